"""The home rank's operators at the edges of their documentation: calls and values that the other
files' cases do not reach."""
import numpy as np
import pytest
import torch

import asynchronous_moe_expert_amd as M

pytestmark = pytest.mark.gpu

F32, BF16, FP8 = torch.float32, torch.bfloat16, torch.float8_e4m3fn


@pytest.mark.parametrize("group", [32, 0])
@pytest.mark.parametrize("size", [1.0, 1e14])
def test_a_group_with_an_infinite_value_stands_for_nan(group, size):
    """gamma[40] infinite while r is ordinary (rows of size 1) and while it is small (1e14): every code of the
    groups that hold the column is NaN, the others' are those of a finite gamma."""
    T, H = 3, 256
    rng = np.random.default_rng(3)
    x = (size * torch.from_numpy(rng.uniform(0.5, 2, (T, H)).astype(np.float32))).cuda()
    gamma = torch.ones(H, device="cuda")
    outs = []
    for g in (1.0, float("inf")):
        gamma[40] = g
        out = torch.zeros(T, H, dtype=torch.uint8, device="cuda")
        scale = torch.zeros(T, H // group if group else 1, device="cuda")
        M.moe_residual_norm(x, None, gamma, 1e-5, out, out_scale=scale, group=group)
        outs.append(out.view(FP8).float().cpu() * scale.repeat_interleave(H // scale.shape[1], 1).cpu())
    finite, got = outs
    hit = torch.zeros(H, dtype=torch.bool)
    hit[32:64] = True
    if group == 0:
        hit[:] = True
    assert got[:, hit].isnan().all()
    assert finite.isfinite().all() and torch.equal(got[:, ~hit], finite[:, ~hit])
