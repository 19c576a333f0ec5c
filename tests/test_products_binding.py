"""The binding's checks of the experts' products' tensors, beyond those of their sizes."""
import ctypes as C
import os

import pytest
import torch

import asynchronous_moe_expert_amd as M


@pytest.fixture(scope="module", autouse=True)
def built():
    from asynchronous_moe_expert_amd import build

    if not (os.path.exists(M.LIB_PATH) and os.path.exists(build.MARSHAL)):
        build.build()


def test_weights_scales_of_another_shape():
    """Scales lie by expert, block of outputs and block of columns: as many of another shape are other weights'."""
    E, N, D = 3, 256, 384
    x, w = torch.zeros(4, D, dtype=torch.uint8), torch.zeros(E, N, D, dtype=torch.uint8)
    offsets, out, xs = torch.zeros(E + 1, dtype=torch.int32), torch.zeros(4, N), torch.zeros(4, 3)
    good = torch.zeros(E, 2, 3)

    def call(scale):
        M.moe_expert_matmul(x, w, offsets, out, x_scale=xs, w_scale=scale)

    for bad in (good.view(E, 6), good.view(6, 3), good.view(E, 3, 2), good.view(1, E, 2, 3), torch.zeros(E + 1, 2, 3)):
        with pytest.raises(M.MoeError, match="w_scale"):
            call(bad)
    for fine in (good, good.view(-1)):
        with pytest.raises(M.MoeError, match="on a GPU"):
            call(fine)


def test_pitches_whose_bytes_pass_64_bits():
    """They are over the limit of 16 MiB like any other that is."""
    from asynchronous_moe_expert_amd import _native as N
    from test_products_cpu import F32, MATMUL, MATMUL_B, SIZE

    lib = M.load()
    for pitch in (1 << 62, 3 << 61, (1 << 63) - 8):
        for name, struct, good, fields in (
                ("moe_expert_matmul", N.ExpertMatmulArgs, MATMUL, ("x_pitch", "w_pitch")),
                ("moe_expert_matmul_backward", N.ExpertMatmulBackwardArgs, MATMUL_B, ("x_pitch", "dout_pitch", "dw_pitch"))):
            for field in fields:
                a = dict(good, dtype=F32, **{field: pitch})
                a.update(dict(out_dtype=F32) if "out_dtype" in a else {})
                a.update({s: (1 << 36) - 8 for s in ("w_stride", "dw_stride") if s in a})
                assert getattr(lib, name)(C.byref(struct(**a)), None) == SIZE, (name, field, pitch)
