"""Every kernel that the cache rule chooses (home.hpp: calls that move 96 MiB of rows or more read them
non-temporally, from 220 MiB on they write them so too), for each type, number of positions and chunks:
a call of that size gives the bits of small calls on its slices, which other tests hold to the oracle."""
import math

import pytest
import torch

import asynchronous_moe_expert_amd as M
from gpu_helpers import sync_err

pytestmark = pytest.mark.gpu

F32, BF16, FP8, I32 = torch.float32, torch.bfloat16, torch.float8_e4m3fn, torch.int32
MIB = 1 << 20
SIZES = {"once": 130 * MIB, "through": 240 * MIB}
PARTS = 10  # slices of at most 24 MiB


def tokens(kind, bytes_per_token):
    T = -(-SIZES[kind] // bytes_per_token)
    moved = T * bytes_per_token
    assert (96 * MIB <= moved < 220 * MIB) if kind == "once" else moved >= 220 * MIB
    return T


def slices(T):
    step = -(-T // PARTS)
    return [(a, min(T, a + step)) for a in range(0, T, step)]


class Make:
    def __init__(self, seed):
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(seed)

    def rows(self, *shape, dtype=F32):
        return torch.randn(*shape, generator=self.g, device="cuda").to(dtype)

    def positions(self, T, K):
        pos = torch.randperm(T * K, generator=self.g, device="cuda").to(I32)
        pos[torch.rand(T * K, generator=self.g, device="cuda") < 0.1] = -1
        return pos.view(T, K)


def zeros(*shape, dtype=F32):
    return torch.zeros(*shape, dtype=torch.uint8 if dtype == FP8 else dtype, device="cuda").view(dtype)


def same(a, b):
    bits = lambda t: t.view(torch.uint8) if t.dtype == FP8 else t  # noqa: E731
    return torch.equal(bits(a), bits(b))


@pytest.mark.parametrize("kind", SIZES)
@pytest.mark.parametrize("rt,ot", [(BF16, BF16), (F32, F32), (BF16, F32), (F32, BF16)])
@pytest.mark.parametrize("K,H", [(2, 2880), (4, 2880), (6, 2880), (8, 7168)])
def test_merge(kind, rt, ot, K, H):
    T = tokens(kind, H * (K * rt.itemsize + ot.itemsize))
    m = Make(T)
    rows, pos, w = m.rows(T * K, H, dtype=rt), m.positions(T, K), m.rows(T, K)
    out, err = zeros(T, H, dtype=ot), zeros(1, dtype=I32)
    M.moe_merge_rows(rows, pos, w, out, err)
    for a, b in slices(T):
        part = zeros(b - a, H, dtype=ot)
        M.moe_merge_rows(rows, pos[a:b], w[a:b], part, err)
        assert same(part, out[a:b]), (a, b)
    assert sync_err(err) == 0 and out.abs().max() > 0


@pytest.mark.parametrize("kind", SIZES)
@pytest.mark.parametrize("dt,rt", [(BF16, BF16), (F32, F32), (BF16, F32), (F32, BF16)])
@pytest.mark.parametrize("K,H", [(2, 2880), (4, 2880), (6, 2880), (8, 7168)])
def test_merge_gradient(kind, dt, rt, K, H):
    T = tokens(kind, H * (2 * K * rt.itemsize + dt.itemsize))
    m = Make(T + 1)
    dout, rows, pos, w = m.rows(T, H, dtype=dt), m.rows(T * K, H, dtype=rt), m.positions(T, K), m.rows(T, K)
    drows, dw, err = zeros(T * K, H, dtype=rt), zeros(T, K), zeros(1, dtype=I32)
    M.moe_merge_rows_backward(dout, rows, pos, w, drows, dw, err)
    small = zeros(T * K, H, dtype=rt)
    for a, b in slices(T):
        part = zeros(b - a, K)
        M.moe_merge_rows_backward(dout[a:b], rows, pos[a:b], w[a:b], small, part, err)
        assert same(part, dw[a:b]), (a, b)
    assert same(small, drows) and sync_err(err) == 0 and dw.abs().max() > 0


@pytest.mark.parametrize("dtype,group", [(F32, 0), (BF16, 0), (FP8, 0), (FP8, 32), (FP8, 128)])
@pytest.mark.parametrize("K,H", [(4, 2880), (1, 7168), (8, 4104)])
def test_sorted_rows(dtype, group, K, H):
    out = F32 if dtype == F32 else BF16
    T, E = tokens("through", H * (K * out.itemsize + dtype.itemsize)), 60
    m = Make(T + 2)
    x = m.rows(T, H, dtype=dtype)
    groups = -(-H // group) if group else 1
    scale = 0.01 + torch.rand(T, groups, generator=m.g, device="cuda") if dtype == FP8 else None
    expert = torch.randint(-1, E, (T, K), generator=m.g, device="cuda", dtype=I32)
    n, err, xs = T * K, zeros(1, dtype=I32), torch.full((T * K, H), 5, dtype=out, device="cuda")
    perm, pos, slot, counts, offsets = (zeros(c, dtype=I32) for c in (n, n, n, E, E + 1))
    M.moe_sort_rows(expert, E, x, xs, perm, pos, counts, offsets, err, zeros(1 << 18, dtype=torch.uint8), row_slot=slot,
                    x_scale=scale, group=group)
    total = int(offsets[E])
    assert total == int((expert >= 0).sum()) and sync_err(err) == 0 and (xs[total:] == 5).all()
    at = torch.arange(H, device="cuda") // (group or H)
    for a, b in slices(total):
        t = slot[a:b].long()
        ref = x.view(torch.uint8)[t].view(FP8).float() * scale[t][:, at] if dtype == FP8 else x[t]
        assert torch.equal(xs[a:b], ref.to(out)), (a, b)  # a product of fp32, rounded once


@pytest.mark.parametrize("kind", SIZES)
@pytest.mark.parametrize("xt,rt", [(BF16, BF16), (BF16, F32), (F32, F32)])
@pytest.mark.parametrize("ot,group", [(F32, 0), (BF16, 0), (FP8, 0), (FP8, 128)])
@pytest.mark.parametrize("H", [4096, 7168, 16384])  # one, two and four chunks per thread
def test_norm(kind, xt, rt, ot, group, H):
    T = tokens(kind, H * (xt.itemsize + 2 * rt.itemsize + ot.itemsize))
    m = Make(T + 3)
    x, res, gamma = m.rows(T, H, dtype=xt), m.rows(T, H, dtype=rt), m.rows(H, dtype=BF16)
    groups = H // group if group else 1

    def call(a, b):
        got = [zeros(b - a, H, dtype=ot), zeros(b - a, H, dtype=rt), zeros(b - a)] + ([zeros(b - a, groups)] if ot == FP8 else [])
        M.moe_residual_norm(x[a:b], res[a:b], gamma, 1e-5, got[0], residual_out=got[1], rstd=got[2],
                            out_scale=got[3] if ot == FP8 else None, group=group)
        return got

    whole = call(0, T)
    for a, b in slices(T):
        for one, part in zip(whole, call(a, b)):
            assert same(one[a:b], part), (a, b)
    assert (whole[2] > 0).all()


@pytest.mark.parametrize("kind", SIZES)
@pytest.mark.parametrize("dt,ht", [(BF16, BF16), (BF16, F32), (F32, F32)])
@pytest.mark.parametrize("H", [512, 4096, 7168, 16384])  # several rows to a workgroup; one, two and four chunks
def test_norm_gradient(kind, dt, ht, H):
    T = tokens(kind, H * (2 * dt.itemsize + 3 * ht.itemsize))
    m = Make(T + 4)
    dout, h, dres, gamma = m.rows(T, H, dtype=dt), m.rows(T, H, dtype=ht), m.rows(T, H, dtype=ht), m.rows(H)
    rstd, ws = 0.5 + torch.rand(T, generator=m.g, device="cuda"), zeros(2048 * H, dtype=torch.uint8)

    def call(a, b):
        got = [zeros(b - a, H, dtype=dt), zeros(b - a, H, dtype=ht), zeros(H)]
        M.moe_residual_norm_backward(dout[a:b], h[a:b], gamma, rstd[a:b], got[0], got[2], ws, dres=dres[a:b], dresidual=got[1])
        return got

    whole = call(0, T)
    ref, size = (torch.zeros(H, dtype=torch.float64, device="cuda") for _ in range(2))
    for a, b in slices(T):
        part = call(a, b)
        assert same(whole[0][a:b], part[0]) and same(whole[1][a:b], part[1]), (a, b)
        t = dout[a:b].double() * h[a:b].double() * rstd[a:b].double()[:, None]
        ref += t.sum(0)
        size += t.abs().sum(0)
    # chains of at most ceil(T / 512) tokens, eight rows' shares, 512 partial sums in runs of 8 and a tree; 3
    # roundings a term
    assert ((whole[2].double() - ref).abs() <= (math.ceil(T / 512) + 30) * 2.0 ** -24 * size).all()


def test_norm_gradient_of_the_largest_number_of_tokens():
    """dx of 2^24 rows of 8 columns, eight of them at a time in a workgroup, 768 MiB: the bits of small calls."""
    T, H = 1 << 24, 8
    m = Make(5)
    dout, h, gamma = m.rows(T, H, dtype=BF16), m.rows(T, H, dtype=BF16), m.rows(H)
    rstd, ws = 0.5 + torch.rand(T, generator=m.g, device="cuda"), zeros(2048 * H, dtype=torch.uint8)
    dx = zeros(T, H, dtype=BF16)
    M.moe_residual_norm_backward(dout, h, gamma, rstd, dx, zeros(H), ws)
    for a in (0, 4091, T // 2 - 5, T - 3000):
        for rows in (500, 3000):  # one row at a time in a workgroup, and several
            part = zeros(rows, H, dtype=BF16)
            M.moe_residual_norm_backward(dout[a:a + rows], h[a:a + rows], gamma, rstd[a:a + rows], part, zeros(H), ws)
            assert same(part, dx[a:a + rows]), (a, rows)
    assert not (dx == 0).all(1).any()
