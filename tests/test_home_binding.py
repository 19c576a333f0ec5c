"""Shapes that hold the right number of elements in another order are refused by the binding (the
checks come before the refusal of tensors that are not on a GPU, which is how a good call ends here)."""
import os

import pytest
import torch

import asynchronous_moe_expert_amd as M

F32, I32, BF16, U8 = torch.float32, torch.int32, torch.bfloat16, torch.uint8


@pytest.fixture(scope="module", autouse=True)
def lib():
    from asynchronous_moe_expert_amd import build

    if not (os.path.exists(M.LIB_PATH) and os.path.exists(build.MARSHAL)):
        build.build()
    return M.load()


def z(*shape, dtype=F32):
    return torch.zeros(*shape, dtype=dtype)


T, K, H, E = 6, 4, 64, 8
ERR = z(1, dtype=I32)


def merge(pos, w):
    M.moe_merge_rows(z(24, H), pos, w, z(T, H), ERR)


def merge_backward(pos, w, dw):
    M.moe_merge_rows_backward(z(T, H), z(24, H), pos, w, z(24, H), dw, ERR)


def sort(pos=z(T * K, dtype=I32), scale=z(T, 2)):
    M.moe_sort_rows(z(T, K, dtype=I32), E, z(T, H, dtype=U8), z(T * K, H, dtype=BF16), None, pos, z(E, dtype=I32),
                    z(E + 1, dtype=I32), ERR, z(1 << 18, dtype=U8), x_scale=scale, group=32)


def norm(scale, group=32):
    M.moe_residual_norm(z(T, H), None, z(H), 1e-5, z(T, H, dtype=U8), out_scale=scale, group=group)


POS, W, PT, WT = z(T, K, dtype=I32), z(T, K), z(K, T, dtype=I32), z(K, T)
REFUSED = [
    (lambda: merge(PT, None), "pos"), (lambda: merge(z(2, T * K // 2, dtype=I32), None), "pos"),
    (lambda: merge(POS, WT), "w"), (lambda: merge(POS.view(-1), WT), "w"), (lambda: merge(POS.view(2, 3, K), None), "pos"),
    (lambda: merge(z(T, 2, 2, dtype=I32), None), "pos"), (lambda: merge(POS, W.view(T, 2, 2)), "w"),
    (lambda: merge_backward(PT, W, W), "pos"), (lambda: merge_backward(POS, WT, W), "w"),
    (lambda: merge_backward(POS, W, WT), "dw"), (lambda: merge_backward(POS, None, WT), "dw"),
    (lambda: sort(pos=PT), "pos"), (lambda: sort(scale=z(2, T)), "x_scale"), (lambda: sort(scale=z(T, 4)), "x_scale"),
    (lambda: norm(z(2, T)), "out_scale"), (lambda: norm(z(T, 4)), "out_scale"), (lambda: norm(z(T, 2), group=0), "out_scale"),
    (lambda: norm(z(T, 1, 2)), "out_scale"),
]
TAKEN = [
    lambda: merge(POS, W), lambda: merge(POS.view(-1), W), lambda: merge(POS, W.view(-1)), lambda: merge(POS.view(-1), None),
    lambda: merge_backward(POS, W, z(T + 2, K)), lambda: merge_backward(POS.view(-1), W, z(T * K + 5)),
    lambda: sort(pos=POS), lambda: sort(pos=z(T + 1, K, dtype=I32)), lambda: sort(scale=z(T * 2)), lambda: sort(scale=z(T + 3, 2)),
    lambda: M.moe_merge_rows(z(24, H), z(0, dtype=I32), z(0, K), z(0, H), ERR),
    lambda: norm(z(T, 2)), lambda: norm(z(T + 1, 2)), lambda: norm(z(2 * T)), lambda: norm(z(T, 1), group=0), lambda: norm(z(T), group=0),
]


@pytest.mark.parametrize("case", range(len(REFUSED)))
def test_refused(case):
    call, what = REFUSED[case]
    with pytest.raises(M.MoeError, match=rf"^{what}:"):
        call()


@pytest.mark.parametrize("case", range(len(TAKEN)))
def test_taken(case):
    with pytest.raises(M.MoeError, match="on a GPU"):
        TAKEN[case]()
