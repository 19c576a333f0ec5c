"""ctypes binding of libmoestep.so.  Argument marshalling only: every step of the path runs
in the library's HIP kernels.  Tensors are torch device tensors (plumbing for device
memory and streams); each function takes the same name as the C call it wraps."""
from __future__ import annotations

import ctypes as C
import os

import torch

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libmoestep.so")

MOE_F32, MOE_BF16, MOE_FP8_E4M3 = 0, 1, 2
MOE_SOFTMAX, MOE_SIGMOID = 0, 1
MOE_BIAS_ON_SCORE = 16  # or-ed to either: the bias is added to the gate's score, not to the logit

ERR_SLOT_RANGE = 1 << 0
ERR_EXPERT_NONLOCAL = 1 << 1
ERR_TOKEN_RANGE = 1 << 2
ERR_KSLOT_RANGE = 1 << 3
ERR_ROW_RANGE = 1 << 4
ERR_STALE_GEN = 1 << 5
ERR_DUPLICATE = 1 << 6

_p = C.c_void_p
_i32 = C.c_int32
_i64 = C.c_int64


class AssembleArgs(C.Structure):
    _fields_ = [("n", _i32), ("slot", _p), ("expert", _p), ("expert_base", _i32), ("E_loc", _i32),
                ("pool", _p), ("P", _i64), ("pool_pitch", _i64), ("H", _i32), ("act_dtype", _i32),
                ("perm", _p), ("pos", _p), ("counts", _p), ("offsets", _p), ("xb", _p), ("err", _p),
                ("row_slot", _p)]


class PackArgs(C.Structure):
    _fields_ = [("E_loc", _i32), ("H", _i32), ("I", _i32), ("w_dtype", _i32), ("wg", _p), ("wu", _p), ("wd", _p),
                ("w_gu", _p), ("w_d", _p)]


class FfnArgs(C.Structure):
    _fields_ = [("n", _i32), ("E_loc", _i32), ("H", _i32), ("I", _i32), ("act_dtype", _i32), ("w_dtype", _i32),
                ("xb", _p), ("offsets", _p), ("w_gu", _p), ("w_d", _p), ("s_gate", _p), ("s_up", _p),
                ("s_down", _p), ("y", _p), ("workspace", _p), ("workspace_bytes", C.c_size_t), ("ev_mid", _p),
                ("perm", _p), ("slot", _p), ("pool", _p), ("P", _i64), ("pool_pitch", _i64), ("row_slot", _p),
                ("plan", _p), ("ev_gu_start", _p), ("ev_gu_stop", _p), ("index", _p)]


class StateC(C.Structure):
    _fields_ = [("acc", _p), ("mask", _p), ("head", _p), ("tgen", _p), ("rflag", _p), ("T_cap", _i32), ("H", _i32)]


class CombineArgs(C.Structure):
    _fields_ = [("m", _i32), ("K", _i32), ("rows", _p), ("row_dtype", _i32), ("row_pitch", _i64),
                ("n_rows", _i64), ("row_idx", _p), ("tok", _p), ("kslot", _p), ("w", _p), ("gen", _p),
                ("state", StateC), ("out", _p), ("out_dtype", _i32), ("out_pitch", _i64), ("rel_list", _p),
                ("rel_count", _p), ("err", _p), ("workspace", _p), ("workspace_bytes", C.c_size_t)]


class RouteArgs(C.Structure):
    _fields_ = [("T", _i32), ("E", _i32), ("K", _i32), ("logits", _p), ("dtype", _i32), ("pitch", _i64), ("bias", _p),
                ("score", _i32), ("renorm", _i32), ("scale", C.c_float), ("expert", _p), ("w", _p)]


class RouteBackwardArgs(C.Structure):
    _fields_ = [("T", _i32), ("E", _i32), ("K", _i32), ("logits", _p), ("dtype", _i32), ("pitch", _i64),
                ("expert", _p), ("dw", _p), ("score", _i32), ("renorm", _i32), ("scale", C.c_float), ("dlogits", _p),
                ("dlogits_pitch", _i64), ("err", _p)]


class SortRowsArgs(C.Structure):
    _fields_ = [("T", _i32), ("K", _i32), ("H", _i32), ("expert_base", _i32), ("E_loc", _i32), ("expert", _p),
                ("x", _p), ("x_dtype", _i32), ("x_pitch", _i64), ("x_scale", _p), ("group", _i32), ("xs", _p),
                ("xs_pitch", _i64), ("perm", _p), ("pos", _p), ("counts", _p), ("offsets", _p), ("row_slot", _p),
                ("err", _p), ("workspace", _p), ("workspace_bytes", C.c_size_t)]


class MergeRowsArgs(C.Structure):
    _fields_ = [("T", _i32), ("K", _i32), ("H", _i32), ("rows", _p), ("row_dtype", _i32), ("row_pitch", _i64),
                ("n_rows", _i64), ("pos", _p), ("w", _p), ("out", _p), ("out_dtype", _i32), ("out_pitch", _i64),
                ("err", _p)]


class MergeRowsBackwardArgs(C.Structure):
    _fields_ = [("T", _i32), ("K", _i32), ("H", _i32), ("dout", _p), ("dout_dtype", _i32), ("dout_pitch", _i64),
                ("rows", _p), ("row_dtype", _i32), ("row_pitch", _i64), ("n_rows", _i64), ("pos", _p), ("w", _p),
                ("drows", _p), ("drows_pitch", _i64), ("dw", _p), ("err", _p)]


class ResidualNormArgs(C.Structure):
    _fields_ = [("T", _i32), ("H", _i32), ("x", _p), ("x_dtype", _i32), ("x_pitch", _i64), ("residual", _p),
                ("res_dtype", _i32), ("res_pitch", _i64), ("gamma", _p), ("gamma_dtype", _i32), ("eps", C.c_float),
                ("out", _p), ("out_dtype", _i32), ("out_pitch", _i64), ("out_scale", _p), ("group", _i32),
                ("residual_out", _p), ("res_out_pitch", _i64), ("rstd", _p), ("row_list", _p), ("row_count", _p),
                ("err", _p)]


class ResidualNormBackwardArgs(C.Structure):
    _fields_ = [("T", _i32), ("H", _i32), ("dout", _p), ("dtype", _i32), ("dout_pitch", _i64), ("h", _p),
                ("h_dtype", _i32), ("h_pitch", _i64), ("gamma", _p), ("gamma_dtype", _i32), ("rstd", _p),
                ("dres", _p), ("dres_pitch", _i64), ("dx", _p), ("dx_pitch", _i64), ("dresidual", _p),
                ("dresidual_pitch", _i64), ("dgamma", _p), ("workspace", _p), ("workspace_bytes", C.c_size_t)]


class ExpertMatmulArgs(C.Structure):
    _fields_ = [("n", _i32), ("E_loc", _i32), ("N", _i32), ("D", _i32), ("offsets", _p), ("x", _p), ("dtype", _i32),
                ("x_rows", _i64), ("x_pitch", _i64), ("row_slot", _p), ("x_scale", _p), ("w", _p),
                ("w_transposed", _i32), ("w_pitch", _i64), ("w_stride", _i64), ("w_scale", _p), ("out", _p),
                ("out_dtype", _i32), ("out_pitch", _i64), ("err", _p)]


class ExpertMatmulBackwardArgs(C.Structure):
    _fields_ = [("n", _i32), ("E_loc", _i32), ("N", _i32), ("D", _i32), ("offsets", _p), ("dout", _p),
                ("dout_pitch", _i64), ("x", _p), ("x_pitch", _i64), ("dtype", _i32), ("accumulate", _i32), ("dw", _p),
                ("dw_dtype", _i32), ("dw_pitch", _i64), ("dw_stride", _i64)]


class SwigluArgs(C.Structure):
    _fields_ = [("n", _i32), ("I", _i32), ("gu", _p), ("dtype", _i32), ("gu_pitch", _i64), ("count", _p), ("h", _p),
                ("h_dtype", _i32), ("h_pitch", _i64), ("h_scale", _p), ("group", _i32)]


class SwigluBackwardArgs(C.Structure):
    _fields_ = [("n", _i32), ("I", _i32), ("gu", _p), ("dtype", _i32), ("gu_pitch", _i64), ("dh", _p),
                ("dh_pitch", _i64), ("count", _p), ("dgu", _p), ("dgu_pitch", _i64), ("h", _p), ("h_pitch", _i64)]


class QuantizeWeightsArgs(C.Structure):
    _fields_ = [("E_loc", _i32), ("N", _i32), ("D", _i32), ("w", _p), ("dtype", _i32), ("w_pitch", _i64),
                ("w_stride", _i64), ("transposed", _i32), ("codes", _p), ("codes_pitch", _i64),
                ("codes_stride", _i64), ("scale", _p)]


_STRUCTS = [AssembleArgs, PackArgs, FfnArgs, StateC, CombineArgs, RouteArgs, RouteBackwardArgs, SortRowsArgs,
            MergeRowsArgs, MergeRowsBackwardArgs, ResidualNormArgs, ResidualNormBackwardArgs, ExpertMatmulArgs,
            ExpertMatmulBackwardArgs, SwigluArgs, SwigluBackwardArgs, QuantizeWeightsArgs]
EXPORTS = ["moe_assemble", "moe_pack_ffn_weights", "moe_ffn_workspace_size", "moe_expert_ffn_grouped",
           "moe_state_reset", "moe_combine_release", "moe_combine_plan", "moe_combine_apply",
           "moe_combine_workspace_size", "moe_strerror", "moe_version", "moe_struct_size",
           "moe_combine_release_noalloc", "moe_combine_noalloc_max_arrivals", "moe_route", "moe_route_backward",
           "moe_sort_rows", "moe_sort_rows_workspace_size", "moe_merge_rows", "moe_merge_rows_backward",
           "moe_residual_norm", "moe_residual_norm_backward", "moe_residual_norm_backward_workspace_size",
           "moe_expert_matmul", "moe_expert_matmul_backward", "moe_swiglu", "moe_swiglu_backward",
           "moe_quantize_weights"]


class MoeError(RuntimeError):
    pass


_lib = None


def load(path: str = LIB_PATH) -> C.CDLL:
    """Loads the HIP library; raises if it has not been built (there is no fallback)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise MoeError(f"libmoestep.so not found at {path}; build it with "
                       "`python -m asynchronous_moe_expert_amd.build` (no CPU fallback exists)")
    lib = C.CDLL(path)
    for name, args in [("moe_assemble", [C.POINTER(AssembleArgs), _p]),
                       ("moe_pack_ffn_weights", [C.POINTER(PackArgs), _p]),
                       ("moe_expert_ffn_grouped", [C.POINTER(FfnArgs), _p]),
                       ("moe_state_reset", [C.POINTER(StateC), C.c_uint32, _p]),
                       ("moe_combine_release", [C.POINTER(CombineArgs), _p]),
                       ("moe_combine_plan", [C.POINTER(CombineArgs), _p]),
                       ("moe_combine_apply", [C.POINTER(CombineArgs), _p]),
                       ("moe_combine_release_noalloc", [C.POINTER(CombineArgs), _p]),
                       ("moe_route", [_p, _p]),
                       ("moe_route_backward", [_p, _p]),
                       ("moe_sort_rows", [_p, _p]),
                       ("moe_merge_rows", [_p, _p]),
                       ("moe_merge_rows_backward", [_p, _p]),
                       ("moe_residual_norm", [_p, _p]),
                       ("moe_residual_norm_backward", [_p, _p]),
                       ("moe_expert_matmul", [_p, _p]),
                       ("moe_expert_matmul_backward", [_p, _p]),
                       ("moe_swiglu", [_p, _p]),
                       ("moe_swiglu_backward", [_p, _p]),
                       ("moe_quantize_weights", [_p, _p]),
                       ("moe_version", []), ("moe_strerror", [C.c_int])]:
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = C.c_int
    lib.moe_strerror.restype = C.c_char_p
    lib.moe_ffn_workspace_size.argtypes = [_i32, _i32, _i32, _i32, _i32]
    lib.moe_ffn_workspace_size.restype = C.c_size_t
    lib.moe_combine_workspace_size.argtypes = [_i32]
    lib.moe_combine_workspace_size.restype = C.c_size_t
    lib.moe_combine_noalloc_max_arrivals.argtypes = []
    lib.moe_combine_noalloc_max_arrivals.restype = C.c_size_t
    for name in ("moe_sort_rows_workspace_size", "moe_residual_norm_backward_workspace_size"):
        getattr(lib, name).argtypes = [_i32]
        getattr(lib, name).restype = C.c_size_t
    lib.moe_struct_size.argtypes = [C.c_int]
    lib.moe_struct_size.restype = C.c_size_t
    for k, s in enumerate(_STRUCTS):
        if lib.moe_struct_size(k) != C.sizeof(s):
            raise MoeError(f"struct layout mismatch for {s.__name__}: library {lib.moe_struct_size(k)} "
                           f"vs binding {C.sizeof(s)}")
    _lib = lib
    return lib


def _ptr(t) -> int | None:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _check(rc: int, what: str) -> None:
    if rc != 0:
        raise MoeError(f"{what}: {load().moe_strerror(rc).decode()} ({rc})")


def dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return MOE_F32
    if t.dtype == torch.bfloat16:
        return MOE_BF16
    if t.dtype in (torch.uint8, torch.float8_e4m3fn):
        return MOE_FP8_E4M3
    raise MoeError(f"unsupported dtype {t.dtype}")


def moe_version() -> int:
    return load().moe_version()


def moe_strerror(rc: int) -> str:
    return load().moe_strerror(rc).decode()


def moe_ffn_workspace_size(n_max: int, E_loc: int, H: int, I: int, act_dtype: int) -> int:
    return load().moe_ffn_workspace_size(n_max, E_loc, H, I, act_dtype)


def assemble_args(slot, expert, expert_base: int, E_loc: int, pool, perm, pos, counts, offsets, xb, err,
                  n: int | None = None, row_slot=None, H: int | None = None) -> AssembleArgs:
    """The moe_assemble argument struct (for moe_assemble, or as moe_ffn_args.index)."""
    if H is None:
        H = pool.shape[1] if xb is None else xb.shape[1]
    return AssembleArgs(int(slot.numel() if n is None else n), _ptr(slot), _ptr(expert), expert_base, E_loc,
                        _ptr(pool), pool.shape[0], pool.stride(0), H, dtype_code(pool), _ptr(perm),
                        _ptr(pos), _ptr(counts), _ptr(offsets), _ptr(xb), _ptr(err), _ptr(row_slot))


def moe_assemble(slot, expert, expert_base: int, E_loc: int, pool, perm, pos, counts, offsets, xb, err,
                 n: int | None = None, stream=None, row_slot=None) -> None:
    """pool: [P][pitch] (f32 or bf16); xb: [>= n][H] of the same dtype (or None);
    row_slot: optional [>= n] int32 output, the pool slot of each batch row."""
    a = assemble_args(slot, expert, expert_base, E_loc, pool, perm, pos, counts, offsets, xb, err, n=n,
                      row_slot=row_slot)
    _check(load().moe_assemble(C.byref(a), _stream(stream)), "moe_assemble")


def moe_pack_ffn_weights(wg, wu, wd, w_gu, w_d, w_dtype: int, stream=None) -> None:
    E, I, H = wg.shape
    a = PackArgs(E, H, I, w_dtype, _ptr(wg), _ptr(wu), _ptr(wd), _ptr(w_gu), _ptr(w_d))
    _check(load().moe_pack_ffn_weights(C.byref(a), _stream(stream)), "moe_pack_ffn_weights")


def moe_expert_ffn_grouped(n: int, E_loc: int, H: int, I: int, act_dtype: int, w_dtype: int, xb, offsets, w_gu,
                           w_d, y, workspace, s_gate=None, s_up=None, s_down=None, ev_mid: int | None = None,
                           stream=None, gather=None, plan: "CombineArgs | None" = None,
                           ev_gu: tuple[int, int] | None = None, index: "AssembleArgs | None" = None) -> None:
    """gather=(perm, slot, pool) or (perm, slot, pool, row_slot): read batch rows from the pool
    (gather-on-load; with row_slot, pool row row_slot[r] and perm/slot unused); xb may be None.
    plan: the arguments (combine_args) of a moe_combine_plan call that this call enqueues as
    well, inside the gate/up launch where it fits.  ev_gu: (start, stop) hipEvent_t handles
    that the weight-streaming gate/up kernel records around itself.  index: the arguments
    (assemble_args, xb None) of a moe_assemble call that this call does as well, inside the
    gate/up launch where it fits; offsets and gather are then taken from it."""
    perm = slot = pool = row_slot = None
    P = pitch = 0
    if gather is not None:
        perm, slot, pool = gather[:3]
        row_slot = gather[3] if len(gather) > 3 else None
        P, pitch = pool.shape[0], pool.stride(0)
    a = FfnArgs(n, E_loc, H, I, act_dtype, w_dtype, _ptr(xb), _ptr(offsets), _ptr(w_gu), _ptr(w_d),
                _ptr(s_gate), _ptr(s_up), _ptr(s_down), _ptr(y), _ptr(workspace),
                workspace.numel() * workspace.element_size(), ev_mid, _ptr(perm), _ptr(slot), _ptr(pool), P, pitch,
                _ptr(row_slot), None if plan is None else C.addressof(plan), *(ev_gu or (None, None)),
                None if index is None else C.addressof(index))
    _check(load().moe_expert_ffn_grouped(C.byref(a), _stream(stream)), "moe_expert_ffn_grouped")


class CombineState:
    """Device tensors of the per-token combine state (allocated here with torch)."""

    def __init__(self, T_cap: int, H: int, device="cuda"):
        self.T_cap, self.H = T_cap, H
        self.acc = torch.empty((T_cap, H), dtype=torch.float32, device=device)
        self.mask = torch.empty(T_cap, dtype=torch.int32, device=device)
        self.head = torch.empty(T_cap, dtype=torch.int32, device=device)
        self.tgen = torch.empty(T_cap, dtype=torch.int32, device=device)
        self.rflag = torch.empty((T_cap + 15) // 16 * 16, dtype=torch.uint8, device=device)

    def c(self) -> StateC:
        return StateC(_ptr(self.acc), _ptr(self.mask), _ptr(self.head), _ptr(self.tgen), _ptr(self.rflag),
                      self.T_cap, self.H)


def moe_state_reset(state: CombineState, gen0: int = 0, stream=None) -> None:
    s = state.c()
    _check(load().moe_state_reset(C.byref(s), gen0, _stream(stream)), "moe_state_reset")


def moe_combine_workspace_size(m_max: int) -> int:
    return load().moe_combine_workspace_size(m_max)


def moe_combine_noalloc_max_arrivals() -> int:
    return load().moe_combine_noalloc_max_arrivals()


def _combine_args(rows, row_idx, tok, kslot, w, gen, K, state, out, rel_list, rel_count, err, workspace, m, n_rows):
    return CombineArgs(int(tok.numel() if m is None else m), K, _ptr(rows), dtype_code(rows), rows.stride(0),
                       rows.shape[0] if n_rows is None else n_rows, _ptr(row_idx), _ptr(tok), _ptr(kslot), _ptr(w),
                       _ptr(gen), state.c(), _ptr(out), dtype_code(out), out.stride(0), _ptr(rel_list),
                       _ptr(rel_count), _ptr(err), _ptr(workspace),
                       0 if workspace is None else workspace.numel() * workspace.element_size())


def combine_args(rows, row_idx, tok, kslot, w, gen, K: int, state: CombineState, out, rel_list, rel_count, err,
                 workspace, m: int | None = None, n_rows: int | None = None) -> CombineArgs:
    """The argument struct of a combine call (for moe_expert_ffn_grouped's plan)."""
    return _combine_args(rows, row_idx, tok, kslot, w, gen, K, state, out, rel_list, rel_count, err, workspace, m,
                         n_rows)


def moe_combine_release(rows, row_idx, tok, kslot, w, gen, K: int, state: CombineState, out, rel_list, rel_count,
                        err, workspace, m: int | None = None, n_rows: int | None = None, stream=None,
                        part: str = "release") -> None:
    """rows: [n_rows][pitch] f32/bf16 result rows; out: [T_cap][pitch] f32/bf16.
    part = "plan" / "apply" calls moe_combine_plan / moe_combine_apply instead; part =
    "noalloc" calls moe_combine_release_noalloc (the library's static scratch; workspace
    may be None)."""
    a = _combine_args(rows, row_idx, tok, kslot, w, gen, K, state, out, rel_list, rel_count, err, workspace, m,
                      n_rows)
    combine_call(a, part, stream)


def combine_call(a: CombineArgs, part: str = "release", stream=None) -> None:
    """moe_combine_release / _plan / _apply on an argument struct from combine_args."""
    fn = {"release": "moe_combine_release", "plan": "moe_combine_plan", "apply": "moe_combine_apply",
          "noalloc": "moe_combine_release_noalloc"}[part]
    _check(getattr(load(), fn)(C.byref(a), _stream(stream)), fn)


# ------------------------------------------------- the home rank's side and the experts' products
# The checks of these calls' tensors (device, type, shape, stride) and their argument structs are
# made by the compiled module _marshal, which costs a call 0.3 us where the same in Python took
# 2-5 us beside a launch of 3 us.  Tensors on another device than the current one are worked on
# where they are.  The calls write into the given buffers and record nothing for torch's autograd,
# whether a tensor requires a gradient or not: the gradients are calls of their own, which a training
# step (or a torch.autograd.Function around a pair of them) makes itself.

_marshal = None
_HOME = ("moe_route", "moe_route_backward", "moe_sort_rows", "moe_merge_rows", "moe_merge_rows_backward",
         "moe_residual_norm", "moe_residual_norm_backward", "moe_expert_matmul", "moe_expert_matmul_backward",
         "moe_swiglu", "moe_swiglu_backward", "moe_quantize_weights")
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _home():
    """The module _marshal, with the library's entry points.  It compares the sizes of the argument
    structs that it was built with with the library's."""
    global _marshal
    if _marshal is None:
        lib = load()
        try:
            from . import _marshal as m
        except ImportError as e:
            raise MoeError(f"_marshal.so could not be loaded ({e}); build it with "
                           "`python -m asynchronous_moe_expert_amd.build`") from None
        m.setup(MoeError, *(C.cast(getattr(lib, name), _p).value
                            for name in ("moe_strerror", "moe_version", "moe_struct_size") + _HOME))
        _marshal = m
    return _marshal


def _stream_object(stream, at: int):
    """`stream` (an object or a handle) of device `at` as torch knows it."""
    if hasattr(stream, "cuda_stream"):
        return stream
    handle = _stream(stream)
    return torch.cuda.ExternalStream(handle, device=at) if handle else torch.cuda.default_stream(at)


def keep_for(stream, at: int, tensors) -> None:
    """Records what a call on `stream` works on, unless that is the current stream of the tensors'
    device `at`, so that the allocator keeps it until the call's work is done."""
    if stream is None or _stream(stream) == _raw_stream(at):
        return
    stream = _stream_object(stream, at)
    for t in tensors:
        if t is not None:
            t.record_stream(stream)


def _capturing(stream) -> bool:
    with torch.cuda.stream(stream):
        return torch.cuda.is_current_stream_capturing()


def after_current(stream, at: int) -> None:
    """`stream` goes on after what device `at`'s current stream has been given so far.  For a buffer made within a
    call on `stream`: the allocator hands out memory that work of the current stream, and of no other, may still
    be using."""
    if stream is None or _stream(stream) == _raw_stream(at):
        return
    stream, current = _stream_object(stream, at), torch.cuda.current_stream(at)
    if _capturing(stream) != _capturing(current):
        raise MoeError("a call that makes its buffers was given another stream than the current one while one of the two "
                       "is captured; make the call once before")
    stream.wait_stream(current)


def _elsewhere(call, args, tensors, stream) -> None:
    """A call on a given stream, or with tensors that are not on the current device."""
    at = tensors[0].get_device()
    if at < 0:
        call(*args, 0)  # refuses: not on a GPU
        return
    where = getattr(stream, "device", None)
    if where is not None and where.index != at:
        raise MoeError(f"a stream of {where} for tensors on {tensors[0].device}")
    with torch.cuda.device(at):
        call(*args, _raw_stream(at) if stream is None else _stream(stream))
    keep_for(stream, at, tensors)


def moe_route(logits, expert, w, bias=None, score: int = MOE_SOFTMAX, renorm: bool = True, scale: float = 1.0,
              stream=None) -> None:
    """logits [T][E] (f32 or bf16); out: expert [T][K] int32, w [T][K] f32.  bias [E] f32 moves the
    choice only: it is added to the logits, or with score = MOE_SIGMOID | MOE_BIAS_ON_SCORE (or MOE_SOFTMAX
    | ...) to the gate's scores, as the balancing bias of a router trained without an auxiliary loss is."""
    call, at = (_marshal or _home()).moe_route, logits.get_device()
    if stream is None and at >= 0 and at == _device():
        call(logits, expert, w, bias, score, renorm, scale, _raw_stream(at))
    else:
        _elsewhere(call, (logits, expert, w, bias, score, renorm, scale), (logits, expert, w, bias), stream)


def moe_route_backward(logits, expert, dw, dlogits, err, score: int = MOE_SOFTMAX, renorm: bool = True,
                       scale: float = 1.0, stream=None) -> None:
    """expert [T][K] as moe_route gave it, dw [T][K] f32; out: dlogits [T][E] of the logits' type."""
    call, at = (_marshal or _home()).moe_route_backward, logits.get_device()
    if stream is None and at >= 0 and at == _device():
        call(logits, expert, dw, dlogits, err, score, renorm, scale, _raw_stream(at))
    else:
        t = (logits, expert, dw, dlogits, err)
        _elsewhere(call, t + (score, renorm, scale), t, stream)


def moe_sort_rows_workspace_size(n_max: int) -> int:
    return load().moe_sort_rows_workspace_size(n_max)


def moe_sort_rows(expert, E_loc: int, x, xs, perm, pos, counts, offsets, err, workspace, expert_base: int = 0,
                  row_slot=None, x_scale=None, group: int = 0, stream=None) -> None:
    """expert [T][K] int32; x [T][H] (f32, bf16, or fp8 with x_scale [T][groups] f32), xs [T * K][H]
    of x's type (bf16 for fp8); xs None: the index alone (x may be None then).  perm and row_slot
    are optional, and so is the workspace where moe_sort_rows_workspace_size(T * K) is 0."""
    call, at = (_marshal or _home()).moe_sort_rows, expert.get_device()
    if stream is None and at >= 0 and at == _device():
        call(expert, E_loc, x, xs, perm, pos, counts, offsets, err, workspace, expert_base, row_slot, x_scale, group,
             _raw_stream(at))
    else:
        _elsewhere(call, (expert, E_loc, x, xs, perm, pos, counts, offsets, err, workspace, expert_base, row_slot,
                          x_scale, group),
                   (expert, x, xs, perm, pos, counts, offsets, err, workspace, row_slot, x_scale), stream)


def moe_merge_rows(rows, pos, w, out, err, stream=None) -> None:
    """rows [n_rows][H]; pos (int32) and w (f32, or None: 1) [T][K]; out [T][H].  f32 or bf16 each.
    With the gradient of moe_sort_rows' xs as rows and w None, out is the gradient of its x."""
    call, at = (_marshal or _home()).moe_merge_rows, rows.get_device()
    if stream is None and at >= 0 and at == _device():
        call(rows, pos, w, out, err, _raw_stream(at))
    else:
        t = (rows, pos, w, out, err)
        _elsewhere(call, t, t, stream)


def moe_merge_rows_backward(dout, rows, pos, w, drows, dw, err, stream=None) -> None:
    """dout [T][H]; rows and drows [n_rows][H] of one type; pos, w and dw [T][K].  drows or dw (and
    then rows) may be None."""
    call, at = (_marshal or _home()).moe_merge_rows_backward, dout.get_device()
    if stream is None and at >= 0 and at == _device():
        call(dout, rows, pos, w, drows, dw, err, _raw_stream(at))
    else:
        t = (dout, rows, pos, w, drows, dw, err)
        _elsewhere(call, t, t, stream)


def moe_residual_norm(x, residual, gamma, eps: float, out, residual_out=None, rstd=None, out_scale=None,
                      group: int = 0, row_list=None, row_count=None, err=None, stream=None) -> None:
    """x, residual (optional) [T][H]; gamma [H]; out [T][H] f32, bf16 or fp8 (then out_scale [T][groups]
    f32).  Optional outputs: residual_out [T][H], rstd [T].  row_list [T], row_count [1] (int32): only
    these rows, with err."""
    call, at = (_marshal or _home()).moe_residual_norm, x.get_device()
    if stream is None and at >= 0 and at == _device():
        call(x, residual, gamma, eps, out, residual_out, rstd, out_scale, group, row_list, row_count, err,
             _raw_stream(at))
    else:
        _elsewhere(call, (x, residual, gamma, eps, out, residual_out, rstd, out_scale, group, row_list, row_count, err),
                   (x, residual, gamma, out, residual_out, rstd, out_scale, row_list, row_count, err), stream)


def moe_residual_norm_backward_workspace_size(H: int) -> int:
    return load().moe_residual_norm_backward_workspace_size(H)


def moe_residual_norm_backward(dout, h, gamma, rstd, dx, dgamma, workspace, dres=None, dresidual=None,
                               stream=None) -> None:
    """dout [T][H], h [T][H] (the forward's residual_out, or x), rstd [T]; out: dx [T][H] of dout's type,
    dresidual [T][H] of h's, dgamma [H] f32 (with the workspace); each may be None.  dres [T][H] of h's
    type is added to dx and dresidual."""
    call, at = (_marshal or _home()).moe_residual_norm_backward, dout.get_device()
    if stream is None and at >= 0 and at == _device():
        call(dout, h, gamma, rstd, dx, dgamma, workspace, dres, dresidual, _raw_stream(at))
    else:
        t = (dout, h, gamma, rstd, dx, dgamma, workspace, dres, dresidual)
        _elsewhere(call, t, t, stream)


def moe_expert_matmul(x, w, offsets, out, err=None, row_slot=None, x_scale=None, w_scale=None, transposed: bool = False,
                      stream=None) -> None:
    """x [n][D], or with row_slot [n] (and err) [rows][D]; w [E][N][D], transposed [E][D][N]; offsets [E + 1] int32;
    out [n][N].  f32, bf16 (out bf16 or f32), or fp8 with x_scale [rows][ceil(D / 128)] and w_scale
    [E][ceil(N / 128)][ceil(D / 128)] f32 (out bf16 or f32).  Any strides of rows and matrices.  With transposed
    and the gradient of a forward product's out as x, out is the gradient of its rows."""
    call, at = (_marshal or _home()).moe_expert_matmul, x.get_device()
    if stream is None and at >= 0 and at == _device():
        call(x, w, offsets, out, err, row_slot, x_scale, w_scale, transposed, _raw_stream(at))
    else:
        t = (x, w, offsets, out, err, row_slot, x_scale, w_scale)
        _elsewhere(call, t + (transposed,), t, stream)


def moe_expert_matmul_backward(dout, x, offsets, dw, accumulate: bool = False, stream=None) -> None:
    """dout [n][N] and x [n][D] of one type (f32 or bf16), offsets [E + 1]; out: dw [E][N][D] (f32, or bf16 from
    bf16), added to with accumulate."""
    call, at = (_marshal or _home()).moe_expert_matmul_backward, dout.get_device()
    if stream is None and at >= 0 and at == _device():
        call(dout, x, offsets, dw, accumulate, _raw_stream(at))
    else:
        t = (dout, x, offsets, dw)
        _elsewhere(call, t + (accumulate,), t, stream)


def moe_swiglu(gu, h, h_scale=None, group: int = 0, count=None, stream=None) -> None:
    """gu [n][2 I] (f32 or bf16): gate columns, then up columns; h [n][I] f32, bf16 or fp8 (then h_scale
    [n][groups] f32).  count: one int32 on the device, the rows to compute (offsets[E:] for the rows that
    moe_sort_rows placed)."""
    call, at = (_marshal or _home()).moe_swiglu, gu.get_device()
    if stream is None and at >= 0 and at == _device():
        call(gu, h, h_scale, count, group, _raw_stream(at))
    else:
        t = (gu, h, h_scale, count)
        _elsewhere(call, t + (group,), t, stream)


def moe_swiglu_backward(gu, dh, dgu, h=None, count=None, stream=None) -> None:
    """gu and dgu [n][2 I], dh and (optional, the forward's rows again) h [n][I], all f32 or all bf16.  dgu may
    be gu."""
    call, at = (_marshal or _home()).moe_swiglu_backward, gu.get_device()
    if stream is None and at >= 0 and at == _device():
        call(gu, dh, dgu, h, count, _raw_stream(at))
    else:
        t = (gu, dh, dgu, h, count)
        _elsewhere(call, t, t, stream)


def moe_quantize_weights(w, codes, scale, transposed: bool = False, stream=None) -> None:
    """w [E][N][D] f32 or bf16; out: codes [E][N][D] fp8 and scale [E][ceil(N / 128)][ceil(D / 128)] f32, or with
    transposed those of each w[e]'s transpose."""
    call, at = (_marshal or _home()).moe_quantize_weights, w.get_device()
    if stream is None and at >= 0 and at == _device():
        call(w, codes, scale, transposed, _raw_stream(at))
    else:
        t = (w, codes, scale)
        _elsewhere(call, t + (transposed,), t, stream)
