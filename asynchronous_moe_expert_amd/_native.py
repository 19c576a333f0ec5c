"""ctypes binding of libmoestep.so.  Argument marshalling only: every step of the path runs
in the library's HIP kernels.  Tensors are torch device tensors (plumbing for device
memory and streams); each function takes the same name as the C call it wraps."""
from __future__ import annotations

import ctypes as C
import os
import struct

import torch

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libmoestep.so")

MOE_F32, MOE_BF16, MOE_FP8_E4M3 = 0, 1, 2
MOE_SOFTMAX, MOE_SIGMOID = 0, 1

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


_STRUCTS = [AssembleArgs, PackArgs, FfnArgs, StateC, CombineArgs, RouteArgs, RouteBackwardArgs, SortRowsArgs,
            MergeRowsArgs, MergeRowsBackwardArgs, ResidualNormArgs, ResidualNormBackwardArgs]
EXPORTS = ["moe_assemble", "moe_pack_ffn_weights", "moe_ffn_workspace_size", "moe_expert_ffn_grouped",
           "moe_state_reset", "moe_combine_release", "moe_combine_plan", "moe_combine_apply",
           "moe_combine_workspace_size", "moe_strerror", "moe_version", "moe_struct_size",
           "moe_combine_release_noalloc", "moe_combine_noalloc_max_arrivals", "moe_route", "moe_route_backward",
           "moe_sort_rows", "moe_sort_rows_workspace_size", "moe_merge_rows", "moe_merge_rows_backward",
           "moe_residual_norm", "moe_residual_norm_backward", "moe_residual_norm_backward_workspace_size"]


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


# ------------------------------------------------------------------ the home rank's side
# These calls check their tensors (device, type, shape, stride) before marshalling: a view that
# the kernels cannot address is refused with a MoeError, and tensors on another device than the
# current one are worked on where they are.  A decode step's calls take the GPU 3-5 us each, so
# the host path is kept short: the argument struct is packed as bytes in the struct's own layout
# (0.4 us; a ctypes.Structure takes four times as long to fill), the checks test for what is right
# first, and the current stream's handle is read directly (0.1 us; a torch.cuda.Stream object
# 1.9 us).  moe_residual_norm of 64 rows: 9.7 us a call before, 3.0 us of them the launch itself.

_F32, _BF16, _I32 = torch.float32, torch.bfloat16, torch.int32
_ROWS = (_F32, _BF16)
_FP8 = (torch.uint8, torch.float8_e4m3fn)
_ROWS8 = _ROWS + _FP8
_CODE = {_F32: MOE_F32, _BF16: MOE_BF16, torch.uint8: MOE_FP8_E4M3, torch.float8_e4m3fn: MOE_FP8_E4M3}


def _packer(cls) -> struct.Struct:
    """Packs the fields of an argument struct in its native layout."""
    chars = {_i32: "i", _i64: "q", _p: "P", C.c_size_t: "N", C.c_float: "f"}
    s = struct.Struct("@" + "".join(chars[t] for _, t in cls._fields_) + "0P")
    if s.size != C.sizeof(cls):
        raise MoeError(f"packed layout of {cls.__name__}: {s.size} bytes, {C.sizeof(cls)} expected")
    return s


_HOME = {"moe_route": _packer(RouteArgs), "moe_route_backward": _packer(RouteBackwardArgs),
         "moe_sort_rows": _packer(SortRowsArgs), "moe_merge_rows": _packer(MergeRowsArgs),
         "moe_merge_rows_backward": _packer(MergeRowsBackwardArgs), "moe_residual_norm": _packer(ResidualNormArgs),
         "moe_residual_norm_backward": _packer(ResidualNormBackwardArgs)}

_home: dict = {}  # name -> (pack, the library's function)


def _home_entry(name: str):
    _home[name] = entry = _HOME[name].pack, getattr(load(), name)
    return entry


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _mat(what: str, t, rows: int, cols: int, types) -> int:
    """A [rows][cols] device tensor of one of `types` whose rows are contiguous; its pitch."""
    if t.dtype not in types:
        raise MoeError(f"{what}: unsupported dtype {t.dtype}")
    if t.shape != (rows, cols):
        raise MoeError(f"{what}: shape {tuple(t.shape)}, expected ({rows}, {cols})")
    s0, s1 = t.stride()
    if s1 == 1 and s0 >= cols and rows > 1:
        return s0
    if s1 != 1 and cols > 1:
        raise MoeError(f"{what}: the elements of a row must be contiguous")
    if rows > 1 and s0 < cols:
        raise MoeError(f"{what}: rows overlap (stride {s0} for {cols} elements)")
    return s0 if rows > 1 else cols


def _vec(what: str, t, n: int, *types) -> int:
    """A contiguous device tensor of one of `types` with at least n elements; its address, 0 for None."""
    if t is None:
        return 0
    if t.dtype not in types:
        raise MoeError(f"{what}: unsupported dtype {t.dtype}")
    if t.numel() < n:
        raise MoeError(f"{what}: {t.numel()} elements, at least {n} expected")
    if not t.is_contiguous():
        raise MoeError(f"{what}: must be contiguous")
    return t.data_ptr()


def _each(what: str, t, T: int, K: int, dtype) -> int:
    """A contiguous device tensor of shape (T, K); its address."""
    if t.dtype is not dtype or t.shape != (T, K) or not t.is_contiguous():
        _mat(what, t, T, K, (dtype,))
        _vec(what, t, T * K, dtype)
    return t.data_ptr()


def _shape(what: str, t) -> tuple[int, int]:
    s = t.shape
    if len(s) != 2:
        raise MoeError(f"{what}: {len(s)} dimensions, 2 expected")
    return s


def _room(workspace) -> int:
    if workspace is None:
        return 0
    if not workspace.is_contiguous():
        raise MoeError("workspace: must be contiguous")
    return workspace.numel() * workspace.element_size()


def _home_call(name: str, values, tensors, stream) -> None:
    """One call of the library on the device that its tensors are on.  With a stream other than
    the current one, the tensors are recorded on it, so that the allocator keeps them until the
    call's work is done."""
    pack, fn = _home.get(name) or _home_entry(name)
    try:
        args = pack(*values)
    except (struct.error, OverflowError, TypeError) as e:
        raise MoeError(f"{name}: an argument is over the documented limits ({e})") from None
    at = tensors[0].get_device()
    for t in tensors:
        if t is not None and t.get_device() != at:
            raise MoeError(f"{name}: tensors on {tensors[0].device} and {t.device}")
    if at < 0:
        raise MoeError(f"{name}: tensors must be on a GPU, got {tensors[0].device}")
    handle = current = _raw_stream(at)
    if stream is not None:
        where = getattr(stream, "device", None)
        if where is not None and where.index != at:
            raise MoeError(f"{name}: a stream of {where} for tensors on {tensors[0].device}")
        handle = _stream(stream)
    if _device() == at:
        rc = fn(args, handle)
    else:
        with torch.cuda.device(at):
            rc = fn(args, handle)
    if rc != 0:
        _check(rc, name)
    if handle != current:
        if not hasattr(stream, "cuda_stream"):
            stream = torch.cuda.ExternalStream(handle, device=at) if handle else torch.cuda.default_stream(at)
        for t in tensors:
            if t is not None:
                t.record_stream(stream)


def _score(score, renorm) -> tuple[int, int]:
    if score not in (MOE_SOFTMAX, MOE_SIGMOID):
        raise MoeError(f"score must be MOE_SOFTMAX or MOE_SIGMOID, got {score!r}")
    return score, 1 if renorm else 0


def moe_route(logits, expert, w, bias=None, score: int = MOE_SOFTMAX, renorm: bool = True, scale: float = 1.0,
              stream=None) -> None:
    """logits [T][E] (f32 or bf16); out: expert [T][K] int32, w [T][K] f32."""
    T, E = _shape("logits", logits)
    K = _shape("expert", expert)[1]
    pitch = _mat("logits", logits, T, E, _ROWS)
    score, renorm = _score(score, renorm)
    _home_call("moe_route", (T, E, K, logits.data_ptr(), _CODE[logits.dtype], pitch, _vec("bias", bias, E, _F32), score,
                             renorm, scale, _each("expert", expert, T, K, _I32), _each("w", w, T, K, _F32)),
               (logits, expert, w, bias), stream)


def moe_route_backward(logits, expert, dw, dlogits, err, score: int = MOE_SOFTMAX, renorm: bool = True,
                       scale: float = 1.0, stream=None) -> None:
    """expert [T][K] as moe_route gave it, dw [T][K] f32; out: dlogits [T][E] of the logits' type."""
    T, E = _shape("logits", logits)
    K = _shape("expert", expert)[1]
    pitch = _mat("logits", logits, T, E, _ROWS)
    dpitch = _mat("dlogits", dlogits, T, E, (logits.dtype,))
    score, renorm = _score(score, renorm)
    _home_call("moe_route_backward",
               (T, E, K, logits.data_ptr(), _CODE[logits.dtype], pitch, _each("expert", expert, T, K, _I32),
                _each("dw", dw, T, K, _F32), score, renorm, scale, dlogits.data_ptr(), dpitch,
                _vec("err", err, 1, _I32)), (logits, expert, dw, dlogits, err), stream)


def moe_sort_rows_workspace_size(n_max: int) -> int:
    return load().moe_sort_rows_workspace_size(n_max)


def _groups(H: int, group: int) -> int:
    if group not in (0, 32, 64, 128):
        raise MoeError(f"group must be 0, 32, 64 or 128, got {group}")
    return (H + group - 1) // group if group else 1


def moe_sort_rows(expert, E_loc: int, x, xs, perm, pos, counts, offsets, err, workspace, expert_base: int = 0,
                  row_slot=None, x_scale=None, group: int = 0, stream=None) -> None:
    """expert [T][K] int32; x [T][H] (f32, bf16, or fp8 with x_scale [T][groups] f32), xs [T * K][H]
    of x's type (bf16 for fp8); xs None: the index alone (x may be None then).  perm and row_slot
    are optional."""
    T, K = _shape("expert", expert)
    n = T * K
    H, code, xp, xsp, xd, xsd, sd = 8, MOE_BF16, 8, 8, 0, 0, 0
    if xs is not None:
        if x is None:
            raise MoeError("x: required with xs")
        H = _shape("xs", xs)[1]
        xp = _mat("x", x, T, H, _ROWS8)
        code = _CODE[x.dtype]
        xsp = _mat("xs", xs, n, H, (_BF16,) if code == MOE_FP8_E4M3 else (x.dtype,))
        xd, xsd = x.data_ptr(), xs.data_ptr()
        if code == MOE_FP8_E4M3:
            if x_scale is None:
                raise MoeError("x_scale: required for fp8 rows")
            sd = _vec("x_scale", x_scale, T * _groups(H, group), _F32)
        else:
            x_scale = None
    else:
        x = x_scale = None
    _home_call("moe_sort_rows",
               (T, K, H, expert_base, E_loc, _each("expert", expert, T, K, _I32), xd, code, xp, sd, group, xsd, xsp,
                _vec("perm", perm, n, _I32), _vec("pos", pos, n, _I32), _vec("counts", counts, E_loc, _I32),
                _vec("offsets", offsets, E_loc + 1, _I32), _vec("row_slot", row_slot, n, _I32),
                _vec("err", err, 1, _I32), 0 if workspace is None else workspace.data_ptr(), _room(workspace)),
               (expert, x, xs, perm, pos, counts, offsets, err, workspace, row_slot, x_scale), stream)


def _positions(pos, w, T: int) -> tuple[int, int, int]:
    """pos: int32, T x K elements in token order ([T][K] or flat), w f32 like it or None; K and their
    addresses."""
    n = pos.numel()
    K = n // T if T else (pos.shape[-1] if pos.dim() > 1 else 1)
    if n != T * K:
        raise MoeError(f"pos: {n} elements are not a whole number for each of {T} tokens")
    if w is not None and w.numel() != n:
        raise MoeError(f"w: {w.numel()} elements, {n} expected")
    return K, _vec("pos", pos, n, _I32), _vec("w", w, n, _F32)


def moe_merge_rows(rows, pos, w, out, err, stream=None) -> None:
    """rows [n_rows][H]; pos (int32) and w (f32, or None: 1) [T][K]; out [T][H].  f32 or bf16 each.
    With the gradient of moe_sort_rows' xs as rows and w None, out is the gradient of its x."""
    T, H = _shape("out", out)
    K, posd, wd = _positions(pos, w, T)
    n_rows = _shape("rows", rows)[0]
    rp = _mat("rows", rows, n_rows, H, _ROWS)
    op = _mat("out", out, T, H, _ROWS)
    _home_call("moe_merge_rows", (T, K, H, rows.data_ptr(), _CODE[rows.dtype], rp, n_rows, posd, wd, out.data_ptr(),
                                  _CODE[out.dtype], op, _vec("err", err, 1, _I32)), (rows, pos, w, out, err), stream)


def moe_merge_rows_backward(dout, rows, pos, w, drows, dw, err, stream=None) -> None:
    """dout [T][H]; rows and drows [n_rows][H] of one type; pos, w and dw [T][K].  drows or dw (and
    then rows) may be None."""
    T, H = _shape("dout", dout)
    K, posd, wd = _positions(pos, w, T)
    dp = _mat("dout", dout, T, H, _ROWS)
    one = rows if rows is not None else drows
    if one is None or (drows is None and dw is None) or (dw is not None and rows is None):
        raise MoeError("moe_merge_rows_backward: drows, or dw with rows, must be given")
    n_rows, rp, drp, rd, drd = _shape("rows", one)[0], H, H, 0, 0
    if rows is not None:
        rp, rd = _mat("rows", rows, n_rows, H, _ROWS), rows.data_ptr()
    if drows is not None:
        drp, drd = _mat("drows", drows, n_rows, H, (rows.dtype,) if rows is not None else _ROWS), drows.data_ptr()
    _home_call("moe_merge_rows_backward",
               (T, K, H, dout.data_ptr(), _CODE[dout.dtype], dp, rd, _CODE[one.dtype], rp, n_rows, posd, wd, drd, drp,
                _vec("dw", dw, T * K, _F32), _vec("err", err, 1, _I32)), (dout, rows, pos, w, drows, dw, err), stream)


def moe_residual_norm(x, residual, gamma, eps: float, out, residual_out=None, rstd=None, out_scale=None,
                      group: int = 0, row_list=None, row_count=None, err=None, stream=None) -> None:
    """x, residual (optional) [T][H]; gamma [H]; out [T][H] f32, bf16 or fp8 (then out_scale [T][groups]
    f32).  Optional outputs: residual_out [T][H], rstd [T].  row_list [T], row_count [1] (int32): only
    these rows, with err."""
    T, H = _shape("x", x)
    xp = _mat("x", x, T, H, _ROWS)
    op = _mat("out", out, T, H, _ROWS8)
    rt, rp, rop, rd, rod, sd = x.dtype, H, H, 0, 0, 0
    if residual is not None:
        rt = residual.dtype
        rp, rd = _mat("residual", residual, T, H, _ROWS), residual.data_ptr()
    if residual_out is not None:
        if residual is None:
            rt = residual_out.dtype
        rop, rod = _mat("residual_out", residual_out, T, H, (rt,) if residual is not None else _ROWS), residual_out.data_ptr()
    oc = _CODE[out.dtype]
    if oc == MOE_FP8_E4M3:
        if out_scale is None:
            raise MoeError("out_scale: required for fp8 output")
        sd = _vec("out_scale", out_scale, T * _groups(H, group), _F32)
    else:
        out_scale = None
    _home_call("moe_residual_norm",
               (T, H, x.data_ptr(), _CODE[x.dtype], xp, rd, _CODE[rt], rp, _vec("gamma", gamma, H, _F32, _BF16),
                _CODE[gamma.dtype], eps, out.data_ptr(), oc, op, sd, group, rod, rop, _vec("rstd", rstd, T, _F32),
                _vec("row_list", row_list, T, _I32), _vec("row_count", row_count, 1, _I32), _vec("err", err, 1, _I32)),
               (x, residual, gamma, out, residual_out, rstd, out_scale, row_list, row_count, err), stream)


def moe_residual_norm_backward_workspace_size(H: int) -> int:
    return load().moe_residual_norm_backward_workspace_size(H)


def moe_residual_norm_backward(dout, h, gamma, rstd, dx, dgamma, workspace, dres=None, dresidual=None,
                               stream=None) -> None:
    """dout [T][H], h [T][H] (the forward's residual_out, or x), rstd [T]; out: dx [T][H] of dout's type,
    dresidual [T][H] of h's, dgamma [H] f32 (with the workspace); each may be None.  dres [T][H] of h's
    type is added to dx and dresidual."""
    T, H = _shape("dout", dout)
    dp = _mat("dout", dout, T, H, _ROWS)
    hp = _mat("h", h, T, H, _ROWS)
    p = []
    for what, t, like in (("dres", dres, h), ("dx", dx, dout), ("dresidual", dresidual, h)):
        p += (0, H) if t is None else (t.data_ptr(), _mat(what, t, T, H, (like.dtype,)))
    _home_call("moe_residual_norm_backward",
               (T, H, dout.data_ptr(), _CODE[dout.dtype], dp, h.data_ptr(), _CODE[h.dtype], hp,
                _vec("gamma", gamma, H, _F32, _BF16), _CODE[gamma.dtype], _vec("rstd", rstd, T, _F32), *p,
                _vec("dgamma", dgamma, H, _F32), 0 if workspace is None else workspace.data_ptr(), _room(workspace)),
               (dout, h, gamma, rstd, dx, dgamma, workspace, dres, dresidual), stream)
