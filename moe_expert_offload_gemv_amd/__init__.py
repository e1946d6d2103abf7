"""Python binding of libmoe_offload.so (include/moe_offload.h).

Argument marshalling only: every step of the MoE layer runs in the HIP
kernels and the host runtime of the shared library. Device buffers are torch
cuda tensors (passed by data_ptr()); host buffers are numpy arrays. The
functions keep the C names and raise MoeError on a negative return code.
If the library has not been built this module raises on first use; there is
no fallback path.
"""
from __future__ import annotations

import ctypes as C
import os

import numpy as np

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "lib", "libmoe_offload.so")

MOE_OK = 0
MOE_E_INVAL = -1
MOE_E_NOMEM = -2
MOE_E_HIP = -3
MOE_E_STATE = -4
MOE_E_CAPTURING = -5
MOE_E_RANGE = -6
MOE_Q4_32_F16 = 1
MOE_ACCUMULATE = 1
MOE_F32 = 0
MOE_F16 = 1
MOE_BF16 = 2
MOE_Q8_32 = 3
MOE_MAX_SWAP_LEAD = 8
MOE_STATIC_SCRATCH_BYTES = 16777216
MOE_COLD_GPU = 0
MOE_COLD_CPU = 1
MOE_HOST_COHERENT = 0
MOE_HOST_NONCOHERENT = 1
MOE_POOL_PER_LAYER = 0
MOE_POOL_GLOBAL = 1

EXPORTED = [
    "moe_expert_bytes", "moe_create", "moe_destroy", "moe_register_layer", "moe_register_router", "moe_seed",
    "moe_forward", "moe_prefill", "moe_cache_step", "moe_get_info", "moe_get_slot_table", "moe_get_stamps",
    "moe_get_miss_log", "moe_get_counts", "moe_last_error", "moe_profile", "moe_preheat", "moe_measure_read_bandwidth",
    "moe_forward_static_scratch",
    "moe_add_rmsnorm", "moe_q4_split", "moe_q4_matmul", "moe_q4_workspace_bytes", "moe_router_balance",
    "moe_router_balance_workspace_bytes", "moe_router_balance_grad",
]


class moe_config(C.Structure):
    _fields_ = [
        ("n_layers", C.c_int32), ("n_experts", C.c_int32), ("top_k", C.c_int32), ("hidden", C.c_int32),
        ("ffn", C.c_int32), ("quant", C.c_int32), ("pool_budget_bytes", C.c_int64), ("reserve_bytes", C.c_int64),
        ("window_tokens", C.c_int32), ("admit_misses", C.c_int32), ("max_batch_tokens", C.c_int32),
        ("max_prefill_tokens", C.c_int32), ("device", C.c_int32), ("host_alloc", C.c_int32),
        ("host_sets", C.c_int32), ("stream", C.c_void_p), ("capture_picks", C.c_int32), ("pool_mode", C.c_int32),
        ("swaps_per_step", C.c_int32), ("swap_lead", C.c_int32), ("cold_exec", C.c_int32),
        ("cpu_threads", C.c_int32), ("decode_launches", C.c_int32), ("decode_sync_polls", C.c_int32),
    ]


class moe_info(C.Structure):
    _fields_ = [(n, C.c_int64) for n in ("slots_per_layer", "expert_bytes", "pool_bytes", "host_bytes",
                                        "staging_experts", "clock", "steps", "host_threads", "host_isa",
                                        "pool_budget_bytes", "free_bytes_at_sizing")]


class moe_step_stats(C.Structure):
    _fields_ = [(n, C.c_int64) for n in ("step", "tokens", "hits", "misses", "admissions", "evictions",
                                        "hot_bytes", "cold_bytes", "copied_bytes", "copied_pcie_bytes",
                                        "distinct_experts", "distinct_cold_experts")]

    def as_dict(self):
        return {n: int(getattr(self, n)) for n, _ in self._fields_}


class moe_profile_stats(C.Structure):
    _fields_ = [("forwards", C.c_int64), ("route_ms", C.c_double), ("hot_gateup_ms", C.c_double),
                ("hot_down_ms", C.c_double), ("cold_gateup_ms", C.c_double), ("cold_down_ms", C.c_double),
                ("hot_picks", C.c_int64), ("cold_picks", C.c_int64), ("gateup_bytes_per_pick", C.c_int64),
                ("down_bytes_per_pick", C.c_int64), ("prefill_passes", C.c_int64),
                ("prefill_gateup_ms", C.c_double), ("prefill_down_ms", C.c_double), ("prefill_pairs", C.c_int64),
                ("prefill_tiles", C.c_int64), ("prefill_staged", C.c_int64), ("prefill_prep_ms", C.c_double),
                ("prefill_stage_ms", C.c_double), ("host_forwards", C.c_int64),
                ("host_expert_passes", C.c_int64), ("host_picks", C.c_int64), ("host_wait_ms", C.c_double),
                ("host_compute_ms", C.c_double), ("layer_forwards", C.c_int64), ("hot_layer_ms", C.c_double),
                ("cold_layer_ms", C.c_double)]

    def as_dict(self):
        return {n: getattr(self, n) for n, _ in self._fields_}


class MoeError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"[{code}] {msg}")
        self.code = code


_lib = None


def lib():
    """The loaded shared library (raises if it was not built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with python -m moe_expert_offload_gemv_amd.build")
        L = C.CDLL(LIB_PATH)
        vp, i32, i64, u32, f32 = C.c_void_p, C.c_int32, C.c_int64, C.c_uint32, C.c_float
        sig = {
            "moe_expert_bytes": (i64, [i32, i32]),
            "moe_create": (C.c_int, [C.POINTER(moe_config), C.POINTER(vp)]),
            "moe_destroy": (C.c_int, [vp]),
            "moe_register_layer": (C.c_int, [vp, i32, vp, vp, vp]),
            "moe_register_router": (C.c_int, [vp, i32, vp]),
            "moe_seed": (C.c_int, [vp, vp]),
            "moe_forward": (C.c_int, [vp, i32, i32, vp, vp, vp, vp, vp, u32]),
            "moe_forward_static_scratch": (C.c_int, [vp, i32, i32, vp, vp, vp, vp, vp, u32]),
            "moe_prefill": (C.c_int, [vp, i32, i32, vp, vp, vp, u32]),
            "moe_cache_step": (C.c_int, [vp, C.POINTER(moe_step_stats)]),
            "moe_get_info": (C.c_int, [vp, C.POINTER(moe_info)]),
            "moe_get_slot_table": (C.c_int, [vp, i32, vp]),
            "moe_get_stamps": (C.c_int, [vp, i32, vp]),
            "moe_get_miss_log": (C.c_int, [vp, vp, i64, C.POINTER(i64)]),
            "moe_get_counts": (C.c_int, [vp, vp]),
            "moe_last_error": (C.c_char_p, [vp]),
            "moe_profile": (C.c_int, [vp, i32, C.POINTER(moe_profile_stats)]),
            "moe_preheat": (C.c_int, [vp, i32, i32, C.POINTER(i32)]),
            "moe_measure_read_bandwidth": (C.c_int, [vp, i64, i32, i32, vp, C.POINTER(C.c_double)]),
            "moe_add_rmsnorm": (C.c_int, [i32, vp, i32, i32, i32, vp, i64, i32, vp, i64, vp, i64, vp, f32, i32, vp, i64,
                                          vp, i64]),
            "moe_q4_split": (C.c_int, [i32, i32, vp, vp, vp]),
            "moe_q4_matmul": (C.c_int, [i32, vp, i32, i32, i32, i32, vp, i64, vp, i64, vp, vp, i32, vp, i64, vp, i64,
                                        u32]),
            "moe_q4_workspace_bytes": (i64, [i32, i32, i32, i32]),
            "moe_router_balance": (C.c_int, [i32, vp, i32, i32, i32, i32, vp, i64, vp, f32, f32, vp, vp, vp, vp, vp, i64,
                                             u32]),
            "moe_router_balance_workspace_bytes": (i64, [i32, i32]),
            "moe_router_balance_grad": (C.c_int, [i32, vp, i32, i32, i32, vp, i64, vp, vp, vp, vp, f32, f32, i32, vp,
                                                  i64, u32]),
        }
        for name, (res, args) in sig.items():
            f = getattr(L, name)
            f.restype, f.argtypes = res, args
        _lib = L
    return _lib


def _check(ctx, rc: int) -> None:
    if rc != MOE_OK:
        msg = lib().moe_last_error(ctx) if ctx else b""
        raise MoeError(rc, (msg or b"").decode(errors="replace"))


def _dptr(t):
    """Device address of a torch cuda tensor (None -> NULL)."""
    if t is None:
        return None
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError("device arguments must be contiguous cuda tensors")
    return t.data_ptr()


def _hptr(a, dtype):
    a = np.ascontiguousarray(a, dtype=dtype)
    return a, a.ctypes.data


# ---------------------------------------------------------------------------

def moe_expert_bytes(hidden: int, ffn: int) -> int:
    return int(lib().moe_expert_bytes(hidden, ffn))


def moe_create(n_layers, n_experts, top_k, hidden, ffn, pool_budget_bytes, reserve_bytes=0, window_tokens=64,
               admit_misses=2, max_batch_tokens=64, max_prefill_tokens=0, device=0, host_alloc=MOE_HOST_COHERENT,
               host_sets=0, stream=None, capture_picks=None, pool_mode=0, swaps_per_step=0, swap_lead=0,
               cold_exec=MOE_COLD_GPU, cpu_threads=0, decode_launches=0, decode_sync_polls=0):
    """Returns an opaque context handle.

    stream: a torch.cuda.Stream, a raw hipStream_t int, or None for torch's
    current stream on the device (0, the null stream, is a valid handle).
    capture_picks: None for top_k (one token's picks per layer; 0 with cold_exec=MOE_COLD_CPU), 0 for off.
    cold_exec: MOE_COLD_GPU (zero-copy reads of cold experts) or MOE_COLD_CPU (host threads compute them).
    pool_mode: MOE_POOL_PER_LAYER (slots per layer) or MOE_POOL_GLOBAL (one pool for all layers).
    swaps_per_step: admissions per cache step (0: no limit); swap_lead: cache steps an admission waits
    for its copy before its table entry flips (0: at once).
    decode_launches: 1 for one launch per layer where the decode shape allows it, 0 or 2 for two (the default).
    decode_sync_polls: bound of the one-launch down work-groups' wait (0: the default, 2^20 polls).
    """
    if capture_picks is None:
        capture_picks = 0 if cold_exec == MOE_COLD_CPU else top_k
    if stream is None:
        stream = 0
        try:
            import torch

            if torch.cuda.is_available():
                stream = torch.cuda.current_stream(device).cuda_stream
        except ImportError:
            pass
    elif not isinstance(stream, int):
        stream = stream.cuda_stream
    cfg = moe_config(n_layers, n_experts, top_k, hidden, ffn, MOE_Q4_32_F16, pool_budget_bytes, reserve_bytes,
                     window_tokens, admit_misses, max_batch_tokens, max_prefill_tokens, device, host_alloc,
                     host_sets, stream, capture_picks, pool_mode, swaps_per_step, swap_lead, cold_exec, cpu_threads,
                     decode_launches, decode_sync_polls)
    out = C.c_void_p()
    rc = lib().moe_create(C.byref(cfg), C.byref(out))
    if rc != MOE_OK:
        raise MoeError(rc, "moe_create: " + (lib().moe_last_error(None) or b"").decode(errors="replace"))
    return out.value


def moe_destroy(ctx) -> None:
    _check(None, lib().moe_destroy(ctx))


def moe_register_layer(ctx, layer: int, gate, up, down) -> None:
    g, gp = _hptr(gate, np.uint8)
    u, up_ = _hptr(up, np.uint8)
    d, dp = _hptr(down, np.uint8)
    _check(ctx, lib().moe_register_layer(ctx, layer, gp, up_, dp))


def moe_register_router(ctx, layer: int, w_router) -> None:
    w, wp = _hptr(w_router, np.float32)
    _check(ctx, lib().moe_register_router(ctx, layer, wp))


def moe_seed(ctx, freq=None) -> None:
    if freq is None:
        _check(ctx, lib().moe_seed(ctx, None))
    else:
        f, fp = _hptr(freq, np.uint32)
        _check(ctx, lib().moe_seed(ctx, fp))


def moe_forward(ctx, layer: int, n_tokens: int, x, logits, y, ids=None, w=None, flags: int = 0) -> None:
    _check(ctx, lib().moe_forward(ctx, layer, n_tokens, _dptr(x), _dptr(logits), _dptr(y), _dptr(ids), _dptr(w),
                                  flags))


def moe_forward_static_scratch(ctx, layer: int, n_tokens: int, x, logits, y, ids=None, w=None,
                               flags: int = 0) -> None:
    _check(ctx, lib().moe_forward_static_scratch(ctx, layer, n_tokens, _dptr(x), _dptr(logits), _dptr(y),
                                                 _dptr(ids), _dptr(w), flags))


def moe_prefill(ctx, layer: int, n_tokens: int, x, logits, y, flags: int = 0) -> None:
    _check(ctx, lib().moe_prefill(ctx, layer, n_tokens, _dptr(x), _dptr(logits), _dptr(y), flags))


def moe_preheat(ctx, layer: int, max_experts: int) -> int:
    """Admit the cold experts the last prompt pass (of `layer`) used; returns how many were admitted."""
    n = C.c_int32(0)
    _check(ctx, lib().moe_preheat(ctx, layer, max_experts, C.byref(n)))
    return int(n.value)


def moe_cache_step(ctx) -> dict:
    s = moe_step_stats()
    _check(ctx, lib().moe_cache_step(ctx, C.byref(s)))
    return s.as_dict()


def moe_get_info(ctx) -> dict:
    s = moe_info()
    _check(ctx, lib().moe_get_info(ctx, C.byref(s)))
    return {n: int(getattr(s, n)) for n, _ in s._fields_}


def moe_get_slot_table(ctx, layer: int, n_experts: int) -> np.ndarray:
    out = np.empty(n_experts, np.int32)
    _check(ctx, lib().moe_get_slot_table(ctx, layer, out.ctypes.data))
    return out


def moe_get_stamps(ctx, layer: int, slots: int) -> np.ndarray:
    out = np.zeros(max(slots, 1), np.uint32)
    _check(ctx, lib().moe_get_stamps(ctx, layer, out.ctypes.data))
    return out[:slots]


def moe_get_miss_log(ctx) -> np.ndarray:
    n = C.c_int64()
    _check(ctx, lib().moe_get_miss_log(ctx, None, 0, C.byref(n)))
    out = np.empty(max(n.value, 1), np.uint64)
    _check(ctx, lib().moe_get_miss_log(ctx, out.ctypes.data, n.value, C.byref(n)))
    return out[: n.value]


def moe_get_counts(ctx, n_layers: int, n_experts: int) -> np.ndarray:
    out = np.empty((n_layers, n_experts), np.uint32)
    _check(ctx, lib().moe_get_counts(ctx, out.ctypes.data))
    return out


def moe_profile(ctx, enable: int = -1) -> dict:
    s = moe_profile_stats()
    _check(ctx, lib().moe_profile(ctx, enable, C.byref(s)))
    return s.as_dict()


def moe_measure_read_bandwidth(buf=None, nbytes: int = 0, reps: int = 3, host_coherent: bool = True,
                               stream=None) -> float:
    """GB/s of a plain 128-bit streaming read kernel: over the cuda tensor buf
    (HBM), or with buf None over nbytes of pinned host memory the library
    allocates (zero-copy over PCIe). A measurement aid, not the MoE path."""
    import torch

    if buf is not None:
        nbytes = buf.numel() * buf.element_size()
    s = stream if stream is not None else torch.cuda.current_stream()
    out = C.c_double(0.0)
    rc = lib().moe_measure_read_bandwidth(_dptr(buf), int(nbytes), int(reps), 1 if host_coherent else 0,
                                          s.cuda_stream, C.byref(out))
    if rc != MOE_OK:
        raise MoeError(rc, "moe_measure_read_bandwidth failed")
    return out.value


def moe_last_error(ctx) -> str:
    return (lib().moe_last_error(ctx) or b"").decode(errors="replace")


# ---------------------------------------------------------------------------
# Operators beside the experts: torch tensors of any strided rows on one
# device, issued on that device's current torch stream (or `stream`: a
# torch.cuda.Stream or a raw hipStream_t int). A call of theirs takes a few
# microseconds on the GPU, so the checks here are kept to a few of the host.

_types = {}  # torch dtype -> type code, filled with torch's first use
_dtypes = {}  # name -> torch dtype, likewise: comparing names would format one per argument and call
_raw_stream = None


def _dense():
    """The library's handle, with the torch side set up."""
    global _raw_stream
    if _raw_stream is None:
        import torch

        _types.update({torch.float32: MOE_F32, torch.float16: MOE_F16, torch.bfloat16: MOE_BF16, torch.int8: MOE_Q8_32})
        _dtypes.update({str(d): d for d in (torch.float32, torch.float16, torch.int32, torch.uint8, torch.bool)})
        # the stream's handle without a Stream object around it, where this torch has that
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda dev: torch.cuda.current_stream(dev).cuda_stream)
    return _lib or lib()


def _fail(rc: int):
    """Raises what a call without a context left in this thread's message."""
    raise MoeError(rc, moe_last_error(None))


def _stream_of(stream, dev):
    if stream is None:
        return _raw_stream(dev)
    return stream if isinstance(stream, int) else stream.cuda_stream


def _rows(name, t, dev, shape):
    """(type code, address, row stride) of a 2-d tensor whose rows are contiguous runs of values."""
    if t.shape != shape or t.get_device() != dev or dev < 0 or t.dtype not in _types:
        raise ValueError(f"{name}: {t.dtype} {tuple(t.shape)} on {t.device}; fp32, fp16, bf16 or int8 of shape "
                         f"{tuple(shape)} on cuda device {max(dev, 0)} is needed")
    stride, step = t.stride()
    width = shape[1]
    if stride < width or step != 1:
        if (step != 1 and width > 1) or (stride < width and shape[0] > 1):
            raise ValueError(f"{name}: rows must be contiguous and must not overlap, strides {t.stride()}")
        stride = max(stride, width)
    return _types[t.dtype], t.data_ptr(), stride


def _flat(name, t, dev, shape, dtype):
    """Address of a contiguous tensor (None -> NULL); dtype: its name in torch."""
    if t is None:
        return None
    if t.shape != shape or t.get_device() != dev or dev < 0 or t.dtype is not _dtypes[dtype] or not t.is_contiguous():
        raise ValueError(f"{name}: {t.dtype} {tuple(t.shape)} on {t.device}; a contiguous {dtype} tensor of shape "
                         f"{tuple(shape)} on cuda device {max(dev, 0)} is needed")
    return t.data_ptr()


def _fits(*values) -> bool:
    """Whether ctypes hands each on as it is: it cuts an int to an int32 parameter's bits without a word."""
    return all(-0x80000000 <= v <= 0x7FFFFFFF for v in values)


def _dims(name, t, n):
    """The shape of a tensor of n dimensions (two: rows)."""
    shape = t.shape
    if len(shape) != n or shape[0] > 0x7FFFFFFF or shape[1] > 0x7FFFFFFF:
        raise ValueError(f"{name}: shape {tuple(shape)}; {n} dimensions of at most 2147483647 are needed")
    return shape


def _number(name, v):
    if not -0x80000000 <= v <= 0xFFFFFFFF:  # within it the library sees the value, or one that it refuses
        raise ValueError(f"{name}: {v} is out of range")
    return v


def _workspace(t, dev, stream, make):
    """(tensor, address, bytes) of the workspace tensor given, or of a new one from torch."""
    if t is None:
        t = make()
        if t is None:
            return None, None, 0
        if stream is not None:  # torch's allocator would hand its memory on by the current stream's order
            raise ValueError("workspace: a call on a stream of its own needs one")
    if t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"workspace: a contiguous tensor on cuda device {dev} is needed")
    return t, t.data_ptr(), t.numel() * t.element_size()


def moe_add_rmsnorm(x, weight, out, residual=None, residual_out=None, scales=None, eps=1e-6, stream=None) -> None:
    """out = RMS norm of x + residual (x without one) times weight; residual_out = x + residual.

    x [T][H] fp32, fp16 or bf16; weight fp32 [H] or None; out [T][H] of those types, or int8 with
    scales fp32 [T][H/32] (MOE_Q8_32). residual [T][H] is updated in place unless residual_out is given.
    """
    L = _dense()
    shape, dev = _dims("x", x, 2), x.get_device()
    T, H = shape
    xt, xp, xs = _rows("x", x, dev, shape)
    ot, op, os_ = _rows("out", out, dev, shape)
    rt, rp, rs, rop, ros = xt, None, 0, None, 0
    if residual is not None:
        rt, rp, rs = _rows("residual", residual, dev, shape)
        rop, ros = rp, rs
        if residual_out is not None:
            rot, rop, ros = _rows("residual_out", residual_out, dev, shape)
            if rot != rt:
                raise ValueError(f"residual_out: {residual_out.dtype}, but the residual is {residual.dtype}")
    elif residual_out is not None:
        raise ValueError("residual_out: there is no residual")
    sp, ss = None, 0
    if scales is not None:
        st, sp, ss = _rows("scales", scales, dev, (T, H // 32))
        if st != MOE_F32:
            raise ValueError(f"scales: {scales.dtype}")
    wp = _flat("weight", weight, dev, (H,), "torch.float32")
    rc = L.moe_add_rmsnorm(dev, _stream_of(stream, dev), T, H, xt, xp, xs, rt, rp, rs, rop, ros, wp, eps, ot, op, os_, sp,
                           ss)
    if rc:
        _fail(rc)


def moe_q4_split(blocks):
    """(nibbles uint8 [rows][k/32][16], scales fp16 [rows][k/32]) of canonical blocks uint8 [rows][k/32][18]."""
    b = np.ascontiguousarray(blocks, np.uint8)
    if b.ndim != 3 or b.shape[2] != 18:
        raise ValueError(f"blocks of shape [rows][k/32][18] are needed, got {b.shape}")
    nib, scl = np.empty(b.shape[:2] + (16,), np.uint8), np.empty(b.shape[:2], np.float16)
    rc = lib().moe_q4_split(b.shape[0], 32 * b.shape[1], b.ctypes.data, nib.ctypes.data, scl.ctypes.data)
    if rc:
        _fail(rc)
    return nib, scl


def moe_q4_workspace_bytes(n_tokens: int, n_out: int, k: int, x_type: int) -> int:
    return int(lib().moe_q4_workspace_bytes(n_tokens, n_out, k, x_type)) if _fits(n_tokens, n_out, k, x_type) else -1


def moe_q4_workspace(x, nibbles):
    """A workspace tensor for moe_q4_matmul of x with these weights (None if it needs none)."""
    L = _dense()
    T, K = _dims("x", x, 2)
    N = _dims("nibbles", nibbles, 3)[0]
    return _q4_workspace(x, nibbles, L.moe_q4_workspace_bytes(T, N, K, _types.get(x.dtype, -1)))


def _q4_workspace(x, nibbles, n):
    if n < 0:
        raise ValueError(f"no product of x {x.dtype} {tuple(x.shape)} with weights {tuple(nibbles.shape)}")
    if n:
        import torch

        return torch.empty(n, dtype=torch.uint8, device=x.device)
    return None


def moe_q4_matmul(x, nibbles, w_scales, y, scales=None, workspace=None, flags: int = 0, stream=None) -> None:
    """y [T][N] = x [T][K] times the 4-bit weights [N][K] (nibbles, w_scales: the planes of moe_q4_split).

    x fp32, fp16, bf16, or int8 with scales fp32 [T][K/32]; y fp32, fp16 or bf16. Without a workspace
    a call that needs one allocates it from torch.
    """
    L = _dense()
    shape, dev = _dims("x", x, 2), x.get_device()
    T, K = shape
    N = _dims("nibbles", nibbles, 3)[0]
    xt, xp, xs = _rows("x", x, dev, shape)
    np_ = _flat("nibbles", nibbles, dev, (N, K // 32, 16), "torch.uint8")
    wp = _flat("w_scales", w_scales, dev, (N, K // 32), "torch.float16")
    yt, yp, ys = _rows("y", y, dev, (T, N))
    sp, ss = None, 0
    if scales is not None:
        st, sp, ss = _rows("scales", scales, dev, (T, K // 32))
        if st != MOE_F32:
            raise ValueError(f"scales: {scales.dtype}")
    workspace, kp, kn = _workspace(workspace, dev, stream,
                                   lambda: _q4_workspace(x, nibbles, L.moe_q4_workspace_bytes(T, N, K, xt)))
    rc = L.moe_q4_matmul(dev, _stream_of(stream, dev), T, N, K, xt, xp, xs, sp, ss, np_, wp, yt, yp, ys, kp, kn,
                         _number("flags", flags))
    if rc:
        _fail(rc)


def moe_router_balance_workspace_bytes(n_tokens: int, n_experts: int) -> int:
    return int(lib().moe_router_balance_workspace_bytes(n_tokens, n_experts)) if _fits(n_tokens, n_experts) else -1


def moe_router_balance_workspace(logits):
    """A workspace tensor for moe_router_balance of these logits."""
    import torch

    n = moe_router_balance_workspace_bytes(*_dims("logits", logits, 2))
    if n < 0:
        raise ValueError(f"no balance of logits {tuple(logits.shape)}")
    return torch.empty(n, dtype=torch.uint8, device=logits.device)


def moe_router_balance(logits, top_k: int, counts, load, stats, lse, valid=None, balance=0.0, z=0.0, workspace=None,
                       flags: int = 0, stream=None) -> None:
    """Per-expert counts, loads and the balance and z losses of logits [T][E] (see moe_offload.h).

    counts int32 [E], load fp32 [E], stats fp32 [4] and lse fp32 [T] are outputs; valid uint8 or bool [T] leaves
    out tokens. Without a workspace the call allocates it from torch.
    """
    L = _dense()
    shape, dev = _dims("logits", logits, 2), logits.get_device()
    T, E = shape
    zt, zp, zs = _rows("logits", logits, dev, shape)
    vp = None
    if valid is not None:
        vp = _flat("valid", valid, dev, (T,), "torch.bool" if valid.dtype is _dtypes["torch.bool"] else "torch.uint8")
    cp = _flat("counts", counts, dev, (E,), "torch.int32")
    lp = _flat("load", load, dev, (E,), "torch.float32")
    tp = _flat("stats", stats, dev, (4,), "torch.float32")
    ep = _flat("lse", lse, dev, (T,), "torch.float32")
    workspace, kp, kn = _workspace(workspace, dev, stream, lambda: moe_router_balance_workspace(logits))
    rc = L.moe_router_balance(dev, _stream_of(stream, dev), T, E, _number("top_k", top_k), zt, zp, zs, vp, balance, z, cp, lp,
                              tp, ep, kp, kn, _number("flags", flags))
    if rc:
        _fail(rc)


def moe_router_balance_grad(logits, load, stats, lse, dlogits, dloss=None, balance=0.0, z=0.0, flags: int = 0,
                            stream=None) -> None:
    """dlogits [T][E] = gradient of stats[0] to the logits, times dloss (fp32 [1], None: 1)."""
    L = _dense()
    shape, dev = _dims("logits", logits, 2), logits.get_device()
    T, E = shape
    zt, zp, zs = _rows("logits", logits, dev, shape)
    lp = _flat("load", load, dev, (E,), "torch.float32")
    tp = _flat("stats", stats, dev, (4,), "torch.float32")
    ep = _flat("lse", lse, dev, (T,), "torch.float32")
    gp = _flat("dloss", dloss, dev, (1,), "torch.float32")
    dt, dp, ds = _rows("dlogits", dlogits, dev, shape)
    rc = L.moe_router_balance_grad(dev, _stream_of(stream, dev), T, E, zt, zp, zs, lp, tp, ep, gp, balance, z, dt, dp, ds,
                                   _number("flags", flags))
    if rc:
        _fail(rc)
