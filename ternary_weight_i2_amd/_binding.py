"""ctypes binding of libbitnet_i2s.so (C ABI in include/bitnet_i2s.h).

Argument marshalling only: each function checks the dtype, shape, device
and contiguity of every torch tensor it is given (so a wrong K or a short
output buffer is refused on the host, never read or written out of bounds),
passes ``data_ptr()`` and the current HIP stream, and raises ``BitnetError``
on a non-zero status.  Every step of the computation
runs in the library's HIP kernels; nothing here computes a result.
"""
from __future__ import annotations

import ctypes
import functools
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libbitnet_i2s.so")
# the same library built with per-launch start/end stamps of the decode GEMV
# (include/bitnet_i2s_stamps.h); a measurement aid, never loaded by default
_STAMPS_PATH = os.path.join(_HERE, "libbitnet_i2s_stamps.so")

OK, E_NULL, E_SHAPE, E_ALIGN, E_DTYPE, E_VALUE, E_HIP = range(7)
F32, BF16 = 0, 1
GEMV_MAX_N = 64
LINEAR_FUSED_MAX_N = 2     # bitnet_linear_i2s: one fused launch up to this N


MAX_GROUP = 8


class I2SMatrix(ctypes.Structure):
    """Mirror of bitnet_i2s_matrix."""
    _fields_ = [("packed", ctypes.c_void_p), ("M", ctypes.c_int64),
                ("w_scale", ctypes.c_float), ("dot", ctypes.c_void_p),
                ("y", ctypes.c_void_p)]


KV4_PAGE = 64              # tokens of a page of the 4-bit cache
W4_BY_GROUP = 0x1000       # W4Desc.group: the steps lie group by group


class KV4Batch(ctypes.Structure):
    """Mirror of bitnet_kv4_batch."""
    _fields_ = [("cache", ctypes.c_void_p), ("n_pages", ctypes.c_int64),
                ("n_kv_heads", ctypes.c_int64), ("head_dim", ctypes.c_int64),
                ("table", ctypes.c_void_p), ("max_pages", ctypes.c_int64),
                ("kv_len", ctypes.c_void_p), ("q_start", ctypes.c_void_p),
                ("n_seqs", ctypes.c_int64)]


class RotaryPlan(ctypes.Structure):
    """Mirror of bitnet_rotary_plan."""
    _fields_ = [("turns", ctypes.c_void_p), ("rot", ctypes.c_int64),
                ("interleaved", ctypes.c_int), ("magnitude", ctypes.c_double)]


class W4Desc(ctypes.Structure):
    """Mirror of bitnet_w4_matrix."""
    _fields_ = [("codes", ctypes.c_void_p), ("steps", ctypes.c_void_p), ("M", ctypes.c_int64),
                ("K", ctypes.c_int64), ("group", ctypes.c_int64)]


class BitnetError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"bitnet status {status}: {msg}")
        self.status = status


_lib = None


def lib_path() -> str:
    return _LIB_PATH


def load() -> ctypes.CDLL:
    """Load the HIP library; raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    _lib = _open(_LIB_PATH)
    return _lib


def use_library(which: str) -> None:
    """Route every call through the product library ("main") or its
    instrumented twin ("stamps", which also records per-launch start/end
    stamps of the decode GEMV).  Both must have been built."""
    global _lib
    if which == "main":
        _lib = _open(_LIB_PATH)
    elif which == "stamps":
        L = _open(_STAMPS_PATH)
        L.bitnet_stamps_reset.argtypes = [ctypes.c_int, ctypes.c_void_p]
        L.bitnet_stamps_reset.restype = ctypes.c_int
        L.bitnet_stamps_read.argtypes = [ctypes.POINTER(ctypes.c_uint64), ctypes.c_int]
        L.bitnet_stamps_read.restype = ctypes.c_int
        _lib = L
    else:
        raise ValueError(which)


def stamps_reset(rewind: bool = False) -> None:
    """Clear the stamp slots on the current stream (instrumented library)."""
    import torch
    _check(load().bitnet_stamps_reset(int(rewind), torch.cuda.current_stream().cuda_stream))


def stamps_read(max_launches: int) -> list[tuple[int, int]]:
    """[(start, end)] in 100 MHz ticks for the launches since the last rewind."""
    buf = (ctypes.c_uint64 * (2 * max_launches))()
    n = load().bitnet_stamps_read(buf, max_launches)
    if n < 0:
        raise BitnetError(E_HIP, "bitnet_stamps_read failed")
    return [(buf[2 * i], buf[2 * i + 1]) for i in range(n)]


def _open(path: str) -> ctypes.CDLL:
    if not os.path.exists(path):
        raise RuntimeError(
            f"{path} is missing: build it with __graft_entry__.build() "
            "(there is no fallback implementation)")
    L = ctypes.CDLL(path)
    p, i64, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_float
    L.bitnet_pack_i2s.argtypes = [p, i64, i64, p, p]
    L.bitnet_quant_act_i8.argtypes = [p, ctypes.c_int, i64, i64, p, p, p, p]
    sig = [p, f32, i64, i64, p, p, p, i64, p, p, p]
    L.bitnet_gemv_i2s_i8.argtypes = sig
    L.bitnet_gemm_i2s_i8.argtypes = sig
    L.bitnet_gemv_i2s_lut.argtypes = sig
    L.bitnet_linear_i2s.argtypes = [p, ctypes.c_int, i64, i64, ctypes.POINTER(I2SMatrix),
                                    ctypes.c_int, p, p, p, p]
    L.bitnet_linear_i2s.restype = ctypes.c_int
    L.bitnet_gemm_i2s_i8_group.argtypes = [ctypes.POINTER(I2SMatrix), ctypes.c_int, i64, p, p, p,
                                           i64, p]
    L.bitnet_gemm_i2s_i8_group.restype = ctypes.c_int
    L.bitnet_gemv_i2s_i8_group.argtypes = L.bitnet_gemm_i2s_i8_group.argtypes
    L.bitnet_gemv_i2s_i8_group.restype = ctypes.c_int
    L.bitnet_ffn_act_quant_i8.argtypes = [p, p, p, f32, i64, i64, p, p, p, p]
    L.bitnet_ffn_act_quant_i8.restype = ctypes.c_int
    L.bitnet_absmean_i2s.argtypes = [p, ctypes.c_int, i64, i64, p, ctypes.POINTER(ctypes.c_float), p]
    L.bitnet_absmean_i2s.restype = ctypes.c_int
    L.bitnet_pack_i2s_f32.argtypes = [p, i64, i64, p, ctypes.POINTER(ctypes.c_float), p]
    L.bitnet_pack_i2s_f32.restype = ctypes.c_int
    i32, kv4 = ctypes.c_int, ctypes.POINTER(KV4Batch)
    L.bitnet_block_norm_quant_i8.argtypes = [p, i32, i32, p, p, i64, f32, p, p, i32, p, f32, i64,
                                             i64, p, p, p, p, p]
    L.bitnet_block_norm_quant_i8.restype = ctypes.c_int
    L.bitnet_kv4_append.argtypes = [kv4, p, i64, p, i64, i32, i64, p]
    L.bitnet_kv4_append.restype = ctypes.c_int
    L.bitnet_kv4_read.argtypes = [kv4, p, p, i32, i64, p]
    L.bitnet_kv4_read.restype = ctypes.c_int
    L.bitnet_attn_kv4_workspace.argtypes = [i64] * 8
    L.bitnet_attn_kv4_workspace.restype = i64
    L.bitnet_attn_kv4.argtypes = [kv4, p, i64, i32, i64, i64, f32, i64, i64, i64, p, p, i64, p]
    L.bitnet_attn_kv4.restype = ctypes.c_int
    plan = ctypes.POINTER(RotaryPlan)
    L.bitnet_rotary.argtypes = [plan, p, i64, i32, i64, i64, i64, p, i32, p, i64, p]
    L.bitnet_rotary.restype = ctypes.c_int
    L.bitnet_rotary_kv4_append.argtypes = [kv4, plan, p, i64, p, i64, i64, p, i64, p, i64, i32, i64,
                                           p, p]
    L.bitnet_rotary_kv4_append.restype = ctypes.c_int
    L.bitnet_kv4_weigh_workspace.argtypes = [i64] * 8
    L.bitnet_kv4_weigh_workspace.restype = i64
    L.bitnet_kv4_weigh.argtypes = [kv4, p, i64, i32, i64, i64, f32, i64, i64, i64, p, f32, p, p, i64, p]
    L.bitnet_kv4_weigh.restype = ctypes.c_int
    L.bitnet_kv4_evict.argtypes = [kv4, p, p, i64, i64, i64, i64, p, p, p, i64, p]
    L.bitnet_kv4_evict_workspace.argtypes, L.bitnet_kv4_evict_workspace.restype = [i64] * 3, i64
    L.bitnet_kv4_evict.restype = ctypes.c_int
    w4 = ctypes.POINTER(W4Desc)
    for fn, args in (("bitnet_pack_w4", [p, i32, w4, p]), ("bitnet_pack_w4_codes", [p, p, w4, p]),
                     ("bitnet_w4_rows", [w4, p, i64, p, i32, p]),
                     ("bitnet_linear_w4", [p, i32, i64, w4, p, p, i64, p])):
        getattr(L, fn).argtypes, getattr(L, fn).restype = args, ctypes.c_int
    L.bitnet_linear_w4_workspace.argtypes, L.bitnet_linear_w4_workspace.restype = [i64] * 3, i64
    for fn in ("bitnet_pack_i2s", "bitnet_quant_act_i8", "bitnet_gemv_i2s_i8",
               "bitnet_gemm_i2s_i8", "bitnet_gemv_i2s_lut", "bitnet_abi_version"):
        getattr(L, fn).restype = ctypes.c_int
    L.bitnet_abi_version.argtypes = []
    L.bitnet_last_error.argtypes = []
    L.bitnet_last_error.restype = ctypes.c_char_p
    return L


def _check(status: int) -> None:
    if status != OK:
        msg = load().bitnet_last_error().decode(errors="replace")
        raise BitnetError(status, msg)


def _stream(t) -> int:
    import torch
    return torch.cuda.current_stream(t.device).cuda_stream


def _ptr(t) -> int | None:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensor must live on the GPU")
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return t.data_ptr()


def _expect(t, name, dtype, shape, device=None):
    """Refuse a tensor of the wrong dtype, shape or device before any launch."""
    if t is None:
        raise ValueError(f"{name} is required")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, the other operands on {device}")


def _expect_tokens(xq, x_scale, x_sum):
    """Quantised tokens xq[N][K] int8 with s[N] fp32 and sum[N] int32 -> (N, K)."""
    import torch
    if xq is None or xq.dim() != 2:
        raise ValueError("xq must be a 2-D [N][K] tensor")
    N, K = xq.shape
    _expect(xq, "xq", torch.int8, (N, K))
    _expect(x_scale, "x_scale", torch.float32, (N,), xq.device)
    _expect(x_sum, "x_sum", torch.int32, (N,), xq.device)
    return N, K


def _expect_packed(P, K, device, name="packed"):
    """I2_S weights [M][K/4] uint8 for reduction length K -> M."""
    import torch
    if P is None or P.dim() != 2:
        raise ValueError(f"{name} must be a 2-D [M][K/4] tensor")
    if K % 4:
        raise ValueError(f"K={K} is not a multiple of 4")
    _expect(P, name, torch.uint8, (P.shape[0], K // 4), device)
    return P.shape[0]


def _expect_outputs(dot, y, N, M, device, name=""):
    import torch
    if dot is not None:
        _expect(dot, f"{name}dot", torch.int32, (N, M), device)
    if y is not None:
        _expect(y, f"{name}y", torch.float32, (N, M), device)


def abi_version() -> int:
    return load().bitnet_abi_version()


def pack(w):
    """int8 ternary W[M][K] (cuda) -> uint8 I2_S packed[M][K/4]."""
    import torch
    if w.dtype != torch.int8 or w.dim() != 2:
        raise TypeError("w must be a 2-D int8 tensor")
    M, K = w.shape
    if K % 4:
        raise ValueError(f"K={K} is not a multiple of 4")
    out = torch.empty((M, K // 4), dtype=torch.uint8, device=w.device)
    _check(load().bitnet_pack_i2s(_ptr(w), M, K, _ptr(out), _stream(w)))
    return out


def absmean_pack(w, out=None):
    """fp32 or bf16 weights W[M][K] (cuda) -> (uint8 I2_S packed[M][K/4], AbsMean
    scale alpha as a Python float)."""
    import torch
    if w.dim() != 2:
        raise TypeError("w must be 2-D [M][K]")
    dt = {torch.float32: F32, torch.bfloat16: BF16}.get(w.dtype)
    if dt is None:
        raise TypeError("w must be float32 or bfloat16")
    M, K = w.shape
    if K % 4:
        raise ValueError(f"K={K} is not a multiple of 4")
    packed = out if out is not None else torch.empty((M, K // 4), dtype=torch.uint8,
                                                     device=w.device)
    _expect(packed, "out", torch.uint8, (M, K // 4), w.device)
    alpha = ctypes.c_float(0.0)
    _check(load().bitnet_absmean_i2s(_ptr(w), dt, M, K, _ptr(packed), ctypes.byref(alpha),
                                     _stream(w)))
    return packed, alpha.value


def pack_f32(w, out=None):
    """fp32 weights already ternary in value, W[M][K] (cuda) -> (packed I2_S by
    sign with the 1e-6 zero threshold, max|w| as a Python float)."""
    import torch
    if w.dtype != torch.float32 or w.dim() != 2:
        raise TypeError("w must be a 2-D float32 tensor")
    M, K = w.shape
    if K % 4:
        raise ValueError(f"K={K} is not a multiple of 4")
    packed = out if out is not None else torch.empty((M, K // 4), dtype=torch.uint8,
                                                     device=w.device)
    _expect(packed, "out", torch.uint8, (M, K // 4), w.device)
    wmax = ctypes.c_float(0.0)
    _check(load().bitnet_pack_i2s_f32(_ptr(w), M, K, _ptr(packed), ctypes.byref(wmax),
                                      _stream(w)))
    return packed, wmax.value


def quant_act(x, out=None):
    """fp32 or bf16 x[N][K] (cuda) -> (int8 xq[N][K], fp32 s[N], int32 xsum[N])."""
    import torch
    if x.dim() != 2:
        raise TypeError("x must be 2-D [N][K]")
    dt = {torch.float32: F32, torch.bfloat16: BF16}.get(x.dtype)
    if dt is None:
        raise TypeError("x must be float32 or bfloat16")
    N, K = x.shape
    if out is None:
        xq = torch.empty((N, K), dtype=torch.int8, device=x.device)
        s = torch.empty((N,), dtype=torch.float32, device=x.device)
        xs = torch.empty((N,), dtype=torch.int32, device=x.device)
    else:
        xq, s, xs = out
        _expect(xq, "xq", torch.int8, (N, K), x.device)
        _expect(s, "x_scale", torch.float32, (N,), x.device)
        _expect(xs, "x_sum", torch.int32, (N,), x.device)
    _check(load().bitnet_quant_act_i8(_ptr(x), dt, N, K, _ptr(xq), _ptr(s),
                                      _ptr(xs), _stream(x)))
    return xq, s, xs


def _matmul(fn, packed, w_scale, xq, x_scale, x_sum, want_dot, want_y, out):
    import torch
    N, K = _expect_tokens(xq, x_scale, x_sum)
    M = _expect_packed(packed, K, xq.device)
    if out is not None:
        dot, y = out
        _expect_outputs(dot, y, N, M, xq.device)
    else:
        dot = torch.empty((N, M), dtype=torch.int32, device=xq.device) if want_dot else None
        y = torch.empty((N, M), dtype=torch.float32, device=xq.device) if want_y else None
    _check(fn(_ptr(packed), float(w_scale), M, K, _ptr(xq), _ptr(x_scale),
              _ptr(x_sum), N, _ptr(dot), _ptr(y), _stream(xq)))
    return dot, y


def gemv(packed, w_scale, xq, x_scale, x_sum, want_dot=True, want_y=True, out=None):
    """Decode matmul (1..64 tokens) -> (int32 dot[N][M] | None, fp32 y[N][M] | None)."""
    return _matmul(load().bitnet_gemv_i2s_i8, packed, w_scale, xq, x_scale, x_sum,
                   want_dot, want_y, out)


def gemv_lut(packed, w_scale, xq, x_scale, x_sum, want_dot=True, want_y=True, out=None):
    """Decode matmul by table lookup (K <= 8192) -> (dot | None, y | None),
    the same values as gemv."""
    return _matmul(load().bitnet_gemv_i2s_lut, packed, w_scale, xq, x_scale, x_sum,
                   want_dot, want_y, out)


def gemm(packed, w_scale, xq, x_scale, x_sum, want_dot=True, want_y=True, out=None):
    """Prefill matmul (any token count, int8 MFMA) -> (dot | None, y | None)."""
    return _matmul(load().bitnet_gemm_i2s_i8, packed, w_scale, xq, x_scale, x_sum,
                   want_dot, want_y, out)


def _mats_out(mats, N, K, device, want_dot, want_y, out):
    import torch
    if not 1 <= len(mats) <= MAX_GROUP:
        raise ValueError(f"{len(mats)} matrices; a call takes 1..{MAX_GROUP}")
    for i, (P, _) in enumerate(mats):
        _expect_packed(P, K, device, f"mats[{i}] packed")
    if out is not None:
        if len(out) != len(mats):
            raise ValueError("out must hold one (dot, y) pair per matrix")
        for i, ((P, _), (d, y)) in enumerate(zip(mats, out)):
            _expect_outputs(d, y, N, P.shape[0], device, f"out[{i}] ")
        return out
    res = []
    for P, _ in mats:
        M = P.shape[0]
        res.append((torch.empty((N, M), dtype=torch.int32, device=device) if want_dot else None,
                    torch.empty((N, M), dtype=torch.float32, device=device) if want_y else None))
    return res


def _mat_array(mats, out):
    arr = (I2SMatrix * len(mats))()
    for i, ((P, ws), (d, y)) in enumerate(zip(mats, out)):
        arr[i] = I2SMatrix(_ptr(P), P.shape[0], float(ws), _ptr(d), _ptr(y))
    return arr


def gemm_group(mats, xq, x_scale, x_sum, want_dot=True, want_y=True, out=None):
    """Prefill matmul of every (packed, w_scale) in ``mats`` by the same
    quantised tokens, one MFMA launch -> [(dot | None, y | None) per matrix]."""
    N, K = _expect_tokens(xq, x_scale, x_sum)
    out = _mats_out(mats, N, K, xq.device, want_dot, want_y, out)
    _check(load().bitnet_gemm_i2s_i8_group(_mat_array(mats, out), len(mats), K, _ptr(xq),
                                           _ptr(x_scale), _ptr(x_sum), N, _stream(xq)))
    return out


def gemv_group(mats, xq, x_scale, x_sum, want_dot=True, want_y=True, out=None):
    """Decode matmul (N <= 64 quantised tokens) of every (packed, w_scale) in
    ``mats`` -> [(dot | None, y | None) per matrix]."""
    N, K = _expect_tokens(xq, x_scale, x_sum)
    out = _mats_out(mats, N, K, xq.device, want_dot, want_y, out)
    _check(load().bitnet_gemv_i2s_i8_group(_mat_array(mats, out), len(mats), K, _ptr(xq),
                                           _ptr(x_scale), _ptr(x_sum), N, _stream(xq)))
    return out


def ffn_act_quant(g, u, gamma=None, eps=1e-5, out=None):
    """sqrelu(g) * u -> RMS sub-norm (gain gamma or 1, eps) -> int8 tokens for
    the down projection: fp32 g, u [N][F] (cuda) -> (xq, s, xsum)."""
    import torch
    if g.dtype != torch.float32 or u.dtype != torch.float32 or g.shape != u.shape or g.dim() != 2:
        raise TypeError("g and u must be float32 tensors of the same 2-D shape")
    N, F = g.shape
    if u.device != g.device:
        raise ValueError("g and u must be on the same device")
    if gamma is not None:
        _expect(gamma, "gamma", torch.float32, (F,), g.device)
    if out is None:
        out = (torch.empty((N, F), dtype=torch.int8, device=g.device),
               torch.empty((N,), dtype=torch.float32, device=g.device),
               torch.empty((N,), dtype=torch.int32, device=g.device))
    xq, xs, xsum = out
    _expect(xq, "xq", torch.int8, (N, F), g.device)
    _expect(xs, "x_scale", torch.float32, (N,), g.device)
    _expect(xsum, "x_sum", torch.int32, (N,), g.device)
    _check(load().bitnet_ffn_act_quant_i8(_ptr(g), _ptr(u), _ptr(gamma), float(eps), N, F,
                                          _ptr(xq), _ptr(xs), _ptr(xsum), _stream(g)))
    return xq, xs, xsum


def ffn(x, gate, up, down, gamma=None, eps=1e-5):
    """The squared-ReLU gated FFN block on I2_S weights, as three library calls:
    bitnet_linear_i2s(x, [gate, up]) -> bitnet_ffn_act_quant_i8 -> the down
    projection (decode or prefill kernel by N).  gate/up/down are
    (packed, w_scale) pairs; x is fp32/bf16 [N][K] (cuda).
    Returns (dot, y) of the down projection."""
    outs, _ = linear(x, [gate, up])
    (_, g), (_, u) = outs
    xq, xs, xsum = ffn_act_quant(g, u, gamma, eps)
    P, ws = down
    if xq.shape[0] <= GEMV_MAX_N:
        return gemv(P, ws, xq, xs, xsum)
    return gemm(P, ws, xq, xs, xsum)


def linear(x, mats, want_dot=True, want_y=True, out=None, qout=None):
    """Linear layer step: quantise tokens x[N][K] (fp32/bf16, cuda) and multiply
    them by every (packed, w_scale) in ``mats`` -- one fused launch for N <= 2;
    for N > 2 the library quantises into ``qout`` first (allocated here if
    None), then runs the batched-decode (N <= 64) or grouped prefill kernels.

    Returns ([(dot | None, y | None) per matrix], (xq, s, xsum) | None)."""
    import torch
    if x.dim() != 2:
        raise TypeError("x must be 2-D [N][K]")
    dt = {torch.float32: F32, torch.bfloat16: BF16}.get(x.dtype)
    if dt is None:
        raise TypeError("x must be float32 or bfloat16")
    N, K = x.shape
    out = _mats_out(mats, N, K, x.device, want_dot, want_y, out)
    if qout is None and N > LINEAR_FUSED_MAX_N:
        qout = (torch.empty((N, K), dtype=torch.int8, device=x.device),
                torch.empty((N,), dtype=torch.float32, device=x.device),
                torch.empty((N,), dtype=torch.int32, device=x.device))
    xq, xs, xsum = qout if qout is not None else (None, None, None)
    if qout is not None:
        _expect(xq, "qout xq", torch.int8, (N, K), x.device)
        _expect(xs, "qout x_scale", torch.float32, (N,), x.device)
        _expect(xsum, "qout x_sum", torch.int32, (N,), x.device)
    _check(load().bitnet_linear_i2s(_ptr(x), dt, N, K, _mat_array(mats, out), len(mats),
                                    _ptr(xq), _ptr(xs), _ptr(xsum), _stream(x)))
    return out, qout


def _launch(fn, device, *args):
    """fn(*args, the device's current stream), with the device current."""
    import torch
    if device.type != "cuda":
        raise ValueError("tensor must live on the GPU")
    index = device.index
    if index == torch._C._cuda_getDevice():
        status = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(index):
            status = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    if status:
        _check(status)


def _float_code(dtype, name):
    """BITNET_F32 or BITNET_BF16."""
    import torch
    if dtype == torch.float32:
        return F32
    if dtype == torch.bfloat16:
        return BF16
    raise TypeError(f"{name} must be float32 or bfloat16, got {dtype}")


def _at(t, name, dtype, shape, device):
    """The pointer of an operand that may be None, refused before any launch if it
    is not contiguous or not what is expected."""
    if t is None:
        return None
    if t.dtype != dtype or t.shape != shape or t.device != device:
        _expect(t, name, dtype, shape, device)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def block_norm_quant(b, res=None, post_norm=False, post_gamma=None, gate=None, scale=1.0,
                     gamma=None, eps=1e-5, want_v=False, want_q=True, out=None):
    """The boundary between two blocks: norm of the block's output b[N][F]
    (``post_norm``, gain ``post_gamma``), times ``gate`` ([F] or [N][F]) and
    ``scale``, added to the residual stream ``res``; then the norm (gain
    ``gamma``) whose tokens the next block takes, as int8 for the matmuls
    (``want_q``) and / or as they are (``want_v``).

    b and res are fp32 or bf16; h and v have res's type (b's without a res).
    ``out``: (h, v, (xq, s, xsum)) to write into, None where not wanted; h may
    be ``res`` itself.  Returns (h | None, v | None, (xq, s, xsum) | None)."""
    import torch
    if b.dim() != 2:
        raise TypeError("b must be 2-D [N][F]")
    shape, dev = b.shape, b.device
    N, F = shape
    f32 = torch.float32
    stream = b.dtype if res is None else res.dtype
    bd, sd = _float_code(b.dtype, "b"), _float_code(stream, "res")
    if post_gamma is not None and not post_norm:
        raise ValueError("post_gamma without post_norm")
    gate_rows = gate is not None and gate.dim() != 1
    if not b.is_contiguous():
        raise ValueError("b must be contiguous")
    res_at = _at(res, "res", stream, shape, dev)
    h = v = q = h_at = v_at = xq_at = xs_at = xsum_at = None
    if out is None:     # tensors made here need no checks
        if res is not None:
            h = torch.empty_like(res)
            h_at = h.data_ptr()
        if want_v:
            v = torch.empty_like(b, dtype=stream)
            v_at = v.data_ptr()
        if want_q:
            xs = torch.empty(N, dtype=f32, device=dev)
            xq, xsum = torch.empty_like(b, dtype=torch.int8), torch.empty_like(xs, dtype=torch.int32)
            q = (xq, xs, xsum)
            xq_at, xs_at, xsum_at = xq.data_ptr(), xs.data_ptr(), xsum.data_ptr()
    else:
        h, v, q = out
        if h is not None and res is None:
            raise ValueError("h without res")
        h_at, v_at = _at(h, "h", stream, shape, dev), _at(v, "v", stream, shape, dev)
        if q is not None:
            xq, xs, xsum = q
            if xq is None or xs is None or xsum is None:
                raise ValueError("xq, x_scale and x_sum come together")
            xq_at, xs_at = _at(xq, "xq", torch.int8, shape, dev), _at(xs, "x_scale", f32, (N,), dev)
            xsum_at = _at(xsum, "x_sum", torch.int32, (N,), dev)
    _launch(load().bitnet_block_norm_quant_i8, dev, b.data_ptr(), bd,
            1 if post_norm else 0, _at(post_gamma, "post_gamma", f32, (F,), dev),
            _at(gate, "gate", f32, shape if gate_rows else (F,), dev), F if gate_rows else 0, scale,
            res_at, h_at, sd, _at(gamma, "gamma", f32, (F,), dev), eps, N, F, v_at, xq_at, xs_at,
            xsum_at)
    return h, v, q


def kv4_cache(n_pages, n_kv_heads, head_dim, device="cuda"):
    """A 4-bit key/value cache of ``n_pages`` pages of 64 tokens (uninitialised:
    what no token was written to is never used), uint8 [n_pages][n_kv_heads]
    [72 * head_dim]."""
    import torch
    if head_dim not in (64, 128, 256):
        raise ValueError(f"head_dim={head_dim} must be 64, 128 or 256")
    return torch.empty((n_pages, n_kv_heads, 72 * head_dim), dtype=torch.uint8, device=device)


def _kv4_batch(cache, table, kv_len, q_start, rows=True):
    """Cache and sequences (without ``rows``: no q_start) -> (bitnet_kv4_batch, kv heads, head_dim)."""
    import torch
    i32 = torch.int32
    if cache.dim() != 3 or cache.dtype != torch.uint8 or cache.shape[2] % 72:
        raise TypeError("cache must be uint8 [n_pages][n_kv_heads][72 * head_dim]")
    dev = cache.device
    if table.dim() != 2:
        raise ValueError("table must be 2-D [n_seqs][max_pages]")
    B, P = table.shape
    n_pages, heads, rec = cache.shape
    if kv_len is None or (rows and q_start is None):
        raise ValueError("kv_len and q_start are required")
    at = _at(table, "table", i32, (B, P), dev)
    lens, start = _at(kv_len, "kv_len", i32, (B,), dev), _at(q_start, "q_start", i32, (B + 1,), dev)
    return KV4Batch(_ptr(cache), n_pages, heads, rec // 72, at, P, lens, start, B), heads, rec // 72


def _rows(t, name, heads, dim, device):
    """[N][heads][dim] with any stride between tokens -> that stride."""
    if t.dim() != 3 or t.shape[1] != heads or t.shape[2] != dim:
        raise ValueError(f"{name} must have shape [N][{heads}][{dim}], got {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, the cache on {device}")
    n, (token, head, one) = t.shape[0], t.stride()
    if n and (one != 1 or (heads > 1 and head != dim)):
        raise ValueError(f"{name}: the values of a token must be contiguous")
    return token if n > 1 else heads * dim


def kv4_append(cache, table, kv_len, q_start, k, v):
    """Quantise keys and values k, v [N][n_kv_heads][head_dim] (fp32 or bf16, any
    stride between tokens) into the cache, as the last positions of their
    sequences: rows q_start[b] .. q_start[b+1] - 1 end at position kv_len[b] - 1
    (kv_len counts them already).  table [B][max_pages], kv_len [B], q_start
    [B+1]: int32 on the device, read when the kernel runs."""
    batch, heads, dim = _kv4_batch(cache, table, kv_len, q_start)
    if v.dtype != k.dtype or v.shape != k.shape:
        raise TypeError("k and v must have the same shape and type")
    dev = cache.device
    _launch(load().bitnet_kv4_append, dev, batch, k.data_ptr(), _rows(k, "k", heads, dim, dev),
            v.data_ptr(), _rows(v, "v", heads, dim, dev), _float_code(k.dtype, "k"), k.shape[0])


_put = object.__setattr__


class _Fixed:
    """An object whose attributes stay as they were made: its descriptor is made once."""
    __slots__ = ()

    def __setattr__(self, name, value):
        raise AttributeError(f"{type(self).__name__}.{name} cannot be changed: make another")


class Rotary(_Fixed):
    """Rotary positions: turns per position of each pair of channels (``turns`` [rot / 2]
    int64 on the device, 64-bit fractions of a turn), the pairs (i, i + rot / 2) or
    (2 i, 2 i + 1) (``interleaved``) of the first rot channels, and what cosine and sine
    are multiplied by.  rotary_plan makes one from a base."""
    __slots__ = ("turns", "interleaved", "magnitude", "_plan")

    def __init__(self, turns, interleaved=False, magnitude=1.0):
        import torch
        if turns.dim() != 1 or turns.dtype != torch.int64 or not turns.is_contiguous():
            raise TypeError("turns must be a contiguous 1-D int64 tensor")
        interleaved, magnitude = bool(interleaved), float(magnitude)
        _put(self, "turns", turns)
        _put(self, "interleaved", interleaved)
        _put(self, "magnitude", magnitude)
        _put(self, "_plan", RotaryPlan(turns.data_ptr(), 2 * turns.shape[0], interleaved, magnitude))


def rotary_plan(rot, base=10000.0, factor=1.0, length=0, low=1.0, high=32.0, freqs=None,
                interleaved=False, magnitude=1.0, device="cuda"):
    """A Rotary of ``rot`` channels: base^(-2 i / rot) radians per position, or ``freqs``
    [rot / 2] (any numbers) in its place.  For contexts longer than trained for: ``factor``
    divides every frequency (positions interpolated), or with ``length`` (the context
    trained for) those that turn fewer than ``low`` times over it, none that turns more
    than ``high`` times, and a share of it in between."""
    import math

    import torch
    if rot < 2 or rot % 2:
        raise ValueError(f"rot={rot} must be even and positive")
    freqs = [base ** (-2 * i / rot) for i in range(rot // 2)] if freqs is None else [float(f) for f in freqs]
    if len(freqs) != rot // 2 or not all(math.isfinite(f) for f in freqs):
        raise ValueError(f"freqs must be {rot // 2} finite numbers")
    if not factor > 0 or not length >= 0 or (length and not low < high):
        raise ValueError("factor must be positive, length not negative and low below high")
    turns = []
    for f in freqs:
        kept = 0.0
        if length:
            kept = min(max((length * abs(f) / (2 * math.pi) - low) / (high - low), 0.0), 1.0)
        f *= kept + (1 - kept) / factor
        t = int(f / (2 * math.pi) * 2.0 ** 64) % 2 ** 64     # whole turns fall away
        turns.append(t - 2 ** 64 if t >= 2 ** 63 else t)
    return Rotary(torch.tensor(turns, dtype=torch.int64, device=device), interleaved, magnitude)


def _plan_of(plan, device):
    if plan.turns.device != device:
        raise ValueError(f"the plan's turns are on {plan.turns.device}, the rows on {device}")
    return plan._plan


def rotary(x, plan, positions, inverse=False, out=None):
    """Rows x [N][heads][dim] (fp32 or bf16, any stride between tokens; dim a multiple of 8)
    turned to ``positions`` [N] (int32, on the device) by a Rotary; ``inverse`` turns back,
    which is the gradient's way.  ``out``: rows like x's, or x itself."""
    import torch
    if x.dim() != 3:
        raise ValueError("x must be 3-D [N][heads][dim]")
    N, heads, dim = x.shape
    dev = x.device
    code, stride = _float_code(x.dtype, "x"), _rows(x, "x", heads, dim, dev)
    if out is None:
        out = torch.empty((N, heads, dim), dtype=x.dtype, device=dev)
        to = heads * dim
    else:
        if out.dtype != x.dtype or out.shape != x.shape:
            raise TypeError("out must have x's shape and type")
        to = _rows(out, "out", heads, dim, dev)
    _launch(load().bitnet_rotary, dev, _plan_of(plan, dev), x.data_ptr(), stride, code, N, heads, dim,
            _at(positions, "positions", torch.int32, (N,), dev), 1 if inverse else 0, out.data_ptr(), to)
    return out


def rotary_kv4_append(cache, table, kv_len, q_start, q, k, v, plan, offset=None, out=None):
    """q [N][n_heads][head_dim] and k [N][n_kv_heads][head_dim] turned to their positions by a
    Rotary, k and v appended to the cache as kv4_append does: one launch.  A row's position is
    its place in the cache plus ``offset`` [B] (int32, on the device) of its sequence.
    Returns the turned q, in ``out`` if given (which may be q); rows of no sequence are left
    as they are there."""
    import torch
    batch, kv_heads, dim = _kv4_batch(cache, table, kv_len, q_start)
    if q.dim() != 3:
        raise ValueError("q must be 3-D [N][n_heads][head_dim]")
    if v.dtype != k.dtype or v.shape != k.shape:
        raise TypeError("k and v must have the same shape and type")
    if q.dtype != k.dtype or q.shape[0] != k.shape[0]:
        raise TypeError("q and k must have the same type and as many rows")
    N, heads, dev = q.shape[0], q.shape[1], cache.device
    at_q, at_k, at_v = _rows(q, "q", heads, dim, dev), _rows(k, "k", kv_heads, dim, dev), _rows(v, "v", kv_heads, dim, dev)
    if out is None:
        out = torch.empty((N, heads, dim), dtype=q.dtype, device=dev)
        to = heads * dim
    else:
        if out.dtype != q.dtype or out.shape != q.shape:
            raise TypeError("out must have q's shape and type")
        to = _rows(out, "out", heads, dim, dev)
    _launch(load().bitnet_rotary_kv4_append, dev, batch, _plan_of(plan, dev), q.data_ptr(), at_q,
            out.data_ptr(), to, heads, k.data_ptr(), at_k, v.data_ptr(), at_v, _float_code(q.dtype, "q"),
            N, _at(offset, "offset", torch.int32, (batch.n_seqs,), dev))
    return out


def kv4_read(cache, table, kv_len, q_start, n, dtype=None, out=None):
    """What the cache holds at the last positions of each sequence (q_start as
    in kv4_append, n rows in all) -> (k, v) [n][n_kv_heads][head_dim], fp32 or
    bf16 (``dtype``).  ``out``: (k, v) to write into, one of them may be None."""
    import torch
    batch, heads, dim = _kv4_batch(cache, table, kv_len, q_start)
    dev, shape = cache.device, (n, heads, dim)
    if out is None:
        dtype = dtype or torch.float32
        k = torch.empty(shape, dtype=dtype, device=dev)
        v = torch.empty_like(k)
        out, at = (k, v), (k.data_ptr(), v.data_ptr())
    else:
        k, v = out
        if k is None and v is None:
            raise ValueError("k and v are both None")
        dtype = dtype or (k if k is not None else v).dtype
        at = _at(k, "k", dtype, shape, dev), _at(v, "v", dtype, shape, dev)
    _launch(load().bitnet_kv4_read, dev, batch, *at, _float_code(dtype, "out"), n)
    return out


def attn_kv4(q, cache, table, kv_len, q_start, scale=None, window=0, sinks=0, max_kv=None,
             out=None, workspace=None):
    """Causal attention of q [N][n_heads][head_dim] (fp32 or bf16, any stride
    between tokens) over the 4-bit cache, for single tokens and prompts: row
    q_start[b] + i stands at position kv_len[b] - (q_start[b+1] - q_start[b]) + i
    and sees the positions up to its own; with a ``window`` the last ``window``
    of them and the first ``sinks``.  A row that sees nothing gets zeros, one with a
    NaN or an infinity in its q NaN.

    scale: 1 / sqrt(head_dim) if None.  max_kv: the longest kv_len expected (the
    table's capacity if None); it tunes the launch and changes no result beyond
    rounding.  workspace: a uint8 tensor for calls that must not allocate
    (attn_kv4_workspace bytes); one for each call that may run at once.
    Returns out [N][n_heads][head_dim] in q's type."""
    import torch
    batch, kv_heads, dim = _kv4_batch(cache, table, kv_len, q_start)
    if q.dim() != 3:
        raise ValueError("q must be 3-D [N][n_heads][head_dim]")
    L, dev, dtype, shape = load(), cache.device, q.dtype, q.shape
    N, heads = shape[0], shape[1]
    code, stride = _float_code(dtype, "q"), _rows(q, "q", heads, dim, dev)
    most = KV4_PAGE * batch.max_pages
    max_kv = most if max_kv is None else min(max_kv, most)
    need = L.bitnet_attn_kv4_workspace(batch.n_seqs, N, heads, kv_heads, dim, max_kv, window, sinks)
    if need < 0:
        raise BitnetError(E_SHAPE, L.bitnet_last_error().decode(errors="replace"))
    if out is None:
        out = torch.empty(shape, dtype=dtype, device=dev)
        at = out.data_ptr()
    else:
        at = _at(out, "out", dtype, shape, dev)
    if workspace is None:
        if need:
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    elif workspace.dtype != torch.uint8 or workspace.device != dev or workspace.numel() < need:
        raise ValueError(f"workspace must be {need} bytes of uint8 on {dev}")
    _launch(L.bitnet_attn_kv4, dev, batch, q.data_ptr(), stride, code, N, heads,
            dim ** -0.5 if scale is None else scale, window, sinks, max_kv,
            at, None if workspace is None else _ptr(workspace),
            0 if workspace is None else workspace.numel())
    return out


def attn_kv4_workspace(n_seqs, n, n_heads, n_kv_heads, head_dim, max_kv, window=0, sinks=0):
    """Bytes of workspace that attn_kv4 takes for these sizes: not fewer for a smaller
    max_kv, so ask with the call's own (attn_kv4 takes at most the table's capacity)."""
    need = load().bitnet_attn_kv4_workspace(n_seqs, n, n_heads, n_kv_heads, head_dim, max_kv,
                                            window, sinks)
    if need < 0:
        raise BitnetError(E_SHAPE, load().bitnet_last_error().decode(errors="replace"))
    return need


def kv4_weights(cache):
    """The array that kv4_weigh and kv4_evict keep beside a cache: fp32 [n_pages][n_kv_heads]
    [64], uninitialised (a token's weight begins at 0 in the call that weighs its row)."""
    import torch
    return torch.empty((*cache.shape[:2], KV4_PAGE), dtype=torch.float32, device=cache.device)


def kv4_weigh(weights, q, cache, table, kv_len, q_start, decay=1.0, scale=None, window=0, sinks=0,
              max_kv=None, out=None, workspace=None):
    """Adds what each cached token is weighed with by the attention of q's rows (the softmax
    weights of attn_kv4 with the same arguments, summed over the rows and the heads that
    share a kv head) to ``decay`` times its weight so far; tokens of the rows themselves begin
    at 0.  ``weights`` fp32 [n_pages][n_kv_heads][64] is updated, or with ``out`` left as it is (None will do with
    a decay of 0).  Sequences without rows keep theirs.  workspace: as in attn_kv4
    (kv4_weigh_workspace bytes).  Long chunks are quicker in a call of their own than among many
    single tokens.  Returns out."""
    import torch
    batch, kv_heads, dim = _kv4_batch(cache, table, kv_len, q_start)
    if q.dim() != 3:
        raise ValueError("q must be 3-D [N][n_heads][head_dim]")
    L, dev = load(), cache.device
    N, heads = q.shape[0], q.shape[1]
    code, stride = _float_code(q.dtype, "q"), _rows(q, "q", heads, dim, dev)
    shape = (*cache.shape[:2], KV4_PAGE)
    at = _at(weights, "weights", torch.float32, shape, dev)
    if out is None:
        out = weights
    to = _at(out, "out", torch.float32, shape, dev)
    most = KV4_PAGE * batch.max_pages
    max_kv = most if max_kv is None else min(max_kv, most)
    need = L.bitnet_kv4_weigh_workspace(batch.n_seqs, N, heads, kv_heads, dim, max_kv, window, sinks)
    if need < 0:
        raise BitnetError(E_SHAPE, L.bitnet_last_error().decode(errors="replace"))
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    elif workspace.dtype != torch.uint8 or workspace.device != dev or workspace.numel() < need:
        raise ValueError(f"workspace must be {need} bytes of uint8 on {dev}")
    _launch(L.bitnet_kv4_weigh, dev, batch, q.data_ptr(), stride, code, N, heads,
            dim ** -0.5 if scale is None else scale, window, sinks, max_kv, at, decay, to,
            _ptr(workspace), workspace.numel())
    return out


def kv4_weigh_workspace(n_seqs, n, n_heads, n_kv_heads, head_dim, max_kv, window=0, sinks=0):
    """Bytes of workspace that kv4_weigh takes for these sizes, with the call's own max_kv."""
    need = load().bitnet_kv4_weigh_workspace(n_seqs, n, n_heads, n_kv_heads, head_dim, max_kv, window, sinks)
    if need < 0:
        raise BitnetError(E_SHAPE, load().bitnet_last_error().decode(errors="replace"))
    return need


def kv4_evict(cache, weights, table, kv_len, new_table, keep, sinks=0, recent=0, out=None,
              workspace=None):
    """Copies what is kept of each sequence to the pages of ``new_table`` [B][new_max_pages], kv
    head by kv head: its first ``sinks`` tokens, its last ``recent`` ones, and of the others
    those of the largest weight, ``keep`` in all (or all there are), in order, weights and all.  The new pages must be
    none that a sequence of the call has; the old ones are left as they are, to be handed out again.

    Returns (new_len [B], index [B][n_kv_heads][keep]: the places that the tokens had, -1
    behind the last), int32, in ``out`` if given (other memory than kv_len).  The step after goes on with new_table and new_len; its
    positions are kv_len - new_len further on (rotary_kv4_append's offset).  workspace: as in
    attn_kv4 (kv4_evict_workspace bytes, none for tables of fewer than 320 pages, which
    take fewer launches too)."""
    import torch
    i32, dev = torch.int32, cache.device
    if weights is None or new_table is None or new_table.dim() != 2:
        raise ValueError("weights and a 2-D new_table are required")
    batch, heads, _ = _kv4_batch(cache, table, kv_len, None, rows=False)
    B = batch.n_seqs
    at_w = _at(weights, "weights", torch.float32, (*cache.shape[:2], KV4_PAGE), dev)
    if out is None:
        new_len = torch.empty(B, dtype=i32, device=dev)
        index = torch.empty((B, heads, max(keep, 0)), dtype=i32, device=dev)
    else:
        new_len, index = out
    L, ws = load(), None
    need = L.bitnet_kv4_evict_workspace(B, heads, batch.max_pages)
    if need > 0:
        if workspace is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
        elif workspace.dtype != torch.uint8 or workspace.device != dev or workspace.numel() < need:
            raise ValueError(f"workspace must be {need} bytes of uint8 on {dev}")
        ws = _ptr(workspace)
    _launch(L.bitnet_kv4_evict, dev, batch, at_w,
            _at(new_table, "new_table", i32, (B, new_table.shape[1]), dev), new_table.shape[1], keep, sinks, recent,
            _at(new_len, "new_len", i32, (B,), dev), _at(index, "index", i32, (B, heads, keep), dev),
            ws, max(need, 0))
    return new_len, index


def kv4_evict_workspace(n_seqs, n_kv_heads, max_pages):
    """Bytes of workspace that kv4_evict takes for n_seqs tables of max_pages entries."""
    need = load().bitnet_kv4_evict_workspace(n_seqs, n_kv_heads, max_pages)
    if need < 0:
        raise BitnetError(E_SHAPE, load().bitnet_last_error().decode(errors="replace"))
    return need


# groups of a block's 128 channels, by the last two sizes of the steps in either order
_W4_PER_BLOCK = {s: p for p in (1, 2, 4) for s in ((16, p), (p, 16))}


class W4Matrix(_Fixed):
    """A matrix of 4-bit weights [M][K] as pack_w4 lays it out: ``codes`` uint8
    [ceil(M/16)][K/128][64][16], ``steps`` fp16 [ceil(M/16)][K/128][16][128/group] or, group by
    group, [ceil(M/16)][K/128][128/group][16], and the number of its ``rows`` M (all of the tiles' if None)."""
    __slots__ = ("codes", "steps", "rows", "k", "group", "_desc")

    def __init__(self, codes, steps, rows=None):
        import torch
        shape, groups = codes.shape, steps.shape
        if codes.dtype != torch.uint8 or len(shape) != 4 or shape[2] != 64 or shape[3] != 16:
            raise TypeError("codes must be uint8 [tiles][K/128][64][16]")
        per = _W4_PER_BLOCK.get(tuple(groups[2:]))
        if steps.dtype != torch.float16 or per is None or groups[:2] != shape[:2]:
            raise TypeError("steps must be float16 [tiles][K/128][16][128/group] or [tiles][K/128][128/group][16]")
        if steps.device != codes.device or not codes.is_contiguous() or not steps.is_contiguous():
            raise ValueError("codes and steps must be contiguous, on one device")
        tiles, k, group = shape[0], 128 * shape[1], 128 // per
        rows = 16 * tiles if rows is None else rows
        if not 16 * (tiles - 1) < rows <= 16 * tiles and (tiles or rows):
            raise ValueError(f"{rows} rows are not {tiles} tiles of 16")
        _put(self, "codes", codes)
        _put(self, "steps", steps)
        _put(self, "rows", rows)
        _put(self, "k", k)
        _put(self, "group", group)
        _put(self, "_desc", W4Desc(codes.data_ptr(), steps.data_ptr(), rows, k,
                                   group | (W4_BY_GROUP if groups[3] == 16 else 0)))

    @classmethod
    def empty(cls, rows, k, group=64, device="cuda"):
        """An uninitialised matrix, for pack_w4's ``out``."""
        import torch
        if k % 128 or group not in (32, 64, 128):
            raise ValueError(f"K={k} must be a multiple of 128 and group={group} 32, 64 or 128")
        tiles = -(-rows // 16)
        return cls(torch.empty((tiles, k // 128, 64, 16), dtype=torch.uint8, device=device),
                   torch.empty((tiles, k // 128, 16, 128 // group), dtype=torch.float16, device=device), rows)


def _w4_out(out, shape, group, device):
    if out is None:
        return W4Matrix.empty(*shape, group, device)
    if (out.rows, out.k, out.group) != (*shape, group) or out.codes.device != device:
        raise ValueError(f"out must be a {shape[0]} x {shape[1]} matrix of group {group} on {device}")
    return out


def pack_w4(w, group=64, out=None):
    """fp32 or bf16 weights w[M][K] (cuda) -> a W4Matrix: 4 bits a weight and a step for each
    ``group`` (32, 64 or 128) channels of a row."""
    if w.dim() != 2 or not w.is_contiguous():
        raise TypeError("w must be 2-D [M][K] and contiguous")
    code = _float_code(w.dtype, "w")
    out = _w4_out(out, tuple(w.shape), group, w.device)
    _launch(load().bitnet_pack_w4, w.device, w.data_ptr(), code, out._desc)
    return out


def pack_w4_codes(w, steps, out=None):
    """Weights that are 4-bit already: int8 w[M][K] in -8 .. 7 and fp16 steps [M][K/group] ->
    a W4Matrix."""
    import torch
    if w.dim() != 2 or w.dtype != torch.int8 or not w.is_contiguous():
        raise TypeError("w must be int8 [M][K] and contiguous")
    M, K = w.shape
    if steps.dim() != 2 or steps.shape[1] == 0 or K % steps.shape[1]:
        raise ValueError("steps must be 2-D [M][K/group]")
    group = K // steps.shape[1]
    at = _at(steps, "steps", torch.float16, (M, K // group), w.device)
    out = _w4_out(out, (M, K), group, w.device)
    _launch(load().bitnet_pack_w4_codes, w.device, w.data_ptr(), at, out._desc)
    return out


def w4_rows(mat, ids=None, dtype=None, out=None):
    """Rows ``ids`` (int32, on the device; all rows if None) of a W4Matrix as fp32 or bf16
    [n][K]: an embedding's lookup.  An id outside the matrix gives zeros."""
    import torch
    dev = mat.codes.device
    n = mat.rows if ids is None else ids.shape[0]
    if out is None:
        dtype = dtype or torch.float32
        out = torch.empty((n, mat.k), dtype=dtype, device=dev)
    at = _at(out, "out", dtype or out.dtype, (n, mat.k), dev)
    _launch(load().bitnet_w4_rows, dev, mat._desc, _at(ids, "ids", torch.int32, (n,), dev), n, at,
            _float_code(out.dtype, "out"))
    return out


def linear_w4(x, mat, out=None, workspace=None):
    """x [N][K] (fp32 or bf16, any N) times a W4Matrix -> y [N][M] fp32.  workspace: a uint8
    tensor for calls that must not allocate (linear_w4_workspace bytes, often none);
    one for each call that may run at once."""
    import torch
    if x.dim() != 2 or x.shape[1] != mat.k:
        raise ValueError(f"x must be 2-D [N][{mat.k}], got {tuple(x.shape)}")
    N, dev = x.shape[0], mat.codes.device
    at = _at(x, "x", x.dtype, x.shape, dev)
    if out is None:
        out = torch.empty((N, mat.rows), dtype=torch.float32, device=dev)
        to = out.data_ptr()
    else:
        to = _at(out, "out", torch.float32, (N, mat.rows), dev)
    L, ws = load(), None
    need = _w4_need(N, mat.rows, mat.k)
    if need > 0:
        if workspace is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
        elif workspace.dtype != torch.uint8 or workspace.device != dev or workspace.numel() < need:
            raise ValueError(f"workspace must be {need} bytes of uint8 on {dev}")
        ws = _ptr(workspace)
    _launch(L.bitnet_linear_w4, dev, at, _float_code(x.dtype, "x"), N, mat._desc, to, ws, max(need, 0))
    return out


@functools.lru_cache(maxsize=1024)
def _w4_need(n, rows, k):   # of the sizes alone
    return load().bitnet_linear_w4_workspace(n, rows, k)


def linear_w4_workspace(n, rows, k):
    """Bytes of workspace that linear_w4 takes for n tokens and a matrix of rows x k."""
    need = load().bitnet_linear_w4_workspace(n, rows, k)
    if need < 0:
        raise BitnetError(E_SHAPE, load().bitnet_last_error().decode(errors="replace"))
    return need


def _matmuls(tokens, mats):
    """y of every (packed, w_scale) in ``mats`` for fp32 / bf16 tokens [N][K] or
    quantised ones (xq, s, xsum)."""
    x = tokens[0] if isinstance(tokens, tuple) else tokens
    if x.shape[0] == 0:     # nothing to multiply, and empty tensors have no address
        return [y for _, y in _mats_out(mats, 0, x.shape[1], x.device, False, True, None)]
    if not isinstance(tokens, tuple):
        return [y for _, y in linear(tokens, mats, want_dot=False)[0]]
    group = gemv_group if x.shape[0] <= GEMV_MAX_N else gemm_group
    return [y for _, y in group(mats, *tokens, want_dot=False)]


def attn_block(tokens, q, k, v, o, cache, table, kv_len, q_start, gamma=None, eps=1e-5, rotary=None,
               window=0, sinks=0, max_kv=None, offset=None, weights=None, decay=1.0):
    """The attention block on I2_S weights and a 4-bit cache: q, k and v projections
    (one grouped launch) -> keys and values appended to the cache -> attention over
    it -> RMS sub-norm (gain gamma or 1) and int8 tokens -> the o projection.

    tokens: fp32 / bf16 [N][hidden], or quantised as block_norm_quant gives them.
    q, k, v, o: (packed, w_scale) pairs; head_dim and the kv heads are the cache's.
    rotary: a Rotary (positions as in rotary_kv4_append, with its ``offset``), or called
    with q [N][n_heads][head_dim] and k [N][n_kv_heads][head_dim] (fp32) and returns them with
    their positions applied.
    weights: what kv4_weigh keeps of each cached token, updated by this step's attention
    (with ``decay``).  The rest as in attn_kv4.
    Returns y [N][hidden] fp32, the block's output for the next block_norm_quant; rows
    of no sequence (padding) have no attention, and their y is unspecified."""
    if offset is not None and not isinstance(rotary, Rotary):
        raise ValueError("offset without a Rotary")
    yq, yk, yv = _matmuls(tokens, [q, k, v])
    N, kv_heads, dim = yq.shape[0], cache.shape[1], cache.shape[2] // 72
    qh = yq.view(N, yq.shape[1] // dim, dim)
    kh, vh = yk.view(N, kv_heads, dim), yv.view(N, kv_heads, dim)
    if isinstance(rotary, Rotary):
        qh = rotary_kv4_append(cache, table, kv_len, q_start, qh, kh, vh, rotary, offset, out=qh)
    else:
        if rotary is not None:
            qh, kh = rotary(qh, kh)
        kv4_append(cache, table, kv_len, q_start, kh, vh)
    if weights is not None:
        kv4_weigh(weights, qh, cache, table, kv_len, q_start, decay, window=window, sinks=sinks, max_kv=max_kv)
    a = attn_kv4(qh, cache, table, kv_len, q_start, window=window, sinks=sinks, max_kv=max_kv)
    _, _, inner = block_norm_quant(a.view(yq.shape), gamma=gamma, eps=eps)
    return _matmuls(inner, [o])[0]
