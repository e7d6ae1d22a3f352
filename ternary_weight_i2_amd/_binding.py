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


class KV4Batch(ctypes.Structure):
    """Mirror of bitnet_kv4_batch."""
    _fields_ = [("cache", ctypes.c_void_p), ("n_pages", ctypes.c_int64),
                ("n_kv_heads", ctypes.c_int64), ("head_dim", ctypes.c_int64),
                ("table", ctypes.c_void_p), ("max_pages", ctypes.c_int64),
                ("kv_len", ctypes.c_void_p), ("q_start", ctypes.c_void_p),
                ("n_seqs", ctypes.c_int64)]


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


def _kv4_batch(cache, table, kv_len, q_start):
    """Cache and sequences -> (bitnet_kv4_batch, kv heads, head_dim)."""
    import torch
    i32 = torch.int32
    if cache.dim() != 3 or cache.dtype != torch.uint8 or cache.shape[2] % 72:
        raise TypeError("cache must be uint8 [n_pages][n_kv_heads][72 * head_dim]")
    dev = cache.device
    if table.dim() != 2:
        raise ValueError("table must be 2-D [n_seqs][max_pages]")
    B, P = table.shape
    n_pages, heads, rec = cache.shape
    if kv_len is None or q_start is None:
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
               window=0, sinks=0, max_kv=None):
    """The attention block on I2_S weights and a 4-bit cache: q, k and v projections
    (one grouped launch) -> keys and values appended to the cache -> attention over
    it -> RMS sub-norm (gain gamma or 1) and int8 tokens -> the o projection.

    tokens: fp32 / bf16 [N][hidden], or quantised as block_norm_quant gives them.
    q, k, v, o: (packed, w_scale) pairs; head_dim and the kv heads are the cache's.
    rotary: called with q [N][n_heads][head_dim] and k [N][n_kv_heads][head_dim]
    (fp32), returns them with their positions applied.  The rest as in attn_kv4.
    Returns y [N][hidden] fp32, the block's output for the next block_norm_quant; rows
    of no sequence (padding) have no attention, and their y is unspecified."""
    yq, yk, yv = _matmuls(tokens, [q, k, v])
    N, kv_heads, dim = yq.shape[0], cache.shape[1], cache.shape[2] // 72
    qh = yq.view(N, yq.shape[1] // dim, dim)
    kh, vh = yk.view(N, kv_heads, dim), yv.view(N, kv_heads, dim)
    if rotary is not None:
        qh, kh = rotary(qh, kh)
    kv4_append(cache, table, kv_len, q_start, kh, vh)
    a = attn_kv4(qh, cache, table, kv_len, q_start, window=window, sinks=sinks, max_kv=max_kv)
    _, _, inner = block_norm_quant(a.view(yq.shape), gamma=gamma, eps=eps)
    return _matmuls(inner, [o])[0]
