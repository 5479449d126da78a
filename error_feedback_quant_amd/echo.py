"""Thin ctypes binding of libecho (include/echo.h), same call names.

Argument marshalling only: every step of the path runs in the HIP kernels of
libecho.so.  Tensors are passed by device pointer (``tensor.data_ptr()``);
PyTorch provides device memory and streams.  A non-zero status raises
``EchoError``.  Importing this module loads libecho.so and raises if it has
not been built -- there is no fallback path.
"""
from __future__ import annotations

import ctypes
import os
import re
from ctypes import POINTER, Structure, c_char_p, c_float, c_int, c_int64, c_size_t, c_uint16, c_void_p

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libecho.so")
HEADER = os.path.join(os.path.dirname(PKG), "include", "echo.h")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is not built; run __graft_entry__.build() (hipcc, gfx950) first")
# torch brings its own HIP runtime (libamdhip64, SONAME libamdhip64.so.7) and
# owns the device memory and streams passed to libecho, so it must be loaded
# first: libecho.so then binds to that same runtime instead of pulling a
# second copy into the process.
import torch  # noqa: E402,F401

_lib = ctypes.CDLL(LIB_PATH)

OK, EINVAL, EALIGN, EUNSUP, ESHAPE, EHIP, ETOOBIG = 0, -1, -2, -3, -4, -5, -6
OUT_F32, OUT_BF16 = 0, 1
F32, BF16, I8 = 0, 1, 2
ERR_NEGATED = 1
QUANT_NAIVE, QUANT_SYMMETRIC = 2, 4
X_ALL = 8
QUANT_MSE = 16
QUANTS = {"zero_aware": 0, "naive": QUANT_NAIVE, "symmetric": QUANT_SYMMETRIC, "mse": QUANT_MSE}
MAX_P = 8


class EchoError(RuntimeError):
    def __init__(self, fn, rc):
        msg = _lib.echo_status_str(rc).decode()
        if rc == EHIP:
            msg += f" (hipError {_lib.echo_last_hip_error()})"
        super().__init__(f"{fn}: {msg} [{rc}]")
        self.rc = rc


class SimArgs(Structure):
    """Mirror of echo_sim_args."""
    _fields_ = [
        ("P", c_int), ("bits", c_int), ("group", c_int), ("tiles", c_int),
        ("out_dtype", c_int), ("ef", c_int), ("quant", c_int), ("alpha", c_float), ("beta", c_float),
        ("n", c_int64),
        ("x", c_void_p * MAX_P), ("comp", c_void_p * MAX_P), ("slow", c_void_p * MAX_P),
        ("err", c_void_p * MAX_P), ("out", c_void_p * MAX_P),
        ("workspace", c_void_p), ("workspace_bytes", c_size_t),
    ]


class NormArgs(Structure):
    """Mirror of echo_norm_args."""
    _fields_ = [
        ("T", c_int64), ("H", c_int64),
        ("ld_x", c_int64), ("ld_r", c_int64), ("ld_r_out", c_int64), ("ld_h", c_int64), ("ld_gate", c_int64),
        ("gate_tokens", c_int64),
        ("x_dtype", c_int), ("r_dtype", c_int), ("w_dtype", c_int), ("h_dtype", c_int), ("post", c_int),
        ("eps", c_float), ("res_scale", c_float), ("block_scale", c_float),
        ("x", c_void_p), ("r", c_void_p), ("w_post", c_void_p), ("w_pre", c_void_p), ("gate", c_void_p),
        ("r_out", c_void_p), ("h", c_void_p), ("h_scale", c_void_p),
    ]


class NormGrads(Structure):
    """Mirror of echo_norm_grads."""
    _fields_ = [
        ("ld_dh", c_int64), ("ld_dr_out", c_int64), ("ld_dx", c_int64), ("ld_dr", c_int64), ("ld_dgate", c_int64),
        ("dh_dtype", c_int),
        ("dh", c_void_p), ("dr_out", c_void_p), ("dx", c_void_p), ("dr", c_void_p),
        ("dw_post", c_void_p), ("dw_pre", c_void_p), ("dgate", c_void_p),
        ("workspace", c_void_p), ("workspace_bytes", c_size_t),
    ]


_lib.echo_status_str.restype = c_char_p
_lib.echo_status_str.argtypes = [c_int]
_lib.echo_last_hip_error.restype = c_int
_lib.echo_last_hip_error.argtypes = []
_lib.echo_quantize_ef.restype = c_int
_lib.echo_quantize_ef.argtypes = [c_void_p, c_void_p, c_int64, c_int, c_int, c_int64, c_int64, c_int, c_int,
                                  c_void_p, c_void_p, c_void_p, c_int, c_void_p]
_lib.echo_reduce_segment.restype = c_int
_lib.echo_reduce_segment.argtypes = [c_void_p, c_void_p, c_void_p, c_void_p, c_int, c_int, c_int64, c_int64,
                                     c_int64, c_int, c_int, c_void_p, c_void_p, c_void_p, c_int, c_void_p]
_lib.echo_gather_dequant.restype = c_int
_lib.echo_gather_dequant.argtypes = [c_void_p, c_void_p, c_int64, c_int64, c_int64, c_int, c_int, c_int,
                                     c_void_p, c_int, c_void_p]
_lib.echo_compensate.restype = c_int
_lib.echo_compensate.argtypes = [c_void_p, c_void_p, c_void_p, c_int64, c_float, c_float, c_void_p]
_lib.echo_gemm_quantize_ef.restype = c_int
_lib.echo_gemm_quantize_ef.argtypes = [c_void_p, c_void_p, c_int64, c_int64, c_int64, c_void_p, c_int, c_int,
                                       c_int, c_int, c_void_p, c_void_p, c_void_p, c_void_p, c_int, c_void_p]
_lib.echo_allreduce_sim_workspace_bytes.restype = c_size_t
_lib.echo_allreduce_sim_workspace_bytes.argtypes = [c_int, c_int64, c_int, c_int]
_lib.echo_allreduce_sim.restype = c_int
_lib.echo_allreduce_sim.argtypes = [POINTER(SimArgs), c_void_p, c_int]
_lib.echo_allreduce_sim_noalloc.restype = c_int
_lib.echo_allreduce_sim_noalloc.argtypes = [POINTER(SimArgs), c_void_p]
_lib.echo_noalloc_scratch_bytes.restype = c_size_t
_lib.echo_noalloc_scratch_bytes.argtypes = []
_lib.echo_quantize_tokens.restype = c_int
_lib.echo_quantize_tokens.argtypes = [c_void_p, c_int64, c_int, c_int64, c_int64, c_void_p, c_int64, c_void_p, c_void_p]
_lib.echo_gemm_int8.restype = c_int
_lib.echo_gemm_int8.argtypes = [c_void_p, c_int64, c_void_p, c_void_p, c_int64, c_void_p, c_void_p, c_int64, c_int64,
                                c_int64, c_void_p, c_int64, c_int, c_void_p]
_lib.echo_linear_int8_workspace_bytes.restype = c_size_t
_lib.echo_linear_int8_workspace_bytes.argtypes = [c_int64, c_int64, c_int64]
_lib.echo_linear_int8.restype = c_int
_lib.echo_linear_int8.argtypes = [c_void_p, c_int64, c_int, c_void_p, c_int64, c_void_p, c_void_p, c_int64, c_int64,
                                  c_int64, c_void_p, c_int64, c_int, c_void_p, c_size_t, c_void_p]
_lib.echo_block_norm.restype = c_int
_lib.echo_block_norm.argtypes = [POINTER(NormArgs), c_void_p]
_lib.echo_block_norm_backward_workspace_bytes.restype = c_size_t
_lib.echo_block_norm_backward_workspace_bytes.argtypes = [c_int64, c_int64]
_lib.echo_block_norm_backward.restype = c_int
_lib.echo_block_norm_backward.argtypes = [POINTER(NormArgs), POINTER(NormGrads), c_void_p]


def lib():
    return _lib


def declared_functions():
    """Function names declared in include/echo.h."""
    text = open(HEADER).read()
    return sorted(set(re.findall(r"^\s*(?:const\s+)?[a-z_0-9]+\s*\*?\s*(echo_[a-z_0-9]+)\s*\(", text, re.M)))


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


# torch's handle of a device's current stream; building a torch.cuda.Stream
# for it costs 2.7 us, a third of a small call
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_gpu_seen = False


def _stream(s):
    if s is None:
        global _gpu_seen
        if not _gpu_seen:
            if not torch.cuda.is_available():
                return None
            _gpu_seen = True
        if _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(s, int):
        return s
    return s.cuda_stream


def _check(fn, rc):
    if rc != OK:
        raise EchoError(fn, rc)


def echo_quantize_ef(x, comp, n, P, rank, tile_begin, tile_len, bits, group, codes, params, err,
                     flags=0, stream=None):
    _check("echo_quantize_ef", _lib.echo_quantize_ef(
        _ptr(x), _ptr(comp), n, P, rank, tile_begin, tile_len, bits, group, _ptr(codes), _ptr(params),
        _ptr(err), flags, _stream(stream)))


def echo_gemm_quantize_ef(a, w, M, N, K, comp, P, rank, bits, group, codes, params, err, x_out, flags=0,
                          stream=None):
    _check("echo_gemm_quantize_ef", _lib.echo_gemm_quantize_ef(
        _ptr(a), _ptr(w), M, N, K, _ptr(comp), P, rank, bits, group, _ptr(codes), _ptr(params), _ptr(err),
        _ptr(x_out), flags, _stream(stream)))


def echo_reduce_segment(own_x, own_comp, peer_codes, peer_params, P, owner, n, tile_begin, tile_len, bits,
                        group, sum_codes, sum_params, own_err, flags=0, stream=None):
    pc = (c_void_p * max(P, 1))(*[_ptr(t) for t in peer_codes])
    pp = (c_void_p * max(P, 1))(*[_ptr(t) for t in peer_params])
    _check("echo_reduce_segment", _lib.echo_reduce_segment(
        _ptr(own_x), _ptr(own_comp), pc, pp, P, owner, n, tile_begin, tile_len, bits, group,
        _ptr(sum_codes), _ptr(sum_params), _ptr(own_err), flags, _stream(stream)))


def echo_gather_dequant(sum_codes, sum_params, n, tile_begin, tile_len, P, bits, group, out, out_dtype,
                        stream=None):
    _check("echo_gather_dequant", _lib.echo_gather_dequant(
        _ptr(sum_codes), _ptr(sum_params), n, tile_begin, tile_len, P, bits, group, _ptr(out), out_dtype,
        _stream(stream)))


def echo_compensate(err, comp_next, slow, n, alpha, beta, stream=None):
    _check("echo_compensate", _lib.echo_compensate(
        _ptr(err), _ptr(comp_next), _ptr(slow), n, alpha, beta, _stream(stream)))


def echo_allreduce_sim_workspace_bytes(P, n, bits, group=128):
    return int(_lib.echo_allreduce_sim_workspace_bytes(P, n, bits, group))


def make_sim_args(xs, outs, workspace, bits=4, group=128, tiles=1, out_dtype=OUT_F32, ef=False,
                  alpha=1.0, beta=0.0, comps=None, slows=None, errs=None, workspace_bytes=None,
                  quant="zero_aware"):
    """Fill an echo_sim_args from lists of tensors (one per simulated rank)."""
    P = len(xs)
    a = SimArgs()
    a.P, a.bits, a.group, a.tiles, a.out_dtype, a.ef = P, bits, group, tiles, out_dtype, 1 if ef else 0
    a.quant = QUANTS[quant]
    a.alpha, a.beta = alpha, beta
    a.n = xs[0].numel() if P else 0
    for r in range(P):
        a.x[r] = _ptr(xs[r])
        a.out[r] = _ptr(outs[r])
        a.comp[r] = _ptr(comps[r]) if comps is not None else None
        a.slow[r] = _ptr(slows[r]) if slows is not None else None
        a.err[r] = _ptr(errs[r]) if errs is not None else None
    a.workspace = _ptr(workspace)
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    a.workspace_bytes = workspace_bytes
    return a


def echo_allreduce_sim(args: SimArgs, streams=None):
    """streams: None (torch's current stream only) or a list of torch streams / handles."""
    if streams is None:
        arr, ns = (c_void_p * 1)(_stream(None)), 1
    else:
        arr, ns = (c_void_p * len(streams))(*[_stream(s) for s in streams]), len(streams)
    _check("echo_allreduce_sim", _lib.echo_allreduce_sim(ctypes.byref(args), arr, ns))


def echo_allreduce_sim_noalloc(args: SimArgs, stream=None):
    """The allocation-free call: args.workspace is ignored; every stage runs
    on `stream` (a torch stream or handle; None = torch's current stream)."""
    _check("echo_allreduce_sim_noalloc", _lib.echo_allreduce_sim_noalloc(ctypes.byref(args), _stream(stream)))


def echo_noalloc_scratch_bytes() -> int:
    return int(_lib.echo_noalloc_scratch_bytes())


# ---------------------------------------------------------- block operators --

_DTYPES = {torch.float32: F32, torch.bfloat16: BF16, torch.int8: I8}


def echo_quantize_tokens(x, ldx, x_dtype, T, K, codes, ldq, scales, stream=None):
    _check("echo_quantize_tokens", _lib.echo_quantize_tokens(
        _ptr(x), ldx, x_dtype, T, K, _ptr(codes), ldq, _ptr(scales), _stream(stream)))


def echo_gemm_int8(x, ldx, sx, w, ldw, sw, bias, M, N, K, y, ldy, y_dtype, stream=None):
    _check("echo_gemm_int8", _lib.echo_gemm_int8(
        _ptr(x), ldx, _ptr(sx), _ptr(w), ldw, _ptr(sw), _ptr(bias), M, N, K, _ptr(y), ldy, y_dtype, _stream(stream)))


def echo_linear_int8_workspace_bytes(M, N, K) -> int:
    return int(_lib.echo_linear_int8_workspace_bytes(M, N, K))


def echo_linear_int8(x, ldx, x_dtype, w, ldw, sw, bias, M, N, K, y, ldy, y_dtype, workspace, workspace_bytes=None,
                     stream=None):
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check("echo_linear_int8", _lib.echo_linear_int8(
        _ptr(x), ldx, x_dtype, _ptr(w), ldw, _ptr(sw), _ptr(bias), M, N, K, _ptr(y), ldy, y_dtype, _ptr(workspace),
        workspace_bytes, _stream(stream)))


_FLOATS = (F32, BF16)


def _refuse(t, shape, what, kinds):
    want = " or ".join(str(d) for d, k in _DTYPES.items() if k in kinds)
    raise ValueError(f"{what}: {tuple(t.shape)} {t.dtype} strides {t.stride()}, expected {tuple(shape)} of {want} in "
                     "rows of contiguous elements")


def _rows(t, shape, what, kinds):
    """(pointer, row distance, type) of a matrix of contiguous rows; the C side cannot see a tensor's shape."""
    ld = t.stride()
    kind = _DTYPES.get(t.dtype)
    if t.shape != shape or kind not in kinds or (ld[1] != 1 and shape[1] > 1):
        _refuse(t, shape, what, kinds)
    return t.data_ptr(), ld[0], kind


def _vector(t, n, what, kind):
    if t.numel() != n or t.dim() != 1 or _DTYPES.get(t.dtype) != kind or not t.is_contiguous():
        _refuse(t, (n,), what, (kind,))
    return t.data_ptr()


def make_norm_args(x, r=None, r_out=None, h=None, h_scale=None, post=True, w_post=None, w_pre=None, gate=None,
                   gate_tokens=0, res_scale=1.0, block_scale=1.0, eps=1e-5):
    """Fill an echo_norm_args from tensors: x, r, r_out and h are [T, H] in
    contiguous rows (an 8-bit h may be wider), w_post and w_pre [H], gate
    [ceil(T / gate_tokens), H].  It can be kept and used again while the
    tensors live."""
    shape = x.shape
    T, H = shape
    px, ld_x, kx = _rows(x, shape, "x", _FLOATS)
    pr = ld_r = po = ld_o = ph = ld_h = pg = ld_g = ps = 0
    kr, kh = kx, F32
    if r is not None:
        pr, ld_r, kr = _rows(r, shape, "r", _FLOATS)
        if r_out is not None:
            po, ld_o, _ = _rows(r_out, shape, "r_out", (kr,))
    elif r_out is not None:
        po, ld_o, kr = _rows(r_out, shape, "r_out", _FLOATS)
    if h is not None:
        if h.dtype == torch.int8:
            n, wide = h.shape
            if wide < H:
                _refuse(h, shape, "h", (I8,))
            ph, ld_h, kh = _rows(h, (n, wide) if n == T else shape, "h", (I8,))
            if h_scale is not None:
                ps = _vector(h_scale, T, "h_scale", F32)
        else:
            ph, ld_h, kh = _rows(h, shape, "h", _FLOATS)
    w = w_post if w_post is not None else w_pre if w_pre is not None else gate
    kw = F32 if w is None else _DTYPES.get(w.dtype)
    if kw not in _FLOATS:
        raise ValueError(f"weights of {w.dtype}")
    pp = _vector(w_post, H, "w_post", kw) if w_post is not None else 0
    pw = _vector(w_pre, H, "w_pre", kw) if w_pre is not None else 0
    if gate is not None:
        if gate_tokens < 1:
            raise ValueError("a gate needs gate_tokens >= 1")
        gate_tokens = min(gate_tokens, max(T, 1))          # a field of 64 bits
        pg, ld_g, _ = _rows(gate, (-(-T // gate_tokens), H), "gate", (kw,))
    else:
        gate_tokens = 0
    return NormArgs(T, H, ld_x, ld_r, ld_o, ld_h, ld_g, gate_tokens, kx, kr, kw, kh, 1 if post else 0, eps, res_scale,
                    block_scale, px, pr, pp, pw, pg, po, ph, ps)


def make_norm_grads(dh=None, dr_out=None, dx=None, dr=None, dw_post=None, dw_pre=None, dgate=None, workspace=None,
                    workspace_bytes=None):
    """Fill an echo_norm_grads from tensors, shaped as in make_norm_args.
    Whether they fit its arguments (shape, types of dx, dr and dr_out, rows of
    dgate) is checked by echo_block_norm_backward."""
    first = dh if dh is not None else dr_out if dr_out is not None else dx if dx is not None else dr
    shape = None if first is None else first.shape
    H = 0 if shape is None else shape[1]
    ph = ld_h = pu = ld_u = px = ld_x = pr = ld_r = pg = ld_g = 0
    kh, kx, ku, kr, rows = F32, None, None, None, None
    if dh is not None:
        ph, ld_h, kh = _rows(dh, shape, "dh", _FLOATS)
    if dr_out is not None:
        pu, ld_u, ku = _rows(dr_out, shape, "dr_out", _FLOATS)
    if dx is not None:
        px, ld_x, kx = _rows(dx, shape, "dx", _FLOATS)
    if dr is not None:
        pr, ld_r, kr = _rows(dr, shape, "dr", _FLOATS)
    pp = _vector(dw_post, H, "dw_post", F32) if dw_post is not None else 0
    pw = _vector(dw_pre, H, "dw_pre", F32) if dw_pre is not None else 0
    if dgate is not None:
        rows = dgate.shape[0]
        pg, ld_g, _ = _rows(dgate, (rows, H), "dgate", (F32,))
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    g = NormGrads(ld_h, ld_u, ld_x, ld_r, ld_g, kh, ph, pu, px, pr, pp, pw, pg, _ptr(workspace), workspace_bytes)
    g.fits = (shape, kx, ku, kr, rows)
    return g


def echo_block_norm(args: NormArgs, stream=None):
    _check("echo_block_norm", _lib.echo_block_norm(ctypes.byref(args), _stream(stream)))


def echo_block_norm_backward_workspace_bytes(T, H) -> int:
    return int(_lib.echo_block_norm_backward_workspace_bytes(T, H))


def echo_block_norm_backward(args: NormArgs, grads: NormGrads, stream=None):
    shape, kx, ku, kr, rows = getattr(grads, "fits", (None,) * 5)      # set by make_norm_grads
    if ((shape is not None and shape != (args.T, args.H)) or kx not in (None, args.x_dtype)
            or ku not in (None, args.r_dtype) or kr not in (None, args.r_dtype)
            or (rows is not None and rows != (-(-args.T // args.gate_tokens) if args.gate else 0))):
        raise ValueError("the gradients' shapes or types do not fit the forward call's arguments")
    _check("echo_block_norm_backward", _lib.echo_block_norm_backward(
        ctypes.byref(args), ctypes.byref(grads), _stream(stream)))
