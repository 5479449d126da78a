"""Plain 64-bit forms of the serving operators with error bounds, shared by
the CPU and GPU tests.

Bounds.  u = 2^-24 (fp32), B = 2^-8 (bfloat16): half a step relative to the
value.  A matrix instruction may cut instead of round, so an addition inside
one counts 2 u.  Magnitudes are carried with absolute values, so cancellation
is inside the bound.
"""
import numpy as np
import torch

U = 2.0 ** -24
BF = 2.0 ** -8
TINY = np.float32(2.0 ** -100)


def quant8(x):
    """Codes and scales of rows (last dimension) in the operator's own fp32 operations."""
    x = np.asarray(x, np.float32)
    bad = ~np.isfinite(x).all(axis=-1)
    a = np.maximum(np.abs(np.where(bad[..., None], np.float32(0), x)).max(axis=-1, initial=0).astype(np.float32), TINY)
    s = a / np.float32(127)
    q = np.rint(np.where(bad[..., None], np.float32(0), x) * (np.float32(127) / a)[..., None]).astype(np.int8)
    return q, np.where(bad, np.float32(np.nan), s)


def quant4(x):
    """Codes, scale and zero point (as binary16 bits) of groups (last
    dimension): the zero-aware quantizer in its own fp32 operations."""
    x = np.asarray(x, np.float32)
    bad = ~np.isfinite(x).all(axis=-1)
    x = np.where(bad[..., None], np.float32(0), x)
    lo, hi = np.minimum(x.min(-1, initial=0), np.float32(0)), np.maximum(x.max(-1, initial=0), np.float32(0))
    with np.errstate(over="ignore"):
        s = ((hi - lo) / np.float32(15)).astype(np.float16)
    s = np.where(s == 0, np.float16(2.0 ** -24), s)
    s = np.where(np.isinf(s), np.float16(65504), s)
    inv = np.float32(1) / s.astype(np.float32)
    z = np.clip(np.rint(-lo * inv), 0, 15).astype(np.float32) + np.float32(0)
    q = np.clip(np.rint(x * inv[..., None]) + z[..., None], 0, 15).astype(np.uint8)
    flat = hi == lo
    s, z = np.where(flat, np.float16(0), s), np.where(flat, np.float32(0), z).astype(np.float16)
    q = np.where((flat | bad)[..., None], np.uint8(0), q)
    return q, np.where(bad, np.uint16(0x7E00), s.view(np.uint16)), np.where(bad, np.uint16(0), z.view(np.uint16))


def pack4(q):
    if q.shape[-1] % 2:
        q = np.concatenate([q, np.zeros_like(q[..., :1])], -1)
    return q[..., 0::2] | (q[..., 1::2] << 4)


def unpack4(b, n):
    return np.stack([b & 15, b >> 4], -1).reshape(*b.shape[:-1], -1)[..., :n]


def quant_groups(x, group):
    """Packed codes [T, ceil(K / 2)] and parameters [T, groups, 2] (uint16) of rows."""
    T, K = x.shape
    codes, params = np.zeros((T, K), np.uint8), np.zeros((T, -(-K // group), 2), np.uint16)
    for g, k in enumerate(range(0, K, group)):
        codes[:, k:k + group], params[:, g, 0], params[:, g, 1] = quant4(x[:, k:k + group])
    return pack4(codes), params


def linear4(x, codes, params, group, bias):
    """y in float64 and the bound of its fp32 evaluation: in a group the sums
    of x (16 + q) and of x run at most 3 * group deep with terms of up to
    31 |x| and |x|, the latter times 16 + z; joining adds the groups and 8
    waves."""
    M, K = x.shape
    q = unpack4(codes, K).astype(np.float64)
    y, tol = np.zeros((M, codes.shape[0])), np.zeros((M, codes.shape[0]))
    depth = params.shape[1] + 16
    for g, k in enumerate(range(0, K, group)):
        s = params[:, g, 0].view(np.float16).astype(np.float64)
        z = params[:, g, 1].view(np.float16).astype(np.float64)
        xs = x[:, k:k + group]
        part = (xs @ (q[:, k:k + group] - z[:, None]).T) * s
        mag = np.abs(xs) @ (16 + q[:, k:k + group]).T + np.abs(xs).sum(1)[:, None] * (16 + z)
        y += part
        tol += (2 * 3 * group + 4) * U * mag * s + depth * U * mag * s
    if bias is not None:
        y = y + bias
        tol = tol + U * np.abs(y)
    return y, tol + 2.0 ** -140


def values(kind, codes, scale, width):
    """A cache's rows in float64: codes [..., width] (or packed), scale [...] (or [..., 2] binary16)."""
    if kind == "bf16":
        return codes.double()
    if kind == "i8":
        return codes.double() * scale.double()[..., None]
    n = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)[..., :width].double()
    return (n - scale[..., 1:].double()) * scale[..., :1].double()


def attention(q, k, v, sees, scale, offset=None):
    """One sequence and one head: q [n, D], k and v [L, D] in float64, sees
    [n, L].  Returns out, lse and their bounds before out is rounded.

    offset: for 4-bit codes (16 + z) * s of k and of v ([L], [L]), whose
    products are summed and taken off again.
    Scores: D products, each exact, summed in fp32, then three roundings.  A
    score off by dx changes a weight by its share dx, and the weights' sum by
    as much.  A weight times v's scale is rounded to bfloat16; sums over L
    tokens, the joins and the division follow."""
    n, D = q.shape
    L = k.shape[0]
    if L == 0 or n == 0:
        return (torch.zeros(n, D, dtype=torch.double), torch.full((n,), -torch.inf, dtype=torch.double),
                torch.zeros(n, D, dtype=torch.double), torch.zeros(n, dtype=torch.double))
    x = torch.mm(q, k.t().contiguous()) * scale
    mag = torch.mm(q.abs(), k.abs().t().contiguous()) * abs(scale)
    vmag = v.abs()
    if offset is not None:
        mag = mag + 2 * q.abs().sum(1)[:, None] * offset[0] * abs(scale)
    dx = torch.where(sees, (2 * D + 8) * U * mag, 0.0).amax(1)
    x = x.masked_fill(~sees, -torch.inf)
    lse = torch.logsumexp(x, 1)
    empty = ~sees.any(1)
    p = torch.exp(x - torch.where(empty, 0.0, lse)[:, None]).masked_fill(~sees, 0.0)
    v = torch.where(sees.any(0)[:, None], v, 0.0)                # what nobody sees may be anything
    vmag = torch.where(sees.any(0)[:, None], vmag, 0.0)
    out, omag = torch.mm(p, v), torch.mm(p, vmag)
    off = torch.mm(p, torch.where(sees.any(0), offset[1], 0.0)[:, None]) if offset is not None else 0.0
    sums = (2 * L + 64) * U
    tol = omag * (1.01 * BF + 2 * dx[:, None] + sums) + off * 2 * (sums + 2 * U)
    return out, lse, tol + 2.0 ** -120, dx + (L + 64) * U + 4 * U * lse.abs().nan_to_num(posinf=0.0, neginf=0.0)


def outside(got, want, tol):
    """Where a tensor is not the rounding, to its type, of any value within
    tol of want (rounding keeps order)."""
    lo, hi, g = (want - tol).to(got.dtype).double(), (want + tol).to(got.dtype).double(), got.double()
    return ~((lo <= g) & (g <= hi))
