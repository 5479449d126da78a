"""How far the serving operators' arithmetic is off in norm, step by step in
numpy, and the limits that lie between the kernels' forms and forms that leave a
step out.  The bounds of tests/_serve_ref.py hold for every element and every
input; they are too wide to tell these forms apart."""
import numpy as np

import _serve_ref as ref

# fp32 tokens, normal values, K = 4096, any group: the kernel's form is off by
# 0.96e-7 to 1.6e-7 of y's norm, with the matrix instruction's sums rounded or cut
# after 4, 8, 16 or all 32 products; without one of its steps by 2.1e-7 or more.
LINEAR_LIMIT = 1.9e-7
# Attention of few rows: the error's norm against that of the 64-bit result
# rounded once to bf16.  Weights in two parts leave 2^-17 of a weight beside the
# output's 2^-9, a share of 1e-4 of the norm after squaring; scores, sums and the
# joins are good to 2^-18.  Weights in one part add what comes near the output's
# own rounding: 1.15 times and more.
ATTENTION_LIMIT = 1.05


def nearest(v):
    return v.astype(np.float32)


def cut(v):
    f = v.astype(np.float32)
    return np.where(np.abs(f.astype(np.float64)) > np.abs(v), np.nextafter(f, np.float32(0)), f)


def parts_of(x, n):
    """x as n bfloat16 parts by truncation, each of the rest before it."""
    got, rest = [], x.astype(np.float32)
    for _ in range(n):
        p = (rest.view(np.uint32) & np.uint32(0xFFFF0000)).view(np.float32)
        got.append(p.astype(np.float64))
        rest = rest - p
    return got


def linear_form(x, codes, params, group, parts=3, apart=True, centre=True, chunk=32, rounded=nearest):
    """The product of fp32 tokens with 16 + q: `parts` of x, the lower ones' sums `apart`, `centre` taken off after each 32 elements;
    a matrix instruction rounds after every `chunk` products."""
    (M, K), N = x.shape, codes.shape[0]
    assert K % group == 0
    q = 16 + ref.unpack4(codes, K).astype(np.float64)
    xp, unit = parts_of(x, parts), max(128, group)
    waves = [np.zeros((M, N), np.float32) for _ in range(8)]
    for g, k in enumerate(range(0, K, group)):
        s, z = (params[:, g, i].view(np.float16).astype(np.float64) for i in (0, 1))
        acc = [np.zeros((M, N), np.float32) for _ in range(2)]      # of the first part and of the others
        xs = [np.zeros((M, 1), np.float32) for _ in range(2)]
        for f in range(k, k + group, 32):
            for what in ("ones", "codes") + (("centre",) if centre else ()):
                sums = xs if what == "ones" else acc
                for i, p in enumerate(xp):
                    for c in range(f, f + 32, chunk):
                        t = p[:, c:c + chunk]
                        t = t @ q[:, c:c + chunk].T if what == "codes" else t.sum(1, keepdims=True) * (-24 if what == "centre" else 1)
                        at = 1 if i and apart else 0
                        sums[at] = rounded(sums[at] + t)
        a, b = (nearest(v[0].astype(np.float64) + v[1]).astype(np.float64) for v in (acc, xs))
        w = waves[k // unit % 8]
        w[:] = nearest(s * nearest(((8 if centre else -16) - z) * b + a) + w)
    y = waves[0]
    for w in waves[1:]:
        y = y + w
    return y


def linear_case(group, M, N, K):
    rng = np.random.default_rng([group, M, N, K])
    x = rng.standard_normal((M, K)).astype(np.float32)
    w = (rng.standard_normal((N, K)) * K ** -0.5).astype(np.float32)
    return x, w


def off(y, want):
    return float(np.linalg.norm(np.asarray(y, np.float64) - want) / np.linalg.norm(want))


def bf16(v):
    """Rounded to bfloat16, by way of fp32 (as the kernels' values come)."""
    w = np.asarray(v, np.float32).view(np.uint32).astype(np.uint64)
    return ((w + 0x7FFF + (w >> np.uint64(16) & np.uint64(1))) & np.uint64(0xFFFF0000)).astype(np.uint32).view(np.float32).astype(np.float64)


def attention_form(codes, scale_of_v, offset, scores, parts):
    """Outputs of rows with these scores [n, L] over v = (codes - offset) * scale_of_v ([L, D], [L], [L]): weights times v's scale as
    `parts` bfloat16 parts times codes, the offset (16 + the zero point under 16 + c, or none) taken off by unrounded weights."""
    p = np.exp(scores - scores.max(1, keepdims=True))
    w = p * scale_of_v
    held = np.zeros_like(w)
    for _ in range(parts):
        held = held + bf16(w - held)
    return bf16((held @ codes - (w * offset).sum(1, keepdims=True)) / p.sum(1, keepdims=True))


def over_rounding(out, want):
    """The error's norm against that of want's own rounding to bfloat16."""
    return float(np.linalg.norm(out - want) / np.linalg.norm(bf16(want) - want))
