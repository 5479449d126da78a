"""echo_quantize_tokens, echo_gemm_int8 and echo_linear_int8 on the GPU against
plain forms: the sums are exact integers, so every comparison is bit for bit
(codes, scales, fp32 outputs, and bf16 outputs as torch rounds them)."""
import numpy as np
import pytest
import torch

import _block_ref as ref
from _helpers import DEV, say

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def echo():
    from error_feedback_quant_amd import echo as e
    assert torch.cuda.is_available()
    return e


def matrix(rows, cols, ld, dtype, values, offset=0, fill=7):
    """[rows, cols] view with row distance ld, `offset` elements into an allocation that ends with the last row."""
    n = offset + (max(rows, 1) - 1) * ld + cols
    buf = torch.full((n,), fill, dtype=dtype, device=DEV)
    v = torch.as_strided(buf, (rows, cols), (ld, 1), offset)
    if values is not None:
        v.copy_(values.to(dtype))
    return buf, v


def codes(rng, rows, cols):
    return torch.from_numpy(rng.integers(-128, 128, (rows, cols), dtype=np.int64).astype(np.int8))


def untouched(buf, view, fill=7):
    """Everything outside the view still holds the fill."""
    mask = torch.ones_like(buf, dtype=torch.bool)
    torch.as_strided(mask, view.shape, view.stride(), view.storage_offset()).fill_(False)
    assert bool((buf[mask] == fill).all())


def same_bits(got, want):
    got, want = got.cpu(), want.cpu()
    assert got.shape == want.shape and got.dtype == want.dtype
    if got.is_floating_point():
        nan = torch.isnan(want)
        assert torch.equal(torch.isnan(got), nan)
        got, want = got.masked_fill(nan, 0), want.masked_fill(nan, 0)
    assert torch.equal(got, want), f"{int((got != want).sum())} of {got.numel()} differ"


QUANT = [(T, K, pad, off) for T, K in [(1, 1), (1, 4096), (3, 7), (64, 1024), (33, 1001), (5, 131071), (700, 200), (2, 16384)]
         for pad, off in [(0, 0), (16, 0), (3, 1)]]


@pytest.mark.parametrize("T,K,pad,off", QUANT)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_quantize_tokens(echo, T, K, pad, off, dt):
    say("quantize", T, K, pad, off, dt)
    rng = np.random.default_rng(T * 1000 + K)
    v = torch.from_numpy(rng.standard_normal((T, K)).astype(np.float32))
    v[T // 2] *= 1e-30 if T % 2 else 20
    v[-1, K // 2] = 100.0
    _, x = matrix(T, K, K + pad, DT[dt], v, off)
    qb, q = matrix(T, K, K + pad, torch.int8, None, off)
    sb, s = matrix(1, T, T, torch.float32, None, off)
    echo.echo_quantize_tokens(x, K + pad, echo.BF16 if dt == "bf16" else echo.F32, T, K, q, K + pad, s)
    torch.cuda.synchronize()
    wq, ws = ref.quantize_tokens(x.float().cpu().numpy())
    same_bits(q, torch.from_numpy(wq))
    same_bits(s[0], torch.from_numpy(ws))
    untouched(qb, q)
    untouched(sb, s)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_quantize_edge_tokens(echo, dt):
    """Zeros, values below the floor of the scale, halves, the largest values,
    an infinity, a NaN; and tokens around them keep their own results."""
    say("quantize edges", dt)
    K = 300
    rng = np.random.default_rng(3)
    v = torch.from_numpy(rng.standard_normal((12, K)).astype(np.float32))
    v[1] = 0
    v[2] = 1e-38
    v[3] = torch.arange(K) % 255 - 127.0
    v[3, 0] = 127.0
    v[4] = 3e38
    v[5, 17] = float("inf")
    v[6, K - 1] = float("nan")
    v[7, 0] = float("-inf")
    v[8] = -0.0
    v[9] = torch.arange(K).float() * 0.5 - 63.5
    v[9, 0] = 127.0
    _, x = matrix(12, K, K, DT[dt], v)
    q = torch.empty(12, K, dtype=torch.int8, device=DEV)
    s = torch.empty(12, device=DEV)
    echo.echo_quantize_tokens(x, K, echo.BF16 if dt == "bf16" else echo.F32, 12, K, q, K, s)
    torch.cuda.synchronize()
    wq, ws = ref.quantize_tokens(x.float().cpu().numpy())
    same_bits(q, torch.from_numpy(wq))
    same_bits(s, torch.from_numpy(ws))
    assert bool(torch.isnan(s[5:8]).all()) and not bool(q[5:8].any())


def test_quantize_no_columns(echo):
    """K = 0 still gives every token its (smallest) scale."""
    s = torch.full((5,), 7.0, device=DEV)
    echo.echo_quantize_tokens(None, 0, echo.F32, 5, 0, None, 0, s)
    torch.cuda.synchronize()
    same_bits(s, torch.from_numpy(ref.quantize_tokens(np.zeros((5, 0), np.float32))[1]))


def run_gemm(echo, M, N, K, ydt, bias, padx=0, padw=0, pady=0, off=0, seed=0, ones=False):
    rng = np.random.default_rng(seed + M * 7 + N * 3 + K)
    xv, wv = codes(rng, M, K), codes(rng, N, K)
    if ones:                      # the largest possible sum
        xv.fill_(-128)
        wv.fill_(-128)
    sx = torch.from_numpy(rng.uniform(0.001, 0.1, M).astype(np.float32))
    sw = torch.from_numpy(rng.uniform(0.001, 0.1, N).astype(np.float32))
    b = torch.from_numpy(rng.standard_normal(N).astype(np.float32)) if bias else None
    _, x = matrix(M, K, K + padx, torch.int8, xv, off, fill=101)
    _, w = matrix(N, K, K + padw, torch.int8, wv, off, fill=-99)
    yb, y = matrix(M, N, N + pady, DT[ydt], None, off)
    echo.echo_gemm_int8(x, K + padx, sx.to(DEV), w, K + padw, sw.to(DEV), b.to(DEV) if bias else None, M, N, K,
                        y, N + pady, echo.BF16 if ydt == "bf16" else echo.F32)
    torch.cuda.synchronize()
    want = torch.from_numpy(ref.gemm_int8(xv.numpy(), sx.numpy(), wv.numpy(), sw.numpy(), b.numpy() if bias else None))
    same_bits(y, want.to(DT[ydt]))
    untouched(yb, y)


SHAPES = [(1, 1, 1), (1, 64, 64), (1, 4096, 512), (1, 1000, 4097), (2, 33, 100), (5, 31, 15), (7, 17, 16), (8, 520, 1024),
          (16, 256, 256), (17, 300, 129), (31, 65, 640), (33, 130, 1000), (48, 100, 64), (64, 1024, 1024), (65, 63, 127),
          (100, 257, 128), (128, 128, 384), (129, 255, 383), (200, 500, 1001), (256, 256, 256), (257, 513, 640),
          (300, 1000, 255), (512, 768, 1152), (777, 1001, 3583), (1025, 260, 96), (260, 1030, 2048)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("layout", ["plain", "padded", "odd"])
def test_gemm_int8(echo, M, N, K, layout):
    say("gemm int8", M, N, K, layout)
    up16 = -K % 16
    if layout == "plain":
        run_gemm(echo, M, N, K, "f32", False)
        run_gemm(echo, M, N, K, "bf16", True)
    elif layout == "padded":      # rows at multiples of 16 bytes whatever K is
        run_gemm(echo, M, N, K, "bf16", False, padx=up16, padw=up16 + 16, pady=-N % 8)
        run_gemm(echo, M, N, K, "f32", True, padx=up16 + 32, padw=up16, pady=-N % 8 + 8)
    else:
        run_gemm(echo, M, N, K, "bf16", True, padx=3, padw=1, pady=5, off=1)
        run_gemm(echo, M, N, K, "f32", False, padx=up16, padw=1, pady=1, off=3)


@pytest.mark.parametrize("M,N", [(1, 40), (20, 48), (70, 80), (300, 260)])
def test_gemm_int8_longest_sum(echo, M, N):
    """K at its limit with every code -128: the sum is 2^14 * 131071, 16384 below 2^31."""
    say("gemm longest sum", M, N)
    run_gemm(echo, M, N, 131071, "f32", False, padx=1, padw=1, ones=True)
    run_gemm(echo, M, N, 131071, "f32", True)


@pytest.mark.parametrize("M,N,K", [(4096, 4096, 3584), (2048, 4096, 4096), (1, 4096, 4096), (64, 4096, 1024), (300, 8192, 4096),
                                   (3000, 2050, 4096)])
def test_gemm_int8_workload_shapes(echo, M, N, K):
    """Whole outputs against float64 products on the GPU (exact: below 2^53)."""
    say("gemm workload", M, N, K)
    g = torch.Generator(device=DEV).manual_seed(M + N)
    x = torch.randint(-127, 128, (M, K), generator=g, device=DEV, dtype=torch.int8)
    w = torch.randint(-127, 128, (N, K), generator=g, device=DEV, dtype=torch.int8)
    sx, sw = torch.rand(M, generator=g, device=DEV), torch.rand(N, generator=g, device=DEV)
    want = ((x.double() @ w.double().t().contiguous()).float() * sx[:, None]) * sw
    for dt, kind in ((torch.float32, echo.F32), (torch.bfloat16, echo.BF16)):
        y = torch.full((M, N), 7.0, dtype=dt, device=DEV)
        echo.echo_gemm_int8(x, K, sx, w, K, sw, None, M, N, K, y, N, kind)
        torch.cuda.synchronize()
        same_bits(y, want.to(dt))


@pytest.mark.parametrize("M,N", [(4096, 4096), (2048, 4096), (1024, 4096), (512, 4096), (200, 4100), (100, 4096), (40, 8200)])
@pytest.mark.parametrize("K", [128, 300, 1155])
@pytest.mark.parametrize("pad", [0, 1, 4])
def test_gemm_int8_every_tile(echo, M, N, K, pad):
    """Sizes that fill the chip with each tile, with rows at multiples of 16
    bytes (pad 0), at words and at odd places; whole stages and a rest of K."""
    say("gemm tiles", M, N, K, pad)
    g = torch.Generator(device=DEV).manual_seed(M + N + K)
    ld = -(-K // 16) * 16 + pad
    x = torch.randint(-128, 128, (M, ld), generator=g, device=DEV, dtype=torch.int8)[:, :K]
    w = torch.randint(-128, 128, (N, ld), generator=g, device=DEV, dtype=torch.int8)[:, :K]
    sx, sw, b = torch.rand(M, generator=g, device=DEV), torch.rand(N, generator=g, device=DEV), torch.rand(N, generator=g, device=DEV)
    want = ((x.double() @ w.double().t().contiguous()).float() * sx[:, None]) * sw + b
    y = torch.full((M, N + pad), 7.0, dtype=torch.bfloat16, device=DEV)
    echo.echo_gemm_int8(x, ld, sx, w, ld, sw, b, M, N, K, y, N + pad, echo.BF16)
    torch.cuda.synchronize()
    same_bits(y[:, :N].contiguous(), want.bfloat16())
    assert bool((y[:, N:] == 7).all())


@pytest.mark.parametrize("M", [1, 40, 300])
def test_gemm_int8_far_rows(echo, M):
    """Row distances that put operands and outputs past 2^31 elements."""
    N, K = 40, 200
    ld = (1 << 31) // (M - 1) + 1000 if M > 1 else K
    ldw = (1 << 31) // (N - 1) + 1001
    say("gemm far rows", M, ld, ldw)
    rng = np.random.default_rng(M)
    xv, wv = codes(rng, M, K), codes(rng, N, K)
    _, x = matrix(M, K, ld, torch.int8, xv)
    _, w = matrix(N, K, ldw, torch.int8, wv)
    s, t = torch.rand(M, device=DEV), torch.rand(N, device=DEV)
    yb, y = matrix(M, N, ld if M > 1 else N, torch.bfloat16, None)
    echo.echo_gemm_int8(x, ld, s, w, ldw, t, None, M, N, K, y, ld if M > 1 else N, echo.BF16)
    torch.cuda.synchronize()
    same_bits(y, torch.from_numpy(ref.gemm_int8(xv.numpy(), s.cpu().numpy(), wv.numpy(), t.cpu().numpy(), None)).bfloat16())


def test_gemm_int8_most_channels(echo):
    """More channels than one launch of the few-token form holds (2^27), three codes each."""
    N, K = (1 << 27) + 5, 3
    say("gemm most channels", N)
    g = torch.Generator(device=DEV).manual_seed(2)
    x = torch.tensor([[100, -128, 7]], dtype=torch.int8, device=DEV)
    w = torch.randint(-128, 128, (N, K), generator=g, device=DEV, dtype=torch.int8)
    sx, sw = torch.full((1,), 0.01, device=DEV), torch.rand(N, generator=g, device=DEV)
    y = torch.empty(1, N, dtype=torch.bfloat16, device=DEV)
    echo.echo_gemm_int8(x, K, sx, w, K, sw, None, 1, N, K, y, N, echo.BF16)
    torch.cuda.synchronize()
    acc = 100 * w[:, 0].int() - 128 * w[:, 1].int() + 7 * w[:, 2].int()
    same_bits(y[0], ((acc.float() * sx) * sw).bfloat16())


@pytest.mark.parametrize("M", [1, 70])
def test_gemm_int8_empty_sum_and_bad_scales(echo, M):
    """K = 0 gives the bias; a NaN scale makes its own token (or channel) NaN and no other."""
    N = 50
    say("gemm empty sum", M)
    b = torch.randn(N, device=DEV)
    one = torch.ones(max(M, N), device=DEV)
    y = torch.full((M, N), 7.0, device=DEV)
    echo.echo_gemm_int8(None, 0, one, None, 0, one, b, M, N, 0, y, N, echo.F32)
    torch.cuda.synchronize()
    same_bits(y, b.expand(M, N).contiguous())
    x = torch.randint(-127, 128, (M, 96), device=DEV, dtype=torch.int8)
    w = torch.randint(-127, 128, (N, 96), device=DEV, dtype=torch.int8)
    sx, sw = one[:M].clone(), one[:N].clone()
    sx[M // 2], sw[3] = float("nan"), float("inf")
    echo.echo_gemm_int8(x, 96, sx, w, 96, sw, None, M, N, 96, y, N, echo.F32)
    torch.cuda.synchronize()
    same_bits(y, torch.from_numpy(ref.gemm_int8(x.cpu().numpy(), sx.cpu().numpy(), w.cpu().numpy(), sw.cpu().numpy(), None)))


LINEAR = [(1, 1, 1), (1, 300, 4096), (1, 4096, 1000), (2, 50, 333), (4, 128, 64), (9, 1000, 1024), (16, 65, 3584), (27, 512, 3584),
          (40, 100, 1001), (64, 512, 1024), (130, 300, 500), (700, 1030, 640)]


@pytest.mark.parametrize("M,N,K", LINEAR)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("pad,off", [(0, 0), (5, 1)])
def test_linear_is_quantize_then_product(echo, M, N, K, dt, pad, off):
    say("linear", M, N, K, dt, pad, off)
    rng = np.random.default_rng(M + N + K)
    v = torch.from_numpy(rng.standard_normal((M, K)).astype(np.float32))
    v[0] *= 50
    if M > 2:
        v[1, 0] = float("nan")
    _, x = matrix(M, K, K + pad, DT[dt], v, off)
    wv = codes(rng, N, K)
    _, w = matrix(N, K, K + pad, torch.int8, wv, off)
    sw = torch.from_numpy(rng.uniform(0.001, 0.1, N).astype(np.float32))
    b = torch.from_numpy(rng.standard_normal(N).astype(np.float32)) if M % 2 else None
    need = echo.echo_linear_int8_workspace_bytes(M, N, K)
    ws = torch.full((need + 64,), 77, dtype=torch.uint8, device=DEV)
    wq, wsc = ref.quantize_tokens(x.float().cpu().numpy())
    want = torch.from_numpy(ref.gemm_int8(wq, wsc, wv.numpy(), sw.numpy(), None if b is None else b.numpy()))
    for ydt, kind in ((torch.float32, echo.F32), (torch.bfloat16, echo.BF16)):
        yb, y = matrix(M, N, N + pad, ydt, None, off)
        echo.echo_linear_int8(x, K + pad, echo.BF16 if dt == "bf16" else echo.F32, w, K + pad, sw.to(DEV),
                              None if b is None else b.to(DEV), M, N, K, y, N + pad, kind, ws, need)
        torch.cuda.synchronize()
        same_bits(y, want.to(ydt))
        untouched(yb, y)
    assert bool((ws[need:] == 77).all())


@pytest.mark.parametrize("M", [1, 600])
def test_linear_on_another_stream_and_in_a_graph(echo, M):
    """The call runs on the stream it is given, and a captured call gives the
    eager call's bits on every replay (new inputs and eager work between)."""
    N, K = 320, 512
    say("linear stream and graph", M)
    w = torch.randint(-127, 128, (N, K), device=DEV, dtype=torch.int8)
    sw = torch.rand(N, device=DEV)
    x = torch.randn(M, K, device=DEV)
    ws = torch.empty(echo.echo_linear_int8_workspace_bytes(M, N, K) + 16, dtype=torch.uint8, device=DEV)
    y = torch.empty(M, N, device=DEV)
    call = lambda out, s: echo.echo_linear_int8(x, K, echo.F32, w, K, sw, None, M, N, K, out, N, echo.F32, ws, stream=s)  # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        x.mul_(1.5)
    call(y, side)
    torch.cuda.current_stream().wait_stream(side)
    want = torch.empty_like(y)
    call(want, None)
    torch.cuda.synchronize()
    same_bits(y, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(y, None)
    for k in range(4):
        x.copy_(torch.randn(M, K, device=DEV) * (k + 1))
        y.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        got = y.clone()
        call(want, None)
        torch.cuda.synchronize()
        same_bits(got, want)
