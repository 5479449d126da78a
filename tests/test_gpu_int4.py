"""The 4-bit layer on the GPU: the group quantizer bit for bit, the product
against 64 bits within derived bounds."""
import numpy as np
import pytest
import torch

import _serve_ref as ref
from _helpers import DEV, say
from error_feedback_quant_amd import echo

pytestmark = pytest.mark.gpu
KINDS = {torch.bfloat16: echo.BF16, torch.float32: echo.F32}


def rows(rng, n, k, pad, dtype, scale=1.0):
    v = torch.from_numpy((rng.standard_normal((n, k + pad)) * scale).astype(np.float32)).to(dtype)
    return v.to(DEV)[:, :k]


def quantize(x, group, pad=0):
    """Codes and parameters in buffers whose rest is marked, checked for writes outside the rows."""
    T, K = x.shape
    nb, ng = (K + 1) // 2, -(-K // group)
    codes = torch.full((T, nb + pad), 0xA5, dtype=torch.uint8, device=DEV)
    params = torch.full((T, ng + pad, 2), -7.0, dtype=torch.float16, device=DEV)
    echo.echo_quantize_groups(x, x.stride(0), KINDS[x.dtype], T, K, group, codes, nb + pad, params, ng + pad)
    torch.cuda.synchronize()
    assert bool((codes[:, nb:] == 0xA5).all()) and bool((params[:, ng:] == -7).all())
    return codes[:, :nb], params[:, :ng]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("group", [32, 64, 128, 256])
@pytest.mark.parametrize("T,K,pad", [(1, 1, 0), (1, 4096, 0), (3, 31, 1), (5, 257, 3), (2, 8, 8), (130, 96, 0), (7, 1000, 5),
                                     (33, 3583, 0), (2, 70001, 1)])
def test_quantize_groups(dtype, group, T, K, pad):
    say("quantize_groups", dtype, group, T, K, pad)
    rng = np.random.default_rng([group, T, K])
    x = rows(rng, T, K, pad, dtype)
    x *= torch.from_numpy(np.exp2(rng.integers(-30, 20, (T, 1)).astype(np.float32))).to(DEV).to(dtype)
    x[0, :min(K, group)] = 0
    x[-1, K // 2:] = x[-1, K // 2:].abs()
    codes, params = quantize(x, group, pad)
    want_c, want_p = ref.quant_groups(x.float().cpu().numpy(), group)
    np.testing.assert_array_equal(codes.cpu().numpy(), want_c)
    np.testing.assert_array_equal(params.contiguous().view(torch.int16).cpu().numpy().view(np.uint16), want_p)


@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan"), 3.4e38, 1e-45])
def test_quantize_groups_of_extremes(value):
    say("quantize extremes", value)
    rng = np.random.default_rng(1)
    x = rows(rng, 4, 300, 0, torch.float32)
    x[1, 70], x[2, 299] = value, -value
    codes, params = quantize(x, 64)
    want_c, want_p = ref.quant_groups(x.cpu().numpy(), 64)
    np.testing.assert_array_equal(codes.cpu().numpy(), want_c)
    np.testing.assert_array_equal(params.contiguous().view(torch.int16).cpu().numpy().view(np.uint16), want_p)


def linear(x, codes, params, group, bias, N, y_dtype, pad=0):
    M, K = x.shape
    y = torch.full((M + 1, N + pad), 77.0, dtype=y_dtype, device=DEV)
    need = echo.echo_linear_int4_workspace_bytes(M, N, K, group)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    echo.echo_linear_int4(x, x.stride(0), KINDS[x.dtype], codes, codes.stride(0), params, params.stride(0) // 2, group, bias, M, N, K,
                          y, y.stride(0), KINDS[y_dtype], ws)
    torch.cuda.synchronize()
    assert bool((y[M] == 77).all()) and bool((y[:M, N:] == 77).all())
    return y[:M, :N]


SHAPES = [(1, 4096, 4096), (1, 16, 128), (2, 1, 1), (5, 17, 33), (1, 1001, 3583), (16, 64, 256), (17, 130, 300), (13, 33, 5000),
          (31, 48, 1024), (33, 1000, 777), (64, 128, 512), (65, 40, 130), (200, 20, 96), (3, 100, 31),
          (24, 64, 512), (30, 48, 516), (40, 8200, 300), (300, 2000, 260), (20, 4000, 8400)]


@pytest.mark.parametrize("dtypes", [(torch.bfloat16, torch.bfloat16), (torch.float32, torch.float32), (torch.bfloat16, torch.float32)])
@pytest.mark.parametrize("group", [32, 64, 128, 256])
@pytest.mark.parametrize("shape", SHAPES)
def test_linear_int4(dtypes, group, shape):
    M, N, K = shape
    say("linear_int4", dtypes, group, shape)
    rng = np.random.default_rng([group, M, N, K])
    pad = (M + N) % 3
    x, w = rows(rng, M, K, pad, dtypes[0]), rows(rng, N, K, 0, torch.float32, K ** -0.5)
    bias = torch.from_numpy(rng.standard_normal(N).astype(np.float32)).to(DEV) if N % 2 else None
    codes, params = quantize(w, group, pad)
    y = linear(x, codes, params, group, bias, N, dtypes[1], pad)
    want, tol = ref.linear4(x.double().cpu().numpy(), codes.cpu().numpy(),
                            params.contiguous().view(torch.int16).cpu().numpy().view(np.uint16), group,
                            None if bias is None else bias.double().cpu().numpy())
    bad = ref.outside(y.cpu(), torch.from_numpy(want), torch.from_numpy(tol))
    assert not bool(bad.any()), (int(bad.sum()), bad.nonzero()[:4])
    again = linear(x, codes, params, group, bias, N, dtypes[1], pad)
    assert torch.equal(again.contiguous().view(torch.int16), y.contiguous().view(torch.int16))


def test_weight_rows_anywhere():
    """Rows of codes and x at odd addresses, the last one ending where its buffer ends."""
    say("odd rows")
    rng = np.random.default_rng(9)
    M, N, K, g = 3, 50, 1003, 128
    w = rows(rng, N, K, 0, torch.float32)
    c0, p0 = quantize(w, g)
    for shift in (1, 2, 3):
        flat = torch.empty(shift + (N - 1) * 503 + 502, dtype=torch.uint8, device=DEV)
        codes = flat[shift:].as_strided((N, 502), (503, 1))
        codes.copy_(c0)
        xb = torch.empty(shift + M * 1007, dtype=torch.bfloat16, device=DEV)
        x = xb[shift:].as_strided((M, K), (1007, 1))
        x.copy_(torch.from_numpy(rng.standard_normal((M, K)).astype(np.float32)))
        y = linear(x, codes, p0, g, None, N, torch.float32)
        want, tol = ref.linear4(x.double().cpu().numpy(), c0.cpu().numpy(),
                                p0.contiguous().view(torch.int16).cpu().numpy().view(np.uint16), g, None)
        assert not bool(ref.outside(y.cpu(), torch.from_numpy(want), torch.from_numpy(tol)).any()), shift


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_tokens_without_numbers(dtype):
    """A token with an infinity or a NaN is NaN throughout; the others keep their bits."""
    say("linear_int4 no numbers", dtype)
    rng = np.random.default_rng(4)
    x, w = rows(rng, 20, 500, 0, dtype), rows(rng, 40, 500, 0, torch.float32)
    codes, params = quantize(w, 128)
    clean = linear(x, codes, params, 128, None, 40, torch.float32)
    x[3, 499], x[17, 0], x[18, 200] = float("inf"), float("nan"), float("-inf")
    y = linear(x, codes, params, 128, None, 40, torch.float32)
    hit = torch.zeros(20, dtype=torch.bool, device=DEV)
    hit[[3, 17, 18]] = True
    assert bool(y[hit].isnan().all()) and torch.equal(y[~hit], clean[~hit])


@pytest.mark.parametrize("M", [3, 20, 100])
@pytest.mark.parametrize("kind", [echo.BF16, echo.F32])
def test_no_inputs_give_the_bias(M, kind):
    say("K = 0", M, kind)
    bias = torch.arange(5, dtype=torch.float32, device=DEV)
    for b, want in ((bias, bias), (None, torch.zeros_like(bias))):
        y = torch.full((M, 5), 9.0, device=DEV)
        echo.echo_linear_int4(None, 0, kind, None, 0, None, 0, 32, b, M, 5, 0, y, 5, echo.F32)
        torch.cuda.synchronize()
        assert torch.equal(y, want.expand(M, 5))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M", [24, 70])
def test_one_token_is_the_same_in_any_batch(dtype, M):
    """The split of K is one for all forms: a token's outputs have the same bits alone, in a small batch and in one that is laid out."""
    say("linear_int4 batches", dtype, M)
    rng = np.random.default_rng(M)
    x, w = rows(rng, M, 1284, 0, dtype), rows(rng, 70, 1284, 0, torch.float32)
    for group in (32, 64, 128, 256):
        codes, params = quantize(w, group)
        whole = linear(x, codes, params, group, None, 70, torch.float32)
        for m in (1, 16, 20):
            part = linear(x[:m].contiguous(), codes, params, group, None, 70, torch.float32)
            assert torch.equal(part, whole[:m]), (group, m)


def test_a_layer_in_a_graph():
    """Quantization and product, laid out and not, captured and replayed with other inputs beside eager work."""
    say("linear_int4 in a graph")
    gen = torch.Generator(device=DEV).manual_seed(2)
    N, K, g = 96, 640, 128
    w = torch.empty(N, K, device=DEV)
    xs = [torch.empty(m, K, dtype=torch.bfloat16, device=DEV) for m in (3, 50)]
    ys = [torch.empty(x.shape[0], N, device=DEV) for x in xs]
    codes, params = torch.empty(N, K // 2, dtype=torch.uint8, device=DEV), torch.empty(N, K // g, 2, dtype=torch.float16, device=DEV)
    ws = [torch.empty(echo.echo_linear_int4_workspace_bytes(x.shape[0], N, K, g), dtype=torch.uint8, device=DEV) for x in xs]

    def step():
        echo.echo_quantize_groups(w, K, echo.F32, N, K, g, codes, K // 2, params, K // g)
        for x, y, s in zip(xs, ys, ws):
            echo.echo_linear_int4(x, K, echo.BF16, codes, K // 2, params, K // g, g, None, x.shape[0], N, K, y, N, echo.F32, s)

    def inputs():
        for t in (w, *xs):
            t.copy_(torch.randn(t.shape, generator=gen, device=DEV))

    inputs()
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        inputs()
        graph.replay()
        torch.cuda.synchronize()
        got = [y.clone() for y in ys]
        for y in ys:
            y.zero_()
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(ys, got)), i
