"""Cases of the operators around a tensor-parallel block: the 8-bit integer
product and linear layer, and the norms that close one block and open the
next, forward and backward.

Shapes are those of the repository's workloads (a single 64 x 1024 call, the
2048 x 4096 depth chain, the 32 x 4096 x 1024 training message, the 4096 x
4096 x 3584 down projection at TP = 4) and generic ones.  T and M count tokens,
H is the width of the stream, N and K the outputs and inputs of a layer.

run() computes a case in elementary torch operations in 32 bits, or, with
``own`` set, through the framework's entry points.
"""
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZES = {"bf16": 2, "f32": 4}
EPS = 1e-5
TINY = 2.0 ** -100           # smallest token magnitude that sets a scale


def _product(name, M, N, K, y="bf16", bias=False, pad=0):
    """Codes and scales in hand, the product out."""
    return dict(name=name, op="product", M=M, N=N, K=K, y=y, bias=bias, pad=pad)


def _linear(name, M, N, K, x="bf16", y="bf16", bias=False, pad=0):
    """Activations quantized token by token, then the product."""
    return dict(name=name, op="linear", M=M, N=N, K=K, x=x, y=y, bias=bias, pad=pad)


def _norm(name, T, H, x="bf16", r="bf16", w="bf16", h="bf16", post=True, gate=0, res=1.0, blk=1.0, pad=0,
          op="norm", N=0):
    """gate: tokens that share one row of the gate, 0 for none.  op "norm" is
    the forward pass, "backward" its gradients, "norm_product" the forward
    pass to 8 bits followed by the next layer's product of N outputs."""
    return dict(name=name, op=op, T=T, H=H, x=x, r=r, w=w, h=h, post=post, gate=gate, res=res, blk=blk, pad=pad, N=N)


def listed():
    return [
        # one token of one request through a square projection: latency, the weight is all there is to read
        _linear("linear_one_token", 1, 4096, 4096),
        # a decode batch of a few requests through a TP = 4 down projection with bias, an odd number of tokens
        _linear("linear_decode_batch", 27, 4096, 3584, bias=True),
        # a long prefill through a square projection
        _linear("linear_prefill", 16384, 4096, 4096),
        # partial sums of a TP = 4 down projection, as they enter the all-reduce
        _product("product_down_projection", 4096, 4096, 3584),
        # a ragged batch through a layer whose sizes fit no tile, into fp32 with bias
        _product("product_ragged", 777, 1001, 3583, y="f32", bias=True),
        # the single-call message: both norms around the residual
        _norm("norm_call", 64, 1024),
        # a chain-sized message, fp32 stream, a gate row for each sequence of 600 tokens (the last one cut short)
        _norm("norm_gated_chain", 2048, 4096, r="f32", gate=600, res=0.8, blk=0.5),
        # the training message: 32 sequences of 4096
        _norm("norm_training", 32 * 4096, 1024),
        # a decode step from the stream into the next projection: norm to 8 bits, then the product
        _norm("norm_product_decode", 8, 4096, op="norm_product", N=4096),
        # gradients of a ragged fp32 batch of odd width
        _norm("backward_ragged", 333, 1537, x="f32", r="f32", w="f32", h="f32", gate=1000, op="backward"),
        # gradients of the gated chain message
        _norm("backward_gated_chain", 2048, 4096, r="f32", gate=600, res=0.8, blk=0.5, op="backward"),
        # gradients of the training message
        _norm("backward_training", 32 * 4096, 1024, op="backward"),
    ]


def _between(rng, lo, hi):
    """An integer spread over the logarithm of [lo, hi]; half of the larger ones are rounded to a multiple of 64."""
    v = int(round(lo * (hi / lo) ** rng.random()))
    return max(lo, v // 64 * 64) if v >= 128 and rng.random() < 0.5 else v


def draw(rng):
    op = rng.choice(["product", "linear", "norm", "norm_product", "backward"])
    pad = rng.choice([0, 0, 16, 5])
    if op in ("product", "linear"):
        N, K = _between(rng, 48, 8192), _between(rng, 64, 8192)
        M = _between(rng, 1, max(2, min(16384, (1 << 38) // (N * K), (1 << 26) // max(N, K))))
        # a linear layer's output is bf16: its codes carry 8 bits, so an fp32 output would hold no more
        return (_product("", M, N, K, y=rng.choice(["bf16", "f32"]), bias=rng.random() < 0.5, pad=pad) if op == "product"
                else _linear("", M, N, K, x=rng.choice(["bf16", "f32"]), bias=rng.random() < 0.5, pad=pad)) | {"name": "drawn"}
    H = _between(rng, 64, 8192)
    few = op == "norm_product"
    T = _between(rng, 1, 2048 if few else max(2, min(131072, (1 << 26) // H)))
    return _norm("drawn", T, H, x=rng.choice(["bf16", "f32"]), r=rng.choice(["bf16", "f32"]),
                 w=rng.choice(["bf16", "f32"]), h="bf16" if few else rng.choice(["bf16", "f32"]),
                 post=rng.random() < 0.75, gate=rng.choice([0, 1, _between(rng, 1, 4096), 1 << 20]),
                 res=rng.choice([1.0, 0.8]), blk=rng.choice([1.0, 0.22]), pad=pad, op=op,
                 N=_between(rng, 48, 8192) if few else 0)


# ------------------------------------------------------------------- inputs --

def _rows(gen, rows, cols, pad, dtype, scale=1.0, outliers=0.0):
    """[rows, cols] normal values in rows of cols + pad, a share of them 20 times larger (as activations have)."""
    buf = torch.randn(rows, cols + pad, generator=gen, device="cuda") * scale
    if outliers:
        buf *= 1.0 + 19.0 * (torch.rand(rows, cols + pad, generator=gen, device="cuda") < outliers)
    return buf.to(dtype)[:, :cols]


def _codes(v, pad):
    """8-bit codes and scales of each row of v, codes in rows of cols + pad."""
    s = v.float().abs().amax(1).clamp(min=TINY) / 127.0
    q = torch.zeros(v.shape[0], v.shape[1] + pad, dtype=torch.int8, device=v.device)
    q[:, :v.shape[1]] = torch.round(v.float() / s[:, None]).clamp(-127, 127).to(torch.int8)
    return q[:, :v.shape[1]], s


def _weight(gen, N, K, pad):
    return _codes(_rows(gen, N, K, 0, torch.float32, K ** -0.5), pad)


def _groups(c):
    return -(-c["T"] // c["gate"]) if c["gate"] else 0


def prepare(case, seed):
    c, gen = dict(case), torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": c}
    pad = c["pad"]
    if c["op"] in ("product", "linear"):
        M, N, K = c["M"], c["N"], c["K"]
        if c["op"] == "product":
            s["xq"], s["sx"] = _codes(_rows(gen, M, K, 0, torch.bfloat16, 1.0, 0.001), pad)
        else:
            s["x"] = _rows(gen, M, K, pad, DTYPES[c["x"]], 1.0, 0.001)
        s["wq"], s["sw"] = _weight(gen, N, K, pad)
        s["bias"] = torch.randn(N, generator=gen, device="cuda") if c["bias"] else None
        s["y"] = torch.empty(M, N, dtype=DTYPES[c["y"]], device="cuda")
        return s
    T, H = c["T"], c["H"]
    s["x"] = _rows(gen, T, H, pad, DTYPES[c["x"]], 0.7, 0.001)
    s["r"] = _rows(gen, T, H, pad, DTYPES[c["r"]], 1.5)
    for k in ("w_post", "w_pre"):
        s[k] = (1.0 + 0.2 * torch.randn(H, generator=gen, device="cuda")).to(DTYPES[c["w"]])
    s["gate"] = (0.5 + 0.3 * torch.randn(_groups(c), H, generator=gen, device="cuda")).to(DTYPES[c["w"]]) if c["gate"] else None
    if c["op"] == "backward":
        s["dh"] = _rows(gen, T, H, pad, DTYPES[c["h"]], 1e-3)
        s["dr_out"] = _rows(gen, T, H, pad, DTYPES[c["r"]], 1e-3)
        s["dx"] = torch.empty(T, H, dtype=DTYPES[c["x"]], device="cuda")
        s["dr"] = torch.empty(T, H, dtype=DTYPES[c["r"]], device="cuda")
        s["dw_post"], s["dw_pre"] = (torch.empty(H, device="cuda") for _ in range(2))
        s["dgate"] = torch.empty(_groups(c), H, device="cuda") if c["gate"] else None
        return s
    s["r_out"] = torch.empty(T, H, dtype=DTYPES[c["r"]], device="cuda")
    if c["op"] == "norm":
        s["h"] = torch.empty(T, H, dtype=DTYPES[c["h"]], device="cuda")
        return s
    s["hq"] = torch.empty(T, -(-H // 16) * 16, dtype=torch.int8, device="cuda")
    s["sh"] = torch.empty(T, device="cuda")
    s["wq"], s["sw"] = _weight(gen, c["N"], H, pad)
    s["y"] = torch.empty(T, c["N"], dtype=torch.bfloat16, device="cuda")
    return s


# -------------------------------------------------------------- plain forms --

def _quantize(v):
    a = v.abs().amax(1).clamp(min=TINY)
    return torch.round(v * (127.0 / a)[:, None]), a / 127.0


def _scaled(xq, sx, s, out):
    y = (xq.float() @ s["wq"].float().t()) * sx[:, None] * s["sw"]
    if s.get("bias") is not None:
        y = y + s["bias"]
    return y.to(out)


def _forward(c, s):
    """r', h before rounding, and what the gradients need."""
    x, r = s["x"].float(), s["r"].float()
    g = s["gate"].float()[torch.arange(c["T"], device="cuda") // c["gate"]] if c["gate"] else None
    kx = torch.rsqrt((x * x).mean(1, keepdim=True) + EPS) if c["post"] else None
    z = x * kx * s["w_post"].float() if c["post"] else x
    rn = c["res"] * r + c["blk"] * (z if g is None else g * z)
    kr = torch.rsqrt((rn * rn).mean(1, keepdim=True) + EPS)
    return rn, rn * kr * s["w_pre"].float(), (x, g, kx, z, kr)


def _backward(c, s):
    rn, _, (x, g, kx, z, kr) = _forward(c, s)
    n = rn * kr
    dh = s["dh"].float()
    dn = dh * s["w_pre"].float()
    d = s["dr_out"].float() + kr * (dn - n * (dn * n).mean(1, keepdim=True))
    got = {"dr": (c["res"] * d).to(DTYPES[c["r"]]), "dw_pre": (dh * n).sum(0)}
    d = c["blk"] * d
    if g is not None:
        v = d * z
        more = _groups(c) * c["gate"] - c["T"] if _groups(c) > 1 else 0
        if more:
            v = torch.cat([v, v.new_zeros(more, c["H"])])
        got["dgate"] = v.view(_groups(c), -1, c["H"]).sum(1)
        d = d * g
    if c["post"]:
        n = x * kx
        got["dw_post"] = (d * n).sum(0)
        d = d * s["w_post"].float()
        d = kx * (d - n * (d * n).mean(1, keepdim=True))
    got["dx"] = d.to(DTYPES[c["x"]])
    return got


def _plain(c, s):
    if c["op"] == "product":
        return {"y": _scaled(s["xq"], s["sx"], s, DTYPES[c["y"]])}
    if c["op"] == "linear":
        return {"y": _scaled(*_quantize(s["x"].float()), s, DTYPES[c["y"]])}
    if c["op"] == "backward":
        return _backward(c, s)
    rn, h, _ = _forward(c, s)
    rn = rn.to(DTYPES[c["r"]])
    if c["op"] == "norm":
        return {"r_out": rn, "h": h.to(DTYPES[c["h"]])}
    return {"r_out": rn, "y": _scaled(*_quantize(h), s, torch.bfloat16)}


# ------------------------------------------------------ the framework's own --

def _own(c, s):
    from error_feedback_quant_amd import echo
    kind = {"bf16": echo.OUT_BF16, "f32": echo.OUT_F32}
    if c["op"] in ("product", "linear"):
        M, N, K, y, w = c["M"], c["N"], c["K"], s["y"], s["wq"]
        if c["op"] == "product":
            echo.echo_gemm_int8(s["xq"], s["xq"].stride(0), s["sx"], w, w.stride(0), s["sw"], s["bias"], M, N, K,
                                y, N, kind[c["y"]])
        else:
            ws = torch.empty(echo.echo_linear_int8_workspace_bytes(M, N, K), dtype=torch.uint8, device="cuda")
            echo.echo_linear_int8(s["x"], s["x"].stride(0), kind[c["x"]], w, w.stride(0), s["sw"], s["bias"], M, N, K,
                                  y, N, kind[c["y"]], ws)
        return {"y": y}
    post = dict(post=c["post"], w_post=s["w_post"] if c["post"] else None, w_pre=s["w_pre"], gate=s["gate"],
                gate_tokens=c["gate"], res_scale=c["res"], block_scale=c["blk"], eps=EPS)
    if c["op"] == "backward":
        a = echo.make_norm_args(s["x"], s["r"], **post)
        ws = torch.empty(echo.echo_block_norm_backward_workspace_bytes(c["T"], c["H"]), dtype=torch.uint8, device="cuda")
        got = {"dx": s["dx"], "dr": s["dr"], "dw_pre": s["dw_pre"]}
        if c["post"]:
            got["dw_post"] = s["dw_post"]
        if c["gate"]:
            got["dgate"] = s["dgate"]
        echo.echo_block_norm_backward(a, echo.make_norm_grads(s["dh"], s["dr_out"], workspace=ws, **got))
        return got
    if c["op"] == "norm":
        echo.echo_block_norm(echo.make_norm_args(s["x"], s["r"], r_out=s["r_out"], h=s["h"], **post))
        return {"r_out": s["r_out"], "h": s["h"]}
    echo.echo_block_norm(echo.make_norm_args(s["x"], s["r"], r_out=s["r_out"], h=s["hq"], h_scale=s["sh"], **post))
    echo.echo_gemm_int8(s["hq"], s["hq"].stride(0), s["sh"], s["wq"], s["wq"].stride(0), s["sw"], None,
                        c["T"], c["N"], c["H"], s["y"], c["N"], echo.OUT_BF16)
    return {"r_out": s["r_out"], "y": s["y"]}


def run(state):
    return (_own if own else _plain)(state["case"], state)


# ---------------------------------------------------------------- the work --

def work(case):
    c = case
    if c["op"] in ("product", "linear"):
        M, N, K = c["M"], c["N"], c["K"]
        data = M * K * (1 if c["op"] == "product" else SIZES[c["x"]]) + N * K + M * N * SIZES[c["y"]]
        scales = 4 * (N + (M if c["op"] == "product" else 0) + (N if c["bias"] else 0))
        return {"bytes": data + scales, "flops": 2 * M * N * K}
    n, G = c["T"] * c["H"], _groups(c)
    small = (G + 1 + c["post"]) * c["H"] * SIZES[c["w"]]
    if c["op"] == "backward":
        return {"bytes": n * (2 * SIZES[c["x"]] + 3 * SIZES[c["r"]] + SIZES[c["h"]]) + small
                + (G + 1 + c["post"]) * c["H"] * 4, "flops": 30 * n}
    data = n * (SIZES[c["x"]] + 2 * SIZES[c["r"]]) + small
    if c["op"] == "norm":
        return {"bytes": data + n * SIZES[c["h"]], "flops": 11 * n}
    return {"bytes": data + c["N"] * (c["H"] + 4) + 2 * c["T"] * c["N"], "flops": 11 * n + 2 * n * c["N"]}


# ------------------------------------------------------- the same in 64 bits --

def exact(case, seed):
    """The definitions in float64 (gradients by differentiation of the forward pass)."""
    c, s = case, prepare(case, seed)
    wide = lambda t: None if t is None else t.double()  # noqa: E731

    def layer(codes, scale):
        y = torch.mm(codes * scale, wide(s["wq"]).t().contiguous()) * wide(s["sw"])
        return y if s.get("bias") is None else y + wide(s["bias"])

    def coded(v):
        scale = torch.clamp(v.abs().max(dim=1, keepdim=True).values, min=TINY) / 127
        return torch.round(v / scale), scale

    if c["op"] == "product":
        return {"y": layer(wide(s["xq"]), wide(s["sx"])[:, None])}
    if c["op"] == "linear":
        return {"y": layer(*coded(wide(s["x"])))}
    leaf = {k: wide(s[k]) for k in ("x", "r", "w_post", "w_pre", "gate")}
    if c["op"] == "backward":
        leaf = {k: None if v is None else v.requires_grad_() for k, v in leaf.items()}

    def unit(v):
        return v / torch.sqrt(v.pow(2).sum(1, keepdim=True) / c["H"] + EPS)

    branch = unit(leaf["x"]) * leaf["w_post"] if c["post"] else leaf["x"]
    if c["gate"]:
        branch = branch * leaf["gate"].repeat_interleave(c["gate"] if _groups(c) > 1 else c["T"], 0)[:c["T"]]
    stream = leaf["r"] * c["res"] + branch * c["blk"]
    h = unit(stream) * leaf["w_pre"]
    if c["op"] == "norm":
        return {"r_out": stream, "h": h}
    if c["op"] == "norm_product":
        return {"r_out": stream, "y": layer(*coded(h))}
    ((h * wide(s["dh"])).sum() + (stream * wide(s["dr_out"])).sum()).backward()
    return {"d" + k: leaf[k].grad for k in ("x", "r", "w_pre", "w_post", "gate") if leaf[k] is not None
            and leaf[k].grad is not None}
