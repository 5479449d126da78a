"""Cases of a rank's serving step between the norm's output and the message of
the all-reduce: layers with 4-bit weights, the quantized paged cache, and the
attention of new tokens over it.

M counts tokens, N and K the outputs and inputs of a layer.  B sequences have
up to `new` new tokens each and are up to `ctx` long with them; hq query heads
share hkv heads of the cache, D wide; a page holds `page` tokens.  Widths of
layers are the repository's workloads' (4096, and 3584 of a down projection at
TP = 4) and generic ones; 8 and 2 heads are a quarter of 32 and 8.

run() computes a case in elementary torch operations in 32 bits, or, with
``own`` set, through the framework's entry points.
"""
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZES = {"bf16": 2, "f32": 4}
KIND_BYTES = {"bf16": 2.0, "i8": 1.0, "i4": 0.5}
TINY = 2.0 ** -100           # smallest magnitude that sets an 8-bit scale


def _layer(name, M, N, K, group=128, x="bf16", y="bf16", bias=False, pad=0, op="linear"):
    """op "linear": codes and parameters in hand; "requantize": the weight goes to 4 bits first."""
    return dict(name=name, op=op, M=M, N=N, K=K, group=group, x=x, y=y, bias=bias, pad=pad)


def _cache(name, op, B, new, ctx, hkv=8, D=128, page=64, kind="i8", x="bf16", mix="all"):
    """op "write": new tokens into the cache, and back as values; "read": the last `new` tokens of each sequence."""
    return dict(name=name, op=op, B=B, new=new, ctx=ctx, hkv=hkv, D=D, page=page, kind=kind, x=x, mix=mix)


def _attention(name, B, new, ctx, hq=32, hkv=8, D=128, page=64, kind="i8", mix="all", window=0, causal=True):
    """mix "all": `new` new tokens and `ctx` long, every one; "ragged": new tokens and lengths up to these; "one": the
    first sequence has `new` new tokens, the others one, lengths up to ctx."""
    return dict(name=name, op="attention", B=B, new=new, ctx=ctx, hq=hq, hkv=hkv, D=D, page=page, kind=kind, mix=mix,
                window=window, causal=causal)


def listed():
    return [
        # one token of one request through a square projection: latency, the weight is all there is to read
        _layer("int4_one_token", 1, 4096, 4096),
        # a ragged decode batch through a layer whose sizes fit no tile, fp32 in and out, fine groups
        _layer("int4_ragged", 13, 1001, 3583, group=32, x="f32", y="f32", bias=True),
        # a weight that has just been updated goes to 4 bits and serves a batch of requests
        _layer("int4_requantized", 64, 8192, 8192, op="requantize"),
        # the same of an odd TP = 4 down projection
        _layer("int4_requantized_ragged", 27, 1001, 3583, group=64, bias=True, pad=5, op="requantize"),
        # a decode step of a batch writes its new tokens: latency
        _cache("cache_write_step", "write", 64, 1, 2048, mix="ragged"),
        # a prompt's chunk into a 4-bit cache
        _cache("cache_write_chunk", "write", 4, 4096, 6000, kind="i4"),
        # whole sequences back as values, as when they move to another engine
        _cache("cache_read_whole", "read", 8, 8192, 8192, mix="ragged"),
        # one request of one TP = 4 rank, one token: latency
        _attention("attention_one_request", 1, 1, 4096, hq=8, hkv=2),
        # a decode step over a 4-bit cache, sequences of all lengths
        _attention("attention_decode_batch", 64, 1, 16384, kind="i4", mix="ragged"),
        # drafted tokens of a batch over a sliding window, narrow heads, bf16
        _attention("attention_drafted", 24, 5, 5000, hq=16, hkv=2, D=64, page=16, kind="bf16", window=1024, mix="ragged"),
        # a chunk of a prompt beside decoding sequences, bf16
        _attention("attention_mixed", 8, 512, 8192, kind="bf16", mix="one"),
        # a whole prompt: work of the matrix cores
        _attention("attention_prompt", 1, 8192, 8192),
    ]


def _between(rng, lo, hi):
    """An integer spread over the logarithm of [lo, hi]; half of the larger ones are rounded to a multiple of 64."""
    v = int(round(lo * (hi / lo) ** rng.random()))
    return max(lo, v // 64 * 64) if v >= 128 and rng.random() < 0.5 else v


def draw(rng):
    op = rng.choice(["linear", "requantize", "write", "read", "attention", "attention", "attention"])
    if op in ("linear", "requantize"):
        both = rng.choice(["bf16", "f32"]) if op == "linear" else "bf16"
        return _layer("drawn", _between(rng, 1, 64), _between(rng, 48, 8192), _between(rng, 64, 8192),
                      group=rng.choice([32, 64, 128, 256]), x=both, y=both, bias=rng.random() < 0.5,
                      pad=rng.choice([0, 0, 16, 5]), op=op)
    D, page, kind = rng.choice([64, 128, 128, 256, 80, 96]), rng.choice([16, 64, 128, 24]), rng.choice(["bf16", "i8", "i4"])
    hkv, mix = rng.choice([1, 2, 4, 8]), rng.choice(["all", "ragged", "one"])
    B = _between(rng, 1, 64)
    if op != "attention":
        new = _between(rng, 1, min(8192, (1 << 25) // (B * hkv * D)))
        return _cache("drawn", op, B, new, new + _between(rng, 1, 1024), hkv, D, page, kind, rng.choice(["bf16", "f32"]), mix)
    G = rng.choice([1, 2, 3, 4, 8])
    ctx = _between(rng, 1, min(65536, (1 << 27) // (B * hkv * D)))
    new = rng.choice([1, 1, _between(rng, 1, 8), _between(rng, 1, 2048)])
    new = max(1, min(new, ctx, (1 << 29) // (B * ctx * hkv * G)))
    return _attention("drawn", B, new, ctx, hkv * G, hkv, D, page, kind, mix, rng.choice([0, 0, _between(rng, 1, 4096)]),
                      rng.random() < 0.8)


# ------------------------------------------------------------------- inputs --

def _rows(gen, rows, cols, pad, dtype, scale=1.0, outliers=0.0):
    """[rows, cols] normal values in rows of cols + pad, a share of them 20 times larger (as activations have)."""
    buf = torch.randn(rows, cols + pad, generator=gen, device="cuda") * scale
    if outliers:
        buf *= 1.0 + 19.0 * (torch.rand(rows, cols + pad, generator=gen, device="cuda") < outliers)
    return buf.to(dtype)[:, :cols]


def _pack(q):
    """4-bit codes two a byte, the even one low."""
    if q.shape[-1] % 2:
        q = torch.nn.functional.pad(q, (0, 1))
    return (q[..., 0::2] | (q[..., 1::2] << 4)).to(torch.uint8)


def _unpack(b, n):
    return torch.stack([b & 15, b >> 4], -1).flatten(-2)[..., :n]


def _quant4(u):
    """Codes, scale (binary16) and zero point of the groups in u's last dimension, in single fp32 operations."""
    lo, hi = u.amin(-1).clamp(max=0.0), u.amax(-1).clamp(min=0.0)
    s = ((hi - lo) / 15.0).half().float()
    s = torch.where(s == 0, torch.full_like(s, 2.0 ** -24), s).clamp(max=65504.0)
    flat = hi == lo
    inv = torch.where(flat, torch.zeros_like(s), 1.0 / s)
    z = torch.round(-lo * inv).clamp(0, 15)
    q = (torch.round(u * inv[..., None]) + z[..., None]).clamp(0, 15)
    return q.to(torch.uint8), torch.where(flat, torch.zeros_like(s), s), z


def _groups_of(w, group):
    """[rows, cols] as [rows, groups, group], the last group filled up with its first value (which changes no bound)."""
    n, k = w.shape
    more = -k % group
    if more:
        w = torch.cat([w, w[:, k - k % group:k - k % group + 1].expand(n, more)], 1)
    return w.reshape(n, -1, group)


def _params(s, z):
    """(scale, zero) as pairs of binary16."""
    return torch.stack([s.half(), z.half()], -1).contiguous()


def _weight4(w, group):
    """Packed codes [N, ceil(K / 2)] and parameters [N, groups, 2] of a weight."""
    q, s, z = _quant4(_groups_of(w.float(), group))
    return _pack(q.reshape(w.shape[0], -1)[:, :w.shape[1]]), _params(s, z)


def _quant8(u):
    a = u.abs().amax(-1).clamp(min=TINY)
    return torch.round(u * (127.0 / a)[..., None]).to(torch.int8), a / 127.0


def _lengths(c):
    """New tokens and length of each sequence, from the case alone."""
    rng = random.Random("%d %d %d %s" % (c["B"], c["new"], c["ctx"], c["mix"]))
    new = [c["new"] if c["mix"] == "all" or b == 0 else 1 if c["mix"] == "one" else rng.randint(1, c["new"]) for b in range(c["B"])]
    return new, [c["ctx"] if c["mix"] == "all" or b == 0 else rng.randint(max(n, c["ctx"] // 8), max(n, c["ctx"]))
                 for b, n in enumerate(new)]


def _ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device="cuda")


def prepare(case, seed):
    c, gen = dict(case), torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": c}
    if c["op"] in ("linear", "requantize"):
        M, N, K = c["M"], c["N"], c["K"]
        s["x"] = _rows(gen, M, K, c["pad"], DTYPES[c["x"]], 1.0, 0.001)
        w = _rows(gen, N, K, c["pad"], torch.bfloat16, K ** -0.5)
        if c["op"] == "linear":
            s["wq"], s["wp"] = _weight4(w, c["group"])
        else:
            s["w"] = w
            s["wq"] = torch.empty(N, (K + 1) // 2, dtype=torch.uint8, device="cuda")
            s["wp"] = torch.empty(N, -(-K // c["group"]), 2, dtype=torch.float16, device="cuda")
        s["bias"] = torch.randn(N, generator=gen, device="cuda") if c["bias"] else None
        s["y"] = torch.empty(M, N, dtype=DTYPES[c["y"]], device="cuda")
        return s
    new, lens = _lengths(c)
    B, Hk, D, page, kind = c["B"], c["hkv"], c["D"], c["page"], c["kind"]
    counts = [-(-n // page) for n in lens]
    pages, wide = sum(counts) + 3, max(counts)
    order = torch.randperm(pages, generator=gen, device="cuda").int()
    first = torch.cumsum(_ints([0] + counts[:-1]), 0)
    at = torch.arange(wide, device="cuda")
    s["table"] = torch.where(at < _ints(counts)[:, None], order[(first[:, None] + at).clamp(max=pages - 1)], -1).int()
    s["starts"] = torch.cumsum(_ints([0] + new), 0).int()
    s["lens"], s["new"], s["max_new"], s["max_len"], s["T"] = _ints(lens), _ints(new), max(new), max(lens), sum(new)
    for part in ("k", "v"):
        full = torch.randn(pages, Hk, page, D, generator=gen, device="cuda")
        if part == "k":                      # a few channels of the keys are larger in every token
            full *= 1.0 + 3.0 * (torch.rand(Hk, 1, D, generator=gen, device="cuda") < 0.03)
        if kind == "bf16":
            s[part], s[part + "_scale"] = full.bfloat16(), None
        elif kind == "i8":
            s[part], s[part + "_scale"] = _quant8(full)
        else:
            q, sc, z = _quant4(full)
            s[part], s[part + "_scale"] = _pack(q), _params(sc, z)
    if c["op"] == "attention":
        s["q"] = _rows(gen, s["T"], c["hq"] * D, 0, torch.bfloat16, 1.5)
        s["out"] = torch.empty(s["T"], c["hq"] * D, dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.empty(s["T"], c["hq"], device="cuda")
        return s
    if c["op"] == "write":
        s["k_new"], s["v_new"] = (_rows(gen, s["T"], Hk * D, 0, DTYPES[c["x"]], 1.0, 0.001) for _ in range(2))
    s["k_out"], s["v_out"] = (torch.empty(s["T"], Hk * D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    return s


# -------------------------------------------------------------- plain forms --

def _plain_linear(c, s):
    if c["op"] == "requantize":
        s["wq"], s["wp"] = _weight4(s["w"], c["group"])
    p = s["wp"].float().repeat_interleave(c["group"], 1)[:, :c["K"]]
    w = (_unpack(s["wq"], c["K"]).float() - p[..., 1]) * p[..., 0]
    y = s["x"].float() @ w.t()
    return {"y": (y if s["bias"] is None else y + s["bias"]).to(DTYPES[c["y"]])}


def _values(c, codes, scale):
    if c["kind"] == "bf16":
        return codes.float()
    if c["kind"] == "i8":
        return codes.float() * scale[..., None]
    p = scale.float()
    return (_unpack(codes, c["D"]).float() - p[..., 1:]) * p[..., :1]


def _places(c, s):
    """Page and slot of every new token, in the order of the tokens."""
    row = torch.repeat_interleave(torch.arange(c["B"], device="cuda"), s["new"], output_size=s["T"])
    pos = torch.arange(s["T"], device="cuda") - s["starts"][row] + (s["lens"] - s["new"])[row]
    return s["table"][row, pos // c["page"]].long(), pos % c["page"]


def _plain_cache(c, s):
    page, slot = _places(c, s)
    got = {}
    for part in ("k", "v"):
        if c["op"] == "write":
            u = s[part + "_new"].float().view(s["T"], c["hkv"], c["D"])
            if c["kind"] == "bf16":
                s[part][page, :, slot] = u.bfloat16()
            elif c["kind"] == "i8":
                s[part][page, :, slot], s[part + "_scale"][page, :, slot] = _quant8(u)
            else:
                q, sc, z = _quant4(u)
                s[part][page, :, slot], s[part + "_scale"][page, :, slot] = _pack(q), _params(sc, z)
        sc = None if s[part + "_scale"] is None else s[part + "_scale"][page, :, slot]
        got[part] = _values(c, s[part][page, :, slot], sc).bfloat16().view(s["T"], -1)
    return got


def _plain_attention(c, s):
    B, Hk, D, G, n, L = c["B"], c["hkv"], c["D"], c["hq"] // c["hkv"], s["max_new"], s["max_len"]
    at = torch.arange(L, device="cuda")
    page, slot = s["table"][:, at // c["page"]].long().clamp(min=0), (at % c["page"]).expand(B, L)
    k, v = (_values(c, s[p][page, :, slot], None if s[p + "_scale"] is None else s[p + "_scale"][page, :, slot])
            .transpose(1, 2).contiguous() for p in ("k", "v"))
    i = torch.arange(n, device="cuda")
    there = i < s["new"][:, None]
    row = (s["starts"][:-1, None] + i).clamp(max=s["T"] - 1).long()
    q = s["q"].float()[row].view(B, n, Hk, G, D).transpose(1, 2).reshape(B, Hk, n * G, D)
    pos = (s["lens"] - s["new"])[:, None] + i
    seen = (at <= pos[..., None]) if c["causal"] else (at < s["lens"][:, None, None]).expand(B, n, L)
    if c["window"]:
        seen = seen & (at > pos[..., None] - c["window"])
    seen = seen[:, None, :, None, :]
    x = (q @ k.transpose(2, 3)).view(B, Hk, n, G, L) * D ** -0.5
    x = torch.where(seen, x, -torch.inf)
    m = x.amax(-1, keepdim=True)
    x = torch.exp(x - torch.where(m == -torch.inf, 0.0, m))
    l = x.sum(-1, keepdim=True)
    o = (x.view(B, Hk, n * G, L) @ v).view(B, Hk, n, G, D) / torch.where(l == 0, 1.0, l)
    o = o.permute(0, 2, 1, 3, 4)[there].reshape(s["T"], -1).bfloat16()
    return {"out": o, "lse": (m + torch.log(l)).permute(0, 2, 1, 3, 4)[there].reshape(s["T"], -1)}


# ------------------------------------------------------ the framework's own --

def _own(c, s):
    from error_feedback_quant_amd import echo
    kind = {"bf16": echo.BF16, "f32": echo.F32}
    if c["op"] in ("linear", "requantize"):
        M, N, K, g, w, p = c["M"], c["N"], c["K"], c["group"], s["wq"], s["wp"]
        if c["op"] == "requantize":
            echo.echo_quantize_groups(s["w"], s["w"].stride(0), echo.BF16, N, K, g, w, w.stride(0), p, p.shape[1])
        ws = torch.empty(echo.echo_linear_int4_workspace_bytes(M, N, K, g), dtype=torch.uint8, device="cuda")
        echo.echo_linear_int4(s["x"], s["x"].stride(0), kind[c["x"]], w, w.stride(0), p, p.shape[1], g, s["bias"], M, N, K,
                              s["y"], N, kind[c["y"]], ws)
        return {"y": s["y"]}
    cache = echo.make_cache(s["k"], s["v"], s["k_scale"], s["v_scale"])
    seqs = echo.make_seqs(s["starts"], s["lens"], s["table"], s["T"], max_new=s["max_new"], max_len=s["max_len"])
    if c["op"] == "attention":
        a = echo.make_attention_args(cache, seqs, s["q"], s["out"], c["hq"], lse=s["lse"], causal=c["causal"], window=c["window"])
        ws = torch.empty(echo.echo_cache_attention_workspace_bytes(a), dtype=torch.uint8, device="cuda")
        echo.echo_cache_attention(a, ws)
        return {"out": s["out"], "lse": s["lse"]}
    if c["op"] == "write":
        echo.echo_cache_write(cache, seqs, s["k_new"], s["v_new"])
    echo.echo_cache_read(cache, seqs, s["k_out"], s["v_out"])
    return {"k": s["k_out"], "v": s["v_out"]}


def _plain(c, s):
    if c["op"] in ("linear", "requantize"):
        return _plain_linear(c, s)
    return _plain_attention(c, s) if c["op"] == "attention" else _plain_cache(c, s)


def run(state):
    return (_own if own else _plain)(state["case"], state)


# ---------------------------------------------------------------- the work --

def work(case):
    c = case
    if c["op"] in ("linear", "requantize"):
        M, N, K = c["M"], c["N"], c["K"]
        w = N * ((K + 1) // 2) + 4 * N * -(-K // c["group"])
        data = M * K * SIZES[c["x"]] + M * N * SIZES[c["y"]] + (4 * N if c["bias"] else 0)
        return {"bytes": data + w + (2 * N * K + w if c["op"] == "requantize" else 0), "flops": 2 * M * N * K}
    new, lens = _lengths(c)
    row = c["D"] * KIND_BYTES[c["kind"]] + (0 if c["kind"] == "bf16" else 4)     # a token's codes and scale in one head
    T, Hk = sum(new), c["hkv"]
    if c["op"] != "attention":
        through = T * Hk * 2 * (row + 2 * c["D"])                                # codes in, values out
        more = T * Hk * 2 * (row + c["D"] * SIZES[c["x"]]) if c["op"] == "write" else 0
        return {"bytes": through + more, "flops": 4 * T * Hk * c["D"]}
    W = c["window"] or max(lens) + 1
    tokens = pairs = 0
    for n, l in zip(new, lens):
        tokens += min(l, W + n - 1)
        if c["causal"]:
            full = max(0, min(n, l - W + 1))             # rows at the end whose window is all there
            pairs += full * W + sum(range(l - n + 1, l - full + 1))
        else:
            pairs += sum(min(l, W + i) for i in range(n))
    return {"bytes": tokens * Hk * 2 * row + T * c["hq"] * (4 * c["D"] + 4), "flops": 4 * c["hq"] * c["D"] * pairs}


# ------------------------------------------------------- the same in 64 bits --

def _exact4(u):
    """(codes - zero) and scale of groups in float64; the scale is a binary16."""
    low, high = torch.clamp(u.min(-1, keepdim=True).values, max=0), torch.clamp(u.max(-1, keepdim=True).values, min=0)
    step = ((high - low) / 15).to(torch.float16).double()
    step = torch.clamp(torch.where(step == 0, 2.0 ** -24, step), max=65504)
    zero = torch.clamp(torch.round(-low / step), 0, 15)
    code = torch.clamp(torch.round(u / step) + zero, 0, 15) - zero
    return torch.where(high == low, 0.0, code * step)


def _nibbles(b, n):
    w = b.long()
    both = torch.zeros(*w.shape[:-1], 2 * w.shape[-1], dtype=torch.double, device=w.device)
    both[..., ::2], both[..., 1::2] = w % 16, w // 16
    return both[..., :n]


def exact(case, seed):
    """The definitions in float64, sequence by sequence."""
    c, s = case, prepare(case, seed)
    if c["op"] in ("linear", "requantize"):
        K, g = c["K"], c["group"]
        w = s["w"].double() if c["op"] == "requantize" else _nibbles(s["wq"], K)
        for k in range(0, K, g):
            if c["op"] == "requantize":
                w[:, k:k + g] = _exact4(w[:, k:k + g])
            else:
                p = s["wp"][:, k // g].double()
                w[:, k:k + g] = (w[:, k:k + g] - p[:, 1:]) * p[:, :1]
        y = torch.mm(s["x"].double(), w.t().contiguous())
        return {"y": y if s["bias"] is None else y + s["bias"].double()}
    new, lens = _lengths(c)
    H, D, kind = c["hkv"], c["D"], c["kind"]

    def kept(part, pages):
        """All tokens of these pages as values: [heads, tokens, D]."""
        if kind == "bf16":
            v = s[part][pages].double()
        elif kind == "i8":
            v = s[part][pages].double() * s[part + "_scale"][pages].double().unsqueeze(-1)
        else:
            p = s[part + "_scale"][pages].double()
            v = (_nibbles(s[part][pages], D) - p[..., 1].unsqueeze(-1)) * p[..., 0].unsqueeze(-1)
        return v.transpose(0, 1).reshape(H, -1, D)

    if c["op"] == "write":
        got = {}
        for part in ("k", "v"):
            u = s[part + "_new"].double().view(-1, H, D)
            if kind == "i8":
                step = torch.clamp(u.abs().max(-1, keepdim=True).values, min=TINY) / 127
                u = torch.round(u / step) * step
            elif kind == "i4":
                u = _exact4(u)
            got[part] = u.reshape(len(u), -1)
        return got
    parts = {"k": [], "v": [], "out": [], "lse": []}
    at = 0
    for b in range(c["B"]):
        n, l = new[b], lens[b]
        pages = s["table"][b, :-(-l // c["page"])].long()
        k, v = kept("k", pages)[:, :l], kept("v", pages)[:, :l]
        if c["op"] == "read":
            for part, t in (("k", k), ("v", v)):
                parts[part].append(t[:, l - n:].transpose(0, 1).reshape(n, -1))
            continue
        q = s["q"][at:at + n].double().view(n, c["hq"], D).transpose(0, 1)
        at += n
        place, key = torch.arange(l - n, l, device="cuda")[:, None], torch.arange(l, device="cuda")
        hidden = (key > place) if c["causal"] else (key >= l).expand(n, l)
        if c["window"]:
            hidden = hidden | (key <= place - c["window"])
        outs, sums = [], []
        for h in range(c["hq"]):
            x = torch.mm(q[h], k[h // (c["hq"] // H)].t().contiguous()) / D ** 0.5
            x = x.masked_fill(hidden, -torch.inf)
            sums.append(torch.logsumexp(x, 1))
            outs.append(torch.mm(torch.exp(x - sums[-1][:, None]), v[h // (c["hq"] // H)].contiguous()))
        parts["out"].append(torch.stack(outs, 1).reshape(n, -1))
        parts["lse"].append(torch.stack(sums, 1))
    return {p: torch.cat(t) for p, t in parts.items() if t}
