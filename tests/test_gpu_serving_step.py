"""The serving operators together, as a tensor-parallel decode step uses them:
the query, key and value layer in 4 bits, the cache, the attention over it, the
output layer's partial sums and their low-bit all-reduce, for P simulated
ranks."""
import pytest
import torch

import _serve_ref as ref
from _helpers import DEV, say
from error_feedback_quant_amd import echo

pytestmark = pytest.mark.gpu


class Rank:
    """A rank's share of the heads, its weights in 4 bits and its cache."""

    def __init__(self, gen, hidden, q_heads, heads, D, kind, pages, page):
        self.q_heads, self.heads, self.D = q_heads, heads, D
        self.sizes = [q_heads * D, heads * D, heads * D]
        self.qkv = self.quantized(torch.randn(sum(self.sizes), hidden, generator=gen, device=DEV) * hidden ** -0.5)
        self.o = self.quantized(torch.randn(hidden, q_heads * D, generator=gen, device=DEV) * (q_heads * D) ** -0.5)
        dt, width = {"bf16": (torch.bfloat16, D), "i8": (torch.int8, D), "i4": (torch.uint8, D // 2)}[kind]
        shape = (pages, heads, page)
        self.k, self.v = (torch.zeros(*shape, width, dtype=dt, device=DEV) for _ in range(2))
        self.ks = self.vs = None
        if kind != "bf16":
            more = (2,) if kind == "i4" else ()
            self.ks, self.vs = (torch.zeros(*shape, *more, dtype=torch.float16 if kind == "i4" else torch.float32, device=DEV) for _ in range(2))
        self.cache = echo.make_cache(self.k, self.v, self.ks, self.vs)

    @staticmethod
    def quantized(w):
        n, k = w.shape
        codes = torch.empty(n, k // 2, dtype=torch.uint8, device=DEV)
        params = torch.empty(n, -(-k // 128), 2, dtype=torch.float16, device=DEV)
        echo.echo_quantize_groups(w, k, echo.F32, n, k, 128, codes, k // 2, params, params.shape[1])
        return codes, params

    def layer(self, x, weight, out):
        codes, params = weight
        m, k = x.shape
        n = codes.shape[0]
        ws = torch.empty(echo.echo_linear_int4_workspace_bytes(m, n, k, 128), dtype=torch.uint8, device=DEV)
        echo.echo_linear_int4(x, x.stride(0), echo.BF16, codes, codes.stride(0), params, params.shape[1], 128, None, m, n, k, out, out.stride(0),
                              echo.BF16, ws)

    def step(self, x, seqs, out):
        T = x.shape[0]
        qkv = torch.empty(T, sum(self.sizes), dtype=torch.bfloat16, device=DEV)
        self.layer(x, self.qkv, qkv)
        q, k, v = qkv.split(self.sizes, 1)                       # rows at a distance: no copies
        echo.echo_cache_write(self.cache, seqs, k, v)
        o = torch.empty(T, self.sizes[0], dtype=torch.bfloat16, device=DEV)
        args = echo.make_attention_args(self.cache, seqs, q, o, self.q_heads)
        ws = torch.empty(echo.echo_cache_attention_workspace_bytes(args), dtype=torch.uint8, device=DEV)
        echo.echo_cache_attention(args, ws)
        self.layer(o, self.o, out)
        return q, k, v, o

    def plain(self, weight, n):
        codes, params = weight
        p = params.double().repeat_interleave(128, 1)[:, :n]
        return (torch.stack([codes & 15, codes >> 4], -1).flatten(-2)[:, :n].double() - p[..., 1]) * p[..., 0]


@pytest.mark.parametrize("kind", ["bf16", "i8", "i4"])
def test_prompts_then_single_tokens(kind):
    """Three prompts in one call, then three steps of a token each.  Every stage against its plain form on the stage's own inputs: a
    layer within half a step of bfloat16 and its fp32 sums, the attention's result against all tokens so far within the bound of its
    weights' rounding, the all-reduced message against the ranks' sum within the quantizer's step."""
    say("serving step", kind)
    hidden, D, page, P = 512, 64, 16, 2
    gen = torch.Generator(device=DEV).manual_seed(3)
    lens = [37, 5, 64]
    pages = 24
    ranks = [Rank(gen, hidden, 4, 2, D, kind, pages, page) for _ in range(P)]
    table = torch.randperm(pages, generator=gen, device=DEV).int().view(3, 8)
    done = [[[], []] for _ in range(3)]                          # per sequence: k, v that rank 0 was given
    for step in range(4):
        new = list(lens) if step == 0 else [1, 1, 1]
        now = [n + step for n in lens]
        T = sum(new)
        starts = torch.tensor([0, new[0], new[0] + new[1], T], dtype=torch.int32, device=DEV)
        seqs = echo.make_seqs(starts, torch.tensor(now, dtype=torch.int32, device=DEV), table, T, max_new=max(new), max_len=max(now))
        rows = -(-T // (2 * P)) * 2 * P                          # the message is whole groups for every rank
        x = torch.randn(T, hidden, generator=gen, device=DEV).bfloat16()
        parts = [torch.zeros(rows, hidden, dtype=torch.bfloat16, device=DEV) for _ in range(P)]
        outs = [torch.empty(rows, hidden, device=DEV) for _ in range(P)]
        for r, rank in enumerate(ranks):
            q, k, v, o = rank.step(x, seqs, parts[r][:T])
            # the layers
            for a, weight, y in ((x, rank.qkv, torch.cat([q, k, v], 1)), (o, rank.o, parts[r][:T])):
                w = rank.plain(weight, a.shape[1])
                want = a.double() @ w.t()
                mag = a.double().abs() @ (w.abs() + 32 * weight[1][..., 0].double().repeat_interleave(128, 1)[:, :a.shape[1]]).t()
                assert not bool(ref.outside(y, want, 2 * 400 * ref.U * mag).any())
            if r:
                continue
            # the attention over everything so far
            at = 0
            for b, n in enumerate(new):
                done[b][0].append(k[at:at + n].clone())
                done[b][1].append(v[at:at + n].clone())
                L = now[b]
                ids = table[b, :-(-L // page)].long()
                held = []
                for t, sc in ((rank.k, rank.ks), (rank.v, rank.vs)):
                    u = ref.values(kind, t[ids], None if sc is None else sc[ids], D)
                    held.append(u.transpose(0, 1).reshape(rank.heads, -1, D)[:, :L])
                for given, kept in zip(done[b], held):           # the cache holds what was written, to its step
                    u = torch.cat(given).view(L, rank.heads, D).transpose(0, 1).double()
                    span = u.amax(-1, keepdim=True).clamp(min=0) - u.amin(-1, keepdim=True).clamp(max=0)
                    step_of = {"bf16": 0.0, "i8": 0.51 / 127, "i4": 1.01 / 15}[kind]
                    size = u.abs().amax(-1, keepdim=True) if kind == "i8" else span
                    assert bool(((u - kept).abs() <= step_of * size + 1e-12).all())
                pos = torch.arange(L - n, L, device=DEV)[:, None]
                sees = torch.arange(L, device=DEV)[None] <= pos
                offs = None
                for hq in range(rank.q_heads):
                    h = hq // (rank.q_heads // rank.heads)
                    if kind == "i4":
                        offs = tuple(((16 + sc[ids][..., 1].double()) * sc[ids][..., 0].double()).transpose(0, 1).reshape(rank.heads, -1)[h, :L]
                                     for sc in (rank.ks, rank.vs))
                    want, _, tol, _ = (t.to(DEV) for t in ref.attention(q[at:at + n].view(n, -1, D)[:, hq].double(), held[0][h], held[1][h],
                                                                         sees, D ** -0.5, offs))
                    assert not bool(ref.outside(o[at:at + n].view(n, -1, D)[:, hq], want, tol).any()), (step, b, hq)
                at += n
        # the message
        ws = torch.empty(echo.echo_allreduce_sim_workspace_bytes(P, rows * hidden, 8), dtype=torch.uint8, device=DEV)
        echo.echo_allreduce_sim(echo.make_sim_args([p.view(-1) for p in parts], [t.view(-1) for t in outs], ws, bits=8, out_dtype=echo.OUT_F32))
        torch.cuda.synchronize()
        total = sum(p.double() for p in parts)
        # a push and a requantization, each off by a step of its group's span over 255 at most
        span = 2 * max(float(p.float().abs().max()) for p in parts + [total.float()])
        assert float((outs[0].double() - total).abs().max()) <= 2 * P * 1.01 * span / 255
        assert torch.equal(outs[0], outs[1])
