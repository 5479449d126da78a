"""One tensor-parallel MLP block in 8 bits around the low-bit all-reduce.

P simulated ranks hold a column-parallel up projection and a row-parallel
down projection, both quantized to 8 bits by rows of their [N, K] form:

  1. echo_block_norm closes the previous block: post norm of its all-reduced
     output, gate, residual sum, pre norm to 8-bit codes with a scale a token;
  2. every rank: echo_gemm_int8 (up), the activation, echo_linear_int8 (down),
     whose bf16 output is the rank's partial sums;
  3. echo_allreduce_sim sums them in 4 or 8 bits, with error feedback;
  4. echo_block_norm closes this block; in training, echo_block_norm_backward
     gives the gradients of the norms, the gate and the residual stream.

Run on an MI355X:  python examples/tp_block.py [tokens] [hidden] [ffn] [bits]
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from error_feedback_quant_amd import echo  # noqa: E402

EPS = 1e-5


def quantize_rows(w):
    """8-bit codes of a weight by rows, laid out once: (codes, scales)."""
    n, k = w.shape
    q = torch.empty(n, -(-k // 16) * 16, dtype=torch.int8, device=w.device)     # rows at 16 bytes: the fastest loads
    s = torch.empty(n, device=w.device)
    echo.echo_quantize_tokens(w, w.stride(0), echo.F32, n, k, q, q.stride(0), s)
    return q, s


class TpMlp:
    """The block's weights and buffers; call it with the previous block's output and the residual stream."""

    def __init__(self, tokens, hidden, ffn, P=4, bits=4, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, generator=g, device=device)  # noqa: E731
        self.T, self.H, self.F, self.P = tokens, hidden, ffn // P, P
        self.up = [rnd(self.F, hidden) * hidden ** -0.5 for _ in range(P)]
        self.down = [rnd(hidden, self.F) * ffn ** -0.5 for _ in range(P)]
        self.up_q, self.down_q = [quantize_rows(w) for w in self.up], [quantize_rows(w) for w in self.down]
        self.norm = {k: 1 + 0.1 * rnd(hidden) for k in ("w_post", "w_pre")}
        self.gate = 0.5 + 0.1 * rnd(1, hidden)
        bf16 = dict(dtype=torch.bfloat16, device=device)
        self.r = torch.empty(tokens, hidden, **bf16)
        self.hq = torch.empty(tokens, -(-hidden // 16) * 16, dtype=torch.int8, device=device)
        self.hs = torch.empty(tokens, device=device)
        self.a = torch.empty(tokens, self.F, **bf16)
        n = tokens * hidden
        self.parts = [torch.empty(tokens, hidden, **bf16) for _ in range(P)]
        self.outs = [torch.empty(tokens, hidden, **bf16) for _ in range(P)]
        self.comps = [torch.zeros(n, device=device) for _ in range(P)]
        need = echo.echo_linear_int8_workspace_bytes(tokens, hidden, self.F)
        self.ws = torch.empty(max(need, 16), dtype=torch.uint8, device=device)
        self.reduce_ws = torch.empty(echo.echo_allreduce_sim_workspace_bytes(P, n, bits), dtype=torch.uint8, device=device)
        self.reduce = echo.make_sim_args([p.view(-1) for p in self.parts], [o.view(-1) for o in self.outs], self.reduce_ws,
                                         bits=bits, out_dtype=echo.OUT_BF16, ef=True, comps=self.comps)

    def __call__(self, x, r):
        """The block's all-reduced output and the residual stream it adds to."""
        T, H, F = self.T, self.H, self.F
        echo.echo_block_norm(echo.make_norm_args(x, r, r_out=self.r, h=self.hq, h_scale=self.hs, gate=self.gate,
                                                 gate_tokens=T, eps=EPS, **self.norm))
        for p in range(self.P):
            q, s = self.up_q[p]
            echo.echo_gemm_int8(self.hq, self.hq.stride(0), self.hs, q, q.stride(0), s, None, T, F, H, self.a, F, echo.BF16)
            act = torch.nn.functional.silu(self.a)
            q, s = self.down_q[p]
            echo.echo_linear_int8(act, F, echo.BF16, q, q.stride(0), s, None, T, H, F, self.parts[p], H, echo.BF16, self.ws)
        echo.echo_allreduce_sim(self.reduce)
        return self.outs[0], self.r

    def plain(self, x, r):
        """The same block in fp32 without any quantization."""
        unit = lambda v: v * torch.rsqrt((v * v).mean(1, keepdim=True) + EPS)  # noqa: E731
        s = r.float() + self.gate * unit(x.float()) * self.norm["w_post"]
        h = unit(s) * self.norm["w_pre"]
        return sum(torch.nn.functional.silu(h @ u.t()) @ d.t() for u, d in zip(self.up, self.down)), s


def main(tokens=2048, hidden=4096, ffn=14336, bits=4):
    block = TpMlp(tokens, hidden, ffn, bits=bits)
    g = torch.Generator(device="cuda").manual_seed(1)
    x, r = (torch.randn(tokens, hidden, generator=g, device="cuda").bfloat16() for _ in range(2))
    out, stream = block(x, r)
    want, want_stream = block.plain(x, r)
    err = float((out.float() - want).norm() / want.norm())
    print(f"block of {tokens} x {hidden}, ffn {ffn}, {bits}-bit all-reduce: output off fp32 by {err:.4f} (relative 2-norm), "
          f"stream by {float((stream.float() - want_stream).norm() / want_stream.norm()):.5f}")
    # the norms that close this block, forward and backward (a training step
    # keeps what it needs: the block's output and the stream)
    h = torch.empty_like(stream)
    args = echo.make_norm_args(out, stream, r_out=torch.empty_like(stream), h=h, gate=block.gate, gate_tokens=tokens,
                               eps=EPS, **block.norm)
    echo.echo_block_norm(args)
    grads = dict(dx=torch.empty_like(out), dr=torch.empty_like(stream), dgate=torch.empty_like(block.gate),
                 **{"d" + k: torch.empty(hidden, device="cuda") for k in block.norm})
    ws = torch.empty(echo.echo_block_norm_backward_workspace_bytes(tokens, hidden), dtype=torch.uint8, device="cuda")
    echo.echo_block_norm_backward(args, echo.make_norm_grads(dh=torch.ones_like(h), workspace=ws, **grads))
    print("gradients of the sum of h: " + ", ".join(f"|{k}| = {float(v.float().norm()):.4g}" for k, v in grads.items()))
    return err, grads


if __name__ == "__main__":
    main(*(int(v) for v in sys.argv[1:]))
