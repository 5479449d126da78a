"""The steps that the 4-bit layer and the attention of few rows take for
accuracy: a form without one of them is past the limits of tests/_serve_forms.py."""
import numpy as np
import pytest
import torch

import _serve_forms as forms
import _serve_ref as ref
from _helpers import DEV, say
from test_gpu_attention import Case
from test_gpu_cache import KINDS
from test_gpu_int4 import linear, quantize

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("group", [32, 64, 128, 256])
@pytest.mark.parametrize("M", [1, 13, 40])
def test_fp32_tokens(group, M):
    """As they are, and laid out first (past 16 tokens)."""
    say("fp32 tokens", group, M)
    N, K = 512, 4096
    x, w = (torch.from_numpy(v).to(DEV) for v in forms.linear_case(group, M, N, K))
    codes, params = quantize(w, group)
    y = linear(x, codes, params, group, None, N, torch.float32)
    want, _ = ref.linear4(x.double().cpu().numpy(), codes.cpu().numpy(), params.contiguous().view(torch.int16).cpu().numpy().view(np.uint16),
                          group, None)
    assert forms.off(y.cpu().numpy(), want) < forms.LINEAR_LIMIT


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("new,lens", [([1, 3], [300, 2000]), ([1], [20000])])
def test_few_rows(kind, D, new, lens):
    """In one part of the tokens and in several that are joined: the error is the output's rounding."""
    c = Case(kind, 2, 4, D, 16, new, lens)
    out, _ = c.check()
    got, want, t = [], [], 0
    for b, n in enumerate(new):
        k, v, offs = c.sequence(b)
        for h in range(2):
            for g in range(4):
                q = c.q[t:t + n].view(n, -1, D)[:, 4 * h + g].double()
                want.append(ref.attention(q, k[h], v[h], c.sees(b), c.scale, offs[h])[0].cpu().numpy())
                got.append(out[t:t + n, 4 * h + g].double().cpu().numpy())
        t += n
    assert forms.over_rounding(np.concatenate(got), np.concatenate(want)) < forms.ATTENTION_LIMIT
