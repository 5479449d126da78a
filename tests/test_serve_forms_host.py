"""The limits of tests/_serve_forms.py tell the kernels' forms from forms that
leave a step out: planted on the host, in the plain forms."""
import numpy as np
import pytest

import _serve_forms as forms
import _serve_ref as ref


@pytest.mark.parametrize("group", [32, 64, 128, 256])
def test_limit_of_fp32_tokens(group):
    x, w = forms.linear_case(group, 13, 96, 4096)
    codes, params = ref.quant_groups(w, group)
    want, _ = ref.linear4(x.astype(np.float64), codes, params, group, None)

    def off(**how):
        return forms.off(forms.linear_form(x, codes, params, group, **how), want)
    for rounded in (forms.nearest, forms.cut):
        for chunk in (4, 32):
            assert off(chunk=chunk, rounded=rounded) < forms.LINEAR_LIMIT / 1.15
        for planted in (dict(centre=False), dict(apart=False), dict(parts=2), dict(parts=1), dict(apart=False, centre=False)):
            assert off(rounded=rounded, **planted) > forms.LINEAR_LIMIT * 1.1, planted


@pytest.mark.parametrize("kind", ["bf16", "i8", "i4"])
@pytest.mark.parametrize("L", [300, 3000])
def test_limit_of_few_rows(kind, L):
    rng = np.random.default_rng(L)
    scores, v = 1.5 * rng.standard_normal((8, L)), rng.standard_normal((L, 128)).astype(np.float32)
    if kind == "bf16":
        codes, scale, z, base = forms.bf16(v), np.ones(L), np.zeros(L), 0
    elif kind == "i8":
        codes, scale = ref.quant8(v)
        z, base = np.zeros(L), 0
    else:
        codes, scale, z = ref.quant4(v)
        scale, z, base = scale.view(np.float16), z.view(np.float16).astype(np.float64), 16
    codes, scale = codes.astype(np.float64), scale.astype(np.float64)
    p = np.exp(scores - scores.max(1, keepdims=True))
    want = p @ ((codes - z[:, None]) * scale[:, None]) / p.sum(1, keepdims=True)

    def over(parts):
        return forms.over_rounding(forms.attention_form(codes + base, scale, z + base, scores, parts), want)
    assert over(2) < 1.01 and over(1) > 1.15
