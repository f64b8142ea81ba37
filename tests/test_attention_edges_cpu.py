"""What can be known of the softmax-attention operators' corners without a GPU: score factors outside fp32's normal
range are refused, and the gradient's formula, which the kernel is held to, is that of the differences."""
import pytest
import torch

import attention_ref as ref
from test_attention_cpu import INVALID, P, decode, lib  # noqa: F401  (lib is a fixture)

# scores are formed as q . k times |scale| log2(e), with a cap times |scale| / softcap and softcap log2(e)
FACTORS = [
    dict(scale=3e38),                     # times log2(e): infinite
    dict(scale=-2.5e38),
    dict(scale=1e-39), dict(scale=-1e-45),
    dict(scale=0.1, softcap=1e38),        # a quotient below the smallest normal number
    dict(scale=1e-30, softcap=1e9),
    dict(scale=1.0, softcap=3e38),        # times log2(e): infinite
    dict(scale=0.0, softcap=3e38),
    dict(scale=1e38, softcap=1e-3),
]


@pytest.mark.parametrize("kw", FACTORS, ids=str)
def test_decode_refuses_factors_outside_the_normal_range(lib, kw):  # noqa: F811
    for scales in (dict(), dict(ksc=P, vsc=P)):
        assert decode(lib, **kw, **scales, b=0) == INVALID  # (an empty batch would launch nothing)


@pytest.mark.parametrize("kw", [dict(scale=0.0), dict(scale=-0.1), dict(scale=2e38), dict(scale=1e-37), dict(scale=0.0, softcap=50.0),
                                dict(scale=0.1, softcap=1e30), dict(scale=1e-20, softcap=1e-3), dict(scale=0.1, softcap=2e36)], ids=str)
def test_decode_takes_factors_inside_it(lib, kw):  # noqa: F811
    assert decode(lib, **kw, b=0) == 0  # (an empty batch: nothing is launched)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot,eps,weights", [(16, 1e-6, True), (32, 0.0, True), (0, 1e-2, True), (16, 1e-6, False)])
def test_gradient_formula_against_differences(rot, eps, weights, interleaved):
    g = torch.Generator().manual_seed(5)
    tokens, h, d = 3, 2, 32
    x, dy = (torch.randn(tokens, h, d, generator=g, dtype=torch.float64) for _ in range(2))
    w = 1 + 0.3 * torch.randn(d, generator=g, dtype=torch.float64) if weights else None
    pos = torch.tensor([0, 3, 17], dtype=torch.int32)
    tab = ref.table(rot, 20) if rot else None
    dx, dw, _, _ = ref.norm_rope_bwd(x, w, eps, tab, pos, interleaved, dy)
    f = lambda x, w: (ref.norm_rope(x, w, eps, tab, pos, interleaved)[0] * dy).sum()
    for _ in range(4):
        ux, uw = torch.randn(x.shape, generator=g, dtype=torch.float64), torch.randn(d, generator=g, dtype=torch.float64)
        e = 1e-5
        ahead, behind = (f(x + s * ux, None if w is None else w + s * uw) for s in (e, -e))
        want = (dx * ux).sum() + (0 if w is None else (dw * uw).sum())
        # central differences: e^2 / 6 times a third derivative of order 1 to 10^3, and 2^-53 / e of rounding
        assert abs((ahead - behind) / (2 * e) - want) <= 1e-6 * (1 + abs(want))
