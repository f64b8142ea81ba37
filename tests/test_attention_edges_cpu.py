"""What can be known of the softmax-attention operators' corners without a GPU."""
import pytest

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
