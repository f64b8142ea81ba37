"""The softmax-attention entry points refuse bad arguments on the host, before anything is launched
(CPU only: no call here reaches a kernel), and the binding checks its tensors."""
import ctypes

import pytest
import torch

import kimi_delta_attention_24_b200 as kda
from kimi_delta_attention_24_b200 import build as kbuild

P = 0x10000000  # an aligned address that is never dereferenced: validation fails first
OK, INVALID, UNSUPPORTED, SMALL = 0, 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    return kda.load()


def rope(lib, bwd=False, append=False, **kw):
    a = dict(q=P, k=P, v=P, qs=2048, ks=2048, vs=2048, wq=P, wk=P, eps=1e-6, tab=P, pos=P, qo=P, ko=P, dq=P, dk=P, dwq=P, dwk=P,
             tokens=4, hq=8, hk=2, d=128, rot=128, most=100, inter=0, ws=P, ws_bytes=1 << 30, kc=P, vc=P, ksc=None, vsc=None,
             slots=P, pages=4, page=16, kstep=2 * 16 * 128, vstep=2 * 16 * 128)
    a.update(kw)
    common = [a["wq"], a["wk"], a["eps"], a["tab"], a["pos"]]
    sizes = [a["tokens"], a["hq"], a["hk"], a["d"], a["rot"], a["most"], a["inter"]]
    if bwd:
        return lib.kda_qk_norm_rope_bwd(a["qo"], a["ko"], a["q"], a["k"], a["qs"], a["ks"], *common, a["dq"], a["dk"], a["dwq"], a["dwk"],
                                        *sizes, a["ws"], a["ws_bytes"], None)
    if append:
        return lib.kda_kv_append(a["q"], a["k"], a["v"], a["qs"], a["ks"], a["vs"], *common, a["qo"], a["kc"], a["vc"], a["ksc"],
                                 a["vsc"], a["slots"], *sizes, a["pages"], a["page"], a["kstep"], a["vstep"], a["ws"], None)
    return lib.kda_qk_norm_rope(a["q"], a["k"], a["qs"], a["ks"], *common, a["qo"], a["ko"], *sizes, a["ws"], None)


ROPE_BAD = [
    (dict(d=24), UNSUPPORTED), (dict(d=144, qs=4096, ks=4096), UNSUPPORTED), (dict(d=0), UNSUPPORTED),
    (dict(rot=8), UNSUPPORTED), (dict(rot=144), UNSUPPORTED), (dict(rot=-16), UNSUPPORTED),
    (dict(tokens=-1), INVALID), (dict(tokens=1 << 31), INVALID), (dict(hq=-1), INVALID), (dict(hk=1 << 17), INVALID),
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(q=P + 8), INVALID), (dict(k=P + 2), INVALID), (dict(qo=None), INVALID),
    (dict(qs=1023), INVALID), (dict(qs=1016), INVALID), (dict(ks=255), INVALID), (dict(qs=2044), INVALID),
    (dict(tab=None), INVALID), (dict(pos=None), INVALID), (dict(tab=P + 4), INVALID), (dict(pos=P + 2), INVALID), (dict(most=-1), INVALID),
    (dict(wq=P + 4), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID),
    (dict(inter=2), INVALID), (dict(ws=P + 16), INVALID),
    (dict(tokens=(1 << 31) - 1, hq=65535, qs=1 << 23), INVALID),
]


@pytest.mark.parametrize("kw,status", ROPE_BAD, ids=lambda x: str(x))
def test_rope_refusals(lib, kw, status):
    assert rope(lib, **kw) == status
    assert rope(lib, bwd=True, **kw) == status
    assert rope(lib, append=True, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(dq=None), INVALID), (dict(dk=P + 4), INVALID), (dict(dwq=None), INVALID), (dict(wk=None), INVALID), (dict(dwk=P + 1), INVALID),
    (dict(ws=None), INVALID), (dict(ws_bytes=4096), SMALL)])
def test_rope_bwd_refusals(lib, kw, status):
    assert rope(lib, bwd=True, **kw) == status


CACHE_BAD = [
    (dict(page=4), UNSUPPORTED), (dict(page=24), UNSUPPORTED), (dict(page=2048), UNSUPPORTED), (dict(pages=0), INVALID),
    (dict(pages=1 << 27, page=16), INVALID), (dict(kc=None), INVALID), (dict(vc=P + 8), INVALID),
    (dict(ksc=P), INVALID), (dict(vsc=P), INVALID), (dict(ksc=P + 2, vsc=P), INVALID),
    (dict(kstep=2 * 16 * 128 - 8), INVALID), (dict(vstep=2 * 16 * 128 + 4), INVALID),
    (dict(ksc=P, vsc=P, kstep=2 * 16 * 128 + 8), INVALID), (dict(kstep=1 << 38), INVALID),
]


@pytest.mark.parametrize("kw,status", CACHE_BAD + [(dict(v=None), INVALID), (dict(vs=100), INVALID), (dict(slots=None), INVALID),
                                                   (dict(slots=P + 1), INVALID), (dict(hk=0), INVALID)], ids=lambda x: str(x))
def test_append_refusals(lib, kw, status):
    assert rope(lib, append=True, **kw) == status


def read(lib, **kw):
    a = dict(kc=P, vc=P, ksc=None, vsc=None, tab=P, cu=P, ko=P, vo=P, n=2, total=10, hk=2, d=128, pages=4, page=16, wide=3,
             kstep=2 * 16 * 128, vstep=2 * 16 * 128, ws=P)
    a.update(kw)
    return lib.kda_kv_read(a["kc"], a["vc"], a["ksc"], a["vsc"], a["tab"], a["cu"], a["ko"], a["vo"], a["n"], a["total"], a["hk"],
                           a["d"], a["pages"], a["page"], a["wide"], a["kstep"], a["vstep"], a["ws"], None)


@pytest.mark.parametrize("kw,status", CACHE_BAD + [
    (dict(d=40), UNSUPPORTED), (dict(n=-1), INVALID), (dict(total=-1), INVALID), (dict(total=1 << 31), INVALID), (dict(wide=-1), INVALID),
    (dict(wide=1 << 28), INVALID), (dict(cu=None), INVALID), (dict(tab=None), INVALID), (dict(ko=None), INVALID), (dict(vo=P + 8), INVALID),
    (dict(ws=P + 4), INVALID), (dict(hk=0), INVALID)], ids=lambda x: str(x))
def test_read_refusals(lib, kw, status):
    assert read(lib, **kw) == status


def decode(lib, **kw):
    a = dict(q=P, kc=P, vc=P, ksc=None, vsc=None, tab=P, lens=P, scale=0.1, softcap=0.0, window=0, out=2 * P, lse=None, b=2, new=1,
             hq=8, hk=2, d=128, pages=4, page=16, wide=3, kstep=2 * 16 * 128, vstep=2 * 16 * 128, ws=P, ws_bytes=1 << 30)
    a.update(kw)
    return lib.kda_attn_decode(a["q"], a["kc"], a["vc"], a["ksc"], a["vsc"], a["tab"], a["lens"], a["scale"], a["softcap"], a["window"],
                               a["out"], a["lse"], a["b"], a["new"], a["hq"], a["hk"], a["d"], a["pages"], a["page"], a["wide"],
                               a["kstep"], a["vstep"], a["ws"], a["ws_bytes"], None)


@pytest.mark.parametrize("kw,status", CACHE_BAD + [
    (dict(d=136), UNSUPPORTED), (dict(d=8), UNSUPPORTED), (dict(b=-1), INVALID), (dict(new=-1), INVALID), (dict(hq=7), INVALID),
    (dict(hq=0), INVALID), (dict(hk=0), INVALID), (dict(wide=-1), INVALID), (dict(wide=1 << 27), INVALID), (dict(window=-1), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID), (dict(softcap=-1.0), INVALID),
    (dict(softcap=float("inf")), INVALID), (dict(softcap=1e-40, scale=1.0), INVALID), (dict(q=None), INVALID), (dict(q=P + 8), INVALID),
    (dict(out=None), INVALID), (dict(out=P), INVALID), (dict(lse=P + 2), INVALID), (dict(lens=None), INVALID), (dict(tab=None), INVALID),
    (dict(tab=P + 2), INVALID), (dict(ws=None), INVALID), (dict(ws=P + 128), INVALID), (dict(ws_bytes=1000), SMALL),
    (dict(new=1 << 20), INVALID), (dict(b=1 << 30, new=2), INVALID), (dict(b=(1 << 31) - 1), INVALID)], ids=lambda x: str(x))
def test_decode_refusals(lib, kw, status):
    assert decode(lib, **kw) == status


def test_workspace_sizes(lib):
    assert lib.kda_qk_norm_rope_bwd_workspace_size() >= 256 + 296 * 128 * 4  # a partial sum for each of two CTAs on 148 SMs
    size = kda.attn_decode_workspace_size
    # two partial results of a unit's rows (at most 16 at a time) for each of at least two CTAs on each of 148 SMs
    assert size(1, 32, 8, 128) >= 256 + 2 * 296 * 4 * (128 + 2) * 4
    assert size(4, 32, 8, 128) >= 256 + 2 * 296 * 16 * (128 + 2) * 4
    assert size(20, 32, 8, 64) >= 256 + 2 * 296 * 16 * (64 + 2) * 4
    assert size(1, 7, 2, 128) == size(0, 8, 8, 128) == size(1, 8, 8, 72) == 256


def test_binding_checks_its_tensors(lib):
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    cache = torch.zeros(2, 2, 16, 64, dtype=torch.bfloat16)
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        kda.qk_norm_rope(x, x)  # not on a GPU
    with pytest.raises(ValueError):
        kda.qk_norm_rope_bwd(x, x, x, x)
    with pytest.raises(ValueError):
        kda.kv_append(x, x, cache, cache, i)
    with pytest.raises(ValueError):
        kda.kv_read(cache, cache, i.view(1, 4), i[:2], x, x)
    with pytest.raises(ValueError):
        kda.attn_decode(x, cache, cache, i.view(4, 1), i, 1.0)
