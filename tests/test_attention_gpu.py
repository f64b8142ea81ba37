"""The softmax-attention operators (norm + rotation and its gradient, the paged cache's write and read,
decode attention) against their formulas in 64 bits (attention_ref.py, which derives the tolerances)."""
import math

import pytest
import torch

import attention_ref as ref
import kimi_delta_attention_24_b200 as kda

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
F8 = torch.float8_e4m3fn


def dev(*ts):
    out = [None if t is None else t.cuda() for t in ts]
    return out if len(out) > 1 else out[0]


def within(got, want, tol, what):
    got = got.double().cpu()
    same = (got == want) | (torch.isnan(got) & torch.isnan(want))
    bad = ~(same | ((got - want).abs() <= tol))
    if bad.any():
        i = tuple(int(x) for x in bad.nonzero()[0])
        over = ((got - want).abs() / tol)[bad].max()
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {i}: got {got[i]}, want {want[i]} "
                             f"+- {tol[i]}, worst {over} tolerances")


def bits(t):
    return t.contiguous().view(torch.uint8)


# ------------------------------------------------------------------------------------ norm and rotation
ROPE = [
    # tokens, hq, hk, d, rot, interleaved, norm q, norm k
    (1, 1, 1, 128, 128, False, True, True),
    (1, 32, 8, 128, 128, True, True, True),
    (7, 5, 3, 16, 16, False, True, True),
    (33, 9, 2, 80, 80, True, True, True),
    (33, 4, 4, 80, 48, False, True, False),
    (129, 12, 12, 96, 96, False, True, True),
    (65, 3, 1, 64, 32, True, False, True),
    (64, 8, 2, 112, 0, False, True, True),
    (17, 6, 6, 48, 16, False, False, False),
    (300, 13, 7, 128, 64, False, True, True),
    # more items than a full device takes at once: one head group per item, and several
    (5003, 5, 1, 128, 64, True, True, True),
    (1601, 64, 16, 96, 96, False, True, True),
    (9001, 3, 1, 48, 32, False, True, True),
]


def rope_inputs(case, seed, strided=True):
    tokens, hq, hk, d, rot, inter, nq, nk = case
    g = torch.Generator().manual_seed(seed)
    qkv = torch.randn(tokens, hq + 2 * hk, d, generator=g).to(BF)
    w = lambda on: (1 + 0.3 * torch.randn(d, generator=g)) if on else None
    wq, wk = w(nq), w(nk)
    tab = ref.table(rot, 5000) if rot else None
    pos = torch.randint(0, 5000, (tokens,), generator=g, dtype=torch.int32) if rot else None
    return qkv, wq, wk, tab, pos


@pytest.mark.parametrize("case", ROPE, ids=lambda c: "-".join(str(int(x)) for x in c))
def test_norm_rope(cuda_device, case):
    tokens, hq, hk, d, rot, inter, *_ = case
    qkv, wq, wk, tab, pos = rope_inputs(case, 1)
    x = qkv.cuda()
    q, k = x[:, :hq], x[:, hq:hq + hk]
    qo, ko = kda.qk_norm_rope(q, k, *dev(wq, wk), 1e-6, *dev(tab, pos), interleaved=inter)
    for got, src, w, what in ((qo, qkv[:, :hq], wq, "q"), (ko, qkv[:, hq:hq + hk], wk, "k")):
        y, mag = ref.norm_rope(src, w, 1e-6, tab, pos, inter)
        within(got, y, ref.norm_rope_tol(y, mag), what)
    # one of the two alone, contiguous, in place: the same bits
    qc = q.contiguous()
    only, none = kda.qk_norm_rope(qc, None, *dev(wq, None), 1e-6, *dev(tab, pos), interleaved=inter, q_out=qc)
    assert none is None and only is qc and torch.equal(bits(qc), bits(qo))
    none, only = kda.qk_norm_rope(None, k, *dev(None, wk), 1e-6, *dev(tab, pos), interleaved=inter)
    assert none is None and torch.equal(bits(only), bits(ko))


def test_norm_rope_special_rows(cuda_device):
    """Zero rows, rows with infinities and NaN, tiny rows: what the formula gives, and only there."""
    d = 128
    x = torch.randn(8, 2, d, generator=torch.Generator().manual_seed(3)).to(BF)
    x[0] = 0
    x[1, 0, 5] = math.inf
    x[2, 1, 127] = math.nan
    x[3] = 1e-30
    tab, pos = ref.table(d, 64), torch.arange(8, dtype=torch.int32)
    w = torch.ones(d)
    out, _ = kda.qk_norm_rope(x.cuda(), None, w.cuda(), None, 1e-6, *dev(tab, pos))
    y, mag = ref.norm_rope(x, w, 1e-6, tab, pos, False)
    got = out.cpu().double()
    assert torch.equal(got[0], torch.zeros(2, d, dtype=torch.float64))
    assert torch.isnan(got[1, 0]).any() and torch.isnan(got[2, 1]).all()
    rest = torch.ones(8, 2, dtype=torch.bool)
    rest[1, 0] = rest[2, 1] = False
    within(out.cpu()[rest], y[rest], ref.norm_rope_tol(y, mag)[rest], "rest")


def test_norm_rope_skips_positions_out_of_range(cuda_device):
    d, tab = 64, ref.table(64, 10)
    x = torch.randn(4, 3, d).to(BF).cuda()
    pos = torch.tensor([9, 10, -1, 0], dtype=torch.int32).cuda()
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    out = torch.full_like(x, 7.0)
    kda.qk_norm_rope(x, None, None, None, 1e-6, tab.cuda(), pos, q_out=out, workspace=ws)
    assert kda.read_device_status(ws) == 1 and kda.read_device_status(ws) == 0
    assert (out[1:3] == 7).all() and not (out[0] == 7).any() and torch.equal(out[3], x[3])


@pytest.mark.parametrize("case", ROPE, ids=lambda c: "-".join(str(int(x)) for x in c))
def test_norm_rope_bwd(cuda_device, case):
    tokens, hq, hk, d, rot, inter, *_ = case
    qkv, wq, wk, tab, pos = rope_inputs(case, 2)
    g = torch.Generator().manual_seed(4)
    gq, gk = torch.randn(tokens, hq, d, generator=g).to(BF), torch.randn(tokens, hk, d, generator=g).to(BF)
    x = qkv.cuda()
    r = kda.qk_norm_rope_bwd(*dev(gq, gk), x[:, :hq], x[:, hq:hq + hk], *dev(wq, wk), 1e-6, *dev(tab, pos), interleaved=inter)
    again = kda.qk_norm_rope_bwd(*dev(gq, gk), x[:, :hq], x[:, hq:hq + hk], *dev(wq, wk), 1e-6, *dev(tab, pos), interleaved=inter)
    for n, src, w, dy in (("q", qkv[:, :hq], wq, gq), ("k", qkv[:, hq:hq + hk], wk, gk)):
        dx, dw, dx_tol, dw_tol = ref.norm_rope_bwd(src, w, 1e-6, tab, pos, inter, dy)
        within(r["d" + n], dx, dx_tol, "d" + n)
        assert torch.equal(bits(r["d" + n]), bits(again["d" + n]))
        if w is None:
            assert r[f"d{n}_weight"] is None
        else:
            within(r[f"d{n}_weight"], dw, dw_tol, f"d{n}_weight")
            assert torch.equal(r[f"d{n}_weight"], again[f"d{n}_weight"])


def test_norm_rope_bwd_of_no_token(cuda_device):
    z = torch.empty(0, 2, 64, dtype=BF, device="cuda")
    w = torch.ones(64, device="cuda")
    r = kda.qk_norm_rope_bwd(z, z, z, z, w, w)
    assert r["dq"].shape == z.shape and not r["dq_weight"].any() and not r["dk_weight"].any()
    q, k = kda.qk_norm_rope(z, z, w, w)
    assert q.shape == z.shape and k.shape == z.shape


def test_norm_rope_bwd_against_differences():
    """The formula's gradient (which the kernel is held to) against central differences in 64 bits."""
    g = torch.Generator().manual_seed(5)
    tokens, h, d = 3, 2, 32
    x = torch.randn(tokens, h, d, generator=g, dtype=torch.float64)
    w = 1 + 0.3 * torch.randn(d, generator=g, dtype=torch.float64)
    dy = torch.randn(tokens, h, d, generator=g, dtype=torch.float64)
    pos = torch.tensor([0, 3, 17], dtype=torch.int32)
    for inter in (False, True):
        tab = ref.table(16, 20)
        dx, dw, _, _ = ref.norm_rope_bwd(x, w, 1e-6, tab, pos, inter, dy)
        f = lambda x, w: (ref.norm_rope(x, w, 1e-6, tab, pos, inter)[0] * dy).sum()
        for _ in range(3):
            ux, uw = torch.randn(x.shape, generator=g, dtype=torch.float64), torch.randn(d, generator=g, dtype=torch.float64)
            e = 1e-5
            diff = (f(x + e * ux, w + e * uw) - f(x - e * ux, w - e * uw)) / (2 * e)
            want = (dx * ux).sum() + (dw * uw).sum()
            assert abs(diff - want) <= 1e-6 * (1 + abs(want))


# ------------------------------------------------------------------------------------ the cache
@pytest.mark.parametrize("quant", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("case,page", [(ROPE[0], 8), (ROPE[1], 16), (ROPE[2], 64), (ROPE[3], 32), (ROPE[4], 16), (ROPE[6], 128),
                                       (ROPE[7], 8), (ROPE[8], 1024), (ROPE[9], 16),
                                       (ROPE[10], 16), (ROPE[11], 64), (ROPE[12], 8)], ids=lambda c: str(c).replace(" ", ""))
def test_append(cuda_device, case, page, quant):
    tokens, hq, hk, d, rot, inter, *_ = case
    qkv, wq, wk, tab, pos = rope_inputs(case, 6)
    gen = torch.Generator().manual_seed(7)
    pages = -(-tokens // page) + 2
    kc, ks = ref.make_cache(gen, pages, hk, page, d, quant, fill=3.0)
    vc, vs = ref.make_cache(gen, pages, hk, page, d, quant, fill=3.0)
    slots = torch.randperm(pages * page, generator=gen)[:tokens].to(torch.int32)
    if tokens > 4:
        slots[2] = -1
        slots[tokens - 1] = -7
    x = qkv.cuda()
    kcd, vcd, ksd, vsd = dev(kc, vc, ks, vs)
    q_out = torch.full((tokens, hq, d), 9.0, dtype=BF, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    got = kda.kv_append(x[:, hq:hq + hk], x[:, hq + hk:], kcd, vcd, slots.cuda(), k_scale=ksd, v_scale=vsd, q=x[:, :hq],
                        q_out=q_out, q_weight=dev(wq), k_weight=dev(wk), cos_sin=dev(tab), positions=dev(pos), interleaved=inter,
                        workspace=ws)
    assert got is q_out and kda.read_device_status(ws) == 0
    on = slots >= 0
    y, mag = ref.norm_rope(qkv[:, :hq], wq, 1e-6, tab, pos, inter)
    within(q_out.cpu()[on], y[on], ref.norm_rope_tol(y, mag)[on], "q")
    assert (q_out.cpu()[~on] == 9).all()
    at = slots[on].long()
    p, r = at // page, at % page
    ky, kmag = (t[on] for t in ref.norm_rope(qkv[:, hq:hq + hk], wk, 1e-6, tab, pos, inter))
    v = qkv[:, hq + hk:][on]
    kn, vn = kcd.cpu(), vcd.cpu()
    if not quant:
        within(kn[p, :, r], ky, ref.norm_rope_tol(ky, kmag), "k")
        assert torch.equal(bits(vn[p, :, r]), bits(v))
    else:
        codes, scales = ref.quantise(v.float())
        assert torch.equal(vsd.cpu()[p, :, r], scales)
        assert torch.equal(bits(vn[p, :, r]), bits(codes))
        s = ksd.cpu().double()[p, :, r]
        want = (ky.abs().amax(-1) / 448).clamp(min=ref.SCALE_FLOOR)
        # a scale is as exact as the row's largest value and one division; a code half a step from the
        # quotient (2^-4 of it, 2^-10 where the steps are even), which the chain and the scale move a little
        stol = (ref.CHAIN * kmag.amax(-1) / 448) + 2 * ref.F32 * want
        assert ((s - want).abs() <= stol).all()
        vals = kn[p, :, r].float().double() * s[..., None]
        within(vals, ky, (ref.E4M3 * ky.abs() + 2.0 ** -10 * want[..., None]) * (1 + 2.0 ** -8) + 2 * ref.CHAIN * kmag, "k values")
    # every other row stayed as it was
    for now, was in ((kn, kc), (vn, vc)) + (((ksd.cpu(), ks), (vsd.cpu(), vs)) if quant else ()):
        keep = torch.ones(pages, now.shape[1], page, dtype=torch.bool)
        keep[p, :, r] = False
        assert torch.equal(bits(now)[..., :].view(pages, now.shape[1], page, -1)[keep],
                           bits(was)[..., :].view(pages, now.shape[1], page, -1)[keep])


def test_append_special_rows(cuda_device):
    """Zero and tiny rows quantise to their values, rows with an infinity or NaN read back as NaN."""
    d, page = 64, 16
    v = torch.randn(6, 2, d).to(BF)
    v[0] = 0
    v[1] = 1e-38
    v[2, 0, 3] = math.inf
    v[3, 1, 0] = math.nan
    v[4] = 3e38
    k = torch.zeros_like(v)
    kc, ks = ref.make_cache(None, 2, 2, page, d, True)
    vc, vs = ref.make_cache(None, 2, 2, page, d, True)
    kc, ks, vc, vs = dev(kc, ks, vc, vs)
    kda.kv_append(*dev(k, v), kc, vc, torch.arange(10, 16, dtype=torch.int32).cuda(), k_scale=ks, v_scale=vs)
    out_k, out_v = torch.zeros(16, 2, d, dtype=BF, device="cuda"), torch.zeros(16, 2, d, dtype=BF, device="cuda")
    kda.kv_read(kc, vc, torch.zeros(1, 1, dtype=torch.int32).cuda(), torch.tensor([0, 16], dtype=torch.int32).cuda(), out_k,
                out_v, k_scale=ks, v_scale=vs)
    got = out_v.cpu()[10:]
    assert (got[0] == 0).all() and (got[1] == 0).all()  # (1e-38 / 2^-64 is below the smallest code)
    assert torch.isnan(got[2, 0]).all() and not torch.isnan(got[2, 1]).any()
    assert torch.isnan(got[3, 1]).all() and not torch.isnan(got[3, 0]).any()
    assert (got[4] == v[4]).all() or ((got[4].double() - v[4].double()).abs() <= 2 * ref.BF16 * v[4].double().abs()).all()
    assert (out_k.cpu()[10:] == 0).all()


def test_append_skips_bad_slots_and_positions(cuda_device):
    d, page = 64, 8
    kc = torch.zeros(2, 1, page, d, dtype=BF, device="cuda")
    vc = torch.zeros_like(kc)
    k = torch.ones(4, 1, d, dtype=BF, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    kda.kv_append(k, k, kc, vc, torch.tensor([3, 16, 15, 4], dtype=torch.int32).cuda(), cos_sin=ref.table(64, 5).cuda(),
                  positions=torch.tensor([0, 0, 5, 4], dtype=torch.int32).cuda(), workspace=ws)
    assert kda.read_device_status(ws) == 1
    wrote = (vc.view(16, d) != 0).any(-1)
    assert wrote.nonzero().flatten().tolist() == [3, 4]


@pytest.mark.parametrize("quant", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("d,hk,page", [(16, 1, 8), (64, 3, 16), (80, 2, 64), (128, 8, 16)])
def test_read(cuda_device, d, hk, page, quant):
    gen = torch.Generator().manual_seed(8)
    lens = [0, 1, page - 1, page, 0, page + 1, 3 * page + 5, 0]
    pages = sum(-(-n // page) for n in lens) + 1
    kc, ks = ref.make_cache(gen, pages, hk, page, d, quant)
    vc, vs = ref.make_cache(gen, pages, hk, page, d, quant)
    tab = ref.fill_sequences(gen, lens, kc, vc, ks, vs)
    cu = torch.tensor([0] + lens, dtype=torch.int32).cumsum(0).to(torch.int32)
    total = int(cu[-1]) + 3
    k_out, v_out = (torch.full((total, hk, d), 5.0, dtype=BF, device="cuda") for _ in range(2))
    kcd, vcd, ksd, vsd = dev(kc, vc, ks, vs)
    kda.kv_read(kcd, vcd, tab.cuda(), cu.cuda(), k_out, v_out, k_scale=ksd, v_scale=vsd)
    for out, cache, scale in ((k_out, kc, ks), (v_out, vc, vs)):
        want = torch.cat([ref.cached_rows(cache, scale, tab[b, :-(-n // page)].long(), n) for b, n in enumerate(lens)])
        # the value of a code and its scale in fp32, rounded once (a product of 4 and 24 bits: rounded to fp32 first)
        assert torch.equal(bits(out.cpu()[:-3]), bits(want.float().to(BF)))
        assert (out[-3:] == 5).all()
    # offsets out of order, a sequence longer than its table, one beyond the rows: nothing is written
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    for bad in ([0, 5, 3, 3, 3, 3, 3, 3, 3], [1, 1, 1, 1, 1, 1, 1, 1, 1], [0] + [10000] * 8, [0] + [total + 1] * 8):
        k_out.fill_(5)
        kda.kv_read(kcd, vcd, tab.cuda(), torch.tensor(bad, dtype=torch.int32).cuda(), k_out, v_out, k_scale=ksd, v_scale=vsd,
                    workspace=ws)
        assert kda.read_device_status(ws) == 1 and (k_out == 5).all()
    # a page number out of range: its rows stay, the others are read
    wrong = tab.clone()
    wrong[6, 1] = pages
    kda.kv_read(kcd, vcd, wrong.cuda(), cu.cuda(), k_out, v_out, k_scale=ksd, v_scale=vsd, workspace=ws)
    assert kda.read_device_status(ws) == 1
    r0 = int(cu[6])
    assert (k_out[r0 + page:r0 + 2 * page] == 5).all() and not (k_out[r0:r0 + page] == 5).all()


@pytest.mark.parametrize("quant", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("d,hk,longest", [(64, 5, 9001), (128, 3, 9001), (80, 11, 3001), (128, 1, 30001), (128, 2, 30001), (64, 1, 30001),
                                          (48, 2, 30001), (64, 1, 9001), (64, 2, 9001), (128, 1, 9001)])
def test_read_many_rows(cuda_device, d, hk, longest, quant):
    """More rows than the groups of a full device; documents of odd lengths over shared random pages."""
    gen = torch.Generator().manual_seed(d)
    page, pages, lens = 16, 50, [longest, 0, 1999, 1, 0, 2, 16383]
    if quant:
        kc, vc = (torch.randint(0, 127, (pages, hk, page, d), generator=gen, dtype=torch.uint8).view(torch.float8_e4m3fn) for _ in range(2))
        ks, vs = (torch.rand(pages, hk, page, generator=gen) for _ in range(2))
    else:
        kc, vc = (torch.randn(pages, hk, page, d, generator=gen).to(BF) for _ in range(2))
        ks = vs = None
    tab = torch.randint(0, pages, (len(lens), 1876), generator=gen, dtype=torch.int32)
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32)
    total = int(cu[-1]) + 2
    k_out, v_out = (torch.full((total, hk, d), 9.0, dtype=BF, device="cuda") for _ in range(2))
    ksd, vsd = dev(ks, vs)
    kda.kv_read(kc.cuda(), vc.cuda(), tab.cuda(), cu.cuda(), k_out, v_out, k_scale=ksd, v_scale=vsd)
    for out, cache, scale in ((k_out, kc, ks), (v_out, vc, vs)):
        got = out.cpu()
        assert (got[-2:] == 9).all()
        for b, n in enumerate(lens):
            j = torch.arange(n)
            p, r = tab[b].long()[j // page], j % page
            want = cache[p, :, r] if scale is None else (cache[p, :, r].float() * scale[p, :, r][..., None]).to(BF)
            assert torch.equal(bits(got[int(cu[b]):int(cu[b + 1])]), bits(want))


# ------------------------------------------------------------------------------------ decode attention
def run_decode(lens, new, hk, group, d, page, quant, softcap=0.0, window=0, seed=11, extra=2, scale=None, max_pages=None,
               k_std=1.0, v_std=1.0, mutate=None, repeat=False):
    gen = torch.Generator().manual_seed(seed)
    first = [max(0, n - new - window + 1) if window else 0 for n in lens]
    pages = sum(-(-n // page) for n in lens) + extra
    kc, ks = ref.make_cache(gen, pages, hk, page, d, quant)
    vc, vs = ref.make_cache(gen, pages, hk, page, d, quant)
    tab = ref.fill_sequences(gen, lens, kc, vc, ks, vs, first=first, k_std=k_std, v_std=v_std, max_pages=max_pages)
    q = torch.randn(len(lens), new, hk * group, d, generator=gen).to(BF)
    scale = d ** -0.5 if scale is None else scale
    if mutate:
        mutate(q, kc, vc, ks, vs, tab)
    args = [t.cuda() if t is not None else None for t in (q, kc, vc, tab, torch.tensor(lens, dtype=torch.int32))]
    ksd, vsd = dev(ks, vs)
    lse = torch.full(q.shape[:3], 99.0, device="cuda")
    ws = torch.full((kda.attn_decode_workspace_size(new, hk * group, hk, d),), 255, dtype=torch.uint8, device="cuda")
    ws[:256].zero_()  # (the rest may hold anything)
    out = torch.full(q.shape, 99.0, dtype=BF, device="cuda")
    kda.attn_decode(*args, scale, out=out, lse=lse, k_scale=ksd, v_scale=vsd, softcap=softcap, window=window, workspace=ws)
    assert kda.read_device_status(ws) == 0
    o, l, ot, lt = ref.attention(q, kc, vc, tab, lens, scale, ks, vs, softcap, window)
    if max_pages is None and tab.shape[1] * page <= 1024:
        # a table wide enough for long sequences: few short units are not split over CTAs, these are
        args[3] = torch.nn.functional.pad(tab, (0, 1024 // page + 1 - tab.shape[1]), value=-1).cuda()
        lse2 = torch.full(q.shape[:3], 99.0, device="cuda")
        out2 = kda.attn_decode(*args, scale, lse=lse2, k_scale=ksd, v_scale=vsd, softcap=softcap, window=window)
        assert torch.equal(torch.isfinite(out2).cpu(), torch.isfinite(o))
        rows = torch.isfinite(o).all(3)  # (where a seen value row is no number, lse may be none either)
        for got, want, tol, fine in ((out2, o, ot, torch.isfinite(o)), (lse2, l, lt, rows)):
            within(torch.where(fine, got.cpu().double(), 0.0), torch.where(fine, want, 0.0), torch.where(fine, tol, 1.0), "wide table")
        args[3] = tab.cuda()
    if repeat:
        o2 = kda.attn_decode(*args, scale, k_scale=ksd, v_scale=vsd, softcap=softcap, window=window)
        assert torch.equal(bits(o2), bits(out))
    return out, lse, o, l, ot, lt


def check_decode(*a, **k):
    out, lse, o, l, ot, lt = run_decode(*a, **k)
    within(out, o, ot, "out")
    within(lse, l, lt, "lse")


EDGE_LENS = [0, 1, 2, 3, 7, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 200, 257]


@pytest.mark.parametrize("quant", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("d", [16, 48, 64, 80, 112, 128])
@pytest.mark.parametrize("page", [8, 16, 64])
def test_decode_lengths(cuda_device, d, page, quant):
    check_decode(EDGE_LENS, 1, 2, 4, d, page, quant, repeat=True)


@pytest.mark.parametrize("quant", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("hk,group,new", [(1, 1, 1), (3, 1, 3), (1, 16, 1), (2, 5, 3), (1, 17, 1), (2, 8, 4), (1, 3, 16), (1, 16, 5),
                                          (1, 96, 1), (12, 1, 2)])
@pytest.mark.parametrize("d", [64, 128])
def test_decode_rows(cuda_device, hk, group, new, d, quant):
    check_decode([0, 1, 2, 5, 18, 64, 130], new, hk, group, d, 16, quant)


@pytest.mark.parametrize("quant", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 64, 100, 1000])
@pytest.mark.parametrize("new", [1, 4])
def test_decode_window(cuda_device, window, new, quant):
    """Pages and rows before the window are unwritten: the table there is -1, the rows NaN."""
    check_decode([0, 1, 3, 40, 64, 129, 300], new, 2, 3, 64, 16, quant, window=window)


@pytest.mark.parametrize("quant", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("softcap", [0.5, 30.0])
def test_decode_softcap(cuda_device, softcap, quant):
    check_decode([1, 20, 150], 2, 2, 4, 128, 32, quant, softcap=softcap, k_std=4.0)


@pytest.mark.parametrize("quant", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("d", [64, 128])
def test_decode_split_and_joined(cuda_device, d, quant):
    """One long sequence over every CTA of the device, beside short ones; then several long ones."""
    check_decode([9000, 3, 0, 70], 1, 1, 8, d, 16, quant, repeat=True)
    check_decode([2500, 1, 3100, 2047], 2, 2, 2, d, 64, quant, repeat=True)
    check_decode([4000], 3, 1, 12, d, 32, quant)  # two row blocks
    check_decode([5000, 1200], 1, 2, 4, d, 16, quant, window=2000)


@pytest.mark.parametrize("quant", [False, True], ids=["bf16", "e4m3"])
def test_decode_peaked_and_large_scores(cuda_device, quant):
    check_decode([700, 33], 1, 1, 4, 128, 16, quant, k_std=30.0)      # nearly one key takes all
    check_decode([700, 33], 1, 1, 4, 128, 16, quant, scale=0.0)       # all keys alike
    check_decode([700, 33], 1, 1, 4, 64, 16, quant, scale=-0.2, v_std=1e4)
    check_decode([300], 1, 1, 4, 64, 16, quant, k_std=1e-6, v_std=1e-8)


def test_decode_scales_far_apart(cuda_device):
    """Value rows whose magnitudes differ by 2^40: the weights of both kinds keep their bits."""
    def mutate(q, kc, vc, ks, vs, tab):
        ok = ~torch.isnan(vs)
        flip = torch.rand(vs.shape, generator=torch.Generator().manual_seed(1)) < 0.5
        vs[ok & flip] *= 2.0 ** -40
        q *= 0.1
    check_decode([500, 77], 1, 2, 4, 128, 16, True, mutate=mutate)
    def all_small(q, kc, vc, ks, vs, tab):
        vs[~torch.isnan(vs)] *= 2.0 ** -50
    check_decode([500, 77], 1, 2, 4, 64, 16, True, mutate=all_small)


def test_decode_small_queries(cuda_device):
    """Queries far below and above fp16's range keep their bits against an e4m3 cache."""
    for f in (1e-12, 1e-6, 1e6, 1e12):
        def mutate(q, kc, vc, ks, vs, tab):
            q *= f
        check_decode([200, 17], 1, 1, 4, 128, 16, True, mutate=mutate, scale=128 ** -0.5 / f)


@pytest.mark.parametrize("d", [64, 128])
def test_decode_nonfinite_values_in_unseen_rows(cuda_device, d):
    """Infinities and NaN in value rows reach the queries that see them and no other (new tokens, window)."""
    lens, new, window = [40, 129, 6], 4, 20
    def mutate(q, kc, vc, ks, vs, tab):
        for b, n in enumerate(lens):
            for j, x in ((n - 1, math.inf), (n - 2, math.nan), (max(0, n - new - window + 1), -math.inf)):
                vc[int(tab[b, j // 16]), :, j % 16, 3] = x
                kc[int(tab[b, j // 16]), 0, j % 16, 5] = kc[int(tab[b, j // 16]), 0, j % 16, 5]
    out, lse, o, l, ot, lt = run_decode(lens, new, 2, 3, d, 16, False, window=window, mutate=mutate)
    got = out.cpu().double()
    assert torch.equal(torch.isfinite(got), torch.isfinite(o))
    fine = torch.isfinite(o)
    within(torch.where(fine, got, 0.0), torch.where(fine, o, 0.0), torch.where(fine, ot, 1.0), "finite rows")
    within(lse, l, lt, "lse")


@pytest.mark.parametrize("quant", [False, True], ids=["bf16", "e4m3"])
def test_decode_nonfinite_rows_that_are_seen(cuda_device, quant):
    def mutate(q, kc, vc, ks, vs, tab):
        if quant:
            vs[int(tab[0, 0]), 0, 2] = math.nan   # as kv_append marks such a row
        else:
            kc[int(tab[0, 0]), 0, 2, 1] = math.nan
    out, *_ , o, l, ot, lt = run_decode([50, 60], 1, 2, 2, 64, 16, quant, mutate=mutate)
    got = out.cpu().double()
    assert torch.isnan(got[0, 0, :2]).all()
    within(got[0, 0, 2:], o[0, 0, 2:], ot[0, 0, 2:], "other head")
    within(got[1], o[1], ot[1], "other sequence")


@pytest.mark.parametrize("quant", [False, True], ids=["bf16", "e4m3"])
def test_decode_shared_pages_and_page_strides(cuda_device, quant):
    """Sequences that share their first pages; K and V side by side in one pool of pages."""
    gen = torch.Generator().manual_seed(21)
    hk, page, d, pages = 2, 16, 64, 9
    kc, ks = ref.make_cache(gen, pages, hk, page, d, quant)
    vc, vs = ref.make_cache(gen, pages, hk, page, d, quant)
    tab = ref.fill_sequences(gen, [6 * 16], kc, vc, ks, vs)
    table = torch.stack([tab[0], tab[0].flip(0), tab[0]])
    lens = [90, 96, 40]
    pool = torch.stack([kc.view(torch.uint8), vc.view(torch.uint8)], 1).cuda()
    kcd, vcd = pool[:, 0].view(kc.dtype), pool[:, 1].view(vc.dtype)
    assert kcd.stride(0) == 2 * hk * page * d
    q = torch.randn(3, 1, 4, d, generator=gen).to(BF)
    ksd, vsd = dev(ks, vs)
    out = kda.attn_decode(q.cuda(), kcd, vcd, table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), 0.125, k_scale=ksd, v_scale=vsd)
    o, _, ot, _ = ref.attention(q, kc, vc, table, lens, 0.125, ks, vs)
    within(out, o, ot, "out")
    k_out, v_out = (torch.empty(90, hk, d, dtype=BF, device="cuda") for _ in range(2))
    kda.kv_read(kcd, vcd, table[:1].cuda(), torch.tensor([0, 90], dtype=torch.int32).cuda(), k_out, v_out, k_scale=ksd, v_scale=vsd)
    assert torch.equal(bits(v_out.cpu()), bits(ref.cached_rows(vc, vs, tab[0].long(), 90).float().to(BF)))


@pytest.mark.parametrize("quant", [False, True], ids=["bf16", "e4m3"])
def test_offsets_beyond_32_bits(cuda_device, quant):
    """A pool of more than 2^31 elements (2^32 for e4m3): its last pages are written, read and attended to."""
    hk, page, d = 8, 64, 128
    per_page = hk * page * d
    pages = (1 << (32 if quant else 31)) // per_page + 40
    dt = F8 if quant else BF
    kc = torch.zeros(pages, hk, page, d, dtype=torch.uint8 if quant else BF, device="cuda").view(dt)
    vc = torch.zeros(pages, hk, page, d, dtype=torch.uint8 if quant else BF, device="cuda").view(dt)
    ks, vs = (torch.zeros(pages, hk, page, device="cuda") if quant else None for _ in range(2))
    n = 100
    table = torch.tensor([[pages - 1, pages - 3]], dtype=torch.int32)
    j = torch.arange(n)
    slots = (table[0, j // page].long() * page + j % page).to(torch.int32)
    gen = torch.Generator().manual_seed(5)
    k, v, q = (torch.randn(n, h, d, generator=gen).to(BF) for h in (hk, hk, 16))
    kda.kv_append(*dev(k, v), kc, vc, slots.cuda(), k_scale=ks, v_scale=vs)
    k_out, v_out = (torch.empty(n, hk, d, dtype=BF, device="cuda") for _ in range(2))
    kda.kv_read(kc, vc, table.cuda(), torch.tensor([0, n], dtype=torch.int32).cuda(), k_out, v_out, k_scale=ks, v_scale=vs)
    if quant:
        codes, sc = ref.quantise(v.float())
        assert torch.equal(bits(v_out.cpu()), bits((codes.float() * sc[..., None]).to(BF)))
    else:
        assert torch.equal(bits(v_out.cpu()), bits(v)) and torch.equal(bits(k_out.cpu()), bits(k))
    out = kda.attn_decode(q[:1].cuda(), kc, vc, table.cuda(), torch.tensor([n], dtype=torch.int32).cuda(), d ** -0.5, k_scale=ks, v_scale=vs)
    last = table[0].long()
    small_k, small_v = kc[last.cuda()].cpu(), vc[last.cuda()].cpu()
    sk, sv = (None if t is None else t[last.cuda()].cpu() for t in (ks, vs))
    o, _, ot, _ = ref.attention(q[:1, None], small_k, small_v, torch.tensor([[0, 1]], dtype=torch.int32), [n], d ** -0.5, sk, sv)
    within(out, o[:, 0], ot[:, 0], "out")


def test_decode_many_sequences(cuda_device):
    """More units than CTAs, and a batch longer than the block that scans the lengths."""
    gen = torch.Generator().manual_seed(9)
    lens = torch.randint(0, 40, (700,), generator=gen).tolist()
    lens[300] = 150
    check_decode(lens, 1, 2, 1, 16, 8, False)


@pytest.mark.parametrize("b,hk", [(147, 1), (148, 1), (149, 1), (74, 2), (511, 1), (512, 1), (513, 1), (600, 8)])
def test_decode_batches_where_the_form_changes(cuda_device, b, hk):
    """A unit per SM and one more; the lengths that fit shared memory and one more; beyond them with a share per warp."""
    gen = torch.Generator().manual_seed(b)
    lens = torch.randint(0, 30, (b,), generator=gen).tolist()
    lens[b // 3] = 170
    check_decode(lens, 1, hk, 2, 16, 8, b % 2 == 1)


@pytest.mark.parametrize("quant", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("new,group", [(1, 4), (3, 4), (4, 6)])
def test_decode_short_window_in_long_sequences(cuda_device, new, group, quant):
    """Few units with few keys each although the tables are long: not split, from the window's first key on."""
    check_decode([5000, 1200, 3, 0, 2049], new, 2, group, 128, 16, quant, window=300)
    check_decode([1300, 4111], new, 1, group, 64, 64, quant, window=33)


@pytest.mark.parametrize("quant", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("d,new,group,window", [(64, 1, 1, 0), (128, 3, 2, 9), (128, 2, 6, 0), (48, 5, 5, 0)])
def test_decode_very_many_units(cuda_device, d, new, group, window, quant):
    """So many (sequence, kv head, rows) units that every warp takes a share of its own."""
    gen = torch.Generator().manual_seed(19)
    rows = new * group
    blocks = -(-rows // (8 if rows <= 8 else 16))
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    b = -(-4 * 4 * 2 * sms // (12 * blocks)) + 1
    lens = torch.randint(0, 20, (b,), generator=gen).tolist()
    lens[0], lens[b // 2], lens[-1] = 0, 300, 65
    # (the formulas over a few of the sequences: the shortest, the longest, and some others)
    gen2 = torch.Generator().manual_seed(11)
    pages = sum(-(-n // 16) for n in lens) + 2
    kc, ks = ref.make_cache(gen2, pages, 12, 16, d, quant)
    vc, vs = ref.make_cache(gen2, pages, 12, 16, d, quant)
    tab = ref.fill_sequences(gen2, lens, kc, vc, ks, vs)
    q = torch.randn(b, new, 12 * group, d, generator=gen2).to(BF)
    lse = torch.full(q.shape[:3], 99.0, device="cuda")
    ksd, vsd = dev(ks, vs)
    args = [t.cuda() for t in (q, kc, vc, tab, torch.tensor(lens, dtype=torch.int32))]
    out = kda.attn_decode(*args, 0.2, lse=lse, k_scale=ksd, v_scale=vsd, window=window)
    pick = sorted({0, 1, 2, b // 3, b // 2, b // 2 + 1, b - 2, b - 1})
    o, l, ot, lt = ref.attention(q[pick], kc, vc, tab[pick], [lens[i] for i in pick], 0.2, ks, vs, 0.0, window)
    within(out.cpu()[pick], o, ot, "out")
    within(lse.cpu()[pick], l, lt, "lse")
    # every other row: the call gives the same with the sequences one by one in a small batch
    few = torch.arange(3, b, max(1, b // 40))
    small = kda.attn_decode(args[0][few], args[1], args[2], args[3][few].contiguous(), args[4][few].contiguous(), 0.2, k_scale=ksd,
                            v_scale=vsd, window=window)
    # (the two forms add the same terms in other orders: a rounding of the result, and 2^-9 of P V's size)
    a, c = out[few].float(), small.float()
    assert ((a - c).abs() <= 2 * ref.BF16 * c.abs() + 2.0 ** -9 * vsize(vc, vs)).all()


def vsize(vc, vs):
    """The largest magnitude of a written value."""
    v = vc.float() if vs is None else vc.float() * vs[..., None]
    return float(v[torch.isfinite(v)].abs().max())


def test_decode_lengths_and_pages_out_of_range(cuda_device):
    gen = torch.Generator().manual_seed(2)
    kc, _ = ref.make_cache(gen, 8, 1, 16, 64, False)
    vc, _ = ref.make_cache(gen, 8, 1, 16, 64, False)
    tab = ref.fill_sequences(gen, [40, 20, 48], kc, vc, None, None, max_pages=3)
    q = torch.randn(3, 1, 2, 64, generator=gen).to(BF)
    ws = kda.new_attn_decode_workspace(1, 2, 1, 64, "cuda")
    args = lambda t, n: (q.cuda(), kc.cuda(), vc.cuda(), t.cuda(), torch.tensor(n, dtype=torch.int32).cuda(), 0.125)
    out = kda.attn_decode(*args(tab, [-5, 20, 1000]), workspace=ws)
    assert kda.read_device_status(ws) == 1
    o, _, ot, _ = ref.attention(q, kc, vc, tab, [0, 20, 48], 0.125)
    within(out, o, ot, "clamped lengths")
    bad = tab.clone()
    bad[0, 1] = 8
    out = kda.attn_decode(*args(bad, [40, 20, 48]), workspace=ws)
    assert kda.read_device_status(ws) == 1
    o, _, ot, _ = ref.attention(q, kc, vc, tab, [40, 20, 48], 0.125)
    within(out[1:], o[1:], ot[1:], "the other sequences")


def test_decode_empty_batch_and_no_pages(cuda_device):
    kc = torch.zeros(1, 1, 16, 64, dtype=BF, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    out = kda.attn_decode(torch.empty(0, 2, 64, dtype=BF, device="cuda"), kc, kc, torch.empty(0, 1, **i32), torch.empty(0, **i32), 1.0)
    assert out.shape == (0, 2, 64)
    lse = torch.zeros(2, 2, device="cuda")
    out = kda.attn_decode(torch.ones(2, 2, 64, dtype=BF, device="cuda"), kc, kc, torch.empty(2, 0, **i32), torch.zeros(2, **i32), 1.0, lse=lse)
    assert (out == 0).all() and (lse == -math.inf).all()


# ------------------------------------------------------------------------------------ streams and graphs
@pytest.mark.parametrize("quant", [False, True], ids=["bf16", "e4m3"])
def test_serving_steps_in_a_graph_beside_kda_decode(cuda_device, quant):
    """A hybrid model's decoding steps: a softmax layer (append, attend) and a KDA layer (its state pool)
    captured once and replayed, against the formulas over what the cache holds."""
    gen = torch.Generator().manual_seed(31)
    b, hk, group, d, page, steps = 3, 2, 4, 128, 16, 20
    hq = hk * group
    lens0 = [30, 1, 15]
    wide = 4
    kc, ks = ref.make_cache(gen, b * wide + 1, hk, page, d, quant)
    vc, vs = ref.make_cache(gen, b * wide + 1, hk, page, d, quant)
    tab = torch.randperm(b * wide + 1, generator=gen)[:b * wide].view(b, wide).to(torch.int32)
    kc, vc, ks, vs = dev(kc, vc, ks, vs)
    wq, wk = (1 + 0.1 * torch.randn(d, generator=gen) for _ in range(2))
    rope = ref.table(d, 128)
    # prefill: every sequence's first tokens, packed
    pos = torch.cat([torch.arange(n) for n in lens0])
    owner = torch.cat([torch.full((n,), i) for i, n in enumerate(lens0)])
    slot = lambda o, p: (tab[o, p // page] * page + p % page).to(torch.int32)
    qkv = torch.randn(len(pos), hq + 2 * hk, d, generator=gen).to(BF).cuda()
    kda.kv_append(qkv[:, hq:hq + hk], qkv[:, hq + hk:], kc, vc, slot(owner, pos).cuda(), k_scale=ks, v_scale=vs, k_weight=wk.cuda(),
                  cos_sin=rope.cuda(), positions=pos.to(torch.int32).cuda())
    # static buffers of one step
    sq = torch.zeros(b, hq + 2 * hk, d, dtype=BF, device="cuda")
    spos, sslot, slen = (torch.zeros(b, dtype=torch.int32, device="cuda") for _ in range(3))
    q_out = torch.zeros(b, hq, d, dtype=BF, device="cuda")
    out = torch.zeros(b, hq, d, dtype=BF, device="cuda")
    lse = torch.zeros(b, hq, device="cuda")
    ws = kda.new_attn_decode_workspace(1, hq, hk, d, "cuda")
    state = torch.zeros(b, hq, 128, 128, device="cuda")
    kq, kk, kv, kg = (torch.zeros(b, hq, 128, dtype=BF, device="cuda") for _ in range(4))
    kbeta, kout = torch.zeros(b, hq, dtype=BF, device="cuda"), torch.zeros(b, hq, 128, dtype=BF, device="cuda")
    A_log, dt = torch.zeros(hq, device="cuda"), torch.zeros(hq, 128, device="cuda")
    tabd, wqd, wkd, roped = dev(tab, wq, wk, rope)

    def step():
        kda.kv_append(sq[:, hq:hq + hk], sq[:, hq + hk:], kc, vc, sslot, k_scale=ks, v_scale=vs, q=sq[:, :hq], q_out=q_out,
                      q_weight=wqd, k_weight=wkd, cos_sin=roped, positions=spos)
        kda.attn_decode(q_out, kc, vc, tabd, slen, d ** -0.5, out=out, lse=lse, k_scale=ks, v_scale=vs, workspace=ws)
        kda.decode(kq, kk, kv, kg, kbeta, 128 ** -0.5, kout, A_log, dt, -5.0, state, state)

    sslot.fill_(-1)  # the warm-up writes nothing
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    state.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    kstate = state.clone()
    for i in range(steps):
        lens = [n + i + 1 for n in lens0]
        pos = torch.tensor(lens) - 1
        new = torch.randn(b, hq + 2 * hk, d, generator=gen).to(BF)
        sq.copy_(new)
        spos.copy_(pos.to(torch.int32))
        sslot.copy_(slot(torch.arange(b), pos))
        slen.copy_(torch.tensor(lens, dtype=torch.int32))
        kv.copy_(torch.randn(b, hq, 128, generator=gen).to(BF))
        kk.copy_(torch.randn(b, hq, 128, generator=gen).to(BF))
        graph.replay()
        y, mag = ref.norm_rope(new[:, :hq], wq, 1e-6, rope, pos, False)
        within(q_out, y, ref.norm_rope_tol(y, mag), f"q of step {i}")
        if i % 5 == 4:
            cpu = lambda t: None if t is None else t.cpu()
            o, l, ot, lt = ref.attention(q_out.cpu()[:, None], kc.cpu(), vc.cpu(), tab, lens, d ** -0.5, cpu(ks), cpu(vs))
            within(out, o[:, 0], ot[:, 0], f"out of step {i}")
            within(lse, l[:, 0], lt[:, 0], f"lse of step {i}")
    assert kda.read_device_status(ws) == 0 and not torch.equal(state, kstate)


def test_two_streams_at_once(cuda_device):
    """Two calls in flight on two streams, each with its own workspace, and calls that allocate on a side stream."""
    gen = torch.Generator().manual_seed(41)
    kc, _ = ref.make_cache(gen, 70, 2, 16, 64, False)
    vc, _ = ref.make_cache(gen, 70, 2, 16, 64, False)
    lens = [600, 300]
    tab = ref.fill_sequences(gen, lens, kc, vc, None, None)
    q = torch.randn(2, 1, 8, 64, generator=gen).to(BF)
    args = [t.cuda() for t in (q, kc, vc, tab, torch.tensor(lens, dtype=torch.int32))]
    want = kda.attn_decode(*args, 0.125)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[], []]
    for _ in range(20):
        for s, o in zip(streams, outs):
            o.append(kda.attn_decode(*args, 0.125, stream=s.cuda_stream))
    torch.cuda.synchronize()
    for o in outs:
        for t in o:
            assert torch.equal(bits(t), bits(want))
