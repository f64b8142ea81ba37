"""Corners of the softmax-attention operators that their documentation allows, against the formulas in 64 bits
(attention_ref.py, which derives the tolerances)."""
import ctypes
import math
import threading

import pytest
import torch

import attention_ref as ref
import kimi_delta_attention_24_b200 as kda
from test_attention_gpu import BF, bits, dev, run_decode, within

pytestmark = pytest.mark.gpu


def bwd_inputs(tokens, hq, hk, d, rot, seed):
    g = torch.Generator().manual_seed(seed)
    qkv = torch.randn(tokens, hq + 2 * hk, d, generator=g).to(BF)
    wq, wk = (1 + 0.3 * torch.randn(d, generator=g) for _ in range(2))
    tab = ref.table(rot, 500) if rot else None
    pos = torch.randint(1, 500, (tokens,), generator=g, dtype=torch.int32) if rot else None
    gq, gk = (torch.randn(tokens, h, d, generator=g).to(BF) for h in (hq, hk))
    return qkv[:, :hq], qkv[:, hq:hq + hk], wq, wk, tab, pos, gq, gk


# ------------------------------------------------------------------------------------ the gradient
# The weights' gradients: at the sizes here a lane adds up to 32 rows, a block up to 32 lanes, and the last
# launch 35 blocks' sums in each of 8 slices; with the 14 roundings of a term below 128 units of 2^-24 (the
# reference's tolerance counts 96).
DW_MORE = 128 / 96


@pytest.mark.parametrize("tokens,hq,hk,d,rot", [
    (1, 1, 1, 64, 64), (5, 5, 1, 128, 64), (33, 9, 2, 80, 80), (300, 13, 7, 128, 0),
    # enough tokens for several turns of two heads each, and heads that do not fill them
    (3301, 20, 1, 128, 128), (3301, 18, 3, 128, 64), (6701, 24, 1, 64, 32)])
def test_bwd_without_epsilon(cuda_device, tokens, hq, hk, d, rot):
    """eps = 0: 1 / sqrt(mean x^2) of the places behind the last head, which hold no row, is infinite."""
    q, k, wq, wk, tab, pos, gq, gk = bwd_inputs(tokens, hq, hk, d, rot, 51)
    r = kda.qk_norm_rope_bwd(*dev(gq, gk, q, k, wq, wk), 0.0, *dev(tab, pos))
    for n, x, w, dy in (("q", q, wq, gq), ("k", k, wk, gk)):
        dx, dw, dx_tol, dw_tol = ref.norm_rope_bwd(x, w, 0.0, tab, pos, False, dy)
        within(r["d" + n], dx, dx_tol, "d" + n)
        within(r[f"d{n}_weight"], dw, dw_tol * DW_MORE, f"d{n}_weight")


@pytest.mark.parametrize("d,rot,hq,hk", [(64, 64, 3, 1), (128, 64, 4, 2)])
def test_bwd_of_skipped_tokens(cuda_device, d, rot, hq, hk):
    """A token whose position is out of range has no output, so its gradients are zero, whatever its rows hold;
    it adds nothing to the weights' gradients, and the status word tells of it."""
    tokens = 45
    q, k, wq, wk, tab, pos, gq, gk = bwd_inputs(tokens, hq, hk, d, rot, 52)
    off = torch.zeros(tokens, dtype=torch.bool)
    off[[0, 7, 8, 44]] = True
    pos[0], pos[7], pos[8], pos[44] = 500, -1, 1 << 30, -(1 << 31)
    q[7, 1, 3], k[8, 0, 5], gq[44, 0, 0], gk[0, 0, 1] = math.nan, math.inf, math.nan, -math.inf
    ws = torch.zeros(kda.load().kda_qk_norm_rope_bwd_workspace_size(), dtype=torch.uint8, device="cuda")
    args = dev(gq, gk, q, k, wq, wk), dev(tab, pos)
    # (memory that earlier tensors left behind would show in rows that are not written)
    left = [torch.full((tokens, h, d), 7.0, dtype=BF, device="cuda") for h in (hq, hk)]
    del left
    r = kda.qk_norm_rope_bwd(*args[0], 1e-6, *args[1], workspace=ws)
    assert kda.read_device_status(ws) == 1 and kda.read_device_status(ws) == 0
    for n, x, w, dy in (("q", q, wq, gq), ("k", k, wk, gk)):
        dx, dw, dx_tol, dw_tol = ref.norm_rope_bwd(x[~off], w, 1e-6, tab, pos[~off], False, dy[~off])
        got = r["d" + n].cpu()
        within(got[~off], dx, dx_tol, "d" + n)
        assert (got[off] == 0).all()
        within(r[f"d{n}_weight"], dw, dw_tol, f"d{n}_weight")


@pytest.mark.parametrize("tokens,hq,hk,d", [(33, 5, 2, 80), (1201, 9, 3, 64)])
def test_bwd_in_the_place_of_its_inputs(cuda_device, tokens, hq, hk, d):
    """The C function with dq in d_q_out's place and dk in d_k_out's: the bits of the call with its own outputs."""
    q, k, wq, wk, tab, pos, gq, gk = bwd_inputs(tokens, hq, hk, d, d - d % 32, 53)
    q, k, wq, wk, tab, pos, gq, gk = dev(q.contiguous(), k.contiguous(), wq, wk, tab, pos, gq, gk)
    want = kda.qk_norm_rope_bwd(gq, gk, q, k, wq, wk, 1e-6, tab, pos)
    lib = kda.load()
    ws = torch.zeros(lib.kda_qk_norm_rope_bwd_workspace_size(), dtype=torch.uint8, device="cuda")
    dwq, dwk = torch.empty(d, device="cuda"), torch.empty(d, device="cuda")
    p = lambda t: ctypes.c_void_p(t.data_ptr())
    st = lib.kda_qk_norm_rope_bwd(p(gq), p(gk), p(q), p(k), hq * d, hk * d, p(wq), p(wk), 1e-6, p(tab), p(pos), p(gq), p(gk), p(dwq), p(dwk),
                                  tokens, hq, hk, d, tab.shape[1], tab.shape[0], 0, p(ws), ws.numel(),
                                  ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert st == 0 and kda.read_device_status(ws) == 0
    for got, name in ((gq, "dq"), (gk, "dk"), (dwq, "dq_weight"), (dwk, "dk_weight")):
        assert torch.equal(bits(got), bits(want[name]))


def test_bwd_of_rows_that_are_no_numbers(cuda_device):
    """Infinities and NaN in rows and in their gradients: where the formula has a number, that number."""
    tokens, hq, hk, d = 40, 3, 2, 64
    q, k, wq, wk, tab, pos, gq, gk = bwd_inputs(tokens, hq, hk, d, 32, 54)
    q[3, 1, 60], q[9, 0, 2], gq[11, 2, 50] = math.inf, math.nan, -math.inf
    k[:, :, 5], gk[20, 1, 7] = 0, math.nan
    for wq_, wk_ in ((wq, wk), (None, None)):
        r = kda.qk_norm_rope_bwd(*dev(gq, gk, q, k, wq_, wk_), 1e-6, *dev(tab, pos))
        for n, x, w, dy in (("q", q, wq_, gq), ("k", k, wk_, gk)):
            want = ref.norm_rope_bwd(x, w, 1e-6, tab, pos, False, dy)
            for got, y, tol in ((r["d" + n], want[0], want[2]), (r[f"d{n}_weight"], want[1], want[3])):
                if y is None:
                    continue
                fine = torch.isfinite(y)
                assert torch.equal(torch.isfinite(got.cpu()), fine)
                within(torch.where(fine, got.cpu().double(), 0.0), torch.where(fine, y, 0.0), torch.where(fine, tol, 1.0), n)


# ------------------------------------------------------------------------------------ the cache
@pytest.mark.parametrize("quant", [False, True], ids=["bf16", "e4m3"])
def test_append_into_pages_that_lie_apart(cuda_device, quant):
    """K and V of a page side by side in one pool: the same bytes as in caches of their own, and no others."""
    gen = torch.Generator().manual_seed(61)
    tokens, hk, d, page, pages = 50, 3, 80, 16, 7
    kc, ks = ref.make_cache(gen, pages, hk, page, d, quant, fill=3.0)
    vc, vs = ref.make_cache(gen, pages, hk, page, d, quant, fill=3.0)
    qkv = torch.randn(tokens, 3 * hk, d, generator=gen).to(BF).cuda()
    k, v = qkv[:, hk:2 * hk], qkv[:, 2 * hk:]
    slots = torch.randperm(pages * page, generator=gen)[:tokens].to(torch.int32).cuda()
    own = dev(kc, vc, ks, vs)
    kda.kv_append(k, v, own[0], own[1], slots, k_scale=own[2], v_scale=own[3])
    raw = [t.view(torch.uint8) for t in (kc, vc)]
    pool = torch.stack([raw[0], torch.full_like(raw[0], 0x55), raw[1]], 1).cuda()
    kd, vd = pool[:, 0].view(kc.dtype), pool[:, 2].view(vc.dtype)
    ksd, vsd = dev(ks, vs)
    kda.kv_append(k, v, kd, vd, slots, k_scale=ksd, v_scale=vsd)
    for got, want in ((kd, own[0]), (vd, own[1])) + (((ksd, own[2]), (vsd, own[3])) if quant else ()):
        assert torch.equal(bits(got), bits(want))
    assert (pool[:, 1] == 0x55).all()


# ------------------------------------------------------------------------------------ decode attention
def compare_where_finite(out, lse, o, l, ot, lt, lse_rows):
    """The formula's numbers where it has them, and no number where it has none (lse: in the given rows)."""
    got = out.cpu().double()
    fine = torch.isfinite(o)
    assert torch.equal(torch.isfinite(got), fine)
    within(torch.where(fine, got, 0.0), torch.where(fine, o, 0.0), torch.where(fine, ot, 1.0), "out")
    within(torch.where(lse_rows, lse.cpu().double(), 0.0), torch.where(lse_rows, l, 0.0), torch.where(lse_rows, lt, 1.0), "lse")


@pytest.mark.parametrize("quant,what,softcap", [(False, "k nan", 0.0), (False, "k nan", 20.0), (False, "k inf", 0.0), (True, "k scale", 0.0),
                                                (True, "k scale", 20.0), (True, "v scale", 0.0), (True, "v scale", 20.0)])
@pytest.mark.parametrize("d,new,group", [(64, 4, 3), (128, 3, 2)])
def test_decode_keys_that_only_some_queries_see(cuda_device, d, new, group, quant, what, softcap):
    """A key, or a scale, that is no number in the last token's row and in the first one of the oldest query's
    window: it reaches the queries that see it and no other."""
    lens, window = [40, 129, 7], 20
    odd = [(b, j) for b, n in enumerate(lens) for j in (n - 1, max(0, n - new - window + 1))]
    def mutate(q, kc, vc, ks, vs, tab):
        if what == "k inf":
            q.abs_()  # (scores of plus infinity: no number comes of them)
            q += 0.1
        for b, j in odd:
            p, r = int(tab[b, j // 16]), j % 16
            if what.startswith("k n") or what == "k inf":
                kc[p, 0, r, 5] = math.inf if what == "k inf" else math.nan
            else:
                (vs if what == "v scale" else ks)[p, 0, r] = math.nan
    out, lse, o, l, ot, lt = run_decode(lens, new, 2, group, d, 16, quant, window=window, mutate=mutate, softcap=softcap)
    sees = torch.zeros(len(lens), new, 2 * group, dtype=torch.bool)
    for b, j in odd:
        for t in range(new):
            last = lens[b] - new + t
            sees[b, t, :group] |= last - window < j <= last
    assert sees.any() and not sees[:, :, :group].all()
    assert torch.equal(torch.isfinite(o).all(3), ~sees)
    compare_where_finite(out, lse, o, l, ot, lt, ~sees)


def test_decode_largest_queries(cuda_device):
    """Queries up to bf16's largest power of two, against keys as small."""
    def mutate(q, kc, vc, ks, vs, tab):
        q *= 2.0 ** 124
        q[..., 3] = torch.where(q[..., 3] > 0, 2.0 ** 127, -2.0 ** 127).to(BF)
        q[0, 0, 1, 4] = 1.5 * 2.0 ** 127
        if ks is not None:
            ks *= 2.0 ** -60
        else:
            kc *= 2.0 ** -60
    for quant in (False, True):
        out, lse, o, l, ot, lt = run_decode([200, 17], 1, 1, 4, 128, 16, quant, mutate=mutate, scale=2.0 ** -66)
        within(out, o, ot, "out")
        within(lse, l, lt, "lse")


@pytest.mark.parametrize("softcap,window", [(0.0, 0), (30.0, 50)])
def test_decode_scales_over_the_allowed_range(cuda_device, softcap, window):
    """Value scales from about 2^-58 to 2^24: keys of either kind count in the sums (lse shows it)."""
    def mutate(q, kc, vc, ks, vs, tab):
        ok = ~torch.isnan(vs)
        small = torch.rand(vs.shape, generator=torch.Generator().manual_seed(3)) < 0.5
        vs[ok & small] *= 2.0 ** -51
        vs[ok & ~small] *= 2.0 ** 31
    out, lse, o, l, ot, lt = run_decode([500, 77, 3], 2, 2, 4, 128, 16, True, mutate=mutate, softcap=softcap, window=window)
    within(out, o, ot, "out")
    within(lse, l, lt, "lse")


def test_decode_small_weights_keep_their_bits(cuda_device):
    """e4m3 cache: channels to which only keys of weights 2^-22 to 2^-27 of the largest add.  A weight is rounded to
    fp16 as p s 2^14 relative to a reference within a factor of two of the largest: 2^-11 of it down to 2^-28 of the
    reference, so here as for the large ones."""
    gen = torch.Generator().manual_seed(71)
    n, d, page, group = 3, 64, 16, 4
    for drop in (22, 23, 24, 25, 26, 26, 27, 27):
        kc, ks = ref.make_cache(gen, 2, 1, page, d, True)
        vc, vs = ref.make_cache(gen, 2, 1, page, d, True)
        tab = ref.fill_sequences(gen, [n], kc, vc, ks, vs)
        q = torch.zeros(1, 1, group, d, dtype=BF)
        q[..., 0] = 1.0
        j = torch.arange(n)
        p, r = tab[0].long()[j // page], j % page
        # scores: 0 for the first key, about -drop ln 2 for the others; values: the first key's in channel 0 alone
        k = torch.zeros(n, d)
        k[1:, 0] = -drop * math.log(2.0) * (1 + 0.02 * torch.rand(n - 1, generator=gen))
        v = 1 + torch.rand(n, d, generator=gen)
        v[0, 1:], v[1:, 0] = 0, 0
        for cache, scale, x in ((kc, ks, k), (vc, vs, v)):
            c, s = ref.quantise(x)
            cache.view(torch.uint8)[p, 0, r] = c.view(torch.uint8)
            scale[p, 0, r] = s
        args = [t.cuda() for t in (q, kc, vc, tab, torch.tensor([n], dtype=torch.int32))]
        out = kda.attn_decode(*args, 1.0, k_scale=ks.cuda(), v_scale=vs.cuda())
        o, _, _, _ = ref.attention(q, kc, vc, tab, [n], 1.0, ks, vs)
        # the output's rounding, a weight's (2^-11), and below 2^-14 for scores, exponentials and sums (all terms
        # of a channel have one sign); 2^-39 of the largest p s (s 448 <= 2) for each key that is subnormal
        tol = (ref.BF16 + (1 + ref.BF16) * (2.0 ** -11 + 2.0 ** -14)) * o.abs() + n * 2.0 ** -38
        within(out, o, tol, f"weights of 2^-{drop}")


@pytest.mark.parametrize("n", [1, 300, 20000])
def test_decode_zeroed_cache(cuda_device, n):
    """A cache of zeros, its scales zero too: every key alike, out 0 and lse log n."""
    kc = torch.zeros(1, 2, 64, 64, device="cuda").to(torch.float8_e4m3fn)
    ks = torch.zeros(1, 2, 64, device="cuda")
    table = torch.zeros(1, 320, dtype=torch.int32, device="cuda")
    lse = torch.zeros(1, 4, device="cuda")
    q = torch.ones(1, 4, 64, dtype=BF, device="cuda")
    out = kda.attn_decode(q, kc, kc, table, torch.tensor([n], dtype=torch.int32, device="cuda"), 0.125, k_scale=ks, v_scale=ks, lse=lse)
    assert (out == 0).all()
    # sums of n equal terms (their rounding is below n 2^-24, and a term's below 2^-20), a scale's logarithm of -80
    want = torch.full((1, 4), math.log(n), dtype=torch.float64)
    within(lse, want, torch.full_like(want, (n + 300) * ref.F32 + 2.0 ** -20 + 100 * 4 * ref.F32), "lse")


@pytest.mark.parametrize("quant", [False, True], ids=["bf16", "e4m3"])
def test_calls_from_two_host_threads(cuda_device, quant):
    """Append and attend from two threads at once, each with a stream, a cache and a workspace of its own."""
    gen = torch.Generator().manual_seed(81)
    hk, group, d, page, n = 2, 4, 64, 16, 300
    sides = []
    for _ in range(2):
        kc, ks = ref.make_cache(gen, 20, hk, page, d, quant, fill=0.0)
        vc, vs = ref.make_cache(gen, 20, hk, page, d, quant, fill=0.0)
        tab = torch.randperm(20, generator=gen)[None, :19].to(torch.int32)
        qkv = torch.randn(n, hk * (group + 2), d, generator=gen).to(BF)
        j = torch.arange(n)
        slots = (tab[0].long()[j // page] * page + j % page).to(torch.int32)
        sides.append([t if t is None else t.cuda() for t in (kc, vc, ks, vs, tab, qkv, slots)])
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()

    def work(side, stream, outs):
        kc, vc, ks, vs, tab, qkv, slots = side
        hq = hk * group
        ws = kda.new_attn_decode_workspace(1, hq, hk, d, "cuda")
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            for _ in range(50):
                q = kda.kv_append(qkv[:, hq:hq + hk], qkv[:, hq + hk:], kc, vc, slots, k_scale=ks, v_scale=vs, q=qkv[:, :hq])
                outs.append(kda.attn_decode(q[-1:], kc, vc, tab, lens, d ** -0.5, k_scale=ks, v_scale=vs, workspace=ws))
        stream.synchronize()

    results = [[], []]
    threads = [threading.Thread(target=work, args=(s, torch.cuda.Stream(), o)) for s, o in zip(sides, results)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for (kc, vc, ks, vs, tab, qkv, slots), outs in zip(sides, results):
        assert len(outs) == 50
        cpu = lambda t: None if t is None else t.cpu()
        o, _, ot, _ = ref.attention(qkv.cpu()[None, -1:, :hk * group], kc.cpu(), vc.cpu(), tab.cpu(), [n], d ** -0.5, cpu(ks), cpu(vs))
        for got in outs:
            assert torch.equal(bits(got), bits(outs[0]))
        within(outs[0], o[:, 0], ot[:, 0], "out")
