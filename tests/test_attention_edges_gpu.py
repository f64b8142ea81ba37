"""Corners of the softmax-attention operators that their documentation allows, against the formulas in 64 bits
(attention_ref.py, which derives the tolerances)."""
import math

import pytest
import torch

import attention_ref as ref
import kimi_delta_attention_24_b200 as kda
from test_attention_gpu import BF, dev, run_decode, within

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


# ------------------------------------------------------------------------------------ decode attention
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
