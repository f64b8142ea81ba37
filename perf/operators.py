"""The softmax-attention operators that serve beside the KDA layers of a hybrid model, as cases with plain forms:

  rope, rope_bwd   per-head RMS norms of queries and keys with the position rotation, and their gradient
  append           the same, with keys and values written into a paged cache (bf16, or e4m3 with a scale per row)
  read             a paged cache read back into packed bf16 rows
  decode           attention of one or a few new tokens per sequence over the paged cache

`run` computes the plain form (elementary torch operations in fp32, rounded once) unless `own` is set; then it calls the
package's entry points.
"""
import math

import torch

own = False

EPS = 1e-6
MAX_POS = 1 << 17          # rows of the rotation table
SCALE_FLOOR = 2.0 ** -64   # smallest scale of a quantised row
DECODE_BYTES_MOST = 1.4e9  # cache bytes of the largest decode case
DECODE_SCORES_MOST = 1e8   # and its scores


def listed():
    return [
        # one decoding step of 8 requests: 40 heads each, nothing but launch latency
        dict(name="rope_8_tokens", op="rope", tokens=8, hq=32, hk=8, d=128, rot=128, interleaved=False, norm=True),
        # a 32K-token prefill with 96 query heads
        dict(name="rope_prefill_32k", op="rope", tokens=32768, hq=96, hk=12, d=128, rot=64, interleaved=True, norm=True),
        # gradients of a short packed batch (two documents of 200 tokens), 12 heads
        dict(name="rope_bwd_400", op="rope_bwd", tokens=400, hq=12, hk=12, d=96, rot=96, interleaved=False, norm=True),
        # gradients of a 4096-token training step, 96 query heads
        dict(name="rope_bwd_4k", op="rope_bwd", tokens=4096, hq=96, hk=12, d=128, rot=128, interleaved=False, norm=True),
        # a decoding step of 256 requests into an e4m3 cache, a few of them padding
        dict(name="append_256_e4m3", op="append", tokens=256, pad=5, hq=32, hk=8, d=128, rot=128, interleaved=False, norm=True,
             page=16, quant=True),
        # a prefill chunk of odd length into a bf16 cache, rotation over part of the head
        dict(name="append_4097_bf16", op="append", tokens=4097, pad=0, hq=32, hk=8, d=128, rot=64, interleaved=False, norm=True,
             page=64, quant=False),
        # one cached document for a continued prefill
        dict(name="read_200_bf16", op="read", batch=1, longest=200, hk=8, d=64, page=16, quant=False),
        # eight cached documents of up to 32K tokens from an e4m3 cache
        dict(name="read_8_docs_e4m3", op="read", batch=8, longest=32768, hk=8, d=128, page=64, quant=True),
        # one request, one short document: the latency of a single step
        dict(name="decode_1x333", op="decode", batch=1, longest=333, new=1, hk=8, group=4, d=128, page=16, quant=False,
             softcap=0.0, window=0),
        # an ordinary batch of ragged documents of up to 4096 tokens
        dict(name="decode_64x4k", op="decode", batch=64, longest=4096, new=1, hk=8, group=4, d=128, page=16, quant=False,
             softcap=0.0, window=0),
        # four speculative tokens per request, capped scores, a sliding window, e4m3, small heads
        dict(name="decode_48x8k_spec", op="decode", batch=48, longest=8192, new=4, hk=4, group=3, d=64, page=32, quant=True,
             softcap=30.0, window=3000),
        # few very long documents, 96 query heads, e4m3
        dict(name="decode_8x128k", op="decode", batch=8, longest=131072, new=1, hk=8, group=12, d=128, page=64, quant=True,
             softcap=0.0, window=0),
    ]


def _log_int(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 0.49)))))))


def draw(rng):
    op = rng.choice(["rope", "rope_bwd", "append", "read", "decode", "decode"])
    d = rng.choice([64, 128, 128, 16 * rng.randint(1, 8)])
    quant = rng.random() < 0.5
    page = rng.choice([8, 16, 32, 64, 128])
    if op in ("rope", "rope_bwd", "append"):
        hk = rng.choice([1, 2, 4, 7, 8, 12])
        hq = hk * rng.choice([1, 2, 3, 4, 8])
        rot = rng.choice([d, d, 16 * rng.randint(1, d // 16), 0])
        most = {"rope": 32768 * 108 * 128, "rope_bwd": 4096 * 108 * 128, "append": 4097 * 48 * 128}[op]
        tokens = _log_int(rng, 1, min(32768, most // (d * (hq + 2 * hk))))
        c = dict(op=op, tokens=tokens, hq=hq, hk=hk, d=d, rot=rot, interleaved=rng.random() < 0.4,
                 norm=op == "rope_bwd" or rng.random() < 0.8)
        if op == "append":
            c.update(pad=min(tokens - 1, rng.randint(0, 9)), page=page, quant=quant)
        return c
    hk = rng.choice([1, 2, 4, 8, 12])
    if op == "read":
        batch = _log_int(rng, 1, 64)
        return dict(op=op, batch=batch, longest=_log_int(rng, 1, min(65536, 8 * 32768 * 8 * 128 // (batch * hk * d))), hk=hk, d=d,
                    page=page, quant=quant)
    batch = _log_int(rng, 1, 256)
    row = batch * hk * 2 * d * (1 if quant else 2)
    new, group = rng.choice([1, 1, 1, 2, 3, 4, 5]), rng.choice([1, 2, 3, 4, 6, 8, 12, 16])
    most = min(DECODE_BYTES_MOST / row, DECODE_SCORES_MOST / (batch * hk * new * group))
    longest = _log_int(rng, 1, max(1, min(131072, int(most))))
    return dict(op=op, batch=batch, longest=longest, new=new, hk=hk, group=group, d=d, page=page, quant=quant,
                softcap=rng.choice([0.0, 0.0, 30.0]), window=rng.choice([0, 0, rng.randint(1, longest)]))


def _lengths(case):
    """Ragged lengths of a case: one sequence has the longest, the others are uniform down to one token."""
    g = torch.Generator().manual_seed(case["batch"] * 1000003 + case["longest"])
    n = torch.randint(1, case["longest"] + 1, (case["batch"],), generator=g, dtype=torch.int64)
    n[0] = case["longest"]
    return n


def _table(rot, device):
    """cos and sin of every position's angles (base 10000), formed in 64 bits: fp32 [MAX_POS, rot]."""
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=device) / rot)
    a = torch.arange(MAX_POS, dtype=torch.float64, device=device)[:, None] * inv
    return torch.cat([a.cos(), a.sin()], 1).float()


def _random_cache(gen, pages, hk, page, d, quant, device):
    """A pool of cache pages as written from N(0, 1) rows: bf16 [pages, hk, page, d], or e4m3 codes and their scales."""
    x = torch.empty(pages, hk, page, d, dtype=torch.bfloat16, device=device).normal_(generator=gen)
    if not quant:
        return x, None
    scale = torch.empty(pages, hk, page, device=device).uniform_(2.0, 4.0, generator=gen) / 448
    return (x / scale[..., None]).clamp_(-448, 448).to(torch.float8_e4m3fn), scale


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    op, d, hk = case["op"], case["d"], case["hk"]
    s = {"case": case}
    if op in ("rope", "rope_bwd", "append"):
        t, hq = case["tokens"], case["hq"]
        # the projection's output: queries, keys and values of a token side by side
        qkv = torch.empty(t, hq + 2 * hk, d, dtype=torch.bfloat16, device=dev).normal_(generator=gen)
        s.update(q=qkv[:, :hq], k=qkv[:, hq:hq + hk], v=qkv[:, hq + hk:])
        s["cos_sin"] = _table(case["rot"], dev) if case["rot"] else None
        s["positions"] = torch.randint(0, MAX_POS, (t,), generator=gen, device=dev, dtype=torch.int32)
        s["wq"] = 1 + 0.2 * torch.randn(d, generator=gen, device=dev) if case["norm"] else None
        s["wk"] = 1 + 0.2 * torch.randn(d, generator=gen, device=dev) if case["norm"] else None
        if op == "rope_bwd":
            s["gq"] = torch.empty(t, hq, d, dtype=torch.bfloat16, device=dev).normal_(generator=gen)
            s["gk"] = torch.empty(t, hk, d, dtype=torch.bfloat16, device=dev).normal_(generator=gen)
        if op == "append":
            page = case["page"]
            pages = -(-t // page) + 3
            s["kc"], s["ks"] = _random_cache(gen, pages, hk, page, d, case["quant"], dev)
            s["vc"], s["vs"] = _random_cache(gen, pages, hk, page, d, case["quant"], dev)
            s["slots"] = torch.randperm(pages * page, generator=gen, device=dev)[:t].to(torch.int32)
            if case["pad"]:
                s["slots"][t - case["pad"]:] = -1
            s["q_out"] = torch.zeros(t, hq, d, dtype=torch.bfloat16, device=dev)
        return s
    page, b = case["page"], case["batch"]
    n = _lengths(case)
    n = n[torch.randperm(b, generator=torch.Generator().manual_seed(seed))]
    wide = -(-case["longest"] // page)
    need = -(-n // page)
    pages = int(need.sum()) + 2
    s["kc"], s["ks"] = _random_cache(gen, pages, hk, page, d, case["quant"], dev)
    s["vc"], s["vs"] = _random_cache(gen, pages, hk, page, d, case["quant"], dev)
    order = torch.randperm(pages, generator=gen, device=dev).to(torch.int32)
    first = torch.cumsum(need, 0) - need
    at = first[:, None] + torch.arange(wide)[None]
    at = torch.where(torch.arange(wide)[None] < need[:, None], at, 0)
    s["table"] = order[at.to(dev)].contiguous()
    if op == "read":
        cu = torch.zeros(b + 1, dtype=torch.int32)
        cu[1:] = torch.cumsum(n, 0)
        s["cu"] = cu.to(dev)
        total = int(cu[-1])
        s["k_out"] = torch.zeros(total, hk, d, dtype=torch.bfloat16, device=dev)
        s["v_out"] = torch.zeros(total, hk, d, dtype=torch.bfloat16, device=dev)
        return s
    hq = hk * case["group"]
    s["lens"] = n.to(torch.int32).to(dev)
    s["q"] = torch.empty(b, case["new"], hq, d, dtype=torch.bfloat16, device=dev).normal_(generator=gen)
    s["scale"] = d ** -0.5
    s["lse"] = torch.empty(b, case["new"], hq, device=dev)
    return s


def _rotate(x, cos_sin, positions, interleaved):
    """The rotation of the first rot channels of fp32 x [tokens, heads, d]."""
    if cos_sin is None:
        return x
    rot = cos_sin.shape[1]
    cs = cos_sin[positions.long()][:, None]
    c, s = cs[..., :rot // 2], cs[..., rot // 2:]
    y = x.clone()
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * c - b * s, b * c + a * s
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = a * c - b * s, b * c + a * s
    return y


def _norm(x, w):
    x = x.float()
    return x if w is None else x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w


def _norm_rope_bwd(x, w, dy, cos_sin, positions, interleaved):
    back = None if cos_sin is None else torch.cat([cos_sin[:, :cos_sin.shape[1] // 2], -cos_sin[:, cos_sin.shape[1] // 2:]], 1)
    g = _rotate(dy.float(), back, positions, interleaved)
    x = x.float()
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    xh = x * r
    u = g * w
    dx = r * (u - xh * (u * xh).mean(-1, keepdim=True))
    return dx.to(torch.bfloat16), (g * xh).sum((0, 1))


def _write(cache, scales, x, slots):
    """Rows of fp32 x [tokens, hk, d] into slots of the paged cache; negative slots are skipped."""
    page = cache.shape[2]
    keep = slots >= 0
    at = slots[keep].long()
    x = x[keep]
    if scales is None:
        cache[at // page, :, at % page] = x.to(torch.bfloat16)
        return
    sc = (x.abs().amax(-1) / 448).clamp(min=SCALE_FLOOR)
    scales[at // page, :, at % page] = sc
    codes = (x / sc[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    cache.view(torch.uint8)[at // page, :, at % page] = codes.view(torch.uint8)


def _gather(cache, scales, table):
    """fp32 [batch, hk, width * page, d]: every page of each sequence's table row."""
    b, wide = table.shape
    p = table.long()
    if scales is None:
        x = cache[p].float()
    else:
        x = cache.view(torch.uint8)[p].view(torch.float8_e4m3fn).float() * scales[p][..., None]
    return x.transpose(1, 2).reshape(b, cache.shape[1], wide * cache.shape[2], cache.shape[3])


def run(s):
    case, op = s["case"], s["case"]["op"]
    if own:
        import kimi_delta_attention_24_b200 as kda
        if op == "rope":
            q, k = kda.qk_norm_rope(s["q"], s["k"], s["wq"], s["wk"], EPS, s["cos_sin"], s["positions"],
                                    interleaved=case["interleaved"])
            return {"q": q, "k": k}
        if op == "rope_bwd":
            return kda.qk_norm_rope_bwd(s["gq"], s["gk"], s["q"], s["k"], s["wq"], s["wk"], EPS, s["cos_sin"], s["positions"],
                                        interleaved=case["interleaved"])
        if op == "append":
            kda.kv_append(s["k"], s["v"], s["kc"], s["vc"], s["slots"], k_scale=s["ks"], v_scale=s["vs"], q=s["q"],
                          q_out=s["q_out"], q_weight=s["wq"], k_weight=s["wk"], eps=EPS, cos_sin=s["cos_sin"],
                          positions=s["positions"], interleaved=case["interleaved"])
            return {"q": s["q_out"], "k_cache": s["kc"], "v_cache": s["vc"], "k_scale": s["ks"], "v_scale": s["vs"]}
        if op == "read":
            kda.kv_read(s["kc"], s["vc"], s["table"], s["cu"], s["k_out"], s["v_out"], k_scale=s["ks"], v_scale=s["vs"])
            return {"k": s["k_out"], "v": s["v_out"]}
        out = kda.attn_decode(s["q"], s["kc"], s["vc"], s["table"], s["lens"], s["scale"], lse=s["lse"], k_scale=s["ks"],
                              v_scale=s["vs"], softcap=case["softcap"], window=case["window"])
        return {"out": out, "lse": s["lse"]}

    if op == "rope":
        return {n: _rotate(_norm(s[n], s["w" + n]), s["cos_sin"], s["positions"], case["interleaved"]).to(torch.bfloat16)
                for n in ("q", "k")}
    if op == "rope_bwd":
        dq, dwq = _norm_rope_bwd(s["q"], s["wq"], s["gq"], s["cos_sin"], s["positions"], case["interleaved"])
        dk, dwk = _norm_rope_bwd(s["k"], s["wk"], s["gk"], s["cos_sin"], s["positions"], case["interleaved"])
        return {"dq": dq, "dk": dk, "dq_weight": dwq, "dk_weight": dwk}
    if op == "append":
        q, k = (_rotate(_norm(s[n], s["w" + n]), s["cos_sin"], s["positions"], case["interleaved"]) for n in ("q", "k"))
        keep = (s["slots"] >= 0)[:, None, None]
        s["q_out"].copy_(torch.where(keep, q.to(torch.bfloat16), s["q_out"]))
        _write(s["kc"], s["ks"], k, s["slots"])
        _write(s["vc"], s["vs"], s["v"].float(), s["slots"])
        return {"q": s["q_out"], "k_cache": s["kc"], "v_cache": s["vc"], "k_scale": s["ks"], "v_scale": s["vs"]}
    if op == "read":
        cu = s["cu"].long()
        row = torch.arange(s["k_out"].shape[0], device=cu.device)
        b = torch.searchsorted(cu, row, right=True) - 1
        t = row - cu[b]
        page = s["kc"].shape[2]
        p = s["table"][b, t // page].long()
        at = (p, slice(None), t % page)
        if s["ks"] is None:
            s["k_out"].copy_(s["kc"][at])
            s["v_out"].copy_(s["vc"][at])
        else:
            for_k, for_v = ((s[c].view(torch.uint8)[at].view(torch.float8_e4m3fn).float() * s[m][at][..., None])
                            for c, m in (("kc", "ks"), ("vc", "vs")))
            s["k_out"].copy_(for_k)
            s["v_out"].copy_(for_v)
        return {"k": s["k_out"], "v": s["v_out"]}
    q = s["q"].float()
    b, new, hq, d = q.shape
    hk = case["hk"]
    # rows of one kv head together: [b, hk, new * group, d]
    q = q.view(b, new, hk, case["group"], d).permute(0, 2, 1, 3, 4).reshape(b, hk, new * case["group"], d)
    z = torch.matmul(q, _gather(s["kc"], s["ks"], s["table"]).transpose(2, 3)) * s["scale"]
    if case["softcap"]:
        z = case["softcap"] * torch.tanh(z / case["softcap"])
    j = torch.arange(z.shape[3], device=z.device)
    p = (s["lens"][:, None] - new + torch.arange(new, device=z.device)).repeat_interleave(case["group"], 1)[:, :, None]
    seen = j <= p
    if case["window"]:
        seen = seen & (j > p - case["window"])
    seen = seen[:, None]
    z = z.masked_fill(~seen, -math.inf)
    m = z.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    e = torch.exp(z - m)
    l = e.sum(-1, keepdim=True)
    o = torch.matmul(e, _gather(s["vc"], s["vs"], s["table"])) / torch.where(l == 0, 1.0, l)
    lse = (m + torch.log(l))[..., 0]
    o = o.view(b, hk, new, case["group"], d).permute(0, 2, 1, 3, 4).reshape(b, new, hq, d).to(torch.bfloat16)
    s["lse"].copy_(lse.view(b, hk, new, case["group"]).permute(0, 2, 1, 3).reshape(b, new, hq))
    return {"out": o, "lse": s["lse"]}


def work(case):
    op, d, hk = case["op"], case["d"], case["hk"]
    if op in ("rope", "rope_bwd", "append"):
        t, h = case["tokens"], case["hq"] + hk
        side = t * (4 + 4 * case["rot"]) + (8 * d if case["norm"] else 0)
        if op == "rope":
            return {"bytes": t * h * d * 4 + side, "flops": t * h * d * 8}
        if op == "rope_bwd":
            return {"bytes": t * h * d * 6 + side + 8 * d, "flops": t * h * d * 16}
        live = t - case["pad"]
        row = hk * (d + 4) if case["quant"] else hk * 2 * d
        return {"bytes": live * (case["hq"] * d * 4 + hk * 4 * d + 2 * row + 8 + 4 * case["rot"]) + (8 * d if case["norm"] else 0),
                "flops": live * h * d * 8}
    token = hk * 2 * ((d + 4) if case["quant"] else 2 * d)
    lens = _lengths(case)
    n = int(lens.sum())
    if op == "read":
        return {"bytes": n * (token + hk * 4 * d) + 4 * n / case["page"], "flops": n * hk * 2 * d}
    rows = case["batch"] * case["new"] * hk * case["group"]
    if case["window"]:
        n = int(lens.clamp(max=case["window"] + case["new"] - 1).sum())
    return {"bytes": n * token + rows * (4 * d + 4), "flops": 4 * n * case["new"] * hk * case["group"] * d}


# --------------------------------------------------------------------------------------------------------------------
# the definitions in 64 bits

def _exact_rotation(n, rot, positions, interleaved, table, sign):
    """Each pair of channels as a complex number times e^{i angle}."""
    z = torch.complex(table[positions.long(), :rot // 2].double(), sign * table[positions.long(), rot // 2:].double())[:, None]
    head, tail = n[..., :rot], n[..., rot:]
    if interleaved:
        w = torch.view_as_complex(head.reshape(*head.shape[:-1], rot // 2, 2).contiguous()) * z
        head = torch.view_as_real(w).reshape(head.shape)
    else:
        w = torch.complex(head[..., :rot // 2].contiguous(), head[..., rot // 2:].contiguous()) * z
        head = torch.cat([w.real, w.imag], -1)
    return torch.cat([head, tail], -1)


def _exact_forward(case, s, n):
    x = s[n].double()
    if case["norm"]:
        x = x / (x.pow(2).sum(-1, keepdim=True) / case["d"] + EPS).sqrt() * s["w" + n].double()
    return _exact_rotation(x, case["rot"], s["positions"], case["interleaved"], s["cos_sin"], 1.0) if case["rot"] else x


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "rope":
        return {n: _exact_forward(case, s, n) for n in ("q", "k")}
    if op == "rope_bwd":
        r = {}
        for n in ("q", "k"):
            g = s["g" + n].double()
            if case["rot"]:
                g = _exact_rotation(g, case["rot"], s["positions"], case["interleaved"], s["cos_sin"], -1.0)
            x, w = s[n].double(), s["w" + n].double()
            v = x.pow(2).sum(-1, keepdim=True) / case["d"] + EPS
            r["d" + n] = g * w / v.sqrt() - x * (g * w * x).sum(-1, keepdim=True) / (case["d"] * v.pow(1.5))
            r["d" + n + "_weight"] = (g * x / v.sqrt()).flatten(0, 1).sum(0)
        return r
    if op == "append":
        page = case["page"]
        live = case["tokens"] - case["pad"]
        q = s["q_out"].double()
        q[:live] = _exact_forward(case, s, "q")[:live]
        r = {"q": q, "k_cache": None, "v_cache": None, "k_scale": None, "v_scale": None}
        at = s["slots"][:live].long()
        for n, x in (("k", _exact_forward(case, s, "k")), ("v", s["v"].double())):
            x = x[:live]
            if case["quant"]:  # the codes are a choice of rounding; the scales are numbers
                scale = s[n + "s"].double()
                scale[at // page, :, at % page] = torch.maximum(x.abs().max(-1).values / 448, torch.tensor(SCALE_FLOOR, device=x.device).double())
                r[n + "_scale"] = scale
            else:
                cache = s[n + "c"].double()
                cache[at // page, :, at % page] = x
                r[n + "_cache"] = cache
        return r
    hk, d, page = case["hk"], case["d"], case["page"]

    def rows(cache, scale, b, first, last):
        """Tokens first .. last - 1 of sequence b in 64 bits: [tokens, hk, d]."""
        pages = s["table"][b, first // page:-(-last // page)].long()
        x = cache.view(torch.uint8)[pages].view(cache.dtype) if scale is not None else cache[pages]
        x = x.double()
        if scale is not None:
            x = x * scale[pages].double().unsqueeze(-1)
        x = x.permute(0, 2, 1, 3).reshape(-1, hk, d)
        return x[first % page:first % page + last - first]

    if op == "read":
        cu = s["cu"].tolist()
        return {n: torch.cat([rows(s[n + "c"], s[n + "s"], b, 0, cu[b + 1] - cu[b]) for b in range(case["batch"])])
                for n in ("k", "v")}
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    lse = torch.full(out.shape[:3], -math.inf, dtype=torch.float64, device=out.device)
    for b, length in enumerate(s["lens"].tolist()):
        for t in range(case["new"]):
            last = length - case["new"] + t + 1
            first = max(0, last - case["window"]) if case["window"] else 0
            if last <= first:
                continue
            k, v = rows(s["kc"], s["ks"], b, first, last), rows(s["vc"], s["vs"], b, first, last)
            q = s["q"][b, t].double().view(hk, case["group"], d)
            z = torch.einsum("hgd,jhd->hgj", q, k) * s["scale"]
            if case["softcap"]:
                z = case["softcap"] * torch.tanh(z / case["softcap"])
            lse[b, t] = torch.logsumexp(z, -1).flatten()
            out[b, t] = torch.einsum("hgj,jhd->hgd", torch.softmax(z, -1), v).reshape(-1, d)
    return {"out": out, "lse": lse}
