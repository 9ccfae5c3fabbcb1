"""The operators of a serving step around the sparse attention, as measured cases.

Four operators, in the order a step calls them:

  layout   block tables and slot maps from request lengths (``batch_layout``)
  qk       norms of queries and keys with the position rotation, the keys
           written into the paged FP8 cache (``qk_norm_rope``)
  mla      attention of a chunk of new tokens over the paged cache (``chunk_mla``)
  verify   drafted tokens checked against the target's probabilities
           (``verify_draft``)

With ``own`` false ``run`` computes them in plain torch operations (32 bits, 64
where a result hangs on a comparison); with ``own`` true it makes the library's
calls.  ``exact`` gives the same from the definitions in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"


# ---- cases -----------------------------------------------------------------------


def listed():
    return [
        # one decode step of a small batch: latency only
        dict(name="layout decode 8", op="layout", req=8, new=1, ctx=4096, page=64),
        # a speculative verify step, 8 tokens at most for each of 128 requests of 64K context
        dict(name="layout verify 128x8", op="layout", req=128, new=8, ctx=65536, page=64),
        # a mixed step of 512 requests that bring up to 2,001 tokens each (prompts admitted whole), small pages
        dict(name="layout prompts 512x2001", op="layout", req=512, new=2001, ctx=8191, page=16),
        # decode of 128 requests: 64 absorbed query heads and the latent row that goes into the FP8 cache
        dict(name="qk decode 128 fp8", op="qk", tokens=128, heads=64, k_heads=1, d=576, rope=64, q_norm=576, k_norm=512,
             interleaved=True, cache=True, max_pos=65536),
        # a prefill chunk of the same model
        dict(name="qk prefill 8192 fp8", op="qk", tokens=8192, heads=64, k_heads=1, d=576, rope=64, q_norm=576,
             k_norm=512, interleaved=True, cache=True, max_pos=65536),
        # grouped-query heads of 128, rotated in halves over the whole head, keys kept in 16 bits; an odd token count
        dict(name="qk grouped 4099 bf16", op="qk", tokens=4099, heads=32, k_heads=8, d=128, rope=128, q_norm=128,
             k_norm=128, interleaved=False, cache=False, max_pos=131072),
        # the small head shape: one token of each of two requests over 512 positions
        dict(name="mla tiny 2x1 ctx 512", op="mla", heads=16, dl=64, dr=16, req=2, new=1, ctx=512, ragged=False, page=16),
        # dense decode: 32 ragged requests of up to 8,192 positions (KV splits fill the GPU)
        dict(name="mla decode 32x1 ctx 8192", op="mla", heads=64, dl=512, dr=64, req=32, new=1, ctx=8192, ragged=True,
             page=64),
        # dense verify: up to 8 drafted tokens of 16 requests, a page size that does not divide the kernel's tiles
        dict(name="mla verify 16x8 ctx 4096", op="mla", heads=64, dl=512, dr=64, req=16, new=8, ctx=4096, ragged=True,
             page=48),
        # a prefill chunk of 1,024 tokens at the end of a 16K context
        dict(name="mla chunk 1x1024 ctx 16384", op="mla", heads=64, dl=512, dr=64, req=1, new=1024, ctx=16384,
             ragged=False, page=64),
        # four requests, drafts without probabilities (each drafted token taken as certain), a small odd vocabulary
        dict(name="verify 4x4 certain", op="verify", req=4, draft=4, vocab=32003, probs=False),
        # 128 requests of up to 8 drafted tokens with the draft's probabilities over a large vocabulary
        dict(name="verify 128x8 probs", op="verify", req=128, draft=8, vocab=131072, probs=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("layout", "qk", "mla", "verify"))
    if op == "layout":
        req, new = _log(rng, 1, 1024), _log(rng, 1, 2001)
        return dict(op=op, req=req, new=min(new, max(1, 1_000_000 // req)), ctx=_log(rng, 1, 65536),
                    page=rng.choice((1, 16, 48, 64, 128)))
    if op == "qk":
        if rng.random() < 0.5:
            h, kh, d, rope, qn, kn = 64, 1, 576, 64, rng.choice((0, 576)), 512
            cache = True
        else:
            d = rng.choice((64, 80, 128, 256))
            rope = rng.choice((16, 32, 64)) if d != 128 else 128
            h, kh, qn, kn = rng.choice((8, 16, 32)), rng.choice((1, 2, 8)), d, d
            cache = kh == 1
        return dict(op=op, tokens=_log(rng, 1, 8192), heads=h, k_heads=kh, d=d, rope=rope, q_norm=qn, k_norm=kn,
                    interleaved=rng.random() < 0.5, cache=cache, max_pos=_log(rng, 512, 1 << 18))
    if op == "mla":
        big = rng.random() < 0.75
        req, new = _log(rng, 1, 32), _log(rng, 1, 256)
        ctx = _log(rng, 1, 16384)
        new = min(new, ctx, max(1, (1 << 23) // (req * ctx)))
        return dict(op=op, heads=64 if big else 16, dl=512 if big else 64, dr=64 if big else 16, req=req, new=new,
                    ctx=ctx, ragged=rng.random() < 0.7, page=rng.choice((1, 16, 48, 64, 128)))
    return dict(op=op, req=_log(rng, 1, 128), draft=rng.randint(0, 8), vocab=_log(rng, 1000, 131072),
                probs=rng.random() < 0.6)


# ---- inputs ----------------------------------------------------------------------


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 7919 + 17)
    return g


def _ints(lo, hi, n, g):
    """int32 [n], uniform in lo..hi (both included)."""
    return torch.randint(lo, hi + 1, (n,), generator=g, device=DEV, dtype=torch.int32)


def prepare(case, seed):
    g = _gen(seed)
    return dict({"layout": _prepare_layout, "qk": _prepare_qk, "mla": _prepare_mla, "verify": _prepare_verify}[case["op"]](case, g),
                case=case)


def _prepare_layout(c, g):
    R, P = c["req"], c["page"]
    ctx = _ints(0, c["ctx"], R, g)
    new = _ints(1, c["new"], R, g)
    # a request holds the pages of its context, and sometimes one more (of tokens that were rejected)
    held = (ctx + P - 1) // P + _ints(0, 1, R, g)
    stride = (c["ctx"] + c["new"] + P - 1) // P + 1
    num_pages = R * stride
    perm = torch.randperm(num_pages, generator=g, device=DEV).to(torch.int32).view(R, stride)
    mask = torch.arange(stride, device=DEV)[None, :] < held[:, None]
    free = perm[~mask]
    free = free[torch.randperm(free.numel(), generator=g, device=DEV)].contiguous()
    table = torch.where(mask, perm, torch.full_like(perm, -1)).contiguous()
    return dict(ctx=ctx, new=new, held=held, table=table, free=free, used=torch.zeros(1, dtype=torch.int32, device=DEV),
                num_pages=num_pages, capacity=R * c["new"])


def _prepare_qk(c, g):
    T, d, rope = c["tokens"], c["d"], c["rope"]
    q = torch.randn((T, c["heads"], d), generator=g, device=DEV).to(torch.bfloat16)
    # the keys are the last columns of a wider projection: a strided view
    wide = torch.randn((T, 64 + c["k_heads"] * d), generator=g, device=DEV).to(torch.bfloat16)
    k = wide[:, 64:].unflatten(1, (c["k_heads"], d))
    qw = 1 + 0.1 * torch.randn(c["q_norm"], generator=g, device=DEV) if c["q_norm"] else None
    kw = 1 + 0.1 * torch.randn(c["k_norm"], generator=g, device=DEV) if c["k_norm"] else None
    pos = _ints(0, c["max_pos"] - 1, T, g)
    freq = 10000.0 ** (-torch.arange(0, rope, 2, device=DEV, dtype=torch.float64) / rope)
    angle = torch.arange(c["max_pos"], device=DEV, dtype=torch.float64)[:, None] * freq[None, :]
    s = dict(q=q, k=k, qw=qw, kw=kw, pos=pos, cos_sin=torch.cat((angle.cos(), angle.sin()), 1).float())
    if c["cache"]:
        slots = (2 * T + 63) // 64 * 64
        s["slot"] = torch.randperm(slots, generator=g, device=DEV)[:T].to(torch.int32)
        s["kv"] = torch.zeros((slots, d), dtype=torch.uint8, device=DEV)
        s["kv_scale"] = torch.zeros(slots, dtype=torch.float32, device=DEV)
    return s


def _prepare_mla(c, g):
    R, n, P = c["req"], c["new"], c["page"]
    dqk = c["dl"] + c["dr"]
    if c["ragged"]:
        q_len = _ints(1, n, R, g)
        kv_len = torch.maximum(_ints((c["ctx"] + 1) // 2, c["ctx"], R, g), q_len)
    else:
        q_len = torch.full((R,), n, dtype=torch.int32, device=DEV)
        kv_len = torch.full((R,), c["ctx"], dtype=torch.int32, device=DEV)
    stride = (c["ctx"] + P - 1) // P
    num_pages = R * stride
    table = torch.randperm(num_pages, generator=g, device=DEV).to(torch.int32).view(R, stride).contiguous()
    rows = torch.randn((num_pages * P, dqk), generator=g, device=DEV)
    scale = rows.abs().amax(1) / 448.0
    kv = (rows / scale[:, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
    # tokens request after request, padded with -1 to the batch's capacity
    j = torch.arange(n, device=DEV, dtype=torch.int32)[None, :]
    live = j < q_len[:, None]
    order = torch.argsort((~live).flatten().to(torch.int8), stable=True)
    req = torch.where(live, torch.arange(R, device=DEV, dtype=torch.int32)[:, None], -1).flatten()[order]
    pos = torch.where(live, (kv_len - q_len)[:, None] + j, -1).flatten()[order]
    q = torch.randn((R * n, c["heads"], dqk), generator=g, device=DEV).to(torch.bfloat16)
    return dict(q=q, kv=kv, kv_scale=scale.contiguous(), table=table, q_req=req.to(torch.int32).contiguous(),
                q_pos=pos.to(torch.int32).contiguous(), softmax_scale=dqk ** -0.5)


def _prepare_verify(c, g):
    R, n, V = c["req"], c["draft"], c["vocab"]
    drafts = _ints(0, n, R, g)
    cu = torch.zeros(R + 1, dtype=torch.int32, device=DEV)
    cu[1:] = torch.cumsum(drafts + 1, 0)
    rows = int(cu[-1])
    target = torch.randn((rows, V), generator=g, device=DEV) * 3.0
    # the draft model's logits: the target's with some noise (a draft has the target's row
    # that it is checked by; the row after a request's last draft has none, and is not read)
    draft = torch.softmax(target + torch.randn((rows, V), generator=g, device=DEV), 1)
    target = torch.softmax(target, 1)
    # a token from the draft's distribution: the smallest of exponential clocks
    tok = (draft / torch.empty((rows, V), device=DEV).exponential_(generator=g)).argmax(1).to(torch.int32)
    return dict(target=target, draft=draft if c["probs"] else None, tok=tok, cu=cu,
                u_accept=torch.rand(rows, generator=g, device=DEV), u_sample=torch.rand(R, generator=g, device=DEV),
                ctx=_ints(0, 65536, R, g))


# ---- one pass --------------------------------------------------------------------


def run(state):
    op = state["case"]["op"]
    if own:
        return {"layout": _own_layout, "qk": _own_qk, "mla": _own_mla, "verify": _own_verify}[op](state)
    return {"layout": _plain_layout, "qk": _plain_qk, "mla": _plain_mla, "verify": _plain_verify}[op](state)


def _own_layout(s):
    import dsa_sparse_mla_topk_gb300 as dsa

    lay = dsa.batch_layout(s["ctx"], s["new"], s["held"], s["table"], s["free"], s["used"], page_size=s["case"]["page"],
                           num_pages=s["num_pages"], capacity=s["capacity"])
    return dict(cu_q=lay.cu_q, q_req=lay.q_req, q_pos=lay.q_pos, slot=lay.slot, ctx=lay.ctx_len, held=lay.pages_held,
                used=lay.free_used, table=s["table"])


def _own_qk(s):
    import dsa_sparse_mla_topk_gb300 as dsa

    c = s["case"]
    q, k = dsa.qk_norm_rope(s["q"], s["k"], s["pos"], s["cos_sin"], d_rope=c["rope"], q_weight=s["qw"], k_weight=s["kw"],
                            eps=1e-6, interleaved=c["interleaved"], slot=s.get("slot"), kv=s.get("kv"),
                            kv_scale=s.get("kv_scale"))
    return _qk_out(s, q, k)


def _own_mla(s):
    import dsa_sparse_mla_topk_gb300 as dsa

    c = s["case"]
    out, lse = dsa.chunk_mla(s["q"], s["kv"], s["kv_scale"], s["table"], s["q_req"], s["q_pos"], d_latent=c["dl"],
                             d_rope=c["dr"], page_size=c["page"], softmax_scale=s["softmax_scale"], max_ctx=c["ctx"])
    return dict(out=out, lse=lse)


def _own_verify(s):
    import dsa_sparse_mla_topk_gb300 as dsa

    tokens, num, ctx = dsa.verify_draft(s["target"], s["tok"], s["cu"], s["u_accept"], s["u_sample"],
                                        draft_probs=s["draft"], ctx_len=s["ctx"], max_out=s["case"]["draft"] + 1)
    return dict(tokens=tokens, num=num, ctx=ctx)


def _plain_layout(s):
    ctx, new, held, table, free, used = (s[x] for x in ("ctx", "new", "held", "table", "free", "used"))
    P, R, cap = s["case"]["page"], ctx.numel(), s["capacity"]
    cu = torch.zeros(R + 1, dtype=torch.int32, device=ctx.device)
    cu[1:] = torch.cumsum(new, 0)
    total = (ctx + new + P - 1) // P
    need = torch.where(new > 0, (total - held).clamp(min=0), 0)
    upto = torch.cumsum(need, 0)
    fits = (need == 0) | (used + upto <= free.numel())
    need = torch.where(fits, need, 0)
    first = upto - need
    col = torch.arange(table.shape[1], device=ctx.device)[None, :]
    fresh = (col >= held[:, None]) & (col < (held + need)[:, None])
    at = (used + first[:, None] + col - held[:, None]).clamp(0, max(0, free.numel() - 1))
    table.copy_(torch.where(fresh, free[at], table))
    t = torch.arange(cap, device=ctx.device)
    r = torch.searchsorted(cu[1:].long(), t, right=True).clamp(max=R - 1)
    live = (t < cu[-1]) & fits[r]
    pos = torch.where(live, ctx[r] + t - cu[r], 0)
    slot = table[r, pos // P] * P + pos % P
    kept = torch.where(fits, torch.maximum(held, total), held)
    return dict(cu_q=cu, q_req=torch.where(live, r, -1).to(torch.int32), q_pos=torch.where(live, pos, -1).to(torch.int32),
                slot=torch.where(live, slot, -1).to(torch.int32), ctx=torch.where(fits, ctx + new, ctx).to(torch.int32),
                held=kept.to(torch.int32), used=(used + need.sum()).to(torch.int32), table=table)


def _norm_rope(x, w, cos, sin, rope, interleaved):
    """fp32 [T, H, d]: the first len(w) values normed, then the last `rope` values rotated."""
    if w is not None:
        h = x[..., :w.numel()]
        h = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + 1e-6) * w
        x = torch.cat((h, x[..., w.numel():]), -1)
    r = x[..., x.shape[-1] - rope:]
    a, b = (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., :rope // 2], r[..., rope // 2:])
    c, s = cos[:, None, :], sin[:, None, :]
    a, b = a * c - b * s, a * s + b * c
    r = torch.stack((a, b), -1).flatten(-2) if interleaved else torch.cat((a, b), -1)
    return torch.cat((x[..., :x.shape[-1] - rope], r), -1)


def _qk_out(s, q, k):
    if s["case"]["cache"]:  # the cache's codes as the values they stand for, and the rows' scales
        return dict(q=q, kv=s["kv"].view(torch.float8_e4m3fn), kv_scale=s["kv_scale"])
    return dict(q=q, k=k)


def _plain_qk(s):
    c = s["case"]
    cs = s["cos_sin"][s["pos"].long()]
    cos, sin = cs[:, :c["rope"] // 2], cs[:, c["rope"] // 2:]
    q = _norm_rope(s["q"].float(), s["qw"], cos, sin, c["rope"], c["interleaved"]).to(torch.bfloat16)
    k = _norm_rope(s["k"].float(), s["kw"], cos, sin, c["rope"], c["interleaved"])
    if c["cache"]:
        k = k[:, 0]
        scale = k.abs().amax(1) / 448.0
        code = (k / scale[:, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
        s["kv"][s["slot"].long()] = code
        s["kv_scale"][s["slot"].long()] = scale
    return _qk_out(s, q, k.to(torch.bfloat16))


def _plain_mla(s):
    c = s["case"]
    R, n, P, H = c["req"], c["new"], c["page"], c["heads"]
    pos = torch.arange(c["ctx"], device=s["q"].device)
    slot = s["table"].long()[:, pos // P] * P + pos % P
    k = s["kv"][slot].view(torch.float8_e4m3fn).float() * s["kv_scale"][slot][..., None]
    # the tokens by request: row R takes the padding
    t = torch.arange(R * n, device=s["q"].device)
    r = torch.where(s["q_req"] >= 0, s["q_req"], R).long()
    start = torch.searchsorted(r, torch.arange(R + 1, device=r.device))
    j = t - start[r]
    j = torch.where(r < R, j, 0)
    q = torch.zeros((R + 1, n, H, s["q"].shape[2]), device=r.device)
    q[r, j] = s["q"].float()
    last = torch.full((R + 1, n), -1, dtype=torch.long, device=r.device)
    last[r, j] = s["q_pos"].long()
    z = torch.matmul(q[:R].flatten(1, 2), k.transpose(1, 2)).view(R, n, H, -1) * s["softmax_scale"]
    z = z.masked_fill((pos[None, None, :] > last[:R, :, None])[:, :, None, :], -math.inf)
    m = z.amax(-1, keepdim=True)
    z = z.sub_(torch.where(m == -math.inf, 0.0, m)).exp_()
    l = z.sum(-1, keepdim=True)
    o = torch.matmul(z.flatten(1, 2), k[..., :c["dl"]]).view(R, n, H, -1) / torch.where(l > 0, l, 1.0)
    lse = (m + l.log())[..., 0]
    rr = r.clamp(max=R - 1)
    live = r < R
    out = torch.where(live[:, None, None], o[rr, j], 0.0).to(torch.bfloat16)
    return dict(out=out, lse=torch.where(live[:, None], lse[rr, j], -math.inf))


def _plain_verify(s):
    R, n, V = s["case"]["req"], s["case"]["draft"], s["case"]["vocab"]
    cu, dev = s["cu"].long(), s["cu"].device
    drafts = cu[1:] - cu[:-1] - 1
    i = torch.arange(n + 1, device=dev)[None, :]
    real = i < drafts[:, None]
    row = torch.where(real, cu[:-1, None] + i, 0)
    tok = s["tok"].long()[row]
    p = s["target"].flatten()[row * V + tok].double()
    q = torch.ones_like(p) if s["draft"] is None else s["draft"].flatten()[row * V + tok].double()
    a = torch.cumprod(((s["u_accept"][row].double() * q < p) & real).long(), 1).sum(1)
    w = s["target"][cu[:-1] + a].double()
    bad = (a < drafts)[:, None]  # a rejected draft: its share of the probability is taken off
    if s["draft"] is None:
        less = torch.where(bad, torch.zeros_like(w).scatter_(1, tok.gather(1, a[:, None]), 2.0), 0.0)
    else:
        less = torch.where(bad, s["draft"][cu[:-1] + a].double(), 0.0)
    rest = (w - less).clamp(min=0)
    w = torch.where(rest.sum(1, keepdim=True) > 0, rest, w)
    cum = torch.cumsum(w, 1)
    y = (cum <= s["u_sample"].double()[:, None] * cum[:, -1:]).sum(1).clamp(max=V - 1)
    tokens = torch.where(i < a[:, None], tok, torch.where(i == a[:, None], y[:, None], -1))
    return dict(tokens=tokens.to(torch.int32), num=(a + 1).to(torch.int32), ctx=(s["ctx"] + a + 1).to(torch.int32))


# ---- what a pass cannot do without -------------------------------------------------


def work(case):
    c = case
    if c["op"] == "layout":
        R, cap = c["req"], c["req"] * c["new"]
        fresh = R * c["new"] / 2 / c["page"]  # pages taken, about: half the largest length for each request
        return dict(bytes=12 * R + 4 + 8 * fresh + 4 * R + 4 * (R + 1) + 12 * cap + 8 * R + 4, flops=4 * cap)
    if c["op"] == "qk":
        T, d = c["tokens"], c["d"]
        q = T * c["heads"] * d
        k = T * c["k_heads"] * d
        table = T * c["rope"] * 4 + 4 * T
        keys = k * 2 + (k + 8 * T if c["cache"] else k * 2)
        return dict(bytes=4 * q + keys + table + 4 * (c["q_norm"] + c["k_norm"]), flops=6 * (q + k))
    if c["op"] == "mla":
        R, n, dqk = c["req"], c["new"], c["dl"] + c["dr"]
        kv = c["ctx"] * (0.75 if c["ragged"] else 1.0)
        tok = R * ((n + 1) / 2 if c["ragged"] else n)
        seen = max(1.0, kv - n / 2)
        return dict(bytes=R * kv * (dqk + 4) + tok * c["heads"] * (2 * dqk + 2 * c["dl"] + 4),
                    flops=2 * tok * c["heads"] * seen * (dqk + c["dl"]))
    # verify: one row of the target for each request, and the draft's row where a token was
    # rejected (about half of them here); the drafted tokens' own probabilities
    R, n, V = c["req"], c["draft"], c["vocab"]
    per = V * 4 * (1.5 if c["probs"] else 1.0)
    return dict(bytes=R * (per + n / 2 * 16 + 4 * (n + 1) + 16), flops=3 * R * V)


# ---- the definitions in 64 bits ----------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    return {"layout": _exact_layout, "qk": _exact_qk, "mla": _exact_mla, "verify": _exact_verify}[case["op"]](s)


def _exact_layout(s):
    c = s["case"]
    ctx, new, held = (s[x].tolist() for x in ("ctx", "new", "held"))
    table, free, used, P = s["table"].cpu().numpy().copy(), s["free"].tolist(), int(s["used"]), c["page"]
    left = len(free) - used
    cu, req, pos, slot, asked = [0], [], [], [], 0
    taken = 0
    for r in range(len(ctx)):
        total = -(-(ctx[r] + new[r]) // P)
        need = max(0, total - held[r]) if new[r] > 0 else 0
        asked += need
        ok = need == 0 or asked <= left
        if ok:
            for x in range(need):
                table[r, held[r] + x] = free[used + asked - need + x]
            taken += need
        p = np.arange(ctx[r], ctx[r] + new[r])
        req.append(np.full(new[r], r if ok else -1))
        pos.append(p if ok else np.full(new[r], -1))
        slot.append(table[r, p // P].astype(np.int64) * P + p % P if ok else np.full(new[r], -1))
        cu.append(cu[-1] + new[r])
        if ok:
            ctx[r] += new[r]
            held[r] = max(held[r], total)
    pad = np.full(s["capacity"] - cu[-1], -1)
    i32 = lambda v: np.asarray(v, dtype=np.int32)  # noqa: E731
    return dict(cu_q=i32(cu), q_req=i32(np.concatenate(req + [pad])), q_pos=i32(np.concatenate(pos + [pad])),
                slot=i32(np.concatenate(slot + [pad])), ctx=i32(ctx), held=i32(held), used=i32([used + taken]), table=table)


def _exact_rows(x, w, pos, rope, interleaved, cos_sin):
    x = x.double()
    d = x.shape[-1]
    if w is not None:
        m = w.numel()
        rms = (x[..., :m].pow(2).sum(-1, keepdim=True) / m + 1e-6).sqrt()
        x[..., :m] = x[..., :m] / rms * w.double()
    t = cos_sin[pos.long()].double()
    z = torch.complex(t[:, :rope // 2], t[:, rope // 2:])[:, None, :]
    i = torch.arange(rope // 2, device=x.device)
    at = (d - rope + 2 * i, d - rope + 2 * i + 1) if interleaved else (d - rope + i, d - rope // 2 + i)
    v = torch.complex(x[..., at[0]], x[..., at[1]]) * z
    x[..., at[0]], x[..., at[1]] = v.real, v.imag
    return x


def _exact_qk(s):
    c = s["case"]
    q = _exact_rows(s["q"], s["qw"], s["pos"], c["rope"], c["interleaved"], s["cos_sin"])
    k = _exact_rows(s["k"], s["kw"], s["pos"], c["rope"], c["interleaved"], s["cos_sin"])
    if not c["cache"]:
        return dict(q=q, k=k)
    kv = torch.zeros(s["kv"].shape, dtype=torch.float64, device=DEV)
    scale = torch.zeros(s["kv_scale"].shape, dtype=torch.float64, device=DEV)
    top = k[:, 0].abs().amax(1) / 448
    kv[s["slot"].long()] = k[:, 0] / top[:, None]
    scale[s["slot"].long()] = top
    return dict(q=q, kv=kv, kv_scale=scale)


def _e4m3_values():
    b = np.arange(256)
    e, m = (b >> 3) & 15, b & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e.astype(float) - 10))
    v[(b & 127) == 127] = np.nan
    return np.where(b >= 128, -v, v)


def _exact_mla(s):
    c = s["case"]
    P, dl = c["page"], c["dl"]
    values = torch.from_numpy(_e4m3_values()).to(DEV)
    req, pos = s["q_req"].tolist(), s["q_pos"].tolist()
    out = torch.zeros((len(req), c["heads"], dl), dtype=torch.float64, device=DEV)
    lse = torch.full((len(req), c["heads"]), -math.inf, dtype=torch.float64, device=DEV)
    for r in range(c["req"]):
        rows = [t for t in range(len(req)) if req[t] == r]
        end = max(pos[t] for t in rows) + 1
        slots = torch.tensor([int(p) * P + o for p in s["table"][r].tolist() for o in range(P)][:end], device=DEV)
        x = values[s["kv"][slots].long()] * s["kv_scale"][slots].double()[:, None]
        for at in range(0, len(rows), 128):
            part = rows[at:at + 128]
            z = torch.einsum("thd,kd->thk", s["q"][part].double(), x) * s["softmax_scale"]
            seen = torch.arange(end, device=DEV)[None, :] <= torch.tensor([pos[t] for t in part], device=DEV)[:, None]
            z = torch.where(seen[:, None, :], z, -math.inf)
            n = torch.logsumexp(z, -1)
            lse[part] = n
            out[part] = torch.einsum("thk,kd->thd", torch.exp(z - n[..., None]), x[:, :dl])
    return dict(out=out, lse=lse)


def _exact_verify(s):
    c = s["case"]
    cu = s["cu"].tolist()
    tok, ua, us, ctx = s["tok"].tolist(), s["u_accept"].tolist(), s["u_sample"].tolist(), s["ctx"].tolist()
    tokens = np.full((c["req"], c["draft"] + 1), -1, dtype=np.int32)
    num = []
    for r in range(c["req"]):
        a, n, at = 0, cu[r + 1] - cu[r] - 1, cu[r]
        while a < n:
            x = tok[at + a]
            q = 1.0 if s["draft"] is None else float(s["draft"][at + a, x])
            if not ua[at + a] * q < float(s["target"][at + a, x]):
                break
            tokens[r, a] = x
            a += 1
        p = s["target"][at + a].cpu().numpy().astype(np.float64)
        w = p
        if a < n:
            w = p.copy()
            if s["draft"] is None:
                w[tok[at + a]] = 0
            else:
                w = np.maximum(p - s["draft"][at + a].cpu().numpy().astype(np.float64), 0)
            if w.sum() == 0:
                w = p
        cum = np.cumsum(w)
        tokens[r, a] = min(int(np.searchsorted(cum, us[r] * cum[-1], side="right")), len(w) - 1)
        num.append(a + 1)
    i32 = lambda v: np.asarray(v, dtype=np.int32)  # noqa: E731
    return dict(tokens=tokens, num=i32(num), ctx=i32(ctx) + i32(num))
