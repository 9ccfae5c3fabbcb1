"""Latent attention's other form, the products around it, and the log probabilities
of a step's tokens, as measured cases.

  absorb   queries into the latent space of the cache (``absorb_q``)
  project  attention's latent outputs to the heads' values (``project_out``)
  expand   cached latent rows to every head's keys and values (``expand_kv``)
  prompt   attention over those, for prompts and their chunks (``prompt_mla``)
  logp     log probabilities, entropy, rank and alternatives of tokens
           (``token_logprobs``)

With ``own`` false ``run`` computes them in plain torch operations in 32 bits;
with ``own`` true it makes the library's calls.  ``exact`` gives the same from
the definitions in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"


# ---- cases -----------------------------------------------------------------------

# head shapes: heads, width of a head's key without position, rotated width, value width, latent width
LARGE = dict(heads=64, dn=128, dr=64, dv=128, dl=512)
SMALL = dict(heads=16, dn=32, dr=16, dv=32, dl=64)


def listed():
    return [
        # one decode step of eight requests: latency, and the weights' one read
        dict(LARGE, name="absorb decode 8", op="absorb", tokens=8),
        # an odd number of tokens of a prefill chunk
        dict(LARGE, name="absorb chunk 4099", op="absorb", tokens=4099),
        # decode of 128 requests
        dict(LARGE, name="project decode 128", op="project", tokens=128),
        # a large prefill chunk
        dict(LARGE, name="project chunk 8192", op="project", tokens=8192),
        # the cached prefixes of five short requests, a page size that no tile divides
        dict(LARGE, name="expand 5x ctx 333", op="expand", req=5, ctx=333, ragged=True, page=48),
        # a long context before a chunk of it is prefilled
        dict(LARGE, name="expand 1x16384", op="expand", req=1, ctx=16384, ragged=False, page=64),
        # the small head shape: two short prompts
        dict(SMALL, name="prompt small 2x200", op="prompt", req=2, new=200, ctx=200, ragged=True),
        # eight prompts of up to 2,048 tokens admitted together, on up to 1,000 cached positions
        dict(LARGE, name="prompt 8x2048 ragged", op="prompt", req=8, new=2048, ctx=3048, ragged=True),
        # a prefill chunk of 1,024 tokens at the end of a 16K context
        dict(LARGE, name="prompt 1024 of 16384", op="prompt", req=1, new=1024, ctx=16384, ragged=False),
        # one long prompt from its first token
        dict(LARGE, name="prompt 1x8192", op="prompt", req=1, new=8192, ctx=8192, ragged=False),
        # a decode step of four requests, a small odd vocabulary, fp32 logits, five alternatives
        dict(name="logp 4x32003 fp32", op="logp", rows=4, vocab=32003, dtype="float32", top=5, masked=0.0),
        # a verify step's 1,024 rows over a large vocabulary whose last part is masked, 20 alternatives
        dict(name="logp 1024x131072 bf16", op="logp", rows=1024, vocab=131072, dtype="bfloat16", top=20, masked=0.02),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("absorb", "project", "expand", "prompt", "logp"))
    shape = LARGE if rng.random() < 0.8 else SMALL
    if op in ("absorb", "project"):
        return dict(shape, op=op, tokens=_log(rng, 1, 8192))
    if op == "expand":
        req = _log(rng, 1, 64)
        return dict(shape, op=op, req=req, ctx=_log(rng, 1, 16384 // req), ragged=rng.random() < 0.7,
                    page=rng.choice((1, 16, 48, 64, 128)))
    if op == "prompt":
        req, new = _log(rng, 1, 32), _log(rng, 1, 4096)
        cached = 0 if rng.random() < 0.4 else _log(rng, 1, 8192)
        new = min(new, max(1, int(math.sqrt((1 << 25) // req))))
        cached = min(cached, max(0, (1 << 25) // (req * new) - new))
        return dict(shape, op=op, req=req, new=new, ctx=new + min(cached, 65536 // req), ragged=rng.random() < 0.7)
    vocab = _log(rng, 1000, 262144)
    return dict(op=op, rows=_log(rng, 1, min(1024, (1 << 26) // vocab)), vocab=vocab,
                dtype=rng.choice(("float32", "bfloat16", "float16")), top=rng.choice((0, 1, 5, 20)),
                masked=rng.choice((0.0, 0.02, 0.5)))


# ---- inputs ----------------------------------------------------------------------


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 6151 + 29)
    return g


def _ints(lo, hi, n, g):
    """int32 [n], uniform in lo..hi (both included)."""
    return torch.randint(lo, hi + 1, (n,), generator=g, device=DEV, dtype=torch.int32)


def _bf16(shape, g):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16)


def _weight(c, g):
    """The up-projection of every head's keys and values, as it stands in a checkpoint."""
    w = torch.randn((c["heads"], c["dn"] + c["dv"], c["dl"]), generator=g, device=DEV)
    return (w * c["dl"] ** -0.5).to(torch.bfloat16)


def _starts(lengths):
    cu = torch.zeros(lengths.numel() + 1, dtype=torch.int32, device=DEV)
    cu[1:] = torch.cumsum(lengths, 0)
    return cu


def prepare(case, seed):
    g = _gen(seed)
    make = {"absorb": _prepare_absorb, "project": _prepare_project, "expand": _prepare_expand, "prompt": _prepare_prompt,
            "logp": _prepare_logp}[case["op"]]
    return dict(make(case, g), case=case)


def _prepare_absorb(c, g):
    return dict(q=_bf16((c["tokens"], c["heads"], c["dn"] + c["dr"]), g), w=_weight(c, g))


def _prepare_project(c, g):
    return dict(o=_bf16((c["tokens"], c["heads"], c["dl"]), g), w=_weight(c, g))


def _prepare_expand(c, g):
    R, P, d = c["req"], c["page"], c["dl"] + c["dr"]
    ctx = _ints((c["ctx"] + 1) // 2, c["ctx"], R, g) if c["ragged"] else torch.full((R,), c["ctx"], dtype=torch.int32, device=DEV)
    stride = (c["ctx"] + P - 1) // P
    table = torch.randperm(R * stride, generator=g, device=DEV).to(torch.int32).view(R, stride).contiguous()
    rows = torch.randn((R * stride * P, d), generator=g, device=DEV)
    scale = rows.abs().amax(1) / 448.0
    kv = (rows / scale[:, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
    # the buffers that a program keeps for the expanded rows, of the largest batch's size: rows
    # behind the last request stay as they are
    n = R * c["ctx"]
    return dict(kv=kv, scale=scale.contiguous(), table=table, ctx=ctx, w=_weight(c, g),
                out_kv=torch.zeros((n, c["heads"], c["dn"] + c["dv"]), dtype=torch.bfloat16, device=DEV),
                out_rope=torch.zeros((n, c["dr"]), dtype=torch.bfloat16, device=DEV),
                out_cu=torch.zeros(R + 1, dtype=torch.int32, device=DEV))


def _prepare_prompt(c, g):
    R, n, H = c["req"], c["new"], c["heads"]
    if c["ragged"]:
        new = _ints((n + 1) // 2, n, R, g)
        ctx = new + _ints(0, c["ctx"] - n, R, g)
    else:
        new = torch.full((R,), n, dtype=torch.int32, device=DEV)
        ctx = torch.full((R,), c["ctx"], dtype=torch.int32, device=DEV)
    cu_q, cu_k = _starts(new), _starts(ctx)
    T, N = R * n, R * c["ctx"]  # the batch's capacities: the tokens past cu_q[R] are padding
    t = torch.arange(T, device=DEV, dtype=torch.int32)
    r = torch.searchsorted(cu_q[1:], t, right=True).clamp(max=R - 1)
    pos = torch.where(t < cu_q[-1], ctx[r] - new[r] + t - cu_q[r], -1).to(torch.int32)
    return dict(q=_bf16((T, H, c["dn"] + c["dr"]), g), kv=_bf16((N, H, c["dn"] + c["dv"]), g), rope=_bf16((N, c["dr"]), g),
                cu_q=cu_q, cu_k=cu_k, pos=pos, scale=(c["dn"] + c["dr"]) ** -0.5)


def _prepare_logp(c, g):
    z = torch.randn((c["rows"], c["vocab"]), generator=g, device=DEV) * 3.0
    cut = int(c["vocab"] * (1 - c["masked"]))
    if cut < c["vocab"]:
        z[:, cut:] = -math.inf
    # sampled tokens: the smallest of exponential clocks
    tok = (z - torch.empty_like(z).exponential_(generator=g).log_()).argmax(1).to(torch.int32)
    return dict(z=z.to(getattr(torch, c["dtype"])), tok=tok)


# ---- one pass --------------------------------------------------------------------


def run(state):
    op = state["case"]["op"]
    if own:
        return {"absorb": _own_absorb, "project": _own_project, "expand": _own_expand, "prompt": _own_prompt, "logp": _own_logp}[op](state)
    return {"absorb": _plain_absorb, "project": _plain_project, "expand": _plain_expand, "prompt": _plain_prompt,
            "logp": _plain_logp}[op](state)


def _own_absorb(s):
    import dsa_sparse_mla_topk_gb300 as dsa

    return dsa.absorb_q(s["q"], s["w"], d_rope=s["case"]["dr"])


def _own_project(s):
    import dsa_sparse_mla_topk_gb300 as dsa

    return dsa.project_out(s["o"], s["w"], d_nope=s["case"]["dn"])


def _own_expand(s):
    import dsa_sparse_mla_topk_gb300 as dsa

    x = dsa.expand_kv(s["kv"], s["scale"], s["table"], s["ctx"], s["w"], d_rope=s["case"]["dr"], page_size=s["case"]["page"],
                      out=dsa.ExpandedKV(s["out_kv"], s["out_rope"], s["out_cu"]))
    return dict(kv=x.kv, k_rope=x.k_rope, cu_k=x.cu_k)


def _own_prompt(s):
    import dsa_sparse_mla_topk_gb300 as dsa

    out, lse = dsa.prompt_mla(s["q"], s["kv"], s["rope"], s["cu_q"], s["cu_k"], s["pos"], d_nope=s["case"]["dn"],
                              softmax_scale=s["scale"])
    return dict(out=out, lse=lse)


def _own_logp(s):
    import dsa_sparse_mla_topk_gb300 as dsa

    r = dsa.token_logprobs(s["z"], s["tok"], top=s["case"]["top"])
    return dict(logprob=r.logprob, entropy=r.entropy, rank=r.rank, top_ids=r.top_ids, top_logprobs=r.top_logprobs)


def _plain_absorb(s):
    dn = s["case"]["dn"]
    x = torch.matmul(s["q"][..., :dn].float().transpose(0, 1), s["w"][:, :dn].float()).transpose(0, 1)
    return torch.cat((x.to(torch.bfloat16), s["q"][..., dn:]), -1)


def _plain_project(s):
    dn = s["case"]["dn"]
    x = torch.matmul(s["o"].float().transpose(0, 1), s["w"][:, dn:].float().transpose(1, 2))
    return x.transpose(0, 1).to(torch.bfloat16).contiguous()


def _plain_expand(s):
    c, P = s["case"], s["case"]["page"]
    cu = _starts(s["ctx"])
    pos = torch.arange(c["ctx"], device=DEV)
    live = pos[None, :] < s["ctx"][:, None]
    slot = (s["table"].long()[:, pos // P] * P + pos % P)[live]
    x = s["kv"][slot].view(torch.float8_e4m3fn).float() * s["scale"][slot][:, None]
    n = slot.numel()
    y = torch.matmul(x[:, :c["dl"]], s["w"].float().flatten(0, 1).t())
    s["out_kv"][:n] = y.view(n, c["heads"], -1).to(torch.bfloat16)
    s["out_rope"][:n] = x[:, c["dl"]:].to(torch.bfloat16)
    s["out_cu"].copy_(cu)
    return dict(kv=s["out_kv"], k_rope=s["out_rope"], cu_k=s["out_cu"])


def _plain_prompt(s):
    c = s["case"]
    R, n, m, H, dn = c["req"], c["new"], c["ctx"], c["heads"], c["dn"]
    # the requests side by side, each padded to the largest
    i, j = torch.arange(n, device=DEV), torch.arange(m, device=DEV)
    q_len, k_len = s["cu_q"].diff(), s["cu_k"].diff()
    here = i[None, :] < q_len[:, None]
    row = torch.where(here, s["cu_q"][:-1, None] + i, 0)
    col = (s["cu_k"][:-1, None] + j).clamp(max=s["kv"].shape[0] - 1)
    q = s["q"].float()[row].transpose(1, 2)                                     # [R, H, n, dn + dr]
    kv = s["kv"].float()[col].transpose(1, 2)                                   # [R, H, m, dn + dv]
    rope = s["rope"].float()[col][:, None].expand(-1, H, -1, -1)
    z = torch.matmul(q, torch.cat((kv[..., :dn], rope), -1).transpose(2, 3)).mul_(s["scale"])
    last = torch.where(here, s["pos"][row], -1)
    seen = (j[None, None, :] <= last[:, :, None]) & (j[None, None, :] < k_len[:, None, None])
    z.masked_fill_(~seen[:, None], -math.inf)
    top = z.amax(-1, keepdim=True)
    z.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    l = z.sum(-1, keepdim=True)
    o = torch.matmul(z, kv[..., dn:]) / torch.where(l > 0, l, 1.0)
    lse = (top + l.log())[..., 0]
    out = torch.zeros((R * n, H, c["dv"]), dtype=torch.bfloat16, device=DEV)
    out_lse = torch.full((R * n, H), -math.inf, device=DEV)
    out[row[here]] = o.transpose(1, 2)[here].to(torch.bfloat16)
    out_lse[row[here]] = lse.transpose(1, 2)[here]
    return dict(out=out, lse=out_lse)


def _plain_logp(s):
    z, tok = s["z"].float(), s["tok"].long()[:, None]
    top = z.amax(1, keepdim=True)
    d = z - top
    e = d.exp()
    total = e.sum(1, keepdim=True, dtype=torch.float64)  # 64 bits: a sure token's logarithm is next to nothing
    log_total = total.log()
    at = d.gather(1, tok)
    logprob = (at.double() - log_total).float()
    entropy = (log_total - (e * torch.where(d == -math.inf, 0.0, d)).sum(1, keepdim=True, dtype=torch.float64) / total).float()
    col = torch.arange(z.shape[1], device=DEV)[None, :]
    rank = ((d > at) | ((d == at) & (col < tok))).sum(1)
    ids = torch.sort(z, dim=1, descending=True, stable=True)[1][:, :s["case"]["top"]]
    return dict(logprob=logprob[:, 0], entropy=entropy[:, 0], rank=rank.to(torch.int32), top_ids=ids.to(torch.int32),
                top_logprobs=(d.gather(1, ids).double() - log_total).float())


# ---- what a pass cannot do without -------------------------------------------------


def work(case):
    c = case
    if c["op"] == "logp":
        size = 4 if c["dtype"] == "float32" else 2
        return dict(bytes=c["rows"] * (c["vocab"] * size + 16 + 8 * c["top"]), flops=5 * c["rows"] * c["vocab"])
    H, dn, dr, dv, dl = (c[x] for x in ("heads", "dn", "dr", "dv", "dl"))
    if c["op"] == "absorb":
        return dict(bytes=2 * c["tokens"] * H * (dn + dl + 2 * dr) + 2 * H * dn * dl, flops=2 * c["tokens"] * H * dn * dl)
    if c["op"] == "project":
        return dict(bytes=2 * c["tokens"] * H * (dl + dv) + 2 * H * dv * dl, flops=2 * c["tokens"] * H * dv * dl)
    if c["op"] == "expand":
        n = c["req"] * c["ctx"] * (0.75 if c["ragged"] else 1.0)
        return dict(bytes=n * (dl + dr + 4 + 2 * H * (dn + dv) + 2 * dr) + 2 * H * (dn + dv) * dl,
                    flops=2 * n * H * (dn + dv) * dl)
    new = c["new"] * (0.75 if c["ragged"] else 1.0)
    ctx = new + (c["ctx"] - c["new"]) * (0.5 if c["ragged"] else 1.0)
    pairs = c["req"] * new * (ctx - (new - 1) / 2)
    return dict(bytes=2 * c["req"] * (new * H * (dn + dr + dv + 2) + ctx * (H * (dn + dv) + dr)),
                flops=2 * pairs * H * (dn + dr + dv))


# ---- the definitions in 64 bits ----------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    return {"absorb": _exact_absorb, "project": _exact_project, "expand": _exact_expand, "prompt": _exact_prompt,
            "logp": _exact_logp}[case["op"]](s)


def _exact_absorb(s):
    dn, dl = s["case"]["dn"], s["case"]["dl"]
    y = torch.empty((*s["q"].shape[:2], dl + s["case"]["dr"]), dtype=torch.float64, device=DEV)
    for h in range(s["case"]["heads"]):
        y[:, h, :dl] = s["q"][:, h, :dn].double() @ s["w"][h, :dn].double()
        y[:, h, dl:] = s["q"][:, h, dn:].double()
    return y


def _exact_project(s):
    return torch.stack([s["o"][:, h].double() @ s["w"][h, s["case"]["dn"]:].double().t() for h in range(s["case"]["heads"])], 1)


def _e4m3_values():
    b = torch.arange(256, device=DEV)
    e, m = (b >> 3) & 15, (b & 7).double()
    v = torch.where(e == 0, m * 2.0 ** -9, (8 + m) * torch.pow(2.0, e.double() - 10))
    v = torch.where((b & 127) == 127, math.nan, v)
    return torch.where(b >= 128, -v, v)


def _exact_expand(s):
    c, values = s["case"], _e4m3_values()
    kv, rope = torch.zeros_like(s["out_kv"], dtype=torch.float64), torch.zeros_like(s["out_rope"], dtype=torch.float64)
    cu, w = [0], s["w"].double()
    for r, n in enumerate(s["ctx"].tolist()):
        pages = s["table"][r].tolist()
        slots = torch.tensor([pages[p // c["page"]] * c["page"] + p % c["page"] for p in range(n)], device=DEV)
        x = values[s["kv"][slots].long()] * s["scale"][slots].double()[:, None]
        kv[cu[-1]:cu[-1] + n] = torch.einsum("nl,hdl->nhd", x[:, :c["dl"]], w)
        rope[cu[-1]:cu[-1] + n] = x[:, c["dl"]:]
        cu.append(cu[-1] + n)
    return dict(kv=kv, k_rope=rope, cu_k=torch.tensor(cu, dtype=torch.int32))


def _exact_prompt(s):
    c, dn = s["case"], s["case"]["dn"]
    out = torch.zeros((s["q"].shape[0], c["heads"], c["dv"]), dtype=torch.float64, device=DEV)
    lse = torch.full(out.shape[:2], -math.inf, dtype=torch.float64, device=DEV)
    cu_q, cu_k, pos = s["cu_q"].tolist(), s["cu_k"].tolist(), s["pos"].tolist()
    for r in range(c["req"]):
        for at in range(cu_q[r], cu_q[r + 1], 512):
            to = min(at + 512, cu_q[r + 1])
            end = max(pos[at:to]) + 1
            rows = slice(cu_k[r], cu_k[r] + end)
            k, q = s["kv"][rows], s["q"][at:to].double()
            z = torch.einsum("thd,khd->htk", q[..., :dn], k[..., :dn].double())
            z = (z + torch.einsum("thd,kd->htk", q[..., dn:], s["rope"][rows].double())) * s["scale"]
            hide = torch.arange(end, device=DEV)[None, :] > torch.tensor(pos[at:to], device=DEV)[:, None]
            z[:, hide] = -math.inf
            n = torch.logsumexp(z, -1)
            lse[at:to] = n.t()
            out[at:to] = torch.einsum("htk,khd->thd", torch.exp(z - n[..., None]), k[..., dn:].double())
    return dict(out=out, lse=lse)


def _exact_logp(s):
    k, made = s["case"]["top"], []
    for z, t in zip(s["z"], s["tok"].tolist()):
        z = z.double()
        lp = torch.log_softmax(z, 0)
        p = lp.exp()
        entropy = -torch.where(p > 0, p * lp, 0.0).sum()
        rank = int((z > z[t]).sum() + (z[:t] == z[t]).sum())
        ids = []
        if k:
            near = torch.nonzero(z >= torch.topk(z, k)[0][-1])[:, 0]
            ids = sorted(near.tolist(), key=dict(zip(near.tolist(), (-z[near]).tolist())).get)[:k]  # stable: lower ids first
        made.append((float(lp[t]), float(entropy), rank, ids, lp[ids].tolist() if k else []))
    lp, entropy, rank, ids, top = zip(*made)
    f64 = lambda v, *shape: torch.tensor(v, dtype=torch.float64).view(*shape)  # noqa: E731
    i32 = lambda v, *shape: torch.tensor(v, dtype=torch.int32).view(*shape)  # noqa: E731
    n = len(made)
    return dict(logprob=f64(lp, n), entropy=f64(entropy, n), rank=i32(rank, n), top_ids=i32(ids, n, k), top_logprobs=f64(top, n, k))
