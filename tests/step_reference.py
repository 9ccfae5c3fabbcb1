"""Plain 64-bit definitions of the serving step's operators (numpy), for the tests."""
import numpy as np

BAD_QPOS, BAD_INDEX, BAD_PAGE, NO_PAGES = 1, 2, 4, 16


def batch_layout(ctx, new, held, table, free, used, *, page_size, num_pages, capacity):
    """Returns (dict of outputs, dev status); table is copied."""
    ctx, new, held, table = ctx.astype(np.int64), new.astype(np.int64), held.astype(np.int64), table.copy()
    P, status = page_size, 0
    left = len(free) - used
    if used < 0 or left < 0:
        status, left = status | BAD_INDEX, 0
    cu = [0]
    req, pos, slot = (np.full(capacity, -1, dtype=np.int64) for _ in range(3))
    asked, taken, tokens, full = 0, 0, 0, False
    ctx_out, held_out = ctx.copy(), held.copy()
    for r in range(len(ctx)):
        n, need, ok = int(new[r]), 0, True
        if ctx[r] < 0 or n < 0 or held[r] < 0:
            status |= BAD_QPOS
            n, ok = 0, False
        elif n > 0:
            total = -(-(ctx[r] + n) // P)
            if total > table.shape[1] or ctx[r] + n > 2**31 - 1:
                status |= BAD_INDEX
                ok = False
            else:
                need = max(0, int(total - held[r]))
        tokens += n
        asked += need
        if tokens > capacity and n > 0:
            status |= BAD_INDEX
            ok, full = False, True
        if ok and need > 0 and asked > left:
            status |= NO_PAGES
            ok = False
        first = cu[-1]
        cu.append(first if full else first + n)
        if not ok:
            continue
        for x in range(need):
            table[r, held[r] + x] = free[used + asked - need + x]
        if need:
            taken = asked
        for j in range(n):
            p = int(ctx[r]) + j
            t = first + j
            req[t], pos[t] = r, p
            page = table[r, p // P]
            if 0 <= page < num_pages:
                slot[t] = int(page) * P + p % P
            else:
                status |= BAD_PAGE
        ctx_out[r] = ctx[r] + n
        held_out[r] = held[r] + need
    return dict(cu_q=np.array(cu), q_req=req, q_pos=pos, slot=slot, ctx_len=ctx_out, pages_held=held_out,
                free_used=np.array([used + taken]), table=table), status


def norm_rope(x, weight, pos, cos_sin, d_rope, interleaved, eps):
    """x [T, H, d] float64 -> the normed and rotated rows."""
    y = x.astype(np.float64).copy()
    n, d = 0 if weight is None else len(weight), y.shape[2]
    if n:
        rms = np.sqrt((y[..., :n] ** 2).mean(-1, keepdims=True) + eps)
        y[..., :n] = y[..., :n] * weight.astype(np.float64) / rms
    h = d_rope // 2
    for i in range(h):
        a, b = (d - d_rope + 2 * i, d - d_rope + 2 * i + 1) if interleaved else (d - d_rope + i, d - h + i)
        c, s = (cos_sin[pos, j].astype(np.float64)[:, None] for j in (i, h + i))
        ya, yb = y[..., a].copy(), y[..., b].copy()
        y[..., a], y[..., b] = ya * c - yb * s, ya * s + yb * c
    return y


def verify_draft(p, q, tok, cu, u_accept, u_sample, max_out):
    """Returns (tokens, num_out, status); p, q float32 rows (q None: certain drafts)."""
    R, V = len(cu) - 1, p.shape[1]
    tokens = np.full((R, max_out), -1, dtype=np.int64)
    num, status = np.zeros(R, dtype=np.int64), 0

    def clean(x):  # NaN and negative values count as 0, values above 1 as 1
        x = np.where(np.isnan(x), 0.0, x.astype(np.float64))
        return np.clip(x, 0.0, 1.0)

    for r in range(R):
        lo, hi = int(cu[r]), int(cu[r + 1])
        if lo < 0 or hi < lo or hi > len(p):
            status |= BAD_INDEX
            continue
        if hi == lo:
            continue
        n, a = hi - lo - 1, 0
        if n > max_out - 1:
            n, status = max_out - 1, status | BAD_INDEX
        while a < n:
            x = int(tok[lo + a])
            if not 0 <= x < V:
                status |= BAD_INDEX
                break
            qx = 1.0 if q is None else float(q[lo + a, x])
            if not float(u_accept[lo + a]) * qx < float(p[lo + a, x]):
                break
            tokens[r, a] = x
            a += 1
        w = clean(p[lo + a])
        if a < n:
            if q is None:
                rest = w.copy()
                if 0 <= tok[lo + a] < V:
                    rest[tok[lo + a]] = 0
            else:
                rest = np.maximum(w - clean(q[lo + a]), 0)
            if rest.sum() > 0:
                w = rest
        c = np.cumsum(w)
        tokens[r, a] = min(int(np.searchsorted(c, float(u_sample[r]) * c[-1], side="right")), V - 1)
        num[r] = a + 1
    return tokens, num, status
