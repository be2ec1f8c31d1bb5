"""Plain 64-bit forms of the paged step's operators (numpy, one row at a time)."""
import numpy as np

PAGE = 16


def pages(n):
    return -(-int(n) // PAGE)


def resize(old, new, table, free, n_free, T, n_pages):
    """paged_resize: (status, cu, slot, pos, table, free, n_free), inputs untouched."""
    B, mp = table.shape
    table, free = table.copy(), free.copy()
    fail = lambda s: (s, np.zeros(B + 1, int), np.full(T, -1), np.full(T, -1), table, free, n_free)  # noqa: E731
    take = [(b, i) for b in range(B) for i in range(pages(max(old[b], 0)), pages(max(new[b], 0)))]
    give = [(b, i) for b in range(B) for i in range(pages(max(new[b], 0)), pages(max(old[b], 0)))]
    rows = [max(0, int(n) - int(o)) for o, n in zip(old, new)]
    A, R = len(take), len(give)
    if min(old) < 0 or min(new) < 0 or not 0 <= n_free <= n_pages or sum(rows) > T or n_free - A + R > n_pages:
        return fail(1)
    if max(old) > PAGE * mp or max(new) > PAGE * mp:
        return fail(2)
    if A > n_free:
        return fail(3)
    moved = [free[n_free - 1 - i] for i in range(A)] + [table[b, i] for b, i in give]
    if any(not 0 <= p < n_pages for p in moved):
        return fail(1)
    for i, (b, j) in enumerate(take):
        table[b, j] = free[n_free - 1 - i]
    cu = np.concatenate([[0], np.cumsum(rows)])
    slot, pos = np.full(T, -1), np.full(T, -1)
    for b in range(B):
        for t in range(rows[b]):
            p = old[b] + t
            pos[cu[b] + t] = p
            pg = table[b, p // PAGE]
            if 0 <= pg < n_pages:
                slot[cu[b] + t] = pg * PAGE + p % PAGE
    for k, (b, j) in enumerate(give):
        free[n_free - A + R - 1 - k] = table[b, j]
        table[b, j] = -1
    return 0, cu, slot, pos, table, free, n_free - A + R


def rope(x, p, base):
    """Half-split rotation of the last dimension by position p."""
    d = x.shape[-1]
    a = float(p) * float(base) ** (-2.0 * np.arange(d // 2) / d)
    c, s = np.cos(a), np.sin(a)
    u, v = x[..., :d // 2], x[..., d // 2:]
    return np.concatenate([u * c - v * s, v * c + u * s], -1)


def head_norm(x, g, eps):
    return x if g is None else x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * g


def attend(q, K, V, allowed, scale, cap):
    """q [G][d], K, V [n][d], allowed [n]: (out [G][d], sum of p |v|)."""
    if not allowed.any():
        z = np.zeros((q.shape[0], V.shape[1]))
        return z, z
    K, V = K[allowed], V[allowed]
    s = q @ K.T * scale
    if cap > 0:
        s = cap * np.tanh(s / cap)
    e = np.exp(s - s.max(1, keepdims=True))
    e /= e.sum(1, keepdims=True)
    return e @ V, e @ np.abs(V)


def chunk_attn(q, kp, vp, table, cu, kv_len, scale, window=0, cap=0.0, out=None):
    """gqa_chunk_attn: out [T][nq][d] (rows of nobody from `out`) and sum_j p_j |v_j|."""
    T, nq, d = q.shape
    P, nkv = kp.shape[:2]
    G = nq // nkv
    out = np.zeros((T, nq, d)) if out is None else out.copy()
    mag = np.zeros((T, nq, d))
    for b in range(len(kv_len)):
        L = min(int(kv_len[b]), PAGE * table.shape[1])
        pg = np.repeat(table[b], PAGE)[:max(L, 0)]
        ok = (pg >= 0) & (pg < P)
        at = np.where(ok, pg, 0)
        off = np.arange(len(pg)) % PAGE
        n = cu[b + 1] - cu[b]
        for i in range(n):
            p = L - n + i
            j = np.arange(len(pg))
            see = ok & (j <= p) & ((j > p - window) if window else True)
            for g in range(nkv):
                r = cu[b] + i
                hs = slice(g * G, (g + 1) * G)
                out[r, hs], mag[r, hs] = attend(q[r, hs], kp[at, g, off], vp[at, g, off], see, scale, cap)
    return out, mag


def chunk_attn_on_device(q, kp, vp, table, cu, kv_len, scale, window=0, cap=0.0):
    """chunk_attn for long sequences: the same in 64-bit torch on q's device, one (sequence, kv
    head, block of rows) at a time. Pools without NaN; every row in a sequence, every page good."""
    import torch
    T, nq, d = q.shape
    nkv = kp.shape[1]
    G = nq // nkv
    out = torch.zeros((T, nq, d), dtype=torch.float64, device=q.device)
    mag = torch.zeros_like(out)
    for b in range(len(kv_len)):
        L, n = int(kv_len[b]), int(cu[b + 1] - cu[b])
        j = torch.arange(L, device=q.device)
        pg = torch.as_tensor(table[b], device=q.device).long()[j // PAGE]
        for g in range(nkv):
            K, V = kp[pg, g, j % PAGE].double(), vp[pg, g, j % PAGE].double()
            for r in range(0, n, 512):
                i = torch.arange(r, min(n, r + 512), device=q.device)
                p = (L - n + i)[:, None, None]
                s = torch.einsum("tgd,jd->tgj", q[cu[b] + i, g * G:(g + 1) * G].double(), K) * scale
                if cap > 0:
                    s = cap * torch.tanh(s / cap)
                hide = j > p
                if window:
                    hide = hide | (j <= p - window)
                e = torch.softmax(s.masked_fill(hide, -float("inf")), -1)
                out[cu[b] + i, g * G:(g + 1) * G] = e @ V
                mag[cu[b] + i, g * G:(g + 1) * G] = e @ V.abs()
    return out.cpu().numpy(), mag.cpu().numpy()


def softmax(l):
    m = l.max()
    if m == -np.inf:
        return np.zeros_like(l)
    e = np.exp(l - m)
    return e / e.sum()


def verify(target, draft, tok, count, temp, u, us):
    """spec_verify of one sequence: (accepted, next token)."""
    n, V = tok.shape[0], target.shape[1]
    count = min(max(int(count), 0), n)
    target = np.asarray(target, np.float64)
    acc = 0
    if not temp > 0:
        while acc < count and target[acc].max() > -np.inf and tok[acc] == target[acc].argmax():
            acc += 1
        return acc, int(target[acc].argmax()) if target[acc].max() > -np.inf else -1
    row = lambda l: softmax(np.asarray(l, np.float64) / np.float64(temp))  # noqa: E731
    while acc < count:
        x = tok[acc]
        if not 0 <= x < V:
            break
        q = 1.0 if draft is None else row(draft[acc])[x]
        if not np.float64(u[acc]) * q < row(target[acc])[x]:
            break
        acc += 1
    p = row(target[acc])
    w = p
    if acc < count:
        if draft is not None:
            w = np.maximum(p - row(draft[acc]), 0)
        elif 0 <= tok[acc] < V:
            w = p.copy()
            w[tok[acc]] = 0
    if not w.sum() > 0:
        w = p
    if not w.sum() > 0:
        return acc, -1
    C = np.cumsum(w)
    hit = np.nonzero((C > np.float64(us) * C[-1]) & (w > 0))[0]
    return acc, int(hit[0]) if len(hit) else int(np.nonzero(w > 0)[0][-1])
