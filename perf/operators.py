"""Cases of the paged serving operators: block tables and slot maps (paged_resize), rotary
positions with the append to the paged cache (paged_rope_append), attention of new rows over
the cache (gqa_chunk_attn) and the verification of drafted tokens (spec_verify).

run() computes each operator in plain torch operations, or with ``own`` set through the
package's entry points. Sizes are those of the shapes in synth/configs.py (heads 32/8 x 128,
16/16 x 128, 9/3 x 64, 4/2 x 64; vocabularies 128256, 151936, 49152) or generic ones."""
import math
import random

import torch

own = False

PAGE = 16


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one decode step of 64 sequences: one new row each, a few of them start a page
        dict(name="resize-decode-b64", op="resize", B=64, new=1, ctx=2048, shrink=0, T=64, mix=1),
        # admission and retirement in one step: prompts of very different lengths come in,
        # a third of the sequences give pages back
        dict(name="resize-mixed-b500", op="resize", B=500, new=300, ctx=4096, shrink=1, T=100000, mix=2),
        # one decode step of a batch of 32, 32/8 heads of 128
        dict(name="append-decode-t32", op="append", T=32, pad=0, nq=32, nkv=8, d=128, base=500000.0, ctx=4096,
             norm=0, mix=3),
        # a ragged step of a small model with QK-norm, with rows left over behind the last sequence
        dict(name="append-ragged-t777", op="append", T=777, pad=23, nq=9, nkv=3, d=64, base=10000.0, ctx=100000,
             norm=1, mix=4),
        # a step full of prompt tokens
        dict(name="append-prompt-t8192", op="append", T=8192, pad=0, nq=32, nkv=8, d=128, base=500000.0, ctx=8192,
             norm=0, mix=5),
        # the check of four drafted tokens for one user
        dict(name="chunk-verify-b1", op="chunk", lens="5@4096", nq=32, nkv=8, d=128, window=0, cap=0.0),
        # the same for a batch of 32 at ragged contexts
        dict(name="chunk-verify-b32", op="chunk", lens="r32:5-8@1000-8000/6", nq=32, nkv=8, d=128, window=0, cap=0.0),
        # a continuous batch: decodes at ragged contexts beside three prompt chunks, odd sizes
        dict(name="chunk-mixed-b24", op="chunk", lens="r21:1-1@30-3000/7,511@0,300@1234,77@4001", nq=9, nkv=3, d=64,
             window=0, cap=0.0),
        # a prompt chunk under a sliding window and a score cap, one kv head for each query head
        dict(name="chunk-window-cap", op="chunk", lens="1500@2500", nq=16, nkv=16, d=128, window=1024, cap=50.0),
        # a long prompt in one go
        dict(name="chunk-prompt-8192", op="chunk", lens="8192@0", nq=32, nkv=8, d=128, window=0, cap=0.0),
        # four drafted tokens of one user, the draft model's logits given
        dict(name="verify-b1-v128256", op="verify", B=1, n=4, V=128256, ld=128256, draft=1, greedy=0, mix=8),
        # seven of each of 32 users, some with fewer drafts, some asking for the greedy token
        dict(name="verify-b32-v128256", op="verify", B=32, n=7, V=128256, ld=128256, draft=1, greedy=1, mix=9),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["resize", "append", "chunk", "chunk", "verify"])
    mix = rng.randrange(1 << 30)
    if op == "resize":
        B = _log(rng, 1, 1000)
        new = _log(rng, 1, max(1, min(2000, 100000 // (2 * B))))
        return dict(op=op, B=B, new=new, ctx=_log(rng, 16, 16000), shrink=rng.randrange(2), T=2 * B * new, mix=mix)
    nq, nkv, d = rng.choice([(32, 8, 128), (16, 16, 128), (9, 3, 64), (4, 2, 64), (24, 2, 128), (8, 1, 64)])
    if op == "append":
        T = _log(rng, 1, 8000)
        return dict(op=op, T=T, pad=rng.choice([0, rng.randrange(T)]), nq=nq, nkv=nkv, d=d,
                    base=rng.choice([10000.0, 500000.0]), ctx=_log(rng, 100, 200000), norm=rng.randrange(2), mix=mix)
    if op == "chunk":
        B = _log(rng, 1, 40)
        most = 7000 // B  # rows and contexts that keep a drawn case below the largest listed one
        hi = _log(rng, 1, max(1, most))
        ctx = _log(rng, 1, 8000 if B > 2 or hi < 1000 else 2000)
        lens = "r%d:%d-%d@%d-%d/%d" % (B, max(1, hi // 4), hi, ctx // 8, ctx, mix)
        return dict(op=op, lens=lens, nq=nq, nkv=nkv, d=d, window=rng.choice([0, 0, _log(rng, 1, 5000)]),
                    cap=rng.choice([0.0, 0.0, 50.0, 30.0]))
    V = rng.choice([128256, 151936, 49152, _log(rng, 500, 100000)])
    n = rng.randrange(1, 9)
    B = _log(rng, 1, max(1, min(64, 30000000 // (V * (n + 1)))))
    return dict(op=op, B=B, n=n, V=V, ld=V + rng.choice([0, 0, 1, 64]), draft=rng.randrange(2),
                greedy=rng.randrange(2), mix=mix)


def _rows(spec):
    """[(new rows, rows cached before them)] of "5@4096" or "r32:5-8@1000-8000/6" (32 drawn from
    these ranges, the last number seeds the draw), comma-separated."""
    out = []
    for part in spec.split(","):
        if part[0] != "r":
            n, c = part.split("@")
            out.append((int(n), int(c)))
            continue
        body, seed = part[1:].split("/")
        count, rest = body.split(":")
        ns, cs = rest.split("@")
        r = random.Random(int(seed))
        (n0, n1), (c0, c1) = (tuple(map(int, s.split("-"))) for s in (ns, cs))
        out += [(r.randint(n0, n1), r.randint(c0, c1)) for _ in range(int(count))]
    return out


def _lengths(case):
    """(old, new) lengths of a resize case."""
    r = random.Random(case["mix"])
    old, new, left, back = [], [], case["T"], case["T"]
    for b in range(case["B"]):
        o = r.randint(0, case["ctx"])
        if case["shrink"] and r.random() < 0.34:
            n = o - min(back, r.randint(0, o))
            back -= o - n
        else:
            n = o + min(left, r.randint(1, 2 * case["new"]) if case["new"] > 1 else 1)
            left -= n - o
        old.append(o)
        new.append(n)
    return old, new


def _pages(length):
    return -(-length // PAGE)


# ------------------------------------------------------------------ work

def work(case):
    op = case["op"]
    if op == "resize":
        old, new = _lengths(case)
        rows = sum(max(0, n - o) for o, n in zip(old, new))
        back = sum(max(0, o - n) for o, n in zip(old, new))
        pages = sum(abs(_pages(n) - _pages(o)) for o, n in zip(old, new))
        # there and back: lengths in, row starts out, slots and positions of every new row and
        # of the T buffer behind them out, one table entry and one free-list entry a page moved
        return dict(bytes=2 * (4 * (2 * case["B"] + case["B"] + 1) + 8 * case["T"] + 8 * pages),
                    flops=2 * (rows + back + pages))
    if op == "append":
        heads = case["nq"] + 2 * case["nkv"]
        rows = case["T"] - case["pad"]
        return dict(bytes=rows * heads * case["d"] * (4 + 2) + 8 * case["T"],
                    flops=rows * (case["nq"] + case["nkv"]) * case["d"] * (3 + 4 * case["norm"]))
    if op == "chunk":
        nq, nkv, d, win = case["nq"], case["nkv"], case["d"], case["window"]
        flops = bytes_ = 0
        for n, c in _rows(case["lens"]):
            seen = sum(min(c + i + 1, win) if win else c + i + 1 for i in range(n))
            keys = min(c + n, win + n - 1) if win else c + n
            flops += 4 * d * nq * seen
            bytes_ += 2 * 2 * nq * d * n + 2 * 2 * nkv * d * keys + 4 * _pages(keys) + 8
        return dict(bytes=bytes_, flops=flops)
    B, n, V = case["B"], case["n"], case["V"]
    rows = B * (n + 1) + (B * n if case["draft"] else 0)
    return dict(bytes=4 * rows * V + 4 * B * (3 * n + 6), flops=4 * rows * V)


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    return dict(case=case, **{"resize": _prep_resize, "append": _prep_append, "chunk": _prep_chunk,
                              "verify": _prep_verify}[case["op"]](case, _gen(seed)))


def _prep_resize(case, g):
    """Sequences of a running server: their pages drawn from a shuffled pool, the rest free."""
    old, new = _lengths(case)
    B = case["B"]
    mp = _pages(max(max(old), max(new))) + 3
    held = [_pages(o) for o in old]
    n_pages = max(sum(max(_pages(o), _pages(n)) for o, n in zip(old, new)), 1) + 5
    perm = torch.randperm(n_pages, device="cuda", generator=g).int()
    table = torch.full((B, mp), -1, dtype=torch.int32, device="cuda")
    held_t = _ints(held).long()
    at = torch.arange(mp, device="cuda")[None, :]
    first = (held_t.cumsum(0) - held_t)[:, None]
    inside = at < held_t[:, None]
    table[inside] = perm[(first + at)[inside]]
    free = torch.full((n_pages,), -1, dtype=torch.int32, device="cuda")
    n_free = n_pages - sum(held)
    free[:n_free] = perm[sum(held):]
    T = case["T"]
    out = lambda n: torch.empty(n, dtype=torch.int32, device="cuda")  # noqa: E731
    return dict(old=_ints(old), new=_ints(new), table=table, free=free, n_free=_ints([n_free]), T=T,
                cu=out(B + 1), slot=out(T), pos=out(T), status=out(1), cu2=out(B + 1), slot2=out(T), pos2=out(T),
                status2=out(1))


def _slots(rows, n_pages, g):
    """A shuffled pool's block table for sequences of the given total lengths."""
    held = [_pages(r) for r in rows]
    mp = max(max(held), 1)
    perm = torch.randperm(n_pages, device="cuda", generator=g).int()
    table = torch.full((len(rows), mp), -1, dtype=torch.int32, device="cuda")
    held_t = _ints(held).long()
    at = torch.arange(mp, device="cuda")[None, :]
    inside = at < held_t[:, None]
    table[inside] = perm[((held_t.cumsum(0) - held_t)[:, None] + at)[inside]]
    return table


def _prep_append(case, g):
    """The QKV projection's fp32 rows of a step: rows of several sequences, each at its own
    position, to distinct slots of the pool; the last `pad` rows belong to nobody."""
    T, nq, nkv, d = case["T"], case["nq"], case["nkv"], case["d"]
    n_pages = _pages(T) + 9
    qkv = torch.randn((T, (nq + 2 * nkv) * d), device="cuda", generator=g)
    slot = torch.randperm(n_pages * PAGE, device="cuda", generator=g)[:T].int()
    pos = torch.randint(0, case["ctx"], (T,), device="cuda", generator=g).int()
    if case["pad"]:
        slot[T - case["pad"]:] = -1
        pos[T - case["pad"]:] = -1
    norm = lambda: 1 + 0.1 * torch.randn(d, device="cuda", generator=g) if case["norm"] else None  # noqa: E731
    pool = lambda: torch.randn((n_pages, nkv, PAGE, d), device="cuda", generator=g).bfloat16()  # noqa: E731
    return dict(qkv=qkv, slot=slot, pos=pos, q_norm=norm(), k_norm=norm(), k_pool=pool(), v_pool=pool(),
                q_out=torch.zeros((T, nq, d), dtype=torch.bfloat16, device="cuda"))


def _prep_chunk(case, g):
    rows = _rows(case["lens"])
    nq, nkv, d = case["nq"], case["nkv"], case["d"]
    T = sum(n for n, _ in rows)
    n_pages = sum(_pages(n + c) for n, c in rows) + 2
    table = _slots([n + c for n, c in rows], n_pages, g)
    pool = lambda: torch.randn((n_pages, nkv, PAGE, d), device="cuda", generator=g).bfloat16()  # noqa: E731
    cu = [0]
    for n, _ in rows:
        cu.append(cu[-1] + n)
    return dict(q=torch.randn((T, nq, d), device="cuda", generator=g).bfloat16(), k_pool=pool(), v_pool=pool(),
                table=table, cu=_ints(cu), kv_len=_ints([n + c for n, c in rows]), rows=rows,
                scale=1 / math.sqrt(d), out=torch.empty((T, nq, d), dtype=torch.bfloat16, device="cuda"))


def _prep_verify(case, g):
    """Logits of a target and a draft model that mostly agree, drafts drawn from the draft
    model's distribution, so that most drafts are accepted and some are not."""
    B, n, V, ld = case["B"], case["n"], case["V"], case["ld"]
    r = random.Random(case["mix"])
    full = torch.randn((B, n + 1, ld), device="cuda", generator=g).mul_(2.5)
    draft = (full[:, :n] + 0.5 * torch.randn((B, n, ld), device="cuda", generator=g))
    temp = [0.0 if case["greedy"] and r.random() < 0.3 else r.uniform(0.5, 1.3) for _ in range(B)]
    temp_t = torch.tensor(temp, device="cuda")
    count = [n if r.random() < 0.7 else r.randint(0, n) for _ in range(B)]
    t = torch.where(temp_t > 0, temp_t, torch.ones_like(temp_t))[:, None, None]
    noise = -torch.log(-torch.log(torch.rand((B, n, V), device="cuda", generator=g).clamp_(1e-30, 1 - 1e-7)))
    drawn = (draft[:, :, :V] / t + noise).argmax(-1)
    tok = torch.where(temp_t[:, None] > 0, drawn, draft[:, :, :V].argmax(-1))
    del noise
    out = lambda *s: torch.empty(s, dtype=torch.int32, device="cuda")  # noqa: E731
    return dict(target=full[:, :, :V], draft=draft[:, :, :V] if case["draft"] else None, tok=tok.int().contiguous(),
                count=_ints(count), temp=temp_t, u=torch.rand((B, n), device="cuda", generator=g),
                us=torch.rand((B,), device="cuda", generator=g), accepted=out(B), tokens=out(B, n + 1))


# ------------------------------------------------------------------ one pass

def run(state):
    op = state["case"]["op"]
    if own:
        return {"resize": _own_resize, "append": _own_append, "chunk": _own_chunk, "verify": _own_verify}[op](state)
    return {"resize": _plain_resize, "append": _plain_append, "chunk": _plain_chunk, "verify": _plain_verify}[op](state)


def _own_resize(s):
    import decoder_only_transformer_layer_b200 as dec
    dec.paged_resize(s["old"], s["new"], s["table"], s["free"], s["n_free"], s["cu"], s["slot"], s["pos"], s["status"])
    # and back, as after a step whose rows are all rejected: the pages return in their old order
    dec.paged_resize(s["new"], s["old"], s["table"], s["free"], s["n_free"], s["cu2"], s["slot2"], s["pos2"],
                     s["status2"])
    return {k: s[k] for k in ("table", "free", "n_free", "cu", "slot", "pos", "status", "cu2", "slot2", "pos2",
                              "status2")}


def _own_append(s):
    import decoder_only_transformer_layer_b200 as dec
    c = s["case"]
    dec.paged_rope_append(s["qkv"], s["slot"], s["pos"], s["q_out"], s["k_pool"], s["v_pool"], c["base"],
                          q_norm=s["q_norm"], k_norm=s["k_norm"], eps=1e-6)
    return {k: s[k] for k in ("q_out", "k_pool", "v_pool")}


def _own_chunk(s):
    import decoder_only_transformer_layer_b200 as dec
    c = s["case"]
    return dec.gqa_chunk_attn(s["q"], s["k_pool"], s["v_pool"], s["table"], s["cu"], s["kv_len"], s["scale"], s["out"],
                              window=c["window"], softcap=c["cap"])


def _own_verify(s):
    import decoder_only_transformer_layer_b200 as dec
    dec.spec_verify(s["target"], s["draft"], s["tok"], s["count"], s["temp"], s["u"], s["us"], s["accepted"],
                    s["tokens"])
    return {"accepted": s["accepted"], "tokens": s["tokens"]}


# ------------------------------------------------------------------ plain forms

def _resize_once(old, new, table, free, n_free, T):
    """One resize in torch operations; the cases never fail, so there is no failure path here."""
    B, mp = table.shape
    P = free.numel()
    old, new, F = old.long(), new.long(), n_free.long()
    held, want = (old + PAGE - 1) // PAGE, (new + PAGE - 1) // PAGE
    take, give = (want - held).clamp(min=0), (held - want).clamp(min=0)
    rows = (new - old).clamp(min=0)
    cu = torch.cat([rows.new_zeros(1), rows.cumsum(0)])
    i = torch.arange(P, device=table.device)
    spare = B * mp  # a place for what is not written
    flat = torch.cat([table.reshape(-1), table.new_zeros(1)])
    stack = torch.cat([free, free.new_zeros(1)])
    # pages taken: the i-th of all, in the order of sequences and of their pages, is free[F - 1 - i]
    end = take.cumsum(0)
    b = torch.searchsorted(end, i, right=True).clamp(max=B - 1)
    ok = i < end[-1]
    where = torch.where(ok, b * mp + held[b] + i - (end[b] - take[b]), spare)
    got = stack[torch.where(ok, F - 1 - i, P)]
    # pages given back: the k-th of all goes to free[F - taken + given - 1 - k]
    gend = give.cumsum(0)
    gb = torch.searchsorted(gend, i, right=True).clamp(max=B - 1)
    gok = i < gend[-1]
    gwhere = torch.where(gok, gb * mp + want[gb] + i - (gend[gb] - give[gb]), spare)
    page = flat[gwhere]
    flat[where] = got
    flat[gwhere] = -1
    stack[torch.where(gok, F - end[-1] + gend[-1] - 1 - i, P)] = page
    table.copy_(flat[:-1].view(B, mp))
    free.copy_(stack[:-1])
    n_free.copy_(F - end[-1] + gend[-1])
    # the new rows' slots and positions
    t = torch.arange(T, device=table.device)
    rb = torch.searchsorted(cu[1:], t, right=True).clamp(max=B - 1)
    p = old[rb] + t - cu[rb]
    ok = t < cu[-1]
    pg = table.long()[rb, torch.where(ok, p // PAGE, 0)]
    slot = torch.where(ok, pg * PAGE + p % PAGE, -1)
    return cu.int(), slot.int(), torch.where(ok, p, -1).int(), torch.zeros(1, dtype=torch.int32, device=table.device)


def _plain_resize(s):
    cu, slot, pos, status = _resize_once(s["old"], s["new"], s["table"], s["free"], s["n_free"], s["T"])
    cu2, slot2, pos2, status2 = _resize_once(s["new"], s["old"], s["table"], s["free"], s["n_free"], s["T"])
    return dict(table=s["table"], free=s["free"], n_free=s["n_free"], cu=cu, slot=slot, pos=pos, status=status,
                cu2=cu2, slot2=slot2, pos2=pos2, status2=status2)


def _plain_append(s):
    c = s["case"]
    T, nq, nkv, d = c["T"], c["nq"], c["nkv"], c["d"]
    x = s["qkv"].view(T, nq + 2 * nkv, d)
    q, k, v = x[:, :nq], x[:, nq:nq + nkv], x[:, nq + nkv:]
    if c["norm"]:
        q = q * torch.rsqrt(q.square().mean(-1, keepdim=True) + 1e-6) * s["q_norm"]
        k = k * torch.rsqrt(k.square().mean(-1, keepdim=True) + 1e-6) * s["k_norm"]
    inv = c["base"] ** (-2.0 * torch.arange(d // 2, device=x.device, dtype=torch.float64) / d)
    a = s["pos"].double()[:, None] * inv
    cos, sin = torch.cos(a).float()[:, None], torch.sin(a).float()[:, None]
    h = d // 2
    turn = lambda y: torch.cat([y[..., :h] * cos - y[..., h:] * sin, y[..., h:] * cos + y[..., :h] * sin], -1)  # noqa: E731
    live = (s["slot"] >= 0)
    s["q_out"].copy_(torch.where(live[:, None, None], turn(q).bfloat16(), s["q_out"]))
    # a row that belongs to nobody repeats row 0's store
    row = torch.where(live, torch.arange(T, device=x.device), 0)
    at = s["slot"][row].long()
    s["k_pool"][at // PAGE, :, at % PAGE] = turn(k).bfloat16()[row]
    s["v_pool"][at // PAGE, :, at % PAGE] = v.bfloat16()[row]
    return dict(q_out=s["q_out"], k_pool=s["k_pool"], v_pool=s["v_pool"])


def _plain_chunk(s):
    c = s["case"]
    nq, nkv, d = c["nq"], c["nkv"], c["d"]
    out, at = s["out"], 0
    for b, (n, cached) in enumerate(s["rows"]):
        L = n + cached
        pages = s["table"][b, :_pages(L)].long()
        K = s["k_pool"][pages].transpose(1, 2).reshape(-1, nkv, d)[:L].float()
        V = s["v_pool"][pages].transpose(1, 2).reshape(-1, nkv, d)[:L].float()
        q = s["q"][at:at + n].float().view(n, nkv, nq // nkv, d).permute(1, 2, 0, 3).reshape(nkv, -1, d)
        S = torch.matmul(q, K.permute(1, 2, 0)).mul_(s["scale"])  # [nkv][G n][L]
        if c["cap"] > 0:
            S.div_(c["cap"]).tanh_().mul_(c["cap"])
        p = torch.arange(cached, L, device=q.device)[:, None]
        j = torch.arange(L, device=q.device)[None, :]
        hide = (j > p) | (j <= p - c["window"]) if c["window"] else j > p
        S.view(nkv, -1, n, L).masked_fill_(hide, -math.inf)
        S.sub_(S.amax(-1, keepdim=True)).exp_()
        O = torch.matmul(S, V.transpose(0, 1)) / S.sum(-1, keepdim=True)
        out[at:at + n] = O.view(nkv, -1, n, d).permute(2, 0, 1, 3).reshape(n, nq, d).bfloat16()
        at += n
    return out


def _plain_verify(s):
    target, draft, tok, count = s["target"], s["draft"], s["tok"].long(), s["count"].long()
    B, n1, V = target.shape
    n = n1 - 1
    warm = s["temp"] > 0
    t = torch.where(warm, s["temp"], torch.ones_like(s["temp"])).double()[:, None, None]
    # probabilities in 64 bits: a sampled token lies next to the borders of the cumulative sums
    p = torch.softmax(target.double() / t, -1)
    if draft is None:
        q = torch.zeros_like(p[:, :n]).scatter_(2, tok[:, :, None], 1.0)
    else:
        q = torch.softmax(draft.double() / t, -1)
    best = target.argmax(-1)
    at = lambda x: x.gather(2, tok[:, :, None])[:, :, 0]  # noqa: E731
    take = torch.where(warm[:, None], s["u"].double() * at(q) < at(p[:, :n]), tok == best[:, :n])
    i = torch.arange(n, device=tok.device)[None, :]
    take = (take & (i < count[:, None])).long().cumprod(1)
    acc = take.sum(1)
    rows = torch.arange(B, device=tok.device)
    pr = p[rows, acc]
    qr = torch.where((acc < count)[:, None], q[rows, acc.clamp(max=n - 1)], 0.0)
    w = (pr - qr).clamp(min=0)
    w = torch.where(w.sum(-1, keepdim=True) > 0, w, pr)
    C = w.cumsum(-1)
    hit = (C > s["us"].double()[:, None] * C[:, -1:]) & (w > 0)
    last = V - 1 - (w > 0).flip(-1).int().argmax(-1)
    pick = torch.where(hit.any(-1), hit.int().argmax(-1), last)
    pick = torch.where(warm, pick, best[rows, acc])
    col = torch.arange(n1, device=tok.device)[None, :]
    padded = torch.cat([tok, tok.new_zeros(B, 1)], 1)
    tokens = torch.where(col < acc[:, None], padded, torch.where(col == acc[:, None], pick[:, None], -1))
    return dict(accepted=acc.int(), tokens=tokens.int())


# ------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    if case["op"] == "append":
        return _exact_append(case, prepare(case, seed))
    if case["op"] == "chunk":
        return _exact_chunk(case, prepare(case, seed))
    return None  # whole numbers


def _exact_append(case, s):
    nq, nkv, d = case["nq"], case["nkv"], case["d"]
    keep = torch.nonzero(s["slot"] >= 0)[:, 0]
    heads = s["qkv"].double()[keep].unflatten(1, (-1, d))
    z = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                    s["pos"][keep].double()[:, None]
                    * torch.exp(-math.log(case["base"]) * torch.arange(0, d, 2, device="cuda").double() / d))

    def rotated(x, gain):
        if gain is not None:
            x = x / torch.sqrt((x * x).mean(2, keepdim=True) + 1e-6) * gain.double()
        y = torch.complex(x[..., : d // 2].contiguous(), x[..., d // 2:].contiguous()) * z[:, None]
        return torch.cat([y.real, y.imag], 2)

    out = {k: s[k].double() for k in ("q_out", "k_pool", "v_pool")}
    out["q_out"][keep] = rotated(heads[:, :nq], s["q_norm"])
    page, off = s["slot"][keep].long().div(PAGE, rounding_mode="floor"), s["slot"][keep].long().remainder(PAGE)
    out["k_pool"][page, :, off] = rotated(heads[:, nq:nq + nkv], s["k_norm"])
    out["v_pool"][page, :, off] = heads[:, nq + nkv:]
    return out


def _exact_chunk(case, s):
    nq, nkv, d = case["nq"], case["nkv"], case["d"]
    G = nq // nkv
    cu, table = s["cu"].tolist(), s["table"].long()
    out = torch.zeros((cu[-1], nq, d), dtype=torch.float64, device="cuda")
    for b, (n, cached) in enumerate(s["rows"]):
        idx = torch.arange(n + cached, device="cuda")
        page, off = table[b][idx // PAGE], idx % PAGE
        p = idx[cached:]
        seen = idx[None] <= p[:, None]
        if case["window"]:
            seen &= idx[None] > p[:, None] - case["window"]
        for h in range(nq):
            K, V = s["k_pool"][page, h // G, off].double(), s["v_pool"][page, h // G, off].double()
            for r in range(0, n, 1024):  # a block of rows at a time
                e = (s["q"][cu[b] + r:cu[b] + min(n, r + 1024), h].double() @ K.T) * s["scale"]
                if case["cap"] > 0:
                    e = case["cap"] * torch.tanh(e / case["cap"])
                e = torch.where(seen[r:r + 1024], e, torch.full_like(e, -math.inf))
                out[cu[b] + r:cu[b] + min(n, r + 1024), h] = torch.softmax(e, 1) @ V
    return out
