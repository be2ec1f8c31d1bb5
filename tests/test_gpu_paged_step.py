"""The paged step's operators against their plain 64-bit forms: paged_resize, paged_rope_append,
gqa_chunk_attn, spec_verify, and a step of all four."""
import math

import numpy as np
import pytest
import torch

import _paged_plain as plain
import decoder_only_transformer_layer_b200 as dec

pytestmark = pytest.mark.gpu

I32 = dict(dtype=torch.int32, device="cuda")


def ints(v):
    return torch.tensor(np.ascontiguousarray(v, dtype=np.int32), device="cuda")


def f64(t):
    return t.double().cpu().numpy()


# ------------------------------------------------------------------ paged_resize

def pool_state(old, mp, n_pages, seed):
    rng = np.random.default_rng(seed)
    perm = rng.permutation(n_pages)
    table = np.full((len(old), mp), -1)
    at = 0
    for b, o in enumerate(old):
        k = plain.pages(o)
        table[b, :k] = perm[at:at + k]
        at += k
    free = np.full(n_pages, -1)
    free[:n_pages - at] = perm[at:]
    return table, free, n_pages - at


def run_resize(old, new, table, free, n_free, T):
    B = len(old)
    out = dict(table=ints(table), free=ints(free), n_free=ints([n_free]), cu=torch.full((B + 1,), 77, **I32),
               slot=torch.full((T,), 77, **I32), pos=torch.full((T,), 77, **I32), status=torch.full((1,), 77, **I32))
    dec.paged_resize(ints(old), ints(new), out["table"], out["free"], out["n_free"], out["cu"], out["slot"],
                     out["pos"], out["status"])
    torch.cuda.synchronize()
    return {k: v.cpu().numpy() for k, v in out.items()}


def check_resize(old, new, table, free, n_free, T):
    got = run_resize(old, new, table, free, n_free, T)
    s, cu, slot, pos, t2, f2, n2 = plain.resize(old, new, table, free, n_free, T, len(free))
    assert got["status"][0] == s
    for k, v in dict(cu=cu, slot=slot, pos=pos, table=t2, free=f2, n_free=[n2]).items():
        assert np.array_equal(got[k], v), k
    return got


@pytest.mark.parametrize("B,hi,T_extra,seed", [(1, 1, 0, 0), (1, 40, 5, 1), (7, 100, 0, 2), (33, 300, 100, 3),
                                               (1000, 60, 9, 4), (1025, 33, 0, 5), (4096, 20, 1, 6), (50, 3000, 7, 7)])
def test_resize_random(B, hi, T_extra, seed):
    rng = np.random.default_rng(seed)
    old = rng.integers(0, hi + 1, B)
    new = np.where(rng.random(B) < 0.2, old, rng.integers(0, hi + 1, B))
    mp = plain.pages(hi) + 1
    n_pages = sum(plain.pages(o) + plain.pages(n) for o, n in zip(old, new)) + 1
    table, free, n_free = pool_state(old, mp, n_pages, seed)
    T = int(np.maximum(new - old, 0).sum()) + T_extra
    got = check_resize(old, new, table, free, n_free, T)
    # and back: table and free list as before
    back = run_resize(new, old, got["table"], got["free"], int(got["n_free"][0]), int(np.maximum(old - new, 0).sum()))
    assert back["status"][0] == 0 and back["n_free"][0] == n_free
    assert np.array_equal(back["table"], table) and np.array_equal(back["free"][:n_free], free[:n_free])


def test_resize_page_borders_and_no_rows():
    for o in (0, 1, 15, 16, 17, 31, 32):
        for n in (0, 1, 15, 16, 17, 31, 32):
            old, new = np.array([o, 5]), np.array([n, 5])
            check_resize(old, new, *pool_state(old, 3, 9, o * 40 + n), max(0, n - o))


def test_resize_failures_change_nothing():
    old, new = np.array([20, 40]), np.array([50, 10])
    table, free, n_free = pool_state(old, 4, 12, 1)
    assert check_resize(old, new, table, free, n_free, 29)["status"][0] == 1      # one row too many for T
    assert check_resize(np.array([-1, 40]), new, table, free, n_free, 60)["status"][0] == 1
    assert check_resize(old, np.array([50, -3]), table, free, n_free, 60)["status"][0] == 1
    assert check_resize(old, np.array([65, 10]), table, free, n_free, 60)["status"][0] == 2
    assert check_resize(old, new, table, free, 1, 60)["status"][0] == 3           # two pages wanted, one free
    assert check_resize(old, new, table, free, 13, 60)["status"][0] == 1          # more free than there are
    assert check_resize(old, new, table, free, -1, 60)["status"][0] == 1
    assert check_resize(old, np.array([0, 0]), table, free, 9, 60)["status"][0] == 1  # the list overflows
    for bad_page in (-1, 12, 1 << 30):
        t = table.copy()
        t[1, 1] = bad_page                                                        # given back
        assert check_resize(old, new, t, free, n_free, 60)["status"][0] == 1
        f = free.copy()
        f[n_free - 2] = bad_page                                                  # taken
        assert check_resize(old, new, table, f, n_free, 60)["status"][0] == 1
        t = table.copy()
        t[0, 1] = bad_page                                                        # kept: its rows have no slot
        got = check_resize(old, new, t, free, n_free, 60)
        assert got["status"][0] == 0 and (got["slot"][:12] == -1).all() and (got["pos"][:12] >= 20).all()


def test_resize_many_rows_and_large_tables():
    # one long prompt beside many short ones, over more than one thread block a cluster
    old = np.array([0] + [3] * 600)
    new = np.array([60000] + [5] * 600)
    check_resize(old, new, *pool_state(old, 3750, 4800, 3), 60000 + 1200 + 17)


@pytest.mark.parametrize("T", [4095, 4096, 4097, 5000])
def test_resize_row_counts_around_the_two_ways_of_placing_them(T):
    old, new = np.array([7, 30, 0]), np.array([7 + 100, 12, T - 100])
    check_resize(old, new, *pool_state(old, 330, 400, T), T)          # exactly full
    check_resize(old, new, *pool_state(old, 330, 400, T), T + 1000)   # rows left over
    check_resize(old, new, *pool_state(old, 330, 400, T), T - 1)      # one too many: refused
    table, free, n_free = pool_state(old, 330, 400, T)
    table[0, 0] = 400                                                 # a kept page outside the pool
    check_resize(old, new, table, free, n_free, T)


# ------------------------------------------------------------------ paged_rope_append

@pytest.mark.parametrize("T,nq,nkv,d,norms,far,pad", [
    (1, 4, 2, 64, 0, 10, 0), (5, 32, 8, 128, 0, 4096, 0), (37, 9, 3, 64, 3, 1000000, 4), (64, 16, 16, 128, 1, 300, 0),
    (3, 8, 1, 128, 2, 2 ** 31 - 1, 1), (700, 4, 4, 64, 3, 5000, 0), (2000, 5, 1, 128, 3, 100, 13)])
def test_rope_append(T, nq, nkv, d, norms, far, pad):
    rng = np.random.default_rng(T)
    n_pages = plain.pages(T) + 3
    width = (nq + 2 * nkv) * d
    base = 500000.0 if far > 4096 else 10000.0
    big = torch.tensor(rng.normal(size=(T, width + 24)), dtype=torch.float32, device="cuda")
    qkv = big[:, 8:8 + width]  # rows with a stride
    slot = rng.permutation(n_pages * 16)[:T]
    pos = rng.integers(0, far, T)
    pos[0] = far - 1
    gone = rng.permutation(T)[:pad]
    slot[gone] = rng.choice([-1, -7, n_pages * 16, 2 ** 31 - 1], pad)
    g = [torch.tensor(1 + 0.3 * rng.normal(size=d), dtype=torch.float32, device="cuda") if norms & k else None
         for k in (1, 2)]
    pools = [torch.tensor(rng.normal(size=(n_pages, nkv, 16, d)), device="cuda").bfloat16() for _ in range(2)]
    q_out = torch.tensor(rng.normal(size=(T, nq, d)), device="cuda").bfloat16()
    want = [f64(q_out)] + [f64(p) for p in pools]
    tol = [np.zeros(w.shape) for w in want]
    x = f64(qkv).reshape(T, nq + 2 * nkv, d)
    gn = [None if y is None else f64(y) for y in g]
    eps = float(np.float32(1e-6))
    for t in range(T):
        if not 0 <= slot[t] < n_pages * 16:
            continue
        pg, off = divmod(int(slot[t]), 16)
        q, k = plain.head_norm(x[t, :nq], gn[0], eps), plain.head_norm(x[t, nq:nq + nkv], gn[1], eps)
        for w, tl, at, y, z in ((want[0], tol[0], (t,), plain.rope(q, pos[t], base), q),
                                (want[1], tol[1], (pg, slice(None), off), plain.rope(k, pos[t], base), k),
                                (want[2], tol[2], (pg, slice(None), off), x[t, nq + nkv:], None)):
            w[at] = y
            # half a bf16 step; the fp32 products and their sum (2^-24 each), the rounded cosine and
            # sine (2^-24 each, 2^-22 of their evaluation) and the norm's factor (2^-21), all relative
            # to the pair's length, which is at most the sum of its two values
            pair = 0 if z is None else np.tile(np.abs(z[..., :d // 2]) + np.abs(z[..., d // 2:]), 2)
            tl[at] = np.abs(y) * 2.0 ** -8 + pair * 2.0 ** -20
    dec.paged_rope_append(qkv, ints(slot), ints(pos), q_out, pools[0], pools[1], base, q_norm=g[0], k_norm=g[1])
    torch.cuda.synchronize()
    for name, got, w, tl in zip("qkv", [q_out] + pools, want, tol):
        err = np.abs(f64(got) - w)
        assert (err <= tl).all(), f"{name}: {np.max(err - tl):.3e} above"  # 0 where nothing is written


# ------------------------------------------------------------------ gqa_chunk_attn

def chunk_inputs(rows, nq, nkv, d, seed, extra_rows=0, holes=False):
    """rows: [(n, kv_len)]; returns device tensors of a shuffled pool whose unused places hold NaN."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rng = np.random.default_rng(seed)
    held = [plain.pages(max(L, 0)) for _, L in rows]
    n_pages = sum(held) + 3
    mp = max(held + [1]) + 1
    perm = rng.permutation(n_pages)
    table = np.full((len(rows), mp), -1)
    at = 0
    kp, vp = (torch.full((n_pages, nkv, 16, d), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for b, (n, L) in enumerate(rows):
        table[b, :held[b]] = perm[at:at + held[b]]
        at += held[b]
        for j in range(held[b]):
            r = min(16, L - 16 * j)
            for p in (kp, vp):
                p[table[b, j], :, :r] = torch.randn((nkv, r, d), device="cuda", generator=g).bfloat16()
    T = sum(n for n, _ in rows) + extra_rows
    q = torch.randn((T, nq, d), device="cuda", generator=g).bfloat16()
    cu = np.concatenate([[0], np.cumsum([n for n, _ in rows])])
    return q, kp, vp, table, cu, np.array([L for _, L in rows])


def check_chunk(inp, scale=None, window=0, cap=0.0, q_view=None, workspace=None, on_device=False):
    q, kp, vp, table, cu, lens = inp
    T, nq, d = q.shape
    scale = float(np.float32(scale or 1 / math.sqrt(d)))
    start = torch.full((T, nq, d), 3.0, dtype=torch.bfloat16, device="cuda")
    out = start.clone()
    dec.gqa_chunk_attn(q if q_view is None else q_view, kp, vp, ints(table), ints(cu), ints(lens), scale, out,
                       window=window, softcap=cap, workspace=workspace)
    dec.check_standalone()
    if on_device:
        want, mag = plain.chunk_attn_on_device(q, torch.nan_to_num(kp), torch.nan_to_num(vp), table, cu, lens, scale,
                                               window, float(np.float32(cap)))
    else:
        want, mag = plain.chunk_attn(f64(q), f64(kp), f64(vp), table, cu, lens, scale, window, float(np.float32(cap)),
                                     f64(start))
    got = f64(out)
    # the unused places of the pool hold NaN; a row is NaN only where it attends one of them
    assert np.array_equal(np.isnan(got), np.isnan(want))
    got, want, mag = (np.nan_to_num(x, nan=0.0) for x in (got, want, mag))
    # half a bf16 step of the result; each weight rounded to bf16 (half a step, 2^-8 relative) and
    # off by its score's error (fp32 sums of d products: below 2^-11 for these inputs)
    tol = np.abs(want) * 2.0 ** -8 + mag * (2.0 ** -8 + 2.0 ** -11) + 1e-30
    bad = np.abs(got - want) > tol
    assert not bad.any(), f"{bad.sum()} of {bad.size} off, worst {np.max(np.abs(got - want) - tol):.3e}"
    assert np.array_equal(got[cu[-1]:], f64(start)[cu[-1]:])  # rows of nobody
    return out


@pytest.mark.parametrize("nq,nkv,d", [(32, 8, 128), (16, 16, 128), (9, 3, 64), (4, 2, 64), (16, 1, 128), (24, 2, 64),
                                      (5, 1, 128), (7, 1, 64), (22, 2, 128), (26, 2, 64)])
def test_chunk_heads(nq, nkv, d):
    check_chunk(chunk_inputs([(1, 1), (5, 300), (70, 70), (33, 140), (1, 129)], nq, nkv, d, nq * d))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rows", [
    [(1, 1)], [(1, 16)], [(1, 17)], [(1, 127)], [(1, 128)], [(1, 129)], [(2, 2)], [(3, 1000)], [(128, 128)],
    [(129, 129)], [(64, 64)], [(65, 200)], [(257, 300)], [(1, 2500)], [(8, 2111)]], ids=str)
def test_chunk_lengths(rows, d):
    check_chunk(chunk_inputs(rows, 8, 2, d, sum(map(sum, rows))))


def test_chunk_empty_and_short_sequences():
    # no new rows, no cache, fewer cache rows than new ones (the first rows see nothing), rows behind the last
    check_chunk(chunk_inputs([(0, 0), (0, 50), (3, 0), (4, 2), (1, 20), (0, 0), (200, 130), (2, 2)], 8, 2, 128, 1,
                             extra_rows=9))
    check_chunk(chunk_inputs([(0, 0)], 4, 2, 64, 2, extra_rows=3))
    check_chunk(chunk_inputs([(5, 0)], 4, 2, 64, 2))


@pytest.mark.parametrize("window", [1, 2, 15, 16, 100, 128, 129, 300, 100000])
@pytest.mark.parametrize("cap", [0.0, 30.0])
def test_chunk_window_and_cap(window, cap):
    check_chunk(chunk_inputs([(150, 420), (1, 333), (7, 7), (2, 1)], 8, 2, 128, window), window=window, cap=cap,
                scale=0.3)
    check_chunk(chunk_inputs([(90, 200), (1, 150)], 3, 1, 64, window), window=window, cap=cap, scale=0.3)


def test_chunk_many_sequences():
    rng = np.random.default_rng(8)
    check_chunk(chunk_inputs([(int(rng.integers(0, 4)), int(rng.integers(3, 90))) for _ in range(700)], 4, 2, 64, 8))


def test_chunk_mixed_prompts_and_decodes():
    check_chunk(chunk_inputs([(1, 700), (300, 300), (1, 5), (130, 900), (1, 2048), (8, 1500)], 8, 2, 128, 9))


@pytest.mark.parametrize("rows,nq,nkv,d,window,cap", [
    ([(1, 3000 + 37 * i) for i in range(30)], 32, 8, 128, 0, 0.0),             # many blocks and several tiles a run
    ([(1 + i % 9, 2000 + 101 * i) for i in range(40)], 32, 8, 128, 0, 0.0),
    ([(1, 128 * (1 + i)) for i in range(40)], 16, 16, 128, 0, 0.0),            # lengths at block borders
    ([(2500, 4100)], 32, 8, 128, 0, 0.0),                                      # many tiles a run
    ([(3000, 3000), (1, 9000), (700, 2000)], 16, 16, 128, 0, 0.0),
    ([(1500, 2500), (1, 3000), (1100, 1100)], 16, 16, 128, 1024, 50.0),
    ([(2000, 2600), (5, 5000)] + [(1, 777)] * 30, 9, 3, 64, 0, 0.0),
    ([(2000, 2600), (5, 5000)] + [(1, 777)] * 30, 9, 3, 64, 130, 0.0),
    ([(900, 5000)], 24, 2, 128, 0, 100.0),
    ([(1, 20000), (16, 9000)], 16, 1, 128, 0, 0.0)],
    ids=lambda v: f"{len(v)}seqs" if isinstance(v, list) else str(v))
def test_chunk_long(rows, nq, nkv, d, window, cap):
    check_chunk(chunk_inputs(rows, nq, nkv, d, len(rows) + nq), window=window, cap=cap, on_device=True)


def test_chunk_strided_q_rows():
    q, kp, vp, table, cu, lens = inp = chunk_inputs([(40, 100), (3, 50)], 8, 2, 128, 10)
    wide = torch.full((q.shape[0], 12 * 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 256:256 + 1024] = q.reshape(q.shape[0], -1)
    view = wide[:, 256:256 + 1024].unflatten(1, (8, 128))
    assert torch.equal(check_chunk(inp, q_view=view), check_chunk(inp))


def test_chunk_bad_pages_are_not_attended():
    inp = chunk_inputs([(20, 200), (1, 170), (3, 60)], 8, 2, 128, 11)
    table = inp[3]
    table[0, 3], table[1, 0], table[1, 10], table[2, :4] = -1, 1 << 30, inp[1].shape[0], -5
    check_chunk(inp)
    check_chunk(inp, window=40)


def test_chunk_lengths_beyond_the_table_count_as_the_table():
    q, kp, vp, table, cu, lens = chunk_inputs([(30, 100), (1, 64), (5, 200)], 8, 2, 128, 17)
    for extra in (1, 5000, 2 ** 31 - 1 - 16 * table.shape[1]):
        check_chunk((q, kp, vp, table, cu, np.array([100, 16 * table.shape[1] + extra, 200])))
        check_chunk((q, kp, vp, table, cu, np.array([100, 64, 16 * table.shape[1] + extra])), window=150)


def test_chunk_row_starts_out_of_order_stay_in_the_buffer():
    # the call promises nothing for such starts but that it keeps to its buffers
    q, kp, vp, table, cu, lens = chunk_inputs([(30, 100), (1, 64), (5, 200)], 8, 2, 128, 18)
    guard = torch.full((3 * q.shape[0], 8, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    out = guard[q.shape[0]:2 * q.shape[0]]
    for starts in ([0, 40, 20, 36], [-5, 10, 2 ** 30, 36], [36, 0, 0, 36], [-2 ** 31, 2 ** 31 - 1, 5, 7]):
        dec.gqa_chunk_attn(q, kp, vp, ints(table), ints(starts), ints(lens), 0.1, out)
        dec.check_standalone()
        assert (guard[:q.shape[0]] == 3.0).all() and (guard[2 * q.shape[0]:] == 3.0).all()


def test_explicit_streams_and_workspaces():
    q, kp, vp, table, cu, lens = inp = chunk_inputs([(30, 300), (1, 640)], 8, 2, 128, 19)
    want = check_chunk(inp)
    out = torch.zeros_like(q)
    side = torch.cuda.Stream()
    args = (q, kp, vp, ints(table), ints(cu), ints(lens), 128 ** -0.5, out)
    torch.cuda.synchronize()
    with pytest.raises(ValueError):
        dec.gqa_chunk_attn(*args, stream=side.cuda_stream)  # whose memory would that be?
    ws = torch.empty(dec.lib().gqa_chunk_attn_workspace(128), dtype=torch.uint8, device="cuda")
    dec.gqa_chunk_attn(*args, stream=side.cuda_stream, workspace=ws)
    side.synchronize()
    assert torch.equal(out, want)
    with pytest.raises(dec.DecError):
        dec.gqa_chunk_attn(*args, workspace=ws[:-16])
    with pytest.raises(dec.DecError):
        dec.gqa_chunk_attn(*args, workspace=torch.empty(ws.numel() + 8, dtype=torch.uint8, device="cuda")[8:])
    with pytest.raises(ValueError):
        dec.gqa_chunk_attn(*args, workspace=ws.cpu())


def test_two_captured_graphs_at_once():
    """Each graph has its own workspace (torch allocates it from the graph's pool); replayed side by
    side again and again, with other lengths in between, they give what eager calls give."""
    a, b = chunk_inputs([(200, 900), (1, 2000)], 8, 2, 128, 41), chunk_inputs([(5, 700)] * 12, 8, 2, 64, 42)
    outs, graphs, lens, kept = [], [], [], []
    for i in (a, b):
        args = [ints(v) for v in i[3:]]
        out = torch.zeros_like(i[0])
        dec.gqa_chunk_attn(i[0], i[1], i[2], *args, i[0].shape[2] ** -0.5, out)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            dec.gqa_chunk_attn(i[0], i[1], i[2], *args, i[0].shape[2] ** -0.5, out)
        outs.append(out)
        graphs.append(g)
        lens.append(args[2])
        kept.append(args)  # a graph's inputs have to live as long as it does
    streams = [torch.cuda.Stream() for _ in graphs]
    for cut in (0, 50, 3):
        for i, t in zip((a, b), lens):
            t.copy_(ints(i[5] - cut))
        torch.cuda.synchronize()
        for _ in range(5):
            for g, st in zip(graphs, streams):
                with torch.cuda.stream(st):
                    g.replay()
        torch.cuda.synchronize()
        for i, out in zip((a, b), outs):
            want = check_chunk((i[0], i[1], i[2], i[3], i[4], i[5] - cut))
            assert torch.equal(out, want)


@pytest.mark.parametrize("way", ["eager", "two streams", "captured"])
def test_calls_that_read_what_the_last_one_wrote(way):
    """Chains of calls, each reading what the kernel, copy or other stream's kernel just before it
    writes, give the same bits as with a synchronisation after each."""
    T, nq, nkv, d, n_pages = 320, 8, 2, 64, 40
    rng = np.random.default_rng(5)
    x = torch.tensor(rng.normal(size=(T, (nq + 2 * nkv) * d)), dtype=torch.float32, device="cuda")
    table = ints(rng.permutation(n_pages).reshape(2, 20))
    old, new, lens = ints([0, 0]), ints([300, 20]), ints([300, 20])
    u, us = torch.rand(T // 4, 3, device="cuda"), torch.rand(T // 4, device="cuda")

    def buffers():
        bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        z = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
        return dict(qkv=x.clone(), q=bf(T, nq, d), k=bf(n_pages, nkv, 16, d), v=bf(n_pages, nkv, 16, d),
                    a=bf(T, nq, d), b=bf(T, nq, d), table=torch.full_like(table, -1), free=table.flatten().clone(),
                    n_free=ints([n_pages]), cu=z(3), slot=z(T), pos=z(T), status=z(1) + 9, tok=z(T // 4, 3),
                    acc=z(T // 4), toks=z(T // 4, 4))

    def chain(s, after, streams):
        last = torch.cuda.current_stream()
        for k in range(6):
            st = streams[k % len(streams)] if streams else last
            st.wait_stream(last)
            with torch.cuda.stream(st):
                dec.paged_resize(old, new, s["table"], s["free"], s["n_free"], s["cu"], s["slot"], s["pos"], s["status"])
                after()
                dec.paged_rope_append(s["qkv"], s["slot"], s["pos"], s["q"], s["k"], s["v"], 1e4)
                after()
                dec.gqa_chunk_attn(s["q"], s["k"], s["v"], s["table"], s["cu"], lens, 0.125, s["a"])
                after()
                dec.gqa_chunk_attn(s["a"], s["k"], s["v"], s["table"], s["cu"], lens, 0.125, s["b"])
                after()
                s["q"].copy_(s["b"])
                after()
                dec.gqa_chunk_attn(s["q"], s["k"], s["v"], s["table"], s["cu"], lens, 0.125, s["a"])
                after()
                s["qkv"][:, :nq * d].add_(s["a"].reshape(T, nq * d))  # the next rows and the logits
                after()
                dec.spec_verify(s["qkv"].view(T // 4, 4, -1), None, s["tok"], None, None, u, us, s["acc"], s["toks"])
                after()
                s["tok"].copy_(s["toks"][:, :3].clamp_min(0))
                dec.paged_resize(new, old, s["table"], s["free"], s["n_free"], s["cu"], s["slot"], s["pos"], s["status"])
                after()
            last = st
        torch.cuda.current_stream().wait_stream(last)

    want, got = buffers(), buffers()
    chain(want, torch.cuda.synchronize, None)
    side = [torch.cuda.Stream() for _ in range(2)] if way != "eager" else None
    if way == "captured":
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            chain(got, lambda: None, side)
        g.replay()
    else:
        chain(got, lambda: None, side)
    torch.cuda.synchronize()
    assert want["status"].item() == 0 and want["toks"].max() > 0
    for name in want:
        assert torch.equal(got[name], want[name]), name


def test_first_call_of_a_process_may_be_captured():
    import subprocess
    import sys
    code = """
import torch
import decoder_only_transformer_layer_b200 as dec
i = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
bf = lambda *s: torch.ones(s, dtype=torch.bfloat16, device="cuda")
q, k, v, out = bf(3, 8, 64), bf(2, 2, 16, 64), bf(2, 2, 16, 64), bf(3, 8, 64) * 0
qkv, slot, pos = torch.ones(3, 12 * 64, device="cuda"), i(0, 1, 2), i(0, 1, 2)
table, cu, n = i(0, 1).view(1, 2), i(0, 3), i(3)
t, tok, u, us = torch.randn(1, 3, 100, device="cuda"), i(1, 2).view(1, 2), torch.rand(1, 2, device="cuda"), torch.rand(1, device="cuda")
acc, toks = i(0), i(0, 0, 0).view(1, 3)
f, nf, c2, st = i(0, 1, 2, 3), i(4), i(0, 0), i(9)
t2, z = i(-1, -1).view(1, 2), i(0)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    dec.paged_resize(z, n, t2, f, nf, c2, slot, pos, st)
    dec.paged_rope_append(qkv, slot, pos, q, k, v, 1e4)
    dec.gqa_chunk_attn(q, k, v, table, cu, n, 0.125, out)
    dec.spec_verify(t, None, tok, None, None, u, us, acc, toks)
g.replay()
torch.cuda.synchronize()
assert st.item() == 0 and (out == 1).all() and toks.max() < 100
print("ok")
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300,
                       cwd=__import__("os").path.dirname(__import__("os").path.dirname(__import__("os").path.abspath(__file__))))
    assert r.returncode == 0 and "ok" in r.stdout, r.stderr[-2000:]


def test_chunk_masked_places_hold_anything():
    # a key that is NaN or infinite reaches the rows that see it, and no other row
    inp = chunk_inputs([(200, 330), (3, 40)], 8, 2, 128, 12)
    q, kp, vp, table, cu, lens = inp
    base = check_chunk(inp)
    for pool in (kp, vp):
        for val in (float("nan"), float("inf"), -float("inf")):
            keep = pool.clone()
            j = 250  # position of new row 120 of sequence 0
            pool[table[0, j // 16], :, j % 16, 5] = val
            out = torch.empty_like(base)
            dec.gqa_chunk_attn(q, kp, vp, ints(table), ints(cu), ints(lens), 128 ** -0.5, out)
            before, after = slice(0, 120), slice(120, 200)
            assert torch.equal(out[before], base[before]) and torch.equal(out[200:], base[200:])
            if pool is kp and val != val:
                assert torch.isnan(out[after]).all()
            if pool is vp:
                assert (~torch.isfinite(out[after, :, 5])).all()
                others = torch.arange(128, device="cuda") != 5
                assert torch.isfinite(out[after][:, :, others]).all()
            pool.copy_(keep)


def test_chunk_large_scores():
    # scores of some hundreds: weights of one key after another, the running maximum moves far
    inp = chunk_inputs([(30, 900), (1, 400)], 8, 2, 128, 13)
    q, kp, vp, table, cu, lens = inp
    scale = 4.0
    out = torch.empty_like(q)
    dec.gqa_chunk_attn(q, kp, vp, ints(table), ints(cu), ints(lens), scale, out)
    want, mag = plain.chunk_attn(f64(q), np.nan_to_num(f64(kp)), np.nan_to_num(f64(vp)), table, cu, lens, scale)
    # scores up to about 4 * 5 * 11 = 200: an fp32 sum of 128 products is off by at most 2^-24 * 128 of
    # the sum of magnitudes (4 * 128 * 0.64 * 1.3 = 430), 3.3e-3, which moves a weight by that fraction
    tol = np.abs(want) * 2.0 ** -8 + mag * (2.0 ** -8 + 7e-3)
    assert (np.abs(f64(out) - want) <= tol).all()


def test_chunk_repeats_bitwise_whatever_the_workspace_holds():
    inp = chunk_inputs([(50, 800), (1, 3000), (300, 300)], 8, 2, 128, 14)
    need = dec.lib().gqa_chunk_attn_workspace(128)
    outs = []
    for fill in (0, 255, 77):
        ws = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
        outs.append(check_chunk(inp, workspace=ws))
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


def test_chunk_agrees_with_decode_attention():
    q, kp, vp, table, cu, lens = chunk_inputs([(1, 77), (1, 1000), (1, 1)], 32, 8, 128, 15)
    kp, vp = torch.nan_to_num(kp), torch.nan_to_num(vp)
    a, b = torch.empty_like(q), torch.empty_like(q)
    t = ints(np.maximum(table, 0))
    dec.gqa_chunk_attn(q, kp, vp, t, ints(cu), ints(lens), 128 ** -0.5, a)
    dec.gqa_decode_attn(q, None, None, kp, vp, t, ints(lens - 1), 32, 8, 128, 128 ** -0.5, 0, 1e4, b)
    assert (a.float() - b.float()).abs().max() <= 2.0 ** -6 * b.float().abs().max()


# ------------------------------------------------------------------ spec_verify

def verify_inputs(B, n, V, draft, seed, ld_extra=0, sharp=2.5):
    rng = np.random.default_rng(seed)
    ld = V + ld_extra
    t = torch.tensor(rng.normal(size=(B, n + 1, ld)) * sharp, dtype=torch.float32, device="cuda")
    d = (t[:, :n] + 0.5 * torch.tensor(rng.normal(size=(B, n, ld)), dtype=torch.float32, device="cuda"))
    temp = rng.uniform(0.4, 1.5, B).astype(np.float32)
    tok = np.zeros((B, n), int)
    dn = d[:, :, :V].cpu().numpy()
    for b in range(B):
        for i in range(n):
            tok[b, i] = rng.choice(V, p=plain.softmax(dn[b, i].astype(np.float64) / temp[b]))
    return dict(target=t[:, :, :V], draft=d[:, :, :V] if draft else None, tok=tok, count=None, temp=temp,
                u=rng.random((B, n)).astype(np.float32), us=rng.random(B).astype(np.float32))


def check_verify(x):
    B, n1, V = x["target"].shape
    acc = torch.full((B,), 77, **I32)
    tokens = torch.full((B, n1), 77, **I32)
    dev = lambda v: None if v is None else torch.tensor(v, device="cuda")  # noqa: E731
    dec.spec_verify(x["target"], x["draft"], ints(x["tok"]), None if x["count"] is None else ints(x["count"]),
                    dev(x["temp"]), dev(x["u"]), dev(x["us"]), acc, tokens)
    acc, tokens = acc.cpu().numpy(), tokens.cpu().numpy()
    t, d = x["target"].cpu().numpy(), None if x["draft"] is None else x["draft"].cpu().numpy()
    for b in range(B):
        a, nxt = plain.verify(t[b], None if d is None else d[b], x["tok"][b], n1 - 1 if x["count"] is None else x["count"][b],
                              1.0 if x["temp"] is None else x["temp"][b], x["u"][b], x["us"][b])
        want = list(x["tok"][b][:a]) + [nxt] + [-1] * (n1 - 1 - a)
        assert acc[b] == a and list(tokens[b]) == want, (b, acc[b], a, tokens[b], want)
    return acc


@pytest.mark.parametrize("B,n,V,draft,ld", [(1, 1, 2, 1, 0), (3, 4, 1000, 1, 0), (3, 4, 1001, 0, 0), (5, 2, 777, 1, 3),
                                            (1, 8, 49152, 1, 0), (4, 3, 32003, 0, 1), (64, 2, 257, 1, 7),
                                            (2, 4, 128256, 1, 64), (17, 0, 5000, 0, 0), (2, 64, 300, 1, 0), (9, 3, 1, 1, 0)])
def test_verify(B, n, V, draft, ld):
    accs = [check_verify(verify_inputs(B, n, V, draft, 100 * s + V, ld)) for s in range(3)]
    if draft and B * n >= 20 and V > 2:
        assert 0 < np.sum(accs) < 3 * B * n  # some drafts accepted, some not


def test_verify_counts_greedy_and_no_temperature():
    x = verify_inputs(24, 5, 3001, 1, 7)
    x["count"] = np.arange(24) % 9 - 2  # below 0 and above n too
    check_verify(x)
    x["temp"][::3] = 0.0
    x["temp"][1::6] = -1.0
    best = x["target"].argmax(-1).cpu().numpy()
    x["tok"][::3] = best[::3, :5]
    x["tok"][6, 2] += 1
    check_verify(x)
    x["temp"] = None
    check_verify(x)


def test_verify_greedy_ties_go_to_the_lowest_index():
    x = verify_inputs(2, 3, 40000, 0, 9)
    x["temp"][:] = 0
    x["target"][:, :, 123] = 50.0
    x["target"][:, :, [9000, 124, 39999]] = 50.0
    x["tok"][:] = 123
    x["tok"][1, 1] = 124
    assert list(check_verify(x)) == [3, 1]


def test_verify_tokens_outside_the_vocabulary_are_rejected():
    for draft in (0, 1):
        x = verify_inputs(4, 3, 500, draft, 11)
        x["tok"][0, 0], x["tok"][1, 1], x["tok"][2, 2], x["tok"][3, 0] = -1, 500, 2 ** 31 - 1, -2 ** 31
        check_verify(x)


def test_verify_borders():
    # uniforms of 0 and just below 1; equal distributions (always accepted); point masses
    x = verify_inputs(6, 3, 900, 1, 12)
    x["us"][:] = [0, 1 - 2.0 ** -24, 0.5, 0, 1 - 2.0 ** -24, 0.3]
    x["u"][:3], x["u"][3:] = 0.0, 1 - 2.0 ** -24
    check_verify(x)
    x["draft"] = x["target"][:, :3].clone()
    assert (check_verify(x) == 3).all()
    x = verify_inputs(6, 3, 900, 0, 13)
    x["target"][:, :, 17] = 200.0  # all the mass there
    x["tok"][:3], x["tok"][3:] = 17, 18
    x["u"][3:] = 0.5
    assert list(check_verify(x)) == [3, 3, 3, 0, 0, 0]


def test_verify_masked_logits():
    x = verify_inputs(4, 2, 5000, 1, 14)
    x["target"][:, :, 100:4900] = -math.inf
    x["draft"][:, :, 2000:] = -math.inf
    x["tok"][0, 0], x["tok"][1, 0] = 300, 4950
    check_verify(x)
    x["target"][2] = -math.inf  # nothing to choose from
    check_verify(x)
    x["target"][3, 1:] = torch.finfo(torch.float32).min
    x["target"][3, 1:, 7] = 0.0
    check_verify(x)


def test_verify_logits_that_are_not_finite_stay_in_the_buffers():
    # not allowed, and the tokens mean nothing; but they are tokens
    for val in (float("nan"), float("inf")):
        for draft in (0, 1):
            x = verify_inputs(6, 3, 3000, draft, 16)
            x["target"][1:3, 1] = val
            x["target"][3, 0, 55] = val
            if draft:
                x["draft"][4, 0, 5:] = val
            acc, tokens = torch.full((6,), 77, **I32), torch.full((6, 4), 7777, **I32)
            dec.spec_verify(x["target"], x["draft"], ints(x["tok"]), None, torch.tensor(x["temp"]).cuda(),
                            torch.tensor(x["u"]).cuda(), torch.tensor(x["us"]).cuda(), acc, tokens)
            assert ((acc >= 0) & (acc <= 3)).all() and ((tokens >= -1) & (tokens < 3000)).all()


def test_verify_close_calls_are_decided_in_64_bits():
    # u next to p / q: above and below by a few steps of u's own type, where fp32 sums cannot tell
    x = verify_inputs(64, 1, 20011, 1, 15)
    t, d = x["target"].cpu().numpy().astype(np.float64), x["draft"].cpu().numpy().astype(np.float64)
    for b in range(64):
        i = x["tok"][b, 0]
        r = plain.softmax(t[b, 0] / np.float64(x["temp"][b]))[i] / plain.softmax(d[b, 0] / np.float64(x["temp"][b]))[i]
        u = np.float32(min(r, 0.99))
        for _ in range(b % 4):
            u = np.nextafter(u, np.float32(0 if b % 8 < 4 else 1))
        x["u"][b, 0] = u
    check_verify(x)


# ------------------------------------------------------------------ together

class Step:
    """Buffers of a step of fixed size, as a serving loop keeps them."""

    def __init__(self, B, T, nq, nkv, d, n_pages, mp):
        self.shape = (nq, nkv, d)
        self.old, self.new = torch.zeros(B, **I32), torch.zeros(B, **I32)
        self.table = torch.full((B, mp), -1, **I32)
        self.free = torch.arange(n_pages, **I32)
        self.n_free = torch.tensor([n_pages], **I32)
        self.cu = torch.zeros(B + 1, **I32)
        self.slot, self.pos, self.status = torch.zeros(T, **I32), torch.zeros(T, **I32), torch.zeros(1, **I32)
        self.kp, self.vp = (torch.full((n_pages, nkv, 16, d), float("nan"), dtype=torch.bfloat16, device="cuda")
                            for _ in range(2))
        self.qkv = torch.zeros((T, (nq + 2 * nkv) * d), device="cuda")
        self.q, self.out = (torch.zeros((T, nq, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))

    def __call__(self):
        dec.paged_resize(self.old, self.new, self.table, self.free, self.n_free, self.cu, self.slot, self.pos,
                         self.status)
        dec.paged_rope_append(self.qkv, self.slot, self.pos, self.q, self.kp, self.vp, 10000.0)
        dec.gqa_chunk_attn(self.q, self.kp, self.vp, self.table, self.cu, self.new, self.shape[2] ** -0.5, self.out)


def expected(history, nq, nkv, d, new_rows):
    """out rows of the last `new_rows` of each sequence's whole QKV history [(n_b, width)]."""
    outs = []
    for x, n in zip(history, new_rows):
        L = len(x)
        h = x.reshape(L, nq + 2 * nkv, d)
        bf = lambda y: torch.tensor(y).bfloat16().double().numpy()  # noqa: E731
        rot = np.stack([plain.rope(h[p, :nq + nkv], p, 10000.0) for p in range(L)]) if L else h[:, :nq + nkv]
        q, k, v = bf(rot[:, :nq]), bf(rot[:, nq:]), bf(h[:, nq + nkv:])
        for p in range(L - n, L):
            G = nq // nkv
            outs.append(np.concatenate([plain.attend(q[p, g * G:(g + 1) * G], k[:, g], v[:, g], np.arange(L) <= p,
                                                     d ** -0.5, 0.0)[0] for g in range(nkv)]))
    return np.array(outs)


@pytest.mark.parametrize("captured", [False, True])
def test_steps_of_a_serving_loop(captured):
    """Prompts in, decode, drafts in and rejected, a sequence retired and replaced, with the
    step run eagerly or replayed from one captured graph."""
    nq, nkv, d, B, T = 8, 2, 128, 3, 200
    s = Step(B, T, nq, nkv, d, 60, 20)
    run = s
    if captured:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            s()  # nothing to do: no rows
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            s()
        run = graph.replay
    rng = np.random.default_rng(21)
    width = (nq + 2 * nkv) * d
    history = [np.zeros((0, width)) for _ in range(B)]
    #        prompts        decode       drafts       two rejected    another one in the place of sequence 1
    plan = [[70, 33, 0], [71, 34, 90], [76, 39, 95], [74, 36, 92], [75, 0, 93], [80, 110, 94], [80, 110, 94]]
    for new in plan:
        old = [len(h) for h in history]
        s.old.copy_(ints(old))
        s.new.copy_(ints(new))
        rows = [max(0, n - o) for o, n in zip(old, new)]
        x = rng.normal(size=(T, width)).astype(np.float32)
        s.qkv.copy_(torch.tensor(x))
        s.out.fill_(7.0)
        run()
        assert s.status.item() == 0
        at = 0
        for b in range(B):
            history[b] = np.concatenate([history[b][:new[b]], x[at:at + rows[b]].astype(np.float64)])
            at += rows[b]
        got = f64(s.out)
        assert (got[at:] == 7.0).all()
        want = expected(history, nq, nkv, d, rows)
        if at:
            # the bar of the fused decode test: a rotated value may round to the other side in fp32
            # (2^-8 relative), which moves the output by a small part of its scale
            assert np.max(np.abs(got[:at] - want)) <= 2.0 ** -5 * np.max(np.abs(want))
        held = sum(plain.pages(n) for n in new)
        assert s.n_free.item() == 60 - held
        pages = np.concatenate([s.table.cpu().numpy().ravel(), s.free[:60 - held].cpu().numpy()])
        assert sorted(p for p in pages if p >= 0) == list(range(60))  # every page once
    dec.check_standalone()


def test_two_streams_at_once_match_one_after_the_other():
    a = chunk_inputs([(300, 900), (1, 2000)], 8, 2, 128, 31)
    b = chunk_inputs([(1, 500)] * 20, 8, 2, 64, 32)
    xs = [verify_inputs(4, 3, 30000, 1, 33), verify_inputs(4, 3, 30000, 1, 34)]
    alone = [check_chunk(a), check_chunk(b)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.empty_like(a[0]), torch.empty_like(b[0])]
    dev = [[ints(v) for v in i[3:]] for i in (a, b)]
    acc = [torch.zeros(4, **I32) for _ in xs]
    toks = [torch.zeros((4, 4), **I32) for _ in xs]
    args = [[x["target"], x["draft"], ints(x["tok"]), None, torch.tensor(x["temp"]).cuda(), torch.tensor(x["u"]).cuda(),
             torch.tensor(x["us"]).cuda()] for x in xs]
    torch.cuda.synchronize()
    for _ in range(10):
        for k, (i, st) in enumerate(zip((a, b), streams)):
            with torch.cuda.stream(st):
                dec.gqa_chunk_attn(i[0], i[1], i[2], *dev[k], i[0].shape[2] ** -0.5, outs[k])
                dec.spec_verify(*args[k], acc[k], toks[k])
    torch.cuda.synchronize()
    # check_chunk scales by the fp32 value of the same factor
    assert torch.equal(outs[0], alone[0]) and torch.equal(outs[1], alone[1])
    for k, x in enumerate(xs):
        assert np.array_equal(check_verify(x), acc[k].cpu().numpy())


def test_decoder_verify_then_spec_verify_then_truncate():
    """The whole of a speculative step on a Decoder: drafts in, logits of every position, greedy
    verification on the device, rejected rows dropped; the tokens are those of plain greedy decoding."""
    import synth
    from synth import configs
    cfg = dict(configs.TINY)
    d = dec.Decoder(cfg, synth.make_weights(cfg))
    prompt = synth.tokens(16, cfg["vocab"], 1000)
    d.prefill(0, prompt, 0)
    seq = [int(d.last_argmax(1)[0])]
    for _ in range(8):
        d.step([seq[-1]], [16 + len(seq) - 1])
        seq.append(int(d.last_argmax(1)[0]))
    d.reset(0)
    d.prefill(0, prompt, 0)
    got = [int(d.last_argmax(1)[0])]
    n = 3
    logits = torch.empty((1, n + 1, cfg["vocab"]), device="cuda")
    acc, tokens = torch.zeros(1, **I32), torch.zeros((1, n + 1), **I32)
    while len(got) < 9:
        L = d.seq_len(0)
        k = len(got)
        drafts = (seq[k:k + n] + [0] * n)[:n]
        if k % 2:
            drafts[1] = (drafts[1] + 1) % cfg["vocab"]  # a wrong one
        d.verify(0, [got[-1]] + drafts, L, logits[0])
        dec.spec_verify(logits, None, ints([drafts]), None, torch.zeros(1, device="cuda"),
                        torch.zeros((1, n), device="cuda"), torch.zeros(1, device="cuda"), acc, tokens)
        a = int(acc.item())
        got += [int(t) for t in tokens[0, :a + 1]]
        d.truncate(0, L + a + 1)
    assert got[:9] == seq[:9]
    d.close()
