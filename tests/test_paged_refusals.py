"""Argument checks of the paged step's entry points: refused on the host, before any CUDA call."""
import ctypes as C

import numpy as np
import pytest
import torch

import _paged_plain as plain
import decoder_only_transformer_layer_b200 as dec

P = 1 << 20  # a non-null, aligned address that is never used: every call below is refused

RESIZE = dict(old_len=P, new_len=P, B=4, block_table=P, max_pages=8, page_size=16, free_pages=P, n_pages=32, n_free=P,
              cu_rows=P, slot=P, row_pos=P, T=16, status=P, stream=None)
APPEND = dict(qkv=P, ld=1536, q_norm=None, k_norm=None, eps=1e-6, rope_base=1e4, slot=P, row_pos=P, T=4, nq=8, nkv=2,
              d=128, page_size=16, q_out=P, k_pool=P, v_pool=P, n_pages=32, stream=None)
CHUNK = dict(q=P, ldq=1024, k_pool=P, v_pool=P, n_pages=32, block_table=P, max_pages=8, cu_rows=P, kv_len=P, B=4, T=16,
             nq=8, nkv=2, d=128, page_size=16, scale=0.1, window=0, softcap=0.0, out=P, workspace=P,
             workspace_bytes=1 << 40, stream=None)
VERIFY = dict(target=P, target_row=1000, target_seq=5000, draft=P, draft_row=1000, draft_seq=4000, draft_tok=P,
              n_draft=None, temperature=None, u_accept=P, u_sample=P, B=2, n=4, V=1000, n_accepted=P, tokens=P,
              workspace=P, workspace_bytes=1 << 40, stream=None)
BAD, UNSUP = 1, 7


def nan():
    return float("nan")


CASES = [("paged_resize", RESIZE, BAD, {k: None}) for k in
         ("old_len", "new_len", "block_table", "free_pages", "n_free", "cu_rows", "slot", "row_pos", "status")]
CASES += [("paged_resize", RESIZE, s, c) for s, c in (
    (BAD, dict(B=0)), (BAD, dict(T=-1)), (BAD, dict(max_pages=0)), (BAD, dict(n_pages=0)), (UNSUP, dict(page_size=32)),
    (UNSUP, dict(B=4097)), (UNSUP, dict(n_pages=1 << 28)), (UNSUP, dict(max_pages=1 << 28)),
    (UNSUP, dict(T=(1 << 30) + 1)))]
CASES += [("paged_rope_append", APPEND, BAD, {k: None}) for k in
          ("qkv", "slot", "row_pos", "q_out", "k_pool", "v_pool")]
CASES += [("paged_rope_append", APPEND, s, c) for s, c in (
    (BAD, dict(T=-1)), (BAD, dict(nq=0)), (BAD, dict(nkv=0)), (BAD, dict(ld=1535)), (BAD, dict(rope_base=0.0)),
    (BAD, dict(rope_base=nan())), (BAD, dict(q_norm=P, eps=nan())), (BAD, dict(k_norm=P, eps=-1.0)),
    (UNSUP, dict(d=96)), (UNSUP, dict(page_size=8)), (UNSUP, dict(n_pages=1 << 28)), (BAD, dict(n_pages=0)),
    (UNSUP, dict(q_out=P + 8)), (UNSUP, dict(k_pool=P + 2)), (UNSUP, dict(v_pool=P + 4)), (UNSUP, dict(q_norm=P + 4)),
    (UNSUP, dict(k_norm=P + 8)), (UNSUP, dict(T=(1 << 30) + 1)), (UNSUP, dict(nq=1 << 21, ld=1 << 40)))]
CASES += [("gqa_chunk_attn", CHUNK, BAD, {k: None}) for k in
          ("q", "k_pool", "v_pool", "block_table", "cu_rows", "kv_len", "out", "workspace")]
CASES += [("gqa_chunk_attn", CHUNK, s, c) for s, c in (
    (BAD, dict(B=0)), (BAD, dict(T=-1)), (BAD, dict(nq=9)), (BAD, dict(nkv=0)), (BAD, dict(ldq=1016)),
    (UNSUP, dict(ldq=1028)), (UNSUP, dict(q=P + 8)), (UNSUP, dict(k_pool=P + 2)), (UNSUP, dict(out=P + 4)),
    (UNSUP, dict(workspace=P + 4)), (BAD, dict(workspace_bytes=0)), (BAD, dict(scale=0.0)), (BAD, dict(scale=nan())),
    (BAD, dict(scale=float("inf"))), (BAD, dict(window=-1)), (BAD, dict(softcap=-1.0)), (BAD, dict(softcap=nan())),
    (UNSUP, dict(scale=2.0 ** -41)), (UNSUP, dict(scale=2.0 ** 41)), (UNSUP, dict(softcap=2.0 ** -21)),
    (UNSUP, dict(d=80, ldq=1024)), (UNSUP, dict(page_size=32)), (UNSUP, dict(nq=34, nkv=2, ldq=8192)),
    (UNSUP, dict(B=4097)), (UNSUP, dict(max_pages=1 << 27)), (UNSUP, dict(n_pages=1 << 27)))]
CASES += [("spec_verify", VERIFY, BAD, {k: None}) for k in
          ("target", "draft_tok", "u_accept", "u_sample", "n_accepted", "tokens", "workspace")]
CASES += [("spec_verify", VERIFY, s, c) for s, c in (
    (BAD, dict(B=0)), (BAD, dict(n=-1)), (BAD, dict(V=0)), (BAD, dict(target_row=999)), (BAD, dict(target_seq=-1)),
    (BAD, dict(draft_row=999)), (BAD, dict(draft_seq=-1)), (BAD, dict(workspace=P + 8)), (BAD, dict(workspace_bytes=0)),
    (UNSUP, dict(n=65)), (UNSUP, dict(B=8000)), (UNSUP, dict(V=(1 << 30) + 1, target_row=1 << 31, draft_row=1 << 31)))]


@pytest.mark.parametrize("name,good,status,change", CASES, ids=lambda v: None if isinstance(v, dict) and len(v) > 3 else str(v))
def test_refused(name, good, status, change):
    args = dict(good, **change)
    assert set(change) <= set(good)
    assert getattr(dec.lib(), name)(*args.values()) == status
    assert dec.lib().dec_last_error()


def test_nothing_to_do_is_fine():
    assert dec.lib().paged_rope_append(*dict(APPEND, T=0, qkv=None, slot=None, row_pos=None, q_out=None).values()) == 0
    assert dec.lib().gqa_chunk_attn(*dict(CHUNK, T=0, q=None, out=None).values()) == 0


def test_workspace_sizes():
    L = dec.lib()
    assert L.gqa_chunk_attn_workspace(64) > 0 and L.gqa_chunk_attn_workspace(128) > 0
    assert L.gqa_chunk_attn_workspace(96) == 0
    assert L.spec_verify_workspace(1, 0, 1) > 0 and L.spec_verify_workspace(0, 1, 1) == 0


def test_wrappers_refuse_what_an_address_would_hide():
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(TypeError):  # lengths of another type
        dec.paged_resize(torch.zeros(2), i(2), i(2, 3), i(9), i(1), i(3), i(4), i(4), i(1))
    with pytest.raises(ValueError):  # row starts too short
        dec.paged_resize(i(2), i(2), i(2, 3), i(9), i(1), i(2), i(4), i(4), i(1))
    with pytest.raises(ValueError):  # a transposed table
        dec.paged_resize(i(2), i(2), i(3, 2).t(), i(9), i(1), i(3), i(4), i(4), i(1))
    with pytest.raises(ValueError):  # on the host
        dec.paged_resize(i(2), i(2), i(2, 3), i(9), i(1), i(3), i(4), i(4), i(1))
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    pool = bf(5, 2, 16, 64)
    with pytest.raises(ValueError):  # heads apart
        dec.gqa_chunk_attn(bf(4, 8, 64)[:, ::2], pool, pool, i(1, 4), i(2), i(1), 1.0, bf(4, 4, 64))
    with pytest.raises(TypeError):
        dec.gqa_chunk_attn(torch.zeros(4, 4, 64), pool, pool, i(1, 4), i(2), i(1), 1.0, bf(4, 4, 64))
    with pytest.raises(ValueError):  # values of a row apart
        dec.paged_rope_append(torch.zeros(4, 1024)[:, ::2], i(4), i(4), bf(4, 4, 64), pool, pool, 1e4)
    f = torch.zeros
    with pytest.raises(ValueError):
        dec.spec_verify(f(2, 4, 50), f(2, 4, 50), i(2, 3), None, None, f(2, 3), f(2), i(2), i(2, 4))
    with pytest.raises(TypeError):
        dec.spec_verify(f(2, 4, 50).half(), None, i(2, 3), None, None, f(2, 3), f(2), i(2), i(2, 4))


def test_plain_verify_keeps_the_target_distribution():
    """The plain form the GPU is held to: over a fine grid of uniforms, the first emitted token
    follows the target's distribution whatever the draft's (here three tokens, exactly)."""
    rng = np.random.default_rng(3)
    t, d = rng.normal(size=(2, 3)), rng.normal(size=(1, 3))
    p, q = plain.softmax(t[0]), plain.softmax(d[0])
    N = 400
    grid = (np.arange(N) + 0.5) / N
    got = np.zeros(3)
    for x in range(3):
        for u in grid:
            acc, _ = plain.verify(t, d, np.array([x]), 1, 1.0, [u], 0.5)
            if acc:
                got[x] += q[x] / N
            else:
                for us in (np.arange(20) + 0.5) / 20:
                    got[plain.verify(t, d, np.array([x]), 1, 1.0, [u], us)[1]] += q[x] / N / 20
    # each grid puts a border off by at most half a cell: 1/(2N) for u per token, 1/40 of the
    # rejected mass for us
    rej = 1 - np.minimum(p, q).sum()
    assert np.abs(got - p).max() <= 3 / (2 * N) + rej * 2 / 40


def test_plain_resize_back_restores_everything():
    rng = np.random.default_rng(5)
    for _ in range(30):
        B, n_pages = 6, 80
        old, new = rng.integers(0, 120, B), rng.integers(0, 120, B)
        perm = rng.permutation(n_pages)
        table = np.full((B, 8), -1)
        at = 0
        for b in range(B):
            k = plain.pages(old[b])
            table[b, :k] = perm[at:at + k]
            at += k
        free = np.full(n_pages, -1)
        free[:n_pages - at] = perm[at:]
        s, cu, slot, pos, t2, f2, n2 = plain.resize(old, new, table, free, n_pages - at, 800, n_pages)
        assert s == 0
        s, _, _, _, t3, f3, n3 = plain.resize(new, old, t2, f2, n2, 800, n_pages)
        assert s == 0 and n3 == n_pages - at
        assert np.array_equal(t3, table) and np.array_equal(f3[:n3], free[:n3])


def test_library_names_are_bound():
    for f in ("paged_resize", "paged_rope_append", "gqa_chunk_attn", "spec_verify"):
        assert getattr(dec.lib(), f).restype == C.c_int and f in dec.__all__


def test_wrappers_name_a_missing_tensor():
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    f = torch.zeros
    pool = bf(5, 2, 16, 64)
    calls = (
        (dec.paged_resize, [i(2), i(2), i(2, 3), i(9), i(1), i(3), i(4), i(4), i(1)], range(9)),
        (dec.paged_rope_append, [f(4, 512), i(4), i(4), bf(4, 4, 64), pool, pool, 1e4], range(6)),
        (dec.gqa_chunk_attn, [bf(4, 4, 64), pool, pool, i(1, 4), i(2), i(1), 1.0, bf(4, 4, 64)], (0, 1, 2, 3, 4, 5, 7)),
        (dec.spec_verify, [f(2, 4, 50), None, i(2, 3), None, None, f(2, 3), f(2), i(2), i(2, 4)], (0, 2, 5, 6, 7, 8)))
    for call, args, needed in calls:
        for k in needed:
            for wrong in (None, [1, 2]):
                with pytest.raises(TypeError, match="expected a torch tensor"):
                    call(*args[:k], wrong, *args[k + 1:])


def test_wait_hook_takes_known_barriers_only():
    L = dec.lib()
    assert L.dec_test_chunk_wait(-1) == BAD and L.dec_test_chunk_wait(11) == BAD
    assert L.dec_test_chunk_wait(0) == 0


def test_a_workspace_for_the_largest_call_serves_smaller_ones():
    size = dec.lib().spec_verify_workspace
    Bs, ns, Vs = [*range(1, 80), 147, 148, 149, 300, 500], [*range(0, 10), 31, 63, 64], [1, 500, 4096, 4097, 8192, 32003,
                                                                                        49152, 128256, 151936, 1 << 20]
    for n in ns:
        for V in Vs:
            sizes = [size(B, n, V) for B in Bs]
            assert sizes == sorted(sizes) and sizes[0] > 0
    for B in Bs:
        for V in Vs:
            sizes = [size(B, n, V) for n in ns]
            assert sizes == sorted(sizes)
        for n in ns:
            sizes = [size(B, n, V) for V in Vs]
            assert sizes == sorted(sizes)
    # and each serves the call itself: one piece a row at least, the pieces the launch takes at most
    for B in Bs:
        for n in ns:
            for V in Vs:
                rows, s = B * (2 * n + 1), -(-V // 4096)
                while s > 1 and rows * s > 148 * 32:
                    s = (s + 1) // 2
                assert size(B, n, V) >= 16 * rows * s
