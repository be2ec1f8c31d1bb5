"""The paged step's operators at the ends of what their documentation allows."""
import math

import numpy as np
import pytest
import torch

import decoder_only_transformer_layer_b200 as dec
from test_gpu_paged_step import I32, check_chunk, check_verify, chunk_inputs, ints, verify_inputs

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ spec_verify

def run_verify(x):
    """(accepted, tokens) of the inputs of verify_inputs."""
    B, n1, _ = x["target"].shape
    acc, tokens = torch.full((B,), 77, **I32), torch.full((B, n1), 77, **I32)
    dev = lambda v: None if v is None else torch.tensor(v, device="cuda")  # noqa: E731
    dec.spec_verify(x["target"], x["draft"], ints(x["tok"]), None if x["count"] is None else ints(x["count"]),
                    dev(x["temp"]), dev(x["u"]), dev(x["us"]), acc, tokens)
    return acc.cpu().numpy(), tokens.cpu().numpy()


def test_verify_temperatures_and_counts_written_just_before_the_call():
    x = verify_inputs(40, 4, 9001, 1, 51)
    rng = np.random.default_rng(51)
    sets = [(torch.tensor(rng.choice([0.0, 0.3, 1.0, 2.0], 40).astype(np.float32)).cuda(), ints(rng.integers(0, 5, 40)))
            for _ in range(8)]
    temp, count = torch.ones(40, device="cuda"), torch.zeros(40, **I32)
    rest = (torch.tensor(x["u"]).cuda(), torch.tensor(x["us"]).cuda())
    tok = ints(x["tok"])

    def call(t, c, after):
        acc, tokens = torch.zeros(40, **I32), torch.zeros((40, 5), **I32)
        temp.copy_(t)
        count.copy_(c)
        after()
        dec.spec_verify(x["target"], x["draft"], tok, count, temp, *rest, acc, tokens)
        return acc, tokens

    want = [call(t, c, torch.cuda.synchronize) for t, c in sets]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [call(t, c, lambda: None) for t, c in sets]
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert torch.equal(g[0], w[0]) and torch.equal(g[1], w[1])


@pytest.mark.parametrize("draft", [0, 1])
def test_verify_at_infinite_temperature(draft):
    """Every token that is not masked is as likely as any other."""
    x = verify_inputs(12, 4, 3000, draft, 52)
    x["temp"][:9] = math.inf
    if not draft:
        x["u"][:, :2] /= 3000  # about 1 / V: some of these drafts are accepted
    acc = check_verify(x)
    assert (acc[:9] == 4).all() if draft else 0 < acc[:9].sum() < 36
    # with masked tokens: as logits of 0 at temperature 1
    x["target"][:, :, 100:2500] = -math.inf
    flat = dict(x, target=torch.where(torch.isinf(x["target"]), -math.inf, 0.0), temp=np.ones(12, np.float32))
    if draft:
        x["draft"][:, :, 2000:] = -math.inf
        flat["draft"] = torch.where(torch.isinf(x["draft"]), -math.inf, 0.0)
    x["temp"][:] = math.inf
    x["tok"][:] = np.random.default_rng(52).integers(0, 3000, (12, 4))
    check_verify(flat)
    for got, want in zip(run_verify(x), run_verify(flat)):
        assert np.array_equal(got, want)


def test_verify_temperatures_far_from_one():
    """The distribution depends on logits over temperature, at any scale of the two."""
    x = verify_inputs(40, 3, 2000, 1, 53)
    scale = np.float32(2.0) ** np.repeat([-116, -60, 60, 116], 10).astype(np.float32)
    for k in ("target", "draft"):
        x[k] = x[k] * torch.tensor(scale, device="cuda")[:, None, None]
    x["temp"] = x["temp"] * scale
    acc = check_verify(x)
    assert 0 < acc.sum() < 120
    # one token has everything; nearly equal chances
    x = verify_inputs(8, 3, 2000, 1, 54)
    x["temp"][:] = [1e-30, 1e-38, 1e-45, 1e-10, 1e10, 1e30, 3e38, 1e5]
    check_verify(x)


def test_verify_greedy_rows_without_a_token_accept_nothing():
    x = verify_inputs(6, 3, 3000, 0, 55)
    x["temp"][:5] = [0.0, -1.0, 0.0, 0.0, 0.0]
    x["target"][:4, 1] = -math.inf
    x["target"][4] = -math.inf
    best = x["target"].argmax(-1).cpu().numpy()
    x["tok"][:] = best[:, :3]
    x["tok"][:5, 1] = [2 ** 31 - 1, 2 ** 31 - 1, 0, -1, 2 ** 31 - 1]
    x["tok"][4, 0] = 2 ** 31 - 1
    assert list(check_verify(x)[:5]) == [1, 1, 1, 1, 0]


def test_verify_close_calls_of_long_rows():
    """Acceptances next to equality where a thread sums 65536 values in fp32: equal logits, at which every
    step rounds the same way. 37 sequences of 64 places put a row into one piece."""
    B, n, V = 37, 64, 1 << 24
    t = torch.empty((1, n + 1, V), device="cuda")  # the counts see to it that only two rows are used
    t[:, 0] = -0.714
    t[:, 0, :4096] = 0.0  # every thread's first largest value
    t[:, 0, 9000] = 14.0
    t[:, 1] = 0.0
    t[:, 1, 7] = 40.0  # the token after an accepted draft
    w = math.exp(float(np.float32(-0.714)))
    p = math.exp(14.0) / (math.exp(14.0) + 4096 + (V - 4097) * w)
    u = np.zeros((B, n), np.float32)
    u[:, 0] = (p * (1 + (np.arange(B) - 18.5) * 1e-5)).astype(np.float32)
    acc, tokens = torch.zeros(B, **I32), torch.zeros((B, n + 1), **I32)
    dec.spec_verify(t.expand(B, n + 1, V), None, ints(np.full((B, n), 9000)), torch.ones(B, **I32), None,
                    torch.tensor(u).cuda(), torch.full((B,), 0.5, device="cuda"), acc, tokens)
    # the nearest uniform is 5e-6 of p away, many steps of its type
    want = (u[:, 0].astype(np.float64) < p).astype(int)
    assert 0 < want.sum() < B and np.array_equal(acc.cpu().numpy(), want)
    tokens = tokens.cpu().numpy()
    assert (tokens[want == 1, 0] == 9000).all() and (tokens[want == 1, 1] == 7).all()


@pytest.mark.parametrize("B,n,V", [(9, 3, 3000), (10, 3, 3000), (16, 2, 3000), (17, 2, 3000), (18, 2, 5000), (19, 2, 3000),
                                   (36, 2, 3000), (37, 2, 3000), (73, 2, 1500), (74, 2, 1500), (75, 2, 1500),
                                   (147, 1, 1000), (148, 1, 1000), (149, 1, 1000), (300, 1, 1000), (100, 7, 20000),
                                   (40, 30, 4097)])
def test_verify_batches_around_the_ways_of_sharing_the_work(B, n, V):
    check_verify(verify_inputs(B, n, V, 1, B + n))


@pytest.mark.parametrize("B,n", [(508, 64), (65535, 0)])
def test_verify_most_rows(B, n):
    check_verify(verify_inputs(B, n, 24, 1, 56))


# ------------------------------------------------------------------ gqa_chunk_attn

@pytest.mark.parametrize("d,kind", [(128, k) for k in range(1, 11)] + [(64, k) for k in (1, 4, 5, 7)])
def test_chunk_wait_that_runs_out_is_reported_and_the_next_call_is_correct(d, kind):
    """Whichever barrier never completes, with loads and products in flight: the call ends with an
    error status, and the next one finds shared memory and TMEM in order."""
    # eight tiles of six blocks a CTA, the last of each cleaned; some tiles of two sub-tiles
    rows = [(2, 700)] * 590 + [(100, 700)] * 5
    inp = chunk_inputs(rows, 8, 2, d, 61)
    q, kp, vp, table, cu, lens = inp
    args = (q, kp, vp, ints(table), ints(cu), ints(lens), d ** -0.5)
    want, got = torch.zeros_like(q), torch.zeros_like(q)
    dec.gqa_chunk_attn(*args, want)
    dec.check_standalone()
    dec.test_chunk_wait(kind)
    try:
        dec.gqa_chunk_attn(*args, got)
        with pytest.raises(dec.DecError) as e:
            dec.check_standalone()
        assert e.value.status == "TIMEOUT"
    finally:
        dec.test_chunk_wait(0)
    dec.check_standalone()  # the word was cleared
    for _ in range(2):
        got.zero_()
        dec.gqa_chunk_attn(*args, got)
        dec.check_standalone()
        assert torch.equal(got, want)

@pytest.mark.parametrize("cap", [0.0, 30.0])
@pytest.mark.parametrize("val", [math.inf, -math.inf])
def test_chunk_scores_that_are_not_finite(val, cap):
    """A score of -inf leaves its key out, one of +inf makes its row NaN; under a cap both are the cap."""
    inp = chunk_inputs([(200, 330), (3, 40), (1, 600), (2, 700)], 8, 2, 128, 62)
    table = inp[3]
    for b, j in ((0, 250), (0, 20), (1, 39), (2, 300), (3, 699)):
        inp[1][table[b, j // 16], :, j % 16, 5] = val
    out = check_chunk(inp, cap=cap)
    assert torch.isnan(out).any() == (cap == 0.0)



@pytest.mark.parametrize("rows", [[(1, 1)], [(3, 40), (1, 600)], [(2, 3000)], [(130, 5000)]], ids=str)
def test_chunk_rows_whose_scores_are_all_minus_infinity(rows):
    """Such a row gives zeros, in one piece or in many; under a cap its scores are all the same."""
    q, kp, vp, table, cu, lens = chunk_inputs(rows, 8, 2, 128, 64)
    q.abs_().clamp_min_(0.125)
    kp.fill_(-math.inf)
    out = torch.full_like(q, 3.0)
    dec.gqa_chunk_attn(q, kp, vp, ints(table), ints(cu), ints(lens), 0.1, out)
    dec.check_standalone()
    assert (out == 0).all()
    check_chunk((q, kp, vp, table, cu, lens), cap=20.0)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("window", [0, 1, 500])
def test_chunk_values_that_are_not_numbers_stay_with_the_rows_that_see_them(window, d):
    """V holds NaN at the end, next to it, at window's edges and in the middle, in tiles cut into many
    pieces too: a row's result is NaN in that column exactly where it sees such a key."""
    rows = [(3, 3000), (200, 1500), (1, 700), (2, 129), (40, 20)]
    inp = chunk_inputs(rows, 8, 2, d, 66)
    table = inp[3]
    for col, (b, j) in enumerate([(0, 2998), (0, 2498), (0, 2999), (1, 900), (1, 1420), (1, 1299), (2, 699), (2, 199),
                                  (3, 127), (3, 128), (4, 19), (4, 0)]):
        inp[2][table[b, j // 16], :, j % 16, 5 * col] = float("nan")
    check_chunk(inp, window=window)



def test_chunk_most_sequences():
    rng = np.random.default_rng(65)
    check_chunk(chunk_inputs([(int(rng.integers(0, 3)), int(rng.integers(2, 40))) for _ in range(4096)], 2, 1, 64, 65))



def test_a_check_reports_and_clears_every_kind_of_time_out():
    """A wait of gqa_chunk_attn and one of the tensor-core GEMM run out: one check tells, and the next
    call of either is correct."""
    from _util import to_dev_bf16
    from test_gpu_boundary import _gemm_case
    W, x, _ = _gemm_case()
    Wd, xd = to_dev_bf16(W, torch), to_dev_bf16(x, torch)
    y, good = (torch.zeros((x.shape[0], W.shape[0]), device="cuda") for _ in range(2))
    q, kp, vp, table, cu, lens = chunk_inputs([(2, 300)] * 40, 8, 2, 64, 63)
    args = (q, kp, vp, ints(table), ints(cu), ints(lens), 0.125)
    want, got = torch.zeros_like(q), torch.zeros_like(q)
    dec.weight_gemv(Wd, xd, good)
    dec.gqa_chunk_attn(*args, want)
    dec.check_standalone()
    dec.test_gemm_wait(1, 1 << 21)
    dec.test_chunk_wait(7)
    try:
        dec.weight_gemv(Wd, xd, y)
        dec.gqa_chunk_attn(*args, got)
        with pytest.raises(dec.DecError) as e:
            dec.check_standalone()
        assert e.value.status == "TIMEOUT"
    finally:
        dec.test_gemm_wait(0, 0)
        dec.test_chunk_wait(0)
    dec.check_standalone()  # nothing is left of either
    dec.weight_gemv(Wd, xd, y)
    dec.gqa_chunk_attn(*args, got)
    dec.check_standalone()
    assert torch.equal(y, good) and torch.equal(got, want)


@pytest.mark.parametrize("used", [False, True])
def test_a_check_of_one_stream_does_not_wait_for_others(used):
    """Nothing goes through the default stream, which would wait for every stream that is not marked
    as independent of it (here one that sleeps for about two seconds)."""
    import os
    import subprocess
    import sys
    code = f"""
import ctypes, time
import torch
import decoder_only_transformer_layer_b200 as dec
bf = lambda *s: torch.ones(s, dtype=torch.bfloat16, device="cuda")
i = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
q, k, v, out = bf(3, 8, 64), bf(2, 2, 16, 64), bf(2, 2, 16, 64), bf(3, 8, 64) * 0
args = (q, k, v, i(0, 1).view(1, 2), i(0, 3), i(3), 0.125, out)
side = torch.cuda.Stream()
handle = ctypes.c_uint64(0)
assert torch.cuda.cudart().cudaStreamCreate(ctypes.addressof(handle)) == 0
slow = torch.cuda.ExternalStream(handle.value)
for sleep in (1000, 1 << 32):
    torch.cuda.synchronize()
    with torch.cuda.stream(slow):
        torch.cuda._sleep(sleep)
    with torch.cuda.stream(side):
        if {used}:
            dec.gqa_chunk_attn(*args)
        t0 = time.monotonic()
        dec.check_standalone()
        waited = time.monotonic() - t0
    assert sleep == 1000 or not slow.query()
    torch.cuda.synchronize()
assert waited < 0.5, waited
print("ok")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300, cwd=root)
    assert r.returncode == 0 and "ok" in r.stdout, r.stderr[-2000:]
