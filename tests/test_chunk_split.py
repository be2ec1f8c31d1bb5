"""The work split of gqa_chunk_attn, checked on the host: every (tile, key block) of every kv head
in one run, tiles cut between runs joined from the run that starts them."""
import numpy as np
import pytest

import decoder_only_transformer_layer_b200 as dec


def check(rows, G, nkv, window=0, max_pages=None):
    n = [r for r, _ in rows]
    L = [k for _, k in rows]
    cu = np.concatenate([[0], np.cumsum(n)])
    mp = max_pages or max(1, -(-max(L) // 16))
    assert dec.test_chunk_split(cu, L, mp, G, nkv, window) == 0, (rows, G, nkv, window)


@pytest.mark.parametrize("G", [1, 2, 3, 4, 5, 7, 8, 9, 12, 13, 16])
@pytest.mark.parametrize("window", [0, 1, 17, 128, 1000, 2 ** 31 - 1])
def test_random_lengths(G, window):
    rng = np.random.default_rng(G * 1000 + window % 999)
    for _ in range(40):
        B = int(rng.integers(1, 40))
        hi = int(rng.choice([2, 40, 700]))
        rows = []
        for _ in range(B):
            n = int(rng.integers(0, hi))
            rows.append((n, n + int(rng.integers(-5, int(rng.choice([2, 200, 5000]))))))
        check(rows, G, int(rng.integers(1, 9)), window)


def test_borders():
    for n, L in [(0, 0), (1, 0), (1, 1), (5, 2), (128, 128), (129, 128), (300, 4), (1, 128), (1, 129), (8192, 8192),
                 (8192, 100000), (100000, 100000), (1, 2 ** 28)]:
        for window in (0, 1, 128, 5000):
            check([(n, L)], 4, 8, window)
    check([(1, 1000000)] * 500, 8, 1)
    check([(3, 50)] * 4096, 4, 8)


def test_hostile_arrays_stay_in_range():
    # row starts that descend or leave the buffer and lengths beyond the table are taken into range
    for cu in ([0, 50, 20, 70], [-5, 10, 1 << 30, 70], [70, 0, 0, 70]):
        assert dec.test_chunk_split(cu, [100, -7, 1 << 30], 10, 4, 2) == 0
