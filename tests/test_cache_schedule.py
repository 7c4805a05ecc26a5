"""How the attention over caches of per-sequence length shares its key tiles (host computation, the
code the kernel runs; no GPU needed): every tile of every unit is taken once, in order, the workers'
shares (tiles, and unit_cost more for each unit begun) are even, the partial results of a cut unit lie in
slots that no other unit uses, and the tiles are numbered without gaps."""
import random

import pytest

from transformer_gqa_attention_gb300 import _build, abi


@pytest.fixture(scope="module", autouse=True)
def _built():
    _build.build()


def check(lens, n_new, S_max, units, workers, cost):
    pieces = abi.attn_debug_cache_schedule(lens, n_new, S_max, units, cost, workers)
    tiles = [max(1, -(-(n + n_new) // 128)) if 0 <= n <= S_max - n_new else 1 for n in lens]
    want = [(b, u, t) for b in range(len(lens)) for u in range(units) for t in range(tiles[b])]
    got = [(b, u, t) for _, b, u, first, n, *_ in pieces for t in range(first, first + n)]
    assert got == want
    places = sum((t + cost) * units for t in tiles)
    share = places / min(workers, places)
    load = {}
    number = 0
    for c, b, u, first, n, _, _, flat in pieces:
        assert n > 0 and flat == number
        number += n
        load[c] = load.get(c, 0) + n + (cost if first == 0 and c in load else 0)
    assert max(load.values()) <= share + 1
    assert [c for c, *_ in pieces] == sorted(c for c, *_ in pieces)
    cut, used = {}, {}
    for c, b, u, first, n, slot, last, _ in pieces:
        if slot < 0:
            assert first == 0 and n == tiles[b] and last == c
            continue
        assert slot not in used and slot // 2 == c
        used[slot] = (b, u)
        cut.setdefault((b, u), []).append((c, first, slot, last))
    for parts in cut.values():  # slots 2 f + 1, then 2 c of every worker up to the last
        f = parts[0][0]
        assert len({p[3] for p in parts}) == 1
        assert [p[2] for p in parts] == [2 * f + 1] + [2 * c for c in range(f + 1, parts[0][3] + 1)]
        assert parts[0][1] == 0 and len(parts) >= 2


@pytest.mark.parametrize("cost", [0, 2, 3, 6, 9])
@pytest.mark.parametrize("workers", [1, 2, 7, 76, 148, 304])
@pytest.mark.parametrize("lens", [[0], [1], [127], [128], [129], [32000], [0, 0, 0], [5, 4000, 128, 1], [-1, 70, 2 ** 31 - 1],
                                  [300] * 33])
def test_small_batches(lens, workers, cost):
    for units in (1, 8, 16, 32):
        for n_new in (0, 1, 26):
            check(lens, n_new, 40000, units, workers, cost)


def test_random_batches():
    rng = random.Random(1)
    for _ in range(40):
        B = rng.choice([1, 3, 40, 385, 800, 1024])
        top = rng.choice([10, 1000, 20000])
        check([rng.randint(-1, top) for _ in range(B)], rng.choice([0, 1, 64]), top + 64, rng.choice([1, 2, 8]),
              rng.choice([76, 152, 304]), rng.choice([2, 3, 6]))


def test_arguments():
    for kw in (dict(units=0), dict(unit_cost=-1), dict(workers=0), dict(n_new=-1), dict(S_max=0)):
        a = dict(n_new=1, S_max=10, units=1, unit_cost=2, workers=2) | kw
        with pytest.raises(abi.GQAError):
            abi.attn_debug_cache_schedule([1], **a)
    with pytest.raises(abi.GQAError):
        abi.attn_debug_cache_schedule([], 1, 10, 1, 2, 2)
