"""The largest numbers of workers that share key tiles (host computation, no GPU needed): shares are
found in 32-bit arithmetic, which holds for up to 32768 workers; more are refused."""
import pytest

from transformer_gqa_attention_gb300 import _build, abi


@pytest.fixture(scope="module", autouse=True)
def _built():
    _build.build()


@pytest.mark.parametrize("lens,units,workers", [([1048576] * 2, 3, 32768), ([1000000, 0, 77, 900000], 2, 30011),
                                                ([100000] * 11, 4, 32767)])
def test_every_tile_is_taken_once_in_order(lens, units, workers):
    pieces = abi.attn_debug_cache_schedule(lens, 0, 1048576, units, 2, workers)
    tiles = [max(1, -(-n // 128)) for n in lens]
    want = iter([(b, u) for b in range(len(lens)) for u in range(units)])
    at, unit = 0, next(want)
    worker = -1
    for c, b, u, first, n, *_ in pieces:
        if at == tiles[unit[0]]:
            at, unit = 0, next(want)
        assert (b, u, first) == (*unit, at) and n > 0 and worker <= c < workers
        at, worker = at + n, c
    assert at == tiles[unit[0]] and next(want, None) is None


@pytest.mark.parametrize("workers", [32769, 100000, 2 ** 31 - 1])
def test_more_workers_are_refused(workers):
    with pytest.raises(abi.GQAError) as err:
        abi.attn_debug_cache_schedule([1048576] * 40, 0, 1048576, 8, 2, workers)
    assert err.value.status == 1
