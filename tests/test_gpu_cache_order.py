"""Order between the warps of the cache attention kernels (GPU): workers with many tiles whose
maximum stays, so that nothing but the hand-over of a tile separates its readers from the next
tile's writers; and tiles of drafted positions that every row sees, none of whose values is cleared
before CTA 0 of a pair is told that the other's half is there.  Results are held to float64 and to the
same bits from call to call."""
import numpy as np
import pytest
import torch

from oracle import cache_oracle as co
from tests import gpu_util as gu
from transformer_gqa_attention_gb300 import abi

pytestmark = pytest.mark.gpu
DEV = gu.DEV
CALLS = 12


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from transformer_gqa_attention_gb300 import _build
    _build.build()


@pytest.fixture(scope="module")
def ctx():
    def zeros(*shape):
        return torch.zeros(*shape, dtype=torch.bfloat16, device=DEV)
    c = abi.attn_create(zeros(4096, 4096), zeros(1024, 4096), zeros(1024, 4096), zeros(4096, 4096))
    abi.attn_sync_status(c)
    yield c
    abi.attn_destroy(c)


def draw(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16)


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def check_h(got, ref, av, mag):
    """One rounding of the result to bf16 (2^-8 of it), one of each weight to bf16 (2^-8 of the mean of
    |v|), and scores of 128 products added in fp32."""
    d = 2 * 2.0 ** -17 * mag / 128 ** 0.5 + 2.0 ** -20
    tol = 2.0 ** -8 * np.abs(ref) + (1 + 2.0 ** -8) * (2.0 ** -8 + d) * av + 1e-30
    assert np.isfinite(got).all()
    assert (np.abs(got - ref) / tol).max() <= 1
    return d


@pytest.mark.parametrize("B,length", [(16, 2000), (40, 1500)])
def test_counted_decode_of_many_tiles_whose_maximum_stays(ctx, B, length):
    S = length + 9
    k, v, q = draw(1, B, S, 8, 128), draw(2, B, S, 8, 128), draw(3, B, 4096)
    k[:, :128] *= 2  # the first tile has the largest scores
    lens = [length - 61 * (b % 5) for b in range(B)]
    kd, vd, qd = k.to(DEV), v.to(DEV), q.to(DEV)
    w = torch.zeros(CALLS, B, 8, S, device=DEV)
    h = torch.full((CALLS, B, 4096), float("nan"), dtype=torch.bfloat16, device=DEV)
    for i in range(CALLS):
        abi.attn_decode_attention_weights(ctx, qd, kd, vd, B, S, ints(lens), w[i], h[i])
    abi.attn_sync_status(ctx)
    for i in range(1, CALLS):
        assert torch.equal(h[i].view(torch.int16), h[0].view(torch.int16)), i
        assert torch.equal(w[i].view(torch.int32), w[0].view(torch.int32)), i
    some = [0, B // 2, B - 1]
    ref, av, wr, mag = co.cache_attention(gu.np64(q[some]).reshape(3, 1, 8, 4, 128), gu.np64(k[some]),
                                          gu.np64(v[some]), [lens[b] for b in some])
    d = check_h(gu.np64(h[0, some]).reshape(ref.shape), ref, av, mag)
    # a weight: its score's error and a handful of fp32 roundings of sums of positive numbers
    assert (np.abs(gu.np64(w[0, some]) - wr) <= (d + 2.0 ** -20) * wr + 1e-30).all()


@pytest.mark.parametrize("T,lens", [(40, [88, 216, 1112]), (64, [64, 0, 192, 4032]), (128, [0, 128, 896]),
                                    (200, [56, 312]), (256, [0, 128, 2048])])
def test_tree_of_a_pair_whose_last_tiles_are_seen_by_every_row(ctx, T, lens):
    B, S = len(lens), max(lens) + T
    assert any((n + T) % 128 == 0 for n in lens)
    k, v, q = draw(4, B, S, 8, 128), draw(5, B, S, 8, 128), draw(6, B, T, 4096)
    vis = np.ones((B, T, T), dtype=bool)
    mask = torch.from_numpy(co.mask_words(vis)).to(DEV)
    kd, vd, qd = k.to(DEV), v.to(DEV), q.to(DEV)
    h = torch.full((CALLS, B, T, 4096), float("nan"), dtype=torch.bfloat16, device=DEV)
    for i in range(CALLS):
        abi.attn_tree_attention(ctx, qd, B, T, mask, kd, vd, S, ints(lens), h[i])
    abi.attn_sync_status(ctx)
    for i in range(1, CALLS):
        assert torch.equal(h[i].view(torch.int16), h[0].view(torch.int16)), i
    ref, av, _, mag = co.cache_attention(gu.np64(q).reshape(B, T, 8, 4, 128), gu.np64(k), gu.np64(v), lens, vis, T)
    check_h(gu.np64(h[0]).reshape(ref.shape), ref, av, mag)
