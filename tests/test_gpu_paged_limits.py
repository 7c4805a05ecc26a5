"""GPU checks of the paged-cache operators at the ends of their ranges: scores of any size, scales at
both ends of fp32, maxima that rise or stand alone, sums of very small weights, descriptions and
outputs that overlap."""
import math

import numpy as np
import pytest
import torch

from oracle import paged_oracle as po
from tests import gpu_util as gu
from tests.test_gpu_paged import Cache, attend, check, context, ints, query, reported, scrub, tables
from transformer_gqa_attention_gb300 import abi

pytestmark = pytest.mark.gpu
DEV = gu.DEV
NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from transformer_gqa_attention_gb300 import _build
    _build.build()


def code_of(x):
    """e4m3 codes of numbers that e4m3 holds exactly."""
    v = po.e4m3_values()
    x = np.asarray(x, dtype=np.float64)
    at = np.argsort(np.where(np.isnan(v), np.inf, v), kind="stable")[:254]
    i = at[np.searchsorted(v[at], x)]
    assert np.array_equal(v[i], x)
    return i.astype(np.uint8)


def put(c, i, pages, x):
    """Positions 0 .. n - 1 of a sequence: x [n, n_kv, 128], exact in the pool's type."""
    at = np.arange(len(x))
    idx = torch.from_numpy(np.asarray(pages)[at // c.page].astype(np.int64)), torch.from_numpy(at % c.page)
    rows = torch.from_numpy(code_of(x)) if c.e4m3 else torch.from_numpy(x).to(torch.bfloat16).view(torch.int16)
    c.raw(i)[idx] = rows.to(DEV)


# Queries 2^power times whole numbers up to 3 against keys of such numbers: products and sums of them are
# whole numbers below 2^11 times 2^power, exact in fp32, and two scores that differ do so by 2^power / sqrt(128)
# at least, so that from 2^13 on the weights are equal shares of the keys with the largest score and nothing
# (e^-700) of the others.  Shares add up exactly; the sum of values rounds with 2^-24 of it for each term that is not
# zero (at most 200 in these draws: 2^-16 together), the quotient and the scale with 2^-22, and h once with 2^-8.
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("power", [13, 22, 25, 30, 36, 60, 100])
@pytest.mark.parametrize("lens", [[1, 17, 300], [20000]])
def test_scores_of_any_size(lens, power, e4m3):
    n_kv = 2
    n_pages = sum(-(-n // 32) for n in lens)
    c = Cache(n_pages, 32, n_kv, e4m3, seed=power)
    for s in c.scales if e4m3 else ():
        s.fill_(0.5)
    t = tables(lens, 32, n_pages, seed=power)
    rng = np.random.default_rng(power + len(lens))
    keys = [rng.integers(-3, 4, (n, n_kv, 128)).astype(np.float64) for n in lens]
    qs = rng.integers(-3, 4, (len(lens), n_kv, 4, 128)).astype(np.float64)
    keys[-1][:, 0] = np.where(qs[-1, 0, 0] >= 0, -np.abs(keys[-1][:, 0]) - (keys[-1][:, 0] == 0),
                              np.abs(keys[-1][:, 0]))  # one head whose scores are all negative
    for b, k in enumerate(keys):
        put(c, 0, t[b], k)
    scrub(c, t, lens)
    q = torch.from_numpy(qs * 2.0 ** power).reshape(len(lens), -1).to(torch.bfloat16).to(DEV)
    h = attend(c, q, t, lens)
    assert not reported(c.ctx)
    vn = c.numbers(1)
    for b, n in enumerate(lens):
        got = gu.np64(h[b]).reshape(n_kv, 4, 128)
        v = po.gather(vn, t[b], n)
        e = np.einsum("ghd,sgd->ghs", qs[b], keys[b])
        a = (e == e.max(-1, keepdims=True)).astype(np.float64)
        assert a.sum(-1).max() <= 200
        a /= a.sum(-1, keepdims=True)
        ref, mean = np.einsum("ghs,sgd->ghd", a, v), np.einsum("ghs,sgd->ghd", a, np.abs(v))
        assert np.all(np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -15 * mean), (b, n)


@pytest.mark.parametrize("broken", [NAN, math.inf, -0.01])
def test_a_broken_key_scale_shows(broken):
    c = Cache(8, 32, 4, True, seed=30)
    t, lens = np.arange(8, dtype=np.int32).reshape(2, 4), [100, 128]
    scrub(c, t, lens)
    c.scales[0][1] = broken
    h = attend(c, query(2, 4), t, lens)
    assert not reported(c.ctx)
    odd = torch.isnan(h[:2]).cpu().view(2, 4, 512)
    assert odd[:, 1].all() and not odd[:, [0, 2, 3]].any()


@pytest.mark.parametrize("scale", [NAN, math.inf, -0.01, 0.0])
def test_an_empty_sequence_is_zero_whatever_the_scales(scale):
    c = Cache(8, 32, 4, True, seed=33)
    t, lens = np.arange(8, dtype=np.int32).reshape(2, 4), [0, 60]
    scrub(c, t, lens)
    for s in c.scales:
        s[2] = scale
    q = query(2, 4)
    h = attend(c, q, t, lens)
    assert not reported(c.ctx)
    assert (h[0] == 0).all()
    assert torch.isfinite(h[1].view(4, 512)[[0, 1, 3]]).all()


def test_keys_of_zeros_under_scales_that_overflow():
    """Scores of exactly 0 where query times scale passes fp32: the mean of the values."""
    c = Cache(8, 32, 2, True, seed=31)
    t, lens = np.arange(8, dtype=np.int32).reshape(2, 4), [100, 37]
    c.raw(0).zero_()
    scrub(c, t, lens)
    c.scales[0].fill_(1e30)
    h = attend(c, query(2, 2, size=1e30), t, lens)
    assert not reported(c.ctx)
    check(c, query(2, 2, size=0.0), t, lens, h)


def test_values_of_tiny_scales():
    c = Cache(80, 64, 2, True, seed=32)
    lens = [5000, 37]
    t = tables(lens, 64, 80)
    scrub(c, t, lens)
    q = query(2, 2)
    for scale in (1e-30, 1e-34, 1e-36, 2.0 ** -126):
        c.scales[1].fill_(scale)
        h = attend(c, q, t, lens)
        assert not reported(c.ctx)
        vn = c.numbers(1)
        for b, n in enumerate(lens):
            ref, mean, mag = po.decode(gu.np64(q[b]).reshape(2, 4, 128), po.gather(c.numbers(0), t[b], n), po.gather(vn, t[b], n))
            d = 2 * 2.0 ** -17 * 1.02 * mag / math.sqrt(128) + 2.0 ** -20
            # 2^-134: half of bf16's smallest step
            tol = 2.0 ** -8 * np.abs(ref) + (1 + 2.0 ** -8) * (2.0 ** -11 + d) * mean + 2.0 ** -133
            assert np.all(np.abs(gu.np64(h[b]).reshape(2, 4, 128) - ref) <= tol), (scale, b)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("n_pages,page,n_kv,order,gaps", [
    (3, 8, 2, (2, 0, 1), (0, 0, 0)), (3, 8, 2, (0, 2, 1), (0, 128, 0)), (3, 8, 2, (1, 0, 2), (64, 0, 256)),
    (1, 8, 2, (0, 1, 2), (0, 256, 0)), (2, 16, 1, (1, 2, 0), (128, 0, 16)), (4, 8, 3, (0, 1, 2), (128, 0, 384))])
def test_keys_and_values_that_overlap_are_refused(n_pages, page, n_kv, order, gaps, e4m3):
    """Every distance of the two pools against their rows' elements one by one (host only).  order: extents (pages, slots,
    heads) from the narrowest stride on, with `gaps` elements left behind each of them."""
    extent, stride, at = (n_pages, page, n_kv), [0, 0, 0], 128
    for i, gap in zip(order, gaps):
        stride[i] = at + gap
        at = stride[i] * extent[i]
    grid = [np.arange(n) * s for n, s in zip(extent, stride)]
    rows = (grid[0][:, None, None] + grid[1][:, None] + grid[2]).reshape(-1)
    held = np.zeros(3 * at + 1024, dtype=bool)
    held[(rows[:, None] + np.arange(128)).reshape(-1) + at + 512] = True
    size = 1 if e4m3 else 2
    memory = torch.zeros((3 * at + 1024) * size, dtype=torch.uint8, device=DEV)
    base = memory.data_ptr() + (at + 512) * size
    ctx, answers = context(n_kv), set()
    for d in range(-at - 256, at + 256, 16):
        meets = bool(held[rows + at + 512 + d].any() or held[rows + at + 512 + d + 127].any())
        try:
            abi.attn_paged_destroy(abi.attn_paged_create(ctx, base, base + d * size, n_pages, page, "e4m3" if e4m3 else "bf16", *stride))
            got = 0
        except abi.GQAError as e:
            got = e.status
        assert got == (1 if meets else 0), d
        answers.add(got)
    assert answers == {0, 1}


@pytest.mark.parametrize("e4m3,beside", [(False, True), (True, True), (False, False)])
def test_heads_over_the_pools_are_refused(e4m3, beside):
    """The output between pages of a pool with room between them, and on each row and scale of it."""
    n_pages, page, n_kv, B = 3, 8, 2, 1
    size, row, bytes_h = (1, 128, 2048) if e4m3 else (2, 256, 2048)
    rows = page * n_kv * row                               # of a page's keys
    room = 2 * rows + 3 * bytes_h                          # from page to page, where keys and values lie side by side
    memory = torch.zeros(bytes_h + n_pages * room, dtype=torch.uint8, device=DEV)
    k = memory.data_ptr() + bytes_h
    v = k + (rows if beside else n_pages * rows)
    strides = ((room if beside else rows) // size, n_kv * 128, 128)
    scales = [torch.ones(512, device=DEV) for _ in range(2)] if e4m3 else [None, None]
    ctx = context(n_kv)
    p = abi.attn_paged_create(ctx, k, v, n_pages, page, "e4m3" if e4m3 else "bf16", *strides, *scales)
    q = torch.zeros(B, n_kv * 512, dtype=torch.bfloat16, device=DEV)
    t, lens = ints([[0, 1, 2]]), ints([20])

    def status(h):
        try:
            abi.attn_paged_decode_attention(ctx, p, q, B, t, 3, lens, h)
            return 0
        except abi.GQAError as e:
            return e.status
    held = np.zeros(len(memory), dtype=bool)
    for first in (k, v):
        for n in range(n_pages):
            at = first - memory.data_ptr() + n * strides[0] * size
            held[at:at + rows] = True
    free = 0
    for at in range(0, len(memory) - bytes_h + 1, 16 if beside else 256):
        want = 1 if held[at:at + bytes_h].any() else 0
        assert status(memory.data_ptr() + at) == want, at
        free += want == 0
    assert free
    for s in scales if e4m3 else ():
        assert status(s) == 1 and status(s.data_ptr() - 2032) == 1
    abi.attn_paged_destroy(p)
    abi.attn_sync_status(ctx)


# ------------------------------------------------------------------------------- weights of every size
def held(c, t, b, n):
    return [po.gather(c.numbers(i), t[b], n) for i in range(2)]


def check_weights(c, q, k, v, h):
    """One sequence.  As `check` of the paged operators, but with e4m3 pages the weights enter the product as fp16
    of 2^15 times them: 2^-11 of the value at most, and 2^-40 of the largest weight for those below 2^-29 of it."""
    ref, mean, mag = po.decode(gu.np64(q).reshape(c.n_kv, 4, 128), k, v)
    w = 2.0 ** -11 if c.e4m3 else 2.0 ** -8
    d = 2 * 2.0 ** -17 * 1.02 * mag / math.sqrt(128) + 2.0 ** -20
    small = len(k) * 2.0 ** -40 * np.abs(v).max() if c.e4m3 else 0.0
    got = gu.np64(h).reshape(c.n_kv, 4, 128)
    assert np.all(np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + (1 + 2.0 ** -8) * (w + d) * mean + small)
    return ref


@pytest.mark.parametrize("lens", [[1, 90, 700], [9000], [(b * 977) % 3000 for b in range(24)]])
def test_e4m3_weights_keep_eleven_bits(lens):
    n_pages = sum(-(-n // 32) for n in lens) + 2
    c = Cache(n_pages, 32, 4, True, seed=40)
    t = tables(lens, 32, n_pages, seed=40)
    scrub(c, t, lens)
    q = query(len(lens), 4)
    h = attend(c, q, t, lens)
    assert not reported(c.ctx)
    for b, n in enumerate(lens):
        if n:
            check_weights(c, q[b], *held(c, t, b, n), h[b])


@pytest.mark.parametrize("n", [640, 5120])
@pytest.mark.parametrize("falling", [False, True])
@pytest.mark.parametrize("e4m3", [False, True])
def test_scores_that_rise_or_fall_with_the_position(e4m3, falling, n):
    """Key s a multiple of the queries that grows (shrinks) with s up to a score near 40: a new maximum in every stage."""
    c = Cache(n // 64, 64, 1, e4m3, seed=41)
    if e4m3:
        c.scales[0].fill_(0.2)
    t = np.random.default_rng(n).permutation(n // 64).astype(np.int32)[None]
    q = query(1, 1)
    q[0] = q[0, :128].repeat(4)
    ramp = np.linspace(1.0, 0.0, n) if falling else np.linspace(0.0, 1.0, n)
    k = torch.from_numpy(ramp[:, None] * gu.np64(q[0, :128]) * (8.0 if e4m3 else 1.6))
    rows = k.to(torch.float8_e4m3fn).view(torch.uint8) if e4m3 else k.to(torch.bfloat16).view(torch.int16)
    at = np.arange(n)
    c.raw(0)[torch.from_numpy(t[0, at // 64].astype(np.int64)), torch.from_numpy(at % 64)] = rows[:, None].to(DEV)
    h = attend(c, q, t, [n])
    assert not reported(c.ctx)
    check_weights(c, q[0], *held(c, t, 0, n), h[0])


@pytest.mark.parametrize("at", [2, 3000, -1])
@pytest.mark.parametrize("e4m3", [False, True])
def test_one_key_far_above_the_others(e4m3, at):
    """In the first tile, in the middle and as the last key: nearly all of the weight of one head."""
    n, n_kv = 5000, 2
    c = Cache(80, 64, n_kv, e4m3, seed=42)
    if e4m3:
        c.scales[0].fill_(0.1)
    t = np.random.default_rng(42).permutation(80).astype(np.int32)[None]
    rng = np.random.default_rng(43)
    q = query(1, n_kv)
    k = rng.integers(-3, 4, (n, n_kv, 128)).astype(np.float64)
    q0 = gu.np64(q[0]).reshape(n_kv, 4, 128)[:, 0]
    k[at] = np.clip(np.round(q0), -6, 6) * 8
    if not e4m3:
        k = k / 8
    put(c, 0, t[0], k)
    scrub(c, t, [n])
    h = attend(c, q, t, [n])
    assert not reported(c.ctx)
    kn, vn = held(c, t, 0, n)
    ref = check_weights(c, q[0], kn, vn, h[0])
    assert np.abs(ref[:, 0] - vn[at]).max() < 0.05 * np.abs(vn).max()


def test_many_small_weights_beside_a_large_one():
    """400000 e4m3 keys of 2^-26 of the largest weight, whose values alone make the result."""
    n, page = 400001, 64
    n_pages = -(-n // page)
    c = Cache(n_pages, page, 1, True, seed=44)
    t = np.random.default_rng(44).permutation(n_pages).astype(np.int32)[None]
    c.raw(0).zero_()
    c.raw(1).fill_(int(code_of([1.0])[0]))
    c.scales[0].fill_(1.0)
    c.scales[1].fill_(1.0)
    q = torch.zeros(1, 512, dtype=torch.bfloat16, device=DEV)
    q[0, ::128] = 26 * math.log(2.0) * math.sqrt(128.0) / 448
    first = int(t[0, 0])
    c.raw(0)[first, 0, 0, 0] = int(code_of([448.0])[0])
    c.raw(1)[first, 0] = 0
    h = attend(c, q, t, [n])
    assert not reported(c.ctx)
    e = float(q[0, 0]) * 448 / math.sqrt(128.0)
    ref = (n - 1) / (n - 1 + math.exp(e))
    assert 0.004 < ref < 0.008
    # sums of n equal terms in fp32 in at most 32 parts a CTA: 2^-24 of them for each of the 100 terms of a lane in a row
    # of tiles, under 2^-12 in all; the score 26 to 2^-20; the weights 2^-11; h 2^-8
    assert np.all(np.abs(gu.np64(h[0]) - ref) <= (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -12 + 2.0 ** -15) * ref)
