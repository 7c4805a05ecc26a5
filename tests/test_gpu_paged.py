"""GPU checks of the rotation by position and of the paged-cache operators against their float64
definitions.

Tolerances.  A rotated value is gain (a cos - b sin) in fp32, rounded once to bf16 (half a step,
2^-8 of the value).  Its angle is off by at most pi 2^-25 (nearest fp32 to half a revolution's
fraction), pi 2^-31 (bits of it that are dropped) and position x frequency x 2^-51 (at a million: 2^-31); sine and
cosine by 2 units of 2^-24; the factor, the products and the sum round with 2^-24 each:
less than 8 units of 2^-24 = 2^-21 of gain (|a| + |b|) together.
e4m3: half a step, 2^-4 of the value (or 2^-10, half the smallest step), the value off by two more
roundings, of the scale's reciprocal and the product, 2^-23.
h: with a the exact weights, the weights enter the product as bf16 (2^-8 of the value at most), the
scores are off by at most 128 * 2^-24 * sum|q_i k_i| (fp32 sums of 128 exact products, scaled keys another
2^-23 of it) and the exponentials by 2^-22, and h is rounded to bf16 once:
    |h - ref| <= 2^-8 |ref| + (1 + 2^-8)(2^-8 + d) sum a|v|,  d = 2 * 2^-17 * 1.02 sum|q_i k_i| / sqrt(128) + 2^-20
(the factor 2: numerator and denominator)."""
import math

import numpy as np
import pytest
import torch

from oracle import paged_oracle as po
from tests import gpu_util as gu
from transformer_gqa_attention_gb300 import abi

pytestmark = pytest.mark.gpu
DEV = gu.DEV
NAN = float("nan")
THETA = 500000.0
MORE = {"plain": {}, "linear": dict(factor=4.0), "bands": dict(factor=8.0, low=1.0, high=4.0, context=8192.0),
        "ramp": dict(factor=16.0, low=1.0, high=32.0, context=4096.0)}
SHAPE_STATUS = 2


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from transformer_gqa_attention_gb300 import _build
    _build.build()


_ctx = {}


def context(n_kv=8):
    """A context over zero weights (these operators do not use them)."""
    if n_kv not in _ctx:
        z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device=DEV)  # noqa: E731
        _ctx[n_kv] = abi.attn_create_shard(z(512 * n_kv, 4096), z(128 * n_kv, 4096), z(128 * n_kv, 4096),
                                           z(4096, 512 * n_kv), n_kv)
        abi.attn_sync_status(_ctx[n_kv])
    return _ctx[n_kv]


def ints(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device=DEV)


def reported(ctx):
    """Whether a value of some earlier call was out of range."""
    try:
        abi.attn_sync_status(ctx)
        return False
    except abi.GQAError as e:
        assert e.status == SHAPE_STATUS
        return True


def turn(layout="pairs", rot=128, scaling="plain"):
    return (abi.attn_rope_init(layout, rot, THETA, scaling, **MORE[scaling]),
            *po.frequencies(rot, THETA, scaling, **MORE[scaling]))


# ------------------------------------------------------------------------------- rotations
POSITIONS = [0, 1, 2, 63, 4095, 131071, 999999, -1, -70000]


@pytest.mark.parametrize("heads", [1, 3, 8, 32, 41])
@pytest.mark.parametrize("layout,rot,scaling", [("pairs", 128, "plain"), ("halves", 128, "bands"), ("pairs", 64, "ramp"),
                                                ("halves", 96, "linear"), ("pairs", 16, "plain"),
                                                ("halves", 16, "ramp"), ("halves", 112, "plain")])
def test_rotation(layout, rot, scaling, heads):
    rope, w, gain = turn(layout, rot, scaling)
    rng = np.random.default_rng(heads + rot)
    for n in (1, 9, 333):
        pos = np.concatenate([POSITIONS, rng.integers(-1000000, 1000000, 333)])[:n]
        wide = heads * 128 + 8 * (n % 3)
        x = torch.from_numpy(rng.standard_normal((n, wide))).to(torch.bfloat16).to(DEV)
        out = torch.full((n, heads * 128 + 16), NAN, dtype=torch.bfloat16, device=DEV)
        before = x.clone()
        abi.attn_rope_apply(context(), rope, x, n, heads, wide, ints(pos), out, out.shape[1])
        abi.attn_sync_status(context())
        assert torch.equal(x, before) and out[:, heads * 128:].isnan().all()
        ref, size = po.rotate(gu.np64(x[:, :heads * 128]).reshape(n, heads, 128), pos, layout, w, gain)
        got = gu.np64(out[:, :heads * 128]).reshape(n, heads, 128)
        tol = 2.0 ** -8 * np.abs(ref) + 2.0 ** -21 * gain * size
        assert np.all(np.abs(got - ref) <= tol)
        assert np.array_equal(got[..., rot:], ref[..., rot:])
        abi.attn_rope_apply(context(), rope, x, n, heads, wide, ints(pos), x, wide)  # in place
        abi.attn_sync_status(context())
        assert torch.equal(x[:, :heads * 128], out[:, :heads * 128]) and torch.equal(x[:, heads * 128:], before[:, heads * 128:])


def test_rotation_passes_infinities_and_nans_on():
    rope, _, _ = turn("pairs", 64)
    x = torch.ones(2, 128, dtype=torch.bfloat16, device=DEV)
    x[0, 2], x[0, 70], x[1, 100] = math.inf, math.inf, NAN
    out = torch.empty_like(x)
    abi.attn_rope_apply(context(), rope, x, 2, 1, 128, ints([5, 6]), out, 128)
    abi.attn_sync_status(context())
    odd = ~torch.isfinite(out).cpu()
    want = torch.zeros(2, 128, dtype=torch.bool)
    want[0, 2] = want[0, 3] = want[0, 70] = want[1, 100] = True
    assert torch.equal(odd, want)


@pytest.mark.parametrize("rot,scaling", [(128, "plain"), (128, "bands"), (64, "ramp"), (16, "linear")])
def test_table(rot, scaling):
    rope, w, gain = turn("pairs", rot, scaling)
    rng = np.random.default_rng(rot)
    for n in (1, 5, 1000):
        pos = np.concatenate([POSITIONS, rng.integers(-1000000, 1000000, 1000)])[:n]
        R = torch.full((n + 1, 64, 2), NAN, device=DEV)
        abi.attn_rope_table(context(), rope, ints(pos), n, R)
        abi.attn_sync_status(context())
        ang = np.asarray(pos, dtype=np.float64)[:, None] * w
        ref = np.zeros((n, 64, 2))
        ref[..., 0] = 1.0
        ref[:, :rot // 2] = np.stack([np.cos(ang), np.sin(ang)], -1) * gain
        assert np.all(np.abs(gu.np64(R[:n]) - ref) <= 2.0 ** -21 * gain)
        assert torch.isnan(R[n]).all()


# ------------------------------------------------------------------------------- pools
class Cache:
    """Two pools, their description, and what they hold as float64 [page, slot, head, 128]."""

    def __init__(self, n_pages, page, n_kv, e4m3, heads_first=False, beside=False, seed=0, fill="normal"):
        rng = np.random.default_rng(seed)
        self.n_pages, self.page, self.n_kv, self.e4m3, self.heads_first = n_pages, page, n_kv, e4m3, heads_first
        mid = (n_kv, page) if heads_first else (page, n_kv)
        shape = (n_pages, 2, *mid, 128) if beside else (2, n_pages, *mid, 128)
        if e4m3:
            both = torch.from_numpy(rng.integers(0, 256, shape).astype(np.uint8)).to(DEV)
            if fill != "any":
                both[(both & 127) == 127] = 0x38  # no NaN
        else:
            both = torch.from_numpy(rng.standard_normal(shape)).to(torch.bfloat16).to(DEV)
        if fill == "nan":
            both.fill_(0x7F if e4m3 else NAN)
        self.k, self.v = (both[:, 0], both[:, 1]) if beside else (both[0], both[1])
        scale = lambda: torch.from_numpy(rng.uniform(0.002, 0.02, 8).astype(np.float32)).to(DEV)  # noqa: E731
        self.scales = (scale(), scale()) if e4m3 else (None, None)
        st = self.k.stride()
        self.strides = (st[0], st[2], st[1]) if heads_first else (st[0], st[1], st[2])
        self.ctx = context(n_kv)
        self.p = abi.attn_paged_create(self.ctx, self.k, self.v, n_pages, page, "e4m3" if e4m3 else "bf16",
                                       *self.strides, *self.scales)

    def __del__(self):
        abi.attn_paged_destroy(getattr(self, "p", None))

    def raw(self, c):
        """A pool's bits [page, slot, head, 128]."""
        t = (self.k, self.v)[c]
        t = t if self.e4m3 else t.view(torch.int16)
        return (t.transpose(1, 2) if self.heads_first else t)

    def codes(self, c):
        """Its numbers, before the scale."""
        bits = self.raw(c).contiguous().cpu()
        return po.e4m3_values()[bits.numpy()] if self.e4m3 else bits.view(torch.bfloat16).double().numpy()

    def numbers(self, c):
        x = self.codes(c)
        return x * gu.np64(self.scales[c][:self.n_kv])[:, None] if self.e4m3 else x


def tables(lens, page, n_pages, seed=0, room=1):
    """Pages of each sequence, no two the same, -7 behind the last."""
    rng = np.random.default_rng(seed)
    need = [-(-n // page) for n in lens]
    t = np.full((len(lens), max(1, max(need)) + room), -7, dtype=np.int32)
    order, at = rng.permutation(n_pages), 0
    for b, k in enumerate(need):
        t[b, :k] = order[at:at + k]
        at += k
    assert at <= n_pages
    return t


# ------------------------------------------------------------------------------- append
@pytest.mark.parametrize("n_kv", [1, 2, 3, 5, 8])
@pytest.mark.parametrize("page,heads_first,beside", [(8, False, False), (24, True, False), (64, False, True),
                                                     (256, True, True)])
@pytest.mark.parametrize("e4m3,layout,rot,scaling", [(False, "pairs", 128, "plain"), (True, "halves", 128, "bands"),
                                                     (False, "halves", 48, "ramp"), (True, None, 0, None)])
def test_append(e4m3, layout, rot, scaling, page, heads_first, beside, n_kv):
    lens, new, T = [0, 1, page - 1, page, 2 * page + 3, 5, 0], [9, 1, 1, 0, 8, 9, 3], 9
    c = Cache(40, page, n_kv, e4m3, heads_first, beside, seed=page)
    t = tables([a + n for a, n in zip(lens, new)], page, 40)
    t[3, :] = -7  # nothing new: its pages are not looked at
    rng = np.random.default_rng(n_kv)
    rows = torch.from_numpy(rng.standard_normal((len(lens), T, 2 * n_kv * 128 + 8))).to(torch.bfloat16).to(DEV)
    k, v = rows[:, :, 8:8 + n_kv * 128], rows[:, :, 8 + n_kv * 128:]
    for b, n in enumerate(new):
        rows[b, n:] = NAN
    want = [c.raw(0).clone(), c.raw(1).clone()]
    first = ints([70000 + b for b in range(len(lens))]) if scaling == "bands" else None
    rope, w, gain = turn(layout, rot, scaling) if layout else (None, np.zeros(0), 1.0)
    abi.attn_paged_append(c.ctx, c.p, k, v, len(lens), T, rows.stride(0), rows.stride(1), rope, first, ints(t), t.shape[1],
                          ints(lens), ints(new))
    assert not reported(c.ctx)
    got = [c.codes(0), c.codes(1)]
    for b, (a, n) in enumerate(zip(lens, new)):
        at = np.arange(a, a + n)
        pages, slots = t[b, at // page], at % page
        start = a if first is None else 70000 + b
        kr, size = po.rotate(gu.np64(k[b, :n]).reshape(n, n_kv, 128), start + np.arange(n), layout or "pairs", w, gain)
        for i, (ref, s) in enumerate(((kr, size), (gu.np64(v[b, :n]).reshape(n, n_kv, 128), 0.0))):
            x = got[i][pages, slots]
            off = 2.0 ** -21 * gain * s
            if e4m3:
                sc = gu.np64(c.scales[i][:n_kv])[:, None]
                ref, off = ref / sc, off / sc
                off = off + 2.0 ** -23 * np.abs(ref)
                top = np.minimum(np.abs(ref), po.E4M3_TOP)
                step = np.maximum(2.0 ** -4 * (top + off), 2.0 ** -10)
                ref = np.clip(ref, -po.E4M3_TOP, po.E4M3_TOP)
            else:
                step = 2.0 ** -8 * np.abs(ref)
            assert np.all(np.abs(x - ref) <= step + off)
            if not layout and not e4m3:
                assert np.array_equal(x, ref)
        for i in range(2):  # the rest stays as it was
            want[i][torch.from_numpy(pages.astype(np.int64)), torch.from_numpy(slots)] = \
                c.raw(i)[torch.from_numpy(pages.astype(np.int64)), torch.from_numpy(slots)]
    assert torch.equal(want[0], c.raw(0)) and torch.equal(want[1], c.raw(1))


def test_append_of_whole_rows_and_of_a_dense_cache():
    """T for every sequence, dense [B, S, n_kv, 128] sources, one token and one sequence with any stride."""
    c = Cache(64, 16, 8, False, fill="nan")
    for B, T, S in ((3, 40, 64), (1, 70, 70), (5, 1, 9), (1, 1, 1)):
        dense = torch.randn(2, B, S, 8, 128, device=DEV).to(torch.bfloat16)
        lens = [7 * b for b in range(B)]
        t = tables([n + T for n in lens], 16, 64, seed=T)
        abi.attn_paged_append(c.ctx, c.p, dense[0], dense[1], B, T, dense.stride(1) if B > 1 else -5,
                              1024 if T > 1 else 3, None, None, ints(t), t.shape[1], ints(lens))
        assert not reported(c.ctx)
        for b, n in enumerate(lens):
            at = np.arange(n, n + T)
            idx = torch.from_numpy(t[b, at // 16].astype(np.int64)), torch.from_numpy(at % 16)
            assert torch.equal(c.k[idx], dense[0, b, :T]) and torch.equal(c.v[idx], dense[1, b, :T])


def test_append_rounds_e4m3_at_its_ends():
    c = Cache(2, 8, 1, True)
    vals = [0.0, -0.0, 448.0, 449.0, 470.0, 1e6, -1e6, math.inf, -math.inf, NAN, 2.0 ** -9, 2.0 ** -10, 1.5 * 2.0 ** -10,
            -2.0 ** -6, 17.0, 19.0]
    k = torch.zeros(1, 1, 128, dtype=torch.bfloat16, device=DEV)
    k[0, 0, :len(vals)] = torch.tensor(vals, device=DEV)
    for s in c.scales:
        s.fill_(0.25)
    abi.attn_paged_append(c.ctx, c.p, (k * 0.25).contiguous(), k, 1, 1, 0, 0, None, None, ints([[1]]), 1, ints([3]))
    assert not reported(c.ctx)
    got = c.codes(0)[1, 3, 0, :len(vals)]
    # 449 is 448 in bf16; halfway cases go to the even neighbour
    want = [0, 0, 448, 448, 448, 448, -448, 448, -448, NAN, 2.0 ** -9, 0, 2.0 ** -9, -2.0 ** -6, 16, 20]
    assert np.array_equal(got, np.array(want), equal_nan=True)
    assert np.array_equal(c.codes(1)[1, 3, 0, 2:9], [448, 448, 448, 448, -448, 448, -448])


def test_append_leaves_out_what_is_out_of_range():
    page, T = 16, 4
    lens = [3, -1, 45, 44, 5, 0, 14, 2 ** 31 - 1]
    new = [4, 2, 4, 4, 5, -1, 4, 1]
    ok = [4, 0, 0, 4, 0, 0, 2, 0]  # the seventh runs from a good page onto a bad one
    for bad in (-1, 40, 2 ** 31 - 1, -2 ** 31):
        c = Cache(40, page, 2, False, seed=3)
        t = np.arange(24, dtype=np.int32).reshape(8, 3)
        t[6, 1] = bad
        rows = torch.randn(2, 8, T, 256, device=DEV).to(torch.bfloat16)
        want = [c.k.clone(), c.v.clone()]
        for b, n in enumerate(ok):
            for s in range(lens[b], lens[b] + n):
                for i in range(2):
                    want[i][t[b, s // page], s % page] = rows[i, b, s - lens[b]].view(2, 128)
        abi.attn_paged_append(c.ctx, c.p, rows[0], rows[1], 8, T, 4 * 256, 256, None, None, ints(t), 3, ints(lens), ints(new))
        assert reported(c.ctx) and not reported(c.ctx)
        assert torch.equal(c.k, want[0]) and torch.equal(c.v, want[1])


# ------------------------------------------------------------------------------- attention
def attend(c, q, t, lens, stream=None):
    B = len(lens)
    h = torch.full((B + 1, c.n_kv * 512), NAN, dtype=torch.bfloat16, device=DEV)
    h[B] = 7.0
    abi.attn_paged_decode_attention(c.ctx, c.p, q, B, ints(t), t.shape[1], ints(lens), h, stream)
    return h


def check(c, q, t, lens, h, left_out=()):
    kn, vn = c.numbers(0), c.numbers(1)
    assert (h[len(lens)] == 7.0).all()
    for b, n in enumerate(lens):
        got = gu.np64(h[b]).reshape(c.n_kv, 4, 128)
        if b in left_out:
            assert np.isnan(got).all(), b
            continue
        ref, mean, mag = po.decode(gu.np64(q[b]).reshape(c.n_kv, 4, 128), po.gather(kn, t[b], n), po.gather(vn, t[b], n))
        d = 2 * 2.0 ** -17 * 1.02 * mag / math.sqrt(128) + 2.0 ** -20
        tol = 2.0 ** -8 * np.abs(ref) + (1 + 2.0 ** -8) * (2.0 ** -8 + d) * mean
        assert np.all(np.abs(got - ref) <= tol), (b, n, float(np.max(np.abs(got - ref) - tol)))


def query(B, n_kv, seed=0, size=1.5):
    rng = np.random.default_rng(seed + 99)
    return torch.from_numpy(rng.standard_normal((B, n_kv * 512)) * size).to(torch.bfloat16).to(DEV)


def scrub(c, t, lens):
    """NaN in every slot that no sequence holds."""
    held = torch.zeros(c.n_pages, c.page, dtype=torch.bool)
    for b, n in enumerate(lens):
        at = np.arange(n)
        held[torch.from_numpy(t[b, at // c.page].astype(np.int64)), torch.from_numpy(at % c.page)] = True
    for i in range(2):
        c.raw(i)[~held.to(DEV)] = 0x7F if c.e4m3 else 0x7FC0


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("n_kv", [1, 3, 8])
@pytest.mark.parametrize("page,heads_first,beside", [(8, False, False), (16, True, False), (24, False, True),
                                                     (32, True, True), (48, False, False), (64, False, False),
                                                     (128, True, False), (136, False, False), (512, False, False)])
def test_attention(page, heads_first, beside, n_kv, e4m3):
    lens = [0, 1, 7, page - 1, page, page + 1, 63, 64, 65, 127, 128, 129, 3 * page + 5, 700, 0, 1500]
    n_pages = sum(-(-n // page) for n in lens) + 2
    c = Cache(n_pages, page, n_kv, e4m3, heads_first, beside, seed=page + n_kv)
    t = tables(lens, page, n_pages, seed=n_kv)
    scrub(c, t, lens)
    q = query(len(lens), n_kv)
    h = attend(c, q, t, lens)
    assert not reported(c.ctx)
    check(c, q, t, lens, h)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("B,lens", [(1, [20000]), (2, [40000, 3]), (5, [0, 9000, 1, 0, 12345]), (40, None), (1, [1]), (1, [0])])
def test_attention_of_long_and_ragged_batches(B, lens, e4m3):
    lens = lens or [(b * 977) % 3000 for b in range(B)]
    n_pages = sum(-(-n // 32) for n in lens) + 2
    c = Cache(n_pages, 32, 8, e4m3, seed=B)
    t = tables(lens, 32, n_pages, seed=B)
    scrub(c, t, lens)
    q = query(B, 8)
    h = attend(c, q, t, lens)
    assert not reported(c.ctx)
    check(c, q, t, lens, h)
    for _ in range(3):  # the same bits every time
        again = attend(c, q, t, lens)
        assert torch.equal(h[:B].view(torch.int16), again[:B].view(torch.int16))


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("n_kv,lens", [(1, [2000]), (1, [2200]), (1, [4100]), (1, [8200]), (1, [8400]), (1, [20000]),
                                       (1, [39000, 900, 0, 17000]), (2, [30000]), (3, [19000, 40]), (4, [24000, 5000]),
                                       (8, [6000]), (7, [11000, 300])])
def test_units_of_many_pieces(n_kv, lens, e4m3):
    """Up to a piece for every CTA: joined at once, in groups of eight and of sixteen."""
    n_pages = sum(-(-n // 64) for n in lens) + 2
    c = Cache(n_pages, 64, n_kv, e4m3, seed=n_kv)
    t = tables(lens, 64, n_pages, seed=n_kv)
    scrub(c, t, lens)
    q = query(len(lens), n_kv, lens[0])
    h = attend(c, q, t, lens)
    assert not reported(c.ctx)
    check(c, q, t, lens, h)
    bits = h[:len(lens)].view(torch.int16).clone()
    for _ in range(20):
        assert torch.equal(attend(c, q, t, lens)[:len(lens)].view(torch.int16), bits)
    if lens[0] > 5000:  # a page that is out of range, in the middle
        bad = t.copy()
        bad[0, 40] = -1
        h = attend(c, q, bad, lens)
        assert reported(c.ctx)
        check(c, q, t, lens, h, left_out=(0,))


def test_attention_of_the_most_sequences():
    lens = [(b * 37) % 90 for b in range(1024)]
    n_pages = sum(-(-n // 16) for n in lens) + 2
    c = Cache(n_pages, 16, 2, False)
    t = tables(lens, 16, n_pages)
    scrub(c, t, lens)
    q = query(1024, 2)
    h = attend(c, q, t, lens)
    assert not reported(c.ctx)
    check(c, q, t, lens, h)


@pytest.mark.parametrize("order", [(2, 0, 1), (1, 0, 2), (1, 2, 0), (2, 1, 0)])
@pytest.mark.parametrize("e4m3", [False, True])
def test_pools_in_other_orders(order, e4m3):
    """Pages, slots and heads in any order in memory, with room between them: append, then attend."""
    n_pages, page, n_kv, B = 7, 24, 3, 3
    rng = np.random.default_rng(sum(order) + 4 * e4m3)
    kind = torch.uint8 if e4m3 else torch.bfloat16
    extent = (n_pages, page, n_kv)
    place = [extent[i] + (2 if i == order[1] else 0) for i in order]  # two more of the middle extent than are used
    c = Cache.__new__(Cache)
    c.n_pages, c.page, c.n_kv, c.e4m3, c.heads_first, c.ctx = n_pages, page, n_kv, e4m3, False, context(n_kv)
    whole = [torch.full((*place, 144), 0x7F if e4m3 else NAN, dtype=kind, device=DEV) for _ in range(2)]
    back = [order.index(i) for i in range(3)]
    c.k, c.v = (w.permute(*back, 3)[:n_pages, :page, :n_kv, :128] for w in whole)
    c.scales = (torch.full((8,), 0.03, device=DEV), torch.full((8,), 0.02, device=DEV)) if e4m3 else (None, None)
    c.p = abi.attn_paged_create(c.ctx, c.k, c.v, n_pages, page, "e4m3" if e4m3 else "bf16", *c.k.stride()[:3], *c.scales)
    lens, t = [70, 24, 1], np.array([[4, 0, 6], [2, -1, -1], [5, 9, 9]], dtype=np.int32)
    new = torch.from_numpy(rng.standard_normal((2, B, 70, n_kv, 128))).to(torch.bfloat16).to(DEV)
    abi.attn_paged_append(c.ctx, c.p, new[0], new[1], B, 70, new.stride(1), new.stride(2), None, None, ints(t), 3, ints([0] * B),
                          ints(lens))
    assert not reported(c.ctx)
    q = query(B, n_kv)
    h = attend(c, q, t, lens)
    assert not reported(c.ctx)
    check(c, q, t, lens, h)
    held = [c.k.clone(), c.v.clone()]
    for i, pool in enumerate((c.k, c.v)):  # what is not a held slot is as it was
        for b, n in enumerate(lens):
            at = np.arange(n)
            pool[torch.from_numpy(t[b, at // page].astype(np.int64)), torch.from_numpy(at % page)] = 0x7F if e4m3 else NAN
        assert torch.equal(whole[i].view(torch.uint8), torch.full_like(whole[i], 0x7F if e4m3 else NAN).view(torch.uint8))
        assert not torch.equal(held[i].view(torch.uint8), pool.contiguous().view(torch.uint8))


@pytest.mark.parametrize("seed", range(24))
def test_drawn_geometries(seed):
    rng = np.random.default_rng(1000 + seed)
    n_kv, page = int(rng.choice([1, 2, 3, 4, 5, 7, 8])), 8 * int(rng.choice([1, 2, 3, 4, 5, 8, 11, 16, 32, 40]))
    e4m3, B = bool(rng.integers(0, 2)), int(rng.choice([1, 2, 3, 7, 20, 45]))
    top = int(rng.choice([10, 130, 700, 2500, 9000 if B < 4 else 900]))
    lens = [int(n) for n in rng.integers(0, top + 1, B)]
    n_pages = sum(-(-n // page) for n in lens) + 1
    c = Cache(n_pages, page, n_kv, e4m3, bool(rng.integers(0, 2)), bool(rng.integers(0, 2)), seed=seed)
    t = tables(lens, page, n_pages, seed=seed, room=int(rng.integers(0, 5)))
    scrub(c, t, lens)
    q = query(B, n_kv, seed)
    h = attend(c, q, t, lens)
    assert not reported(c.ctx)
    check(c, q, t, lens, h)


def test_sequences_that_share_pages():
    c = Cache(12, 64, 8, True, seed=5)
    t = np.array([[3, 4, 5], [3, 4, 6], [3, 3, 3], [9, 4, 3]], dtype=np.int32)
    lens = [170, 150, 192, 129]
    q = query(4, 8)
    h = attend(c, q, t, lens)
    assert not reported(c.ctx)
    check(c, q, t, lens, h)


@pytest.mark.parametrize("e4m3", [False, True])
def test_lengths_and_pages_out_of_range(e4m3):
    lens = [100, -1, 60, 193, 192, 130, 2 ** 31 - 1, -2 ** 31, 128, 5]
    c = Cache(30, 64, 8, e4m3, seed=6)
    for bad in (-1, 30, 2 ** 31 - 1, -2 ** 31):
        t = np.arange(30, dtype=np.int32).reshape(10, 3)
        t[5, 1], t[8, 2], t[9, 0] = bad, bad, bad  # the second of three pages; one that is not read; the only one
        q = query(10, 8)
        h = attend(c, q, t, lens)
        assert reported(c.ctx) and not reported(c.ctx)
        check(c, q, t, [n if 0 <= n <= 192 else 0 for n in lens], h, left_out=(1, 3, 5, 6, 7, 9))


@pytest.mark.parametrize("e4m3", [False, True])
def test_peaked_and_rising_scores(e4m3):
    """One key far above the others in a late tile, scores that rise with the position, and all equal."""
    n = 5000
    c = Cache(80, 64, 2, e4m3, seed=8)
    t = np.stack([np.random.default_rng(b).permutation(80)[:79] for b in range(3)]).astype(np.int32)
    q = query(3, 2)
    q[1] *= 6.0
    q[2] = 0.0
    h = attend(c, q, t, [n, n, n])
    assert not reported(c.ctx)
    check(c, q, t, [n, n, n], h)
    # rising: key s is a multiple of the query that grows with s (one kv head, one sequence)
    one = Cache(80, 64, 1, False, seed=9)
    qr = query(1, 1)
    qr[0] = qr[0, :128].repeat(4)
    ramp = torch.linspace(0.0, 1.0, 80 * 64, device=DEV)[:, None] * qr[0, :128].float()[None]
    order = np.arange(80, dtype=np.int32)[None]
    one.k.copy_(ramp.to(torch.bfloat16).view(80, 64, 1, 128))
    h = attend(one, qr, order, [80 * 64])
    assert not reported(one.ctx)
    check(one, qr, order, [80 * 64], h)


@pytest.mark.parametrize("e4m3", [False, True])
def test_nan_and_large_numbers(e4m3):
    """A NaN in a key or value that is seen reaches the heads that see it and no others."""
    c = Cache(8, 32, 4, e4m3, seed=10)
    t, lens = np.arange(8, dtype=np.int32).reshape(2, 4), [100, 100]
    q = query(2, 4)
    nan = 0x7F if e4m3 else 0x7FC0
    c.raw(0)[0, 5, 1, 3] = nan                 # sequence 0, kv head 1: a key
    c.raw(1)[5, 9, 2, 77] = nan                # sequence 1, kv head 2: one element of a value
    h = attend(c, q, t, lens)
    assert not reported(c.ctx)
    odd = torch.isnan(h[:2]).cpu().view(2, 4, 4, 128)
    want = torch.zeros(2, 4, 4, 128, dtype=torch.bool)
    want[0, 1] = True
    want[1, 2, :, 77] = True
    assert torch.equal(odd, want)


def test_queries_of_any_size_against_e4m3_keys():
    """Queries enter the products with the exponent of their row taken out: huge and tiny ones hold."""
    c = Cache(8, 32, 2, True, seed=11)
    t, lens = np.arange(8, dtype=np.int32).reshape(2, 4), [100, 37]
    for size, scale in ((1e5, 1e-7), (1e-6, 1e3), (1e30, 1e-32), (0.0, 1.0)):
        c.scales[0].fill_(scale)
        q = query(2, 2, size=size)
        h = attend(c, q, t, lens)
        assert not reported(c.ctx)
        check(c, q, t, lens, h)


@pytest.mark.parametrize("scale", [1e-30, 1e-7, 1.0])
def test_queries_of_nothing_against_e4m3_keys(scale):
    """Scores that are all the same however small the scale: the mean of the values, also behind keys that are left out."""
    c = Cache(8, 32, 2, True, seed=12)
    t, lens = np.arange(8, dtype=np.int32).reshape(2, 4), [100, 37]
    scrub(c, t, lens)
    c.scales[0].fill_(scale)
    for size in (0.0, 1e-38):
        q = query(2, 2, size=size)
        h = attend(c, q, t, lens)
        assert not reported(c.ctx)
        check(c, q, t, lens, h)


def test_pools_past_two_to_the_32():
    """Pages whose byte offsets (and element offsets) pass 2^32."""
    n_pages, page = 36000, 128
    need = 2 * n_pages * page * 1024 * 2
    if torch.cuda.mem_get_info()[0] < need + (8 << 30):
        pytest.skip("not enough free memory")
    c = Cache.__new__(Cache)
    c.n_pages, c.page, c.n_kv, c.e4m3, c.heads_first = n_pages, page, 8, False, False
    both = torch.zeros(2, n_pages, page, 8, 128, dtype=torch.bfloat16, device=DEV)
    c.k, c.v, c.scales, c.ctx = both[0], both[1], (None, None), context(8)
    assert (n_pages - 1) * c.k.stride(0) > 2 ** 32
    c.p = abi.attn_paged_create(c.ctx, c.k, c.v, n_pages, page, "bf16", *c.k.stride()[:3])
    t = np.array([[n_pages - 1, 1, n_pages - 2], [17000, 35000, 33000]], dtype=np.int32)
    lens, T = [0, 100], 140
    new = torch.randn(2, 2, T, 8, 128, device=DEV).to(torch.bfloat16)
    abi.attn_paged_append(c.ctx, c.p, new[0], new[1], 2, T, new.stride(1), new.stride(2), None, None, ints(t), 3, ints(lens))
    assert not reported(c.ctx)
    dense = []
    for b in range(2):
        for i, pool in enumerate((c.k, c.v)):
            at = np.arange(lens[b], lens[b] + T)
            assert torch.equal(pool[torch.from_numpy(t[b, at // page].astype(np.int64)), torch.from_numpy(at % page)], new[i, b])
        at = np.arange(lens[b] + T)
        idx = torch.from_numpy(t[b, at // page].astype(np.int64)), torch.from_numpy(at % page)
        dense.append([gu.np64(c.k[idx]), gu.np64(c.v[idx])])
    q = query(2, 8)
    h = attend(c, q, t, [T, 100 + T])
    assert not reported(c.ctx)
    for b in range(2):
        ref, mean, mag = po.decode(gu.np64(q[b]).reshape(8, 4, 128), *dense[b])
        d = 2 * 2.0 ** -17 * 1.02 * mag / math.sqrt(128) + 2.0 ** -20
        tol = 2.0 ** -8 * np.abs(ref) + (1 + 2.0 ** -8) * (2.0 ** -8 + d) * mean
        assert np.all(np.abs(gu.np64(h[b]).reshape(8, 4, 128) - ref) <= tol)


# ------------------------------------------------------------------------------- the largest calls
def test_the_most_tokens():
    n = 262144
    rope, w, gain = turn("halves", 32, "bands")
    gen = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randn(n, 256, generator=gen, device=DEV).to(torch.bfloat16)
    pos = torch.randint(-1000000, 1000000, (n,), generator=gen, device=DEV, dtype=torch.int32)
    out = torch.full((n + 1, 256), NAN, dtype=torch.bfloat16, device=DEV)
    abi.attn_rope_apply(context(), rope, x, n, 2, 256, pos, out, 256)
    R = torch.full((n + 1, 64, 2), NAN, device=DEV)
    abi.attn_rope_table(context(), turn()[0], pos, n, R)
    abi.attn_sync_status(context())
    assert out[n].isnan().all() and not out[:n].isnan().any() and R[n].isnan().all() and not R[:n].isnan().any()
    rows = np.r_[0:5, n // 2:n // 2 + 5, n - 5:n]
    ref, size = po.rotate(gu.np64(x[rows]).reshape(-1, 2, 128), gu.np64(pos[rows]), "halves", w, gain)
    got = gu.np64(out[rows]).reshape(-1, 2, 128)
    assert np.all(np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -21 * gain * size)
    ang = gu.np64(pos[rows])[:, None] * turn()[1]
    assert np.all(np.abs(gu.np64(R[rows]) - np.stack([np.cos(ang), np.sin(ang)], -1)) <= 2.0 ** -21)
    # as many new positions, of 1024 sequences, some of them left out
    B, T, page = 1024, 256, 64
    c = Cache(5 * B, page, 1, False, fill="nan")
    new = torch.randint(0, T + 1, (B,), generator=gen, device=DEV, dtype=torch.int32)
    lens = torch.randint(0, 64, (B,), generator=gen, device=DEV, dtype=torch.int32)
    table = torch.randperm(5 * B, generator=gen, device=DEV).int().view(B, 5)
    k = torch.randn(2, B, T, 128, generator=gen, device=DEV).to(torch.bfloat16)
    abi.attn_paged_append(c.ctx, c.p, k[0], k[1], B, T, T * 128, 128, None, None, table, 5, lens, new)
    assert not reported(c.ctx)
    at = lens[:, None].long() + torch.arange(T, device=DEV)
    live = torch.arange(T, device=DEV) < new[:, None]
    where = torch.gather(table.long(), 1, at // page)[live], (at % page)[live]
    for i, pool in enumerate((c.k, c.v)):
        assert torch.equal(pool[where][:, 0], k[i][live])
        assert int(pool.isnan().all(-1).logical_not().sum()) == int(new.sum())


@pytest.mark.parametrize("e4m3", [False, True])
def test_one_page_for_all_positions(e4m3):
    """A page as long as the longest cache: a dense cache of several sequences described as pages."""
    c = Cache(2, 1048576, 1, e4m3, seed=20)
    lens, t = [90000, 1], np.array([[1], [0]], dtype=np.int32)
    q = query(2, 1)
    h = attend(c, q, t, lens)
    assert not reported(c.ctx)
    codes = [c.raw(i)[:, :lens[0]].contiguous().cpu() for i in range(2)]
    x = [po.e4m3_values()[b.numpy()] * float(c.scales[i][0]) if e4m3 else b.view(torch.bfloat16).double().numpy()
         for i, b in enumerate(codes)]
    for b, n in enumerate(lens):
        ref, mean, mag = po.decode(gu.np64(q[b]).reshape(1, 4, 128), x[0][t[b, 0], :n], x[1][t[b, 0], :n])
        d = 2 * 2.0 ** -17 * 1.02 * mag / math.sqrt(128) + 2.0 ** -20
        assert np.all(np.abs(gu.np64(h[b]).reshape(1, 4, 128) - ref)
                      <= 2.0 ** -8 * np.abs(ref) + (1 + 2.0 ** -8) * (2.0 ** -8 + d) * mean)


@pytest.mark.parametrize("given", [(False, False), (True, False), (False, True)])
def test_scales_that_are_left_out_are_one(given):
    c = Cache(6, 16, 2, True, seed=21)
    abi.attn_paged_destroy(c.p)
    held = tuple(s if g else None for s, g in zip(c.scales, given))
    c.p = abi.attn_paged_create(c.ctx, c.k, c.v, 6, 16, "e4m3", *c.strides, *held)
    c.scales = tuple(s if g else torch.ones(8, device=DEV) for s, g in zip(c.scales, given))
    for pool in (c.k, c.v):
        pool.fill_(0x7F)
    t, n = np.array([[3, 0, 5]], dtype=np.int32), 41
    new = torch.randn(2, 1, n, 2, 128, device=DEV).to(torch.bfloat16) * 0.25
    abi.attn_paged_append(c.ctx, c.p, new[0], new[1], 1, n, 0, 256, None, None, ints(t), 3, ints([0]))
    assert not reported(c.ctx)
    at = np.arange(n)
    for i in range(2):
        got, ref = c.numbers(i)[t[0, at // 16], at % 16], gu.np64(new[i, 0])
        scale = gu.np64(c.scales[i][:2])[:, None]
        ref = np.clip(ref, -448 * scale, 448 * scale)
        assert np.all(np.abs(got - ref) <= np.maximum((2.0 ** -4 + 2.0 ** -20) * np.abs(ref), 2.0 ** -10 * scale))
    q = query(1, 2)
    h = attend(c, q, t, [n])
    assert not reported(c.ctx)
    check(c, q, t, [n], h)


# ------------------------------------------------------------------------------- refusals
def test_descriptions_that_are_refused():
    ctx = context(8)
    k = torch.zeros(4, 16, 8, 128, dtype=torch.bfloat16, device=DEV)
    v = torch.zeros_like(k)

    def code(*strides, n_pages=4, ctx=ctx):
        try:
            abi.attn_paged_destroy(abi.attn_paged_create(ctx, k, v, n_pages, 16, "bf16", *strides))
            return 0
        except abi.GQAError as e:
            return e.status
    assert code(16384, 1024, 128) == 0 and code(16384, 128, 2048) == 0
    assert code(-1, 1024, 128, n_pages=1) == 0          # an extent of 1: not read
    assert code(16384, 1024, 64) == 1                   # heads overlap
    assert code(16384, 1000, 128) == 1                  # slots overlap
    assert code(16376, 1024, 128) == 1                  # pages overlap
    assert code(16384, 1024, 128 + 4) == 3              # not 16 bytes
    assert code(16384, 0, 128) == 2 and code(16384, 1024, -128) == 2 and code(1 << 40, 1024, 128) == 2


def test_calls_that_are_refused_on_the_context():
    c, other = Cache(4, 16, 2, False), context(8)
    q, h = query(1, 8), torch.zeros(1, 4096, dtype=torch.bfloat16, device=DEV)
    t, n = ints([[0, 1]]), ints([5])

    def status(fn, *a):
        with pytest.raises(abi.GQAError) as e:
            fn(*a)
        return e.value.status
    assert status(abi.attn_paged_decode_attention, other, c.p, q, 1, t, 2, n, h) == 1            # another number of kv heads
    assert status(abi.attn_paged_decode_attention, c.ctx, c.p, q, 1, t, 65537, n, h) == 2        # over a million positions
    assert status(abi.attn_paged_decode_attention, c.ctx, c.p, q, 1, t, 2, n, q) == 1            # h over q
    assert status(abi.attn_paged_append, c.ctx, c.p, c.k, c.v, 1, 2, 0, 256, None, None, t, 2, n) == 1   # the pools themselves
    assert status(abi.attn_paged_append, c.ctx, c.p, q, q, 1, 2, 0, 128, None, None, t, 2, n) == 2       # rows overlap
    x, R, d = torch.zeros(1, 1, 4096, dtype=torch.bfloat16, device=DEV), torch.zeros(1, 64, 2, device=DEV), torch.zeros(1, 1, 4096, device=DEV)
    assert status(abi.attn_decode_paged, other, c.p, x, 1, R, t, 2, n, d) == 1
    assert status(abi.attn_decode_paged_residual, c.ctx, c.p, x, 1, R, t, 2, n, d) == 1          # no norm weight
    abi.attn_sync_status(c.ctx)
    abi.attn_sync_status(other)
