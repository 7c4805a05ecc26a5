"""GPU checks of the cache operators (tree attention, commit, decode attention with key weights,
eviction) against their float64 definitions.

Tolerances.  h: with a the exact weights, the kernel's P is bf16 (half a step, 2^-9 relative to
the power of two below it, so at most 2^-8 of the value), its scores are off by at most
128 * 2^-24 * sum|q_i k_i| (fp32 sums of 128 exact products) and its exponentials by 2^-22, and h
is rounded to bf16 once:
    |h - ref| <= 2^-8 |ref| + (1 + 2^-8)(2^-8 + d) sum a|v|,  d = 2 * 2^-17 sum|q_i k_i| / sqrt(128) + 2^-20
(the factor 2: numerator and denominator).  The key weights stay fp32: |w - ref| <= d * (sum of a)
+ 2^-22 |w|.  Moved keys, values, weights and positions are compared bit for bit."""
import numpy as np
import pytest
import torch

from oracle import cache_oracle as co
from tests import gpu_util as gu
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


_ctx = {}


def context(n_kv=8):
    """A context over zero weights (the attention-only operators do not use them)."""
    if n_kv not in _ctx:
        z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device=DEV)  # noqa: E731
        _ctx[n_kv] = abi.attn_create_shard(z(512 * n_kv, 4096), z(128 * n_kv, 4096), z(128 * n_kv, 4096),
                                           z(4096, 512 * n_kv), n_kv)
        abi.attn_sync_status(_ctx[n_kv])
    return _ctx[n_kv]


@pytest.fixture(scope="module", autouse=True)
def _contexts():
    yield
    for c in _ctx.values():
        abi.attn_destroy(c)
    _ctx.clear()


def ints(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device=DEV)


def random_trees(rng, B, T):
    return np.stack([co.tree_visibility([int(rng.integers(-1, t)) if t else -1 for t in range(T)]) for _ in range(B)])


def draw_cache(gen, B, S, n_kv, ends, scale=1.0):
    """Caches filled up to ends[b]; NaN behind."""
    k = torch.randn(B, S, n_kv, 128, generator=gen) * scale
    v = torch.randn(B, S, n_kv, 128, generator=gen)
    for b, e in enumerate(ends):
        k[b, e:] = NAN
        v[b, e:] = NAN
    return k.to(torch.bfloat16), v.to(torch.bfloat16)


def check_h(got, ref, av, mag, what=""):
    got = np.asarray(got)
    assert np.isfinite(got).all(), f"{what}: non-finite values"
    d = 2 * 2.0 ** -17 * mag / 128 ** 0.5 + 2.0 ** -20
    tol = 2.0 ** -8 * np.abs(ref) + (1 + 2.0 ** -8) * (2.0 ** -8 + d) * av + 1e-30
    worst = (np.abs(got - ref) / tol).max(initial=0)
    assert worst <= 1, f"{what}: {worst:.2f} of the bound"
    return d


def run_tree(seed, lens, T, n_kv=8, vis=None, S=None, scale=1.0, spoil=True, ramp=0.0):
    rng = np.random.default_rng(seed)
    gen = torch.Generator().manual_seed(seed)
    B = len(lens)
    S = S or max(lens) + T + 3
    vis = random_trees(rng, B, T) if vis is None else vis
    k, v = draw_cache(gen, B, S, n_kv, [n + T for n in lens], scale)
    if ramp:
        k = (k.float() * (1 + ramp * torch.arange(S)[None, :, None, None] / 128)).to(torch.bfloat16)
    if spoil:  # a drafted position that nobody sees may hold anything
        for b in range(B):
            for j in np.flatnonzero(~vis[b].any(0)):
                k[b, lens[b] + j] = NAN
                v[b, lens[b] + j] = float("inf")
    q = torch.randn(B, T, n_kv * 512, generator=gen).to(torch.bfloat16)
    h = torch.full((B, T, n_kv * 512), NAN, dtype=torch.bfloat16, device=DEV)
    ctx = context(n_kv)
    kd, vd = k.to(DEV), v.to(DEV)
    abi.attn_tree_attention(ctx, q.to(DEV), B, T, torch.from_numpy(co.mask_words(vis)).to(DEV), kd, vd, S, ints(lens), h)
    abi.attn_sync_status(ctx)
    assert torch.equal(kd.cpu().view(torch.int16), k.view(torch.int16))
    ref, av, _, mag = co.cache_attention(gu.np64(q).reshape(B, T, n_kv, 4, 128), gu.np64(k), gu.np64(v), lens, vis, T)
    check_h(gu.np64(h).reshape(ref.shape), ref, av, mag, f"T={T} lens={lens} n_kv={n_kv}")
    return gu.np64(h).reshape(ref.shape)


@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 16, 31, 32, 33, 40, 63, 64, 65, 96, 129, 256])
def test_tree_attention_at_every_tree_size(T):
    run_tree(T, [130, 0, 61], T)


@pytest.mark.parametrize("lens", [[0], [1], [63], [64], [127], [128], [129], [255], [256], [1000], [5, 700, 0, 2050]])
@pytest.mark.parametrize("T", [1, 5, 32, 50])
def test_tree_attention_at_tile_edges(lens, T):
    run_tree(1000 + T, lens, T)


@pytest.mark.parametrize("n_kv", [1, 2, 3, 5, 7])
def test_tree_attention_on_head_shards(n_kv):
    run_tree(50 + n_kv, [300, 17, 128], 12, n_kv=n_kv)
    run_tree(60 + n_kv, [300, 17, 128], 45, n_kv=n_kv)


@pytest.mark.parametrize("T", [6, 40, 70])
def test_tree_rows_that_see_little_or_nothing(T):
    # padding rows (no bits, not seen by others), tokens without their own bit, and a prefix of 0
    rng = np.random.default_rng(T)
    vis = random_trees(rng, 4, T)
    for b, n in enumerate((T - 3, T // 2, 1, T)):
        vis[b, n:] = False
        vis[b, :, n:] = False
    vis[3] &= ~np.eye(T, dtype=bool)
    h = run_tree(70 + T, [0, 40, 0, 0], T, vis=vis)
    assert (h[0, T - 3:] == 0).all() and (h[2, 1:] == 0).all()
    assert (h[3, 0] == 0).all()  # the root without its own bit sees nothing
    run_tree(71 + T, [0, 5], T, vis=np.zeros((2, T, T), dtype=bool))


def test_mask_bits_beyond_the_tree_are_ignored():
    T, lens = 37, [90]
    rng = np.random.default_rng(3)
    vis = random_trees(rng, 1, T)
    gen = torch.Generator().manual_seed(3)
    k, v = draw_cache(gen, 1, 200, 8, [127])
    q = torch.randn(1, T, 4096, generator=gen).to(torch.bfloat16).to(DEV)
    outs = []
    for high in (0, -1):
        words = co.mask_words(vis)
        words[:, :, 1] |= high << (T - 32) if high else 0
        h = torch.full((1, T, 4096), NAN, dtype=torch.bfloat16, device=DEV)
        abi.attn_tree_attention(context(), q, 1, T, torch.from_numpy(words).to(DEV), k.to(DEV), v.to(DEV), 200,
                                ints(lens), h)
        abi.attn_sync_status(context())
        outs.append(h)
    assert torch.isfinite(outs[0].float()).all() and torch.equal(outs[0], outs[1])


@pytest.mark.parametrize("T", [3, 32, 64])
def test_tree_attention_with_peaked_scores(T):
    # scores spread over hundreds: late maxima force rescales, most weights underflow
    run_tree(90 + T, [1500, 3, 640], T, scale=30.0)


@pytest.mark.parametrize("T", [1, 3, 7, 12, 24, 50, 130])
def test_tree_attention_with_rising_scores(T):
    # scores grow from key tile to key tile, so that nearly every tile rescales O and l
    run_tree(95 + T, [2500, 700], T, n_kv=2, ramp=4.0)
    run_tree(96 + T, [500] * 40, T, n_kv=2, ramp=4.0)


def test_tree_attention_over_a_long_prefix():
    run_tree(91, [20000], 20, n_kv=2)
    run_tree(92, [9000, 12000], 64, n_kv=1)


@pytest.mark.parametrize("T", [2, 20, 48, 100])
def test_tree_attention_with_more_units_than_ctas(T):
    # whole units of several key tiles beside cut ones
    run_tree(94, [(53 * b) % 700 for b in range(40)], T)


@pytest.mark.parametrize("T", [20, 40, 103])
def test_tree_attention_of_many_short_units_with_rising_scores(T):
    # units of one to six tiles, several to a worker, whose maximum grows from tile to tile
    lens = [int(n) for n in np.random.default_rng(T).integers(0, 700, 30)]
    run_tree(15 + T, lens, T, ramp=2.0)


def test_causal_chain_equals_the_prefill_mask():
    # a chain (every token sees all before it) is a causal prefill of T positions
    T, L = 24, 200
    run_tree(93, [L, L], T, vis=np.stack([np.tril(np.ones((T, T), dtype=bool))] * 2))


@pytest.mark.parametrize("bad", [-1, 62, 2 ** 31 - 1, -2 ** 31])
def test_tree_prefix_out_of_range(bad):
    T, S, ctx = 4, 65, context()
    gen = torch.Generator().manual_seed(5)
    k, v = draw_cache(gen, 3, S, 8, [24] * 3)
    vis = np.stack([np.eye(T, dtype=bool)] * 3)
    q = torch.randn(3, T, 4096, generator=gen).to(torch.bfloat16)
    h = torch.zeros(3, T, 4096, dtype=torch.bfloat16, device=DEV)
    lens = [20, bad, 20]
    abi.attn_tree_attention(ctx, q.to(DEV), 3, T, torch.from_numpy(co.mask_words(vis)).to(DEV), k.to(DEV), v.to(DEV),
                            S, ints(lens), h)
    with pytest.raises(abi.GQAError) as err:
        abi.attn_sync_status(ctx)
    assert err.value.status == 2
    abi.attn_sync_status(ctx)  # read and cleared
    assert torch.isnan(h[1].float()).all()
    ref, av, _, mag = co.cache_attention(gu.np64(q[[0, 2]]).reshape(2, T, 8, 4, 128), gu.np64(k[[0, 2]]),
                                         gu.np64(v[[0, 2]]), [20, 20], vis, T)
    check_h(gu.np64(h[[0, 2]]).reshape(ref.shape), ref, av, mag)


# ------------------------------------------------------------------------------------- weights
def run_weights(seed, lens, n_kv=8, S=None, scale=1.0, steps=1, ramp=0.0):
    gen = torch.Generator().manual_seed(seed)
    B = len(lens)
    S = S or max(lens) + 5
    k, v = draw_cache(gen, B, S, n_kv, lens, scale)
    if ramp:
        k = (k.float() * (1 + ramp * torch.arange(S)[None, :, None, None] / 128)).to(torch.bfloat16)
    w0 = torch.rand(B, n_kv, S, generator=gen)
    for b, n in enumerate(lens):
        w0[b, :, n:] = NAN  # not touched
    w = w0.to(DEV)
    ctx, kd, vd = context(n_kv), k.to(DEV), v.to(DEV)
    total, d_sum = gu.np64(w0), 0.0
    for _ in range(steps):
        q = torch.randn(B, n_kv * 512, generator=gen).to(torch.bfloat16)
        h = torch.full((B, n_kv * 512), NAN, dtype=torch.bfloat16, device=DEV)
        abi.attn_decode_attention_weights(ctx, q.to(DEV), kd, vd, B, S, ints(lens), w, h)
        abi.attn_sync_status(ctx)
        ref, av, wr, mag = co.cache_attention(gu.np64(q).reshape(B, 1, n_kv, 4, 128), gu.np64(k), gu.np64(v), lens)
        d = check_h(gu.np64(h).reshape(ref.shape), ref, av, mag, f"h, lens={lens}")
        total = total + wr
        d_sum = d_sum + d * wr
    got = gu.np64(w)
    assert (np.isnan(got) == np.isnan(gu.np64(w0))).all()
    live = ~np.isnan(got)
    tol = d_sum + steps * 2.0 ** -22 * total + 1e-30
    worst = (np.abs(got - total)[live] / tol[live]).max(initial=0)
    assert worst <= 1, f"weights, lens={lens}: {worst:.2f} of the bound"


@pytest.mark.parametrize("lens", [[1], [2], [127], [128], [129], [256], [257], [1000], [0, 5, 0], [700, 3, 2049, 0, 64],
                                  list(range(1, 400, 13))])
def test_decode_attention_weights(lens):
    run_weights(200 + len(lens), lens)


@pytest.mark.parametrize("n_kv", [1, 2, 3, 6])
def test_decode_attention_weights_on_head_shards(n_kv):
    run_weights(220 + n_kv, [333, 64, 1], n_kv=n_kv)


def test_decode_attention_weights_accumulate_over_steps():
    run_weights(230, [300, 90], steps=3)


def test_decode_attention_weights_long_and_peaked():
    run_weights(231, [30000, 100], n_kv=1)
    run_weights(232, [3000, 700], scale=20.0)
    run_weights(234, [2500, 700], ramp=4.0)
    run_weights(235, [500] * 40, n_kv=2, ramp=4.0)


def test_decode_attention_weights_many_sequences():
    run_weights(233, [(37 * b) % 90 for b in range(600)], n_kv=1)


@pytest.mark.parametrize("bad", [-1, 65, 2 ** 31 - 1])
def test_weights_length_out_of_range(bad):
    S, ctx = 64, context()
    gen = torch.Generator().manual_seed(6)
    k, v = draw_cache(gen, 2, S, 8, [40, 40])
    w = torch.ones(2, 8, S, device=DEV)
    h = torch.zeros(2, 4096, dtype=torch.bfloat16, device=DEV)
    q = torch.randn(2, 4096, generator=gen).to(torch.bfloat16).to(DEV)
    abi.attn_decode_attention_weights(ctx, q, k.to(DEV), v.to(DEV), 2, S, ints([bad, 40]), w, h)
    with pytest.raises(abi.GQAError) as err:
        abi.attn_sync_status(ctx)
    assert err.value.status == 2
    assert torch.isnan(h[0].float()).all() and torch.isfinite(h[1].float()).all()
    assert (w[0] == 1).all() and abs(float(w[1].sum()) - 8 * (S + 4)) < 0.01


# -------------------------------------------------------------------------------------- commit
def bits(t):
    return t.cpu().view(torch.int16).numpy()


@pytest.mark.parametrize("n_kv", [8, 1, 3])
@pytest.mark.parametrize("T", [1, 5, 33, 256])
@pytest.mark.parametrize("alias", [False, True])
def test_commit_moves_the_accepted_path(n_kv, T, alias):
    rng = np.random.default_rng(T)
    B, S = 6, 300 + T
    gen = torch.Generator().manual_seed(T)
    k, v = draw_cache(gen, B, S, n_kv, [S - 7] * B)  # NaN payloads move like any other bits
    lens = [0, 3, 299, 300, 17, 128]
    counts = [0, T, 1, min(T, 4), T // 2, max(0, T - 1)]
    paths = [sorted(rng.choice(T, size=c, replace=False).tolist()) for c in counts]
    table = np.full((B, T), -77, dtype=np.int32)  # entries past n_accept are not read
    for b, p in enumerate(paths):
        table[b, :len(p)] = p
    ctx, kd, vd, ld = context(n_kv), k.to(DEV), v.to(DEV), ints(lens)
    new = ld if alias else torch.full((B,), -5, dtype=torch.int32, device=DEV)
    abi.attn_cache_commit(ctx, kd, vd, B, S, T, ld, ints(table), ints(counts), new)
    abi.attn_sync_status(ctx)
    assert new.tolist() == [n + c for n, c in zip(lens, counts)]
    for got, was in ((kd, k), (vd, v)):
        assert np.array_equal(bits(got), co.commit(bits(was), lens, paths))


@pytest.mark.parametrize("path,count,length", [([2, 2, 3], 3, 10), ([3, 1, 2], 3, 10), ([0, 1, 5], 3, 10),
                                               ([-1, 0, 1], 3, 10), ([0, 1, 2], -1, 10), ([0, 1, 2], 6, 10),
                                               ([0, 1, 2], 3, -1), ([0, 1, 2], 3, 28)])
def test_commit_leaves_a_bad_sequence_alone(path, count, length):
    T, S, ctx = 5, 32, context()
    gen = torch.Generator().manual_seed(9)
    k, v = draw_cache(gen, 2, S, 8, [S, S])
    kd, vd = k.to(DEV), v.to(DEV)
    new = torch.zeros(2, dtype=torch.int32, device=DEV)
    table = np.array([path + [0, 0], [1, 4, 0, 0, 0]], dtype=np.int32)
    abi.attn_cache_commit(ctx, kd, vd, 2, S, T, ints([length, 7]), ints(table), ints([count, 2]), new)
    with pytest.raises(abi.GQAError) as err:
        abi.attn_sync_status(ctx)
    assert err.value.status == 2
    assert new.tolist() == [length, 9]
    for got, was in ((kd, k), (vd, v)):
        assert np.array_equal(bits(got), co.commit(bits(was), [0, 7], [[], [1, 4]]))


# ------------------------------------------------------------------------------------ eviction
def run_evict(w, lens, budget, n_first, n_recent, n_kv, S, S_out=None, seed=0):
    """In place where S_out is None.  w [B, n_kv, S] fp32 (CPU)."""
    B = len(lens)
    gen = torch.Generator().manual_seed(seed)
    k, v = draw_cache(gen, B, S, n_kv, [S] * B)
    ctx, kd, vd, wd, ld = context(n_kv), k.to(DEV), v.to(DEV), w.to(DEV), ints(lens)
    kept = torch.full((B, n_kv, budget), -9, dtype=torch.int32, device=DEV)
    if S_out is None:
        S_out, ok, ov, ow, new = S, kd, vd, wd, ld
        rest_k, rest_v = bits(k), bits(v)
    else:
        ok = torch.full((B, S_out, n_kv, 128), 7.0, dtype=torch.bfloat16, device=DEV)
        ov = torch.full((B, S_out, n_kv, 128), -3.0, dtype=torch.bfloat16, device=DEV)
        ow = torch.full((B, n_kv, S_out), NAN, device=DEV)
        new = torch.full((B,), -5, dtype=torch.int32, device=DEV)
        rest_k, rest_v = bits(ok), bits(ov)
    in_place = ok is kd
    abi.attn_cache_evict(ctx, kd, vd, wd, B, S, ld, budget, n_first, n_recent, ok, ov, ow, S_out, kept, new)
    abi.attn_sync_status(ctx)
    assert new.tolist() == [min(n, budget) for n in lens]
    want_k, want_v, want_w = rest_k.copy(), rest_v.copy(), w.numpy().copy() if in_place else np.zeros((B, n_kv, S_out), np.float32)
    want_kept = np.full((B, n_kv, budget), -1, dtype=np.int32)
    wn = w.numpy()
    for b, n in enumerate(lens):
        for g in range(n_kv):
            at = co.evict_positions(wn[b, g].tolist(), n, budget, n_first, n_recent)
            want_kept[b, g, :len(at)] = at
            want_k[b, :len(at), g] = bits(k)[b, at, g]
            want_v[b, :len(at), g] = bits(v)[b, at, g]
            if in_place:
                want_w[b, g, len(at):n] = 0
            want_w[b, g, :len(at)] = wn[b, g, at]
    assert np.array_equal(kept.cpu().numpy(), want_kept)
    assert np.array_equal(bits(ok), want_k) and np.array_equal(bits(ov), want_v)
    assert np.array_equal(ow.cpu().numpy().view(np.int32), want_w.view(np.int32))
    if not in_place:
        assert np.array_equal(bits(kd), bits(k)) and np.array_equal(bits(vd), bits(v))


def heavy(seed, *shape):
    return torch.exp(2 * torch.randn(*shape, generator=torch.Generator().manual_seed(seed)))


@pytest.mark.parametrize("S_out", [None, 130])
@pytest.mark.parametrize("budget,n_first,n_recent", [(100, 4, 16), (1, 0, 0), (1, 1, 0), (1, 0, 1), (64, 40, 24),
                                                     (64, 0, 0), (65, 1, 63), (130, 3, 5)])
def test_evict(budget, n_first, n_recent, S_out):
    lens = [130, 0, 1, 64, 65, 100, 101, 129]
    run_evict(heavy(1, 8, 3, 140), lens, budget, n_first, n_recent, 3, 140, S_out)


@pytest.mark.parametrize("S_out", [None, 2600])
@pytest.mark.parametrize("n_kv", [8, 1])
def test_evict_long(n_kv, S_out):
    run_evict(heavy(2, 2, n_kv, 9000), [9000, 2611], 2600, 5, 300, n_kv, 9000, S_out)


@pytest.mark.parametrize("S_out", [None, 40])
def test_evict_ties_and_special_weights(S_out):
    w = heavy(3, 6, 2, 200)
    w[0] = 1.0                                              # all equal: the lowest positions stay
    w[1] = torch.round(w[1])                                # many ties
    w[2, :, ::2] = 0.0
    w[2, :, 1::4] = -0.0                                    # -0 ties with +0
    w[3, :, 10:180] = NAN                                   # fewer numbers than the budget wants
    w[4, :, ::3] = float("inf")
    w[4, :, 1::3] = -float("inf")
    w[5] = -w[5]
    w[5, :, 50:60] = 1e-42                                  # subnormal, above everything negative
    run_evict(w, [200] * 6, 40, 2, 6, 2, 200, S_out)


@pytest.mark.parametrize("B,n_kv,length", [(1, 1, 70000), (1, 8, 40000), (3, 5, 20000), (33, 2, 5000), (40, 8, 600)])
def test_evict_at_every_share_of_a_head(B, n_kv, length):
    # one to eight CTAs per head, slices of one and of several staged chunks
    S = length + 3
    w = heavy(5, B, n_kv, S)
    w[0, 0, 100:4000] = 0.25                                # a plateau that the cut may fall into
    run_evict(w, [max(0, length - 17 * b) for b in range(B)], length // 3, 3, 40, n_kv, S, length // 3 + 2)


def test_evict_many_sequences():
    run_evict(heavy(4, 300, 1, 50), [(7 * b) % 51 for b in range(300)], 20, 1, 4, 1, 50)


@pytest.mark.parametrize("bad", [-1, 51])
@pytest.mark.parametrize("in_place", [True, False])
def test_evict_length_out_of_range(bad, in_place):
    ctx, gen = context(), torch.Generator().manual_seed(4)
    k, v = draw_cache(gen, 2, 50, 8, [50, 50])
    kd, vd, w, lens = k.to(DEV), v.to(DEV), torch.ones(2, 8, 50, device=DEV), ints([bad, 50])
    kept = torch.zeros(2, 8, 20, dtype=torch.int32, device=DEV)
    outs = (kd, vd, w) if in_place else tuple(torch.ones_like(t) for t in (kd, vd, w))
    was = [t.clone() for t in outs]
    new = lens if in_place else torch.zeros_like(lens)
    abi.attn_cache_evict(ctx, kd, vd, w, 2, 50, lens, 20, 2, 2, *outs, 50, kept, new)
    with pytest.raises(abi.GQAError) as err:
        abi.attn_sync_status(ctx)
    assert err.value.status == 2
    assert new.tolist() == [0, 20] and (kept[0] == -1).all() and (kept[1] >= 0).all()
    for t, u in zip(outs, was):
        assert torch.equal(t[0], u[0])


def test_evict_refuses_partial_overlaps():
    ctx = context()
    pool = torch.zeros(4 * 64 * 8 * 128, dtype=torch.bfloat16, device=DEV)
    part = 64 * 8 * 128
    k, v, a, c = (pool[i * part:(i + 1) * part] for i in range(4))
    w, ow = torch.zeros(8, 64, device=DEV), torch.zeros(8, 64, device=DEV)
    lens, kept = ints([64]), torch.zeros(8, 16, dtype=torch.int32, device=DEV)
    for outs in ((pool[part - 128:], c, ow), (a, pool[2 * part - 256:], ow), (a, c, w[:, 4:])):
        with pytest.raises(abi.GQAError) as err:
            abi.attn_cache_evict(ctx, k, v, w, 1, 64, lens, 16, 0, 0, *outs, 32, kept, torch.zeros_like(lens))
        assert err.value.status == 1
    abi.attn_cache_evict(ctx, k, v, w, 1, 64, lens, 16, 0, 0, a, c, ow, 32, kept, torch.zeros_like(lens))
    abi.attn_sync_status(ctx)


def test_outputs_that_overlap_each_other_are_refused():
    ctx = context()
    part = 64 * 8 * 128
    pool = torch.zeros(6 * part, dtype=torch.bfloat16, device=DEV)
    k, v, a, c = (pool[i * part:(i + 1) * part] for i in range(4))
    w, ow = torch.zeros(8, 64, device=DEV), torch.zeros(8, 64, device=DEV)
    lens, kept, new = ints([64]), torch.zeros(8 * 16, dtype=torch.int32, device=DEV), ints([0])
    good = dict(ck=k, cv=v, ok=a, ov=c, ow=ow, kept=kept, new=new, S_out=64)

    def evict(**kw):
        d = {**good, **kw}
        abi.attn_cache_evict(ctx, d["ck"], d["cv"], w, 1, 64, lens, 16, 0, 0, d["ok"], d["ov"], d["ow"], d["S_out"],
                             d["kept"], d["new"])

    for bad in (dict(ov=a), dict(ov=pool[2 * part + 128:]), dict(new=kept), dict(kept=ow), dict(kept=w.view(torch.int32)),
                dict(new=ow.view(torch.int32)), dict(ck=k, cv=k, ok=k, ov=k, ow=w), dict(kept=a.view(torch.int32)),
                dict(ok=k, ov=v, ow=w, kept=lens)):
        with pytest.raises(abi.GQAError) as err:
            evict(**bad)
        assert err.value.status == 1, bad.keys()
    evict()
    evict(new=lens)
    with pytest.raises(abi.GQAError) as err:  # K and V of a commit lie apart
        abi.attn_cache_commit(ctx, k, k, 1, 64, 4, ints([8]), ints([0, 1, 2, 3]), ints([4]), new)
    assert err.value.status == 1
    abi.attn_sync_status(ctx)


# ------------------------------------------------------------------------------- failure path
@pytest.mark.parametrize("weights", [False, True])
def test_a_wait_that_runs_out_is_reported(weights):
    # the last worker issues no loads: its waits run out, the status says so, and the next call is right
    ctx = context()
    gen = torch.Generator().manual_seed(11)
    k, v = (t.to(DEV) for t in draw_cache(gen, 2, 900, 8, [800, 800]))
    q = torch.randn(2, 3, 4096, generator=gen).to(torch.bfloat16).to(DEV)
    h = torch.zeros(2, 3, 4096, dtype=torch.bfloat16, device=DEV)
    words = torch.from_numpy(co.mask_words(np.stack([np.eye(3, dtype=bool)] * 2))).to(DEV)
    abi.attn_debug_inject_timeout(ctx, "cache_attn")
    if weights:
        w = torch.zeros(2, 8, 900, device=DEV)
        abi.attn_decode_attention_weights(ctx, q, k, v, 2, 900, ints([700, 700]), w, h)
    else:
        abi.attn_tree_attention(ctx, q, 2, 3, words, k, v, 900, ints([700, 700]), h)
    with pytest.raises(abi.GQAError) as err:
        abi.attn_sync_status(ctx)
    assert err.value.status == 5
    abi.attn_sync_status(ctx)
    if weights:
        run_weights(12, [700, 700], S=900)
    else:
        run_tree(12, [700, 700], 3, S=900)


@pytest.mark.parametrize("T", [40, 200])
def test_a_wait_of_a_pair_that_runs_out_is_reported(T):
    # more than 32 tokens: the last pair of CTAs issues no loads, and the call after is right
    ctx = context()
    gen = torch.Generator().manual_seed(13)
    k, v = (t.to(DEV) for t in draw_cache(gen, 2, 900, 8, [800, 800]))
    q = torch.randn(2, T, 4096, generator=gen).to(torch.bfloat16).to(DEV)
    h = torch.zeros(2, T, 4096, dtype=torch.bfloat16, device=DEV)
    mask = torch.from_numpy(co.mask_words(np.stack([np.eye(T, dtype=bool)] * 2))).to(DEV)
    abi.attn_debug_inject_timeout(ctx, "cache_attn")
    abi.attn_tree_attention(ctx, q, 2, T, mask, k, v, 900, ints([600, 600]), h)
    with pytest.raises(abi.GQAError) as err:
        abi.attn_sync_status(ctx)
    assert err.value.status == 5
    abi.attn_sync_status(ctx)
    run_tree(14, [600, 600], T, S=900)
