"""GPU checks of the cache operators at the ends of what they accept: caches past 2^32 bytes, the
largest batch, caches of a few positions, buffers that go on behind the call's last row, two contexts
on two streams at once, graphs replayed with other lengths."""
import numpy as np
import pytest
import torch

from oracle import cache_oracle as co
from tests import gpu_util as gu
from tests.test_gpu_cache_ops import bits, check_h, context, heavy, ints, random_trees
from transformer_gqa_attention_gb300 import abi

pytestmark = pytest.mark.gpu
DEV = gu.DEV


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from transformer_gqa_attention_gb300 import _build
    _build.build()


def new_context(n_kv=8):
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device=DEV)  # noqa: E731
    ctx = abi.attn_create_shard(z(512 * n_kv, 4096), z(128 * n_kv, 4096), z(128 * n_kv, 4096), z(4096, 512 * n_kv), n_kv)
    abi.attn_sync_status(ctx)
    return ctx


def words(vis):
    return torch.from_numpy(co.mask_words(vis)).to(DEV)


def attend64(q, k, v, seen):
    """One kv head on the GPU in 64 bits: q [T, 4, 128], k, v [L, 128], seen [T, L]."""
    e = torch.einsum("thd,ld->thl", q.double(), k.double()) / 128 ** 0.5
    e.masked_fill_(~seen[:, None, :], -float("inf"))
    a = torch.softmax(e, -1)
    return a, torch.einsum("thl,ld->thd", a, v.double()), torch.einsum("thl,ld->thd", a, v.double().abs())


@pytest.fixture(scope="module")
def big():
    """Two sequences of 2^20 positions, 8 kv heads: 4.3 GB each of keys and values."""
    S = 1 << 20
    gen = torch.Generator(device=DEV).manual_seed(1)
    k = torch.randn(2, S, 8, 128, generator=gen, device=DEV, dtype=torch.bfloat16)
    v = torch.randn(2, S, 8, 128, generator=gen, device=DEV, dtype=torch.bfloat16)
    yield k, v, S
    del k, v
    torch.cuda.empty_cache()


@pytest.mark.parametrize("T", [3, 40])
def test_tree_attention_past_32_bit_offsets(big, T):
    k, v, S = big
    lens = [700, S - T]
    vis = random_trees(np.random.default_rng(T), 2, T)
    q = torch.randn(2, T, 4096, device=DEV, dtype=torch.bfloat16)
    h = torch.empty(2, T, 4096, device=DEV, dtype=torch.bfloat16)
    abi.attn_tree_attention(context(), q, 2, T, words(vis), k, v, S, ints(lens), h)
    abi.attn_sync_status(context())
    for b, g in ((0, 3), (1, 0), (1, 7)):
        end = lens[b] + T
        seen = torch.ones(T, end, dtype=torch.bool, device=DEV)
        seen[:, lens[b]:] = torch.from_numpy(vis[b]).to(DEV)
        _, ref, av = attend64(q[b].view(T, 8, 4, 128)[:, g], k[b, :end, g], v[b, :end, g], seen)
        # sum |q_i k_i| of 128 products of unit normals: well below 250
        check_h(gu.np64(h[b].view(T, 8, 4, 128)[:, g]), ref.cpu().numpy(), av.cpu().numpy(), 250.0, f"sequence {b}")


def test_weights_and_eviction_past_32_bit_offsets(big):
    k, v, S = big
    lens = [700, S]
    q = torch.randn(2, 4096, device=DEV, dtype=torch.bfloat16)
    h = torch.empty(2, 4096, device=DEV, dtype=torch.bfloat16)
    w = torch.rand(2, 8, S, device=DEV) * 1e-6
    was = w.double()
    abi.attn_decode_attention_weights(context(), q, k, v, 2, S, ints(lens), w, h)
    abi.attn_sync_status(context())
    for b, g in ((0, 2), (1, 0), (1, 7)):
        a, ref, av = attend64(q[b].view(1, 8, 4, 128)[:, g], k[b, :lens[b], g], v[b, :lens[b], g],
                              torch.ones(1, lens[b], dtype=torch.bool, device=DEV))
        d = check_h(gu.np64(h[b].view(1, 8, 4, 128)[:, g]), ref.cpu().numpy(), av.cpu().numpy(), 250.0)
        got, want = w[b, g].double(), was[b, g].clone()
        want[:lens[b]] += a.sum((0, 1))
        tol = d * (want - was[b, g]) + 2.0 ** -22 * want
        assert ((got - want).abs() <= tol).all()
    budget = 2000
    out = [torch.zeros(2, budget, 8, 128, device=DEV, dtype=torch.bfloat16) for _ in range(2)]
    ow, kept, new = torch.zeros(2, 8, budget, device=DEV), torch.zeros(2, 8, budget, device=DEV, dtype=torch.int32), ints([0, 0])
    abi.attn_cache_evict(context(), k, v, w, 2, S, ints(lens), budget, 4, 100, *out, ow, budget, kept, new)
    abi.attn_sync_status(context())
    assert new.tolist() == [700, budget]
    for g in (0, 7):
        middle = w[1, g, 4:S - 100]
        top = torch.sort(middle, descending=True, stable=True).indices[:budget - 104].sort().values + 4
        want = torch.cat([torch.arange(4, device=DEV), top, torch.arange(S - 100, S, device=DEV)])
        assert torch.equal(kept[1, g].long(), want)
        for o, c in zip(out, (k, v)):
            assert torch.equal(o[1, :, g].view(torch.int16), c[1, want, g].view(torch.int16))
        assert torch.equal(ow[1, g], w[1, g, want])


def test_commit_past_32_bit_offsets(big):
    k, v, S = big
    T, at = 9, S - 20
    was = [c[1, at:].clone() for c in (k, v)]
    path = [1, 2, 5, 8]
    table = np.zeros((2, T), dtype=np.int32)
    table[1, :4] = path
    new = ints([0, 0])
    abi.attn_cache_commit(context(), k, v, 2, S, T, ints([5, at]), ints(table), ints([0, 4]), new)
    abi.attn_sync_status(context())
    assert new.tolist() == [5, at + 4]
    for c, w in zip((k, v), was):
        want = w.clone()
        want[:4] = w[path]
        assert torch.equal(c[1, at:].view(torch.int16), want.view(torch.int16))


def test_the_largest_batch():
    B, S, n_kv = 1024, 70, 1
    rng = np.random.default_rng(2)
    gen = torch.Generator().manual_seed(2)
    lens = rng.integers(0, 60, size=B).tolist()
    k, v = (torch.randn(B, S, n_kv, 128, generator=gen).to(torch.bfloat16) for _ in range(2))
    for T in (1, 8, 10):
        vis = random_trees(rng, B, T)
        q = torch.randn(B, T, 512 * n_kv, generator=gen).to(torch.bfloat16)
        h = torch.empty(B, T, 512 * n_kv, dtype=torch.bfloat16, device=DEV)
        abi.attn_tree_attention(context(n_kv), q.to(DEV), B, T, words(vis), k.to(DEV), v.to(DEV), S, ints(lens), h)
        abi.attn_sync_status(context(n_kv))
        ref, av, _, mag = co.cache_attention(gu.np64(q).reshape(B, T, n_kv, 4, 128), gu.np64(k), gu.np64(v), lens, vis, T)
        check_h(gu.np64(h).reshape(ref.shape), ref, av, mag, f"T={T}")


@pytest.mark.parametrize("T", [1, 2, 37, 256])
def test_a_cache_that_only_holds_the_tree(T):
    vis = random_trees(np.random.default_rng(T), 2, T)
    gen = torch.Generator().manual_seed(T)
    k, v = (torch.randn(2, T, 2, 128, generator=gen).to(torch.bfloat16) for _ in range(2))
    q = torch.randn(2, T, 1024, generator=gen).to(torch.bfloat16)
    h = torch.empty(2, T, 1024, dtype=torch.bfloat16, device=DEV)
    abi.attn_tree_attention(context(2), q.to(DEV), 2, T, words(vis), k.to(DEV), v.to(DEV), T, ints([0, 0]), h)
    abi.attn_sync_status(context(2))
    ref, av, _, mag = co.cache_attention(gu.np64(q).reshape(2, T, 2, 4, 128), gu.np64(k), gu.np64(v), [0, 0], vis, T)
    check_h(gu.np64(h).reshape(ref.shape), ref, av, mag)


@pytest.mark.parametrize("T", [1, 5, 33, 70])
def test_nothing_is_written_behind_the_last_row(T):
    # every output lies in a larger buffer of a known pattern, and the inputs stay as they are
    B, S, n_kv = 3, 300, 3
    gen = torch.Generator().manual_seed(T)
    k, v = (torch.randn(B, S, n_kv, 128, generator=gen).to(torch.bfloat16).to(DEV) for _ in range(2))
    q = torch.randn(B, T, 512 * n_kv, generator=gen).to(torch.bfloat16).to(DEV)
    lens, mask = ints([100, 0, 200]), words(random_trees(np.random.default_rng(T), B, T))
    inputs = [k, v, q, lens, mask]
    was = [t.clone() for t in inputs]
    h = torch.full((B + 2, T, 512 * n_kv), 7.0, dtype=torch.bfloat16, device=DEV)
    abi.attn_tree_attention(context(n_kv), q, B, T, mask, k, v, S, lens, h)
    w = torch.full((B + 1, n_kv, S), 7.0, device=DEV)
    h1 = torch.full((B + 2, 512 * n_kv), 7.0, dtype=torch.bfloat16, device=DEV)
    abi.attn_decode_attention_weights(context(n_kv), q, k, v, B, S, lens, w, h1)
    abi.attn_sync_status(context(n_kv))
    assert (h[B:] == 7).all() and (h1[B:] == 7).all() and (w[B] == 7).all()
    for b, n in enumerate((100, 0, 200)):
        assert (w[b, :, n:] == 7).all()
    for a, b in zip(inputs, was):
        assert torch.equal(a.view(torch.int16) if a.dtype == torch.bfloat16 else a,
                           b.view(torch.int16) if b.dtype == torch.bfloat16 else b)


def test_two_contexts_on_two_streams_at_once():
    ctxs, streams = [new_context(), new_context()], [torch.cuda.Stream(), torch.cuda.Stream()]
    try:
        cases = []
        for i, T in enumerate((20, 60)):
            rng, gen = np.random.default_rng(i), torch.Generator().manual_seed(i)
            lens = [900 + 300 * i, 50, 2000]
            vis = random_trees(rng, 3, T)
            k, v = (torch.randn(3, 2100, 8, 128, generator=gen).to(torch.bfloat16) for _ in range(2))
            q = torch.randn(3, T, 4096, generator=gen).to(torch.bfloat16)
            ref = co.cache_attention(gu.np64(q).reshape(3, T, 8, 4, 128), gu.np64(k), gu.np64(v), lens, vis, T)
            h = torch.empty(3, T, 4096, dtype=torch.bfloat16, device=DEV)
            cases.append((T, [q.to(DEV), words(vis), k.to(DEV), v.to(DEV), ints(lens)], h, ref))
        torch.cuda.synchronize()
        for _ in range(20):
            for ctx, s, (T, (q, m, k, v, lens), h, _) in zip(ctxs, streams, cases):
                abi.attn_tree_attention(ctx, q, 3, T, m, k, v, 2100, lens, h, stream=s)
        for ctx, s, (T, _, h, (ref, av, _, mag)) in zip(ctxs, streams, cases):
            abi.attn_sync_status(ctx, stream=s)
            check_h(gu.np64(h).reshape(ref.shape), ref, av, mag, f"T={T}")
    finally:
        for c in ctxs:
            abi.attn_destroy(c)


def test_results_do_not_change_from_run_to_run():
    # split sequences are merged in a fixed order: the same bits every time, alone and from a graph
    T, S, lens = 30, 5100, [5000, 40, 3000]
    gen = torch.Generator().manual_seed(3)
    k, v = (torch.randn(3, S, 8, 128, generator=gen).to(torch.bfloat16).to(DEV) for _ in range(2))
    q = torch.randn(3, T, 4096, generator=gen).to(torch.bfloat16).to(DEV)
    mask, ld = words(random_trees(np.random.default_rng(3), 3, T)), ints(lens)
    h, h1 = (torch.empty(3, n, 4096, dtype=torch.bfloat16, device=DEV) for n in (T, 1))
    w = torch.zeros(3, 8, S, device=DEV)
    q1 = q[:, 0].contiguous()

    def run():
        w.zero_()
        abi.attn_tree_attention(context(), q, 3, T, mask, k, v, S, ld, h)
        abi.attn_decode_attention_weights(context(), q1, k, v, 3, S, ld, w, h1)

    run()
    first = [t.clone() for t in (h, h1, w)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    for again in (run, run, g.replay, g.replay):
        for t in (h, h1, w):
            t.fill_(float("nan"))
        again()
        torch.cuda.synchronize()
        abi.attn_sync_status(context())
        for a, b in zip((h, h1, w), first):
            assert torch.equal(a.view(torch.int16) if a.dtype == torch.bfloat16 else a,
                               b.view(torch.int16) if b.dtype == torch.bfloat16 else b)


def test_eviction_replayed_with_other_lengths():
    # a captured decode-and-evict step follows the lengths and weights that the device holds
    B, n_kv, S, budget = 2, 8, 120, 50
    ctx = context(n_kv)
    gen = torch.Generator().manual_seed(4)
    k0, v0 = (torch.randn(B, S, n_kv, 128, generator=gen).to(torch.bfloat16) for _ in range(2))
    kd, vd, wd, ld = torch.empty_like(k0, device=DEV), torch.empty_like(v0, device=DEV), torch.zeros(B, n_kv, S, device=DEV), ints([0, 0])
    kept = torch.zeros(B, n_kv, budget, dtype=torch.int32, device=DEV)

    def step():
        abi.attn_cache_evict(ctx, kd, vd, wd, B, S, ld, budget, 2, 10, kd, vd, wd, S, kept, ld)

    step()
    abi.attn_sync_status(ctx)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for i, lens in enumerate(([120, 30], [51, 90], [50, 120])):
        w = heavy(i, B, n_kv, S)
        for dst, src in ((kd, k0), (vd, v0), (wd, w), (ld, ints(lens))):
            dst.copy_(src)
        g.replay()
        torch.cuda.synchronize()
        abi.attn_sync_status(ctx)
        assert ld.tolist() == [min(n, budget) for n in lens]
        for b, n in enumerate(lens):
            for h in range(n_kv):
                at = co.evict_positions(w[b, h].tolist(), n, budget, 2, 10)
                assert kept[b, h, :len(at)].tolist() == at
                assert np.array_equal(bits(kd)[b, :len(at), h], bits(k0)[b, at, h])


def test_growing_from_small_to_large_calls():
    # the scratch grows under calls of every kind, one after another on one context
    ctx = new_context()
    try:
        gen = torch.Generator().manual_seed(5)
        for T, lens in ((1, [3]), (9, [700, 20]), (33, [100]), (200, [900, 0, 300]), (2, [50])):
            B, S = len(lens), max(lens) + T
            rng = np.random.default_rng(T)
            vis = random_trees(rng, B, T)
            k, v = (torch.randn(B, S, 8, 128, generator=gen).to(torch.bfloat16) for _ in range(2))
            q = torch.randn(B, T, 4096, generator=gen).to(torch.bfloat16)
            h = torch.empty(B, T, 4096, dtype=torch.bfloat16, device=DEV)
            abi.attn_tree_attention(ctx, q.to(DEV), B, T, words(vis), k.to(DEV), v.to(DEV), S, ints(lens), h)
            w, h1 = torch.zeros(B, 8, S, device=DEV), torch.empty(B, 4096, dtype=torch.bfloat16, device=DEV)
            abi.attn_decode_attention_weights(ctx, q[:, 0].contiguous().to(DEV), k.to(DEV), v.to(DEV), B, S, ints(lens), w, h1)
            abi.attn_sync_status(ctx)
            ref, av, _, mag = co.cache_attention(gu.np64(q).reshape(B, T, 8, 4, 128), gu.np64(k), gu.np64(v), lens, vis, T)
            check_h(gu.np64(h).reshape(ref.shape), ref, av, mag, f"T={T}")
            assert np.allclose(gu.np64(w).sum(-1), [[4.0 if n else 0.0] * 8 for n in lens], rtol=1e-5)
    finally:
        abi.attn_destroy(ctx)
