"""GPU checks of the block over caches of per-sequence length: attn_prefill_tree and
attn_decode_weights (and their residual forms) against the float64 block, the cache operators run
one after another as a server runs them, replay from CUDA graphs with other lengths, and use on a
second stream."""
import numpy as np
import pytest
import torch

from oracle import cache_oracle as co
from oracle import gqa_oracle as orc
from tests import gpu_util as gu
from transformer_gqa_attention_gb300 import abi
from transformer_gqa_attention_gb300 import inputs as gin

pytestmark = pytest.mark.gpu
DEV = gu.DEV
EPS = 1e-5
# Key weights of a block step: Q_r and K_r are bf16, each element off by 2^-8 / sqrt(12) of itself
# (root mean square), so a score of 128 products of q, k ~ N(0, 1.28^2) is off by
# sqrt(2 * 128) * 1.28^2 * 1.1e-3 / sqrt(128) = 2.6e-3 and its weight by as much: four times that.
TOL_W_REL_L1 = 1e-2


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from transformer_gqa_attention_gb300 import _build
    _build.build()


@pytest.fixture(scope="module")
def blk():
    b = gu.Block(gin.make_custom(seed=400, B=1, T=1))
    b.norm = gin.norm_weight(400)
    abi.attn_set_norm(b.ctx, b.norm.to(DEV), EPS)
    abi.attn_sync_status(b.ctx)
    yield b
    b.close()


def ints(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device=DEV)


def words(vis):
    return torch.from_numpy(co.mask_words(vis)).to(DEV)


def tree(rng, B, T):
    """(visibility [B, T, T], depth of each token [B, T])"""
    parents = [[int(rng.integers(-1, t)) if t else -1 for t in range(T)] for _ in range(B)]
    vis = np.stack([co.tree_visibility(p) for p in parents])
    return vis, vis.sum(-1) - 1


def draw(seed, lens, T, S, n_kv=8):
    """(x [B, T, 4096], caches filled to lens[b] and NaN behind), bf16 on the CPU."""
    gen = torch.Generator().manual_seed(seed)
    B = len(lens)
    x = torch.randn(B, T, 4096, generator=gen).to(torch.bfloat16)
    k, v = (torch.randn(B, S, n_kv, 128, generator=gen) for _ in range(2))
    for b, n in enumerate(lens):
        k[b, n:] = v[b, n:] = float("nan")
    return x, k.to(torch.bfloat16), v.to(torch.bfloat16)


def rope(positions):
    p = np.asarray(positions)
    return gin.rope_table(p.reshape(-1)).reshape(*p.shape, 64, 2).contiguous()


def check_caches(kd, vd, ck, cv, was_k, was_v, lens, T):
    for got, ref, was in ((kd, ck, was_k), (vd, cv, was_v)):
        g = got.cpu()
        for b, n in enumerate(lens):
            gu.assert_close(gu.np64(g[b, n:n + T]), ref[b, n:n + T], gu.TOL_BF16_REL_L1, gu.TOL_BF16_MAX, "cache")
            for a, z in ((0, n), (n + T, g.shape[1])):
                assert torch.equal(g[b, a:z].view(torch.int16), was[b, a:z].view(torch.int16))


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("T,lens", [(1, [5, 0]), (5, [40, 130, 0]), (21, [64, 7, 300]), (40, [0, 99]), (70, [17, 256])])
def test_prefill_tree_matches_the_block(blk, T, lens, residual):
    rng = np.random.default_rng(T)
    B, S = len(lens), max(lens) + T + 4
    vis, depth = tree(rng, B, T)
    x, k, v = draw(500 + T, lens, T, S)
    R = rope(np.asarray(lens)[:, None] + depth)
    kd, vd = k.to(DEV), v.to(DEV)
    out = torch.full((B, T, 4096), float("nan"), device=DEV)
    fn = abi.attn_prefill_tree_residual if residual else abi.attn_prefill_tree
    fn(blk.ctx, x.to(DEV), B, T, R.to(DEV), words(vis), kd, vd, S, ints(lens), out)
    abi.attn_sync_status(blk.ctx)
    x64 = gin.to_f64(x)
    xin = orc.rms_norm(x64, gin.to_f64(blk.norm), EPS) if residual else x64
    ref, ck, cv, _ = co.block_ragged(xin, *blk.w64, gin.to_f64(R), gu.np64(k), gu.np64(v), lens, vis)
    got = gu.np64(out) - (x64 if residual else 0.0)
    gu.assert_close(got, ref, 7e-3 if residual else gu.TOL_REL_L1, gu.TOL_MAX, f"tree block T={T}")
    if not residual:
        check_caches(kd, vd, ck, cv, k, v, lens, T)


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("lens", [[0], [40, 130, 0, 63], [(11 * b) % 50 for b in range(70)]])
def test_decode_weights_matches_the_block(blk, lens, residual):
    B, S = len(lens), max(lens) + 3
    x, k, v = draw(520 + B, lens, 1, S)
    R = rope(np.asarray(lens) + 1000)  # after an eviction a token's position is past its slot
    kd, vd = k.to(DEV), v.to(DEV)
    w0 = torch.rand(B, 8, S, generator=torch.Generator().manual_seed(B))
    w = w0.to(DEV)
    out = torch.full((B, 1, 4096), float("nan"), device=DEV)
    fn = abi.attn_decode_weights_residual if residual else abi.attn_decode_weights
    fn(blk.ctx, x.to(DEV), B, R.to(DEV), kd, vd, S, ints(lens), w, out)
    abi.attn_sync_status(blk.ctx)
    x64 = gin.to_f64(x)
    xin = orc.rms_norm(x64, gin.to_f64(blk.norm), EPS) if residual else x64
    ref, ck, cv, wr = co.block_ragged(xin, *blk.w64, gin.to_f64(R)[:, None], gu.np64(k), gu.np64(v), lens)
    gu.assert_close(gu.np64(out) - (x64 if residual else 0.0), ref, 7e-3 if residual else gu.TOL_REL_L1, gu.TOL_MAX)
    added = gu.np64(w) - gu.np64(w0)
    assert np.abs(added - wr).sum() <= TOL_W_REL_L1 * wr.sum()
    assert (gu.np64(w)[wr == 0] == gu.np64(w0)[wr == 0]).all()
    if not residual:
        check_caches(kd, vd, ck, cv, k, v, lens, 1)


def test_tree_block_on_a_head_shard():
    inp = gin.make_custom(seed=410, B=1, T=1)
    n, T, lens = 2, 9, [30, 0]
    w = [inp.wq[512:512 + 512 * n].contiguous(), inp.wk[128:128 + 128 * n].contiguous(),
         inp.wv[128:128 + 128 * n].contiguous(), inp.wo[:, 512:512 + 512 * n].contiguous()]
    ctx = abi.attn_create_shard(*[t.to(DEV) for t in w], n)
    try:
        vis, depth = tree(np.random.default_rng(4), 2, T)
        S = 44
        x, k, v = draw(411, lens, T, S, n)
        R = rope(np.asarray(lens)[:, None] + depth)
        kd, vd, out = k.to(DEV), v.to(DEV), torch.full((2, T, 4096), float("nan"), device=DEV)
        abi.attn_prefill_tree(ctx, x.to(DEV), 2, T, R.to(DEV), words(vis), kd, vd, S, ints(lens), out)
        abi.attn_sync_status(ctx)
        ref, ck, cv, _ = co.block_ragged(gin.to_f64(x), *[gin.to_f64(t) for t in w], gin.to_f64(R), gu.np64(k),
                                         gu.np64(v), lens, vis)
        gu.assert_close(gu.np64(out), ref)
        check_caches(kd, vd, ck, cv, k, v, lens, T)
        with pytest.raises(abi.GQAError) as err:  # the residual form needs the whole block
            abi.attn_prefill_tree_residual(ctx, x.to(DEV), 2, T, R.to(DEV), words(vis), kd, vd, S, ints(lens), out)
        assert err.value.status == 1
    finally:
        abi.attn_destroy(ctx)


@pytest.mark.parametrize("T,bad", [(3, 18), (3, -1), (60, 1)])
def test_a_sequence_out_of_range_is_not_written(blk, T, bad):
    S = 60 if T == 60 else 20
    lens, ok = [0, bad], [0]
    vis, depth = tree(np.random.default_rng(5), 2, T)
    x, k, v = draw(540 + T, [0, S], T, S)
    R = rope(depth)
    kd, vd, out = k.to(DEV), v.to(DEV), torch.zeros(2, T, 4096, device=DEV)
    abi.attn_prefill_tree(blk.ctx, x.to(DEV), 2, T, R.to(DEV), words(vis), kd, vd, S, ints(lens), out)
    with pytest.raises(abi.GQAError) as err:
        abi.attn_sync_status(blk.ctx)
    assert err.value.status == 2
    assert torch.isnan(out[1]).all()
    for got, was in ((kd, k), (vd, v)):
        assert torch.equal(got[1].cpu().view(torch.int16), was[1].view(torch.int16))
    ref, _, _, _ = co.block_ragged(gin.to_f64(x[:1]), *blk.w64, gin.to_f64(R[:1]), gu.np64(k[:1]), gu.np64(v[:1]), ok,
                                   vis[:1])
    gu.assert_close(gu.np64(out[:1]), ref)


class Mirror:
    """The float64 course of a server's steps on two sequences."""

    def __init__(self, w64, S):
        self.w, self.k, self.v = w64, np.zeros((2, S, 8, 128)), np.zeros((2, S, 8, 128))

    def step(self, x, R, lens, vis=None):
        ref, self.k, self.v, w = co.block_ragged(gin.to_f64(x), *self.w, gin.to_f64(R), self.k, self.v, lens, vis)
        return ref, w


def test_verify_commit_decode_evict_in_a_row(blk):
    # prompt, drafted tree, accepted paths of different length, two counted decode steps, eviction
    # in place, one more decode step
    S, P, T, B = 64, 20, 11, 2
    rng = np.random.default_rng(6)
    gen = torch.Generator().manual_seed(6)
    x = lambda t: torch.randn(B, t, 4096, generator=gen).to(torch.bfloat16)  # noqa: E731
    m = Mirror(blk.w64, S)
    kd, vd = gu.empty_cache(B, S)
    w = torch.zeros(B, 8, S, device=DEV)
    lens = [P, P]
    ld = ints(lens)

    x0 = x(P)
    R0 = gin.rope_table(np.arange(P))
    d = torch.empty(B, P, 4096, device=DEV)
    abi.attn_prefill(blk.ctx, x0.to(DEV), B, P, R0.to(DEV), True, kd, vd, S, 0, d)
    ref, _ = m.step(x0, R0[None].expand(B, -1, -1, -1), [0, 0], np.stack([np.tril(np.ones((P, P), bool))] * B))
    gu.assert_close(gu.np64(d), ref, what="prompt")

    vis, depth = tree(rng, B, T)
    x1, R1 = x(T), rope(P + depth)
    d = torch.empty(B, T, 4096, device=DEV)
    abi.attn_prefill_tree(blk.ctx, x1.to(DEV), B, T, R1.to(DEV), words(vis), kd, vd, S, ld, d)
    ref, _ = m.step(x1, R1, lens, vis)
    gu.assert_close(gu.np64(d), ref, what="tree")

    paths = [np.flatnonzero(vis[0, T - 1]).tolist(), []]  # the last token's branch; nothing
    table = np.zeros((B, T), dtype=np.int32)
    table[0, :len(paths[0])] = paths[0]
    abi.attn_cache_commit(blk.ctx, kd, vd, B, S, T, ld, ints(table), ints([len(p) for p in paths]), ld)
    m.k, m.v = co.commit(m.k, lens, paths), co.commit(m.v, lens, paths)
    lens = [n + len(p) for n, p in zip(lens, paths)]
    assert ld.tolist() == lens

    total = np.zeros((B, 8, S))
    pos = np.array(lens)
    for step in range(3):
        x2, R2 = x(1), rope(pos + step)
        d = torch.empty(B, 1, 4096, device=DEV)
        abi.attn_decode_weights(blk.ctx, x2.to(DEV), B, R2.to(DEV), kd, vd, S, ld, w, d)
        ref, wr = m.step(x2, R2[:, None], lens)
        gu.assert_close(gu.np64(d), ref, what=f"decode step {step}")
        total += wr
        assert np.abs(gu.np64(w) - total).sum() <= TOL_W_REL_L1 * total.sum()
        ld += 1
        lens = [n + 1 for n in lens]
        if step == 1:
            budget = 15
            before = w.cpu().numpy()
            kept = torch.zeros(B, 8, budget, dtype=torch.int32, device=DEV)
            abi.attn_cache_evict(blk.ctx, kd, vd, w, B, S, ld, budget, 2, 4, kd, vd, w, S, kept, ld)
            at = kept.cpu().numpy()
            for b in range(B):
                for g in range(8):
                    assert at[b, g].tolist() == co.evict_positions(before[b, g].tolist(), lens[b], budget, 2, 4)
                    for c in (m.k, m.v):
                        c[b, :budget, g] = c[b, at[b, g], g]
                    total[b, g, :budget] = total[b, g, at[b, g]]
                    total[b, g, budget:] = 0
            lens = [budget, budget]
            assert ld.tolist() == lens
    abi.attn_sync_status(blk.ctx)


def test_replay_with_other_lengths_and_after_the_workspace_grew(blk):
    # one graph of verify + commit; the lengths, the tree and the path are device memory, so a
    # replay follows them.  In between a larger call outgrows the workspace that the graph uses.
    T, S, B = 6, 96, 2
    ctx = abi.attn_create(*blk.w)
    try:
        rng = np.random.default_rng(7)
        kd, vd = (torch.zeros(B, S, 8, 128, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        xd = torch.zeros(B, T, 4096, dtype=torch.bfloat16, device=DEV)
        Rd = torch.zeros(B, T, 64, 2, device=DEV)
        md = torch.zeros(B, T, 1, dtype=torch.int32, device=DEV)
        ld, pd, nd = ints([0, 0]), ints(np.zeros((B, T))), ints([0, 0])
        new, out = ints([0, 0]), torch.empty(B, T, 4096, device=DEV)

        def step():
            abi.attn_prefill_tree(ctx, xd, B, T, Rd, md, kd, vd, S, ld, out)
            abi.attn_cache_commit(ctx, kd, vd, B, S, T, ld, pd, nd, new)

        step()  # sizes the workspace
        abi.attn_sync_status(ctx)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        for round_, lens in enumerate(([3, 80], [90, 0], [41, 64])):
            vis, depth = tree(rng, B, T)
            x, k, v = draw(560 + round_, lens, T, S)
            R = rope(np.asarray(lens)[:, None] + depth)
            paths = [np.flatnonzero(vis[b, T - 1]).tolist() for b in range(B)]
            table = np.zeros((B, T), dtype=np.int32)
            for b, p in enumerate(paths):
                table[b, :len(p)] = p
            for dst, src in ((kd, k), (vd, v), (xd, x), (Rd, R), (md, torch.from_numpy(co.mask_words(vis))),
                             (ld, ints(lens)), (pd, ints(table)), (nd, ints([len(p) for p in paths]))):
                dst.copy_(src)
            g.replay()
            torch.cuda.synchronize()
            abi.attn_sync_status(ctx)
            ref, ck, _, _ = co.block_ragged(gin.to_f64(x), *blk.w64, gin.to_f64(R), gu.np64(k), gu.np64(v), lens, vis)
            gu.assert_close(gu.np64(out), ref, what=f"replay {round_}")
            assert new.tolist() == [n + len(p) for n, p in zip(lens, paths)]
            want = co.commit(ck, lens, paths)
            for b, n in enumerate(lens):
                gu.assert_close(gu.np64(kd[b, n:n + len(paths[b])]), want[b, n:n + len(paths[b])],
                                gu.TOL_BF16_REL_L1, gu.TOL_BF16_MAX)
            if round_ == 0:  # a much larger call on the same context
                big = torch.zeros(4, 1024, 4096, dtype=torch.bfloat16, device=DEV)
                bk, bv = gu.empty_cache(4, 1024)
                bd = torch.empty(4, 1024, 4096, device=DEV)
                abi.attn_prefill(ctx, big, 4, 1024, torch.zeros(1024, 64, 2, device=DEV), True, bk, bv, 1024, 0, bd)
                junk = [torch.full((1 << 20,), float("nan"), device=DEV) for _ in range(8)]  # reuse of freed memory
                torch.cuda.synchronize()
                del junk
    finally:
        abi.attn_destroy(ctx)


def test_a_call_that_has_to_grow_is_refused_while_capturing(blk):
    ctx = abi.attn_create(*blk.w)
    try:
        T, S = 4, 16
        vis, depth = tree(np.random.default_rng(8), 1, T)
        x, k, v = draw(570, [5], T, S)
        args = (x.to(DEV), 1, T, rope(5 + depth).to(DEV), words(vis), k.to(DEV), v.to(DEV), S, ints([5]))
        out = torch.zeros(1, T, 4096, device=DEV)
        mark = torch.zeros(1, device=DEV)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            mark += 1
            with pytest.raises(abi.GQAError) as err:
                abi.attn_prefill_tree(ctx, *args, out)
            assert err.value.status == 4
        g.replay()  # the capture itself stayed valid
        torch.cuda.synchronize()
        assert mark.item() == 1 and (out == 0).all()
        abi.attn_prefill_tree(ctx, *args, out)
        abi.attn_sync_status(ctx)
        ref, _, _, _ = co.block_ragged(gin.to_f64(x), *blk.w64, gin.to_f64(rope(5 + depth)), gu.np64(k), gu.np64(v),
                                       [5], vis)
        gu.assert_close(gu.np64(out), ref)
    finally:
        abi.attn_destroy(ctx)


def test_a_refused_capture_leaves_nothing_behind(blk):
    # the block's workspace is large enough, the scratch of the attention is not: no kernel is recorded
    ctx = abi.attn_create(*blk.w)
    try:
        T, S = 4, 300
        vis, depth = tree(np.random.default_rng(12), 1, T)
        x, k, v = draw(575, [200], T, S)
        kd, vd = k.to(DEV), v.to(DEV)
        bk, bv = gu.empty_cache(1, 256)
        abi.attn_prefill(ctx, torch.zeros(1, 256, 4096, dtype=torch.bfloat16, device=DEV), 1, 256,
                         torch.zeros(256, 64, 2, device=DEV), True, bk, bv, 256, 0, torch.empty(1, 256, 4096, device=DEV))
        out = torch.zeros(1, T, 4096, device=DEV)
        w = torch.zeros(1, 8, S, device=DEV)
        args = (x.to(DEV), 1, T, rope(200 + depth).to(DEV), words(vis), kd, vd, S, ints([200]), out)
        steps = (x[:, :1].contiguous().to(DEV), 1, rope(200 + depth)[:, 0].contiguous().to(DEV), kd, vd, S, ints([200]), w,
                 out[:, :1].contiguous())
        mark = torch.zeros(1, device=DEV)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            mark += 1
            for call, a in ((abi.attn_prefill_tree, args), (abi.attn_decode_weights, steps)):
                with pytest.raises(abi.GQAError) as err:
                    call(ctx, *a)
                assert err.value.status == 4
        g.replay()
        torch.cuda.synchronize()
        assert mark.item() == 1 and (out == 0).all() and (w == 0).all()
        assert torch.equal(kd.cpu().view(torch.int16), k.view(torch.int16))
        assert torch.equal(vd.cpu().view(torch.int16), v.view(torch.int16))
    finally:
        abi.attn_destroy(ctx)


def test_on_a_second_stream_behind_other_work(blk):
    # lengths, mask and queries are written on the stream just before the calls that read them
    T, S, B = 12, 700, 3
    lens = [600, 3, 88]
    vis, depth = tree(np.random.default_rng(9), B, T)
    x, k, v = draw(580, lens, T, S)
    R = rope(np.asarray(lens)[:, None] + depth)
    host = [t.to(DEV) for t in (x, R, torch.from_numpy(co.mask_words(vis)), k, v, ints(lens))]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        dev = [torch.zeros_like(t) for t in host]
        out = torch.empty(B, T, 4096, device=DEV)
        torch.cuda._sleep(2_000_000)
        for d, h in zip(dev, host):
            d.copy_(h)
        abi.attn_prefill_tree(blk.ctx, dev[0], B, T, dev[1], dev[2], dev[3], dev[4], S, dev[5], out, stream=s)
        abi.attn_sync_status(blk.ctx, stream=s)
    ref, _, _, _ = co.block_ragged(gin.to_f64(x), *blk.w64, gin.to_f64(R), gu.np64(k), gu.np64(v), lens, vis)
    gu.assert_close(gu.np64(out), ref)


def test_profile_names_the_cache_kernels(blk):
    T, S = 3, 40
    vis, depth = tree(np.random.default_rng(10), 1, T)
    x, k, v = draw(590, [9], T, S)
    ld, w = ints([9]), torch.ones(1, 8, S, device=DEV)
    kd, vd = k.to(DEV), v.to(DEV)
    abi.attn_profile_begin(blk.ctx)
    abi.attn_prefill_tree(blk.ctx, x.to(DEV), 1, T, rope(9 + depth).to(DEV), words(vis), kd, vd, S, ld,
                          torch.empty(1, T, 4096, device=DEV))
    abi.attn_cache_commit(blk.ctx, kd, vd, 1, S, T, ld, ints([[0, 0, 0]]), ints([1]), ld)
    abi.attn_cache_evict(blk.ctx, kd, vd, w, 1, S, ld, 8, 1, 1, kd, vd, w, S, torch.zeros(1, 8, 8, dtype=torch.int32,
                                                                                         device=DEV), ld)
    prof = abi.attn_profile_end(blk.ctx)
    assert all(prof[n][1] >= 1 for n in ("qkv_splitk", "cache_attn", "cache_commit", "evict_select", "evict_move",
                                         "out_splitk")), prof
