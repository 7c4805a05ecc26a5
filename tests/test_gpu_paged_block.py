"""GPU checks of the paged cache in use: the block's decode step over pages behind a prompt whose keys
and values were appended from a dense cache; queries, keys and values of a fused projection rotated,
appended and attended; captured graphs, streams and contexts beside one another."""
import math

import numpy as np
import pytest
import torch

from oracle import gqa_oracle as orc
from oracle import paged_oracle as po
from tests import gpu_util as gu
from transformer_gqa_attention_gb300 import abi
from transformer_gqa_attention_gb300 import inputs as gin

pytestmark = pytest.mark.gpu
DEV = gu.DEV


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from transformer_gqa_attention_gb300 import _build
    _build.build()


def ints(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device=DEV)


class Pools:
    def __init__(self, ctx, n_pages, page, dtype="bf16", n_kv=8):
        kind = torch.uint8 if dtype == "e4m3" else torch.bfloat16
        nan = 0x7F if dtype == "e4m3" else float("nan")
        self.k = torch.full((n_pages, page, n_kv, 128), nan, dtype=kind, device=DEV)
        self.v = torch.full_like(self.k, nan)
        self.scales = [torch.full((8,), 1.0 / 32, device=DEV) for _ in range(2)] if dtype == "e4m3" else [None, None]
        self.p = abi.attn_paged_create(ctx, self.k, self.v, n_pages, page, dtype, *self.k.stride()[:3], *self.scales)

    def __del__(self):
        abi.attn_paged_destroy(self.p)


# Against the dense cache of the same bf16 numbers: the block's own bar (bf16 intermediates).
# With e4m3 pages a key or value is off by a uniform error over half a step, 2^-4 of it at most and
# 2^-4 / sqrt(3) = 0.036 rms.  A score is q k / sqrt(128) with |q|, |k| near 128^0.5 1.28 = 14.5 (x of unit
# variance, weights of 0.02: elements near 1.28), so it is off by 0.036 14.5 14.5 / (11.3 11.3) = 0.06 rms, each
# weight by as much of itself; with the values' own 0.036 the heads and Delta move by 0.07 to 0.1 of
# the values' size, which is at most 5 times what is left of 40 of them averaged with uneven weights: 0.5.
@pytest.mark.parametrize("B,page,dtype,residual", [(1, 16, "bf16", False), (3, 24, "bf16", True), (5, 64, "e4m3", False),
                                                   (70, 16, "bf16", False), (66, 8, "bf16", True)])
def test_decode_steps_behind_an_appended_prompt(B, page, dtype, residual):
    T, steps = 37, 3
    inp = gin.make_custom(seed=900 + B, B=B, T=T)
    blk = gu.Block(inp)
    try:
        ctx, S = blk.ctx, T + steps
        if residual:
            abi.attn_set_norm(ctx, gin.norm_weight(1).to(DEV))
        dense = gu.empty_cache(B, S)
        blk.prefill(inp.x.to(DEV), inp.R.to(DEV), *dense)
        per = -(-S // page)
        pools = Pools(ctx, B * per + 1, page, dtype)
        t = np.random.default_rng(B).permutation(B * per + 1)[:B * per].reshape(B, per).astype(np.int32)
        lens, table = ints([0] * B), ints(t)
        abi.attn_paged_append(ctx, pools.p, *dense, B, T, S * 1024, 1024, None, None, table, per, lens)
        lens += T
        gen = torch.Generator().manual_seed(B)
        for i in range(steps):
            x = torch.randn(B, 1, 4096, generator=gen).to(torch.bfloat16).to(DEV)
            rope = abi.attn_rope_init("pairs", 128, gin.ROPE_THETA)
            R = torch.empty(B, 64, 2, device=DEV)
            abi.attn_rope_table(ctx, rope, lens, B, R)
            got, want = torch.empty(B, 1, 4096, device=DEV), torch.empty(B, 1, 4096, device=DEV)
            step, ref = ((abi.attn_decode_paged_residual, abi.attn_decode_residual) if residual
                         else (abi.attn_decode_paged, abi.attn_decode))
            step(ctx, pools.p, x, B, R, table, per, lens, got)
            abi.attn_sync_status(ctx)
            ref(ctx, x, B, T + i, gin.rope_table([T + i]).to(DEV), *dense, S, want)
            abi.attn_sync_status(ctx)
            lens += 1
            a, b = gu.np64(got), gu.np64(want)
            if residual:
                a, b = a - gu.np64(x), b - gu.np64(x)
            if dtype == "bf16":
                gu.assert_close(a, b, what=f"step {i}")
            else:
                assert np.isfinite(a).all() and np.linalg.norm(a - b) <= 0.5 * np.linalg.norm(b)
            at = np.arange(T + i + 1)
            for pool, d in zip((pools.k, pools.v), dense):
                rows = pool[torch.from_numpy(t[:, at // page].astype(np.int64)), torch.from_numpy(at % page)]
                if dtype == "bf16":
                    gu.assert_close(gu.np64(rows), gu.np64(d[:, :T + i + 1]), gu.TOL_BF16_REL_L1, gu.TOL_BF16_MAX)
                else:
                    x8 = po.e4m3_values()[rows.cpu().numpy()] / 32
                    r = gu.np64(d[:, :T + i + 1])
                    assert np.all(np.abs(x8 - r) <= (2.0 ** -4 + 2.0 ** -6) * np.abs(r) + 2.0 ** -15)
    finally:
        blk.close()


def test_decode_step_against_the_oracle():
    """Sequences of different lengths, with the rows a length or page out of range gives."""
    B, page = 4, 32
    inp = gin.make_custom(seed=940, B=B, T=1, start_pos=90, S_max=96, fill_cache=True)
    blk = gu.Block(inp)
    try:
        pools = Pools(blk.ctx, 16, page)
        t = np.arange(16, dtype=np.int32).reshape(B, 4)[:, :3]
        t[2, 1] = 99
        lens = [90, 0, 40, 96]  # the last one has no room left
        rows = [g.to(DEV) for g in (inp.cache_k, inp.cache_v)]
        table = ints(np.arange(16, dtype=np.int32).reshape(B, 4)[:, :3])
        abi.attn_paged_append(blk.ctx, pools.p, *rows, B, 90, 96 * 1024, 1024, None, None, table, 3, ints([0] * B),
                              ints([90, 0, 40, 90]))
        abi.attn_sync_status(blk.ctx)
        before = pools.k.clone(), pools.v.clone()
        rope = abi.attn_rope_init("pairs", 128, gin.ROPE_THETA)
        R = torch.empty(B, 64, 2, device=DEV)
        abi.attn_rope_table(blk.ctx, rope, ints(lens), B, R)
        out = torch.zeros(B, 1, 4096, device=DEV)
        x = inp.x.to(DEV)
        abi.attn_decode_paged(blk.ctx, pools.p, x, B, R, ints(t), 3, ints(lens), out)
        with pytest.raises(abi.GQAError) as e:
            abi.attn_sync_status(blk.ctx)
        assert e.value.status == 2
        assert torch.isnan(out[2]).all() and torch.isnan(out[3]).all()
        changed = [(n, s) for n in range(16) for s in range(page)
                   if not torch.equal(pools.k[n, s].view(torch.int16), before[0][n, s].view(torch.int16))]
        assert changed == [(2, 26), (4, 0)]
        for b in (0, 1):
            n = lens[b]
            ck = np.zeros((1, n + 1, 8, 128))
            cv = np.zeros((1, n + 1, 8, 128))
            ck[:, :n], cv[:, :n] = gin.to_f64(inp.cache_k)[b:b + 1, :n], gin.to_f64(inp.cache_v)[b:b + 1, :n]
            ref, _ = orc.attention_decode(gin.to_f64(inp.x)[b:b + 1], *blk.w64, gu.np64(R[b:b + 1]), ck, cv, n)
            gu.assert_close(gu.np64(out[b:b + 1]), ref, what=str(b))
    finally:
        blk.close()


@pytest.mark.parametrize("B", [2, 70])
def test_captured_block_steps(B):
    """A step of the block with its rotation table and its lengths in one graph, against the dense block step by step."""
    T, page, steps = 21, 8, 14
    inp = gin.make_custom(seed=970 + B, B=B, T=T)
    blk = gu.Block(inp)
    try:
        ctx, S = blk.ctx, T + steps
        dense = gu.empty_cache(B, S)
        blk.prefill(inp.x.to(DEV), inp.R.to(DEV), *dense)
        per = -(-S // page)
        pools = Pools(ctx, B * per, page)
        table, lens = ints(np.random.default_rng(B).permutation(B * per).reshape(B, per)), ints([0] * B)
        abi.attn_paged_append(ctx, pools.p, *dense, B, T, S * 1024, 1024, None, None, table, per, lens)
        lens += T
        rope = abi.attn_rope_init("pairs", 128, gin.ROPE_THETA)
        x = torch.empty(B, 1, 4096, dtype=torch.bfloat16, device=DEV)
        R, got, want = torch.empty(B, 64, 2, device=DEV), torch.empty(B, 1, 4096, device=DEV), torch.empty(B, 1, 4096, device=DEV)

        def step():
            abi.attn_rope_table(ctx, rope, lens, B, R)
            abi.attn_decode_paged(ctx, pools.p, x, B, R, table, per, lens, got)
            lens.add_(1)

        gen = torch.Generator(device=DEV).manual_seed(B)
        g = torch.cuda.CUDAGraph()
        for i in range(steps):
            x.normal_(generator=gen)
            if i == 0:
                step()
                torch.cuda.synchronize()
                with torch.cuda.graph(g):
                    step()
            else:
                g.replay()
            abi.attn_sync_status(ctx)
            abi.attn_decode(ctx, x, B, T + i, gin.rope_table([T + i]).to(DEV), *dense, S, want)
            abi.attn_sync_status(ctx)
            gu.assert_close(gu.np64(got), gu.np64(want), what=f"step {i}")
        assert lens.tolist() == [S] * B
    finally:
        blk.close()


@pytest.mark.parametrize("n_kv,first", [(2, 4), (1, 7), (3, 0)])
def test_decode_step_of_a_head_shard(n_kv, first):
    """The shard's partial Delta over pages against its Delta over a dense cache."""
    B, T, page = 3, 29, 16
    inp = gin.make_custom(seed=960 + n_kv, B=B, T=T)
    rows = lambda w, n: w[n * first:n * (first + n_kv)].contiguous().to(DEV)  # noqa: E731
    ctx = abi.attn_create_shard(rows(inp.wq, 512), rows(inp.wk, 128), rows(inp.wv, 128),
                                inp.wo[:, 512 * first:512 * (first + n_kv)].contiguous().to(DEV), n_kv)
    try:
        dense = [torch.zeros(B, T + 1, n_kv, 128, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
        delta = torch.empty(B, T, 4096, device=DEV)
        abi.attn_prefill(ctx, inp.x.to(DEV), B, T, inp.R.to(DEV), True, *dense, T + 1, 0, delta)
        pools = Pools(ctx, 8, page, n_kv=n_kv)
        table = ints([[5, 2], [0, 7], [3, 1]])
        abi.attn_paged_append(ctx, pools.p, *dense, B, T, (T + 1) * n_kv * 128, n_kv * 128, None, None, table, 2, ints([0] * B))
        x, R1 = inp.x[:, :1].contiguous().to(DEV), gin.rope_table([T]).to(DEV)
        got, want = torch.empty(B, 1, 4096, device=DEV), torch.empty(B, 1, 4096, device=DEV)
        abi.attn_decode_paged(ctx, pools.p, x, B, R1.expand(B, 64, 2).contiguous(), table, 2, ints([T] * B), got)
        abi.attn_decode(ctx, x, B, T, R1, *dense, T + 1, want)
        abi.attn_sync_status(ctx)
        gu.assert_close(gu.np64(got), gu.np64(want))
    finally:
        abi.attn_destroy(ctx)


def _zero_context(n_kv):
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device=DEV)  # noqa: E731
    ctx = abi.attn_create_shard(z(512 * n_kv, 4096), z(128 * n_kv, 4096), z(128 * n_kv, 4096), z(4096, 512 * n_kv), n_kv)
    abi.attn_sync_status(ctx)
    return ctx


class Server:
    """Steps of a caller with projections of its own: fused rows in, heads out, all by one context."""

    def __init__(self, n_kv, B, room, page, layout="halves", rot=64):
        self.n_kv, self.B, self.page, self.layout = n_kv, B, page, layout
        self.per = -(-room // page)
        self.ctx = _zero_context(n_kv)
        self.pools = Pools(self.ctx, B * self.per, page, n_kv=n_kv)
        self.t = np.random.default_rng(B).permutation(B * self.per).reshape(B, self.per).astype(np.int32)
        self.table = ints(self.t)
        self.lens = torch.zeros(B, dtype=torch.int32, device=DEV)
        self.rope = abi.attn_rope_init(layout, rot, 10000.0)
        self.w, _ = po.frequencies(rot, 10000.0)
        self.rows = torch.empty(B, 6 * n_kv * 128, dtype=torch.bfloat16, device=DEV)
        self.q = torch.empty(B, 4 * n_kv * 128, dtype=torch.bfloat16, device=DEV)
        self.h = torch.empty_like(self.q)
        self.past = [[] for _ in range(B)]

    def step(self, stream=None):
        n, row = self.n_kv * 128, 6 * self.n_kv * 128
        abi.attn_rope_apply(self.ctx, self.rope, self.rows, self.B, 4 * self.n_kv, row, self.lens, self.q, 4 * n, stream)
        abi.attn_paged_append(self.ctx, self.pools.p, self.rows[:, 4 * n:], self.rows[:, 5 * n:], self.B, 1, row, 0,
                              self.rope, None, self.table, self.per, self.lens, None, stream)
        self.lens += 1
        abi.attn_paged_decode_attention(self.ctx, self.pools.p, self.q, self.B, self.table, self.per, self.lens, self.h, stream)

    def check(self):
        """Each head against the definition over the rows seen so far (one more rounding each of q and k)."""
        abi.attn_sync_status(self.ctx)
        n = self.n_kv
        rows = gu.np64(self.rows).reshape(self.B, 6 * n, 128)
        for b in range(self.B):
            self.past[b].append(rows[b])
            p = np.stack(self.past[b])
            at = np.arange(len(p))
            bf = lambda x: torch.from_numpy(x).to(torch.bfloat16).double().numpy()  # noqa: E731
            k = bf(po.rotate(p[:, 4 * n:5 * n], at, self.layout, self.w)[0])
            q = bf(po.rotate(p[-1:, :4 * n], at[-1:], self.layout, self.w)[0])[0].reshape(n, 4, 128)
            ref, mean, _ = po.decode(q, k, p[:, 5 * n:])
            # an ulp of bf16 in q or k where fp32 fell on the other side of a border: 2^-8 of a product at most for few
            # elements; scores near 12 move by less than 2^-7 all told
            got = gu.np64(self.h[b]).reshape(n, 4, 128)
            assert np.all(np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + (2.0 ** -7 + 2.0 ** -6) * mean)


@pytest.mark.parametrize("n_kv,layout,rot", [(8, "pairs", 128), (2, "halves", 64)])
def test_rotate_append_attend(n_kv, layout, rot):
    s = Server(n_kv, 6, 40, 16, layout, rot)
    gen = torch.Generator(device=DEV).manual_seed(3)
    for _ in range(20):
        s.rows.normal_(generator=gen)
        s.step()
        s.check()
    abi.attn_destroy(s.ctx)


def test_a_captured_step_follows_the_lengths():
    s = Server(5, 5, 300, 24)
    gen = torch.Generator(device=DEV).manual_seed(4)
    s.rows.normal_(generator=gen)
    s.step()  # makes room
    s.check()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        s.step()
    for _ in range(25):
        s.rows.normal_(generator=gen)
        g.replay()
        s.check()
    abi.attn_destroy(s.ctx)


def test_a_graph_outlives_the_growth_of_the_scratch():
    small, gen = Server(8, 1, 64, 8), torch.Generator(device=DEV).manual_seed(5)
    small.rows.normal_(generator=gen)
    small.step()
    small.check()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        small.step()
    # larger calls on the same context in between
    big = Pools(small.ctx, 2048, 64)
    lens, t = ints([8000] * 16), ints(np.arange(2048).reshape(16, 128))
    big.k.normal_(generator=gen)
    big.v.normal_(generator=gen)
    q, h = torch.randn(16, 4096, device=DEV).to(torch.bfloat16), torch.empty(16, 4096, dtype=torch.bfloat16, device=DEV)
    for _ in range(5):
        abi.attn_paged_decode_attention(small.ctx, big.p, q, 16, t, 128, lens, h)
        first = h.clone()
        small.rows.normal_(generator=gen)
        g.replay()
        small.check()
        abi.attn_paged_decode_attention(small.ctx, big.p, q, 16, t, 128, lens, h)
        abi.attn_sync_status(small.ctx)
        assert torch.equal(h.view(torch.int16), first.view(torch.int16))
    abi.attn_destroy(small.ctx)


def test_two_contexts_on_two_streams():
    a, b = Server(8, 3, 64, 16), Server(8, 7, 64, 32)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    gen = torch.Generator(device=DEV).manual_seed(6)
    for _ in range(15):
        for s in (a, b):
            s.rows.normal_(generator=gen)
        torch.cuda.synchronize()
        for s, st in zip((a, b), streams):
            with torch.cuda.stream(st):
                s.step()
        torch.cuda.synchronize()
        a.check()
        b.check()
    for s in (a, b):
        abi.attn_destroy(s.ctx)


def test_paged_and_dense_attention_in_turn():
    """Calls that share the context's counters and scratch."""
    inp = gin.make_custom(seed=950, B=2, T=1, start_pos=700, S_max=704, fill_cache=True)
    blk = gu.Block(inp)
    try:
        pools = Pools(blk.ctx, 48, 32)
        table = ints(np.arange(48).reshape(2, 24)[:, :22])
        dense = [g.to(DEV) for g in (inp.cache_k, inp.cache_v)]
        abi.attn_paged_append(blk.ctx, pools.p, *dense, 2, 700, 704 * 1024, 1024, None, None, table, 22, ints([0, 0]))
        x, R1 = inp.x.to(DEV), gin.rope_table([700]).to(DEV)
        R = R1.expand(2, 64, 2).contiguous()
        weights = torch.zeros(2, 8, 704, device=DEV)
        outs = [torch.empty(2, 1, 4096, device=DEV) for _ in range(3)]
        for _ in range(4):
            abi.attn_decode(blk.ctx, x, 2, 700, R1, *dense, 704, outs[0])
            abi.attn_decode_paged(blk.ctx, pools.p, x, 2, R, table, 22, ints([700, 700]), outs[1])
            abi.attn_decode_weights(blk.ctx, x, 2, R, *dense, 704, ints([700, 700]), weights, outs[2])
            abi.attn_sync_status(blk.ctx)
            gu.assert_close(gu.np64(outs[1]), gu.np64(outs[0]))
            gu.assert_close(gu.np64(outs[2]), gu.np64(outs[0]))
    finally:
        blk.close()


def test_steps_are_profiled():
    s = Server(8, 2, 64, 16)
    s.rows.normal_()
    s.step()
    abi.attn_profile_begin(s.ctx)
    s.step()
    got = abi.attn_profile_end(s.ctx)
    assert [got[k][1] for k in ("rope", "paged_append", "paged_attn")] == [1, 1, 1]
    assert all(got[k][0] > 0 for k in ("rope", "paged_append", "paged_attn"))
    abi.attn_destroy(s.ctx)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_waits_that_run_out(dtype):
    ctx = _zero_context(8)
    pools = Pools(ctx, 64, 64, dtype)
    for c in (pools.k, pools.v):
        c.copy_(torch.randint(0, 100, c.shape, device=DEV, dtype=torch.uint8) if dtype == "e4m3" else torch.randn(c.shape, device=DEV))
    t, lens = ints(np.arange(64).reshape(2, 32)), ints([2048, 1500])
    q, h = torch.randn(2, 4096, device=DEV).to(torch.bfloat16), torch.empty(2, 4096, dtype=torch.bfloat16, device=DEV)
    abi.attn_paged_decode_attention(ctx, pools.p, q, 2, t, 32, lens, h)
    abi.attn_sync_status(ctx)
    want = h.clone()
    abi.attn_debug_inject_timeout(ctx, "paged_attn")
    abi.attn_paged_decode_attention(ctx, pools.p, q, 2, t, 32, lens, h)
    with pytest.raises(abi.GQAError) as e:
        abi.attn_sync_status(ctx)
    assert e.value.status == 5
    for _ in range(2):
        h.fill_(0)
        abi.attn_paged_decode_attention(ctx, pools.p, q, 2, t, 32, lens, h)
        abi.attn_sync_status(ctx)
        assert torch.equal(h.view(torch.int16), want.view(torch.int16))
    abi.attn_destroy(ctx)
