"""GPU checks of the block's decode step over pages against what its pages hold: with the captured Q_r
the heads are attention in float64 over the stored numbers, Delta is their product with W_O, and the
stored new keys and values are those of the projections rounded to the pages' type."""
import math

import numpy as np
import pytest
import torch

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


class Step:
    """A block (or the shard of kv heads first .. first + n_kv - 1) over pages that hold random numbers of the size of
    its own keys and values."""

    def __init__(self, lens, page, e4m3, n_kv=8, first=0, residual=False, room=4, seed=0):
        self.lens, self.page, self.e4m3, self.n_kv, self.residual, B = lens, page, e4m3, n_kv, residual, len(lens)
        inp = gin.make_custom(seed=800 + seed, B=1, T=1)
        rows = lambda w, n: w[n * first:n * (first + n_kv)].contiguous()  # noqa: E731
        w = [rows(inp.wq, 512), rows(inp.wk, 128), rows(inp.wv, 128), inp.wo[:, 512 * first:512 * (first + n_kv)].contiguous()]
        self.w64 = [gin.to_f64(t) for t in w]
        self.ctx = abi.attn_create_shard(*[t.to(DEV) for t in w], n_kv) if n_kv < 8 else abi.attn_create(*[t.to(DEV) for t in w])
        if residual:
            abi.attn_set_norm(self.ctx, gin.norm_weight(1).to(DEV))
        self.per = -(-(max(lens) + room) // page)
        n_pages = B * self.per
        gen = torch.Generator(device=DEV).manual_seed(seed)
        self.gen = gen
        pools = [1.3 * torch.randn(n_pages, page, n_kv, 128, generator=gen, device=DEV) for _ in range(2)]
        self.scales = [torch.rand(8, generator=gen, device=DEV) * 0.02 + 0.02 for _ in range(2)] if e4m3 else [None, None]
        self.pools = [((p * 32).to(torch.float8_e4m3fn).view(torch.uint8) if e4m3 else p.to(torch.bfloat16)) for p in pools]
        self.p = abi.attn_paged_create(self.ctx, *self.pools, n_pages, page, "e4m3" if e4m3 else "bf16",
                                       *self.pools[0].stride()[:3], *self.scales)
        self.t = np.random.default_rng(seed).permutation(n_pages).reshape(B, self.per).astype(np.int32)
        self.table, self.dev_lens = ints(self.t), ints(lens)
        self.rope = abi.attn_rope_init("pairs", 128, gin.ROPE_THETA)
        self.x = torch.empty(B, 1, 4096, dtype=torch.bfloat16, device=DEV)
        self.R = torch.empty(B, 64, 2, device=DEV)
        self.out = torch.empty(B, 1, 4096, device=DEV)

    def draw(self):
        self.x.normal_(generator=self.gen)

    def call(self):
        abi.attn_rope_table(self.ctx, self.rope, self.dev_lens, len(self.lens), self.R)
        step = abi.attn_decode_paged_residual if self.residual else abi.attn_decode_paged
        step(self.ctx, self.p, self.x, len(self.lens), self.R, self.table, self.per, self.dev_lens, self.out)
        self.dev_lens.add_(1)

    def numbers(self, i, b, n):
        at = np.arange(n)
        idx = torch.from_numpy(self.t[b, at // self.page].astype(np.int64)), torch.from_numpy(at % self.page)
        x = self.pools[i][idx]
        if not self.e4m3:
            return gu.np64(x)
        return po.e4m3_values()[x.cpu().numpy()] * gu.np64(self.scales[i][:self.n_kv])[:, None]

    def check(self, sample=None):
        abi.attn_sync_status(self.ctx)
        n_kv, B = self.n_kv, len(self.lens)
        q, h = (gu.np64(gu.device_view(p, (B, 512 * n_kv))).reshape(B, n_kv, 4, 128) for p in abi.attn_debug_buffers(self.ctx))
        x = gu.np64(self.x)[:, 0]
        if self.residual:
            x = x / np.sqrt((x ** 2).mean(-1, keepdims=True) + 1e-5) * gin.to_f64(gin.norm_weight(1))
        delta = gu.np64(self.out)[:, 0] - (gu.np64(self.x)[:, 0] if self.residual else 0.0)
        sample = list(range(B)) if sample is None else sample
        gu.assert_close(delta[sample], h[sample].reshape(len(sample), -1) @ self.w64[3].T)
        w, _ = po.frequencies(128, gin.ROPE_THETA)
        for b in sample:
            n = self.lens[b]
            k, v = self.numbers(0, b, n + 1), self.numbers(1, b, n + 1)
            ref, mean, mag = po.decode(q[b], k, v)
            d = 2 * 2.0 ** -17 * 1.02 * mag / math.sqrt(128) + 2.0 ** -20
            tol = 2.0 ** -8 * np.abs(ref) + (1 + 2.0 ** -8) * ((2.0 ** -11 if self.e4m3 else 2.0 ** -8) + d) * mean
            assert np.all(np.abs(h[b] - ref) <= tol), b
            # the new key and value: a half step of e4m3 (2^-4 of it, or half the smallest step) behind a rounding to bf16
            # of a projection in fp32 (with the norm's weight rounded into the matrix in the residual form)
            new_k = po.rotate((x[b] @ self.w64[1].T).reshape(1, n_kv, 128), [n], "pairs", w)[0][0]
            new_v = (x[b] @ self.w64[2].T).reshape(n_kv, 128)
            for i, (got, want) in enumerate(((k[n], new_k), (v[n], new_v))):
                if self.e4m3:
                    sc = gu.np64(self.scales[i][:n_kv])[:, None]
                    err = np.abs(got - want) - (2.0 ** -4 * np.abs(want) + 2.0 ** -10 * sc)
                    assert err.max() <= 2.0 ** -7 * np.abs(want).max(), (b, i)
                else:
                    gu.assert_close(got, want, gu.TOL_BF16_REL_L1, gu.TOL_BF16_MAX)
        self.lens = [n + 1 for n in self.lens]

    def close(self):
        abi.attn_paged_destroy(self.p)
        abi.attn_destroy(self.ctx)


@pytest.mark.parametrize("lens,page,n_kv,residual", [
    ([37], 16, 8, False), ([0, 5, 15, 16, 90], 16, 8, False), ([700, 1, 64], 64, 8, True), ([40, 23, 24], 24, 2, False),
    ([9] * 30 + [0] * 6 + [130] * 34, 8, 8, True), ([300, 1000], 128, 1, False), ([50] * 3, 32, 5, False)])
@pytest.mark.parametrize("e4m3", [True, False])
def test_step_over_what_the_pages_hold(lens, page, n_kv, residual, e4m3):
    s = Step(lens, page, e4m3, n_kv, first=8 - n_kv, residual=residual, seed=len(lens) + page)
    for _ in range(3):
        s.draw()
        s.call()
        s.check()
    s.close()


@pytest.mark.parametrize("residual", [False, True])
def test_captured_steps_over_e4m3_pages(residual):
    s = Step([3, 60, 0, 17], 16, True, residual=residual, room=12, seed=7)
    s.draw()
    s.call()
    s.check()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s.call()
    for _ in range(8):
        s.draw()
        g.replay()
        s.check()
    s.close()


@pytest.mark.parametrize("e4m3", [True, False])
def test_step_of_the_most_sequences(e4m3):
    lens = [(b * 37) % 70 for b in range(1024)]
    s = Step(lens, 8, e4m3, room=1, seed=3)
    s.draw()
    s.call()
    s.check(sample=[0, 1, 2, 63, 64, 500, 511, 512, 1000, 1022, 1023])
    assert torch.isfinite(s.out).all()
    s.close()
