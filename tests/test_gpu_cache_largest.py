"""The largest tree block (GPU): 1024 sequences of 256 drafted tokens, 262144 in all.  A chain behind
an empty prefix is a causal prefill, so attn_prefill on the same inputs writes the same keys and values
and gives the same Delta but for the rounding of the probabilities to bf16."""
import numpy as np
import pytest
import torch

from tests import gpu_util as gu
from transformer_gqa_attention_gb300 import abi
from transformer_gqa_attention_gb300 import inputs as gin

pytestmark = pytest.mark.gpu
DEV = gu.DEV


@pytest.mark.parametrize("B,T", [(1024, 256), (1024, 1), (7, 255)])
def test_a_chain_behind_nothing_is_a_causal_prefill(B, T):
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from transformer_gqa_attention_gb300 import _build
    _build.build()
    blk = gu.Block(gin.make_custom(seed=710, B=1, T=1))
    try:
        gen = torch.Generator(device=DEV).manual_seed(711)
        x = torch.randn(B, T, 4096, generator=gen, device=DEV, dtype=torch.bfloat16)
        R = gin.rope_table(np.arange(T)).to(DEV)
        chain = torch.from_numpy(np.tril(np.ones((T, T), dtype=np.uint32)))
        W = (T + 31) // 32
        words = np.zeros((T, W), dtype=np.uint32)
        for j in range(T):
            words[:, j // 32] |= chain[:, j].numpy() << np.uint32(j % 32)
        mask = torch.from_numpy(words.view(np.int32)).to(DEV).expand(B, T, W).contiguous()
        Rt = R.expand(B, T, 64, 2).contiguous()
        lens = torch.zeros(B, dtype=torch.int32, device=DEV)
        caches = [torch.full((B, T, 8, 128), float("nan"), dtype=torch.bfloat16, device=DEV) for _ in range(4)]
        ref = torch.full((B, T, 4096), float("nan"), device=DEV)
        got = torch.full((B, T, 4096), float("nan"), device=DEV)
        abi.attn_prefill(blk.ctx, x, B, T, R, True, caches[0], caches[1], T, 0, ref)
        abi.attn_prefill_tree(blk.ctx, x, B, T, Rt, mask, caches[2], caches[3], T, lens, got)
        abi.attn_sync_status(blk.ctx)
        for a, b in ((0, 2), (1, 3)):
            assert torch.equal(caches[a].view(torch.int16), caches[b].view(torch.int16))
        # both are within the block's bounds of the exact Delta, so within twice them of each other
        err, top, total = 0.0, 0.0, 0.0
        for b in range(0, B, 64):
            d = (got[b:b + 64] - ref[b:b + 64]).abs()
            assert torch.isfinite(d).all()
            err += float(d.sum(dtype=torch.float64))
            total += float(ref[b:b + 64].abs().sum(dtype=torch.float64))
            top = max(top, float(d.max()))
        assert err <= 2 * gu.TOL_REL_L1 * total and top <= 2 * gu.TOL_MAX * float(ref.abs().max())
    finally:
        blk.close()
