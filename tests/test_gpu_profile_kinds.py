"""What the per-kernel profile writes (GPU): as many kinds as its caller's arrays have room for."""
import ctypes

import numpy as np
import pytest
import torch

from tests import gpu_util as gu
from transformer_gqa_attention_gb300 import abi
from transformer_gqa_attention_gb300 import inputs as gin

pytestmark = pytest.mark.gpu
DEV = gu.DEV
ROOM = 24


def test_profile_writes_no_more_kinds_than_there_is_room_for():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from transformer_gqa_attention_gb300 import _build
    _build.build()
    blk = gu.Block(gin.make_custom(seed=700, B=1, T=1))
    try:
        L, x = abi.lib(), torch.zeros(1, 2, 4096, dtype=torch.bfloat16, device=DEV)
        R = gin.rope_table(np.arange(2)).to(DEV)
        mask, ld = torch.ones(1, 2, 1, dtype=torch.int32, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
        ck, cv = gu.empty_cache(1, 8)
        out = torch.empty(1, 2, 4096, device=DEV)

        def profile(end):
            ms, n = (ctypes.c_double * ROOM)(*[-1.0] * ROOM), (ctypes.c_int * ROOM)(*[-1] * ROOM)
            abi.attn_profile_begin(blk.ctx)
            abi.attn_prefill_tree(blk.ctx, x, 1, 2, R, mask, ck, cv, 8, ld, out)
            assert end(ms, n) == 0
            return list(ms), list(n)

        kinds = len(abi.KERNEL_KINDS)
        stream = torch.cuda.current_stream().cuda_stream
        ms, n = profile(lambda m, c: L.attn_profile_end(blk.ctx, m, c, stream))
        assert n[1] == 1 and ms[1] > 0 and n[5] == 1  # qkv_splitk, out_splitk
        assert ms[7:] == [-1.0] * (ROOM - 7) and n[7:] == [-1] * (ROOM - 7)
        for room in (0, 3, kinds, ROOM):
            ms, n = profile(lambda m, c: L.attn_profile_end_kinds(blk.ctx, m, c, room, stream))
            assert ms[room:] == [-1.0] * (ROOM - room) and n[room:] == [-1] * (ROOM - room)
            assert n[:room] == [0, 1, 0, 0, 0, 1, 0, 1, 1][:room] + [0] * (room - 9)
            assert all((m > 0) == (c > 0) for m, c in zip(ms[:room], n[:room]))
    finally:
        blk.close()
