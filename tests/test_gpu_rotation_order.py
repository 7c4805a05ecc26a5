"""The rotation table R as the last thing written on the stream before a call (GPU).

A step's rotations are gathered just before the step, into the same buffer every time.  Kernels
start before the one in front of them has finished, so each must wait for it before it reads R.
Here R is the output of another call of the library, whose last kernel lets the next one start long
before it writes: a step that reads R early gets the step before's, or NaN.  Results are compared
bit for bit with those of the same R, written and waited for."""
import pytest
import torch

from tests import gpu_util as gu
from transformer_gqa_attention_gb300 import abi
from transformer_gqa_attention_gb300 import inputs as gin

pytestmark = pytest.mark.gpu
DEV = gu.DEV
STEPS = 4


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from transformer_gqa_attention_gb300 import _build
    _build.build()


@pytest.fixture(scope="module")
def blk():
    b = gu.Block(gin.make_custom(seed=600, B=1, T=1))
    yield b
    b.close()


class Writer:
    """Writes R: Delta of a small prefill, 4096 floats (32 rows of R) per token."""

    def __init__(self, blk, rows, seed):
        self.blk, self.n = blk, (rows + 31) // 32
        gen = torch.Generator().manual_seed(seed)
        self.x = [torch.randn(1, self.n, 4096, generator=gen).to(torch.bfloat16).to(DEV) for _ in range(STEPS)]
        self.rope = gin.rope_table(torch.arange(self.n).numpy()).to(DEV)
        self.ck, self.cv = gu.empty_cache(1, self.n)
        self.R = torch.full((1, self.n, 4096), float("nan"), device=DEV)

    def __call__(self, step):
        abi.attn_prefill(self.blk.ctx, self.x[step], 1, self.n, self.rope, True, self.ck, self.cv, self.n, 0, self.R)


def check(blk, rows, seed, call):
    """call(step, R) -> outputs, of a step's own buffers."""
    write = Writer(blk, rows, seed)
    ref = []
    for i in range(STEPS):
        write(i)
        abi.attn_sync_status(blk.ctx)
        ref.append(call(i, write.R))
        abi.attn_sync_status(blk.ctx)
    for outs in ref:
        assert torch.isfinite(outs[0]).all()
    assert not torch.equal(ref[0][0], ref[1][0])
    write.R.fill_(float("nan"))
    torch.cuda.synchronize()
    got = []
    for i in range(STEPS):  # nothing between the writer's last kernel and the call's first
        write(i)
        got.append(call(i, write.R))
    abi.attn_sync_status(blk.ctx)
    for i, (g, r) in enumerate(zip(got, ref)):
        for a, b in zip(g, r):
            assert torch.equal(a.view(torch.int8), b.view(torch.int8)), f"step {i}"


def drawn(seed, *shape):
    gen = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=gen).to(torch.bfloat16).to(DEV)


def buffers(seed, B, T, S):
    """Every step's own x, caches and output, made before the first call."""
    return [(drawn(seed + i, B, T, 4096), drawn(seed + 50 + i, B, S, 8, 128), drawn(seed + 90 + i, B, S, 8, 128))
            for i in range(STEPS)]


@pytest.mark.parametrize("B,T", [(2, 1), (3, 9), (5, 11), (4, 21), (3, 70)])
def test_tree_block_reads_the_rotations_behind_the_kernel_that_writes_them(blk, B, T):
    S = 100 + T
    lens = torch.tensor([(37 * b) % 100 for b in range(B)], dtype=torch.int32, device=DEV)
    W = (T + 31) // 32
    mask = torch.full((B, T, W), -1, dtype=torch.int32, device=DEV)
    bufs = [[(x, k.clone(), v.clone(), torch.empty(B, T, 4096, device=DEV)) for x, k, v in buffers(10, B, T, S)]
            for _ in range(2)]
    turn = iter(range(2 * STEPS))

    def call(step, R):
        x, k, v, out = bufs[next(turn) // STEPS][step]
        abi.attn_prefill_tree(blk.ctx, x, B, T, R, mask, k, v, S, lens, out)
        return out, k, v

    check(blk, B * T, 1, call)


@pytest.mark.parametrize("B", [1, 33, 70])
def test_counted_decode_reads_the_rotations_behind_the_kernel_that_writes_them(blk, B):
    S = 60
    lens = torch.tensor([(17 * b) % 59 for b in range(B)], dtype=torch.int32, device=DEV)
    bufs = [[(x, k.clone(), v.clone(), torch.empty(B, 1, 4096, device=DEV), torch.zeros(B, 8, S, device=DEV))
             for x, k, v in buffers(20, B, 1, S)] for _ in range(2)]
    turn = iter(range(2 * STEPS))

    def call(step, R):
        x, k, v, out, w = bufs[next(turn) // STEPS][step]
        abi.attn_decode_weights(blk.ctx, x, B, R, k, v, S, lens, w, out)
        return out, k, v, w

    check(blk, B, 2, call)


@pytest.mark.parametrize("B,T", [(1, 1), (2, 16), (1, 60), (4, 16), (1, 100), (2, 300)])
def test_prefill_reads_the_rotations_behind_the_kernel_that_writes_them(blk, B, T):
    S = T + 3
    bufs = [[(x, k.clone(), v.clone(), torch.empty(B, T, 4096, device=DEV)) for x, k, v in buffers(30, B, T, S)]
            for _ in range(2)]
    turn = iter(range(2 * STEPS))

    def call(step, R):
        x, k, v, out = bufs[next(turn) // STEPS][step]
        abi.attn_prefill(blk.ctx, x, B, T, R, True, k, v, S, 2, out)
        return out, k, v

    check(blk, T, 3, call)


@pytest.mark.parametrize("B", [1, 40, 80])
def test_decode_reads_the_rotation_behind_the_kernel_that_writes_it(blk, B):
    S = 90
    bufs = [[(x, k.clone(), v.clone(), torch.empty(B, 1, 4096, device=DEV)) for x, k, v in buffers(40, B, 1, S)]
            for _ in range(2)]
    turn = iter(range(2 * STEPS))

    def call(step, R):
        x, k, v, out = bufs[next(turn) // STEPS][step]
        abi.attn_decode(blk.ctx, x, B, 80, R, k, v, S, out)
        return out, k, v

    check(blk, 1, 4, call)


@pytest.mark.parametrize("B,T", [(1, 16), (4, 16), (2, 100)])
@pytest.mark.parametrize("tree", [False, True])
def test_residual_forms_read_what_the_kernels_in_front_write(blk, B, T, tree):
    """R by the call in front, each row's 1 / rms by the call's own first kernel."""
    abi.attn_set_norm(blk.ctx, gin.norm_weight(600).to(DEV), 1e-5)
    S = T + 40
    lens = torch.tensor([(13 * b) % 40 for b in range(B)], dtype=torch.int32, device=DEV)
    mask = torch.full((B, T, (T + 31) // 32), -1, dtype=torch.int32, device=DEV)
    # each step's x has another size, and with it another 1 / rms
    bufs = [[(x * 2.0 ** i, k.clone(), v.clone(), torch.empty(B, T, 4096, device=DEV))
             for i, (x, k, v) in enumerate(buffers(60, B, T, S))] for _ in range(2)]
    turn = iter(range(2 * STEPS))

    def call(step, R):
        x, k, v, out = bufs[next(turn) // STEPS][step]
        if tree:
            abi.attn_prefill_tree_residual(blk.ctx, x, B, T, R, mask, k, v, S, lens, out)
        else:
            abi.attn_prefill_residual(blk.ctx, x, B, T, R, True, k, v, S, 2, out)
        return out, k, v

    check(blk, B * T if tree else T, 5, call)
