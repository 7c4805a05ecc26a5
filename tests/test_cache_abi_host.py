"""Host-side refusals of the cache operators (no GPU needed): null and misaligned pointers, sizes
out of range, outputs that overlap inputs.  Addresses are fake and never dereferenced: every call
here is refused before anything is enqueued."""
import ctypes

import pytest

from transformer_gqa_attention_gb300 import _build, abi

vp = ctypes.c_void_p
STEP = 1 << 33  # fake buffers far apart
INVALID, SHAPE, ALIGN = 1, 2, 3


@pytest.fixture(scope="module", autouse=True)
def _built():
    _build.build()


# argument names in call order, with a valid value each; pointers are named in PTRS
CALLS = {
    "attn_tree_attention": dict(ctx=0, q_r=1, B=2, T=8, tree_mask=2, cache_k=3, cache_v=4, S_max=64, prefix_len=5, h=6),
    "attn_prefill_tree": dict(ctx=0, x=1, B=2, T=8, R=2, tree_mask=3, cache_k=4, cache_v=5, S_max=64, prefix_len=6,
                              delta=7),
    "attn_prefill_tree_residual": dict(ctx=0, x=1, B=2, T=8, R=2, tree_mask=3, cache_k=4, cache_v=5, S_max=64,
                                       prefix_len=6, h_out=7),
    "attn_cache_commit": dict(ctx=0, cache_k=1, cache_v=2, B=2, S_max=64, T=8, prefix_len=3, path=4, n_accept=5,
                              new_len=6),
    "attn_decode_attention_weights": dict(ctx=0, q_r=1, cache_k=2, cache_v=3, B=2, S_max=64, kv_len=4, weights=5, h=6),
    "attn_decode_weights": dict(ctx=0, x=1, B=2, R=2, cache_k=3, cache_v=4, S_max=64, kv_len=5, weights=6, delta=7),
    "attn_decode_weights_residual": dict(ctx=0, x=1, B=2, R=2, cache_k=3, cache_v=4, S_max=64, kv_len=5, weights=6,
                                         h_out=7),
    "attn_cache_evict": dict(ctx=0, cache_k=1, cache_v=2, weights=3, B=2, S_max=64, kv_len=4, budget=32, n_first=2,
                             n_recent=4, out_k=5, out_v=6, out_weights=7, S_out=48, kept=8, new_len=9),
}
SIZES = {"B", "T", "S_max", "budget", "n_first", "n_recent", "S_out"}


def status(fn, **changed):
    args = []
    for name, value in CALLS[fn].items():
        if name in SIZES:
            args.append(changed.get(name, value))
        else:
            args.append(vp(changed.get(name, (value + 1) * STEP)))
    return abi.raw_status(fn, *args, None)


def pointers(fn):
    return [n for n in CALLS[fn] if n not in SIZES]


@pytest.mark.parametrize("fn", CALLS)
def test_null_pointers_are_refused(fn):
    for name in pointers(fn):
        assert status(fn, **{name: None}) == INVALID, name


@pytest.mark.parametrize("fn", CALLS)
def test_misaligned_pointers_are_refused(fn):
    for name in pointers(fn)[1:]:
        for off in (2, 4, 8):
            assert status(fn, **{name: 40 * STEP + off}) == ALIGN, (name, off)


@pytest.mark.parametrize("fn", CALLS)
def test_sizes_out_of_range_are_refused(fn):
    bad = [dict(B=0), dict(B=-1), dict(B=1025), dict(S_max=0), dict(S_max=(1 << 20) + 1)]
    if "T" in CALLS[fn]:
        bad += [dict(T=0), dict(T=257, S_max=1024), dict(T=65)]
    if "budget" in CALLS[fn]:
        bad += [dict(budget=0), dict(budget=49), dict(n_first=-1), dict(n_recent=-1), dict(n_first=29),
                dict(n_first=(1 << 31) - 1, n_recent=(1 << 31) - 1), dict(S_out=0), dict(S_out=(1 << 20) + 1)]
    for kw in bad:
        assert status(fn, **kw) == SHAPE, kw


def test_commit_refuses_lengths_that_overlap():
    at = 4 * STEP  # prefix_len
    assert status("attn_cache_commit", B=8, new_len=at + 16) == INVALID
    assert status("attn_cache_commit", new_len=6 * STEP) == INVALID                 # n_accept
    assert status("attn_cache_commit", B=8, new_len=5 * STEP + 48) == INVALID       # inside path


def test_evict_refuses_outputs_that_overlap_inputs():
    k, v, w = 2 * STEP, 3 * STEP, 4 * STEP
    fn = "attn_cache_evict"
    assert status(fn, out_k=k) == INVALID                                            # only one in place
    assert status(fn, out_k=k, out_v=v, out_weights=w) == INVALID                    # in place with another S_out
    assert status(fn, out_k=v, out_v=k, out_weights=w, S_out=64) == INVALID          # crossed
    assert status(fn, B=8, new_len=5 * STEP + 16) == INVALID                         # inside kv_len


def test_kernel_kinds_match_the_header():
    import os
    import re
    src = open(os.path.join(os.path.dirname(__file__), "..", "include", "gqa_attn.h")).read()
    kinds = re.findall(r"GQA_KERNEL_([A-Z_]+) = (\d+),", src)
    assert [k.lower() for k, _ in kinds] == list(abi.KERNEL_KINDS)
    assert int(re.search(r"GQA_KERNEL_KINDS = (\d+)", src).group(1)) == len(abi.KERNEL_KINDS)
