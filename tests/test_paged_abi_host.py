"""Rotations set up on the host, and the refusals of the paged-cache entry points (no GPU needed).
Addresses are fake and never dereferenced: every call here is refused before the context is used."""
import ctypes
import math
import os
import shutil
import subprocess

import numpy as np
import pytest

from oracle import paged_oracle as po
from transformer_gqa_attention_gb300 import _build, abi
from transformer_gqa_attention_gb300 import inputs as gin

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
vp = ctypes.c_void_p
STEP = 1 << 33  # fake buffers far apart
INVALID, SHAPE, ALIGN = 1, 2, 3
MORE = {"plain": {}, "linear": dict(factor=4.0), "bands": dict(factor=8.0, low=1.0, high=4.0, context=8192.0),
        "ramp": dict(factor=16.0, low=1.0, high=32.0, context=4096.0)}


@pytest.fixture(scope="module", autouse=True)
def _built():
    _build.build()


# ------------------------------------------------------------------------------- rotations
@pytest.mark.parametrize("scaling", MORE)
@pytest.mark.parametrize("rot,theta", [(128, 500000.0), (96, 10000.0), (16, 1.0e6)])
def test_frequencies(rot, theta, scaling):
    r = abi.attn_rope_init("pairs", rot, theta, scaling, **MORE[scaling])
    w, gain = po.frequencies(rot, theta, scaling, **MORE[scaling])
    got = np.array([t / 2.0 ** 64 * 2 * math.pi for t in r.turns])
    # a few roundings in 64 bits, and 2^-64 of a revolution
    assert np.all(np.abs(got[:rot // 2] - w) <= 2.0 ** -48 * w + 2.0 ** -61) and not got[rot // 2:].any()
    assert abs(r.gain - gain) <= 2.0 ** -24 * gain and r.rot_dim == rot


def test_bands_are_the_scaled_table_of_the_inputs():
    r = abi.attn_rope_init("pairs", 128, gin.ROPE_THETA, "bands", **MORE["bands"])
    w = gin.scaled_frequencies(gin.ROPE_THETA ** (-2.0 * np.arange(64) / 128))
    assert np.allclose(np.array(list(r.turns), dtype=np.float64) / 2.0 ** 64 * 2 * math.pi, w, rtol=1e-13, atol=1e-18)


@pytest.mark.parametrize("bad,code", [
    (dict(layout=2), INVALID), (dict(layout=-1), INVALID), (dict(rot=0), SHAPE), (dict(rot=8), SHAPE),
    (dict(rot=120), SHAPE), (dict(rot=144), SHAPE), (dict(theta=1.0), INVALID), (dict(theta=math.nan), INVALID),
    (dict(theta=math.inf), INVALID), (dict(kind=4), INVALID), (dict(kind=-1), INVALID),
    (dict(kind=1, factor=0.5), INVALID), (dict(kind=1, factor=math.nan), INVALID), (dict(kind=2, low=4.0), INVALID),
    (dict(kind=2, low=0.0), INVALID), (dict(kind=3, context=0.0), INVALID), (dict(kind=3, high=math.inf), INVALID)])
def test_rotations_that_are_refused(bad, code):
    v = dict(layout=0, rot=128, theta=10000.0, kind=0, factor=2.0, low=1.0, high=4.0, context=4096.0) | bad
    how = abi.RopeScaling(v["kind"], v["factor"], v["low"], v["high"], v["context"])
    r = abi.Rope()
    r.check = 77
    assert abi.lib().attn_rope_init(ctypes.byref(r), v["layout"], v["rot"], v["theta"], ctypes.byref(how)) == code
    assert r.check == 77  # left as it was
    assert abi.lib().attn_rope_init(None, 0, 128, 10000.0, None) == INVALID


@pytest.mark.skipif(shutil.which("gcc") is None, reason="needs gcc")
def test_the_bindings_structures_are_the_headers(tmp_path):
    prog = ('#include <gqa_attn.h>\n#include <stdio.h>\nint main(void) { printf("%zu %zu", sizeof(gqa_rope), '
            'sizeof(gqa_rope_scaling)); return 0; }\n')
    exe = str(tmp_path / "sizes")
    subprocess.run(["gcc", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), "-xc", "-", "-o", exe], input=prog,
                   text=True, check=True)
    out = subprocess.run([exe], capture_output=True, text=True, check=True).stdout
    assert out == f"{ctypes.sizeof(abi.Rope)} {ctypes.sizeof(abi.RopeScaling)}"


# ------------------------------------------------------------------------------- refusals
_TURN = None


def turn():
    global _TURN
    _TURN = _TURN or abi.attn_rope_init("pairs", 128, 500000.0)
    return _TURN


# argument names in call order, with a valid value each; fake addresses are numbers of buffers
CALLS = {
    "attn_rope_apply": dict(ctx=0, rope="rope", x=1, n_tok=4, n_heads=32, stride=4096, positions=2, out=3,
                            out_stride=4096),
    "attn_rope_table": dict(ctx=0, rope="rope", positions=1, n_tok=4, R=2),
    "attn_paged_create": dict(ctx=0, k_pages=1, v_pages=2, n_pages=4, page_size=16, dtype=1, stride_page=16384,
                              stride_pos=1024, stride_head=128, k_scale=3, v_scale=4, handle="handle"),
    "attn_paged_append": dict(ctx=0, paged=1, k=2, v=3, B=2, T=4, stride_b=4096, stride_t=1024, rope="rope", rope_pos=4,
                              page_table=5, max_pages=8, kv_len=6, n_new=7),
    "attn_paged_decode_attention": dict(ctx=0, paged=1, q_r=2, B=2, page_table=3, max_pages=8, kv_len=4, h=5),
    "attn_decode_paged": dict(ctx=0, paged=1, x=2, B=2, R=3, page_table=4, max_pages=8, kv_len=5, delta=6),
    "attn_decode_paged_residual": dict(ctx=0, paged=1, x=2, B=2, R=3, page_table=4, max_pages=8, kv_len=5, h_out=6),
}
SIZES = {"n_tok", "n_heads", "stride", "out_stride", "n_pages", "page_size", "dtype", "stride_page", "stride_pos",
         "stride_head", "B", "T", "stride_b", "stride_t", "max_pages"}
OPTIONAL = {"attn_paged_create": {"k_scale", "v_scale"}, "attn_paged_append": {"rope", "rope_pos", "n_new"}}


def status(fn, **changed):
    handle = vp()
    args = []
    for name, value in CALLS[fn].items():
        value = changed.get(name, value if name in SIZES or isinstance(value, str) else (value + 1) * STEP)
        if value == "rope":
            value = ctypes.byref(turn())
        elif value == "handle":
            value = ctypes.byref(handle)
        elif isinstance(value, abi.Rope):
            value = ctypes.byref(value)
        elif name not in SIZES:
            value = None if value is None else vp(value)
        args.append(value)
    if fn != "attn_paged_create":
        args.append(None)
    return abi.raw_status(fn, *args)


def pointers(fn):
    return [n for n, v in CALLS[fn].items() if n not in SIZES and not isinstance(v, str)]


@pytest.mark.parametrize("fn", CALLS)
def test_null_pointers_are_refused(fn):
    for name in [n for n in CALLS[fn] if n not in SIZES]:
        if name not in OPTIONAL.get(fn, ()):
            assert status(fn, **{name: None}) == INVALID, name


@pytest.mark.parametrize("fn", CALLS)
def test_misaligned_pointers_are_refused(fn):
    for name in pointers(fn):
        if name not in ("ctx", "paged"):
            value = (CALLS[fn][name] + 1) * STEP
            assert status(fn, **{name: value + 8}) == ALIGN, name


@pytest.mark.parametrize("fn", [f for f in CALLS if "B" in CALLS[f]])
def test_sizes_out_of_range(fn):
    for bad in (dict(B=0), dict(B=1025), dict(B=-1), dict(max_pages=0), dict(max_pages=-4)):
        assert status(fn, **bad) == SHAPE, bad


def test_rotations_of_a_call():
    fn = "attn_rope_apply"
    for bad in (dict(n_tok=0), dict(n_tok=262145), dict(n_heads=0), dict(n_heads=1025), dict(stride=4088),
                dict(out_stride=0), dict(stride=-4096), dict(stride=1 << 31), dict(out_stride=1 << 31)):
        assert status(fn, **bad) == SHAPE, bad
    assert status(fn, stride=4100) == ALIGN and status(fn, out_stride=4100) == ALIGN
    x = 2 * STEP
    assert status(fn, out=x, out_stride=8192) == INVALID          # in place with another stride
    assert status(fn, out=x + 16) == INVALID                      # overlaps
    assert status(fn, out=x + 2 * 3 * 4096) == INVALID            # the last row
    assert status(fn, out=3 * STEP - 4 * 4096) == INVALID         # over the positions
    for name in ("attn_rope_apply", "attn_rope_table", "attn_paged_append"):
        assert status(name, rope=abi.Rope()) == INVALID           # not set up
    halves = abi.attn_rope_init("halves", 64, 500000.0)
    assert status("attn_rope_table", rope=halves) == INVALID
    assert status("attn_rope_table", n_tok=0) == SHAPE and status("attn_rope_table", n_tok=262145) == SHAPE


def test_descriptions():
    fn = "attn_paged_create"
    for bad in (dict(n_pages=0), dict(page_size=0), dict(page_size=4), dict(page_size=20), dict(page_size=1048584),
                dict(page_size=-16)):
        assert status(fn, **bad) == SHAPE, bad
    assert status(fn, dtype=2) == INVALID and status(fn, dtype=-1) == INVALID
    assert status(fn, dtype=0) == INVALID                         # scales with bf16
    assert status(fn, dtype=0, v_scale=None) == INVALID
    assert status(fn, v_pages=2 * STEP) == INVALID                # one pool twice


def test_appends():
    fn = "attn_paged_append"
    for bad in (dict(T=0), dict(B=1024, T=257), dict(stride_b=-4096), dict(stride_t=-1024), dict(stride_b=1 << 31),
                dict(stride_t=1 << 31)):
        assert status(fn, **bad) == SHAPE, bad
    assert status(fn, stride_b=4100) == ALIGN and status(fn, stride_t=1028) == ALIGN
