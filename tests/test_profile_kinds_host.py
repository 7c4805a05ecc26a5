"""The per-kernel profile as programs call it that were built with this header, and with one that
had fewer kernel kinds (no GPU needed)."""
import ctypes
import os
import re
import shutil
import subprocess

import pytest

from transformer_gqa_attention_gb300 import _build, abi

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_the_binding_names_every_kind():
    src = open(os.path.join(ROOT, "include", "gqa_attn.h")).read()
    assert int(re.search(r"GQA_KERNEL_KINDS = (\d+)", src).group(1)) == len(abi.KERNEL_KINDS)


def test_null_context_and_negative_counts_are_refused():
    _build.build()
    ms, n = (ctypes.c_double * 13)(*[-1.0] * 13), (ctypes.c_int * 13)(*[-1] * 13)
    L = abi.lib()
    assert L.attn_profile_end(None, ms, n, None) == 1
    assert L.attn_profile_end_kinds(None, ms, n, 13, None) == 1
    assert L.attn_profile_end_kinds(ctypes.c_void_p(0x10000), ms, n, -1, None) == 1  # before the context is used
    assert list(ms) == [-1.0] * 13 and list(n) == [-1] * 13


@pytest.mark.skipif(shutil.which("gcc") is None, reason="needs gcc")
def test_a_program_built_with_the_header_asks_for_its_own_number_of_kinds():
    prog = "#include <gqa_attn.h>\nint f(gqa_ctx *c, double *m, int *n) { return attn_profile_end(c, m, n, 0); }\n"
    out = subprocess.run(["gcc", "-E", "-P", "-I", os.path.join(ROOT, "include"), "-"], input=prog, text=True,
                         capture_output=True, check=True).stdout
    assert "return attn_profile_end_kinds(c, m, n, GQA_KERNEL_KINDS, 0);" in out
    subprocess.run(["gcc", "-fsyntax-only", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), "-xc", "-"], input=prog,
                   text=True, check=True)
