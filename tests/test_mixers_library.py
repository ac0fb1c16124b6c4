"""What the built library holds of the mixers' kernels: the variants that a call reaches, and no others."""

import os
import re

import pytest

import packed_varlen_gated_amd as pkv


@pytest.fixture(scope="module")
def names():
    if not os.path.exists(pkv.LIB_PATH):
        from packed_varlen_gated_amd import build
        build.build(verbose=False)
    return open(pkv.LIB_PATH, "rb").read()


def _variants(names, kernel):
    """{(type, head dimensions)} of a kernel's instances, from their mangled names."""
    found = re.findall(kernel.encode() + rb"I(DF16b|f)Li(\d+)E(?:Li(\d+)E)?", names)
    return {(("bf16" if t == b"DF16b" else "f32"),) + tuple(int(d) for d in dims if d) for t, *dims in found}


@pytest.mark.parametrize("kernel", ["attn_simple_fwd", "attn_simple_dq", "attn_simple_dkv"])
def test_attention_off_the_bf16_matrix_path(names, kernel):
    assert _variants(names, kernel) == {("f32", 32), ("f32", 64), ("f32", 128), ("bf16", 32)}


def test_linear_token_by_token(names):
    dims = (32, 64, 128)
    assert _variants(names, "linear_serial_kernel") == (
        {("f32", a, b) for a in dims for b in dims} | {("bf16", a, b) for a in dims for b in dims if 32 in (a, b)})
