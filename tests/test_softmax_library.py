"""What the built library holds of the softmax layer's kernels: the variants that a call reaches, and no others."""

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


def _variants(names, kernel, pattern):
    """{template arguments} of a kernel's instances, from their mangled names."""
    found = re.findall(rb"\d" + kernel.encode() + b"I" + pattern + b"E", names)
    return {tuple(x.decode() for x in f) if isinstance(f, tuple) else f.decode() for f in found}


TYPES = {("f", "32"), ("f", "64"), ("f", "128"), ("DF16b", "32")}


def test_windowed_forward(names):
    assert _variants(names, "attn_fwd_kernel", rb"Li(\d+)ELi(\d+)ELb([01])E") == {
        (d, s, w) for d in ("64", "128") for s, w in (("1", "0"), ("2", "0"), ("1", "1"))}


def test_windowed_reverse(names):
    assert _variants(names, "attn_window_dq_kernel", rb"Li(\d+)E") == {"64", "128"}
    assert _variants(names, "attn_window_dkv_kernel", rb"Li(\d+)ELi(\d+)ELb([01])E") == {
        (d, k, f) for d in ("64", "128") for k, f in (("1", "0"), ("2", "0"), ("4", "0"), ("4", "1"))}


@pytest.mark.parametrize("kernel", ["attn_simple_fwd", "attn_simple_dq", "attn_simple_dkv"])
def test_windows_off_the_bf16_matrix_path(names, kernel):
    assert _variants(names, kernel, rb"(DF16b|f)Li(\d+)ELb([01])E") == {t + (w,) for t in TYPES for w in "01"}


def test_paged(names):
    assert _variants(names, "attn_paged_kernel", rb"Li(\d+)ELb([01])E") == {(d, b) for d in ("64", "128") for b in "01"}
    assert _variants(names, "attn_paged_join_kernel", rb"Li(\d+)E") == {"64", "128"}
    for kernel in ("attn_paged_simple_kernel", "attn_paged_simple_join_kernel"):
        assert _variants(names, kernel, rb"(DF16b|f)Li(\d+)E") == TYPES


def test_norms_with_rotation(names):
    every = {(t, d, i) for t in ("f", "DF16b") for d in ("32", "64", "128") for i in "01"}
    assert _variants(names, "qk_norm_rope_kernel", rb"(DF16b|f)Li(\d+)ELb([01])E") == every
    assert _variants(names, "qk_norm_rope_bwd_kernel", rb"(DF16b|f)Li(\d+)ELb([01])E") == every
    assert _variants(names, "qk_norm_rope_dw_kernel", rb"Li(\d+)E") == {"32", "64", "128"}
