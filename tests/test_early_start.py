"""Kernels launched with programmatic stream serialisation start while the kernel before them may
still be writing their inputs.  Those that can come right behind a caller's kernel read the caller's
memory after their wait, and not through the read-only path (__ldg), which asks for memory that does
not change as long as the kernel runs."""

import os
import re

import pytest

FIRST = [("router.cu", "router_sgemm_kernel"), ("router_tc.cu", "router_tc_kernel"),
         ("grouped_gemm.cu", "grouped_gemm_kernel"), ("gemm_fp4.cu", "gemm_fp4_kernel"),
         ("quant_fp4.cu", "quantize_fp4_kernel"), ("quant_fp4.cu", "dequantize_fp4_kernel")]


def _body(text, name):
    """The text of a kernel's body, without comments."""
    text = re.sub(r"//[^\n]*", "", text)
    start = re.search(r"__global__[^;{]*\b" + name + r"\s*\(", text).end()
    at = text.index("{", start)
    depth = 0
    for i in range(at, len(text)):
        depth += (text[i] == "{") - (text[i] == "}")
        if depth == 0:
            return text[at:i + 1]
    raise AssertionError(name)


@pytest.mark.parametrize("source,kernel", FIRST)
def test_first_kernels_do_not_use_the_read_only_path(repo_root, source, kernel):
    with open(os.path.join(repo_root, "sparse_moe_layer_fp32_b200", "csrc", source)) as f:
        body = _body(f.read(), kernel)
    assert "pdl_wait()" in body
    assert "__ldg(" not in body and "ld.global.nc" not in body
