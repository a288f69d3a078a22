"""Outputs that share memory with an operand: the host's test against sets of addresses, and the
operators' refusals (answered before any CUDA call)."""

import ctypes
import os
import random
import subprocess

import pytest

import sparse_moe_layer_fp32_b200 as bm

SHIM = """
#include "overlap.h"
extern "C" int overlap(long a, long ar, long aw, long ap, long b, long br, long bw, long bp) {
  return beam::overlap({(const void*)a, ar, aw, ap}, {(const void*)b, br, bw, bp});
}
"""


@pytest.fixture(scope="module")
def overlap(repo_root, tmp_path_factory):
    at = tmp_path_factory.mktemp("overlap")
    (at / "shim.cpp").write_text(SHIM)
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-I",
                    os.path.join(repo_root, "sparse_moe_layer_fp32_b200", "csrc"), str(at / "shim.cpp"), "-o",
                    str(at / "shim.so")], check=True)
    f = ctypes.CDLL(str(at / "shim.so")).overlap
    f.argtypes = [ctypes.c_long] * 8
    return f


def _bytes(at, rows, width, pitch):
    return {at + r * pitch + c for r in range(rows) for c in range(width)}


def test_against_sets_of_addresses(overlap):
    rng = random.Random(1)
    seen = [0, 0]
    for _ in range(20000):
        pitch = rng.randint(1, 12)
        spans = []
        for _ in range(2):
            p = pitch if rng.random() < 0.6 else rng.randint(1, 12)
            spans.append((1000 + rng.randint(0, 60), rng.randint(1, 6), rng.randint(1, p), p))
        want = not _bytes(*spans[0]).isdisjoint(_bytes(*spans[1]))
        seen[want] += 1
        assert bool(overlap(*spans[0], *spans[1])) == want, spans
    assert min(seen) > 3000


def test_far_pitches_and_nothing(overlap):
    assert not overlap(0, 4, 4, 4, 1000, 4, 4, 4)                     # a null pointer is no matrix
    assert not overlap(1000, 0, 4, 4, 1000, 4, 4, 4)
    big = 1 << 40
    assert overlap(1000, 1 << 22, 16, big, 1000 + big, 1, 1, 1)       # beyond 62 bits in all
    assert not overlap(1000, 1 << 22, 16, big, 1016 + big, 1, 1, 1)
    assert overlap(1 << 46, 1 << 31, 512, 1024, (1 << 46) + 511, 1 << 31, 512, 1024)
    assert not overlap(1 << 46, 1 << 31, 512, 1024, (1 << 46) + 512, 1 << 31, 512, 1024)


BAD = bm.ERR_INVALID_ARG
P = 1 << 20  # addresses that nothing reads: every call below is refused
ROWS, N, K, GROUPS = 40, 16, 32, 2


@pytest.mark.parametrize("size,out_type", [(2, bm.TYPE_BF16), (4, bm.TYPE_FP32)])
def test_grouped_products_refuse(size, out_type):
    lib, t = bm.lib(), bm.TYPE_BF16
    x, w, off = P, 2 * P, 3 * P
    x_end, w_end = x + ROWS * K * 2, w + GROUPS * N * K * 2
    for y in (x - ROWS * N * size + 16, x + 16, x_end - 16, w, w_end - 16, off - 16, off):
        assert lib.beam_moe_grouped_gemm(x, K, w, off, ROWS, GROUPS, N, K, t, y, N, out_type, None) == BAD
    dy_end = x + ROWS * N * 2
    for dx in (x + 16, dy_end - 16, w_end - 16, off):
        assert lib.beam_moe_grouped_gemm_dgrad(x, N, w, off, ROWS, GROUPS, N, K, t, dx, K, out_type, None) == BAD
    for dw in (x + 16, dy_end - 16, w + 16, off, off - 16):
        assert lib.beam_moe_grouped_gemm_wgrad(x, N, w, K, off, ROWS, GROUPS, N, K, t, dw, out_type, None) == BAD
    # columns of one larger matrix that meet
    assert lib.beam_moe_grouped_gemm(x, 64, w, off, ROWS, GROUPS, N, K, t, x + (K - 8) * 2, 64 * 2 // size, out_type,
                                     None) == BAD


def test_fp4_refuses():
    lib, rows, cols = bm.lib(), 10, 64
    src, codes, sf, alpha = P, 2 * P, 3 * P, 4 * P

    def quantise(form, src=src, codes=codes, sf=sf, alpha_out=alpha):
        return lib.beam_moe_quantize_fp4(form, src, bm.TYPE_BF16, cols, rows, cols, 1.0, codes, 32, sf, 16, alpha_out,
                                         None)

    def back(form, codes=codes, sf=sf, alpha=alpha, out=src):
        return lib.beam_moe_dequantize_fp4(form, codes, 32, sf, 16, alpha, rows, cols, out, bm.TYPE_BF16, cols, None)

    for form in (bm.FP4_MX, bm.FP4_NV):
        assert quantise(form, codes=src + 16) == BAD
        assert quantise(form, sf=src + rows * cols * 2 - 16) == BAD
        assert quantise(form, sf=codes + 16) == BAD
        assert back(form, out=codes) == BAD
        assert back(form, out=sf - rows * cols * 2 + 16) == BAD
    assert quantise(bm.FP4_NV, alpha_out=src + 8) == BAD
    assert quantise(bm.FP4_NV, alpha_out=codes) == BAD
    assert quantise(bm.FP4_NV, alpha_out=sf + 16) == BAD
    assert back(bm.FP4_NV, alpha=src + 4) == BAD

    a, asf, b, bsf, al, be, out = (i * P for i in range(1, 8))
    for form in (bm.FP4_MX, bm.FP4_NV):
        for at in (a, a + 32 * 4 - 2, asf + 16, b - 2, bsf) + ((al, be + 2) if form == bm.FP4_NV else ()):
            assert lib.beam_moe_gemm_fp4(form, a, 32, asf, 16, al, b, 32, bsf, 16, be, 4, 8, 64, at, bm.TYPE_BF16, 8,
                                         None) == BAD
