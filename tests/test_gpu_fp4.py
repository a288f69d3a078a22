"""MXFP4 and NVFP4 on caller buffers: the quantiser bit for bit against the oracle, its inverse,
and the product of two quantised matrices against the same sum in 64 bits.

Bound of a product's element: the products of codes and scales are exact in the tensor core; a
sum is aligned to its largest term and cut off below FP32's last bit (the next power of two
bounds its growth), at most 2^-22 of S = sum |a||b| for each 16 terms; NVFP4's two tensor scales
multiply once each, 2^-24 of the value twice; then one rounding to the output's type."""

import os
import subprocess
import sys

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

from oracle import mxfp4, nvfp4  # noqa: E402

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
BLOCK = {"mxfp4": 32, "nvfp4": 16}


@pytest.fixture(scope="module")
def bm():
    import sparse_moe_layer_fp32_b200 as m
    yield m
    m.beam_moe_check_operators()


def _draw(shape, kind, seed, scale=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(kind)


def _oracle(x, fmt, alpha):
    v = x.float().cpu().numpy()
    if fmt == "mxfp4":
        return mxfp4.quantize_mxfp4(v)
    return nvfp4.quantize_nvfp4(v, np.float32(alpha))


def _values(codes, sf, fmt, alpha=None):
    """The 64-bit values of a quantised matrix."""
    c, s = codes.cpu().numpy(), sf.cpu().numpy()
    if fmt == "mxfp4":
        return torch.from_numpy(mxfp4.dequantize_mxfp4(c, s)).cuda()
    q = nvfp4.e2m1_decode(nvfp4.unpack_nibbles(c))
    d = nvfp4.e4m3_decode(s).repeat(16, axis=-1) * (1.0 if alpha is None else float(alpha))
    return torch.from_numpy(q * d).cuda()


def _norm(packed):
    c = nvfp4.unpack_nibbles(packed)
    c[c == 8] = 0
    return c


def _close(got, ref, size, k):
    info = torch.finfo(got.dtype)
    acc = (k + 15) // 16 * 2.0 ** -22 * size + 2.0 ** -23 * ref.abs()
    bound = acc + info.eps / 2 * (ref.abs() + acc) + info.smallest_normal * info.eps / 2
    off = (got.double() - ref).abs()
    assert bool((off <= bound).all()), ((off / bound).max().item(), off.max().item())


SIZES = [(1, 32), (1, 5120), (3, 96), (7, 288), (33, 256), (129, 544), (300, 1536)]


@pytest.mark.parametrize("kind", [BF16, FP16, FP32])
@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_quantise_and_back(bm, rows, cols, fmt, kind):
    x = _draw((rows, cols), kind, rows + cols)
    x[0, :32] = 0
    alpha = 0.0019 if fmt == "nvfp4" else None
    codes, sf, scale = bm.beam_moe_quantize_fp4(x, fmt, alpha=alpha)
    rc, rs = _oracle(x, fmt, alpha)
    np.testing.assert_array_equal(sf.cpu().numpy(), rs)
    np.testing.assert_array_equal(_norm(codes.cpu().numpy()), _norm(rc))
    assert (scale is None) == (fmt == "mxfp4") and (scale is None or scale.item() == np.float32(alpha))
    for out in (BF16, FP16, FP32):
        back = bm.beam_moe_dequantize_fp4(codes, sf, fmt, alpha=scale, out_dtype=out)
        want = _values(codes, sf, fmt, scale.item() if scale is not None else None)
        info = torch.finfo(out)
        # one FP32 rounding by alpha, one to the output's type
        bound = (info.eps / 2 + 2.0 ** -24) * 1.001 * want.abs() + info.smallest_normal * info.eps / 2
        assert back.dtype == out and bool(((back.double() - want).abs() <= bound).all())


def test_nvfp4_scale_found_on_the_device(bm):
    x = _draw((70, 352), BF16, 5, 3.0)
    codes, sf, scale = bm.beam_moe_quantize_fp4(x, "nvfp4")
    want = np.float32(x.float().abs().max().item()) / np.float32(2688.0)
    assert scale.item() == want
    rc, rs = _oracle(x, "nvfp4", want)
    np.testing.assert_array_equal(sf.cpu().numpy(), rs)
    np.testing.assert_array_equal(_norm(codes.cpu().numpy()), _norm(rc))
    # the framework's FP32 quantiser gives the same codes
    c2, s2, a2 = bm.beam_moe_quantize_nvfp4(x.float())
    assert a2.item() == scale.item() and torch.equal(s2, sf) and torch.equal(c2, codes)
    codes, sf, scale = bm.beam_moe_quantize_fp4(torch.zeros(4, 64, dtype=FP16, device="cuda"), "nvfp4")
    assert scale.item() == 0 and not codes.any() and not sf.any()
    assert not bm.beam_moe_dequantize_fp4(codes, sf, "nvfp4", alpha=scale).any()


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_non_finite_blocks_read_back_as_nan(bm, fmt):
    x = _draw((4, 128), FP32, 6)
    x[1, 40], x[2, 127], x[3, 0] = float("nan"), float("inf"), float("-inf")
    codes, sf, scale = bm.beam_moe_quantize_fp4(x, fmt)
    if fmt == "nvfp4":
        assert scale.item() == np.float32(x[torch.isfinite(x)].abs().max().item()) / np.float32(2688.0)
    back = bm.beam_moe_dequantize_fp4(codes, sf, fmt, alpha=scale, out_dtype=FP32)
    bad = ~torch.isfinite(x.view(4, -1, BLOCK[fmt])).all(-1, keepdim=True).expand(-1, -1, BLOCK[fmt]).reshape(4, 128)
    assert bool((torch.isnan(back) == bad).all())
    assert not codes.view(4, -1, BLOCK[fmt] // 2)[bad.view(4, -1, BLOCK[fmt])[..., 0]].any()


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_extreme_magnitudes(bm, fmt):
    # each block at another power of two, over FP32's whole range, and on the borders 6 * 2^e
    e = torch.arange(-149, 128, dtype=torch.float64, device="cuda")
    top = torch.cat([torch.exp2(e), 1.5 * torch.exp2(e[2:]), 1.4999 * torch.exp2(e[20:])]).float()
    x = top[:, None] * torch.linspace(-1, 1, 32, device="cuda")[None, :]
    x[:, 31] = top
    codes, sf, scale = bm.beam_moe_quantize_fp4(x, fmt, alpha=1.0 if fmt == "nvfp4" else None)
    rc, rs = _oracle(x, fmt, 1.0)
    np.testing.assert_array_equal(sf.cpu().numpy(), rs)
    np.testing.assert_array_equal(_norm(codes.cpu().numpy()), _norm(rc))


def test_quotients_near_every_e2m1_border(bm):
    # NVFP4 divides by scale * alpha; quotients on a border between two codes and a few units in
    # the last place around it, for many divisors, where the code hangs on the last bit of the
    # IEEE quotient; and the same through BF16 and FP16, whose quotients meet borders exactly
    rng = np.random.default_rng(77)
    borders = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], np.float32)
    for alpha in (np.float32(1.0), np.float32(0.37), np.float32(1e-3), np.float32(3.1e-5), np.float32(2.0 ** -9),
                  np.float32(3e-31), np.float32(2e31)):
        rows = []
        for code in rng.choice(np.arange(8, 127), 40, replace=False):
            d = np.float32(nvfp4.e4m3_decode(np.uint8(code)) * alpha)
            top = np.float32(np.float32(6.0) * d)  # gives the block this scale
            for b in borders:
                base = np.float32(b * d)
                near = [base]
                for to in (np.float32(0), np.float32(np.inf)):
                    v = base
                    for _ in range(7):
                        v = np.nextafter(v, to)
                        near.append(v)
                rows.append(np.array([top, *near], np.float32) * np.where(rng.random(16) < 0.5, -1, 1))
        v = np.stack(rows).reshape(-1, 32).astype(np.float32)
        for kind in (FP32, BF16, FP16):
            x = torch.from_numpy(v).cuda().to(kind)
            x = torch.where(torch.isfinite(x), x, 0)
            codes, sf, _ = bm.beam_moe_quantize_fp4(x, "nvfp4", alpha=float(alpha))
            rc, rs = _oracle(x, "nvfp4", alpha)
            np.testing.assert_array_equal(sf.cpu().numpy(), rs)
            np.testing.assert_array_equal(_norm(codes.cpu().numpy()), _norm(rc))


def test_strides_of_the_quantiser(bm):
    whole = _draw((50, 320), BF16, 7)
    x = whole[:, 32:256]
    for fmt in ("mxfp4", "nvfp4"):
        a = bm.beam_moe_quantize_fp4(x, fmt, alpha=0.002 if fmt == "nvfp4" else None)
        b = bm.beam_moe_quantize_fp4(x.contiguous(), fmt, alpha=0.002 if fmt == "nvfp4" else None)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        # a slice of the columns reads back as a slice
        n = BLOCK[fmt]
        part = bm.beam_moe_dequantize_fp4(a[0][:, 32:64], a[1][:, 64 // n:128 // n], fmt, alpha=a[2])
        assert torch.equal(part, bm.beam_moe_dequantize_fp4(*a[:2], fmt, alpha=a[2])[:, 64:128])


def test_bytes_between_the_rows_stay(bm):
    # codes and scales are written to their columns only
    lib, x = bm.lib(), _draw((20, 160), BF16, 8)
    codes = torch.full((20, 112), 0xA5, dtype=torch.uint8, device="cuda")
    sf = torch.full((20, 32), 0xA5, dtype=torch.uint8, device="cuda")
    for form, n in ((bm.FP4_MX, 5), (bm.FP4_NV, 10)):
        assert lib.beam_moe_quantize_fp4(form, x.data_ptr(), bm.TYPE_BF16, 160, 20, 160, 0.002, codes.data_ptr(), 112,
                                         sf.data_ptr(), 32, None, torch.cuda.current_stream().cuda_stream) == bm.OK
        torch.cuda.synchronize()
        assert bool((codes[:, 80:] == 0xA5).all()) and bool((sf[:, n:] == 0xA5).all())
        assert not bool((sf[:, :n] == 0xA5).all())


PRODUCTS = [(1, 1, 32), (1, 256, 256), (3, 40, 64), (33, 129, 288), (64, 512, 512), (257, 300, 96), (160, 264, 1056),
            (1, 5120, 1536), (700, 520, 1312), (2100, 136, 224),
            # a tile shared by several pairs: few tiles, long sums, up to 64 rows
            (1, 300, 2592), (5, 8192, 2560), (20, 520, 5120), (21, 1000, 5120), (32, 129, 5120), (64, 256, 2816),
            (65, 256, 2816)]


@pytest.mark.parametrize("out", [BF16, FP16, FP32])
@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("m,n,k", PRODUCTS)
def test_product(bm, m, n, k, fmt, out):
    a, b = _draw((m, k), BF16, 20), _draw((n, k), FP32, 21, 0.1)
    b *= torch.exp2(torch.randint(-3, 4, (n, 1), device="cuda").float())
    qa, qb = bm.beam_moe_quantize_fp4(a, fmt), bm.beam_moe_quantize_fp4(b, fmt)
    y = bm.beam_moe_gemm_fp4(qa[0], qa[1], qb[0], qb[1], fmt, alpha_a=qa[2], alpha_b=qb[2], out_dtype=out)
    assert y.shape == (m, n) and y.dtype == out
    va, vb = (_values(q[0], q[1], fmt, None if q[2] is None else q[2].item()) for q in (qa, qb))
    _close(y, va @ vb.t(), va.abs() @ vb.abs().t(), k)


@pytest.mark.parametrize("alpha_a,alpha_b,scale,code", [
    # the product of the scales underflows (to 0, or to a few bits) or overflows; the result does not
    (1e-23, 1e-23, 0x7E, 0x7), (3e-42, 0.4, 0x7E, 0x7), (2e-20, 3e-24, 0x7E, 0x7), (2e-24, 1e-21, 0x7E, 0x7),
    (-1e-23, 1e-23, 0x7E, 0x7), (2e38, 40.0, 0x01, 0x1), (30.0, 3e38, 0x01, 0x1), (1e20, -1e19, 0x01, 0x1),
    # ordinary ones, a zero, and results that overflow or vanish for good
    (0.37, 1.3, 0x38, 0x2), (0.0, 3e38, 0x7E, 0x7), (1e30, 1e30, 0x7E, 0x7), (1e-40, 1e-40, 0x7E, 0x7)])
@pytest.mark.parametrize("out", [BF16, FP16, FP32])
@pytest.mark.parametrize("m,n,k", [(1, 300, 2592), (70, 130, 288), (33, 129, 96)])
def test_tensor_scales_of_any_size(bm, m, n, k, out, alpha_a, alpha_b, scale, code):
    g = torch.Generator(device="cuda")
    g.manual_seed(50)
    codes = [torch.randint(0, 256, (r, k // 2), generator=g, device="cuda", dtype=torch.uint8) & 0x88 | 0x11 * code
             for r in (m, n)]
    for c in codes:
        c[-1] = 0  # sums of zero stay zero
    sf = [torch.full((r, (k // 16 + 15) // 16 * 16), scale, dtype=torch.uint8, device="cuda")[:, :k // 16]
          for r in (m, n)]
    al = [torch.tensor([v], dtype=FP32, device="cuda") for v in (alpha_a, alpha_b)]
    y = bm.beam_moe_gemm_fp4(codes[0], sf[0], codes[1], sf[1], "nvfp4", alpha_a=al[0], alpha_b=al[1], out_dtype=out)
    # the tensor scales multiply the reference's sums: those of codes and block scales are exact in 64
    # bits (multiples of 2^-20 below 2^35), where with the scales in every term a sum that cancels to
    # zero left a rounding of 1e-16 of terms of 1e66
    va, vb, by = _values(codes[0], sf[0], "nvfp4"), _values(codes[1], sf[1], "nvfp4"), al[0].item() * al[1].item()
    ref, size = (va @ vb.t()) * by, (va.abs() @ vb.abs().t()) * abs(by)
    top = torch.finfo(out).max
    over = ref.abs() > 2 * top  # (no reference lies between the type's largest value and twice that)
    assert not bool(((ref.abs() > top) & ~over).any())
    assert torch.equal(torch.isinf(y), over) and torch.equal(torch.sign(y)[over].double(), torch.sign(ref)[over])
    y, ref, size = (torch.where(over, 0, t) for t in (y, ref, size))
    _close(y, ref, size, k)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_product_strides_and_padding(bm, fmt):
    # operands that are column slices, an output inside a larger one, NaN bytes between the
    # rows' scales
    m, n, k, blk = 70, 200, 256, BLOCK[fmt]
    qa, qb = bm.beam_moe_quantize_fp4(_draw((m, 768), BF16, 22), fmt), bm.beam_moe_quantize_fp4(
        _draw((n, 768), BF16, 23), fmt)
    start = 512 if fmt == "mxfp4" else 256  # scale columns that start on 16 bytes
    ops = []
    for q in (qa, qb):
        sf = torch.full((q[1].shape[0], 64), 0xFF if fmt == "mxfp4" else 0x7F, dtype=torch.uint8, device="cuda")
        sf = sf[:, 16:16 + k // blk]
        sf.copy_(q[1][:, start // blk:(start + k) // blk])
        ops.append((q[0][:, start // 2:(start + k) // 2], sf, q[2]))
    want = bm.beam_moe_gemm_fp4(ops[0][0].contiguous(), ops[0][1], ops[1][0].contiguous(), ops[1][1], fmt,
                                alpha_a=ops[0][2], alpha_b=ops[1][2])
    va, vb = (_values(c, s, fmt, None if al is None else al.item()) for c, s, al in ops)
    _close(want, va @ vb.t(), va.abs() @ vb.abs().t(), k)
    for width, at in ((n + 16, 8), (n + 3, 1), (n + 4, 1), (n + 2, 2)):
        whole = torch.full((m, width), 5.0, dtype=BF16, device="cuda")
        bm.beam_moe_gemm_fp4(ops[0][0], ops[0][1], ops[1][0], ops[1][1], fmt, alpha_a=ops[0][2], alpha_b=ops[1][2],
                             out=whole[:, at:at + n])
        assert torch.equal(whole[:, at:at + n], want)
        assert bool((whole[:, :at] == 5.0).all()) and bool((whole[:, at + n:] == 5.0).all())


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_product_of_non_finite_blocks(bm, fmt):
    a, b = _draw((40, 320), BF16, 24), _draw((90, 320), BF16, 25)
    a[7, 100], b[50, 319] = float("nan"), float("inf")
    qa, qb = bm.beam_moe_quantize_fp4(a, fmt), bm.beam_moe_quantize_fp4(b, fmt)
    y = bm.beam_moe_gemm_fp4(qa[0], qa[1], qb[0], qb[1], fmt, alpha_a=qa[2], alpha_b=qb[2])
    bad = torch.zeros_like(y, dtype=torch.bool)
    bad[7], bad[:, 50] = True, True
    assert bool((torch.isnan(y) == bad).all())


def test_the_library_quantisers_weights(bm):
    # weights from beam_moe_quantize_nvfp4: their scales' rows need a multiple of 16 bytes
    w, x = _draw((384, 512), FP32, 26, 0.02), _draw((9, 512), BF16, 27)
    qw, qx = bm.beam_moe_quantize_nvfp4(w), bm.beam_moe_quantize_fp4(x, "nvfp4", alpha=0.002)
    y = bm.beam_moe_gemm_fp4(qx[0], qx[1], qw[0], qw[1], "nvfp4", alpha_a=qx[2], alpha_b=qw[2], out_dtype=FP32)
    va, vb = _values(qx[0], qx[1], "nvfp4", qx[2].item()), _values(qw[0], qw[1], "nvfp4", qw[2].item())
    _close(y, va @ vb.t(), va.abs() @ vb.abs().t(), 512)


def test_single_rows_of_any_pitch(bm):
    # the distance to a row that is not there does not matter
    for fmt in ("mxfp4", "nvfp4"):
        x = _draw((1, 67 + 64), BF16, 40)[:, :64]
        q = bm.beam_moe_quantize_fp4(x, fmt)
        assert all(torch.equal(a, b) for a, b in zip(q[:2], bm.beam_moe_quantize_fp4(x.contiguous(), fmt)[:2]))
        w = bm.beam_moe_quantize_fp4(_draw((24, 64), BF16, 41), fmt)
        y = bm.beam_moe_gemm_fp4(q[0], q[1].contiguous(), w[0], w[1], fmt, alpha_a=q[2], alpha_b=w[2])
        assert torch.equal(y, bm.beam_moe_gemm_fp4(q[0], q[1], w[0], w[1], fmt, alpha_a=q[2], alpha_b=w[2]))


def test_captured_before_any_other_call():
    # the first use of the kernels in a process may be inside a capture
    code = (
        "import torch, sparse_moe_layer_fp32_b200 as bm\n"
        "x = torch.randn(40, 256, device='cuda').bfloat16(); w = torch.randn(3, 64, 256, device='cuda').bfloat16()\n"
        "off = torch.tensor([0, 10, 10, 40], dtype=torch.int32, device='cuda')\n"
        "torch.cuda.synchronize(); g = torch.cuda.CUDAGraph()\n"
        "with torch.cuda.graph(g):\n"
        "    y = bm.beam_moe_grouped_gemm(x, w, off); dw = bm.beam_moe_grouped_gemm_wgrad(y, x, off)\n"
        "    q = bm.beam_moe_quantize_fp4(x, 'nvfp4'); z = bm.beam_moe_gemm_fp4(q[0], q[1], q[0], q[1], 'nvfp4')\n"
        "g.replay(); torch.cuda.synchronize()\n"
        "assert torch.equal(y, bm.beam_moe_grouped_gemm(x, w, off)), 'forward'\n"
        "assert torch.equal(dw, bm.beam_moe_grouped_gemm_wgrad(y, x, off)), 'wgrad'\n"
        "assert torch.equal(z, bm.beam_moe_gemm_fp4(q[0], q[1], q[0], q[1], 'nvfp4')), 'product'\n"
        "bm.beam_moe_check_operators(); print('fine')\n")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    done = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert done.returncode == 0 and "fine" in done.stdout, done.stderr[-2000:]


def test_nothing_to_do(bm):
    for fmt in ("mxfp4", "nvfp4"):
        codes, sf, alpha = bm.beam_moe_quantize_fp4(torch.empty(0, 64, dtype=BF16, device="cuda"), fmt)
        assert bm.beam_moe_dequantize_fp4(codes, sf, fmt, alpha=alpha).shape == (0, 64)
        q = bm.beam_moe_quantize_fp4(_draw((5, 64), BF16, 28), fmt)
        assert bm.beam_moe_gemm_fp4(codes, sf, q[0], q[1], fmt).shape == (0, 5)
        assert bm.beam_moe_gemm_fp4(q[0], q[1], codes, sf, fmt).shape == (5, 0)


def test_tensor_scale_of_an_empty_matrix(bm):
    # the scale that was given, else 0; written on the call's stream
    none, side = torch.empty(0, 64, dtype=BF16, device="cuda"), torch.cuda.Stream()
    assert bm.beam_moe_quantize_fp4(none, "nvfp4", alpha=0.002)[2].item() == np.float32(0.002)
    assert bm.beam_moe_quantize_fp4(none, "nvfp4")[2].item() == 0
    scale = bm.beam_moe_quantize_fp4(none, "nvfp4", alpha=0.002, stream=side)[2]
    side.synchronize()
    assert scale.item() == np.float32(0.002)


def test_streams_and_a_replayed_graph(bm):
    m, n, k = 70, 300, 544
    x, w = _draw((m, k), BF16, 29), _draw((n, k), BF16, 30)
    for fmt in ("mxfp4", "nvfp4"):
        qw = bm.beam_moe_quantize_fp4(w, fmt)

        def linear(v, out=None, stream=None):
            q = bm.beam_moe_quantize_fp4(v, fmt, stream=stream)
            return bm.beam_moe_gemm_fp4(q[0], q[1], qw[0], qw[1], fmt, alpha_a=q[2], alpha_b=qw[2], out=out,
                                        out_dtype=BF16, stream=stream)

        want = linear(x)
        streams = [torch.cuda.Stream() for _ in range(3)]
        torch.cuda.synchronize()
        got = []
        for i in range(15):
            with torch.cuda.stream(streams[i % 3]):
                got.append(linear(x))
        torch.cuda.synchronize()
        assert all(torch.equal(g, want) for g in got)
        out = torch.empty_like(want)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            linear(x, out)
        for seed in (31, 32):
            x.copy_(_draw((m, k), BF16, seed))
            graph.replay()
            assert torch.equal(out, linear(x))


def test_refusals(bm):
    x = _draw((4, 64), BF16, 33)
    codes, sf, alpha = bm.beam_moe_quantize_fp4(x, "nvfp4")
    for call in (lambda: bm.beam_moe_quantize_fp4(x, "fp4"),
                 lambda: bm.beam_moe_quantize_fp4(x.double(), "mxfp4"),
                 lambda: bm.beam_moe_quantize_fp4(x.t(), "mxfp4"),
                 lambda: bm.beam_moe_quantize_fp4(x.cpu(), "mxfp4"),
                 lambda: bm.beam_moe_quantize_fp4(x, "nvfp4", alpha=-1.0),
                 lambda: bm.beam_moe_quantize_fp4(x, "nvfp4", alpha=float("nan")),
                 lambda: bm.beam_moe_dequantize_fp4(codes, sf, "mxfp4"),
                 lambda: bm.beam_moe_dequantize_fp4(codes.int(), sf, "nvfp4"),
                 lambda: bm.beam_moe_dequantize_fp4(codes, sf, "nvfp4", alpha=alpha.double()),
                 lambda: bm.beam_moe_gemm_fp4(codes, sf, codes[:, :16], sf[:, :2], "nvfp4"),
                 lambda: bm.beam_moe_gemm_fp4(codes, sf, codes, sf[:3], "nvfp4"),
                 lambda: bm.beam_moe_gemm_fp4(codes, sf, codes, sf, "nvfp4", alpha_a=torch.ones(1)),
                 lambda: bm.beam_moe_gemm_fp4(codes, sf, codes, sf, "nvfp4", out=torch.empty(4, 5, device="cuda"))):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(bm.BeamMoeError) as err:  # more rows than 32 bits count
        bm.beam_moe_gemm_fp4(codes[:1].expand(2 ** 32 + 4, -1), sf[:1].expand(2 ** 32 + 4, -1), codes, sf, "nvfp4")
    assert err.value.status == bm.ERR_UNSUPPORTED
    for call, status in ((lambda: bm.beam_moe_quantize_fp4(x[:, :48].contiguous(), "nvfp4"), bm.ERR_UNSUPPORTED),
                         (lambda: bm.beam_moe_quantize_fp4(x[:, 1:33], "mxfp4"), bm.ERR_INVALID_ARG),
                         # scale rows 4 bytes apart
                         (lambda: bm.beam_moe_gemm_fp4(codes, sf.contiguous(), codes, sf, "nvfp4"),
                          bm.ERR_INVALID_ARG)):
        with pytest.raises(bm.BeamMoeError) as err:
            call()
        assert err.value.status == status
