"""Matrix products grouped by expert (beam_moe_grouped_gemm, _dgrad, _wgrad) against the same
sums in 64 bits.

Bound of every element.  The tensor core adds 16 products to its FP32 accumulator at a time,
aligned to the largest of the 17 and cut off below FP32's last bit (the next power of two
bounds the sum's growth): an error of at most 2^-22 of the magnitude in flight, which is at
most S = sum |a||b|, for each of the ceil(K / 16) additions.  Then one rounding to the output's
type, half a step: eps / 2 of the value, and half of the smallest step near zero."""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def bm():
    import sparse_moe_layer_fp32_b200 as m
    yield m
    m.beam_moe_check_operators()


def _draw(shape, kind, seed, scale=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(kind)


def _offsets(counts, first=0):
    return torch.tensor(np.concatenate([[first], first + np.cumsum(counts)]), dtype=torch.int32, device="cuda")


def _close(got, ref, size, terms, what=""):
    """got against the 64-bit ref; size: sum of the absolute products, terms: their number."""
    info = torch.finfo(got.dtype)
    acc = (terms + 15) // 16 * 2.0 ** -22 * size
    bound = acc + info.eps / 2 * (ref.abs() + acc) + info.smallest_normal * info.eps / 2
    off = (got.double() - ref).abs()
    assert bool((off <= bound).all()), (what, (off / bound).max().item(), off.max().item())


def _fwd_ref(x, w, counts, first=0):
    """(rows, reference, sum of absolute products) for each expert with rows."""
    a = first
    for e, c in enumerate(counts):
        if c:
            xe, we = x[a:a + c].double(), w[e].double()
            yield slice(a, a + c), xe @ we.t(), xe.abs() @ we.abs().t()
        a += c


SHAPES = [  # experts' rows, n, k
    ([1], 8, 8),
    ([5], 256, 64),
    ([0, 1, 0, 3], 128, 256),
    ([256], 512, 512),
    ([257, 31, 0, 33], 264, 328),
    ([64, 700, 3, 0, 129], 520, 1000),
    ([1, 2, 3, 4, 5, 6, 7, 8] * 8, 384, 72),
    ([2500, 100], 768, 136),
    ([17] * 40, 1536, 512),
]


@pytest.mark.parametrize("kind,out", [(BF16, BF16), (FP16, FP16), (BF16, FP32), (FP16, FP32)])
@pytest.mark.parametrize("counts,n,k", SHAPES)
def test_forward(bm, counts, n, k, kind, out):
    rows = sum(counts)
    x, w = _draw((rows, k), kind, 1), _draw((len(counts), n, k), kind, 2, 0.1)
    y = bm.beam_moe_grouped_gemm(x, w, _offsets(counts), out_dtype=out)
    assert y.dtype == out and y.shape == (rows, n)
    for r, ref, size in _fwd_ref(x, w, counts):
        _close(y[r], ref, size, k)


@pytest.mark.parametrize("kind,out", [(BF16, BF16), (FP16, FP16), (BF16, FP32)])
@pytest.mark.parametrize("counts,n,k", SHAPES)
def test_dgrad(bm, counts, n, k, kind, out):
    rows = sum(counts)
    dy, w = _draw((rows, n), kind, 3), _draw((len(counts), n, k), kind, 4, 0.1)
    dx = bm.beam_moe_grouped_gemm_dgrad(dy, w, _offsets(counts), out_dtype=out)
    assert dx.dtype == out and dx.shape == (rows, k)
    for r, ref, size in _fwd_ref(dy, w.transpose(1, 2), counts):
        _close(dx[r], ref, size, n)


@pytest.mark.parametrize("kind,out", [(BF16, BF16), (FP16, FP16), (BF16, FP32)])
@pytest.mark.parametrize("counts,n,k", SHAPES)
def test_wgrad(bm, counts, n, k, kind, out):
    rows = sum(counts)
    dy, x = _draw((rows, n), kind, 5), _draw((rows, k), kind, 6)
    dw = torch.full((len(counts), n, k), 7.0, dtype=out, device="cuda")
    bm.beam_moe_grouped_gemm_wgrad(dy, x, _offsets(counts), out=dw)
    a = 0
    for e, c in enumerate(counts):
        d, v = dy[a:a + c].double(), x[a:a + c].double()
        _close(dw[e], d.t() @ v, d.abs().t() @ v.abs(), max(c, 1), e)
        a += c


def test_nothing_to_do(bm):
    w = _draw((3, 16, 32), BF16, 7)
    none = torch.zeros(4, dtype=torch.int32, device="cuda")
    assert bm.beam_moe_grouped_gemm(_draw((0, 32), BF16, 8), w, none).shape == (0, 16)
    assert bm.beam_moe_grouped_gemm_dgrad(_draw((0, 16), BF16, 8), w, none).shape == (0, 32)
    dw = bm.beam_moe_grouped_gemm_wgrad(_draw((0, 16), BF16, 8), _draw((0, 32), BF16, 8), none)
    assert dw.shape == (3, 16, 32) and not dw.any()
    # rows, but no expert's: nothing is written
    y = torch.full((40, 16), 3.0, dtype=BF16, device="cuda")
    bm.beam_moe_grouped_gemm(_draw((40, 32), BF16, 9), w, none + 20, out=y)
    assert bool((y == 3.0).all())
    dw = bm.beam_moe_grouped_gemm_wgrad(_draw((40, 16), BF16, 8), _draw((40, 32), BF16, 8), none + 20)
    assert not dw.any()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_rows_of_others_stay_out(bm, bad):
    # rows before the first expert, behind the last one and another expert's rows hold values
    # that would spread: no other expert's result sees them, and the outputs' own rows there
    # stay as they were
    counts, first, rows, n, k = [37, 50, 0, 70], 11, 200, 264, 200
    x, dy = _draw((rows, k), BF16, 10), _draw((rows, n), BF16, 11)
    w = _draw((4, n, k), BF16, 12, 0.1)
    off = _offsets(counts, first)
    last = first + sum(counts)
    for t in (x, dy):
        t[:first] = bad
        t[last:] = bad
        t[first + 37:first + 87] = bad  # expert 1
    w[1] = bad
    y = torch.full((rows, n), 5.0, dtype=BF16, device="cuda")
    dx = torch.full((rows, k), 5.0, dtype=BF16, device="cuda")
    bm.beam_moe_grouped_gemm(x, w, off, out=y)
    bm.beam_moe_grouped_gemm_dgrad(dy, w, off, out=dx)
    dw = bm.beam_moe_grouped_gemm_wgrad(dy, x, off)
    for t in (y, dx):
        assert bool((t[:first] == 5.0).all()) and bool((t[last:] == 5.0).all())
        assert not bool(torch.isfinite(t[first + 37:first + 87]).any())
    for e, (r, ref, size) in zip((0, 1, 3), _fwd_ref(x, w, counts, first)):
        if e != 1:
            _close(y[r], ref, size, k)
    for e, (r, ref, size) in zip((0, 1, 3), _fwd_ref(dy, w.transpose(1, 2), counts, first)):
        if e != 1:
            _close(dx[r], ref, size, n)
    assert not bool(torch.isfinite(dw[1]).any()) and not dw[2].any()
    for e, a, c in ((0, first, 37), (3, first + 87, 70)):
        d, v = dy[a:a + c].double(), x[a:a + c].double()
        _close(dw[e], d.t() @ v, d.abs().t() @ v.abs(), c, e)


def test_ragged_ends_are_zeroed_in_time(bm):
    # wgrad: every second expert's rows are NaN and none ends on a multiple of 16, so that each
    # sum's last rows are followed by NaN; many times, with other work on the GPU
    counts = [1, 33, 15, 17, 250, 5, 300, 63, 65, 129, 7, 47] * 4
    n, k = 1536, 520
    x, dy = _draw((sum(counts), k), BF16, 60), _draw((sum(counts), n), BF16, 61)
    a = 0
    for e, c in enumerate(counts):
        if e % 2:
            x[a:a + c] = float("nan")
            dy[a:a + c] = float("inf")
        a += c
    off = _offsets(counts)
    first = bm.beam_moe_grouped_gemm_wgrad(dy, x, off)
    a = 0
    for e, c in enumerate(counts):
        if e % 2 == 0:
            d, v = dy[a:a + c].double(), x[a:a + c].double()
            _close(first[e], d.t() @ v, d.abs().t() @ v.abs(), c, e)
        a += c
    noise, side = torch.zeros(1 << 26, device="cuda"), torch.cuda.Stream()
    for i in range(200):
        with torch.cuda.stream(side):
            noise.add_(1.0)
        again = bm.beam_moe_grouped_gemm_wgrad(dy, x, off)
        assert torch.equal(again[::2], first[::2]), i


def test_row_strides(bm):
    counts, n, k = [40, 3, 90], 264, 136
    rows = sum(counts)
    x = _draw((rows, k + 24), FP16, 13)[:, 8:8 + k]  # starts on a 16-byte boundary, rows further apart
    dy = _draw((rows, n + 8), FP16, 14)[:, :n]
    w = _draw((3, n, k), FP16, 15, 0.1)
    off = _offsets(counts)
    whole = torch.full((rows, n + 16), 5.0, dtype=FP16, device="cuda")
    bm.beam_moe_grouped_gemm(x, w, off, out=whole[:, 8:8 + n])
    assert bool((whole[:, :8] == 5.0).all()) and bool((whole[:, 8 + n:] == 5.0).all())
    for r, ref, size in _fwd_ref(x, w, counts):
        _close(whole[r, 8:8 + n], ref, size, k)
    whole = torch.full((rows, k + 16), 5.0, dtype=FP32, device="cuda")
    bm.beam_moe_grouped_gemm_dgrad(dy, w, off, out=whole[:, 8:8 + k])
    assert bool((whole[:, :8] == 5.0).all()) and bool((whole[:, 8 + k:] == 5.0).all())
    for r, ref, size in _fwd_ref(dy, w.transpose(1, 2), counts):
        _close(whole[r, 8:8 + k], ref, size, n)
    same = bm.beam_moe_grouped_gemm_wgrad(dy.contiguous(), x.contiguous(), off)
    assert torch.equal(bm.beam_moe_grouped_gemm_wgrad(dy, x, off), same)


def test_bad_offsets_are_clamped(bm):
    # read as their running maximum within [0, rows]; no access leaves the buffers
    rows, n, k = 96, 72, 64
    x, w = _draw((rows, k), BF16, 16), _draw((5, n, k), BF16, 17, 0.1)
    off = torch.tensor([-7, 20, 10, 1 << 30, -(1 << 31), 50], dtype=torch.int32, device="cuda")
    y = bm.beam_moe_grouped_gemm(x, w, off)
    want = bm.beam_moe_grouped_gemm(x, w, torch.tensor([0, 20, 20, 96, 96, 96], dtype=torch.int32, device="cuda"))
    assert torch.equal(y, want)
    dw = bm.beam_moe_grouped_gemm_wgrad(y, x, off)
    assert not dw[1].any() and not dw[3].any() and not dw[4].any() and bool(torch.isfinite(dw).all())


def test_most_groups(bm):
    g = torch.Generator().manual_seed(18)
    counts = torch.randint(0, 4, (1024,), generator=g).tolist()
    n, k = 40, 24
    x, w = _draw((sum(counts), k), BF16, 19), _draw((1024, n, k), BF16, 20)
    y = bm.beam_moe_grouped_gemm(x, w, _offsets(counts))
    for r, ref, size in _fwd_ref(x, w, counts):
        _close(y[r], ref, size, k)
    dw = bm.beam_moe_grouped_gemm_wgrad(y, x, _offsets(counts), out_dtype=FP32)
    a = 0
    for e, c in enumerate(counts):
        d, v = y[a:a + c].double(), x[a:a + c].double()
        _close(dw[e], d.t() @ v, d.abs().t() @ v.abs(), max(c, 1), e)
        a += c


def test_output_past_32_bits(bm):
    # 2^31 elements are passed in y (forward) and in dy (wgrad)
    rows, n, k = 1_000_000, 2560, 8
    counts = [400_000, 599_990, 10]
    x, w = _draw((rows, k), BF16, 21), _draw((3, n, k), BF16, 22)
    y = bm.beam_moe_grouped_gemm(x, w, _offsets(counts))
    for e, a, b in ((0, 399_000, 400_000), (1, 400_000, 401_000), (1, 998_000, 999_990), (2, 999_990, rows)):
        xe, we = x[a:b].double(), w[e].double()
        _close(y[a:b], xe @ we.t(), xe.abs() @ we.abs().t(), k, (e, a))
    dw = bm.beam_moe_grouped_gemm_wgrad(y, x, _offsets(counts), out_dtype=FP32)
    d, v = y[999_990:].double(), x[999_990:].double()
    _close(dw[2], d.t() @ v, d.abs().t() @ v.abs(), 10)


def test_streams_and_a_replayed_graph(bm):
    counts, n, k = [30, 0, 200, 26], 264, 136
    rows = sum(counts)
    x, w = _draw((rows, k), BF16, 23), _draw((4, n, k), BF16, 24, 0.1)
    off = _offsets(counts)
    plain = [bm.beam_moe_grouped_gemm(x, w, off), bm.beam_moe_grouped_gemm_dgrad(_draw((rows, n), BF16, 25), w, off)]
    # two streams at once
    dy = _draw((rows, n), BF16, 25)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        got[0].append(bm.beam_moe_grouped_gemm(x, w, off, stream=streams[0]))
        got[1].append(bm.beam_moe_grouped_gemm_dgrad(dy, w, off, stream=streams[1]))
    torch.cuda.synchronize()
    assert all(torch.equal(v, plain[0]) for v in got[0]) and all(torch.equal(v, plain[1]) for v in got[1])
    # captured once, replayed with other rows and other borders
    y, dx = torch.empty_like(plain[0]), torch.empty_like(plain[1])
    dw = torch.empty_like(w)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bm.beam_moe_grouped_gemm(x, w, off, out=y)
        bm.beam_moe_grouped_gemm_dgrad(y, w, off, out=dx)
        bm.beam_moe_grouped_gemm_wgrad(y, x, off, out=dw)
    for counts in ([30, 0, 200, 26], [0, 256, 0, 0], [64, 64, 64, 64]):
        off.copy_(_offsets(counts))
        x.copy_(_draw((rows, k), BF16, sum(counts[:2])))
        graph.replay()
        want = bm.beam_moe_grouped_gemm(x, w, off)
        assert torch.equal(y, want)
        assert torch.equal(dx, bm.beam_moe_grouped_gemm_dgrad(want, w, off))
        assert torch.equal(dw, bm.beam_moe_grouped_gemm_wgrad(want, x, off))
        for r, ref, size in _fwd_ref(x, w, counts):
            _close(y[r], ref, size, k)


def test_gradients_against_differences(bm):
    # L = sum(c * y): dL/dx and dL/dw by the operators against central differences of L in 64
    # bits along random directions, L being linear in each operand (no truncation error)
    counts, n, k = [19, 0, 45], 72, 40
    rows = sum(counts)
    x, w, c = _draw((rows, k), BF16, 26), _draw((3, n, k), BF16, 27), _draw((rows, n), BF16, 28)
    off = _offsets(counts)
    dx = bm.beam_moe_grouped_gemm_dgrad(c, w, off, out_dtype=FP32)
    dw = bm.beam_moe_grouped_gemm_wgrad(c, x, off, out_dtype=FP32)

    def loss(xv, wv):
        return sum(((xv[r] @ wv[e].t()) * c[r].double()).sum() for e, r in ((0, slice(0, 19)), (2, slice(19, 64))))

    for seed in range(3):
        vx, vw = _draw((rows, k), FP32, 30 + seed).double(), _draw((3, n, k), FP32, 40 + seed).double()
        xd, wd = x.double(), w.double()
        for grad, num, size in (
                (dx, (loss(xd + vx, wd) - loss(xd - vx, wd)) / 2, (dx.double().abs() * vx.abs()).sum()),
                (dw, (loss(xd, wd + vw) - loss(xd, wd - vw)) / 2, (dw.double().abs() * vw.abs()).sum())):
            v = vx if grad is dx else vw
            # every gradient element is right to 5 steps of 2^-22 of its absolute sum, which is
            # at most ~8 times the element's own typical size here: 2^-17 of the summed sizes
            assert abs((grad.double() * v).sum() - num) <= 2.0 ** -17 * size


def test_refusals(bm):
    x, w = _draw((10, 32), BF16, 50), _draw((2, 16, 32), BF16, 51)
    off = _offsets([4, 6])
    dy = _draw((10, 16), BF16, 52)
    for call in (lambda: bm.beam_moe_grouped_gemm(x.half(), w, off),
                 lambda: bm.beam_moe_grouped_gemm(x.float(), w.float(), off),
                 lambda: bm.beam_moe_grouped_gemm(x, w, off.long()),
                 lambda: bm.beam_moe_grouped_gemm(x, w, off[:2]),
                 lambda: bm.beam_moe_grouped_gemm(x, w, off.cpu()),
                 lambda: bm.beam_moe_grouped_gemm(x[:, :24], w, off),
                 lambda: bm.beam_moe_grouped_gemm(x.t().contiguous().t(), w, off),
                 lambda: bm.beam_moe_grouped_gemm(x, w.transpose(1, 2), off),
                 lambda: bm.beam_moe_grouped_gemm(x, w, off, out=torch.empty(10, 24, dtype=BF16, device="cuda")),
                 lambda: bm.beam_moe_grouped_gemm_dgrad(x, w, off),
                 lambda: bm.beam_moe_grouped_gemm_wgrad(dy[:9], x, off)):
        with pytest.raises(ValueError):
            call()
    # more rows than 32 bits count (one row of memory seen many times)
    many = _draw((1, 32), BF16, 54).expand(2 ** 32 + 10, 32)
    with pytest.raises(bm.BeamMoeError) as err:
        bm.beam_moe_grouped_gemm(many, w, off)
    assert err.value.status == bm.ERR_UNSUPPORTED
    with pytest.raises(bm.BeamMoeError) as err:
        bm.beam_moe_grouped_gemm_wgrad(many[:, :16], many, off)
    assert err.value.status == bm.ERR_UNSUPPORTED
    wide = _draw((10, 34), BF16, 53)
    for call, status in ((lambda: bm.beam_moe_grouped_gemm(wide[:, 1:33], w, off), bm.ERR_INVALID_ARG),
                         (lambda: bm.beam_moe_grouped_gemm(wide[:, :32], w, off), bm.ERR_INVALID_ARG),
                         (lambda: bm.beam_moe_grouped_gemm(x, w, off, out_dtype=FP16), bm.ERR_INVALID_ARG),
                         (lambda: bm.beam_moe_grouped_gemm(x[:, :28].contiguous(), w[:, :, :28].contiguous(), off),
                          bm.ERR_UNSUPPORTED)):
        with pytest.raises(bm.BeamMoeError) as err:
            call()
        assert err.value.status == status


@pytest.mark.parametrize("counts,n,k", SHAPES)
def test_fp16_gradients_in_fp32(bm, counts, n, k):
    rows = sum(counts)
    dy, x, w = _draw((rows, n), FP16, 60), _draw((rows, k), FP16, 61), _draw((len(counts), n, k), FP16, 62, 0.1)
    dx = bm.beam_moe_grouped_gemm_dgrad(dy, w, _offsets(counts), out_dtype=FP32)
    dw = bm.beam_moe_grouped_gemm_wgrad(dy, x, _offsets(counts), out_dtype=FP32)
    assert dx.dtype == dw.dtype == FP32
    for r, ref, size in _fwd_ref(dy, w.transpose(1, 2), counts):
        _close(dx[r], ref, size, n)
    a = 0
    for e, c in enumerate(counts):
        d, v = dy[a:a + c].double(), x[a:a + c].double()
        _close(dw[e], d.t() @ v, d.abs().t() @ v.abs(), max(c, 1), e)
        a += c
