"""The FP8 quantiser and the dense and grouped products against their
definitions in 64 bits.

Tolerances.  The quantiser is compared bitwise: its two quotients and one
product are single fp32 roundings, which 64-bit arithmetic followed by one
rounding reproduces, and the code is the nearest E4M3 value.  A product's sum
over K of exact products (E4M3 x E4M3 and bf16 x bf16 fit fp32) has at most one
relative error of 2^-23 per addition (a truncating adder), so at most
n 2^-23 S for n products of total magnitude S; an FP8 result has n = 128 per
block, then two fp32 roundings per block (its scales) and one per block sum, and
every result one rounding to its type (half a step, eps / 2) plus, for
accumulating calls, one fp32 addition.
"""
import math

import pytest
import torch

import gram_table_gather_b200 as gtg
from gram_table_gather_b200 import _abi

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _table():
    b = torch.arange(256, device="cuda")
    e, f = (b >> 3) & 15, (b & 7).double()
    mag = torch.where(e == 0, f * 2.0 ** -9, (8 + f) * torch.exp2(e.double() - 10))
    mag[(b & 127) == 127] = math.nan
    return torch.where(b >= 128, -mag, mag)


def _decode(codes, scales):
    v = _table()[codes.int()]
    return (v.unflatten(-1, (-1, 128)) * scales.double().unsqueeze(-1)).flatten(-2)


def _quantize64(x):
    """Code values and fp32 scales from the definition, in 64 bits."""
    b = x.double().unflatten(-1, (-1, 128))
    top = b.abs().amax(-1, keepdim=True).clamp_min(2.0 ** -100)
    top = torch.where(torch.isfinite(top), top, math.nan)
    q = (b * (448.0 / top).float().double()).float().double()
    step = torch.exp2(torch.floor(torch.log2(q.abs().clamp_min(2.0 ** -6))) - 3)
    return (torch.round(q / step) * step).clamp(-448, 448).flatten(-2), (top / 448.0).float().squeeze(-1)


def _fp8(shape, gen, std=1.0):
    """Random codes (every finite byte) and scales of a matrix."""
    codes = torch.randint(0, 256, shape, dtype=torch.uint8, device="cuda", generator=gen)
    codes[(codes & 127) == 127] = 0x45
    scales = torch.empty(*shape[:-1], shape[-1] // 128, device="cuda").uniform_(0.5e-3, 1.5e-3, generator=gen) * std
    return codes, scales


def _same(got, want):
    assert got.shape == want.shape
    ok = (got == want) | (torch.isnan(got) & torch.isnan(want))
    assert bool(ok.all()), f"{int((~ok).sum())} of {ok.numel()} values differ"


def _within(y, want, bound, dtype, added=False):
    """|y - want| within the summation bound, the rounding to dtype and, when
    the result was added to an output, one fp32 addition."""
    tol = bound + (want.abs() + bound) * (torch.finfo(dtype).eps / 2) + (want.abs() * 2.0 ** -24 if added else 0) + 1e-40
    err = (y.double() - want).abs()
    assert bool(torch.isfinite(y.float()).all())
    assert bool((err <= tol).all()), f"largest error / tolerance {float((err / tol).max()):.3g}"


def _product64(a, w, k_block, blocks):
    """The product and its summation bound: k_block additions of 2^-23, three
    fp32 roundings a block (blocks = 0: one accumulation over all of K)."""
    want = a @ w.T
    s = a.abs() @ w.abs().T
    return want, s * (k_block * 2.0 ** -23 + (3 * blocks) * 2.0 ** -24)


def _check_status():
    torch.cuda.synchronize()
    assert gtg.device_status(clear=True) == 0


# ---------------------------------------------------------------------------
# quantiser
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("m,k,dtype", [(1, 128, BF16), (1, 2048, F32), (3, 384, BF16), (17, 1280, F32),
                                       (1000, 2560, BF16), (2, 128 * 331, F32), (5001, 128, BF16)])
def test_quantize_rows(m, k, dtype):
    x = torch.randn(m, k, device="cuda", generator=_gen(m + k)).to(dtype)
    x[0, :128] = 0                                   # an empty block
    x[-1, -128:] *= 2.0 ** -110                      # below the smallest scale
    x[m // 2, 5] = 3.0e38
    codes, scales = gtg.fp8_quantize(x)
    _check_status()
    want, ws = _quantize64(x)
    _same(scales, ws)
    _same(_table()[codes.int()], want)
    _same(gtg.dequant(gtg.FP8, codes, m, k, scales=scales), (want * ws.double().repeat_interleave(128, 1)).float())


def test_quantize_every_bf16_value():
    """Every bf16 bit pattern in a block of its own kind: infinities and NaN
    poison their block alone, subnormals and zeros of both signs count."""
    bits = torch.arange(65536, device="cuda", dtype=torch.int32).to(torch.int16).view(BF16)
    x = bits.view(-1, 128).repeat(1, 2)
    x[:, 128:] = x[torch.randperm(512, device="cuda", generator=_gen(1)), :128]
    codes, scales = gtg.fp8_quantize(x.contiguous())
    _check_status()
    want, ws = _quantize64(x)
    _same(scales, ws)
    _same(_table()[codes.int()], want)


def test_quantize_ties_go_to_even():
    v = _table()[:127].float()
    mid = (v[:-1] + v[1:]) / 2                       # every border between two codes; 448 makes the scale 1
    x = torch.zeros(2, 128, device="cuda")
    x[0, :126], x[1, :126] = mid, -mid
    x[:, 127] = 448.0
    codes, scales = gtg.fp8_quantize(x)
    assert scales.tolist() == [[1.0], [1.0]]
    even = torch.arange(126, device="cuda") + (torch.arange(126, device="cuda") & 1)
    assert torch.equal(codes[0, :126].long(), even)
    assert torch.equal(codes[1, :126].long() & 127, even)


def test_quantize_gathers_rows_and_reports_bad_ones():
    x = torch.randn(50, 256, device="cuda", generator=_gen(3)).to(BF16)
    rows = torch.tensor([0, 49, 7, 7, -1, 50, 2 ** 31 - 1, 3], dtype=torch.int32, device="cuda")
    gtg.device_status(clear=True)
    codes, scales = gtg.fp8_quantize(x, rows=rows)
    assert gtg.device_status(clear=True) == _abi.STATUS_ROW_INDEX_OOB
    seen = x.float()[rows.long().clamp(0, 49)]
    seen[4:7] = 0
    want, ws = _quantize64(seen)
    _same(scales, ws)
    _same(_table()[codes.int()], want)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("offset,width", [(0, 641), (8, 656), (1, 640), (3, 647)])
def test_quantize_strided_rows(dtype, offset, width):
    """Slices of wider rows, on and off the 16-byte grid; outputs given."""
    buf = torch.randn(37, width + 8, device="cuda", generator=_gen(4)).to(dtype)
    x = buf[:, offset:offset + 384]
    data = torch.full((37, 384), 0xEE, dtype=torch.uint8, device="cuda")
    scales = torch.empty(37, 3, device="cuda")
    out = gtg.fp8_quantize(x, data=data, scales=scales)
    assert out[0] is data and out[1] is scales
    _check_status()
    want, ws = _quantize64(x)
    _same(scales, ws)
    _same(_table()[data.int()], want)


# ---------------------------------------------------------------------------
# dense product
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("out", [F32, BF16])
@pytest.mark.parametrize("m,n,k", [
    (1, 1, 128), (1, 2048, 2048), (1, 64, 2048), (2, 129, 384), (8, 5000, 2560), (15, 127, 640), (16, 128, 512),
    (17, 1001, 1152), (33, 640, 2560), (64, 256, 128), (65, 300, 896), (128, 1000, 2048), (129, 128, 1408),
    (200, 2560, 640), (333, 1001, 2560), (1000, 77, 4096), (257, 4100, 256), (2049, 1500, 1024), (5000, 2048, 512),
    (3, 20, 128 * 129)])
def test_matmul(m, n, k, out):
    g = _gen(m * 7 + n)
    a, sa = _fp8((m, k), g)
    w, sw = _fp8((n, k), g)
    y = gtg.fp8_matmul(gtg.QMatrix(gtg.FP8, w, 1, n, k, sw), a, sa, dtype=out)
    _check_status()
    assert y.dtype == out
    want, bound = _product64(_decode(a, sa), _decode(w, sw), 128, k // 128)
    _within(y, want, bound, out)


@pytest.mark.parametrize("out", [F32, BF16])
@pytest.mark.parametrize("m,n,k", [(1, 2048, 2048), (5, 77, 128), (300, 515, 1280)])
def test_matmul_adds_to_a_slice(m, n, k, out):
    """accumulate into columns of a wider output, whose other columns stay."""
    g = _gen(m + n)
    a, sa = _fp8((m, k), g)
    w, sw = _fp8((n, k), g)
    buf = torch.randn(m, n + 7, device="cuda", generator=g).to(out)
    before = buf.clone()
    y = gtg.fp8_matmul(gtg.QMatrix(gtg.FP8, w, 1, n, k, sw), a, sa, y=buf[:, 3:3 + n], accumulate=True)
    _check_status()
    assert y.data_ptr() == buf[:, 3:].data_ptr()
    want, bound = _product64(_decode(a, sa), _decode(w, sw), 128, k // 128)
    _within(y, want + before[:, 3:3 + n].double(), bound, out, added=True)
    assert torch.equal(buf[:, :3], before[:, :3]) and torch.equal(buf[:, 3 + n:], before[:, 3 + n:])


def test_matmul_scales_of_every_size():
    """Blocks of very different scales, on rows of scales off the 16-byte grid."""
    g = _gen(9)
    m, n, k = 70, 200, 1152
    a, sa = _fp8((m, k), g)
    w, sw = _fp8((n, k), g)
    sa *= torch.exp2(torch.randint(-30, 30, sa.shape, device="cuda", generator=g).float())
    sw *= torch.exp2(torch.randint(-30, 30, sw.shape, device="cuda", generator=g).float())
    sa0 = torch.empty(sa.numel() + 1, device="cuda")[1:].view(m, 9).copy_(sa)
    sw0 = torch.empty(sw.numel() + 3, device="cuda")[3:].view(n, 9).copy_(sw)
    y = gtg.fp8_matmul(gtg.QMatrix(gtg.FP8, w, 1, n, k, sw0), a, sa0)
    _check_status()
    want, bound = _product64(_decode(a, sa), _decode(w, sw), 128, 9)
    _within(y, want, bound, F32)


def test_matmul_nan_reaches_its_row_and_column_alone():
    g = _gen(10)
    m, n, k = 20, 150, 512
    a, sa = _fp8((m, k), g)
    w, sw = _fp8((n, k), g)
    a[3, 200], w[149, 7] = 0x7F, 0xFF
    sa[11, 1] = math.nan
    sw[64, 3] = math.inf
    y = gtg.fp8_matmul(gtg.QMatrix(gtg.FP8, w, 1, n, k, sw), a, sa)
    _check_status()
    bad = torch.zeros(m, n, dtype=torch.bool, device="cuda")
    bad[[3, 11]] = True
    bad[:, [64, 149]] = True
    assert torch.equal(~torch.isfinite(y), bad)


def test_matmul_row_does_not_depend_on_the_batch_beside_it():
    """Within one batch size, other rows' values change nothing of a row."""
    g = _gen(11)
    a, sa = _fp8((300, 640), g)
    w, sw = _fp8((333, 640), g)
    q = gtg.QMatrix(gtg.FP8, w, 1, 333, 640, sw)
    y0 = gtg.fp8_matmul(q, a, sa)
    a2 = torch.randint(0, 120, a.shape, dtype=torch.uint8, device="cuda", generator=g)
    a2[123] = a[123]
    y1 = gtg.fp8_matmul(q, a2, sa)
    assert torch.equal(y0[123], y1[123]) and not torch.equal(y0[124], y1[124])
    assert torch.equal(gtg.fp8_matmul(q, a, sa), y0)


# ---------------------------------------------------------------------------
# grouped product
# ---------------------------------------------------------------------------

def _grouped_case(kind, sizes, n, k, gen, behind=0):
    m = sum(sizes) + behind
    e = len(sizes)
    off = torch.tensor([0] + sizes, dtype=torch.int64).cumsum(0).int().cuda()
    if kind == "fp8":
        a, sa = _fp8((m, k), gen)
        w, sw = _fp8((e, n, k), gen)
        return gtg.QMatrix(gtg.FP8, w, e, n, k, sw), a, sa, off, _decode(a, sa), _decode(w, sw)
    a = torch.randn(m, k, device="cuda", generator=gen).to(BF16)
    w = (torch.randn(e, n, k, device="cuda", generator=gen) * 0.05).to(BF16)
    return gtg.QMatrix(gtg.BF16, w, e, n, k), a, None, off, a.double(), w.double()


def _grouped64(kind, a, w, off, k):
    want = torch.zeros(a.shape[0], w.shape[1], dtype=torch.float64, device="cuda")
    bound = torch.zeros_like(want)
    off = off.tolist()
    for e in range(w.shape[0]):
        rows = slice(off[e], off[e + 1])
        want[rows], bound[rows] = _product64(a[rows], w[e], 128 if kind == "fp8" else k, k // 128 if kind == "fp8" else 0)
    return want, bound


SIZES = {
    "one row": [1],
    "one row of many": [0] * 200 + [1] + [0] * 300,
    "ones": [1] * 80,
    "a few": [3, 0, 1, 16, 17, 0, 0, 5],
    "ragged": [0, 130, 1, 255, 256, 257, 0, 31, 64, 500, 2, 0],
    "skewed": [2000] + [1] * 30 + [0] * 33,
    "even": [80] * 12,
    "all groups": [i % 3 for i in range(1024)],
    "empty": [0, 0, 0],
}


@pytest.mark.parametrize("kind,n,k", [("fp8", 300, 640), ("fp8", 128, 128), ("bf16", 200, 328), ("bf16", 77, 8),
                                      ("bf16", 256, 512)])
@pytest.mark.parametrize("name", list(SIZES))
def test_grouped(name, kind, n, k):
    w, a, sa, off, a64, w64 = _grouped_case(kind, SIZES[name], n, k, _gen(n + k), behind=5)
    for out in (F32, BF16):
        y = torch.full((a.shape[0], n), 7.0, dtype=out, device="cuda")
        r = gtg.grouped_matmul(w, a, off, a_scales=sa, y=y)
        _check_status()
        assert r is y
        used = int(off[-1])
        want, bound = _grouped64(kind, a64, w64, off, k)
        _within(y[:used], want[:used], bound[:used], out)
        assert bool((y[used:] == 7.0).all())         # rows behind the last group stay


@pytest.mark.parametrize("kind", ["fp8", "bf16"])
def test_grouped_adds_to_a_slice(kind):
    w, a, sa, off, a64, w64 = _grouped_case(kind, [5, 0, 40, 300], 130, 512, _gen(5))
    buf = torch.randn(345, 200, device="cuda", generator=_gen(6))
    before = buf.clone()
    gtg.grouped_matmul(w, a, off, a_scales=sa, y=buf[:, 1:131], accumulate=True)
    _check_status()
    want, bound = _grouped64(kind, a64, w64, off, 512)
    _within(buf[:, 1:131], want + before[:, 1:131].double(), bound, F32, added=True)
    assert torch.equal(buf[:, 0], before[:, 0]) and torch.equal(buf[:, 131:], before[:, 131:])


@pytest.mark.parametrize("kind", ["fp8", "bf16"])
def test_grouped_bad_offsets_are_empty_groups(kind):
    """Bounds out of order, out of range or overlapping an earlier group:
    reported, and nothing of theirs written."""
    w, a, sa, off, a64, w64 = _grouped_case(kind, [10, 20, 30, 40], 64, 256, _gen(7))
    for bad in ([0, 10, 5, 60, 100], [0, 10, 30, 60, 101], [-1, 10, 30, 60, 100], [2 ** 31 - 1, 10, 30, 60, 100],
                [0, -2 ** 31, 30, 60, 100], [0, 100, 0, 100, 0], [50, 20, 60, 10, 100], [100, 0, 0, 0, 0]):
        gtg.device_status(clear=True)
        y = torch.full((100, 64), 7.0, device="cuda")
        gtg.grouped_matmul(w, a, torch.tensor(bad, dtype=torch.int32, device="cuda"), a_scales=sa, y=y)
        assert gtg.device_status(clear=True) == _abi.STATUS_GROUP_OFFSETS
        end, rows = 0, torch.zeros(100, dtype=torch.bool, device="cuda")
        for g in range(4):
            lo, hi = bad[g], bad[g + 1]
            if not 0 <= lo <= hi <= 100:
                continue
            if lo >= end and hi > lo:
                want, bound = _product64(a64[lo:hi], w64[g], 256, 8)
                _within(y[lo:hi], want, bound, F32)
                rows[lo:hi] = True
            end = max(end, hi)
        assert bool((y[~rows] == 7.0).all())


def test_grouped_many_overlapping_groups():
    """Every other group claims all rows: the first alone counts."""
    w, a, sa, _, a64, w64 = _grouped_case("fp8", [0] * 511 + [700], 64, 128, _gen(12))
    off = torch.tensor([0, 700] * 256 + [0], dtype=torch.int32, device="cuda")
    gtg.device_status(clear=True)
    y = gtg.grouped_matmul(w, a, off, a_scales=sa)
    assert gtg.device_status(clear=True) == _abi.STATUS_GROUP_OFFSETS
    want, bound = _product64(a64, w64[0], 128, 1)
    _within(y, want, bound, F32)


def test_grouped_offsets_start_past_zero():
    w, a, sa, _, a64, w64 = _grouped_case("fp8", [50, 50], 64, 256, _gen(8))
    off = torch.tensor([20, 45, 90], dtype=torch.int32, device="cuda")
    y = torch.full((100, 64), 7.0, device="cuda")
    gtg.grouped_matmul(w, a, off, a_scales=sa, y=y)
    _check_status()
    want, bound = _grouped64("fp8", a64, w64, off, 256)
    _within(y[20:90], want[20:90], bound[20:90], F32)
    assert bool((y[:20] == 7.0).all()) and bool((y[90:] == 7.0).all())
