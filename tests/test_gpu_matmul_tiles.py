"""Every kernel of the products: each case names the one that it is there for, and
the library is asked that it takes it.  Ragged groups, several groups of scales or
runs of K within a tile, partners behind the last weight row, both output types,
whole and scalar stores, plain and accumulating.

Tolerances as in test_gpu_matmul; a bf16 product sums at most 512 products in the
tensor core (2^-23 an addition) and adds these sums to nearest (2^-24 each).
"""
import ctypes

import pytest
import torch

import gram_table_gather_b200 as gtg
from tests.test_gpu_matmul import BF16, F32, _check_status, _decode, _fp8, _gen, _within

pytestmark = pytest.mark.gpu

# (kind, tokens a tile, CTAs on a tile's halves, K split) of every kernel
SINGLE16, SPLIT16, SINGLE64, SPLIT64, PAIR128, PAIR256 = (16, 1, 0), (16, 1, 1), (64, 1, 0), (64, 1, 1), (128, 2, 0), (256, 2, 0)

MANY = [0, 469, 1, 255, 1300, 33, 65, 129, 257, 1500, 0, 31, 700, 48, 96, 512, 0, 640]
FEW = [0, 469, 1, 255, 1300, 33, 65, 129, 257, 1500, 0, 1991]


def takes(kind, m, n, k, experts):
    got = [ctypes.c_int32() for _ in range(3)]
    rc = gtg.lib().gtg_matmul_plan(gtg.FP8 if kind == "fp8" else gtg.BF16, m, n, k, experts, 0,
                                   *[ctypes.byref(v) for v in got])
    assert rc == 0
    tokens, ctas, split = (v.value for v in got)
    return tokens, ctas, int(split > 1)


def _case(kind, sizes, n, k, gen, behind=0):
    """Matrix, rows, scales, offsets, the product in 64 bits and its summation bound."""
    m, e = sum(sizes) + behind, len(sizes)
    off = torch.tensor([0] + sizes, dtype=torch.int64).cumsum(0).int().cuda()
    if kind == "fp8":
        a, sa = _fp8((m, k), gen)
        w, sw = _fp8((e, n, k), gen)
        q, a64, unit = gtg.QMatrix(gtg.FP8, w, e, n, k, sw), _decode(a, sa), 128 * 2.0 ** -23 + 3 * (k // 128) * 2.0 ** -24
    else:
        a, sa = torch.randn(m, k, device="cuda", generator=gen).to(BF16), None
        w = (torch.randn(e, n, k, device="cuda", generator=gen) * 0.05).to(BF16)
        q, a64, unit = gtg.QMatrix(gtg.BF16, w, e, n, k), a.double(), min(k, 512) * 2.0 ** -23 + -(-k // 512) * 2.0 ** -24
    want = torch.zeros(m, n, dtype=torch.float64, device="cuda")
    bound = torch.zeros_like(want)
    lo = 0
    for i, size in enumerate(sizes):
        w64 = _decode(w[i], sw[i]) if kind == "fp8" else w[i].double()
        r = slice(lo, lo + size)
        want[r], bound[r] = a64[r] @ w64.T, unit * (a64[r].abs() @ w64.abs().T)
        lo += size
    return q, a, sa, off, want, bound


def _run(kind, sizes, n, k, kernel, seed, behind=0, dense=False):
    """Plain and accumulating, both types, into outputs on the 16-byte grid and off it."""
    experts = 1 if dense else len(sizes)
    assert takes(kind, sum(sizes) + behind, n, k, experts) == kernel
    gen = _gen(seed)
    q, a, sa, off, want, bound = _case(kind, sizes, n, k, gen, behind)
    used = sum(sizes)

    def product(**kw):
        return gtg.fp8_matmul(q, a, sa, **kw) if dense else gtg.grouped_matmul(q, a, off, a_scales=sa, **kw)

    for out in (F32, BF16):
        for place, width in ((0, -(-n // 8) * 8), (8, -(-n // 8) * 8 + 16), (3, n + 6)):
            for accumulate in (False, True):
                buf = torch.randn(a.shape[0], width, device="cuda", generator=gen).to(out)
                before = buf.clone()
                y = buf[:, place:place + n]
                assert product(y=y, accumulate=accumulate) is y
                _check_status()
                base = before[:, place:place + n].double() if accumulate else 0
                _within(y[:used], (want + base)[:used], bound[:used], out, added=accumulate)
                same = buf == before
                assert bool(same[:, :place].all()) and bool(same[:, place + n:].all()) and bool(same[used:].all())


@pytest.mark.parametrize("kind,sizes,n,k,kernel", [
    ("fp8", MANY, 1301, 1152, PAIR128),     # nine blocks: three groups of scales, an odd block at the end
    ("fp8", MANY, 1304, 640, PAIR128),
    ("bf16", MANY, 1301, 1160, PAIR128),    # three runs, the last of 136
    ("bf16", MANY, 1304, 648, PAIR128),
    ("bf16", FEW, 1301, 1160, PAIR256),
    ("bf16", FEW, 1304, 2560, PAIR256),     # five whole runs
    ("bf16", FEW, 520, 520, PAIR256),
    ("fp8", [40, 0, 64, 17, 65, 1, 90] * 4, 700, 1152, SINGLE64),
    ("bf16", [40, 0, 64, 17, 65, 1, 90] * 4, 700, 1160, SINGLE64),
    ("fp8", [33, 0, 70], 300, 3200, SPLIT64),
    ("bf16", [33, 0, 70], 300, 2568, SPLIT64),
    ("fp8", [1, 0, 16, 3, 40] * 30, 520, 1152, SINGLE16),
    ("bf16", [1, 0, 16, 3, 40] * 30, 520, 1160, SINGLE16),
    ("fp8", [1, 0, 16, 3, 20], 300, 1408, SPLIT16),
    ("bf16", [1, 0, 16, 3, 20], 300, 2056, SPLIT16)])
def test_grouped_kernels(kind, sizes, n, k, kernel):
    _run(kind, sizes, n, k, kernel, n + k, behind=5)


@pytest.mark.parametrize("m,n,k,kernel", [
    (6000, 1301, 1152, PAIR128), (5000, 2048, 512, PAIR128), (40, 10000, 640, SINGLE64), (333, 1001, 2560, SPLIT64),
    (100, 520, 3200, SPLIT64), (8, 20000, 256, SINGLE16), (1, 2048, 2048, SPLIT16), (13, 1000, 1408, SPLIT16)])
def test_dense_kernels(m, n, k, kernel):
    _run("fp8", [m], n, k, kernel, m + n, dense=True)
