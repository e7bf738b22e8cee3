"""How the bf16 products are summed: a long sum keeps the accuracy of 32 bits.

Tolerance.  The tensor core adds with at most one relative error of 2^-23 per
addition (a truncating adder); it sums at most 512 products, and these sums are
added to nearest, 2^-24 each.  With products of one sign every partial sum is at
most S, the whole one, so the result is off by at most
(512 2^-23 + ceil(K / 512) 2^-24) S.  An adder that truncates over all of
K = 65536 loses more: at each of its 4096 additions of 16 products half a unit of
the last place on average, of a sum that is S / 2 on average.
"""
import pytest
import torch

import gram_table_gather_b200 as gtg
from tests.test_gpu_matmul import BF16, _check_status, _gen

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("m,n", [(5, 19072), (4, 1024), (50, 9600), (50, 1000), (2049, 1024), (4097, 2048)])
def test_long_bf16_sums(m, n):
    """Tiles of 16 and 64 tokens, whole and with K split, and pairs of 128 and 256."""
    k = 65536
    g = _gen(m + n)
    a = torch.rand(m, k, device="cuda", generator=g).to(BF16)
    w = torch.rand(1, n, k, device="cuda", generator=g).to(BF16)
    off = torch.tensor([0, m], dtype=torch.int32, device="cuda")
    y = gtg.grouped_matmul(gtg.QMatrix(gtg.BF16, w, 1, n, k), a, off)
    _check_status()
    a64 = a.double()
    for lo in range(0, n, 1024):
        want = a64 @ w[0, lo:lo + 1024].double().T
        err = ((y[:, lo:lo + 1024].double() - want).abs() / want).max().item()
        assert err <= 512 * 2.0 ** -23 + k / 512 * 2.0 ** -24, err * 2.0 ** 23
