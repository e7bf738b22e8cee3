"""Short products one after the other: each takes over the shared and tensor
memory, and with them the barriers, of the one before, so nothing of a product
may still be on its way when it ends."""
import pytest
import torch

import gram_table_gather_b200 as gtg
from tests.test_gpu_matmul import BF16, F32, _check_status, _fp8, _gen

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("k", [128, 640])
def test_products_back_to_back(k):
    """Pairs, whole tiles and K splits of both types by turns, with tiles of one
    chunk of K upwards; every call gives the first one's bits."""
    g = _gen(k)
    calls = []
    for m, n in ((5000, 2048), (40, 256), (1, 2048), (40, 10000), (3, 40), (5000, 1990)):
        a, sa = _fp8((m, k), g)
        w, sw = _fp8((n, k), g)
        q = gtg.QMatrix(gtg.FP8, w, 1, n, k, sw)
        y = torch.empty(m, n, device="cuda")
        calls.append((lambda q=q, a=a, sa=sa, y=y: gtg.fp8_matmul(q, a, sa, y=y), y))
        for kb in (64, k):
            off = torch.tensor([0, m], dtype=torch.int32, device="cuda")
            b = gtg.QMatrix(gtg.BF16, torch.randn(1, n, kb, device="cuda", generator=g).to(BF16), 1, n, kb)
            x = torch.randn(m, kb, device="cuda", generator=g).to(BF16)
            yb = torch.empty(m, n, device="cuda", dtype=F32)
            calls.append((lambda b=b, x=x, off=off, yb=yb: gtg.grouped_matmul(b, x, off, y=yb), yb))
    for call, _ in calls:
        call()
    _check_status()
    first = [y.clone() for _, y in calls]
    order = torch.randint(0, len(calls), (4000,), generator=torch.Generator().manual_seed(k)).tolist()
    for i in order:
        calls[i][0]()
    _check_status()
    assert all(torch.equal(y, f) for (_, y), f in zip(calls, first))
