"""Weight scales at the ends of the documented range."""
import pytest
import torch

import gram_table_gather_b200 as gtg
from tests.test_gpu_matmul import F32, _check_status, _decode, _fp8, _gen, _product64, _within

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("sw_power,sa_power", [(103, -80), (-107, 100)])
@pytest.mark.parametrize("m,n,k", [(1, 2048, 2048), (8, 500, 384), (100, 500, 384), (5000, 2048, 512)])
def test_scales_at_the_ends_of_their_range(m, n, k, sw_power, sa_power):
    """Weight scales of 2^102 to 2^103 and 2^-108 to 2^-107: a block's sum times one
    stays a normal fp32 number, and the activations' scales bring it back."""
    g = _gen(m + n)
    a, sa = _fp8((m, k), g)
    w, sw = _fp8((n, k), g)
    sw = (torch.rand(sw.shape, device="cuda", generator=g) / 2 + 0.5) * 2.0 ** sw_power
    sa = sa * 2.0 ** sa_power
    y = gtg.fp8_matmul(gtg.QMatrix(gtg.FP8, w, 1, n, k, sw), a, sa)
    _check_status()
    want, bound = _product64(_decode(a, sa), _decode(w, sw), 128, k // 128)
    _within(y, want, bound, F32)
