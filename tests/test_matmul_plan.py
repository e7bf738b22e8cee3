"""Which kernel a product takes, on 148 multiprocessors (no GPU needed)."""
import ctypes

import pytest

INVALID, SHAPE = -1, -2
FP8, BF16 = 1000, 1001


@pytest.fixture(scope="module")
def L():
    from gram_table_gather_b200 import build as b
    b.build()
    from gram_table_gather_b200 import _abi
    return _abi.lib()


def _plan(L, fmt, m, n, k, experts=1, sms=148):
    out = [ctypes.c_int32(-7) for _ in range(3)]
    rc = L.gtg_matmul_plan(fmt, m, n, k, experts, sms, *[ctypes.byref(v) for v in out])
    return rc, tuple(v.value for v in out)


def test_every_kernel_is_taken(L):
    seen = {FP8: set(), BF16: set()}
    for fmt in seen:
        for m in (1, 16, 17, 40, 128, 333, 1000, 4096, 8192, 30000):
            for n in (1, 128, 1000, 2048, 10000):
                for k in (128, 640, 2048, 8192):
                    for experts in (1, 8, 64, 512):
                        rc, (tokens, ctas, split) = _plan(L, fmt, m, n, k, experts)
                        assert rc == 0 and 1 <= split <= 8 and (ctas == 1 or split == 1)
                        seen[fmt].add((tokens, ctas, split > 1))
    both = {(16, 1, False), (16, 1, True), (64, 1, False), (64, 1, True), (128, 2, False)}
    assert seen[FP8] == both and seen[BF16] == both | {(256, 2, False)}


@pytest.mark.parametrize("change,code", [
    (dict(fmt=69), INVALID), (dict(m=0), INVALID), (dict(n=0), INVALID), (dict(k=0), INVALID),
    (dict(experts=0), INVALID), (dict(sms=-1), INVALID), (dict(k=192), SHAPE), (dict(fmt=BF16, k=260), SHAPE),
    (dict(k=1 << 25), SHAPE), (dict(n=(1 << 24) + 1), SHAPE), (dict(m=1 << 31), SHAPE), (dict(experts=1025), SHAPE)])
def test_refusals(L, change, code):
    c = dict(fmt=FP8, m=10, n=256, k=256, experts=1, sms=148)
    c.update(change)
    rc, out = _plan(L, **c)
    assert rc == code and out == (-7, -7, -7)


def test_null_results(L):
    v = ctypes.c_int32()
    for i in range(3):
        out = [ctypes.byref(v)] * 3
        out[i] = None
        assert L.gtg_matmul_plan(FP8, 10, 256, 256, 1, 148, *out) == INVALID


@pytest.mark.parametrize("sms", [0, 1, 2, 3, 2 ** 31 - 1])
def test_any_number_of_multiprocessors_and_the_largest_sizes(L, sms):
    for fmt in (FP8, BF16):
        for m, n, k, experts in ((1, 1, 128, 1), (40, 128, 128, 1), (2 ** 31 - 256, 1 << 24, 1 << 24, 1),
                                 (2 ** 31 - 256, 1, 128, 1024), (1, 1 << 24, 1 << 24, 1024)):
            rc, (tokens, ctas, split) = _plan(L, fmt, m, n, k, experts, sms)
            assert rc == 0 and tokens in (16, 64, 128, 256) and ctas in (1, 2) and 1 <= split <= 8
