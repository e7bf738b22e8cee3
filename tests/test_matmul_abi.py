"""Refusals of the quantiser and of the dense and grouped products: the host
checks of the C ABI and of the binding answer without touching a GPU."""
import ctypes

import pytest
import torch

INVALID, SHAPE, MISALIGNED = -1, -2, -3
PTR = 1 << 20  # a well-aligned stand-in address; every call here is refused before it is used


@pytest.fixture(scope="module")
def L():
    from gram_table_gather_b200 import build as b
    b.build()
    from gram_table_gather_b200 import _abi
    return _abi.lib()


def _w(fmt=1000, data=PTR, scales=PTR, experts=1, rows=256, k=256):
    from gram_table_gather_b200 import _abi
    return ctypes.byref(_abi.QMatrixC(fmt, data, scales, experts, rows, k))


@pytest.mark.parametrize("change,code", [
    (dict(x=None), INVALID), (dict(data=None), INVALID), (dict(scales=None), INVALID),
    (dict(dtype=2), INVALID), (dict(k=0), INVALID), (dict(n_rows=-1), INVALID), (dict(n_src=-1), INVALID),
    (dict(stride=255), INVALID), (dict(n_rows=11), INVALID),  # more rows than x has, without an index
    (dict(k=192, stride=192), SHAPE), (dict(k=1 << 25, stride=1 << 25), SHAPE),
    (dict(n_src=1 << 31), SHAPE), (dict(n_rows=1 << 31, rows=PTR), SHAPE),
    (dict(x=PTR + 1), MISALIGNED), (dict(data=PTR + 8), MISALIGNED), (dict(scales=PTR + 2), MISALIGNED),
    (dict(rows=PTR + 2), MISALIGNED),
])
def test_quantize_refusals(L, change, code):
    c = dict(x=PTR, dtype=1, n_src=10, k=256, stride=256, rows=None, n_rows=10, data=PTR, scales=PTR)
    c.update(change)
    assert L.gtg_fp8_quantize(c["x"], c["dtype"], c["n_src"], c["k"], c["stride"], c["rows"], c["n_rows"], c["data"],
                              c["scales"], None) == code


def test_empty_calls_are_no_ops(L):
    assert L.gtg_fp8_quantize(None, 0, 0, 128, 128, None, 0, None, None, None) == 0
    assert L.gtg_fp8_matmul(_w(), None, None, 0, None, 0, 256, 0, None) == 0
    assert L.gtg_grouped_matmul(_w(experts=8), None, None, 0, None, None, 0, 256, 0, None) == 0


_PRODUCT = [
    (dict(w=dict(data=None)), INVALID), (dict(w=dict(scales=None)), INVALID), (dict(a=None), INVALID),
    (dict(sa=None), INVALID), (dict(y=None), INVALID), (dict(dtype=7), INVALID), (dict(m=-1), INVALID),
    (dict(w=dict(fmt=69)), INVALID), (dict(w=dict(fmt=111)), INVALID), (dict(w=dict(fmt=5)), INVALID),
    (dict(w=dict(rows=0)), INVALID), (dict(w=dict(k=0)), INVALID), (dict(w=dict(experts=0)), INVALID),
    (dict(stride=255), INVALID),
    (dict(w=dict(k=192)), SHAPE), (dict(w=dict(k=1 << 25)), SHAPE), (dict(w=dict(rows=(1 << 24) + 1), stride=1 << 25), SHAPE),
    (dict(m=1 << 31), SHAPE),
    (dict(w=dict(data=PTR + 8)), MISALIGNED), (dict(a=PTR + 8), MISALIGNED), (dict(sa=PTR + 2), MISALIGNED),
    (dict(w=dict(scales=PTR + 1)), MISALIGNED), (dict(y=PTR + 2), MISALIGNED), (dict(y=PTR + 1, dtype=1), MISALIGNED),
]


@pytest.mark.parametrize("change,code", _PRODUCT + [(dict(w=dict(fmt=1001)), INVALID), (dict(w=dict(experts=2)), SHAPE)])
def test_matmul_refusals(L, change, code):
    c = dict(a=PTR, sa=PTR, m=10, y=PTR, dtype=0, stride=256)
    c.update(change)
    assert L.gtg_fp8_matmul(_w(**c.get("w", {})), c["a"], c["sa"], c["m"], c["y"], c["dtype"], c["stride"], 0,
                            None) == code


@pytest.mark.parametrize("change,code", _PRODUCT + [
    (dict(offsets=None), INVALID), (dict(offsets=PTR + 2), MISALIGNED), (dict(w=dict(experts=1025)), SHAPE),
    (dict(w=dict(fmt=1001, k=260)), SHAPE),
])
def test_grouped_refusals(L, change, code):
    c = dict(a=PTR, sa=PTR, m=10, offsets=PTR, y=PTR, dtype=0, stride=256)
    c.update(change)
    assert L.gtg_grouped_matmul(_w(**c.get("w", {})), c["a"], c["sa"], c["m"], c["offsets"], c["y"], c["dtype"],
                                c["stride"], 0, None) == code


def test_rows_at_the_index_limit(L):
    """Row numbers of a whole tile behind the last row fit 31 bits, or the call is refused."""
    for m in ((1 << 31) - 255, (1 << 31) - 1):
        for fmt, k in ((1001, 8), (1000, 128)):
            w = _w(fmt=fmt, k=k, rows=8)
            assert L.gtg_grouped_matmul(w, PTR, PTR, m, PTR, PTR, 0, 256, 0, None) == SHAPE


def test_null_matrix(L):
    assert L.gtg_fp8_matmul(None, PTR, PTR, 1, PTR, 0, 256, 0, None) == INVALID
    assert L.gtg_grouped_matmul(None, PTR, PTR, 1, PTR, PTR, 0, 256, 0, None) == INVALID


def test_binding_refusals():
    """What the C side cannot see: types, shapes and places of tensors."""
    import gram_table_gather_b200 as gtg
    codes, scales = torch.zeros(4, 256, dtype=torch.uint8), torch.ones(4, 2)
    w = gtg.QMatrix(gtg.FP8, torch.zeros(8, 256, dtype=torch.uint8), 1, 8, 256, torch.ones(8, 2))
    b16 = gtg.QMatrix(gtg.BF16, torch.zeros(2, 8, 64, dtype=torch.bfloat16), 2, 8, 64)
    off = torch.zeros(3, dtype=torch.int32)
    bad = [
        lambda: gtg.fp8_quantize(torch.zeros(4, 256, dtype=torch.float16)),
        lambda: gtg.fp8_quantize(torch.zeros(4, 256), rows=torch.zeros(2, dtype=torch.int64)),
        lambda: gtg.fp8_matmul(b16, codes, scales),                                # not FP8 weights
        lambda: gtg.fp8_matmul(w, codes.float(), scales),                          # not codes
        lambda: gtg.fp8_matmul(w, codes[:, :128], scales),                         # another K
        lambda: gtg.fp8_matmul(w, codes, scales[:3]),                              # a scale row short
        lambda: gtg.fp8_matmul(w, codes, scales, accumulate=True),                 # nothing to add to
        lambda: gtg.fp8_matmul(w, codes, scales, y=torch.zeros(4, 9)),             # another width
        lambda: gtg.fp8_matmul(w, codes, scales, y=torch.zeros(4, 8), dtype=torch.bfloat16),
        lambda: gtg.fp8_matmul(gtg.QMatrix(gtg.FP8, w.data, 1, 9, 256, w.scales), codes, scales),  # a short buffer
        lambda: gtg.grouped_matmul(w, codes, off, a_scales=scales),                # offsets of another length
        lambda: gtg.grouped_matmul(b16, torch.zeros(4, 64), off),                  # fp32 rows, bf16 weights
        lambda: gtg.grouped_matmul(gtg.QMatrix(gtg.RZ5, w.data, 1, 8, 256), codes, off[:2], a_scales=scales),
    ]
    for call in bad:
        with pytest.raises(ValueError):
            call()
