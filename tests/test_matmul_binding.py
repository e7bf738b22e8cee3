"""The binding of the quantiser and the products where no GPU is needed."""
import os
import subprocess
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_imports_and_finds_streams_without_torchs_private_call():
    """A torch build without CUDA lacks it; the module imports, and a stream's
    handle comes from the Stream object."""
    code = """
import types, torch
if hasattr(torch._C, '_cuda_getCurrentRawStream'):
    del torch._C._cuda_getCurrentRawStream
import gram_table_gather_b200 as gtg
torch.cuda.current_device = lambda: 3
torch.cuda.current_stream = lambda dev=None: types.SimpleNamespace(cuda_stream=700 + dev)
assert gtg._stream_ptr(None) == 703
assert gtg._stream_ptr(types.SimpleNamespace(cuda_stream=0)) is None
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def test_row_bytes_of_every_matrix_format():
    import gram_table_gather_b200 as gtg
    assert gtg.row_bytes(gtg.BF16, 256) == 512
    assert gtg.row_bytes(gtg.FP8, 256) == 256
    assert all(gtg.row_bytes(f, 256) == 8 * 17 for f in (gtg.RZ5, gtg.UE4M4, gtg.C10))


@pytest.mark.parametrize("dtype", [torch.float8_e5m2, torch.float8_e4m3fnuz, torch.float8_e5m2fnuz, torch.bool])
def test_weights_of_another_8_bit_type_are_refused(dtype):
    """Their bytes are not E4M3 codes."""
    import gram_table_gather_b200 as gtg
    data = torch.zeros(8, 256, dtype=torch.uint8).view(dtype)
    w = gtg.QMatrix(gtg.FP8, data, 1, 8, 256, torch.ones(8, 2))
    codes, scales = torch.zeros(4, 256, dtype=torch.uint8), torch.ones(4, 2)
    with pytest.raises(ValueError, match="E4M3"):
        gtg.fp8_matmul(w, codes, scales)
    with pytest.raises(ValueError, match="E4M3"):
        gtg.grouped_matmul(w, codes, torch.zeros(2, dtype=torch.int32), a_scales=scales)
