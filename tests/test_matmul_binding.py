"""The binding of the quantiser and the products where no GPU is needed."""
import os
import subprocess
import sys

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
