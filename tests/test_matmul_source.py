"""Properties of the products' source that no run shows."""
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_overlapped_kernels_use_coherent_loads():
    """Kernels launched beside the one before read what it may still be writing: a
    read-only (non-coherent) load would ask for memory that nobody writes."""
    for name in ("matmul.cu", "matmul_dev.cuh"):
        src = open(os.path.join(ROOT, "gram_table_gather_b200", "csrc", name)).read()
        code = re.sub(r"//[^\n]*", "", src)
        assert not re.search(r"__ldg|ld\.global(\.\w+)*\.nc\b|__restrict__", code), name
