"""Rules of the chunk attention's source that a run shows only by hanging."""
import pathlib
import re

import sparse_depth_token_gb300

CSRC = pathlib.Path(sparse_depth_token_gb300.__file__).parent / "csrc"


def test_successors_start_after_the_tensor_memory_is_taken():
    """A grid lets its successors start once every CTA of it holds its tensor memory. Before that, a
    successor's CTA on the same SM could take the columns that a CTA of the grid waits for (a third
    kernel held them), and keep them while it waits for that grid to end."""
    text = re.sub(r"//[^\n]*", "", (CSRC / "cache_chunk_tc.cu").read_text())
    kernel = text[text.index("__global__"):]
    at = [kernel.index(name + "(") for name in ("tmem_alloc", "__syncthreads", "pdl_trigger", "pdl_wait")]
    assert at == sorted(at)
    for name in ("tmem_alloc", "pdl_trigger", "pdl_wait"):
        assert kernel.count(name + "(") == 1, name
