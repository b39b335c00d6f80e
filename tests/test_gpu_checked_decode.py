"""The decoding-loop operators on the bounds-checked debug build: their GPU
tests run again in a child process with libtsd_checked.so, where an index
outside a buffer sets TSD_DEV_BOUNDS in the status word that every one of
those tests requires to be clear."""

import os
import subprocess
import sys

import pytest

from tree_speculative_decoding_ancestor_b200 import build

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.mark.gpu
def test_decode_operators_on_the_checked_build(cuda_device):
    lib = build.build(checked=True)
    files = [os.path.join(HERE, f"test_gpu_{n}.py")
             for n in ("rope", "commit_paged", "chunk_attention", "sample", "decode_loop")]
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider",
                        "-k", "not large_offsets and not 70000", *files],
                       env=dict(os.environ, TSD_LIBRARY=lib), capture_output=True, text=True,
                       timeout=600, cwd=os.path.dirname(HERE))
    assert r.returncode == 0 and " passed" in r.stdout, r.stdout[-3000:] + r.stderr[-2000:]
