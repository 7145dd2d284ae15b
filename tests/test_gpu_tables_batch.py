"""Page tables of batches around the size at which the sums in shared memory pass the default 48 KB."""
import os
import subprocess
import sys

import numpy as np
import pytest

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))  # (as a script)
from gpu_helpers import lib
from oracle import kv_cache as kc
from test_gpu_kv_cache import make_tables, run_tables, same

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))


def check_batch(bsp, B):
    a = make_tables(np.random.default_rng(B), B, 16, 40, 3)
    tot, n = int((-(-(a[0].astype(np.int64) + a[1]) // 16)).sum()), int(a[1].sum())
    same(run_tables(bsp, *a, 16, tot + 3, n + 2), kc.tables(*a, 16, tot + 3, n + 2))


@pytest.mark.parametrize("B", [4078, 4079, 4095])
def test_first_batch_of_a_process(B):
    """No larger batch before it: nothing else has raised the kernel's limit."""
    r = subprocess.run([sys.executable, __file__, str(B)], cwd=os.path.dirname(HERE), capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


@pytest.mark.parametrize("B", [4079, 4096, 4097, 16384])
def test_batch(B):
    check_batch(lib(), B)


if __name__ == "__main__":
    check_batch(lib(), int(sys.argv[1]))
