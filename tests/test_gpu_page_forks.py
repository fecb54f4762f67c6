"""Forks of caches whose staged columns fill a block's shared memory, or take several strips of it."""
import subprocess
import sys

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

# (requests, columns): 4 R (2 + columns) bytes are staged.  Exactly 48 KB, and 12 bytes less; past 48 KB; past what a block has.
SHAPES = [(64, 190), (63, 193), (100, 150), (2048, 40), (900, 60)]


def forks(shapes):
    import torch
    import kv_cache_eviction_split_gb300 as kv
    from tests.test_gpu_pages import Model, _fork
    kv.load()
    for R, cols in shapes:
        rng = np.random.default_rng(R)
        lens = rng.integers(0, 16 * cols + 1, R)
        lens[:2] = 16 * cols, 16 * cols - 15
        m = Model(kv, R, 1, 1, 64, 16, cols, int((-(-lens // 16)).sum()), lens)
        for parents in (rng.integers(-1, R, R).tolist(), [1] * (R // 2) + list(range(R // 2, R))):
            _fork(m, parents)
            torch.cuda.synchronize()
            m.fork(parents)
            m.check()


@pytest.mark.parametrize("shape", SHAPES)
def test_forks_in_a_process_of_their_own(cuda_lib, shape):
    """The first fork of a process: nothing has asked for more shared memory before."""
    code = "from tests.test_gpu_page_forks import forks; forks([%r])" % (shape,)
    p = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert p.returncode == 0, p.stderr[-2000:]
