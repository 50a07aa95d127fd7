"""Pool calls that find no memory for a table: an error, and a pool as it was (CPU). Each
runs in a process of its own whose address space is cut off; an exception that leaves
the library ends it."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SCRIPT = """
import resource, sys
import numpy as np
sys.path.insert(0, %r)
import paged_kv_decode_25_gb300 as mi
N, what = 1 << 26, sys.argv[1]
def cut(more):
    with open("/proc/self/statm") as f:
        used = int(f.read().split()[0]) * resource.getpagesize()
    resource.setrlimit(resource.RLIMIT_AS, (used + more, resource.getrlimit(resource.RLIMIT_AS)[1]))
pool = mi.Pool(N, 4, N - 1)
assert pool.alloc(1, 100) == 0
lib, h = mi.load(), pool.handle
ids, big = np.array([0, 1], np.int32), np.array([16 * (N - 1000), 200], np.int32)
if what == "alloc":
    free = pool.num_free()
    cut(64 << 20)
    assert pool.alloc(0, int(big[0])) == mi.MI_ERR_INVALID_ARG
    assert pool.num_free() == free and mi.mi_kv_pool_seq_blocks(h, 0) is None
    assert pool.alloc(1, int(big[0])) == mi.MI_ERR_INVALID_ARG
    assert mi.mi_kv_pool_seq_blocks(h, 1, 100).tolist() == list(range(7))
    assert pool.alloc(0, 1000) == 0
else:
    free = pool.num_free()
    cut(64 << 20)
    assert lib.mi_kv_pool_alloc_batch(h, ids.ctypes.data, big.ctypes.data, 2) == mi.MI_ERR_INVALID_ARG
    assert pool.num_free() == free and mi.mi_kv_pool_seq_blocks(h, 0) is None
    assert mi.mi_kv_pool_seq_blocks(h, 1, 100).tolist() == list(range(7))
print("done")
""" % ROOT


@pytest.mark.parametrize("what", ["alloc", "alloc_batch"])
def test_no_memory_for_a_table(what):
    from paged_kv_decode_25_gb300 import build
    build.build()
    p = subprocess.run([sys.executable, "-c", SCRIPT, what], capture_output=True, text=True, timeout=300)
    assert p.returncode == 0 and p.stdout == "done\n", (p.returncode, p.stderr[-2000:])
