"""No C++ exception leaves the library: the batch calls of many entries, in a process that has no memory left for a copy
of them (CPU only: every call returns before it launches anything)."""
import subprocess
import sys

import pytest

CHILD = r"""
import ctypes, resource, sys
import numpy as np
lib = ctypes.CDLL(sys.argv[1])
COUNT, M, dropout = 2_000_000, int(sys.argv[3]), sys.argv[4] == "dropout"
fake, vp, sz = 0x10000, ctypes.c_void_p, ctypes.c_size_t
if sys.argv[2] == "grads":      # x, t, u, dy, dA, dB, M, N, K
    items = np.tile(np.array([fake] * 6 + [M, 64, 128], dtype=np.int64), (COUNT, 1))
else:                           # x, w, out, M, C
    items = np.tile(np.array([fake] * 3 + [M, 128], dtype=np.int64), (COUNT, 1))
drops = np.zeros((COUNT, 3), dtype=np.uint64)
drops[:, 2] = np.float64(0.25).view(np.uint64)
name = {"grads": "qlora_lora_grads_batch", "down": "qlora_lora_down_batch", "u": "qlora_lora_u_batch"}[sys.argv[2]]
f = getattr(lib, name + ("_dropout" if dropout else ""))
args = [vp(items.ctypes.data)] + ([vp(drops.ctypes.data)] if dropout else []) + [COUNT, 8]
args += ([] if sys.argv[2] == "grads" else [ctypes.c_float(1.0)]) + [0, vp(0), sz(0), vp(0)]
now = next(int(l.split()[1]) for l in open("/proc/self/status") if l.startswith("VmSize:")) * 1024
resource.setrlimit(resource.RLIMIT_AS, (now + (16 << 20), resource.RLIM_INFINITY))
status = f(*args)
resource.setrlimit(resource.RLIMIT_AS, (resource.RLIM_INFINITY, resource.RLIM_INFINITY))
print("status", status)
"""


# no rows: nothing to do; rows, but no workspace for them
@pytest.mark.parametrize("call,dropout,M,status", [("down", "dropout", 0, 0), ("down", "dropout", 4, -4), ("down", "", 0, 0),
                                                   ("u", "", 0, 0), ("grads", "dropout", 4, -4)])
def test_batches_need_no_memory_of_their_own(call, dropout, M, status):
    from bit_nf4_quantized_15_amd import build
    r = subprocess.run([sys.executable, "-c", CHILD, build.OUT, call, str(M), dropout], capture_output=True, text=True,
                       timeout=120)
    assert r.returncode == 0 and f"status {status}" in r.stdout, (r.returncode, r.stdout, r.stderr[-500:])
