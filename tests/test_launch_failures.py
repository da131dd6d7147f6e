"""What the expert operators return where a HIP call fails, without a GPU:
a library put before HIP's own in a child process stands for the calls."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SHIM = r"""
#include <stdlib.h>
static int launches;
static int fails(const char* call) { const char* f = getenv("FAILS"); return f && f[0] == call[0]; }
int hipFuncSetAttribute(const void* f, int a, int v) { return fails("attribute"); }
int __hipPushCallConfiguration(void) { return 0; }
int __hipPopCallConfiguration(void) { return 0; }
int hipLaunchKernel(void) { ++launches; return 0; }
int hipGetLastError(void) { return fails("launch"); }
int launches_so_far(void) { return launches; }
"""

CHILD = r"""
import ctypes, sys
sys.path.insert(0, sys.argv[1])
from lossless_bf16_exponent_zc_amd import experts
L, shim, P = experts.lib(), ctypes.CDLL(sys.argv[2]), 0x10000
calls = []
# dense products of few rows, small, mid, pair and wide tiles, in order and in runs; weight gradients of every shape
for rows, n, k in ((8, 128, 128), (100, 512, 128), (1024, 4096, 7168), (8192, 600, 128), (4096, 4096, 256), (65536, 4096, 256)):
    calls.append(lambda rows=rows, n=n, k=k: L.zc_expert_product(P, P, rows, P, P, 1, n, k, None, None, P, n, 0, None))
for rows, n, k in ((256, 64, 64), (256, 4096, 4096), (4096, 4096, 7168), (128, 2000, 2000), (256, 2000, 2000), (32768, 1024, 1024)):
    need = L.zc_expert_weight_grad_workspace_bytes(rows, 1, n, k)
    calls.append(lambda rows=rows, n=n, k=k, need=need: L.zc_expert_weight_grad(P, P, P, P, rows, 1, n, k, None, P, 0, P if need else None, need, None))
for call in calls:
    before = shim.launches_so_far()
    rc = call()
    print(rc, shim.launches_so_far() - before)
"""


def run(tmp_path, fails):
    src, lib = tmp_path / "shim.c", tmp_path / "shim.so"
    src.write_text(SHIM)
    subprocess.run(["gcc", "-shared", "-fPIC", str(src), "-o", str(lib)], check=True)
    before = os.environ.get("LD_PRELOAD")
    env = dict(os.environ, LD_PRELOAD=str(lib) + (":" + before if before else ""), FAILS=fails)
    r = subprocess.run([sys.executable, "-c", CHILD, ROOT, str(lib)], env=env, capture_output=True, text=True, timeout=110)
    assert r.returncode == 0, r.stderr
    return [tuple(map(int, line.split())) for line in r.stdout.splitlines()]


def test_calls_that_launch(tmp_path):
    got = run(tmp_path, "")
    assert len(got) == 12 and all(rc == 0 and launches >= 1 for rc, launches in got)


def test_a_failed_launch_is_reported(tmp_path):
    assert all(rc == 5 for rc, _ in run(tmp_path, "launch"))


def test_nothing_is_launched_without_the_lds_it_needs(tmp_path):
    """Kernels with more LDS than the default ask for it first; few rows need none."""
    got = run(tmp_path, "attribute")
    assert got[0] == (0, 1)
    assert got[1:] == [(5, 0)] * 11
