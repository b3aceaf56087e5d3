"""The launches of the weight-only operators, without a GPU: a stand-in for the HIP
runtime's launch and attribute calls records them in a process of its own;
nothing runs on a device."""

import json
import os
import subprocess
import sys

import pytest

from w4a4_quantized_diffusion_amd import svdq

STUB = r"""
#include <cstdio>
#include <cstddef>
struct dim3_ { unsigned x, y, z; };
extern "C" {
static dim3_ grid, block;
static size_t shared;
static void* stream;
int __hipPushCallConfiguration(dim3_ g, dim3_ b, size_t shm, void* s) {
  grid = g, block = b, shared = shm, stream = s;
  return 0;
}
int __hipPopCallConfiguration(dim3_* g, dim3_* b, size_t* shm, void** s) {
  *g = grid, *b = block, *shm = shared, *s = stream;
  return 0;
}
int hipFuncSetAttribute(const void* f, int attr, int value) {
  std::printf("attr %p %d %d\n", f, attr, value);
  return 0;
}
int hipLaunchKernel(const void* f, dim3_ g, dim3_ b, void**, size_t shm, void*) {
  std::printf("launch %p %zu\n", f, shm);
  return 0;
}
int hipGetLastError() { return 0; }
}
"""

RUN = r"""
import ctypes, json, sys
ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)
lib = ctypes.CDLL(sys.argv[2])
libc = ctypes.CDLL(None)
P, L, I = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
def at(i): return P((i + 1) << 36)
big = ctypes.c_size_t(1 << 35)
for call in json.loads(sys.argv[3]):
    op, m, k, n = call[:4]
    if op == "a16":
        st = lib.svdq_linear_w4a16(at(0), I(0), L(m), L(k), L(n), I(16), I(0), at(1), at(2), at(3), at(4),
                                   at(5), at(6), P(None), I(0), at(8), I(call[4]), at(9), big, P(None))
    elif op == "linear_grad":
        st = lib.awq_linear_w4a16_grad(at(0), L(m), L(k), L(n), I(64), at(1), at(2), at(3), at(4), I(0),
                                       at(5), big, P(None))
    else:
        st = lib.awq_gated_w4a16_grad(at(0), at(1), at(2), L(m), L(k), L(n), I(64), at(3), at(4), at(5),
                                      at(6), at(7), at(8), I(0), at(9), at(10), at(11), at(12), big, P(None))
    assert st == 0, (call, st)
    libc.fflush(None)
"""

ATTRIBUTE = 8                       # hipFuncAttributeMaxDynamicSharedMemorySize
LDS = 160 << 10


@pytest.fixture(scope="module")
def record(tmp_path_factory):
    """calls -> {function: [(attribute set before or None, the launch's dynamic LDS)]}."""
    if not os.path.exists(svdq.LIB_PATH):
        pytest.fail("libsvdq.so is not built (run __graft_entry__.build())")
    d = tmp_path_factory.mktemp("stub")
    (d / "stub.cpp").write_text(STUB)
    subprocess.run(["g++", "-shared", "-fPIC", "-o", str(d / "stub.so"), str(d / "stub.cpp")], check=True)

    def run(calls):
        r = subprocess.run([sys.executable, "-c", RUN, str(d / "stub.so"), svdq.LIB_PATH, json.dumps(calls)],
                           capture_output=True, text=True)
        assert r.returncode == 0, r.stderr
        now, out = {}, {}
        for line in r.stdout.splitlines():
            w = line.split()
            if w[0] == "attr":
                assert int(w[2]) == ATTRIBUTE
                now[w[1]] = int(w[3])
            else:
                out.setdefault(w[1], []).append((now.get(w[1]), int(w[2])))
        assert out, r.stdout
        return out

    return run


CALLS = [["a16", 64, 4096, 256, 0], ["a16", 54, 7424, 256, 0], ["a16", 49, 2048, 256, 0],
         ["a16", 61, 2752, 10928, 0], ["a16", 50, 512, 12288, 1], ["a16", 64, 4096, 12288, 1],
         ["linear_grad", 1, 4096, 512], ["linear_grad", 40, 4096, 4096], ["linear_grad", 33, 4096, 8192],
         ["gated_grad", 20, 2048, 5456], ["gated_grad", 29, 2048, 1024], ["gated_grad", 64, 512, 4096]]


def test_lds_attribute_is_one_value_per_function(record):
    """Functions that need more than 64 KB of dynamic LDS get one value of the
    attribute, whatever the call's size: two host threads with calls of two sizes
    cannot lower it between each other's setting and launch."""
    large = 0
    for f, launches in record(CALLS + CALLS[::-1]).items():
        values = {a for a, _ in launches if a is not None}
        assert len(values) <= 1, (f, values)
        for a, shm in launches:
            assert shm <= (a if a is not None else 64 << 10) <= LDS
            large += shm > 64 << 10
    assert large >= 6
