"""The launches of the operators around a block, without a GPU: a stand-in for the HIP
runtime's registration, launch and attribute calls records them in a process of its own;
nothing runs on a device."""

import json
import os
import subprocess
import sys

import pytest

from w4a4_quantized_diffusion_amd import svdq

STUB = r"""
#include <cstddef>
#include <cstdio>
#include <cstring>
struct dim3_ { unsigned x, y, z; };
extern "C" {
static dim3_ grid, block;
static size_t shared;
static void* stream;
static const void* read[64];
static int reads;
void __hipRegisterFunction(void**, const void* f, char*, const char* name, unsigned, void*, void*, void*,
                           void*, int*) {
  std::printf("name %p %s\n", f, name);
  if (std::strstr(name, "res_grad_kernel") && reads < 64) read[reads++] = f;
}
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
// (res_grad_kernel's first three arguments are or begin with an address)
int hipLaunchKernel(const void* f, dim3_ g, dim3_ b, void** args, size_t shm, void*) {
  size_t a[3] = {};
  for (int i = 0; i < reads; ++i)
    if (read[i] == f)
      for (int k = 0; k < 3; ++k) std::memcpy(&a[k], args[k], sizeof(size_t));
  std::printf("launch %p %u %u %zu %zu %zu %zu\n", f, g.x, b.x, shm, a[0], a[1], a[2]);
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
P, L, I, F = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float
class Vec(ctypes.Structure):
    _fields_ = [("data", P), ("dtype", I), ("ld", L)]
def at(i): return P((i + 1) << 40)
def vec(i, ld): return ctypes.byref(Vec((i + 1) << 40, 1, ld))
big = ctypes.c_size_t(1 << 39)
print("begin")
for op, a in json.loads(sys.argv[3]):
    if op == "norm_grad":
        m, d, images, dt = a
        st = lib.svdq_block_norm_grad(at(0), I(dt), at(1), at(2), I(dt), at(3), I(dt), L(m), L(d),
                                      L(images), I(0), F(1e-6), vec(4, 0), vec(5, d), vec(6, 0), vec(7, d),
                                      vec(8, d), at(9), at(10), at(11), at(12), at(13), at(14), at(15),
                                      at(16), big, P(None))
    elif op == "res_grad":
        m, k, n, images, dt, dgate = a
        st = lib.awq_linear_w4a16_res_grad(at(0), I(dt), at(1), L(m), L(k), L(n), I(64), at(2), at(3),
                                           at(4), I(0), vec(5, n), L(images), at(6), at(7),
                                           at(8) if dgate else P(None), at(9), big, P(None))
    else:
        t, e, top, k, n = a
        st = lib.awq_moe_w4a16(at(0), at(1), I(0), L(t), L(e), I(top), L(k), L(n), I(64), at(2), at(3),
                               at(4), at(5), at(6), at(7), at(8), at(9), at(10), I(0), I(1), at(11),
                               P(None), P(None), at(12), big, P(None))
    assert st == 0, (op, a, st)
    print("call")
    libc.fflush(None)
    sys.stdout.flush()
"""


@pytest.fixture(scope="module")
def record(tmp_path_factory):
    """calls -> for each, [(kernel, workgroups, threads, dynamic LDS, attribute set
    before or None, res_grad_kernel's first three arguments)]."""
    if not os.path.exists(svdq.LIB_PATH):
        pytest.fail("libsvdq.so is not built (run __graft_entry__.build())")
    d = tmp_path_factory.mktemp("stub")
    (d / "stub.cpp").write_text(STUB)
    subprocess.run(["g++", "-shared", "-fPIC", "-o", str(d / "stub.so"), str(d / "stub.cpp")], check=True)

    def run(calls):
        r = subprocess.run([sys.executable, "-u", "-c", RUN, str(d / "stub.so"), svdq.LIB_PATH,
                            json.dumps(calls)], capture_output=True, text=True)
        assert r.returncode == 0, r.stderr
        names, attrs, out, now = {}, {}, [], []
        for line in r.stdout.splitlines():
            w = line.split()
            if w[0] == "name":
                names[w[1]] = w[2]
            elif w[0] == "attr":
                assert int(w[2]) == 8                  # hipFuncAttributeMaxDynamicSharedMemorySize
                attrs[w[1]] = int(w[3])
            elif w[0] == "launch":
                v = [int(x) for x in w[2:]]
                now.append((names[w[1]], v[0], v[1], v[2], attrs.get(w[1]), tuple(v[3:])))
            elif w[0] == "call":
                out.append(now)
                now = []
        assert len(out) == len(calls)
        return out

    return run


@pytest.mark.parametrize("images,rows,n", [(1 << 20, 1, 16384), (1 << 20, 1, 8192), (1 << 20, 3, 4096),
                                            (1 << 19, 2, 16400), (1 << 20, 1, 64), (7, 5000, 12288)])
@pytest.mark.parametrize("dgate", [False, True])
def test_res_grad_launches_fit(record, images, rows, n, dgate):
    """A launch has fewer than 2^32 threads, whatever images and N are, and the launches
    over dY, Z and the gate follow one another without a gap."""
    for dt, size in ((1, 2), (0, 4)):
        launches, = record([["res_grad", [images * rows, 64, n, images, dt, dgate]]])
        for kernel, groups, threads, *_ in launches:
            assert 0 < groups and groups * threads < 1 << 32, kernel
        first = [l for l in launches if "res_grad_kernel" in l[0]]
        blocks = -(-n // 512)
        total = sum(l[1] for l in first)
        parts, rest = divmod(total, blocks * images)
        assert rest == 0 and 1 <= parts <= rows
        done = 0
        for _, groups, _, _, _, (dy, z, gate) in first:
            assert groups % (blocks * parts) == 0
            assert dy == (1 << 40) + done * rows * n * size and z == (2 << 40) + done * rows * n * 2
            assert gate == (6 << 40) + done * n * 2
            done += groups // (blocks * parts)
        assert done == images


CALLS = [["norm_grad", [m, d, images, dt]] for m, d, images in ((6, 8200, 2), (4, 16384, 1), (9, 12288, 3))
         for dt in (0, 1)]
CALLS += [["moe", a] for a in ([64, 8, 2, 4096, 128], [40, 64, 8, 2048, 256], [64, 2, 2, 8192, 64],
                               [50, 40, 6, 1024, 192], [33, 4, 2, 8256, 64], [1, 8, 2, 8192, 128])]


def test_lds_attribute_is_one_value_per_function(record):
    """Functions that need more than 64 KB of dynamic LDS get one value of the attribute,
    whatever the call's size: two host threads with calls of two sizes cannot lower it
    between each other's setting and launch."""
    values, large = {}, set()
    for launches in record(CALLS + CALLS[::-1]):
        for kernel, _, _, shm, attr, _ in launches:
            assert shm <= (attr if attr is not None else 64 << 10) <= 160 << 10, kernel
            if attr is not None:
                values.setdefault(kernel, set()).add(attr)
            if shm > 64 << 10:
                large.add(kernel)
    assert all(len(v) == 1 for v in values.values()), values
    assert any("block_norm_grad" in k for k in large) and any("moe_down" in k for k in large)


def test_moe_forms(record):
    """Wide layers need no slices: two launches, 32 columns a workgroup of the second."""
    for k, launches in ((8192, 2), (8256, 2), (4096, 3)):
        for t in (5, 64):
            got, = record([["moe", [t, 8, 2, k, 128]]])
            assert len(got) == launches
            assert "moe_down_kernel" in got[1][0] and got[1][1] == k // 32 * (1 if launches == 2 else 2)
    got, = record([["moe", [1, 8, 2, 8192, 128]]])
    assert len(got) == 2 and got[1][1] == 8192 // 32
