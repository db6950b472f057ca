"""Prompt and tree calls on several devices of one process: a kernel's limit of
dynamic shared memory belongs to one device, so it has to be raised on each
before the first launch there; and a deterministic call is laid out the same on
each.  The library's objects are linked against a
stand-in of the few runtime calls they make, which writes down what it is asked."""
from __future__ import annotations

import ctypes
import os
import shutil
import subprocess

import pytest

from paged_kv_gqa_02_gb300 import build, ops

OBJECTS = ("pa_packed_f32", "pa_packed_tc", "pa_pages", "pa_serving_api")

FAKE = r"""
#include <cuda_runtime_api.h>
static int dev = 0, count = 0, sms = 152;
struct Entry { int dev, launch; const void* func; long long bytes; };
static unsigned grid = 0;
static Entry entries[4096];
static void put(int launch, const void* f, long long n) { entries[count++ & 4095] = {dev, launch, f, n}; }
static int fake_encode() { return 0; }
extern "C" {
void fake_device(int d) { dev = d; count = 0; }
void fake_sms(int n) { sms = n; }
unsigned fake_grid() { return grid; }  // of the last launch with more than 48 KB
int fake_entry(int i, int* d, int* launch, const void** f, long long* n) {
    if (i >= count) return 0;
    *d = entries[i].dev, *launch = entries[i].launch, *f = entries[i].func, *n = entries[i].bytes;
    return 1;
}
cudaError_t cudaGetDevice(int* d) { *d = dev; return cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr, int) { *v = sms; return cudaSuccess; }
cudaError_t cudaFuncSetAttribute(const void* f, cudaFuncAttribute a, int v) {
    if (a == cudaFuncAttributeMaxDynamicSharedMemorySize) put(0, f, v);
    return cudaSuccess;
}
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* c, const void* f, void**) {
    put(1, f, (long long)c->dynamicSmemBytes);
    if (c->dynamicSmemBytes > 48 * 1024) grid = c->gridDim.x;
    return cudaSuccess;
}
cudaError_t cudaGetDriverEntryPointByVersion(const char*, void** f, unsigned, unsigned long long,
                                             cudaDriverEntryPointQueryResult* r) {
    *f = (void*)fake_encode;
    *r = cudaDriverEntryPointSuccess;
    return cudaSuccess;
}
// what the compiler's own start-up code refers to
void** __cudaRegisterFatBinary(void*) { static void* h; return &h; }
void __cudaRegisterFatBinaryEnd(void**) {}
void __cudaUnregisterFatBinary(void**) {}
void __cudaRegisterFunction() {}
void __cudaRegisterVar() {}
int __cudaGetKernel() { return 0; }
int __cudaLaunchKernel() { return 0; }
int __cudaPopCallConfiguration() { return 0; }
}
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    build.build()
    objects = [os.path.join(build.BUILD_DIR, n + ".o") for n in OBJECTS]
    if not all(map(os.path.exists, objects)):
        build.build(force=True)
    at = tmp_path_factory.mktemp("fake")
    src, out = str(at / "fake.cpp"), str(at / "libfake.so")
    open(src, "w").write(FAKE)
    include = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(build.nvcc()))), "include")
    subprocess.run([cxx, "-shared", "-fPIC", "-Wl,-Bsymbolic", "-I", include, src, *objects, "-o", out], check=True)
    L = ctypes.CDLL(out)
    vp = ctypes.c_void_p
    P, R = ctypes.POINTER(ops.Params), ctypes.POINTER(ops.Rows)
    L.pa_prompt.argtypes = [P, R] + [vp] * 7
    L.pa_tree.argtypes = [P, R] + [vp] * 11 + [ctypes.c_size_t, vp, vp]
    return L


def entries(lib):
    out, i = [], 0
    d, launch, f, n = ctypes.c_int(), ctypes.c_int(), ctypes.c_void_p(), ctypes.c_longlong()
    while lib.fake_entry(i, ctypes.byref(d), ctypes.byref(launch), ctypes.byref(f), ctypes.byref(n)):
        out.append((d.value, bool(launch.value), f.value, n.value))
        i += 1
    return out


@pytest.mark.parametrize("op", ("prompt", "tree"))
@pytest.mark.parametrize("d", (64, 128))
@pytest.mark.parametrize("dtype,out_dtype", [("f32", "f32"), ("f16", "f16"), ("f16", "f32"), ("bf16", "bf16"), ("bf16", "f32")])
def test_shared_memory_is_allowed_on_every_device(lib, op, d, dtype, out_dtype):
    p = ops.make_params(num_seqs=2, num_q_heads=8, num_kv_heads=2, head_dim=d, page_size=16, num_pages=10,
                        max_blocks_per_seq=4, max_context_len=64, dtype=dtype, out_dtype=out_dtype)
    r, at = ops.make_rows(5, 3), ctypes.c_void_p(1 << 20)  # aligned, never read: nothing is launched
    allowed = {}
    for dev in (0, 1, 0, 63, 64, 70, 70, 1):
        lib.fake_device(dev)
        if op == "prompt":
            assert lib.pa_prompt(p, r, at, at, at, at, at, None, None) == 0
        else:
            assert lib.pa_tree(p, r, *[at] * 11, 1 << 40, None, None) == 0
        big = 0
        for where, launch, func, n in entries(lib):
            assert where == dev
            if not launch:
                assert dev >= 64 or (dev, func) not in allowed, "asked for again"
                allowed[dev, func] = n
            elif n > 48 * 1024:  # what a kernel may take unasked
                big += 1
                assert allowed.get((dev, func), 0) >= n, f"device {dev}: {n} bytes not allowed"
        assert big == 1


@pytest.mark.parametrize("hq,hkv,d", [(16, 2, 128), (8, 8, 64), (32, 8, 128)])
@pytest.mark.parametrize("op", ("prompt", "tree"))
def test_a_deterministic_call_is_laid_out_the_same_on_every_device(lib, op, hq, hkv, d):
    """A 16-bit row's bits depend on whether a unit has one tile of rows or two, a tree's on the number of shares."""
    at = ctypes.c_void_p(1 << 20)
    seen = {0: set(), 1: set()}
    for deterministic in (0, 1):
        p = ops.make_params(num_seqs=1, num_q_heads=hq, num_kv_heads=hkv, head_dim=d, page_size=16, num_pages=10,
                            max_blocks_per_seq=4, max_context_len=64, dtype="bf16", deterministic=deterministic)
        for n in ((1000, 2500, 4000, 6000) if op == "prompt" else (500,)):
            grids = []
            for sms in (40, 80, 148, 152, 160):
                lib.fake_sms(sms)
                lib.fake_device(0)
                if op == "prompt":
                    assert lib.pa_prompt(p, ops.make_rows(n, n), at, at, at, at, at, None, None) == 0
                else:
                    assert lib.pa_tree(p, ops.make_rows(n, n), *[at] * 11, 1 << 40, None, None) == 0
                grids.append(lib.fake_grid())
            lib.fake_sms(152)
            seen[deterministic].add(len(set(grids)))
    assert seen[1] == {1} and max(seen[0]) > 1
