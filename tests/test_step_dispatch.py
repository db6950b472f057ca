"""What the calls around the step's attention launch, and what they refuse by their arguments' places, on the host: the
library's objects are linked against a stand-in of the few runtime calls they make, which writes down what it is asked
and launches nothing.  No test here needs a GPU."""
from __future__ import annotations

import ctypes
import os
import shutil
import subprocess

import pytest

from paged_kv_gqa_02_gb300 import build, ops

OBJECTS = ("pa_step_api", "pa_rotate", "pa_verify", "pa_key_weights", "pa_key_weights_tc", "pa_evict")

FAKE = r"""
#include <cuda_runtime_api.h>
static int dev = 0, launches = 0, clusters[64], fits[17], fails = 0;
static int fake_encode() { return 0; }
extern "C" {
void fake_device(int d) { dev = d; launches = 0; }
// how many clusters of each size there are at once; a negative one: the question fails
void fake_fits(int size, int n) { fits[size] = n; }
int fake_launches(int* sizes) {
    for (int i = 0; i < launches && i < 64; ++i) sizes[i] = clusters[i];
    return launches;
}
cudaError_t cudaGetDevice(int* d) { *d = dev; return cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr, int) { *v = 152; return cudaSuccess; }
cudaError_t cudaFuncSetAttribute(const void*, cudaFuncAttribute, int) { return cudaSuccess; }
cudaError_t cudaGetLastError() { return cudaSuccess; }
cudaError_t cudaOccupancyMaxActiveClusters(int* n, const void*, const cudaLaunchConfig_t* c) {
    *n = fits[c->attrs[0].val.clusterDim.x];
    return *n < 0 ? cudaErrorInvalidValue : cudaSuccess;
}
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* c, const void*, void**) {
    int size = 0;
    for (unsigned i = 0; i < c->numAttrs; ++i)
        if (c->attrs[i].id == cudaLaunchAttributeClusterDimension) size = int(c->attrs[i].val.clusterDim.x);
    if (launches < 64) clusters[launches] = size;
    ++launches;
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
SHAPE = 2


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
    vp, i32, P, R = ctypes.c_void_p, ctypes.c_int32, ctypes.POINTER(ops.Params), ctypes.POINTER(ops.Rows)
    L.pa_verify.argtypes = [P, R, i32] + [vp] * 15
    L.pa_evict.argtypes = [P] + [vp] * 7 + [i32, i32] + [vp] * 5
    return L


def place(n):
    return ctypes.c_void_p(n << 24)  # aligned, far apart, never read


def evict(lib, **kw):
    p = ops.make_params(num_seqs=4, num_q_heads=2, num_kv_heads=2, head_dim=64, page_size=16, num_pages=10, max_blocks_per_seq=4,
                        max_context_len=64, dtype="bf16")
    a = {x: place(i + 1) for i, x in enumerate(("kc", "vc", "bt", "cl", "ref", "w", "keep", "out", "kept", "lens"))}
    a.update(kw)
    names = list(a)
    lib.fake_device(0)
    return lib.pa_evict(p, *(a[x] for x in names[:7]), 0, 0, *(a[x] for x in names[7:]), None, None)


def test_evict_refuses_outputs_over_its_inputs(lib):
    """4 sequences: 16 bytes of lengths; 2 heads of 64 slots: 2048 bytes of weights."""
    def at(n, off):
        return ctypes.c_void_p((n << 24) + off)
    assert evict(lib) == 0
    for other in ("cl", "keep"):
        for off in (0, 4, 12, -4, -12):
            assert evict(lib, **{other: at(99, 0), "lens": at(99, off)}) == SHAPE, (other, off)
        for off in (16, -16, 64):
            assert evict(lib, **{other: at(99, 0), "lens": at(99, off)}) == 0, (other, off)
    for off in (0, 16, 512, 2032, -16, -2032):
        assert evict(lib, w=at(99, 0), out=at(99, off)) == SHAPE, off
    for off in (2048, -2048):
        assert evict(lib, w=at(99, 0), out=at(99, off)) == 0, off
    assert evict(lib, keep=at(98, 0), cl=at(98, 0)) == 0  # both are read only


ON_A_GB300 = {16: 7, 8: 15, 6: 23, 5: 28, 4: 36, 3: 46, 2: 76, 1: 152}


def cluster_of(lib, seqs, vocab, dev, fits):
    """CTAs to a sequence of a verification on a device that answers `fits`."""
    for size in range(17):
        lib.fake_fits(size, fits.get(size, -1))
    lib.fake_device(dev)
    p, r = ops.verify_params(num_seqs=seqs, dtype="bf16"), ops.make_rows(2 * seqs, 2)
    assert lib.pa_verify(p, r, vocab, *[place(1)] * 13, None, None) == 0
    sizes = (ctypes.c_int * 64)()
    assert lib.fake_launches(sizes) == 2
    return sizes[0]


def test_clusters_of_a_verification(lib):
    """As wide as fit at once for all sequences, by the device's own answer; one CTA where it has none."""
    for seqs, size in ((1, 16), (7, 16), (8, 8), (15, 8), (17, 8), (18, 6), (23, 6), (24, 5), (28, 5), (36, 4), (46, 3), (76, 2), (77, 1), (500, 1)):
        assert cluster_of(lib, seqs, 131072, 0, ON_A_GB300) == size, seqs
    # a unit of eight tokens for every second thread of 512
    for vocab, size in ((32768, 16), (32767, 8), (16384, 8), (8192, 4), (4096, 2), (4095, 1), (1, 1)):
        assert cluster_of(lib, 1, vocab, 1, ON_A_GB300) == size, vocab
    small = {16: 0, 8: 0, 6: 1, 5: 1, 4: 2, 3: 3, 2: 5, 1: 10}  # a part of a GPU
    for seqs, size in ((1, 6), (2, 4), (3, 3), (5, 2), (6, 1)):
        assert cluster_of(lib, seqs, 131072, 2, small) == size, seqs
    assert cluster_of(lib, 14, 131072, 3, {**ON_A_GB300, 8: 12}) == 6  # no two more than it says
    for seqs in (1, 2):  # the question fails
        assert cluster_of(lib, seqs, 131072, 4, {}) == 1
