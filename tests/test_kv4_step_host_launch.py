"""What digest and select launch, on stand-ins for the CUDA runtime: grids and
clusters that follow from the sizes (no GPU needed)."""

import ctypes
import shutil
import subprocess
from pathlib import Path

import pytest

import mla_decode_query_gb300 as mq
from mla_decode_query_gb300 import build
from mla_decode_query_gb300.mlaqp import _SIGNATURES

STAND_INS = r"""
#include "mlaqp_host.h"
#include "mlaqp_kv4_launch.h"

#include <cstring>
#include <string>

extern "C" {
int device = 0;                                // the current one
int sms[2] = {152, 152};
int room[2][2] = {{1, 1}, {1, 1}};             // clusters of 16 that a device has room for: BF16 queries, E4M3
unsigned grid = 0, threads = 0, cluster = 0;   // of the last launch
int launches = 0;
static std::string names[16];
static const void* functions[16];
static int n_functions = 0;

cudaError_t cudaGetDevice(int* d) { *d = device; return cudaSuccess; }
cudaError_t cudaSetDevice(int d) { device = d; return cudaSuccess; }
cudaError_t cudaGetLastError() { return cudaSuccess; }
cudaError_t cudaFuncGetAttributes(cudaFuncAttributes*, const void*) { return cudaSuccess; }
cudaError_t cudaFuncSetAttribute(const void*, cudaFuncAttribute, int) { return cudaSuccess; }
cudaError_t cudaMemcpyFromSymbol(void*, const void*, size_t, size_t, cudaMemcpyKind) { return cudaSuccess; }
cudaError_t cudaMemcpyToSymbol(const void*, const void*, size_t, size_t, cudaMemcpyKind) { return cudaSuccess; }
cudaError_t cudaOccupancyMaxActiveClusters(int* n, const void* fn, const cudaLaunchConfig_t*) {
  *n = 0;
  for (int i = 0; i < n_functions; ++i)
    if (functions[i] == fn) *n = room[device][names[i].find("Lb1E") != std::string::npos];
  return cudaSuccess;
}
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* cfg, const void*, void**) {
  grid = cfg->gridDim.x;
  threads = cfg->blockDim.x;
  cluster = 1;
  for (unsigned i = 0; i < cfg->numAttrs; ++i)
    if (cfg->attrs[i].id == cudaLaunchAttributeClusterDimension) cluster = cfg->attrs[i].val.clusterDim.x;
  ++launches;
  return cudaSuccess;
}
// what nvcc's host code calls when a library is loaded
void** __cudaRegisterFatBinary(void*) { static void* handle; return &handle; }
void __cudaRegisterFatBinaryEnd(void**) {}
void __cudaUnregisterFatBinary(void**) {}
void __cudaRegisterFunction(void**, const char* host, char*, const char* name, int, void*, void*, void*, void*, int*) {
  functions[n_functions] = host;
  names[n_functions++] = name;
}
void __cudaRegisterVar(void**, char*, char*, const char*, int, size_t, int, int) {}
int __cudaGetKernel(void**, const void*) { return 0; }
int __cudaLaunchKernel(void*, dim3, dim3, void**, size_t, void*) { return 0; }
int __cudaPopCallConfiguration(dim3*, dim3*, size_t*, void*) { return 0; }
int64_t mlaqp_kv4_page_bytes(int page_size) { return 400 * page_size; }
}

namespace mlaqp {
int host_fail(int status, const std::string&) { return status; }
int host_fail_cuda(const char*, cudaError_t) { return 3; }
int host_device(int asked, int* resolved, int* sm_count) {
  *resolved = asked < 0 ? device : asked;
  *sm_count = sms[*resolved];
  return 0;
}
cudaError_t kv4_rope_setup() { return cudaSuccess; }
cudaError_t kv4_append_rope(const Kv4RopeParams&, bool, cudaStream_t) { return cudaSuccess; }
}  // namespace mlaqp
"""

A = 1 << 24  # fake, aligned device addresses, never dereferenced


@pytest.fixture(scope="module")
def stand_in_library(tmp_path_factory):
    d = tmp_path_factory.mktemp("kv4_step_launch")
    (d / "stand_ins.cpp").write_text(STAND_INS)
    cuda = Path(build.nvcc_path()).resolve().parent.parent / "include"
    include = [f"-I{build.INCLUDE}", f"-I{build.CSRC}"]
    jobs = [[build.nvcc_path(), "-gencode", "arch=compute_103a,code=compute_103a", "-O1", "-std=c++17", "-Xcompiler", "-fPIC",
             *include, "-c", str(build.CSRC / f"mlaqp_kv4_{u}.cu"), "-o", str(d / f"{u}.o")] for u in ("digest", "select", "step_api")]
    jobs.append([shutil.which("g++"), "-std=c++17", "-fPIC", *include, f"-I{cuda}", "-c", str(d / "stand_ins.cpp"), "-o",
                 str(d / "stand_ins.o")])
    for p in [subprocess.Popen(j) for j in jobs]:
        assert p.wait() == 0
    so = d / "libkv4_step_launch.so"
    # -Bsymbolic: its own stand-ins, not what libraries loaded before it export
    subprocess.run([shutil.which("g++"), "-shared", "-Wl,-Bsymbolic", *(str(d / f"{u}.o") for u in ("stand_ins", "digest", "select",
                                                                                               "step_api")), "-o", str(so)], check=True)
    return so


@pytest.fixture
def lib(stand_in_library, tmp_path):
    copy = tmp_path / "lib.so"  # a library of its own: what is ready is kept once per process
    shutil.copy(stand_in_library, copy)
    lib = ctypes.CDLL(str(copy))
    for name, (res, args) in _SIGNATURES.items():
        if hasattr(lib, name):
            getattr(lib, name).restype, getattr(lib, name).argtypes = res, args
    return lib


def _int(lib, name):
    return ctypes.c_int.in_dll(lib, name)


def _digest(lib, n, max_new, table_stride, num_pages, page_size=16):
    st = lib.mlaqp_kv4_digest(1 << 40, 400 * page_size, num_pages, page_size, A, table_stride, 64, 2 * A, 3 * A, 4 * A, n, max_new,
                              1 << 44, 1168, None)
    assert st == mq.MLAQP_OK
    return _int(lib, "grid").value, _int(lib, "threads").value


@pytest.mark.parametrize("n,max_new,table_stride,num_pages,jobs", [
    (3, 17, 100, 1000, 6),                       # ceil(17 / 16) pages an item
    (3, 16, 100, 1000, 3),
    (3, (1 << 31) - 1, 4, 1000, 12),             # no row holds more than four
    (3, (1 << 31) - 1, 1 << 31, 5, 15),          # no sequence more than the pool
    (64, (1 << 31) - 1, 8, 1 << 20, 512),
    (1, 1 << 20, 2, 1 << 20, 2),
])
def test_digest_looks_up_no_more_pages_than_there_can_be(lib, n, max_new, table_stride, num_pages, jobs):
    # so few that four warps a page find room at once: a CTA each
    assert _digest(lib, n, max_new, table_stride, num_pages) == (jobs, 128)


def _select(lib, e4m3=0, B=1, table_stride=8192):
    st = lib.mlaqp_kv4_select(A, 576 * 16, e4m3, 1 << 40, 1168, 8192, 16, 2 * A, table_stride, 4, 3 * A, None, B, 1, 16, 4, 1, 1,
                              4 * A, 4, 5 * A, 6 * A, 1 << 20, None)
    assert st == mq.MLAQP_OK
    assert _int(lib, "grid").value == B * _int(lib, "cluster").value
    return _int(lib, "cluster").value


def _rooms(lib, *rooms):
    at = (ctypes.c_int * 4).in_dll(lib, "room")
    at[:] = [n for device in rooms for n in device]


@pytest.mark.parametrize("order", [(0, 1), (1, 0)])
def test_wide_clusters_on_the_devices_that_have_room(lib, order):
    _rooms(lib, (1, 1), (0, 0))
    for device in order:
        assert lib.mlaqp_kv4_step_prewarm(device) == mq.MLAQP_OK
    for device in (0, 1, 0):
        _int(lib, "device").value = device
        assert _select(lib) == (16, 8)[device]


def test_wide_clusters_of_the_kernels_that_have_room(lib):
    _rooms(lib, (1, 0), (0, 1))
    for device in (0, 1):
        _int(lib, "device").value = device
        assert (_select(lib, 0), _select(lib, 1)) == ((16, 8), (8, 16))[device]


@pytest.mark.parametrize("B,table_stride,cluster", [(1, 8192, 16), (1, 1024, 16), (1, 512, 16), (1, 256, 8), (1, 100, 4), (1, 32, 1)])
def test_clusters_follow_the_table(lib, B, table_stride, cluster):
    assert _select(lib, B=B, table_stride=table_stride) == cluster
