"""Host side of the 4-bit cache on stand-ins for the device and the kernels:
kernels of one group that cannot be made ready refuse the calls that need
them, and no others (no GPU needed)."""

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

extern "C" {
int fail_rows = 0, fail_pages = 0, fail_attend16 = 0, fail_attend32 = 0, launches = 0, setups = 0;
cudaError_t cudaGetDevice(int* d) { *d = 0; return cudaSuccess; }
cudaError_t cudaSetDevice(int) { return cudaSuccess; }
cudaError_t cudaGetLastError() { return cudaSuccess; }
}

namespace mlaqp {
int host_fail(int status, const std::string&) { return status; }
int host_fail_cuda(const char*, cudaError_t) { return 3; }
int host_device(int, int* resolved, int* sm_count) { *resolved = 0; *sm_count = 152; return 0; }
static cudaError_t up(int fail) { ++setups; return fail ? cudaErrorInvalidKernelImage : cudaSuccess; }
static cudaError_t launch() { ++launches; return cudaSuccess; }
cudaError_t kv4_rows_setup() { return up(fail_rows); }
cudaError_t kv4_pages_setup() { return up(fail_pages); }
cudaError_t kv4_attend_setup(int rows) { return up(rows == 16 ? fail_attend16 : fail_attend32); }
int kv4_attend_rows(int q_len, int H) { return q_len * H <= 16 ? 16 : 32; }
cudaError_t kv4_append(const Kv4RowsParams&, cudaStream_t) { return launch(); }
cudaError_t kv4_gather(const Kv4RowsParams&, cudaStream_t) { return launch(); }
cudaError_t kv4_extend(const Kv4PagesParams&, cudaStream_t) { return launch(); }
cudaError_t kv4_fork(const Kv4PagesParams&, int, cudaStream_t) { return launch(); }
cudaError_t kv4_release(const Kv4PagesParams&, cudaStream_t) { return launch(); }
cudaError_t kv4_compact(const Kv4PagesParams&, int, cudaStream_t) { return launch(); }
cudaError_t kv4_copy_pages(const Kv4PagesParams&, int, cudaStream_t) { return launch(); }
cudaError_t kv4_attend(const Kv4AttendParams&, bool, int, cudaStream_t) { return launch(); }
int64_t kv4_pages_workspace(int, int) { return 64; }
int64_t kv4_attend_workspace(int, int, int, int) { return 64; }
}  // namespace mlaqp
"""

A = 1 << 24  # fake, aligned device addresses, never dereferenced
TABLES = (A, 8, 4, 2 * A, 3 * A, 64, 16)
POOL = (8 * A, 6400, 6400 * 64, 3)


def _attend(lib, q_len):
    return lib.mlaqp_kv4_attend(A, 576 * 16, 0, None, 8 * A, 6400, 64, 16, 4 * A, 4, 3, 5 * A, None, 3, q_len, 16, 0.07,
                                2 * A, 512 * 16, 3 * A, 16 * A, 1 << 20, None)


CALLS = {
    "rows": [lambda lib: lib.mlaqp_kv4_append(A, 576, A + 1024, 576, 8 * A, 6400, 64, 16, 4 * A, 3, None),
             lambda lib: lib.mlaqp_kv4_gather(8 * A, 6400, 64, 16, 4 * A, 3, A, 576, None)],
    "pages": [lambda lib: lib.mlaqp_kv4_extend(*TABLES, 4 * A, 5 * A, 2, 6 * A, 4, None),
              lambda lib: lib.mlaqp_kv4_fork(*TABLES, 4 * A, 5 * A, 2, *POOL, 7 * A, 1 << 20, None),
              lambda lib: lib.mlaqp_kv4_release(*TABLES, 4 * A, 2, None),
              lambda lib: lib.mlaqp_kv4_compact(*TABLES, *POOL, 6 * A, 7 * A, 1 << 20, None),
              lambda lib: lib.mlaqp_kv4_copy_pages(*POOL, 64, 16, A, 2 * A, 2, None)],
    "attend16": [lambda lib: _attend(lib, 1)],
    "attend32": [lambda lib: _attend(lib, 2)],
}


@pytest.fixture(scope="module")
def stand_in_library(tmp_path_factory):
    d = tmp_path_factory.mktemp("kv4_host")
    (d / "stand_ins.cpp").write_text(STAND_INS)
    cuda = Path(build.nvcc_path()).resolve().parent.parent / "include"
    so = d / "libkv4_host.so"
    # -Bsymbolic: its own stand-ins, not what libraries loaded before it export
    subprocess.run([shutil.which("g++"), "-std=c++17", "-shared", "-fPIC", "-Wl,-Bsymbolic", f"-I{build.INCLUDE}",
                    f"-I{build.CSRC}", f"-I{cuda}", "-x", "c++", str(build.CSRC / "mlaqp_kv4_api.cu"), str(d / "stand_ins.cpp"), "-o", str(so)], check=True)
    return so


def _load(so, tmp_path):
    copy = tmp_path / "lib.so"  # a library of its own: what is ready is kept once per process
    shutil.copy(so, copy)
    lib = ctypes.CDLL(str(copy))
    for name, (res, args) in _SIGNATURES.items():
        if hasattr(lib, name):
            getattr(lib, name).restype, getattr(lib, name).argtypes = res, args
    return lib


@pytest.mark.parametrize("broken", ["none", "rows", "pages", "attend16", "attend32"])
def test_only_the_calls_that_need_them_are_refused(stand_in_library, tmp_path, broken):
    lib = _load(stand_in_library, tmp_path)
    if broken != "none":
        ctypes.c_int.in_dll(lib, f"fail_{broken}").value = 1
    launches = ctypes.c_int.in_dll(lib, "launches")
    for group, calls in CALLS.items():
        for call in calls:
            before = launches.value
            want = mq.MLAQP_ERR_CUDA if group == broken else mq.MLAQP_OK
            assert call(lib) == want, group
            assert launches.value - before == (group != broken)
    assert lib.mlaqp_kv4_attend_workspace(3, 1, 16, -1) == (-1 if broken == "attend16" else 64)
    assert lib.mlaqp_kv4_attend_workspace(3, 2, 16, -1) == (-1 if broken == "attend32" else 64)
    assert lib.mlaqp_kv4_prewarm(-1) == (mq.MLAQP_OK if broken == "none" else mq.MLAQP_ERR_CUDA)


def test_kernels_are_made_ready_once_by_the_first_call(stand_in_library, tmp_path):
    lib = _load(stand_in_library, tmp_path)
    assert CALLS["rows"][0](lib) == mq.MLAQP_OK
    assert ctypes.c_int.in_dll(lib, "setups").value == 4
    for _ in range(3):
        for calls in CALLS.values():
            for call in calls:
                assert call(lib) == mq.MLAQP_OK
    assert lib.mlaqp_kv4_prewarm(-1) == mq.MLAQP_OK
    assert ctypes.c_int.in_dll(lib, "setups").value == 4
