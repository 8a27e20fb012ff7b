"""Host side of the calls around the attention over the 4-bit cache on
stand-ins for the device and the kernels: kernels that cannot be made ready
refuse the calls that need them, and no others (no GPU needed)."""

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
int fail_rope = 0, fail_digest = 0, fail_select = 0, launches = 0, setups = 0;
cudaError_t cudaGetDevice(int* d) { *d = 0; return cudaSuccess; }
cudaError_t cudaSetDevice(int) { return cudaSuccess; }
cudaError_t cudaGetLastError() { return cudaSuccess; }
int64_t mlaqp_kv4_page_bytes(int page_size) { return 400 * page_size; }
}

namespace mlaqp {
int host_fail(int status, const std::string&) { return status; }
int host_fail_cuda(const char*, cudaError_t) { return 3; }
int host_device(int, int* resolved, int* sm_count) { *resolved = 0; *sm_count = 152; return 0; }
static cudaError_t up(int fail) { ++setups; return fail ? cudaErrorInvalidKernelImage : cudaSuccess; }
static cudaError_t launch() { ++launches; return cudaSuccess; }
cudaError_t kv4_rope_setup() { return up(fail_rope); }
cudaError_t kv4_digest_setup() { return up(fail_digest); }
cudaError_t kv4_select_setup() { return up(fail_select); }
cudaError_t kv4_append_rope(const Kv4RopeParams&, bool, cudaStream_t) { return launch(); }
cudaError_t kv4_digest(const Kv4DigestParams&, int, cudaStream_t) { return launch(); }
cudaError_t kv4_select(const Kv4SelectParams&, bool, int, cudaStream_t) { return launch(); }
}  // namespace mlaqp
"""

A = 1 << 24  # fake, aligned device addresses, never dereferenced
CALLS = {
    "rope": lambda lib: lib.mlaqp_kv4_append_rope(A, 576, 2 * A, 1e-6, A + 1024, 576, 3 * A, 1024, 64, 3 * A, 1024, 64, 16, 4 * A,
                                                  5 * A, 300, 0, 8 * A, 6400, 64, 16, 6 * A, 3, None),
    "digest": lambda lib: lib.mlaqp_kv4_digest(8 * A, 6400, 64, 16, A, 8, 4, 2 * A, 3 * A, 4 * A, 2, 17, 16 * A, 1168, None),
    "select": lambda lib: lib.mlaqp_kv4_select(A, 576 * 16, 0, 16 * A, 1168, 64, 16, 2 * A, 8, 4, 3 * A, None, 3, 2, 16, 4, 1, 1,
                                               4 * A, 4, 5 * A, 6 * A, 1 << 20, None),
}


@pytest.fixture(scope="module")
def stand_in_library(tmp_path_factory):
    d = tmp_path_factory.mktemp("kv4_step_host")
    (d / "stand_ins.cpp").write_text(STAND_INS)
    cuda = Path(build.nvcc_path()).resolve().parent.parent / "include"
    so = d / "libkv4_step_host.so"
    # -Bsymbolic: its own stand-ins, not what libraries loaded before it export
    subprocess.run([shutil.which("g++"), "-std=c++17", "-shared", "-fPIC", "-Wl,-Bsymbolic", f"-I{build.INCLUDE}",
                    f"-I{build.CSRC}", f"-I{cuda}", "-x", "c++", str(build.CSRC / "mlaqp_kv4_step_api.cu"),
                    str(d / "stand_ins.cpp"), "-o", str(so)], check=True)
    return so


def _load(so, tmp_path):
    copy = tmp_path / "lib.so"  # a library of its own: what is ready is kept once per process
    shutil.copy(so, copy)
    lib = ctypes.CDLL(str(copy))
    for name, (res, args) in _SIGNATURES.items():
        if hasattr(lib, name):
            getattr(lib, name).restype, getattr(lib, name).argtypes = res, args
    return lib


@pytest.mark.parametrize("broken", ["none", *CALLS])
def test_only_the_calls_that_need_them_are_refused(stand_in_library, tmp_path, broken):
    lib = _load(stand_in_library, tmp_path)
    if broken != "none":
        ctypes.c_int.in_dll(lib, f"fail_{broken}").value = 1
    launches = ctypes.c_int.in_dll(lib, "launches")
    for group, call in CALLS.items():
        before = launches.value
        assert call(lib) == (mq.MLAQP_ERR_CUDA if group == broken else mq.MLAQP_OK), group
        assert launches.value - before == (group != broken)
    assert lib.mlaqp_kv4_step_prewarm(-1) == (mq.MLAQP_OK if broken == "none" else mq.MLAQP_ERR_CUDA)


def test_kernels_are_made_ready_once_by_the_first_call(stand_in_library, tmp_path):
    lib = _load(stand_in_library, tmp_path)
    setups = ctypes.c_int.in_dll(lib, "setups")
    assert CALLS["select"](lib) == mq.MLAQP_OK
    assert setups.value == 3
    for _ in range(3):
        for call in CALLS.values():
            assert call(lib) == mq.MLAQP_OK
    assert lib.mlaqp_kv4_step_prewarm(-1) == mq.MLAQP_OK
    assert setups.value == 3
