"""The paged handle's host side over a fake CUDA runtime (fake_cuda_runtime.cpp, fake_paged_launches.cu): its device, its status word."""
import ctypes
import os
import subprocess

import pytest

from head_partitioned_sparse_b200 import binding as B
from head_partitioned_sparse_b200 import build

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    so = tmp_path_factory.mktemp("fake") / "libfake.so"
    # -Bsymbolic: its own runtime, also where torch has loaded the real one
    subprocess.run([build._nvcc(), "-gencode", "arch=compute_100a,code=sm_100a", "-O1", "-std=c++17", "--shared", "-cudart", "none",
                    "-Xcompiler", "-fPIC", "-Xlinker", "-Bsymbolic", "-I", build.CSRC, "-I", os.path.join(build.ROOT, "include"), "-o", str(so),
                    os.path.join(build.CSRC, "spa_paged.cu"), os.path.join(HERE, "fake_paged_launches.cu"), os.path.join(HERE, "fake_cuda_runtime.cpp")], check=True)
    lib = ctypes.CDLL(str(so))
    for name in ("spa_paged_create", "spa_paged_destroy", "spa_paged_status", "spa_kv_append_paged"):
        getattr(lib, name).argtypes = B._SIGS[name][1]
    lib.fake_last_error.restype = ctypes.c_char_p
    return lib


def var(lib, name):
    return ctypes.c_int.in_dll(lib, name)


@pytest.fixture()
def handle(lib):
    var(lib, "fake_device").value = 0
    h = ctypes.c_void_p()
    cfg = B.make_paged_config(max_batch=1, n_q_heads=1, n_kv_heads=1, kv_dtype=B.SPA_BF16, page_format=B.SPA_PAGE_INT4,
                              page_size=16, n_pages=1, max_pages=1)
    assert lib.spa_paged_create(ctypes.byref(h), ctypes.byref(cfg), None) == B.SPA_OK
    yield h
    if h.value:
        lib.spa_paged_destroy(h)
    assert var(lib, "fake_allocs").value == 0


def append(lib, h):
    X = 0x10000
    assert lib.spa_kv_append_paged(h, X, None, X, None, X, None, 1, 1, X, X, None) == B.SPA_OK


def test_status_keeps_what_was_set_after_it_was_read(lib, handle):
    """Appends of another stream may set a bit between the read of the status word and its clearing."""
    append(lib, handle)
    var(lib, "hook_after_read").value = 16        # a block_table entry
    assert lib.spa_paged_status(handle, None) == B.SPA_ERR_DEVICE_RANGE
    assert b"position" in lib.fake_last_error() and b"block_table" not in lib.fake_last_error()
    assert lib.spa_paged_status(handle, None) == B.SPA_ERR_DEVICE_RANGE
    assert b"block_table" in lib.fake_last_error() and b"position" not in lib.fake_last_error()
    assert lib.spa_paged_status(handle, None) == B.SPA_OK


def test_status_needs_the_handles_device(lib, handle):
    append(lib, handle)
    var(lib, "fake_device").value = 1
    assert lib.spa_paged_status(handle, None) == B.SPA_ERR_INVALID_ARG
    assert b"device" in lib.fake_last_error()
    var(lib, "fake_device").value = 0
    assert lib.spa_paged_status(handle, None) == B.SPA_ERR_DEVICE_RANGE
    assert lib.spa_paged_status(handle, None) == B.SPA_OK


def test_destroy_waits_for_the_handles_device(lib, handle):
    var(lib, "fake_device").value = 1
    var(lib, "fake_synced_on").value = var(lib, "fake_freed_on").value = -1
    assert lib.spa_paged_destroy(handle) == B.SPA_OK
    handle.value = None
    assert var(lib, "fake_synced_on").value == 0 and var(lib, "fake_freed_on").value == 0
    assert var(lib, "fake_device").value == 1
