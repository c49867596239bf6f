"""The front ends of the gated linear recurrence and of the norms around a block (api_glr.cpp, api_block.cpp) under
AddressSanitizer and UBSan, host code only: their checks' tests against an instrumented build, as
tests/test_sanitizers_delta_cpu.py does for the delta rule's."""
import os

import pytest

from test_sanitizers_cpu import CSRC, HOST_SAN, OUT, ROOT, _asan_runtime_clang, _nm_has_asan, _pytest_child, _regular_objects, _run


@pytest.fixture(scope="module")
def san_library():
    bd, objs = _regular_objects()
    os.makedirs(OUT, exist_ok=True)
    common = [bd.hipcc(), "--offload-arch=" + bd.ARCH, "-O1", "-g", "-std=c++17", "-fPIC", "-Wall",
              "-I" + os.path.join(ROOT, "include"), "-I" + CSRC, *bd.DEVICE_FLAGS, *HOST_SAN]
    sources = ("api.cpp", "api_glr.cpp", "api_block.cpp", "log.cpp")
    names = [os.path.splitext(src)[0] + ".o" for src in sources]
    san_objs = []
    for src, name in zip(sources, names):
        obj = os.path.join(OUT, "block_" + name)
        _run(common + ["-c", "-o", obj, os.path.join(CSRC, src)])
        san_objs.append(obj)
    rest = [o for o in objs if os.path.basename(o) not in names]
    lib = os.path.join(OUT, "libssmscan_block_san.so")
    _run([bd.hipcc(), "--offload-arch=" + bd.ARCH, "-shared", "-fPIC", *HOST_SAN, "-shared-libsan", "-o", lib]
         + san_objs + rest)
    assert _nm_has_asan(lib)
    return lib


@pytest.mark.parametrize("name", ["test_glr_abi_cpu.py", "test_block_abi_cpu.py"])
def test_checks_under_asan_and_ubsan(san_library, name):
    text = _pytest_child([os.path.join(ROOT, "tests", name)],
                         {"LD_PRELOAD": _asan_runtime_clang(), "SSM_SCAN_LIBRARY": san_library}, timeout=600)
    assert " passed" in text
