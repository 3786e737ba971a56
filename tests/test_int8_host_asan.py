"""Host code of the 8-bit integer operators under AddressSanitizer (CPU only): int8_api.cpp with
the library's other host sources instrumented for the host only (-Xarch_host before each
-fsanitize=), linked with the GPU objects of the normal build."""
import os
import shutil

import pytest

from test_host_asan import BUILD, CSRC, GPU_OBJECTS, HIPCC, HOST_SOURCES, ROOT, _check_run, _run

OBJECTS = GPU_OBJECTS + ["int8", "norm_quant"]
SOURCES = HOST_SOURCES + ["int8_api.cpp"]


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not found")
def test_int8_host_code_under_address_sanitizer(tmp_path):
    missing = [o for o in OBJECTS if not os.path.exists(os.path.join(BUILD, o + ".o"))]
    if missing:
        pytest.skip(f"build the library first: {missing}")
    flags = ["-x", "hip", "--offload-arch=gfx950", "-std=c++17", "-O1", "-g", "-fPIC",
             "-I", os.path.join(ROOT, "include"), "-I", CSRC,
             "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
             "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fno-omit-frame-pointer"]
    objs = []
    for src in [os.path.join(CSRC, s) for s in SOURCES] + [os.path.join(ROOT, "tests", "asan", "int8_checks.cpp")]:
        obj = str(tmp_path / (os.path.basename(src) + ".o"))
        _run([HIPCC, "-c", src, "-o", obj] + flags)
        objs.append(obj)
    exe = str(tmp_path / "int8_checks")
    _run([HIPCC, "--offload-arch=gfx950", "-o", exe] + objs +
         [os.path.join(BUILD, o + ".o") for o in OBJECTS] +
         ["-Xarch_host", "-fsanitize=address"])
    _check_run(exe, {}, "int8_checks")
