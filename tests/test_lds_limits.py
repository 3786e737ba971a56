"""Launches from several host threads whose LDS depends on the sizes, without a GPU: see
asan/lds_limit_checks.cpp, which replaces the runtime's launch calls by records."""
import os
import subprocess

import pytest

from skinny_gemm_projection_amd import build

HIPCC = build.hipcc()
SOURCE = os.path.join(build.ROOT, "tests", "asan", "lds_limit_checks.cpp")


@pytest.mark.skipif(not os.path.exists(HIPCC) or not os.path.exists(SOURCE), reason="hipcc or source not found")
def test_no_call_lowers_the_limit_of_another(tmp_path):
    objects = [os.path.join(build.BUILD, os.path.splitext(s)[0] + ".o") for s in build.SOURCES]
    missing = [o for o in objects if not os.path.exists(o)]
    if missing:
        pytest.skip(f"build the library first: {missing}")
    obj, exe = str(tmp_path / "checks.o"), str(tmp_path / "lds_limit_checks")
    for cmd in ([HIPCC, "-c", "-x", "hip", "--offload-arch=gfx950", "-std=c++17", "-O1", SOURCE, "-o", obj,
                 "-I", build.INCLUDE, "-I", build.CSRC],
                [HIPCC, "--offload-arch=gfx950", "-o", exe, obj] + objects):
        r = subprocess.run(cmd, capture_output=True, text=True, timeout=600)
        assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=100)
    assert r.returncode == 0 and "lds_limit_checks: ok" in r.stdout, r.stdout + r.stderr
