"""The host tests of the layer operators, the grouped products and the q4_G products again, with their
argument checks built under AddressSanitizer and UBSan (CPU only).

The entry points' sources, which hold all of the host's arithmetic on sizes, are compiled with both (host
code only) into a library that takes the rest, launchers included, from the built libmmq.so. The package,
copied next to it, runs the host tests in a child process with the ASan runtime preloaded; any report
aborts the child and fails this test.
"""
import os
import shutil
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

import pytest

from tests import test_abi_sanitized as san

pytest.importorskip("q4_q8_int8_amd")

SOURCES = ["api.cpp", "moe_api.cpp", "grouped_api.cpp", "q4g_api.cpp"]
TESTS = ["test_layer_host.py", "test_grouped_host.py", "test_q4g_host.py", "test_sizes_host.py"]


@pytest.mark.skipif(not os.path.exists(san.build.HIPCC), reason="hipcc not found")
def test_entry_points_under_asan_and_ubsan():
    runtime = san._asan_runtime()
    if not runtime:
        pytest.skip("no ASan runtime next to the ROCm clang")
    tmp = tempfile.mkdtemp(prefix="mmq_san_")
    try:
        pkg = os.path.join(tmp, "pkg", "q4_q8_int8_amd")
        os.makedirs(pkg)

        def compile_one(src):
            obj = os.path.join(tmp, src + ".o")
            r = subprocess.run([san.build.HIPCC, *san.build.FLAGS, *san.SAN, "-c",
                                os.path.join(san.build.CSRC, src), "-o", obj],
                               capture_output=True, text=True)
            assert r.returncode == 0, r.stderr[-2000:]
            return obj

        with ThreadPoolExecutor(len(SOURCES)) as ex:
            objs = list(ex.map(compile_one, SOURCES))
        lib = os.path.join(pkg, "libmmq.so")
        rest = os.path.join(tmp, "libmmq_rest.so")
        shutil.copy(san.build.LIB, rest)
        r = subprocess.run([san.build.HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC",
                            "-Xarch_host", "-fsanitize=address", "-Xarch_host",
                            "-fsanitize=undefined", "-shared-libasan", *objs, rest,
                            f"-Wl,-rpath,{tmp}", "-o", lib], capture_output=True, text=True)
        assert r.returncode == 0, r.stderr[-2000:]
        nm = subprocess.run(["nm", "-D", lib], capture_output=True, text=True, check=True).stdout
        assert "__asan_report" in nm and "__ubsan_handle" in nm and "T mmq_q4K_grouped\n" in nm
        shutil.copy(os.path.join(san.ROOT, "q4_q8_int8_amd", "__init__.py"), pkg)
        shutil.copytree(os.path.join(san.ROOT, "include"), os.path.join(tmp, "pkg", "include"))
        runner = os.path.join(tmp, "run.py")
        with open(runner, "w") as f:
            f.write(san.RUNNER.replace("sys.argv[2]]", "*sys.argv[2:]]"))
        env = dict(os.environ, LD_PRELOAD=runtime,
                   ASAN_OPTIONS="detect_leaks=0:alloc_dealloc_mismatch=0:halt_on_error=1",
                   UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
        r = subprocess.run([sys.executable, runner, os.path.join(tmp, "pkg"),
                            *(os.path.join(san.ROOT, "tests", t) for t in TESTS),
                            "-k", "not compiler"],   # (those that only compile)
                           capture_output=True, text=True, env=env, cwd=san.ROOT, timeout=600)
        out = r.stdout + r.stderr
        assert r.returncode == 0, out[-4000:]
        assert "passed" in out and "ERROR: AddressSanitizer" not in out \
            and "runtime error" not in out, out[-4000:]
    finally:
        shutil.rmtree(tmp, ignore_errors=True)
