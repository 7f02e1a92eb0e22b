"""The host-side argument checks of the operators around the SSD layer under
AddressSanitizer and UndefinedBehaviorSanitizer (CPU only, no GPU call), as
test_abi_sanitized.py runs those of the other entry points."""
import glob
import os
import shutil
import subprocess
import sys

import pytest

from test_abi_sanitized import PKG, ROCM, ROOT

FILES = ("test_block_abi_host.py", "test_block_limits_host.py", "test_block_workspace_host.py")


def test_block_host_checks_under_asan_and_ubsan(tmp_path):
    objs = sorted(o for o in glob.glob(os.path.join(PKG, "_build", "*.o"))
                  if os.path.basename(o) not in ("ssm_abi.cpp.o", "ssm_calib.hip.o"))
    if not objs or not shutil.which("g++"):
        pytest.skip("the library's objects are not built (run __graft_entry__.build()) or g++ is missing")
    asan = subprocess.run(["g++", "-print-file-name=libasan.so"], capture_output=True, text=True).stdout.strip()
    if not os.path.exists(asan):
        pytest.skip("libasan is not installed")
    san = ["-fsanitize=address,undefined", "-fno-sanitize-recover=undefined", "-fno-omit-frame-pointer"]
    obj, lib = str(tmp_path / "ssm_abi_san.o"), str(tmp_path / "libssm_san.so")
    subprocess.run(["g++", "-std=c++17", "-O1", "-g", "-fPIC", "-D__HIP_PLATFORM_AMD__", *san,
                    "-I", os.path.join(ROCM, "include"), "-I", os.path.join(ROOT, "include"),
                    "-c", os.path.join(PKG, "csrc", "ssm_abi.cpp"), "-o", obj], check=True)
    subprocess.run(["g++", "-shared", *san, "-o", lib, obj, *objs, "-L", os.path.join(ROCM, "lib"),
                    "-lamdhip64", "-Wl,-rpath," + os.path.join(ROCM, "lib")], check=True)
    env = dict(os.environ, SSM_LIBRARY=lib, LD_PRELOAD=asan,
               ASAN_OPTIONS="detect_leaks=0:halt_on_error=1:abort_on_error=1",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    # the binding-with-torch case is left out: torch is not built with the sanitizer
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-p", "no:cacheprovider",
                        "-k", "not binding_refuses_cpu_tensors", *(os.path.join(ROOT, "tests", f) for f in FILES)],
                       env=env, capture_output=True, text=True, cwd=ROOT, timeout=600)
    out = r.stdout[-4000:] + r.stderr[-4000:]
    assert r.returncode == 0, out
    assert "ERROR: AddressSanitizer" not in out and "runtime error" not in out, out
    assert " passed" in r.stdout, out
