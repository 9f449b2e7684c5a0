"""The training entry points' host-side checks under AddressSanitizer and
UndefinedBehaviorSanitizer (api.cpp rebuilt with them on the host side, the
kernels as built). CPU only: no call reaches the GPU."""
import glob
import os
import shutil
import subprocess

import pytest

from test_sanitizers_cpu import CSRC, ENV, HERE, HIPCC, ROOT, SAN


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not installed")
def test_training_validation_under_asan_ubsan(tmp_path):
    flags = ["--offload-arch=gfx950", "-O1", "-g", "-std=c++17", "-fPIC",
             "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
             "-I", os.path.join(ROOT, "include")]
    objs = []
    for src in sorted(glob.glob(os.path.join(CSRC, "*.hip")) + glob.glob(os.path.join(CSRC, "*.cpp"))):
        base = os.path.basename(src)
        obj = str(tmp_path / (base + ".o"))
        built = os.path.join(ROOT, "_build", base + ".o")
        if base != "api.cpp" and os.path.exists(built):
            shutil.copy(built, obj)
        else:
            extra = SAN if base == "api.cpp" else ["-O3"]
            subprocess.run([HIPCC] + flags + extra + ["-c", src, "-o", obj], check=True, capture_output=True)
        objs.append(obj)
    lib = str(tmp_path / "libbimamba_asan.so")
    subprocess.run([HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", "-o", lib] + objs, check=True,
                   capture_output=True)
    exe = str(tmp_path / "abi_train_asan")
    subprocess.run(["/opt/rocm/llvm/bin/clang", "-O1", "-g", "-fsanitize=address,undefined",
                    "-fno-sanitize-recover=all", "-I", os.path.join(ROOT, "include"),
                    os.path.join(HERE, "abi_train_main.c"), lib, "-Wl,-rpath," + str(tmp_path),
                    "-L/opt/rocm/lib", "-lamdhip64", "-Wl,-rpath,/opt/rocm/lib", "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, env=ENV, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "runtime error" not in r.stderr, r.stderr
    assert "abi training checks: ok" in r.stdout, r.stdout
