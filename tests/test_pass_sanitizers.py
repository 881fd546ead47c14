"""The host code of the verifier's pass (argument checks, planning, extents, rotary angles) under AddressSanitizer and
UndefinedBehaviorSanitizer on the CPU, sanitizers on the host side only, with every test of tests/test_pass_abi_cpu.py
run against it in a child process."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "lossless_draft_verification_04_amd", "csrc")
SOURCES = ["sv_pass_api.hip", "sv_rope.hip", "sv_kv.hip", "sv_kv_attention.hip"]
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

pytestmark = pytest.mark.slow


def test_pass_host_code_under_asan_and_ubsan(tmp_path):
    so = str(tmp_path / "libspecverify_pass_san.so")
    flags = ["--offload-arch=gfx950", "-O1", "-g", "-std=c++17", "-fPIC", "-shared", "-ffp-contract=off",
             "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
             "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
             "-Xarch_host", "-fno-sanitize-recover=undefined"]
    subprocess.run([HIPCC, *flags, "-I" + os.path.join(ROOT, "include"), *[os.path.join(CSRC, f) for f in SOURCES],
                    "-o", so], check=True, capture_output=True)
    clang = os.path.join(os.path.dirname(os.path.dirname(HIPCC)), "lib", "llvm", "lib", "clang")
    rt = [os.path.join(d, f) for d, _, fs in os.walk(clang) for f in fs if f == "libclang_rt.asan-x86_64.so"]
    assert rt, "clang ASan runtime not found"
    script = (
        "import ctypes, sys\n"
        f"sys.path.insert(0, {ROOT!r})\n"
        "from lossless_draft_verification_04_amd import specverify as svx\n"
        f"L = ctypes.CDLL({so!r})\n"
        "for name, (args, res) in svx._PASS_SIGS.items():\n"
        "    fn = getattr(L, name); fn.argtypes = args; fn.restype = res\n"
        "L.sv_status_string = svx._lib.sv_status_string\n"
        "svx._lib = L\n"
        "import tests.test_pass_abi_cpu as T\n"
        "T.L = L\n"
        "names = [k for k in dir(T) if k.startswith('test_')]\n"
        "for k in names:\n"
        "    getattr(T, k)()\n"
        "print('ran', len(names))\n")
    env = dict(os.environ, LD_PRELOAD=rt[0], ASAN_OPTIONS="detect_leaks=0:abort_on_error=1",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    res = subprocess.run([sys.executable, "-c", script], cwd=ROOT, env=env, capture_output=True, text=True, timeout=900)
    tail = (res.stdout + res.stderr)[-3000:]
    assert res.returncode == 0, tail
    assert "ran " in res.stdout and "runtime error" not in res.stderr, tail
