"""The host side of the operators beside KDA (argument checks, size
arithmetic, launch plans) rebuilt with AddressSanitizer and
UndefinedBehaviorSanitizer on the host pass only, together with the rest of
the library, and its C-ABI tests run against that build (no GPU needed)."""
import os
import sys
from concurrent.futures import ThreadPoolExecutor

import pytest

from test_sanitizers_cpu import HIPCC, OUT, ROOT, _clang_asan_runtime, _env, _run


@pytest.mark.skipif(_clang_asan_runtime() is None or not os.path.exists(HIPCC), reason="needs hipcc and clang's ASan")
def test_hybrid_host_code_under_asan_and_ubsan():
    from gated_delta_rule_91_amd.build import SOURCES
    out = OUT + "_hybrid"
    os.makedirs(out, exist_ok=True)
    csrc = os.path.join(ROOT, "gated_delta_rule_91_amd", "csrc")
    names = [os.path.splitext(s)[0] for s in SOURCES]
    flags = ["--offload-arch=gfx950", "-O1", "-g", "-std=c++17", "-fPIC",
             "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops", "-I", os.path.join(ROOT, "include"),
             "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
             "-Xarch_host", "-fno-sanitize-recover=undefined", "-Xarch_host", "-fno-omit-frame-pointer"]

    def compile_one(name):
        return _run([HIPCC, *flags, "-c", os.path.join(csrc, name + ".hip"), "-o", os.path.join(out, name + ".o")])

    with ThreadPoolExecutor(os.cpu_count() or 1) as ex:
        for rc, msg in ex.map(compile_one, names):
            assert rc == 0, msg
    lib = os.path.join(out, "libkda_san.so")
    rc, msg = _run([HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC",
                    *[os.path.join(out, n + ".o") for n in names], "-o", lib])
    assert rc == 0, msg
    rc, msg = _run([sys.executable, "-m", "pytest", "-q", "-x", "-m", "not gpu", "-p", "no:cacheprovider",
                    os.path.join(ROOT, "tests", "test_hybrid_abi_cpu.py")],
                   env=_env(_clang_asan_runtime(), KDA_LIB=lib))
    assert rc == 0 and "passed" in msg, msg[:3000]
    assert "ERROR: AddressSanitizer" not in msg and "runtime error" not in msg, msg[:3000]
