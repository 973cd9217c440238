"""The C-ABI tests again, against a copy of libmxq whose host validation layer
(api.hip) is built with AddressSanitizer, in a child process with the sanitizer
runtime preloaded. Any out-of-bounds or use-after-free access in argument
checking, workspace sizing or launch set-up aborts the child and fails here."""

import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_abi_under_host_address_sanitizer():
    from microscaling_precision_quantization_amd import build as b
    rt = b.asan_runtime()
    if rt is None or shutil.which(b.HIPCC) is None and not os.path.exists(b.HIPCC):
        pytest.skip("no hipcc / clang AddressSanitizer runtime")
    lib = b.build_asan()
    env = dict(os.environ, MXQ_LIBRARY=lib, LD_PRELOAD=rt, ASAN_OPTIONS="detect_leaks=0:abort_on_error=1")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-p", "no:cacheprovider", "-m", "not gpu",
                        os.path.join(ROOT, "tests", "test_abi.py")], cwd=ROOT, env=env, capture_output=True,
                       text=True, timeout=600)
    assert r.returncode == 0, (r.stdout[-3000:] + r.stderr[-3000:])
    assert "AddressSanitizer" not in r.stderr
    assert " passed" in r.stdout


def test_abi_of_the_norms_and_the_router_under_host_address_sanitizer():
    from microscaling_precision_quantization_amd import build as b
    rt = b.asan_runtime()
    if rt is None or shutil.which(b.HIPCC) is None and not os.path.exists(b.HIPCC):
        pytest.skip("no hipcc / clang AddressSanitizer runtime")
    env = dict(os.environ, MXQ_LIBRARY=b.build_asan(), LD_PRELOAD=rt, ASAN_OPTIONS="detect_leaks=0:abort_on_error=1")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-p", "no:cacheprovider", "-m", "not gpu",
                        os.path.join(ROOT, "tests", "test_abi_block.py")], cwd=ROOT, env=env, capture_output=True,
                       text=True, timeout=600)
    assert r.returncode == 0, (r.stdout[-3000:] + r.stderr[-3000:])
    assert "AddressSanitizer" not in r.stderr
    assert " passed" in r.stdout
