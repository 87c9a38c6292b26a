"""The host code of the operators beside the MoE layer under AddressSanitizer
and UndefinedBehaviorSanitizer (ops_driver.c), as test_host_sanitizers does for
the layer's.  No device is touched."""

import os
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest

from moe_decode_layer_sigmoid_amd import build as lib_build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HERE = os.path.join(ROOT, "tests", "sanitize")
SAN_ENV = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=0",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")


def _run(cmd, **kw):
    res = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True, **kw)
    return res.returncode, res.stdout


def test_ops_host_checks_under_asan_ubsan(tmp_path):
    try:
        hipcc = lib_build.hipcc()
    except RuntimeError as e:
        pytest.skip(str(e))
    flags = lib_build.FLAGS  # -O3: the kernels' asm operands are constants only when inlined
    san = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
           "-Xarch_host", "-fno-sanitize-recover=all", "-Xarch_host", "-fno-omit-frame-pointer"]
    inc = ["-I", os.path.join(ROOT, "include"), "-I", lib_build.CSRC]
    jobs = [[hipcc, *flags, *san, *inc, "-c", os.path.join(lib_build.CSRC, "ops", src), "-o",
             str(tmp_path / src.replace(".hip", ".o"))] for src in lib_build.OPS_SOURCES]
    jobs.append([hipcc, *san, *inc, "-x", "c", "-c", os.path.join(HERE, "ops_driver.c"), "-o",
                 str(tmp_path / "driver.o")])
    with ThreadPoolExecutor(max(1, min(len(jobs), os.cpu_count() or 1))) as ex:
        results = list(ex.map(_run, jobs))
    for cmd, (rc, out) in zip(jobs, results):
        assert rc == 0, " ".join(cmd) + "\n" + out
    exe = str(tmp_path / "ops_san")
    rc, out = _run([hipcc, "--offload-arch=" + lib_build.ARCH, *san, *[j[-1] for j in jobs], "-o", exe])
    assert rc == 0, out
    rc, out = _run([exe], env=SAN_ENV, timeout=300)
    assert rc == 0 and "ops checks: ok" in out, out
