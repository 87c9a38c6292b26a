"""The block-scaled product's kernels stage codes HBM -> LDS with loads that
write LDS directly, which the compiler does not order later LDS reads after.
This compiles product.hip for gfx950 to assembly (no GPU needed) and checks in
program order that the kernels whose waves read only what they loaded
themselves wait for all of it (s_waitcnt vmcnt(0)) before any read, and that
those that hand buffers over between waves wait and pass a barrier."""

import os
import re
import subprocess

import pytest

from moe_decode_layer_sigmoid_amd import build as lib_build


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    try:
        hipcc = lib_build.hipcc()
    except RuntimeError as e:
        pytest.skip(str(e))
    out = tmp_path_factory.mktemp("asm") / "product.s"
    cmd = [hipcc, *(f for f in lib_build.FLAGS if f != "-fPIC"), "-I", os.path.join(lib_build.ROOT, "include"),
           "-I", lib_build.CSRC, "--cuda-device-only", "-S",
           os.path.join(lib_build.CSRC, "ops", "product.hip"), "-o", str(out)]
    res = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    assert res.returncode == 0, res.stdout[-2000:]
    asm, got = out.read_text(), {}
    for name in re.findall(r"^(_Z\S*product_\w*kernel\S*):", asm, re.M):
        at = asm.index("\n" + name + ":")
        got[name] = [x.strip() for x in asm[at:asm.index(".Lfunc_end", at)].splitlines()]
    return got


def test_waves_wait_for_their_own_loads(kernels):
    checked = 0
    for name, body in kernels.items():
        if "rows_kernel" not in name and "deal_kernel" not in name:
            continue
        pending = seen = False
        for line in body:
            if line.startswith("global_load_lds"):
                pending = seen = True
            elif line.startswith("s_waitcnt") and "vmcnt(0)" in line:
                pending = False
            elif line.startswith("ds_read"):
                assert not pending, "%s: %s before its loads are waited for" % (name, line)
        checked += seen
    assert checked == 6  # four of rows, two that deal


def test_buffers_are_handed_over_behind_a_wait_and_a_barrier(kernels):
    """From a staging load to a barrier there is a wait on the loads."""
    checked = 0
    for name, body in kernels.items():
        if "14product_kernel" not in name:
            continue
        loads = waited = 0
        for line in body:
            if line.startswith("global_load_lds"):
                loads, waited = loads + 1, False
            elif line.startswith("s_waitcnt") and "vmcnt" in line:
                waited = True
            elif line.startswith("s_barrier"):
                assert loads == 0 or waited, name
        checked += loads > 0
    assert checked >= 20
