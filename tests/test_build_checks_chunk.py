"""The build's register check for the 8-bit cache's chunk kernel, whose warpgroups re-split their registers too (CPU only).

With any other count than kLaunchRegs every call of it would be refused at run time, so the build has to fail.
"""
import os
import subprocess

import pytest

from exact_tiled_attention_47_b200 import build
from test_build_checks import report

SRC = "constexpr int kLaunchRegs = 128;\n"
NAME = "_ZN2fa16kv8_chunk_kernelILb0ELb0ELi64EEEvNS_9AttParamsEi"


def test_the_planned_count_passes_with_spills():
    build.check_planned_registers("fa_kv8_chunk.cu", SRC, report(128, 12, NAME) + report(60, name="kv8_combine_kernel"))


@pytest.mark.parametrize("rep", [report(127, name=NAME), report(128, name=NAME) + report(136, name=NAME + "2"), report(128, name="other"), ""])
def test_other_counts_or_nothing_fail(rep):
    with pytest.raises(RuntimeError):
        build.check_planned_registers("fa_kv8_chunk.cu", SRC, rep)


@pytest.mark.parametrize("extra", [[], ["-DFA_DEBUG"]])
def test_real_chunk_object_passes_the_check(extra):
    src = os.path.join(build.CSRC, "fa_kv8_chunk.cu")
    r = subprocess.run([build.nvcc()] + build.ARCH + build.CFLAGS + extra + ["-Xptxas", "-v", "-c", src, "-o", os.devnull],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    with open(src) as fh:
        build.check_planned_registers("fa_kv8_chunk.cu", fh.read(), r.stdout + r.stderr)


def test_every_kernel_that_re_splits_registers_is_planned():
    for name in os.listdir(build.CSRC):
        with open(os.path.join(build.CSRC, name)) as fh:
            if name.endswith(".cu") and "regs_increase<" in fh.read():
                assert name in build.REGISTER_PLANNED, name
