"""The recurrence's kernels hold a block of a batch in registers: the compiler's own report of
their resources, for the flags that the library is built with, names none that spills."""
import os
import re
import subprocess

import pytest

from gated_delta_rule_46_amd import build


def test_no_kernel_spills():
    if not os.path.exists(build.HIPCC):
        pytest.skip("no compiler")
    src = os.path.join(build.CSRC, "kda_glr.hip")
    r = subprocess.run([build.HIPCC, *build.FLAGS, *build.EXTRA.get("kda_glr.hip", []), "--offload-device-only", "-c", src,
                        "-o", os.devnull, "-Rpass-analysis=kernel-resource-usage"], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    names = re.findall(r"Function Name: (\S+)", r.stderr)
    scratch = [int(n) for n in re.findall(r"ScratchSize \[bytes/lane\]: (\d+)", r.stderr)]
    assert len(names) == len(scratch) > 20
    assert not [n for n, s in zip(names, scratch) if s]
