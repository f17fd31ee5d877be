"""The tiled MXFP4 kernels hold all of a lane's values in registers: what the compiler put into scratch memory would be
waited for together with the direct loads and the stores that are meant to be in flight."""
import os
import re
import subprocess

import pytest

import __graft_entry__ as entry

CSRC = os.path.join(entry.PKG, "csrc")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")


@pytest.mark.parametrize("source", ["mx_tile128.hip", "mx_tile256.hip", "mx_ffn_forward128.hip", "mx_ffn_forward256.hip",
                                    "mx_ffn_backward128.hip"])
def test_no_scratch(source):
    got = subprocess.run([HIPCC, *entry.HIPCC_FLAGS, "-I", os.path.join(entry.ROOT, "include"), "-S", "--cuda-device-only",
                          os.path.join(CSRC, source), "-o", "-"], capture_output=True, text=True, check=True).stdout
    used = re.findall(r"\.private_segment_fixed_size:\s*(\d+)", got)
    names = re.findall(r"^\s*\.amdhsa_kernel (\S+)", got, flags=re.M)
    assert len(used) == len(names) >= 4
    assert set(used) == {"0"}, dict(zip(names, used))
