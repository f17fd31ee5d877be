"""The LDS address register (M0) of the tiled MXFP4 kernels' direct loads, in the code the compiler
makes of them: several loads share what one instruction set it to."""
import os
import re
import subprocess

import pytest

import __graft_entry__ as entry

CSRC = os.path.join(entry.PKG, "csrc")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

# Code that holds a value of its own in M0 across a load.
SNIPPET = """
#include "mx_tile.h"
using namespace nvfp4;
extern "C" __global__ void own_m0(const char* p, int at, int bytes) {
    uint32_t own;
    asm volatile("s_movk_i32 %0, 0x77" : "={m0}"(own));
    set_m0(at);
    dma16_at<0>(make_rsrc(p, bytes), threadIdx.x * 16, 0);
    asm volatile("s_setprio 0 ; %0" ::"{m0}"(own));
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}
"""


def device_code(path):
    got = subprocess.run([HIPCC, *entry.HIPCC_FLAGS, "-I", os.path.join(entry.ROOT, "include"), "-I", CSRC, "-S",
                          "--cuda-device-only", str(path), "-o", "-"], capture_output=True, text=True, check=True).stdout
    lines = (re.sub(r"\s*;.*", "", line).strip() for line in got.splitlines())
    return [line for line in lines if line and not line.startswith(".")]


def test_set_m0_says_that_it_changes_m0(tmp_path):
    (tmp_path / "snippet.hip").write_text(SNIPPET)
    code = device_code(tmp_path / "snippet.hip")
    load = next(i for i, line in enumerate(code) if line.startswith("buffer_load") and line.endswith("lds"))
    use = next(i for i, line in enumerate(code) if line.startswith("s_setprio"))
    assert load < use and any(line.startswith("s_mov_b32 m0,") for line in code[load:use])      # put back


@pytest.mark.parametrize("source", ["mx_tile128.hip", "mx_tile256.hip"])
def test_nothing_else_writes_m0(source):
    """set_m0 and dma16 write it with a wait state behind; any other write would be the compiler's."""
    code = device_code(os.path.join(CSRC, source))
    writes = [i for i, line in enumerate(code) if re.match(r"\S+ m0,", line)]
    assert len(writes) > 20
    assert all(code[i].startswith("s_mov_b32") and code[i + 1] == "s_nop 0" for i in writes)
    assert not [line for line in code if re.search(r",.*\bm0\b", line)]     # nor does anything read it
