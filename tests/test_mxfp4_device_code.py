"""What the compiler is told about the MXFP4 kernels, read from the intermediate
code it makes of their sources (no GPU): properties that no output shows."""
import functools
import os
import re
import subprocess

import pytest

from weight_only_quantized_msd_amd import build as B


@functools.lru_cache(maxsize=None)
def kernels(source):
    """name -> lines of intermediate code, for each kernel of a source, with the library's own flags."""
    if not os.path.exists(B.HIPCC):
        pytest.skip("no hipcc")
    r = subprocess.run([B.HIPCC] + B._flags(source) + ["-S", "-emit-llvm", "--offload-device-only", "-o", "-",
                                                       os.path.join(B.CSRC, source)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    found, lines = {}, None
    for line in r.stdout.splitlines():
        m = re.match(r"define .*amdgpu_kernel void @(\w+)\(", line)
        if m:
            lines = found.setdefault(m.group(1), [])
        elif line == "}":
            lines = None
        elif lines is not None:
            lines.append(line)
    return found


@pytest.mark.parametrize("kernel", ["mx_moe_up_kernel", "mx_moe_down_kernel"])
def test_lists_of_pairs_are_fenced_before_other_lanes_read_them(kernel):
    """Lanes write entries of the wave's list in LDS (16 bits each) that other lanes read."""
    seen = 0
    for name, lines in kernels("mx_moe.hip").items():
        if kernel not in name:
            continue
        writes = [i for i, s in enumerate(lines) if re.search(r"store i16 .*addrspace\(3\)", s)]
        reads = [i for i, s in enumerate(lines) if re.search(r"load i16, ptr addrspace\(3\)", s)]
        assert writes and reads and max(writes) < min(reads)
        assert any("fence syncscope(\"wavefront\")" in s for s in lines[max(writes):min(reads)]), name
        seen += 1
    assert seen >= 2
