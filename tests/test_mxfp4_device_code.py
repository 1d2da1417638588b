"""What the compiler makes of the MXFP4 kernels (no GPU), read from its intermediate
code and its assembly of their sources: properties that no output shows."""
import functools
import os
import re
import subprocess

import pytest

from weight_only_quantized_msd_amd import build as B


@functools.lru_cache(maxsize=None)
def kernels(source):
    """name -> lines of intermediate code, for each kernel of a source, with the library's own flags."""
    found, lines = {}, None
    for line in compiled(source, "-emit-llvm").splitlines():
        m = re.match(r"define .*amdgpu_kernel void @(\w+)\(", line)
        if m:
            lines = found.setdefault(m.group(1), [])
        elif line == "}":
            lines = None
        elif lines is not None:
            lines.append(line)
    return found


def compiled(source, *more):
    if not os.path.exists(B.HIPCC):
        pytest.skip("no hipcc")
    r = subprocess.run([B.HIPCC] + B._flags(source) + ["-S", "--offload-device-only", *more, "-o", "-",
                                                       os.path.join(B.CSRC, source)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return r.stdout


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


# The tiled products wait by counting the loads in flight.  A load whose value has no
# use is taken out, and a wait that counts it would then be too short.
# P: a wave's copies of a stage; S: its scale loads of a K-tile or quad.

def gemm4_loads(TM, TN, WVM, WVN):
    waves, S = WVM * WVN, TM + TN
    P = TM * WVM // waves + -(-TN * WVN // waves)
    # three stages ahead, four phases of the loop, three of a last quad; scales ahead and in the loop's first phase
    return 10 * P, 2 * S


def gemm16_loads(TM, TN):
    P = TM + TN
    # three stages ahead, three K-tiles of the loop, three after it; scales of two K-tiles ahead, in the loop's three
    # K-tiles and in the first after it
    return 9 * P, 6 * TN


@pytest.mark.parametrize("source,kernel,loads", [("mx_gemm4.hip", "mx_gemm4_kernel", gemm4_loads),
                                                 ("mx_gemm16.hip", "mx_gemm16_kernel", gemm16_loads)])
def test_every_load_that_a_wait_counts_is_there(source, kernel, loads):
    found, name = {}, None
    for line in compiled(source).splitlines():
        m = re.match(r"(_Z\w+):", line)
        if m:
            name = m.group(1)
        elif name and kernel in name and "buffer_load_dword" in line:
            at = found.setdefault(name, [0, 0])
            at[0 if re.search(r"\blds\b", line) else 1] += 1
    assert len(found) >= 6
    for name, got in found.items():
        dtype, *tile = map(int, re.findall(r"Li(\d+)E", name))
        paths = 2 if kernel == "mx_gemm16_kernel" and dtype == 0 else 1       # fp16: weights exact in fp16, or not
        assert got == [paths * n for n in loads(*tile)], name
