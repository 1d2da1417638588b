"""Which kernels a call of the C ABI launches, and how large, found without a GPU: a
child process makes the calls on a stand-in for the HIP runtime (launch_stub.cpp)."""
import ctypes
import json
import os
import subprocess
import sys

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
A = 0x10000                                             # an aligned address that nothing reads


def launched(tmp_path, calls):
    """(all kernels' names, per call (status, [(kernel, workgroups, threads of one)])) of [(function, arguments)]."""
    from weight_only_quantized_msd_amd import build as B
    if not os.path.exists(B.LIB_PATH):
        pytest.skip("the library is not built")
    include = os.path.join(os.path.dirname(os.path.dirname(B.HIPCC)), "include")
    stub = str(tmp_path / "launch_stub.so")
    r = subprocess.run(["g++", "-O1", "-std=c++17", "-fPIC", "-shared", "-D__HIP_PLATFORM_AMD__", "-isystem", include,
                        os.path.join(HERE, "launch_stub.cpp"), "-o", stub], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    first = ":".join(filter(None, [stub, os.environ.get("LD_PRELOAD")]))
    r = subprocess.run([sys.executable, os.path.abspath(__file__)], input=json.dumps(calls),
                       env=dict(os.environ, LD_PRELOAD=first, HIP_STUB=stub), capture_output=True, text=True, timeout=100)
    assert r.returncode == 0, r.stdout + r.stderr
    kernels, each = json.loads(r.stdout)
    names = subprocess.run(["c++filt"], input="\n".join(kernels), capture_output=True, text=True, check=True)
    plain = dict(zip(kernels, (n.split("(")[0].replace("void ", "").replace("wqbmm::", "") for n in names.stdout.split("\n"))))
    return set(plain.values()), [(status, [(plain[k], g, b) for k, g, b in some]) for status, some in each]


def child():
    sys.path.insert(0, os.path.dirname(HERE))
    from weight_only_quantized_msd_amd import _lib as L
    lib, stub = L.lib(), ctypes.CDLL(os.environ["HIP_STUB"])
    stub.stub_kernel.restype = stub.stub_launched.restype = ctypes.c_char_p
    stub.stub_grid.restype = stub.stub_block.restype = ctypes.c_uint32
    each = []
    for name, args in json.loads(sys.stdin.read()):
        stub.stub_reset()
        status = getattr(lib, name)(*args)
        each.append((status, [(stub.stub_launched(i).decode(), stub.stub_grid(i), stub.stub_block(i))
                              for i in range(stub.stub_launches())]))
    print(json.dumps(([stub.stub_kernel(i).decode() for i in range(stub.stub_kernels())], each)))


def route(T, E, k=1, dtype=1):
    return "wqbmm_moe_route", [A, dtype, E, T, E, k, 1, A, A, None]


def group(T, k, G):
    return "wqbmm_group_rows", [A, T, k, G, A, A, A, None]


def grouped(S, G, K, N, dtype=1, act=0, gated=0, R=None, ld=None):
    """R: x's rows, if the places have rows of their own."""
    return "wqbmm_mxfp4_grouped_matmul", [A, dtype, ld or K, S if R is None else R, None if R is None else A, A, G, S, K, N,
                                          A, A, act, gated, None]


def combine(T, k, H, dtype=1):
    return "wqbmm_moe_combine", [A, dtype, H, T, H, A, A, T, k, None, 0, A, H, None]


def lora(M, L, r, K, N, dtype=1):
    return "wqbmm_lora_matmul", [A, dtype, K, M, K, N, r, L, A, A, None, A, A, None, 0, A, N, None]


if __name__ == "__main__":
    child()
