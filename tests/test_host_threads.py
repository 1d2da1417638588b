"""Calls of several host threads, without a GPU: the library as it is built, on a
stand-in for the HIP runtime (hip_stub.cpp) that notes every launch.  A call passes
operands from one launch to the next in its stream's workspace, so no other call may
launch on that workspace in between.  The calls run in a child process."""
import ctypes
import os
import subprocess
import sys
import threading

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
PER_THREAD = 2                                          # hipStreamPerThread
A = 0x10000                                             # an aligned address that nothing reads


def calls(L):
    """name -> (call on a stream, of several launches)"""
    lib = L.lib()
    return {
        "mxfp4": lambda s: lib.wqbmm_mxfp4_matmul(A, 0, 2080, A, 300, 2080, 72, A, 1, s),
        "16bit": lambda s: lib.wqbmm_mxfp4_matmul(A, 0, 2080, A, 100, 2080, 72, A, 0, s),
        "moe": lambda s: lib.wqbmm_mxfp4_moe(A, 0, 512, 40, 512, 96, 6, 2, 1, A, A, A, A, A, A, s),
        "moe_one": lambda s: lib.wqbmm_mxfp4_moe(A, 0, 512, 1, 512, 96, 6, 2, 1, A, A, A, A, A, A, s),
        "msd_decode": lambda s: lib.wqbmm_a16w4_msd(A, A, A, 128, 16, 512, 256, A, s),
        "msd_prefill": lambda s: lib.wqbmm_a16w4_msd(A, A, A, 128, 256, 512, 256, A, s),
    }


def child():
    sys.path.insert(0, os.path.dirname(HERE))
    from weight_only_quantized_msd_amd import _lib as L
    stub = ctypes.CDLL(os.environ["HIP_STUB"])
    stub.stub_stream_of.restype = ctypes.c_size_t
    all_calls = calls(L)

    def run(names, streams, repeat=12):
        """Each thread makes its call `repeat` times on its stream, all at once."""
        stub.stub_reset()
        start, wrong = threading.Barrier(len(names)), []

        def work(i):
            stub.stub_thread(i)
            start.wait()
            for _ in range(repeat):
                status = all_calls[names[i]](streams[i])
                if status != 0:
                    wrong.append((names[i], status))

        threads = [threading.Thread(target=work, args=(i,)) for i in range(len(names))]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        assert not wrong, wrong[0]
        return [(stub.stub_thread_of(i), stub.stub_stream_of(i)) for i in range(stub.stub_launches())]

    per_call = {}
    for name in all_calls:
        run([name], [0x50], 1)                          # the workspace grows here
        per_call[name] = len(run([name], [0x50], 1))
        assert per_call[name] >= 2, (name, per_call[name])
    for names in (["mxfp4", "mxfp4"], ["moe", "moe_one"], ["16bit", "moe"], ["msd_prefill", "mxfp4"],
                  ["msd_decode", "msd_prefill", "moe"]):
        log = run(names, [0x50] * len(names))
        at = 0
        while at < len(log):                            # whole calls, one after another
            who = log[at][0]
            n = per_call[names[who]]
            assert [t for t, _ in log[at:at + n]] == [who] * n, (names, at, log[at:at + n])
            at += n
    # other streams have workspaces of their own and do not wait for each other
    log = run(["mxfp4", "mxfp4"], [0x60, 0x70])
    assert stub.stub_allocations() == 2
    assert any(a != b for (a, _), (b, _) in zip(log, log[1:len(log) // 2]))
    # one handle, another stream in each thread
    run(["moe", "moe"], [PER_THREAD, PER_THREAD])
    assert stub.stub_allocations() >= 2, "two threads' own streams share a workspace"
    print("threads ok")


def test_calls_of_several_threads(tmp_path):
    from weight_only_quantized_msd_amd import build as B
    if not os.path.exists(B.LIB_PATH):
        pytest.skip("the library is not built")
    include = os.path.join(os.path.dirname(os.path.dirname(B.HIPCC)), "include")
    stub = str(tmp_path / "hip_stub.so")
    r = subprocess.run(["g++", "-O1", "-std=c++17", "-fPIC", "-shared", "-D__HIP_PLATFORM_AMD__", "-isystem", include,
                        os.path.join(HERE, "hip_stub.cpp"), "-o", stub, "-lpthread"], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    first = ":".join(filter(None, [stub, os.environ.get("LD_PRELOAD")]))
    r = subprocess.run([sys.executable, os.path.abspath(__file__)],
                       env=dict(os.environ, LD_PRELOAD=first, HIP_STUB=stub), capture_output=True, text=True, timeout=100)
    assert r.returncode == 0 and "threads ok" in r.stdout, r.stdout + r.stderr


if __name__ == "__main__":
    child()
