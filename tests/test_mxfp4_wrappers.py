"""The MXFP4 wrappers' own ways, without a GPU."""
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_a_stream_of_another_device_is_refused():
    torch = pytest.importorskip("torch")
    from weight_only_quantized_msd_amd import _mxfp4 as M
    M._load()

    class Stream:                                       # as torch.cuda.Stream
        device, cuda_stream = torch.device("cuda", 1), 0

    def work(raw):
        raise AssertionError("launched on another device than the tensors'")

    with pytest.raises(ValueError, match="stream is on cuda:1"):
        M._on(torch.device("cuda", 0), Stream(), work)


def test_another_build_of_the_library_is_the_only_one(tmp_path):
    """WQBMM_LIB selects it: the package's own must not be loaded beside it for the short calls."""
    pytest.importorskip("torch")
    from weight_only_quantized_msd_amd import build as B
    if not os.path.exists(B.LIB_PATH):
        pytest.skip("the library is not built")
    other = str(tmp_path / "libother.so")
    shutil.copy(B.LIB_PATH, other)
    r = subprocess.run([sys.executable, "-c",
                        "from weight_only_quantized_msd_amd import _mxfp4 as M; M._load(); "
                        "print({l.split()[-1] for l in open('/proc/self/maps') if l.rstrip().endswith('.so')})"],
                       cwd=ROOT, env=dict(os.environ, WQBMM_LIB=other), capture_output=True, text=True)
    assert r.returncode == 0 and other in r.stdout and "libwqbmm.so" not in r.stdout, r.stdout + r.stderr
