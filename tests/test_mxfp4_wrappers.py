"""The MXFP4 wrappers' own ways, without a GPU."""

import pytest


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
