"""Host threads that call on one stream at the same time get what each of them
gets alone (the calls with `stream` given release the interpreter's lock)."""
import threading

import numpy as np
import pytest

from test_gpu_mxfp4 import random_weights, tiled

pytestmark = pytest.mark.gpu


def test_threads_on_one_stream():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import weight_only_quantized_msd_amd as W
    rng = np.random.default_rng(5)
    H, inter, E, k, N = 544, 96, 6, 2, 72
    w, gate_up, down = (tiled(torch, *random_weights(rng, s)) for s in ((N, H), (E, 2 * inter, H), (E, H, inter)))
    router = torch.randn(E, H, device="cuda").bfloat16()
    stream = torch.cuda.Stream()

    def call(i, x):
        if i % 2:
            return W.wqbmm_mxfp4_matmul(x, w, N, activations="mxfp4" if i % 4 == 1 else "16bit", stream=stream)
        return W.wqbmm_mxfp4_moe(x, router, gate_up, down, inter, k, stream=stream)[0]

    rows = [40, 300, 1, 130]
    xs = [torch.randn(m, H, device="cuda").bfloat16() for m in rows]
    torch.cuda.synchronize()
    want = [call(i, x) for i, x in enumerate(xs)]       # the workspace grows here
    stream.synchronize()
    got, start = [[] for _ in xs], threading.Barrier(len(xs))

    def work(i):
        start.wait()
        for _ in range(100):
            got[i].append(call(i, xs[i]))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(xs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    stream.synchronize()
    for i, outs in enumerate(got):
        assert len(outs) == 100 and all(torch.equal(y, want[i]) for y in outs), rows[i]
