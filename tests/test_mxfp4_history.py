"""The MXFP4 calls have no gradients: what they return for inputs that require one
must not look as if it had none to give."""
import numpy as np
import pytest


def test_history_ends_in_an_error():
    torch = pytest.importorskip("torch")
    from weight_only_quantized_msd_amd import _mxfp4 as M
    M._load()
    x = torch.ones(2, 3, requires_grad=True)
    out, ids = M._with_history("a call", (torch.zeros(2, 3), torch.zeros(2, dtype=torch.int32)), x)
    assert out.requires_grad and not ids.requires_grad
    with pytest.raises(RuntimeError, match="a call has no gradient"):
        (out * 2).sum().backward()
    assert x.grad is None
    with pytest.raises(RuntimeError, match="y given"):
        M._refuse_given_output(torch.zeros(1), "a call", x)
    y = torch.zeros(2, 3)
    with torch.no_grad():
        assert M._with_history("a call", (y,), x)[0] is y
        M._refuse_given_output(y, "a call", x)
    assert M._with_history("a call", (y,), x.detach())[0] is y
    M._refuse_given_output(None, "a call", x)


@pytest.mark.gpu
@pytest.mark.parametrize("on_a_stream", [False, True])
def test_calls_with_inputs_that_require_a_gradient(on_a_stream):
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import weight_only_quantized_msd_amd as W
    from test_gpu_mxfp4 import random_weights, tiled
    rng = np.random.default_rng(0)
    T, H, inter, E, k, N = 3, 64, 32, 4, 2, 48
    o = {"stream": torch.cuda.current_stream()} if on_a_stream else {}
    w, gate_up, down = (tiled(torch, *random_weights(rng, s)) for s in ((N, H), (E, 2 * inter, H), (E, H, inter)))
    x, router = torch.randn(T, H, device="cuda").bfloat16(), torch.randn(E, H, device="cuda").bfloat16()
    want, layer = W.wqbmm_mxfp4_matmul(x, w, N), W.wqbmm_mxfp4_moe(x, router, gate_up, down, inter, k)
    assert not want.requires_grad and not any(t.requires_grad for t in layer)
    for act in ("16bit", "mxfp4"):
        xg = x.clone().requires_grad_()
        y = W.wqbmm_mxfp4_matmul(xg, w, N, activations=act, **o)
        assert y.requires_grad and (act != "16bit" or torch.equal(y.detach(), want))
        with pytest.raises(RuntimeError, match="no gradient"):
            y.sum().backward()
        with torch.no_grad():
            assert not W.wqbmm_mxfp4_matmul(xg, w, N, activations=act, **o).requires_grad
        with pytest.raises(RuntimeError, match="y given"):
            W.wqbmm_mxfp4_matmul(xg, w, N, activations=act, y=torch.empty_like(want), **o)
    for which in (0, 1):
        inputs = [x.clone(), router.clone()]
        inputs[which].requires_grad_()
        got = W.wqbmm_mxfp4_moe(*inputs, gate_up, down, inter, k, **o)
        assert all(torch.equal(a.detach(), b) for a, b in zip(got, layer))
        assert got[0].requires_grad and not got[1].requires_grad and got[2].requires_grad
        for out in (got[0], got[2]):
            with pytest.raises(RuntimeError, match="no gradient"):
                out.sum().backward(retain_graph=True)
        with pytest.raises(RuntimeError, match="y given"):
            W.wqbmm_mxfp4_moe(*inputs, gate_up, down, inter, k, y=torch.empty_like(x), **o)
