"""The wrappers of the operators whose weights depend on the row: matrices whose rows
overlap (expanded ones, overlapping windows) are refused, by the short way and the
long one.  Without a GPU the wrappers get tensors that only say that they are on one."""
import pytest


def overlapping(torch, rows, cols, **o):
    """A bias for every row, and windows eight values apart."""
    yield torch.zeros(cols, **o).expand(rows, cols)
    yield torch.zeros(8 * rows + cols, **o).as_strided((rows, cols), (8, 1))


def calls(torch, W, wrap, **o):
    """name of the matrix -> a call with it"""
    T, k, E, S, H, L, r = 6, 2, 16, 12, 64, 2, 8
    half, int32 = dict(o, dtype=torch.float16), dict(o, dtype=torch.int32)
    z, base, weights = wrap(torch.zeros(S, H, **half)), wrap(torch.zeros(T, H, **half)), wrap(torch.zeros(T, k, **o))
    slots, offsets, rows = (wrap(torch.zeros(*s, **int32)) for s in ((T, k), (L + 1,), (T,)))
    x, a, b = (wrap(torch.zeros(*s, **half)) for s in ((T, H), (L, r, H), (L, H, r)))
    return [
        ("logits", (T, E), o, lambda t: W.wqbmm_moe_route(t, k)),
        ("z", (S, H), half, lambda t: W.wqbmm_moe_combine(t, slots, weights)),
        ("base", (T, H), half, lambda t: W.wqbmm_moe_combine(z, slots, weights, base=t)),
        ("y", (T, H), half, lambda t: W.wqbmm_moe_combine(z, slots, weights, y=t)),
        ("base", (T, H), half, lambda t: W.wqbmm_moe_combine(z, slots, weights, base=t, y=t)),
        ("x", (T, H), half, lambda t: W.wqbmm_lora_matmul(t, a, b, offsets, rows)),
        ("base", (T, H), half, lambda t: W.wqbmm_lora_matmul(x, a, b, offsets, rows, base=t)),
        ("y", (T, H), half, lambda t: W.wqbmm_lora_matmul(x, a, b, offsets, rows, base=base, y=t)),
        ("base", (T, H), half, lambda t: W.wqbmm_lora_matmul(x, a, b, offsets, rows, base=t, y=t)),
    ]


def refused(torch, W, wrap, **o):
    for name, shape, options, call in calls(torch, W, wrap, **o):
        for t in overlapping(torch, *shape, **options):
            with pytest.raises((ValueError, W.WqbmmError)) as e:
                call(wrap(t))
                raise AssertionError(f"{name} with strides {t.stride()} was let through")
            if isinstance(e.value, W.WqbmmError):
                assert e.value.status == W.WQBMM_ERR_INVALID, (name, t.stride())
            else:
                assert f"the rows of {name} must not overlap" in str(e.value)


def test_overlapping_rows_are_refused_without_a_gpu(monkeypatch):
    torch = pytest.importorskip("torch")
    import weight_only_quantized_msd_amd as W
    from weight_only_quantized_msd_amd import _mxfp4 as M
    M._load()

    class OnADevice(torch.Tensor):
        is_cuda = True

    # the library refuses the call's arguments before it looks for a device
    monkeypatch.setattr(M, "_on", lambda device, stream, work: work(0))
    refused(torch, W, lambda t: t.as_subclass(OnADevice))


@pytest.mark.gpu
def test_overlapping_rows_are_refused():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import weight_only_quantized_msd_amd as W
    refused(torch, W, lambda t: t, device="cuda")
    # one row overlaps with none
    slots, weights = torch.tensor([[0]], dtype=torch.int32, device="cuda"), torch.ones(1, 1, device="cuda")
    bias = torch.ones(64, dtype=torch.float16, device="cuda")
    assert (W.wqbmm_moe_combine(bias.expand(1, 64), slots, weights, base=bias.expand(1, 64)) == 2).all()
