"""The refusals of the MXFP4 C ABI with the library's host code (msd_api.cpp,
mx_api.cpp) under AddressSanitizer and UndefinedBehaviorSanitizer, as
test_sanitized.py does for the int4 operator: their extents go up to 2^63 - 1."""
import glob
import os

import pytest

from test_sanitized import _run


def test_mxfp4_validation_under_asan_ubsan():
    rts = glob.glob("/opt/rocm/lib/llvm/lib/clang/*/lib/linux/libclang_rt.asan-x86_64.so")
    if not rts:
        pytest.skip("clang's ASan runtime is not installed")
    from weight_only_quantized_msd_amd.build import build_host_sanitized
    lib = build_host_sanitized()
    first = ":".join(filter(None, [rts[0], os.environ.get("LD_PRELOAD")]))
    out = _run({"LD_PRELOAD": first, "WQBMM_LIB": lib}, ["tests/test_mxfp4.py", "-k", "c_abi or tiled_weight_bytes"])
    assert "failed" not in out and "skipped" not in out
