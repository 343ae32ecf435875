"""Further host-side refusals and the plans' handling of streams and devices; these run without a GPU."""
import ctypes

import pytest
import torch

import semi_autoregressive_drafting_gb300 as ds

P = ctypes.c_void_p(256)
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    from semi_autoregressive_drafting_gb300 import _build, _lib
    _build.build()
    return _lib.load()


@pytest.mark.parametrize("T,ok", [(3.5e-39, False), (2.95e-39, False), (4.2e-39, False), (4.3e-39, True),
                                  (1e-38, True), (3e38, True)])
def test_temperature_whose_scale_overflows(lib, T, ok):
    # log2(e) / T is infinite from about 4.24e-39 down, 1 / T only from 2.94e-39
    want = 0 if ok else 1
    assert lib.dspark_token_logprobs(0, 100, T, 0, P, 100, P, 2, P, P, P, P, P, P, P, BIG, None) == want
    assert lib.dspark_token_logprobs_grad(0, 100, T, 0, P, 100, P, P, P, P, P, P, 100, None) == want
