"""Limits of the calls over vocabulary rows and cache blocks that their
refusals state (no GPU needed)."""

import ctypes

import pytest

from test_vocab_reference import _status, lib  # noqa: F401

D, E = ctypes.c_void_p(16), ctypes.c_void_p(32)
LOGPROBS = dict(logits=D, dtype=0, R=2, V=64, stride=64, tokens=D, T=1.0, K=4, logprob=D, rank=D, entropy=D, ids=D,
                lps=D, err=D, stream=None)
DISTILL = dict(student=D, dtype=0, R=2, V=64, stride=64, ids=D, lp=D, K=4, w=None, T=1.0, tail=1, loss=D, stats=None,
               grad=E, grad_stride=64, err=None, stream=None)
BACKWARD = dict(student=D, dtype=0, R=2, V=64, stride=64, ids=D, lp=D, K=4, stats=D, gl=None, T=1.0, grad=E,
                grad_stride=64, stream=None)


@pytest.mark.parametrize("T", [2.0 ** -149, 1e-39, 4.2e-39, 2.0 ** -126 - 2.0 ** -149])
@pytest.mark.parametrize("name,good", [("spec_token_logprobs", LOGPROBS), ("spec_distill_topk", DISTILL),
                                       ("spec_distill_topk_backward", BACKWARD)])
def test_temperatures_whose_reciprocal_has_no_32_bits(lib, name, good, T):  # noqa: F811
    assert _status(lib, name, good, T=T) == 2
    assert _status(lib, name, good, T=T, R=0) == 2
    assert _status(lib, name, good, T=2.0 ** -126) == 1  # taken: the pointers are no device's
