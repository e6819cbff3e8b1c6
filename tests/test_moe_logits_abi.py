"""Refusals of the router's FP32 logits: every argument is checked before any HIP call, so no GPU is needed."""
import pytest
import torch

from deterministic_gated_ffn_amd import binding

FAKE = 1 << 20  # a 16-byte aligned stand-in address; never dereferenced by these calls
EINVAL, EUNSUPPORTED = 1, 2
NAMES = "x ldx w ldw logits ld M H E dtype stream".split()


def test_refusals():
    lib = binding.load()
    d = dict(x=FAKE, ldx=64, w=FAKE, ldw=64, logits=FAKE, ld=60, M=5, H=64, E=60, dtype=binding.DGF_BF16, stream=None)
    for change, status, text in (
            (dict(M=-1), EINVAL, b"negative"), (dict(H=-1), EINVAL, b"negative"), (dict(E=0), EINVAL, b"E=0"),
            (dict(E=1025, ld=1025), EUNSUPPORTED, b"E <= 1024"), (dict(M=(1 << 21) + 1), EUNSUPPORTED, b"2^21"),
            (dict(H=1 << 23), EUNSUPPORTED, b"2^23"), (dict(dtype=binding.DGF_FP32), EUNSUPPORTED, b"FP32"),
            (dict(dtype=9), EINVAL, b"dtype"), (dict(x=None), EINVAL, b"x is NULL"), (dict(w=FAKE + 2), EINVAL, b"w_router is not"),
            (dict(ldx=56), EINVAL, b"x: leading"), (dict(ldw=68), EINVAL, b"w_router: leading"),
            (dict(logits=None), EINVAL, b"logits is NULL"), (dict(logits=FAKE + 2), EINVAL, b"logits is not aligned"),
            (dict(ld=59), EINVAL, b"logits: leading")):
        got = lib.dgf_moe_logits(*[{**d, **change}[n] for n in NAMES])
        assert got == status and text in lib.dgf_last_error(), (change, got, lib.dgf_last_error())
    assert lib.dgf_moe_logits(*[{**d, "M": 0, "x": None, "logits": None}[n] for n in NAMES]) == 0


def test_binding_refusals():
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(8, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU tensor"):
        binding.moe_logits(x, w)
    with pytest.raises(TypeError, match="float32"):
        binding.moe_logits(x.float(), w)
