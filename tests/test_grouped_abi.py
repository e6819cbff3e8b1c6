"""Grouped products without rows or columns: an empty matrix may be NULL, also in the second term.  Nothing is launched."""
import pytest

from deterministic_gated_ffn_amd import binding

FAKE = 1 << 20  # a 16-byte aligned stand-in address; never dereferenced by these calls
NAMES = "layout A lda B ldb sb A2 lda2 B2 ldb2 sb2 rows T offsets C ldc sc M N K E dtype stream".split()


@pytest.mark.parametrize("layout", [binding.DGF_NT, binding.DGF_NN])
def test_second_term_without_tokens(layout):
    lib = binding.load()
    d = dict(layout=layout, A=None, lda=64, B=FAKE, ldb=64, sb=64 * 64, A2=None, lda2=64, B2=FAKE, ldb2=64, sb2=64 * 64, rows=None,
             T=0, offsets=FAKE, C=None, ldc=64, sc=0, M=0, N=64, K=64, E=4, dtype=binding.DGF_BF16, stream=None)
    call = lambda **c: lib.dgf_gemm_grouped(*[{**d, **c}[n] for n in NAMES])  # noqa: E731
    assert call() == 0
    assert call(M=0, rows=FAKE) == 0
    full = dict(A=FAKE, C=FAKE, M=8, T=8)
    for change in (dict(A2=None), dict(A2=FAKE, B2=None)):
        assert call(**full, **change) == 1 and b"both" in lib.dgf_last_error()
    assert call(layout=binding.DGF_TN, A=FAKE, M=64, K=0) == 1 and b"both" in lib.dgf_last_error()
    assert call(layout=binding.DGF_TN, A=FAKE, A2=FAKE, M=64, K=0) == 1 and b"one pair" in lib.dgf_last_error()
