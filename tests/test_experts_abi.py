"""Refusals of the mixture of experts over many tokens, dropout and the 4-bit weights:
every argument is checked before any HIP call, so no GPU is needed."""
import ctypes

import pytest
import torch

from deterministic_gated_ffn_amd import binding

FAKE = 1 << 20  # a 16-byte aligned stand-in address; never dereferenced by these calls
BF = binding.DGF_BF16
NT, NN, TN = binding.DGF_NT, binding.DGF_NN, binding.DGF_TN
EINVAL, EUNSUPPORTED, EWORKSPACE = 1, 2, 3
nan, inf = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    return binding.load()


def check(lib, fn, names, defaults, refusals):
    names = names.split()
    assert set(defaults) == set(names)

    def call(**change):
        assert set(change) <= set(names), change
        return fn(*[{**defaults, **change}[n] for n in names])

    for change, status, text in refusals:
        got = call(**change)
        assert got == status and text in lib.dgf_last_error(), (change, got, lib.dgf_last_error())
    return call


GROUPED = "layout A lda B ldb sb A2 lda2 B2 ldb2 sb2 rows T offsets C ldc sc M N K E dtype stream"


def test_grouped_refusals(lib):
    d = dict(layout=NT, A=FAKE, lda=64, B=FAKE, ldb=64, sb=64 * 32, A2=None, lda2=0, B2=None, ldb2=0, sb2=0, rows=FAKE,
             T=10, offsets=FAKE, C=FAKE, ldc=32, sc=0, M=20, N=32, K=64, E=4, dtype=BF, stream=None)
    call = check(lib, lib.dgf_gemm_grouped, GROUPED, d, (
        (dict(layout=3), EINVAL, b"layout"), (dict(dtype=binding.DGF_FP32), EUNSUPPORTED, b"FP32"),
        (dict(dtype=8), EINVAL, b"dtype"), (dict(M=-1), EINVAL, b"negative"), (dict(E=0), EINVAL, b"E=0"),
        (dict(E=1025), EUNSUPPORTED, b"E <= 1024"), (dict(M=(1 << 25) + 1), EUNSUPPORTED, b"2^25"),
        (dict(N=1 << 23, ldc=1 << 23), EUNSUPPORTED, b"2^23"), (dict(K=1 << 23), EUNSUPPORTED, b"2^23"),
        (dict(M=1 << 25, N=(1 << 23) - 8, ldc=(1 << 23) - 8), EUNSUPPORTED, b"tiles"),
        (dict(A2=FAKE), EINVAL, b"A2 and B2"), (dict(B2=FAKE), EINVAL, b"A2 and B2"), (dict(T=-1), EINVAL, b"T=-1"),
        (dict(T=(1 << 25) + 1), EUNSUPPORTED, b"T="), (dict(rows=FAKE + 2), EINVAL, b"rows"),
        (dict(offsets=None), EINVAL, b"offsets is NULL"), (dict(offsets=FAKE + 1), EINVAL, b"offsets"),
        (dict(A=None), EINVAL, b"A is NULL"), (dict(lda=56), EINVAL, b"A: leading"), (dict(B=FAKE + 8), EINVAL, b"B is not"),
        (dict(ldb=68), EINVAL, b"multiple of 8"), (dict(sb=64 * 31), EINVAL, b"B: expert stride"),
        (dict(sb=64 * 32 + 4), EINVAL, b"B: expert stride"), (dict(C=None), EINVAL, b"C is NULL"),
        (dict(ldc=24), EINVAL, b"C: leading"), (dict(lda=1 << 23), EUNSUPPORTED, b"limit"),
        (dict(A2=FAKE, B2=FAKE, lda2=64, ldb2=32), EINVAL, b"B2: leading"),
        (dict(A2=FAKE, B2=FAKE, lda2=32, ldb2=64, sb2=2048), EINVAL, b"A2: leading")))
    assert call(M=0, A=None, B=None, C=None, offsets=None) == 0 and call(N=0) == 0  # nothing to write
    d.update(layout=TN, lda=24, ldb=32, sb=0, ldc=32, sc=24 * 32, M=24, N=32, K=20, rows=None, T=0)
    call = check(lib, lib.dgf_gemm_grouped, GROUPED, d, (
        (dict(A2=FAKE, B2=FAKE), EINVAL, b"one pair"), (dict(lda=16), EINVAL, b"A: leading"),
        (dict(sc=24 * 32 - 8), EINVAL, b"C: expert stride"), (dict(K=(1 << 25) + 1), EUNSUPPORTED, b"2^25"),
        (dict(M=1 << 22, N=1 << 22, lda=1 << 22, ldb=1 << 22, ldc=1 << 22, sc=1 << 44), EUNSUPPORTED, b"tiles")))
    assert call(N=0) == 0 and call(M=0) == 0


def test_route_refusals(lib):
    names = "logits ld ids probs offsets rows pos M E k renorm ws ws_bytes dtype stream"
    d = dict(logits=FAKE, ld=60, ids=FAKE, probs=FAKE, offsets=FAKE, rows=FAKE, pos=FAKE, M=500, E=60, k=4, renorm=1, ws=FAKE,
             ws_bytes=1 << 20, dtype=BF, stream=None)
    check(lib, lib.dgf_moe_route, names, d, (
        (dict(M=-1), EINVAL, b"negative"), (dict(k=0), EINVAL, b"k=0"), (dict(k=61), EINVAL, b"k=61"),
        (dict(E=0), EINVAL, b"E=0"), (dict(E=1025, ld=1025), EUNSUPPORTED, b"E <= 1024"), (dict(k=17), EUNSUPPORTED, b"k <= 16"),
        (dict(M=(1 << 21) + 1), EUNSUPPORTED, b"2^21"), (dict(dtype=5), EINVAL, b"dtype"), (dict(ld=59), EINVAL, b"logits: leading"),
        (dict(logits=None), EINVAL, b"logits is NULL"), (dict(logits=FAKE + 1), EINVAL, b"aligned"),
        (dict(logits=FAKE + 2, dtype=binding.DGF_FP32), EINVAL, b"aligned"), (dict(ids=None), EINVAL, b"ids"),
        (dict(probs=FAKE + 2), EINVAL, b"probs"), (dict(offsets=None), EINVAL, b"offsets"), (dict(rows=None), EINVAL, b"rows"),
        (dict(pos=FAKE + 1), EINVAL, b"pos"), (dict(ws=None), EWORKSPACE, b"workspace"),
        (dict(ws_bytes=8), EWORKSPACE, b"workspace"), (dict(ws=FAKE + 8), EWORKSPACE, b"workspace")))
    assert lib.dgf_moe_route_workspace(500, 60, 4) >= 32 * 60 * 2
    assert lib.dgf_moe_route_workspace(1, 60, 4) == 0 and lib.dgf_moe_route_workspace(500, 60, 61) == 0
    names = "dprobs logits ld ids probs dlogits ld_d M E k renorm dtype stream"
    d = dict(dprobs=FAKE, logits=FAKE, ld=64, ids=FAKE, probs=FAKE, dlogits=FAKE, ld_d=64, M=3, E=60, k=4, renorm=0, dtype=BF,
             stream=None)
    call = check(lib, lib.dgf_moe_route_bwd, names, d, (
        (dict(dprobs=None), EINVAL, b"dprobs"), (dict(ids=FAKE + 2), EINVAL, b"ids"), (dict(probs=None), EINVAL, b"probs"),
        (dict(logits=None), EINVAL, b"logits is NULL"), (dict(dlogits=None), EINVAL, b"dlogits is NULL"),
        (dict(ld_d=59), EINVAL, b"dlogits: leading"), (dict(k=0), EINVAL, b"k=0"), (dict(dtype=-1), EINVAL, b"dtype")))
    assert call(M=0, logits=None, dlogits=None, dprobs=None) == 0


def test_combine_refusals(lib):
    names = "o ld_o R pos probs y ldy M H k dtype stream"
    d = dict(o=FAKE, ld_o=64, R=12, pos=FAKE, probs=FAKE, y=FAKE, ldy=64, M=6, H=64, k=2, dtype=BF, stream=None)
    call = check(lib, lib.dgf_moe_combine, names, d, (
        (dict(M=-1), EINVAL, b"negative"), (dict(k=0), EINVAL, b"k=0"), (dict(k=17), EUNSUPPORTED, b"k <= 16"),
        (dict(R=(1 << 25) + 1), EUNSUPPORTED, b"2^25"), (dict(o=None), EINVAL, b"o is NULL"), (dict(o=FAKE + 2), EINVAL, b"o is not"),
        (dict(ld_o=56), EINVAL, b"o: leading"), (dict(pos=None), EINVAL, b"pos"), (dict(probs=FAKE + 2), EINVAL, b"probs"),
        (dict(y=None), EINVAL, b"y is NULL"), (dict(ldy=60), EINVAL, b"y: leading"), (dict(dtype=2), EUNSUPPORTED, b"FP32")))
    assert call(M=0, o=None, y=None, pos=None) == 0
    names = "dy lddy o ld_o R pos probs d_o ld_do dprobs M H k dtype stream"
    d = dict(dy=FAKE, lddy=64, o=FAKE, ld_o=64, R=12, pos=FAKE, probs=FAKE, d_o=FAKE, ld_do=64, dprobs=FAKE, M=6, H=64, k=2,
             dtype=BF, stream=None)
    call = check(lib, lib.dgf_moe_combine_bwd, names, d, (
        (dict(probs=None), EINVAL, b"dprobs without probs"), (dict(dprobs=FAKE + 2), EINVAL, b"dprobs"),
        (dict(o=None), EINVAL, b"o is NULL"), (dict(dy=None), EINVAL, b"dy is NULL"), (dict(d_o=None), EINVAL, b"d_o is NULL"),
        (dict(ld_do=32), EINVAL, b"d_o: leading"), (dict(H=0), EINVAL, b"H must"), (dict(pos=FAKE + 3), EINVAL, b"pos")))
    assert call(M=0, dy=None, o=None, d_o=None) == 0


def test_dropout_refusals(lib):
    names = "x ldx res ld_res alpha p rng z ldz M H dtype stream"
    d = dict(x=FAKE, ldx=64, res=FAKE, ld_res=64, alpha=1.0, p=0.1, rng=FAKE, z=FAKE, ldz=64, M=4, H=64, dtype=BF, stream=None)
    call = check(lib, lib.dgf_dropout, names, d, (
        (dict(p=-0.1), EINVAL, b"p="), (dict(p=1.0), EINVAL, b"p="), (dict(p=nan), EINVAL, b"p="), (dict(p=inf), EINVAL, b"p="),
        (dict(p=1 - 2.0 ** -18), EINVAL, b"p="), (dict(alpha=nan), EINVAL, b"alpha"), (dict(rng=None), EINVAL, b"rng"),
        (dict(rng=FAKE + 4), EINVAL, b"rng"), (dict(x=None), EINVAL, b"x is NULL"), (dict(res=FAKE + 2), EINVAL, b"res is not"),
        (dict(ldz=56), EINVAL, b"z: leading"), (dict(M=-2), EINVAL, b"negative"), (dict(dtype=2), EUNSUPPORTED, b"FP32"),
        (dict(H=1 << 23, ldx=1 << 23), EUNSUPPORTED, b"limit")))
    assert call(M=0, x=None, z=None, rng=None) == 0


def test_4_bit_refusals(lib):
    names = "w ldw codes scales N K group dtype stream"
    d = dict(w=FAKE, ldw=128, codes=FAKE, scales=FAKE, N=32, K=128, group=64, dtype=BF, stream=None)
    bad = ((dict(group=48), EINVAL, b"group=48"), (dict(group=0), EINVAL, b"group=0"), (dict(N=0), EINVAL, b"rows and columns"),
           (dict(K=0), EINVAL, b"rows and columns"), (dict(w=None), EINVAL, b"w is NULL"), (dict(codes=None), EINVAL, b"codes"),
           (dict(scales=None), EINVAL, b"scales"), (dict(codes=FAKE + 8), EINVAL, b"codes"), (dict(scales=FAKE + 4), EINVAL, b"scales"),
           (dict(ldw=120), EINVAL, b"w: leading"), (dict(dtype=2), EUNSUPPORTED, b"FP32"), (dict(K=1 << 23), EUNSUPPORTED, b"2^23"),
           (dict(N=1 << 19, K=1 << 18, ldw=1 << 18), EUNSUPPORTED, b"2^26 tiles"))
    check(lib, lib.dgf_pack4, names, d, bad)
    check(lib, lib.dgf_unpack4, "codes scales w ldw N K group dtype stream", d, bad)
    d = dict(x=FAKE, ldx=128, codes=FAKE, scales=FAKE, y=FAKE, ldy=32, M=3, N=32, K=128, group=64, dtype=BF, stream=None)
    call = check(lib, lib.dgf_gemm_w4, "x ldx codes scales y ldy M N K group dtype stream", d, (
        (dict(M=65537), EUNSUPPORTED, b"65536"), (dict(x=None), EINVAL, b"x is NULL"), (dict(y=FAKE + 2), EINVAL, b"y is not"),
        (dict(codes=None), EINVAL, b"codes"), (dict(group=16), EINVAL, b"group"), (dict(ldy=24), EINVAL, b"y: leading")))
    assert call(M=0, x=None, y=None) == 0
    names = "x ldx gc gs uc us dc ds y ldy M H I group ws ws_bytes dtype stream"
    d = dict(x=FAKE, ldx=64, gc=FAKE, gs=FAKE, uc=FAKE, us=FAKE, dc=FAKE, ds=FAKE, y=FAKE, ldy=64, M=2, H=64, I=96, group=32,
             ws=FAKE, ws_bytes=1 << 20, dtype=BF, stream=None)
    call = check(lib, lib.dgf_ffn_fwd_w4, names, d, (
        (dict(gc=None), EINVAL, b"gate"), (dict(us=None), EINVAL, b"up"), (dict(dc=FAKE + 2), EINVAL, b"down"),
        (dict(ws=None), EWORKSPACE, b"workspace"), (dict(ws_bytes=64), EWORKSPACE, b"workspace"), (dict(I=0), EINVAL, b"rows and"),
        (dict(M=-1), EINVAL, b"negative"), (dict(y=None), EINVAL, b"y is NULL")))
    assert call(M=0, x=None, ws=None) == 0
    assert lib.dgf_ffn_fwd_w4_workspace(2, 64, 96) == 8192 and lib.dgf_ffn_fwd_w4_workspace(0, 64, 96) == 0


def test_binding_refusals():
    """The binding names the tensor that does not fit before anything reaches the library."""
    b, off = torch.zeros(8, 64, dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int32)
    w = torch.zeros(2, 32, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="layout"):
        binding.gemm_grouped("TT", b, w, off)
    with pytest.raises(TypeError, match="float32"):
        binding.gemm_grouped("NT", b.float(), w, off)
    with pytest.raises(ValueError, match="GPU tensor"):
        binding.gemm_grouped("NT", b, w, off)
    with pytest.raises(TypeError, match="bfloat16, float16 or float32"):
        binding.moe_route(b.long(), 2)
    with pytest.raises(ValueError, match="row-major"):
        binding.moe_route(b.t(), 2)
    with pytest.raises(ValueError, match="GPU tensor"):
        binding.moe_route(b, 2)
    with pytest.raises(ValueError, match="GPU tensor"):
        binding.moe_combine(b, off.view(1, 3))
    with pytest.raises(ValueError, match="GPU tensor"):
        binding.dropout(b, 0.1, torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError, match="GPU tensor"):
        binding.pack4(b)
    p = binding.Packed4(torch.zeros(1, 1, 1024, dtype=torch.uint8), torch.zeros(1, 1, 16, 2).bfloat16(), (8, 64), 64)
    with pytest.raises(ValueError, match="GPU tensor"):
        binding.unpack4(p)
    with pytest.raises(TypeError, match="int32"):
        binding._flat_of(off.long(), torch.int32, (3,), 0, "offsets")
    with pytest.raises(ValueError, match="device"):
        binding._flat_of(off, torch.int32, (3,), 0, "offsets")


def test_signatures_have_c_types():
    for name in ("dgf_gemm_grouped", "dgf_moe_route", "dgf_moe_route_bwd", "dgf_moe_combine_bwd", "dgf_dropout", "dgf_ffn_fwd_w4"):
        res, args = binding.SIGNATURES[name]
        assert res is ctypes.c_int and args[-1] is ctypes.c_void_p and args[-2] is ctypes.c_int, name
