"""Refusals of the operators around the FFN (norms, 8-bit checkpoints, mixture of
experts): every argument is checked before any HIP call, so no GPU is needed."""
import ctypes

import pytest
import torch

from deterministic_gated_ffn_amd import binding

FAKE = 1 << 20  # a 16-byte aligned stand-in address; never dereferenced by these calls
BF = binding.DGF_BF16
EINVAL, EUNSUPPORTED, EWORKSPACE = 1, 2, 3
nan, inf = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    return binding.load()


def refused(lib, status, want, text):
    assert status == want, (status, lib.dgf_last_error())
    assert text in lib.dgf_last_error(), lib.dgf_last_error()


def caller(fn, names, defaults):
    def call(**change):
        unknown = set(change) - set(names)
        assert not unknown, unknown
        return fn(*[{**defaults, **change}[n] for n in names])
    return call


@pytest.fixture
def norm_fwd(lib):
    names = ("res ld_res y ld_y w_post gate ld_gate alpha w_next eps z ld_z h ld_h rstd M H dtype stream").split()
    return caller(lib.dgf_norm_fwd, names, dict(
        res=FAKE, ld_res=64, y=FAKE, ld_y=64, w_post=FAKE, gate=FAKE, ld_gate=0, alpha=1.0, w_next=FAKE, eps=1e-6,
        z=FAKE, ld_z=64, h=FAKE, ld_h=64, rstd=FAKE, M=4, H=64, dtype=BF, stream=None))


def test_norm_fwd_refusals(lib, norm_fwd):
    for change, status, text in (
            (dict(dtype=binding.DGF_FP32), EUNSUPPORTED, b"FP32"), (dict(dtype=9), EINVAL, b"dtype"),
            (dict(M=-1), EINVAL, b"negative"), (dict(M=(1 << 21) + 1), EUNSUPPORTED, b"limits"),
            (dict(H=0), EINVAL, b"H must"), (dict(H=16385, ld_res=16392), EUNSUPPORTED, b"H=16385"),
            (dict(eps=0.0), EINVAL, b"eps"), (dict(eps=nan), EINVAL, b"eps"), (dict(eps=inf), EINVAL, b"eps"),
            (dict(alpha=nan), EINVAL, b"alpha"), (dict(alpha=inf), EINVAL, b"alpha"),
            (dict(y=None), EINVAL, b"need a block output"),
            (dict(y=None, w_post=None, gate=None, alpha=0.5), EINVAL, b"need a block output"),
            (dict(y=None, w_post=None, gate=None, w_next=None, h=None), EINVAL, b"nothing to compute"),
            (dict(h=None), EINVAL, b"w_next and h"), (dict(w_next=None), EINVAL, b"w_next and h"),
            (dict(res=None), EINVAL, b"res is NULL"), (dict(z=None), EINVAL, b"z is NULL"),
            (dict(res=FAKE + 2), EINVAL, b"aligned"), (dict(ld_res=56), EINVAL, b"leading dimension"),
            (dict(ld_y=60), EINVAL, b"leading dimension"), (dict(ld_h=68), EINVAL, b"multiple of 8"),
            (dict(ld_z=1 << 23), EUNSUPPORTED, b"limit"), (dict(w_post=FAKE + 8), EINVAL, b"w_post"),
            (dict(w_next=FAKE + 2), EINVAL, b"w_next"), (dict(gate=FAKE + 2), EINVAL, b"gate"),
            (dict(ld_gate=8), EINVAL, b"gate"), (dict(rstd=FAKE + 2), EINVAL, b"rstd")):
        refused(lib, norm_fwd(**change), status, text)
    assert norm_fwd(M=0, res=None, y=None, z=None, h=None) == 0  # no rows: no launch


def test_norm_bwd_refusals(lib):
    names = ("dz ld_dz dh ld_dh z ld_z y ld_y w_post gate ld_gate alpha w_next rstd dres ld_dres dy ld_dy dw_post dgate "
             "ld_dgate dw_next M H ws ws_bytes dtype stream").split()
    call = caller(lib.dgf_norm_bwd, names, dict(
        dz=FAKE, ld_dz=64, dh=FAKE, ld_dh=64, z=FAKE, ld_z=64, y=FAKE, ld_y=64, w_post=FAKE, gate=FAKE, ld_gate=64,
        alpha=1.0, w_next=FAKE, rstd=FAKE, dres=FAKE, ld_dres=64, dy=FAKE, ld_dy=64, dw_post=FAKE, dgate=FAKE, ld_dgate=64,
        dw_next=FAKE, M=4, H=64, ws=FAKE, ws_bytes=1 << 20, dtype=BF, stream=None))
    for change, status, text in (
            (dict(dtype=7), EINVAL, b"dtype"), (dict(H=20000), EUNSUPPORTED, b"H=20000"),
            (dict(dh=None), EINVAL, b"dh and w_next"), (dict(w_next=None, dw_next=None), EINVAL, b"dh and w_next"),
            (dict(dz=None, dh=None, w_next=None, dw_next=None), EINVAL, b"no gradient"),
            (dict(w_post=None), EINVAL, b"dw_post without"), (dict(gate=None), EINVAL, b"dgate without"),
            (dict(dh=None, w_next=None), EINVAL, b"dw_next without"),
            (dict(y=None, w_post=None, gate=None, dw_post=None, dgate=None, alpha=2.0), EINVAL, b"need a block output"),
            (dict(z=None), EINVAL, b"z is NULL"), (dict(dres=None), EINVAL, b"dres is NULL"),
            (dict(dy=None), EINVAL, b"dy is NULL"), (dict(rstd=None), EINVAL, b"rstd"),
            (dict(dw_post=FAKE + 1), EINVAL, b"2-byte"), (dict(ld_dgate=32), EINVAL, b"dgate"),
            (dict(ld_gate=0, dgate=FAKE + 1), EINVAL, b"dgate"),
            (dict(ws=None), EWORKSPACE, b"workspace"), (dict(ws_bytes=64), EWORKSPACE, b"workspace"),
            (dict(ws=FAKE + 4), EWORKSPACE, b"workspace")):
        refused(lib, call(**change), status, text)
    assert lib.dgf_norm_bwd_workspace(4, 64) == 3 * 4 * 64 * 4
    assert lib.dgf_norm_bwd_workspace(0, 64) == 0 and lib.dgf_norm_bwd_workspace(4, 1 << 20) == 0


def test_pack8_refusals(lib):
    names = "x ldx q ld_q scales ld_s M N dtype stream".split()
    d = dict(x=FAKE, ldx=200, q=FAKE, ld_q=208, scales=FAKE, ld_s=4, M=3, N=200, dtype=BF, stream=None)
    for fn, order in ((lib.dgf_pack8, names), (lib.dgf_unpack8, "q ld_q scales ld_s x ldx M N dtype stream".split())):
        call = caller(fn, order, d)
        for change, status, text in (
                (dict(x=None), EINVAL, b"x is NULL"), (dict(q=None), EINVAL, b"codes is NULL"),
                (dict(scales=None), EINVAL, b"scales is NULL"), (dict(q=FAKE + 8), EINVAL, b"codes are not 16-byte"),
                (dict(scales=FAKE + 2), EINVAL, b"4-byte"), (dict(ld_q=199), EINVAL, b"codes"),
                (dict(ld_q=204), EINVAL, b"codes"), (dict(ld_s=3), EINVAL, b"4 blocks"), (dict(ldx=196), EINVAL, b"x:"),
                (dict(ld_q=1 << 23), EUNSUPPORTED, b"limit"), (dict(N=-1), EINVAL, b"negative"),
                (dict(dtype=binding.DGF_FP32), EUNSUPPORTED, b"FP32")):
            refused(lib, call(**change), status, text)
        assert call(M=0, x=None, q=None, scales=None) == 0 and call(N=0) == 0


def test_q8_backward_refusals(lib):
    act = caller(lib.dgf_act_bwd_q8, "da ldda g_q g_s u_q u_s ld_q ld_s dg du a ld_out M N dtype stream".split(), dict(
        da=FAKE, ldda=64, g_q=FAKE, g_s=FAKE, u_q=FAKE, u_s=FAKE, ld_q=64, ld_s=1, dg=FAKE, du=FAKE, a=None, ld_out=64,
        M=2, N=64, dtype=BF, stream=None))
    for change, text in ((dict(da=None), b"da is NULL"), (dict(g_q=None), b"g: the codes"), (dict(u_s=None), b"u: the scales"),
                         (dict(du=None), b"du is NULL"), (dict(a=FAKE + 2), b"a is not"), (dict(ld_s=0), b"scales")):
        refused(lib, act(**change), EINVAL, text)
    assert act(M=0) == 0
    fwd = caller(lib.dgf_ffn_fwd_q8, ("x ldx wg ldwg wu ldwu wd ldwd y ldy g_q g_s u_q u_s ld_q ld_s M H I ws ws_bytes dtype "
                                      "stream").split(), dict(
        x=FAKE, ldx=64, wg=FAKE, ldwg=64, wu=FAKE, ldwu=64, wd=FAKE, ldwd=96, y=FAKE, ldy=64, g_q=FAKE, g_s=FAKE, u_q=FAKE,
        u_s=FAKE, ld_q=96, ld_s=2, M=4, H=64, I=96, ws=FAKE, ws_bytes=1 << 30, dtype=BF, stream=None))
    refused(lib, fwd(g_q=None), EINVAL, b"g: the codes")
    refused(lib, fwd(ld_s=1), EINVAL, b"2 blocks")
    refused(lib, fwd(ws_bytes=8), EWORKSPACE, b"workspace")
    refused(lib, fwd(x=None), EINVAL, b"x is NULL")
    refused(lib, fwd(H=1 << 17, ldx=1 << 17, ldwg=1 << 17, ldwu=1 << 17, ldy=1 << 17), EUNSUPPORTED, b"too deep")
    assert lib.dgf_ffn_fwd_q8_workspace(20, 512, 768) >= lib.dgf_ffn_fwd_workspace(20, 512, 768) + 2 * 20 * 768 * 2
    assert lib.dgf_ffn_fwd_q8_workspace(0, 512, 768) == 0


def test_moe_refusals(lib):
    names = ("x ldx wr ldr wg ldg sg wu ldu su wd ldd sd y ldy ids probs M H I E e0 El k renorm ws ws_bytes dtype "
             "stream").split()
    call = caller(lib.dgf_moe_fwd, names, dict(
        x=FAKE, ldx=64, wr=FAKE, ldr=64, wg=FAKE, ldg=64, sg=64 * 32, wu=FAKE, ldu=64, su=64 * 32, wd=FAKE, ldd=32, sd=64 * 32,
        y=FAKE, ldy=64, ids=None, probs=None, M=4, H=64, I=32, E=8, e0=0, El=8, k=2, renorm=1, ws=FAKE, ws_bytes=1 << 24,
        dtype=BF, stream=None))
    for change, status, text in (
            (dict(k=0), EINVAL, b"k=0"), (dict(k=9), EINVAL, b"k=9"), (dict(El=0), EINVAL, b"experts [0"),
            (dict(e0=-1), EINVAL, b"experts [-1"), (dict(e0=1), EINVAL, b"experts [1"), (dict(El=9), EINVAL, b"experts"),
            (dict(H=0), EINVAL, b"positive"), (dict(E=0), EINVAL, b"positive"), (dict(M=129), EUNSUPPORTED, b"M <= 128"),
            (dict(E=1025), EUNSUPPORTED, b"E <= 1024"), (dict(E=64, k=17), EUNSUPPORTED, b"k <= 16"),
            (dict(I=(1 << 17) + 8), EUNSUPPORTED, b"I <= "), (dict(M=-1), EINVAL, b"negative"),
            (dict(x=None), EINVAL, b"x is NULL"), (dict(wr=FAKE + 2), EINVAL, b"w_router"), (dict(wg=None), EINVAL, b"w_gate"),
            (dict(sg=64 * 31), EINVAL, b"w_gate: expert stride"), (dict(su=64 * 32 + 4), EINVAL, b"w_up: expert stride"),
            (dict(ldd=24), EINVAL, b"w_down"), (dict(y=None), EINVAL, b"y is NULL"), (dict(ids=FAKE + 2), EINVAL, b"ids"),
            (dict(ws=None), EWORKSPACE, b"workspace"), (dict(ws_bytes=100), EWORKSPACE, b"workspace"),
            (dict(dtype=binding.DGF_FP32), EUNSUPPORTED, b"FP32")):
        refused(lib, call(**change), status, text)
    assert call(M=0, x=None, y=None, ws=None) == 0
    assert lib.dgf_moe_fwd_workspace(4, 64, 32, 8, 8, 2) > 0
    assert lib.dgf_moe_fwd_workspace(129, 64, 32, 8, 8, 2) == 0 and lib.dgf_moe_fwd_workspace(4, 64, 32, 8, 9, 2) == 0


def test_binding_refusals():
    """The binding names the tensor that does not fit before anything reaches the library."""
    b, h = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(4, 64, dtype=torch.float16)
    f = torch.zeros(4, 64)
    w = torch.ones(64, dtype=torch.bfloat16)
    with pytest.raises(TypeError, match="float32"):
        binding.norm_fwd(f, w_next=w)
    with pytest.raises(ValueError, match="GPU tensor"):
        binding.norm_fwd(b, w_next=w)
    with pytest.raises(ValueError, match="expanded"):
        binding._gate(w.expand(4, 64), 4, 64, b)
    with pytest.raises(ValueError, match="rstd"):
        binding.norm_bwd(b, None, b)
    with pytest.raises(ValueError, match="GPU tensor"):
        binding.pack8(b)
    codes, scales = torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4, 1)
    with pytest.raises(TypeError, match="bfloat16 or float16"):
        binding.unpack8(binding.Packed8(codes, scales, torch.float32))
    with pytest.raises(ValueError, match="GPU tensors"):
        binding.unpack8(binding.Packed8(codes, scales, torch.bfloat16))
    with pytest.raises(ValueError, match="out"):
        binding.norm_fwd(b, w_next=w, out=b)
    with pytest.raises(TypeError, match="int8"):
        binding.unpack8(binding.Packed8(codes.float(), scales, torch.bfloat16))
    with pytest.raises(ValueError, match="GPU tensor"):
        binding.moe_fwd(b, torch.zeros(8, 64, dtype=torch.bfloat16), *[torch.zeros(8, 64, 64, dtype=torch.bfloat16)] * 3, 2)
    with pytest.raises(TypeError, match="float16"):
        binding.ffn_fwd_q8(b, h, h, h)


def test_signatures_have_c_types():
    for name in ("dgf_norm_fwd", "dgf_norm_bwd", "dgf_moe_fwd", "dgf_pack8", "dgf_act_bwd_q8", "dgf_ffn_bwd_q8"):
        res, args = binding.SIGNATURES[name]
        assert res is ctypes.c_int and args[-1] is ctypes.c_void_p and args[-2] is ctypes.c_int, name
