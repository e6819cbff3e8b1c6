"""GPU: activation checkpoints in 8 bits (pack8, unpack8), the activation's
backward from them (act_bwd_q8) and the FFN that keeps them (ffn_fwd_q8,
ffn_bwd_q8).

The format is exact: scales and codes are compared bit for bit with the same
FP32 operations in numpy.  Against FP64, a value reads back within half a step
(A / 254) plus three FP32 roundings of A, then one rounding to the stored type.
act_bwd_q8's outputs are off by one rounding (u = 2^-8 BF16, 2^-11 FP16) and at
most 16 FP32 roundings of the terms' magnitudes."""
import numpy as np
import pytest
import torch

import oracle
from deterministic_gated_ffn_amd import binding as dgf

pytestmark = pytest.mark.gpu

BF, FH = torch.bfloat16, torch.float16
U = {BF: 2.0 ** -8, FH: 2.0 ** -11}
TINY = {BF: 2.0 ** -134, FH: 2.0 ** -25}


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible: the GPU tests need an MI355X")
    dgf.load()


def rows(gen, shape, dt, scale=1.0, pad=0):
    ld = -(-shape[-1] // 8) * 8 + pad
    buf = torch.full((*shape[:-1], ld), float("nan"), dtype=dt)
    buf[..., :shape[-1]] = (torch.randn(shape, generator=gen) * scale).to(dt)
    return buf.cuda()[..., :shape[-1]]


def quantise(x):
    """The format's FP32 operations, block by block (x: FP32 numpy [M, N])."""
    M, N = x.shape
    nb = -(-N // 64)
    b = np.zeros((M, nb * 64), np.float32)
    b[:, :N] = x
    b = b.reshape(M, nb, 64)
    top = np.abs(b).max(2)
    dead = top < np.float32(2.0 ** -119)
    with np.errstate(all="ignore"):
        s = np.where(dead, np.float32(0), top / np.float32(127)).astype(np.float32)
        inv = np.where(dead, np.float32(0), np.float32(127) / top).astype(np.float32)
        q = np.rint(b * inv[..., None])
    bad = ~np.isfinite(b).all(2)
    s[bad], q[bad] = np.nan, 0
    return q.reshape(M, -1)[:, :N].astype(np.int8), s


def same_bits(a, b):
    return np.array_equal(np.asarray(a), np.asarray(b), equal_nan=np.asarray(a).dtype.kind == "f")


SHAPES = [(1, 1), (1, 63), (3, 64), (2, 65), (5, 130), (17, 200), (9, 513), (1, 12288), (33, 5461), (300, 64), (2, 40000)]


@pytest.mark.parametrize("dt", [BF, FH])
@pytest.mark.parametrize("M,N", SHAPES)
def test_codes_scales_and_what_they_read_back_as(M, N, dt):
    gen = torch.Generator().manual_seed(M + N)
    x = rows(gen, (M, N), dt, 1.7, pad=8)
    p = dgf.pack8(x)
    xf = x.float().cpu().numpy()
    q, s = quantise(xf)
    assert same_bits(p.scales.cpu().numpy(), s)
    assert same_bits(p.codes.cpu().numpy(), q)
    back = dgf.unpack8(p)
    assert back.dtype == dt and back.shape == x.shape
    want = torch.from_numpy(q.astype(np.float32) * np.repeat(s, 64, 1)[:, :N]).to(dt)
    assert torch.equal(back.cpu(), want)
    top = np.repeat(s.astype(np.float64) * 127, 64, 1)[:, :N]
    off = np.abs(back.double().cpu().numpy() - xf)
    assert (off <= top / 254 + 3 * 2.0 ** -24 * top + U[dt] * (np.abs(xf) + top / 254) + TINY[dt]).all()


def test_blocks_of_zeros_tiny_infinite_and_nan_values():
    x = torch.zeros(6, 192, dtype=BF)
    x[0, 64:128] = torch.randn(64)
    x[1, :64] = 2.0 ** -130                      # below 2^-119: kept as zeros
    x[2, :64] = 2.0 ** -118
    x[3, 70] = float("inf")
    x[4, 130] = float("nan")
    x[5] = torch.finfo(BF).max
    x[5, 64:] *= -1
    back = dgf.unpack8(dgf.pack8(x.cuda())).cpu()
    assert (back[0, :64] == 0).all() and (back[0, 128:] == 0).all() and (back[0, 64:128] != 0).any()
    assert (back[1] == 0).all()
    assert torch.equal(back[2], x[2])
    assert torch.isnan(back[3, 64:128]).all() and (back[3, :64] == 0).all() and (back[3, 128:] == 0).all()
    assert torch.isnan(back[4, 128:]).all() and (back[4, :128] == 0).all()
    assert torch.equal(back[5], x[5])


def test_offsets_past_32_bits():
    # the last rows' codes, values and outputs lie past 2^32 bytes
    ld, N = (1 << 22) + 8, 100
    M = (1 << 32) // ld + 3
    codes = torch.empty((M, ld), dtype=torch.int8, device="cuda")[:, :N]
    x = torch.randn(M, N, generator=torch.Generator().manual_seed(1)).to(BF).cuda()
    x = torch.nn.functional.pad(x, (0, 4))[:, :N]
    p = dgf.pack8(x)
    codes.copy_(p.codes)
    wide = torch.empty((M, ld), dtype=BF, device="cuda")[:, :N]
    wide.copy_(x)
    far = dgf.pack8(wide)
    assert torch.equal(far.codes, p.codes) and torch.equal(far.scales, p.scales)
    assert torch.equal(dgf.unpack8(dgf.Packed8(codes, p.scales, BF)), dgf.unpack8(p))


def act64(da, g, u):
    sg = 1.0 / (1.0 + torch.exp(-g))
    ds = sg * (1.0 + g * (1.0 - sg))
    size = sg * (1.0 + (g * (1.0 - sg)).abs())
    return {"dg": (da * u * ds, (da * u).abs() * size), "du": (da * g * sg, (da * g * sg).abs()),
            "a": (g * sg * u, (g * sg * u).abs())}


@pytest.mark.parametrize("dt", [BF, FH])
@pytest.mark.parametrize("M,N", SHAPES)
def test_activation_backward_from_8_bits(M, N, dt):
    gen = torch.Generator().manual_seed(M * N)
    g, u, da = rows(gen, (M, N), dt, 2.0), rows(gen, (M, N), dt, 1.3), rows(gen, (M, N), dt, 0.5, pad=16)
    pg, pu = dgf.pack8(g), dgf.pack8(u)
    got = dict(zip(("dg", "du", "a"), dgf.act_bwd_q8(da, pg, pu)))
    read = lambda p: (p.codes.float() * p.scales.repeat_interleave(64, 1)[:, :N]).double().cpu()  # noqa: E731
    for k, (want, size) in act64(da.double().cpu(), read(pg), read(pu)).items():
        off = (got[k].double().cpu() - want).abs()
        assert (off <= U[dt] * want.abs() + 16 * 2.0 ** -24 * size + TINY[dt]).all(), k


def test_activation_backward_against_differences():
    """dG, dU along random directions against central differences of the FP64
    activation at the values read back (error O(step^2)); roundings: u sum |g v|."""
    M, N, dt = 4, 130, FH
    gen = torch.Generator().manual_seed(2)
    pg, pu = dgf.pack8(rows(gen, (M, N), dt, 1.5)), dgf.pack8(rows(gen, (M, N), dt))
    da = rows(gen, (M, N), dt, 0.5)
    dg, du, _ = dgf.act_bwd_q8(da, pg, pu)
    read = lambda p: (p.codes.float() * p.scales.repeat_interleave(64, 1)[:, :N]).double().cpu()  # noqa: E731
    g, u, w, step = read(pg), read(pu), da.double().cpu(), 2.0 ** -13
    loss = lambda g, u: (w * g / (1 + torch.exp(-g)) * u).sum()  # noqa: E731
    for grad, where in ((dg, 0), (du, 1)):
        v = torch.randn(M, N, generator=gen, dtype=torch.float64)
        at = lambda t: loss(g + t * v, u) if where == 0 else loss(g, u + t * v)  # noqa: E731
        diff = (at(step) - at(-step)) / (2 * step)
        gv = grad.double().cpu() * v
        assert abs(gv.sum() - diff) <= 2 * U[dt] * gv.abs().sum() + 1e-6


def bits(t):
    return t.detach().contiguous().cpu().view(torch.int16).numpy().view(np.uint16)


# 4 and 20 tokens: the fused gate/up kernel, whose g and u are packed after it (H = 512);
# H = 200: a ragged last leaf through the streaming join; 160 tokens: the tiled kernel
@pytest.mark.parametrize("dt", [BF, FH])
@pytest.mark.parametrize("M,H,I", [(4, 512, 768), (20, 512, 200), (1, 200, 77), (48, 256, 640), (160, 256, 648), (130, 320, 333)])
def test_ffn_with_8_bit_checkpoint(M, H, I, dt):
    gen = torch.Generator().manual_seed(M + H + I)
    x, dy = rows(gen, (M, H), dt), rows(gen, (M, H), dt)
    wg, wu, wd = (rows(gen, s, dt, 0.05) for s in ((I, H), (I, H), (H, I)))
    y, g, u = dgf.ffn_fwd(x, wg, wu, wd, training=True)
    y8, g8, u8 = dgf.ffn_fwd_q8(x, wg, wu, wd)
    assert torch.equal(y8, y)
    for p, t in ((g8, g), (u8, u)):
        q = dgf.pack8(t)
        assert torch.equal(p.codes, q.codes) and torch.equal(p.scales, q.scales)
    r = dgf.ffn_bwd_q8(dy, x, g8, u8, wg, wu, wd)
    # the same backward from its parts
    da = dgf.gemm_tree("NN", dy, wd)
    dg, du, a = dgf.act_bwd_q8(da, g8, u8)
    want = {"dX": dgf.tree_combine([dgf.gemm_tree("NN", dg, wg).contiguous(), dgf.gemm_tree("NN", du, wu).contiguous()]),
            "dW_gate": dgf.gemm_tree("TN", dg, x), "dW_up": dgf.gemm_tree("TN", du, x), "dW_down": dgf.gemm_tree("TN", dy, a)}
    for k, t in want.items():
        assert np.array_equal(bits(r[k]), bits(t)), k
    # and close to the backward from the 16-bit g and u: a block's values are off by at most
    # 1/254 of its largest, about 1/80 of a normal block's root mean square in the worst place
    # and 0.6% in the mean square, so a gradient that sums hundreds of them moves by about 1%
    full = dgf.ffn_bwd(dy, x, g, u, wg, wu, wd)
    for k in full:
        a, b = full[k].double().cpu(), r[k].double().cpu()
        assert (a - b).norm() <= 0.03 * a.norm(), k


def test_ffn_with_8_bit_checkpoint_has_the_oracle_s_output():
    M, H, I = 5, 256, 320
    rng = np.random.default_rng(0)
    x, wg, wu, wd = (oracle.f32_to_bf16_bits((rng.standard_normal(s) * k).astype(np.float32))
                     for s, k in (((M, H), 1.0), ((I, H), 0.05), ((I, H), 0.05), ((H, I), 0.05)))
    dev = [torch.from_numpy(b.view(np.int16)).cuda().view(BF) for b in (x, wg, wu, wd)]
    y, g8, u8 = dgf.ffn_fwd_q8(*dev)
    o = oracle.ffn_fwd(x, wg, wu, wd)
    assert np.array_equal(bits(y), o["y"])
    for p, name in ((g8, "g"), (u8, "u")):
        q, s = quantise((o[name].astype(np.uint32) << 16).view(np.float32))
        assert same_bits(p.codes.cpu().numpy(), q) and same_bits(p.scales.cpu().numpy(), s)


def test_another_stream_and_empty_inputs():
    gen = torch.Generator().manual_seed(9)
    x = rows(gen, (50, 700), BF)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    p = dgf.pack8(x, stream=side)
    back = dgf.unpack8(p, stream=side)
    side.synchronize()
    assert torch.equal(back, dgf.unpack8(dgf.pack8(x)))
    assert dgf.unpack8(dgf.pack8(x[:0])).shape == (0, 700)
    w = [rows(gen, s, BF, 0.05) for s in ((64, 32), (64, 32), (32, 64))]
    x0 = rows(gen, (1, 32), BF)[:0]
    y, g, u = dgf.ffn_fwd_q8(x0, *w)
    r = dgf.ffn_bwd_q8(y, x0, g, u, *w)
    assert y.shape == (0, 32) and all((bits(r[k]) == 0).all() for k in ("dW_gate", "dW_up", "dW_down"))
