"""4-bit weights: packing bit for bit, products against FP64 on the values that the codes stand for.

Tolerances.  A product's codes enter the matrix core as 24 + c and -24 times the
activations' sum takes the excess out, so its rounding goes by S' = sum |x| s 48:
one of 2^-23 S' for every block of 8 columns (and of the excess) in a wave's share
of K, and 12 for the sums over groups and waves: (K / 4 + 12) 2^-23 S' covers any
split.  The activation of the FFN is silu (slope at most 1.1) of such a product
times another, kept to 2^-16 of its value."""
import pytest
import torch

from deterministic_gated_ffn_amd import binding as dgf

pytestmark = pytest.mark.gpu
BF, FH = torch.bfloat16, torch.float16
nan, inf = float("nan"), float("inf")


def rows(gen, M, K, dtype, scale=1.0, pad=0):
    buf = torch.full((M, (K + 7) // 8 * 8 + pad), nan, dtype=dtype, device="cuda")
    buf[:, :K] = (torch.randn(M, K, generator=gen, device="cuda") * scale).to(dtype)
    return buf[:, :K]


def quantised(w, group):
    """(codes int, scales) [N, groups, group] by definition: s = rnd(A / 7), c = rint(w / s) in [-7, 7]."""
    N, K = w.shape
    ng = -(-K // group)
    b = torch.nn.functional.pad(w.float(), (0, ng * group - K)).view(N, ng, group)
    s = (b.abs().amax(2) / 7.0).to(w.dtype)
    sf = s.float()[..., None]
    return torch.where(sf > 0, torch.round(b / sf).clamp(-7, 7), 0.0), s


def values(w, group):
    c, s = quantised(w, group)
    return (c.double() * s.double()[..., None]).view(w.shape[0], -1)[:, :w.shape[1]]


@pytest.mark.parametrize("dtype", [BF, FH], ids=str)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("N,K", [(1, 1), (16, 128), (17, 129), (5, 31), (33, 500), (100, 1003), (8, 4096)])
def test_pack(dtype, group, N, K):
    gen = torch.Generator(device="cuda").manual_seed(N + K)
    w = rows(gen, N, K, dtype, 0.03, pad=8)
    w[0, 0] = 0
    if K > 300:
        w[0, :group] = 0           # a group of zeros
        w[-1, :8] = -w[-1].abs().max()
    p = dgf.pack4(w, group=group)
    c, s = quantised(w, group)
    tn, tk = -(-N // 16), -(-K // 128)
    # the documented layout, read back on the host
    q = p.codes.view(torch.int32).cpu().view(tn, tk, 4, 16, 4).long() & 0xFFFFFFFF  # lane = 16 g + row; dword i
    full = torch.empty(tn * 16, tk * 128, dtype=torch.long)
    for col in range(128):
        i, g, e = col // 32, col % 32 // 8, col % 8
        v = q[:, :, g, :, i] >> (4 * (e // 2) + 16 * (e % 2)) & 15
        full[:, col::128] = v.permute(0, 2, 1).reshape(tn * 16, tk) - 8
    want = torch.nn.functional.pad(c.view(N, -1).cpu().long(), (0, max(0, tk * 128 - c.shape[1] * group)))[:, :tk * 128]
    assert torch.equal(full[:N], want) and not full[N:].any()
    sc = p.scales.permute(0, 2, 1, 3).reshape(tn * 16, -1)
    assert torch.equal(sc[:N, :s.shape[1]], s)
    u = dgf.unpack4(p)
    assert u.shape == (N, K) and torch.equal(u, values(w, group).float().to(dtype))


def test_pack_special_groups():
    w = torch.zeros(4, 256, dtype=FH, device="cuda")
    w[0, 3], w[1, 70], w[2, :] = nan, -inf, 65504.0
    w[3, :64] = 5.96e-8  # A / 7 rounds to zero
    u = dgf.unpack4(dgf.pack4(w, group=64))
    assert u[0, :64].isnan().all() and not u[0, 64:].any()
    assert u[1, 64:128].isnan().all() and not u[1, :64].any() and not u[3].any()
    assert (u[2] - 65504.0).abs().max() <= 65504 * 2.0 ** -10


@pytest.mark.parametrize("dtype", [BF, FH], ids=str)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (1, 4096, 1024), (2, 17, 129), (5, 1411, 1003), (16, 48, 128), (17, 100, 2051),
                                   (33, 64, 640), (64, 33, 96), (100, 130, 260)])
def test_product(dtype, group, M, N, K):
    gen = torch.Generator(device="cuda").manual_seed(M + N + K)
    w, x = rows(gen, N, K, dtype, K ** -0.5), rows(gen, M, K, dtype, pad=8 * (M % 2))
    p = dgf.pack4(w, group=group)
    y = dgf.gemm_w4(x, p)
    W, X = values(w, group), x.double()
    s = quantised(w, group)[1].double().repeat_interleave(group, 1)[:, :K]
    want, size = X @ W.t(), 48 * (X.abs() @ s.t())
    tol = torch.finfo(dtype).eps / 2 * want.abs() + (K / 4 + 12) * 2.0 ** -23 * size + (2.0 ** -25 if dtype == FH else 0)
    assert ((y.double() - want).abs() <= tol).all()
    assert torch.equal(y, dgf.gemm_w4(x, p))
    # a token's result does not depend on the others
    assert torch.equal(dgf.gemm_w4(x[-1:], p)[0], y[-1])


@pytest.mark.parametrize("dtype", [BF, FH], ids=str)
@pytest.mark.parametrize("M,H,I,group", [(1, 512, 768, 64), (3, 77, 130, 32), (16, 256, 256, 128), (31, 1003, 411, 64),
                                         (70, 128, 1000, 32)])
def test_ffn(dtype, M, H, I, group):
    gen = torch.Generator(device="cuda").manual_seed(M + H)
    ws = [rows(gen, I, H, dtype, H ** -0.5), rows(gen, I, H, dtype, H ** -0.5), rows(gen, H, I, dtype, I ** -0.5)]
    x = rows(gen, M, H, dtype)
    p = [dgf.pack4(w, group=group) for w in ws]
    y = dgf.ffn_fwd_w4(x, *p)
    X = x.double()
    wg, wu, wd = (values(w, group) for w in ws)
    scales = [quantised(w, group)[1].double().repeat_interleave(group, 1)[:, :w.shape[1]] for w in ws]
    err = (H / 4 + 12) * 2.0 ** -23 * 48
    g, u = X @ wg.t(), X @ wu.t()
    a = torch.nn.functional.silu(g) * u
    da = 1.1 * err * ((X.abs() @ scales[0].t()) * u.abs() + (X.abs() @ scales[1].t()) * g.abs()) + (2.0 ** -16 + 2.0 ** -20) * a.abs()
    want = a @ wd.t()
    tol = torch.finfo(dtype).eps / 2 * want.abs() + (I / 4 + 12) * 2.0 ** -23 * 48 * (a.abs() @ scales[2].t()) + da @ wd.abs().t()
    assert ((y.double() - want).abs() <= tol + (2.0 ** -25 if dtype == FH else 0)).all()
    assert torch.equal(dgf.ffn_fwd_w4(x[-1:], *p)[0], y[-1])


def test_large_activations_fp16():
    """Activations far past FP16's range pass between the kernels."""
    gen = torch.Generator(device="cuda").manual_seed(0)
    ws = [rows(gen, 64, 128, FH, 4.0), rows(gen, 64, 128, FH, 4.0), rows(gen, 128, 64, FH, 1e-4)]
    x = rows(gen, 2, 128, FH, 10.0)
    y = dgf.ffn_fwd_w4(x, *[dgf.pack4(w) for w in ws])
    wg, wu, wd = (values(w, 64) for w in ws)
    a = torch.nn.functional.silu(x.double() @ wg.t()) * (x.double() @ wu.t())
    assert a.abs().max() > 1e5 and torch.isfinite(y).all()
    want = a @ wd.t()
    assert ((y.double() - want).norm() / want.norm()) < 2.0 ** -10


def test_captured_products_follow_their_inputs():
    gen = torch.Generator(device="cuda").manual_seed(9)
    p = [dgf.pack4(rows(gen, *s, BF, 0.05)) for s in ((256, 192), (256, 192), (192, 256))]
    x = rows(gen, 20, 192, BF)
    dgf.ffn_fwd_w4(x, *p)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = dgf.ffn_fwd_w4(x, *p)
    for _ in range(3):
        x.copy_(rows(gen, 20, 192, BF))
        graph.replay()
        want = dgf.ffn_fwd_w4(x, *p)
        torch.cuda.synchronize()
        assert torch.equal(y, want)


@pytest.mark.parametrize("dtype", [BF, FH], ids=str)
@pytest.mark.parametrize("N,K,group", [(1000, 2304, 64), (520, 4099, 128), (12304, 2048, 32), (300, 6400, 128)])
def test_a_row_does_not_depend_on_the_batch(dtype, N, K, group):
    """Wide enough that the waves start at different tiles, and every number of row tiles a workgroup."""
    gen = torch.Generator(device="cuda").manual_seed(N)
    w = dgf.pack4(rows(gen, N, K, dtype, K ** -0.5), group)
    gate, up = (dgf.pack4(rows(gen, K, N, dtype, N ** -0.5), group) for _ in range(2))
    x, h = rows(gen, 130, K, dtype), rows(gen, 130, N, dtype)
    y, z = dgf.gemm_w4(x, w), dgf.ffn_fwd_w4(h, gate, up, w)
    for lo, hi in ((0, 1), (7, 9), (20, 36), (40, 57), (60, 92), (66, 130)):
        assert torch.equal(dgf.gemm_w4(x[lo:hi], w), y[lo:hi]), (lo, hi)
        assert torch.equal(dgf.ffn_fwd_w4(h[lo:hi], gate, up, w), z[lo:hi]), (lo, hi)
