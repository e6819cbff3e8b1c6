"""4-bit weights where the result is known exactly.

The inputs are whole numbers times powers of two, and so are the scales: as long as
the sum of the magnitudes stays below 2^24 units, FP32 sums in any order are exact, and the
output is the exact value rounded once.  A missing column, a wrong scale and an
operand in fewer bits all change it.  (silu(g) is g itself, in FP32, from g = 20 on:
exp(-20) is less than half a step at 1.)"""
import pytest
import torch

from deterministic_gated_ffn_amd import binding as dgf

pytestmark = pytest.mark.gpu
BF, FH = torch.bfloat16, torch.float16
nan, inf = float("nan"), float("inf")
BITS = 2.0 ** 24


def matrix(t, dtype):
    """The values as a row-major GPU matrix whose rows end in NaN (never to be used)."""
    M, K = t.shape
    buf = torch.full((M, (K + 7) // 8 * 8), nan, dtype=dtype, device="cuda")
    buf[:, :K] = t.to(dtype)
    return buf[:, :K]


def draw_codes(gen, N, K, group, lo=-7, hi=7):
    """Codes [N, K], the first of every group +-7 (so that its scale is the unit the weights are given in)."""
    c = torch.randint(lo, hi + 1, (N, K), generator=gen).double()
    c[:, ::group] = 7.0 if lo >= 0 else 7.0 * (1 - 2 * torch.randint(0, 2, c[:, ::group].shape, generator=gen).double())
    return c


def packed(c, unit, dtype, group):
    p = dgf.pack4(matrix(c * unit, dtype), group=group)
    assert torch.equal(dgf.unpack4(p).double().cpu(), c * unit)
    return p


def once(t, dtype):
    return t.float().to(dtype)  # (exact in FP32)


@pytest.mark.parametrize("dtype", [BF, FH], ids=str)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M,N,K", [(1, 40, 7), (1, 33, 1024), (3, 17, 129), (16, 100, 2051), (17, 48, 1003), (33, 4100, 640),
                                   (70, 8200, 133), (100, 60, 4096)])
def test_product(dtype, group, M, N, K):
    gen = torch.Generator().manual_seed(M + N + K)
    c = draw_codes(gen, N, K, group)
    x = torch.randint(-8, 9, (M, K), generator=gen).double()
    x[:, -1] = 5.0
    assert 56 * K < BITS
    y = dgf.gemm_w4(matrix(x, dtype), packed(c, 2.0 ** -6, dtype, group))
    assert torch.equal(y.cpu(), once(x @ c.T * 2.0 ** -6, dtype))


@pytest.mark.parametrize("dtype,large,small", [(BF, 2.0 ** 100, 2.0 ** -10), (FH, 2.0 ** 15, 2.0 ** -14)], ids=str)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M", [1, 20])
def test_large_activations_at_codes_of_zero(dtype, large, small, group, M):
    """A code of 0 takes nothing from its activation, however large that is."""
    gen = torch.Generator().manual_seed(M)
    N, K = 50, 700
    c = draw_codes(gen, N, K, group)
    out = torch.arange(3, K, 32)  # (never the first of a group)
    c[:, out] = 0.0
    x = torch.randint(-8, 9, (M, K), generator=gen).double()
    p = packed(c, 2.0 ** -3, dtype, group)
    want = once(x @ c.T * small * 2.0 ** -3, dtype)
    x *= small
    x[:, out] = large * (1 - 2 * torch.randint(0, 2, (M, len(out)), generator=gen).double())
    assert torch.equal(dgf.gemm_w4(matrix(x, dtype), p).cpu(), want)


@pytest.mark.parametrize("dtype", [BF, FH], ids=str)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M", [1, 20])
def test_infinite_activations(dtype, group, M):
    """An infinity times a code is an infinity of its sign, times a code of 0 a NaN; other tokens do not see it."""
    gen = torch.Generator().manual_seed(M)
    N, K = 60, 300
    c = draw_codes(gen, N, K, group)
    x = torch.randint(-8, 9, (M, K), generator=gen).double()
    x[M // 2, 70] = -inf
    c[:4, 70] = 0.0
    y = dgf.gemm_w4(matrix(x, dtype), packed(c, 2.0 ** -3, dtype, group))
    want = (x[:, None, :] * c * 2.0 ** -3).sum(2)
    assert want.isinf().any() and want.isnan().any()
    assert torch.equal(y.cpu().nan_to_num(nan=12345.0), once(want, dtype).nan_to_num(nan=12345.0))


@pytest.mark.parametrize("dtype", [BF, FH], ids=str)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M,H,I", [(1, 512, 768), (4, 77, 130), (16, 256, 256), (31, 1003, 411), (70, 128, 1000),
                                   (18, 1003, 8200), (40, 1000, 8200), (20, 45, 4500), (33, 2048, 520)])
def test_ffn(dtype, group, M, H, I):
    """Every form of the two kernels: ragged and whole widths, one to three row tiles a workgroup."""
    gen = torch.Generator().manual_seed(M + H + I)
    cg, cu = draw_codes(gen, I, H, group, 4, 5), draw_codes(gen, I, H, group)
    cd = draw_codes(gen, H, I, group, -1, 1)
    x = torch.zeros(M, H, dtype=torch.double)
    for m in range(M):  # 6 columns, the last one among them
        x[m, torch.randperm(H - 1, generator=gen)[:5]] = 1.0
    x[:, -1] = 1.0
    g, u = x @ cg.T, x @ cu.T
    assert g.min() >= 20
    a = g * u  # 11 bits and a sign
    assert (a.abs() @ cd.abs().T).max() < BITS
    y = dgf.ffn_fwd_w4(matrix(x, dtype), packed(cg, 1.0, dtype, group), packed(cu, 0.25, dtype, group), packed(cd, 2.0 ** -10, dtype, group))
    assert torch.equal(y.cpu(), once(a @ cd.T * 2.0 ** -12, dtype))


@pytest.mark.parametrize("dtype", [BF, FH], ids=str)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M", [1, 9, 18, 40])
def test_activations_pass_whole(dtype, group, M):
    """Activations of 20 bits, of which the second product takes differences of a few units: every bit counts."""
    gen = torch.Generator().manual_seed(M)
    H, I = 40, 300
    digits = torch.randint(0, 8, (I, 6), generator=gen)  # of u, base 8
    digits[1::2, 1:] = digits[::2, 1:]                   # pairs that differ in the last one
    digits[::32] = 0                                     # the columns of the second product that hold a group's 7
    cg, cu, cd = torch.zeros(I, H).double(), torch.zeros(I, H).double(), torch.zeros(H, I).double()
    cg[:, ::group] = cu[:, ::group] = cd[:, ::group] = 7.0
    cg[:, 7], cu[:, 1:7] = 6.0, digits.double()
    for n in range(H):
        i = 2 * n + 2 + 128 * (n % 2)
        cd[n, i], cd[n, i + 1] = (1.0, -1.0) if i % 32 else (0.0, 0.0)
    x = torch.zeros(M, H).double()
    x[:, 1:7] = 8.0 ** torch.arange(6) * torch.tensor([1.0, -1.0, 0.5, -0.25, 0.125])[torch.arange(M) % 5, None]
    x[:, 7] = 4.0  # g = 24
    a = 24.0 * (x @ cu.T)
    y = dgf.ffn_fwd_w4(matrix(x, dtype), packed(cg, 1.0, dtype, group), packed(cu, 1.0, dtype, group), packed(cd, 2.0 ** -4, dtype, group))
    assert torch.equal(y.cpu(), once(a @ cd.T * 2.0 ** -4, dtype))


@pytest.mark.parametrize("dtype", [BF, FH], ids=str)
@pytest.mark.parametrize("M", [1, 20])
def test_infinite_activations_pass(dtype, M):
    """An infinite activation is an infinity in the second product too, and only its token's."""
    H, I, group = 40, 72, 32
    cg, cu, cd = torch.zeros(I, H).double(), torch.zeros(I, H).double(), torch.zeros(H, I).double()
    cg[:, ::group] = cu[:, ::group] = cd[:, ::group] = 7.0
    cg[5, 3], cg[6, 4] = 7.0, 1.0
    cu[5, 3], cu[6, 4] = -7.0, 2.0
    cd[:30, 5] = torch.arange(30).double() % 8 - 4
    cd[:, 6] = 3.0
    x = torch.zeros(M, H).double()
    x[:, 4] = 32.0
    x[M // 2, 3] = inf
    y = dgf.ffn_fwd_w4(matrix(x, dtype), *(packed(c, 1.0, dtype, group) for c in (cg, cu, cd)))
    a = torch.zeros(M, I).double()
    a[:, 6] = 32.0 * 64.0
    want = a @ cd.T
    # every other row of gate and up has a code of 0 there: 0 times infinity
    want[M // 2] = nan
    assert torch.equal(y.cpu().nan_to_num(nan=12345.0), once(want, dtype).nan_to_num(nan=12345.0))
    if dtype == BF:  # finite inputs whose activation overflows
        x[M // 2, 3] = 2.0 ** 70
        y = dgf.ffn_fwd_w4(matrix(x, dtype), *(packed(c, 1.0, dtype, group) for c in (cg, cu, cd)))
        want = a @ cd.T
        want[M // 2] = torch.where(cd[:, 5] == 0, nan, torch.where(cd[:, 5] > 0, -inf, inf))
        assert torch.equal(y.cpu().nan_to_num(nan=12345.0), once(want, dtype).nan_to_num(nan=12345.0))
