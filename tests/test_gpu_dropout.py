"""Dropout from a counter-based generator: the mask by the published algorithm in
numpy, values to one rounding (FP32 products and one sum before it)."""
import numpy as np
import pytest
import torch

from deterministic_gated_ffn_amd import binding as dgf

pytestmark = pytest.mark.gpu
BF, FH = torch.bfloat16, torch.float16


def philox(seed, step, n, first=0):
    """Philox-4x32-10 (Salmon et al. 2011) at counters {first..first+n-1, step}, [n, 4] words."""
    c = np.zeros((4, n), dtype=np.uint64)
    at = np.arange(first, first + n)
    c[0], c[1] = at & 0xFFFFFFFF, at >> 32
    c[2], c[3] = step & 0xFFFFFFFF, step >> 32 & 0xFFFFFFFF
    k0, k1 = seed & 0xFFFFFFFF, seed >> 32 & 0xFFFFFFFF
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        s = np.uint64(32)
        low = np.uint64(0xFFFFFFFF)
        c = np.stack([(b >> s) ^ c[1] ^ np.uint64(k0), b & low, (a >> s) ^ c[3] ^ np.uint64(k1), a & low])
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    return c.T.astype(np.uint32)


def test_oracle_known_answers():
    """The published vectors: counter and key of zeros, and of ones throughout."""
    assert philox(0, 0, 1)[0].tolist() == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]


def mask(M, H, p, seed, step):
    words = philox(seed, step, M * -(-H // 8))
    draws = np.stack([words & 0xFFFF, words >> 16], 2).reshape(M, -1)[:, :H]
    return torch.from_numpy(draws >= int(round(p * 65536))).cuda()


def rng_of(seed, step):
    return torch.tensor([seed, step], dtype=torch.int64, device="cuda")


def rows(M, H, dtype, seed, pad=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    buf = torch.full((M, (H + 7) // 8 * 8 + pad), float("nan"), dtype=dtype, device="cuda")
    buf[:, :H] = torch.randn(M, H, generator=gen, device="cuda").to(dtype)
    return buf[:, :H]


@pytest.mark.parametrize("dtype", [BF, FH], ids=str)
@pytest.mark.parametrize("M,H", [(1, 1), (1, 7), (3, 8), (5, 77), (129, 1003), (40, 16384)])
@pytest.mark.parametrize("p,alpha", [(0.0, None), (0.1, None), (0.5, 1.0), (0.25, 0.5), (65535 / 65536, 1.0)])
def test_values(dtype, M, H, p, alpha):
    seed, step = 0x7EDCBA9876543210, (3 << 40) + 5
    x = rows(M, H, dtype, 1, pad=8 * (M % 2))
    res = rows(M, H, dtype, 2) if alpha is not None else None
    z = dgf.dropout(x, p, rng_of(seed, step), res=res, alpha=1.0 if alpha is None else alpha)
    keep = mask(M, H, p, seed, step)
    cut = round(p * 65536)
    want = torch.where(keep, x.double() * (65536 / (65536 - cut)), 0.0)
    size = want.abs()
    if res is not None:
        want, size = want + alpha * res.double(), size + abs(alpha) * res.double().abs()
    tiny = 2.0 ** -25 if dtype == FH else 0.0
    fits = want.abs() < torch.finfo(dtype).max
    err = (z.double() - want).abs()
    assert (err <= torch.finfo(dtype).eps / 2 * want.abs() + 4 * 2.0 ** -24 * size + tiny)[fits].all()
    assert torch.isinf(z[~fits]).all()


def test_a_dropped_infinity_is_gone():
    x = torch.full((4, 64), float("inf"), dtype=BF, device="cuda")
    x[:, ::2] = float("nan")
    z = dgf.dropout(x, 0.5, rng_of(1, 2))
    keep = mask(4, 64, 0.5, 1, 2)
    assert (z[~keep] == 0).all() and not torch.isfinite(z[keep]).any()


def test_gradient_is_the_same_call():
    """z is linear in x: <dropout(x), d> = <x, dropout(d)>, the same mask in both."""
    x, d = rows(64, 256, FH, 3), rows(64, 256, FH, 4)
    r = rng_of(9, 1)
    z, dx = dgf.dropout(x, 0.3, r), dgf.dropout(d, 0.3, r)
    assert torch.equal(z == 0, dx == 0) or ((z == 0) ^ (dx == 0)).sum() == ((x == 0) ^ (d == 0)).sum()
    a, b = (z.double() * d.double()).sum(), (x.double() * dx.double()).sum()
    assert abs(a - b) <= 2 * 2.0 ** -11 * (z.double() * d.double()).abs().sum()


def test_rows_and_share():
    """The mask goes by row, column and step alone, and drops its share: 6 standard deviations of 2^20 draws."""
    x = torch.ones(1024, 1024, dtype=BF, device="cuda")
    one = dgf.dropout(x, 0.1, rng_of(5, 0))
    assert torch.equal(one[:100], dgf.dropout(x[:100], 0.1, rng_of(5, 0)))
    assert abs((one == 0).double().mean().item() - round(6553.6) / 65536) < 6 * (0.09 / 2 ** 20) ** 0.5
    for other in (rng_of(6, 0), rng_of(5, 1)):
        same = ((dgf.dropout(x, 0.1, other) == 0) & (one == 0)).double().mean().item()
        assert abs(same - 0.01) < 6 * (0.0099 / 2 ** 20) ** 0.5


def test_in_place():
    x, res = rows(33, 77, BF, 5), rows(33, 77, BF, 6)
    want = dgf.dropout(x, 0.2, rng_of(1, 1), res=res)
    for into in (x.clone(memory_format=torch.preserve_format), res):
        buf = torch.empty(33, 80, dtype=BF, device="cuda")[:, :77]
        buf.copy_(into)
        got = dgf.dropout(buf if into is not res else x, 0.2, rng_of(1, 1), res=buf if into is res else res, out=buf)
        assert got is buf and torch.equal(got, want)


def test_replays_draw_new_masks():
    """A captured call whose graph advances the step, against eager calls at the same steps."""
    x = rows(50, 300, BF, 7)
    r = rng_of(3, 100)
    inc = torch.tensor([0, 1], dtype=torch.int64, device="cuda")
    dgf.dropout(x, 0.4, r)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        z = dgf.dropout(x, 0.4, r)
        r.add_(inc)
    seen = []
    for n in range(4):
        g.replay()
        want = dgf.dropout(x, 0.4, rng_of(3, 100 + n))
        torch.cuda.synchronize()
        assert torch.equal(z, want)
        seen.append(z.clone())
    assert not torch.equal(seen[0], seen[1])


def test_more_than_2_to_the_32_pieces():
    """Rows on both sides of the 2^32nd piece of 8 values, in place: the mask goes on with the counter's second word."""
    M, H = 1 << 21, 16392
    x = torch.ones(M, H, dtype=BF, device="cuda")
    dgf.dropout(x, 0.5, rng_of(5, 6), out=x)
    per = H // 8
    for m in (0, (1 << 32) // per - 1, (1 << 32) // per, (1 << 32) // per + 1, M - 1):
        words = philox(5, 6, per, m * per)
        keep = torch.from_numpy((np.stack([words & 0xFFFF, words >> 16], 2).reshape(-1) >= 32768)).cuda()
        assert torch.equal(x[m], torch.where(keep, 2.0, 0.0).to(BF)), m
