"""Grouped products of two terms, in both types.  The inputs are small whole numbers, so every FP32 sum
is exact and the output is the exact value rounded once."""
import pytest
import torch

from deterministic_gated_ffn_amd import binding as dgf

pytestmark = pytest.mark.gpu
BF, FH = torch.bfloat16, torch.float16


def whole(gen, shape, dtype, most, pad=0):
    *lead, cols = shape
    buf = torch.full((*lead, (cols + 7) // 8 * 8 + pad), float("nan"), dtype=dtype, device="cuda")
    buf[..., :cols] = torch.randint(-most, most + 1, shape, generator=gen, device="cuda").to(dtype)
    return buf[..., :cols]


@pytest.mark.parametrize("dtype", [BF, FH], ids=str)
@pytest.mark.parametrize("layout", ["NT", "NN"])
@pytest.mark.parametrize("T,N,K,counts", [(1, 8, 1, [1]), (5, 33, 70, [0, 5, 0, 9]), (40, 130, 515, [64, 0, 3, 129, 1]),
                                          (700, 300, 96, [300, 5, 900, 0]), (2100, 513, 40, [4000, 3000]), (60, 1411, 1003, [2] * 30)])
def test_two_terms(dtype, layout, T, N, K, counts):
    gen = torch.Generator(device="cuda").manual_seed(T + N + K)
    E, R = len(counts), sum(counts)
    offsets = torch.tensor([0, *torch.tensor(counts).cumsum(0).tolist()], dtype=torch.int32, device="cuda")
    rows = torch.randint(0, T, (R,), generator=gen, device="cuda", dtype=torch.int32)
    rows[R // 2] = -1  # a row of zeros
    shape = (E, N, K) if layout == "NT" else (E, K, N)
    A, A2 = whole(gen, (T, K), dtype, 4, pad=8), whole(gen, (T, K), dtype, 4)
    B, B2 = whole(gen, shape, dtype, 4), whole(gen, shape, dtype, 4, pad=16)
    assert 2 * 16 * K < 2 ** 24
    c = dgf.gemm_grouped(layout, A, B, offsets, rows=rows, add=(A2, B2))
    want = torch.zeros(R, N, dtype=torch.float64, device="cuda")
    for e in range(E):
        r = slice(int(offsets[e]), int(offsets[e + 1]))
        for a, b in ((A, B), (A2, B2)):
            picked = a.double()[rows[r].long().clamp(min=0)] * (rows[r] >= 0)[:, None]
            want[r] += picked @ (b[e].double().t() if layout == "NT" else b[e].double())
    assert torch.equal(c, want.float().to(dtype))
    # the terms' order does not matter to whole numbers, and one term alone is the other's absence
    assert torch.equal(c, dgf.gemm_grouped(layout, A2, B2, offsets, rows=rows, add=(A, B)))
    one = dgf.gemm_grouped(layout, A, B, offsets, rows=rows).double() + dgf.gemm_grouped(layout, A2, B2, offsets, rows=rows).double()
    assert (one - want).abs().max() <= torch.finfo(dtype).eps * 16 * K * 2
