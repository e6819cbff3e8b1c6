"""Matrix products grouped by expert against FP64, over ragged rows.

Tolerance of an output: half a step of its type, and of its FP32 sum one rounding
of 2^-23 (the matrix core truncates) for every block of 8 of the K contraction
elements and each of the terms, relative to the sum of the products' magnitudes."""
import pytest
import torch

from deterministic_gated_ffn_amd import binding as dgf

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float16]
nan = float("nan")


def rand(gen, *shape, dtype, scale=1.0, pad=0):
    """Normal values in rows with a leading dimension of a multiple of 8 (and pad more); what lies between rows is NaN."""
    *lead, cols = shape
    buf = torch.full((*lead, (cols + 7) // 8 * 8 + pad), nan, dtype=dtype, device="cuda")
    v = buf[..., :cols]
    v.copy_(torch.randn(*shape, generator=gen, device="cuda") * scale)
    return v


def ints(*values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def reference(layout, A, B, off, rows, add=None):
    """(values, sums of magnitudes) in FP64; rows of no expert NaN."""
    R = rows.numel() if rows is not None else A.shape[0]
    where = rows.long() if rows is not None else torch.arange(R, device="cuda")
    if layout == "TN":
        R = A.shape[0]
        where = rows.long() if rows is not None else torch.arange(R, device="cuda")
        out = [[f(A[lo:hi].double()).t() @ f(B[where[lo:hi]].double()) for lo, hi in zip(off, off[1:])] for f in (torch.clone, torch.abs)]
        return torch.stack(out[0]), torch.stack(out[1])
    N = B.shape[1] if layout == "NT" else B.shape[2]
    v = torch.full((R, N), nan, dtype=torch.float64, device="cuda")
    s = v.clone()
    for e, (lo, hi) in enumerate(zip(off, off[1:])):
        v[lo:hi] = s[lo:hi] = 0
        for a, b in [(A, B)] + ([add] if add is not None else []):
            a, b = a[where[lo:hi]].double(), b[e].double()
            b = b.t() if layout == "NT" else b
            v[lo:hi] += a @ b
            s[lo:hi] += a.abs() @ b.abs()
    return v, s


def check(got, ref, mags, K, terms=1):
    live = ~torch.isnan(ref)
    tol = torch.finfo(got.dtype).eps / 2 * ref.abs() + (K / 8 + 8) * terms * 2.0 ** -23 * mags
    if got.dtype == torch.float16:
        tol += 2.0 ** -25  # half a step below its normal range
    bad = (live & ~((got.double() - ref).abs() <= tol)).sum().item()
    assert bad == 0, (bad, (got.double() - ref)[live].abs().max().item())


def make(layout, off, T, M, N, K, dtype, gen, pad=0):
    E, R = len(off) - 1, off[-1]
    if layout == "TN":
        return rand(gen, R, M, dtype=dtype, pad=pad), rand(gen, T, N, dtype=dtype, pad=pad)
    A = rand(gen, T, K, dtype=dtype, pad=pad)
    return A, rand(gen, E, *((N, K) if layout == "NT" else (K, N)), dtype=dtype, scale=K ** -0.5 if K else 1.0, pad=pad)


# offsets with empty experts at the ends and between, one row, 63 to 65 rows, several tiles, one expert only
RAGGED = [[0, 1], [0, 0, 1, 1, 3], [0, 63, 127, 192, 192], [0, 300, 300, 301, 813], [0] * 66 + [5, 70]]


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("layout", ["NT", "NN", "TN"])
@pytest.mark.parametrize("off", RAGGED, ids=lambda o: f"{len(o) - 1}x{o[-1]}")
@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (24, 17, 8), (100, 136, 63), (129, 300, 65), (264, 520, 200)])
def test_ragged_sizes(dtype, layout, off, M, N, K):
    gen = torch.Generator(device="cuda").manual_seed(M * 1000 + K)
    R = off[-1]
    T = max(1, R // 2)
    A, B = make(layout, off, T, M, N, K, dtype, gen, pad=8 * (K % 2))
    rows = torch.randint(0, T, (R,), generator=gen, device="cuda", dtype=torch.int32)
    got = dgf.gemm_grouped(layout, A, B, ints(*off), rows=rows)
    ref, mags = reference(layout, A, B, off, rows)
    check(got, ref, mags, R if layout == "TN" else K)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("layout", ["NT", "NN", "TN"])
def test_large_tiles(dtype, layout):
    """Enough tiles for the widest form, remainders of every size, no row list."""
    gen = torch.Generator(device="cuda").manual_seed(5)
    counts = [256, 1, 511, 130, 64, 0, 705, 320, 257, 192, 900, 1000]
    off = [0]
    for c in counts:
        off.append(off[-1] + c)
    A, B = make(layout, off, off[-1], 1032, 1300, 456, dtype, gen)
    got = dgf.gemm_grouped(layout, A, B, ints(*off))
    ref, mags = reference(layout, A, B, off, None)
    check(got, ref, mags, max(counts) if layout == "TN" else 456)


@pytest.mark.parametrize("layout,M,N,K,rows", [("NT", 0, 4000, 8, 1), ("NN", 0, 4000, 40, 1), ("TN", 520, 530, 0, 3),
                                               ("NT", 0, 9300, 8, 70)])
def test_many_tiles_each(layout, M, N, K, rows):
    """1024 experts of a few rows and many columns: 40 and more tiles for a workgroup."""
    gen = torch.Generator(device="cuda").manual_seed(8)
    E = 1024 if rows < 70 else 256
    off = list(range(0, E * rows + 1, rows))
    A, B = make(layout, off, E * rows, M, N, K, torch.bfloat16, gen)
    got = dgf.gemm_grouped(layout, A, B, ints(*off))
    assert torch.equal(got, dgf.gemm_grouped(layout, A, B, ints(*off)))
    for e in range(0, E, 8):  # (in parts: FP64 takes four times the memory)
        o = [x - off[e] for x in off[e:e + 9]]
        a, b = A[off[e]:off[e + 8]], (B[off[e]:off[e + 8]] if layout == "TN" else B[e:e + 8])
        ref, mags = reference(layout, a, b, o, None)
        check(got[e:e + 8] if layout == "TN" else got[off[e]:off[e + 8]], ref, mags, rows if layout == "TN" else K)


@pytest.mark.parametrize("layout", ["NT", "NN"])
@pytest.mark.parametrize("K", [0, 5, 64, 100, 513])
@pytest.mark.parametrize("listed", [False, True])
def test_second_term(layout, K, listed):
    gen = torch.Generator(device="cuda").manual_seed(K)
    off = [0, 70, 70, 333]
    A, B = make(layout, off, 333, 0, 200, K, torch.bfloat16, gen)
    A2, B2 = make(layout, off, 333, 0, 200, K, torch.bfloat16, gen, pad=16)
    rows = torch.randperm(333, generator=gen, device="cuda").int() if listed else None
    got = dgf.gemm_grouped(layout, A, B, ints(*off), rows=rows, add=(A2, B2))
    ref, mags = reference(layout, A, B, off, rows, (A2, B2))
    check(got, ref, mags, K, 2)
    if K == 0:
        assert not got.any()


@pytest.mark.parametrize("layout", ["NT", "NN"])
def test_rows_of_no_expert_stay(layout):
    """A range of the experts writes its own rows only, and nothing past its columns."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    off = [0, 40, 200, 230, 300]
    A, B = make(layout, off, 320, 0, 77, 96, torch.bfloat16, gen)
    full = torch.full((320, 88), 7.0, dtype=torch.bfloat16, device="cuda")
    out = full[:, :77]
    dgf.gemm_grouped(layout, A, B[1:3], ints(*off)[1:4], out=out)
    ref, mags = reference(layout, A, B, off, None)
    assert (full[:, 77:] == 7).all() and (out[:40] == 7).all() and (out[230:] == 7).all()
    check(out[40:230], ref[40:230], mags[40:230], 96)


def test_tn_sums_its_rows_only():
    """Rows of no expert, NaN here, are not read into a sum; an expert without rows gives +0."""
    gen = torch.Generator(device="cuda").manual_seed(2)
    A, B = rand(gen, 90, 50, dtype=torch.float16), rand(gen, 90, 60, dtype=torch.float16)
    for t in (A, B):
        t[:10], t[71:] = nan, nan
    off = [10, 30, 30, 71]
    got = dgf.gemm_grouped("TN", A, B, ints(*off))
    ref, mags = reference("TN", A, B, off, None)
    check(got, ref, mags, 41)
    assert (got[1].view(torch.int16) == 0).all()


@pytest.mark.parametrize("layout", ["NT", "NN", "TN"])
def test_no_rows(layout):
    A, B = torch.empty(0, 48, device="cuda").half(), torch.ones(3, 48, 48, device="cuda").half()
    off = ints(0, 0, 0, 0)
    if layout == "TN":
        got = dgf.gemm_grouped("TN", A, A, off, out=torch.ones(3, 48, 48, device="cuda").half())
        assert got.shape == (3, 48, 48) and not got.any()
    else:
        assert dgf.gemm_grouped(layout, A, B, off).shape == (0, 48)


@pytest.mark.parametrize("layout", ["NT", "NN", "TN"])
def test_a_row_does_not_depend_on_the_others(layout):
    """The same rows in other company, and the same call again, give the same bits."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    off = [0, 300, 700]
    A, B = make(layout, off, 700, 640, 512, 320, torch.bfloat16, gen)
    got = dgf.gemm_grouped(layout, A, B, ints(*off))
    assert torch.equal(got, dgf.gemm_grouped(layout, A, B, ints(*off)))
    if layout == "TN":
        alone = dgf.gemm_grouped("TN", A[300:], B[300:], ints(0, 400))
        assert torch.equal(alone[0], got[1])
    else:
        alone = dgf.gemm_grouped(layout, A[300:301], B[1:], ints(0, 1))
        assert torch.equal(alone[0], got[300])


@pytest.mark.parametrize("layout", ["NT", "TN"])
def test_offsets_and_lists_out_of_range(layout):
    """Whatever the device arrays hold, reads and writes stay within the operands."""
    gen = torch.Generator(device="cuda").manual_seed(4)
    A, B = make(layout, [0, 50, 100], 100, 40, 40, 64, torch.bfloat16, gen)
    rows = torch.arange(100, device="cuda", dtype=torch.int32)
    rows[3], rows[60] = -5, 1 << 30
    got = dgf.gemm_grouped(layout, A, B, ints(0, 50, 100), rows=rows)
    clean, at = rows.clone(), torch.tensor([3, 60], device="cuda")
    clean[at] = 0
    if layout == "TN":
        Z = A.clone()
        Z[at] = 0
        ref, mags = reference("TN", Z, B, [0, 50, 100], clean)
    else:
        ref, mags = reference("NT", A, B, [0, 50, 100], clean)
        ref[at], mags[at] = 0, 0
    check(got, ref, mags, 100)
    for off in ((-7, 50, 1 << 30), (90, 20, 50), (1 << 30, -(1 << 30), 60)):
        dgf.gemm_grouped(layout, A, B, ints(*off), rows=rows)
    torch.cuda.synchronize()


def test_list_into_a_matrix_past_4_gib():
    T, K = 300_000, 8200
    A = torch.zeros(T, K, dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(6)
    rows = ints(T - 1, 0, 270_000, 131_072)
    A[rows.long()] = rand(gen, 4, K, dtype=torch.bfloat16)
    B = rand(gen, 2, 24, K, dtype=torch.bfloat16, scale=K ** -0.5)
    ref, mags = reference("NT", A, B, [0, 2, 4], rows)
    check(dgf.gemm_grouped("NT", A, B, ints(0, 2, 4), rows=rows), ref, mags, K)
    D = rand(gen, 4, 24, dtype=torch.bfloat16)
    ref, mags = reference("TN", D, A, [0, 2, 4], rows)
    check(dgf.gemm_grouped("TN", D, A, ints(0, 2, 4), rows=rows), ref, mags, 4)


def test_other_stream():
    gen = torch.Generator(device="cuda").manual_seed(7)
    off = [0, 100, 256]
    A, B = make("NT", off, 256, 0, 128, 128, torch.bfloat16, gen)
    o = ints(*off)
    want = dgf.gemm_grouped("NT", A, B, o)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = dgf.gemm_grouped("NT", A, B, o, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got, want)
