"""Routing of tokens to experts and the experts' outputs back to tokens: plans
equal to the definition's, weights and gradients against FP64.

Tolerances: probs and the gradient's P are exponentials (2 units of 2^-24 each,
and half a unit of the argument's rounding for every unit of |l| up to 32), an
FP32 sum over at most E / 64 + 6 steps and a division: (E / 64 + 48) 2^-24 of the
value.  A sum of k products of FP32 values is off by (k + 1) 2^-24 of their
magnitudes' sum, a dot product over H by (H / 512 + 16) 2^-24 of them."""
import math

import pytest
import torch

from deterministic_gated_ffn_amd import binding as dgf

pytestmark = pytest.mark.gpu
inf, nan = math.inf, math.nan
U = 2.0 ** -24
BF, FH, F32 = torch.bfloat16, torch.float16, torch.float32


def plan_of(logits, k, renorm):
    """The plan by definition, token by token on the host."""
    l = logits.detach().cpu().double().tolist()
    top = torch.finfo(F32).max
    M, E = len(l), logits.shape[1]
    ids, probs, lists = [], [], [[] for _ in range(E)]
    for m, row in enumerate(l):
        row = [-inf if math.isnan(v) else min(v, top) for v in row]
        order = sorted((e for e in range(E) if row[e] > -inf), key=lambda e: (-row[e], e))[:k]
        over = order if renorm else [e for e in range(E) if row[e] > -inf]
        den = sum(math.exp(row[e] - row[order[0]]) for e in over) if order else 1.0
        ids.append(order + [-1] * (k - len(order)))
        probs.append([math.exp(row[e] - row[order[0]]) / den for e in order] + [0.0] * (k - len(order)))
        for j, e in enumerate(order):
            lists[e].append(m * k + j)
    offsets, rows, pos = [0], [], [-1] * (M * k)
    for one in lists:
        for n in one:
            pos[n] = len(rows)
            rows.append(n // k)
        offsets.append(len(rows))
    rows += [-1] * (M * k - len(rows))
    return ids, probs, offsets, rows, pos


def check_plan(logits, k, renorm, **kw):
    got = dgf.moe_route(logits, k, renorm=renorm, **kw)
    M, E = logits.shape
    ids, probs, offsets, rows, pos = plan_of(logits, k, renorm)
    assert got.ids.tolist() == ids and got.offsets.tolist() == offsets
    assert got.rows.tolist() == rows and got.pos.view(-1).tolist() == pos
    want = torch.tensor(probs, dtype=torch.float64).view(M, k)
    err = (got.probs.cpu().double() - want).abs()
    assert (err <= (E / 64 + 48) * U * want + 2.0 ** -126).all(), err.max()
    return got


def logits_of(M, E, dtype, seed=0, pad=0):
    gen = torch.Generator().manual_seed(seed)
    t = torch.full((M, E + pad), nan, dtype=dtype)
    t[:, :E] = (torch.randn(M, E, generator=gen) * 2).to(dtype)
    return t.cuda()[:, :E]


@pytest.mark.parametrize("dtype", [BF, FH, F32], ids=str)
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("M,E,k", [(1, 1, 1), (1, 128, 8), (3, 5, 5), (63, 64, 16), (64, 65, 3), (65, 60, 4), (257, 128, 8),
                                   (1000, 200, 1), (300, 1000, 6), (5000, 8, 2)])
def test_plan(dtype, renorm, M, E, k):
    """16-bit logits tie often; 5000 tokens give a workgroup several tokens a wave."""
    check_plan(logits_of(M, E, dtype, seed=M + E, pad=E % 3), k, renorm)


@pytest.mark.parametrize("M", [9, 200])
@pytest.mark.parametrize("renorm", [True, False])
def test_masks_and_special_logits(M, renorm):
    l = logits_of(M, 70, F32, seed=3)
    l[0] = -inf                      # goes nowhere
    l[1, 3:] = -inf                  # fewer open experts than choices
    l[2] = nan
    l[3, 5], l[3, 60] = nan, nan
    l[4, 7], l[4, 66] = inf, inf     # two infinities share the token
    l[5] = 0.0
    l[5, ::2] = -0.0                 # one value: the lowest indices
    l[6] = torch.finfo(F32).min      # a finite mask still leaves an order
    l[6, 69] = 1.0
    l[7, :66] = -inf
    l[8] = torch.finfo(F32).max
    plan = check_plan(l, 4, renorm)
    assert plan.ids[0].tolist() == [-1] * 4 and plan.pos[0].tolist() == [-1] * 4 and not plan.probs[0].any()
    assert plan.ids[5].tolist() == [0, 1, 2, 3] and plan.ids[4, :2].tolist() == [7, 66]


@pytest.mark.parametrize("M", [40, 700])
def test_one_expert_takes_all(M):
    l = torch.zeros(M, 9, device="cuda")
    l[:, 4] = 1.0
    plan = check_plan(l, 1, True)
    assert plan.offsets.tolist() == [0] * 5 + [M] * 5
    none = check_plan(torch.full((M, 9), -inf, device="cuda"), 2, False)
    assert none.offsets.tolist() == [0] * 10 and (none.rows == -1).all()


def test_no_tokens():
    plan = dgf.moe_route(torch.empty(0, 12, device="cuda"), 3)
    assert plan.offsets.tolist() == [0] * 13 and plan.ids.shape == (0, 3) and plan.rows.shape == (0,)
    d = dgf.moe_route_bwd(plan.probs, torch.empty(0, 12, device="cuda"), plan.ids, plan.probs)
    assert d.shape == (0, 12)


def test_many_tokens():
    """Past what one token a wave covers, against the sort of torch."""
    M, E, k = 70001, 96, 6
    l = logits_of(M, E, BF, seed=8)
    plan = dgf.moe_route(l, k)
    top, ids = torch.sort(l.float(), dim=1, descending=True, stable=True)
    ids = ids[:, :k].reshape(-1)
    assert torch.equal(plan.ids.view(-1).long(), ids)
    key, order = torch.sort(ids, stable=True)
    assert torch.equal(plan.rows.long(), order // k)
    assert torch.equal(plan.pos.view(-1).long()[order], torch.arange(M * k, device="cuda"))
    assert torch.equal(plan.offsets.long(), torch.searchsorted(key, torch.arange(E + 1, device="cuda")))


@pytest.mark.parametrize("dtype", [BF, FH, F32], ids=str)
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("M,E,k", [(1, 1, 1), (5, 60, 4), (130, 128, 8), (33, 1000, 16)])
def test_gradient(dtype, renorm, M, E, k):
    """Against the formula's in FP64 (probs as the forward gave them), and differences of the definition."""
    l = logits_of(M, E, dtype, seed=E + k)
    if M > 4 and E > 8:
        l[1] = -inf
        l[2, 3:] = -inf
        l[3, 5] = nan
    plan = dgf.moe_route(l, k, renorm=renorm)
    gen = torch.Generator(device="cuda").manual_seed(1)
    dp = torch.randn(M, k, generator=gen, device="cuda")
    dp[plan.ids < 0] = nan  # the gradient of a weight that is not there is not read
    d = dgf.moe_route_bwd(dp, l, plan.ids, plan.probs, renorm=renorm)
    assert d.dtype == dtype and d.shape == (M, E)

    live = plan.ids >= 0
    at = torch.where(live, plan.ids, E).long()
    g = torch.zeros(M, E + 1, dtype=torch.float64, device="cuda").scatter_(1, at, torch.where(live, dp, 0.0).double())[:, :E]
    x = torch.nan_to_num(l.double(), nan=-inf, neginf=-inf)
    chosen = torch.zeros(M, E + 1, dtype=torch.bool, device="cuda").scatter_(1, at, True)[:, :E]

    def weights(x):
        e = torch.exp(x - x.amax(1, keepdim=True).clamp(min=-1e300))
        e = torch.where(chosen, e, 0.0) if renorm else e
        return e / e.sum(1, keepdim=True).clamp(min=1e-300)

    P = weights(x)
    want = P * (g - (P * g).sum(1, keepdim=True))
    size = P * (g.abs() + (P * g).abs().sum(1, keepdim=True))
    tol = torch.finfo(dtype).eps / 2 * want.abs() + 2 * (E / 64 + k + 48) * U * size + (2.0 ** -25 if dtype == FH else 2.0 ** -134)
    assert ((d.double() - want).abs() <= tol).all()
    # along a random direction, by central differences in FP64 (their own error: h^2, and rounding / h)
    v = torch.randn(M, E, generator=gen, device="cuda", dtype=torch.float64)
    h = 1e-4
    diff = ((weights(x + h * v) - weights(x - h * v)) * g).sum(1) / (2 * h)
    along = torch.where(want != 0, want * v, 0.0).sum(1)
    assert (diff - along).abs().max() < 1e-6 * (1 + g.abs().sum(1).max())


# ------------------------------------------------------------------ combine
def combine_case(M, H, k, dtype, R=None, pad=0, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    R = M * k if R is None else R

    def rows(n):
        buf = torch.full((n, (H + 7) // 8 * 8 + pad), nan, dtype=dtype, device="cuda")
        buf[:, :H] = torch.randn(n, H, generator=gen, device="cuda").to(dtype)
        return buf[:, :H]

    pos = torch.full((M * k,), -1, dtype=torch.int32, device="cuda")
    some = torch.randperm(M * k, generator=gen, device="cuda")[:min(R, M * k)]
    pos[some] = torch.randperm(R, generator=gen, device="cuda")[:some.numel()].int()
    return rows(R), pos.view(M, k), torch.rand(M, k, generator=gen, device="cuda"), rows(M)


@pytest.mark.parametrize("dtype", [BF, FH], ids=str)
@pytest.mark.parametrize("M,H,k,short", [(1, 1, 1, 0), (1, 2048, 8, 0), (7, 77, 3, 5), (33, 1003, 2, 0), (10, 4096, 4, 7),
                                         (5, 9000, 16, 11), (300, 512, 8, 100), (4, 120, 6, 24)])
def test_combine(dtype, M, H, k, short):
    """Some pairs without a row; an outsider among the positions; padding is NaN."""
    o, pos, probs, dy = combine_case(M, H, k, dtype, R=M * k - short, pad=8 * (M % 2), seed=H)
    if short:
        pos.view(-1)[(pos.view(-1) < 0).nonzero()[0]] = 1 << 30
    live = (pos >= 0) & (pos < o.shape[0])
    rows = torch.where(live, pos, 0).long()
    O = (o.double()[rows] if o.shape[0] else torch.zeros(M, k, H, device="cuda", dtype=torch.float64)) * live[..., None]
    half = torch.finfo(dtype).eps / 2
    tiny = 2.0 ** -25 if dtype == FH else 0.0
    for w in (probs, None):
        y = dgf.moe_combine(o, pos, w)
        W = (torch.ones_like(probs) if w is None else w).double()[..., None]
        want, size = (W * O).sum(1), (W * O).abs().sum(1)
        assert ((y.double() - want).abs() <= half * want.abs() + (k + 1) * U * size + tiny).all()
        d_o, dprobs = dgf.moe_combine_bwd(dy, o, pos, w)
        assert d_o.shape == o.shape
        D = (W * dy.double()[:, None]).expand(M, k, H)[live]
        assert ((d_o[pos[live].long()].double() - D).abs() <= (half + U) * D.abs() + tiny).all()
        if w is None:
            assert dprobs is None
            continue
        terms = dy.double()[:, None] * O
        assert ((dprobs.double() - terms.sum(2)).abs() <= (H / 512 + 16) * U * terms.abs().sum(2)).all()
        assert not dprobs[~live].any()


def test_combine_leaves_other_rows():
    lib = dgf.load()
    o, pos, probs, dy = combine_case(3, 64, 2, BF, R=10)
    d_o = torch.full((10, 64), 5.0, dtype=BF, device="cuda")
    dprobs = torch.empty(3, 2, device="cuda")
    st = lib.dgf_moe_combine_bwd(dy.data_ptr(), 64, o.data_ptr(), 64, 10, pos.data_ptr(), probs.data_ptr(), d_o.data_ptr(),
                                 64, dprobs.data_ptr(), 3, 64, 2, dgf.DGF_BF16, torch.cuda.current_stream().cuda_stream)
    assert st == 0
    other = torch.ones(10, dtype=torch.bool, device="cuda")
    other[pos.view(-1).long()] = False
    assert other.sum() == 4 and (d_o[other] == 5).all() and not (d_o[~other] == 5).all(1).any()


def test_combine_without_rows():
    """No expert took anything: zeros, whatever lies at o."""
    pos = torch.full((4, 2), -1, dtype=torch.int32, device="cuda")
    y = dgf.moe_combine(torch.empty(0, 32, dtype=BF, device="cuda"), pos, torch.ones(4, 2, device="cuda"))
    assert y.shape == (4, 32) and (y.view(torch.int16) == 0).all()


def test_captured_routing_follows_its_inputs():
    """A graph of routing and combination, replayed on new logits between eager calls."""
    M, E, k = 300, 60, 4
    l = logits_of(M, E, F32, seed=11)
    o = torch.randn(M * k, 96, device="cuda").to(BF)
    dgf.moe_combine(o, dgf.moe_route(l, k).pos)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        plan = dgf.moe_route(l, k)
        y = dgf.moe_combine(o, plan.pos, plan.probs)
    for seed in (21, 22, 23):
        l.copy_(logits_of(M, E, F32, seed=seed))
        o.normal_()
        g.replay()
        want = dgf.moe_route(l, k)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(plan, want))
        assert torch.equal(y, dgf.moe_combine(o, want.pos, want.probs))
