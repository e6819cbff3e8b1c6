"""GPU: a mixture of experts trained as block.py composes it, against FP64 autograd
with the same choices and the same dropout mask, captured in a HIP graph, and the
FFN served with 4-bit weights.

Every stage boundary is rounded to BF16: about 20 roundings (2^-9 in the mean
square each at most, adding in quadrature) stay below 3% in the 2-norm; the
router's gradient is a difference of two sums of like size, twice that."""
import pytest
import torch

from deterministic_gated_ffn_amd import binding as dgf
from deterministic_gated_ffn_amd.block import FfnBlock4, MoeTrainBlock

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
EPS = 1e-6


def rand(gen, *shape, scale=1.0, shift=0.0):
    return (torch.randn(shape, generator=gen) * scale + shift).to(BF).cuda()


def norm64(t, w):
    return t * torch.rsqrt(t.square().mean(-1, keepdim=True) + EPS) * w


def off(a, b):
    return ((a.double().cpu() - b).norm() / b.norm()).item()


def make(M, H, I, E, seed=0):
    gen = torch.Generator().manual_seed(seed)
    w = dict(w_in=rand(gen, H, scale=0.05, shift=1.0), w_router=rand(gen, E, H, scale=2 * H ** -0.5),
             w_gate=rand(gen, E, I, H, scale=H ** -0.5), w_up=rand(gen, E, I, H, scale=H ** -0.5),
             w_down=rand(gen, E, H, I, scale=I ** -0.5))
    return w, rand(gen, M, H), rand(gen, M, H, scale=0.1)


def layer64(q, ids, keep, renorm):
    """The layer in FP64 with these choices and this dropout factor."""
    h = norm64(q["x"], q["w_in"])
    chosen = torch.softmax(h @ q["w_router"].T, 1).gather(1, ids)
    probs = chosen / chosen.sum(1, keepdim=True) if renorm else chosen
    y = 0
    for j in range(ids.shape[1]):
        e = ids[:, j]
        g, u = (torch.einsum("mih,mh->mi", q[n][e], h) for n in ("w_gate", "w_up"))
        y = y + probs[:, j, None] * torch.einsum("mhi,mi->mh", q["w_down"][e], g * torch.sigmoid(g) * u)
    return q["x"] + keep * y


NAMES = {"dx": "x", "dw_in": "w_in", "dw_router": "w_router", "dW_gate": "w_gate", "dW_up": "w_up", "dW_down": "w_down"}


@pytest.mark.parametrize("renorm", [True, False])
def test_gradients_by_differences(renorm):
    """Each gradient along a random direction against central differences of the FP64 layer.
    An error of 3% (6% for the router) in the 2-norm is along a normal direction normal
    itself, of that deviation: 5 deviations.  The differences' own error, 1e-8 of it, is far below."""
    w, x, dz = make(40, 64, 72, 5, seed=4)
    rng = torch.tensor([3, 9], device="cuda")
    block = MoeTrainBlock(**w, top_k=2, p_drop=0.25, renorm=renorm, eps=EPS)
    _, saved = block.forward(x, rng)
    grads = block.backward(dz, saved)
    ids = saved[4].ids.long().cpu()
    keep = dgf.dropout(torch.ones_like(x), 0.25, rng).double().cpu()
    q = {n: t.double().cpu() for n, t in {**w, "x": x}.items()}
    gen = torch.Generator().manual_seed(5)
    for name, of in NAMES.items():
        v = torch.randn(q[of].shape, generator=gen, dtype=torch.float64)
        step = 1e-4
        up, down = ((dz.double().cpu() * layer64({**q, of: q[of] + s * v}, ids, keep, renorm)).sum() for s in (step, -step))
        d = grads[name].double().cpu()
        share = 0.06 if name == "dw_router" else 0.03
        assert abs((up - down) / (2 * step) - (d * v).sum()) <= 5 * share * d.norm(), name


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("M,H,I,E,k,p", [(1, 64, 72, 4, 2, 0.0), (37, 128, 200, 6, 2, 0.25), (300, 256, 320, 20, 4, 0.1),
                                         (700, 320, 264, 60, 8, 0.5)])
def test_training_step(M, H, I, E, k, p, renorm):
    w, x, dz = make(M, H, I, E)
    rng = torch.tensor([7, 3], device="cuda")
    block = MoeTrainBlock(**w, top_k=k, p_drop=p, renorm=renorm, eps=EPS)
    z, saved = block.forward(x, rng)
    grads = block.backward(dz, saved)
    ids = saved[4].ids.long().cpu()
    keep = dgf.dropout(torch.ones_like(x), p, rng).double().cpu()  # 0 or 1 / (1 - p)

    q = {n: t.double().cpu().requires_grad_() for n, t in {**w, "x": x}.items()}
    z64 = layer64(q, ids, keep, renorm)
    z64.backward(dz.double().cpu())
    assert off(z, z64.detach()) <= 0.03
    assert set(grads) == set(NAMES)
    for n, of in NAMES.items():
        assert grads[n].shape == q[of].shape
        want = q[of].grad
        if want.norm() == 0:  # one choice of one expert's weight: no gradient to the router
            assert grads[n].abs().max() < 1e-3
            continue
        assert off(grads[n], want) <= (0.06 if n == "dw_router" else 0.03), (n, off(grads[n], want))
    # experts without a token have a gradient of zeros
    idle = [e for e in range(E) if e not in set(ids.view(-1).tolist())]
    assert all(not grads[n][e].any() for e in idle for n in ("dW_gate", "dW_up", "dW_down"))
    again = block.backward(dz, block.forward(x, rng)[1])
    assert all(torch.equal(grads[n], again[n]) for n in grads)


def test_captured_step():
    """Forward and backward in one graph that advances the dropout's step, against eager steps."""
    w, x, dz = make(200, 128, 136, 10, seed=2)
    rng = torch.tensor([11, 0], device="cuda")
    one = torch.tensor([0, 1], device="cuda")
    block = MoeTrainBlock(**w, top_k=2, p_drop=0.2)

    def step(r):
        z, saved = block.forward(x, r)
        return {"z": z, **block.backward(dz, saved)}

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(rng)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(rng)
        rng.add_(one)
    for n in range(4):
        x.copy_(rand(torch.Generator().manual_seed(50 + n), 200, 128))
        graph.replay()
        want = step(torch.tensor([11, n], device="cuda"))
        torch.cuda.synchronize()
        for name in want:
            assert torch.equal(out[name], want[name]), (n, name)


def test_two_streams():
    """Two layers in flight at once on their own streams give what each gives alone."""
    sets = [make(150, 128, 264, 8, seed=s) for s in (5, 6)]
    rng = torch.tensor([1, 1], device="cuda")
    blocks = [MoeTrainBlock(**w, top_k=2, p_drop=0.1) for w, _, _ in sets]
    want = [b.backward(dz, b.forward(x, rng)[1]) for b, (_, x, dz) in zip(blocks, sets)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [None, None]
    for _ in range(3):
        for i, (b, (_, x, dz)) in enumerate(zip(blocks, sets)):
            got[i] = b.backward(dz, b.forward(x, rng, stream=streams[i])[1], stream=streams[i])
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(a[n], b[n]) for n in b)


@pytest.mark.parametrize("M", [1, 5, 40])
def test_served_in_4_bits(M):
    gen = torch.Generator().manual_seed(M)
    H, I = 256, 328
    w = [rand(gen, I, H, scale=H ** -0.5), rand(gen, I, H, scale=H ** -0.5), rand(gen, H, I, scale=I ** -0.5)]
    w_in, w_out, gate = rand(gen, H, scale=0.05, shift=1.0), rand(gen, H, scale=0.05, shift=1.0), rand(gen, H, shift=0.5)
    x = rand(gen, M, H)
    block = FfnBlock4(w_in, *w, w_out, group=32, gate=gate, alpha=0.9)
    z = block(x)
    d = lambda t: t.double().cpu()  # noqa: E731
    wg, wu, wd = (d(dgf.unpack4(p)) for p in block.w)
    h = norm64(d(x), d(w_in))
    g = h @ wg.T
    z64 = 0.9 * d(x) + d(gate) * norm64((g * torch.sigmoid(g) * (h @ wu.T)) @ wd.T, d(w_out))
    assert off(z, z64) <= 0.03


def test_the_example_runs(capsys):
    from deterministic_gated_ffn_amd import block
    block._demo(M=64, H=128, I=256, E=4, k=2)
    assert "4 bits" in capsys.readouterr().out
