"""GPU: the FFN half of a layer (block.py) put together from the library's calls,
against the same layer in FP64 and its gradient by differences, and captured in
a HIP graph.

The layer rounds to the stored type at every stage boundary and keeps g and u in
8 bits, so it is compared in the 2-norm: about 20 roundings of BF16 (2^-9 in the
mean square each at most, adding in quadrature) and the checkpoint's steps (0.6%
of g and u) stay below 3%."""
import pytest
import torch

from deterministic_gated_ffn_amd import binding as dgf
from deterministic_gated_ffn_amd.block import FfnBlock, MoeBlock

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible: the GPU tests need an MI355X")
    dgf.load()


def rand(gen, *shape, scale=1.0, shift=0.0):
    return (torch.randn(shape, generator=gen) * scale + shift).to(BF).cuda()


def norm64(t, w):
    return t * torch.rsqrt(t.square().mean(-1, keepdim=True) + EPS) * w


def ffn64(h, wg, wu, wd):
    g = h @ wg.T
    return (g * torch.sigmoid(g) * (h @ wu.T)) @ wd.T


def make(M, H, I, seed=0):
    gen = torch.Generator().manual_seed(seed)
    w = dict(w_in=rand(gen, H, scale=0.05, shift=1.0), w_gate=rand(gen, I, H, scale=0.05),
             w_up=rand(gen, I, H, scale=0.05), w_down=rand(gen, H, I, scale=0.05),
             w_out=rand(gen, H, scale=0.05, shift=1.0), gate=rand(gen, H, scale=0.1, shift=0.5))
    return w, rand(gen, M, H), rand(gen, M, H, scale=0.1)


def off(a, b):
    return ((a.double().cpu() - b).norm() / b.norm()).item()


@pytest.mark.parametrize("M,H,I", [(1, 256, 640), (24, 512, 768), (160, 320, 520)])
def test_training_step(M, H, I):
    w, x, dz = make(M, H, I)
    block = FfnBlock(**w, alpha=0.9, eps=EPS)
    z, saved = block.forward(x)
    grads = block.backward(dz, saved)
    p = {k: t.double().cpu().requires_grad_() for k, t in {**w, "x": x}.items()}
    z64 = 0.9 * p["x"] + p["gate"] * norm64(ffn64(norm64(p["x"], p["w_in"]), p["w_gate"], p["w_up"], p["w_down"]), p["w_out"])
    z64.backward(dz.double().cpu())
    assert off(z, z64.detach()) <= 0.03
    names = {"dx": "x", "dw_in": "w_in", "dw_out": "w_out", "dgate": "gate", "dW_gate": "w_gate", "dW_up": "w_up",
             "dW_down": "w_down"}
    assert set(grads) == set(names)
    for k, n in names.items():
        assert off(grads[k], p[n].grad) <= 0.03, (k, off(grads[k], p[n].grad))
    # the step is the calls' own bits, run to run
    again = block.backward(dz, block.forward(x)[1])
    assert all(torch.equal(grads[k], again[k]) for k in grads)


def test_served_batch():
    M, H, I, E, k = 6, 256, 192, 12, 3
    w, x, _ = make(M, H, I, seed=2)
    gen = torch.Generator().manual_seed(3)
    wr, wg, wu, wd = (rand(gen, *s, scale=0.05) for s in ((E, H), (E, I, H), (E, I, H), (E, H, I)))
    w_next = rand(gen, H, scale=0.05, shift=1.0)
    z, h = MoeBlock(w["w_in"], wr, wg, wu, wd, w["w_out"], k, gate=w["gate"], eps=EPS)(x, w_next=w_next)
    d = lambda t: t.double().cpu()  # noqa: E731
    hin = norm64(d(x), d(w["w_in"])).to(BF).double()  # the block's input is rounded once; the routing follows it
    top, ids = (hin @ d(wr).T).topk(k, dim=1)
    p = torch.softmax(top, 1)
    y = torch.stack([sum(p[m, j] * ffn64(hin[m], d(wg)[e], d(wu)[e], d(wd)[e]) for j, e in enumerate(ids[m].tolist()))
                     for m in range(M)])
    z64 = d(x) + d(w["gate"]) * norm64(y, d(w["w_out"]))
    assert off(z, z64) <= 0.03
    assert off(h, norm64(z64, d(w_next))) <= 0.03


def test_training_step_replays_from_a_hip_graph():
    w, x, dz = make(96, 256, 384, seed=4)
    block = FfnBlock(**w, eps=EPS)

    def step():
        z, saved = block.forward(x)
        return {"z": z, **block.backward(dz, saved)}

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    gen = torch.Generator().manual_seed(5)
    for i in range(4):
        x.copy_(rand(gen, 96, 256))
        dz.copy_(rand(gen, 96, 256, scale=0.1))
        graph.replay()
        eager = step()
        torch.cuda.synchronize()
        for k in eager:
            assert torch.equal(out[k], eager[k]), (i, k)


def test_explicit_stream():
    w, x, dz = make(40, 256, 384, seed=6)
    block = FfnBlock(**w, eps=EPS)
    z, saved = block.forward(x)
    want = block.backward(dz, saved)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    z2, saved2 = block.forward(x, stream=side)
    got = block.backward(dz, saved2, stream=side)
    side.synchronize()
    assert torch.equal(z, z2)
    for k in want:
        assert torch.equal(want[k], got[k]), k
