"""GPU: a mixture of experts trained in FP16, against FP64 autograd with the same choices and
the same dropout mask.

Every stage boundary is rounded to FP16: about 20 roundings (2^-11 each at most, adding in
quadrature: 0.22%) stay below 0.4% in the 2-norm; the router's gradient is a difference of two
sums of like size, twice that."""
import pytest
import torch

from deterministic_gated_ffn_amd import binding as dgf
from deterministic_gated_ffn_amd.block import MoeTrainBlock
from tests.test_gpu_experts_block import EPS, NAMES, layer64, make, off

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("M,H,I,E,k,p", [(37, 128, 200, 6, 2, 0.25), (300, 256, 320, 20, 4, 0.0), (500, 320, 264, 60, 8, 0.5)])
def test_training_step(M, H, I, E, k, p, renorm):
    w, x, dz = make(M, H, I, E, seed=1)
    w, x, dz = {n: t.half() for n, t in w.items()}, x.half(), dz.half()
    rng = torch.tensor([7, 3], device="cuda")
    block = MoeTrainBlock(**w, top_k=k, p_drop=p, renorm=renorm, eps=EPS)
    z, saved = block.forward(x, rng)
    grads = block.backward(dz, saved)
    ids = saved[4].ids.long().cpu()
    keep = dgf.dropout(torch.ones_like(x), p, rng).double().cpu()
    q = {n: t.double().cpu().requires_grad_() for n, t in {**w, "x": x}.items()}
    z64 = layer64(q, ids, keep, renorm)
    z64.backward(dz.double().cpu())
    assert z.dtype == torch.float16 and off(z, z64.detach()) <= 0.004
    for n, of in NAMES.items():
        assert grads[n].dtype == torch.float16
        assert off(grads[n], q[of].grad) <= (0.008 if n == "dw_router" else 0.004), (n, off(grads[n], q[of].grad))


def test_no_tokens():
    """A batch without tokens: nothing comes out, and the gradients of the weights are zeros."""
    w, x, dz = make(4, 64, 72, 6)
    block = MoeTrainBlock(**w, top_k=2, p_drop=0.1)
    rng = torch.tensor([1, 2], device="cuda")
    z, saved = block.forward(x[:0], rng)
    grads = block.backward(dz[:0], saved)
    assert z.shape == (0, 64) and grads["dx"].shape == (0, 64)
    assert all(grads[n].shape == w[of].shape and not grads[n].any() for n, of in NAMES.items() if of != "x")
