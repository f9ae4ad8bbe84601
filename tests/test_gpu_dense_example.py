"""The fine-tuning example on the GPU: its gradients against 64-bit autograd of the same block, and
its loss falling."""
import os
import sys

import pytest
import torch

from dense_ref import d, half_step

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_gradients_of_the_block_against_autograd():
    import finetune
    T, H, I, E, k, V = 50, 128, 64, 6, 2, 301
    b = finetune.Block(H, I, E, k, V)
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.empty((T, H), dtype=torch.bfloat16, device="cuda").normal_(0, 1, generator=g)
    t = torch.randint(0, V, (T,), generator=g, device="cuda", dtype=torch.int32)
    t[::7] = -1
    dnll = torch.where(t >= 0, 1.0 / T, 0.0).float()
    nll, lse, saved = b.forward(x, t)
    grads = b.backward(lse, saved, dnll)
    w, groups = d(saved[2]), saved[3]
    off, slots = groups.offsets.cpu(), groups.slot_list.cpu().long()
    p = {n: d(v).requires_grad_() for n, v in b.params.items()}
    x64, y = d(x), torch.zeros((T, H), dtype=torch.float64)
    for e in range(E):
        s = slots[int(off[e]):int(off[e + 1])]
        xe = x64[s // k]
        h = torch.nn.functional.silu(xe @ p["gate"][e].T) * (xe @ p["up"][e].T)
        y = y.index_add(0, s // k, w.reshape(-1)[s][:, None] * (h @ p["down"][e].T))
    r = x64 + y
    o = r + torch.nn.functional.gelu(r @ p["proj"].T + p["bias"])
    keep = (t >= 0).cpu()
    ref = torch.nn.functional.cross_entropy((o @ p["head"].T)[keep], t.cpu().long()[keep], reduction="none")
    (ref.sum() / T).backward()
    # a value passes at most ten roundings to bf16 on its way (h, r, pre, o, ds, do, dz, dr, dy, dg),
    # each off by at most half a step of itself
    lim = 10 * half_step(torch.bfloat16)
    ref = ref.detach()
    got = d(nll)[keep]
    assert float((got - ref).norm() / ref.norm()) <= lim
    assert not nll[~keep.cuda()].any()
    for n, v in p.items():
        rel = float((d(grads[n]) - v.grad).norm() / v.grad.norm())
        assert rel <= lim, f"{n}: {rel}"


def test_the_example_learns():
    import finetune
    losses, one = finetune.train(steps=20, tokens=200, H=256, I=128, E=8, k=2, V=1003, log=None)
    assert all(l == l for l in losses)
    assert losses[-1] < 0.5 * losses[0], losses
