"""The mixture-of-experts block of examples/moe_block_step.py: its reduced
gradients against autograd on a plain model, and that training goes down with
states in 8 and in 32 bits."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ex():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    spec = importlib.util.spec_from_file_location("moe_block_step", os.path.join(ROOT, "examples", "moe_block_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def plain_gradients(ex, job, x, target):
    """Autograd in 64 bits, the mean over the dp ranks; the choices of experts as the block makes them."""
    p = {k: v.double().requires_grad_(True) for k, v in job.params.items()}
    loss = 0
    for d in range(ex.DP):
        v = x[d].double()
        h = (v - v.mean(1, keepdim=True)) / (v.var(1, correction=0, keepdim=True) + 1e-5).sqrt() * p["norm.w"] + p["norm.b"]
        rounded = h.to(torch.bfloat16).float() @ job.params["router"].float().T
        idx = rounded.topk(ex.TOP_K, 1).indices
        w = (h @ p["router"].T).gather(1, idx).softmax(1)
        y = v
        for j in range(ex.TOP_K):
            up, down = p["up"][idx[:, j]], p["down"][idx[:, j]]
            y = y + w[:, j:j + 1] * torch.einsum("tdf,tf->td", down, torch.relu(torch.einsum("tfd,td->tf", up, h)))
        loss = loss + (y - target[d].double()).square().mean() / ex.DP
    loss.backward()
    return float(loss.detach()), {k: v.grad for k, v in p.items()}


def test_reduced_gradients_are_those_of_the_block(ex):
    job = ex.Job(8)
    x, target = ex.data(1)
    loss = float(torch.stack([ex.forward_backward(job, d, x[d], target[d]) for d in range(ex.DP)]).mean())
    want_loss, want = plain_gradients(ex, job, x, target)
    job.update(0.0)
    logical = torch.empty(sum(v.numel() for v in want.values()), device="cuda")
    ex.grs.grs_state_to_logical(job.plan, job.acc.data_ptr(), logical.data_ptr(), job.stream())
    torch.cuda.synchronize()
    assert abs(loss / want_loss - 1) < 0.02
    at = 0
    for k in ex.NAMES:
        n = want[k].numel()
        got = logical[at:at + n].double().view(want[k].shape)
        at += n
        # activations, gradients and products in bf16: 2^-8 each, several in a row
        rel = float((got - want[k]).norm() / want[k].norm())
        assert rel < 0.03, (k, rel)
    job.close()


def test_training_goes_down_in_both_forms(ex):
    last = {}
    for states in (32, 8):
        losses, status = ex.train(40, states)
        assert status == (ex.grs.GRS_OK, ex.grs.GRS_OK)
        assert losses[-1] < 0.5 * losses[0], (states, losses[0], losses[-1])
        last[states] = losses[-1]
    assert last[8] < 1.25 * last[32]
