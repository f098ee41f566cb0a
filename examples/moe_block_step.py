"""Training steps of a sequence-sharded mixture-of-experts block, from the
layer norm to the update with states in 8 bits.

A job of tp 2 x dp 2 ranks, simulated in one GPU's memory as everywhere in
this library.  The block is y = x + experts(norm(x)), the loss the mean square
of y - target.  Its parameters show three owners:

  norm.w, norm.b  PARTIAL_SUM   each tp rank normalises its part of the
                                sequence; the backward pass writes the part's
                                dw and db straight into the rank's buffer
  router          REPLICA_AVG   computed alike on every tp rank
  up, down        LOCAL_SHARD   a tp rank holds half of the experts and sorts
                                the tokens that go to them

A step: grs_layernorm_forward, grs_moe_sort / dispatch, the experts' products
(torch), grs_moe_combine; the same back; grs_reduce_all by owner and
grs_grad_norm_sq on the plan; grs_tensors_adamw8_step (or adamw_step) over the
plan's arrays; grs_gather_params.

    python examples/moe_block_step.py [--steps 40] [--states 8|32]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from gradient_reduction_sharded_gb300 import grs  # noqa: E402

TP, DP = 2, 2
TOKENS, HIDDEN, EXPERTS, TOP_K, FFN = 512, 256, 8, 2, 128
LOCAL = EXPERTS // TP  # experts of a tp rank
NAMES = ("norm.w", "norm.b", "router", "up", "down")
SHAPES = {"norm.w": (HIDDEN,), "norm.b": (HIDDEN,), "router": (EXPERTS, HIDDEN), "up": (EXPERTS, FFN, HIDDEN),
          "down": (EXPERTS, HIDDEN, FFN)}
OWNERS = {"norm.w": grs.GRS_PARTIAL_SUM, "norm.b": grs.GRS_PARTIAL_SUM, "router": grs.GRS_REPLICA_AVG,
          "up": grs.GRS_LOCAL_SHARD, "down": grs.GRS_LOCAL_SHARD}


def ptr(t):
    return t.data_ptr()


class Job:
    """Parameters, rank buffers and optimizer state of the simulated job."""

    def __init__(self, states: int = 8, seed: int = 0):
        dev = "cuda"
        g = torch.Generator(device=dev).manual_seed(seed)
        numels = [torch.Size(SHAPES[n]).numel() for n in NAMES]
        self.states = states
        self.plan = grs.grs_plan_create(numels, [OWNERS[n] for n in NAMES], TP * DP, TP, 1, DP, 25 << 20)
        info = grs.grs_plan_query(self.plan)
        n = self.n = info["n_state_pad"]
        # Where each tensor's gradient lies in a rank's buffer.
        self.place = []
        for i in range(len(NAMES)):
            t = grs.grs_tensor_info(self.plan, i)
            self.place.append((grs.grs_bucket_info(self.plan, t["bucket"])["rank_offset"] + t["bucket_offset"], t["per_rank"]))
        self.grads = [torch.zeros(info["n_rank_pad"], dtype=torch.bfloat16, device=dev) for _ in range(TP * DP)]
        self.acc = torch.zeros(n, device=dev)
        self.ws = torch.zeros(info["workspace_bytes"], dtype=torch.uint8, device=dev)
        self.norm = torch.zeros(1, dtype=torch.float64, device=dev)
        # The parameters, and the fp32 master in the plan's layout.
        std = {"norm.w": 0.0, "norm.b": 0.0, "router": 0.02, "up": HIDDEN ** -0.5, "down": FFN ** -0.5}
        values = [torch.randn(SHAPES[k], generator=g, device=dev) * std[k] + (k == "norm.w") for k in NAMES]
        self.master = torch.empty(n, device=dev)
        grs.grs_state_from_logical(self.plan, ptr(torch.cat([v.reshape(-1) for v in values])), ptr(self.master), self.stream())
        self.flat = self.master.to(torch.bfloat16)
        self.params = {k: torch.empty(SHAPES[k], dtype=torch.bfloat16, device=dev) for k in NAMES}
        self.gather()
        # The plan's arrays are a list of one tensor for the list's AdamW.
        self.list = grs.grs_tensors_create([n])
        li = grs.grs_tensors_query(self.list)
        table = lambda t: torch.tensor([ptr(t)], dtype=torch.int64, device=dev)  # noqa: E731
        self.acc_table, self.flat_table = table(self.acc), table(self.flat)
        ns, nb = li["n_state"], li["n_blocks"]
        self.master = torch.cat([self.master, torch.zeros(ns - n, device=dev)])  # the list rounds up to whole blocks
        if states == 8:
            self.state = [torch.zeros(ns, dtype=torch.uint8, device=dev), torch.zeros(nb, device=dev),
                          torch.zeros(ns, dtype=torch.uint8, device=dev), torch.zeros(nb, device=dev)]
        else:
            self.state = [torch.zeros(ns, device=dev), torch.zeros(ns, device=dev)]
        self.step = 0

    def stream(self):
        return torch.cuda.current_stream().cuda_stream

    def gather(self):
        grs.grs_gather_params(self.plan, ptr(self.flat), [ptr(self.params[k]) for k in NAMES], self.stream())

    def grad(self, rank: int, name: str) -> torch.Tensor:
        """The part of a rank's gradient buffer that is this tensor's."""
        off, per_rank = self.place[NAMES.index(name)]
        return self.grads[rank][off:off + per_rank]

    def update(self, lr: float, max_norm: float = 1.0):
        """Reduce by owner, clip by the global norm, AdamW, bf16 parameters."""
        self.step += 1
        st = self.stream()
        grs.grs_reduce_all(self.plan, [ptr(t) for t in self.grads], ptr(self.acc), 0, 1, ptr(self.ws), st)
        grs.grs_grad_norm_sq(self.plan, ptr(self.acc), 1, ptr(self.ws), 1, ptr(self.norm), st)
        hp = grs.make_adamw(lr, 0.9, 0.99, 1e-8, 0.0, max_norm, self.step, 1)
        if self.states == 8:
            grs.grs_tensors_adamw8_step(self.list, hp, self.step, ptr(self.norm), ptr(self.acc_table), grs.GRS_DTYPE_FP32,
                                        ptr(self.master), *(ptr(t) for t in self.state), ptr(self.flat_table), st)
        else:
            grs.grs_tensors_adamw_step(self.list, hp, ptr(self.norm), ptr(self.acc_table), grs.GRS_DTYPE_FP32, ptr(self.master),
                                       *(ptr(t) for t in self.state), ptr(self.flat_table), st)
        self.gather()

    def close(self):
        torch.cuda.synchronize()
        grs.grs_tensors_destroy(self.list)
        grs.grs_plan_destroy(self.plan)


def experts_forward(p, t, offsets, xs):
    """The products of tp rank t's experts on their rows (offsets: host list)."""
    mid = torch.zeros(xs.shape[0], FFN, dtype=torch.bfloat16, device="cuda")
    ys = torch.zeros_like(xs)
    for e in range(LOCAL):
        rows = slice(offsets[e], offsets[e + 1])
        mid[rows] = torch.relu(xs[rows] @ p["up"][t * LOCAL + e].T)
        ys[rows] = mid[rows] @ p["down"][t * LOCAL + e].T
    return mid, ys


def experts_backward(p, t, offsets, xs, mid, dys, d_up, d_down):
    """Gradients of the experts' weights (into the rank's buffer) and of their rows."""
    dxs = torch.zeros_like(xs)
    for e in range(LOCAL):
        rows = slice(offsets[e], offsets[e + 1])
        d_down[e] = dys[rows].T @ mid[rows]
        d_mid = (dys[rows] @ p["down"][t * LOCAL + e]) * (mid[rows] > 0)
        d_up[e] = d_mid.T @ xs[rows]
        dxs[rows] = d_mid @ p["up"][t * LOCAL + e]
    return dxs


def forward_backward(job: Job, dp: int, x: torch.Tensor, target: torch.Tensor) -> torch.Tensor:
    """The loss of one dp rank's tokens (a device scalar); gradients into its tp ranks' buffers."""
    p, st, dev = job.params, job.stream(), "cuda"
    half = TOKENS // TP
    bf16 = grs.GRS_DTYPE_BF16
    norm = grs.make_norm(half, HIDDEN, 1e-5, bf16, bf16, bf16)
    norm_ws = torch.empty(grs.grs_layernorm_workspace_bytes(norm), dtype=torch.uint8, device=dev)
    # Each tp rank normalises its part of the sequence; an all-gather would bring the parts together.
    h = torch.empty(TOKENS, HIDDEN, dtype=torch.bfloat16, device=dev)
    mean, rstd = torch.empty(TOKENS, device=dev), torch.empty(TOKENS, device=dev)
    for t in range(TP):
        part = slice(t * half, (t + 1) * half)
        grs.grs_layernorm_forward(norm, ptr(x[part]), ptr(p["norm.w"]), ptr(p["norm.b"]), ptr(h[part]), ptr(mean[part]), ptr(rstd[part]), st)
    # The router, alike on every tp rank.
    logits = h.float() @ p["router"].float().T
    top = logits.topk(TOP_K, 1)
    ids = top.indices.to(torch.int32).contiguous()
    weights = top.values.softmax(1).contiguous()
    # Each tp rank's experts on the tokens that go to them; an all-reduce would add the parts up.
    y = x.float()
    kept = []
    n = TOKENS * TOP_K
    for t in range(TP):
        moe = grs.make_moe(TOKENS, TOP_K, EXPERTS, t * LOCAL, (t + 1) * LOCAL, HIDDEN, bf16)
        offsets = torch.empty(LOCAL + 1, dtype=torch.int32, device=dev)
        row_slot, slot_row = (torch.empty(n, dtype=torch.int32, device=dev) for _ in range(2))
        ws = torch.empty(grs.grs_moe_workspace_bytes(moe), dtype=torch.uint8, device=dev)
        grs.grs_moe_sort(moe, ptr(ids), ptr(offsets), ptr(row_slot), ptr(slot_row), ptr(ws), st)
        xs = torch.zeros(n, HIDDEN, dtype=torch.bfloat16, device=dev)
        grs.grs_moe_dispatch(moe, ptr(h), ptr(slot_row), ptr(xs), st)
        off = offsets.tolist()
        mid, ys = experts_forward(p, t, off, xs)
        out = torch.empty(TOKENS, HIDDEN, dtype=torch.bfloat16, device=dev)
        grs.grs_moe_combine(moe, ptr(ys), ptr(slot_row), ptr(weights), ptr(out), st)
        y += out.float()
        kept.append((moe, off, slot_row, xs, mid, ys))
    diff = y - target.float()
    loss = diff.square().mean()
    dy = (diff * (2.0 / diff.numel())).to(torch.bfloat16)
    # Back.
    dh = torch.zeros(TOKENS, HIDDEN, device=dev)
    dweights = torch.zeros(TOKENS, TOP_K, device=dev)
    for t, (moe, off, slot_row, xs, mid, ys) in enumerate(kept):
        rank = dp * TP + t
        dys, dw = torch.zeros_like(ys), torch.empty(TOKENS, TOP_K, device=dev)
        grs.grs_moe_combine_backward(moe, ptr(dy), ptr(ys), ptr(slot_row), ptr(weights), ptr(dys), ptr(dw), st)
        dxs = experts_backward(p, t, off, xs, mid, dys, job.grad(rank, "up").view(LOCAL, FFN, HIDDEN), job.grad(rank, "down").view(LOCAL, HIDDEN, FFN))
        part = torch.empty(TOKENS, HIDDEN, dtype=torch.bfloat16, device=dev)
        grs.grs_moe_dispatch_backward(moe, ptr(dxs), ptr(slot_row), ptr(part), st)
        dh += part.float()
        dweights += dw  # 0 where the choice is another rank's
    d_top = weights * (dweights - (weights * dweights).sum(1, keepdim=True))
    d_logits = torch.zeros_like(logits).scatter_(1, top.indices, d_top)
    dh += d_logits @ p["router"].float()
    d_router = d_logits.T @ h.float()
    dh = dh.to(torch.bfloat16)
    dx = torch.empty_like(dh)
    for t in range(TP):
        rank, part = dp * TP + t, slice(t * half, (t + 1) * half)
        job.grad(rank, "router").copy_(d_router.reshape(-1))
        grs.grs_layernorm_backward(norm, ptr(dh[part]), ptr(x[part]), ptr(p["norm.w"]), ptr(mean[part]), ptr(rstd[part]), ptr(dx[part]),
                                   ptr(job.grad(rank, "norm.w")), ptr(job.grad(rank, "norm.b")), ptr(norm_ws), st)
    return loss


def data(seed: int):
    """Tokens of each dp rank and what the block shall make of them."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(DP, TOKENS, HIDDEN, generator=g, device="cuda").to(torch.bfloat16)
    mix = torch.randn(HIDDEN, HIDDEN, generator=torch.Generator(device="cuda").manual_seed(99), device="cuda") * HIDDEN ** -0.5
    return x, (x.float() + 0.5 * torch.relu(x.float() @ mix)).to(torch.bfloat16)


def train(steps: int, states: int = 8, lr: float = 3e-3):
    """Losses of `steps` steps on one batch, and the status of the plan's and the list's checks."""
    job = Job(states)
    x, target = data(1)
    losses = []
    for _ in range(steps):
        losses.append(torch.stack([forward_backward(job, d, x[d], target[d]) for d in range(DP)]).mean())
        job.update(lr)
    status = (grs.grs_check_device_errors(job.plan, job.stream()), grs.grs_tensors_check_device_errors(job.list, job.stream()))
    job.close()
    return [float(v) for v in losses], status


if __name__ == "__main__":
    a = argparse.ArgumentParser()
    a.add_argument("--steps", type=int, default=40)
    a.add_argument("--states", type=int, choices=(8, 32), default=8)
    a = a.parse_args()
    losses, status = train(a.steps, a.states)
    for i in range(0, a.steps, max(1, a.steps // 8)):
        print(f"step {i:4d}  loss {losses[i]:.5f}")
    print(f"last       loss {losses[-1]:.5f}  (states in {a.states} bits, device checks {status})")
