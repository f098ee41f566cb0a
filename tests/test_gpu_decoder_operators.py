"""The operators of a decoder's parameters in a row, as a training step uses
them: embedding, layer norm, norms of queries and keys with rotation, tokens
sorted by expert, the experts' products, and back into the gradient buffers of
a rank; against autograd on a plain model in 64 bits.  Also: capture into a
graph as a process's first call, two streams at once, the checked build."""
import os
import re
import subprocess
import sys

import pytest
import torch

from operators_support import binding, ptr, stream

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")


def empty(*shape, dtype=BF):
    return torch.empty(*shape, dtype=dtype, device="cuda")


T, V, D, HQ, HK, HD, E, K, F = 320, 700, 256, 4, 2, 64, 6, 2, 192
SHAPES = {"embed": (V, D), "norm.w": (D,), "norm.b": (D,), "qkv": ((HQ + 2 * HK) * HD, D), "o": (D, HQ * HD), "q_norm": (HD,), "k_norm": (HD,),
          "up": (E, F, D), "down": (E, D, F)}


def causal(q, k, v):
    """Attention of grouped heads, [T, heads, HD]."""
    k, v = (x.repeat_interleave(HQ // HK, 1) for x in (k, v))
    s = torch.einsum("thd,shd->hts", q, k) * HD ** -0.5
    s = s.masked_fill(torch.ones(T, T, device="cuda").triu(1).bool(), float("-inf"))
    return torch.einsum("hts,shd->thd", s.softmax(-1), v)


def step(p, ids, pos, experts, weights, g_out, grads):
    """Forward and backward through the entry points; the parameters' gradients go to `grads`."""
    grs, st = binding(), stream()
    bf, f32 = grs.GRS_DTYPE_BF16, grs.GRS_DTYPE_FP32
    emb = grs.make_embedding(T, 0, V, D, D ** 0.5, bf, bf)
    norm = grs.make_norm(T, D, 1e-5, bf, bf, bf)
    wide = (HQ + 2 * HK) * HD
    qk = grs.make_qk_norm(T, HQ, HK, HD, HD, 1e-6, bf, bf, bf, ld_q=wide, ld_k=wide)
    moe = grs.make_moe(T, K, E, 0, E, D, bf)
    up, down = grs.make_experts(T * K, E, D, F, bf, bf), grs.make_experts(T * K, E, F, D, bf, bf)
    turns = torch.tensor(grs.grs_rope_turns([1e4 ** (-2 * i / HD) for i in range(HD // 2)]), dtype=torch.uint64, device="cuda")
    need = [grs.grs_embedding_workspace_bytes(emb), grs.grs_layernorm_workspace_bytes(norm), grs.grs_qk_norm_workspace_bytes(qk),
            grs.grs_moe_workspace_bytes(moe), grs.grs_experts_workspace_bytes(up), grs.grs_experts_workspace_bytes(down)]
    ws = torch.empty(max(need + [16]), dtype=torch.uint8, device="cuda")  # one for all: the calls follow one another

    x, h, mean, rstd = empty(T, D), empty(T, D), empty(T, dtype=torch.float32), empty(T, dtype=torch.float32)
    grs.grs_embedding_forward(emb, ptr(ids), ptr(p["embed"]), ptr(x), st)
    grs.grs_layernorm_forward(norm, ptr(x), ptr(p["norm.w"]), ptr(p["norm.b"]), ptr(h), ptr(mean), ptr(rstd), st)
    joint = h @ p["qkv"].T
    q, k = empty(T, HQ * HD), empty(T, HK * HD)
    kin = joint[:, HQ * HD:]
    grs.grs_qk_norm_forward(qk, ptr(joint), ptr(kin), ptr(p["q_norm"]), ptr(p["k_norm"]), ptr(pos), ptr(turns), ptr(q), ptr(k), st)
    att_in = [a.detach().float().requires_grad_(True) for a in (q.view(T, HQ, HD), k.view(T, HK, HD), joint[:, (HQ + HK) * HD:].reshape(T, HK, HD))]
    att = causal(*att_in)
    a = att.detach().reshape(T, -1).to(BF)
    y = a @ p["o"].T
    off, row_slot, slot_row = (empty(n, dtype=torch.int32) for n in (E + 1, T * K, T * K))
    xs, mid, ys, out = empty(T * K, D), empty(T * K, F), empty(T * K, D), empty(T, D)
    grs.grs_moe_sort(moe, ptr(experts), ptr(off), ptr(row_slot), ptr(slot_row), ptr(ws), st)
    grs.grs_moe_dispatch(moe, ptr(y), ptr(slot_row), ptr(xs), st)
    grs.grs_experts_forward(up, ptr(xs), ptr(p["up"]), ptr(off), ptr(mid), ptr(ws), st)
    act = mid.relu()
    grs.grs_experts_forward(down, ptr(act), ptr(p["down"]), ptr(off), ptr(ys), ptr(ws), st)
    grs.grs_moe_combine(moe, ptr(ys), ptr(slot_row), ptr(weights), ptr(out), st)

    dys, dweights, dact, dxs, dy = empty(T * K, D), empty(T * K, dtype=torch.float32), empty(T * K, F), empty(T * K, D), empty(T, D)
    grs.grs_moe_combine_backward(moe, ptr(g_out), ptr(ys), ptr(slot_row), ptr(weights), ptr(dys), ptr(dweights), st)
    grs.grs_experts_backward(down, ptr(dys), ptr(act), ptr(p["down"]), ptr(off), ptr(dact), ptr(grads["down"]), ptr(ws), st)
    dmid = dact * (mid > 0)
    grs.grs_experts_backward(up, ptr(dmid), ptr(xs), ptr(p["up"]), ptr(off), ptr(dxs), ptr(grads["up"]), ptr(ws), st)
    grs.grs_moe_dispatch_backward(moe, ptr(dxs), ptr(slot_row), ptr(dy), st)
    grads["o"].copy_(dy.float().T @ a.float())
    att.backward((dy @ p["o"]).float().view(T, HQ, HD))
    dq, dk, dv = (t.grad.reshape(T, -1).to(BF) for t in att_in)
    djoint = empty(T, wide)
    djoint[:, (HQ + HK) * HD:] = dv
    dkin = djoint[:, HQ * HD:]
    grs.grs_qk_norm_backward(qk, ptr(dq), ptr(dk), ptr(joint), ptr(kin), ptr(p["q_norm"]), ptr(p["k_norm"]), ptr(pos), ptr(turns), ptr(djoint), ptr(dkin),
                             ptr(grads["q_norm"]), ptr(grads["k_norm"]), ptr(ws), st)
    grads["qkv"].copy_(djoint.float().T @ h.float())
    dh, dx = djoint @ p["qkv"], empty(T, D)
    grs.grs_layernorm_backward(norm, ptr(dh), ptr(x), ptr(p["norm.w"]), ptr(mean), ptr(rstd), ptr(dx), ptr(grads["norm.w"]), ptr(grads["norm.b"]),
                               ptr(ws), st)
    grs.grs_embedding_backward(emb, ptr(ids), ptr(dx), ptr(grads["embed"]), ptr(ws), st)
    return out, dweights


def plain(p, ids, pos, experts, weights):
    x = p["embed"][ids.long()] * D ** 0.5
    h = (x - x.mean(1, keepdim=True)) / (x.var(1, correction=0, keepdim=True) + 1e-5).sqrt() * p["norm.w"] + p["norm.b"]
    q, k, v = (h @ p["qkv"].T).split([HQ * HD, HK * HD, HK * HD], 1)
    angle = pos.double()[:, None, None] * torch.tensor([1e4 ** (-2 * i / HD) for i in range(HD // 2)], dtype=torch.float64, device="cuda")

    def turned(x, w):
        x = x.reshape(T, -1, HD)
        u = x / (x.square().mean(-1, keepdim=True) + 1e-6).sqrt() * w
        a, b = u.chunk(2, -1)
        return torch.cat((a * angle.cos() - b * angle.sin(), a * angle.sin() + b * angle.cos()), -1)

    y = causal(turned(q, p["q_norm"]), turned(k, p["k_norm"]), v.reshape(T, HK, HD)).reshape(T, -1) @ p["o"].T
    out = 0
    for j in range(K):
        e = experts.view(T, K)[:, j].long()
        m = torch.relu(torch.einsum("tfd,td->tf", p["up"][e], y))
        out = out + weights.view(T, K)[:, j:j + 1] * torch.einsum("tdf,tf->td", p["down"][e], m)
    return out


def test_gradients_of_a_block_of_them_all():
    g = torch.Generator(device="cuda").manual_seed(4)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    p = {k: (rnd(*s) * (0.1 if k == "embed" else s[-1] ** -0.5) if len(s) > 1 else 1 + 0.1 * rnd(*s)).to(BF) for k, s in SHAPES.items()}
    ids = torch.randint(0, V, (T,), generator=g, device="cuda", dtype=torch.int32)
    ids[:90] = 5
    pos = (torch.arange(T, device="cuda") + 1000).to(torch.int32)
    experts = torch.stack([torch.randperm(E, generator=g, device="cuda")[:K] for _ in range(T)]).to(torch.int32).reshape(-1)
    weights = torch.rand(T * K, generator=g, device="cuda") + 0.2
    g_out = rnd(T, D).to(BF)
    grads = {k: torch.full(s, 7.0, dtype=BF, device="cuda") for k, s in SHAPES.items()}
    out, dweights = step(p, ids, pos, experts, weights, g_out, grads)
    grs = binding()
    assert grs.grs_operators_check_device_errors(stream()) == grs.GRS_OK
    p64 = {k: v.double().requires_grad_(True) for k, v in p.items()}
    w64 = weights.double().requires_grad_(True)
    want = plain(p64, ids, pos, experts, w64)
    want.backward(g_out.double())
    # Twelve tensors in a row are rounded to bf16 (2^-9 of their norm each on average, 2^-8 at most), forward and backward.
    rel = lambda a, b: float((a.double() - b).norm() / b.norm())  # noqa: E731
    assert rel(out, want.detach()) < 12 * 2.0 ** -8
    assert rel(dweights, w64.grad) < 12 * 2.0 ** -8
    for k in SHAPES:
        assert rel(grads[k], p64[k].grad) < 24 * 2.0 ** -8, k


CAPTURE = '''
import sys; sys.path[:0] = [%r, %r]
import torch
from operators_support import binding, ptr, stream
from test_gpu_experts import Case
from test_gpu_qk_norm import Case as Qk
from test_gpu_embedding import tokens
grs = binding()
c, q = Case([300, 0, 40], 264, 136, "bf16", "fp32"), Qk(50, 4, 2, 128, 128, "bf16", "bf16", "fp32")
ids = tokens(3000, 0, 900)
s = grs.make_embedding(3000, 0, 900, 64, 1.0, 0, 1)
ws = torch.empty(grs.grs_embedding_workspace_bytes(s), dtype=torch.uint8, device="cuda")
dy, dt = torch.randn(3000, 64, device="cuda").bfloat16(), torch.empty(900, 64, device="cuda")
def calls():
    grs.grs_embedding_backward(s, ptr(ids), ptr(dy), ptr(dt), ptr(ws), stream())
    return [c.forward(), *c.backward(), *q.forward(), *(t for p in q.backward() for t in p), dt]
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    out = calls()
graph.replay()
torch.cuda.synchronize()
got = [t.clone() for t in out]
for a, b in zip(got, calls()):
    assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
print("same")
'''


def test_capture_as_the_first_call_of_a_process():
    r = subprocess.run([sys.executable, "-c", CAPTURE % (ROOT, os.path.join(ROOT, "tests"))], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("same"), r.stdout[-2000:] + r.stderr[-2000:]


def test_two_streams_at_once():
    from test_gpu_embedding import tokens
    from test_gpu_experts import Case
    from test_gpu_qk_norm import Case as Qk
    grs = binding()
    cases = [(Case([900, 7, 0, 400], 520, 264, "bf16", "bf16", seed=i), Qk(2000, 8, 2, 64, 64, "bf16", "bf16", "fp32", seed=i)) for i in range(2)]
    emb = []
    for i in range(2):
        s = grs.make_embedding(20000, 0, 5000, 128, 1.0, grs.GRS_DTYPE_BF16, grs.GRS_DTYPE_FP32)
        emb.append((s, tokens(20000, 0, 5000, seed=i), torch.randn(20000, 128, device="cuda").bfloat16(), torch.empty(5000, 128, device="cuda"),
                    torch.empty(grs.grs_embedding_workspace_bytes(s), dtype=torch.uint8, device="cuda")))

    def calls(i):
        c, q = cases[i]
        s, ids, dy, dt, ws = emb[i]
        grs.grs_embedding_backward(s, ptr(ids), ptr(dy), ptr(dt), ptr(ws), stream())
        return [c.forward(), *c.backward(), *q.forward(), *(t for p in q.backward() for t in p), dt.clone()]

    want = [calls(0), calls(1)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = []
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got.append(calls(i))
        torch.cuda.synchronize()
        for a, b in zip(want[0] + want[1], got[0] + got[1]):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_suites_pass_on_the_checked_build():
    from gradient_reduction_sharded_gb300 import _build
    lib = _build.build_checked()
    r = subprocess.run([sys.executable, "-m", "pytest", "-x", "-q", "-p", "no:cacheprovider", "-m", "gpu", "tests/test_gpu_experts.py",
                        "tests/test_gpu_embedding.py", "tests/test_gpu_qk_norm.py"], cwd=ROOT, env=dict(os.environ, GRS_LIBRARY=lib),
                       capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, r.stdout[-4000:] + r.stderr[-2000:]
    m = re.search(r"(\d+) passed", r.stdout)
    assert m and int(m.group(1)) >= 200, r.stdout[-2000:]
