"""What the operators of a mixture-of-experts decoder's remaining parameters
cost: the products of the experts with rows sorted by expert (LOCAL_SHARD
weights), the embedding (a replicated or vocabulary-sharded table) and the
norms of queries and keys with the position rotation (PARTIAL_SUM weights),
each forward and backward.

`own` selects the side `run` takes: the plain form in elementary torch
operations, or the framework's entry points.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
ESIZE = {"bf16": 2, "fp32": 4}
EPS = 1e-6
BASE = 1e6  # of the rotation's frequencies


# ------------------------------------------------------------------- cases

def listed():
    return [
        # One decoding step: 5 tokens x 4 choices over the 32 experts of the MoE workload, gate or up product: latency.
        {"name": "experts_fwd_few", "op": "experts_fwd", "rows": 20, "tail": 0, "experts": 32, "in": 2048, "out": 768, "act": "bf16"},
        # A microbatch of 16384 tokens x 8 choices, the same product.
        {"name": "experts_fwd_batch", "op": "experts_fwd", "rows": 131072, "tail": 0, "experts": 32, "in": 2048, "out": 768, "act": "bf16"},
        # Widths that divide nothing, a rank with 12 of the experts (the rows behind theirs are other ranks'), gradients in fp32.
        {"name": "experts_bwd_odd", "op": "experts_bwd", "rows": 3001, "tail": 1503, "experts": 12, "in": 1027, "out": 519, "act": "bf16", "grad": "fp32"},
        # Backward of an uneven microbatch through the down product, weights' gradients in the rank buffer's bf16.
        {"name": "experts_bwd_batch", "op": "experts_bwd", "rows": 36006, "tail": 0, "experts": 32, "in": 768, "out": 2048, "act": "bf16", "grad": "bf16"},
        # The new tokens of 7 sequences, the MoE workload's table: latency.
        {"name": "embed_fwd_token", "op": "embed_fwd", "tokens": 7, "vocab": 151936, "begin": 0, "end": 151936, "hidden": 2048, "act": "bf16", "scaled": False, "none": 0.0},
        # A microbatch of 16 sequences of 2048 tokens, vectors scaled by sqrt(d).
        {"name": "embed_fwd_batch", "op": "embed_fwd", "tokens": 32768, "vocab": 151936, "begin": 0, "end": 151936, "hidden": 2048, "act": "bf16", "scaled": True, "none": 0.0},
        # A vocabulary-sharded table of odd sizes in fp32, a third of the batch padding.
        {"name": "embed_bwd_odd", "op": "embed_bwd", "tokens": 3001, "vocab": 9973, "begin": 4987, "end": 9973, "hidden": 519, "act": "fp32", "grad": "fp32", "scaled": True, "none": 0.3},
        # Backward of a microbatch of 16384 tokens, the whole table's gradient in the rank buffer's bf16.
        {"name": "embed_bwd_batch", "op": "embed_bwd", "tokens": 16384, "vocab": 151936, "begin": 0, "end": 151936, "hidden": 2048, "act": "bf16", "grad": "bf16", "scaled": False, "none": 0.0},
        # One new token far into a sequence, 16 + 16 heads of 128 (the MoE workload's attention): latency.
        {"name": "qk_fwd_token", "op": "qk_fwd", "tokens": 1, "q_heads": 16, "k_heads": 16, "dim": 128, "rot": 128, "pairs": False, "far": 1000000, "act": "bf16", "par": "bf16", "packed": True},
        # A microbatch of 16384 tokens of the same attention, queries and keys inside the joint projection's rows.
        {"name": "qk_fwd_batch", "op": "qk_fwd", "tokens": 16384, "q_heads": 16, "k_heads": 16, "dim": 128, "rot": 128, "pairs": False, "far": 0, "act": "bf16", "par": "bf16", "packed": True},
        # Heads of 80 with 40 of them rotated in neighbouring pairs, fp32, a ragged number of tokens.
        {"name": "qk_bwd_odd", "op": "qk_bwd", "tokens": 1531, "q_heads": 5, "k_heads": 1, "dim": 80, "rot": 40, "pairs": True, "far": 4000, "act": "fp32", "par": "fp32", "grad": "fp32", "packed": False},
        # Backward with grouped heads: 32 query and 4 key heads of 64, as the 1.1B decoder has them.
        {"name": "qk_bwd_batch", "op": "qk_bwd", "tokens": 16384, "q_heads": 32, "k_heads": 4, "dim": 64, "rot": 64, "pairs": False, "far": 0, "act": "bf16", "par": "bf16", "grad": "bf16", "packed": True},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["experts_fwd", "experts_bwd", "embed_fwd", "embed_bwd", "qk_fwd", "qk_bwd"])
    act = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    grad = rng.choice(["bf16", "fp32"]) if act == "bf16" else "fp32"
    while True:
        if op.startswith("experts"):
            width = lambda: _log(rng, 8, 1024) * 8 + rng.choice([0, 0, 0, 0, 3, 4])  # noqa: E731
            rows = _log(rng, 1, 131072)
            c = {"op": op, "rows": rows, "tail": rng.choice([0, 0, rows // 3]), "experts": _log(rng, 1, 128), "in": width(), "out": width(), "act": act}
            # fp32 is for small models and for checks.
            most = (1e10 if act == "fp32" else 4e11, 1e9)
            if c["experts"] * c["in"] * c["out"] > 4e8:
                continue
        elif op.startswith("embed"):
            vocab = _log(rng, 50, 151936)
            begin = rng.choice([0, 0, vocab // 2])
            c = {"op": op, "tokens": _log(rng, 1, 65536), "vocab": vocab, "begin": begin, "end": vocab, "hidden": _log(rng, 8, 512) * 8 + rng.choice([0, 0, 0, 3]),
                 "act": act, "scaled": rng.choice([True, False]), "none": rng.choice([0.0, 0.0, 0.4])}
            most = (math.inf, 2.6e8 if op == "embed_fwd" else 6.5e8)
        else:
            dim = rng.choice([32, 64, 64, 80, 96, 128, 128, 192, 256])
            heads = _log(rng, 1, 8)
            c = {"op": op, "tokens": _log(rng, 1, 65536), "q_heads": heads * rng.choice([1, 2, 4, 8]), "k_heads": heads, "dim": dim,
                 "rot": rng.choice([dim, dim, dim // 2, 0]), "pairs": rng.choice([False, False, True]), "far": rng.choice([0, 0, 100000, 2000000]),
                 "act": act, "par": rng.choice(["bf16", "fp32"]) if act == "bf16" else "fp32", "packed": rng.choice([True, False])}
            most = (math.inf, 2.6e8 if op == "qk_fwd" else 2.2e8)
        if op.endswith("bwd"):
            c["grad"] = grad
        w = work(c)
        if w["flops"] <= most[0] and w["bytes"] <= most[1]:
            return c


def work(case):
    op, e = case["op"], ESIZE[case["act"]]
    if op.startswith("experts"):
        m, k, n = case["rows"], case["in"], case["out"]
        some = min(case["experts"], m) * k * n  # weights that are read: at most an expert a row
        if op == "experts_fwd":
            return {"bytes": (m * k + m * n + some) * e + 4 * (case["experts"] + 1), "flops": 2 * m * k * n}
        # dys and xs in, weights in; dxs out, every weight's gradient out
        return {"bytes": (2 * m * k + m * n + some) * e + case["experts"] * k * n * ESIZE[case["grad"]] + 4 * (case["experts"] + 1), "flops": 4 * m * k * n}
    if op.startswith("embed"):
        t, d, share = case["tokens"], case["hidden"], (case["end"] - case["begin"]) / case["vocab"] * (1 - case["none"])
        if op == "embed_fwd":  # a vector in for every token of this table, one out for each token
            return {"bytes": int((1 + share) * t * d * e + 4 * t), "flops": t * d}
        return {"bytes": int(share * t * d * e + 4 * t + (case["end"] - case["begin"]) * d * ESIZE[case["grad"]]), "flops": 2 * int(share * t * d)}
    n, d = case["tokens"] * (case["q_heads"] + case["k_heads"]) * case["dim"], case["dim"]
    if op == "qk_fwd":
        return {"bytes": 2 * n * e + 4 * case["tokens"] + 2 * d * ESIZE[case["par"]], "flops": 10 * n}
    return {"bytes": 3 * n * e + 4 * case["tokens"] + 2 * d * (ESIZE[case["par"]] + ESIZE[case["grad"]]), "flops": 20 * n}


# ------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(shape, std, g, dtype):
    return torch.randn(shape, generator=g, device="cuda").mul_(std).to(dtype)


def _experts_inputs(case, seed):
    g = _gen(seed)
    m, n_e, k, n, act = case["rows"], case["experts"], case["in"], case["out"], DT[case["act"]]
    all_rows = m + case["tail"]
    # Uneven experts, as a router without balance fills them; some may be empty.
    ids = torch.multinomial(torch.randn(n_e, generator=g, device="cuda").softmax(0), m, replacement=True, generator=g)
    offsets = torch.zeros(n_e + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = torch.bincount(ids, minlength=n_e).cumsum(0)
    s = {"case": case, "offsets": offsets, "xs": _normal((all_rows, k), 1.0, g, act), "w": _normal((n_e, n, k), k ** -0.5, g, act),
         "bounds": offsets.tolist()}
    if case["op"] == "experts_fwd":
        s["ys"] = torch.zeros(all_rows, n, dtype=act, device="cuda")
    else:
        s["dys"] = _normal((all_rows, n), 1e-2, g, act)
        s["dxs"] = torch.zeros_like(s["xs"])
        s["dw"] = torch.zeros(s["w"].shape, dtype=DT[case["grad"]], device="cuda")
    return s


def _embed_inputs(case, seed):
    g = _gen(seed)
    t, v, d, act = case["tokens"], case["vocab"], case["hidden"], DT[case["act"]]
    # Token frequencies fall as 1 / rank; ids in no order of frequency. -1: padding, no token of any table.
    rank = torch.rand(t, generator=g, device="cuda", dtype=torch.float64).mul_(math.log(v + 1)).exp_().long().sub_(1).clamp_(0, v - 1)
    ids = torch.randperm(v, generator=g, device="cuda")[rank].to(torch.int32)
    ids[torch.rand(t, generator=g, device="cuda") < case["none"]] = -1
    s = {"case": case, "ids": ids, "scale": torch.tensor(math.sqrt(d) if case["scaled"] else 1.0).item()}  # an fp32 number
    if case["op"] == "embed_fwd":
        s["table"] = _normal((case["end"] - case["begin"], d), 0.02, g, act)
    else:
        s["dy"] = _normal((t, d), 1e-2, g, act)
    return s


def _qk_inputs(case, seed):
    g = _gen(seed)
    t, d, act, par = case["tokens"], case["dim"], DT[case["act"]], DT[case["par"]]
    q, k = case["q_heads"] * d, case["k_heads"] * d
    wide = q + 2 * k if case["packed"] else 0  # queries, keys and values in one row

    def both(std):
        joint = _normal((t, wide or q + k), std, g, act)
        a, b = joint[:, :q], joint[:, q:q + k]
        return (a, b) if wide else (a.contiguous(), b.contiguous())

    s = {"case": case}
    s["q"], s["k"] = both(2.0)
    s["wq"], s["wk"] = ((1 + 0.1 * torch.randn(d, generator=g, device="cuda")).to(par) for _ in range(2))
    # A few sequences one behind the other, from `far` on.
    first = torch.randint(1, max(2, t // 3), (1,), generator=g, device="cuda")
    s["pos"] = ((torch.arange(t, device="cuda") % first) + case["far"]).to(torch.int32)
    r = case["rot"]
    s["inv_freq"] = torch.tensor([BASE ** (-2 * i / r) for i in range(r // 2)], dtype=torch.float64, device="cuda")
    if case["op"] == "qk_bwd":
        s["dqo"], s["dko"] = _normal((t, q), 1e-2, g, act), _normal((t, k), 1e-2, g, act)
    return s


def _inputs(case, seed):
    op = case["op"]
    return (_experts_inputs if op.startswith("experts") else _embed_inputs if op.startswith("embed") else _qk_inputs)(case, seed)


def prepare(case, seed):
    s = _inputs(case, seed)
    if not own:
        return s
    from gradient_reduction_sharded_gb300 import grs
    dt = {"bf16": grs.GRS_DTYPE_BF16, "fp32": grs.GRS_DTYPE_FP32}
    act, grad = dt[case["act"]], dt[case.get("grad", "fp32")]
    op = case["op"]
    if op.startswith("experts"):
        s["shape"] = grs.make_experts(case["rows"] + case["tail"], case["experts"], case["in"], case["out"], act, grad)
        size = grs.grs_experts_workspace_bytes(s["shape"])
    elif op.startswith("embed"):
        s["shape"] = grs.make_embedding(case["tokens"], case["begin"], case["end"], case["hidden"], s["scale"], act, grad)
        size = grs.grs_embedding_workspace_bytes(s["shape"])
        rows = case["tokens"] if op == "embed_fwd" else case["end"] - case["begin"]
        s["out"] = torch.empty(rows, case["hidden"], dtype=DT[case["act"] if op == "embed_fwd" else case["grad"]], device="cuda")
    else:
        q, k = s["q"], s["k"]
        s["shape"] = grs.make_qk_norm(case["tokens"], case["q_heads"], case["k_heads"], case["dim"], case["rot"], EPS, act, dt[case["par"]], grad,
                                      interleaved=case["pairs"], ld_q=q.stride(0), ld_k=k.stride(0), ld_qo=q.shape[1], ld_ko=k.shape[1])
        size = grs.grs_qk_norm_workspace_bytes(s["shape"])
        s["turns"] = torch.tensor(grs.grs_rope_turns(s["inv_freq"].tolist()), dtype=torch.uint64, device="cuda")
        if op == "qk_fwd":
            s["qo"], s["ko"] = (torch.empty(x.shape, dtype=x.dtype, device="cuda") for x in (q, k))
        else:
            # The gradients go where queries and keys lie in the joint projection's gradient.
            s["dq"], s["dk"] = (torch.empty_strided(x.shape, x.stride(), dtype=x.dtype, device="cuda") for x in (q, k))
            s["dwq"], s["dwk"] = (torch.empty(case["dim"], dtype=DT[case["grad"]], device="cuda") for _ in range(2))
    s["ws"] = torch.empty(max(16, size), dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------- one pass

def run(state):
    return (_own if own else _plain)(state)


def _own(s):
    from gradient_reduction_sharded_gb300 import grs
    op, st = s["case"]["op"], torch.cuda.current_stream().cuda_stream
    p = lambda k: s[k].data_ptr()  # noqa: E731
    if op == "experts_fwd":
        grs.grs_experts_forward(s["shape"], p("xs"), p("w"), p("offsets"), p("ys"), p("ws"), st)
        return {"ys": s["ys"]}
    if op == "experts_bwd":
        grs.grs_experts_backward(s["shape"], p("dys"), p("xs"), p("w"), p("offsets"), p("dxs"), p("dw"), p("ws"), st)
        return {"dxs": s["dxs"], "dw": s["dw"]}
    if op == "embed_fwd":
        grs.grs_embedding_forward(s["shape"], p("ids"), p("table"), p("out"), st)
        return {"y": s["out"]}
    if op == "embed_bwd":
        grs.grs_embedding_backward(s["shape"], p("ids"), p("dy"), p("out"), p("ws"), st)
        return {"dtable": s["out"]}
    if op == "qk_fwd":
        grs.grs_qk_norm_forward(s["shape"], p("q"), p("k"), p("wq"), p("wk"), p("pos"), p("turns"), p("qo"), p("ko"), st)
        return {"q": s["qo"], "k": s["ko"]}
    grs.grs_qk_norm_backward(s["shape"], p("dqo"), p("dko"), p("q"), p("k"), p("wq"), p("wk"), p("pos"), p("turns"), p("dq"), p("dk"),
                             p("dwq"), p("dwk"), p("ws"), st)
    return {"dq": s["dq"], "dk": s["dk"], "dwq": s["dwq"], "dwk": s["dwk"]}


def _plain(s):
    return {"experts_fwd": _plain_experts_fwd, "experts_bwd": _plain_experts_bwd, "embed_fwd": _plain_embed_fwd, "embed_bwd": _plain_embed_bwd,
            "qk_fwd": _plain_qk_fwd, "qk_bwd": _plain_qk_bwd}[s["case"]["op"]](s)


# ys[r] = w[e] xs[r] for the rows of expert e; dxs[r] = w[e]^T dys[r]; dw[e] = sum over its rows of dys[r] xs[r]^T.
# The experts' rows differ in number, so they go one by one; rows behind the last expert's are left as they are.

def _plain_experts_fwd(s):
    for e, (a, b) in enumerate(zip(s["bounds"], s["bounds"][1:])):
        s["ys"][a:b] = s["xs"][a:b].float() @ s["w"][e].float().T
    return {"ys": s["ys"]}


def _plain_experts_bwd(s):
    for e, (a, b) in enumerate(zip(s["bounds"], s["bounds"][1:])):
        dy = s["dys"][a:b].float()
        s["dxs"][a:b] = dy @ s["w"][e].float()
        s["dw"][e] = dy.T @ s["xs"][a:b].float()
    return {"dxs": s["dxs"], "dw": s["dw"]}


# y[t] = scale * table[id], zeros for an id that the table does not hold; its gradient.

def _plain_embed_fwd(s):
    row = s["ids"].long() - s["case"]["begin"]
    held = (row >= 0) & (row < s["table"].shape[0])
    y = s["table"][row.clamp(0, s["table"].shape[0] - 1)].float() * s["scale"]
    return {"y": torch.where(held[:, None], y, torch.zeros_like(y)).to(s["table"].dtype)}


def _plain_embed_bwd(s):
    c = s["case"]
    n = c["end"] - c["begin"]
    row = s["ids"].long() - c["begin"]
    row = torch.where((row >= 0) & (row < n), row, torch.full_like(row, n))  # one row more takes what is not held
    d = torch.zeros(n + 1, c["hidden"], device="cuda").index_add_(0, row, s["dy"].float() * s["scale"])
    return {"dtable": d[:n].to(DT[c["grad"]])}


# h = x / sqrt(mean(x^2) + eps) and u = h * w for each head; then each pair of the first `rot`
# elements, (i, i + rot / 2) or (2 i, 2 i + 1), is turned by position * inv_freq[i].

def _angles(s):
    a = s["pos"].double()[:, None] * s["inv_freq"]
    return a.cos().float()[:, None, :], a.sin().float()[:, None, :]


def _turn(u, cos, sin, c):
    r, y = c["rot"], u.clone()
    one, two = (slice(0, r, 2), slice(1, r, 2)) if c["pairs"] else (slice(0, r // 2), slice(r // 2, r))
    y[..., one] = u[..., one] * cos - u[..., two] * sin
    y[..., two] = u[..., two] * cos + u[..., one] * sin
    return y


def _heads(x, c):
    return x.unflatten(1, (-1, c["dim"])).float()


def _plain_qk_fwd(s):
    c = s["case"]
    cos, sin = _angles(s)

    def one(x, w):
        x = _heads(x, c)
        r = 1 / ((x * x).sum(2, keepdim=True) / float(c["dim"]) + EPS).sqrt()
        return _turn(x * r * w.float(), cos, sin, c).flatten(1).to(s["q"].dtype)

    return {"q": one(s["q"], s["wq"]), "k": one(s["k"], s["wk"])}


def _plain_qk_bwd(s):
    c = s["case"]
    cos, sin = _angles(s)

    def one(dy, x, w):
        x, du = _heads(x, c), _turn(_heads(dy, c), cos, -sin, c)
        r = 1 / ((x * x).sum(2, keepdim=True) / float(c["dim"]) + EPS).sqrt()
        h, dh = x * r, du * w.float()
        dx = r * (dh - h * ((dh * h).sum(2, keepdim=True) / float(c["dim"])))
        return dx.flatten(1).to(s["q"].dtype), (du * h).sum((0, 1)).to(DT[c["grad"]])

    dq, dwq = one(s["dqo"], s["q"], s["wq"])
    dk, dwk = one(s["dko"], s["k"], s["wk"])
    return {"dq": dq, "dk": dk, "dwq": dwq, "dwk": dwk}


# ------------------------------------------------------------------- 64 bits

def exact(case, seed):
    s, op = _inputs(case, seed), case["op"]
    if op.startswith("experts"):
        xs, w, at = s["xs"], s["w"], s["bounds"]
        used = at[-1]
        counts = [at[i + 1] - at[i] for i in range(case["experts"])]
        part = lambda x: x[:used].double().split(counts)  # noqa: E731
        if op == "experts_fwd":
            ys = torch.zeros_like(s["ys"], dtype=torch.float64)
            torch.cat([torch.einsum("rk,nk->rn", x, m.double()) for x, m in zip(part(xs), w)], out=ys[:used])
            return {"ys": ys}
        dxs = torch.zeros_like(xs, dtype=torch.float64)
        torch.cat([torch.einsum("rn,nk->rk", d, m.double()) for d, m in zip(part(s["dys"]), w)], out=dxs[:used])
        return {"dxs": dxs, "dw": torch.stack([torch.einsum("rn,rk->nk", d, x) for d, x in zip(part(s["dys"]), part(xs))])}
    if op == "embed_fwd":
        table = torch.nn.functional.pad(s["table"], (0, 0, 0, 1)).double().mul_(s["scale"])  # a row of zeros at the end
        last = table.shape[0] - 1
        where = torch.tensor([i - case["begin"] if case["begin"] <= i < case["end"] else last for i in s["ids"].tolist()], device="cuda")
        return {"y": table.index_select(0, where)}
    if op == "embed_bwd":
        ids, order = s["ids"].sort(stable=True)
        d = torch.zeros(case["end"] - case["begin"], case["hidden"], dtype=torch.float64, device="cuda")
        held = (ids >= case["begin"]) & (ids < case["end"])
        if bool(held.any()):
            rows, counts = torch.unique_consecutive(ids[held], return_counts=True)
            dy = s["dy"].double().index_select(0, order[held])
            d[rows.long() - case["begin"]] = torch.segment_reduce(dy, "sum", lengths=counts, axis=0)
        return {"dtable": d.mul_(s["scale"])}
    d, r = case["dim"], case["rot"]
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), torch.outer(s["pos"].double(), s["inv_freq"])).unsqueeze(1)

    def rotated(u, by):
        z = u[..., :r]
        z = torch.complex(z[..., 0::2].contiguous(), z[..., 1::2].contiguous()) if case["pairs"] else torch.complex(*(h.contiguous() for h in z.chunk(2, -1)))
        z = torch.view_as_real(z * by)
        z = z.flatten(-2) if case["pairs"] else z.transpose(-1, -2).flatten(-2)
        return torch.cat([z, u[..., r:]], -1)

    out = {}
    for name, heads in (("q", case["q_heads"]), ("k", case["k_heads"])):
        x, w = s[name].double().reshape(-1, heads, d), s["w" + name].double()
        inv = x.pow(2).mean(-1, keepdim=True).add(EPS).pow(-0.5)
        if op == "qk_fwd":
            out[name] = rotated(x * inv * w, turn).flatten(1)
            continue
        du = rotated(s["d" + name + "o"].double().reshape(-1, heads, d), turn.conj())
        dh = du * w
        dot = torch.einsum("thd,thd->th", dh, x).unsqueeze(2)
        out["d" + name] = (inv * dh - inv.pow(3) * x * dot / d).flatten(1)
        out["dw" + name] = torch.einsum("thd,thd->d", du, x * inv)
    return out
