"""What the training operators beside the gradient reduction cost: layer
norm (forward, backward), tokens sorted by expert and back (forward,
backward), and AdamW over a list of tensors with states in 32 or 8 bits.

`own` selects the side `run` takes: the plain form in elementary torch
operations, or the framework's entry points.
"""
import math

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
ESIZE = {"bf16": 2, "fp32": 4}
BLOCK = 256  # elements of one scale of the 8-bit states, and the alignment of each tensor in the state arrays
HP = {"lr": 1e-3, "beta1": 0.9, "beta2": 0.999, "eps": 1e-8, "weight_decay": 0.01, "max_norm": 1.0}


# ------------------------------------------------------------------- cases

def listed():
    return [
        # The update of the hand-sized model (six tensors) in its first step: latency.
        {"name": "adamw32_tiny", "op": "adamw32", "d": 64, "layers": 1, "ffn": 128, "vocab": 100, "grad": "fp32",
         "step": 1, "n_micro": 1, "shift": 0},
        # A model whose sizes divide nothing, bf16 gradients packed at an odd address, 4 microbatches summed.
        {"name": "adamw32_odd", "op": "adamw32", "d": 519, "layers": 9, "ffn": 1411, "vocab": 9973, "grad": "bf16",
         "step": 200, "n_micro": 4, "shift": 1},
        # The same update as the 67M-parameter plan's, states in 8 bits, fp32 gradients (the accumulator).
        {"name": "adamw8_67M", "op": "adamw8", "d": 1024, "layers": 4, "ffn": 4096, "vocab": 1001, "grad": "fp32",
         "step": 200, "n_micro": 1, "shift": 0},
        # The 1.1B decoder's list (d 2048, 22 layers, ffn 5632, vocabulary 32000), bf16 gradients.
        {"name": "adamw8_1B", "op": "adamw8", "d": 2048, "layers": 22, "ffn": 5632, "vocab": 32000, "grad": "bf16",
         "step": 1000, "n_micro": 1, "shift": 0},
        # One new token of the 1.1B decoder's width.
        {"name": "ln_fwd_token", "op": "ln_fwd", "rows": 1, "cols": 2048, "act": "bf16", "par": "bf16", "pad": 0},
        # A microbatch of 16 sequences of 2048 tokens.
        {"name": "ln_fwd_batch", "op": "ln_fwd", "rows": 32768, "cols": 2048, "act": "bf16", "par": "bf16", "pad": 0},
        # Backward of one sequence, the weight's gradient in the rank buffer's bf16.
        {"name": "ln_bwd_sequence", "op": "ln_bwd", "rows": 8192, "cols": 2048, "act": "bf16", "par": "bf16", "pad": 0},
        # Backward of a per-head norm: 4096 tokens x 16 heads of 128, rows inside a wider projection.
        {"name": "ln_bwd_heads", "op": "ln_bwd", "rows": 65536, "cols": 128, "act": "bf16", "par": "fp32", "pad": 256},
        # An odd width in fp32, a ragged number of rows.
        {"name": "ln_bwd_odd", "op": "ln_bwd", "rows": 1531, "cols": 1027, "act": "fp32", "par": "fp32", "pad": 0},
        # A handful of tokens through 32 experts: latency.
        {"name": "moe_fwd_few", "op": "moe_fwd", "tokens": 5, "top_k": 4, "experts": 32, "hidden": 2048, "act": "bf16"},
        # A microbatch of the MoE workload's width and number of experts, 8 experts a token.
        {"name": "moe_fwd_batch", "op": "moe_fwd", "tokens": 16384, "top_k": 8, "experts": 32, "hidden": 2048, "act": "bf16"},
        # Backward of an uneven microbatch.
        {"name": "moe_bwd_batch", "op": "moe_bwd", "tokens": 6001, "top_k": 6, "experts": 32, "hidden": 2048, "act": "bf16"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["adamw32", "adamw8", "ln_fwd", "ln_bwd", "moe_fwd", "moe_bwd"])
    if op.startswith("adamw"):
        most = 3e9 if op == "adamw32" else 17e9
        while True:
            d = _log(rng, 24, 2048)
            if rng.random() < 0.5:
                d = max(24, d // 8 * 8)
            c = {"op": op, "d": d, "layers": _log(rng, 1, 24), "ffn": _log(rng, d, 4 * d), "vocab": _log(rng, 50, 32000),
                 "grad": rng.choice(["bf16", "fp32"]), "step": _log(rng, 1, 10000), "n_micro": rng.choice([1, 1, 4, 8]),
                 "shift": rng.choice([0, 0, 1])}
            if work(c)["bytes"] <= most:
                return c
    act = rng.choice(["bf16", "bf16", "fp32"])
    if op.startswith("ln"):
        while True:
            cols = _log(rng, 16, 16384)
            if rng.random() < 0.6:
                cols = max(16, cols // 16 * 16)
            rows = _log(rng, 1, 1 << 18)
            if rows * cols * ESIZE[act] * (2 if op == "ln_fwd" else 3) <= (268e6 if op == "ln_fwd" else 100e6):
                return {"op": op, "rows": rows, "cols": cols, "act": act, "par": rng.choice(["bf16", "fp32"]) if act == "bf16" else "fp32",
                        "pad": rng.choice([0, 0, 16, 64])}
    while True:
        k = rng.choice([1, 2, 4, 6, 8])
        c = {"op": op, "tokens": _log(rng, 1, 16384), "top_k": k, "experts": max(k, _log(rng, 4, 256)),
             "hidden": _log(rng, 8, 512) * 8 + rng.choice([0, 0, 0, 3]), "act": act}
        if work(c)["bytes"] <= (1.2e9 if op == "moe_fwd" else 6e8):
            return c


def work(case):
    op = case["op"]
    if op.startswith("adamw"):
        n = sum(_numels(case))
        g = ESIZE[case["grad"]]
        # gradient in, master in and out, bf16 parameter out, both moments in and out
        return {"bytes": n * (g + 8 + 2 + (16 if op == "adamw32" else 4 + 16 / BLOCK)), "flops": n * (16 if op == "adamw32" else 30)}
    e = ESIZE[case["act"]]
    if op.startswith("ln"):
        n = case["rows"] * case["cols"]
        p = case["cols"] * ESIZE[case["par"]]
        if op == "ln_fwd":
            return {"bytes": 2 * n * e + 8 * case["rows"] + 2 * p, "flops": 8 * n}
        return {"bytes": 3 * n * e + 8 * case["rows"] + 3 * p, "flops": 14 * n}
    t, k, d = case["tokens"], case["top_k"], case["hidden"]
    if op == "moe_fwd":  # ids in, maps out; dispatch: x in, rows out; combine: rows and weights in, y out
        return {"bytes": t * k * 12 + 2 * (t * d + t * k * d) * e + t * k * 8, "flops": 2 * t * k * d}
    # dy, rows in, their gradients out, weights in and out, map in twice; expert input gradients in, dx out
    return {"bytes": 2 * t * d * e + 3 * t * k * d * e + t * k * 16, "flops": 4 * t * k * d}


# ------------------------------------------------------------------- inputs

def _numels(c):
    """Parameters of a decoder of these sizes, in model order."""
    d, kv = c["d"], max(1, c["d"] // 8)
    layer = [d, d * d, kv * d, kv * d, d * d, d, c["ffn"] * d, c["ffn"] * d, d * c["ffn"]]
    return [c["vocab"] * d] + layer * c["layers"] + [d, c["vocab"] * d]


def _layout(numels):
    """Offset of each tensor in the state arrays, and their length."""
    off, at = [], 0
    for n in numels:
        off.append(at)
        at += -(-n // BLOCK) * BLOCK
    return off, at


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(n, std, g, dtype):
    return torch.randn(n, generator=g, device="cuda").mul_(std).to(dtype)


def _adamw_inputs(case, seed):
    g = _gen(seed)
    numels = _numels(case)
    off, n = _layout(numels)
    live = torch.zeros(n, dtype=torch.bool, device="cuda")
    for o, k in zip(off, numels):
        live[o:o + k] = True
    gdt, sh = DT[case["grad"]], case["shift"]
    s = {"case": case, "numels": numels, "off": off, "n": n, "first": case["step"] == 1}
    s["grads"] = torch.zeros(n + 8, dtype=gdt, device="cuda")[sh:sh + n]
    s["grads"].copy_(_normal(n, 1e-3 * case["n_micro"], g, gdt).mul_(live))
    s["params"] = torch.zeros(n + 8, dtype=torch.bfloat16, device="cuda")[sh:sh + n]
    s["master"] = _normal(n, 0.02, g, torch.float32).mul_(live)
    s["params"].copy_(s["master"])
    used = torch.tensor(float(sum(numels)), dtype=torch.float64, device="cuda")
    # The squared norm of the whole job's gradient, as the other ranks' parts add up to it.
    s["norm_sq"] = (used * 1e-6 * (1.0 + 0.1 * (seed % 7))).reshape(1)
    s["seed"] = (seed * 0x9E3779B97F4A7C15 + case["step"]) % (1 << 64)
    if case["op"] == "adamw32":
        s["m"] = torch.zeros(n, device="cuda")
        s["v"] = torch.zeros(n, device="cuda")
        if not s["first"]:
            s["m"].copy_(_normal(n, 3e-4, g, torch.float32).mul_(live))
            s["v"].copy_(_normal(n, 1e-3, g, torch.float32).square_().mul_(live))
        return s
    nb = n // BLOCK
    s["m8"] = torch.zeros(n, dtype=torch.uint8, device="cuda")
    s["s8"] = torch.zeros(n, dtype=torch.uint8, device="cuda")
    s["m_scale"] = torch.zeros(nb, device="cuda")
    s["s_scale"] = torch.zeros(nb, device="cuda")
    if not s["first"]:
        m = (torch.randn(n, generator=g, device="cuda") * 60).clamp_(-240, 240).mul_(live)
        s["m8"].copy_(m.to(torch.float8_e4m3fn).view(torch.uint8))
        m = (torch.randn(n, generator=g, device="cuda").abs_() * 60 + 1).clamp_(max=240).mul_(live)
        s["s8"].copy_(m.to(torch.float8_e4m3fn).view(torch.uint8))
        del m
        for k, base in (("m_scale", -18), ("s_scale", -16)):
            s[k].copy_(torch.ldexp(torch.ones(nb, device="cuda"), torch.randint(base - 2, base + 2, (nb,), generator=g, device="cuda")))
    return s


def _ln_inputs(case, seed):
    g = _gen(seed)
    rows, cols, act, par = case["rows"], case["cols"], DT[case["act"]], DT[case["par"]]

    def rect(std, mean=0.0):
        wide = torch.zeros(rows, cols + case["pad"], dtype=act, device="cuda")
        wide[:, :cols] = torch.randn(rows, cols, generator=g, device="cuda") * std + mean
        return wide[:, :cols]

    s = {"case": case, "x": rect(1.5, 0.3), "w": (1 + 0.1 * torch.randn(cols, generator=g, device="cuda")).to(par),
         "b": (0.1 * torch.randn(cols, generator=g, device="cuda")).to(par), "eps": 1e-5}
    if case["op"] == "ln_bwd":
        s["dy"] = rect(1e-2)
        x = s["x"].float()
        s["mean"] = x.mean(1)
        s["rstd"] = 1 / ((x - s["mean"][:, None]).square().mean(1) + s["eps"]).sqrt()
    return s


def _moe_inputs(case, seed):
    g = _gen(seed)
    t, k, d, act = case["tokens"], case["top_k"], case["hidden"], DT[case["act"]]
    # Uneven experts, k different ones a token, weights that sum to 1.
    logits = torch.randn(t, case["experts"], generator=g, device="cuda") + torch.randn(case["experts"], generator=g, device="cuda")
    top = logits.topk(k, 1)
    s = {"case": case, "ids": top.indices.to(torch.int32).contiguous(), "weights": top.values.softmax(1).contiguous(),
         "ys": _normal((t * k, d), 0.5, g, act)}
    if case["op"] == "moe_fwd":
        s["x"] = _normal((t, d), 1.0, g, act)
    else:
        s["dy"] = _normal((t, d), 1e-2, g, act)
        s["dxs"] = _normal((t * k, d), 1e-2, g, act)
        s["slot_row"] = _sorted_rows(s["ids"], case["experts"])[2].reshape(t, k)
    return s


def _inputs(case, seed):
    return (_adamw_inputs if case["op"].startswith("adamw") else _ln_inputs if case["op"].startswith("ln") else _moe_inputs)(case, seed)


class _List:
    """The framework's handle of a list of tensors, destroyed with the state."""

    def __init__(self, numels):
        from gradient_reduction_sharded_gb300 import grs
        self.grs, self.handle = grs, grs.grs_tensors_create(numels)
        self.info = grs.grs_tensors_query(self.handle)

    def __del__(self):
        if self.grs is not None:
            torch.cuda.synchronize()
            self.grs.grs_tensors_destroy(self.handle)


def prepare(case, seed):
    s = _inputs(case, seed)
    if not own:
        return s
    from gradient_reduction_sharded_gb300 import grs
    if case["op"].startswith("adamw"):
        s["list"] = _List(s["numels"])
        info = s["list"].info
        assert info["n_state"] == s["n"]
        ptrs = lambda t: torch.tensor([t.data_ptr() + o * t.element_size() for o in s["off"]], dtype=torch.int64, device="cuda")  # noqa: E731
        s["grad_ptrs"], s["param_ptrs"] = ptrs(s["grads"]), ptrs(s["params"])
        s["ws"] = torch.zeros(info["workspace_bytes"], dtype=torch.uint8, device="cuda")
        s["norm_out"] = torch.zeros(1, dtype=torch.float64, device="cuda")
    elif case["op"].startswith("ln"):
        dt = {"bf16": grs.GRS_DTYPE_BF16, "fp32": grs.GRS_DTYPE_FP32}
        x = s["x"]
        s["shape"] = grs.make_norm(x.shape[0], x.shape[1], s["eps"], dt[case["act"]], dt[case["par"]], dt[case["par"]],
                                   ld_x=x.stride(0), ld_y=x.shape[1], ld_dy=x.stride(0), ld_dx=x.shape[1])
        s["ws"] = torch.empty(max(16, grs.grs_layernorm_workspace_bytes(s["shape"])), dtype=torch.uint8, device="cuda")
        s["y"] = torch.empty(x.shape, dtype=x.dtype, device="cuda")
        s["out"] = [torch.empty(x.shape[0], device="cuda") for _ in range(2)] if case["op"] == "ln_fwd" else \
            [torch.empty_like(s["w"]) for _ in range(2)]
    else:
        t, k, d = case["tokens"], case["top_k"], case["hidden"]
        s["shape"] = grs.make_moe(t, k, case["experts"], 0, case["experts"], d,
                                  {"bf16": grs.GRS_DTYPE_BF16, "fp32": grs.GRS_DTYPE_FP32}[case["act"]])
        s["ws"] = torch.empty(max(16, grs.grs_moe_workspace_bytes(s["shape"])), dtype=torch.uint8, device="cuda")
        s["rows"] = torch.empty_like(s["ys"])
        s["y"] = torch.empty(t, d, dtype=s["ys"].dtype, device="cuda")
        if case["op"] == "moe_fwd":
            s["offsets"] = torch.empty(case["experts"] + 1, dtype=torch.int32, device="cuda")
            s["row_slot"] = torch.empty(t * k, dtype=torch.int32, device="cuda")
            s["slot_row"] = torch.empty(t * k, dtype=torch.int32, device="cuda")
        else:
            s["dweights"] = torch.empty_like(s["weights"])
    return s


# ------------------------------------------------------------------- one pass

def run(state):
    return (_own if own else _plain)(state)


def _own(s):
    from gradient_reduction_sharded_gb300 import grs
    c, st = s["case"], torch.cuda.current_stream().cuda_stream
    p = lambda k: s[k].data_ptr()  # noqa: E731
    op = c["op"]
    if op.startswith("adamw"):
        h, dt = s["list"].handle, grs.GRS_DTYPE_BF16 if c["grad"] == "bf16" else grs.GRS_DTYPE_FP32
        hp = grs.make_adamw(HP["lr"], HP["beta1"], HP["beta2"], HP["eps"], HP["weight_decay"], HP["max_norm"], c["step"], c["n_micro"])
        if op == "adamw32":
            grs.grs_tensors_norm_sq(h, p("grad_ptrs"), dt, c["n_micro"], p("ws"), p("norm_out"), st)
            grs.grs_tensors_adamw_step(h, hp, p("norm_out"), p("grad_ptrs"), dt, p("master"), p("m"), p("v"), p("param_ptrs"), st)
            return {"norm_sq": s["norm_out"], "master": s["master"], "m": s["m"], "v": s["v"], "params": s["params"]}
        grs.grs_tensors_adamw8_step(h, hp, s["seed"], p("norm_sq"), p("grad_ptrs"), dt, p("master"), p("m8"), p("m_scale"),
                                    p("s8"), p("s_scale"), p("param_ptrs"), st)
        return _state8(s)
    if op == "ln_fwd":
        grs.grs_layernorm_forward(s["shape"], p("x"), p("w"), p("b"), p("y"), s["out"][0].data_ptr(), s["out"][1].data_ptr(), st)
        return {"y": s["y"], "mean": s["out"][0], "rstd": s["out"][1]}
    if op == "ln_bwd":
        grs.grs_layernorm_backward(s["shape"], p("dy"), p("x"), p("w"), p("mean"), p("rstd"), p("y"), s["out"][0].data_ptr(),
                                   s["out"][1].data_ptr(), p("ws"), st)
        return {"dx": s["y"], "dw": s["out"][0], "db": s["out"][1]}
    if op == "moe_fwd":
        grs.grs_moe_sort(s["shape"], p("ids"), p("offsets"), p("row_slot"), p("slot_row"), p("ws"), st)
        grs.grs_moe_dispatch(s["shape"], p("x"), p("slot_row"), p("rows"), st)
        grs.grs_moe_combine(s["shape"], p("ys"), p("slot_row"), p("weights"), p("y"), st)
        return {"offsets": s["offsets"], "row_slot": s["row_slot"], "slot_row": s["slot_row"], "xs": s["rows"], "y": s["y"]}
    grs.grs_moe_combine_backward(s["shape"], p("dy"), p("ys"), p("slot_row"), p("weights"), p("rows"), p("dweights"), st)
    grs.grs_moe_dispatch_backward(s["shape"], p("dxs"), p("slot_row"), p("y"), st)
    return {"dys": s["rows"], "dweights": s["dweights"], "dx": s["y"]}


def _state8(s):
    """The states as they stand: E4M3 numbers in units of each block's scale, and the scales."""
    return {"master": s["master"], "params": s["params"], "m": s["m8"].view(torch.float8_e4m3fn), "m_scale": s["m_scale"],
            "s": s["s8"].view(torch.float8_e4m3fn), "s_scale": s["s_scale"]}


def _plain(s):
    op = s["case"]["op"]
    if op == "adamw32":
        return _plain_adamw32(s)
    if op == "adamw8":
        return _plain_adamw8(s)
    if op.startswith("ln"):
        return _plain_ln_fwd(s) if op == "ln_fwd" else _plain_ln_bwd(s)
    return _plain_moe_fwd(s) if op == "moe_fwd" else _plain_moe_bwd(s)


# AdamW (decoupled weight decay) on the clipped, microbatch-averaged gradient.

def _consts(c):
    f = lambda v: float(np.float32(v))  # noqa: E731
    lr, b1, b2, wd = f(HP["lr"]), f(HP["beta1"]), f(HP["beta2"]), f(HP["weight_decay"])
    return {"decay": f(1 - lr * wd), "b1": b1, "omb1": f(1 - b1), "b2": b2, "omb2": f(1 - b2), "eps": f(HP["eps"]),
            "step_size": f(lr / (1 - b1 ** c["step"])), "inv_bc2": f(1 / math.sqrt(1 - b2 ** c["step"])), "inv_m": f(1 / c["n_micro"])}


def _gscale(norm_sq, k):
    one = torch.ones_like(norm_sq, dtype=torch.float32)
    cr = (one * HP["max_norm"]) / (norm_sq.to(torch.float32).sqrt() + 1e-6)
    return torch.minimum(cr, one) * k["inv_m"]


def _moments(g, p, m, v, k):
    """(p, m, sqrt(v), v) after the step."""
    m = m * k["b1"] + g * k["omb1"]
    v = v * k["b2"] + (g * k["omb2"]) * g
    s = v.sqrt()
    p = p * k["decay"] - (m / (s * k["inv_bc2"] + k["eps"])) * k["step_size"]
    return p, m, s, v


def _plain_adamw32(s):
    k = _consts(s["case"])
    g = s["grads"].float()
    norm_sq = (g * k["inv_m"]).square().double().sum().reshape(1)
    p, m, _, v = _moments(g * _gscale(norm_sq, k), s["master"], s["m"], s["v"], k)
    s["master"].copy_(p)
    s["m"].copy_(m)
    s["v"].copy_(v)
    s["params"].copy_(p)
    return {"norm_sq": norm_sq, "master": s["master"], "m": s["m"], "v": s["v"], "params": s["params"]}


# 32-bit mixing: odd multipliers from the golden ratio and the square roots of
# 2 and 3, shifts that fold the high half down.
_A, _B, _C = 0x9E3779B9, 0x6A09E667, 0xBB67AE85


def _mix(x):
    x ^= x >> 16
    x = x * _A & 0xFFFFFFFF
    x ^= x >> 15
    x = x * _C & 0xFFFFFFFF
    return x ^ x >> 16


def _signed(c):
    return c - (1 << 32) if c >> 31 else c


def _random(n, seed):
    """32 random bits for each element of the state arrays, from the seed and the element's index."""
    key0 = _mix(((seed & 0xFFFFFFFF) + _A) & 0xFFFFFFFF)
    key1 = _mix(key0 ^ seed >> 32)
    i = torch.arange(n, device="cuda")
    x = i.to(torch.int32) ^ _signed(key0) ^ (i >> 32).to(torch.int32) * _B
    del i
    x = (x ^ x >> 16 & 0xFFFF) * _signed(_A) ^ _signed(key1)
    x = (x ^ x >> 15 & 0x1FFFF) * _signed(_C)
    return x ^ x >> 16 & 0xFFFF


def _to8(x, r16, positive):
    """(codes, scales): E4M3 numbers of each block in units of a power of two that
    brings the block's largest magnitude into (128, 256], rounded up with the
    probability of the fraction cut off; a positive number of the second kind
    never becomes zero. A block that holds NaN or infinity gets the scale NaN."""
    bits = x.abs().view(torch.int32).reshape(-1, BLOCK)
    top = bits.amax(1).long()
    bad = top >= 0x7F800000
    e = ((top + 0x7FFFFF >> 23) - 8).clamp_(1, 247).to(torch.int32)
    scale = (e << 23).view(torch.float32)
    y = (x.abs().reshape(-1, BLOCK) * ((254 - e) << 23).view(torch.float32)[:, None]) * 2.0 ** -120
    code = y.view(torch.int32) + (r16.reshape(-1, BLOCK) << 4 | 8) >> 20
    if positive:
        code = torch.maximum(code, (bits > 0).to(torch.int32))
    code = code | (x.view(torch.int32).reshape(-1, BLOCK) >> 31 & 0x80)
    code = torch.where(bad[:, None], torch.zeros_like(code), code)
    return code.to(torch.uint8).reshape(-1), torch.where(bad, torch.full_like(scale, math.nan), scale)


def _from8(code, scale):
    return (code.view(torch.float8_e4m3fn).float().reshape(-1, BLOCK) * scale[:, None]).reshape(-1)


def _plain_adamw8(s):
    k = _consts(s["case"])
    g = s["grads"].float() * _gscale(s["norm_sq"], k)
    p, m, r, _ = _moments(g, s["master"], _from8(s["m8"], s["m_scale"]), _from8(s["s8"], s["s_scale"]).square(), k)
    s["master"].copy_(p)
    s["params"].copy_(p)
    del g, p
    bits = _random(s["n"], s["seed"])
    for key, scale, x, r16 in (("m8", "m_scale", m, bits & 0xFFFF), ("s8", "s_scale", r, bits >> 16 & 0xFFFF)):
        code, sc = _to8(x, r16, key == "s8")
        s[key].copy_(code)
        s[scale].copy_(sc)
    return _state8(s)


def _plain_ln_fwd(s):
    x = s["x"].float()
    mean = x.sum(1) / float(x.shape[1])
    xc = x - mean[:, None]
    rstd = 1 / ((xc * xc).sum(1) / float(x.shape[1]) + s["eps"]).sqrt()
    y = xc * rstd[:, None] * s["w"].float() + s["b"].float()
    return {"y": y.to(s["x"].dtype), "mean": mean, "rstd": rstd}


def _plain_ln_bwd(s):
    dy = s["dy"].float()
    h = (s["x"].float() - s["mean"][:, None]) * s["rstd"][:, None]
    dh = dy * s["w"].float()
    c = float(h.shape[1])
    dx = s["rstd"][:, None] * (dh - (dh.sum(1) / c)[:, None] - h * ((dh * h).sum(1) / c)[:, None])
    return {"dx": dx.to(s["x"].dtype), "dw": (dy * h).sum(0).to(s["w"].dtype), "db": dy.sum(0).to(s["w"].dtype)}


def _sorted_rows(ids, experts):
    """(offsets, row_slot, slot_row): the slots (token, choice) sorted by expert, the order of slots kept within one."""
    flat = ids.reshape(-1)
    hit = (flat[None, :] == torch.arange(experts, dtype=torch.int32, device="cuda")[:, None]).to(torch.int32)
    offsets = torch.zeros(experts + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = hit.sum(1).cumsum(0)
    before = hit.cumsum(1, dtype=torch.int32).gather(0, flat.long()[None, :])[0] - 1
    slot_row = offsets[flat.long()] + before
    row_slot = torch.empty_like(slot_row)
    row_slot[slot_row.long()] = torch.arange(flat.numel(), dtype=torch.int32, device="cuda")
    return offsets, row_slot, slot_row


def _plain_moe_fwd(s):
    k = s["case"]["top_k"]
    offsets, row_slot, slot_row = _sorted_rows(s["ids"], s["case"]["experts"])
    xs = s["x"][row_slot.long() // k]
    y = (s["ys"][slot_row.long()].float().reshape(-1, k, xs.shape[1]) * s["weights"][:, :, None]).sum(1)
    return {"offsets": offsets, "row_slot": row_slot, "slot_row": slot_row, "xs": xs, "y": y.to(s["x"].dtype)}


def _plain_moe_bwd(s):
    rows = s["slot_row"].long()
    dy = s["dy"].float()[:, None, :]
    dys = torch.empty_like(s["ys"])
    dys[rows] = (dy * s["weights"][:, :, None]).to(dys.dtype)
    dweights = (s["ys"][rows].float() * dy).sum(2)
    return {"dys": dys, "dweights": dweights, "dx": s["dxs"][rows].float().sum(1).to(s["dy"].dtype)}


# ------------------------------------------------------------------- 64 bits

def exact(case, seed):
    s, op = _inputs(case, seed), case["op"]
    if op.startswith("adamw"):
        hp = {k: float(np.float32(v)) for k, v in HP.items()}  # the numbers as the call takes them
        b1, b2, lr = hp["beta1"], hp["beta2"], hp["lr"]
        g = s["grads"].double() / case["n_micro"]
        norm_sq = g.dot(g) if op == "adamw32" else s["norm_sq"][0]
        g *= min(1.0, hp["max_norm"] / (math.sqrt(float(norm_sq)) + 1e-6))
        if op == "adamw32":
            m, v = s["m"].double(), s["v"].double()
        else:
            wide = lambda code, scale: torch.mul(s[code].view(torch.float8_e4m3fn).to(torch.float64).view(-1, BLOCK), s[scale].double().view(-1, 1)).view(-1)  # noqa: E731
            m, v = wide("m8", "m_scale"), wide("s8", "s_scale").pow(2)
        m = torch.lerp(g, m, b1)
        v = torch.lerp(g.pow(2), v, b2)
        hat = (v / (1 - b2 ** case["step"])).sqrt_().add_(hp["eps"])
        p = s["master"].double() * (1 - lr * hp["weight_decay"]) - lr / (1 - b1 ** case["step"]) * (m / hat)
        if op == "adamw32":
            return {"norm_sq": norm_sq.reshape(1), "master": p, "m": m, "v": v, "params": p}
        return {"master": p, "params": p, "m": None, "m_scale": None, "s": None, "s_scale": None}
    if op.startswith("ln"):
        x, w = s["x"].double(), s["w"].double()
        var, mean = torch.var_mean(x, 1, correction=0)
        rstd = (var + s["eps"]).pow(-0.5)
        if op == "ln_fwd":
            return {"y": torch.addcmul(s["b"].double(), (x - mean.unsqueeze(1)) * rstd.unsqueeze(1), w), "mean": mean, "rstd": rstd}
        mean, rstd, dy = s["mean"].double(), s["rstd"].double(), s["dy"].double()
        h = torch.einsum("rc,r->rc", x - mean.unsqueeze(1), rstd)
        dh = torch.einsum("rc,c->rc", dy, w)
        dx = dh - dh.mean(1, keepdim=True) - h * torch.einsum("rc,rc->r", dh, h).div(w.numel()).unsqueeze(1)
        return {"dx": dx * rstd.unsqueeze(1), "dw": torch.einsum("rc,rc->c", dy, h), "db": dy.sum(0)}
    t, k = case["tokens"], case["top_k"]
    ids = s["ids"].reshape(-1).cpu().numpy()
    order = np.argsort(ids, kind="stable")
    row = np.empty_like(order)
    row[order] = np.arange(t * k)
    rows, order = torch.from_numpy(row).cuda().reshape(t, k), torch.from_numpy(order).cuda()
    wt = s["weights"].double()
    if op == "moe_fwd":
        counts = np.bincount(ids, minlength=case["experts"])
        y = torch.zeros(t, case["hidden"], dtype=torch.float64, device="cuda")
        for j in range(k):
            y.addcmul_(s["ys"].index_select(0, rows[:, j]).double(), wt[:, j:j + 1])
        return {"offsets": torch.from_numpy(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)), "row_slot": order.to(torch.int32),
                "slot_row": rows.reshape(-1).to(torch.int32), "xs": s["x"].double().index_select(0, order // k), "y": y}
    dy = s["dy"].double()
    dys = dy.index_select(0, order // k) * wt.reshape(-1)[order].unsqueeze(1)
    dw = torch.stack([torch.einsum("td,td->t", s["ys"].index_select(0, rows[:, j]).double(), dy) for j in range(k)], 1)
    dx = sum(s["dxs"].index_select(0, rows[:, j]).double() for j in range(k))
    return {"dys": dys, "dweights": dw, "dx": dx}
