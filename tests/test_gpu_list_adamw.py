"""AdamW over a list of tensors, states in 32 and in 8 bits, on the GPU.

Expected values: numpy in 64 bits from the formulas; for the 8-bit codes a
restatement in numpy's float32, which rounds every product and sum as IEEE
arithmetic does, so the codes have to be equal bit for bit.
"""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

B = 256
HP = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01)
# Sizes: one element, an empty tensor, around a block and around a tile of 2048, several tiles.
SIZES = [[1], [5, 0, 255, 256, 257], [2047, 2048, 2049, 1, 7 * 2048 + 300], [100003, 31, 65536]]
# fp32 arithmetic against 64 bits: under ten roundings a result, each at most 2^-24 of an operand, and a
# master whose update is not larger than itself by orders of magnitude.
RTOL, ATOL = 1e-5, 1e-7


@pytest.fixture(scope="module")
def grs():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from gradient_reduction_sharded_gb300 import grs as g
    return g


def f32(x):
    return float(np.float32(x))


class List:
    """A list with gradients (one buffer a tensor, starting `shift` elements into its storage) and states."""

    def __init__(self, grs, numels, bf16=False, shift=0, seed=0, skip=()):
        self.grs, self.numels, self.skip = grs, numels, set(skip)
        self.h = grs.grs_tensors_create(numels)
        self.info = grs.grs_tensors_query(self.h)
        self.n = self.info["n_state"]
        self.off = [grs.grs_tensors_offset(self.h, i) for i in range(len(numels))]
        rng = np.random.default_rng(seed)
        dt = torch.bfloat16 if bf16 else torch.float32
        self.dt = grs.GRS_DTYPE_BF16 if bf16 else grs.GRS_DTYPE_FP32
        self.store, self.pstore = [], []
        g = np.zeros(self.n, np.float32)
        for i, k in enumerate(numels):
            x = torch.from_numpy((rng.standard_normal(k) * 1e-2).astype(np.float32)).to(dt)
            buf = torch.full((k + 16,), float("nan"), dtype=dt, device="cuda")
            buf[shift:shift + k] = x.cuda()
            self.store.append(buf)
            self.pstore.append(torch.full((k + 16,), 7.0, dtype=torch.bfloat16, device="cuda"))
            g[self.off[i]:self.off[i] + k] = x.float().numpy()
        self.g = g
        self.shift = shift
        table = lambda bufs, size, skip: torch.tensor([0 if i in skip else b.data_ptr() + shift * size for i, b in enumerate(bufs)],  # noqa: E731
                                                      dtype=torch.int64, device="cuda")
        self.gp, self.pp = table(self.store, 2 if bf16 else 4, self.skip), table(self.pstore, 2, ())
        self.live = np.zeros(self.n, bool)
        for i, k in enumerate(numels):
            if i not in self.skip:
                self.live[self.off[i]:self.off[i] + k] = True
        self.used = np.zeros(self.n, bool)
        for i, k in enumerate(numels):
            self.used[self.off[i]:self.off[i] + k] = True
        self.rng = rng
        self.master = self.fill(0.02)
        self.ws = torch.zeros(self.info["workspace_bytes"], dtype=torch.uint8, device="cuda")
        self.norm = torch.zeros(1, dtype=torch.float64, device="cuda")

    def fill(self, std, square=False):
        """Random state; the padding holds NaN."""
        x = (self.rng.standard_normal(self.n) * std).astype(np.float32)
        x = x * x if square else x
        x[~self.used] = np.nan
        return torch.from_numpy(x).cuda()

    def stream(self):
        return torch.cuda.current_stream().cuda_stream

    def params(self):
        """The bf16 parameters; what lies around each is untouched."""
        got = np.zeros(self.n, np.float32)
        for i, k in enumerate(self.numels):
            p = self.pstore[i].float().cpu().numpy()
            assert (p[:self.shift] == 7).all() and (p[self.shift + k:] == 7).all()
            got[self.off[i]:self.off[i] + k] = p[self.shift:self.shift + k]
        return got

    def close(self):
        torch.cuda.synchronize()
        assert self.grs.grs_tensors_check_device_errors(self.h, self.stream()) != self.grs.GRS_ERR_BOUNDS
        self.grs.grs_tensors_destroy(self.h)


def step64(g, p, m, v, step, c, n_micro):
    """One AdamW step in 64 bits with the hyper-parameters as fp32 numbers."""
    lr, b1, b2, eps, wd = (f32(HP[k]) for k in ("lr", "beta1", "beta2", "eps", "weight_decay"))
    g = g.astype(np.float64) * c / n_micro
    m = b1 * m.astype(np.float64) + (1 - b1) * g
    v = b2 * v.astype(np.float64) + (1 - b2) * g * g
    p = p.astype(np.float64) * (1 - lr * wd) - lr / (1 - b1 ** step) * m / (np.sqrt(v) / math.sqrt(1 - b2 ** step) + eps)
    return p, m, v


def clip(S, max_norm):
    return min(1.0, max_norm / (math.sqrt(S) + 1e-6)) if max_norm > 0 else 1.0


@pytest.mark.parametrize("numels", SIZES)
@pytest.mark.parametrize("bf16,shift", [(False, 0), (True, 0), (True, 1), (False, 3), (True, 8)])
def test_norm(grs, numels, bf16, shift):
    t = List(grs, numels, bf16, shift, seed=1, skip=[1] if len(numels) > 2 else [])
    grs.grs_tensors_norm_sq(t.h, t.gp.data_ptr(), t.dt, 3, t.ws.data_ptr(), t.norm.data_ptr(), t.stream())
    a = float(t.norm.cpu()[0])
    grs.grs_tensors_norm_sq(t.h, t.gp.data_ptr(), t.dt, 3, t.ws.data_ptr(), t.norm.data_ptr(), t.stream())
    want = float(np.sum(t.g[t.live].astype(np.float64) ** 2)) / 9
    # a tile's sum passes through at most 8 + 5 + 8 additions of positive fp32 numbers
    assert abs(a - want) <= 22 * 2.0 ** -24 * want
    assert float(t.norm.cpu()[0]) == a
    assert grs.grs_tensors_check_device_errors(t.h, t.stream()) == grs.GRS_OK
    t.close()


def test_norm_flags_a_nonfinite_gradient(grs):
    t = List(grs, [300, 4000])
    t.store[1][77] = float("inf")
    grs.grs_tensors_norm_sq(t.h, t.gp.data_ptr(), t.dt, 1, t.ws.data_ptr(), t.norm.data_ptr(), t.stream())
    assert grs.grs_tensors_check_device_errors(t.h, t.stream()) == grs.GRS_ERR_NONFINITE
    assert grs.grs_tensors_check_device_errors(t.h, t.stream()) == grs.GRS_OK
    t.close()


@pytest.mark.parametrize("numels", SIZES)
@pytest.mark.parametrize("bf16,shift,max_norm,n_micro", [(False, 0, 1.0, 1), (True, 0, 0.0, 4), (True, 1, 0.05, 1), (False, 1, 0.05, 8)])
def test_step_in_32_bits(grs, numels, bf16, shift, max_norm, n_micro):
    skip = [2] if len(numels) > 2 else []
    t = List(grs, numels, bf16, shift, seed=2, skip=skip)
    m, v = t.fill(1e-3), t.fill(1e-2, square=True)
    before = [x.cpu().numpy() for x in (t.master, m, v)]
    S = 0.7
    t.norm.fill_(S)
    hp = grs.make_adamw(*HP.values(), max_norm, 5, n_micro)
    grs.grs_tensors_adamw_step(t.h, hp, t.norm.data_ptr(), t.gp.data_ptr(), t.dt, t.master.data_ptr(), m.data_ptr(),
                               v.data_ptr(), t.pp.data_ptr(), t.stream())
    torch.cuda.synchronize()
    want = step64(t.g, *before, 5, clip(S, max_norm), n_micro)
    got = [x.cpu().numpy() for x in (t.master, m, v)]
    params = t.params()
    for a, b, old in zip(got, want, before):
        assert (np.abs(a - b)[t.live] <= ATOL + RTOL * np.abs(b[t.live])).all()
        kept = t.used & ~t.live
        assert np.array_equal(a[kept], old[kept])  # a tensor without a gradient
    bf = torch.from_numpy(got[0]).to(torch.bfloat16).float().numpy()
    assert np.array_equal(params[t.live], bf[t.live])
    if not skip:
        for a in got:
            assert (a[~t.used] == 0).all()  # padding held NaN
    t.close()


def test_step_equals_the_plan_update_bit_for_bit(grs):
    """A plan's arrays as a list of one tensor: the same bits as grs_clip_adamw_step."""
    plan = grs.grs_plan_create([70001, 300], [0, 0], 1, 1, 1, 1, 1 << 30)
    n = grs.grs_plan_query(plan)["n_state_pad"]
    used = 70301
    t = List(grs, [n], seed=3)
    t.store[0][used:n] = 0
    m, v = t.fill(1e-3), t.fill(1e-2, square=True)
    for x in (t.master, m, v):
        x[used:] = 0
    copies = [x.clone() for x in (t.master, m, v)]
    p2 = torch.zeros(n, dtype=torch.int16, device="cuda")
    t.norm.fill_(3.0)
    hp = grs.make_adamw(*HP.values(), 1.0, 9, 2)
    grs.grs_tensors_adamw_step(t.h, hp, t.norm.data_ptr(), t.gp.data_ptr(), t.dt, t.master.data_ptr(), m.data_ptr(),
                               v.data_ptr(), t.pp.data_ptr(), t.stream())
    grs.grs_clip_adamw_step(plan, hp, t.norm.data_ptr(), t.store[0].data_ptr(), *(x.data_ptr() for x in copies),
                            p2.data_ptr(), t.stream())
    torch.cuda.synchronize()
    for a, b in zip((t.master, m, v), copies):
        assert torch.equal(a[:n].view(torch.int32), b[:n].view(torch.int32))
    assert torch.equal(t.pstore[0][:n].view(torch.int16), p2)
    t.close()
    grs.grs_plan_destroy(plan)


# ---------------------------------------------------------------- 8 bits

def e4m3(code):
    """The number of a code: sign, 4 exponent bits of bias 7, 3 mantissa bits."""
    code = code.astype(np.int64)
    e, f = code >> 3 & 15, code & 7
    x = np.where(e == 0, f * 2.0 ** -9, (8 + f) * 2.0 ** (e.astype(np.float64) - 10))
    return np.where(code & 128, -x, x)


def mix(x):
    x = x ^ x >> 16
    x = x * 0x9E3779B9 & 0xFFFFFFFF
    x = x ^ x >> 15
    x = x * 0xBB67AE85 & 0xFFFFFFFF
    return x ^ x >> 16


def random_bits(n, seed):
    k0 = mix((seed & 0xFFFFFFFF) + 0x9E3779B9 & 0xFFFFFFFF)
    k1 = mix(k0 ^ seed >> 32)
    x = np.arange(n, dtype=np.uint64) ^ np.uint64(k0)  # indexes below 2^32
    x = x ^ x >> np.uint64(16)
    x = x * np.uint64(0x9E3779B9) & np.uint64(0xFFFFFFFF) ^ np.uint64(k1)
    x = x ^ x >> np.uint64(15)
    x = x * np.uint64(0xBB67AE85) & np.uint64(0xFFFFFFFF)
    return (x ^ x >> np.uint64(16)).astype(np.int64)


def to8(x, r16, positive):
    """Codes and scales of float32 x by stochastic rounding, in 64-bit arithmetic on whole numbers."""
    x = x.reshape(-1, B)
    top = np.abs(x).max(1)
    scale = np.maximum(np.exp2(np.ceil(np.log2(np.maximum(top, 1e-300).astype(np.float64))) - 8), 2.0 ** -126)
    y = np.abs(x).astype(np.float64) / scale[:, None]
    e = np.maximum(np.floor(np.log2(np.maximum(y, 1e-300))), -6)  # exponent of the code, -6 for subnormals
    ulp = np.exp2(e - 3)
    k = np.floor(y / ulp)
    # the fraction beyond the code in units of 2^-20, as far as fp32 holds it, plus the random number
    frac = np.floor((y / ulp - k) * 2 ** 20)
    k += frac + (r16.reshape(-1, B) * 16 + 8) >= 2 ** 20
    val = k * ulp
    if positive:
        val = np.where((x > 0) & (val == 0), 2.0 ** -9, val)
    return np.copysign(val, x).reshape(-1), scale.astype(np.float32)


def random_state8(t, seed):
    rng = np.random.default_rng(seed)
    m8 = rng.integers(0, 0x79, t.n).astype(np.uint8) | (rng.integers(0, 2, t.n).astype(np.uint8) << 7)
    s8 = rng.integers(1, 0x79, t.n).astype(np.uint8)
    ms = np.exp2(rng.integers(-20, -14, t.n // B)).astype(np.float32)
    ss = np.exp2(rng.integers(-18, -13, t.n // B)).astype(np.float32)
    return m8, ms, s8, ss


def run8(grs, t, st, hp, seed):
    d = [torch.from_numpy(np.ascontiguousarray(x)).cuda() for x in st]
    grs.grs_tensors_adamw8_step(t.h, hp, seed, t.norm.data_ptr(), t.gp.data_ptr(), t.dt, t.master.data_ptr(), d[0].data_ptr(),
                                d[1].data_ptr(), d[2].data_ptr(), d[3].data_ptr(), t.pp.data_ptr(), t.stream())
    torch.cuda.synchronize()
    return [x.cpu().numpy() for x in d]


@pytest.mark.parametrize("numels", SIZES)
@pytest.mark.parametrize("bf16,shift,seed", [(False, 0, 1), (True, 1, (1 << 63) + 12345), (True, 0, 0)])
def test_step_in_8_bits(grs, numels, bf16, shift, seed):
    skip = [2] if len(numels) > 2 else []
    t = List(grs, numels, bf16, shift, seed=4, skip=skip)
    st = random_state8(t, 5)
    p0 = t.master.cpu().numpy()
    S, step = 0.5, 40
    t.norm.fill_(S)
    hp = grs.make_adamw(*HP.values(), 1.0, step, 2)
    got = run8(grs, t, st, hp, seed)
    F = np.float32
    m0 = (e4m3(st[0]).reshape(-1, B) * st[1][:, None]).reshape(-1)
    s0 = (e4m3(st[2]).reshape(-1, B) * st[3][:, None]).reshape(-1)
    c = clip(S, 1.0)
    # master against 64 bits
    want = step64(t.g, p0, m0, s0 * s0, step, c, 2)
    p = t.master.cpu().numpy()
    assert (np.abs(p - want[0])[t.live] <= ATOL + RTOL * np.abs(want[0][t.live])).all()
    assert np.array_equal(t.params()[t.live], torch.from_numpy(p).to(torch.bfloat16).float().numpy()[t.live])
    # the moments in float32, rounding by rounding
    gscale = F(F(1.0) / F(np.sqrt(F(S)) + F(1e-6)))
    gscale = F(min(gscale, F(1)) * F(0.5))
    g = t.g * gscale
    b1, b2 = F(HP["beta1"]), F(HP["beta2"])
    m = m0.astype(F) * b1 + g * F(1 - float(b1))
    s0 = s0.astype(F)
    s = np.sqrt(s0 * s0 * b2 + (g * F(1 - float(b2))) * g)
    m[~t.used], s[~t.used] = 0, 0
    bits = random_bits(t.n, seed)
    for x, code, scale, r16, pos in ((m, got[0], got[1], bits & 0xFFFF, False), (s, got[2], got[3], bits >> 16, True)):
        val, sc = to8(x, r16, pos)
        on = t.live | ~t.used
        if skip:
            lo = t.off[2]
            on[lo:lo + -(-numels[2] // B) * B] = False
        assert np.array_equal(e4m3(code)[on], val[on])
        assert np.array_equal(scale[on[::B]], sc[on[::B]])
    if skip:
        lo, hi = t.off[2], t.off[2] + numels[2]
        for a, b in zip(got[::2], st[::2]):
            assert np.array_equal(a[lo:hi], b[lo:hi])
    t.close()


def test_rounding_is_unbiased(grs):
    """The mean over seeds is the unrounded value, to six standard deviations of such a mean."""
    t = List(grs, [2048], seed=6)
    st = random_state8(t, 7)
    t.norm.fill_(1e-6)
    hp = grs.make_adamw(*HP.values(), 0.0, 40, 1)
    K = 400
    sums = [np.zeros(t.n), np.zeros(t.n)]
    for k in range(K):
        got = run8(grs, t, st, hp, 1000 + k)
        for j in range(2):
            sums[j] += (e4m3(got[2 * j]).reshape(-1, B) * got[2 * j + 1][:, None]).reshape(-1)
    m0 = (e4m3(st[0]).reshape(-1, B) * st[1][:, None]).reshape(-1)
    s0 = (e4m3(st[2]).reshape(-1, B) * st[3][:, None]).reshape(-1)
    _, m, v = step64(t.g, np.zeros(t.n), m0, s0 * s0, 40, 1.0, 1)
    for j, x in enumerate((m, np.sqrt(v))):
        unit = (got[2 * j + 1][:, None] * np.ones(B)).reshape(-1)
        y = np.abs(x) / unit
        gap = np.exp2(np.maximum(np.floor(np.log2(np.maximum(y, 2.0 ** -9))), -6) - 3) * unit
        dev = (sums[j] / K - x) / (gap / 2 / math.sqrt(K))  # a two-point variable has at most half the gap as its deviation
        keep = y > 2.0 ** -9 if j else np.ones(t.n, bool)
        assert np.abs(dev[keep]).max() < 6
        assert abs(dev[keep].mean()) < 6 / math.sqrt(keep.sum())
    t.close()


def test_moving_average_follows_a_falling_gradient(grs):
    """sqrt(v) starts 10 times too large: nearest rounding would leave every code where it is; the average has to
    follow sqrt of v's own course within 6 % (variance that rounding adds to v: about 5 %, 2.5 % of sqrt(v))."""
    n, steps = 1 << 16, 800
    t = List(grs, [n], seed=8)
    t.store[0][:n] = 1e-2
    st = [np.zeros(n, np.uint8), np.full(n // B, 2.0 ** -10, np.float32), np.full(n, 0x70, np.uint8),
          np.full(n // B, 0.1 / 128, np.float32)]
    d = [torch.from_numpy(x).cuda() for x in st]
    hp = grs.make_adamw(*HP.values(), 0.0, 1000, 1)
    for k in range(steps):
        grs.grs_tensors_adamw8_step(t.h, hp, k, None, t.gp.data_ptr(), t.dt, t.master.data_ptr(), d[0].data_ptr(), d[1].data_ptr(),
                                    d[2].data_ptr(), d[3].data_ptr(), None, t.stream())
    s = e4m3(d[2].cpu().numpy()).reshape(-1, B) * d[3].cpu().numpy()[:, None].astype(np.float64)
    a = f32(0.999) ** steps
    want = math.sqrt(0.01 * a + 1e-4 * (1 - a))
    assert abs(s.mean() / want - 1) < 0.06, (s.mean(), want)
    t.close()


def test_zero_and_tiny_and_nonfinite_blocks(grs):
    t = List(grs, [4 * B], seed=9)
    t.store[0][:4 * B] = 0
    t.store[0][B] = 1e-30           # block 1: far below everything else
    t.store[0][2 * B + 3] = float("nan")
    t.store[0][3 * B:4 * B] = 1e-2
    t.store[0][3 * B + 9] = 1e-12   # positive sqrt(v) below the smallest code
    st = [np.zeros(4 * B, np.uint8), np.zeros(4, np.float32), np.zeros(4 * B, np.uint8), np.zeros(4, np.float32)]
    hp = grs.make_adamw(*HP.values(), 0.0, 1, 1)
    got = run8(grs, t, st, hp, 3)
    p = t.master.cpu().numpy()
    assert (got[0][:B] == 0).all() and (got[2][:B] == 0).all() and np.isfinite(p[:2 * B]).all()
    assert np.isnan(got[1][2]) and np.isnan(got[3][2]) and (got[0][2 * B:3 * B] == 0).all()
    assert np.isnan(p[2 * B + 3]) and np.isfinite(np.delete(p[2 * B:3 * B], 3)).all()
    assert got[2][3 * B + 9] == 1  # never zero
    t.close()


def test_magnitudes_over_the_whole_range(grs):
    """Blocks whose moments are huge (beyond one scaling product) and tiny (at the smallest scale): the codes bit for bit."""
    factors = [1e18, 1e10, 1.0, 1e-10, 1e-18, 3e-36]
    t = List(grs, [len(factors) * B], seed=14)
    g = t.g * np.repeat(np.array(factors, np.float32), B)
    t.store[0][:t.n] = torch.from_numpy(g).cuda()
    st = [np.zeros(t.n, np.uint8), np.zeros(t.n // B, np.float32), np.zeros(t.n, np.uint8), np.zeros(t.n // B, np.float32)]
    hp = grs.make_adamw(*HP.values(), 0.0, 1, 1)
    got = run8(grs, t, st, hp, 77)
    F = np.float32
    m = g * F(1 - float(F(0.9)))
    s = np.sqrt((g * F(1 - float(F(0.999)))) * g)
    bits = random_bits(t.n, 77)
    for x, code, scale, r16, pos in ((m, got[0], got[1], bits & 0xFFFF, False), (s, got[2], got[3], bits >> 16, True)):
        val, sc = to8(x, r16, pos)
        assert np.array_equal(e4m3(code), val) and np.array_equal(scale, sc)
    assert np.isfinite(t.master.cpu().numpy()).all()
    t.close()


def test_indexes_beyond_32_bits(grs):
    """A tensor of more than 2^32 elements: its last blocks' states, whose random numbers take the high word, and its norm."""
    n = (1 << 32) + 5000
    h = grs.grs_tensors_create([n])
    info = grs.grs_tensors_query(h)
    N = info["n_state"]
    free = torch.cuda.mem_get_info()[0]
    if free < 12 * N:
        pytest.skip("needs about 52 GB of device memory")
    g = torch.zeros(N, dtype=torch.bfloat16, device="cuda")
    master = torch.zeros(N, device="cuda")
    m8, s8 = torch.zeros(N, dtype=torch.uint8, device="cuda"), torch.zeros(N, dtype=torch.uint8, device="cuda")
    ms, ss = torch.zeros(N // B, device="cuda"), torch.zeros(N // B, device="cuda")
    lo = N - 4096 - B
    tail = torch.randn(n - lo, generator=torch.Generator().manual_seed(1)).mul(1e-2).to(torch.bfloat16)
    g[lo:n] = tail.cuda()
    table = lambda x: torch.tensor([x.data_ptr()], dtype=torch.int64, device="cuda")  # noqa: E731
    gp = table(g)
    ws = torch.zeros(info["workspace_bytes"], dtype=torch.uint8, device="cuda")
    norm = torch.zeros(1, dtype=torch.float64, device="cuda")
    st = torch.cuda.current_stream().cuda_stream
    grs.grs_tensors_norm_sq(h, gp.data_ptr(), grs.GRS_DTYPE_BF16, 1, ws.data_ptr(), norm.data_ptr(), st)
    hp = grs.make_adamw(*HP.values(), 0.0, 1, 1)
    grs.grs_tensors_adamw8_step(h, hp, 5, None, gp.data_ptr(), grs.GRS_DTYPE_BF16, master.data_ptr(), m8.data_ptr(), ms.data_ptr(),
                                s8.data_ptr(), ss.data_ptr(), None, st)
    torch.cuda.synchronize()
    x = np.zeros(N - lo, np.float32)
    x[:n - lo] = tail.float().numpy()
    want = float(np.sum(x.astype(np.float64) ** 2))
    assert abs(float(norm.cpu()[0]) - want) <= 22 * 2.0 ** -24 * want
    idx = np.arange(lo, N, dtype=np.uint64)
    k0 = mix(5 + 0x9E3779B9 & 0xFFFFFFFF)
    k1 = mix(k0)
    y = (idx & np.uint64(0xFFFFFFFF)) ^ np.uint64(k0) ^ ((idx >> np.uint64(32)) * np.uint64(0x6A09E667) & np.uint64(0xFFFFFFFF))
    y = ((y ^ y >> np.uint64(16)) * np.uint64(0x9E3779B9) & np.uint64(0xFFFFFFFF)) ^ np.uint64(k1)
    y = (y ^ y >> np.uint64(15)) * np.uint64(0xBB67AE85) & np.uint64(0xFFFFFFFF)
    bits = (y ^ y >> np.uint64(16)).astype(np.int64)
    F = np.float32
    m = x * F(1 - float(F(0.9)))
    s = np.sqrt((x * F(1 - float(F(0.999)))) * x)
    for v, code, scale, r16, pos in ((m, m8, ms, bits & 0xFFFF, False), (s, s8, ss, bits >> 16, True)):
        val, sc = to8(v, r16, pos)
        assert np.array_equal(e4m3(code[lo:].cpu().numpy()), val)
        assert np.array_equal(scale[lo // B:].cpu().numpy(), sc)
    want = step64(x, np.zeros(N - lo), np.zeros(N - lo), np.zeros(N - lo), 1, 1.0, 1)[0]
    assert np.abs(master[lo:].cpu().numpy() - want).max() <= ATOL + RTOL * np.abs(want).max()
    assert int(m8[:lo].max()) == 0 and float(master[:1 << 20].abs().max()) == 0
    grs.grs_tensors_destroy(h)
    del g, master, m8, s8
    torch.cuda.empty_cache()


def test_only_empty_tensors(grs):
    t = List(grs, [0, 0])
    t.norm.fill_(5.0)
    grs.grs_tensors_norm_sq(t.h, t.gp.data_ptr(), t.dt, 1, t.ws.data_ptr(), t.norm.data_ptr(), t.stream())
    assert float(t.norm.cpu()[0]) == 0.0
    hp = grs.make_adamw(*HP.values(), 1.0, 1, 1)
    x = torch.zeros(16, device="cuda").data_ptr()
    grs.grs_tensors_adamw_step(t.h, hp, t.norm.data_ptr(), t.gp.data_ptr(), t.dt, x, x, x, t.pp.data_ptr(), t.stream())
    grs.grs_tensors_adamw8_step(t.h, hp, 1, t.norm.data_ptr(), t.gp.data_ptr(), t.dt, x, x, x, x, x, t.pp.data_ptr(), t.stream())
    t.close()


@pytest.mark.parametrize("numels", SIZES)
def test_pack_and_unpack(grs, numels):
    t = List(grs, numels, seed=10)
    m, v = t.fill(1e-3), t.fill(1e-3, square=True)
    m8, s8 = (torch.full((t.n,), 0xFF, dtype=torch.uint8, device="cuda") for _ in range(2))
    ms, ss = (torch.zeros(t.n // B, device="cuda") for _ in range(2))
    m2, v2 = torch.empty_like(m), torch.empty_like(v)
    pack = lambda a, b: grs.grs_tensors_pack8(t.h, a.data_ptr(), b.data_ptr(), m8.data_ptr(), ms.data_ptr(), s8.data_ptr(), ss.data_ptr(), t.stream())  # noqa: E731
    unpack = lambda a, b: grs.grs_tensors_unpack8(t.h, m8.data_ptr(), ms.data_ptr(), s8.data_ptr(), ss.data_ptr(), a.data_ptr(), b.data_ptr(), t.stream())  # noqa: E731
    pack(m, v)
    unpack(m2, v2)
    for x, y, sc in ((m, m2, ms), (v.sqrt(), v2.sqrt(), ss)):
        x, y = x.cpu().numpy(), y.cpu().numpy()
        unit = np.repeat(sc.cpu().numpy(), B)
        assert (y[~t.used] == 0).all()
        x, y, unit = x[t.used], y[t.used], unit[t.used]
        # nearest of 4 significant bits: 2^-4 of the value; half a unit of the last place, 2^-10, below the normal range;
        # a positive sqrt(v) may be lifted to the smallest code 2^-9
        assert (np.abs(x - y) <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -9 * unit) * (1 + 1e-6)).all()
    m3, v3 = torch.empty_like(m), torch.empty_like(v)
    pack(m2, v2)
    unpack(m3, v3)
    torch.cuda.synchronize()
    assert torch.equal(m2, m3) and torch.equal(v2, v3)
    t.close()


def test_8_bit_training_follows_32_bits(grs):
    """A quadratic bowl: both forms reach its bottom."""
    n = 5000
    target = torch.randn(n, device="cuda", generator=torch.Generator(device="cuda").manual_seed(3))
    left = {}
    for form in (32, 8):
        t = List(grs, [n], seed=11)
        w = t.pstore[0][:n]
        w.copy_(t.master[:n])
        m, v = torch.zeros(t.n, device="cuda"), torch.zeros(t.n, device="cuda")
        m8, s8 = torch.zeros(t.n, dtype=torch.uint8, device="cuda"), torch.zeros(t.n, dtype=torch.uint8, device="cuda")
        ms, ss = torch.zeros(t.n // B, device="cuda"), torch.zeros(t.n // B, device="cuda")
        for k in range(1, 301):
            t.store[0][:n] = w.float() - target
            hp = grs.make_adamw(1e-2, 0.9, 0.999, 1e-8, 0.0, 0.0, k, 1)
            if form == 32:
                grs.grs_tensors_adamw_step(t.h, hp, None, t.gp.data_ptr(), t.dt, t.master.data_ptr(), m.data_ptr(), v.data_ptr(),
                                           t.pp.data_ptr(), t.stream())
            else:
                grs.grs_tensors_adamw8_step(t.h, hp, k, None, t.gp.data_ptr(), t.dt, t.master.data_ptr(), m8.data_ptr(), ms.data_ptr(),
                                            s8.data_ptr(), ss.data_ptr(), t.pp.data_ptr(), t.stream())
        left[form] = float((t.master[:n] - target).square().mean())
        t.close()
    assert left[32] < 0.05 and left[8] < 2 * left[32] + 0.01, left


def test_refusals(grs):
    t = List(grs, [600], seed=12)
    hp = grs.make_adamw(*HP.values(), 1.0, 1, 1)
    ok = t.master.data_ptr()
    gp, norm, s = t.gp.data_ptr(), t.norm.data_ptr(), t.stream()
    bad_step = grs.make_adamw(*HP.values(), 1.0, 0, 1)
    bad_micro = grs.make_adamw(*HP.values(), 1.0, 1, 0)
    step = lambda hp=hp, n=norm, g=gp, dt=t.dt, p=ok, m=ok, v=ok, pp=None: grs.grs_tensors_adamw_step(t.h, hp, n, g, dt, p, m, v, pp, s)  # noqa: E731
    step8 = lambda m8=ok, ms=ok, s8=ok, ss=ok, n=norm: grs.grs_tensors_adamw8_step(t.h, hp, 1, n, gp, t.dt, ok, m8, ms, s8, ss, None, s)  # noqa: E731
    inv, ali = grs.GRS_ERR_INVALID_ARG, grs.GRS_ERR_ALIGNMENT
    for call, status in ((lambda: step(hp=bad_step), inv), (lambda: step(hp=bad_micro), inv), (lambda: step(n=None), inv),
                         (lambda: step(g=None), inv), (lambda: step(dt=2), inv), (lambda: step(dt=-1), inv),
                         (lambda: step(p=None), inv), (lambda: step(m=None), inv), (lambda: step(p=ok + 4), ali),
                         (lambda: step(v=ok + 8), ali), (lambda: step(g=gp + 4), ali), (lambda: step(pp=gp + 2), ali),
                         (lambda: step8(m8=None), inv), (lambda: step8(ss=None), inv), (lambda: step8(s8=ok + 8), ali),
                         (lambda: step8(ms=ok + 2), ali), (lambda: step8(n=norm + 4), ali),
                         (lambda: grs.grs_tensors_norm_sq(t.h, gp, 7, 1, t.ws.data_ptr(), norm, s), inv),
                         (lambda: grs.grs_tensors_norm_sq(t.h, gp, 0, 0, t.ws.data_ptr(), norm, s), inv),
                         (lambda: grs.grs_tensors_norm_sq(t.h, gp, 0, 1, t.ws.data_ptr() + 8, norm, s), ali),
                         (lambda: grs.grs_tensors_pack8(t.h, ok, None, ok, ok, ok, ok, s), inv),
                         (lambda: grs.grs_tensors_unpack8(t.h, ok, ok, ok, ok, ok + 4, ok, s), ali)):
        with pytest.raises(grs.GrsError) as e:
            call()
        assert e.value.status == status
    t.close()


def test_on_another_stream(grs):
    """The work goes to the given stream: after an event on it, the results are there."""
    t = List(grs, [30000], seed=13)
    m, v = torch.zeros(t.n, device="cuda"), torch.zeros(t.n, device="cuda")
    p0 = t.master.cpu().numpy()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    hp = grs.make_adamw(*HP.values(), 1.0, 1, 1)
    grs.grs_tensors_norm_sq(t.h, t.gp.data_ptr(), t.dt, 1, t.ws.data_ptr(), t.norm.data_ptr(), side.cuda_stream)
    grs.grs_tensors_adamw_step(t.h, hp, t.norm.data_ptr(), t.gp.data_ptr(), t.dt, t.master.data_ptr(), m.data_ptr(), v.data_ptr(),
                               None, side.cuda_stream)
    side.synchronize()
    S = float(np.sum(t.g.astype(np.float64) ** 2))
    want = step64(t.g, p0, np.zeros(t.n), np.zeros(t.n), 1, clip(S, 1.0), 1)[0]
    got = t.master.cpu().numpy()
    assert (np.abs(got - want)[t.used] <= ATOL + RTOL * np.abs(want[t.used])).all()
    t.close()
