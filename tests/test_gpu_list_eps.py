"""The 8-bit step's parameter for every eps that a caller may give: as the
32-bit step's from the same states, also where eps is below fp32's normal
numbers and all there is in the denominator."""
import math

import numpy as np
import pytest
import torch

from test_gpu_list_adamw import B, HP, List, grs, random_state8  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("eps", [1e-8, 1e-30, 2.0 ** -100, 1.2e-38, 1e-38, 1e-40, 2.0 ** -149, 1.0, 1e10])
@pytest.mark.parametrize("step", [1, 300])
def test_any_eps(grs, eps, step):  # noqa: F811
    t = List(grs, [6 * B], seed=21)
    g = t.store[0]
    g[:B] = 0                    # no gradient and no state: the parameter only decays
    g[B:2 * B] = 1e-25           # v underflows, m does not
    g[2 * B:3 * B] = -1e-22
    g[3 * B:4 * B] *= 1e15
    hp = grs.make_adamw(HP["lr"], HP["beta1"], HP["beta2"], eps, HP["weight_decay"], 0.0, step, 1)
    if step == 1:
        st = [np.zeros(t.n, np.uint8), np.zeros(t.n // B, np.float32), np.zeros(t.n, np.uint8), np.zeros(t.n // B, np.float32)]
    else:
        st = list(random_state8(t, 22))
        for x in st[::2]:
            x[:3 * B] = 0
    d = [torch.from_numpy(np.ascontiguousarray(x)).cuda() for x in st]
    m, v = torch.empty(t.n, device="cuda"), torch.empty(t.n, device="cuda")
    grs.grs_tensors_unpack8(t.h, *(x.data_ptr() for x in d), m.data_ptr(), v.data_ptr(), t.stream())
    p8, p32 = t.master.clone(), t.master.clone()
    grs.grs_tensors_adamw8_step(t.h, hp, 5, None, t.gp.data_ptr(), t.dt, p8.data_ptr(), *(x.data_ptr() for x in d), None, t.stream())
    grs.grs_tensors_adamw_step(t.h, hp, None, t.gp.data_ptr(), t.dt, p32.data_ptr(), m.data_ptr(), v.data_ptr(), None, t.stream())
    torch.cuda.synchronize()
    old, a, b = (x.double().cpu() for x in (t.master, p8, p32))
    assert torch.isfinite(b).all() and torch.isfinite(a).all()
    decay = 1 - float(np.float32(HP["lr"])) * float(np.float32(HP["weight_decay"]))
    # the quotient and its products within 2^-21 of themselves, two roundings of the parameter's size
    bound = 2.0 ** -21 * (b - old * decay).abs() + 2.0 ** -22 * torch.maximum(old.abs(), b.abs()) + 2.0 ** -149
    assert ((a - b).abs() <= bound).all(), float(((a - b).abs() - bound).max())
    assert not math.isnan(float(a.sum()))
    t.close()
