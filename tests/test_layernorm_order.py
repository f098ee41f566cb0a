"""The order in which dw and db of wide rows are added up: fixed by the shape,
not by what a device says of itself."""
import glob
import os

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_no_launch_asks_the_device_how_much_it_holds():
    """A grid that depends on the answer changes the order of sums from one device to another."""
    for path in glob.glob(os.path.join(ROOT, "gradient_reduction_sharded_gb300", "csrc", "kernels_l*.cu")) + \
            glob.glob(os.path.join(ROOT, "gradient_reduction_sharded_gb300", "csrc", "kernels_moe.cu")):
        with open(path) as f:
            src = f.read()
        for call in ("cudaOccupancy", "cudaGetDeviceProperties", "cudaDeviceGetAttribute", "multiProcessorCount"):
            assert call not in src, (path, call)


def parts_of(rows, cols, act):
    """Clusters, and so parts, of a wide matrix."""
    e = 16 if act == "bf16" else 8
    peers = 2
    while peers * 512 * e < cols:
        peers *= 2
    span = -(-(-(-cols // 8)) // peers) * 8
    threads = -(-(-(-span // e)) // 32) * 32
    at_once = 1 if act == "bf16" else 3 if threads <= 320 else 2
    return min(rows, {2: (76, 152, 228), 4: (36, 74, 110), 8: (15, 36, 51)}[peers][at_once - 1])


def db32(dy, n):
    """db as n parts of the rows k, k + n, ... and the sum of the parts, addition by addition in fp32."""
    rows, cols = dy.shape
    parts = torch.zeros(n, cols, device=dy.device)
    for r in range(0, rows, n):
        take = dy[r:r + n].float()
        parts[:len(take)] += take
    blocks = -(-2 * cols // 32)
    warps = 32 if blocks <= 152 or n > 160 else 16 if n > 80 else 8
    s = torch.zeros(warps, cols, device=dy.device)
    for k in range(0, n, warps):
        take = parts[k:k + warps]
        s[:len(take)] += take
    if warps == 32:
        for o in (16, 8, 4, 2, 1):
            s = s + s[torch.arange(32, device=s.device) ^ o]
        return s[0]
    out = s[0].clone()
    for k in range(1, warps):
        out += s[k]
    return out


@pytest.mark.gpu
@pytest.mark.parametrize("rows,cols,act", [(300, 8200, "bf16"), (500, 16384, "bf16"), (1000, 20000, "bf16"), (150, 65536, "bf16"), (90, 40008, "bf16"),
                                           (700, 4104, "fp32"), (1500, 8192, "fp32"), (400, 12000, "fp32"), (333, 16384, "fp32"), (200, 20000, "fp32"),
                                           (150, 32768, "fp32"), (10, 16384, "fp32")])
def test_db_is_added_up_in_the_order_of_the_shape(rows, cols, act):
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from gradient_reduction_sharded_gb300 import grs
    g = torch.Generator(device="cuda").manual_seed(rows + cols)
    dt = torch.bfloat16 if act == "bf16" else torch.float32
    x, dy = (torch.randn(rows, cols, generator=g, device="cuda").to(dt) for _ in range(2))
    mean, rstd = torch.zeros(rows, device="cuda"), torch.ones(rows, device="cuda")
    code = grs.GRS_DTYPE_BF16 if act == "bf16" else grs.GRS_DTYPE_FP32
    s = grs.make_norm(rows, cols, 1e-5, code, code, grs.GRS_DTYPE_FP32)
    ws = torch.empty(grs.grs_layernorm_workspace_bytes(s), dtype=torch.uint8, device="cuda")
    dw, db, dx = torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda"), torch.empty_like(x)
    want = db32(dy, parts_of(rows, cols, act))
    for out in (dx.data_ptr(), None):
        grs.grs_layernorm_backward(s, dy.data_ptr(), x.data_ptr(), None, mean.data_ptr(), rstd.data_ptr(), out, dw.data_ptr(), db.data_ptr(),
                                   ws.data_ptr(), torch.cuda.current_stream().cuda_stream)
        assert torch.equal(db, want)
