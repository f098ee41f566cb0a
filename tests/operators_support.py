"""Helpers of the tests of the experts' products, the embedding and the query
and key norms: types, half steps of rounding, comparison element by element."""
import torch

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def binding():
    from gradient_reduction_sharded_gb300 import grs
    return grs


def dtype_code(name):
    return {"bf16": binding().GRS_DTYPE_BF16, "fp32": binding().GRS_DTYPE_FP32}[name]


def stream():
    return torch.cuda.current_stream().cuda_stream


def half(name):
    """Relative error of one rounding to the type."""
    return torch.finfo(DT[name]).eps / 2


def ptr(t):
    return None if t is None else t.data_ptr()


def close(got, want, limit, what):
    """got (rounded) within `limit` (64-bit tensor of absolute errors) of want (64 bits)."""
    off = (got.double() - want).abs()
    bad = ~(off <= limit)
    assert not bool(bad.any()), (what, int(bad.sum()), float((off - limit).nan_to_num(float("inf")).max()), bad.nonzero()[:4].tolist())
