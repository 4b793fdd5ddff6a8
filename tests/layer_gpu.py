"""Helpers of the GPU tests of the operators around the recurrence: seeded inputs rounded to the
storage type on the host, so that the float64 oracle sees the device's values, and the error
measures. Tolerances count roundings: one of bfloat16 is at most 2^-8 of the value, one of float32
2^-24."""
import numpy as np

HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def torch_dtype(dtype):
    import torch

    return torch.bfloat16 if dtype == "bf16" else torch.float32


def rounded(a, dtype):
    import torch

    return torch.from_numpy(np.ascontiguousarray(a)).float().to(torch_dtype(dtype)).double().numpy()


def dev(a, dtype="f32"):
    """a as a GPU tensor of the storage type (its values are already rounded)."""
    import torch

    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).float().to(torch_dtype(dtype)).cuda()


def host(t):
    return None if t is None else t.double().cpu().numpy()


def rel(a, b):
    """2-norm of the difference over that of b."""
    a, b = np.asarray(a, np.float64).reshape(-1), np.asarray(b, np.float64).reshape(-1)
    assert a.shape == b.shape
    n = float(np.linalg.norm(b))
    d = float(np.linalg.norm(a - b))
    return d / n if n > 0 else d


def cu_of(lens):
    return [int(v) for v in np.concatenate([[0], np.cumsum(lens)])]
