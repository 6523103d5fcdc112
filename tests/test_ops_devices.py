"""step, rms_norm and linear refuse tensors of different GPUs, and a stream of
another GPU, on the host.  The tensors here name a device and have no memory, so
the refusals are tested without a GPU."""
from __future__ import annotations

from types import SimpleNamespace

import pytest
import torch

import chunked_gated_delta_gb300 as kda

BF16, F32, I32, F8 = torch.bfloat16, torch.float32, torch.int32, torch.float8_e4m3fn


class Named(torch.Tensor):
    """A tensor of a device, shape and type, without memory."""

    @staticmethod
    def __new__(cls, shape, dtype, device="cuda:0"):
        return torch.Tensor._make_wrapper_subclass(cls, shape, dtype=dtype, device=device)

    @classmethod
    def __torch_dispatch__(cls, func, types, args=(), kwargs=None):
        raise AssertionError(f"{func} was called")


STEP = {"q": ((2, 1, 4, 64), BF16), "k": ((2, 1, 4, 64), BF16), "v": ((2, 1, 4, 64), BF16), "g": ((2, 1, 4, 64), F32),
        "beta": ((2, 1, 4), BF16), "state": ((3, 4, 64, 64), F32), "slots": ((2,), I32), "out": ((2, 1, 4, 64), BF16),
        "status": ((1,), I32)}
PACKED = dict(STEP, **{n: ((1, 2, *s[2:]), t) for n, (s, t) in STEP.items() if n in ("q", "k", "v", "g", "beta", "out")},
              cu_seqlens=((3,), I32))
NORM = {"x": ((5, 64), BF16), "weight": ((64,), BF16), "residual": ((5, 64), BF16), "out": ((5, 64), BF16),
        "residual_out": ((5, 64), BF16)}
LINEAR = {"x": ((5, 64), F8), "w": ((32, 64), F8), "bias": ((32,), F32), "residual": ((5, 32), BF16),
          "x_scale": ((5,), F32), "w_scale": ((32,), F32), "out": ((5, 32), BF16), "status": ((1,), I32)}
CALLS = {"step": (kda.step, STEP, {}), "packed step": (kda.step, PACKED, {}),
         "rms_norm": (kda.rms_norm, NORM, {}), "linear": (kda.linear, LINEAR, {"out_dtype": BF16})}


@pytest.mark.parametrize("call,other", [(c, n) for c, (_, a, _) in CALLS.items() for n in a])
def test_one_tensor_on_another_gpu(call, other):
    fn, args, kw = CALLS[call]
    given = {n: Named(shape, dtype, "cuda:1" if n == other else "cuda:0") for n, (shape, dtype) in args.items()}
    with pytest.raises(TypeError, match="on one device"):
        fn(**given, **kw)


@pytest.mark.parametrize("call", list(CALLS))
def test_a_stream_of_another_gpu(call):
    fn, args, kw = CALLS[call]
    given = {n: Named(shape, dtype) for n, (shape, dtype) in args.items()}
    with pytest.raises(TypeError, match="stream must be of the tensors' device"):
        fn(**given, **kw, stream=SimpleNamespace(cuda_stream=0, device_index=1))
