"""GPU tests of SiLU over its whole range, behind the convolution and as the norm's gate.

y e^y is a normal number of either format down to about -91 and subnormal below. The activation itself is
good to 2^-16 (bf16, 2^-17 from -80 on) and, with the library's exponential (1 ulp, 2^-23, taken twice below
-80) and three more roundings, to 2^-21 (fp32); the norm's mean square, root and two products put
8 2^-24 more. Results below the smallest normal number, 2^-126, may lose their bits."""
from __future__ import annotations

import numpy as np
import pytest

import prompt_ref as ref
from test_gpu_prompt import HALF, _close, _code, _dt, _np, _rrs

pytestmark = pytest.mark.gpu

OWN = {"bf16": 2.0 ** -16, "f32": 2.0 ** -21}


def _arguments(torch, dtype):
    """-130 .. 130, dense around the place where e^-y leaves fp32."""
    y = torch.cat([torch.linspace(-130, 130, 4096), torch.linspace(-93, -79, 4096)])
    return y.to(_dt(torch, dtype)).cuda()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_convolution(dtype):
    rrs, torch = _rrs()
    x = _arguments(torch, dtype).view(8, 1024)
    w = torch.zeros(2, 1024, device="cuda")
    w[1] = 1  # the sum is the row itself, exactly
    want = ref.silu(_np(x))
    tol = (HALF[dtype] + OWN[dtype]) * np.abs(want) + 2.0 ** -126
    conv = rrs.make_conv(8, 1024, 2, _code(rrs, dtype))
    y, win = torch.empty_like(x), torch.zeros(8, 1, 1024, dtype=x.dtype, device="cuda")
    rrs.seed_decode_conv(conv, x, w, None, win, y)
    _close(_np(y), want, tol)
    off = torch.arange(9, dtype=torch.int32, device="cuda")
    rrs.seed_prefill_conv(conv, x, off, w, None, win, y)
    _close(_np(y), want, tol)
    odd = x[:, 1:1000].contiguous()
    y = torch.empty_like(odd)
    rrs.seed_decode_conv(rrs.make_conv(8, 999, 2, _code(rrs, dtype)), odd, w[:, 1:1000].contiguous(), None,
                         torch.zeros(8, 1, 999, dtype=x.dtype, device="cuda"), y)
    _close(_np(y), want[:, 1:1000], tol[:, 1:1000])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim", [64, 63])
def test_gate_of_the_norm(dtype, dim):
    rrs, torch = _rrs()
    z = _arguments(torch, dtype)[:128 * dim].view(16, 8, dim) if dim == 64 else _arguments(torch, dtype)[-128 * dim:].view(16, 8, dim)
    x, w = torch.ones_like(z), torch.ones(8, dim, device="cuda")
    y = torch.empty_like(z)
    rrs.seed_norm_rows(x, w, y, gate=z, eps=0.0)
    want, _, mag = ref.norm_rows(_np(x), _np(w), _np(z), 0.0, False, None, None)
    _close(_np(y), want, HALF[dtype] * np.abs(want) + (OWN[dtype] + 2.0 ** -21) * mag + 2.0 ** -126)
