"""Angles of rotary positions on the GPU against sixty decimal digits: off by what include/gk_prompt.h
says, at frequencies below and far above one, over the whole range of positions."""
import math
from decimal import Decimal, getcontext

import numpy as np
import pytest
import torch

import paged_fp8_kv_gk_gb300 as gk

pytestmark = pytest.mark.gpu
TURN = Decimal("6.28318530717958647692528676655900576839433879875021164194988918461563281257")


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    gk.lib()


@pytest.mark.parametrize("theta", [10.0, 1e4, 150000.0])
@pytest.mark.parametrize("factor", [None, 4.0, 1e-3, 1e-6, 2.5e-9])
def test_angles(theta, factor):
    getcontext().prec = 70
    pos = np.concatenate((np.arange(-3, 40), [131071, 999983, -(2 ** 20) - 1, 2 ** 31 - 1, -2 ** 31]))
    n, R = len(pos), 64
    cos, sin = (torch.empty(n, R // 2, device="cuda") for _ in range(2))
    scaling = dict(scaling="none") if factor is None else dict(scaling="linear", factor=factor)
    gk.gk_rope_table(dict(rot_dim=R, theta=theta, **scaling), torch.as_tensor(pos, dtype=torch.int32).cuda(), cos, sin)
    cos, sin = (x.double().cpu().numpy() for x in (cos, sin))
    for e in range(R // 2):
        f = (-Decimal(theta).ln() * e / (R // 2)).exp() / Decimal(1.0 if factor is None else factor)
        for i, p in enumerate(pos.tolist()):
            turns = f * p / TURN
            a = float((turns - turns.to_integral_value()) * TURN)
            slack = abs(p) * (float(f) * 2.0 ** -50 + 2.0 ** -60) + 2.0 ** -50      # and of the doubles here
            for got, want in ((cos[i, e], math.cos(a)), (sin[i, e], math.sin(a))):
                assert abs(got - want) <= slack + 2.0 ** -22 * abs(want), (e, p, got, want, slack)
