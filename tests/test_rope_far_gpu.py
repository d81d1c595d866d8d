"""RoPE tables at far positions against angles in 60 decimal digits."""
import math
from decimal import Decimal, getcontext

import pytest
import torch

from looped_transformer_cross_gb300 import lla

pytestmark = pytest.mark.gpu

TWO_PI = Decimal("6.28318530717958647692528676655900576839433879875021164194988918")


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from looped_transformer_cross_gb300 import build
    build.build()


@pytest.mark.parametrize("d,base,kind,factor", [(128, 10000.0, "plain", 1.0), (64, 500000.0, "linear", 3.0)])
@pytest.mark.parametrize("pos0", [0, (1 << 20) + 1, (1 << 28) - 3, (1 << 31) - 5])
def test_far_positions(d, base, kind, factor, pos0):
    """Off by the frequency's fp64 rounding, 2^-52 of the angle, and the two functions' own 1.3 * 2^-24."""
    getcontext().prec = 60
    cos, sin = lla.rope_table_scaled(lla.dims(1, 1, 16, 16, d_head=d, rope_base=base), 5, lla.rope_scaling(kind, factor), pos0)
    for f in range(d // 2):
        theta = Decimal(base) ** (Decimal(-2 * f) / d) / Decimal(factor)
        for i in range(5):
            angle = (pos0 + i) * theta
            rest = float(angle % TWO_PI)
            tol = float(angle) * 2.0 ** -52 + 1.3 * 2.0 ** -24
            assert abs(float(cos[i, f]) - math.cos(rest)) <= tol and abs(float(sin[i, f]) - math.sin(rest)) <= tol, (f, i)
