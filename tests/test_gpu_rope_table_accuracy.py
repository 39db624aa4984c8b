"""Accuracy of the rotary table relative to its values, and of negative frequencies."""
import math
from decimal import Decimal, getcontext

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def da():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from split_kv_decode_attention_gb300 import binding as B
    from split_kv_decode_attention_gb300 import build as cuda_build
    cuda_build.build()
    B.lib()
    return B


# What the kernel rounds, in units of 2^-24.  The remainder's angle x: its sum, 2 pi /
# 2^64 and their product, 1 each.  Into sin x these 3 go at most as they are (x cot x <=
# 1), into cos x by x tan x <= pi / 4: 2.4.  The polynomial's inner part is at most a
# tenth (sine) or 0.41 (cosine) of the value and takes four roundings: 0.4 or 1.7.  The
# last step 1, the amplitude's product 1.  At most 6.1 in all; the truncated series and
# the terms of second order are a tenth.  The angle itself: F is half a unit of 2^-64
# turns off, once per position (and its fp64 terms a little), and the low word's 32 bits
# become 24, up to 2^7 such units near a zero crossing.
RELATIVE = 6.5 * 2.0 ** -24


def phase_error(pos):
    return 2 * math.pi * (abs(pos) * 2.0 ** -65 * 1.25 + 2.0 ** -56)


PI = Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899")


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("first,count", [(0, 1200), (131072 - 300, 300), ((1 << 24) + 7, 200), ((1 << 31) - 100, 100)])
def test_relative_error(da, first, count, sign):
    getcontext().prec = 70
    f = torch.tensor([1.0, 0.7310585786300049, 0.1, 3.0e-3, 3.0e-5, 7.1e-7, 2.5, 1e-9], dtype=torch.float64)
    out = da.rope_table((sign * f).cuda(), count, first=first).cpu().double()
    n = f.numel()
    for i, x in enumerate(f.tolist()):
        a = [float((Decimal(first + r) * Decimal(x)) % (2 * PI)) for r in range(count)]
        a = torch.tensor(a, dtype=torch.float64)
        for col, want in ((i, a.cos()), (n + i, sign * a.sin())):
            # (the reference's angle is rounded to 53 bits)
            tol = RELATIVE * want.abs() + phase_error(first + count) + a * 2.0 ** -53 + 2.0 ** -60
            over = (out[:, col] - want).abs() - tol
            assert bool((over <= 0).all()), (x, col, int(over.argmax()), float(over.max()))
