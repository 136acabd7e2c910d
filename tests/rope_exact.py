"""Rotation plans and angles in 70 decimal digits."""
import math
from decimal import Decimal, getcontext

getcontext().prec = 70
PI = Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899862803")


def turns(rot, theta, scaling="none", factor=1.0, original=0.0, low=1.0, high=4.0):
    """Turns per position of each pair, as the header defines them."""
    ln = Decimal(theta).ln()
    f = [(-ln * 2 * i / rot).exp() for i in range(rot // 2)]
    fac = Decimal(factor)
    if scaling == "linear":
        f = [x / fac for x in f]
    elif scaling == "yarn":
        at = lambda t: rot * math.log(original / (t * 2 * math.pi)) / (2 * math.log(theta))  # noqa: E731
        a, b = max(math.floor(at(high)), 0), min(math.ceil(at(low)), rot - 1)
        span = Decimal(b - a) if b > a else Decimal("0.001")
        m = [min(max((i - a) / span, Decimal(0)), Decimal(1)) for i in range(rot // 2)]
        f = [x * (1 - t) + x / fac * t for x, t in zip(f, m)]
    elif scaling == "wavelength":
        lo, hi = Decimal(low), Decimal(high)
        m = [min(max((Decimal(original) * x / (2 * PI) - lo) / (hi - lo), Decimal(0)), Decimal(1))
             for x in f]
        f = [x * t + x / fac * (1 - t) for x, t in zip(f, m)]
    return [x / (2 * PI) for x in f]


def rows(positions, t):
    """[(cos, sin)] per position and pair, right to 64 bits."""
    out = []
    for pos in positions:
        row = []
        for x in t:
            y = x * int(pos)
            a = float((y - y.to_integral_value()) * 2 * PI)
            row.append((math.cos(a), math.sin(a)))
        out.append(row)
    return out
