"""Rotary angles to fifty digits."""
from decimal import Decimal, getcontext
import math

PI = Decimal("3.14159265358979323846264338327950288419716939937510582")


def frequencies(n, theta):
    """theta^(-2 i / n), i < n / 2."""
    getcontext().prec = 50
    ln = Decimal(theta).ln()
    return [(-Decimal(2 * i) / Decimal(n) * ln).exp() for i in range(n // 2)]


def turn(position, frequency):
    """(cosine, sine) of the angle, reduced in fifty digits."""
    getcontext().prec = 50
    a = Decimal(position) * frequency
    a -= (a / (2 * PI)).to_integral_value() * 2 * PI
    return math.cos(float(a)), math.sin(float(a))
