"""The gated product's activations in 64 bits, and the bound of their fp32 steps: with u = 2^-24 a relative
(1.3 |g| w + 6) u for silu and (7.3 |t| w + 6) u for gelu, t = 2 sqrt(2 / pi) (g + 0.044715 g^3) and
w = 1 / (1 + e^t), from the roundings of the exponent (of the constant and the product 1.3, of t 6), of the
exponential and the reciprocal (2 each) and of the sum and the product; below |g| 2^-126 nothing may be left.
A result below fp32's normal numbers is rounded to its subnormals, whose half step is 2^-150 whatever the value:
u relative counts the last product's rounding only above 2^-126."""
import math

import numpy as np

U = 2.0 ** -24


def activation(g, kind):
    """(act(g), bound of its fp32 value) of fp64 g."""
    t = g if kind == "silu" else 2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)
    with np.errstate(over="ignore"):
        a = g / (1 + np.exp(-t))
        w = 1 / (1 + np.exp(t))
    steps = (1.3 if kind == "silu" else 7.3) * np.abs(t) * w + 6
    return a, 1.001 * steps * U * np.abs(a) + np.abs(g) * 2.0 ** -126 + 2.0 ** -150
