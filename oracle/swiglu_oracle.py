"""CPU oracle of the gated activation and its gradient (numpy, float64), with bounds of what
FP32 arithmetic may add. Test infrastructure only: it shares no code with the GPU path.

Bounds. t = e^-g is 2^(-g log2 e): the product's rounding and that of the constant put the exponent
off by at most 1.5 |g| 2^-24, ex2 adds 2^-22, the sum 1 + t 2^-24 and the reciprocal 2^-23, so
s = 1 / (1 + t) is off by e(g) = |g| 2^-23 + 2^-21 of itself, or it is below 2^-126 and 0."""
import numpy as np


def sigmoid(g):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-g))


def sigmoid_error(g):
    return np.abs(g) * 2.0 ** -23 + 2.0 ** -21


def forward(g, u):
    return g * sigmoid(g) * u


def forward_error(g, u):
    """Of FP32 arithmetic: s, two products, and the sigmoids taken as 0."""
    h = np.abs(forward(g, u))
    return h * (sigmoid_error(g) + 2.0 ** -23) + np.abs(g * u) * 2.0 ** -126 + 2.0 ** -148


def backward(g, u, dh):
    """(dg, du)."""
    s = sigmoid(g)
    return dh * u * s * (1 + g * (1 - s)), dh * g * s


def backward_error(g, u, dh):
    """Of FP32 arithmetic. 1 - s carries s's error and a rounding, 1 + g (1 - s) one more, and
    three products follow."""
    s, e = sigmoid(g), sigmoid_error(g)
    a = np.abs(1 + g * (1 - s))
    dg = np.abs(dh * u) * (s * (np.abs(g) * (s * e + 2.0 ** -24) + a * (e + 2.0 ** -22))
                           + (1 + np.abs(g)) * 2.0 ** -126)
    du = np.abs(dh * g) * (s * (e + 2.0 ** -23) + 2.0 ** -126)
    return dg + 2.0 ** -147, du + 2.0 ** -147
