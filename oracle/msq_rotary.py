"""Plain oracle of rotary positions (numpy): the angle in fp64, its cosine and sine in fp64 times
the amplitude and rounded to fp32, then fp32 with one rounding an operation."""
from __future__ import annotations

import numpy as np

F32 = np.float32


def pairs(dims, interleaved):
    """(first, second) dims of the pairs."""
    i = np.arange(dims // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + dims // 2)


def rotate(x, positions, freq, interleaved=False, amplitude=1.0):
    """x [rows][heads][dim] as fp32, positions [rows], freq fp64 [dims / 2]: fp32."""
    x = np.asarray(x, F32)
    angle = np.asarray(positions, np.float64)[:, None] * np.asarray(freq, np.float64)
    c, s = (F32(amplitude * f(angle))[:, None, :] for f in (np.cos, np.sin))
    lo, hi = pairs(2 * len(freq), interleaved)
    a, b = x[..., lo], x[..., hi]
    y = x.copy()
    with np.errstate(invalid="ignore", over="ignore"):
        y[..., lo] = (a * c) - (b * s)
        y[..., hi] = (b * c) + (a * s)
    return y


def rotate64(x, positions, freq, interleaved=False, amplitude=1.0):
    """The same in fp64 throughout, by complex numbers."""
    x = np.asarray(x, np.float64)
    lo, hi = pairs(2 * len(freq), interleaved)
    z = (x[..., lo] + 1j * x[..., hi]) * (amplitude * np.exp(1j * np.outer(positions, freq)))[:, None, :]
    y = x.copy()
    y[..., lo], y[..., hi] = z.real, z.imag
    return y
