"""The polynomials behind the rotary angles, checked on the CPU: the coefficients
in the kernel source are the Chebyshev interpolants that its comment names, and
the kernel's steps replayed in float32 stay within 1.1e-7 of cos and sin at
phases all around the turn, the borders between quarters among them."""
import os
import re

import numpy as np
from numpy.polynomial import chebyshev, polynomial

SRC = os.path.join(os.path.dirname(__file__), "..", "sparse_attention_diffusion_mcs_b200", "csrc", "rotary.cuh")


def coefficients():
    body = open(SRC).read()
    fn = body[body.index("void turn_sincos("):]
    fn = fn[:fn.index("\n}\n")]
    v = [float(x) for x in re.findall(r"(-?[0-9]\.[0-9]{9}e[-+][0-9]+)f", fn)]
    assert len(v) == 8
    return np.array([v[3], v[2], v[1], v[0]]), np.array([v[7], v[6], v[5], v[4]])


def interpolant(f):
    n = 400
    k = np.cos(np.pi * (np.arange(n) + 0.5) / n)
    p = chebyshev.cheb2poly(chebyshev.chebfit(k, f((k + 1) / 32), 3))       # in k = 32 z - 1
    out, power = np.zeros(1), np.ones(1)
    for a in p:
        out, power = polynomial.polyadd(out, a * power), polynomial.polymul(power, [-1.0, 32.0])
    return out


def test_coefficients_are_the_interpolants():
    s, c = coefficients()
    np.testing.assert_allclose(s, interpolant(lambda z: np.sin(np.pi * np.sqrt(z)) / np.sqrt(z)), rtol=1e-6)
    np.testing.assert_allclose(c, interpolant(lambda z: (np.cos(np.pi * np.sqrt(z)) - 1) / z), rtol=1e-6)


def test_replayed_steps_are_within_the_bound():
    s, c = (v.astype(np.float32) for v in coefficients())
    f32 = np.float32
    fma = lambda a, b, k: (a.astype(np.float64) * b + k).astype(f32)
    rng = np.random.default_rng(0)
    near = np.arange(-64, 64, dtype=np.int64)
    phase = np.concatenate([rng.integers(0, 2 ** 32, 400_000)] + [e * 2 ** 29 + near for e in range(8)]) % 2 ** 32
    q = ((phase + 2 ** 29) % 2 ** 32) >> 30
    r = (phase - (q << 30)) % 2 ** 32
    r = np.where(r >= 2 ** 31, r - 2 ** 32, r)
    assert np.abs(r).max() <= 2 ** 29
    x = r.astype(f32) * f32(2.0 ** -31)
    z = x * x
    u = fma(fma(fma(z, s[3], s[2]), z, s[1]), z, s[0]) * x
    v = fma(fma(fma(fma(z, c[3], c[2]), z, c[1]), z, c[0]), z, 1.0)
    a, b = np.where(q & 1, u, v), np.where(q & 1, v, u)
    cos, sin = np.where((q + 1) & 2, -a, a), np.where(q & 2, -b, b)
    t = phase * (np.pi / 2 ** 31)
    assert np.abs(cos - np.cos(t)).max() <= 1.1e-7
    assert np.abs(sin - np.sin(t)).max() <= 1.1e-7
