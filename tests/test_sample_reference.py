"""The reference of drawing and judging against closed forms and brute force, and the kernel's arithmetic of weights, done in the same
32-bit steps on the CPU."""
import math

import numpy as np
import pytest

from tests import sample_reference as ref


def test_settings_by_hand():
    l = np.log(np.array([0.1, 0.4, 0.2, 0.2, 0.1]))
    assert np.allclose(ref.distribution(l), [0.1, 0.4, 0.2, 0.2, 0.1])
    assert np.allclose(ref.distribution(l, top_k=2), [0, 2 / 3, 1 / 3, 0, 0])  # of equal logits the lower index stays
    assert np.allclose(ref.distribution(l, top_p=0.59), [0, 2 / 3, 1 / 3, 0, 0])
    assert np.allclose(ref.distribution(l, top_p=0.61), [0, 0.5, 0.25, 0.25, 0])
    assert np.allclose(ref.distribution(l, top_p=0.0), [0, 1, 0, 0, 0])
    assert np.allclose(ref.distribution(l, min_p=0.3), [0, 0.5, 0.25, 0.25, 0])
    assert np.allclose(ref.distribution(l, temperature=0.0), [0, 1, 0, 0, 0])
    assert np.allclose(ref.distribution(l, temperature=0.5), np.array([1, 16, 4, 4, 1]) / 26)
    assert np.allclose(ref.distribution(l, top_k=3, top_p=0.7), [0, 2 / 3, 1 / 3, 0, 0])  # top_p of what top_k left: 0.5 < 0.7 <= 0.75
    assert not ref.distribution([-np.inf, np.nan]).any()
    assert np.allclose(ref.distribution([0.0, np.inf, 3.0, np.inf]), [0, 0.5, 0, 0.5])
    assert [ref.pick(np.array([0.25, 0.0, 0.5, 0.25]), u) for u in (0.0, 0.2, 0.25, 0.7, 0.75, 0.999, 1.0)] == [0, 0, 2, 2, 3, 3, 3]


def test_judging_keeps_the_targets_distribution():
    """Over all uniform numbers, what a position ends with is distributed as the target: by sums over the draft, not by drawing."""
    rng = np.random.default_rng(0)
    for _ in range(20):
        p, q = rng.dirichlet(np.ones(6)), rng.dirichlet(np.ones(6))
        q[rng.integers(6)] = 0.0
        q /= q.sum()
        out = np.zeros(6)
        for x in range(6):
            if q[x] == 0:
                continue
            accept = min(1.0, p[x] / q[x])
            out[x] += q[x] * accept
            rest = np.maximum(p - q, 0)
            out += q[x] * (1 - accept) * rest / rest.sum()
        assert np.allclose(out, p)
        x = int(rng.integers(6))
        ids, n = ref.verify([p, p], [x], [[0.0, 0.3], [0.0, 0.6]], q[None])
        assert n == (p[x] > 0) and ids[0] == (x if p[x] > 0 else ids[0]) and len(ids) == 2


def weight(l, m, temperature):
    """The kernel's weight of a token of y >= -6, in its steps: fp32 operations (a fused multiply-add rounds once), whole numbers of 2^-44."""
    f = np.float32
    c = 1.4426950408889634 / temperature
    hi = f(c)
    lo = f(c - float(hi))

    def fma(a, b, c):
        return f(np.longdouble(a) * np.longdouble(b) + np.longdouble(c))

    diff = f(l - m)
    back = f(diff - l)
    lost = f(f(l - f(diff - back)) + f(f(-m) - back))
    p = f(diff * hi)
    e = fma(lost, hi, fma(diff, lo, fma(diff, hi, -p)))
    n = int(np.rint(float(p) * 64))
    r = f(f(p - f(n / 64)) + e)
    q = f(r * fma(r, fma(r, f(0.0555041087), f(0.2402265070)), f(0.6931471806)))
    entry = 2.0 ** (28 + (n % 64) / 64)
    s = int(np.rint(entry)) + int(np.rint(float(q) * float(f(entry))))
    return s << (16 + (n // 64))


@pytest.mark.parametrize("temperature", [1.0, 0.3, 0.8, 1.7, 25.0])
def test_weights_are_exact_to_28_bits(temperature):
    rng = np.random.default_rng(1)
    t = float(np.float32(temperature))
    for _ in range(3000):
        m = np.float32(rng.normal() * 8)
        l = np.float32(m - np.float32(rng.uniform(0, 5.5 * t)))
        want = math.exp((float(l) - float(m)) / t)
        if want < 2.0**-7.9:
            continue
        # half a unit of the table's entry and of the product, of at least 2^28, the cubic's next term, and what 32 bits lose of r and q
        assert abs(weight(l, m, t) / 2.0**44 - want) <= want * (2.0**-28 + 4e-11 + 2 * 2.0**-24 * 0.0055)
    assert weight(np.float32(3.5), np.float32(3.5), t) == 1 << 44
