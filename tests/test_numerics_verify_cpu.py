"""CPU checks of the running sums behind the verification of drafts: pairs of floats, the sum and what it lost.

Units of 2^-48 of the sum (u = 2^-24 squared), worst case. An addition to a pair is exact but for the addition to its second
part, which is at most j u of the sum after j additions: j units then, (n^2 + n) / 2 over n additions. Two pairs with second
parts of up to m u together take 2 m + 1 units. A lane has its values of a run in two pairs, in windows of n = 8 kFlush additions to
each; a window's pair goes to that of all windows, which is settled (exact): (n^2 + n) / 2 + 2 n + 1, and 3 for each window, 3 for the two
together. A warp's sum takes 35 more, and what follows (running sums over the runs, a run's parts, and the tokens in a
part) 511. For 2^-38 these are at most 1024 together.

The additions are restated here in f32 from their definitions; the number of values that a pair takes is read from the source.
"""
import os
import re
from fractions import Fraction

import numpy as np
import pytest

F = np.float32
CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_ternary_matmul_gb300", "csrc", "verify.cu")
UNIT = Fraction(1, 2 ** 48)
BEHIND = 511  # units of what follows a warp's sum


@pytest.fixture(scope="module")
def flush():
    """Times 512 values of a run, 16 of a lane, 8 of each of its two pairs."""
    return int(re.search(r"constexpr int kFlush = (\d+);", open(CSRC).read()).group(1))


def add(p, w):
    h, lo = p
    s = F(h + w)
    b = F(s - h)
    return s, F(lo + F(F(h - F(s - b)) + F(w - b)))


def plus(a, b):
    lo = F(a[1] + b[1])
    h, e = add((a[0], F(0)), b[0])
    return h, F(e + lo)


def window_to(all_, p):
    s = F(all_[0] + p[0])
    b = F(s - all_[0])
    return s, F(F(F(all_[0] - F(s - b)) + F(p[0] - b)) + F(all_[1] + p[1]))


def settled(p):
    h = F(p[0] + p[1])
    return h, F(p[1] - F(h - p[0]))


def exact(p):
    return Fraction(float(p[0])) + Fraction(float(p[1]))


def lane_sum(values, flush):
    """Of a lane's values in their order, 16 of them an iteration."""
    total, pairs, n = [(F(0), F(0))] * 2, [(F(0), F(0))] * 2, 0

    def window():
        return [settled(window_to(t, p)) for t, p in zip(total, pairs)], [(F(0), F(0))] * 2
    for i in range(0, len(values), 16):
        for j, w in enumerate(values[i: i + 16]):
            pairs[j % 2] = add(pairs[j % 2], F(w))
        n += 1
        if n % flush == 0:
            total, pairs = window()
    total, pairs = window()
    return settled(plus(*total))


def warp_sum(lanes):
    n = 16
    while n:
        lanes = [plus(lanes[i], lanes[i ^ n]) for i in range(32)]
        n //= 2
    return settled(lanes[0])


def falling(n):
    """1, then n - 1 floats below half its spacing, each of which makes the second part round down by nearly half a step."""
    p, out = (F(1), F(0)), [F(1)]
    for _ in range(n - 1):
        at = Fraction(float(p[1])) + Fraction(1, 2 ** 24) * (1 - Fraction(1, 64))
        step = Fraction(2) ** (int(np.floor(np.log2(float(at)))) - 23)
        w = F(float((at // step) * step + step / 2 - Fraction(1, 2 ** 48) - Fraction(float(p[1]))))
        if not 0 < w < 2.0 ** -24:
            w = F(2.0 ** -24 * (1 - 2.0 ** -6))
        p = add(p, w)
        out.append(w)
    return out


def rows(r, flush):
    n = 8 * flush
    window = falling(n)
    yield "falling", [w for w in window for _ in range(2)]                  # both pairs
    yield "falling, many", [w for _ in range(4) for x in (window, window[::-1]) for w in x for _ in range(2)]
    yield "growing", list((2.0 ** np.linspace(-30, 0, 8 * n)).astype(F))
    yield "one large", [F(0.5)] + [F(2.0 ** -45)] * (8 * n - 1)
    for _ in range(4):
        yield "random", list(np.exp(r.randn(4 * n) * 3).astype(F))
        yield "just below half a step", list(np.where(r.rand(4 * n) < 0.02, F(1), (r.rand(4 * n) * 2.0 ** -24).astype(F)))


def test_what_a_bound_of_running_sums_leaves_for_a_lane(flush):
    n = 8 * flush
    assert (n * n + n) // 2 + (2 * n + 1) + 3 + 35 + BEHIND <= 1024, "2^-38 of the total is not held"


def test_a_lane_and_a_warp(flush):
    r, n = np.random.RandomState(1), 8 * flush
    for name, values in rows(r, flush):
        got, want = lane_sum(values, flush), sum(Fraction(float(v)) for v in values)
        windows = -(-len(values) // (2 * n)) + 1
        bound = ((n * n + n) // 2 + 2 * n + 4 + 3 * windows) * UNIT * want
        assert abs(exact(got) - want) <= bound, name
        lanes = [[F(F(2.0 ** -r.randint(0, 3)) * v) for v in values] for _ in range(32)]
        got = warp_sum([lane_sum(x, flush) for x in lanes])
        want = sum(Fraction(float(v)) for x in lanes for v in x)
        bound = ((n * n + n) // 2 + 2 * n + 4 + 3 * windows + 35) * UNIT * want
        assert abs(exact(got) - want) <= bound, name
        assert abs(exact(got) - want) <= 2 * UNIT * 512 * want, name     # 2^-38


def test_one_pair_alone(flush):
    """The additions that a pair takes, rounded down one after the other as far as they can be: within 2^-39 of their sum."""
    values = falling(8 * flush)
    p = (F(0), F(0))
    for v in values:
        p = add(p, v)
    want = sum(Fraction(float(v)) for v in values)
    assert abs(exact(p) - want) <= UNIT * 512 * want
