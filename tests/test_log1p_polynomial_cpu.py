"""The polynomial that stands for log1p(w) / w in the scan's softplus, with its coefficients as the source has them."""
import os
import re

import numpy as np

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "linear_recurrence_sequence_gb300", "csrc",
                      "ssm.cuh")


def _coefficients():
    m = re.search(r"kLog1p\[10\] = \{([^}]*)\}", open(SOURCE).read())
    c = [np.float32(v.strip().rstrip("f")) for v in m.group(1).split(",")]
    assert len(c) == 10
    return c


def test_within_the_stated_error():
    stated = re.search(r"log1p\(w\) / w on \[0, 1\] within ([0-9.e+-]+) of itself", open(SOURCE).read())
    assert stated, "the source states the polynomial's error"
    c = [float(v) for v in _coefficients()]   # FP32 values, evaluated in 64 bits
    w = np.concatenate([np.linspace(0.0, 1.0, 400001)[1:], np.logspace(-30, 0, 20001)])
    p = np.zeros_like(w)
    for v in reversed(c):
        p = p * w + v
    worst = float(np.abs(p * w / np.log1p(w) - 1.0).max())
    assert worst <= float(stated.group(1))
    assert worst >= 0.9 * float(stated.group(1))   # nor is it a looser figure than the code's


def test_the_steps_bound_has_room_for_it():
    """dt = w p(w) (+ max(r, 0)) within 2^-21, besides the rounding of the exponential's argument: the polynomial's own error;
    2^-24 of each of Horner's sums s_k, which counts w^k times; ex2's 2^-22 of w, of which log1p(w) feels the part
    w / ((1 + w) log1p(w)); and 2^-24 of the last product."""
    w = np.linspace(0.0, 1.0, 100001)[1:]
    c = [float(v) for v in _coefficients()]
    s, rounding = np.zeros_like(w), np.zeros_like(w)
    for k in range(9, -1, -1):
        s = s * w + c[k]
        rounding += 2.0 ** -24 * np.abs(s) * w ** k
    bound = 2.4e-8 + rounding / s + 2.0 ** -22 * w / ((1 + w) * np.log1p(w)) + 2.0 ** -24
    assert float(bound.max()) <= 2.0 ** -21
