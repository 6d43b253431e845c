"""Attention with modified scores, without a GPU: what the binding refuses, and the polynomials of the cap."""
import os
import re

import numpy as np
import pytest

from transformer_encoder_bert_b200 import Scores

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "transformer_encoder_bert_b200", "csrc")


def test_a_scale_or_cap_of_zero_is_not_taken_for_the_default():
    """The struct's 0 means the default scale, or no cap: a caller's 0, or what float32 rounds to it, is refused."""
    for kw in (dict(scale=0.0), dict(scale=-0.0), dict(scale=1e-50), dict(cap=1e-50)):
        with pytest.raises(ValueError, match="zero as a float32"):
            Scores(**kw)
    assert Scores().c.scale == 0 and Scores(cap=0.0).c.cap == 0 and Scores(cap=0).c.cap == 0
    assert Scores(scale=-0.5).c.scale == -0.5


def _coefficients(text, start):
    """The float literals of the first braces after `start`."""
    body = text[text.index(start):]
    body = body[body.index("{", body.index("=")) + 1:]
    return np.array([float(x) for x in re.findall(r"-?\d+\.?\d*(?:e[+-]?\d+)?(?=f)", body[: body.index("}")])])


# (file, what the coefficients follow, how many, range, largest relative error that the comments state)
@pytest.mark.parametrize("name,start,count,top,stated", [
    ("scored.cuh", "struct TanhSmall", 5, 0.5, 2.9e-8),
    ("scored_tc.cuh", "uint64_t tanh_over_x2", 9, 1.25, 1.9e-8),
])
def test_polynomials_of_the_cap(name, start, count, top, stated):
    """tanh(x) / x in powers of x^2, evaluated in 64 bits: the largest relative error over the range is the stated one."""
    with open(os.path.join(CSRC, name)) as f:
        text = f.read()
    c = _coefficients(text, start)
    assert len(c) == count and (c == c.astype(np.float32)).all()
    x = np.linspace(1e-4, top, 200_001)
    z, p = x * x, np.full_like(x, c[-1])
    for k in c[-2::-1]:
        p = p * z + k
    worst = np.abs(p * x / np.tanh(x) - 1).max()
    assert stated * 0.98 < worst < stated * 1.03, worst
    assert f"{stated:.1e}".replace("e-0", "e-") in text
