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
