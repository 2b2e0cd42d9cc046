"""Edges of the operators beside the GEMV: what a caller can hand them that the
plain cases of test_operators.py do not, against the same 64-bit forms. GPU
tests need a B200."""
import ctypes

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import quantized_gemv_stagq_b200 as Q
from tests import operator_oracle as R
from tests.test_operators import BF16, EFORMAT, EINVAL, F16, F32, Case, assert_rounded, rnd

gpu = pytest.mark.gpu


# ------------------------------------------------------------------- masses

@gpu
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("tokens", [2, 40, 700])
def test_a_query_that_is_not_finite_spoils_no_mass_that_it_does_not_see(tokens, bad):
    # the oldest of three new tokens, one of KV head 0's two query heads: it
    # does not see the last two positions, whose masses come from the others
    c = Case([tokens, 5], 2, 128, 16, 64, F16)
    q = rnd((6, 4 * 128), 3, F16)
    q[0, 128 + 7] = bad
    mass = torch.zeros(2, 2, c.width * 16, device="cuda")
    out = c.attend(q.cuda(), 3, mass).view(2, 3, 4, 128).cpu()
    clean = q.clone()
    clean[0, 128 + 7] = 0
    want, p, bound, p_bound = R.attention(clean.view(2, 3, 4, 128), c.k, c.v, c.lens_l, 3, 128 ** -0.5)
    seen = max(tokens - 2, 0)
    if seen:
        assert torch.isnan(out[0, 0, 1]).all() and torch.isnan(mass[0, 0, :seen]).all()
    else:
        assert not out[0, 0, 1].any()
    others = torch.ones(2, 3, 4, dtype=torch.bool)
    others[0, 0, 1] = False
    assert_rounded(out[others], want[others], F16, bound[others][:, None])
    got = mass.double().cpu()
    for b, h, lo in ((0, 0, seen), (0, 1, 0), (1, 0, 0), (1, 1, 0)):
        n = c.lens_l[b]
        assert ((got[b, h, lo:n] - p[b, h, lo:n]).abs() <= p_bound[b, h, lo:n] + 2.0 ** -24 * p[b, h, lo:n]).all(), (b, h)
        assert not got[b, h, n:].any()
    Q.stagq_ops_check(0)
