"""The range of eps of ula_norm_rotate: refused outside of it (on the host, without a GPU), and right at its ends."""

import ctypes

import numpy as np
import pytest

from serving_pb_lru_amd import ula
from test_norm_weigh_lightest_refusals import EINVAL, norm_args


@pytest.mark.parametrize("eps", [2.0 ** -127, 2.0 ** -149, 2.0 ** -126 * (1 - 2.0 ** -23), 2.0 ** 96 * (1 + 2.0 ** -23), 3e38])
def test_refused(eps):
    assert ula.lib().ula_norm_rotate(ctypes.byref(norm_args(eps=eps)), 0) == EINVAL


def test_taken():
    for eps in (2.0 ** -126, 2.0 ** 96):               # an empty call, which has its arguments checked
        args = norm_args(eps=eps, n=0)
        assert ula.lib().ula_norm_rotate(ctypes.byref(args), 0) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dim", [64, 6, 256])
@pytest.mark.parametrize("eps", [2.0 ** -126, 2.0 ** -100, 2.0 ** 40, 2.0 ** 96])
def test_rows_around_the_root_of_eps(dim, eps):
    """Rows far below the root of eps, around it and far above, up to squares that overflow. Tolerance of
    test_norm_gpu.py: squares below 2^-126 add at most 2^-150 each to the mean, 2^-24 of the least eps, halved by the
    root, and an overflowing row's mean is 2^24 times the largest eps; results below 2^-126 have steps of 2^-149."""
    import torch
    from serving_pb_lru_amd import norm_rotate
    from test_norm_gpu import wanted
    from test_rows_gpu import assert_within, f64
    rng = np.random.default_rng([dim, int(np.log2(eps)) + 200])
    at = np.log2(eps) / 2
    size = np.array([s for s in at + np.array([-40, -14, -12, -6, -2, 0, 2, 13, 40, 80]) if s < 120] + [63.0, 110.0, 120.0])
    x = (rng.standard_normal((1, len(size), dim)) * 2.0 ** size[None, :, None]).astype(np.float32)
    got = f64(norm_rotate(torch.from_numpy(x).cuda(), eps=eps)[0])
    want, tol = wanted(x.astype(np.float64), None, eps, None, None, 0, 1.0, False, "fp32")
    assert_within(got, want, tol + 2.0 ** -148)
