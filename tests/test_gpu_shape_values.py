"""The repetition penalty's quotient over the whole range of fp32: one division
rounds by at most half a unit in the last place of its result (of the smallest
subnormal below the normal range); the corrected reciprocal adds at most 2^-22
of a unit to that."""

import numpy as np
import pytest
import torch

import draft_verification_amd as sdv
from tests.parity_util import to_np

pytestmark = pytest.mark.gpu

DEV = "cuda"


def _float(g, lo, hi, n):
    """n positive floats with biased exponents lo..hi."""
    bits = g.integers(lo, hi + 1, n).astype(np.uint32) << 23 | g.integers(0, 1 << 23, n).astype(np.uint32)
    return np.maximum(bits, 1).view(np.float32)


@pytest.mark.parametrize("y,rep", [((100, 150), (120, 134)), ((27, 254), (1, 253)), ((0, 0), (120, 134)),
                                   ((0, 40), (120, 134)), ((0, 40), (1, 253)), ((0, 254), (0, 0)),
                                   ((0, 254), (253, 254)), ((0, 254), (0, 254))])
def test_quotient(y, rep):
    g = np.random.default_rng(y[0] + 1000 * rep[0] + rep[1])
    R, V = 256, 8192
    x = _float(g, *y, R * V).reshape(R, V)
    r = _float(g, *rep, R)
    i32 = lambda a: torch.as_tensor(a, dtype=torch.int32).to(DEV)  # noqa: E731
    got = sdv.sd_logit_shape(torch.as_tensor(x).to(DEV), i32(np.arange(R)), i32(np.zeros(R)), V, gamma_max=0,
                             repetition=torch.as_tensor(r).to(DEV), seen=i32(np.full((R, V // 32), -1)))
    assert (got["status"] == 0).all()
    got = to_np(got["logits"]).astype(np.float64)
    want = x.astype(np.float64) / r[:, None].astype(np.float64)
    top = float(np.finfo(np.float32).max)
    with np.errstate(over="ignore"):
        unit = np.spacing(np.minimum(want, top).astype(np.float32)).astype(np.float64)
    over = want >= top * (1 + 2.0 ** -25)       # rounds to infinity
    assert np.isinf(got[over]).all()
    off = np.abs(got - want)[~over] / unit[~over]
    assert off.max(initial=0.0) <= 0.5 + 2.0 ** -22, off.max()
