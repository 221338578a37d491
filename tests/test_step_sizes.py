"""Sizes past 32 bits are refused, not cut to their low half."""

import pytest
import torch

import draft_verification_amd as sdv
from draft_verification_amd import _lib

BIG = 1 << 32


def test_what_fits():
    for sizes in (0, 5 | 64, (1 << 31) - 1, -1, -1 | 7, -(1 << 31)):
        _lib._fits("f", sizes)
    for sizes in (1 << 31, BIG, BIG + 64, 3 | BIG, -BIG + 64, -(1 << 31) - 1):
        with pytest.raises(sdv.SdvError) as e:
            _lib._fits("f", sizes)
        assert e.value.code == _lib.SD_EUNSUPPORTED


@pytest.mark.gpu
def test_calls_refuse_them():
    i = lambda *k: torch.zeros(k, dtype=torch.int32, device="cuda")  # noqa: E731
    x, seq = torch.zeros((4, 64), device="cuda"), torch.zeros(2, dtype=torch.int64, device="cuda")
    calls = [
        lambda n: sdv.sd_logit_shape(x, i(2), i(2) - 1, 64 + n, gamma_max=1),
        lambda n: sdv.sd_logit_shape(x, i(2), i(2) - 1, 64, gamma_max=1 + n),
        lambda n: sdv.sd_token_counts(i(2, 3), i(2, 2), i(2, 64), 64 + n),
        lambda n: sdv.sd_token_counts(i(8), i(2, 2), i(2, 64), 64, start=seq, length=i(2), max_length=4 + n),
        lambda n: sdv.sd_slot_reserve(seq, i(2) - 1, i(2, 4), i(8), i(1), 16, 3 + n, max_rows=6),
        lambda n: sdv.sd_slot_reserve(seq, i(2) - 1, i(2, 4), i(8), i(1), 16 + n, 3),
        lambda n: sdv.sd_slot_commit(seq, i(2) - 1, i(2), i(2, 4), i(8), i(1), 16, q_max=3 + n),
        lambda n: sdv.sd_slot_commit(seq, i(2) - 1, i(2), i(2, 4), i(8), i(1), 16 + n, q_max=3),
    ]
    for k, call in enumerate(calls):
        call(0)
        for n in (1 << 32, -(1 << 32)):
            with pytest.raises(sdv.SdvError):
                call(n)
                pytest.fail(f"call {k} took a size cut to 32 bits")
    torch.cuda.synchronize()
