"""Keys that pa_append_quant neither norms nor turns, wholly or in their unturned part: the codes are
those of the fp16 numbers themselves, bit for bit, halves between two codes and zeroes of both signs
among them."""

import numpy as np
import pytest

from tests.quant_reference import BORDERS, quantise
from tests.test_quant_cache import QuantCase, check

gpu = pytest.mark.gpu


def exact_rows(case, seed):
    """Key rows with borders between two codes, zeroes of both signs, and normal numbers beside them."""
    rng = np.random.default_rng(seed)
    k = case.qkv[:, case.qh:case.qh + case.kvh]
    kind = rng.integers(0, 4, k.shape)
    sign = rng.choice([-1.0, 1.0], k.shape)
    ties = rng.choice(BORDERS, k.shape) * 2.0 ** -5
    k[...] = np.where(kind == 0, k, sign * np.where(kind < 3, ties, 0.0)).astype(np.float16)
    assert (ties.astype(np.float16) == ties).all()  # numbers of fp16
    return case


@gpu
@pytest.mark.parametrize("norm", ["none", "query"])
@pytest.mark.parametrize("hd,rotary,interleaved", [
    (64, 0, False), (128, 0, False), (256, 0, False), (128, 64, False), (256, 64, True), (64, 16, True),
    (256, 128, False)])
def test_codes_of_unturned_elements(hd, rotary, interleaved, norm):
    case = exact_rows(QuantCase([33, 2, 70], [60, 2, 90], norm=norm, hd=hd, rotary=rotary, qh=6, kvh=3,
                                interleaved=interleaved), hd + rotary)
    got, flags = case.run()
    check(case, got, flags)
    # the largest element of a row may be a turned one, so the scale is the row's own
    for b, n in enumerate(case.new):
        for j in range(int(n)):
            t = int(case.ctx[b] - n + j)
            at = int(case.bt[b, t // case.ps]), t % case.ps
            k = case.qkv[int(case.qs[b]) + j, case.qh:case.qh + case.kvh].astype(np.float64)
            scale = 2.0 ** (got[2]["k"][at].astype(np.float64) - 127)[:, None]
            if rotary == 0:
                assert np.array_equal(got[1]["k"][at], quantise(k)[0])
            # under a scale of 1 (its row's largest number is put at 448) codes are those of k / scale
            row = np.append(np.clip(k / scale, -448, 448), np.full((case.kvh, 1), 448.0), axis=1)
            codes, one = quantise(row)
            assert (one == 127).all()
            assert np.array_equal(got[1]["k"][at][:, rotary:], codes[:, rotary:-1])
