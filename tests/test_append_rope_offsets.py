"""pa_append_rope where some sequence's offsets are wrong: that sequence is flagged and left out, and
every other one is written."""

import numpy as np
import pytest

from paged_kv_cache_63_gb300 import lib
from tests.test_append_rope import Case, check

gpu = pytest.mark.gpu


@gpu
@pytest.mark.parametrize("batch", [5, 32, 33, 64, 100, 1100])
def test_a_bad_offset_costs_its_own_sequences_alone(batch):
    rng = np.random.default_rng(batch)
    case = Case([3] * batch, [4] * batch, qh=2, kvh=1, ps=8, pad=2)
    for at in sorted({1, batch // 2, batch - 1, *rng.integers(1, batch, 4).tolist()}):
        for value in (0, case.total + 1, 1 << 30, -1):
            qs = case.qs.copy()
            qs[at] = value
            if at == 1 and value == 0:
                continue  # an empty sequence, and one of more tokens than its context
            rows = set(range(3 * (at - 1), 3 * (at + 1)))
            check(case, *case.run(qs=qs), want_flags=lib.PA_DEVERR_QUERY_START, skip=rows)


@gpu
def test_the_last_offset_too_small():
    case = Case([2] * 40, [2] * 40, qh=2, kvh=1, ps=8)
    qs = case.qs.copy()
    qs[-1] = 70
    check(case, *case.run(qs=qs), want_flags=lib.PA_DEVERR_QUERY_START, skip={78, 79})
