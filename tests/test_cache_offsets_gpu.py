"""Offsets of query rows out of range in the paged cache's attention: the status, the rows of the requests that
are right, and the rows that no request owns."""
import numpy as np
import pytest

import test_cache_gpu as tc

pytestmark = pytest.mark.gpu
fp = tc.fp
FAR = 2 ** 31 - 1


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("reqs,cu,status", [
    # by columns: rows of the second request behind q, a negative start, an end before the start, starts behind q, an
    # end far behind it
    ([(200, 2), (90, 1)], [0, 2, 9], 5), ([(200, 2), (90, 1)], [-3, 2, 3], 5), ([(200, 2), (90, 1)], [0, 2, 1], 0),
    ([(200, 2), (90, 1)], [5, 7, 9], 5), ([(200, 2), (90, 1)], [0, FAR, 3], 5), ([(200, 2), (90, 1)], [1, 1, 3], 0),
    # by tiles, which leave requests of few columns to the other form or take them too
    ([(300, 80), (90, 1)], [0, 80, 90], 5), ([(300, 80), (90, 1)], [-3, 77, 81], 5), ([(300, 80), (90, 1)], [0, 81, 1], 0),
    ([(300, 80), (90, 1)], [5, 85, 81], 5), ([(300, 80), (90, 1)], [0, FAR, 3], 5), ([(300, 80), (90, 1)], [0, 2, 1], 0),
    ([(300, 80), (90, 1)], [-2 ** 31, 2, 4], 5), ([(300, 80), (90, 1)], [7, 7, 81], 0), ([(300, 80), (90, 1)], [FAR, FAR, FAR], 0),
])
def test_offsets(fp, reqs, cu, status, dtype):
    import torch
    h_q, h = (4, 2) if reqs[0][1] == 2 else (8, 2)
    s = tc.attn_case(fp, reqs, h_q, h, 32, dtype, "bf16", seed=5)
    total = s["q"].shape[0]
    out = torch.full((total, h_q, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((h_q, total), 7.0, device="cuda")
    s["c"].attn(s["q"], tc.i32(s["table"]), tc.i32(s["lens"]), cu_seqlens_q=tc.i32(cu), max_q=max(m for _, m in reqs), out=out,
                lse=lse)
    assert s["c"].device_status() == status
    owned = np.zeros(total, bool)
    for r in range(2):
        a, b = cu[r], cu[r + 1]
        if a < 0 or b <= a or a >= total:
            continue
        rows = slice(a, min(b, total))
        assert not owned[rows].any()
        owned[rows] = True
        if b - a > s["lens"][r] + total:                # every one of its rows lies before the first key
            assert not out[rows].any() and bool(torch.isneginf(lse[:, rows]).all())
            continue
        one = dict(s, qv=s["qv"][rows], table=s["table"][r:r + 1], lens=[s["lens"][r]], lq=[b - a])
        tc.check_attn(one, out[rows], lse[:, rows], rows=rows.stop - a)
    assert bool((out[torch.from_numpy(~owned)] == 3).all()) and bool((lse[:, torch.from_numpy(~owned)] == 7).all())
