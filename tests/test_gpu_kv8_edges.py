"""The operators over an 8-bit paged cache at the edges of what their arguments may be: scales, scores and values
over the whole range of their types, units that leave a slot idle, sizes at the top of the range."""
import math

import pytest
import torch

from block_sparse_long_rope_b200 import star
from tests import kv8_util as U
from tests.kv8_util import E4M3, INT8, ints
from tests.test_gpu_kv8 import BOUNDS, _attend, _attend_case, _status, _wide

pytestmark = pytest.mark.gpu


# ---- units that leave a slot of the chunk kernel without rows ---------------------------------------
@pytest.mark.parametrize("D,page", [(128, 64), (64, 16)])
@pytest.mark.parametrize("g", [1, 2])
def test_attend_slots_without_rows_behind_slow_ends(D, page, g):
    """Row tiles of 256 rows whose last rows meet NaN values at the causal edge (a slow way out), each
    followed by one of few rows, which leaves the other slot idle over a whole context."""
    lens, new, Hkv = [20000, 9001, 300, 12000], [300 // g, 260 // g, 300 // g, 20], 4
    q, cu, table, kp, vp, ks, vs = _attend_case(lens, new, Hkv * g, Hkv, D, page, E4M3, 79)
    max_new = max(new)
    clean, lse0, ws = _attend(q, cu, lens, table, kp, vp, ks, vs, max_new=max_new)
    U.check_attend(clean, lse0, U.attend_plain(q, cu, lens, table, kp, vp, ks, vs))
    hit = torch.zeros(q.shape[0], Hkv, D, dtype=torch.bool, device="cuda")
    for b, (L, T) in enumerate(zip(lens, new)):
        for back in range(2, T, 3):  # every third new token's value row
            t, dim, head = T - back, (7 * back) % D, back % Hkv
            at = L - back
            vp.view(torch.uint8)[int(table[b, at // page]), head, at % page, dim] = 0x7F if back % 2 else 0xFF
            hit[cu[b] + t:cu[b + 1], head, dim] = True
    hit = hit.repeat_interleave(g, 1)
    for _ in range(3):
        o, lse, _ = _attend(q, cu, lens, table, kp, vp, ks, vs, max_new=max_new, ws=ws)
        assert _status(ws) == "STAR_OK"
        assert torch.equal(torch.isnan(o), hit) and torch.equal(lse, lse0)
        assert torch.equal(o[~hit], clean[~hit])
