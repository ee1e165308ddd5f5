"""What kvc_kv4_append_rotated reports of tokens that are not written: a position past the table, whatever the slot; nothing of a
token whose position is negative."""
import pytest

import entropy_coding_02_amd as kvc
import kv4_spec_ref as spec
from gpu_util import say
from test_gpu_kv4 import draw, fresh, same_pool, status

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("with_q", [False, True])
def test_a_position_past_the_table_is_reported_whatever_the_slot(dt, with_q):
    import torch
    H, D, G, P, Hq, n = 2, 64, 32, 16, 3, 2
    tab = torch.from_numpy(spec.table(100, D)).cuda()
    cache, ref = fresh(H, D, G, P, n)
    k, q = draw((1, H, D), dt, 11).cuda(), draw((1, Hq, D), dt, 12).cuda()
    for slot, pos, want in ((-1, 100, True), (-5, 1 << 40, True), (n * P, 100, True), (3, 100, True), (n * P, 5, True),
                            (-1, 5, False), (-1, -1, False), (n * P, -1, False), (1 << 40, -(1 << 40), False)):
        say(f"[gpu] kv4 rotated, slot {slot}, position {pos}")
        kvc.kv4_append_rotated(cache, k, k, torch.tensor([slot]).cuda(), torch.tensor([pos]).cuda(), tab, q=q if with_q else None)
        assert status(cache) == (kvc.KVC_DEV_BAD_INDEX if want else 0), (slot, pos)
    same_pool(cache, ref)  # nothing was written
