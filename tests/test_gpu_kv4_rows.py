"""Query rows that no sequence has: the padding of a captured batch."""
import pytest

import entropy_coding_02_amd as kvc
from gpu_util import say
from test_gpu_kv4 import build, draw, status, widen

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cu", [(0, 1, 3), (0, 2, 4), (2, 3, 5), (3, 3, 3)])
@pytest.mark.parametrize("keys,room,max_q,n_q", [
    (300, 320, 2, 9),          # one split
    (5000, 5056, 2, 9),        # split: the rows are joined by a second kernel
    (5000, 80000, 2, 9),       # in more than eight
    (300, 1 << 19, 64, 70),    # blocks of 128 rows, split
    (5000, 5056, 2, 40000)])   # far more rows than the sequences may have
def test_rows_of_no_sequence_are_left_alone(cu, keys, room, max_q, n_q):
    import torch
    say(f"[gpu] kv4 rows of no sequence cu={cu} keys={keys} room={room} n_q={n_q}")
    P, R, H, D = 64, 2, 2, 128
    cache, _, table, _ = build(H, D, 64, P, [keys, keys], "bf16", 91)
    table = torch.from_numpy(widen(table, room, P)).cuda()
    lens = torch.tensor([keys, keys], dtype=torch.int32).cuda()
    q = draw((n_q, H * R, D), "bf16", 92).cuda()
    bounds = torch.tensor(cu, dtype=torch.int32).cuda()
    out = torch.full_like(q, 7.0)
    lse = torch.full((n_q, H * R), 7.0, dtype=torch.float32, device="cuda")
    work = torch.full((kvc.kv4_work_bytes(cache, n_q, H * R, 2, table.shape[1], max_q),), 0x3C, dtype=torch.uint8, device="cuda")
    kvc.kv4_attention(cache, q, table, lens, cu_q=bounds, max_q=max_q, out=out, lse=lse, work=work)
    assert status(cache) == 0
    a, b = cu[0], cu[-1]
    assert (out[:a] == 7.0).all() and (out[b:] == 7.0).all() and (lse[:a] == 7.0).all() and (lse[b:] == 7.0).all()
    if b > a:  # and the others are what a call without the padding gives
        want, wl = kvc.kv4_attention(cache, q[a:b].contiguous(), table, lens, cu_q=bounds - a, max_q=max_q, return_lse=True)
        assert torch.equal(out[a:b], want) and torch.equal(lse[a:b], wl)
