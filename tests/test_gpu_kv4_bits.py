"""Codes of groups whose values pass the fp16 range, bit for bit."""
import numpy as np
import pytest

import entropy_coding_02_amd as kvc
from gpu_util import say
from test_gpu_kv4 import f32, fresh, same_pool, status, tdt

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("D,G", [(64, 32), (128, 64), (256, 128)])
def test_values_past_the_range_count_as_its_border(dt, D, G):
    """Minima next to 65504, where lo rounds up or down, beside one value past it; and the same below zero."""
    import torch
    H, P = 1, 16
    low = [65400.0, 65472.0, 65480.0, 65488.0, 65490.0, 65500.0, 65503.0, 65504.0, 60000.0, 0.0, -65504.0, -7e4]
    high = [65504.0, 65519.0, 65520.0, 70000.0, 3e38]
    rows = [(a, b, sign) for a in low for b in high for sign in (1.0, -1.0)]
    say(f"[gpu] kv4 past the range {dt} D={D} G={G} rows={len(rows)}")
    x = np.zeros((len(rows), H, D), np.float32)
    for r, (a, b, sign) in zip(x, rows):
        r[0] = a
        r[0, 5::G] = b
        r[0, 9::G] = min(b, (a + 65504.0) / 2)
        r *= np.float32(sign)
    t = torch.from_numpy(x).to(tdt(dt))
    slots = np.arange(len(rows))
    cache, ref = fresh(H, D, G, P, -(-len(rows) // P))
    kvc.kv4_append(cache, t.cuda(), t.flip(0).cuda(), torch.from_numpy(slots).cuda())
    assert status(cache) == 0
    ref.write(f32(t), f32(t.flip(0)), slots)
    same_pool(cache, ref)
