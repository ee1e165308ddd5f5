"""What kvc_kv4_tree_attention reports of sequences without a key: parents that are no earlier token."""
import numpy as np
import pytest

import entropy_coding_02_amd as kvc
from gpu_util import say
from test_gpu_kv4 import build, draw, status
from test_gpu_kv4_tree import call, trees
from test_gpu_kv4_tree_rows import roomy

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H,D,G,rows", [(1, 64, 32, 24), (1, 64, 32, 4), (2, 128, 64, 128)])
@pytest.mark.parametrize("length", [0, -7, 2])
def test_a_bad_parent_of_a_sequence_without_keys_is_reported(H, D, G, rows, length):
    import torch
    R, nq = 4, rows // 4
    lens, pars = [200, length], trees([nq, nq], 41)
    say(f"[gpu] kv4 tree, bad parents, {length} keys, {rows} rows")
    cache, ref, table, slots = build(H, D, G, 16, lens, "bf16", 41)
    if rows == 128:
        table = roomy(table, H, 16, rows)
    q = draw((2 * nq, H * R, D), "bf16", 73)
    good, gl = call(cache, q, table, lens, pars)
    assert status(cache) == 0
    for at, entry in ((nq - 1, nq - 1), (0, 0), (nq // 2, -2)):
        worse = list(pars[1])
        worse[at] = entry
        out, lse = call(cache, q, table, lens, [pars[0], worse])
        assert status(cache) == kvc.KVC_DEV_BAD_INDEX, (at, entry)
        assert torch.equal(out[:nq], good[:nq])
        if length <= 0:
            assert (out[nq:] == 0).all() and np.isneginf(lse[nq:].cpu().numpy()).all()
