"""kvc_kv4_append_rotated refuses q_out in k's or v's place, and with every tensor in a place of its own what else it has to (no
GPU: the call returns before any HIP call)."""
import pytest
import torch

import entropy_coding_02_amd as kvc
from test_kv4_abi import OK, desc
from test_kv4_spec_abi import append

FAR = {n: OK + (i << 20) for i, n in enumerate(("k", "v", "q", "q_out"))}


@pytest.mark.parametrize("other", ["k", "v"])
def test_queries_turned_in_the_place_of_keys_or_values(other):
    if torch.cuda.device_count():
        pytest.skip("accepted calls would launch on stand-in addresses")
    assert append(**FAR) == kvc.KVC_ERR_HIP  # as far as the missing device
    assert append(**{**FAR, "q_out": FAR[other]}) == kvc.KVC_ERR_ARG
    assert append(**{**FAR, "q": FAR[other], "q_out": FAR[other]}) == kvc.KVC_ERR_ARG
    assert append(**{**FAR, "q": FAR[other]}) == kvc.KVC_ERR_HIP  # read by both


def test_other_refusals():
    if torch.cuda.device_count():
        pytest.skip("accepted calls would launch on stand-in addresses")
    at = FAR["q_out"]
    for kw in (dict(k=None), dict(v=None), dict(k=OK + 1), dict(v=at + 1), dict(q=at + 1), dict(q_out=at + 1), dict(q=None),
               dict(q_out=None), dict(q=at + 2, dtype=1), dict(n_tokens=-1), dict(n_tokens=1 << 41), dict(dtype=3), dict(dtype=-1),
               dict(slots=None), dict(slots=OK + 4), dict(positions=None), dict(positions=OK + 4), dict(table=None),
               dict(table=OK + 8), dict(n_positions=-1), dict(rot=0), dict(rot=8), dict(rot=24), dict(rot=144), dict(rot=-16),
               dict(n_q_heads=0), dict(n_q_heads=-3), dict(n_q_heads=65537), dict(q=at, q_out_token_stride=640),
               dict(q=at, q_out_head_stride=256), dict(codes=None), dict(codes=OK + 8), dict(params=None), dict(params=OK + 4),
               dict(st=OK + 2), dict(d=desc(D=64), rot=80)):
        assert append(**{**FAR, **kw}) == kvc.KVC_ERR_ARG, kw
    for kw in (dict(q=at), dict(q_out_token_stride=640), dict(q=None, q_out=None, n_q_heads=0), dict(rot=16), dict(interleaved=1)):
        assert append(**{**FAR, **kw}) == kvc.KVC_ERR_HIP, kw
