"""The 4-bit cache's calls on a stream that is not the current one."""
import pytest

import entropy_coding_02_amd as kvc
from gpu_util import say
from test_gpu_kv4 import build, draw, status

pytestmark = pytest.mark.gpu


def busy(x):
    """Some milliseconds of work on the current stream."""
    for _ in range(20):
        x = x @ x
    return x


@pytest.mark.parametrize("handle", [False, True])
def test_attention_on_a_given_stream(handle):
    """While the call waits on its stream, the current one allocates and fills blocks of the workspace's size."""
    import torch
    say(f"[gpu] kv4 attention stream= handle={handle}")
    cache, _, table, _ = build(2, 128, 64, 64, [9001], "bf16", 16)
    q, tab = draw((1, 8, 128), "bf16", 60).cuda(), torch.from_numpy(table).cuda()
    lens, x = torch.tensor([9001], dtype=torch.int32).cuda(), torch.zeros((4096, 4096), dtype=torch.bfloat16, device="cuda")
    want, wl = kvc.kv4_attention(cache, q, tab, lens, return_lse=True)
    nb = kvc.kv4_work_bytes(cache, 1, 8, 1, tab.shape[1], 1)
    assert nb > 0
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        busy(x)
    out, lse = kvc.kv4_attention(cache, q, tab, lens, return_lse=True, stream=s.cuda_stream if handle else s)
    others = [torch.full((nb,), 7, dtype=torch.uint8, device="cuda") for _ in range(8)]
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, wl)
    assert all(bool((t == 7).all()) for t in others)
    assert status(cache) == 0


def test_read_on_a_given_stream():
    """What the current stream still writes to memory that was given back must not be in the rows."""
    import torch
    say("[gpu] kv4 read stream=")
    T, H, D = 3000, 2, 128
    cache, _, _, slots = build(H, D, 64, 64, [T], "f16", 17)
    at = torch.from_numpy(slots[0]).cuda()
    want = kvc.kv4_read(cache, at)
    x = torch.zeros((4096, 4096), dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    given_back = [torch.empty((T, H, D), dtype=torch.float16, device="cuda") for _ in range(4)]
    busy(x)
    for t in given_back:
        t.fill_(7.0)
    del t, given_back
    got = kvc.kv4_read(cache, at, stream=s)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert status(cache) == 0
