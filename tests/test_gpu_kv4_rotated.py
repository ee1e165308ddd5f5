"""kvc_kv4_append_rotated on the GPU: codes, parameters and turned queries bit for bit (the definition rounds every operation)."""
import math

import numpy as np
import pytest

import entropy_coding_02_amd as kvc
import kv4_ref
import kv4_spec_ref as spec
from gpu_util import say
from test_gpu_kv4 import SHAPES, draw, f32, fresh, same_pool, status, tdt

pytestmark = pytest.mark.gpu

N_POS = 5000


def bits(t):
    import torch
    return t.contiguous().view({2: torch.int16, 4: torch.int32}[t.element_size()])


def turned(q, tab, pos, interleaved):
    """What q becomes, rounded to its type."""
    import torch
    return torch.from_numpy(spec.rotate(f32(q), tab, pos, interleaved)).to(q.dtype)


def inputs(T, H, D, Hq, dt, seed=1):
    k, v, q = draw((T, H, D), dt, seed), draw((T, H, D), dt, seed + 1, 0.01), draw((T, Hq, D), dt, seed + 2)
    pos = np.random.default_rng(seed).integers(0, N_POS, T)
    pos[0], pos[-1] = 0, N_POS - 1
    return k, v, q, pos


def cuda(*xs):
    import torch
    return [(torch.from_numpy(x) if isinstance(x, np.ndarray) else x).cuda() for x in xs]


@pytest.mark.parametrize("H,D,G,P", SHAPES)
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,order,Hq", [(1, "run", 1), (2, "mixed", 3), (37, "run", 8), (45, "mixed", 5), (45, "skipped", 7)])
def test_bits(H, D, G, P, dt, T, order, Hq):
    import torch
    say(f"[gpu] kv4 rotated H={H} D={D} G={G} P={P} {dt} T={T} {order} Hq={Hq}")
    n = -(-48 // P) + 2
    rng = np.random.default_rng(T)
    slots = (np.arange(T) + P if order == "run" else rng.permutation(n * P)[:T]).astype(np.int64)
    if order == "skipped":
        slots[::5] = -1
    k, v, q, pos = inputs(T, H, D, Hq, dt)
    for rot, inter in ((D, False), (D, True), (D // 2, False), (48, True), (16, False)):
        tab = spec.table(N_POS, rot)
        cache, ref = fresh(H, D, G, P, n)
        out = kvc.kv4_append_rotated(cache, *cuda(k, v, slots, pos, tab), q=q.cuda(), interleaved=inter)
        assert status(cache) == 0
        ref.write(spec.rotate(f32(k), tab, pos, inter), f32(v), slots)
        same_pool(cache, ref)
        assert torch.equal(bits(out.cpu()), bits(turned(q, tab, pos, inter))), (rot, inter)


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
def test_without_q_and_in_place(dt):
    import torch
    H, D, G, P, T, Hq = 2, 128, 64, 16, 21, 6
    k, v, q, pos = inputs(T, H, D, Hq, dt, 7)
    tab, slots = spec.table(N_POS, D), np.arange(3, 3 + T)
    for inter in (False, True):
        a, ref = fresh(H, D, G, P, 3)
        b, _ = fresh(H, D, G, P, 3)
        assert kvc.kv4_append_rotated(a, *cuda(k, v, slots, pos, tab), interleaved=inter) is None
        # q, k and v lie in one tensor, as a projection leaves them; q is turned where it is
        qkv = torch.cat([q, k, v], 1).cuda()
        qd, kd, vd = qkv.split([Hq, H, H], 1)
        assert kvc.kv4_append_rotated(b, kd, vd, *cuda(slots, pos, tab), q=qd, q_out=qd, interleaved=inter) is qd
        assert status(a) == 0 and status(b) == 0
        ref.write(spec.rotate(f32(k), tab, pos, inter), f32(v), slots)
        same_pool(a, ref)
        same_pool(b, ref)
        assert torch.equal(bits(qkv[:, :Hq].cpu()), bits(turned(q, tab, pos, inter)))
        assert torch.equal(qkv[:, Hq:].cpu(), torch.cat([k, v], 1))


def test_strides():
    import torch
    H, D, G, P, T, Hq = 3, 128, 64, 16, 21, 4
    tab = spec.table(N_POS, 96)
    big = draw((T, 3, Hq + 1, D + 1), "bf16", 5).cuda()
    k, v, q = big[:, 0, :H, :D], big[:, 1, 1:H + 1, 1:], big[:, 2, 1:, 1:]
    for k, v, q in ((k, v, q), (k.flip(0), v[:1].expand(T, H, D), q.transpose(0, 1).contiguous().transpose(0, 1))):
        cache, ref = fresh(H, D, G, P, 3)
        pos, slots = np.arange(T) * 200, np.arange(5, 5 + T)
        out = torch.full((T, Hq + 2, 2, D + 3), 7.0, dtype=torch.bfloat16, device="cuda")
        view = out[:, :Hq, 1, 3:]
        kvc.kv4_append_rotated(cache, k, v, *cuda(slots, pos, tab), q=q, q_out=view)
        assert status(cache) == 0
        ref.write(spec.rotate(f32(k), tab, pos, False), f32(v), slots)
        same_pool(cache, ref)
        assert torch.equal(bits(view.cpu()), bits(turned(q.cpu(), tab, pos, False)))
        assert (out[:, Hq:] == 7.0).all() and (out[:, :, 0] == 7.0).all() and (out[:, :, 1, :3] == 7.0).all()


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
def test_skipped_and_bad_tokens(dt):
    import torch
    H, D, G, P, Hq, n = 2, 64, 32, 16, 3, 2
    T = 9
    k, v, q, pos = inputs(T, H, D, Hq, dt, 11)
    tab = spec.table(100, 64)
    pos = np.array([0, 99, -1, 5, 100, 1 << 40, -(1 << 40), 7, 8], np.int64)
    slots = np.array([0, 1, 2, -1, 4, 5, 6, n * P, 1 << 40], np.int64)
    cache, ref = fresh(H, D, G, P, n)
    out = torch.full((T, Hq, D), 3.0, dtype=tdt(dt), device="cuda")
    kvc.kv4_append_rotated(cache, *cuda(k, v, slots, pos, tab), q=q.cuda(), q_out=out)
    assert status(cache) == kvc.KVC_DEV_BAD_INDEX
    there = (pos >= 0) & (pos < 100)
    ok = there & (slots >= 0) & (slots < n * P)
    at = np.where(there, pos, 0)
    ref.write(spec.rotate(f32(k), tab, at, False), f32(v), np.where(ok, slots, -1))
    same_pool(cache, ref)
    want = turned(q, tab, at, False)
    want[torch.from_numpy(~there)] = 3.0  # rows of tokens without a position are left alone
    assert torch.equal(bits(out.cpu()), bits(want))
    # a skipped token, whatever its slot and position, is no finding
    keep = (pos < 0) | (slots < 0)
    kvc.kv4_append_rotated(cache, *cuda(k[keep], v[keep], slots[keep], pos[keep], tab))
    assert status(cache) == 0
    same_pool(cache, ref)


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
def test_values_past_fp16_and_not_finite(dt):
    import torch
    H, D, G, P = 1, 64, 32, 16
    big = 65504.0 if dt == "f16" else 3.0e38
    tab = spec.table(8, 64)
    k = np.full((6, H, D), 1.0, np.float32)
    k[0, 0, :32], k[0, 0, 32:] = 60000.0, -60000.0  # turned by 1: past the fp16 range
    k[1, 0, 3] = math.inf                           # reaches its partner's group too
    k[2, 0, 40] = math.nan
    k[3, 0, 5], k[3, 0, 37] = big, -big             # sums past fp32, where the type holds such values
    k[4, 0, 9] = -0.0
    kt = torch.from_numpy(k).to(tdt(dt))
    slots, pos = np.arange(6), np.array([1, 2, 3, 1, 0, 7])
    cache, ref = fresh(H, D, G, P, 1)
    q = kt.expand(6, 1, D).contiguous()
    out = kvc.kv4_append_rotated(cache, *cuda(kt, torch.ones_like(kt), slots, pos, tab), q=q.cuda())
    assert status(cache) == kvc.KVC_DEV_NONFINITE
    turn = spec.rotate(f32(kt), tab, pos, False)
    ref.write(turn, np.ones_like(k), slots)
    same_pool(cache, ref)
    want = torch.from_numpy(turn).to(tdt(dt))
    assert torch.equal(torch.isnan(out.cpu()), torch.isnan(want))
    fine = ~torch.isnan(want)
    assert torch.equal(out.cpu()[fine], want[fine])


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("Hq", [1, 30])
def test_many_tokens_equal_few_at_a_time(dt, Hq):
    """A call that fills the chip gives the bytes of small calls, with odd counts of heads and tokens."""
    import torch
    H, D, G, P, T = 5, 64, 32, 32, 14003
    n = -(-T // P)
    k, v, q = draw((T, H, D), dt, 41).cuda(), draw((T, H, D), dt, 42, 0.1).cuda(), draw((T, Hq, D), dt, 43).cuda()
    rng = np.random.default_rng(6)
    slots, pos = cuda(rng.permutation(n * P)[:T].astype(np.int64), rng.integers(-1, N_POS, T))
    tab = torch.from_numpy(spec.table(N_POS, 64)).cuda()
    a, _ = fresh(H, D, G, P, n)
    b, _ = fresh(H, D, G, P, n)
    big, few = torch.full_like(q, 3.0), torch.full_like(q, 3.0)
    kvc.kv4_append_rotated(a, k, v, slots, pos, tab, q=q, q_out=big)
    for t in range(0, T, 400):
        at = slice(t, t + 400)
        kvc.kv4_append_rotated(b, k[at], v[at], slots[at], pos[at], tab, q=q[at], q_out=few[at])
    assert status(a) == 0 and status(b) == 0
    assert torch.equal(a.codes, b.codes) and torch.equal(bits(a.params), bits(b.params)) and torch.equal(bits(big), bits(few))
    i = np.random.default_rng(7).integers(0, T, 50)
    there = (pos[i] >= 0).cpu()
    want = turned(q[i].cpu(), spec.table(N_POS, 64), np.maximum(pos[i].cpu().numpy(), 0), False)
    assert torch.equal(bits(big[i].cpu()[there]), bits(want[there]))


def test_position_zero_is_kv4_append():
    import torch
    H, D, G, P, T = 4, 128, 32, 64, 100
    k, v = draw((T, H, D), "bf16", 51).cuda(), draw((T, H, D), "bf16", 52).cuda()
    slots = torch.arange(T).cuda()
    a, _ = fresh(H, D, G, P, 2)
    b, _ = fresh(H, D, G, P, 2)
    kvc.kv4_append(a, k, v, slots)
    kvc.kv4_append_rotated(b, k, v, slots, torch.zeros_like(slots), torch.from_numpy(spec.table(1, D)).cuda())
    assert torch.equal(a.codes, b.codes) and torch.equal(bits(a.params), bits(b.params))


def test_nothing_to_write():
    import torch
    cache, ref = fresh(2, 64, 32, 16, 1)
    e = torch.empty((0, 2, 64), dtype=torch.float16, device="cuda")
    none = torch.empty((0,), dtype=torch.int64, device="cuda")
    tab = torch.from_numpy(spec.table(4, 64)).cuda()
    assert kvc.kv4_append_rotated(cache, e, e, none, none, tab, q=e).shape == (0, 2, 64)
    assert status(cache) == 0
    same_pool(cache, ref)
    # an empty table holds no position
    one = torch.zeros((1,), dtype=torch.int64, device="cuda")
    k = torch.ones((1, 2, 64), dtype=torch.float16, device="cuda")
    kvc.kv4_append_rotated(cache, k, k, one, one, tab[:0])
    assert status(cache) == kvc.KVC_DEV_BAD_INDEX
    same_pool(cache, ref)


def test_a_given_stream():
    import torch
    from test_gpu_kv4_streams import busy
    H, D, T = 2, 128, 3000
    k, v, q, pos = inputs(T, H, D, 4, "bf16", 61)
    slots, tab = np.arange(T), spec.table(N_POS, D)
    args = cuda(k, v, slots, pos, tab)
    qd, x = q.cuda(), torch.zeros((4096, 4096), dtype=torch.bfloat16, device="cuda")
    a, _ = fresh(H, D, 64, 64, 47)
    b, _ = fresh(H, D, 64, 64, 47)
    want = kvc.kv4_append_rotated(a, *args, q=qd)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    given_back = [torch.empty_like(qd) for _ in range(4)]
    busy(x)
    for t in given_back:
        t.fill_(7.0)
    del t, given_back
    got = kvc.kv4_append_rotated(b, *args, q=qd, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(bits(got), bits(want)) and torch.equal(a.codes, b.codes) and status(b) == 0
