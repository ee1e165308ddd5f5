"""The resident 4-bit cache on the GPU: written codes and parameters bit for
bit, values read back, and attention against 64-bit references.

Tolerance of attention.  out is rounded once: half a step of its type.  In
fp32 before it: a logit's error is at most delta = (D + 16) 2^-24 scale
max_j sum_c |q_c| (|lo| + 31 s) log2e (D products and sums, the start -qs and
the few steps after, on operands up to 31 s and lo, where a value is lo + code s); it moves every p by
delta and their normalised sum by 2 delta max|v|.  p s enters as two bf16
terms, off by 2^-18 of itself, times up to 31: 31 * 2^-18 max s.  exp2, the
sums over n keys (pairwise over waves, at most n/32 + 32 steps in a lane) and the
division: (n/32 + 64) 2^-24 of (max|v| + 31 max s).  lse: delta plus those steps of |lse| + 1.
"""
import math

import numpy as np
import pytest

import entropy_coding_02_amd as kvc
import kv4_ref
from gpu_util import say

pytestmark = pytest.mark.gpu

EPS = {"bf16": 2.0 ** -7, "f16": 2.0 ** -10, "f32": 2.0 ** -23}


def tdt(name):
    import torch
    return {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}[name]


def draw(shape, dt, seed, spread=1.0):
    import torch
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g) * spread
    x[..., :3] += 6.0 * spread
    return x.to(tdt(dt))


def f32(t):
    return t.float().cpu().numpy()


def status(cache):
    import torch
    torch.cuda.synchronize()
    s = int(cache.dev_status.item())
    cache.dev_status.zero_()
    return s


def same_pool(cache, ref):
    assert np.array_equal(cache.codes.cpu().numpy(), ref.codes_bytes())
    got, want = cache.params.cpu().numpy(), ref.params()
    assert np.array_equal(got, want, equal_nan=True)  # as numbers: -0 is 0


SHAPES = [  # H, D, G, P
    (1, 64, 32, 16), (3, 64, 64, 32), (2, 128, 32, 16), (5, 128, 64, 64), (2, 128, 128, 16), (1, 256, 32, 16),
    (3, 256, 64, 32), (1, 256, 128, 16)]


def fresh(H, D, G, P, n):
    cache = kvc.Kv4Cache(H, D, n, page_tokens=P, group=G)
    cache.codes.zero_()
    cache.params.zero_()
    return cache, kv4_ref.Pool(H, D, G, P, n)


@pytest.mark.parametrize("H,D,G,P", SHAPES)
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,order", [(1, "run"), (2, "mixed"), (37, "run"), (45, "mixed"), (45, "skipped")])
def test_append_bits_and_read(H, D, G, P, dt, T, order):
    import torch
    say(f"[gpu] kv4 append H={H} D={D} G={G} P={P} {dt} T={T} {order}")
    n = -(-48 // P) + 2
    cache, ref = fresh(H, D, G, P, n)
    rng = np.random.default_rng(T)
    slots = np.arange(T) + P if order == "run" else rng.permutation(n * P)[:T]
    if order == "skipped":
        slots[::5] = -1
    k, v = draw((T, H, D), dt, 1), draw((T, H, D), dt, 2, 0.01)
    st = torch.from_numpy(slots.astype(np.int64)).cuda()
    kvc.kv4_append(cache, k.cuda(), v.cuda(), st)
    assert status(cache) == 0
    ref.write(f32(k), f32(v), slots)
    same_pool(cache, ref)
    for out in ("f32", "f16", "bf16"):
        got = kvc.kv4_read(cache, st, dtype=tdt(out))
        for kv in (0, 1):
            want = torch.from_numpy(ref.value(kv, np.where(slots < 0, 0, slots)).astype(np.float32))  # fp32 first
            want[torch.from_numpy(slots < 0)] = 0
            assert torch.equal(got[kv].cpu(), want.to(tdt(out))), (out, kv)
    assert status(cache) == 0


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
def test_append_edge_values(dt):
    import torch
    H, D, G, P = 1, 128, 32, 16
    cache, ref = fresh(H, D, G, P, 2)
    x = np.zeros((8, H, D), np.float32)
    x[0] = 2.5                                  # constant
    x[1, 0, ::2] = 65504.0                      # the whole fp16 range
    x[1, 0, 1::2] = -65504.0
    x[2, 0] = 6e-8 * np.arange(D)               # subnormal lo and s
    x[3, 0] = 1e-7 * (np.arange(D) % 3)         # s below half the smallest fp16
    x[4, 0, ::3] = -0.0
    x[5, 0] = 70000.0 * np.sign(np.arange(D) - 60.5)  # past the fp16 range where the type holds it
    x[6, 0] = np.arange(D) / 7.0
    x[7, 0] = -1000.0 - np.arange(D) * 0.5
    t = torch.from_numpy(x).to(tdt(dt))
    t = torch.where(torch.isfinite(t), t, torch.zeros_like(t)) if dt == "f16" else t
    slots = torch.arange(8, 16).cuda()
    kvc.kv4_append(cache, t.cuda(), t.flip(0).cuda(), slots)
    assert status(cache) == 0
    ref.write(f32(t), f32(t.flip(0)), np.arange(8, 16))
    same_pool(cache, ref)
    k16, _ = kvc.kv4_read(cache, slots, dtype=torch.float16)
    assert torch.isfinite(k16).all()


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("D,G", [(64, 32), (128, 128), (256, 64)])
def test_append_nonfinite(dt, bad, D, G):
    import torch
    H, P = 2, 16
    cache, ref = fresh(H, D, G, P, 2)
    k, v = draw((6, H, D), dt, 3), draw((6, H, D), dt, 4)
    k[1, 1, D - 1] = bad
    v[4, 0, 5] = bad
    slots = torch.arange(3, 9).cuda()
    kvc.kv4_append(cache, k.cuda(), v.cuda(), slots)
    assert status(cache) == kvc.KVC_DEV_NONFINITE
    ref.write(f32(k), f32(v), np.arange(3, 9))
    same_pool(cache, ref)
    rk, rv = kvc.kv4_read(cache, slots, dtype=torch.float16)
    assert int(torch.isnan(rk).sum()) == G and int(torch.isnan(rv).sum()) == G
    assert torch.isnan(rk[1, 1, D - 1]) and torch.isnan(rv[4, 0, 5])


def test_append_and_read_strides():
    import torch
    H, D, G, P, T = 3, 128, 64, 16, 21
    big = draw((T, 2, H + 1, D + 1), "bf16", 5).cuda()
    for k, v in ((big[:, 0, :H, :D], big[:, 1, 1:, 1:]), (big[:, 0, :H, :D].flip(0).contiguous()[::2], big[::2, 1, :H, :D]),
                 (big[:, 0, :H, :D].transpose(0, 1).contiguous().transpose(0, 1), big[:, 1, :H, :D])):
        cache, ref = fresh(H, D, G, P, 3)
        n = k.shape[0]
        slots = torch.arange(5, 5 + n).cuda()
        kvc.kv4_append(cache, k, v, slots)
        ref.write(f32(k), f32(v), np.arange(5, 5 + n))
        assert status(cache) == 0
        same_pool(cache, ref)
        out = torch.full((n, H + 2, 2, D + 3), 7.0, dtype=torch.float16, device="cuda")
        kvc.kv4_read(cache, slots, k=out[:, :H, 0, :D], v=out[:, 2:, 1, 3:])
        for kv, view in ((0, out[:, :H, 0, :D]), (1, out[:, 2:, 1, 3:])):
            want = torch.from_numpy(ref.value(kv, np.arange(5, 5 + n)).astype(np.float32)).half()
            assert torch.equal(view.cpu(), want)
        assert (out[:, H:, 0] == 7.0).all() and (out[:, :2, 1] == 7.0).all() and (out[:, 2:, 1, :3] == 7.0).all()


def test_read_one_side_only():
    import torch
    cache, ref = fresh(2, 64, 32, 16, 2)
    k, v = draw((9, 2, 64), "f16", 6), draw((9, 2, 64), "f16", 7)
    slots = torch.arange(9).cuda()
    kvc.kv4_append(cache, k.cuda(), v.cuda(), slots)
    out = torch.zeros((9, 2, 64), dtype=torch.float32, device="cuda")
    for kv, args in ((0, (out.data_ptr(), None)), (1, (None, out.data_ptr()))):
        rc = kvc.lib().kvc_kv4_read(cache.ref, cache.codes.data_ptr(), cache.params.data_ptr(), slots.data_ptr(), 9, *args,
                                    128, 64, 128, 64, kvc.KVC_F32, None, torch.cuda.current_stream().cuda_stream)
        assert rc == kvc.KVC_OK
        ref.write(f32(k), f32(v), np.arange(9))
        assert np.array_equal(out.cpu().numpy(), ref.value(kv, np.arange(9)).astype(np.float32))


def test_bad_slots_are_flagged_and_skipped():
    import torch
    H, D, G, P, n = 2, 128, 64, 16, 2
    cache, ref = fresh(H, D, G, P, n)
    k, v = draw((8, H, D), "bf16", 8), draw((8, H, D), "bf16", 9)
    slots = np.array([0, 1, n * P, 3, -7, 1 << 40, 30, 31], np.int64)
    st = torch.from_numpy(slots).cuda()
    kvc.kv4_append(cache, k.cuda(), v.cuda(), st)
    assert status(cache) == kvc.KVC_DEV_BAD_INDEX
    ref.write(f32(k), f32(v), slots)
    same_pool(cache, ref)
    rk, rv = kvc.kv4_read(cache, st)
    assert status(cache) == kvc.KVC_DEV_BAD_INDEX
    gone = torch.from_numpy((slots < 0) | (slots >= n * P)).cuda()
    assert (rk[gone] == 0).all() and (rv[gone] == 0).all() and (rk[~gone] != 0).any()


# ------------------------------------------------------------------- attention

def build(H, D, G, P, lens, dt, seed, spare=2, junk=True):
    """A pool whose sequences of the given lengths lie in shuffled pages; what no sequence holds is NaN."""
    import torch
    pages = [-(-max(l, 0) // P) for l in lens]
    n = sum(pages) + spare
    cache, ref = fresh(H, D, G, P, n)
    if junk:
        cache.codes.fill_(0xA5)
        cache.params.fill_(math.nan)
    order = np.random.default_rng(seed).permutation(n)
    table = np.full((len(lens), max(pages + [1])), -1, np.int32)
    a, slots = 0, []
    for b, (l, m) in enumerate(zip(lens, pages)):
        table[b, :m] = order[a:a + m]
        a += m
        t = np.arange(max(l, 0))
        slots.append(table[b, t // P].astype(np.int64) * P + t % P)
    every = np.concatenate(slots)
    k, v = draw((len(every), H, D), dt, seed + 1, 0.7), draw((len(every), H, D), dt, seed + 2, 0.3)
    if len(every):
        kvc.kv4_append(cache, k.cuda(), v.cuda(), torch.from_numpy(every).cuda())
        ref.write(f32(k), f32(v), every)
    return cache, ref, table, slots


def check(cache, ref, table, slots, lens, nqs, R, dt, causal=True, window=0, softcap=0.0, scale=None, seed=50, **call):
    import torch
    H, D = ref.H, ref.D
    n_q = sum(nqs)
    q = draw((n_q, H * R, D), dt, seed)
    cu = np.concatenate([[0], np.cumsum(nqs)]).astype(np.int32)
    scale = D ** -0.5 if scale is None else scale
    out, lse = kvc.kv4_attention(cache, q.cuda(), torch.from_numpy(table).cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                                 cu_q=torch.from_numpy(cu).cuda(), max_q=max(nqs), causal=causal, window=window,
                                 softcap=softcap, scale=scale, return_lse=True, **call)
    assert status(cache) == 0
    compare(out, lse, q, ref, slots, lens, nqs, R, dt, causal, window, softcap, scale)
    return out, lse


def compare(out, lse, q, ref, slots, lens, nqs, R, dt, causal, window, softcap, scale):
    out, lse, q64 = out.double().cpu().numpy(), lse.double().cpu().numpy(), q.double().numpy()
    D = ref.D
    a = 0
    for b, nq in enumerate(nqs):
        l = max(lens[b], 0)
        pos = l - nq + np.arange(nq)
        for h in range(ref.H):
            hs = slice(h * R, (h + 1) * R)
            k, v = ref.value(0, slots[b])[:, h], ref.value(1, slots[b])[:, h]
            wo, wl = kv4_ref.attention(q64[a:a + nq, hs], k, v, pos, l, causal, window, softcap, scale)
            got, gl = out[a:a + nq, hs], lse[a:a + nq, hs]
            empty = np.isneginf(wl)
            assert np.array_equal(np.isneginf(gl), empty) and (got[empty] == 0).all()
            if l == 0 or empty.all():
                continue
            ks, kl = (np.repeat(x[0, slots[b], h].astype(np.float64), ref.G, -1) for x in (ref.s, ref.lo))
            reach = (np.abs(kl) + 31 * ks).max(0)
            delta = (D + 16) * 2.0 ** -24 * abs(scale) * 1.4427 * (np.abs(q64[a:a + nq, hs]) @ reach)
            smax, vmax = ref.s[1, slots[b], h].astype(np.float64).max(), np.abs(v).max()
            steps = (l / 32 + 64) * 2.0 ** -24
            tol = EPS[dt] / 2 * np.abs(wo) + (2 * delta * vmax + 31 * 2.0 ** -18 * smax + steps * (vmax + 31 * smax))[..., None]
            assert (np.abs(got - wo) <= tol)[~empty].all(), (b, h, np.abs(got - wo).max(), tol.min())
            assert (np.abs(gl - wl) <= delta + steps * (np.abs(wl) + 1))[~empty].all(), (b, h)
        a += nq


@pytest.mark.parametrize("H,D,G,P", SHAPES)
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_decode_lengths(H, D, G, P, dt):
    lens = [1, 0, 15, 16, 17, 31, 33, 128, 129, 300, 5, -3]
    say(f"[gpu] kv4 decode H={H} D={D} G={G} P={P} {dt}")
    cache, ref, table, slots = build(H, D, G, P, lens, dt, 11)
    check(cache, ref, table, slots, lens, [1] * len(lens), 4, dt)


@pytest.mark.parametrize("R", [1, 3, 7, 8, 16, 17])
@pytest.mark.parametrize("D,G", [(64, 32), (128, 64), (256, 128)])
def test_head_ratios(R, D, G):
    lens = [70, 259]
    say(f"[gpu] kv4 R={R} D={D}")
    cache, ref, table, slots = build(2, D, G, 32, lens, "f16", 12)
    check(cache, ref, table, slots, lens, [1, 1], R, "f16")


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("H,D,G,P", [(2, 64, 32, 16), (1, 128, 64, 64), (2, 128, 128, 32), (1, 256, 64, 16)])
def test_several_queries(H, D, G, P, dt, causal):
    # more queries than keys leave rows without a key
    lens, nqs = [3, 0, 64, 200, 131, 90], [5, 2, 64, 1, 37, 90]
    say(f"[gpu] kv4 queries H={H} D={D} G={G} P={P} {dt} causal={causal}")
    cache, ref, table, slots = build(H, D, G, P, lens, dt, 13)
    check(cache, ref, table, slots, lens, nqs, 3, dt, causal=causal)


@pytest.mark.parametrize("window", [1, 2, 31, 100, 128, 10000])
@pytest.mark.parametrize("D,G", [(64, 64), (128, 64), (256, 32)])
def test_window(window, D, G):
    import torch
    lens, nqs = [300, 17, 160, 5], [40, 1, 3, 9]
    say(f"[gpu] kv4 window={window} D={D}")
    cache, ref, table, slots = build(2, D, G, 16, lens, "bf16", 14)
    # pages wholly behind every query's window have been given away
    for b, (l, n) in enumerate(zip(lens, nqs)):
        table[b, :max(0, l - n - window + 1) // 16] = -1
    check(cache, ref, table, slots, lens, nqs, 2, "bf16", window=window)


@pytest.mark.parametrize("softcap,scale", [(30.0, None), (5.0, 1.0), (0.0, 2.0), (0.0, 0.0), (50.0, -0.5)])
def test_softcap_and_scale(softcap, scale):
    lens, nqs = [300, 33], [1, 20]
    say(f"[gpu] kv4 softcap={softcap} scale={scale}")
    cache, ref, table, slots = build(2, 128, 64, 16, lens, "f16", 15)
    check(cache, ref, table, slots, lens, nqs, 4, "f16", softcap=softcap, scale=scale)


@pytest.mark.parametrize("dt,lens", [("bf16", [5000]), ("f16", [9001, 37]), ("bf16", [2049, 0, 4096])])
def test_long_keys_are_split(dt, lens):
    say(f"[gpu] kv4 split {lens}")
    cache, ref, table, slots = build(2, 128, 64, 64, lens, dt, 16)
    assert kvc.kv4_work_bytes(cache, len(lens), 8, len(lens), table.shape[1], 1) > 0
    check(cache, ref, table, slots, lens, [1] * len(lens), 4, dt)
    check(cache, ref, table, slots, lens, [1] * len(lens), 4, dt, window=3000)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("D,G,R", [(64, 32, 4), (128, 64, 4), (128, 128, 1), (256, 64, 2)])
def test_prompt_pieces(dt, D, G, R):
    lens, nqs = [700, 333], [300, 333]
    say(f"[gpu] kv4 prompt D={D} G={G} R={R} {dt}")
    cache, ref, table, slots = build(2, D, G, 32, lens, dt, 17)
    check(cache, ref, table, slots, lens, nqs, R, dt)
    check(cache, ref, table, slots, lens, nqs, R, dt, window=150)


def test_nan_reaches_only_rows_that_attend():
    import torch
    lens, nqs = [80], [80]
    cache, ref, table, slots = build(1, 128, 64, 16, lens, "bf16", 18)
    k = torch.zeros((1, 1, 128), dtype=torch.bfloat16, device="cuda")
    v = k.clone()
    v[0, 0, 100] = math.nan  # token 50, second group of V
    kvc.kv4_append(cache, k, v, torch.from_numpy(slots[0][50:51]).cuda())
    assert status(cache) == kvc.KVC_DEV_NONFINITE
    q = draw((80, 2, 128), "bf16", 51).cuda()
    out, lse = kvc.kv4_attention(cache, q, torch.from_numpy(table).cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                                 return_lse=True)
    nan = torch.isnan(out)
    assert not nan[:50].any() and not nan[:, :, :64].any() and nan[50:, :, 64:].all() and torch.isfinite(lse).all()
    v[0, 0, 100] = 0.0
    k[0, 0, 3] = math.inf
    kvc.kv4_append(cache, k, v, torch.from_numpy(slots[0][50:51]).cuda())
    assert status(cache) == kvc.KVC_DEV_NONFINITE
    q[7, 1, 5] = math.nan
    out, lse = kvc.kv4_attention(cache, q, torch.from_numpy(table).cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                                 return_lse=True)
    nan = torch.isnan(out).all(-1)
    assert torch.equal(nan, torch.isnan(out).any(-1)) and torch.equal(nan, torch.isnan(lse))
    want = torch.zeros((80, 2), dtype=torch.bool, device="cuda")
    want[50:] = True
    want[7, 1] = True
    assert torch.equal(nan, want)


def test_attention_strides_and_given_buffers():
    import torch
    lens, nqs, R, H, D = [100, 40], [3, 2], 2, 3, 128
    cache, ref, table, slots = build(H, D, 64, 16, lens, "f16", 19)
    wide = torch.full((2, 9), -5, dtype=torch.int32)
    wide[:, :table.shape[1]] = torch.from_numpy(table)
    big = torch.full((5, 3, H * R, D + 1), 7.0, dtype=torch.float16, device="cuda")
    q = draw((5, H * R, D), "f16", 52)
    qd = torch.zeros((5, H * R + 1, D + 1), dtype=torch.float16, device="cuda")[:, 1:, 1:]
    qd.copy_(q)
    lse = torch.empty((5, H * R), dtype=torch.float32, device="cuda")
    out = big[:, 1, :, 1:]
    work = torch.empty(kvc.kv4_work_bytes(cache, 5, H * R, 2, table.shape[1], 3), dtype=torch.uint8, device="cuda")
    kvc.kv4_attention(cache, qd, wide.cuda()[:, :table.shape[1]], torch.tensor(lens, dtype=torch.int32).cuda(),
                      cu_q=torch.tensor([0, 3, 5], dtype=torch.int32).cuda(), max_q=3, out=out, lse=lse, work=work)
    assert status(cache) == 0
    compare(out, lse, q, ref, slots, lens, nqs, R, "f16", True, 0, 0.0, D ** -0.5)
    assert (big[:, 0] == 7.0).all() and (big[:, 2] == 7.0).all() and (big[:, 1, :, 0] == 7.0).all()


def test_bad_pages_and_lengths_are_flagged():
    import torch
    lens = [100, 100]
    cache, ref, table, slots = build(1, 64, 32, 16, lens, "bf16", 20)
    q = draw((2, 4, 64), "bf16", 53)

    def call(tab, ln, cu=(0, 1, 2)):
        out, lse = kvc.kv4_attention(cache, q.cuda(), torch.from_numpy(tab).cuda(), torch.tensor(ln, dtype=torch.int32).cuda(),
                                     cu_q=torch.tensor(cu, dtype=torch.int32).cuda(), max_q=1, return_lse=True)
        return status(cache), out, lse

    st, good, lse = call(table, lens)
    assert st == 0
    compare(good, lse, q, ref, slots, lens, [1, 1], 4, "bf16", True, 0, 0.0, 0.125)
    for entry in (-1, cache.n_pages, 2 ** 31 - 1):
        t = table.copy()
        t[1, 2] = entry
        st, out, _ = call(t, lens)
        assert st == kvc.KVC_DEV_BAD_INDEX and torch.equal(out[0], good[0])  # the other sequence is untouched
    st, out, _ = call(table, [100, table.shape[1] * 16 + 1])
    assert st == kvc.KVC_DEV_BAD_INDEX and torch.equal(out[0], good[0])
    st, out, _ = call(table, lens, cu=(0, 1, 3))
    assert st == kvc.KVC_DEV_BAD_INDEX and torch.equal(out[0], good[0])
    st, out, _ = call(table, lens, cu=(-4, 1, 2))
    assert st == kvc.KVC_DEV_BAD_INDEX


def test_pool_past_32_bits():
    """Slots whose bytes lie past 2^32."""
    import torch
    H, D, G, P = 8, 128, 64, 64
    n = (1 << 32) // (2 * H * P * D // 2) + 40
    cache = kvc.Kv4Cache(H, D, n, page_tokens=P, group=G)
    assert cache.codes.numel() > 1 << 32
    lens = [150]
    pages = np.array([n - 1, n - 17, 3], np.int32)
    t = np.arange(150)
    slots = pages[t // P].astype(np.int64) * P + t % P
    k, v = draw((150, H, D), "bf16", 61), draw((150, H, D), "bf16", 62)
    st = torch.from_numpy(slots).cuda()
    kvc.kv4_append(cache, k.cuda(), v.cuda(), st)
    small = kv4_ref.Pool(H, D, G, P, 3)
    near = np.arange(150)
    small.write(f32(k), f32(v), near)
    got = kvc.kv4_read(cache, st, dtype=torch.float32)
    for kv in (0, 1):
        assert np.array_equal(got[kv].cpu().numpy(), small.value(kv, near).astype(np.float32))
    q = draw((1, 16, D), "bf16", 63)
    out, lse = kvc.kv4_attention(cache, q.cuda(), torch.from_numpy(pages[None]).cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                                 return_lse=True)
    assert status(cache) == 0
    compare(out, lse, q, small, [near], lens, [1], 2, "bf16", True, 0, 0.0, D ** -0.5)


def test_other_stream_and_repeat():
    import torch
    lens = [700, 20, 333]
    cache, ref, table, slots = build(2, 128, 64, 16, lens, "bf16", 21)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    args = dict(table=torch.from_numpy(table).cuda(), lens=torch.tensor(lens, dtype=torch.int32).cuda(), q=draw((3, 8, 128), "bf16", 54).cuda())
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        a, la = kvc.kv4_attention(cache, args["q"], args["table"], args["lens"], return_lse=True)
        b, lb = kvc.kv4_attention(cache, args["q"], args["table"], args["lens"], return_lse=True)
    s.synchronize()
    assert torch.equal(a, b) and torch.equal(la, lb)  # a fixed order of sums
    compare(a, la, args["q"].cpu(), ref, slots, lens, [1, 1, 1], 4, "bf16", True, 0, 0.0, 128 ** -0.5)


def test_step_in_a_graph():
    """A serving step (write the new token, attend) captured once and replayed as the cache grows."""
    import torch
    H, R, D, P, B = 2, 4, 128, 16, 3
    lens = [400, 17, 63]
    grow = 3
    cache, ref, table, slots = build(H, D, 64, P, [l + grow for l in lens], "bf16", 22)
    k, v = draw((grow, B, H, D), "bf16", 71), draw((grow, B, H, D), "bf16", 72)
    q = draw((grow, B, H * R, D), "bf16", 73)
    tab = torch.from_numpy(table).cuda()
    sk, sv, sq = (torch.zeros_like(x[0]).cuda() for x in (k, v, q))
    slot = torch.full((B,), -1, dtype=torch.int64, device="cuda")
    length = torch.tensor(lens, dtype=torch.int32).cuda()
    work = torch.empty(kvc.kv4_work_bytes(cache, B, H * R, B, table.shape[1], 1), dtype=torch.uint8, device="cuda")
    out, lse = torch.empty_like(sq), torch.empty((B, H * R), dtype=torch.float32, device="cuda")

    def step():
        kvc.kv4_append(cache, sk, sv, slot)
        kvc.kv4_attention(cache, sq, tab, length, out=out, lse=lse, work=work)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for i in range(grow):
        at = np.array([slots[b][l + i] for b, l in enumerate(lens)])
        ref.write(f32(k[i]), f32(v[i]), at)
        sk.copy_(k[i]), sv.copy_(v[i]), sq.copy_(q[i])
        slot.copy_(torch.from_numpy(at))
        length.copy_(torch.tensor([l + i + 1 for l in lens], dtype=torch.int32))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        now = [l + i + 1 for l in lens]
        compare(out, lse, q[i], ref, [slots[b][:n] for b, n in enumerate(now)], now, [1] * B, R, "bf16", True, 0, 0.0, D ** -0.5)
        again, lse2 = kvc.kv4_attention(cache, sq, tab, length, return_lse=True)
        assert torch.equal(again, out) and torch.equal(lse2, lse)
    assert status(cache) == 0


def test_codec_to_cache_and_back():
    """The whole path: fp16 KV coded, decoded into the 4-bit cache, attended over, read back and coded again."""
    import torch
    import kvgen
    cfg = kvgen.CONFIGS["c2"].scaled(n_layers=2, n_tokens=300, layer_bins=((0, 2, 32),))
    L, T, C, H, D, R = 2, 300, cfg.n_channels, 8, 128, 4
    kv, _ = kvgen.generate(cfg)
    d = kvc.Desc(L, C, T, cfg.bins(), cfg.chunk_tokens)
    buf = kvc.alloc(d)
    kvc.encode(buf, torch.from_numpy(kv.view(np.int16)).cuda())
    kvc.decode(buf)
    dec = buf.out[: kv.size].view(L, 2, T, H, D)
    slots = torch.arange(T, device="cuda") + 64
    table = torch.arange(1, 6, dtype=torch.int32, device="cuda").view(1, 5)
    back = torch.empty_like(dec)
    for layer in range(L):
        cache, ref = kvc.Kv4Cache(H, D, 6), kv4_ref.Pool(H, D, 64, 64, 6)
        kvc.kv4_append(cache, dec[layer, 0], dec[layer, 1], slots)
        q = draw((1, H * R, D), "f16", 80 + layer, 0.2)
        out, lse = kvc.kv4_attention(cache, q.cuda(), table, torch.tensor([T], dtype=torch.int32).cuda(), return_lse=True)
        kvc.kv4_read(cache, slots, k=back[layer, 0], v=back[layer, 1])
        assert status(cache) == 0
        at = np.arange(T) + 64
        ref.write(f32(dec[layer, 0]), f32(dec[layer, 1]), at)
        compare(out, lse, q, ref, [at], [T], [1], R, "f16", True, 0, 0.0, D ** -0.5)
        for kv_ in (0, 1):
            assert np.array_equal(back[layer, kv_].cpu().numpy(), kv4_ref.to16(ref.value(kv_, at)))
    kvc.encode(buf, back)
    kvc.decode(buf)
    torch.cuda.synchronize()
    assert int(buf.dev_status.item()) == 0


# ----------------------------------------- blocks of 128 rows: many queries, or a long table

def widen(table, keys, P):
    """The same sequences under a table of room for `keys` keys (the launch goes by the table's width)."""
    wide = np.full((table.shape[0], keys // P), -1, np.int32)
    wide[:, :table.shape[1]] = table
    return wide


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("H,D,G,P,R", [(2, 64, 32, 16, 4), (1, 64, 64, 32, 5), (2, 128, 32, 64, 3), (2, 128, 64, 16, 4),
                                       (1, 128, 128, 32, 8), (1, 256, 64, 32, 4), (1, 256, 128, 16, 2)])
def test_wide_blocks_split(H, D, G, P, R, dt):
    lens, nqs = [700, 130, 0, 65, 3], [150, 130, 7, 1, 40]
    say(f"[gpu] kv4 wide H={H} D={D} G={G} P={P} R={R} {dt}")
    cache, ref, table, slots = build(H, D, G, P, lens, dt, 31)
    table = widen(table, 65536, P)
    check(cache, ref, table, slots, lens, nqs, R, dt)
    check(cache, ref, table, slots, lens, nqs, R, dt, causal=False)
    check(cache, ref, table, slots, lens, nqs, R, dt, softcap=20.0, scale=-0.3)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("window", [0, 2100, 4000])
def test_wide_blocks_window_and_pages_given_away(dt, window):
    lens, nqs, P = [5000, 2300], [64, 40], 32
    say(f"[gpu] kv4 wide window={window} {dt}")
    cache, ref, table, slots = build(1, 128, 64, P, lens, dt, 32)
    for b, (l, n) in enumerate(zip(lens, nqs)):
        if window:
            table[b, :max(0, l - n - window + 1) // P] = -1
    check(cache, ref, widen(table, 1 << 19, P), slots, lens, nqs, 2, dt, window=window)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_wide_blocks_unsplit(dt):
    B = 33
    lens = [int(x) for x in np.random.default_rng(5).integers(1, 200, B)]
    nqs = [min(l, 32) for l in lens]
    nqs[0], lens[0] = 32, 190
    say(f"[gpu] kv4 wide unsplit {dt}")
    cache, ref, table, slots = build(8, 64, 64, 16, lens, dt, 33)
    assert kvc.kv4_work_bytes(cache, sum(nqs), 32, B, 4096 // 16, 32) >= 0
    check(cache, ref, widen(table, 4096, 16), slots, lens, nqs, 4, dt)


def test_wide_blocks_bad_page_and_nan():
    import torch
    lens, nqs, P, R = [300], [300], 16, 2
    cache, ref, table, slots = build(1, 128, 64, P, lens, "bf16", 34)
    wide = widen(table, 1 << 19, P)
    q = draw((300, R, 128), "bf16", 91)
    args = (q.cuda(), torch.from_numpy(wide).cuda(), torch.tensor(lens, dtype=torch.int32).cuda())
    good = kvc.kv4_attention(cache, *args)
    assert status(cache) == 0
    bad = wide.copy()
    bad[0, 3] = cache.n_pages
    out = kvc.kv4_attention(cache, args[0], torch.from_numpy(bad).cuda(), args[2])
    assert status(cache) == kvc.KVC_DEV_BAD_INDEX
    assert torch.equal(out[:48], good[:48])  # rows before the page
    v = torch.zeros((1, 1, 128), dtype=torch.bfloat16, device="cuda")
    v[0, 0, 100] = math.nan
    kvc.kv4_append(cache, torch.zeros_like(v), v, torch.from_numpy(slots[0][150:151]).cuda())
    assert status(cache) == kvc.KVC_DEV_NONFINITE
    out, lse = kvc.kv4_attention(cache, *args, return_lse=True)
    nan = torch.isnan(out)
    assert not nan[:150].any() and not nan[:, :, :64].any() and nan[150:, :, 64:].all() and torch.isfinite(lse).all()


@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_tiny_and_huge_values(dt):
    """V and K far from 1: s near the ends of fp16, q beyond its range."""
    import torch
    H, D, G, P = 1, 128, 64, 16
    lens = [200]
    for kmul, vmul, qmul in ((1.0, 1e-3, 1.0), (1.0, 6000.0, 1.0), (1000.0, 1.0, 1e-4), (1e-3, 1.0, 3e4)):
        cache, ref = fresh(H, D, G, P, 14)
        k, v = draw(lens + [H, D], dt, 95, kmul), draw(lens + [H, D], dt, 96, vmul)
        slots = np.arange(lens[0])
        kvc.kv4_append(cache, k.cuda(), v.cuda(), torch.from_numpy(slots).cuda())
        ref.write(f32(k), f32(v), slots)
        table = np.arange(13, dtype=np.int32)[None]
        q = (draw((40, 4, D), "bf16", 97).float() * qmul).clamp(-6e4, 6e4).to(tdt(dt))
        for tab in (table, widen(table, 1 << 19, P)):
            out, lse = kvc.kv4_attention(cache, q.cuda(), torch.from_numpy(tab).cuda(),
                                         torch.tensor(lens, dtype=torch.int32).cuda(), return_lse=True)
            assert status(cache) == 0
            compare(out, lse, q, ref, [slots], lens, [40], 4, dt, True, 0, 0.0, D ** -0.5)


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
def test_many_tokens_equal_few_at_a_time(dt):
    """A call that fills the chip gives the bytes and values of small calls."""
    import torch
    H, D, G, P, T = 5, 64, 32, 32, 14003
    n = -(-T // P)
    k, v = draw((T, H, D), dt, 41).cuda(), draw((T, H, D), dt, 42, 0.1).cuda()
    slots = torch.from_numpy(np.random.default_rng(6).permutation(n * P)[:T].astype(np.int64)).cuda()
    slots[1000:9000] = torch.arange(1000, 9000).cuda()  # runs too; a slot met twice is written last by the later call
    slots = torch.where(torch.isin(slots, torch.arange(1000, 9000).cuda()) &
                        ((torch.arange(T).cuda() < 1000) | (torch.arange(T).cuda() >= 9000)), -1, slots)
    a, _ = fresh(H, D, G, P, n)
    b, _ = fresh(H, D, G, P, n)
    kvc.kv4_append(a, k, v, slots)
    for t in range(0, T, 4000):
        kvc.kv4_append(b, k[t:t + 4000], v[t:t + 4000], slots[t:t + 4000])
    assert status(a) == 0 and status(b) == 0
    assert torch.equal(a.codes, b.codes) and torch.equal(a.params.view(torch.int16), b.params.view(torch.int16))
    big = kvc.kv4_read(a, slots, dtype=tdt(dt))
    for t in range(0, T, 4000):
        few = kvc.kv4_read(b, slots[t:t + 4000], dtype=tdt(dt))
        for x, y in zip(big, few):
            assert torch.equal(x[t:t + 4000], y)


def test_every_scale_has_its_reciprocal():
    """Codes of groups whose s takes every positive fp16 value that it can: 1/s has to be rounded correctly."""
    import torch
    H, D, G, P = 1, 64, 32, 256
    bits = np.arange(1, 0x7C00, dtype=np.uint16)
    s = bits.view(np.float16).astype(np.float32)
    s = s[s <= 4366.0]  # 15 s within fp16
    rng = np.random.default_rng(8)
    x = (rng.random((len(s), 1, D)).astype(np.float32) * 15.0) * s[:, None, None]
    x[:, 0, ::G] = 0.0
    x[:, 0, 1::G] = (15.0 * s)[:, None]
    T = len(s)
    n = -(-T // P)
    cache, _ = fresh(H, D, G, P, n)
    t = torch.from_numpy(x)
    slots = torch.arange(T).cuda()
    kvc.kv4_append(cache, t.cuda(), t.cuda(), slots)
    assert status(cache) == 0
    got = kvc.kv4_read(cache, slots, dtype=torch.float32)
    c, sq, lo = kv4_ref.quantise(x, G)
    want = kv4_ref.values(c, sq, lo, G).astype(np.float32)
    assert len(np.unique(sq)) > 0.99 * len(s)
    for y in got:
        assert np.array_equal(y.cpu().numpy(), want)


@pytest.mark.parametrize("wide", [False, True])
def test_average_of_many_keys_keeps_its_last_bit(wide):
    """20000 keys, fp16: out is a small average of large terms (lo and s n cancel).  Its relative rms error is that
    of one rounding, at most half a step, 2^-11, uniform: 2^-11 / sqrt(3), with a tenth more for all before it."""
    import torch
    H, D, G, P, R, T = 2, 128, 64, 64, 8, 20000
    n = -(-T // P)
    cache, ref = kvc.Kv4Cache(H, D, n, page_tokens=P, group=G), kv4_ref.Pool(H, D, G, P, n)
    k, v = draw((T, H, D), "f16", 101), torch.randn((T, H, D), generator=torch.Generator().manual_seed(102)).half()
    slots = np.arange(T)
    kvc.kv4_append(cache, k.cuda(), v.cuda(), torch.from_numpy(slots).cuda())
    ref.write(f32(k), f32(v), slots)
    nq = 32 if wide else 1
    q = draw((nq, H * R, D), "f16", 103, 0.5)
    table = np.arange(n, dtype=np.int32)[None]
    tab = widen(table, 1 << 19, P) if wide else table
    out, lse = kvc.kv4_attention(cache, q.cuda(), torch.from_numpy(tab).cuda(), torch.tensor([T], dtype=torch.int32).cuda(),
                                 return_lse=True)
    assert status(cache) == 0
    got, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
    off, of, ol = [], [], []
    for h in range(H):
        hs = slice(h * R, (h + 1) * R)
        wo, wl = kv4_ref.attention(q[:, hs].double().numpy(), ref.value(0, slots)[:, h], ref.value(1, slots)[:, h],
                                   T - nq + np.arange(nq), T, True, 0, 0.0, D ** -0.5)
        off.append(got[:, hs] - wo), of.append(wo), ol.append((gl[:, hs] - wl) / wl)
    rms = lambda x: float(np.sqrt(np.mean(np.square(x))))  # noqa: E731
    assert rms(off) <= 1.1 * 2.0 ** -11 / math.sqrt(3) * rms(of)
    assert rms(ol) < 1e-6


def test_example_runs_them_together():
    import os
    import sys
    import torch
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    sys.path.insert(0, os.path.join(root, "examples"))
    try:
        import resident_cache
    finally:
        sys.path.pop(0)
    r = resident_cache.main(n_tokens=300, n_steps=70)  # the steps pass the end of a page
    assert r["status"] == 0 and torch.isfinite(r["out"]).all() and r["out"].abs().sum() > 0
    # 4 bits a channel, 16 levels over a group's range: half a step of 1/15 of it, uniform, against the rms of what
    # lies in it (at least an eighth of its range for 64 values of any smooth density)
    assert r["rms_error"] <= 8 / 15 / math.sqrt(12)


def test_wide_blocks_in_a_graph():
    """A prompt piece captured, replayed with other queries and lengths, each replay against the eager call."""
    import torch
    lens, nq, R, P = [260, 90], 64, 4, 16
    cache, ref, table, slots = build(2, 128, 64, P, lens, "bf16", 35)
    tab = torch.from_numpy(widen(table, 65536, P)).cuda()
    q = draw((2 * nq, 2 * R, 128), "bf16", 111).cuda()
    length = torch.tensor(lens, dtype=torch.int32).cuda()
    work = torch.empty(kvc.kv4_work_bytes(cache, 2 * nq, 2 * R, 2, tab.shape[1], nq), dtype=torch.uint8, device="cuda")
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], dtype=torch.float32, device="cuda")

    def step():
        kvc.kv4_attention(cache, q, tab, length, out=out, lse=lse, work=work)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for i in range(3):
        q.copy_(draw(tuple(q.shape), "bf16", 112 + i))
        length.copy_(torch.tensor([l - 13 * i for l in lens], dtype=torch.int32))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        again, lse2 = kvc.kv4_attention(cache, q, tab, length, return_lse=True)
        assert torch.equal(again, out) and torch.equal(lse2, lse)
        now = [l - 13 * i for l in lens]
        compare(out, lse, q.cpu(), ref, [s[:n] for s, n in zip(slots, now)], now, [nq] * 2, R, "bf16", True, 0, 0.0, 128 ** -0.5)
    assert status(cache) == 0


@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_wide_blocks_of_256_channels_in_fine_groups(dt):
    lens, nqs = [333, 64, 0], [140, 64, 9]
    say(f"[gpu] kv4 wide D=256 G=32 {dt}")
    cache, ref, table, slots = build(2, 256, 32, 16, lens, dt, 36)
    table = widen(table, 65536, 16)
    check(cache, ref, table, slots, lens, nqs, 2, dt)
    check(cache, ref, table, slots, lens, nqs, 2, dt, causal=False, softcap=15.0)
