"""Attention over the 4-bit cache against 64 bits, as near as kv4_close asks: every shape and type, both kernels, split
and unsplit, windows, soft caps, rows without keys."""
import numpy as np
import pytest

import entropy_coding_02_amd as kvc
import kv4_close
import kv4_ref
from gpu_util import say
from test_gpu_kv4 import SHAPES, f32, fresh, status, widen

pytestmark = pytest.mark.gpu


def hold(H, D, G, P, lens, n_q, R, dt, seed):
    """Sequences of the given lengths in shuffled pages; what no sequence holds is NaN."""
    import torch
    pages = [-(-l // P) for l in lens]
    n = sum(pages) + 1
    cache, ref = fresh(H, D, G, P, n)
    cache.codes.fill_(0xA5)
    cache.params.fill_(float("nan"))
    order, a = np.random.default_rng(seed).permutation(n), 0
    table, slots = np.full((len(lens), max(pages + [1])), -1, np.int32), []
    for b, (l, m) in enumerate(zip(lens, pages)):
        table[b, :m] = order[a:a + m]
        a += m
        t = np.arange(l)
        slots.append(table[b, t // P].astype(np.int64) * P + t % P)
    every = np.concatenate(slots)
    k, v, q = kv4_close.inputs((len(every), H, D), (n_q, H * R, D), dt, seed)
    kvc.kv4_append(cache, k.cuda(), v.cuda(), torch.from_numpy(every).cuda())
    ref.write(f32(k), f32(v), every)
    return cache, ref, table, slots, q


def run(H, D, G, P, lens, nqs, R, dt, room=0, seed=7, **call):
    """room: the table has pages for as many keys.  Outputs and lse, here and in 64 bits, and V's largest s."""
    import torch
    cache, ref, table, slots, q = hold(H, D, G, P, lens, sum(nqs), R, dt, seed)
    if room:
        table = widen(table, room, P)
    cu = torch.from_numpy(np.concatenate([[0], np.cumsum(nqs)]).astype(np.int32)).cuda()
    out, lse = kvc.kv4_attention(cache, q.cuda(), torch.from_numpy(table).cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                                 cu_q=cu, max_q=max(nqs), return_lse=True, **call)
    assert status(cache) == 0
    got, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
    wo, wl, q64, a = np.zeros_like(got), np.full_like(gl, -np.inf), q.double().numpy(), 0
    for l, n, at in zip(lens, nqs, slots):
        for h in range(H if l else 0):
            hs = slice(h * R, (h + 1) * R)
            k, v = ref.value(0, at)[:, h], ref.value(1, at)[:, h]
            assert np.abs(q64[a:a + n, hs] @ k.T).max() * D ** -0.5 < kv4_close.MOST
            wo[a:a + n, hs], wl[a:a + n, hs] = kv4_ref.attention(
                q64[a:a + n, hs], k, v, l - n + np.arange(n), l, call.get("causal", True), call.get("window", 0),
                call.get("softcap", 0.0), D ** -0.5)
        a += n
    assert (got[np.isneginf(wl)] == 0).all()
    return got, gl, wo, wl, float(ref.s[1].astype(np.float64).max())


def near(*args, **call):
    got, gl, wo, wl, _ = run(*args, **call)
    dt = args[7]
    o, e = kv4_close.out_off(got, wo, dt), kv4_close.lse_off(gl, wl)
    assert o <= 1 and e <= 1, (o, e)


@pytest.mark.parametrize("H,D,G,P", SHAPES)
@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("room", [0, 8192])
def test_decode(H, D, G, P, dt, room):
    say(f"[gpu] kv4 close decode H={H} D={D} G={G} P={P} {dt} room={room}")
    lens = [1, 0, 15, 16, 17, 31, 33, 128, 129, 300, 511, 512, 513, 700]
    near(H, D, G, P, lens, [1] * len(lens), 4, dt, room)


@pytest.mark.parametrize("H,D,G,P", SHAPES)
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_long_decode(H, D, G, P, dt):
    say(f"[gpu] kv4 close long decode H={H} D={D} G={G} P={P} {dt}")
    near(H, D, G, P, [5001, 37, 2048], [1, 1, 1], 4, dt)
    near(H, D, G, P, [5001, 37, 2048], [1, 1, 1], 4, dt, window=3001)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_very_long_decode(dt):
    say(f"[gpu] kv4 close 30001 keys {dt}")
    near(1, 128, 64, 64, [30001], [1], 8, dt)


@pytest.mark.parametrize("H,D,G,P", SHAPES)
@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("room", [0, 65536, 1 << 19])
@pytest.mark.parametrize("call", [dict(), dict(causal=False), dict(window=100), dict(softcap=6.0)],
                         ids=lambda c: "-".join(c) or "plain")
def test_several_queries(H, D, G, P, dt, room, call):
    say(f"[gpu] kv4 close queries H={H} D={D} G={G} P={P} {dt} room={room} {call}")
    # more queries than keys leave rows without a key; with room enough, blocks of 128 rows
    near(H, D, G, P, [333, 3, 64, 0, 131], [150, 5, 64, 2, 1], 3, dt, room, **call)


@pytest.mark.parametrize("R", [1, 2, 5, 8, 16, 17, 33])
@pytest.mark.parametrize("D,G", [(64, 32), (128, 64), (256, 128)])
def test_head_ratios(R, D, G):
    say(f"[gpu] kv4 close R={R} D={D}")
    near(2, D, G, 32, [70, 259], [1, 5], R, "f16")


@pytest.mark.parametrize("H,D,G,P", SHAPES)
@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("room", [0, 65536])
def test_one_key_a_row(H, D, G, P, dt, room):
    """out is the key's value lo + s n, which has few bits: one case of a hundred lies exactly between two numbers of the
    type, and some next to 0.  By element: half a step, and as for a dominant key 2^-22 of p s times 15 and the fp32
    steps of p s n and p lo, 2^-18 of the largest s."""
    say(f"[gpu] kv4 close one key H={H} D={D} G={G} P={P} {dt} room={room}")
    got, gl, wo, wl, smax = run(H, D, G, P, [333, 64, 1], [150, 64, 1], 3, dt, room, window=1)
    assert (np.abs(got - wo) <= kv4_close.STEP[dt] / 2 * np.abs(wo) + 2.0 ** -18 * smax).all()
    assert kv4_close.lse_off(gl, wl) <= 1


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("D,G", [(64, 64), (128, 64), (256, 128)])
@pytest.mark.parametrize("wide", [False, True])
def test_rounding_errors_do_not_add_up_over_many_keys(dt, D, G, wide):
    """20000 keys in one split, V of either sign: outputs are averages a hundred times smaller than what is summed.  A
    sum of N terms of either sign, rounded to fp32 at every step of 32, is off by about 2^-24 sqrt(N / 32) of itself,
    2^-19.4; with the logits' share and the two terms' as in kv4_close, of which most averages out: 2^-16 of |out|, in
    the mean, beyond the rounding, and four steps."""
    import torch
    say(f"[gpu] kv4 close 20000 keys {dt} D={D} G={G} wide={wide}")
    T, P, H, R, B, nq = 20000, 64, 8, 4, 64 if wide else 256, 32 if wide else 1
    n = -(-T // P)
    cache, ref = kvc.Kv4Cache(H, D, n, page_tokens=P, group=G), kv4_ref.Pool(2, D, G, P, n)  # two heads are looked at
    g = torch.Generator().manual_seed(21)
    t = {"bf16": torch.bfloat16, "f16": torch.float16}[dt]
    k, v, q = (torch.randn(s, generator=g).to(t) for s in ((T, H, D), (T, H, D), (nq, H * R, D)))
    slots = np.arange(T)
    kvc.kv4_append(cache, k.cuda(), v.cuda(), torch.from_numpy(slots).cuda())
    # as many sequences as leave no call for splits, all over the same pages with the same queries
    table = torch.arange(n, dtype=torch.int32).repeat(B, 1).cuda()
    lens = torch.full((B,), T, dtype=torch.int32).cuda()
    assert kvc.kv4_work_bytes(cache, B * nq, H * R, B, n, nq) == 0
    out, lse = kvc.kv4_attention(cache, q.repeat(B, 1, 1).cuda(), table, lens, return_lse=True)
    assert status(cache) == 0
    ref.write(f32(k[:, :2]), f32(v[:, :2]), slots)
    got, gl = out[:nq, :2 * R].double().cpu().numpy(), lse[:nq, :2 * R].double().cpu().numpy()
    wo, wl = np.zeros_like(got), np.zeros_like(gl)
    for h in range(2):
        hs = slice(h * R, (h + 1) * R)
        wo[:, hs], wl[:, hs] = kv4_ref.attention(q[:, hs].double().numpy(), ref.value(0, slots)[:, h], ref.value(1, slots)[:, h],
                                                 T - nq + np.arange(nq), T, True, 0, 0.0, D ** -0.5)
    off = np.abs(got - kv4_close.rounded(wo, dt)).sum()
    assert off <= 2.0 ** -16 * np.abs(wo).sum() + 4 * kv4_close.STEP[dt] * np.abs(wo).max()
    assert kv4_close.lse_off(gl, wl) <= 1
