"""kvc_kv4_tree_attention on the GPU over values of very different sizes, in blocks of 128 rows: sequences enough that a block
has all of its sequence's keys, or thousands.  All of them hold the same pages and ask the same, so one is compared with 64
bits, and the others with it.

Tolerance, row by row, with p normalised and out = sum_j p_j v_j:
  a key's logit is off by delta_j = (D + 16) 2^-24 scale log2e sum_c |q_c| (|lo_jc| + 31 s_jc), every product and sum rounded,
  and its exponential by 2^-18 (half a step of an exponent below 64, and its own last place): sum_j p_j delta_j |v_j - out|;
  p s enters as two fp16 terms, 22 bits of it, and none below 2^-25 where the row's largest p s is 2^7 or more, times codes up
  to 7.5 from their middle: 7.5 sum_j (2^-22 p_j s_j + 2^-32 max_i p_i s_i), s of the channel's group, of the key's largest in the maximum;
  sums over n keys, at most n/32 + 64 steps: as many 2^-24 of sum_j p_j (|mid_j| + 7.5 s_j), twice (the sum that divides);
  one rounding to the type.
lse: the largest p_j delta_j's sum, and those steps of |lse| + 1."""
import numpy as np
import pytest

import entropy_coding_02_amd as kvc
import kv4_ref
import kv4_spec_ref as spec
from gpu_util import say
from test_gpu_kv4 import EPS, build, f32, status, tdt
from test_gpu_kv4_tree import call, check, trees
from test_gpu_kv4_tree_rows import roomy

pytestmark = pytest.mark.gpu

R, N, P = 4, 32, 64  # heads of a group, tokens of a tree, of a page: 128 rows


def near(out, lse, q, ref, slots, ok, dt):
    """out [n][R][D], lse [n][R] of KV head 0 within what the docstring allows."""
    D, G = ref.D, ref.G
    out, lse, q = (t.double().cpu().numpy() for t in (out, lse, q))
    k, v = ref.value(0, slots)[:, 0], ref.value(1, slots)[:, 0]
    ks, kl, vs, vl = (np.repeat(x[i, slots, 0].astype(np.float64), G, -1) for i in (0, 1) for x in (ref.s, ref.lo))
    mid, top = np.abs(vl + 7.5 * vs), vs.max(-1)
    steps = (len(slots) / 32 + 64) * 2.0 ** -24
    for i in range(out.shape[0]):
        see = ok[i]
        for r in range(out.shape[1]):
            x = k[see] @ q[i, r] * D ** -0.5
            m = x.max()
            p = np.exp(x - m)
            total = p.sum()
            p /= total
            want = p @ v[see]
            delta = (D + 16) * 2.0 ** -24 * D ** -0.5 * 1.4427 * ((np.abs(kl) + 31 * ks)[see] @ np.abs(q[i, r])) + 2.0 ** -18
            tol = (p * delta) @ np.abs(v[see] - want) * 1.01
            tol += 7.5 * (2.0 ** -22 * (p @ vs[see]) + see.sum() * 2.0 ** -32 * (p * top[see]).max())
            tol += 2 * steps * (p @ (mid + 7.5 * vs)[see]) + EPS[dt] / 2 * np.abs(want)
            off = np.abs(out[i, r] - want)
            assert (off <= tol).all(), (i, r, off.max(), tol[off.argmax()], want[off.argmax()])
            wl = m + np.log(total)
            assert abs(lse[i, r] - wl) <= p @ delta + steps * (abs(wl) + 1), (i, r, lse[i, r], wl)


def shared(B, D, G, logits, sizes, dt, seed, tree="bushy", signed=True):
    """One tree of N tokens behind len(logits) - N keys, which B sequences hold; the keys' logits about as given, the values' sizes."""
    import torch
    T = len(logits)
    g = torch.Generator().manual_seed(seed)
    k = torch.randn((T, 1, D), generator=g) * 0.05 + torch.tensor(logits).view(T, 1, 1) * D ** -0.5
    v = (torch.rand((T, 1, D), generator=g) * 0.5 + 0.5) * torch.tensor(sizes).view(T, 1, 1)
    if signed:
        v = v * torch.where(torch.rand(v.shape, generator=g) < 0.5, -1.0, 1.0)
    q = 1.0 + torch.randn((N, R, D), generator=g) * 0.05
    k, v, q = (t.to(tdt(dt)) for t in (k, v, q))
    n = -(-T // P)
    cache, ref = kvc.Kv4Cache(1, D, n, page_tokens=P, group=G), kv4_ref.Pool(1, D, G, P, n)
    slots = np.arange(T)
    kvc.kv4_append(cache, k.cuda(), v.cuda(), torch.from_numpy(slots).cuda())
    ref.write(f32(k), f32(v), slots)
    par = trees([N], seed, tree)[0]
    table = np.tile(np.arange(n, dtype=np.int32), (B, 1))
    return cache, ref, q, table, slots, par


def run(B, cache, q, table, T, par):
    out, lse = call(cache, q.repeat(B, 1, 1), table, [T] * B, [par] * B)
    assert status(cache) == 0
    out, lse = out.view(B, N, R, -1), lse.view(B, N, R)
    assert (out == out[:1]).all() and (lse == lse[:1]).all()
    return out[0], lse[0]


def kinds(kind, T):
    """Logits and sizes of V."""
    logits, sizes = np.zeros(T, np.float32), np.full(T, 0.1, np.float32)
    if kind.startswith("beside"):  # the key that rows look at has a neighbour 2^k times the others that they do not
        logits[37], logits[38] = 12.0, -48.0
        sizes[38] *= 2.0 ** int(kind[6:])
    elif kind == "first":          # a large tile, then many small keys of a larger weight in all
        logits[16:] = -8.6
        logits[:16] -= 20.0
        logits[5] = 0.0
        sizes[:16], sizes[16:] = 4096.0, 0.01
    elif kind == "huge":
        logits[:] = -7.14
        logits[3] = 0.0
        sizes[:], sizes[3] = 0.007, 50000.0
    elif kind == "tiles":          # from 2^-12 to 2^10, a tile of 16 keys each
        sizes = 2.0 ** ((np.arange(T) // 16 * 7) % 23 - 12.0)
        logits -= 0.4 * np.log2(sizes)
    elif kind == "last":           # small ones first
        logits[:-N - 16] = 3.0
        sizes[:-N - 16], sizes[-N - 16:] = 0.001, 8000.0
    return logits.astype(np.float32), sizes.astype(np.float32)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("kind", ["beside12", "beside16", "beside18", "first", "huge", "tiles", "last"])
def test_sizes_that_differ(kind, dt):
    T, B = 8192, 1024
    say(f"[gpu] kv4 tree of many rows, values of sizes {kind} {dt}")
    logits, sizes = kinds(kind, T)
    cache, ref, q, table, slots, par = shared(B, 128, 64, logits, sizes, dt, 3, signed=kind not in ("first", "huge"))
    out, lse = run(B, cache, q, table, T, par)
    near(out, lse, q, ref, slots, spec.sees(par, T, 0), dt)


@pytest.mark.parametrize("D,G", [(128, 32), (128, 128), (256, 32), (256, 64), (64, 32)])
@pytest.mark.parametrize("kind", ["beside18", "huge", "tiles"])
def test_sizes_that_differ_by_shape(D, G, kind):
    T, B = 4000, 1024
    say(f"[gpu] kv4 tree of many rows, values of sizes {kind} D={D} G={G}")
    logits, sizes = kinds(kind, T)
    cache, ref, q, table, slots, par = shared(B, D, G, logits, sizes, "bf16", 4, signed=kind != "huge")
    out, lse = run(B, cache, q, table, T, par)
    near(out, lse, q, ref, slots, spec.sees(par, T, 0), "bf16")


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("D,G", [(128, 32), (128, 64), (128, 128), (256, 64), (64, 32)])
def test_few_heavy_keys(D, G, dt):
    """Outputs that a handful of keys make: a share of 2^-11 of each would show."""
    T, B = 1500, 1024
    say(f"[gpu] kv4 tree of many rows, few heavy keys D={D} G={G} {dt}")
    logits = np.full(T, -30.0, np.float32)
    logits[np.random.default_rng(5).permutation(T - N)[:6]] = 0.0
    cache, ref, q, table, slots, par = shared(B, D, G, logits, np.ones(T, np.float32), dt, 5)
    out, lse = run(B, cache, q, table, T, par)
    near(out, lse, q, ref, slots, spec.sees(par, T, 0), dt)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("D,G", [(128, 32), (128, 64), (64, 32), (256, 64)])
def test_a_sibling_far_larger_changes_nothing(D, G, dt):
    """Whatever lies, finite, at a key that a token does not see: every bit of its outputs stays."""
    import torch
    T, B = 1000 + N, 256
    say(f"[gpu] kv4 tree of many rows, a far larger sibling D={D} G={G} {dt}")
    cache, ref, q, table, slots, par = shared(B, D, G, np.zeros(T, np.float32), np.full(T, 1e-3, np.float32), dt, 6)
    out, lse = run(B, cache, q, table, T, par)
    ok = spec.sees(par, T, 0)
    near(out, lse, q, ref, slots, ok, dt)
    for tok in (0, 3, N - 1):
        unseen = torch.from_numpy(~ok[:, T - N + tok]).cuda()
        assert unseen.any()
        k, v = torch.full((2, 1, 1, D), 3.0).to(tdt(dt)), torch.full((1, 1, D), 60000.0).to(tdt(dt))
        v[..., ::2] *= -1
        at = torch.tensor([T - N + tok]).cuda()
        before = cache.codes.clone(), cache.params.clone()
        kvc.kv4_append(cache, k[0].cuda(), v.cuda(), at)
        o, l = run(B, cache, q, table, T, par)
        assert torch.equal(o[unseen], out[unseen]) and torch.equal(l[unseen], lse[unseen])
        assert not torch.equal(o[~unseen], out[~unseen])
        cache.codes.copy_(before[0])
        cache.params.copy_(before[1])


@pytest.mark.parametrize("D,G,dt,softcap", [(128, 32, "f16", 0.0), (128, 64, "f16", 20.0), (128, 128, "bf16", 0.0), (256, 64, "f16", 0.0),
                                            (64, 64, "bf16", 20.0)])
def test_a_window_within_long_sequences(D, G, dt, softcap):
    """Windows that mask inside such blocks, by the path, with and without a cap."""
    lens, nqs, H = [6000, 700, 5700] * 4, [60, 31, 64] * 4, 4
    say(f"[gpu] kv4 tree of many rows, long windows D={D} G={G} {dt}")
    cache, ref, table, slots = build(H, D, G, 32, lens, dt, 37)
    check(cache, ref, table, slots, lens, trees(nqs, 37), 2, dt, window=2500, softcap=softcap)


@pytest.mark.parametrize("D,G,heads,n,dt", [(256, 32, 2, 1024, "f16"), (256, 32, 1, 590, "bf16"), (128, 64, 8, 640, "f16"), (128, 128, 2, 128, "bf16"),
                                            (128, 32, 1, 1024, "bf16")])
def test_paths_that_fill_a_block(D, G, heads, n, dt):
    """The largest trees whose paths a block of 128 rows still has room for, and one that goes to tiles."""
    lens = [n + 333, n + 64]
    say(f"[gpu] kv4 tree of {n}, {heads} heads of {D}, G={G} {dt}")
    cache, ref, table, slots = build(1, D, G, 64, lens, dt, 38)
    check(cache, ref, roomy(table, 1, 64, n * heads), slots, lens, [trees([n], 38)[0], trees([n], 39, "chain")[0]], heads, dt)
