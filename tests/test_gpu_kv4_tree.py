"""kvc_kv4_tree_attention on the GPU against 64 bits, over trees of every kind.

Tolerance: that of test_gpu_kv4.py, whose derivation holds for these kernels (the logits are the same; p s, or p, enters as
two fp16 terms, nearer than the bf16 ones counted there), and one more for bf16 outputs of trees of more than 32 rows, whose p
may be one fp16 term: with p_j (1 + d_j), |d_j| <= 2^-11 (fp16's half step), in the sum that divides too,
    out' - out = sum_j p_j d_j (v_j - out) / sum_j p_j (1 + d_j),
at most 2^-11 / (1 - 2^-11) of sum_j p_j |v_j - out|, p normalised."""
import math

import numpy as np
import pytest

import entropy_coding_02_amd as kvc
import kv4_spec_ref as spec
from gpu_util import say
from test_gpu_kv4 import EPS, SHAPES, build, draw, status

pytestmark = pytest.mark.gpu


def trees(nqs, seed, shape="bushy"):
    rng = np.random.default_rng(seed)
    return [spec.random_tree(n, rng, shape) for n in nqs]


def ints(x):
    import torch
    return torch.tensor(x, dtype=torch.int32).cuda()


def call(cache, q, table, lens, pars, **kw):
    import torch
    nqs = [len(p) for p in pars]
    cu = np.concatenate([[0], np.cumsum(nqs)])
    return kvc.kv4_tree_attention(cache, q.cuda(), torch.from_numpy(table).cuda(), ints(lens), ints(sum(pars, [])), cu_q=ints(cu),
                                  max_q=max(nqs), return_lse=True, **kw)


def check(cache, ref, table, slots, lens, pars, R, dt, window=0, softcap=0.0, scale=None, seed=50, **kw):
    q = draw((sum(len(p) for p in pars), ref.H * R, ref.D), dt, seed)
    scale = ref.D ** -0.5 if scale is None else scale
    out, lse = call(cache, q, table, lens, pars, window=window, softcap=softcap, scale=scale, **kw)
    assert status(cache) == 0
    compare(out, lse, q, ref, slots, lens, pars, R, dt, window, softcap, scale)
    return out, lse


def compare(out, lse, q, ref, slots, lens, pars, R, dt, window, softcap, scale):
    out, lse, q64 = out.double().cpu().numpy(), lse.double().cpu().numpy(), q.double().cpu().numpy()
    D, a = ref.D, 0
    for b, par in enumerate(pars):
        n, l = len(par), max(lens[b], 0)
        ok = spec.sees(par, l, window)
        for h in range(ref.H):
            hs = slice(h * R, (h + 1) * R)
            k, v = ref.value(0, slots[b])[:, h], ref.value(1, slots[b])[:, h]
            wo, wl = spec.attention(q64[a:a + n, hs], k, v, ok, softcap, scale)
            got, gl = out[a:a + n, hs], lse[a:a + n, hs]
            empty = np.isneginf(wl)
            assert np.array_equal(np.isneginf(gl), empty) and (got[empty] == 0).all()
            if empty.all():
                continue
            ks, kl = (np.repeat(x[0, slots[b], h].astype(np.float64), ref.G, -1) for x in (ref.s, ref.lo))
            reach = (np.abs(kl) + 31 * ks).max(0)
            delta = (D + 16) * 2.0 ** -24 * abs(scale) * 1.4427 * (np.abs(q64[a:a + n, hs]) @ reach)
            smax, vmax = ref.s[1, slots[b], h].astype(np.float64).max(), np.abs(v).max()
            steps = (l / 32 + 64) * 2.0 ** -24
            tol = EPS[dt] / 2 * np.abs(wo) + (2 * delta * vmax + 31 * 2.0 ** -18 * smax + steps * (vmax + 31 * smax))[..., None]
            if dt == "bf16" and max(len(p) for p in pars) * R > 32:
                tol += 2.0 ** -11 / (1 - 2.0 ** -11) * spec.spread(q64[a:a + n, hs], k, v, ok, softcap, scale)
            assert (np.abs(got - wo) <= tol)[~empty].all(), (b, h, np.abs(got - wo).max(), tol.min())
            assert (np.abs(gl[~empty] - wl[~empty]) <= (delta + steps * (np.abs(np.where(empty, 0, wl)) + 1))[~empty]).all(), (b, h)
        a += n


@pytest.mark.parametrize("H,D,G,P", SHAPES)
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_lengths_and_sizes(H, D, G, P, dt):
    lens, nqs = [1, 9, 33, 64, 65, 200, 131, 300], [1, 9, 2, 1, 33, 40, 7, 64]
    say(f"[gpu] kv4 tree H={H} D={D} G={G} P={P} {dt}")
    cache, ref, table, slots = build(H, D, G, P, lens, dt, 11)
    check(cache, ref, table, slots, lens, trees(nqs, 1), 4, dt)


@pytest.mark.parametrize("R", [1, 2, 3, 5, 8, 17])
@pytest.mark.parametrize("D,G", [(64, 32), (128, 64), (256, 128)])
def test_head_ratios(R, D, G):
    lens, nqs = [70, 259, 40], [16, 33, 5]
    say(f"[gpu] kv4 tree R={R} D={D}")
    cache, ref, table, slots = build(2, D, G, 32, lens, "f16", 12)
    check(cache, ref, table, slots, lens, trees(nqs, 2), R, "f16")


@pytest.mark.parametrize("shape", ["chain", "flat", "bushy"])
@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 100, 257])
def test_kinds_of_trees(shape, n):
    lens = [n + 3, n + 45, n]
    say(f"[gpu] kv4 tree {shape} of {n}")
    cache, ref, table, slots = build(1, 64, 64, 16, lens, "f16", 13)
    check(cache, ref, table, slots, lens, trees([n] * 3, 3, shape), 2, "f16")


@pytest.mark.parametrize("R", [1, 2])
def test_the_largest_tree(R):
    lens = [1024 + 31, 1024 + 700]
    say(f"[gpu] kv4 tree of 1024, R={R}")
    cache, ref, table, slots = build(1, 64, 32, 64, lens, "f16", 14)
    check(cache, ref, table, slots, lens, trees([1024, 900], 4), R, "f16")
    check(cache, ref, table, slots, lens, trees([1024, 1024], 5, "chain"), R, "f16", window=100)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_more_tokens_than_keys(dt):
    """Rows without a key, and sequences without any."""
    lens, nqs = [3, 0, 20, -5, 1], [9, 4, 40, 3, 2]
    say(f"[gpu] kv4 tree short {dt}")
    cache, ref, table, slots = build(2, 128, 64, 16, lens, dt, 15)
    for shape in ("bushy", "chain", "flat"):
        check(cache, ref, table, slots, lens, trees(nqs, 6, shape), 3, dt)
        check(cache, ref, table, slots, lens, trees(nqs, 6, shape), 3, dt, window=2)


@pytest.mark.parametrize("window", [1, 2, 3, 31, 100, 128, 10000])
@pytest.mark.parametrize("D,G", [(64, 64), (128, 64), (256, 32)])
def test_window(window, D, G):
    """Windows shorter than the paths too; pages wholly behind the first token's window have been given away."""
    lens, nqs = [300, 37, 160, 9, 400], [40, 1, 13, 9, 64]
    say(f"[gpu] kv4 tree window={window} D={D}")
    cache, ref, table, slots = build(2, D, G, 16, lens, "bf16", 16)
    for b, (l, n) in enumerate(zip(lens, nqs)):
        table[b, :max(0, l - n - window + 1) // 16] = -1
    for shape in ("bushy", "chain"):
        check(cache, ref, table, slots, lens, trees(nqs, 7, shape), 2, "bf16", window=window)


@pytest.mark.parametrize("softcap,scale", [(30.0, None), (5.0, 1.0), (0.0, 2.0), (0.0, 0.0), (50.0, -0.5)])
def test_softcap_and_scale(softcap, scale):
    lens, nqs = [300, 33], [24, 20]
    say(f"[gpu] kv4 tree softcap={softcap} scale={scale}")
    cache, ref, table, slots = build(2, 128, 64, 16, lens, "f16", 17)
    check(cache, ref, table, slots, lens, trees(nqs, 8), 4, "f16", softcap=softcap, scale=scale)


@pytest.mark.parametrize("dt,lens,nqs", [("bf16", [5000], [33]), ("f16", [9001, 37], [5, 37]), ("bf16", [2049, 0, 4096], [3, 2, 60]),
                                         ("f16", [12345], [64])])
def test_long_keys_are_split(dt, lens, nqs):
    say(f"[gpu] kv4 tree split {lens}")
    cache, ref, table, slots = build(2, 128, 64, 64, lens, dt, 18)
    assert kvc.kv4_tree_work_bytes(cache, sum(nqs), 8, len(lens), table.shape[1], max(nqs)) > 0
    check(cache, ref, table, slots, lens, trees(nqs, 9), 4, dt)
    check(cache, ref, table, slots, lens, trees(nqs, 9), 4, dt, window=3000)


@pytest.mark.parametrize("D,G", [(64, 32), (128, 128), (256, 64)])
def test_a_chain_is_causal_attention(D, G):
    """The outputs of kv4_attention: both near the same value, a step of the type apart at most where it lies between two,
    and what p in one term may move it by (above)."""
    import torch
    lens, nq = [500, 129, 64], 20
    cache, ref, table, slots = build(2, D, G, 32, lens, "bf16", 19)
    q = draw((3 * nq, 8, D), "bf16", 51).cuda()
    tab, par = torch.from_numpy(table).cuda(), ints(list(range(-1, nq - 1)) * 3)
    for kw in (dict(), dict(window=37), dict(softcap=10.0)):
        a, la = kvc.kv4_tree_attention(cache, q, tab, ints(lens), par, return_lse=True, **kw)
        b, lb = kvc.kv4_attention(cache, q, tab, ints(lens), return_lse=True, **kw)
        moved = torch.empty(a.shape, dtype=torch.float64)
        for i, l in enumerate(lens):
            for hd in range(2):
                at, hs = slice(i * nq, (i + 1) * nq), slice(4 * hd, 4 * hd + 4)
                k, v = ref.value(0, slots[i])[:, hd], ref.value(1, slots[i])[:, hd]
                ok = spec.sees(list(range(-1, nq - 1)), l, kw.get("window", 0))
                moved[at, hs] = torch.from_numpy(spec.spread(q[at, hs].double().cpu().numpy(), k, v, ok, kw.get("softcap", 0.0), D ** -0.5))
        moved = moved.cuda() * (2.0 ** -11 / (1 - 2.0 ** -11))
        assert ((a.double() - b.double()).abs() <= 2.0 ** -7 * b.double().abs() + 1e-6 + moved).all()
        assert ((la - lb).abs() <= 2.0 ** -20 * (lb.abs() + 1)).all()
    assert status(cache) == 0


@pytest.mark.parametrize("nq", [4, 40])
def test_what_a_token_does_not_see_does_not_reach_it(nq):
    """NaN in a sibling's keys and values, and behind the sequence."""
    import torch
    n0, R = 70, 4
    lens, pars = [n0 + nq], trees([nq], 10)
    cache, ref, table, slots = build(1, 128, 64, 16, lens, "bf16", 20)
    q = draw((nq, R, 128), "bf16", 52)
    good, _ = call(cache, q, table, lens, pars)
    bad = 1
    seen = spec.sees(pars[0], lens[0], 0)[:, n0 + bad]
    assert seen.any() and not seen.all()
    for side in (0, 1):
        x = torch.zeros((2, 1, 1, 128), dtype=torch.bfloat16, device="cuda")
        x[side, 0, 0, 100] = math.nan
        kvc.kv4_append(cache, x[0], x[1], torch.from_numpy(slots[0][n0 + bad:n0 + bad + 1]).cuda())
        assert status(cache) == kvc.KVC_DEV_NONFINITE
        out, lse = call(cache, q, table, lens, pars)
        nan = torch.isnan(out).any(-1).any(-1).cpu().numpy()
        assert np.array_equal(nan, seen)
        assert torch.equal(out[torch.from_numpy(~seen).cuda()], good[torch.from_numpy(~seen).cuda()])
    assert status(cache) == 0


def test_bad_parents_pages_and_lengths_are_flagged():
    import torch
    lens, nqs = [100, 100], [6, 6]
    cache, ref, table, slots = build(1, 64, 32, 16, lens, "bf16", 21)
    q = draw((12, 4, 64), "bf16", 53)
    pars = trees(nqs, 11)
    good, lse = call(cache, q, table, lens, pars)
    assert status(cache) == 0
    compare(good, lse, q, ref, slots, lens, pars, 4, "bf16", 0, 0.0, 0.125)
    for worse in ([-1, 1, 0, 0, 0, 0], [-1, 0, -2, 0, 0, 0], [5, 0, 0, 0, 0, 0], [-1, 0, 2 ** 31 - 1, 0, 0, 0], [-1, 0, 0, 0, 5, 0],
                  [-1, 0, 0, -2 ** 31, 0, 0], [-1, 0, 65536, 0, 0, 0], [-1, 65535, 0, 0, 0, 0]):
        out, _ = call(cache, q, table, lens, [pars[0], worse])
        assert status(cache) == kvc.KVC_DEV_BAD_INDEX and torch.equal(out[:6], good[:6])
        # a bad parent is none
        mended, ml = call(cache, q, table, lens, [pars[0], [p if -1 <= p < i else -1 for i, p in enumerate(worse)]])
        assert status(cache) == 0 and torch.equal(out, mended)
    for entry in (-1, cache.n_pages, 2 ** 31 - 1):
        t = table.copy()
        t[1, 2] = entry
        out, _ = call(cache, q, t, lens, pars)
        assert status(cache) == kvc.KVC_DEV_BAD_INDEX and torch.equal(out[:6], good[:6])
    out, _ = call(cache, q, table, [100, table.shape[1] * 16 + 1], pars)
    assert status(cache) == kvc.KVC_DEV_BAD_INDEX and torch.equal(out[:6], good[:6])
    for cu in ((0, 6, 13), (0, 6, 5), (-4, 6, 12), (0, 6, 2 ** 31 - 1), (0, 2 ** 31 - 1, 12), (0, 0, 12)):
        kvc.kv4_tree_attention(cache, q.cuda(), torch.from_numpy(table).cuda(), ints(lens), ints(sum(pars, [])), cu_q=ints(cu), max_q=6)
        assert status(cache) == kvc.KVC_DEV_BAD_INDEX, cu


@pytest.mark.parametrize("lens", [[100, 40], [9000, 40]])
def test_strides_given_buffers_and_rows_of_no_sequence(lens):
    import torch
    pars, R, H, D = trees([11, 5], 12), 2, 3, 128
    cache, ref, table, slots = build(H, D, 64, 16, lens, "f16", 22)
    wide = torch.full((2, table.shape[1] + 9), -5, dtype=torch.int32)
    wide[:, :table.shape[1]] = torch.from_numpy(table)
    n_q = 20  # two before the first sequence's, two behind the last's
    big = torch.full((n_q, 3, H * R, D + 1), 7.0, dtype=torch.float16, device="cuda")
    q = draw((n_q, H * R, D), "f16", 54)
    qd = torch.zeros((n_q, H * R + 1, D + 1), dtype=torch.float16, device="cuda")[:, 1:, 1:]
    qd.copy_(q)
    lse = torch.full((n_q, H * R), 5.0, dtype=torch.float32, device="cuda")
    out = big[:, 1, :, 1:]
    work = torch.empty(kvc.kv4_tree_work_bytes(cache, n_q, H * R, 2, table.shape[1], 11), dtype=torch.uint8, device="cuda")
    par = ints([99, 99] + pars[0] + pars[1] + [99, 99])
    kvc.kv4_tree_attention(cache, qd, wide.cuda()[:, :table.shape[1]], ints(lens), par, cu_q=ints([2, 13, 18]), max_q=11, out=out,
                           lse=lse, work=work)
    assert status(cache) == 0
    compare(out[2:18], lse[2:18], q[2:18], ref, slots, lens, pars, R, "f16", 0, 0.0, D ** -0.5)
    assert (big[:, 0] == 7.0).all() and (big[:, 2] == 7.0).all() and (big[:, 1, :, 0] == 7.0).all()
    for t in (big, lse):
        rest = t[[0, 1, 18, 19]]
        assert (rest == rest.flatten()[0]).all()


def test_other_streams_and_repeats():
    import torch
    from test_gpu_kv4_streams import busy
    lens, nqs = [9001, 20, 333], [30, 20, 7]
    cache, ref, table, slots = build(2, 128, 64, 16, lens, "bf16", 23)
    pars = trees(nqs, 13)
    q, tab, ln, par, cu = draw((57, 8, 128), "bf16", 55).cuda(), torch.from_numpy(table).cuda(), ints(lens), ints(sum(pars, [])), ints([0, 30, 50, 57])
    want, wl = kvc.kv4_tree_attention(cache, q, tab, ln, par, cu_q=cu, max_q=30, return_lse=True)
    again, al = kvc.kv4_tree_attention(cache, q, tab, ln, par, cu_q=cu, max_q=30, return_lse=True)
    assert torch.equal(want, again) and torch.equal(wl, al)  # a fixed order of sums
    nb = kvc.kv4_tree_work_bytes(cache, 57, 8, 3, tab.shape[1], 30)
    x = torch.zeros((4096, 4096), dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        busy(x)
    out, lse = kvc.kv4_tree_attention(cache, q, tab, ln, par, cu_q=cu, max_q=30, return_lse=True, stream=s)
    others = [torch.full((nb,), 7, dtype=torch.uint8, device="cuda") for _ in range(8)]
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, wl) and all(bool((t == 7).all()) for t in others)
    assert status(cache) == 0


@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_tiny_and_huge_values(dt):
    import torch
    from test_gpu_kv4 import f32, fresh, tdt
    H, D, G, P, T, n = 1, 128, 64, 16, 200, 40
    pars = trees([n], 14)
    for kmul, vmul, qmul in ((1.0, 1e-3, 1.0), (1.0, 6000.0, 1.0), (1000.0, 1.0, 1e-4), (1e-3, 1.0, 3e4)):
        cache, ref = fresh(H, D, G, P, 14)
        k, v = draw((T, H, D), dt, 95, kmul), draw((T, H, D), dt, 96, vmul)
        slots = np.arange(T)
        kvc.kv4_append(cache, k.cuda(), v.cuda(), torch.from_numpy(slots).cuda())
        ref.write(f32(k), f32(v), slots)
        q = (draw((n, 4, D), dt, 97).float() * qmul).clamp(-6e4, 6e4).to(tdt(dt))
        out, lse = call(cache, q, np.arange(13, dtype=np.int32)[None], [T], pars)
        assert status(cache) == 0
        compare(out, lse, q, ref, [slots], [T], pars, 4, dt, 0, 0.0, D ** -0.5)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_sums_over_many_keys_keep_every_key(dt):
    """Near enough to 64 bits that a lost key among thousands shows (kv4_close)."""
    import kv4_close
    import torch
    from test_gpu_kv4 import f32
    import kv4_ref
    H, D, G, P, R, T, n = 2, 128, 64, 64, 4, 6000, 24
    pages = -(-T // P)
    cache, ref = kvc.Kv4Cache(H, D, pages, page_tokens=P, group=G), kv4_ref.Pool(H, D, G, P, pages)
    k, v, q = kv4_close.inputs((T, H, D), (n, H * R, D), dt, 60)
    slots = np.arange(T)
    kvc.kv4_append(cache, k.cuda(), v.cuda(), torch.from_numpy(slots).cuda())
    ref.write(f32(k), f32(v), slots)
    pars = trees([n], 15)
    out, lse = call(cache, q, np.arange(pages, dtype=np.int32)[None], [T], pars)
    assert status(cache) == 0
    ok = spec.sees(pars[0], T, 0)
    for h in range(H):
        hs = slice(h * R, (h + 1) * R)
        wo, wl = spec.attention(q[:, hs].double().numpy(), ref.value(0, slots)[:, h], ref.value(1, slots)[:, h], ok, 0.0, D ** -0.5)
        assert kv4_close.lse_off(lse[:, hs].double().cpu().numpy(), wl) <= 1.0
        assert kv4_close.out_off(out[:, hs].double().cpu().numpy(), wo, dt) <= 1.0


def outlying(H, D, G, P, R, T, n, dt, table_of=lambda t: t):
    """One channel of each group 64 times the others: what the others lose to its s shows, channel by channel."""
    import torch
    from test_gpu_kv4 import f32, fresh
    cache, ref = fresh(H, D, G, P, -(-T // P))
    k, v = draw((T, H, D), dt, 61), draw((T, H, D), dt, 62)
    v[..., ::G] = v[..., ::G].abs() * 64
    slots = np.arange(T)
    kvc.kv4_append(cache, k.cuda(), v.cuda(), torch.from_numpy(slots).cuda())
    ref.write(f32(k), f32(v), slots)
    pars, q = trees([n], 16), draw((n, H * R, D), dt, 63, 3.0)
    out, lse = call(cache, q, table_of(np.arange(-(-T // P), dtype=np.int32)[None]), [T], pars)
    assert status(cache) == 0
    compare(out, lse, q, ref, [slots], [T], pars, R, dt, 0, 0.0, D ** -0.5)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("n,R", [(3, 2), (16, 2), (24, 4)])
def test_outlying_channels(dt, n, R):
    outlying(2, 128, 64, 16, R, 70, n, dt)
