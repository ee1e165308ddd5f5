"""kvc_kv4_tree_attention on the GPU with trees of many rows: blocks of 128 rows, which the kernel takes where 7/8 of
their waves have rows and the tables' keys fill the chip, here by tables far wider than the sequences are long.

Tolerance: test_gpu_kv4_tree.py's, which counts p's one term for bf16."""
import math

import numpy as np
import pytest

import entropy_coding_02_amd as kvc
import kv4_spec_ref as spec
from gpu_util import say
from test_gpu_kv4 import build, draw, f32, fresh, status, tdt
from test_gpu_kv4_tree import call, check, compare, ints, outlying, trees

pytestmark = pytest.mark.gpu


def roomy(table, H, P, rows):
    """The table with room for so many keys that blocks of 128 rows are taken; what no sequence reaches is no page."""
    tiles = -(-rows // 128)
    assert -(-rows // 32) * 8 >= tiles * 28, "rows that fill the blocks"
    pages = 1024 * (-(-512 // (len(table) * H * tiles))) // P
    wide = np.full((len(table), max(pages, table.shape[1])), -1, table.dtype)
    wide[:, :table.shape[1]] = table
    return wide


@pytest.mark.parametrize("H,D,G,P", [(2, 128, 32, 16), (1, 128, 64, 64), (3, 128, 128, 32), (2, 256, 32, 128), (1, 256, 32, 16)])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_lengths_and_sizes(H, D, G, P, dt):
    lens, nqs = [1, 9, 33, 64, 65, 200, 131, 300, 1030], [1, 9, 2, 1, 32, 30, 7, 31, 3]
    say(f"[gpu] kv4 tree of many rows H={H} D={D} G={G} P={P} {dt}")
    cache, ref, table, slots = build(H, D, G, P, lens, dt, 31)
    check(cache, ref, roomy(table, H, P, 128), slots, lens, trees(nqs, 31), 4, dt)


@pytest.mark.parametrize("R,nq", [(1, 128), (1, 225), (2, 57), (3, 42), (5, 51), (7, 16), (17, 15), (33, 30)])
def test_head_ratios(R, nq):
    lens, nqs = [70, 259, 400], [16, nq, 5]
    say(f"[gpu] kv4 tree of many rows R={R} n={nq}")
    cache, ref, table, slots = build(2, 128, 64, 32, lens, "f16", 32)
    check(cache, ref, roomy(table, 2, 32, nq * R), slots, lens, trees(nqs, 32), R, "f16")


@pytest.mark.parametrize("D,R", [(128, 1), (128, 2), (256, 1)])
def test_the_largest_tree(D, R):
    lens = [1024 + 31, 1024 + 300]
    say(f"[gpu] kv4 tree of 1024, many rows, D={D} R={R}")
    cache, ref, table, slots = build(1, D, 32, 64, lens, "bf16", 33)
    table = roomy(table, 1, 64, 1024 * R)
    check(cache, ref, table, slots, lens, trees([1024, 900], 33), R, "bf16")
    check(cache, ref, table, slots, lens, trees([1024, 1024], 34, "chain"), R, "bf16", window=100)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_more_tokens_than_keys(dt):
    lens, nqs = [3, 0, 20, -5, 1, 41], [9, 4, 40, 3, 2, 42]
    say(f"[gpu] kv4 tree of many rows, few keys, {dt}")
    cache, ref, table, slots = build(2, 128, 64, 16, lens, dt, 35)
    for shape in ("bushy", "chain", "flat"):
        for window in (0, 2):
            check(cache, ref, roomy(table, 2, 16, 126), slots, lens, trees(nqs, 35, shape), 3, dt, window=window)


@pytest.mark.parametrize("window", [1, 3, 31, 128, 30000])
@pytest.mark.parametrize("D,G", [(256, 32), (128, 64)])
def test_window(window, D, G):
    """A short window leaves too few keys for such blocks: both kinds from one workspace's size."""
    lens, nqs = [300, 37, 160, 9, 400], [40, 1, 13, 9, 64]
    say(f"[gpu] kv4 tree of many rows, window={window} D={D}")
    cache, ref, table, slots = build(2, D, G, 16, lens, "bf16", 36)
    for b, (l, n) in enumerate(zip(lens, nqs)):
        table[b, :max(0, l - n - window + 1) // 16] = -1
    check(cache, ref, roomy(table, 2, 16, 128), slots, lens, trees(nqs, 36), 2, "bf16", window=window)


def test_a_window_within_long_sequences():
    """Long enough for such blocks even so: what rows of one wave do not all see."""
    lens, nqs, H = [9000, 700, 8700] * 4, [60, 31, 64] * 4, 8
    say("[gpu] kv4 tree of many rows, long windows")
    cache, ref, table, slots = build(H, 128, 32, 64, lens, "bf16", 37)
    check(cache, ref, table, slots, lens, trees(nqs, 37), 2, "bf16", window=2500)


@pytest.mark.parametrize("softcap,scale", [(30.0, None), (5.0, 1.0), (0.0, 2.0), (0.0, 0.0), (50.0, -0.5)])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_softcap_and_scale(softcap, scale, dt):
    lens, nqs = [300, 33], [32, 20]
    say(f"[gpu] kv4 tree of many rows, softcap={softcap} scale={scale} {dt}")
    cache, ref, table, slots = build(2, 128, 64, 16, lens, dt, 38)
    check(cache, ref, roomy(table, 2, 16, 128), slots, lens, trees(nqs, 38), 4, dt, softcap=softcap, scale=scale)


@pytest.mark.parametrize("dt,lens,nqs", [("bf16", [5000], [57]), ("f16", [9001, 137], [64, 37]), ("bf16", [2049, 0, 4096], [3, 2, 60])])
def test_long_keys_are_split(dt, lens, nqs):
    say(f"[gpu] kv4 tree of many rows, split {lens}")
    cache, ref, table, slots = build(2, 128, 64, 64, lens, dt, 39)
    table = roomy(table, 2, 64, max(nqs) * 4)
    check(cache, ref, table, slots, lens, trees(nqs, 39), 4, dt)
    check(cache, ref, table, slots, lens, trees(nqs, 39), 4, dt, window=70000)


@pytest.mark.parametrize("G", [32, 64, 128])
def test_what_a_token_does_not_see_does_not_reach_it(G):
    """NaN in a sibling's keys and values, and in one that all see."""
    import torch
    n0, nq, R = 170, 32, 4
    lens, pars = [n0 + nq], trees([nq], 40)
    cache, ref, table, slots = build(1, 128, G, 16, lens, "bf16", 40)
    table = roomy(table, 1, 16, nq * R)
    q = draw((nq, R, 128), "bf16", 72)
    good, _ = call(cache, q, table, lens, pars)
    for key in (n0 + 1, 75):
        seen = spec.sees(pars[0], lens[0], 0)[:, key]
        assert seen.any()
        for side in (0, 1):
            x = torch.zeros((2, 1, 1, 128), dtype=torch.bfloat16, device="cuda")
            x[side, 0, 0, 100] = math.nan
            kvc.kv4_append(cache, x[0], x[1], torch.from_numpy(slots[0][key:key + 1]).cuda())
            assert status(cache) == kvc.KVC_DEV_NONFINITE
            out, lse = call(cache, q, table, lens, pars)
            nan = torch.isnan(out).any(-1).any(-1).cpu().numpy()
            assert np.array_equal(nan, seen)
            assert torch.equal(out[torch.from_numpy(~seen).cuda()], good[torch.from_numpy(~seen).cuda()])
            if side:  # V's: the groups of that channel alone
                only = torch.isnan(out).any(0).any(0).cpu().numpy()
                assert np.array_equal(only, np.arange(128) // G == 100 // G)
    assert status(cache) == 0


def test_bad_parents_and_pages_are_flagged():
    import torch
    lens, nqs = [200, 200], [32, 32]
    cache, ref, table, slots = build(2, 128, 32, 16, lens, "bf16", 41)
    table = roomy(table, 2, 16, 128)
    q = draw((64, 8, 128), "bf16", 73)
    pars = trees(nqs, 41)
    good, lse = call(cache, q, table, lens, pars)
    assert status(cache) == 0
    for at, entry in ((3, 3), (5, -7), (31, 2 ** 31 - 1), (0, 65535)):
        worse = list(pars[1])
        worse[at] = entry
        out, _ = call(cache, q, table, lens, [pars[0], worse])
        assert status(cache) == kvc.KVC_DEV_BAD_INDEX and torch.equal(out[:32], good[:32])
        worse[at] = -1
        mended, _ = call(cache, q, table, lens, [pars[0], worse])
        assert status(cache) == 0 and torch.equal(out, mended)
    for entry in (-1, cache.n_pages, 2 ** 31 - 1):
        t = table.copy()
        t[1, 2] = entry
        out, _ = call(cache, q, t, lens, pars)
        assert status(cache) == kvc.KVC_DEV_BAD_INDEX and torch.equal(out[:32], good[:32])


def test_strides_and_rows_of_no_sequence():
    import torch
    lens, pars, R, H, D = [400, 40], trees([32, 5], 42), 4, 2, 128
    cache, ref, table, slots = build(H, D, 64, 16, lens, "f16", 42)
    table = roomy(table, H, 16, 128)
    n_q = 41  # two before the first sequence's, two behind the last's
    big = torch.full((n_q, 3, H * R, D + 1), 7.0, dtype=torch.float16, device="cuda")
    q = draw((n_q, H * R, D), "f16", 74)
    qd = torch.zeros((n_q, H * R + 1, D + 1), dtype=torch.float16, device="cuda")[:, 1:, 1:]
    qd.copy_(q)
    lse = torch.full((n_q, H * R), 5.0, dtype=torch.float32, device="cuda")
    kvc.kv4_tree_attention(cache, qd, torch.from_numpy(table).cuda(), ints(lens), ints([99, 99] + pars[0] + pars[1] + [99, 99]),
                           cu_q=ints([2, 34, 39]), max_q=32, out=big[:, 1, :, 1:], lse=lse)
    assert status(cache) == 0
    compare(big[2:39, 1, :, 1:], lse[2:39], q[2:39], ref, slots, lens, pars, R, "f16", 0, 0.0, D ** -0.5)
    assert (big[:, 0] == 7.0).all() and (big[:, 2] == 7.0).all() and (big[:, 1, :, 0] == 7.0).all()
    for t in (big, lse):
        rest = t[[0, 1, 39, 40]]
        assert (rest == rest.flatten()[0]).all()


def test_repeats_give_the_same():
    import torch
    lens, nqs = [9001, 20, 333], [32, 20, 7]
    cache, ref, table, slots = build(2, 128, 64, 16, lens, "bf16", 43)
    table, pars, q = roomy(table, 2, 16, 128), trees(nqs, 43), draw((59, 8, 128), "bf16", 75)
    want, wl = call(cache, q, table, lens, pars)
    for _ in range(3):
        out, lse = call(cache, q, table, lens, pars)
        assert torch.equal(out, want) and torch.equal(lse, wl)
    assert status(cache) == 0


@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_tiny_and_huge_values(dt):
    """V's terms are scaled by 16 keys' largest value: of one size, and of very different ones side by side."""
    import torch
    H, D, G, P, T, n = 1, 128, 64, 16, 200, 32
    pars = trees([n], 44)
    for kmul, vmul, qmul, uneven in ((1.0, 1e-3, 1.0, 0), (1.0, 6000.0, 1.0, 0), (1000.0, 1.0, 1e-4, 0), (1e-3, 1.0, 3e4, 0), (1.0, 30.0, 1.0, 1)):
        cache, ref = fresh(H, D, G, P, 14)
        k, v = draw((T, H, D), dt, 95, kmul), draw((T, H, D), dt, 96, vmul)
        if uneven:
            v[::3] /= 4096
        slots = np.arange(T)
        kvc.kv4_append(cache, k.cuda(), v.cuda(), torch.from_numpy(slots).cuda())
        ref.write(f32(k), f32(v), slots)
        q = (draw((n, 4, D), dt, 97).float() * qmul).clamp(-6e4, 6e4).to(tdt(dt))
        out, lse = call(cache, q, roomy(np.arange(13, dtype=np.int32)[None], H, P, 128), [T], pars)
        assert status(cache) == 0
        compare(out, lse, q, ref, [slots], [T], pars, 4, dt, 0, 0.0, D ** -0.5)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_sums_over_many_keys_keep_every_key(dt):
    """bf16's p in one term: 6000 roundings of 2^-11 at most, to either side, of shares sum_j p_j^2 <= 1/1000 of which moves an
    output by some 2^-12 * 0.5 / sqrt(1000) = 2^-18, well below what kv4_close allows in the mean."""
    import kv4_close
    import kv4_ref
    import torch
    H, D, G, P, R, T, n = 2, 128, 64, 64, 4, 6000, 32
    pages = -(-T // P)
    cache, ref = kvc.Kv4Cache(H, D, pages, page_tokens=P, group=G), kv4_ref.Pool(H, D, G, P, pages)
    k, v, q = kv4_close.inputs((T, H, D), (n, H * R, D), dt, 60)
    slots = np.arange(T)
    kvc.kv4_append(cache, k.cuda(), v.cuda(), torch.from_numpy(slots).cuda())
    ref.write(f32(k), f32(v), slots)
    pars = trees([n], 45)
    out, lse = call(cache, q, roomy(np.arange(pages, dtype=np.int32)[None], H, P, n * R), [T], pars)
    assert status(cache) == 0
    ok = spec.sees(pars[0], T, 0)
    for h in range(H):
        hs = slice(h * R, (h + 1) * R)
        wo, wl = spec.attention(q[:, hs].double().numpy(), ref.value(0, slots)[:, h], ref.value(1, slots)[:, h], ok, 0.0, D ** -0.5)
        assert kv4_close.lse_off(lse[:, hs].double().cpu().numpy(), wl) <= 1.0
        assert kv4_close.out_off(out[:, hs].double().cpu().numpy(), wo, dt) <= 1.0


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("D,G", [(128, 64), (256, 32)])
def test_outlying_channels(D, G, dt):
    outlying(2, D, G, 16, 4, 70, 32, dt, lambda t: roomy(t, 2, 16, 128))


def test_captured_and_on_two_streams():
    """Replays follow what lengths, queries and parents hold then; calls on two streams at once keep to their own."""
    import torch
    lens, nqs, H, R = [700, 45], [32, 20], 2, 4
    cache, ref, table, slots = build(H, 128, 64, 16, lens, "bf16", 45)
    pars = [trees(nqs, 45 + i) for i in range(3)]
    qs = [draw((52, H * R, 128), "bf16", 76 + i) for i in range(3)]
    want = [call(cache, q, roomy(table, H, 16, 128), lens, p) for q, p in zip(qs, pars)]
    tab, ln, cu = torch.from_numpy(roomy(table, H, 16, 128)).cuda(), ints(lens), ints([0, 32, 52])
    q, par = qs[0].cuda(), ints(sum(pars[0], []))
    nb = kvc.kv4_tree_work_bytes(cache, 52, H * R, 2, tab.shape[1], 32)
    out, lse = torch.empty_like(q), torch.empty((52, H * R), dtype=torch.float32, device="cuda")
    work = torch.empty(nb, dtype=torch.uint8, device="cuda")
    run = lambda: kvc.kv4_tree_attention(cache, q, tab, ln, par, cu_q=cu, max_q=32, out=out, lse=lse, work=work)
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for i in (1, 2, 0, 1):
        q.copy_(qs[i])
        par.copy_(ints(sum(pars[i], [])))
        out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[i][0]) and torch.equal(lse, want[i][1])
        again, _ = call(cache, qs[i], roomy(table, H, 16, 128), lens, pars[i])
        assert torch.equal(again, want[i][0])
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    dev = [(a.cuda(), ints(sum(p, []))) for a, p in zip(qs, pars)]
    torch.cuda.synchronize()
    for i, s in enumerate(streams * 3):
        a, p = dev[i % 2]
        got.append(kvc.kv4_tree_attention(cache, a, tab, ln, p, cu_q=cu, max_q=32, return_lse=True, stream=s))
    torch.cuda.synchronize()
    for i, (o, l) in enumerate(got):
        assert torch.equal(o, want[i % 2][0]) and torch.equal(l, want[i % 2][1])
    assert status(cache) == 0


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("D,R,nq", [(128, 4, 17), (128, 3, 32), (256, 2, 33)])
def test_groups_of_32_fill_fewer(D, R, nq, dt):
    """With groups of 32 three of four waves with rows are enough, the last of them part of one."""
    lens, nqs, H = [300, 77, 500], [nq, 3, 9], 2
    cache, ref, table, slots = build(H, D, 32, 16, lens, dt, 46)
    check(cache, ref, roomy(table, H, 16, 128), slots, lens, trees(nqs, 46), R, dt)
