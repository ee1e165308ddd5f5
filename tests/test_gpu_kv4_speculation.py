"""Speculative decoding as a serving loop does it: drafted trees written, attended and kept, step after step, eagerly and in
a captured graph, against the same steps in 64 bits."""
import numpy as np
import pytest

import entropy_coding_02_amd as kvc
import kv4_ref
import kv4_spec_ref as spec
from gpu_util import say
from test_gpu_kv4 import build, draw, f32, fresh, same_pool, status
from test_gpu_kv4_tree import compare, ints

pytestmark = pytest.mark.gpu

H, R, D, G, P, B, N, L = 2, 4, 128, 64, 16, 3, 12, 2  # N drafted tokens a sequence, L layers


class Loop:
    """The device side: fixed buffers, one step."""

    def __init__(self, lens, steps):
        import torch
        room = [l + (steps + 1) * N for l in lens]
        self.pages = -(-max(room) // P)
        n_pages = B * self.pages
        self.table = np.random.default_rng(5).permutation(n_pages).astype(np.int32).reshape(B, self.pages)
        self.caches, self.refs = zip(*(fresh(H, D, G, P, n_pages) for _ in range(L)))
        self.tab = torch.from_numpy(self.table).cuda()
        self.rope = spec.table(4096, D)
        self.rope_d = torch.from_numpy(self.rope).cuda()
        f = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        self.k, self.v, self.q, self.qt, self.out = f(L, B * N, H, D), f(L, B * N, H, D), f(L, B * N, H * R, D), f(L, B * N, H * R, D), f(L, B * N, H * R, D)
        self.lse = torch.zeros((L, B * N, H * R), dtype=torch.float32, device="cuda")
        self.slots = torch.full((B * N,), -1, dtype=torch.int64, device="cuda")
        self.positions = torch.full((B * N,), -1, dtype=torch.int64, device="cuda")
        self.base, self.kv_len, self.n_keep = ints([0] * B), ints([0] * B), ints([0] * B)
        self.parents, self.path = ints([-1] * (B * N)), ints([[-1] * N] * B)
        nb = kvc.kv4_tree_work_bytes(self.caches[0], B * N, H * R, B, self.pages, N)
        self.work = torch.empty(max(nb, 16), dtype=torch.uint8, device="cuda")

    def slots_of(self, b, n):
        t = np.arange(n)
        return self.table[b, t // P].astype(np.int64) * P + t % P

    def draft(self):
        for i, cache in enumerate(self.caches):
            kvc.kv4_append_rotated(cache, self.k[i], self.v[i], self.slots, self.positions, self.rope_d, q=self.q[i], q_out=self.qt[i])
            kvc.kv4_tree_attention(cache, self.qt[i], self.tab, self.kv_len, self.parents, out=self.out[i], lse=self.lse[i], work=self.work)

    def accept(self):
        kvc.kv4_keep(self.caches, self.tab, self.base, self.path, self.n_keep)


def captured(f):
    import torch
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        f()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        f()
    return g.replay


@pytest.mark.parametrize("graph", [False, True])
def test_steps(graph):
    import torch
    say(f"[gpu] kv4 speculation graph={graph}")
    steps, lens = 5, [100, 0, 37]
    loop = Loop(lens, steps)
    rng = np.random.default_rng(17)
    # the prompts, rotated by their positions
    for i, (cache, ref) in enumerate(zip(loop.caches, loop.refs)):
        pos = np.concatenate([np.arange(l) for l in lens])
        at = np.concatenate([loop.slots_of(b, l) for b, l in enumerate(lens)])
        k, v = draw((len(pos), H, D), "bf16", 200 + i), draw((len(pos), H, D), "bf16", 210 + i)
        kvc.kv4_append_rotated(cache, k.cuda(), v.cuda(), torch.from_numpy(at).cuda(), torch.from_numpy(pos).cuda(), loop.rope_d)
        ref.write(spec.rotate(f32(k), loop.rope, pos, False), f32(v), at)
    draft, accept = (captured(loop.draft), captured(loop.accept)) if graph else (loop.draft, loop.accept)
    base = list(lens)
    for step in range(steps):
        pars = [spec.random_tree(N, rng, ("bushy", "chain", "flat", "bushy", "bushy")[step]) for _ in range(B)]
        way = [[spec.path(p, i) for i in range(N)] for p in pars]
        slots = [loop.slots_of(b, base[b] + N) for b in range(B)]
        at = np.concatenate([s[-N:] for s in slots])
        pos = np.concatenate([[base[b] + len(w) - 1 for w in way[b]] for b in range(B)])
        loop.slots.copy_(torch.from_numpy(at)), loop.positions.copy_(torch.from_numpy(pos))
        loop.base.copy_(torch.tensor(base)), loop.kv_len.copy_(torch.tensor(base) + N)
        loop.parents.copy_(torch.tensor(sum(pars, [])))
        kvq = [[draw((B * N, n, D), "bf16", 1000 * step + 10 * i + j) for j, n in enumerate((H, H, H * R))] for i in range(L)]
        for i, (k, v, q) in enumerate(kvq):
            loop.k[i].copy_(k), loop.v[i].copy_(v), loop.q[i].copy_(q)
        torch.cuda.synchronize()
        draft()
        torch.cuda.synchronize()
        for i, (k, v, q) in enumerate(kvq):
            ref = loop.refs[i]
            ref.write(spec.rotate(f32(k), loop.rope, pos, False), f32(v), at)
            qt = torch.from_numpy(spec.rotate(f32(q), loop.rope, pos, False)).to(torch.bfloat16)
            assert torch.equal(loop.qt[i].cpu(), qt)
            now = [b + N for b in base]
            compare(loop.out[i], loop.lse[i], qt, ref, slots, now, pars, R, "bf16", 0, 0.0, D ** -0.5)
        kept = [w[int(rng.integers(N))] for w in way]
        kept[step % B] = kept[step % B] if step % 2 else []  # a sequence that accepts nothing
        loop.path.copy_(torch.tensor([p + [-1] * (N - len(p)) for p in kept]))
        loop.n_keep.copy_(torch.tensor([len(p) for p in kept]))
        torch.cuda.synchronize()
        accept()
        torch.cuda.synchronize()
        for ref, cache in zip(loop.refs, loop.caches):
            for b in range(B):
                spec.keep(ref, slots[b], base[b], kept[b])
            same_pool(cache, ref)
            assert status(cache) == 0
        base = [b + len(p) for b, p in zip(base, kept)]
    assert max(base) > 100


def test_pool_past_32_bits():
    """Slots whose bytes lie past 2^32: written, attended, kept."""
    import torch
    h, p = 8, 64
    n = (1 << 32) // (2 * h * p * D // 2) + 40
    cache = kvc.Kv4Cache(h, D, n, page_tokens=p)
    assert cache.codes.numel() > 1 << 32
    T, nq = 150, 20
    pages = np.array([n - 1, n - 17, 3], np.int32)
    t = np.arange(T)
    slots, pos = pages[t // p].astype(np.int64) * p + t % p, t.copy()
    k, v, q = draw((T, h, D), "bf16", 61), draw((T, h, D), "bf16", 62), draw((nq, 2 * h, D), "bf16", 63)
    rope = spec.table(200, D)
    kvc.kv4_append_rotated(cache, k.cuda(), v.cuda(), torch.from_numpy(slots).cuda(), torch.from_numpy(pos).cuda(), torch.from_numpy(rope).cuda())
    small, near = kv4_ref.Pool(h, D, 64, p, 3), np.arange(T)
    small.write(spec.rotate(f32(k), rope, pos, False), f32(v), near)
    par = [spec.random_tree(nq, np.random.default_rng(1))]
    tab = torch.from_numpy(pages[None]).cuda()
    out, lse = kvc.kv4_tree_attention(cache, q.cuda(), tab, ints([T]), ints(par[0]), return_lse=True)
    compare(out, lse, q, small, [near], [T], par, 2, "bf16", 0, 0.0, D ** -0.5)
    way = [2, 3, 7, 15]
    kvc.kv4_keep(cache, tab, ints([T - nq]), ints([way]), ints([4]))
    spec.keep(small, near, T - nq, way)
    got = kvc.kv4_read(cache, torch.from_numpy(slots).cuda(), dtype=torch.float32)
    for kv in (0, 1):
        assert np.array_equal(got[kv].cpu().numpy(), small.value(kv, near).astype(np.float32))
    assert status(cache) == 0
