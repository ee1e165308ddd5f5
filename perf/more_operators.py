"""Measured cases of speculative serving from the paged 4-bit KV cache: drafted tokens written with the rotation of their
positions, attention for a tree of them over the cache, and the accepted path kept.

Rotation.  Token t at position p turns the first `rot` channels of each head of k and q by the angles p base^(-2i/rot),
i = 0 .. rot/2 - 1; `table` [positions][rot] fp32 holds their cosines, then their sines.  Pair i is channels (i, i + rot/2),
or (2i, 2i + 1) where interleaved:  a' = a cos - b sin,  b' = b cos + a sin,  fp32, every operation rounded on its own.  k' is
quantised as it is, v as it came, q' is rounded to its type.

Cache format.  A row is the D channels of one (token, K or V, kv head), cut into groups of G channels.  Per group, in
fp32, every operation rounded on its own, x clamped to +-65504:

    lo = fp16(min x),  s = fp16((max x - min x) * fp32(1/15)),  inv = 1 / s (0 where s is 0),
    code = clamp(round_half_even((x - lo) * inv), 0, 15),  the code stands for  lo + code * s.

Codes live in pages of P tokens, uint8 [n_pages][2][H][P*D/2], K and V halves ordered for the attention that reads them
(pack_k, pack_v); (s, lo) pairs live in fp16 [n_pages][2][H][D/G][P][2].  Slot = page * P + token in page.

Tree attention.  A sequence's last n cached keys are n drafted tokens, n queries stand at them; parents[i] < i is the
drafted token that i follows, -1: the last one before the tree.  Query i sees the keys before the tree and, of the
drafted ones, itself and its ancestors; with a window only keys less than `window` steps of its own path back.

Keeping.  After verification token path[i] of a sequence's tree becomes its i-th token past the base, path rising.
"""
import math

import numpy as np
import torch

own = False


# ------------------------------------------------------------------ the cases

def listed():
    bf, hf = "bf16", "f16"
    return [
        # one new token for each of 64 running sequences, 8 kv heads of 128 channels under 32 query heads: pure latency
        dict(name="rotate_step", kind="rotate", tokens=64, H=8, R=4, D=128, G=64, P=64, rot=128, interleaved=False,
             dtype=bf, scattered=True),
        # an odd piece of a small-head model that turns half of its channels, in neighbouring pairs
        dict(name="rotate_odd", kind="rotate", tokens=1001, H=5, R=3, D=64, G=32, P=16, rot=32, interleaved=True,
             dtype=hf, scattered=False),
        # one layer's q, K and V of a 32K prompt (the 70B-class shape, 1024 channels of K and V)
        dict(name="rotate_prompt", kind="rotate", tokens=32768, H=8, R=4, D=128, G=64, P=64, rot=128, interleaved=False,
             dtype=hf, scattered=False),
        # one user, a small tree after a short prompt
        dict(name="tree_short", kind="tree", B=1, nq=8, chain=False, kv=300, ragged=False, H=8, R=4, D=128, G=64, P=64,
             window=0, softcap=0.0, dtype=bf),
        # a serving batch, every sequence with its own tree of up to 24 tokens at its own length up to 8192
        dict(name="tree_batch", kind="tree", B=16, nq=24, chain=False, kv=8192, ragged=True, H=8, R=4, D=128, G=64, P=64,
             window=0, softcap=0.0, dtype=bf),
        # sliding-window heads of 64 channels with fine groups and capped logits, odd batch and ratio
        dict(name="tree_window", kind="tree", B=33, nq=13, chain=False, kv=6001, ragged=True, H=4, R=7, D=64, G=32, P=16,
             window=2047, softcap=30.0, dtype=hf),
        # the widest trees, 64 tokens under 64 query heads, fp16: the most arithmetic of a batch
        dict(name="tree_wide", kind="tree", B=4, nq=64, chain=False, kv=16000, ragged=True, H=8, R=8, D=128, G=64, P=64,
             window=0, softcap=0.0, dtype=hf),
        # one user with an 80,000-token context (the 34B-class shape) and a tree of 60
        dict(name="tree_long", kind="tree", B=1, nq=60, chain=False, kv=80000, ragged=False, H=8, R=8, D=128, G=64, P=64,
             window=0, softcap=0.0, dtype=bf),
        # eight sequences' accepted paths kept in one layer: pure latency
        dict(name="keep_one", kind="keep", B=8, L=1, nodes=32, keep=6, H=8, D=128, G=64, P=64),
        # sixteen sequences' accepted paths kept in all 80 layers
        dict(name="keep_layers", kind="keep", B=16, L=80, nodes=32, keep=8, H=8, D=128, G=64, P=64),
        # a chain of 4 drafted tokens each, written, attended and kept
        dict(name="step_chain", kind="step", B=32, nq=4, chain=True, kv=4096, ragged=True, H=8, R=4, D=128, G=64, P=64,
             window=0, softcap=0.0, rot=128, interleaved=False, dtype=bf),
        # a verification step as a serving loop makes it with trees of up to 32 tokens
        dict(name="step_tree", kind="step", B=8, nq=32, chain=False, kv=16384, ragged=True, H=8, R=8, D=128, G=64, P=64,
             window=0, softcap=0.0, rot=128, interleaved=False, dtype=bf),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    D = rng.choice([64, 128, 128, 256])
    G = rng.choice([g for g in (32, 64, 128) if g <= D])
    H, P, R = rng.randint(1, 8), rng.choice([16, 32, 64, 128]), rng.choice([1, 2, 3, 4, 5, 7, 8])
    base = dict(H=H, D=D, G=G, P=P)
    turn = dict(rot=rng.choice([D, D, D // 2, 16 * rng.randint(1, D // 16)]), interleaved=rng.random() < 0.3)
    kind = rng.choice(["rotate", "rotate", "tree", "tree", "tree", "keep", "step"])
    if kind == "keep":
        keep = rng.randint(1, 10)
        return dict(kind="keep", B=_log(rng, 1, 16), L=_log(rng, 1, 64), nodes=rng.randint(2 * keep, 64), keep=keep, **base)
    if kind == "rotate":
        T, dtype = _log(rng, 1, 24000), rng.choice(["bf16", "f16", "f32"])
        return dict(kind="rotate", tokens=T // 2 + 1 if dtype == "f32" else T, R=min(R, 4), dtype=dtype,
                    scattered=T <= 512 and rng.random() < 0.5, **turn, **base)
    nq, B = _log(rng, 1, 96), _log(rng, 1, 32)
    most = 1 << 36  # of q rows * keys * channels: below the largest listed case
    kv = _log(rng, nq, max(nq, min(65536, 262144 // B, most // (B * nq * H * R * D))))
    d = dict(kind=kind, B=B, nq=nq, chain=rng.random() < 0.2, kv=kv, ragged=rng.random() < 0.7, R=R,
             window=rng.choice([0, 0, 0, _log(rng, 1, 4096)]), softcap=rng.choice([0.0, 0.0, 30.0, 50.0]),
             dtype=rng.choice(["bf16", "f16"]), **base)
    return dict(d, **turn) if kind == "step" else d


# --------------------------------------------------- the format, in elementary operations

def group_quantise(x, G):
    """x [..., D] -> codes uint8 [..., D], scale and lo fp16 [..., D/G]."""
    g = x.float().clamp(-65504.0, 65504.0).unflatten(-1, (-1, G))
    mn, mx = g.amin(-1), g.amax(-1)
    lo = mn.half()
    s = ((mx - mn) * (1.0 / 15.0)).half()  # the constant rounds to fp32 in an fp32 product
    s32 = s.float()
    inv = torch.where(s32 > 0, (1.0 / s32.double()).float(), torch.zeros_like(s32))
    c = torch.round((g - lo.float().unsqueeze(-1)) * inv.unsqueeze(-1)).clamp(0.0, 15.0)
    return c.to(torch.uint8).flatten(-2), s, lo


def pack_k(c):
    """codes [..., D] -> bytes [..., D/2]: dword (h, t) of a row holds channels 32t + 8h .. + 7, low nibble first."""
    b = c[..., 0::2] | (c[..., 1::2] << 4)
    return b.unflatten(-1, (-1, 4, 4)).transpose(-3, -2).flatten(-3)


def pack_v(c):
    """codes [..., D] -> bytes [..., 16, D/64, 2]: two-byte piece (n, u) holds channels 64u + 16i + n, i = 0 .. 3."""
    c = c.unflatten(-1, (-1, 4, 16)).movedim(-1, -3)
    return c[..., 0::2] | (c[..., 1::2] << 4)


def views(codes, c):
    """The K view [..., pages, H, P, D/2] and the V view [..., pages, H, P/4, 16, D/64, 4, 2] of a code pool: four tokens'
    pieces lie side by side."""
    H, P, D = c["H"], c["P"], c["D"]
    k, v = codes.unbind(-3)
    return k.unflatten(-1, (P, D // 2)), v.unflatten(-1, (P // 4, 16, D // 64, 4, 2))


def write_plain(codes, params, c, k, v, slots):
    page, off = slots // c["P"], slots % c["P"]
    kc, ks, kl = group_quantise(k, c["G"])
    vc, vs, vl = group_quantise(v, c["G"])
    K, V = views(codes, c)
    K[page, :, off] = pack_k(kc)
    V[page, :, off // 4, :, :, off % 4] = pack_v(vc)
    params[page, 0, :, :, off] = torch.stack([ks, kl], -1)
    params[page, 1, :, :, off] = torch.stack([vs, vl], -1)


def nibbles(b):
    """bytes [..., n] -> codes [..., 2n], low nibble first."""
    return torch.stack([b & 15, b >> 4], -1).flatten(-2)


def values(code, p, G):
    """codes [..., D], (s, lo) [..., D/G, 2] -> fp32 values."""
    p = p.float()
    return (code.float().unflatten(-1, (-1, G)) * p[..., 0:1] + p[..., 1:2]).flatten(-2)


def read_plain(codes, params, c, slots):
    page, off = slots // c["P"], slots % c["P"]
    K, V = views(codes, c)
    kb = K[page, :, off].unflatten(-1, (4, -1, 4)).transpose(-3, -2).flatten(-3)
    vn = nibbles(V[page, :, off // 4, :, :, off % 4]).movedim(-3, -1).flatten(-3)
    return (values(nibbles(kb), params[page, 0, :, :, off], c["G"]),
            values(vn, params[page, 1, :, :, off], c["G"]))


def rounded(x, dtype):
    """A value can pass its group's largest by the scale's rounding: what fp16 holds is clamped."""
    return (x.clamp(-65504.0, 65504.0) if dtype == torch.float16 else x).to(dtype)


# ------------------------------------------------------- the operators, plain

def rotate_plain(x, table, positions, c):
    """x [T][heads][D] turned, fp32."""
    r = c["rot"]
    cs = table[positions].unsqueeze(1)
    cos, sin = cs[..., :r // 2], cs[..., r // 2:]
    x = x.float()
    a, b = (x[..., 0:r:2], x[..., 1:r:2]) if c["interleaved"] else (x[..., :r // 2], x[..., r // 2:r])
    a, b = a * cos - b * sin, b * cos + a * sin
    return torch.cat([torch.stack([a, b], -1).flatten(-2) if c["interleaved"] else torch.cat([a, b], -1), x[..., r:]], -1)


def sees_plain(parents, cu, nq, window):
    """[B][nq][nq]: whether query i sees drafted token j, and each one's depth [B][nq]."""
    B = cu.numel() - 1
    i = torch.arange(nq, device=cu.device)
    real = i < (cu[1:] - cu[:-1]).unsqueeze(1)
    par = torch.where(real, parents.long()[torch.where(real, cu[:-1].unsqueeze(1) + i, 0)], -1)
    up = (par.unsqueeze(-1) == i).float() + torch.eye(nq, device=cu.device)
    for _ in range(max(1, nq - 1).bit_length()):  # one step up, two, four, ...
        up = (torch.matmul(up, up) > 0).float()
    depth = up.sum(-1) - 1.0
    sees = up > 0
    if window > 0:
        sees = sees & (depth.unsqueeze(-1) - depth.unsqueeze(1) < window)
    return sees & real.unsqueeze(-1), depth.view(B, nq)


def attend_plain(s, q):
    c = s["case"]
    table, lens, cu = s["pages"], s["lens"].long(), s["cu"].long()
    B, H, R, D, P, nq = table.shape[0], c["H"], c["R"], c["D"], c["P"], s["max_q"]
    T = table.shape[1] * P
    slots = (table.long().unsqueeze(-1) * P + torch.arange(P, device=q.device)).flatten()
    k, v = read_plain(s["codes"], s["params"], c, slots)  # [B*T][H][D]
    k, v = (t.view(B, T, H, D).transpose(1, 2).contiguous() for t in (k, v))
    n = cu[1:] - cu[:-1]
    i = torch.arange(nq, device=q.device)
    real = i < n.unsqueeze(1)  # [B][nq]
    idx = torch.where(real, cu[:-1].unsqueeze(1) + i, 0)
    qp = q.float()[idx].view(B, nq, H, R, D).permute(0, 2, 3, 1, 4).reshape(B, H, R * nq, D)
    x = torch.matmul(qp, k.transpose(-1, -2).contiguous()) * s["scale"]
    if c["softcap"] > 0:
        x = c["softcap"] * torch.tanh(x / c["softcap"])
    sees, depth = sees_plain(s["parents"], cu, nq, c["window"])
    j = torch.arange(T, device=q.device)
    base = lens - n
    ok = (j < base.unsqueeze(1)).unsqueeze(1) & real.unsqueeze(-1)  # [B][nq][T]
    if c["window"] > 0:
        ok = ok & (j > ((base.unsqueeze(1) + depth).unsqueeze(-1) - c["window"]))
    at = j - base.unsqueeze(1)  # [B][T]: which drafted token a key is
    inside = (at >= 0) & (at < n.unsqueeze(1))
    ok = ok | (inside.unsqueeze(1) & sees.gather(2, at.clamp(0, nq - 1).unsqueeze(1).expand(B, nq, T)))
    x = x.view(B, H, R, nq, T).masked_fill_(~ok.view(B, 1, 1, nq, T), -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    e = x.sub_(m).exp_()
    l = e.sum(-1, keepdim=True)
    o = torch.matmul(e.view(B, H, R * nq, T), v).view(B, H, R, nq, D) / torch.where(l > 0, l, torch.ones_like(l))
    lse = (m + l.log()).squeeze(-1)
    o = o.permute(0, 3, 1, 2, 4).reshape(B, nq, H * R, D)[real]
    return o.to(q.dtype), lse.permute(0, 3, 1, 2).reshape(B, nq, H * R)[real]


def keep_plain(codes, params, c, s):
    """codes [..., n_pages, 2, H, P*D/2] and params, of one layer or several: token base + path[i] moves to base + i."""
    path, base, P = s["path"].long(), s["base"].long().unsqueeze(1), c["P"]
    i = torch.arange(path.shape[1], device=path.device)
    real = i < s["n_keep"].unsqueeze(1)
    b = torch.arange(path.shape[0], device=path.device).unsqueeze(1).expand_as(path)[real]
    to, of = (base + i)[real], (base + path)[real]
    tp, to, fp, of = s["pages"][b, to // P].long(), to % P, s["pages"][b, of // P].long(), of % P
    K, V = views(codes, c)
    K[..., tp, :, to, :] = K[..., fp, :, of, :]  # indexing copies before anything is written
    V[..., tp, :, to // 4, :, :, to % 4, :] = V[..., fp, :, of // 4, :, :, of % 4, :]
    params[..., tp, :, :, :, to, :] = params[..., fp, :, :, :, of, :]


# --------------------------------------------------------------- inputs

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
POSITIONS = 1 << 17


def make_kv(shape, dtype, g, is_key):
    """K has a few channels that are large in every token, V is centred: what caches look like."""
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)
    H, D = shape[-2:]
    if is_key:
        mean = torch.randn((H, D), generator=g, device="cuda") * 0.5
        big = torch.rand((H, D), generator=g, device="cuda") < 0.03
        x = x.add_(torch.where(big, mean * 12.0, mean))
    return x.to(dtype)


def make_pool(c, n_pages, g, dtype):
    """A code pool and its parameters, every token of it quantised from drawn K and V."""
    H, D, P = c["H"], c["D"], c["P"]
    codes = torch.empty((n_pages, 2, H, P * D // 2), dtype=torch.uint8, device="cuda")
    params = torch.empty((n_pages, 2, H, D // c["G"], P, 2), dtype=torch.float16, device="cuda")
    piece = max(1, (1 << 26) // (P * H * D))  # pages at a time: bounded temporaries
    for a in range(0, n_pages, piece):
        b = min(n_pages, a + piece)
        slots = torch.arange(a * P, b * P, device="cuda")
        shape = (slots.numel(), H, D)
        write_plain(codes, params, c, make_kv(shape, dtype, g, True), make_kv(shape, dtype, g, False), slots)
    return codes, params


def make_table(rot, count):
    """Cosines and sines of the positions' angles, computed in 64 bits."""
    i = torch.arange(rot // 2, device="cuda", dtype=torch.float64)
    angle = torch.arange(count, device="cuda", dtype=torch.float64).unsqueeze(1) * 10000.0 ** (-2.0 * i / rot)
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def sizes(c):
    """Drafted tokens of each sequence: by the case, so that outputs keep their shapes."""
    if not c["ragged"]:
        return [c["nq"]] * c["B"]
    n = np.random.default_rng(c["B"] + c["nq"]).integers(max(1, c["nq"] // 2), c["nq"] + 1, c["B"])
    return [int(x) for x in n]


def lengths(c, seed):
    """Keys a sequence holds, its drafted ones among them."""
    if not c["ragged"]:
        return [c["kv"]] * c["B"]
    r, kv = np.random.default_rng(1000 + seed), c["kv"]
    lens = [max(int(x), m) for x, m in zip(r.integers(max(1, kv // 4), kv + 1, c["B"]), sizes(c))]
    lens[int(r.integers(c["B"]))] = kv
    return lens


def trees(c, seed):
    """Each sequence's parents: a chain, or a tree of the kind that keeps the likeliest continuations of every step."""
    r = np.random.default_rng(2000 + seed)
    if c["chain"]:
        return [list(range(-1, n - 1)) for n in sizes(c)]
    return [[int(r.integers(max(-1, i // 4 - 2), max(0, i // 2))) for i in range(n)] for n in sizes(c)]


def path_to(parents, i):
    """The drafted tokens from the tree's first level to i."""
    return (path_to(parents, parents[i]) if parents[i] >= 0 else []) + [i]


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = np.random.default_rng(3000 + seed)
    H, D, P = c["H"], c["D"], c["P"]
    s = {"case": c}
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    if c["kind"] == "rotate":
        T, dtype = c["tokens"], DT[c["dtype"]]
        n_pages = T if c["scattered"] else -(-T // P)
        s["codes"] = torch.zeros((n_pages, 2, H, P * D // 2), dtype=torch.uint8, device="cuda")
        s["params"] = torch.zeros((n_pages, 2, H, D // c["G"], P, 2), dtype=torch.float16, device="cuda")
        pages, t = torch.randperm(n_pages, generator=g, device="cuda"), torch.arange(T, device="cuda")
        if c["scattered"]:  # each token ends another sequence's last page, at its own position
            s["slots"] = pages[t] * P + torch.randint(0, P, (T,), generator=g, device="cuda")
            s["positions"] = torch.randint(0, POSITIONS, (T,), generator=g, device="cuda")
        else:  # a piece of a long prompt
            s["slots"] = pages[t // P] * P + t % P
            s["positions"] = int(r.integers(0, POSITIONS - T)) + t
    elif c["kind"] == "keep":
        # a wide first level, of which the likeliest is accepted: what is kept is not overwritten, and a second pass does the same
        B, L, N, K = c["B"], c["L"], c["nodes"], c["keep"]
        base = r.integers(0, 2 * P, B)
        M = -(-(2 * P + N) // P)
        n_pages = B * M
        s["codes"] = torch.randint(0, 256, (L, n_pages, 2, H, P * D // 2), dtype=torch.uint8, generator=g, device="cuda")
        s["params"] = torch.randn((L, n_pages, 2, H, D // c["G"], P, 2), generator=g, device="cuda").half()
        s["pages"] = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32).view(B, M)
        path = [[0] + sorted(int(x) for x in r.choice(np.arange(K, N), K - 1, replace=False)) for _ in range(B)]
        s.update(base=ints(base), path=ints(path), n_keep=ints(r.integers(0, K + 1, B)))
    else:
        lens, n, par, dtype = lengths(c, seed), sizes(c), trees(c, seed), DT[c["dtype"]]
        B, M = c["B"], -(-max(lens) // P)
        n_pages = sum(-(-l // P) for l in lens) + 1
        s["codes"], s["params"] = make_pool(c, n_pages, g, dtype)
        order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
        s["pages"] = torch.zeros((B, M), dtype=torch.int32, device="cuda")
        a = 0
        for b, l in enumerate(lens):
            m = -(-l // P)
            s["pages"][b, :m] = order[a:a + m]
            a += m
        cu = [int(x) for x in np.concatenate([[0], np.cumsum(n)])]
        s.update(lens=ints(lens), cu=ints(cu), max_q=max(n), scale=1.0 / math.sqrt(D), parents=ints(sum(par, [])))
        if c["kind"] == "step":
            base = [l - m for l, m in zip(lens, n)]
            depth = [[len(path_to(p, i)) - 1 for i in range(len(p))] for p in par]
            at = torch.cat([b + torch.arange(m, device="cuda") for b, m in zip(base, n)])
            of = torch.repeat_interleave(torch.arange(B, device="cuda"), torch.tensor(n, device="cuda"))
            s["slots"] = s["pages"][of, at // P].long() * P + at % P
            s["positions"] = torch.tensor([b + d for b, x in zip(base, depth) for d in x], device="cuda")
            kept = [path_to(p, int(r.integers(len(p)))) for p in par]
            s.update(base=ints(base), n_keep=ints([len(x) for x in kept]),
                     path=ints([x + [-1] * (max(n) - len(x)) for x in kept]))
        else:
            s["q"] = torch.randn((cu[-1], H * c["R"], D), generator=g, device="cuda").to(dtype)
    if "slots" in s:
        T = s["slots"].numel()
        s["k"], s["v"] = make_kv((T, H, D), dtype, g, True), make_kv((T, H, D), dtype, g, False)
        s["q"] = torch.randn((T, H * c["R"], D), generator=g, device="cuda").to(dtype)
        s["table"] = make_table(c["rot"], POSITIONS)
    if own:  # the handles and the workspace that a serving program keeps
        import entropy_coding_02_amd as kvc
        pools = zip(s["codes"], s["params"]) if c["kind"] == "keep" else [(s["codes"], s["params"])]
        s["caches"] = [kvc.Kv4Cache(H, D, n_pages, page_tokens=P, group=c["G"], codes=a, params=b) for a, b in pools]
        if "parents" in s:
            s["work"] = torch.empty(kvc.kv4_tree_work_bytes(s["caches"][0], s["q"].shape[0], H * c["R"], c["B"], M, s["max_q"]),
                                    dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------- a pass

def run(state):
    s = state
    c = s["case"]
    if own:
        import entropy_coding_02_amd as kvc
        cache, q = s["caches"][0], s.get("q")
        if "slots" in s:
            q = kvc.kv4_append_rotated(cache, s["k"], s["v"], s["slots"], s["positions"], s["table"], q=q,
                                       interleaved=c["interleaved"])
        if "parents" in s:
            out = kvc.kv4_tree_attention(cache, q, s["pages"], s["lens"], s["parents"], cu_q=s["cu"], max_q=s["max_q"],
                                         window=c["window"], softcap=c["softcap"], scale=s["scale"], return_lse=True,
                                         work=s["work"])
        if "path" in s:
            kvc.kv4_keep(s["caches"], s["pages"], s["base"], s["path"], s["n_keep"])
        if c["kind"] == "keep":
            return s["codes"], s["params"]
        if c["kind"] == "tree":
            return out
        back = kvc.kv4_read(cache, s["slots"], dtype=q.dtype)
        return (q, *back) if c["kind"] == "rotate" else (*out, *back)
    if c["kind"] == "keep":
        keep_plain(s["codes"], s["params"], c, s)
        return s["codes"], s["params"]
    q = s["q"]
    if "slots" in s:
        write_plain(s["codes"], s["params"], c, rotate_plain(s["k"], s["table"], s["positions"], c), s["v"], s["slots"])
        q = rotate_plain(q, s["table"], s["positions"], c).to(q.dtype)
    if "parents" in s:
        out = attend_plain(s, q)
        if c["kind"] == "tree":
            return out
        keep_plain(s["codes"], s["params"], c, s)
    back = tuple(rounded(x, q.dtype) for x in read_plain(s["codes"], s["params"], c, s["slots"]))
    return (q, *back) if c["kind"] == "rotate" else (*out, *back)


def _rotate_work(c, tokens):
    size, row = 4 if c["dtype"] == "f32" else 2, c["D"] // 2 + 4 * (c["D"] // c["G"])
    kv, heads = 2 * tokens * c["H"], c["H"] * c["R"]
    b = kv * (c["D"] * size + row) + 2 * tokens * heads * c["D"] * size + tokens * (4 * c["rot"] + 16)
    return b, kv * c["D"] * 8 + 3 * tokens * (heads + c["H"]) * c["rot"]


def work(case):
    c = case
    H, D, G = c["H"], c["D"], c["G"]
    row = D // 2 + 4 * (D // G)  # a cached row
    if c["kind"] == "keep":
        n = c["B"] * c["keep"] // 2
        return {"bytes": 4 * n * c["L"] * H * row + 4 * n, "flops": 0}
    size = 4 if c["dtype"] == "f32" else 2
    if c["kind"] == "rotate":
        b, f = _rotate_work(c, c["tokens"])
        n = 2 * c["tokens"] * H
        return {"bytes": b + n * (row + D * size), "flops": f + 2 * n * D}
    W, Hq, lens, par = c["window"], H * c["R"], lengths(c, 0), trees(c, 0)
    keys = pairs = 0
    for l, p in zip(lens, par):
        base = l - len(p)
        steps = np.array([len(path_to(p, i)) for i in range(len(p))])  # itself and its ancestors
        first = np.maximum(0, base + steps - W) if W else np.zeros_like(steps)
        keys += len(p) + max(0, base - int(first[0]))
        pairs += int((np.maximum(0, base - first) + (np.minimum(steps, W) if W else steps)).sum())
    n = sum(sizes(c))
    b = 2 * keys * H * row + n * (Hq * (4 * D + 4) + 4) + 4 * sum(-(-l // c["P"]) for l in lens)
    f = 4 * pairs * Hq * D
    if c["kind"] == "step":
        rb, rf = _rotate_work(c, n)
        b, f = b + rb + 2 * n * H * (row + D * size) + 4 * n * H * row, f + rf
    return {"bytes": b, "flops": f}


# ------------------------------------------- the definition in 64 bits, written apart

def _r32(x):
    return x.float().double()


def _r16(x):
    return x.float().half().double()  # x holds fp32 values here: one rounding


def _decode_rows(s, page, off, kv):
    """Values [n][H][D] in float64 of the tokens (page, off), gathered code by code from the byte layout."""
    c = s["case"]
    H, D, G = c["H"], c["D"], c["G"]
    ch = torch.arange(D, device="cuda")
    if kv == 0:
        nib = ch % 2
        byte = off.view(-1, 1) * (D // 2) + 4 * ((ch % 32) // 8 * (D // 32) + ch // 32) + (ch % 8) // 2
    else:
        nib = (ch // 16) % 2
        byte = (off.view(-1, 1) // 4) * (2 * D) + (ch % 16) * (D // 8) + (ch // 64) * 8 + (off.view(-1, 1) % 4) * 2 + (ch % 64) // 32
    pool = s["codes"][:, kv]
    heads = torch.arange(H, device="cuda")
    raw = pool[page.view(-1, 1, 1), heads.view(1, H, 1), byte.view(-1, 1, D)]
    code = torch.where(nib == 0, raw & 15, raw >> 4).double()
    sc = s["params"][:, kv][page.view(-1, 1, 1), heads.view(1, H, 1), (ch // G).view(1, 1, D), off.view(-1, 1, 1)].double()
    return sc[..., 1] + code * sc[..., 0]


def _quantised(x, G):
    """The values that x [n][H][D] stands for once written: the definition's fp32 steps carried out in float64."""
    x = x.double().clamp(-65504.0, 65504.0)
    n, H, D = x.shape
    g = x.reshape(n, H, D // G, G)
    lo, hi = g.min(-1, keepdim=True).values, g.max(-1, keepdim=True).values
    s = _r16(_r32(_r32(hi - lo) * float(np.float32(1.0) / np.float32(15.0))))
    lo = _r16(lo)
    inv = torch.where(s > 0, _r32(1.0 / s), 0.0)
    code = _r32(_r32(g - lo) * inv).round().clamp(0, 15)
    return (lo + code * s).reshape(n, H, D)


def _turned(s, x, steps):
    """x rotated in float64; steps: with the definition's roundings to fp32."""
    c = s["case"]
    half, t = c["rot"] // 2, s["table"].double()[s["positions"]][:, None]
    fix = _r32 if steps else (lambda y: y)
    x, y = x.double(), x.double().clone()
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + half)
        cos, sin = t[..., i], t[..., half + i]
        y[..., a] = fix(fix(x[..., a] * cos) - fix(x[..., b] * sin))
        y[..., b] = fix(fix(x[..., b] * cos) + fix(x[..., a] * sin))
    return y


def _attended(s, q, new=None):
    """out and lse in float64; new: the drafted tokens' (k, v) as they were written."""
    c = s["case"]
    H, R, W, P = c["H"], c["R"], c["window"], c["P"]
    cu, par, outs, lses = s["cu"].tolist(), s["parents"].tolist(), [], []
    for b, l in enumerate(s["lens"].tolist()):
        t = torch.arange(l, device="cuda")
        page = s["pages"][b].long()[t // P]
        k, v = (_decode_rows(s, page, t % P, kv) for kv in (0, 1))
        n = cu[b + 1] - cu[b]
        if new is not None:
            k[l - n:], v[l - n:] = (x[cu[b]:cu[b + 1]] for x in new)
        ok = np.zeros((n, l), bool)
        for i in range(n):
            way = path_to(par[cu[b]:cu[b + 1]], i)  # its position is the last key's before the tree plus the way's length
            ok[i, max(0, l - n + len(way) - W) if W else 0:l - n] = True
            ok[i, [l - n + j for j in (way[-W:] if W else way)]] = True
        ok = torch.from_numpy(ok).cuda()
        qb = q[cu[b]:cu[b + 1]].double()
        o, e = torch.empty_like(qb), torch.empty((n, H * R), dtype=torch.float64, device="cuda")
        for h in range(H * R):
            x = (qb[:, h] @ k[:, h // R].T) * s["scale"]
            if c["softcap"] > 0:
                x = c["softcap"] * torch.tanh(x / c["softcap"])
            x = torch.where(ok, x, -math.inf)
            e[:, h] = torch.logsumexp(x, -1)
            o[:, h] = torch.exp(x - e[:, h:h + 1]) @ v[:, h // R]
        outs.append(o)
        lses.append(e)
    return torch.cat(outs), torch.cat(lses)


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["kind"] == "keep":
        # bytes are moved: a token's are found by its index in the layout, one token after the other
        P, D = c["P"], c["D"]
        codes, params = s["codes"].cpu().numpy(), s["params"].cpu()
        was, pwas = codes.copy(), params.clone()
        byte = np.arange(P * D // 2)
        owner = (byte // (D // 2), byte // (2 * D) * 4 + byte % 8 // 2)  # which token of its page a byte of K, of V is
        pages, path, kept, base = (s[n].tolist() for n in ("pages", "path", "n_keep", "base"))
        for b in range(c["B"]):
            for i in range(kept[b]):
                to, of = divmod(base[b] + i, P), divmod(base[b] + path[b][i], P)
                tp, fp = pages[b][to[0]], pages[b][of[0]]
                for kv in (0, 1):
                    codes[:, tp, kv, :, owner[kv] == to[1]] = was[:, fp, kv, :, owner[kv] == of[1]]
                params[:, tp, :, :, :, to[1]] = pwas[:, fp, :, :, :, of[1]]
        return torch.from_numpy(codes), params
    if c["kind"] == "tree":
        return _attended(s, s["q"])
    k, v = _quantised(_turned(s, s["k"], True), c["G"]), _quantised(s["v"], c["G"])
    if c["kind"] == "rotate":
        return _turned(s, s["q"], False), k, v
    q = _turned(s, s["q"], True).to(s["q"].dtype)  # what the attention is given
    out, lse = _attended(s, q, (k, v))
    cu, kept, path = s["cu"].tolist(), s["n_keep"].tolist(), s["path"].tolist()
    back = [x.clone() for x in (k, v)]
    for b in range(c["B"]):
        for i in range(kept[b]):
            for x, y in zip(back, (k, v)):
                x[cu[b] + i] = y[cu[b] + path[b][i]]
    return out, lse, *back
