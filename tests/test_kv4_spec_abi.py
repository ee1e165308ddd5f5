"""Sizes and refusals of kvc_kv4_append_rotated, kvc_kv4_tree_attention and kvc_kv4_keep (no GPU: these calls return before
any HIP call), and of their Python side, with stand-ins for device tensors."""
import ctypes

import pytest
import torch

import entropy_coding_02_amd as kvc
from test_kv4_abi import BAD, OK, attn, desc
from test_kv4_binding import ALLOCATED, Fake, calls, pool  # noqa: F401


def rotated(**kw):
    a = dict(k=OK, v=OK, q=OK, q_out=OK, k_token_stride=256, k_head_stride=128, v_token_stride=256, v_head_stride=128,
             q_token_stride=512, q_head_stride=128, q_out_token_stride=512, q_out_head_stride=128, slots=OK, positions=OK,
             table=OK, n_tokens=2, n_positions=100, n_q_heads=4, rot=128, interleaved=0, dtype=2)
    a.update(kw)
    return kvc.KvcKv4Rotated(**a)


def append(d=None, codes=OK, params=OK, st=None, **kw):
    return kvc.lib().kvc_kv4_append_rotated(d or desc(), ctypes.byref(rotated(**kw)), codes, params, st, None)


def tree(d=None, parents=OK, codes=OK, params=OK, st=None, **kw):
    return kvc.lib().kvc_kv4_tree_attention(d or desc(), ctypes.byref(attn(**kw)), parents, codes, params, st, None)


def keep(d=None, pools=(OK, OK, OK + 64, OK + 64), n_pools=2, table=OK, stride=4, max_pages=4, base=OK, path=OK, path_stride=3,
         max_path=3, n_keep=OK, n_seqs=2, st=None):
    a = None if pools is None else (ctypes.c_void_p * len(pools))(*pools)
    return kvc.lib().kvc_kv4_keep(d or desc(), a, n_pools, table, stride, max_pages, base, path, path_stride, max_path, n_keep,
                                  n_seqs, st, None)


@pytest.mark.parametrize("bad", BAD)
def test_bad_descriptors(bad):
    d = desc(**bad)
    assert append(d) == tree(d) == keep(d) == kvc.KVC_ERR_ARG
    assert kvc.lib().kvc_kv4_tree_work_bytes(d, 1, 1, 8, 4, 1) == kvc.KVC_ERR_ARG


def test_append_rotated_refusals():
    assert kvc.lib().kvc_kv4_append_rotated(desc(), None, OK, OK, None, None) == kvc.KVC_ERR_ARG
    for kw in (dict(k=None), dict(v=None), dict(k=OK + 1), dict(v=OK + 1), dict(q=OK + 1), dict(q_out=OK + 1), dict(q=None),
               dict(q_out=None), dict(q=OK + 2, dtype=1), dict(n_tokens=-1), dict(n_tokens=1 << 41), dict(dtype=3), dict(dtype=-1),
               dict(slots=None), dict(slots=OK + 4), dict(positions=None), dict(positions=OK + 4), dict(table=None),
               dict(table=OK + 8), dict(n_positions=-1), dict(rot=0), dict(rot=8), dict(rot=24), dict(rot=144), dict(rot=-16),
               dict(n_q_heads=0), dict(n_q_heads=-3), dict(n_q_heads=65537), dict(q_out_token_stride=640),
               dict(q_out_head_stride=256), dict(codes=None), dict(codes=OK + 8), dict(params=None), dict(params=OK + 4), dict(st=OK + 2)):
        assert append(**kw) == kvc.KVC_ERR_ARG, kw
    assert append(d=desc(D=64), rot=80) == kvc.KVC_ERR_ARG
    assert append(n_tokens=0, k=None, v=None, q=None, q_out=None, slots=None, positions=None, table=None) == kvc.KVC_OK


def test_tree_attention_refusals():
    assert kvc.lib().kvc_kv4_tree_attention(desc(), None, OK, OK, OK, None, None) == kvc.KVC_ERR_ARG
    for kw in (dict(parents=None), dict(parents=OK + 2), dict(causal=0), dict(causal=2), dict(max_q=1025, n_q=2050), dict(q=None),
               dict(out=None), dict(lse=OK + 2), dict(page_table=None), dict(kv_len=None), dict(cu_q=OK + 2), dict(n_q=-1),
               dict(n_seqs=-1), dict(max_q=-1), dict(n_q_heads=5), dict(dtype=1), dict(window=-1), dict(softcap=-1.0),
               dict(softcap=float("nan")), dict(scale=float("inf")), dict(cu_q=None), dict(max_pages=1 << 27),
               dict(codes=None), dict(params=OK + 4), dict(st=OK + 1)):
        assert tree(**kw) == kvc.KVC_ERR_ARG, kw
    for kw in (dict(n_q=0), dict(n_seqs=0), dict(max_q=0)):
        assert tree(q=None, out=None, parents=None, **kw) == kvc.KVC_OK, kw


def test_tree_workspace():
    d, lib = desc(n=10000), kvc.lib()
    need = lib.kvc_kv4_tree_work_bytes(d, 8, 1, 4, 512, 8)  # 8192 keys: split
    assert need > 0 and need % (8 * 4 * 130 * 4) == 0
    a = dict(n_q=8, n_seqs=1, max_q=8, max_pages=512, cu_q=None, d=d)
    for kw, want in ((dict(work=None), kvc.KVC_ERR_ARG), (dict(work=OK + 4), kvc.KVC_ERR_ARG),
                     (dict(work_bytes=need - 1), kvc.KVC_ERR_CAPACITY)):
        assert tree(**{**a, **kw}) == want
    assert lib.kvc_kv4_tree_work_bytes(d, 0, 0, 4, 0, 0) == 0
    for n_q, n_seqs, heads, pages, max_q in ((1, 1, 3, 4, 1), (2050, 1, 4, 4, 1025), (-1, 1, 4, 4, 1), (1, 1, 4, 1 << 27, 1)):
        assert lib.kvc_kv4_tree_work_bytes(d, n_q, n_seqs, heads, pages, max_q) == kvc.KVC_ERR_ARG


@pytest.mark.parametrize("D,G", [(64, 64), (128, 64), (256, 32), (256, 64)])
def test_tree_workspace_covers_every_window(D, G):
    """The size does not know the window, which may change the launch.  (Accepted calls fail at it: there is no device.)"""
    import numpy as np
    if torch.cuda.device_count():
        pytest.skip("accepted calls would launch on stand-in addresses")
    rng = np.random.default_rng(D)
    for _ in range(300):
        H, R, B = (int(rng.integers(1, n)) for n in (17, 13, 40))
        max_q, pages = int(2 ** rng.uniform(0, 10)), int(2 ** rng.uniform(0, 12))
        d = desc(H, D, G, 32, pages)
        need = kvc.lib().kvc_kv4_tree_work_bytes(d, B * max_q, B, H * R, pages, max_q)
        assert need >= 0
        for window in [0] + [int(2 ** rng.uniform(0, 17)) for _ in range(4)] + [2047, pages * 16]:
            assert tree(d, cu_q=None, n_q=B * max_q, n_seqs=B, n_q_heads=H * R, max_pages=pages, max_q=max_q, window=window,
                        work=OK if need else None, work_bytes=need) == kvc.KVC_ERR_HIP


def test_keep_refuses_a_pool_given_twice():
    assert keep(pools=(OK, OK, OK, OK + 64)) == keep(pools=(OK, OK, OK + 64, OK)) == kvc.KVC_ERR_ARG
    assert keep(n_pools=4097) == kvc.KVC_ERR_ARG


def test_keep_refusals():
    for kw in (dict(pools=None), dict(pools=(OK, None)), dict(pools=(None, OK)), dict(pools=(OK, OK, OK + 8, OK)),
               dict(pools=(OK, OK + 4, OK, OK)), dict(n_pools=-1), dict(table=None), dict(table=OK + 2), dict(max_pages=-1),
               dict(max_pages=1 << 27), dict(base=None), dict(base=OK + 2), dict(path=None), dict(path=OK + 1), dict(max_path=-1),
               dict(n_keep=None), dict(n_keep=OK + 3), dict(n_seqs=-1), dict(n_seqs=1 << 24), dict(st=OK + 2)):
        assert keep(**kw) == kvc.KVC_ERR_ARG, kw
    for kw in (dict(n_pools=0), dict(n_seqs=0)):
        assert keep(pools=None, table=None, base=None, path=None, n_keep=None, **kw) == kvc.KVC_OK, kw


def test_packed_arguments_match_the_structure():
    fields = [n for n, _ in kvc.KvcKv4Rotated._fields_]
    assert kvc._ROTATED.size == ctypes.sizeof(kvc.KvcKv4Rotated)
    got = kvc.KvcKv4Rotated.from_buffer_copy(kvc._ROTATED.pack(*range(1, len(fields) + 1)))
    assert [getattr(got, n) for n in fields] == list(range(1, len(fields) + 1))


# --------------------------------------------------------------- the Python side

@pytest.fixture
def made(calls, monkeypatch):  # noqa: F811
    """`calls`, with this file's entry points recorded too."""
    lib = kvc._load()
    for n in ("kvc_kv4_append_rotated", "kvc_kv4_tree_attention", "kvc_kv4_keep"):
        setattr(lib, n, lambda *a, n=n: calls.append((n, a)) or kvc.KVC_OK)
    return calls


F16, I32, I64, F32 = torch.float16, torch.int32, torch.int64, torch.float32


def turn(cache, T=3, **kw):
    H, D = cache.n_kv_heads, cache.head_dim
    a = dict(k=Fake((T, H, D), F16), v=Fake((T, H, D), F16), slots=Fake((T,), I64), positions=Fake((T,), I64),
             table=Fake((50, D), F32), q=Fake((T, 4, D), F16))
    a.update(kw)
    return kvc.kv4_append_rotated(cache, a.pop("k"), a.pop("v"), a.pop("slots"), a.pop("positions"), a.pop("table"), **a)


def grow(cache, n=5, **kw):
    a = dict(q=Fake((n, 4, cache.head_dim), F16), page_table=Fake((1, 200), I32), kv_len=Fake((1,), I32), parents=Fake((n,), I32))
    a.update(kw)
    return kvc.kv4_tree_attention(cache, a.pop("q"), a.pop("page_table"), a.pop("kv_len"), a.pop("parents"), **a)


def hold(caches, B=2, **kw):
    a = dict(page_table=Fake((B, 9), I32), base=Fake((B,), I32), path=Fake((B, 4), I32), n_keep=Fake((B,), I32))
    a.update(kw)
    return kvc.kv4_keep(caches, *(a.pop(n) for n in ("page_table", "base", "path", "n_keep")), **a)


def test_what_a_call_allocates_belongs_to_its_stream(made):
    out = turn(pool(), stream=1234)
    assert ALLOCATED == [out] and out.home.cuda_stream == 1234 and made[-1][1][-1] == 1234
    grow(pool(), return_lse=True, stream=1234)
    assert len(ALLOCATED) == 4 and all(t.home.cuda_stream == 1234 for t in ALLOCATED) and made[-1][1][-1] == 1234
    turn(pool())
    grow(pool())
    hold(pool())
    assert all(t.home is None for t in ALLOCATED[4:]) and all(a[-1] == 77 for _, a in made[-3:])


def test_append_rotated_arguments(made):
    cache = pool()
    q = Fake((3, 4, 64), F16)
    assert turn(cache, q=q, q_out=q, table=Fake((50, 32), F32), interleaved=True) is q and not ALLOCATED
    a = kvc.KvcKv4Rotated.from_buffer_copy(made[-1][1][1])
    assert (a.q, a.q_out, a.rot, a.interleaved, a.n_positions, a.n_q_heads, a.n_tokens) == (q.address, q.address, 32, 1, 50, 4, 3)
    assert turn(cache, q=None) is None
    a = kvc.KvcKv4Rotated.from_buffer_copy(made[-1][1][1])
    assert a.q is None and a.q_out is None


def test_what_is_refused(made):
    cache, far = pool(), lambda *s: Fake(s[:-1], s[-1], device=1)  # noqa: E731
    bad = [lambda: turn(cache, k=Fake((3, 2, 32), F16)), lambda: turn(cache, v=Fake((4, 2, 64), F16)),
           lambda: turn(cache, v=Fake((3, 2, 64), F32)), lambda: turn(cache, q=Fake((3, 4, 64), torch.bfloat16)),
           lambda: turn(cache, q=Fake((2, 4, 64), F16)), lambda: turn(cache, q=Fake((3, 256), F16)),
           lambda: turn(cache, q=None, q_out=Fake((3, 4, 64), F16)), lambda: turn(cache, q_out=Fake((3, 5, 64), F16)),
           lambda: turn(cache, q_out=Fake((3, 4, 64), F16, strides=(0, 64, 1))), lambda: turn(cache, slots=Fake((3,), I32)),
           lambda: turn(cache, positions=Fake((2,), I64)), lambda: turn(cache, table=Fake((64,), F32)),
           lambda: turn(cache, table=Fake((50, 64), torch.float64)), lambda: turn(cache, table=Fake((50, 64), F32, strides=(128, 1))),
           lambda: turn(cache, k=Fake((3, 2, 64), torch.float64), v=Fake((3, 2, 64), torch.float64), q=None),
           lambda: turn(cache, table=far(50, 64, F32)), lambda: turn(cache, positions=far(3, I64)),
           lambda: turn(cache, q=far(3, 4, 64, F16)), lambda: turn(cache, q_out=far(3, 4, 64, F16)),
           lambda: grow(cache, parents=Fake((4,), I32)), lambda: grow(cache, parents=Fake((5,), I64)),
           lambda: grow(cache, parents=far(5, I32)), lambda: grow(cache, parents=Fake((5,), I32, strides=(2,))),
           lambda: grow(cache, work=far(1 << 24, torch.uint8)),
           lambda: hold([]), lambda: hold([cache, cache]), lambda: hold([cache, pool(H=3)]), lambda: hold([cache, pool(device=1)]),
           lambda: hold(cache, path=Fake((2, 4), I64)), lambda: hold(cache, path=Fake((3, 4), I32)), lambda: hold(cache, path=Fake((8,), I32)),
           lambda: hold(cache, path=Fake((2, 4), I32, strides=(1, 2))), lambda: hold(cache, page_table=far(2, 9, I32)),
           lambda: hold(cache, base=Fake((3,), I32)), lambda: hold(cache, n_keep=Fake((2,), I64)), lambda: hold(cache, n_keep=far(2, I32))]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    with pytest.raises(kvc.KvcError):
        grow(cache, n=1025)  # a tree that a block does not hold
    assert not made


def test_keep_in_several_caches(made):
    caches = [pool() for _ in range(70)]
    hold(caches, path=Fake((2, 4), I32, strides=(9, 1)))
    a = made[-1][1]
    assert list((ctypes.c_void_p * 140).from_buffer_copy(a[1])) == [p for c in caches for p in (c.codes_ptr, c.params_ptr)]
    assert a[2] == 70 and a[8:10] == (9, 4) and a[-2] == caches[0].status_ptr
