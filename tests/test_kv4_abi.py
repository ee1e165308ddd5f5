"""The kvc_kv4_* entry points' sizes and refusals (no GPU: these calls return
before any HIP call), and the reference's own pins."""
import ctypes

import numpy as np
import pytest

import entropy_coding_02_amd as kvc
import kv4_ref

OK = 1 << 20  # an aligned stand-in address; nothing is launched on these paths


def desc(H=2, D=128, G=64, P=16, n=3):
    return kvc.KvcKv4Desc(H, D, G, P, n)


@pytest.mark.parametrize("D,G", [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128), (256, 32), (256, 64), (256, 128)])
@pytest.mark.parametrize("P", [16, 64, 256])
def test_sizes(D, G, P):
    d, lib = desc(5, D, G, P, 7), kvc.lib()
    assert lib.kvc_kv4_codes_bytes(d) == 7 * 2 * 5 * P * D // 2
    assert lib.kvc_kv4_params_bytes(d) == 7 * 2 * 5 * (D // G) * P * 4


def test_sizes_pass_32_bits():
    d = desc(8, 128, 64, 256, 1 << 24)
    assert kvc.lib().kvc_kv4_codes_bytes(d) == (1 << 24) * 2 * 8 * 256 * 64


BAD = [dict(H=0), dict(H=1025), dict(D=32), dict(D=96), dict(D=512), dict(G=16), dict(G=48), dict(G=256), dict(D=64, G=128),
       dict(P=8), dict(P=24), dict(P=512), dict(P=0), dict(P=-16), dict(n=0), dict(n=-1), dict(n=1 << 31)]


@pytest.mark.parametrize("bad", BAD)
def test_bad_descriptors(bad):
    d, lib = desc(**bad), kvc.lib()
    assert lib.kvc_kv4_codes_bytes(d) == kvc.KVC_ERR_ARG
    assert lib.kvc_kv4_params_bytes(d) == kvc.KVC_ERR_ARG
    assert lib.kvc_kv4_append(d, OK, OK, 1, 0, 0, 0, 0, 0, OK, OK, OK, None, None) == kvc.KVC_ERR_ARG
    assert lib.kvc_kv4_read(d, OK, OK, OK, 1, OK, OK, 0, 0, 0, 0, 0, None, None) == kvc.KVC_ERR_ARG
    assert lib.kvc_kv4_work_bytes(d, 1, 1, 8, 4, 1) == kvc.KVC_ERR_ARG


def test_append_and_read_refusals():
    d, lib = desc(), kvc.lib()

    def ap(k=OK, v=OK, n=1, dt=0, slots=OK, codes=OK, params=OK, st=None):
        return lib.kvc_kv4_append(d, k, v, n, 256, 128, 256, 128, dt, slots, codes, params, st, None)

    def rd(codes=OK, params=OK, slots=OK, n=1, k=OK, v=OK, dt=0, st=None):
        return lib.kvc_kv4_read(d, codes, params, slots, n, k, v, 256, 128, 256, 128, dt, st, None)

    for kw in (dict(k=None), dict(v=None), dict(k=OK + 1), dict(v=OK + 1), dict(k=OK + 2, dt=1), dict(n=-1), dict(dt=3),
               dict(dt=-1), dict(slots=None), dict(slots=OK + 4), dict(codes=None), dict(codes=OK + 8),
               dict(params=None), dict(params=OK + 4), dict(st=OK + 2)):
        assert ap(**kw) == kvc.KVC_ERR_ARG, kw
    for kw in (dict(k=None, v=None), dict(k=OK + 1), dict(v=OK + 1), dict(n=-1), dict(dt=3), dict(slots=None),
               dict(slots=OK + 4), dict(codes=None), dict(params=None), dict(st=OK + 2)):
        assert rd(**kw) == kvc.KVC_ERR_ARG, kw
    assert ap(n=0, k=None, v=None, slots=None) == kvc.KVC_OK
    assert rd(n=0, k=None, v=None, slots=None) == kvc.KVC_OK


def attn(**kw):
    a = dict(q=OK, out=OK, lse=None, q_token_stride=512, q_head_stride=128, out_token_stride=512, out_head_stride=128,
             page_table=OK, table_stride=4, kv_len=OK, cu_q=OK, n_q=3, n_seqs=2, n_q_heads=4, max_pages=4, max_q=2,
             dtype=2, causal=1, window=0, softcap=0.0, scale=0.1, work=OK, work_bytes=1 << 30)
    a.update(kw)
    return kvc.KvcKv4Attn(**a)


def test_attention_refusals():
    d, lib = desc(), kvc.lib()

    def call(codes=OK, params=OK, st=None, **kw):
        return lib.kvc_kv4_attention(d, ctypes.byref(attn(**kw)), codes, params, st, None)

    assert lib.kvc_kv4_attention(d, None, OK, OK, None, None) == kvc.KVC_ERR_ARG
    for kw in (dict(q=None), dict(out=None), dict(q=OK + 1), dict(out=OK + 1), dict(lse=OK + 2), dict(page_table=None),
               dict(page_table=OK + 2), dict(kv_len=None), dict(kv_len=OK + 2), dict(cu_q=OK + 2), dict(n_q=-1),
               dict(n_seqs=-1), dict(max_q=-1), dict(max_pages=-1), dict(n_q_heads=5), dict(n_q_heads=1),
               dict(n_q_heads=0), dict(dtype=1), dict(dtype=7), dict(window=-1), dict(window=4, causal=0),
               dict(softcap=-1.0), dict(softcap=float("nan")), dict(softcap=float("inf")), dict(scale=float("nan")),
               dict(scale=float("inf")), dict(cu_q=None), dict(max_pages=1 << 27), dict(max_q=1 << 30),
               dict(codes=None), dict(codes=OK + 8), dict(params=None), dict(st=OK + 1)):
        assert call(**kw) == kvc.KVC_ERR_ARG, kw
    # nothing to do: no launch, whatever the pointers
    for kw in (dict(n_q=0), dict(n_seqs=0), dict(max_q=0)):
        assert call(q=None, out=None, **kw) == kvc.KVC_OK, kw


def test_attention_workspace():
    d, lib = desc(n=10000), kvc.lib()
    need = lib.kvc_kv4_work_bytes(d, 1, 1, 4, 512, 1)  # 8192 keys, one row tile a head: split
    assert need > 0 and need % (4 * 130 * 4) == 0
    a = dict(n_q=1, n_seqs=1, max_q=1, max_pages=512, cu_q=None)
    for kw, want in ((dict(work=None), kvc.KVC_ERR_ARG), (dict(work=OK + 4), kvc.KVC_ERR_ARG),
                     (dict(work_bytes=need - 1), kvc.KVC_ERR_CAPACITY)):
        assert lib.kvc_kv4_attention(d, ctypes.byref(attn(**{**a, **kw})), OK, OK, None, None) == want
    assert lib.kvc_kv4_work_bytes(d, 0, 0, 4, 0, 0) == 0
    assert lib.kvc_kv4_work_bytes(d, 1, 1, 3, 4, 1) == kvc.KVC_ERR_ARG


def test_binding_refuses_host_tensors():
    import torch
    with pytest.raises(ValueError):
        kvc.Kv4Cache(2, 64, 4, codes=torch.zeros(4 * 2 * 2 * 64 * 32, dtype=torch.uint8),
                     params=torch.zeros((4, 2, 2, 1, 64, 2), dtype=torch.float16))
    with pytest.raises(kvc.KvcError):
        kvc.Kv4Cache(2, 96, 4, device="cpu")


def test_reference_round_trip_and_bound():
    """|value - x| <= s/2 for a value inside the codes' range, plus the roundings of s and lo."""
    rng = np.random.default_rng(0)
    x = rng.standard_normal((50, 128)).astype(np.float16).astype(np.float32)
    c, s, lo = kv4_ref.quantise(x, 32)
    y = kv4_ref.values(c, s, lo, 32)
    s64 = np.repeat(s.astype(np.float64), 32, -1)
    # s is off by at most 2^-11 of itself, so the top code by 15 * 2^-11 s; the quotient's fp32 roundings by 15 * 2^-23 s
    assert (np.abs(y - x) <= s64 * (0.5 + 15 * 2.0 ** -11 + 15 * 2.0 ** -22)).all()
    assert c.min() == 0 and c.max() == 15
    const, s, lo = kv4_ref.quantise(np.full((1, 64), 2.5, np.float32), 64)
    assert (const == 0).all() and s[0, 0] == 0 and lo[0, 0] == 2.5


def test_reference_layouts_are_permutations():
    for D in (64, 128, 256):
        seen = set()
        for off in range(16):
            for c in range(D):
                seen.add(kv4_ref.v_byte(D, off, c))
        assert len(seen) == 16 * D and max(b for b, _ in seen) == 16 * D // 2 - 1
        code = np.arange(D) % 16
        assert sorted(np.concatenate([kv4_ref.pack_k(code) & 15, kv4_ref.pack_k(code) >> 4])) == sorted(code)


def test_packed_arguments_match_the_structure():
    """The binding packs kvc_kv4_attn itself: same size, and every field where the structure has it."""
    fields = [n for n, _ in kvc.KvcKv4Attn._fields_]
    assert kvc._ATTN.size == ctypes.sizeof(kvc.KvcKv4Attn)
    vals = [0.5 + i if n in ("softcap", "scale") else i + 1 for i, n in enumerate(fields)]
    got = kvc.KvcKv4Attn.from_buffer_copy(kvc._ATTN.pack(*vals))
    assert [getattr(got, n) for n in fields] == vals


@pytest.mark.parametrize("D,G", [(64, 64), (128, 64), (256, 32), (256, 64)])
def test_workspace_covers_every_window(D, G):
    """kvc_kv4_work_bytes does not know the window, which may change the launch: with that much workspace no
    call is refused.  (Accepted calls fail at the launch: there is no device.)"""
    import torch
    if torch.cuda.device_count():
        pytest.skip("accepted calls would launch on stand-in addresses")
    lib = kvc.lib()
    rng = np.random.default_rng(D)
    for _ in range(400):
        H, R, B = (int(rng.integers(1, n)) for n in (17, 13, 40))
        max_q = int(2 ** rng.uniform(0, 11))
        pages = int(2 ** rng.uniform(0, 12))
        d = desc(H, D, G, 32, pages)
        need = lib.kvc_kv4_work_bytes(d, B * max_q, B, H * R, pages, max_q)
        assert need >= 0
        for window in [0] + [int(2 ** rng.uniform(0, 17)) for _ in range(4)] + [2047, 2000, pages * 16]:
            a = attn(cu_q=None, n_q=B * max_q, n_seqs=B, n_q_heads=H * R, max_pages=pages, max_q=max_q, window=window,
                     work=OK if need else None, work_bytes=need)
            assert lib.kvc_kv4_attention(d, ctypes.byref(a), OK, OK, None, None) == kvc.KVC_ERR_HIP


def test_launch_limits():
    """Sizes whose launches would pass 2^24 blocks are refused, the largest products without overflow."""
    d, lib = desc(H=1024, D=64, G=64, n=10), kvc.lib()
    big = (1 << 31) - 1
    for n_q, n_seqs, heads, pages, max_q in ((big, big, 1024 * 2000000, big, big), (1 << 20, 1 << 14, 1024, 4, 64),
                                            (1, 1, 1024, 4, 1 << 18), (1 << 21, 1, 1024, 4, 1)):
        assert lib.kvc_kv4_work_bytes(d, n_q, n_seqs, heads, pages, max_q) == kvc.KVC_ERR_ARG
    assert lib.kvc_kv4_work_bytes(d, 1 << 13, 1 << 13, 1024, 4, 1) == 0
