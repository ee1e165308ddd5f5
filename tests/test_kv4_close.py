"""The closeness of kv4_close accepts a rounded result and rejects planted mistakes (no GPU)."""
import numpy as np
import pytest

import kv4_close
import kv4_ref

D, G = 128, 64


def problem(n, nq, R, dt, seed=0):
    k, v, q = (t.float().numpy() for t in kv4_close.inputs((n, 1, D), (nq, R, D), dt, seed))
    kq, vq = (kv4_ref.quantise(x[:, 0], G) for x in (k, v))
    return q.astype(np.float64), kq, vq


def attend(q, kq, vq, n, keep=slice(None), window=0, scale=D ** -0.5, causal=True):
    k, v = kv4_ref.values(*kq, G), kv4_ref.values(*vq, G)
    pos = n - len(q) + np.arange(len(q))
    return kv4_ref.attention(q, k[keep], v[keep], pos, len(k[keep]), causal, window, 0.0, scale)


def judged(got, gl, wo, wl, dt):
    return kv4_close.out_off(kv4_close.rounded(got, dt), wo, dt), kv4_close.lse_off(gl.astype(np.float32).astype(np.float64), wl)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("n,nq", [(40, 1), (700, 32), (5000, 4), (9001, 4)])
def test_accepts_what_is_off_by_fp32_steps(n, nq, dt):
    q, kq, vq = problem(n, nq, 4, dt)
    wo, wl = attend(q, kq, vq, n)
    assert np.abs(q @ kv4_ref.values(*kq, G).T).max() * D ** -0.5 < kv4_close.MOST
    rng = np.random.default_rng(1)
    e = 1 + rng.uniform(-1, 1, wo.shape) * 2.0 ** -18
    o, l = judged(wo * e, wl + rng.uniform(-1, 1, wl.shape) * 2.0 ** -19, wo, wl, dt)
    assert o < 0.75 and l < 0.75


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("n,nq", [(700, 32), (5000, 4), (9001, 4)])
@pytest.mark.parametrize("mistake", ["first key lost", "last key lost", "one key in a tile lost", "window one short",
                                     "scale", "code 0 for 1"])
def test_rejects_one_lost_key_and_the_like(n, nq, dt, mistake):
    q, kq, vq = problem(n, nq, 4, dt)
    window = n // 2
    wo, wl = attend(q, kq, vq, n, window=window if mistake == "window one short" else 0, causal=mistake[0] == "w")
    if mistake == "window one short":
        got = attend(q, kq, vq, n, window=window - 1)
    elif mistake == "scale":
        got = attend(q, kq, vq, n, scale=D ** -0.5 * (1 + 2.0 ** -14), causal=False)
    elif mistake == "code 0 for 1":
        got = attend(q, kq, (np.where(vq[0] == 1, 0, vq[0]).astype(np.uint8), *vq[1:]), n, causal=False)
        assert judged(*got, wo, wl, dt)[0] > 1
        return
    else:
        lost = {"first key lost": 0, "last key lost": n - 1, "one key in a tile lost": n // 2}[mistake]
        got = attend(q, kq, vq, n, keep=np.arange(n) != lost, causal=False)
    o, l = judged(*got, wo, wl, dt)
    assert l > 1, (o, l)
    assert o > 1 or mistake == "scale" or n > 700, (o, l)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_rejects_wrong_values(dt):
    q, kq, vq = problem(700, 32, 4, dt)
    wo, wl = attend(q, kq, vq, 700)
    lo = vq[2].copy()
    lo[:, 1] = 0  # one group's lo lost
    shifted = (vq[0], vq[1], np.roll(vq[2], 1, 0))  # parameters of the token before
    for got in (np.zeros_like(wo), wo * (1 + 2.0 ** -12), np.roll(wo, 1, -1), attend(q, kq, (vq[0], vq[1], lo), 700)[0],
                attend(q, kq, shifted, 700)[0]):
        assert judged(got, wl, wo, wl, dt)[0] > 1
    empty = wl.copy()
    empty[3, 1] = -np.inf
    assert judged(wo, empty, wo, wl, dt)[1] > 1
