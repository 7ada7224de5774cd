"""Refusals of the 4-bit cache, the evicting cache and the rotary axes: host-side checks, no GPU work."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
import sink_aware_sliding_b200 as swa
from sink_aware_sliding_b200 import build as swa_build

A = 1 << 12  # an aligned address that is never used: each call is refused, or has nothing to do
ODD = A + 4
BAD, UNSUP, OK = swa.SWA_ERR_INVALID_ARG, swa.SWA_ERR_UNSUPPORTED, swa.SWA_OK


@pytest.fixture(scope="module")
def lib():
    swa_build.build()
    return swa.library()


def call(lib, name, order, base, **kw):
    args = dict(base, **kw)
    return getattr(lib, name)(*(args[n] for n in order.split()))


KV4 = dict(k=A, v=A, kc=A, vc=A, sk=A, sv=A, pos=A, q=A, out=A, lse=None, B=1, P=4, Hq=4, Hkv=2, d=128, W=8, S=2,
           n=3, scale=0.1, dt=0, stream=None)


@pytest.mark.parametrize("kw,want", [
    (dict(P=-1), BAD), (dict(B=-1), BAD), (dict(Hkv=0), BAD), (dict(W=0), BAD), (dict(S=-1), BAD), (dict(d=96), UNSUP),
    (dict(k=None), BAD), (dict(v=ODD), BAD), (dict(kc=None), BAD), (dict(vc=ODD), BAD), (dict(sk=None), BAD),
    (dict(sv=ODD), BAD), (dict(P=0), OK), (dict(B=0), OK), (dict(P=0, S=0, sk=None, sv=None), OK)])
def test_kv4_fill(lib, kw, want):
    assert call(lib, "swa_kv4_cache_fill", "k v P kc vc sk sv B Hkv d W S stream", KV4, **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(pos=None), BAD), (dict(pos=A + 2), BAD), (dict(k=ODD), BAD), (dict(W=0), BAD), (dict(d=256), UNSUP),
    (dict(B=1 << 20, Hkv=1 << 12), UNSUP), (dict(B=0), OK), (dict(sk=None), BAD)])
def test_kv4_append(lib, kw, want):
    assert call(lib, "swa_kv4_cache_append", "k v pos kc vc sk sv B Hkv d W S stream", KV4, **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(n=-1), BAD), (dict(pos=None), BAD), (dict(dt=2), BAD), (dict(dt=5), BAD), (dict(out=None), BAD),
    (dict(out=ODD), BAD), (dict(n=0), OK), (dict(B=0), OK), (dict(d=32), UNSUP)])
def test_kv4_read(lib, kw, want):
    assert call(lib, "swa_kv4_cache_read", "pos n kc vc sk sv out out dt B Hkv d W S stream", KV4, **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(Hq=3), BAD), (dict(Hq=18), UNSUP), (dict(scale=0.0), BAD), (dict(scale=float("nan")), BAD), (dict(dt=1), BAD),
    (dict(q=None), BAD), (dict(out=ODD), BAD), (dict(pos=A + 1), BAD), (dict(lse=A + 2), BAD), (dict(kc=None), BAD),
    (dict(B=5000), UNSUP), (dict(B=0), OK), (dict(d=80), UNSUP), (dict(W=2 ** 31 - 1, S=2 ** 31 - 1), UNSUP),
    (dict(W=2 ** 30), UNSUP)])
def test_kv4_decode(lib, kw, want):
    assert call(lib, "swa_kv4_decode", "q kc vc sk sv pos out lse B Hq Hkv d W S scale dt stream", KV4, **kw) == want


def test_kv4_row_bytes(lib):
    assert [swa.swa_kv4_row_bytes(d) for d in (64, 128, 96, 0, -64)] == [40, 80, 0, 0, 0]


HH = dict(q=A, k=A, v=A, lse=A, si=A, kc=A, vc=A, sp=A, sc=A, pos=A, slot=None, out=A, B=1, Hq=4, Hkv=2, L=16, d=128,
          C=8, S=2, recent=3, n_obs=4, W=16, scale=0.1, decay=1.0, dt=0, stream=None)


@pytest.mark.parametrize("kw,want", [
    (dict(n_obs=-1), BAD), (dict(n_obs=17), BAD), (dict(L=-1), BAD), (dict(W=0), BAD), (dict(S=-1), BAD),
    (dict(q=ODD), BAD), (dict(k=None), BAD), (dict(lse=None), BAD), (dict(lse=A + 2), BAD), (dict(sc=A + 1), BAD),
    (dict(d=96), UNSUP), (dict(scale=-1.0), BAD), (dict(Hq=5), BAD), (dict(B=0), OK), (dict(L=0, n_obs=0), OK),
    (dict(B=2 ** 20, L=2 ** 20), UNSUP)])
def test_hh_scores(lib, kw, want):
    assert call(lib, "swa_hh_scores", "q k lse sc B Hq Hkv L d n_obs W S scale stream", HH, **kw) == want


def test_hh_scores_of_prompts_whose_positions_and_windows_leave_32_bits(lib):
    order = "q k lse sc B Hq Hkv L d n_obs W S scale stream"
    for L in (2 ** 30 - 128, 2 ** 30 + 1, 2 ** 31 - 200):
        assert call(lib, "swa_hh_scores", order, HH, B=1, Hq=1, Hkv=1, d=64, L=L, W=2 ** 31 - 1, n_obs=1) == UNSUP
    assert call(lib, "swa_hh_scores", order, HH, B=2 ** 28, Hq=8, Hkv=8, d=64, L=1, n_obs=1) == UNSUP


CACHE = [(dict(recent=0), BAD), (dict(S=-1), BAD), (dict(S=6), BAD), (dict(C=0), BAD), (dict(C=16385), UNSUP),
         (dict(d=32), UNSUP), (dict(kc=None), BAD), (dict(vc=ODD), BAD), (dict(sp=A + 2), BAD), (dict(sc=None), BAD),
         (dict(B=-1), BAD), (dict(Hkv=0), BAD), (dict(B=0), OK), (dict(B=2 ** 22), UNSUP)]


@pytest.mark.parametrize("kw,want", CACHE + [(dict(L=-1), BAD), (dict(k=None), BAD), (dict(si=A + 2), BAD),
                                             (dict(L=2 ** 31 - 1), UNSUP)])
def test_hh_fill(lib, kw, want):
    assert call(lib, "swa_hh_cache_fill", "k v si L kc vc sp sc B Hkv d C S recent stream", HH, **kw) == want


@pytest.mark.parametrize("kw,want", CACHE + [(dict(k=None), BAD), (dict(v=ODD), BAD), (dict(pos=None), BAD),
                                             (dict(slot=A + 2), BAD)])
def test_hh_append(lib, kw, want):
    assert call(lib, "swa_hh_cache_append", "k v pos kc vc sp sc slot B Hkv d C S recent stream", HH, **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(C=0), BAD), (dict(C=16385), UNSUP), (dict(Hq=3), BAD), (dict(Hq=18), UNSUP), (dict(Hq=0), BAD),
    (dict(scale=float("inf")), BAD), (dict(decay=-0.1), BAD), (dict(decay=1.5), BAD), (dict(decay=float("nan")), BAD),
    (dict(dt=1), BAD), (dict(q=None), BAD), (dict(out=ODD), BAD), (dict(lse=A + 2), BAD), (dict(sp=None), BAD),
    (dict(B=0), OK), (dict(d=48), UNSUP)])
def test_hh_decode(lib, kw, want):
    assert call(lib, "swa_hh_decode", "q kc vc sp sc out lse B Hq Hkv d C scale decay dt stream", HH, **kw) == want


ROPE = dict(q=A, k=A, pos=A, T=4, Hq=2, Hkv=1, d=64, qs=128, ks=64, sec=(8, 12, 12), layout=0, base=1e4, inv=0, dt=0)


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), BAD), (dict(Hq=-1), BAD), (dict(sec=()), BAD), (dict(sec=(8, 12, 11)), BAD), (dict(sec=(40, -8)), BAD),
    (dict(sec=(8, 12, 12), layout=2), BAD), (dict(sec=(12, 10, 10), layout=2, T=0), OK), (dict(layout=3), BAD),
    (dict(layout=-1), BAD), (dict(base=0.0), BAD), (dict(base=float("inf")), BAD), (dict(dt=2), BAD), (dict(d=96), UNSUP),
    (dict(sec=(8, 8, 8, 4, 4)), UNSUP), (dict(qs=127), BAD), (dict(qs=132), BAD), (dict(ks=60), BAD),
    (dict(q=ODD), BAD), (dict(k=ODD), BAD), (dict(pos=None), BAD), (dict(pos=A + 2), BAD), (dict(T=0), OK),
    (dict(Hq=0, k=None), OK), (dict(T=2 ** 62), UNSUP)])
def test_rope_axes(lib, kw, want):
    a = dict(ROPE, **kw)
    sec = (ctypes.c_int32 * max(1, len(a["sec"])))(*a["sec"])
    assert lib.swa_rope_axes_qk(a["q"], a["k"], a["pos"], a["T"], a["Hq"], a["Hkv"], a["d"], a["qs"], a["ks"], sec,
                                len(a["sec"]), a["layout"], a["base"], a["inv"], a["dt"], None) == want


@pytest.mark.parametrize("sinks", [0, 2])
def test_an_empty_batch_of_the_4bit_cache_has_nothing_to_do(lib, sinks):
    """Tensors without elements have no address; wrong sizes are refused all the same."""
    none = dict(B=0, S=sinks, k=None, v=None, kc=None, vc=None, sk=None, sv=None, pos=None, q=None, out=None)
    for name, order in (("swa_kv4_cache_fill", "k v P kc vc sk sv B Hkv d W S stream"),
                        ("swa_kv4_cache_append", "k v pos kc vc sk sv B Hkv d W S stream"),
                        ("swa_kv4_cache_read", "pos n kc vc sk sv out out dt B Hkv d W S stream"),
                        ("swa_kv4_decode", "q kc vc sk sv pos out lse B Hq Hkv d W S scale dt stream")):
        assert call(lib, name, order, KV4, **none) == OK
        for wrong, want in ((dict(W=0), BAD), (dict(S=-1), BAD), (dict(Hkv=0), BAD), (dict(d=96), UNSUP)):
            assert call(lib, name, order, KV4, **dict(none, **wrong)) == want
    assert call(lib, "swa_kv4_cache_fill", "k v P kc vc sk sv B Hkv d W S stream", KV4, **dict(none, P=-1)) == BAD
    assert call(lib, "swa_kv4_cache_read", "pos n kc vc sk sv out out dt B Hkv d W S stream", KV4, **dict(none, n=-1)) == BAD


def test_binding_refuses_tensors_that_are_not_on_the_gpu(lib):
    t = torch.zeros(1, 2, 128, dtype=torch.bfloat16)
    u = torch.zeros(1, 2, 8, 80, dtype=torch.uint8)
    p = torch.zeros(1, dtype=torch.int32)
    c = torch.zeros(1, 2, 8, 128, dtype=torch.bfloat16)
    s = torch.zeros(1, 2, 8)
    for f in (lambda: swa.swa_kv4_cache_append(t, t, p, u, u, None, None, 8, 0),
              lambda: swa.swa_kv4_cache_fill(t[None], t[None], u, u, None, None, 8, 0),
              lambda: swa.swa_kv4_cache_read(p[None], u, u, None, None, t[None], t[None], 8, 0),
              lambda: swa.swa_kv4_decode(t, u, u, None, None, p, t, None, 8, 0),
              lambda: swa.swa_hh_scores(t[None], t[None], s, s, 1, 1, 0),
              lambda: swa.swa_hh_cache_fill(t[None], t[None], s, c, c, s.int(), s, 0, 1),
              lambda: swa.swa_hh_cache_append(t, t, p, c, c, s.int(), s, None, 0, 1),
              lambda: swa.swa_hh_decode(t, c, c, s.int(), s, t, None),
              lambda: swa.swa_rope_axes_qk(t, None, p[None], (64,)),
              lambda: swa.swa_rope_axes_qk(t, None, p[None], (64,), layout="other")):
        with pytest.raises(ValueError):
            f()


# ---------------------------------------------------------------- the oracle's own pins
def test_oracle_kv4_is_within_half_a_step_and_packs_by_hand():
    rng = np.random.default_rng(0)
    x = torch.from_numpy(rng.standard_normal((20, 64))).bfloat16()
    code, step, lo = oracle.kv4_quantise(x)
    err = np.abs(oracle.kv4_values(x) - x.double().numpy()).reshape(20, 2, 32)
    # half a step, and what rounding the step to bf16 (2^-8) moves at code 15
    assert (err <= (0.5 + 15 * 2.0 ** -8) * step[..., None] + 1e-12).all()
    ramp = torch.zeros(64)
    ramp[:32] = torch.arange(32) % 16  # step 1, lo 0: the codes are the values
    ramp[32:] = 3.0                    # constant: step 0, lo 3
    row = oracle.kv4_pack(ramp.bfloat16())
    nib = np.stack([row[:32] & 15, row[:32] >> 4], -1).reshape(8, 2, 4)
    np.testing.assert_array_equal(nib[:, 0].reshape(-1), np.arange(32) % 16)
    assert (nib[:, 1] == 0).all()
    np.testing.assert_array_equal(row[32:].view("<u2"), [0x3f80, 0, 0, 0x4040])


def test_oracle_eviction_by_hand():
    nan = float("nan")
    assert oracle.hh_select([5, 1, 9, 9, 2, 0], 4, 1, 1) == [0, 2, 3, 5]
    assert oracle.hh_select([0, 7, 7, 7, 0], 3, 1, 1) == [0, 1, 4]
    assert oracle.hh_select([0, nan, -np.inf, 0], 3, 1, 1) == [0, 2, 3]
    assert oracle.hh_victim([0, 5, 3, 4], [0.0, 9, 2, 1], 6, 1, 2) == 3
    assert oracle.hh_victim([0, 5, 3, 4], [0.0, 9, 2, 1], 6, 1, 3) == 2
    assert oracle.hh_victim([0, 6, 3, 4], [0.0, 9, 2, 1], 6, 1, 2) == 1
    assert oracle.hh_victim([0, 5, -1, -1], [0.0, 9, 2, 1], 6, 1, 2) == 2
    assert oracle.hh_victim([0, 8, 9], [3.0, 2, 2], 6, 1, 2) == 1


def test_oracle_rotation_by_hand():
    x = np.zeros((1, 1, 64))
    x[..., 0] = x[..., 1] = 1.0
    pos = np.array([[np.pi / 2], [np.pi]])
    y = oracle.rope_axes(x, pos, (1, 31), "sections", base=1.0)
    np.testing.assert_allclose(y[0, 0, [0, 32, 1, 33]], [0, 1, -1, 0], atol=1e-15)
    y = oracle.rope_axes(x, pos, (16, 16), "interleaved", base=1.0, inverse=True)
    np.testing.assert_allclose(y[0, 0, [0, 32, 1, 33]], [0, -1, -1, 0], atol=1e-15)
    pos = np.array([[0.0], [1.0]])
    one = oracle.rope_axes(np.ones((1, 1, 64)), pos, (16, 16), "per_axis")
    two = oracle.rope(np.ones((1, 1, 32)), np.array([1]))
    np.testing.assert_allclose(one[0, 0, 16:32], two[0, 0, :16], rtol=1e-12)
