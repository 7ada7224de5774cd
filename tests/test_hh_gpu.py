"""The cache that evicts by accumulated attention weight, on the GPU (through the C ABI), against the fp64 oracle.

Tolerances.  Scores of q and k are float32 sums of d exact products: at most (d + 16) 2^-24 of sum |q||k| scale, and
2^-20 to allow for the matrix unit's own alignment; dz below.  The exponential adds 2^-21.  A weight is then off by
(dz + dlse + 2^-20) relative, a log-sum-exp by dz plus a rounding of its value, an output by 2 dz max|v| plus what the two
bf16 parts of the softmax numerators leave (2^-16), and a bf16 output by its rounding, 2^-8."""
import math

import numpy as np
import pytest
import torch

import oracle
import sink_aware_sliding_b200 as swa

pytestmark = pytest.mark.gpu


def rand(shape, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).bfloat16()


def dz_of(q, k, scale):
    size = scale * math.sqrt(float((q ** 2).sum(-1).max()) * float((k ** 2).sum(-1).max()))
    return size * ((q.shape[-1] + 16) * 2.0 ** -24 + 2.0 ** -20) + 2.0 ** -21


# ---------------------------------------------------------------- scores of a prompt
@pytest.mark.parametrize("d,Hq,H", [(64, 2, 2), (128, 4, 1), (128, 6, 2)])
@pytest.mark.parametrize("L,n_obs,W,S", [(1, 1, 1, 0), (5, 3, 5, 2), (128, 128, 128, 0), (129, 1, 129, 0),
                                        (300, 300, 300, 0), (300, 77, 50, 4), (700, 130, 128, 0), (400, 400, 1, 3),
                                        (513, 256, 600, 200), (260, 0, 260, 0)])
def test_scores_match_oracle(d, Hq, H, L, n_obs, W, S):
    B = 2
    q, k = rand((B, L, Hq, d), L), rand((B, L, H, d), L + 1)
    out = torch.empty(B, L, Hq, d, device="cuda", dtype=torch.bfloat16)
    lse = torch.empty(B, Hq, L, device="cuda")
    swa.swa_fwd(q.cuda(), k.cuda(), k.cuda(), out, lse, W, S)
    scale = 1 / math.sqrt(d)
    exact = oracle.swa_fwd(q, k, k, W, S, scale)[1]
    dlse = float(np.abs(lse.double().cpu().numpy() - exact).max())
    assert dlse < 1e-3
    score = torch.full((B, H, L), 7.0, device="cuda")
    swa.swa_hh_scores(q.cuda(), k.cuda(), lse, score, n_obs, W, S)
    assert swa.swa_device_error() == 0
    want = oracle.hh_scores(q, k, n_obs, W, S, scale)
    got = score.double().cpu().numpy()
    tol = (dz_of(q.double(), k.double(), scale) + dlse + 2.0 ** -18) * want + 1e-9
    assert (np.abs(got - want) <= tol).all(), np.abs(got - want).max()
    if n_obs:
        np.testing.assert_allclose(got.sum(-1), n_obs * Hq // H, rtol=1e-3)


def test_scores_of_large_logits_and_an_odd_scale():
    B, L, H, d = 1, 200, 1, 64
    q, k = rand((B, L, H, d), 1, 4.0), rand((B, L, H, d), 2, 4.0)
    lse = torch.empty(B, H, L, device="cuda")
    swa.swa_fwd(q.cuda(), k.cuda(), k.cuda(), torch.empty_like(q, device="cuda"), lse, L, 0, scale=0.3)
    exact = oracle.swa_fwd(q, k, k, L, 0, 0.3)[1]
    dlse = float(np.abs(lse.double().cpu().numpy() - exact).max())
    score = torch.empty(B, H, L, device="cuda")
    swa.swa_hh_scores(q.cuda(), k.cuda(), lse, score, L, L, 0, scale=0.3)
    want = oracle.hh_scores(q, k, L, L, 0, 0.3)
    tol = (dz_of(q.double(), k.double(), 0.3) + dlse + 2.0 ** -18) * want + 1e-9
    assert (np.abs(score.double().cpu().numpy() - want) <= tol).all()


# ---------------------------------------------------------------- filling from a prompt
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("L,C,S,recent", [(0, 5, 1, 2), (1, 1, 0, 1), (7, 9, 2, 3), (9, 9, 2, 3), (10, 9, 2, 3),
                                          (300, 50, 4, 46), (300, 50, 4, 20), (5000, 600, 0, 1), (4097, 4096, 16, 512)])
@pytest.mark.parametrize("kind", ["plain", "ties", "odd"])
def test_fill_keeps_what_the_oracle_keeps(d, L, C, S, recent, kind):
    B, H = 2, 2
    k, v = rand((B, L, H, d), 1), rand((B, L, H, d), 2)
    rng = np.random.default_rng(L + C)
    s = rng.random((B, H, L)).astype(np.float32) ** 8
    if kind == "ties":
        s = np.floor(s * 4).astype(np.float32)
    if kind == "odd" and L:
        s -= np.float32(0.5)
        flat = s.reshape(-1)
        at = rng.integers(0, flat.size, 12)
        flat[at] = np.array([np.inf, -np.inf, np.nan, -np.nan, 0.0, -0.0, 1e-40, -1e-40, 3e38, -3e38, np.nan, 0.0])
    kc, vc = (torch.full((B, H, C, d), 5.0, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    sp = torch.full((B, H, C), 77, device="cuda", dtype=torch.int32)
    score = torch.full((B, H, C), 77.0, device="cuda")
    swa.swa_hh_cache_fill(k.cuda(), v.cuda(), torch.from_numpy(s).cuda(), kc, vc, sp, score, S, recent)
    torch.cuda.synchronize()
    for b in range(B):
        for h in range(H):
            keep = oracle.hh_select(s[b, h], C, S, recent)
            n = len(keep)
            assert sp[b, h].cpu().tolist() == keep + [-1] * (C - n)
            np.testing.assert_array_equal(score[b, h, :n].cpu().numpy(), s[b, h, keep])
            assert (score[b, h, n:] == 0).all()
            assert torch.equal(kc[b, h, :n].cpu(), k[b, keep, h]) and torch.equal(vc[b, h, :n].cpu(), v[b, keep, h])
            assert (kc[b, h, n:] == 5).all() and (vc[b, h, n:] == 5).all()


@pytest.mark.parametrize("B,H,L,C", [(1, 2, 60001, 1000), (1, 1, 500003, 3000), (40, 4, 50001, 700), (5, 4, 9000, 2500)])
def test_fill_of_long_prompts(B, H, L, C):
    """Prompts whose keys do not fit shared memory, and one whose do, with many ties."""
    d, S, recent = 64, 4, 100
    k = rand((B, L, H, d), 1)
    s = np.floor(np.random.default_rng(3).random((B, H, L)) * 400).astype(np.float32)  # many ties
    kc, vc = (torch.zeros(B, H, C, d, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    sp, score = torch.zeros(B, H, C, device="cuda", dtype=torch.int32), torch.zeros(B, H, C, device="cuda")
    swa.swa_hh_cache_fill(k.cuda(), (-k).cuda(), torch.from_numpy(s).cuda(), kc, vc, sp, score, S, recent)
    torch.cuda.synchronize()
    for b, h in {(0, 0), (B - 1, H - 1), (B // 2, 0)}:
        keep = oracle.hh_select(s[b, h], C, S, recent)
        assert sp[b, h].cpu().tolist() == keep
        assert torch.equal(kc[b, h].cpu(), k[b, keep, h]) and torch.equal(vc[b, h].cpu(), -k[b, keep, h])
        np.testing.assert_array_equal(score[b, h].cpu().numpy(), s[b, h, keep])


# ---------------------------------------------------------------- appending
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("C,S,recent", [(1, 0, 1), (4, 1, 3), (5, 0, 1), (300, 4, 64), (700, 0, 512)])
def test_append_evicts_what_the_oracle_evicts(d, C, S, recent):
    B, H = 3, 2
    kc, vc = (torch.zeros(B, H, C, d, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    sp = torch.full((B, H, C), -1, device="cuda", dtype=torch.int32)
    score = torch.zeros(B, H, C, device="cuda")
    slot = torch.empty(B, H, device="cuda", dtype=torch.int32)
    rng = np.random.default_rng(C)
    steps = list(range(C + 40)) + [C + 39, C + 39, 3, 10 ** 9, 2 ** 31 - 1, 5]
    if C >= 300:
        # start full, so that every step evicts
        sp.copy_(torch.stack([torch.randperm(C).int() for _ in range(B * H)]).view(B, H, C))
        steps = steps[C:]
    for n, p in enumerate(steps):
        s = rng.random((B, H, C)).astype(np.float32)
        if n % 3 == 1:
            s = np.floor(s * 3).astype(np.float32)
        if n % 7 == 5:
            s[0, 0, rng.integers(0, C)] = np.nan
            s[1, 0, rng.integers(0, C)] = -np.inf
            s[2, 1, rng.integers(0, C)] = -0.0
        score.copy_(torch.from_numpy(s))
        before = sp.cpu().numpy()
        old = [t.clone() for t in (kc, vc)]
        k, v = rand((B, H, d), 2 * n), rand((B, H, d), 2 * n + 1)
        pos = [p, p, -1 if n % 4 == 2 else p]
        swa.swa_hh_cache_append(k.cuda(), v.cuda(), torch.tensor(pos, dtype=torch.int32, device="cuda"), kc, vc, sp,
                                score, slot, S, recent)
        torch.cuda.synchronize()
        want_sp, want_s = before.copy(), s.copy()
        for b in range(B):
            for h in range(H):
                if pos[b] < 0:
                    assert int(slot[b, h]) == -1
                    continue
                i = oracle.hh_victim(before[b, h], s[b, h], p, S, recent)
                assert int(slot[b, h]) == i, (n, b, h)
                want_sp[b, h, i], want_s[b, h, i] = p, 0
                old[0][b, h, i], old[1][b, h, i] = k[b, h].cuda(), v[b, h].cuda()
        np.testing.assert_array_equal(sp.cpu().numpy(), want_sp)
        np.testing.assert_array_equal(score.cpu().numpy(), want_s)
        assert torch.equal(kc, old[0]) and torch.equal(vc, old[1])


def test_append_without_a_place_for_the_slot():
    kc, vc = (torch.zeros(1, 1, 4, 64, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    sp, score = torch.full((1, 1, 4), -1, device="cuda", dtype=torch.int32), torch.zeros(1, 1, 4, device="cuda")
    k = rand((1, 1, 64), 1).cuda()
    swa.swa_hh_cache_append(k, k, torch.zeros(1, device="cuda", dtype=torch.int32), kc, vc, sp, score, None, 0, 1)
    assert sp.flatten().tolist() == [0, -1, -1, -1] and torch.equal(kc[0, 0, 0], k[0, 0])


# ---------------------------------------------------------------- decoding
def check_decode(q, kc, vc, sp, s, scale=None, decay=1.0, f32=True):
    B, Hq, d = q.shape
    H = kc.shape[1]
    out = torch.full((B, Hq, d), 7.0, device="cuda", dtype=torch.float32 if f32 else torch.bfloat16)
    lse, score = torch.full((B, Hq), 7.0, device="cuda"), torch.from_numpy(s).cuda()
    swa.swa_hh_decode(q.cuda(), kc.cuda(), vc.cuda(), torch.from_numpy(sp).cuda(), score, out, lse, scale, decay)
    torch.cuda.synchronize()
    scale = scale or 1 / math.sqrt(d)
    occ = sp >= 0
    k64 = np.where(occ[..., None], kc.double().numpy(), 0.0)
    v64 = np.where(occ[..., None], vc.double().numpy(), 0.0)
    wo, wl, ws = oracle.hh_decode(q, k64, v64, sp, s, scale, decay)
    dz = dz_of(q.double(), torch.from_numpy(k64), scale)
    go, gl, gs = (t.double().cpu().numpy() for t in (out, lse, score))
    tol = (2 * dz + 2.0 ** -16) * np.abs(v64).max() + 1e-30 + (0 if f32 else 2.0 ** -8 * np.abs(wo))
    assert (np.abs(go - wo) <= tol).all(), (np.abs(go - wo).max(), dz)
    empty = np.isneginf(wl)
    assert np.array_equal(empty, np.isneginf(gl))
    fine = ~empty
    assert (np.abs(gl[fine] - wl[fine]) <= dz + 2.0 ** -22 * np.abs(wl[fine]) + 1e-6).all()
    np.testing.assert_array_equal(score.cpu().numpy()[~occ], s[~occ])
    added = ws - decay * s
    tol_s = 2 * (dz + 2.0 ** -19) * added + 2.0 ** -22 * np.abs(ws) + 1e-9
    assert (np.abs(gs - ws) <= tol_s)[occ].all(), np.abs(gs - ws).max()


def cache(B, H, C, d, seed, share, scale=1.0):
    rng = np.random.default_rng(seed)
    sp = rng.permutation(4 * C)[:C].astype(np.int32) + np.zeros((B, H, 1), np.int32)
    sp = np.where(rng.random((B, H, C)) < share, sp, -1).astype(np.int32)
    return rand((B, H, C, d), seed, scale), rand((B, H, C, d), seed + 1), sp, rng.random((B, H, C)).astype(np.float32)


@pytest.mark.parametrize("d,Hq,H", [(64, 2, 2), (64, 8, 1), (128, 8, 2), (128, 7, 1), (128, 3, 3), (64, 12, 4)])
@pytest.mark.parametrize("C,share", [(1, 1.0), (15, 1.0), (16, 0.5), (130, 1.0), (500, 0.05), (700, 0.9)])
def test_decode_matches_oracle(d, Hq, H, C, share):
    B = 4
    k, v, sp, s = cache(B, H, C, d, C + d, share)
    sp[1, 0] = -1  # nothing occupied
    check_decode(rand((B, Hq, d), 3), k, v, sp, s)
    check_decode(rand((B, Hq, d), 4), k, v, sp, s, decay=0.75, f32=False)


@pytest.mark.parametrize("B,H,G,C", [(1, 1, 8, 16384), (1, 8, 4, 2048), (40, 4, 2, 300), (2, 2, 1, 5000)])
def test_decode_long_and_wide(B, H, G, C):
    k, v, sp, s = cache(B, H, C, 128, 7, 0.95)
    check_decode(rand((B, H * G, 128), 8), k, v, sp, s)


def test_decode_large_logits_and_decay_zero():
    k, v, sp, s = cache(2, 2, 100, 64, 9, 0.8, scale=6.0)
    check_decode(rand((2, 4, 64), 10, 6.0), k, v, sp, s, scale=0.5, decay=0.0)


def test_empty_slots_may_hold_anything():
    k, v, sp, s = cache(1, 2, 90, 128, 11, 0.6)
    for t, x in ((k, float("nan")), (v, float("inf"))):
        t[torch.from_numpy(sp) < 0] = x
    s[sp < 0] = np.nan
    check_decode(rand((1, 4, 128), 12), k, v, sp, s)


# ---------------------------------------------------------------- together
def test_a_prompt_and_generated_tokens_in_turn():
    """Forward, scores, fill, then append and decode step by step, against an oracle that follows the library's
    choices (each choice is checked on the library's own scores, which rounding may order differently)."""
    B, L, steps, Hq, H, d, C, S, recent = 2, 150, 40, 4, 2, 64, 60, 2, 16
    scale = 1 / math.sqrt(d)
    q, k, v = rand((B, L + steps, Hq, d), 1), rand((B, L + steps, H, d), 2), rand((B, L + steps, H, d), 3)
    qp, kp, vp = (t[:, :L].contiguous().cuda() for t in (q, k, v))
    out, lse = torch.empty_like(qp), torch.empty(B, Hq, L, device="cuda")
    swa.swa_fwd(qp, kp, vp, out, lse, L, 0)
    si = torch.empty(B, H, L, device="cuda")
    swa.swa_hh_scores(qp, kp, lse, si, 32, L, 0)
    kc, vc = (torch.zeros(B, H, C, d, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    sp, sc = torch.full((B, H, C), -1, device="cuda", dtype=torch.int32), torch.zeros(B, H, C, device="cuda")
    swa.swa_hh_cache_fill(kp, vp, si, kc, vc, sp, sc, S, recent)
    slot = torch.empty(B, H, device="cuda", dtype=torch.int32)
    o, l = torch.empty(B, Hq, d, device="cuda"), torch.empty(B, Hq, device="cuda")
    for p in range(L, L + steps):
        before, sb = sp.cpu().numpy(), sc.cpu().numpy()
        swa.swa_hh_cache_append(k[:, p].contiguous().cuda(), v[:, p].contiguous().cuda(),
                                torch.full((B,), p, dtype=torch.int32, device="cuda"), kc, vc, sp, sc, slot, S, recent)
        mid = sc.double().cpu().numpy()
        swa.swa_hh_decode(q[:, p].contiguous().cuda(), kc, vc, sp, sc, o, l)
        torch.cuda.synchronize()
        held = sp.cpu().numpy()
        for b in range(B):
            for h in range(H):
                assert int(slot[b, h]) == oracle.hh_victim(before[b, h], sb[b, h], p, S, recent)
                assert set(range(S)) <= set(held[b, h]) and set(range(p - recent + 1, p + 1)) <= set(held[b, h])
                assert torch.equal(kc[b, h].cpu(), k[b, held[b, h], h])
        wo, wl, ws = oracle.hh_decode(q[:, p], kc.cpu(), vc.cpu(), held, mid, scale)
        dz = dz_of(q.double(), k.double(), scale)
        assert np.abs(o.double().cpu().numpy() - wo).max() <= (2 * dz + 2.0 ** -16) * float(v.abs().max())
        assert np.abs(sc.double().cpu().numpy() - ws).max() <= 2 * (dz + 2.0 ** -19) * Hq + 2.0 ** -22 * ws.max()


def test_captured_and_on_two_streams():
    B, H, Hq, d, C = 3, 2, 8, 128, 400
    k, v, sp, s = cache(B, H, C, d, 13, 0.9)
    q = rand((B, Hq, d), 14).cuda()

    def fresh():
        return ([t.cuda() for t in (k, v)] + [torch.from_numpy(sp).cuda(), torch.from_numpy(s).cuda()],
                torch.zeros(B, Hq, d, device="cuda"), torch.zeros(B, Hq, device="cuda"))

    kn = rand((B, H, d), 15).cuda()
    pos = torch.full((B,), 5 * C, dtype=torch.int32, device="cuda")

    def step(st):
        c, out, lse = st
        swa.swa_hh_cache_append(kn, kn, pos, *c, None, 2, 8)
        swa.swa_hh_decode(q, *c, out, lse)

    want = fresh()
    for _ in range(3):
        step(want)
    a, b = fresh(), fresh()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(a)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        graph.replay()
        with torch.cuda.stream(side):
            step(b)
    torch.cuda.synchronize()
    for st in (a, b):
        for x, y in zip(st[0] + [st[1], st[2]], want[0] + [want[1], want[2]]):
            assert torch.equal(x, y)


def test_scores_wait_that_runs_out_is_reported_and_leaves_the_library_usable():
    """The load warp issues nothing (test hook): every wait ends at its limit, the status says so, and the next call
    works."""
    B, L, H, d = 1, 300, 2, 128
    q, k = rand((B, L, H, d), 1).cuda(), rand((B, L, H, d), 2).cuda()
    lse = torch.empty(B, H, L, device="cuda")
    swa.swa_fwd(q, k, k, torch.empty_like(q), lse, L, 0)
    want, got = torch.empty(B, H, L, device="cuda"), torch.empty(B, H, L, device="cuda")
    swa.swa_hh_scores(q, k, lse, want, L, L, 0)
    assert swa.swa_device_error() == 0
    old = swa.swa_set_wait_timeout_ns(2_000_000)
    swa.swa_set_debug_flags(1)
    try:
        swa.swa_hh_scores(q, k, lse, got, L, L, 0)
        assert swa.swa_device_error() == swa.SWA_ERR_DEVICE_TIMEOUT
    finally:
        swa.swa_set_debug_flags(0)
        swa.swa_set_wait_timeout_ns(old)
    swa.swa_hh_scores(q, k, lse, got, L, L, 0)
    assert swa.swa_device_error() == 0 and torch.equal(got, want)


def test_scores_captured_twice_and_replayed_in_turn():
    """Two graphs of the same call on different inputs share nothing."""
    B, L, H, d = 1, 260, 2, 64
    sets = []
    for s in (1, 5):
        q, k = rand((B, L, H, d), s).cuda(), rand((B, L, H, d), s + 1).cuda()
        lse, score = torch.empty(B, H, L, device="cuda"), torch.empty(B, H, L, device="cuda")
        swa.swa_fwd(q, k, k, torch.empty_like(q), lse, L, 0)
        swa.swa_hh_scores(q, k, lse, score, 100, L, 0)
        sets.append((q, k, lse, score, score.clone()))
    torch.cuda.synchronize()
    graphs = []
    for q, k, lse, score, _ in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            swa.swa_hh_scores(q, k, lse, score, 100, L, 0)
        graphs.append(g)
    for _ in range(3):
        for (_, _, _, score, _), g in zip(sets, graphs):
            score.zero_()
            g.replay()
    torch.cuda.synchronize()
    for _, _, _, score, want in sets:
        assert torch.equal(score, want)


def test_calls_on_a_stream_given_by_hand_and_without_sequences():
    st = torch.cuda.Stream()
    k, v, sp, s = cache(2, 2, 64, 64, 3, 1.0)
    args = [t.cuda() for t in (k, v)] + [torch.from_numpy(sp).cuda(), torch.from_numpy(s).cuda()]
    q = rand((2, 4, 64), 4).cuda()
    outs = [torch.zeros(2, 4, 64, device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    swa.swa_hh_decode(q, *args, outs[0], None, stream=st)
    st.synchronize()
    args[3].copy_(torch.from_numpy(s))
    swa.swa_hh_decode(q, *args, outs[1], None)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[1]) and float(outs[0].abs().sum()) > 0
    none = [t[:0] for t in args]
    swa.swa_hh_decode(q[:0], *none, outs[0][:0], None)
    swa.swa_hh_cache_append(k[:0, :, 0].contiguous().cuda(), v[:0, :, 0].contiguous().cuda(),
                            torch.zeros(0, dtype=torch.int32, device="cuda"), *none, None, 0, 1)
    torch.cuda.synchronize()


@pytest.mark.parametrize("C,d", [(1001, 128), (2045, 64)])
def test_fills_of_the_same_cache_one_after_another(C, d):
    """Capacities whose heads share sectors of slot_pos, filled again and again in place with other prompts, eagerly and
    in a graph: the copying kernel, which starts while the choice is still being written, takes the new positions."""
    B, H, L, S, recent = 4, 8, 5000, 3, 200
    sets = []
    for seed in range(3):
        k, s = rand((B, L, H, d), seed).cuda(), torch.rand(B, H, L, generator=torch.Generator().manual_seed(seed)).cuda()
        always = (torch.arange(L, device="cuda") < S) | (torch.arange(L, device="cuda") >= L - recent)
        keep = s.masked_fill(always, 2.0).sort(dim=-1, descending=True, stable=True)[1][..., :C].sort(-1)[0]
        at = keep.transpose(1, 2)[..., None].expand(-1, -1, -1, d)
        sets.append((k, -k, s, keep.int(), k.gather(1, at).transpose(1, 2)))
    kc, vc = (torch.zeros(B, H, C, d, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    sp = torch.full((B, H, C), L - 1, device="cuda", dtype=torch.int32)  # valid, and wrong
    score = torch.zeros(B, H, C, device="cuda")
    k, v, s = (torch.empty_like(x) for x in sets[0][:3])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        swa.swa_hh_cache_fill(k, v, s, kc, vc, sp, score, S, recent)
    for n in range(12):
        kn, vn, sn, keep, rows = sets[n % 3]
        if n % 2:
            for x, y in zip((k, v, s), (kn, vn, sn)):
                x.copy_(y)
            graph.replay()
        else:
            swa.swa_hh_cache_fill(kn, vn, sn, kc, vc, sp, score, S, recent)
        assert torch.equal(sp, keep), n
        assert torch.equal(kc, rows) and torch.equal(vc, -rows), n


def test_integers_that_do_not_fit_32_bits_are_refused():
    """ctypes would drop their upper bits: 2^32 + 1 would be 1.  A window of any size from L on means all keys."""
    k, v, sp, s = (t.cuda() for t in map(torch.as_tensor, cache(1, 2, 8, 64, 3, 1.0)))
    x, lse, big = rand((1, 4, 2, 64), 4).cuda(), torch.zeros(1, 2, 4, device="cuda"), 2 ** 32
    pos = torch.zeros(1, device="cuda", dtype=torch.int32)
    for f in (lambda: swa.swa_hh_scores(x, x, lse, lse.clone(), big + 1, 4, 0),
              lambda: swa.swa_hh_scores(x, x, lse, lse.clone(), 1, 4, big),
              lambda: swa.swa_hh_cache_fill(x, x, lse, k, v, sp, s, big, 1),
              lambda: swa.swa_hh_cache_fill(x, x, lse, k, v, sp, s, 0, big + 1),
              lambda: swa.swa_hh_cache_append(x[:, 0], x[:, 0], pos, k, v, sp, s, None, 0, -big + 1),
              lambda: swa.swa_hh_cache_append(x[:, 0], x[:, 0], pos, k, v, sp, s, None, big, 1),
              lambda: swa.swa_kv4_cache_append(x[:, 0], x[:, 0], pos, *[torch.zeros(1, 2, 8, 40, device="cuda",
                                               dtype=torch.uint8) for _ in range(2)], None, None, 8, -big),
              lambda: swa.swa_rope_axes_qk(x[0], None, pos.expand(1, 4).contiguous(), (big + 32,))):
        with pytest.raises(ValueError, match="32 bits"):
            f()
    scores = []
    for window in (4, 2 ** 31, big + 1, 2 ** 63 - 1):
        scores.append(torch.empty(1, 2, 4, device="cuda"))
        swa.swa_hh_scores(x, x, lse, scores[-1], 4, window, 0)
    torch.cuda.synchronize()
    assert all(torch.equal(scores[0], y) for y in scores[1:])


@pytest.mark.parametrize("L,n_obs", [(128, 128), (300, 200), (5000, 600)])
def test_scores_waits_of_a_nanosecond_leave_the_library_usable(L, n_obs):
    """With a time limit that any wait may exceed, whichever warp gives up first, while others are through with their
    lists or not: the call ends, reports it or does not, and the next call gives the same bits as ever."""
    B, H, G, d = 2, 2, 2, 128
    q, k = rand((B, L, H * G, d), 1).cuda(), rand((B, L, H, d), 2).cuda()
    lse = torch.empty(B, H * G, L, device="cuda")
    swa.swa_fwd(q, k, k, torch.empty_like(q), lse, L, 0)
    want, got = torch.empty(B, H, L, device="cuda"), torch.empty(B, H, L, device="cuda")
    swa.swa_hh_scores(q, k, lse, want, n_obs, L, 0)
    assert swa.swa_device_error() == 0
    for _ in range(5):
        old = swa.swa_set_wait_timeout_ns(1)
        try:
            swa.swa_hh_scores(q, k, lse, got, n_obs, L, 0)
            assert swa.swa_device_error() in (0, swa.SWA_ERR_DEVICE_TIMEOUT)
        finally:
            swa.swa_set_wait_timeout_ns(old)
        swa.swa_hh_scores(q, k, lse, got, n_obs, L, 0)
        assert swa.swa_device_error() == 0 and torch.equal(got, want)


@pytest.mark.parametrize("d", [64, 128])
def test_scores_of_log_sum_exps_from_elsewhere(d):
    """Sums too small for the logits (another window, another scale): every column gives 2^x as far as a float goes, and
    an infinity beyond; a NaN stays one.  One query at a time has weight, on all the ways a column can take."""
    B, H, L, n_obs = 1, 1, 256, 8
    q, k = torch.zeros(B, L, H, d).bfloat16().cuda(), rand((B, L, H, d), 1).cuda()
    for x in (-100.0, 0.0, 100.0, 119.3, 121.0, 125.0, 127.25, 128.25, 130.0, 256.0, 300.5, 1e4, math.inf, math.nan):
        for t in range(L - n_obs, L):
            lse = torch.full((B, H, L), 150 * math.log(2), device="cuda")
            lse[..., t] = -x * math.log(2)
            score = torch.empty(B, H, L, device="cuda")
            swa.swa_hh_scores(q, k, lse, score, n_obs, L, 0)
            got = score[0, 0, :L - n_obs].double().cpu().numpy()
            # x in the kernel: the float32 log-sum-exp (2^-24 of it) times log2(e), rounded again
            want = math.nan if x != x else math.inf if x > 128 else 2.0 ** x
            if x != x or x > 128:
                np.testing.assert_array_equal(got, want)
            else:  # and seven columns of 2^-126 at most
                assert (np.abs(got - want) <= (abs(x) * 2.0 ** -22 + 2.0 ** -20) * want + 8 * 2.0 ** -126).all(), (x, t)
    assert swa.swa_device_error() == 0


@pytest.mark.parametrize("B,H,L,C,d", [(20, 8, 2500, 1601, 128), (10, 16, 30001, 3203, 64), (32, 8, 3000, 700, 128)])
def test_fills_of_more_heads_than_the_gpu_takes_at_once(B, H, L, C, d):
    """A block for every SM and more, few and many rows a head: copied by the choosing block or by a kernel of its own."""
    S, recent = 4, 100
    g = torch.Generator(device="cuda").manual_seed(1)
    k = torch.randn(B, L, H, d, device="cuda", generator=g).bfloat16()
    s = torch.rand(B, H, L, device="cuda", generator=g)
    kc, vc = (torch.zeros(B, H, C, d, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    sp, score = torch.full((B, H, C), L - 1, device="cuda", dtype=torch.int32), torch.zeros(B, H, C, device="cuda")
    swa.swa_hh_cache_fill(k, -k, s, kc, vc, sp, score, S, recent)
    at = torch.arange(L, device="cuda")
    rank = s.masked_fill((at < S) | (at >= L - recent), 2.0)
    keep = rank.sort(dim=-1, descending=True, stable=True)[1][..., :C].sort(-1)[0]
    assert torch.equal(sp, keep.int()) and torch.equal(score, s.gather(-1, keep))
    rows = k.gather(1, keep.transpose(1, 2)[..., None].expand(-1, -1, -1, d)).transpose(1, 2)
    assert torch.equal(kc, rows) and torch.equal(vc, -rows)
