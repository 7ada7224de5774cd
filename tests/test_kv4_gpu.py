"""4-bit ring cache on the GPU (through the C ABI) against the fp64 oracle: packed rows bit for bit, values
read back, the decode step, and a run of prompt, appends and decodes.

Tolerances of the decode.  The kernel rounds p * step to fp16 (relative 2^-11 of the value with truncation and
the fp16 product's rounding together; finfo(float16).eps / 2 = 2^-11), and a code is at most 15, so that an output
moves by at most 2^-11 * max(15 step).  A score is a float32 sum of d products of magnitude sum |q||k| scale: at most
(d + 16) 2^-24 of that (and 2^-20 to allow for the matrix unit's own alignment), and an output moves by twice the
score's error times max |v|, a log-sum-exp by once.  A bf16 output is rounded by at most half a step, 2^-8."""
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


class Cache:
    def __init__(self, B, H, d, W, S, fill=0):
        row = swa.swa_kv4_row_bytes(d)
        self.kc, self.vc = (torch.full((B, H, W, row), fill, dtype=torch.uint8, device="cuda") for _ in range(2))
        self.sk, self.sv = (torch.full((B, H, S, row), fill, dtype=torch.uint8, device="cuda") for _ in range(2))
        self.W, self.S = W, S

    def args(self):
        return self.kc, self.vc, self.sk, self.sv


def bounds(q, k, v, scale, seen):
    """Largest allowed error of an output (before its rounding) and of a log-sum-exp; k, v [n, d] values."""
    k, v = k[seen], v[seen]
    size = scale * (np.abs(q) @ np.abs(k).T).max()
    dz = size * ((q.shape[-1] + 16) * 2.0 ** -24 + 2.0 ** -20) + 2.0 ** -21
    span = max(float(oracle.kv4_quantise(v)[1].max()) * 15, 0.0)
    return 2.0 ** -11 * span + 2 * dz * np.abs(v).max() + 1e-30, dz + 4e-7 * 40


def check_decode(c, q, pos, kval, vval, scale=None, f32=True):
    """Decode and compare; kval, vval [B, H, W + S, d] are the values in the slots."""
    B, Hq, d = q.shape
    H = kval.shape[1]
    out = torch.full((B, Hq, d), 7.0, device="cuda", dtype=torch.float32 if f32 else torch.bfloat16)
    lse = torch.full((B, Hq), 7.0, device="cuda")
    swa.swa_kv4_decode(q.cuda(), *c.args(), torch.tensor(pos, dtype=torch.int32, device="cuda"), out, lse, c.W, c.S,
                       scale)
    torch.cuda.synchronize()
    scale = scale or 1 / math.sqrt(d)
    got, gl, q64 = out.double().cpu().numpy(), lse.double().cpu().numpy(), q.double().numpy()
    for b in range(B):
        p = int(pos[b])
        i = np.arange(c.W + c.S)
        seen = np.where(i < c.W, i < min(p + 1, c.W), i - c.W < min(c.S, max(0, p - c.W + 1)))
        for h in range(Hq):
            kv = h // (Hq // H)
            if not seen.any():
                assert (got[b, h] == 0).all() and gl[b, h] == -np.inf
                continue
            z = scale * kval[b, kv][seen] @ q64[b, h]
            e = np.exp(z - z.max())
            want, wl = e @ vval[b, kv][seen] / e.sum(), z.max() + np.log(e.sum())
            tol, tl = bounds(q64[b, h], kval[b, kv], vval[b, kv], scale, seen)
            tol = tol + (0 if f32 else 2.0 ** -8 * np.abs(want))
            assert (np.abs(got[b, h] - want) <= tol).all(), (b, h, np.abs(got[b, h] - want).max(), tol)
            assert abs(gl[b, h] - wl) <= tl, (b, h, gl[b, h], wl)


def slots(kval, B, H, W, S, d, seed, scale=1.0):
    return rand((B, H, W, d), seed, scale), rand((B, H, S, d), seed + 1, scale)


def filled(B, H, d, W, S, seed, scale=1.0):
    """A cache whose every slot holds something, and the values."""
    c = Cache(B, H, d, W, S)
    vals = []
    for ring, sink, s in ((c.kc, c.sk, seed), (c.vc, c.sv, seed + 10)):
        r, k = rand((B, H, W, d), s, scale), rand((B, H, S, d), s + 1, scale)
        ring.copy_(torch.from_numpy(oracle.kv4_pack(r)))
        if S:
            sink.copy_(torch.from_numpy(oracle.kv4_pack(k)))
        vals.append(np.concatenate([oracle.kv4_values(r), oracle.kv4_values(k)], 2))
    return c, vals[0], vals[1]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("P,W,S", [(1, 1, 0), (5, 8, 3), (8, 8, 8), (9, 8, 4), (200, 64, 4), (70, 64, 70), (33, 7, 0)])
def test_fill_is_bit_exact(d, P, W, S):
    B, H = 2, 3
    k, v = rand((B, P, H, d), P + d), rand((B, P, H, d), P + d + 1)
    c = Cache(B, H, d, W, S, fill=171)
    swa.swa_kv4_cache_fill(k.cuda(), v.cuda(), *c.args(), W, S)
    torch.cuda.synchronize()
    for x, ring, sink in ((k, c.kc, c.sk), (v, c.vc, c.sv)):
        rows = oracle.kv4_pack(x)
        want_ring = np.full((B, H, W, rows.shape[-1]), 171, dtype=np.uint8)
        want_sink = np.full((B, H, S, rows.shape[-1]), 171, dtype=np.uint8)
        for p in range(max(0, P - W), P):
            want_ring[:, :, p % W] = rows[:, p]
        for p in range(min(P, S)):
            want_sink[:, :, p] = rows[:, p]
        np.testing.assert_array_equal(ring.cpu().numpy(), want_ring)
        np.testing.assert_array_equal(sink.cpu().numpy(), want_sink)


@pytest.mark.parametrize("d", [64, 128])
def test_groups_of_every_kind_are_quantised_as_defined(d):
    """Constant groups, zeros, tiny and large values, one outlier, and values that lie on a rounding border."""
    B, H, P = 1, 1, 64
    x = rand((B, P, H, d), 5).float()
    x[0, 0] = 0
    x[0, 1] = 2.5
    x[0, 2] = -3
    x[0, 3] *= 1e-30
    x[0, 4] *= 1e30
    x[0, 5] *= 1e-38  # steps below 2^-126
    x[0, 6, 0, 7] = 1000
    x[0, 7, 0, :] = torch.arange(d) % 32  # 31 / 15 steps
    x[0, 8, 0, :] = (torch.arange(d) % 31).float() / 2  # step 1: halves are borders
    x[0, 9, 0, ::2] = -0.0
    k = x.bfloat16()
    c = Cache(B, H, d, P, 0)
    swa.swa_kv4_cache_fill(k.cuda(), (-k).cuda(), *c.args(), P, 0)
    out = [torch.empty(B, P, H, d, device="cuda") for _ in range(2)]
    swa.swa_kv4_cache_read(torch.arange(P, dtype=torch.int32, device="cuda")[None], *c.args(), *out, P, 0)
    torch.cuda.synchronize()
    for got, src in zip(out, (k, -k)):
        # one float32 rounding of code * step + lo
        np.testing.assert_array_equal(got.cpu().numpy(), oracle.kv4_values(src).astype(np.float32))


@pytest.mark.parametrize("d", [64, 128])
def test_append_and_read_back(d):
    B, H, W, S = 4, 2, 6, 3
    c = Cache(B, H, d, W, S)
    held = {}
    for step in range(20):
        pos = [step, step + 5, -1 if step % 3 == 0 else step, 2 ** 31 - 30 + step]
        k, v = rand((B, H, d), step), rand((B, H, d), 100 + step)
        swa.swa_kv4_cache_append(k.cuda(), v.cuda(), torch.tensor(pos, dtype=torch.int32, device="cuda"), *c.args(),
                                 W, S)
        for b, p in enumerate(pos):
            if p >= 0:
                held[b, p] = (oracle.kv4_values(k[b]), oracle.kv4_values(v[b]))
    ask = torch.full((B, 8), -1, dtype=torch.int32)
    ask[0, :6] = torch.arange(14, 20)
    ask[0, 6:] = torch.tensor([0, 2])
    ask[1, 0] = 24
    ask[2, 0] = 19
    ask[3, 1] = 2 ** 31 - 11
    for dt in (torch.float32, torch.bfloat16):
        ko, vo = (torch.full((B, 8, H, d), 9.0, device="cuda", dtype=dt) for _ in range(2))
        swa.swa_kv4_cache_read(ask.cuda(), *c.args(), ko, vo, W, S)
        torch.cuda.synchronize()
        for b in range(B):
            for i in range(8):
                p = int(ask[b, i])
                want = held[b, p] if p >= 0 else (np.zeros((H, d)),) * 2
                for got, w in zip((ko, vo), want):
                    w = torch.from_numpy(w).float().to(dt)
                    assert torch.equal(got[b, i].cpu(), w), (b, i)


@pytest.mark.parametrize("d,Hq,H", [(64, 2, 2), (64, 8, 1), (128, 8, 2), (128, 7, 1), (128, 3, 3), (64, 12, 4)])
@pytest.mark.parametrize("W,S", [(1, 0), (15, 1), (16, 16), (130, 4), (700, 20)])
def test_decode_matches_oracle(d, Hq, H, W, S):
    B = 5
    c, kv, vv = filled(B, H, d, W, S, W + d)
    pos = [W + S + 3, 0, W - 1, W, -1]
    check_decode(c, rand((B, Hq, d), 3), pos, kv, vv)
    check_decode(c, rand((B, Hq, d), 4), pos, kv, vv, f32=False)


@pytest.mark.parametrize("B,W", [(1, 4096), (3, 20000), (40, 257)])
def test_decode_long_and_wide(B, W):
    """Every size of cluster."""
    c, kv, vv = filled(B, 2, 128, W, 4, 11)
    check_decode(c, rand((B, 8, 128), 12), [2 * W] * (B - 1) + [W // 2], kv, vv)


@pytest.mark.parametrize("qs,ks,vs", [(1e-12, 1, 1), (1, 1e-20, 1e-20), (1e4, 1e-4, 1e6), (8, 8, 1e15), (0, 1, 1)])
def test_decode_over_the_range_of_values(qs, ks, vs):
    """Magnitudes far from 1, large scores (one key takes all), zero queries, and steps that differ by 2^40 within
    one cache: the keys' order is turned so that the largest come first for one head and last for the other."""
    B, H, d, W = 2, 2, 128, 200
    c, kv, vv = filled(B, H, d, W, 0, 21)
    k = rand((B, H, W, d), 22, ks)
    v = rand((B, H, W, d), 23, vs).float()
    v[:, 0, 50:] *= 2.0 ** -20
    v[:, 1, :150] *= 2.0 ** -20
    v = v.bfloat16()
    c.kc.copy_(torch.from_numpy(oracle.kv4_pack(k)))
    c.vc.copy_(torch.from_numpy(oracle.kv4_pack(v)))
    check_decode(c, rand((B, 4, d), 24, qs), [W, W // 3], oracle.kv4_values(k), oracle.kv4_values(v))


def test_slots_that_are_not_visible_are_not_read_into_the_result():
    """A ring that is not full: what lies behind the last position holds NaN parameters."""
    B, H, d, W, S = 1, 1, 128, 64, 4
    c, kv, vv = filled(B, H, d, W, S, 31)
    for t in (c.kc, c.vc):
        t[:, :, 20:] = 255  # bf16 0xffff is a NaN
    for t in (c.sk, c.sv):
        t[:] = 255
    check_decode(c, rand((B, 4, d), 32), [19], kv, vv)


def test_a_prompt_and_generated_tokens_in_turn():
    """Fill, then append and decode step by step, against attention over the quantised history."""
    B, P, steps, H, Hq, d, W, S = 2, 90, 30, 2, 4, 64, 50, 3
    c = Cache(B, H, d, W, S)
    hist = [rand((B, P + steps, H, d), s) for s in (41, 42)]
    swa.swa_kv4_cache_fill(hist[0][:, :P].contiguous().cuda(), hist[1][:, :P].contiguous().cuda(), *c.args(), W, S)
    vals = [oracle.kv4_values(x) for x in hist]
    for p in range(P, P + steps):
        pos = torch.full((B,), p, dtype=torch.int32, device="cuda")
        swa.swa_kv4_cache_append(hist[0][:, p].contiguous().cuda(), hist[1][:, p].contiguous().cuda(), pos, *c.args(),
                                 W, S)
        q = rand((B, Hq, d), p)
        out, lse = torch.empty(B, Hq, d, device="cuda"), torch.empty(B, Hq, device="cuda")
        swa.swa_kv4_decode(q.cuda(), *c.args(), pos, out, lse, W, S)
        seen = oracle.visible_mask(p + 1, W, S)[p]
        for b in range(B):
            for h in range(Hq):
                k, v = vals[0][b, :p + 1, h // 2], vals[1][b, :p + 1, h // 2]
                z = k[seen] @ q[b, h].double().numpy() / math.sqrt(d)
                e = np.exp(z - z.max())
                tol, tl = bounds(q[b, h].double().numpy(), k, v, 1 / math.sqrt(d), seen)
                assert np.abs(out[b, h].double().cpu().numpy() - e @ v[seen] / e.sum()).max() <= tol
                assert abs(float(lse[b, h]) - z.max() - np.log(e.sum())) <= tl


def test_captured_and_on_two_streams():
    """A captured step replayed with new inputs, while another stream decodes from another cache; results as alone."""
    B, H, Hq, d, W, S = 3, 2, 8, 128, 300, 4
    ca, _, _ = filled(B, H, d, W, S, 51)
    cb, _, _ = filled(B, H, d, W, S, 61)
    q = rand((B, Hq, d), 52).cuda()
    pos = torch.tensor([400, 20, 299], dtype=torch.int32, device="cuda")
    kn, vn = rand((B, H, d), 53).cuda(), rand((B, H, d), 54).cuda()

    def step(c, out, lse):
        swa.swa_kv4_cache_append(kn, vn, pos, *c.args(), W, S)
        swa.swa_kv4_decode(q, *c.args(), pos, out, lse, W, S)

    alone = []
    for c in (ca, cb):
        out, lse = torch.empty(B, Hq, d, device="cuda", dtype=torch.bfloat16), torch.empty(B, Hq, device="cuda")
        step(c, out, lse)
        alone.append((out, lse))
    torch.cuda.synchronize()
    out, lse = torch.zeros_like(alone[0][0]), torch.zeros_like(alone[0][1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(ca, out, lse)
    side = torch.cuda.Stream()
    ob, lb = torch.zeros_like(out), torch.zeros_like(lse)
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        graph.replay()
        with torch.cuda.stream(side):
            step(cb, ob, lb)
    torch.cuda.synchronize()
    assert torch.equal(out, alone[0][0]) and torch.equal(lse, alone[0][1])
    assert torch.equal(ob, alone[1][0]) and torch.equal(lb, alone[1][1])


def test_many_sequences_and_repeated_calls_agree_bit_for_bit():
    """A decode's sums are taken in an order that the sizes give: the same call gives the same bits."""
    B, H, Hq, d, W, S = 70, 3, 6, 64, 90, 2
    c, kv, vv = filled(B, H, d, W, S, 71)
    q = rand((B, Hq, d), 72)
    check_decode(c, q, [(37 * b) % 200 for b in range(B)], kv, vv)
    pos = torch.tensor([(37 * b) % 200 for b in range(B)], dtype=torch.int32, device="cuda")
    outs = [torch.empty(B, Hq, d, device="cuda") for _ in range(3)]
    for o in outs:
        swa.swa_kv4_decode(q.cuda(), *c.args(), pos, o, None, W, S)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


def test_constant_rows_of_any_size():
    """Groups of one value have step 0 and carry it in their minimum: the output is that value."""
    B, H, Hq, d, W = 1, 1, 8, 128, 40
    for value in (3.0, -1e9, 1e25, 0.0):
        c = Cache(B, H, d, W, 0)
        v = torch.full((B, W, H, d), value).bfloat16()
        swa.swa_kv4_cache_fill(rand((B, W, H, d), 1).cuda(), v.cuda(), *c.args(), W, 0)
        out = torch.empty(B, Hq, d, device="cuda")
        swa.swa_kv4_decode(rand((B, Hq, d), 2).cuda(), *c.args(), torch.full((1,), W - 1, dtype=torch.int32,
                                                                            device="cuda"), out, None, W, 0)
        want = float(v[0, 0, 0, 0])
        # the two bf16 parts of the softmax numerators leave 2^-16, the sums 40 * 2^-24
        assert float((out - want).abs().max()) <= (2.0 ** -16 + 40 * 2.0 ** -24 + 2.0 ** -20) * abs(want)


def test_a_prompt_that_fills_the_ring_many_times_over_and_a_wide_batch():
    """More sequences than blocks in z, and positions that wrap the ring several times."""
    B, P, H, d, W, S = 300, 23, 1, 64, 5, 2
    k, v = rand((B, P, H, d), 81), rand((B, P, H, d), 82)
    c = Cache(B, H, d, W, S)
    swa.swa_kv4_cache_fill(k.cuda(), v.cuda(), *c.args(), W, S)
    torch.cuda.synchronize()
    rows = oracle.kv4_pack(k)
    for p in range(P - W, P):
        np.testing.assert_array_equal(c.kc[:, :, p % W].cpu().numpy(), rows[:, p])
    np.testing.assert_array_equal(c.sk.cpu().numpy()[:, 0], rows[:, :S, 0])


def test_captured_behind_copies_and_a_join_of_streams():
    """The decode may start before the kernel in front of it ends; behind a copy, a memset, an event of another stream
    or at a graph's very start there is none, and it has to wait for those all the same."""
    B, H, Hq, d, W, S = 2, 2, 8, 128, 500, 4
    c, _, _ = filled(B, H, d, W, S, 91)
    q = rand((B, Hq, d), 92).cuda()
    pos = torch.tensor([600, 77], dtype=torch.int32, device="cuda")
    want = torch.empty(B, Hq, d, device="cuda")
    swa.swa_kv4_decode(q, *c.args(), pos, want, None, W, S)
    torch.cuda.synchronize()
    qin, pin = torch.zeros_like(q), torch.zeros_like(pos)
    big, host = torch.zeros(64 << 20, device="cuda"), q.cpu().pin_memory()
    outs = [torch.zeros(B, Hq, d, device="cuda") for _ in range(4)]
    side = torch.cuda.Stream()

    def copied(out):
        qin.copy_(host, non_blocking=True)
        pin.copy_(pos)
        swa.swa_kv4_decode(qin, *c.args(), pin, out, None, W, S)

    def behind_a_kernel(out):
        big.add_(1.0)  # takes longer than a launch
        qin.copy_(q * 1.0)
        swa.swa_kv4_decode(qin, *c.args(), pos, out, None, W, S)

    def joined(out):
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            big.add_(1.0)
            qin.copy_(q * 1.0)
        pin.copy_(pos)
        torch.cuda.current_stream().wait_stream(side)
        swa.swa_kv4_decode(qin, *c.args(), pin, out, None, W, S)

    def alone(out):
        swa.swa_kv4_decode(q, *c.args(), pos, out, None, W, S)

    for f, out in zip((copied, behind_a_kernel, joined, alone), outs):
        f(out)  # eagerly
        torch.cuda.synchronize()
        assert torch.equal(out, want), f.__name__
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            f(out)
        for _ in range(3):
            qin.zero_()
            pin.zero_()
            out.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want), f.__name__


def check_parts(q, c, pos, kq, vq, coarse):
    """Decode and compare with weights and terms of each element in 64 bits; kq, vq = (codes, steps, minima) of the slots'
    rows, as kv4_quantise gives them.  coarse(weights, steps, sums of the code terms) is what the rounding of numerators times
    steps may move each element by."""
    B, Hq, d = q.shape
    H = vq[0].shape[1]
    out, lse = torch.full((B, Hq, d), 7.0, device="cuda"), torch.full((B, Hq), 7.0, device="cuda")
    swa.swa_kv4_decode(q.cuda(), *c.args(), torch.tensor(pos, dtype=torch.int32, device="cuda"), out, lse, c.W, c.S)
    torch.cuda.synchronize()
    got, gl, q64 = out.double().cpu().numpy(), lse.double().cpu().numpy(), q.double().numpy()
    for b in range(B):
        n = min(int(pos[b]) + 1, c.W)
        for h in range(Hq):
            kv = h // (Hq // H)
            kc, ks, kl = (x[b, kv, :n] for x in kq)
            vc, vs, vl = (x[b, kv, :n] for x in vq)
            k = kc * np.repeat(ks, 32, -1) + np.repeat(kl, 32, -1)
            z = k @ q64[b, h] / math.sqrt(d)
            w = np.exp(z - z.max())
            total = w.sum()
            w, wl = w / total, z.max() + np.log(total)
            step, low = np.repeat(vs, 32, -1), np.repeat(vl, 32, -1)
            want = w @ (vc * step + low)
            # sums of the terms' sizes: minima carry two bf16 parts (2^-16), the products of a warp's 16 keys each are
            # added up in float32 (2^-22 a step, n / 64 steps at least four warps apart, and the merge)
            minima, codes = w @ np.abs(low), w @ (vc * step)
            size = (np.abs(q64[b, h]) @ np.abs(k).T).max() / math.sqrt(d)
            dz = size * ((d + 16) * 2.0 ** -24 + 2.0 ** -20) + 2.0 ** -20
            tol = coarse(w, vs, codes) + 2.0 ** -16 * minima + (2 * dz + (n / 64 + 16) * 2.0 ** -22) * (minima + codes)
            assert (np.abs(got[b, h] - want) <= tol + 1e-36).all(), (b, h, (np.abs(got[b, h] - want) - tol).max())
            assert abs(gl[b, h] - wl) <= dz + 2.0 ** -22 * abs(wl) + 2.0 ** -18, (b, h, gl[b, h], wl)


def eleven_bits(w, vs, codes):
    """fp16 numerators with one reference for all groups: 2^-11 of the largest term."""
    return 2.0 ** -11 * 15 * float(vs.max())


def packed(k, v, W):
    """A cache of these rows [B, H, W, d], and their codes, steps and minima."""
    B, H, _, d = k.shape
    c = Cache(B, H, d, W, 0)
    c.kc.copy_(torch.from_numpy(oracle.kv4_pack(k)))
    c.vc.copy_(torch.from_numpy(oracle.kv4_pack(v)))
    return c, oracle.kv4_quantise(k), oracle.kv4_quantise(v)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,W", [(1, 64), (1, 128), (1, 256), (2, 4096), (150, 300)])
@pytest.mark.parametrize("large", [1e12, 1e15, -1e25])
def test_keys_without_values_count_beside_keys_of_large_ones(d, B, W, large):
    """Half of the rows of V are zero, in front for one KV head and behind for the other, so that whole tiles, and with
    few tiles whole warps, see nothing else; logits are near each other, so that every key has its share of the sum."""
    H = 2
    k, v = rand((B, H, W, d), 1, 0.05), rand((B, H, W, d), 2).float() * large
    if large < 0:
        v = torch.full((B, H, W, d), large)  # groups of one value: no steps
    v[:, 0, :W // 2] = 0
    v[:, 1, W // 2:] = 0
    c, kq, vq = packed(k, v.bfloat16(), W)
    check_parts(rand((B, 2 * H, d), 3), c, [W - 1] * B, kq, vq, eleven_bits)


def sixteen_bits(w, vs, codes):
    """Numerators in two bf16 parts (2^-18) times steps in two again (2^-17): of each term, wherever the largest is."""
    return 1.5 * 2.0 ** -17 * codes


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,W", [(1, 40), (2, 700), (150, 130)])
@pytest.mark.parametrize("power", [-20, 0, 16, 20, 30, 40])
def test_groups_of_small_steps_beside_one_of_large_ones(d, B, W, power):
    """One group of V lies 2^power above the others, under a peaked softmax: every group keeps its own bits."""
    H = 2
    k, v = rand((B, H, W, d), 1), rand((B, H, W, d), 2).float()
    v[..., 32:64] *= 2.0 ** power
    c, kq, vq = packed(k, v.bfloat16(), W)
    check_parts(rand((B, 4 * H, d), 3, 3.0), c, [W - 1] * B, kq, vq, sixteen_bits)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("W", [32, 200, 3000])
@pytest.mark.parametrize("at", [0, -1])
def test_a_large_value_of_negligible_weight_takes_no_bits_from_the_others(d, W, at):
    """One key, in front or behind, with V 2^40 above the others and a weight of about 2^-40 or 2^-60 of theirs."""
    B, H, G = 2, 2, 4
    side = torch.sign(rand((H, 1, d), 5).float())
    k, v = rand((B, H, W, d), 1, 0.1).float(), rand((B, H, W, d), 2).float()
    power = torch.tensor([40.0, 60.0]).view(1, H, 1)
    k[:, :, at] = (-side * power[..., None] * math.log(2) / math.sqrt(d)).squeeze(2)
    v[:, :, at] *= 2.0 ** 40
    q = (side + 0.1 * rand((B, H, G, d), 3).float()).flatten(1, 2).bfloat16()
    c, kq, vq = packed(k.bfloat16(), v.bfloat16(), W)
    check_parts(q, c, [W - 1] * B, kq, vq, sixteen_bits)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("scale", [1e-27, 1e-12, 1e12, 1e27])
def test_values_of_any_size_keep_sixteen_bits(d, scale):
    B, H, W = 2, 2, 500
    c, kq, vq = packed(rand((B, H, W, d), 1), (rand((B, H, W, d), 2).float() * scale).bfloat16(), W)
    check_parts(rand((B, 4 * H, d), 3), c, [W - 1, 77], kq, vq, sixteen_bits)


def test_constant_rows_next_to_the_largest_that_fill_takes():
    """Values of 2^126: sums over keys, warps and blocks stay finite."""
    for B, W in ((1, 4096), (150, 100)):
        H, d = 2, 64
        v = torch.full((B, H, W, d), 2.0 ** 126)
        v[:, 1] *= -1
        c, kq, vq = packed(rand((B, H, W, d), 1, 0.1), v.bfloat16(), W)
        check_parts(rand((B, 2 * H, d), 3), c, [W - 1] * B, kq, vq, sixteen_bits)


def test_a_group_that_is_not_finite_keeps_to_itself():
    """Infinite or NaN parameters in one group of V: the other groups come out as without them, to the last bits."""
    B, H, Hq, d, W = 1, 2, 8, 128, 300
    k, v = rand((B, H, W, d), 1), rand((B, H, W, d), 2)
    q, pos = rand((B, Hq, d), 3).cuda(), torch.full((B,), W - 1, dtype=torch.int32, device="cuda")
    outs = []
    for word in (None, [0x80, 0x7f, 0x80, 0xff], [0xc0, 0x7f, 0xc0, 0x7f]):
        c, _, _ = packed(k, v, W)
        if word:
            c.vc[:, :, 40, d // 2 + 4:d // 2 + 8] = torch.tensor(word, dtype=torch.uint8, device="cuda")
        outs.append(torch.empty(B, Hq, d, device="cuda"))
        swa.swa_kv4_decode(q, *c.args(), pos, outs[-1], None, W, 0)
    torch.cuda.synchronize()
    rest = torch.arange(d) // 32 != 1
    for out in outs[1:]:
        assert not torch.isfinite(out[..., 32:64]).any()
        assert float((out - outs[0])[..., rest].abs().max()) <= 2.0 ** -20 * float(outs[0].abs().max())


@pytest.mark.parametrize("d", [64, 128])
def test_reads_behind_fills_of_the_same_cache(d):
    """Filled again and again in place with other prompts and read at once, eagerly and in a graph: the read, which starts
    while the fill still writes, takes the new rows, and the new positions of a copy."""
    B, P, H, W, S = 4, 3001, 3, 2500, 5
    c = Cache(B, H, d, W, S)
    first = torch.arange(P - W, P, dtype=torch.int32).expand(B, -1).contiguous().cuda()
    asks = [first, first.flip(1).contiguous()]
    prompts = [rand((B, P, H, d), n).cuda() for n in range(3)]
    want = [torch.from_numpy(oracle.kv4_values(x.cpu())).float().cuda()[:, P - W:] for x in prompts]
    k, ask = torch.empty_like(prompts[0]), torch.empty_like(first)
    ko, vo = (torch.zeros(B, W, H, d, device="cuda") for _ in range(2))

    def both(x, at):
        swa.swa_kv4_cache_fill(x, x, *c.args(), W, S)
        swa.swa_kv4_cache_read(at, *c.args(), ko, vo, W, S)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both(k, ask)
    for n in range(12):
        x, at = prompts[n % 3], asks[n // 2 % 2]
        if n % 2:
            k.copy_(x)
            ask.copy_(at)
            graph.replay()
        else:
            both(x, at)
        w = want[n % 3] if n // 2 % 2 == 0 else want[n % 3].flip(1)
        assert torch.equal(ko, w) and torch.equal(vo, w), n


@pytest.mark.parametrize("S", [0, 3])
def test_calls_without_sequences(S):
    c = Cache(2, 2, 64, 9, S)
    none = [t[:0] for t in c.args()] if S else [c.kc[:0], c.vc[:0], None, None]
    k, pos = rand((2, 4, 2, 64), 1).cuda(), torch.zeros(2, device="cuda", dtype=torch.int32)
    swa.swa_kv4_cache_fill(k[:0], k[:0], *none, 9, S)
    swa.swa_kv4_cache_append(k[:0, 0], k[:0, 0], pos[:0], *none, 9, S)
    swa.swa_kv4_cache_read(pos[:0, None], *none, k[:0, :1], k[:0, :1], 9, S)
    swa.swa_kv4_decode(k[:0, 0], *none, pos[:0], k[:0, 0], None, 9, S)
    torch.cuda.synchronize()


def test_missing_tensors_are_refused_by_name():
    c = Cache(1, 2, 64, 9, 3)
    k, pos = rand((1, 2, 64), 1).cuda(), torch.zeros(1, device="cuda", dtype=torch.int32)
    for sinks in ((None, None), (c.sk, None), (None, c.sv)):
        for f in (lambda: swa.swa_kv4_cache_fill(k[None], k[None], c.kc, c.vc, *sinks, 9, 3),
                  lambda: swa.swa_kv4_cache_append(k, k, pos, c.kc, c.vc, *sinks, 9, 3),
                  lambda: swa.swa_kv4_cache_read(pos[None], c.kc, c.vc, *sinks, k[None], k[None], 9, 3),
                  lambda: swa.swa_kv4_decode(k, c.kc, c.vc, *sinks, pos, k, None, 9, 3)):
            with pytest.raises(ValueError, match="sink_k" if sinks[0] is None else "sink_v"):
                f()
    with pytest.raises(ValueError, match="pos"):
        swa.swa_kv4_cache_append(k, k, None, c.kc, c.vc, c.sk, c.sv, 9, 3)
    with pytest.raises(ValueError, match="v_new"):
        swa.swa_kv4_cache_append(k, None, pos, c.kc, c.vc, c.sk, c.sv, 9, 3)


@pytest.mark.parametrize("G", [1, 3, 4, 5, 7, 8])
@pytest.mark.parametrize("d", [64, 128])
def test_numerators_keep_sixteen_bits_for_every_number_of_heads(G, d):
    """Up to four heads the numerators' low parts share a product with the high ones, with more they have their own."""
    B, H, W = 3, 2, 450
    k, v = rand((B, H, W, d), 1), rand((B, H, W, d), 2).float()
    v[..., :32] *= 2.0 ** 25
    v[:, 1, 100:300] *= 2.0 ** -30
    c, kq, vq = packed(k, v.bfloat16(), W)
    check_parts(rand((B, H * G, d), 3, 2.0), c, [W - 1, 31, 200], kq, vq, sixteen_bits)
