"""Rotary positions with several axes on the GPU (through the C ABI) against the oracle's complex rotation in fp64.

Tolerances: the angle is exact to fp64 and rounded to float32 in [-pi, pi] (2^-23 absolute), cosine and sine add two
float32 roundings, and the rotation three: below 2^-20 of the pair's length; a bf16 result is rounded by 2^-8."""
import numpy as np
import pytest
import torch

import oracle
import sink_aware_sliding_b200 as swa

pytestmark = pytest.mark.gpu


def rand(shape, seed, dtype):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g).to(dtype)


def positions(n, T, seed):
    g = torch.Generator().manual_seed(seed)
    p = torch.randint(0, 300000, (n, T), generator=g, dtype=torch.int32)
    p[:, :1] = 0
    p[0, -1] = 2 ** 31 - 1
    p[-1, T // 2] = -7
    return p


def check(got, want, dtype):
    d = want.shape[-1]
    pair = np.sqrt(want[..., :d // 2] ** 2 + want[..., d // 2:] ** 2)
    tol = 2.0 ** -20 * np.concatenate([pair, pair], -1)
    if dtype == torch.bfloat16:
        tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(want) + 1e-38
    err = np.abs(got.double().cpu().numpy() - want)
    assert (err <= tol).all(), (err - tol).max()


SECTIONS = {64: [(32,), (16, 16), (8, 12, 12), (2, 0, 30), (8, 8, 8, 8)],
            128: [(64,), (32, 32), (16, 24, 24), (24, 20, 20), (1, 0, 63), (16, 16, 16, 16), (40, 8, 8, 8)]}


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("layout", ["sections", "per_axis", "interleaved"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,Hq,H,inverse", [(1, 1, 1, False), (3, 8, 2, True), (37, 5, 5, False), (301, 7, 1, True)])
def test_matches_oracle(d, layout, dtype, T, Hq, H, inverse):
    for n, sec in enumerate(SECTIONS[d]):
        if layout == "interleaved" and any(a + len(sec) * (s - 1) >= d // 2 for a, s in enumerate(sec) if a and s):
            continue
        q, k, pos = rand((T, Hq, d), n, dtype), rand((T, H, d), n + 50, dtype), positions(len(sec), T, n)
        qd, kd = q.cuda(), k.cuda()
        swa.swa_rope_axes_qk(qd, kd, pos.cuda(), sec, layout=layout, inverse=inverse, rope_base=5e5)
        torch.cuda.synchronize()
        check(qd, oracle.rope_axes(q, pos.numpy(), sec, layout, 5e5, inverse), dtype)
        check(kd, oracle.rope_axes(k, pos.numpy(), sec, layout, 5e5, inverse), dtype)


@pytest.mark.parametrize("d", [64, 128])
def test_one_axis_is_the_plain_rotation(d):
    """Equal positions on all axes, or one axis: what swa_rope_qk computes, but for the sines' last bits."""
    T = 50
    q, p = rand((T, 4, d), 1, torch.bfloat16), positions(1, T, 2).clamp(min=0)
    want = q.cuda()
    swa.swa_rope_qk(want, None, p[0].cuda())
    for sec, layout in (((d // 2,), "sections"), ((d // 4, d // 4), "sections"), ((d // 4, d // 4), "interleaved")):
        got = q.cuda()
        swa.swa_rope_axes_qk(got, None, p.expand(len(sec), -1).contiguous().cuda(), sec, layout=layout)
        x, y = got.double().cpu().numpy(), want.double().cpu().numpy()
        assert (np.abs(x - y) <= 2.0 ** -7 * np.abs(y) + 1e-4).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_views_of_one_projection(dtype):
    """q and k inside one [T, (Hq + 2 H) d] output: only they turn."""
    T, Hq, H, d = 33, 4, 2, 128
    sec = (16, 24, 24)
    x, pos = rand((T, (Hq + 2 * H) * d), 3, dtype), positions(3, T, 4)
    xd = x.cuda()
    qv = xd[:, :Hq * d].unflatten(1, (Hq, d))
    kv = xd[:, Hq * d:(Hq + H) * d].unflatten(1, (H, d))
    swa.swa_rope_axes_qk(qv, kv, pos.cuda(), sec)
    torch.cuda.synchronize()
    got = xd.cpu()
    q, k = x[:, :Hq * d].reshape(T, Hq, d), x[:, Hq * d:(Hq + H) * d].reshape(T, H, d)
    check(got[:, :Hq * d].reshape(T, Hq, d), oracle.rope_axes(q, pos.numpy(), sec, "sections"), dtype)
    check(got[:, Hq * d:(Hq + H) * d].reshape(T, H, d), oracle.rope_axes(k, pos.numpy(), sec, "sections"), dtype)
    assert torch.equal(got[:, (Hq + H) * d:], x[:, (Hq + H) * d:])


@pytest.mark.parametrize("layout", ["sections", "per_axis", "interleaved"])
def test_inverse_is_the_gradient(layout):
    """The rotation is linear, y = R x: d(g . y)/dx = R^T g, by differences of g . R(x + h e) in fp64 on the oracle, and
    by the formula; and the inverse undoes the rotation."""
    T, H, d, sec = 4, 1, 64, (12, 10, 10)
    x, g, pos = rand((T, H, d), 5, torch.float32), rand((T, H, d), 6, torch.float32), positions(3, T, 7)
    got = g.cuda()
    swa.swa_rope_axes_qk(got, None, pos.cuda(), sec, layout=layout, inverse=True)
    grad = np.zeros((T, H, d))
    for i in range(d):
        h = np.zeros((T, H, d))
        h[..., i] = 0.5
        up, down = (oracle.rope_axes(x.double().numpy() + s * h, pos.numpy(), sec, layout) for s in (1, -1))
        grad[..., i] = (g.double().numpy() * (up - down)).sum(-1)
    check(got, oracle.rope_axes(g, pos.numpy(), sec, layout, inverse=True), torch.float32)
    assert np.abs(got.double().cpu().numpy() - grad).max() <= 2.0 ** -20 * np.sqrt(2) * float(g.abs().max())
    back = x.cuda()
    swa.swa_rope_axes_qk(back, None, pos.cuda(), sec, layout=layout)
    swa.swa_rope_axes_qk(back, None, pos.cuda(), sec, layout=layout, inverse=True)
    assert (back.cpu() - x).abs().max() <= 2.0 ** -18 * float(x.abs().max())


def test_gradients_through_rotation_and_attention():
    """Rotate, attend, swa_bwd, rotate the gradients back: against differences of the whole in fp64 along one direction."""
    B, L, H, d, W, S, sec = 1, 40, 2, 64, 16, 2, (8, 12, 12)
    q, k, v, do = (rand((L, H, d), s, torch.bfloat16) for s in (1, 2, 3, 4))
    pos = positions(3, L, 5)
    qr, kr = q.cuda(), k.cuda()
    swa.swa_rope_axes_qk(qr, kr, pos.cuda(), sec)
    out, lse = torch.empty(B, L, H, d, device="cuda", dtype=torch.bfloat16), torch.empty(B, H, L, device="cuda")
    swa.swa_fwd(qr[None], kr[None], v[None].cuda(), out, lse, W, S)
    dq, dk, dv = (torch.empty(B, L, H, d, device="cuda") for _ in range(3))
    swa.swa_bwd(qr[None], kr[None], v[None].cuda(), out, do[None].cuda(), lse, dq, dk, dv, W, S)
    swa.swa_rope_axes_qk(dq[0], dk[0], pos.cuda(), sec, inverse=True)
    torch.cuda.synchronize()
    wq, wk, _ = oracle.swa_bwd(oracle.rope_axes(q, pos.numpy(), sec, "sections")[None],
                               oracle.rope_axes(k, pos.numpy(), sec, "sections")[None], v[None], do[None], W, S, d ** -0.5)
    for got, want in ((dq, wq), (dk, wk)):
        want = oracle.rope_axes(want[0], pos.numpy(), sec, "sections", inverse=True)
        err = np.abs(got[0].double().cpu().numpy() - want)
        # the bounds of the backward pass (1e-2, mean 1e-3), and q, k rounded to bf16 once more after the rotation
        assert err.max() <= 2e-2 * max(1.0, np.abs(want).max()) and err.mean() <= 2e-3 * max(1.0, np.abs(want).mean())
