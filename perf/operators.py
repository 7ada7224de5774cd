"""Cases of the fixed-memory decoding operators: what is measured, in plain torch and through the library.

Four families, each with the cases a serving program meets:
  kv4_prompt  fill a 4-bit ring cache from a prompt, and read the kept positions back
  kv4_step    one generated token on a 4-bit ring cache: append, then attend
  hh_scores   attention weight that each prompt key received from the last queries
  hh_fill     keep a prompt's heaviest positions in a cache of fixed capacity
  hh_step     one generated token on that cache: evict and append, then attend and accumulate
  rope        rotary positions with several axes, in place, and its inverse for gradients
"""
import math

import torch

if torch.cuda.is_available():
    torch.backends.cuda.matmul.allow_tf32 = False

own = False  # False: `run` computes the plain forms; True: it calls the library

GROUP = 32  # elements of a row that share a scale and a minimum in the 4-bit cache


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # a short prompt in a small sliding-window layer: 300 tokens, more than two windows, odd sizes
        dict(name="kv4_prompt_short", kind="kv4_prompt", B=1, P=300, Hkv=2, d=64, W=129, S=3),
        # four long prompts of a grouped-query layer: the last 4096 positions and 4 sinks stay
        dict(name="kv4_prompt_long", kind="kv4_prompt", B=4, P=16384, Hkv=8, d=128, W=4096, S=4),
        # one sequence, one token: the latency a single user sees
        dict(name="kv4_step_single", kind="kv4_step", B=1, Hq=32, Hkv=8, d=128, W=4096, S=4, ragged=False),
        # a full serving batch past its window: the cache's bytes decide
        dict(name="kv4_step_batch64", kind="kv4_step", B=64, Hq=32, Hkv=8, d=128, W=4096, S=4, ragged=False),
        # many heads of their own (no sharing), short prompts, the last 64 queries observe
        dict(name="hh_scores_short", kind="hh_scores", B=2, L=2048, Hq=16, Hkv=16, d=64, W=2048, S=0, n_obs=64),
        # a long prompt of a grouped-query layer, the last 512 queries observe all of it
        dict(name="hh_scores_long", kind="hh_scores", B=1, L=32768, Hq=32, Hkv=8, d=128, W=32768, S=0, n_obs=512),
        # a prompt a little longer than the cache, odd sizes
        dict(name="hh_fill_short", kind="hh_fill", B=2, L=1000, Hkv=4, d=64, C=515, S=4, recent=128),
        # long prompts of a batch, an eighth is kept
        dict(name="hh_fill_long", kind="hh_fill", B=4, L=16384, Hkv=8, d=128, C=2048, S=4, recent=512),
        # one sequence, one token
        dict(name="hh_step_single", kind="hh_step", B=1, Hq=32, Hkv=8, d=128, C=2048, S=4, recent=512, fill=1.0),
        # a full serving batch on full caches
        dict(name="hh_step_batch64", kind="hh_step", B=64, Hq=32, Hkv=8, d=128, C=2048, S=4, recent=512, fill=1.0),
        # the next token of a batch: queries and keys turn by time, height and width, one launch's latency
        dict(name="rope_step", kind="rope", T=64, Hq=32, Hkv=8, d=128, axes=3, layout="interleaved", dtype="bf16",
             inverse=False),
        # a clip of 16 frames of 30 x 34 patches: gradients in float32 turn back
        dict(name="rope_clip_grad", kind="rope", T=16320, Hq=32, Hkv=8, d=128, axes=3, layout="sections", dtype="f32",
             inverse=True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["kv4_prompt", "kv4_step", "kv4_step", "hh_scores", "hh_fill", "hh_step", "hh_step", "rope"])
    d = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 3, 4, 5, 8])
    G = rng.choice([1, 2, 3, 4, 7, 8])
    B = _log_int(rng, 1, 64)
    if kind == "kv4_prompt":
        W = _log_int(rng, 1, 4096)
        c = dict(kind=kind, B=B, P=_log_int(rng, 1, 16384), Hkv=Hkv, d=d, W=W, S=rng.randint(0, 16))
        while c["B"] > 1 and c["B"] * c["P"] > 65536:
            c["B"] -= 1
        return c
    if kind == "kv4_step":
        c = dict(kind=kind, B=B, Hq=Hkv * G, Hkv=Hkv, d=d, W=_log_int(rng, 1, 16384), S=rng.randint(0, 40),
                 ragged=rng.random() < 0.5)
        while c["B"] > 1 and c["B"] * Hkv * c["W"] > 64 * 8 * 4096:
            c["B"] -= 1
        return c
    if kind == "hh_scores":
        L = _log_int(rng, 1, 16384)
        c = dict(kind=kind, B=rng.randint(1, 4), L=L, Hq=Hkv * G, Hkv=Hkv, d=d,
                 W=L if rng.random() < 0.5 else _log_int(rng, 1, L), S=rng.randint(0, 8),
                 n_obs=_log_int(rng, 1, min(L, 600)))
        while c["B"] > 1 and c["B"] * L * c["n_obs"] * c["Hq"] > 32768 * 512 * 32:
            c["B"] -= 1
        while c["n_obs"] > 1 and c["B"] * L * c["n_obs"] * c["Hq"] > 32768 * 512 * 32:
            c["n_obs"] //= 2
        return c
    if kind == "hh_fill":
        S, recent = rng.randint(0, 8), _log_int(rng, 1, 512)
        c = dict(kind=kind, B=B, L=_log_int(rng, 1, 16384), Hkv=Hkv, d=d, C=S + recent + _log_int(rng, 1, 2048), S=S,
                 recent=recent)
        while c["B"] > 1 and c["B"] * c["L"] > 65536:
            c["B"] -= 1
        return c
    if kind == "hh_step":
        S, recent = rng.randint(0, 8), _log_int(rng, 1, 512)
        c = dict(kind=kind, B=B, Hq=Hkv * G, Hkv=Hkv, d=d, C=S + recent + _log_int(rng, 1, 4096), S=S, recent=recent,
                 fill=rng.choice([1.0, 1.0, 0.9, 0.3]))
        while c["B"] > 1 and c["B"] * Hkv * c["C"] > 64 * 8 * 2048:
            c["B"] -= 1
        return c
    axes = rng.randint(1, 4)
    return dict(kind="rope", T=_log_int(rng, 1, 16000), Hq=Hkv * G, Hkv=Hkv, d=d, axes=axes,
                layout=rng.choice(["sections", "per_axis", "interleaved"]), dtype=rng.choice(["bf16", "f32"]),
                inverse=rng.random() < 0.5)


def _sections(c):
    """Pairs of each axis: the first axis a quarter or what is left, the others alike."""
    half, n = c["d"] // 2, c["axes"]
    if n == 1:
        return [half]
    rest = half // n if c["layout"] != "per_axis" else (3 * half // 4) // (n - 1)
    return [half - rest * (n - 1)] + [rest] * (n - 1)


# ------------------------------------------------------------------ the inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _row_bytes(d):
    return d // 2 + d // GROUP * 4


def prepare(case, seed):
    c, g = case, _gen(seed)
    kind, B, d = c["kind"], c.get("B"), c["d"]
    s = dict(case=c, kind=kind)
    dev = dict(device="cuda")
    if kind == "kv4_prompt":
        P, H, W, S = c["P"], c["Hkv"], c["W"], c["S"]
        s["k"], s["v"] = _randn(g, B, P, H, d), _randn(g, B, P, H, d)
        for n, rows in (("kc", W), ("vc", W), ("sk", S), ("sv", S)):
            s[n] = torch.zeros(B, H, rows, _row_bytes(d), dtype=torch.uint8, **dev)
        kept = list(range(min(S, max(0, P - W)))) + list(range(max(0, P - W), P))
        s["kept"] = torch.tensor(kept, dtype=torch.int32, **dev).expand(B, -1).contiguous()
        s["ko"] = torch.zeros(B, len(kept), H, d, dtype=torch.bfloat16, **dev)
        s["vo"] = torch.zeros_like(s["ko"])
    elif kind == "kv4_step":
        H, Hq, W, S = c["Hkv"], c["Hq"], c["W"], c["S"]
        for n, rows in (("kc", W), ("vc", W), ("sk", S), ("sv", S)):
            s[n] = torch.empty(B, H, rows, _row_bytes(d), dtype=torch.uint8, **dev)
            for b in range(B):
                s[n][b] = _pack4(_randn(g, H, rows, d))
        s["pos"] = torch.full((B,), W + S + 17, dtype=torch.int32, **dev)
        if c["ragged"]:
            s["pos"] = torch.randint(0, 2 * W + 2, (B,), generator=g, dtype=torch.int32, **dev)
        s["q"], s["kn"], s["vn"] = _randn(g, B, Hq, d), _randn(g, B, H, d), _randn(g, B, H, d)
        s["out"] = torch.zeros(B, Hq, d, dtype=torch.bfloat16, **dev)
        s["lse"] = torch.zeros(B, Hq, **dev)
    elif kind == "hh_scores":
        L, H, Hq = c["L"], c["Hkv"], c["Hq"]
        s["q"], s["k"] = _randn(g, B, L, Hq, d), _randn(g, B, L, H, d)
        s["lse"] = torch.zeros(B, Hq, L, **dev)
        for b in range(B):  # what the forward pass left for the queries that observe
            z = _obs_logits(s["q"][b:b + 1, L - c["n_obs"]:], s["k"][b:b + 1], c, torch.float32)
            s["lse"][b, :, L - c["n_obs"]:] = torch.logsumexp(z, -1).reshape(Hq, c["n_obs"])
        s["score"] = torch.zeros(B, H, L, **dev)
    elif kind == "hh_fill":
        L, H, C = c["L"], c["Hkv"], c["C"]
        s["k"], s["v"] = _randn(g, B, L, H, d), _randn(g, B, L, H, d)
        # accumulated weights: a few keys hold most of it
        s["score_in"] = torch.rand(B, H, L, generator=g, **dev).pow(8) * 4
        s["kc"] = torch.zeros(B, H, C, d, dtype=torch.bfloat16, **dev)
        s["vc"] = torch.zeros_like(s["kc"])
        s["slot_pos"] = torch.full((B, H, C), -1, dtype=torch.int32, **dev)
        s["score"] = torch.zeros(B, H, C, **dev)
    elif kind == "hh_step":
        H, Hq, C = c["Hkv"], c["Hq"], c["C"]
        s["kc"], s["vc"] = _randn(g, B, H, C, d), _randn(g, B, H, C, d)
        s["score"] = torch.rand(B, H, C, generator=g, **dev).pow(8) * 4
        n = max(1, int(c["fill"] * C))
        # the first positions, the last ones, and a choice of those between, in any order
        last = 4 * C
        mid = torch.rand(B, H, last - c["S"] - c["recent"], generator=g, **dev).argsort(-1)[..., :C] + c["S"]
        order = torch.cat([torch.arange(c["S"], **dev).expand(B, H, -1),
                           torch.arange(last - c["recent"] + 1, last, **dev).expand(B, H, -1), mid], -1)[..., :n]
        shuffle = torch.rand(B, H, C, generator=g, **dev).argsort(-1)
        full = torch.full((B, H, C), -1, dtype=torch.int64, **dev)
        full[..., :n] = order
        s["slot_pos"] = full.gather(-1, shuffle).to(torch.int32)
        s["score"] = torch.where(s["slot_pos"] >= 0, s["score"], torch.zeros_like(s["score"]))
        s["pos"] = torch.full((B,), last, dtype=torch.int32, **dev)
        s["q"], s["kn"], s["vn"] = _randn(g, B, Hq, d), _randn(g, B, H, d), _randn(g, B, H, d)
        s["out"] = torch.zeros(B, Hq, d, dtype=torch.bfloat16, **dev)
        s["lse"] = torch.zeros(B, Hq, **dev)
        s["slot"] = torch.zeros(B, H, dtype=torch.int32, **dev)
    else:
        T = c["T"]
        dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
        s["q"], s["k"] = _randn(g, T, c["Hq"], d, dtype=dt), _randn(g, T, c["Hkv"], d, dtype=dt)
        # axis 0: time, far into a stream; the others: places in a frame
        s["positions"] = torch.stack([
            torch.randint(0, 200000 if a == 0 else 64, (T,), generator=g, dtype=torch.int32, **dev)
            for a in range(c["axes"])])
        s["sections"] = _sections(c)
    return s


# ------------------------------------------------------------------ plain forms
def _quant4(x):
    """Codes, scales and minima of rows [..., d], by groups of 32 elements; every step rounds to 32 bits."""
    r = x.float().unflatten(-1, (-1, GROUP))
    lo, hi = r.amin(-1, keepdim=True), r.amax(-1, keepdim=True)
    scale = ((hi - lo) * torch.tensor(1 / 15, dtype=torch.float32, device=x.device)).bfloat16().float()
    scale = torch.where(scale >= 2.0 ** -126, scale, torch.zeros_like(scale))
    inv = torch.where(scale > 0, 1 / scale, torch.zeros_like(scale))
    return torch.round((r - lo) * inv).clamp(0, 15), scale, lo


def _pack4(x):
    """Rows [..., d] as the cache holds them: d/2 bytes of codes, then scale and minimum of each group in bf16."""
    code, scale, lo = _quant4(x)
    code = code.to(torch.uint8).unflatten(-1, (8, 4)).transpose(-3, -2).flatten(-3)
    pairs = code.unflatten(-1, (-1, 2))
    par = torch.cat([scale, lo], -1).bfloat16().flatten(-2).contiguous().view(torch.uint8)
    return torch.cat([pairs[..., 0] | (pairs[..., 1] << 4), par], -1)


def _unpack4(rows, d, dtype=torch.float32):
    """The values that packed rows [..., row_bytes] stand for."""
    raw, par = rows[..., :d // 2], rows[..., d // 2:].contiguous().view(torch.bfloat16).to(dtype)
    code = torch.stack([raw & 15, raw >> 4], -1).flatten(-2)
    code = code.unflatten(-1, (8, d // GROUP, 4)).transpose(-3, -2).flatten(-2).to(dtype)
    par = par.unflatten(-1, (-1, 2))
    return (code * par[..., :1] + par[..., 1:]).flatten(-2)


def _plain_kv4_prompt(s):
    c = s["case"]
    P, W, S, d = c["P"], c["W"], c["S"], c["d"]
    first, n_sink = max(0, P - W), min(S, P)
    slots = torch.arange(first, P, device="cuda") % W
    for x, ring, sink, out in (("k", "kc", "sk", "ko"), ("v", "vc", "sv", "vo")):
        rows = s[x].transpose(1, 2)
        s[ring][:, :, slots] = _pack4(rows[:, :, first:])
        s[sink][:, :, :n_sink] = _pack4(rows[:, :, :n_sink])
        p = s["kept"][0].long()
        got = torch.cat([s[sink][:, :, p[p < S]], s[ring][:, :, p[p >= S] % W]], 2)
        s[out].copy_(_unpack4(got, d).transpose(1, 2))
    return s["ko"], s["vo"]


def _write_row(ring, sink, row, pos, W, S):
    b = torch.arange(row.shape[0], device="cuda")
    ring[b, :, pos % W] = row
    if S:
        at = pos.clamp(max=S - 1)
        sink[b, :, at] = torch.where((pos < S)[:, None, None], row, sink[b, :, at])


def _plain_kv4_step(s):
    c = s["case"]
    W, S, d, H = c["W"], c["S"], c["d"], c["Hkv"]
    pos = s["pos"].long()
    _write_row(s["kc"], s["sk"], _pack4(s["kn"]), pos, W, S)
    _write_row(s["vc"], s["sv"], _pack4(s["vn"]), pos, W, S)
    i = torch.arange(W + S, device="cuda")
    n_ring, n_sink = (pos + 1).clamp(max=W), (pos - W + 1).clamp(0, S)
    seen = torch.where(i < W, i < n_ring[:, None], i - W < n_sink[:, None])[:, None, None]
    k = torch.cat([_unpack4(s["kc"], d), _unpack4(s["sk"], d)], 2)
    z = (s["q"].float().unflatten(1, (H, -1)) / math.sqrt(d)) @ k.transpose(-1, -2)
    del k
    z = z.masked_fill(~seen, -math.inf)
    m = z.amax(-1, keepdim=True)
    e = torch.exp(z - m)
    total = e.sum(-1, keepdim=True)
    v = torch.cat([_unpack4(s["vc"], d), _unpack4(s["sv"], d)], 2)
    v = v.masked_fill(~seen[:, :, 0, :, None], 0.0)
    s["out"].copy_((e @ v / total).flatten(1, 2))
    s["lse"].copy_((m + torch.log(total)).flatten(1))
    return s["out"], s["lse"]


def _obs_logits(q, k, c, dtype):
    """Scaled scores [B, Hkv, G * n_obs, L] of the queries that observe, -inf where a key is not visible."""
    n, L, H = q.shape[1], k.shape[1], c["Hkv"]
    qg = q.to(dtype).unflatten(2, (H, -1)).permute(0, 2, 3, 1, 4).flatten(2, 3)
    z = qg @ k.to(dtype).permute(0, 2, 3, 1) / math.sqrt(c["d"])
    t, j = torch.arange(L - n, L, device="cuda")[:, None], torch.arange(L, device="cuda")
    seen = (j <= t) & ((j > t - c["W"]) | (j < c["S"]))
    return z.unflatten(2, (-1, n)).masked_fill(~seen, -math.inf).flatten(2, 3)


def _plain_hh_scores(s):
    c = s["case"]
    n = c["n_obs"]
    z = _obs_logits(s["q"][:, c["L"] - n:], s["k"], c, torch.float32)
    lse = s["lse"][..., c["L"] - n:].unflatten(1, (c["Hkv"], -1)).flatten(2, 3)
    s["score"].copy_(torch.exp(z - lse[..., None]).sum(2))
    return s["score"]


def _plain_hh_fill(s):
    c = s["case"]
    L, C, S, recent = c["L"], c["C"], c["S"], c["recent"]
    j = torch.arange(L, device="cuda")
    if L > C:
        always = (j < S) | (j >= L - recent)
        rank = s["score_in"].masked_fill(always, math.inf)
        keep = torch.sort(rank, dim=-1, descending=True, stable=True)[1][..., :C].sort(-1)[0]
    else:
        keep = j.expand(c["B"], c["Hkv"], L)
    n = keep.shape[-1]
    at = keep.transpose(1, 2)[..., None].expand(-1, -1, -1, c["d"])
    s["kc"][:, :, :n] = s["k"].gather(1, at).transpose(1, 2)
    s["vc"][:, :, :n] = s["v"].gather(1, at).transpose(1, 2)
    s["slot_pos"].fill_(-1)[..., :n] = keep.to(torch.int32)
    s["score"].zero_()[..., :n] = s["score_in"].gather(-1, keep)
    return s["kc"], s["vc"], s["slot_pos"], s["score"]


def _plain_hh_step(s):
    c = s["case"]
    H, d = c["Hkv"], c["d"]
    pos, sp, score = s["pos"].long()[:, None, None], s["slot_pos"].long(), s["score"]
    same, empty = sp == pos, sp < 0
    may_go = (sp >= c["S"]) & (sp <= pos - c["recent"])
    # in this order: the slot of the same position, an empty one, the lightest that may go, the lightest
    rank = torch.where(same, 0, torch.where(empty, 1, torch.where(may_go, 2, 3)))
    best = rank.amin(-1, keepdim=True)
    w = torch.where(rank == best, torch.where(best < 2, torch.zeros_like(score), score), math.inf)
    slot = w.argmin(-1)
    s["slot"].copy_(slot)
    at = slot[..., None]
    s["kc"].scatter_(2, at[..., None].expand(-1, -1, -1, d), s["kn"][:, :, None])
    s["vc"].scatter_(2, at[..., None].expand(-1, -1, -1, d), s["vn"][:, :, None])
    s["slot_pos"].scatter_(2, at, pos.expand(-1, H, -1).to(torch.int32))
    score.scatter_(2, at, 0.0)
    seen = (s["slot_pos"] >= 0)[:, :, None]
    z = (s["q"].float().unflatten(1, (H, -1)) / math.sqrt(d)) @ s["kc"].float().transpose(-1, -2)
    z = z.masked_fill(~seen, -math.inf)
    m = z.amax(-1, keepdim=True)
    e = torch.exp(z - m)
    total = e.sum(-1, keepdim=True)
    v = s["vc"].float().masked_fill(~seen[:, :, 0, :, None], 0.0)
    s["out"].copy_((e @ v / total).flatten(1, 2))
    s["lse"].copy_((m + torch.log(total)).flatten(1))
    score.add_((e / total).sum(2))
    return s["out"], s["lse"], s["score"], s["slot"], s["slot_pos"]


def _axis_of_pair(c, sections):
    """The axis and the frequency of each pair of a head's elements."""
    half, n = c["d"] // 2, len(sections)
    i = torch.arange(half, device="cuda")
    ends = torch.tensor(sections, device="cuda").cumsum(0)
    if c["layout"] == "interleaved":
        size = torch.tensor(sections, device="cuda")[i % n]
        return torch.where(i // n < size, i % n, 0), 10000.0 ** (-i.double() / half)
    axis = (i[:, None] >= ends).sum(-1)
    if c["layout"] == "per_axis":
        size = torch.tensor(sections, device="cuda")[axis]
        return axis, 10000.0 ** (-(i - (ends[axis] - size)).double() / size.double())
    return axis, 10000.0 ** (-i.double() / half)


def _plain_rope(s):
    c = s["case"]
    axis, theta = _axis_of_pair(c, s["sections"])
    angle = s["positions"].double()[axis].T * theta  # far positions need 64 bits
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    if c["inverse"]:
        sin = -sin
    for x in (s["q"], s["k"]):
        lo, hi = x.float().chunk(2, -1)
        x.copy_(torch.cat([lo * cos - hi * sin, lo * sin + hi * cos], -1))
    return s["q"], s["k"]


# ------------------------------------------------------------------ one pass
def run(state):
    s, c = state, state["case"]
    if not own:
        return {"kv4_prompt": _plain_kv4_prompt, "kv4_step": _plain_kv4_step, "hh_scores": _plain_hh_scores,
                "hh_fill": _plain_hh_fill, "hh_step": _plain_hh_step, "rope": _plain_rope}[s["kind"]](s)
    import sink_aware_sliding_b200 as swa
    if s["kind"] == "kv4_prompt":
        swa.swa_kv4_cache_fill(s["k"], s["v"], s["kc"], s["vc"], s["sk"], s["sv"], c["W"], c["S"])
        swa.swa_kv4_cache_read(s["kept"], s["kc"], s["vc"], s["sk"], s["sv"], s["ko"], s["vo"], c["W"], c["S"])
        return s["ko"], s["vo"]
    if s["kind"] == "kv4_step":
        swa.swa_kv4_cache_append(s["kn"], s["vn"], s["pos"], s["kc"], s["vc"], s["sk"], s["sv"], c["W"], c["S"])
        swa.swa_kv4_decode(s["q"], s["kc"], s["vc"], s["sk"], s["sv"], s["pos"], s["out"], s["lse"], c["W"], c["S"])
        return s["out"], s["lse"]
    if s["kind"] == "hh_scores":
        swa.swa_hh_scores(s["q"], s["k"], s["lse"], s["score"], c["n_obs"], c["W"], c["S"])
        return s["score"]
    if s["kind"] == "hh_fill":
        swa.swa_hh_cache_fill(s["k"], s["v"], s["score_in"], s["kc"], s["vc"], s["slot_pos"], s["score"], c["S"],
                              c["recent"])
        return s["kc"], s["vc"], s["slot_pos"], s["score"]
    if s["kind"] == "hh_step":
        swa.swa_hh_cache_append(s["kn"], s["vn"], s["pos"], s["kc"], s["vc"], s["slot_pos"], s["score"], s["slot"],
                                c["S"], c["recent"])
        swa.swa_hh_decode(s["q"], s["kc"], s["vc"], s["slot_pos"], s["score"], s["out"], s["lse"])
        return s["out"], s["lse"], s["score"], s["slot"], s["slot_pos"]
    swa.swa_rope_axes_qk(s["q"], s["k"], s["positions"], s["sections"], layout=c["layout"], inverse=c["inverse"])
    return s["q"], s["k"]


# ------------------------------------------------------------------ what a pass cannot do without
def _pairs(L, n_obs, W, S):
    """Visible (query, key) pairs of the last n_obs queries of a sequence of L tokens."""
    total = 0
    for t in range(L - n_obs, L):
        first = max(0, t - W + 1)
        total += t + 1 - first + min(S, first)
    return total


def work(case):
    c = case
    kind, d, B, H = c["kind"], c["d"], c.get("B"), c["Hkv"]
    if kind == "kv4_prompt":
        kept = min(c["P"], c["W"]) + min(c["S"], max(0, c["P"] - c["W"]))
        # the prompt's rows in, the packed rows out, their values out
        return {"bytes": 2 * B * H * kept * (2 * d + _row_bytes(d) + 2 * d), "flops": 2 * B * H * kept * d * 6}
    if kind == "kv4_step":
        rows = c["W"] + c["S"] if not c["ragged"] else c["W"] * 3 // 4 + c["S"] // 2
        return {"bytes": 2 * B * H * (rows * _row_bytes(d) + 2 * d) + 4 * B * c["Hq"] * (d + 1),
                "flops": 4 * B * c["Hq"] * rows * d}
    if kind == "hh_scores":
        keys = min(c["L"], c["W"] + c["n_obs"] + c["S"])
        return {"bytes": 2 * B * d * (keys * H + c["n_obs"] * c["Hq"]) + 4 * B * (c["Hq"] * c["n_obs"] + H * c["L"]),
                "flops": 2 * d * B * c["Hq"] * _pairs(c["L"], c["n_obs"], c["W"], c["S"])}
    if kind == "hh_fill":
        kept = min(c["L"], c["C"])
        return {"bytes": B * H * (4 * c["L"] + kept * (8 * d + 4) + 4 * c["C"]), "flops": B * H * c["L"]}
    if kind == "hh_step":
        return {"bytes": B * H * (c["C"] * 12 + int(c["fill"] * c["C"]) * 4 * d) + 4 * B * c["Hq"] * (d + 1),
                "flops": 4 * B * c["Hq"] * int(c["fill"] * c["C"]) * d}
    size = 2 if c["dtype"] == "bf16" else 4
    return {"bytes": 2 * size * c["T"] * (c["Hq"] + H) * d + 4 * c["axes"] * c["T"],
            "flops": 3 * c["T"] * (c["Hq"] + H) * d}


# ------------------------------------------------------------------ the definitions in 64 bits
def _e4(x):
    """The values that rows hold once they are in 4 bits: the definition rounds the scale to bf16, and its
    reciprocal and the scaled distance from the minimum to 32 bits; what follows is exact."""
    shape = x.shape
    r = x.double().reshape(-1, GROUP)
    lo, hi = r.min(1).values, r.max(1).values
    step = ((hi - lo).float().double() * torch.tensor(1 / 15).to(r.device).double()).float().bfloat16().double()
    ok = step >= 2.0 ** -126
    inv = torch.where(ok, 1 / torch.where(ok, step, torch.ones_like(step)), torch.zeros_like(step)).float().double()
    step = torch.where(ok, step, torch.zeros_like(step))
    dist = (r - lo[:, None]).float().double()
    code = torch.round((dist * inv[:, None]).float().double()).clamp(0, 15)
    return (code * step[:, None] + lo[:, None]).reshape(shape)


def _e_attend(q, k, v, seen):
    """softmax over the seen keys: q [H, G, d], k and v [H, n, d] in 64 bits, seen [H, n]."""
    z = torch.einsum("hgd,hnd->hgn", q.double(), k) / math.sqrt(q.shape[-1])
    z = z.masked_fill(~seen[:, None], -math.inf)
    lse = torch.logsumexp(z, -1)
    p = torch.exp(z - lse[..., None])
    return torch.einsum("hgn,hnd->hgd", p, v.masked_fill(~seen[..., None], 0.0)), lse, p


def exact(case, seed):
    s, c = prepare(case, seed), case
    kind, B, d, H = c["kind"], c.get("B"), c["d"], c["Hkv"]
    if kind == "kv4_prompt":
        at = s["kept"][0].long()
        return _e4(s["k"][:, at]), _e4(s["v"][:, at])
    if kind == "kv4_step":
        outs, lses = [], []
        for b in range(B):
            p = int(s["pos"][b])
            keys = []
            for ring, sink, new in (("kc", "sk", "kn"), ("vc", "sv", "vn")):
                rows = torch.cat([_unpack4(s[ring][b], d, torch.float64), _unpack4(s[sink][b], d, torch.float64)], 1)
                rows[:, p % c["W"]] = _e4(s[new][b])
                if p < c["S"]:
                    rows[:, c["W"] + p] = _e4(s[new][b])
                keys.append(rows)
            i = torch.arange(c["W"] + c["S"], device="cuda")
            first = max(0, p - c["W"] + 1)
            seen = (i < min(p + 1, c["W"])) | ((i >= c["W"]) & (i - c["W"] < min(c["S"], first)))
            o, lse, _ = _e_attend(s["q"][b].unflatten(0, (H, -1)), keys[0], keys[1], seen.expand(H, -1))
            outs.append(o.flatten(0, 1))
            lses.append(lse.flatten())
        return torch.stack(outs), torch.stack(lses)
    if kind == "hh_scores":
        n, L, G = c["n_obs"], c["L"], c["Hq"] // H
        score = torch.zeros(B, H, L, dtype=torch.float64, device="cuda")
        t, j = torch.arange(L - n, L, device="cuda")[:, None], torch.arange(L, device="cuda")
        seen = (j <= t) & ((t - j < c["W"]) | (j < c["S"]))
        for b in range(B):
            for h in range(c["Hq"]):
                z = s["q"][b, L - n:, h].double() @ s["k"][b, :, h // G].double().T / math.sqrt(d)
                w = torch.exp(z - s["lse"][b, h, L - n:].double()[:, None])
                score[b, h // G] += torch.where(seen, w, torch.zeros_like(w)).sum(0)
        return score
    if kind == "hh_fill":
        kc, vc = s["kc"].double(), s["vc"].double()
        sp, score = s["slot_pos"].clone(), s["score"].double()
        L, C = c["L"], c["C"]
        j = torch.arange(L, device="cuda")
        always = (j < c["S"]) | (j >= L - c["recent"])
        for b in range(B):
            for h in range(H):
                kept = j
                if L > C:
                    free = C - int(always.sum())
                    w = s["score_in"][b, h][~always].double().cpu()
                    chosen = j[~always].cpu()[torch.argsort(-w, stable=True)[:free]].to("cuda")
                    kept = torch.cat([j[always], chosen]).sort().values
                m = kept.numel()
                kc[b, h, :m], vc[b, h, :m] = s["k"][b, kept, h].double(), s["v"][b, kept, h].double()
                sp[b, h, :m], score[b, h, :m] = kept.to(torch.int32), s["score_in"][b, h, kept].double()
        return kc, vc, sp, score
    if kind == "hh_step":
        outs, lses, scores, slots, places = [], [], [], [], []
        for b in range(B):
            p = int(s["pos"][b])
            sp, score = s["slot_pos"][b].long().clone(), s["score"][b].double()
            host, light = sp.cpu(), score.cpu()
            slot = []
            for h in range(H):
                for may in (host[h] == p, host[h] < 0, (host[h] >= c["S"]) & (host[h] <= p - c["recent"]), host[h] >= 0):
                    at = may.nonzero().flatten()
                    if at.numel():
                        w = light[h, at] if bool((host[h, at] >= 0).all()) else torch.zeros(at.numel())
                        slot.append(int(at[int((w == w.min()).nonzero()[0])]))
                        break
            k, v = s["kc"][b].double(), s["vc"][b].double()
            h, at = torch.arange(H, device="cuda"), torch.tensor(slot, device="cuda")
            k[h, at], v[h, at] = s["kn"][b].double(), s["vn"][b].double()
            sp[h, at], score[h, at] = p, 0.0
            o, lse, w = _e_attend(s["q"][b].unflatten(0, (H, -1)), k, v, sp >= 0)
            outs.append(o.flatten(0, 1))
            lses.append(lse.flatten())
            scores.append(score + w.sum(1))
            slots.append(at.to(torch.int32))
            places.append(sp.to(torch.int32))
        return torch.stack(outs), torch.stack(lses), torch.stack(scores), torch.stack(slots), torch.stack(places)
    half, axes, sec = d // 2, c["axes"], s["sections"]
    turn = torch.zeros(c["T"], half, dtype=torch.float64, device="cuda")
    done = [0] * axes
    for i in range(half):
        if c["layout"] == "interleaved":
            a = i % axes if i // axes < sec[i % axes] else 0
        else:
            a = next(n for n in range(axes) if i < sum(sec[:n + 1]))
        power = done[a] / sec[a] if c["layout"] == "per_axis" else i / half
        done[a] += 1
        turn[:, i] = s["positions"][a].double() / 10000.0 ** power
    turn = torch.polar(torch.ones_like(turn), -turn if c["inverse"] else turn)[:, None]
    outs = []
    for x in (s["q"], s["k"]):
        z = torch.complex(x[..., :half].double(), x[..., half:].double()) * turn
        outs.append(torch.cat([z.real, z.imag], -1))
    return tuple(outs)
