"""Products of 8-bit floating point with a scale for each block of 128, and the gated feed-forward
projections on them, in plain form and by the library's kernels.

A weight W [N, K] is held as e4m3 codes Q and one power of two (e8m0) for each block of 128 x 128:
W = S Q.  The rows that meet it are rounded to e4m3 in blocks of 128 along the summed axis, each with
the least power of two s >= 2^-127 for which |r| <= 448 s; r / s is exact, so a code is one rounding of
the value itself.  Two kinds of operator, dense and with one weight per expert (the rows of each expert
lying together):

  fwd        y  = xq W^T
  bwd        dx = dyq W
  gated_fwd  h  = act(g) u,  g = xq Wgate^T,  u = xq Wup^T; for training g and u are returned in bf16 too
  gated_bwd  dx = dgq Wgate + duq Wup,  dg = dh u act'(g),  du = dh act(g), from those g and u

act is silu, or gelu in its tanh form.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 128
LARGEST = 2 * 4480 * 16384 * 6144             # products of a row's and a weight's value: both projections of the widest block


def _case(name, op, M, N, K, out="bf16", act="", save=False, E=0, active=0, skew=0.0, pad=0):
    return dict(name=name, op=op, M=M, N=N, K=K, out=out, act=act, save=save, E=E, active=active, skew=skew, pad=pad)


def listed():
    return [
        # one sequence generating one token: latency, and the weight's bytes
        _case("fwd_token", "fwd", 1, 6144, 6144),
        # a short prompt of an odd length, widths that end inside a block, single-precision output
        _case("fwd_prompt777", "fwd", 777, 4240, 2832, out="f32"),
        # the widest projection over a whole image's or prompt's tokens
        _case("fwd_prompt4480", "fwd", 4480, 16384, 6144),
        # training, a short batch: gradient of the input, single-precision output
        _case("bwd_509", "bwd", 509, 2944, 2048, out="f32"),
        # training, the widest projection over a whole batch
        _case("bwd_4480", "bwd", 4480, 16384, 6144),
        # four sequences generating with 8 of 64 experts each: 32 rows on 27 experts
        _case("grouped_tokens32", "fwd", 32, 2816, 2048, E=64, active=27, skew=0.2),
        # training with experts, a long batch, unevenly spread
        _case("grouped_bwd_8192", "bwd", 8192, 2816, 2048, E=64, active=64, skew=0.6),
        # eight sequences generating together through a gated block
        _case("gated_tokens8", "gated_fwd", 8, 16384, 6144, act="silu"),
        # training, both projections of the widest block over a whole batch
        _case("gated_4480", "gated_fwd", 4480, 16384, 6144, act="silu", save=True),
        # training, a middling batch: gradient through both projections
        _case("gated_bwd_2049", "gated_bwd", 2049, 8192, 4096, act="gelu"),
        # a prompt of 1024 tokens with 8 of 64 experts each, unevenly spread, padded to 8300 rows
        _case("grouped_gated_prompt", "gated_fwd", 8192, 1408, 2048, act="silu", E=64, active=61, skew=0.6, pad=108),
        # training with gated experts, a short batch
        _case("grouped_gated_bwd_1030", "gated_bwd", 1030, 2064, 1280, act="silu", E=16, active=13, skew=0.8, pad=4),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["fwd", "bwd", "gated_fwd", "gated_bwd"])
    grouped, gated = rng.random() < 0.5, op.startswith("gated")
    while True:
        # whole blocks or widths that end inside one
        N, K = (s * _log_int(rng, 256 // s, top // s) for s, top in ((rng.choice([16, 128]), 16384 if not grouped else 6144),
                                                                     (rng.choice([16, 128]), 16384 if not grouped else 4096)))
        M = _log_int(rng, 1, 4480 if not grouped else 8192)
        E = _log_int(rng, 1, 128) if grouped else 0
        times = 2 if gated else 1
        if times * M * N * K <= LARGEST and times * max(E, 1) * N * K <= 400_000_000:
            break
    summed = K if op == "fwd" else N
    return dict(op=op, M=M, N=N, K=K, out="f32" if not gated and summed <= 8192 and rng.random() < 0.4 else "bf16",
                act=rng.choice(["silu", "gelu"]) if gated else "", save=op == "gated_fwd" and rng.random() < 0.5, E=E,
                active=rng.randint(1, min(E, M)) if grouped else 0, skew=rng.choice([0.0, 0.4, 1.0]) if grouped else 0.0,
                pad=rng.choice([0, 0, 1, 77]) if grouped else 0)


def _counts(case):
    """Rows of each expert that has any, largest first: every one at least 1, M in all."""
    a = case["active"]
    share = np.arange(1, a + 1, dtype=np.float64) ** -case["skew"]
    c = 1 + np.floor((case["M"] - a) * share / share.sum()).astype(np.int64)
    c[: case["M"] - int(c.sum())] += 1
    return c


def _blocks(n):
    return (n + BLOCK - 1) // BLOCK


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    M, N, K, E, op = case["M"], case["N"], case["K"], case["E"], case["op"]
    gated, bwd = op.startswith("gated"), op.endswith("bwd")
    lead = (E,) if E else ()
    dev = dict(device="cuda")
    state = dict(case=case, codes=[], scales=[])
    for _ in range(2 if gated else 1):
        # bell-shaped values; a block's scale follows its largest one, so most blocks share two or three
        q = torch.empty(*lead, N, K, dtype=torch.float32, **dev)
        q.normal_(0.0, 90.0, generator=g)
        state["codes"].append(q.clamp_(-448, 448).to(torch.float8_e4m3fn))
        del q
        top = round(math.log2(math.sqrt(K) * 90 / (1.3 if gated else 1.0)))
        e = torch.randint(-1, 2, (*lead, _blocks(N), _blocks(K)), generator=g, **dev) + (127 - top)
        state["scales"].append(e.to(torch.uint8).view(torch.float8_e8m0fnu))
    rows = M + case["pad"]
    width = N if bwd else K
    x = torch.randn(rows, width, generator=g, **dev)
    if bwd:     # gradients: small, and of very different size from token to token
        x *= 1e-3 * torch.exp(torch.randn(rows, 1, generator=g, **dev))
    else:       # activations: a few channels far larger than the rest
        loud = torch.randperm(width, generator=g, **dev)[: max(1, width // 128)]
        x[:, loud] *= 12.0
    state["x"] = x.to(torch.bfloat16)
    if op == "gated_bwd":       # what the forward pass saved
        state["gate"] = (torch.randn(rows, N, generator=g, **dev) * 1.5).to(torch.bfloat16)
        state["up"] = (torch.randn(rows, N, generator=g, **dev) * 1.5).to(torch.bfloat16)
    if E:
        counts = np.zeros(E, np.int64)
        counts[np.random.default_rng(seed).permutation(E)[: case["active"]]] = _counts(case)
        state["counts"] = counts.tolist()
        state["offsets"] = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, **dev)
    if own:     # the handles of the layer that a program keeps, over the same tensors
        import bit_quantized_frozen_b200 as sq
        state["w"] = [sq.GroupedWeight(E, N, K, q, s, fmt=sq.SQ_FMT_FP8_BLOCK) if E
                      else sq.Weight(sq.SQ_FMT_FP8_BLOCK, N, K, q, s) for q, s in zip(state["codes"], state["scales"])]
    return state


# ---- plain form ---------------------------------------------------------------------------------

def _rounded(v):
    """The rows of v [..., width] after the rounding to e4m3 in blocks of 128."""
    width = v.shape[-1]
    b = torch.nn.functional.pad(v, (0, -width % BLOCK)).unflatten(-1, (-1, BLOCK))
    top = b.abs().amax(dim=-1, keepdim=True)
    m, e = torch.frexp(top)                                   # top = m 2^e, 1/2 <= m < 1; 448 = 0.875 * 2^9
    e = (e - 9 + (m > 0.875)).clamp(min=-127)
    q = torch.ldexp(b, -e).to(torch.float8_e4m3fn).float()
    return torch.ldexp(q, e).flatten(-2)[..., :width]


def _weight(codes, scales):
    """W in 32 bits."""
    N, K = codes.shape[-2:]
    s = scales.float().repeat_interleave(BLOCK, dim=-1)[..., :K].repeat_interleave(BLOCK, dim=-2)[..., :N, :]
    return codes.float() * s


def _act(g, kind):
    """(act(g), act'(g))"""
    if kind == "silu":
        s = 1 / (1 + torch.exp(-g))
        return g * s, s * (1 + g * (1 - s))
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (g + 0.044715 * g * g * g))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 3 * 0.044715 * g * g)


def _forward(case, x, weights):
    r = _rounded(x.float())
    y = [r @ w.transpose(-1, -2) for w in weights]
    if case["op"] == "fwd":
        return y
    h = _act(y[0], case["act"])[0] * y[1]
    return [h] + y if case["save"] else [h]


def _backward(case, dy, weights, gate=None, up=None):
    dy = dy.float()
    if case["op"] == "bwd":
        return [_rounded(dy) @ weights[0]]
    a, slope = _act(gate.float(), case["act"])
    return [_rounded(dy * up.float() * slope) @ weights[0] + _rounded(dy * a) @ weights[1]]


def _plain(state):
    case = state["case"]
    f = _backward if case["op"].endswith("bwd") else _forward
    rows = [state[k] for k in ("x", "gate", "up") if k in state]
    dtypes = [torch.float32 if case["out"] == "f32" else torch.bfloat16, torch.bfloat16, torch.bfloat16]
    if not case["E"]:
        out = f(case, rows[0], [_weight(q, s) for q, s in zip(state["codes"], state["scales"])], *rows[1:])
        return tuple(o.to(t) for o, t in zip(out, dtypes))
    # the experts that have rows, each with its rows padded to the largest number; rows of no expert are 0
    counts, dev = state["counts"], state["x"].device
    some = [e for e, n in enumerate(counts) if n]
    most = max(counts)
    n = torch.tensor([counts[e] for e in some], device=dev)
    at = torch.arange(most, device=dev)
    live = at < n[:, None]
    index = ((n.cumsum(0) - n)[:, None] + at)[live]
    pick = torch.tensor(some, device=dev)

    def spread(t):
        wide = t.new_zeros(len(some), most, t.shape[1])
        wide[live] = t[index]
        return wide

    # (the experts are picked as bytes: 8-bit types have no indexing of their own)
    codes = [q.view(torch.uint8)[pick].view(q.dtype) for q in state["codes"]]
    scales = [s.view(torch.uint8)[pick].view(s.dtype) for s in state["scales"]]
    weights = [_weight(q, s) for q, s in zip(codes, scales)]
    out = f(case, spread(rows[0]), weights, *(spread(r) for r in rows[1:]))
    whole = [torch.zeros(rows[0].shape[0], o.shape[-1], dtype=t, device=dev) for o, t in zip(out, dtypes)]
    for w, o in zip(whole, out):
        w[index] = o[live].to(w.dtype)
    return tuple(whole)


def run(state):
    if not own:
        return _plain(state)
    import bit_quantized_frozen_b200 as sq
    case, w, x = state["case"], state["w"], state["x"]
    op, bf16, act = case["op"], case["out"] == "bf16", case["act"]
    if case["E"]:
        off = state["offsets"]
        if op == "fwd":
            return (sq.grouped_fwd_fp8(w[0], x, off, out_bf16=bf16),)
        if op == "bwd":
            return (sq.grouped_bwd_dx_fp8(w[0], x, off, out_bf16=bf16),)
        if op == "gated_fwd":
            out = sq.grouped_gated_fwd_fp8(w[0], w[1], x, off, act=act, save=case["save"], out_bf16=bf16)
            return out if case["save"] else (out,)
        return (sq.grouped_gated_bwd_dx_fp8(w[0], w[1], x, state["gate"], state["up"], off, act=act, out_bf16=bf16),)
    if op == "fwd":
        return (sq.linear_fwd_fp8(w[0], x, out_bf16=bf16),)
    if op == "bwd":
        return (sq.linear_bwd_dx_fp8(w[0], x, out_bf16=bf16),)
    if op == "gated_fwd":
        out = sq.gated_fwd_fp8(w[0], w[1], x, act=act, save=case["save"], out_bf16=bf16)
        return out if case["save"] else (out,)
    return (sq.gated_bwd_dx_fp8(w[0], w[1], x, state["gate"], state["up"], act=act, out_bf16=bf16),)


def work(case):
    M, N, K, op = case["M"], case["N"], case["K"], case["op"]
    bwd, projections = op.endswith("bwd"), 2 if op.startswith("gated") else 1
    experts, rows = (case["active"], M + case["pad"]) if case["E"] else (1, M)
    size = 2 if case["out"] == "bf16" else 4
    layer = projections * (N * K + _blocks(N) * _blocks(K))
    read = 2 * M * N * (3 if op == "gated_bwd" else 1) if bwd else 2 * M * K
    write = size * rows * (K if bwd else N) + (4 * rows * N if case["save"] else 0)
    return {"bytes": experts * layer + read + write + (4 * (case["E"] + 1) if case["E"] else 0),
            "flops": 2 * projections * M * N * K}


# ---- the definition in 64 bits ------------------------------------------------------------------

def _exact_rows(v):
    """Rows rounded to e4m3 in blocks of 128: v [m, width] in 64 bits."""
    out = torch.empty_like(v)
    for b in range(0, v.shape[1], BLOCK):
        r = v[:, b:b + BLOCK]
        top = r.abs().max(dim=1, keepdim=True).values
        e = torch.ceil(torch.log2(torch.where(top > 0, top, torch.ones_like(top)) / 448.0))
        e = torch.where(448.0 * torch.exp2(e - 1) >= top, e - 1, e)       # log2 may be off next to a whole number
        e = torch.where(448.0 * torch.exp2(e) < top, e + 1, e).clamp(min=-127)
        t = r / torch.exp2(e)
        # e4m3: 3 bits behind the leading one, steps of 2^-9 below 2^-6
        step = torch.exp2(torch.floor(torch.log2(t.abs().clamp(min=2.0 ** -6))) - 3)
        out[:, b:b + BLOCK] = torch.round(t / step) * step * torch.exp2(e)
    return out


def _exact_weight(codes, scales, N, K):
    n, k = torch.arange(N, device="cuda") // BLOCK, torch.arange(K, device="cuda") // BLOCK
    return codes.to(torch.float64) * torch.exp2(scales.view(torch.uint8).to(torch.float64) - 127.0)[n][:, k]


def _exact_act(g, kind):
    if kind == "silu":
        return g * torch.sigmoid(g), torch.sigmoid(g) + g * torch.sigmoid(g) * torch.sigmoid(-g)
    # 0.5 (1 + tanh z) = sigmoid(2 z)
    z = 2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)
    dz = 2 * math.sqrt(2 / math.pi) * (1 + 0.134145 * g ** 2)
    return g * torch.sigmoid(z), torch.sigmoid(z) + g * torch.sigmoid(z) * torch.sigmoid(-z) * dz


def exact(case, seed):
    state = prepare(case, seed)
    N, K, op, d = case["N"], case["K"], case["op"], torch.float64
    rows = state["x"].shape[0]
    groups = [(0, rows, None)]
    if case["E"]:
        ends = np.cumsum(state["counts"])
        groups = [(int(e - n), int(e), i) for i, (e, n) in enumerate(zip(ends, state["counts"])) if n]
    widths = [K] if op.endswith("bwd") else [N, N, N] if case["save"] else [N]
    outs = tuple(torch.zeros(rows, w, dtype=d, device="cuda") for w in widths)
    for lo, hi, e in groups:
        W = [_exact_weight(*((q, s) if e is None else (q[e], s[e])), N, K) for q, s in zip(state["codes"], state["scales"])]
        v = state["x"][lo:hi].to(d)
        if op == "fwd":
            got = [torch.einsum("mk,nk->mn", _exact_rows(v), W[0])]
        elif op == "bwd":
            got = [torch.einsum("mn,nk->mk", _exact_rows(v), W[0])]
        elif op == "gated_fwd":
            v = _exact_rows(v)
            gate, up = (torch.einsum("mk,nk->mn", v, w) for w in W)
            got = [_exact_act(gate, case["act"])[0] * up, gate, up]
        else:
            a, slope = _exact_act(state["gate"][lo:hi].to(d), case["act"])
            dg, du = _exact_rows(v * state["up"][lo:hi].to(d) * slope), _exact_rows(v * a)
            got = [torch.einsum("mn,nk->mk", dg, W[0]) + torch.einsum("mn,nk->mk", du, W[1])]
        for o, x in zip(outs, got):
            o[lo:hi] = x
    return outs
