"""The 8-bit integer products of the int8 per-row layer, in plain form and by the library's kernels.

The layer is W = lora_up lora_down^T + H256(diag(s_w) Q): int8 codes Q [N, K], one fp32 scale per
output channel, a rank-16 bf16 branch, rotated by the block-diagonal Hadamard matrix of order 256
over K.  Four operators, each a product of 8-bit integers with one scale per token and one per
channel:

  fwd          y  = s_x s_w (q_x Q^T) + (x lora_down) lora_up^T,  q_x = int8 codes of H x per token
  bwd          dx = H(s_g (q_g Q)) + (dy lora_up) lora_down^T,    q_g = int8 codes of dy s_w per token
  grouped_fwd  the forward with one layer per expert, the rows of each expert lying together
  grouped_bwd  its input gradient

The codes of a row r are rint(r (1 / s)), s = max|r| / 127, in single precision with one rounding
per operation; the rotation is the radix-2 transform with strides 1, 2, ..., 128.  The plain form
keeps that order, so that a value next to a rounding border falls on the same side.
"""
import math

import numpy as np
import torch

own = False

RANK = 16
LARGEST = dict(M=4480, N=16384, K=6144)        # tokens, output and input features of the largest product


def _case(name, op, M, N, K, out="bf16", lora=True, E=0, active=0, skew=0.0, pad=0):
    return dict(name=name, op=op, M=M, N=N, K=K, out=out, lora=lora, E=E, active=active, skew=skew, pad=pad)


def listed():
    return [
        # one sequence generating one token: latency, and the weight's bytes
        _case("fwd_token", "fwd", 1, 6144, 6144),
        # two dozen sequences generating together
        _case("fwd_tokens24", "fwd", 24, 16384, 6144),
        # a short prompt of an odd length through a layer of odd multiples of 128 and 256, no
        # low-rank branch, single-precision output
        _case("fwd_prompt777", "fwd", 777, 4224, 2816, out="f32", lora=False),
        # the widest projection over a whole image's or prompt's tokens
        _case("fwd_prompt4480", "fwd", 4480, 16384, 6144),
        # training, a short batch: gradient of the input
        _case("bwd_509", "bwd", 509, 2944, 2048, out="f32"),
        # training, the widest projection over a whole batch
        _case("bwd_4480", "bwd", 4480, 16384, 6144, out="f32"),
        # four sequences generating with 8 of 64 experts each: 32 rows on 27 experts
        _case("grouped_tokens32", "grouped_fwd", 32, 2816, 2048, E=64, active=27, skew=0.2),
        # a prompt of 1024 tokens with 8 of 64 experts each, unevenly spread, padded to 8300 rows
        _case("grouped_prompt", "grouped_fwd", 8192, 2816, 2048, E=64, active=61, skew=0.6, pad=108),
        # few large experts, single-precision output
        _case("grouped_wide", "grouped_fwd", 6001, 6144, 4096, out="f32", E=8, active=8, skew=0.4),
        # training with experts: a short batch, and a long one
        _case("grouped_bwd_300", "grouped_bwd", 300, 2048, 1280, out="f32", E=16, active=13, skew=0.8, pad=4),
        _case("grouped_bwd_8192", "grouped_bwd", 8192, 2816, 2048, E=64, active=64, skew=0.6),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["fwd", "bwd", "grouped_fwd", "grouped_bwd"])
    grouped = op.startswith("grouped")
    largest = LARGEST["M"] * LARGEST["N"] * LARGEST["K"]
    while True:
        N = 128 * _log_int(rng, 1, 128 if not grouped else 48)
        K = 256 * _log_int(rng, 1, 64 if not grouped else 16)
        M = _log_int(rng, 1, 4480 if not grouped else 8192)
        E = _log_int(rng, 1, 128) if grouped else 0
        if M * N * K <= largest and max(E, 1) * N * K <= 400_000_000:
            break
    active = rng.randint(1, min(E, M)) if grouped else 0
    return dict(op=op, M=M, N=N, K=K, out=rng.choice(["bf16", "f32"]), lora=rng.random() < 0.7, E=E,
                active=active, skew=rng.choice([0.0, 0.4, 1.0]) if grouped else 0.0,
                pad=rng.choice([0, 0, 1, 77]) if grouped else 0)


def _counts(case):
    """Rows of each expert that has any, largest first: every one at least 1, M in all."""
    a = case["active"]
    share = np.arange(1, a + 1, dtype=np.float64) ** -case["skew"]
    c = 1 + np.floor((case["M"] - a) * share / share.sum()).astype(np.int64)
    c[: case["M"] - int(c.sum())] += 1
    return c


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    M, N, K, E = case["M"], case["N"], case["K"], case["E"]
    grouped, bwd = E > 0, case["op"].endswith("bwd")
    lead = (E,) if grouped else ()
    dev = dict(device="cuda")
    state = dict(case=case)
    # codes of a builder: bell-shaped, the MSE-chosen scale clipping the tails
    q = torch.empty(*lead, N, K, dtype=torch.float32, **dev)
    q.normal_(0.0, 38.0, generator=g)
    state["codes"] = q.round_().clamp_(-127, 127).to(torch.int8)
    del q
    state["scales"] = (torch.rand(*lead, N, generator=g, **dev) + 0.5) * (0.026 / math.sqrt(K))
    if case["lora"]:
        state["lora_up"] = (torch.randn(*lead, N, RANK, generator=g, **dev) * 0.2).to(torch.bfloat16)
        state["lora_down"] = (torch.randn(*lead, K, RANK, generator=g, **dev) * (0.6 / math.sqrt(K))).to(torch.bfloat16)
    else:
        state["lora_up"] = state["lora_down"] = None
    rows, width = M + case["pad"], N if bwd else K
    x = torch.randn(rows, width, generator=g, **dev)
    if bwd:     # gradients: small, and of very different size from token to token
        x *= 1e-3 * torch.exp(torch.randn(rows, 1, generator=g, **dev))
    else:       # activations: a few channels far larger than the rest
        loud = torch.randperm(width, generator=g, **dev)[: max(1, width // 128)]
        x[:, loud] *= 12.0
    state["x"] = x.to(torch.bfloat16)
    if grouped:
        counts = np.zeros(E, np.int64)
        counts[np.random.default_rng(seed).permutation(E)[: case["active"]]] = _counts(case)
        state["counts"] = counts.tolist()
        state["offsets"] = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, **dev)
    if own:     # the handle of the layer that a program keeps, over the same tensors
        import bit_quantized_frozen_b200 as sq
        parts = (state["codes"], state["scales"], state["lora_up"], state["lora_down"])
        state["w"] = (sq.GroupedWeight(E, N, K, *parts) if grouped
                      else sq.Weight(sq.SQ_FMT_INT8_ROW, N, K, parts[0], parts[1], None, parts[2], parts[3]))
    return state


# ---- plain form ---------------------------------------------------------------------------------

def _rotate(v):
    """H256 over every 256 columns: radix-2 butterflies, strides 1, 2, ..., 128, then 1/16."""
    rows, width = v.shape
    for stride in (1, 2, 4, 8, 16, 32, 64, 128):
        v = v.reshape(rows, width // (2 * stride), 2, stride)
        a, b = v[:, :, 0], v[:, :, 1]
        v = torch.stack((a + b, a - b), dim=2)
    return v.reshape(rows, width) * 0.0625


def _quantise(v):
    """(codes as numbers, scales) of the rows of v."""
    s = v.abs().amax(dim=1, keepdim=True) / torch.full((1, 1), 127.0, device=v.device)
    inv = torch.where(s > 0, torch.reciprocal(s), torch.zeros_like(s))
    return (v * inv).round().clamp(-127, 127), s


def _plain_fwd(x, codes, scales, up, down, dtype):
    x = x.float()
    q, s = _quantise(_rotate(x))
    y = (q @ codes.float().t()) * (s * scales)
    if up is not None:
        y += (x @ down.float()) @ up.float().t()
    return y.to(dtype)


def _plain_bwd(dy, codes, scales, up, down, dtype):
    dy = dy.float()
    q, s = _quantise(dy * scales)
    dx = _rotate((q @ codes.float()) * s)
    if up is not None:
        dx += (dy @ up.float()) @ down.float().t()
    return dx.to(dtype)


def _grouped(state, f, dtype, width):
    """f over the rows of each expert that has any; rows outside every group are 0."""
    out = torch.zeros(state["x"].shape[0], width, dtype=dtype, device=state["x"].device)
    at = 0
    for e, n in enumerate(state["counts"]):
        if n:
            up, down = (None, None) if state["lora_up"] is None else (state["lora_up"][e], state["lora_down"][e])
            out[at:at + n] = f(state["x"][at:at + n], state["codes"][e], state["scales"][e], up, down, dtype)
            at += n
    return out


def run(state):
    case = state["case"]
    op, bf16 = case["op"], case["out"] == "bf16"
    if own:
        import bit_quantized_frozen_b200 as sq
        if op == "fwd":
            return sq.linear_fwd_w8a8(state["w"], state["x"], out_bf16=bf16)
        if op == "bwd":
            return sq.linear_bwd_dx_w8a8(state["w"], state["x"], out_bf16=bf16)
        f = sq.grouped_fwd_w8a8 if op == "grouped_fwd" else sq.grouped_bwd_dx_w8a8
        return f(state["w"], state["x"], state["offsets"], out_bf16=bf16)
    dtype = torch.bfloat16 if bf16 else torch.float32
    f = _plain_bwd if op.endswith("bwd") else _plain_fwd
    if case["E"]:
        return _grouped(state, f, dtype, case["K"] if op.endswith("bwd") else case["N"])
    return f(state["x"], state["codes"], state["scales"], state["lora_up"], state["lora_down"], dtype)


def work(case):
    M, N, K = case["M"], case["N"], case["K"]
    bwd, experts = case["op"].endswith("bwd"), case["active"] if case["E"] else 1
    size = 2 if case["out"] == "bf16" else 4
    layer = N * K + 4 * N + (2 * RANK * (N + K) if case["lora"] else 0)
    rows = 2 * M * (N if bwd else K) + size * (M + case["pad"]) * (K if bwd else N)
    return {"bytes": experts * layer + rows + (4 * (case["E"] + 1) if case["E"] else 0),
            "flops": 2 * M * N * K + (2 * RANK * M * (N + K) if case["lora"] else 0)}


# ---- the definition in 64 bits ------------------------------------------------------------------
#
# The codes are whole numbers that the definition gives by single-precision operations with one
# rounding each; they are formed that way here too.  All that is computed from them is in 64 bits.

def _hadamard():
    """The Sylvester matrix of order 256 over 16: entry (i, j) is (-1)^(number of ones in i & j) / 16."""
    i = np.arange(256)
    ones = np.array([bin(v).count("1") for v in range(256)])
    return torch.tensor(np.where(ones[i[:, None] & i[None, :]] % 2 == 0, 1.0, -1.0) / 16.0, dtype=torch.float64,
                        device="cuda")


def _single_rotation(v):
    """Column k becomes v[k] + v[k ^ h] where k has no bit h, else v[k ^ h] - v[k]; h = 1, 2, ..., 128; over 16."""
    k = torch.arange(v.shape[1], device=v.device)
    h = 1
    while h < 256:
        other = v[:, k ^ h]
        v = torch.where((k & h) != 0, other - v, other + v)
        h *= 2
    return v / 16.0


def _single_codes(r):
    largest = r.abs().max(dim=1).values
    s = torch.div(largest, torch.full_like(largest, 127.0))
    q = torch.round(r * torch.where(s > 0, torch.ones_like(s) / s, s)[:, None])
    return torch.clamp(q, -127.0, 127.0).double(), s.double()[:, None]


def exact(case, seed):
    state = prepare(case, seed)
    H, d = _hadamard(), torch.float64
    bwd = case["op"].endswith("bwd")
    rows = state["x"].shape[0]
    bounds = [(0, rows, None)]
    if case["E"]:
        ends = np.cumsum(state["counts"])
        bounds = [(int(e - n), int(e), i) for i, (e, n) in enumerate(zip(ends, state["counts"])) if n]
    out = torch.zeros(rows, case["K"] if bwd else case["N"], dtype=d, device="cuda")
    for lo, hi, e in bounds:
        pick = (lambda t: t) if e is None else (lambda t: t[e])
        Q, sw, v = pick(state["codes"]).to(d), pick(state["scales"]), state["x"][lo:hi].float()
        q, s = _single_codes(v * sw if bwd else _single_rotation(v))
        if bwd:
            z = torch.einsum("rbk,kj->rbj", (torch.einsum("mn,nk->mk", q, Q) * s).view(hi - lo, -1, 256), H)
            z = z.reshape(hi - lo, -1)
        else:
            z = torch.einsum("mk,nk->mn", q, Q) * s * sw.to(d)
        if state["lora_up"] is not None:
            up, down = pick(state["lora_up"]).to(d), pick(state["lora_down"]).to(d)
            z += v.to(d) @ up @ down.t() if bwd else v.to(d) @ down @ up.t()
        out[lo:hi] = z
    return out
