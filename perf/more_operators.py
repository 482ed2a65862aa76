"""What is measured of linear attention with a decay for each head (prompts, gradients, single
tokens) and of group norm, channels last, with an activation (forward and backward).

With ``own`` false, ``run`` computes an operator in its plain form (elementary torch
operations in float32, rounded once at the end); with ``own`` true it makes the calls of
``mamba_ssd_chunked_02_amd`` that a program makes.  ``exact`` gives the same outputs in
float64 from the definitions: the recurrence token by token, the norm by its sums.

Shapes: q [b, L, H, K], k [b, L, G, K], v [b, L, G, V] (packed: b = 1, sequences given by
cu_seqlens; head h reads group h G / H), decay [H] (logarithms), states [sequences, H, K, V];
the norm's x [samples, positions, channels].
"""
import math
import random

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
CHUNK = 64  # tokens of a block of the plain form


def listed():
    return [
        # a short odd request in float32 that goes on from a state: latency
        {"name": "linattn_short", "op": "lin_fwd", "dtype": "f32", "batch": 3, "seqlen": 77,
         "heads": 5, "groups": 5, "keys": 40, "values": 56, "nseq": 0, "carry": True},
        # the layer workload's tokens, d_model 768: 12 heads, keys of 64, values expanded twice
        {"name": "linattn_layer", "op": "lin_fwd", "dtype": "bf16", "batch": 2, "seqlen": 2048,
         "heads": 12, "groups": 12, "keys": 64, "values": 128, "nseq": 0, "carry": False},
        # prompts: 16 packed sequences, 65536 tokens in all
        {"name": "linattn_prompts", "op": "lin_fwd", "dtype": "bf16", "batch": 1,
         "seqlen": 65536, "heads": 16, "groups": 16, "keys": 128, "values": 128, "nseq": 16,
         "carry": True},
        # one long document through wide heads: few of them, so its tokens must be split
        {"name": "linattn_long", "op": "lin_fwd", "dtype": "bf16", "batch": 1, "seqlen": 32768,
         "heads": 8, "groups": 8, "keys": 256, "values": 256, "nseq": 0, "carry": False},
        # training: the layer workload's gradients
        {"name": "linattn_train", "op": "lin_bwd", "dtype": "bf16", "batch": 2, "seqlen": 2048,
         "heads": 12, "groups": 12, "keys": 64, "values": 128, "nseq": 0, "carry": False},
        # training in float32 on packed sequences of odd lengths; 4 heads share keys and values
        {"name": "linattn_train_shared", "op": "lin_bwd", "dtype": "f32", "batch": 1,
         "seqlen": 3001, "heads": 8, "groups": 2, "keys": 96, "values": 72, "nseq": 7,
         "carry": True},
        # one token of one sequence through the layer workload's heads: latency
        {"name": "linattn_token_one", "op": "lin_step", "dtype": "bf16", "batch": 1, "heads": 12,
         "groups": 12, "keys": 64, "values": 128, "spare": 0},
        # one new token for each of 64 sequences of a wide layer
        {"name": "linattn_token_batch", "op": "lin_step", "dtype": "bf16", "batch": 64,
         "heads": 32, "groups": 32, "keys": 128, "values": 128, "spare": 0},
        # the gated norm of every head's output, token by token, of the layer workload
        {"name": "gnorm_heads", "op": "gn_fwd", "dtype": "bf16", "samples": 4096, "positions": 1,
         "channels": 1536, "groups": 12, "form": "gate"},
        # its gradients for 8192 tokens of 16 heads of 128
        {"name": "gnorm_heads_train", "op": "gn_bwd", "dtype": "bf16", "samples": 8192,
         "positions": 1, "channels": 2048, "groups": 16, "form": "gate"},
        # 8 feature maps of 64 x 64 positions in front of a scan over their positions
        {"name": "gnorm_map", "op": "gn_fwd", "dtype": "bf16", "samples": 8, "positions": 4096,
         "channels": 320, "groups": 32, "form": "silu"},
        # training in float32 on small maps with an odd side (35 x 35)
        {"name": "gnorm_map_train", "op": "gn_bwd", "dtype": "f32", "samples": 4,
         "positions": 1225, "channels": 192, "groups": 8, "form": "silu"},
    ]


def _size(rng, lo, hi):
    """A whole number, evenly spread over the logarithm of [lo, hi]."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["lin_fwd", "lin_fwd", "lin_bwd", "lin_bwd", "lin_step", "gn_fwd", "gn_bwd"])
    case = {"op": op, "dtype": rng.choice(["bf16", "bf16", "f32"])}
    if op in ("gn_fwd", "gn_bwd"):
        groups = _size(rng, 1, 48)
        channels = groups * _size(rng, 3, 3000 / groups)
        most = 1.6e7 / channels
        positions = 1 if rng.random() < 0.4 else _size(rng, 2, max(2, most / 2))
        case |= {"samples": _size(rng, 1, max(1, most / positions)), "positions": positions,
                 "channels": channels, "groups": groups,
                 "form": rng.choice(["plain", "silu", "gate"])}
        return case
    groups = _size(rng, 1, 16)
    heads = groups * rng.choice([1, 1, 1, 2, 4])
    keys, values = 8 * _size(rng, 2, 32), 8 * _size(rng, 2, 32)
    case |= {"heads": heads, "groups": groups, "keys": keys, "values": values}
    area = heads * keys * values
    if op == "lin_step":
        return case | {"batch": _size(rng, 1, max(1, min(256, 3.3e7 / area))),
                       "spare": rng.choice([0, 5])}
    packed = rng.random() < 0.5
    tokens = _size(rng, 1, min(65536, (1.7e10 if op == "lin_fwd" else 3.0e9) / area))
    batch = 1 if packed else min(tokens, rng.randint(1, 8))
    return case | {"batch": batch, "seqlen": tokens // batch,
                   "nseq": rng.randint(1, 24) if packed else 0, "carry": rng.random() < 0.5}


def _lengths(case, seed):
    """Lengths of a packed batch's sequences; of more than twelve, one is empty."""
    r = random.Random(seed * 6151 + 29)
    n, total = case["nseq"], case["seqlen"]
    cuts = [r.uniform(0.1, 3.0) for _ in range(n)]
    if n > 12 and total < 65536:
        cuts[r.randrange(n)] = 0.0
    lengths = [int(total * c / sum(cuts)) for c in cuts]
    lengths[max(range(n), key=lengths.__getitem__)] += total - sum(lengths)
    return lengths


def prepare(case, seed):
    dev, dt, op = "cuda", DTYPES[case["dtype"]], case["op"]
    g = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape, scale=1.0, dtype=torch.float32):
        return (scale * torch.randn(shape, generator=g, device=dev)).to(dtype)

    s = {"op": op}
    if op in ("gn_fwd", "gn_bwd"):
        n, P, C, G = (case[k] for k in ("samples", "positions", "channels", "groups"))
        # every channel has an offset and a size of its own
        x = normal(n, P, C) * (0.5 + torch.rand(C, generator=g, device=dev)) + 0.3 * normal(C)
        s |= {"x": x.to(dt), "groups": G, "weight": 1 + normal(C, scale=0.2),
              "bias": normal(C, scale=0.2), "eps": 1e-5,
              "activation": "silu" if case["form"] == "silu" else None,
              "z": normal(n, P, C, dtype=dt) if case["form"] == "gate" else None}
        if op == "gn_bwd":
            xg = s["x"].double().view(n, P, G, C // G)
            mean = xg.mean((1, 3))
            var = (xg - mean[:, None, :, None]).square().mean((1, 3))
            s |= {"dy": normal(n, P, C, dtype=dt), "mean": mean.float(),
                  "rstd": torch.rsqrt(var + s["eps"]).float()}
        return s
    b, H, G, K, V = (case[k] for k in ("batch", "heads", "groups", "keys", "values"))
    # a head forgets over 32 tokens (the first) to 512 (the last)
    fades = torch.linspace(math.log(1 / 32), math.log(1 / 512), H, dtype=torch.float64)
    s |= {"decay": torch.log1p(-torch.exp(fades)).float().to(dev), "scale": K ** -0.5}
    if op == "lin_step":
        # a pool of states, the batch's in any order; the new states go to a second pool
        lead, sequences = (b,), b + case["spare"]
        s["slots"] = torch.randperm(sequences, generator=g, device=dev)[:b].to(torch.int32)
    else:
        L = case["seqlen"]
        lead, sequences, s["cu"] = (b, L), b, None
        if case["nseq"]:
            lengths = _lengths(case, seed)
            s["cu"] = torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32,
                                   device=dev)
            sequences = len(lengths)
    # q, k and v are views of one projection's output
    proj = normal(*lead, H * K + G * (K + V), dtype=dt)
    q, k, v = proj.split([H * K, G * K, G * V], dim=-1)
    s |= {"q": q.unflatten(-1, (H, K)), "k": k.unflatten(-1, (G, K)),
          "v": v.unflatten(-1, (G, V))}
    carried = op == "lin_step" or case["carry"]
    s["state"] = normal(sequences, H, K, V) if carried else None
    if op == "lin_bwd":
        s["dy"] = normal(*lead, H, V, dtype=dt)
        s["d_final"] = normal(sequences, H, K, V, scale=0.3) if carried else None
    if op == "lin_step":
        s["new_state"] = torch.zeros_like(s["state"])
    return s


def run(s):
    return (_own if own else _plain)[s["op"]](s)


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    op = case["op"]
    if op in ("gn_fwd", "gn_bwd"):
        n = case["samples"] * case["positions"] * case["channels"]
        gated = int(case["form"] == "gate")
        stats = 8 * case["samples"] * case["groups"]
        if op == "gn_fwd":
            return {"bytes": (2 + gated) * n * e + stats + 8 * case["channels"],
                    "flops": 8 * n + 6 * n * (case["form"] != "plain")}
        return {"bytes": (3 + 2 * gated) * n * e + stats + 16 * case["channels"],
                "flops": 16 * n + 12 * n * (case["form"] != "plain")}
    H, G, K, V = (case[k] for k in ("heads", "groups", "keys", "values"))
    tokens = case["batch"] * case.get("seqlen", 1)
    heads, shared = tokens * H * e, tokens * G * e
    if op == "lin_step":
        return {"bytes": 8 * tokens * H * K * V + (heads + shared) * (K + V) + 4 * H,
                "flops": 5 * tokens * H * K * V}
    state = 4 * (case["nseq"] or case["batch"]) * H * K * V
    if op == "lin_fwd":
        return {"bytes": (heads + shared) * (K + V) + state * (1 + case["carry"]) + 4 * H,
                "flops": 4 * tokens * H * K * V}
    # reads q, k, v, dy, writes dq, dk, dv, dinit_state
    return {"bytes": heads * (2 * K + V) + 2 * shared * (K + V) + state * (1 + 2 * case["carry"]),
            "flops": 10 * tokens * H * K * V}


# ---- the framework's calls -----------------------------------------------------------------

def _library():
    import mamba_ssd_chunked_02_amd as ssd
    return ssd


def _own_lin_fwd(s):
    return _library().ssd_linattn_fwd(s["q"], s["k"], s["v"], s["decay"], scale=s["scale"],
                                      init_state=s["state"], cu_seqlens=s["cu"])


def _own_lin_bwd(s):
    return _library().ssd_linattn_bwd(s["q"], s["k"], s["v"], s["decay"], s["dy"],
                                      scale=s["scale"], init_state=s["state"],
                                      cu_seqlens=s["cu"], d_final=s["d_final"])


def _own_lin_step(s):
    y = _library().ssd_linattn_step(s["q"], s["k"], s["v"], s["decay"], s["state"],
                                    scale=s["scale"], slots=s["slots"],
                                    new_state=s["new_state"])
    return y, s["new_state"]


def _own_gn_fwd(s):
    return _library().ssd_groupnorm_fwd(s["x"], s["groups"], s["weight"], s["bias"], z=s["z"],
                                        activation=s["activation"], eps=s["eps"])


def _own_gn_bwd(s):
    return _library().ssd_groupnorm_bwd(s["x"], s["groups"], s["weight"], s["bias"], s["mean"],
                                        s["rstd"], s["dy"], z=s["z"],
                                        activation=s["activation"])


_own = {"lin_fwd": _own_lin_fwd, "lin_bwd": _own_lin_bwd, "lin_step": _own_lin_step,
        "gn_fwd": _own_gn_fwd, "gn_bwd": _own_gn_bwd}


# ---- the plain forms -----------------------------------------------------------------------

def _powers(decay, n):
    """exp(n decay) for whole n >= 0 in float64, rounded to float32."""
    return torch.exp(n.double() * decay.double()).float()


def _spans(lead, cu, device):
    """First token and length of every sequence."""
    if cu is None:
        b, L = lead
        first = torch.arange(b, device=device) * L
        return first, torch.full_like(first, L)
    c = cu.long()
    return c[:-1], c[1:] - c[:-1]


def _linear(q, k, v, decay, cu, init, reverse, power):
    """Outputs q_t S_t (float32, tokens flat) and the states behind the last tokens, of
    S_t = exp(decay) S_(t-1) + k_t^T v_t over the tokens in order, or in reverse.  The state
    that comes in meets the first token times exp(power decay).  In blocks of CHUNK tokens:
    scores within a block, and a product with the state that enters it."""
    lead, H = q.shape[:2], decay.numel()
    T, dev = lead.numel(), q.device
    q, k, v = (t.reshape(T, t.shape[2], t.shape[3]).float() for t in (q, k, v))
    first, length = _spans(lead, cu, dev)
    S = first.numel()
    # block m is block `at` of sequence `seq`; m past the last block has no tokens
    count = (length + CHUNK - 1) // CHUNK
    ends = count.cumsum(0)
    M = T // CHUNK + S
    m = torch.arange(M, device=dev)
    seq = torch.searchsorted(ends, m, right=True).clamp(max=S - 1)
    at = m - (ends - count)[seq]
    step = at[:, None] * CHUNK + torch.arange(CHUNK, device=dev)
    inside = (step < length[seq][:, None]) & (m < ends[-1])[:, None]
    token = torch.where(inside, first[seq][:, None] + (length[seq][:, None] - 1 - step if reverse else step), 0)

    def blocks(t):
        t = torch.where(inside[..., None, None], t[token], torch.zeros((), device=dev))
        return t.repeat_interleave(H // t.shape[2], dim=2).transpose(1, 2)  # [M, H, CHUNK, .]

    qb, kb, vb = blocks(q), blocks(k), blocks(v)
    r = torch.arange(CHUNK, device=dev)
    back = r[:, None] - r
    fade = torch.where(back >= 0, _powers(decay[:, None, None], back.clamp(min=0)), 0.0)
    y = torch.matmul(torch.matmul(qb, kb.transpose(2, 3)) * fade, vb)
    # what each block adds to the state, as of its own last token
    filled = inside.sum(1)
    left = (filled[:, None] - 1 - r).clamp(min=0)
    add = torch.matmul((kb * _powers(decay[:, None], left[:, None])[..., None]).transpose(2, 3), vb)
    K, V = add.shape[2:]
    flat = add.transpose(0, 1).reshape(H, M, K * V)
    # the state entering block m, as of its first token
    gap = at[:, None] - at - 1
    earlier = (seq[:, None] == seq) & (gap >= 0)
    W = torch.where(earlier, _powers(decay[:, None, None], gap.clamp(min=0) * CHUNK + 1), 0.0)
    come = torch.matmul(W, flat).view(H, M, K, V).transpose(0, 1)
    if init is not None:
        come = come + init[seq] * _powers(decay, (at * CHUNK + power)[:, None])[..., None, None]
    y = y + torch.matmul(qb * _powers(decay[:, None], r)[..., None], come)
    # the states behind the last tokens
    sid = torch.arange(S, device=dev)
    rest = length[:, None] - at * CHUNK - filled
    mine = (sid[:, None] == seq) & (filled > 0)
    W = torch.where(mine, _powers(decay[:, None, None], rest.clamp(min=0)), 0.0)
    final = torch.matmul(W, flat).view(H, S, K, V).transpose(0, 1)
    if init is not None:
        before = (length + power - 1).clamp(min=0)
        kept = init * _powers(decay, before[:, None])[..., None, None]
        final = final + torch.where((length > 0)[:, None, None, None], kept, init)
    out = torch.zeros((T, H, V), device=dev)
    out[token[inside]] = y.transpose(1, 2)[inside]
    return out.view(*lead, H, V), final


def _plain_lin_fwd(s):
    y, final = _linear(s["q"], s["k"], s["v"], s["decay"], s["cu"], s["state"], False, 1)
    return (s["scale"] * y).to(s["q"].dtype), final


def _shared(d, G):
    """Gradients of heads summed over the heads of a group."""
    return d.unflatten(2, (G, -1)).sum(3)


def _plain_lin_bwd(s):
    q, k, v, dy, decay, cu, c = (s[n] for n in ("q", "k", "v", "dy", "decay", "cu", "scale"))
    dt, G, H = q.dtype, k.shape[2], q.shape[2]
    turned = None if s["state"] is None else s["state"].transpose(2, 3)
    dq, _ = _linear(dy, v, k, decay, cu, turned, False, 1)
    qs = q.float() * c
    df = s["d_final"]
    # R_t = qs_t^T dy_t + exp(decay) R_(t+1), to which d_final comes at the last token
    dv, R = _linear(k.repeat_interleave(H // G, 2), qs, dy, decay, cu, df, True, 0)
    dk, _ = _linear(v.repeat_interleave(H // G, 2), dy, qs, decay, cu,
                    None if df is None else df.transpose(2, 3), True, 0)
    _, length = _spans(q.shape[:2], cu, q.device)
    last = _powers(decay, (length > 0)[:, None].expand(-1, H))[..., None, None]
    return {"dq": (c * dq).to(dt), "dk": _shared(dk, G).to(dt), "dv": _shared(dv, G).to(dt),
            "dinit_state": R * last}


def _plain_lin_step(s):
    H, at = s["q"].shape[1], s["slots"].long()
    q, k, v = (s[n].float().repeat_interleave(H // s[n].shape[1], dim=1) for n in ("q", "k", "v"))
    h = torch.exp(s["decay"])[:, None, None] * s["state"][at] + k[..., None] * v[:, :, None]
    s["new_state"][at] = h
    return (s["scale"] * torch.matmul(q[:, :, None], h)[:, :, 0]).to(s["q"].dtype), s["new_state"]


def _normed(s):
    """(x - mean) rstd and u in float32, by group, and what goes with them."""
    n, P, C = s["x"].shape
    G = s["groups"]
    x = s["x"].float().view(n, P, G, C // G)
    if "mean" in s:
        mean, rstd = s["mean"], s["rstd"]
    else:
        mean = x.mean((1, 3))
        rstd = torch.rsqrt((x - mean[:, None, :, None]).square().mean((1, 3)) + s["eps"])
    xh = (x - mean[:, None, :, None]) * rstd[:, None, :, None]
    return xh, (xh.view(n, P, C) * s["weight"] + s["bias"]), mean, rstd


def _plain_gn_fwd(s):
    _, u, mean, rstd = _normed(s)
    if s["activation"] == "silu":
        u = u * torch.sigmoid(u)
    if s["z"] is not None:
        z = s["z"].float()
        u = u * (z * torch.sigmoid(z))
    return u.to(s["x"].dtype), mean, rstd


def _plain_gn_bwd(s):
    xh, u, _, rstd = _normed(s)
    n, P, C = s["x"].shape
    dt, du, out = s["x"].dtype, s["dy"].float(), {}
    if s["z"] is not None:
        z = s["z"].float()
        sig = torch.sigmoid(z)
        out["dz"] = (du * u * (sig * (1 + z * (1 - sig)))).to(dt)
        du = du * (z * sig)
    if s["activation"] == "silu":
        sig = torch.sigmoid(u)
        du = du * (sig * (1 + u * (1 - sig)))
    g = (du * s["weight"]).view(xh.shape)
    mean_g, mean_gx = g.mean((1, 3), keepdim=True), (g * xh).mean((1, 3), keepdim=True)
    dx = rstd[:, None, :, None] * (g - mean_g - xh * mean_gx)
    return out | {"dx": dx.view(n, P, C).to(dt), "dbias": du.sum((0, 1)),
                  "dweight": (du * xh.view(n, P, C)).sum((0, 1))}


_plain = {"lin_fwd": _plain_lin_fwd, "lin_bwd": _plain_lin_bwd, "lin_step": _plain_lin_step,
          "gn_fwd": _plain_gn_fwd, "gn_bwd": _plain_gn_bwd}


# ---- the definitions in float64 ------------------------------------------------------------

def _padded(t, bounds):
    """[sequences, longest, ...] in float64, zeros behind each sequence's end."""
    flat = t.reshape(-1, *t.shape[2:])
    out = flat.new_zeros((len(bounds), max(1, max(b - a for a, b in bounds)), *flat.shape[1:]),
                         dtype=torch.float64)
    for i, (a, b) in enumerate(bounds):
        out[i, :b - a] = flat[a:b]
    return out


def _flat(t, bounds, lead):
    return torch.cat([t[i, :b - a] for i, (a, b) in enumerate(bounds)]).reshape(*lead, *t.shape[2:])


def _exact_lin(case, s):
    b, L = s["q"].shape[:2]
    if s["cu"] is None:
        bounds = [(i * L, (i + 1) * L) for i in range(b)]
    else:
        cu = s["cu"].tolist()
        bounds = list(zip(cu[:-1], cu[1:]))
    H, G, c = case["heads"], case["groups"], s["scale"]
    lam = torch.exp(s["decay"].double())[:, None, None]
    q = _padded(s["q"], bounds)
    k, v = (_padded(s[n], bounds).repeat_interleave(H // G, 2) for n in ("k", "v"))
    S, longest = q.shape[:2]
    K, V = k.shape[-1], v.shape[-1]
    h = q.new_zeros((S, H, K, V)) if s["state"] is None else s["state"].double()
    ends = torch.tensor([z - a for a, z in bounds], device=q.device)
    least = min(z - a for a, z in bounds)
    if case["op"] == "lin_fwd":
        y = torch.zeros_like(v)
        for t in range(longest):
            new = torch.addcmul(lam * h, k[:, t, :, :, None], v[:, t, :, None])
            h = new if t < least else torch.where((t < ends)[:, None, None, None], new, h)
            y[:, t] = torch.matmul(q[:, t, :, None], h)[:, :, 0]
        return c * _flat(y, bounds, (b, L)), h
    dy = _padded(s["dy"], bounds)
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    for t in range(longest):
        h = torch.addcmul(lam * h, k[:, t, :, :, None], v[:, t, :, None])
        dq[:, t] = c * torch.matmul(h, dy[:, t, ..., None])[..., 0]
    # the gradient of the state behind token t
    R = q.new_zeros((S, H, K, V)) if s["d_final"] is None else s["d_final"].double()
    for t in reversed(range(longest)):
        new = torch.addcmul(R, c * q[:, t, :, :, None], dy[:, t, :, None])
        dk[:, t] = torch.matmul(new, v[:, t, ..., None])[..., 0]
        dv[:, t] = torch.matmul(k[:, t, :, None], new)[:, :, 0]
        R = lam * new if t < least else torch.where((t < ends)[:, None, None, None], lam * new, R)

    def shared(d):
        return d.view(*d.shape[:2], G, H // G, d.shape[-1]).sum(3)

    return {"dq": _flat(dq, bounds, (b, L)), "dk": _flat(shared(dk), bounds, (b, L)),
            "dv": _flat(shared(dv), bounds, (b, L)), "dinit_state": R}


def _exact_step(case, s):
    rep, at = case["heads"] // case["groups"], s["slots"].long()
    q = s["q"].double()
    k, v = (s[n].double().repeat_interleave(rep, 1) for n in ("k", "v"))
    h = torch.exp(s["decay"].double())[:, None, None] * s["state"].double()[at]
    h += k[..., None] * v[:, :, None]
    pool = s["new_state"].double()
    pool[at] = h
    return s["scale"] * (q[..., None] * h).sum(2), pool


def _exact_norm(case, s):
    n, P, C, G = (case[k] for k in ("samples", "positions", "channels", "groups"))
    x = s["x"].double().view(n, P, G, -1)
    N = P * (C // G)
    if case["op"] == "gn_bwd":
        mean, rstd = s["mean"].double(), s["rstd"].double()
    else:
        mean = x.sum((1, 3)) / N
        rstd = ((x - mean[:, None, :, None]).square().sum((1, 3)) / N + s["eps"]) ** -0.5
    xh = ((x - mean[:, None, :, None]) * rstd[:, None, :, None]).view(n, P, C)
    w, bias = s["weight"].double(), s["bias"].double()
    u = xh * w + bias
    z = None if s["z"] is None else s["z"].double()
    if case["op"] == "gn_fwd":
        if case["form"] == "silu":
            u = u / (1 + torch.exp(-u))
        if z is not None:
            u = u * z / (1 + torch.exp(-z))
        return u, mean, rstd
    du, out = s["dy"].double(), {}
    if z is not None:
        sig = 1 / (1 + torch.exp(-z))
        out["dz"] = du * u * (sig + z * sig * (1 - sig))
        du = du * z * sig
    if case["form"] == "silu":
        sig = 1 / (1 + torch.exp(-u))
        du = du * (sig + u * sig * (1 - sig))
    g = (du * w).view(n, P, G, -1)
    xg = xh.view(n, P, G, -1)
    s1, s2 = g.sum((1, 3), keepdim=True) / N, (g * xg).sum((1, 3), keepdim=True) / N
    dx = rstd[:, None, :, None] * (g - s1 - xg * s2)
    return out | {"dx": dx.reshape(n, P, C), "dbias": du.sum((0, 1)), "dweight": (du * xh).sum((0, 1))}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("gn"):
        return _exact_norm(case, s)
    return (_exact_step if case["op"] == "lin_step" else _exact_lin)(case, s)
