"""What is measured of the operators around the scan: the short causal convolution, the
selective scan with a learned decay per channel and state entry, their single-token forms,
the single-token form of the SSD scan, and layer norm; each forward and, where it is
trained, backward.

With ``own`` false, ``run`` computes an operator in its plain form (elementary torch
operations in float32, rounded once at the end); with ``own`` true it makes the calls of
``mamba_ssd_chunked_02_amd`` that a program makes.  ``exact`` gives the same outputs in
float64 from the recurrences, token by token.

Shapes: x [b, L, E] (packed: b = 1, sequences given by cu_seqlens), B and C [b, L, G, N],
decay rates A [N, E] (negative), states [sequences, N, E], convolution weight [W, E] and
state [sequences, W - 1, E].
"""
import math
import random

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
LOG2E = 1.4426950408889634


def listed():
    return [
        # prompts: 16 packed sequences of 256 to 8192 tokens through the convolution of a
        # Mamba-2 layer (24 heads x 64 channels and B, C of 128 states)
        {"name": "conv_prompts", "op": "conv_fwd", "dtype": "bf16", "batch": 1, "seqlen": 65536,
         "channels": 1792, "width": 4, "nseq": 16, "carry": True},
        # training: the same layer's gradients for 2 x 2048 tokens, in float32
        {"name": "conv_train", "op": "conv_bwd", "dtype": "f32", "batch": 2, "seqlen": 2048,
         "channels": 1792, "width": 4, "nseq": 0, "carry": False},
        # one new token for each of 64 sequences of a wide layer (80 x 64 + 2 x 128 channels)
        {"name": "conv_token", "op": "conv_step", "dtype": "bf16", "batch": 64, "channels": 5376,
         "width": 4, "spare": 0},
        # a short odd request in float32 that goes on from a state: latency
        {"name": "scan_short", "op": "scan_fwd", "dtype": "f32", "batch": 3, "seqlen": 77,
         "channels": 203, "states": 16, "groups": 1, "gated": True, "nseq": 0, "carry": True},
        # the layer workload: 2 x 2048 tokens, d_model 768 expanded twice
        {"name": "scan_layer", "op": "scan_fwd", "dtype": "bf16", "batch": 2, "seqlen": 2048,
         "channels": 1536, "states": 16, "groups": 1, "gated": True, "nseq": 0, "carry": False},
        # prompts: 16 packed sequences, 65536 tokens in all
        {"name": "scan_prompts", "op": "scan_fwd", "dtype": "bf16", "batch": 1, "seqlen": 65536,
         "channels": 1536, "states": 16, "groups": 1, "gated": True, "nseq": 16, "carry": True},
        # training: the layer workload's gradients
        {"name": "scan_train", "op": "scan_bwd", "dtype": "bf16", "batch": 2, "seqlen": 2048,
         "channels": 1536, "states": 16, "groups": 1, "gated": True, "nseq": 0, "carry": False},
        # one new token for each of 128 sequences, d_model 2560 expanded twice
        {"name": "scan_token", "op": "scan_step", "dtype": "bf16", "batch": 128, "channels": 5120,
         "states": 16, "groups": 1, "gated": True, "spare": 0},
        # one token of one sequence through the layer workload's scan: latency
        {"name": "ssd_token_one", "op": "ssd_step", "dtype": "bf16", "batch": 1, "heads": 24,
         "headdim": 64, "states": 128, "groups": 1, "spare": 0},
        # one new token for each of 64 sequences through the wide workload's scan
        {"name": "ssd_token_batch", "op": "ssd_step", "dtype": "bf16", "batch": 64, "heads": 80,
         "headdim": 64, "states": 128, "groups": 1, "spare": 0},
        # the norm in front of the layer workload's block
        {"name": "norm_layer", "op": "norm_fwd", "dtype": "bf16", "rows": 4096, "width": 768},
        # training: the norm's gradients at the wide workload's 8192 tokens
        {"name": "norm_train", "op": "norm_bwd", "dtype": "bf16", "rows": 8192, "width": 2560},
    ]


def _size(rng, lo, hi):
    """A whole number, evenly spread over the logarithm of [lo, hi]."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["conv_fwd", "conv_bwd", "conv_step", "scan_fwd", "scan_bwd", "scan_step",
                     "ssd_step", "norm_fwd", "norm_bwd"])
    case = {"op": op, "dtype": rng.choice(["bf16", "bf16", "f32"])}
    if op in ("norm_fwd", "norm_bwd"):
        width = _size(rng, 33, 16384)
        case |= {"rows": _size(rng, 1, 4e7 / width), "width": width}
    elif op == "ssd_step":
        groups = rng.choice([1, 1, 2])
        case |= {"batch": _size(rng, 1, 64), "heads": groups * _size(rng, 1, 24),
                 "headdim": 16 * rng.randint(1, 8), "states": rng.choice([16, 32, 64, 128]),
                 "groups": groups, "spare": rng.choice([0, 3])}
    elif op == "conv_step":
        case |= {"batch": _size(rng, 1, 256), "channels": _size(rng, 33, 8000),
                 "width": rng.choice([2, 3, 4]), "spare": rng.choice([0, 5])}
    elif op == "scan_step":
        groups = rng.choice([1, 1, 2])
        case |= {"batch": _size(rng, 1, 256), "channels": groups * _size(rng, 33, 2600),
                 "states": rng.choice([8, 16, 16, 32]), "groups": groups,
                 "gated": rng.random() < 0.7, "spare": rng.choice([0, 5])}
    else:
        packed = rng.random() < 0.5
        if op.startswith("conv"):
            channels, most = _size(rng, 33, 6000), 1.0e8
            case |= {"width": rng.choice([2, 3, 4, 4])}
        else:
            groups = rng.choice([1, 1, 2])
            states = rng.choice([8, 16, 16, 32])
            channels = groups * _size(rng, 33, 2600)
            most = (4.0e8 if op == "scan_fwd" else 1.0e8) / states
            case |= {"states": states, "groups": groups, "gated": rng.random() < 0.7}
        tokens = _size(rng, 1, min(65536, most / channels))
        batch = 1 if packed else min(tokens, rng.randint(1, 8))
        case |= {"batch": batch, "seqlen": tokens // batch, "channels": channels,
                 "nseq": rng.randint(1, 24) if packed else 0, "carry": rng.random() < 0.5}
    return case


def _lengths(case, seed):
    """Lengths of a packed batch's sequences; of more than twelve, one is empty."""
    r = random.Random(seed * 7919 + 17)
    n, total = case["nseq"], case["seqlen"]
    cuts = [r.uniform(0.1, 3.2) for _ in range(n)]
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
    if op.startswith("norm"):
        rows, width = case["rows"], case["width"]
        # rows of a residual stream: each with an offset and a size of its own
        x = normal(rows, width) * (0.5 + torch.rand((rows, 1), generator=g, device=dev))
        s |= {"x": (x + 0.3 * normal(rows, 1)).to(dt), "weight": 1 + normal(width, scale=0.2),
              "bias": normal(width, scale=0.2), "eps": 1e-5}
        if op == "norm_bwd":
            xf = s["x"].float()
            mean = xf.mean(1)
            s |= {"dy": normal(rows, width, dtype=dt), "mean": mean,
                  "rstd": torch.rsqrt((xf - mean[:, None]).square().mean(1) + s["eps"])}
        return s
    b = case["batch"]
    if op in ("conv_step", "scan_step", "ssd_step"):
        # a pool of states, the batch's in any order; the new states go to a second pool
        slots = torch.randperm(b + case["spare"], generator=g, device=dev)[:b].to(torch.int32)
        s["slots"], s["lead"] = slots, (b,)
        sequences = b + case["spare"]
    else:
        L = case["seqlen"]
        s["lead"], s["cu"] = (b, L), None
        sequences = b
        if case["nseq"]:
            lengths = _lengths(case, seed)
            s["cu"] = torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32,
                                   device=dev)
            sequences = len(lengths)
    lead = s["lead"]
    if op.startswith("conv"):
        E, W = case["channels"], case["width"]
        s |= {"x": normal(*lead, E, dtype=dt), "weight": normal(W, E, scale=W ** -0.5),
              "bias": normal(E, scale=0.3)}
        if op == "conv_step" or case["carry"]:
            s["state"] = normal(sequences, W - 1, E, dtype=dt)
        else:
            s["state"] = None
        if op == "conv_bwd":
            s["dy"] = normal(*lead, E, dtype=dt)
            s["d_final"] = normal(sequences, W - 1, E, dtype=dt) if case["carry"] else None
    elif op == "ssd_step":
        H, P, N, G = case["heads"], case["headdim"], case["states"], case["groups"]
        s |= {"x": normal(b, H, P, dtype=dt), "d_raw": normal(b, H, dtype=dt), "d_init": -4.6,
              "B": normal(b, G, N, dtype=dt), "C": normal(b, G, N, dtype=dt),
              "state": normal(sequences, H, N, P, scale=0.1)}
    else:
        E, N, G = case["channels"], case["states"], case["groups"]
        # the step's bias puts the steps between 0.001 and 0.1, and the decay rates start as
        # -1, -2, ... -N in every channel
        step = torch.exp(torch.rand(E, generator=g, device=dev) * math.log(100.0)) * 1e-3
        rates = torch.arange(1, N + 1, device=dev, dtype=torch.float32)[:, None]
        rank = max(1, E // 32)
        # B and C are views of one projection's output, behind the step's low-rank part
        proj = normal(*lead, rank + 2 * G * N, dtype=dt)
        B, C = (p.unflatten(-1, (G, N)) for p in proj[..., rank:].split(G * N, dim=-1))
        s |= {"x": normal(*lead, E, dtype=dt), "d_raw": normal(*lead, E, dtype=dt),
              "d_init": step + torch.log(-torch.expm1(-step)),
              "A": -rates * torch.exp(normal(N, E, scale=0.1)), "B": B, "C": C,
              "D": 1 + normal(E, scale=0.1),
              "z": normal(*lead, E, dtype=dt) if case["gated"] else None}
        if op == "scan_step" or case["carry"]:
            s["state"] = normal(sequences, N, E, scale=0.3)
        else:
            s["state"] = None
        if op == "scan_bwd":
            s["dy"] = normal(*lead, E, dtype=dt)
            s["d_final"] = normal(sequences, N, E, scale=0.3) if case["carry"] else None
    if op.endswith("step"):
        s["new_state"] = torch.zeros_like(s["state"])
    return s


def run(s):
    return (_own if own else _plain)[s["op"]](s)


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    op = case["op"]
    if op.startswith("norm"):
        n = case["rows"] * case["width"]
        if op == "norm_fwd":
            return {"bytes": 2 * n * e + 8 * case["rows"] + 8 * case["width"], "flops": 8 * n}
        return {"bytes": 3 * n * e + 8 * case["rows"] + 12 * case["width"], "flops": 14 * n}
    b = case["batch"]
    if op == "ssd_step":
        heads = b * case["heads"]
        state = heads * case["states"] * case["headdim"]
        rows = heads * (2 * case["headdim"] + 1) + 2 * b * case["groups"] * case["states"]
        return {"bytes": 8 * state + rows * e, "flops": 5 * state}
    E = case["channels"]
    if op == "conv_step":
        W = case["width"]
        return {"bytes": b * E * e * (2 * (W - 1) + 2) + 4 * (W + 1) * E,
                "flops": b * E * (2 * W + 5)}
    tokens = b * case.get("seqlen", 1)
    sequences = case.get("nseq") or b
    if op.startswith("conv"):
        W = case["width"]
        state = sequences * (W - 1) * E * e * case["carry"]
        if op == "conv_fwd":
            return {"bytes": 2 * tokens * E * e + 4 * (W + 1) * E + state + sequences * (W - 1) * E * e,
                    "flops": tokens * E * (2 * W + 5)}
        return {"bytes": 3 * tokens * E * e + 8 * (W + 1) * E + 3 * state,
                "flops": tokens * E * (6 * W + 12)}
    N, gated = case["states"], int(case["gated"])
    BC = 2 * tokens * case["groups"] * N * e
    if op == "scan_step":
        return {"bytes": 8 * b * N * E + b * E * e * (3 + gated) + BC + 4 * E * (N + 2),
                "flops": 7 * b * N * E + 16 * b * E}
    state = 4 * sequences * N * E
    if op == "scan_fwd":
        return {"bytes": tokens * E * e * (3 + gated) + BC + 4 * E * (N + 2) + state * (1 + case["carry"]),
                "flops": 7 * tokens * N * E + 16 * tokens * E}
    return {"bytes": tokens * E * e * (5 + 2 * gated) + 2 * BC + 8 * E * (N + 2) + 3 * state * case["carry"],
            "flops": 20 * tokens * N * E + 40 * tokens * E}


# ---- the framework's calls -----------------------------------------------------------------

def _library():
    import mamba_ssd_chunked_02_amd as ssd
    return ssd


def _own_conv_fwd(s):
    return _library().ssd_conv_fwd(s["x"], s["weight"], s["bias"], init_state=s["state"],
                                   cu_seqlens=s["cu"])


def _own_conv_bwd(s):
    return _library().ssd_conv_bwd(s["x"], s["weight"], s["bias"], s["dy"], init_state=s["state"],
                                   cu_seqlens=s["cu"], d_final=s["d_final"])


def _own_conv_step(s):
    y = _library().ssd_conv_step(s["x"], s["state"], s["weight"], s["bias"], slots=s["slots"],
                                 new_state=s["new_state"])
    return y, s["new_state"]


def _own_scan_fwd(s):
    return _library().ssd_selscan_fwd(s["x"], s["d_raw"], s["d_init"], s["A"], s["B"], s["C"],
                                      D=s["D"], z=s["z"], init_state=s["state"],
                                      cu_seqlens=s["cu"])


def _own_scan_bwd(s):
    return _library().ssd_selscan_bwd(s["x"], s["d_raw"], s["d_init"], s["A"], s["B"], s["C"],
                                      s["dy"], D=s["D"], z=s["z"], init_state=s["state"],
                                      cu_seqlens=s["cu"], d_final=s["d_final"])


def _own_scan_step(s):
    y = _library().ssd_selscan_step(s["x"], s["d_raw"], s["d_init"], s["A"], s["B"], s["C"],
                                    s["state"], D=s["D"], z=s["z"], slots=s["slots"],
                                    new_state=s["new_state"])
    return y, s["new_state"]


def _own_ssd_step(s):
    y = _library().ssd_step(s["x"], s["d_raw"], s["d_init"], s["B"], s["C"], s["state"],
                            slots=s["slots"], new_state=s["new_state"])
    return y, s["new_state"]


def _own_norm_fwd(s):
    return _library().ssd_norm_fwd(s["x"], s["weight"], s["bias"], eps=s["eps"])


def _own_norm_bwd(s):
    return _library().ssd_norm_bwd(s["x"], s["weight"], s["mean"], s["rstd"], s["dy"])


_own = {"conv_fwd": _own_conv_fwd, "conv_bwd": _own_conv_bwd, "conv_step": _own_conv_step,
        "scan_fwd": _own_scan_fwd, "scan_bwd": _own_scan_bwd, "scan_step": _own_scan_step,
        "ssd_step": _own_ssd_step, "norm_fwd": _own_norm_fwd, "norm_bwd": _own_norm_bwd}


# ---- the plain forms -----------------------------------------------------------------------

def _sequences(s):
    """For each of the flattened tokens its sequence and that sequence's first and last token."""
    T = s["x"].shape[:-1].numel()
    t = torch.arange(T, device=s["x"].device)
    if s["cu"] is None:
        L = s["x"].shape[1]
        q = t // L
        first = torch.arange(0, T, L, device=t.device)
        last = first + L - 1
    else:
        cu = s["cu"].long()
        q = torch.searchsorted(cu[1:].contiguous(), t, right=True)
        first, last = cu[:-1], cu[1:] - 1
    return t, q, first, last


def _silu_slope(v):
    sig = torch.sigmoid(v)
    return sig * (1 + v * (1 - sig))


def _conv_inputs(s):
    """Every token's W inputs [T, W, E] in float32: its sequence's, or its initial state's."""
    W, E = s["weight"].shape
    t, q, first, _ = _sequences(s)
    x = s["x"].reshape(-1, E).float()
    back = torch.arange(W - 1, -1, -1, device=t.device)
    at = t[:, None] - back
    before = at < first[q][:, None]
    taken = x[at.clamp(min=0)]
    if s["state"] is None:
        return torch.where(before[..., None], torch.zeros((), device=t.device), taken), at, before
    # position -1 of a sequence is the state's last row
    row = (at - first[q][:, None] + W - 1).clamp(0, W - 2)
    carried = s["state"].float()[q[:, None].expand_as(row), row]
    return torch.where(before[..., None], carried, taken), at, before


def _plain_conv_fwd(s):
    W, E = s["weight"].shape
    taken, _, _ = _conv_inputs(s)
    v = (taken * s["weight"]).sum(1) + s["bias"]
    y = (v * torch.sigmoid(v)).to(s["x"].dtype).reshape(s["x"].shape)
    # the last W - 1 inputs of each sequence, its initial state's rows where it is shorter
    _, _, first, last = _sequences(s)
    at = last[:, None] - torch.arange(W - 2, -1, -1, device=y.device)
    x = s["x"].reshape(-1, E)
    final = x[at.clamp(0, x.shape[0] - 1)]
    before = at < first[:, None]
    if s["state"] is None:
        carried = torch.zeros_like(final)
    else:
        row = (at - first[:, None] + W - 1).clamp(0, W - 2)
        carried = torch.gather(s["state"], 1, row[..., None].expand(-1, -1, E))
    return y, torch.where(before[..., None], carried, final)


def _plain_conv_bwd(s):
    W, E = s["weight"].shape
    taken, at, before = _conv_inputs(s)
    t, q, first, last = _sequences(s)
    v = (taken * s["weight"]).sum(1) + s["bias"]
    dv = s["dy"].reshape(-1, E).float() * _silu_slope(v)
    # the input of token t meets tap W - 1 - k of token t + k, in the same sequence
    ahead = t[:, None] + torch.arange(W - 1, -1, -1, device=t.device)
    inside = ahead <= last[q][:, None]
    dx = (torch.where(inside[..., None], dv[ahead.clamp(max=t.numel() - 1)],
                      torch.zeros((), device=t.device)) * s["weight"]).sum(1)
    out = {"dweight": (taken * dv[:, None]).sum(0), "dbias": dv.sum(0)}
    # gradients of the states: rows that lie in front of the sequence
    S = first.numel()
    dinit = torch.zeros((S, W - 1, E), device=t.device)
    i, k = before.nonzero(as_tuple=True)
    dinit.index_put_((q[i], at[i, k] - first[q[i]] + W - 1), dv[i] * s["weight"][k], accumulate=True)
    if s["d_final"] is not None:
        df = s["d_final"].float()
        at = last[:, None] - torch.arange(W - 2, -1, -1, device=t.device)
        front = (at < first[:, None])[..., None]
        none = torch.zeros((), device=t.device)
        row = (at - first[:, None] + W - 1).clamp(0, W - 2)
        dinit.index_put_((torch.arange(S, device=t.device)[:, None].expand_as(row), row),
                         torch.where(front, df, none), accumulate=True)
        dx.index_put_((at.clamp(0, max(t.numel() - 1, 0)),), torch.where(front, none, df), accumulate=True)
    dt = s["x"].dtype
    return out | {"dx": dx.to(dt).reshape(s["x"].shape), "dinit_state": dinit.to(dt)}


def _plain_conv_step(s):
    W = s["weight"].shape[0]
    slots = s["slots"].long()
    taken = torch.cat([s["state"][slots], s["x"][:, None]], dim=1)
    v = (taken.float() * s["weight"]).sum(1) + s["bias"]
    s["new_state"][slots] = taken[:, 1:]
    return (v * torch.sigmoid(v)).to(s["x"].dtype), s["new_state"]


def _softplus(z):
    return z.clamp(min=0) + torch.log1p(torch.exp(-z.abs()))


def _running(a, b):
    """h_t = a_t h_{t-1} + b_t along dim 0 (h_{-1} = 0), by doubling; writes over a and b."""
    k, T = 1, a.shape[0]
    while k < T:
        b[k:] = torch.addcmul(b[k:], a[k:], b[:-k])
        a[k:] = a[k:] * a[:-k]
        k *= 2
    return b


def _per_channel(m, E):
    """[T, G, N] -> [T, N, E]: each channel its group's row."""
    T, G, N = m.shape
    return m[:, :, :, None].expand(T, G, N, E // G).transpose(1, 2).reshape(T, N, E)


def _scan_parts(s):
    """Steps, decays and states of every token, in float32 [T, (N,) E]."""
    E = s["x"].shape[-1]
    _, q, first, last = _sequences(s)
    z = s["d_raw"].reshape(-1, E).float() + s["d_init"]
    x = s["x"].reshape(-1, E).float()
    d = _softplus(z)
    a = torch.exp(d[:, None] * s["A"])
    B = _per_channel(s["B"].flatten(0, 1).float(), E)
    b = B * (d * x)[:, None]
    some = last >= first
    if s["state"] is not None:
        b[first[some]] += a[first[some]] * s["state"][some]
    a0 = a.clone()
    a0[first[some]] = 0
    return {"z": z, "x": x, "d": d, "a": a, "B": B, "h": _running(a0, b), "q": q, "first": first,
            "last": last, "some": some}


def _scan_output(s, p):
    E = s["x"].shape[-1]
    C = _per_channel(s["C"].flatten(0, 1).float(), E)
    return C, (C * p["h"]).sum(1) + s["D"] * p["x"]


def _plain_scan_fwd(s):
    E = s["x"].shape[-1]
    p = _scan_parts(s)
    _, y = _scan_output(s, p)
    if s["z"] is not None:
        z = s["z"].reshape(-1, E).float()
        y = y * (z * torch.sigmoid(z))
    S, N = p["first"].numel(), s["A"].shape[0]
    final = torch.zeros((S, N, E), device=y.device) if s["state"] is None else s["state"].clone()
    final[p["some"]] = p["h"][p["last"][p["some"]]]
    return y.to(s["x"].dtype).reshape(s["x"].shape), final


def _plain_scan_bwd(s):
    E, N = s["x"].shape[-1], s["A"].shape[0]
    G, dt = s["B"].shape[2], s["x"].dtype
    p = _scan_parts(s)
    C, v = _scan_output(s, p)
    a, h, d, x, first, last, some = (p[k] for k in ("a", "h", "d", "x", "first", "last", "some"))
    dy = s["dy"].reshape(-1, E).float()
    out = {}
    if s["z"] is not None:
        z = s["z"].reshape(-1, E).float()
        out["dz"] = (dy * v * _silu_slope(z)).to(dt).reshape(s["x"].shape)
        dy = dy * (z * torch.sigmoid(z))
    # the gradient of every token's state: g_t = C_t dy_t + a_{t+1} g_{t+1}
    g = C * dy[:, None]
    after = torch.zeros_like(a)
    after[:-1] = a[1:]
    after[last[some]] = 0
    if s["d_final"] is not None:
        g[last[some]] += s["d_final"][some]
    g = _running(after.flip(0), g.flip(0)).flip(0)
    before = torch.zeros_like(h)
    before[1:] = h[:-1]
    before[first[some]] = 0 if s["state"] is None else s["state"][some]
    T = x.shape[0]
    groups = (T, N, G, E // G)
    slope = g * a * before
    gB = (g * p["B"]).sum(1)
    dd = x * gB + (slope * s["A"]).sum(1)
    dd_raw = dd * torch.sigmoid(p["z"])
    dinit = torch.zeros((first.numel(), N, E), device=x.device)
    if s["d_final"] is not None:
        dinit += s["d_final"]
    dinit[some] = a[first[some]] * g[first[some]]
    shape = s["x"].shape
    return out | {
        "dx": (dy * s["D"] + d * gB).to(dt).reshape(shape),
        "dd_raw": dd_raw.to(dt).reshape(shape),
        "dd_init": dd_raw.sum(0),
        "dA": (d[:, None] * slope).sum(0),
        "dB": (g * (d * x)[:, None]).reshape(groups).sum(3).transpose(1, 2).to(dt).reshape(s["B"].shape),
        "dC": (h * dy[:, None]).reshape(groups).sum(3).transpose(1, 2).to(dt).reshape(s["C"].shape),
        "dD": (dy * x).sum(0),
        "dinit_state": dinit,
    }


def _plain_scan_step(s):
    E = s["x"].shape[-1]
    slots = s["slots"].long()
    x = s["x"].float()
    d = _softplus(s["d_raw"].float() + s["d_init"])
    h = torch.exp(d[:, None] * s["A"]) * s["state"][slots] + _per_channel(s["B"].float(), E) * (d * x)[:, None]
    s["new_state"][slots] = h
    y = (_per_channel(s["C"].float(), E) * h).sum(1) + s["D"] * x
    if s["z"] is not None:
        z = s["z"].float()
        y = y * (z * torch.sigmoid(z))
    return y.to(s["x"].dtype), s["new_state"]


def _plain_ssd_step(s):
    H, G = s["x"].shape[1], s["B"].shape[1]
    slots = s["slots"].long()
    d = _softplus(s["d_raw"].float() + s["d_init"])
    B, C = (s[k].float().repeat_interleave(H // G, dim=1) for k in ("B", "C"))
    h = torch.exp(-d)[:, :, None, None] * s["state"][slots] \
        + B[..., None] * (d[..., None] * s["x"].float())[:, :, None]
    s["new_state"][slots] = h
    return (C[..., None] * h).sum(2).to(s["x"].dtype), s["new_state"]


def _plain_norm_fwd(s):
    x = s["x"].float()
    mean = x.mean(1)
    centred = x - mean[:, None]
    rstd = torch.rsqrt(centred.square().mean(1) + s["eps"])
    return (centred * rstd[:, None] * s["weight"] + s["bias"]).to(s["x"].dtype), mean, rstd


def _plain_norm_bwd(s):
    dy = s["dy"].float()
    xhat = (s["x"].float() - s["mean"][:, None]) * s["rstd"][:, None]
    dxhat = dy * s["weight"]
    dx = s["rstd"][:, None] * (dxhat - dxhat.mean(1, keepdim=True)
                               - xhat * (dxhat * xhat).mean(1, keepdim=True))
    return {"dx": dx.to(s["x"].dtype), "dweight": (dy * xhat).sum(0), "dbias": dy.sum(0)}


_plain = {"conv_fwd": _plain_conv_fwd, "conv_bwd": _plain_conv_bwd, "conv_step": _plain_conv_step,
          "scan_fwd": _plain_scan_fwd, "scan_bwd": _plain_scan_bwd, "scan_step": _plain_scan_step,
          "ssd_step": _plain_ssd_step, "norm_fwd": _plain_norm_fwd, "norm_bwd": _plain_norm_bwd}


# ---- the definitions, token by token in float64 ----------------------------------------------

def _spans(s):
    """(first flattened token, length) of every sequence."""
    if s["cu"] is None:
        b, L = s["x"].shape[:2]
        return [(i * L, L) for i in range(b)]
    cu = s["cu"].tolist()
    return [(u, v - u) for u, v in zip(cu[:-1], cu[1:])]


def _exact_conv(s):
    W, E = s["weight"].shape
    op, w, bias = s["op"], s["weight"].double(), s["bias"].double()
    if op == "conv_step":
        new, y = s["new_state"].double(), []
        for i, slot in enumerate(s["slots"].tolist()):
            window = torch.cat([s["state"][slot].double(), s["x"][i:i + 1].double()])
            v = bias + torch.einsum("we,we->e", window, w)
            y.append(v / (1 + torch.exp(-v)))
            new[slot] = window[1:]
        return torch.stack(y), new
    x = s["x"].reshape(-1, E).double()
    y, final = torch.zeros_like(x), []
    dx, dw, db, dinit = torch.zeros_like(x), torch.zeros_like(w), torch.zeros_like(bias), []
    for i, (u, n) in enumerate(_spans(s)):
        front = torch.zeros((W - 1, E), dtype=torch.float64, device=x.device) if s["state"] is None \
            else s["state"][i].double()
        line = torch.cat([front, x[u:u + n]])
        final.append(line[n:])
        v = bias.repeat(n, 1)
        for k in range(W):
            v = v + line[k:k + n] * w[k]
        sig = 1 / (1 + torch.exp(-v))
        y[u:u + n] = v * sig
        if op == "conv_bwd":
            dv = s["dy"].reshape(-1, E)[u:u + n].double() * (sig + v * sig * (1 - sig))
            dline = torch.zeros_like(line)
            for k in range(W):
                dline[k:k + n] += dv * w[k]
                dw[k] += (dv * line[k:k + n]).sum(0)
            if s["d_final"] is not None:
                dline[n:] += s["d_final"][i].double()
            db += dv.sum(0)
            dx[u:u + n] = dline[W - 1:]
            dinit.append(dline[:W - 1])
    if op == "conv_fwd":
        return y.reshape(s["x"].shape), torch.stack(final)
    return {"dx": dx.reshape(s["x"].shape), "dweight": dw, "dbias": db, "dinit_state": torch.stack(dinit)}


def _exact_scan(s):
    op, A = s["op"], s["A"].double()
    N, E = A.shape
    G = s["B"].shape[-2]
    dev = A.device
    group = torch.arange(E, device=dev) // (E // G)
    if op == "scan_step":
        spans = [(i, 1) for i in range(s["x"].shape[0])]
        start = s["state"][s["slots"].long()].double()
    else:
        spans = _spans(s)
        start = torch.zeros((len(spans), N, E), dtype=torch.float64, device=dev) if s["state"] is None \
            else s["state"].double()
    flat = {k: s[k].reshape(-1, E).double() for k in ("x", "d_raw", "z", "dy") if s.get(k) is not None}
    Bm, Cm = (s[k].reshape(-1, G, N).double() for k in ("B", "C"))
    x, raw = flat["x"], flat["d_raw"] + s["d_init"].double()
    d = torch.logaddexp(raw, torch.zeros_like(raw))
    D = s["D"].double()
    # sequences side by side, longest first, one token of each at a time
    order = sorted(range(len(spans)), key=lambda i: -spans[i][1])
    heads = torch.tensor([spans[i][0] for i in order], device=dev)
    sizes = [spans[i][1] for i in order]
    alive = [sum(n > t for n in sizes) for t in range(sizes[0])]
    h = start[torch.tensor(order, device=dev)].clone()
    y = D * x
    train = op == "scan_bwd"
    kept = []
    for t, m in enumerate(alive):
        at = heads[:m] + t
        if train:
            kept.append(h[:m].clone())
        b, c = Bm[at][:, group].transpose(1, 2), Cm[at][:, group].transpose(1, 2)
        dt = d[at][:, None]
        h[:m] = torch.exp(dt * A) * h[:m] + dt * b * x[at][:, None]
        y[at] += (c * h[:m]).sum(1)
    back = torch.empty(len(order), dtype=torch.long, device=dev)
    back[torch.tensor(order, device=dev)] = torch.arange(len(order), device=dev)
    if "z" in flat:
        sig = torch.sigmoid(flat["z"])
        gate = flat["z"] * sig
    else:
        gate = torch.ones_like(x)
    if not train:
        out = (y * gate).reshape(s["x"].shape)
        if op == "scan_fwd":
            return out, h[back]
        new = s["new_state"].double()
        new[s["slots"].long()] = h[back]
        return out, new
    dyv = flat["dy"] * gate
    res = {"dx": dyv * D, "dd_raw": torch.zeros_like(x), "dB": torch.zeros_like(Bm), "dC": torch.zeros_like(Cm),
           "dA": torch.zeros_like(A), "dD": (dyv * x).sum(0)}
    if "z" in flat:
        res["dz"] = flat["dy"] * y * (sig + gate * (1 - sig))
    g = torch.zeros_like(h) if s["d_final"] is None else s["d_final"].double()[torch.tensor(order, device=dev)]
    for t in range(len(alive) - 1, -1, -1):
        m = alive[t]
        at, old = heads[:m] + t, kept[t]
        b, c = Bm[at][:, group].transpose(1, 2), Cm[at][:, group].transpose(1, 2)
        dt, xt, gy = d[at][:, None], x[at][:, None], dyv[at][:, None]
        a = torch.exp(dt * A)
        now = a * old + dt * b * xt
        gt = g[:m] + c * gy
        res["dC"][at] = (now * gy).reshape(m, N, G, -1).sum(3).transpose(1, 2)
        res["dB"][at] = (gt * dt * xt).reshape(m, N, G, -1).sum(3).transpose(1, 2)
        res["dx"][at] += (gt * dt * b).sum(1)
        res["dd_raw"][at] = (gt * (b * xt + A * a * old)).sum(1) * torch.sigmoid(raw[at])
        res["dA"] += (gt * dt * a * old).sum(0)
        g[:m] = gt * a
    res["dd_init"] = res["dd_raw"].sum(0)
    res["dinit_state"] = g[back]
    like = {"dx": "x", "dd_raw": "x", "dz": "x", "dB": "B", "dC": "C"}
    return {k: v.reshape(s[like[k]].shape) if k in like else v for k, v in res.items()}


def _exact_ssd_step(s):
    H, G = s["x"].shape[1], s["B"].shape[1]
    group = torch.arange(H, device=s["x"].device) // (H // G)
    raw = s["d_raw"].double() + s["d_init"]
    new, y = s["new_state"].double(), []
    for i, slot in enumerate(s["slots"].tolist()):
        d = torch.logaddexp(raw[i], torch.zeros_like(raw[i]))
        outer = torch.einsum("hn,hp->hnp", s["B"][i].double()[group], s["x"][i].double())
        h = torch.exp(-d)[:, None, None] * s["state"][slot].double() + d[:, None, None] * outer
        new[slot] = h
        y.append(torch.einsum("hn,hnp->hp", s["C"][i].double()[group], h))
    return torch.stack(y), new


def _exact_norm(s):
    x, w = s["x"].double(), s["weight"].double()
    if s["op"] == "norm_fwd":
        var, mean = torch.var_mean(x, dim=1, correction=0)
        rstd = 1 / torch.sqrt(var + s["eps"])
        return (x - mean[:, None]) * rstd[:, None] * w + s["bias"].double(), mean, rstd
    rstd = s["rstd"].double()[:, None]
    hat, dy = (x - s["mean"].double()[:, None]) * rstd, s["dy"].double()
    v = dy * w
    n = x.shape[1]
    dx = rstd / n * (n * v - v.sum(1, keepdim=True) - hat * (v * hat).sum(1, keepdim=True))
    return {"dx": dx, "dweight": torch.einsum("re,re->e", dy, hat), "dbias": dy.sum(0)}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op.startswith("conv"):
        return _exact_conv(s)
    if op.startswith("scan"):
        if case.get("seqlen", 1) * case["channels"] * case["states"] > 4e8 and op == "scan_bwd":
            return None
        return _exact_scan(s)
    return _exact_ssd_step(s) if op == "ssd_step" else _exact_norm(s)
