"""Cases of the selective state space layer's operators, as a user's program calls them.

Five operators, named by a case's "op":

  scan_fwd   the selective scan over prompts or training sequences: y and the final states
  scan_bwd   its gradients with respect to every input, the parameters and the initial states
  scan_step  one token of every sequence on a pool of states (decode)
  conv_bwd   the gradients of the short causal depthwise convolution in front of the scan
  q4_matvec  a few rows times a matrix of 4-bit weights with group scales (the projections of a decode step)

`own` chooses between the plain form (elementary torch operations in 32 bits) and the
framework's entry points; `exact` evaluates the definitions token by token in 64 bits.
"""
import math
import random

import torch

own = False

DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one long prompt of a 32 x 128-channel layer
        {"name": "scan_fwd one prompt", "op": "scan_fwd", "B": 1, "T": 4096, "D": 4096, "S": 16, "G": 1,
         "dtype": "bf16", "gate": True, "init": False},
        # the forward half of a training step on long sequences
        {"name": "scan_fwd training batch", "op": "scan_fwd", "B": 4, "T": 8192, "D": 4096, "S": 16, "G": 1,
         "dtype": "bf16", "gate": True, "init": False},
        # packed prompts of very different lengths that continue earlier states, in fp32
        {"name": "scan_fwd packed", "op": "scan_fwd", "packed": 64, "longest": 2048, "D": 2048, "S": 8, "G": 2,
         "dtype": "f32", "gate": False, "init": True},
        # the backward half of a training step
        {"name": "scan_bwd training batch", "op": "scan_bwd", "B": 4, "T": 4096, "D": 4096, "S": 16, "G": 1,
         "dtype": "bf16", "gate": True, "init": False},
        # packed training sequences, odd sizes, gradients down to the initial states
        {"name": "scan_bwd packed, odd", "op": "scan_bwd", "packed": 13, "longest": 1500, "D": 1000, "S": 12, "G": 4,
         "dtype": "f32", "gate": True, "init": True},
        # decode, a single request: latency
        {"name": "scan_step 1 request", "op": "scan_step", "N": 1, "slots": 8, "D": 4096, "S": 16, "G": 1,
         "dtype": "bf16", "gate": True},
        # decode, a full batch on a larger pool
        {"name": "scan_step 512 requests", "op": "scan_step", "N": 512, "slots": 640, "D": 4096, "S": 16, "G": 1,
         "dtype": "bf16", "gate": True},
        # the convolution in front of a 32-head layer (2 * 32 * 128 + 32 * 128 channels), training
        {"name": "conv_bwd training batch", "op": "conv_bwd", "B": 4, "T": 8192, "D": 12288, "W": 4, "act": "silu",
         "dtype": "bf16", "init": False},
        # packed sequences, odd sizes, gradients of the initial inputs too
        {"name": "conv_bwd packed, odd", "op": "conv_bwd", "packed": 37, "longest": 1000, "D": 1048, "W": 3,
         "act": "silu", "dtype": "f32", "init": True},
        # a square projection of one token: latency
        {"name": "q4_matvec 1 row", "op": "q4_matvec", "M": 1, "N": 4096, "K": 4096, "group": 128, "dtype": "bf16",
         "scales": "bf16", "zeros": False},
        # a wide projection of a few requests, small groups with zero points
        {"name": "q4_matvec 5 rows", "op": "q4_matvec", "M": 5, "N": 12288, "K": 4096, "group": 32, "dtype": "bf16",
         "scales": "bf16", "zeros": True},
        # a large matrix and a decode batch
        {"name": "q4_matvec 32 rows", "op": "q4_matvec", "M": 32, "N": 16384, "K": 8192, "group": 128,
         "dtype": "bf16", "scales": "bf16", "zeros": False},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _size(v):
    return v + 8 if v == 3072 else v


def draw(rng):
    op = rng.choice(["scan_fwd", "scan_bwd", "scan_step", "conv_bwd", "q4_matvec"])
    c = {"op": op, "dtype": rng.choice(["bf16", "bf16", "f32"])}
    if op == "q4_matvec":
        group = rng.choice([32, 64, 128])
        k = group * _log(rng, 1, 8192 // group)
        return {**c, "M": _log(rng, 1, 32), "N": _size(_log(rng, 17, 16384)),
                "K": k + group if k == 3072 else k, "group": group,
                "scales": rng.choice(["bf16", "f32"]), "zeros": rng.random() < 0.5}
    if op == "conv_bwd":
        c |= {"W": rng.choice([2, 3, 4]), "act": rng.choice(["silu", "none"]), "D": _size(8 * _log(rng, 8, 1024)),
              "init": rng.random() < 0.5}
        most = (1 << 27) // c["D"]
    else:
        G = rng.choice([1, 1, 2, 4])
        c |= {"G": G, "S": rng.choice([4, 8, 16, 16, 24, 32]), "D": _size(G * _log(rng, 64 // G, 6144 // G)),
              "gate": rng.random() < 0.7}
        if op == "scan_step":
            n = _log(rng, 1, 512)
            return {**c, "N": n, "slots": n + rng.randrange(0, 100)}
        c["init"] = rng.random() < 0.5
        most = (1 << 29) // (c["D"] * c["S"])
    tokens = _size(_log(rng, 16, max(32, min(16384, most))))
    if rng.random() < 0.5:
        n = rng.randrange(2, 65)
        return {**c, "packed": n, "longest": _size(max(2, 5 * tokens // n))}
    B = _log(rng, 1, min(8, tokens))
    return {**c, "B": B, "T": _size(max(1, tokens // B))}


def _lengths(c):
    """Token counts of the case's sequences: all alike, or log-uniform in [1, longest] for packed ones."""
    if "B" in c:
        return [c["T"]] * c["B"]
    r = random.Random("%s %s" % (c["packed"], c["longest"]))
    return [_log(r, 1, c["longest"]) for _ in range(c["packed"])]


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    dt = DT[c["dtype"]]

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=DEV)

    def rand(*shape):
        return torch.rand(*shape, generator=g, device=DEV)

    if c["op"] == "q4_matvec":
        M, N, K, gr = c["M"], c["N"], c["K"], c["group"]
        return {"case": c, "x": randn(M, K).to(dt),
                "qweight": torch.randint(0, 256, (N, K // 2), generator=g, device=DEV, dtype=torch.uint8),
                "scales": ((0.5 + rand(N, K // gr)) * (0.2 * K ** -0.5)).to(DT[c["scales"]]),
                "zeros": torch.randint(6, 11, (N, K // gr), generator=g, device=DEV, dtype=torch.uint8)
                if c["zeros"] else None,
                "bias": 0.1 * randn(N)}
    D = c["D"]
    if c["op"] == "scan_step":
        N, lens, cu = c["N"], [1] * c["N"], None
        lead = (N, 1)
    else:
        lens = _lengths(c)
        N = len(lens)
        if "B" in c:
            cu, lead = None, (c["B"], c["T"])
        else:
            cu = torch.tensor([sum(lens[:i]) for i in range(N + 1)], dtype=torch.int32, device=DEV)
            lead = (1, sum(lens))
    s = {"case": c, "cu": cu, "lens": lens, "x": randn(*lead, D).to(dt)}
    if c["op"] == "conv_bwd":
        W = c["W"]
        s |= {"weight": randn(D, W) * W ** -0.5, "bias": 0.1 * randn(D), "dout": randn(*lead, D).to(dt),
              "init": randn(N, W - 1, D).to(dt) if c["init"] else None,
              "dfinal": randn(N, W - 1, D).to(dt) if c["init"] else None}
    else:
        S, G = c["S"], c["G"]
        step = torch.exp(math.log(1e-3) + rand(D) * math.log(100.0))      # step sizes in [1e-3, 1e-1]
        s |= {"delta": (0.5 * randn(*lead, D)).to(dt), "dt_bias": torch.log(torch.expm1(step)),
              "A": -(torch.arange(1, S + 1, device=DEV) * torch.exp(0.1 * randn(D, S))),
              "B": randn(*lead, G, S).to(dt), "C": randn(*lead, G, S).to(dt), "D": 1.0 + 0.1 * randn(D),
              "z": randn(*lead, D).to(dt) if c["gate"] else None}
        if c["op"] == "scan_step":
            s |= {"state": 0.3 * randn(c["slots"], D, S),
                  "slots": torch.randperm(c["slots"], generator=g, device=DEV)[:N].to(torch.int32)}
        else:
            s["h0"] = 0.3 * randn(N, D, S) if c["init"] else None
            if c["op"] == "scan_bwd":
                s |= {"dout": randn(*lead, D).to(dt), "dht": randn(N, D, S) if c["init"] else None}
    # where each sequence starts and ends among the tokens, as the plain forms index them
    ends = torch.tensor(lens, device=DEV).cumsum(0)
    s |= {"starts": ends - torch.tensor(lens, device=DEV), "last": ends - 1}
    torch.cuda.synchronize()
    return s


# -------------------------------------------------------------- plain forms

def _sigmoid(v):
    return 1.0 / (1.0 + torch.exp(-v))


def _flat(v, *tail):
    return v.float().reshape(-1, *tail)


def _recurrence(a, b, longest):
    """h_t = a_t h_{t-1} + b_t along the first axis by doubling (a is 0 where a sequence starts); overwrites both."""
    k = 1
    while k < longest:
        b[k:] += a[k:] * b[:-k]
        a[k:] = a[k:] * a[:-k]
        k *= 2
    return b


def _scan_terms(s):
    c = s["case"]
    D, S, G = c["D"], c["S"], c["G"]
    x, raw = _flat(s["x"], D), _flat(s["delta"], D) + s["dt_bias"]
    dt = raw.clamp(min=0) + torch.log1p(torch.exp(-raw.abs()))
    Bd = _flat(s["B"], G, 1, S)
    Cd = _flat(s["C"], G, 1, S)
    decay = torch.exp(dt[:, :, None] * s["A"])
    u = ((dt * x).view(-1, G, D // G, 1) * Bd).view(-1, D, S)
    return x, raw, dt, Bd, Cd, decay, u


def _plain_scan_fwd(s):
    c = s["case"]
    D, S, G = c["D"], c["S"], c["G"]
    x, _, _, _, Cd, a, h = _scan_terms(s)
    if s["h0"] is not None:
        h[s["starts"]] += a[s["starts"]] * s["h0"]
    a[s["starts"]] = 0.0
    h = _recurrence(a, h, max(s["lens"]))
    y = (h.view(-1, G, D // G, S) * Cd).sum(-1).view(-1, D) + s["D"] * x
    if s["z"] is not None:
        z = _flat(s["z"], D)
        y = y * z * _sigmoid(z)
    return [y.view(s["x"].shape).to(s["x"].dtype), h[s["last"]]]


def _plain_scan_step(s):
    c = s["case"]
    D, S, G = c["D"], c["S"], c["G"]
    x, _, _, _, Cd, a, u = _scan_terms(s)
    at = s["slots"].long()
    h = a * s["state"][at] + u
    s["state"][at] = h
    y = (h.view(-1, G, D // G, S) * Cd).sum(-1).view(-1, D) + s["D"] * x
    if s["z"] is not None:
        z = _flat(s["z"], D)
        y = y * z * _sigmoid(z)
    return [y.view(s["x"].shape).to(s["x"].dtype), s["state"]]


def _plain_scan_bwd(s):
    c = s["case"]
    D, S, G = c["D"], c["S"], c["G"]
    starts, last, longest, dtype = s["starts"], s["last"], max(s["lens"]), s["x"].dtype
    x, raw, dt, Bd, Cd, decay, h = _scan_terms(s)
    a = decay.clone()
    if s["h0"] is not None:
        h[starts] += a[starts] * s["h0"]
    a[starts] = 0.0
    h = _recurrence(a, h, longest)
    dy = _flat(s["dout"], D)
    out = {}
    if s["z"] is not None:
        z = _flat(s["z"], D)
        sg = _sigmoid(z)
        y = (h.view(-1, G, D // G, S) * Cd).sum(-1).view(-1, D) + s["D"] * x
        out["dz"] = (dy * y * sg * (1 + z * (1 - sg))).view(s["x"].shape).to(dtype)
        dy = dy * z * sg
    # the adjoint of h: the same recurrence backwards in time, with the next token's decay
    adj = (dy.view(-1, G, D // G, 1) * Cd).view(-1, D, S)
    if s["dht"] is not None:
        adj[last] += s["dht"]
    a = torch.zeros_like(decay)
    a[:-1] = decay[1:]
    a[last] = 0.0
    adj = _recurrence(a.flip(0), adj.flip(0), longest).flip(0)
    del a
    out["dC"] = (h.view(-1, G, D // G, S) * dy.view(-1, G, D // G, 1)).sum(2)
    out["dB"] = (adj.view(-1, G, D // G, S) * (dt * x).view(-1, G, D // G, 1)).sum(2)
    gB = (adj.view(-1, G, D // G, S) * Bd).sum(-1).view(-1, D)
    # decay times the state before the token
    h[1:] = h[:-1].clone()
    h[starts] = s["h0"] if s["h0"] is not None else 0.0
    if s["h0"] is not None:
        out["dh0"] = decay[starts] * adj[starts]
    w = adj * decay * h
    out["dA"] = (w * dt[:, :, None]).sum(0)
    ddt = ((w * s["A"]).sum(-1) + gB * x) * _sigmoid(raw)
    out["dx"] = (gB * dt + s["D"] * dy).view(s["x"].shape).to(dtype)
    out["ddelta"] = ddt.view(s["x"].shape).to(dtype)
    out["dD"] = (dy * x).sum(0)
    out["ddt_bias"] = ddt.sum(0)
    out["dB"] = out["dB"].view(s["B"].shape).to(dtype)
    out["dC"] = out["dC"].view(s["C"].shape).to(dtype)
    return out


def _plain_conv_bwd(s):
    c = s["case"]
    D, W = c["D"], c["W"]
    x, dy = _flat(s["x"], D), _flat(s["dout"], D)
    n_tok, N, dtype = x.shape[0], len(s["lens"]), s["x"].dtype
    lens = torch.tensor(s["lens"], device=DEV)
    seq = torch.repeat_interleave(torch.arange(N, device=DEV), lens)
    # every sequence with W - 1 rows in front of it (its earlier inputs) and W - 1 rows of zeros behind it
    pad = 2 * (W - 1)
    at = torch.arange(n_tok, device=DEV) + seq * pad + (W - 1)
    rows = (s["starts"] + torch.arange(N, device=DEV) * pad)[:, None] + torch.arange(W - 1, device=DEV)
    ext = torch.zeros(n_tok + N * pad, D, device=DEV)
    ext[at] = x
    if s["init"] is not None:
        ext[rows] = s["init"].float()
    taps = at[:, None] - (W - 1) + torch.arange(W, device=DEV)      # [tokens, W] rows of ext
    u = (ext[taps] * s["weight"].t()).sum(1) + s["bias"]
    if c["act"] == "silu":
        sg = _sigmoid(u)
        dy = dy * sg * (1 + u * (1 - sg))
    out = {"dweight": (ext[taps] * dy[:, None, :]).sum(0).t().contiguous(), "dbias": dy.sum(0)}
    ext.zero_()
    ext[at] = dy
    # the row that holds input j was read by the outputs of rows j .. j + W - 1, through weights W - 1 .. 0
    reads = torch.arange(W - 1, -1, -1, device=DEV)
    dx = (ext[at[:, None] + reads] * s["weight"].t()).sum(1)
    d0 = (ext[rows[:, :, None] + reads] * s["weight"].t()).sum(2)
    if s["dfinal"] is not None:
        # row L + j of a sequence's inputs (counted with the earlier ones) is row j of its final state
        both = torch.zeros_like(ext)
        both[at], both[rows] = dx, d0
        both[rows + lens[:, None]] += s["dfinal"].float()
        dx, d0 = both[at], both[rows]
    out["dx"] = dx.view(s["x"].shape).to(dtype)
    if s["init"] is not None:
        out["dinitial_state"] = d0.to(dtype)
    return out


def _plain_q4_matvec(s):
    c = s["case"]
    q = s["qweight"].to(torch.int32)
    q = torch.stack((q & 15, q >> 4), -1).view(c["N"], -1, c["group"])
    zero = 8 if s["zeros"] is None else s["zeros"].to(torch.int32)[:, :, None]
    w = ((q - zero).float() * s["scales"].float()[:, :, None]).view(c["N"], c["K"])
    return (s["x"].float() @ w.t() + s["bias"]).to(s["x"].dtype)


def run(state):
    s, op = state, state["case"]["op"]
    if not own:
        return {"scan_fwd": _plain_scan_fwd, "scan_bwd": _plain_scan_bwd, "scan_step": _plain_scan_step,
                "conv_bwd": _plain_conv_bwd, "q4_matvec": _plain_q4_matvec}[op](s)
    from gated_deltanet_chunked_gdn_gb300 import binding as gdn
    if op == "q4_matvec":
        return gdn.gdn_q4_matvec(s["x"], s["qweight"], s["scales"], zeros=s["zeros"], bias=s["bias"])
    if op == "conv_bwd":
        g = gdn.gdn_causal_conv1d_bwd(s["x"], s["weight"], s["dout"], bias=s["bias"], activation=s["case"]["act"],
                                      initial_state=s["init"], dfinal_state=s["dfinal"], cu_seqlens=s["cu"])
        return {k: v for k, v in g.items() if v is not None and k != "workspace"}
    if op == "scan_step":
        y = gdn.gdn_selective_scan_step(s["x"], s["delta"], s["A"], s["B"], s["C"], s["state"], D=s["D"], z=s["z"],
                                        dt_bias=s["dt_bias"], state_indices=s["slots"])
        return [y, s["state"]]
    if op == "scan_fwd":
        y, ht = gdn.gdn_selective_scan_fwd(s["x"], s["delta"], s["A"], s["B"], s["C"], D=s["D"], z=s["z"],
                                           dt_bias=s["dt_bias"], h0=s["h0"], cu_seqlens=s["cu"])
        return [y, ht]
    g = gdn.gdn_selective_scan_bwd(s["x"], s["delta"], s["A"], s["B"], s["C"], s["dout"], D=s["D"], z=s["z"],
                                   dt_bias=s["dt_bias"], h0=s["h0"], dht=s["dht"], cu_seqlens=s["cu"])
    return {k: v for k, v in g.items() if v is not None and k != "workspace"}


# ---------------------------------------------------- the definitions, 64 bits

def _exact_q4(s):
    c = s["case"]
    y = torch.empty(c["M"], c["N"], dtype=torch.float64, device=DEV)
    x = s["x"].double().view(c["M"], -1, c["group"])
    for n in range(0, c["N"], 2048):
        b = s["qweight"][n:n + 2048]
        low, high = (b % 16).double(), (b // 16).double()
        w = torch.empty(b.shape[0], c["K"], dtype=torch.float64, device=DEV)
        w[:, 0::2], w[:, 1::2] = low, high
        w = w.view(b.shape[0], -1, c["group"])
        w = w - (8.0 if s["zeros"] is None else s["zeros"][n:n + 2048].double()[:, :, None])
        per = torch.einsum("mgk,ngk->mng", x, w)
        y[:, n:n + 2048] = (per * s["scales"][n:n + 2048].double()).sum(-1) + s["bias"][n:n + 2048].double()
    return y


def _exact_conv_bwd(s):
    c = s["case"]
    D, W, N = c["D"], c["W"], len(s["lens"])
    x, dy, w = s["x"].reshape(-1, D), s["dout"].reshape(-1, D), s["weight"].double()
    dx = torch.empty(x.shape, dtype=torch.float64, device=DEV)
    dw, db = torch.zeros(D, W, dtype=torch.float64, device=DEV), torch.zeros(D, dtype=torch.float64, device=DEV)
    d0 = torch.empty(N, W - 1, D, dtype=torch.float64, device=DEV) if s["init"] is not None else None
    p = 0
    for n, L in enumerate(s["lens"]):
        head = s["init"][n].double() if s["init"] is not None else x.new_zeros(W - 1, D, dtype=torch.float64)
        e = torch.cat([head, x[p:p + L].double()])
        u = s["bias"].double() + sum(w[:, i] * e[i:i + L] for i in range(W))
        g = dy[p:p + L].double()
        if c["act"] == "silu":
            sg = torch.sigmoid(u)
            g = g * (sg + u * sg * (1 - sg))
        de = torch.zeros_like(e)
        if s["dfinal"] is not None:
            de[L:] += s["dfinal"][n].double()
        for i in range(W):
            de[i:i + L] += w[:, i] * g
            dw[:, i] += (e[i:i + L] * g).sum(0)
        db += g.sum(0)
        dx[p:p + L] = de[W - 1:]
        if d0 is not None:
            d0[n] = de[:W - 1]
        p += L
    out = {"dx": dx.view(s["x"].shape), "dweight": dw, "dbias": db}
    if d0 is not None:
        out["dinitial_state"] = d0
    return out


def _exact_scan(s, backward):
    """Token after token, all sequences that are that long at once."""
    c = s["case"]
    D, S, G, N = c["D"], c["S"], c["G"], len(s["lens"])
    of = torch.arange(D, device=DEV) // (D // G)
    f64 = dict(dtype=torch.float64, device=DEV)
    order = sorted(range(N), key=lambda n: -s["lens"][n])                 # longest first
    idx = torch.tensor(order, device=DEV)
    starts = [sum(s["lens"][:n]) for n in order]
    starts = torch.tensor(starts, device=DEV)
    lens = [s["lens"][n] for n in order]
    A, Dp, bias = s["A"].double(), s["D"].double(), s["dt_bias"].double()
    tok = {k: s[k].reshape(-1, *s[k].shape[2:]) for k in ("x", "delta", "B", "C", "z", "dout")
           if s.get(k) is not None}

    def at(t, m):
        r = starts[:m] + t
        g = {k: v[r].double() for k, v in tok.items()}
        g["raw"] = g["delta"] + bias
        g["dt"] = torch.nn.functional.softplus(g["raw"], threshold=40.0)
        g["a"] = torch.exp(g["dt"][:, :, None] * A)
        g["Bd"], g["Cd"] = g["B"][:, of], g["C"][:, of]
        return r, g

    if "slots" in s:
        h = s["state"][s["slots"].long()][idx].double()
    else:
        h = s["h0"][idx].double() if s["h0"] is not None else torch.zeros(N, D, S, **f64)
    n_tok = tok["x"].shape[0]
    y = torch.empty(n_tok, D, **f64)
    before = torch.empty(n_tok, D, S, **f64) if backward else None
    for t in range(max(lens)):
        m = sum(1 for v in lens if v > t)
        r, g = at(t, m)
        if backward:
            before[r] = h[:m]
        h[:m] = g["a"] * h[:m] + (g["dt"] * g["x"])[:, :, None] * g["Bd"]
        y[r] = (h[:m] * g["Cd"]).sum(-1) + Dp * g["x"]
    if not backward:
        if "z" in tok:
            z = tok["z"].double()
            y = y * z * torch.sigmoid(z)
        back = torch.empty_like(h)
        back[idx] = h
        if "slots" in s:
            pool = s["state"].double()
            pool[s["slots"].long()] = back
            back = pool
        return [y.view(s["x"].shape), back]
    out = {k: torch.empty(n_tok, D, **f64) for k in ("dx", "ddelta")}
    out |= {k: torch.empty(n_tok, G, S, **f64) for k in ("dB", "dC")}
    out |= {"dA": torch.zeros(D, S, **f64), "dD": torch.zeros(D, **f64), "ddt_bias": torch.zeros(D, **f64)}
    if "z" in tok:
        out["dz"] = torch.empty(n_tok, D, **f64)
    adj = s["dht"][idx].double() if s["dht"] is not None else torch.zeros(N, D, S, **f64)
    for t in reversed(range(max(lens))):
        m = sum(1 for v in lens if v > t)
        r, g = at(t, m)
        dy = g["dout"]
        if "z" in tok:
            sg = torch.sigmoid(g["z"])
            out["dz"][r] = dy * y[r] * (sg + g["z"] * sg * (1 - sg))
            dy = dy * g["z"] * sg
        hb = before[r]
        hn = g["a"] * hb + (g["dt"] * g["x"])[:, :, None] * g["Bd"]
        adj[:m] += dy[:, :, None] * g["Cd"]
        out["dC"][r] = (hn * dy[:, :, None]).view(m, G, D // G, S).sum(2)
        out["dB"][r] = (adj[:m] * (g["dt"] * g["x"])[:, :, None]).view(m, G, D // G, S).sum(2)
        gB = (adj[:m] * g["Bd"]).sum(-1)
        w = adj[:m] * g["a"] * hb
        ddt = ((w * A).sum(-1) + gB * g["x"]) * torch.sigmoid(g["raw"])
        out["dx"][r] = gB * g["dt"] + Dp * dy
        out["ddelta"][r] = ddt
        out["dA"] += (w * g["dt"][:, :, None]).sum(0)
        out["dD"] += (dy * g["x"]).sum(0)
        out["ddt_bias"] += ddt.sum(0)
        adj[:m] = g["a"] * adj[:m]
    if s["h0"] is not None:
        out["dh0"] = torch.empty_like(adj)
        out["dh0"][idx] = adj
    for k in ("dx", "ddelta", "dz"):
        if k in out:
            out[k] = out[k].view(s["x"].shape)
    for k in ("dB", "dC"):
        out[k] = out[k].view(s["B"].shape)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "q4_matvec":
        return _exact_q4(s)
    if case["op"] == "conv_bwd":
        return _exact_conv_bwd(s)
    return _exact_scan(s, case["op"] == "scan_bwd")


# --------------------------------------------------------------------- work

def work(case):
    c = case
    e = 2 if c["dtype"] == "bf16" else 4
    if c["op"] == "q4_matvec":
        M, N, K, gr = c["M"], c["N"], c["K"], c["group"]
        groups = N * (K // gr)
        return {"bytes": N * K // 2 + groups * ((2 if c["scales"] == "bf16" else 4) + int(c["zeros"])) + M * (N + K) * e
                + 4 * N, "flops": 2 * M * N * K}
    N = c["N"] if c["op"] == "scan_step" else len(_lengths(c))
    tokens = N if c["op"] == "scan_step" else sum(_lengths(c))
    D = c["D"]
    if c["op"] == "conv_bwd":
        W = c["W"]
        return {"bytes": 3 * tokens * D * e + (3 * N * (W - 1) * D * e if c["init"] else 0) + 8 * D * (W + 1),
                "flops": tokens * D * (6 * W + 8)}
    S, G = c["S"], c["G"]
    gate = int(c["gate"])
    params = 4 * D * (S + 2)
    if c["op"] == "scan_step":
        return {"bytes": tokens * e * (D * (3 + gate) + 2 * G * S) + 8 * N * D * S + params, "flops": 7 * tokens * D * S}
    states = 4 * N * D * S
    if c["op"] == "scan_fwd":
        return {"bytes": tokens * e * (D * (3 + gate) + 2 * G * S) + states * (1 + int(c["init"])) + params,
                "flops": 7 * tokens * D * S}
    return {"bytes": tokens * e * (D * (5 + 2 * gate) + 4 * G * S) + 3 * states * int(c["init"]) + 2 * params,
            "flops": 22 * tokens * D * S}
