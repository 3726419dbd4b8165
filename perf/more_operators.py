"""Cases of linear attention with a decay for each head and of the norms around a block, as a user's program calls them.

Five operators, named by a case's "op":

  attn_fwd       decayed linear attention over prompts or training sequences: outputs and final states
  attn_bwd       its gradients with respect to every input and the initial states
  attn_step      one token of every sequence on a pool of states (decode)
  gated_norm     the norm of a mixer's output, head by head, times its gate: silu(z) * rms(x) * weight
  residual_norm  between two blocks: the norm after the one, its gate, the scaled residual sum, the norm before the next

The norms run forward ("fwd") or forward and backward ("train").  `own` chooses between the plain form (elementary
torch operations in 32 bits, decays in 64) and the framework's entry points; `exact` evaluates the definitions in 64
bits: the recurrence token by token, its gradients by the sums over all pairs of tokens.
"""
import math
import random

import torch

own = False

DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6
CHUNK = 64      # tokens a block of the plain form


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one long prompt, two value heads to a query head
        {"name": "attn_fwd one prompt", "op": "attn_fwd", "B": 1, "T": 8192, "Hqk": 16, "Hv": 32, "K": 128, "V": 128,
         "dtype": "bf16", "decay": "token", "init": False},
        # the forward half of a training step on long sequences
        {"name": "attn_fwd training batch", "op": "attn_fwd", "B": 4, "T": 8192, "Hqk": 32, "Hv": 32, "K": 128,
         "V": 128, "dtype": "bf16", "decay": "token", "init": False},
        # packed prompts of very different lengths that continue earlier states, fixed decays, in fp32
        {"name": "attn_fwd packed", "op": "attn_fwd", "packed": 37, "longest": 1500, "Hqk": 4, "Hv": 12, "K": 64,
         "V": 128, "dtype": "f32", "decay": "head", "init": True},
        # the backward half of a training step
        {"name": "attn_bwd training batch", "op": "attn_bwd", "B": 4, "T": 4096, "Hqk": 32, "Hv": 32, "K": 128,
         "V": 128, "dtype": "bf16", "decay": "token", "init": False},
        # packed training sequences, one key head for all value heads, gradients down to the initial states
        {"name": "attn_bwd packed, odd", "op": "attn_bwd", "packed": 13, "longest": 1500, "Hqk": 1, "Hv": 6, "K": 128,
         "V": 64, "dtype": "f32", "decay": "token", "init": True},
        # decode, a single request: latency
        {"name": "attn_step 1 request", "op": "attn_step", "N": 1, "slots": 8, "Hqk": 16, "Hv": 32, "K": 128,
         "V": 128, "dtype": "bf16", "decay": "token"},
        # decode, a full batch on a larger pool
        {"name": "attn_step 512 requests", "op": "attn_step", "N": 512, "slots": 640, "Hqk": 32, "Hv": 32, "K": 128,
         "V": 128, "dtype": "bf16", "decay": "token"},
        # a decode step of a few requests: latency
        {"name": "gated_norm 5 rows", "op": "gated_norm", "rows": 5, "H": 32, "V": 128, "dtype": "bf16", "dir": "fwd"},
        # training
        {"name": "gated_norm training batch", "op": "gated_norm", "rows": 16384, "H": 32, "V": 128, "dtype": "bf16",
         "dir": "train"},
        # a decode step of one request, residuals in fp32
        {"name": "residual_norm 1 row", "op": "residual_norm", "rows": 1, "D": 4096, "dtype": "bf16",
         "residual": "f32", "post": True, "gate": "channel", "weight": True, "dir": "fwd"},
        # a long prompt
        {"name": "residual_norm prompt", "op": "residual_norm", "rows": 8192, "D": 4096, "dtype": "bf16",
         "residual": "bf16", "post": True, "gate": "channel", "weight": True, "dir": "fwd"},
        # training, odd sizes, a gate of its own for each token
        {"name": "residual_norm training, odd", "op": "residual_norm", "rows": 4099, "D": 2500, "dtype": "f32",
         "residual": "f32", "post": True, "gate": "token", "weight": True, "dir": "train"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attn_fwd", "attn_fwd", "attn_bwd", "attn_bwd", "attn_step", "gated_norm", "residual_norm"])
    c = {"op": op, "dtype": rng.choice(["bf16", "bf16", "f32"])}
    if op == "gated_norm":
        H, V = _log(rng, 1, 64), _log(rng, 16, 512)
        most = (1 << 26) // (H * V)
        return {**c, "rows": _log(rng, 1, most), "H": H, "V": V, "dir": rng.choice(["fwd", "train"])}
    if op == "residual_norm":
        D = _log(rng, 64, 16384)
        return {**c, "rows": _log(rng, 1, (1 << 25) // D), "D": D,
                "residual": "f32" if c["dtype"] == "f32" else rng.choice(["bf16", "f32"]),
                "post": rng.random() < 0.7, "gate": rng.choice(["none", "channel", "token"]),
                "weight": rng.random() < 0.9, "dir": rng.choice(["fwd", "train"])}
    per, Hqk = rng.choice([1, 1, 2, 4, 6]), _log(rng, 1, 32)
    Hv = min(64, Hqk * per) // Hqk * Hqk
    c |= {"Hqk": Hqk, "Hv": Hv, "K": rng.choice([64, 128, 128, 256]), "V": rng.choice([64, 128, 128, 256]),
          "decay": rng.choice(["token", "token", "head"])}
    if op == "attn_step":
        n = _log(rng, 1, max(1, min(512, (1 << 28) // (Hv * c["K"] * c["V"]))))
        return {**c, "N": n, "slots": n + rng.randrange(0, 100)}
    c["init"] = rng.random() < 0.5
    # tokens by what the largest listed case of the kind computes
    most = (1 << (34 if op == "attn_fwd" else 33)) // (Hv * c["K"] * c["V"])
    if c["dtype"] == "f32":
        most //= 4
    tokens = _log(rng, 16, max(32, min(32768, most)))
    if rng.random() < 0.5:
        n = rng.randrange(2, 65)
        return {**c, "packed": n, "longest": max(2, 4 * tokens // n)}
    B = _log(rng, 1, min(8, tokens))
    return {**c, "B": B, "T": max(1, tokens // B)}


def _lengths(c):
    """Token counts of the case's sequences: all alike, or log-uniform in [1, longest] for packed ones."""
    if "B" in c:
        return [c["T"]] * c["B"]
    r = random.Random("%s %s" % (c["packed"], c["longest"]))
    return [_log(r, 1, c["longest"]) for _ in range(c["packed"])]


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    c = case
    gen = torch.Generator(device=DEV).manual_seed(int(seed))
    dt = DT[c["dtype"]]

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device=DEV)

    def rand(*shape):
        return torch.rand(*shape, generator=gen, device=DEV)

    if c["op"] == "gated_norm":
        shape = (c["rows"], c["H"], c["V"])
        s = {"case": c, "x": (2.0 * randn(*shape)).to(dt), "z": randn(*shape).to(dt),
             "weight": 1.0 + 0.1 * randn(c["V"]), "dy": randn(*shape).to(dt)}
        torch.cuda.synchronize()
        return s
    if c["op"] == "residual_norm":
        shape, rdt = (c["rows"], c["D"]), DT[c["residual"]]
        s = {"case": c, "y": randn(*shape).to(dt), "residual": (3.0 * randn(*shape)).to(rdt),
             "post_weight": 1.0 + 0.1 * randn(c["D"]) if c["post"] else None,
             "gate": {"none": None, "channel": 0.5 + 0.1 * randn(c["D"]), "token": rand(*shape).to(dt)}[c["gate"]],
             "weight": 1.0 + 0.1 * randn(c["D"]) if c["weight"] else None, "scale": 0.7,
             "dh": randn(*shape).to(rdt), "dn": randn(*shape).to(dt) if c["weight"] else None}
        torch.cuda.synchronize()
        return s

    Hqk, Hv, K, V = c["Hqk"], c["Hv"], c["K"], c["V"]
    cu = None
    if c["op"] == "attn_step":
        lens, lead = [1] * c["N"], (c["N"], 1)
    else:
        lens = _lengths(c)
        if "B" in c:
            lead = (c["B"], c["T"])
        else:
            cu = torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device=DEV)
            lead = (1, sum(lens))
    N = len(lens)
    s = {"case": c, "lens": lens, "cu": cu, "scale": K ** -0.5,
         "q": randn(*lead, Hqk, K).to(dt), "k": (randn(*lead, Hqk, K) * K ** -0.5).to(dt),
         "v": randn(*lead, Hv, V).to(dt)}
    if c["decay"] == "head":       # slopes of a fixed geometric series
        s["g"] = -torch.exp2(-8.0 * torch.arange(1, Hv + 1, device=DEV) / Hv)
    else:                          # -rate * softplus(step), as a layer makes them
        step = torch.log1p(torch.exp(randn(*lead, Hv) - 2.0))
        s["g"] = -(torch.exp(rand(Hv) * math.log(16.0)) * step)
    if c["op"] == "attn_step":
        s |= {"state": 0.3 * randn(c["slots"], Hv, K, V),
              "slots": torch.randperm(c["slots"], generator=gen, device=DEV)[:N].to(torch.int32)}
    else:
        s["h0"] = 0.3 * randn(N, Hv, K, V) if c["init"] else None
        if c["op"] == "attn_bwd":
            s |= {"do": randn(*lead, Hv, V).to(dt), "dht": 0.3 * randn(N, Hv, K, V) if c["init"] else None}
        s |= _blocks(lens)
    torch.cuda.synchronize()
    return s


def _blocks(lens):
    """Tables of the plain form: its blocks of CHUNK tokens, each within one sequence."""
    at, first, last, base = [], [], [], 0
    for n in lens:
        first.append(len(at))
        for p in range(0, n, CHUNK):
            at.append([base + p + i if p + i < n else -1 for i in range(CHUNK)])
        last.append(len(at) - 1)
        base += n
    at = torch.tensor(at, device=DEV)
    where = torch.empty(base, dtype=torch.long, device=DEV)      # a token's place among the blocks' rows
    flat = at.reshape(-1)
    where[flat[flat >= 0]] = torch.nonzero(flat >= 0)[:, 0]
    return {"at": at.clamp(min=0), "live": at >= 0, "first": torch.tensor(first, device=DEV),
            "last": torch.tensor(last, device=DEV), "where": where, "most": max(-(-n // CHUNK) for n in lens)}


# -------------------------------------------------------------- plain forms

def _sigmoid(v):
    return 1.0 / (1.0 + torch.exp(-v))


def _to_blocks(s, t, heads):
    """[B, T, H, D] as fp32 [blocks, heads, CHUNK, D], zeros past a sequence's end."""
    t = t.reshape(-1, *t.shape[2:])[s["at"]].float() * s["live"][:, :, None, None]
    return t.transpose(1, 2).repeat_interleave(heads // t.shape[2], dim=1)


def _from_blocks(s, t, like, heads):
    """Back to [B, T, heads, D] in the type of `like`, heads that share one summed."""
    t = t.reshape(t.shape[0], heads, -1, *t.shape[2:]).sum(2)
    t = t.transpose(1, 2).reshape(-1, heads, t.shape[-1])[s["where"]]
    return t.view(*like.shape[:2], heads, -1).to(like.dtype)


def _decays(s):
    """Sums of the log decays within the blocks (64 bits) [blocks, heads, CHUNK]."""
    c, g = s["case"], s["g"].double()
    if c["decay"] == "head":
        g = s["live"][:, :, None] * g
    else:
        g = g.view(-1, c["Hv"])[s["at"]] * s["live"][:, :, None]
    return g.cumsum(1).transpose(1, 2)


def _recurrence(a, b, longest):
    """b_c += a_c b_{c-1} along the blocks by doubling (a is 0 where a sequence starts); overwrites both."""
    k = 1
    while k < longest:
        b[k:] += a[k:, :, None, None] * b[:-k]
        a[k:] = a[k:] * a[:-k]
        k *= 2
    return b


def _states(s, k, v, sums):
    """States before every block and after the sequences."""
    total = sums[:, :, -1:]
    after = (k * torch.exp(total - sums).float()[..., None]).transpose(2, 3) @ v
    a = torch.exp(total[..., 0]).float()
    if s["h0"] is not None:
        after[s["first"]] += a[s["first"]][:, :, None, None] * s["h0"]
    a[s["first"]] = 0.0
    after = _recurrence(a, after, s["most"])
    before = torch.zeros_like(after)
    before[1:] = after[:-1]
    before[s["first"]] = s["h0"] if s["h0"] is not None else 0.0
    return before, after


def _within(sums):
    """exp(b_i - b_j) for j <= i, else 0."""
    i = torch.arange(CHUNK, device=DEV)
    d = sums[..., :, None] - sums[..., None, :]
    return torch.exp(torch.where(i[:, None] >= i, d, torch.full_like(d, -math.inf))).float()


def _plain_fwd(s):
    c, Hv = s["case"], s["case"]["Hv"]
    q, k, v = (_to_blocks(s, s[n], Hv) for n in ("q", "k", "v"))
    sums = _decays(s)
    before, after = _states(s, k, v, sums)
    o = ((q @ k.transpose(2, 3)) * _within(sums)) @ v + torch.exp(sums).float()[..., None] * (q @ before)
    return [_from_blocks(s, o * s["scale"], s["v"], Hv), after[s["last"]]]


def _plain_bwd(s):
    c, Hv = s["case"], s["case"]["Hv"]
    q, k, v, do = (_to_blocks(s, s[n], Hv) for n in ("q", "k", "v", "do"))
    q = q * s["scale"]
    sums = _decays(s)
    total = sums[:, :, -1:]
    before, after = _states(s, k, v, sums)
    up = torch.exp(sums).float()[..., None]                 # from a block's start to the token
    down = torch.exp(total - sums).float()[..., None]       # from the token to the block's end
    # adjoints of the states after every block, and of the initial ones
    adj = (q * up).transpose(2, 3) @ do
    a = torch.exp(total[..., 0]).float()
    end = torch.zeros_like(a)
    end[:-1] = a[:-1]
    if s["dht"] is not None:
        adj[s["last"]] += a[s["last"]][:, :, None, None] * s["dht"]
    end[s["last"]] = 0.0
    adj = _recurrence(end.flip(0), adj.flip(0), s["most"]).flip(0)     # adjoint of the state before each block
    G = torch.zeros_like(adj)
    G[:-1] = adj[1:]
    G[s["last"]] = s["dht"] if s["dht"] is not None else 0.0
    M = _within(sums)
    qk, dov = (q @ k.transpose(2, 3)) * M, do @ v.transpose(2, 3)
    both = qk * dov
    dov = dov * M
    from_state = up * (do @ before.transpose(2, 3))
    to_state = down * (v @ G.transpose(2, 3))
    dq = (dov @ k + from_state) * s["scale"]
    dk = dov.transpose(2, 3) @ q + to_state
    dv = qk.transpose(2, 3) @ do + down * (k @ G)
    db = both.double().sum(3) - both.double().sum(2) + ((q * from_state).double() - (k * to_state).double()).sum(3)
    dg = db.flip(2).cumsum(2).flip(2) + (G * after).double().sum((2, 3))[..., None]
    dg = (dg * s["live"][:, None, :]).transpose(1, 2)
    if c["decay"] == "head":
        dg = dg.sum((0, 1)).float()
    else:
        dg = dg.reshape(-1, Hv)[s["where"]].view(s["g"].shape).float()
    out = {"dq": _from_blocks(s, dq, s["q"], c["Hqk"]), "dk": _from_blocks(s, dk, s["k"], c["Hqk"]),
           "dv": _from_blocks(s, dv, s["v"], Hv), "dg": dg}
    if s["h0"] is not None:
        out["dh0"] = adj[s["first"]]
    return out


def _plain_step(s):
    c = s["case"]
    N, Hqk, Hv = c["N"], c["Hqk"], c["Hv"]
    q, k = (s[n].float().view(N, Hqk, c["K"]).repeat_interleave(Hv // Hqk, dim=1) for n in ("q", "k"))
    v = s["v"].float().view(N, Hv, c["V"])
    at = s["slots"].long()
    a = torch.exp(s["g"].view(-1, Hv))[..., None, None]
    h = a * s["state"][at] + k[..., None] * v[..., None, :]
    s["state"][at] = h
    o = s["scale"] * (q[..., None] * h).sum(2)
    return [o.view(s["v"].shape).to(s["v"].dtype), s["state"]]


def _rms(x):
    """1 / root mean square of the last dimension."""
    return torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)


def _rms_bwd(d, xhat, r):
    """Gradient of xhat = x r with respect to x."""
    return r * (d - xhat * (d * xhat).mean(-1, keepdim=True))


def _plain_gated_norm(s):
    x, z = s["x"].float(), s["z"].float()
    r, sg = _rms(x), _sigmoid(z)
    xhat, gate = x * r, z * sg
    y = (xhat * s["weight"] * gate).to(s["x"].dtype)
    if s["case"]["dir"] == "fwd":
        return {"y": y}
    dy = s["dy"].float()
    du = dy * gate
    dz = dy * xhat * s["weight"] * sg * (1 + z * (1 - sg))
    return {"y": y, "dx": _rms_bwd(du * s["weight"], xhat, r).to(y.dtype), "dz": dz.to(y.dtype),
            "dweight": (du * xhat).sum((0, 1))}


def _plain_residual_norm(s):
    c = s["case"]
    y, gate = s["y"].float(), s["gate"].float() if s["gate"] is not None else None
    u = y
    if c["post"]:
        r1 = _rms(y)
        yhat = y * r1
        u = yhat * s["post_weight"]
    h = s["residual"].float() + s["scale"] * (u * gate if gate is not None else u)
    out = {"h": h.to(s["residual"].dtype)}
    if c["weight"]:
        r2 = _rms(h)
        hhat = h * r2
        out["n"] = (hhat * s["weight"]).to(s["y"].dtype)
    if c["dir"] == "fwd":
        return out
    dh = s["dh"].float()
    if c["weight"]:
        dn = s["dn"].float()
        out["dweight"] = (dn * hhat).sum(0)
        dh = dh + _rms_bwd(dn * s["weight"], hhat, r2)
    out["dresidual"] = dh.to(s["residual"].dtype)
    du = s["scale"] * dh
    if gate is not None:
        dgate = du * u
        out["dgate"] = dgate.sum(0) if c["gate"] == "channel" else dgate.to(s["gate"].dtype)
        du = du * gate
    if c["post"]:
        out["dpost_weight"] = (du * yhat).sum(0)
        du = _rms_bwd(du * s["post_weight"], yhat, r1)
    out["dy"] = du.to(s["y"].dtype)
    return out


def run(state):
    s, c, op = state, state["case"], state["case"]["op"]
    if not own:
        return {"attn_fwd": _plain_fwd, "attn_bwd": _plain_bwd, "attn_step": _plain_step,
                "gated_norm": _plain_gated_norm, "residual_norm": _plain_residual_norm}[op](s)
    from gated_deltanet_chunked_gdn_gb300 import binding as gdn
    if op == "attn_fwd":
        o, ht = gdn.gdn_linear_attn_fwd(s["q"], s["k"], s["v"], s["g"], scale=s["scale"], h0=s["h0"],
                                        cu_seqlens=s["cu"])
        return [o, ht]
    if op == "attn_bwd":
        g = gdn.gdn_linear_attn_bwd(s["q"], s["k"], s["v"], s["g"], s["do"], scale=s["scale"], h0=s["h0"],
                                    dht=s["dht"], cu_seqlens=s["cu"])
        return {k: g[k] for k in ("dq", "dk", "dv", "dg", "dh0") if g[k] is not None}
    if op == "attn_step":
        o = gdn.gdn_linear_attn_step(s["q"], s["k"], s["v"], s["g"], s["state"], scale=s["scale"],
                                     state_indices=s["slots"])
        return [o, s["state"]]
    train = c["dir"] == "train"
    if op == "gated_norm":
        y, rstd = gdn.gdn_gated_norm_fwd(s["x"], s["z"], s["weight"], eps=EPS, save_rstd=train)
        out = {"y": y}
        if train:
            g = gdn.gdn_gated_norm_bwd(s["x"], s["z"], s["weight"], rstd, s["dy"])
            out |= {k: g[k] for k in ("dx", "dz", "dweight")}
        return out
    h, n, rstd = gdn.gdn_residual_norm_fwd(s["y"], s["residual"], post_weight=s["post_weight"], gate=s["gate"],
                                           residual_scale=s["scale"], weight=s["weight"], eps=EPS, save_rstd=train)
    out = {"h": h}
    if n is not None:
        out["n"] = n
    if train:
        g = gdn.gdn_residual_norm_bwd(s["y"], s["residual"], rstd, s["dh"], s["dn"], post_weight=s["post_weight"],
                                      gate=s["gate"], residual_scale=s["scale"], weight=s["weight"])
        out |= {k: g[k] for k in ("dweight", "dresidual", "dgate", "dpost_weight", "dy") if g[k] is not None}
    return out


# ---------------------------------------------------- the definitions, 64 bits

def _each_sequence(s):
    p = 0
    for n, L in enumerate(s["lens"]):
        yield n, p, L
        p += L


def _log_decays(s):
    c = s["case"]
    g = s["g"].double()
    return g.expand(sum(s["lens"]), c["Hv"]) if c["decay"] == "head" else g.reshape(-1, c["Hv"])


def _exact_fwd(s):
    """Token after token, all sequences that are that long at once."""
    c = s["case"]
    Hv, K, V, N = c["Hv"], c["K"], c["V"], len(s["lens"])
    of = torch.arange(Hv, device=DEV) // (Hv // c["Hqk"])
    order = sorted(range(N), key=lambda n: -s["lens"][n])
    starts = torch.tensor([sum(s["lens"][:n]) for n in order], device=DEV)
    lens = [s["lens"][n] for n in order]
    idx = torch.tensor(order, device=DEV)
    q, k, v = (s[n].reshape(-1, *s[n].shape[2:]) for n in ("q", "k", "v"))
    a = torch.exp(_log_decays(s))
    if c["op"] == "attn_step":
        h = s["state"][s["slots"].long()].double()
    else:
        h = s["h0"][idx].double() if s["h0"] is not None else torch.zeros(N, Hv, K, V, dtype=torch.float64, device=DEV)
    o = torch.empty(v.shape, dtype=torch.float64, device=DEV)
    for t in range(max(lens)):
        m = sum(1 for L in lens if L > t)
        r = starts[:m] + t
        h[:m].mul_(a[r][:, :, None, None])
        h[:m].addcmul_(k[r].double()[:, of, :, None], v[r].double()[:, :, None, :])
        o[r] = s["scale"] * torch.matmul(q[r].double()[:, of, None, :], h[:m])[:, :, 0]
    o = o.view(s["v"].shape)
    if c["op"] == "attn_step":
        pool = s["state"].double()
        pool[s["slots"].long()] = h
        return [o, pool]
    ht = torch.empty_like(h)
    ht[idx] = h
    return [o, ht]


def _exact_bwd(s):
    """Sums over all pairs of tokens of a sequence, one head after the other."""
    c = s["case"]
    Hqk, Hv, K, V = c["Hqk"], c["Hv"], c["K"], c["V"]
    if Hv * sum(L * L for L in s["lens"]) > 3e9 or Hv * len(s["lens"]) > 1500:
        return None
    q, k, v, do = (s[n].reshape(-1, *s[n].shape[2:]) for n in ("q", "k", "v", "do"))
    g = _log_decays(s)
    f64 = dict(dtype=torch.float64, device=DEV)
    out = {"dq": torch.zeros(q.shape, **f64), "dk": torch.zeros(k.shape, **f64), "dv": torch.zeros(v.shape, **f64),
           "dg": torch.zeros(g.shape, **f64)}
    if s["h0"] is not None:
        out["dh0"] = torch.zeros(s["h0"].shape, **f64)
    for n, p, L in _each_sequence(s):
        at = slice(p, p + L)
        for h in range(Hv):
            hq = h // (Hv // Hqk)
            Q, Kt, X, D = s["scale"] * q[at, hq].double(), k[at, hq].double(), v[at, h].double(), do[at, h].double()
            b = g[at, h].cumsum(0)
            M = torch.exp((b[:, None] - b[None, :]).tril_()).tril_()
            A, W = (Q @ Kt.t()).mul_(M), (D @ X.t()).mul_(M)
            out["dq"][at, hq] += s["scale"] * (W @ Kt)
            out["dk"][at, hq] += W.t() @ Q
            out["dv"][at, h] = A.t() @ D
            # pairs counted once with their decays: M is in A and in W
            w = torch.where(M > 0, A * W / torch.where(M > 0, M, torch.ones_like(M)), torch.zeros_like(M))
            db = w.sum(1) - w.sum(0)
            if s["h0"] is not None:
                h0, dht = s["h0"][n, h].double(), s["dht"][n, h].double()
                e, d = torch.exp(b)[:, None], torch.exp(b[-1] - b)[:, None]
                fq, fk = e * (D @ h0.t()), d * (X @ dht.t())
                out["dq"][at, hq] += s["scale"] * fq
                out["dk"][at, hq] += fk
                out["dv"][at, h] += d * (Kt @ dht)
                out["dh0"][n, h] = (e * Q).t() @ D + torch.exp(b[-1]) * dht
                ht = torch.exp(b[-1]) * h0 + (d * Kt).t() @ X
                db += (Q * fq).sum(1) - (Kt * fk).sum(1)
                db[-1] += (dht * ht).sum()
            out["dg"][at, h] = db.flip(0).cumsum(0).flip(0)
    for name in ("q", "k", "v"):
        out["d" + name] = out["d" + name].view(s[name].shape)
    out["dg"] = out["dg"].sum(0) if c["decay"] == "head" else out["dg"].view(s["g"].shape)
    return out


def _exact_norms(s):
    """The forward forms in 64 bits, and their gradients by reverse mode."""
    c = s["case"]
    train = c["dir"] == "train"
    names = ("x", "z", "weight") if c["op"] == "gated_norm" else ("y", "residual", "post_weight", "gate", "weight")
    t = {n: s[n].double().requires_grad_(train) for n in names if s[n] is not None}

    def norm(v):
        return v / torch.sqrt(v.pow(2).mean(-1, keepdim=True) + EPS)

    if c["op"] == "gated_norm":
        out = {"y": norm(t["x"]) * t["weight"] * torch.nn.functional.silu(t["z"])}
        up = {"y": s["dy"]}
    else:
        u = norm(t["y"]) * t["post_weight"] if c["post"] else t["y"]
        out = {"h": t["residual"] + s["scale"] * t["gate"] * u if "gate" in t else t["residual"] + s["scale"] * u}
        up = {"h": s["dh"]}
        if c["weight"]:
            out["n"] = norm(out["h"]) * t["weight"]
            up["n"] = s["dn"]
    if train:
        grads = torch.autograd.grad([out[n] for n in up], list(t.values()), [up[n].double() for n in up])
        out |= {"d" + n: g for n, g in zip(t, grads)}
    return {n: v.detach() for n, v in out.items()}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("gated_norm", "residual_norm"):
        return _exact_norms(s)
    return _exact_bwd(s) if case["op"] == "attn_bwd" else _exact_fwd(s)


# --------------------------------------------------------------------- work

def work(case):
    c = case
    e = 2 if c["dtype"] == "bf16" else 4
    train = c.get("dir") == "train"
    if c["op"] == "gated_norm":
        n = c["rows"] * c["H"] * c["V"]
        return {"bytes": n * e * (6 if train else 3) + 4 * c["V"] * (2 if train else 1), "flops": n * (26 if train else 10)}
    if c["op"] == "residual_norm":
        n, r = c["rows"] * c["D"], 4 if c["residual"] == "f32" else 2
        token, w = c["gate"] == "token", int(c["weight"])
        vec = 4 * c["D"] * (int(c["post"]) + w + int(c["gate"] == "channel"))
        fwd = n * (e * (1 + w + int(token)) + 2 * r) + vec
        # the gradients' half reads what comes from above besides, and writes a gradient for every input
        bwd = n * (e * (w + 1 + int(token)) + 2 * r) + vec
        return {"bytes": fwd + (bwd if train else 0), "flops": n * (30 if train else 10)}
    Hqk, Hv, K, V = c["Hqk"], c["Hv"], c["K"], c["V"]
    N = c["N"] if c["op"] == "attn_step" else len(_lengths(c))
    tokens = N if c["op"] == "attn_step" else sum(_lengths(c))
    state = 4 * N * Hv * K * V
    g = 4 * Hv * (tokens if c["decay"] == "token" else 1)
    rows = tokens * e * 2 * (Hqk * K + Hv * V)
    if c["op"] == "attn_step":
        return {"bytes": rows + g + 2 * state, "flops": 5 * tokens * Hv * K * V}
    if c["op"] == "attn_fwd":
        return {"bytes": rows + g + state * (1 + int(c["init"])), "flops": 4 * tokens * Hv * K * V}
    return {"bytes": 2 * rows - tokens * e * Hv * V + 2 * g + 3 * state * int(c["init"]),
            "flops": 10 * tokens * Hv * K * V}
