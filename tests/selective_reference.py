"""The selective state space layer's operators from their definitions, token by
token in 64 bits (torch, CPU).  Used by the tests only; gradients by autograd."""
import torch


def lengths(B, T, lens):
    return [T] * B if lens is None else list(lens)


def scan(x, delta, A, B, C, D=None, z=None, dt_bias=None, softplus=True, h0=None, lens=None):
    """(y, ht) of the scan; x [B, T, D], B and C [B, T, G, S]; lens: packed sequences."""
    d64 = lambda t: None if t is None else t.double()
    x, delta, A, B, C, D, z, dt_bias, h0 = map(d64, (x, delta, A, B, C, D, z, dt_bias, h0))
    nb, T, d = x.shape
    G, S = B.shape[2:]
    tok = lambda t, *tail: t.reshape(-1, *tail)
    x_, de, B_, C_ = tok(x, d), tok(delta, d), tok(B, G, S), tok(C, G, S)
    dt = de + dt_bias if dt_bias is not None else de
    if softplus:
        dt = torch.nn.functional.softplus(dt, threshold=50.0)
    Bd, Cd = B_.repeat_interleave(d // G, 1), C_.repeat_interleave(d // G, 1)      # [tokens, D, S]
    ys, hts, p = [], [], 0
    for n, L in enumerate(lengths(nb, T, lens)):
        h = h0[n] if h0 is not None else torch.zeros(d, S, dtype=torch.float64)
        for t in range(p, p + L):
            h = torch.exp(dt[t][:, None] * A) * h + (dt[t] * x_[t])[:, None] * Bd[t]
            y = (h * Cd[t]).sum(-1)
            ys.append(y + D * x_[t] if D is not None else y)
        hts.append(h)
        p += L
    y = torch.stack(ys).reshape(x.shape) if ys else torch.zeros(x.shape, dtype=torch.float64)
    if z is not None:
        y = y * z * torch.sigmoid(z)
    return y, torch.stack(hts)


def scan_grads(inputs, dout, dht=None, **kw):
    """Gradients of <dout, y> + <dht, ht> with respect to every tensor of ``inputs`` (a dict of scan's arguments)."""
    leaves = {k: v.double().requires_grad_() for k, v in inputs.items() if v is not None}
    y, ht = scan(**leaves, **kw)
    total = (y * dout.double()).sum()
    if dht is not None:
        total = total + (ht * dht.double()).sum()
    got = torch.autograd.grad(total, list(leaves.values()), allow_unused=True)
    return {k: torch.zeros_like(v) if g is None else g for (k, v), g in zip(leaves.items(), got)}


def conv(x, weight, bias=None, activation="silu", initial_state=None, lens=None):
    """(y, final state) of the causal depthwise convolution."""
    d64 = lambda t: None if t is None else t.double()
    x, weight, bias, initial_state = map(d64, (x, weight, bias, initial_state))
    nb, T, d = x.shape
    W = weight.shape[1]
    x_, ys, finals, p = x.reshape(-1, d), [], [], 0
    for n, L in enumerate(lengths(nb, T, lens)):
        head = initial_state[n] if initial_state is not None else torch.zeros(W - 1, d, dtype=torch.float64)
        ext = torch.cat([head, x_[p:p + L]])
        u = sum(weight[:, w] * ext[w:w + L] for w in range(W))
        ys.append(u + bias if bias is not None else u)
        finals.append(ext[L:L + W - 1])
        p += L
    u = torch.cat(ys).reshape(x.shape)
    return (u * torch.sigmoid(u) if activation == "silu" else u), torch.stack(finals)


def q4_weights(qweight, scales, zeros=None):
    """[N, K] weights that 4-bit codes stand for."""
    n, half = qweight.shape
    q = torch.stack((qweight & 15, qweight >> 4), -1).reshape(n, scales.shape[1], -1).double()
    zero = zeros.double()[:, :, None] if zeros is not None else 8.0
    return ((q - zero) * scales.double()[:, :, None]).reshape(n, 2 * half)


def make_scan(B, T, D, S, G, dtype, gate=True, bias=True, skip=True, init=False, lens=None, seed=0):
    """Inputs with step sizes in [1e-3, 1e-1] and decay rates -1 .. -S, as such layers start from."""
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g)
    if lens is not None:
        B, T = 1, sum(lens)
    N = B if lens is None else len(lens)
    step = torch.exp(-6.9 + 4.6 * torch.rand(D, generator=g))
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    return {"x": rn(B, T, D).to(dt), "delta": (0.5 * rn(B, T, D)).to(dt),
            "A": -(torch.arange(1, S + 1) * torch.exp(0.1 * rn(D, S))), "B": rn(B, T, G, S).to(dt),
            "C": rn(B, T, G, S).to(dt), "D": 1 + 0.1 * rn(D) if skip else None,
            "z": rn(B, T, D).to(dt) if gate else None,
            "dt_bias": torch.log(torch.expm1(step)) if bias else None, "h0": 0.3 * rn(N, D, S) if init else None}
