"""Decayed linear attention and the norms around a block from their definitions, in 64 bits on the tensors' device:
the recurrence token by token, its gradients by the adjoint recurrence; the norms' gradients by their formulas."""
import torch


def sequences(q, cu):
    if cu is None:
        return [(n, n * q.shape[1], (n + 1) * q.shape[1]) for n in range(q.shape[0])]
    c = cu.tolist()
    return [(n, c[n], c[n + 1]) for n in range(len(c) - 1)]


def _flat(q, k, v, g):
    Hv = v.shape[2]
    of = torch.arange(Hv, device=v.device) // (Hv // q.shape[2])
    q, k = (t.double().reshape(-1, *t.shape[2:])[:, of] for t in (q, k))
    v = v.double().reshape(-1, *v.shape[2:])
    g = g.double().expand(v.shape[0], Hv) if g.dim() == 1 else g.double().reshape(-1, Hv)
    return q, k, v, g


def forward(q, k, v, g, scale, h0=None, cu=None):
    Q, K, X, L = _flat(q, k, v, g)
    seqs = sequences(q, cu)
    o = torch.zeros_like(X)
    ht = torch.zeros(len(seqs), X.shape[1], Q.shape[2], X.shape[2], dtype=torch.float64, device=v.device)
    for n, a, b in seqs:
        S = h0[n].double().clone() if h0 is not None else torch.zeros_like(ht[n])
        for t in range(a, b):
            S = torch.exp(L[t])[:, None, None] * S + K[t][:, :, None] * X[t][:, None, :]
            o[t] = scale * (Q[t][:, :, None] * S).sum(1)
        ht[n] = S
    return o.view(v.shape), ht


def backward(q, k, v, g, do, scale, h0=None, dht=None, cu=None):
    Q, K, X, L = _flat(q, k, v, g)
    D = do.double().reshape(X.shape)
    seqs = sequences(q, cu)
    dq, dk, dv, dg = torch.zeros_like(Q), torch.zeros_like(K), torch.zeros_like(X), torch.zeros_like(L)
    dh0 = torch.zeros(len(seqs), X.shape[1], Q.shape[2], X.shape[2], dtype=torch.float64, device=v.device)
    for n, a, b in seqs:
        S = [h0[n].double() if h0 is not None else torch.zeros_like(dh0[n])]
        for t in range(a, b):
            S.append(torch.exp(L[t])[:, None, None] * S[-1] + K[t][:, :, None] * X[t][:, None, :])
        G = dht[n].double().clone() if dht is not None else torch.zeros_like(dh0[n])
        for t in reversed(range(a, b)):
            i = t - a + 1
            dq[t] = scale * (S[i] * D[t][:, None, :]).sum(2)
            G = G + scale * Q[t][:, :, None] * D[t][:, None, :]
            dk[t] = (G * X[t][:, None, :]).sum(2)
            dv[t] = (G * K[t][:, :, None]).sum(1)
            G = torch.exp(L[t])[:, None, None] * G
            dg[t] = (G * S[i - 1]).sum((1, 2))
        dh0[n] = G
    R = X.shape[1] // q.shape[2]
    out = {"dq": dq.view(-1, q.shape[2], R, q.shape[3]).sum(2).view(q.shape),
           "dk": dk.view(-1, q.shape[2], R, q.shape[3]).sum(2).view(q.shape), "dv": dv.view(v.shape),
           "dg": dg.sum(0) if g.dim() == 1 else dg.view(g.shape), "dh0": dh0}
    return out


def rms(x, eps):
    return 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)


def rms_backward(a, xhat, r):
    return r * (a - xhat * (a * xhat).mean(-1, keepdim=True))


def gated_norm(x, z, w, eps, dy=None):
    x, w = x.double(), w.double()
    r = rms(x, eps)
    xhat = x * r
    s = torch.sigmoid(z.double()) if z is not None else None
    gate = z.double() * s if z is not None else torch.ones_like(x)
    y = xhat * w * gate
    if dy is None:
        return y
    dy = dy.double()
    out = {"dx": rms_backward(dy * gate * w, xhat, r), "dweight": (dy * gate * xhat).flatten(0, -2).sum(0)}
    if z is not None:
        out["dz"] = dy * xhat * w * s * (1 + z.double() * (1 - s))
    return out


def residual_norm(y, res, pw, gate, scale, w, eps, dh=None, dn=None):
    y = y.double()
    r1 = rms(y, eps)
    yhat = y * r1
    u = yhat * pw.double() if pw is not None else y
    gt = gate.double() if gate is not None else torch.ones_like(y)
    h = res.double() + scale * gt * u
    r2 = rms(h, eps)
    hhat = h * r2
    n = hhat * w.double() if w is not None else None
    if dh is None and dn is None:
        return h, n
    d = dh.double() if dh is not None else torch.zeros_like(h)
    out = {}
    if w is not None:
        out["dweight"] = (dn.double() * hhat).reshape(-1, h.shape[-1]).sum(0)
        d = d + rms_backward(dn.double() * w.double(), hhat, r2)
    out["dresidual"] = d
    if gate is not None:
        dg = scale * d * u
        out["dgate"] = dg if gate.shape == y.shape else dg.reshape(-1, h.shape[-1]).sum(0)
    du = scale * d * gt
    if pw is not None:
        out["dpost_weight"] = (du * yhat).reshape(-1, h.shape[-1]).sum(0)
        du = rms_backward(du * pw.double(), yhat, r1)
    out["dy"] = du
    return out


def rel(x, ref):
    """Relative Frobenius error; inputs of any type."""
    x, ref = x.detach().double(), ref.detach().double()
    n = float(torch.linalg.vector_norm(ref))
    d = float(torch.linalg.vector_norm(x - ref))
    return d / n if n else d
