"""A decayed linear attention layer on the library's operators, and a stack of mixers with norms around them:

    q, k, v, z = in_proj(u);  a = a_proj(u)
    g     = -exp(A_log) softplus(a + dt_bias)            (or one fixed decay a head)
    o     = linear_attn(q, k, v, g)
    out   = out_proj(silu(z) * rms_norm(o) * norm_weight)       head by head

    Stack:  n = norm(h);  y = mixer(n);  h = h + scale * gate * post_norm(y);  n = norm(h);  ...

A stack's mixers are layers of this module or selective layers.  Training and prompts multiply by bf16 weights (torch);
a decode step reads 4-bit weights with group scales (``quantize_``).  A layer's states live in a pool with a slot for
every sequence.
"""
from __future__ import annotations

import math

import torch

from . import binding as gdn
from .selective_layer import _first_order, quantize


class LinearAttention(torch.autograd.Function):
    """gdn_linear_attn_fwd / _bwd from zero states."""

    @staticmethod
    def forward(ctx, q, k, v, g, scale, cu_seqlens):
        ctx.save_for_backward(q, k, v, g, cu_seqlens)
        ctx.scale = scale
        return gdn.gdn_linear_attn_fwd(q, k, v, g, scale=scale, cu_seqlens=cu_seqlens, output_final_state=False)[0]

    @staticmethod
    @_first_order
    def backward(ctx, do):
        q, k, v, g, cu = ctx.saved_tensors
        d = gdn.gdn_linear_attn_bwd(q, k, v, g, do.contiguous(), scale=ctx.scale, cu_seqlens=cu)
        return d["dq"], d["dk"], d["dv"], d["dg"], None, None


class GatedNorm(torch.autograd.Function):
    """gdn_gated_norm_fwd / _bwd; z may be None."""

    @staticmethod
    def forward(ctx, x, z, weight, eps):
        y, rstd = gdn.gdn_gated_norm_fwd(x, z, weight, eps=eps, save_rstd=True)
        ctx.save_for_backward(x, z, weight, rstd)
        return y

    @staticmethod
    @_first_order
    def backward(ctx, dy):
        x, z, weight, rstd = ctx.saved_tensors
        d = gdn.gdn_gated_norm_bwd(x, z, weight, rstd, dy.contiguous())
        return d["dx"], d["dz"], d["dweight"], None


class ResidualNorm(torch.autograd.Function):
    """gdn_residual_norm_fwd / _bwd: (h, n) of a block's output y and the residual."""

    @staticmethod
    def forward(ctx, y, residual, post_weight, gate, scale, weight, eps):
        h, n, rstd = gdn.gdn_residual_norm_fwd(y, residual, post_weight=post_weight, gate=gate, residual_scale=scale,
                                               weight=weight, eps=eps, save_rstd=True)
        ctx.save_for_backward(y, residual, post_weight, gate, weight, rstd)
        ctx.scale = scale
        ctx.set_materialize_grads(False)
        return h, n

    @staticmethod
    @_first_order
    def backward(ctx, dh, dn):
        y, residual, post_weight, gate, weight, rstd = ctx.saved_tensors
        if weight is None:
            dn = None   # there was no n
        else:
            dn = torch.zeros_like(y, memory_format=torch.contiguous_format) if dn is None else dn.contiguous()
        d = gdn.gdn_residual_norm_bwd(y, residual, rstd, None if dh is None else dh.contiguous(), dn,
                                      post_weight=post_weight, gate=gate, residual_scale=ctx.scale, weight=weight)
        return d["dy"], d["dresidual"], d["dpost_weight"], d["dgate"], None, d["dweight"], None


PROJECTIONS = ("in_proj", "a_proj", "out_proj")


class LinearLayer(torch.nn.Module):
    """width: the model's; heads q/k heads and value_heads value heads (a multiple) of K and V dims (64, 128 or 256);
    decay "token" (from the input) or "head" (a fixed geometric series of slopes, not trained)."""

    def __init__(self, width, heads, value_heads=None, K=128, V=128, decay="token", eps=1e-6, device="cuda"):
        super().__init__()
        if decay not in ("token", "head"):
            raise ValueError('decay must be "token" or "head"')
        self.Hqk, self.Hv, self.K, self.V, self.eps = heads, value_heads or heads, K, V, eps
        bf = dict(dtype=torch.bfloat16, device=device)

        def matrix(n, k):
            return torch.nn.Parameter(torch.randn(n, k, **bf) * k ** -0.5)

        self.in_proj = matrix(2 * self.Hqk * K + 2 * self.Hv * V, width)
        self.out_proj = matrix(width, self.Hv * V)
        self.norm_weight = torch.nn.Parameter(torch.ones(V, device=device))
        self.decay = decay
        if decay == "token":
            self.a_proj = matrix(self.Hv, width)
            self.A_log = torch.nn.Parameter(torch.log(1 + 15 * torch.rand(self.Hv, device=device)))
            step = torch.exp(torch.rand(self.Hv, device=device) * math.log(100) + math.log(1e-3))   # in [1e-3, 1e-1]
            self.dt_bias = torch.nn.Parameter(torch.log(torch.expm1(step)))
        else:
            self.register_buffer("slopes", -torch.exp2(-8.0 * torch.arange(1, self.Hv + 1, device=device) / self.Hv))

    @property
    def q4(self):
        """{projection: (codes, scales)} of step(), or None before quantize_()."""
        b = self._buffers
        return {k: (b[k + "_codes"], b[k + "_scales"]) for k in PROJECTIONS if k + "_codes" in b} or None

    def _load_from_state_dict(self, state_dict, prefix, *args):
        """A checkpoint of a quantized layer brings its 4-bit weights; those of a layer that gets other parameters
        without any are dropped."""
        names = [k + kind for k in PROJECTIONS if hasattr(self, k) for kind in ("_codes", "_scales")]
        if all(prefix + k in state_dict for k in names):
            for k in names:
                self.register_buffer(k, torch.empty_like(state_dict[prefix + k], device=self.in_proj.device))
        elif any(prefix + k in state_dict for k in PROJECTIONS):
            for k in names:
                self._buffers.pop(k, None)
        super()._load_from_state_dict(state_dict, prefix, *args)

    def _split(self, p):
        """q, k, v, z [..., heads, dim] as slices of the projection's rows."""
        qk, vz = self.Hqk * self.K, self.Hv * self.V
        q, k, v, z = p.split([qk, qk, vz, vz], dim=-1)
        return (q.unflatten(-1, (self.Hqk, self.K)), k.unflatten(-1, (self.Hqk, self.K)),
                v.unflatten(-1, (self.Hv, self.V)), z.unflatten(-1, (self.Hv, self.V)))

    def _log_decay(self, a):
        if self.decay == "head":
            return self.slopes
        return -torch.exp(self.A_log) * torch.nn.functional.softplus(a.float() + self.dt_bias)

    def _decays(self, u):
        return self._log_decay(u @ self.a_proj.t() if self.decay == "token" else None)

    def _scale(self):
        return self.K ** -0.5

    def forward(self, u, cu_seqlens=None):
        """u [B, T, width] (packed with cu_seqlens when B == 1), with gradients."""
        q, k, v, z = self._split(u @ self.in_proj.t())
        o = LinearAttention.apply(q, k, v, self._decays(u), self._scale(), cu_seqlens)
        return GatedNorm.apply(o, z, self.norm_weight, self.eps).flatten(-2) @ self.out_proj.t()

    # ------------------------------------------------------------- serving

    def new_states(self, slots):
        """A zeroed pool [slots, Hv, K, V]."""
        return torch.zeros(slots, self.Hv, self.K, self.V, device=self.in_proj.device)

    @torch.no_grad()
    def quantize_(self, group=32):
        """4-bit copies of the projections for step(): buffers, which move and are saved with the layer.  To be called
        again when the parameters have changed."""
        for k in PROJECTIONS:
            if hasattr(self, k):
                codes, scales = quantize(getattr(self, k), group)
                self.register_buffer(k + "_codes", codes)
                self.register_buffer(k + "_scales", scales)
        return self

    @torch.no_grad()
    def prompt(self, u, states, slots, cu_seqlens=None):
        """New sequences' prompts; their states go to the pool's rows ``slots`` (int32).  A slot outside the pool means
        "no state": the outputs are computed and nothing is kept."""
        q, k, v, z = self._split(u @ self.in_proj.t())
        o, _ = gdn.gdn_linear_attn_fwd(q, k, v, self._decays(u), scale=self._scale(), cu_seqlens=cu_seqlens, ht=states,
                                       state_indices=slots)
        return gdn.gdn_gated_norm_fwd(o, z, self.norm_weight, eps=self.eps)[0].flatten(-2) @ self.out_proj.t()

    @torch.no_grad()
    def step(self, u, states, slots):
        """One token of every sequence: u [N, width] on the pool's rows ``slots``, with the 4-bit weights."""
        q4 = self.q4
        if q4 is None:
            raise RuntimeError("step() multiplies by 4-bit weights: call quantize_() first")
        q, k, v, z = self._split(gdn.gdn_q4_matvec(u, *q4["in_proj"]))
        g = self._log_decay(gdn.gdn_q4_matvec(u, *q4["a_proj"])[:, None] if self.decay == "token" else None)
        o = gdn.gdn_linear_attn_step(q[:, None], k[:, None], v[:, None], g, states, scale=self._scale(),
                                     state_indices=slots)
        y, _ = gdn.gdn_gated_norm_fwd(o[:, 0], z, self.norm_weight, eps=self.eps)
        return gdn.gdn_q4_matvec(y.flatten(1), *q4["out_proj"])


class Stack(torch.nn.Module):
    """Mixers (LinearLayer, SelectiveLayer) with a norm before and after each, a gate a channel and a scaled residual
    sum: n = norm(h), h = h + scale * gate * post_norm(mixer(n)).  Between two mixers all of it is one pass.  Returns
    the last norm's output.  residual_dtype: of the sums h (the mixers' type, or float32)."""

    def __init__(self, mixers, width, scale=1.0, residual_dtype=torch.bfloat16, eps=1e-6, device="cuda"):
        super().__init__()
        self.mixers = torch.nn.ModuleList(mixers)
        self.scale, self.residual_dtype, self.eps = scale, residual_dtype, eps
        ones = [torch.nn.Parameter(torch.ones(width, device=device)) for _ in range(3 * len(mixers) + 1)]
        n = len(mixers)
        self.first_weight = ones[0]
        self.post_weights = torch.nn.ParameterList(ones[1:n + 1])
        self.gates = torch.nn.ParameterList(ones[n + 1:2 * n + 1])
        self.weights = torch.nn.ParameterList(ones[2 * n + 1:])

    def forward(self, u, cu_seqlens=None):
        n = GatedNorm.apply(u.unsqueeze(-2), None, self.first_weight, self.eps).squeeze(-2)
        h = u.to(self.residual_dtype).contiguous()
        for mixer, post, gate, weight in zip(self.mixers, self.post_weights, self.gates, self.weights):
            h, n = ResidualNorm.apply(mixer(n, cu_seqlens), h, post, gate, self.scale, weight, self.eps)
        return n

    def new_states(self, slots):
        return [m.new_states(slots) for m in self.mixers]

    def quantize_(self, group=32):
        for m in self.mixers:
            m.quantize_(group)
        return self

    @torch.no_grad()
    def _serve(self, u, mix):
        n, _ = gdn.gdn_gated_norm_fwd(u.unsqueeze(-2), None, self.first_weight, eps=self.eps)
        n, h = n.squeeze(-2), u.to(self.residual_dtype, copy=True).contiguous()
        for i, (post, gate, weight) in enumerate(zip(self.post_weights, self.gates, self.weights)):
            h, n, _ = gdn.gdn_residual_norm_fwd(mix(i, n), h, post_weight=post, gate=gate, residual_scale=self.scale,
                                                weight=weight, eps=self.eps, h=h)
        return n

    def prompt(self, u, states, slots, cu_seqlens=None):
        return self._serve(u, lambda i, n: self.mixers[i].prompt(n, states[i], slots, cu_seqlens))

    def step(self, u, states, slots):
        return self._serve(u, lambda i, n: self.mixers[i].step(n, states[i], slots))
