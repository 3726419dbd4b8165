"""A selective state space layer on the library's operators, for training, prompts
and decoding:

    x, z  = in_proj(u)                       (two halves of one product)
    x     = silu(causal_conv1d(x))
    dt, B, C = x_proj(x);  delta = dt_proj(dt)
    y     = selective_scan(x, delta, A, B, C, D, z)
    out   = out_proj(y)

Training and prompts multiply by bf16 weights (torch); a decode step reads 4-bit
weights with group scales (``quantize``), since a token's time is its weights' bytes.
States live in pools with a slot for every sequence: the last W - 1 inputs of the
convolution and the scan's state.
"""
from __future__ import annotations

import functools
import math

import torch

from . import binding as gdn


class _FirstOrder(torch.autograd.Function):
    """Gradients as they are; differentiating them again raises."""

    @staticmethod
    def forward(ctx, anchor, *grads):
        return grads

    @staticmethod
    def backward(ctx, *_):
        raise RuntimeError("the selective layer's operators have first derivatives only: their gradients cannot be "
                           "differentiated again")


def _first_order(backward):
    """For a backward that torch cannot differentiate.  Under create_graph its gradients would count as constants;
    here they depend on something, so that a second derivative through them raises, whether or not the incoming
    gradient needs one (the operator's inputs, which they depend on too, may)."""

    @functools.wraps(backward)
    def call(ctx, *dys):
        with torch.no_grad():
            grads = backward(ctx, *dys)
        if not torch.is_grad_enabled():   # no graph of the gradients is wanted
            return grads
        some = [i for i, g in enumerate(grads) if g is not None]
        anchor = torch.zeros((), device=grads[some[0]].device, requires_grad=True)
        grads = list(grads)
        for i, g in zip(some, _FirstOrder.apply(anchor, *(grads[i] for i in some))):
            grads[i] = g
        return tuple(grads)
    return call


class CausalConv1d(torch.autograd.Function):
    """gdn_causal_conv1d_fwd / _bwd from zero initial inputs."""

    @staticmethod
    def forward(ctx, x, weight, bias, cu_seqlens):
        ctx.save_for_backward(x, weight, bias, cu_seqlens)
        return gdn.gdn_causal_conv1d_fwd(x, weight, bias, "silu", cu_seqlens=cu_seqlens)

    @staticmethod
    @_first_order
    def backward(ctx, dy):
        x, weight, bias, cu = ctx.saved_tensors
        g = gdn.gdn_causal_conv1d_bwd(x, weight, dy.contiguous(), bias=bias, activation="silu", cu_seqlens=cu)
        return g["dx"], g["dweight"], g["dbias"], None


class SelectiveScan(torch.autograd.Function):
    """gdn_selective_scan_fwd / _bwd from zero states."""

    @staticmethod
    def forward(ctx, x, delta, A, B, C, D, z, dt_bias, cu_seqlens):
        ctx.save_for_backward(x, delta, A, B, C, D, z, dt_bias, cu_seqlens)
        return gdn.gdn_selective_scan_fwd(x, delta, A, B, C, D=D, z=z, dt_bias=dt_bias, cu_seqlens=cu_seqlens,
                                          output_final_state=False)[0]

    @staticmethod
    @_first_order
    def backward(ctx, dy):
        x, delta, A, B, C, D, z, dt_bias, cu = ctx.saved_tensors
        g = gdn.gdn_selective_scan_bwd(x, delta, A, B, C, dy.contiguous(), D=D, z=z, dt_bias=dt_bias, cu_seqlens=cu)
        return (*(g[k] for k in ("dx", "ddelta", "dA", "dB", "dC", "dD", "dz", "ddt_bias")), None)


def quantize(w: torch.Tensor, group: int = 64):
    """(qweight, scales) of a weight matrix [N, K] for gdn_q4_matvec: codes of the nearest multiples of a scale per
    group of K, with 8 for zero; scales in bf16."""
    N, K = w.shape
    g = w.float().view(N, K // group, group)
    scales = (g.abs().amax(-1) / 7).clamp(min=1e-12).to(torch.bfloat16)
    q = (torch.round(g / scales.float()[..., None]) + 8).clamp(0, 15).to(torch.uint8).view(N, K)
    return (q[:, 0::2] | (q[:, 1::2] << 4)).contiguous(), scales


def dequantize(qweight: torch.Tensor, scales: torch.Tensor) -> torch.Tensor:
    """The weights that the codes stand for, fp32."""
    q = torch.stack((qweight & 15, qweight >> 4), -1).view(qweight.shape[0], scales.shape[1], -1).float() - 8
    return (q * scales.float()[..., None]).view(qweight.shape[0], -1)


PROJECTIONS = ("in_proj", "x_proj", "dt_proj", "out_proj")


class SelectiveLayer(torch.nn.Module):
    """width: the model's; channels D, states S a channel, groups G that share B and C, W taps, rank of the step."""

    def __init__(self, width, channels, states=16, groups=1, taps=4, rank=None, device="cuda"):
        super().__init__()
        rank = rank or max(32, 32 * (width // 512))
        self.D, self.S, self.G, self.W, self.rank = channels, states, groups, taps, rank
        bf = dict(dtype=torch.bfloat16, device=device)

        def matrix(n, k):
            return torch.nn.Parameter(torch.randn(n, k, **bf) * k ** -0.5)

        self.in_proj = matrix(2 * channels, width)
        self.x_proj = matrix(rank + 2 * groups * states, channels)
        self.dt_proj = matrix(channels, rank)
        self.out_proj = matrix(width, channels)
        self.conv_weight = torch.nn.Parameter(torch.randn(channels, taps, device=device) * taps ** -0.5)
        self.conv_bias = torch.nn.Parameter(torch.zeros(channels, device=device))
        self.A_log = torch.nn.Parameter(torch.log(torch.arange(1, states + 1, device=device).float()).repeat(channels, 1))
        self.Dskip = torch.nn.Parameter(torch.ones(channels, device=device))
        step = torch.exp(torch.rand(channels, device=device) * math.log(100) + math.log(1e-3))   # in [1e-3, 1e-1]
        self.dt_bias = torch.nn.Parameter(torch.log(torch.expm1(step)))

    @property
    def q4(self):
        """{projection: (codes, scales)} of step(), or None before quantize_()."""
        b = self._buffers
        return {k: (b[k + "_codes"], b[k + "_scales"]) for k in PROJECTIONS} if "A" in b else None

    def _load_from_state_dict(self, state_dict, prefix, *args):
        """A checkpoint of a quantized layer brings its 4-bit weights; those of a layer that gets other parameters
        without any are dropped."""
        names = [k + kind for k in PROJECTIONS for kind in ("_codes", "_scales")] + ["A"]
        if all(prefix + k in state_dict for k in names):
            for k in names:
                self.register_buffer(k, torch.empty_like(state_dict[prefix + k], device=self.in_proj.device))
        elif any(prefix + k in state_dict for k in (*PROJECTIONS, "A_log")):
            for k in names:
                self._buffers.pop(k, None)
        super()._load_from_state_dict(state_dict, prefix, *args)

    def _split(self, dbc):
        dt, B, C = dbc.split([self.rank, self.G * self.S, self.G * self.S], dim=-1)
        return dt, B.unflatten(-1, (self.G, self.S)), C.unflatten(-1, (self.G, self.S))

    def forward(self, u, cu_seqlens=None):
        """u [B, T, width] (packed with cu_seqlens when B == 1), with gradients."""
        x, z = (u @ self.in_proj.t()).chunk(2, dim=-1)
        x = CausalConv1d.apply(x.contiguous(), self.conv_weight, self.conv_bias, cu_seqlens)
        dt, B, C = self._split(x @ self.x_proj.t())
        y = SelectiveScan.apply(x, dt @ self.dt_proj.t(), -torch.exp(self.A_log), B, C, self.Dskip, z, self.dt_bias,
                                cu_seqlens)
        return y @ self.out_proj.t()

    # ------------------------------------------------------------- serving

    def new_states(self, slots):
        """Zeroed pools: (convolution inputs [slots, W - 1, D], scan states [slots, D, S])."""
        dev = self.in_proj.device
        return (torch.zeros(slots, self.W - 1, self.D, dtype=torch.bfloat16, device=dev),
                torch.zeros(slots, self.D, self.S, device=dev))

    @torch.no_grad()
    def quantize_(self, group=32):
        """4-bit copies of the projections (and the decay rates) for step(): buffers, which move and are saved with
        the layer.  To be called again when the parameters have changed."""
        for k in PROJECTIONS:
            codes, scales = quantize(getattr(self, k), group)
            self.register_buffer(k + "_codes", codes)
            self.register_buffer(k + "_scales", scales)
        self.register_buffer("A", -torch.exp(self.A_log))
        return self

    @torch.no_grad()
    def prompt(self, u, states, slots, cu_seqlens=None):
        """New sequences' prompts; their states go to the pools' rows ``slots`` (int32).  A slot outside the pools
        means "no state": the outputs are computed and nothing is kept.  Malformed cu_seqlens leave the scan's pool
        as it is."""
        conv, scan = states
        n = cu_seqlens.numel() - 1 if cu_seqlens is not None else u.shape[0]
        x, z = (u @ self.in_proj.t()).chunk(2, dim=-1)
        x = gdn.gdn_causal_conv1d_fwd(x.contiguous(), self.conv_weight, self.conv_bias, "silu", conv_state=conv,
                                      cache_indices=slots, has_initial_state=torch.zeros(n, dtype=torch.int32,
                                                                                         device=u.device),
                                      cu_seqlens=cu_seqlens)
        dt, B, C = self._split(x @ self.x_proj.t())
        y, _ = gdn.gdn_selective_scan_fwd(x, dt @ self.dt_proj.t(), -torch.exp(self.A_log), B, C, D=self.Dskip, z=z,
                                          dt_bias=self.dt_bias, cu_seqlens=cu_seqlens, ht=scan, state_indices=slots)
        return y @ self.out_proj.t()

    @torch.no_grad()
    def step(self, u, states, slots):
        """One token of every sequence: u [N, width] on the pools' rows ``slots``, with the 4-bit weights."""
        conv, scan = states
        q4 = self.q4
        if q4 is None:
            raise RuntimeError("step() multiplies by 4-bit weights: call quantize_() first")

        def product(v, name):
            return gdn.gdn_q4_matvec(v, *q4[name])

        x, z = product(u, "in_proj").chunk(2, dim=-1)
        x = gdn.gdn_causal_conv1d_fwd(x.contiguous()[:, None], self.conv_weight, self.conv_bias, "silu",
                                      conv_state=conv, cache_indices=slots)
        dt, B, C = self._split(product(x[:, 0], "x_proj"))
        delta = product(dt, "dt_proj")
        y = gdn.gdn_selective_scan_step(x, delta[:, None], self.A, B[:, None], C[:, None], scan, D=self.Dskip,
                                        z=z[:, None], dt_bias=self.dt_bias, state_indices=slots)
        return product(y[:, 0], "out_proj")
