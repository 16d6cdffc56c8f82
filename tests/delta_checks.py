"""The gated delta rule and the norms around a block in float64, written as
plainly as their definitions, and inputs for their tests.

Runs on whatever device the inputs are on; shares nothing with the library.
"""
import math

import torch

F64 = torch.float64


def gated_delta(q, k, v, dt, A, beta, dt_bias=None, dt_softplus=True, beta_sigmoid=True,
                scale=None, h0=None, cu_seqlens=None):
    """Token by token: (y, last_state) in float64."""
    q, k, v, dt, A, beta = (t.to(F64) for t in (q, k, v, dt, A, beta))
    batch, L, H, P = v.shape
    G, N = q.shape[2:]
    scale = 1 / math.sqrt(N) if scale is None else scale
    if dt_bias is not None:
        dt = dt + dt_bias.to(F64)
    step = torch.logaddexp(dt, torch.zeros_like(dt)) if dt_softplus else dt
    a = torch.exp(step * A)
    b = 1 / (1 + torch.exp(-beta)) if beta_sigmoid else beta
    spans = [(i, 0, L) for i in range(batch)]
    if cu_seqlens is not None:
        cu = [min(max(int(c), 0), L) for c in cu_seqlens.tolist()]
        spans = [(0, lo, max(lo, hi)) for lo, hi in zip(cu, cu[1:])]
    y = torch.full((batch, L, H, P), float("nan"), dtype=F64, device=v.device)
    last = torch.zeros(len(spans), H, P, N, dtype=F64, device=v.device)
    if h0 is not None:
        last += h0.to(F64)
    per = H // G
    for i, (r, lo, hi) in enumerate(spans):
        S = last[i]
        for t in range(lo, hi):
            kt = k[r, t].repeat_interleave(per, 0)[:, None, :]
            qt = q[r, t].repeat_interleave(per, 0)[:, None, :]
            S = S * a[r, t][:, None, None]
            u = b[r, t][:, None] * (v[r, t] - (S * kt).sum(-1))
            S = S + u[:, :, None] * kt
            y[r, t] = scale * (S * qt).sum(-1)
        last[i] = S
    return y, last


def delta_inputs(batch, L, H, P, G, N, dtype, seed=0, device="cuda", h0=False, seqs=None,
                 signed=False):
    g = torch.Generator(device=device).manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device=device)  # noqa: E731
    def unit(t):
        t = t if signed else torch.nn.functional.silu(t)
        return torch.nn.functional.normalize(t, dim=-1)
    d = dict(q=unit(rnd(batch, L, G, N)).to(dtype), k=unit(rnd(batch, L, G, N)).to(dtype),
             v=rnd(batch, L, H, P).to(dtype), dt=rnd(batch, L, H).to(dtype),
             beta=rnd(batch, L, H).to(dtype),
             A=-(1 + 15 * torch.rand(H, generator=g, device=device)))
    step = 1e-3 + 0.099 * torch.rand(H, generator=g, device=device)
    d["dt_bias"] = torch.log(torch.expm1(step))
    d["h0"] = 0.25 * rnd(seqs or batch, H, P, N) if h0 else None
    return d


def gated_rmsnorm(x, z, w, eps, group, before):
    """y in float64; differentiable in float64 leaves."""
    gate = z / (1 + torch.exp(-z))
    a = x if before else x * gate
    a = a.reshape(*x.shape[:-1], -1, group)
    n = a / torch.sqrt(a.pow(2).sum(-1, keepdim=True) / group + eps)
    y = (n * w.reshape(-1, group)).reshape(x.shape)
    return y * gate if before else y


def rmsnorm(r, w, eps):
    return r / torch.sqrt(r.pow(2).mean(-1, keepdim=True) + eps) * w


def worst(got, want, terms=None):
    """Largest |difference| over the largest |value|, or over the largest of
    the `terms` whose difference the value is; infinite where a value is
    missing or not finite."""
    got, want = got.detach().to(F64).cpu(), want.detach().cpu()
    if got.shape != want.shape or not torch.isfinite(got).all():
        return math.inf
    if not want.numel():
        return 0.0
    size = want.abs().max()
    if terms is not None:
        size = torch.maximum(size, terms.detach().to(F64).cpu().abs().max())
    return float((got - want).abs().max() / size.clamp(min=1e-300))
