"""Plain 64-bit token-by-token references of the decode and backward operators
(torch, any device), and the tolerances their tests use.

The state is H = S^T [d_k, d_v]; per token
    Hd = e^g H,  u = v - Hd^T k,  H' = Hd + beta k u^T,  o = scale H'^T q.
"""
from __future__ import annotations

import torch

# A bf16 rounding is off by at most half a step, 2^-8 of the value, so a tensor
# rounded once is off by at most 2^-8 of its norm; the f32 arithmetic before it
# adds far less (F32_REL below).
BF16_REL = 2.0 ** -8
# f32 products of d <= 128 terms: a rounding is 2^-24, a sum of 128 terms is off
# by at most 128 roundings (7.6e-6) of its terms' size and, the roundings being
# unrelated, by about sqrt(128) of them (6.7e-7); a dozen such products follow
# one another, which adds up to 128 * 2^-24 * 12 / sqrt(12) at the most.
F32_REL = 128 * 2.0 ** -24 * 12 ** 0.5


def offsets(lens):
    cu = [0]
    for x in lens:
        cu.append(cu[-1] + int(x))
    return cu


def rel(a, b) -> float:
    """2-norm of a - b over that of b (of b = 0: the norm of a)."""
    a, b = a.detach().cpu().double(), b.detach().cpu().double()
    n = float(b.norm())
    return float((a - b).norm()) / (n if n else 1.0)


def _rows64(q, k, v, g, beta):
    vpg = v.shape[1] // q.shape[1]
    return (q.double().repeat_interleave(vpg, 1), k.double().repeat_interleave(vpg, 1),
            v.double(), g.double().exp(), beta.double())


def forward(q, k, v, g, beta, lens, h0=None, scale=1.0):
    """o [T, H_v, d] and the final states [N, H_v, d, d] in 64 bits."""
    q, k, v, a, beta = _rows64(q, k, v, g, beta)
    T, Hv, d = v.shape
    o, out, cu = torch.zeros_like(v), [], offsets(lens)
    for b in range(len(lens)):
        h = v.new_zeros(Hv, d, d) if h0 is None else h0[b].double()
        for t in range(cu[b], cu[b + 1]):
            h = a[t][:, None, None] * h
            u = v[t] - torch.einsum("hij,hi->hj", h, k[t])
            h = h + torch.einsum("h,hi,hj->hij", beta[t], k[t], u)
            o[t] = scale * torch.einsum("hij,hi->hj", h, q[t])
        out.append(h)
    return o, torch.stack(out)


def backward(q, k, v, g, beta, lens, do, h0=None, dhT=None, scale=1.0):
    """The gradients (dq, dk, dv, dg, dbeta, dh0) in 64 bits."""
    Hk = q.shape[1]
    q, k, v, a, beta = _rows64(q, k, v, g, beta)
    do = do.double()
    T, Hv, d = v.shape
    dq, dk, dv = torch.zeros_like(v), torch.zeros_like(v), torch.zeros_like(v)
    dg, dbeta, dh0, cu = torch.zeros_like(beta), torch.zeros_like(beta), [], offsets(lens)
    for b in range(len(lens)):
        h = v.new_zeros(Hv, d, d) if h0 is None else h0[b].double()
        kept = []
        for t in range(cu[b], cu[b + 1]):
            hd = a[t][:, None, None] * h
            u = v[t] - torch.einsum("hij,hi->hj", hd, k[t])
            h = hd + torch.einsum("h,hi,hj->hij", beta[t], k[t], u)
            kept.append((hd, u, h))
        dh = v.new_zeros(Hv, d, d) if dhT is None else dhT[b].double()
        for t in range(cu[b + 1] - 1, cu[b] - 1, -1):
            hd, u, h = kept.pop()
            dq[t] = scale * torch.einsum("hij,hj->hi", h, do[t])
            dh = dh + scale * torch.einsum("hi,hj->hij", q[t], do[t])
            w = torch.einsum("hij,hi->hj", dh, k[t])
            dbeta[t] = (w * u).sum(-1)
            du = beta[t][:, None] * w
            dv[t] = du
            dk[t] = beta[t][:, None] * torch.einsum("hij,hj->hi", dh, u) - \
                torch.einsum("hij,hj->hi", hd, du)
            dh = dh - torch.einsum("hi,hj->hij", k[t], du)
            dg[t] = (dh * hd).sum((-2, -1))
            dh = a[t][:, None, None] * dh
        dh0.append(dh)
    vpg = Hv // Hk
    dq, dk = (x.view(T, Hk, vpg, d).sum(2) for x in (dq, dk))
    return dq, dk, dv, dg, dbeta, torch.stack(dh0)


def rows(gen, T, Hk, Hv, d, device="cpu"):
    """q, k (unit length), v bf16, g = logsigmoid(N(2, 1)), beta = sigmoid(N(0, 1))."""
    def n(*shape):
        return torch.randn(shape, generator=gen).to(device)

    def unit(x):
        return (x / x.norm(dim=-1, keepdim=True).clamp_min(1e-6)).to(torch.bfloat16)

    return (unit(n(T, Hk, d)), unit(n(T, Hk, d)), n(T, Hv, d).to(torch.bfloat16),
            torch.nn.functional.logsigmoid(n(T, Hv) + 2.0), torch.sigmoid(n(T, Hv)))
