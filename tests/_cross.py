"""Attention of queries to keys of another length in plain fp64 on the device, with elementwise
bounds on what the kernels may be off by.  Nothing here calls the library.

Bounds: u = 2^-24.  A score of d products of bf16 numbers, accumulated and scaled in fp32, is off by
s = 2 (d + 16) u of the largest absolute score sum of its row; a weight by 2 s, the exponential
(7.5e-5 where it is a polynomial, ex2.approx 2^-22) and the row's sum.  Sums of n terms add n 2^-23 of
the absolute sum.  P and dS enter the second products in bf16 (2^-8 of themselves), outputs round to
bf16 (2^-8)."""
from __future__ import annotations

import math

import torch

U = 2.0 ** -24
HALF = 2.0 ** -8
EXP = 1e-4


def visible(nq, nk, causal, device):
    i = torch.arange(nq, device=device)[:, None]
    j = torch.arange(nk, device=device)[None]
    return j <= i + (nk - nq) if causal else torch.ones((nq, nk), dtype=torch.bool, device=device)


def scores(q, k, causal, scale):
    """x [H, nq, nk] (-inf where masked) and the largest absolute score sum of each row."""
    G = q.shape[0] // k.shape[0]
    k = k.repeat_interleave(G, 0)
    seen = visible(q.shape[1], k.shape[1], causal, q.device)
    x = torch.where(seen, scale * q @ k.transpose(1, 2), -math.inf)
    size = scale * (q.abs() @ k.abs().transpose(1, 2))
    top = size.amax(-1) if k.shape[1] else size.new_zeros(size.shape[:2])
    return x, seen, top


def forward(q, k, v, causal, scale):
    """fp64 q [H, nq, d], k, v [Hkv, nk, d] -> o, lse and their bounds."""
    G = q.shape[0] // k.shape[0]
    v = v.repeat_interleave(G, 0)
    x, seen, top = scores(q, k, causal, scale)
    nk, d = v.shape[1], v.shape[2]
    if nk:
        lse = torch.logsumexp(x, -1)
    else:
        lse = x.new_full(x.shape[:2], -math.inf)
    w = torch.where(seen, torch.exp(x - torch.where(lse == -math.inf, 0.0, lse)[..., None]), 0.0)
    o, size = w @ v, w @ v.abs()
    s = 2 * (d + 16) * U * top
    rel = HALF + EXP + 2 * s[..., None] + 2 * (nk + 64) * 2 * U
    lse_room = s + EXP + (nk + 64) * 2 * U + 8 * U * torch.where(lse == -math.inf, 0.0, lse).abs()
    return o, lse, HALF * o.abs() + rel * size + 1e-30, lse_room


def backward(q, k, v, o, dout, lse, causal, scale):
    """{name: (gradient, bound)} from the o and lse that the kernels were given."""
    Hkv, G = k.shape[0], q.shape[0] // k.shape[0]
    nq, nk, d = q.shape[1], k.shape[1], q.shape[2]
    x, seen, top = scores(q, k, causal, scale)
    kk, vv = k.repeat_interleave(G, 0), v.repeat_interleave(G, 0)
    none = (lse == -math.inf)[..., None]
    p = torch.where(seen & ~none, torch.exp(x - torch.where(none, 0.0, lse[..., None])), 0.0)
    delta = (o * dout).sum(-1, keepdim=True)
    ds = p * (dout @ vv.transpose(1, 2) - delta)
    e_p = (2 * 2 * (d + 16) * U * top + 8 * U * torch.where(none[..., 0], 0.0, lse).abs() + 2 ** -21)
    e_dp = 2 * (d + 16) * U * (dout.abs() @ vv.abs().transpose(1, 2)
                               + (o * dout).abs().sum(-1, keepdim=True))
    off_p = p * (HALF + e_p[..., None])
    off_s = ds.abs() * (HALF + 2 * e_p[..., None]) + 1.1 * p * e_dp
    add = lambda n: 2 * (n + 64) * 2 * U

    def group(y):
        return y.reshape(Hkv, G, nk, d).sum(1)

    dq = scale * ds @ kk
    dk, dv = group(scale * ds.transpose(1, 2) @ q), group(p.transpose(1, 2) @ dout)
    bq = scale * (off_s + add(nk) * ds.abs()) @ kk.abs()
    bk = group(scale * (off_s + add(nq * G) * ds.abs()).transpose(1, 2) @ q.abs())
    bv = group((off_p + add(nq * G) * p).transpose(1, 2) @ dout.abs())
    return {n: (y, HALF * y.abs() + b * 1.01 + 1e-30) for n, y, b in
            (("dq", dq, bq), ("dk", dk, bk), ("dv", dv, bv))}


def inside(name, got, want, bound):
    err = (got.double() - want).abs()
    # (both infinite of one sign: no difference)
    err = torch.where(got.double() == want, 0.0, err)
    bad = ~(err <= bound)
    assert not bad.any(), (name, int(bad.sum()), float((err - bound)[bad].max()),
                           [int(i) for i in bad.nonzero()[0]])
