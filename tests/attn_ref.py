"""64-bit references of the attention operators, and how far a kernel may be
from them.

Bounds (u = eps / 2 of the I/O dtype, f = 2^-23: one fp32 operation of a
tensor core, whose adds may truncate):

* A score is an fp32 dot product of D terms, then one or two more fp32
  operations and the exponential: its error is at most
  d = (D + 16) * f * max_j scale * sum_i |q_i k_ji|, plus 16 f * |s|.
* A weight is off by a factor within 1 +- 2 d (numerator and sum), and its
  rounding to the dtype by 1 +- u; below the normal range of fp16 (weights
  are at most 1 relative to the row's maximum, the sum is at least 1) the
  rounding is at most 2^-25 absolutely.
* Sums over L keys add at most (L + 64) * f relative to sum p_j |v_j|, and
  the output's rounding u * |out| (2^-25 below fp16's normal range).

With a = sum_j p_j |v_j| an element of the output is therefore within
  (2 u + 2 d + (L + 64) f) * a * 1.01 + [fp16] 2^-25 (sum_j |v_j| / l + 1)
and the log-sum-exp within d + (L + 64) f + 4 f |lse|.
"""
import math

import torch

F = 2.0 ** -23


def attend(q, k, v, first, scale, dtype, causal=True):
    """q [n, H, D], k [L, D] or [H, L, D], v alike, fp64; row i sees keys 0 .. first + i (causal) or all.
    Returns out, lse and their error bounds."""
    n, H, D = q.shape
    L = k.shape[-2]
    dev = q.device
    if k.dim() == 2:
        k, v = k.expand(H, L, D), v.expand(H, L, v.shape[-1])
    q = q.transpose(0, 1)
    s = torch.matmul(q, k.transpose(1, 2)) * scale
    mag = torch.matmul(q.abs(), k.abs().transpose(1, 2)) * abs(scale)
    if causal:
        gone = torch.arange(L, device=dev)[None, :] > first + torch.arange(n, device=dev)[:, None]
    else:
        gone = torch.zeros(n, L, dtype=torch.bool, device=dev)
    s = s.masked_fill(gone, -math.inf)
    mag = mag.masked_fill(gone, 0.0)
    some = ~gone.all(dim=-1)                                       # [n]
    m = s.amax(dim=-1, keepdim=True) if L else torch.full((H, n, 1), -math.inf, dtype=torch.float64, device=dev)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    e = torch.exp(s - m)
    l = e.sum(-1, keepdim=True)
    p = e / torch.where(l == 0, torch.ones_like(l), l)
    out = torch.matmul(p, v)
    lse = (m + torch.log(l)).squeeze(-1)
    u = torch.finfo(dtype).eps / 2
    d = (D + 16) * F * (mag.amax(-1) if L else torch.zeros(H, n, dtype=torch.float64, device=dev)) + 16 * F * m.abs().squeeze(-1)
    a = torch.matmul(p, v.abs())
    tol = (2 * u + 2 * d[..., None] + (L + 64) * F) * a * 1.01
    if dtype == torch.float16:
        tol = tol + 2.0 ** -25 * (v.abs().sum(-2, keepdim=True) / l.clamp(min=1.0) + 1.0)
    ltol = d + (L + 64) * F + 4 * F * torch.where(torch.isinf(lse), torch.zeros_like(lse), lse.abs())
    out = torch.where(some[None, :, None], out, torch.zeros_like(out))
    return out.transpose(0, 1), lse.transpose(0, 1), tol.transpose(0, 1), ltol.transpose(0, 1)


def check(name, got, ref, tol):
    got = got.double()
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    inf = torch.isinf(ref)
    assert torch.equal(inf, torch.isinf(got)) and torch.equal(got[inf], ref[inf]), f"{name}: infinities"
    assert torch.isfinite(got[~inf]).all(), f"{name}: non-finite values"
    over = (got - ref)[~inf].abs() / tol[~inf].clamp(min=1e-300)
    if over.numel():
        assert over.max().item() <= 1.0, f"{name}: error {over.max().item():.3g} times the bound"


def rope(x, cos, sin):
    """De-interleave and rotate halves, in x's type (fp64): x [..., 64]."""
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.cat((a * cos[..., :32] - b * sin[..., :32], b * cos[..., 32:] + a * sin[..., 32:]), dim=-1)
