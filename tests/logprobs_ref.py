"""Log probabilities of tokens, entropy, top alternatives and gradient in 64 bits (torch on the
CPU), with bounds on what fp32 arithmetic may be off by."""
from __future__ import annotations

import torch


def forward(x, tokens, scale, top=0):
    """x [rows, vocab] of any type. (results, bounds): dicts of 64-bit tensors.

    With d = scale (x - m) and S = sum exp(d): the exponent d log2(e) is rounded three times and
    the approximate exponential adds 2^-22, so a weight is off by 2^-21 + |d| 2^-22 relatively; a
    thread adds up at most vocab / 512 + 32 terms of S and T one after the other. Hence S is off by
    ds = 2^-21 + 2^-22 E|d| + (vocab / 512 + 32) 2^-24 relatively (E: over p) and log S by that and
    2^-23 of itself; T / S = E d by 2 ds E|d| + 2^-22 E d^2. The given logit's d is rounded twice."""
    y = x.double()
    live = (tokens >= 0) & (tokens < y.shape[1])
    m = y.amax(1, keepdim=True)
    none = m == -torch.inf
    d = torch.where(none, torch.zeros_like(y), (y - m) * scale)
    w = torch.where(none, torch.zeros_like(y), d.exp())
    S = torch.where(none, torch.ones_like(m), w.sum(1, keepdim=True))
    p, log_s = w / S, S.log()
    dd = torch.where(p > 0, d, torch.zeros_like(d))
    mean, mean_abs, mean_sq = ((p * z).sum(1) for z in (dd, dd.abs(), dd * dd))
    log_p = torch.where(none, torch.full_like(y, -torch.inf), d - log_s)
    entropy = torch.where(none[:, 0], torch.zeros_like(mean), log_s[:, 0] - mean)
    ds = 2.0 ** -21 + 2.0 ** -22 * mean_abs + (y.shape[1] / 512 + 32) * 2.0 ** -24
    d_log_s = ds + 2.0 ** -23 * log_s[:, 0].abs()
    at = tokens.long().clamp(0, y.shape[1] - 1)[:, None]

    def of(i):  # log p of columns i and its bound
        v = log_p.gather(1, i)
        e = 2.0 ** -22 * d.gather(1, i).abs() + d_log_s[:, None] + 2.0 ** -23 * v.abs()
        return v, torch.where(v.isinf(), torch.zeros_like(e), e)

    order = torch.sort(torch.nan_to_num(y, nan=-torch.inf, posinf=torch.inf, neginf=-torch.inf) + 0.0,
                       dim=1, descending=True, stable=True).indices[:, :top]
    v, e = of(at)
    tv, te = of(order)
    zero = torch.zeros(())
    pick = lambda z, other=zero: torch.where(live.view(-1, *[1] * (z.dim() - 1)), z, other.to(z.dtype))  # noqa: E731
    got = {"logprob": pick(v[:, 0]), "entropy": pick(entropy),
           "stats": pick(torch.cat([m, torch.where(none, torch.zeros_like(log_s), log_s)], 1)),
           "top_logprob": pick(tv), "top_token": pick(order, torch.tensor(-1))}
    bound = {"logprob": e[:, 0], "top_logprob": te,
             "entropy": d_log_s + 2 * ds * mean_abs + 2.0 ** -22 * (mean_sq + mean_abs + entropy.abs()),
             "stats": torch.stack([torch.zeros_like(ds), d_log_s], 1)}
    return got, bound


def backward(x, tokens, scale, d_logprob=None, d_entropy=None, d_top=None, top_token=None):
    """(gradient by autograd of the definition in 64 bits, bound before the last rounding).

    p's exponent is off by 2^-22 (|d| + log S + 2) and by log S's own error (see forward): `rel`
    of p together; the factor g + h (log p + H) by 2^-22 of its terms' magnitudes and by H's error."""
    y = x.double()
    # (-inf as a far number: its weight is 0, and the derivative by it still the formula's)
    y = torch.where(y.isinf(), torch.full_like(y, -1e5 / scale), y).requires_grad_()
    live = (tokens >= 0) & (tokens < y.shape[1]) & (x.double().amax(1) != -torch.inf)
    at = tokens.long().clamp(0, y.shape[1] - 1)[:, None]
    log_p = torch.log_softmax(scale * y, 1)
    p = log_p.exp()
    loss = torch.zeros((y.shape[0],), dtype=torch.float64)
    g = torch.zeros_like(loss)
    if d_logprob is not None:
        loss = loss + d_logprob.double() * log_p.gather(1, at)[:, 0]
        g = g + d_logprob.double().abs()
    H = -(p * torch.where(p > 0, log_p, torch.zeros_like(p))).sum(1)
    h = torch.zeros_like(loss) if d_entropy is None else d_entropy.double()
    loss = loss + h * H
    if d_top is not None:
        loss = loss + (d_top.double() * log_p.gather(1, top_token.long().clamp(min=0))).sum(1)
        g = g + d_top.double().abs().sum(1)
    (dx,) = torch.autograd.grad(torch.where(live, loss, torch.zeros_like(loss)).sum(), y)
    got, bound = forward(x, tokens, scale)
    lp = torch.where(p > 0, log_p, torch.zeros_like(p)).abs().detach()
    d_log_s = bound["stats"][:, 1:]
    rel = 2.0 ** -21 + 2.0 ** -22 * (lp + 2 * got["stats"][:, 1:].abs() + 2) + 2 * d_log_s
    size = g[:, None] + h.abs()[:, None] * (lp + H.detach()[:, None])
    err = p.detach() * (size * (rel + 2.0 ** -21) + h.abs()[:, None] * (bound["entropy"][:, None] + d_log_s))
    return dx, scale * (err + 2.0 ** -22 * dx.abs() / scale) + 2.0 ** -140
