"""The top-k distillation loss in 64 bits for every listed mass, with bounds for float32.

Plain torch in double precision on the CPU, from the formulas in include/ob.h: the gradient is
the loss's derivative also where the listed mass S = sum p exceeds 1 (p_rest is 0 there, and the
student's q counts S times), and where the student has no mass that float32 shows outside the list a p_rest
within a sum's rounding is 0.

Logits are taken relative to their row's largest, dz <= 0, which leaves q and the loss as they
are. EPS is float32's unit roundoff. An exponent dz is formed with at most 4 roundings of its own
size; a log-sum-exp has those of its terms, weighted with their shares, and C = 32 EPS for the
exponentials, the sum and the logarithm. p = exp(t - lse) has the roundings of t and lse, at most
4 EPS of either, and C. Products and sums of these take C of the terms' sizes.
"""
import math

import torch

from student_ref import C, EPS, HALF_ULP, TINY

INF = float("inf")


def rest_slack(top_lse, K):
    """The largest p_rest that is taken as rounding where the student has no mass outside the list."""
    return EPS * (4 * abs(top_lse) + K / 32 + 16)


def _rounded(bound, value, dtype):
    return bound + HALF_ULP.get(dtype, 0.0) * (value.abs() + bound) + TINY.get(dtype, 0.0)


def distill(logits, index, top, top_lse=None, temperature=1.0, weight=None, dloss=None):
    """{name: (value, bound)} of loss and dlogits (of sum(dloss*loss)), logits [N, V]."""
    z = logits.detach().double().cpu()
    N, V = z.shape
    K = index.shape[1]
    index = index.cpu().long()
    here = (index >= 0) & (index < V)
    t = torch.where(here, top.detach().double().cpu(), torch.full(index.shape, -INF, dtype=torch.float64))
    w = torch.ones(N, dtype=torch.float64) if weight is None else weight.double().cpu()
    up = torch.ones(N, dtype=torch.float64) if dloss is None else dloss.detach().double().cpu()
    loss, eloss = torch.zeros(N, dtype=torch.float64), torch.zeros(N, dtype=torch.float64)
    d, ed = torch.zeros_like(z), torch.zeros_like(z)
    for n in range(N):
        live = t[n] > -INF
        if w[n] == 0 or (top_lse is None and not bool(live.any())):
            continue
        dz = (z[n] - z[n].max()) / temperature
        ez = torch.nan_to_num(4 * EPS * dz.abs(), posinf=0.0)
        lse = torch.logsumexp(dz, 0)
        lq = dz - lse
        q = torch.exp(lq)
        es = (q * ez).sum() + C
        elq = ez + es + 4 * EPS * lse.abs()
        if top_lse is None:
            tn = (t[n] - t[n].max()) / temperature
            tl = torch.logsumexp(tn, 0)
        else:
            tn, tl = t[n] / temperature, top_lse[n].double().cpu()
        lp = tn - tl
        p = torch.exp(lp)
        ep = p * (torch.nan_to_num(4 * EPS * tn.abs(), posinf=0.0) + 4 * EPS * tl.abs() + C)
        k = index[n].clamp(0, V - 1)
        has = p > 0
        loss[n] = (p[has] * (lp[has] - lq[k[has]])).sum()
        sizes = p[has] * (lp[has].abs() + lq[k[has]].abs())
        # p's own error counts with its factor, log p's and log q's with p
        eloss[n] = ((ep[has] * (1 + lp[has].abs() + lq[k[has]].abs())) + p[has] * elq[k[has]] + C * sizes).sum()
        total = torch.zeros(V, dtype=torch.float64)
        etotal = torch.zeros(V, dtype=torch.float64)
        total.index_add_(0, index[n][here[n]], p[here[n]])
        etotal.index_add_(0, index[n][here[n]], ep[here[n]])
        listed = torch.zeros(V, dtype=torch.bool)
        listed[index[n][here[n]]] = True
        outside = torch.where(listed, torch.full_like(dz, -INF), dz)
        lrest = torch.logsumexp(outside, 0)
        mass, emass = p.sum(), ep.sum() + C * p.sum() + 4 * EPS
        rest = torch.zeros((), dtype=torch.float64)
        if top_lse is not None:
            rest = torch.clamp(1 - mass, min=0)
            if float(outside.max()) < -126 * math.log(2) and rest <= rest_slack(float(tl), K):
                rest = torch.zeros_like(rest)
            lqr = lrest - lse
            if rest > 0:
                loss[n] += rest * (torch.log(rest) - lqr)
            if lqr > -INF:
                # p_rest log p_rest near 0 moves by the mass's error times its logarithm
                size = 1 + torch.log(torch.maximum(rest, emass)).abs() + lqr.abs()
                esr = (torch.exp(outside - lrest) * ez).sum() + C
                eloss[n] += emass * size + rest * (esr + es + C * size)
        soft = torch.exp(outside - lrest) if lrest > -INF else torch.zeros_like(q)
        factor = mass + rest if top_lse is not None else torch.ones_like(mass)
        esoft = torch.exp(outside - lrest) * (ez + (soft * ez).sum() + C) if lrest > -INF else soft
        d[n] = factor * q - torch.where(listed, total, rest * soft)
        ed[n] = (factor * q * (elq + C) + q * emass * float(top_lse is not None)
                 + torch.where(listed, etotal + EPS * total, rest * esoft + emass * soft * float(top_lse is not None)))
    f = (w * up / temperature)[:, None]
    el = w.abs() * eloss + EPS * (w * loss).abs()
    return {"loss": (w * loss, el),
            "dlogits": (d * f, _rounded(ed * f.abs() + 4 * EPS * (d * f).abs(), d * f, logits.dtype))}
