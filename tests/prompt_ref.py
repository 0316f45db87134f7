"""Attention of whole prompts and its gradients in 64 bits on the CPU: the
reference of the tests, with the error bounds the kernels are held to.

A batch is given as flat rows: q [T, Hq, D], k, v [T, Hkv, D] and the rows'
ranges (offsets cu of B + 1 entries); rows outside them belong to nothing.
"""
import math

import torch

U = 2.0 ** -24                              # half an fp32 step, relative
SLACK = 1 + 2.0 ** -6                       # terms of second order
# what an fp32 exponential, product or operand below the smallest normal number
# may lose: each is taken as zero by the hardware (2^-126, twice on the way)
TINY = 2.0 ** -125


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def band(L, window):
    """Which tokens (columns) each row attends to."""
    m = torch.ones((L, L), dtype=torch.bool).tril()
    return m.triu(1 - window) if window else m


def _heads(x, lo, hi):
    return x[lo:hi].double().transpose(0, 1)            # [heads, L, D]


def _logits(q, k, scale, window):
    """s of one head, -inf where a row does not attend; and how far an fp32
    logit may be off: sums of D products, their scaling by c = scale log2 e
    (rounded) and, in units of the exponent, the difference to a rounded
    maximum or log sum."""
    s = scale * (q @ k.t())
    D = q.shape[1]
    err = (D + 2) * U * abs(scale) * (q.abs() @ k.abs().t()) + 4 * U * s.abs()
    seen = band(q.shape[0], window) & (s > -math.inf)     # (a weight of zero is as none)
    return s.masked_fill(~seen, -math.inf), err.masked_fill(~seen, 0.0), seen


def forward(q, k, v, cu, scale, window=0):
    """o and lse of every row (NaN outside the sequences), and their bounds.

    With h the half step of the inputs' type: a weight relative to the row's
    maximum is off by e (its logit's error) + 4 u + 4 u (|s| + |m|), with e the
    largest of the row, so that a normalised weight is off by at most 2 of
    these and (N + 16) u for the sum of N; rounding it to an operand adds h,
    the product's sums (N + 16) u, all relative to sum w |v|; storing o adds
    h |o|.  lse adds the errors of the maximum and of the sum's logarithm.
    """
    h = half_step(q.dtype)
    G = q.shape[1] // k.shape[1]
    o = torch.full(q.shape, math.nan, dtype=torch.float64)
    lse = torch.full(q.shape[:2], math.nan, dtype=torch.float64)
    ob, lb = torch.zeros_like(o), torch.zeros_like(lse)
    for lo, hi in zip(cu[:-1], cu[1:]):
        L = hi - lo
        if L == 0:
            continue
        qs, ks, vs = (_heads(x, lo, hi) for x in (q, k, v))
        for hq in range(q.shape[1]):
            kk, vv = ks[hq // G], vs[hq // G]
            s, err, seen = _logits(qs[hq], kk, scale, window)
            n = seen.sum(1, keepdim=True)
            w = torch.softmax(s, 1).masked_fill(n == 0, 0.0)
            big = s.masked_fill(~seen, 0).abs().amax(1, keepdim=True)
            e = err.amax(1, keepdim=True) + 4 * U + 8 * U * big
            rel = 2 * e + (n + 16) * U
            o[lo:hi, hq] = w @ vv
            ob[lo:hi, hq] = ((rel + (h if h > U else 0) + (n + 16) * U) * (w @ vv.abs())
                             + h * o[lo:hi, hq].abs()
                             + TINY * (1 + seen.double() @ vv.abs())) * SLACK
            x = torch.logsumexp(s, 1)
            lse[lo:hi, hq] = x
            lb[lo:hi, hq] = (rel[:, 0] + 4 * U * (x.abs() + big[:, 0] + 1)) * SLACK
    return o, lse, ob, lb


def backward(q, k, v, o, lse, do, cu, scale, window=0):
    """dq, dk, dv for the o and lse given (those of the kernel), and bounds.

    w = e^{s - lse}: off by rel = e + 4 u + 4 u |lse| relative; do.v and
    do.o by (D + 2) u of their sums of magnitudes; ds = w (do.v - delta) by
    w times these and (rel + 4 u) of itself.  Operands are rounded (h), sums
    of N terms add (N + 16) u, results are rounded once.
    """
    h = half_step(q.dtype)
    hp = h if h > U else 0                  # fp32 operands are not rounded
    D, Hkv = q.shape[2], k.shape[1]
    G = q.shape[1] // Hkv
    grads = [torch.full(x.shape, math.nan, dtype=torch.float64) for x in (q, k, v)]
    bounds = [torch.zeros_like(x) for x in grads]
    a = abs(scale)
    for lo, hi in zip(cu[:-1], cu[1:]):
        L = hi - lo
        if L == 0:
            continue
        qs, ks, vs, os, gs = (_heads(x, lo, hi) for x in (q, k, v, o, do))
        ls = lse[lo:hi].double().t()
        for hk in range(Hkv):
            kk, vv = ks[hk], vs[hk]
            dk, dv, bk, bv = (torch.zeros_like(kk) for _ in range(4))
            for hq in range(hk * G, hk * G + G):
                s, err, seen = _logits(qs[hq], kk, scale, window)
                x = ls[hq][:, None]
                w = torch.where(seen & (x > -math.inf), torch.exp(s - x), torch.zeros(()).double())
                rel = torch.where(seen, err + 4 * U + 4 * U * x.abs().nan_to_num(posinf=0), 0.0)
                g = gs[hq]
                dp, dpe = g @ vv.t(), (D + 2) * U * (g.abs() @ vv.abs().t())
                de = (g * os[hq]).sum(1, keepdim=True)
                dee = (D + 2) * U * (g * os[hq]).abs().sum(1, keepdim=True)
                ds = w * (dp - de)
                dse = (w * (dpe + dee) + (rel + 4 * U) * ds.abs()
                       + torch.where(seen, TINY * (1 + (dp - de).abs()), 0.0))
                n = seen.sum(1, keepdim=True) + 16
                m = G * seen.sum(0)[:, None] + 16
                y = scale * (ds @ kk)
                grads[0][lo:hi, hq] = y
                bounds[0][lo:hi, hq] = SLACK * (
                    a * ((dse + (hp + n * U) * ds.abs()) @ kk.abs()) + (h + 2 * U) * y.abs() + TINY)
                dk += scale * (ds.t() @ qs[hq])
                bk += a * ((dse + hp * ds.abs()).t() @ qs[hq].abs()
                           + m * U * (ds.abs().t() @ qs[hq].abs()))
                dv += w.t() @ g
                bv += (w * (rel + hp) + TINY * seen).t() @ g.abs() + m * U * (w.t() @ g.abs())
            grads[1][lo:hi, hk], grads[2][lo:hi, hk] = dk, dv
            bounds[1][lo:hi, hk] = SLACK * (bk + (h + 2 * U) * dk.abs() + TINY)
            bounds[2][lo:hi, hk] = SLACK * (bv + (h + 2 * U) * dv.abs() + TINY)
    return grads, bounds
