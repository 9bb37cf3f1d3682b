"""Packed attention again in 64 bits, one sequence and head at a time, and the
error bounds of the kernels' arithmetic.

Bounds.  Half a step of a type, relative to the value, is finfo.eps / 2:
bf16 2^-8, fp32 2^-24; fp32 sums count 2^-23 a term (the tensor cores may
truncate).  With s the scaled scores, E = (d + 4) 2^-23 scale max_j sum_i |q_i k_ji|
(the score's sum and the roundings of its scaling) and n the row's keys:
  O    every P is rounded once to bf16, the result once more:
       (2^-8 + 2 E + 2^-21 + (n + d) 2^-23) sum_j P_j |v_j| + 2^-8 |O|.
  LSE  E + 2^-22 (exponential) + (n + 64) 2^-23 (sum) + 2^-21 |LSE| (logarithm,
       conversion).
The gradients are taken, as the kernels do, from the O and LSE that they are
given:  P = exp(s - LSE),  D = dO . O,  dS = P (dP - D).
  P    off by r_P = E + 2^-21 + 2^-22 |LSE| (exponent), and 2^-8 in the bf16 form
       that both products read.
  dV   (2^-8 + r_P + n_q 2^-23) sum_i P |dO| + 2^-8 |dV|, n_q the queries summed.
  dS   P's error, and its own rounding to bf16: e_S = (2 2^-8 + 2^-16 + r_P) |dS|
       + (d + 4) 2^-23 P (sum |dO| |v| + sum |dO| |O|) from the sums dP and D.
  dK   scale (sum_i e_S |q| + n_q 2^-23 sum_i |dS| |q|) + 2^-8 |dK|, dQ likewise.
(1.02: products of two errors.)"""
import math

import torch

F64 = torch.float64


def visible(Lq, Lk, causal):
    see = torch.ones(Lq, Lk, dtype=torch.bool)
    return see.tril(Lk - Lq) if causal else see


def fwd(Q, K, V, cu_q, cu_k, causal, scale):
    """O, LSE and their bounds (CPU inputs, cu as lists)."""
    Tq, Hq, d = Q.shape
    G = Hq // K.shape[1]
    O, Ot = torch.zeros(Tq, Hq, d, dtype=F64), torch.zeros(Tq, Hq, d, dtype=F64)
    L, Lt = torch.full((Hq, Tq), -math.inf, dtype=F64), torch.zeros(Hq, Tq, dtype=F64)
    for b in range(len(cu_q) - 1):
        q0, q1, k0, k1 = cu_q[b], cu_q[b + 1], cu_k[b], cu_k[b + 1]
        if q1 == q0 or k1 == k0:
            continue
        see = visible(q1 - q0, k1 - k0, causal)
        some, n = see.any(1), see.sum(1)
        for h in range(Hq):
            q, k, v = Q[q0:q1, h].to(F64), K[k0:k1, h // G].to(F64), V[k0:k1, h // G].to(F64)
            s = (q @ k.T * scale).masked_fill(~see, -math.inf)
            E = (d + 4) * 2.0 ** -23 * scale * (q.abs() @ k.abs().T).masked_fill(~see, 0).amax(1)
            lse = torch.where(some, torch.logsumexp(s, 1), torch.tensor(-math.inf, dtype=F64))
            p = torch.exp(s - lse.masked_fill(~some, 0.0)[:, None]).masked_fill(~see, 0.0)
            o = p @ v
            O[q0:q1, h], L[h, q0:q1] = o, lse
            Ot[q0:q1, h] = 1.02 * ((2.0 ** -8 + 2 * E + 2.0 ** -21 + (n + d) * 2.0 ** -23)[:, None] * (p @ v.abs())
                                   + 2.0 ** -8 * o.abs())
            Lt[h, q0:q1] = E + 2.0 ** -22 + (n + 64) * 2.0 ** -23 + 2.0 ** -21 * lse.masked_fill(~some, 0.0).abs()
    return O, L, Ot, Lt


def bwd(Q, K, V, O, dO, LSE, cu_q, cu_k, causal, scale):
    """[(dQ, bound), (dK, bound), (dV, bound)] from the given O and LSE."""
    Tq, Hq, d = Q.shape
    G = Hq // K.shape[1]
    out = [[torch.zeros(t.shape, dtype=F64), torch.zeros(t.shape, dtype=F64)] for t in (Q, K, V)]
    u = 2.0 ** -23
    for b in range(len(cu_q) - 1):
        q0, q1, k0, k1 = cu_q[b], cu_q[b + 1], cu_k[b], cu_k[b + 1]
        if q1 == q0 or k1 == k0:
            continue
        see = visible(q1 - q0, k1 - k0, causal)
        nq = (q1 - q0) * G
        for h in range(Hq):
            q, k, v = Q[q0:q1, h].to(F64), K[k0:k1, h // G].to(F64), V[k0:k1, h // G].to(F64)
            o, do, lse = O[q0:q1, h].to(F64), dO[q0:q1, h].to(F64), LSE[h, q0:q1].to(F64)
            none = torch.isneginf(lse)
            lse = lse.masked_fill(none, 0.0)
            hide = ~see | none[:, None]
            p = torch.exp((q @ k.T * scale - lse[:, None]).masked_fill(hide, -math.inf))
            E = (d + 4) * u * scale * (q.abs() @ k.abs().T).masked_fill(hide, 0).amax(1)
            rP = (E + 2.0 ** -21 + 2.0 ** -22 * lse.abs())[:, None]
            dp, D = do @ v.T, (do * o).sum(1, keepdim=True)
            ds = p * (dp - D)
            eS = (2 * 2.0 ** -8 + 2.0 ** -16 + rP) * ds.abs() + (d + 4) * u * p * (do.abs() @ v.abs().T + (do * o).abs().sum(1, keepdim=True))
            out[0][0][q0:q1, h] = scale * (ds @ k)
            out[0][1][q0:q1, h] = 1.02 * scale * ((eS + (k1 - k0) * u * ds.abs()) @ k.abs())
            out[1][0][k0:k1, h // G] += scale * (ds.T @ q)
            out[1][1][k0:k1, h // G] += 1.02 * scale * ((eS + nq * u * ds.abs()).T @ q.abs())
            out[2][0][k0:k1, h // G] += p.T @ do
            out[2][1][k0:k1, h // G] += 1.02 * (((2.0 ** -8 + rP + nq * u) * p).T @ do.abs())
    return [(x, t + 2.0 ** -8 * x.abs()) for x, t in out]
