"""The paged cache calls again in 64 bits, one sequence and head at a time, and
the error bounds of the kernels' arithmetic.

Bounds.  Half a step of a type, relative to the value, is finfo.eps / 2:
bf16 2^-8, fp16 2^-11, fp32 2^-24.  With A = sum_j p_j |v_j| / l:
  O    the P of the value product is rounded once (bf16, or fp16 over an 8-bit
       cache; l sums the unrounded P), the result once to bf16:
       half_P A + 2^-8 |O|.  fp16 P below 2^-14 of the row's largest is off by at
       most 2^-25 of it: 2^-25 sum_j |v_j| / l, with l >= 1 in those units.  The
       fp32 sums add at most (n + d) 2^-23 of the magnitudes they add (2^-23 and not
       2^-24: the tensor cores may truncate), and the exponent's argument is off
       by E (below), which moves every p by at most the factor e^E.
  LSE  E = (d + 4) 2^-23 scale max_j sum_i |q_i k_ji|: the score's sum and the two
       roundings of its scaling; the exponential (2^-22 relative) and the sum
       ((n / 32 + 64) 2^-23: a lane adds one key in 32, then lanes, warps and parts
       are joined) add to log l; 2^-22 |LSE| covers the final conversions.
  A row's weight P = exp(s - LSE) is off by the factor exp(E + the LSE's error)."""
import math

import torch

F64 = torch.float64


def flat(pool, table_row, n, scale=None):
    """Rows 0 .. n of a sequence: [Hkv, n, d] in 64 bits."""
    pages, Hkv, page, d = pool.shape
    out = torch.empty(Hkv, n, d, dtype=F64)
    for p in range(n):
        out[:, p] = pool[int(table_row[p // page]), :, p % page].to(F64)
    return out if scale is None else out * scale.to(F64)[:, None, None]


def decode(Q, kc, vc, table, lens, scale, ks=None, vs=None):
    """Per sequence: O, LSE, weights and the bounds of their errors (CPU inputs)."""
    B, Hq, d = Q.shape
    Hkv = kc.shape[1]
    G = Hq // Hkv
    half = 2.0 ** -11 if ks is not None else 2.0 ** -8
    res = []
    for b in range(B):
        n = int(lens[b])
        r = dict(O=torch.zeros(Hq, d, dtype=F64), LSE=torch.full((Hq,), -math.inf, dtype=F64),
                 W=torch.zeros(Hkv, n, dtype=F64))
        r["O_tol"], r["LSE_tol"], r["W_tol"] = (torch.zeros_like(r[k]) for k in ("O", "LSE", "W"))
        if n:
            k, v = flat(kc, table[b], n, ks), flat(vc, table[b], n, vs)
            for h in range(Hq):
                q = Q[b, h].to(F64)
                s = (k[h // G] @ q) * scale
                lse = torch.logsumexp(s, 0)
                p = torch.exp(s - lse)
                E = (d + 4) * 2.0 ** -23 * scale * float((k[h // G].abs() @ q.abs()).max())
                e_lse = E + 2.0 ** -22 + (n / 32 + 64) * 2.0 ** -23 + 2.0 ** -22 * abs(float(lse))
                o, A = p @ v[h // G], p @ v[h // G].abs()
                r["O"][h], r["LSE"][h] = o, lse
                r["LSE_tol"][h] = e_lse
                # (half a step more than the bound's first order: products of two errors)
                r["O_tol"][h] = 1.01 * ((half + 2 * E + 2.0 ** -21 + (n + d) * 2.0 ** -23) * A + 2.0 ** -8 * o.abs())
                if ks is not None:
                    r["O_tol"][h] += 2.0 ** -25 * v[h // G].abs().sum(0) * math.exp(float(s.max() - lse))
                r["W"][h // G] += p
                r["W_tol"][h // G] += p * (1.01 * (E + e_lse + 2.0 ** -21)) + 2.0 ** -120
        res.append(r)
    return res


def evict(w, n, budget, recent):
    """Positions that one head keeps (w: its weights, a list of floats)."""
    if n <= budget:
        return list(range(n))
    old = n - recent
    order = sorted(range(old), key=lambda i: (-w[i] if w[i] == w[i] else math.inf, w[i] != w[i], i))
    return sorted(order[:budget - recent]) + list(range(old, n))


def make_cache(lens, Hkv, d, page, e4m3=False, seed=0, extra_pages=3, layout="heads", poison=True):
    """Pools, a shuffled page table and scales on the CPU.  Slots that no
    sequence holds are NaN (``poison``), as are the pages nobody owns."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // page) for n in lens]
    pages = sum(need) + extra_pages
    ids = torch.randperm(pages, generator=g).to(torch.int32)
    W = max(1, max(need))
    table = torch.full((len(lens), W), -1, dtype=torch.int32)
    at = 0
    for b, k in enumerate(need):
        table[b, :k] = ids[at:at + k]
        at += k
    shape = (pages, Hkv, page, d)
    live = torch.zeros(pages, page, dtype=torch.bool)
    for b, n in enumerate(lens):
        for p in range(n):
            live[int(table[b, p // page]), p % page] = True
    pools = []
    ks = vs = None
    if e4m3:
        ks, vs = torch.rand(Hkv, generator=g) * 0.02 + 0.005, torch.rand(Hkv, generator=g) * 0.02 + 0.005
    for s in (ks, vs):
        x = torch.randn(shape, generator=g)
        if s is not None:
            x = (x / s[:, None, None]).clamp(-448, 448)
        if poison:
            x = torch.where(live[:, None, :, None], x, torch.nan)
        x = x.to(torch.float8_e4m3fn if e4m3 else torch.bfloat16)
        if layout == "rows":  # [pages, page_size, Hkv, d] in memory
            x = x.transpose(1, 2).contiguous().transpose(1, 2)
        pools.append(x)
    return dict(kc=pools[0], vc=pools[1], table=table, lens=torch.tensor(lens, dtype=torch.int32), ks=ks, vs=vs,
                free=[int(i) for i in ids[at:]])


def dev(c):
    return {k: (v.cuda() if isinstance(v, torch.Tensor) else v) for k, v in c.items()}
