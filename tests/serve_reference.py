"""Plain attention in 64 bits for the packed and paged tests, with the error
that a correct kernel may have.

Derivation of the tolerance, per output element, for 16-bit inputs and output
of half step u (bf16 2^-8, fp16 2^-11):
  - every weight p is rounded once to 16 bits: at most u times A = sum p |v| / sum p;
  - the output is rounded once: u |o| (plus the smallest fp16 step's half);
  - a score is a sum of 128 fp32 products: at most 128 2^-24 R with R = max_j c
    sum_c |q_c k_jc| in log2 units, twice (score and running maximum); 2^x has a
    relative error below 2^-20: the weight is off by e = ln 2 (2 x 132 x 2^-24
    R) + 2^-20, the quotient by 2 e A;
  - sums over n keys in fp32: (n + 64) 2^-24 A, for numerator and denominator;
  - fp16 weights below 2^-31 of the largest vanish: n 2^-31 max |v|.
The logarithm of the sum: e + (n + 64) 2^-24 + 2^-21 |lse|.
"""
import math

import torch

D = 128
HALF = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


def attend(q, k, v, limit, scale=None):
    """One key head: q [rows, D], k, v [keys, D], row i sees the first limit[i]
    keys.  Returns o, lse and their tolerances, in float64."""
    u, n = HALF[q.dtype], k.shape[0]
    c = 1 / math.sqrt(D) if scale is None else scale
    q, k, v = q.double(), k.double(), v.double()
    hidden = torch.arange(n, device=q.device) >= limit[:, None]
    seen_k = torch.nan_to_num(k, nan=0.0, posinf=0.0, neginf=0.0)
    x = (q @ seen_k.T * c).masked_fill(hidden, -math.inf)
    if n == 0:
        x = x.reshape(q.shape[0], 0)
    top = x.amax(-1, keepdim=True) if n else torch.full((q.shape[0], 1), -math.inf, device=q.device, dtype=q.dtype)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = torch.exp(x - top)
    total = p.sum(-1, keepdim=True)
    some = total > 0
    safe = torch.where(some, total, torch.ones_like(total))
    fin = torch.isfinite(v)
    vf = torch.where(fin, v, torch.zeros_like(v))
    o = p @ vf / safe
    a = p @ vf.abs() / safe
    # elements that are not finite reach exactly the rows that see them
    seen = (~hidden).double()
    for kind, val in ((torch.isnan(v), math.nan), (v == math.inf, math.inf), (v == -math.inf, -math.inf)):
        if bool(kind.any()):
            hit = (seen @ kind.double()) > 0
            o = torch.where(hit, o + val, o)
    lse = torch.where(some, top + safe.log(), torch.full_like(top, -math.inf)).squeeze(-1)
    r = (q.abs() @ seen_k.abs().T * c).masked_fill(hidden, 0.0).amax(-1, keepdim=True) * math.log2(math.e) if n else top * 0
    e = math.log(2) * 2 * 132 * 2.0 ** -24 * r + 2.0 ** -20
    vmax = vf.abs().max() if n else 0.0
    tol = u * (a + torch.nan_to_num(o, nan=0.0, posinf=0.0, neginf=0.0).abs()) + (2 * e + 2 * (n + 64) * 2.0 ** -24) * a \
        + n * 2.0 ** -31 * vmax + 2.0 ** -25
    tol_lse = e.squeeze(-1) + (n + 64) * 2.0 ** -24 + 2.0 ** -21 * torch.nan_to_num(lse, neginf=0.0).abs()
    return o, lse, tol, tol_lse


def check(got, want, tol, what):
    got = got.double()
    odd = ~torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{what}: NaN in other places"
    assert torch.equal(got[odd & ~torch.isnan(want)], want[odd & ~torch.isnan(want)]), f"{what}: infinities differ"
    off = (got - want).abs()[~odd] / tol.expand_as(want)[~odd]
    worst = float(off.max()) if off.numel() else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3f} of the tolerance"
    return worst


def packed(q, k, v, cu_q, cu_k, causal, scale=None):
    """o, lse and tolerances [total_q, Hq, ...] over packed sequences (cu lists on the host)."""
    Hq, G = q.shape[1], q.shape[1] // k.shape[1]
    o = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(o)
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device=q.device)
    tl = torch.zeros_like(lse)
    for i in range(len(cu_q) - 1):
        lq, lk = cu_q[i + 1] - cu_q[i], cu_k[i + 1] - cu_k[i]
        if lq == 0:
            continue
        rows = torch.arange(lq, device=q.device)
        limit = (rows + 1 + lk - lq).clamp(0, lk) if causal else torch.full_like(rows, lk)
        s = slice(cu_q[i], cu_q[i + 1])
        for h in range(Hq):
            o[s, h], lse[s, h], tol[s, h], tl[s, h] = attend(
                q[s, h], k[cu_k[i]:cu_k[i + 1], h // G], v[cu_k[i]:cu_k[i + 1], h // G], limit, scale)
    return o, lse, tol, tl


def paged(pool, layer, rows, lens, q, seqs, cu_q, scale=None):
    """The same over a cache: rows[r] the page list of table row r, lens[r] its tokens."""
    Hkv, page = pool.shape[3], pool.shape[4]
    ks, vs, ck = [], [], [0]
    for s in seqs:
        n = lens[s] if s >= 0 else 0
        pages = torch.tensor(rows[s][:-(-n // page)] if n else [], dtype=torch.long, device=q.device)
        for out, x in ((ks, pool[0, layer]), (vs, pool[1, layer])):
            out.append(x[pages].transpose(1, 2).reshape(-1, Hkv, D)[:n])
        ck.append(ck[-1] + n)
    return packed(q, torch.cat(ks), torch.cat(vs), cu_q, ck, True, scale)
