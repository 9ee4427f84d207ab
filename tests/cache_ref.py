"""Plain 64-bit forms of the cache operators, and the bounds their results are held to.

The bounds count roundings.  eps(t) / 2 is half a step of type t relative to
the value.  A logit y = scale q.k is a sum of d exact products in fp32, so it
is off by at most Y = (d + 8) 2^-23 scale sum|q||k| (the tensor cores may
truncate: a whole step an addition), plus the roundings of its scaled value.
A weight exp(y - lse) is off by a factor of at most 1 + R,

    R = 2 Y + 2^-22 (|y| + |lse|) + 2^-20

(2^-20: ex2 and lg2, each a few units in the last place).
"""
import math

import torch

F64 = torch.float64
EX2_FLOOR = 1e-36          # results of ex2 below 2^-126 are flushed to zero


def visible(N_Q, N_K, causal, n):
    see = torch.arange(N_K)[None, :].expand(N_Q, N_K) < n
    if causal:
        see = see & (torch.arange(N_K)[None, :] <= torch.arange(N_Q)[:, None] + (N_K - N_Q))
    return see


def key_mass(q, k, scale, causal, kv_len=None, lse=None):
    """(mass, lse, bound of mass, bound of lse), 64-bit, of CPU tensors."""
    B, H, N_Q, d = q.shape
    Hk, N_K = k.shape[1:3]
    G = H // Hk
    mass, bound = torch.zeros(B, Hk, N_K, dtype=F64), torch.full((B, Hk, N_K), G * N_Q * EX2_FLOOR, dtype=F64)
    out, out_bound = torch.full((B, H, N_Q), -math.inf, dtype=F64), torch.zeros(B, H, N_Q, dtype=F64)
    for b in range(B):
        n = N_K if kv_len is None else int(kv_len[b])
        see = visible(N_Q, N_K, causal, n)
        for h in range(H):
            qd, kd = q[b, h].to(F64), k[b, h // G].to(F64)
            kd = torch.where((torch.arange(N_K) < n)[:, None], kd, torch.zeros_like(kd))
            y = torch.where(see, qd @ kd.T * scale, torch.tensor(-math.inf, dtype=F64))
            Y = (d + 8) * 2.0 ** -23 * scale * (qd.abs() @ kd.abs().T)
            l = torch.logsumexp(y, 1) if N_K else torch.full((N_Q,), -math.inf, dtype=F64)
            out[b, h] = l
            size = torch.where(see, y.abs(), torch.zeros_like(y))
            out_bound[b, h] = Y.amax(1) + 2.0 ** -22 * (size.amax(1) + l.abs().nan_to_num(posinf=0.0)) + 2.0 ** -20
            used = l if lse is None else lse[b, h].to(F64)
            ok = torch.isfinite(used)
            w = torch.where(see & ok[:, None], torch.exp(y - torch.where(ok, used, torch.zeros_like(used))[:, None]),
                            torch.zeros_like(y))
            R = Y + Y.amax(1, keepdim=True) + 2.0 ** -22 * (size + torch.where(ok, used, torch.zeros_like(used))
                                                            .abs()[:, None]) + 2.0 ** -20
            R = R + 2.0 ** -24 * (40 + G * N_Q / 64)            # the sum's own roundings
            mass[b, h // G] += w.sum(0)
            bound[b, h // G] += (w * R).sum(0)
    return mass, out, bound, out_bound


def tokens(pages, table_row, n, hk):
    """[n, d]: the tokens of one sequence and key head."""
    page = pages.shape[2]
    t = torch.arange(n)
    return pages[table_row.long()[t // page], hk, t % page]


def decode(q, k_pages, v_pages, table, lens, scale, mass=None):
    """(out, lse, mass, bounds of the three), 64-bit, of CPU tensors; tokens of pages that do not exist are skipped."""
    B, H, d = q.shape
    pages, Hk, page, _ = k_pages.shape
    G = H // Hk
    step = torch.finfo(q.dtype).eps / 2
    out, ob = torch.zeros(B, H, d, dtype=F64), torch.full((B, H, d), 1e-30, dtype=F64)
    lse, lb = torch.full((B, H), -math.inf, dtype=F64), torch.zeros(B, H, dtype=F64)
    new, mb = (None, None) if mass is None else (mass.to(F64).clone(), torch.zeros(mass.shape, dtype=F64))
    for b in range(B):
        n = int(lens[b])
        t = torch.arange(n)
        pg = table[b].long()[t // page]
        ok = (pg >= 0) & (pg < pages)
        if not ok.any():
            continue
        t, pg = t[ok], pg[ok]
        for h in range(H):
            kd, vd = k_pages[pg, h // G, t % page].to(F64), v_pages[pg, h // G, t % page].to(F64)
            qd = q[b, h].to(F64)
            y = kd @ qd * scale
            Y = (d + 8) * 2.0 ** -23 * scale * (kd.abs() @ qd.abs())
            l = torch.logsumexp(y, 0)
            w = torch.exp(y - l)
            R = Y + Y.max() + 2.0 ** -22 * (y.abs() + l.abs()) + 2.0 ** -20
            o = w @ vd
            out[b, h], lse[b, h] = o, l
            # weights rounded to 16 bits (fp16: 2^-24 of the scale below its normal range), sums of n terms, the output
            tiny = 2.0 ** -40 if q.dtype == torch.float16 else 0.0
            ob[b, h] += ((w * (R + step + 2.0 ** -23 * (n / 16 + 16))) @ vd.abs() + o.abs() * (R.max() + step)
                         + tiny * w.max() * vd.abs().sum(0))
            lb[b, h] = Y.max() + 2.0 ** -22 * (y.abs().max() + l.abs()) + 2.0 ** -20 + 2.0 ** -24 * (n / 16 + 16)
            if mass is not None:
                new[b, h // G, t] += w
                mb[b, h // G, t] += w * (R + 2.0 ** -24 * (n / 16 + 16)) + EX2_FLOOR
    if mass is not None:
        mb += 2.0 ** -24 * (G + 1) * new.abs()
        mb[new == mass.to(F64)] = 0.0                             # untouched slots keep their bits
    out_b = ob + torch.finfo(q.dtype).tiny * torch.finfo(q.dtype).eps
    return out, lse, new, out_b, lb, mb


def evict_slots(mass, pos, n, budget, recent, next_pos):
    """Source slot of every slot below the new length of one (sequence, key head)."""
    keep = min(n, budget)

    def rank(t):
        m = float(mass[t])
        new = recent > 0 and int(pos[t]) >= next_pos - recent
        return (0 if new else 1, 0.0 if new else -(m if m > 0 else 0.0), t)      # the newest rank alike

    kept = sorted(range(n), key=rank)[:keep]
    have = set(kept)
    movers = iter(sorted(t for t in kept if t >= keep))
    return [t if t in have else next(movers) for t in range(keep)]


def evict(k_pages, v_pages, table, lens, mass, budget, recent=0, pos=None, next_pos=None, skip=()):
    """(new_len, mass, pos, k_pages, v_pages) of CPU tensors; the sequences in `skip` stay as they are."""
    page = k_pages.shape[2]
    B, Hk, cap = mass.shape
    new_len = torch.empty(B, dtype=torch.int32)
    m2, p2 = torch.zeros_like(mass), None if pos is None else torch.full_like(pos, -1)
    k2, v2 = k_pages.clone(), v_pages.clone()
    for b in range(B):
        n = int(lens[b])
        new_len[b] = n if b in skip else min(n, budget)
        for h in range(Hk):
            src = (list(range(n)) if b in skip else
                   evict_slots(mass[b, h], None if pos is None else pos[b, h], n, budget, recent,
                               0 if next_pos is None else int(next_pos[b])))
            for t, s in enumerate(src):
                m2[b, h, t] = mass[b, h, s]
                if pos is not None:
                    p2[b, h, t] = pos[b, h, s]
                if t != s:
                    a, c = int(table[b, t // page]), int(table[b, s // page])
                    k2[a, h, t % page] = k_pages[c, h, s % page]
                    v2[a, h, t % page] = v_pages[c, h, s % page]
    return new_len, m2, p2, k2, v2
