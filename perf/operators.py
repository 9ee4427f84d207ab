"""Cases and plain forms of the cache operators, for timing and comparison.

Three operators that belong to one path, serving with a bounded key-value
cache:

  key_mass  the attention weight that every key has received, summed over the
            query rows (the column sums of the softmax matrix), after a prompt
  decode    attention of one new token a sequence over a paged cache, which
            also adds the token's weights to the keys' accumulated ones
  evict     keeps, in every sequence and key head, the tokens with the largest
            accumulated weight and the newest ones, and closes the gaps

``run`` computes an operator in elementary torch operations in 32 bits, or,
with ``own`` set, calls the package.  ``exact`` computes the same from the
definition in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
LOG2_PAIRS = 31          # most query-key pairs (all heads) of a key_mass case


# --------------------------------------------------------------------- cases
def listed():
    return [
        # key_mass: a first small call, the latency of one tile
        dict(name="mass_tiny_128", op="key_mass", B=1, H=1, Hk=1, NQ=128, NK=128, d=64, causal=False, dtype="bf16",
             given=True, pad=False),
        # key_mass: a batch of ordinary prompts whose training forward left its log-sum-exps
        dict(name="mass_causal_2k_d64", op="key_mass", B=2, H=8, Hk=8, NQ=2048, NK=2048, d=64, causal=True,
             dtype="bf16", given=True, pad=False),
        # key_mass: a long prompt with grouped key heads
        dict(name="mass_causal_8k_gqa", op="key_mass", B=1, H=32, Hk=8, NQ=8192, NK=8192, d=128, causal=True,
             dtype="bf16", given=True, pad=False),
        # key_mass: only the prompt's last rows vote on a long, padded prompt; no log-sum-exps at hand
        dict(name="mass_window_64k", op="key_mass", B=4, H=8, Hk=2, NQ=61, NK=65536, d=128, causal=True,
             dtype="fp16", given=False, pad=True),
        # decode: one short sequence, the latency of a call
        dict(name="decode_one_short", op="decode", B=1, H=8, Hk=2, d=64, page=16, lo=77, hi=77, dtype="bf16",
             layout="HND", mass=False),
        # decode: a serving batch of very different lengths that feeds an eviction policy
        dict(name="decode_ragged_gqa", op="decode", B=24, H=32, Hk=8, d=128, page=64, lo=1, hi=8192, dtype="bf16",
             layout="HND", mass=True),
        # decode: as many key heads as query heads, token-major pages of an odd size
        dict(name="decode_mha_odd_pages", op="decode", B=7, H=16, Hk=16, d=64, page=24, lo=301, hi=2500, dtype="fp16",
             layout="NHD", mass=True),
        # decode: few sequences, long caches
        dict(name="decode_long_128k", op="decode", B=4, H=32, Hk=8, d=128, page=64, lo=131000, hi=131072,
             dtype="bf16", layout="HND", mass=False),
        # evict: one sequence a page over its budget
        dict(name="evict_one_page", op="evict", B=1, Hk=8, d=128, page=16, lo=1040, hi=1040, budget=1024, recent=32,
             dtype="bf16", layout="HND", fresh=False),
        # evict: a serving batch, each sequence up to a page over its budget
        dict(name="evict_serving_4k", op="evict", B=32, Hk=8, d=128, page=64, lo=4097, hi=4160, budget=4096,
             recent=128, dtype="bf16", layout="HND", fresh=False),
        # evict: prompts compressed to an eighth after the prefill
        dict(name="evict_prompt_32k", op="evict", B=4, Hk=8, d=128, page=64, lo=32700, hi=32768, budget=4096,
             recent=512, dtype="bf16", layout="HND", fresh=True),
        # evict: lengths below and above the budget, token-major pages of an odd size
        dict(name="evict_ragged_d64", op="evict", B=13, Hk=16, d=64, page=24, lo=1, hi=5000, budget=1001, recent=65,
             dtype="fp16", layout="NHD", fresh=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["key_mass", "decode", "evict"])
    d, dtype = rng.choice([64, 128]), rng.choice(["bf16", "fp16"])
    Hk = rng.choice([1, 2, 3, 4, 8])
    H = Hk * rng.choice([1, 2, 4, 5, 8])
    if op == "key_mass":
        B = _log(rng, 1, 8)
        NK = _log(rng, 1, 65536)
        most = max(1, min(NK, (1 << LOG2_PAIRS) // (B * H * NK), 16384))
        NQ = _log(rng, 1, most)
        return dict(op=op, B=B, H=H, Hk=Hk, NQ=NQ, NK=NK, d=d, causal=rng.random() < 0.7, dtype=dtype,
                    given=rng.random() < 0.5, pad=rng.random() < 0.4)
    B = _log(rng, 1, 48)
    page = rng.choice([1, 8, 16, 24, 32, 64, 100, 128, 256])
    hi = _log(rng, 1, max(1, min(131072, 4194304 // (B * Hk))))
    lo = _log(rng, 1, hi)
    layout = rng.choice(["HND", "NHD"])
    if op == "decode":
        return dict(op=op, B=B, H=H, Hk=Hk, d=d, page=page, lo=lo, hi=hi, dtype=dtype, layout=layout,
                    mass=rng.random() < 0.5)
    budget = _log(rng, 1, hi)
    return dict(op=op, B=B, Hk=Hk, d=d, page=page, lo=lo, hi=hi, budget=budget, recent=rng.randint(0, budget),
                dtype=dtype, layout=layout, fresh=rng.random() < 0.5)


def _lengths(c):
    """B lengths spread over [lo, hi] by their logarithm (the same for every seed, which only orders them)."""
    B, lo, hi = c["B"], c["lo"], c["hi"]
    if B == 1:
        return [hi]
    return [min(hi, max(lo, int(round(lo * (hi / lo) ** (i / (B - 1)))))) for i in range(B)]


def _key_lengths(c):
    """Key lengths of a padded batch: from all of N_K down to half of it."""
    B, NK = c["B"], c["NK"]
    return [max(1, NK - (NK * i) // (2 * B)) for i in range(B)]


# -------------------------------------------------------------------- inputs
def _dtype(c):
    return torch.bfloat16 if c["dtype"] == "bf16" else torch.float16


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    dt = _dtype(c)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=DEV, dtype=dt)

    s = {"case": c}
    if c["op"] == "key_mass":
        B, H, Hk, NQ, NK, d = c["B"], c["H"], c["Hk"], c["NQ"], c["NK"], c["d"]
        s["k"] = randn(B, Hk, NK, d)
        # queries lean towards one key each, so that some keys collect much more weight than others
        s["q"] = randn(B, H, NQ, d)
        liked = (torch.rand(B, Hk, NQ, generator=g, device=DEV).square() * NK).long().clamp_(max=NK - 1)
        lean = torch.gather(s["k"], 2, liked[..., None].expand(B, Hk, NQ, d)).repeat_interleave(H // Hk, dim=1)
        s["q"] = (s["q"] + 0.5 * lean).to(dt)
        s["kv_len"] = torch.tensor(_key_lengths(c), dtype=torch.int32, device=DEV) if c["pad"] else None
        s["scale"] = 1.0 / math.sqrt(d)
        s["lse"] = _lse_plain(s) if c["given"] else None
        return s
    B, Hk, d, page = c["B"], c["Hk"], c["d"], c["page"]
    lens = torch.tensor(_lengths(c), dtype=torch.int32, device=DEV)
    lens = lens[torch.randperm(B, generator=g, device=DEV)]
    per = -(-c["hi"] // page)
    pages = B * per + 3
    s["table"] = torch.randperm(pages, generator=g, device=DEV)[:B * per].view(B, per).to(torch.int32)
    s["len"] = lens
    shape = (pages, Hk, page, d) if c["layout"] == "HND" else (pages, page, Hk, d)
    s["k"], s["v"] = randn(*shape), randn(*shape)
    if c["layout"] == "NHD":
        s["k"], s["v"] = s["k"].transpose(1, 2), s["v"].transpose(1, 2)
    cap = per * page
    if c["op"] == "decode":
        s["q"] = 1.5 * randn(B, c["H"], d)
        s["scale"] = 1.0 / math.sqrt(d)
        s["mass"] = torch.rand(B, Hk, cap, generator=g, device=DEV) if c["mass"] else None
        s["mass_out"] = torch.empty_like(s["mass"]) if c["mass"] else None
        return s
    # accumulated weights have a long tail, and some tokens were never looked at
    mass = torch.randn(B, Hk, cap, generator=g, device=DEV).mul_(2.0).exp_()
    s["mass"] = torch.where(torch.rand(B, Hk, cap, generator=g, device=DEV) < 0.05, torch.zeros_like(mass), mass)
    slot = torch.arange(cap, device=DEV, dtype=torch.int32).expand(B, Hk, cap)
    if not c["fresh"]:
        # earlier evictions left the budget's slots in no order of age
        low = min(c["budget"], cap)
        order = torch.rand(B, Hk, low, generator=g, device=DEV).argsort(dim=-1).to(torch.int32)
        slot = torch.cat([order, slot[..., low:]], dim=-1)
    s["pos"] = slot.contiguous()
    s["next_pos"] = lens.clone()
    return s


# --------------------------------------------------------------- plain forms
def _visible(s):
    """[B, 1, NQ or 1, NK] truth values: which keys a row sees."""
    c = s["case"]
    NQ, NK = c["NQ"], c["NK"]
    j = torch.arange(NK, device=DEV)
    see = torch.ones(1, 1, 1, NK, dtype=torch.bool, device=DEV)
    if c["causal"]:
        i = torch.arange(NQ, device=DEV)
        see = (j[None, :] <= i[:, None] + (NK - NQ))[None, None]
    if s["kv_len"] is not None:
        see = see & (j[None, None, None, :] < s["kv_len"].view(-1, 1, 1, 1))
    return see


def _logits(s):
    c = s["case"]
    k = s["k"].float().repeat_interleave(c["H"] // c["Hk"], dim=1)
    x = torch.matmul(s["q"].float() * s["scale"], k.transpose(2, 3))
    return x.masked_fill_(~_visible(s), -math.inf)


def _lse_plain(s):
    x = _logits(s)
    m = x.amax(dim=-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    return (m + x.sub_(m).exp_().sum(dim=-1, keepdim=True).log()).squeeze(-1)


def _key_mass_plain(s):
    c = s["case"]
    x = _logits(s)
    lse = s["lse"]
    if lse is None:
        m = x.amax(dim=-1, keepdim=True)
        m = torch.where(m == -math.inf, torch.zeros_like(m), m)
        lse = (m + (x - m).exp_().sum(dim=-1, keepdim=True).log()).squeeze(-1)
    # a row without a visible key has the log-sum-exp -inf and weighs nothing
    p = x.sub_(torch.where(lse == -math.inf, torch.zeros_like(lse), lse)[..., None]).exp_()
    mass = p.sum(dim=2).view(c["B"], c["Hk"], c["H"] // c["Hk"], c["NK"]).sum(dim=2)
    return (mass,) if c["given"] else (mass, lse)


def _gather(pages, table):
    """[B, Hk, cap, d] in 32 bits: the tokens of every sequence in the order of its slots."""
    B, per = table.shape
    x = pages[table.long()]                                     # [B, per, Hk, page, d]
    return x.permute(0, 2, 1, 3, 4).reshape(B, x.shape[2], per * x.shape[3], x.shape[4]).float()


def _decode_plain(s):
    c = s["case"]
    B, H, Hk, d = c["B"], c["H"], c["Hk"], c["d"]
    k, v = _gather(s["k"], s["table"]), _gather(s["v"], s["table"])
    q = (s["q"].float() * s["scale"]).view(B, Hk, H // Hk, d)
    x = torch.matmul(q, k.transpose(2, 3))                      # [B, Hk, G, cap]
    see = torch.arange(x.shape[-1], device=DEV) < s["len"].view(B, 1, 1, 1)
    x = x.masked_fill_(~see, -math.inf)
    m = x.amax(dim=-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    e = (x - m).exp_()
    sums = e.sum(dim=-1, keepdim=True)
    lse = (m + sums.log()).reshape(B, H)
    p = e / torch.where(sums == 0, torch.ones_like(sums), sums)
    o = torch.matmul(p, v).reshape(B, H, d).to(s["q"].dtype)
    if s["mass"] is None:
        return o, lse
    return o, lse, s["mass"] + p.sum(dim=2)


def _evict_plain(s):
    """Tokens ranked by (recent, weight, lowest slot); the kept ones of the slots past the budget fill, in
    order, the slots of the evicted ones before it."""
    c = s["case"]
    mass, pos, lens = s["mass"], s["pos"], s["len"].view(-1, 1, 1)
    B, Hk, cap = mass.shape
    slot = torch.arange(cap, device=DEV).expand(B, Hk, cap)
    live = slot < lens
    new_len = torch.clamp(lens, max=c["budget"])
    weight = torch.where(mass > 0, mass, torch.zeros_like(mass)).double()
    recent = (pos >= s["next_pos"].view(-1, 1, 1) - c["recent"]) & live
    weight = torch.where(recent, math.inf, torch.where(live, weight, -1.0))
    order = torch.sort(weight, dim=-1, descending=True, stable=True).indices
    kept = torch.zeros(B, Hk, cap, dtype=torch.bool, device=DEV)
    kept.scatter_(2, order, slot < new_len)
    hole, mover = (slot < new_len) & ~kept, (slot >= new_len) & kept
    # the n-th mover goes to the n-th hole
    nth_hole = torch.where(hole, hole.long().cumsum(-1) - 1, cap)
    nth_mover = torch.where(mover, mover.long().cumsum(-1) - 1, cap)
    source = torch.zeros(B, Hk, cap + 1, dtype=torch.long, device=DEV).scatter_(2, nth_mover, slot)[..., :cap]
    source = torch.where(hole, torch.gather(source, 2, nth_hole.clamp(max=cap - 1)), slot)
    done = slot < new_len
    out_mass = torch.where(done, torch.gather(mass, 2, source), torch.zeros_like(mass))
    out_pos = torch.where(done, torch.gather(pos, 2, source), torch.full_like(pos, -1))
    b, h, t = hole.nonzero(as_tuple=True)
    u = source[b, h, t]
    page = s["k"].shape[2]
    at = s["table"].long()
    for_to, from_ = (at[b, t // page], h, t % page), (at[b, u // page], h, u % page)
    s["k"][for_to] = s["k"][from_]
    s["v"][for_to] = s["v"][from_]
    return new_len.view(-1).to(torch.int32), out_mass, out_pos, s["k"], s["v"]


def run(state):
    s, c = state, state["case"]
    if own:
        import attention_kl_divergence_attn_b200 as skl
        if c["op"] == "key_mass":
            mass, lse = skl.streamkl_key_mass(s["q"], s["k"], s["lse"], s["scale"], c["causal"], kv_len=s["kv_len"])
            return (mass,) if c["given"] else (mass, lse)
        if c["op"] == "decode":
            o, lse = skl.streamkl_decode(s["q"], s["k"], s["v"], s["table"], s["len"], s["scale"], mass=s["mass"],
                                         mass_out=s["mass_out"])
            return (o, lse) if s["mass"] is None else (o, lse, s["mass_out"])
        new_len, mass, pos = skl.streamkl_evict(s["k"], s["v"], s["table"], s["len"], s["mass"], c["budget"],
                                                recent=c["recent"], pos=s["pos"], next_pos=s["next_pos"])
        return new_len, mass, pos, s["k"], s["v"]
    return {"key_mass": _key_mass_plain, "decode": _decode_plain, "evict": _evict_plain}[c["op"]](s)


# ---------------------------------------------------------------------- work
def work(case):
    c = case
    if c["op"] == "key_mass":
        B, H, Hk, NQ, NK, d = c["B"], c["H"], c["Hk"], c["NQ"], c["NK"], c["d"]
        pairs = 0
        for n in (_key_lengths(c) if c["pad"] else [NK] * B):
            if c["causal"]:
                # row i sees min(n, i + NK - NQ + 1) keys
                full = max(0, min(NQ, NQ - (n - (NK - NQ)) + 1)) if n - (NK - NQ) >= 1 else NQ
                part = NQ - full
                pairs += full * n + part * (NK - NQ + 1) + part * (part - 1) // 2
            else:
                pairs += NQ * n
        keys = sum(_key_lengths(c)) if c["pad"] else B * NK
        return {"bytes": 2 * d * (B * H * NQ + Hk * keys) + 4 * B * H * NQ + 4 * B * Hk * NK,
                "flops": 2 * d * H * pairs}
    lens = _lengths(c)
    B, Hk, d, page = c["B"], c["Hk"], c["d"], c["page"]
    cap = -(-c["hi"] // page) * page
    tables = 4 * sum(-(-n // page) for n in lens) + 4 * B
    if c["op"] == "decode":
        by = 4 * d * Hk * sum(lens) + tables + 4 * d * B * c["H"] + 4 * B * c["H"]
        if c["mass"]:
            by += 8 * B * Hk * cap
        return {"bytes": by, "flops": 4 * d * c["H"] * sum(lens)}
    moved = 0.0
    for n in lens:
        over = n - c["budget"]
        if over > 0:
            new = min(c["recent"], n)
            moved += min(new, over) + max(0, over - new) * (c["budget"] - new) / max(1, n - new)
    return {"bytes": 8 * Hk * sum(lens) + 8 * B * Hk * cap + tables + 8 * d * Hk * moved,
            "flops": 2 * Hk * sum(lens)}


# --------------------------------------------------------------------- exact
def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    return {"key_mass": _key_mass_exact, "decode": _decode_exact, "evict": _evict_exact}[c["op"]](s, c)


def _key_mass_exact(s, c):
    B, H, Hk, NQ, NK = c["B"], c["H"], c["Hk"], c["NQ"], c["NK"]
    mass = torch.zeros(B, Hk, NK, dtype=torch.float64, device=DEV)
    lse = torch.full((B, H, NQ), -math.inf, dtype=torch.float64, device=DEV)
    step = max(1, (1 << 26) // NK)
    for b in range(B):
        n = NK if s["kv_len"] is None else int(s["kv_len"][b])
        for h in range(H):
            kd = s["k"][b, h // (H // Hk), :n].double()
            for i0 in range(0, NQ, step):
                y = s["q"][b, h, i0:i0 + step].double() @ kd.T * s["scale"]
                if c["causal"]:
                    last = torch.arange(i0, i0 + y.shape[0], device=DEV)[:, None] + (NK - NQ)
                    y = torch.where(torch.arange(n, device=DEV)[None, :] > last, -math.inf, y)
                l = torch.logsumexp(y, dim=1)
                lse[b, h, i0:i0 + step] = l
                used = l if s["lse"] is None else s["lse"][b, h, i0:i0 + step].double()
                seen = used > -math.inf
                mass[b, h // (H // Hk), :n] += torch.exp(y[seen] - used[seen, None]).sum(dim=0)
    return (mass,) if c["given"] else (mass, lse)


def _decode_exact(s, c):
    B, H, Hk, d, page = c["B"], c["H"], c["Hk"], c["d"], c["page"]
    G = H // Hk
    o = torch.zeros(B, H, d, dtype=torch.float64, device=DEV)
    lse = torch.full((B, H), -math.inf, dtype=torch.float64, device=DEV)
    mass = None if s["mass"] is None else s["mass"].double()
    for b, n in enumerate(s["len"].tolist()):
        if n == 0:
            continue
        t = torch.arange(n, device=DEV)
        at = s["table"][b].long()[t // page]
        for h in range(Hk):
            kd, vd = s["k"][at, h, t % page].double(), s["v"][at, h, t % page].double()
            y = s["q"][b, h * G:(h + 1) * G].double() @ kd.T * s["scale"]
            w = torch.softmax(y, dim=1)
            lse[b, h * G:(h + 1) * G] = torch.logsumexp(y, dim=1)
            o[b, h * G:(h + 1) * G] = w @ vd
            if mass is not None:
                mass[b, h, :n] += w.sum(dim=0)
    return (o, lse) if mass is None else (o, lse, mass)


def _evict_exact(s, c):
    page = c["page"]
    mass, pos = torch.zeros_like(s["mass"]), torch.full_like(s["pos"], -1)
    news = []
    for b, n in enumerate(s["len"].tolist()):
        keep = min(n, c["budget"])
        news.append(keep)
        for h in range(c["Hk"]):
            w = s["mass"][b, h, :n].cpu().double().clamp(min=0.0)
            p = s["pos"][b, h, :n].cpu()
            w[p >= int(s["next_pos"][b]) - c["recent"]] = math.inf
            rank = torch.argsort(-w, stable=True)
            stay = rank[:keep].sort().values
            src = torch.arange(keep)
            free = torch.ones(keep, dtype=torch.bool)
            free[stay[stay < keep]] = False
            src[free] = stay[stay >= keep]
            mass[b, h, :keep] = s["mass"][b, h, src.to(DEV)]
            pos[b, h, :keep] = s["pos"][b, h, src.to(DEV)]
            to = torch.arange(keep)[free].to(DEV)
            fr = src[free].to(DEV)
            at = s["table"][b].long()
            for x in (s["k"], s["v"]):
                x[at[to // page], h, to % page] = x[at[fr // page], h, fr % page]
    return (torch.tensor(news, dtype=torch.int32, device=DEV), mass.double(), pos, s["k"].double(), s["v"].double())
