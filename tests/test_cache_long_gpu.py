"""Evictions whose keys do not fit in a CTA's shared memory, up to the longest cache that is taken."""

import pytest
import torch

from attention_kl_divergence_attn_b200 import streamkl_check, streamkl_evict
from test_cache_gpu import BF, assert_evicted, gen, policy_inputs

pytestmark = pytest.mark.gpu


def evicted(k, v, table, lens, mass, budget, recent, pos, nxt):
    """cache_ref.evict without a loop over the slots."""
    page = k.shape[2]
    B, Hk, cap = mass.shape
    m2, p2, k2, v2 = torch.zeros_like(mass), torch.full_like(pos, -1), k.clone(), v.clone()
    for b in range(B):
        n, keep = int(lens[b]), min(int(lens[b]), budget)
        row = table[b].long()
        for h in range(Hk):
            m, at = mass[b, h, :n], pos[b, h, :n]
            key = torch.where(m > 0, m.view(torch.int32).long(), 0)        # a positive float's bits grow with it
            key = torch.where((at >= int(nxt[b]) - recent) & (recent > 0), 1 << 40, key)
            kept = torch.zeros(n, dtype=torch.bool)
            kept[torch.argsort(-key, stable=True)[:keep]] = True
            src = torch.arange(keep)
            src[~kept[:keep]] = torch.arange(keep, n)[kept[keep:]]
            m2[b, h, :keep], p2[b, h, :keep] = m[src], at[src]
            to = torch.arange(keep)[~kept[:keep]]
            fr = src[to]
            for x, y in ((k2, k), (v2, v)):
                x[row[to // page], h, to % page] = y[row[fr // page], h, fr % page]
    return torch.tensor([min(int(n), budget) for n in lens], dtype=torch.int32), m2, p2, k2, v2


def pages_for(g, lens, Hk, d, page, room):
    """(k, v, table): pages in random order; the table's unused columns name no page.  Any bits will do for rows."""
    used = [-(-n // page) for n in lens]
    order = torch.randperm(sum(used), generator=g).to(torch.int32)
    table = torch.full((len(lens), -(-room // page)), -1, dtype=torch.int32)
    first = 0
    for b, u in enumerate(used):
        table[b, :u] = order[first:first + u]
        first += u
    n = max(1, sum(used)) * Hk * page * d
    k = torch.randint(-2 ** 15, 2 ** 15, (n,), generator=g, dtype=torch.int16)
    return [x.view(BF).view(-1, Hk, page, d) for x in (k, k.flip(0))] + [table]


def run(g, lens, Hk, page, room, budget, recent, ties=None):
    k, v, table = pages_for(g, lens, Hk, 64, page, room)
    cap = table.shape[1] * page
    mass, pos, nxt = policy_inputs(g, len(lens), Hk, cap, lens)
    if ties:
        mass = (mass * ties).nan_to_num(0.0, 1e3, 0.0).clamp(-1, 50).round()    # few distinct weights
    n = torch.tensor(lens, dtype=torch.int32)
    want = evicted(k, v, table, lens, mass, budget, recent, pos, nxt)
    dev = [x.cuda() for x in (k, v, table, n, mass, pos, nxt)]
    got = streamkl_evict(*dev[:5], budget, recent=recent, pos=dev[5], next_pos=dev[6])
    assert streamkl_check() == 0
    assert_evicted(got, want, dev[0], dev[1])


@pytest.mark.parametrize("ties", [None, 4.0])
def test_one_long_sequence(ties):
    # eight CTAs of 1172 words of 32 slots: keys are read again in every pass
    run(gen(400), (300001,), 1, 64, 300001, 100000, 5000, ties)


@pytest.mark.parametrize("ties", [None, 4.0])
def test_many_rows_with_room(ties):
    # more rows than SMs: one CTA a row, whose room is past what it keeps keys of
    short = [(7 * i) % 101 for i in range(17)]
    run(gen(401), (40000, *short, 33333), 8, 64, 40000, 3000, 100, ties)


def test_clusters_that_the_room_asks_for():
    # more rows than SMs and more room than one CTA deals with
    run(gen(402), (270000, *[(5 * i) % 33 for i in range(149)]), 1, 128, 300000, 4096, 64)


@pytest.mark.parametrize("budget", [1, 1 << 20, (1 << 21) - 1])
def test_longest_cache(budget):
    run(gen(403), (1 << 21,), 1, 256, 1 << 21, budget, min(budget, 1000), 1.0 if budget > 1 else None)


def test_one_slot_more_is_refused():
    t = torch.zeros(1, (1 << 21) + 1, dtype=torch.int32, device="cuda")
    k = torch.zeros(2, 1, 1, 64, dtype=BF, device="cuda")
    with pytest.raises(RuntimeError):
        streamkl_evict(k, k.clone(), t, torch.ones(1, dtype=torch.int32, device="cuda"),
                       torch.zeros(1, 1, (1 << 21) + 1, device="cuda"), 1)
