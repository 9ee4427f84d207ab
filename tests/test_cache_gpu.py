"""The cache operators (key mass, paged decode, eviction) against 64-bit forms, elementwise."""
import math

import pytest
import torch

import attention_kl_divergence_attn_b200 as skl
import cache_ref as ref
from attention_kl_divergence_attn_b200 import (StreamKLError, streamkl_check, streamkl_decode, streamkl_evict,
                                               streamkl_fwd, streamkl_key_mass)

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


def gen(seed):
    return torch.Generator().manual_seed(seed)


def randn(g, *shape, dtype=BF, std=1.0):
    return (torch.randn(*shape, generator=g) * std).to(dtype)


def within(got, want, bound, what):
    got, want = got.detach().cpu().double(), want.double()
    same = (got == want) | (got.isnan() & want.isnan())
    bad = ~same & ~((got - want).abs() <= bound)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} outside, first at {bad.nonzero()[0].tolist()}: "
                           f"{got[bad][0]!r} for {want[bad][0]!r} +- {bound.expand_as(want)[bad][0]!r}")


# ------------------------------------------------------------------ key mass
MASS = [
    # B, H, Hk, N_Q, N_K, d, causal, dtype, lengths
    (1, 1, 1, 1, 1, 64, False, BF, None),
    (1, 1, 1, 128, 128, 64, False, BF, None),
    (2, 4, 2, 129, 129, 128, True, FP, None),
    (1, 5, 1, 61, 700, 64, True, BF, None),
    (3, 6, 3, 200, 333, 128, False, FP, (333, 1, 0)),
    (3, 6, 2, 200, 333, 64, True, BF, (332, 130, 17)),
    (1, 2, 2, 1, 5000, 128, True, BF, None),
    (1, 8, 2, 1, 4097, 64, False, FP, (4000,)),
    (1, 3, 3, 1500, 1501, 64, True, BF, None),
    (1, 1, 1, 3000, 40, 128, False, BF, None),
    (1, 4, 1, 63, 12000, 128, True, FP, None),
    # many tiles a run
    (2, 8, 2, 1700, 1750, 64, True, BF, None),
    (2, 8, 4, 1500, 1601, 128, False, FP, (1601, 900)),
    (2, 12, 3, 40, 30000, 128, True, FP, None),
    (1, 9, 1, 17, 60000, 64, False, BF, (59990,)),
]


@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("case", MASS, ids=lambda c: "x".join(str(x) for x in c[:7]))
def test_key_mass(case, given):
    B, H, Hk, N_Q, N_K, d, causal, dtype, lens = case
    g = gen(N_Q * 7 + N_K)
    q, k = randn(g, B, H, N_Q, d, dtype=dtype, std=1.5), randn(g, B, Hk, N_K, d, dtype=dtype)
    kv = None if lens is None else torch.tensor(lens, dtype=torch.int32)
    for b, n in enumerate(lens or ()):              # what lies in padding is never looked at
        k[b, :, n:] = torch.tensor([math.inf, math.nan, -math.inf, 3.0], dtype=dtype).repeat(d // 4)
    scale = 0.11
    lse = None
    if given:
        lse = ref.key_mass(q, k, scale, causal, kv)[1].float()
        lse[0, 0, 0] = -math.inf                    # rows that the caller leaves out
        lse[0, -1, N_Q // 2] = math.inf
    want, want_lse, bound, lse_bound = ref.key_mass(q, k, scale, causal, kv, lse)
    args = (q.cuda(), k.cuda(), None if lse is None else lse.cuda(), scale, causal)
    mass, got_lse = streamkl_key_mass(*args, kv_len=None if kv is None else kv.cuda())
    assert streamkl_check() == 0
    within(mass, want, bound, "mass")
    if given:
        assert torch.equal(got_lse.cpu(), lse)
    else:
        within(got_lse, want_lse, lse_bound, "lse")
    again, _ = streamkl_key_mass(*args, kv_len=None if kv is None else kv.cuda())
    assert torch.equal(mass, again)


def test_key_mass_strides():
    # token-major tensors and heads cut out of a wider projection
    g = gen(1)
    q = randn(g, 2, 150, 6, 192)[..., 64:].transpose(1, 2)
    k = randn(g, 2, 170, 2, 256)[..., 128:].transpose(1, 2)
    want, want_lse, bound, lb = ref.key_mass(q, k, 0.09, True)
    qc = torch.empty(2, 150, 6, 192, dtype=BF, device="cuda")[..., 64:].transpose(1, 2)
    kc = torch.empty(2, 170, 2, 256, dtype=BF, device="cuda")[..., 128:].transpose(1, 2)
    qc.copy_(q), kc.copy_(k)
    mass, lse = streamkl_key_mass(qc, kc, None, 0.09, True)
    assert streamkl_check() == 0
    within(mass, want, bound, "mass")
    within(lse, want_lse, lb, "lse")


def test_key_mass_pieces_accumulate():
    # a prompt in three pieces of query rows, each seeing the keys up to its end
    g = gen(2)
    q, k = randn(g, 1, 4, 500, 64), randn(g, 1, 2, 500, 64)
    want, _, bound, _ = ref.key_mass(q, k, 0.125, True)
    qc, kc = q.cuda(), k.cuda()
    mass = torch.full((1, 2, 500), math.nan, device="cuda")
    for lo, hi in ((0, 130), (130, 131), (131, 500)):
        # the causal diagonal ends at the last key, so the piece's keys are a slice
        part = torch.zeros(1, 2, hi, device="cuda") if lo == 0 else mass[..., :hi].contiguous()
        if lo:
            part[..., prev:] = 0
        streamkl_key_mass(qc[:, :, lo:hi], kc[:, :, :hi], None, 0.125, True, out=part, accumulate=True)
        mass[..., :hi] = part
        prev = hi
    assert streamkl_check() == 0
    within(mass, want, bound + 3 * 2.0 ** -24 * want, "mass")


def test_key_mass_from_the_forward():
    # the log-sum-exps that streamkl_fwd leaves behind
    g = gen(3)
    q, k = randn(g, 2, 4, 300, 128), randn(g, 2, 2, 310, 128)
    kv = torch.tensor([310, 200], dtype=torch.int32)
    _, lse, _, _ = streamkl_fwd(q.cuda(), k.cuda(), q.cuda(), k.cuda(), 0.1, 0.1, True, kv_len=kv.cuda())
    mass, _ = streamkl_key_mass(q.cuda(), k.cuda(), lse, 0.1, True, kv_len=kv.cuda())
    assert streamkl_check() == 0
    want, want_lse, bound, lb = ref.key_mass(q, k, 0.1, True, kv, lse.cpu())
    within(mass, want, bound, "mass")
    # every row with a key hands out a weight of 1 (off by its log-sum-exp's own error)
    rows = torch.isfinite(want_lse).sum((1, 2)).double()
    total = mass.double().sum((1, 2)).cpu()
    assert ((total - rows).abs() <= rows * (lb[torch.isfinite(want_lse)].max() + 1e-3) * 1.01).all()


def test_key_mass_infinite_key():
    # a key that every row weighs with exp(-inf) received nothing
    g = gen(18)
    q, k = randn(g, 1, 2, 70, 64), randn(g, 1, 2, 300, 64)
    q[..., 5] = q[..., 5].abs() + 0.5
    k[..., 5] = k[..., 5].abs()
    k[0, :, 33, 5] = -math.inf
    want = ref.key_mass(q, torch.where(k.isinf(), torch.tensor(-1e4, dtype=BF), k), 0.125, False)
    mass, lse = streamkl_key_mass(q.cuda(), k.cuda())
    assert streamkl_check() == 0
    assert torch.equal(mass[0, :, 33], torch.zeros_like(mass[0, :, 33]))
    other = torch.arange(300) != 33
    within(mass[..., other.cuda()], want[0][..., other], want[2][..., other], "mass")
    within(lse, want[1], want[3], "lse")


def test_overlapping_outputs_are_refused():
    q, k = torch.randn(1, 2, 8, 64, device="cuda").to(BF), torch.randn(1, 2, 8, 64, device="cuda").to(BF)
    lse = torch.zeros(1, 2, 8, device="cuda")
    with pytest.raises(ValueError):
        streamkl_key_mass(q, k, lse, out=lse)
    t, n = torch.zeros(1, 1, dtype=torch.int32, device="cuda"), torch.full((1,), 8, dtype=torch.int32, device="cuda")
    pages = k.clone()
    q1 = q[:, :, 0].contiguous()
    with pytest.raises(ValueError):
        streamkl_decode(q1, pages, k, t, n, out=(q1, torch.empty(1, 2, device="cuda")))
    mass = torch.zeros(3, 2, 8, device="cuda").view(-1)
    with pytest.raises(ValueError):
        streamkl_decode(q1, pages, k, t, n, mass=mass[:16].view(1, 2, 8), mass_out=mass[8:24].view(1, 2, 8))
    with pytest.raises(ValueError):
        streamkl_evict(pages, k, t, n, mass[:16].view(1, 2, 8), 4, out=(n, torch.empty(1, 2, 8, device="cuda"), None))
    with pytest.raises(ValueError):
        streamkl_evict(pages, pages, t, n, mass[:16].view(1, 2, 8), 4)
    assert streamkl_check() == 0


def test_key_mass_empty():
    q, k = torch.empty(2, 4, 0, 64, dtype=BF, device="cuda"), torch.randn(2, 2, 7, 64, device="cuda").to(BF)
    out = torch.full((2, 2, 7), math.nan, device="cuda")
    mass, lse = streamkl_key_mass(q, k, None, out=out)
    assert mass is out and torch.equal(out, torch.zeros_like(out)) and lse.shape == (2, 4, 0)
    out.fill_(3)
    assert torch.equal(streamkl_key_mass(q, k, None, out=out, accumulate=True)[0], torch.full_like(out, 3))
    assert streamkl_key_mass(q[:0], k[:0])[0].shape == (0, 2, 7)
    assert streamkl_check() == 0


def test_key_mass_bad_length_is_reported_and_clamped():
    g = gen(4)
    q, k = randn(g, 2, 1, 10, 64), randn(g, 2, 1, 50, 64)
    kv = torch.tensor([51, -1], dtype=torch.int32)
    mass, _ = streamkl_key_mass(q.cuda(), k.cuda(), None, 0.1, kv_len=kv.cuda())
    with pytest.raises(StreamKLError):
        streamkl_check()
    assert streamkl_check() == 0
    want, _, bound, _ = ref.key_mass(q, k, 0.1, False, kv.clamp(0, 50))
    within(mass, want, bound, "mass")


# -------------------------------------------------------------------- decode
def cache(g, lens, Hk, d, page, dtype, layout="HND", spare=2, std=1.0):
    """(k_pages, v_pages, table): CPU, pages in random order, junk in every slot that no sequence holds."""
    per = max(1, max(-(-n // page) for n in lens))
    pages = len(lens) * per + spare
    table = torch.randperm(pages, generator=g)[:len(lens) * per].view(len(lens), per).to(torch.int32)
    out = []
    for _ in range(2):
        x = randn(g, pages, Hk, page, d, dtype=dtype, std=std)
        live = torch.zeros(pages, page, dtype=torch.bool)
        for b, n in enumerate(lens):
            t = torch.arange(n)
            live[table[b].long()[t // page], t % page] = True
        x.masked_fill_(~live[:, None, :, None], math.nan)
        out.append(x.transpose(1, 2).contiguous().transpose(1, 2) if layout == "NHD" else x)
    return out[0], out[1], table


def on_gpu(x):
    y = torch.empty_strided(x.shape, x.stride(), dtype=x.dtype, device="cuda")
    return y.copy_(x)


DECODE = [
    # H, Hk, d, page, dtype, layout, lengths
    (1, 1, 64, 1, BF, "HND", (1,)),
    (8, 2, 64, 16, BF, "HND", (77,)),
    (4, 4, 128, 24, FP, "NHD", (0, 1, 15, 16, 17, 63, 64, 65)),
    (5, 1, 128, 64, BF, "NHD", (1000, 0, 3)),
    (16, 1, 64, 100, FP, "HND", (129, 300)),
    (17, 1, 128, 8, BF, "HND", (200, 64)),
    (66, 2, 64, 32, FP, "NHD", (130, 1, 0, 257)),
    (6, 3, 128, 256, BF, "HND", (2000, 5, 1024, 1, 700, 0, 0, 31)),
    (32, 8, 128, 64, BF, "HND", (9000,)),
    (2, 1, 64, 48, FP, "HND", (40001, 12)),
]


@pytest.mark.parametrize("with_mass", [False, True])
@pytest.mark.parametrize("case", DECODE, ids=lambda c: "x".join(str(x) for x in c[:4]) + c[5] + str(len(c[6])))
def test_decode(case, with_mass):
    H, Hk, d, page, dtype, layout, lens = case
    g = gen(sum(lens) + H)
    B = len(lens)
    k, v, table = cache(g, lens, Hk, d, page, dtype, layout)
    q = randn(g, B, H, d, dtype=dtype, std=2.0)
    n = torch.tensor(lens, dtype=torch.int32)
    mass = torch.rand(B, Hk, table.shape[1] * page + 3, generator=g) if with_mass else None
    want = ref.decode(q, k, v, table, n, 0.13, mass)
    dev = [on_gpu(x) for x in (q, k, v, table, n)]
    mc = mass.cuda() if with_mass else None
    mo = torch.full_like(mc, math.nan) if with_mass else None
    out, lse = streamkl_decode(*dev, 0.13, mass=mc, mass_out=mo)
    assert streamkl_check() == 0
    within(out, want[0], want[3], "out")
    within(lse, want[1], want[4], "lse")
    if with_mass:
        within(mo, want[2], want[5], "mass")
        assert torch.equal(mc.cpu(), mass)
    again = streamkl_decode(*dev, 0.13, mass=mc)                 # in place
    assert torch.equal(again[0], out) and torch.equal(again[1], lse)
    if with_mass:
        assert torch.equal(mc, mo)


def test_decode_many_sequences():
    # more sequences than threads in a block, most of them empty
    g = gen(5)
    lens = [int(x) for x in torch.randint(0, 90, (700,), generator=g) * (torch.rand(700, generator=g) < 0.2)]
    k, v, table = cache(g, lens, 2, 64, 16, BF)
    q = randn(g, 700, 4, 64)
    n = torch.tensor(lens, dtype=torch.int32)
    want = ref.decode(q, k, v, table, n, 0.125)
    out, lse = streamkl_decode(*[on_gpu(x) for x in (q, k, v, table, n)])
    assert streamkl_check() == 0
    within(out, want[0], want[3], "out")
    within(lse, want[1], want[4], "lse")


def test_decode_contiguous_cache_and_views():
    # one page a sequence, q cut out of a fused projection, table rows with a stride
    g = gen(6)
    lens = (333, 64, 500)
    k, v, _ = cache(g, lens, 2, 128, 512, BF, spare=0)
    table = torch.arange(3, dtype=torch.int32)[:, None]
    live = [torch.arange(512) < n for n in lens]
    for x in (k, v):
        for b in range(3):
            x[b] = torch.where(live[b][None, :, None], randn(g, 2, 512, 128), torch.tensor(math.nan, dtype=BF))
    wide = randn(g, 3, 12, 128)
    want = ref.decode(wide[:, 2:10], k, v, table, torch.tensor(lens), 0.1)
    tc = torch.full((3, 5), -7, dtype=torch.int32, device="cuda")
    tc[:, 1:2] = table.cuda()
    out, lse = streamkl_decode(wide.cuda()[:, 2:10], k.cuda(), v.cuda(), tc[:, 1:2],
                               torch.tensor(lens, dtype=torch.int32, device="cuda"), 0.1)
    assert streamkl_check() == 0
    within(out, want[0], want[3], "out")
    within(lse, want[1], want[4], "lse")


def test_decode_shared_prefix():
    # two sequences over the same pages (an expanded table)
    g = gen(7)
    k, v, table = cache(g, (150,), 2, 64, 32, FP)
    q = randn(g, 2, 4, 64, dtype=FP)
    n = torch.tensor([150, 70], dtype=torch.int32)
    want = ref.decode(q, k, v, table.expand(2, -1), n, 0.125)
    out, lse = streamkl_decode(q.cuda(), k.cuda(), v.cuda(), table.cuda().expand(2, -1), n.cuda(), 0.125)
    assert streamkl_check() == 0
    within(out, want[0], want[3], "out")
    within(lse, want[1], want[4], "lse")


def test_decode_extreme_logits():
    # one token takes all, and a long tail far below it
    g = gen(8)
    for dtype in (BF, FP):
        k, v, table = cache(g, (3000, 3000), 1, 128, 64, dtype, std=4.0)
        q = randn(g, 2, 3, 128, dtype=dtype, std=6.0)
        n = torch.tensor([3000, 2999], dtype=torch.int32)
        want = ref.decode(q, k, v, table, n, 1.0)
        out, lse = streamkl_decode(*[on_gpu(x) for x in (q, k, v, table, n)], 1.0)
        assert streamkl_check() == 0
        within(out, want[0], want[3], "out")
        within(lse, want[1], want[4], "lse")


def test_decode_bad_lengths_and_pages():
    g = gen(9)
    lens = (100, 96, 40, 64)
    k, v, table = cache(g, lens, 2, 64, 16, BF)
    q = randn(g, 4, 4, 64)
    table[0, 2], table[0, 5] = -1, k.shape[0]                    # tokens 32..47 and 80..95 do not exist
    table[3] = k.shape[0] + 5                                    # nothing exists
    mass = torch.rand(4, 2, table.shape[1] * 16, generator=g)
    want = ref.decode(q, k, v, table, torch.tensor(lens), 0.2, mass)
    mc = mass.cuda()
    out, lse = streamkl_decode(q.cuda(), k.cuda(), v.cuda(), table.cuda(),
                               torch.tensor(lens, dtype=torch.int32, device="cuda"), 0.2, mass=mc)
    with pytest.raises(StreamKLError):
        streamkl_check()
    assert streamkl_check() == 0
    within(out, want[0], want[3], "out")
    within(lse, want[1], want[4], "lse")
    within(mc, want[2], want[5], "mass")
    # lengths outside the table are clamped to it
    k, v, table = cache(g, (112, 112), 1, 64, 16, BF)
    n = torch.tensor([113, -5], dtype=torch.int32)
    want = ref.decode(q[:2, :2], k, v, table, n.clamp(0, 112), 0.2)
    out, lse = streamkl_decode(q[:2, :2].cuda(), k.cuda(), v.cuda(), table.cuda(), n.cuda(), 0.2)
    with pytest.raises(StreamKLError):
        streamkl_check()
    within(out, want[0], want[3], "out")
    within(lse, want[1], want[4], "lse")


def test_decode_offsets_past_32_bits():
    # the used pages lie past 2^32 elements of the cache
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB")
    g = gen(10)
    page, Hk, d = 64, 2, 128
    pages = (1 << 32) // (Hk * page * d) + 9
    big = torch.empty(pages, Hk, page, d, dtype=BF, device="cuda")
    lens, last = (200, 130), pages - 1
    table = torch.tensor([[last, last - 2, 0, last - 1], [last - 3, last - 5, last - 4, 1]], dtype=torch.int32)
    small, stable = torch.empty(8, Hk, page, d, dtype=BF), torch.arange(8, dtype=torch.int32).view(2, 4)
    small.copy_(randn(g, 8, Hk, page, d))
    big[table.view(-1).long().cuda()] = small.cuda()
    q = randn(g, 2, 4, d)
    n = torch.tensor(lens, dtype=torch.int32)
    want = ref.decode(q, small, small, stable, n, 0.1)
    out, lse = streamkl_decode(q.cuda(), big, big, table.cuda(), n.cuda(), 0.1)
    assert streamkl_check() == 0
    within(out, want[0], want[3], "out")
    within(lse, want[1], want[4], "lse")
    # and moved there by an eviction
    mass = torch.rand(2, Hk, 256, generator=g)
    big2 = torch.empty_strided(big.shape, big.stride(), dtype=BF, device="cuda")
    big2[table.view(-1).long().cuda()] = small.cuda()
    want = ref.evict(small, small, stable, n, mass, 70)
    got = streamkl_evict(big, big2, table.cuda(), n.cuda(), mass.cuda(), 70)
    assert streamkl_check() == 0
    assert torch.equal(got[1].cpu(), want[1])
    for x in (big, big2):
        assert torch.equal(x[table.view(-1).long().cuda()].cpu(), want[3])


# --------------------------------------------------------------------- evict
EVICT = [
    # Hk, d, page, layout, lengths, budget, recent
    (1, 64, 16, "HND", (1,), 1, 0),
    (2, 64, 16, "HND", (33, 32, 31, 0), 32, 5),
    (3, 128, 24, "NHD", (500, 70, 1), 100, 100),
    (2, 128, 1, "HND", (40,), 39, 0),
    (1, 64, 64, "NHD", (1500, 1100, 2100), 1024, 64),
    (2, 64, 100, "HND", (3000,), 1, 1),
    (2, 64, 100, "HND", (300, 10), 0, 0),
    (1, 128, 256, "HND", (5000, 5000), 4999, 0),
]


def assert_evicted(got, want, k, v):
    for a, b, what in zip((*got, k, v), want, ("new_len", "mass", "pos", "k", "v")):
        if b is None:
            assert a is None
            continue
        a = a.cpu()
        if a.dtype in (BF, FP):
            a, b = a.contiguous().view(torch.int16), b.contiguous().view(torch.int16)
        elif a.dtype == torch.float32:
            a, b = a.view(torch.int32), b.view(torch.int32)
        assert torch.equal(a, b), what


def policy_inputs(g, B, Hk, cap, lens):
    mass = torch.randn(B, Hk, cap, generator=g).mul(2).exp()
    mass[torch.rand(B, Hk, cap, generator=g) < 0.2] = 0.0
    mass[torch.rand(B, Hk, cap, generator=g) < 0.1] = 1.5         # ties
    odd = torch.tensor([math.nan, -math.nan, -1.0, -0.0, math.inf, -math.inf, 1e-42])
    at = torch.rand(B, Hk, cap, generator=g) < 0.05
    mass[at] = odd[torch.randint(0, len(odd), (int(at.sum()),), generator=g)]
    pos = torch.rand(B, Hk, cap, generator=g).argsort(-1).to(torch.int32)
    return mass, pos, torch.tensor([n for n in lens], dtype=torch.int32)


@pytest.mark.parametrize("case", EVICT, ids=lambda c: "x".join(str(x) for x in (*c[:3], c[3], len(c[4]), *c[5:])))
def test_evict(case):
    Hk, d, page, layout, lens, budget, recent = case
    g = gen(sum(lens) + budget)
    k, v, table = cache(g, lens, Hk, d, page, BF, layout)
    cap = table.shape[1] * page + 5
    mass, pos, nxt = policy_inputs(g, len(lens), Hk, cap, lens)
    n = torch.tensor(lens, dtype=torch.int32)
    want = ref.evict(k, v, table, n, mass, budget, recent, pos, nxt)
    kc, vc, tc, nc, mc, pc, xc = [on_gpu(x) for x in (k, v, table, n, mass, pos, nxt)]
    got = streamkl_evict(kc, vc, tc, nc, mc, budget, recent=recent, pos=pc, next_pos=xc)
    assert streamkl_check() == 0
    assert_evicted(got, want, kc, vc)
    for a, b in ((mc, mass), (pc, pos), (tc, table), (nc, n)):
        assert torch.equal(a.cpu().view(torch.int32), b.view(torch.int32))       # inputs stay
    if recent == 0:                                               # without positions
        kc, vc = on_gpu(k), on_gpu(v)
        got = streamkl_evict(kc, vc, tc, nc, mc, budget)
        assert_evicted(got, (want[0], want[1], None, want[3], want[4]), kc, vc)


def test_evict_long():
    # more slots than fit in shared memory, few distinct weights
    g = gen(11)
    lens, page, budget = (50001, 60000), 128, 20000
    k, v, table = cache(g, lens, 1, 64, page, FP)
    cap = table.shape[1] * page
    mass, pos, nxt = policy_inputs(g, 2, 1, cap, lens)
    mass[1] = (mass[1] > 1).float()
    n = torch.tensor(lens, dtype=torch.int32)
    want = ref.evict(k, v, table, n, mass, budget, 500, pos, nxt)
    kc, vc, tc, nc, mc, pc, xc = [on_gpu(x) for x in (k, v, table, n, mass, pos, nxt)]
    got = streamkl_evict(kc, vc, tc, nc, mc, budget, recent=500, pos=pc, next_pos=xc)
    assert streamkl_check() == 0
    assert_evicted(got, want, kc, vc)


@pytest.mark.parametrize("columns", [7, 2000])        # few entries, and more than a sequence looks through itself
def test_evict_leaves_shared_and_bad_pages(columns):
    g = gen(12)
    lens = (100, 100, 20, 100, 64, 100, 100)
    k, v, table = cache(g, lens, 2, 64, 16, BF)
    k, v = k.nan_to_num(1.0), v.nan_to_num(2.0)
    table[2, 1] = table[1, 3]          # a short sequence shares a page with one that evicts
    table[3, 4] = table[3, 2]          # one page twice
    table[4, 3] = -2                   # no such page, and nothing to evict
    table[5, 0] = k.shape[0]           # no such page
    table[6, 6] = table[0, 6]          # both evict
    mass, pos, nxt = policy_inputs(g, 7, 2, 112, lens)
    n = torch.tensor(lens, dtype=torch.int32)
    lens2 = (100, 100, 20, 100, 64, 100, 50)
    for lengths, skip in ((lens, (0, 1, 2, 3, 4, 5, 6)), (lens2, (1, 2, 3, 4, 5))):
        # with 50 tokens the last sequence does not reach the page that it shares
        n = torch.tensor(lengths, dtype=torch.int32)
        budget = 64
        if lengths is lens2:
            budget = 49
        want = ref.evict(k, v, table.clamp(0, k.shape[0] - 1), n, mass, budget, 3, pos, nxt, skip=skip)
        kc, vc = k.cuda(), v.cuda()
        wide = torch.full((7, columns), -9, dtype=torch.int32)
        wide[:, :7] = table
        got = streamkl_evict(kc, vc, wide.cuda(), n.cuda(), mass.cuda(), budget, recent=3, pos=pos.cuda(),
                             next_pos=nxt.cuda())
        with pytest.raises(StreamKLError):
            streamkl_check()
        assert streamkl_check() == 0
        assert_evicted(got, want, kc, vc)


@pytest.mark.parametrize("columns", [4, 5000])
def test_evict_shared_prefix_without_eviction(columns):
    # sharing is fine while nobody evicts
    g = gen(13)
    k, v, table = cache(g, (60,), 1, 64, 16, BF)
    mass, pos, nxt = policy_inputs(g, 2, 1, 64, (60, 30))
    n = torch.tensor([60, 30], dtype=torch.int32)
    kc, vc = k.cuda(), v.cuda()
    wide = torch.zeros(1, columns, dtype=torch.int32)
    wide[:, :4] = table
    got = streamkl_evict(kc, vc, wide.cuda().expand(2, -1), n.cuda(), mass.cuda(), 60)
    assert streamkl_check() == 0
    assert got[0].tolist() == [60, 30]
    assert torch.equal(kc.cpu().view(torch.int16), k.view(torch.int16))
    # and both stay as they are when one does
    got = streamkl_evict(kc, vc, wide.cuda().expand(2, -1), n.cuda(), mass.cuda(), 40)
    with pytest.raises(StreamKLError):
        streamkl_check()
    assert got[0].tolist() == [60, 30]
    assert torch.equal(kc.cpu().view(torch.int16), k.view(torch.int16))


def test_evict_many_columns():
    # a table of more entries than a sequence looks through itself, used far into its rows
    g = gen(19)
    lens = (9000, 3, 8000)
    k, v, table = cache(g, lens, 1, 64, 1, BF)
    mass, pos, nxt = policy_inputs(g, 3, 1, 9000, lens)
    n = torch.tensor(lens, dtype=torch.int32)
    want = ref.evict(k, v, table, n, mass, 100, 10, pos, nxt)
    kc, vc, tc, nc, mc, pc, xc = [on_gpu(x) for x in (k, v, table, n, mass, pos, nxt)]
    got = streamkl_evict(kc, vc, tc, nc, mc, 100, recent=10, pos=pc, next_pos=xc)
    assert streamkl_check() == 0
    assert_evicted(got, want, kc, vc)


# ------------------------------------------------------- streams, graphs, use
def test_two_streams_and_two_graphs():
    """Calls on two streams at once, and two captured graphs replayed side by side, do not share scratch."""
    g = gen(14)
    sets = []
    for s in range(2):
        lens = (3000 + 11 * s, 77, 1500)
        k, v, table = cache(g, lens, 2, 128, 64, BF)
        q = randn(g, 3, 8, 128, std=2.0)
        n = torch.tensor(lens, dtype=torch.int32)
        mass = torch.rand(3, 2, table.shape[1] * 64, generator=g)
        qq, kk = randn(g, 1, 4, 70, 64), randn(g, 1, 2, 6000, 64)
        sets.append([on_gpu(x) for x in (q, k.nan_to_num(0.0), v.nan_to_num(0.0), table, n, mass, qq, kk)])

    def work(x):
        q, k, v, table, n, mass, qq, kk = x
        kc, vc = k.clone(), v.clone()
        o, lse = streamkl_decode(q, kc, vc, table, n, mass=mass, mass_out=(mo := torch.empty_like(mass)))
        new, m2, _ = streamkl_evict(kc, vc, table, n, mo, 1024)
        o2, lse2 = streamkl_decode(q, kc, vc, table, new)
        km, kl = streamkl_key_mass(qq, kk, causal=True)
        return [o, lse, mo, new, m2, o2, lse2, km, kl, kc, vc]

    base = [work(x) for x in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    outs = [[], []]
    for _ in range(5):
        for i, (s, x) in enumerate(zip(streams, sets)):
            with torch.cuda.stream(s):
                outs[i].append(work(x))
    torch.cuda.synchronize()
    for i in range(2):
        for got in outs[i]:
            assert all(torch.equal(a, b) for a, b in zip(got, base[i]))
    graphs, caught = [], []
    for x in sets:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            caught.append(work(x))
        graphs.append(graph)
    for _ in range(3):
        for s, graph in zip(streams, graphs):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(a, b) for a, b in zip(caught[i], base[i]))
    assert streamkl_check() == 0


def test_stream_argument():
    g = gen(15)
    k, v, table = cache(g, (500,), 2, 64, 16, BF)
    q = randn(g, 1, 4, 64)
    n = torch.tensor([500], dtype=torch.int32)
    dev = [on_gpu(x) for x in (q, k, v, table, n)]
    base = streamkl_decode(*dev)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = streamkl_decode(*dev, stream=s)
    s.synchronize()
    assert torch.equal(got[0], base[0]) and torch.equal(got[1], base[1])
    assert streamkl_check(stream=s) == 0


def test_serving_with_a_bounded_cache():
    """Prompt, key mass, eviction to a budget, then tokens with an eviction whenever a sequence is a page over it."""
    g = gen(16)
    B, H, Hk, d, page, N, budget, recent, steps = 3, 8, 2, 64, 16, 150, 64, 16, 40
    lens = [150, 90, 40]
    scale = 0.2
    q, k, v = randn(g, B, H, N, d, std=2.0), randn(g, B, Hk, N, d), randn(g, B, Hk, N, d)
    kv = torch.tensor(lens, dtype=torch.int32)
    _, lse, _, _ = streamkl_fwd(q.cuda(), k.cuda(), q.cuda(), k.cuda(), scale, scale, False, kv_len=kv.cuda())
    per = -(-N // page) + 1
    cap = per * page
    table = torch.randperm(B * per, generator=g).view(B, per).to(torch.int32)
    kp = torch.full((B * per, Hk, page, d), math.nan, dtype=BF)
    vp = kp.clone()
    for b in range(B):
        for t in range(lens[b]):
            kp[table[b, t // page], :, t % page] = k[b, :, t]
            vp[table[b, t // page], :, t % page] = v[b, :, t]
    # on the GPU
    kc, vc, tc, length, nxt = kp.cuda(), vp.cuda(), table.cuda(), kv.cuda(), kv.cuda().clone()
    mass = torch.zeros(B, Hk, cap, device="cuda")
    mass[..., :N] = streamkl_key_mass(q.cuda(), k.cuda(), lse, scale, False, kv_len=kv.cuda())[0]
    pos = torch.arange(cap, dtype=torch.int32, device="cuda").expand(B, Hk, cap).contiguous()
    # 64-bit, on the CPU, from the definition; the slots' order follows the GPU's masses, which decide near ties
    for step in range(steps):
        if step % page == 0:
            before = [x.cpu() for x in (kc, vc, length, mass, pos, nxt)]
            length, mass, pos = streamkl_evict(kc, vc, tc, length, mass, budget, recent=recent, pos=pos, next_pos=nxt)
            want = ref.evict(before[0], before[1], table, before[2], before[3], budget, recent, before[4], before[5])
            assert_evicted((length, mass, pos), want, kc, vc)
        qs, ks, vs = randn(g, B, H, d, std=2.0), randn(g, B, Hk, d), randn(g, B, Hk, d)
        at = length.long()
        rows = torch.arange(B, device="cuda")
        page_at = tc.long()[rows, at // page]
        kc[page_at, :, at % page], vc[page_at, :, at % page] = ks.cuda(), vs.cuda()
        pos[rows, :, at] = nxt[:, None]
        mass[rows, :, at] = 0.0
        length, nxt = length + 1, nxt + 1
        before = mass.cpu()
        out, lse = streamkl_decode(qs.cuda(), kc, vc, tc, length, scale, mass=mass)
        want = ref.decode(qs, kc.cpu(), vc.cpu(), table, length.cpu(), scale, before)
        within(out, want[0], want[3], f"out {step}")
        within(lse, want[1], want[4], f"lse {step}")
        within(mass, want[2], want[5], f"mass {step}")
    assert streamkl_check() == 0
    assert length.tolist() == [min(n, budget) + 8 for n in (150, 90)] + [min(40 + 32, budget) + 8]
    assert nxt.tolist() == [n + steps for n in lens]


@pytest.mark.parametrize("case", [0, 1])
def test_checked_build(case):
    """The bounds-checked build finds every access of the key-mass kernels in bounds."""
    from attention_kl_divergence_attn_b200 import build as kbuild
    from test_bounds_gpu import library
    B, H, Hk, N_Q, N_K, d, causal, dtype, lens = MASS[(5, 10)[case]]
    g = gen(17)
    q, k = randn(g, B, H, N_Q, d, dtype=dtype).cuda(), randn(g, B, Hk, N_K, d, dtype=dtype).cuda()
    kv = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    want = streamkl_key_mass(q, k, None, 0.1, causal, kv_len=kv)
    assert streamkl_check() == 0
    with library(kbuild.build(checked=True)):
        got = streamkl_key_mass(q, k, None, 0.1, causal, kv_len=kv)
        assert streamkl_check() == 0
    for a, b in zip(got, want):
        torch.testing.assert_close(a, b, rtol=1e-6, atol=1e-6)


# --------------------------------------------------------------------- sweeps
@pytest.mark.parametrize("seed", range(30))
def test_key_mass_sweep(seed):
    import random
    rng = random.Random(seed)
    Hk = rng.choice([1, 1, 2, 3])
    G = rng.choice([1, 1, 2, 3, 7, 16, 130 if seed % 3 == 0 else 4])
    N_K = rng.choice([1, 63, 64, 127, 128, 129, 255, 256, 257, 400, 777])
    N_Q = rng.choice([1, 2, 5, 31, 32, 33, 60, 64, 65, 120, 128, 129, 256, 300])
    causal = rng.random() < 0.6
    if causal:
        N_Q = min(N_Q, N_K)
    if G > 16:
        N_Q = min(N_Q, 40)
    B, d, dtype = rng.randint(1, 4), rng.choice([64, 128]), rng.choice([BF, FP])
    lens = None if rng.random() < 0.5 else [rng.choice([0, 1, N_K, rng.randint(0, N_K)]) for _ in range(B)]
    g = gen(1000 + seed)
    q, k = randn(g, B, G * Hk, N_Q, d, dtype=dtype, std=1.5), randn(g, B, Hk, N_K, d, dtype=dtype)
    kv = None if lens is None else torch.tensor(lens, dtype=torch.int32)
    want, want_lse, bound, lse_bound = ref.key_mass(q, k, 0.1, causal, kv)
    out = torch.full((B, Hk, N_K), math.nan, device="cuda")
    mass, lse = streamkl_key_mass(q.cuda(), k.cuda(), None, 0.1, causal, kv_len=None if kv is None else kv.cuda(),
                                  out=out)
    assert streamkl_check() == 0
    within(mass, want, bound, "mass")
    within(lse, want_lse, lse_bound, "lse")


@pytest.mark.parametrize("seed", range(30))
def test_decode_and_evict_sweep(seed):
    import random
    rng = random.Random(seed)
    Hk, G = rng.choice([1, 2, 3, 8]), rng.choice([1, 2, 3, 5, 16, 17, 40])
    page, d = rng.choice([1, 3, 16, 24, 64, 100, 256]), rng.choice([64, 128])
    dtype, layout = rng.choice([BF, FP]), rng.choice(["HND", "NHD"])
    top = rng.choice([1, 40, 300, 512, 513, 1500])
    lens = [rng.choice([0, 1, rng.randint(0, top), top]) for _ in range(rng.randint(1, 6))]
    g = gen(2000 + seed)
    B = len(lens)
    k, v, table = cache(g, lens, Hk, d, page, dtype, layout)
    q = randn(g, B, G * Hk, d, dtype=dtype, std=2.0)
    n = torch.tensor(lens, dtype=torch.int32)
    cap = table.shape[1] * page
    mass, pos, nxt = policy_inputs(g, B, Hk, cap, lens)
    dev = [on_gpu(x) for x in (k, v, table, n)]
    weight = mass.nan_to_num(0.0, 1.0, 1.0).clamp(min=0.0)
    want = ref.decode(q, k, v, table, n, 0.12, weight)
    wc = weight.cuda()
    out, lse = streamkl_decode(q.cuda(), *dev, 0.12, mass=wc)
    assert streamkl_check() == 0
    within(out, want[0], want[3], "out")
    within(lse, want[1], want[4], "lse")
    within(wc, want[2], want[5], "mass")
    budget = rng.randint(0, top + 3)
    recent = rng.randint(0, budget)
    want = ref.evict(k, v, table, n, mass, budget, recent, pos, nxt)
    got = streamkl_evict(*dev, mass.cuda(), budget, recent=recent, pos=pos.cuda(), next_pos=nxt.cuda())
    assert streamkl_check() == 0
    assert_evicted(got, want, dev[0], dev[1])


def test_short_caches_in_a_graph():
    # a row a CTA and its weights in one kernel, captured and replayed on new lengths
    g = gen(20)
    k, v, table = cache(g, (100, 60), 2, 64, 16, BF)
    k, v = k.nan_to_num(0.5), v.nan_to_num(0.5)
    q = randn(g, 2, 8, 64)
    mass = torch.rand(2, 2, 112, generator=g)
    kc, vc, tc, qc, mc = k.cuda(), v.cuda(), table.cuda(), q.cuda(), mass.cuda()
    n = torch.tensor([100, 60], dtype=torch.int32, device="cuda")
    mo = torch.empty_like(mc)
    streamkl_decode(qc, kc, vc, tc, n, mass=mc, mass_out=mo)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = streamkl_decode(qc, kc, vc, tc, n, mass=mc, mass_out=mo)
        new, m2, _ = streamkl_evict(kc.clone(), vc.clone(), tc, n, mo, 32)
    for lens in ((100, 60), (7, 0), (112, 33)):
        n.copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        want = ref.decode(q, k, v, table, lens, 0.125, mass)
        within(out, want[0], want[3], "out")
        within(lse, want[1], want[4], "lse")
        within(mo, want[2], want[5], "mass")
        assert new.tolist() == [min(x, 32) for x in lens]
    assert streamkl_check() == 0
