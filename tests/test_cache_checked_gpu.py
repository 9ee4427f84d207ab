"""The cache operators through the bounds-checked build.  Key mass: items that runs share, items without a tile,
packed heads, sums added to, log-sum-exps given and computed.  Decode and eviction: rows split and whole, every way
to look for shared pages, bad pages and lengths."""
import random

import pytest
import torch

from attention_kl_divergence_attn_b200 import (StreamKLError, build as kbuild, streamkl_check, streamkl_decode,
                                               streamkl_evict, streamkl_key_mass)
from test_bounds_gpu import library
from test_cache_gpu import BF, DECODE, EVICT, FP, MASS, cache, gen, on_gpu, policy_inputs, randn

pytestmark = pytest.mark.gpu

EMPTY = [                                                 # batch elements and key tiles without a visible key
    (3, 4, 2, 130, 700, 64, True, BF, (0, 700, 257)),
    (4, 6, 2, 33, 1500, 128, False, FP, (0, 0, 1500, 3)),
    (2, 16, 1, 5, 40000, 64, False, BF, (0, 39999)),
    (2, 3, 3, 1000, 1000, 128, True, BF, (0, 0)),
]


def drawn(seed):
    rng = random.Random(seed)
    Hk, G, B = rng.choice([1, 2, 3]), rng.choice([1, 2, 7, 20]), rng.randint(1, 4)
    N_K = rng.choice([1, 128, 255, 257, 900, 5000])
    N_Q = min(rng.choice([1, 31, 64, 65, 129, 400]), N_K)
    lens = None if rng.random() < 0.3 else tuple(rng.choice([0, 1, N_K, rng.randint(0, N_K)]) for _ in range(B))
    return B, Hk * G, Hk, N_Q, N_K, rng.choice([64, 128]), rng.random() < 0.6, rng.choice([BF, FP]), lens


@pytest.mark.parametrize("case", MASS + EMPTY + [drawn(s) for s in range(12)],
                         ids=lambda c: "x".join(str(x) for x in c[:7]))
def test_key_mass_stays_in_bounds(case):
    B, H, Hk, N_Q, N_K, d, causal, dtype, lens = case
    g = gen(300 + N_Q + N_K)
    q, k = randn(g, B, H, N_Q, d, dtype=dtype).cuda(), randn(g, B, Hk, N_K, d, dtype=dtype).cuda()
    kv = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")

    def calls():
        mass, lse = streamkl_key_mass(q, k, None, 0.1, causal, kv_len=kv)
        again, _ = streamkl_key_mass(q, k, lse, 0.1, causal, kv_len=kv)
        twice, _ = streamkl_key_mass(q, k, lse, 0.1, causal, kv_len=kv, out=mass.clone(), accumulate=True)
        assert streamkl_check() == 0
        return mass, lse, again, twice

    want = calls()
    with library(kbuild.build(checked=True)):
        got = calls()
    for a, b in zip(got, want):
        torch.testing.assert_close(a, b, rtol=1e-6, atol=1e-6)
    assert torch.equal(want[0], want[2]) and torch.equal(want[3], 2 * want[0])


def same(got, want):
    for a, b in zip(got, want):
        assert (a is None) == (b is None)
        if a is not None:
            bits = torch.int16 if a.element_size() == 2 else torch.int32
            assert torch.equal(a.contiguous().view(bits), b.contiguous().view(bits))


def serve(H, Hk, d, page, dtype, layout, lens, budget, recent, seed):
    """Decode with and without weights, then an eviction of the same cache, in both builds: the same bits."""
    g = gen(seed)
    k, v, table = cache(g, lens, Hk, d, page, dtype, layout)
    cap = table.shape[1] * page + 5
    mass, pos, nxt = policy_inputs(g, len(lens), Hk, cap, lens)
    q = randn(g, len(lens), H, d, dtype=dtype)
    n = torch.tensor(lens, dtype=torch.int32)
    qc, tc, nc, mc, pc, xc = [x.cuda() for x in (q, table, n, mass.nan_to_num(0.0, 1.0, 0.0).abs(), pos, nxt)]

    def calls():
        kc, vc = on_gpu(k), on_gpu(v)
        out = list(streamkl_decode(qc, kc, vc, tc, nc, 0.1))
        out += streamkl_decode(qc, kc, vc, tc, nc, 0.1, mass=mc, mass_out=(mo := torch.empty_like(mc)))
        out += streamkl_evict(kc, vc, tc, nc, mo, budget, recent=recent, pos=pc, next_pos=xc)
        assert streamkl_check() == 0
        return [*out, mo, kc, vc]

    want = calls()
    with library(kbuild.build(checked=True)):
        got = calls()
    same(got, want)


@pytest.mark.parametrize("case", DECODE, ids=lambda c: "x".join(str(x) for x in c[:4]) + c[5] + str(len(c[6])))
def test_decode_stays_in_bounds(case):
    H, Hk, d, page, dtype, layout, lens = case
    serve(H, Hk, d, page, dtype, layout, lens, max(1, max(lens) // 3), max(lens) // 9, 310 + H)


@pytest.mark.parametrize("case", EVICT, ids=lambda c: "x".join(str(x) for x in (*c[:3], c[3], len(c[4]), *c[5:])))
def test_evict_stays_in_bounds(case):
    Hk, d, page, layout, lens, budget, recent = case
    serve(2 * Hk, Hk, d, page, BF, layout, lens, budget, recent, 330 + budget)


@pytest.mark.parametrize("lens,page,budget", [((60000, 50001), 128, 20000), ((9000, 3, 8000), 1, 100)],
                         ids=["clusters", "columns"])
def test_long_tables_stay_in_bounds(lens, page, budget):
    serve(3, 1, 64, page, FP, "HND", lens, budget, 50, 350)


@pytest.mark.parametrize("columns", [7, 2000])
def test_bad_input_stays_in_bounds(columns):
    """Bad pages and lengths are reported as such, and lead to no access that the checked build would report."""
    g = gen(360)
    k, v, table = cache(g, (100, 100, 64), 2, 64, 16, BF)
    k, v = k.nan_to_num(1.0).cuda(), v.nan_to_num(1.0).cuda()
    wide = torch.full((3, columns), -9, dtype=torch.int32)
    wide[:, :7] = table
    wide[0, 3], wide[1, 0] = 10 ** 9, -5
    mass, q = torch.rand(3, 2, 112, generator=g).cuda(), randn(g, 3, 4, 64).cuda()
    n = torch.tensor([100, 113, -1], dtype=torch.int32, device="cuda")
    with library(kbuild.build(checked=True)):
        streamkl_decode(q, k, v, wide.cuda(), n, mass=mass)
        streamkl_evict(k, v, wide.cuda(), n, mass, 40)
        with pytest.raises(StreamKLError) as e:
            streamkl_check()
        assert "invalid argument" in str(e.value)             # not an access out of bounds
        assert streamkl_check() == 0
