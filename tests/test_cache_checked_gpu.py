"""Every access of the key-mass kernels through the bounds-checked build: items that runs share, items without a
tile, packed heads, sums added to, log-sum-exps given and computed."""
import random

import pytest
import torch

from attention_kl_divergence_attn_b200 import build as kbuild, streamkl_check, streamkl_key_mass
from test_bounds_gpu import library
from test_cache_gpu import BF, FP, MASS, gen, randn

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
