"""Outputs of the cache operators that overlap an input or another output are refused, in the C ABI and the binding."""
import ctypes

import pytest
import torch

import attention_kl_divergence_attn_b200 as skl
from attention_kl_divergence_attn_b200 import (build as kbuild, streamkl_check, streamkl_decode, streamkl_evict,
                                               streamkl_key_mass)
from test_cache_args import decode, evict, mass, strides

BF = torch.bfloat16
# The C calls below have addresses that nothing lies at, so no call that might be accepted may meet a GPU.
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="addresses of nothing: only where no kernel can run")


@pytest.fixture(scope="module")
def L():
    kbuild.build()
    return skl.lib()


def apart(*names):
    """Addresses a gigabyte apart."""
    return {n: (i + 1) << 30 for i, n in enumerate(names)}


MASS = apart("q", "k", "kv", "lse", "mass")
DECODE = dict(apart("q", "k", "v", "table", "len", "out", "lse", "mass", "mo"), cap=32)
EVICT = apart("k", "v", "table", "len", "mass", "pos", "nxt", "new", "mo", "po")
# bytes of each tensor for the sizes of test_cache_args
SIZE = {"mass": dict(q=4 * 8 * 128, k=2 * 9 * 128, kv=4, lse=4 * 32, mass=4 * 18),
        "decode": dict(q=2 * 4 * 128, k=3 * 2 * 16 * 128, v=3 * 2 * 16 * 128, table=16, len=8, out=2 * 4 * 128,
                       lse=32, mass=4 * 2 * 2 * 32, mo=4 * 2 * 2 * 32),
        "evict": dict(k=3 * 2 * 16 * 128, v=3 * 2 * 16 * 128, table=16, len=8, mass=4 * 4 * 32, pos=4 * 4 * 32, nxt=8,
                      new=8, mo=4 * 4 * 32, po=4 * 4 * 32)}
CALL = {"mass": (mass, MASS), "decode": (decode, DECODE), "evict": (evict, EVICT)}
PAIRS = ([("mass", "mass", x) for x in ("q", "k", "kv", "lse")] + [("mass", "lse", x) for x in ("q", "k", "kv")]
         + [("decode", o, x) for o in ("out", "lse", "mo") for x in ("q", "k", "v", "table", "len", "mass", "out", "lse")
            if o != x]
         + [("evict", o, x) for o in ("new", "mo", "po")
            for x in ("k", "v", "table", "len", "mass", "pos", "nxt", "new", "mo") if o != x]
         + [("evict", o, x) for o in ("k", "v") for x in ("table", "len", "mass", "pos", "nxt")])


@no_gpu
@pytest.mark.parametrize("op,out,other", PAIRS, ids="-".join)
def test_overlap_is_refused(L, op, out, other):
    call, at = CALL[op]
    size = SIZE[op]
    ok = call(L, **at)
    assert ok not in (0, 1, 5)                          # no device
    align = 16 if out in ("q", "k", "v", "out") else 4
    # the output's start on the other's last bytes, its end on the other's first, and one past each
    last = (size[other] - 1) // align * align
    assert call(L, **{**at, out: at[other] + last}) == 1
    assert call(L, **{**at, out: at[other] - (size[out] - 1) // align * align}) == 1
    up = lambda n: -(-n // align) * align
    assert call(L, **{**at, out: at[other] + up(size[other])}) == ok
    assert call(L, **{**at, out: at[other] - up(size[out])}) == ok


@no_gpu
def test_what_may_lie_together(L):
    ok = mass(L, **MASS)
    assert mass(L, **{**MASS, "q": MASS["k"]}) == ok                               # inputs
    assert mass(L, **{**MASS, "given": 1, "kv": MASS["lse"]}) == ok
    assert decode(L, **{**DECODE, "mo": DECODE["mass"]}) == ok                     # in place
    assert decode(L, **{**DECODE, "k": DECODE["v"]}) == ok
    pages = strides(2 * 2 * 16 * 64, 16 * 64, 64)                                  # keys and values page by page
    at = {**EVICT, "v": EVICT["k"] + 2 * 16 * 128}
    assert evict(L, **{**at, "ks": pages, "vs": pages}) == ok


@no_gpu
def test_spans_follow_the_strides(L):
    # the last of B = 2 rows of the table, of 3 pages far apart, of 4 heads far apart
    far = 1 << 26
    ok = decode(L, **DECODE)
    assert decode(L, **{**DECODE, "ts": far, "lse": DECODE["table"] + 4 * far + 4}) == 1
    assert decode(L, **{**DECODE, "ts": far, "lse": DECODE["table"] + 4 * far + 8}) == ok
    s = strides(far, 16 * 64, 64)
    end = 2 * (2 * far + 2 * 16 * 64)
    assert decode(L, **{**DECODE, "ks": s, "lse": DECODE["k"] + end - 4}) == 1
    assert decode(L, **{**DECODE, "ks": s, "lse": DECODE["k"] + end}) == ok
    s = strides(8, far, 64)                                                        # (a batch of one has no stride)
    end = 2 * (3 * far + 8 * 64)
    assert mass(L, **{**MASS, "qs": s, "mass": MASS["q"] + end - 4}) == 1
    assert mass(L, **{**MASS, "qs": s, "mass": MASS["q"] + end}) == ok
    # strides as large as any, whose end is past the address space
    s = strides(1 << 38, 1 << 38, 1 << 38)
    assert decode(L, **{**DECODE, "pages": 1 << 30, "ks": s, "lse": 1 << 62}) == 1


@pytest.mark.gpu
def test_binding_names_overlaps():
    """Each combination that the binding lets through to the library comes back as a ValueError, and nothing ran."""
    dev = "cuda"
    k = torch.randn(2, 2, 16, 64, device=dev).to(BF)
    v = k.clone()
    q = torch.randn(1, 4, 64, device=dev).to(BF)
    table, n = torch.tensor([[0, 1]], dtype=torch.int32, device=dev), torch.tensor([20], dtype=torch.int32, device=dev)
    o, lse = torch.empty(1, 4, 64, dtype=BF, device=dev), torch.empty(1, 4, device=dev)
    mass = torch.rand(1, 2, 32, device=dev)

    def flat(t, dtype, *shape):
        return t.view(-1).view(dtype)[:torch.Size(shape).numel()].view(shape)

    for out in ((flat(k, BF, 1, 4, 64), lse), (flat(v, BF, 1, 4, 64), lse), (o, flat(o, torch.float32, 1, 4)),
                (o, flat(mass, torch.float32, 1, 4)), (o, flat(k, torch.float32, 1, 4))):
        with pytest.raises(ValueError):
            streamkl_decode(q, k, v, table, n, mass=mass, out=out)
    for out in ((None, None), (o, None), (None, lse)):
        with pytest.raises(ValueError):
            streamkl_decode(q, k, v, table, n, out=out)
    for other in (k, v, q):
        with pytest.raises(ValueError):
            streamkl_decode(q, k, v, table, n, mass=mass, mass_out=flat(other, torch.float32, 1, 2, 32)[:, :, :32])
    with pytest.raises(ValueError):                               # in place, on the keys
        streamkl_decode(q, k, v, table, n, mass=flat(k, torch.float32, 1, 2, 32))
    pos, nxt = torch.zeros(1, 2, 32, dtype=torch.int32, device=dev), torch.tensor([20], dtype=torch.int32, device=dev)
    new, m2, p2 = torch.empty_like(n), torch.empty_like(mass), torch.empty_like(pos)
    for out in ((flat(p2, torch.int32, 1), m2, p2), (new, flat(k, torch.float32, 1, 2, 32), p2),
                (new, m2, flat(v, torch.int32, 1, 2, 32)), (new, m2, flat(m2, torch.int32, 1, 2, 32)),
                (flat(table, torch.int32, 1), m2, p2)):
        with pytest.raises(ValueError):
            streamkl_evict(k, v, table, n, mass, 8, pos=pos, next_pos=nxt, out=out)
    with pytest.raises(ValueError):
        streamkl_evict(k, v, table, n, flat(v, torch.float32, 1, 2, 32), 8)
    qq, kk = torch.randn(1, 2, 8, 64, device=dev).to(BF), torch.randn(1, 2, 8, 64, device=dev).to(BF)
    for other in (qq, kk):
        with pytest.raises(ValueError):
            streamkl_key_mass(qq, kk, out=flat(other, torch.float32, 1, 2, 8))
    assert streamkl_check() == 0
    # and what only looks close is taken
    both = torch.randn(2, 2, 2, 16, 64, device=dev).to(BF)         # a page's keys, then its values
    streamkl_evict(both[:, 0], both[:, 1], table, n, mass, 8, pos=pos, next_pos=nxt, out=(new, m2, p2))
    streamkl_decode(q, both[:, 0], both[:, 1], table, new, mass=m2, out=(o, lse))
    assert streamkl_check() == 0
