"""The cache operators' refusals, and their 64-bit forms against torch's own softmax (no GPU needed)."""
import ctypes
import math

import pytest
import torch

import cache_ref as ref
from attention_kl_divergence_attn_b200 import (build as kbuild, streamkl_decode, streamkl_evict, streamkl_key_mass)


@pytest.fixture(scope="module")
def L():
    kbuild.build()
    import attention_kl_divergence_attn_b200 as skl
    return skl.lib()


def p(x=16):
    return ctypes.c_void_p(x) if x else None


def strides(*s):
    return (ctypes.c_longlong * len(s))(*s)


def mass(L, **kw):
    a = dict(q=16, qs=None, k=16, ks=None, dtype=0, B=1, H=4, Hk=2, N_Q=8, N_K=9, d=64, scale=0.1, causal=0, kv=0,
             lse=16, given=0, mass=16, acc=0, ws=16, wsb=256, sc=16, scb=1 << 30)
    a.update(kw)
    return L.streamkl_key_mass(p(a["q"]), a["qs"], p(a["k"]), a["ks"], a["dtype"], a["B"], a["H"], a["Hk"], a["N_Q"],
                               a["N_K"], a["d"], a["scale"], a["causal"], p(a["kv"]), p(a["lse"]), a["given"],
                               p(a["mass"]), a["acc"], p(a["ws"]), a["wsb"], p(a["sc"]), a["scb"], None)


def decode(L, **kw):
    a = dict(q=16, qs=None, k=16, ks=None, v=16, vs=None, dtype=0, B=2, H=4, Hk=2, d=64, pages=3, page=16, table=16,
             maxp=2, ts=2, len=16, scale=0.1, out=16, lse=16, mass=0, mo=0, cap=0, ws=16, wsb=256, sc=16,
             scb=1 << 30)
    a.update(kw)
    return L.streamkl_decode(p(a["q"]), a["qs"], p(a["k"]), a["ks"], p(a["v"]), a["vs"], a["dtype"], a["B"], a["H"],
                             a["Hk"], a["d"], a["pages"], a["page"], p(a["table"]), a["maxp"], a["ts"], p(a["len"]),
                             a["scale"], p(a["out"]), p(a["lse"]), p(a["mass"]), p(a["mo"]), a["cap"], p(a["ws"]),
                             a["wsb"], p(a["sc"]), a["scb"], None)


def evict(L, **kw):
    a = dict(k=16, ks=None, v=32, vs=None, B=2, Hk=2, d=64, pages=3, page=16, table=16, maxp=2, ts=2, len=16, mass=48,
             pos=64, nxt=80, cap=32, budget=16, recent=4, new=96, mo=112, po=128, ws=16, wsb=256, sc=16,
             scb=1 << 30)
    a.update(kw)
    return L.streamkl_evict(p(a["k"]), a["ks"], p(a["v"]), a["vs"], a["B"], a["Hk"], a["d"], a["pages"], a["page"],
                            p(a["table"]), a["maxp"], a["ts"], p(a["len"]), p(a["mass"]), p(a["pos"]), p(a["nxt"]),
                            a["cap"], a["budget"], a["recent"], p(a["new"]), p(a["mo"]), p(a["po"]), p(a["ws"]),
                            a["wsb"], p(a["sc"]), a["scb"], None)


COMMON = [(dict(ws=0), 5), (dict(wsb=255), 5), (dict(ws=20), 1), (dict(d=96), 2), (dict(d=256), 2), (dict(B=-1), 1),
          (dict(Hk=0), 1), (dict(k=24), 1)]


@pytest.mark.parametrize("kw,rc", COMMON + [
    (dict(H=3), 1), (dict(dtype=2), 1), (dict(causal=2), 1), (dict(causal=1, N_Q=10), 1), (dict(N_K=0), 1),
    (dict(scale=0.0), 1), (dict(scale=math.inf), 1), (dict(scale=math.nan), 1), (dict(lse=0), 1), (dict(mass=0), 1),
    (dict(mass=18), 1), (dict(lse=18), 1), (dict(kv=18), 1), (dict(given=2), 1), (dict(acc=2), 1), (dict(q=0), 1),
    (dict(q=24), 1), (dict(sc=20), 1), (dict(N_Q=1 << 25), 1), (dict(sc=0), 5), (dict(scb=100), 5), (dict(qs=strides(4096, 512, 60)), 1),
    (dict(ks=strides(1, 0, 64)), 1), (dict(ks=strides(1, 576, -64)), 1)])
def test_key_mass_refusals(L, kw, rc):
    assert mass(L, **kw) == rc


@pytest.mark.parametrize("kw,rc", COMMON + [
    (dict(H=3), 1), (dict(dtype=2), 1), (dict(scale=0.0), 1), (dict(scale=math.inf), 1), (dict(page=0), 1),
    (dict(maxp=-1), 1), (dict(pages=-1), 1), (dict(q=0), 1), (dict(v=0), 1), (dict(v=24), 1), (dict(len=0), 1),
    (dict(len=18), 1), (dict(table=0), 1), (dict(table=18), 1), (dict(out=0), 1), (dict(out=24), 1), (dict(lse=0), 1),
    (dict(lse=18), 1), (dict(mass=16), 1), (dict(mo=16), 1), (dict(mass=18, mo=32, cap=32), 1), (dict(cap=-1), 1),
    (dict(sc=0, maxp=99), 5), (dict(scb=100, maxp=99), 5), (dict(sc=20), 1), (dict(ts=-1), 1),
    (dict(qs=strides(256, 60)), 1),
    (dict(ks=strides(2048, 1024, 0)), 1), (dict(vs=strides(2048, -1024, 64)), 1)])
def test_decode_refusals(L, kw, rc):
    assert decode(L, **kw) == rc


@pytest.mark.parametrize("kw,rc", COMMON + [
    (dict(budget=-1), 1), (dict(recent=-1), 1), (dict(recent=17), 1), (dict(pos=0), 1), (dict(nxt=0), 1),
    (dict(po=0), 1), (dict(pos=0, recent=0), 1), (dict(len=0), 1), (dict(new=0), 1), (dict(new=16, len=16), 1),
    (dict(mass=0), 1), (dict(mo=0), 1), (dict(mo=48), 1), (dict(po=64), 1), (dict(cap=-1), 1), (dict(sc=0), 5),
    (dict(scb=16), 5), (dict(cap=1 << 22, page=1 << 16, maxp=64), 2), (dict(table=0), 1), (dict(ts=-1), 1), (dict(v=16), 1), (dict(mass=50), 1), (dict(pos=66), 1),
    (dict(ks=strides(2048, 1024, 60)), 1)])
def test_evict_refusals(L, kw, rc):
    assert evict(L, **kw) == rc


def test_nothing_to_do_needs_no_device(L):
    assert mass(L, B=0, mass=0, lse=0, q=0, k=0) == 0
    assert decode(L, B=0) == 0 and decode(L, H=0, Hk=1) == 0
    assert evict(L, B=0) == 0


def test_binding_refuses_cpu_tensors_and_bad_types():
    q, k = torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16), torch.zeros(1, 1, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        streamkl_key_mass(q, k)
    t, n = torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(TypeError):
        streamkl_decode(q[:, :, 0], k, k, t, n)
    with pytest.raises(TypeError):
        streamkl_evict(k, k, t, n, torch.zeros(1, 1, 4), 2)
    with pytest.raises(TypeError):
        streamkl_key_mass([[1.0]], k)
    with pytest.raises(TypeError):
        streamkl_key_mass(q.float(), k)


# ---------------------------------------------------------- the 64-bit forms
def test_reference_key_mass_against_softmax():
    g = torch.Generator().manual_seed(0)
    q, k = torch.randn(2, 4, 5, 64, generator=g), torch.randn(2, 2, 7, 64, generator=g)
    m, lse, _, _ = ref.key_mass(q, k, 0.3, True)
    x = torch.einsum("bhid,bhjd->bhij", q.double(), k.double().repeat_interleave(2, 1)) * 0.3
    x = x.masked_fill(torch.ones(5, 7).triu(3).bool(), -math.inf)
    torch.testing.assert_close(m, torch.softmax(x, -1).sum(2).view(2, 2, 2, 7).sum(2))
    torch.testing.assert_close(lse, torch.logsumexp(x, -1))


def test_reference_decode_is_attention_of_the_last_row():
    g = torch.Generator().manual_seed(1)
    kp, vp = torch.randn(6, 2, 4, 64, generator=g), torch.randn(6, 2, 4, 64, generator=g)
    table = torch.tensor([[3, 1, 5]])
    q = torch.randn(1, 4, 64, generator=g)
    o, lse, m, _, _, _ = ref.decode(q, kp, vp, table, [10], 0.2, torch.zeros(1, 2, 12))
    k = kp[[3, 1, 5]].transpose(0, 1).reshape(2, 12, 64)[:, :10].double().repeat_interleave(2, 0)
    v = vp[[3, 1, 5]].transpose(0, 1).reshape(2, 12, 64)[:, :10].double().repeat_interleave(2, 0)
    x = torch.einsum("hd,htd->ht", q[0].double(), k) * 0.2
    w = torch.softmax(x, -1)
    torch.testing.assert_close(o[0], torch.einsum("ht,htd->hd", w, v))
    torch.testing.assert_close(lse[0], torch.logsumexp(x, -1))
    torch.testing.assert_close(m[0, :, :10], w.view(2, 2, 10).sum(1))


def test_reference_eviction_by_hand():
    m = torch.tensor([0.5, 2.0, 0.1, 2.0, 0.1, 9.0, math.nan, 0.3])
    pos = torch.tensor([0, 1, 2, 3, 4, 5, 6, 7])
    # newest: 7; then 9.0, 2.0 (slot 1), 2.0 (slot 3): of the first four slots 0 and 2 are free, 5 and 7 move there
    assert ref.evict_slots(m, pos, 8, 4, 1, 8) == [5, 1, 7, 3]
    assert ref.evict_slots(m, pos, 8, 4, 0, 8) == [0, 1, 5, 3]
    assert ref.evict_slots(m, pos, 3, 4, 0, 8) == [0, 1, 2]
