"""The cache operators at the ends of their documented ranges."""
import ctypes

import pytest
import torch

import attention_kl_divergence_attn_b200 as skl
import cache_ref as ref
from attention_kl_divergence_attn_b200 import streamkl_check, streamkl_decode, streamkl_evict, streamkl_key_mass
from test_cache_gpu import assert_evicted, cache, gen, policy_inputs, randn

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


def ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def longs(*s):
    return (ctypes.c_longlong * len(s))(*s)


@pytest.mark.parametrize("columns", [1, 2000])        # the table looked through, and pages claimed
def test_evict_huge_page_size(columns):
    """A contiguous cache as pages of 2^31 - 1 slots, of which few exist: bad and shared pages are still found."""
    g = gen(200)
    Hk, d, room, page, budget = 2, 64, 128, 2 ** 31 - 1, 40
    lens = (100, 80, 100, 30)
    k, v = randn(g, 2, Hk, room, d), randn(g, 2, Hk, room, d)
    table = torch.full((4, columns), -1, dtype=torch.int32)
    table[:, 0] = torch.tensor([1, 9, 0, 0])              # its own, none, and one page for two
    mass, pos, nxt = policy_inputs(g, 4, Hk, room, lens)
    n = torch.tensor(lens, dtype=torch.int32)
    want = ref.evict(k, v, table[:, :1].clamp(0, 1), n, mass, budget, 5, pos, nxt, skip=(1, 2, 3))
    kc, vc, tc, nc, mc, pc, xc = [x.cuda() for x in (k, v, table, n, mass, pos, nxt)]
    new, m2, p2 = torch.empty_like(nc), torch.empty_like(mc), torch.empty_like(pc)
    L = skl.lib()
    size = L.streamkl_evict_scratch_size(4, Hk, 2, page, columns, room, budget)
    word = torch.zeros(256, dtype=torch.uint8, device="cuda")
    scratch = torch.empty(size, dtype=torch.uint8, device="cuda")
    strides = longs(Hk * room * d, room * d, d)
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    rc = L.streamkl_evict(ptr(kc), strides, ptr(vc), strides, 4, Hk, d, 2, page, ptr(tc), columns, columns, ptr(nc),
                          ptr(mc), ptr(pc), ptr(xc), room, budget, 5, ptr(new), ptr(m2), ptr(p2), ptr(word), 256,
                          ptr(scratch), size, stream)
    assert rc == 0
    code = ctypes.c_uint(0)
    assert L.streamkl_check(ptr(word), stream, ctypes.byref(code)) == 1 and code.value & 0xff == 0b11000
    assert_evicted((new, m2, p2), want, kc, vc)


@pytest.mark.parametrize("H,Hk", [(4, 2), (40, 2), (0, 2)])
@pytest.mark.parametrize("in_place", [False, True])
def test_decode_without_room(H, Hk, in_place):
    """A table without a column: nothing to attend to, and the accumulated weights stay (or are copied) whole."""
    g = gen(201)
    mass = torch.rand(3, Hk, 1500, generator=g)
    mc = mass.cuda()
    mo = mc if in_place else torch.full_like(mc, float("nan"))
    k = randn(g, 2, Hk, 16, 64).cuda()
    out, lse = streamkl_decode(randn(g, 3, H, 64).cuda(), k, k, torch.zeros(3, 0, dtype=torch.int32, device="cuda"),
                               torch.zeros(3, dtype=torch.int32, device="cuda"), 0.1, mass=mc, mass_out=mo)
    assert streamkl_check() == 0
    assert torch.equal(mo.cpu(), mass) and torch.equal(mc.cpu(), mass)
    assert torch.equal(out.cpu(), torch.zeros(3, H, 64, dtype=BF))
    assert torch.equal(lse.cpu(), torch.full((3, H), -float("inf")))


def test_decode_weights_without_a_column():
    """Weights without a column leave no room for a slot, which is not the same as no weights: refused."""
    k = torch.zeros(2, 1, 16, 64, dtype=BF, device="cuda")
    q, n = k[:1, :, 0].contiguous(), torch.full((1,), 5, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        streamkl_decode(q, k, k, torch.zeros(1, 1, dtype=torch.int32, device="cuda"), n,
                        mass=torch.empty(1, 1, 0, device="cuda"))
    streamkl_decode(q, k, k, torch.zeros(1, 0, dtype=torch.int32, device="cuda"), n - 5,
                    mass=torch.empty(1, 1, 0, device="cuda"))
    assert streamkl_check() == 0


def test_key_mass_item_of_millions_of_tiles():
    """2^18 heads of 1024 rows over one key head: every 256 keys take seconds, longer than any other wait may last.

    The heads are windows of one tensor of rows.  Keys of zeros receive a weight of 1 (2^0) from every row, so
    their sums are exact: 2^28, of terms and partial sums that are multiples of 64 below 2^30.
    """
    if torch.cuda.mem_get_info()[0] < 8 << 30:
        pytest.skip("needs 8 GB")
    H, N_Q, d = 1 << 18, 1024, 64
    N_K = 256 * torch.cuda.get_device_properties(0).multi_processor_count
    g = gen(202)
    rows = randn(g, H + N_Q - 1, d)
    q = rows.cuda().as_strided((1, H, N_Q, d), (0, d, d, 1))
    k = torch.zeros(1, 1, N_K, d, dtype=BF)
    k[0, 0, 300, 0] = 2.0
    lse = torch.zeros(1, H, N_Q, device="cuda")
    mass, _ = streamkl_key_mass(q, k.cuda(), lse, 0.125)
    assert streamkl_check() == 0
    got = mass[0, 0].cpu()
    zero = torch.arange(N_K) != 300
    assert torch.equal(got[zero], torch.full((N_K - 1,), float(H * N_Q)))
    # row r is in min(r + 1, N_Q, ...) windows
    times = torch.minimum(torch.arange(1, H + N_Q), torch.arange(H + N_Q - 1, 0, -1)).clamp(max=N_Q).double()
    want = float((times * torch.exp(0.125 * 2.0 * rows[:, 0].double())).sum())
    # a sum of 64 terms a tile half, added H N_Q / 128 times: half a step each
    assert abs(float(got[300]) - want) <= want * (2.0 ** -24 * (H * N_Q / 128 + 64) + 2.0 ** -20)


def test_calls_from_several_threads():
    """Host threads on streams of their own, in shapes that no other call has had: every result as from one thread."""
    from concurrent.futures import ThreadPoolExecutor

    g = gen(203)
    sets = []
    for i in range(4):
        lens = (900 + 37 * i, 13 + i, 450)
        k, v, table = cache(g, lens, 2, 64, 24 + 8 * i, BF)
        q, qq = randn(g, 3, 6, 64), randn(g, 1, 2, 90 + i, 64)
        n, mass = torch.tensor(lens, dtype=torch.int32), torch.rand(3, 2, table.shape[1] * (24 + 8 * i), generator=g)
        sets.append([x.cuda() for x in (q, k.nan_to_num(0.0), v.nan_to_num(0.0), table, n, mass, qq)])

    def work(x):
        q, k, v, table, n, mass, qq = x
        kc, vc = k.clone(), v.clone()
        out = list(streamkl_decode(q, kc, vc, table, n, mass=mass, mass_out=(mo := torch.empty_like(mass))))
        out += streamkl_evict(kc, vc, table, n, mo, 300)[:2]
        out += streamkl_key_mass(qq, qq, causal=True)
        return [*out, mo, kc, vc]

    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()

    def on_stream(i):
        with torch.cuda.stream(streams[i]):
            got = [work(sets[i]) for _ in range(30)]
        streams[i].synchronize()
        return got

    with ThreadPoolExecutor(len(sets)) as pool:
        many = list(pool.map(on_stream, range(len(sets))))
    for x, got in zip(sets, many):
        want = work(x)
        for one in got:
            assert all(torch.equal(a, b) for a, b in zip(one, want))
    assert streamkl_check() == 0
