"""Errors that are smaller than the bounds of cache_ref: decode's products with the values, off by the output's own
rounding and not by one of the weights; fp16 logits of key mass, without a systematic part."""
import math

import pytest
import torch

import cache_ref as ref
from attention_kl_divergence_attn_b200 import streamkl_check, streamkl_decode, streamkl_key_mass
from test_cache_gpu import cache, gen, on_gpu, randn, within

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16

# A weight p is two parts.  hi is truncated from p (1 - s), s = 2^-16 (bf16) or 2^-11 (fp16), which leaves
# lo < p (eps + s), and lo is rounded by half a step: eps / 2 (eps + s), 2^-14.9 or 2^-20.4 of the weight.
SPLIT = {BF: 2.0 ** -8 * (2.0 ** -7 + 2.0 ** -16), FP: 2.0 ** -11 * (2.0 ** -10 + 2.0 ** -11)}


def bound(q, k, v, table, lens, scale):
    """What the output may be off by (cache_ref's terms, the weights' rounding replaced by that of their parts)."""
    B, H, d = q.shape
    page, G = k.shape[2], H // k.shape[1]
    step = torch.finfo(q.dtype).eps / 2
    out = torch.full((B, H, d), torch.finfo(q.dtype).tiny * torch.finfo(q.dtype).eps + 1e-30, dtype=torch.float64)
    for b in range(B):
        n = int(lens[b])
        if n == 0:
            continue
        t = torch.arange(n)
        pg = table[b].long()[t // page]
        for h in range(H):
            kd, vd, qd = k[pg, h // G, t % page].double(), v[pg, h // G, t % page].double(), q[b, h].double()
            y = kd @ qd * scale
            Y = (d + 8) * 2.0 ** -23 * scale * (kd.abs() @ qd.abs())
            l = torch.logsumexp(y, 0)
            w = torch.exp(y - l)
            R = Y + Y.max() + 2.0 ** -22 * (y.abs() + l.abs()) + 2.0 ** -20
            tiny = 2.0 ** -40 if q.dtype == FP else 0.0              # a part below fp16's normal range
            # two products a tile of 16 tokens, each sum a whole step of fp32
            out[b, h] += ((w * (R + SPLIT[q.dtype] + 2.0 ** -23 * (n / 8 + 32))) @ vd.abs()
                          + (w @ vd).abs() * (R.max() + step) + tiny * w.max() * vd.abs().sum(0))
    return out


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens", [(2, 3, 4, 5, 7, 0, 11, 16, 33), (700, 2, 1100, 40)], ids=["short", "split"])
def test_weights_keep_their_bits(lens, d, dtype):
    # a few tokens of like weight whose values nearly cancel: the weights' error is what is left
    g = gen(100 + len(lens) + d)
    k, v, table = cache(g, lens, 2, d, 16, dtype)
    q = randn(g, len(lens), 6, d, dtype=dtype, std=0.5)
    n = torch.tensor(lens, dtype=torch.int32)
    scale = 0.5 / math.sqrt(d)
    want = ref.decode(q, k, v, table, n, scale)
    out, lse = streamkl_decode(*[on_gpu(x) for x in (q, k, v, table, n)], scale)
    assert streamkl_check() == 0
    within(out, want[0], bound(q, k, v, table, n, scale), "out")
    within(lse, want[1], want[4], "lse")


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_infinite_value(sign, dtype):
    # an infinite value of a token with any weight makes its column infinite, and no other
    g = gen(110)
    k, v, table = cache(g, (40, 700), 1, 64, 16, dtype)
    for b, t in ((0, 3), (1, 640)):
        v[table[b, t // 16], 0, t % 16, 5] = sign * math.inf
    q = randn(g, 2, 3, 64, dtype=dtype, std=0.5)
    n = torch.tensor([40, 700], dtype=torch.int32)
    out, _ = streamkl_decode(*[on_gpu(x) for x in (q, k, v, table, n)], 0.1)
    assert streamkl_check() == 0
    assert torch.equal(out[..., 5].float().cpu(), torch.full((2, 3), sign * math.inf))
    other = torch.arange(64) != 5
    want = ref.decode(q, k, v.clamp(-100, 100), table, n, 0.1)
    within(out[..., other.cuda()], want[0][..., other], want[3][..., other], "out")


@pytest.mark.parametrize("d", [64, 128])
def test_fp16_logits_are_not_too_small(d):
    """Key mass of single rows, lse 0: exp(y), off by the logit's error.  Its systematic part, the slope of the error
    over y, is held to the scale's own rounding (2^-24) and a third of the correction for the tensor cores' rounding
    towards zero: (d / 16 + 1) / 2 additions' worth of half a step, 0.36 2^-23 each."""
    g = gen(120 + d)
    q = randn(g, 64, 1, 1, d, dtype=FP)
    k = (randn(g, 64, 1, 4000, d, dtype=FP).float() + q.float()).to(FP)
    scale = float(torch.tensor(1 / math.sqrt(d), dtype=torch.float32))
    y = (q.cuda().double() @ k.cuda().double().transpose(2, 3)).squeeze(2) * scale
    mass, _ = streamkl_key_mass(q.cuda(), k.cuda(), torch.zeros(64, 1, 1, device="cuda"), scale)
    assert streamkl_check() == 0
    err = mass.double() / torch.exp(y) - 1
    slope = float((err * y).sum() / (y * y).sum())
    assert abs(slope) <= 2.0 ** -24 + 0.36 * (d / 16 + 1) / 2 * 2.0 ** -23 / 3, slope
