"""GPU accuracy of attention over the 4-bit cache, per query head and group of 64
dims: V scales that differ between groups, heads and tokens, scores that rise late,
and long requests, within the bounds of _int4_bound."""
import numpy as np
import pytest
import torch

import paged_fp8_kv_attn_b200 as pkv

import _cache_reference as ref
import _int4_bound as tight
from test_gpu_cache_ops import Cache, attention_case, cuda, values

pytestmark = pytest.mark.gpu

# G, H, D, P: every compiled form (one and two KV heads an item, groups past 8)
SHAPES = [(8, 2, 128, 64), (4, 2, 128, 16), (7, 1, 128, 32), (12, 1, 128, 16), (8, 2, 64, 16),
          (3, 2, 64, 128), (5, 1, 64, 64), (16, 1, 64, 32)]


def scaled(bits, k):
    """bf16 bits times 2^k."""
    return ref.f32_bits_to_bf16((ref.bf16(bits) * 2.0 ** k).astype(np.float32))


def set_key(p, table, b, t, value, head=slice(None)):
    """Token t of request b: every dim of K is `value`."""
    P = p.shape[2]
    at = table[b, t // P], head, t % P
    p.k[at] = 0
    p.kp[at] = 0
    p.kp[at + (slice(None), 1)] = ref.f32_bits_to_bf16(np.float32(value))


def raise_scale(p, table, b, t, k, group=slice(None)):
    """Token t of request b: V's scale and minimum times 2^k."""
    P = p.shape[2]
    at = table[b, t // P], slice(None), t % P, group
    p.vp[at] = scaled(p.vp[at], k)


def run(p, q, table, lens, sm, label, window=0, sinks=0, ctas=(0, 1, 7, -2)):
    c = Cache(p)
    B, Hq, D = q.shape
    want = tight.attend(q, p, table, lens, sm, window, sinks)
    for n in ctas:
        ws = c.workspace(B, Hq, n)
        out, lse = c.attend(cuda(q), cuda(table), cuda(lens), sm, ws, window, sinks, num_ctas=n)
        torch.cuda.synchronize()
        assert pkv.workspace_status(ws) == 0
        w = tight.check(values(out), values(lse), want, f"{label} ctas={n}")
        print(f"{label} ctas={n}: {w[0]:.3f} {w[1]:.3f}")


@pytest.mark.parametrize("G,H,D,P", SHAPES)
def test_drawn_values(cuda_device, G, H, D, P):
    p, q, table, lens = attention_case("int4", [1, 64, 65, 700, 333], G, H, D, P, seed=31)
    run(p, q, table, lens, D ** -0.5, "drawn")
    run(p, q, table, lens, D ** -0.5, "window", window=70, sinks=9)


@pytest.mark.parametrize("G,H,D,P", SHAPES)
@pytest.mark.parametrize("k", [10, 20, 40])
def test_a_scale_that_no_weight_falls_on(cuda_device, G, H, D, P, k):
    """One token, first, in the middle or last, whose V scale is 2^k times the others' and
    whose weight is e^-60 of them or less: the others keep their bits."""
    n = 513
    p, q, table, lens = attention_case("int4", [n] * 4, G, H, D, P, seed=32)
    q = ref.f32_bits_to_bf16(np.abs(ref.bf16(q)).astype(np.float32))      # query sums well above 0
    sm = D ** -0.5
    low = ref.bf16(q).sum(-1).min(-1) * sm
    for b, t in enumerate((0, 200, n - 1, 63)):
        set_key(p, table, b, t, -100.0 / low[b])
        raise_scale(p, table, b, t, k)
    run(p, q, table, lens, sm, f"2^{k}")


@pytest.mark.parametrize("G,H,P", [(8, 2, 64), (3, 1, 16), (11, 1, 32)])
@pytest.mark.parametrize("k", [-20, 20, 40])
def test_groups_of_different_scale(cuda_device, G, H, P, k):
    """The last 64 dims of every V row 2^k times the first 64."""
    p, q, table, lens = attention_case("int4", [300, 65, 1, 900], G, H, 128, P, seed=33)
    p.vp[..., 1, :] = scaled(p.vp[..., 1, :], k)
    run(p, q, table, lens, 0.09, f"2^{k}")
    run(p, q, table, lens, 0.09, f"2^{k} window", window=130, sinks=3)


@pytest.mark.parametrize("G,H,D,P", SHAPES)
def test_heads_with_weights_on_different_scales(cuda_device, G, H, D, P):
    """Even query heads put their weight on a token of a V scale of 2^24, the odd ones none."""
    p, q, table, lens = attention_case("int4", [400, 700], G, H, D, P, seed=34)
    x = np.abs(ref.bf16(q))
    x[:, 1::2] *= -1.0
    q = ref.f32_bits_to_bf16(x.astype(np.float32))
    sm = D ** -0.5
    for b, t in enumerate((130, 699)):
        set_key(p, table, b, t, 120.0 / (x[b].sum(-1)[0::2].min() * sm))
        raise_scale(p, table, b, t, 24)
    run(p, q, table, lens, sm, "heads")


@pytest.mark.parametrize("G,H,D,P", SHAPES)
@pytest.mark.parametrize("jump", [11.0, 40.0, 150.0, 700.0])
def test_scores_that_rise_late(cuda_device, G, H, D, P, jump):
    """The last 3 tokens' scores are far above the others', their V scales 2^-24 of them."""
    p, q, table, lens = attention_case("int4", [500, 130], G, H, D, P, seed=35)
    q = ref.f32_bits_to_bf16(np.abs(ref.bf16(q)).astype(np.float32))
    sm = D ** -0.5
    sums = ref.bf16(q).sum(-1) * sm
    for b in range(2):
        for t in range(lens[b] - 3):
            raise_scale(p, table, b, t, 24)
        for t in range(lens[b] - 3, lens[b]):
            set_key(p, table, b, t, (jump + 40.0) / sums[b].min())
    run(p, q, table, lens, sm, f"jump {jump}")


@pytest.mark.parametrize("G,H,D,P", [(8, 2, 128, 64), (5, 1, 64, 16)])
def test_long_request(cuda_device, G, H, D, P):
    """40,001 tokens over several splits, and a window with sinks over most of them.  The
    tokens at the window's and the sinks' edges, those in front of and behind them
    (hidden) and the last one score far above the rest, e^10 and e^20 of it: an edge that
    is off by one token, or a part of a split that is lost or counted twice, passes
    neither bound."""
    n, window, sinks = 40001, 30011, 100
    p, q, table, lens = attention_case("int4", [n], G, H, D, P, seed=36)
    q = ref.f32_bits_to_bf16(np.abs(ref.bf16(q)).astype(np.float32))
    sm = D ** -0.5
    one = 1.0 / (ref.bf16(q).sum(-1).mean() * sm)      # the key of a score of about 1
    for t in range(n):
        set_key(p, table, 0, t, 0.5 * one)
    for t in (0, sinks - 1, n - window, n - 1):
        set_key(p, table, 0, t, 10 * one)
    run(p, q, table, lens, sm, "long", ctas=(0, 148, 296, -16))
    for t in (sinks, n - window - 1):
        set_key(p, table, 0, t, 20 * one)
    run(p, q, table, lens, sm, "long window", window=window, sinks=sinks, ctas=(0, 296, -8))
    good = tight.attend(q, p, table, lens, sm, window, sinks)
    for w, s in ((window + 1, sinks), (window - 1, sinks), (window, sinks + 1), (window, sinks - 1)):
        o, l, _, _ = tight.attend(q, p, table, lens, sm, w, s)
        with pytest.raises(AssertionError):
            tight.check(o, good[1], good)
        with pytest.raises(AssertionError):
            tight.check(good[0], l, good)


@pytest.mark.parametrize("G,H,D,P", SHAPES)
@pytest.mark.parametrize("at", [0, 70, 299])
def test_the_only_weighted_token_comes_back(cuda_device, G, H, D, P, at):
    """One token, first or late, with all the weight (the others have e^-50 of it at most):
    its weight is 1 and rounds to nothing, so an output is its value to 2^-20 of its two
    parts, and the half step of bf16."""
    n = 300
    p, q, table, lens = attention_case("int4", [n] * 3, G, H, D, P, seed=37)
    q = ref.f32_bits_to_bf16(np.abs(ref.bf16(q)).astype(np.float32))
    sm = D ** -0.5
    sums = ref.bf16(q).sum(-1) * sm
    for b in range(3):
        set_key(p, table, b, at, (110.0 + 0.37 * b) / sums[b].min())
    c = Cache(p)
    _, a, m = p.rows("v", table[:, at // P], np.full(3, at % P))
    want = np.repeat((a + m).reshape(3, H, 1, D), G, 2).reshape(3, H * G, D)
    parts = np.repeat((np.abs(a) + np.abs(m)).reshape(3, H, 1, D), G, 2).reshape(3, H * G, D)
    half = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(want), 2.0 ** -126))) - 8)
    for ctas in (0, 1, 7, -2):
        ws = c.workspace(3, H * G, ctas)
        out, _ = c.attend(cuda(q), cuda(table), cuda(lens), sm, ws, num_ctas=ctas)
        err = np.abs(values(out) - want)
        assert (err <= half + 2.0 ** -20 * parts).all(), (ctas, (err / (half + 2.0 ** -20 * parts)).max())
