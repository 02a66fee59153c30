"""Lengths up to 2^31 - 1: page tables of 2^24 entries of 128 tokens a request, of
which the calls read what they use."""
import numpy as np
import pytest
import torch

import paged_fp8_kv_attn_b200 as pkv

import _cache_reference as ref
from test_gpu_cache_ops import KINDS, Cache, bits, cuda, normal_bits, values

pytestmark = pytest.mark.gpu

P, MP = 128, 1 << 24
LENS = (2**31 - 1, 2**31 - 64, 2**31 - 127, 2**31 - 128)


@pytest.fixture(scope="module")
def rows():
    """A page-table row over 30 pages, their tags, and the row's expected tags."""
    rng = np.random.Generator(np.random.PCG64(1))
    table = rng.integers(0, 30, (1, MP)).astype(np.int32)
    tags = rng.integers(0, 2**32, 30, dtype=np.uint64).astype(np.uint32)
    return table, tags, tags[table]


@pytest.mark.parametrize("length", LENS)
@pytest.mark.parametrize("window", [0, 1, 100, 2**31 - 1])
def test_tag_check(cuda_device, rows, length, window):
    table, tags, expected = rows
    g_table, g_tags, g_exp = cuda(table), cuda(tags), cuda(expected)
    lens = torch.tensor([length], dtype=torch.int32, device="cuda")
    abort = torch.full((1,), 9, dtype=torch.uint8, device="cuda")

    def check():
        if window:
            pkv.kv_tag_check_window(g_tags, g_table, g_exp, lens, P, window, 3, abort)
        else:
            pkv.kv_tag_check(g_tags, g_table, g_exp, lens, P, abort)
        return int(abort)

    last = (length - 1) // P
    assert check() == 0
    g_exp[0, last] += 1                   # the entry of the newest token
    assert check() == 1
    g_exp[0, last] -= 1
    g_exp[0, last // 2] += 1              # hidden by a window
    assert check() == (window in (0, 2**31 - 1))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("length", LENS)
def test_check_append_and_expected_tags(cuda_device, rows, kind, length):
    """A stale page aborts the request, whose token is then not written; rebuilt tags let
    it pass."""
    table, tags, expected = rows
    p = ref.Pools(kind, 30, 2, P, 64, 0.1, 0.1, seed=2)
    c = Cache(p)
    rng = np.random.Generator(np.random.PCG64(3))
    k, v = normal_bits(rng, (1, 2, 64)), normal_bits(rng, (1, 2, 64))
    g_table, g_tags, g_exp = cuda(table), cuda(tags), cuda(expected)
    lens = torch.tensor([length], dtype=torch.int32, device="cuda")
    abort = torch.full((1,), 9, dtype=torch.uint8, device="cuda")
    call = getattr(pkv, f"kv_check_append_{kind}")
    g_exp[0, (length - 1) // P] += 1
    args = (g_tags, g_table, g_exp, lens, P, cuda(k), cuda(v), *c.scales, *c.pools, abort)
    call(*args)
    assert int(abort) == 1
    c.same(p)
    pkv.kv_expected_tags(g_tags, g_table, lens, P, g_exp)
    call(*args)
    assert int(abort) == 0
    p.write([table[0, (length - 1) // P] * P + (length - 1) % P], k, v)
    c.same(p)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("G,H,D", [(4, 2, 128), (2, 1, 64)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (100, 5), (700, 300)])
def test_window_attention(cuda_device, rows, kind, G, H, D, window, sinks):
    """The same as a request of the sinks' pages and the window's alone."""
    table = rows[0]
    p = ref.Pools(kind, 30, H, P, D, 0.1, 0.1, seed=4)
    c = Cache(p)
    rng = np.random.Generator(np.random.PCG64(5))
    q = normal_bits(rng, (len(LENS), H * G, D))
    short = np.stack([np.concatenate([table[0, :4], table[0, (n - 1) // P - 8:][:9]]) for n in LENS])
    short_lens = np.array([12 * P + (n - 1) % P + 1 for n in LENS], np.int32)
    want = ref.attend(q, p, short, short_lens, 0.1, window, sinks)
    gq, gt = cuda(q), cuda(np.repeat(table, len(LENS), 0))
    gl = cuda(np.array(LENS, np.int32))
    for n in (0, 1, 40, -2):
        ws = c.workspace(len(LENS), H * G, n)
        out, lse = c.attend(gq, gt, gl, 0.1, ws, window, sinks, num_ctas=n)
        torch.cuda.synchronize()
        assert pkv.workspace_status(ws) == 0
        ref.check_attention(values(out), values(lse), want, f"ctas={n}")
        # a visible page that is none kills its request only
        gt[1, (LENS[1] - 1) // P] = 30
        out, lse = c.attend(gq, gt, gl, 0.1, ws, window, sinks, num_ctas=n)
        torch.cuda.synchronize()
        gt[1, (LENS[1] - 1) // P] = int(table[0, (LENS[1] - 1) // P])
        assert not out[1].any() and torch.isneginf(lse[1]).all()
        live = [0, 2, 3]
        ref.check_attention(values(out)[live], values(lse)[live], [x[live] for x in want], f"ctas={n}")
