"""CPU checks of the 4-bit cache, slot, page-table and window calls: what they
refuse on the host, and the references that their GPU tests use."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
import paged_fp8_kv_attn_b200 as pkv
from paged_fp8_kv_attn_b200 import build as pkv_build

import _cache_reference as ref

A = ctypes.c_void_p(256)     # a non-null, aligned address; no call here reaches the device
ODD = ctypes.c_void_p(257)


@pytest.fixture(scope="module")
def lib():
    pkv_build.build()
    return pkv.library()


def _tables(lib, **kw):
    a = dict(old=A, new=A, batch=2, page=16, free=A, cap=4, nf=A, nfo=A, pages=8, table=A, mp=4,
             tags=None, exp=None, slots=A, tokens=8, cu=A, failed=A)
    a.update(kw)
    return lib.kv_extend_tables(a["old"], a["new"], a["batch"], a["page"], a["free"], a["cap"],
                                a["nf"], a["nfo"], a["pages"], a["table"], a["mp"], a["tags"],
                                a["exp"], a["slots"], a["tokens"], a["cu"], a["failed"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(batch=-1), 1), (dict(tokens=-1), 1), (dict(cap=-1), 1), (dict(pages=0), 1),
    (dict(mp=0), 1), (dict(page=48), 3), (dict(page=0), 3), (dict(cap=9), 1),
    (dict(pages=1 << 27, page=16), 3), (dict(tags=A), 1), (dict(exp=A), 1), (dict(old=None), 1),
    (dict(table=None), 1), (dict(failed=None), 1), (dict(free=None), 1), (dict(slots=None), 1),
    (dict(cu=None), 1), (dict(nf=None), 1), (dict(nfo=None), 1), (dict(table=ODD), 1),
    (dict(slots=ctypes.c_void_p(258)), 1),
])
def test_extend_tables_refuses(lib, kw, status):
    assert _tables(lib, **kw) == status, lib.pkv_last_error()


def _write_int4(lib, **kw):
    a = dict(k=A, v=A, ks=128, vs=128, slots=A, t=4, h=2, d=64, page=16, kc=A, kp=A, vc=A, vp=A, np=8)
    a.update(kw)
    return lib.kv_write_slots_int4(a["k"], a["v"], a["ks"], a["vs"], a["slots"], a["t"], a["h"],
                                   a["d"], a["page"], a["kc"], a["kp"], a["vc"], a["vp"], a["np"],
                                   None)


@pytest.mark.parametrize("kw,status", [
    (dict(t=-1), 1), (dict(h=0), 1), (dict(d=96), 3), (dict(page=24), 3), (dict(np=0), 1),
    (dict(np=1 << 30), 3), (dict(ks=120), 1), (dict(vs=132), 1), (dict(k=None), 1),
    (dict(slots=None), 1), (dict(kp=None), 1), (dict(vc=None), 1), (dict(k=ctypes.c_void_p(264)), 1),
    (dict(vp=ctypes.c_void_p(264)), 1), (dict(kc=ODD), 1),
])
def test_slot_calls_refuse(lib, kw, status):
    assert _write_int4(lib, **kw) == status, lib.pkv_last_error()


def test_slot_calls_refuse_scales_and_accept_no_tokens(lib):
    assert lib.kv_write_slots_fp8(A, A, 128, 128, A, 4, 2, 64, 16, 0.0, 1.0, A, A, 8, None) == 1
    assert lib.kv_read_slots_fp8(A, 4, 2, 64, 16, 1.0, float("inf"), A, A, 8, A, A, 128, 128, None) == 1
    assert lib.kv_read_slots_int4(A, 4, 2, 64, 16, A, A, A, None, 8, A, A, 128, 128, None) == 1
    assert lib.kv_write_slots_bf16(None, None, 128, 128, None, 0, 2, 64, 16, None, None, 8, None) == 0
    assert lib.kv_read_slots_int4(None, 0, 2, 64, 16, None, None, None, None, 8, None, None, 128, 128,
                                  None) == 0


def _attn(lib, kind, **kw):
    a = dict(k=A, kp=A, v=A, vp=A, mp=4, b=2, hq=4, h=2, d=64, page=16, np=8, sm=0.1, w=8, s=0,
             ws=A, q=A)
    a.update(kw)
    rest = [A, a["mp"], A, a["b"], a["hq"], a["h"], a["d"], a["page"], a["np"], a["sm"]]
    end = [None, A, A, a["ws"], 1 << 20, 4, None]
    if kind == "int4":
        return lib.paged_decode_attn_int4(a["q"], a["k"], a["kp"], a["v"], a["vp"], *rest, *end)
    if kind == "int4_window":
        return lib.paged_decode_attn_int4_window(a["q"], a["k"], a["kp"], a["v"], a["vp"], *rest,
                                                 a["w"], a["s"], *end)
    if kind == "fp8_window":
        return lib.paged_decode_attn_fp8_window(a["q"], a["k"], a["v"], 1.0, 1.0, *rest, a["w"],
                                                a["s"], *end)
    return lib.paged_decode_attn_bf16_window(a["q"], a["k"], a["v"], *rest, a["w"], a["s"], *end)


@pytest.mark.parametrize("kind", ["int4", "int4_window", "fp8_window", "bf16_window"])
@pytest.mark.parametrize("kw,status", [
    (dict(hq=5), 1), (dict(hq=34), 3), (dict(d=96), 3), (dict(page=8), 3), (dict(mp=0), 1),
    (dict(sm=float("nan")), 1), (dict(q=None), 1), (dict(k=ODD), 1), (dict(ws=None), 2),
    (dict(b=-1), 1),
])
def test_attention_refuses(lib, kind, kw, status):
    assert _attn(lib, kind, **kw) == status, lib.pkv_last_error()


@pytest.mark.parametrize("kind", ["int4", "int4_window"])
def test_int4_attention_refuses_missing_parameters(lib, kind):
    assert _attn(lib, kind, kp=None) == 1
    assert _attn(lib, kind, vp=ctypes.c_void_p(264)) == 1


@pytest.mark.parametrize("kind", ["int4_window", "fp8_window", "bf16_window"])
def test_window_attention_refuses_bad_windows(lib, kind):
    assert _attn(lib, kind, w=0) == 1 and b"window" in lib.pkv_last_error()
    assert _attn(lib, kind, w=-5) == 1
    assert _attn(lib, kind, s=-1) == 1 and b"sinks" in lib.pkv_last_error()


def test_other_int4_calls_refuse(lib):
    assert lib.kv_tag_check_window(A, 8, A, A, 4, A, 2, 16, 0, 0, A, None, None) == 1
    assert lib.kv_tag_check_window(A, 8, A, A, 4, A, 2, 16, 4, -1, A, None, None) == 1
    assert lib.kv_append_int4(A, A, A, 4, A, 2, 2, 96, 16, A, A, A, A, 8, None, None) == 3
    assert lib.kv_append_int4(A, A, A, 4, A, 2, 2, 64, 16, A, None, A, A, 8, None, None) == 1
    assert lib.kv_check_append_int4(A, 8, A, A, 4, A, 2, 16, A, A, 2, 64, A, A, A, ODD, A, None,
                                    None) == 1
    assert lib.kv_requant_pages_int4(A, 8, A, A, None, 8, A, 2, 2, 16, 64, None) == 1
    assert lib.kv_requant_pages_int4(A, 8, A, A, A, 8, A, -1, 2, 16, 64, None) == 1
    assert lib.paged_decode_attn_workspace_size(2, 4, 64, 8, 128, 296) > 0
    assert lib.paged_decode_attn_workspace_size(3, 4, 64, 8, 128, 296) == 0


def test_binding_refuses_host_tensors():
    t = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.kv_extend_tables(t, t, 16, t, t[:1], t.view(4, 1), t, t, t, t[:1], 4)
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.kv_write_slots_bf16(x, x, t, x.view(4, 1, 2, 64), x.view(4, 1, 2, 64))


# ---------------------------------------------------------------------------
# the references themselves
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("seed", range(3))
def test_reference_int4_values(seed):
    """|value - x| is at most half a code step, and the range's ends come back
    within the rounding of s to bf16 (15 codes of 2^-8 of it, and the clamp)."""
    rng = np.random.Generator(np.random.PCG64(seed))
    x = rng.standard_normal((50, 128)) * np.exp(rng.uniform(-30, 30, (50, 1)))
    bits = ref.f32_bits_to_bf16(x.astype(np.float32))
    codes, params = ref.int4_pack(bits)
    back, val = ref.int4_unpack(codes, params), ref.bf16(bits)
    s = np.repeat(ref.bf16(params)[..., 0], 64, axis=-1)
    # half a step; the top value may also fall short by s's rounding, 15 s 2^-8
    assert (np.abs(back - val) <= s * (0.5 + 15 * 2.0 ** -8) * (1 + 1e-6)).all()
    group = val.reshape(50, 2, 64)
    assert np.array_equal(ref.bf16(params)[..., 1], group.min(-1))


def test_reference_int4_specials():
    x = np.zeros((5, 64), np.float32)
    x[1, 3] = np.nan
    x[2, 5] = np.inf
    x[3, 0], x[3, 1] = 3.3e38, -3.3e38
    x[4] = -0.0
    codes, params = ref.int4_pack(ref.f32_bits_to_bf16(x))
    back = ref.int4_unpack(codes, params)
    assert np.array_equal(back[0], np.zeros(64)) and np.array_equal(back[4], np.zeros(64))
    assert np.isnan(back[1:4]).all() and not codes.any()
    assert not params[4].any()      # a zero minimum is +0


def test_reference_attention_against_the_oracle():
    """attend() without a window is the C oracle's attention, to 1e-12."""
    for kind in ("fp8", "bf16"):
        p = ref.Pools(kind, 9, 2, 16, 64, 0.1, 0.2, seed=4)
        rng = np.random.Generator(np.random.PCG64(1))
        table = rng.permutation(9)[:8].reshape(2, 4).astype(np.int32)
        lens = np.array([50, 1], np.int32)
        q = ref.f32_bits_to_bf16(rng.standard_normal((2, 6, 64)).astype(np.float32))
        o, l, _, _ = ref.attend(q, p, table, lens, 0.125)
        ks, vs = (0.1, 0.2) if kind == "fp8" else (1.0, 1.0)
        oo, ol = oracle.paged_decode_attn(q, p.k, p.v, table, lens, 2, 16, 0.125, ks, vs)
        assert np.allclose(o, oo, rtol=1e-12, atol=1e-12) and np.allclose(l, ol, rtol=1e-12)


def test_reference_window_is_a_shorter_request():
    """With a window and no sinks the result is that of the last tokens alone; a
    page that holds none of them does not matter."""
    p = ref.Pools("int4", 6, 1, 16, 64, seed=5)
    rng = np.random.Generator(np.random.PCG64(2))
    q = ref.f32_bits_to_bf16(rng.standard_normal((1, 2, 64)).astype(np.float32))
    table = np.array([[3, 1, 0, 5]], np.int32)
    a = ref.attend(q, p, table, np.array([60]), 0.125, window=12)
    hidden = np.array([[-1, 99, -7, 5]], np.int32)
    b = ref.attend(q, p, hidden, np.array([60]), 0.125, window=12)
    c = ref.attend(q, p, np.array([[5]], np.int32), np.array([12]), 0.125)
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[0], c[0])
    assert np.array_equal(ref.visible(100, 10, 3), [0, 1, 2, *range(90, 100)])
    assert np.array_equal(ref.visible(5, 10, 3), range(5))


def test_reference_tables():
    out = ref.extend_tables([0, 20, 5, 31], [16, 33, 5, 65], 16, [7, 8, 9, 2], 4,
                            np.full((4, 5), -1, np.int32), 10, 70)
    assert out["table"][0, 0] == 2 and out["table"][1, 2] == 9
    # the last request needs 3 pages (entries 2..4), two are left: it fails
    assert out["failed"].tolist() == [0, 0, 0, 1] and out["free"] == 2
    assert out["cu"].tolist() == [0, 16, 29, 29, 63]
    assert out["slots"][:16].tolist() == list(range(32, 48)) and (out["slots"][29:] == -1).all()
    # (request 1's own page was never filled in, so its first 12 tokens have no slot)
    assert (out["slots"][16:28] == -1).all() and out["slots"][28] == 9 * 16
