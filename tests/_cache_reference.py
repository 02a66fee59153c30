"""Plain 64-bit restatements of the cache operators, for their tests: the 4-bit
format, token writes and reads by slot, page tables from lengths, and decode
attention over a list of visible tokens.  numpy only; no code of the library.
"""
from __future__ import annotations

import numpy as np

import oracle

GROUP = 64
BF16_STEP, F16_STEP, F32_STEP = 2.0 ** -8, 2.0 ** -11, 2.0 ** -24   # half a step, relative


def f32_bits_to_bf16(x):
    """bf16 bit patterns of binary32 values, round to nearest even (NaN: 0x7FC0)."""
    u = np.asarray(x, np.float32).view(np.uint32).astype(np.uint64)
    r = ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)
    return np.where(np.isnan(x), np.uint16(0x7FC0), r)


def bf16(bits):
    return oracle.bf16_to_double(bits)


# ---------------------------------------------------------------------------
# the 4-bit format
# ---------------------------------------------------------------------------

def int4_pack(bits):
    """bf16 bits [..., D] -> (codes uint8 [..., D/2], params bf16 bits [..., D/64, 2])."""
    x = bf16(bits).astype(np.float32)
    x = x.reshape(*x.shape[:-1], -1, GROUP)
    with np.errstate(all="ignore"):
        lo, hi = x.min(-1), x.max(-1)
        lo = lo + np.float32(0)
        r = (hi - lo).astype(np.float32) + np.float32(0)
        bad = ~np.isfinite(x).all(-1) | ~np.isfinite(r)
        s_bits = f32_bits_to_bf16((r / np.float32(15)).astype(np.float32))
        s = bf16(s_bits).astype(np.float32)
        q = (x - lo[..., None]).astype(np.float32) / np.where(s == 0, np.float32(1), s)[..., None]
        code = np.minimum(np.rint(q.astype(np.float32)), 15)
    code = np.where((bad | (s == 0))[..., None], 0, code).astype(np.uint8)
    code = code.reshape(*code.shape[:-2], -1)
    nan = np.uint16(0x7FC0)
    params = np.stack([np.where(bad, nan, s_bits), np.where(bad, nan, f32_bits_to_bf16(lo))], -1)
    return code[..., 0::2] | (code[..., 1::2] << 4), params.astype(np.uint16)


def int4_split(codes, params):
    """(s * code, m) as fp64 [..., D]: the value is their sum."""
    n = np.empty((*codes.shape[:-1], 2 * codes.shape[-1]))
    n[..., 0::2], n[..., 1::2] = codes & 15, codes >> 4
    p = np.repeat(bf16(params), GROUP, axis=-2)
    return n * p[..., 0], p[..., 1]


def int4_unpack(codes, params):
    a, m = int4_split(codes, params)
    return a + m


# ---------------------------------------------------------------------------
# slots
# ---------------------------------------------------------------------------

class Pools:
    """The K and V pools of one cache on the host.  kind: fp8, bf16 or int4."""

    def __init__(self, kind, num_pages, heads, page, dim, k_scale=1.0, v_scale=1.0, seed=0):
        rng = np.random.Generator(np.random.PCG64(seed))
        self.kind, self.shape = kind, (num_pages, heads, page, dim)
        self.k_scale, self.v_scale = k_scale, v_scale
        self.k, self.kp = self._fill(rng)
        self.v, self.vp = self._fill(rng)

    def _fill(self, rng):
        x = rng.standard_normal(self.shape)
        x[rng.random(self.shape) < 0.01] *= 20.0
        bits = f32_bits_to_bf16(x.astype(np.float32))
        return self._pack(bits, self.k_scale)

    def _pack(self, bits, scale):
        if self.kind == "int4":
            return int4_pack(bits)
        return (oracle.quantize_bf16(np.ascontiguousarray(bits), scale) if self.kind == "fp8"
                else bits), None

    def write(self, slot_map, k_bits, v_bits):
        NP, _, P, _ = self.shape
        for i, s in enumerate(np.asarray(slot_map)):
            if not 0 <= s < NP * P:
                continue
            for x, p, bits, scale in ((self.k, self.kp, k_bits, self.k_scale),
                                      (self.v, self.vp, v_bits, self.v_scale)):
                a, b = self._pack(bits[i], scale)
                x[s // P, :, s % P] = a
                if p is not None:
                    p[s // P, :, s % P] = b

    def rows(self, which, pages, offs):
        """fp64 [T][Hkv][D] values, and the part of them that weights multiply in the
        V product (INT4: s * code; otherwise the values)."""
        x, p, scale = ((self.k, self.kp, self.k_scale) if which == "k"
                       else (self.v, self.vp, self.v_scale))
        x = x[pages, :, offs]
        if self.kind == "int4":
            a, m = int4_split(x, p[pages, :, offs])
            return a + m, a, m
        val = (oracle.e4m3_decode(x) * float(np.float32(scale)) if self.kind == "fp8" else bf16(x))
        return val, val, np.zeros_like(val)

    def read(self, slot_map):
        """fp64 values [T][Hkv][D] of K and V (zeros where there is no slot)."""
        NP, H, P, D = self.shape
        slot_map = np.asarray(slot_map)
        have = (slot_map >= 0) & (slot_map < NP * P)
        back = []
        for which in "kv":
            out = np.zeros((slot_map.size, H, D))
            out[have] = self.rows(which, slot_map[have] // P, slot_map[have] % P)[0]
            back.append(out)
        return back


# ---------------------------------------------------------------------------
# page tables
# ---------------------------------------------------------------------------

def extend_tables(old, new, P, free, num_free, table, num_pages, max_tokens, tags=None,
                  expected=None):
    """Request by request; returns a dict of the outputs (inputs are not changed)."""
    table = table.copy()
    expected = None if expected is None else expected.copy()
    MP = table.shape[1]
    num_free = min(max(int(num_free), 0), len(free))
    slots = np.full(max_tokens, -1, np.int32)
    cu, failed, asked, left = [0], [], 0, num_free
    for b, (o, n) in enumerate(zip(map(int, old), map(int, new))):
        fine = 0 <= o <= n <= MP * P
        first, last = -(-o // P), -(-n // P)
        need = last - first if fine else 0
        asked += need
        ok = fine and (need == 0 or asked <= num_free)
        if ok:
            for j in range(first, last):
                left -= 1
                table[b, j] = free[left]
                if tags is not None and 0 <= free[left] < num_pages:
                    expected[b, j] = tags[free[left]]
        count = n - o if 0 <= o <= n else 0
        if ok:
            for i in range(count):
                t, page = cu[-1] + i, int(table[b, (o + i) // P])
                if t < max_tokens and 0 <= page < num_pages:
                    slots[t] = page * P + (o + i) % P
        cu.append(min(cu[-1] + count, 2 ** 31 - 1))
        failed.append(0 if ok else 1)
    return {"table": table, "expected": expected, "slots": slots, "cu": np.array(cu, np.int32),
            "failed": np.array(failed, np.uint8), "free": left}


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------

def visible(length, window, sinks):
    t = np.arange(length)
    return t if not window else t[(t >= length - window) | (t < sinks)]


def attend(q_bits, pools, table, lens, sm_scale, window=0, sinks=0, abort=None):
    """(out, lse, out_tol, lse_tol) in fp64: the definition, and what its roundings allow.

    With w_t the softmax weights, the kernels round (1) each weight (INT4: weight
    times scale) to f16, or bf16 over a BF16 cache, before the V product: half a
    step of the part of the values it multiplies, and over FP8 and BF16 caches
    once more in the sum they divide by; (2) weights below f16's normal range to
    multiples of 2^-24, INT4: of the largest scale: half of that per token;
    (3) scores and sums in binary32: D + 8 steps of the sum of the products'
    magnitudes, which moves a weight by that factor and the output by twice it
    (numerator and denominator); (4) the output to bf16.
    """
    NP, H, P, D = pools.shape
    B, Hq, _ = q_bits.shape
    G = Hq // H
    out, lse = np.zeros((B, Hq, D)), np.full((B, Hq), -np.inf)
    out_tol, lse_tol = np.zeros((B, Hq, D)), np.zeros((B, Hq))
    q = bf16(q_bits).reshape(B, H, G, D)
    sm = float(np.float32(sm_scale))
    MP = table.shape[1]
    weight_step = BF16_STEP if pools.kind == "bf16" else F16_STEP
    for b in range(B):
        L = int(lens[b])
        if (abort is not None and abort[b]) or not 1 <= L <= MP * P:
            continue
        t = visible(L, window, sinks)
        pages = table[b, t // P]
        if ((pages < 0) | (pages >= NP)).any():
            continue
        k, ka, km = pools.rows("k", pages, t % P)
        v, va, vm = pools.rows("v", pages, t % P)
        s = np.einsum("hgd,thd->hgt", q[b], k) * sm
        size = np.einsum("hgd,thd->hgt", np.abs(q[b]), np.abs(ka) + np.abs(km)).max(-1) * sm
        top = s.max(-1, keepdims=True)
        e = np.exp(s - top)
        tot = e.sum(-1, keepdims=True)
        w = e / tot
        o = np.einsum("hgt,thd->hgd", w, v)
        mag = np.einsum("hgt,thd->hgd", w, np.abs(va))
        mag_m = np.einsum("hgt,thd->hgd", w, np.abs(vm))
        moved = ((D + 8) * 2 * F32_STEP * size + 2.0 ** -20)[..., None]
        once = 1 if pools.kind == "int4" else 2
        small = 0.0
        if pools.kind != "bf16":
            # (of the head: a NaN elsewhere is not part of the bound)
            unit = 15.0 * np.nanmax(bf16(pools.vp[pages, :, t % P])[..., 0], axis=(0, 2)) \
                if pools.kind == "int4" else np.nanmax(np.abs(v), axis=(0, 2))
            small = (len(t) * 2.0 ** -25 * unit)[:, None, None]
        tol = weight_step * once * mag + small + 2 * moved * (mag + mag_m)
        out[b], lse[b] = o.reshape(Hq, D), (top + np.log(tot))[..., 0].reshape(Hq)
        out_tol[b] = (BF16_STEP * (np.abs(o) + tol) + tol).reshape(Hq, D)
        lse_tol[b] = (moved[..., 0] + 4 * F32_STEP * (np.abs(lse[b]).reshape(H, G) + 1)).reshape(Hq)
    return out, lse, out_tol, lse_tol


def check_attention(got_out, got_lse, want, label=""):
    """Every output against attend()'s."""
    out, lse, out_tol, lse_tol = want
    dead = np.isneginf(lse)
    assert np.isneginf(got_lse[dead]).all() and not got_out[dead].any(), f"{label}: dead rows"
    nan = np.isnan(out)
    assert np.isnan(got_out[nan]).all(), f"{label}: NaN values lost"
    fine = ~nan & ~dead[..., None]
    err = np.abs(got_out - out)
    worst = np.max(err[fine] / out_tol[fine], initial=0.0)
    assert worst <= 1.0, f"{label}: output error {worst:.3f} of its bound"
    fin = np.isfinite(lse)
    lworst = np.max(np.abs(got_lse[fin] - lse[fin]) / lse_tol[fin], initial=0.0)
    assert lworst <= 1.0, f"{label}: lse error {lworst:.3f} of its bound"
    assert np.isnan(got_lse[np.isnan(lse)]).all(), f"{label}: NaN lse lost"
    return worst, lworst
