"""Measured cases of the paged-cache operators: page tables and slot maps, slot writes and reads, decode
attention over a 4-bit cache, and decode attention with a sliding window and sinks.

``run`` computes them in elementary torch operations in 32 bits (``own`` false) or through the library
(``own`` true); ``exact`` computes them from their definitions in 64 bits.

The 4-bit cache holds, per token, KV head and group of 64 dims, 4-bit codes and a bf16 pair (s, m); the value is
s * code + m, with m the group's minimum, s = bf16((max - min) / 15) and
code = min(15, round_half_even((x - m) / s)), each step of the quotient in binary32.
"""
import math
import random

import numpy as np
import torch

own = False

GROUP = 64          # dims that share a (scale, minimum) pair of the 4-bit cache
OUTLIER_P = 0.01    # K and V are N(0, 1) with 1% of the elements times 20, as the decode workloads draw them
OUTLIER_MUL = 20.0


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _tables(name, batch, page, ctx_lo, ctx_hi, new_lo, new_hi, shape_seed):
    return {"name": name, "op": "tables", "batch": batch, "page": page, "ctx_lo": ctx_lo, "ctx_hi": ctx_hi,
            "new_lo": new_lo, "new_hi": new_hi, "shape_seed": shape_seed}


def _slots(name, kv, tokens, hkv, d, page, skip):
    return {"name": name, "op": "slots", "kv": kv, "tokens": tokens, "hkv": hkv, "d": d, "page": page,
            "skip": skip}


def _attn(name, kv, batch, lo, hi, hq, hkv, d, page, window, sinks, aborted, shape_seed):
    return {"name": name, "op": "attn", "kv": kv, "batch": batch, "lo": lo, "hi": hi, "hq": hq, "hkv": hkv,
            "d": d, "page": page, "window": window, "sinks": sinks, "aborted": aborted,
            "shape_seed": shape_seed}


def listed():
    return [
        # one decode step of 64 requests: one token each, a new page for some
        _tables("tables_decode_b64", 64, 64, 1024, 16384, 1, 1, 11),
        # a prefill step: prompts of odd lengths on empty and half-filled rows, small pages
        _tables("tables_prefill_b48", 48, 16, 0, 2000, 1, 2047, 12),
        # the new tokens of a decode batch of 64, then read back
        _slots("slots_int4_decode_t64", "int4", 64, 8, 128, 64, 0.0),
        # a prefill chunk of 8,192 tokens
        _slots("slots_int4_prefill_t8192", "int4", 8192, 8, 128, 64, 0.0),
        # a padded FP8 chunk: odd token count, a quarter of the rows carry no slot
        _slots("slots_fp8_padded_t5001", "fp8", 5001, 8, 128, 16, 0.25),
        # a single request at the sweep's context: latency
        _attn("attn_int4_b1_l8192", "int4", 1, 8192, 8192, 64, 8, 128, 64, 0, 0, 0.0, 21),
        # the concurrency sweep's largest batch
        _attn("attn_int4_b64_l8192", "int4", 64, 8192, 8192, 64, 8, 128, 64, 0, 0, 0.0, 22),
        # ragged batch of short and long odd lengths with a few aborted requests, 64-dim heads, small pages
        _attn("attn_int4_b96_ragged_d64", "int4", 96, 1, 8190, 48, 8, 64, 16, 0, 0, 0.03, 23),
        # two requests at the longest context of the ragged workload
        _attn("attn_int4_b2_l131072", "int4", 2, 131071, 131072, 32, 8, 128, 128, 0, 0, 0.0, 24),
        # a window layer of the sweep's batch, FP8
        _attn("window_fp8_b64_w1024", "fp8", 64, 8192, 8192, 64, 8, 128, 64, 1024, 4, 0.0, 25),
        # ragged lengths around an odd window, BF16, two heads a group
        _attn("window_bf16_b32_w4095", "bf16", 32, 3, 16384, 16, 8, 128, 32, 4095, 5, 0.03, 26),
        # long contexts over the 4-bit cache with 64 sinks
        _attn("window_int4_b8_l65536", "int4", 8, 60001, 65536, 64, 8, 128, 64, 16384, 64, 0.0, 27),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    seed = rng.randrange(1 << 20)
    page = rng.choice([16, 32, 64, 128])
    op = rng.choice(["tables", "slots", "attn", "attn", "window", "window"])
    if op == "tables":
        batch = _log(rng, 1, 1024)
        new_hi = 1 if rng.random() < 0.5 else _log(rng, 2, max(2, min(4096, 65536 // batch)))
        case = _tables("", batch, page, rng.choice([0, 1, 500]), _log(rng, 501, 16384), rng.choice([0, 1]),
                       new_hi, seed)
    elif op == "slots":
        hkv, d = rng.choice([1, 2, 3, 8]), rng.choice([64, 128])
        case = _slots("", rng.choice(["int4", "fp8", "bf16"]), _log(rng, 1, 8192 * 8 * 128 // (hkv * d) // 2), hkv, d,
                      page, rng.choice([0.0, 0.1]))
    else:
        hkv, d = rng.choice([1, 2, 3, 4, 8]), rng.choice([64, 128])
        group = rng.choice([1, 2, 3, 4, 5, 6, 8, 12, 16])
        batch = _log(rng, 1, 128)
        hi = _log(rng, 16, min(131072, 64 * 8192 // batch))
        lo = rng.choice([1, max(1, hi // 3), hi])
        window, sinks = 0, 0
        if op == "window":
            window, sinks = _log(rng, 1, hi), rng.choice([0, 1, 4, 64, 100])
        kv = "int4" if op == "attn" else rng.choice(["fp8", "bf16", "int4"])
        case = _attn("", kv, batch, lo, hi, hkv * group, hkv, d, page, window, sinks, rng.choice([0.0, 0.05]), seed)
    del case["name"]
    return case


# ---------------------------------------------------------------------------
# shapes that a case fixes (lengths do not depend on the inputs' seed)
# ---------------------------------------------------------------------------

def _table_shape(case):
    r = random.Random(case["shape_seed"])
    old = [r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["batch"])]
    new = [o + r.randint(case["new_lo"], case["new_hi"]) for o in old]
    return old, new


def _attn_shape(case):
    r = random.Random(case["shape_seed"])
    lens = [r.randint(case["lo"], case["hi"]) for _ in range(case["batch"])]
    dead = [r.random() < case["aborted"] for _ in range(case["batch"])]
    return lens, dead


def _ceil(a, b):
    return -(-a // b)


def _visible(case, length):
    if not case["window"]:
        return length
    return min(length, case["window"] + min(case["sinks"], max(0, length - case["window"])))


def work(case):
    if case["op"] == "tables":
        old, new = _table_shape(case)
        pages = sum(_ceil(n, case["page"]) - _ceil(o, case["page"]) for o, n in zip(old, new))
        tokens = sum(new) - sum(old)
        # lengths in, offsets and flags out, slots out, free ids and tags in, table entries and expected tags out
        return {"bytes": case["batch"] * (8 + 4 + 1) + 4 * tokens + 16 * pages, "flops": tokens + pages}
    if case["op"] == "slots":
        row = case["hkv"] * case["d"]
        held = {"int4": row / 2 + row // GROUP * 4, "fp8": row, "bf16": 2 * row}[case["kv"]]
        n = case["tokens"] * (1.0 - case["skip"])
        # write: values in, codes out; read: codes in, values out; the slots twice
        return {"bytes": int(2 * n * (2 * row + held + held) + 2 * case["tokens"] * 2 * row + 8 * case["tokens"]),
                "flops": int(8 * n * row)}
    lens, dead = _attn_shape(case)
    seen = [_visible(case, n) for n, x in zip(lens, dead) if not x]
    row = case["hkv"] * case["d"]
    held = {"int4": row / 2 + row // GROUP * 4, "fp8": row, "bf16": 2 * row}[case["kv"]]
    io = case["batch"] * case["hq"] * (4 * case["d"] + 4)
    return {"bytes": int(2 * sum(seen) * held + io + sum(4 * _ceil(n, case["page"]) for n in seen)),
            "flops": 4 * sum(seen) * case["hq"] * case["d"]}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _draw_kv(shape, g):
    x = torch.randn(shape, generator=g, device="cuda")
    u = torch.rand(shape, generator=g, device="cuda")
    return torch.where(u < OUTLIER_P, x * OUTLIER_MUL, x).to(torch.bfloat16)


def _pack_int4(x):
    """bf16 [..., D] -> (codes uint8 [..., D/2], params bf16 [..., D/64, 2])."""
    f = x.float().unflatten(-1, (-1, GROUP))
    lo, hi = f.amin(-1, keepdim=True) + 0.0, f.amax(-1, keepdim=True)
    # (divisors are tensors: a division by a number is a product with its reciprocal on the GPU)
    s = ((hi - lo) / torch.full_like(hi, 15.0)).to(torch.bfloat16).float()
    code = torch.where(s > 0, torch.round((f - lo) / s), torch.zeros_like(f)).clamp(max=15.0)
    code = code.to(torch.uint8).flatten(-2)
    codes = code[..., 0::2] | (code[..., 1::2] << 4)
    return codes, torch.cat([s, lo], -1).to(torch.bfloat16)


def _unpack_int4(codes, params):
    n = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).float().unflatten(-1, (-1, GROUP))
    p = params.float()
    return (n * p[..., 0:1] + p[..., 1:2]).flatten(-2)


def _pack_fp8(x, scale):
    y = x.float()
    return (y / torch.full_like(y, scale)).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


class _State:
    pass


def _pool(kv, pages, hkv, page, d, g):
    """A cache pool of one tensor, filled as a prefill leaves it: a dict of its buffers."""
    if kv == "bf16":
        x = torch.empty((pages, hkv, page, d), dtype=torch.bfloat16, device="cuda")
    elif kv == "fp8":
        x = torch.empty((pages, hkv, page, d), dtype=torch.uint8, device="cuda")
    else:
        x = torch.empty((pages, hkv, page, d // 2), dtype=torch.uint8, device="cuda")
        p = torch.empty((pages, hkv, page, d // GROUP, 2), dtype=torch.bfloat16, device="cuda")
    scale = OUTLIER_MUL * 5.5 / 448.0
    step = max(1, (1 << 25) // (hkv * page * d))
    for at in range(0, pages, step):
        v = _draw_kv((min(step, pages - at), hkv, page, d), g)
        if kv == "bf16":
            x[at: at + step] = v
        elif kv == "fp8":
            x[at: at + step] = _pack_fp8(v, scale)
        else:
            x[at: at + step], p[at: at + step] = _pack_int4(v)
    return {"x": x, "p": p if kv == "int4" else None, "scale": scale if kv == "fp8" else 1.0}


def prepare(case, seed):
    st = _State()
    st.case = case
    g = _gen(seed)
    rng = np.random.Generator(np.random.PCG64(int(seed)))
    page = case["page"]
    if case["op"] == "tables":
        old, new = _table_shape(case)
        b = case["batch"]
        used = [_ceil(o, page) for o in old]
        need = sum(_ceil(n, page) for n in new) - sum(used)
        st.num_pages = sum(used) + need + 7
        st.max_pages = max(1, max(_ceil(n, page) for n in new))
        perm = rng.permutation(st.num_pages).astype(np.int32)
        table = np.full((b, st.max_pages), -1, dtype=np.int32)
        at = 0
        for i, n in enumerate(used):
            table[i, :n] = perm[at: at + n]
            at += n
        tags = rng.integers(0, 1 << 31, st.num_pages).astype(np.int32)
        st.tokens = sum(new) - sum(old) + 3          # a padded step: three rows carry no token
        st.old = torch.tensor(old, dtype=torch.int32, device="cuda")
        st.new = torch.tensor(new, dtype=torch.int32, device="cuda")
        st.free = torch.from_numpy(perm[at:].copy()).cuda()
        st.num_free = torch.tensor([perm.size - at], dtype=torch.int32, device="cuda")
        st.num_free_out = torch.zeros(1, dtype=torch.int32, device="cuda")
        st.table = torch.from_numpy(table).cuda()
        st.tags = torch.from_numpy(tags).cuda()
        st.expected = torch.zeros((b, st.max_pages), dtype=torch.int32, device="cuda")
        st.slots = torch.zeros(st.tokens, dtype=torch.int32, device="cuda")
        st.cu = torch.zeros(b + 1, dtype=torch.int32, device="cuda")
        st.failed = torch.zeros(b, dtype=torch.uint8, device="cuda")
        return st
    hkv, d = case["hkv"], case["d"]
    if case["op"] == "slots":
        t = case["tokens"]
        pages = _ceil(t, page) + 5
        slots = rng.permutation(pages)[: _ceil(t, page)].astype(np.int64)
        slots = (slots[:, None] * page + np.arange(page)[None, :]).reshape(-1)[:t].astype(np.int32)
        slots[rng.random(t) < case["skip"]] = -1
        st.slots = torch.from_numpy(slots).cuda()
        st.k_new, st.v_new = _draw_kv((t, hkv, d), g), _draw_kv((t, hkv, d), g)
        st.k, st.v = _pool(case["kv"], pages, hkv, page, d, g), _pool(case["kv"], pages, hkv, page, d, g)
        st.k_back, st.v_back = torch.empty_like(st.k_new), torch.empty_like(st.v_new)
        return st
    lens, dead = _attn_shape(case)
    b, hq = case["batch"], case["hq"]
    used = [_ceil(n, page) for n in lens]
    perm = rng.permutation(sum(used) + 3).astype(np.int32)
    table = np.full((b, max(used)), -1, dtype=np.int32)
    at = 0
    for i, n in enumerate(used):
        table[i, :n] = perm[at: at + n]
        at += n
    st.table = torch.from_numpy(table).cuda()
    st.lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
    st.abort = torch.tensor(dead, dtype=torch.uint8, device="cuda") if any(dead) else None
    st.q = torch.randn((b, hq, d), generator=g, device="cuda").to(torch.bfloat16)
    st.k, st.v = (_pool(case["kv"], perm.size, hkv, page, d, g) for _ in range(2))
    st.sm = 1.0 / math.sqrt(d)
    st.out = torch.empty((b, hq, d), dtype=torch.bfloat16, device="cuda")
    st.lse = torch.empty((b, hq), dtype=torch.float32, device="cuda")
    st.work = torch.zeros(64 << 20, dtype=torch.uint8, device="cuda")
    return st


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(st):
    op = st.case["op"]
    if own:
        return {"tables": _own_tables, "slots": _own_slots, "attn": _own_attn}[op](st)
    return {"tables": _plain_tables, "slots": _plain_slots, "attn": _plain_attn}[op](st)


def _own_tables(st):
    import paged_fp8_kv_attn_b200 as pkv
    pkv.kv_extend_tables(st.old, st.new, st.case["page"], st.free, st.num_free, st.table, st.slots, st.cu,
                         st.failed, st.num_free_out, st.num_pages, page_tags=st.tags, expected_tags=st.expected)
    return {"table": st.table, "expected": st.expected, "slots": st.slots, "cu": st.cu, "failed": st.failed,
            "free": st.num_free_out}


def _plain_tables(st):
    page, b = st.case["page"], st.case["batch"]
    old, new = st.old.long(), st.new.long()
    first = (old + page - 1) // page
    fine = (old >= 0) & (new >= old) & (new <= st.max_pages * page)
    need = torch.where(fine, (new + page - 1) // page - first, 0)
    upto = need.cumsum(0)
    served = fine & ((upto <= st.num_free) | (need == 0))
    got = torch.where(served, need, 0)
    begin = upto - need
    # new table entries: entry j of a served row takes the (begin + j - first)-th page from the stack's top
    j = torch.arange(st.max_pages, device="cuda")
    k = j[None, :] - first[:, None]
    fresh = (k >= 0) & (k < got[:, None])
    at = (st.num_free - 1 - begin[:, None] - k).clamp(0, st.free.numel() - 1)
    page_ids = st.free[at]
    table = torch.where(fresh, page_ids, st.table)
    expected = torch.where(fresh, st.tags[page_ids.long()], st.expected)
    # slots of the packed new tokens
    count = torch.where((old >= 0) & (new > old), new - old, 0)
    cu = torch.cat([torch.zeros(1, dtype=torch.long, device="cuda"), count.cumsum(0)])
    t = torch.arange(st.tokens, device="cuda")
    row = torch.searchsorted(cu, t, right=True) - 1
    real = row < b
    row = row.clamp(max=b - 1)
    pos = (old[row] + t - cu[row]).clamp(0, st.max_pages * page - 1)
    entry = table[row, pos // page].long()
    ok = real & served[row] & (entry >= 0) & (entry < st.num_pages)
    slots = torch.where(ok, entry * page + pos % page, -1)
    return {"table": table, "expected": expected, "slots": slots.int(), "cu": cu.int(),
            "failed": (~served).to(torch.uint8), "free": (st.num_free - got.sum()).int()}


def _own_slots(st):
    import paged_fp8_kv_attn_b200 as pkv
    kv = st.case["kv"]
    if kv == "int4":
        pools = (st.k["x"], st.k["p"], st.v["x"], st.v["p"])
        pkv.kv_write_slots_int4(st.k_new, st.v_new, st.slots, *pools)
        pkv.kv_read_slots_int4(st.slots, *pools, st.k_back, st.v_back)
    elif kv == "fp8":
        pkv.kv_write_slots_fp8(st.k_new, st.v_new, st.slots, st.k["scale"], st.v["scale"], st.k["x"], st.v["x"])
        pkv.kv_read_slots_fp8(st.slots, st.k["scale"], st.v["scale"], st.k["x"], st.v["x"], st.k_back, st.v_back)
    else:
        pkv.kv_write_slots_bf16(st.k_new, st.v_new, st.slots, st.k["x"], st.v["x"])
        pkv.kv_read_slots_bf16(st.slots, st.k["x"], st.v["x"], st.k_back, st.v_back)
    return {"k": st.k_back, "v": st.v_back}


def _plain_slots(st):
    page = st.case["page"]
    have = st.slots >= 0
    at = st.slots.long()[have]
    where = (at // page, slice(None), at % page)      # [page][head][slot] rows of the pool
    back = {}
    for name, new, pool in (("k", st.k_new, st.k), ("v", st.v_new, st.v)):
        x = new[have]
        if st.case["kv"] == "int4":
            pool["x"][where], pool["p"][where] = _pack_int4(x)
            got = _unpack_int4(pool["x"][where], pool["p"][where])
        elif st.case["kv"] == "fp8":
            pool["x"][where] = _pack_fp8(x, pool["scale"])
            got = pool["x"][where].view(torch.float8_e4m3fn).float() * pool["scale"]
        else:
            pool["x"][where] = x
            got = pool["x"][where]
        out = torch.zeros_like(new)
        out[have] = got.to(torch.bfloat16)
        back[name] = out
    return back


def _own_attn(st):
    import paged_fp8_kv_attn_b200 as pkv
    c = st.case
    win = (c["window"], c["sinks"]) if c["window"] else ()
    rest = (st.table, st.lens, st.sm, *win, st.out, st.lse, st.work)
    if c["kv"] == "int4":
        f = pkv.paged_decode_attn_int4_window if win else pkv.paged_decode_attn_int4
        f(st.q, st.k["x"], st.k["p"], st.v["x"], st.v["p"], *rest, abort=st.abort)
    elif c["kv"] == "fp8":
        pkv.paged_decode_attn_fp8_window(st.q, st.k["x"], st.v["x"], st.k["scale"], st.v["scale"], *rest,
                                         abort=st.abort)
    else:
        pkv.paged_decode_attn_bf16_window(st.q, st.k["x"], st.v["x"], *rest, abort=st.abort)
    return {"out": st.out, "lse": st.lse}


def _plain_attn(st):
    c = st.case
    b, hkv, d = c["batch"], c["hkv"], c["d"]
    ids = st.table.clamp(min=0).long()

    def dense(pool):   # [B][Hkv][MP * P][D] in 32 bits
        x = pool["x"][ids].transpose(1, 2).flatten(2, 3)
        if c["kv"] == "int4":
            return _unpack_int4(x, pool["p"][ids].transpose(1, 2).flatten(2, 3))
        if c["kv"] == "fp8":
            return x.view(torch.float8_e4m3fn).float() * pool["scale"]
        return x.float()

    q = st.q.float().unflatten(1, (hkv, -1))
    s = (q @ dense(st.k).transpose(2, 3)) * st.sm                         # [B][Hkv][G][T]
    t = torch.arange(s.shape[-1], device="cuda")[None, :]
    lens = st.lens[:, None].long()
    see = t < lens
    if c["window"]:
        see = see & ((t >= lens - c["window"]) | (t < c["sinks"]))
    if st.abort is not None:
        see = see & (st.abort[:, None] == 0)
    s = s.masked_fill(~see[:, None, None, :], -math.inf)
    top = s.amax(-1, keepdim=True)
    e = torch.exp(s - torch.where(torch.isfinite(top), top, 0.0))
    total = e.sum(-1, keepdim=True)
    out = (e @ dense(st.v)) / torch.where(total > 0, total, 1.0)
    lse = (top + torch.log(total)).squeeze(-1)
    return {"out": out.flatten(1, 2).to(torch.bfloat16), "lse": lse.flatten(1)}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "tables":
        return _exact_tables(st)
    if case["op"] == "slots":
        return {"k": _exact_round_trip(st, st.k_new, st.k), "v": _exact_round_trip(st, st.v_new, st.v)}
    return _exact_attn(st)


def _exact_tables(st):
    """The rows request by request, pages taken from the free stack one after another."""
    page = st.case["page"]
    old, new = _table_shape(st.case)
    free, left = st.free.tolist(), int(st.num_free)
    tags = st.tags.cpu().numpy()
    table, expected = st.table.cpu().numpy().copy(), st.expected.cpu().numpy().copy()
    slots, cu, failed = np.full(st.tokens, -1, dtype=np.int32), [0], np.zeros(st.case["batch"], dtype=np.uint8)
    for b, (o, n) in enumerate(zip(old, new)):
        for j in range(_ceil(o, page), _ceil(n, page)):
            left -= 1
            table[b, j] = free[left]
            expected[b, j] = tags[free[left]]
        pos = np.arange(o, n)
        slots[cu[-1]: cu[-1] + n - o] = table[b, pos // page] * page + pos % page
        cu.append(cu[-1] + n - o)
    back = {"table": table, "expected": expected, "slots": slots, "cu": np.array(cu, dtype=np.int32),
            "failed": failed, "free": np.array([left], dtype=np.int32)}
    return {k: torch.from_numpy(v).cuda() for k, v in back.items()}


def _exact_round_trip(st, new, pool):
    """What the cache holds of each written token, from the formats' definitions."""
    kv = st.case["kv"]
    x = new.double()
    if kv == "int4":
        # the quotient's steps are binary32 by definition: computed in 64 bits and rounded to 32
        r32 = lambda v: v.to(torch.float32).double()  # noqa: E731
        blocks = x.reshape(*x.shape[:-1], -1, GROUP)
        low = torch.min(blocks, dim=-1, keepdim=True).values
        span = r32(torch.max(blocks, dim=-1, keepdim=True).values - low)
        step = r32(span / torch.full_like(span, 15.0)).to(torch.bfloat16).double()
        n = torch.round(r32(r32(blocks - low) / torch.where(step == 0, 1.0, step)))
        n = torch.minimum(n, torch.full_like(n, 15.0)) * (step != 0)
        held = (low + step * n).reshape(x.shape)
    elif kv == "fp8":
        # the nearest of the 127 non-negative E4M3 values, ties to the even code
        code = torch.arange(127, dtype=torch.float64, device="cuda")
        e, f = torch.div(code, 8, rounding_mode="floor"), code % 8
        grid = torch.where(e == 0, f * 2.0 ** -9, (1 + f / 8) * 2.0 ** (e - 7))
        scale = float(np.float32(pool["scale"]))
        y = (x / torch.full_like(x, scale)).to(torch.float32).double()
        a = y.abs().clamp(max=448.0)
        up = torch.searchsorted(grid, a.contiguous()).clamp(max=126)
        dn = (up - 1).clamp(min=0)
        du, dd = grid[up] - a, a - grid[dn]
        pick = torch.where((du < dd) | ((du == dd) & (up % 2 == 0)), up, dn)
        held = grid[pick] * torch.sign(y) * scale
    else:
        held = x
    return held * (st.slots >= 0)[:, None, None]


def _exact_attn(st):
    c = st.case
    lens, dead = _attn_shape(c)
    hq, hkv, d, page = c["hq"], c["hkv"], c["d"], c["page"]
    out = torch.zeros((c["batch"], hq, d), dtype=torch.float64, device="cuda")
    lse = torch.full((c["batch"], hq), -math.inf, dtype=torch.float64, device="cuda")
    for i, (n, gone) in enumerate(zip(lens, dead)):
        if gone:
            continue
        keep = torch.arange(n, device="cuda")
        if c["window"]:
            keep = keep[(keep >= n - c["window"]) | (keep < c["sinks"])]
        pages, offs = st.table[i].long()[keep // page], keep % page

        def rows(pool):   # [T][Hkv][D]
            x = pool["x"][pages, :, offs]
            if c["kv"] == "fp8":
                return x.view(torch.float8_e4m3fn).double() * float(np.float32(pool["scale"]))
            if c["kv"] == "bf16":
                return x.double()
            par = pool["p"][pages, :, offs].double()
            val = torch.empty((*x.shape[:2], d), dtype=torch.float64, device="cuda")
            val[..., 0::2], val[..., 1::2] = (x % 16).double(), (x // 16).double()
            for k in range(d // GROUP):
                part = val[..., k * GROUP: (k + 1) * GROUP]
                part.mul_(par[:, :, k, 0, None]).add_(par[:, :, k, 1, None])
            return val

        k, v = rows(st.k), rows(st.v)
        q = st.q[i].double().reshape(hkv, hq // hkv, d)
        s = torch.einsum("hgd,thd->hgt", q, k) * float(np.float32(st.sm))
        z = torch.logsumexp(s, dim=-1)
        out[i] = torch.einsum("hgt,thd->hgd", torch.exp(s - z[..., None]), v).reshape(hq, d)
        lse[i] = z.reshape(hq)
    return {"out": out, "lse": lse}
