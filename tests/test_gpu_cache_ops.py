"""GPU parity of the 4-bit cache, the slot calls, the page tables and the
windowed attention, against the 64-bit references of _cache_reference: bytes and
whole numbers exactly, attention within the bound that its roundings allow."""
import numpy as np
import pytest
import torch

import oracle
import paged_fp8_kv_attn_b200 as pkv

import _cache_reference as ref

pytestmark = pytest.mark.gpu

KINDS = ("int4", "fp8", "bf16")


def cuda(a):
    """A host array on the GPU (uint16 as bf16 bits, uint32 as int32)."""
    a = np.ascontiguousarray(a)
    if a.dtype == np.uint16:
        return torch.from_numpy(a.view(np.int16)).cuda().view(torch.bfloat16)
    return torch.from_numpy(a.view(np.int32) if a.dtype == np.uint32 else a).cuda()


def bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def values(t):
    return t.float().cpu().numpy().astype(np.float64)


class Cache:
    """A host cache's pools on the GPU."""

    def __init__(self, p):
        self.p = p
        self.k, self.v = cuda(p.k), cuda(p.v)
        self.kp, self.vp = (None, None) if p.kp is None else (cuda(p.kp), cuda(p.vp))

    @property
    def pools(self):
        return (self.k, self.v) if self.kp is None else (self.k, self.kp, self.v, self.vp)

    @property
    def scales(self):
        return (self.p.k_scale, self.p.v_scale) if self.p.kind == "fp8" else ()

    def write(self, k, v, slots, **kw):
        getattr(pkv, f"kv_write_slots_{self.p.kind}")(k, v, slots, *self.scales, *self.pools, **kw)

    def read(self, slots, k, v):
        getattr(pkv, f"kv_read_slots_{self.p.kind}")(slots, *self.scales, *self.pools, k, v)

    def attend(self, q, table, lens, sm, ws, window=0, sinks=0, abort=None, num_ctas=0, out=None):
        B, Hq, D = q.shape
        if out is None:
            out = (torch.full((B, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda"),
                   torch.full((B, Hq), 7.0, device="cuda"))
        win, tail = ((window, sinks), "_window") if window else ((), "")
        args = (self.k, self.kp, self.v, self.vp) if self.kp is not None else \
            (self.k, self.v, *self.scales)
        getattr(pkv, f"paged_decode_attn_{self.p.kind}{tail}")(
            q, *args, table, lens, sm, *win, *out, ws, abort=abort, num_ctas=num_ctas)
        return out

    def workspace(self, B, Hq, num_ctas=0):
        kind = {"fp8": pkv.PKV_KV_FP8, "bf16": pkv.PKV_KV_BF16, "int4": pkv.PKV_KV_INT4}[self.p.kind]
        n = pkv.paged_decode_attn_workspace_size(kind, B, Hq, self.p.shape[1], self.p.shape[3],
                                                 num_ctas)
        return torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")

    def same(self, p):
        for a, b in ((self.k, p.k), (self.v, p.v), (self.kp, p.kp), (self.vp, p.vp)):
            if b is None:
                continue
            got = a.cpu().numpy() if b.dtype == np.uint8 else bits(a)
            bad = np.argwhere(got != b)
            assert bad.size == 0, f"{len(bad)} entries differ, first at {bad[0]}"


def normal_bits(rng, shape):
    x = rng.standard_normal(shape)
    x[rng.random(shape) < 0.01] *= 20.0
    return ref.f32_bits_to_bf16(x.astype(np.float32))


# ---------------------------------------------------------------------------
# slots
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T,H,D,P", [(1, 1, 64, 16), (7, 3, 64, 32), (129, 8, 128, 64),
                                     (1, 20, 128, 128), (300, 2, 128, 16), (33, 5, 64, 128)])
def test_write_and_read_slots(cuda_device, kind, T, H, D, P):
    rng = np.random.Generator(np.random.PCG64(T * H + D))
    NP = -(-T // P) + 3
    p = ref.Pools(kind, NP, H, P, D, 0.11, 0.23, seed=T)
    c = Cache(p)
    slots = rng.permutation(NP * P)[:T].astype(np.int32)
    drop = rng.random(T) < 0.2
    slots[drop] = rng.choice([-1, NP * P, -2**31, 2**31 - 1], int(drop.sum()))
    k, v = normal_bits(rng, (T, H, D)), normal_bits(rng, (T, H, D))
    c.write(cuda(k), cuda(v), cuda(slots))
    p.write(slots, k, v)
    torch.cuda.synchronize()
    c.same(p)
    back = [torch.full((T, H, D), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    c.read(cuda(slots), *back)
    for got, want in zip(back, p.read(slots)):
        assert np.array_equal(bits(got) & 0x7FFF, oracle.bf16_from_double(want) & 0x7FFF)
        assert np.array_equal(values(got), ref.bf16(oracle.bf16_from_double(want)))


@pytest.mark.parametrize("kind", KINDS)
def test_slots_with_strided_rows(cuda_device, kind):
    """K and V as parts of one wider row, the rows behind and between left alone."""
    rng = np.random.Generator(np.random.PCG64(3))
    T, H, D, P = 21, 2, 64, 16
    p = ref.Pools(kind, 4, H, P, D, 0.1, 0.1, seed=1)
    c = Cache(p)
    wide = normal_bits(rng, (T + 2, 5 * H * D + 8))
    g = cuda(wide)
    part = lambda x, i: x[1: T + 1, 8 + i * H * D: 8 + (i + 1) * H * D].unflatten(1, (H, D))  # noqa: E731
    slots = rng.permutation(4 * P)[:T].astype(np.int32)
    c.write(part(g, 3), part(g, 1), cuda(slots))
    host = torch.from_numpy(wide.view(np.int16))
    p.write(slots, *(part(host, i).numpy().view(np.uint16) for i in (3, 1)))
    torch.cuda.synchronize()
    c.same(p)
    out = torch.full((T + 2, 5 * H * D + 8), 7.0, dtype=torch.bfloat16, device="cuda")
    c.read(cuda(slots), part(out, 0), part(out, 4))
    want = p.read(slots)
    for i, w in zip((0, 4), want):
        assert np.array_equal(values(part(out, i)), ref.bf16(oracle.bf16_from_double(w)))
    part(out, 0).fill_(7.0)
    part(out, 4).fill_(7.0)
    assert (out == 7.0).all()


def test_int4_values_every_range(cuda_device):
    """Groups of every magnitude, flat ones, signed zeros, subnormals, ties, NaN, Inf and
    ranges beyond binary32, through the append-format write, bit for bit."""
    rng = np.random.Generator(np.random.PCG64(12))
    T, H, D = 4000, 1, 128
    x = (rng.standard_normal((T, H, D)) * np.exp2(rng.integers(-140, 120, (T, 1, 1)))).astype(np.float32)
    b = ref.f32_bits_to_bf16(x)
    b[:500] = rng.integers(0, 65536, (500, H, D)).astype(np.uint16)          # any pattern
    b[500:600] = rng.integers(0, 2, (100, H, D)).astype(np.uint16) << 15      # +-0
    b[600:700] = b[600:700, :, :1]                                            # flat
    b[700:900] = ref.f32_bits_to_bf16(rng.integers(0, 31, (200, H, D)).astype(np.float32) / 2)  # ties
    b[900:1000] = rng.integers(0, 128, (100, H, D)).astype(np.uint16)         # subnormals
    p = ref.Pools("int4", T // 16, H, 16, D)
    c = Cache(p)
    slots = np.arange(T, dtype=np.int32)
    c.write(cuda(b), cuda(b), cuda(slots))
    p.write(slots, b, b)
    torch.cuda.synchronize()
    c.same(p)


@pytest.mark.parametrize("P,D,H", [(16, 64, 1), (64, 128, 8), (32, 128, 3), (128, 64, 4)])
def test_int4_append_check_append_and_requant(cuda_device, P, D, H):
    rng = np.random.Generator(np.random.PCG64(P + D + H))
    B, MP, NP = 37, 6, 260
    table = rng.permutation(NP)[: B * MP].reshape(B, MP).astype(np.int32)
    lens = rng.integers(1, MP * P + 1, B).astype(np.int32)
    lens[:4] = [0, MP * P + 1, -3, MP * P]
    table[5] = -1
    table[6] = NP
    abort = (rng.random(B) < 0.2).astype(np.uint8)
    k, v = normal_bits(rng, (B, H, D)), normal_bits(rng, (B, H, D))

    def slot_of(skip):
        s = np.full(B, -1, np.int64)
        for i in range(B):
            if not skip[i] and 1 <= lens[i] <= MP * P:
                page = table[i, (lens[i] - 1) // P]
                s[i] = page * P + (lens[i] - 1) % P if 0 <= page < NP else -1
        return s

    p = ref.Pools("int4", NP, H, P, D, seed=2)
    c = Cache(p)
    pkv.kv_append_int4(cuda(k), cuda(v), cuda(table), cuda(lens), P, *c.pools, abort=cuda(abort))
    p.write(slot_of(abort), k, v)
    torch.cuda.synchronize()
    c.same(p)

    tags = rng.integers(0, 2**32, NP, dtype=np.uint64).astype(np.uint32)
    expected = tags[np.clip(table, 0, NP - 1)].copy()
    expected[10, 0] += np.uint32(1)
    want, n_want = oracle.kv_tag_check(tags, table, expected, lens, P)
    got = torch.full((B,), 9, dtype=torch.uint8, device="cuda")
    n = torch.full((1,), 9, dtype=torch.int32, device="cuda")
    pkv.kv_check_append_int4(cuda(tags), cuda(table), cuda(expected), cuda(lens), P, cuda(v),
                             cuda(k), *c.pools, got, n)
    p.write(slot_of(want), v, k)
    torch.cuda.synchronize()
    assert np.array_equal(got.cpu().numpy(), want) and int(n) == n_want
    c.same(p)

    src = normal_bits(rng, (5, H, P, D))
    ids = np.array([0, 4, 2, -1, 3, 5, 1], np.int32)
    to = np.array([7, 3, 0, 1, NP, 2, 255], np.int32)
    pkv.kv_requant_pages_int4(cuda(src), cuda(ids), c.k, c.kp, cuda(to))
    for s, d in zip(ids, to):
        if 0 <= s < 5 and 0 <= d < NP:
            p.k[d], p.kp[d] = ref.int4_pack(src[s])
    torch.cuda.synchronize()
    c.same(p)


# ---------------------------------------------------------------------------
# page tables
# ---------------------------------------------------------------------------

def run_tables(old, new, P, free, num_free, table, num_pages, tokens, tags=None, expected=None,
               in_place=False):
    B = table.shape[0]
    g = dict(table=cuda(table), slots=torch.full((tokens,), 77, dtype=torch.int32, device="cuda"),
             cu=torch.full((B + 1,), 77, dtype=torch.int32, device="cuda"),
             failed=torch.full((B,), 77, dtype=torch.uint8, device="cuda"))
    nf = torch.tensor([num_free], dtype=torch.int32, device="cuda")
    g["free"] = nf if in_place else torch.full((1,), 77, dtype=torch.int32, device="cuda")
    g["expected"] = None if expected is None else cuda(expected)
    pkv.kv_extend_tables(cuda(old), cuda(new), P, cuda(free), nf, g["table"], g["slots"], g["cu"],
                         g["failed"], g["free"], num_pages,
                         page_tags=None if tags is None else cuda(tags), expected_tags=g["expected"])
    torch.cuda.synchronize()
    return g


def same_tables(g, want):
    for k in ("table", "slots", "cu", "failed"):
        got = g[k].cpu().numpy()
        assert np.array_equal(got, want[k]), (k, np.argwhere(got != want[k])[:4])
    assert int(g["free"]) == want["free"]
    if want["expected"] is not None:
        assert np.array_equal(g["expected"].cpu().numpy().view(np.uint32), want["expected"])


@pytest.mark.parametrize("B", [1, 2, 31, 64, 511, 512, 513, 1500])
@pytest.mark.parametrize("seed", range(3))
def test_extend_tables_random(cuda_device, B, seed):
    """Rows that grow by nothing, one token and many; rows with bad lengths; too few free
    pages; bad ids in the table and on the stack; a short and a long slot map."""
    rng = np.random.Generator(np.random.PCG64(100 * seed + B))
    P = int(rng.choice([16, 32, 64, 128]))
    MP = int(rng.integers(1, 12))
    old = rng.integers(0, MP * P + 1, B)
    new = np.minimum(old + rng.integers(0, 3 * P, B) * rng.integers(0, 2, B), MP * P)
    wrong = rng.random(B) < 0.1
    old[wrong] = rng.integers(-5, MP * P, wrong.sum())
    new[wrong] = rng.integers(-5, MP * P + 40, wrong.sum())
    old, new = old.astype(np.int32), new.astype(np.int32)
    need = int(sum(max(0, -(-n // P) - -(-o // P)) for o, n in zip(old.tolist(), new.tolist())))
    NP = B * MP + need + 5
    cap = need + int(rng.integers(1, 5))
    free = rng.permutation(NP)[:cap].astype(np.int32)
    free[rng.random(cap) < 0.03] = rng.choice([-1, NP])
    table = rng.integers(-2, NP + 2, (B, MP)).astype(np.int32)
    num_free = [cap, int(need * 0.6), cap + 9][seed]
    tokens = int(sum(max(0, n - o) for o, n in zip(old.tolist(), new.tolist()) if o >= 0))
    tokens = max(0, tokens + [5, -3, 4099][seed])
    tags = rng.integers(0, 2**32, NP, dtype=np.uint64).astype(np.uint32)
    expected = rng.integers(0, 2**32, (B, MP), dtype=np.uint64).astype(np.uint32)
    want = ref.extend_tables(old, new, P, free, num_free, table, NP, tokens, tags, expected)
    same_tables(run_tables(old, new, P, free, num_free, table, NP, tokens, tags, expected,
                           in_place=seed == 1), want)


def test_extend_tables_long_rows_and_sums_past_32_bits(cuda_device):
    """A long prefill, and lengths whose sums pass 2^31: later rows keep their flags."""
    big = 2**31 - 1
    old = np.array([0, 3, big - 5, 0, 7, 8], np.int32)
    new = np.array([70001, 3, big, big, big, 9], np.int32)
    P, MP, NP = 16, 4400, 5000
    free = np.arange(NP, dtype=np.int32)
    table = np.full((6, MP), 11, np.int32)
    want = ref.extend_tables(old, new, P, free, NP, table, NP, 70100)
    assert want["failed"].tolist() == [0, 0, 1, 1, 1, 0]
    same_tables(run_tables(old, new, P, free, NP, table, NP, 70100), want)


def test_extend_tables_empty_batch_and_no_slots(cuda_device):
    z = np.zeros(0, np.int32)
    g = run_tables(z, z, 16, np.arange(4, dtype=np.int32), 3, np.zeros((0, 2), np.int32), 9, 6)
    assert int(g["free"]) == 3 and g["cu"].tolist() == [0] and g["slots"].tolist() == [-1] * 6
    old, new = np.array([0], np.int32), np.array([17], np.int32)
    g = run_tables(old, new, 16, np.array([5, 6], np.int32), 2, np.zeros((1, 2), np.int32), 9, 0)
    assert g["table"].tolist() == [[6, 5]] and g["cu"].tolist() == [0, 17] and int(g["free"]) == 0


def test_extend_tables_unaligned_slot_map(cuda_device):
    """The slot map as a part of a larger buffer, at every 4-byte offset; words around it stay."""
    old, new = np.array([5, 0, 30], np.int32), np.array([40, 21, 31], np.int32)
    free, table = np.arange(8, dtype=np.int32), np.arange(9, dtype=np.int32).reshape(3, 3)
    want = ref.extend_tables(old, new, 16, free, 8, table, 9, 60)
    for at in range(4):
        buf = torch.full((70,), 55, dtype=torch.int32, device="cuda")
        nf = torch.tensor([8], dtype=torch.int32, device="cuda")
        cu = torch.zeros(4, dtype=torch.int32, device="cuda")
        failed = torch.zeros(3, dtype=torch.uint8, device="cuda")
        pkv.kv_extend_tables(cuda(old), cuda(new), 16, cuda(free), nf, cuda(table),
                             buf[at: at + 60], cu, failed, nf, 9)
        got = buf.cpu().numpy()
        assert np.array_equal(got[at: at + 60], want["slots"])
        assert (got[:at] == 55).all() and (got[at + 60:] == 55).all()


# ---------------------------------------------------------------------------
# tag check with a window
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("window,sinks", [(1, 0), (17, 3), (64, 16), (40, 40), (10**6, 2), (5, 10**6)])
def test_tag_check_window(cuda_device, window, sinks):
    rng = np.random.Generator(np.random.PCG64(window % 1000 + sinks % 1000))
    B, MP, P, NP = 300, 12, 16, 500
    tags = rng.integers(0, 2**32, NP, dtype=np.uint64).astype(np.uint32)
    table = rng.integers(0, NP, (B, MP)).astype(np.int32)
    table[rng.random((B, MP)) < 0.03] = -1
    expected = tags[np.clip(table, 0, NP - 1)].copy()
    expected[rng.random((B, MP)) < 0.03] += np.uint32(1)
    lens = rng.integers(-2, MP * P + 3, B).astype(np.int32)
    want = np.zeros(B, np.uint8)
    for b in range(B):
        L = int(lens[b])
        if not 1 <= L <= MP * P:
            want[b] = 1
            continue
        for j in np.unique(ref.visible(L, window, sinks) // P):
            if table[b, j] < 0 or tags[table[b, j]] != expected[b, j]:
                want[b] = 1
    got = torch.full((B,), 9, dtype=torch.uint8, device="cuda")
    n = torch.zeros(1, dtype=torch.int32, device="cuda")
    pkv.kv_tag_check_window(cuda(tags), cuda(table), cuda(expected), cuda(lens), P, window, sinks,
                            got, n)
    torch.cuda.synchronize()
    assert np.array_equal(got.cpu().numpy(), want) and int(n) == want.sum()


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------

def attention_case(kind, lens, G, H, D, P, seed, spare=3, extra_pages=2):
    rng = np.random.Generator(np.random.PCG64(seed))
    lens = np.asarray(lens, np.int32)
    B = lens.size
    used = [max(0, -(-int(n) // P)) if n < 10**5 else 0 for n in lens]
    MP = max(used) + extra_pages
    NP = sum(used) + spare
    perm = rng.permutation(NP).astype(np.int32)
    table = np.full((B, MP), -1, np.int32)
    at = 0
    for i, n in enumerate(used):
        table[i, :n] = perm[at: at + n]
        at += n
    p = ref.Pools(kind, NP, H, P, D, 0.13, 0.17, seed=seed)
    q = ref.f32_bits_to_bf16(rng.standard_normal((B, H * G, D)).astype(np.float32))
    return p, q, table, lens


def run_attention(p, q, table, lens, window=0, sinks=0, abort=None, ctas=(0,)):
    c = Cache(p)
    B, Hq, D = q.shape
    sm = D ** -0.5
    want = ref.attend(q, p, table, lens, sm, window, sinks, abort)
    for n in ctas:
        ws = c.workspace(B, Hq, n)
        out, lse = c.attend(cuda(q), cuda(table), cuda(lens), sm, ws, window, sinks,
                            None if abort is None else cuda(abort), n)
        torch.cuda.synchronize()
        assert pkv.workspace_status(ws) == 0
        ref.check_attention(values(out), values(lse), want, f"ctas={n}")


SHAPES = [  # G, H, D, P
    (8, 8, 128, 64), (1, 1, 64, 16), (8, 2, 64, 32), (16, 1, 128, 16), (12, 2, 64, 128),
    (3, 3, 128, 32), (5, 4, 128, 128), (1, 2, 64, 64),
]


@pytest.mark.parametrize("G,H,D,P", SHAPES)
def test_int4_attention(cuda_device, G, H, D, P):
    lens = [1, 2, P - 1, P, P + 1, 63, 64, 65, 700, 0, -4, 333]
    p, q, table, lens = attention_case("int4", lens, G, H, D, P, seed=G * H + D)
    abort = np.zeros(len(lens), np.uint8)
    abort[[3, 8]] = 1
    table[4, 0] = p.shape[0]          # a page outside the pool
    run_attention(p, q, table, lens, abort=abort, ctas=(0, 1, 7, 148, -1, -2, -8))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("G,H,D,P", SHAPES)
def test_window_attention(cuda_device, kind, G, H, D, P):
    lens = [1, 5, P, 130, 131, 64, 400, 0, 257, 700]
    p, q, table, lens = attention_case(kind, lens, G, H, D, P, seed=G + H + D)
    abort = np.zeros(len(lens), np.uint8)
    abort[3] = 1
    for window, sinks, ctas in ((1, 0, (0, 5)), (100, 4, (0, 1, 19, -2)), (64, 64, (0,)),
                                (17, 200, (0, -4)), (640, 1, (0, 148)), (5000, 3, (0,))):
        run_attention(p, q, table, lens, window, sinks, abort, ctas)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D,P", [(128, 16), (64, 64), (128, 128)])
def test_window_hides_pages_and_values(cuda_device, kind, D, P):
    """Hidden page ids of any value and hidden values of NaN change nothing."""
    p, q, table, lens = attention_case(kind, [500, 321, 64, 30], 4, 2, D, P, seed=8)
    window, sinks = 70, 5
    nan = {"int4": 0, "fp8": 0x7F, "bf16": 0x7FC0}[kind]
    for b, L in enumerate(lens):
        seen = set(ref.visible(int(L), window, sinks).tolist())
        for j in range(-(-int(L) // P)):
            toks = range(j * P, min((j + 1) * P, int(L)))
            hid = [t for t in toks if t not in seen]
            for t in hid:
                page, o = table[b, j], t % P
                p.k[page, :, o], p.v[page, :, o] = nan, nan
                if p.kp is not None:
                    p.kp[page, :, o], p.vp[page, :, o] = 0x7FC0, 0x7F80
        for j in range(-(-int(L) // P)):
            toks = range(j * P, min((j + 1) * P, int(L)))
            if not any(t in seen for t in toks):
                table[b, j] = [-1, 10**6, -2**31][j % 3]
    run_attention(p, q, table, lens, window, sinks, ctas=(0, 1, 33, -2))
    # a visible entry that names no page kills the request
    table[0, (int(lens[0]) - 1) // P] = -1
    run_attention(p, q, table, lens, window, sinks)


@pytest.mark.parametrize("kind", ("int4",))
@pytest.mark.parametrize("D", [64, 128])
def test_int4_attention_special_values(cuda_device, kind, D):
    """A NaN token makes its head's outputs NaN and nothing else; scales of very different
    sizes, zero scales, large and tiny queries."""
    P, H = 16, 2
    p, q, table, lens = attention_case(kind, [200, 77, 300, 40], 4, H, D, P, seed=3)
    rng = np.random.Generator(np.random.PCG64(5))
    # request 0: a NaN group of K in head 1, token 150; request 1: of V, head 0, last group
    p.kp[table[0, 150 // P], 1, 150 % P, 0] = 0x7FC0
    p.vp[table[1, 70 // P], 0, 70 % P, -1] = 0x7FC0
    # request 2: V's scales over 60 powers of two, and zero ones
    for j in range(-(-300 // P)):
        e = rng.integers(-40, 20, (H, P, D // 64))
        p.vp[table[2, j], :, :, :, 0] = ref.f32_bits_to_bf16(np.exp2(e).astype(np.float32))
        p.vp[table[2, j], :, 0, :, 0] = 0
    q[3] = ref.f32_bits_to_bf16((ref.bf16(q[3]) * 2.0 ** -100).astype(np.float32))
    run_attention(p, q, table, lens, ctas=(0, 1, 20, -2))
    q[2] = 0
    run_attention(p, q, table, lens, window=33, sinks=2)


def test_int4_attention_long_request(cuda_device):
    """One request of 40,001 tokens over every split, and with a window over most of it."""
    p, q, table, lens = attention_case("int4", [40001], 8, 2, 128, 64, seed=6)
    run_attention(p, q, table, lens, ctas=(0, 1, 148, 296, -16))
    run_attention(p, q, table, lens, window=30011, sinks=100, ctas=(0, 296, -8))


def test_int4_work_split_choice(cuda_device):
    """Short requests: one launch, clusters of one CTA; long ones on few items: split-K.
    The choice is one of the splits that the other tests run."""
    size, ctas, launches = pkv.paged_decode_attn_plan(pkv.PKV_KV_INT4, 128, 64, 8, 128, 1, 16)
    assert (size, launches) == (1, 1) and ctas >= 128
    size, ctas, launches = pkv.paged_decode_attn_plan(pkv.PKV_KV_INT4, 2, 32, 8, 128, 1024, 128)
    assert (size, launches) == (0, 2) and ctas >= 148


@pytest.mark.parametrize("kind", KINDS)
def test_attention_of_a_batch_without_requests(cuda_device, kind):
    """Every request padded (length 0) or invalid, by every work split: dead outputs, and
    the calls around it keep their order."""
    p, q, table, lens = attention_case(kind, [0, -1, 0, 10**6, 0], 4, 2, 64, 16, seed=2,
                                       extra_pages=3, spare=9)
    c = Cache(p)
    gq, gt, gl = cuda(q), cuda(table[:, :3].copy()), cuda(lens)
    for window in (0, 20):
        for n in (0, 1, 40, -1, -2):
            out, lse = c.attend(gq, gt, gl, 0.1, c.workspace(5, 8, n), window, 2 if window else 0,
                                num_ctas=n) if kind == "int4" or window else (None, None)
            if out is not None:
                torch.cuda.synchronize()
                assert not out.any() and torch.isneginf(lse).all()


@pytest.mark.parametrize("kind", ["int4", "bf16"])
def test_offsets_past_32_bits(cuda_device, kind):
    """A pool whose code bytes (INT4: parameter bytes too) pass 2^32 and 2^31: the last
    pages are written, read and attended to."""
    H, P, D = 8, 128, 128
    NP = {"int4": 2**32 // (H * P * D // 2) + 40, "bf16": 2**32 // (H * P * D * 2) + 40}[kind]
    small = ref.Pools(kind, 40, H, P, D, seed=9)
    big = {n: torch.zeros((NP, *getattr(small, n).shape[1:]), device="cuda",
                          dtype=torch.uint8 if getattr(small, n).dtype == np.uint8 else torch.bfloat16)
           for n in ("k", "v", "kp", "vp") if getattr(small, n) is not None}
    for n, t in big.items():
        t[NP - 40:] = cuda(getattr(small, n))
    c = Cache.__new__(Cache)
    c.p, c.k, c.v, c.kp, c.vp = small, big["k"], big["v"], big.get("kp"), big.get("vp")
    rng = np.random.Generator(np.random.PCG64(1))
    T = 300
    at = rng.permutation(40 * P)[:T].astype(np.int32)
    k, v = normal_bits(rng, (T, H, D)), normal_bits(rng, (T, H, D))
    c.write(cuda(k), cuda(v), cuda(at + (NP - 40) * P))
    small.write(at, k, v)
    back = [torch.empty((T, H, D), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    c.read(cuda(at + (NP - 40) * P), *back)
    for got, want in zip(back, small.read(at)):
        assert np.array_equal(values(got), ref.bf16(oracle.bf16_from_double(want)))
    table = rng.permutation(40)[:30].reshape(3, 10).astype(np.int32)
    lens = np.array([1280, 999, 5], np.int32)
    q = ref.f32_bits_to_bf16(rng.standard_normal((3, 2 * H, D)).astype(np.float32))
    for window, sinks in ((0, 0), (300, 7)):
        want = ref.attend(q, small, table, lens, 0.09, window, sinks)
        out, lse = c.attend(cuda(q), cuda(table + NP - 40), cuda(lens), 0.09, c.workspace(3, 2 * H),
                            window, sinks)
        torch.cuda.synchronize()
        ref.check_attention(values(out), values(lse), want)


# ---------------------------------------------------------------------------
# a run of them together
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("kind", KINDS)
def test_prefill_and_decode_steps(cuda_device, kind):
    """A prefill chunk and then decode steps, captured once as a graph and replayed on new
    inputs: lengths -> tables and slots -> write -> check -> windowed and full attention."""
    B, H, G, D, P, MP, NP = 5, 2, 4, 128, 16, 20, 90
    rng = np.random.Generator(np.random.PCG64(17))
    p = ref.Pools(kind, NP, H, P, D, 0.1, 0.1, seed=3)
    c = Cache(p)
    tags = rng.integers(0, 2**32, NP, dtype=np.uint64).astype(np.uint32)
    free = rng.permutation(NP).astype(np.int32)
    table, expected = np.full((B, MP), -1, np.int32), np.zeros((B, MP), np.uint32)
    old, new = np.zeros(B, np.int32), np.array([70, 1, 33, 160, 16], np.int32)
    T, num_free = 400, NP
    g_old, g_new = cuda(old), cuda(new)
    g_table, g_exp, g_tags, g_free = cuda(table), cuda(expected), cuda(tags), cuda(free)
    nf = torch.tensor([NP], dtype=torch.int32, device="cuda")
    slots = torch.zeros(T, dtype=torch.int32, device="cuda")
    cu, failed = torch.zeros(B + 1, dtype=torch.int32, device="cuda"), torch.zeros(B, dtype=torch.uint8, device="cuda")
    gk, gv = (torch.zeros((T, H, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    gq = torch.zeros((B, H * G, D), dtype=torch.bfloat16, device="cuda")
    abort, n_abort = torch.zeros(B, dtype=torch.uint8, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    ws, ws2 = c.workspace(B, H * G), c.workspace(B, H * G)
    outs = [(torch.zeros((B, H * G, D), dtype=torch.bfloat16, device="cuda"),
             torch.zeros((B, H * G), device="cuda")) for _ in range(2)]

    def step():
        pkv.kv_extend_tables(g_old, g_new, P, g_free, nf, g_table, slots, cu, failed, nf, NP,
                             page_tags=g_tags, expected_tags=g_exp)
        c.write(gk, gv, slots)
        pkv.kv_tag_check(g_tags, g_table, g_exp, g_new, P, abort, n_abort)
        c.attend(gq, g_table, g_new, 0.08, ws, abort=abort, out=outs[0])
        c.attend(gq, g_table, g_new, 0.08, ws2, 25, 3, abort, out=outs[1])

    graph = None
    for it in range(6):
        k, v = normal_bits(rng, (T, H, D)), normal_bits(rng, (T, H, D))
        q = normal_bits(rng, (B, H * G, D))
        for dst, src in ((gk, k), (gv, v), (gq, q), (g_old, old), (g_new, new)):
            dst.copy_(cuda(src))
        if it == 2:
            # (capture runs nothing)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
        if graph is None:
            step()
        else:
            graph.replay()
        torch.cuda.synchronize()
        want = ref.extend_tables(old, new, P, free, num_free, table, NP, T, tags, expected)
        table, expected, num_free = want["table"], want["expected"], want["free"]
        assert np.array_equal(g_table.cpu().numpy(), table) and int(nf) == num_free
        assert np.array_equal(slots.cpu().numpy(), want["slots"]) and not abort.any()
        p.write(want["slots"], k, v)
        c.same(p)
        for (o, l), (w, s) in zip(outs, ((0, 0), (25, 3))):
            ref.check_attention(values(o), values(l), ref.attend(q, p, table, new, 0.08, w, s), f"step {it}")
        old = new.copy()
        new = new + rng.integers(0, 3, B).astype(np.int32)


@pytest.mark.parametrize("kind", KINDS)
def test_two_streams_with_their_own_workspaces(cuda_device, kind):
    """Calls on two streams at once, on streams that are not the current one."""
    p, q, table, lens = attention_case(kind, [300, 40, 900], 8, 2, 128, 64, seed=21)
    c = Cache(p)
    want = [ref.attend(q, p, table, lens, 0.1, w, 2 if w else 0) for w in (0, 90)]
    gq, gt, gl = cuda(q), cuda(table), cuda(lens)
    streams = [torch.cuda.Stream() for _ in range(2)]
    wss = [c.workspace(3, 16) for _ in range(2)]
    outs = [(torch.zeros_like(gq), torch.zeros((3, 16), device="cuda")) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for i, w in enumerate((0, 90)):
            with torch.cuda.stream(streams[i]):
                if kind != "int4" and w == 0:
                    c.attend(gq, gt, gl, 0.1, wss[i], out=outs[i])
                else:
                    c.attend(gq, gt, gl, 0.1, wss[i], w, 2 if w else 0, out=outs[i])
    torch.cuda.synchronize()
    for (o, l), w in zip(outs, want):
        ref.check_attention(values(o), values(l), w)


def test_binding_refuses(cuda_device):
    p, q, table, lens = attention_case("int4", [30, 20], 2, 2, 64, 16, seed=1)
    c = Cache(p)
    ws = c.workspace(2, 4)
    gq, gt, gl = cuda(q), cuda(table), cuda(lens)
    with pytest.raises(ValueError, match="out must be"):
        c.attend(gq, gt, gl, 0.1, ws, out=(torch.zeros((2, 3, 64), dtype=torch.bfloat16, device="cuda"),
                                           torch.zeros((2, 4), device="cuda")))
    with pytest.raises(pkv.PagedKVError, match="workspace"):
        c.attend(gq, gt, gl, 0.1, ws[:256])
    with pytest.raises(pkv.PagedKVError, match="window"):
        c.attend(gq, gt, gl, 0.1, ws, window=-1)
    with pytest.raises(ValueError, match="k_params must be"):
        pkv.paged_decode_attn_int4(gq, c.k, c.kp[:1], c.v, c.vp, gt, gl, 0.1,
                                   torch.empty_like(gq), torch.empty((2, 4), device="cuda"), ws)
    rows = torch.zeros((3, 2, 64), dtype=torch.bfloat16, device="cuda")
    s = torch.zeros(3, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="contiguously"):
        c.write(rows.transpose(1, 2).contiguous().transpose(1, 2), rows, s)
    with pytest.raises(ValueError, match="must be"):
        c.write(rows[:2], rows, s)
    with pytest.raises(pkv.PagedKVError, match="aligned"):
        off = torch.zeros(3 * 128 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(3, 2, 64)
        c.write(off, off, s)
    with pytest.raises(ValueError, match="together"):
        run_tables(np.zeros(1, np.int32), np.ones(1, np.int32), 16, np.zeros(1, np.int32), 1,
                   np.zeros((1, 1), np.int32), 4, 1, tags=np.zeros(4, np.uint32))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("between", [False, True])
def test_attention_sees_the_tables_of_the_call_before(cuda_device, kind, between):
    """Tables, (a slot write,) and attention back to back, with no synchronisation: the
    attention kernel may be scheduled early but must not read rows from before.  Both
    of two states are attended to in turn, and compared with the same call made alone."""
    B, H, D, P, NP = 48, 2, 64, 16, 1600
    rng = np.random.Generator(np.random.PCG64(2))
    p = ref.Pools(kind, NP, H, P, D, 0.1, 0.1, seed=11)
    c = Cache(p)
    old, new = np.zeros(B, np.int32), rng.integers(300, 500, B).astype(np.int32)
    MP, T = 32, int(new.sum())
    assert -(-new // P).sum() <= NP
    stacks = [cuda(rng.permutation(NP).astype(np.int32)) for _ in range(2)]
    nf, nfo = (torch.tensor([NP], dtype=torch.int32, device="cuda") for _ in range(2))
    table = torch.full((B, MP), -1, dtype=torch.int32, device="cuda")
    slots = torch.zeros(T, dtype=torch.int32, device="cuda")
    cu_tokens, failed = torch.zeros(B + 1, dtype=torch.int32, device="cuda"), torch.zeros(B, dtype=torch.uint8, device="cuda")
    g_old, g_new, q = cuda(old), cuda(new), cuda(normal_bits(rng, (B, 2 * H, D)))
    rows = torch.zeros((1, H, D), dtype=torch.bfloat16, device="cuda")
    nowhere = torch.full((1,), -1, dtype=torch.int32, device="cuda")
    ws = c.workspace(B, 2 * H)

    def tables(i):
        pkv.kv_extend_tables(g_old, g_new, P, stacks[i], nf, table, slots, cu_tokens, failed, nfo, NP)

    want = []
    for i in range(2):
        tables(i)
        torch.cuda.synchronize()
        want.append([t.clone() for t in c.attend(q, table, g_new, 0.1, ws)])
        torch.cuda.synchronize()
    outs = [tuple(torch.zeros_like(t) for t in want[0]) for _ in range(40)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()   # (replayed, the kernels follow one another at once)
    with torch.cuda.graph(graph):
        for n, out in enumerate(outs):
            tables(n % 2)
            if between:
                c.write(rows, rows, nowhere)
            c.attend(q, table, g_new, 0.1, ws, out=out)
    graph.replay()
    torch.cuda.synchronize()
    for n, out in enumerate(outs):
        for got, w in zip(out, want[n % 2]):
            assert torch.equal(got, w), f"call {n}"
