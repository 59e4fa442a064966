"""GPU parity of the paged 4-bit KV cache (append with rotary embedding, gather, page copies) and of attention over it,
against float64 (kv_reference.py).

Tolerances.  Codes and scales are bit-exact: x / s of fp16 values is a half-integer exactly or at least 2^-13 (relative)
away from one, and -min / 7 at least 2^-15 away from an fp16 rounding boundary, both far above an fp32 rounding.
A gathered value is the exact product rounded once to fp16.  A rotated value: cos and sin rounded to fp32, two products and
a sum rounded in fp32 stay within 2^-22 (|x| + |y|), then half an fp16 step.
Attention: the weights are rounded to fp16 before and after V's scale (2^-11 each: 2^-10 of sum w |v|); scores carry an
absolute error e from their fp32 arithmetic, (D / 32 + 2) 2^-24 times sum |q (code) s| and 2^-24 |s| (in the exponent's
units, here below 64), which moves weights by 2 e ln 2 < 2^-14: together (2^-10 + 2^-14) sum w |v|.  Products
weight * V scale below fp16's normal range are off by up to 2^-25, times |code - 7| <= 8, with the largest weight at 2^9 or
more (at 1 or more from the first V scale of 2 on): 2^-31 (2^-22) a token; weights themselves there by 2^-34 (2^-25) of |v|.
Then half an fp16 step of the result (2^-11, or 2^-25 for subnormals)."""
import numpy as np
import pytest

import kv_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def zt():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from int4_group_quantized_q4f16_b200 import zt_q4
    return zt_q4


def cuda(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def fp16(rng, *shape, by=1.0):
    return (rng.standard_normal(shape) * by).astype(np.float16)


def same_bytes(cache, pool):
    got = cache.pages[0].cpu().numpy().reshape(pool.raw.shape)
    bad = np.argwhere(got != pool.raw)
    assert not len(bad), f"{len(bad)} bytes differ, first at (page, head, tile, byte) {bad[:5].tolist()}: " \
                         f"{[(int(got[tuple(i)]), int(pool.raw[tuple(i)])) for i in bad[:5]]}"


def tables(rng, lens, page, spare=2):
    """A page table in random order and the number of pages; entries behind a sequence's pages are out of range."""
    width = [-(-n // page) for n in lens]
    order = rng.permutation(sum(width) + spare)
    table = np.full((len(lens), max(max(width), 1)), 2**31 - 1, np.int32)
    at = 0
    for b, w in enumerate(width):
        table[b, :w] = order[at:at + w]
        at += w
    return table, sum(width) + spare


def filled(zt, rng, lens, page, heads, D, k_by=1.0, v_by=1.0, edit=None):
    """A cache holding random rows, written by the reference into random bytes."""
    table, n = tables(rng, lens, page)
    raw = rng.integers(0, 256, (n, zt.kv_page_bytes(page, heads, D)), dtype=np.uint8)
    pool = ref.Pool(raw, page, heads, D)
    for b, m in enumerate(lens):
        for p in range(m):
            k, v = fp16(rng, heads, D, by=k_by), fp16(rng, heads, D, by=v_by)
            if edit:
                edit(b, p, k, v)
            pool.write(table[b, p // page], p % page, k, v)
    return zt.KvCache(cuda(raw), page, heads, D), pool, table


def check_attention(zt, cache, pool, q, lens, table, scale=None, large_v=False, **more):
    import torch
    tokens, D = q.shape[1], q.shape[3]
    plan = zt.KvAttention(cache, cuda(q), cuda(np.asarray(lens, np.int32)), cuda(table), scale=scale, **more)
    got = plan.run().cpu().numpy()
    again = plan.run().clone()
    torch.cuda.synchronize()
    assert cache.errors() == 0
    assert np.array_equal(again.cpu().numpy().view(np.uint16), got.view(np.uint16)), "two runs differ"
    for b, n in enumerate(lens):
        k, v = pool.values(table[b, :-(-n // pool.page)], n)
        with np.errstate(all="ignore"):
            want, mag = ref.attention(q[b], k, v, [n - tokens + 1 + i for i in range(tokens)], scale or D ** -0.5)
        top = np.nanmax(np.abs(v), initial=0.0)
        tol = (2.0**-10 + 2.0**-14) * mag + 2.0**-11 * np.abs(want) + 2.0**-25 + n * 2.0**(0 if large_v else -9) * (2.0**-22 + 2.0**-25 * top)
        assert np.array_equal(np.isnan(got[b]), np.isnan(want)), f"sequence {b}: NaN in other places"
        fine = ~np.isnan(want)
        err = np.abs(got[b].astype(np.float64) - want)
        assert (err <= tol)[fine].all(), (b, n, float((err - tol)[fine].max()), float(err[fine].max()))
    return got


# ------------------------------------------------------------- append, gather --
@pytest.mark.parametrize("D,heads,page", [(64, 3, 16), (96, 32, 64), (128, 8, 32), (128, 1, 1024)])
def test_append_is_bit_exact_and_gathers_back(zt, D, heads, page):
    rng = np.random.default_rng(D + heads)
    lens = [1, 16, 37, 2 * page + 5 if page < 100 else 40, 0, 8]
    table, n = tables(rng, lens, page)
    raw = rng.integers(0, 256, (n, zt.kv_page_bytes(page, heads, D)), dtype=np.uint8)
    want = ref.Pool(raw.copy(), page, heads, D)
    cache = zt.KvCache(cuda(raw), page, heads, D)
    places = [(b, p) for b, m in enumerate(lens) for p in range(m)]
    rng.shuffle(places)
    places = places[:-7] + [(0, -1), (99, -1)] + places[-7:]            # padding rows, and a second call
    rows = len(places)
    # values of every kind: zeros, ties, one-sided groups, subnormals, the largest
    x = fp16(rng, rows, 2 * heads + 1, D)
    x[1] = 0
    x[2] = np.float16(-1.5)
    x[3] = np.abs(x[3])
    x[4] *= np.float16(6e-8)
    x[5] = np.float16(65504) * np.sign(x[5])
    x[6] = np.rint(x[6] * 4) / 4
    x[7, :, :32] = np.inf
    x[8, :, 33] = np.nan
    seq, pos = (np.array(c, np.int32) for c in zip(*places))
    dev, (sd, pd, td) = cuda(x), (cuda(a) for a in (seq, pos, table))
    for part in (slice(0, rows - 7), slice(rows - 7, rows)):
        zt.KvAppend(cache, dev[part, :heads], dev[part, heads:2 * heads], sd[part], pd[part], td).run()
    for i, (b, p) in enumerate(places):
        if p >= 0:
            want.write(table[b, p // page], p % page, x[i, :heads], x[i, heads:2 * heads])
    same_bytes(cache, want)
    k, v = zt.KvGather(cache, sd, pd, td, k=cuda(np.full((rows, heads, D), 9, np.float16))).run()
    k, v = k.cpu().numpy(), v.cpu().numpy()
    assert cache.errors() == 0
    for i, (b, p) in enumerate(places):
        if p < 0:
            assert (k[i] == 9).all()
            continue
        wk, wv = (ref.dequantize(*ref.quantize(y)).astype(np.float16) for y in (x[i, :heads], x[i, heads:2 * heads]))
        assert np.array_equal(k[i], wk, equal_nan=True) and np.array_equal(v[i], wv, equal_nan=True), i


@pytest.mark.parametrize("D,heads,page,where", [(64, 2, 16, "in order"), (96, 3, 32, "in order"), (128, 1, 64, "in order"),
                                                 (96, 2, 16, "backwards"), (96, 2, 16, "two by two"), (64, 1, 48, "gaps")])
def test_append_runs(zt, D, heads, page, where):
    """Rows as prompts and steps bring them: runs of consecutive positions that start and end anywhere in a tile and in a
    window of rows, runs that touch, padding inside them, rows of a tile in other orders."""
    rng = np.random.default_rng(D + heads + len(where))
    spans = [(0, 40), (3, 4), (12, 45), (5, 5), (31, 33), (9, 25), (15, 17), (2, 50), (0, 16), (7, 8), (16, 79)]
    places = [(b, p) for b, (lo, hi) in enumerate(spans) for p in range(lo, hi)]
    if where == "backwards":
        places = places[::-1]
    elif where == "two by two":
        places = [x for i in range(0, len(places), 4) for x in places[i + 2:i + 4] + places[i:i + 2]]
    elif where == "gaps":
        places = [(b, p if rng.random() < 0.8 else -1) for b, p in places]
    table, n = tables(rng, [hi for _, hi in spans], page)
    raw = rng.integers(0, 256, (n, zt.kv_page_bytes(page, heads, D)), dtype=np.uint8)
    want, cache, rows = ref.Pool(raw.copy(), page, heads, D), zt.KvCache(cuda(raw), page, heads, D), len(places)
    x = fp16(rng, rows, 2 * heads, D)
    seq, pos = (np.array(c, np.int32) for c in zip(*places))
    dev, (sd, pd, td) = cuda(x), (cuda(a) for a in (seq, pos, table))
    zt.KvAppend(cache, dev[:, :heads], dev[:, heads:], sd, pd, td).run()
    for i, (b, p) in enumerate(places):
        if p >= 0:
            want.write(table[b, p // page], p % page, x[i, :heads], x[i, heads:])
    same_bytes(cache, want)
    k, v = (t.cpu().numpy() for t in zt.KvGather(cache, sd, pd, td, k=cuda(np.full((rows, heads, D), 9, np.float16)),
                                                 v=cuda(np.full((rows, heads, D), 9, np.float16))).run())
    assert cache.errors() == 0
    for i, (b, p) in enumerate(places):
        wk, wv = (ref.dequantize(*ref.quantize(y)).astype(np.float16) if p >= 0 else np.full((heads, D), 9, np.float16)
                  for y in (x[i, :heads], x[i, heads:]))
        assert np.array_equal(k[i], wk) and np.array_equal(v[i], wv), (i, b, p)


@pytest.mark.parametrize("D,heads,q_heads", [(64, 2, 6), (96, 32, 32), (128, 8, 32)])
def test_append_rotates(zt, D, heads, q_heads):
    rng = np.random.default_rng(D)
    rows, page, theta = 21, 16, 10000.0
    pos = np.array([0, 1, 2, 131071, 2**20 + 3] + list(range(100, 100 + rows - 5)), np.int32)
    # every row a sequence of its own whose table points the pages it needs at one page
    table = np.repeat(np.arange(rows, dtype=np.int32)[:, None], int(pos.max()) // page + 1, 1)
    raw = rng.integers(0, 256, (rows, zt.kv_page_bytes(page, heads, D)), dtype=np.uint8)
    want = ref.Pool(raw.copy(), page, heads, D)
    cache = zt.KvCache(cuda(raw), page, heads, D)
    x = fp16(rng, rows, q_heads + 2 * heads, D)
    dev = cuda(x)
    q, k = zt.KvAppend(cache, dev[:, q_heads:q_heads + heads], dev[:, q_heads + heads:], cuda(np.arange(rows, dtype=np.int32)),
                       cuda(pos), cuda(table), q=dev[:, :q_heads], theta=theta).run()
    q, k = q.cpu().numpy(), k.cpu().numpy()
    assert cache.errors() == 0
    half = D // 2
    for got, src in ((q, x[:, :q_heads]), (k, x[:, q_heads:q_heads + heads])):
        exact = ref.rotate(src, pos, theta)
        mag = np.abs(src.astype(np.float64))
        mag = mag + np.concatenate([mag[..., half:], mag[..., :half]], -1)
        assert (np.abs(got - exact) <= 2.0**-11 * np.abs(exact) + 2.0**-25 + 2.0**-22 * mag).all()
    assert np.array_equal(q[0], x[0, :q_heads]) and np.array_equal(k[0], x[0, q_heads:q_heads + heads])   # position 0
    for i in range(rows):
        want.write(i, pos[i] % page, k[i], x[i, q_heads + heads:])
    same_bytes(cache, want)


def test_append_reports_places_out_of_range(zt):
    """Bad pages, positions and sequences set the error bit and write nothing; the other rows are stored."""
    rng = np.random.default_rng(5)
    page, heads, D = 16, 2, 64
    table = np.array([[1, -1], [7, 0]], np.int32)              # -1 and 7 are not pages of a pool of 4
    raw = rng.integers(0, 256, (4, zt.kv_page_bytes(page, heads, D)), dtype=np.uint8)
    want = ref.Pool(raw.copy(), page, heads, D)
    cache = zt.KvCache(cuda(raw), page, heads, D)
    seq = np.array([0, 0, 1, 1, 0, 2, -1], np.int32)
    pos = np.array([3, 16, 0, 17, 32, 0, 0], np.int32)
    k, v = fp16(rng, 7, heads, D), fp16(rng, 7, heads, D)
    args = cuda(seq), cuda(pos), cuda(table)
    zt.KvAppend(cache, cuda(k), cuda(v), *args).run()
    assert cache.errors() == zt.ZT_Q4_KV_ERR_PLACE
    want.write(1, 3, k[0], v[0])
    want.write(0, 1, k[3], v[3])
    same_bytes(cache, want)
    cache.clear_errors()
    assert cache.errors() == 0
    gk, _ = zt.KvGather(cache, *args, k=cuda(np.full((7, heads, D), 9, np.float16))).run()
    assert cache.errors() == zt.ZT_Q4_KV_ERR_PLACE
    assert [(gk[i] == 9).all().item() for i in range(7)] == [False, True, True, False, True, True, True]


def test_offsets_beyond_32_bits(zt):
    """Pages behind the first 4 GiB of a pool: append, gather, attention and copies reach them."""
    import torch
    page, heads, D = 1024, 32, 128
    size = zt.kv_page_bytes(page, heads, D)
    n = (5 << 30) // size
    cache = zt.KvCache(torch.zeros((n, size), dtype=torch.uint8, device="cuda"), page, heads, D)
    rng = np.random.default_rng(1)
    k, v = fp16(rng, 3, heads, D), fp16(rng, 3, heads, D)
    table = cuda(np.array([[n - 1], [n - 2]], np.int32))
    seq, pos = cuda(np.zeros(3, np.int32)), cuda(np.array([0, 1, 2], np.int32))
    zt.KvAppend(cache, cuda(k), cuda(v), seq, pos, table).run()
    zt.KvCopy(cache, cuda(np.array([n - 1], np.int32)), cuda(np.array([n - 2], np.int32))).run()
    for b in (0, 1):
        gk, gv = zt.KvGather(cache, seq + b, pos, table).run()
        assert np.array_equal(gk.cpu().numpy(), ref.dequantize(*ref.quantize(k)).astype(np.float16))
        assert np.array_equal(gv.cpu().numpy(), ref.dequantize(*ref.quantize(v)).astype(np.float16))
    q = cuda(fp16(rng, 2, 1, heads, D))
    q[1] = q[0]
    out = zt.KvAttention(cache, q, cuda(np.array([3, 3], np.int32)), table).run()
    torch.cuda.synchronize()
    assert cache.errors() == 0 and out.abs().sum() > 0
    assert torch.equal(out[0], out[1])


@pytest.mark.parametrize("layers", [1, 3])
def test_copy_pages(zt, layers):
    import torch
    rng = np.random.default_rng(layers)
    page, heads, D, n = 48, 3, 96, 11
    raw = rng.integers(0, 256, (layers, n, zt.kv_page_bytes(page, heads, D)), dtype=np.uint8)
    cache = zt.KvCache(cuda(raw), page, heads, D)
    src, dst = np.array([3, 3, 10, 5, 8], np.int32), np.array([0, 1, 2, 5, 9], np.int32)
    zt.KvCopy(cache, cuda(src), cuda(dst)).run()
    raw[:, dst] = raw[:, src]
    assert np.array_equal(cache.pages.cpu().numpy(), raw) and cache.errors() == 0
    zt.KvCopy(cache, cuda(np.array([n, 2, -1, 4], np.int32)), cuda(np.array([0, n, 1, 6], np.int32))).run()
    raw[:, 6] = raw[:, 4]
    assert np.array_equal(cache.pages.cpu().numpy(), raw) and cache.errors() == zt.ZT_Q4_KV_ERR_PLACE
    zt.KvCopy(cache, torch.empty(0, dtype=torch.int32, device="cuda"), torch.empty(0, dtype=torch.int32, device="cuda")).run()


def test_calls_without_rows(zt):
    """Empty tensors, with and without rotation: nothing is launched, nothing changes."""
    import torch
    rng = np.random.default_rng(14)
    raw = rng.integers(0, 256, (3, zt.kv_page_bytes(16, 2, 64)), dtype=np.uint8)
    cache = zt.KvCache(cuda(raw), 16, 2, 64)
    x, no = cuda(fp16(rng, 5, 8, 64)), torch.empty(0, dtype=torch.int32, device="cuda")
    table = cuda(np.zeros((1, 2), np.int32))
    for part in (x[:0], x[2:2], x[5:]):
        assert zt.KvAppend(cache, part[:, 4:6], part[:, 6:], no, no, table).run() == (None, None)
        q, k = zt.KvAppend(cache, part[:, 4:6], part[:, 6:], no, no, table, q=part[:, :4], theta=1e4).run()
        assert q.shape == (0, 4, 64) and k.shape == (0, 2, 64)
        k, v = zt.KvGather(cache, no, no, table).run()
        assert k.shape == v.shape == (0, 2, 64)
    assert cache.errors() == 0 and np.array_equal(cache.pages[0].cpu().numpy(), raw)


# ------------------------------------------------------------------ attention --
LENS = [0, 1, 15, 16, 17, 33, 100, 257]


@pytest.mark.parametrize("D,q_heads,heads,tokens,page", [
    (64, 4, 4, 1, 16), (96, 4, 4, 1, 64), (128, 8, 2, 1, 32), (128, 5, 1, 1, 16), (64, 16, 2, 1, 48), (96, 9, 1, 1, 16),
    (128, 16, 1, 1, 16), (128, 17, 1, 1, 16), (64, 2, 2, 4, 16), (96, 6, 2, 3, 32), (128, 4, 2, 16, 16), (64, 40, 2, 1, 16)])
def test_attention(zt, D, q_heads, heads, tokens, page):
    rng = np.random.default_rng(D * 100 + q_heads * 10 + tokens)
    cache, pool, table = filled(zt, rng, LENS, page, heads, D)
    check_attention(zt, cache, pool, fp16(rng, len(LENS), tokens, q_heads, D, by=2.0), LENS, table)


@pytest.mark.parametrize("D,q_heads,heads,tokens,page", [(128, 4, 1, 1, 64), (96, 2, 2, 1, 64), (64, 3, 1, 1, 16),
                                                         (128, 12, 1, 1, 48), (96, 5, 1, 5, 16), (64, 1, 1, 2, 1024)])
def test_attention_long_sequences(zt, D, q_heads, heads, tokens, page):
    """Sequences cut between many CTAs, next to short ones; up to 25 columns a head."""
    rng = np.random.default_rng(D)
    lens = [5, 7001, 0, 1300, 1]
    cache, pool, table = filled(zt, rng, lens, page, heads, D)
    check_attention(zt, cache, pool, fp16(rng, len(lens), tokens, q_heads, D, by=2.0), lens, table)


def test_attention_split_changes_nothing_but_rounding(zt):
    """The same sequence alone, among others and behind a wider page table (which of the launch shapes is taken goes by
    that) agrees within the tolerance; each of them repeats bit for bit."""
    rng = np.random.default_rng(12)
    lens, D = [900, 33, 900, 700], 128
    cache, pool, table = filled(zt, rng, lens, 32, 2, D)
    q = fp16(rng, 4, 1, 8, D, by=2.0)
    wide = np.concatenate([table, np.zeros((4, 40), np.int32)], 1)
    for t in (table, wide):
        check_attention(zt, cache, pool, q, lens, t)
        check_attention(zt, cache, pool, q[:1], lens[:1], t[:1])


def test_attention_reports_a_workspace_that_was_not_zeroed(zt):
    import torch
    rng = np.random.default_rng(13)
    lens = [6000]
    cache, pool, table = filled(zt, rng, lens, 64, 1, 64)
    nbytes = zt.kv_attention_workspace_bytes(1, 1, 64, 1)
    dirty = torch.full((nbytes,), 0xEE, dtype=torch.uint8, device="cuda")
    zt.KvAttention(cache, cuda(fp16(rng, 1, 1, 1, 64)), cuda(np.array(lens, np.int32)), cuda(table), workspace=dirty).run()
    torch.cuda.synchronize()
    assert cache.errors() == zt.ZT_Q4_KV_ERR_WORKSPACE


def test_attention_many_sequences(zt):
    """More sequences than one warp's prefix sum, most of them a single token or none."""
    rng = np.random.default_rng(3)
    lens = [int(n) for n in rng.integers(0, 4, 300)]
    lens[123] = 90
    cache, pool, table = filled(zt, rng, lens, 16, 1, 64)
    check_attention(zt, cache, pool, fp16(rng, len(lens), 1, 2, 64), lens, table)


def test_attention_scale_and_strides(zt):
    """q as the first heads of a QKV buffer, out as rows of a wider one, a scale of the caller's."""
    import torch
    rng = np.random.default_rng(4)
    lens, D = [40, 3], 96
    cache, pool, table = filled(zt, rng, lens, 16, 2, D)
    q = fp16(rng, 2, 1, 4, D)
    got = check_attention(zt, cache, pool, q, lens, table, scale=0.25)
    wide = torch.full((2, 1, 9, D), 7.0, dtype=torch.float16, device="cuda")
    wide[:, :, :4] = cuda(q)
    out = torch.full((2, 1, 6, D), 7.0, dtype=torch.float16, device="cuda")
    zt.KvAttention(cache, wide[:, :, :4], cuda(np.array(lens, np.int32)), cuda(table), scale=0.25, out=out[:, :, 1:5]).run()
    out = out.cpu().numpy()
    assert np.array_equal(out[:, :, 1:5], got) and (out[:, :, 0] == 7).all() and (out[:, :, 5] == 7).all()


@pytest.mark.parametrize("v_by", [1e-4, 100.0, 8000.0])
def test_attention_value_ranges(zt, v_by):
    """Tiny values, and scales of 2 and more, which change the weights' offset within a segment."""
    rng = np.random.default_rng(6)
    lens = [200, 33]

    def edit(b, p, k, v):
        if v_by > 1 and p % 3:
            v[:] = v / np.float16(v_by)
    cache, pool, table = filled(zt, rng, lens, 16, 2, 128, v_by=v_by, edit=edit)
    check_attention(zt, cache, pool, fp16(rng, 2, 1, 4, 128, by=2.0), lens, table, large_v=v_by > 1)


@pytest.mark.parametrize("D,q_heads,heads,tokens", [(64, 4, 2, 1), (96, 6, 2, 3), (128, 8, 1, 1), (128, 16, 2, 2)])
@pytest.mark.parametrize("by", [1e-3, 1e-4, 1e-5, 3e-7, 1.0, 2000.0, 16000.0])
def test_attention_query_ranges(zt, D, q_heads, heads, tokens, by):
    """Queries down to fp16's smallest values and up to its largest, with a scale that makes up for it: the scores are those of
    queries near 1, and so is what a call may be off by (the powers of two that q and the scale exchange are exact)."""
    rng = np.random.default_rng(D + tokens)
    lens = [512, 37]
    cache, pool, table = filled(zt, rng, lens, 32, heads, D)
    q = np.clip(rng.standard_normal((2, tokens, q_heads, D)) * by, -65504, 65504).astype(np.float16)
    check_attention(zt, cache, pool, q, lens, table, scale=2.0 / by * D ** -0.5)


def test_attention_queries_of_different_sizes(zt):
    """Heads of all sizes beside one another, values of all sizes within a head, a head of zeros."""
    rng = np.random.default_rng(19)
    lens, D = [700, 33, 2000], 96
    cache, pool, table = filled(zt, rng, lens, 32, 1, D)
    q = rng.standard_normal((3, 1, 9, D)) * np.array([1, 1e-1, 1e-2, 1e-3, 1e-4, 1e-5, 10, 0, 1])[:, None]
    q[:, :, 8] *= 2.0 ** -rng.integers(0, 22, (3, 1, D))
    check_attention(zt, cache, pool, q.astype(np.float16), lens, table, scale=0.5)
    check_attention(zt, cache, pool, q[:, :, 2:6].astype(np.float16), lens, table, scale=300.0)


def test_attention_queries_that_are_not_finite(zt):
    """A head with an infinity or a NaN gives NaN; the others are not touched by it."""
    rng = np.random.default_rng(20)
    lens, D = [300], 64
    cache, pool, table = filled(zt, rng, lens, 32, 1, D)
    q = fp16(rng, 1, 2, 5, D)
    q[0, 0, 1, 7], q[0, 1, 3, 40], q[0, 1, 4, 0] = np.nan, np.nan, np.inf
    got = check_attention(zt, cache, pool, q, lens, table)
    assert np.isnan(got).any(-1).tolist() == [[[False, True, False, False, False], [False, False, False, True, True]]]


@pytest.mark.parametrize("n", [20, 300, 7000])
def test_attention_part_of_nan_scores(zt, n):
    """Tokens whose scores are all NaN make up a warp's or a CTA's whole share of a sequence: the result is NaN all the same."""
    rng = np.random.default_rng(21)
    for lo, hi in ((0, 16), (n - 1, n), (n // 2, n // 2 + 1)):
        def edit(b, p, k, v):
            if lo <= p < hi:
                k[0, 5] = np.inf
        cache, pool, table = filled(zt, rng, [n], 16, 2, 64, edit=edit)
        got = check_attention(zt, cache, pool, fp16(rng, 1, 1, 4, 64), [n], table)
        assert np.isnan(got[0, 0, :2]).all() and np.isfinite(got[0, 0, 2:]).all()


@pytest.mark.parametrize("n", [300, 7000])
@pytest.mark.parametrize("scale", [2.0**-8, 2.0**-4, 0.125, 1.0, 2.0**20, 2.0**60])
def test_attention_scores_of_any_size(zt, n, scale):
    """Scores up to 2^90, each of them exact in fp32 (a common value times small whole numbers), some equal: the largest ones
    share the weight, all others lie too far below to count, and nothing overflows."""
    rng = np.random.default_rng(22)
    c = rng.permutation(np.r_[np.full(n - n // 3, 512), np.full(n // 3 - 5, 1023), np.full(5, 1024)]).astype(np.float16)

    def edit(b, p, k, v):
        k[:] = c[p]
    cache, pool, table = filled(zt, rng, [n], 16, 1, 64, edit=edit)
    q = np.full((1, 1, 3, 64), 1024, np.float16)
    q[0, 0, 1:] = np.float16([[-1024], [16384]])
    check_attention(zt, cache, pool, q, [n], table, scale=scale)


@pytest.mark.parametrize("scale", [0.5, 0.3, 0.7, 1.1])
def test_attention_weights_at_the_largest_scale_below_two(zt, scale):
    """V scales of 1.999 and weights as far above the reference as they come without a rescale, at scores of up to 2^17 in the
    exponent, whose roundings are 2^-7: weight * V scale is fp16's largest value nearly.  All V are alike, so the output is
    V's value whatever the weights; it is off by their product's rounding and its own, 2^-11 each, and fp32 sums."""
    rng = np.random.default_rng(23)
    D, heads, seqs, page = 64, 16, 40, 80
    k, v = np.zeros((page, heads, D), np.float16), np.full((page, heads, D), 15.992, np.float16)
    k[:, :, 0], k[64:, :, 32:] = 64.0, 1.0
    pool = ref.Pool(np.zeros((1, zt.kv_page_bytes(page, heads, D)), np.uint8), page, heads, D)
    for p in range(page):
        pool.write(0, p, k[p], v[p])
    cache = zt.KvCache(cuda(pool.raw.reshape(1, -1)), page, heads, D)
    q = np.zeros((seqs, 16, heads, D), np.float16)
    q[..., 0] = rng.uniform(100, 2**17 * np.log(2) / 64 / scale, q.shape[:-1])
    q[..., 32:40] = 6 * np.log(2) / scale / 8                   # later tokens: 6 powers of two more ...
    q[..., 40] = rng.uniform(-0.03, 0.03, q.shape[:-1])         # ... and a little
    out = zt.KvAttention(cache, cuda(q), cuda(np.full(seqs, page, np.int32)), cuda(np.zeros((seqs, 1), np.int32)), scale=scale).run()
    want = pool.values([0], page)[1][0, 0, 0]
    assert want == 8 * np.float64(np.float16(1.999))
    assert (np.abs(out.cpu().numpy() - want) <= (2.0**-10 + 2.0**-16) * want).all() and cache.errors() == 0


@pytest.mark.parametrize("bits", [16, 18, 20, 22])
@pytest.mark.parametrize("top", [16.5, 40.0, 300.0, 4000.0, 60000.0])
def test_attention_small_weights_beside_a_large_value(zt, top, bits):
    """Tokens of weight 2^-bits beside one whose V scale is 2^e or more, which a warp's whole run follows.  Their products with
    their scale s = 0.3 are rounded at 2^off 2^-bits s, off = min(9, 13 - e): off by 2^-11 of themselves, or by half of fp16's
    smallest step, 2^-25.  The output's own rounding is 2^-11 (2^-25 where it is subnormal), fp32 sums and scores 2^-16."""
    rng = np.random.default_rng(24)
    D, heads, n, seqs, page = 64, 8, 200, 600, 208
    pool = ref.Pool(np.zeros((1, zt.kv_page_bytes(page, heads, D)), np.uint8), page, heads, D)
    first = int(rng.integers(0, 16))
    for p in range(n):
        k, v = np.full((heads, D), 1.0 if p == first else 0.0, np.float16), np.full((heads, D), 2.4, np.float16)
        if p == first:
            v[:, :32], v[:, 32:] = 0.0, top
        pool.write(0, p, k, v)
    cache = zt.KvCache(cuda(pool.raw.reshape(1, -1)), page, heads, D)
    k, v = pool.values([0], n)
    q, scale = np.ones((seqs, 1, heads, D), np.float16), bits * np.log(2) / D
    out = zt.KvAttention(cache, cuda(q), cuda(np.full(seqs, n, np.int32)), cuda(np.zeros((seqs, 1), np.int32)), scale=scale).run()
    want, _ = ref.attention(q[0], k, v, [n], scale)
    off = min(9, 13 - int(np.floor(np.log2(top / 8))))
    tol = (2.0**-10 + 2.0**-16 + 2.0**-25 / (2.0**(off - bits) * 0.3)) * np.abs(want) + 2.0**-25
    assert (np.abs(out.cpu().numpy()[:, 0].astype(np.float64) - want) <= tol).all() and cache.errors() == 0


def test_attention_sink(zt):
    """One token takes half the weight, thousands of others share the rest: none of it is lost."""
    rng = np.random.default_rng(7)
    D, n = 64, 4000
    u = np.sign(fp16(rng, D)).astype(np.float16)

    def edit(b, p, k, v):
        k[:] = u * np.float16(1.0 if p == 0 else 0.0)
        v[:] = np.float16(0.02) if p else np.float16(0)
    cache, pool, table = filled(zt, rng, [n], 16, 1, D, edit=edit)
    q = np.broadcast_to(u, (1, 1, 2, D)).copy()
    q[0, 0, 1] *= np.float16(2)
    got = check_attention(zt, cache, pool, q, [n], table, scale=np.log(n) / D)
    assert (got[0, 0, 0] > 0.009).all() and (got[0, 0, 1] > 0).all()


def test_attention_hides_what_is_behind(zt):
    """NaN scales behind the sequences' ends (random bytes elsewhere in the tests) and NaN rows that an earlier drafted
    token must not see stay out of the results; rows that see a NaN give NaN."""
    rng = np.random.default_rng(8)
    lens, tokens, D = [19, 5], 3, 96

    def edit(b, p, k, v):
        if p == lens[b] - 1:
            v[0, 40] = np.nan
            k[1, 3] = np.inf
    cache, pool, table = filled(zt, rng, lens, 16, 2, D, edit=edit)
    got = check_attention(zt, cache, pool, fp16(rng, 2, tokens, 2, D), lens, table)
    assert np.isfinite(got[:, :2]).all() and np.isnan(got[:, 2, 0, 32:64]).all() and np.isnan(got[:, 2, 1]).all()
    assert np.isfinite(got[:, 2, 0, :32]).all()


def test_attention_reports_bad_pages_and_lengths(zt):
    """A page out of range is left out with the error bit set; lengths beyond the table are cut, negative ones empty."""
    import torch
    rng = np.random.default_rng(9)
    lens = [40, 33, 16]
    cache, pool, table = filled(zt, rng, lens, 16, 1, 64)
    q = fp16(rng, 3, 1, 1, 64)
    broken = table.copy()
    broken[0, 1] = pool.raw.shape[0]
    out = zt.KvAttention(cache, cuda(q), cuda(np.array(lens, np.int32)), cuda(broken)).run().cpu().numpy()
    assert cache.errors() == zt.ZT_Q4_KV_ERR_PLACE
    cache.clear_errors()
    k, v = pool.values(table[0, :3], 40)
    keep = np.r_[0:16, 32:40]
    want, mag = ref.attention(q[0], k[keep], v[keep], [24], 64 ** -0.5)
    assert (np.abs(out[0] - want) <= 2.0**-9 * mag + 2.0**-11 * np.abs(want) + 2.0**-25).all()
    good = table.copy()
    good[good > 10**6] = 0
    out = zt.KvAttention(cache, cuda(q), cuda(np.array([-5, 33, 10**9], np.int32)), cuda(good)).run()
    torch.cuda.synchronize()
    assert cache.errors() == zt.ZT_Q4_KV_ERR_PLACE and (out[0] == 0).all() and torch.isfinite(out[1]).all()


def test_graph_stream_and_workspace(zt):
    """Captured and replayed with new contents, and on a stream of its own, the calls give what eager calls give; two graphs
    that share a workspace may follow each other."""
    import torch
    rng = np.random.default_rng(10)
    lens, heads, D, page = [70, 1500, 3], 2, 128, 16
    cache, pool, table = filled(zt, rng, lens, page, heads, D)
    q = cuda(fp16(rng, 3, 1, 4, D))
    ld, td = cuda(np.array(lens, np.int32)), cuda(table)
    first = zt.KvAttention(cache, q, ld, td)
    ws = first._keep[5]
    second = zt.KvAttention(cache, q.flip(0).contiguous(), ld, td, workspace=ws)
    want = [first.run().clone(), second.run().clone()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs = []
    with torch.cuda.stream(side):
        for plan in (first, second):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                plan.run()
            graphs.append(g)
        for _ in range(3):
            for g, plan, w in zip(graphs, (first, second), want):
                plan._result.zero_()
                g.replay()
                assert torch.equal(plan._result, w)
        q.mul_(0.5)
        first._result.zero_()
        graphs[0].replay()
        replayed = first._result.clone()
        assert torch.equal(first.run(stream=side), replayed) and not torch.equal(replayed, want[0])
    torch.cuda.synchronize()


def test_runs_on_other_streams_wait_for_the_fills(zt):
    """A workspace, an error word and a cache's memory that are zeroed behind long work on the constructing stream: a run on
    another stream comes after it, whatever the memory held before."""
    import torch
    rng = np.random.default_rng(15)
    lens = [6000]
    cache, pool, table = filled(zt, rng, lens, 64, 1, 64)
    q, ld, td = cuda(fp16(rng, 1, 1, 1, 64)), cuda(np.array(lens, np.int32)), cuda(table)
    out, side = torch.empty_like(q), torch.cuda.Stream()
    want = zt.KvAttention(cache, q, ld, td).run().clone()
    x, zero = cuda(fp16(rng, 1, 2, 64)), cuda(np.zeros(1, np.int32))
    sizes = (zt.kv_attention_workspace_bytes(1, 1, 64, 1), 2 * zt.kv_page_bytes(16, 1, 64), 4)
    torch.cuda.synchronize()
    dirty = [torch.full((n,), 0xEE, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(4)]
    torch.cuda.synchronize()
    del dirty
    torch.cuda._sleep(200_000_000)                  # about 0.1 s
    plan = zt.KvAttention(cache, q, ld, td, out=out)
    other = zt.KvCache.empty(1, 2, 16, 1, 64)
    append = zt.KvAppend(other, x[:, :1], x[:, 1:], zero, zero, zero[None])
    plan.run(stream=side)
    append.run(stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(out, want) and cache.errors() == 0
    raw = ref.Pool(np.zeros((2, other.page_bytes), np.uint8), 16, 1, 64)
    raw.write(0, 0, x[0, :1].cpu().numpy(), x[0, 1:].cpu().numpy())
    torch.cuda.synchronize()
    same_bytes(other, raw)
    assert other.errors() == 0


def test_run_on_the_default_stream_waits_for_a_fill_on_another(zt):
    import torch
    rng = np.random.default_rng(17)
    lens = [6000]
    cache, pool, table = filled(zt, rng, lens, 64, 1, 64)
    q, ld, td = cuda(fp16(rng, 1, 1, 1, 64)), cuda(np.array(lens, np.int32)), cuda(table)
    out, side = torch.empty_like(q), torch.cuda.Stream()
    want = zt.KvAttention(cache, q, ld, td).run().clone()
    with torch.cuda.stream(side):
        dirty = torch.full((zt.kv_attention_workspace_bytes(1, 1, 64, 1),), 0xEE, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        del dirty
        torch.cuda._sleep(200_000_000)
        plan = zt.KvAttention(cache, q, ld, td, out=out)
    plan.run()
    got = out.clone()
    torch.cuda.synchronize()
    assert torch.equal(got, want) and cache.errors() == 0


def test_errors_waits_for_other_streams(zt):
    """A bad page met on a stream that is still busy is in the word that errors() returns."""
    import torch
    cache = zt.KvCache.empty(1, 4, 16, 1, 64)
    x, zero = torch.ones((1, 1, 64), dtype=torch.float16, device="cuda"), cuda(np.zeros(1, np.int32))
    append = zt.KvAppend(cache, x, x, zero, zero, cuda(np.full((1, 1), 99, np.int32)))
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)
    append.run(stream=side)
    assert cache.errors() == zt.ZT_Q4_KV_ERR_PLACE


def test_dropped_plans_keep_their_memory_until_their_runs_end(zt):
    """A plan (with its workspace) and a cache that are let go while their runs on another stream are still to come: memory
    allocated afterwards on the constructing stream is not theirs."""
    import torch
    rng = np.random.default_rng(18)
    lens = [6000]
    cache, pool, table = filled(zt, rng, lens, 64, 1, 64)
    q, ld, td = cuda(fp16(rng, 1, 1, 1, 64)), cuda(np.array(lens, np.int32)), cuda(table)
    out, side = torch.empty_like(q), torch.cuda.Stream()
    want = zt.KvAttention(cache, q, ld, td).run().clone()
    x, zero = cuda(fp16(rng, 1, 2, 64)), cuda(np.zeros(1, np.int32))
    own = zt.KvCache.empty(1, 2, 16, 1, 64)
    plans = [zt.KvAttention(cache, q, ld, td, out=out), zt.KvAppend(own, x[:, :1], x[:, 1:], zero, zero, zero[None]),
             zt.KvGather(own, zero, zero, zero[None])]
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)              # about 0.1 s
    for p in plans:
        kv_back = p.run(stream=side)
    sizes = (zt.kv_attention_workspace_bytes(1, 1, 64, 1), 2 * own.page_bytes, 4)
    del plans, p, own
    dirty = [torch.full((n,), 0xEE, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(4)]
    side.synchronize()
    assert torch.equal(out, want) and cache.errors() == 0
    for got, src in zip(kv_back, (x[:, :1], x[:, 1:])):
        assert np.array_equal(got.cpu().numpy(), ref.dequantize(*ref.quantize(src.cpu().numpy())).astype(np.float16))
    assert all((d == 0xEE).all() for d in dirty)


def test_plans_made_in_a_capture(zt):
    """A plan made while a graph is captured has its fill in the graph: it runs there, on a forked stream too, and is refused
    outside."""
    import torch
    rng = np.random.default_rng(16)
    lens = [3000]
    cache, pool, table = filled(zt, rng, lens, 64, 1, 64)
    q, ld, td = cuda(fp16(rng, 1, 1, 1, 64)), cuda(np.array(lens, np.int32)), cuda(table)
    want = zt.KvAttention(cache, q, ld, td).run().clone()
    outs = [torch.empty_like(q) for _ in range(2)]
    main, fork, graph = torch.cuda.Stream(), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=main):
        fork.wait_stream(main)
        plans = [zt.KvAttention(cache, q, ld, td, out=o) for o in outs]
        plans[0].run()
        plans[1].run(stream=fork)
        main.wait_stream(fork)
    for _ in range(3):
        for o in outs:
            o.fill_(7.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, want) for o in outs) and cache.errors() == 0
    for stream in (None, main, fork):
        with pytest.raises(RuntimeError, match="captured"):
            plans[0].run(stream=stream)


def test_attention_refuses_other_workspaces(zt):
    import torch
    cache = zt.KvCache.empty(1, 4, 16, 2, 64)
    q = torch.zeros((1, 1, 2, 64), dtype=torch.float16, device="cuda")
    lens, table = (torch.zeros(s, dtype=torch.int32, device="cuda") for s in ((1,), (1, 2)))
    n = zt.kv_attention_workspace_bytes(2, 2, 64, 1)
    for bad in (torch.zeros(n, dtype=torch.uint8), torch.zeros(n, dtype=torch.int8, device="cuda"),
                torch.zeros((2, n), dtype=torch.uint8, device="cuda"), torch.zeros(2 * n, dtype=torch.uint8, device="cuda")[::2]):
        with pytest.raises(ValueError, match="workspace"):
            zt.KvAttention(cache, q, lens, table, workspace=bad)
    with pytest.raises(zt.ZtError):
        zt.KvAttention(cache, q, lens, table, workspace=torch.zeros(n - 1, dtype=torch.uint8, device="cuda")).run()
