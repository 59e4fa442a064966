"""The paged 4-bit cache on the host: refusals of every entry point before any
CUDA call (fake addresses are never dereferenced), the binding's checks, and the
page bookkeeping.  No GPU needed."""
import ctypes

import numpy as np
import pytest

from int4_group_quantized_q4f16_b200 import build as zt_build
from int4_group_quantized_q4f16_b200.kv_pages import KvPages

FAKE = 0x10000


@pytest.fixture(scope="module")
def zt():
    zt_build.build()
    from int4_group_quantized_q4f16_b200 import zt_q4
    return zt_q4


def kv(zt, pages=FAKE, n_pages=4, page_size=16, kv_heads=2, head_dim=64, err=None):
    return zt.ZtKv(pages, n_pages, page_size, kv_heads, head_dim, err)


def rows(zt, seq=FAKE, pos=FAKE, n=3, table=FAKE, n_seqs=2, max_pages=2):
    return zt.ZtKvRows(seq, pos, n, table, n_seqs, max_pages)


BAD_KV = [(dict(pages=None), "INVALID_ARG"), (dict(n_pages=0), "INVALID_ARG"), (dict(page_size=8), "INVALID_ARG"),
          (dict(page_size=24), "INVALID_ARG"), (dict(page_size=2048), "INVALID_ARG"), (dict(kv_heads=0), "INVALID_ARG"),
          (dict(head_dim=80), "UNSUPPORTED"), (dict(head_dim=0), "UNSUPPORTED"), (dict(pages=FAKE + 8), "MISALIGNED"),
          (dict(err=FAKE + 2), "MISALIGNED")]
BAD_ROWS = [(dict(seq=None), "INVALID_ARG"), (dict(pos=None), "INVALID_ARG"), (dict(n=-1), "INVALID_ARG"),
            (dict(n=2**25), "INVALID_ARG"), (dict(table=None), "INVALID_ARG"), (dict(n_seqs=0), "INVALID_ARG"),
            (dict(max_pages=0), "INVALID_ARG"), (dict(max_pages=2**28), "INVALID_ARG"), (dict(seq=FAKE + 2), "MISALIGNED"),
            (dict(table=FAKE + 1), "MISALIGNED")]


def status(zt, name):
    return getattr(zt, "ZT_ERR_" + name)


def test_page_bytes(zt):
    f = zt.lib.zt_q4_kv_page_bytes
    assert f(64, 32, 96) == 32 * 4 * 18 * 96 and f(16, 1, 64) == 18 * 64
    for bad in ((0, 1, 64), (17, 1, 64), (16, 0, 64), (16, 1, 32), (16, 1, 256), (-16, 1, 64), (1040, 1, 64)):
        assert f(*bad) == 0
    with pytest.raises(ValueError):
        zt.kv_page_bytes(16, 1, 100)


def test_append_and_gather_refusals(zt):
    app, gat, ref = zt.lib.zt_q4_kv_append, zt.lib.zt_q4_kv_gather, ctypes.byref
    for bad, name in BAD_KV:
        assert app(ref(kv(zt, **bad)), ref(rows(zt)), FAKE, 128, FAKE, 128, None, None) == status(zt, name), bad
        assert gat(ref(kv(zt, **bad)), ref(rows(zt)), FAKE, 128, FAKE, 128, None) == status(zt, name), bad
    for bad, name in BAD_ROWS:
        assert app(ref(kv(zt)), ref(rows(zt, **bad)), FAKE, 128, FAKE, 128, None, None) == status(zt, name), bad
        assert gat(ref(kv(zt)), ref(rows(zt, **bad)), FAKE, 128, FAKE, 128, None) == status(zt, name), bad
    assert app(None, ref(rows(zt)), FAKE, 128, FAKE, 128, None, None) == zt.ZT_ERR_INVALID_ARG
    assert app(ref(kv(zt)), None, FAKE, 128, FAKE, 128, None, None) == zt.ZT_ERR_INVALID_ARG
    for k, ldk, v, ldv, name in ((None, 128, FAKE, 128, "INVALID_ARG"), (FAKE, 128, None, 128, "INVALID_ARG"),
                                 (FAKE, 120, FAKE, 128, "INVALID_ARG"), (FAKE, 128, FAKE, 127, "INVALID_ARG"),
                                 (FAKE + 8, 128, FAKE, 128, "MISALIGNED"), (FAKE, 128, FAKE, 132, "MISALIGNED")):
        assert app(ref(kv(zt)), ref(rows(zt)), k, ldk, v, ldv, None, None) == status(zt, name)
        assert gat(ref(kv(zt)), ref(rows(zt)), k, ldk, v, ldv, None) == status(zt, name)
    # no rows: nothing to launch (and no device needed)
    assert app(ref(kv(zt)), ref(rows(zt, n=0, seq=None, pos=None)), FAKE, 128, FAKE, 128, None, None) == zt.ZT_OK
    assert gat(ref(kv(zt)), ref(rows(zt, n=0)), FAKE, 128, FAKE, 128, None) == zt.ZT_OK


def test_append_rope_refusals(zt):
    def call(theta=1e4, q=None, ld_q=0, q_heads=0, q_out=None, ld_qo=0, k_out=None, ld_ko=0):
        rope = zt.ZtKvRope(theta, q, ld_q, q_heads, q_out, ld_qo, k_out, ld_ko)
        return zt.lib.zt_q4_kv_append(ctypes.byref(kv(zt)), ctypes.byref(rows(zt, n=0)), FAKE, 128, FAKE, 128,
                                      ctypes.byref(rope), None)
    other = 2 * FAKE
    assert call() == zt.ZT_OK and call(q=FAKE, ld_q=256, q_heads=4, q_out=other, ld_qo=256, k_out=other, ld_ko=128) == zt.ZT_OK
    for theta in (0.0, -1.0, float("nan"), float("inf")):
        assert call(theta=theta) == zt.ZT_ERR_INVALID_ARG
    good = dict(q=FAKE, ld_q=256, q_heads=4, q_out=other, ld_qo=256)
    for bad, name in ((dict(q_heads=0), "INVALID_ARG"), (dict(ld_q=248), "INVALID_ARG"), (dict(q_out=None), "INVALID_ARG"),
                      (dict(q_out=FAKE), "INVALID_ARG"), (dict(q=None), "INVALID_ARG"), (dict(ld_qo=260), "MISALIGNED"),
                      (dict(q_out=other + 2), "MISALIGNED"), (dict(k_out=FAKE, ld_ko=128), "INVALID_ARG"),
                      (dict(k_out=other, ld_ko=64), "INVALID_ARG")):
        assert call(**{**good, **bad}) == status(zt, name), bad


def test_copy_refusals(zt):
    f = zt.lib.zt_q4_kv_copy_pages
    size = zt.kv_page_bytes(16, 2, 64)

    def call(src=FAKE, dst=FAKE, n=0, layers=1, layer_bytes=0, **bad):
        return f(ctypes.byref(kv(zt, **bad)), src, dst, n, layers, layer_bytes, None)
    for bad, name in BAD_KV:
        assert call(**bad) == status(zt, name)
    assert call() == zt.ZT_OK and call(layers=2, layer_bytes=4 * size) == zt.ZT_OK
    for bad, name in ((dict(n=-1), "INVALID_ARG"), (dict(n=1, src=None), "INVALID_ARG"), (dict(n=1, dst=None), "INVALID_ARG"),
                      (dict(layers=0), "INVALID_ARG"), (dict(layers=65536), "INVALID_ARG"),
                      (dict(layers=2, layer_bytes=4 * size - 16), "INVALID_ARG"),
                      (dict(layers=2, layer_bytes=4 * size + 8), "MISALIGNED"), (dict(src=FAKE + 1), "MISALIGNED")):
        assert call(**bad) == status(zt, name), bad


def test_attention_refusals(zt):
    ws = zt.kv_attention_workspace_bytes(2, 8, 64, 1)
    assert ws > 0 and zt.kv_attention_workspace_bytes(2, 8, 128, 4) > ws
    for bad in ((0, 8, 64, 1), (2, 7, 64, 1), (2, 1, 64, 1), (2, 8, 32, 1), (2, 8, 64, 0), (2, 8, 64, 17)):
        assert zt.kv_attention_workspace_bytes(*bad) == 0

    def call(q=FAKE, ld_q=512, heads=8, tokens=1, lens=FAKE, table=FAKE, seqs=2, max_pages=2, scale=0.1, out=FAKE, ld=512,
             work=FAKE, nbytes=ws, **bad):
        return zt.lib.zt_q4_kv_attention(ctypes.byref(kv(zt, **bad)), q, ld_q, heads, tokens, lens, table, seqs, max_pages,
                                         scale, out, ld, work, nbytes, None)
    for bad, name in BAD_KV:
        assert call(**bad) == status(zt, name)
    for bad, name in ((dict(q=None), "INVALID_ARG"), (dict(ld_q=504), "INVALID_ARG"), (dict(ld_q=516), "MISALIGNED"),
                      (dict(q=FAKE + 8), "MISALIGNED"), (dict(heads=7), "INVALID_ARG"), (dict(heads=0), "INVALID_ARG"),
                      (dict(tokens=0), "INVALID_ARG"), (dict(tokens=17), "INVALID_ARG"), (dict(lens=None), "INVALID_ARG"),
                      (dict(table=None), "INVALID_ARG"), (dict(seqs=0), "INVALID_ARG"), (dict(seqs=2049), "INVALID_ARG"),
                      (dict(max_pages=0), "INVALID_ARG"), (dict(scale=0.0), "INVALID_ARG"), (dict(scale=-1.0), "INVALID_ARG"),
                      (dict(scale=float("nan")), "INVALID_ARG"), (dict(scale=float("inf")), "INVALID_ARG"),
                      (dict(scale=2.0**65), "INVALID_ARG"), (dict(scale=2.0**-65), "INVALID_ARG"),
                      (dict(out=None), "INVALID_ARG"), (dict(out=FAKE + 1), "MISALIGNED"), (dict(ld=511), "INVALID_ARG"),
                      (dict(work=None), "INVALID_ARG"), (dict(work=FAKE + 8), "MISALIGNED"), (dict(nbytes=ws - 1), "WORKSPACE"),
                      (dict(seqs=2048, max_pages=2**19), "UNSUPPORTED")):
        assert call(**bad) == status(zt, name), bad


def test_prompt_refusals(zt):
    def call(q=FAKE, ld_q=512, k=FAKE, ld_k=128, v=FAKE, ld_v=128, cu_q=FAKE, cu_k=FAKE, seqs=2, total_q=10, total_k=10,
             heads=8, kv_heads=2, dim=64, causal=1, scale=0.1, out=FAKE, ld=512, err=None):
        return zt.lib.zt_q4_prompt_attention(q, ld_q, k, ld_k, v, ld_v, cu_q, cu_k, seqs, total_q, total_k, heads, kv_heads,
                                             dim, causal, scale, out, ld, err, None)
    for bad, name in ((dict(q=None), "INVALID_ARG"), (dict(k=None), "INVALID_ARG"), (dict(v=None), "INVALID_ARG"),
                      (dict(out=None), "INVALID_ARG"), (dict(cu_q=None), "INVALID_ARG"), (dict(cu_k=None), "INVALID_ARG"),
                      (dict(ld_q=504), "INVALID_ARG"), (dict(ld_k=120), "INVALID_ARG"), (dict(ld_v=120), "INVALID_ARG"),
                      (dict(ld=504), "INVALID_ARG"), (dict(ld_q=516), "MISALIGNED"), (dict(ld_k=132), "MISALIGNED"),
                      (dict(q=FAKE + 8), "MISALIGNED"), (dict(out=FAKE + 2), "MISALIGNED"), (dict(v=FAKE + 4), "MISALIGNED"),
                      (dict(cu_q=FAKE + 2), "MISALIGNED"), (dict(err=FAKE + 2), "MISALIGNED"), (dict(seqs=0), "INVALID_ARG"),
                      (dict(seqs=2049), "INVALID_ARG"), (dict(total_q=-1), "INVALID_ARG"), (dict(total_k=2**25), "INVALID_ARG"),
                      (dict(heads=7), "INVALID_ARG"), (dict(kv_heads=0), "INVALID_ARG"), (dict(heads=1), "INVALID_ARG"),
                      (dict(dim=80), "UNSUPPORTED"), (dict(dim=256), "UNSUPPORTED"), (dict(causal=2), "INVALID_ARG"),
                      (dict(scale=0.0), "INVALID_ARG"), (dict(scale=float("inf")), "INVALID_ARG"),
                      (dict(scale=2.0**65), "INVALID_ARG"), (dict(scale=2.0**-65), "INVALID_ARG")):
        assert call(**bad) == status(zt, name), bad
    assert call(total_q=0, q=None, out=None) == zt.ZT_OK


def test_errors_call_refusals(zt):
    assert zt.lib.zt_q4_kv_errors(None, ctypes.byref(ctypes.c_uint(0))) == zt.ZT_ERR_INVALID_ARG
    assert zt.lib.zt_q4_kv_errors(FAKE, None) == zt.ZT_ERR_INVALID_ARG


def test_binding_refuses_host_tensors(zt):
    import torch
    with pytest.raises(ValueError):
        zt.KvCache(torch.zeros(1, 4, zt.kv_page_bytes(16, 2, 64), dtype=torch.uint8), 16, 2, 64)


def test_calls_without_rows_take_null_pointers(zt):
    """An empty tensor's address is null: with n = 0 that is no fault, other arguments are still checked."""
    app, gat, ref = zt.lib.zt_q4_kv_append, zt.lib.zt_q4_kv_gather, ctypes.byref
    none = rows(zt, n=0, seq=None, pos=None)
    assert app(ref(kv(zt)), ref(none), None, 128, None, 128, None, None) == zt.ZT_OK
    assert gat(ref(kv(zt)), ref(none), None, 128, None, 128, None) == zt.ZT_OK
    rope = zt.ZtKvRope(1e4, None, 256, 4, None, 256, None, 128)
    assert app(ref(kv(zt)), ref(none), None, 128, None, 128, ref(rope), None) == zt.ZT_OK
    assert app(ref(kv(zt, head_dim=80)), ref(none), None, 128, None, 128, None, None) == zt.ZT_ERR_UNSUPPORTED
    assert app(ref(kv(zt)), ref(none), FAKE + 8, 128, None, 128, None, None) == zt.ZT_ERR_MISALIGNED
    for call in (lambda: app(ref(kv(zt)), ref(rows(zt)), None, 128, FAKE, 128, None, None),
                 lambda: gat(ref(kv(zt)), ref(rows(zt)), FAKE, 128, None, 128, None)):
        assert call() == zt.ZT_ERR_INVALID_ARG


class OnDevice:
    """A host tensor that says it is on a GPU, for the binding's checks (nothing is launched)."""

    def __init__(self, t, device):
        self._t, self.device, self.is_cuda = t, device, True

    def __getattr__(self, name):
        return getattr(self._t, name)

    def as_strided(self, *args):
        return OnDevice(self._t.as_strided(*args), self.device)


def test_attention_refuses_an_out_of_another_shape(zt):
    """An out with fewer sequences or other tokens than q is refused, also where the storage behind it would have room."""
    import torch
    dev, shape = torch.device("cuda", 0), (4, 2, 8, 64)
    rows = lambda t: zt.KvAttention._rows_of(OnDevice(t, dev), dev, "out", *shape)   # noqa: E731
    big = torch.zeros((8, 4, 16, 128), dtype=torch.float16)
    assert rows(torch.zeros(shape, dtype=torch.float16))[1] == 8 * 64
    for bad in (torch.zeros((8, 2, 8, 64), dtype=torch.float16)[:2], torch.zeros((8, 2, 8, 64), dtype=torch.float16)[:5],
                torch.zeros((9, 1, 8, 64), dtype=torch.float16)[:4], torch.zeros((4, 4, 8, 64), dtype=torch.float16)[:, :1],
                torch.zeros((4, 3, 8, 64), dtype=torch.float16), torch.zeros((2, 4, 8, 64), dtype=torch.float16),
                big[:4, :2, :4, :64], big[:4, :2, :8, :96]):
        with pytest.raises(ValueError, match="out"):
            rows(bad)


def test_binding_refuses_what_an_int_cannot_hold(zt):
    """Strides, rows and table widths beyond the C call's 32-bit integers are refused, not cut off."""
    import torch
    dev = torch.device("cuda", 0)
    meta = lambda *a, **k: OnDevice(torch.empty_strided(*a, device="meta", **k), dev)   # noqa: E731
    half = dict(dtype=torch.float16)
    assert zt._heads(meta((2, 4, 64), (2**31 - 8, 64, 1), **half), dev, "k", 2, 4, 64)[1] == 2**31 - 8
    for stride in (2**31, 2**32 + 256):
        with pytest.raises(ValueError, match="k"):
            zt._heads(meta((2, 4, 64), (stride, 64, 1), **half), dev, "k", 2, 4, 64)
    cache = zt.KvCache.__new__(zt.KvCache)
    cache.device = dev
    ints = lambda *shape: meta(shape, (1,) if len(shape) == 1 else (shape[1], 1), dtype=torch.int32)   # noqa: E731
    assert cache._rows(ints(3), ints(3), ints(2, 5)).n == 3
    for seq, table in ((2**32 + 3, (2, 5)), (3, (2, 2**32 + 1)), (3, (2**31, 1))):
        with pytest.raises(ValueError):
            cache._rows(ints(seq), ints(seq), ints(*table))


# ---------------------------------------------------------------- bookkeeping --
def check(p: KvPages):
    """Every page's holders, recounted from the tables; pages being filled are held once."""
    held = np.zeros(p.n_pages, int)
    for s in p.sequences():
        pages, n = p.pages(s), p.length(s)
        assert len(pages) == -(-n // p.page_size) and len(set(pages)) == len(pages)
        held[pages] += 1
    assert list(held) == p._refs
    for s in p.sequences():
        if p.length(s) % p.page_size:
            assert held[p.pages(s)[-1]] == 1, "a page being filled is shared"


def test_pages_fork_free_compact_keep_contents():
    """A random life of a cache, played on an array of token numbers with the copies that the bookkeeping asks for."""
    rng = np.random.default_rng(0)
    p, size = KvPages(40, 4), 4
    store = np.full((40, size), -1)
    want, names = {}, iter(range(10**6))

    def run(copies):
        src, dst = [c[0] for c in copies], [c[1] for c in copies]
        assert not set(src) & set(dst) and len(set(dst)) == len(dst)
        store[dst] = store[src]

    for step in range(600):
        act = rng.integers(0, 6)
        seqs = p.sequences()
        try:
            if act == 0 or not seqs:
                s = next(names)
                p.add(s)
                want[s] = []
            elif act <= 2:
                s = seqs[rng.integers(len(seqs))]
                k = int(rng.integers(0, 9))
                at = p.extend(s, k)
                assert at == len(want[s])
                for t in range(at, at + k):
                    store[p.pages(s)[t // size], t % size] = step * 100 + t
                    want[s].append(step * 100 + t)
            elif act == 3:
                s, c = seqs[rng.integers(len(seqs))], next(names)
                run(p.fork(s, c))
                want[c] = list(want[s])
            elif act == 4 and len(seqs) > 3:
                s = seqs[rng.integers(len(seqs))]
                p.free(s)
                del want[s]
            else:
                run(p.compact())
                live = p.n_pages - p.free_pages
                assert all(max(p.pages(s), default=0) < max(live, 1) for s in p.sequences())
        except MemoryError:
            p.free(seqs[0])
            del want[seqs[0]]
        check(p)
        for s in p.sequences():
            assert [store[p.pages(s)[t // size], t % size] for t in range(p.length(s))] == want[s]


def test_pages_refusals_change_nothing():
    p = KvPages(3, 16)
    p.add("a")
    assert p.extend("a", 20) == 0 and p.free_pages == 1
    with pytest.raises(MemoryError):
        p.extend("a", 40)
    assert p.length("a") == 20 and p.free_pages == 1
    p.extend("a", 12)
    p.extend("a", 1)
    with pytest.raises(MemoryError):
        p.fork("a", "b")
    assert p.sequences() == ["a"] and p.free_pages == 0
    with pytest.raises(KeyError):
        p.add("a")
    with pytest.raises(KeyError):
        p.free("b")
    with pytest.raises(ValueError):
        p.extend("a", -1)
    with pytest.raises(ValueError):
        KvPages(0, 16)
    assert p.table(["a"]).tolist() == [p.pages("a")] and p.table(["a"], 5).shape == (1, 5)
    with pytest.raises(ValueError):
        p.table(["a"], 2)
