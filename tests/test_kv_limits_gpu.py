"""The cache and both attentions at the ends of what their documentation allows: many sequences, many heads, layers other than
the first, strided results, long lists of rows.  References and tolerances: test_kv_gpu.py and test_prompt_gpu.py."""
import numpy as np
import pytest

import kv_reference as ref
import test_kv_gpu as kv
import test_prompt_gpu as prompt
from test_kv_gpu import cuda, fp16, zt  # noqa: F401  (zt: fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("seqs", [33, 500, 2048])
@pytest.mark.parametrize("causal", [True, False])
def test_prompt_of_many_sequences(zt, seqs, causal):
    """More sequences than a warp has lanes, most of them short or empty, longer ones at the ends and in between."""
    rng = np.random.default_rng(seqs)
    nq = rng.integers(0, 9, seqs)
    nk = np.maximum(nq + rng.integers(-2, 20, seqs), 0)
    for at, n, m in ((0, 300, 300), (seqs - 1, 257, 400), (seqs // 2, 140, 600), (31, 129, 129), (32, 5, 700)):
        nq[at], nk[at] = n, m
    nk[3] = 0
    q, k, v = fp16(rng, nq.sum(), 4, 64, by=1.5), fp16(rng, nk.sum(), 2, 64), fp16(rng, nk.sum(), 2, 64)
    got = prompt.run(zt, q, k, v, nq, nk, causal)
    prompt.check(got, q, k, v, nq, nk, causal, 64 ** -0.5, heads=[0, 3])


@pytest.mark.parametrize("D,heads,kv_heads", [(64, 512, 2), (128, 300, 300)])
def test_prompt_of_many_heads(zt, D, heads, kv_heads):
    rng = np.random.default_rng(heads)
    nq, nk = [3, 130], [50, 131]
    q, k, v = fp16(rng, sum(nq), heads, D, by=1.5), fp16(rng, sum(nk), kv_heads, D), fp16(rng, sum(nk), kv_heads, D)
    prompt.check(prompt.run(zt, q, k, v, nq, nk), q, k, v, nq, nk, True, D ** -0.5, heads=[0, heads // 2, heads - 1])


@pytest.mark.parametrize("D", [64, 96, 128])
def test_attention_of_as_many_sequences_as_there_may_be(zt, D):
    rng = np.random.default_rng(D)
    lens = [int(n) for n in rng.integers(0, 3, zt.ZT_Q4_KV_MAX_SEQS)]
    lens[0], lens[1000], lens[-1] = 70, 333, 40
    cache, pool, table = kv.filled(zt, rng, lens, 16, 1, D)
    kv.check_attention(zt, cache, pool, fp16(rng, len(lens), 1, 2, D), lens, table)


@pytest.mark.parametrize("D,heads,kv_heads,tokens,n", [(64, 2048, 2, 1, 40), (128, 128, 1, 16, 700), (96, 64, 64, 2, 100)])
def test_attention_of_many_heads(zt, D, heads, kv_heads, tokens, n):
    rng = np.random.default_rng(heads + tokens)
    cache, pool, table = kv.filled(zt, rng, [n, 3], 32, kv_heads, D)
    kv.check_attention(zt, cache, pool, fp16(rng, 2, tokens, heads, D), [n, 3], table)


def test_layers_are_apart(zt):
    """Append, gather and attention on each layer of a cache: the layer's own rows, and no other layer's bytes change."""
    import torch
    rng = np.random.default_rng(31)
    layers, page, heads, D, n = 3, 16, 2, 64, 37
    raw = rng.integers(0, 256, (layers, 4, zt.kv_page_bytes(page, heads, D)), dtype=np.uint8)
    cache = zt.KvCache(cuda(raw), page, heads, D)
    table = np.array([[2, 0, 3]], np.int32)
    args = cuda(np.zeros(n, np.int32)), cuda(np.arange(n, dtype=np.int32)), cuda(table)
    q = fp16(rng, 1, 1, 4, D)
    for layer in (1, 2, 0):
        x = fp16(rng, n, 2 * heads, D)
        pool = ref.Pool(raw[layer], page, heads, D)
        for p in range(n):
            pool.write(table[0, p // page], p % page, x[p, :heads], x[p, heads:])
        zt.KvAppend(cache, cuda(x[:, :heads]), cuda(x[:, heads:]), *args, layer=layer).run()
        assert np.array_equal(cache.pages.cpu().numpy(), raw)
        k, v = zt.KvGather(cache, *args, layer=layer).run()
        for got, src in ((k, x[:, :heads]), (v, x[:, heads:])):
            assert np.array_equal(got.cpu().numpy(), ref.dequantize(*ref.quantize(src)).astype(np.float16))
        kv.check_attention(zt, cache, pool, q, [n], table, layer=layer)
    for bad in (-1, layers):
        with pytest.raises(ValueError, match="layer"):
            zt.KvAppend(cache, k, v, *args, layer=bad)
    torch.cuda.synchronize()


def test_append_and_gather_into_strided_rows(zt):
    """Rotated q and k, and rows read back, in the middle of wider rows: what lies beside them stays as it was."""
    import torch
    rng = np.random.default_rng(32)
    heads, q_heads, D, n = 3, 6, 96, 45
    cache = zt.KvCache.empty(1, 3, 16, heads, D)
    x = cuda(fp16(rng, n, q_heads + 2 * heads, D))
    args = cuda(np.zeros(n, np.int32)), cuda(np.arange(n, dtype=np.int32)), cuda(np.array([[1, 2, 0]], np.int32))
    k, v, q = x[:, q_heads:q_heads + heads], x[:, q_heads + heads:], x[:, :q_heads]
    want = [t.clone() for t in zt.KvAppend(cache, k, v, *args, q=q, theta=500.0).run()]
    bytes_ = cache.pages.clone()
    want += [t.clone() for t in zt.KvGather(cache, *args).run()]
    wide = [torch.full((n, h + 3, D), 7.0, dtype=torch.float16, device="cuda") for h in (q_heads, heads, heads, heads)]
    parts = [w[:, 1:-2] for w in wide]
    cache.pages.zero_()
    zt.KvAppend(cache, k, v, *args, q=q, theta=500.0, q_out=parts[0], k_out=parts[1]).run()
    zt.KvGather(cache, *args, k=parts[2], v=parts[3]).run()
    torch.cuda.synchronize()
    assert torch.equal(cache.pages, bytes_) and cache.errors() == 0
    for w, p, t in zip(wide, parts, want):
        assert torch.equal(p, t) and (w[:, 0] == 7).all() and (w[:, -2:] == 7).all()


def test_many_rows(zt):
    """A hundred thousand rows of one call, over sequences of all lengths, in the order of the sequences and shuffled."""
    import torch
    rng = np.random.default_rng(33)
    page, D, lens = 64, 64, [60000, 1, 17, 30000, 9999, 64]
    table, pages = kv.tables(rng, lens, page)
    seq, pos = np.repeat(np.arange(6), lens).astype(np.int32), np.concatenate([np.arange(n) for n in lens]).astype(np.int32)
    x = cuda(fp16(rng, len(seq), 2, D))
    caches = [zt.KvCache.empty(1, pages, page, 1, D) for _ in range(2)]
    order = torch.from_numpy(rng.permutation(len(seq))).cuda()
    sd, pd, td = cuda(seq), cuda(pos), cuda(table)
    zt.KvAppend(caches[0], x[:, :1], x[:, 1:], sd, pd, td).run()
    y, s2, p2 = x[order], sd[order].contiguous(), pd[order].contiguous()
    zt.KvAppend(caches[1], y[:, :1], y[:, 1:], s2, p2, td).run()
    assert torch.equal(caches[0].pages, caches[1].pages) and not caches[0].errors() and not caches[1].errors()
    k, v = zt.KvGather(caches[0], sd, pd, td).run()
    k2, v2 = zt.KvGather(caches[0], s2, p2, td).run()
    assert torch.equal(k[order], k2) and torch.equal(v[order], v2)
    some = rng.integers(0, len(seq), 2000)
    for got, src in ((k, x[:, :1]), (v, x[:, 1:])):
        assert np.array_equal(got.cpu().numpy()[some], ref.dequantize(*ref.quantize(src.cpu().numpy()[some])).astype(np.float16))


@pytest.mark.parametrize("width", [4, 200])
def test_replayed_step_follows_lengths_and_pages(zt, width):
    """One captured decode step (append, then attention, whose launch goes by the table's width), replayed while lengths,
    positions and the page table change: what eager calls on a copy of the cache give, bit for bit."""
    import torch
    rng = np.random.default_rng(width)
    page, heads, D, lens = 16, 2, 64, np.array([14, 0, 31], np.int32)
    cache, other = (zt.KvCache.empty(1, 12, page, heads, D) for _ in range(2))
    table = cuda(np.zeros((3, width), np.int32))
    x, q = cuda(fp16(rng, 3, 2 * heads, D)), cuda(fp16(rng, 3, 1, 4, D))
    seq, pos, ld = cuda(np.arange(3, dtype=np.int32)), cuda(lens), cuda(lens + 1)

    def plans(c):
        return zt.KvAppend(c, x[:, :heads], x[:, heads:], seq, pos, table), zt.KvAttention(c, q, ld, table)
    first, eager = plans(cache), plans(other)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for p in first:
            p.run()
    order = torch.from_numpy(rng.permutation(12).astype(np.int32)).cuda()
    for step in range(20):
        x.copy_(cuda(fp16(rng, 3, 2 * heads, D)))
        q.copy_(cuda(fp16(rng, 3, 1, 4, D)))
        pos.copy_(cuda(lens + step))
        ld.copy_(cuda(lens + step + 1))
        if step == 10:
            ld[1] = 0                                # a padded place in the batch
        table[:, :4] = order.view(3, 4)
        graph.replay()
        for p in eager:
            p.run()
        assert torch.equal(first[1]._result, eager[1]._result) and torch.equal(cache.pages, other.pages), step
        assert step != 10 or not first[1]._result[1].any()
    assert cache.errors() == 0 and other.errors() == 0


def test_calls_at_once(zt):
    """Decode steps and prompts side by side on streams of their own, again and again: each gives what it gives alone."""
    import torch
    rng = np.random.default_rng(34)
    lens = [900, 5000, 1, 300]
    cache, pool, table = kv.filled(zt, rng, lens, 32, 2, 128)
    ld, td = cuda(np.array(lens, np.int32)), cuda(table)
    plans = [zt.KvAttention(cache, cuda(fp16(rng, 4, t, 8, 128)), ld, td) for t in (1, 1, 4)]
    for nq, nk in (([300, 40], [300, 700]), ([9], [5000])):
        plans.append(zt.PromptAttention(cuda(fp16(rng, sum(nq), 4, 96)), cuda(fp16(rng, sum(nk), 2, 96)),
                                        cuda(fp16(rng, sum(nk), 2, 96)), cuda(prompt.offsets(nq)), cuda(prompt.offsets(nk))))
    want = [p.run().clone() for p in plans]
    streams = [torch.cuda.Stream() for _ in plans]
    torch.cuda.synchronize()
    for _ in range(30):
        for p, s in zip(plans, streams):
            with torch.cuda.stream(s):
                p._result.fill_(7.0)
                p.run()
    torch.cuda.synchronize()
    assert all(torch.equal(p._result, w) for p, w in zip(plans, want))
    assert cache.errors() == 0 and not any(p.errors() for p in plans[3:])
