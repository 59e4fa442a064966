"""The attention side of a decoder layer next to the projections, as a program uses them: a prompt through the batched
QKV projection, rotation and append, prompt attention and the output projection; then decode steps through a pass whose
QKV rows are rotated in its epilogue, append, attention over the 4-bit cache and the output projection; with sequences
forked, freed and the pool compacted in between.  Each call is checked against float64 on its own inputs."""
import numpy as np
import pytest

import kv_reference as ref
from int4_group_quantized_q4f16_b200 import synth
from int4_group_quantized_q4f16_b200.kv_pages import KvPages

pytestmark = pytest.mark.gpu

HEADS, KV, D, PAGE, THETA = 4, 2, 64, 16, 10000.0
HIDDEN, WIDTH = HEADS * D, (HEADS + 2 * KV) * D


@pytest.fixture(scope="module")
def zt():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from int4_group_quantized_q4f16_b200 import zt_q4
    return zt_q4


def cuda(a):
    import torch
    a = np.ascontiguousarray(a)
    return torch.from_numpy(a.view(np.int32) if a.dtype == np.uint32 else a).cuda()


class Layer:
    def __init__(self, zt, layers=2, n_pages=24):
        self.zt = zt
        rng = np.random.default_rng(0)
        qkv, s, _ = synth.problem(0, WIDTH, HIDDEN, M=1, proj=0)
        o, so, _ = synth.problem(1, HIDDEN, HIDDEN, M=1, proj=1)
        self.qkv, self.s = cuda(qkv), cuda((s.astype(np.float32) * 4).astype(np.float16))
        self.o, self.so = cuda(o), cuda(so)
        self.cache = zt.KvCache.empty(layers, n_pages, PAGE, KV, D)
        self.cache.pages.random_(0, 256)                       # what is not written may hold anything
        self.pages = KvPages(n_pages, PAGE)
        self.rng = rng

    def table(self, seqs):
        return cuda(self.pages.table(seqs))

    def prompt(self, seqs, lens, layer):
        """The attention output of packed new sequences; their K and V go to `layer` of the cache."""
        import torch
        zt, total = self.zt, sum(lens)
        x = cuda(self.rng.standard_normal((total, HIDDEN)).astype(np.float16))
        qkv = zt.gemm(self.qkv, self.s, x).view(total, HEADS + 2 * KV, D)
        seq = cuda(np.repeat(np.arange(len(seqs)), lens).astype(np.int32))
        pos = cuda(np.concatenate([np.arange(n) for n in lens]).astype(np.int32))
        q, k = zt.KvAppend(self.cache, qkv[:, HEADS:HEADS + KV], qkv[:, HEADS + KV:], seq, pos, self.table(seqs), layer=layer,
                           q=qkv[:, :HEADS], theta=THETA).run()
        cu = cuda(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32))
        out = zt.PromptAttention(q, k, qkv[:, HEADS + KV:], cu, cu).run()
        zt.gemm(self.o, self.so, out.view(total, HIDDEN))
        torch.cuda.synchronize()
        at = 0
        for n in lens:
            sl = slice(at, at + n)
            want, mag = ref.attention(*(t[sl].cpu().numpy().astype(np.float64) for t in (q, k, qkv[:, HEADS + KV:])),
                                      np.arange(n) + 1, D ** -0.5)
            err = np.abs(out[sl].cpu().numpy().astype(np.float64) - want)
            assert (err <= (2.0**-11 + 2.0**-15) * mag + 2.0**-11 * np.abs(want) + 2.0**-24 * (n + 1)).all()
            at += n
        return out

    def decode(self, seqs, x, layer):
        """One token of each sequence (pages already extended): the layer's attention output [n, HEADS, D]."""
        import torch
        zt, n = self.zt, len(seqs)
        lens = np.array([self.pages.length(s) for s in seqs], np.int32)
        pos = cuda(lens - 1)
        qkv = torch.empty((n, WIDTH), dtype=torch.float16, device="cuda")
        rot = (HEADS + KV) * D
        zt.Pass([{"kind": "gemv", "qw": self.qkv[:rot], "scales": self.s[:rot], "x": x, "out": qkv, "ld_out": WIDTH,
                  "rope": {"pos": pos, "head_dim": D, "theta": THETA}},
                 {"kind": "gemv", "qw": self.qkv[rot:], "scales": self.s[rot:], "x": x, "out": qkv[:, rot:], "ld_out": WIDTH}]).run()
        rows, table = qkv.view(n, HEADS + 2 * KV, D), self.table(seqs)
        zt.KvAppend(self.cache, rows[:, HEADS:HEADS + KV], rows[:, HEADS + KV:], cuda(np.arange(n, dtype=np.int32)), pos, table,
                    layer=layer).run()
        out = zt.KvAttention(self.cache, rows[:, None, :HEADS], cuda(lens), table, layer=layer).run()[:, 0]
        zt.gemv(self.o, self.so, out.reshape(n, HIDDEN))
        torch.cuda.synchronize()
        assert self.cache.errors() == 0
        pool = ref.Pool(self.cache.pages[layer].cpu().numpy(), PAGE, KV, D)
        for b, s in enumerate(seqs):
            k, v = pool.values(self.pages.pages(s), int(lens[b]))
            last = rows[b, HEADS:HEADS + KV].cpu().numpy()
            assert np.array_equal(k[-1].astype(np.float16), ref.dequantize(*ref.quantize(last)).astype(np.float16))
            want, mag = ref.attention(rows[b:b + 1, :HEADS].cpu().numpy(), k, v, [int(lens[b])], D ** -0.5)
            err = np.abs(out[b].cpu().numpy().astype(np.float64) - want[0])
            assert (err <= (2.0**-10 + 2.0**-14) * mag[0] + 2.0**-11 * np.abs(want[0]) + 2.0**-24 * (lens[b] + 1)).all()
        return out.cpu().numpy()

    def move(self, copies):
        if copies:
            src, dst = (cuda(np.array(c, np.int32)) for c in zip(*copies))
            self.zt.KvCopy(self.cache, src, dst).run()


def test_prompt_decode_fork_free_and_compact(zt):
    layer = Layer(zt)
    x = cuda(layer.rng.standard_normal((3, HIDDEN)).astype(np.float16))
    lens = {"a": 37, "b": 5, "c": 16}
    for s, n in lens.items():
        layer.pages.add(s)
        layer.pages.extend(s, n)
    for which in (0, 1):
        layer.prompt(list(lens), list(lens.values()), which)
    before = layer.cache.pages[:, layer.pages.pages("a")[:2]].clone()
    layer.move(layer.pages.fork("a", "a2"))
    layer.move(layer.pages.fork("c", "c2"))                      # ends at a page's end: nothing to copy
    for step in range(20):
        seqs = ["a", "b", "a2"] if step % 2 else ["c", "a", "a2"]
        for s in seqs:
            layer.pages.extend(s, 1)
        token = x.roll(step, 0).contiguous()
        token[2] = token[1] if step % 2 == 0 else token[0]       # a2 gets what a gets
        a, twin = (0, 2) if step % 2 else (1, 2)
        for which in (0, 1):
            out = layer.decode(seqs, token, which)
            assert np.array_equal(out[a].view(np.uint16), out[twin].view(np.uint16)), "the fork differs from its parent"
        if step == 6:
            layer.pages.free("b")
            layer.pages.add("b")
            layer.pages.extend("b", 0)
        if step == 9:
            layer.pages.free("c2")
            layer.move(layer.pages.compact())
    assert (layer.cache.pages[:, layer.pages.pages("a2")[:2]] == before).all(), "shared pages changed"


def test_chunked_prompt_behind_a_cached_prefix(zt):
    """A second chunk attends to the first one through the cache: gathered rows, then prompt attention with nk > nq."""
    import torch
    layer = Layer(zt)
    rng, first, second = layer.rng, 50, 33
    layer.pages.add("a")
    layer.pages.extend("a", first + second)
    table, n = layer.table(["a"]), first + second
    rows = cuda(rng.standard_normal((n, HEADS + 2 * KV, D)).astype(np.float16))
    zero = cuda(np.zeros(n, np.int32))
    pos = cuda(np.arange(n, dtype=np.int32))
    q = torch.empty((n, HEADS, D), dtype=torch.float16, device="cuda")
    for sl in (slice(0, first), slice(first, n)):
        zt.KvAppend(layer.cache, rows[sl, HEADS:HEADS + KV], rows[sl, HEADS + KV:], zero[sl], pos[sl], table, layer=1,
                    q=rows[sl, :HEADS], theta=THETA, q_out=q[sl]).run()
    k, v = zt.KvGather(layer.cache, zero, pos, table, layer=1).run()
    out = zt.PromptAttention(q[first:], k, v, cuda(np.array([0, second], np.int32)), cuda(np.array([0, n], np.int32))).run()
    step = zt.KvAttention(layer.cache, q[None, -16:], cuda(np.array([n], np.int32)), table, layer=1).run()
    torch.cuda.synchronize()
    assert layer.cache.errors() == 0
    kk, vv = (t.cpu().numpy().astype(np.float64) for t in (k, v))
    want, mag = ref.attention(q[first:].cpu().numpy(), kk, vv, first + 1 + np.arange(second), D ** -0.5)
    tol = (2.0**-11 + 2.0**-15) * mag + 2.0**-11 * np.abs(want) + 2.0**-24 * n
    assert (np.abs(out.cpu().numpy() - want) <= tol).all()
    # the decode kernel over the same cache: its last 16 tokens (the gathered fp16 rows are within half a step of its values)
    tol = (2.0**-10 + 2.0**-14 + 2.0**-9) * mag[-16:] + 2.0**-11 * np.abs(want[-16:]) + 2.0**-24 * n
    assert (np.abs(step[0].cpu().numpy() - want[-16:]) <= tol).all()
