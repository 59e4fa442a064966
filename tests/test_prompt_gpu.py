"""GPU parity of attention over packed prompts (tcgen05) against float64 (kv_reference.attention).

Tolerances.  A weight is rounded to fp16 (2^-11); scores carry their fp32 accumulation error and that of the exponent's
argument, together below 2^-16 (|score| log2(e) scale stays below 64: 64 * 2^-24, and D products summed in fp32: D 2^-24
sum |q k| scale log2(e) < 2^-17), which moves weights by less than 2^-15; weights below 2^-14 of the reference lose up to
2^-25 of it each, and the reference may lie 2^8 below the largest: 2^-25 max|v| a key.  The output's own rounding adds half
an fp16 step: in all (2^-11 + 2^-15) sum w |v| + 2^-11 |o| + n 2^-25 max|v| + 2^-25."""
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


def offsets(lens):
    return np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)


def check(got, q, k, v, nq, nk, causal, scale, heads=None):
    cq, ck = offsets(nq), offsets(nk)
    heads = range(q.shape[1]) if heads is None else heads
    group = q.shape[1] // k.shape[1]
    for b, (n, m) in enumerate(zip(nq, nk)):
        for h in heads:
            qq, g = q[cq[b]:cq[b] + n, [h]], got[cq[b]:cq[b] + n, h]
            kk, vv = (x[ck[b]:ck[b] + m, [h // group]].astype(np.float64) for x in (k, v))
            with np.errstate(all="ignore"):
                want, mag = ref.attention(qq, kk, vv, [i + 1 + m - n if causal else m for i in range(n)], scale)
            want, mag = want[:, 0], mag[:, 0]
            top = np.nanmax(np.abs(np.where(np.isfinite(vv), vv, np.nan)), initial=0.0) if m else 0.0
            tol = (2.0**-11 + 2.0**-15) * mag + 2.0**-11 * np.abs(want) + m * 2.0**-25 * top + 2.0**-25
            assert np.array_equal(np.isnan(g), np.isnan(want)), (b, h, "NaN in other places")
            fine = np.isfinite(want)
            with np.errstate(invalid="ignore"):
                bad = ((np.abs(g.astype(np.float64) - want) > tol) & fine) | (~fine & ~np.isnan(want) & (g != want))
            assert not bad.any(), (b, h, np.argwhere(bad)[:4].tolist(), float(np.abs(g.astype(np.float64) - want)[fine].max()))


def run(zt, q, k, v, nq, nk, causal=True, scale=None, **more):
    import torch
    plan = zt.PromptAttention(cuda(q), cuda(k), cuda(v), cuda(offsets(nq)), cuda(offsets(nk)), causal=causal, scale=scale, **more)
    got = plan.run().cpu().numpy()
    again = plan.run().cpu().numpy()
    torch.cuda.synchronize()
    assert plan.errors() == 0
    assert np.array_equal(again.view(np.uint16), got.view(np.uint16)), "two runs differ"
    return got


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("D,heads,kv", [(64, 2, 2), (96, 2, 1), (128, 3, 1)])
@pytest.mark.parametrize("nq,nk", [
    ([1], [1]), ([45], [45]), ([128], [128]), ([129], [129]), ([300], [300]),
    ([1, 0, 17, 128, 40, 257], [1, 0, 17, 128, 40, 257]),        # packed, one empty
    ([5, 130, 64], [200, 131, 64]),                               # chunks behind a prefix
    ([200, 7, 140], [3, 0, 139]),                                 # fewer keys than queries: rows that see nothing
])
def test_prompt(zt, D, heads, kv, nq, nk, causal):
    rng = np.random.default_rng(D + sum(nq) + sum(nk))
    q, k, v = fp16(rng, sum(nq), heads, D, by=1.5), fp16(rng, sum(nk), kv, D), fp16(rng, sum(nk), kv, D)
    check(run(zt, q, k, v, nq, nk, causal), q, k, v, nq, nk, causal, D ** -0.5)


@pytest.mark.parametrize("D", [64, 96, 128])
def test_prompt_many_blocks(zt, D):
    """Enough heads and rows that a CTA takes two query tiles (checked on a few heads)."""
    rng = np.random.default_rng(D)
    nq, nk, heads = [700, 513, 31], [700, 1100, 31], 48
    q, k, v = fp16(rng, sum(nq), heads, D, by=1.5), fp16(rng, sum(nk), 12, D), fp16(rng, sum(nk), 12, D)
    check(run(zt, q, k, v, nq, nk), q, k, v, nq, nk, True, D ** -0.5, heads=[0, 7, 47])


def test_prompt_long(zt):
    rng = np.random.default_rng(2)
    nq, D = [4100], 128
    q, k, v = fp16(rng, 4100, 1, D, by=2.0), fp16(rng, 4100, 1, D), fp16(rng, 4100, 1, D)
    check(run(zt, q, k, v, nq, nq), q, k, v, nq, nq, True, D ** -0.5)


def test_prompt_strides_scale_and_other_rows(zt):
    """Views into a QKV buffer, out within a wider one: rows no sequence covers and the heads beside stay as they were."""
    import torch
    rng = np.random.default_rng(3)
    D, heads, kv, n = 96, 4, 2, 150
    qkv = fp16(rng, n + 20, heads + 2 * kv, D)
    dev = cuda(qkv)
    out = torch.full((n + 20, heads + 2, D), 7.0, dtype=torch.float16, device="cuda")
    cu = cuda(np.array([0, 50, n], np.int32))
    zt.PromptAttention(dev[:, :heads], dev[:, heads:heads + kv], dev[:, heads + kv:], cu, cu, scale=0.3, out=out[:, 1:-1]).run()
    out = out.cpu().numpy()
    q, k, v = qkv[:n, :heads], qkv[:n, heads:heads + kv], qkv[:n, heads + kv:]
    check(out[:n, 1:-1], q, k, v, [50, 100], [50, 100], True, 0.3)
    assert (out[n:] == 7).all() and (out[:, 0] == 7).all() and (out[:, -1] == 7).all()


@pytest.mark.parametrize("causal", [True, False])
def test_prompt_ignores_what_is_behind_a_sequence(zt, causal):
    """NaN and infinities in the next sequence's rows, and in rows that no sequence covers, stay out."""
    rng = np.random.default_rng(4)
    D, nq = 128, [37, 5, 129]
    q, k, v = (fp16(rng, sum(nq) + 60, 2, D) for _ in range(3))
    for x in (q, k, v):
        x[37:42] = np.nan
        x[sum(nq):] = np.inf
    got = run(zt, q, k, v, nq, nq, causal)
    assert np.isnan(got[37:42]).all()
    clean = [0, 1, 2]
    for b, at in ((0, slice(0, 37)), (2, slice(42, 171))):
        check(got[at], q[at], k[at], v[at], [nq[b]], [nq[b]], causal, D ** -0.5)


def test_prompt_rescales(zt):
    """Scores that climb by far more than the slack from tile to tile, and fall again; weights that vanish in between."""
    rng = np.random.default_rng(5)
    D, n = 64, 600
    q, k, v = np.ones((n, 1, D), np.float16), np.ones((n, 1, D), np.float16), fp16(rng, n, 1, D)
    k *= np.array([0, 3, -4, 7, 2], np.float16).repeat(120)[:, None, None]
    q[::7] *= np.float16(-1)
    check(run(zt, q, k, v, [n], [n], scale=0.1), q, k, v, [n], [n], True, 0.1)


@pytest.mark.parametrize("nq,nk", [(600, 600), (5, 5000)])
@pytest.mark.parametrize("scale", [2.0**-8, 2.0**-4, 0.125, 1.0, 2.0**20, 2.0**60])
def test_prompt_scores_of_any_size(zt, nq, nk, scale):
    """Scores up to 2^90, each of them exact in fp32 (a common value times small whole numbers), some equal: the largest ones
    that a row sees share the weight, all others lie too far below to count, and nothing overflows."""
    rng = np.random.default_rng(13)
    c = rng.permutation(np.r_[np.full(nk - nk // 3, 512), np.full(nk // 3 - 5, 1023), np.full(5, 1024)])
    q = np.full((nq, 3, 64), 1024, np.float16)
    q[:, 1], q[:, 2] = -1024, 16384
    k, v = np.broadcast_to(c[:, None, None], (nk, 1, 64)).astype(np.float16), fp16(rng, nk, 1, 64)
    check(run(zt, q, k, v, [nq], [nk], scale=scale), q, k, v, [nq], [nk], True, scale)


def test_prompt_bad_offsets_are_left_out(zt):
    """Offsets that decrease or leave the tensors: those sequences count as empty, nothing else is touched."""
    import torch
    rng = np.random.default_rng(6)
    D, n = 64, 100
    q, k, v = (fp16(rng, n, 1, D) for _ in range(3))
    out = torch.full((n, 1, D), 7.0, dtype=torch.float16, device="cuda")
    cu_q = np.array([0, 40, 10, 2**31 - 1, -7, 30], np.int32)     # only [0, 40) is a sequence of q
    cu_k = np.array([0, 40, 40, 40, 40, 40], np.int32)
    plan = zt.PromptAttention(cuda(q), cuda(k), cuda(v), cuda(cu_q), cuda(cu_k), out=out)
    plan.run()
    got = out.cpu().numpy()
    assert plan.errors() == 0
    check(got[:40], q[:40], k[:40], v[:40], [40], [40], True, D ** -0.5)
    assert (got[40:] == 7).all()
    cu_k[1] = n + 1                                                 # no keys then: zeros
    zt.PromptAttention(cuda(q), cuda(k), cuda(v), cuda(cu_q), cuda(cu_k), out=out).run()
    got = out.cpu().numpy()
    assert (got[:40] == 0).all() and (got[40:] == 7).all()


def test_prompt_without_rows_or_keys(zt):
    import torch
    e = lambda n: torch.empty((n, 2, 64), dtype=torch.float16, device="cuda")   # noqa: E731
    cu = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")            # noqa: E731
    assert zt.PromptAttention(e(0), e(3), e(3), cu(0, 0), cu(0, 3)).run().shape == (0, 2, 64)
    out = zt.PromptAttention(torch.ones_like(e(4)), e(0), e(0), cu(0, 4), cu(0, 0), causal=False).run()
    assert (out == 0).all()


def test_prompt_graph_and_stream(zt):
    import torch
    rng = np.random.default_rng(7)
    nq = [300, 20]
    q, k, v = (cuda(fp16(rng, 320, 2, 96)) for _ in range(3))
    cu = cuda(offsets(nq))
    plan = zt.PromptAttention(q, k, v, cu, cu)
    want = plan.run().clone()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            plan.run()
        for _ in range(2):
            plan._result.zero_()
            g.replay()
            assert torch.equal(plan._result, want)
        v.mul_(2)
        g.replay()
        replayed = plan._result.clone()
        assert torch.equal(plan.run(stream=side), replayed) and not torch.equal(replayed, want)
    torch.cuda.synchronize()


@pytest.mark.parametrize("at", [0, 70000, 2**17])
def test_prompt_sink(zt, at):
    """2^17 keys with 2^-26 of the weight of one more, whose value is zero: together 2^-9 of the output.  A weight is 2^-19 as
    the kernel holds it, an fp16 subnormal with a step of 2^-24: off by 2^-6 of itself at most.  The other errors (O summed in
    fp32 in 2^13 steps of 2^-24, the score's 2^-19, the output's rounding 2^-11) stay below 2^-9."""
    n, D = 2**17, 64
    q, k, v = np.ones((1, 1, D), np.float16), np.zeros((n + 1, 1, D), np.float16), np.ones((n + 1, 1, D), np.float16)
    k[at], v[at] = 1.0, 0.0
    got = run(zt, q, k, v, [1], [n + 1], causal=False, scale=26 * np.log(2) / D)
    want = 2.0**-9 / (1 + 2.0**-9)
    assert (np.abs(got.astype(np.float64) - want) <= (2.0**-6 + 2.0**-9) * want).all()


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("D,heads,kv", [(64, 2, 2), (96, 6, 2), (128, 8, 1), (64, 40, 8)])
@pytest.mark.parametrize("nq,nk", [([5], [5000]), ([137], [2724]), ([1], [9000]), ([130, 2, 0], [6000, 37, 3000]),
                                   ([3, 64], [4500, 0]), ([300], [1100])])
def test_prompt_few_rows_long_keys(zt, D, heads, kv, nq, nk, causal):
    """Few query tiles: the keys of each are split between CTAs, parts without keys or with a ragged end among them."""
    rng = np.random.default_rng(D + heads + sum(nk))
    q, k, v = fp16(rng, sum(nq), heads, D, by=1.5), fp16(rng, sum(nk), kv, D), fp16(rng, sum(nk), kv, D)
    check(run(zt, q, k, v, nq, nk, causal), q, k, v, nq, nk, causal, D ** -0.5, heads=sorted({0, heads // 2, heads - 1}))


@pytest.mark.parametrize("D,heads", [(64, 1), (96, 3), (128, 2), (128, 9)])
@pytest.mark.parametrize("nk", [257, 513, 1001, 1025, 1535, 2050, 3079, 4093, 6157])
def test_prompt_split_ragged_ends(zt, D, heads, nk):
    """The part that holds a ragged end leaves its result in the shared memory where that end's V rows were zeroed: ends
    in every 16-key step's middle, in parts of one to several tiles, infinities behind them, the same bits run after run."""
    import torch
    rng = np.random.default_rng(D + heads + nk)
    q, k, v = fp16(rng, 40, heads, D, by=1.5), fp16(rng, nk + 130, 1, D), fp16(rng, nk + 130, 1, D)
    k[nk:], v[nk:] = np.nan, np.inf
    plan = zt.PromptAttention(cuda(q), cuda(k), cuda(v), cuda(offsets([40])), cuda(offsets([nk])), causal=False)
    first = plan.run().clone()
    check(first.cpu().numpy(), q, k[:nk], v[:nk], [40], [nk], False, D ** -0.5, heads=[0, heads - 1])
    for _ in range(20):
        plan._result.fill_(7.0)
        assert torch.equal(plan.run(), first)
    assert plan.errors() == 0


def test_prompt_split_keys_that_are_not_seen(zt):
    """NaN in a long sequence's keys reaches the rows that see them, whichever part they are in; keys behind the sequence do not."""
    rng = np.random.default_rng(11)
    D, n = 64, 8000
    q, k, v = fp16(rng, 130, 1, D), fp16(rng, n + 300, 1, D), fp16(rng, n + 300, 1, D)
    k[n:] = np.nan
    v[n:] = np.inf
    k[n - 65] = np.nan                   # the row that this key belongs to and those behind it see it
    import torch
    cu_q, cu_k = offsets([130]), np.array([0, n], np.int32)
    plan = zt.PromptAttention(cuda(q), cuda(k), cuda(v), cuda(cu_q), cuda(cu_k), causal=True)
    got = plan.run().cpu().numpy()
    assert plan.errors() == 0
    assert np.array_equal(np.isnan(got[:, 0]).all(1), np.arange(130) >= 65) and not np.isnan(got[:65]).any()
    check(got[:65], q[:65], k[:n - 65], v[:n - 65], [65], [n - 65], True, D ** -0.5)


def test_prompt_split_keys_in_a_graph(zt):
    """Split and whole calls after one another in a graph, on a stream of their own: the same bits as outside."""
    import torch
    rng = np.random.default_rng(12)
    plans = []
    for nq, nk in (([9], [5000]), ([300, 40], [300, 700]), ([64], [3000])):
        q, k, v = fp16(rng, sum(nq), 4, 96), fp16(rng, sum(nk), 2, 96), fp16(rng, sum(nk), 2, 96)
        plans.append(zt.PromptAttention(cuda(q), cuda(k), cuda(v), cuda(offsets(nq)), cuda(offsets(nk))))
    want = [p.run().clone() for p in plans]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        outs = [p.run() for p in plans]
    for _ in range(3):
        for out in outs:
            out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want)) and not any(p.errors() for p in plans)
