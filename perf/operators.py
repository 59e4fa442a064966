"""Cases of the attention side of a decoder layer: appending to a paged 4-bit cache, attention over that cache, attention over
whole prompts, and page copies.  Each operator is given in its plain form, as the library's call, and in 64 bits.

The cache.  A pool holds pages of `page` tokens (a multiple of 16); a page holds, for each kv head, page / 16 tiles of 16 tokens.
A tile of head size D is 18 D bytes: the K codes (8 D bytes), the V codes (8 D), the K scales (D) and the V scales (D).  A value is
(code - 7) * scale, one fp16 scale for 32 values of a token.  With G = D / 32, low nibbles first:
  K code of token t, d = 32 g + 8 j + n:                        nibble n of word t * D / 8 + j * G + g
  V code of token t = 8 h + 2 j + e, d = 16 m + 8 i + r:         nibble i of byte 2 e + h of word (m / 2) * 64 + (4 r + j) * 2 + m % 2
  K scale of token t = 8 h + r, group g:                         half (r * G + g) * 2 + h
  V scale of token t = 8 h + 2 j + e, group g:                   half ((j * G + g) * 2 + h) * 2 + e
"""
import random

import torch

own = False

THETA = 10000.0


def listed():
    return [
        # one decode step's new token of one sequence, Phi-3-mini's heads: the smallest call, where latency counts
        {"name": "append_token", "op": "append", "seqs": 1, "new": 1, "past": 1001, "back": False, "mix": 0, "q_heads": 32, "kv_heads": 32, "dim": 96, "page": 64},
        # a chunk of several prompts of different lengths behind a cached prefix, all read back as fp16 for the prompt attention
        {"name": "append_chunk", "op": "append", "seqs": 5, "new": 1337, "past": 700, "back": True, "mix": 1, "q_heads": 32, "kv_heads": 32, "dim": 96, "page": 64},
        # one token of one short sequence, Phi-3-mini's heads
        {"name": "decode_token", "op": "decode", "seqs": 1, "tokens": 1, "longest": 517, "mix": 0, "q_heads": 32, "kv_heads": 32, "dim": 96, "page": 64},
        # one token of one very long sequence, grouped heads: the work is split along the cache
        {"name": "decode_long", "op": "decode", "seqs": 1, "tokens": 1, "longest": 131071, "mix": 0, "q_heads": 32, "kv_heads": 8, "dim": 128, "page": 64},
        # a serving batch of different lengths, grouped heads
        {"name": "decode_batch", "op": "decode", "seqs": 61, "tokens": 1, "longest": 6001, "mix": 2, "q_heads": 32, "kv_heads": 8, "dim": 128, "page": 32},
        # four drafted tokens at a time for a small batch, Phi-3-mini's heads
        {"name": "decode_draft", "op": "decode", "seqs": 7, "tokens": 4, "longest": 3999, "mix": 3, "q_heads": 32, "kv_heads": 32, "dim": 96, "page": 16},
        # a short question, Phi-3-mini's heads
        {"name": "prompt_short", "op": "prompt", "seqs": 1, "longest": 45, "past": 0, "mix": 0, "causal": True, "q_heads": 32, "kv_heads": 32, "dim": 96},
        # packed prompts of different lengths, grouped heads
        {"name": "prompt_packed", "op": "prompt", "seqs": 9, "longest": 1501, "past": 0, "mix": 4, "causal": True, "q_heads": 32, "kv_heads": 8, "dim": 128},
        # a chunk of a prompt against a longer prefix, Phi-3-mini's heads
        {"name": "prompt_chunk", "op": "prompt", "seqs": 2, "longest": 1021, "past": 3100, "mix": 5, "causal": True, "q_heads": 32, "kv_heads": 32, "dim": 96},
        # one long prompt, Llama-7B's heads
        {"name": "prompt_long", "op": "prompt", "seqs": 1, "longest": 8192, "past": 0, "mix": 0, "causal": True, "q_heads": 32, "kv_heads": 32, "dim": 128},
        # a fork: the last, partly filled page of a few sequences, in every layer
        {"name": "copy_fork", "op": "copy", "layers": 32, "pages": 40, "moves": 3, "kv_heads": 8, "dim": 128, "page": 64},
        # compaction of a fragmented pool, in every layer
        {"name": "copy_compact", "op": "copy", "layers": 32, "pages": 301, "moves": 97, "kv_heads": 32, "dim": 96, "page": 64},
    ]


def _between(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    heads, kv, dim = rng.choice([(32, 32, 96), (32, 8, 128), (32, 32, 128), (24, 8, 64), (8, 1, 128), (32, 4, 96)])
    op = rng.choice(["append", "decode", "decode", "prompt", "prompt", "copy"])
    case = {"op": op, "q_heads": heads, "kv_heads": kv, "dim": dim, "mix": rng.randrange(1000)}
    if op == "append":
        seqs = _between(rng, 1, 64)
        case |= {"seqs": seqs, "new": _between(rng, 1, max(1, 4000 // seqs)), "past": _between(rng, 1, 700), "back": rng.random() < 0.5, "page": rng.choice([16, 32, 64, 128])}
    elif op == "decode":
        seqs = _between(rng, 1, 64)
        case |= {"seqs": seqs, "tokens": rng.choice([1, 1, 1, 2, 3, 5, 8]), "longest": _between(rng, 9, 80000 // seqs), "page": rng.choice([16, 32, 64, 128])}
    elif op == "prompt":
        seqs = _between(rng, 1, 16)
        case |= {"seqs": seqs, "longest": _between(rng, 1, 6000 // seqs), "past": rng.choice([0, 0, _between(rng, 1, 4000 // seqs)]), "causal": rng.random() < 0.85}
    else:
        pages = _between(rng, 8, 300)
        case = {"op": op, "kv_heads": kv, "dim": dim, "layers": rng.choice([1, 16, 32]), "pages": pages, "moves": rng.randint(1, pages // 3), "page": rng.choice([16, 32, 64])}
    return case


def _lengths(case, longest, salt):
    """Lengths of the case's sequences: the longest one first, shorter ones, and from four sequences on one of a single token."""
    rng = random.Random(1000 * case["mix"] + salt)
    lens = [longest] + [_between(rng, max(1, longest // 12), longest) for _ in range(case["seqs"] - 1)]
    return lens[:-1] + [1] if len(lens) > 3 else lens


def _sizes(case):
    """(new, past) tokens of each sequence."""
    if case["op"] == "decode":
        lens = [max(n, case["tokens"]) for n in _lengths(case, case["longest"], 1)]
        return [case["tokens"]] * len(lens), [n - case["tokens"] for n in lens]
    new = _lengths(case, case["longest"] if case["op"] == "prompt" else case["new"], 1)
    return new, _lengths(case, case["past"], 2) if case["past"] else [0] * len(new)


def _page_bytes(case):
    return case["kv_heads"] * case["page"] // 16 * 18 * case["dim"]


def work(case):
    if case["op"] == "copy":
        return {"bytes": 2 * case["layers"] * case["moves"] * _page_bytes(case), "flops": 0}
    new, past = _sizes(case)
    hq, hk, d = case["q_heads"], case["kv_heads"], case["dim"]
    if case["op"] == "append":
        rows, back = sum(new), sum(new) + (sum(past) if case["back"] else 0)
        cached = hk * d * 9 // 8  # bytes of a token's K and V in the cache
        return {"bytes": rows * (2 * d * (2 * hq + 3 * hk) + cached) + back * (cached + 4 * hk * d), "flops": rows * 3 * d * (hq + hk)}
    pairs = sum(n * p + (n * (n + 1) // 2 if case.get("causal", True) else n * n) for n, p in zip(new, past))
    kept = sum(new) + sum(past)
    if case["op"] == "decode":
        return {"bytes": kept * hk * d * 9 // 8 + 4 * sum(new) * hq * d, "flops": 4 * pairs * hq * d}
    return {"bytes": 4 * sum(new) * hq * d + 4 * kept * hk * d, "flops": 4 * pairs * hq * d}


# ------------------------------------------------------------------ inputs --
def _normal(gen, *shape, by=1.0):
    return (torch.randn(*shape, generator=gen, device="cuda") * by).half()


def _quantise(x):
    """(codes, scales) of fp16 values [..., D]: D / 32 scales."""
    g = x.float().unflatten(-1, (-1, 32))
    s = torch.maximum(g.amax(-1) / 8, -g.amin(-1) / 7).half()
    s32 = s.float().unsqueeze(-1)
    q = torch.where(s32 > 0, torch.round(g / s32) + 7, torch.full_like(g, 7)).clamp(0, 15)
    return q.flatten(-2).to(torch.uint8), s


def _pack(k, v):
    """Tiles [..., 18 D] (bytes) of fp16 k and v [..., 16, D]."""
    (kq, ks), (vq, vs) = _quantise(k), _quantise(v)
    lead, d = k.shape[:-2], k.shape[-1]
    n = kq.reshape(*lead, 16, d // 32, 4, 4, 2)  # t, g, j, byte, nibble
    n = n.movedim(-3, -4)
    kb = (n[..., 0] | n[..., 1] << 4).reshape(*lead, 8 * d)
    n = vq.reshape(*lead, 2, 4, 2, d // 32, 2, 2, 8)  # h, j, e, m / 2, m % 2, i, r
    n = n[..., 0, :] | n[..., 1, :] << 4  # h, j, e, m / 2, m % 2, r
    a = len(lead)
    vb = n.permute(*range(a), a + 3, a + 5, a + 1, a + 4, a + 2, a).reshape(*lead, 8 * d)
    ksb = ks.reshape(*lead, 2, 8, d // 32).permute(*range(a), a + 1, a + 2, a).contiguous().view(torch.uint8).reshape(*lead, d)
    vsb = vs.reshape(*lead, 2, 4, 2, d // 32).permute(*range(a), a + 1, a + 3, a, a + 2).contiguous().view(torch.uint8).reshape(*lead, d)
    return torch.cat([kb, vb, ksb, vsb], -1)


def _cache(case, gen, lens):
    """A pool whose pages hold random tokens, and a page table in a random order; the pool has a few pages more."""
    width = [-(-n // case["page"]) for n in lens]
    used, hk, d, tiles = sum(width), case["kv_heads"], case["dim"], case["page"] // 16
    spread = torch.rand(d, generator=gen, device="cuda") * 1.5 + 0.5  # some channels of K are wider than others
    shape = (used + 3, hk, tiles, 16, d)
    pool = _pack(_normal(gen, *shape) * spread.half(), _normal(gen, *shape)).reshape(1, used + 3, -1)
    order = torch.randperm(used + 3, generator=gen, device="cuda").int()
    table = torch.zeros(len(lens), max(width), dtype=torch.int32, device="cuda")
    at = 0
    for b, w in enumerate(width):
        table[b, :w] = order[at : at + w]
        at += w
    return pool, table


def _places(new, past):
    """(sequence, position) of the new tokens, sequence by sequence."""
    seq = torch.repeat_interleave(torch.arange(len(new)), torch.tensor(new))
    pos = torch.cat([torch.arange(p, p + n) for n, p in zip(new, past)])
    return seq.int().cuda(), pos.int().cuda()


def _offsets(lens):
    return torch.tensor([0] + list(lens)).cumsum(0).int().cuda()


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    state = {"case": case}
    if case["op"] == "copy":
        n = case["pages"]
        state["pool"] = torch.randint(0, 256, (case["layers"], n, _page_bytes(case)), generator=gen, device="cuda", dtype=torch.uint8)
        order = torch.randperm(n, generator=gen, device="cuda").int()
        state["src"], state["dst"] = order[: case["moves"]].clone(), order[case["moves"] : 2 * case["moves"]].clone()
    else:
        new, past = _sizes(case)
        rows, hq, hk, d = sum(new), case["q_heads"], case["kv_heads"], case["dim"]
    if case["op"] in ("append", "decode"):
        lens = [n + p for n, p in zip(new, past)]
        state["pool"], state["table"] = _cache(case, gen, lens)
        state["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    if case["op"] == "append":
        state["qkv"] = _normal(gen, rows, hq + 2 * hk, d)  # the QKV projection's output
        state["seq"], state["pos"] = _places(new, past)
        state["back_seq"], state["back_pos"] = _places(lens, [0] * len(lens)) if case["back"] else (state["seq"], state["pos"])
    elif case["op"] == "decode":
        state["q"] = _normal(gen, len(lens), case["tokens"], hq, d, by=1.5)
    elif case["op"] == "prompt":
        kept = rows + sum(past)
        state["q"], state["k"], state["v"] = _normal(gen, rows, hq, d, by=1.5), _normal(gen, kept, hk, d), _normal(gen, kept, hk, d)
        state["cu_q"], state["cu_k"] = _offsets(new), _offsets(n + p for n, p in zip(new, past))
    if own:
        state["plans"] = _plans(state)  # the launch plans that a program keeps, as it keeps the library's Pass
    return state


def _plans(state):
    from int4_group_quantized_q4f16_b200 import zt_q4

    case, op = state["case"], state["case"]["op"]
    if op == "prompt":
        return [zt_q4.PromptAttention(state["q"], state["k"], state["v"], state["cu_q"], state["cu_k"], causal=case["causal"])]
    cache = zt_q4.KvCache(state["pool"], page_size=case["page"], kv_heads=case["kv_heads"], head_dim=case["dim"])
    if op == "copy":
        return [zt_q4.KvCopy(cache, state["src"], state["dst"])]
    if op == "decode":
        return [zt_q4.KvAttention(cache, state["q"], state["lens"], state["table"])]
    q, k, v = state["qkv"].split([case["q_heads"], case["kv_heads"], case["kv_heads"]], 1)
    append = zt_q4.KvAppend(cache, k, v, state["seq"], state["pos"], state["table"], q=q, theta=THETA)
    return [append, zt_q4.KvGather(cache, state["back_seq"], state["back_pos"], state["table"])]


# -------------------------------------------------------------- plain form --
def _unpack(tiles, d):
    """K and V values [..., 16, D] (fp32) of tiles [..., 18 D]."""
    lead, a = tiles.shape[:-1], tiles.dim() - 1
    kb, vb, ks, vs = tiles.split([8 * d, 8 * d, d, d], -1)
    n = torch.stack([kb & 15, kb >> 4], -1).reshape(*lead, 16, 4, d // 32, 8).movedim(-2, -3)  # t, g, j, n
    ks = ks.contiguous().view(torch.float16).reshape(*lead, 8, d // 32, 2).permute(*range(a), a + 2, a, a + 1)
    k = (n.reshape(*lead, 16, d // 32, 32).float() - 7) * ks.reshape(*lead, 16, d // 32, 1).float()
    n = torch.stack([vb & 15, vb >> 4], -1).reshape(*lead, d // 32, 8, 4, 2, 2, 2, 2)  # m / 2, r, j, m % 2, e, h, i
    n = n.permute(*range(a), a + 5, a + 2, a + 4, a, a + 3, a + 6, a + 1)  # h, j, e, m / 2, m % 2, i, r
    vs = vs.contiguous().view(torch.float16).reshape(*lead, 4, d // 32, 2, 2).permute(*range(a), a + 2, a, a + 3, a + 1)
    v = (n.reshape(*lead, 16, d // 32, 32).float() - 7) * vs.reshape(*lead, 16, d // 32, 1).float()
    return k.flatten(-2), v.flatten(-2)


def _cached(state):
    """K and V values [B, kv_heads, longest, D] of the sequences in the cache."""
    case = state["case"]
    d = case["dim"]
    pages = state["pool"][0][state["table"].long()]  # B, pages, bytes
    tiles = pages.unflatten(-1, (case["kv_heads"], case["page"] // 16, 18 * d)).transpose(1, 2)
    return [x.flatten(2, 4) for x in _unpack(tiles, d)]


def _softmax_product(s, seen, v):
    """softmax(s) v over the places that are seen; rows that see nothing give zero."""
    s = s.masked_fill(~seen, float("-inf"))
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(top == float("-inf"), torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    return p @ v / torch.where(total == 0, torch.ones_like(total), total)


def _rotate(x, pos):
    """Rotary embedding of x [T, H, D] at positions pos: halves i and i + D / 2 are a pair."""
    d = x.shape[-1]
    angle = pos.double()[:, None] * THETA ** (-2 * torch.arange(d // 2, device=x.device, dtype=torch.float64) / d)
    c, s = angle.cos().float()[:, None], angle.sin().float()[:, None]
    a, b = x.float().chunk(2, -1)
    return torch.cat([a * c - b * s, b * c + a * s], -1).half()


def _store(state, k, v):
    """Writes the quantised rows k and v [T, kv_heads, D] to their places in the pool."""
    case = state["case"]
    d, g, dev = case["dim"], case["dim"] // 32, k.device
    page = state["table"][state["seq"].long(), (state["pos"] // case["page"]).long()].long()
    t, tile = (state["pos"] % 16).long()[:, None, None], (state["pos"] % case["page"] // 16).long()
    head = torch.arange(case["kv_heads"], device=dev)
    base = (page[:, None] * _page_bytes(case) + (head * (case["page"] // 16) + tile[:, None]) * 18 * d)[..., None]
    h, j, e = t // 8, t % 8 // 2, t % 2
    (kq, ks), (vq, vs) = _quantise(k), _quantise(v)
    n = kq.unflatten(-1, (g, 4, 4, 2)).transpose(-4, -3)
    flat = state["pool"].view(-1)
    flat[base + t * (d // 2) + torch.arange(d // 2, device=dev)] = (n[..., 0] | n[..., 1] << 4).flatten(-3)
    n = vq.unflatten(-1, (d // 16, 2, 8))
    m, r = torch.arange(d // 16, device=dev)[:, None], torch.arange(8, device=dev)
    word = ((m // 2 * 64 + r * 8 + m % 2).flatten()) + 2 * j
    flat[base + 8 * d + 4 * word + 2 * e + h] = (n[..., 0, :] | n[..., 1, :] << 4).flatten(-2)
    flat, at = flat.view(torch.float16), torch.arange(g, device=dev)
    flat[base // 2 + 8 * d + (t % 8 * g + at) * 2 + h] = ks
    flat[base // 2 + 8 * d + d // 2 + ((j * g + at) * 2 + h) * 2 + e] = vs


def _plain_append(state):
    case = state["case"]
    q, k, v = state["qkv"].split([case["q_heads"], case["kv_heads"], case["kv_heads"]], 1)
    q, k = _rotate(q, state["pos"]), _rotate(k, state["pos"])
    _store(state, k, v)
    ck, cv = _cached(state)
    at = state["back_seq"].long(), slice(None), state["back_pos"].long()
    return {"q": q, "k": k, "k_back": ck[at].half(), "v_back": cv[at].half()}


def _plain_decode(state):
    case, q = state["case"], state["q"].float()
    k, v = _cached(state)
    b, n, hq, d = q.shape
    hk, longest = case["kv_heads"], k.shape[2]
    q = q.unflatten(2, (hk, hq // hk)).permute(0, 2, 1, 3, 4).flatten(2, 3)  # B, kv_heads, tokens * group, D
    last = state["lens"][:, None] - n + torch.arange(n, device=q.device)  # the last position that a token sees
    seen = torch.arange(longest, device=q.device) <= last.repeat_interleave(hq // hk, 1)[:, None, :, None]
    v = v.masked_fill(torch.arange(longest, device=q.device)[:, None] >= state["lens"][:, None, None, None], 0)
    o = _softmax_product(q @ k.transpose(2, 3) * d**-0.5, seen, v)
    return o.unflatten(2, (n, hq // hk)).permute(0, 2, 1, 3, 4).flatten(2, 3).half()


def _plain_prompt(state):
    case, dev = state["case"], state["q"].device
    hq, hk, d = case["q_heads"], case["kv_heads"], case["dim"]
    q = state["q"].float().transpose(0, 1).unflatten(0, (hk, hq // hk))  # kv_heads, group, T, D
    k, v = state["k"].float().transpose(0, 1)[:, None], state["v"].float().transpose(0, 1)[:, None]
    cu_q, cu_k = state["cu_q"].long(), state["cu_k"].long()
    iq, ik = torch.arange(q.shape[2], device=dev), torch.arange(k.shape[2], device=dev)
    sq, sk = torch.searchsorted(cu_q, iq, right=True) - 1, torch.searchsorted(cu_k, ik, right=True) - 1
    seen = sq[:, None] == sk
    if case["causal"]:
        seen &= (ik - cu_k[sk + 1]) <= (iq - cu_q[sq + 1])[:, None]
    return _softmax_product(q @ k.transpose(2, 3) * d**-0.5, seen, v).flatten(0, 1).transpose(0, 1).half()


def _plain_copy(state):
    words = state["pool"].view(torch.int64)
    words[:, state["dst"].long()] = words[:, state["src"].long()]
    return state["pool"].view(torch.int32)


def run(state):
    if own:
        out = [plan.run() for plan in state["plans"]]
        if state["case"]["op"] == "append":
            (q, k), (k_back, v_back) = out
            return {"q": q, "k": k, "k_back": k_back, "v_back": v_back}
        return state["pool"].view(torch.int32) if state["case"]["op"] == "copy" else out[0]
    return {"append": _plain_append, "decode": _plain_decode, "prompt": _plain_prompt, "copy": _plain_copy}[state["case"]["op"]](state)


# ------------------------------------------------------------------ 64 bits --
def _exact_row(state, which, seq, pos):
    """Values (64 bits) [rows, kv_heads, D] that the pool holds at the places (seq, pos), value by value from the layout's formulas."""
    case = state["case"]
    d, dev = case["dim"], seq.device
    page = state["table"][seq.long(), (pos // case["page"]).long()].long()[:, None, None]
    t, tile = (pos % 16).long()[:, None, None], (pos % case["page"] // 16).long()[:, None, None]
    head, c = torch.arange(case["kv_heads"], device=dev)[:, None], torch.arange(d, device=dev)
    base = page * _page_bytes(case) + (head * (case["page"] // 16) + tile) * (18 * d)
    h, e = t // 8, t % 2
    if which == "k":
        byte, high = t * (d // 2) + (c % 32 // 8 * (d // 32) + c // 32) * 4 + c % 8 // 2, c % 2
        half = 8 * d + (t % 8 * (d // 32) + c // 32) * 2 + h
    else:
        j = t % 8 // 2
        byte, high = 8 * d + ((c // 32) * 64 + (4 * (c % 8) + j) * 2 + c // 16 % 2) * 4 + 2 * e + h, c % 16 // 8
        half = 8 * d + d // 2 + ((j * (d // 32) + c // 32) * 2 + h) * 2 + e
    flat = state["pool"].view(-1)
    code = flat[base + byte].to(torch.int32) >> 4 * high & 15
    return (code.double() - 7) * flat.view(torch.float16)[base // 2 + half].double()


def _exact_quantised(x):
    """What the 4-bit format keeps of fp16 values x [..., D], in 64 bits."""
    g = x.double().unflatten(-1, (-1, 32))
    s = torch.maximum(g.amax(-1, keepdim=True) / 8, g.amin(-1, keepdim=True) / -7).half().double()
    safe = torch.where(s == 0, torch.ones_like(s), s)
    return ((g / safe).round().clamp(-7, 8) * s).flatten(-2)


def _exact_rotated(x, pos):
    d = x.shape[-1]
    freq = torch.tensor([THETA ** (-2.0 * i / d) for i in range(d // 2)], dtype=torch.float64, device=x.device)
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=x.device), pos.double()[:, None, None] * freq)
    z = torch.complex(x[..., : d // 2].double(), x[..., d // 2 :].double()) * turn
    return torch.cat([z.real, z.imag], -1)


def _exact_attention(q, k, v, first, scale):
    """Attention of q [n, heads, D] over k and v [m, kv_heads, D] (64 bits); query i sees the keys up to first + i (all, where first is None)."""
    n, hq, d = q.shape
    m, hk = k.shape[:2]
    out = torch.zeros(n, hq, d, dtype=torch.float64, device=q.device)
    i, j = torch.arange(n, device=q.device), torch.arange(m, device=q.device)
    hidden = j > first + i[:, None] if first is not None else torch.zeros(n, m, dtype=torch.bool, device=q.device)
    for a in range(hq):
        s = (q[:, a] @ k[:, a // (hq // hk)].T) * scale
        s[hidden] = -torch.inf
        p = torch.softmax(s, -1).nan_to_num(0.0) if m else s
        out[:, a] = p @ v[:, a // (hq // hk)]
    return out


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "copy":
        return None  # bytes, not computed numbers
    new, past = _sizes(case)
    if case["op"] == "append":
        hq, hk = case["q_heads"], case["kv_heads"]
        q, k = _exact_rotated(state["qkv"][:, :hq], state["pos"]), _exact_rotated(state["qkv"][:, hq : hq + hk], state["pos"])
        kept_k, kept_v = _exact_quantised(k.half()), _exact_quantised(state["qkv"][:, hq + hk :])
        if case["back"]:
            seq, pos = state["back_seq"], state["back_pos"]
            old_k, old_v = _exact_row(state, "k", seq, pos), _exact_row(state, "v", seq, pos)
            is_new = pos >= torch.tensor(past, device=pos.device)[seq.long()]  # both orders go sequence by sequence
            old_k[is_new], old_v[is_new] = kept_k, kept_v
            kept_k, kept_v = old_k, old_v
        return {"q": q, "k": k, "k_back": kept_k, "v_back": kept_v}
    scale = case["dim"] ** -0.5
    outs = []
    for b, (n, p) in enumerate(zip(new, past)):
        if case["op"] == "decode":
            pos = torch.arange(n + p, device="cuda")
            seq = torch.full_like(pos, b)
            k, v = _exact_row(state, "k", seq, pos), _exact_row(state, "v", seq, pos)
            outs.append(_exact_attention(state["q"][b].double(), k, v, p, scale))
        else:
            q0, k0 = sum(new[:b]), sum(new[:b]) + sum(past[:b])
            k, v = state["k"][k0 : k0 + n + p].double(), state["v"][k0 : k0 + n + p].double()
            outs.append(_exact_attention(state["q"][q0 : q0 + n].double(), k, v, p if case["causal"] else None, scale))
    return torch.stack(outs) if case["op"] == "decode" else torch.cat(outs)
