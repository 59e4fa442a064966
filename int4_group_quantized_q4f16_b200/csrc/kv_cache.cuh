// kv_cache.cuh -- writing, reading back and moving the rows of the paged 4-bit
// KV cache (include/zt_q4.h: zt_q4_kv_append, zt_q4_kv_gather, zt_q4_kv_copy_pages).
#pragma once

#include "kv_common.cuh"

namespace zt {

// Place of row `row` (sequence, position): the kv-head-0 tile that holds it, or
// null for a row to skip (pos < 0: padding) or out of range (error bit).
struct KvRow {
    unsigned char *tile;       // tile of kv head 0; head h is h * head_stride further
    int t;                     // token within the tile
};

__device__ __forceinline__ KvRow kv_row(const KvPlaces &p, int seq, int pos, int tile_bytes)
{
    KvRow r{nullptr, pos & (kKvTile - 1)};
    if (pos < 0) return r;
    const int in_seq = pos / p.page_size;
    int page = -1;
    if (seq >= 0 && seq < p.n_seqs && in_seq < p.max_pages) page = p.table[(long long)seq * p.max_pages + in_seq];
    if (page < 0 || page >= p.n_pages) {
        kv_error(p.err, kErrKvPlace);
        return r;
    }
    r.tile = p.pages + page * p.page_bytes + (long long)((pos - in_seq * p.page_size) / kKvTile) * tile_bytes;
    return r;
}

// A word of V's codes holds four tokens of a tile: 2 j, 2 j + 1, 2 j + 8, 2 j + 9 (bytes 0, 2, 1, 3).  Rows of a call that
// lie in such a word are taken together, so that it is read or written once: a row by itself costs a byte access, and a
// sector, for every two values.
struct KvWord {
    unsigned char *tile;       // of kv head 0
    int row0;                  // call row of the tile's token 0, if it were among them
    int tokens;                // first token | last token << 8 | j << 16: the run of rows that this word's belong to
};
constexpr int kKvWindow = 16;  // rows whose runs a CTA takes

// The words of the runs (rows of consecutive tokens of one tile) that start in rows w0 .. w0 + 15, into `words` (32 at
// most); a run may end up to 15 rows later.  First warp; returns their number, in all threads after a barrier.
template <typename Args>
__device__ __forceinline__ int kv_words(const Args &a, int w0, int tile_bytes, KvWord *words, int *count)
{
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x, row = w0 - 1 + lane;
        KvRow at{nullptr, 0};
        if (row >= 0 && row < a.rows) at = kv_row(a.at, a.seq[row], a.pos[row], tile_bytes);
        const unsigned long long mine = reinterpret_cast<unsigned long long>(at.tile),
                                 before = __shfl_up_sync(0xffffffffu, mine, 1);
        const int t_before = __shfl_up_sync(0xffffffffu, at.t, 1);
        const unsigned starts = __ballot_sync(0xffffffffu, !(lane > 0 && mine && mine == before && at.t == t_before + 1));
        const int start = 31 - __clz(starts & ((2u << lane) - 1u));           // of this lane's run; lane 0 is one
        const unsigned later = starts & ~((2u << lane) - 1u);
        const int end = later ? __ffs(later) - 1 : 32;
        const int first = at.t - (lane - start), last = first + (end - start) - 1, j = (at.t & 7) >> 1;
        int lead = 2 * j + 9;                                                 // the word's first token in the run
        for (int t : {2 * j + 8, 2 * j + 1, 2 * j})
            if (t >= first) lead = t;
        const bool own = mine && start >= 1 && start <= kKvWindow && at.t == lead;
        const unsigned all = __ballot_sync(0xffffffffu, own);
        if (own) words[__popc(all & ((1u << lane) - 1u))] = {at.tile, row - at.t, first | (last << 8) | (j << 16)};
        if (lane == 0) *count = __popc(all);
    }
    __syncthreads();
    return *count;
}

constexpr int kRopeMax = 64;   // pairs of the largest head

struct KvAppendArgs {
    KvPlaces at;
    const int32_t *seq, *pos;
    const __half *k, *v, *q;      // q: null unless rotated
    __half *k_out, *q_out;        // null: not written
    long long ld_k, ld_v, ld_q, ld_k_out, ld_q_out;
    int rows, q_heads, rope;
    int row_ctas, v_ctas;         // CTAs per row (k and q) and per window of 16 rows (v); the rows' come first
    double freq[kRopeMax];        // theta^(-2 i / D)
};

// Scale of 32 values with the largest value mx and the smallest mn: codes 0..15
// stand for -7 .. 8 times it.  A group that holds an infinity or a NaN (bad)
// reads back as NaN.
__device__ __forceinline__ __half kv_scale(float mx, float mn, bool bad)
{
    const __half s = __float2half_rn(fmaxf(mx * 0.125f, __fdiv_rn(-mn, 7.0f)));
    return bad ? __ushort_as_half((unsigned short)0x7E00) : s;
}

// Codes round(x / s) + 7 in 0..15 of eight values, the first in the low nibble.  The quotient is correctly rounded: inv is
// the correctly rounded reciprocal, and one correction of x * inv by its exact remainder then gives the rounded quotient
// (Markstein's theorem; s has 11 significant bits).  x / s of two fp16 values is either exactly a half-integer or further
// from one than an fp32 rounding, so ties go to even as in exact arithmetic.  Adding 1.5 * 2^23 rounds to a whole number
// and leaves it in the low bits; the eight are added up in steps of 16, and what the constants and the sevens add to the
// sum is put right at the end.  x is clamped first, to -7 s and 8 s in fp16: 8 s is exact, and -7 s is off by 2^-11 of
// itself at most, which rounds to the same code.
__device__ __forceinline__ uint32_t kv_codes(const uint32_t (&x)[4], __half s, float sf, float inv)
{
    const __half2 most = __half2half2(__hmul(s, __float2half_rn(8.f))), least = __half2half2(__hmul(s, __float2half_rn(-7.f)));
    const uint64_t inv2 = f2_pack(inv, inv), minus_s = f2_pack(-sf, -sf), magic = f2_pack(12582912.f, 12582912.f);
    uint32_t acc = 0;
#pragma unroll
    for (int c = 3; c >= 0; --c) {
        const float2 v = __half22float2(__hmin2(__hmax2(bits_h2(x[c]), least), most));
        const uint64_t x2 = f2_pack(v.x, v.y), q = f2_mul(x2, inv2);
        const float2 u = f2_split(f2_add(f2_fma(f2_fma(q, minus_s, x2), inv2, q), magic));
        acc = (acc << 4) + __float_as_uint(u.y);
        acc = (acc << 4) + __float_as_uint(u.x);
    }
    // sum of 0x4B400000 * 16^n: 0x3F400000
    return acc - 0x3F400000u + 0x77777777u;
}

// Scale and codes of a group of 32, eight values in each of four neighbouring lanes.  Whole warp.
__device__ __forceinline__ uint32_t kv_quantize(const uint32_t (&w)[4], __half &s)
{
    // the group's largest value and its smallest one's negative in a half2, NaN if there is one
    __half2 hi = bits_h2(w[0]), lo = hi;
#pragma unroll
    for (int c = 1; c < 4; ++c) {
        hi = __hmax2_nan(hi, bits_h2(w[c]));
        lo = __hmin2_nan(lo, bits_h2(w[c]));
    }
    lo = __hneg2(lo);
    __half2 m = __hmax2_nan(__lows2half2(hi, lo), __highs2half2(hi, lo));
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) m = __hmax2_nan(m, bits_h2(__shfl_xor_sync(0xffffffffu, h2_bits(m), o)));
    const float2 ends = __half22float2(m);
    s = kv_scale(ends.x, -ends.y, !(ends.x < INFINITY && ends.y < INFINITY));
    const float sf = __half2float(s);
    // zeros, or a group that reads back as NaN: code 7
    return sf > 0.f ? kv_codes(w, s, sf, __frcp_rn(sf)) : 0x77777777u;
}

constexpr int kAppendThreads = 128;

// CTAs of two kinds.  k and q: by row, for its angles; one thread per 8 values of a head.  RoPE reads the pair's other half
// again (an L1 hit) instead of exchanging it between threads.
// 3008 rows of 3 x 32 heads of 96 with rotation (103 MB, 15.7 us at the memory's rate): 30.8 us, 23.6 without v, bound by
// the chains from load to store; 43.8 with v's codes written byte by byte in the rows' CTAs, 33.6 without the loads
// ahead.  CTAs of 96, 192 and 256 threads: 30.2, 34.3 and 38.6 (the last two, and 33.5 for 128, without the loads ahead).
template <int D>
__device__ __forceinline__ void kv_append_row(const KvAppendArgs &a, int row, int part)
{
    using T = KvTile<D>;
    constexpr int V8 = D / 8;
    __shared__ __align__(16) float turn[2][D / 2];      // cos, sin
    const int pos = a.pos[row];
    const KvRow at = kv_row(a.at, a.seq[row], pos, T::kBytes);
    if (!at.tile) return;
    const int nk = a.at.kv_heads * V8, n = nk + (a.q ? a.q_heads * V8 : 0), stride = a.row_ctas * kAppendThreads;
    const long long head_stride = (long long)(a.at.page_size / kKvTile) * T::kBytes;
    const __half *k = a.k + row * a.ld_k, *q = a.q + row * a.ld_q;
    // Whole warps, so that exchanges name all lanes (a mask per group of four costs several instructions each).  The next
    // values are on their way while these are worked on, the first ones during the angles.
    struct Item {
        bool live, is_q;
        int rel, head, v8;
    };
    auto item = [&](int it0) {
        Item i;
        const int it = min(it0 + (int)(threadIdx.x & 31), n - 1);
        i.live = it == it0 + (int)(threadIdx.x & 31);
        i.is_q = it >= nk;
        i.rel = i.is_q ? it - nk : it;
        i.head = i.rel / V8;
        i.v8 = i.rel - i.head * V8;
        return i;
    };
    uint4 raw = make_uint4(0, 0, 0, 0), other = raw;
    auto fetch = [&](int it0) {
        if (it0 >= n) return;
        const Item i = item(it0);
        const __half *src = (i.is_q ? q : k) + 8 * i.rel;
        raw = *reinterpret_cast<const uint4 *>(src);
        if (a.rope) other = *reinterpret_cast<const uint4 *>(src + (i.v8 >= V8 / 2 ? -D / 2 : D / 2));
    };
    const int from = part * kAppendThreads + (threadIdx.x & ~31);
    fetch(from);
    if (a.rope) {
        for (int i = threadIdx.x; i < D / 2; i += kAppendThreads) {
            double sn, cs;
            sincos((double)pos * a.freq[i], &sn, &cs);
            turn[0][i] = (float)cs;
            turn[1][i] = (float)sn;
        }
        __syncthreads();
    }
    for (int it0 = from; it0 < n; it0 += stride) {
        const Item i = item(it0);
        uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
        const uint4 pair = other;
        fetch(it0 + stride);
        if (a.rope) {
            const bool second = i.v8 >= V8 / 2;
            const int i0 = 8 * (second ? i.v8 - V8 / 2 : i.v8);
            // x c - y s for the first half, x c + y s for the second, each product and sum rounded by itself
            const uint32_t sign = second ? 0u : 0x80008000u;
            const uint32_t y[4] = {pair.x ^ sign, pair.y ^ sign, pair.z ^ sign, pair.w ^ sign};
#pragma unroll
            for (int c = 0; c < 4; c += 2) {
                const float4 cs = *reinterpret_cast<const float4 *>(&turn[0][i0 + 2 * c]),
                             sn = *reinterpret_cast<const float4 *>(&turn[1][i0 + 2 * c]);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float2 xf = __half22float2(bits_h2(w[c + e])), yf = __half22float2(bits_h2(y[c + e]));
                    const float2 r = f2_split(f2_add(f2_mul(f2_pack(xf.x, xf.y), e ? f2_pack(cs.z, cs.w) : f2_pack(cs.x, cs.y)),
                                                     f2_mul(f2_pack(yf.x, yf.y), e ? f2_pack(sn.z, sn.w) : f2_pack(sn.x, sn.y))));
                    w[c + e] = h2_bits(__floats2half2_rn(r.x, r.y));
                }
            }
            __half *dst = i.is_q ? a.q_out : a.k_out;
            if (dst && i.live)
                *reinterpret_cast<uint4 *>(dst + row * (i.is_q ? a.ld_q_out : a.ld_k_out) + 8 * i.rel) =
                    make_uint4(w[0], w[1], w[2], w[3]);
        }
        if (__all_sync(0xffffffffu, i.is_q)) continue;
        __half s;
        const uint32_t codes = kv_quantize(w, s);
        if (!i.live || i.is_q) continue;
        unsigned char *tile = at.tile + i.head * head_stride;
        const int t = at.t, g = i.v8 / 4, j = i.v8 & 3;
        reinterpret_cast<uint32_t *>(tile)[t * V8 + j * T::kG + g] = codes;
        if (j == 0) reinterpret_cast<__half *>(tile + T::kKs)[((t & 7) * T::kG + g) * 2 + (t >> 3)] = s;
    }
}

// v: by windows of 16 rows; one thread per 8 values of a word's tokens, four lanes to a group, words side by side.
template <int D>
__device__ __forceinline__ void kv_append_v(const KvAppendArgs &a, int window, int part)
{
    using T = KvTile<D>;
    __shared__ KvWord words[32];
    __shared__ int count;
    const int n_words = kv_words(a, window * kKvWindow, T::kBytes, words, &count);
    const int n = a.at.kv_heads * T::kG * n_words * 4;
    const long long head_stride = (long long)(a.at.page_size / kKvTile) * T::kBytes;
    for (int it0 = part * kAppendThreads + (threadIdx.x & ~31); it0 < n; it0 += a.v_ctas * kAppendThreads) {
        const int lane = threadIdx.x & 31, q = lane & 3, odd = q & 1;
        const bool live = it0 + lane < n;
        const int unit = (live ? it0 + lane : n - 1) / 4, group = unit / n_words;      // (head, group of 32), word
        const KvWord word = words[unit - group * n_words];
        const int first = word.tokens & 255, last = (word.tokens >> 8) & 255, j = word.tokens >> 16;
        const int head = group / T::kG, g = group - head * T::kG;
        uint32_t w[4][4], even[4], uneven[4];
        __half s[4];
        bool in[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int t = 2 * j + (u & 1) + 8 * (u >> 1);
            in[u] = t >= first && t <= last;
            uint4 raw = make_uint4(0, 0, 0, 0);
            if (in[u]) raw = *reinterpret_cast<const uint4 *>(a.v + (word.row0 + t) * a.ld_v + 32 * group + 8 * q);
            w[u][0] = raw.x, w[u][1] = raw.y, w[u][2] = raw.z, w[u][3] = raw.w;
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            // its neighbour's codes: a byte holds rows r (low nibble) and r + 8 of a 16-row block; the even lane takes
            // r = 0..3, the odd one r = 4..7
            const uint32_t codes = kv_quantize(w[u], s[u]), theirs = __shfl_xor_sync(0xffffffffu, codes, 1);
            const uint32_t lo = ((odd ? theirs : codes) >> (16 * odd)) & 0xFFFFu, hi = ((odd ? codes : theirs) >> (16 * odd)) & 0xFFFFu;
            even[u] = (lo & 0x0F0Fu) | ((hi & 0x0F0Fu) << 4);            // bytes r = 0, 2
            uneven[u] = ((lo >> 4) & 0x0F0Fu) | (hi & 0xF0F0u);          // bytes r = 1, 3
        }
        if (!live) continue;
        unsigned char *tile = word.tile + head * head_stride;
        unsigned char *base = tile + T::kV + 4 * (g * 64 + (16 * odd + j) * 2 + q / 2);
        __half *scales = reinterpret_cast<__half *>(tile + T::kVs) + (j * T::kG + g) * 4;
        if (in[0] && in[1] && in[2] && in[3]) {
            uint32_t *out = reinterpret_cast<uint32_t *>(base);
            const uint32_t e02 = __byte_perm(even[0], even[2], 0x5140), e13 = __byte_perm(even[1], even[3], 0x5140);
            const uint32_t u02 = __byte_perm(uneven[0], uneven[2], 0x5140), u13 = __byte_perm(uneven[1], uneven[3], 0x5140);
            out[0] = __byte_perm(e02, e13, 0x5410);
            out[8] = __byte_perm(u02, u13, 0x5410);
            out[16] = __byte_perm(e02, e13, 0x7632);
            out[24] = __byte_perm(u02, u13, 0x7632);
            if (q == 0)
                *reinterpret_cast<uint2 *>(scales) = make_uint2(h2_bits(__halves2half2(s[0], s[1])), h2_bits(__halves2half2(s[2], s[3])));
        } else {
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (in[u]) {
                    unsigned char *out = base + 2 * (u & 1) + (u >> 1);
                    out[0] = (unsigned char)even[u];
                    out[32] = (unsigned char)uneven[u];
                    out[64] = (unsigned char)(even[u] >> 8);
                    out[96] = (unsigned char)(uneven[u] >> 8);
                    if (q == 0) scales[u] = s[u];
                }
        }
    }
}

template <int D>
__global__ void __launch_bounds__(kAppendThreads) kv_append_kernel(const __grid_constant__ KvAppendArgs a)
{
    kv_pdl_wait();
    const int by_row = a.rows * a.row_ctas, x = (int)gridDim.x - 1 - (int)blockIdx.x;      // windows first
    if (x < by_row) kv_append_row<D>(a, x / a.row_ctas, x % a.row_ctas);
    else kv_append_v<D>(a, (x - by_row) / a.v_ctas, (x - by_row) % a.v_ctas);
}

struct KvGatherArgs {
    KvPlaces at;
    const int32_t *seq, *pos;
    __half *k, *v;
    long long ld_k, ld_v;
    int rows, row_ctas, v_ctas;   // as for the append
};

// fp16((code - 7) * s) of two codes, one rounding: 64 + code (codes at bits 4 and 20) or 1024 + code (at bits 0 and 16)
// and the differences are exact.
__device__ __forceinline__ uint32_t kv_low2(uint32_t w, __half2 s2)
{
    return h2_bits(__hmul2(__hsub2(bits_h2((w & 0x000F000Fu) | 0x64006400u), bits_h2(0x64076407u)), s2));
}
__device__ __forceinline__ uint32_t kv_high2(uint32_t w, __half2 s2)
{
    return h2_bits(__hmul2(__hsub2(bits_h2((w & 0x00F000F0u) | 0x54005400u), bits_h2(0x54705470u)), s2));
}

constexpr int kGatherThreads = 128;

// The append's places backwards: CTAs by row for k, a thread per 8 values of a head, and by windows of rows for v, a thread
// per 8 values of a word's tokens.  4188 rows of 2 x 32 heads of 96 (66 MB, 10.1 us at the memory's rate): 16.0 us; 23.8
// with v read byte by byte in the rows' CTAs.
template <int D>
__device__ __forceinline__ void kv_gather_row(const KvGatherArgs &a, int row, int part)
{
    using T = KvTile<D>;
    constexpr int V8 = D / 8;
    const KvRow at = kv_row(a.at, a.seq[row], a.pos[row], T::kBytes);
    if (!at.tile) return;
    const int n = a.at.kv_heads * V8, t = at.t;
    const long long head_stride = (long long)(a.at.page_size / kKvTile) * T::kBytes;
    for (int it = part * kGatherThreads + threadIdx.x; it < n; it += a.row_ctas * kGatherThreads) {
        const int head = it / V8, v8 = it - head * V8, g = v8 / 4;
        const unsigned char *tile = at.tile + head * head_stride;
        const uint32_t w = reinterpret_cast<const uint32_t *>(tile)[t * V8 + (v8 & 3) * T::kG + g], w8 = w >> 8;
        const __half2 s2 = __half2half2(reinterpret_cast<const __half *>(tile + T::kKs)[((t & 7) * T::kG + g) * 2 + (t >> 3)]);
        const uint32_t v04 = kv_low2(w, s2), v15 = kv_high2(w, s2), v26 = kv_low2(w8, s2), v37 = kv_high2(w8, s2);
        *reinterpret_cast<uint4 *>(a.k + row * a.ld_k + 8 * it) =
            make_uint4(__byte_perm(v04, v15, 0x5410), __byte_perm(v26, v37, 0x5410), __byte_perm(v04, v15, 0x7632),
                       __byte_perm(v26, v37, 0x7632));
    }
}

template <int D>
__device__ __forceinline__ void kv_gather_v(const KvGatherArgs &a, int window, int part)
{
    using T = KvTile<D>;
    __shared__ KvWord words[32];
    __shared__ int count;
    const int n_words = kv_words(a, window * kKvWindow, T::kBytes, words, &count);
    const int n = a.at.kv_heads * T::kG * n_words * 4;
    const long long head_stride = (long long)(a.at.page_size / kKvTile) * T::kBytes;
    for (int it = part * kGatherThreads + threadIdx.x; it < n; it += a.v_ctas * kGatherThreads) {
        const int unit = it / 4, q = it & 3, group = unit / n_words;
        const KvWord word = words[unit - group * n_words];
        const int first = word.tokens & 255, last = (word.tokens >> 8) & 255, j = word.tokens >> 16;
        const int head = group / T::kG, g = group - head * T::kG;
        const unsigned char *tile = word.tile + head * head_stride;
        const uint32_t *codes = reinterpret_cast<const uint32_t *>(tile + T::kV) + g * 64 + j * 2 + q / 2;
        const uint2 scales = *reinterpret_cast<const uint2 *>(tile + T::kVs + (j * T::kG + g) * 8);
        uint32_t w[8];
#pragma unroll
        for (int r = 0; r < 8; ++r) w[r] = codes[8 * r];
#pragma unroll
        for (int r = 0; r < 8; ++r) w[r] >>= 4 * (q & 1);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int t = 2 * j + (u & 1) + 8 * (u >> 1);
            if (t < first || t > last) continue;
            const unsigned byte = 2 * (u & 1) + (u >> 1), pick = byte | ((4 + byte) << 8);      // result bytes 0 and 2
            const __half2 pair = bits_h2(u < 2 ? scales.x : scales.y), s2 = u & 1 ? __high2half2(pair) : __low2half2(pair);
            uint32_t o[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) o[r] = kv_low2(__byte_perm(w[2 * r], w[2 * r + 1], pick), s2);
            *reinterpret_cast<uint4 *>(a.v + (word.row0 + t) * a.ld_v + 32 * group + 8 * q) = make_uint4(o[0], o[1], o[2], o[3]);
        }
    }
}

template <int D>
__global__ void __launch_bounds__(kGatherThreads) kv_gather_kernel(const __grid_constant__ KvGatherArgs a)
{
    kv_pdl_wait();
    const int by_row = a.rows * a.row_ctas, x = (int)gridDim.x - 1 - (int)blockIdx.x;      // windows first
    if (x < by_row) kv_gather_row<D>(a, x / a.row_ctas, x % a.row_ctas);
    else kv_gather_v<D>(a, (x - by_row) / a.v_ctas, (x - by_row) % a.v_ctas);
}

struct KvCopyArgs {
    unsigned char *pages;
    long long page_bytes, layer_bytes;
    int n_pages;
    const int32_t *src, *dst;
    unsigned int *err;
};

// Page src[x] of layer z onto page dst[x], gridDim.y CTAs per page; bound by memory (6.6 TB/s read and written).
__global__ void __launch_bounds__(256) kv_copy_kernel(const KvCopyArgs a)
{
    kv_pdl_wait();
    const int src = a.src[blockIdx.x], dst = a.dst[blockIdx.x];
    if (src < 0 || src >= a.n_pages || dst < 0 || dst >= a.n_pages) {
        if (threadIdx.x == 0) kv_error(a.err, kErrKvPlace);
        return;
    }
    if (src == dst) return;
    unsigned char *layer = a.pages + blockIdx.z * a.layer_bytes;
    const uint4 *from = reinterpret_cast<const uint4 *>(layer + src * a.page_bytes);
    uint4 *to = reinterpret_cast<uint4 *>(layer + dst * a.page_bytes);
    const int n = (int)(a.page_bytes / 16), step = gridDim.y * blockDim.x;
    constexpr int U = 4;   // loads in flight per thread
    for (int i = blockIdx.y * blockDim.x + threadIdx.x; i < n; i += U * step) {
        uint4 w[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (i + u * step < n) w[u] = from[i + u * step];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (i + u * step < n) to[i + u * step] = w[u];
    }
}

}  // namespace zt
