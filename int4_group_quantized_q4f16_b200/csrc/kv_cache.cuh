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

constexpr int kRopeMax = 64;   // pairs of the largest head

struct KvAppendArgs {
    KvPlaces at;
    const int32_t *seq, *pos;
    const __half *k, *v, *q;      // q: null unless rotated
    __half *k_out, *q_out;        // null: not written
    long long ld_k, ld_v, ld_q, ld_k_out, ld_q_out;
    int q_heads, rope;
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

// code = round(x / s) + 7 in 0..15.  The quotient is correctly rounded: inv is the correctly rounded reciprocal, and one
// correction of x * inv by its exact remainder then gives the rounded quotient (Markstein's theorem; s has 11 significant
// bits).  x / s of two fp16 values is either exactly a half-integer or further from one than an fp32 rounding, so ties go
// to even as in exact arithmetic.  Adding 1.5 * 2^23 rounds to a whole number and leaves it in the low bits.
__device__ __forceinline__ uint32_t kv_code(float x, float s, float inv)
{
    const float q = x * inv, t = fmaf(fmaf(-q, s, x), inv, q);
    return (__float_as_uint(__fadd_rn(fminf(fmaxf(t, -7.f), 8.f), 12582912.f)) + 7u) & 15u;
}

// One thread per 8 values of a row's head: 2384 rows of 3 x 32 heads of 96 with rotation 43 us, 85 % of it issue slots
// (the rows' bytes, 82 MB, are 12.5 us).  Taking 16 rows at a time, so that a tile's V bytes leave as whole sectors, took 90 us:
// fewer and longer chains of the same instructions.  A group of 32 is four neighbouring
// lanes.  RoPE reads the pair's other half again (an L1 hit) instead of
// exchanging it between threads.
template <int D>
__global__ void __launch_bounds__(256) kv_append_kernel(const __grid_constant__ KvAppendArgs a)
{
    using T = KvTile<D>;
    constexpr int V8 = D / 8;
    __shared__ float2 turn[D / 2];
    kv_pdl_wait();
    const int row = blockIdx.x;
    const int pos = a.pos[row];
    const KvRow at = kv_row(a.at, a.seq[row], pos, T::kBytes);
    if (!at.tile) return;
    if (a.rope) {
        for (int i = threadIdx.x; i < D / 2; i += blockDim.x) {
            double sn, cs;
            sincos((double)pos * a.freq[i], &sn, &cs);
            turn[i] = make_float2((float)cs, (float)sn);
        }
        __syncthreads();
    }
    const int nk = a.at.kv_heads * V8, nq = a.q ? a.q_heads * V8 : 0, n = 2 * nk + nq;
    const long long head_stride = (long long)(a.at.page_size / kKvTile) * T::kBytes;
    // whole warps, so that exchanges name all lanes (a mask per group of four costs several instructions each)
    for (int it0 = blockIdx.y * blockDim.x + (threadIdx.x & ~31); it0 < n; it0 += gridDim.y * blockDim.x) {
        const bool live = it0 + (int)(threadIdx.x & 31) < n;
        const int it = live ? it0 + (threadIdx.x & 31) : n - 1;
        const int kind = it < nk ? 0 : it < 2 * nk ? 1 : 2;     // k, v, q
        const int rel = it - (kind == 0 ? 0 : kind == 1 ? nk : 2 * nk);
        const int head = rel / V8, v8 = rel % V8;
        const __half *src = kind == 0 ? a.k + row * a.ld_k : kind == 1 ? a.v + row * a.ld_v : a.q + row * a.ld_q;
        src += head * D;
        uint4 raw = *reinterpret_cast<const uint4 *>(src + 8 * v8);
        if (kind != 1 && a.rope) {
            const bool second = v8 >= V8 / 2;
            const int o8 = second ? v8 - V8 / 2 : v8 + V8 / 2, i0 = 8 * (second ? o8 : v8);
            const uint4 other = *reinterpret_cast<const uint4 *>(src + 8 * o8);
            uint32_t *x = reinterpret_cast<uint32_t *>(&raw);
            const uint32_t *y = reinterpret_cast<const uint32_t *>(&other);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const float2 xf = __half22float2(bits_h2(x[c])), yf = __half22float2(bits_h2(y[c]));
                const float2 t0 = turn[i0 + 2 * c], t1 = turn[i0 + 2 * c + 1];
                // each product and sum rounded by itself: x c - y s for the first half, x c + y s for the second
                const float p0 = __fmul_rn(yf.x, t0.y), p1 = __fmul_rn(yf.y, t1.y);
                const float r0 = __fadd_rn(__fmul_rn(xf.x, t0.x), second ? p0 : -p0);
                const float r1 = __fadd_rn(__fmul_rn(xf.y, t1.x), second ? p1 : -p1);
                x[c] = h2_bits(__floats2half2_rn(r0, r1));
            }
            __half *dst = kind == 0 ? a.k_out : a.q_out;
            if (dst && live) {
                dst += row * (kind == 0 ? a.ld_k_out : a.ld_q_out) + head * D + 8 * v8;
                *reinterpret_cast<uint4 *>(dst) = raw;
            }
        }
        if (__all_sync(0xffffffffu, kind == 2)) continue;
        // largest and smallest value of the group, NaN if there is one, two at a time
        const uint32_t *w = reinterpret_cast<const uint32_t *>(&raw);
        __half2 hi = bits_h2(w[0]), lo = hi;
#pragma unroll
        for (int c = 1; c < 4; ++c) {
            hi = __hmax2_nan(hi, bits_h2(w[c]));
            lo = __hmin2_nan(lo, bits_h2(w[c]));
        }
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
            hi = __hmax2_nan(hi, bits_h2(__shfl_xor_sync(0xffffffffu, h2_bits(hi), o)));
            lo = __hmin2_nan(lo, bits_h2(__shfl_xor_sync(0xffffffffu, h2_bits(lo), o)));
        }
        const float mx = __half2float(__hmax_nan(__low2half(hi), __high2half(hi))),
                    mn = __half2float(__hmin_nan(__low2half(lo), __high2half(lo)));
        const __half s = kv_scale(mx, mn, !(mx < INFINITY && mn > -INFINITY));
        const float sf = __half2float(s), inv = __frcp_rn(sf);
        uint32_t codes = 0;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const float2 x = __half22float2(bits_h2(w[c]));
            codes |= kv_code(x.x, sf, inv) << (8 * c) | kv_code(x.y, sf, inv) << (8 * c + 4);
        }
        if (!(sf > 0.f)) codes = 0x77777777u;                // zeros, or a group that reads back as NaN
        unsigned char *tile = at.tile + head * head_stride;
        const int t = at.t, g = v8 / 4;
        // its neighbour's codes: a byte of V holds rows r (low nibble) and r + 8 of a 16-row block
        const uint32_t theirs = __shfl_xor_sync(0xffffffffu, codes, 1);
        if (!live) continue;
        if (kind == 0) {
            const int j = v8 & 3;
            reinterpret_cast<uint32_t *>(tile)[t * V8 + j * T::kG + g] = codes;
            if (j == 0) reinterpret_cast<__half *>(tile + T::kKs)[((t & 7) * T::kG + g) * 2 + (t >> 3)] = s;
        } else if (kind == 1) {
            // the even lane writes r = 0..3, the odd one r = 4..7
            const uint32_t lo = (v8 & 1) ? theirs : codes, hi = (v8 & 1) ? codes : theirs;
            const int h = t >> 3, j = (t & 7) >> 1, e = t & 1, m = v8 / 2, r0 = (v8 & 1) * 4;
            unsigned char *base = tile + T::kV + 2 * e + h;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const uint32_t byte = ((lo >> (4 * (r0 + r))) & 15u) | (((hi >> (4 * (r0 + r))) & 15u) << 4);
                base[4 * ((m / 2) * 64 + (4 * (r0 + r) + j) * 2 + (m & 1))] = (unsigned char)byte;
            }
            if ((v8 & 3) == 0)
                reinterpret_cast<__half *>(tile + T::kVs)[((j * T::kG + g) * 2 + h) * 2 + e] = s;
        }
    }
}

struct KvGatherArgs {
    KvPlaces at;
    const int32_t *seq, *pos;
    __half *k, *v;
    long long ld_k, ld_v;
};

// fp16((code - 7) * s), one rounding: the code and the difference are exact.
__device__ __forceinline__ __half2 kv_value2(uint32_t c0, uint32_t c1, __half2 s2)
{
    const uint32_t v = 0x64006400u | c0 | (c1 << 16);                       // 1024 + code
    return __hmul2(__hsub2(bits_h2(v), bits_h2(0x64076407u)), s2);
}

// One thread per 8 values of a row's head, the append's places backwards: 5511 rows of 2 x 32 heads of 96 24 us (87 MB
// are 13.3 us), bound by issue slots: a V value's nibble is a byte load of its own.
template <int D>
__global__ void __launch_bounds__(256) kv_gather_kernel(const __grid_constant__ KvGatherArgs a)
{
    using T = KvTile<D>;
    constexpr int V8 = D / 8;
    kv_pdl_wait();
    const int row = blockIdx.x;
    const KvRow at = kv_row(a.at, a.seq[row], a.pos[row], T::kBytes);
    if (!at.tile) return;
    const int nk = a.at.kv_heads * V8;
    const long long head_stride = (long long)(a.at.page_size / kKvTile) * T::kBytes;
    const int t = at.t;
    for (int it = blockIdx.y * blockDim.x + threadIdx.x; it < 2 * nk; it += gridDim.y * blockDim.x) {
        const bool is_v = it >= nk;
        const int rel = is_v ? it - nk : it, head = rel / V8, v8 = rel % V8, g = v8 / 4;
        const unsigned char *tile = at.tile + head * head_stride;
        uint32_t codes;
        __half s;
        if (!is_v) {
            codes = reinterpret_cast<const uint32_t *>(tile)[t * V8 + (v8 & 3) * T::kG + g];
            s = reinterpret_cast<const __half *>(tile + T::kKs)[((t & 7) * T::kG + g) * 2 + (t >> 3)];
        } else {
            const int h = t >> 3, j = (t & 7) >> 1, e = t & 1, m = v8 / 2;
            const unsigned char *base = tile + T::kV + 2 * e + h + 4 * ((m / 2) * 64 + j * 2 + (m & 1));
            codes = 0;
#pragma unroll
            for (int r = 0; r < 8; ++r) codes |= ((uint32_t)(base[32 * r] >> (4 * (v8 & 1))) & 15u) << (4 * r);
            s = reinterpret_cast<const __half *>(tile + T::kVs)[((j * T::kG + g) * 2 + h) * 2 + e];
        }
        const __half2 s2 = __half2half2(s);
        uint4 o;
        uint32_t *po = reinterpret_cast<uint32_t *>(&o);
#pragma unroll
        for (int c = 0; c < 4; ++c)
            po[c] = h2_bits(kv_value2((codes >> (8 * c)) & 15u, (codes >> (8 * c + 4)) & 15u, s2));
        __half *dst = (is_v ? a.v + row * a.ld_v : a.k + row * a.ld_k) + head * D + 8 * v8;
        *reinterpret_cast<uint4 *>(dst) = o;
    }
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
