// kv_attn.cuh -- attention of a few query tokens per sequence over the paged
// 4-bit KV cache (include/zt_q4.h: zt_q4_kv_attention).
//
// Mathematics.  For a kv head, the columns are its (query token, query head)
// pairs; per tile of 16 cached tokens
//   S[t][c] = sum_g ks[t][g] (sum_{d in g} kc[t][d] q[d][c] - 7 sum_{d in g} q[d][c])
//   p[t][c] = 2^(scale log2(e) S[t][c] - R[c])
//   O[d][c] += sum_t (vc[t][d] - 7) (p[t][c] vs[t][g(d)])
// and the result is O[d][c] / sum_t p[t][c].  kc and vc are the 4-bit codes, ks
// and vs the fp16 scales of 32 values.
//
// Both products are mma.sync m16n8k16 with the codes as the A operand: a code
// pair masked out of its word is a pair of fp16 subnormals (code * 2^-24, or
// 16 times that for the high nibbles), so unpacking costs one logic instruction
// per two values and the products are exact.  The matrix unit aligns its sums to
// the operands' nominal exponents, and a subnormal's lies up to 2^10 above its
// value: harmless for the 32 terms of a score's group, which are scaled and added
// in fp32, but O runs on over all tiles.  So V's pairs take one fma more, to
// (code - 7) * 2^-10, normal numbers.  The tiles are stored in the order
// of the A fragments (K: tokens by d; V: d by tokens), and p goes from the first
// product's accumulator to the second's B operand with one 8x8 transpose.
// tcgen05 would need the unpacked codes written to shared memory first (4x the
// cache's bytes); the work is bound by the cache's bytes.
//
// R is a reference, not the running maximum: p may exceed 2^kOff.., so O and the
// sum of p are rescaled only when a score passes R by kOff + 2.  kOff keeps p * vs in
// the upper range of fp16: with scales below 2 (values below 14) p * vs stays
// under 2^15, and a weight of 2^-26 of the largest one still has 3 bits.  A tile
// with a larger scale sets the offset to 0 (p <= 4, p * vs <= 4 * 65504 / 7).
// p is rounded to fp16, p * vs once more; sums of p and O are fp32.
//
// Work split.  The (sequence, kv head) segments are laid end to end in tiles and
// cut into equal runs, one per CTA, then one per warp: ragged batches and single
// long sequences balance alike.  Each warp streams its run through a private ring
// of bulk copies (one copy = one tile, K and V).  Segments cut between warps are
// joined in shared memory, segments cut between CTAs by kv_attn_join_kernel,
// always in the order of the tokens: results do not depend on timing.
#pragma once

#include "kv_common.cuh"

namespace zt {

struct KvAttnArgs {
    KvPlaces at;
    const __half *q;
    __half *out;
    const int32_t *lens;
    float *part;               // partial results of segments cut between CTAs
    long long ld_q, ld_out;    // elements between query tokens
    int tokens;                // query tokens per sequence
    int q_heads, group;        // group = q_heads / kv_heads
    int cols, blocks;          // columns of a kv head (tokens * group), and blocks of 8 NT of them
    int ctas;                  // CTAs of the main kernel
    float scale_log2;          // softmax scale * log2(e)
};

template <int D, int NT>
struct KvAttnCfg {
    using T = KvTile<D>;
    static constexpr int kWarps = NT == 1 ? 16 : 8;
    static constexpr int kStages = 4;
    static constexpr int kCols = 8 * NT;
    static constexpr int kPart = kCols * (D + 2);                      // floats: O, then R and the sum of p per column
    static constexpr int kRing = kStages * T::kBytes;                  // per warp; holds the last partial at the end
    static constexpr int kPartBytes = (kPart * 4 + 15) / 16 * 16;
    static_assert(kPartBytes <= kRing, "a warp's last partial goes to its ring");
    static constexpr int kBars = kWarps * kStages * 8;
    static constexpr int kFlags = 3 * kWarps * 4;
    static constexpr int kSmem = kWarps * (kRing + kPartBytes) + kBars + kFlags;   // + the prefix sums, 4 bytes per sequence
};

constexpr int kKvSeqs = 4096;          // sequences per call (prefix sums in shared memory)
constexpr int kKvWarpTiles = 1;        // tiles per warp below which fewer CTAs are used
constexpr float kKvOff = 12.f, kKvSlack = 2.f;

// Runs of tiles: CTA c of n takes [T c / n, T (c + 1) / n).
__device__ __forceinline__ int kv_run(int total, int c, int n) { return (int)((long long)total * c / n); }
__device__ __forceinline__ int kv_owner(int total, int x, int n)
{
    return (int)((((long long)x + 1) * n - 1) / total);
}

// Number of CTAs that share `total` tiles.
__device__ __forceinline__ int kv_ctas(int total, int ctas, int warps)
{
    return max(1, min(ctas, (total + warps * kKvWarpTiles - 1) / (warps * kKvWarpTiles)));
}

// Cached tokens of sequence b: its length, at most what its row of the page table holds.
__device__ __forceinline__ int kv_len(const KvAttnArgs &a, int b)
{
    const int n = a.lens[b], most = a.at.max_pages * a.at.page_size;
    if (n < 0 || n > most) {
        kv_error(a.at.err, kErrKvPlace);
        return n < 0 ? 0 : most;
    }
    return n;
}

__device__ __forceinline__ void kv_mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1, float c0, float c1, float c2, float c3)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}

__device__ __forceinline__ uint32_t kv_transpose(uint32_t v)
{
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

// (code - 7) * 2^-10 of a pair of codes masked out of its word: f undoes the subnormals' 2^-24 (and a high nibble's 16).
__device__ __forceinline__ uint32_t kv_value(uint32_t codes, float f)
{
    return h2_bits(__hfma2(bits_h2(codes), __float2half2_rn(f), __float2half2_rn(-7.f * 0x1p-10f)));
}

__device__ __forceinline__ float kv_exp2(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// N words (N = 2, 3 or 4) at a shared address aligned to 4 N bytes (4 for N = 3).
template <int N>
__device__ __forceinline__ void kv_lds(uint32_t (&w)[N], uint32_t addr)
{
    if constexpr (N == 4)
        asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(addr));
    else if constexpr (N == 2)
        asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr));
    else
#pragma unroll
        for (int i = 0; i < N; ++i) asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w[i]) : "r"(addr + 4 * i));
}

// prefix[b] = tiles of the sequences before b, each counted for every kv head and column block.
__device__ __forceinline__ void kv_prefix(const KvAttnArgs &a, int *prefix)
{
    const int per = a.at.kv_heads * a.blocks;
    for (int b = threadIdx.x; b < a.at.n_seqs; b += blockDim.x)
        prefix[b + 1] = (kv_len(a, b) + kKvTile - 1) / kKvTile * per;
    if (threadIdx.x == 0) prefix[0] = 0;
    __syncthreads();
    if (threadIdx.x < 32) {
        int base = 0;
        for (int b0 = 0; b0 < a.at.n_seqs; b0 += 32) {
            const int b = b0 + threadIdx.x;
            int v = b < a.at.n_seqs ? prefix[b + 1] : 0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, v, o);
                if ((int)threadIdx.x >= o) v += u;
            }
            if (b < a.at.n_seqs) prefix[b + 1] = base + v;
            base += __shfl_sync(0xffffffffu, v, 31);
        }
    }
    __syncthreads();
}

// A position in the run of tiles: sequence, head-and-block, tile.
struct KvCursor {
    int b, hc, tile, tiles, len;
    __device__ __forceinline__ void seek(const KvAttnArgs &a, const int *prefix, int x)
    {
        int lo = 0, hi = a.at.n_seqs;                       // prefix[lo] <= x < prefix[hi]
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (prefix[mid] <= x) lo = mid;
            else hi = mid;
        }
        b = lo;
        enter(a);
        const int rel = x - prefix[b];
        hc = rel / tiles;
        tile = rel - hc * tiles;
    }
    __device__ __forceinline__ void enter(const KvAttnArgs &a)
    {
        len = min(max(a.lens[b], 0), a.at.max_pages * a.at.page_size);
        tiles = (len + kKvTile - 1) / kKvTile;
    }
    // on to the next tile; there is one (the caller counts the run)
    __device__ __forceinline__ void next(const KvAttnArgs &a)
    {
        if (++tile < tiles) return;
        tile = 0;
        if (++hc < a.at.kv_heads * a.blocks) return;
        hc = 0;
        do {
            if (++b >= a.at.n_seqs) {
                b = 0;                                      // behind the last tile: never used
                tiles = 1;
                return;
            }
            enter(a);
        } while (tiles == 0);
    }
};

// Columns of head-and-block hc.
__device__ __forceinline__ int kv_columns(const KvAttnArgs &a, int hc, int kcols)
{
    return min(kcols, a.cols - hc % a.blocks * kcols);
}

// Row of the output for column c of (b, hc).
__device__ __forceinline__ __half *kv_out_row(const KvAttnArgs &a, int b, int hc, int c, int kcols, int D)
{
    const int h = hc / a.blocks, col = (hc - h * a.blocks) * kcols + c;
    const int i = col / a.group, head = h * a.group + (col - i * a.group);
    return a.out + ((long long)b * a.tokens + i) * a.ld_out + head * D;
}

template <int D, int NT>
__global__ void __launch_bounds__(KvAttnCfg<D, NT>::kWarps * 32, 1) kv_attn_kernel(const __grid_constant__ KvAttnArgs a)
{
    using C = KvAttnCfg<D, NT>;
    using T = KvTile<D>;
    constexpr int G = T::kG, W = C::kWarps, S = C::kStages;
    extern __shared__ __align__(128) unsigned char kv_smem_raw[];
    unsigned char *rings = kv_smem_raw;
    float *heads = reinterpret_cast<float *>(kv_smem_raw + W * C::kRing);      // a warp's first partial
    const uint32_t bars = kv_smem(kv_smem_raw) + W * (C::kRing + C::kPartBytes);
    int *prefix = reinterpret_cast<int *>(kv_smem_raw + C::kSmem);
    // all shared memory is dynamic: the opt-in limit leaves no room for a static part
    int *open = prefix - 3 * W;      // 1: the warp's last segment goes on in the next warp
    int *began = prefix - 2 * W;     // 1: that segment began in this warp
    int *first = prefix - W;         // 1: the warp wrote a partial of a segment that began earlier and ended in it

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, j = lane & 3;
    if (lane < S) asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(bars + 8 * (warp * S + lane)) : "memory");
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    kv_pdl_launch();
    kv_pdl_wait();
    kv_prefix(a, prefix);
    const int total = prefix[a.at.n_seqs];
    const int n_ctas = kv_ctas(total, gridDim.x, W);
    if ((int)blockIdx.x >= n_ctas || total == 0) return;
    const int c_lo = kv_run(total, blockIdx.x, n_ctas), c_hi = kv_run(total, blockIdx.x + 1, n_ctas);
    const int lo = c_lo + kv_run(c_hi - c_lo, warp, W), hi = c_lo + kv_run(c_hi - c_lo, warp + 1, W);
    const int n = hi - lo;

    const uint32_t ring = kv_smem(rings) + warp * C::kRing, bar = bars + 8 * warp * S;
    float *tail = reinterpret_cast<float *>(rings + warp * C::kRing);
    float *head_part = heads + warp * (C::kPartBytes / 4);
    const int tpp = a.at.page_size / kKvTile;

    // the copying side runs S tiles ahead
    KvCursor ahead = {};
    unsigned bad = 0;                // stages whose tile has no page
    auto issue = [&](int s) {
        const int in_seq = ahead.tile / tpp;
        const int page = __ldg(a.at.table + (long long)ahead.b * a.at.max_pages + in_seq);
        bad &= ~(1u << s);
        if (page < 0 || page >= a.at.n_pages) {
            bad |= 1u << s;
            if (lane == 0) {
                kv_error(a.at.err, kErrKvPlace);
                asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar + 8 * s) : "memory");
            }
        } else if (lane == 0) {
            const int h = ahead.hc / a.blocks;
            const unsigned char *src = a.at.pages + page * a.at.page_bytes +
                                       ((long long)h * tpp + (ahead.tile - in_seq * tpp)) * T::kBytes;
            asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar + 8 * s), "r"(T::kBytes) : "memory");
            asm volatile(
                "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                    ring + s * T::kBytes),
                "l"(src), "r"(T::kBytes), "r"(bar + 8 * s) : "memory");
        }
        ahead.next(a);
    };

    KvCursor at = {};
    bool is_open = false, did_begin = false, did_first = false;
    if (n > 0) {
        at.seek(a, prefix, lo);
        ahead = at;
        for (int s = 0; s < min(S, n); ++s) issue(s);
    }

    float O[NT][D / 16][4], R[NT][2], L[NT][2], xg[NT][G][2];
    uint32_t qf[NT][G][4];
    int seen[NT][2];                 // tokens that columns 2j and 2j + 1 see
    float off = kKvOff;
    bool fresh = true, dead = false;
    int seg_tile0 = 0;
    for (int x = 0; x < n; ++x) {
        if (fresh) {
            // a new segment: its queries as B fragments, the sums of q per group, the columns' ends
            fresh = false;
            seg_tile0 = at.tile;
            off = kKvOff;
            const int h = at.hc / a.blocks, c0 = (at.hc - h * a.blocks) * C::kCols;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const int col = c0 + nt * 8 + r;
                const bool has = col < a.cols;
                const int i = has ? col / a.group : 0, qh = h * a.group + (has ? col - i * a.group : 0);
                const __half *src = a.q + ((long long)at.b * a.tokens + i) * a.ld_q + qh * D + 8 * j;
#pragma unroll
                for (int g = 0; g < G; ++g) {
                    uint4 w = has ? *reinterpret_cast<const uint4 *>(src + 32 * g) : make_uint4(0, 0, 0, 0);
                    const float2 f0 = __half22float2(bits_h2(w.x)), f1 = __half22float2(bits_h2(w.y)),
                                 f2 = __half22float2(bits_h2(w.z)), f3 = __half22float2(bits_h2(w.w));
                    float sum = ((f0.x + f0.y) + (f1.x + f1.y)) + ((f2.x + f2.y) + (f3.x + f3.y));
                    sum += __shfl_xor_sync(0xffffffffu, sum, 1);
                    sum += __shfl_xor_sync(0xffffffffu, sum, 2);
                    // codes are code * 2^-24, so the zero point's term carries the same factor
                    xg[nt][g][0] = -7.f * 0x1p-24f * __shfl_sync(0xffffffffu, sum, 8 * j);
                    xg[nt][g][1] = -7.f * 0x1p-24f * __shfl_sync(0xffffffffu, sum, 8 * j + 4);
                    // step 0 of a group meets codes 0, 4 | 2, 6 of the lane's word, step 1 codes 1, 5 | 3, 7,
                    // which come with a factor 16
                    const __half2 six = __float2half2_rn(0.0625f);
                    qf[nt][g][0] = __byte_perm(w.x, w.z, 0x5410);
                    qf[nt][g][1] = __byte_perm(w.y, w.w, 0x5410);
                    qf[nt][g][2] = h2_bits(__hmul2(bits_h2(__byte_perm(w.x, w.z, 0x7632)), six));
                    qf[nt][g][3] = h2_bits(__hmul2(bits_h2(__byte_perm(w.y, w.w, 0x7632)), six));
                }
#pragma unroll
                for (int m = 0; m < D / 16; ++m)
#pragma unroll
                    for (int e = 0; e < 4; ++e) O[nt][m][e] = 0.f;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    R[nt][e] = -INFINITY;
                    L[nt][e] = 0.f;
                    seen[nt][e] = at.len - a.tokens + 1 + (c0 + nt * 8 + 2 * j + e) / a.group;
                }
            }
        }
        const int s = x % S;
        if (!dead && !__all_sync(0xffffffffu, tc_wait(bar + 8 * s, (uint32_t)(x / S) & 1u, false))) {
            // the copy did not land in time: report it, give the other copies in flight their time,
            // and go on without reading tiles (the results are incomplete)
            if (lane == 0) kv_error(a.at.err, kErrKvWait);
            for (int y = x + 1; y < min(x + S, n); ++y) tc_wait(bar + 8 * (y % S), (uint32_t)(y / S) & 1u, false);
            __syncwarp();
            dead = true;
        }
        if (!dead && !((bad >> s) & 1u)) {
            const uint32_t tile = ring + s * T::kBytes;
            float P[NT][4];
            {
                uint32_t wa[G], wb[G], ks[G];
                kv_lds<G>(wa, tile + (r * 4 + j) * G * 4);
                kv_lds<G>(wb, tile + ((r + 8) * 4 + j) * G * 4);
                kv_lds<G>(ks, tile + T::kKs + r * G * 4);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) P[nt][e] = 0.f;
#pragma unroll
                for (int g = 0; g < G; ++g) {
                    const float2 sc = __half22float2(bits_h2(ks[g]));
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        float d[4];
                        kv_mma(d, wa[g] & 0x000F000Fu, wb[g] & 0x000F000Fu, (wa[g] >> 8) & 0x000F000Fu,
                               (wb[g] >> 8) & 0x000F000Fu, qf[nt][g][0], qf[nt][g][1], xg[nt][g][0], xg[nt][g][1],
                               xg[nt][g][0], xg[nt][g][1]);
                        kv_mma(d, wa[g] & 0x00F000F0u, wb[g] & 0x00F000F0u, (wa[g] >> 8) & 0x00F000F0u,
                               (wb[g] >> 8) & 0x00F000F0u, qf[nt][g][2], qf[nt][g][3], d[0], d[1], d[2], d[3]);
                        P[nt][0] = fmaf(sc.x, d[0], P[nt][0]);
                        P[nt][1] = fmaf(sc.x, d[1], P[nt][1]);
                        P[nt][2] = fmaf(sc.y, d[2], P[nt][2]);
                        P[nt][3] = fmaf(sc.y, d[3], P[nt][3]);
                    }
                }
            }
            // the V scales of this lane's tokens 2j, 2j + 1 and 2j + 8, 2j + 9
            uint32_t vs[2 * G];
#pragma unroll
            for (int g = 0; g < G; ++g) {
                uint32_t w[2];
                kv_lds<2>(w, tile + T::kVs + (j * G + g) * 8);
                vs[2 * g] = w[0];
                vs[2 * g + 1] = w[1];
            }
            const int t0 = at.tile * kKvTile;
            const bool edge = t0 + kKvTile > at.len - a.tokens + 1;      // some column does not see the whole tile
            if (edge) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (t0 + r + 8 * (e >> 1) >= seen[nt][e & 1]) P[nt][e] = -INFINITY;
                // places behind the sequence's end may hold anything
#pragma unroll
                for (int g = 0; g < G; ++g)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int t = t0 + 8 * h + 2 * j;
                        if (t >= at.len) vs[2 * g + h] = 0u;
                        else if (t + 1 >= at.len) vs[2 * g + h] &= 0xFFFFu;
                    }
            }
            uint32_t any = 0;
#pragma unroll
            for (int g = 0; g < 2 * G; ++g) any |= vs[g];
            const bool large = (any & 0x40004000u) != 0u;                // a scale of 2 or more
            const float sl = a.scale_log2 * 0x1p24f;
            bool lift = large && off > 0.f;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    lift |= fmaxf(P[nt][e], P[nt][e + 2]) * sl > R[nt][e] + (off + kKvSlack);
            if (__any_sync(0xffffffffu, lift)) {
                const float before = off;
                if (__any_sync(0xffffffffu, large)) off = 0.f;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float mx = fmaxf(P[nt][e], P[nt][e + 2]) * sl;
#pragma unroll
                        for (int o = 4; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                        const float ref = fmaxf(mx, R[nt][e] + before) - off;
                        const float f = R[nt][e] == ref ? 1.f : kv_exp2(R[nt][e] - ref);
                        R[nt][e] = ref;
                        L[nt][e] *= f;
#pragma unroll
                        for (int m = 0; m < D / 16; ++m) {
                            O[nt][m][e] *= f;
                            O[nt][m][e + 2] *= f;
                        }
                    }
            }
            uint32_t pt[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                // a column that has seen nothing yet keeps R = -inf: its weights are 2^-inf = 0
                const float r0 = R[nt][0] == -INFINITY ? 0.f : R[nt][0], r1 = R[nt][1] == -INFINITY ? 0.f : R[nt][1];
                const float p0 = kv_exp2(fmaf(P[nt][0], sl, -r0)), p1 = kv_exp2(fmaf(P[nt][1], sl, -r1));
                const float p2 = kv_exp2(fmaf(P[nt][2], sl, -r0)), p3 = kv_exp2(fmaf(P[nt][3], sl, -r1));
                L[nt][0] += p0 + p2;
                L[nt][1] += p1 + p3;
                pt[nt][0] = kv_transpose(h2_bits(__floats2half2_rn(p0, p1)));
                pt[nt][1] = kv_transpose(h2_bits(__floats2half2_rn(p2, p3)));
            }
#pragma unroll
            for (int g = 0; g < G; ++g) {
                uint32_t w[2];
                kv_lds<2>(w, tile + T::kV + (g * 64 + lane * 2) * 4);
                uint32_t va[2][4];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    va[u][0] = kv_value(w[u] & 0x000F000Fu, 0x1p14f);
                    va[u][1] = kv_value(w[u] & 0x00F000F0u, 0x1p10f);
                    va[u][2] = kv_value((w[u] >> 8) & 0x000F000Fu, 0x1p14f);
                    va[u][3] = kv_value((w[u] >> 8) & 0x00F000F0u, 0x1p10f);
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    uint32_t b0 = h2_bits(__hmul2(bits_h2(pt[nt][0]), bits_h2(vs[2 * g])));
                    uint32_t b1 = h2_bits(__hmul2(bits_h2(pt[nt][1]), bits_h2(vs[2 * g + 1])));
                    if (edge) {
                        // a hidden token's scale may be NaN: nothing times NaN is nothing here
                        b0 &= ~__vcmpeq2(pt[nt][0], 0u);
                        b1 &= ~__vcmpeq2(pt[nt][1], 0u);
                    }
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        float (&o)[4] = O[nt][2 * g + u];
                        kv_mma(o, va[u][0], va[u][1], va[u][2], va[u][3], b0, b1, o[0], o[1], o[2], o[3]);
                    }
                }
            }
        }
        __syncwarp();                                                     // all lanes have read the stage
        if (x + S < n && !dead) issue(s);

        const bool ends = at.tile + 1 == at.tiles;
        if (ends || x + 1 == n) {
            const bool begins = seg_tile0 == 0;
            const bool whole = ends && begins;
            float *dst = nullptr;
            if (!whole) {
                if (ends) did_first = true;
                else {
                    is_open = true;
                    did_begin = begins;
                }
                dst = ends ? head_part : tail;
            }
            __syncwarp();
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float l = L[nt][e];
#pragma unroll
                    for (int o = 4; o < 32; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
                    const int c = nt * 8 + 2 * j + e;
                    if (c >= kv_columns(a, at.hc, C::kCols)) continue;
                    if (whole) {
                        __half *row = kv_out_row(a, at.b, at.hc, c, C::kCols, D);
                        const float inv = l == 0.f ? 0.f : 0x1p10f / l;
#pragma unroll
                        for (int m = 0; m < D / 16; ++m) {
                            row[16 * m + r] = __float2half_rn(O[nt][m][e] * inv);
                            row[16 * m + 8 + r] = __float2half_rn(O[nt][m][e + 2] * inv);
                        }
                    } else {
#pragma unroll
                        for (int m = 0; m < D / 16; ++m) {
                            dst[c * D + 16 * m + r] = O[nt][m][e] * 0x1p10f;
                            dst[c * D + 16 * m + 8 + r] = O[nt][m][e + 2] * 0x1p10f;
                        }
                        if (r == 0) {
                            dst[C::kCols * D + c] = R[nt][e];
                            dst[C::kCols * (D + 1) + c] = l;
                        }
                    }
                }
            fresh = true;
        }
        at.next(a);
    }
    if (lane == 0) {
        open[warp] = is_open;
        began[warp] = did_begin;
        first[warp] = did_first;
    }
    __syncthreads();

    // Join the segments that this CTA's warps share: the warp in which such a segment begins, or the
    // first warp with tiles for one that began in an earlier CTA, walks on to where it ends.
    if (n == 0) return;
    KvCursor seg = {};
    auto join = [&](int w_end, bool ends_here, bool began_here) {
        // partials: this warp's tail (or, for a single partial, its head), the tails of the warps between, w_end's head or tail
        float *out_part = a.part + ((long long)blockIdx.x * 2 + (ends_here ? 0 : 1)) * C::kPart;
        for (int c = 0; c < kv_columns(a, seg.hc, C::kCols); ++c) {
            float top = -INFINITY;
            for (int w = warp; w <= w_end; ++w) {
                if (w > warp && kv_run(c_hi - c_lo, w, W) == kv_run(c_hi - c_lo, w + 1, W)) continue;
                const float *p = (w == w_end && ends_here) ? heads + w * (C::kPartBytes / 4)
                                                           : reinterpret_cast<float *>(rings + w * C::kRing);
                top = fmaxf(top, p[C::kCols * D + c]);
            }
            const float ref = top == -INFINITY ? 0.f : top;
            float l = 0.f, acc[D / 32];
#pragma unroll
            for (int e = 0; e < D / 32; ++e) acc[e] = 0.f;
            for (int w = warp; w <= w_end; ++w) {
                if (w > warp && kv_run(c_hi - c_lo, w, W) == kv_run(c_hi - c_lo, w + 1, W)) continue;
                const float *p = (w == w_end && ends_here) ? heads + w * (C::kPartBytes / 4)
                                                           : reinterpret_cast<float *>(rings + w * C::kRing);
                const float f = kv_exp2(p[C::kCols * D + c] - ref);
                l += p[C::kCols * (D + 1) + c] * f;
#pragma unroll
                for (int e = 0; e < D / 32; ++e) acc[e] += p[c * D + 32 * e + lane] * f;
            }
            if (ends_here && began_here) {
                __half *row = kv_out_row(a, seg.b, seg.hc, c, C::kCols, D);
                const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
                for (int e = 0; e < D / 32; ++e) row[32 * e + lane] = __float2half_rn(acc[e] * inv);
            } else {
#pragma unroll
                for (int e = 0; e < D / 32; ++e) out_part[c * D + 32 * e + lane] = acc[e];
                if (lane == 0) {
                    out_part[C::kCols * D + c] = top;
                    out_part[C::kCols * (D + 1) + c] = l;
                }
            }
        }
    };
    int w_first = 0;
    while (kv_run(c_hi - c_lo, w_first, W) == kv_run(c_hi - c_lo, w_first + 1, W)) ++w_first;
    if (warp == w_first && first[warp]) {
        // the segment that came in from an earlier CTA ends in this warp
        seg.seek(a, prefix, lo);
        join(warp, true, false);
    }
    if (open[warp] && (began[warp] || warp == w_first)) {
        seg.seek(a, prefix, hi - 1);
        int w = warp;
        bool ends_here = false;
        while (w + 1 < W) {
            ++w;
            if (kv_run(c_hi - c_lo, w, W) == kv_run(c_hi - c_lo, w + 1, W)) continue;
            if (first[w]) {
                ends_here = true;
                break;
            }
        }
        join(w, ends_here, began[warp]);
    }
}

// One CTA per (segment, column): joins what CTAs of the main kernel left of a
// segment they share, in order; writes zeros for a sequence without tokens.
template <int D, int NT>
__global__ void __launch_bounds__(128) kv_attn_join_kernel(const __grid_constant__ KvAttnArgs a)
{
    using C = KvAttnCfg<D, NT>;
    extern __shared__ int kv_join_prefix[];
    kv_pdl_wait();
    kv_prefix(a, kv_join_prefix);
    const int total = kv_join_prefix[a.at.n_seqs];
    const int per = a.at.kv_heads * a.blocks;
    const int b = blockIdx.x / per, hc = blockIdx.x - b * per, c = blockIdx.y, d = threadIdx.x;
    if (c >= kv_columns(a, hc, C::kCols) || d >= D) return;
    __half *row = kv_out_row(a, b, hc, c, C::kCols, D);
    const int tiles = (kv_join_prefix[b + 1] - kv_join_prefix[b]) / per;
    if (tiles == 0) {
        row[d] = __float2half_rn(0.f);
        return;
    }
    const int n_ctas = kv_ctas(total, a.ctas, C::kWarps);
    const int x0 = kv_join_prefix[b] + hc * tiles, x1 = x0 + tiles;
    const int f = kv_owner(total, x0, n_ctas), l = kv_owner(total, x1 - 1, n_ctas);
    if (f == l) return;                            // one CTA had it all
    auto part = [&](int cta) { return a.part + ((long long)cta * 2 + (cta == l ? 0 : 1)) * C::kPart; };
    float top = -INFINITY;
    for (int i = f; i <= l; ++i) top = fmaxf(top, part(i)[C::kCols * D + c]);
    const float ref = top == -INFINITY ? 0.f : top;
    float sum = 0.f, acc = 0.f;
    for (int i = f; i <= l; ++i) {
        const float *p = part(i);
        const float w = kv_exp2(p[C::kCols * D + c] - ref);
        sum += p[C::kCols * (D + 1) + c] * w;
        acc += p[c * D + d] * w;
    }
    row[d] = __float2half_rn(sum == 0.f ? 0.f : acc / sum);
}

}  // namespace zt
