// attn_tc.cuh -- attention over whole prompts on the 5th-generation tensor cores
// (include/zt_q4.h: zt_q4_prompt_attention).
//
// Mathematics.  For a query row, over the keys that it sees, in tiles of 128:
//   S = q k^T,  p = 2^(scale log2(e) (S - m)),  O += p v,  l += sum p
// and the result is O / l.  m is a reference, at least the largest score so far
// minus 8 / (scale log2(e)): while scores stay below m by that margin (p <= 2^8),
// neither O nor l is rescaled.  p is rounded to fp16 for the second product;
// scores, m, l and O are fp32.
//
// Layout.  A CTA takes two tiles of 128 queries of one head (one where that leaves
// SMs idle) and walks the keys.  Both products are tcgen05.mma (M = 128, kind::f16):
// S [128 x 128] and O [128 x D] live in tensor memory, Q, K and V in shared memory
// in the 128-byte swizzle of their TMA loads (V is the N-major operand as it
// stands), and p goes back to tensor memory, over S, as the second product's A
// operand: a thread owns a row, so the softmax needs no exchange between threads.
//
// Roles.  Warps 0-3 and 4-7: softmax of tile 0 and of tile 1; warp 8: TMA; warp 9:
// mma.  While one tile's softmax runs, the other tile's products run.  One commit
// per S of a tile also covers that tile's previous O += p v (issued before it), so
// a softmax group that has S may rescale O.
//
// Masked places.  Keys behind a sequence's end (the next sequence's, or whatever
// follows) are masked in S; their V rows within the last 16-key step are zeroed in
// shared memory and later steps skipped, so what they hold does not matter.
#pragma once

#include "kv_common.cuh"

namespace zt {

constexpr int kAttnRows = 128, kAttnKeys = 128;
constexpr int kAttnThreads = 384;
constexpr float kAttnSlack = 8.f;      // log2 of the largest weight before a rescale

struct PromptArgs {
    __half *out;
    long long ld_out;
    const int32_t *cu_q, *cu_k;        // [n_seqs + 1]
    int n_seqs, total_q, total_k, q_heads, group, causal;
    int tiles;                         // query tiles per CTA: 1 or 2
    float scale_log2;
    unsigned int *err;
};

template <int D>
struct PromptCfg {
    static constexpr int kAtoms = (D + 63) / 64;                       // 64-column halves of a tile
    static constexpr int kAtom = 128 * 128;                            // bytes
    static constexpr int kTile = kAtoms * kAtom;                       // 16 or 32 KB
    static constexpr int kStages = kAtoms == 2 ? 5 : 8;
    static constexpr int kBars = 1 + 2 * kStages + 6;
    static constexpr int kSmem = 2 * kTile + kStages * kTile + kBars * 8 + 16 + 1024;
    // kind::f16, D f32, A and B f16; the second product's B (V) is N-major (bit 16)
    static constexpr uint32_t kIdescS = (1u << 4) | ((uint32_t)(kAttnKeys >> 3) << 17) | (8u << 24);
    static constexpr uint32_t kIdescO = (1u << 4) | (1u << 16) | ((uint32_t)(D >> 3) << 17) | (8u << 24);
};

// N-major operand in the 128-byte swizzle: 64-column halves one atom apart (leading offset), 8-key groups
// 1024 bytes apart (stride offset).
__device__ __forceinline__ uint64_t attn_desc_v(uint32_t saddr, uint32_t lead)
{
    return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)(lead >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
           ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

__device__ __forceinline__ void attn_tma_3d(uint32_t dst, const CUtensorMap *map, int x, int y, int z, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
            dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar) : "memory");
}

__device__ __forceinline__ void attn_commit(uint32_t bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

// 32 columns of this warp's lanes; attn_ld_wait names the registers before their first use
__device__ __forceinline__ void attn_ld32(uint32_t taddr, uint32_t (&r)[32])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}
__device__ __forceinline__ void attn_ld_wait(uint32_t (&r)[32])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                   "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]),
                   "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]),
                   "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
                 :
                 : "memory");
}
__device__ __forceinline__ void attn_st32(uint32_t taddr, const uint32_t (&r)[32])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}
__device__ __forceinline__ void attn_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ float attn_exp2(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// What a CTA works on: one head's query rows row0 .. of a sequence.
struct PromptItem {
    int q0, k0, nq, nk, row0, head;
    bool any;
};

// Item `id` of the list (sequence, head, block of queries from the last to the first): the heavy blocks of
// a causal prompt start first, and CTAs that run together share a head's keys in L2.  Whole warp.
__device__ __forceinline__ PromptItem prompt_item(const PromptArgs &a, int id, int rows)
{
    PromptItem it{};
    const int lane = threadIdx.x & 31;
    int before = 0;
    for (int b0 = 0; b0 < a.n_seqs; b0 += 32) {
        const int b = b0 + lane;
        int q0 = 0, nq = 0;
        if (b < a.n_seqs) {
            // offsets out of order or range: the sequence is left out
            const int q1 = a.cu_q[b + 1];
            q0 = a.cu_q[b];
            nq = q0 >= 0 && q1 >= q0 && q1 <= a.total_q ? q1 - q0 : 0;
        }
        int mine = (nq + rows - 1) / rows * a.q_heads, upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += u;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, id < before + upto);
        if (hit) {
            const int src = __ffs(hit) - 1;
            const int rel = id - before - __shfl_sync(0xffffffffu, upto - mine, src);
            it.q0 = __shfl_sync(0xffffffffu, q0, src);
            it.nq = __shfl_sync(0xffffffffu, nq, src);
            const int k1 = a.cu_k[b0 + src + 1];
            it.k0 = a.cu_k[b0 + src];
            it.nk = it.k0 >= 0 && k1 >= it.k0 && k1 <= a.total_k ? k1 - it.k0 : 0;
            const int blocks = (it.nq + rows - 1) / rows;
            it.head = rel / blocks;
            it.row0 = (blocks - 1 - (rel - it.head * blocks)) * rows;
            it.any = rel >= 0 && it.head < a.q_heads;       // false only where overlapping sequences overflow the count
            return it;
        }
        before += __shfl_sync(0xffffffffu, upto, 31);
    }
    return it;
}

template <int D>
__global__ void __launch_bounds__(kAttnThreads, 1) prompt_attn_kernel(const __grid_constant__ CUtensorMap map_q,
                                                                      const __grid_constant__ CUtensorMap map_k,
                                                                      const __grid_constant__ CUtensorMap map_v,
                                                                      const __grid_constant__ PromptArgs a)
{
    using C = PromptCfg<D>;
    constexpr int S = C::kStages;
    extern __shared__ __align__(128) unsigned char attn_smem[];
    const uint32_t raw = kv_smem(attn_smem);
    const uint32_t q_s = (raw + 1023u) & ~1023u, ring = q_s + 2 * C::kTile;
    const uint32_t bars = ring + S * C::kTile, slot = bars + C::kBars * 8;
    const uint32_t q_full = bars;
    auto full = [&](int s) { return bars + 8u * (1 + s); };
    auto empty = [&](int s) { return bars + 8u * (1 + S + s); };
    auto s_full = [&](int t) { return bars + 8u * (1 + 2 * S + t); };
    auto p_full = [&](int t) { return bars + 8u * (3 + 2 * S + t); };
    auto o_full = [&](int t) { return bars + 8u * (5 + 2 * S + t); };

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kBars; ++i) {
            const bool p = i >= 3 + 2 * S && i < 5 + 2 * S;
            asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bars + 8 * i), "r"(p ? 128 : 1) : "memory");
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 8) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(slot) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    kv_pdl_launch();
    kv_pdl_wait();
    const int rows = a.tiles * kAttnRows;
    const PromptItem it = prompt_item(a, (int)blockIdx.x, rows);
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    uint32_t tmem;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(tmem) : "r"(slot) : "memory");

    // key tiles of each query tile: those that its last row sees
    auto seen_by = [&](int row) { return a.causal ? min(max(row + 1 + it.nk - it.nq, 0), it.nk) : it.nk; };
    int n_t[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const int first = it.row0 + t * kAttnRows, last = min(first + kAttnRows, it.nq) - 1;
        n_t[t] = it.any && t < a.tiles && last >= first ? (seen_by(last) + kAttnKeys - 1) / kAttnKeys : 0;
    }
    const int n = max(n_t[0], n_t[1]);
    const int kv_head = it.head / a.group;

    if (warp < 8) {
        // ------------------------------------------------------------ softmax
        const int t = warp >> 2, row = it.row0 + t * kAttnRows + (threadIdx.x & 127);
        const bool valid = it.any && t < a.tiles && row < it.nq;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t s_tm = tmem + lanes + 128u * t, o_tm = tmem + lanes + 256u + 128u * t;
        const int seen = seen_by(row);
        const int all_seen = seen_by(it.row0 + t * kAttnRows);      // by every row of the tile
        const float sl = a.scale_log2, slack = kAttnSlack / sl;
        float ref = -INFINITY, l = 0.f;
        bool ok = true;
        for (int j = 0; j < n_t[t] && ok; ++j) {
            ok = __all_sync(0xffffffffu, tc_wait(s_full(t), (uint32_t)j & 1u, false));
            if (!ok) {
                if (lane == 0) kv_error(a.err, kErrKvWait);
                break;
            }
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            uint32_t r[4][32];
#pragma unroll
            for (int c = 0; c < 4; ++c) attn_ld32(s_tm + 32 * c, r[c]);
#pragma unroll
            for (int c = 0; c < 4; ++c) attn_ld_wait(r[c]);
            if (j * kAttnKeys + kAttnKeys > all_seen) {
                const int left = seen - j * kAttnKeys;
#pragma unroll
                for (int c = 0; c < 4; ++c)
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (32 * c + i >= left) r[c][i] = 0xFF800000u;
            }
            float mx = -INFINITY;
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
                for (int i = 0; i < 32; ++i) mx = fmaxf(mx, __uint_as_float(r[c][i]));
            if (__any_sync(0xffffffffu, mx > ref + slack)) {
                const float to = fmaxf(ref, mx);
                const float f = ref == to ? 1.f : attn_exp2((ref - to) * sl);
                ref = to;
                l *= f;
                if (j > 0) {
#pragma unroll 1
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t o[32];
                        attn_ld32(o_tm + 32 * c, o);
                        attn_ld_wait(o);
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                        attn_st32(o_tm + 32 * c, o);
                    }
                }
            }
            const float base = ref == -INFINITY ? 0.f : ref * sl;
            float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int c = 0; c < 4; c += 2) {
                uint32_t p[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    const uint32_t *src = i < 16 ? r[c] : r[c + 1];
                    const int k = 2 * (i & 15);
                    const float p0 = attn_exp2(fmaf(__uint_as_float(src[k]), sl, -base));
                    const float p1 = attn_exp2(fmaf(__uint_as_float(src[k + 1]), sl, -base));
                    sum[2 * (i & 1)] += p0;
                    sum[2 * (i & 1) + 1] += p1;
                    p[i] = h2_bits(__floats2half2_rn(p0, p1));
                }
                attn_st32(s_tm + 16 * c, p);
            }
            l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
            attn_st_wait();
            asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
            asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(p_full(t)) : "memory");
        }
        if (n_t[t] > 0 && ok) {
            ok = __all_sync(0xffffffffu, tc_wait(o_full(t), 0u, false));
            if (!ok && lane == 0) kv_error(a.err, kErrKvWait);
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        }
        if (ok) {
            const float inv = l == 0.f ? 0.f : 1.f / l;
            __half *dst = a.out + (long long)(it.q0 + row) * a.ld_out + it.head * D;
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
                uint32_t o[32];
                if (n_t[t] > 0) {
                    attn_ld32(o_tm + 32 * c, o);
                    attn_ld_wait(o);
                }
                if (valid) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t v[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            v[e] = l == 0.f ? 0u
                                            : h2_bits(__floats2half2_rn(__uint_as_float(o[8 * i + 2 * e]) * inv,
                                                                        __uint_as_float(o[8 * i + 2 * e + 1]) * inv));
                        *reinterpret_cast<uint4 *>(dst + 32 * c + 8 * i) = make_uint4(v[0], v[1], v[2], v[3]);
                    }
                }
            }
        }
        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    } else if (warp == 8) {
        // ---------------------------------------------------------------- TMA
        if (lane == 0 && n > 0) {
            auto tile = [&](uint32_t dst, const CUtensorMap *map, int head, int token, uint32_t bar) {
#pragma unroll
                for (int c = 0; c < C::kAtoms; ++c) attn_tma_3d(dst + c * C::kAtom, map, 64 * c, head, token, bar);
            };
            asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(q_full), "r"(a.tiles * C::kTile)
                         : "memory");
            for (int t = 0; t < a.tiles; ++t) tile(q_s + t * C::kTile, &map_q, it.head, it.q0 + it.row0 + t * kAttnRows, q_full);
            int i = 0;
            for (; i < 2 * n; ++i) {
                const int s = i % S;
                if (i >= S && !tc_wait(empty(s), (uint32_t)(i / S - 1) & 1u, false)) {
                    kv_error(a.err, kErrKvWait);
                    break;
                }
                asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(full(s)), "r"(C::kTile) : "memory");
                tile(ring + s * C::kTile, (i & 1) ? &map_v : &map_k, kv_head, it.k0 + (i >> 1) * kAttnKeys, full(s));
            }
            // every load has landed before the CTA ends (all of them have been used, unless a wait ran out)
            tc_wait(q_full, 0u, false);
            for (int k = max(0, i - S); k < i; ++k)
                if (!tc_wait(full(k % S), (uint32_t)(k / S) & 1u, false)) break;
        }
        __syncwarp();
    } else if (warp == 9 && n > 0) {
        // ---------------------------------------------------------------- mma
        bool ok = true;
        auto wait = [&](uint32_t bar, int par) {
            if (ok && !__all_sync(0xffffffffu, tc_wait(bar, (uint32_t)par & 1u, false))) {
                if (lane == 0) kv_error(a.err, kErrKvWait);
                ok = false;
            }
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        };
        auto scores = [&](int t, int j) {
            const int i = 2 * j;
            const uint64_t dq = tc_desc_sw128(q_s + t * C::kTile), dk = tc_desc_sw128(ring + (i % S) * C::kTile);
            if (lane == 0) {
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const uint64_t at = (uint64_t)((k / 4) * (C::kAtom >> 4) + (k % 4) * 2);
                    asm volatile(
                        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem + 128u * t),
                        "l"(dq + at), "l"(dk + at), "r"(C::kIdescS), "r"(k ? 1u : 0u));
                }
                attn_commit(s_full(t));
            }
        };
        auto values = [&](int t, int j, int steps) {
            const int i = 2 * j + 1;
            const uint64_t dv = attn_desc_v(ring + (i % S) * C::kTile, C::kAtom);
            if (lane == 0)
#pragma unroll
                for (int k = 0; k < kAttnKeys / 16; ++k)
                    if (k < steps)
                        asm volatile(
                            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                            "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(tmem + 256u + 128u * t),
                            "r"(tmem + 128u * t + 8u * k), "l"(dv + (uint64_t)(k * (2048 >> 4))), "r"(C::kIdescO),
                            "r"((j | k) ? 1u : 0u));
        };
        wait(q_full, 0);
        wait(full(0), 0);
        if (ok) {
#pragma unroll
            for (int t = 0; t < 2; ++t)
                if (n_t[t] > 0) scores(t, 0);
            if (lane == 0 && S < 2 * n) attn_commit(empty(0));
        }
        for (int j = 0; j < n && ok; ++j) {
            const int iv = 2 * j + 1, ik = 2 * j + 2;
            wait(full(iv % S), iv / S);
            const int keys = min(kAttnKeys, it.nk - j * kAttnKeys), steps = (keys + 15) / 16;
            if (keys < 16 * steps && ok) {
                // rows behind the end within the last step: zero, whatever follows the sequence
                for (int c = lane; c < (16 * steps - keys) * C::kAtoms * 8; c += 32) {
                    const int row = keys + c / (C::kAtoms * 8), in = c % (C::kAtoms * 8);
                    asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(ring + (iv % S) * C::kTile +
                                                                                 (in / 8) * C::kAtom + row * 128 + (in % 8) * 16),
                                 "r"(0u) : "memory");
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
            }
            if (ik < 2 * n) wait(full(ik % S), ik / S);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                if (j >= n_t[t]) continue;
                wait(p_full(t), j);
                if (!ok) break;
                values(t, j, steps);
                if (j + 1 < n_t[t]) scores(t, j + 1);
                else if (lane == 0) attn_commit(o_full(t));
            }
            if (ok && lane == 0) {
                // only for stages that are loaded again: no arrival is left behind when the CTA ends
                if (iv + S < 2 * n) attn_commit(empty(iv % S));
                if (ik + S < 2 * n) attn_commit(empty(ik % S));
            }
        }
        if (!ok && lane == 0) {
            // what was issued ends before tensor memory is freed
            attn_commit(o_full(0));
            tc_wait(o_full(0), 0u, false);
        }
        __syncwarp();
    }
    __syncthreads();
    if (warp == 8) {
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    }
}

}  // namespace zt
