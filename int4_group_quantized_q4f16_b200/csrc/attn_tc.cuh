// attn_tc.cuh -- attention over whole prompts on the 5th-generation tensor cores
// (include/zt_q4.h: zt_q4_prompt_attention).
//
// Mathematics.  For a query row, over the keys that it sees, in tiles of 128:
//   S = q k^T,  p = 2^(scale log2(e) (S - m) + 7),  O += p v,  l += sum p
// and the result is O / l.  m is a reference, at least the largest score so far
// minus 8 / (scale log2(e)): while no score passes m by more (p <= 2^15), neither O
// nor l is rescaled.  p is rounded to fp16 for the second product, and the 7 keeps it
// in the upper range: of many small weights beside a large one those down to 2^-21 of
// it are rounded like normal numbers, and 2^-31 is not zero yet (2^-14 and 2^-24
// without).  Scores, m, l and O are fp32.  Where scale log2(e) m is so large that its
// rounding would count (2^18), m is taken off the scores first, in the rescale's branch,
// which such rows take at every tile (in a branch of its own before the exponentials: 137
// queries on 2724 keys 27.1 us, packed prompts 75.5, as here 26.9 and 74.4; without, for
// smaller scores only, 26.7 and 75.2).
//
// Layout.  A CTA takes two tiles of 128 queries of one head (one where that leaves
// SMs idle) and walks the keys.  Both products are tcgen05.mma (M = 128, kind::f16):
// S [128 x 128] and O [128 x D] live in tensor memory, Q, K and V in shared memory
// in the 128-byte swizzle of their TMA loads (V is the N-major operand as it
// stands), and p goes back to tensor memory, over S, as the second product's A
// operand: a thread owns a row, so the softmax needs no exchange between threads.
//
// Roles.  Warps 0-3 and 4-7: softmax of tile 0 and of tile 1; warp 8: TMA; warps
// 9 and 10: the products of tile 0 and of tile 1; warp 11: the schedule.  While one tile's softmax runs, the other tile's
// products run; p is handed over in halves, so that O += p v starts on the first 64
// keys.  One commit per S of a tile also covers that tile's previous O += p v (issued
// before it), so a softmax group that has S may rescale O.
//
// What bounds it.  A pair of tiles takes 1024 tensor-core cycles per 128 keys (D = 128;
// 1536 with the shared-memory reads of Q, K and V at 128 bytes a cycle) and 2048 cycles
// of exponentials at 16 a cycle.  Measured at 8192 tokens, 32 heads of 128: 3700 cycles,
// of which a softmax group waits 1050 for its products, and takes 550 for the maxima and
// 1370 for the exponentials.  The groups take turns at the exponentials (without: 548 us,
// with: 504).  Computing 1/8 .. 3/8 of them by polynomial on the fma units made it slower
// (565 .. 647 us): the chain of one tile, not the exponentials' rate, sets the pace.
// 8192 tokens causal: 484-527 us, 1040-1140 TFLOP/s, in bursts; 540-590 us, 930-1020 TFLOP/s,
// call after call, where the power limit holds the clock near 1.5 GHz.  784 before the groups
// took turns, the products had a warp per tile and items were taken in order of their weight.
//
// Schedule.  The grid has a CTA per work item (sequence, head, block of queries), the
// heavy blocks first; a CTA that runs keeps taking items whose CTAs have not been
// launched (clusterlaunchcontrol), so that loads and the first products of an item
// overlap the end of the one before, and barriers and tensor memory are set up once.
//
// Few query tiles on long keys (a chunk behind a prefix): the CTAs of a cluster share an item's keys, leave O, the
// references and the sums in shared memory, and each joins a share of the columns, reading the others' through the
// cluster, in the order of the keys.  No workspace, one launch.
//
// Masked places.  Keys behind a sequence's end (the next sequence's, or whatever
// follows) are masked in S; their V rows within the last 16-key step are zeroed in
// shared memory and later steps skipped, so what they hold does not matter.
#pragma once

#include "kv_common.cuh"

namespace zt {

constexpr int kAttnRows = 128, kAttnKeys = 128;
constexpr int kAttnThreads = 384;
constexpr float kAttnSlack = 8.f;      // scores above the reference before a rescale, in powers of two
constexpr float kAttnLift = 7.f;       // log2 of a weight at the reference
constexpr float kAttnFar = 0x1p18f;    // exponents whose reference is taken off the scores before the product with the scale

struct PromptArgs {
    __half *out;
    long long ld_out;
    const int32_t *cu_q, *cu_k;        // [n_seqs + 1]
    int n_seqs, total_q, total_k, q_heads, group, causal;
    int tiles;                         // query tiles per CTA: 1 or 2
    int splits;                        // CTAs (a cluster) that share an item's keys; more than 1 with one query tile only
    float scale_log2;
    unsigned int *err;
};

template <int D>
struct PromptCfg {
    static constexpr int kAtoms = (D + 63) / 64;                       // 64-column halves of a tile
    static constexpr int kAtom = 128 * 128;                            // bytes
    static constexpr int kTile = kAtoms * kAtom;                       // 16 or 32 KB
    static constexpr int kStages = kAtoms == 2 ? 5 : 8;
    static constexpr int kBars = 2 * kStages + 2 + 2 + 4 + 2 + 2 + 4 + 1 + 2 + 1 + 2;
    static constexpr int kItems = (kBars * 8 + 15) / 16 * 16;                           // two items of 32 bytes, the scheduler's answer
    static constexpr int kSmem = 2 * kTile + kStages * kTile + kItems + 64 + 16 + 16 + 1024;
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

// D (+)= A B: A from shared memory, or from tensor memory; B from shared memory
__device__ __forceinline__ void attn_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc),
        "r"((uint32_t)add));
}
__device__ __forceinline__ void attn_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(idesc),
        "r"((uint32_t)add));
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

__device__ __forceinline__ bool attn_try(uint32_t bar, uint32_t par)
{
    uint32_t done;
    asm volatile("{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(done) : "r"(bar), "r"(par) : "memory");
    return done != 0u;
}

// One lane of a converged warp, in a form that lets the compiler keep operands of the tensor-core instructions in
// uniform registers (a compare with the lane number costs ~200 cycles per instruction: 2.5x the kernel's time).
__device__ __forceinline__ bool attn_elect()
{
    uint32_t e;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
    return e != 0u;
}

__device__ __forceinline__ float attn_max3(float a, float b, float c)
{
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// What a CTA works on: one head's query rows row0 .. of a sequence.
struct PromptItem {
    int q0, k0, nq, nk, row0, head;
    bool any;
};

// Item `id` of the list.  Up to 32 sequences: by block of queries from the longest sequence's last one down, then
// sequence, then head: the heavy blocks of causal prompts start first and light ones fill in at the end.  (By sequence,
// head and block some CTAs had 25 % more tiles than the average at 8192 tokens and 32 heads: 654 us, not 504.)  More
// sequences, which are short ones as a rule: by sequence, then head, then block from the last down.  Whole warp.
__device__ __forceinline__ PromptItem prompt_item(const PromptArgs &a, int id, int rows)
{
    PromptItem it{};
    const int lane = threadIdx.x & 31;
    auto length = [&](int b, int &q0) {
        if (b >= a.n_seqs) return 0;
        // offsets out of order or range: the sequence is left out
        const int q1 = a.cu_q[b + 1];
        q0 = a.cu_q[b];
        return q0 >= 0 && q1 >= q0 && q1 <= a.total_q ? q1 - q0 : 0;
    };
    auto scan = [&](int v) {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += u;
        }
        return v;
    };
    int src = -1, first = 0, q0 = 0, nq = 0, rel = id, blocks = 0;
    if (a.n_seqs <= 32) {
        nq = length(lane, q0);
        blocks = (nq + rows - 1) / rows;
        // the highest level (block index) with at most id items above it
        int lo = 0, hi = __reduce_max_sync(0xffffffffu, blocks);
        if (hi == 0) return it;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (__reduce_add_sync(0xffffffffu, max(blocks - mid, 0)) * a.q_heads > id) lo = mid;
            else hi = mid;
        }
        rel = id - __reduce_add_sync(0xffffffffu, max(blocks - lo - 1, 0)) * a.q_heads;
        const int mine = blocks > lo ? a.q_heads : 0, upto = scan(mine);
        const unsigned hit = __ballot_sync(0xffffffffu, rel < upto);
        if (!hit) return it;
        src = __ffs(hit) - 1;
        it.head = rel - __shfl_sync(0xffffffffu, upto - mine, src);
        it.row0 = lo * rows;
    } else {
        for (int before = 0; first < a.n_seqs; first += 32) {
            nq = length(first + lane, q0);
            blocks = (nq + rows - 1) / rows;
            const int mine = blocks * a.q_heads, upto = scan(mine);
            const unsigned hit = __ballot_sync(0xffffffffu, id < before + upto);
            if (hit) {
                src = __ffs(hit) - 1;
                rel = id - before - __shfl_sync(0xffffffffu, upto - mine, src);
                const int n = __shfl_sync(0xffffffffu, blocks, src);
                it.head = rel / n;
                it.row0 = (n - 1 - (rel - it.head * n)) * rows;
                break;
            }
            before += __shfl_sync(0xffffffffu, upto, 31);
        }
        if (src < 0) return it;
    }
    it.q0 = __shfl_sync(0xffffffffu, q0, src);
    it.nq = __shfl_sync(0xffffffffu, nq, src);
    const int k1 = a.cu_k[first + src + 1];
    it.k0 = a.cu_k[first + src];
    it.nk = it.k0 >= 0 && k1 >= it.k0 && k1 <= a.total_k ? k1 - it.k0 : 0;
    // false only where overlapping sequences overflow the count
    it.any = it.head >= 0 && it.head < a.q_heads && it.row0 >= 0 && it.row0 < it.nq;
    return it;
}

// The cluster's parts of an item, in shared memory: O as [D][128 rows], the rows' references and sums behind it.  A cluster
// barrier separates writing, joining and the end; every thread comes to it, whatever became of its role.
__device__ __forceinline__ void attn_cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ float attn_peer(uint32_t saddr, int rank)
{
    float v;
    asm volatile("{\n\t.reg .b32 at;\n\tmapa.shared::cluster.u32 at, %1, %2;\n\tld.shared::cluster.f32 %0, [at];\n\t}"
                 : "=f"(v) : "r"(saddr), "r"(rank));
    return v;
}

constexpr int kAttnSplits = 8;         // CTAs of a cluster that share an item's keys, at most

// One row's result from N parts, in their order: CTA `rank` of the cluster writes its share of the columns, with 32 reads
// under way at a time.
template <int D, int N>
__device__ __forceinline__ void attn_join(uint32_t part, int row, int rank, float sl, __half *dst)
{
    constexpr int kShare = D / N, kStep = 32 / N;
    static_assert(kShare % kStep == 0 && kStep % 4 == 0, "whole steps, of 8 bytes of the result");
    const uint32_t refs = part + D * kAttnRows * 4 + row * 4, sums = refs + kAttnRows * 4;
    float f[N], sum[N], top = -INFINITY, l = 0.f;
#pragma unroll
    for (int p = 0; p < N; ++p) {
        f[p] = attn_peer(refs, p);
        sum[p] = attn_peer(sums, p);
    }
#pragma unroll
    for (int p = 0; p < N; ++p) top = fmaxf(top, f[p]);
#pragma unroll
    for (int p = 0; p < N; ++p) {
        f[p] = f[p] == top ? 1.f : attn_exp2((f[p] - top) * sl);
        if (sum[p] != 0.f) l += f[p] * sum[p];
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll 1
    for (int d = rank * kShare; d < (rank + 1) * kShare; d += kStep) {
        float o[kStep] = {}, v[N][kStep];
#pragma unroll
        for (int p = 0; p < N; ++p)
#pragma unroll
            for (int e = 0; e < kStep; ++e) v[p][e] = attn_peer(part + ((d + e) * kAttnRows + row) * 4, p);
#pragma unroll
        for (int p = 0; p < N; ++p)
#pragma unroll
            for (int e = 0; e < kStep; ++e)
                if (sum[p] != 0.f) o[e] = fmaf(f[p], v[p][e], o[e]);       // a part without keys has no O
#pragma unroll
        for (int e = 0; e < kStep; e += 4)
            *reinterpret_cast<uint2 *>(dst + d + e) = make_uint2(h2_bits(__floats2half2_rn(o[e] * inv, o[e + 1] * inv)),
                                                                 h2_bits(__floats2half2_rn(o[e + 2] * inv, o[e + 3] * inv)));
    }
}

// SPLIT: an item's keys are shared between the CTAs of a cluster, a CTA has one item.
template <int D, bool SPLIT>
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
    const uint32_t bars = ring + S * C::kTile, items = bars + C::kItems, answer = items + 64, slot = answer + 16;
    auto full = [&](int s) { return bars + 8u * s; };                       // K or V tile loaded
    auto empty = [&](int s) { return bars + 8u * (S + s); };                // and used
    const uint32_t misc = bars + 16u * S;
    const uint32_t q_full = misc, q_empty = misc + 8;                       // the item's Q tiles loaded, and used
    auto s_full = [&](int t) { return misc + 16u + 8u * t; };               // S of tile t there
    auto p_full = [&](int t, int h) { return misc + 32u + 8u * (2 * t + h); };   // half h of its weights there
    auto o_full = [&](int t) { return misc + 64u + 8u * t; };               // O of tile t complete
    auto o_empty = [&](int t) { return misc + 80u + 8u * t; };              // and read
    auto item_full = [&](int i) { return misc + 96u + 8u * i; };            // item slot i written
    auto item_empty = [&](int i) { return misc + 112u + 8u * i; };          // and read by its eleven readers
    const uint32_t answered = misc + 128u, wanted = misc + 152u;            // the scheduler's answer; an item's loads issued
    auto go = [&](int t) { return misc + 136u + 8u * t; };                  // tile t's turn at the exponentials
    auto drain = [&](int t) { return misc + 160u + 8u * t; };               // tile t's products ended, after a wait ran out

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        auto init = [&](uint32_t bar, int n) {
            asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(n) : "memory");
        };
        for (int i = 0; i < S; ++i) {
            init(full(i), 1);
            init(empty(i), 2);
        }
        init(q_full, 1);
        init(q_empty, 2);
        for (int t = 0; t < 2; ++t) {
            init(s_full(t), 1);
            init(p_full(t, 0), 128);
            init(p_full(t, 1), 128);
            init(o_full(t), 1);
            init(o_empty(t), 128);
            init(go(t), 128);
            init(drain(t), 1);
            init(item_full(t), 1);
            init(item_empty(t), 11);
        }
        init(answered, 1);
        init(wanted, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 8) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(slot) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    kv_pdl_launch();
    kv_pdl_wait();
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    uint32_t tmem;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(tmem) : "r"(slot) : "memory");

    // Every wait is bounded; after one ran out its role gives up, and so do, one after the other, those that wait for it.
    bool ok = true;
    auto wait = [&](uint32_t bar, uint32_t phase) {          // whole warp
        // one try without a branch per lane; most waits end there
        if (__all_sync(0xffffffffu, attn_try(bar, phase & 1u))) return;
        if (ok && !__all_sync(0xffffffffu, tc_wait(bar, phase & 1u, false))) {
            if (lane == 0) kv_error(a.err, kErrKvWait);
            ok = false;
        }
    };
    auto arrive = [&](uint32_t bar) { asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory"); };

    // item number k of this CTA, from the schedule; false: there is none
    int q0, k0, nq, nk, row0, head, n_t[2], n;
    [[maybe_unused]] int first_tile = 0;         // of this CTA's part of the keys
    const int share = SPLIT ? (int)(blockIdx.x % (unsigned)a.splits) : 0;
    auto j0 = [&]() { return SPLIT ? first_tile : 0; };
    auto take = [&](int k) {
        wait(item_full(k & 1), (uint32_t)k >> 1);
        const uint32_t at = items + 32u * (k & 1);
        int any = 0;
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(q0), "=r"(k0), "=r"(nq), "=r"(nk) : "r"(at) : "memory");
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(row0), "=r"(head), "=r"(any), "=r"(n) : "r"(at + 16u)
                     : "memory");
        __syncwarp();
        if (lane == 0) arrive(item_empty(k & 1));
        // the same in all lanes; a reduction's result is known to be, and stays in uniform registers
        auto uniform = [](int &v) { v = __reduce_max_sync(0xffffffffu, v); };
        uniform(q0), uniform(k0), uniform(nq), uniform(nk), uniform(row0), uniform(head), uniform(any);
        // key tiles of each query tile: those that its last row sees
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const int first = row0 + t * kAttnRows, last = min(first + kAttnRows, nq) - 1;
            const int seen = a.causal ? min(max(last + 1 + nk - nq, 0), nk) : nk;
            n_t[t] = t < a.tiles && last >= first ? (seen + kAttnKeys - 1) / kAttnKeys : 0;
        }
        if constexpr (SPLIT) {                     // this CTA's part of the keys
            const int each = (n_t[0] + a.splits - 1) / a.splits;
            first_tile = min(share * each, n_t[0]);
            n_t[0] = min(each, n_t[0] - first_tile);
        }
        n = max(n_t[0], n_t[1]);
        return ok && any != 0;
    };

    __half *joined = nullptr;                   // of this thread's row, where the keys are split
    if (warp < 8) {
        // ------------------------------------------------------------ softmax
        asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
        const int t = warp >> 2;
        auto my_n = [&]() { return t ? n_t[1] : n_t[0]; };
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t s_tm = tmem + lanes + 128u * t, o_tm = tmem + lanes + 256u + 128u * t;
        const float sl = a.scale_log2, slack = kAttnSlack / sl;
        uint32_t turn = 0, done = 0, pairs = 0;     // S tiles, O tiles and turns at the exponentials taken so far
        for (int k = 0; take(k); ++k) {
            const int mine = my_n();
            const int row = row0 + t * kAttnRows + (threadIdx.x & 127);
            auto seen_by = [&](int r) { return a.causal ? min(max(r + 1 + nk - nq, 0), nk) : nk; };
            const int seen = seen_by(row), all_seen = seen_by(row0 + t * kAttnRows);      // by this row, by every row
            const int both = min(n_t[0], n_t[1]);
            // base: scale log2(e) ref - 7, 0 without one; limit: the largest score without a rescale
            float ref = -INFINITY, l = 0.f, base = 0.f, limit = -INFINITY;
            for (int j = 0; j < mine && ok; ++j, ++turn) {
                wait(s_full(t), turn);
                if (!ok) break;
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                uint32_t r[4][32];
#pragma unroll
                for (int c = 0; c < 4; ++c) attn_ld32(s_tm + 32 * c, r[c]);
#pragma unroll
                for (int c = 0; c < 4; ++c) attn_ld_wait(r[c]);
                if ((j + j0()) * kAttnKeys + kAttnKeys > all_seen) {
                    const int left = seen - (j + j0()) * kAttnKeys;
#pragma unroll
                    for (int c = 0; c < 4; ++c)
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (32 * c + i >= left) r[c][i] = 0xFF800000u;
                }
                float m4[4];                             // four chains: one would be 64 dependent steps
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    m4[c] = __uint_as_float(r[c][0]);
#pragma unroll
                    for (int i = 1; i < 31; i += 2)
                        m4[c] = attn_max3(m4[c], __uint_as_float(r[c][i]), __uint_as_float(r[c][i + 1]));
                    m4[c] = fmaxf(m4[c], __uint_as_float(r[c][31]));
                }
                const float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
                if (__any_sync(0xffffffffu, mx > limit)) {
                    const float to = fmaxf(ref, mx);
                    const float f = ref == to ? 1.f : attn_exp2((ref - to) * sl);
                    ref = to;
                    l *= f;
                    base = ref == -INFINITY ? 0.f : ref * sl - kAttnLift;
                    limit = __fadd_rd(ref, slack);
                    if (__any_sync(0xffffffffu, fabsf(base) > kAttnFar)) {
                        // too large for some row: the references are taken off the scores, here at every tile
#pragma unroll
                        for (int c = 0; c < 4; ++c)
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                r[c][i] = __float_as_uint(__uint_as_float(r[c][i]) - (ref == -INFINITY ? 0.f : ref));
                        base = -kAttnLift;
                        limit = -INFINITY;
                    }
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
                // The two groups take turns at the exponentials: in step, both would wait for them and then both for
                // the products.
                const bool paired = j < both;
                if (paired) {
                    if (t == 1 || pairs > 0) wait(go(t), pairs - (t == 0));
                    ++pairs;
                    if (!ok) break;
                }
                const uint64_t sl2 = f2_pack(sl, sl), base2 = f2_pack(-base, -base);
                uint64_t sum[2] = {0ull, 0ull};
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t p[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        const uint32_t *src = i < 16 ? r[2 * h] : r[2 * h + 1];
                        const int e = 2 * (i & 15);
                        const uint64_t x = f2_fma(f2_pack(__uint_as_float(src[e]), __uint_as_float(src[e + 1])), sl2, base2);
                        float2 v = f2_split(x);
                        v.x = attn_exp2(v.x);
                        v.y = attn_exp2(v.y);
                        sum[i & 1] = f2_add(sum[i & 1], f2_pack(v.x, v.y));
                        p[i] = h2_bits(__floats2half2_rn(v.x, v.y));
                    }
                    attn_st32(s_tm + 32 * h, p);
                    if (h == 1 && paired) arrive(go(1 - t));
                    attn_st_wait();
                    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
                    arrive(p_full(t, h));
                }
                const float2 s0 = f2_split(sum[0]), s1 = f2_split(sum[1]);
                l += (s0.x + s0.y) + (s1.x + s1.y);
            }
            if (mine > 0) {
                wait(o_full(t), done++);
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            }
            if (!ok) break;
            const float inv = l == 0.f ? 0.f : 1.f / l;
            __half *dst = a.out + (long long)(q0 + row) * a.ld_out + head * D;
            const bool valid = t < a.tiles && row < nq;
            if constexpr (SPLIT) {
                if (t == 1) continue;               // a second query tile: there is none
                // the part of the result goes to the ring, whose tiles have all been used: by warp 9, which O's completion
                // covers; warp 10 only waits for them
                const uint32_t at = ring + (threadIdx.x & 127) * 4, refs = at + D * kAttnRows * 4;
                if (mine > 0) {
#pragma unroll 1
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t o[32];
                        attn_ld32(o_tm + 32 * c, o);
                        attn_ld_wait(o);
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            asm volatile("st.shared.u32 [%0], %1;" ::"r"(at + (32 * c + i) * kAttnRows * 4), "r"(o[i]) : "memory");
                    }
                    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
                    arrive(o_empty(t));
                }
                asm volatile("st.shared.f32 [%0], %1;" ::"r"(refs), "f"(ref) : "memory");
                asm volatile("st.shared.f32 [%0], %1;" ::"r"(refs + kAttnRows * 4), "f"(l) : "memory");
                if (valid) joined = dst;
            } else {
#pragma unroll 1
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t o[32];
                    if (mine > 0) {
                        attn_ld32(o_tm + 32 * c, o);
                        attn_ld_wait(o);
                    }
                    if (c == D / 32 - 1 && mine > 0) {
                        // all of O is in registers or on its way out: the next item's products may start
                        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
                        arrive(o_empty(t));
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
        }
        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    }
    if (warp == 8) {
        // ---------------------------------------------------------------- TMA
        int i = 0, qs = 0;                                        // tiles and items with queries loaded so far
        bool q_open = false;
        for (int k = 0; take(k); ++k) {
            if (n == 0) {
                if (lane == 0) arrive(wanted);
                continue;
            }
            const int kv_head = head / a.group;
            auto tile = [&](uint32_t dst, const CUtensorMap *map, int h, int token, uint32_t bar) {
#pragma unroll
                for (int c = 0; c < C::kAtoms; ++c) attn_tma_3d(dst + c * C::kAtom, map, 64 * c, h, token, bar);
            };
            auto expect = [&](uint32_t bar, int bytes) {
                asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
            };
            if (qs > 0) wait(q_empty, (uint32_t)(qs - 1));
            if (!ok) break;
            if (lane == 0) {
                expect(q_full, a.tiles * C::kTile);
                for (int t = 0; t < a.tiles; ++t) tile(q_s + t * C::kTile, &map_q, head, q0 + row0 + t * kAttnRows, q_full);
            }
            ++qs;
            q_open = true;
            for (int j = 0; j < 2 * n; ++j, ++i) {
                const int s = i % S;
                if (i >= S) wait(empty(s), (uint32_t)(i / S - 1));
                if (!ok) break;
                if (lane == 0) {
                    expect(full(s), C::kTile);
                    tile(ring + s * C::kTile, (j & 1) ? &map_v : &map_k, kv_head, k0 + ((j >> 1) + j0()) * kAttnKeys, full(s));
                }
            }
            if (!ok) break;
            if (lane == 0) arrive(wanted);
        }
        // every load has landed before the CTA ends (all of them have been used, unless a wait ran out)
        if (lane == 0) {
            if (q_open) tc_wait(q_full, (uint32_t)(qs - 1) & 1u, false);
            for (int j = max(0, i - S); j < i; ++j)
                if (!tc_wait(full(j % S), (uint32_t)(j / S) & 1u, false)) break;
        }
        __syncwarp();
    } else if (warp == 9 || warp == 10) {
        // ---------------------------------------------------------------- mma
        // One warp per query tile: what one of them spends between products is hidden by the other's.
        const int t = warp - 9;
        const uint32_t s_tm = tmem + 128u * t, o_tm = tmem + 256u + 128u * t, q_t = q_s + t * C::kTile;
        auto sync_wait = [&](uint32_t bar, uint32_t phase) {
            wait(bar, phase);
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        };
        auto scores = [&](int i) {                                // S with the keys of ring tile i
            const uint64_t dq = tc_desc_sw128(q_t), dk = tc_desc_sw128(ring + (i % S) * C::kTile);
            if (attn_elect()) {
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const uint64_t at = (uint64_t)((k / 4) * (C::kAtom >> 4) + (k % 4) * 2);
                    attn_mma_ss(s_tm, dq + at, dk + at, C::kIdescS, k > 0);
                }
                attn_commit(s_full(t));
            }
        };
        auto values = [&](int j, int i, int h, int steps) {       // O += half h of p v, `steps` 16-key steps
            const uint64_t dv = attn_desc_v(ring + (i % S) * C::kTile + h * 8192, C::kAtom);
            const uint32_t p = s_tm + 32u * h;
            if (attn_elect()) {
                if (steps >= 4) {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        attn_mma_ts(o_tm, p + 8u * k, dv + (uint64_t)(k * 128), C::kIdescO, j > 0 || h > 0 || k > 0);
                } else {
                    for (int k = 0; k < steps; ++k)
                        attn_mma_ts(o_tm, p + 8u * k, dv + (uint64_t)(k * 128), C::kIdescO, j > 0 || h > 0 || k > 0);
                }
            }
        };
        // this warp is done with what `bar` guards: when the products issued so far are, or at once.  Both warps say
        // so for every tile and item, after its load: neither can be a phase ahead of the other.
        auto release = [&](uint32_t bar, bool used) {
            if (attn_elect()) {
                if (used) attn_commit(bar);
                else arrive(bar);
            }
        };
        int base = 0, qs = 0;                                     // ring tiles and Q tiles of the items before
        uint32_t turn = 0, outs = 0;                              // S tiles and O tiles of this query tile so far
        for (int k = 0; take(k); ++k) {
            if (n == 0) continue;
            const int mine = t ? n_t[1] : n_t[0];
            sync_wait(q_full, (uint32_t)qs);
            sync_wait(full(base % S), (uint32_t)(base / S));
            if (!ok) break;
            if (mine > 0) scores(base);
            release(empty(base % S), mine > 0);
            if (mine < 2) release(q_empty, mine > 0);
            for (int j = 0; j < n && ok; ++j) {
                const int iv = base + 2 * j + 1, ik = iv + 1;
                sync_wait(full(iv % S), (uint32_t)(iv / S));
                const int keys = min(kAttnKeys, nk - (j + j0()) * kAttnKeys), steps = (keys + 15) / 16;
                if (keys < 16 * steps && j < mine && ok) {
                    // rows behind the end within the last step: zero, whatever follows the sequence.  Each warp does so
                    // for its own products only (both write the same zeros): O's completion orders these stores before
                    // the tile's next use, and where the keys are split that is tile 0's alone.
                    for (int c = lane; c < (16 * steps - keys) * C::kAtoms * 8; c += 32) {
                        const int row = keys + c / (C::kAtoms * 8), in = c % (C::kAtoms * 8);
                        asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(
                                         ring + (iv % S) * C::kTile + (in / 8) * C::kAtom + row * 128 + (in % 8) * 16),
                                     "r"(0u) : "memory");
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                }
                if (j + 1 < n) sync_wait(full(ik % S), (uint32_t)(ik / S));
                if (j < mine) {
                    if (j == 0 && outs > 0) sync_wait(o_empty(t), outs - 1);
                    sync_wait(p_full(t, 0), turn);
                    if (!ok) break;
                    values(j, iv, 0, steps);
                    sync_wait(p_full(t, 1), turn);
                    if (!ok) break;
                    values(j, iv, 1, steps - 4);
                    ++turn;
                    if (j + 1 < mine) scores(ik);
                    else {
                        release(o_full(t), true);
                        ++outs;
                    }
                }
                if (!ok) break;
                release(empty(iv % S), j < mine);
                if (j + 1 < n) release(empty(ik % S), j + 1 < mine);
                if (j + 2 == mine) release(q_empty, true);        // the last scores have read Q
            }
            if (!ok) break;
            base += 2 * n;
            ++qs;
        }
        // all commits have arrived before shared and tensor memory are given back
        if (ok) {
            if (qs > 0) wait(q_empty, (uint32_t)(qs - 1));
            for (int i = max(0, base - S); i < base; ++i) wait(empty(i % S), (uint32_t)(i / S));
        } else if (attn_elect()) {
            attn_commit(drain(t));                                // what was issued ends first
            tc_wait(drain(t), 0u, false);
        }
        __syncwarp();
    } else if (warp == 11) {
        // ----------------------------------------------------------- schedule
        int id = SPLIT ? (int)(blockIdx.x / (unsigned)a.splits) : (int)blockIdx.x;
        for (int k = 0;; ++k) {
            const PromptItem it = id >= 0 ? prompt_item(a, id, a.tiles * kAttnRows) : PromptItem{};
            // a CTA without an item: the list is shorter than the grid, and so are all that follow
            if (k >= 2) wait(item_empty(k & 1), (uint32_t)(k >> 1) - 1u);
            if (!ok) break;
            if (lane == 0) {
                const uint32_t at = items + 32u * (k & 1);
                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(it.q0), "r"(it.k0), "r"(it.nq), "r"(it.nk)
                             : "memory");
                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at + 16u), "r"(it.row0), "r"(it.head),
                             "r"(it.any ? 1 : 0), "r"(0) : "memory");
                arrive(item_full(k & 1));
            }
            __syncwarp();
            if (!it.any) break;
            if constexpr (SPLIT) {                 // a cluster has one item
                id = -1;
            } else {
                // the next item is taken when this one's loads have been issued: earlier, it would wait here while other
                // CTAs run out of work
                wait(wanted, (uint32_t)k);
                if (!ok) break;
                if (lane == 0) {
                    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], 16;" ::"r"(answered) : "memory");
                    asm volatile(
                        "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                            answer),
                        "r"(answered) : "memory");
                }
                wait(answered, (uint32_t)k);
                if (!ok) break;
                uint32_t got, x;
                asm volatile(
                    "{\n\t.reg .pred p;\n\t.reg .b128 r;\n\t.reg .b32 y, z, w;\n\t"
                    "ld.shared.b128 r, [%2];\n\t"
                    "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
                    "selp.u32 %0, 1, 0, p;\n\tmov.u32 %1, 0;\n\t"
                    "@p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%1, y, z, w}, r;\n\t}"
                    : "=r"(got), "=r"(x)
                    : "r"(answer)
                    : "memory");
                // the answer has been read before the next one may be written over it
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                id = got ? (int)x : -1;
            }
        }
    }
    __syncwarp();
    if constexpr (SPLIT) {
        attn_cluster_sync();
        if (joined) {
            const int r = threadIdx.x & 127;
            if (a.splits == 2) attn_join<D, 2>(ring, r, share, a.scale_log2, joined);
            else if (a.splits == 4) attn_join<D, 4>(ring, r, share, a.scale_log2, joined);
            else attn_join<D, 8>(ring, r, share, a.scale_log2, joined);
        }
        __syncwarp();
        attn_cluster_sync();
    }
    __syncthreads();
    if (warp == 8) {
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    }
}

}  // namespace zt
