// kv_attn.cuh -- attention of a few query tokens per sequence over the paged
// 4-bit KV cache (include/zt_q4.h: zt_q4_kv_attention).
//
// Mathematics.  For a kv head, the columns are its (query token, query head)
// pairs; per tile of 16 cached tokens
//   S[t][c] = sum_g ks[t][g] sum_{d in g} kc[t][d] q[d][c]  +  sum_g ks[t][g] x[g][c],   x[g][c] = -7 sum_{d in g} q[d][c]
//   p[t][c] = 2^(scale log2(e) (S[t][c] - M[c]) + 9)
//   O[d][c] += sum_t (vc[t][d] - 7) (p[t][c] vs[t][g(d)])
// and the result is O[d][c] / sum_t p[t][c].  kc and vc are the 4-bit codes, ks
// and vs the fp16 scales of 32 values.  q is multiplied by a power of two per column
// first, which the column's softmax scale takes back: its largest value lies between
// 2^14 and 2^16, so that neither q / 16 (below) nor x is rounded in fp16's subnormals
// where q is small and the caller's scale large.
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
// M is a reference, not the running maximum: the largest score when it was set (p =
// 2^9 there).  O and the sum of p are rescaled only when a score passes M by 5.5 / (scale
// log2(e)).  That keeps p * vs in the upper range of fp16: with scales below 2 (values
// below 14) p * vs stays under 2^15.5, and a weight of 2^-24 of the largest one still has
// 2 bits.  From the first tile with a scale of 2^e or more on, e > 0, the room is e less,
// first at the cost of the 5.5, down to 1.5, then of the 9.  The difference is taken before the product with the scale: scores may
// be of any size, and near M it is exact.  p goes through the transpose as two fp16
// parts, so that p * vs is rounded once (with p rounded first, the error of a long
// sequence's output was 1.5 times that of its rounding to fp16 alone, not 1.3); sums of p
// and O are fp32.
//
// Work split.  The (sequence, kv head) segments are laid end to end in tiles, each
// with four more that stand for its own cost, and cut into equal runs, one per CTA,
// then one per warp: ragged batches and single long sequences balance alike.  Each
// warp streams its run through a private ring of bulk copies (a tile is K and V),
// two tiles at a time.  Where every segment is short and there are few of them, a
// CTA takes one whole segment.  Segments cut between warps are joined in shared
// memory; of the CTAs that share a segment each leaves its part in the workspace and
// counts itself, and the one that counts last joins them.  Both joins go in the
// order of the tokens: results do not depend on timing.
//
// What bounds it.  One token of 131071 cached ones, 8 kv heads of 128, 4 query heads each
// (151 MB of cache): 47.0 us, 3.2 TB/s; the copies alone, without the products, 25.7 us.  The
// main loop is bound by issue slots and the chains between them (56 % of the slots busy over the
// whole launch, the ALU pipe 47 %, memory 34 %): a pair of tiles takes a warp about 600
// instructions, most of them unpacking codes for the two products.  Joining the warps takes 2 us
// of it and joining the CTAs 5 us, most of that latency.  61 sequences of up to 6001 tokens (174
// MB): 57.5 us; 7 sequences of up to 3999 tokens, 32 kv heads of 96, 4 query tokens (27 MB): 20.9
// us; one sequence of 517 tokens (1.8 MB): 8.15 us, of which streaming takes 4.1, the products 2.7
// and the join 1.1.  Warps: 16 with two pairs of tiles in flight each; 8 with four pairs took 54.0,
// 67.2 and 22.4 us on the first three (then 46.5, 57.0 and 20.9).  Columns: eight at a time.
// Sixteen that share a pass over the tiles (8 warps, for the registers) took 30.1 us where two
// passes of eight take 23.9 (4 sequences of 20000 tokens, 12 columns per kv head; 16 columns: 32.6
// and 24.9), and were faster only where the cache is larger than L2: 131071 tokens of 8 heads, 16
// columns, 79.3 and 81.8; 32 sequences of 8000, 57.4 and 65.0.
// References, in us on the first two: a rounded product scale * M taken off in the multiply-add,
// which holds for scores up to some thousands only, 46.5 and 57.0; with a branch for far ones 47.6
// and 58.3 out of line, 48.1 and 58.9 in the loop; differences first, for any score, as above.
#pragma once

#include "kv_common.cuh"

namespace zt {

struct KvAttnArgs {
    KvPlaces at;
    const __half *q;
    __half *out;
    const int32_t *lens;
    unsigned int *arrived;     // [kKvMaxCtas] zero between calls: partials of a cut segment, counted at its first CTA
    float *part;               // partial results of segments cut between CTAs
    long long ld_q, ld_out;    // elements between query tokens
    int tokens;                // query tokens per sequence
    int q_heads, group;        // group = q_heads / kv_heads
    int cols, blocks;          // columns of a kv head (tokens * group), and blocks of 8 of them
    int whole;                 // 1: a CTA takes one whole segment
    float scale_log2;          // softmax scale * log2(e)
};

template <int D>
struct KvAttnCfg {
    using T = KvTile<D>;
    static constexpr int kWarps = 16;
    static constexpr int kPairs = D == 64 ? 4 : 2;      // ring stages of two tiles
    static constexpr int kStage = 2 * T::kBytes;
    static constexpr int kCols = 8;
    static constexpr int kPart = kCols * (D + 2);                      // floats: O, then R and the sum of p per column
    static constexpr int kRing = kPairs * kStage;                      // per warp; holds the last partial at the end
    static constexpr int kPartBytes = (kPart * 4 + 8 + 15) / 16 * 16;         // and the segment, within a CTA
    static_assert(kPartBytes <= kRing, "a warp's last partial goes to its ring");
    static constexpr int kBars = kWarps * kPairs * 8;
    static constexpr int kFlags = kWarps * (4 + 16) + 32;
    static constexpr int kSmem = kWarps * (kRing + kPartBytes) + kBars + kFlags;   // + KvIndex, 8 bytes per sequence
};

// What starting and ending a segment costs, in tiles.  131071 tokens of 8 heads, 61 ragged sequences, 7 with 4
// query tokens: with 1 49.4, 63.4 and 22.8 us, 2 49.4, 57.5 and 20.9, 4 47.4, 57.7 and 20.9, 8 47.7, 58.0 and 20.7.
constexpr int kKvSegTiles = 4;
constexpr int kKvMaxCtas = 148;        // CTAs that share one call's tiles (and partials in the workspace)
constexpr float kKvOff = 9.f, kKvRoom = 14.5f, kKvSlack = 1.5f;

// Runs of tiles: CTA c of n takes total / n of them, the first total % n CTAs one more.
struct KvRuns {
    int each, more;
    __device__ __forceinline__ KvRuns(int total, int n) : each(total / n), more(total - total / n * n) {}
    __device__ __forceinline__ int start(int c) const { return each * c + min(c, more); }
    __device__ __forceinline__ int owner(int x) const
    {
        return x < more * (each + 1) ? x / (each + 1) : more + (x - more * (each + 1)) / each;
    }
};

// Number of CTAs that share `total` tiles: a tile per warp at least.
__device__ __forceinline__ int kv_ctas(int total, int ctas, int warps)
{
    return max(1, min(ctas, (total + warps - 1) / warps));
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

// (code - 7) * 2^-10 of a pair of codes masked out of its word: the factor (2^14, or 2^10 for the high nibbles' 16
// times larger patterns) undoes the subnormals' 2^-24.
constexpr uint32_t kKvLow = 0x74007400u, kKvHigh = 0x64006400u, kKvMinus7 = 0x9F009F00u;
__device__ __forceinline__ uint32_t kv_value(uint32_t codes, uint32_t f)
{
    return h2_bits(__hfma2(bits_h2(codes), bits_h2(f), bits_h2(kKvMinus7)));
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

// The sequences in shared memory: lengths, and first[b] = virtual tiles (with every segment's kKvSegTiles) of the
// sequences before b.
struct KvIndex {
    int *first, *lens;
    int per, n;                // segments per sequence (kv heads x column blocks), sequences

    __device__ __forceinline__ void build(const KvAttnArgs &a, int *mem)
    {
        n = a.at.n_seqs;
        per = a.at.kv_heads * a.blocks;
        first = mem;
        lens = mem + n + 1;
        const int lane = threadIdx.x & 31;
        if (n <= 32) {
            // every warp by itself (all write the same)
            const int len = lane < n ? kv_len(a, lane) : 0;
            const int upto = scan(lane < n ? ((len + kKvTile - 1) / kKvTile + kKvSegTiles) * per : 0);
            if (lane < n) {
                lens[lane] = len;
                first[lane + 1] = upto;
            }
            if (lane == 0) first[0] = 0;
            __syncwarp();
            return;
        }
        for (int b = threadIdx.x; b < n; b += blockDim.x) lens[b] = kv_len(a, b);
        __syncthreads();
        if (threadIdx.x < 32) {
            int base = 0;
            for (int b0 = 0; b0 < n; b0 += 32) {
                const int b = b0 + lane;
                const int upto = base + scan(b < n ? ((lens[b] + kKvTile - 1) / kKvTile + kKvSegTiles) * per : 0);
                if (b < n) first[b + 1] = upto;
                base = __shfl_sync(0xffffffffu, upto, 31);
            }
            if (lane == 0) first[0] = 0;
        }
        __syncthreads();
    }
    __device__ static __forceinline__ int scan(int v)
    {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, v, o);
            if ((int)(threadIdx.x & 31) >= o) v += u;
        }
        return v;
    }
    __device__ __forceinline__ int total() const { return first[n]; }
};

// A tile: sequence, head-and-block, index within the segment (which may lie behind its last tile, in the virtual ones).
struct KvCursor {
    int b, hc, tile, tiles, len;
    __device__ __forceinline__ void enter(const KvIndex &ix)
    {
        len = ix.lens[b];
        tiles = (len + kKvTile - 1) / kKvTile;
    }
    __device__ __forceinline__ void seek(const KvIndex &ix, int x)
    {
        int lo = 0, hi = ix.n;                              // first[lo] <= x < first[hi]
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (ix.first[mid] <= x) lo = mid;
            else hi = mid;
        }
        b = lo;
        enter(ix);
        const int rel = x - ix.first[b];
        hc = rel / (tiles + kKvSegTiles);
        tile = rel - hc * (tiles + kKvSegTiles);
    }
    // tiles (not virtual ones) before this position, which is x
    __device__ __forceinline__ int before(const KvIndex &ix, int x) const
    {
        return x - kKvSegTiles * (b * ix.per + hc) - max(0, tile - tiles);
    }
    // on to the start of the next segment that has tiles; there is one
    __device__ __forceinline__ void next_segment(const KvIndex &ix)
    {
        tile = 0;
        if (++hc < ix.per) return;
        hc = 0;
        do {
            ++b;
            enter(ix);
        } while (tiles == 0);
    }
};

// b's halves, zero where p's are.  Kept out of line: it is hardly ever needed.
static __device__ __noinline__ uint32_t kv_hide(uint32_t b, uint32_t p) { return b & ~__vcmpeq2(p, 0u); }

// Largest V scale among a lane's, as fp16 bits; a NaN counts as the largest number: columns that see it are lost, and others
// it is hidden from in a sequence's last tiles only.  Out of line: for scales of 2 and more.
template <int N>
struct KvScales {
    uint32_t w[N];
};
template <int N>
static __device__ __noinline__ uint32_t kv_largest(KvScales<N> s)
{
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < N; ++i) m = __vmaxu2(m, s.w[i] & 0x7FFF7FFFu);
    return min(max(m & 0xFFFFu, m >> 16), 0x7BFFu);
}

// Columns of head-and-block hc.
__device__ __forceinline__ int kv_columns(const KvAttnArgs &a, int hc, int kcols)
{
    return a.blocks == 1 ? a.cols : min(kcols, a.cols - hc % a.blocks * kcols);
}

// Row of the output for column c of (b, hc).
__device__ __forceinline__ __half *kv_out_row(const KvAttnArgs &a, int b, int hc, int c, int kcols, int D)
{
    const int h = a.blocks == 1 ? hc : hc / a.blocks, col = (hc - h * a.blocks) * kcols + c;
    const int i = a.tokens == 1 ? 0 : col / a.group, head = h * a.group + (col - i * a.group);
    return a.out + ((long long)b * a.tokens + i) * a.ld_out + head * D;
}

// Zeros for the queries of a sequence without tokens: whole CTA.
__device__ __forceinline__ void kv_zero(const KvAttnArgs &a, int b, int hc, int kcols, int D)
{
    for (int i = threadIdx.x; i < kv_columns(a, hc, kcols) * D; i += blockDim.x)
        kv_out_row(a, b, hc, i / D, kcols, D)[i % D] = __float2half_rn(0.f);
}

__device__ __forceinline__ float kv_lds_f32(uint32_t addr)
{
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr));
    return v;
}

// One column's partial results joined in order by a warp: a lane has values lane, lane + 32, ...
template <int D>
struct KvSum {
    float top = -INFINITY, l = 0.f, acc[D / 32] = {};
    // four partials (reference, sum of p, values); a missing one has the reference -inf, and its values count nothing
    __device__ __forceinline__ void add(const float (&R)[4], const float (&l1)[4], const float (&v)[4][D / 32])
    {
        const float to = fmaxf(fmaxf(fmaxf(R[0], R[1]), fmaxf(R[2], R[3])), top), ref = to == -INFINITY ? 0.f : to;
        const float f = kv_exp2(top - ref);
        l *= f;
#pragma unroll
        for (int e = 0; e < D / 32; ++e) acc[e] *= f;
        top = to;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const float w = kv_exp2(R[u] - ref);
            const bool counts = R[u] != -INFINITY;      // a place without a partial may hold anything
            l += counts ? l1[u] * w : 0.f;
#pragma unroll
            for (int e = 0; e < D / 32; ++e) acc[e] += counts ? v[u][e] * w : 0.f;
        }
    }
    __device__ __forceinline__ void store(__half *row) const
    {
        const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
        for (int e = 0; e < D / 32; ++e) row[32 * e + (threadIdx.x & 31)] = __float2half_rn(acc[e] * inv);
    }
    // as a partial of `cols` columns: values, then references, then sums
    __device__ __forceinline__ void leave(float *part, int c, int cols) const
    {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int e = 0; e < D / 32; ++e) part[c * D + 32 * e + lane] = acc[e];
        if (lane == 0) {
            part[cols * D + c] = top;
            part[cols * (D + 1) + c] = l;
        }
    }
};

template <int D>
__global__ void __launch_bounds__(KvAttnCfg<D>::kWarps * 32, 1) kv_attn_kernel(const __grid_constant__ KvAttnArgs a)
{
    using C = KvAttnCfg<D>;
    using T = KvTile<D>;
    constexpr int G = T::kG, W = C::kWarps, S = C::kPairs;
    extern __shared__ __align__(128) unsigned char kv_smem_raw[];
    unsigned char *rings = kv_smem_raw;
    float *heads = reinterpret_cast<float *>(kv_smem_raw + W * C::kRing);      // a warp's first partial
    const uint32_t bars = kv_smem(kv_smem_raw) + W * (C::kRing + C::kPartBytes);
    int *index = reinterpret_cast<int *>(kv_smem_raw + C::kSmem);
    // all shared memory is dynamic: the opt-in limit leaves no room for a static part
    int4 *starts = reinterpret_cast<int4 *>(index) - W;     // of each warp's run: sequence, head-and-block, tile, tiles
    int4 *chains = starts - 2;       // the segments cut at the run's start and at its end: first CTA (-1: none),
                                     // number of CTAs, sequence, head-and-block
    int *flags = reinterpret_cast<int *>(chains) - W;
                                     // of each warp: 1 it had tiles, 2 its last segment goes on in the next warp,
                                     // 4 and began in it, 8 it wrote the end of a segment that began earlier

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, j = lane & 3;
    const uint32_t ring = kv_smem(rings) + warp * C::kRing, bar = bars + 8 * warp * S;
    if (lane < S) asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(bar + 8 * lane) : "memory");
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    kv_pdl_launch();
    kv_pdl_wait();

    // this CTA's run of tiles: its share of all of them, or one whole segment
    KvIndex ix;
    KvCursor at = {};
    if (a.whole) {
        const int per = a.at.kv_heads * a.blocks;
        at.b = blockIdx.x / per;
        at.hc = blockIdx.x - at.b * per;
        at.len = kv_len(a, at.b);
        at.tiles = (at.len + kKvTile - 1) / kKvTile;
        __syncwarp();
        if (at.tiles == 0) {
            kv_zero(a, at.b, at.hc, C::kCols, D);
            return;
        }
    } else {
        ix.build(a, index);
        for (int b = blockIdx.x; b < ix.n; b += gridDim.x)
            if (ix.lens[b] == 0)
                for (int hc = 0; hc < ix.per; ++hc) kv_zero(a, b, hc, C::kCols, D);
        const int total = ix.total(), n_ctas = kv_ctas(total, gridDim.x, W);
        if ((int)blockIdx.x >= n_ctas) return;
        if (warp == 0) {
            // lane w finds where warp w's run starts (lane W: where the last one ends)
            const KvRuns runs(total, n_ctas);
            const int c_lo = runs.start(blockIdx.x), c_n = runs.start(blockIdx.x + 1) - c_lo;
            const int x = c_lo + (int)((long long)c_n * min(lane, W) / W);
            KvCursor c = {};
            int before = total - kKvSegTiles * ix.n * ix.per;
            if (x < total) {
                c.seek(ix, x);
                before = c.before(ix, x);
            }
            // the segments that this run's start and end cut: their first CTA, and how many share them
            if (lane == 0 || lane == W) {
                int4 chain = make_int4(-1, 0, c.b, c.hc);
                if (x < total && c.tile > 0 && c.tile < c.tiles) {
                    chain.x = runs.owner(x - c.tile);
                    chain.y = runs.owner(x - c.tile + c.tiles - 1) - chain.x + 1;
                }
                chains[lane == W] = chain;
            }
            const int here = __shfl_down_sync(0xffffffffu, before, 1) - before;
            if (lane < W) {
                if (here > 0 && c.tile >= c.tiles) c.next_segment(ix);
                starts[lane] = make_int4(c.b, c.hc, c.tile, here);
            }
        }
        __syncthreads();
    }
    // this warp's run: n tiles from seg on
    KvCursor seg = at;
    int n;
    if (a.whole) {
        seg.tile = at.tiles * warp / W;
        n = at.tiles * (warp + 1) / W - seg.tile;
    } else {
        const int4 s = starts[warp];
        seg.b = s.x;
        seg.hc = s.y;
        seg.tile = s.z;
        n = s.w;
        if (n > 0) seg.enter(ix);
    }

    float *tail = reinterpret_cast<float *>(rings + warp * C::kRing);
    float *head_part = heads + warp * (C::kPartBytes / 4);
    const int tpp = a.at.page_size / kKvTile;

    // The copying side runs kPairs steps ahead.  A step is two tiles of a segment, or one where the segment or
    // the run ends; src walks through the page that ahead's next tile is in.
    KvCursor ahead = {};
    const unsigned char *src = nullptr;
    int in_page = 0, page_at = 0, to_copy = n;
    int entry = 0, entry_b = -1, entry_at = 0;      // lane i holds the table's entry entry_at + i of sequence entry_b
    unsigned bad = 0;                // two bits per stage: tiles that have no page
    auto open_page = [&]() {
        if (ahead.b != entry_b || page_at < entry_at || page_at >= entry_at + 32) {
            entry_b = ahead.b;
            entry_at = page_at;
            const int last = (ahead.tiles - 1) / tpp;
            entry = page_at + lane <= last ? __ldg(a.at.table + (long long)entry_b * a.at.max_pages + page_at + lane) : -1;
        }
        const int page = __shfl_sync(0xffffffffu, entry, page_at - entry_at);
        const bool fine = page >= 0 && page < a.at.n_pages;
        src = fine ? a.at.pages + page * a.at.page_bytes + ((long long)(ahead.hc / a.blocks) * tpp + in_page) * T::kBytes
                   : nullptr;
        if (!fine && lane == 0) kv_error(a.at.err, kErrKvPlace);
    };
    // a step reads the cache once (with several blocks of columns once a block): it should not push out of L2 what is
    // read again, this kernel's code first of all
    uint64_t once;
    asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(once));
    auto copy = [&](int s, int u, int tiles) {      // `tiles` tiles from src on, to place u of stage s
        if (lane == 0 && src)
            asm volatile(
                "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;" ::
                    "r"(ring + s * C::kStage + u * T::kBytes),
                "l"(src), "r"(tiles * T::kBytes), "r"(bar + 8 * s), "l"(once) : "memory");
    };
    auto expect = [&](int s, int tiles) {           // a stage's arrival: the bytes of this many tiles
        if (lane == 0) {
            if (tiles)
                asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar + 8 * s), "r"(tiles * T::kBytes)
                             : "memory");
            else
                asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar + 8 * s) : "memory");
        }
    };
    auto next_page = [&]() {
        in_page = 0;
        ++page_at;
        open_page();
    };
    auto issue = [&](int s) {
        const int step = min(min(2, to_copy), ahead.tiles - ahead.tile);
        if (src && in_page + step <= tpp) {         // both tiles lie side by side
            expect(s, step);
            copy(s, 0, step);
            src += step * T::kBytes;
            in_page += step;
            bad &= ~(3u << (2 * s));
        } else {
            // from one page to the next, or a page out of range; the next page's address is known before
            // the stage's bytes are announced
            const unsigned char *one = src;
            const unsigned miss0 = src ? 0u : 1u;
            if (step == 2) {
                if (++in_page == tpp) next_page();
                else if (src) src += T::kBytes;
            }
            const unsigned miss1 = step == 2 && !src ? 2u : 0u;
            bad = (bad & ~(3u << (2 * s))) | ((miss0 | miss1) << (2 * s));
            expect(s, step - (int)miss0 - (int)(miss1 >> 1));
            const unsigned char *two = src;
            src = one;
            copy(s, 0, 1);
            if (step == 2) {
                src = two;
                copy(s, 1, 1);
            }
            if (src) src += T::kBytes;
            ++in_page;
        }
        to_copy -= step;
        if (to_copy == 0) return;
        ahead.tile += step;
        if (ahead.tile == ahead.tiles) {
            ahead.next_segment(ix);
            in_page = page_at = 0;
            open_page();
        } else if (in_page == tpp) {
            next_page();
        }
    };

    bool is_open = false, did_begin = false, did_first = false;
    if (n > 0) {
        ahead = seg;
        page_at = ahead.tile / tpp;
        in_page = ahead.tile - page_at * tpp;
        open_page();
        for (int s = 0; s < C::kPairs && to_copy > 0; ++s) issue(s);
    }

    float O[D / 16][4], minus_m[2], L[2], most[2];      // -M (0 without one); largest score without a rescale (-inf)
    uint32_t qf[G][4], xq;
    int seen[2];                 // tokens that columns 2j and 2j + 1 see
    float room = kKvRoom;             // less e, where 2^e is the largest power of two among the V scales so far (above 1)
    auto off_of = [](float room) { return fminf(kKvOff, room - kKvSlack); };
    float sl[2];                 // softmax scale of columns 2j and 2j + 1, in the units of S as it is computed
    bool fresh = true, dead = false;
    int seg_tile0 = 0, step = 1, s = 0;
    uint32_t parity = 0;
    for (int x = 0; x < n; x += step) {
        if (fresh) {
            // a new segment: its queries as B fragments, the zero point's term, the columns' ends
            fresh = false;
            seg_tile0 = seg.tile;
            room = kKvRoom;
            const int h = seg.hc / a.blocks, c0 = (seg.hc - h * a.blocks) * C::kCols;
            const int col = c0 + r;
            const bool has = col < a.cols;
            const int i = has ? col / a.group : 0, qh = h * a.group + (has ? col - i * a.group : 0);
            const __half *q = a.q + ((long long)seg.b * a.tokens + i) * a.ld_q + qh * D + 8 * j;
            __half xlo = __float2half_rn(0.f), xhi = xlo;
            uint4 raw[G];
            uint32_t top = 0u;                     // bit patterns of |q| go up with it; an infinity or a NaN lifts by 2^0
#pragma unroll
            for (int g = 0; g < G; ++g) {
                raw[g] = has ? *reinterpret_cast<const uint4 *>(q + 32 * g) : make_uint4(0, 0, 0, 0);
                top = __vmaxu2(top, __vmaxu2(__vmaxu2(raw[g].x & 0x7FFF7FFFu, raw[g].y & 0x7FFF7FFFu),
                                             __vmaxu2(raw[g].z & 0x7FFF7FFFu, raw[g].w & 0x7FFF7FFFu)));
            }
            top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const float big = __half2float(__ushort_as_half((unsigned short)max(top & 0xFFFFu, top >> 16)));
            const int lift = max(0, 14 + 127 - max((int)(__float_as_uint(big) >> 23), 127 - 24));
            const float up = __uint_as_float((uint32_t)(127 + lift) << 23);
#pragma unroll
            for (int e = 0; e < 2; ++e)
                sl[e] = a.scale_log2 * __uint_as_float((uint32_t)(127 + 24 - __shfl_sync(0xffffffffu, lift, 4 * (2 * j + e))) << 23);
#pragma unroll
            for (int g = 0; g < G; ++g) {
                float2 f0 = __half22float2(bits_h2(raw[g].x)), f1 = __half22float2(bits_h2(raw[g].y)),
                       f2 = __half22float2(bits_h2(raw[g].z)), f3 = __half22float2(bits_h2(raw[g].w));
                float sum = ((f0.x + f0.y) + (f1.x + f1.y)) + ((f2.x + f2.y) + (f3.x + f3.y));
                f0.x *= up, f0.y *= up, f1.x *= up, f1.y *= up, f2.x *= up, f2.y *= up, f3.x *= up, f3.y *= up;
                const uint4 w = make_uint4(h2_bits(__float22half2_rn(f0)), h2_bits(__float22half2_rn(f1)),      // exact
                                           h2_bits(__float22half2_rn(f2)), h2_bits(__float22half2_rn(f3)));
                sum += __shfl_xor_sync(0xffffffffu, sum, 1);
                sum += __shfl_xor_sync(0xffffffffu, sum, 2);
                // lane j of a quad keeps the two groups of its k slots: groups 0..3 rounded to fp16 in
                // slots 0..3, what the rounding left in slots 4..7 (2^-8 of them, so that none overflows)
                sum *= -7.f * 0x1p-8f * up;
                const __half high = __float2half_rn(sum);
                const __half part = j < 2 ? high : __float2half_rn(sum - __half2float(high));
                if (g / 2 == (j & 1)) (g & 1 ? xhi : xlo) = part;
                // step 0 of a group meets codes 0, 4 | 2, 6 of the lane's word, step 1 codes 1, 5 | 3, 7,
                // which come with a factor 16
                const __half2 six = __float2half2_rn(0.0625f);
                qf[g][0] = __byte_perm(w.x, w.z, 0x5410);
                qf[g][1] = __byte_perm(w.y, w.w, 0x5410);
                qf[g][2] = h2_bits(__hmul2(bits_h2(__byte_perm(w.x, w.z, 0x7632)), six));
                qf[g][3] = h2_bits(__hmul2(bits_h2(__byte_perm(w.y, w.w, 0x7632)), six));
            }
            xq = h2_bits(__halves2half2(xlo, xhi));
#pragma unroll
            for (int m = 0; m < D / 16; ++m)
#pragma unroll
                for (int e = 0; e < 4; ++e) O[m][e] = 0.f;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                most[e] = -INFINITY;
                minus_m[e] = L[e] = 0.f;
                seen[e] = seg.len - a.tokens + 1 + (c0 + 2 * j + e) / a.group;
            }
        }
        // Two tiles at a time, for independent work between the waits and one look at the maxima; a last
        // odd one goes alone, its missing partner masked.
        step = min(min(2, n - x), seg.tiles - seg.tile);
        if (!dead && !__all_sync(0xffffffffu, tc_wait(bar + 8 * s, parity, false))) {
            // a copy did not land in time: report it, give the other copies in flight their time, and go on
            // without reading tiles (the results are incomplete)
            if (lane == 0) kv_error(a.at.err, kErrKvWait);
            for (int i = 0; i < S && n - x - to_copy > i; ++i)
                tc_wait(bar + 8 * ((s + i) % S), parity ^ (s + i >= S ? 1u : 0u), false);
            __syncwarp();
            dead = true;
        }
        const bool drop0 = dead || ((bad >> (2 * s)) & 1u), drop1 = dead || step < 2 || ((bad >> (2 * s)) & 2u);
        const uint32_t stage = ring + s * C::kStage;
        const uint32_t tile[2] = {stage, stage + T::kBytes};
        float P[2][4];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            uint32_t wa[G], wb[G], ks[G], kz[2];
            kv_lds<G>(wa, tile[u] + (r * 4 + j) * G * 4);
            kv_lds<G>(wb, tile[u] + ((r + 8) * 4 + j) * G * 4);
            kv_lds<G>(ks, tile[u] + T::kKs + r * G * 4);
            // this lane's two groups of scales again, by token: the A operand of the zero point's product.  A slot
            // without a group meets zeros in B; its scale must be this token's, or zero, not another's NaN.
            if constexpr (G == 4) {
                kv_lds<2>(kz, tile[u] + T::kKs + (r * G + 2 * (j & 1)) * 4);
            } else {
                kz[0] = G == 3 && (j & 1) ? ks[G - 1] : ks[0];
                kz[1] = G == 3 && (j & 1) ? 0u : ks[1];
            }
            const uint32_t za = __byte_perm(kz[0], kz[1], 0x5410), zb = __byte_perm(kz[0], kz[1], 0x7632);
#pragma unroll
            for (int g = 0; g < G; ++g) {
                const float2 sc = __half22float2(bits_h2(ks[g]));
                const uint32_t ha = wa[g] >> 8, hb = wb[g] >> 8;
                float d[4];
                float (&p)[4] = P[u];
                kv_mma(d, wa[g] & 0x000F000Fu, wb[g] & 0x000F000Fu, ha & 0x000F000Fu, hb & 0x000F000Fu, qf[g][0],
                       qf[g][1], 0.f, 0.f, 0.f, 0.f);
                kv_mma(d, wa[g] & 0x00F000F0u, wb[g] & 0x00F000F0u, ha & 0x00F000F0u, hb & 0x00F000F0u, qf[g][2],
                       qf[g][3], d[0], d[1], d[2], d[3]);
                const uint64_t lo = f2_pack(sc.x, sc.x), hi = f2_pack(sc.y, sc.y), d01 = f2_pack(d[0], d[1]), d23 = f2_pack(d[2], d[3]);
                const float2 p01 = f2_split(g ? f2_fma(lo, d01, f2_pack(p[0], p[1])) : f2_mul(lo, d01));
                const float2 p23 = f2_split(g ? f2_fma(hi, d23, f2_pack(p[2], p[3])) : f2_mul(hi, d23));
                p[0] = p01.x, p[1] = p01.y, p[2] = p23.x, p[3] = p23.y;
            }
            float z[4];
            kv_mma(z, za, zb, 0u, 0u, xq, 0u, 0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int e = 0; e < 4; ++e) P[u][e] = fmaf(z[e], 0x1p-16f, P[u][e]);
        }
        // the V scales of this lane's tokens 2j, 2j + 1 and 2j + 8, 2j + 9
        uint32_t vs[2][2 * G];
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int g = 0; g < G; g += G % 2 ? 1 : 2) {
                uint32_t w[G % 2 ? 2 : 4];
                kv_lds<G % 2 ? 2 : 4>(w, tile[u] + T::kVs + (j * G + g) * 8);
#pragma unroll
                for (int i = 0; i < (G % 2 ? 2 : 4); ++i) vs[u][2 * g + i] = w[i];
            }
        const int t0 = seg.tile * kKvTile;
        // some column does not see all of both tiles
        const bool edge = t0 + 2 * kKvTile > seg.len - a.tokens + 1 || drop0 || drop1;
        bool mend = false;
        if (__builtin_expect(edge, 0)) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const bool drop = u ? drop1 : drop0;
                const int tu = t0 + u * kKvTile;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (drop || tu + r + 8 * (e >> 1) >= seen[e & 1]) P[u][e] = -INFINITY;
                // places behind the sequence's end may hold anything
#pragma unroll
                for (int g = 0; g < G; ++g)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int t = tu + 8 * h + 2 * j;
                        if (drop || t >= seg.len) vs[u][2 * g + h] = 0u;
                        else if (t + 1 >= seg.len) vs[u][2 * g + h] &= 0xFFFFu;
                    }
            }
        }
        uint32_t any = 0;
#pragma unroll
        for (int g = 0; g < 2 * G; ++g) any |= vs[0][g] | vs[1][g];
        if (__builtin_expect(edge && __any_sync(0xffffffffu, (any & 0x40004000u) != 0u), 0)) {
            // a token may be hidden from some columns only, and its scale be NaN (which the test above
            // catches, among other large ones): nothing times NaN is nothing there
            mend = true;
        }
        const bool large = (any & 0x40004000u) != 0u;                // a scale of 2 or more
        bool lift = false;
        uint32_t met = 0u;
        if (__builtin_expect(large, 0)) {
            KvScales<4 * G> all;
#pragma unroll
            for (int g = 0; g < 2 * G; ++g) {
                all.w[g] = vs[0][g];
                all.w[2 * G + g] = vs[1][g];
            }
            met = kv_largest(all);
            lift = (float)(int)(met >> 10) > kKvRoom + 15.f - room;
        }
#pragma unroll
        for (int e = 0; e < 2; ++e)
            lift |= fmaxf(fmaxf(P[0][e], P[0][e + 2]), fmaxf(P[1][e], P[1][e + 2])) > most[e];
        if (__any_sync(0xffffffffu, lift)) {
            const float before = off_of(room);
            room = fminf(room, kKvRoom + 15.f - (float)(int)(__reduce_max_sync(0xffffffffu, met) >> 10));
            const float off = off_of(room);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float mx = fmaxf(fmaxf(P[0][e], P[0][e + 2]), fmaxf(P[1][e], P[1][e + 2]));
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                const float old = most[e] == -INFINITY ? -INFINITY : -minus_m[e], now = fmaxf(old, mx);
                const float f = kv_exp2(old == now ? off - before : fmaf(old - now, sl[e], off - before));
                minus_m[e] = now == -INFINITY ? 0.f : -now;
                most[e] = __fadd_rd(now, __fdividef(room - off, sl[e]));      // the room has half a power of two to spare
                L[e] *= f;
#pragma unroll
                for (int m = 0; m < D / 16; ++m) {
                    O[m][e] *= f;
                    O[m][e + 2] *= f;
                }
            }
        }
        uint32_t pt[2][2], pl[2][2];      // the weights as B fragments: rounded, and what the rounding left
        const uint64_t m2 = f2_pack(minus_m[0], minus_m[1]), sl2 = f2_pack(sl[0], sl[1]), off2 = f2_pack(off_of(room), off_of(room));
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const float2 x01 = f2_split(f2_fma(f2_add(f2_pack(P[u][0], P[u][1]), m2), sl2, off2));
            const float2 x23 = f2_split(f2_fma(f2_add(f2_pack(P[u][2], P[u][3]), m2), sl2, off2));
            const float p0 = kv_exp2(x01.x), p1 = kv_exp2(x01.y), p2 = kv_exp2(x23.x), p3 = kv_exp2(x23.y);
            const float2 sums = f2_split(f2_add(f2_pack(L[0], L[1]), f2_add(f2_pack(p0, p1), f2_pack(p2, p3))));
            L[0] = sums.x;
            L[1] = sums.y;
            const __half2 h01 = __floats2half2_rn(p0, p1), h23 = __floats2half2_rn(p2, p3);
            const float2 f01 = __half22float2(h01), f23 = __half22float2(h23);
            pt[u][0] = kv_transpose(h2_bits(h01));
            pt[u][1] = kv_transpose(h2_bits(h23));
            pl[u][0] = kv_transpose(h2_bits(__floats2half2_rn(p0 - f01.x, p1 - f01.y)));
            pl[u][1] = kv_transpose(h2_bits(__floats2half2_rn(p2 - f23.x, p3 - f23.y)));
        }
#pragma unroll
        for (int g = 0; g < G; ++g)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                uint32_t w[2], va[2][4];
                kv_lds<2>(w, tile[u] + T::kV + (g * 64 + lane * 2) * 4);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t hi = w[i] >> 8;
                    va[i][0] = kv_value(w[i] & 0x000F000Fu, kKvLow);
                    va[i][1] = kv_value(w[i] & 0x00F000F0u, kKvHigh);
                    va[i][2] = kv_value(hi & 0x000F000Fu, kKvLow);
                    va[i][3] = kv_value(hi & 0x00F000F0u, kKvHigh);
                }
                const __half2 s0 = bits_h2(vs[u][2 * g]), s1 = bits_h2(vs[u][2 * g + 1]);
                uint32_t b0 = h2_bits(__hfma2(bits_h2(pt[u][0]), s0, __hmul2(bits_h2(pl[u][0]), s0)));
                uint32_t b1 = h2_bits(__hfma2(bits_h2(pt[u][1]), s1, __hmul2(bits_h2(pl[u][1]), s1)));
                if (mend) {
                    b0 = kv_hide(b0, pt[u][0]);
                    b1 = kv_hide(b1, pt[u][1]);
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float (&o)[4] = O[2 * g + i];
                    kv_mma(o, va[i][0], va[i][1], va[i][2], va[i][3], b0, b1, o[0], o[1], o[2], o[3]);
                }
            }
        __syncwarp();                                                     // all lanes have read the stage
        if (to_copy > 0 && !dead) issue(s);
        if (++s == S) {
            s = 0;
            parity ^= 1u;
        }

        const bool ends = seg.tile + step == seg.tiles;
        if (ends || x + step == n) {
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
            for (int e = 0; e < 2; ++e) {
                float l = L[e];
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
                const int c = 2 * j + e;
                if (c >= kv_columns(a, seg.hc, C::kCols)) continue;
                if (whole) {
                    __half *row = kv_out_row(a, seg.b, seg.hc, c, C::kCols, D);
                    const float inv = l == 0.f ? 0.f : 0x1p10f / l;
#pragma unroll
                    for (int m = 0; m < D / 16; ++m) {
                        row[16 * m + r] = __float2half_rn(O[m][e] * inv);
                        row[16 * m + 8 + r] = __float2half_rn(O[m][e + 2] * inv);
                    }
                } else {
#pragma unroll
                    for (int m = 0; m < D / 16; ++m) {
                        dst[c * D + 16 * m + r] = O[m][e] * 0x1p10f;
                        dst[c * D + 16 * m + 8 + r] = O[m][e + 2] * 0x1p10f;
                    }
                    if (r == 0) {
                        // without a reference, tokens were not seen, or all of their scores were NaN: those count
                        const float ref = most[e] == -INFINITY ? most[e] : -fmaf(minus_m[e], sl[e], off_of(room));
                        dst[C::kCols * D + c] = l != l ? fmaxf(ref, 0.f) : ref;
                        dst[C::kCols * (D + 1) + c] = l;
                        reinterpret_cast<int *>(dst)[C::kPart] = seg.b;
                        reinterpret_cast<int *>(dst)[C::kPart + 1] = seg.hc;
                    }
                }
            }
            fresh = true;
        }
        seg.tile += step;
        if (ends && x + step < n) seg.next_segment(ix);
    }
    if (lane == 0) flags[warp] = (n > 0 ? 1 : 0) | (is_open ? 2 : 0) | (did_begin ? 4 : 0) | (did_first ? 8 : 0);
    __syncthreads();

    // Join the segments that this CTA's warps share.  Each is a chain of warps: it starts where the segment begins
    // (or at the first warp with tiles, for one that began in an earlier CTA) and ends with the warp that wrote its
    // end (or the last warp with tiles).  All warps see the chains alike and take their columns in turn.
    const int mine = lane < W ? flags[lane] : 0;
    const unsigned some = __ballot_sync(0xffffffffu, mine & 1), opens = __ballot_sync(0xffffffffu, mine & 2),
                   begins = __ballot_sync(0xffffffffu, mine & 4), ends = __ballot_sync(0xffffffffu, mine & 8);
    const unsigned leader = some & (0u - some);
    unsigned left = opens & (begins | leader);
    bool came = (ends & leader) != 0u;            // a segment of an earlier CTA ends in the first warp
    const uint32_t tails_s = kv_smem(rings), heads_s = kv_smem(heads);
#pragma unroll 1
    for (int task = warp; came || left;) {
        // w0's partial (its tail; its head, if it is the whole chain), the tails of the warps between, w1's
        const int w0 = __ffs(came ? leader : left) - 1;
        const unsigned end = came ? leader : ends & ~((2u << w0) - 1u);
        const int w1 = end ? __ffs(end) - 1 : 31 - __clz(some);
        const bool ends_here = end != 0u, whole = ends_here && !came && ((begins >> w0) & 1u);
        const unsigned in = some & ((2u << w1) - 1u) & ~((1u << w0) - 1u);
        if (came) came = false;
        else left &= left - 1;
        auto part = [&](int w) {
            return w == w1 && ends_here ? heads_s + w * C::kPartBytes : tails_s + w * C::kRing;
        };
        int b, hc;
        asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(b), "=r"(hc) : "r"(part(w0) + C::kPart * 4));
        const int tasks = kv_columns(a, hc, C::kCols);
#pragma unroll 1
        for (; task < tasks; task += W) {
            KvSum<D> sum;
#pragma unroll 1
            for (unsigned rest = in; rest;) {
                // four partials at a time, loaded without branches
                float R1[4], l1[4], v[4][D / 32];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const bool has = rest != 0u;
                    const uint32_t p = part(has ? __ffs(rest) - 1 : w0);
                    rest &= rest - 1u;
                    R1[u] = kv_lds_f32(p + (C::kCols * D + task) * 4);
                    l1[u] = kv_lds_f32(p + (C::kCols * (D + 1) + task) * 4);
#pragma unroll
                    for (int e = 0; e < D / 32; ++e) v[u][e] = kv_lds_f32(p + (task * D + 32 * e + lane) * 4);
                    if (!has) R1[u] = -INFINITY;
                }
                sum.add(R1, l1, v);
            }
            if (whole) sum.store(kv_out_row(a, b, hc, task, C::kCols, D));
            else sum.leave(a.part + (2ll * blockIdx.x + (ends_here ? 0 : 1)) * C::kPart, task, C::kCols);
        }
        task -= tasks;                            // the next chain's tasks follow on
        if (task < 0) task += W;
    }
    if (a.whole) return;

    // Parts left in the workspace: the CTA that counts last for a segment joins them.
    if (chains[0].x < 0 && chains[1].x < 0) return;
    __syncthreads();
    if (threadIdx.x < 2) {
        // a segment that covers the whole run is cut at both ends, but left one part
        const int f = chains[threadIdx.x].x, parts = chains[threadIdx.x].y;
        bool joins = false;
        if (f >= 0 && (threadIdx.x == 1 || f != chains[1].x)) {
            __threadfence();
            const unsigned before = atomicAdd(a.arrived + f, 1u);
            joins = before == (unsigned)(parts - 1);
            if (joins) a.arrived[f] = 0u;                   // for the next call
            else if (before >= (unsigned)parts) kv_error(a.at.err, kErrKvWork);
            __threadfence();
        }
        flags[threadIdx.x] = joins;
    }
    __syncthreads();
    for (int k = 0; k < 2; ++k) {
        if (!flags[k]) continue;
        const int4 chain = chains[k];
        const int parts = chain.y, cols = kv_columns(a, chain.w, C::kCols);
        const float *base = a.part + (2ll * chain.x + 1) * C::kPart;      // the last part lies one slot earlier
        // warp w takes column w % cols, and of its parts every q-th: the W / cols warps of a column halve the
        // rounds of loads; what each has goes through shared memory (the rings are done with)
        static_assert(W >= 2 * C::kCols, "two warps a column at least");
        const int q = W / cols;
        float *slots = reinterpret_cast<float *>(rings);
#pragma unroll 1
        for (int c = warp; c < cols * q; c += W) {
            KvSum<D> sum;
            const int col = c % cols;
#pragma unroll 1
            for (int i = c / cols; i < parts; i += 4 * q) {
                float R1[4], l1[4], v[4][D / 32];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int k = i + u * q;
                    const float *p = base + (2 * min(k, parts - 1) - (k >= parts - 1 ? 1 : 0)) * C::kPart;
                    R1[u] = __ldcg(p + C::kCols * D + col);
                    l1[u] = __ldcg(p + C::kCols * (D + 1) + col);
#pragma unroll
                    for (int e = 0; e < D / 32; ++e) v[u][e] = __ldcg(p + col * D + 32 * e + lane);
                    if (k >= parts) R1[u] = -INFINITY;
                }
                sum.add(R1, l1, v);
            }
            sum.leave(slots, c, W);
        }
        __syncthreads();
        if (warp < cols) {
            KvSum<D> sum;
#pragma unroll 1
            for (int i = 0; i < q; i += 4) {
                float R1[4], l1[4], v[4][D / 32];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int c = warp + min(i + u, q - 1) * cols;
                    R1[u] = i + u < q ? slots[W * D + c] : -INFINITY;
                    l1[u] = slots[W * (D + 1) + c];
#pragma unroll
                    for (int e = 0; e < D / 32; ++e) v[u][e] = slots[c * D + 32 * e + lane];
                }
                sum.add(R1, l1, v);
            }
            sum.store(kv_out_row(a, chain.z, chain.w, warp, C::kCols, D));
        }
        __syncthreads();
    }
}

}  // namespace zt
