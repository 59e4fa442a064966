// zt_kv.cu -- C ABI of the paged 4-bit KV cache and of attention over it (see
// include/zt_q4.h for the contract of every entry point): argument checks,
// launch shapes and launches.  Every check runs before the first CUDA call.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>

#include "zt_host.h"
#include "attn_tc.cuh"
#include "kv_attn.cuh"
#include "kv_cache.cuh"
#include "zt_q4.h"

namespace {

using namespace zt;

constexpr int kRowsMax = 1 << 24;

int device_error(cudaError_t e, int status)
{
    g_last_cuda_error = e;
    (void)cudaGetLastError();
    return status;
}

size_t page_bytes(int page_size, int kv_heads, int head_dim)
{
    if (page_size < kKvTile || page_size > 1024 || page_size % kKvTile || kv_heads < 1 || kv_heads > 1024) return 0;
    if (head_dim != 64 && head_dim != 96 && head_dim != 128) return 0;
    return (size_t)kv_heads * (page_size / kKvTile) * 18 * head_dim;
}

int check_kv(const zt_q4_kv *kv)
{
    if (!kv || !kv->pages || kv->n_pages < 1) return ZT_ERR_INVALID_ARG;
    if (kv->head_dim != 64 && kv->head_dim != 96 && kv->head_dim != 128) return ZT_ERR_UNSUPPORTED;
    if (!page_bytes(kv->page_size, kv->kv_heads, kv->head_dim)) return ZT_ERR_INVALID_ARG;
    if (!aligned(kv->pages, 16) || !aligned(kv->err, 4)) return ZT_ERR_MISALIGNED;
    return ZT_OK;
}

// a page table whose positions fit in int
int check_table(const int32_t *table, int n_seqs, int max_pages, int page_size)
{
    if (!table || n_seqs < 1 || max_pages < 1 || (int64_t)max_pages * page_size > INT_MAX) return ZT_ERR_INVALID_ARG;
    return aligned(table, 4) ? ZT_OK : ZT_ERR_MISALIGNED;
}

int check_rows(const zt_q4_kv *kv, const zt_q4_kv_rows *rows)
{
    if (!rows || rows->n < 0 || rows->n > kRowsMax) return ZT_ERR_INVALID_ARG;
    if (rows->n && (!rows->seq || !rows->pos)) return ZT_ERR_INVALID_ARG;
    if (!aligned(rows->seq, 4) || !aligned(rows->pos, 4)) return ZT_ERR_MISALIGNED;
    return check_table(rows->page_table, rows->n_seqs, rows->max_pages, kv->page_size);
}

// fp16 rows read and written 16 bytes at a time; null is fine where there are none
int check_matrix(const void *p, int ld, int64_t width, int rows = 1)
{
    if ((!p && rows) || ld < width) return ZT_ERR_INVALID_ARG;
    return aligned(p, 16) && ld % 8 == 0 ? ZT_OK : ZT_ERR_MISALIGNED;
}

// softmax scales whose products with a score, and whose reciprocals, stay finite
bool scale_ok(float scale) { return scale >= 0x1p-64f && scale <= 0x1p64f; }

KvPlaces places(const zt_q4_kv *kv, const int32_t *table, int n_seqs, int max_pages)
{
    KvPlaces p;
    p.pages = static_cast<unsigned char *>(kv->pages);
    p.page_bytes = (long long)page_bytes(kv->page_size, kv->kv_heads, kv->head_dim);
    p.n_pages = kv->n_pages;
    p.page_size = kv->page_size;
    p.kv_heads = kv->kv_heads;
    p.table = table;
    p.n_seqs = n_seqs;
    p.max_pages = max_pages;
    p.err = kv->err;
    return p;
}

const __half *h(const uint16_t *p) { return reinterpret_cast<const __half *>(p); }
__half *h(uint16_t *p) { return reinterpret_cast<__half *>(p); }

// Launch with programmatic dependent launch: the kernel may start while the one ahead of it on the
// stream ends; it waits for it before it reads anything.
template <typename Args>
int launch(void (*fn)(Args), dim3 grid, int threads, size_t smem, const Args &args, void *stream)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    clear_stale_error();
    const cudaError_t e = cudaLaunchKernelEx(&cfg, fn, args);
    return e == cudaSuccess ? ZT_OK : device_error(e, ZT_ERR_LAUNCH);
}

// CTAs per row or window: few leave most SMs idle, so the items of each are spread until the grid covers the device
// about twice.  (Rows are not spread further: each CTA of a row computes its angles.)
int spread(int parts, int items, int threads)
{
    const int most = std::max(1, (items + threads - 1) / threads);
    return std::max(1, std::min(most, 2 * 148 / std::max(1, parts) + 1));
}

// Grid of an append or a gather: CTAs by row, then by window of rows.
template <typename Args>
int launch_rows(void (*fn)(Args), Args &a, int threads, int row_items, int group_items, void *stream)
{
    const int windows = (a.rows + kKvWindow - 1) / kKvWindow;
    a.row_ctas = spread(a.rows, row_items, threads);
    // Windows have no angles: up to eight times as many CTAs.  Appending and reading back as in kv_cache.cuh, with 256
    // threads: 37.1 and 22.7 us, with these 38.6 and 17.9; a CTA per window 66.4 (windows last) and 26.8.
    a.v_ctas = spread(windows / 8, group_items * 4 * std::min(a.rows, 4), threads);
    const int64_t grid = (int64_t)a.rows * a.row_ctas + (int64_t)windows * a.v_ctas;
    return launch(fn, dim3((unsigned)grid), threads, 0, a, stream);
}

constexpr size_t kArrivedBytes = 1024;     // counters at the workspace's start
static_assert(kArrivedBytes >= kKvMaxCtas * sizeof(unsigned), "one counter per CTA");

size_t part_bytes(int head_dim)
{
    return kArrivedBytes + (size_t)kKvMaxCtas * 2 * 8 * (head_dim + 2) * sizeof(float);
}

// Segments of at most this many tokens (as far as the page table reaches), one wave of them: a CTA takes one
// each, and nothing goes through the workspace.  One sequence, 32 kv heads of 96, whole and split: 100 tokens
// 5.8 and 11.4 us, 517 8.2 and 11.2, 1000 9.2 and 11.6, 2000 13.3 and 12.9; 8 kv heads of 128 with 4 query heads
// each: 1000 tokens 10.5 and 12.6, 2000 tokens 15.3 and 13.2.
constexpr int kWholeTokens = 1024;

template <int D>
int launch_attention(KvAttnArgs &a, void *stream)
{
    using C = KvAttnCfg<D>;
    a.blocks = (a.cols + C::kCols - 1) / C::kCols;
    const int64_t segments = (int64_t)a.at.n_seqs * a.at.kv_heads * a.blocks;
    if (segments * ((int64_t)a.at.max_pages * (a.at.page_size / kKvTile) + kKvSegTiles) > INT_MAX) return ZT_ERR_UNSUPPORTED;
    const size_t index = (2 * (size_t)a.at.n_seqs + 1) * sizeof(int);
    int sms = 0;
    if (resident_ctas(reinterpret_cast<const void *>(&kv_attn_kernel<D>), C::kWarps * 32, C::kSmem + index, sms) < 1)
        return ZT_ERR_DEVICE;
    const int longest = a.at.max_pages * a.at.page_size;
    a.whole = segments <= sms && longest <= kWholeTokens;
    const int ctas = a.whole ? (int)segments : std::min(sms, kKvMaxCtas);
    return launch(kv_attn_kernel<D>, dim3((unsigned)ctas), C::kWarps * 32, C::kSmem + index, a, stream);
}

// fp16 [tokens][heads][D] with rows ld elements apart, boxes of 64 columns x 1 head x 128 tokens, 128-byte
// swizzle; columns and tokens out of range read as zero.
bool tma_map_heads(CUtensorMap *map, const uint16_t *base, int D, int heads, int64_t tokens, int ld)
{
    PFN_cuTensorMapEncodeTiled_v12000 enc = tma_encoder();
    if (!enc) return false;
    cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)tokens};
    cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)ld * 2};
    cuuint32_t box[3] = {64, 1, kAttnRows};
    cuuint32_t estr[3] = {1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<uint16_t *>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Where the items of one query tile fill at most half of the SMs, the keys of an item are split between the CTAs of a
// cluster (2, 4 or 8), at least this many (of the average sequence) to each.  Whole and split: 137 queries, 2724 keys, 32
// heads of 96, 40.4 and 26.9 us; 20 queries, 32020 keys, 32 heads of 128, 406 and 105; 64 queries, 32 heads, 1064 keys 20.3
// and 14.7, 564 keys 13.5 and 12.3; 64 queries, 8 heads, 464 keys 11.7 and 11.9.  With 256 and 512 keys at least: 964 keys
// of 8 heads 14.9 and 18.0, with 128 11.3.
constexpr int kSplitKeys = 128;

template <int D>
int launch_prompt(PromptArgs &a, const uint16_t *q, int ld_q, const uint16_t *k, int ld_k, const uint16_t *v, int ld_v,
                  void *stream)
{
    using C = PromptCfg<D>;
    int sms = 0;
    if (resident_ctas(reinterpret_cast<const void *>(&prompt_attn_kernel<D, false>), kAttnThreads, C::kSmem, sms) < 1 ||
        resident_ctas(reinterpret_cast<const void *>(&prompt_attn_kernel<D, true>), kAttnThreads, C::kSmem, sms) < 1)
        return ZT_ERR_DEVICE;
    const int kv_heads = a.q_heads / a.group;
    CUtensorMap mq, mk, mv;
    if (a.total_k == 0) {             // no keys are read: any valid map will do
        k = v = q;
        ld_k = ld_v = ld_q;
    }
    const int64_t keys = std::max(a.total_k, 1);
    if (!tma_map_heads(&mq, q, D, a.q_heads, a.total_q, ld_q) || !tma_map_heads(&mk, k, D, kv_heads, keys, ld_k) ||
        !tma_map_heads(&mv, v, D, kv_heads, keys, ld_v))
        return ZT_ERR_DEVICE;
    // One query tile per CTA while two would leave SMs without work.  Causal, 32 heads of 128, one and two tiles:
    // 129 tokens 9.0 and 10.1 us, 512 13.8 and 15.1, 900 (4 x 32 items of two) 23.8 and 23.0, 1100 (5 x 32) 26.8
    // and 23.7, 2048 64.2 and 42.0.
    auto items = [&](int tiles) {
        return ((int64_t)a.total_q + tiles * kAttnRows - 1) / (tiles * kAttnRows) * a.q_heads;
    };
    a.tiles = items(2) < sms ? 1 : 2;
    // Every sequence may end with a partial block; CTAs without an item end at once.
    int64_t grid = items(a.tiles) + (int64_t)(a.n_seqs - 1) * a.q_heads;
    a.splits = 1;
    while (a.splits < kAttnSplits && grid * a.splits * 2 <= sms && keys >= (int64_t)a.n_seqs * a.splits * 2 * kSplitKeys) a.splits *= 2;
    grid *= a.splits;
    if (grid > INT_MAX) return ZT_ERR_UNSUPPORTED;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kAttnThreads);
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)a.splits;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = a.splits > 1 ? 2 : 1;
    clear_stale_error();
    const cudaError_t e = cudaLaunchKernelEx(&cfg, a.splits > 1 ? prompt_attn_kernel<D, true> : prompt_attn_kernel<D, false>, mq, mk, mv, (const PromptArgs &)a);
    return e == cudaSuccess ? ZT_OK : device_error(e, ZT_ERR_LAUNCH);
}

}  // namespace

extern "C" {

size_t zt_q4_kv_page_bytes(int page_size, int kv_heads, int head_dim) { return page_bytes(page_size, kv_heads, head_dim); }

int zt_q4_kv_append(const zt_q4_kv *kv, const zt_q4_kv_rows *rows, const uint16_t *k, int ld_k, const uint16_t *v,
                    int ld_v, const zt_q4_kv_rope *rope, void *stream)
{
    int rc = check_kv(kv);
    if (!rc) rc = check_rows(kv, rows);
    if (rc) return rc;
    const int64_t width = (int64_t)kv->kv_heads * kv->head_dim;
    if ((rc = check_matrix(k, ld_k, width, rows->n)) || (rc = check_matrix(v, ld_v, width, rows->n))) return rc;
    if (rope) {
        if (!(rope->theta > 0.f) || rope->theta > 3.0e38f) return ZT_ERR_INVALID_ARG;
        if (rope->q) {
            if (rope->q_heads < 1 || rope->q_heads > 16384) return ZT_ERR_INVALID_ARG;
            const int64_t qw = (int64_t)rope->q_heads * kv->head_dim;
            if ((rc = check_matrix(rope->q, rope->ld_q, qw)) || (rc = check_matrix(rope->q_out, rope->ld_q_out, qw)))
                return rc;
            if (rope->q_out == rope->q) return ZT_ERR_INVALID_ARG;
        } else if (rope->q_out) {
            return ZT_ERR_INVALID_ARG;
        }
        if (rope->k_out && (rc = check_matrix(rope->k_out, rope->ld_k_out, width))) return rc;
        if (rope->k_out && rope->k_out == k) return ZT_ERR_INVALID_ARG;
    }
    if (rows->n == 0) return ZT_OK;
    KvAppendArgs a = {};
    a.at = places(kv, rows->page_table, rows->n_seqs, rows->max_pages);
    a.seq = rows->seq;
    a.pos = rows->pos;
    a.k = h(k);
    a.v = h(v);
    a.ld_k = ld_k;
    a.ld_v = ld_v;
    if (rope) {
        a.rope = 1;
        a.q = h(rope->q);
        a.q_out = h(rope->q_out);
        a.k_out = h(rope->k_out);
        a.ld_q = rope->ld_q;
        a.ld_q_out = rope->ld_q_out;
        a.ld_k_out = rope->ld_k_out;
        a.q_heads = rope->q ? rope->q_heads : 0;
        for (int i = 0; i < kv->head_dim / 2; ++i) a.freq[i] = std::pow((double)rope->theta, -2.0 * i / kv->head_dim);
    }
    a.rows = rows->n;
    const int row_items = (kv->kv_heads + a.q_heads) * kv->head_dim / 8, groups = kv->kv_heads * kv->head_dim / 32;
    if (kv->head_dim == 64) return launch_rows(kv_append_kernel<64>, a, kAppendThreads, row_items, groups, stream);
    if (kv->head_dim == 96) return launch_rows(kv_append_kernel<96>, a, kAppendThreads, row_items, groups, stream);
    return launch_rows(kv_append_kernel<128>, a, kAppendThreads, row_items, groups, stream);
}

int zt_q4_kv_gather(const zt_q4_kv *kv, const zt_q4_kv_rows *rows, uint16_t *k, int ld_k, uint16_t *v, int ld_v,
                    void *stream)
{
    int rc = check_kv(kv);
    if (!rc) rc = check_rows(kv, rows);
    if (rc) return rc;
    const int64_t width = (int64_t)kv->kv_heads * kv->head_dim;
    if ((rc = check_matrix(k, ld_k, width, rows->n)) || (rc = check_matrix(v, ld_v, width, rows->n))) return rc;
    if (rows->n == 0) return ZT_OK;
    KvGatherArgs a = {};
    a.at = places(kv, rows->page_table, rows->n_seqs, rows->max_pages);
    a.seq = rows->seq;
    a.pos = rows->pos;
    a.k = h(k);
    a.v = h(v);
    a.ld_k = ld_k;
    a.ld_v = ld_v;
    a.rows = rows->n;
    const int row_items = kv->kv_heads * kv->head_dim / 8, groups = kv->kv_heads * kv->head_dim / 32;
    if (kv->head_dim == 64) return launch_rows(kv_gather_kernel<64>, a, kGatherThreads, row_items, groups, stream);
    if (kv->head_dim == 96) return launch_rows(kv_gather_kernel<96>, a, kGatherThreads, row_items, groups, stream);
    return launch_rows(kv_gather_kernel<128>, a, kGatherThreads, row_items, groups, stream);
}

int zt_q4_kv_copy_pages(const zt_q4_kv *kv, const int32_t *src, const int32_t *dst, int n, int layers,
                        size_t layer_bytes, void *stream)
{
    const int rc = check_kv(kv);
    if (rc) return rc;
    if (n < 0 || n > kRowsMax || layers < 1 || layers > 65535) return ZT_ERR_INVALID_ARG;
    if (n && (!src || !dst)) return ZT_ERR_INVALID_ARG;
    const size_t bytes = page_bytes(kv->page_size, kv->kv_heads, kv->head_dim);
    if (layers > 1 && layer_bytes < bytes * (size_t)kv->n_pages) return ZT_ERR_INVALID_ARG;
    if (!aligned(src, 4) || !aligned(dst, 4) || (layers > 1 && layer_bytes % 16)) return ZT_ERR_MISALIGNED;
    if (n == 0) return ZT_OK;
    KvCopyArgs a = {};
    a.pages = static_cast<unsigned char *>(kv->pages);
    a.page_bytes = (long long)bytes;
    a.layer_bytes = (long long)layer_bytes;
    a.n_pages = kv->n_pages;
    a.src = src;
    a.dst = dst;
    a.err = kv->err;
    // 16 KB per CTA (256 threads x 4 loads of 16 bytes) until the pages are covered: 3 pages of 147 KB in 32 layers
    // 2.9 us, 97 of 221 KB 207.5 (6.62 TB/s read and written); with 64 KB per CTA 3.5 and 211.6
    const unsigned per_page = (unsigned)std::max<size_t>(1, (bytes + 16383) / 16384);
    return launch(kv_copy_kernel, dim3((unsigned)n, per_page, (unsigned)layers), 256, 0, a, stream);
}

size_t zt_q4_kv_attention_workspace_bytes(int kv_heads, int q_heads, int head_dim, int tokens)
{
    if (kv_heads < 1 || q_heads < kv_heads || q_heads % kv_heads || q_heads > 16384 || tokens < 1 || tokens > 16) return 0;
    if (head_dim != 64 && head_dim != 96 && head_dim != 128) return 0;
    return part_bytes(head_dim);
}

int zt_q4_kv_attention(const zt_q4_kv *kv, const uint16_t *q, int ld_q, int q_heads, int tokens, const int32_t *lens,
                       const int32_t *page_table, int n_seqs, int max_pages, float scale, uint16_t *out, int ld_out,
                       void *workspace, size_t ws_bytes, void *stream)
{
    int rc = check_kv(kv);
    if (!rc) rc = check_table(page_table, n_seqs, max_pages, kv->page_size);
    if (rc) return rc;
    if (!lens || !out || !workspace || n_seqs > ZT_Q4_KV_MAX_SEQS || tokens < 1 || tokens > 16) return ZT_ERR_INVALID_ARG;
    if (q_heads < kv->kv_heads || q_heads % kv->kv_heads || q_heads > 16384) return ZT_ERR_INVALID_ARG;
    if (!scale_ok(scale)) return ZT_ERR_INVALID_ARG;
    const int64_t width = (int64_t)q_heads * kv->head_dim;
    if ((rc = check_matrix(q, ld_q, width))) return rc;
    if (ld_out < width) return ZT_ERR_INVALID_ARG;
    if (!aligned(out, 2) || !aligned(lens, 4) || !aligned(workspace, 16)) return ZT_ERR_MISALIGNED;
    if (ws_bytes < zt_q4_kv_attention_workspace_bytes(kv->kv_heads, q_heads, kv->head_dim, tokens)) return ZT_ERR_WORKSPACE;
    KvAttnArgs a = {};
    a.at = places(kv, page_table, n_seqs, max_pages);
    a.q = h(q);
    a.out = h(out);
    a.lens = lens;
    a.arrived = static_cast<unsigned int *>(workspace);
    a.part = reinterpret_cast<float *>(static_cast<unsigned char *>(workspace) + kArrivedBytes);
    a.ld_q = ld_q;
    a.ld_out = ld_out;
    a.tokens = tokens;
    a.q_heads = q_heads;
    a.group = q_heads / kv->kv_heads;
    a.cols = a.group * tokens;
    a.scale_log2 = scale * 1.4426950408889634f;
    if (kv->head_dim == 64) return launch_attention<64>(a, stream);
    if (kv->head_dim == 96) return launch_attention<96>(a, stream);
    return launch_attention<128>(a, stream);
}

int zt_q4_prompt_attention(const uint16_t *q, int ld_q, const uint16_t *k, int ld_k, const uint16_t *v, int ld_v,
                           const int32_t *cu_q, const int32_t *cu_k, int n_seqs, int total_q, int total_k, int q_heads,
                           int kv_heads, int head_dim, int causal, float scale, uint16_t *out, int ld_out, uint32_t *err,
                           void *stream)
{
    if (!cu_q || !cu_k || n_seqs < 1 || n_seqs > ZT_Q4_KV_MAX_SEQS || total_q < 0 || total_q > kRowsMax || total_k < 0 ||
        total_k > kRowsMax)
        return ZT_ERR_INVALID_ARG;
    if (kv_heads < 1 || kv_heads > 1024 || q_heads < kv_heads || q_heads % kv_heads || q_heads > 16384) return ZT_ERR_INVALID_ARG;
    if (head_dim != 64 && head_dim != 96 && head_dim != 128) return ZT_ERR_UNSUPPORTED;
    if ((causal != 0 && causal != 1) || !scale_ok(scale)) return ZT_ERR_INVALID_ARG;
    const int64_t qw = (int64_t)q_heads * head_dim, kw = (int64_t)kv_heads * head_dim;
    int rc;
    if (!aligned(cu_q, 4) || !aligned(cu_k, 4) || !aligned(err, 4)) return ZT_ERR_MISALIGNED;
    if (total_q && ((rc = check_matrix(q, ld_q, qw)) || (rc = check_matrix(out, ld_out, qw)))) return rc;
    if (total_k && ((rc = check_matrix(k, ld_k, kw)) || (rc = check_matrix(v, ld_v, kw)))) return rc;
    if (total_q == 0) return ZT_OK;
    PromptArgs a = {};
    a.out = h(out);
    a.ld_out = ld_out;
    a.cu_q = cu_q;
    a.cu_k = cu_k;
    a.n_seqs = n_seqs;
    a.total_q = total_q;
    a.total_k = total_k;
    a.q_heads = q_heads;
    a.group = q_heads / kv_heads;
    a.causal = causal;
    a.scale_log2 = scale * 1.4426950408889634f;
    a.err = err;
    if (head_dim == 64) return launch_prompt<64>(a, q, ld_q, k, ld_k, v, ld_v, stream);
    if (head_dim == 96) return launch_prompt<96>(a, q, ld_q, k, ld_k, v, ld_v, stream);
    return launch_prompt<128>(a, q, ld_q, k, ld_k, v, ld_v, stream);
}

int zt_q4_kv_errors(const uint32_t *err, unsigned int *out)
{
    if (!err || !out) return ZT_ERR_INVALID_ARG;
    const cudaError_t e = cudaMemcpy(out, err, sizeof(unsigned int), cudaMemcpyDeviceToHost);
    return e == cudaSuccess ? ZT_OK : device_error(e, ZT_ERR_DEVICE);
}

}  // extern "C"
