// kv_common.cuh -- layout of the paged 4-bit KV cache (include/zt_q4.h, zt_q4_kv)
// and small device helpers of the kernels that read and write it.
#pragma once

#include <cuda_fp16.h>
#include <cstdint>

#include "tc_common.cuh"

namespace zt {

constexpr int kKvTile = 16;               // tokens per tile: one k or m extent of the decode kernel's mma
constexpr unsigned kErrKvPlace = 1u;      // a page index, position or sequence out of range
constexpr unsigned kErrKvWait = 2u;       // a bounded wait ran out
constexpr unsigned kErrKvWork = 4u;       // a workspace that was not zero-filled before its first use

// One kv head's tile: K codes | V codes | K scales | V scales.
template <int D>
struct KvTile {
    static constexpr int kG = D / 32;                 // scales per token
    static constexpr int kCodes = kKvTile * D / 2;    // bytes of K (or V) codes
    static constexpr int kScales = kKvTile * kG * 2;  // bytes of K (or V) scales
    static constexpr int kV = kCodes, kKs = 2 * kCodes, kVs = 2 * kCodes + kScales;
    static constexpr int kBytes = 2 * (kCodes + kScales);   // 18 D
    static_assert(kBytes % 16 == 0, "bulk copies move multiples of 16 bytes");
};

// Where pages, sequences and positions are; every index into it is checked on the device.
struct KvPlaces {
    unsigned char *pages;
    long long page_bytes;
    int n_pages, page_size, kv_heads;
    const int32_t *table;      // [n_seqs][max_pages]
    int n_seqs, max_pages;
    unsigned int *err;         // or null
};

__device__ __forceinline__ void kv_error(unsigned int *err, unsigned bit)
{
    if (err) atomicOr(err, bit);
}

__device__ __forceinline__ uint32_t kv_smem(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void kv_pdl_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void kv_pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

__device__ __forceinline__ uint32_t h2_bits(__half2 h) { return *reinterpret_cast<uint32_t *>(&h); }
__device__ __forceinline__ __half2 bits_h2(uint32_t v) { return *reinterpret_cast<__half2 *>(&v); }

// Two fp32 values in a 64-bit register.
__device__ __forceinline__ uint64_t f2_pack(float a, float b)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 f2_split(uint64_t v)
{
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ uint64_t f2_fma(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

}  // namespace zt
