// zt_host.cu -- host helpers shared by the C ABI's translation units (zt_host.h).
#include "zt_host.h"

#include <functional>
#include <mutex>
#include <unordered_map>

#include "zt_q4.h"

namespace zt {

thread_local cudaError_t g_last_cuda_error = cudaSuccess;

namespace {

struct OccKey {
    const void *fn;
    int dev, threads;
    size_t smem;
    bool operator==(const OccKey &o) const
    {
        return fn == o.fn && dev == o.dev && threads == o.threads && smem == o.smem;
    }
};
struct OccHash {
    size_t operator()(const OccKey &k) const
    {
        return std::hash<const void *>()(k.fn) ^ (size_t)k.dev * 131 ^ (size_t)k.threads * 7919 ^
               k.smem * 104729;
    }
};

std::mutex g_mu;   // guards the tables below
std::unordered_map<OccKey, int, OccHash> g_occ;   // resident CTAs per SM, or -1 if unusable
std::unordered_map<int, int> g_sms;               // device -> SM count

std::unordered_map<uint64_t, bool> g_optin;      // (kernel, device) opted in to the max smem

}  // namespace

int launch_status()
{
    const cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) return ZT_OK;
    g_last_cuda_error = e;
    return ZT_ERR_LAUNCH;
}

int resident_ctas(const void *fn, int threads, size_t smem, int &sms)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) {
        g_last_cuda_error = e;
        return -1;
    }
    std::lock_guard<std::mutex> lk(g_mu);
    auto it_s = g_sms.find(dev);
    if (it_s == g_sms.end()) {
        int n = 0;
        e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess || n < 1) {
            g_last_cuda_error = e;
            return -1;
        }
        it_s = g_sms.emplace(dev, n).first;
    }
    sms = it_s->second;
    const uint64_t fkey = (uint64_t)(uintptr_t)fn * 64u + (uint64_t)dev;
    if (g_optin.find(fkey) == g_optin.end()) {
        int optin = 0;
        e = cudaDeviceGetAttribute(&optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
        if (e == cudaSuccess) e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, optin);
        if (e != cudaSuccess) {
            g_last_cuda_error = e;
            (void)cudaGetLastError();
            return -1;
        }
        g_optin.emplace(fkey, true);
    }
    OccKey key{fn, dev, threads, smem};
    auto it = g_occ.find(key);
    if (it != g_occ.end()) return it->second;
    int nb = 0;
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&nb, fn, threads, smem);
    if (e != cudaSuccess) {
        g_last_cuda_error = e;
        (void)cudaGetLastError();
        return -1;
    }
    g_occ.emplace(key, nb > 0 ? nb : -1);
    return nb > 0 ? nb : -1;
}

PFN_cuTensorMapEncodeTiled_v12000 tma_encoder()
{
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        cudaDriverEntryPointQueryResult q;
        void *p = nullptr;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
        (void)cudaGetLastError();
    });
    return fn;
}

}  // namespace zt
