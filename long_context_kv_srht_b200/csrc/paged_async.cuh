// paged_async.cuh -- what the paged attention kernels share on the asynchronous side: mbarrier waits
// with a limit, and tensor maps of the pages.
#pragma once

#include "paged.cuh"
#include "tcgen05.cuh"

namespace pkv {

namespace {

constexpr uint64_t kWaitLimitNs = 2000000000ull;
constexpr uint32_t kNapNs = 20000;

__device__ unsigned long long g_waits_out;   // waits that ran out (one count a source file)

__device__ __forceinline__ uint64_t now_ns() {
    uint64_t t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}

// Waits for the phase of `parity` to complete; false once a wait of this CTA has run out. The
// instruction holds the warp for a while by itself; the rest of a longer wait is out of line (the
// roles' loops have to share the instruction caches) and short (a spinning warp takes issue slots
// and power from the others).
__device__ __noinline__ bool wait_more(uint32_t bar, uint32_t parity, volatile int32_t* abort,
                                       uint64_t limit) {
    uint64_t t0 = 0;
#pragma unroll 1
    for (int i = 1; !mbar_try_wait(bar, parity); ++i) {
        if (i & 127) continue;
        if (*abort) return false;
        const uint64_t t = now_ns();
        if (t0 == 0) t0 = t;
        if (t - t0 > limit) {
            *abort = 1;
            atomicAdd(&g_waits_out, 1ull);
            return false;
        }
    }
    return true;
}
// The same for a warp that is ahead of the others: asleep for up to kNapNs at a time.
__device__ __noinline__ bool nap_more(uint32_t bar, uint32_t parity, volatile int32_t* abort) {
    uint64_t t0 = 0;
#pragma unroll 1
    while (true) {
        uint32_t ok;
        asm volatile(
            "{\n .reg .pred p;\n"
            " mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n"
            " selp.u32 %0, 1, 0, p;\n}\n"
            : "=r"(ok) : "r"(bar), "r"(parity), "r"(kNapNs) : "memory");
        if (ok) return true;
        if (*abort) return false;
        const uint64_t t = now_ns();
        if (t0 == 0) t0 = t;
        if (t - t0 > kWaitLimitNs) {
            *abort = 1;
            atomicAdd(&g_waits_out, 1ull);
            return false;
        }
    }
}
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity, volatile int32_t* abort,
                                         uint64_t limit = kWaitLimitNs) {
    const uint32_t b = smem_addr(bar);
    return mbar_try_wait(b, parity) || wait_more(b, parity, abort, limit);
}
// the same by a whole warp, which goes on together
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity,
                                          volatile int32_t* abort) {
    return __all_sync(0xffffffffu, wait_for(bar, parity, abort));
}
__device__ __forceinline__ bool warp_nap(uint64_t* bar, uint32_t parity, volatile int32_t* abort) {
    const uint32_t b = smem_addr(bar);
    return __all_sync(0xffffffffu, mbar_try_wait(b, parity) || nap_more(b, parity, abort));
}
__device__ __forceinline__ void arrive(uint64_t* bar) { mbar_arrive(smem_addr(bar)); }

// Whether a wait on the current device has run out since this was last asked, after `st`'s work is
// done. The device only counts up and the host remembers how far it has reported, so a wait that
// runs out on another stream meanwhile is never lost, and of two threads one gets the report.
inline cudaError_t take_waits_out(bool* out, cudaStream_t st) {
    static std::atomic<unsigned long long> reported[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    unsigned long long now = 0;
    e = cudaMemcpyFromSymbolAsync(&now, g_waits_out, sizeof(now), 0, cudaMemcpyDeviceToHost, st);
    if (e == cudaSuccess) e = cudaStreamSynchronize(st);
    if (e != cudaSuccess) return e;
    unsigned long long before = reported[dev].load();
    while (before < now && !reported[dev].compare_exchange_weak(before, now)) {}
    *out = before < now;
    return cudaSuccess;
}

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                 const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                 const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiled encode_tiled() {
    static const EncodeTiled fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                             &r) != cudaSuccess ||
            r != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<EncodeTiled>(p);
    }();
    return fn;
}

// a 3-d tensor of rows of 128 elements (bytes or bf16); boxes of `cols` x r1 x r2, their 128-byte
// rows swizzled in shared memory or not
inline bool encode_rows(CUtensorMap* m, const void* base, bool bytes, bool swizzle, uint64_t n1,
                        uint64_t n2, uint64_t s1, uint64_t s2, uint32_t cols, uint32_t r1,
                        uint32_t r2) {
    const EncodeTiled fn = encode_tiled();
    if (!fn) return false;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), n1, n2}, strides[2] = {s1, s2};
    const cuuint32_t box[3] = {cols, r1, r2}, step[3] = {1, 1, 1};
    return fn(m, bytes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
              const_cast<void*>(base), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
              swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace
}  // namespace pkv
