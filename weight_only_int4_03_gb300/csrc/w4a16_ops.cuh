// w4a16_ops.cuh -- what the decode-step operators (rotary append, paged attention, expert layer)
// share beside the GEMM's own headers: status codes of their entry points, argument helpers and a
// few device primitives.  Kept apart from the GEMM's headers so that the GEMM's sources stay as
// they were measured.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "ptx.cuh"
#include "w4a16.h"

namespace w4 {
namespace ops {

constexpr int STAGE_ARG = 1;
constexpr int STAGE_UNSUPPORTED = 2;
constexpr int STAGE_RESOURCE = 3;
constexpr int STAGE_LAUNCH = 6;
constexpr long long HEADER_BYTES = 256; // status word of a workspace
constexpr int MAX_DEVICES = 64;         // devices whose attributes are cached

inline int status_of(int stage, int detail)
{
    return (stage << 16) | (detail & 0xFFFF);
}

inline int launch_status(cudaError_t err)
{
    return err == cudaSuccess ? 0 : status_of(STAGE_LAUNCH, err);
}

inline bool aligned(const void *p, uintptr_t a)
{
    return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

inline long long round_up(long long v, long long a)
{
    return (v + a - 1) / a * a;
}

// Multiprocessors of the current device; cached (a device's count never changes, and two threads
// that race store the same value).
inline cudaError_t sm_count(int *out)
{
    static int cache[MAX_DEVICES];
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess)
        return err;
    if (dev < MAX_DEVICES) {
        const int v = __atomic_load_n(&cache[dev], __ATOMIC_RELAXED);
        if (v > 0) {
            *out = v;
            return cudaSuccess;
        }
    }
    err = cudaDeviceGetAttribute(out, cudaDevAttrMultiProcessorCount, dev);
    if (err == cudaSuccess && dev < MAX_DEVICES)
        __atomic_store_n(&cache[dev], *out, __ATOMIC_RELAXED);
    return err;
}

// Lets kernel `v` of the N of a family use `bytes` of dynamic shared memory on the current device;
// once per device (a second thread that races sets the same value).
template <class Family, int N>
inline cudaError_t allow_smem(const void *kernel, int v, int bytes)
{
    static int done[N][MAX_DEVICES];
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess)
        return err;
    if (dev < MAX_DEVICES && __atomic_load_n(&done[v][dev], __ATOMIC_RELAXED) >= bytes)
        return cudaSuccess;
    err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (err == cudaSuccess && dev < MAX_DEVICES)
        __atomic_store_n(&done[v][dev], bytes, __ATOMIC_RELAXED);
    return err;
}

// Launch with programmatic stream serialisation: the kernel may start while the previous one on
// the stream drains, and waits (pdl_wait) before it touches memory.
template <class... KArgs, class... Args>
inline cudaError_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem,
                              cudaStream_t stream, Args... args)
{
    cudaLaunchConfig_t lc = {};
    lc.gridDim = grid;
    lc.blockDim = block;
    lc.dynamicSmemBytes = smem;
    lc.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    lc.attrs = attr;
    lc.numAttrs = 1;
    return cudaLaunchKernelEx(&lc, kernel, args...);
}

// --- device helpers --------------------------------------------------------------------------

// The 16-bit types by a template switch: BF false = IEEE half, true = bfloat16.
template <bool BF>
__device__ __forceinline__ float to_float(uint16_t b)
{
    return BF ? __bfloat162float(__ushort_as_bfloat16(b)) : __half2float(__ushort_as_half(b));
}

template <bool BF>
__device__ __forceinline__ uint16_t from_float(float x)
{
    return BF ? __bfloat16_as_ushort(__float2bfloat16_rn(x)) : __half_as_ushort(__float2half_rn(x));
}

template <bool BF>
__device__ __forceinline__ float2 unpack2(uint32_t v)
{
    return make_float2(to_float<BF>((uint16_t)v), to_float<BF>((uint16_t)(v >> 16)));
}

template <bool BF>
__device__ __forceinline__ uint32_t pack2(float lo, float hi)
{
    if (BF) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&v);
    }
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// D (f32 16x8) += A (16x16, row) * B (16x8, col).
template <bool BF>
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1)
{
    if (BF)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
            "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
            "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// D (f32 16x8) = A * B.
template <bool BF>
__device__ __forceinline__ void mma16816_zero(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                              uint32_t a3, uint32_t b0, uint32_t b1)
{
    if (BF)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
            "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
            "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ void ldsm_x4_trans(uint32_t addr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

// 16 bytes from global to shared memory, or 16 zero bytes when `live` is false (nothing is then
// read from src).
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool live)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "r"(live ? 16 : 0)
                 : "memory");
}

// The same with constant byte offsets on both sides.
template <int DST, int SRC>
__device__ __forceinline__ void cp_async16_at(uint32_t dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0 + %2], [%1 + %3], 16;" ::"r"(dst), "l"(src), "n"(DST), "n"(SRC)
                 : "memory");
}

__device__ __forceinline__ void cp_async_commit()
{
    asm volatile("cp.async.commit_group;" ::: "memory");
}

template <int N>
__device__ __forceinline__ void cp_async_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// One acquire-release add at GPU scope: what the block stored before its barrier is visible to
// whoever sees the new count, and the last to arrive sees what the others stored.
__device__ __forceinline__ int arrive_counter(int *counter)
{
    int old;
    asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], 1;" : "=r"(old) : "l"(counter) : "memory");
    return old;
}

} // namespace ops
} // namespace w4
