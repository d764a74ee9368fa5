// The global norm of many gradient tensors, and their clipping by it (gfx950).
//
//   norm = sqrt(sum over all tensors of g^2),  g' = g min(1, max_norm / (norm + 1e-6))
//
// Bound by memory: every value is read for the norm, and read and written again once
// the norm is known.  The tensors' addresses travel in the kernel's arguments, so a
// call copies no table and a captured graph holds its own.
#include "block8.hpp"
#include "common.hpp"
#include "kernels.hpp"

namespace moe {

#pragma clang fp contract(off)

constexpr int kGradThreads = 256;

// First element, count and tensor of chunk c, c ascending from call to call.
__device__ __forceinline__ void grad_chunk(const GradList& a, int64_t c, int& i, int64_t& first, int& count) {
    while (i + 1 < a.n && c >= a.first[i + 1]) ++i;
    first = (c - a.first[i]) * a.chunk;
    const int64_t left = (int64_t)(a.count[i] & ~kGradBf16) - first;
    count = left < a.chunk ? (int)left : a.chunk;
}

// Squares are summed in 64 bits: those of fp32 values do not overflow there, and the
// sum of 10^9 values keeps fp32's precision.  The conversions and additions run at a
// quarter of the load rate's need.
__device__ __forceinline__ double square(float v) { return (double)v * (double)v; }

// Workgroup b sums chunks b, b + grid, ... into its own slot; the last one to finish
// (of a call's last launch) adds all slots in ascending order.
__global__ __launch_bounds__(kGradThreads) void grad_norm_kernel(GradList a, double* partial, int slot0, int slots,
                                                                 int* counter, float* norm) {
    __shared__ double s_sum[kGradThreads / kWave];
    __shared__ int s_last;
    double sum0 = 0.0, sum1 = 0.0;
    int i = 0;
    for (int64_t c = blockIdx.x; c < a.first[a.n]; c += gridDim.x) {
        int64_t first;
        int count;
        grad_chunk(a, c, i, first, count);
        if (a.count[i] & kGradBf16) {
            const uint16_t* g = (const uint16_t*)a.src[i] + first;
            const int whole = ((uintptr_t)g & 15) == 0 ? count & ~7 : 0;
            for (int x = threadIdx.x * 8; x < whole; x += kGradThreads * 8) {
                const intx4 raw = *(const intx4*)(g + x);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    sum0 += square(__builtin_bit_cast(float, (uint32_t)raw[q] << 16));
                    sum1 += square(__builtin_bit_cast(float, (uint32_t)raw[q] & 0xffff0000u));
                }
            }
            for (int x = whole + threadIdx.x; x < count; x += kGradThreads) sum0 += square(bf16_to_f32(g[x]));
        } else {
            const float* g = (const float*)a.src[i] + first;
            const int whole = ((uintptr_t)g & 15) == 0 ? count & ~3 : 0;
#pragma unroll 4
            for (int x = threadIdx.x * 4; x < whole; x += kGradThreads * 4) {
                const floatx4 v = *(const floatx4*)(g + x);
                sum0 += square(v[0]);
                sum1 += square(v[1]);
                sum0 += square(v[2]);
                sum1 += square(v[3]);
            }
            for (int x = whole + threadIdx.x; x < count; x += kGradThreads) sum0 += square(g[x]);
        }
    }
    auto joined = [&](double v) {  // over the workgroup, in a fixed order
#pragma unroll
        for (int s = 1; s < kWave; s *= 2) v += __shfl_xor(v, s, kWave);
        if ((threadIdx.x & 63) == 0) s_sum[threadIdx.x >> 6] = v;
        __syncthreads();
        return ((s_sum[0] + s_sum[1]) + s_sum[2]) + s_sum[3];
    };
    const double sum = joined(sum0 + sum1);
    if (threadIdx.x == 0) {
        __hip_atomic_store(partial + slot0 + blockIdx.x, sum, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        s_last = 0;
        if (norm) {  // the store has reached memory before the workgroup counts in
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            const int before = __hip_atomic_fetch_add(counter, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            if (before == (int)gridDim.x - 1) {
                __hip_atomic_store(counter, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);  // for the next call
                s_last = 1;
            }
        }
    }
    __syncthreads();
    if (!s_last) return;
    double all = 0.0;
    for (int x = threadIdx.x; x < slots; x += kGradThreads)
        all += __hip_atomic_load(partial + x, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    all = joined(all);
    if (threadIdx.x == 0) *norm = (float)sqrt(all);
}

// A NaN norm makes every gradient NaN, an infinite one zero (infinite ones NaN).
__global__ __launch_bounds__(kGradThreads) void grad_clip_kernel(GradList a, const float* norm, float max_norm) {
    const double ratio = (double)max_norm / ((double)*norm + 1e-6);
    const float coef = ratio >= 1.0 ? 1.0f : (float)ratio;
    int i = 0;
    for (int64_t c = blockIdx.x; c < a.first[a.n]; c += gridDim.x) {
        int64_t first;
        int count;
        grad_chunk(a, c, i, first, count);
        if (a.src[i] == a.dst[i] && coef == 1.0f) continue;  // in place and within the bound
        if (a.count[i] & kGradBf16) {
            const uint16_t* g = (const uint16_t*)a.src[i] + first;
            uint16_t* o = (uint16_t*)a.dst[i] + first;
            const int whole = (((uintptr_t)g | (uintptr_t)o) & 15) == 0 ? count & ~7 : 0;
            for (int x = threadIdx.x * 8; x < whole; x += kGradThreads * 8) {
                float v[8];
                unpack_bf16x8(*(const intx4*)(g + x), v);
#pragma unroll
                for (int y = 0; y < 8; ++y) v[y] *= coef;
                *(intx4*)(o + x) = pack_bf16x8(v);
            }
            for (int x = whole + threadIdx.x; x < count; x += kGradThreads)
                o[x] = (uint16_t)pack_bf16x2(bf16_to_f32(g[x]) * coef, 0.0f);
        } else {
            const float* g = (const float*)a.src[i] + first;
            float* o = (float*)a.dst[i] + first;
            const int whole = (((uintptr_t)g | (uintptr_t)o) & 15) == 0 ? count & ~3 : 0;
#pragma unroll 4
            for (int x = threadIdx.x * 4; x < whole; x += kGradThreads * 4) {
                floatx4 v = *(const floatx4*)(g + x);
#pragma unroll
                for (int y = 0; y < 4; ++y) v[y] *= coef;
                *(floatx4*)(o + x) = v;
            }
            for (int x = whole + threadIdx.x; x < count; x += kGradThreads) o[x] = g[x] * coef;
        }
    }
}

// Fills the chunks' size and bounds; returns how many there are.  16384 elements, less
// where that gives too few to spread over the CUs.
static int64_t grad_chunks(GradList& a) {
    uint64_t all = 0;
    for (int i = 0; i < a.n; ++i) all += a.count[i] & ~kGradBf16;
    a.chunk = 16384;
    while (a.chunk > 1024 && all / a.chunk < 1024) a.chunk /= 2;
    a.first[0] = 0;
    for (int i = 0; i < a.n; ++i)
        a.first[i + 1] = a.first[i] + ((int64_t)(a.count[i] & ~kGradBf16) + a.chunk - 1) / a.chunk;
    return a.first[a.n];
}

int launch_grad_norm(GradList a, double* partial, int slot0, bool last, int* counter, float* norm, hipStream_t stream) {
    const int64_t chunks = grad_chunks(a);
    const int grid = (int)(chunks < 1 ? 1 : chunks < kGradSlots ? chunks : kGradSlots);
    hipLaunchKernelGGL(grad_norm_kernel, dim3(grid), dim3(kGradThreads), 0, stream, a, partial, slot0, slot0 + grid,
                       counter, last ? norm : nullptr);
    return slot0 + grid;
}

void launch_grad_clip(GradList a, const float* norm, float max_norm, hipStream_t stream) {
    const int64_t chunks = grad_chunks(a);
    if (chunks == 0) return;
    hipLaunchKernelGGL(grad_clip_kernel, dim3((unsigned)(chunks < 4096 ? chunks : 4096)), dim3(kGradThreads), 0, stream, a,
                       norm, max_norm);
}

}  // namespace moe
