// The global norm of many gradient tensors, and their clipping by it (gfx950).
//
//   norm = sqrt(sum over all tensors of g^2),  g' = g min(1, max_norm / (norm + 1e-6))
//
// Bound by memory: every value is read for the norm, and read and written again once
// the norm is known.  Tensors that are not 16-byte aligned go element by element, for one
// of 4.7e8 values: norm of fp32 276 -> 918 us, of bf16 232 -> 852, clip 637 -> 799 and 300
// -> 698.  The tensors' addresses travel in the kernel's arguments, so a
// call copies no table and a captured graph holds its own.
#include "block8.hpp"
#include "common.hpp"
#include "kernels.hpp"

namespace moe {

#pragma clang fp contract(off)

constexpr int kGradThreads = 256;
constexpr int kGradUnroll = 4;  // 16-byte loads of a thread in flight

// Where chunk c lies: tensor i, its first element there and how many.  The number of
// tensors that end at or before c, counted by the wave: a search would be a chain of
// loads at the start of every workgroup.
struct GradChunk {
    int i, count;
    int64_t first;
};
__device__ __forceinline__ GradChunk grad_chunk(const GradList& a, int64_t c) {
    const int lane = threadIdx.x & 63;
    static_assert(kGradTensors <= 2 * kWave, "two counts");
    int i = __popcll(__ballot(lane < a.n && a.first[lane + 1] <= c));
    if (a.n > kWave) i += __popcll(__ballot(kWave + lane < a.n && a.first[min(kWave + lane + 1, kGradTensors)] <= c));
    GradChunk r;
    r.i = i;
    r.first = (c - a.first[i]) * a.chunk;
    const int64_t left = (int64_t)(a.count[i] & ~kGradBf16) - r.first;
    r.count = left < a.chunk ? (int)left : a.chunk;
    return r;
}

// The norm's squares are summed in 64 bits: those of fp32 values do not overflow there,
// and the sum of 10^9 values keeps fp32's precision.  A CU converts and adds four times
// as fast as it can be fed.
__device__ __forceinline__ double square(float v) { return (double)v * (double)v; }

// Loads and stores leave the caches to others: what passes through is not read again
// soon.  1.4e9 fp32 values: norm 985 -> 905 us, clip 1980 -> 1950 us with such loads and
// 1900 with such stores too.
__device__ __forceinline__ intx4 grad_load(const void* p) { return __builtin_nontemporal_load((const intx4*)p); }
__device__ __forceinline__ void grad_store(void* p, intx4 v) { __builtin_nontemporal_store(v, (intx4*)p); }

struct GradSums {
    double a, b;
};
template <bool kBf16>
__device__ __forceinline__ GradSums grad_squares(const void* src, const GradChunk& k) {
    constexpr int kSize = kBf16 ? 2 : 4, kPer = 16 / kSize;
    const char* g = (const char*)src + k.first * kSize;
    const int whole = ((uintptr_t)g & 15) == 0 ? k.count / kPer : 0;  // vectors
    GradSums s{0.0, 0.0};
    auto take = [&](intx4 raw) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const uint32_t u = (uint32_t)raw[q];
            if (kBf16) {
                s.a += square(__builtin_bit_cast(float, u << 16));
                s.b += square(__builtin_bit_cast(float, u & 0xffff0000u));
            } else if (q & 1) {
                s.b += square(__builtin_bit_cast(float, u));
            } else {
                s.a += square(__builtin_bit_cast(float, u));
            }
        }
    };
    int x = threadIdx.x;
    for (; x + (kGradUnroll - 1) * kGradThreads < whole; x += kGradUnroll * kGradThreads) {
        intx4 v[kGradUnroll];
#pragma unroll
        for (int y = 0; y < kGradUnroll; ++y) v[y] = grad_load(g + (x + y * kGradThreads) * 16);
#pragma unroll
        for (int y = 0; y < kGradUnroll; ++y) take(v[y]);
    }
    for (; x < whole; x += kGradThreads) take(grad_load(g + x * 16));
    for (int e = whole * kPer + threadIdx.x; e < k.count; e += kGradThreads)
        s.a += square(kBf16 ? bf16_to_f32(((const uint16_t*)g)[e]) : ((const float*)g)[e]);
    return s;
}

// Workgroup b sums chunks b, b + grid, ... into its own slot.  The last workgroup to
// finish (of a call's last launch) adds all slots in ascending order.  They count in 32
// to a counter, and the last of 32 to one above them, each in a cache line of its own:
// 2048 workgroups on one counter take 25 us to pass it.  1.4e9 fp32 values: 823 us (6.9 TB/s);
// a layer's few thousand 5.6 us.
__global__ __launch_bounds__(kGradThreads) void grad_norm_kernel(GradList a, double* partial, int slot0, int slots,
                                                                 int* counters, float* norm) {
    __shared__ double s_sum[kGradThreads / kWave];
    __shared__ int s_last;
    double sum0 = 0.0, sum1 = 0.0;
    for (int64_t c = blockIdx.x; c < a.first[a.n]; c += gridDim.x) {
        const GradChunk k = grad_chunk(a, c);
        const GradSums s = a.count[k.i] & kGradBf16 ? grad_squares<true>(a.src[k.i], k) : grad_squares<false>(a.src[k.i], k);
        sum0 += s.a;
        sum1 += s.b;
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
        if (norm) {  // (a call's last launch)
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // the store has reached memory before it is counted
            auto last_of = [&](int line, int n) {  // and the counter is back at zero for the next call
                int* at = counters + line * kGradLineInts;
                if (__hip_atomic_fetch_add(at, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) != n - 1) return false;
                __hip_atomic_store(at, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
                return true;
            };
            const int grid = gridDim.x, team = blockIdx.x / 32, teams = (grid + 31) / 32;
            if (last_of(1 + team, min(32, grid - team * 32)) && last_of(0, teams)) s_last = 1;
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

template <bool kBf16>
__device__ __forceinline__ void grad_scale(const void* src, void* dst, const GradChunk& k, float coef) {
    constexpr int kSize = kBf16 ? 2 : 4, kPer = 16 / kSize;
    const char* g = (const char*)src + k.first * kSize;
    char* o = (char*)dst + k.first * kSize;
    const int whole = (((uintptr_t)g | (uintptr_t)o) & 15) == 0 ? k.count / kPer : 0;  // vectors
    auto scaled = [&](intx4 raw) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const uint32_t u = (uint32_t)raw[q];
            if (kBf16)
                raw[q] = (int)pack_bf16x2(__builtin_bit_cast(float, u << 16) * coef,
                                          __builtin_bit_cast(float, u & 0xffff0000u) * coef);
            else
                raw[q] = __builtin_bit_cast(int, __builtin_bit_cast(float, u) * coef);
        }
        return raw;
    };
    int x = threadIdx.x;
    for (; x + (kGradUnroll - 1) * kGradThreads < whole; x += kGradUnroll * kGradThreads) {
        intx4 v[kGradUnroll];
#pragma unroll
        for (int y = 0; y < kGradUnroll; ++y) v[y] = grad_load(g + (x + y * kGradThreads) * 16);
#pragma unroll
        for (int y = 0; y < kGradUnroll; ++y) grad_store(o + (x + y * kGradThreads) * 16, scaled(v[y]));
    }
    for (; x < whole; x += kGradThreads) grad_store(o + x * 16, scaled(grad_load(g + x * 16)));
    for (int e = whole * kPer + threadIdx.x; e < k.count; e += kGradThreads) {
        if (kBf16) ((uint16_t*)o)[e] = (uint16_t)pack_bf16x2(bf16_to_f32(((const uint16_t*)g)[e]) * coef, 0.0f);
        else ((float*)o)[e] = ((const float*)g)[e] * coef;
    }
}

// A NaN norm makes every gradient NaN, an infinite one zero (infinite ones NaN).  A
// workgroup to a chunk of 4096 elements: 1.4e9 fp32 values 1900 us (5.9 TB/s), against
// 2200 in chunks of 16384 over 4096 workgroups.
__global__ __launch_bounds__(kGradThreads) void grad_clip_kernel(GradList a, const float* norm, float max_norm) {
    const double ratio = (double)max_norm / ((double)*norm + 1e-6);
    const float coef = ratio >= 1.0 ? 1.0f : (float)ratio;
    for (int64_t c = blockIdx.x; c < a.first[a.n]; c += gridDim.x) {
        const GradChunk k = grad_chunk(a, c);
        if (a.src[k.i] == a.dst[k.i] && coef == 1.0f) continue;  // in place and within the bound
        if (a.count[k.i] & kGradBf16) grad_scale<true>(a.src[k.i], a.dst[k.i], k, coef);
        else grad_scale<false>(a.src[k.i], a.dst[k.i], k, coef);
    }
}

// Fills the chunks' size and bounds; returns how many there are.  4096 elements, less
// where that gives too few to spread over the CUs.
static int64_t grad_chunks(GradList& a) {
    uint64_t all = 0;
    for (int i = 0; i < a.n; ++i) all += a.count[i] & ~kGradBf16;
    a.chunk = 4096;
    while (a.chunk > 1024 && all / a.chunk < 512) a.chunk /= 2;
    a.first[0] = 0;
    for (int i = 0; i < a.n; ++i)
        a.first[i + 1] = a.first[i] + ((int64_t)(a.count[i] & ~kGradBf16) + a.chunk - 1) / a.chunk;
    return a.first[a.n];
}

int launch_grad_norm(GradList a, double* partial, int slot0, bool last, int* counters, float* norm,
                     hipStream_t stream) {
    const int64_t chunks = grad_chunks(a);
    const int grid = (int)(chunks < 1 ? 1 : chunks < kGradSlots ? chunks : kGradSlots);
    hipLaunchKernelGGL(grad_norm_kernel, dim3(grid), dim3(kGradThreads), 0, stream, a, partial, slot0, slot0 + grid,
                       counters, last ? norm : nullptr);
    return slot0 + grid;
}

void launch_grad_clip(GradList a, const float* norm, float max_norm, hipStream_t stream) {
    const int64_t chunks = grad_chunks(a);
    if (chunks == 0) return;
    hipLaunchKernelGGL(grad_clip_kernel, dim3((unsigned)(chunks < (1 << 22) ? chunks : (1 << 22))), dim3(kGradThreads), 0,
                       stream, a, norm, max_norm);
}

}  // namespace moe
