// Residual addition with root-mean-square norm, forward and backward (gfx950).
//
//   s = bf16(x + residual),  rstd = 1 / sqrt(mean(s^2) + eps),  y = bf16(s * rstd * w)
//   dx = dsum + rstd * (dy w - xhat mean(dy w xhat)),  xhat = s * rstd
//   dw = sum over rows of dy * xhat
//
// All of it is bound by memory: a few operations per value.  A row is read once
// and kept in registers between its sum and its output; only the backward of
// rows past 16384 columns reads them twice.  A thread holds vectors of eight
// consecutive values (16 bytes of bf16), so an MXFP8 block of 32 is four
// neighbouring lanes.
#include "common.hpp"
#include "kernels.hpp"
#include "mxfp8.hpp"

namespace moe {

#pragma clang fp contract(off)

constexpr int kNormVec = 8;

__device__ __forceinline__ void unpack8(intx4 raw, float (&v)[8]) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        v[2 * q] = __builtin_bit_cast(float, (uint32_t)raw[q] << 16);
        v[2 * q + 1] = __builtin_bit_cast(float, (uint32_t)raw[q] & 0xffff0000u);
    }
}

// Two values rounded to nearest even by the conversion instruction.  It gives what
// f32_to_bf16_rne gives for all 2^32 patterns but the NaN ones (compared one by
// one), and these stay NaN: adding to a pattern carries a NaN whose payload is all
// ones, as a gain or 1/rms read from outside may hold, over into a zero.
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    typedef float floatx2 __attribute__((ext_vector_type(2)));
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(floatx2{a, b}, bf16x2));
}

__device__ __forceinline__ intx4 pack8(const float (&v)[8]) {
    intx4 o;
#pragma unroll
    for (int q = 0; q < 4; ++q) o[q] = (int)pack2(v[2 * q], v[2 * q + 1]);
    return o;
}

// Sum over the kLanes lanes of a row's group.
template <int kLanes = kWave>
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int s = kLanes / 2; s >= 1; s >>= 1) v += __shfl_xor(v, s, kWave);
    return v;
}

// Sum over the workgroup (kWaves waves), the same in every thread and in the
// same order on every call.
template <int kWaves, int kLanes>
__device__ __forceinline__ float group_sum(float v, float* s_sum) {
    v = wave_sum<kLanes>(v);
    if constexpr (kWaves == 1) return v;
    if ((threadIdx.x & 63) == 0) s_sum[threadIdx.x >> 6] = v;
    lds_barrier();  // the stores in flight need not have ended
    float r = s_sum[0];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) r += s_sum[w];
    return r;
}

// The eight values of a lane as part of the 32-value block of its four lanes:
// the codes, and the scale byte (the same in all four).
__device__ __forceinline__ uint64_t block_codes(const float (&v)[8], uint8_t& scale) {
    float m = 0.0f;
#pragma unroll
    for (int c = 0; c < 8; ++c) m = fmaxf(m, fabsf(v[c]));
    m = fmaxf(m, __shfl_xor(m, 1, kWave));
    m = fmaxf(m, __shfl_xor(m, 2, kWave));
    const int e = mx_scale_exp(m);
    scale = (uint8_t)(e + 127);
    const uint32_t lo = fp8x4(ldexpf(v[0], -e), ldexpf(v[1], -e), ldexpf(v[2], -e), ldexpf(v[3], -e));
    const uint32_t hi = fp8x4(ldexpf(v[4], -e), ldexpf(v[5], -e), ldexpf(v[6], -e), ldexpf(v[7], -e));
    return (uint64_t)lo | ((uint64_t)hi << 32);
}

// A row per group of kWaves waves, kNV vectors per thread, or (kWaves = 1) of
// kLanes lanes, 256 / kLanes rows in a workgroup: 262144 rows of 128 with the
// residual and its sum take 48 us (5.5 TB/s) with 16 lanes a row.  On inputs that the
// last cache held in part it was 42 us, against 92 with 64 lanes.
template <int kWaves, int kNV, int kLanes>
__global__ __launch_bounds__(kWaves == 1 ? 256 : kWaves * kWave) void norm_fwd_kernel(NormFwd a) {
    __shared__ float s_sum[kWaves];
    const int lid = kWaves > 1 ? threadIdx.x : threadIdx.x % kLanes;
    const int64_t r = kWaves > 1 ? (int64_t)blockIdx.x : (int64_t)blockIdx.x * (256 / kLanes) + threadIdx.x / kLanes;
    if (kWaves == 1 && r >= a.rows) return;  // whole rows; no barrier follows
    const int nv = a.cols / kNormVec;
    const int64_t base = r * a.cols;
    float v[kNV][8];
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < kNV; ++i) {
        const int p = lid + i * kWaves * kWave;
        intx4 raw = {0, 0, 0, 0};
        if (p < nv) raw = *(const intx4*)(a.x + base + p * kNormVec);
        if (a.residual) {
            intx4 rr = {0, 0, 0, 0};
            if (p < nv) rr = *(const intx4*)(a.residual + base + p * kNormVec);
            float xv[8], rv[8];
            unpack8(raw, xv);
            unpack8(rr, rv);
#pragma unroll
            for (int c = 0; c < 8; ++c) xv[c] += rv[c];
            raw = pack8(xv);
        }
        if (a.summed && p < nv) *(intx4*)(a.summed + base + p * kNormVec) = raw;
        unpack8(raw, v[i]);
#pragma unroll
        for (int c = 0; c < 8; ++c) ss = __builtin_fmaf(v[i][c], v[i][c], ss);
    }
    const float rstd = 1.0f / sqrtf(group_sum<kWaves, kLanes>(ss, s_sum) / (float)a.cols + a.eps);
    if (a.rstd && lid == 0) a.rstd[r] = rstd;
    const int nb = a.cols / 32;
#pragma unroll
    for (int i = 0; i < kNV; ++i) {
        const int p = lid + i * kWaves * kWave;
        if (p >= nv) break;  // in fours: cols is a multiple of 32
        uint8_t sc;
        if (a.ckq) {
            *(uint64_t*)(a.ckq + base + p * kNormVec) = block_codes(v[i], sc);
            if ((p & 3) == 0) a.cks[r * nb + (p >> 2)] = sc;
        }
        const floatx4 w0 = *(const floatx4*)(a.weight + p * kNormVec), w1 = *(const floatx4*)(a.weight + p * kNormVec + 4);
        float y[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) y[c] = v[i][c] * rstd * (c < 4 ? w0[c] : w1[c - 4]);
        const intx4 out = pack8(y);
        *(intx4*)(a.y + base + p * kNormVec) = out;
        if (a.yq) {  // the codes of the rounded y, as the layer's own quantisation of y gives
            unpack8(out, y);
            *(uint64_t*)(a.yq + base + p * kNormVec) = block_codes(y, sc);
            if ((p & 3) == 0) mx_store_scale_byte(a.ys, a.rows, r, p >> 2, nb, sc);
        }
    }
}

void launch_norm_fwd(const NormFwd& a, hipStream_t stream) {
    const int nv = a.cols / kNormVec;
#define NORM_FWD(W, NV, LANES)                                                                            \
    hipLaunchKernelGGL((norm_fwd_kernel<W, NV, LANES>),                                                   \
                       dim3((unsigned)(W > 1 ? a.rows : (a.rows + 256 / LANES - 1) / (256 / LANES))),     \
                       dim3(W > 1 ? W * kWave : 256), 0, stream, a)
    if (nv <= 8) NORM_FWD(1, 1, 8);
    else if (nv <= 16) NORM_FWD(1, 1, 16);
    else if (nv <= 32) NORM_FWD(1, 1, 32);
    else if (nv <= 64) NORM_FWD(1, 1, 64);
    else if (nv <= 128) NORM_FWD(1, 2, 64);
    else if (nv <= 256) NORM_FWD(2, 2, 64);
    else if (nv <= 512) NORM_FWD(4, 2, 64);
    else if (nv <= 1024) NORM_FWD(8, 2, 64);
    else if (nv <= 2048) NORM_FWD(16, 2, 64);
    else NORM_FWD(16, 4, 64);
#undef NORM_FWD
}

// ---------------------------------------------------------------------------
// Backward
// ---------------------------------------------------------------------------

constexpr int kNormParts = 512;   // most partial sums of dw
constexpr int kNarrowVecs = 128;  // vectors of a row that one wave holds, up to two a lane

constexpr int kBwdWaves = 8;      // most waves that hold a row and ask for the next
constexpr int kWideWaves = 16;    // waves of a row past what those hold

// Lanes of a row where one wave holds it, of a 256-thread workgroup's rows; 0 for
// wider rows, a workgroup each.
static int narrow_lanes(int cols) {
    const int nv = cols / kNormVec;
    return nv <= 8 ? 8 : nv <= 16 ? 16 : nv <= 32 ? 32 : nv <= kNarrowVecs ? 64 : 0;
}

int norm_bwd_parts(int64_t rows, int cols) {
    const int lanes = narrow_lanes(cols);
    if (lanes) rows = (rows + 256 / lanes - 1) / (256 / lanes);
    // Few rows: one workgroup takes them all and writes dw itself, which spares a
    // launch (2.5 us of the host's time) and the sums' way through memory.  Four
    // sets of narrow rows, 4 of 512: 3.2 against 5.4 us; 2 rows of 2048 3.9 against
    // 5.6, 2 of 16384 8.5 against 8.9, but 4 of 7168 8.7 against 6.8 and 2 of 32768
    // 15.9 against 14.4.
    if (rows <= (lanes ? 4 : cols <= kNormVec * kWave * kBwdWaves * 4 ? 2 : 1)) return 1;
    return (int)(rows < kNormParts ? rows : kNormParts);
}

// A vector of a row as it lies in memory.
template <bool kCk>
struct NormVec {
    intx4 dy, s;
    uint64_t q;
    int e;
};

// Its s.
template <bool kCk>
__device__ __forceinline__ void norm_values(const NormVec<kCk>& v, float (&s)[8]) {
    if constexpr (kCk) {
        const int e = v.e - 127;
        const uint32_t lo = (uint32_t)v.q, hi = (uint32_t)(v.q >> 32);
        s[0] = __builtin_amdgcn_cvt_f32_fp8(lo, 0); s[1] = __builtin_amdgcn_cvt_f32_fp8(lo, 1);
        s[2] = __builtin_amdgcn_cvt_f32_fp8(lo, 2); s[3] = __builtin_amdgcn_cvt_f32_fp8(lo, 3);
        s[4] = __builtin_amdgcn_cvt_f32_fp8(hi, 0); s[5] = __builtin_amdgcn_cvt_f32_fp8(hi, 1);
        s[6] = __builtin_amdgcn_cvt_f32_fp8(hi, 2); s[7] = __builtin_amdgcn_cvt_f32_fp8(hi, 3);
#pragma unroll
        for (int c = 0; c < 8; ++c) s[c] = ldexpf(s[c], e);
    } else {
        unpack8(v.s, s);
    }
}

// Workgroup b takes rows b, b + parts, ...; dw's partial sums stay in
// registers over them.  The next row is asked for before this one's sum is joined
// over the workgroup, so a row's loads (all of them at once) have the barrier and
// the arithmetic of a row to arrive: 4096 rows of 2048 from the checkpoint 23.3 ->
// 16.2 us, 16384 of 7168 191 -> 179 us (5.2 TB/s).
template <int kNV, bool kCk>
__global__ __launch_bounds__(kBwdWaves * kWave) void norm_bwd_kernel(NormBwd a) {
    __shared__ float s_sum[2][kBwdWaves];
    const int lid = threadIdx.x, waves = blockDim.x / kWave;
    const int nv = a.cols / kNormVec, nb = a.cols / 32;
    float dw[kNV][8];
#pragma unroll
    for (int i = 0; i < kNV; ++i)
#pragma unroll
        for (int c = 0; c < 8; ++c) dw[i][c] = 0.0f;
    // vectors past the row's end repeat its last one; what they give is not used
    auto vec_of = [&](int i) { return min(lid + i * (int)blockDim.x, nv - 1); };
    auto load = [&](int64_t r, int i, NormVec<kCk>& t) {
        const int p = vec_of(i);
        const int64_t at = r * a.cols + p * kNormVec;
        t.dy = *(const intx4*)(a.dy + at);
        if constexpr (kCk) {
            t.q = *(const uint64_t*)(a.ckq + at);
            t.e = a.cks[r * nb + (p >> 2)];
        } else {
            t.s = *(const intx4*)(a.summed + at);
        }
    };
    auto load_ds = [&](int64_t r, int i) {
        return a.dsum ? *(const intx4*)(a.dsum + r * a.cols + vec_of(i) * kNormVec) : intx4{0, 0, 0, 0};
    };
    NormVec<kCk> t[kNV];
    intx4 ds[kNV];
    float rstd = a.rstd[blockIdx.x];  // there are no more workgroups than rows
#pragma unroll
    for (int i = 0; i < kNV; ++i) {
        load(blockIdx.x, i, t[i]);
        ds[i] = load_ds(blockIdx.x, i);
    }
    int half = 0;
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x, half ^= 1) {
        float xh[kNV][8], gy[kNV][8], dv[kNV][8];
        const float rs = rstd;
        float dot = 0.0f;
#pragma unroll
        for (int i = 0; i < kNV; ++i) {
            const bool in = lid + i * (int)blockDim.x < nv;
            norm_values<kCk>(t[i], xh[i]);
            unpack8(t[i].dy, gy[i]);
            unpack8(ds[i], dv[i]);
            const float* wp = a.weight + vec_of(i) * kNormVec;  // cached
            const floatx4 w0 = *(const floatx4*)wp, w1 = *(const floatx4*)(wp + 4);
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                xh[i][c] *= rs;
                dw[i][c] = __builtin_fmaf(gy[i][c], xh[i][c], dw[i][c]);
                gy[i][c] *= c < 4 ? w0[c] : w1[c - 4];
                if (in) dot = __builtin_fmaf(gy[i][c], xh[i][c], dot);
            }
        }
        {
            const int64_t rn = r + gridDim.x < a.rows ? r + gridDim.x : r;
            rstd = a.rstd[rn];
#pragma unroll
            for (int i = 0; i < kNV; ++i) {
                load(rn, i, t[i]);
                ds[i] = load_ds(rn, i);
            }
        }
        dot = wave_sum(dot);
        if (waves > 1) {
            if ((lid & 63) == 0) s_sum[half][lid >> 6] = dot;
            lds_barrier();
            dot = s_sum[half][0];
            for (int v = 1; v < waves; ++v) dot += s_sum[half][v];
        }
        const float mean = dot / (float)a.cols;
#pragma unroll
        for (int i = 0; i < kNV; ++i) {
            const int p = lid + i * (int)blockDim.x;
            if (p >= nv) continue;
            float d[8];
#pragma unroll
            for (int c = 0; c < 8; ++c) d[c] = rs * (gy[i][c] - xh[i][c] * mean) + dv[i][c];
            *(intx4*)(a.dx + r * a.cols + p * kNormVec) = pack8(d);
        }
    }
#pragma unroll
    for (int i = 0; i < kNV; ++i) {
        const int p = lid + i * (int)blockDim.x;
        if (p >= nv) continue;
        float* d = a.partial + (int64_t)blockIdx.x * a.cols + p * kNormVec;
        *(floatx4*)d = floatx4{dw[i][0], dw[i][1], dw[i][2], dw[i][3]};
        *(floatx4*)(d + 4) = floatx4{dw[i][4], dw[i][5], dw[i][6], dw[i][7]};
    }
}

// The same for rows past 16384, sixteen waves and up to four vectors a lane: 128
// registers a lane hold dw's sums but not the row, which is read again after its
// sum (from the L2 or the cache behind it): 2048 rows of 32768 149 us (3.6 TB/s of
// what has to move).  Eight waves of eight vectors that keep the row as fp32 xhat,
// g and dsum (24 registers a vector) spill, and so do sixteen of four: 324 and 265
// us.  A row kept as it lies in memory (8 a vector) has not been built.
template <bool kCk>
__global__ __launch_bounds__(kWideWaves * kWave) void norm_bwd_wide_kernel(NormBwd a) {
    constexpr int kNV = 4, kThreads = kWideWaves * kWave;
    __shared__ float s_sum[2][kWideWaves];
    const int lid = threadIdx.x;
    const int nv = a.cols / kNormVec, nb = a.cols / 32;
    float dw[kNV][8];
#pragma unroll
    for (int i = 0; i < kNV; ++i)
#pragma unroll
        for (int c = 0; c < 8; ++c) dw[i][c] = 0.0f;
    // xhat, dy and the weights of vector p, an address of 32 bits from a scalar one
    auto values = [&](int64_t r, uint32_t p, float rs, float (&xh)[8], float (&gy)[8], float (&w)[8]) {
        const int64_t row = r * a.cols;
        const uint32_t at = p * kNormVec;
        NormVec<kCk> t;
        t.dy = *(const intx4*)(a.dy + row + at);
        if constexpr (kCk) {
            t.q = *(const uint64_t*)(a.ckq + row + at);
            t.e = (a.cks + r * nb)[p >> 2];
        } else {
            t.s = *(const intx4*)(a.summed + row + at);
        }
        const floatx4 w0 = *(const floatx4*)(a.weight + at), w1 = *(const floatx4*)(a.weight + at + 4);
        norm_values<kCk>(t, xh);
        unpack8(t.dy, gy);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            xh[c] *= rs;
            w[c] = c < 4 ? w0[c] : w1[c - 4];
        }
    };
    int half = 0;
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x, half ^= 1) {
        const float rs = a.rstd[r];
        float dot = 0.0f, xh[8], gy[8], w[8];
#pragma unroll
        for (int i = 0; i < kNV; ++i) {
            const uint32_t p = lid + i * kThreads;
            if ((int)p >= nv) break;
            values(r, p, rs, xh, gy, w);
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                dw[i][c] = __builtin_fmaf(gy[c], xh[c], dw[i][c]);
                dot = __builtin_fmaf(gy[c] * w[c], xh[c], dot);
            }
        }
        dot = wave_sum(dot);
        if ((lid & 63) == 0) s_sum[half][lid >> 6] = dot;
        asm volatile("" ::: "memory");  // read again, not kept
        lds_barrier();
        dot = s_sum[half][0];
#pragma unroll
        for (int v = 1; v < kWideWaves; ++v) dot += s_sum[half][v];
        const float mean = dot / (float)a.cols;
#pragma unroll 1
        for (uint32_t p = lid; (int)p < nv; p += kThreads) {
            const int64_t row = r * a.cols;
            float d[8];
            values(r, p, rs, xh, gy, w);
            unpack8(a.dsum ? *(const intx4*)(a.dsum + row + p * kNormVec) : intx4{0, 0, 0, 0}, d);
#pragma unroll
            for (int c = 0; c < 8; ++c) d[c] = rs * (gy[c] * w[c] - xh[c] * mean) + d[c];
            *(intx4*)(a.dx + row + p * kNormVec) = pack8(d);
        }
    }
#pragma unroll
    for (int i = 0; i < kNV; ++i) {
        const int p = lid + i * kThreads;
        if (p >= nv) break;
        float* d = a.partial + (int64_t)blockIdx.x * a.cols + p * kNormVec;
        *(floatx4*)d = floatx4{dw[i][0], dw[i][1], dw[i][2], dw[i][3]};
        *(floatx4*)(d + 4) = floatx4{dw[i][4], dw[i][5], dw[i][6], dw[i][7]};
    }
}

// The same for rows that one wave holds: kLanes lanes a row, 256 / kLanes rows
// of a workgroup side by side, so that narrow rows (a head's) fill their lanes
// and no barrier stands in the loop.  The rows' sums of dw meet in LDS at the
// end. Against a workgroup a row, on inputs that the last cache holds in part:
// 262144 rows of 128 377 -> 47 us, 65536 of 512 103 -> 45 us, 16384 of 1024 37
// -> 26 us; on three such inputs in turn the first two take 52 us (5.1 TB/s).
// Rows of 2048 would need four vectors a lane and 256 registers: 4096 of them
// from the checkpoint take 21 us that way and 18 us with a workgroup each.
template <int kLanes, int kNV, bool kCk>
__global__ __launch_bounds__(256) void norm_bwd_narrow_kernel(NormBwd a) {
    constexpr int kRows = 256 / kLanes;
    __shared__ float s_dw[kRows][kLanes * kNV * kNormVec];
    const int lid = threadIdx.x % kLanes, row = threadIdx.x / kLanes;
    const int nv = a.cols / kNormVec, nb = a.cols / 32;
    auto vec_of = [&](int i) { return min(lid + i * kLanes, nv - 1); };
    NormVec<kCk> t[kNV];
    intx4 ds[kNV];
    float rstd;
    auto load = [&](int64_t r) {
        rstd = a.rstd[r];
#pragma unroll
        for (int i = 0; i < kNV; ++i) {
            const int p = vec_of(i);
            const int64_t at = r * a.cols + p * kNormVec;
            t[i].dy = *(const intx4*)(a.dy + at);
            if constexpr (kCk) {
                t[i].q = *(const uint64_t*)(a.ckq + at);
                t[i].e = a.cks[r * nb + (p >> 2)];
            } else {
                t[i].s = *(const intx4*)(a.summed + at);
            }
            ds[i] = a.dsum ? *(const intx4*)(a.dsum + at) : intx4{0, 0, 0, 0};
        }
    };
    float dw[kNV][8], w[kNV][8];
#pragma unroll
    for (int i = 0; i < kNV; ++i) {
        const float* wp = a.weight + vec_of(i) * kNormVec;
        const floatx4 w0 = *(const floatx4*)wp, w1 = *(const floatx4*)(wp + 4);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            dw[i][c] = 0.0f;
            w[i][c] = c < 4 ? w0[c] : w1[c - 4];
        }
    }
    const int64_t first = (int64_t)blockIdx.x * kRows + row, stride = (int64_t)gridDim.x * kRows;
    load(min(first, a.rows - 1));
    for (int64_t r = first; r < a.rows; r += stride) {
        float xh[kNV][8], gy[kNV][8], dv[kNV][8];
        const float rs = rstd;
        float dot = 0.0f;
#pragma unroll
        for (int i = 0; i < kNV; ++i) {
            norm_values<kCk>(t[i], xh[i]);
            unpack8(t[i].dy, gy[i]);
            unpack8(ds[i], dv[i]);
            const bool in = lid + i * kLanes < nv;
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                xh[i][c] *= rs;
                dw[i][c] = __builtin_fmaf(gy[i][c], xh[i][c], dw[i][c]);
                gy[i][c] *= w[i][c];
                if (in) dot = __builtin_fmaf(gy[i][c], xh[i][c], dot);
            }
        }
        load(min(r + stride, a.rows - 1));
        const float mean = wave_sum<kLanes>(dot) / (float)a.cols;
#pragma unroll
        for (int i = 0; i < kNV; ++i) {
            const int p = lid + i * kLanes;
            float d[8];
#pragma unroll
            for (int c = 0; c < 8; ++c) d[c] = rs * (gy[i][c] - xh[i][c] * mean) + dv[i][c];
            if (p < nv) *(intx4*)(a.dx + r * a.cols + p * kNormVec) = pack8(d);
        }
    }
#pragma unroll
    for (int i = 0; i < kNV; ++i) {
        floatx4* d = (floatx4*)&s_dw[row][(lid + i * kLanes) * kNormVec];
        d[0] = floatx4{dw[i][0], dw[i][1], dw[i][2], dw[i][3]};
        d[1] = floatx4{dw[i][4], dw[i][5], dw[i][6], dw[i][7]};
    }
    __syncthreads();
    for (int c = threadIdx.x; c < a.cols; c += 256) {
        float v[kRows];
#pragma unroll
        for (int g = 0; g < kRows; ++g) v[g] = s_dw[g][c];
#pragma unroll
        for (int n = kRows / 2; n >= 1; n >>= 1)
#pragma unroll
            for (int g = 0; g < n; ++g) v[g] += v[g + n];
        a.partial[(int64_t)blockIdx.x * a.cols + c] = v[0];
    }
}

// dw[c] = the partial sums in a fixed order: 32 columns per workgroup, thread
// (group, column quad) sums every 128th part, then a tree over the groups.
__global__ __launch_bounds__(1024) void norm_dw_kernel(const float* partial, int parts, int cols, float* dw) {
    __shared__ __attribute__((aligned(16))) floatx4 s[128][8];
    const int q = threadIdx.x & 7, g = threadIdx.x >> 3;
    const int c = blockIdx.x * 32 + q * 4;
    floatx4 v = {0, 0, 0, 0};
#pragma unroll 4
    for (int p = g; p < parts; p += 128) v += *(const floatx4*)(partial + (int64_t)p * cols + c);
    s[g][q] = v;
    for (int n = 64; n >= 1; n >>= 1) {
        __syncthreads();
        if (g < n) s[g][q] += s[g + n][q];
    }
    if (g == 0) *(floatx4*)(dw + c) = s[0][q];
}

void launch_norm_bwd(NormBwd a, hipStream_t stream) {
    const int nv = a.cols / kNormVec;
    const int parts = norm_bwd_parts(a.rows, a.cols);
    if (parts == 1) a.partial = a.dw;  // the only part is the sum
#define NORM_BWD(NV)                                                                                             \
    do {                                                                                                         \
        const dim3 block(ceil_div(ceil_div(nv, NV), kWave) * kWave);                                             \
        if (a.ckq)                                                                                               \
            hipLaunchKernelGGL((norm_bwd_kernel<NV, true>), dim3(parts), block, 0, stream, a);              \
        else                                                                                                     \
            hipLaunchKernelGGL((norm_bwd_kernel<NV, false>), dim3(parts), block, 0, stream, a);             \
    } while (0)
#define NORM_BWD_NARROW(LANES, NV)                                                                               \
    do {                                                                                                         \
        if (a.ckq)                                                                                               \
            hipLaunchKernelGGL((norm_bwd_narrow_kernel<LANES, NV, true>), dim3(parts), dim3(256), 0, stream, a); \
        else                                                                                                     \
            hipLaunchKernelGGL((norm_bwd_narrow_kernel<LANES, NV, false>), dim3(parts), dim3(256), 0, stream, a); \
    } while (0)
    if (nv <= 8) NORM_BWD_NARROW(8, 1);
    else if (nv <= 16) NORM_BWD_NARROW(16, 1);
    else if (nv <= 32) NORM_BWD_NARROW(32, 1);
    else if (nv <= 64) NORM_BWD_NARROW(64, 1);
    else if (nv <= kNarrowVecs) NORM_BWD_NARROW(64, 2);
    else if (nv <= 512) NORM_BWD(1);
    else if (nv <= 1024) NORM_BWD(2);
    else if (nv <= 2048) NORM_BWD(4);
    else if (a.ckq)
        hipLaunchKernelGGL(norm_bwd_wide_kernel<true>, dim3(parts), dim3(kWideWaves * kWave), 0, stream, a);
    else
        hipLaunchKernelGGL(norm_bwd_wide_kernel<false>, dim3(parts), dim3(kWideWaves * kWave), 0, stream, a);
#undef NORM_BWD
#undef NORM_BWD_NARROW
    if (parts == 1) return;
    hipLaunchKernelGGL(norm_dw_kernel, dim3(a.cols / 32), dim3(1024), 0, stream, a.partial, parts, a.cols, a.dw);
}

}  // namespace moe
