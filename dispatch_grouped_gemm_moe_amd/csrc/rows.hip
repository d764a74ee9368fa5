// Rows by expert and back (gfx950): what stands on either side of the experts'
// products, forward and backward, and the quantisers of the products' operands.
//
//   dispatch     xs[r(t,j)] = x[t]
//   combine      out[t] = add[t] + sum_j w[t,j] src[r(t,j)]
//   its gradient dsrc[r(t,j)] = w[t,j] dout[t],  dw[t,j] = <src[r(t,j)], dout[t]>
//
// r(t,j) is the row of token t's choice j; one outside the rows is no row (a
// dropped choice).  All of it is bound by memory.  A token's row is read once and
// serves its k rows, so the unit of work is a token, not a row: 16384 tokens of
// 7168 to 8 rows each read 0.23 GB and write 1.9 instead of moving 1.9 twice.
//
// A thread holds vectors of eight consecutive values (16 bytes of bf16); a block of
// 128 that gets one scale is 16 neighbouring lanes.
#include "block8.hpp"
#include "common.hpp"
#include "kernels.hpp"

namespace moe {

#pragma clang fp contract(off)

constexpr int kRowThreads = 256;
constexpr int kRowVec = 8;

// Threads that share a token: a power of two from 16 (a block of 128) to the
// workgroup, so that narrow rows stand side by side in a workgroup.
static int row_lanes_log(int cols) {
    const int nv = (cols + kRowVec - 1) / kRowVec;
    int s = 4;
    while (s < 8 && (1 << s) < nv) ++s;
    return s;
}

static unsigned row_grid(int64_t units) { return (unsigned)(units < (1 << 22) ? units : (1 << 22)); }

// Workgroups that share a token's columns: one where the tokens alone fill the CUs,
// which then reads the token's table once.
static unsigned row_slices(int64_t groups, int cols, int log) {
    const int slices = (cols / kRowVec + (1 << log) - 1) >> log;
    return (unsigned)(groups >= 2048 ? 1 : slices);
}

// An entry of a table that no kernel changes while it is read, of a token that is the
// same in the whole wave: a scalar load.
template <class T>
__device__ __forceinline__ T ld_uniform(const T* p) {
    return *(const __attribute__((address_space(4))) T*)p;
}

// ---------------------------------------------------------------------------
// Dispatch, and the quantiser (a dispatch of every row to itself)
// ---------------------------------------------------------------------------

// A workgroup takes kRowThreads >> log tokens at a time.  kWide: one wave's lanes share
// a token (rows of more than 256 columns).
template <bool kCodes, bool kWide>
__global__ __launch_bounds__(kRowThreads) void rows_dispatch_kernel(RowsDispatch a, int log) {
    const int lanes = 1 << log, per = kRowThreads >> log;
    const int lid = threadIdx.x & (lanes - 1);
    const int sub = kWide ? __builtin_amdgcn_readfirstlane(threadIdx.x >> log) : threadIdx.x >> log;
    const int nv = a.cols / kRowVec;
    int64_t t_lo = 0, t_hi = a.tokens;
    if (a.offsets) {
        t_lo = max(a.offsets[0], 0);
        t_hi = min((int64_t)a.offsets[a.groups], a.tokens);
    }
    for (int64_t t0 = (int64_t)blockIdx.x * per; t0 < t_hi; t0 += (int64_t)gridDim.x * per) {
        const int64_t t = t0 + sub;
        const bool tok = t >= t_lo && t < t_hi;
        // (whole groups of 16 lanes: they share a block's maximum)
        for (int p = blockIdx.y * lanes + lid; (p & ~15) < nv; p += gridDim.y * lanes) {
            const bool live = tok && p < nv;
            intx4 raw = {0, 0, 0, 0};
            float v[8];
            if (live) {
                if (kCodes && a.xf) {
                    const floatx4* s = (const floatx4*)(a.xf + t * a.cols + (int64_t)p * kRowVec);
                    const floatx4 f0 = s[0], f1 = s[1];
#pragma unroll
                    for (int c = 0; c < 8; ++c) v[c] = c < 4 ? f0[c] : f1[c - 4];
                } else {
                    raw = *(const intx4*)(a.x + t * a.cols + (int64_t)p * kRowVec);
                }
            }
            uint64_t q = 0;
            float scale = 0.0f;
            if constexpr (kCodes) {
                if (!a.xf) unpack_bf16x8(raw, v);
                float m = live ? abs_max8(v) : 0.0f;  // past the row's end: zeros
#pragma unroll
                for (int s = 1; s < 16; s *= 2) m = fmaxf(m, __shfl_xor(m, s, kWave));
                const int e = blk_exp(m);
                scale = pow2f(e);
                q = blk_codes8(v, e);
                if (a.xf) raw = pack_bf16x8(v);
            }
            if (!live) continue;
            for (int j = 0; j < a.k; ++j) {
                const int32_t* at = a.tok_row + t * a.k + j;
                const int64_t r = !a.tok_row ? t : kWide ? ld_uniform(at) : *at;
                if (r < 0 || r >= a.rows) continue;  // no row
                if (a.dst) *(intx4*)(a.dst + r * a.cols + (int64_t)p * kRowVec) = raw;
                if constexpr (kCodes) {
                    *(uint64_t*)(a.codes + r * a.cols + (int64_t)p * kRowVec) = q;
                    if ((p & 15) == 0) a.scales[(int64_t)(p >> 4) * a.rows + r] = scale;
                }
            }
        }
    }
}

void launch_rows_dispatch(const RowsDispatch& a, hipStream_t stream) {
    const int log = row_lanes_log(a.cols), per = kRowThreads >> log;
    const int64_t groups = (a.tokens + per - 1) / per;
    const dim3 grid(row_grid(groups), row_slices(groups, a.cols, log));
#define ROWS_DISPATCH(CODES, WIDE) \
    hipLaunchKernelGGL((rows_dispatch_kernel<CODES, WIDE>), grid, dim3(kRowThreads), 0, stream, a, log)
    if (a.codes) {
        if (log >= 6) ROWS_DISPATCH(true, true);
        else ROWS_DISPATCH(true, false);
    } else {
        if (log >= 6) ROWS_DISPATCH(false, true);
        else ROWS_DISPATCH(false, false);
    }
#undef ROWS_DISPATCH
}

// ---------------------------------------------------------------------------
// Combine
// ---------------------------------------------------------------------------

// The sum over a token's rows in fp32, choice by choice in ascending order, rounded
// once.  Eight rows' loads are in flight at a time.
template <bool kWide>
__global__ __launch_bounds__(kRowThreads) void rows_combine_kernel(RowsCombine a, int log) {
    const int lanes = 1 << log, per = kRowThreads >> log;
    const int lid = threadIdx.x & (lanes - 1);
    const int sub = kWide ? __builtin_amdgcn_readfirstlane(threadIdx.x >> log) : threadIdx.x >> log;
    const int nv = a.cols / kRowVec;
    for (int64_t t = (int64_t)blockIdx.x * per + sub; t < a.tokens; t += (int64_t)gridDim.x * per) {
        for (int p = blockIdx.y * lanes + lid; p < nv; p += gridDim.y * lanes) {
            const int64_t col = (int64_t)p * kRowVec;
            float sum[8] = {};
            if (a.add) unpack_bf16x8(*(const intx4*)(a.add + t * a.cols + col), sum);
            for (int j0 = 0; j0 < a.k; j0 += 8) {
                intx4 raw[8];
                float w[8];
                bool in[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    int64_t r = -1;
                    w[j] = 1.0f;
                    if (j0 + j < a.k) {
                        const int64_t at = t * a.k + j0 + j;
                        r = kWide ? ld_uniform(a.tok_row + at) : a.tok_row[at];
                        if (a.w) w[j] = kWide ? ld_uniform(a.w + at) : a.w[at];
                    }
                    in[j] = r >= 0 && r < a.rows;
                    raw[j] = intx4{0, 0, 0, 0};
                    if (in[j]) raw[j] = *(const intx4*)(a.src + r * a.cols + col);
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    float v[8];
                    unpack_bf16x8(raw[j], v);
                    if (in[j])  // (a missing row's weight may be a NaN)
#pragma unroll
                        for (int c = 0; c < 8; ++c) sum[c] = __builtin_fmaf(w[j], v[c], sum[c]);
                }
            }
            *(intx4*)(a.out + t * a.cols + col) = pack_bf16x8(sum);
        }
    }
}

void launch_rows_combine(const RowsCombine& a, hipStream_t stream) {
    const int log = row_lanes_log(a.cols), per = kRowThreads >> log;
    const int64_t groups = (a.tokens + per - 1) / per;
    const dim3 grid(row_grid(groups), row_slices(groups, a.cols, log));
    if (log >= 6) hipLaunchKernelGGL(rows_combine_kernel<true>, grid, dim3(kRowThreads), 0, stream, a, log);
    else hipLaunchKernelGGL(rows_combine_kernel<false>, grid, dim3(kRowThreads), 0, stream, a, log);
}

// ---------------------------------------------------------------------------
// Gradient of combine
// ---------------------------------------------------------------------------

// A token per group of lanes, its slices one after the other: the k dot products
// stay in registers over them and are joined once, in a fixed order.
template <int kK, bool kDot>
__global__ __launch_bounds__(kRowThreads) void rows_combine_bwd_kernel(RowsCombineBwd a, int log, int slices,
                                                                       int64_t units) {
    __shared__ float s_dot[kRowThreads / kWave][kK];
    const int lanes = 1 << log, per = kRowThreads >> log;
    const int lid = threadIdx.x & (lanes - 1), sub = threadIdx.x >> log;
    const int nv = a.cols / kRowVec;
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        const int64_t t = u * per + sub;
        const bool tok = t < a.tokens;
        int64_t r[kK];
        float w[kK], dot[kK];
#pragma unroll
        for (int j = 0; j < kK; ++j) {
            r[j] = tok && j < a.k ? (int64_t)a.tok_row[t * a.k + j] : -1;
            if (r[j] >= a.rows) r[j] = -1;
            w[j] = tok && j < a.k && a.w ? a.w[t * a.k + j] : 1.0f;
            dot[j] = 0.0f;
        }
        for (int s = 0; s < slices; ++s) {
            const int p = s * lanes + lid;
            const bool live = tok && p < nv;
            const int64_t at = (int64_t)p * kRowVec;
            float d[8] = {};
            intx4 raw[kK];
            if (kDot) {
#pragma unroll
                for (int j = 0; j < kK; ++j) {
                    raw[j] = intx4{0, 0, 0, 0};
                    if (live && r[j] >= 0) raw[j] = *(const intx4*)(a.src + r[j] * a.cols + at);
                }
            }
            if (live) unpack_bf16x8(*(const intx4*)(a.dout + t * a.cols + at), d);
#pragma unroll
            for (int j = 0; j < kK; ++j) {
                if (kDot) {
                    float v[8];
                    unpack_bf16x8(raw[j], v);
                    if (r[j] >= 0)
#pragma unroll
                        for (int c = 0; c < 8; ++c) dot[j] = __builtin_fmaf(v[c], d[c], dot[j]);
                }
                if (!a.dsrc && !a.codes) continue;
                float g[8];
#pragma unroll
                for (int c = 0; c < 8; ++c) g[c] = w[j] * d[c];
                const intx4 out = pack_bf16x8(g);
                const bool put = live && r[j] >= 0;
                if (a.dsrc && put) *(intx4*)(a.dsrc + r[j] * a.cols + at) = out;
                if (a.codes) {  // of the rounded gradient, as the quantiser of dsrc gives
                    unpack_bf16x8(out, g);
                    float m = put ? abs_max8(g) : 0.0f;
#pragma unroll
                    for (int x = 1; x < 16; x *= 2) m = fmaxf(m, __shfl_xor(m, x, kWave));
                    const int e = blk_exp(m);
                    if (put) {
                        *(uint64_t*)(a.codes + r[j] * a.cols + at) = blk_codes8(g, e);
                        if ((p & 15) == 0) a.scales[(int64_t)(p >> 4) * a.rows + r[j]] = pow2f(e);
                    }
                }
            }
        }
        if constexpr (kDot) {
            const int span = lanes < kWave ? lanes : kWave;
#pragma unroll
            for (int j = 0; j < kK; ++j)
                for (int s = span / 2; s >= 1; s >>= 1) dot[j] += __shfl_xor(dot[j], s, kWave);
            if (lanes > kWave) {  // one or two tokens' waves: joined in ascending order
                if ((threadIdx.x & 63) == 0)
#pragma unroll
                    for (int j = 0; j < kK; ++j) s_dot[threadIdx.x >> 6][j] = dot[j];
                __syncthreads();
                if (lid == 0)
#pragma unroll
                    for (int j = 0; j < kK; ++j) {
                        const int w0 = threadIdx.x >> 6;
                        float v = s_dot[w0][j];
                        for (int x = 1; x < lanes / kWave; ++x) v += s_dot[w0 + x][j];
                        dot[j] = v;
                    }
                __syncthreads();
            }
            if (tok && lid == 0)
#pragma unroll
                for (int j = 0; j < kK; ++j)
                    if (j < a.k) a.dw[t * a.k + j] = r[j] >= 0 ? dot[j] : 0.0f;
        }
    }
}

void launch_rows_combine_bwd(const RowsCombineBwd& a, hipStream_t stream) {
    const int log = row_lanes_log(a.cols), per = kRowThreads >> log;
    const int slices = (a.cols / kRowVec + (1 << log) - 1) >> log;
    const int64_t units = (a.tokens + per - 1) / per;
#define ROWS_BWD(K)                                                                                             \
    do {                                                                                                        \
        if (a.dw)                                                                                               \
            hipLaunchKernelGGL((rows_combine_bwd_kernel<K, true>), dim3(row_grid(units)), dim3(kRowThreads), 0, \
                               stream, a, log, slices, units);                                                  \
        else                                                                                                    \
            hipLaunchKernelGGL((rows_combine_bwd_kernel<K, false>), dim3(row_grid(units)), dim3(kRowThreads), 0, \
                               stream, a, log, slices, units);                                                  \
    } while (0)
    if (a.k <= 2) ROWS_BWD(2);
    else if (a.k <= 4) ROWS_BWD(4);
    else if (a.k <= 8) ROWS_BWD(8);
    else ROWS_BWD(16);
#undef ROWS_BWD
}

// ---------------------------------------------------------------------------
// Weights in blocks of 128 x 128, and back to bf16
// ---------------------------------------------------------------------------

constexpr int kBwPitch = kBlk + 16;  // bytes of a staged row of codes

// One 128 x 128 block per workgroup.  Thread (i, c), c = tid % 16, holds rows 8 i ..
// 8 i + 7 of the source and columns 8 c .. 8 c + 7.  A transposed source's 8 x 8
// values turn in registers: the eight codes of a column are eight neighbours of a
// row of the result, which leaves through LDS in whole lines.
template <bool kTransposed>
__global__ __launch_bounds__(kRowThreads) void block_quant_weights_kernel(const uint16_t* src, int n, int k,
                                                                          int64_t blocks, uint8_t* codes,
                                                                          float* scales) {
    __shared__ float s_max[kRowThreads / kWave];
    __shared__ __attribute__((aligned(16))) uint8_t s_q[kTransposed ? kBlk * kBwPitch : 16];
    const int nb = blk_count(n), kb = blk_count(k);
    const int rows = kTransposed ? k : n, cols = kTransposed ? n : k;  // of the source
    const int c = threadIdx.x & 15, i = threadIdx.x >> 4;
    for (int64_t b = blockIdx.x; b < blocks; b += gridDim.x) {
        const int64_t g = b / ((int64_t)nb * kb);
        const int in = (int)(b % ((int64_t)nb * kb));
        const int bn = in / kb, bk = in % kb;
        const int r0 = (kTransposed ? bk : bn) * kBlk + 8 * i, c0 = (kTransposed ? bn : bk) * kBlk + 8 * c;
        float v[8][8];
        float m = 0.0f;
#pragma unroll
        for (int x = 0; x < 8; ++x) {
            intx4 raw = {0, 0, 0, 0};
            if (r0 + x < rows && c0 < cols) raw = *(const intx4*)(src + (g * rows + r0 + x) * cols + c0);
            unpack_bf16x8(raw, v[x]);
            m = fmaxf(m, abs_max8(v[x]));
        }
#pragma unroll
        for (int s = 1; s < kWave; s *= 2) m = fmaxf(m, __shfl_xor(m, s, kWave));
        if ((threadIdx.x & 63) == 0) s_max[threadIdx.x >> 6] = m;
        __syncthreads();
        m = fmaxf(fmaxf(s_max[0], s_max[1]), fmaxf(s_max[2], s_max[3]));
        const int e = blk_exp(m);
        if (threadIdx.x == 0) scales[b] = pow2f(e);
        uint8_t* dst = codes + (g * n + (int64_t)bn * kBlk) * k + bk * kBlk;
        if constexpr (!kTransposed) {
#pragma unroll
            for (int x = 0; x < 8; ++x)
                if (r0 + x < rows && c0 < cols) *(uint64_t*)(dst + (int64_t)(8 * i + x) * k + 8 * c) = blk_codes8(v[x], e);
            __syncthreads();  // s_max is read
        } else {
#pragma unroll
            for (int y = 0; y < 8; ++y) {
                float col[8];
#pragma unroll
                for (int x = 0; x < 8; ++x) col[x] = v[x][y];
                *(uint64_t*)(s_q + (8 * c + y) * kBwPitch + 8 * i) = blk_codes8(col, e);
            }
            __syncthreads();
            for (int x = threadIdx.x; x < kBlk * 8; x += kRowThreads) {
                const int row = x >> 3, at = (x & 7) * 16;
                if (bn * kBlk + row < n && bk * kBlk + at < k)
                    *(intx4*)(dst + (int64_t)row * k + at) = *(const intx4*)(s_q + row * kBwPitch + at);
            }
            __syncthreads();
        }
    }
}

void launch_block_quant_weights(const uint16_t* src, int groups, int n, int k, int transposed, uint8_t* codes,
                                float* scales, hipStream_t stream) {
    const int64_t blocks = (int64_t)groups * blk_count(n) * blk_count(k);
    if (transposed)
        hipLaunchKernelGGL(block_quant_weights_kernel<true>, dim3(row_grid(blocks)), dim3(kRowThreads), 0, stream, src, n,
                           k, blocks, codes, scales);
    else
        hipLaunchKernelGGL(block_quant_weights_kernel<false>, dim3(row_grid(blocks)), dim3(kRowThreads), 0, stream, src,
                           n, k, blocks, codes, scales);
}

// Sixteen codes a thread, 16 << log columns of a workgroup's rows.  The scale of row
// r's block b: scales[b][r], or with a matrix of n rows that of its 128 x 128 block,
// [matrix][n / 128][b].
__global__ __launch_bounds__(kRowThreads) void block_dequant_kernel(const uint8_t* codes, const float* scales,
                                                                    int64_t rows, int cols, uint32_t n, uint16_t* dst,
                                                                    int log) {
    const int lanes = 1 << log, per = kRowThreads >> log;
    const int lid = threadIdx.x & (lanes - 1), sub = threadIdx.x >> log;
    const int c = (blockIdx.y * lanes + lid) * 16, b = c / kBlk;
    if (c >= cols) return;  // no barrier follows
    for (int64_t r = (int64_t)blockIdx.x * per + sub; r < rows; r += (int64_t)gridDim.x * per) {
        float s;
        if (n) {
            const uint32_t g = (uint32_t)r / n, in = (uint32_t)r - g * n;
            s = scales[((int64_t)g * blk_count(n) + in / kBlk) * blk_count(cols) + b];
        } else {
            s = scales[b * rows + r];
        }
        const int64_t at = r * cols + c;
        const intx4 q = *(const intx4*)(codes + at);
        float v[2][8];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int d = 0; d < 2; ++d) {
                const uint32_t w = (uint32_t)q[2 * h + d];
                v[h][4 * d] = __builtin_amdgcn_cvt_f32_fp8(w, 0) * s;
                v[h][4 * d + 1] = __builtin_amdgcn_cvt_f32_fp8(w, 1) * s;
                v[h][4 * d + 2] = __builtin_amdgcn_cvt_f32_fp8(w, 2) * s;
                v[h][4 * d + 3] = __builtin_amdgcn_cvt_f32_fp8(w, 3) * s;
            }
        *(intx4*)(dst + at) = pack_bf16x8(v[0]);
        *(intx4*)(dst + at + 8) = pack_bf16x8(v[1]);
    }
}

void launch_block_dequant(const uint8_t* codes, const float* scales, int64_t rows, int cols, int n, uint16_t* dst,
                          hipStream_t stream) {
    int log = 3;
    while (log < 8 && (16 << log) < cols) ++log;
    const int per = kRowThreads >> log;
    const dim3 grid(row_grid((rows + per - 1) / per), (unsigned)((cols / 16 + (1 << log) - 1) >> log));
    hipLaunchKernelGGL(block_dequant_kernel, grid, dim3(kRowThreads), 0, stream, codes, scales, rows, cols, (uint32_t)n,
                       dst, log);
}

}  // namespace moe
