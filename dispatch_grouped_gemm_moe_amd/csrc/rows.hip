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
#include <algorithm>

#include "block8.hpp"
#include "common.hpp"
#include "kernels.hpp"

namespace moe {

#pragma clang fp contract(off)

constexpr int kRowThreads = 256;
constexpr int kRowVec = 8;

// Threads that share a token: a power of two from 16 (a block of 128) to the
// workgroup, so that narrow rows stand side by side in a workgroup.
static int row_lanes_log(int cols, int vec = kRowVec) {
    const int nv = (cols + vec - 1) / vec;
    int s = 4;
    while (s < 8 && (1 << s) < nv) ++s;
    return s;
}

static unsigned row_grid(int64_t units) { return (unsigned)(units < (1 << 22) ? units : (1 << 22)); }

// Workgroups that share a token's columns: one where the tokens alone fill the CUs,
// which then reads the token's table once.
static unsigned row_slices(int64_t groups, int cols, int log, int vec = kRowVec) {
    const int slices = (cols / vec + (1 << log) - 1) >> log;
    return (unsigned)(groups >= 2048 ? 1 : slices);
}

// Loads and stores of rows; kStream: the rows are more than the last cache's 256 MB, so
// they leave the caches to others.  (16384 tokens of 7168 and 8 rows each, 1.9 GB of rows:
// combine 421 -> 365 us, its gradient 764 -> 751, dispatch 412 -> 404; but 20000 tokens of
// 128 and 4 rows each, 20 MB: combine 7.7 -> 9.4.)
template <bool kStream>
__device__ __forceinline__ intx4 ld_row(const void* p) {
    if (kStream) return __builtin_nontemporal_load((const intx4*)p);
    return *(const intx4*)p;
}
template <bool kStream>
__device__ __forceinline__ void st_row(void* p, intx4 v) {
    if (kStream) __builtin_nontemporal_store(v, (intx4*)p);
    else *(intx4*)p = v;
}
static bool streams(int64_t rows, int64_t row_bytes) { return rows * row_bytes > (256ll << 20); }

// An entry of a table that no kernel changes while it is read, of a token that is the
// same in the whole wave: a scalar load.
template <class T>
__device__ __forceinline__ T ld_uniform(const T* p) {
    return *(const __attribute__((address_space(4))) T*)p;
}

// ---------------------------------------------------------------------------
// Dispatch
// ---------------------------------------------------------------------------

// Measured: 16384 tokens of 7168 to 8 rows each 405 us (5.2 TB/s, mostly writes), as codes
// 299 us (3.9 TB/s: scales of neighbouring rows are written by different XCDs), as both 1061
// us (2.9 TB/s: a thread's two stores of bf16 each skip every other 16 bytes, past the caches),
// more than the two calls.
//
// A workgroup takes kRowThreads >> log tokens at a time.  A thread has eight
// consecutive values, or with codes sixteen, which leave as 16 bytes; a block's eight
// lanes share its maximum.  kWide: one wave's lanes share a token.
template <bool kCodes, bool kWide, bool kStream>
__global__ __launch_bounds__(kRowThreads) void rows_dispatch_kernel(RowsDispatch a, int log) {
    constexpr int kParts = kCodes ? 2 : 1, kVec = kParts * kRowVec;
    const int lanes = 1 << log, per = kRowThreads >> log;
    const int lid = threadIdx.x & (lanes - 1);
    const int sub = kWide ? __builtin_amdgcn_readfirstlane(threadIdx.x >> log) : threadIdx.x >> log;
    const int nv = a.cols / kVec;
    int64_t t_lo = 0, t_hi = a.tokens;
    if (a.offsets) {
        // (a last bound below the one before it, as moe_dispatch_layout's error report: no row in
        // the last group, as for the products)
        t_lo = max(a.offsets[0], 0);
        t_hi = min((int64_t)max(a.offsets[a.groups - 1], a.offsets[a.groups]), a.tokens);
    }
    for (int64_t t0 = (int64_t)blockIdx.x * per; t0 < t_hi; t0 += (int64_t)gridDim.x * per) {
        const int64_t t = t0 + sub;
        const bool tok = t >= t_lo && t < t_hi;
        for (int p = blockIdx.y * lanes + lid; (p & ~7) < nv; p += gridDim.y * lanes) {  // whole blocks
            const bool live = tok && p < nv;
            const int64_t col = (int64_t)p * kVec;
            intx4 raw[kParts] = {};
            float v[kParts][8] = {};  // past the row's end: zeros
            if (live) {
                if (kCodes && a.xf) {
#pragma unroll
                    for (int h = 0; h < kParts; ++h)
#pragma unroll
                        for (int c = 0; c < 8; c += 4) {
                            const floatx4 f = *(const floatx4*)(a.xf + t * a.cols + col + 8 * h + c);
#pragma unroll
                            for (int x = 0; x < 4; ++x) v[h][c + x] = f[x];
                        }
                } else {
#pragma unroll
                    for (int h = 0; h < kParts; ++h) raw[h] = *(const intx4*)(a.x + t * a.cols + col + 8 * h);
                }
            }
            intx4 q = {0, 0, 0, 0};
            float scale = 0.0f;
            if constexpr (kCodes) {
                if (!a.xf) {
#pragma unroll
                    for (int h = 0; h < kParts; ++h) unpack_bf16x8(raw[h], v[h]);
                }
                float m = fmaxf(abs_max8(v[0]), abs_max8(v[kParts - 1]));
#pragma unroll
                for (int s = 1; s < 8; s *= 2) m = fmaxf(m, __shfl_xor(m, s, kWave));
                const int e = blk_exp(m);
                scale = pow2f(e);
#pragma unroll
                for (int h = 0; h < kParts; ++h) {
                    const uint64_t c8 = blk_codes8(v[h], e);
                    q[2 * h] = (int)(uint32_t)c8;
                    q[2 * h + 1] = (int)(uint32_t)(c8 >> 32);
                    if (a.xf) raw[h] = pack_bf16x8(v[h]);
                }
            }
            if (!live) continue;
            for (int j = 0; j < a.k; ++j) {
                const int32_t* at = a.tok_row + t * a.k + j;
                const int64_t r = !a.tok_row ? t : kWide ? ld_uniform(at) : *at;
                if (r < 0 || r >= a.rows) continue;  // no row
                if (a.dst) {
#pragma unroll
                    for (int h = 0; h < kParts; ++h) st_row<kStream>(a.dst + r * a.cols + col + 8 * h, raw[h]);
                }
                if constexpr (kCodes) {
                    st_row<kStream>(a.codes + r * a.cols + col, q);
                    if ((p & 7) == 0) a.scales[(int64_t)(p >> 3) * a.rows + r] = scale;
                }
            }
        }
    }
}

void launch_rows_dispatch(const RowsDispatch& a, hipStream_t stream) {
    const int vec = a.codes ? 2 * kRowVec : kRowVec;
    const int log = row_lanes_log(a.cols, vec), per = kRowThreads >> log;
    const int64_t groups = (a.tokens + per - 1) / per;
    const dim3 grid(row_grid(groups), row_slices(groups, a.cols, log, vec));
    const bool big = streams(a.rows, (int64_t)a.cols * ((a.dst ? 2 : 0) + (a.codes ? 1 : 0)));
#define ROWS_DISPATCH(CODES, WIDE, STREAM) \
    hipLaunchKernelGGL((rows_dispatch_kernel<CODES, WIDE, STREAM>), grid, dim3(kRowThreads), 0, stream, a, log)
#define ROWS_DISPATCH2(CODES, WIDE)                  \
    do {                                             \
        if (big) ROWS_DISPATCH(CODES, WIDE, true);   \
        else ROWS_DISPATCH(CODES, WIDE, false);      \
    } while (0)
    if (a.codes) {
        if (log >= 6) ROWS_DISPATCH2(true, true);
        else ROWS_DISPATCH2(true, false);
    } else {
        if (log >= 6) ROWS_DISPATCH2(false, true);
        else ROWS_DISPATCH2(false, false);
    }
#undef ROWS_DISPATCH2
#undef ROWS_DISPATCH
}

// ---------------------------------------------------------------------------
// The quantiser of rows
// ---------------------------------------------------------------------------

// A workgroup takes kC blocks next to each other of 32 / kC rows, eight lanes to a block and
// sixteen values to a lane, so that no width leaves lanes idle but in its last blocks, and the
// scales of neighbouring rows are written together.  Four blocks where they divide the row, one
// where it has just one, else two.  (us, kC of 1, 2, 4 and, before, a workgroup to a row:
// 131072 x 7168 547, 503, 488 (5.8 TB/s), 504; 8191 x 4112 25.4, 21.5, 23.4, 22.3; 24576 x 2048
// 26.0, 25.5, 26.2, 29.3; 64 x 7168 3.4, 3.4, 3.4, 4.0; 80000 x 128 6.8, 7.5, 10.9, 8.7.)
template <int kC, bool kStream>
__global__ __launch_bounds__(kRowThreads) void block_quant_kernel(const uint16_t* x, int64_t rows, int cols,
                                                                  uint8_t* codes, float* scales) {
    constexpr int kR = kRowThreads / 8 / kC;
    const int lid = threadIdx.x & 7, kb = blockIdx.x * kC + (threadIdx.x >> 3) % kC;
    const int col = kb * kBlk + lid * 16;
    if (kb * kBlk >= cols) return;  // a whole block; no barrier follows
    for (int64_t r = (int64_t)blockIdx.y * kR + (threadIdx.x >> 3) / kC; r < rows; r += (int64_t)gridDim.y * kR) {
        const int64_t at = r * cols + col;
        float v[2][8] = {};  // past the row's end: zeros
        if (col < cols) {
            unpack_bf16x8(ld_row<kStream>(x + at), v[0]);
            unpack_bf16x8(ld_row<kStream>(x + at + 8), v[1]);
        }
        float m = fmaxf(abs_max8(v[0]), abs_max8(v[1]));
#pragma unroll
        for (int s = 1; s < 8; s *= 2) m = fmaxf(m, __shfl_xor(m, s, kWave));
        const int e = blk_exp(m);
        if (lid == 0) scales[(int64_t)kb * rows + r] = pow2f(e);
        if (col < cols) {
            const uint64_t lo = blk_codes8(v[0], e), hi = blk_codes8(v[1], e);
            st_row<kStream>(codes + at, intx4{(int)(uint32_t)lo, (int)(uint32_t)(lo >> 32), (int)(uint32_t)hi,
                                              (int)(uint32_t)(hi >> 32)});
        }
    }
}

template <int kC>
static void launch_block_quant(const uint16_t* x, int64_t rows, int cols, uint8_t* codes, float* scales,
                               hipStream_t stream) {
    constexpr int kR = kRowThreads / 8 / kC;
    const dim3 grid((blk_count(cols) + kC - 1) / kC, (unsigned)std::min<int64_t>((rows + kR - 1) / kR, 65535));
    if (streams(rows, 2ll * cols))
        hipLaunchKernelGGL((block_quant_kernel<kC, true>), grid, dim3(kRowThreads), 0, stream, x, rows, cols, codes, scales);
    else
        hipLaunchKernelGGL((block_quant_kernel<kC, false>), grid, dim3(kRowThreads), 0, stream, x, rows, cols, codes, scales);
}

void launch_block_quant(const uint16_t* x, int64_t rows, int cols, uint8_t* codes, float* scales, hipStream_t stream) {
    const int nb = blk_count(cols);
    if (nb == 1) launch_block_quant<1>(x, rows, cols, codes, scales, stream);
    else if (nb % 4 == 0) launch_block_quant<4>(x, rows, cols, codes, scales, stream);
    else launch_block_quant<2>(x, rows, cols, codes, scales, stream);
}

// ---------------------------------------------------------------------------
// Combine
// ---------------------------------------------------------------------------

// The sum over a token's rows in fp32, choice by choice in ascending order, rounded
// once.  Eight rows' loads are in flight at a time.  16384 tokens of 7168 from 8 rows each:
// 366 us (5.8 TB/s).
template <bool kWide, bool kStream>
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
                    if (in[j]) raw[j] = ld_row<kStream>(a.src + r * a.cols + col);
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
#define ROWS_COMBINE(WIDE, STREAM) \
    hipLaunchKernelGGL((rows_combine_kernel<WIDE, STREAM>), grid, dim3(kRowThreads), 0, stream, a, log)
    if (log < 6) ROWS_COMBINE(false, false);
    else if (streams(a.rows, 2ll * a.cols)) ROWS_COMBINE(true, true);
    else ROWS_COMBINE(true, false);
#undef ROWS_COMBINE
}

// ---------------------------------------------------------------------------
// Gradient of combine
// ---------------------------------------------------------------------------

// A token per group of 1 << log lanes, its columns in one go or one piece after the other:
// the k dot products stay in registers over them and are joined once, in a fixed order.
// kWide: one wave's lanes share a token, and its table's entries are scalars.  16384 tokens
// of 7168 from 8 rows each: 766 us (5.2 TB/s); as codes alone 319 (3.8 TB/s), as codes with dw
// 653 (4.7), with all three 1031 (4.8).
template <int kK, bool kDot, bool kWide, bool kStream, int kThreads>
__global__ __launch_bounds__(kThreads) void rows_combine_bwd_kernel(RowsCombineBwd a, int log, int64_t units) {
    __shared__ float s_dot[kThreads / kWave][kK];
    const int lanes = 1 << log, per = kThreads >> log;
    const int lid = threadIdx.x & (lanes - 1);
    const int sub = kWide ? __builtin_amdgcn_readfirstlane(threadIdx.x >> log) : threadIdx.x >> log;
    const int nv = a.cols / kRowVec;
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        const int64_t t = u * per + sub;
        const bool tok = t < a.tokens;
        for (int j0 = 0; j0 < a.k; j0 += kK) {  // kK choices at a time
            int r[kK];
            float w[kK], dot[kK];
#pragma unroll
            for (int j = 0; j < kK; ++j) {
                r[j] = -1;
                w[j] = 1.0f;
                if (tok && j0 + j < a.k) {
                    const int64_t at = t * a.k + j0 + j;
                    r[j] = kWide ? ld_uniform(a.tok_row + at) : a.tok_row[at];
                    if (r[j] >= a.rows) r[j] = -1;
                    if (a.w) w[j] = kWide ? ld_uniform(a.w + at) : a.w[at];
                }
                dot[j] = 0.0f;
            }
            for (int p = lid; (p & ~15) < nv; p += lanes) {  // whole blocks: their lanes share a maximum
                const bool live = tok && p < nv;
                const int64_t col = (int64_t)p * kRowVec;
                float d[8] = {};
                intx4 raw[kK];
                if (kDot) {
#pragma unroll
                    for (int j = 0; j < kK; ++j) {
                        raw[j] = intx4{0, 0, 0, 0};
                        if (live && r[j] >= 0) raw[j] = ld_row<kStream>(a.src + (int64_t)r[j] * a.cols + col);
                    }
                }
                if (live) unpack_bf16x8(*(const intx4*)(a.dout + t * a.cols + col), d);
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
                    const int64_t at = (int64_t)r[j] * a.cols + col;
                    if (a.dsrc && put) st_row<kStream>(a.dsrc + at, out);
                    if (a.codes) {  // of the rounded gradient, as the quantiser of dsrc gives
                        unpack_bf16x8(out, g);
                        float m = put ? abs_max8(g) : 0.0f;
#pragma unroll
                        for (int x = 1; x < 16; x *= 2) m = fmaxf(m, __shfl_xor(m, x, kWave));
                        const int e = blk_exp(m);
                        if (put) {
                            *(uint64_t*)(a.codes + at) = blk_codes8(g, e);
                            if ((p & 15) == 0) a.scales[(int64_t)(p >> 4) * a.rows + r[j]] = pow2f(e);
                        }
                    }
                }
            }
            if constexpr (kDot) {
                const int span = lanes < kWave ? lanes : kWave;
                for (int s = span / 2; s >= 1; s >>= 1)  // (the k exchanges of a step overlap)
#pragma unroll
                    for (int j = 0; j < kK; ++j) dot[j] += __shfl_xor(dot[j], s, kWave);
                if (lanes > kWave) {  // several waves to a token: joined in ascending order
                    if ((threadIdx.x & 63) == 0)
#pragma unroll
                        for (int j = 0; j < kK; ++j) s_dot[threadIdx.x >> 6][j] = dot[j];
                    __syncthreads();
                    if (lid < kK && j0 + lid < a.k) {  // a lane to a choice
                        const int w0 = threadIdx.x >> 6;
                        float v = s_dot[w0][lid];
                        for (int x = 1; x < lanes / kWave; ++x) v += s_dot[w0 + x][lid];
                        if (tok) {
                            const int64_t at = t * a.k + j0 + lid;
                            const int rj = a.tok_row[at];
                            a.dw[at] = rj >= 0 && rj < a.rows ? v : 0.0f;
                        }
                    }
                    __syncthreads();
                } else if (tok && lid == 0) {
#pragma unroll
                    for (int j = 0; j < kK; ++j)
                        if (j0 + j < a.k) a.dw[t * a.k + j0 + j] = r[j] >= 0 ? dot[j] : 0.0f;
                }
            }
        }
    }
}

template <int kK, bool kWide, bool kStream, int kThreads>
static void launch_rows_bwd(const RowsCombineBwd& a, int log, hipStream_t stream) {
    const int per = kThreads >> log;
    const int64_t units = (a.tokens + per - 1) / per;
    const dim3 grid(row_grid(units));
    if (a.dw)
        hipLaunchKernelGGL((rows_combine_bwd_kernel<kK, true, kWide, kStream, kThreads>), grid, dim3(kThreads), 0, stream, a,
                           log, units);
    else
        hipLaunchKernelGGL((rows_combine_bwd_kernel<kK, false, kWide, kStream, kThreads>), grid, dim3(kThreads), 0, stream,
                           a, log, units);
}

template <int kK>
static void launch_rows_bwd(const RowsCombineBwd& a, hipStream_t stream) {
    const int log = row_lanes_log(a.cols);
    // few tokens of wide rows: 1024 threads to a token, which then waits for its rows once (64
    // tokens of 7168 from 8 rows 16.0 -> 11.5 us; 4096 fill the CUs either way)
    if (a.cols > kRowThreads * kRowVec && a.tokens < 1024) launch_rows_bwd<kK, true, false, 1024>(a, 10, stream);
    else if (log < 6) launch_rows_bwd<kK, false, false, kRowThreads>(a, log, stream);
    else if (streams(a.rows, 4ll * a.cols)) launch_rows_bwd<kK, true, true, kRowThreads>(a, log, stream);
    else launch_rows_bwd<kK, true, false, kRowThreads>(a, log, stream);
}

void launch_rows_combine_bwd(const RowsCombineBwd& a, hipStream_t stream) {
    if (a.k <= 2) launch_rows_bwd<2>(a, stream);
    else if (a.k <= 4) launch_rows_bwd<4>(a, stream);
    else launch_rows_bwd<8>(a, stream);
}

// ---------------------------------------------------------------------------
// Weights in blocks of 128 x 128, and back to bf16
// ---------------------------------------------------------------------------

constexpr int kBwPitch = kBlk + 16;  // bytes of a staged row of codes

// One 128 x 128 block per workgroup.  Thread (i, c), c = tid % 16, holds rows 8 i ..
// 8 i + 7 of the source and columns 8 c .. 8 c + 7.  A transposed source's 8 x 8
// values turn in registers: the eight codes of a column are eight neighbours of a
// row of the result, which leaves through LDS in whole lines.  32 matrices of [2048, 7168]:
// 248 us, turned 250 (5.65 TB/s).
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
            if (r0 + x < rows && c0 < cols) raw = ld_row<true>(src + (g * rows + r0 + x) * cols + c0);
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
                    st_row<true>(dst + (int64_t)row * k + at, *(const intx4*)(s_q + row * kBwPitch + at));
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

// Eight codes a thread, whose 16 bytes of values stand next to its neighbours' (sixteen: the
// two stores of a wave each skip every other 16 bytes, 267 -> 277 us for 32 matrices of [2048,
// 7168]), and 8 << log columns of a workgroup's rows.  The scale of row r's block b:
// scales[b][r], or with a matrix of n rows that of its 128 x 128 block, [matrix][n / 128][b].
// kStream as in ld_row, by the size of dst: those matrices 267 -> 245 us (5.7 TB/s), 131072
// rows of 7168 525 -> 503; but 8191 rows of 4112 19.2 -> 24.7.
template <bool kStream>
__global__ __launch_bounds__(kRowThreads) void block_dequant_kernel(const uint8_t* codes, const float* scales,
                                                                    int64_t rows, int cols, uint32_t n, uint16_t* dst,
                                                                    int log) {
    const int lanes = 1 << log, per = kRowThreads >> log;
    const int lid = threadIdx.x & (lanes - 1), sub = threadIdx.x >> log;
    const int c = (blockIdx.y * lanes + lid) * 8, b = c / kBlk;
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
        typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
        const u32x2 q = kStream ? __builtin_nontemporal_load((const u32x2*)(codes + at)) : *(const u32x2*)(codes + at);
        float v[8];
#pragma unroll
        for (int d = 0; d < 2; ++d) {
            const uint32_t w = q[d];
            v[4 * d] = __builtin_amdgcn_cvt_f32_fp8(w, 0) * s;
            v[4 * d + 1] = __builtin_amdgcn_cvt_f32_fp8(w, 1) * s;
            v[4 * d + 2] = __builtin_amdgcn_cvt_f32_fp8(w, 2) * s;
            v[4 * d + 3] = __builtin_amdgcn_cvt_f32_fp8(w, 3) * s;
        }
        st_row<kStream>(dst + at, pack_bf16x8(v));
    }
}

void launch_block_dequant(const uint8_t* codes, const float* scales, int64_t rows, int cols, int n, uint16_t* dst,
                          hipStream_t stream) {
    int log = 4;
    while (log < 8 && (8 << log) < cols) ++log;
    const int per = kRowThreads >> log;
    const dim3 grid(row_grid((rows + per - 1) / per), (unsigned)((cols / 8 + (1 << log) - 1) >> log));
    if (streams(rows, 2ll * cols))
        hipLaunchKernelGGL(block_dequant_kernel<true>, grid, dim3(kRowThreads), 0, stream, codes, scales, rows, cols,
                           (uint32_t)n, dst, log);
    else
        hipLaunchKernelGGL(block_dequant_kernel<false>, grid, dim3(kRowThreads), 0, stream, codes, scales, rows, cols,
                           (uint32_t)n, dst, log);
}

}  // namespace moe
