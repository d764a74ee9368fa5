// The whole MoE layer for a few tokens (gfx950): 1 to kFewTokens tokens, as a
// server decodes them.
//
//   z = x Wr + b,  S = top-k(z),  w = softmax(z_S)
//   h_e = silu(x Wg_e) * (x Wu_e),  out = sum_{e in S} w_e h_e Wd_e (+ shared)
//
// With so few rows per expert every product is a matrix times a handful of
// vectors: what bounds the layer is reading the chosen experts' weights from
// HBM once (3 H I values per expert), not arithmetic.  The tiles of the layer
// kernel spend 128 padded rows per expert; here the weight rows are the M side
// of 16-wide MFMAs and the expert's tokens the N side, so 16 tokens ride on
// every weight fragment and nothing is padded past 16 rows.
//
// Four launches: router (logits, top-k, expert row lists), gate|up with SwiGLU,
// down, and the weighted sum.
#include "common.hpp"
#include "kernels.hpp"
#include "mxfp8.hpp"

namespace moe {

#pragma clang fp contract(off)

// ---------------------------------------------------------------------------
// Router
// ---------------------------------------------------------------------------

constexpr int kFrThreads = 512;
constexpr int kFrEC = 4;         // experts per workgroup
constexpr int kFrTok = 16;       // tokens per workgroup, two per wave
constexpr int kFrSlab = 2048;    // h per LDS slab
constexpr int kFrWL = kFrSlab / kFrThreads;                   // weight rows (16 bytes) per thread and slab
constexpr int kFrXL = kFrTok * kFrSlab / 8 / kFrThreads;      // 16-byte pieces of x per thread and slab

__device__ __forceinline__ float tree64(float v) {
    // halving tree p[l] += p[l+s], s = 32, 16, ..., 1 (the result is lane 0's)
#pragma unroll
    for (int s = 32; s >= 1; s >>= 1) v = v + __shfl_xor(v, s, kWave);
    return v;
}

// Top-k of every token and the experts' row lists, by the workgroup that
// finishes the logits last.  At most 64 tokens: an expert's tokens are one
// 64-bit mask, a row's rank within its expert a population count.
__device__ void few_layout(const FewRoute& a, uint64_t* s_mask, int* s_idx, float* s_w, int* s_off) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int T = a.T, E = a.E, k = a.k;
    for (int e = tid; e < kMaxExperts; e += kFrThreads) s_mask[e] = 0;
    __syncthreads();
    for (int t = wave; t < T; t += kFrThreads / kWave) {
        float v[kMaxExperts / kWave];
        unsigned taken = 0;
#pragma unroll
        for (int q = 0; q < kMaxExperts / kWave; ++q) {
            const int e = lane + q * kWave;
            // written by other workgroups of this launch: read past this XCD's cache
            v[q] = e < E ? __hip_atomic_load(a.logits + (size_t)t * E + e, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT)
                         : 0.0f;
            // a NaN compares with nothing: as the lowest value the order stays
            // total, so every lane picks the same k distinct experts
            if (v[q] != v[q]) v[q] = -INFINITY;
            if (e >= E) taken |= 1u << q;
        }
        float first = 0.0f, den = 0.0f, ez = 0.0f;
        int mine = -1;  // lane j keeps selection j
        for (int j = 0; j < k; ++j) {
            float bv = 0.0f;
            int bi = 0x7fffffff;
#pragma unroll
            for (int q = 0; q < kMaxExperts / kWave; ++q)
                if (!(taken & (1u << q)) && (bi == 0x7fffffff || v[q] > bv)) { bv = v[q]; bi = lane + q * kWave; }
#pragma unroll
            for (int s = 32; s >= 1; s >>= 1) {
                const float ov = __shfl_xor(bv, s, kWave);
                const int oi = __shfl_xor(bi, s, kWave);
                if (oi != 0x7fffffff && (bi == 0x7fffffff || ov > bv || (ov == bv && oi < bi))) { bv = ov; bi = oi; }
            }
            if (j == 0) first = bv;
            const float z = expf(bv - first);
            den = den + z;
            if (lane == j) { mine = bi; ez = z; }
            if ((bi & (kWave - 1)) == lane) taken |= 1u << (bi / kWave);
        }
        if (lane < k) {
            s_idx[t * k + lane] = mine;
            s_w[t * k + lane] = ez / den;
            atomicOr((unsigned long long*)&s_mask[mine], 1ull << t);
        }
    }
    __syncthreads();
    // exclusive prefix of rows and of active experts over the experts (wave 0)
    if (wave == 0) {
        int rows = 0, act = 0;
        for (int e0 = 0; e0 < E; e0 += kWave) {
            const int e = e0 + lane;
            const int c = e < E ? __popcll(s_mask[e]) : 0;
            int inc = c;
#pragma unroll
            for (int s = 1; s < kWave; s <<= 1) {
                const int o = __shfl_up(inc, s, kWave);
                if (lane >= s) inc += o;
            }
            const uint64_t on = __ballot(c > 0);
            const int at = act + __popcll(on & ((1ull << lane) - 1ull));
            if (e < E) s_off[e] = rows + inc - c;
            if (c > 0) {
                a.act_e[at] = e;
                a.act_off[at] = rows + inc - c;
            }
            rows += __shfl(inc, kWave - 1, kWave);
            act += __popcll(on);
        }
        if (lane == 0) {
            if (a.shared) {  // the shared expert takes every token, after the routed rows
                a.act_e[act] = E;
                a.act_off[act] = rows;
                ++act;
                rows += T;
            }
            a.act_off[act] = rows;
            *a.n_act = act;
        }
    }
    __syncthreads();
    for (int i = tid; i < T * k; i += kFrThreads) {
        const int t = i / k, e = s_idx[i];
        const int row = s_off[e] + __popcll(s_mask[e] & ((1ull << t) - 1ull));
        a.row_token[row] = t;
        a.row_w[row] = s_w[i];
        a.slot_row[i] = row;
    }
    if (a.shared)
        for (int t = tid; t < T; t += kFrThreads) {
            a.row_token[T * k + t] = t;
            a.row_w[T * k + t] = 1.0f;
        }
}

// Workgroup (x, y): experts 4x .. 4x+3 for tokens 16y .. 16y+15.  The logits'
// order is moe_route's: lane l sums h = l, l + 64, ... with fused
// multiply-adds, then the halving tree, then the bias.  Slabs of kFrSlab rows
// of the router weight and of the tokens go through LDS, the next slab's loads
// in flight while one is summed.
template <bool kVec4>
__global__ __launch_bounds__(kFrThreads) void few_route_kernel(FewRoute a) {
    __shared__ __attribute__((aligned(16))) float s_wr[kFrSlab][kFrEC];
    __shared__ __attribute__((aligned(16))) uint16_t s_x[kFrTok][kFrSlab];
    __shared__ int s_last;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int e0 = blockIdx.x * kFrEC, t0 = blockIdx.y * kFrTok;
    const int T = a.T, H = a.H, E = a.E;
    const int nt = min(kFrTok, T - t0);
    floatx4 wn[kFrWL];
    intx4 xn[kFrXL];
    auto load = [&](int h0) {
#pragma unroll
        for (int i = 0; i < kFrWL; ++i) {
            const int h = h0 + i * kFrThreads + tid;
            floatx4 v = {0, 0, 0, 0};
            if (h < H) {
                const float* p = a.Wr + (size_t)h * E + e0;
                if (kVec4) {
                    v = *(const floatx4*)p;
                } else {
#pragma unroll
                    for (int q = 0; q < kFrEC; ++q) v[q] = e0 + q < E ? p[q] : 0.0f;
                }
            }
            wn[i] = v;
        }
#pragma unroll
        for (int i = 0; i < kFrXL; ++i) {
            const int p = i * kFrThreads + tid;  // 16-byte piece of the slab: token p / 256
            const int t = p / (kFrSlab / 8), h = h0 + (p % (kFrSlab / 8)) * 8;
            intx4 v = {0, 0, 0, 0};
            if (t < nt && h < H) v = *(const intx4*)(a.x + (size_t)(t0 + t) * H + h);
            xn[i] = v;
        }
    };
    float acc[2][kFrEC] = {};
    load(0);
    for (int h0 = 0; h0 < H; h0 += kFrSlab) {
        __syncthreads();  // the previous slab is summed
#pragma unroll
        for (int i = 0; i < kFrWL; ++i) *(floatx4*)s_wr[i * kFrThreads + tid] = wn[i];
#pragma unroll
        for (int i = 0; i < kFrXL; ++i) {
            const int p = i * kFrThreads + tid;
            *(intx4*)&s_x[p / (kFrSlab / 8)][(p % (kFrSlab / 8)) * 8] = xn[i];
        }
        __syncthreads();
        if (h0 + kFrSlab < H) load(h0 + kFrSlab);
        if (wave * 2 < nt) {
            const int nc = min(kFrSlab, H - h0) / kWave;
#pragma unroll 4
            for (int c = 0; c < nc; ++c) {
                const floatx4 w4 = *(const floatx4*)s_wr[c * kWave + lane];
                const float x0 = bf16_to_f32(s_x[wave * 2][c * kWave + lane]);
                const float x1 = bf16_to_f32(s_x[wave * 2 + 1][c * kWave + lane]);
#pragma unroll
                for (int q = 0; q < kFrEC; ++q) {
                    acc[0][q] = __builtin_fmaf(x0, w4[q], acc[0][q]);
                    acc[1][q] = __builtin_fmaf(x1, w4[q], acc[1][q]);
                }
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int t = t0 + wave * 2 + i;
        if (wave * 2 + i >= nt) break;
#pragma unroll
        for (int q = 0; q < kFrEC; ++q) {
            float v = tree64(acc[i][q]);
            if (lane == 0 && e0 + q < E) {
                if (a.bias) v = v + a.bias[e0 + q];
                __hip_atomic_store(a.logits + (size_t)t * E + e0 + q, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            }
        }
    }
    // MXFP8: the tokens' codes and operand-layout scales, a block of 32 per thread
    if (a.xq) {
        const int nb = H / 32, ng = gridDim.x * gridDim.y;
        for (int i = (blockIdx.y * gridDim.x + blockIdx.x) * kFrThreads + tid; i < T * nb; i += ng * kFrThreads) {
            const int t = i / nb, b = i - t * nb;
            const uint8_t sc = mx_quant_block32(a.x + (size_t)t * H + b * 32, a.xq + (size_t)t * H + b * 32);
            mx_store_scale_byte(a.xs, T, t, b, nb, sc);
        }
    }
    // The workgroup that counts in last lays the rows out; it leaves the
    // counter at zero for the next call.
    __syncthreads();
    if (tid == 0) {
        __atomic_thread_fence(__ATOMIC_RELEASE);
        const int n = gridDim.x * gridDim.y;
        const int before = __hip_atomic_fetch_add(a.counter, 1, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT);
        s_last = before == n - 1;
        if (s_last) __hip_atomic_store(a.counter, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    __syncthreads();
    if (!s_last) return;
    // the slab buffers are free: tables in their place
    uint64_t* s_mask = (uint64_t*)&s_wr[0][0];              // 256 x 8
    int* s_off = (int*)(s_mask + kMaxExperts);              // 256 x 4
    int* s_idx = s_off + kMaxExperts;                       // 64 x 16 x 4
    float* s_w = (float*)(s_idx + kFewTokens * kMaxTopK);   // 64 x 16 x 4
    static_assert(sizeof(s_wr) >= kMaxExperts * 12 + kFewTokens * kMaxTopK * 8, "tables fit the slab");
    few_layout(a, s_mask, s_idx, s_w, s_off);
}

void launch_few_route(const FewRoute& a, hipStream_t stream) {
    const dim3 grid(ceil_div(a.E, kFrEC), ceil_div(a.T, kFrTok));
    if (a.E % 4 == 0 && ((uintptr_t)a.Wr & 15) == 0)
        hipLaunchKernelGGL(few_route_kernel<true>, grid, dim3(kFrThreads), 0, stream, a);
    else
        hipLaunchKernelGGL(few_route_kernel<false>, grid, dim3(kFrThreads), 0, stream, a);
}

// ---------------------------------------------------------------------------
// Expert products
// ---------------------------------------------------------------------------

constexpr int kFgThreads = 512;
constexpr int kFgWaves = kFgThreads / kWave;
constexpr int kFgRows = 64;                 // weight rows per workgroup
constexpr int kFgChunk = 128;               // bytes of a weight row per step: one cache line
constexpr int kFgLd = kFgRows + 4;          // floats of a token's partial sums in LDS

__device__ __forceinline__ intx8 cat8(intx4 a, intx4 b) {
    return intx8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
}

// The operands of one step of a wave: 64 weight rows and up to 16 * MT token
// rows, 128 bytes of each.  Lane l holds, of row l % 16 of each fragment, the
// 16 bytes at 16 (l / 16) of each half line: for bf16 the operands of two
// 16x16x32 MFMAs, for MXFP8 those of one scaled 16x16x128 MFMA, whose scale of
// (row m, block b) comes from lane m + 16 b.
template <bool MX, int N>
struct FewFrag {
    intx4 v[N][2];
    uint32_t s[MX ? N : 1];
};

// One operand of a tile: rows of data and, for MXFP8, their scale dwords
// (`group` bytes from one 128-column group to the next).  Buffer loads: a
// lane's offset stays, the step is the scalar offset, and a buffer of no bytes
// gives zeros without touching memory.
struct FewOperand {
    const void* data;
    const void* scale;
    uint32_t bytes, scale_bytes, group;
};

__device__ __forceinline__ __amdgpu_buffer_rsrc_t few_rsrc(const void* p, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc((void*)p, 0, (int)bytes, 0x00020000);
}

// Fragments of step c of rows of kb bytes: zeros past the row's end, which for
// MXFP8 rows of an odd multiple of 64 columns is in the middle of a line.  (The
// scalar offset counts against the buffer's size, so it is zero there too.)
template <bool MX, int N>
__device__ __forceinline__ void few_load(const FewOperand& o, int kb, int c, const uint32_t (&off)[N],
                                         const uint32_t (&soff)[N], FewFrag<MX, N>& f) {
    const int at = c * kFgChunk;
    const bool in = at < kb, whole = MX ? at + kFgChunk / 2 < kb : in;
    const __amdgpu_buffer_rsrc_t lo = few_rsrc(o.data, in ? o.bytes : 0), hi = few_rsrc(o.data, whole ? o.bytes : 0);
    const __amdgpu_buffer_rsrc_t sc = few_rsrc(o.scale, in ? o.scale_bytes : 0);
    const int lo_at = in ? at : 0, hi_at = whole ? at : 0, sc_at = in ? c * (int)o.group : 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        f.v[i][0] = __builtin_amdgcn_raw_buffer_load_b128(lo, off[i], lo_at, 0);
        f.v[i][1] = __builtin_amdgcn_raw_buffer_load_b128(hi, off[i] + kFgChunk / 2, hi_at, 0);
        if (MX) f.s[i] = __builtin_amdgcn_raw_buffer_load_b32(sc, soff[i], sc_at, 0);
    }
}

template <bool MX, int MT>
__device__ __forceinline__ void few_mfma(const FewFrag<MX, 4>& w, const FewFrag<MX, MT>& x, int shift,
                                         floatx4 (&acc)[4][MT]) {
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (MX) {
                acc[i][m] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                    cat8(w.v[i][0], w.v[i][1]), cat8(x.v[m][0], x.v[m][1]), acc[i][m], 0, 0, 0, (int)(w.s[i] >> shift),
                    0, (int)(x.s[m] >> shift));
            } else {
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    acc[i][m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, w.v[i][j]),
                                                                        __builtin_bit_cast(bf16x8, x.v[m][j]),
                                                                        acc[i][m], 0, 0, 0);
            }
        }
}

// acc[i][m] (+)= weight rows 16 i .. of the tile times token rows 16 m .., over
// the steps wave, wave + 8, ... of the rows' kb bytes.  The weights of one step
// are in flight while the step before is multiplied; the tokens, which come
// from the L2, are loaded in their own step, ahead of the next weights, so that
// waiting for them (loads return in order) leaves those in flight.  Steps past
// the end load zeros, so the loop has one exit and keeps its registers.
template <bool MX, int MT>
__device__ __forceinline__ void few_stream(const FewOperand& wo, const FewOperand& xo, int kb, int wave, int lane,
                                           const uint32_t (&xrow)[MT], const uint32_t (&xsoff)[MT],
                                           floatx4 (&acc)[4][MT]) {
    const uint32_t lo = (uint32_t)(lane >> 4) * 16;
    uint32_t woff[4], wsoff[4], xoff[MT];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        woff[i] = (uint32_t)(i * 16 + (lane & 15)) * (uint32_t)kb + lo;
        wsoff[i] = (uint32_t)(i * 16 + (lane & 15)) * 4;
    }
#pragma unroll
    for (int m = 0; m < MT; ++m) xoff[m] = xrow[m] + lo;
    const int shift = 8 * (lane >> 4);
    FewFrag<MX, 4> w0, w1;
    FewFrag<MX, MT> x;
    auto step = [&](int c, const FewFrag<MX, 4>& w, FewFrag<MX, 4>& next) {
        few_load<MX, MT>(xo, kb, c, xoff, xsoff, x);
        few_load<MX, 4>(wo, kb, c + kFgWaves, woff, wsoff, next);
        __builtin_amdgcn_sched_barrier(0);
        few_mfma<MX, MT>(w, x, shift, acc);
        __builtin_amdgcn_sched_barrier(0);
    };
    few_load<MX, 4>(wo, kb, wave, woff, wsoff, w0);
    for (int c = wave; c * kFgChunk < kb; c += 2 * kFgWaves) {
        step(c, w0, w1);
        step(c + kFgWaves, w1, w0);
    }
}

// One M tile's partial sums of every wave into LDS: s_part[wave][token][row].
// A lane holds rows 4 (l / 16) .. + 3 of each fragment for token l % 16.
template <int MT>
__device__ __forceinline__ void few_stage(const floatx4 (&acc)[4][MT], int m, int wave, int lane, float* s_part) {
    float* d = s_part + ((size_t)wave * 16 + (lane & 15)) * kFgLd + 4 * (lane >> 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) *(floatx4*)(d + 16 * i) = acc[i][m];
}

template <bool MX, int MT>
__device__ __forceinline__ void few_gate_up(const FewGemm& a, int e, int n, int row0, int rows, float* s_part) {
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int H = a.H, I = a.I;
    const uint32_t kb = (uint32_t)H * (MX ? 1 : 2);
    FewOperand wo{}, xo{};
    wo.bytes = kFgRows * kb;
    xo.bytes = (uint32_t)a.T * kb;
    if constexpr (MX) {
        wo.data = a.w1q + ((int64_t)e * 2 * I + (int64_t)n * kFgRows) * H;
        wo.scale = a.s1 + ((int64_t)e * mx_groups(H) * 2 * I + (int64_t)n * kFgRows) * 4;
        wo.group = (uint32_t)2 * I * 4;
        wo.scale_bytes = ((uint32_t)mx_groups(H) - 1) * wo.group + kFgRows * 4;
        xo.data = a.xq;
        xo.scale = a.xs;
        xo.group = (uint32_t)a.T * 4;
        xo.scale_bytes = (uint32_t)mx_groups(H) * xo.group;
    } else {
        wo.data = a.w1 + ((int64_t)e * 2 * I + (int64_t)n * kFgRows) * H;
        xo.data = a.x;
    }
    uint32_t xrow[MT], xsrow[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        const int t = a.row_token[row0 + min(m * 16 + (lane & 15), rows - 1)];
        xrow[m] = (uint32_t)t * kb;
        xsrow[m] = (uint32_t)t * 4;
    }
    floatx4 acc[4][MT];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int m = 0; m < MT; ++m) acc[i][m] = floatx4{0, 0, 0, 0};
    few_stream<MX, MT>(wo, xo, (int)kb, wave, lane, xrow, xsrow, acc);
    // thread (token tid / 32, column tid % 32): the tile's rows are 32 gate
    // columns and the 32 up columns of the same indices
    const int tt = tid >> 5, col = tid & 31;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        if (m * 16 >= rows) break;
        __syncthreads();
        few_stage<MT>(acc, m, wave, lane, s_part);
        __syncthreads();
        float g = 0.0f, u = 0.0f;
#pragma unroll
        for (int w = 0; w < kFgWaves; ++w) {
            g += s_part[(w * 16 + tt) * kFgLd + col];
            u += s_part[(w * 16 + tt) * kFgLd + 32 + col];
        }
        const float h = g / (1.0f + expf(-g)) * u;
        const int r = m * 16 + tt;
        if (MX) {  // the 32 columns of a token are one MXFP8 block, held by half a wave
            float am = fabsf(h);
#pragma unroll
            for (int s = 16; s >= 1; s >>= 1) am = fmaxf(am, __shfl_xor(am, s, kWave));
            const int ex = mx_scale_exp(am);
            const uint32_t code = fp8x4(ldexpf(h, -ex), 0.0f, 0.0f, 0.0f);
            if (r < rows) {
                a.hq[(size_t)(row0 + r) * I + n * 32 + col] = (uint8_t)code;
                if (col == 0) {  // a row's scale dwords are adjacent; the last group's spare bytes are zero
                    uint8_t* d = a.hs + (size_t)(row0 + r) * mx_groups(I) * 4 + n;
                    d[0] = (uint8_t)(ex + 127);
                    if (n + 1 == I / 32)
                        for (int z = 1; (n + z) & 3; ++z) d[z] = 0;
                }
            }
        } else if (r < rows) {
            a.h[(size_t)(row0 + r) * I + n * 32 + col] = f32_to_bf16_rne(h);
        }
    }
}

template <bool MX, int MT>
__device__ __forceinline__ void few_down(const FewGemm& a, int e, int n, int row0, int rows, float* s_part) {
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int H = a.H, I = a.I;
    const uint32_t kb = (uint32_t)I * (MX ? 1 : 2);
    FewOperand wo{}, xo{};
    wo.bytes = kFgRows * kb;
    xo.bytes = (uint32_t)rows * kb;
    if constexpr (MX) {
        wo.data = a.w2q + ((int64_t)e * H + (int64_t)n * kFgRows) * I;
        wo.scale = a.s2 + ((int64_t)e * mx_groups(I) * H + (int64_t)n * kFgRows) * 4;
        wo.group = (uint32_t)H * 4;
        wo.scale_bytes = ((uint32_t)mx_groups(I) - 1) * wo.group + kFgRows * 4;
        xo.data = a.hq + (int64_t)row0 * I;
        xo.scale = a.hs + (int64_t)row0 * mx_groups(I) * 4;
        xo.group = 4;
        xo.scale_bytes = (uint32_t)rows * (uint32_t)mx_groups(I) * 4;
    } else {
        wo.data = a.w2 + ((int64_t)e * H + (int64_t)n * kFgRows) * I;
        xo.data = a.h + (int64_t)row0 * I;
    }
    uint32_t xrow[MT], xsrow[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        const uint32_t r = (uint32_t)min(m * 16 + (lane & 15), rows - 1);
        xrow[m] = r * kb;
        xsrow[m] = r * (uint32_t)mx_groups(I) * 4;
    }
    floatx4 acc[4][MT];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int m = 0; m < MT; ++m) acc[i][m] = floatx4{0, 0, 0, 0};
    few_stream<MX, MT>(wo, xo, (int)kb, wave, lane, xrow, xsrow, acc);
    const int tt = tid >> 5, col = (tid & 31) * 2;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        if (m * 16 >= rows) break;
        __syncthreads();
        few_stage<MT>(acc, m, wave, lane, s_part);
        __syncthreads();
        float y0 = 0.0f, y1 = 0.0f;
#pragma unroll
        for (int w = 0; w < kFgWaves; ++w) {
            y0 += s_part[(w * 16 + tt) * kFgLd + col];
            y1 += s_part[(w * 16 + tt) * kFgLd + col + 1];
        }
        const int r = m * 16 + tt;
        if (r < rows) {
            const float wt = a.row_w[row0 + r];
            float* d = a.y + (size_t)(row0 + r) * H + n * kFgRows + col;
            d[0] = wt * y0;
            d[1] = wt * y1;
        }
    }
}

template <bool kDown, bool MX, int MT>
__device__ __forceinline__ void few_tile(const FewGemm& a, int e, int n, int row0, int rows, float* s_part) {
    if constexpr (kDown) few_down<MX, MT>(a, e, n, row0, rows, s_part);
    else few_gate_up<MX, MT>(a, e, n, row0, rows, s_part);
}

// The tile's code by the 16-row fragments that the expert's rows fill (three
// run as four, the rows past the last repeating it).
template <bool kDown, bool MX, int kMost>
__device__ __forceinline__ void few_tile_rows(const FewGemm& a, int e, int n, int row0, int rows, float* s_part) {
    if (kMost == 1 || rows <= 16) few_tile<kDown, MX, 1>(a, e, n, row0, rows, s_part);
    else if (kMost == 2 || rows <= 32) few_tile<kDown, MX, 2>(a, e, n, row0, rows, s_part);
    else few_tile<kDown, MX, 4>(a, e, n, row0, rows, s_part);
}

// Workgroup b: active expert b / n_tiles, weight rows 64 (b % n_tiles) .. + 63.
// The host sizes the grid for every expert that T * k choices can reach; the
// workgroups past the active ones end at once.  kMost: 16-row fragments of T.
template <bool kDown, bool kMx, int kMost>
__global__ __launch_bounds__(kFgThreads) void few_gemm_kernel(FewGemm a) {
    __shared__ __attribute__((aligned(16))) float s_part[kFgWaves * 16 * kFgLd];
    const int nt = kDown ? a.H / kFgRows : a.I / 32;
    const int i = blockIdx.x / nt, n = blockIdx.x - i * nt;
    if (i >= ld_layout(a.n_act)) return;
    const int e = ld_layout(a.act_e + i), row0 = ld_layout(a.act_off + i), rows = ld_layout(a.act_off + i + 1) - row0;
    if (kMx && e < a.E) few_tile_rows<kDown, true, kMost>(a, e, n, row0, rows, s_part);
    else few_tile_rows<kDown, false, kMost>(a, e, n, row0, rows, s_part);
}

template <bool kDown>
static void launch_few_gemm(const FewGemm& a, int max_act, hipStream_t stream) {
    const dim3 grid((unsigned)max_act * (unsigned)(kDown ? a.H / kFgRows : a.I / 32)), block(kFgThreads);
    const int mt = ceil_div(a.T, 16);  // an expert has at most T rows
#define FEW_LAUNCH(MX, MT) hipLaunchKernelGGL((few_gemm_kernel<kDown, MX, MT>), grid, block, 0, stream, a)
    if (a.xq) {
        if (mt == 1) FEW_LAUNCH(true, 1);
        else if (mt == 2) FEW_LAUNCH(true, 2);
        else FEW_LAUNCH(true, 4);
    } else {
        if (mt == 1) FEW_LAUNCH(false, 1);
        else if (mt == 2) FEW_LAUNCH(false, 2);
        else FEW_LAUNCH(false, 4);
    }
#undef FEW_LAUNCH
}

void launch_few_gate_up(const FewGemm& a, int max_act, hipStream_t s) { launch_few_gemm<false>(a, max_act, s); }
void launch_few_down(const FewGemm& a, int max_act, hipStream_t s) { launch_few_gemm<true>(a, max_act, s); }

// out[t] = sum over slots in order of the weighted rows, then the shared row.
__global__ __launch_bounds__(256) void few_combine_kernel(FewGemm a, int k, int shared, uint16_t* out) {
    const int c = (blockIdx.x * 256 + threadIdx.x) * 2, t = blockIdx.y;
    if (c >= a.H) return;
    float s0 = 0.0f, s1 = 0.0f;
    for (int j = 0; j < k + shared; ++j) {
        const int row = j < k ? a.slot_row[t * k + j] : a.T * k + t;
        const float* y = a.y + (size_t)row * a.H + c;
        s0 += y[0];
        s1 += y[1];
    }
    *(uint32_t*)(out + (size_t)t * a.H + c) = (uint32_t)f32_to_bf16_rne(s0) | ((uint32_t)f32_to_bf16_rne(s1) << 16);
}

void launch_few_combine(const FewGemm& a, int k, int shared, uint16_t* out, hipStream_t stream) {
    hipLaunchKernelGGL(few_combine_kernel, dim3(ceil_div(a.H, 512), a.T), dim3(256), 0, stream, a, k, shared, out);
}

}  // namespace moe
