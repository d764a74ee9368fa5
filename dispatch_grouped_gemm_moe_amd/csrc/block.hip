// Products of rows sorted by expert with their expert's matrix, both in 8-bit
// floating point with one fp32 scale per block of 128 (gfx950).
//
//   out[r][j] = sum_b sa[b][r] sw[g][j / 128][b] P_b,  P_b = sum over block b of a[r][.] w[g][j][.]
//
// and, with a gate and an up matrix, h = silu(gate product) * (up product).  A block
// is as deep as one or two matrix instructions, so P_b comes from a zero accumulator
// and one fused multiply-add per element takes it, scaled, into the fp32 sum.
#include <algorithm>

#include "block8.hpp"
#include "common.hpp"
#include "kernels.hpp"

namespace moe {

#pragma clang fp contract(off)

// A piece of a buffer load that lies past a row's end or a matrix's last row asks for
// this offset: past every buffer here (they hold less than 2 GiB), so it reads as zero.
constexpr uint32_t kNowhere = 0x80000000u;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t blk_rsrc(const void* p, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc((void*)p, 0, bytes, 0x00020000);
}

// Part `slot` of the rows: groups in ascending order, each in parts of kRows rows (the
// last one shorter).  False past the last part.  Offsets outside the rows are cut off,
// so whatever the table holds, no row outside them is named.  Uniform in the wave.
template <int kRows>
__device__ __forceinline__ bool find_part(const int32_t* offsets, int groups, int rows, int slot, int& g, int& row0,
                                          int& count) {
    if (!offsets) {
        g = 0;
        row0 = slot * kRows;
        count = min(rows - row0, kRows);
        return count > 0;
    }
    const int lane = threadIdx.x & 63, per = (groups + kWave - 1) / kWave;
    auto bounds = [&](int e, int& lo, int& hi) {
        lo = min(max(offsets[e], 0), rows);
        hi = min(max(offsets[e + 1], lo), rows);
    };
    int mine = 0;
    for (int i = 0; i < per; ++i) {
        const int e = lane * per + i;
        if (e < groups) {
            int lo, hi;
            bounds(e, lo, hi);
            mine += (hi - lo + kRows - 1) / kRows;
        }
    }
    int upto = mine;  // inclusive sum over the lanes
#pragma unroll
    for (int s = 1; s < kWave; s *= 2) {
        const int v = __shfl_up(upto, s, kWave);
        if (lane >= s) upto += v;
    }
    const uint64_t past = __ballot(upto > slot);
    if (!past) return false;
    const int l = __builtin_ctzll(past);
    int left = slot - __builtin_amdgcn_readlane(upto - mine, l);
    for (int e = l * per;; ++e) {  // ends: lane l's groups hold the part
        int lo, hi;
        bounds(e, lo, hi);
        const int parts = (hi - lo + kRows - 1) / kRows;
        if (left < parts || e == groups - 1) {
            g = __builtin_amdgcn_readfirstlane(e);
            row0 = __builtin_amdgcn_readfirstlane(lo + left * kRows);
            count = __builtin_amdgcn_readfirstlane(min(hi - lo - left * kRows, kRows));
            return true;
        }
        left -= parts;
    }
}

// ---------------------------------------------------------------------------
// Few rows to a group: bound by reading the weights
// ---------------------------------------------------------------------------

constexpr int kBfWaves = 4;

// 16 kTF rows by 16 kNF columns a workgroup, the K blocks dealt to its four waves and
// their sums joined in LDS in a fixed order.  Weight rows are the M side of 16-wide
// MFMAs, rows of a the N side, so a lane ends with four neighbouring columns of a row.
template <int kNF, int kTF, bool kGlu, int kDepth>
__global__ __launch_bounds__(kBfWaves * kWave) void block_few_kernel(BlockGemm a) {
    constexpr int kW = kGlu ? 2 * kNF : kNF;  // weight fragments: the gate's, then the up matrix's
    __shared__ floatx4 s_part[kBfWaves][kW * kTF][kWave];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lr = lane & 15, lq = lane >> 4;
    const int n0 = blockIdx.x * 16 * kNF;
    int g, row0, count;
    for (int slot = blockIdx.y; find_part<16 * kTF>(a.offsets, a.groups, a.rows, slot, g, row0, count);
         slot += gridDim.y) {
        const int kb_n = blk_count(a.k), nb = blk_count(a.n);
        const int64_t wat = (int64_t)g * a.n * a.k;
        const uint32_t wbytes = (uint32_t)a.n * (uint32_t)a.k;
        const __amdgpu_buffer_rsrc_t rw = blk_rsrc(a.w + wat, wbytes), ru = blk_rsrc((kGlu ? a.wu : a.w) + wat, wbytes);
        const __amdgpu_buffer_rsrc_t ra = blk_rsrc(a.a + (int64_t)row0 * a.k, (uint32_t)count * (uint32_t)a.k);
        uint32_t woff[kNF];
        const float *swf[kNF], *suf[kNF];
#pragma unroll
        for (int f = 0; f < kNF; ++f) {
            const int col = n0 + 16 * f + lr;
            woff[f] = col < a.n ? (uint32_t)col * (uint32_t)a.k + lq * 16 : kNowhere;
            const int64_t sat = ((int64_t)g * nb + min(n0 + 16 * f, a.n - 1) / kBlk) * kb_n;
            swf[f] = a.sw + sat;
            suf[f] = (kGlu ? a.swu : a.sw) + sat;
        }
        uint32_t aoff[kTF];
        const float* saf[kTF];
#pragma unroll
        for (int t = 0; t < kTF; ++t) {
            const int r = 16 * t + lr;
            aoff[t] = r < count ? (uint32_t)r * (uint32_t)a.k + lq * 16 : kNowhere;
            saf[t] = a.sa + row0 + min(r, count - 1);
        }
        struct Step {
            intx4 w[kW][2], x[kTF][2];
            float sw[kW], sa[kTF];
        };
        auto load = [&](Step& s, int kb) {
            const uint32_t at = (uint32_t)kb * kBlk + lq * 16;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const bool in = at + 64 * h < (uint32_t)a.k;  // k is a multiple of 16: a piece is inside or not
#pragma unroll
                for (int f = 0; f < kW; ++f) {
                    const uint32_t o = woff[f % kNF];
                    s.w[f][h] = __builtin_amdgcn_raw_buffer_load_b128(
                        f < kNF ? rw : ru, in && o != kNowhere ? o + kb * kBlk + 64 * h : kNowhere, 0, 0);
                }
#pragma unroll
                for (int t = 0; t < kTF; ++t)
                    s.x[t][h] = __builtin_amdgcn_raw_buffer_load_b128(
                        ra, in && aoff[t] != kNowhere ? aoff[t] + kb * kBlk + 64 * h : kNowhere, 0, 0);
            }
            const int ks = min(kb, kb_n - 1);
#pragma unroll
            for (int f = 0; f < kW; ++f) s.sw[f] = (f < kNF ? swf[f % kNF] : suf[f % kNF])[ks];
#pragma unroll
            for (int t = 0; t < kTF; ++t) s.sa[t] = saf[t][(int64_t)ks * a.rows];
        };
        floatx4 acc[kW][kTF] = {};
        auto multiply = [&](const Step& s) {
#pragma unroll
            for (int f = 0; f < kW; ++f) {
                const intx8 w = __builtin_shufflevector(s.w[f][0], s.w[f][1], 0, 1, 2, 3, 4, 5, 6, 7);
#pragma unroll
                for (int t = 0; t < kTF; ++t) {
                    const intx8 x = __builtin_shufflevector(s.x[t][0], s.x[t][1], 0, 1, 2, 3, 4, 5, 6, 7);
                    const floatx4 p =
                        __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, floatx4{}, 0, 0, 0, 0, 0, 0);
                    const float sc = s.sw[f] * s.sa[t];
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[f][t][i] = __builtin_fmaf(p[i], sc, acc[f][t][i]);
                }
            }
        };
        Step st[kDepth];
#pragma unroll
        for (int d = 0; d < kDepth; ++d) load(st[d], wave + kBfWaves * d);
        for (int kb = wave; kb < kb_n; kb += kBfWaves * kDepth) {
#pragma unroll
            for (int d = 0; d < kDepth; ++d) {
                multiply(st[d]);  // past the last block: zeros
                load(st[d], kb + kBfWaves * (kDepth + d));
            }
        }
#pragma unroll
        for (int f = 0; f < kW; ++f)
#pragma unroll
            for (int t = 0; t < kTF; ++t) s_part[wave][f * kTF + t][lane] = acc[f][t];
        __syncthreads();
        auto joined = [&](int i) {
            floatx4 v = s_part[0][i][lane];
#pragma unroll
            for (int x = 1; x < kBfWaves; ++x) v += s_part[x][i][lane];
            return v;
        };
        for (int i = wave; i < kNF * kTF; i += kBfWaves) {
            const int f = i / kTF, t = i % kTF, r = 16 * t + lr, col = n0 + 16 * f + 4 * lq;
            floatx4 v = joined(i);
            if constexpr (kGlu) {
                const floatx4 u = joined(kNF * kTF + i);
#pragma unroll
                for (int x = 0; x < 4; ++x) v[x] = v[x] / (1.0f + __expf(-v[x])) * u[x];
            }
            if (r >= count || col >= a.n) continue;  // n is a multiple of 8: four columns are inside or not
            const int64_t at = (int64_t)(row0 + r) * a.n + col;
            if constexpr (kGlu)
                *(floatx4*)(a.h + at) = v;
            else
                *(uint2*)(a.out + at) = uint2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
        }
        __syncthreads();  // the sums are read
    }
}

// Parts of at most `part` rows that `rows` rows of `groups` groups can fall into.
static int most_parts(int rows, int groups, int part) { return rows / part + (groups < rows ? groups : rows); }

void launch_block_gemm_few(const BlockGemm& a, hipStream_t stream) {
#define BLOCK_FEW(NF, TF, D)                                                                                          \
    do {                                                                                                              \
        const dim3 grid((a.n + 16 * NF - 1) / (16 * NF), std::min(most_parts(a.rows, a.groups, 16 * TF), 65535));                      \
        if (a.wu)                                                                                                     \
            hipLaunchKernelGGL((block_few_kernel<NF, TF, true, D>), grid, dim3(kBfWaves * kWave), 0, stream, a);      \
        else                                                                                                          \
            hipLaunchKernelGGL((block_few_kernel<NF, TF, false, D>), grid, dim3(kBfWaves * kWave), 0, stream, a);     \
    } while (0)
    if (a.rows <= 16 * a.groups) BLOCK_FEW(1, 1, 2);
    else BLOCK_FEW(2, 4, 1);
#undef BLOCK_FEW
}

}  // namespace moe
