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
#include "gemm_tile.hpp"
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

// ---------------------------------------------------------------------------
// Many rows: 256 x 256 tiles
// ---------------------------------------------------------------------------

// Eight waves, two per SIMD, each 64 x 128 of the tile as 2 x 4 fragments of 32 x 32.
// A stage is one block of K: A and B codes as 128-byte rows, the A rows' scales and
// the tile's two weight scales; two stages make the ring.  All of it comes by loads
// straight into LDS through buffer descriptors: what lies past the group's last row,
// the matrix's last row or the row's end reads as zero and moves no memory, so no
// size needs a tile of its own, and a lane's offsets are the same for every tile.
constexpr int kBgStageB = BM * kBlk;
constexpr int kBgStageSA = kBgStageB + BN * kBlk;
constexpr int kBgStageSW = kBgStageSA + BM * 4;       // the first two of four areas that a wave's load fills
constexpr int kBgStage = kBgStageSW + 4 * kWave * 4;
constexpr int kBgRing = 2 * kBgStage;
constexpr int kBgStgPitch = 512;                      // staged bf16 output: 32 rows of 512 bytes
constexpr int kBgMax = kBgRing + 32 * kBgStgPitch;    // SwiGLU: largest |h| of each row's two halves
constexpr int kBgTables = kBgMax + BM * 8;
constexpr int kBgGroups = 512;                        // groups whose tables fit beside them
constexpr int kBgSmem = kBgTables + (3 * kBgGroups + 1) * 4;
static_assert(kBgSmem <= 160 * 1024, "the LDS");
constexpr int kBgThreads = 512;

// What a tile's loads start from, uniform in a wave: codes of this wave's A and B
// rows, the scales of its 64 A rows (waves 0 .. 3), one weight scale (waves 4 and 5).
struct BgSource {
    const uint8_t *a, *b;
    const float* s;
    uint32_t a_bytes, b_bytes, s_bytes;
};

struct BgTile {
    int g, row0, count, n0;  // n0: first output column; count: rows, at most BM; 0: no tile
};

// LDS accesses of the epilogue, in asm: the compiler would wait for the next tile's
// loads into the ring too.
__device__ __forceinline__ uint32_t lds_at(const void* p) { return (uint32_t)(uintptr_t)(lds_void*)p; }
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ void lds_put(uint32_t at, uint32_t v) {
    asm volatile("ds_write_b32 %0, %1" ::"v"(at), "v"(v) : "memory");
}
__device__ __forceinline__ void lds_put2(uint32_t at, u32x2 v) {
    asm volatile("ds_write_b64 %0, %1" ::"v"(at), "v"(v) : "memory");
}
__device__ __forceinline__ void lds_get4x2(uint32_t at0, uint32_t at1, u32x4& d0, u32x4& d1) {
    asm volatile("ds_read_b128 %0, %2\n\tds_read_b128 %1, %3\n\ts_waitcnt lgkmcnt(0)"
                 : "=&v"(d0), "=&v"(d1)
                 : "v"(at0), "v"(at1)
                 : "memory");
}
__device__ __forceinline__ u32x2 lds_get2(uint32_t at) {
    u32x2 d;
    asm volatile("ds_read_b64 %0, %1\n\ts_waitcnt lgkmcnt(0)" : "=&v"(d) : "v"(at) : "memory");
    return d;
}

template <bool kGlu>
__global__ __launch_bounds__(kBgThreads, 2) void block_gemm_kernel(BlockGemm p) {
    constexpr int kCols = kGlu ? BN / 2 : BN;  // output columns of a tile
    extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
    int32_t* s_first = (int32_t*)(smem + kBgTables);  // [groups + 1] M tiles before each group
    int32_t* s_lo = s_first + p.groups + 1;           // [groups] its rows
    int32_t* s_hi = s_lo + p.groups;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave >> 1, wn = wave & 1;
    const int KB = blk_count(p.k), NB = blk_count(p.n), NT = (p.n + kCols - 1) / kCols;

    if (wave == 0) {
        int before = 0;
        for (int e0 = 0; e0 < p.groups; e0 += kWave) {
            const int e = e0 + lane;
            int lo = 0, hi = 0;
            if (e < p.groups) {  // bounds outside the rows are cut off
                lo = p.offsets ? min(max(p.offsets[e], 0), p.rows) : 0;
                hi = p.offsets ? min(max(p.offsets[e + 1], lo), p.rows) : p.rows;
            }
            const int tiles = (hi - lo + BM - 1) / BM;
            int upto = tiles;
#pragma unroll
            for (int s = 1; s < kWave; s *= 2) {
                const int v = __shfl_up(upto, s, kWave);
                if (lane >= s) upto += v;
            }
            if (e < p.groups) {
                s_first[e] = before + upto - tiles;
                s_lo[e] = lo;
                s_hi[e] = hi;
            }
            before += __shfl(upto, kWave - 1, kWave);
        }
        if (lane == 0) s_first[p.groups] = before;
    }
    __syncthreads();
    // Workgroup b runs on XCD b % 8, whose workgroups take neighbouring tiles: group by
    // group, column by column, M tiles fastest, so that they share panels in its L2.
    const int total = __builtin_amdgcn_readfirstlane(s_first[p.groups]) * NT;
    const int xcd = blockIdx.x & 7, per = (total + 7) / 8, step = gridDim.x >> 3;
    const int t_end = min((xcd + 1) * per, total);
    auto tile_at = [&](int t) {
        BgTile r{0, 0, 0, 0};
        if (t >= t_end) return r;
        int e = 0;  // the last group with no more than t tiles before it; it is not empty
        for (int e0 = 0; e0 < p.groups; e0 += kWave) {
            const int x = e0 + lane;
            const uint64_t at = __ballot(x < p.groups && s_first[min(x, p.groups - 1)] * NT <= t);
            if (!at) break;
            e = e0 + 63 - __builtin_clzll(at);
        }
        r.g = e;
        const int f0 = __builtin_amdgcn_readfirstlane(s_first[e]), f1 = __builtin_amdgcn_readfirstlane(s_first[e + 1]);
        const int in = t - f0 * NT, col = in / (f1 - f0);
        r.n0 = col * kCols;
        r.row0 = __builtin_amdgcn_readfirstlane(s_lo[e]) + (in - col * (f1 - f0)) * BM;
        r.count = min(__builtin_amdgcn_readfirstlane(s_hi[e]) - r.row0, BM);
        return r;
    };
    auto source_of = [&](const BgTile& t) {
        BgSource s{};
        if (t.count == 0) return s;
        s.a = p.a + (int64_t)(t.row0 + wave * 32) * p.k;
        s.a_bytes = (uint32_t)max(t.count - wave * 32, 0) * (uint32_t)p.k;
        // B rows 32 wave .. + 31 of the stage: columns n0 + 32 wave; with SwiGLU, for the column
        // half wn = wave / 4 and fragment j = wave % 4, columns n0 + 64 wn + 32 (j % 2) of the
        // gate's (j < 2) or the up matrix, so that a wave ends with both of its columns
        const bool up = kGlu && (wave & 2);
        const int br = t.n0 + (kGlu ? (wave >> 2) * 64 + (wave & 1) * 32 : wave * 32);
        s.b = (up ? p.wu : p.w) + ((int64_t)t.g * p.n + br) * p.k;
        s.b_bytes = (uint32_t)max(p.n - br, 0) * (uint32_t)p.k;
        if (wave < 4) {
            s.s = p.sa + t.row0 + wave * 64;
            s.s_bytes = (uint32_t)max(t.count - wave * 64, 0) * 4;
        } else {  // the tile's first column block (the gate's), and its second (the up matrix's)
            const int nb = t.n0 / kBlk + (kGlu ? 0 : wave & 1);
            s.s = (kGlu && (wave & 1) ? p.swu : p.sw) + ((int64_t)t.g * NB + nb) * KB;
            s.s_bytes = wave < 6 && nb < NB ? 4 : 0;
        }
        return s;
    };
    const int64_t s_step = wave < 4 ? p.rows : 1;  // scales from block to block of K

    // Load i of a stage fills rows 32 wave + 8 i .. + 7: lane l row l / 8, chunk l % 8 in LDS,
    // which holds the row's chunk (l % 8) ^ swz8(row).
    const int c_even = (lane & 7) ^ (lane >> 4), c_odd = c_even ^ 4;
    const uint32_t v_even = (uint32_t)(lane >> 3) * (uint32_t)p.k + c_even * 16;
    const uint32_t v_odd = (uint32_t)((lane >> 3) + 8) * (uint32_t)p.k + c_odd * 16;
    const uint32_t v_two = 16u * (uint32_t)p.k;
    BgSource src, nxt;
    // Stage s of this tile, or past its last the next tile's; past the last tile's last
    // nothing is read and the slot, which no wave reads any more, is filled with zeros.
    auto issue = [&](int s_, int slot) {
        const bool beyond = s_ >= KB;
        const BgSource q = beyond ? nxt : src;
        const int s = beyond ? s_ - KB : s_;
        const int left = q.a ? p.k - s * kBlk : 0;  // bytes of a row from this stage on
        uint8_t* st = smem + slot * kBgStage;
        uint8_t* base = st + wave * 32 * kBlk;
        const __amdgpu_buffer_rsrc_t ra = blk_rsrc(q.a, q.a_bytes), rb = blk_rsrc(q.b, q.b_bytes);
        const bool in_e = c_even * 16 < left, in_o = c_odd * 16 < left;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t v = (i & 1 ? v_odd : v_even) + (i >> 1) * v_two + s * kBlk;
            const uint32_t o = (i & 1 ? in_o : in_e) ? v : kNowhere;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_void*)(base + i * 1024), 16, o, 0, 0, 0);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (lds_void*)(base + kBgStageB + i * 1024), 16, o, 0, 0, 0);
        }
        // (a wave without scales fills its area with zeros: a branch here would let the
        // compiler move every addition of the stage past it)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(blk_rsrc(q.s + s * s_step, left > 0 ? q.s_bytes : 0),
                                                 (lds_void*)(st + kBgStageSA + wave * 256), 4, lane * 4, 0, 0, 0);
    };

    const int fr = lane & 31, half = lane >> 5;
    const int fsw = swz8(fr);  // a fragment's rows differ from fr by multiples of 32
    const int arow = (wm * 32 + fr) * kBlk, brow = kBgStageB + (wn * 128 + fr) * kBlk;
    // The two operands' parts of a K block fall to the lanes alike: K step ks takes chunks
    // 4 ks + half and 4 ks + 2 + half.
    auto read_frag = [&](int slot, int row, intx8 (&f)[2]) {
        const uint8_t* st = smem + slot * kBgStage + row;
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
            const intx4 lo = *(const intx4*)(st + (((4 * ks + half) ^ fsw) * 16));
            const intx4 hi = *(const intx4*)(st + (((4 * ks + 2 + half) ^ fsw) * 16));
            f[ks] = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
        }
    };
    intx8 fa[2][2], fb[2][2];
    float sa[2], sw[kGlu ? 2 : 1], sa_n[2], sw_n[kGlu ? 2 : 1];
    auto read_scales = [&](int slot) {
        const float* st = (const float*)(smem + slot * kBgStage + kBgStageSA);
#pragma unroll
        for (int i = 0; i < 2; ++i) sa_n[i] = st[i * 128 + wm * 32 + fr];
        const float* w = (const float*)(smem + slot * kBgStage + kBgStageSW);
        if constexpr (kGlu) {
            sw_n[0] = w[0];
            sw_n[1] = w[kWave];
        } else {
            sw_n[0] = w[wn * kWave];
        }
    };
    floatx16 acc[2][4];
    // Fragment f = 2 j + i of a stage: both K steps from a zero accumulator, then scaled into
    // the sum.  B is the first operand, so element 4 q + s of lane l is column 8 q + 4 (l / 32) +
    // s of row l % 32: a lane has one row of A, and its scale is one register.  A fragment is
    // added while the next one multiplies, the last one of a stage in the next stage; the
    // order is fixed here, since the compiler's own keeps six products at once and spills.
    floatx16 v[2];
    float sc[2];
    auto multiply = [&](int i, int j, const intx8 (&b)[2]) {
        v[i] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(b[0], fa[i][0], floatx16{}, 0, 0, 0, 0, 0, 0);
        v[i] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(b[1], fa[i][1], v[i], 0, 0, 0, 0, 0, 0);
        __builtin_amdgcn_sched_barrier(0);  // then the additions: the product they take is done by now
    };
    auto add = [&](int i, int j) {
#pragma unroll
        for (int c = 0; c < 16; ++c) acc[i][j][c] = __builtin_fmaf(v[i][c], sc[i], acc[i][j][c]);
    };
    auto pin = [] { __builtin_amdgcn_sched_barrier(0); };

    int t = xcd * per + (blockIdx.x >> 3);
    BgTile tile = tile_at(t);
    if (tile.count == 0) return;
    src = source_of(tile);
    nxt = BgSource{};
    issue(0, 0);
    issue(1, 1);  // KB is at least 2
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    int slot = 0;
    read_frag(0, arow, fa[0]);
    read_frag(0, arow + 128 * kBlk, fa[1]);
    read_frag(0, brow, fb[0]);
    read_scales(0);
    for (;;) {
        t += step;
        const BgTile next = tile_at(t);
        nxt = source_of(next);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = floatx16{};
        v[1] = floatx16{};
        sc[1] = 0.0f;
        for (int s = 0; s < KB; ++s) {
            pin();
            read_frag(slot, brow + 1 * 32 * kBlk, fb[1]);
            multiply(0, 0, fb[0]);
            add(1, 3);  // of the stage before
#pragma unroll
            for (int i = 0; i < 2; ++i) sa[i] = sa_n[i];
#pragma unroll
            for (int x = 0; x < (kGlu ? 2 : 1); ++x) sw[x] = sw_n[x];
            sc[0] = sa[0] * sw[0];
            sc[1] = sa[1] * sw[0];
            pin();
            multiply(1, 0, fb[0]);
            add(0, 0);
            pin();
            read_frag(slot, brow + 2 * 32 * kBlk, fb[0]);
            multiply(0, 1, fb[1]);
            add(1, 0);
            pin();
            multiply(1, 1, fb[1]);
            add(0, 1);
            if constexpr (kGlu) sc[0] = sa[0] * sw[1];
            pin();
            read_frag(slot, brow + 3 * 32 * kBlk, fb[1]);
            multiply(0, 2, fb[0]);
            add(1, 1);
            if constexpr (kGlu) sc[1] = sa[1] * sw[1];
            pin();
            multiply(1, 2, fb[0]);
            add(0, 2);
            pin();
            // stage s + 1 has landed, and no wave reads stage s any more
            asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
            __builtin_amdgcn_s_barrier();
            asm volatile("" ::: "memory");
            issue(s + 2, slot);
            slot ^= 1;
            pin();
            read_frag(slot, brow, fb[0]);
            read_scales(slot);
            multiply(0, 3, fb[1]);
            add(1, 2);
            pin();
            read_frag(slot, arow, fa[0]);
            multiply(1, 3, fb[1]);
            add(0, 3);
            pin();
            read_frag(slot, arow + 128 * kBlk, fa[1]);
        }
        add(1, 3);

        const uint32_t stg = lds_at(smem) + kBgRing;
        int tid = threadIdx.x;  // opaque: the lane addresses are formed here, not kept live
        asm volatile("" : "+v"(tid));
        if constexpr (!kGlu) {
            // 32 rows at a time through LDS, chunk c of row r at c ^ r, out in whole lines
            const int rs = tid & 31, r0 = tid >> 5, ch = tid & 31;
            const uint32_t wrow = stg + rs * kBgStgPitch + 8 * ((tid >> 5) & 1);
            const int wc0 = ((tid >> 6) & 1) * 16;
            const bool col_in = ch * 8 < p.n - tile.n0;  // n is a multiple of 8
#pragma unroll
            for (int b = 0; b < 8; ++b) {  // tile rows 32 b ..: fragment b / 4 of the waves with wm = b % 4
                if (b * 32 >= tile.count) break;
                if (wm == (b & 3)) {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const floatx16& v = acc[b >> 2][j];
                            lds_put2(wrow + (((wc0 + 4 * j + q) ^ rs) << 4),
                                     u32x2{pack_bf16x2(v[4 * q], v[4 * q + 1]), pack_bf16x2(v[4 * q + 2], v[4 * q + 3])});
                        }
                }
                lds_barrier();
                u32x4 d0, d1;
                lds_get4x2(stg + r0 * kBgStgPitch + ((ch ^ r0) << 4),
                           stg + (r0 + 16) * kBgStgPitch + ((ch ^ (r0 + 16)) << 4), d0, d1);
                const int row = b * 32 + r0;
                uint16_t* dst = p.out + (int64_t)(tile.row0 + row) * p.n + tile.n0 + ch * 8;
                if (col_in && row < tile.count) *(u32x4*)dst = d0;
                if (col_in && row + 16 < tile.count) *(u32x4*)(dst + 16 * (int64_t)p.n) = d1;
                lds_barrier();
            }
        } else {
            // h in place of the gate's fragments; a row's block of 128 is two waves' columns
            const int cl = tile.n0 + wn * 64 + 4 * half;
            float m[2] = {0.0f, 0.0f};
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int c = 0; c < 16; ++c) {
                        const float g = acc[i][j][c];
                        float v = g / (1.0f + __expf(-g)) * acc[i][2 + j][c];
                        if (cl + 32 * j + 8 * (c >> 2) >= p.n) v = 0.0f;  // n is a multiple of 16
                        acc[i][j][c] = v;
                        m[i] = fmaxf(m[i], fabsf(v));
                    }
            const uint32_t mx = lds_at(smem) + kBgMax;
            const int rl = wm * 32 + (tid & 31);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                m[i] = fmaxf(m[i], __shfl_xor(m[i], 32, kWave));
                if (half == 0) lds_put(mx + ((128 * i + rl) * 2 + wn) * 4, __builtin_bit_cast(uint32_t, m[i]));
            }
            lds_barrier();
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if (128 * i >= tile.count) break;
                const u32x2 both = lds_get2(mx + (128 * i + rl) * 8);
                // (of values: a cast of the vector's element itself takes its first one)
                const uint32_t m0 = both[0], m1 = both[1];
                const int e = blk_exp(fmaxf(__builtin_bit_cast(float, m0), __builtin_bit_cast(float, m1)));
                const int row = tile.row0 + 128 * i + rl;
                const bool row_in = 128 * i + rl < tile.count;
                if (wn == 0 && half == 0 && row_in) p.hs[(int64_t)(tile.n0 / kBlk) * p.rows + row] = pow2f(e);
                const float inv = pow2f(-e);
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const floatx16& v = acc[i][j];
                        const int col = wn * 64 + 32 * j + 8 * q + 4 * half;
                        lds_put(stg + rl * kBlk + (((col >> 4) ^ swz8(rl)) << 4) + (col & 15),
                                fp8x4(v[4 * q] * inv, v[4 * q + 1] * inv, v[4 * q + 2] * inv, v[4 * q + 3] * inv));
                        if (p.h16 && row_in && cl + 32 * j + 8 * q < p.n)
                            *(u32x2*)(p.h16 + (int64_t)row * p.n + tile.n0 + col) =
                                u32x2{pack_bf16x2(v[4 * q], v[4 * q + 1]), pack_bf16x2(v[4 * q + 2], v[4 * q + 3])};
                    }
                lds_barrier();
                const int r0 = tid >> 3, ch = tid & 7;  // rows r0 and r0 + 64 of these 128
                u32x4 d0, d1;
                lds_get4x2(stg + r0 * kBlk + ((ch ^ swz8(r0)) << 4), stg + (r0 + 64) * kBlk + ((ch ^ swz8(r0 + 64)) << 4),
                           d0, d1);
                uint8_t* dst = p.hq + (int64_t)(tile.row0 + 128 * i + r0) * p.n + tile.n0 + ch * 16;
                const bool col_in = tile.n0 + ch * 16 < p.n;
                if (col_in && 128 * i + r0 < tile.count) *(u32x4*)dst = d0;
                if (col_in && 128 * i + r0 + 64 < tile.count) *(u32x4*)(dst + 64 * (int64_t)p.n) = d1;
                lds_barrier();
            }
        }
        if (next.count == 0) break;
        tile = next;
        src = nxt;
    }
    // zeros may still be on their way into the ring
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}

// Parts of at most `part` rows that `rows` rows of `groups` groups can fall into.
static int most_parts(int rows, int groups, int part) { return rows / part + (groups < rows ? groups : rows); }

// Whether the large tiles are the better ones.
bool block_gemm_large(int64_t rows, int n, int k, int groups) {
    return groups <= kBgGroups && k > kBlk && rows > 64 * groups;
}

static void launch_block_gemm_few(const BlockGemm& a, hipStream_t stream) {
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

void launch_block_gemm(const BlockGemm& a, hipStream_t stream) {
    if (!block_gemm_large(a.rows, a.n, a.k, a.groups)) {
        launch_block_gemm_few(a, stream);
        return;
    }
    const int cols = a.wu ? BN / 2 : BN;
    const int64_t tiles = (int64_t)most_parts(a.rows, a.groups, BM) * ((a.n + cols - 1) / cols);
    const int grid = (int)std::min<int64_t>((tiles + 7) / 8 * 8, 256);  // a multiple of the XCDs
    if (a.wu)
        hipLaunchKernelGGL(block_gemm_kernel<true>, dim3(grid), dim3(kBgThreads), kBgSmem, stream, a);
    else
        hipLaunchKernelGGL(block_gemm_kernel<false>, dim3(grid), dim3(kBgThreads), kBgSmem, stream, a);
}

}  // namespace moe
