// Products of rows sorted by expert with their expert's matrix, both in 8-bit
// floating point with one fp32 scale per block of 128 (gfx950).
//
//   out[r][j] = sum_b sa[b][r] sw[g][j / 128][b] P_b,  P_b = sum over block b of a[r][.] w[g][j][.]
//
// and, with a gate and an up matrix, h = silu(gate product) * (up product).  A block
// is as deep as one or two matrix instructions, so P_b comes from a zero accumulator
// and one fused multiply-add per element takes it, scaled, into the fp32 sum.
//
// The matrix instruction cuts off what lies below 2^-13 of the largest of eight neighbouring
// products.  A product's own output does not show it (its distance from 64 bits is the last
// rounding's, 0.0017, with and without); but of h's codes 1.6 in 1000 are those on the other
// side of a border, where sums in fp32 leave 0.06, and the experts' output is 0.0025 to 0.0026
// away instead of 0.0023 to 0.0024.
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "block8.hpp"
#include "common.hpp"
#include "gemm_tile.hpp"
#include "kernels.hpp"

namespace moe {

#pragma clang fp contract(off)

// A piece of a buffer load that lies past a row's end or a matrix's last row asks for
// this offset: past every buffer here (they hold less than 2 GiB), so it reads as zero.
constexpr uint32_t kNowhere = 0x80000000u;
constexpr int kPastCaches = 2;  // of a buffer load: the non-temporal hint

__device__ __forceinline__ __amdgpu_buffer_rsrc_t blk_rsrc(const void* p, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc((void*)p, 0, bytes, 0x00020000);
}

__device__ __forceinline__ uint32_t lds_at(const void* p) { return (uint32_t)(uintptr_t)(lds_void*)p; }

// Parts of at most `part` rows that `rows` rows of `groups` groups can fall into.  The kernels
// take no more of them, whatever a table holds (where moe_dispatch_layout has reported an
// error it may be anything: groups that overlap could make 2^34 of them).
__host__ __device__ __forceinline__ int most_parts(int rows, int groups, int part) {
    return rows / part + (groups < rows ? groups : rows);
}

// Part `slot` (below most_parts) of the rows: groups in ascending order, each in parts of kRows
// rows (the last one shorter).  False past the last part.  Offsets outside the rows are cut off
// and the count of parts ends at kParts, which no slot reaches, so whatever the table holds, no
// row outside them is named.  Uniform in the wave.
template <int kRows>
__device__ __forceinline__ bool find_part(const int32_t* offsets, int groups, int rows, int slot, int& g, int& row0,
                                          int& count) {
    if (!offsets) {
        g = 0;
        row0 = slot * kRows;
        count = min(rows - row0, kRows);
        return count > 0;
    }
    constexpr int kParts = 1 << 29;  // (a lane has at most 2^10 groups of 2^24 rows: 2^28 parts)
    const int lane = threadIdx.x & 63, per = (groups + kWave - 1) / kWave;
    int lo = 0, hi = 0, mine = 0;  // of the lane's groups: the last one's bounds, their parts
    for (int i = 0; i < per; ++i) {
        const int e = min(lane * per + i, groups);
        lo = min(max(offsets[e], 0), rows);
        hi = min(max(offsets[min(e + 1, groups)], lo), rows);  // past the last group: none
        mine += (hi - lo + kRows - 1) / kRows;
    }
    int upto = mine;  // inclusive sum over the lanes
#pragma unroll
    for (int s = 1; s < kWave; s *= 2) {
        const int v = __shfl_up(upto, s, kWave);
        if (lane >= s) upto = min(upto + v, kParts);
    }
    const uint64_t past = __ballot(upto > slot);
    if (!past) return false;
    const int l = __builtin_ctzll(past);
    int left = slot - __builtin_amdgcn_readlane(upto - mine, l);
    g = l * per;
    if (per == 1) {
        lo = __builtin_amdgcn_readlane(lo, l);
        hi = __builtin_amdgcn_readlane(hi, l);
    } else {
        for (;; ++g) {  // ends: the part is one of lane l's groups'
            lo = min(max(offsets[g], 0), rows);
            hi = min(max(offsets[g + 1], lo), rows);
            const int parts = (hi - lo + kRows - 1) / kRows;
            if (left < parts || g == groups - 1) break;
            left -= parts;
        }
        lo = __builtin_amdgcn_readfirstlane(lo);
        hi = __builtin_amdgcn_readfirstlane(hi);
    }
    row0 = lo + left * kRows;
    count = min(hi - row0, kRows);
    return true;
}

// ---------------------------------------------------------------------------
// Few rows to a group: bound by reading the weights
// ---------------------------------------------------------------------------

constexpr int kBfWaves = 4;
constexpr int kBfRows = 64;           // most rows of a part
constexpr int kBfSlot = 4 * 16 * kBlk;  // a wave's weights of a step: four fragments of 16 rows by a block

// kFrags fragments of 16 weight rows from LDS, fragment f at byte 2048 f: this lane's
// pieces at p0 and p1 of its row.  In one block with its wait: the compiler would wait
// for the loads into the other slot too.
template <int kFrags>
__device__ __forceinline__ void few_frags(uint32_t p0, uint32_t p1, intx8 (&w)[kFrags]) {
    intx4 f[2 * kFrags];
    if constexpr (kFrags == 4) {
        asm volatile(
            "ds_read_b128 %0, %8\n\tds_read_b128 %1, %9\n\t"
            "ds_read_b128 %2, %8 offset:2048\n\tds_read_b128 %3, %9 offset:2048\n\t"
            "ds_read_b128 %4, %8 offset:4096\n\tds_read_b128 %5, %9 offset:4096\n\t"
            "ds_read_b128 %6, %8 offset:6144\n\tds_read_b128 %7, %9 offset:6144\n\t"
            "s_waitcnt lgkmcnt(0)"
            : "=&v"(f[0]), "=&v"(f[1]), "=&v"(f[2]), "=&v"(f[3]), "=&v"(f[4]), "=&v"(f[5]), "=&v"(f[6]), "=&v"(f[7])
            : "v"(p0), "v"(p1)
            : "memory");
    } else if constexpr (kFrags == 2) {
        asm volatile(
            "ds_read_b128 %0, %4\n\tds_read_b128 %1, %5\n\t"
            "ds_read_b128 %2, %4 offset:2048\n\tds_read_b128 %3, %5 offset:2048\n\t"
            "s_waitcnt lgkmcnt(0)"
            : "=&v"(f[0]), "=&v"(f[1]), "=&v"(f[2]), "=&v"(f[3])
            : "v"(p0), "v"(p1)
            : "memory");
    } else {
        static_assert(kFrags == 1, "");
        asm volatile("ds_read_b128 %0, %2\n\tds_read_b128 %1, %3\n\ts_waitcnt lgkmcnt(0)"
                     : "=&v"(f[0]), "=&v"(f[1])
                     : "v"(p0), "v"(p1)
                     : "memory");
    }
#pragma unroll
    for (int x = 0; x < kFrags; ++x) w[x] = __builtin_shufflevector(f[2 * x], f[2 * x + 1], 0, 1, 2, 3, 4, 5, 6, 7);
}

// Rows row0 .. row0 + count - 1 (at most 16 kTF) of group g by columns n0 .. n0 + 16 kNF -
// 1, the K blocks dealt to the workgroup's four waves and their sums joined in LDS in a
// fixed order.  Weight rows are the M side of 16-wide MFMAs, rows of a the N side, so a
// lane ends with four neighbouring columns of a row.
//
// A wave's step is kU blocks of K.  Its weights come straight into one of the wave's own
// two LDS slots in whole lines, eight rows an instruction, asked for a step ahead; the
// rows of a, which every workgroup of the group reads, come from the cache into registers.
//
// Measured: 64 rows x [7168, 2048] in 32 groups 71 us, 408 MB of weights at 5.7 TB/s; 1 row x
// [8192, 8192] 14.4 us (4.7 TB/s); 1 x [2048, 1024] 3.7 us, a launch and a few trips to memory.
template <int kNF, int kTF, bool kGlu, bool kPast>
__device__ __forceinline__ void block_few_part(const BlockGemm& a, int g, int row0, int count, int n0,
                                               uint8_t (*s_w)[2][kBfSlot]) {
    constexpr int kW = kGlu ? 2 * kNF : kNF;  // weight fragments: the gate's, then the up matrix's
    constexpr int kU = 4 / (kW > kTF ? kW : kTF);
    constexpr int kFrags = kW * kU;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lr = lane & 15, lq = lane >> 4;
    const int kb_n = blk_count(a.k), nb = blk_count(a.n);
    const int64_t wat = ((int64_t)g * a.n + n0) * a.k;
    const uint32_t wbytes = (uint32_t)(a.n - n0) * (uint32_t)a.k;  // columns past the last read as zero
    const __amdgpu_buffer_rsrc_t rw = blk_rsrc(a.w + wat, wbytes), ru = blk_rsrc((kGlu ? a.wu : a.w) + wat, wbytes);
    const __amdgpu_buffer_rsrc_t ra = blk_rsrc(a.a + (int64_t)row0 * a.k, (uint32_t)count * (uint32_t)a.k);
    const uint32_t off16 = 16u * (uint32_t)a.k;
    const float *swf[kNF], *suf[kNF];
#pragma unroll
    for (int f = 0; f < kNF; ++f) {
        const int64_t at = ((int64_t)g * nb + min(n0 + 16 * f, a.n - 1) / kBlk) * kb_n;
        swf[f] = a.sw + at;
        suf[f] = (kGlu ? a.swu : a.sw) + at;
    }
    // Load q of a step: rows 8 (q % 2) .. + 7 of fragment q / 2; lane l row l / 8, chunk l % 8 in
    // LDS, which holds the row's chunk (l % 8) ^ swz8(row).
    auto issue = [&](int s, int slot) {
        uint8_t* dst = s_w[wave][slot];
#pragma unroll
        for (int q = 0; q < 2 * kFrags; ++q) {
            const int f = q / 2 % kW, row = 8 * (q & 1) + (lane >> 3);
            const int at = ((s * kBfWaves + wave) * kU + q / 2 / kW) * kBlk + ((lane & 7) ^ (4 * (q & 1) | (lane >> 4))) * 16;
            // k is a multiple of 16: a piece is inside the row or not
            const uint32_t o = at < a.k ? (uint32_t)row * (uint32_t)a.k + at + f % kNF * off16 : kNowhere;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(f < kNF ? rw : ru, (lds_void*)(dst + q * 1024), 16, o, 0, 0,
                                                     kPast ? kPastCaches : 0);
        }
    };
    struct Rows {
        intx4 x[kU][kTF][2];
        float sa[kU][kTF];
    };
    constexpr int kRowLoads = 3 * kU * kTF;
    auto load = [&](int s, Rows& r) {
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int kb = (s * kBfWaves + wave) * kU + u;
            const __amdgpu_buffer_rsrc_t rs = blk_rsrc(a.sa + (int64_t)min(kb, kb_n - 1) * a.rows + row0, count * 4);
#pragma unroll
            for (int t = 0; t < kTF; ++t) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int at = kb * kBlk + 64 * h + lq * 16;
                    const uint32_t o = at < a.k ? (uint32_t)lr * (uint32_t)a.k + at : kNowhere;
                    r.x[u][t][h] = __builtin_amdgcn_raw_buffer_load_b128(ra, o + t * off16, 0, 0);
                }
                r.sa[u][t] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(rs, (16 * t + lr) * 4, 0, 0));
            }
        }
    };
    floatx4 acc[kW][kTF] = {};
    const uint32_t p_row = lds_at(s_w[wave][0]) + lr * kBlk;
    const uint32_t p0 = p_row + ((lq ^ swz8(lr)) << 4), p1 = p_row + (((4 + lq) ^ swz8(lr)) << 4);
    auto step = [&](auto last, int s, int slot, const Rows& cur, Rows& next) {
        if constexpr (decltype(last)::value) {
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        } else {
            load(s + 1, next);
            __builtin_amdgcn_sched_barrier(0);
            issue(s + 1, slot ^ 1);
            __builtin_amdgcn_sched_barrier(0);
            // This step's loads, all older than those, have arrived (scalar loads are not
            // counted).  The count holds because a step that is not the last uses every value it
            // loads in the next one: none is dropped.
            asm volatile("s_waitcnt vmcnt(%0)" ::"n"(kRowLoads + 2 * kFrags) : "memory");
        }
        intx8 w[kFrags];
        few_frags<kFrags>(p0 + slot * kBfSlot, p1 + slot * kBfSlot, w);
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int ks = min((s * kBfWaves + wave) * kU + u, kb_n - 1);
#pragma unroll
            for (int f = 0; f < kW; ++f) {
                // a scalar load: waiting for a vector one would wait for the weights asked for before it
                const float sw = *(const __attribute__((address_space(4))) float*)((f < kNF ? swf[f % kNF] : suf[f % kNF]) + ks);
#pragma unroll
                for (int t = 0; t < kTF; ++t) {
                    const intx8 x = __builtin_shufflevector(cur.x[u][t][0], cur.x[u][t][1], 0, 1, 2, 3, 4, 5, 6, 7);
                    const floatx4 p = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w[u * kW + f], x, floatx4{}, 0, 0,
                                                                                       0, 0, 0, 0);
                    const float sc = sw * cur.sa[u][t];
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[f][t][i] = __builtin_fmaf(p[i], sc, acc[f][t][i]);
                }
            }
        }
    };
    // (a wave's blocks past the last are zeros)
    const int steps = (kb_n + kBfWaves * kU - 1) / (kBfWaves * kU);
    Rows r0, r1;
    load(0, r0);
    __builtin_amdgcn_sched_barrier(0);
    issue(0, 0);
    constexpr std::integral_constant<bool, false> more{};
    constexpr std::integral_constant<bool, true> last{};
    int s = 0;
    for (; s + 2 < steps; s += 2) {
        step(more, s, 0, r0, r1);
        step(more, s + 1, 1, r1, r0);
    }
    if (s + 1 < steps) {
        step(more, s, 0, r0, r1);
        step(last, s + 1, 1, r1, r0);
    } else {
        step(last, s, 0, r0, r1);
    }
    __syncthreads();  // the slots are free
    // the sums go through the slots' memory, one fragment of rows at a time
    floatx4 (*s_part)[kW][kWave] = (floatx4(*)[kW][kWave])s_w;
#pragma unroll
    for (int t = 0; t < kTF; ++t) {
#pragma unroll
        for (int f = 0; f < kW; ++f) s_part[wave][f][lane] = acc[f][t];
        __syncthreads();
        auto joined = [&](int f) {
            floatx4 v = s_part[0][f][lane];
#pragma unroll
            for (int x = 1; x < kBfWaves; ++x) v += s_part[x][f][lane];
            return v;
        };
        for (int f = wave; f < kNF; f += kBfWaves) {
            const int r = 16 * t + lr, col = n0 + 16 * f + 4 * lq;
            floatx4 v = joined(f);
            if constexpr (kGlu) {
                const floatx4 u = joined(kNF + f);
#pragma unroll
                for (int x = 0; x < 4; ++x) v[x] = swiglu(v[x], u[x]);
            }
            if (r >= count || col >= a.n) continue;  // n is a multiple of 8: four columns are inside or not
            const int64_t at = (int64_t)(row0 + r) * a.n + col;
            if constexpr (kGlu)
                *(floatx4*)(a.h + at) = v;
            else
                *(uint2*)(a.out + at) = uint2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
        }
        __syncthreads();
    }
}

template <int kNF, bool kGlu, bool kPast>
__global__ __launch_bounds__(kBfWaves * kWave, 2) void block_few_kernel(BlockGemm a) {
    __shared__ __attribute__((aligned(1024))) uint8_t s_w[kBfWaves][2][kBfSlot];
    int g, row0, count;
    const int most = most_parts(a.rows, a.groups, kBfRows);
    for (int slot = blockIdx.y; slot < most && find_part<kBfRows>(a.offsets, a.groups, a.rows, slot, g, row0, count);
         slot += gridDim.y) {
        const int n0 = blockIdx.x * 16 * kNF;
        if (count <= 16) block_few_part<kNF, 1, kGlu, kPast>(a, g, row0, count, n0, s_w);
        else if (count <= 32) block_few_part<kNF, 2, kGlu, kPast>(a, g, row0, count, n0, s_w);
        else block_few_part<kNF, 4, kGlu, kPast>(a, g, row0, count, n0, s_w);
    }
}

// ---------------------------------------------------------------------------
// Many rows: tiles of up to 256 x 256
// ---------------------------------------------------------------------------

// A tile of eight waves, kWM down and kWN across, each with kFI x kFJ fragments of 32 x
// 32.  A stage is one block of K: A and B codes as 128-byte rows, the A rows' scales and
// the tile's weight scales; kS stages make the ring.  All of it comes by loads straight
// into LDS through buffer descriptors: what lies past the group's last row, the matrix's
// last row or the row's end reads as zero and moves no memory, so no size needs a tile of
// its own, and a lane's offsets are the same for every tile.
//
// Measured: 131072 rows x [7168, 2048] in 32 groups 1765 to 1857 us by card, 2180 to 2072 TFLOP/s; 16384 x [8192, 8192]
// 2540.  That is bound by power: 16384 x [4096, 4096] runs at 2310 with random codes and at
// 3364 with zeros.  512 rows x [7168, 2048] in 32 groups: 79 us, weights at 6.0 TB/s.
constexpr int kBgThreads = 512;
constexpr int kBgGroups = 512;  // groups whose tables fit beside the ring; more run in the few-row form
constexpr int kBgStg = 2048;    // a wave's staged output
constexpr int kBgPatch = 8;     // M tiles of a patch
template <int kWM_, int kWN_, int kFI_, int kFJ_, int kS_>
struct BgShape {
    static constexpr int kWM = kWM_, kWN = kWN_, kFI = kFI_, kFJ = kFJ_, kS = kS_;
    static_assert(kWM * kWN == 8 && kFJ % 2 == 0 && kS >= 2, "eight waves; B fragments alternate between two registers");
    static constexpr int kM = kWM * kFI * 32, kN = kWN * kFJ * 32;
    static constexpr int kStageB = kM * kBlk;
    static constexpr int kStageS = kStageB + kN * kBlk;  // scales: an area of 64 for each wave's load
    static constexpr int kStage = kStageS + 8 * kWave * 4;
    static constexpr int kRing = kS * kStage;
    static constexpr int kMax = kRing + 8 * kBgStg;      // behind the staged output; SwiGLU: largest |h| by row and wave
    static constexpr int kTables = kMax + kM * kWN * 4;
    static constexpr int kSmem = kTables + (3 * kBgGroups + 1) * 4;
    static_assert(kSmem <= 160 * 1024, "the LDS");
    static constexpr int kLoads = (kM + kN) / 64 + 1;    // of a wave and stage
};

// What a tile's loads start from, uniform in a wave: codes of this wave's A and B
// rows, and the scales of 64 A rows (the first kM / 64 waves) or one weight scale.
struct BgSource {
    const uint8_t *a, *b;
    const float* s;
    uint32_t a_bytes, b_bytes, s_bytes;
};

struct BgTile {
    int g, row0, count, n0;  // n0: first output column; count: rows, at most kM; 0: no tile
};

// LDS accesses between two tiles' products, in asm: the compiler would wait for the next
// tile's loads into the ring, and for the stores before them, too.
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ void lds_put(uint32_t at, uint32_t v) {
    asm volatile("ds_write_b32 %0, %1" ::"v"(at), "v"(v) : "memory");
}
__device__ __forceinline__ void lds_put2(uint32_t at, u32x2 v) {
    asm volatile("ds_write_b64 %0, %1" ::"v"(at), "v"(v) : "memory");
}
__device__ __forceinline__ void lds_get4(uint32_t at, u32x4& d) {
    asm volatile("ds_read_b128 %0, %1\n\ts_waitcnt lgkmcnt(0)" : "=&v"(d) : "v"(at) : "memory");
}
// The lane, formed anew where it is needed: kept live over the products it would be spilled,
// and a spilled value's return waits for every load and store before it.
__device__ __forceinline__ int lane_now() {
    int l;
    asm volatile("v_mbcnt_lo_u32_b32 %0, -1, 0\n\tv_mbcnt_hi_u32_b32 %0, -1, %0" : "=v"(l));
    return l;
}

__device__ __forceinline__ int lds_get(uint32_t at) {
    int d;
    asm volatile("ds_read_b32 %0, %1\n\ts_waitcnt lgkmcnt(0)" : "=&v"(d) : "v"(at) : "memory");
    return d;
}

// The wave's own writes, then two reads: LDS serves a wave in order.
__device__ __forceinline__ void lds_put_get(uint32_t at0, uint32_t at1, u32x4& d0, u32x4& d1) {
    asm volatile("s_waitcnt lgkmcnt(0)\n\tds_read_b128 %0, %2\n\tds_read_b128 %1, %3\n\ts_waitcnt lgkmcnt(0)"
                 : "=&v"(d0), "=&v"(d1)
                 : "v"(at0), "v"(at1)
                 : "memory");
}

// A store that leaves the caches alone (in asm: two branches that store the same value to
// the same place, with and without the hint, become one store without it).  The s_nop is the
// two wait states that a store of more than 8 bytes needs on gfx950 before a VALU instruction
// may write its data registers, which the compiler keeps only after stores of its own.
__device__ __forceinline__ void store_past(uint16_t* at, u32x4 v) {
    asm volatile("global_store_dwordx4 %0, %1, off nt\n\ts_nop 1" ::"v"(at), "v"(v) : "memory");
}

template <class C, bool kGlu, bool kPast>
__device__ __forceinline__ void block_gemm_tiles(const BlockGemm& p) {
    constexpr int kFI = C::kFI, kFJ = C::kFJ, kWM = C::kWM, kWN = C::kWN;
    constexpr int kCols = kGlu ? C::kN / 2 : C::kN;  // output columns of a tile
    static_assert(!kGlu || kCols == kBlk, "a block of h is a tile's columns");
    extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
    int32_t* s_first = (int32_t*)(smem + C::kTables);  // [groups + 1] M tiles before each group
    int32_t* s_lo = s_first + p.groups + 1;            // [groups] its rows
    int32_t* s_hi = s_lo + p.groups;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / kWN, wn = wave % kWN;
    const int KB = blk_count(p.k), NB = blk_count(p.n), NT = (p.n + kCols - 1) / kCols;

    if (wave == 0) {
        const int most = most_parts(p.rows, p.groups, C::kM);
        int before = 0;
        for (int e0 = 0; e0 < p.groups; e0 += kWave) {
            const int e = e0 + lane;
            int lo = 0, hi = 0;
            if (e < p.groups) {  // bounds outside the rows are cut off
                lo = p.offsets ? min(max(p.offsets[e], 0), p.rows) : 0;
                hi = p.offsets ? min(max(p.offsets[e + 1], lo), p.rows) : p.rows;
            }
            const int tiles = (hi - lo + C::kM - 1) / C::kM;
            int upto = tiles;
#pragma unroll
            for (int s = 1; s < kWave; s *= 2) {
                const int v = __shfl_up(upto, s, kWave);
                if (lane >= s) upto += v;
            }
            if (e < p.groups) {
                s_first[e] = min(before + upto - tiles, most);
                s_lo[e] = lo;
                s_hi[e] = hi;
            }
            before += __shfl(upto, kWave - 1, kWave);
        }
        if (lane == 0) s_first[p.groups] = min(before, most);
    }
    __syncthreads();
    // Workgroup b runs on XCD b % 8, whose workgroups take neighbouring tiles, so that they
    // share panels in its L2: group by group, kBgPatch M tiles by all columns after the other,
    // M fastest.  32 workgroups then read 8 row and 4 column panels; with all of a group's M
    // tiles first, 16384 x [8192, 8192] took 925 us instead of 862.
    const int total = __builtin_amdgcn_readfirstlane(s_first[p.groups]) * NT;
    const int xcd = blockIdx.x & 7, per = (total + 7) / 8, step = gridDim.x >> 3;
    const int t_end = min((xcd + 1) * per, total);
    const uint32_t t_first = lds_at(smem) + C::kTables, t_lo = t_first + (p.groups + 1) * 4, t_hi = t_lo + p.groups * 4;
    auto uniform = [](uint32_t at) { return __builtin_amdgcn_readfirstlane(lds_get(at)); };
    auto tile_at = [&](int t) {
        BgTile r{0, 0, 0, 0};
        if (t >= t_end) return r;
        const int l = lane_now();
        int e = 0;  // the last group with no more than t tiles before it; it is not empty
        for (int e0 = 0; e0 < p.groups; e0 += kWave) {
            const int x = e0 + l;
            const int before = lds_get(t_first + min(x, p.groups - 1) * 4);
            const uint64_t at = __ballot(x < p.groups && before * NT <= t);
            if (!at) break;
            e = e0 + 63 - __builtin_clzll(at);
        }
        r.g = e;
        const int f0 = uniform(t_first + e * 4), f1 = uniform(t_first + e * 4 + 4);
        const int in = t - f0 * NT, block = in / (kBgPatch * NT), rest = in - block * kBgPatch * NT;
        const int high = min(kBgPatch, f1 - f0 - block * kBgPatch), col = rest / high;
        r.n0 = col * kCols;
        r.row0 = uniform(t_lo + e * 4) + (block * kBgPatch + rest - col * high) * C::kM;
        r.count = min(uniform(t_hi + e * 4) - r.row0, C::kM);
        return r;
    };
    constexpr int kRowsA = C::kM / 8, kRowsB = C::kN / 8;  // rows of a stage that a wave loads
    constexpr int kScaleWaves = C::kM / 64;                // waves that load A scales
    constexpr int kScalesW = kGlu ? 2 : C::kN / kBlk;      // weight scales of a stage
    auto source_of = [&](const BgTile& t) {
        BgSource s{};
        if (t.count == 0) return s;
        s.a = p.a + (int64_t)(t.row0 + wave * kRowsA) * p.k;
        s.a_bytes = (uint32_t)max(t.count - wave * kRowsA, 0) * (uint32_t)p.k;
        // B rows of the stage are columns n0 ..; with SwiGLU, of a wave's kFJ fragments the
        // first half are columns of the gate's, the second the same of the up matrix, so that
        // a wave ends with both (a wave then loads just one fragment's rows)
        static_assert(!kGlu || kRowsB == 32, "");
        const bool up = kGlu && wave % kFJ >= kFJ / 2;
        const int br = t.n0 + (kGlu ? wave / kFJ * (kFJ * 16) + wave % (kFJ / 2) * 32 : wave * kRowsB);
        s.b = (up ? p.wu : p.w) + ((int64_t)t.g * p.n + br) * p.k;
        s.b_bytes = (uint32_t)max(p.n - br, 0) * (uint32_t)p.k;
        if (wave < kScaleWaves) {
            s.s = p.sa + t.row0 + wave * 64;
            s.s_bytes = (uint32_t)max(t.count - wave * 64, 0) * 4;
        } else {  // the tile's column blocks, or the gate's and the up matrix's
            const int x = wave - kScaleWaves, nb = t.n0 / kBlk + (kGlu ? 0 : x);
            s.s = (kGlu && x == 1 ? p.swu : p.sw) + ((int64_t)t.g * NB + min(nb, NB - 1)) * KB;
            s.s_bytes = x < kScalesW && nb < NB ? 4 : 0;
        }
        return s;
    };
    const int64_t s_step = wave < kScaleWaves ? p.rows : 1;  // scales from block to block of K

    // A load fills eight rows of a stage: lane l row l / 8, chunk l % 8 in LDS, which holds the
    // row's chunk (l % 8) ^ swz8(row), that is with bit 2 turned for every other eight rows.
    const int c_even = (lane & 7) ^ (lane >> 4), c_odd = c_even ^ 4;
    uint32_t v_even = (uint32_t)(lane >> 3) * (uint32_t)p.k + c_even * 16;
    uint32_t v_odd = (uint32_t)(lane >> 3) * (uint32_t)p.k + c_odd * 16;
    const uint32_t v_eight = 8u * (uint32_t)p.k;
    BgSource src, nxt;
    // Part x of kParts of the A or the B half (with the scales) of stage s of this tile, or past
    // its last of the next tile's; past the last tile's last nothing is read and the slot, which
    // no wave reads any more, is filled with zeros.
    auto issue = [&](auto half_a, auto part, auto parts, int s_, int slot) {
        constexpr bool kA = decltype(half_a)::value;
        constexpr int kRows = kA ? kRowsA : kRowsB, kPart = decltype(part)::value, kParts = decltype(parts)::value;
        const bool beyond = s_ >= KB;
        const BgSource q = beyond ? nxt : src;
        const int s = beyond ? s_ - KB : s_;
        const int left = q.a ? p.k - s * kBlk : 0;  // bytes of a row from this stage on
        uint8_t* st = smem + slot * C::kStage;
        const __amdgpu_buffer_rsrc_t r = kA ? blk_rsrc(q.a, q.a_bytes) : blk_rsrc(q.b, q.b_bytes);
        const bool in_e = c_even * 16 < left, in_o = c_odd * 16 < left;
#pragma unroll
        for (int i = kRows / 8 * kPart / kParts; i < kRows / 8 * (kPart + 1) / kParts; ++i) {
            // (fewer than sixteen rows to a wave: the wave's own place tells which)
            const bool odd = kRows >= 16 ? (i & 1) : (wave & 1);
            const uint32_t v = (odd ? v_odd : v_even) + i * v_eight + s * kBlk;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                r, (lds_void*)(st + (kA ? 0 : C::kStageB) + wave * kRows * kBlk + i * 1024), 16,
                (odd ? in_o : in_e) ? v : kNowhere, 0, 0,
                kPast && !kA ? kPastCaches : 0);
        }
        // (a wave without scales fills its area with zeros: a branch here would let the
        // compiler move every addition of the stage past it)
        if (!kA && kPart == 0)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(blk_rsrc(q.s + s * s_step, left > 0 ? q.s_bytes : 0),
                                                     (lds_void*)(st + C::kStageS + wave * 256), 4, lane * 4, 0, 0, 0);
    };
    constexpr std::integral_constant<bool, true> kHalfA{};
    constexpr std::integral_constant<bool, false> kHalfB{};
    constexpr std::integral_constant<int, 0> k0{};
    constexpr std::integral_constant<int, 1> k1{};
    constexpr std::integral_constant<int, 2> k2{};
    // With two slots, A's half of a slot is loaded again half a stage before B's: its
    // fragments are in registers before the stage begins.
    constexpr bool kEarlyA = C::kS == 2;
    static_assert(!kEarlyA || kFJ >= 4, "the A half's barrier is not the stage's");

    const int fr = lane & 31, half = lane >> 5;
    const int fsw = swz8(fr);  // a fragment's rows differ from fr by multiples of 32
    const int arow = (wm * 32 + fr) * kBlk, brow = C::kStageB + (wn * kFJ * 32 + fr) * kBlk;
    // The two operands' parts of a K block fall to the lanes alike: K step ks takes chunks
    // 4 ks + half and 4 ks + 2 + half.
    auto read_frag = [&](int slot, int row, intx8 (&f)[2]) {
        const uint8_t* st = smem + slot * C::kStage + row;
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
            const intx4 lo = *(const intx4*)(st + (((4 * ks + half) ^ fsw) * 16));
            const intx4 hi = *(const intx4*)(st + (((4 * ks + 2 + half) ^ fsw) * 16));
            f[ks] = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
        }
    };
    intx8 fa[kFI][2], fb[2][2];
    constexpr int kSW = kGlu ? 2 : 1;  // weight scales of a wave
    float sa[kFI], sw[kSW], sa_n[kFI], sw_n[kSW];
    auto read_scales = [&](int slot) {
        const float* st = (const float*)(smem + slot * C::kStage + C::kStageS);
#pragma unroll
        for (int i = 0; i < kFI; ++i) sa_n[i] = st[(i * kWM + wm) * 32 + fr];
        const float* w = st + kScaleWaves * kWave;
        sw_n[0] = kGlu ? w[0] : w[wn * kFJ * 32 / kBlk * kWave];
        if constexpr (kGlu) sw_n[1] = w[kWave];
    };
    floatx16 acc[kFI][kFJ];
    // Fragment f = j kFI + i of a stage: both K steps from a zero accumulator, then scaled into
    // the sum.  B is the first operand, so element 4 q + s of lane l is column 8 q + 4 (l / 32) +
    // s of row l % 32: a lane has one row of A, and its scale is one register.  A fragment is
    // added while the next one multiplies, the last one of a stage in the next stage; the
    // order is fixed here, since the compiler's own keeps six products at once and spills.
    constexpr int kF = kFI * kFJ;
    floatx16 v[2];
    float sc[2];
    auto multiply = [&](int f) {
        const int i = f % kFI, j = f / kFI;
        v[f & 1] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fb[j & 1][0], fa[i][0], floatx16{}, 0, 0, 0, 0, 0, 0);
        v[f & 1] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fb[j & 1][1], fa[i][1], v[f & 1], 0, 0, 0, 0, 0, 0);
        __builtin_amdgcn_sched_barrier(0);  // then an addition: the product that it takes is done by now
    };
    auto add = [&](int f) {
#pragma unroll
        for (int c = 0; c < 16; ++c)
            acc[f % kFI][f / kFI][c] = __builtin_fmaf(v[f & 1][c], sc[f & 1], acc[f % kFI][f / kFI][c]);
    };
    auto pin = [] { __builtin_amdgcn_sched_barrier(0); };

    int t = xcd * per + (blockIdx.x >> 3);
    BgTile tile = tile_at(t);
    if (tile.count == 0) return;
    src = source_of(tile);
    t += step;
    BgTile next = tile_at(t);
    nxt = source_of(next);
    // (KB is at least kS, so a tile's loads reach no further than the next tile)
#pragma unroll
    for (int s = 0; s < C::kS; ++s) {
        issue(kHalfA, k0, k1, s, s);
        issue(kHalfB, k0, k1, s, s);
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    int slot = 0, freed = 0;
    // An output of more than the last cache's 256 MB whose 64 columns are whole lines leaves the
    // caches to the operands (131072 x [7168, 2048], 32 groups: 1851 -> 1828 us; but 16384 x
    // [2048, 1024], 67 MB: 38.4 -> 42, and 100000 x [2040, 512], part lines: 186 -> 245).
    const bool stream = !kGlu && p.n % 64 == 0 && (int64_t)p.rows * p.n > (128ll << 20);
    // Whether the tile before was whole, so that each wave stored kStores times at least: the first
    // stage then waits for its loads, which are older, and not for those stores too.  (With the
    // line above and nothing else that waits for them between two tiles 1851 -> 1798 us; 65536 x
    // [4096, 1024] in 8 groups 318 -> 298; SwiGLU of 24576 x [1024, 2048], 64 groups 149 -> 144.)
    bool stored = false;
#pragma unroll
    for (int i = 0; i < kFI; ++i) read_frag(0, arow + i * kWM * 32 * kBlk, fa[i]);
    read_frag(0, brow, fb[0]);
    read_scales(0);
    for (;;) {
        asm volatile("" : "+v"(v_even), "+v"(v_odd));  // opaque: the first stage's addresses are not kept
#pragma unroll
        for (int i = 0; i < kFI; ++i)
#pragma unroll
            for (int j = 0; j < kFJ; ++j) acc[i][j] = floatx16{};
        v[(kF - 1) & 1] = floatx16{};
        sc[(kF - 1) & 1] = 0.0f;
        for (int s = 0; s < KB; ++s) {
#pragma unroll
            for (int f = 0; f < kF; ++f) {
                const int i = f % kFI, j = f / kFI;
                pin();
                if (i == 0 && j < kFJ - 1) read_frag(slot, brow + (j + 1) * 32 * kBlk, fb[(j + 1) & 1]);
                if (kEarlyA && i == 0 && j == kFJ / 2) {
                    // every wave has multiplied its A fragments of stage s: they have left LDS
                    asm volatile("" ::: "memory");
                    __builtin_amdgcn_s_barrier();
                    asm volatile("" ::: "memory");
                }
                if (i == 0 && j == kFJ - 1) {
                    // stage s + 1 has landed, and no wave reads stage s any more
                    constexpr int kStores = kGlu ? kFI * kFJ / 2 : 2 * kFI * kFJ;
                    constexpr int kAfter = kEarlyA ? kRowsA / 8 : (C::kS - 2) * C::kLoads;
                    if (stored)
                        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(kAfter + kStores) : "memory");
                    else
                        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(kAfter) : "memory");
                    stored = false;
                    __builtin_amdgcn_s_barrier();
                    asm volatile("" ::: "memory");
                    if (!kEarlyA) issue(kHalfA, k0, k1, s + C::kS, slot);
                    freed = slot;
                    slot = slot == C::kS - 1 ? 0 : slot + 1;
                    read_frag(slot, brow, fb[(j + 1) & 1]);
                    read_scales(slot);
                }
                multiply(f);
                // Loads go out a few at a time under the products: all of a stage's at once, and the
                // waves wait for the address unit to take them (264 -> 252 us for 16384 x [4096, 4096]).
                if (kEarlyA && j == kFJ / 2) {
                    if (kFI == 1) issue(kHalfA, k0, k1, s + C::kS, slot);
                    else if (i == 0) issue(kHalfA, k0, k2, s + C::kS, slot);
                    else issue(kHalfA, k1, k2, s + C::kS, slot);
                }
                if (j == kFJ - 1) {
                    if (kFI == 1) issue(kHalfB, k0, k1, s + C::kS, freed);
                    else if (i == 0) issue(kHalfB, k0, k2, s + C::kS, freed);
                    else issue(kHalfB, k1, k2, s + C::kS, freed);
                }
                if (f == 0) {
                    add(kF - 1);  // of the stage before
#pragma unroll
                    for (int x = 0; x < kFI; ++x) sa[x] = sa_n[x];
#pragma unroll
                    for (int x = 0; x < kSW; ++x) sw[x] = sw_n[x];
                } else {
                    add(f - 1);
                }
                sc[f & 1] = sa[i] * sw[kGlu ? j / (kFJ / 2) : 0];
                pin();
                if (j == kFJ - 1) read_frag(slot, arow + i * kWM * 32 * kBlk, fa[i]);  // of the next stage
            }
        }
        add(kF - 1);

        const uint32_t stg = lds_at(smem) + C::kRing;
        const int l = lane_now();
        if constexpr (!kGlu) {
            // 16 rows of 64 columns at a time through the wave's own block of LDS (chunk c of row r
            // at c ^ swz8(r)) and out in whole lines; no barrier, so the waves part here.  (32 rows of
            // all columns at a time by the whole workgroup, with two barriers each: 6.8 us a tile of
            // 256 x 256.)
            const uint32_t blk = stg + wave * kBgStg;
            const int r16 = l & 15, h2 = (l >> 5) & 1, r0 = l >> 3, ch = l & 7;
            const uint32_t put = blk + r16 * kBlk + 8 * h2;
            const uint32_t g0 = blk + r0 * kBlk + ((ch ^ swz8(r0)) << 4), g1 = blk + (r0 + 8) * kBlk + ((ch ^ swz8(r0 + 8)) << 4);
#pragma unroll
            for (int i = 0; i < kFI; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int row = (i * kWM + wm) * 32 + 16 * h;
                    if (row >= tile.count) break;
#pragma unroll
                    for (int jp = 0; jp < kFJ / 2; ++jp) {
                        if (((l >> 4) & 1) == h) {
#pragma unroll
                            for (int c = 0; c < 8; ++c) {
                                const floatx16& x = acc[i][2 * jp + (c >> 2)];
                                const int q = c & 3;
                                lds_put2(put + ((c ^ swz8(r16)) << 4),
                                         u32x2{pack_bf16x2(x[4 * q], x[4 * q + 1]), pack_bf16x2(x[4 * q + 2], x[4 * q + 3])});
                            }
                        }
                        u32x4 d0, d1;
                        lds_put_get(g0, g1, d0, d1);
                        const int col = tile.n0 + (wn * kFJ + 2 * jp) * 32 + ch * 8;
                        uint16_t* dst = p.out + (int64_t)(tile.row0 + row + r0) * p.n + col;
                        const bool col_in = col < p.n;  // n is a multiple of 8
                        const bool in0 = col_in && row + r0 < tile.count, in1 = col_in && row + r0 + 8 < tile.count;
                        if (stream) {
                            if (in0) store_past(dst, d0);
                            if (in1) store_past(dst + 8 * (int64_t)p.n, d1);
                        } else {
                            if (in0) *(u32x4*)dst = d0;
                            if (in1) *(u32x4*)(dst + 8 * (int64_t)p.n) = d1;
                        }
                    }
                }
        } else {
            // h in place of the gate's fragments; a row's block of 128 is kWN waves' columns
            constexpr int kJ = kFJ / 2;
            const int h2 = l >> 5, c0 = wn * kJ * 32 + 4 * h2;  // this lane's first column of the tile
            const int rl = wm * 32 + (l & 31);
            const uint32_t mx = lds_at(smem) + C::kMax;
            float m[kFI];
#pragma unroll
            for (int i = 0; i < kFI; ++i) {
                m[i] = 0.0f;
#pragma unroll
                for (int j = 0; j < kJ; ++j)
#pragma unroll
                    for (int c = 0; c < 16; ++c) {
                        const float g = acc[i][j][c];
                        const float h = swiglu(g, acc[i][kJ + j][c]);  // (past column n: of zeros)
                        acc[i][j][c] = h;
                        m[i] = fmaxf(m[i], fabsf(h));
                    }
                m[i] = fmaxf(m[i], __shfl_xor(m[i], 32, kWave));
                const float mi = m[i];  // (a cast of the array's element would be of its first one)
                if (h2 == 0)
                    lds_put(mx + ((i * kWM * 32 + rl) * kWN + wn) * 4, __builtin_bit_cast(uint32_t, mi));
            }
            lds_barrier();
            // A wave's columns of 32 rows go through its own block of LDS (chunk c of row r at c ^
            // r / 4) and out; the waves part here.
            constexpr int kChunks = 2 * kJ;  // of 16 codes
            const uint32_t blk = stg + wave * kBgStg;
            auto chunk_at = [&](int r, int c) { return blk + r * (16 * kChunks) + ((c ^ ((r >> 2) & (kChunks - 1))) << 4); };
            const int r = l & 31;
#pragma unroll
            for (int i = 0; i < kFI; ++i) {
                const int base = (i * kWM + wm) * 32;  // the wave's first row of these
                if (base >= tile.count) break;
                u32x4 all;  // the row's maxima (with two waves across, the next row's behind them)
                lds_get4(mx + (base + r) * kWN * 4 / 16 * 16, all);
                const uint32_t a0 = all[0], a1 = all[1], a2 = all[2], a3 = all[3];
                auto f32 = [](uint32_t x) { return __builtin_bit_cast(float, x); };
                const float lo = fmaxf(f32(a0), f32(a1)), hi = fmaxf(f32(a2), f32(a3));
                const int e = blk_exp(kWN == 4 ? fmaxf(lo, hi) : (r & 1 ? hi : lo));
                const int64_t row = tile.row0 + base + r;
                const bool row_in = base + r < tile.count;
                if (wn == 0 && h2 == 0 && row_in) p.hs[(int64_t)(tile.n0 / kBlk) * p.rows + row] = pow2f(e);
                const float inv = pow2f(-e);
#pragma unroll
                for (int j = 0; j < kJ; ++j)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const floatx16& x = acc[i][j];
                        lds_put(chunk_at(r, 2 * j + (q >> 1)) + 8 * (q & 1) + 4 * h2,
                                fp8x4(x[4 * q] * inv, x[4 * q + 1] * inv, x[4 * q + 2] * inv, x[4 * q + 3] * inv));
                        const int col = tile.n0 + c0 + 32 * j + 8 * q;
                        if (p.h16 && row_in && col < p.n)
                            *(u32x2*)(p.h16 + row * p.n + col) =
                                u32x2{pack_bf16x2(x[4 * q], x[4 * q + 1]), pack_bf16x2(x[4 * q + 2], x[4 * q + 3])};
                    }
                const int r0 = l / kChunks, ch = l % kChunks, col = tile.n0 + wn * kJ * 32 + ch * 16;
                uint8_t* dst = p.hq + (int64_t)(tile.row0 + base + r0) * p.n + col;
                u32x4 d0, d1;
                if constexpr (kJ == 2) {  // 16 rows at once
                    lds_put_get(chunk_at(r0, ch), chunk_at(r0 + 16, ch), d0, d1);
                    if (col < p.n && base + r0 + 16 < tile.count) *(u32x4*)(dst + 16 * (int64_t)p.n) = d1;
                } else {
                    static_assert(kJ == 1, "");
                    lds_get4(chunk_at(r0, ch), d0);
                }
                if (col < p.n && base + r0 < tile.count) *(u32x4*)dst = d0;
            }
        }
        if (next.count == 0) break;
        stored = kEarlyA && tile.count == C::kM && tile.n0 + kCols <= p.n;
        tile = next;
        src = nxt;
        t += step;
        next = tile_at(t);
        nxt = source_of(next);
    }
    // zeros may still be on their way into the ring
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}

template <class C, bool kGlu, bool kPast>
__global__ __launch_bounds__(kBgThreads, 2) void block_gemm_kernel(BlockGemm p) {
    block_gemm_tiles<C, kGlu, kPast>(p);
}

using Bg256x256 = BgShape<4, 2, 2, 4, 2>;
using Bg128x256 = BgShape<4, 2, 1, 4, 2>;
using Bg128x128 = BgShape<4, 2, 1, 2, 4>;
using Bg64x256 = BgShape<2, 4, 1, 2, 3>;

enum BlockForm { kFormFew, kForm256x256, kForm128x256, kForm128x128, kForm64x256 };

// Groups with rows, routed evenly.
static double active_groups(int64_t rows, int groups) {
    return groups * (1.0 - pow(1.0 - 1.0 / groups, (double)rows));
}

// Whether the weights' loads leave the caches alone: more than the last cache's 256 MB of them,
// and so few rows to a group that one part holds them and the weights are read once (us: SwiGLU
// of [2048, 7168] in 32 groups, 64 rows 163 -> 155, 512 rows 172 -> 153; [7168, 2048] in 32
// groups, 512 rows 94 -> 87; but 2048 rows 119 -> 133, and 8 rows, which need 105 MB of
// weights, 22.6 -> 24.3).
static bool weights_past_caches(const BlockGemm& a) {
    const double active = active_groups(a.rows, a.groups);
    return a.rows <= active * (kBfRows / 2) && active * a.n * a.k * (a.wu ? 2 : 1) > 256.0 * (1 << 20);
}

// Parts of at most m rows, routed evenly: the sum over groups of the expected ceil(rows / m),
// that is the chance of more than j m rows over all j, a group's rows being normal about their
// mean with its root as deviation.
static double expected_parts(int64_t rows, int groups, int m) {
    if (groups == 1) return (double)((rows + m - 1) / m);
    const double mean = (double)rows / groups, dev = sqrt(mean);
    if (2 * dev > m) return groups * (mean / m + 0.5);
    double sum = active_groups(rows, groups);
    int64_t j = std::max<int64_t>(1, (int64_t)ceil((mean - 4 * dev) / m));
    sum += (double)groups * (j - 1);
    for (; j * m < mean + 4 * dev; ++j) sum += groups * 0.5 * erfc((j * m + 0.5 - mean) / (sqrt(2.0) * dev));
    return sum;
}

// Most of up to `rows` rows whose SwiGLU product may fall to the few-row form, which leaves h in
// fp32 in the caller's workspace: no more for fewer rows, so that a workspace for many serves
// fewer.  All of them where no tile fits, and for narrow outputs, whose h is small beside the
// rows; else a bound that lies above every choice (of 10^6 shapes drawn on logarithmic scales
// the times below would choose it for 3612 rows, or 53 rows to a group, at most).
int64_t block_few_rows(int64_t rows, int n, int k, int groups) {
    if (groups > kBgGroups || n < kBlk || blk_count(k) < Bg128x256::kS) return rows;
    return std::min<int64_t>(rows, std::max(4096, kBfRows * groups));
}

// The form with the least expected time, in us.  A tile takes a block of K in `low` us where
// it is one of few and in `full` us where every CU has one, and `end` us for its epilogue;
// tiles run in rounds of one to a CU, while codes are read at `rate` TB/s.  Larger tiles need
// less of everything for each element, smaller ones fill the CUs sooner and pad a group's rows
// less.  The few-row form needs more the more fragments of 16 rows a part has; past 64 groups a
// workgroup takes longer to find its part.  The constants are fitted to 1200 shapes, 1 to
// 32768 rows, 1 to 256 groups, n up to 7168 and k of 416 to 7168, drawn evenly on
// logarithmic scales, and those below, each timed in every form.  On 400 others the chosen
// form is 1.5 % slower than the best one on average, and more than 10 % slower for 3 in 100.
// The table's contents stay on the device, so the choice knows even routing only: with half of
// the rows in one group 512 rows x [7168, 2048] in 32 groups take 81 us instead of 78, 2048 114
// instead of 106, 512 rows of SwiGLU of [2048, 7168] 134 instead of 100, 1024 of [1024, 2048] in
// 64 groups 41 instead of 29.
// Measured, us, tiles of 256 x 256, 128 x 256, 128 x 128, 64 x 256 and the few-row form (-: not
// timed):
//   1 row x [2048, 1024]       -, -, 8.2, 9.2, 3.7;   64 rows x [4096, 4096]  -, -, 21, 26, 12
//   256 rows x [4096, 4096]    43, 31, 22, 27, 39;    2048 rows               48, 40, 48, 56, 268
//   4096 rows                  61, 78, 91, 104, 531;  16384 rows              234, 299, 344, 394, -
//   16 groups of [4096, 4096]  32 rows -, -, 63, 66, 49;  128 rows            -, -, 67, 69, 53
//   32 groups of [7168, 2048]  64 rows -, -, 85, 77, 71;  512 rows            -, -, 98, 85, 87
//   1024 rows                  112, 103, 100, 96, 116;    2048 rows           125, 113, 108, 113, -
//   3000 rows                  123, 117, 114, 120, -;     8192 rows           186, 196, 216, 226, 957
//   131072 rows                1798, 2272, 2574, 2912, 14243
//   SwiGLU, [2048, 7168]       64 rows -, -, -, 134, 132; 512 rows            -, -, -, 142, 160
//   1500 rows                  206, 179, -, 163, 211;     2048 rows           208, 191, -, 181, -
//   256 groups of [512, 1024]  512 rows -, -, 32, 27, 31; SwiGLU              -, -, -, 50, 58
static BlockForm block_form(int64_t rows, int n, int k, int groups, bool glu) {
    const double r = (double)rows, kb = blk_count(k), active = active_groups(rows, groups);
    const double per_group = r / active, wide = glu ? 2 : 1;
    const double strips = ((n + 15) / 16) * expected_parts(rows, groups, kBfRows) / 256;
    double busy = per_group <= 16 ? 1 : per_group <= 32 ? 1.65 : 2.55;
    if (groups > 1) {  // rows differ from group to group: 1 to 8 rows, 1.2 at 16, 1.65 at 32, 2.55 from 64 on
        const double at = log2(std::min(std::max(per_group, 8.0), 64.0)) - 3;
        busy = at <= 1 ? 1 + 0.2 * at : at <= 2 ? 1.2 + 0.45 * (at - 1) : 1.65 + 0.9 * (at - 2);
    }
    BlockForm best = kFormFew;
    double least = 4.2 + (glu ? 2.2 : 1) * std::max(kb * 0.075 * std::min(busy, 2.0),
                                                    strips * busy * (kb * 0.08 + (groups > kWave ? 0.32 : 0.19)));
    if (groups > kBgGroups) return best;
    if (glu && rows > block_few_rows(rows, n, k, groups)) least = INFINITY;
    const double bytes = wide * active * n * k + r * k;
    const struct { BlockForm form; int m, n, stages; double low, full, end, rate; } tiles[] = {
        {kForm256x256, 256, 256, Bg256x256::kS, 1.5, 1.63, 3.6, 5.0},
        {kForm128x256, 128, 256, Bg128x256::kS, 0.9, 1.08, 2.7, 4.8},
        {kForm128x128, 128, 128, Bg128x128::kS, 0.63, 0.68, 1.4, 5.2},
        {kForm64x256, 64, 256, Bg64x256::kS, 0.735, 0.965, 2.05, 5.5}};
    for (const auto& t : tiles) {
        if (kb < t.stages || (glu && t.n != 256)) continue;  // a block of h is half of 256 columns
        const int cols = glu ? t.n / 2 : t.n;
        const double rounds = expected_parts(rows, groups, t.m) * ((n + cols - 1) / cols) / 256;
        const double run = (rounds <= 1 ? 1 : rounds <= 3 ? ceil(rounds) : rounds + 0.25) *
                           (kb * (rounds <= 1 ? t.low : t.full) + t.end);
        const double read = bytes / (t.rate * 1e6);
        const double us = 3.2 + std::max(run, read) + 0.2 * std::min(run, read);
        if (us < least) {
            least = us;
            best = t.form;
        }
    }
    return best;
}

bool block_gemm_large(int64_t rows, int n, int k, int groups) { return block_form(rows, n, k, groups, true) != kFormFew; }

template <bool kPast>
static void launch_block_gemm_few(const BlockGemm& a, hipStream_t stream) {
#define BLOCK_FEW(NF, GLU)                                                                                      \
    hipLaunchKernelGGL((block_few_kernel<NF, GLU, kPast>),                                                      \
                       dim3((a.n + 16 * NF - 1) / (16 * NF), std::min(most_parts(a.rows, a.groups, kBfRows), 65535)), \
                       dim3(kBfWaves * kWave), 0, stream, a)
    const int64_t strips = (int64_t)((a.n + 15) / 16) * std::min(a.rows, a.groups);
    if (a.wu) {
        if (strips >= 2 * 512) BLOCK_FEW(2, true);
        else BLOCK_FEW(1, true);
    } else {
        if (strips >= 4 * 512) BLOCK_FEW(4, false);
        else if (strips >= 2 * 512) BLOCK_FEW(2, false);
        else BLOCK_FEW(1, false);
    }
#undef BLOCK_FEW
}

template <class C, bool kGlu, bool kPast = false>
static void launch_block_gemm_tiles(const BlockGemm& a, hipStream_t stream) {
    const int cols = kGlu ? C::kN / 2 : C::kN;
    const int64_t tiles = (int64_t)most_parts(a.rows, a.groups, C::kM) * ((a.n + cols - 1) / cols);
    const int grid = (int)std::min<int64_t>((tiles + 7) / 8 * 8, 256);  // a multiple of the XCDs
    hipLaunchKernelGGL((block_gemm_kernel<C, kGlu, kPast>), dim3(grid), dim3(kBgThreads), C::kSmem, stream, a);
}

void launch_block_gemm(const BlockGemm& a, hipStream_t stream) {
    const bool glu = a.wu != nullptr, past = weights_past_caches(a);
    switch (block_form(a.rows, a.n, a.k, a.groups, glu)) {
        case kFormFew:
            if (past) launch_block_gemm_few<true>(a, stream);
            else launch_block_gemm_few<false>(a, stream);
            return;
        case kForm256x256:
            if (glu) launch_block_gemm_tiles<Bg256x256, true>(a, stream);
            else launch_block_gemm_tiles<Bg256x256, false>(a, stream);
            return;
        case kForm128x256:
            if (glu) launch_block_gemm_tiles<Bg128x256, true>(a, stream);
            else launch_block_gemm_tiles<Bg128x256, false>(a, stream);
            return;
        case kForm128x128: launch_block_gemm_tiles<Bg128x128, false>(a, stream); return;
        case kForm64x256:  // (few rows to a group and many weights fall to other tiles at a few sizes only)
            if (glu && past) launch_block_gemm_tiles<Bg64x256, true, true>(a, stream);
            else if (glu) launch_block_gemm_tiles<Bg64x256, true>(a, stream);
            else if (past) launch_block_gemm_tiles<Bg64x256, false, true>(a, stream);
            else launch_block_gemm_tiles<Bg64x256, false>(a, stream);
            return;
    }
}

}  // namespace moe
