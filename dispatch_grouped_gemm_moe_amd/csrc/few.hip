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
// every weight fragment and an expert's rows are padded to 16, 32 or 64 only.
//
// Three launches: the router (logits, top-k, expert row lists), the gate|up
// product with SwiGLU, and the down product with the weighted sum; past 16
// tokens the weighted sum has a launch of its own.  One MXFP8 token of H 7168, I
// 2048, 8 of 32 experts takes 77 us (363 MB of weights: 4.7 TB/s over the call,
// 5.5 over the gate|up product's 44 us), 64 bf16 tokens of the same sizes 537 us
// (2.82 GB, 5.3 TB/s).
//
// Two other forms of the products were built and measured on that one token,
// then 85 us: all three in one launch with tiles handed out by a ticket, down
// tiles waiting on counters, took 159 us (the ticket and the counters shared a
// cache line, on which atomics complete one per 30 ns; with a line each, as the
// counters have now, it was not built again); workgroups that stay and ask for
// their next tile's weights before they reduce the present one, 82 us, and 343
// us against 301 us for 16 tokens with the shared expert, by register spills.
#include "common.hpp"
#include "kernels.hpp"
#include "mxfp8.hpp"

namespace moe {

#pragma clang fp contract(off)

// ---------------------------------------------------------------------------
// Router
// ---------------------------------------------------------------------------

constexpr int kFrEC = 32;         // experts per workgroup: a cache line of a router weight row
constexpr int kFrTok = 4;         // tokens per workgroup, a wave each
constexpr int kFrRes = 16;        // residue groups: group l takes h mod 64 in {l, l + 16, l + 32, l + 48}
constexpr int kFrSlab = 128;      // 64-wide chunks of h per LDS slab

template <int kCtrl>
__device__ __forceinline__ uint32_t dpp_max(uint32_t v) {
    return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, kCtrl, 0xF, 0xF, true));
}

// Largest value of the wave, uniform.
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
    v = dpp_max<0x111>(v);  // row_shr:1, 2, 4, 8: lane 15 of a row has the row's
    v = dpp_max<0x112>(v);
    v = dpp_max<0x114>(v);
    v = dpp_max<0x118>(v);
    v = dpp_max<0x142>(v);  // row_bcast:15, 31: lane 63 has the wave's
    v = dpp_max<0x143>(v);
    return (uint32_t)__builtin_amdgcn_readlane((int)v, kWave - 1);
}

__device__ __forceinline__ int agent_load(const int* p) {
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void agent_store(int* p, int v) {
    __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Whether this workgroup is the last of n to count in; what the others stored
// with agent_store before is then readable with agent_load (both go past the
// XCD's cache, so no cache is written back or dropped).  The last one leaves
// the counter at zero for the next call.
__device__ __forceinline__ bool counts_in_last(int* counter, int n, int* s_flag) {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // this wave's stores have reached memory
    __syncthreads();
    if (threadIdx.x == 0) {
        const int before = __hip_atomic_fetch_add(counter, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        if (before == n - 1) agent_store(counter, 0);
        *s_flag = before == n - 1;
    }
    __syncthreads();
    const bool last = *s_flag != 0;
    __syncthreads();
    return last;
}

// Top-k of one token by one wave: its selections and their softmax weights,
// selection j in lane j.  A lane holds kQ experts, best first, as keys that order
// as the logits do (-0 as +0, NaN as -inf; 0 is below all: none, or chosen), so a
// selection is one maximum over the lanes' first keys.  16 of 256 experts take
// 3.0 us, 8 of 32 1.7; searching all of a lane's logits for every selection took
// 4.8 and 2.8.
template <int kQ>
__device__ __forceinline__ void few_topk(const float* logits, int E, int k, int lane, int& sel, float& weight) {
    uint32_t key[kQ];
    int idx[kQ];
#pragma unroll
    for (int q = 0; q < kQ; ++q) {
        const int e = lane + q * kWave;
        key[q] = 0;
        idx[q] = e;
        if (e < E) {
            const float z = logits[e] + 0.0f;
            const int b = __builtin_bit_cast(int, z == z ? z : -INFINITY);
            key[q] = (uint32_t)b ^ ((uint32_t)(b >> 31) | 0x80000000u);
        }
    }
    // neighbours change places only where that is strictly better: among equal keys the lower expert stays first
#pragma unroll
    for (int n = kQ - 1; n >= 1; --n)
#pragma unroll
        for (int q = 0; q < n; ++q) {
            const bool swap = key[q + 1] > key[q];
            const uint32_t hi = swap ? key[q + 1] : key[q], lo = swap ? key[q] : key[q + 1];
            const int ih = swap ? idx[q + 1] : idx[q], il = swap ? idx[q] : idx[q + 1];
            key[q] = hi, key[q + 1] = lo, idx[q] = ih, idx[q + 1] = il;
        }
    int mine = 0;
    uint32_t mkey = 0, first = 0;
    for (int j = 0; j < k; ++j) {  // k <= E: there is always a key
        const uint32_t m = wave_max(key[0]);
        uint64_t at = __ballot(key[0] == m);
        int from = __builtin_ctzll(at), best = __builtin_amdgcn_readlane(idx[0], from);
        while ((at &= at - 1) != 0) {  // equal logits: the lowest expert
            const int l = __builtin_ctzll(at), e = __builtin_amdgcn_readlane(idx[0], l);
            if (e < best) best = e, from = l;
        }
        if (lane == from) {
#pragma unroll
            for (int q = 0; q + 1 < kQ; ++q) key[q] = key[q + 1], idx[q] = idx[q + 1];
            key[kQ - 1] = 0;
        }
        if (j == 0) first = m;
        if (lane == j) mine = best, mkey = m;
    }
    auto value = [](uint32_t b) { return __builtin_bit_cast(float, (int)b < 0 ? b ^ 0x80000000u : ~b); };
    const float z = expf(value(mkey) - value(first));
    float den = 0.0f;  // summed in slot order
    for (int j = 0; j < k; ++j)
        den = den + __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, z), j));
    sel = mine;
    weight = z / den;
}

// LDS of the row lists.
struct FewLists {
    uint64_t mask[kMaxExperts];  // tokens of each expert
    int off[kMaxExperts];        // its first row
    int wave_rows[kMaxExperts / kWave], wave_act[kMaxExperts / kWave];
    int sel_e[kFewTokens * kMaxTopK];  // every token's selections
    float sel_w[kFewTokens * kMaxTopK];
};

// The experts' row lists.  At most 64 tokens: an expert's tokens are one 64-bit
// mask, and a row's rank within its expert a population count.
template <int kThreads>
__device__ __forceinline__ void few_lists(const FewRoute& a, FewLists& s) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int n = a.T * a.k;
    static_assert(kMaxExperts <= kThreads && kThreads % kWave == 0, "an expert per thread");
    if (tid < kMaxExperts) s.mask[tid] = 0;
    __syncthreads();
    for (int i = tid; i < n; i += kThreads) atomicOr((unsigned long long*)&s.mask[s.sel_e[i]], 1ull << (i / a.k));
    __syncthreads();
    // exclusive prefixes over the experts, of rows and of experts that have any
    int c = 0, inc = 0;
    uint64_t on = 0;
    if (tid < kMaxExperts) {
        c = __popcll(s.mask[tid]);
        inc = c;
#pragma unroll
        for (int d = 1; d < kWave; d <<= 1) {
            const int o = __shfl_up(inc, d, kWave);
            if (lane >= d) inc += o;
        }
        on = __ballot(c > 0);
        if (lane == kWave - 1) {
            s.wave_rows[wave] = inc;
            s.wave_act[wave] = __popcll(on);
        }
    }
    __syncthreads();
    int rows = 0, act = 0;
    for (int w = 0; w < kMaxExperts / kWave; ++w) {
        if (w == wave && tid < kMaxExperts) {
            const int off = rows + inc - c;
            s.off[tid] = off;
            if (c > 0) {
                const int at = act + __popcll(on & ((1ull << lane) - 1ull));
                a.act_e[at] = tid;
                a.act_off[at] = off;
            }
        }
        rows += s.wave_rows[w];
        act += s.wave_act[w];
    }
    if (tid == 0) {
        if (a.shared) {  // the shared expert takes every token, after the routed rows
            a.act_e[act] = a.E;
            a.act_off[act] = rows;
            ++act;
            rows += a.T;
        }
        a.act_off[act] = rows;
        *a.n_act = act;
    }
    __syncthreads();
    for (int i = tid; i < n; i += kThreads) {
        const int t = i / a.k, e = s.sel_e[i];
        const int row = s.off[e] + __popcll(s.mask[e] & ((1ull << t) - 1ull));
        a.row_token[row] = t;
        a.row_w[row] = s.sel_w[i];
        a.slot_row[i] = row;
    }
    if (a.shared && tid < a.T) {
        a.row_token[n + tid] = tid;
        a.row_w[n + tid] = 1.0f;
    }
}

// Workgroup (l, x, y): residues l, l + 16, l + 32, l + 48 of h mod 64, experts
// 32 x .. 32 x + 31, tokens 4 y .. 4 y + 3, a wave per token.  (Eight tokens a
// workgroup gather more of x's lines in one: 16 tokens of H 7168 16.1 against 13.4
// us; 5 tokens over 64 experts, one count less, 9.9 against 10.5.)
//
// The logits' order is moe_route's: p[r] sums h = r, r + 64, ... with fused
// multiply-adds, a halving tree joins the 64 p[r], the bias comes last.  The
// sums over h are chains, but the 64 residues are independent, so they are what
// is spread over workgroups: each asks for its rows of the router weight (whole
// cache lines) and its tokens' values at once and waits for memory once.  What
// this costs is latency and cache lines per workgroup (about 350 lines a
// microsecond), not bytes.  Splitting the experts alone instead (every
// workgroup all of h, 16 bytes of each line) took 26 us for one token of H 7168
// and 32 experts, and 27 us for 64 tokens.
//
// A lane holds expert lane % 32; its half of the wave residues l + 16 half and
// l + 16 half + 32: the first two tree levels stay in the wave.  The workgroup
// of a y that counts in last joins the 16 groups' sums to logits and picks its
// tokens' experts, the last y builds the row lists.  With more than a logit per
// thread to join, the last of an (x, y) joins, the last of a y picks: one count
// more (one token, 64 experts: 9.1 against 7.9 us).
template <bool kVec4>
__global__ __launch_bounds__(kFrTok * kWave) void few_route_kernel(FewRoute a) {
    constexpr int kTok = kFrTok, kThreads = kTok * kWave;
    __shared__ __attribute__((aligned(1024))) float s_wr[kFrSlab * 4][kFrEC];
    __shared__ __attribute__((aligned(16))) float s_x[kTok][2][kFrSlab][2];
    __shared__ float s_logit[kTok][kMaxExperts];
    __shared__ int s_flag;
    static_assert(sizeof(FewLists) <= sizeof(s_wr), "the lists take the slab's place");
    FewLists& s_lists = *(FewLists*)&s_wr[0][0];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int l = blockIdx.x, e0 = blockIdx.y * kFrEC, t0 = blockIdx.z * kTok;
    const int ng = gridDim.y, nz = gridDim.z;
    const int T = a.T, H = a.H, E = a.E, k = a.k;
    const int nt = min(kTok, T - t0), ne = min(kFrEC, E - e0);
    const int half = lane >> 5, el = lane & 31;
    float p0 = 0.0f, p1 = 0.0f;
    for (int c0 = 0; c0 < H / kWave; c0 += kFrSlab) {
        const int nc = min(kFrSlab, H / kWave - c0);
        if (c0) __syncthreads();  // the previous slab is summed
        // LDS row 4 c + j: h = 64 (c0 + c) + l + 16 j
        auto h_of = [&](int r) { return (c0 + (r >> 2)) * kWave + l + 16 * (r & 3); };
        // (the columns past the last expert hold anything: nobody reads their sums)
        if (kVec4) {
            // eight rows per load; a slab's rows are a multiple of four
            if ((lane & 7) * 4 < ne)
                for (int r = wave * 8; r < nc * 4; r += kTok * 8)
                    __builtin_amdgcn_global_load_lds(
                        (gbl_cvoid*)(a.Wr + (size_t)h_of(min(r + (lane >> 3), nc * 4 - 1)) * E + e0 + (lane & 7) * 4),
                        (lds_void*)s_wr[r], 16, 0, 0);
        } else {
            // a row per half wave, eight loads of a thread at once
            constexpr int kRows = kThreads / kFrEC;
            const int q = min(el, ne - 1);
            for (int r0 = tid / kFrEC; r0 < nc * 4; r0 += 8 * kRows) {
                float v[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = a.Wr[(size_t)h_of(min(r0 + j * kRows, nc * 4 - 1)) * E + e0 + q];
#pragma unroll
                for (int j = 0; j < 8; ++j) s_wr[min(r0 + j * kRows, nc * 4 - 1)][el] = v[j];
            }
        }
        if (wave < nt) {
            const uint16_t* xr = a.x + (size_t)(t0 + wave) * H + (size_t)c0 * kWave + l;
            uint16_t v[kFrSlab / kWave][4];
#pragma unroll
            for (int i = 0; i < kFrSlab / kWave; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) v[i][j] = xr[(size_t)min(i * kWave + lane, nc - 1) * kWave + 16 * j];
#pragma unroll
            for (int i = 0; i < kFrSlab / kWave; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) s_x[wave][j & 1][i * kWave + lane][j >> 1] = bf16_to_f32(v[i][j]);
        }
        // MXFP8: the tokens' codes and operand-layout scales, a block of 32 per
        // thread, while the slab is on its way
        if (a.xq && c0 == 0) {
            const int nb = H / 32, n = gridDim.x * ng * nz;
            for (int i = ((blockIdx.z * ng + blockIdx.y) * gridDim.x + l) * kThreads + tid; i < T * nb;
                 i += n * kThreads) {
                const int ti = i / nb, b = i - ti * nb;
                const uint8_t sc = mx_quant_block32(a.x + (size_t)ti * H + b * 32, a.xq + (size_t)ti * H + b * 32);
                mx_store_scale_byte(a.xs, T, ti, b, nb, sc);
            }
        }
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // the loads into LDS too
        __syncthreads();
        if (wave < nt) {
            const float* wr = &s_wr[half][el];
#pragma unroll 8
            for (int c = 0; c < nc; ++c) {
                p0 = __builtin_fmaf(s_x[wave][half][c][0], wr[c * 4 * kFrEC], p0);
                p1 = __builtin_fmaf(s_x[wave][half][c][1], wr[(c * 4 + 2) * kFrEC], p1);
            }
        }
    }
    {
        float v = p0 + p1;                 // p[r] + p[r + 32]
        v = v + __shfl_xor(v, 32, kWave);  // + 16
        if (wave < nt && half == 0 && el < ne)
            agent_store((int*)a.partial + ((size_t)(t0 + wave) * E + e0 + el) * kFrRes + l, __builtin_bit_cast(int, v));
    }
    const bool two = ng > 4 || min(kTok, T) * E > kThreads;
    if (two) {
        if (!counts_in_last(a.counter + (1 + kFewTokens / 4 + blockIdx.z * ng + blockIdx.y) * kFewCounterInts, kFrRes,
                            &s_flag))
            return;
    } else if (!counts_in_last(a.counter + (1 + blockIdx.z) * kFewCounterInts, kFrRes * ng, &s_flag)) {
        return;
    }
    const int j0 = two ? e0 : 0, nj = two ? ne : E;  // the experts to join
    for (int i = tid; i < nt * nj; i += kThreads) {
        const int ti = i / nj, ei = i - ti * nj + j0;
        const uint64_t* q = (const uint64_t*)(a.partial + ((size_t)(t0 + ti) * E + ei) * kFrRes);
        float v[kFrRes];
#pragma unroll
        for (int j = 0; j < kFrRes / 2; ++j) {
            const uint64_t two = __hip_atomic_load(q + j, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            v[2 * j] = __builtin_bit_cast(float, (uint32_t)two);
            v[2 * j + 1] = __builtin_bit_cast(float, (uint32_t)(two >> 32));
        }
#pragma unroll
        for (int d = kFrRes / 2; d >= 1; d >>= 1)
#pragma unroll
            for (int j = 0; j < d; ++j) v[j] = v[j] + v[j + d];
        float z = v[0];
        if (a.bias) z = z + a.bias[ei];
        s_logit[ti][ei] = z;
        if (two) agent_store((int*)a.logits + (size_t)(t0 + ti) * E + ei, __builtin_bit_cast(int, z));
    }
    if (two) {
        if (!counts_in_last(a.counter + (1 + blockIdx.z) * kFewCounterInts, ng, &s_flag)) return;
        for (int i = tid; i < nt * E; i += kThreads)
            s_logit[i / E][i % E] = __builtin_bit_cast(float, agent_load((const int*)a.logits + (size_t)t0 * E + i));
    }
    __syncthreads();
    if (wave < nt) {
        int sel;
        float weight;
        if (E <= kWave) few_topk<1>(s_logit[wave], E, k, lane, sel, weight);
        else few_topk<kMaxExperts / kWave>(s_logit[wave], E, k, lane, sel, weight);
        if (lane < k) {
            const int i = (t0 + wave) * k + lane;
            s_lists.sel_e[i] = sel;
            s_lists.sel_w[i] = weight;
            if (nz > 1) {
                agent_store(a.sel_e + i, sel);
                agent_store((int*)a.sel_w + i, __builtin_bit_cast(int, weight));
            }
        }
    }
    if (nz > 1) {
        if (!counts_in_last(a.counter, nz, &s_flag)) return;
        for (int i = tid; i < T * k; i += kThreads) {
            s_lists.sel_e[i] = agent_load(a.sel_e + i);
            s_lists.sel_w[i] = __builtin_bit_cast(float, agent_load((const int*)a.sel_w + i));
        }
    }
    few_lists<kThreads>(a, s_lists);
}

void launch_few_route(const FewRoute& a, hipStream_t stream) {
    const dim3 grid(kFrRes, ceil_div(a.E, kFrEC), ceil_div(a.T, kFrTok)), block(kFrTok * kWave);
    if (a.E % 4 == 0 && ((uintptr_t)a.Wr & 15) == 0)
        hipLaunchKernelGGL(few_route_kernel<true>, grid, block, 0, stream, a);
    else
        hipLaunchKernelGGL(few_route_kernel<false>, grid, block, 0, stream, a);
}

// ---------------------------------------------------------------------------
// Expert products
// ---------------------------------------------------------------------------

// Four waves, whose partial sums meet in LDS once per tile.  Eight a workgroup
// give a wave half the steps for the same start and epilogue: 61.0 against 54.5
// us a call (7 tokens, H 1024, I 512, 16 of 256 experts, MXFP8), 114 against 90
// (24 tokens, H 2048, I 1024, 6 of 64).  Two double the tokens' loads and the
// epilogue of a wave: 557 against 531 us (64 tokens, H 7168, I 2048, 8 of 32).
constexpr int kFgThreads = 256;
constexpr int kFgWaves = kFgThreads / kWave;
constexpr int kFgRows = 64;                 // weight rows per workgroup
constexpr int kFgChunk = 128;               // bytes of a weight row per step: one cache line
constexpr int kFgLd = kFgRows + 4;          // floats of a token's partial sums in LDS

// What a launch's experts are: bf16, MXFP8, or MXFP8 with the bf16 shared expert.
enum FewKind { kFewBf16 = 0, kFewMx = 1, kFewMxShared = 2 };

__device__ __forceinline__ bf16x8 few_half(intx8 v, int j) {
    return __builtin_bit_cast(bf16x8, j == 0 ? __builtin_shufflevector(v, v, 0, 1, 2, 3)
                                             : __builtin_shufflevector(v, v, 4, 5, 6, 7));
}

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

// Fragments of step c of rows up to byte kb: zeros past it, a row's end, which for
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

// The 32 MXFP8 values of a lane as bf16, scaled (exact: four significand bits
// and a power of two), eight to an operand of a 16x16x32 MFMA.  Bytes 0 .. 15
// lie in block (l / 32) of the line, bytes 16 .. 31 in block 2 + l / 32.
__device__ __forceinline__ void few_widen(const intx4 (&v)[2], uint32_t scales, int lane, bf16x8 (&o)[4]) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    const uint32_t s = scales >> (8 * (lane >> 5));
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const float f = __builtin_bit_cast(float, (s >> (16 * j) & 0xff) << 23);  // its exponent is the scale
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            bf16x2 t[4];
#pragma unroll
            for (int d = 0; d < 2; ++d) {
                t[2 * d] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)v[j][2 * q + d], f, false);
                t[2 * d + 1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)v[j][2 * q + d], f, true);
            }
            o[2 * j + q] = bf16x8{t[0][0], t[0][1], t[1][0], t[1][1], t[2][0], t[2][1], t[3][0], t[3][1]};
        }
    }
}

// kWiden: MXFP8 values go through bf16 MFMAs.  A scaled MFMA adds up eight
// neighbouring products on one exponent and cuts off what lies below 2^-13 of the
// largest one's power of two (measured for every place of the 128); beyond the
// eight it is fp32.  Sums of 1664 random products are off by 1.7e-5 of their norm.
// Too coarse for what is quantised again: 16 of 11648 values of h took another
// code, this way none, in the same time.  The down products take scaled MFMAs:
// their operands were rounded to 2^-4 of a value before, their output is to 2^-8,
// and the cut is at most 7 2^-13 of the eight's largest.
//
// kParts: fragments MT .. of x are the second parts of tokens in two bf16 parts.
template <bool MX, int MT, int kParts, bool kWiden>
__device__ __forceinline__ void few_mfma(const FewFrag<MX, 4>& w, const FewFrag<MX, MT * kParts>& x, int lane,
                                         floatx4 (&acc)[4][MT]) {
    if constexpr (MX && kWiden) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            bf16x8 wb[4];
            few_widen(w.v[i], w.s[i], lane, wb);
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                bf16x8 xb[4];
                few_widen(x.v[m], x.s[m], lane, xb);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    acc[i][m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wb[j], xb[j], acc[i][m], 0, 0, 0);
            }
        }
    } else {
        const int shift = 8 * (lane >> 4);
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (MX) {
                    acc[i][m] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                        cat8(w.v[i][0], w.v[i][1]), cat8(x.v[m][0], x.v[m][1]), acc[i][m], 0, 0, 0,
                        (int)(w.s[i] >> shift), 0, (int)(x.s[m] >> shift));
                } else {
#pragma unroll
                    for (int j = 0; j < 2 * kParts; ++j)
                        acc[i][m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                            __builtin_bit_cast(bf16x8, w.v[i][j & 1]),
                            __builtin_bit_cast(bf16x8, x.v[m + MT * (j >> 1)][j & 1]), acc[i][m], 0, 0, 0);
                }
            }
    }
}

// acc[i][m] (+)= weight rows 16 i .. of the tile times token rows 16 m .., over
// the steps c0 + wave, c0 + wave + 4, ... of the rows' kb bytes up to byte `end`.
// The weights of one step are in flight while the step before is multiplied; the tokens, which come
// from the L2, are loaded in their own step, ahead of the next weights, so that
// waiting for them (loads return in order) leaves those in flight.  Steps past
// the end load zeros, so the loop has one exit and keeps its registers.
template <bool MX, int MT, int kParts, bool kWiden>
__device__ __forceinline__ void few_stream(const FewOperand& wo, const FewOperand& xo, int kb, int c0, int end,
                                           int wave, int lane, const uint32_t (&xrow)[MT * kParts],
                                           const uint32_t (&xsoff)[MT * kParts], floatx4 (&acc)[4][MT]) {
    const uint32_t lo = (uint32_t)(lane >> 4) * 16;
    uint32_t woff[4], wsoff[4], xoff[MT * kParts];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        woff[i] = (uint32_t)(i * 16 + (lane & 15)) * (uint32_t)kb + lo;
        wsoff[i] = (uint32_t)(i * 16 + (lane & 15)) * 4;
    }
#pragma unroll
    for (int m = 0; m < MT * kParts; ++m) xoff[m] = xrow[m] + lo;
    FewFrag<MX, 4> w0, w1;
    FewFrag<MX, MT * kParts> x;
    auto step = [&](int c, const FewFrag<MX, 4>& w, FewFrag<MX, 4>& next) {
        few_load<MX, MT * kParts>(xo, end, c, xoff, xsoff, x);
        few_load<MX, 4>(wo, end, c + kFgWaves, woff, wsoff, next);
        __builtin_amdgcn_sched_barrier(0);
        few_mfma<MX, MT, kParts, kWiden>(w, x, lane, acc);
        __builtin_amdgcn_sched_barrier(0);
    };
    few_load<MX, 4>(wo, end, c0 + wave, woff, wsoff, w0);
    for (int c = c0 + wave; c * kFgChunk < end; c += 2 * kFgWaves) {
        step(c, w0, w1);
        step(c + kFgWaves, w1, w0);
    }
}

// v in two bf16 parts of its sign, neither zero unless v is (or next to nothing):
// the first cut off towards zero, and one step smaller still where that would
// leave nothing, so that an infinite weight gives v's infinity in both products.
__device__ __forceinline__ void few_split(float v, uint16_t& hi, uint16_t& lo) {
    const uint32_t b = __builtin_bit_cast(uint32_t, v);
    hi = (uint16_t)(b >> 16);
    if ((b & 0xffff) == 0 && (hi & 0x7fff) != 0 && (hi & 0x7fff) < 0x7f80) --hi;
    lo = f32_to_bf16_rne((hi & 0x7fff) < 0x7f80 ? v - bf16_to_f32(hi) : v);
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
__device__ __forceinline__ void few_gate_up(const FewGemm& a, int e, int n, int row0, int rows, int z, int counter,
                                            float* s_part) {
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
    const int lines = ((int)kb + kFgChunk - 1) / kFgChunk, splits = a.gu_splits;
    const int end = z + 1 == splits ? (int)kb : lines * (z + 1) / splits * kFgChunk;
    few_stream<MX, MT, 1, true>(wo, xo, (int)kb, lines * z / splits, end, wave, lane, xrow, xsrow, acc);
    // thread (tokens tid / 32, + 8; column tid % 32): the tile's rows are 32 gate
    // columns and the 32 up columns of the same indices
    const int col = tid & 31;
    auto finish = [&](int r, float g, float u) {
        const float h = g / (1.0f + expf(-g)) * u;
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
                        for (int s = 1; (n + s) & 3; ++s) d[s] = 0;
                }
            }
        } else if (r < rows) {
            // Two bf16 parts, operands of the next MFMAs: 2^-15 of h is lost.  One part
            // would add an error as large as the output's own rounding (measured
            // against 64 bits, 0.0024 to 0.0028 instead of 0.0017 of the output).  Where
            // an expert has up to eight rows the parts share a fragment and cost next
            // to nothing (one token, H 2048: 0.5 of 28 us; as products of their own,
            // 2); for 64 tokens of H 7168 the down product takes 196 us instead of 182.
            uint16_t hi, lo;
            few_split(h, hi, lo);
            uint16_t* d = a.h + (size_t)(row0 + r) * 2 * I + n * 32 + col;
            d[0] = hi;
            d[I] = lo;
        }
    };
    // the parts' sums of row r: [row][tile of 32 columns][part][64]
    auto part = [&](int r) { return a.gu_part + ((size_t)(row0 + r) * (I / 32) + n) * splits * kFgRows + col; };
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        if (m * 16 >= rows) break;
        __syncthreads();
        few_stage<MT>(acc, m, wave, lane, s_part);
        __syncthreads();
        for (int tt = tid >> 5; tt < 16; tt += kFgThreads / 32) {
            float g = 0.0f, u = 0.0f;
#pragma unroll
            for (int w = 0; w < kFgWaves; ++w) {
                g += s_part[(w * 16 + tt) * kFgLd + col];
                u += s_part[(w * 16 + tt) * kFgLd + 32 + col];
            }
            const int r = m * 16 + tt;
            if (splits == 1) {
                finish(r, g, u);
            } else if (r < rows) {
                int* d = (int*)part(r) + z * kFgRows;
                agent_store(d, __builtin_bit_cast(int, g));
                agent_store(d + 32, __builtin_bit_cast(int, u));
            }
        }
    }
    if (splits == 1 || !counts_in_last(a.tile_count + counter * kFewCounterInts, splits, (int*)s_part)) return;
    for (int r = tid >> 5; r < ((rows + 1) & ~1); r += kFgThreads / 32) {  // whole waves
        const int* q = (const int*)part(min(r, rows - 1));
        float g = 0.0f, u = 0.0f;
        for (int s = 0; s < splits; ++s) {
            g += __builtin_bit_cast(float, agent_load(q + s * kFgRows));
            u += __builtin_bit_cast(float, agent_load(q + s * kFgRows + 32));
        }
        finish(r, g, u);
    }
}

// kPairs: up to eight rows whose two bf16 parts are rows of their own, 2 r and 2 r
// + 1 (as they lie in memory): both products in one 16-wide fragment.
template <bool MX, int MT, bool kPairs>
__device__ __forceinline__ void few_down(const FewGemm& a, int e, int n, int row0, int rows, float* s_part) {
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int H = a.H, I = a.I;
    const uint32_t kb = (uint32_t)I * (MX ? 1 : 2);
    FewOperand wo{}, xo{};
    wo.bytes = kFgRows * kb;
    constexpr int kParts = MX || kPairs ? 1 : 2;  // of a token in fragments of their own
    xo.bytes = (uint32_t)rows * kb * (MX ? 1 : 2);
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
        xo.data = a.h + (int64_t)row0 * 2 * I;
    }
    uint32_t xrow[MT * kParts], xsrow[MT * kParts];
#pragma unroll
    for (int m = 0; m < MT * kParts; ++m) {
        const uint32_t r = (uint32_t)min(m % MT * 16 + (lane & 15), (kPairs ? 2 * rows : rows) - 1);
        xrow[m] = (r * kParts + m / MT) * kb;
        xsrow[m] = r * (uint32_t)mx_groups(I) * 4;
    }
    floatx4 acc[4][MT];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int m = 0; m < MT; ++m) acc[i][m] = floatx4{0, 0, 0, 0};
    few_stream<MX, MT, kParts, false>(wo, xo, (int)kb, 0, (int)kb, wave, lane, xrow, xsrow, acc);
    const int col = (tid & 31) * 2;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        if (m * 16 >= rows) break;
        __syncthreads();
        few_stage<MT>(acc, m, wave, lane, s_part);
        __syncthreads();
        for (int tt = tid >> 5; tt < 16; tt += kFgThreads / 32) {
            float y0 = 0.0f, y1 = 0.0f;
#pragma unroll
            for (int w = 0; w < kFgWaves; ++w) {
                y0 += s_part[(w * 16 + tt) * kFgLd + col];
                y1 += s_part[(w * 16 + tt) * kFgLd + col + 1];
            }
            int r = m * 16 + tt;
            if constexpr (kPairs) {  // the pair's other part: half a wave further on
                y0 += __shfl_xor(y0, 32, kWave);
                y1 += __shfl_xor(y1, 32, kWave);
                r = tt & 1 ? rows : tt >> 1;
            }
            if (r < rows) {
                const float wt = a.row_w[row0 + r];
                float* d = a.y + (size_t)(row0 + r) * H + n * kFgRows + col;
                d[0] = wt * y0;
                d[1] = wt * y1;
            }
        }
    }
}

template <bool kDown, bool MX, int MT>
__device__ __forceinline__ void few_tile(const FewGemm& a, int e, int n, int row0, int rows, int z, int counter,
                                         float* s_part) {
    if constexpr (kDown) few_down<MX, MT, false>(a, e, n, row0, rows, s_part);
    else few_gate_up<MX, MT>(a, e, n, row0, rows, z, counter, s_part);
}

// The tile's code by the 16-row fragments that the expert's rows fill (three
// run as four, the rows past the last repeating it).
template <bool kDown, bool MX, int kMost>
__device__ __forceinline__ void few_tile_rows(const FewGemm& a, int e, int n, int row0, int rows, int z, int counter,
                                              float* s_part) {
    if (kDown && !MX && rows <= 8) few_down<MX, 1, true>(a, e, n, row0, rows, s_part);
    else if (kMost == 1 || rows <= 16) few_tile<kDown, MX, 1>(a, e, n, row0, rows, z, counter, s_part);
    else if (kMost == 2 || rows <= 32) few_tile<kDown, MX, 2>(a, e, n, row0, rows, z, counter, s_part);
    else few_tile<kDown, MX, 4>(a, e, n, row0, rows, z, counter, s_part);
}

// Workgroup b: active expert b / n_tiles, weight rows 64 (b % n_tiles) .. + 63.
// The host sizes the grid for every expert that T * k choices can reach; the
// workgroups past the active ones end at once.  kMost: 16-row fragments of T.  The
// bound on waves keeps the compiler from spreading over accumulation registers,
// which would halve the waves per SIMD past 16 tokens.
template <bool kDown, bool kMx, int kMost>
__global__ __launch_bounds__(kFgThreads, kMost == 1 ? 1 : (kMost == 4 ? 2 : (kMx || kDown ? 3 : 4))) void few_gemm_kernel(
    FewGemm a) {
    __shared__ __attribute__((aligned(16))) float s_part[kFgWaves * 16 * kFgLd];
    const int nt = kDown ? a.H / kFgRows : a.I / 32;
    const int t = kDown ? blockIdx.x : blockIdx.x / a.gu_splits, z = kDown ? 0 : blockIdx.x - t * a.gu_splits;
    const int i = t / nt, n = t - i * nt;
    // the lists hold an entry for every expert of the grid
    const int n_act = ld_layout(a.n_act), e = ld_layout(a.act_e + i), row0 = ld_layout(a.act_off + i);
    const int rows = ld_layout(a.act_off + i + 1) - row0;
    if (i >= n_act) return;
    if (kMx && e < a.E) few_tile_rows<kDown, true, kMost>(a, e, n, row0, rows, z, t, s_part);
    else few_tile_rows<kDown, false, kMost>(a, e, n, row0, rows, z, t, s_part);
}

template <bool kDown>
static void launch_few_gemm(const FewGemm& a, int max_act, hipStream_t stream) {
    const dim3 grid((unsigned)max_act * (unsigned)(kDown ? a.H / kFgRows : a.I / 32 * a.gu_splits)), block(kFgThreads);
    const int mt = ceil_div(a.T, 16);  // an expert has at most T rows
#define FEW_LAUNCH(MX, MT) hipLaunchKernelGGL((few_gemm_kernel<kDown, MX, MT>), grid, block, 0, stream, a)
    if (mt > 2) {
        if (a.xq) FEW_LAUNCH(true, 4);
        else FEW_LAUNCH(false, 4);
    } else if (kDown || mt == 2) {  // the down product of up to 16 tokens is few_down16_kernel's
        if (a.xq) FEW_LAUNCH(true, 2);
        else FEW_LAUNCH(false, 2);
    } else if constexpr (!kDown) {
        if (a.xq) FEW_LAUNCH(true, 1);
        else FEW_LAUNCH(false, 1);
    }
#undef FEW_LAUNCH
}

int few_gate_up_splits(int64_t tiles, int row_bytes) {
    // As many workgroups as CUs, each wave with about three steps at least: a wave
    // that is alone on its SIMD takes 1.2 us a step.  16 tiles over bf16 rows of H
    // 6784: 29.4 us whole, 10.4 us in eight; 6 over MXFP8 rows of H 6400: 17.3 and
    // 9.7 us in four; 12 over MXFP8 rows of H 2944 stay whole (9.7 us, of which
    // the join would be 3 again).
    const int64_t by_cus = 256 / tiles, by_work = row_bytes / (3 * kFgWaves * kFgChunk);
    const int64_t z = by_work < by_cus ? by_work : by_cus;
    return z < 1 ? 1 : (z > kFewMaxSplits ? kFewMaxSplits : (int)z);
}

void launch_few_gate_up(const FewGemm& a, int max_act, hipStream_t s) { launch_few_gemm<false>(a, max_act, s); }
void launch_few_down(const FewGemm& a, int max_act, hipStream_t s) { launch_few_gemm<true>(a, max_act, s); }

// ---------------------------------------------------------------------------
// Down product and weighted sum of up to 16 tokens
// ---------------------------------------------------------------------------

constexpr int kFdTok = 16;    // tokens
constexpr int kFdCols = 16;   // output columns per workgroup: weight rows of a step
constexpr int kFdBatch = 4;   // cache lines of a row per step
constexpr int kFdSlot = kFdBatch * kFdCols * kFgChunk;  // 8 KB of weights per step
constexpr int kFdRows = kFdTok * (kMaxTopK + 1);

// A value every lane holds alike, as the scalar that it is: a descriptor that
// the compiler keeps in vector registers makes a loop of every load.
__device__ __forceinline__ uint32_t scalar(uint32_t v) { return (uint32_t)__builtin_amdgcn_readfirstlane((int)v); }
__device__ __forceinline__ const void* scalar(const void* p) {
    const uint64_t v = (uint64_t)p;
    return (const void*)((uint64_t)scalar((uint32_t)v) | (uint64_t)scalar((uint32_t)(v >> 32)) << 32);
}

// A part of an expert's product with 16 output columns, taken by one wave.
struct FewUnit {
    const void *w, *x;        // weight rows, the expert's token rows
    const void *ws, *xs;      // MXFP8: their scales
    uint32_t ws_bytes, xs_bytes;
    int row0, rows;           // token rows
    int kb, end;              // bytes of a row, last line of the part + 1
    int mx;
    bool pairs;               // bf16 rows few enough that their two parts are rows of one fragment
};

// Output columns 16 n .. 16 n + 15 of every token, over all active experts: the
// workgroup's waves deal the (expert, part of the row) units among them, each
// runs through its units without a pause (a unit's first weights are asked for
// while the one before is multiplied) and adds the weighted results up per
// token in LDS; one barrier, and the waves' sums are added in order.  Nothing
// goes through memory, and there is no launch for the weighted sum.
//
// There are H / 16 workgroups, fewer than CUs in a small layer, so what one CU
// can draw from memory counts.  Loads of 16 rows x 64 bytes in the MFMA's lane
// order reach 36 GB/s a CU, 8 rows x one line straight into LDS 50 GB/s; the
// fragments are then read from LDS, the 16-byte pieces of a row swizzled by
// its index so that 16 rows fall on distinct banks.  H 7168, I 2048: 25.1 us for
// one MXFP8 token (8 experts, 121 MB, 4.8 TB/s), 171 us for 16 bf16 ones (939 MB,
// 5.5 TB/s).
//
// The two bf16 parts of an expert's h lie as rows 2 r and 2 r + 1: up to eight
// rows are one fragment, whose neighbouring columns are added at the end; past
// that the second parts are loaded and multiplied on their own.
template <int kKind, int kFdWaves>
__global__ __launch_bounds__(kFdWaves * kWave) void few_down16_kernel(FewGemm a, int max_act, int max_rows,
                                                                      uint16_t* out) {
    constexpr int kFdThreads = kFdWaves * kWave;
    __shared__ int s_flag;
    constexpr bool kMx = kKind != kFewBf16;
    __shared__ __attribute__((aligned(1024))) uint8_t s_w[kFdWaves][2][kFdSlot];
    __shared__ __attribute__((aligned(16))) float s_sum[kFdWaves][kFdTok][kFdCols];
    __shared__ int s_token[kFdRows], s_e[kMaxExperts + 1], s_off[kMaxExperts + 2];
    __shared__ float s_weight[kFdRows];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int n = blockIdx.x, splits = gridDim.y, H = a.H, I = a.I;
    // the tables, up to what T and k allow: all asked for at once
    const int n_act = ld_layout(a.n_act);
    for (int i = tid; i < max_rows; i += kFdThreads) {
        s_token[i] = a.row_token[i];
        s_weight[i] = a.row_w[i];
    }
    for (int i = tid; i <= max_act; i += kFdThreads) s_off[i] = a.act_off[i];
    for (int i = tid; i < max_act; i += kFdThreads) s_e[i] = a.act_e[i];
    for (int i = tid; i < kFdWaves * kFdTok * kFdCols; i += kFdThreads) (&s_sum[0][0][0])[i] = 0.0f;
    // parts per expert (2^log_parts): as few as spread the units evenly enough (to a tenth)
    const int lines = (I * (kMx ? 1 : 2) + kFgChunk - 1) / kFgChunk, batches = (lines + kFdBatch - 1) / kFdBatch;
    const int stride = kFdWaves * splits;
    int log_parts = 0;
    while ((2 << log_parts) <= batches &&
           10 * ceil_div(n_act << log_parts, stride) * stride > 11 * (n_act << log_parts))
        ++log_parts;
    const int units = n_act << log_parts;
    __syncthreads();

    // unit u and its first line; past the last one, the first again with no lines
    auto unit_of = [&](int u, int& c0) {
        FewUnit t;
        const int live = (u - units) >> 31;
        u &= live;
        const int i = u >> log_parts, part = u - (i << log_parts);
        const int e = (int)scalar((uint32_t)s_e[i]);
        t.row0 = (int)scalar((uint32_t)s_off[i]);
        t.rows = (int)scalar((uint32_t)s_off[i + 1]) - t.row0;
        t.mx = kKind == kFewMx || (kKind == kFewMxShared && e < a.E) ? 1 : 0;
        t.kb = t.mx ? I : 2 * I;
        t.pairs = kKind != kFewMx && !t.mx && t.rows <= kFdTok / 2;
        const int ln = (t.kb + kFgChunk - 1) / kFgChunk, bt = (ln + kFdBatch - 1) / kFdBatch;
        c0 = (bt * part >> log_parts) * kFdBatch;
        t.end = min((bt * (part + 1) >> log_parts) * kFdBatch, ln);
        if (!live) t.end = c0;
        const int64_t wrow = (int64_t)e * H + (int64_t)n * kFdCols;
        const uint32_t groups = (uint32_t)mx_groups(I);
        t.w = scalar((t.mx ? a.w2q : (const uint8_t*)a.w2) + wrow * t.kb);
        t.x = scalar(t.mx ? a.hq + (int64_t)t.row0 * I : (const uint8_t*)(a.h + (int64_t)t.row0 * 2 * I));
        if (kMx) {
            t.ws = scalar(a.s2 + ((int64_t)e * groups * H + (int64_t)n * kFdCols) * 4);
            t.ws_bytes = scalar(t.mx ? (groups - 1) * (uint32_t)H * 4 + kFdCols * 4 : 0);
            t.xs = scalar(a.hs + (int64_t)t.row0 * groups * 4);
            t.xs_bytes = scalar(t.mx ? (uint32_t)t.rows * groups * 4 : 0);
        }
        t.kb = (int)scalar((uint32_t)t.kb);
        t.end = (int)scalar((uint32_t)t.end);
        c0 = (int)scalar((uint32_t)c0);
        return t;
    };

    const uint32_t lo = (uint32_t)(lane >> 4) * 16, lr = (uint32_t)lane & 15;
    const int shift = 8 * (lane >> 4);
    struct Scales { uint32_t s[kMx ? kFdBatch : 1]; };
    // Ask for the weights of step (t, c) into the slot, load q taking rows 8 (q %
    // 2) .. + 7 of line c + q / 2.  Past the part's end its last line is repeated
    // (and dropped); past the end of an MXFP8 row, in the middle of a line,
    // its first half (against zero scale bytes).  And for the scale dwords; a bf16
    // unit has none: no bytes, at scalar offset 0 (it counts against the size).
    auto issue = [&](const FewUnit& t, int c, int slot, Scales& f) {
        uint8_t* dst = s_w[wave][slot];
        const int last = max(t.end - 1, 0);
#pragma unroll
        for (int q = 0; q < 2 * kFdBatch; ++q) {
            const int line = min(c + q / 2, last);
            const uint32_t row = (uint32_t)(q & 1) * 8 + (uint32_t)(lane >> 3);
            const uint32_t half = kMx && line * kFgChunk + kFgChunk / 2 >= t.kb ? 3 : 7;
            const uint32_t piece = (((uint32_t)lane & 7) ^ (row & 7)) & half;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(few_rsrc(t.w, (uint32_t)(kFdCols * t.kb)), (lds_void*)(dst + q * 1024),
                                                     16, row * (uint32_t)t.kb + piece * 16, line * kFgChunk, 0, 0);
        }
        if constexpr (kMx) {
#pragma unroll
            for (int j = 0; j < kFdBatch; ++j)
                f.s[j] = __builtin_amdgcn_raw_buffer_load_b32(few_rsrc(t.ws, t.ws_bytes), lr * 4,
                                                              t.mx ? min(c + j, last) * H * 4 : 0, 0);
        }
    };
    // The weight fragments of a slot: of line j this lane's pieces lane / 16 and
    // 4 + lane / 16 of row lane % 16.  In one block with its wait: the compiler
    // would wait for the loads into the other slot too.
    static_assert(kFdBatch == 4 && kFdCols * kFgChunk == 2048, "the offsets below");
    auto frags = [&](int slot, intx8 (&w)[kFdBatch]) {
        const uint32_t g = (uint32_t)lane >> 4, sw = lr & 7;
        const uint32_t row = (uint32_t)(uintptr_t)(lds_void*)s_w[wave][slot] + lr * kFgChunk;
        const uint32_t p0 = row + (g ^ sw) * 16, p1 = row + ((4 + g) ^ sw) * 16;
        intx4 f[2 * kFdBatch];
        asm volatile(
            "ds_read_b128 %0, %8\n\tds_read_b128 %1, %9\n\t"
            "ds_read_b128 %2, %8 offset:2048\n\tds_read_b128 %3, %9 offset:2048\n\t"
            "ds_read_b128 %4, %8 offset:4096\n\tds_read_b128 %5, %9 offset:4096\n\t"
            "ds_read_b128 %6, %8 offset:6144\n\tds_read_b128 %7, %9 offset:6144\n\t"
            "s_waitcnt lgkmcnt(0)"
            : "=&v"(f[0]), "=&v"(f[1]), "=&v"(f[2]), "=&v"(f[3]), "=&v"(f[4]), "=&v"(f[5]), "=&v"(f[6]), "=&v"(f[7])
            : "v"(p0), "v"(p1)
            : "memory");
#pragma unroll
        for (int j = 0; j < kFdBatch; ++j) w[j] = __builtin_shufflevector(f[2 * j], f[2 * j + 1], 0, 1, 2, 3, 4, 5, 6, 7);
    };
    floatx4 acc = {0, 0, 0, 0};
    int u = blockIdx.y * kFdWaves + wave, c;
    FewUnit t = unit_of(u, c);
    Scales f0, f1;
    issue(t, c, 0, f0);
    auto step = [&](int slot, const Scales& f, Scales& next) {
        const FewUnit cur = t;
        const int c0 = c;
        constexpr int kXl = kKind == kFewMx ? 0 : kFdBatch;
        intx8 x[kFdBatch], xl[kXl + 1];  // xl: the second parts, where they are not rows of their own
        uint32_t xs[kMx ? kFdBatch : 1];
        const uint32_t r = (uint32_t)min((int)lr, (cur.pairs ? 2 * cur.rows : cur.rows) - 1);  // past the last: that again
        const int last = max(cur.end - 1, 0);
        const bool two = kKind != kFewMx && !cur.mx && !cur.pairs;
        const uint32_t xoff = r * (uint32_t)(two ? 2 * cur.kb : cur.kb) + lo;
        const __amdgpu_buffer_rsrc_t d = few_rsrc(cur.x, (uint32_t)(cur.mx ? cur.rows : 2 * cur.rows) * (uint32_t)cur.kb);
#pragma unroll
        for (int j = 0; j < kFdBatch; ++j) {
            const int line = min(c0 + j, last), at = line * kFgChunk;
            const int hi = kMx && at + kFgChunk / 2 >= cur.kb ? at : at + kFgChunk / 2;
            const intx4 p0 = __builtin_amdgcn_raw_buffer_load_b128(d, xoff, at, 0);
            const intx4 p1 = __builtin_amdgcn_raw_buffer_load_b128(d, xoff, hi, 0);
            x[j] = __builtin_shufflevector(p0, p1, 0, 1, 2, 3, 4, 5, 6, 7);
            if constexpr (kMx)
                xs[j] = __builtin_amdgcn_raw_buffer_load_b32(few_rsrc(cur.xs, cur.xs_bytes),
                                                             r * (uint32_t)mx_groups(I) * 4, cur.mx ? line * 4 : 0, 0);
        }
        if (two) {
#pragma unroll
            for (int j = 0; j < kXl; ++j) {
                const int at = min(c0 + j, last) * kFgChunk + cur.kb;
                const intx4 p0 = __builtin_amdgcn_raw_buffer_load_b128(d, xoff, at, 0);
                const intx4 p1 = __builtin_amdgcn_raw_buffer_load_b128(d, xoff, at + kFgChunk / 2, 0);
                xl[j] = __builtin_shufflevector(p0, p1, 0, 1, 2, 3, 4, 5, 6, 7);
            }
        }
        c += kFdBatch;
        const bool flush = c >= cur.end;
        if (flush) {
            u += stride;
            t = unit_of(u, c);
        }
        __builtin_amdgcn_sched_barrier(0);
        issue(t, c, slot ^ 1, next);
        __builtin_amdgcn_sched_barrier(0);
        // everything before the next step's weights has arrived
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"(2 * kFdBatch + (kMx ? kFdBatch : 0)) : "memory");
        intx8 w[kFdBatch];
        frags(slot, w);
        if (c0 + kFdBatch > cur.end) {  // zero times zero past the part's end, whatever the last line holds
#pragma unroll
            for (int j = 0; j < kFdBatch; ++j)
                if (c0 + j >= cur.end) {
                    w[j] = x[j] = intx8{};
                    if constexpr (kKind != kFewMx) xl[j] = intx8{};
                }
        }
        if (two) {
#pragma unroll
            for (int j = 0; j < kXl; ++j) {
                acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(few_half(w[j], 0), few_half(xl[j], 0), acc, 0, 0, 0);
                acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(few_half(w[j], 1), few_half(xl[j], 1), acc, 0, 0, 0);
            }
        }
#pragma unroll
        for (int j = 0; j < kFdBatch; ++j) {
            if (kKind == kFewMx || (kKind == kFewMxShared && cur.mx)) {
                if constexpr (kMx)
                    acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w[j], x[j], acc, 0, 0, 0, (int)(f.s[j] >> shift),
                                                                           0, (int)(xs[j] >> shift));
            } else {
                acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(few_half(w[j], 0), few_half(x[j], 0), acc, 0, 0, 0);
                acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(few_half(w[j], 1), few_half(x[j], 1), acc, 0, 0, 0);
            }
        }
        __builtin_amdgcn_sched_barrier(0);
        if (flush) {  // lane: columns 4 (l / 16) .. + 3 of token row l % 16, or of the part of row l % 16 / 2
            int tr = (int)lr;
            if (kKind != kFewMx && cur.pairs) {
#pragma unroll
                for (int q = 0; q < 4; ++q) {  // + the neighbour's
                    const float v = acc[q];
                    acc[q] = v + __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), 0xB1,
                                                                                    0xF, 0xF, true));
                }
                tr = tr & 1 ? cur.rows : tr >> 1;
            }
            if (tr < cur.rows) {
                floatx4* d = (floatx4*)&s_sum[wave][s_token[cur.row0 + tr]][4 * (lane >> 4)];
                const float wt = s_weight[cur.row0 + tr];
                floatx4 v = *d;
#pragma unroll
                for (int q = 0; q < 4; ++q) v[q] = __builtin_fmaf(wt, acc[q], v[q]);
                *d = v;
            }
            acc = floatx4{0, 0, 0, 0};
        }
    };
    while (u < units) {  // the second step may be past the last unit
        step(0, f0, f1);
        step(1, f1, f0);
    }
    __syncthreads();
    // T x 16 sums, two a thread
    const int tok = tid / (kFdCols / 2), col = tid % (kFdCols / 2) * 2;
    static_assert(kFdTok * kFdCols / 2 <= kFdThreads, "two sums a thread");
    float s0 = 0.0f, s1 = 0.0f;
    if (tok < a.T) {
#pragma unroll
        for (int w = 0; w < kFdWaves; ++w) {
            s0 += s_sum[w][tok][col];
            s1 += s_sum[w][tok][col + 1];
        }
    }
    if (splits > 1) {
        uint64_t* part = (uint64_t*)a.y + ((size_t)n * splits * a.T + tok) * (kFdCols / 2) + col / 2;
        const size_t next = (size_t)a.T * (kFdCols / 2);
        if (tok < a.T)
            __hip_atomic_store(part + blockIdx.y * next,
                               (uint64_t)__builtin_bit_cast(uint32_t, s0) |
                                   (uint64_t)__builtin_bit_cast(uint32_t, s1) << 32,
                               __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        if (!counts_in_last(a.tile_count + n * kFewCounterInts, splits, &s_flag)) return;
        s0 = s1 = 0.0f;
        if (tok < a.T)
            for (int z = 0; z < splits; ++z) {
                const uint64_t two = __hip_atomic_load(part + z * next, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
                s0 += __builtin_bit_cast(float, (uint32_t)two);
                s1 += __builtin_bit_cast(float, (uint32_t)(two >> 32));
            }
    }
    if (tok < a.T)
        *(uint32_t*)(out + (size_t)tok * H + n * kFdCols + col) =
            (uint32_t)f32_to_bf16_rne(s0) | ((uint32_t)f32_to_bf16_rne(s1) << 16);
}

int few_down16_splits(int H, int64_t column_kb) {
    // As many workgroups as CUs, each with about 100 KB to read at least.  64
    // column blocks of 750 KB take 26.4 us whole and 16.8 us in four (7 tokens, H
    // 1024, 16 of 256 experts), 128 of 590 KB 22.7 and 19.8 us in two; 128 of 192
    // KB (9.0 us whole) stay whole: each part reads the row lists anew and the last
    // to finish reads every part's sums.
    const int n = H / kFdCols;
    static_assert(256 / (kFewMaxSplitTiles + 1) < 2, "a counter for every column block that is split");
    const int64_t by_work = column_kb / 100, by_cus = 256 / n;
    const int64_t z = by_work < by_cus ? by_work : by_cus;
    return z < 1 ? 1 : (z > kFewMaxSplits ? kFewMaxSplits : (int)z);
}

void launch_few_down16(const FewGemm& a, int max_act, int max_rows, int shared, int splits, uint16_t* out,
                       hipStream_t stream) {
    const dim3 grid(a.H / kFdCols, splits);
#define FEW_DOWN16(KIND, WAVES)                                                                            \
    hipLaunchKernelGGL((few_down16_kernel<KIND, WAVES>), grid, dim3(WAVES * kWave), 0, stream, a, max_act, \
                       max_rows, out)
    // With more column blocks than CUs, two workgroups of four waves fit a CU and
    // even its load out: one token of H 7168, MXFP8, 27.7 -> 25.1 us, H 4608 and I
    // 512 11.1 -> 7.2 us.  With fewer, eight waves ask for more at once: H 3584, I
    // 2048, 8 experts 12.0 us against 13.6 us in four waves and twice the parts.
    if (a.H / kFdCols > 256) {
        if (!a.xq) FEW_DOWN16(kFewBf16, 4);
        else if (!shared) FEW_DOWN16(kFewMx, 4);
        else FEW_DOWN16(kFewMxShared, 4);
    } else {
        if (!a.xq) FEW_DOWN16(kFewBf16, 8);
        else if (!shared) FEW_DOWN16(kFewMx, 8);
        else FEW_DOWN16(kFewMxShared, 8);
    }
#undef FEW_DOWN16
}

// out[t] = the weighted rows of the slots in order, then the shared expert's.
__global__ __launch_bounds__(256) void few_combine_kernel(FewGemm a, int k, int shared, uint16_t* out) {
    const int col = (blockIdx.x * 256 + threadIdx.x) * 2, t = blockIdx.y;
    if (col >= a.H) return;
    float s0 = 0.0f, s1 = 0.0f;
    for (int j0 = 0; j0 < k; j0 += 8) {
        uint64_t two[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int row = ld_layout(a.slot_row + t * k + min(j0 + j, k - 1));
            two[j] = *(const uint64_t*)(a.y + (size_t)row * a.H + col);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j0 + j < k) {
                s0 += __builtin_bit_cast(float, (uint32_t)two[j]);
                s1 += __builtin_bit_cast(float, (uint32_t)(two[j] >> 32));
            }
    }
    if (shared) {
        const uint64_t two = *(const uint64_t*)(a.y + (size_t)(a.T * k + t) * a.H + col);
        s0 += __builtin_bit_cast(float, (uint32_t)two);
        s1 += __builtin_bit_cast(float, (uint32_t)(two >> 32));
    }
    *(uint32_t*)(out + (size_t)t * a.H + col) = (uint32_t)f32_to_bf16_rne(s0) | ((uint32_t)f32_to_bf16_rne(s1) << 16);
}

void launch_few_combine(const FewGemm& a, int k, int shared, uint16_t* out, hipStream_t stream) {
    hipLaunchKernelGGL(few_combine_kernel, dim3(ceil_div(a.H, 512), a.T), dim3(256), 0, stream, a, k, shared, out);
}

}  // namespace moe
