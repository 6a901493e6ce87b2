// Softmax cross entropy of an output layer whose vocabulary is split over R ranks, and
// its gradients, without the logits in memory.
//
// With z = h W^T (W: the ranks' weights W_r [Vs, K], one below the other), target t_i:
//   lse_i  = log sum_v exp z_iv                    loss_i = lse_i - z_{i, t_i}
//   d_iv   = dloss_i * (exp(z_iv - lse_i) - [v = t_i])
//   dh     = d W                                   dW_r = d_r^T h
//
// Four products on the tensor cores, which are what bounds it (2 M V K operations
// forward, three times that backward, the logits being formed a second time, and five
// times with d in two parts):
//   kLogSum   z, whose epilogue leaves the maximum of 64 or 128 columns of a row and the
//             sum of exp(z - maximum): 8 bytes for what would be 256 and more.  A small
//             kernel joins the tiles' pairs; pieces of the vocabulary as large as the
//             buffer holds pairs for.
//   kDLogits  z again, whose epilogue leaves d for one piece of the vocabulary, in two bf16 parts;
//   kDH       d W, in fp32 sums over the pieces;
//   kDW       d^T h, rounded to bf16 once; the tiles of both in one launch (kGrads), the
//             long ones of kDH first.
// The tensor cores multiply bf16, and d has more bits: bf16(d) and bf16(d - bf16(d)), one behind
// the other along the contraction, are d to 2^-16 of a term.  With the first alone, which a caller
// may choose, dh and dw are as far from 64 bits as two roundings, 2.4e-3, instead of one, 1.7e-3.
// (tf32 has the rate of the two parts and 2^-11.)  Maxima, sums, lse and all sums of products are fp32.
//
// One kernel body for the four, the CTA-pair scheme of the GEMM kernels: 256x256 tiles,
// each CTA staging its 128 rows of A and 128 columns of B by TMA (six stages of 32 KB),
// the leader issuing cta_group::2 products into two accumulators of 256 TMEM columns, so
// the epilogue of one tile runs under the products of the next.  What differs is which
// tensor lies along the contraction: h and W_r in kLogSum and kDLogits and d in kDH do,
// W_r in kDH, d and h in kDW lie across it, which the tensor cores read as it is
// (MN-major operands), so nothing is transposed in memory.  Nothing waits on another
// pair: a grid of any size is right, and it is persistent only for its two accumulators.
// Tiles are taken in groups of rows whose operand stays in L2 while the other one
// streams past (16 rows of tiles: forward 1055 us, 8: 1076).
//
// Measured, 4096 tokens, K = 4096, vocabulary 65536 over 8 ranks: forward 1.07 ms, 2.05 PFLOP/s, in
// a long run 1.25; forward and backward 7.8 to 7.9 ms, 1.67 to 1.7 PFLOP/s of what is multiplied, the
// rate that the power limit leaves a library's product (8.1 to 8.3 ms in a long run; d in one part 5.2 to 5.4).  One
// token, K = 2048, vocabulary 32000: 28.3 us, 4.6 TB/s, of which 7 are the two kernels' starts and
// ends.  77 tokens, K = 1000, vocabulary 11001, both directions: 48 us, the latencies of five kernels (d in one part 43).
#include <cuda_bf16.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <cmath>

#include "rows.cuh"

namespace are {
namespace {

constexpr int kTile = kXentTile;  // rows and columns of a pair's tile
constexpr uint32_t kHalf = 128 * 64 * 2;  // a CTA's part of an operand: 128 rows or columns, 64 of the contraction
constexpr uint32_t kStageBytes = 2 * kHalf;
constexpr uint32_t kBox = 4096;           // an epilogue warp's staging buffer: 32 rows of 128 bytes; two a warp
// Blocks of 64 of the contraction that the tensor cores add up before the logits' sums go on in registers.  Their fp32 sums
// are cut, not rounded, at every step of 16: over the whole of K = 4096 the losses of 4096 tokens were 1.5e-6 off, and the
// loss of one foreseen token at K = 2048, whose logit of 10 came out 4e-5 too small, 1.8e-5.  With rounded sums of parts of
// 512 the 4096 losses are 1.7e-7 off (a product in fp32 3.1e-7), of 1024 3.6e-7, of 256 0.9e-7; reading the accumulators holds
// the products up: 1077, 1070 and 1102 us in a forward pass.  One CTA's tiles, of few tokens, mostly wait for memory: with parts
// of 256 one token's loss is 3.4e-7 off (K = 2048, vocabulary 32000, the mean of 40), of 128 2.1e-7, as a product in fp32 is, of 64
// 1.7e-7, in 27.8, 28.3 and 29.1 us.
constexpr int kPartPair = 8, kPartOne = 2;

template <int PASS, bool PAIR>
struct Shape {
    // four epilogue warps; sixteen for the logits, whose columns are in registers: 64 a thread, and the 128 of one CTA's tile
    static constexpr int kEpi = PASS == kXentGrads || !PAIR ? 4 : 16;
    static constexpr int kThreads = 128 + 32 * kEpi;  // and a TMA producer, an MMA issuer, a TMEM allocator, an idle warp
    static constexpr int kBoxes = PASS == kXentLogSum ? 0 : PASS == kXentDLogits && PAIR ? 16 : 8;  // staging buffers
    static constexpr int kStages = kBoxes == 16 ? 5 : 6;
    static constexpr int kBars = 2 * kStages + 4 + 1;
    static constexpr size_t kSmem = 1024 + (size_t)kStages * kStageBytes + (size_t)kBoxes * kBox + kBars * 8 + 16;
    static_assert(kSmem <= 232448, "shared memory budget");
};
constexpr float kLog2e = 1.4426950408889634f;

// Instruction descriptor: D fp32, A and B bf16, which of them lie across the contraction, `side` rows and columns.
__device__ __forceinline__ uint32_t idesc(bool a_across, bool b_across, int side) {
    return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)a_across << 15) | ((uint32_t)b_across << 16) |
           ((uint32_t)(side >> 3) << 17) | ((uint32_t)(side >> 4) << 24);
}

// Shared-memory matrix descriptor: 128B swizzle, tcgen05 version bit.
__device__ __forceinline__ uint64_t sdesc(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)((lbo >> 4) & 0x3FFFu) << 16) |
           ((uint64_t)((sbo >> 4) & 0x3FFFu) << 32) | (1ull << 46) | (2ull << 61);
}

// Bounded wait on an mbarrier phase: after a timeout the CTA's roles give up one after the other.
__device__ __noinline__ bool wait_slow(uint64_t* bar, uint32_t parity, volatile uint32_t* abort_flag, const XentParams& p,
                                       int id, int unit) {
    const uint64_t t0 = ptx::globaltimer();
    while (!ptx::mbar_try_wait(bar, parity)) {
        if (*abort_flag) return false;
        if (ptx::globaltimer() - t0 > p.timeout_ns) {
            record_error(p.status, ARE_DEV_PIPE_TIMEOUT, blockIdx.x, id, unit);
            *abort_flag = 1u;
            return false;
        }
    }
    return true;
}
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, volatile uint32_t* abort_flag, const XentParams& p,
                                     int id, int unit) {
    if (ptx::mbar_try_wait(bar, parity)) return true;
    return wait_slow(bar, parity, abort_flag, p, id, unit);
}
// Wait for a copy or product that was issued (it completes by itself), whatever the abort flag says.
__device__ __noinline__ void drain(uint64_t* bar, uint32_t parity, const XentParams& p) {
    const uint64_t t0 = ptx::globaltimer();
    while (!ptx::mbar_try_wait(bar, parity))
        if (ptx::globaltimer() - t0 > p.timeout_ns) break;
}

__device__ __forceinline__ int quotient(int n, const Divisor& d) { return (int)(((uint64_t)(uint32_t)n * d.mul) >> d.shift); }

struct Tile {
    int kind;      // which product: kXentLogSum, kXentDLogits, kXentDH, kXentDW
    int tm, tn, split;
    int kb0, kb1;  // its part of the contraction, in blocks of 64
};

// Order of the tiles: the first grid's, then the second's; in a grid a split's tiles together; inside, groups of p.group
// rows of tiles, column by column.
template <int PASS>
__device__ __forceinline__ Tile tile_of(const XentParams& p, int u) {
    Tile t;
    t.kind = PASS;
    if (PASS == kXentGrads) t.kind = u < p.grid[0].units ? kXentDH : kXentDW;
    const bool second = PASS == kXentGrads && u >= p.grid[0].units;
    const XentGrid& g = p.grid[second ? 1 : 0];
    if (second) u -= p.grid[0].units;
    t.split = quotient(u, g.per_split);
    u -= t.split * (g.tiles_m * g.tiles_n);
    const int n = quotient(u, g.per_group), first = n * p.group, left = g.tiles_m - first;
    const bool whole = left >= p.group;
    u -= n * (p.group * g.tiles_n);
    t.tn = quotient(u, whole ? g.rows : g.last_rows);
    t.tm = first + (u - t.tn * (whole ? p.group : left));
    t.kb0 = quotient(g.num_kb * t.split, g.parts);
    t.kb1 = quotient(g.num_kb * (t.split + 1), g.parts);
    return t;
}

// A vocabulary tile (p.tile columns of one rank) of the piece: the rank, and its first column there.
struct Place {
    int rank, col;
};
__device__ __forceinline__ Place place_of(const XentParams& p, int tile) {
    const int v = p.tile0 + tile, r = quotient(v, p.per_rank);
    return Place{r, (v - r * p.rank_tiles) * p.tile};
}
// Columns of the tile that are in the vocabulary, 0..side.
__device__ __forceinline__ int columns_of(const XentParams& p, const Place& at, int side) {
    const int64_t left = min((int64_t)p.Vs - at.col, p.vocab - ((int64_t)at.rank * p.Vs + at.col));
    return left < 0 ? 0 : left > side ? side : (int)left;
}

__device__ __forceinline__ int64_t target_of(const XentParams& p, int row) {
    const int64_t t = p.wide ? static_cast<const int64_t*>(p.targets)[row] : static_cast<const int32_t*>(p.targets)[row];
    return t >= 0 && t < p.vocab ? t : -1;
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
    __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&v);
}

// 16-byte chunk c of a 128B-swizzled staging row.
__device__ __forceinline__ uint4* chunk_at(uint8_t* base, int row, int c) {
    return reinterpret_cast<uint4*>(base + row * 128 + ((c ^ (row & 7)) << 4));
}

// Two staging buffers a warp (kXentGrads), each free again once the store before the last has read it.
struct Stager {
    uint8_t* base;
    int n;
    __device__ __forceinline__ uint8_t* next() {
        uint8_t* b = base + (n++ & 1) * kBox;
        if ((threadIdx.x & 31) == 0) ptx::bulk_wait_read1();
        __syncwarp();
        return b;
    }
};

// The hidden states with zeros in the rows that have no target: d is 0 there, but 0 times an infinity or a NaN, which padding
// may hold, is none.  dW's product reads the copy in h's place.  kXentDLogits' epilogue warps make it before their first tile,
// under its products (a launch of its own took 10 us of 5 ms at 4096 x 4096, 2 of 40 at 77 x 1000).  Its warps are those of the
// first piece's tiles: for a vocabulary of a few hundred they are few (128 tokens, K = 8192, vocabulary 100: 125 us for all).
__device__ __forceinline__ void copy_rows(const XentParams& p, int warp, int warps) {
    const int lane = threadIdx.x & 31, packs = p.K >> 3;
    for (int64_t row = warp; row < p.M; row += warps) {
        const bool on = target_of(p, (int)row) >= 0;
        const uint4* from = p.rows_from + row * packs;
        uint4* to = p.rows_to + row * packs;
        constexpr int U = 4;  // packs in flight
        for (int i0 = lane; i0 < packs; i0 += 32 * U) {
            uint4 v[U];
#pragma unroll
            for (int j = 0; j < U; ++j) v[j] = on && i0 + 32 * j < packs ? from[i0 + 32 * j] : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
            for (int j = 0; j < U; ++j)
                if (i0 + 32 * j < packs) to[i0 + 32 * j] = v[j];
        }
    }
}

template <int PASS, bool PAIR>
__global__ void __launch_bounds__(Shape<PASS, PAIR>::kThreads, 1) xent_kernel(const __grid_constant__ XentParams p) {
    constexpr int kStages = Shape<PASS, PAIR>::kStages, kEpi = Shape<PASS, PAIR>::kEpi, kPart = PAIR ? kPartPair : kPartOne;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sA = smem;
    uint8_t* sB = sA + kStages * kHalf;
    uint8_t* sOut = sB + kStages * kHalf;
    uint64_t* full = reinterpret_cast<uint64_t*>(sOut + Shape<PASS, PAIR>::kBoxes * kBox);
    uint64_t* empty = full + kStages;
    uint64_t* tfull = empty + kStages;
    uint64_t* tempty = tfull + 2;
    uint64_t* mma_done = tempty + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 1);
    volatile uint32_t* abort_flag = tmem_slot + 1;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int kSide = PAIR ? 256 : 128;  // rows and columns of a tile
    const int q = PAIR ? (int)ptx::cluster_ctarank() : 0;  // 0 = leader
    const int first = PAIR ? blockIdx.x >> 1 : blockIdx.x, pairs = PAIR ? gridDim.x >> 1 : gridDim.x;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) { ptx::mbar_init(&full[s], 1); ptx::mbar_init(&empty[s], 1); }
        for (int s = 0; s < 2; ++s) { ptx::mbar_init(&tfull[s], 1); ptx::mbar_init(&tempty[s], PAIR ? 2 * kEpi : kEpi); }
        ptx::mbar_init(mma_done, 1);
        *abort_flag = 0u;
        ptx::fence_mbar_init();
        ptx::fence_proxy_async_shared();
    }
    if (warp == 2) {
        if (PAIR) {
            ptx::tmem_alloc_pair(tmem_slot, 2 * kSide);
            ptx::tmem_relinquish_pair();
        } else {
            ptx::tmem_alloc(tmem_slot, 2 * kSide);
            ptx::tmem_relinquish();
        }
    }
    if (warp == 0 && lane == 0) {
        ptx::prefetch_tmap(&p.tmA);
        for (int r = 0; r < p.R; ++r) ptx::prefetch_tmap(&p.tmW[r]);
        if (PASS == kXentGrads) {
            ptx::prefetch_tmap(&p.tmA2);
            ptx::prefetch_tmap(&p.tmB);
        }
    }
    __syncwarp();
    ptx::tc_fence_before();
    if (PAIR) ptx::cluster_sync();
    else __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    ptx::grid_launch_dependents();
    ptx::grid_wait();  // nothing of the caller's or of the buffers is touched before

    if (warp == 0) {
        // ------------------------------------------------------------ TMA producer (both CTAs)
        const bool issuer = ptx::elect_one();
        const uint64_t pol = ptx::policy_evict_normal();
        int stage = 0;
        uint32_t ph = 0, issued = 0, issued_ph = 0;
        bool aborted = false;
        for (int u = first; u < p.units && !aborted; u += pairs) {
            const Tile t = tile_of<PASS>(p, u);
            const bool dh = PASS == kXentGrads && t.kind == kXentDH, dw = PASS == kXentGrads && !dh;
            const Place at = place_of(p, PASS == kXentGrads ? 0 : t.tn);
            const int a0 = t.tm * kSide + q * 128, b0 = t.tn * kSide + q * 128;
            // rows of A behind the last one are not loaded: whatever the buffers hold, it enters no other row's sums
            const bool has_a = dw || a0 < p.M, both_a = dw || t.tm * kSide + 128 < p.M;
            const uint32_t a_bytes = dw ? kHalf : (uint32_t)p.a_rows * 128;
            for (int kb = t.kb0; kb < t.kb1; ++kb) {
                const bool ok = wait(&empty[stage], ph ^ 1u, abort_flag, p, 30, u);
                if (!__all_sync(0xFFFFFFFFu, ok)) {
                    aborted = true;
                    break;
                }
                if (issuer) {
                    // both CTAs' copies complete on the leader's barrier
                    uint8_t *a = sA + stage * kHalf, *b = sB + stage * kHalf;
                    const int k = kb * 64;
                    if (!PAIR) {
                        ptx::mbar_arrive_expect_tx(&full[stage], kHalf + a_bytes);
                        ptx::tma_load_2d(a, &p.tmA, &full[stage], k, a0, pol);
                        ptx::tma_load_2d(b, &p.tmW[at.rank], &full[stage], k, at.col, pol);
                    }
                    const uint32_t fb = PAIR ? ptx::mapa_shared(ptx::smem_u32(&full[stage]), 0) : 0;
                    if (PAIR && q == 0) ptx::mbar_arrive_expect_tx(&full[stage], 2 * kHalf + (both_a ? 2 * a_bytes : a_bytes));
                    if (!PAIR) {
                    } else if (dw) {
                        // d's first and second part in turn, with the same block of h
                        const int part = (kb & p.second) * p.columns, row = (kb >> p.second) * 64;
                        for (int i = 0; i < 2; ++i) {
                            ptx::tma_load_2d_pair(a + i * 8192, &p.tmA2, fb, part + a0 + i * 64, row, pol);
                            ptx::tma_load_2d_pair(b + i * 8192, &p.tmB, fb, b0 + i * 64, row, pol);
                        }
                    } else {
                        if (has_a) ptx::tma_load_2d_pair(a, &p.tmA, fb, dh ? (kb & p.second) * p.columns + (kb >> p.second) * 64 : k, a0, pol);
                        if (dh) {
                            const int block = kb >> p.second;
                            const Place w = place_of(p, block >> 2);
                            const int v = w.col + (block & 3) * 64;
                            for (int i = 0; i < 2; ++i)
                                ptx::tma_load_2d_pair(b + i * 8192, &p.tmW[w.rank], fb, b0 + i * 64, v, pol);
                        } else {
                            ptx::tma_load_2d_pair(b, &p.tmW[at.rank], fb, k, at.col + q * 128, pol);
                        }
                    }
                }
                __syncwarp();
                issued |= 1u << stage;
                issued_ph = (issued_ph & ~(1u << stage)) | (ph << stage);
                if (++stage == kStages) { stage = 0; ph ^= 1u; }
            }
        }
        if (q == 0) {
            for (int s = 0; s < kStages; ++s)
                if (issued & (1u << s)) drain(&full[s], (issued_ph >> s) & 1u, p);
        } else if (aborted) {
            // this CTA's copies land on the leader's barriers: give them time to land
            const uint64_t t0 = ptx::globaltimer();
            while (ptx::globaltimer() - t0 < 50000) {}
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer (leader only)
        if (q == 0) {
            const bool issuer = ptx::elect_one();
            int stage = 0, it = 0;
            uint32_t ph = 0;
            constexpr bool kAcrossB = PASS == kXentGrads;
            bool ok = true;
            for (int u = first; u < p.units && ok; u += pairs) {
                const Tile t = tile_of<PASS>(p, u);
                // along the contraction: rows of 128 bytes, 32 of them a step; across: two groups of 64 columns, 16 rows a step
                const bool across_a = PASS == kXentGrads && t.kind == kXentDW;
                const uint64_t adesc = sdesc(ptx::smem_u32(sA), across_a ? 8192 : 16, 1024);
                const uint64_t bdesc = sdesc(ptx::smem_u32(sB), kAcrossB ? 8192 : 16, 1024);
                const int step_a = across_a ? 128 : 2, step_b = kAcrossB ? 128 : 2;
                const uint32_t id = idesc(across_a, kAcrossB, kSide);
                // an accumulator holds the whole sum, or a part of it (kPart blocks)
                for (int kb = t.kb0; kb < t.kb1; ++kb) {
                    const int in_part = PASS == kXentGrads ? kb - t.kb0 : (kb - t.kb0) % kPart;
                    const bool last = kb == t.kb1 - 1 || (PASS != kXentGrads && in_part == kPart - 1);
                    const int buf = it & 1;
                    if (in_part == 0) {
                        ok = __all_sync(0xFFFFFFFFu, wait(&tempty[buf], ((uint32_t)(it >> 1) & 1u) ^ 1u, abort_flag, p, 31, u));
                        if (!ok) break;
                        ptx::tc_fence_after();
                    }
                    ok = __all_sync(0xFFFFFFFFu, wait(&full[stage], ph, abort_flag, p, 32, u));
                    if (!ok) break;
                    ptx::tc_fence_after();
                    if (issuer) {
                        const uint32_t d = tmem_base + buf * kSide;
                        const uint64_t ad = adesc + (uint64_t)(stage * (kHalf >> 4)), bd = bdesc + (uint64_t)(stage * (kHalf >> 4));
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk) {
                            const uint64_t ak = ad + (uint64_t)(kk * step_a), bk = bd + (uint64_t)(kk * step_b);
                            if (PAIR) ptx::umma_bf16_pair(d, ak, bk, id, in_part != 0 || kk != 0);
                            else ptx::umma_bf16(d, ak, bk, id, in_part != 0 || kk != 0);
                        }
                        if (PAIR) ptx::umma_commit_pair_multicast(&empty[stage], 0x3);
                        else ptx::umma_commit(&empty[stage]);
                        if (last) {
                            if (PAIR) ptx::umma_commit_pair_multicast(&tfull[buf], 0x3);
                            else ptx::umma_commit(&tfull[buf]);
                        }
                    }
                    __syncwarp();
                    if (++stage == kStages) { stage = 0; ph ^= 1u; }
                    if (last) ++it;
                }
            }
            if (issuer) {
                if (PAIR) ptx::umma_commit_pair(mma_done);
                else ptx::umma_commit(mma_done);
            }
            __syncwarp();
            drain(mma_done, 0, p);
        }
    } else if (warp >= 4 && PASS != kXentGrads) {
        // ------------------------------------------------------------ the logits: a thread owns a group of a row's columns
        constexpr int kGroups = kEpi / 4, kCols = kSide / kGroups;
        const int w = warp & 3, group = (warp - 4) >> 2;
        uint8_t* const box = sOut + (warp - 4) * (kCols / 64) * kBox;
        const uint64_t scale = ptx::pair(kLog2e, kLog2e);
        int part = 0;
        bool ok = true;
        if (PASS == kXentDLogits && p.rows_from) copy_rows(p, blockIdx.x * kEpi + warp - 4, gridDim.x * kEpi);
        for (int u = first; u < p.units; u += pairs) {
            const Tile t = tile_of<PASS>(p, u);
            uint64_t z[kCols / 2];  // pairs of columns
#pragma unroll
            for (int i = 0; i < kCols / 2; ++i) z[i] = 0ull;
            for (int kb = t.kb0; kb < t.kb1; kb += kPart, ++part) {
                const int buf = part & 1;
                ok = __all_sync(0xFFFFFFFFu, wait(&tfull[buf], (uint32_t)(part >> 1) & 1u, abort_flag, p, 33, u));
                if (!ok) break;
                ptx::tc_fence_after();
                const uint32_t acc = tmem_base + ((uint32_t)(w * 32) << 16) + buf * kSide + group * kCols;
#pragma unroll
                for (int j = 0; j < kCols; j += 16) {
                    uint32_t v[16];
                    ptx::tmem_ld16(acc + j, v);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        z[j / 2 + i] = ptx::add2(z[j / 2 + i], ptx::pair(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])));
                }
                // the accumulator goes back to the leader's MMA warp (with a release it went 2000 cycles later, when the
                // stores in flight had ended: forward 1053 us for 1047, 128 tokens' gradients 185 for 157)
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (PAIR) ptx::mbar_arrive_cluster_relaxed(ptx::mapa_shared(ptx::smem_u32(&tempty[buf]), 0));
                    else ptx::mbar_arrive(&tempty[buf]);
                }
                __syncwarp();
            }
            if (!ok) break;
            const Place at = place_of(p, t.tn);
            const int cols = max(0, min(kCols, columns_of(p, at, kSide) - group * kCols));  // of the group, in the vocabulary
            const int m0 = t.tm * kSide + q * 128 + w * 32, m = m0 + lane;                  // the warp's rows, the thread's
            const int64_t tgt = m < p.M ? target_of(p, m) : -1;
            const int64_t column = tgt - ((int64_t)at.rank * p.Vs + at.col + group * kCols);
            const int mine = tgt >= 0 && column >= 0 && column < cols ? (int)column : -1;  // the target's column, if it is here
            float target = 0.f;
            if (mine >= 0) {
#pragma unroll
                for (int i = 0; i < kCols / 2; ++i) {
                    const float2 e = ptx::unpair(z[i]);
                    target = 2 * i == mine ? e.x : 2 * i + 1 == mine ? e.y : target;
                }
            }
            if (PASS == kXentLogSum) {
                if (mine >= 0) p.target_logit[m] = target;
                float top = -INFINITY, sum[4] = {0.f, 0.f, 0.f, 0.f};
                if (cols > 0) {
                    if (cols < kCols) {
#pragma unroll
                        for (int i = 0; i < kCols / 2; ++i) {
                            const float2 e = ptx::unpair(z[i]);
                            z[i] = ptx::pair(2 * i < cols ? e.x : -INFINITY, 2 * i + 1 < cols ? e.y : -INFINITY);
                        }
                    }
#pragma unroll
                    for (int i = 0; i < kCols / 2; ++i) {
                        const float2 e = ptx::unpair(z[i]);
                        top = fmaxf(top, fmaxf(e.x, e.y));
                    }
                    // the difference is formed before the scaling: a row's largest logit has exactly exp 1
                    const uint64_t minus = ptx::pair(-top, -top);
#pragma unroll
                    for (int i = 0; i < kCols / 2; ++i) {
                        const float2 e = ptx::unpair(ptx::mul2(ptx::add2(z[i], minus), scale));
                        sum[(2 * i) & 3] += ex2(e.x);
                        sum[(2 * i + 1) & 3] += ex2(e.y);
                    }
                }
                if (m < p.M)
                    p.stats[((size_t)m * p.grid[0].tiles_n + t.tn) * kGroups + group] = make_float2(top, (sum[0] + sum[1]) + (sum[2] + sum[3]));
            } else {
                const bool on = tgt >= 0;  // a row without a target has no gradient, whatever its logits
                const float lse = on ? p.lse[m] : 0.f, g = on ? p.dloss[m] : 0.f;
                const uint64_t minus = ptx::pair(-lse, -lse), g2 = ptx::pair(g, g);
                // g (p - 1) for the target: the difference before the rounding, and without cancellation where p is near 1
                const float own = mine >= 0 ? g * expm1f(target - lse) : 0.f;
#pragma unroll
                for (int i = 0; i < kCols / 2; ++i) {
                    const float2 e = ptx::unpair(ptx::mul2(ptx::add2(z[i], minus), scale));
                    float2 x = ptx::unpair(ptx::mul2(ptx::pair(ex2(e.x), ex2(e.y)), g2));
                    x.x = !on || 2 * i >= cols ? 0.f : 2 * i == mine ? own : x.x;
                    x.y = !on || 2 * i + 1 >= cols ? 0.f : 2 * i + 1 == mine ? own : x.y;
                    z[i] = ptx::pair(x.x, x.y);
                }
                // d rounded to bf16, and what that rounding left, which is rounded in its turn
                for (int part = 0; part <= p.second; ++part) {
                    __syncwarp();
                    if (lane == 0) ptx::bulk_wait_read0();
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < kCols / 8; ++i) {
                        uint32_t d[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float2 x = ptx::unpair(z[4 * i + j]);
                            d[j] = bf16x2(x.x, x.y);
                            z[4 * i + j] = ptx::pair(x.x - __uint_as_float(d[j] << 16), x.y - __uint_as_float(d[j] & 0xFFFF0000u));
                        }
                        *chunk_at(box + (i / 8) * kBox, lane, i % 8) = make_uint4(d[0], d[1], d[2], d[3]);
                    }
                    ptx::fence_proxy_async_shared();
                    __syncwarp();
                    if (lane == 0) {
                        if (m0 < p.M)
                            for (int i = 0; i < kCols / 64; ++i)
                                ptx::tma_store_2d(&p.tmOut[0], box + i * kBox, part * p.columns + t.tn * kSide + group * kCols + i * 64, m0);
                        ptx::bulk_commit();
                    }
                }
            }
            __syncwarp();
        }
        if (lane == 0) ptx::bulk_wait0();
    } else if (warp >= 4) {
        // ------------------------------------------------------------ epilogue: a thread owns a row of the CTA's half
        const int w = warp - 4;
        Stager out{sOut + w * 2 * kBox, 0};
        int it = 0;
        for (int u = first; u < p.units; u += pairs, ++it) {
            const Tile t = tile_of<PASS>(p, u);
            const int buf = it & 1;
            const bool dw = t.kind == kXentDW;
            const Place at = place_of(p, dw ? t.tm : 0);
            const int m0 = t.tm * kSide + q * 128 + w * 32;        // the warp's rows of the tile
            const int r0 = dw ? at.col + q * 128 + w * 32 : m0;   // and of dh, or of a rank's dW
            // a row without a target, or behind the vocabulary, is zeros: its d is, but 0 times an infinity or a NaN is none
            const bool on = dw ? r0 + lane - at.col < columns_of(p, at, kSide) : m0 + lane < p.M && target_of(p, m0 + lane) >= 0;
            if (!__all_sync(0xFFFFFFFFu, wait(&tfull[buf], (uint32_t)(it >> 1) & 1u, abort_flag, p, 33, u))) break;
            ptx::tc_fence_after();
            const uint32_t acc = tmem_base + ((uint32_t)(w * 32) << 16) + buf * kSide;

            if (t.kind == kXentDH && p.sums) {
                // fp32 sums of this split, over the pieces
                for (int c = 0; c < kTile && t.tn * kTile + c < p.K; c += 32) {
                    uint32_t v[32];
                    ptx::tmem_ld32(acc + c, v);
                    uint8_t* box = out.next();
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        *chunk_at(box, lane, i) = on ? make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]) : make_uint4(0u, 0u, 0u, 0u);
                    ptx::fence_proxy_async_shared();
                    __syncwarp();
                    if (lane == 0) {
                        if (m0 < p.M) {
                            if (p.add) ptx::tma_add_3d(&p.tmDH, box, t.tn * kTile + c, m0, t.split);
                            else ptx::tma_store_3d(&p.tmDH, box, t.tn * kTile + c, m0, t.split);
                        }
                        ptx::bulk_commit();
                    }
                    __syncwarp();
                }
            } else {
                // bf16 results: rows of dh, or of a rank's dW
                const bool store = r0 < (dw ? p.Vs : p.M);
                const CUtensorMap* map = dw ? &p.tmOut[at.rank] : &p.tmDH;
                for (int c = 0; c < kTile && t.tn * kTile + c < p.K; c += 64) {
                    uint8_t* box = out.next();
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        uint32_t v[32];
                        ptx::tmem_ld32(acc + c + half * 32, v);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            uint32_t d[4];
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                d[j] = on ? bf16x2(__uint_as_float(v[8 * i + 2 * j]), __uint_as_float(v[8 * i + 2 * j + 1])) : 0u;
                            *chunk_at(box, lane, half * 4 + i) = make_uint4(d[0], d[1], d[2], d[3]);
                        }
                    }
                    ptx::fence_proxy_async_shared();
                    __syncwarp();
                    if (lane == 0) {
                        if (store) ptx::tma_store_2d(map, box, t.tn * kTile + c, r0);
                        ptx::bulk_commit();
                    }
                    __syncwarp();
                }
            }
            // the accumulator goes back to the leader's MMA warp
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (PAIR) ptx::mbar_arrive_cluster_relaxed(ptx::mapa_shared(ptx::smem_u32(&tempty[buf]), 0));
                else ptx::mbar_arrive(&tempty[buf]);
            }
        }
        if (lane == 0) ptx::bulk_wait0();
    }

    __syncwarp();
    ptx::tc_fence_before();
    if (PAIR) ptx::cluster_sync();
    else __syncthreads();
    ptx::tc_fence_after();
    if (warp == 2) {
        __syncwarp();
        if (PAIR) ptx::tmem_dealloc_pair(tmem_base, 2 * kSide);
        else ptx::tmem_dealloc(tmem_base, 2 * kSide);
    }
}

// Joins the tiles' (maximum, sum) pairs of a row, and the pieces' before; after the last
// piece lse = max + log(sum) and loss = (max - z_t) + log(sum), which for a token that is
// foreseen has no large terms.  A warp a row.
__global__ void __launch_bounds__(256) xent_join_kernel(const float2* stats, float2* carry, const float* target_logit,
                                                        const void* targets, int wide, int64_t vocab, float* loss, float* lse,
                                                        int M, int tiles, int first, int last) {
    const int row = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    ptx::grid_launch_dependents();
    ptx::grid_wait();
    if (row >= M) return;
    const float2* at = stats + (size_t)row * tiles;
    float top = -INFINITY, sum = 0.f;
    if (!first && lane == 0) {
        const float2 c = carry[row];
        top = c.x;
        sum = c.y;
    }
    constexpr int U = 8;  // pairs in flight
    for (int i0 = lane; i0 < tiles; i0 += 32 * U) {
        float2 v[U];
#pragma unroll
        for (int j = 0; j < U; ++j) v[j] = i0 + 32 * j < tiles ? at[i0 + 32 * j] : make_float2(-INFINITY, 0.f);
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const float hi = fmaxf(top, v[j].x);
            // (a tile outside the vocabulary has maximum -inf and sum 0)
            sum = (hi == top ? sum : sum * ex2((top - hi) * kLog2e)) + (hi == v[j].x ? v[j].y : v[j].y * ex2((v[j].x - hi) * kLog2e));
            top = hi;
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float x = __shfl_xor_sync(0xFFFFFFFFu, top, o), y = __shfl_xor_sync(0xFFFFFFFFu, sum, o);
        const float hi = fmaxf(top, x);
        const float a = hi == top ? sum : sum * ex2((top - hi) * kLog2e), b = hi == x ? y : y * ex2((x - hi) * kLog2e);
        sum = a + b;  // the same in both lanes: a sum does not depend on the order of two terms
        top = hi;
    }
    if (lane) return;
    if (!last) {
        carry[row] = make_float2(top, sum);
        return;
    }
    const float rest = logf(sum);
    lse[row] = top + rest;
    const int64_t t = wide ? static_cast<const int64_t*>(targets)[row] : static_cast<const int32_t*>(targets)[row];
    loss[row] = t >= 0 && t < vocab ? (top - target_logit[row]) + rest : 0.f;
}

// dh = the splits' fp32 sums, in their order, rounded to bf16 once.
__global__ void __launch_bounds__(256) xent_dh_kernel(const float4* sums, uint2* dh, int64_t quads, int splits) {
    ptx::grid_launch_dependents();
    ptx::grid_wait();
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < quads; i += (int64_t)gridDim.x * 256) {
        float4 a = sums[i];
        constexpr int U = 8;  // sets in flight
        for (int s0 = 1; s0 < splits; s0 += U) {
            float4 b[U];
#pragma unroll
            for (int j = 0; j < U; ++j)
                if (s0 + j < splits) b[j] = sums[(s0 + j) * quads + i];
#pragma unroll
            for (int j = 0; j < U; ++j)
                if (s0 + j < splits) { a.x += b[j].x; a.y += b[j].y; a.z += b[j].z; a.w += b[j].w; }
        }
        dh[i] = make_uint2(bf16x2(a.x, a.y), bf16x2(a.z, a.w));
    }
}

template <int PASS, bool PAIR = true>
cudaError_t launch(XentParams& p, int clusters, cudaStream_t s) {
    p.units = 0;
    p.per_rank = Divisor(p.rank_tiles);
    for (XentGrid& g : p.grid) {
        p.units += g.units = g.tiles_m * g.tiles_n * g.splits;
        if (g.units == 0) continue;
        g.per_split = Divisor(g.tiles_m * g.tiles_n);
        g.per_group = Divisor(p.group * g.tiles_n);
        g.rows = Divisor(p.group);
        g.last_rows = Divisor((g.tiles_m - 1) % p.group + 1);
        g.parts = Divisor(g.splits);
    }
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = PAIR ? 2 : 1;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1] = dependent_launch();  // a CTA comes up on an SM that the kernel before has left
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(PAIR ? 2 * std::min(p.units, clusters) : std::min(p.units, 2 * clusters)));
    cfg.blockDim = dim3(Shape<PASS, PAIR>::kThreads);
    cfg.dynamicSmemBytes = Shape<PASS, PAIR>::kSmem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, xent_kernel<PASS, PAIR>, p);
}

// Up to 128 tokens the logits' tiles are 128 x 128, each of one CTA: of a pair's 256 rows half would be empty, and its
// product of 256 x 256 x 64 takes 0.27 us whatever it holds, as long as the copies do.
constexpr int kFewTokens = 128;
constexpr int kGroup = 16;  // rows of tiles whose operand stays in L2: 4096 rows

// dh's sums as a map [splits, M, K] of fp32, 128B-swizzled boxes of 32 columns x 32 rows.
cudaError_t make_tmap_sums(CUtensorMap* m, const void* base, uint64_t K, uint64_t M, uint64_t splits) {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q);
    if (e != cudaSuccess || q != cudaDriverEntryPointSuccess || fn == nullptr) return cudaErrorNotSupported;
    const cuuint64_t dims[3] = {K, M, splits}, strides[2] = {K * 4, K * M * 4};
    const cuuint32_t box[3] = {32, 32, 1}, each[3] = {1, 1, 1};
    const CUresult r = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn)(
        m, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, const_cast<void*>(base), dims, strides, box, each, CU_TENSOR_MAP_INTERLEAVE_NONE,
        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

int ceil256(int64_t n) { return (int)((n + kTile - 1) / kTile); }

}  // namespace

template <int PASS>
static are_launch_info launched(int kernel, const XentParams& p, bool few, int clusters) {
    return few ? are_launch_info{kernel, std::min(p.units, 2 * clusters), Shape<PASS, false>::kThreads, 1, 0, 0, 0, p.group}
               : are_launch_info{kernel, 2 * std::min(p.units, clusters), Shape<PASS, true>::kThreads, 2, 0, 0, 0, p.group};
}

template <int PASS, bool PAIR>
static cudaError_t opt_in_xent() {
    return cudaFuncSetAttribute(xent_kernel<PASS, PAIR>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Shape<PASS, PAIR>::kSmem);
}

cudaError_t xent_prepare(int* clusters) {
    for (cudaError_t e : {opt_in_xent<kXentLogSum, true>(), opt_in_xent<kXentLogSum, false>(), opt_in_xent<kXentDLogits, true>(),
                          opt_in_xent<kXentDLogits, false>(), opt_in_xent<kXentGrads, true>()})
        if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = 2;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2048);
    cfg.blockDim = dim3(Shape<kXentLogSum, true>::kThreads);
    cfg.dynamicSmemBytes = Shape<kXentDLogits, true>::kSmem;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaOccupancyMaxActiveClusters(clusters, xent_kernel<kXentDLogits, true>, &cfg);
}

// Sets of sums that dh's contraction over the vocabulary is split into, at most `most`.  Few tokens have few tiles, and
// the pairs that would have none take parts of the contraction; from half a wave of tiles on, two to four parts make the
// last wave fuller (4096 tokens, K = 4096: 256 tiles are 3.4 waves of 76; in two parts 6.7: 170 -> 150 us a piece).
static int dh_splits(int tiles, int clusters, int most) {
    int best = std::max(1, std::min(clusters / tiles, most));
    auto filled = [&](int s) { return (double)tiles * s / (((int64_t)tiles * s + clusters - 1) / clusters * clusters); };
    if (best == 1)
        for (int s = 2; s <= std::min(4, most); ++s)
            if (filled(s) > filled(best) + 0.04) best = s;
    return best;
}

// Rows of rank r's weights that are in the vocabulary.  Those behind are not read, and count as zeros where a tile has them:
// whatever they hold, infinities and NaN too, enters nothing.
static int64_t rows_in(const XentCall& c, int r) { return std::max<int64_t>(0, std::min(c.Vs, c.vocab - r * c.Vs)); }
static int last_rank(const XentCall& c) { return (int)((c.vocab - 1) / c.Vs); }
// Vocabulary tiles, up to the last that holds some of the vocabulary.
static int tiles_in(const XentCall& c, int tile, int rank_tiles) {
    const int r = last_rank(c);
    return r * rank_tiles + (int)((rows_in(c, r) + tile - 1) / tile);
}

static void common(XentParams& p, const XentCall& c, const XentBuffers& b) {
    p.M = (int)c.M;
    p.K = (int)c.K;
    p.Vs = (int)c.Vs;
    p.vocab = c.vocab;
    p.tile = kTile;
    p.rank_tiles = ceil256(c.Vs);
    p.targets = c.targets;
    p.wide = c.wide;
    p.status = b.status;
    p.timeout_ns = b.timeout_ns;
    p.R = last_rank(c) + 1;  // ranks behind have none of the vocabulary
    p.group = kGroup;
    p.a_rows = (int)std::min<int64_t>((c.M + 7) / 8 * 8, 128);
}

cudaError_t launch_xent_forward(const XentCall& c, const XentBuffers& b, cudaStream_t s, are_launch_info* info) {
    XentParams p{};
    common(p, c, b);
    cudaError_t e = make_tmap_bf16(&p.tmA, c.h, (uint64_t)c.K, (uint64_t)c.M, 64, p.a_rows);
    for (int r = 0; r < p.R && e == cudaSuccess; ++r)
        e = make_tmap_bf16(&p.tmW[r], c.w[r], (uint64_t)c.K, (uint64_t)rows_in(c, r), 64, 128);
    if (e != cudaSuccess) return e;
    const bool few = c.M <= kFewTokens;
    if (few) {
        p.tile = 128;
        p.rank_tiles = (int)((c.Vs + 127) / 128);
    }
    const int total = tiles_in(c, p.tile, p.rank_tiles), each = few ? 1 : 4;  // pairs of a row that a tile leaves
    const int fit = (int)std::min<int64_t>(total, (int64_t)(b.sizes.d_bytes / ((size_t)c.M * 8 * each)));
    p.stats = static_cast<float2*>(b.d);
    float2* carry = static_cast<float2*>(b.rows);
    p.target_logit = reinterpret_cast<float*>(carry + c.M);
    XentGrid& g = p.grid[0];
    g = XentGrid{ceil256(c.M), 0, 1, (int)((c.K + 63) / 64), 0};
    for (p.tile0 = 0; p.tile0 < total && e == cudaSuccess; p.tile0 += g.tiles_n) {
        g.tiles_n = std::min(fit, total - p.tile0);
        e = few ? launch<kXentLogSum, false>(p, b.clusters, s) : launch<kXentLogSum>(p, b.clusters, s);
        if (p.tile0 == 0) *info = launched<kXentLogSum>(ARE_KERNEL_CROSS_ENTROPY, p, few, b.clusters);
        if (e != cudaSuccess) return e;
        e = launch_dependent(xent_join_kernel, dim3((unsigned)((c.M + 7) / 8)), 256, 0, s, p.stats, carry, p.target_logit,
                             c.targets, c.wide, c.vocab, c.loss, c.lse, (int)c.M, each * g.tiles_n, p.tile0 == 0,
                             p.tile0 + g.tiles_n == total);
    }
    return e;
}

cudaError_t launch_xent_backward(const XentCall& c, const XentBuffers& b, cudaStream_t s, are_launch_info* info) {
    XentParams z{};  // the logits and their gradient
    common(z, c, b);
    z.lse = c.lse;
    z.dloss = c.dloss;
    XentParams d = z;  // the products with it
    const bool few = c.M <= kFewTokens;
    if (few) {
        z.tile = 128;
        z.rank_tiles *= 2;  // halves of the tiles that the products take
    }
    const int total = tiles_in(c, kTile, d.rank_tiles), tiles_m = ceil256(c.M), tiles_k = ceil256(c.K);
    const int most = (int)std::min<int64_t>(total, (int64_t)(b.sizes.d_bytes / ((size_t)c.M * kTile * 2)));
    z.second = d.second = b.parts - 1;
    const int even = (total + most - 1) / most, piece = (total + even - 1) / even;
    const int pieces = (total + piece - 1) / piece, left = total - (pieces - 1) * piece;  // the last piece's tiles, 1..piece
    cudaError_t e = make_tmap_bf16(&z.tmA, c.h, (uint64_t)c.K, (uint64_t)c.M, 64, z.a_rows);
    for (int r = 0; r < c.R && c.has_dw && e == cudaSuccess; ++r) {
        // rows of dW that no tile has
        const int64_t from = r < z.R - 1 ? c.Vs : r >= z.R ? 0 : std::min<int64_t>(c.Vs, (int64_t)ceil256(rows_in(c, r)) * kTile);
        if (from < c.Vs) e = cudaMemsetAsync(c.dw[r] + from * c.K, 0, (size_t)(c.Vs - from) * c.K * 2, s);
    }
    for (int r = 0; r < z.R && e == cudaSuccess; ++r) {
        e = make_tmap_bf16(&z.tmW[r], c.w[r], (uint64_t)c.K, (uint64_t)rows_in(c, r), 64, 128);
        if (e == cudaSuccess) e = make_tmap_bf16(&d.tmW[r], c.w[r], (uint64_t)c.K, (uint64_t)rows_in(c, r), 64, 64);
        if (e == cudaSuccess && c.has_dw) e = make_tmap_bf16(&d.tmOut[r], c.dw[r], (uint64_t)c.K, (uint64_t)c.Vs, 64, 32);
    }
    if (e == cudaSuccess) e = make_tmap_bf16(&d.tmB, b.h, (uint64_t)c.K, (uint64_t)c.M, 64, 64);
    const int splits = dh_splits(tiles_m * tiles_k, b.clusters,
                                 (int)std::min({(int64_t)(b.sizes.sum_bytes / ((size_t)c.M * c.K * 4)), (int64_t)piece / 2, (int64_t)4 * left}));
    d.sums = pieces > 1 || splits > 1;
    if (e == cudaSuccess && c.dh)
        e = d.sums ? make_tmap_sums(&d.tmDH, b.sums, (uint64_t)c.K, (uint64_t)c.M, (uint64_t)splits)
                   : make_tmap_bf16(&d.tmDH, c.dh, (uint64_t)c.K, (uint64_t)c.M, 64, 32);
    if (c.has_dw) {
        z.rows_from = reinterpret_cast<const uint4*>(c.h);
        z.rows_to = static_cast<uint4*>(b.h);
    }
    for (int t0 = 0; t0 < total && e == cudaSuccess; t0 += piece) {
        const int n = std::min(piece, total - t0);
        z.tile0 = d.tile0 = t0;
        z.grid[0] = XentGrid{tiles_m, few ? 2 * n : n, 1, (int)((c.K + 63) / 64), 0};
        if (few) z.tile0 = 2 * t0;
        if (c.dh) d.grid[0] = XentGrid{tiles_m, tiles_k, splits, 4 * n * b.parts, 0};
        if (c.has_dw) d.grid[1] = XentGrid{n, tiles_k, 1, (int)((c.M + 63) / 64) * b.parts, 0};
        z.columns = d.columns = n * kTile;
        const uint64_t cols = (uint64_t)n * kTile * b.parts;
        if (t0 == 0 || n != piece) {  // the piece's d [M, parts, columns]: as an output, along and across the contraction
            e = make_tmap_bf16(&z.tmOut[0], b.d, cols, (uint64_t)c.M, 64, 32);
            if (e == cudaSuccess) e = make_tmap_bf16(&d.tmA, b.d, cols, (uint64_t)c.M, 64, d.a_rows);
            if (e == cudaSuccess) e = make_tmap_bf16(&d.tmA2, b.d, cols, (uint64_t)c.M, 64, 64);
        }
        if (e == cudaSuccess) e = few ? launch<kXentDLogits, false>(z, b.clusters, s) : launch<kXentDLogits>(z, b.clusters, s);
        if (t0 == 0) *info = launched<kXentDLogits>(ARE_KERNEL_CROSS_ENTROPY_BACKWARD, z, few, b.clusters);
        z.rows_from = nullptr;
        d.add = t0 > 0;
        if (e == cudaSuccess) e = launch<kXentGrads>(d, b.clusters, s);
    }
    if (e == cudaSuccess && c.dh && d.sums) {
        const int64_t quads = c.M * c.K / 4;
        e = launch_dependent(xent_dh_kernel, dim3((unsigned)std::min<int64_t>((quads + 255) / 256, 16 * b.clusters)), 256, 0, s,
                             static_cast<const float4*>(b.sums), reinterpret_cast<uint2*>(c.dh), quads, splits);
    }
    return e;
}

}  // namespace are
