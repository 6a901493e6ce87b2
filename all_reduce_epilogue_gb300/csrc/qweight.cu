// The row-parallel linear of a few tokens with 4-bit weights, all-reduced over
// R ranks:
//   out[m][n] = bf16( sum_{r=0..R-1} sum_k x_r[m][k] * (u_r[n][k] - z_r[n][g]) * s_r[n][g] ),
//   g = k / group,
// with tokens x in bf16, or in FP8 E4M3 codes times a scale per group of k.
//
// Bound by the weights' bytes: M tokens use each of them M times.  What
// competes with the bytes is the integer work of unpacking the codes, so that
// is made as small as it gets:
//  * A code in bits 0..3 of a bf16 is the subnormal u * 2^-133; in bits 4..7 it is
//    u * 2^-129, as the first binade of normal numbers goes on in the same steps.
//    So a word of 8 codes becomes four operand registers of m16n8k16 tensor
//    instructions (16 rows of weights, 16 of k, 8 tokens, fp32 sums) by four
//    masks and a shift: the pairs (0, 4) (1, 5) (2, 6) (3, 7).  The tokens are
//    staged in that order, scaled up to match, the odd k by 2^-4 less.
//    (Codes made into normal numbers take 7 to 11 instructions a word.  FP8
//    operands would take 3, but FP8 mma.sync is not native here: it measured 36
//    cycles a sub-core for 32 of k, 16-bit ones 8.2 for 16.)
//  * Such an instruction adds its 16 products and the sum so far to 25 bits below
//    the largest of their exponents, and counts a subnormal's as 2^-126: 7 bits
//    above u = 1.  What it cuts of each is up to 2^-18 of the largest token whose
//    code is not zero (in units of the code), 17 times 2^-18 in all.  In fp16, with
//    3 bits of mantissa more to be subnormal in, that was 2^-15; normal numbers
//    (from E4M3, which reads a code byte as u * 2^-9) have 2^-25 of u times the
//    token, and measured 6 to 11 % slower (one token 18.5 us for 16.6, 64 75.5 for
//    70.9; all codes in bits 4..7, 2^-22: 17.8 and 76).  The output's rounding to
//    bf16 is 2^-9 of what is left after the ranks and groups have been added up.
//  * The tokens enter exactly: bf16 as they are, FP8 codes times 2^7 or times their
//    power-of-two scales, scaled per token and 256 of k by the power of two that
//    takes the largest value to 2^14..2^15, which their scale in fp32 undoes, and
//    all by 2^109.  What is 2^-112 of the largest or less may lose bits.
//  * The zero point leaves the sums: sum (u - z) x = sum u x - z sum x, with
//    sum x per token and group in fp32.  The scales are applied in fp32, once
//    per group, to the tensor instruction's fp32 sums.  No weight is rounded.
//  * bf16 values that are not finite are staged as zeros, and their tokens'
//    outputs get the products that hold them one by one at the end.
//
// The codes are read once, into a ring of shared memory per warp (16-byte
// asynchronous copies ahead of their use, no barrier between warps).  A cluster
// owns a run of row groups; each of its CTAs takes one rank's (or, where R is
// small, part of a rank's) K range for all of them.  At the end the CTAs add
// their fp32 sums over distributed shared memory, r ascending: no partial sum
// goes through global memory and the order never varies.
//  * In tiles of 8 tokens (qweight_few_kernel), a CTA stages its tokens itself,
//    and the (group, K) items of a CTA are dealt to its warps in equal contiguous
//    runs of 16-row groups.  R = 8, one token, 7168 x 2048: 17 us, 3.7 TB/s of
//    codes; issue slots are 51 % used (about 70 % in the loop over the codes,
//    which is 60 % of the time), DRAM 37 %; the rest is start and cluster sum.
//  * In tiles of 16 or 32 (qweight_tokens_kernel, then qweight_wide_kernel), they
//    are staged once, in global memory, and come in tiles of K by bulk copies; a warp
//    owns 32 rows, which share the tokens' operands, and their sums stay in
//    registers.  R = 8: 16 tokens, 8192 x 4096, groups of 64: 46 us (4 of them
//    staging), 3.1 TB/s; 64 tokens, 7168 x 2048: 71 us, tensor pipes 47 %, issue
//    44 %, at the four warps a scheduler that the registers allow.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <algorithm>
#include <type_traits>

#include "are_internal.h"
#include "ptx.cuh"

namespace are {
namespace {

using ptx::add2;
using ptx::fma2;
using ptx::mul2;
using ptx::pair;
using ptx::unpair;

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxSmem = 113 * 1024;       // two CTAs an SM

// What the tokens are: bf16, or FP8 codes with fp32 or with power-of-two scales.
enum Tokens { kBf16, kFp8, kFp8Pow2 };

// The shape of the kernel for TT token tiles of 8.  An item (a ring slot) is 2 KB of codes.
template <int TT>
struct Shape {
    static constexpr int TOK = TT * 8;
    static constexpr bool OWN = TT >= 2;              // a warp owns its rows
    static constexpr int RT = OWN ? 2 : 1;            // 16-row tiles of a group
    static constexpr int ROWS = RT * 16;
    static constexpr int ITEM = OWN ? 128 : 256;      // k of a slot
    static constexpr int DEPTH = 3;                   // ring slots of a warp
    static constexpr int PITCH = ITEM / 2;            // bytes of a row's codes, in 16-byte pieces that swizzle() permutes
    static constexpr int SLOT = ROWS * PITCH;
    static constexpr int RING = kWarps * DEPTH * SLOT;
    static constexpr int LD = ROWS + 4;               // floats between a sum's tokens: 4 token pairs x 8 rows in 32 banks
    static constexpr int UNITS = 8;                   // units of 8 k a thread stages of a K tile (TT = 1)
};

// What the places of row g's 16-byte pieces are xored with (times 16), its bits reversed: then the 4-, 8- and 16-byte
// reads of 4 lanes of each of 8 rows meet no bank twice, in rows of 64 bytes as of 128.
template <int PITCH>
__device__ __forceinline__ uint32_t swizzle(int g) {
    return (uint32_t)((g & 1) << 2 | (g & 2) | (g >> 2 & 1)) % (PITCH / 16) * 16u;
}

// Shared memory of the kernel for wide tiles, of each of its two buffers, and its K tile: 512 k where they fit.
template <int TT, bool QX, int WSTEPS, int STEPS>
struct Wide {
    static constexpr int TILE = TT == 2 && WSTEPS >= 2 ? 512 : 256;
    static constexpr int WROWS = kWarps * Shape<TT>::ROWS + 1;                 // odd: a row's groups fall into different banks
    static constexpr int XS = 2 * Shape<TT>::TOK * TILE;                        // bytes
    static constexpr int XSUM = TILE / (STEPS * 32) * Shape<TT>::TOK;           // words
    static constexpr int XSC = QX ? XSUM : TILE / 256 * Shape<TT>::TOK;         // (a token group is STEPS * 32 or more)
    static constexpr int WSC = TILE / (WSTEPS * 32) * WROWS;
    static constexpr int SMEM = Shape<TT>::RING + 2 * XS + 8 * (XSUM + XSC + WSC) + 32;
    static_assert(SMEM <= kMaxSmem && 8 * WSC % 16 == 0, "two CTAs an SM, barriers aligned");
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid) {
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// (No load here is a non-coherent one: the kernel may start while the one before it in the stream still writes what it
// reads after grid_wait, and such loads want memory that nothing writes in the kernel's lifetime.)
//
// Loads under a predicate: a register keeps its value where it is false, and no
// branch stands between one load and the next (a branch each had every load
// wait for the one before: 12 thousand cycles for 24 of them).
__device__ __forceinline__ void ldg_if(uint4& v, const void* p, bool on) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %5, 0;\n\t@q ld.global.cg.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}"
        : "+r"(v.x), "+r"(v.y), "+r"(v.z), "+r"(v.w)
        : "l"(p), "r"((uint32_t)on));
}
__device__ __forceinline__ void ldg_if(uint2& v, const void* p, bool on) {
    asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %3, 0;\n\t@q ld.global.cg.v2.u32 {%0, %1}, [%2];\n\t}"
                 : "+r"(v.x), "+r"(v.y)
                 : "l"(p), "r"((uint32_t)on));
}
__device__ __forceinline__ void ldg_u16_if(uint32_t& v, const void* p, bool on) {
    asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %2, 0;\n\t@q ld.global.u16 %0, [%1];\n\t}"
                 : "+r"(v)
                 : "l"(p), "r"((uint32_t)on));
}
__device__ __forceinline__ void ldg_u8_if(uint32_t& v, const void* p, bool on) {
    asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %2, 0;\n\t@q ld.global.cg.u8 %0, [%1];\n\t}"
                 : "+r"(v)
                 : "l"(p), "r"((uint32_t)on));
}

__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}
__device__ __forceinline__ uint2 ld_shared_v2(uint32_t addr) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t ld_shared(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ float2 ld_cluster_f2(uint32_t addr) {
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t ld_cluster(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

// Adds one; what was read from shared memory before is not read later, by this thread or by who sees the sum.
__device__ __forceinline__ uint32_t atom_add_acq_rel(uint32_t* p) {
    uint32_t v;
    asm volatile("atom.acq_rel.cta.shared::cta.add.u32 %0, [%1], 1;" : "=r"(v) : "r"(ptx::smem_u32(p)) : "memory");
    return v;
}

// d (+)= a (weights) * b (tokens).
template <bool FIRST>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t* a, uint32_t b0, uint32_t b1) {
    if (FIRST)
        asm(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%10, %10, %10, %10};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
    else
        asm(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Two floats of tokens as bf16.
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&b);
}
__device__ __forceinline__ float2 fp8x2_to_float2(uint32_t v) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(v & 0xFFFFu), __NV_E4M3);
    return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// A word's codes: pairs (0, 4) and (2, 6) times 2^-133, (1, 5) and (3, 7) times 2^-129.
template <int HALF>
__device__ __forceinline__ void codes8(uint32_t w, uint32_t (&a0)[4], uint32_t (&a1)[4]) {
    a0[HALF] = w & 0x000F000Fu;
    a0[2 + HALF] = w & 0x00F000F0u;
    w >>= 8;
    a1[HALF] = w & 0x000F000Fu;
    a1[2 + HALF] = w & 0x00F000F0u;
}

// A token's power of two, 2^(141 - top) with `top` the biased exponent of its
// largest value (at most 2^127, which is enough for subnormal ones; `top` is 0
// for them and for zeros), and what undoes it.
__device__ __forceinline__ float scale_of(uint32_t top) {
    return __uint_as_float(min(268u - top, 254u) << 23);
}
__device__ __forceinline__ float unscale_of(uint32_t top) {
    return top < 15u ? __uint_as_float(0x00400000u) : __uint_as_float((top - 14u) << 23);
}

// Tokens m0 .. m0 + toks of rank r, k from t0 to kend, as a tile of `tile_k` k in the order of the tensor
// instruction's operands, with their sums and scales; tokens up to `rows` are written, those that do
// not exist as zeros.  A warp takes a token's 256 k at a time, a unit of 8 k a lane; its (at most UNITS)
// loads are in flight together with those of `between`.
//   xs   : [k / 32][TT][lane] units of 8 k in bf16
//   xsum : [k / GRAIN][TOK] sum x * 2^-24
//   xsc  : [k / 256, or k / xgroup with kFp8][TOK] the tokens' scales
//   bad  : bit m: token m has a value that is not finite
template <int TT, Tokens KIND, int SPAN, int GRAIN, int UNITS, typename Between>
__device__ __forceinline__ void stage_tokens(const QweightParams& p, int r, int m0, int rows, int toks, int t0, int kend,
                                             int tile_k, uint8_t* xs, float* xsum, float* xsc, uint32_t* bad,
                                             Between between) {
    constexpr int TOK = TT * 8;
    const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;  // warp: uniform
    int tokp = 1, toksh = 0;
    while (tokp < rows) tokp <<= 1, ++toksh;
    const int todo = ((tile_k + 255) >> 8) * tokp;  // (256 k, token) rows, the token innermost
    uint4 v[UNITS];
    constexpr int BYTES = KIND == kBf16 ? 2 : 1;
    const uint8_t* from = static_cast<const uint8_t*>(p.x[r]) + ((int64_t)m0 * p.K + t0 + lane * 8) * BYTES;  // (32 rows of K <= 2^20: within 2^31)
#pragma unroll
    for (int j = 0; j < UNITS; ++j) {
        v[j] = make_uint4(0u, 0u, 0u, 0u);
        const int i = warp + j * kWarps, m = i & (tokp - 1), k = (i >> toksh) * 256;
        const bool in = i < todo && m < toks && t0 + lane * 8 + k < kend;
        const uint8_t* at = from + (m * p.K + k) * BYTES;
        if constexpr (KIND == kBf16) {
            ldg_if(v[j], at, in);
        } else {
            uint2 b = make_uint2(0u, 0u);
            ldg_if(b, at, in);
            v[j].x = b.x;
            v[j].y = b.y;
            if (KIND == kFp8Pow2)
                ldg_u8_if(v[j].z, static_cast<const uint8_t*>(p.xscale[r]) + (int64_t)(m0 + m) * p.xgroups + ((t0 + lane * 8 + k) >> p.xgroup_shift), in);
        }
    }
    between();
    // two rows at a time, so that one's steps fill the waits of the other's
#pragma unroll
    for (int j0 = 0; j0 < UNITS; j0 += 2) {
        if (warp + j0 * kWarps >= todo) break;
        float x[2][8], sum[2];  // the even k, 0 2 4 6, times 1; and the odd
        int m[2], k[2];         // k within the tile
        bool in[2];
        uint32_t top[2] = {0u, 0u};
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int i = warp + (j0 + e) * kWarps;
            m[e] = i & (tokp - 1);
            k[e] = (i >> toksh) * 256 + lane * 8;
            in[e] = i < todo && m[e] < rows && k[e] < tile_k;
            uint4& w = v[j0 + e];
            if constexpr (KIND != kBf16) {
                const float2 f[4] = {fp8x2_to_float2(w.x), fp8x2_to_float2(w.x >> 16), fp8x2_to_float2(w.y), fp8x2_to_float2(w.y >> 16)};
#pragma unroll
                for (int i4 = 0; i4 < 4; ++i4) {
                    x[e][i4] = f[i4].x;
                    x[e][4 + i4] = f[i4].y;
                }
            }
            if constexpr (KIND == kFp8) {  // for the sums' unit
#pragma unroll
                for (int i8 = 0; i8 < 8; ++i8) x[e][i8] *= 128.f;
            } else if constexpr (KIND == kFp8Pow2) {
                // The largest value goes to 2^14..2^15, as for bf16, whatever scales the codes of zero are under.
                // `largest`: of the lanes' scale bytes plus biased exponents; within what keeps the factor that undoes it,
                // 2^(largest - 268) * 2^12, a normal number (2^129 and more, which fp32 does not hold, may leave bf16)
                float a = 0.f;
#pragma unroll
                for (int i8 = 0; i8 < 8; ++i8) a = fmaxf(a, fabsf(x[e][i8]));
                const uint32_t own = a == 0.f || w.z == 255u ? 0u : w.z + (__float_as_uint(a) >> 23);
                const int largest = min(max((int)__reduce_max_sync(0xFFFFFFFFu, own), 141), 383);
                // 2^(w.z - 127) * 2^(268 - largest), biased (at most 150 where a code is not zero); a NaN scale
                const int mul = max(min((int)w.z - largest + 268, 150), 0);
#pragma unroll
                for (int i8 = 0; i8 < 8; ++i8) x[e][i8] *= __uint_as_float(w.z == 255u ? 0x7FC00000u : (uint32_t)mul << 23);
                if (lane == 0 && in[e]) xsc[(k[e] >> 8) * TOK + m[e]] = __uint_as_float((uint32_t)(largest - 129) << 23);
            } else {
                top[e] = __vmaxu2(__vmaxu2(w.x & 0x7F807F80u, w.y & 0x7F807F80u), __vmaxu2(w.z & 0x7F807F80u, w.w & 0x7F807F80u));
            }
        }
        if constexpr (KIND == kBf16) {
            // the largest exponents
#pragma unroll
            for (int e = 0; e < 2; ++e) top[e] = __reduce_max_sync(0xFFFFFFFFu, max(top[e] >> 23, top[e] >> 7 & 0xFFu));
            if (top[0] == 255u || top[1] == 255u) {
                // values that are not finite: zeros here, and their tokens are noted
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    if (top[e] != 255u) continue;
                    if (lane == 0) atomicOr(bad, 1u << m[e]);
                    uint32_t* w = &v[j0 + e].x;
                    uint32_t t = 0u;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if ((w[i] & 0x7F800000u) == 0x7F800000u) w[i] &= 0x0000FFFFu;
                        if ((w[i] & 0x00007F80u) == 0x00007F80u) w[i] &= 0xFFFF0000u;
                        t = __vmaxu2(t, w[i] & 0x7F807F80u);
                    }
                    top[e] = __reduce_max_sync(0xFFFFFFFFu, max(t >> 23, t >> 7 & 0xFFu));
                }
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float mul = scale_of(top[e]);
                const uint32_t w[4] = {v[j0 + e].x, v[j0 + e].y, v[j0 + e].z, v[j0 + e].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[e][i] = bf_lo(w[i]) * mul;
                    x[e][4 + i] = bf_hi(w[i]) * mul;
                }
                // (a row's first lane is in the tile wherever the row has a lane in it)
                if (lane == 0 && in[e]) xsc[(k[e] >> 8) * TOK + m[e]] = unscale_of(top[e]) * 0x1p12f;
            }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            // unit u of SPAN k is lane c4's, in step st
            const int u = lane % (SPAN / 8), st = k[e] / SPAN * (SPAN / 32) + u % (SPAN / 32), c4 = u / (SPAN / 32);
            const float(&y)[8] = x[e];
            if (in[e])
                *reinterpret_cast<uint4*>(xs + (((st * TT + (m[e] >> 3)) * 8 + (m[e] & 7)) * 4 + c4) * 16) =
                    make_uint4(bf16x2(y[0] * 0x1p109f, y[2] * 0x1p109f), bf16x2(y[4] * 0x1p105f, y[6] * 0x1p105f),
                               bf16x2(y[1] * 0x1p109f, y[3] * 0x1p109f), bf16x2(y[5] * 0x1p105f, y[7] * 0x1p105f));
            sum[e] = ((y[0] + y[1]) + (y[2] + y[3])) + ((y[4] + y[5]) + (y[6] + y[7]));
        }
        // sum x over each GRAIN of k, in the weights' unit
#pragma unroll
        for (int o = 1; o < GRAIN / 8; o <<= 1)
#pragma unroll
            for (int e = 0; e < 2; ++e) sum[e] += __shfl_xor_sync(0xFFFFFFFFu, sum[e], o);
#pragma unroll
        for (int e = 0; e < 2; ++e)
            if ((lane & (GRAIN / 8 - 1)) == 0 && in[e]) xsum[k[e] / GRAIN * TOK + m[e]] = sum[e] * 0x1p-24f;
    }
    if constexpr (KIND == kFp8) {
        const int x0 = t0 >> p.xgroup_shift;
        for (int u = threadIdx.x; u < (tile_k >> p.xgroup_shift) * TOK; u += kThreads) {
            const int m = u % TOK, gi = u / TOK;
            const bool in = m < toks && x0 + gi < p.xgroups;
            xsc[u] = in ? __ldcg(static_cast<const float*>(p.xscale[r]) + (int64_t)(m0 + m) * p.xgroups + x0 + gi) : 0.f;
        }
    }
}

// The tokens of a launch, staged once for all CTAs that read them: CTA (rank, token tile, 256 k).
template <int TT, Tokens KIND, int STEPS>
__global__ void __launch_bounds__(kThreads) qweight_tokens_kernel(const __grid_constant__ QweightParams p) {
    constexpr int TOK = TT * 8, GRAIN = STEPS * 32;
    __shared__ uint32_t bad;
    if (threadIdx.x == 0) bad = 0u;
    const int chunks = p.kp >> 8, chunk = (int)blockIdx.x % chunks, b = (int)blockIdx.x / chunks;
    const int m0 = b % p.tiles_m * TOK, k0 = chunk * 256;
    // in this order: the kernel that follows knows that all that ran before this one has ended
    ptx::grid_wait();
    ptx::grid_launch_dependents();
    const int fshift = KIND == kFp8 ? p.xgroup_shift : 8;
    stage_tokens<TT, KIND, GRAIN < 64 ? 32 : 64, GRAIN, TT>(
        p, b / p.tiles_m, m0, TOK, min(TOK, p.M - m0), k0, p.K, 256, p.tokens + ((size_t)b * p.kp + k0) * (TOK * 2),
        p.sums + ((size_t)b * p.kp + k0) / GRAIN * TOK, p.scales + (((size_t)b * p.kp + k0) >> fshift) * TOK, &bad,
        [] { __syncthreads(); });
    __syncthreads();
    if (threadIdx.x == 0) p.flags[blockIdx.x] = bad;
}

// Bounded wait for a tile's copies; after a timeout every wait of the CTA returns at once.
__device__ __forceinline__ void tile_wait(uint64_t* bar, uint32_t parity, volatile uint32_t* abort, const QweightParams& p) {
    if (ptx::mbar_try_wait(bar, parity)) return;
    const uint64_t t0 = ptx::globaltimer();
    while (!ptx::mbar_try_wait(bar, parity)) {
        if (*abort) return;
        if (ptx::globaltimer() - t0 > p.timeout_ns) {
            record_error(p.status, ARE_DEV_PIPE_TIMEOUT, blockIdx.x, -6, -1);
            *abort = 1u;
            return;
        }
    }
}

// A group's scale and zero point (0..255: exact in bf16), in a word.
__device__ __forceinline__ uint32_t scale_word(uint32_t scale, uint32_t zero) {
    return scale | (__float_as_uint((float)zero) & 0xFFFF0000u);
}

// 128 k of a warp's rows times the tokens.  A lane reads its codes of a step of 32 k, or of up to four steps that share
// the scales at once, which permutes their k; the tokens are staged in the same order.
//   at    : row g's codes of the first row tile (shared memory), sw its swizzle, BLK the 128 k of them
//   xat   : the lane's token operands
//   words : the lane's row's scale word, of the block's first group; a group's words are `wrows` apart
//   sums, scales: the lane's token pair's, of the block's first row
//   acc   : [row tile][token tile][row g, g + 8] of the token pair
template <int TT, int WSTEPS, int STEPS, int BLK>
__device__ __forceinline__ void products(uint64_t (&acc)[Shape<TT>::RT][TT][2], uint32_t at, uint32_t sw, int c, uint32_t xat, const uint32_t* words,
                                         int wrows, const float* sums, const float* scales, int fshift) {
    using S = Shape<TT>;
    constexpr int TOK = S::TOK, RT = S::RT, PITCH = S::PITCH;
    constexpr bool OWN = S::OWN;
    // Two row tiles take the 128 k in two parts, whose operands fit the registers, and TB token tiles at a time; one
    // takes CH chains of sums: a dependent instruction waits for the one before it.
    constexpr int PARTS = OWN ? 2 : 1, SP = 4 / PARTS, TB = OWN ? 2 : 1, CH = OWN ? 1 : 2;
    constexpr bool KEEP = STEPS > SP;  // a group's sums outlive a part
    float d[KEEP ? TT : TB][RT][CH][4];
#pragma unroll
    for (int part = 0; part < PARTS; ++part) {
        const int s0 = part * SP;
        uint32_t a[RT][SP][2][4];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            uint32_t lo[SP], hi[SP];
            const uint32_t from = at + rt * 16 * PITCH;
            if (STEPS == 4 && SP == 4) {
                const uint32_t o = ((uint32_t)c * 16u ^ sw) ^ (BLK * 64u);
                const uint4 l4 = ld_shared_v4(from + o), h4 = ld_shared_v4(from + 8 * PITCH + o);
                lo[0] = l4.x; lo[1] = l4.y; lo[SP - 2] = l4.z; lo[SP - 1] = l4.w;
                hi[0] = h4.x; hi[1] = h4.y; hi[SP - 2] = h4.z; hi[SP - 1] = h4.w;
            } else if (STEPS >= 2) {
#pragma unroll
                for (int st = 0; st < SP; st += 2) {
                    const uint32_t o = (((uint32_t)c / 2u * 16u ^ sw) ^ (BLK * 64u + (s0 + st) / 2 * 32u)) + (uint32_t)c % 2u * 8u;
                    const uint2 l2 = ld_shared_v2(from + o), h2 = ld_shared_v2(from + 8 * PITCH + o);
                    lo[st] = l2.x; lo[st + 1] = l2.y;
                    hi[st] = h2.x; hi[st + 1] = h2.y;
                }
            } else {
#pragma unroll
                for (int st = 0; st < SP; ++st) {
                    const uint32_t o = (sw ^ (BLK * 64u + (s0 + st) * 16u)) + (uint32_t)c * 4u;
                    lo[st] = ld_shared(from + o);
                    hi[st] = ld_shared(from + 8 * PITCH + o);
                }
            }
#pragma unroll
            for (int st = 0; st < SP; ++st) {
                codes8<0>(lo[st], a[rt][st][0], a[rt][st][1]);
                codes8<1>(hi[st], a[rt][st][0], a[rt][st][1]);
            }
        }
        // the scales and negated zero points of the rows' groups that end in this part, once for all tokens, in pairs
        constexpr int WG = SP / WSTEPS > 0 ? SP / WSTEPS : 1;
        uint64_t ws[WG][RT][2], wz[WG][RT][2];
        if ((s0 + SP) % WSTEPS == 0 || STEPS <= SP) {
#pragma unroll
            for (int i = 0; i < WG; ++i)
#pragma unroll
                for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const uint32_t word = words[(s0 / WSTEPS + i) * wrows + rt * 16 + half * 8];
                        ws[i][rt][half] = pair(__uint_as_float(word << 16), __uint_as_float(word << 16));
                        const float z = __uint_as_float((word & 0xFFFF0000u) ^ 0x80000000u);
                        wz[i][rt][half] = pair(z, z);
                    }
        }
#pragma unroll
        for (int tb = 0; tb < TT; tb += TB) {
            uint4 b[TB][SP];
#pragma unroll
            for (int st = 0; st < SP; ++st)
#pragma unroll
                for (int t = 0; t < TB; ++t) b[t][st] = ld_shared_v4(xat + ((s0 + st) * TT + tb + t) * 512);
#pragma unroll
            for (int st = 0; st < SP; ++st) {
#pragma unroll
                for (int t = 0; t < TB; ++t)
#pragma unroll
                    for (int rt = 0; rt < RT; ++rt) {
                        float(&to)[CH][4] = d[KEEP ? tb + t : t][rt];
                        const bool first = (s0 + st) % STEPS == 0;
                        if (first) mma<true>(to[0], a[rt][st][0], b[t][st].x, b[t][st].y);
                        else mma<false>(to[0], a[rt][st][0], b[t][st].x, b[t][st].y);
                        if (CH == 2 && first) mma<true>(to[CH - 1], a[rt][st][1], b[t][st].z, b[t][st].w);
                        else mma<false>(to[CH - 1], a[rt][st][1], b[t][st].z, b[t][st].w);
                    }
                if ((s0 + st) % STEPS != STEPS - 1) continue;
#pragma unroll
                for (int t = 0; t < TB; ++t) {
                    const int tok = (tb + t) * 8;
                    const uint64_t sum = *reinterpret_cast<const uint64_t*>(sums + (s0 + st) / STEPS * TOK + tok);
                    const uint64_t f = *reinterpret_cast<const uint64_t*>(scales + ((s0 + st) * 32 >> fshift) * TOK + tok);
#pragma unroll
                    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            const uint64_t sc = ws[st / WSTEPS][rt][half], z = wz[st / WSTEPS][rt][half];
                            const float(&d2)[CH][4] = d[KEEP ? tb + t : t][rt];
                            uint64_t y = pair(d2[0][half * 2], d2[0][half * 2 + 1]);
                            if (CH == 2) y = add2(y, pair(d2[CH - 1][half * 2], d2[CH - 1][half * 2 + 1]));
                            uint64_t& e = acc[rt][tb + t][half];
                            e = fma2(mul2(sc, f), fma2(z, sum, y), e);
                        }
                }
            }
        }
    }
}

// Adds the cluster's sums, r ascending, and writes the outputs.  red: [slot_of(group)][rtoks][LD]; bad: tokens
// of this CTA's K range that hold a value that is not finite, whose products are added here.
template <int TT, bool NOTED, typename Slot>
__device__ __forceinline__ void combine(const QweightParams& p, int q, int m0, int toks, int group0, int groups,
                                        const float* red, const uint32_t* bad, Slot slot_of) {
    constexpr int ROWS = Shape<TT>::ROWS, LD = Shape<TT>::LD;
    __syncwarp();
    ptx::cluster_sync();
    constexpr int PAIRS = ROWS / 2;  // pairs of rows of a group
    const uint32_t base = ptx::smem_u32(red), bad_addr = ptx::smem_u32(bad);
    uint32_t any = 0u;
    if (NOTED) {
#pragma unroll
        for (int j = 0; j < kMaxRanks; ++j)
            if (j < p.cluster) any |= ld_cluster(ptx::mapa_shared(bad_addr, (uint32_t)j));
    }
    // the cluster's threads take the (token, group, pair) in turn
    for (int u = q * kThreads + threadIdx.x; u < groups * PAIRS * toks; u += p.cluster * kThreads) {
        const int pair = u % PAIRS, a = u / PAIRS % groups, m = u / PAIRS / groups;
        const int n = (group0 + a) * ROWS + pair * 2;
        if (n < p.N) {
            const uint32_t addr = base + (uint32_t)((slot_of(a) * p.rtoks + m) * LD + pair * 2) * 4u;
            float2 s = make_float2(0.f, 0.f);
#pragma unroll
            for (int j = 0; j < kMaxRanks; ++j) {
                if (j < p.cluster) {
                    const float2 v = ld_cluster_f2(ptx::mapa_shared(addr, (uint32_t)j));
                    s.x += v.x;
                    s.y += v.y;
                }
            }
            if (NOTED && (any >> m & 1u)) {  // products of values that are not finite
                for (int j = 0; j < p.cluster; ++j) {
                    const int rj = j / p.splits, k0 = j % p.splits * p.split_k, k1 = min(p.K, k0 + p.split_k);
                    const int64_t row = (int64_t)(m0 + m) * p.K;
                    for (int k = k0; k < k1; ++k) {
                        const float xv = __uint_as_float((uint32_t)__ldcg(static_cast<const uint16_t*>(p.x[rj]) + row + k) << 16);
                        if ((__float_as_uint(xv) & 0x7F800000u) != 0x7F800000u) continue;
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int64_t at = (int64_t)(n + i) * p.groups + (k >> p.group_shift);
                            const uint32_t byte = p.codes[rj][((int64_t)(n + i) * p.K + k) >> 1];
                            const int u = (int)(k & 1 ? byte >> 4 : byte & 15u), z = p.zero[rj] ? p.zero[rj][at] : 8;
                            const float w = (float)(u - z) * __uint_as_float((uint32_t)p.scale[rj][at] << 16);
                            (i ? s.y : s.x) += xv * w;
                        }
                    }
                }
            }
            const __nv_bfloat162 o = __floats2bfloat162_rn(s.x, s.y);
            for (int v = 0; v < p.nviews; ++v)
                *reinterpret_cast<__nv_bfloat162*>(p.views[v] + (int64_t)(m0 + m) * p.N + n) = o;
        }
    }
    __syncwarp();
    ptx::cluster_sync();  // no CTA leaves while another reads its sums
}

// Up to 8 tokens a tile.
// fp32 token scales (QX) are applied with the weights'; power-of-two scales go
// into the staged tokens.
// WSTEPS: steps of 32 k in a weight group; STEPS: those that share both scales,
// the smaller of the weight and the token group.
template <Tokens KIND, int WSTEPS, int STEPS>
__global__ void __launch_bounds__(kThreads, 2) qweight_few_kernel(const __grid_constant__ QweightParams p) {
    extern __shared__ __align__(128) uint8_t qw_smem[];
    constexpr int TT = 1;
    constexpr bool QX = KIND == kFp8;
    using S = Shape<TT>;
    constexpr int TOK = S::TOK, ROWS = S::ROWS, ITEM = S::ITEM, PITCH = S::PITCH, LD = S::LD;
    constexpr int SLOT = S::SLOT, DEPTH = S::DEPTH, UNITS = S::UNITS;
    constexpr int GRAIN = STEPS * 32;       // k that share both scales
    // What the sums lack of 2^24 (the codes' 2^-133 times the tokens' 2^109): 2^12 of it is in the staged scales, or 2^7 in
    // the tokens.  So outputs down to bf16's smallest normal ones keep bits enough in fp32 sums.
    constexpr float UNIT = QX ? 0x1p17f : 0x1p12f;
    const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;  // warp: uniform
    const int g = lane >> 2, c = lane & 3;
    const int q = (int)(blockIdx.x % p.cluster);
    const int tile = (int)(blockIdx.x / p.cluster);
    const int m0 = tile % p.tiles_m * TOK, group0 = tile / p.tiles_m * p.run;
    const int groups = min(p.run, (p.N + ROWS - 1) / ROWS - group0);  // of ROWS rows
    const int r = q / p.splits;
    const int kbeg = q % p.splits * p.split_k, kend = min(p.K, kbeg + p.split_k);  // never empty
    const int tiles = (kend - kbeg + p.tile_k - 1) / p.tile_k;
    const int toks = min(TOK, p.M - m0);

    const uint32_t ring = ptx::smem_u32(qw_smem) + warp * (DEPTH * SLOT);
    const int fshift = QX ? p.xgroup_shift : 8, frows = QX ? p.tile_k >> fshift : (p.tile_k + 255) >> 8;
    const int wrows = p.run * ROWS + 1;                              // odd: a row's groups fall into different banks
    uint8_t* xs = qw_smem + S::RING;                                 // as stage_tokens writes them
    float* xsum = reinterpret_cast<float*>(xs + 2 * TOK * p.tile_k);
    float* xsc = xsum + p.tile_k / GRAIN * TOK;
    uint32_t* wsc = reinterpret_cast<uint32_t*>(xsc + frows * TOK);  // [k >> group][wrows]: scale | zero point << 16, in bf16
    uint32_t* bad = wsc + (((p.tile_k >> p.group_shift) * wrows + 3) & ~3);
    float* red = reinterpret_cast<float*>(bad + 4);                       // [group + warp][rtoks][LD]

    // this warp's items of a K tile: [first, first + count), item = group * per + K index
    const int per = p.tile_k / ITEM, all = groups * per;
    const int first = warp * all / kWarps;
    const int count = (warp + 1) * all / kWarps - first;

    // ---- the stream of codes, DEPTH - 1 items ahead of their use, by asynchronous copies.  N is a
    // multiple of 8: 8 rows exist or not.
    constexpr int LPR = ITEM / 32, RPI = 32 / LPR, CP = ROWS / RPI;  // lanes a row of codes, rows an instruction, instructions
    const int64_t rstep = (int64_t)RPI * (p.K >> 1);
    const int64_t lane_off = (int64_t)(lane / LPR) * (p.K >> 1) + lane % LPR * 16;
    const uint32_t lane_to = (uint32_t)(lane / LPR * PITCH) + ((uint32_t)(lane % LPR * 16) ^ swizzle<PITCH>(lane / LPR));
    static_assert(RPI == 4, "a row 4 further has the lowest bit of its swizzle the other way");
    const uint8_t* fcodes = nullptr;
    int ftl = -1, fleft = 0, fkk = 0, fgl = 0, fk = 0, fn = 0;
    auto seek = [&]() {  // group fgl, K index fkk of tile ftl
        const int n = (group0 + fgl) * ROWS;
        fk = kbeg + ftl * p.tile_k + fkk * ITEM;
        fn = p.N - n;
        fcodes = p.codes[r] + (((int64_t)n * p.K + fk) >> 1) + lane_off;
    };
    auto fetch = [&](uint32_t slot) {
        if (fleft == 0) {
            if (count > 0 && ftl + 1 < tiles) {
                ++ftl;
                fleft = count;
                fgl = first / per;
                fkk = first % per;
                seek();
            } else {
                cp_commit();
                return;
            }
        }
        const uint32_t to = slot + lane_to;
        if (fn >= ROWS && fk + ITEM <= kend) {
#pragma unroll
            for (int j = 0; j < CP; ++j) cp_async16((to ^ (j & 1) * 16u) + j * RPI * PITCH, fcodes + j * rstep);
        } else {  // rows or K that end within the item: zeros
            const bool kin = fk + lane % LPR * 32 < kend;
#pragma unroll
            for (int j = 0; j < CP; ++j) {
                const bool in = kin && j * RPI < fn;
                cp_async16((to ^ (j & 1) * 16u) + j * RPI * PITCH, in ? fcodes + j * rstep : p.codes[r], in);
            }
        }
        cp_commit();
        fk += ITEM;
        fcodes += ITEM / 2;
        --fleft;
        if (++fkk == per) {
            fkk = 0;
            ++fgl;
            seek();
        }
    };

    if (threadIdx.x == 0) *bad = 0u;
    if (toks < TOK) {  // tokens that do not exist: zeros, which no tile overwrites
        for (int u = threadIdx.x; u < TOK * p.tile_k / 8; u += kThreads)
            *reinterpret_cast<uint4*>(xs + u * 16) = make_uint4(0u, 0u, 0u, 0u);
        for (int u = threadIdx.x; u < p.tile_k / GRAIN * TOK; u += kThreads) xsum[u] = 0.f;
        for (int u = threadIdx.x; u < frows * TOK; u += kThreads) xsc[u] = 0.f;
    }
    ptx::grid_launch_dependents();
    ptx::grid_wait();
#pragma unroll
    for (int i = 0; i < DEPTH - 1; ++i) fetch(ring + i * SLOT);

    // The rows' scales and zero points: neighbouring lanes take a row's neighbouring groups (lanes on rows
    // of their own would touch a sector each with every load); what does not exist weighs nothing.
    const bool zeros = p.zero[r] != nullptr;
    const int tg = p.tile_k >> p.group_shift;
    int tsh = 0;
    while (1 << tsh < tg) ++tsh;
    // a thread's group of the tile is fixed; its rows are wstep apart
    const int wgi = threadIdx.x & ((1 << tsh) - 1), wrow = threadIdx.x >> tsh, wstep = kThreads >> tsh;
    const int wleft = min(p.run * ROWS, p.N - group0 * ROWS);
    const int64_t wbase = (int64_t)group0 * ROWS * p.groups;  // the same for the CTA; its rows' offsets fit 32 bits
    const int wat = wrow * p.groups + wgi, wjump = wstep * p.groups;
    constexpr int WUNITS = 16;  // of a round
    uint32_t sv[WUNITS], zv[WUNITS];
    auto load_scales = [&](int t0, int round) {
        const bool on = wgi < tg && (t0 >> p.group_shift) + wgi < p.groups;
        const int at = wat + (t0 >> p.group_shift) + round * WUNITS * wjump;
        const uint16_t* sp = p.scale[r] + wbase + at;
        const uint8_t* zp = p.zero[r] + wbase + at;
#pragma unroll
        for (int j = 0; j < WUNITS; ++j) {
            const bool in = on && wrow + (round * WUNITS + j) * wstep < wleft;
            sv[j] = 0u;
            zv[j] = 8u;
            ldg_u16_if(sv[j], sp, in);
            ldg_u8_if(zv[j], zp, in && zeros);
            sp += wjump;
            zp += wjump;
        }
    };
    auto store_scales = [&](int t0) {
        for (int round = 0; round * WUNITS * wstep < p.run * ROWS; ++round) {
            if (round) load_scales(t0, round);
            uint32_t* to = wsc + wgi * wrows + wrow + round * WUNITS * wstep;
#pragma unroll
            for (int j = 0; j < WUNITS; ++j)
                if (wgi < tg && wrow + (round * WUNITS + j) * wstep < p.run * ROWS) to[j * wstep] = scale_word(sv[j], zv[j]);
        }
    };
    auto stage = [&](int tl) {
        const int t0 = kbeg + tl * p.tile_k;
        stage_tokens<TT, KIND, GRAIN, GRAIN, UNITS>(p, r, m0, toks, toks, t0, kend, p.tile_k, xs, xsum, xsc, bad, [&] {
            load_scales(t0, 0);  // in flight with the tokens
            __syncthreads();     // every warp is done with the tile before (first: with clearing)
        });
        store_scales(t0);
        __syncthreads();
    };
    uint64_t acc[1][TT][2];
#pragma unroll
    for (int t = 0; t < TT; ++t)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[0][t][j] = 0ull;
    const uint32_t xs_addr = ptx::smem_u32(xs) + lane * 16u, sw = swizzle<PITCH>(g);
    uint32_t cur = ring;
    const uint32_t ring_end = ring + DEPTH * SLOT;
#pragma unroll 1
    for (int tl = 0; tl < tiles; ++tl) {
        stage(tl);
        const int ktile = kbeg + tl * p.tile_k;
        int gl = first / per, kk = first % per;
#pragma unroll 1
        for (int left = count; left > 0; --left) {
            cp_wait<DEPTH - 2>();
            __syncwarp();  // every lane's copies have landed, and every lane has left the slot refilled now
            const uint32_t next = cur + SLOT == ring_end ? ring : cur + SLOT;
            fetch(cur == ring ? ring_end - SLOT : cur - SLOT);  // the slot before
            const uint32_t at = cur + g * PITCH;
            cur = next;
            if (ktile + kk * ITEM < kend) {
                auto block = [&](auto blk) {
                    constexpr int BLK = decltype(blk)::value;
                    const int kt = kk * ITEM + BLK * 128;  // within the tile
                    products<TT, WSTEPS, STEPS, BLK>(acc, at, sw, c, xs_addr + (uint32_t)((kt >> 5) * TT * 512),
                                                     wsc + (kt >> p.group_shift) * wrows + gl * ROWS + g, wrows,
                                                     xsum + kt / GRAIN * TOK + 2 * c, xsc + (kt >> fshift) * TOK + 2 * c, fshift);
                };
                block(std::integral_constant<int, 0>());
                block(std::integral_constant<int, 1>());
            }
            if (++kk == per || left == 1) {
                // the warp leaves a group: its sums go to the slot of (group, warp), which no other
                // warp touches; along a CTA's items either index grows, so group + warp is unique
                float* to = red + (gl + warp) * p.rtoks * LD + g;
#pragma unroll
                for (int t = 0; t < TT; ++t) {
                    float* e = to + (t * 8 + 2 * c) * LD;
                    const float2 v01 = unpair(acc[0][t][0]), v23 = unpair(acc[0][t][1]);
                    const float v[4] = {v01.x, v01.y, v23.x, v23.y};
                    if (t * 8 + 2 * c >= p.rtoks) {
                    } else if (tl == 0) {
                        e[0] = v[0] * UNIT; e[LD] = v[1] * UNIT; e[8] = v[2] * UNIT; e[LD + 8] = v[3] * UNIT;
                    } else {
                        e[0] = fmaf(v[0], UNIT, e[0]); e[LD] = fmaf(v[1], UNIT, e[LD]);
                        e[8] = fmaf(v[2], UNIT, e[8]); e[LD + 8] = fmaf(v[3], UNIT, e[LD + 8]);
                    }
                    acc[0][t][0] = acc[0][t][1] = 0ull;
                }
                kk = 0;
                ++gl;
            }
        }
    }
    cp_wait<0>();
    __syncthreads();

    // ---- the sums: of a group over the CTA's warps (into the slot of its first warp), then over the
    // cluster, r ascending.  Item i belongs to warp (8 (i + 1) - 1) / all.
    auto slot_of = [&](int a) { return a + (kWarps * (a * per + 1) - 1) / all; };
    for (int a = warp; a < groups; a += kWarps) {
        const int s0 = slot_of(a), w0 = s0 - a, w1 = (kWarps * (a * per + per) - 1) / all;
        for (int w = w0 + 1; w <= w1; ++w) {
            if ((w + 1) * all / kWarps == w * all / kWarps) continue;  // a warp without items
            for (int m = lane >> 4; m < toks; m += 2)
                red[(s0 * p.rtoks + m) * LD + (lane & 15)] += red[((a + w) * p.rtoks + m) * LD + (lane & 15)];
        }
    }
    combine<TT, KIND == kBf16>(p, q, m0, toks, group0, groups, red, bad, slot_of);
}

// Tiles of 16 or 32 tokens: a warp owns 32 rows.  The staged tokens come in tiles of K by bulk copies, the
// weights' scales with plain loads spread over the items of the tile before, both a tile ahead.
template <int TT, bool QX, int WSTEPS, int STEPS>
__global__ void __launch_bounds__(kThreads, 2) qweight_wide_kernel(const __grid_constant__ QweightParams p) {
    extern __shared__ __align__(128) uint8_t qw_smem[];
    using S = Shape<TT>;
    using W = Wide<TT, QX, WSTEPS, STEPS>;
    constexpr int TOK = S::TOK, RT = S::RT, ROWS = S::ROWS, ITEM = S::ITEM, PITCH = S::PITCH, LD = S::LD;
    constexpr int SLOT = S::SLOT, DEPTH = S::DEPTH, TILE = W::TILE, PER = TILE / ITEM, WROWS = W::WROWS;
    constexpr int GRAIN = STEPS * 32;       // k that share both scales
    constexpr float UNIT = QX ? 0x1p17f : 0x1p12f;  // as in qweight_few_kernel
    const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;  // warp: uniform
    const int g = lane >> 2, c = lane & 3;
    const int q = (int)(blockIdx.x % p.cluster);
    const int tile = (int)(blockIdx.x / p.cluster);
    const int m0 = tile % p.tiles_m * TOK, group0 = tile / p.tiles_m * kWarps;
    const int groups = min(kWarps, (p.N + ROWS - 1) / ROWS - group0);
    const int r = q / p.splits;
    const int kbeg = q % p.splits * p.split_k, kend = min(p.K, kbeg + p.split_k);  // never empty
    const int tiles = (kend - kbeg + TILE - 1) / TILE;
    const bool active = warp < groups;

    const uint32_t ring = ptx::smem_u32(qw_smem) + warp * (DEPTH * SLOT);
    const int fshift = QX ? p.xgroup_shift : 8;
    uint8_t* xs = qw_smem + S::RING;                                      // [buffer] as stage_tokens writes them
    float* xsum = reinterpret_cast<float*>(xs + 2 * W::XS);
    float* xsc = xsum + 2 * W::XSUM;
    uint32_t* wsc = reinterpret_cast<uint32_t*>(xsc + 2 * W::XSC);        // [buffer][group][WROWS]: scale | zero point << 16, in bf16
    uint32_t* bad = wsc + 2 * W::WSC;
    volatile uint32_t* abort = bad + 1;                                   // a wait has run out
    uint32_t* left = bad + 2;                                             // by buffer: warps that have left a tile, of all so far
    uint64_t* full = reinterpret_cast<uint64_t*>(bad + 4);                // a buffer's copies have landed
    float* red = reinterpret_cast<float*>(qw_smem);                       // the ring's place, when the products are done

    // the stream of codes, DEPTH - 1 items ahead of their use
    constexpr int LPR = ITEM / 32, RPI = 32 / LPR, CP = ROWS / RPI;  // lanes a row of codes, rows an instruction, instructions
    const int frow = (group0 + warp) * ROWS, fn = p.N - frow;
    const int rstep = RPI * (p.K >> 1);                              // p.K <= 2^20: a warp's rows are within 2^31 of each other
    int fk = kbeg;
    const uint8_t* fcodes = p.codes[r] + (((int64_t)frow * p.K + kbeg) >> 1) + lane / LPR * (p.K >> 1) + lane % LPR * 16;
    const uint32_t lane_to = (uint32_t)(lane / LPR * PITCH) + ((uint32_t)(lane % LPR * 16) ^ swizzle<PITCH>(lane / LPR));
    static_assert(RPI == 8, "a row 8 further has the same swizzle");
    auto fetch = [&](uint32_t slot) {
        if (active && fk < kend) {
            const uint32_t to = slot + lane_to;
            if (fn >= ROWS && fk + ITEM <= kend) {
#pragma unroll
                for (int j = 0; j < CP; ++j) cp_async16(to + j * RPI * PITCH, fcodes + (int64_t)j * rstep);
            } else {  // rows (8 exist or not: N is a multiple of 8) or K that end within the item: zeros
                const bool kin = fk + lane % LPR * 32 < kend;
#pragma unroll
                for (int j = 0; j < CP; ++j) {
                    const bool in = kin && j * RPI < fn;
                    cp_async16(to + j * RPI * PITCH, in ? fcodes + (int64_t)j * rstep : p.codes[r], in);
                }
            }
            fk += ITEM;
            fcodes += ITEM / 2;
        }
        cp_commit();
    };

    // a tile of the staged tokens, by one thread: the first two at the start, then by the warp that is the last
    // to leave the tile two before
    const int b = r * p.tiles_m + tile % p.tiles_m;
    auto copy_tile = [&](int tl) {
        const int t0 = kbeg + tl * TILE, kl = min(TILE, min(kbeg + p.split_k, p.kp) - t0), buf = tl & 1;
        const size_t at = (size_t)b * p.kp + t0;
        const uint32_t nx = (uint32_t)kl * (TOK * 2), ns = (uint32_t)(kl / GRAIN) * (TOK * 4), nf = (uint32_t)(kl >> fshift) * (TOK * 4);
        ptx::mbar_arrive_expect_tx(&full[buf], nx + ns + nf);
        ptx::bulk_load(xs + buf * W::XS, p.tokens + at * (TOK * 2), nx, &full[buf]);
        ptx::bulk_load(xsum + buf * W::XSUM, p.sums + at / GRAIN * TOK, ns, &full[buf]);
        ptx::bulk_load(xsc + buf * W::XSC, p.scales + (at >> fshift) * TOK, nf, &full[buf]);
    };

    // The scales and zero points of the warp's rows in a tile, STEP rows apart, NE of them with an item: neighbouring
    // lanes take a row's neighbouring groups; what does not exist weighs nothing.
    constexpr int TG = TILE / (WSTEPS * 32), STEP = 32 / TG, NE = TG / PER;
    static_assert(ROWS == 32 && NE * PER == TG, "an item's share of the scales");
    const bool zeros = p.zero[r] != nullptr;
    const int wgi = lane % TG, wrow = lane / TG;
    const int64_t wbase = (int64_t)frow * p.groups;  // the warp's rows are within 2^31 of it
    uint32_t sv[NE], zv[NE];
    auto load_scales = [&](int tl, int kk) {
        const int gi = (kbeg + tl * TILE) / (WSTEPS * 32) + wgi;
#pragma unroll
        for (int j = 0; j < NE; ++j) {
            const int row = wrow + (kk * NE + j) * STEP;
            const int64_t at = wbase + (row * p.groups + gi);
            const bool in = gi < p.groups && row < fn;
            sv[j] = 0u;
            zv[j] = 8u;
            ldg_u16_if(sv[j], p.scale[r] + at, in);
            ldg_u8_if(zv[j], p.zero[r] + at, in && zeros);
        }
    };
    uint32_t* wto = wsc + wgi * WROWS + warp * ROWS + wrow;
    auto store_scales = [&](int tl, int kk) {
#pragma unroll
        for (int j = 0; j < NE; ++j) wto[(tl & 1) * W::WSC + (kk * NE + j) * STEP] = scale_word(sv[j], zv[j]);
    };

    if (threadIdx.x == 0) {
        *bad = 0u;
        left[0] = left[1] = 0u;
        *abort = 0u;
        ptx::mbar_init(&full[0], 1);
        ptx::mbar_init(&full[1], 1);
        ptx::fence_mbar_init();
        ptx::fence_proxy_async_shared();
    }
    ptx::grid_launch_dependents();
    // The kernel before is the one that stages the tokens, and lets this one start when all that ran before it has
    // ended: the weights can be read, the tokens after the wait.
#pragma unroll
    for (int i = 0; i < DEPTH - 1; ++i) fetch(ring + i * SLOT);
    for (int kk = 0; kk < PER; ++kk) {
        load_scales(0, kk);
        store_scales(0, kk);
    }
    ptx::grid_wait();
    __syncthreads();  // the barriers and `bad`
    if (threadIdx.x == 0) {
        ptx::fence_proxy_async_global();
        copy_tile(0);
        if (tiles > 1) copy_tile(1);
    }
    if (!QX) {
        const int chunks = ((kend + 255) >> 8) - (kbeg >> 8);
        for (int i = threadIdx.x; i < chunks; i += kThreads) {
            const uint32_t v = __ldcg(p.flags + (size_t)b * (p.kp >> 8) + (kbeg >> 8) + i);
            if (v) atomicOr(bad, v);
        }
    }

    uint64_t acc[RT][TT][2];
#pragma unroll
    for (int a = 0; a < RT; ++a)
#pragma unroll
        for (int t = 0; t < TT; ++t)
#pragma unroll
            for (int j = 0; j < 2; ++j) acc[a][t][j] = 0ull;
    const uint32_t xs_addr = ptx::smem_u32(xs) + lane * 16u, sw = swizzle<PITCH>(g);
    const uint32_t* words = wsc + warp * ROWS + g;
    const float *sums = xsum + 2 * c, *scales = xsc + 2 * c;
    uint32_t cur = ring;
    const uint32_t ring_end = ring + DEPTH * SLOT;
#pragma unroll 1
    for (int tl = 0; tl < tiles; ++tl) {
        const int buf = tl & 1;
        tile_wait(&full[buf], (uint32_t)(tl >> 1) & 1u, abort, p);
        const bool more = tl + 1 < tiles;
#pragma unroll(TT == 2 ? PER : 1)
        for (int kk = 0; kk < PER; ++kk) {
            if (more) load_scales(tl + 1, kk);
            cp_wait<DEPTH - 2>();
            __syncwarp();  // every lane's copies have landed, its scales are stored, and it has left the slot refilled now
            const uint32_t next = cur + SLOT == ring_end ? ring : cur + SLOT;
            fetch(cur == ring ? ring_end - SLOT : cur - SLOT);  // the slot before
            if (active && kbeg + tl * TILE + kk * ITEM < kend)
                products<TT, WSTEPS, STEPS, 0>(acc, cur + g * PITCH, sw, c,
                                            xs_addr + (uint32_t)(buf * W::XS + kk * (4 * TT * 512)),
                                            words + buf * W::WSC + kk * (4 / WSTEPS * WROWS), WROWS,
                                            sums + buf * W::XSUM + kk * (4 / STEPS * TOK),
                                            scales + buf * W::XSC + (kk * ITEM >> fshift) * TOK, fshift);
            cur = next;
            if (more) store_scales(tl + 1, kk);
        }
        // a warp is at most a tile ahead of another (its next tile's copies start when all have left this one), so
        // the count of this tile is whole before one of the next but one begins
        __syncwarp();
        if (lane == 0 && tl + 2 < tiles && !*abort && atom_add_acq_rel(&left[buf]) % kWarps == kWarps - 1) copy_tile(tl + 2);
    }
    cp_wait<0>();
    __syncthreads();
    if (threadIdx.x == 0 && *abort) {  // the CTA must not end before its copies have landed
        const int n = min(tiles, (int)(left[0] / kWarps + left[1] / kWarps) + 2);
        for (int tl = max(n - 2, 0); tl < n; ++tl) {
            const uint64_t t0 = ptx::globaltimer();
            while (!ptx::mbar_try_wait(&full[tl & 1], (uint32_t)(tl >> 1) & 1u))
                if (ptx::globaltimer() - t0 > p.timeout_ns) break;
        }
    }
    if (active) {
        float* to = red + warp * p.rtoks * LD + g;
#pragma unroll
        for (int t = 0; t < TT; ++t) {
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                if (t * 8 + 2 * c >= p.rtoks) break;
                float* e = to + (t * 8 + 2 * c) * LD + rt * 16;
                const float2 v01 = unpair(acc[rt][t][0]), v23 = unpair(acc[rt][t][1]);
                e[0] = v01.x * UNIT; e[LD] = v01.y * UNIT;
                e[8] = v23.x * UNIT; e[LD + 8] = v23.y * UNIT;
            }
        }
    }
    combine<TT, !QX>(p, q, m0, min(TOK, p.M - m0), group0, groups, red, bad, [](int a) { return a; });
}

typedef void (*Kernel)(QweightParams);

// A launch's kernel and the shared memory that it takes (0: by its sizes).
struct Choice {
    Kernel kernel;
    size_t smem;
};
template <int TT, Tokens KIND, int WSTEPS, int STEPS>
Choice choice() {
    constexpr bool QX = KIND == kFp8;  // (wide tiles: the staged bf16 and power-of-two tokens look alike)
    if constexpr (TT == 1) return {qweight_few_kernel<KIND, WSTEPS, STEPS>, 0};
    else return {qweight_wide_kernel<TT, QX, WSTEPS, STEPS>, Wide<TT, QX, WSTEPS, STEPS>::SMEM};
}
template <int TT, Tokens KIND, int WSTEPS>
Choice kernel_of(int steps) {
    if constexpr (KIND != kFp8 || WSTEPS == 1) return choice<TT, KIND, WSTEPS, WSTEPS>();
    else if constexpr (WSTEPS == 2) return steps == 1 ? choice<TT, KIND, 2, 1>() : choice<TT, KIND, 2, 2>();
    else return steps == 1 ? choice<TT, KIND, 4, 1>() : steps == 2 ? choice<TT, KIND, 4, 2>() : choice<TT, KIND, 4, 4>();
}
template <int TT, Tokens KIND>
Choice kernel_of(int wsteps, int steps) {
    return wsteps == 1 ? kernel_of<TT, KIND, 1>(steps) : wsteps == 2 ? kernel_of<TT, KIND, 2>(steps) : kernel_of<TT, KIND, 4>(steps);
}
template <int TT>
Choice kernel_of(Tokens kind, int wsteps, int steps) {
    return kind == kBf16 ? kernel_of<TT, kBf16>(wsteps, steps) : kind == kFp8 ? kernel_of<TT, kFp8>(wsteps, steps) : kernel_of<TT, kFp8Pow2>(wsteps, steps);
}
// The kernel of a token tile and of the groups' sizes in steps of 32; steps <= wsteps.
Choice kernel_of(int tt, Tokens kind, int wsteps, int steps) {
    return tt == 1 ? kernel_of<1>(kind, wsteps, steps) : tt == 2 ? kernel_of<2>(kind, wsteps, steps) : kernel_of<4>(kind, wsteps, steps);
}

// The kernel that stages the tokens for it (TT >= 2).
template <int TT, Tokens KIND>
Kernel tokens_kernel_of(int steps) {
    return steps == 1 ? qweight_tokens_kernel<TT, KIND, 1> : steps == 2 ? qweight_tokens_kernel<TT, KIND, 2> : qweight_tokens_kernel<TT, KIND, 4>;
}
template <int TT>
Kernel tokens_kernel_of(Tokens kind, int steps) {
    return kind == kBf16 ? tokens_kernel_of<TT, kBf16>(steps) : kind == kFp8 ? tokens_kernel_of<TT, kFp8>(steps) : tokens_kernel_of<TT, kFp8Pow2>(steps);
}
Kernel tokens_kernel_of(int tt, Tokens kind, int steps) {
    return tt == 2 ? tokens_kernel_of<2>(kind, steps) : tokens_kernel_of<4>(kind, steps);
}

void cluster_config(cudaLaunchConfig_t& cfg, cudaLaunchAttribute (&attr)[2], int cluster, size_t smem) {
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)cluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    // the kernel comes up while the one before it runs out, and waits for its end (grid_wait)
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
}

struct HostShape {
    int rows, item, ring, ld, units;
};
template <int TT>
HostShape host_shape() {
    using S = Shape<TT>;
    return {S::ROWS, S::ITEM, S::RING, S::LD, S::UNITS};
}

HostShape host_shape(int tt) { return tt == 1 ? host_shape<1>() : tt == 2 ? host_shape<2>() : host_shape<4>(); }

// How a launch over p.M tokens in tiles of 8 tt is cut, and what it is expected to cost, in items of 2 KB of codes.
struct Cut {
    int splits, split_k, run;
    int64_t cost;
};

// Splits of a rank's K (of whole 256 k): of what the busiest CTA does one after the other, its items, its start and
// end, and a little for each CTA more that the cluster adds up.
//  * tt = 1: items of 16 rows x 256 k, the run's by all warps; staging a token's 256 k costs as half an item.
//    (R = 1, 4096 x 4096, 8 tokens: 8.2 us in clusters of 8; 14.8 without a split, each CTA staging all of K.)
//  * tt = 2, 4: items of 32 rows x 128 k, a warp each; one with 32 tokens takes 15/8 as long as with 16.
//    (R = 8, 7168 x 2048: 23 us a launch of one wave with 16, 38 with 32.)
Cut cut_of(const QweightParams& p, const QweightDevice& dev, int tt) {
    const HostShape shape = host_shape(tt);
    const bool own = tt >= 2;
    const int64_t groups = (p.N + shape.rows - 1) / shape.rows, tiles_m = (p.M + tt * 8 - 1) / (tt * 8);
    const int most = own ? kWarps : 24;  // groups a CTA has room for
    const int whole = 256 / shape.item, items_k = (p.K + shape.item - 1) / shape.item;
    Cut best{};
    for (int sp = 1; sp * p.R <= kMaxRanks && sp <= items_k; ++sp) {
        const int per = ((items_k + sp - 1) / sp + whole - 1) / whole * whole;
        if ((items_k + per - 1) / per != sp) continue;  // a split would be empty
        const int resident = dev.clusters[sp * p.R];
        const int64_t run = own ? kWarps : std::min<int64_t>((groups * tiles_m + resident - 1) / resident, most);
        const int64_t waves = ((groups + run - 1) / run * tiles_m + resident - 1) / resident;
        const int64_t busiest = own ? (tt == 2 ? 8 * per + 4 : 15 * per + 8) : run * per + std::min(p.M, 8) * per / 2 + 20;
        const int64_t cost = waves * busiest + (own ? 1 : 2) * sp;
        if (best.cost == 0 || cost < best.cost) best = Cut{sp, per * shape.item, (int)run, cost};
    }
    return best;
}

// One launch over p.M tokens with token tiles of 8 tt.
cudaError_t launch_tiles(QweightParams& p, const QweightDevice& dev, int tt, int* grid, int* cluster, cudaStream_t s) {
    const int tok = tt * 8, wsteps = 1 << (p.group_shift - 5);
    const HostShape shape = host_shape(tt);
    const int rows = shape.rows, item = shape.item, ring = shape.ring, ld = shape.ld;
    const bool own = tt >= 2;
    const bool qx = p.qx && !p.xpow2;
    const int shift = qx && p.xgroup_shift < p.group_shift ? p.xgroup_shift : p.group_shift;
    const int64_t groups = (p.N + rows - 1) / rows;
    p.tiles_m = (p.M + tok - 1) / tok;
    p.rtoks = p.M < tok ? (p.M + 1) / 2 * 2 : tok;
    const int slot = own ? 0 : p.rtoks * ld * 4;                // bytes of a group's sums beside the ring
    const Cut cut = cut_of(p, dev, tt);
    p.splits = cut.splits;
    p.split_k = cut.split_k;
    p.run = cut.run;
    p.cluster = p.R * p.splits;
    const int steps = 1 << (shift - 5);
    const Tokens kind = !p.qx ? kBf16 : p.xpow2 ? kFp8Pow2 : kFp8;
    const Choice k = kernel_of(tt, kind, wsteps, steps);
    size_t smem = k.smem;
    if (!own) {
        // K tile: at most `units` units of 8 k a thread, and as long as the tokens fit what the rest
        // leaves; a multiple of an item and of 128
        // (an item of 128 k holds its groups' scales whole: 128 is the largest group)
        const int xstep = item * tok * 2 + (item >> shift) * tok * 4 + (qx ? item >> p.xgroup_shift : (item + 255) / 256) * tok * 4 +
                          (item >> p.group_shift) * (p.run * rows + 1) * 4;
        const int fixed = ring + 32 + (p.run + kWarps) * slot;
        const int units = shape.units * 8 * kThreads / (tok * item), split_items = p.split_k / item;
        const int room = std::min((kMaxSmem - fixed) / xstep, units);
        if (room < 1) return cudaErrorInvalidValue;
        p.tiles_k = (split_items + room - 1) / room;
        const int tile_items = (split_items + p.tiles_k - 1) / p.tiles_k;
        p.tiles_k = (split_items + tile_items - 1) / tile_items;
        p.tile_k = tile_items * item;
        smem = (size_t)fixed + (size_t)tile_items * xstep;
    }

    const int64_t runs = (groups + p.run - 1) / p.run;
    *cluster = p.cluster;
    *grid = (int)(runs * p.tiles_m * p.cluster);
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    cfg.stream = s;
    if (own) {
        cluster_config(cfg, attr, 1, 0);
        cfg.gridDim = dim3((unsigned)(p.R * p.tiles_m * (p.kp >> 8)));
        const cudaError_t e = cudaLaunchKernelEx(&cfg, tokens_kernel_of(tt, kind, steps), p);
        if (e != cudaSuccess) return e;
    }
    cluster_config(cfg, attr, p.cluster, smem);
    cfg.gridDim = dim3((unsigned)*grid);
    return cudaLaunchKernelEx(&cfg, k.kernel, p);
}

}  // namespace

cudaError_t qweight_prepare(QweightDevice& dev) {
    cudaError_t e = cudaSuccess;
    for (int tt = 1; tt <= 4; tt *= 2)
        for (Tokens kind : {kBf16, kFp8, kFp8Pow2})
            for (int wsteps = 1; wsteps <= 4; wsteps *= 2)
                for (int steps = 1; steps <= wsteps; steps *= 2)
                    if (e == cudaSuccess)
                        e = cudaFuncSetAttribute(kernel_of(tt, kind, wsteps, steps).kernel,
                                                 cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
    // clusters of each size that are resident at once, at the largest shared memory a launch takes
    for (int c = 1; c <= kMaxRanks && e == cudaSuccess; ++c) {
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute attr[2];
        cluster_config(cfg, attr, c, kMaxSmem);
        cfg.gridDim = dim3((unsigned)c);
        cfg.numAttrs = 1;
        e = cudaOccupancyMaxActiveClusters(&dev.clusters[c], kernel_of(2, kFp8, 1, 1).kernel, &cfg);
        if (e == cudaSuccess && dev.clusters[c] < 1) dev.clusters[c] = 1;
    }
    return e;
}

cudaError_t launch_qweight(QweightParams& p, const QweightDevice& dev, uint8_t* scratch, size_t scratch_bytes, int* grid,
                           int* variant, int* cluster, cudaStream_t s) {
    // In tiles of 8 tokens a CTA stages its own; tiles of 16 or 32, whichever is expected to end first, are staged by
    // a kernel before (each CTA staging them again took 30 to 50 % of the time at 16 and 64 tokens), as many at
    // once as the scratch holds.  That kernel and its launch cost as much as 30 items:
    //  * R = 8, 7168 x 2048: 8 tokens 19.2 us in a tile of 8, 22.9 in one of 16; 16 tokens 47 and 21.7; 64 tokens 71 in 32s;
    //  * R = 4, 1024 x 2048: 12 tokens 8.3 and 11.0; 64 tokens 17.5 and 15.8;
    //  * R = 2, 512 x 512: 8 tokens 5.1 and 6.1, 64 tokens 6.1 and 7.0.
    // Rows too long for a staged tile go by 8 tokens.  More than 32 tokens a tile need 200 registers a thread:
    // spilled to 128 they took 139 us at R = 8, M = 64, N = 7168, K = 2048.
    p.kp = (p.K + 255) / 256 * 256;
    // of a token tile: bf16 tokens, sums and scales of at least 32 k, and a flag word per 256 k
    auto tile_bytes = [&](int t) { return (size_t)p.R * p.kp / 32 * (t * 8 * (64 + 4 + 4) + 4); };
    int tt = p.force_tile == 8 || (p.M <= 8 && p.force_tile == 0) || tile_bytes(2) > scratch_bytes ? 1 : 2;
    if (tt == 2 && p.force_tile != 16 && tile_bytes(4) <= scratch_bytes &&
        (p.force_tile == 32 || (p.M > 16 && cut_of(p, dev, 4).cost <= cut_of(p, dev, 2).cost)))
        tt = 4;
    if (p.force_tile == 0 && tt > 1 && cut_of(p, dev, 1).cost <= cut_of(p, dev, tt).cost + 30) tt = 1;
    const int tok = tt * 8, M = p.M;
    const int all = (M + tok - 1) / tok, most = tt == 1 ? all : (int)std::min<size_t>(all, scratch_bytes / tile_bytes(tt));
    *variant = tt;
    for (int first = 0; first < all; first += most) {
        const int rest = M - first * tok;
        const int tiles = std::min(most, all - first);
        p.M = std::min(rest, tiles * tok);
        const size_t k = (size_t)p.R * tiles * p.kp;
        p.tokens = scratch;
        p.sums = reinterpret_cast<float*>(scratch + k * tok * 2);
        p.scales = p.sums + k / 32 * tok;
        p.flags = reinterpret_cast<uint32_t*>(p.scales + k / 32 * tok);
        const cudaError_t e = launch_tiles(p, dev, tt, grid, cluster, s);
        if (e != cudaSuccess) return e;
        for (int r = 0; r < p.R; ++r) {
            p.x[r] = static_cast<const uint8_t*>(p.x[r]) + (size_t)p.M * p.K * (p.qx ? 1 : 2);
            if (p.qx) p.xscale[r] = static_cast<const uint8_t*>(p.xscale[r]) + (size_t)p.M * p.xgroups * (p.xpow2 ? 1 : 4);
        }
        for (int v = 0; v < p.nviews; ++v) p.views[v] += (size_t)p.M * p.N;
    }
    return cudaSuccess;
}

}  // namespace are
