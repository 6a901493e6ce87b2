// The row-parallel linear of a few tokens with 4-bit weights, all-reduced over
// R ranks:
//   out[m][n] = bf16( sum_{r=0..R-1} sum_k x_r[m][k] * (u_r[n][k] - z_r[n][g]) * s_r[n][g] ),
//   g = k / group,
// with tokens x in bf16, or in FP8 E4M3 codes times a scale per group of k.
//
// Bound by the weights' bytes: M tokens use each of them M times.  So the
// codes are read once, straight into a ring of shared memory per warp (16-byte
// asynchronous copies, no barrier between warps), and meet the tokens in
// m16n8k16 tensor instructions whose 16 rows are weight rows and whose 8
// columns are tokens.  Integers u - z are exact in bf16, so every product is
// exact and the group scales are applied in fp32, once per group, to the
// tensor instruction's fp32 sums: no weight is ever rounded.
//
// A word of 8 codes gives the pairs (k, k+4), k = 0..3, of one MMA operand
// register by a shift and a masked OR that places a code in the mantissa of
// 128.0; the tokens are laid into shared memory in the same order of k, so
// nothing is shuffled.
//
// One cluster computes one tile of output rows: its CTAs take the ranks (and
// splits of K where R is small) and add their fp32 sums over distributed
// shared memory, r ascending, so no partial sum goes through global memory and
// the order never varies.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "are_internal.h"
#include "ptx.cuh"

namespace are {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kItemK = 256;               // codes of a row in one ring slot
constexpr int kRowBytes = kItemK / 2 + 16;  // 144: 36 words, 8 rows start in 8 different bank quads
constexpr int kSlotBytes = 16 * kRowBytes;
constexpr int kDepth = 4;                 // ring slots of a warp
constexpr int kRingBytes = kWarps * kDepth * kSlotBytes;
constexpr int kMaxSmem = 227 * 1024;

__device__ __forceinline__ void cp_async16(void* dst, const void* src, bool valid) {
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(ptx::smem_u32(dst)), "l"(src),
                 "r"(valid ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t sub2(uint32_t a, uint32_t b) {
    __nv_bfloat162 r = __hsub2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
    return *reinterpret_cast<uint32_t*>(&r);
}

// The codes i and i + 4 of a word as the bf16 pair 128 + u, then u - z exactly.
template <int I>
__device__ __forceinline__ uint32_t codes2(uint32_t w, uint32_t z2) {
    return sub2(((w >> (4 * I)) & 0x000F000Fu) | 0x43004300u, z2);
}

__device__ __forceinline__ uint32_t fp8x2_to_bf16x2(uint32_t v) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(v & 0xFFFFu), __NV_E4M3);
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    const __nv_bfloat162 b = __floats2bfloat162_rn(f.x, f.y);  // exact: 4 significant bits
    return *reinterpret_cast<const uint32_t*>(&b);
}

__device__ __forceinline__ float e8m0_to_float(uint32_t b) {
    return __uint_as_float(b == 255u ? 0x7FC00000u : b == 0u ? 0x00400000u : b << 23);
}

// 8 consecutive k of a token in the order of the weight pairs: 0 4 1 5 2 6 3 7.
__device__ __forceinline__ uint4 pair_order(uint32_t w0, uint32_t w1, uint32_t w2, uint32_t w3) {
    return make_uint4(__byte_perm(w0, w2, 0x5410), __byte_perm(w0, w2, 0x7632), __byte_perm(w1, w3, 0x5410),
                      __byte_perm(w1, w3, 0x7632));
}

__device__ __forceinline__ float2 ld_cluster_f2(uint32_t addr) {
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
    return v;
}

// TT: token tiles of 8.  QX: tokens in 8 bits with scales.
template <int TT, bool QX>
__global__ void __launch_bounds__(kThreads, 2) qweight_kernel(const __grid_constant__ QweightParams p, int ks_shift) {
    extern __shared__ __align__(128) uint8_t qw_smem[];
    constexpr int TOK = TT * 8;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, c = lane & 3;
    const int KS = 1 << ks_shift, BN = (kWarps >> ks_shift) * 16;
    const int rowgroup = warp >> ks_shift, ks = warp & (KS - 1);
    const int cluster = p.R * p.splits;
    const int q = (int)(blockIdx.x % cluster);
    const int tile = (int)(blockIdx.x / cluster);
    const int m0 = (tile % p.tiles_m) * TOK, n0 = (tile / p.tiles_m) * BN;
    const int r = q / p.splits;
    const int kbeg = (q % p.splits) * p.split_k, kend = min(p.K, kbeg + p.split_k);
    const int len = max(kend - kbeg, 0);
    const int tiles = (len + p.tile_k - 1) / p.tile_k;
    const int items = p.tile_k / (kItemK * KS);  // of a warp in a tile
    const int granule = QX ? min(p.group_shift, p.xgroup_shift) : p.group_shift;

    uint8_t* ring = qw_smem + warp * (kDepth * kSlotBytes);
    uint8_t* xs = qw_smem + kRingBytes;                                    // [tile_k / 32][TOK][4] units of 8 k
    uint32_t* wsc = reinterpret_cast<uint32_t*>(xs + TOK * p.tile_k * 2);  // [groups of the tile][BN]: scale | 128 + zero
    float* xsc = reinterpret_cast<float*>(wsc + (p.tile_k >> p.group_shift) * BN);  // [xgroups of the tile][TOK]

    // asynchronous copies of this warp's codes, item by item
    const uint8_t* codes = p.codes[r];
    const int total = tiles * items;
    auto fetch = [&](int i) {
        if (i < total) {
            const int k0 = kbeg + (i * KS + ks) * kItemK;
            uint8_t* slot = ring + (i % kDepth) * kSlotBytes;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int row = j * 4 + (lane >> 3), col = (lane & 7) * 16;
                const int n = n0 + rowgroup * 16 + row, k = k0 + col * 2;
                const bool ok = n < p.N && k < kend;
                cp_async16(slot + row * kRowBytes + col, codes + (ok ? ((int64_t)n * p.K + k) / 2 : 0), ok);
            }
        }
        cp_commit();
    };
#pragma unroll
    for (int i = 0; i < kDepth - 1; ++i) fetch(i);

    float acc[TT][4];
#pragma unroll
    for (int t = 0; t < TT; ++t)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[t][j] = 0.f;

    for (int tl = 0; tl < tiles; ++tl) {
        const int t0 = kbeg + tl * p.tile_k;
        if (tl) __syncthreads();
        // the tile's tokens
        for (int u = threadIdx.x; u < TOK * p.tile_k / 8; u += kThreads) {
            const int m = m0 + (u >> 2) % TOK, k = t0 + u / (4 * TOK) * 32 + (u & 3) * 8;
            uint4 v = make_uint4(0u, 0u, 0u, 0u);
            if (m < p.M && k < kend) {
                if (QX) {
                    const uint2 b = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(p.x[r]) +
                                                                         (int64_t)m * p.K + k));
                    v = pair_order(fp8x2_to_bf16x2(b.x), fp8x2_to_bf16x2(b.x >> 16), fp8x2_to_bf16x2(b.y),
                                   fp8x2_to_bf16x2(b.y >> 16));
                } else {
                    const uint4 b = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.x[r]) +
                                                                         (int64_t)m * p.K + k));
                    v = pair_order(b.x, b.y, b.z, b.w);
                }
            }
            *reinterpret_cast<uint4*>(xs + u * 16) = v;
        }
        // its weight scales and zero points; groups and rows that do not exist weigh nothing
        const int tg = p.tile_k >> p.group_shift, g0 = t0 >> p.group_shift;
        for (int u = threadIdx.x; u < tg * BN; u += kThreads) {
            const int gi = u % tg, n = u / tg;
            uint32_t v = 0x43080000u;
            if (n0 + n < p.N && g0 + gi < p.groups) {
                const int64_t at = (int64_t)(n0 + n) * p.groups + g0 + gi;
                v = __ldg(p.scale[r] + at);
                v |= (0x4300u + (p.zero[r] ? (uint32_t)__ldg(p.zero[r] + at) : 8u)) << 16;
            }
            wsc[gi * BN + n] = v;
        }
        if (QX) {
            const int xg = p.tile_k >> p.xgroup_shift, x0 = t0 >> p.xgroup_shift;
            for (int u = threadIdx.x; u < xg * TOK; u += kThreads) {
                const int gi = u % xg, m = u / xg;
                float v = 0.f;
                if (m0 + m < p.M && x0 + gi < p.xgroups) {
                    const int64_t at = (int64_t)(m0 + m) * p.xgroups + x0 + gi;
                    v = p.xpow2 ? e8m0_to_float(__ldg(static_cast<const uint8_t*>(p.xscale[r]) + at))
                                : __ldg(static_cast<const float*>(p.xscale[r]) + at);
                }
                xsc[gi * TOK + m] = v;
            }
        }
        __syncthreads();

        for (int it = 0; it < items; ++it) {
            const int i = tl * items + it;
            cp_wait<kDepth - 2>();
            __syncwarp();
            const int kt = (it * KS + ks) * kItemK;  // within the tile
            if (t0 + kt < kend) {
                const uint8_t* slot = ring + (i % kDepth) * kSlotBytes;
                float d[TT][4];
#pragma unroll
                for (int st = 0; st < kItemK / 32; ++st) {
                    const int k = kt + st * 32;
                    const int gi = k >> p.group_shift;
                    if ((st & ((1 << (granule - 5)) - 1)) == 0) {
#pragma unroll
                        for (int t = 0; t < TT; ++t)
#pragma unroll
                            for (int j = 0; j < 4; ++j) d[t][j] = 0.f;
                    }
                    const uint32_t slo = wsc[gi * BN + rowgroup * 16 + g], shi = wsc[gi * BN + rowgroup * 16 + g + 8];
                    const uint32_t zlo = __byte_perm(slo, slo, 0x3232), zhi = __byte_perm(shi, shi, 0x3232);
                    const uint32_t wlo = *reinterpret_cast<const uint32_t*>(slot + g * kRowBytes + (st * 4 + c) * 4);
                    const uint32_t whi = *reinterpret_cast<const uint32_t*>(slot + (g + 8) * kRowBytes + (st * 4 + c) * 4);
                    const uint32_t a0[4] = {codes2<0>(wlo, zlo), codes2<0>(whi, zhi), codes2<1>(wlo, zlo), codes2<1>(whi, zhi)};
                    const uint32_t a1[4] = {codes2<2>(wlo, zlo), codes2<2>(whi, zhi), codes2<3>(wlo, zlo), codes2<3>(whi, zhi)};
#pragma unroll
                    for (int t = 0; t < TT; ++t) {
                        const uint4 b = *reinterpret_cast<const uint4*>(xs + ((((k >> 5) * TOK + t * 8 + g) << 2) + c) * 16);
                        mma16816(d[t], a0, b.x, b.y);
                        mma16816(d[t], a1, b.z, b.w);
                    }
                    if (((st + 1) & ((1 << (granule - 5)) - 1)) == 0) {
                        const float fl = __uint_as_float(slo << 16), fh = __uint_as_float(shi << 16);
#pragma unroll
                        for (int t = 0; t < TT; ++t) {
                            if (QX) {
                                const float2 x2 = *reinterpret_cast<const float2*>(xsc + (k >> p.xgroup_shift) * TOK + t * 8 + 2 * c);
                                acc[t][0] = fmaf(fl * x2.x, d[t][0], acc[t][0]);
                                acc[t][1] = fmaf(fl * x2.y, d[t][1], acc[t][1]);
                                acc[t][2] = fmaf(fh * x2.x, d[t][2], acc[t][2]);
                                acc[t][3] = fmaf(fh * x2.y, d[t][3], acc[t][3]);
                            } else {
                                acc[t][0] = fmaf(fl, d[t][0], acc[t][0]);
                                acc[t][1] = fmaf(fl, d[t][1], acc[t][1]);
                                acc[t][2] = fmaf(fh, d[t][2], acc[t][2]);
                                acc[t][3] = fmaf(fh, d[t][3], acc[t][3]);
                            }
                        }
                    }
                }
            }
            __syncwarp();  // every lane has read the slot that the next copies overwrite
            fetch(i + kDepth - 1);
        }
    }
    cp_wait<0>();
    __syncthreads();

    // this CTA's sums, [ks][token][row]; a token's rows are padded so that the four tokens a
    // store touches start in four different bank groups
    float* red = reinterpret_cast<float*>(qw_smem);
    const int ld = BN + 4;
#pragma unroll
    for (int t = 0; t < TT; ++t) {
        float* at = red + (size_t)ks * TOK * ld + rowgroup * 16 + g;
        const int m = t * 8 + 2 * c;
        at[m * ld] = acc[t][0];
        at[(m + 1) * ld] = acc[t][1];
        at[m * ld + 8] = acc[t][2];
        at[(m + 1) * ld + 8] = acc[t][3];
    }
    if (KS > 1) {
        __syncthreads();
        for (int u = threadIdx.x; u < TOK * BN; u += kThreads) {
            const int at = u / BN * ld + u % BN;
            float v = red[at];
            for (int j = 1; j < KS; ++j) v += red[j * TOK * ld + at];
            red[at] = v;
        }
    }
    __syncwarp();
    ptx::cluster_sync();
    const int toks = min(TOK, p.M - m0), half = BN / 2;
    const uint32_t base = ptx::smem_u32(red);
    for (int u = q * kThreads + threadIdx.x; u < toks * half; u += cluster * kThreads) {
        const int m = u / half, n = (u % half) * 2;
        if (n0 + n < p.N) {
            float2 s = make_float2(0.f, 0.f);
            for (int j = 0; j < cluster; ++j) {
                const float2 v = ld_cluster_f2(ptx::mapa_shared(base + (uint32_t)(m * ld + n) * 4u, (uint32_t)j));
                s.x += v.x;
                s.y += v.y;
            }
            const __nv_bfloat162 o = __floats2bfloat162_rn(s.x, s.y);
            for (int v = 0; v < p.nviews; ++v)
                *reinterpret_cast<__nv_bfloat162*>(p.views[v] + (int64_t)(m0 + m) * p.N + n0 + n) = o;
        }
    }
    __syncwarp();
    ptx::cluster_sync();  // no CTA leaves while another reads its sums
}

typedef void (*Kernel)(QweightParams, int);

Kernel kernel_of(int tt, bool qx) {
    switch (tt) {
        case 1: return qx ? qweight_kernel<1, true> : qweight_kernel<1, false>;
        case 2: return qx ? qweight_kernel<2, true> : qweight_kernel<2, false>;
        case 4: return qx ? qweight_kernel<4, true> : qweight_kernel<4, false>;
        default: return qx ? qweight_kernel<8, true> : qweight_kernel<8, false>;
    }
}

}  // namespace

cudaError_t qweight_prepare() {
    cudaError_t e = cudaSuccess;
    for (int tt = 1; tt <= 8; tt *= 2)
        for (int qx = 0; qx < 2; ++qx)
            if (e == cudaSuccess)
                e = cudaFuncSetAttribute(kernel_of(tt, qx != 0), cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
    return e;
}

cudaError_t launch_qweight(QweightParams& p, bool qx, int num_sms, int* grid, int* variant, int* cluster,
                           cudaStream_t s) {
    const int tt = p.M <= 8 ? 1 : p.M <= 16 ? 2 : p.M <= 32 ? 4 : 8;
    const int tok = tt * 8;
    p.tiles_m = (p.M + tok - 1) / tok;
    // Splits of K: as many as the cluster has room for and 512 of K each.
    p.splits = 8 / p.R;
    while (p.splits > 1 && p.K < p.splits * 512) --p.splits;
    const int range = (p.K + p.splits - 1) / p.splits;
    // Warps share a row tile's K range (fewer rows a CTA) while there are fewer than two CTAs an SM.
    int ks = 0;
    auto ctas = [&](int k) {
        const int bn = 128 >> k;
        return (int64_t)((p.N + bn - 1) / bn) * p.tiles_m * p.R * p.splits;
    };
    while (ks < 3 && ctas(ks) < 2 * num_sms && (kItemK << (ks + 1)) <= range && tok << ks <= 64) ++ks;
    const int unit = kItemK << ks;
    p.split_k = (range + unit - 1) / unit * unit;
    // tokens of a tile: up to 32 KB
    p.tile_k = 16384 / tok / unit * unit;
    if (p.tile_k < unit) p.tile_k = unit;
    if (p.tile_k > p.split_k) p.tile_k = p.split_k;
    const int bn = 128 >> ks;
    size_t smem = kRingBytes + (size_t)tok * p.tile_k * 2 + (size_t)(p.tile_k >> p.group_shift) * bn * 4 +
                  (qx ? (size_t)(p.tile_k >> p.xgroup_shift) * tok * 4 : 0);
    const size_t red = (size_t)(tok << ks) * (bn + 4) * 4;
    if (smem < red) smem = red;
    p.smem = (uint32_t)smem;

    *cluster = p.R * p.splits;
    *grid = (int)ctas(ks);
    *variant = tt * 8 + (1 << ks);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)*grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)*cluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel_of(tt, qx), p, ks);
}

}  // namespace are
