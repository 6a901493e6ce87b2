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
// A cluster owns a run of 16-row groups; each of its CTAs takes one rank's (or,
// where R is small, part of a rank's) K range for all of them, so that its
// tokens go to shared memory once.  The (group, 256 of K) items of a CTA are
// dealt to its warps in equal contiguous runs.  At the end the CTAs add their
// fp32 sums over distributed shared memory, r ascending: no partial sum goes
// through global memory and the order never varies.
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "are_internal.h"
#include "ptx.cuh"

namespace are {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kItemK = 256;                 // codes of a row in one ring slot
constexpr int kRowBytes = kItemK / 2 + 16;  // 144: 36 words, so that 8 rows start in 8 different bank quads
constexpr int kSlotBytes = 16 * kRowBytes;
constexpr int kDepth = 3;                   // ring slots of a warp, and the length of the unrolled loop
constexpr int kRingBytes = kWarps * kDepth * kSlotBytes;
constexpr int kRedLd = 20;                  // floats between a sum's tokens: 8 rows of 4 token pairs in 32 banks
constexpr int kMaxSmem = 113 * 1024;        // two CTAs an SM

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

// The same on a zero accumulator.
__device__ __forceinline__ void mma16816_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

__device__ __forceinline__ uint32_t sub2(uint32_t a, uint32_t b) {
    __nv_bfloat162 r = __hsub2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
    return *reinterpret_cast<uint32_t*>(&r);
}

// The codes i and i + 4 of a word as the bf16 pair 128 + u, then u - z exactly.
template <int I>
__device__ __forceinline__ uint32_t codes2(uint32_t w, uint32_t z2) {
    uint32_t v;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(v) : "r"(w >> (4 * I)), "r"(0x000F000Fu), "r"(0x43004300u));
    return sub2(v, z2);
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

// TT: token tiles of 8.  QX: tokens in 8 bits with scales.  WSTEPS: steps of
// 32 k in a weight group; STEPS: those that share both scales, the smaller of
// the weight and the token group.
template <int TT, bool QX, int WSTEPS, int STEPS>
__global__ void __launch_bounds__(kThreads, 2) qweight_kernel(const __grid_constant__ QweightParams p) {
    extern __shared__ __align__(128) uint8_t qw_smem[];
    constexpr int TOK = TT * 8;
    constexpr int NS = 4 / WSTEPS;  // an item has 8 / WSTEPS weight groups x 2 row halves, NS for each of a row's lanes
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, c = lane & 3;
    const int cluster = p.R * p.splits;
    const int q = (int)(blockIdx.x % cluster);
    const int tile = (int)(blockIdx.x / cluster);
    const int m0 = (tile % p.tiles_m) * TOK, group0 = (tile / p.tiles_m) * p.run;
    const int groups = min(p.run, (p.N + 15) / 16 - group0);  // of 16 rows
    const int r = q / p.splits;
    const int kbeg = (q % p.splits) * p.split_k, kend = min(p.K, kbeg + p.split_k);

    uint8_t* ring = qw_smem + warp * (kDepth * kSlotBytes);
    uint8_t* xs = qw_smem + kRingBytes;                                // [tile_k / 32][TOK][4] units of 8 k
    float* red = reinterpret_cast<float*>(xs + TOK * p.tile_k * 2);    // [slot][TOK][kRedLd]
    float* xsc = red + (p.run + kWarps) * TOK * kRedLd;                // [token groups of the tile][TOK]

    // this warp's items of a K tile: [first, first + count), item = group * per + K index
    const int per = p.tile_k / kItemK, all = groups * per;
    const int first = warp * all / kWarps, count = (warp + 1) * all / kWarps - first;

    // ---- the stream of items, two ahead of their use: codes by asynchronous copies (16 rows of 128
    // bytes, 8 lanes a row, 4 rows apart), the weight scales and zero points by loads.  Lane c of a
    // row quad loads row half c & 1 of the weight groups (c >> 1) + 2j.  N is a multiple of 8: a row
    // half exists or not for all lanes.
    const int64_t row4 = (int64_t)p.K * 2;  // bytes of four rows of codes
    const uint8_t* fcodes = nullptr;
    int64_t fscale = 0;
    int ftl = -1, fleft = 0, fkk = 0, fgl = 0, fk = 0;
    bool ffull = false;
    uint32_t sreg[kDepth][NS], zreg[kDepth][NS];
    auto seek = [&]() {  // pointers of group fgl, K index fkk of tile ftl
        const int n = (group0 + fgl) * 16;
        fk = kbeg + ftl * p.tile_k + fkk * kItemK;
        ffull = n + 16 <= p.N;
        fcodes = p.codes[r] + (((int64_t)(n + (lane >> 3)) * p.K + fk) >> 1) + (lane & 7) * 16;
        fscale = (int64_t)(n + g + 8 * (c & 1)) * p.groups + (fk >> p.group_shift) + (c >> 1);
    };
    auto fetch = [&](uint32_t (&sv)[NS], uint32_t (&zv)[NS], uint8_t* to) {
        if (fleft == 0) {
            if (count > 0 && ftl + 1 < p.tiles_k) {
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
        const bool kin = fk + (lane & 7) * 32 < kend;
        const uint8_t* from = kin ? fcodes : p.codes[r];
        const int64_t step = kin ? row4 : 0;
        uint8_t* at = to + (lane >> 3) * kRowBytes + (lane & 7) * 16;
        cp_async16(at, from, kin);
        cp_async16(at + 4 * kRowBytes, from + step, kin);
        cp_async16(at + 8 * kRowBytes, ffull ? from + 2 * step : from, kin && ffull);
        cp_async16(at + 12 * kRowBytes, ffull ? from + 3 * step : from, kin && ffull);
        cp_commit();
        const bool nin = ffull || (c & 1) == 0;
#pragma unroll
        for (int j = 0; j < NS; ++j) {
            sv[j] = 0u;  // what does not exist weighs nothing
            zv[j] = 8u;
            if (nin && fk + ((c >> 1) + 2 * j) * (WSTEPS * 32) < kend) {
                sv[j] = __ldg(p.scale[r] + fscale + 2 * j);
                if (p.zero[r]) zv[j] = __ldg(p.zero[r] + fscale + 2 * j);
            }
        }
        fk += kItemK;
        fcodes += kItemK / 2;
        fscale += 8 / WSTEPS;
        --fleft;
        if (++fkk == per) {
            fkk = 0;
            ++fgl;
            seek();
        }
    };
    ptx::grid_launch_dependents();
    ptx::grid_wait();
    fetch(sreg[0], zreg[0], ring);
    fetch(sreg[1], zreg[1], ring + kSlotBytes);

    // ---- a K tile's tokens, in bf16 and in the order of the weight pairs; token scales
    auto stage = [&](int tl) {
        const int t0 = kbeg + tl * p.tile_k;
        if (tl) __syncthreads();
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
        if (QX) {
            const int xg = p.tile_k >> p.xgroup_shift, x0 = t0 >> p.xgroup_shift;
            for (int u = threadIdx.x; u < xg * TOK; u += kThreads) {
                const int m = u % TOK, gi = u / TOK;
                float v = 0.f;
                if (m0 + m < p.M && x0 + gi < p.xgroups) {
                    const int64_t at = (int64_t)(m0 + m) * p.xgroups + x0 + gi;
                    v = p.xpow2 ? e8m0_to_float(__ldg(static_cast<const uint8_t*>(p.xscale[r]) + at))
                                : __ldg(static_cast<const float*>(p.xscale[r]) + at);
                }
                xsc[u] = v;
            }
        }
        __syncthreads();
    };

    float acc[TT][4];
#pragma unroll
    for (int t = 0; t < TT; ++t)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[t][j] = 0.f;
    int tl = -1, left = 0, gl = 0, kk = 0;
    // One item.  PH: its ring slot and the place of its scales, fixed in the unrolled loop (moving a
    // register whose load is in flight would wait for it).
    auto item = [&](auto ph) {
        constexpr int PH = decltype(ph)::value;
        constexpr int NEXT = (PH + 2) % kDepth;
        if (left == 0) {
            stage(++tl);
            left = count;
            gl = first / per;
            kk = first % per;
        }
        cp_wait<kDepth - 2>();
        __syncwarp();  // every lane's copies have landed, and every lane has left the slot refilled next
        fetch(sreg[NEXT], zreg[NEXT], ring + NEXT * kSlotBytes);
        const uint8_t* at = ring + PH * kSlotBytes + g * kRowBytes + c * 4;
        uint32_t word[NS];  // scale | 128 + zero, as two bf16
#pragma unroll
        for (int j = 0; j < NS; ++j) word[j] = sreg[PH][j] | ((0x4300u + zreg[PH][j]) << 16);
        const int kt = kk * kItemK;
        if (kbeg + tl * p.tile_k + kt < kend) {
            const uint8_t* xat = xs + (kt >> 5) * (TOK * 64) + lane * 16;
            float d[TT][4];
            uint32_t slo = 0, shi = 0, zlo = 0, zhi = 0;
#pragma unroll
            for (int st = 0; st < kItemK / 32; ++st) {
                if (st % WSTEPS == 0) {
                    const int gi = st / WSTEPS;  // lane 2 * (gi & 1) + half of the quad has it at j = gi / 2
                    slo = __shfl_sync(0xFFFFFFFFu, word[gi / 2], (lane & 28) + (gi & 1) * 2);
                    shi = __shfl_sync(0xFFFFFFFFu, word[gi / 2], (lane & 28) + (gi & 1) * 2 + 1);
                    zlo = __byte_perm(slo, slo, 0x3232);
                    zhi = __byte_perm(shi, shi, 0x3232);
                }
                const uint32_t wlo = *reinterpret_cast<const uint32_t*>(at + st * 16);
                const uint32_t whi = *reinterpret_cast<const uint32_t*>(at + 8 * kRowBytes + st * 16);
                const uint32_t a0[4] = {codes2<0>(wlo, zlo), codes2<0>(whi, zhi), codes2<1>(wlo, zlo), codes2<1>(whi, zhi)};
                const uint32_t a1[4] = {codes2<2>(wlo, zlo), codes2<2>(whi, zhi), codes2<3>(wlo, zlo), codes2<3>(whi, zhi)};
#pragma unroll
                for (int t = 0; t < TT; ++t) {
                    const uint4 b = *reinterpret_cast<const uint4*>(xat + st * (TOK * 64) + t * 512);
                    if (st % STEPS == 0) mma16816_first(d[t], a0, b.x, b.y);
                    else mma16816(d[t], a0, b.x, b.y);
                    mma16816(d[t], a1, b.z, b.w);
                }
                if (st % STEPS == STEPS - 1) {
                    const float fl = __uint_as_float(slo << 16), fh = __uint_as_float(shi << 16);
#pragma unroll
                    for (int t = 0; t < TT; ++t) {
                        if (QX) {
                            const float2 x2 = *reinterpret_cast<const float2*>(
                                xsc + ((kt + st * 32) >> p.xgroup_shift) * TOK + t * 8 + 2 * c);
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
        --left;
        if (++kk == per || left == 0) {
            // the warp leaves a group: its sums go to the slot of (group, warp), which no other
            // warp touches; along a CTA's items either index grows, so group + warp is unique
            float* to = red + (gl + warp) * TOK * kRedLd + g;
#pragma unroll
            for (int t = 0; t < TT; ++t) {
                float* e = to + (t * 8 + 2 * c) * kRedLd;
                if (tl == 0) {
                    e[0] = acc[t][0]; e[kRedLd] = acc[t][1]; e[8] = acc[t][2]; e[kRedLd + 8] = acc[t][3];
                } else {
                    e[0] += acc[t][0]; e[kRedLd] += acc[t][1]; e[8] += acc[t][2]; e[kRedLd + 8] += acc[t][3];
                }
                acc[t][0] = acc[t][1] = acc[t][2] = acc[t][3] = 0.f;
            }
            kk = 0;
            ++gl;
        }
    };
    if (count == 0) {  // a warp without items helps to stage the tokens
        for (int i = 0; i < p.tiles_k; ++i) stage(i);
    } else {
        const int total = p.tiles_k * count;
        int i = 0;
        for (; i + kDepth <= total; i += kDepth) {
            item(std::integral_constant<int, 0>{});
            item(std::integral_constant<int, 1>{});
            item(std::integral_constant<int, 2>{});
        }
        if (i < total) item(std::integral_constant<int, 0>{});
        if (i + 1 < total) item(std::integral_constant<int, 1>{});
    }
    cp_wait<0>();
    __syncthreads();

    // ---- the sums: of a group over the CTA's warps (into the slot of its first warp), then over the
    // cluster, r ascending.  Item i belongs to warp (8 (i + 1) - 1) / all.
    const int toks = min(TOK, p.M - m0);
    auto warp_of = [&](int i) { return (kWarps * (i + 1) - 1) / all; };
    for (int a = warp; a < groups; a += kWarps) {
        const int w0 = warp_of(a * per), w1 = warp_of(a * per + per - 1);
        for (int w = w0 + 1; w <= w1; ++w) {
            if ((w + 1) * all / kWarps == w * all / kWarps) continue;  // a warp without items
            for (int m = lane >> 4; m < toks; m += 2)
                red[((a + w0) * TOK + m) * kRedLd + (lane & 15)] += red[((a + w) * TOK + m) * kRedLd + (lane & 15)];
        }
    }
    __syncwarp();
    ptx::cluster_sync();
    const uint32_t base = ptx::smem_u32(red);
    for (int a = q + cluster * warp; a < groups; a += cluster * kWarps) {
        const int n = (group0 + a) * 16 + (lane & 7) * 2;
        const int s0 = a + warp_of(a * per);
        if (n < p.N) {
            for (int m = lane >> 3; m < toks; m += 4) {
                const uint32_t addr = base + (uint32_t)((s0 * TOK + m) * kRedLd + (lane & 7) * 2) * 4u;
                float2 s = make_float2(0.f, 0.f);
#pragma unroll
                for (int j = 0; j < kMaxRanks; ++j) {
                    if (j < cluster) {
                        const float2 v = ld_cluster_f2(ptx::mapa_shared(addr, (uint32_t)j));
                        s.x += v.x;
                        s.y += v.y;
                    }
                }
                const __nv_bfloat162 o = __floats2bfloat162_rn(s.x, s.y);
                for (int v = 0; v < p.nviews; ++v)
                    *reinterpret_cast<__nv_bfloat162*>(p.views[v] + (int64_t)(m0 + m) * p.N + n) = o;
            }
        }
    }
    __syncwarp();
    ptx::cluster_sync();  // no CTA leaves while another reads its sums
}

typedef void (*Kernel)(QweightParams);

template <int TT, bool QX, int WSTEPS>
Kernel kernel_of(int steps) {
    if constexpr (!QX || WSTEPS == 1) return qweight_kernel<TT, QX, WSTEPS, WSTEPS>;
    else if constexpr (WSTEPS == 2) return steps == 1 ? qweight_kernel<TT, QX, 2, 1> : qweight_kernel<TT, QX, 2, 2>;
    else return steps == 1 ? qweight_kernel<TT, QX, 4, 1> : steps == 2 ? qweight_kernel<TT, QX, 4, 2> : qweight_kernel<TT, QX, 4, 4>;
}
template <int TT, bool QX>
Kernel kernel_of(int wsteps, int steps) {
    return wsteps == 1 ? kernel_of<TT, QX, 1>(steps) : wsteps == 2 ? kernel_of<TT, QX, 2>(steps) : kernel_of<TT, QX, 4>(steps);
}
template <int TT>
Kernel kernel_of(bool qx, int wsteps, int steps) {
    return qx ? kernel_of<TT, true>(wsteps, steps) : kernel_of<TT, false>(wsteps, steps);
}
// The kernel of a token tile and of the groups' sizes in steps of 32; steps <= wsteps.
Kernel kernel_of(int tt, bool qx, int wsteps, int steps) {
    return tt == 1 ? kernel_of<1>(qx, wsteps, steps) : tt == 2 ? kernel_of<2>(qx, wsteps, steps) : kernel_of<4>(qx, wsteps, steps);
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

}  // namespace

cudaError_t qweight_prepare(QweightDevice& dev) {
    cudaError_t e = cudaSuccess;
    for (int tt = 1; tt <= 4; tt *= 2)
        for (int qx = 0; qx < 2; ++qx)
            for (int wsteps = 1; wsteps <= 4; wsteps *= 2)
                for (int steps = 1; steps <= wsteps; steps *= 2)
                    if (e == cudaSuccess)
                        e = cudaFuncSetAttribute(kernel_of(tt, qx != 0, wsteps, steps),
                                                 cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
    // clusters of each size that are resident at once, at the largest shared memory a launch takes
    for (int c = 1; c <= kMaxRanks && e == cudaSuccess; ++c) {
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute attr[2];
        cluster_config(cfg, attr, c, kMaxSmem);
        cfg.gridDim = dim3((unsigned)c);
        e = cudaOccupancyMaxActiveClusters(&dev.clusters[c], kernel_of(4, true, 1, 1), &cfg);
        if (e == cudaSuccess && dev.clusters[c] < 1) dev.clusters[c] = 1;
    }
    return e;
}

cudaError_t launch_qweight(QweightParams& p, bool qx, const QweightDevice& dev, int* grid, int* variant, int* cluster,
                           cudaStream_t s) {
    const int tt = p.M <= 8 ? 1 : p.M <= 16 ? 2 : 4;
    const int tok = tt * 8;
    p.tiles_m = (p.M + tok - 1) / tok;
    const int groups = (p.N + 15) / 16;
    // Splits of a rank's K: those that leave the busiest CTA the fewest items (an item is 16 rows
    // by 256 of K), where a split also costs about one item more to join.
    const int items_k = (p.K + kItemK - 1) / kItemK;
    int64_t best = 0;
    for (int sp = 1; sp * p.R <= kMaxRanks && sp <= items_k; ++sp) {
        const int64_t rounds = (int64_t)((groups + dev.clusters[sp * p.R] - 1) / dev.clusters[sp * p.R]) * p.tiles_m;
        const int64_t cost = rounds * ((items_k + sp - 1) / sp) + sp;
        if (sp == 1 || cost < best) {
            best = cost;
            p.splits = sp;
        }
    }
    *cluster = p.R * p.splits;
    p.split_k = (items_k + p.splits - 1) / p.splits * kItemK;
    // Groups a cluster: an even share for every resident cluster, as far as their sums fit shared memory.
    const int slot = tok * kRedLd * 4;
    const int most = 36 * 1024 / slot - kWarps;
    p.run = (groups + dev.clusters[*cluster] - 1) / dev.clusters[*cluster];
    if (p.run > most) p.run = most;
    // K tile: as long as the tokens fit what is left
    const int xstep = kItemK * tok * 2 + (qx ? (kItemK >> p.xgroup_shift) * tok * 4 : 0);
    const int room = (kMaxSmem - kRingBytes - (p.run + kWarps) * slot) / xstep;  // items of K
    const int split_items = p.split_k / kItemK;
    p.tiles_k = (split_items + room - 1) / room;
    const int tile_items = (split_items + p.tiles_k - 1) / p.tiles_k;
    p.tile_k = tile_items * kItemK;
    const size_t smem = (size_t)kRingBytes + (size_t)(p.run + kWarps) * slot + (size_t)tile_items * xstep;

    const int runs = (groups + p.run - 1) / p.run;
    *grid = runs * p.tiles_m * *cluster;
    *variant = tt;
    const int shift = qx && p.xgroup_shift < p.group_shift ? p.xgroup_shift : p.group_shift;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    cluster_config(cfg, attr, *cluster, smem);
    cfg.gridDim = dim3((unsigned)*grid);
    cfg.stream = s;
    return cudaLaunchKernelEx(&cfg, kernel_of(tt, qx, 1 << (p.group_shift - 5), 1 << (shift - 5)), p);
}

}  // namespace are
