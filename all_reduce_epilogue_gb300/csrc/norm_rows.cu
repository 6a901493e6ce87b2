// Row-streaming kernels around the residual add and RMSNorm after an
// all-reduce: the group-quantised forward (FP8 E4M3 codes with one scale per
// group of columns) and the backward pass.
//
// Forward, per row i (partials x_r, residual e, width N):
//   h = sum_{r=0..R-1} x_r + e          (fp32, r ascending; the sum starts at
//                                        +0.0, so an all -0.0 sum is +0.0)
//   y = h * rsqrt(mean(h^2) + eps) * gamma
//   per group of G columns: a = max|y|,  scale = a / 448 or a power of two,
//   code = e4m3(y / scale)
// With z = h * gamma, y / scale is z * 448 / max|z|: the code of the fp32 form
// needs no inv, and two roundings (of 448 / max|z| and of the product, the
// rounding error of z going in through an fma) decide it.  z is formed at the
// size of y, h times the power of two below inv, so it leaves fp32's range only
// where y does.
// Backward (dy = sum_r dy_r the all-reduced output gradient, d_res the
// gradient of the updated residual, inv = rsqrt(mean(h^2) + eps)):
//   dh      = inv * dy * gamma - h * inv^3 * mean(dy * gamma * h) + d_res
//   dgamma  = sum_i dy_i * h_i * inv_i
//
// Both are bound by HBM: every input byte is read once, every output written
// once, and one row's sums decide nothing about another's.  A block owns whole
// rows (row = block, block + grid, ...).  One producer warp streams the row's
// sources (R partials, residual / h, gradient of the residual) with 1D bulk
// copies into a ring of stages, stage (row, k) holding the k-th slice of
// blockDim-32 packs of 8 columns of every source; consumer thread t owns pack
// t of every slice, so a row lives in registers between the two passes over
// it (statistics, then outputs) and the ring already fills with the next row
// meanwhile.  A thread owns the same columns in every row, which lets the
// backward pass keep its dgamma sums in registers until the block ends; a
// small kernel adds the blocks' rows of them (4 us).
// Measured (a copy moves 6.78 TB/s): forward, R = 8, 4096 x 7168: 99 us,
// 6.2 TB/s; backward, R = 8, 4096 x 7168: 97 us, 6.7 TB/s; R = 1, 16384 x 4096:
// 90 us, 6.0 TB/s.  One row of 7168 at R = 8: 3.9 us, all latency.  Narrow rows
// are below both rates (R = 1, 16384 x 2048 backward 57 us, 4.7 TB/s, issue
// slots 58 % used): what each row costs besides its bytes, a barrier of the
// block, two sums over its warps and a turn of the ring, is for one or two packs
// a thread.  So their arithmetic is in pairs of columns, and an SM takes as many
// blocks as its registers hold (16384 x 1024: 34 us; two blocks 43).
#include <cuda_fp8.h>

#include <algorithm>

#include "rows.cuh"

namespace are {
namespace {

// ------------------------------------------------------------ quantised forward
// The larger magnitude, NaN if one is.
__device__ __forceinline__ float max_abs(float a, float b) {
    float v;
    asm("{\n\t.reg .f32 x, y;\n\tabs.f32 x, %1;\n\tabs.f32 y, %2;\n\tmax.NaN.f32 %0, x, y;\n\t}" : "=f"(v) : "f"(a), "f"(b));
    return v;
}

// n / d from an approximate reciprocal of d, corrected once by the remainder (Markstein 1990: the quotient's
// remainder is exact in an fma).  The reciprocal is off by 2^-23 of its value at most and n * rcp by less than 2^-22, so
// the corrected quotient before its rounding is off by less than 2^-44: correctly rounded unless n / d is within that of
// a tie.  No over- or underflow on the way.
__device__ __forceinline__ float quotient(float n, float d, float rcp) {
    const float q = n * rcp;
    return fmaf(fmaf(-d, q, n), rcp, q);
}
__device__ __forceinline__ float approx_rcp(float d) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(d));
    return r;
}

// Scale of a group whose largest |z| is `top` and largest |y| = top * m is
// finite (1 <= m < 2), and the factor that takes z to code range.
struct GroupScale {
    float factor;
    uint32_t stored;  // fp32 bits, or the E8M0 byte
};

template <bool POW2>
__device__ __forceinline__ GroupScale group_scale(float top, float m) {
    GroupScale s;
    const float a = top * m;
    if (POW2) {
        // the smallest power of two X with a / X <= 448 = 1.75 * 2^8, as a biased exponent >= 0
        const uint32_t u = __float_as_uint(a);
        int e = (int)(u >> 23) - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
        e = u == 0 ? 127 : max(e, 0);
        s.stored = (uint32_t)e;
        s.factor = m * __uint_as_float((uint32_t)(254 - e) << 23);  // m * 2^(127 - e), e <= 247: exact
    } else {
        // at least 2^-126, so that its reciprocal is finite
        const bool tiny = a < 448 * 1.17549435e-38f;
        const float sc = tiny ? 1.17549435e-38f : quotient(a, 448.f, 1.f / 448.f);
        s.stored = __float_as_uint(a == 0.f ? 1.f : sc);
        // (the reciprocal of the largest magnitudes would be a denormal)
        s.factor = tiny ? m * 8.50705917e37f : top < 0x1p120f ? quotient(448.f, top, approx_rcp(top)) : __fdiv_rn(448.f, top);
    }
    return s;
}

template <int PPT, bool POW2, int THREADS, int BLOCKS>
__global__ void __launch_bounds__(THREADS, BLOCKS)
    norm_quant_rows_kernel(const __grid_constant__ RowsParams p) {
    extern __shared__ __align__(128) uint8_t rows_smem[];
    const Ring g = carve(rows_smem, p);
    ring_init(g, p);
    ptx::grid_launch_dependents();
    ptx::grid_wait();
    if (threadIdx.x >= p.nt) {
        produce(g, p);
        return;
    }
    const int t = threadIdx.x, lane = t & 31, w = t >> 5, nwarps = p.nt >> 5;
    const int P = p.N >> 3;
    const size_t step = (size_t)p.nt * 16;
    constexpr bool kGammaRegs = PPT <= 4;
    Pack gam[kGammaRegs ? PPT : 1];
    if (kGammaRegs) {
#pragma unroll
        for (int k = 0; k < PPT; ++k) {
            const int pk = t + k * p.nt;
            if (pk < P) load8(p.gamma + pk * 8, gam[k]);
        }
    }
    int s = 0, buf = 0;
    uint32_t ph = 0;
    for (int64_t row = blockIdx.x; row < p.M; row += gridDim.x, buf ^= 1) {
        Pack h[PPT];
        uint64_t ss2 = 0ull;
#pragma unroll
        for (int k = 0; k < PPT; ++k) {
            if (k < p.slices) {
                const int pk = t + k * p.nt;
                ring_wait(&g.full[s], ph, g, p);
                const uint8_t* at = g.stage + (size_t)s * p.stage_bytes + t * 16;
                if (pk < P) {
                    sum_ranks<false>(at, p.R, step, h[k]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) h[k][i] = add2(h[k][i], 0ull);  // a sum of -0.0 counts as +0.0
                    if (p.has_res) {
                        Pack e;
                        unpack8(*reinterpret_cast<const uint4*>(at + p.R * step), e);
#pragma unroll
                        for (int i = 0; i < 4; ++i) h[k][i] = add2(h[k][i], e[i]);
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) ss2 = fma2(h[k][i], h[k][i], ss2);
                }
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(&g.empty[s]);
                if (++s == p.stages) { s = 0; ph ^= 1u; }
                if (p.res_out && pk < P) ptx::st_stream_v4(p.res_out + row * (int64_t)p.N + pk * 8, pack8(h[k]));
            }
        }
        // one barrier a row: the next row's partial sums go to the other buffer
        float* red = g.red + buf * 64;
        const float ss = warp_sum(both(ss2));
        if (lane == 0) red[w] = ss;
        consumer_bar(p.nt);
        // inv = two * m: a power of two (0 for 0, infinite for NaN) and 1 <= m < 2
        const uint32_t inv = __float_as_uint(rsqrtf(red_total(red, nwarps) * p.inv_n + p.eps));
        const float two = __uint_as_float(inv & 0x7F800000u), m = __uint_as_float((inv & 0x7FFFFFu) | 0x3F800000u);
        const uint64_t two2 = pair(two, two), minus = pair(-1.f, -1.f);
#pragma unroll
        for (int k = 0; k < PPT; ++k) {
            if (k < p.slices) {
                const int pk = t + k * p.nt;
                const bool in = pk < P;
                Pack gk;
                if (kGammaRegs) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) gk[i] = gam[kGammaRegs ? k : 0][i];
                } else if (in) {
                    load8(p.gamma + pk * 8, gk);
                }
                float top = 0.f;  // largest |z|
                if (in) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        h[k][i] = mul2(h[k][i], two2);
                        const float2 z = unpair(mul2(h[k][i], gk[i]));
                        top = max_abs(top, max_abs(z.x, z.y));
                    }
                }
                // a group is 4, 8 or 16 neighbouring lanes (p.nt is a multiple of 32)
                for (int o = 1; o < p.group_packs; o <<= 1) top = max_abs(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
                if (in) {
                    uint2 q;
                    uint32_t stored;
                    if (top * m <= 3.40282347e38f) {
                        const GroupScale gs = group_scale<POW2>(top, m);
                        stored = gs.stored;
                        const uint64_t factor = pair(gs.factor, gs.factor);
                        uint32_t c[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const uint64_t z = mul2(h[k][i], gk[i]), lost = fma2(h[k][i], gk[i], mul2(z, minus));
                            c[i] = (uint32_t)__nv_cvt_float2_to_fp8x2(unpair(fma2(z, factor, mul2(lost, factor))),
                                                                      __NV_SATFINITE, __NV_E4M3);
                        }
                        q = make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
                    } else {  // not finite: NaN codes under a NaN scale
                        stored = POW2 ? 0xFFu : 0x7FC00000u;
                        q = make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
                    }
                    ptx::st_stream_v2(p.out_q + row * (int64_t)p.N + pk * 8, q);
                    if ((lane & (p.group_packs - 1)) == 0) {
                        const int64_t at = row * (int64_t)p.groups + pk / p.group_packs;
                        if (POW2) static_cast<uint8_t*>(p.out_scale)[at] = (uint8_t)stored;
                        else static_cast<uint32_t*>(p.out_scale)[at] = stored;
                    }
                }
            }
        }
    }
}

// --------------------------------------------------------------------- backward
template <int PPT, bool ONE, int THREADS, int BLOCKS>
__global__ void __launch_bounds__(THREADS, BLOCKS) norm_backward_rows_kernel(const __grid_constant__ RowsParams p) {
    extern __shared__ __align__(128) uint8_t rows_smem[];
    const Ring g = carve(rows_smem, p);
    ring_init(g, p);
    ptx::grid_launch_dependents();
    ptx::grid_wait();
    if (threadIdx.x >= p.nt) {
        produce(g, p);
        return;
    }
    const int t = threadIdx.x, lane = t & 31, w = t >> 5, nwarps = p.nt >> 5;
    const int P = p.N >> 3;
    const size_t step = (size_t)p.nt * 16;
    // a thread reads only the gamma words that it writes here: no barrier.  (Not by non-coherent loads: the kernel before
    // may have been writing gamma when this one started, before grid_wait.)
#pragma unroll
    for (int k = 0; k < PPT; ++k) {
        const int pk = t + k * p.nt;
        if (pk < P) {
            reinterpret_cast<float4*>(g.extra)[pk * 2] = reinterpret_cast<const float4*>(p.gamma)[pk * 2];
            reinterpret_cast<float4*>(g.extra)[pk * 2 + 1] = reinterpret_cast<const float4*>(p.gamma)[pk * 2 + 1];
        }
    }
    Pack dg[PPT];
#pragma unroll
    for (int k = 0; k < PPT; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) dg[k][i] = 0ull;
    int s = 0, buf = 0;
    uint32_t ph = 0;
    for (int64_t row = blockIdx.x; row < p.M; row += gridDim.x, buf ^= 1) {
        Pack dy[ONE ? 1 : PPT];
        uint4 dv[ONE ? PPT : 1], hv[PPT], ev[PPT];  // one rank's dy stays packed
        uint64_t s1 = 0ull, s2 = 0ull;
#pragma unroll
        for (int k = 0; k < PPT; ++k) {
            if (k < p.slices) {
                const int pk = t + k * p.nt;
                ring_wait(&g.full[s], ph, g, p);
                const uint8_t* at = g.stage + (size_t)s * p.stage_bytes + t * 16;
                if (pk < P) {
                    Pack& d = dy[ONE ? 0 : k];
                    sum_ranks<ONE>(at, p.R, step, d);
                    if (ONE) dv[k] = *reinterpret_cast<const uint4*>(at);
                    hv[k] = *reinterpret_cast<const uint4*>(at + p.R * step);
                    if (p.has_res) ev[k] = *reinterpret_cast<const uint4*>(at + (p.R + 1) * step);
                    Pack h, gk;
                    unpack8(hv[k], h);
                    load8(g.extra + pk * 8, gk);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        s1 = fma2(h[i], h[i], s1);
                        s2 = fma2(mul2(d[i], gk[i]), h[i], s2);
                    }
                }
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(&g.empty[s]);
                if (++s == p.stages) { s = 0; ph ^= 1u; }
            }
        }
        float* red = g.red + buf * 64;
        const float c1 = warp_sum(both(s1)), c2 = warp_sum(both(s2));
        if (lane == 0) {
            red[w] = c1;
            red[32 + w] = c2;
        }
        consumer_bar(p.nt);
        const float inv = rsqrtf(red_total(red, nwarps) * p.inv_n + p.eps);
        const float m = inv * (red_total(red + 32, nwarps) * p.inv_n) * inv;  // inv^2 * mean(dy gamma h): dh = inv dy gamma - m (h inv) + d_res
        const uint64_t inv2 = pair(inv, inv), m2 = pair(-m, -m);
#pragma unroll
        for (int k = 0; k < PPT; ++k) {
            if (k < p.slices) {
                const int pk = t + k * p.nt;
                if (pk < P) {
                    Pack h, gk, e = {}, o;
                    unpack8(hv[k], h);
                    load8(g.extra + pk * 8, gk);
                    if (p.has_res) unpack8(ev[k], e);
                    Pack& d = dy[ONE ? 0 : k];
                    if (ONE) unpack8(dv[k], d);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint64_t xh = mul2(h[i], inv2);
                        o[i] = fma2(mul2(d[i], gk[i]), inv2, fma2(xh, m2, e[i]));
                        dg[k][i] = fma2(d[i], xh, dg[k][i]);
                    }
                    ptx::st_stream_v4(p.res_out + row * (int64_t)p.N + pk * 8, pack8(o));
                }
            }
        }
    }
    if (p.dgamma) {
        float* to = p.dgamma + (size_t)blockIdx.x * p.N;
#pragma unroll
        for (int k = 0; k < PPT; ++k) {
            const int pk = t + k * p.nt;
            if (pk < P) {
                const float2 a = unpair(dg[k][0]), b = unpair(dg[k][1]), c = unpair(dg[k][2]), d = unpair(dg[k][3]);
                *reinterpret_cast<float4*>(to + pk * 8) = make_float4(a.x, a.y, b.x, b.y);
                *reinterpret_cast<float4*>(to + pk * 8 + 4) = make_float4(c.x, c.y, d.x, d.y);
            }
        }
    }
}

// dgamma[j] = sum over the blocks' partial rows, in an order that the number of
// rows alone decides: 64 strands of every 64th row, then the strands.
// blockIdx.y: a second set of partial rows right behind the first (the LayerNorm's dbeta).
__global__ void __launch_bounds__(256) dgamma_sum_kernel(const float* part, float* dgamma, float* second, int rows, int N) {
    if (blockIdx.y) {
        part += (size_t)rows * N;
        dgamma = second;
    }
    __shared__ float4 sum[8][4];
    const int c = threadIdx.x & 3, strand = threadIdx.x >> 2;
    const int col = (blockIdx.x * 4 + c) * 4;
    ptx::grid_launch_dependents();
    ptx::grid_wait();
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    if (col < N) {
        float4 v[5];
        for (int r0 = strand; r0 < rows; r0 += 5 * 64) {
#pragma unroll
            for (int i = 0; i < 5; ++i)
                v[i] = r0 + i * 64 < rows ? __ldcg(reinterpret_cast<const float4*>(part + (size_t)(r0 + i * 64) * N + col))
                                          : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int i = 0; i < 5; ++i) {
                a.x += v[i].x; a.y += v[i].y; a.z += v[i].z; a.w += v[i].w;
            }
        }
    }
    for (int o = 4; o < 32; o <<= 1) {  // the 8 strands of a warp
        a.x += __shfl_xor_sync(0xFFFFFFFFu, a.x, o);
        a.y += __shfl_xor_sync(0xFFFFFFFFu, a.y, o);
        a.z += __shfl_xor_sync(0xFFFFFFFFu, a.z, o);
        a.w += __shfl_xor_sync(0xFFFFFFFFu, a.w, o);
    }
    if ((threadIdx.x & 31) < 4) sum[threadIdx.x >> 5][c] = a;
    __syncthreads();
    if (threadIdx.x < 16) {
        const int out = blockIdx.x * 16 + threadIdx.x;
        float t = 0.f;
        for (int w = 0; w < 8; ++w) t += reinterpret_cast<const float*>(sum[w])[threadIdx.x];
        if (out < N) dgamma[out] = t;
    }
}

// Packs a thread holds, of a row of P.  Forward: about 256 threads a block.
// Backward, whose state is 24 registers a pack (20 with one rank): up to 256
// threads, two blocks an SM; above, as few packs as 16 warps allow, which may
// have 128 registers each (17 warps: 96) in one block an SM.  R = 3,
// 1001 x 5000: two packs 16 us, three in two blocks an SM 17; R = 8,
// 4096 x 7168: two packs 97 us, four in two blocks 102; R = 4, 2048 x 10240:
// three packs 51 us, in 17 warps 71, eight 81; 2048 x 16384: five packs 106 us,
// four in 17 warps 115, eight 132.
// With no more rows than SMs a block has its SM alone, and a forward row takes
// up to 512 threads (R = 8, 7168 columns: one row 3.9 us, with 224 threads 5.4;
// 152 rows 4.5 and 5.7.  Backward it costs: R = 4, 150 x 4096: 6.1 us, with 256
// threads 5.4).
int packs_per_thread(int P, bool alone) {
    if (alone && P <= 1024) return P <= 512 ? 1 : 2;
    return P <= 256 ? 1 : P <= 512 ? 2 : P <= 2048 ? 4 : 8;
}
int backward_packs_per_thread(int P) { return P <= 256 ? 1 : P <= 960 ? 2 : P <= 1440 ? 3 : P <= 1920 ? 4 : 5; }

}  // namespace

cudaLaunchAttribute dependent_launch() {
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    return attr;
}

RowsPlan rows_plan(RowsParams& p, int num_sms) {
    const int P = p.N / 8;
    p.extra_words = p.backward ? p.N : 0;
    p.red_words = 2 * 2 * 32;  // [buffer][statistic][warp]
    return rows_shape(p, p.backward ? backward_packs_per_thread(P) : packs_per_thread(P, p.M <= num_sms), num_sms);
}

// The kernel of a plan: blocks of up to 288 threads leave room for two on an SM.
template <bool POW2>
void (*quant_kernel(int ppt, int threads))(RowsParams) {
    switch (ppt) {
        case 1: return threads <= 288 ? norm_quant_rows_kernel<1, POW2, 288, 2> : norm_quant_rows_kernel<1, POW2, 544, 1>;
        case 2: return threads <= 288 ? norm_quant_rows_kernel<2, POW2, 288, 2> : norm_quant_rows_kernel<2, POW2, 544, 1>;
        case 4: return threads <= 288 ? norm_quant_rows_kernel<4, POW2, 288, 2> : norm_quant_rows_kernel<4, POW2, 544, 1>;
        default: return norm_quant_rows_kernel<8, POW2, 544, 1>;
    }
}

template <bool ONE>
void (*backward_kernel(int ppt, int threads))(RowsParams) {
    switch (ppt) {
        case 1: return norm_backward_rows_kernel<1, ONE, 288, 2>;
        case 2: return threads <= 288 ? norm_backward_rows_kernel<2, ONE, 288, 2> : norm_backward_rows_kernel<2, ONE, 512, 1>;
        case 3: return norm_backward_rows_kernel<3, ONE, 512, 1>;
        case 4: return norm_backward_rows_kernel<4, ONE, 512, 1>;
        default: return norm_backward_rows_kernel<5, ONE, 512, 1>;
    }
}

cudaError_t rows_prepare() {
    cudaError_t e = cudaSuccess;
    for (int ppt : {1, 2, 4, 8})
        for (int threads : {288, 544}) {
            if (e == cudaSuccess) e = opt_in(quant_kernel<false>(ppt, threads));
            if (e == cudaSuccess) e = opt_in(quant_kernel<true>(ppt, threads));
        }
    for (int ppt : {1, 2, 3, 4, 5})
        for (int threads : {288, 512})
            for (bool one : {false, true})
                if (e == cudaSuccess)
                    e = opt_in(one ? backward_kernel<true>(ppt, threads) : backward_kernel<false>(ppt, threads));
    return e;
}

cudaError_t launch_norm_quant_rows(const RowsParams& p, const RowsPlan& plan, bool pow2, cudaStream_t s) {
    auto* kernel = pow2 ? quant_kernel<true>(plan.ppt, plan.threads) : quant_kernel<false>(plan.ppt, plan.threads);
    return launch_dependent(kernel, plan.grid, plan.threads, plan.smem, s, p);
}

cudaError_t launch_row_sums(const float* part, float* first, float* second, int rows, int N, cudaStream_t s) {
    return launch_dependent(dgamma_sum_kernel, dim3((N + 15) / 16, second ? 2 : 1), 256, 0, s, part, first, second, rows, N);
}

cudaError_t launch_norm_backward_rows(RowsParams& p, const RowsPlan& plan, float* scratch, float* dgamma,
                                      cudaStream_t s) {
    // a single block's sums are the result
    p.dgamma = dgamma == nullptr ? nullptr : plan.grid == 1 ? dgamma : scratch;
    auto* kernel = p.R == 1 ? backward_kernel<true>(plan.ppt, plan.threads) : backward_kernel<false>(plan.ppt, plan.threads);
    cudaError_t e = launch_dependent(kernel, plan.grid, plan.threads, plan.smem, s, p);
    if (e == cudaSuccess && dgamma != nullptr && plan.grid > 1)
        e = launch_row_sums(scratch, dgamma, nullptr, plan.grid, p.N, s);
    return e;
}

size_t norm_backward_scratch_words(int64_t n_max, int num_sms) {
    // rows of N from an SM's blocks.  rows_plan fits kRowsThreads / (nt + 32) of them, ten at most: with a pack a thread,
    // N <= 8 nt, less than 8 * kRowsThreads columns; with two, N > 2048 and nt >= 160, three blocks at most and less than
    // twice that
    const int64_t n = n_max < kBackwardMaxN ? n_max : kBackwardMaxN, most = 8 * kRowsThreads;
    return (size_t)std::max(std::max(2 * n, std::min(3 * n, 2 * most)), std::min(kRowsThreads / 64 * n, most)) * num_sms;
}

}  // namespace are
