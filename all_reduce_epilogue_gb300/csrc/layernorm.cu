// All-reduce + residual add + LayerNorm and its backward pass, on the row-streaming
// scheme of the RMSNorm's (norm_rows.cu).
//
// Forward, per row (partials x_r, residual e, width N):
//   h = sum_{r=0..R-1} x_r + e        (fp32, r ascending from +0.0)
//   y = (h - mean) * rsqrt(var + eps) * gamma + beta,   var = mean((h - mean)^2)
// Backward (dy = sum_r dy_r, g = dy * gamma, xhat = (h - mean) * inv):
//   dh     = inv * (g - mean(g) - xhat * mean(g * xhat)) + d_res
//   dgamma = sum_i dy_i * xhat_i,  dbeta = sum_i dy_i
//
// The variance is a sum of squares around the mean, not mean(h^2) - mean^2, which
// loses a row whose mean is large against its spread.  It takes one exchange over the
// block all the same: a warp sums its columns, takes the squares (and the products
// with g) around its own mean m_w, and the block joins the warps' sums,
//   sum (h - mean)^2 = sum_w Q_w + n_w (m_w - mean)^2,
//   sum g (h - mean) = sum_w C_w + G_w (m_w - mean)
// (Chan, Golub and LeVeque 1979): shuffles within the warp instead of a second
// barrier of the block.
#include <algorithm>

#include "rows.cuh"

namespace are {
namespace {

constexpr int kStat = 32;                     // words of one statistic: one a warp
constexpr int kRedSet = 4 * kStat;            // words of one exchange
constexpr int kRedAll = 2 * kRedSet + 2 * kStat;  // two exchanges in turn, the warps' columns and their reciprocals

// Columns that warp w owns.
__device__ __forceinline__ int warp_columns(int w, const RowsParams& p) {
    const int P = p.N >> 3;
    int n = 0;
    for (int k = 0; k < p.slices; ++k) {
        const int left = P - (w * 32 + k * p.nt);
        n += left < 0 ? 0 : left > 32 ? 32 : left;
    }
    return n * 8;
}

// Words behind the last warp stay zero, so the joins may run over whole float4s.
__device__ __forceinline__ void init_columns(const Ring& g, const RowsParams& p) {
    if (threadIdx.x < (unsigned)(p.nt >> 5)) {
        const float n = (float)warp_columns(threadIdx.x, p);
        g.red[2 * kRedSet + threadIdx.x] = n;
        g.red[2 * kRedSet + kStat + threadIdx.x] = 1.f / n;
    }
    __syncthreads();
}

__device__ __forceinline__ float quad(const float4& v) { return (v.x + v.y) + (v.z + v.w); }

// The row's mean from the warps' sums.
__device__ __forceinline__ float join_mean(const float* red, int nwarps, float inv_n) {
    float t = 0.f;
    for (int w = 0; w < nwarps; w += 4) t += quad(*reinterpret_cast<const float4*>(red + w));
    return t * inv_n;
}

__device__ __forceinline__ float4 at4(const float* p) { return *reinterpret_cast<const float4*>(p); }

// sum (h - mean)^2 from the warps' sums S, squares Q around their own means, and columns n (1/n).
__device__ __forceinline__ float join_squares(const float* S, const float* Q, const float* n, int nwarps, float mean) {
    float t = 0.f;
    for (int w = 0; w < nwarps; w += 4) {
        const float4 s = at4(S + w), q = at4(Q + w), c = at4(n + w), r = at4(n + kStat + w);
        const float a = fmaf(s.x, r.x, -mean), b = fmaf(s.y, r.y, -mean), d = fmaf(s.z, r.z, -mean), e = fmaf(s.w, r.w, -mean);
        t += (fmaf(c.x * a, a, q.x) + fmaf(c.y * b, b, q.y)) + (fmaf(c.z * d, d, q.z) + fmaf(c.w * e, e, q.w));
    }
    return t;
}

// sum g (h - mean) from the warps' G = sum g and C = sum g (h - m_w).
__device__ __forceinline__ float join_products(const float* S, const float* G, const float* C, const float* n, int nwarps,
                                               float mean) {
    float t = 0.f;
    for (int w = 0; w < nwarps; w += 4) {
        const float4 s = at4(S + w), g = at4(G + w), c = at4(C + w), r = at4(n + kStat + w);
        t += (fmaf(g.x, fmaf(s.x, r.x, -mean), c.x) + fmaf(g.y, fmaf(s.y, r.y, -mean), c.y)) +
             (fmaf(g.z, fmaf(s.z, r.z, -mean), c.z) + fmaf(g.w, fmaf(s.w, r.w, -mean), c.w));
    }
    return t;
}

// ---------------------------------------------------------------------- forward
// Where gamma and beta come from: registers (up to two packs a thread), gamma from
// registers and beta from shared memory (four), both from the caches (eight).
template <int PPT, int THREADS, int BLOCKS>
__global__ void __launch_bounds__(THREADS, BLOCKS) layernorm_rows_kernel(const __grid_constant__ RowsParams p) {
    extern __shared__ __align__(128) uint8_t rows_smem[];
    const Ring g = carve(rows_smem, p);
    ring_init(g, p);
    init_columns(g, p);
    ptx::grid_launch_dependents();
    ptx::grid_wait();
    if (threadIdx.x >= p.nt) {
        produce(g, p);
        return;
    }
    const int t = threadIdx.x, lane = t & 31, w = t >> 5, nwarps = p.nt >> 5;
    const int P = p.N >> 3;
    const size_t step = (size_t)p.nt * 16;
    constexpr bool kGammaRegs = PPT <= 4, kBetaRegs = PPT <= 2, kBetaShared = PPT == 4;
    const float* cols = g.red + 2 * kRedSet;
    const float inv_cols = cols[kStat + w];
    Pack gam[kGammaRegs ? PPT : 1], bet[kBetaRegs ? PPT : 1];
#pragma unroll
    for (int k = 0; k < PPT; ++k) {
        const int pk = t + k * p.nt;
        if (kGammaRegs && pk < P) load8(p.gamma + pk * 8, gam[k]);
        if (kBetaRegs && pk < P) {
#pragma unroll
            for (int i = 0; i < 4; ++i) bet[k][i] = 0ull;
            if (p.beta) load8(p.beta + pk * 8, bet[k]);
        }
        // a thread reads only the words that it writes here: no barrier
        if (kBetaShared && pk < P) {
            const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
            float4* to = reinterpret_cast<float4*>(g.extra) + pk * 2;
            to[0] = p.beta ? reinterpret_cast<const float4*>(p.beta)[pk * 2] : zero;
            to[1] = p.beta ? reinterpret_cast<const float4*>(p.beta)[pk * 2 + 1] : zero;
        }
    }
    int s = 0, buf = 0;
    uint32_t ph = 0;
    for (int64_t row = blockIdx.x; row < p.M; row += gridDim.x, buf ^= 1) {
        Pack h[PPT];
        uint64_t sum2 = 0ull;
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
                    for (int i = 0; i < 4; ++i) sum2 = add2(h[k][i], sum2);
                }
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(&g.empty[s]);
                if (++s == p.stages) { s = 0; ph ^= 1u; }
                if (p.res_out && pk < P) ptx::st_stream_v4(p.res_out + row * (int64_t)p.N + pk * 8, pack8(h[k]));
            }
        }
        float* red = g.red + buf * kRedSet;
        const float S = warp_sum(both(sum2));
        const float own = S * inv_cols;  // the warp's mean
        const uint64_t own2 = pair(-own, -own);
        uint64_t q2 = 0ull;
#pragma unroll
        for (int k = 0; k < PPT; ++k) {
            if (k < p.slices && t + k * p.nt < P) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint64_t c = add2(h[k][i], own2);
                    q2 = fma2(c, c, q2);
                }
            }
        }
        const float Q = warp_sum(both(q2));
        if (lane == 0) {
            red[w] = S;
            red[kStat + w] = Q;
        }
        consumer_bar(p.nt);
        const float mean = join_mean(red, nwarps, p.inv_n);
        const float inv = rsqrtf(join_squares(red, red + kStat, cols, nwarps, mean) * p.inv_n + p.eps);
        const uint64_t mean2 = pair(-mean, -mean), inv2 = pair(inv, inv);
#pragma unroll
        for (int k = 0; k < PPT; ++k) {
            if (k < p.slices) {
                const int pk = t + k * p.nt;
                if (pk < P) {
                    Pack gk, bk, o;
                    if (kGammaRegs) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) gk[i] = gam[kGammaRegs ? k : 0][i];
                    } else {
                        load8(p.gamma + pk * 8, gk);
                    }
                    if (kBetaRegs) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) bk[i] = bet[kBetaRegs ? k : 0][i];
                    } else if (kBetaShared) {
                        load8(g.extra + pk * 8, bk);
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i) bk[i] = 0ull;
                        if (p.beta) load8(p.beta + pk * 8, bk);
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[i] = fma2(mul2(add2(h[k][i], mean2), inv2), gk[i], bk[i]);
                    ptx::st_stream_v4(p.out + row * (int64_t)p.N + pk * 8, pack8(o));
                }
            }
        }
    }
}

// --------------------------------------------------------------------- backward
// dbeta's sums: in registers up to two packs a thread, above in the thread's own words
// of shared memory (with dgamma's they would not fit the 128 registers of 16 warps).
template <int PPT, bool ONE, int THREADS, int BLOCKS>
__global__ void __launch_bounds__(THREADS, BLOCKS) layernorm_backward_rows_kernel(const __grid_constant__ RowsParams p) {
    extern __shared__ __align__(128) uint8_t rows_smem[];
    const Ring g = carve(rows_smem, p);
    ring_init(g, p);
    init_columns(g, p);
    ptx::grid_launch_dependents();
    ptx::grid_wait();
    if (threadIdx.x >= p.nt) {
        produce(g, p);
        return;
    }
    const int t = threadIdx.x, lane = t & 31, w = t >> 5, nwarps = p.nt >> 5;
    const int P = p.N >> 3;
    const size_t step = (size_t)p.nt * 16;
    constexpr bool kRegs = PPT <= 2;
    const float* cols = g.red + 2 * kRedSet;
    const float inv_cols = cols[kStat + w];
    float* const beta_sums = g.extra + p.N;
    // a thread reads only the words that it writes here: no barrier
    Pack dg[PPT], db[kRegs ? PPT : 1];
#pragma unroll
    for (int k = 0; k < PPT; ++k) {
        const int pk = t + k * p.nt;
#pragma unroll
        for (int i = 0; i < 4; ++i) dg[k][i] = 0ull;
        if (kRegs) {
#pragma unroll
            for (int i = 0; i < 4; ++i) db[kRegs ? k : 0][i] = 0ull;
        }
        if (pk < P) {
            reinterpret_cast<float4*>(g.extra)[pk * 2] = reinterpret_cast<const float4*>(p.gamma)[pk * 2];
            reinterpret_cast<float4*>(g.extra)[pk * 2 + 1] = reinterpret_cast<const float4*>(p.gamma)[pk * 2 + 1];
            if (!kRegs) {
                reinterpret_cast<float4*>(beta_sums)[pk * 2] = make_float4(0.f, 0.f, 0.f, 0.f);
                reinterpret_cast<float4*>(beta_sums)[pk * 2 + 1] = make_float4(0.f, 0.f, 0.f, 0.f);
            }
        }
    }
    int s = 0, buf = 0;
    uint32_t ph = 0;
    for (int64_t row = blockIdx.x; row < p.M; row += gridDim.x, buf ^= 1) {
        Pack dy[ONE ? 1 : PPT];
        uint4 dv[ONE ? PPT : 1], hv[PPT], ev[PPT];  // one rank's dy stays packed
        uint64_t sum2 = 0ull;
#pragma unroll
        for (int k = 0; k < PPT; ++k) {
            if (k < p.slices) {
                const int pk = t + k * p.nt;
                ring_wait(&g.full[s], ph, g, p);
                const uint8_t* at = g.stage + (size_t)s * p.stage_bytes + t * 16;
                if (pk < P) {
                    if (ONE) dv[k] = *reinterpret_cast<const uint4*>(at);
                    else sum_ranks<false>(at, p.R, step, dy[ONE ? 0 : k]);
                    hv[k] = *reinterpret_cast<const uint4*>(at + p.R * step);
                    if (p.has_res) ev[k] = *reinterpret_cast<const uint4*>(at + (p.R + 1) * step);
                    Pack h;
                    unpack8(hv[k], h);
#pragma unroll
                    for (int i = 0; i < 4; ++i) sum2 = add2(h[i], sum2);
                }
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(&g.empty[s]);
                if (++s == p.stages) { s = 0; ph ^= 1u; }
            }
        }
        float* red = g.red + buf * kRedSet;
        const float S = warp_sum(both(sum2));
        const float own = S * inv_cols;  // the warp's mean
        const uint64_t own2 = pair(-own, -own);
        uint64_t q2 = 0ull, g2 = 0ull, c2 = 0ull;
#pragma unroll
        for (int k = 0; k < PPT; ++k) {
            if (k < p.slices && t + k * p.nt < P) {
                Pack h, gk;
                unpack8(hv[k], h);
                load8(g.extra + (t + k * p.nt) * 8, gk);
                Pack& d = dy[ONE ? 0 : k];
                if (ONE) unpack8(dv[k], d);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint64_t c = add2(h[i], own2), gi = mul2(d[i], gk[i]);
                    q2 = fma2(c, c, q2);
                    g2 = add2(gi, g2);
                    c2 = fma2(gi, c, c2);
                }
            }
        }
        const float Q = warp_sum(both(q2)), G = warp_sum(both(g2)), C = warp_sum(both(c2));
        if (lane == 0) {
            red[w] = S;
            red[kStat + w] = Q;
            red[2 * kStat + w] = G;
            red[3 * kStat + w] = C;
        }
        consumer_bar(p.nt);
        const float mean = join_mean(red, nwarps, p.inv_n);
        const float inv = rsqrtf(join_squares(red, red + kStat, cols, nwarps, mean) * p.inv_n + p.eps);
        const float a = join_mean(red + 2 * kStat, nwarps, p.inv_n);  // mean(g)
        const float b = join_products(red, red + 2 * kStat, red + 3 * kStat, cols, nwarps, mean) * p.inv_n * inv;  // mean(g xhat)
        const uint64_t mean2 = pair(-mean, -mean), inv2 = pair(inv, inv), b2 = pair(-inv * b, -inv * b),
                       a2 = pair(-a, -a);
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
                        const uint64_t xh = mul2(add2(h[i], mean2), inv2);
                        o[i] = fma2(fma2(d[i], gk[i], a2), inv2, fma2(xh, b2, e[i]));
                        dg[k][i] = fma2(d[i], xh, dg[k][i]);
                        if (kRegs) db[kRegs ? k : 0][i] = add2(db[kRegs ? k : 0][i], d[i]);
                    }
                    ptx::st_stream_v4(p.res_out + row * (int64_t)p.N + pk * 8, pack8(o));
                    if (!kRegs && p.dbeta) {
                        Pack v;
                        load8(beta_sums + pk * 8, v);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            reinterpret_cast<uint64_t*>(beta_sums + pk * 8)[i] = add2(v[i], d[i]);
                    }
                }
            }
        }
    }
#pragma unroll
    for (int k = 0; k < PPT; ++k) {
        const int pk = t + k * p.nt;
        if (pk < P) {
            const size_t at = (size_t)blockIdx.x * p.N + pk * 8;
            if (p.dgamma) {
#pragma unroll
                for (int i = 0; i < 4; ++i) reinterpret_cast<uint64_t*>(p.dgamma + at)[i] = dg[k][i];
            }
            if (p.dbeta) {
                Pack v;
                if (!kRegs) load8(beta_sums + pk * 8, v);
#pragma unroll
                for (int i = 0; i < 4; ++i) reinterpret_cast<uint64_t*>(p.dbeta + at)[i] = kRegs ? db[kRegs ? k : 0][i] : v[i];
            }
        }
    }
}

// Packs a thread holds, of a row of P: as the RMSNorm's kernels, whose registers these have.
int packs_per_thread(int P, bool alone) {
    if (alone && P <= 1024) return P <= 512 ? 1 : 2;
    return P <= 256 ? 1 : P <= 512 ? 2 : P <= 2048 ? 4 : 8;
}
int backward_packs_per_thread(int P) { return P <= 256 ? 1 : P <= 960 ? 2 : P <= 1440 ? 3 : P <= 1920 ? 4 : 5; }

// The kernel of a plan: blocks of up to 288 threads leave room for two on an SM.
void (*forward_kernel(int ppt, int threads))(RowsParams) {
    switch (ppt) {
        case 1: return threads <= 288 ? layernorm_rows_kernel<1, 288, 2> : layernorm_rows_kernel<1, 544, 1>;
        case 2: return threads <= 288 ? layernorm_rows_kernel<2, 288, 2> : layernorm_rows_kernel<2, 544, 1>;
        case 4: return threads <= 288 ? layernorm_rows_kernel<4, 288, 2> : layernorm_rows_kernel<4, 544, 1>;
        default: return layernorm_rows_kernel<8, 544, 1>;
    }
}

template <bool ONE>
void (*backward_kernel(int ppt, int threads))(RowsParams) {
    switch (ppt) {
        case 1: return layernorm_backward_rows_kernel<1, ONE, 288, 2>;
        case 2:
            return threads <= 288 ? layernorm_backward_rows_kernel<2, ONE, 288, 2> : layernorm_backward_rows_kernel<2, ONE, 512, 1>;
        case 3: return layernorm_backward_rows_kernel<3, ONE, 512, 1>;
        case 4: return layernorm_backward_rows_kernel<4, ONE, 512, 1>;
        default: return layernorm_backward_rows_kernel<5, ONE, 512, 1>;
    }
}

}  // namespace

RowsPlan layernorm_plan(RowsParams& p, int num_sms) {
    const int P = p.N / 8;
    const int ppt = p.backward ? backward_packs_per_thread(P) : packs_per_thread(P, p.M <= num_sms);
    p.extra_words = p.backward ? (ppt <= 2 ? p.N : 2 * p.N) : ppt == 4 ? p.N : 0;
    p.red_words = kRedAll;
    return rows_shape(p, ppt, num_sms);
}

cudaError_t layernorm_prepare() {
    cudaError_t e = cudaSuccess;
    for (int ppt : {1, 2, 4, 8})
        for (int threads : {288, 544})
            if (e == cudaSuccess) e = opt_in(forward_kernel(ppt, threads));
    for (int ppt : {1, 2, 3, 4, 5})
        for (int threads : {288, 512})
            for (bool one : {false, true})
                if (e == cudaSuccess)
                    e = opt_in(one ? backward_kernel<true>(ppt, threads) : backward_kernel<false>(ppt, threads));
    return e;
}

cudaError_t launch_layernorm_rows(const RowsParams& p, const RowsPlan& plan, cudaStream_t s) {
    return launch_dependent(forward_kernel(plan.ppt, plan.threads), plan.grid, plan.threads, plan.smem, s, p);
}

cudaError_t launch_layernorm_backward_rows(RowsParams& p, const RowsPlan& plan, float* scratch, float* dgamma, float* dbeta,
                                           cudaStream_t s) {
    // a single block's sums are the results; otherwise dbeta's partial rows lie right behind dgamma's
    const bool one = plan.grid == 1;
    float* const second = scratch + (dgamma ? (size_t)plan.grid * p.N : 0);
    p.dgamma = dgamma == nullptr ? nullptr : one ? dgamma : scratch;
    p.dbeta = dbeta == nullptr ? nullptr : one ? dbeta : second;
    auto* kernel = p.R == 1 ? backward_kernel<true>(plan.ppt, plan.threads) : backward_kernel<false>(plan.ppt, plan.threads);
    cudaError_t e = launch_dependent(kernel, plan.grid, plan.threads, plan.smem, s, p);
    if (e == cudaSuccess && !one && (dgamma || dbeta))
        e = launch_dependent(dgamma_sum_kernel, dim3((p.N + 15) / 16, dgamma && dbeta ? 2 : 1), 256, 0, s, scratch,
                             dgamma ? dgamma : dbeta, dbeta, plan.grid, p.N);
    return e;
}

}  // namespace are
