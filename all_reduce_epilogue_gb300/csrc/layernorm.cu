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
// The forward pass's variance is a sum of squares around the mean, not mean(h^2) -
// mean^2, which loses a row whose mean is large against its spread.  It takes one
// exchange over the block all the same: a warp sums its columns, takes the squares
// around its own mean m_w, and the block joins the warps' sums,
//   sum (h - mean)^2 = sum_w Q_w + n_w (m_w - mean)^2
// (Chan, Golub and LeVeque 1979): shuffles within the warp instead of a second
// barrier of the block.
//
// Bound by HBM, as the RMSNorm's: every input once, every output once.  Measured (a
// copy moves 6.78 TB/s): forward, R = 8, 4096 x 7168: 98 us, 6.6 TB/s; R = 1,
// 16384 x 4096: 89 us, 6.0 TB/s, x 768: 21 us, 4.8 TB/s, x 64: 3.2 us; one row of 7168, R = 8:
// 4.1 us, all latency.  Backward, R = 1, 16384 x 7168: 153 us, 6.1 TB/s, x 4096:
// 93 us, 5.8 TB/s, x 768: 34 us, 3.0 TB/s (a row's exchange and joins for one pack a
// thread), x 264: 18 us, x 64: 9.4; R = 3, 1001 x 5000: 16.8 us, 6.6 rows an SM and 4 us for the sums of the
// blocks' partial rows.
#include <algorithm>

#include "rows.cuh"

namespace are {
namespace {

constexpr int kRedWarps = 32;
constexpr int kWarps = 16;                  // backward: warps of a block, at most
constexpr int kRedAll = 2 * kRedWarps * 4;  // two exchanges in turn: forward two sums a warp, backward up to six
static_assert(2 * 6 * kWarps <= kRedAll, "words of an exchange");

// The join is spread over a warp's lanes: lane l has the sums of warp l modulo `ways`, the
// power of two that holds the block's warps, so sums over `ways` neighbouring lanes are
// the block's, in every lane.  (A thread that ran through all the warps' sums by itself took
// 28 % of the backward kernel's instructions at 4096 columns.)
struct Join {
    int ways;
    float n, inv_n;    // this lane's warp's columns, 0 behind the last warp
    float own_inv_n;   // the reciprocal of the thread's own warp's
};

__device__ __forceinline__ Join make_join(const RowsParams& p) {
    const int lane = threadIdx.x & 31, nwarps = p.nt >> 5, P = p.N >> 3;
    Join j;
    j.ways = 1;
    while (j.ways < nwarps) j.ways <<= 1;
    const int w = lane & (j.ways - 1);
    int n = 0;
    if (w < nwarps) {
        for (int k = 0; k < p.slices; ++k) {
            const int left = P - (w * 32 + k * p.nt);
            n += left < 0 ? 0 : left > 32 ? 32 : left;
        }
    }
    j.n = (float)(n * 8);
    j.inv_n = n ? 1.f / j.n : 0.f;
    j.own_inv_n = __shfl_sync(0xFFFFFFFFu, j.inv_n, threadIdx.x >> 5);
    return j;
}

__device__ __forceinline__ float join_sum(float v, int ways) {
    for (int o = 1; o < ways; o <<= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// ---------------------------------------------------------------------- forward
// Where gamma and beta come from: registers (up to two packs a thread), gamma from
// registers and beta from shared memory (three, four), both from the caches (eight).
template <int PPT, int THREADS, int BLOCKS>
__global__ void __launch_bounds__(THREADS, BLOCKS) layernorm_rows_kernel(const __grid_constant__ RowsParams p) {
    extern __shared__ __align__(128) uint8_t rows_smem[];
    const Ring g = carve(rows_smem, p);
    ring_init(g, p);
    ptx::grid_launch_dependents();
    ptx::grid_wait();
    if (threadIdx.x >= p.nt) {
        produce(g, p);
        return;
    }
    const int t = threadIdx.x, lane = t & 31, w = t >> 5;
    const int P = p.N >> 3;
    const size_t step = (size_t)p.nt * 16;
    constexpr bool kGammaRegs = PPT <= 4, kBetaRegs = PPT <= 2, kBetaShared = PPT == 3 || PPT == 4;
    const Join join = make_join(p);
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
        float2* red = reinterpret_cast<float2*>(g.red) + buf * kRedWarps;
        const float S = warp_sum(both(sum2));
        const float own = S * join.own_inv_n;  // the warp's mean
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
        if (lane == 0) red[w] = make_float2(S, Q);
        consumer_bar(p.nt);
        const float2 v = red[lane & (join.ways - 1)];
        const float mean = join_sum(v.x, join.ways) * p.inv_n;
        const float off = fmaf(v.x, join.inv_n, -mean);
        const float inv = rsqrtf(join_sum(fmaf(join.n * off, off, v.y), join.ways) * p.inv_n + p.eps);
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

// Rows of up to 1024 columns, many of them (see narrow()): 8, 16 or 32 lanes take a row each, so a row costs no barrier and no
// turn of a ring, and an SM has up to 128 rows in flight.
constexpr int kNarrowWarps = 8;

template <int PPT>
__global__ void __launch_bounds__(kNarrowWarps * 32, PPT <= 2 ? 4 : 3) layernorm_narrow_kernel(const __grid_constant__ RowsParams p) {
    const int lane = threadIdx.x & 31, G = p.lanes, l = lane & (G - 1), P = p.N >> 3, per_warp = 32 / G;
    ptx::grid_launch_dependents();
    ptx::grid_wait();
    const int64_t warps = (int64_t)gridDim.x * kNarrowWarps;
    for (int64_t w = (int64_t)blockIdx.x * kNarrowWarps + (threadIdx.x >> 5); w * per_warp < p.M; w += warps) {
        const int64_t row = w * per_warp + lane / G;
        const bool there = row < p.M;  // (all lanes stay for the exchanges)
        Pack h[PPT];
        uint64_t sum2 = 0ull;
        const int64_t at = row * p.N + l * 8;
        auto load = [&](const uint16_t* from, int k) {
            return there && l + k * G < P ? ptx::ld_stream_v4(from + at + k * G * 8) : make_uint4(0u, 0u, 0u, 0u);
        };
        {
            uint4 v[PPT];
#pragma unroll
            for (int k = 0; k < PPT; ++k) v[k] = load(p.src[0], k);
            // the ranks in turn, a rank's loads under the additions of the one before
            for (int r = 1; r < p.nsrc; ++r) {
                uint4 next[PPT];
#pragma unroll
                for (int k = 0; k < PPT; ++k) next[k] = load(p.src[r], k);
#pragma unroll
                for (int k = 0; k < PPT; ++k) {
                    Pack f;
                    unpack8(v[k], f);
#pragma unroll
                    for (int i = 0; i < 4; ++i) h[k][i] = r == 1 ? f[i] : add2(h[k][i], f[i]);
                    if (p.has_res && r == p.nsrc - 1) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) h[k][i] = add2(h[k][i], 0ull);  // a sum of -0.0 counts as +0.0
                    }
                    v[k] = next[k];
                }
            }
#pragma unroll
            for (int k = 0; k < PPT; ++k) {
                Pack f;
                unpack8(v[k], f);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    h[k][i] = p.nsrc == 1 ? f[i] : add2(h[k][i], f[i]);
                    if (!p.has_res) h[k][i] = add2(h[k][i], 0ull);
                    sum2 = add2(h[k][i], sum2);
                }
            }
        }
        if (p.res_out && there) {
#pragma unroll
            for (int k = 0; k < PPT; ++k)
                if (l + k * G < P) ptx::st_stream_v4(p.res_out + at + k * G * 8, pack8(h[k]));
        }
        float sum = both(sum2);
        for (int o = 1; o < G; o <<= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
        const float mean = sum * p.inv_n;
        const uint64_t mean2 = pair(-mean, -mean);
        uint64_t q2 = 0ull;
#pragma unroll
        for (int k = 0; k < PPT; ++k) {
            if (l + k * G < P) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    h[k][i] = add2(h[k][i], mean2);
                    q2 = fma2(h[k][i], h[k][i], q2);
                }
            }
        }
        float q = both(q2);
        for (int o = 1; o < G; o <<= 1) q += __shfl_xor_sync(0xFFFFFFFFu, q, o);
        const float inv = rsqrtf(q * p.inv_n + p.eps);
        const uint64_t inv2 = pair(inv, inv);
        if (there) {
#pragma unroll
            for (int k = 0; k < PPT; ++k) {
                if (l + k * G < P) {
                    Pack g, b = {}, o;
                    load8(p.gamma + (l + k * G) * 8, g);
                    if (p.beta) load8(p.beta + (l + k * G) * 8, b);
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[i] = fma2(mul2(h[k][i], inv2), g[i], b[i]);
                    ptx::st_stream_v4(p.out + at + k * G * 8, pack8(o));
                }
            }
        }
    }
}

// --------------------------------------------------------------------- backward
// The backward pass needs four sums a row, and takes them in one pass: H = sum h,
// Q = sum h^2, G = sum g, C = sum g h, from which mean = H / N, var = Q / N - mean^2 and
// sum g (h - mean) = C - mean G.  Where the mean is large against the spread these
// differences lose what the terms have: a row with mean^2 > 4 var takes Q and C again,
// around the mean, from the registers that still hold it (one more exchange; the same row
// always does, whatever its neighbours are).  Elsewhere the differences cost at most a factor
// of 5 of the sums' relative error, 2^-21 or so.
constexpr float kSpread = 4.f;

template <int N>
struct Reduced {
    // Sums of N (a power of two) values over the warp; lane l ends up with the sum of value l / (32 / N).
    // With each of the first steps a lane sends half of what it has and keeps the other half.
    static __device__ __forceinline__ float run(float (&v)[N]) {
        const int lane = threadIdx.x & 31;
        int o = 16;
#pragma unroll
        for (int n = N; n > 1; n >>= 1, o >>= 1) {
            const bool upper = lane & o;
#pragma unroll
            for (int i = 0; i < n / 2; ++i)
                v[i] = (upper ? v[i + n / 2] : v[i]) + __shfl_xor_sync(0xFFFFFFFFu, upper ? v[i] : v[i + n / 2], o);
        }
        float t = v[0];
        for (; o > 0; o >>= 1) t += __shfl_xor_sync(0xFFFFFFFFu, t, o);
        return t;
    }
};

// The block's sums of a row, in every thread, from what its warps left: `at[s * step + w]`, statistic s of warp w,
// zero behind the last warp; eight lanes add up each statistic.
struct RowSums {
    float Q, G, C, H;
};
__device__ __forceinline__ RowSums block_sums(const float* at, int step, int nwarps) {
    const int lane = threadIdx.x & 31;
    const float* mine = at + (lane >> 3) * step + (lane & 7);
    float v = mine[0];
    if (nwarps > 8) v += mine[8];
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return RowSums{__shfl_sync(0xFFFFFFFFu, v, 0), __shfl_sync(0xFFFFFFFFu, v, 8), __shfl_sync(0xFFFFFFFFu, v, 16),
                   __shfl_sync(0xFFFFFFFFu, v, 24)};
}

// What a row's outputs need: dh = inv * (g - a) - (h - mean) * inv * b + d_res, as pairs.
struct RowCoefs {
    uint64_t mean2, inv2, a2, b2;
};
__device__ __forceinline__ RowCoefs row_coefs(float mean, float var, float a, float products, const RowsParams& p) {
    const float inv = rsqrtf(var + p.eps), b = -inv * (products * p.inv_n * inv);
    return RowCoefs{pair(-mean, -mean), pair(inv, inv), pair(-a, -a), pair(b, b)};
}

// The four sums' terms of one pack, and Q's and C's around the mean.
__device__ __forceinline__ void add_terms(const Pack& h, const Pack& d, const Pack& g, uint64_t& Q, uint64_t& G, uint64_t& C,
                                          uint64_t& H) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint64_t gi = mul2(d[i], g[i]);
        H = add2(h[i], H);
        Q = fma2(h[i], h[i], Q);
        G = add2(gi, G);
        C = fma2(gi, h[i], C);
    }
}
__device__ __forceinline__ void add_centred(const Pack& h, const Pack& d, const Pack& g, uint64_t mean2, uint64_t& Q, uint64_t& C) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint64_t c = add2(h[i], mean2);
        Q = fma2(c, c, Q);
        C = fma2(mul2(d[i], g[i]), c, C);
    }
}
__device__ __forceinline__ void outputs(const Pack& h, const Pack& d, const Pack& g, const Pack& e, const RowCoefs& c, Pack& o,
                                        Pack& dg) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint64_t xh = mul2(add2(h[i], c.mean2), c.inv2);
        o[i] = fma2(fma2(d[i], g[i], c.a2), c.inv2, fma2(xh, c.b2, e[i]));
        dg[i] = fma2(d[i], xh, dg[i]);
    }
}

// dbeta's sums: in registers up to two packs a thread, above in the thread's own words
// of shared memory (with dgamma's they would not fit the 128 registers of 16 warps).
template <int PPT, bool ONE, int THREADS, int BLOCKS>
__global__ void __launch_bounds__(THREADS, BLOCKS) layernorm_backward_rows_kernel(const __grid_constant__ RowsParams p) {
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
    constexpr bool kRegs = PPT <= 2;
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
        uint64_t Q = 0ull, G = 0ull, C = 0ull, H = 0ull;
#pragma unroll
        for (int k = 0; k < PPT; ++k) {
            if (k < p.slices) {
                const int pk = t + k * p.nt;
                ring_wait(&g.full[s], ph, g, p);
                const uint8_t* at = g.stage + (size_t)s * p.stage_bytes + t * 16;
                if (pk < P) {
                    Pack h, gk;
                    Pack& d = dy[ONE ? 0 : k];
                    sum_ranks<ONE>(at, p.R, step, d);
                    if (ONE) dv[k] = *reinterpret_cast<const uint4*>(at);
                    hv[k] = *reinterpret_cast<const uint4*>(at + p.R * step);
                    if (p.has_res) ev[k] = *reinterpret_cast<const uint4*>(at + (p.R + 1) * step);
                    unpack8(hv[k], h);
                    load8(g.extra + pk * 8, gk);
                    add_terms(h, d, gk, Q, G, C, H);
                }
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(&g.empty[s]);
                if (++s == p.stages) { s = 0; ph ^= 1u; }
            }
        }
        float* red = g.red + buf * (6 * kWarps);  // [Q, G, C, H, and Q, C around the mean][warp]
        float v[4] = {both(Q), both(G), both(C), both(H)};
        const float part = Reduced<4>::run(v);
        if ((lane & 7) == 0) red[(lane >> 3) * kWarps + w] = part;
        consumer_bar(p.nt);
        const RowSums sums = block_sums(red, kWarps, nwarps);
        const float mean = sums.H * p.inv_n;
        float var = fmaf(sums.Q, p.inv_n, -mean * mean), products = fmaf(-mean, sums.G, sums.C);
        if (!(mean * mean <= kSpread * var)) {
            uint64_t cq = 0ull, cc = 0ull;
            const uint64_t mean2 = pair(-mean, -mean);
#pragma unroll
            for (int k = 0; k < PPT; ++k) {
                if (k < p.slices && t + k * p.nt < P) {
                    Pack h, gk;
                    unpack8(hv[k], h);
                    load8(g.extra + (t + k * p.nt) * 8, gk);
                    Pack& d = dy[ONE ? 0 : k];
                    if (ONE) unpack8(dv[k], d);
                    add_centred(h, d, gk, mean2, cq, cc);
                }
            }
            const float q = warp_sum(both(cq)), c = warp_sum(both(cc));
            if (lane == 0) {
                red[4 * kWarps + w] = q;
                red[5 * kWarps + w] = c;
            }
            consumer_bar(p.nt);
            var = red_total(red + 4 * kWarps, nwarps) * p.inv_n;
            products = red_total(red + 5 * kWarps, nwarps);
        }
        const RowCoefs coefs = row_coefs(mean, var, sums.G * p.inv_n, products, p);
#pragma unroll
        for (int k = 0; k < PPT; ++k) {
            if (k < p.slices) {
                const int pk = t + k * p.nt;
                if (pk < P) {
                    Pack gk, e = {}, o, h;
                    unpack8(hv[k], h);
                    load8(g.extra + pk * 8, gk);
                    if (p.has_res) unpack8(ev[k], e);
                    Pack& d = dy[ONE ? 0 : k];
                    if (ONE) unpack8(dv[k], d);
                    outputs(h, d, gk, e, coefs, o, dg[k]);
                    ptx::st_stream_v4(p.res_out + row * (int64_t)p.N + pk * 8, pack8(o));
                    if (kRegs) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) db[kRegs ? k : 0][i] = add2(db[kRegs ? k : 0][i], d[i]);
                    } else if (p.dbeta) {
                        Pack b;
                        load8(beta_sums + pk * 8, b);
#pragma unroll
                        for (int i = 0; i < 4; ++i) reinterpret_cast<uint64_t*>(beta_sums + pk * 8)[i] = add2(b[i], d[i]);
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

// Rows of up to 4096 columns: a block takes ROWS of them at a time, whose sums share one
// exchange and whose latencies run side by side (one row at a time, 16384 x 4096 took 138 us
// for a floor of 79: neither memory nor the issue slots were busy, but every row went through
// 25 shuffles, a barrier and the join one after the other).  It has no producer warp, which
// leaves 128 registers a thread: behind the barrier everyone has read the rows, so warp 0
// sends the ring's next copies from there.
constexpr int kSmallThreads = 512;  // threads an SM, at 128 registers

template <int PPT, int ROWS, bool ONE>
__global__ void __launch_bounds__(256, 2) layernorm_backward_small_kernel(const __grid_constant__ RowsParams p) {
    extern __shared__ __align__(128) uint8_t rows_smem[];
    Ring g;  // (for ring_wait)
    g.stage = rows_smem;
    g.extra = reinterpret_cast<float*>(rows_smem + (size_t)p.stages * p.stage_bytes);
    g.red = g.extra + p.extra_words;
    g.full = reinterpret_cast<uint64_t*>(g.red + p.red_words);
    g.abort = reinterpret_cast<volatile uint32_t*>(g.full + kMaxStages);
    const int t = threadIdx.x, lane = t & 31, w = t >> 5, nwarps = p.nt >> 5, P = p.N >> 3, S = p.stages;
    if (t == 0) {
        for (int s = 0; s < S; ++s) ptx::mbar_init(&g.full[s], 1);
        *g.abort = 0u;
        ptx::fence_mbar_init();
        ptx::fence_proxy_async_shared();
    }
    for (int i = t; i < p.red_words; i += p.nt) g.red[i] = 0.f;
    __syncthreads();
    ptx::grid_launch_dependents();
    ptx::grid_wait();

    // this block's k-th row (M and more: none)
    auto row_at = [&](int64_t k) { return (blockIdx.x + k / ROWS * gridDim.x) * ROWS + k % ROWS; };
    const uint32_t bytes = (uint32_t)p.N * 2u;
    const uint64_t pol = ptx::policy_evict_first();
    auto send = [&](int64_t k) {  // warp 0
        const int64_t row = row_at(k);
        if (row >= p.M) return;
        const int s = (int)(k % S);
        if (lane == 0) ptx::mbar_arrive_expect_tx(&g.full[s], bytes * (uint32_t)p.nsrc);
        __syncwarp();
        if (lane < p.nsrc)
            ptx::bulk_load_hint(g.stage + (size_t)s * p.stage_bytes + (size_t)lane * bytes, p.src[lane] + row * (int64_t)p.N, bytes,
                                &g.full[s], pol);
    };
    if (w == 0)
        for (int k = 0; k < S; ++k) send(k);

    // a thread reads only the gamma words that it writes here
#pragma unroll
    for (int k = 0; k < PPT; ++k) {
        const int pk = t + k * p.nt;
        if (pk < P) {
            reinterpret_cast<float4*>(g.extra)[pk * 2] = reinterpret_cast<const float4*>(p.gamma)[pk * 2];
            reinterpret_cast<float4*>(g.extra)[pk * 2 + 1] = reinterpret_cast<const float4*>(p.gamma)[pk * 2 + 1];
        }
    }
    Pack dg[PPT], db[PPT];
#pragma unroll
    for (int k = 0; k < PPT; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) dg[k][i] = db[k][i] = 0ull;
    int s = 0, buf = 0;
    uint32_t ph = 0;
    int64_t k0 = 0;
    for (int64_t row0 = (int64_t)blockIdx.x * ROWS; row0 < p.M; row0 += (int64_t)gridDim.x * ROWS, k0 += ROWS, buf ^= 1) {
        Pack dy[ONE ? 1 : ROWS][ONE ? 1 : PPT];
        uint4 dv[ONE ? ROWS : 1][ONE ? PPT : 1], hv[ROWS][PPT], ev[ROWS][PPT];
        float v[4 * ROWS];  // Q, G, C, H of each row
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            uint64_t Q = 0ull, G = 0ull, C = 0ull, H = 0ull;
            if (row0 + r < p.M) {
                ring_wait(&g.full[s], ph, g, p);
                const uint8_t* at = g.stage + (size_t)s * p.stage_bytes + t * 16;
#pragma unroll
                for (int k = 0; k < PPT; ++k, at += p.nt * 16) {
                    const int pk = t + k * p.nt;
                    if (pk < P) {
                        Pack h, gk, d1;
                        Pack& d = ONE ? d1 : dy[ONE ? 0 : r][ONE ? 0 : k];
                        if (ONE) dv[ONE ? r : 0][ONE ? k : 0] = *reinterpret_cast<const uint4*>(at);
                        hv[r][k] = *reinterpret_cast<const uint4*>(at + p.R * bytes);
                        if (p.has_res) ev[r][k] = *reinterpret_cast<const uint4*>(at + (p.R + 1) * bytes);
                        if (ONE) unpack8(dv[ONE ? r : 0][ONE ? k : 0], d);
                        else sum_ranks<false>(at, p.R, bytes, d);
                        unpack8(hv[r][k], h);
                        load8(g.extra + pk * 8, gk);
                        add_terms(h, d, gk, Q, G, C, H);
                    }
                }
            }
            v[r] = both(Q);
            v[ROWS + r] = both(G);
            v[2 * ROWS + r] = both(C);
            v[3 * ROWS + r] = both(H);
            if (++s == S) { s = 0; ph ^= 1u; }
        }
        const float part = Reduced<4 * ROWS>::run(v);  // lane l: value l / (8 / ROWS)
        float* red = g.red + buf * (ROWS * 6 * 8);  // [statistic][row][warp]
        constexpr int kPer = 8 / ROWS;
        if (lane % kPer == 0) red[(lane / kPer) * 8 + w] = part;
        __syncthreads();
        if (w == 0) {
#pragma unroll
            for (int r = 0; r < ROWS; ++r) send(k0 + S + r);
        }
        float mean[ROWS], var[ROWS], a[ROWS], products[ROWS];
        bool far = false;  // the same in every thread of the block
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            const RowSums sums = block_sums(red + r * 8, ROWS * 8, nwarps);
            mean[r] = sums.H * p.inv_n;
            var[r] = fmaf(sums.Q, p.inv_n, -mean[r] * mean[r]);
            a[r] = sums.G * p.inv_n;
            products[r] = fmaf(-mean[r], sums.G, sums.C);
            far |= !(mean[r] * mean[r] <= kSpread * var[r]);
        }
        if (far) {
            float* again = red + 4 * ROWS * 8;
#pragma unroll
            for (int r = 0; r < ROWS; ++r) {
                uint64_t cq = 0ull, cc = 0ull;
                const uint64_t mean2 = pair(-mean[r], -mean[r]);
#pragma unroll
                for (int k = 0; k < PPT; ++k) {
                    if (row0 + r < p.M && t + k * p.nt < P) {
                        Pack h, gk, d1;
                        unpack8(hv[r][k], h);
                        load8(g.extra + (t + k * p.nt) * 8, gk);
                        if (ONE) unpack8(dv[ONE ? r : 0][ONE ? k : 0], d1);
                        add_centred(h, ONE ? d1 : dy[ONE ? 0 : r][ONE ? 0 : k], gk, mean2, cq, cc);
                    }
                }
                const float q = warp_sum(both(cq)), c = warp_sum(both(cc));
                if (lane == 0) {
                    again[r * 8 + w] = q;
                    again[(ROWS + r) * 8 + w] = c;
                }
            }
            __syncthreads();
#pragma unroll
            for (int r = 0; r < ROWS; ++r) {
                if (!(mean[r] * mean[r] <= kSpread * var[r])) {
                    var[r] = red_total(again + r * 8, nwarps) * p.inv_n;
                    products[r] = red_total(again + (ROWS + r) * 8, nwarps);
                }
            }
        }
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            if (row0 + r >= p.M) continue;
            const RowCoefs coefs = row_coefs(mean[r], var[r], a[r], products[r], p);
#pragma unroll
            for (int k = 0; k < PPT; ++k) {
                const int pk = t + k * p.nt;
                if (pk < P) {
                    Pack h, gk, e = {}, o, d1;
                    unpack8(hv[r][k], h);
                    if (p.has_res) unpack8(ev[r][k], e);
                    load8(g.extra + pk * 8, gk);
                    if (ONE) unpack8(dv[ONE ? r : 0][ONE ? k : 0], d1);
                    const Pack& d = ONE ? d1 : dy[ONE ? 0 : r][ONE ? 0 : k];
                    outputs(h, d, gk, e, coefs, o, dg[k]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) db[k][i] = add2(db[k][i], d[i]);
                    ptx::st_stream_v4(p.res_out + (row0 + r) * (int64_t)p.N + pk * 8, pack8(o));
                }
            }
        }
    }
    if (w == 0 && *g.abort) {
        // the block must not end before its copies have landed (they have, unless a wait ran out)
        for (int64_t k = k0 > S ? k0 - S : 0; k < k0 + S; ++k) {
            if (row_at(k) >= p.M) break;
            const uint64_t t0 = ptx::globaltimer();
            while (!ptx::mbar_try_wait(&g.full[k % S], (uint32_t)(k / S) & 1u))
                if (ptx::globaltimer() - t0 > p.timeout_ns) break;
        }
    }
#pragma unroll
    for (int k = 0; k < PPT; ++k) {
        const int pk = t + k * p.nt;
        if (pk < P) {
            const size_t at = (size_t)blockIdx.x * p.N + pk * 8;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (p.dgamma) reinterpret_cast<uint64_t*>(p.dgamma + at)[i] = dg[k][i];
                if (p.dbeta) reinterpret_cast<uint64_t*>(p.dbeta + at)[i] = db[k][i];
            }
        }
    }
}

// The same rows by lanes, backward: a lane has the same columns in every row that it takes, and a block joins its lanes' and
// warps' sums in a fixed order at its end.
constexpr int kNarrowBackWarps = 4;

template <int PPT, bool ONE>
__global__ void __launch_bounds__(kNarrowBackWarps * 32, PPT == 1 ? 6 : 5)
    layernorm_backward_narrow_kernel(const __grid_constant__ RowsParams p) {
    __shared__ float sums[2][512];
    const int lane = threadIdx.x & 31, wb = threadIdx.x >> 5, G = p.lanes, l = lane & (G - 1), P = p.N >> 3, per_warp = 32 / G;
    ptx::grid_launch_dependents();
    ptx::grid_wait();
    Pack dg[PPT], db[PPT];
#pragma unroll
    for (int k = 0; k < PPT; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) dg[k][i] = db[k][i] = 0ull;
    const int64_t warps = (int64_t)gridDim.x * kNarrowBackWarps;
    for (int64_t w = (int64_t)blockIdx.x * kNarrowBackWarps + wb; w * per_warp < p.M; w += warps) {
        const int64_t row = w * per_warp + lane / G;
        const bool there = row < p.M;  // (all lanes stay for the exchanges; a row that is not there is zeros)
        const int64_t at = row * p.N + l * 8;
        auto load = [&](const uint16_t* from, int k) {
            return there && l + k * G < P ? ptx::ld_stream_v4(from + at + k * G * 8) : make_uint4(0u, 0u, 0u, 0u);
        };
        Pack dy[ONE ? 1 : PPT];
        uint4 dv[PPT], hv[PPT], ev[PPT];
#pragma unroll
        for (int k = 0; k < PPT; ++k) dv[k] = load(p.src[0], k);
#pragma unroll
        for (int k = 0; k < PPT; ++k) hv[k] = load(p.src[p.R], k);
        if (p.has_res) {
#pragma unroll
            for (int k = 0; k < PPT; ++k) ev[k] = load(p.src[p.R + 1], k);
        }
        if (!ONE) {
#pragma unroll
            for (int k = 0; k < PPT; ++k) unpack8(dv[k], dy[ONE ? 0 : k]);
            for (int r = 1; r < p.R; ++r) {
#pragma unroll
                for (int k = 0; k < PPT; ++k) dv[k] = load(p.src[r], k);
#pragma unroll
                for (int k = 0; k < PPT; ++k) {
                    Pack f;
                    unpack8(dv[k], f);
#pragma unroll
                    for (int i = 0; i < 4; ++i) dy[ONE ? 0 : k][i] = add2(dy[ONE ? 0 : k][i], f[i]);
                }
            }
        }
        uint64_t sum2 = 0ull;
#pragma unroll
        for (int k = 0; k < PPT; ++k) {
            Pack h;
            unpack8(hv[k], h);
#pragma unroll
            for (int i = 0; i < 4; ++i) sum2 = add2(h[i], sum2);
        }
        float H = both(sum2);
        for (int o = 1; o < G; o <<= 1) H += __shfl_xor_sync(0xFFFFFFFFu, H, o);
        const float mean = H * p.inv_n;
        const uint64_t mean2 = pair(-mean, -mean);
        uint64_t q2 = 0ull, g2 = 0ull, c2 = 0ull;
#pragma unroll
        for (int k = 0; k < PPT; ++k) {
            if (l + k * G < P) {
                Pack h, gk, d1;
                unpack8(hv[k], h);
                load8(p.gamma + (l + k * G) * 8, gk);
                if (ONE) unpack8(dv[k], d1);
                const Pack& d = ONE ? d1 : dy[ONE ? 0 : k];
                add_centred(h, d, gk, mean2, q2, c2);
#pragma unroll
                for (int i = 0; i < 4; ++i) g2 = fma2(d[i], gk[i], g2);
            }
        }
        float Q = both(q2), A = both(g2), C = both(c2);
        for (int o = 1; o < G; o <<= 1) {
            Q += __shfl_xor_sync(0xFFFFFFFFu, Q, o);
            A += __shfl_xor_sync(0xFFFFFFFFu, A, o);
            C += __shfl_xor_sync(0xFFFFFFFFu, C, o);
        }
        const RowCoefs coefs = row_coefs(mean, Q * p.inv_n, A * p.inv_n, C, p);
        if (there) {
#pragma unroll
            for (int k = 0; k < PPT; ++k) {
                if (l + k * G < P) {
                    Pack h, gk, e = {}, o, d1;
                    unpack8(hv[k], h);
                    if (p.has_res) unpack8(ev[k], e);
                    load8(p.gamma + (l + k * G) * 8, gk);
                    if (ONE) unpack8(dv[k], d1);
                    const Pack& d = ONE ? d1 : dy[ONE ? 0 : k];
                    outputs(h, d, gk, e, coefs, o, dg[k]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) db[k][i] = add2(db[k][i], d[i]);
                    ptx::st_stream_v4(p.res_out + at + k * G * 8, pack8(o));
                }
            }
        }
    }
    // the lanes of a warp that have the same columns, then the warps in turn
    for (int w = 0; w < kNarrowBackWarps; ++w) {
        if (wb == w) {
#pragma unroll
            for (int k = 0; k < PPT; ++k) {
                const int pk = l + k * G;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float2 a = unpair(dg[k][i]), b = unpair(db[k][i]);
                    for (int o = G; o < 32; o <<= 1) {
                        a.x += __shfl_xor_sync(0xFFFFFFFFu, a.x, o);
                        a.y += __shfl_xor_sync(0xFFFFFFFFu, a.y, o);
                        b.x += __shfl_xor_sync(0xFFFFFFFFu, b.x, o);
                        b.y += __shfl_xor_sync(0xFFFFFFFFu, b.y, o);
                    }
                    if (lane < G && pk < P) {
                        float2* const g = reinterpret_cast<float2*>(sums[0] + pk * 8) + i;
                        float2* const t = reinterpret_cast<float2*>(sums[1] + pk * 8) + i;
                        const float2 x = w ? *g : make_float2(0.f, 0.f), y = w ? *t : make_float2(0.f, 0.f);
                        *g = make_float2(x.x + a.x, x.y + a.y);
                        *t = make_float2(y.x + b.x, y.y + b.y);
                    }
                }
            }
        }
        __syncthreads();
    }
    for (int j = threadIdx.x; j < p.N; j += kNarrowBackWarps * 32) {
        if (p.dgamma) p.dgamma[(size_t)blockIdx.x * p.N + j] = sums[0][j];
        if (p.dbeta) p.dbeta[(size_t)blockIdx.x * p.N + j] = sums[1][j];
    }
}

// Lanes a row rather than a block: where a row is hardly more than its exchange (R = 8, 16384 x 64: 4.0 us, a block 15.5), and
// with few sources where there are many rows (R = 1, 16384 x 264: 10.7 us for 16.7, x 1024 26.5 for 29.5; 4000 x 1024 8.9 for
// 8.0; with eight, whose loads the ring keeps further ahead, 16384 x 264 26.9 for 22.1).
bool narrow(int P, int sources, int64_t M, int num_sms) {
    return P <= 16 ? M > 4 * (int64_t)num_sms : P <= 128 && sources <= 3 && M > 32 * (int64_t)num_sms;
}

// Backward, where a block already takes four such rows at a time: R = 1, 16384 x 64: 9.4 us for 17.2, x 264 17.9 for 25.9, 4000
// x 264 10.0 for 12.0, 1500 x 64 5.9 for 7.2; R = 4, 16384 x 64 10.3 for 20.2, but 4000 x 264 12.4 for 10.5.
bool narrow_backward(int P, int sources, int64_t M, int num_sms) {
    return (P <= 16 || (P <= 64 && sources <= 3)) && M > 8 * (int64_t)num_sms;
}

// Packs a thread holds, of a row of P.  A row alone takes as many warps as it fills.  Up to 512 packs several blocks of an SM
// hide one another's latencies (R = 1, 16384 x 2048, in us: one pack a thread and two blocks 55, two packs and four 51; 4096 x
// 1536 15.0 and 10.6), above one block of up to 16 warps has the shortest row (R = 1, 16384 x 10000: four packs 289, three 225;
// R = 8, 1001 x 7168: 28.1, two 24.6, though 16384 rows of it take 387 for 382).  Up to 640 four packs leave room for three
// blocks, which many rows use (R = 1, 16384 x 5120: two packs 150, four 117; R = 8, 1001 rows: 19.6 and 22.6).
int packs_per_thread(int P, int64_t M, int num_sms) {
    if (M <= num_sms && P <= 1024) return P <= 512 ? 1 : 2;
    if (P > 512 && P <= 640 && M > 16 * (int64_t)num_sms) return 4;
    return P <= 128 ? 1 : P <= 1024 ? 2 : P <= 1536 ? 3 : P <= 2048 ? 4 : 8;
}
// Backward, three packs for a little more than two blocks of two hold: two blocks an SM have two rows' latencies side by side,
// but need more rows to pay for their partial sums (R = 3: 16384 x 4104 119 us for 150 with one block, 4096 x 5120 41 for 46,
// 1001 x 5120 17.3 for 16.7; R = 1: 16384 x 4104 113 for 121, 4096 x 5120 41 for 40).  Two packs with 16 warps and a
// producer leave 96 registers a thread, enough for one rank's dy, which stays packed (R = 1: 16384 x 8192 182 us for 219 with
// three packs; R = 3: 241 for 219).
int backward_packs_per_thread(int P, int R, int sources, int64_t M, int num_sms) {
    if (P > 512 && P <= 672 && M * sources > 100 * (int64_t)num_sms) return 3;
    return P <= 256 ? 1 : P <= (R == 1 ? 1024 : 960) ? 2 : P <= 1440 ? 3 : P <= 1920 ? 4 : 5;
}

// The kernel of a plan: blocks of up to 288 threads leave room for two on an SM.
void (*forward_kernel(int ppt, int threads))(RowsParams) {
    switch (ppt) {
        case 1: return threads <= 288 ? layernorm_rows_kernel<1, 288, 2> : layernorm_rows_kernel<1, 544, 1>;
        case 2: return threads <= 288 ? layernorm_rows_kernel<2, 288, 2> : layernorm_rows_kernel<2, 544, 1>;
        case 3: return layernorm_rows_kernel<3, 544, 1>;
        case 4: return threads <= 288 ? layernorm_rows_kernel<4, 288, 2> : layernorm_rows_kernel<4, 544, 1>;
        default: return layernorm_rows_kernel<8, 544, 1>;
    }
}

template <bool ONE>
void (*backward_kernel(int ppt, int threads, int rows, int lanes))(RowsParams) {
    if (lanes) return ppt == 1 ? layernorm_backward_narrow_kernel<1, ONE> : layernorm_backward_narrow_kernel<2, ONE>;
    if (rows == 4) return layernorm_backward_small_kernel<1, 4, ONE>;
    if (rows == 2) return layernorm_backward_small_kernel<2, 2, ONE>;
    switch (ppt) {
        case 1: return layernorm_backward_rows_kernel<1, ONE, 288, 2>;
        case 2:
            if (ONE && threads > 512) return layernorm_backward_rows_kernel<2, true, 544, 1>;
            return threads <= 288 ? layernorm_backward_rows_kernel<2, ONE, 288, 2> : layernorm_backward_rows_kernel<2, ONE, 512, 1>;
        case 3: return layernorm_backward_rows_kernel<3, ONE, 512, 1>;
        case 4: return layernorm_backward_rows_kernel<4, ONE, 512, 1>;
        default: return layernorm_backward_rows_kernel<5, ONE, 512, 1>;
    }
}

}  // namespace

RowsPlan layernorm_plan(RowsParams& p, int num_sms) {
    const int P = p.N / 8;
    p.lanes = 0;
    p.rows = 1;
    if (p.backward ? narrow_backward(P, p.nsrc, p.M, num_sms) : narrow(P, p.nsrc, p.M, num_sms)) {
        RowsPlan plan;
        p.lanes = P <= 8 ? 8 : P <= 16 ? 16 : 32;
        plan.ppt = (P + p.lanes - 1) / p.lanes;
        const int warps = p.backward ? kNarrowBackWarps : kNarrowWarps;
        const int resident = p.backward ? (plan.ppt == 1 ? 6 : 5) : plan.ppt <= 2 ? 4 : 3;
        plan.threads = warps * 32;
        plan.smem = 0;
        const int64_t rows = warps * (32 / p.lanes), blocks = (p.M + rows - 1) / rows;
        plan.grid = (int)std::min<int64_t>(blocks, (int64_t)num_sms * resident);
        return plan;
    }
    const int ppt = p.backward ? backward_packs_per_thread(P, p.R, p.nsrc, p.M, num_sms) : packs_per_thread(P, p.M, num_sms);
    const int one_nt = ((P + ppt - 1) / ppt + 31) / 32 * 32;
    if (p.backward && ppt <= 2 && P <= 512 && p.M > (int64_t)num_sms * (kRowsThreads / (one_nt + 32))) {
        // several rows at a time, where there is more than a round of single ones and the ring holds that many for every
        // block that an SM's registers hold
        RowsPlan plan;
        plan.ppt = ppt;
        p.rows = ppt == 1 ? 4 : 2;
        p.nt = one_nt;
        p.slices = ppt;
        p.extra_words = p.N;
        p.red_words = 2 * p.rows * 6 * 8;
        p.stage_bytes = p.nsrc * p.N * 2;
        const int64_t items = (p.M + p.rows - 1) / p.rows, rounds = (items + num_sms - 1) / num_sms;
        const int blocks = (int)std::min<int64_t>(rounds, std::min(kSmallThreads / p.nt, 10));
        const size_t fixed = (size_t)(p.extra_words + p.red_words) * 4 + kMaxStages * 8 + 16;
        const size_t room = (blocks == 1 ? kRowsSmemLimit : kRowsSmemSm / blocks - 1024) - fixed;
        p.stages = (int)std::min<size_t>(room / p.stage_bytes, kMaxStages);
        plan.smem = fixed + (size_t)p.stages * p.stage_bytes;
        plan.threads = p.nt;
        plan.grid = (int)std::min<int64_t>(items, (int64_t)blocks * num_sms);
        if (p.stages >= p.rows) return plan;
        p.rows = 1;
    }
    p.extra_words = p.backward ? (ppt <= 2 ? p.N : 2 * p.N) : ppt == 3 || ppt == 4 ? p.N : 0;
    p.red_words = kRedAll;
    return rows_shape(p, ppt, num_sms);
}

cudaError_t layernorm_prepare() {
    cudaError_t e = cudaSuccess;
    for (int ppt : {1, 2, 3, 4, 8})
        for (int threads : {288, 544})
            if (e == cudaSuccess) e = opt_in(forward_kernel(ppt, threads));
    for (int ppt : {1, 2, 3, 4, 5})
        for (int threads : {288, 512, 544})
            for (bool one : {false, true})
                if (e == cudaSuccess)
                    e = opt_in(one ? backward_kernel<true>(ppt, threads, 1, 0) : backward_kernel<false>(ppt, threads, 1, 0));
    for (int rows : {2, 4})
        for (bool one : {false, true})
            if (e == cudaSuccess) e = opt_in(one ? backward_kernel<true>(0, 0, rows, 0) : backward_kernel<false>(0, 0, rows, 0));
    return e;
}

cudaError_t launch_layernorm_rows(const RowsParams& p, const RowsPlan& plan, cudaStream_t s) {
    auto* kernel = p.lanes == 0   ? forward_kernel(plan.ppt, plan.threads)
                   : plan.ppt == 1 ? layernorm_narrow_kernel<1>
                   : plan.ppt == 2 ? layernorm_narrow_kernel<2>
                   : plan.ppt == 3 ? layernorm_narrow_kernel<3>
                                   : layernorm_narrow_kernel<4>;
    return launch_dependent(kernel, plan.grid, plan.threads, plan.smem, s, p);
}

cudaError_t launch_layernorm_backward_rows(RowsParams& p, const RowsPlan& plan, float* scratch, float* dgamma, float* dbeta,
                                           cudaStream_t s) {
    // a single block's sums are the results; otherwise dbeta's partial rows lie right behind dgamma's
    const bool one = plan.grid == 1;
    float* const second = scratch + (dgamma ? (size_t)plan.grid * p.N : 0);
    p.dgamma = dgamma == nullptr ? nullptr : one ? dgamma : scratch;
    p.dbeta = dbeta == nullptr ? nullptr : one ? dbeta : second;
    auto* kernel = p.R == 1 ? backward_kernel<true>(plan.ppt, plan.threads, p.rows, p.lanes)
                            : backward_kernel<false>(plan.ppt, plan.threads, p.rows, p.lanes);
    cudaError_t e = launch_dependent(kernel, plan.grid, plan.threads, plan.smem, s, p);
    if (e == cudaSuccess && !one && (dgamma || dbeta))
        e = launch_row_sums(scratch, dgamma ? dgamma : dbeta, dgamma ? dbeta : nullptr, plan.grid, p.N, s);
    return e;
}

}  // namespace are
