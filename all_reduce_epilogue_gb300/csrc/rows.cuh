// What the row-streaming kernels share: the ring of stages that a producer warp fills
// with slices of a row's sources, fp32 arithmetic in pairs of columns, sums over a
// block's warps, and their launch.
#pragma once
#include <cuda_bf16.h>

#include "are_internal.h"
#include "ptx.cuh"

namespace are {
namespace {

constexpr int kMaxStages = 16;
constexpr size_t kRowsSmemLimit = 227 * 1024;   // a block
constexpr size_t kRowsSmemSm = 228 * 1024;      // an SM, 1 KB of it for each block
constexpr int kRowsThreads = 640;               // threads an SM at the 96 registers of blocks up to 288

using ptx::add2;
using ptx::fma2;
using ptx::mul2;
using ptx::pair;
using ptx::unpair;

// A pack of 8 columns in fp32 is four pairs: their arithmetic is two columns an instruction.
typedef uint64_t Pack[4];

__device__ __forceinline__ void unpack8(const uint4& v, Pack& f) {
    f[0] = pair(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xFFFF0000u));
    f[1] = pair(__uint_as_float(v.y << 16), __uint_as_float(v.y & 0xFFFF0000u));
    f[2] = pair(__uint_as_float(v.z << 16), __uint_as_float(v.z & 0xFFFF0000u));
    f[3] = pair(__uint_as_float(v.w << 16), __uint_as_float(v.w & 0xFFFF0000u));
}

__device__ __forceinline__ uint32_t pack2(uint64_t v) {
    const float2 f = unpair(v);
    __nv_bfloat162 b = __floats2bfloat162_rn(f.x, f.y);
    return *reinterpret_cast<uint32_t*>(&b);
}

__device__ __forceinline__ uint4 pack8(const Pack& f) {
    return make_uint4(pack2(f[0]), pack2(f[1]), pack2(f[2]), pack2(f[3]));
}

// 8 fp32 words, 16-byte aligned (shared or global memory).
__device__ __forceinline__ void load8(const float* at, Pack& f) {
    const float4 a = reinterpret_cast<const float4*>(at)[0], b = reinterpret_cast<const float4*>(at)[1];
    f[0] = pair(a.x, a.y);
    f[1] = pair(a.z, a.w);
    f[2] = pair(b.x, b.y);
    f[3] = pair(b.z, b.w);
}

__device__ __forceinline__ float both(uint64_t v) {
    const float2 f = unpair(v);
    return f.x + f.y;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

struct Ring {
    uint8_t* stage;
    uint64_t* full;
    uint64_t* empty;
    float* red;
    float* extra;               // p.extra_words fp32 of the kernel's own (backward: gamma)
    volatile uint32_t* abort;
};

__device__ __forceinline__ Ring carve(uint8_t* base, const RowsParams& p) {
    Ring g;
    g.stage = base;
    g.extra = reinterpret_cast<float*>(base + (size_t)p.stages * p.stage_bytes);
    g.red = g.extra + p.extra_words;
    g.full = reinterpret_cast<uint64_t*>(g.red + p.red_words);
    g.empty = g.full + kMaxStages;
    g.abort = reinterpret_cast<volatile uint32_t*>(g.empty + kMaxStages);
    return g;
}

// Bounded wait on a barrier phase; after a timeout every wait of the block
// returns at once, and the block runs to its end without waiting.
__device__ __forceinline__ bool ring_wait(uint64_t* bar, uint32_t parity, const Ring& g, const RowsParams& p) {
    if (ptx::mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = ptx::globaltimer();
    while (!ptx::mbar_try_wait(bar, parity)) {
        if (*g.abort) return false;
        if (ptx::globaltimer() - t0 > p.timeout_ns) {
            record_error(p.status, ARE_DEV_PIPE_TIMEOUT, blockIdx.x, -5, -1);
            *g.abort = 1u;
            return false;
        }
    }
    return true;
}

__device__ __forceinline__ void consumer_bar(int nt) {
    __syncwarp();
    asm volatile("bar.sync 1, %0;" ::"r"(nt) : "memory");
}

__device__ __forceinline__ void ring_init(const Ring& g, const RowsParams& p) {
    if (threadIdx.x == 0) {
        for (int s = 0; s < p.stages; ++s) {
            ptx::mbar_init(&g.full[s], 1);
            ptx::mbar_init(&g.empty[s], p.nt / 32);
        }
        *g.abort = 0u;
        ptx::fence_mbar_init();
        ptx::fence_proxy_async_shared();
    }
    for (int i = threadIdx.x; i < p.red_words; i += blockDim.x) g.red[i] = 0.f;
    __syncthreads();
}

// The producer warp: lane i copies source i's slice.
__device__ __forceinline__ void produce(const Ring& g, const RowsParams& p) {
    const int lane = threadIdx.x & 31;
    const uint64_t pol = ptx::policy_evict_first();
    const uint16_t* src = lane < p.nsrc ? p.src[lane] : nullptr;
    int s = 0;
    uint32_t ph = 0;
    int64_t issued = 0;
    bool ok = true;
    for (int64_t row = blockIdx.x; row < p.M && ok; row += gridDim.x) {
        for (int k = 0; k < p.slices; ++k) {
            ok = ring_wait(&g.empty[s], ph ^ 1u, g, p);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok) break;
            const int c0 = k * p.nt * 8;
            const uint32_t bytes = (uint32_t)min(p.nt * 8, p.N - c0) * 2u;
            if (lane == 0) ptx::mbar_arrive_expect_tx(&g.full[s], bytes * (uint32_t)p.nsrc);
            __syncwarp();
            if (src)
                ptx::bulk_load_hint(g.stage + (size_t)s * p.stage_bytes + (size_t)lane * p.nt * 16,
                                    src + row * (int64_t)p.N + c0, bytes, &g.full[s], pol);
            ++issued;
            if (++s == p.stages) { s = 0; ph ^= 1u; }
        }
    }
    // the block must not end before its copies have landed (they have, unless a wait ran out)
    if (lane == 0 && !ok) {
        const int n = issued < p.stages ? (int)issued : p.stages;
        for (int i = 1; i <= n; ++i) {
            const int64_t j = issued - i;
            const uint64_t t0 = ptx::globaltimer();
            while (!ptx::mbar_try_wait(&g.full[j % p.stages], (uint32_t)(j / p.stages) & 1u))
                if (ptx::globaltimer() - t0 > p.timeout_ns) break;
        }
    }
}

template <int R>
__device__ __forceinline__ void sum_more(const uint8_t* at, size_t step, Pack& f) {
#pragma unroll
    for (int r = 1; r < R; ++r) {
        Pack v;
        unpack8(*reinterpret_cast<const uint4*>(at + r * step), v);
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = add2(f[i], v[i]);
    }
}

// Sum of the R partials of this thread's pack, r ascending from +0.0.  ONE: R is
// 1, the common case of the backward pass, without the code of the other ranks.
// The usual numbers of ranks have code of their own: with a branch a rank, each
// load waits for the one before (one row of 7168, R = 8: 5.7 us, without 5.4;
// R = 8, 8192 x 512: 15.2 and 14.0; backward R = 4, 2000 x 2048: 14.1 and 12.5.
// A case for every number makes the code too long: one row 6.1 us).
template <bool ONE>
__device__ __forceinline__ void sum_ranks(const uint8_t* at, int R, size_t step, Pack& f) {
    unpack8(*reinterpret_cast<const uint4*>(at), f);
    if constexpr (!ONE) {
        if (R == 8) {
            sum_more<8>(at, step, f);
        } else if (R == 4) {
            sum_more<4>(at, step, f);
        } else if (R == 2) {
            sum_more<2>(at, step, f);
        } else if (R > 1) {
            sum_more<3>(at, step, f);
#pragma unroll
            for (int r = 3; r < kMaxRanks - 1; ++r) {
                if (r < R) {
                    Pack v;
                    unpack8(*reinterpret_cast<const uint4*>(at + r * step), v);
#pragma unroll
                    for (int i = 0; i < 4; ++i) f[i] = add2(f[i], v[i]);
                }
            }
        }
    }
}

// Sum over the consumer threads of one statistic, the same bits in every
// thread.  `red` holds one word per warp, zero behind the last one.
__device__ __forceinline__ float red_total(const float* red, int nwarps) {
    float t = 0.f;
    for (int w = 0; w < nwarps; w += 4) {
        const float4 v = *reinterpret_cast<const float4*>(red + w);
        t += (v.x + v.y) + (v.z + v.w);
    }
    return t;
}

// Launches on the programmatic dependency: the kernel comes up while the one
// before it in the stream runs out, and waits for its end before it touches
// global memory (grid_wait).  That hides the launch and the prologue.
template <typename... P, typename... A>
cudaError_t launch_dependent(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t s, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr = dependent_launch();
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

template <typename F>
cudaError_t opt_in(F f) {
    return cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kRowsSmemLimit);
}

// The launch shape of rows whose threads own `ppt` packs each; p.extra_words and p.red_words are set.
inline RowsPlan rows_shape(RowsParams& p, int ppt, int num_sms) {
    RowsPlan plan;
    const int P = p.N / 8;
    plan.ppt = ppt;
    p.nt = ((P + plan.ppt - 1) / plan.ppt + 31) / 32 * 32;
    p.slices = (P + p.nt - 1) / p.nt;
    p.stage_bytes = p.nsrc * p.nt * 16;
    const int fit = p.nt > 256 ? 1 : kRowsThreads / (p.nt + 32);  // blocks of an SM
    const int64_t rounds = (p.M + num_sms - 1) / num_sms;
    const int blocks = (int)(rounds < fit ? rounds : fit);
    const size_t fixed = (size_t)(p.extra_words + p.red_words) * 4 + 2 * kMaxStages * 8 + 16;
    const size_t room = (blocks == 1 ? kRowsSmemLimit : kRowsSmemSm / blocks - 1024) - fixed;
    p.stages = (int)(room / p.stage_bytes);
    if (p.stages > kMaxStages) p.stages = kMaxStages;
    plan.smem = fixed + (size_t)p.stages * p.stage_bytes;
    plan.threads = p.nt + 32;
    plan.grid = (int)(p.M < (int64_t)blocks * num_sms ? p.M : (int64_t)blocks * num_sms);
    return plan;
}

}  // namespace
}  // namespace are
