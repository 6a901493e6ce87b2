// Lookup in an embedding table whose vocabulary is split over R ranks, and its gradient.
//
//   out_i    = scale * table[id_i]                      (0 where id_i is outside the vocabulary)
//   dtable_v = scale * sum_{i : id_i = v} dy_i          (every row of every rank is written)
//
// In a tensor-parallel model each rank looks up the tokens of its own rows, has zeros for the
// others, and the all-reduce adds R partials of which one is not zero: on one GPU that sum is
// the row itself, read from the rank that has it.
//
// Both are bound by memory: forward 4 bytes an output element, backward 2 for dy and 2 for
// each element of the tables, most of which are zeros.  The gradient's sums go by the tokens
// sorted by (id, position): a token's rows meet in fp32 in the order of their positions, whatever
// the hardware's order is.
//   1. A cluster of eight CTAs sorts the ids, stable, up to 10 bits a pass (a warp ranks its own run of
//      tokens by matching digits, counters per warp and digit keep the order), in shared memory for up to
//      131072 tokens, in runs of that for more; up to 2048 tokens one CTA does.  Beside it, on the other
//      SMs, a second kernel writes the tables' zeros, which mostly takes longer.
//   2. The sorted tokens are cut into chunks of equal length, whatever the ids: a token that makes
//      up a tenth of a batch is then work for a tenth of the chunks.  A chunk's sums that do not
//      reach its ends are results; the others are partial rows.
//   3. The partial rows of an id are added in order.
// Rows that tokens touch are written twice, first with zeros: knowing them in step 1 would mean
// that the zeros wait for the sort (with the rest of the zeros in step 3 the three took 159 us).
// Up to 512 tokens a kernel of its own does all of it.
//
// Measured, 16384 x 4096, vocabulary 65536 over 8 ranks, 6000 of them in the text: lookup 31.5 us, 5.8 TB/s of
// the bytes it cannot do without (8.6 with the rows that come again, which are in L2); gradient 124 us,
// 5.3 TB/s: zeros 82 us, the sort below them, sums 33, join 8; added to tables that are there 76 us for
// 33: sort 16, sums 52 (a row of the table is loaded where its sum ends, and nothing runs under that), join 8.
// 300 x 1032, vocabulary 11001: 8.7 us; 16384 x 1032: 34 (one CTA's sort 63).
#include <algorithm>

#include "rows.cuh"

namespace are {
namespace {

constexpr int kSortThreads = 1024, kSortWarps = 32;
constexpr int kSortCluster = 8;       // CTAs
constexpr int kSortOne = 2048;        // tokens that one CTA sorts: 16.2 us with sums and join at 1024 x 1032, a cluster 17.5; at 4096 24.0 and 20.7
constexpr int kMaxBins = 1024;
template <int ITEMS>  // of a thread
constexpr size_t kSortSmem = (size_t)ITEMS * kSortThreads * 8 + (size_t)kSortWarps * kMaxBins * 2 + 4 * kMaxBins * 4 + 64 * 4;
static_assert(kSortSmem<16> <= kRowsSmemLimit, "shared memory budget");
constexpr int kZeroThreads = 512, kZeroBlocks = 2;  // of an SM
constexpr int kThreads = 128;
constexpr int kShort = 16;            // chunks behind its first one through which one warp adds up an id's sum
constexpr int kSumBlocks = 6;         // blocks of the sums on an SM

template <typename T>
__device__ __forceinline__ uint32_t id_as(const EmbedParams& p, int64_t i) {
    const int64_t v = static_cast<const T*>(p.ids)[i];
    return v >= 0 && v < p.V ? (uint32_t)v : p.V;  // V: none
}
__device__ __forceinline__ uint32_t id_of(const EmbedParams& p, int64_t i) {
    return p.wide ? id_as<int64_t>(p, i) : id_as<int32_t>(p, i);
}

__device__ __forceinline__ uint16_t* row_of(uint16_t* const* tables, uint32_t id, const EmbedParams& p) {
    const uint32_t r = id / p.Vs;
    return tables[r] + (size_t)(id - r * p.Vs) * p.N;
}

// ---------------------------------------------------------------------- forward
// A thread takes up to four packs of 8 columns, a block's threads consecutive ones of one or more rows.
__global__ void __launch_bounds__(kThreads) embed_kernel(const __grid_constant__ EmbedParams p) {
    const int P = p.N >> 3;
    const int64_t at = (int64_t)blockIdx.x * (kThreads * 4), row0 = at / P;
    const int in0 = (int)(at - row0 * P);
    ptx::grid_launch_dependents();
    ptx::grid_wait();
    uint4 v[4];
    int64_t row[4];
    int col[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t i = (uint32_t)in0 + j * kThreads + threadIdx.x, r = i / (uint32_t)P;
        row[j] = row0 + r;
        col[j] = (int)(i - r * P) * 8;
        v[j] = make_uint4(0u, 0u, 0u, 0u);
        if (row[j] < p.M) {
            const uint32_t id = id_of(p, row[j]);
            if (id < p.V) v[j] = *reinterpret_cast<const uint4*>(row_of(p.tables, id, p) + col[j]);
        }
    }
    const uint64_t scale = pair(p.scale, p.scale);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (row[j] < p.M) {
            if (p.scale != 1.f) {
                Pack f;
                unpack8(v[j], f);
#pragma unroll
                for (int i = 0; i < 4; ++i) f[i] = mul2(f[i], scale);
                v[j] = pack8(f);
            }
            *reinterpret_cast<uint4*>(p.out + row[j] * p.N + col[j]) = v[j];
        }
    }
}

// ------------------------------------------------------------------------- sort
// Exclusive sum over the block's threads; `warps` holds 32 words.
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t* warps) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    uint32_t x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();  // (the words' last readers are done)
    if (lane == 31) warps[w] = x;
    __syncthreads();
    if (w == 0) {
        uint32_t s = warps[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, s, o);
            if (lane >= o) s += y;
        }
        warps[lane] = s;
    }
    __syncthreads();
    return x - v + (w ? warps[w - 1] : 0u);
}

// The CTAs of a cluster sort as one: each ranks a part of the tokens, in their order, and writes its items to the places that
// all parts' counts give them, in whichever CTA's shared memory that is.
template <bool CLUSTER, int ITEMS>
__global__ void __launch_bounds__(kSortThreads, 1) embed_sort_kernel(const __grid_constant__ EmbedParams p) {
    extern __shared__ __align__(128) uint8_t smem[];
    uint32_t* skey = reinterpret_cast<uint32_t*>(smem);
    uint32_t* sidx = skey + ITEMS * kSortThreads;
    uint16_t* count = reinterpret_cast<uint16_t*>(sidx + ITEMS * kSortThreads);   // [warp][bin]
    uint32_t* local = reinterpret_cast<uint32_t*>(count + kSortWarps * kMaxBins);  // where this CTA's items of a bin begin in the run
    uint32_t* first = local + kMaxBins;                                            // where the bin does
    uint32_t* global = first + kMaxBins;                                           // and where its next items go in the whole order
    uint32_t* totals = global + kMaxBins;                                          // this CTA's items of a bin
    uint32_t* scan = totals + kMaxBins;
    const int t = threadIdx.x, lane = t & 31, w = t >> 5;
    constexpr int C = CLUSTER ? kSortCluster : 1;
    const int q = CLUSTER ? (int)ptx::cluster_ctarank() : 0;
    const int M = (int)p.M, bins = 1 << p.digit_bits, run = C * ITEMS * kSortThreads;
    const bool one = M <= run;
    const uint32_t mask = bins - 1;
    uint16_t* mine = count + w * bins;
    auto sync = [] {
        __syncwarp();
        if (CLUSTER) ptx::cluster_sync();
        else __syncthreads();
    };
    // the sum over the CTAs of a bin's total, and over those before this one
    auto joined = [&](int bin, uint32_t& before) {
        uint32_t all = 0;
        before = 0;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const uint32_t x = CLUSTER ? ptx::ld_cluster_u32(ptx::mapa_shared(ptx::smem_u32(totals + bin), c)) : totals[bin];
            before += c < q ? x : 0u;
            all += x;
        }
        return all;
    };
    if (p.accumulate) ptx::grid_launch_dependents();
    ptx::grid_wait();
    if (q == 0 && t < 2) p.crossing[t] = 0;
    for (int pass = 0; pass < p.passes; ++pass) {
        const int shift = pass * p.digit_bits;
        const uint32_t *from_key = p.keys[(pass & 1) ^ 1], *from_idx = p.idx[(pass & 1) ^ 1];
        uint32_t *to_key = p.keys[pass & 1], *to_idx = p.idx[pass & 1];
        if (!one) {
            for (int b = t; b < bins; b += kSortThreads) totals[b] = 0;
            __syncthreads();
            for (int i = q * kSortThreads + t; i < M; i += C * kSortThreads)
                atomicAdd(&totals[((pass == 0 ? id_of(p, i) : from_key[i]) >> shift) & mask], 1u);
            sync();
            uint32_t before, n = t < bins ? joined(t, before) : 0u;
            const uint32_t at = block_scan(n, scan);
            if (t < bins) global[t] = at;
            sync();  // the totals have been read
        }
        for (int c0 = 0; c0 < M; c0 += run) {
            const int n = min(run, M - c0), per = (n + C * kSortThreads - 1) / (C * kSortThreads);  // items of a thread
            const int part = per * kSortThreads;                                                    // of a CTA
            for (int i = t; i < kSortWarps * bins / 2; i += kSortThreads) reinterpret_cast<uint32_t*>(count)[i] = 0;
            __syncthreads();
            // a warp has a run of per * 32 items, in their order; an item's place among the warp's of its digit
            uint32_t key[ITEMS], idx[ITEMS], place[ITEMS / 2];
            const int s0 = w * per * 32 + lane, i0 = q * part + s0;  // its first item in the CTA's part, in the run
            // one kind of source a loop, so that its loads run side by side
            auto items = [&](auto load) {
#pragma unroll
                for (int j = 0; j < ITEMS; ++j)
                    if (j < per && i0 + j * 32 < n) load(j, j * 32);
            };
            if (pass > 0 && one) items([&](int j, int k) { key[j] = skey[s0 + k]; idx[j] = sidx[s0 + k]; });
            else if (pass > 0) items([&](int j, int k) { key[j] = from_key[c0 + i0 + k]; idx[j] = from_idx[c0 + i0 + k]; });
            else if (p.wide) items([&](int j, int k) { key[j] = id_as<int64_t>(p, c0 + i0 + k); idx[j] = c0 + i0 + k; });
            else items([&](int j, int k) { key[j] = id_as<int32_t>(p, c0 + i0 + k); idx[j] = c0 + i0 + k; });
            // the zeros' kernel may begin: the loads of the ids, which would wait behind its stores, are on their way
            if (pass == 0 && c0 == 0) ptx::grid_launch_dependents();
#pragma unroll
            for (int j = 0; j < ITEMS; ++j) {
                if (j < per) {
                    const bool in = i0 + j * 32 < n;
                    const uint32_t d = in ? (key[j] >> shift) & mask : 0xFFFFFFFFu;
                    const uint32_t same = __match_any_sync(0xFFFFFFFFu, d);
                    const int leader = __ffs(same) - 1;
                    uint32_t before = 0;
                    if (lane == leader && in) {
                        before = mine[d];
                        mine[d] = (uint16_t)(before + __popc(same));
                    }
                    before = __shfl_sync(0xFFFFFFFFu, before, leader) + __popc(same & ((1u << lane) - 1u));
                    if (j & 1) place[j / 2] |= before << 16;
                    else place[j / 2] = before;
                    __syncwarp();
                }
            }
            __syncthreads();
            if (t < bins) {
                uint32_t total = 0;
#pragma unroll 8
                for (int v = 0; v < kSortWarps; ++v) {
                    const uint32_t x = count[v * bins + t];
                    count[v * bins + t] = (uint16_t)total;
                    total += x;
                }
                totals[t] = total;
            }
            sync();  // the CTAs' totals are there, and their items in registers
            uint32_t before = 0;
            const uint32_t all = t < bins ? joined(t, before) : 0u, at = block_scan(all, scan);
            if (t < bins) {
                first[t] = at;
                local[t] = at + before;
            }
            __syncthreads();
#pragma unroll
            for (int j = 0; j < ITEMS; ++j) {
                if (j < per && i0 + j * 32 < n) {
                    const uint32_t d = (key[j] >> shift) & mask;
                    const uint32_t to = local[d] + mine[d] + ((place[j / 2] >> (16 * (j & 1))) & 0xFFFFu);
                    if (CLUSTER) {
                        const uint32_t c = to / part, in = to - c * part;
                        ptx::st_cluster_u32(ptx::mapa_shared(ptx::smem_u32(skey + in), c), key[j]);
                        ptx::st_cluster_u32(ptx::mapa_shared(ptx::smem_u32(sidx + in), c), idx[j]);
                    } else {
                        skey[to] = key[j];
                        sidx[to] = idx[j];
                    }
                }
            }
            sync();
            if (!one || pass == p.passes - 1) {
                for (int i = t; i < part && q * part + i < n; i += kSortThreads) {
                    const uint32_t k = skey[i], d = (k >> shift) & mask, i_run = q * part + i;
                    const uint32_t to = one ? i_run : global[d] + (i_run - first[d]);
                    to_key[to] = k;
                    to_idx[to] = sidx[i];
                }
                if (!one) {
                    __syncthreads();
                    if (t < bins) global[t] += all;
                    sync();  // the items have left; global memory of this pass, too, is the next pass's input
                }
            }
        }
    }
}

// Zeros in the tables.  Behind the sort it begins when all of the sort's CTAs have passed their wait, so what came before them
// has ended; it ends after the sort, so that who waits for it waits for both.
__global__ void __launch_bounds__(kZeroThreads) embed_zero_kernel(const __grid_constant__ EmbedParams p) {
    if (p.M == 0) ptx::grid_wait();
    ptx::grid_launch_dependents();
    const int64_t packs = (int64_t)p.Vs * (p.N >> 3), step = (int64_t)gridDim.x * kZeroThreads;
    for (int r = 0; r < p.R; ++r) {
        uint4* to = reinterpret_cast<uint4*>(p.tables[r]);
        for (int64_t i = (int64_t)blockIdx.x * kZeroThreads + threadIdx.x; i < packs; i += step) to[i] = make_uint4(0u, 0u, 0u, 0u);
    }
    ptx::grid_wait();
}

// ------------------------------------------------------------------------- sums
// A thread's place: which chunk, which 8 columns.  Rows narrower than the block leave room for several chunks.
struct Where {
    int64_t chunk;
    int pack;
};
__device__ __forceinline__ Where where(const EmbedParams& p) {
    const int sub = threadIdx.x / p.width;
    Where x{(int64_t)blockIdx.x * p.block_chunks + sub, (int)(blockIdx.y * p.width + threadIdx.x - sub * p.width)};
    if (sub >= p.block_chunks || x.chunk >= p.chunks || x.pack >= p.N >> 3) x.pack = -1;
    return x;
}

__device__ __forceinline__ void store_row(const EmbedParams& p, uint32_t id, int pack, const Pack& sum) {
    uint4* to = reinterpret_cast<uint4*>(row_of(p.tables, id, p)) + pack;
    const uint64_t scale = pair(p.scale, p.scale);
    Pack f = {};
    if (p.accumulate) unpack8(*to, f);
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = fma2(sum[i], scale, f[i]);
    *to = pack8(f);
}

__device__ __forceinline__ void store_part(const EmbedParams& p, int64_t row, int pack, const Pack& sum) {
    uint64_t* to = reinterpret_cast<uint64_t*>(p.part + row * p.N + pack * 8);
#pragma unroll
    for (int i = 0; i < 4; ++i) to[i] = sum[i];
}

// Partial rows: 2c, the sum that goes on from the chunk before c; 2c + 1, the one that starts in c and goes on behind.
// A block's tokens come through shared memory, 512 at a time, so that a thread's loads of dy wait for no other.
__global__ void __launch_bounds__(kThreads, kSumBlocks) embed_sum_kernel(const __grid_constant__ EmbedParams p) {
    constexpr int kTokens = 512, U = 8;  // U: rows in flight
    __shared__ uint32_t keys[kTokens], order[kTokens];
    const Where x = where(p);
    const int t = threadIdx.x, sub = t / p.width;
    const int tile = min((int)p.chunk, kTokens / p.block_chunks);  // tokens of a chunk at a time
    const int64_t block0 = (int64_t)blockIdx.x * p.block_chunks;
    ptx::grid_launch_dependents();
    ptx::grid_wait();
    const int64_t first = x.chunk * p.chunk;
    const int n = x.pack < 0 ? 0 : (int)min(p.chunk, p.M - first);
    const uint32_t prev = n && first > 0 ? p.sorted[first - 1] : p.V, next = n && first + n < p.M ? p.sorted[first + n] : p.V;
    Pack sum = {};
    uint32_t cur = p.V;
    bool started = false;  // the current sum starts in this chunk
    for (int at = 0; at < (int)p.chunk; at += tile) {
        __syncthreads();
        for (int i = t; i < tile * p.block_chunks; i += blockDim.x) {
            const int c = i / tile, j = at + i - c * tile;
            const int64_t from = (block0 + c) * p.chunk + j;
            const bool in = j < (int)p.chunk && from < p.M;
            keys[i] = in ? p.sorted[from] : p.V;
            order[i] = in ? p.order[from] : 0u;
        }
        __syncthreads();
        const int end = min(tile, n - at);
        for (int i0 = 0; i0 < end; i0 += U) {
            uint32_t key[U];
            uint4 v[U];
#pragma unroll
            for (int j = 0; j < U; ++j) {
                key[j] = i0 + j < end ? keys[sub * tile + i0 + j] : p.V;
                if (key[j] < p.V) v[j] = ptx::ld_stream_v4(p.dy + (size_t)order[sub * tile + i0 + j] * p.N + x.pack * 8);
            }
#pragma unroll
            for (int j = 0; j < U; ++j) {
                if (key[j] >= p.V) continue;
                if (key[j] != cur) {
                    if (cur < p.V) {
                        if (started) store_row(p, cur, x.pack, sum);
                        else store_part(p, 2 * x.chunk, x.pack, sum);
                    }
                    started = at + i0 + j > 0 || key[j] != prev;
                    cur = key[j];
#pragma unroll
                    for (int i = 0; i < 4; ++i) sum[i] = 0ull;
                }
                Pack f;
                unpack8(v[j], f);
#pragma unroll
                for (int i = 0; i < 4; ++i) sum[i] = add2(sum[i], f[i]);
            }
        }
    }
    if (cur < p.V) {
        if (!started) store_part(p, 2 * x.chunk, x.pack, sum);
        else if (cur == next) {
            store_part(p, 2 * x.chunk + 1, x.pack, sum);
            if (x.pack == 0) {  // listed, in any order: those that go on for long from the front, the others from the end
                const int64_t far = (x.chunk + 1 + kShort) * p.chunk;
                if (far < p.M && p.sorted[far] == cur) p.crossing[2 + atomicAdd(p.crossing, 1u)] = (uint32_t)x.chunk;
                else p.crossing[1 + p.chunks - atomicAdd(p.crossing + 1, 1u)] = (uint32_t)x.chunk;
            }
        } else {
            store_row(p, cur, x.pack, sum);
        }
    }
}

// Ids that cross chunks: a sum starts in a listed chunk and goes on through the next ones, up to kShort of them, which one
// warp adds up, or more, of which a block's warps take equal runs, in order, and add the runs' sums in order.  (An id that
// makes up much of a batch has hundreds: 16384 tokens of 64 ids, 512 columns, a thread alone: 75 us.)
constexpr int kJoinWarps = 8;

// sum += the partial rows 2c of the chunks c0 .. c1 - 1
__device__ __forceinline__ void add_parts(const EmbedParams& p, int64_t c0, int64_t c1, int pack, Pack& sum) {
    constexpr int U = 4;  // rows in flight
    for (int64_t c = c0; c < c1; c += U) {
        Pack v[U];
#pragma unroll
        for (int j = 0; j < U; ++j)
            if (c + j < c1) load8(p.part + 2 * (c + j) * p.N + pack * 8, v[j]);
#pragma unroll
        for (int j = 0; j < U; ++j) {
            if (c + j < c1) {
#pragma unroll
                for (int i = 0; i < 4; ++i) sum[i] = add2(sum[i], v[j][i]);
            }
        }
    }
}

__global__ void __launch_bounds__(kJoinWarps * 32) embed_join_kernel(const __grid_constant__ EmbedParams p) {
    __shared__ uint64_t runs[kJoinWarps][4][32];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, P = p.N >> 3, slabs = (P + 31) / 32;
    ptx::grid_launch_dependents();
    ptx::grid_wait();
    const int64_t longs = (int64_t)p.crossing[0] * slabs, shorts = (int64_t)p.crossing[1] * slabs;
    for (int64_t i = blockIdx.x; i < longs; i += gridDim.x) {
        const int64_t chunk = p.crossing[2 + i / slabs];
        const int pack = (int)(i % slabs) * 32 + lane;
        const uint32_t id = p.sorted[(chunk + 1) * p.chunk];
        // the last chunk that begins with this id: 32 places at a time
        int64_t lo = chunk + 1, hi = p.chunks;  // lo does, hi does not
        while (hi - lo > 1) {
            const int64_t step = (hi - lo + 31) / 32, at = lo + (lane + 1) * step;
            const int far = __popc(__ballot_sync(0xFFFFFFFFu, at < hi && p.sorted[at * p.chunk] == id));  // (lanes that have it come first)
            hi = min(hi, lo + (far + 1) * step);
            lo += far * step;
        }
        const int64_t n = lo - chunk;
        Pack sum = {};
        if (pack < P) {
            if (w == 0) load8(p.part + (2 * chunk + 1) * p.N + pack * 8, sum);
            add_parts(p, chunk + 1 + n * w / kJoinWarps, chunk + 1 + n * (w + 1) / kJoinWarps, pack, sum);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) runs[w][k][lane] = sum[k];
        __syncthreads();
        if (w == 0 && pack < P) {
            for (int r = 1; r < kJoinWarps; ++r)
#pragma unroll
                for (int k = 0; k < 4; ++k) sum[k] = add2(sum[k], runs[r][k][lane]);
            store_row(p, id, pack, sum);
        }
        __syncthreads();
    }
    for (int64_t i = (int64_t)(gridDim.x - 1 - blockIdx.x) * kJoinWarps + w; i < shorts; i += (int64_t)gridDim.x * kJoinWarps) {
        const int64_t chunk = p.crossing[1 + p.chunks - i / slabs];
        const int pack = (int)(i % slabs) * 32 + lane;
        const int64_t at = chunk + 1 + lane;
        const uint32_t key = lane < kShort && at < p.chunks ? p.sorted[at * p.chunk] : p.V;
        const uint32_t id = __shfl_sync(0xFFFFFFFFu, key, 0);
        const int n = __popc(__ballot_sync(0xFFFFFFFFu, key == id));
        if (pack >= P) continue;
        Pack sum;
        load8(p.part + (2 * chunk + 1) * p.N + pack * 8, sum);
        add_parts(p, chunk + 1, chunk + 1 + n, pack, sum);
        store_row(p, id, pack, sum);
    }
}

// -------------------------------------------------------------------- few tokens
// Up to kFew tokens one launch does it all.  A warp takes a token and 256 columns and looks through the ids: the warp of an
// id's first token sums all of its rows, or, if there are many, the block's warps sum equal runs of them, in order.  (A
// warp's neighbours have the next tokens, so an id's columns lie in different blocks.)  Other blocks write zeros to the rows
// that no token has, which a table of the ids tells.  (300 x 1032, vocabulary 11001: 8.7 us, sort, sums and join 12.8, a
// block instead of a warp for each token 11.3; 513 tokens, which the sort takes, 13.5 us, 512 10.9.)
constexpr int kFew = kEmbedFew, kFewWarps = 8, kFewThreads = 32 * kFewWarps, kSlots = 1024;
constexpr int kHot = 32;  // rows that one warp sums
static_assert(kHot * kFewWarps <= kFew, "a list for each warp");
constexpr uint32_t kNone = 0xFFFFFFFFu;

__device__ __forceinline__ uint32_t slot_of(uint32_t id) { return (id * 2654435761u) >> 22; }

__global__ void __launch_bounds__(kFewThreads) embed_few_kernel(const __grid_constant__ EmbedParams p, int zero_blocks) {
    __shared__ uint32_t keys[kFew];
    __shared__ union {
        uint32_t slots[kSlots];
        struct {
            uint32_t list[kFew], hot[kFewWarps], many;
            uint64_t runs[kFewWarps][4][32];
        };
    } sh;
    const int t = threadIdx.x, lane = t & 31, w = t >> 5, M = (int)p.M, P = p.N >> 3;
    ptx::grid_launch_dependents();
    ptx::grid_wait();
    for (int i = t; i < M; i += kFewThreads) keys[i] = id_of(p, i);
    if ((int)blockIdx.x < zero_blocks) {
        for (int i = t; i < kSlots; i += kFewThreads) sh.slots[i] = kNone;
        __syncthreads();
        for (int i = t; i < M; i += kFewThreads) {
            const uint32_t k = keys[i];
            if (k >= p.V) continue;
            uint32_t s = slot_of(k);  // at most 512 of the 1024 slots are taken: the search ends
            for (uint32_t was; (was = atomicCAS(&sh.slots[s], kNone, k)) != kNone && was != k;) s = (s + 1) & (kSlots - 1);
        }
        __syncthreads();
        const int64_t packs = (int64_t)p.Vs * P, step = (int64_t)zero_blocks * kFewThreads;
        for (int r = 0; r < p.R; ++r) {
            uint4* to = reinterpret_cast<uint4*>(p.tables[r]);
            for (int64_t i = (int64_t)blockIdx.x * kFewThreads + t; i < packs; i += step) {
                const uint32_t id = r * p.Vs + (uint32_t)(packs <= 0xFFFFFFFFu ? (uint32_t)i / (uint32_t)P : i / P);
                uint32_t s = slot_of(id), k;
                while ((k = sh.slots[s]) != kNone && k != id) s = (s + 1) & (kSlots - 1);
                if (k == kNone) to[i] = make_uint4(0u, 0u, 0u, 0u);
            }
        }
        return;
    }
    const int slabs = (P + 31) / 32, first = (int)(blockIdx.x - zero_blocks) * kFewWarps;
    __syncthreads();
    // item i: token i % M, slab i / M
    auto add_rows = [&](const uint32_t* list, int n, int pack, Pack& sum) {
        constexpr int U = 8;  // rows in flight
        for (int c = 0; c < n; c += U) {
            uint4 v[U];
#pragma unroll
            for (int j = 0; j < U; ++j)
                if (c + j < n) v[j] = ptx::ld_stream_v4(p.dy + (size_t)list[c + j] * p.N + pack * 8);
#pragma unroll
            for (int j = 0; j < U; ++j) {
                if (c + j < n) {
                    Pack f;
                    unpack8(v[j], f);
#pragma unroll
                    for (int i = 0; i < 4; ++i) sum[i] = add2(sum[i], f[i]);
                }
            }
        }
    };
    // the tokens of `id` from `from` on, in order, into a list, up to `most` of them; how many there are
    auto find = [&](uint32_t id, int from, uint32_t* list, int most) {
        int n = 0;
        for (int j0 = from & ~31; j0 < M; j0 += 32) {
            const int j = j0 + lane;
            const uint32_t with = __ballot_sync(0xFFFFFFFFu, j >= from && j < M && keys[j] == id);
            const int at = n + __popc(with & ((1u << lane) - 1u));
            if ((with >> lane & 1) && at < most) list[at] = j;
            n += __popc(with);
        }
        __syncwarp();
        return n;
    };
    {
        const int item = first + w, token = item % M;
        const uint32_t id = item < slabs * M ? keys[token] : p.V;
        bool mine = id < p.V;
        for (int j0 = 0; j0 < token && mine; j0 += 32) mine = !__any_sync(0xFFFFFFFFu, j0 + lane < token && keys[j0 + lane] == id);
        uint32_t* const list = sh.list + w * kHot;
        const int n = mine ? find(id, token, list, kHot) : 0, pack = item / M * 32 + lane;
        if (lane == 0) sh.hot[w] = n > kHot;
        if (n > 0 && n <= kHot && pack < P) {
            Pack sum = {};
            add_rows(list, n, pack, sum);
            store_row(p, id, pack, sum);
        }
    }
    for (int h = 0; h < kFewWarps; ++h) {
        __syncthreads();
        if (!sh.hot[h]) continue;  // the same for the whole block
        const int item = first + h, token = item % M, pack = item / M * 32 + lane;
        if (w == 0) {
            const int n = find(keys[token], token, sh.list, kFew);
            if (lane == 0) sh.many = n;
        }
        __syncthreads();
        const int n = sh.many, c0 = n * w / kFewWarps;
        Pack sum = {};
        if (pack < P) add_rows(sh.list + c0, n * (w + 1) / kFewWarps - c0, pack, sum);
#pragma unroll
        for (int i = 0; i < 4; ++i) sh.runs[w][i][lane] = sum[i];
        __syncthreads();
        if (w == 0 && pack < P) {
            for (int r = 1; r < kFewWarps; ++r)
#pragma unroll
                for (int i = 0; i < 4; ++i) sum[i] = add2(sum[i], sh.runs[r][i][lane]);
            store_row(p, keys[token], pack, sum);
        }
    }
}

}  // namespace

template <bool CLUSTER, int ITEMS>
static cudaError_t opt_in_sort() {
    return cudaFuncSetAttribute(embed_sort_kernel<CLUSTER, ITEMS>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSortSmem<ITEMS>);
}
cudaError_t embed_prepare() {
    for (cudaError_t e : {opt_in_sort<false, 4>(), opt_in_sort<true, 4>(), opt_in_sort<true, 16>()})
        if (e != cudaSuccess) return e;
    return cudaSuccess;
}

template <bool CLUSTER, int ITEMS>
static cudaError_t launch_sort(const EmbedParams& p, cudaStream_t s) {
    cudaLaunchAttribute attr[2];
    attr[0] = dependent_launch();
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = kSortCluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(CLUSTER ? kSortCluster : 1);
    cfg.blockDim = dim3(kSortThreads);
    cfg.dynamicSmemBytes = kSortSmem<ITEMS>;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = CLUSTER ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, embed_sort_kernel<CLUSTER, ITEMS>, p);
}

// Keys and positions twice, and the list of chunks (of 8 tokens or more) in which an id starts that goes on behind.
size_t embed_sort_bytes(int64_t M_max) { return (size_t)M_max * 16 + (size_t)(M_max / 8 + 4) * 4; }

cudaError_t launch_embedding(const EmbedParams& p, int* grid, cudaStream_t s) {
    const int64_t packs = p.M * (p.N / 8), blocks = (packs + kThreads * 4 - 1) / (kThreads * 4);
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    *grid = (int)blocks;
    return launch_dependent(embed_kernel, dim3((unsigned)blocks), kThreads, 0, s, p);
}

cudaError_t launch_embedding_backward(EmbedParams& p, void* sort, float* scratch, int num_sms, int* grid, cudaStream_t s) {
    if (p.M > 0 && p.M <= kFew) {
        const int zeros = p.accumulate ? 0 : 4 * num_sms;
        *grid = zeros + ((int)p.M * ((p.N / 8 + 31) / 32) + 7) / 8;  // a warp an item, eight a block
        return launch_dependent(embed_few_kernel, dim3((unsigned)*grid), kFewThreads, 0, s, p, zeros);
    }
    // passes of equal length, of 10 bits at most; V itself stands for "no id"
    int bits = 1;
    while (bits < 32 && (p.V >> bits)) ++bits;
    p.passes = (bits + 9) / 10;
    p.digit_bits = (bits + p.passes - 1) / p.passes;
    uint32_t* words = static_cast<uint32_t*>(sort);
    for (int i = 0; i < 2; ++i) {
        p.keys[i] = words + (2 * i) * p.M;
        p.idx[i] = words + (2 * i + 1) * p.M;
    }
    p.crossing = words + 4 * p.M;
    const int last = (p.passes - 1) & 1;
    p.sorted = p.keys[last];
    p.order = p.idx[last];
    p.part = scratch;
    // a row's packs over blocks of equal width, or several chunks in a block
    const int P = p.N / 8, slabs = (P + kThreads - 1) / kThreads;
    p.width = (P + slabs - 1) / slabs;
    p.block_chunks = kThreads / p.width;
    // as many chunks as run at once (16384 x 4096: 222 of 74 tokens, 32 us; 373 of 44, which take a second round, 36),
    // two partial rows each, of those that a workspace of this width has, so that the order of the sums goes by the
    // sizes alone
    const int64_t rows = (int64_t)two_sums_words(p.N, num_sms) / p.N;
    const int64_t most = std::min<int64_t>(rows / 2, (int64_t)num_sms * kSumBlocks / slabs * p.block_chunks);
    p.chunk = std::max<int64_t>(8, (p.M + most - 1) / most);
    p.chunks = (p.M + p.chunk - 1) / p.chunk;
    const bool cluster = p.M > kSortOne;
    *grid = p.M == 0 ? 0 : cluster ? kSortCluster : 1;
    cudaError_t e = cudaSuccess;
    // (four items a thread need no spilled registers: 16384 x 1032 34 us, with room for 16 38)
    if (p.M > 0)
        e = !cluster                                 ? launch_sort<false, 4>(p, s)
            : p.M <= 4 * kSortCluster * kSortThreads ? launch_sort<true, 4>(p, s)
                                                     : launch_sort<true, 16>(p, s);
    // zeros on the SMs that the sort leaves: with a share for its own they would end late
    if (e == cudaSuccess && !p.accumulate) e = launch_dependent(embed_zero_kernel, dim3((unsigned)(kZeroBlocks * (num_sms - *grid))), kZeroThreads, 0, s, p);
    if (e != cudaSuccess || p.M == 0) return e;
    const int threads = (p.width * p.block_chunks + 31) / 32 * 32;
    const dim3 blocks((unsigned)((p.chunks + p.block_chunks - 1) / p.block_chunks), (unsigned)slabs);
    e = launch_dependent(embed_sum_kernel, blocks, threads, 0, s, p);
    if (e == cudaSuccess && p.chunks > 1)
        e = launch_dependent(embed_join_kernel, dim3((unsigned)std::min<int64_t>(3 * num_sms, p.chunks * ((P + 31) / 32))),
                             kJoinWarps * 32, 0, s, p);
    return e;
}

}  // namespace are
