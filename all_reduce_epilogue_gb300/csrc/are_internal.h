// Internal interfaces between the C-ABI layer (api.cu) and the kernels.
#pragma once
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "../../include/are.h"
#include "xent_sizes.h"

namespace are {

constexpr int kMaxRanks = 8;

// Device status word: first error wins (code 0 = no error).
struct DevStatus {
    uint32_t code;
    uint32_t where;
    int32_t a;
    int32_t b;
};

__device__ __forceinline__ void record_error(DevStatus* st, uint32_t code, uint32_t where, int32_t a, int32_t b) {
    if (atomicCAS(&st->code, 0u, code) == 0u) {
        st->where = where;
        st->a = a;
        st->b = b;
        __threadfence();
    }
}

// ------------------------------------------------------------------ AR+RMSNorm
constexpr uint32_t kSentinelF32 = 0x80000000u;  // -0.0 as an fp32 word
constexpr int kArThreads = 512;   // 1 producer warp + 7 phase-A warps + 8 phase-B warps
constexpr int kMaxArStages = 8;   // phase-A shared-memory stages (upper bound)
constexpr int kArRingSlots = 8;   // staging ring slots (chunks) when the rows wrap

struct ArParams {
    const uint16_t* x[kMaxRanks];  // R bf16 partials [M, N]
    const uint16_t* residual;      // bf16 [M, N] or nullptr
    const float* gamma;            // fp32 [N]
    uint16_t* out;                 // bf16 [M, N]
    uint16_t* residual_out;        // bf16 [M, N] or nullptr: bf16(h), h = canon(s) + residual
    uint8_t* out_q;                // FP8 E4M3 [M, N] or nullptr (then `out` is written)
    float* out_scale;              // fp32 [M] with out_q: the per-row scale
    uint32_t* staging;             // fp32 words, armed with the sentinel (chunk rows, see ring_slots)
    DevStatus* status;
    unsigned long long* counters;  // debug counters
    int R;
    int M;
    int N;
    int packs_per_row;  // N / 8
    int chunk_rows;     // rows per pipeline chunk (<= grid)
    int num_chunks;
    int ring_slots;     // 0: chunk c's rows at c*chunk_rows; else staging slot c % ring_slots
    int stages;         // phase-A shared-memory stages (set by ar_rmsnorm_smem_plan)
    int res_in_smem;    // residual rows streamed into shared memory (set by ar_rmsnorm_smem_plan)
    int gamma_in_smem;  // gamma copied into shared memory once per block (set by ar_rmsnorm_smem_plan)
    float eps;
    float inv_n;
    uint32_t flags;
    int64_t debug_arg;
    uint64_t timeout_ns;
};

// Packs-per-thread variant for a row of `packs_per_row` 8-element packs (0 if too wide).
int ar_rmsnorm_ppt(int packs_per_row);
constexpr int kArMaxPpt = 20;
// Choose the phase-A stage count and whether residual rows go through shared
// memory (needs p.N and p.residual set).
void ar_rmsnorm_smem_plan(ArParams& p);
// Largest grid that is fully co-resident for the packs-per-thread variant `ppt`.
int ar_rmsnorm_resident_blocks(int ppt, int num_sms);
cudaError_t launch_ar_rmsnorm(const ArParams& p, int ppt, int grid, cudaStream_t stream);
// One-shot AR+RMSNorm for small messages (one row per block, no staging).
size_t ar_oneshot_smem_bytes(int R, int N, bool residual);
bool ar_oneshot_fits(int R, int N, bool residual);
cudaError_t ar_oneshot_prepare();
cudaError_t launch_ar_oneshot(const ArParams& p, int ppt, int grid, cudaStream_t stream);
int ar_oneshot_threads();
// Fill n 32-bit words with v.
cudaError_t launch_fill_u32(uint32_t* dst, uint32_t v, size_t n, cudaStream_t stream);

// ------------------------------------------------------------------ row-streaming norm kernels
constexpr int kRowSources = kMaxRanks + 2;
constexpr int64_t kBackwardMaxN = 16384;  // widest row whose dgamma sums fit a block's registers

struct RowsParams {
    const uint16_t* src[kRowSources];  // bf16 [M, N] each: the R partials, then residual (forward) or h and d_res (backward)
    const float* gamma;                // fp32 [N]
    const float* beta;                 // LayerNorm forward: fp32 [N] or nullptr
    uint16_t* out;                     // LayerNorm forward: bf16 [M, N]
    uint16_t* res_out;                 // bf16 [M, N]: h or nullptr (forward); dh (backward)
    uint8_t* out_q;                    // forward: FP8 E4M3 codes [M, N]
    void* out_scale;                   // forward: [M, groups] fp32 or E8M0 bytes
    float* dgamma;                     // backward: partial sums [grid, N], or nullptr
    float* dbeta;                      // LayerNorm backward: the same
    DevStatus* status;
    int64_t M;
    int R;
    int N;
    int nsrc;           // sources in use
    int has_res;        // the last source (residual, d_res) is there
    int groups;         // forward: scales a row
    int group_packs;    // forward: 8-column packs a group (4, 8, 16)
    int backward;       // the backward pass (gamma in shared memory, fewer threads)
    int extra_words;    // fp32 words of shared memory of the kernel's own, a multiple of 4 (set by the plans)
    int red_words;      // words that a block's sums are exchanged in, a multiple of 4 (set by the plans)
    int lanes;          // LayerNorm: lanes that take a row (8, 16, 32), 0: a block does (set by layernorm_plan)
    int rows;           // LayerNorm backward: rows that a block takes at a time (set by layernorm_plan)
    int nt;             // consumer threads, a multiple of 32 (set by rows_plan)
    int slices;         // slices of nt packs a row (set by rows_plan)
    int stages;         // ring stages (set by rows_plan)
    int stage_bytes;    // (set by rows_plan)
    float eps;
    float inv_n;
    uint64_t timeout_ns;
};

// The attribute of a launch on the programmatic dependency (norm_rows.cu).
cudaLaunchAttribute dependent_launch();

struct RowsPlan {
    int ppt;      // packs of a row a thread owns at most (template variant)
    int threads;  // nt + the producer warp
    int grid;
    size_t smem;
};

// Fills p's plan fields from p.N, p.M, p.nsrc and p.backward.
RowsPlan rows_plan(RowsParams& p, int num_sms);
cudaError_t rows_prepare();
cudaError_t launch_norm_quant_rows(const RowsParams& p, const RowsPlan& plan, bool pow2, cudaStream_t stream);
// scratch: norm_backward_scratch_words() floats; dgamma may be nullptr.
cudaError_t launch_norm_backward_rows(RowsParams& p, const RowsPlan& plan, float* scratch, float* dgamma,
                                      cudaStream_t stream);
size_t norm_backward_scratch_words(int64_t n_max, int num_sms);
// Of the LayerNorm's, which sums dbeta too, and of the embedding's.
inline size_t two_sums_words(int64_t n_max, int num_sms) { return 2 * norm_backward_scratch_words(n_max, num_sms); }

// The columns' sums over `rows` partial rows [rows, N], and with `second` over as many right behind them.
cudaError_t launch_row_sums(const float* part, float* first, float* second, int rows, int N, cudaStream_t stream);

// LayerNorm on the same rows (layernorm.cu).  scratch: two_sums_words() floats; dgamma and dbeta may be nullptr.
RowsPlan layernorm_plan(RowsParams& p, int num_sms);
cudaError_t layernorm_prepare();
cudaError_t launch_layernorm_rows(const RowsParams& p, const RowsPlan& plan, cudaStream_t stream);
cudaError_t launch_layernorm_backward_rows(RowsParams& p, const RowsPlan& plan, float* scratch, float* dgamma,
                                           float* dbeta, cudaStream_t stream);

// ------------------------------------------------------------------ 4-bit weights, few tokens
struct QweightParams {
    const void* x[kMaxRanks];            // bf16 [M, K], or FP8 E4M3 codes [M, K]
    const void* xscale[kMaxRanks];       // fp32 or E8M0 [M, xgroups] (8-bit tokens)
    const uint8_t* codes[kMaxRanks];     // [N, K/2], the lower four bits first
    const uint16_t* scale[kMaxRanks];    // bf16 [N, groups]
    const uint8_t* zero[kMaxRanks];      // [N, groups] or nullptr (8)
    uint16_t* views[kMaxRanks];          // distinct outputs, bf16 [M, N]
    int R, nviews;
    int M, N, K;
    int group_shift, groups;             // log2 of the weight group, groups a row
    int qx;                              // tokens in 8 bits
    int xgroup_shift, xgroups;           // of the token scales
    int xpow2;
    int force_tile;                      // 0: by size; 8, 16, 32: tokens a tile; -1: 16 or 32
    DevStatus* status;
    unsigned long long timeout_ns;
    // set by launch_qweight:
    int kp;                              // K, up to whole 256
    uint8_t* tokens;                     // staged tokens [R][tiles_m][kp / 32][tile]: bf16 operands
    float* sums;                         // their sums [R][tiles_m][kp / shared group][tile]
    float* scales;                       // their scales [R][tiles_m][kp / 256 or xgroup][tile]
    uint32_t* flags;                     // [R][tiles_m][kp / 256]: tokens with a value that is not finite
    int cluster;                         // CTAs a cluster: R * splits
    int splits;                          // K splits of a rank
    int split_k;                         // K range of a split
    int tile_k, tiles_k;                 // K range of a shared-memory tile, tiles of a split
    int tiles_m;                         // token tiles
    int run;                             // row groups of a cluster
    int rtoks;                           // tokens of a tile that have sums, even
};

// What the launch shape depends on: resident clusters by cluster size.
struct QweightDevice {
    int clusters[kMaxRanks + 1];
};

cudaError_t qweight_prepare(QweightDevice& dev);
// Bytes of a rank's staged tokens: a tile of 32 of K = 28672 with groups of 32, or more of shorter rows.
constexpr size_t kQweightScratch = 2u << 20;
// Chooses the launch shape and launches (in parts, if `scratch` does not hold all tokens); `grid`, `variant` and `cluster` report it.
cudaError_t launch_qweight(QweightParams& p, const QweightDevice& dev, uint8_t* scratch, size_t scratch_bytes, int* grid,
                           int* variant, int* cluster, cudaStream_t s);

// ------------------------------------------------------------------ GEMM + reduce
constexpr int kBM = 128;
constexpr int kBN = 256;
constexpr int kBK = 64;
constexpr int kStages = 3;            // mainloop shared-memory stages
constexpr int kPStages = 3;           // partial_buf stages
constexpr int kSubBytes = 16384;      // one 128-row x 128-byte sub-tile
constexpr int kTilePartBytes = 131072;  // fp32 128x256 partial (bf16 uses the first half)
constexpr int kGemmThreads = 256;
constexpr int kPieceWords = 64;       // debug piece log words per tile
constexpr int kChunkCap = 64;         // completion counters per owner segment (largest chunk count)
constexpr unsigned long long kChunkQ = 1ull << 32;  // counter advance per completed chunk

enum GemmMode : int { kModeRS = 0, kModeAR = 1 };

struct GemmParams {
    CUtensorMap tmA[kMaxRanks];
    CUtensorMap tmB[kMaxRanks];
    CUtensorMap tmOut[kMaxRanks];  // GEMM+RS: owner segments (64 x H boxes); GEMM+AR: the distinct views
                                   // (64 x 128 boxes for the one-CTA kernel, 64 x 16 for the pair kernel)
    // CTA-pair kernel: the partial slots as [R][T][16 sub-tiles][128 rows][16 words], boxes of
    // 8 sub-tiles x 16 rows (one 8 KB partial-buffer stage of a row slice's 16-row group)
    CUtensorMap tmPart;
    are_bf16* views[kMaxRanks];  // GEMM+AR: distinct output views; GEMM+RS with rs_split: the owner
                                 // segments (row groups that no box covers: st.global)
    uint8_t* part;       // [R][T][tile part bytes]
    uint32_t* mask;      // [T]
    DevStatus* status;
    int32_t* pieces;     // debug piece log [T][kPieceWords]
    unsigned long long* counters;  // debug counters (wait profile)
    int R;
    int M, N, K;
    int S;               // owner segment rows (RS)
    int H;               // output box height (RS)
    int nviews;          // distinct output views (AR)
    int tiles_m, tiles_n, num_tiles, num_units, num_kb;
    int pairs_m, num_pair_units;  // CTA-pair kernel: 256-row tile pairs, R units per pair
    int block_tiles;     // CTA-pair kernel: tile pairs per rank block (0 = ranks innermost)
    int rs_split;        // CTA-pair kernel, GEMM+RS: 1 = every unit reduces its row slice of the tile
                         // (two-shot, as GEMM+AR); 0 = the running sum is pushed along the ranks
    int rank_group;      // CTA-pair kernel: ranks run together inside a block (1 = rank by rank)
    uint32_t* cons;      // CTA-pair kernel, GEMM+AR: row-slice readers done per tile (0 between calls)
    int group_m;         // tile raster: rows of tiles (pairs) per group
    // chunked owner-segment completion (GEMM+RS; chunk_ctr == nullptr: off)
    unsigned long long* chunk_ctr;  // [R][kChunkCap] monotonic completion counters
    uint32_t* chunk_host;           // [R][kChunkCap] completed generation, host-mapped (may be null)
    int chunks;          // requested chunks per owner segment
    // destination-rotated order of the pair kernel (rot_pc == 0: raster order)
    int rot_pc;          // pair rows per order chunk
    int rot_cs;          // order chunks per owner segment
    int rot_ps;          // pair rows per owner segment
    int rot_w;           // tile columns per destination rotation (stripe)
    uint32_t flags;
    int64_t debug_arg;
    uint64_t timeout_ns;
};

// ------------------------------------------------------------------ embedding (embedding.cu)
struct EmbedParams {
    uint16_t* tables[kMaxRanks];  // bf16 [Vs, N]: the tables (forward, read only) or their gradients
    const void* ids;              // [M]
    const uint16_t* dy;           // backward: bf16 [M, N]
    uint16_t* out;                // forward: bf16 [M, N]
    int64_t M;
    int N, R;
    uint32_t Vs, V;               // rows of a rank, of all ranks
    int wide;                     // ids of 64 bits
    int accumulate;
    float scale;
    // backward, set at the launch
    uint32_t* keys[2];            // ids, and the tokens' positions, between the passes of the sort
    uint32_t* idx[2];
    const uint32_t* sorted;       // after the last pass
    const uint32_t* order;
    int passes, digit_bits;
    int64_t chunk, chunks;        // sorted tokens of a chunk
    uint32_t* crossing;           // how many chunks have an id that starts in them and goes on behind, and which
    int width, block_chunks;      // 8-column packs of a row that a block takes; chunks it takes
    float* part;                  // [2 chunks, N]
};

constexpr int kEmbedFew = 512;  // tokens whose gradient is one launch
cudaError_t embed_prepare();
size_t embed_sort_bytes(int64_t M_max);
cudaError_t launch_embedding(const EmbedParams& p, int* grid, cudaStream_t stream);
// sort: embed_sort_bytes(M); scratch: two_sums_words(N, num_sms) floats.  Up to kEmbedFew tokens need neither.
cudaError_t launch_embedding_backward(EmbedParams& p, void* sort, float* scratch, int num_sms, int* grid, cudaStream_t stream);

// ------------------------------------------------------------------ cross entropy (cross_entropy.cu)
enum XentPass : int { kXentLogSum = 0, kXentDLogits = 1, kXentDH = 2, kXentDW = 3, kXentGrads = 4 };

// n / d for n < 2^31 as a product and a shift (Granlund and Montgomery 1994): with s = ceil(log2 d) and mul = floor(2^(31+s) / d)
// + 1 the product is less than n 2^-(31+s) <= 1/d too large.
struct Divisor {
    uint32_t mul = 0, shift = 0;
    Divisor() = default;
    explicit Divisor(uint32_t d) {
        uint32_t s = 0;
        while ((1ull << s) < d) ++s;
        mul = (uint32_t)((1ull << (31 + s)) / d + 1);
        shift = 31 + s;
    }
};

struct XentGrid {
    int tiles_m, tiles_n;  // 256 x 256
    int splits;            // parts of the contraction
    int num_kb;            // its blocks of 64
    int units;             // tiles_m * tiles_n * splits (set at the launch, as what follows)
    Divisor per_split, per_group, rows, last_rows, parts;  // tiles of a split, of a group; rows of a group, of the last one; splits
};

struct XentParams {
    CUtensorMap tmA, tmA2, tmB;   // A; kXentDW's A (d) and B (h)
    CUtensorMap tmW[kMaxRanks];   // B of the others: the ranks' weights
    CUtensorMap tmOut[kMaxRanks]; // d, or the ranks' dW
    CUtensorMap tmDH;             // dh or its sums
    const void* targets;
    const float* lse;
    const float* dloss;
    float2* stats;                // kXentLogSum: [M, tiles_n, groups of columns] (maximum, sum of exp) pairs
    float* target_logit;          // [M]
    DevStatus* status;
    int64_t vocab;                // columns of all ranks that count
    int M, K, Vs, R;
    int wide;                     // targets of 64 bits
    int tile;                     // columns of a vocabulary tile: 256, or 128 of one CTA
    int rank_tiles, tile0;        // vocabulary tiles of a rank; the piece's first
    Divisor per_rank;             // rank_tiles (set at the launch)
    XentGrid grid[2];             // the second: kXentDW's in kXentGrads
    int a_rows;                   // rows of A that a copy takes: 128, fewer if M is less
    int group;                    // rows of tiles taken together
    int units;                    // (set at the launch)
    int sums, add;                // kXentDH: fp32 sums, added to what is there
    int second, columns;          // d has a second bf16 part (1) or not (0), which lies `columns` behind the first
    const uint4* rows_from;       // kXentDLogits: h, or nullptr
    uint4* rows_to;               // and its copy with zeros in the rows that have no target
    uint64_t timeout_ns;
};

struct XentCall {
    const are_bf16* h;
    const are_bf16* w[kMaxRanks];
    const void* targets;
    int wide;
    int R;
    int64_t M, Vs, K, vocab;
    float* loss;                  // forward
    float* lse;                   // forward: written; backward: read
    const float* dloss;           // backward
    are_bf16* dh;                 // backward, or nullptr
    are_bf16* dw[kMaxRanks];      // backward
    bool has_dw;
};

struct XentBuffers {
    void *d, *sums, *h, *rows;
    XentSizes sizes;
    int parts;                    // bf16 parts of d: 2, or 1
    int clusters;
    DevStatus* status;
    uint64_t timeout_ns;
};

cudaError_t xent_prepare(int* clusters);
cudaError_t launch_xent_forward(const XentCall& c, const XentBuffers& b, cudaStream_t stream, are_launch_info* info);
cudaError_t launch_xent_backward(const XentCall& c, const XentBuffers& b, cudaStream_t stream, are_launch_info* info);

size_t gemm_smem_bytes();
cudaError_t gemm_prepare_kernels();
// bf16 [outer, inner] row-major tensor map, 128B-swizzled boxes of box_inner x box_outer.
cudaError_t make_tmap_bf16(CUtensorMap* m, const void* base, uint64_t inner, uint64_t outer, uint32_t box_inner,
                           uint32_t box_outer);
// The pair kernel's partial slots for T tiles and R ranks as a 5-D map (see GemmParams::tmPart).
cudaError_t make_tmap_part(CUtensorMap* m, const void* part, uint64_t T, uint64_t R);
cudaError_t launch_gemm_reduce(const GemmParams& p, int mode, int grid, cudaStream_t stream);
// CTA-pair variant (cta_group::2 UMMA, 256x256 per pair); grid = 2 x clusters.
cudaError_t launch_gemm_pair(const GemmParams& p, int mode, int grid, cudaStream_t stream);
// Largest number of co-resident 2-CTA clusters of the pair kernel on the current
// device (0 if unavailable); valid after gemm_prepare_kernels() on that device.
int gemm_pair_max_clusters();
int gemm_pair_threads();

}  // namespace are
