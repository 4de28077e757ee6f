// api.cu -- host layer of the C ABI: the pool object, argument validation,
// the split-KV plan and kernel launches.  Nothing here allocates or
// synchronises on the append / decode path.
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <limits>
#include <mutex>
#include <new>

#include "kernels.h"
#include "kv_block_manager.h"
#include "kv_mla.h"
#include "kv_paged.h"

struct kv_pool {
    int num_blocks, block_size, kv_heads, head_dim, device;
    kv_dtype dtype;
    size_t elem;            // bytes per cached element
    size_t pool_bytes;      // bytes of the K pool (= bytes of the V pool)
    void* base;             // the single allocation
    uint8_t* k;
    uint8_t* v;
    float* k_scale;
    float* v_scale;
    uint32_t* err;
    CUtensorMap tmk, tmv;   // 5-D tile maps of the K and V pools; latent pools: the map
                            // with the stage box of the producer-warp decode (tmk) and of
                            // the three-CTA decode (tmv)
    CUtensorMap tmt;        // latent pools with blocks of 64: one 128-byte piece of a block
                            // per box (the wide tcgen05 decode)
    CUtensorMap tmh;        // latent pools with blocks of 64: one 128-byte piece of 32 slots
                            // per box (the narrow tcgen05 decode)
    CUtensorMap tmsk[3], tmsv[3]; // K and V pools in boxes of 16 slots of 1, 2, 4 kv heads (the span kernel)
    CUtensorMap tmpk, tmpv; // K and V pools in octets of slots (the shared prefix pass)
    int has_tc;
    int num_sms;
    int mla;                // 1: latent pool (one cached vector per token, no V half)
};

namespace {

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn()
{
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000,
                                             cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(ptr);
    });
    return fn;
}

constexpr size_t kAlign = 256;
size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Failure-path test hook of the decode kernels (kv_debug_decode_stall).
std::atomic<int> g_stop_stage{-1};
std::atomic<unsigned long long> g_consumer_wait_ns{0};

// Restores the caller's current device on scope exit.
struct DeviceGuard {
    int prev = -1;
    bool ok = false;
    explicit DeviceGuard(int dev)
    {
        if (cudaGetDevice(&prev) != cudaSuccess) return;
        ok = (prev == dev) || cudaSetDevice(dev) == cudaSuccess;
    }
    ~DeviceGuard()
    {
        if (prev >= 0) cudaSetDevice(prev);
    }
};

bool variant_supported(kv_dtype dtype, int head_dim, int block_size)
{
    if (block_size != 16 && block_size != 32) return false;
    if (dtype == KV_DTYPE_BF16) return head_dim == 64 || head_dim == 128;
    if (dtype == KV_DTYPE_FP8_E4M3) return head_dim == 128;
    return false;
}

// Tile map of one pool half: dims (innermost first) = 128-byte row piece,
// pieces per token row, kv head, slot, block; a box is one block of one kv
// head, written to shared memory with the 128-byte swizzle.
kv_status encode_pool_map(const kv_pool* p, uint8_t* base, CUtensorMap* map, int slots_per_box = 0,
                          int pieces_per_box = 0)
{
    EncodeTiledFn fn = encode_fn();
    if (fn == nullptr) return KV_ERR_CUDA;
    const cuuint64_t row = static_cast<cuuint64_t>(p->head_dim) * p->elem;
    const cuuint64_t per_piece = 128 / p->elem;
    const cuuint64_t dims[5] = {per_piece, row / 128, static_cast<cuuint64_t>(p->kv_heads),
                                static_cast<cuuint64_t>(p->block_size),
                                static_cast<cuuint64_t>(p->num_blocks)};
    const cuuint64_t strides[4] = {128, row, row * p->kv_heads, row * p->kv_heads * p->block_size};
    const cuuint32_t box[5] = {static_cast<cuuint32_t>(per_piece),
                               static_cast<cuuint32_t>(pieces_per_box > 0 ? pieces_per_box
                                                                          : row / 128), 1,
                               static_cast<cuuint32_t>(slots_per_box > 0 ? slots_per_box
                                                                         : p->block_size), 1};
    const cuuint32_t estride[5] = {1, 1, 1, 1, 1};
    const CUtensorMapDataType dt = p->dtype == KV_DTYPE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                             : CU_TENSOR_MAP_DATA_TYPE_UINT8;
    CUresult r = fn(map, dt, 5, base, dims, strides, box, estride, CU_TENSOR_MAP_INTERLEAVE_NONE,
                    CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? KV_OK : KV_ERR_CUDA;
}

// Tile map of one pool half for the span kernel: dims (innermost first) = 128-byte row piece, pieces
// per token row, slot, kv head, block; a box is 16 slots of `heads` kv heads, written head by head,
// each as encode_pool_map's tile.
kv_status encode_span_map(const kv_pool* p, uint8_t* base, int heads, CUtensorMap* map)
{
    EncodeTiledFn fn = encode_fn();
    if (fn == nullptr) return KV_ERR_CUDA;
    const cuuint64_t row = static_cast<cuuint64_t>(p->head_dim) * p->elem;
    const cuuint64_t token = row * p->kv_heads;
    const cuuint64_t dims[5] = {128 / p->elem, row / 128, static_cast<cuuint64_t>(p->block_size),
                                static_cast<cuuint64_t>(p->kv_heads), static_cast<cuuint64_t>(p->num_blocks)};
    const cuuint64_t strides[4] = {128, token, row, token * p->block_size};
    const cuuint32_t box[5] = {static_cast<cuuint32_t>(128 / p->elem), static_cast<cuuint32_t>(row / 128), 16,
                               static_cast<cuuint32_t>(heads), 1};
    const cuuint32_t estride[5] = {1, 1, 1, 1, 1};
    const CUtensorMapDataType dt = p->dtype == KV_DTYPE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                             : CU_TENSOR_MAP_DATA_TYPE_UINT8;
    CUresult r = fn(map, dt, 5, base, dims, strides, box, estride, CU_TENSOR_MAP_INTERLEAVE_NONE,
                    CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? KV_OK : KV_ERR_CUDA;
}

// Tile map of one pool half for the shared prefix pass: dims (innermost first) = 128-byte row
// piece, slot of an octet, pieces per token row, octet of slots (of all blocks), kv head; a box
// is one block of one kv head, written as octets of [piece][8 slots][128 bytes] with the 128-byte
// swizzle -- 8-row groups of the tensor cores' operand layout one after another.
kv_status encode_octet_map(const kv_pool* p, uint8_t* base, CUtensorMap* map)
{
    EncodeTiledFn fn = encode_fn();
    if (fn == nullptr) return KV_ERR_CUDA;
    const cuuint64_t row = static_cast<cuuint64_t>(p->head_dim) * p->elem;
    const cuuint64_t token = row * p->kv_heads;
    const cuuint64_t dims[5] = {128 / p->elem, 8, row / 128,
                                static_cast<cuuint64_t>(p->num_blocks) * (p->block_size / 8),
                                static_cast<cuuint64_t>(p->kv_heads)};
    const cuuint64_t strides[4] = {token, 128, 8 * token, row};
    const cuuint32_t box[5] = {static_cast<cuuint32_t>(128 / p->elem), 8, static_cast<cuuint32_t>(row / 128),
                               static_cast<cuuint32_t>(p->block_size / 8), 1};
    const cuuint32_t estride[5] = {1, 1, 1, 1, 1};
    const CUtensorMapDataType dt = p->dtype == KV_DTYPE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                             : CU_TENSOR_MAP_DATA_TYPE_UINT8;
    CUresult r = fn(map, dt, 5, base, dims, strides, box, estride, CU_TENSOR_MAP_INTERLEAVE_NONE,
                    CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? KV_OK : KV_ERR_CUDA;
}

// Tile map of the absorbed queries [batch, q_heads, MLA_DK] (bf16) for the narrow
// tcgen05 decode: dims (innermost first) = number, head, sequence; a box is one 64-number
// piece of min(16, q_heads) heads, written to shared memory with the 128-byte swizzle
// (heads past q_heads read as zeros).
kv_status encode_query_map(const uint16_t* q, int q_heads, int batch, CUtensorMap* map)
{
    EncodeTiledFn fn = encode_fn();
    if (fn == nullptr) return KV_ERR_CUDA;
    const cuuint64_t row = static_cast<cuuint64_t>(kvp::MLA_DK) * 2;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(kvp::MLA_DK), static_cast<cuuint64_t>(q_heads),
                                static_cast<cuuint64_t>(batch)};
    const cuuint64_t strides[2] = {row, row * static_cast<cuuint64_t>(q_heads)};
    const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(q_heads < kvp::MLA_TCN_HEADS ? q_heads
                                                                                       : kvp::MLA_TCN_HEADS), 1};
    const cuuint32_t estride[3] = {1, 1, 1};
    CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint16_t*>(q), dims, strides, box,
                    estride, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? KV_OK : KV_ERR_CUDA;
}

struct Plan {
    int group, rows, head_tile, head_groups, split_blocks, max_splits;
    int cta_heads, cta_per_sm;  // kv heads per CTA (1: paged_decode_main), its CTAs per SM
};

// Split-KV plan.  Automatic chunk size: about eight chunks per SM over the
// worst case (every sequence at max_blocks), kept between 64 and 192 blocks --
// long enough that a CTA's start and epilogue are a small part of its life,
// short enough that the last CTAs to start (the remainder chunks, launched
// last) end soon.  Measured on GB300 for the Llama-3-8B-shaped, ragged and
// long-context batches, the best chunks lie between 96 and 256 blocks.
kv_status make_plan(const kv_pool* pl, int batch, int q_heads, int q_len, int max_blocks,
                    int split_tokens, Plan* out)
{
    if (pl == nullptr || batch < 0 || q_heads <= 0 || q_len <= 0 || max_blocks <= 0 ||
        split_tokens < 0)
        return KV_ERR_INVALID_ARG;
    if (q_heads % pl->kv_heads != 0) return KV_ERR_INVALID_ARG;
    if (split_tokens % pl->block_size != 0) return KV_ERR_INVALID_ARG;
    if (static_cast<long long>(max_blocks) * pl->block_size > std::numeric_limits<int>::max())
        return KV_ERR_INVALID_ARG;
    if (static_cast<long long>(q_heads / pl->kv_heads) * q_len > 4096) return KV_ERR_UNSUPPORTED;
    Plan p;
    p.group = q_heads / pl->kv_heads;
    p.rows = p.group * q_len;
    p.head_tile = kvp::head_tile_for_group(p.rows);
    p.head_groups = (p.rows + p.head_tile - 1) / p.head_tile;
    // CTA shape.  With the automatic chunk, decode rows of one tile per kv head run the
    // kernel whose CTA covers a group of kv heads where it is built: two kv heads of a
    // bf16 pool of head_dim 128 and blocks of 16 (three CTAs per SM), four of an fp8 pool
    // of head_dim 128 and blocks of 32 (two per SM) -- measured on GB300 faster than one
    // CTA per kv head with the automatic chunk (Llama-3-8B-shaped layer 95.7 against
    // 99.4-101.1 us; fp8 batch 328 against 334 us).  A chunk given by the caller keeps one
    // CTA per kv head: for the same chunk that grid has more CTAs, which long chunks need
    // to fill the GPU (long-context batch, 4,096-token chunks: 385 against 479 us).
    p.cta_heads = 1;
    p.cta_per_sm = 3;
    if (split_tokens == 0 && p.head_tile == 8) {
        const bool fp8 = pl->dtype == KV_DTYPE_FP8_E4M3;
        const int hc = fp8 ? 4 : 2, ct = fp8 ? 2 : 3;
        if (pl->kv_heads % hc == 0 &&
            kvp::decode_heads_supported(fp8, pl->head_dim, pl->block_size, p.head_tile, hc, ct)) {
            p.cta_heads = hc;
            p.cta_per_sm = ct;
        }
    }
    if (split_tokens > 0) {
        p.split_blocks = split_tokens / pl->block_size;
    } else {
        const long long units = static_cast<long long>(batch > 0 ? batch : 1) * pl->kv_heads *
                                p.head_groups;
        const long long work = units * max_blocks;
        const long long target = static_cast<long long>(pl->num_sms > 0 ? pl->num_sms : 148) * 8;
        long long sb = (work + target - 1) / target;
        // (the two-head CTA measured best at up to 128 blocks on the ragged batch: 201 us
        // at 2,048 tokens against 217 us at 3,072)
        const long long most = p.cta_heads == 2 ? 128 : 192;
        if (sb < 64) sb = 64;
        if (sb > most) sb = most;
        p.split_blocks = static_cast<int>(sb);
    }
    if (p.split_blocks > max_blocks) p.split_blocks = max_blocks;
    p.max_splits = (max_blocks + p.split_blocks - 1) / p.split_blocks;
    if (p.max_splits > 65535) return KV_ERR_UNSUPPORTED;      // grid z limit
    *out = p;
    return KV_OK;
}

// Plan of the span kernel, whose tiles see at most `span_blocks` blocks of a sequence: units of
// (sequence, group of kv heads, row tile), and a grid of the CTAs that are resident together, or
// fewer where ranges of the least length cover everything.
struct SpanPlan {
    int rows, head_tile, head_groups, heads, least, ctas;
    long long units;
};

// Least positions of a CTA's range with the automatic choice: with fewer, small calls have more pieces
// to merge, with more, fewer SMs at work (one sequence of 480 tokens: 5 10.4 us, 6 10.8, 10 12.6; four
// samples of one prompt 17.2, 17.1, 21.6; larger calls do not depend on it).
constexpr int kSpanLeast = 2 + kvp::SPAN_PAD;

// Tokens a group has to save at least, (members - 1) x shared, to be computed once: less costs more in
// runs of the shared pass, pieces and their merge than it saves.  With 0 / 1,024 / 2,048 / 2,560 / 4,096:
//   32 groups of 8 behind 512 tokens                              161 / 161 / 163 / 165 / 173 us
//   four samples of 512 tokens                                    16.1 / 16.1 / 15.2 / 15.3 / 15.1
//   41 pairs of sequences behind 1,364, 8 kv heads                60 / 62 / 53 / 53 / 53
//   46 pairs behind 22 (8-bit)                                    42 / 17 / 17 / 17 / 17
//   16 pairs behind 2,196, 8 kv heads (8-bit)                     - / 52 / 47 / 37 / 37
//   12 pairs behind 3,102, 2 kv heads (8-bit)                     29 / 29 / 32 / 34 / 24
//   125 sequences behind 35, 3 new tokens (8-bit)                 - / 77 / 77 / 77 / 60
// With nothing shared at all the last five take 47 / 17 / 32 / 19 / 56 us: pairs, and many members behind
// little, want more than 2,048 tokens, the many groups of the first line fewer.  What sharing saves are
// bytes (kv heads and element size count too), what it costs is a pass and its runs; a rule by tokens
// alone is off by up to 42 % on single calls.
constexpr int kShareTokens = 2048;

kv_status make_span_plan(const kv_pool* pl, int batch, int q_heads, int q_len, int max_blocks,
                         int span_blocks, int split_tokens, SpanPlan* out)
{
    if (pl == nullptr || pl->mla || batch < 0 || q_heads <= 0 || q_len <= 0 || max_blocks <= 0 || split_tokens < 0)
        return KV_ERR_INVALID_ARG;
    if (q_heads % pl->kv_heads != 0 || split_tokens % pl->block_size != 0) return KV_ERR_INVALID_ARG;
    if (static_cast<long long>(max_blocks) * pl->block_size > std::numeric_limits<int>::max())
        return KV_ERR_INVALID_ARG;
    if (static_cast<long long>(q_heads / pl->kv_heads) * q_len > 4096) return KV_ERR_UNSUPPORTED;
    SpanPlan p;
    p.rows = q_heads / pl->kv_heads * q_len;
    p.head_tile = kvp::head_tile_for_group(p.rows);
    p.head_groups = (p.rows + p.head_tile - 1) / p.head_tile;
    const long long subs = static_cast<long long>(span_blocks) * (pl->block_size / 16) + kvp::SPAN_PAD;
    if (p.head_groups * subs > (1 << 30)) return KV_ERR_UNSUPPORTED;        // positions of a kv head group
    const long long resident = static_cast<long long>(pl->num_sms) * kvp::SPAN_CTAS;
    p.least = split_tokens > 0 ? split_tokens / 16 : kSpanLeast;
    // Kv heads per CTA.  Four (where they divide): a warp owns its rows, and a unit's beginning and
    // end are paid once for four heads -- 64 x 4,096 tokens of 8 heads, 8-bit: 125 us, with two heads
    // 148, with one 203; bf16 163 / 166 / 184.  Two where four would leave CTAs without work, so that
    // the same tokens are spread over twice the CTAs: 4 x 512 tokens of 8 heads 12.1 / 11.0 / 11.4 us,
    // 16 x 512 14.2 / 12.8 / 14.7; with the grid just full they are even (64 x 512 tokens of 4 heads
    // 15.7 / 16.3 / 20.5).
    const auto cut = [&](int heads) {
        p.heads = heads;
        p.units = static_cast<long long>(batch) * (pl->kv_heads / heads) * p.head_groups;
        const long long most = (p.units * subs + p.least - 1) / p.least;
        p.ctas = static_cast<int>(most < resident ? most : resident);
    };
    cut(pl->kv_heads % 4 == 0 ? 4 : pl->kv_heads % 2 == 0 ? 2 : 1);
    if (p.heads == 4 && p.ctas < resident) cut(2);
    *out = p;
    return KV_OK;
}

// Window as the kernel takes it: one that covers every position is none.
int effective_window(const kv_pool* pl, int window, int max_blocks)
{
    return window >= static_cast<long long>(max_blocks) * pl->block_size ? 0 : window;
}

// Most blocks that a tile's rows see: window + q_len - 1 tokens at any offset, or all.
int masked_span_blocks(const kv_pool* pl, int q_len, int max_blocks, int window)
{
    if (window <= 0) return max_blocks;
    const long long tokens = static_cast<long long>(window) + q_len - 1;
    const long long blocks = (tokens + pl->block_size - 2) / pl->block_size + 1;
    return blocks < max_blocks ? static_cast<int>(blocks) : max_blocks;
}

kv_status make_masked_plan(const kv_pool* pl, int batch, int q_heads, int q_len, int max_blocks,
                           int window, int split_tokens, SpanPlan* out)
{
    if (pl == nullptr || window < 0 || q_len <= 0 || max_blocks <= 0) return KV_ERR_INVALID_ARG;
    window = effective_window(pl, window, max_blocks);
    return make_span_plan(pl, batch, q_heads, q_len, max_blocks,
                          masked_span_blocks(pl, q_len, max_blocks, window), split_tokens, out);
}

// Workspace layout (only when a sequence can have several chunks): partial
// outputs [batch, q_heads, max_splits, d], (max, sum) pairs [batch, q_heads,
// max_splits, 2], then one ticket per (sequence, kv head, head tile).
struct WorkspaceLayout {
    size_t part_o, part_ml, tickets, ticket_bytes, total;
};

WorkspaceLayout workspace_layout(const kv_pool* pl, int batch, const Plan& p)
{
    WorkspaceLayout w{0, 0, 0, 0, 0};
    if (p.max_splits <= 1) return w;
    const size_t n = static_cast<size_t>(batch) * pl->kv_heads * p.rows * p.max_splits;
    w.part_ml = round_up(n * pl->head_dim * sizeof(float), kAlign);
    w.tickets = w.part_ml + round_up(n * 2 * sizeof(float), kAlign);
    w.ticket_bytes = static_cast<size_t>(batch) * pl->kv_heads * p.head_groups * sizeof(int);
    w.total = w.tickets + w.ticket_bytes;
    return w;
}

size_t workspace_bytes_for(const kv_pool* pl, int batch, const Plan& p)
{
    return workspace_layout(pl, batch, p).total;
}

// Workspace of the span kernel: tickets, then the pieces of cut units, two per CTA and head: (max, sum)
// pairs, partial outputs.  The tickets' place does not depend on the call's sizes: whatever call
// used the workspace before, they are zero.
struct SpanLayout {
    size_t part_ml, part_o, total;
};

SpanLayout span_layout(const kv_pool* pl, const SpanPlan& p)
{
    SpanLayout w;
    const size_t rows = static_cast<size_t>(p.ctas) * 2 * p.heads * p.head_tile;
    w.part_ml = round_up(static_cast<size_t>(pl->num_sms) * kvp::SPAN_CTAS * 2 * 4 * sizeof(int), kAlign);
    w.part_o = w.part_ml + round_up(rows * 2 * sizeof(float), kAlign);
    w.total = w.part_o + round_up(rows * pl->head_dim * sizeof(float), kAlign);
    return w;
}

// The shared prefix pass's part of a workspace (behind the span kernel's): run entries, log-sum-exps,
// partial outputs.  Pieces: one per run and one per range border of the grid (one CTA per SM).
struct PrefixLayout {
    size_t runs, piece_lse, piece_o, total;
    long long pieces;
};

PrefixLayout prefix_layout(const kv_pool* pl, int batch, const SpanPlan& p, int n_groups)
{
    PrefixLayout w{0, 0, 0, 0, 0};
    if (n_groups == 0 || batch < 2) return w;
    const long long runs = kvp::prefix_run_slots(batch, pl->kv_heads, p.rows, n_groups);
    w.pieces = runs + pl->num_sms;
    w.piece_lse = round_up(static_cast<size_t>(runs) * sizeof(int2), kAlign);
    w.piece_o = w.piece_lse + static_cast<size_t>(w.pieces) * 256 * sizeof(float4);
    w.total = w.piece_o + static_cast<size_t>(w.pieces) * 256 * pl->head_dim * sizeof(float);
    return w;
}

kv_status check_device(const kv_pool* pl)
{
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) return KV_ERR_CUDA;
    return dev == pl->device ? KV_OK : KV_ERR_INVALID_ARG;
}

}  // namespace

extern "C" {

int kv_abi_version(void) { return KV_PAGED_ABI_VERSION; }

const char* kv_status_string(kv_status s)
{
    switch (s) {
    case KV_OK: return "ok";
    case KV_ERR_INVALID_ARG: return "invalid argument";
    case KV_ERR_OUT_OF_MEMORY: return "out of device memory";
    case KV_ERR_OUT_OF_BLOCKS: return "out of KV cache blocks";
    case KV_ERR_UNSUPPORTED: return "unsupported configuration";
    case KV_ERR_CUDA: return "CUDA error";
    case KV_ERR_DEVICE_CHECK: return "device-side check failed";
    }
    return "unknown status";
}

kv_status kv_pool_create(int num_blocks, int block_size, int kv_heads, int head_dim,
                         kv_dtype dtype, int device, kv_pool** out)
{
    if (out == nullptr) return KV_ERR_INVALID_ARG;
    *out = nullptr;
    if (num_blocks <= 0 || block_size <= 0 || kv_heads <= 0 || head_dim <= 0 || device < 0)
        return KV_ERR_INVALID_ARG;
    if (dtype != KV_DTYPE_BF16 && dtype != KV_DTYPE_FP8_E4M3) return KV_ERR_INVALID_ARG;
    if (!variant_supported(dtype, head_dim, block_size)) return KV_ERR_UNSUPPORTED;
    const size_t elem = dtype == KV_DTYPE_BF16 ? 2 : 1;
    const long double bytes = static_cast<long double>(num_blocks) * block_size * kv_heads *
                              head_dim * elem;
    if (bytes >= static_cast<long double>(1ull << 40)) return KV_ERR_UNSUPPORTED;

    int ndev = 0;
    if (cudaGetDeviceCount(&ndev) != cudaSuccess || device >= ndev) return KV_ERR_CUDA;
    DeviceGuard guard(device);
    if (!guard.ok) return KV_ERR_CUDA;

    kv_pool* p = new (std::nothrow) kv_pool();
    if (p == nullptr) return KV_ERR_OUT_OF_MEMORY;
    p->num_blocks = num_blocks;
    p->block_size = block_size;
    p->kv_heads = kv_heads;
    p->head_dim = head_dim;
    p->device = device;
    p->dtype = dtype;
    p->elem = elem;
    p->pool_bytes = static_cast<size_t>(bytes);
    const size_t half = round_up(p->pool_bytes, kAlign);
    const size_t scales = round_up(sizeof(float) * kv_heads, kAlign);
    const size_t total = 2 * half + 2 * scales + kAlign;
    if (cudaMalloc(&p->base, total) != cudaSuccess) {
        cudaGetLastError();
        delete p;
        return KV_ERR_OUT_OF_MEMORY;
    }
    uint8_t* b = static_cast<uint8_t*>(p->base);
    p->k = b;
    p->v = b + half;
    p->k_scale = reinterpret_cast<float*>(b + 2 * half);
    p->v_scale = reinterpret_cast<float*>(b + 2 * half + scales);
    p->err = reinterpret_cast<uint32_t*>(b + 2 * half + 2 * scales);

    kv_status st = KV_OK;
    if (cudaMemset(p->base, 0, total) != cudaSuccess) st = KV_ERR_CUDA;
    if (st == KV_OK) {
        float* ones = new (std::nothrow) float[kv_heads];
        if (ones == nullptr) {
            st = KV_ERR_OUT_OF_MEMORY;
        } else {
            for (int h = 0; h < kv_heads; ++h) ones[h] = 1.0f;
            if (cudaMemcpy(p->k_scale, ones, sizeof(float) * kv_heads, cudaMemcpyHostToDevice) !=
                    cudaSuccess ||
                cudaMemcpy(p->v_scale, ones, sizeof(float) * kv_heads, cudaMemcpyHostToDevice) !=
                    cudaSuccess)
                st = KV_ERR_CUDA;
            delete[] ones;
        }
    }
    if (st == KV_OK && cudaDeviceGetAttribute(&p->num_sms, cudaDevAttrMultiProcessorCount, device) !=
                           cudaSuccess)
        st = KV_ERR_CUDA;
    if (st == KV_OK) st = encode_pool_map(p, p->k, &p->tmk);
    if (st == KV_OK) st = encode_pool_map(p, p->v, &p->tmv);
    for (int i = 0; i < 3 && kv_heads % (1 << i) == 0; ++i) {
        if (st == KV_OK) st = encode_span_map(p, p->k, 1 << i, &p->tmsk[i]);
        if (st == KV_OK) st = encode_span_map(p, p->v, 1 << i, &p->tmsv[i]);
    }
    if (st == KV_OK) st = encode_octet_map(p, p->k, &p->tmpk);
    if (st == KV_OK) st = encode_octet_map(p, p->v, &p->tmpv);
    if (st == KV_OK) {
        const bool fp8 = dtype == KV_DTYPE_FP8_E4M3;
        for (int nt : {8, 16}) {
            cudaError_t e = fp8 ? kvp::prepare_decode_fp8(head_dim, block_size, nt)
                                : kvp::prepare_decode_bf16(head_dim, block_size, nt);
            if (e == cudaSuccess)
                for (int hc : {1, 2, 4})
                    if (e == cudaSuccess)
                        e = fp8 ? kvp::prepare_span_fp8(head_dim, nt, hc) : kvp::prepare_span_bf16(head_dim, nt, hc);
            if (e != cudaSuccess) st = KV_ERR_CUDA;
        }
        if (kvp::prepare_decode_heads(fp8, head_dim, block_size) != cudaSuccess) st = KV_ERR_CUDA;
        if (kvp::prepare_norm_rope_append(head_dim, fp8) != cudaSuccess) st = KV_ERR_CUDA;
        if (kvp::prepare_prefix(fp8, head_dim, block_size) != cudaSuccess) st = KV_ERR_CUDA;
    }
    if (st == KV_OK && cudaDeviceSynchronize() != cudaSuccess) st = KV_ERR_CUDA;
    if (st != KV_OK) {
        cudaGetLastError();
        cudaFree(p->base);
        delete p;
        return st;
    }
    *out = p;
    return KV_OK;
}

kv_status kv_pool_destroy(kv_pool* pool)
{
    if (pool == nullptr) return KV_OK;
    kv_status st = KV_OK;
    {
        DeviceGuard guard(pool->device);
        if (!guard.ok || cudaDeviceSynchronize() != cudaSuccess) st = KV_ERR_CUDA;
        if (cudaFree(pool->base) != cudaSuccess) st = KV_ERR_CUDA;
    }
    delete pool;
    return st;
}

kv_status kv_pool_tensors(const kv_pool* pool, void** k_pool, void** v_pool, float** k_scale,
                          float** v_scale)
{
    if (pool == nullptr) return KV_ERR_INVALID_ARG;
    if (k_pool) *k_pool = pool->k;
    if (v_pool) *v_pool = pool->v;
    if (k_scale) *k_scale = pool->k_scale;
    if (v_scale) *v_scale = pool->v_scale;
    return KV_OK;
}

kv_status kv_pool_shape(const kv_pool* pool, int* num_blocks, int* block_size, int* kv_heads,
                        int* head_dim, kv_dtype* dtype, int* device)
{
    if (pool == nullptr) return KV_ERR_INVALID_ARG;
    if (num_blocks) *num_blocks = pool->num_blocks;
    if (block_size) *block_size = pool->block_size;
    if (kv_heads) *kv_heads = pool->kv_heads;
    if (head_dim) *head_dim = pool->head_dim;
    if (dtype) *dtype = pool->dtype;
    if (device) *device = pool->device;
    return KV_OK;
}

kv_status kv_pool_set_scales(kv_pool* pool, const float* k_scale_host, const float* v_scale_host)
{
    if (pool == nullptr) return KV_ERR_INVALID_ARG;
    for (const float* s : {k_scale_host, v_scale_host}) {
        if (s == nullptr) continue;
        for (int h = 0; h < pool->kv_heads; ++h)
            if (!(std::isfinite(s[h]) && s[h] > 0.f)) return KV_ERR_INVALID_ARG;
    }
    DeviceGuard guard(pool->device);
    if (!guard.ok) return KV_ERR_CUDA;
    const size_t n = sizeof(float) * pool->kv_heads;
    if (k_scale_host && cudaMemcpy(pool->k_scale, k_scale_host, n, cudaMemcpyHostToDevice) != cudaSuccess)
        return KV_ERR_CUDA;
    if (v_scale_host && cudaMemcpy(pool->v_scale, v_scale_host, n, cudaMemcpyHostToDevice) != cudaSuccess)
        return KV_ERR_CUDA;
    return KV_OK;
}

kv_status kv_pool_device_errors(kv_pool* pool, uint32_t* bits, int clear)
{
    if (pool == nullptr || bits == nullptr) return KV_ERR_INVALID_ARG;
    DeviceGuard guard(pool->device);
    if (!guard.ok || cudaDeviceSynchronize() != cudaSuccess) return KV_ERR_CUDA;
    if (cudaMemcpy(bits, pool->err, sizeof(uint32_t), cudaMemcpyDeviceToHost) != cudaSuccess)
        return KV_ERR_CUDA;
    if (clear && cudaMemset(pool->err, 0, sizeof(uint32_t)) != cudaSuccess) return KV_ERR_CUDA;
    return *bits ? KV_ERR_DEVICE_CHECK : KV_OK;
}

kv_status paged_kv_append(kv_pool* pool, const void* k_new, const void* v_new, int num_tokens,
                          const int32_t* token_seq, const int32_t* token_pos,
                          const int32_t* block_tables, int max_blocks,
                          const int32_t* context_lens, int batch, void* stream)
{
    if (pool == nullptr || num_tokens < 0 || batch < 0 || max_blocks <= 0)
        return KV_ERR_INVALID_ARG;
    if (num_tokens == 0) return KV_OK;
    if (k_new == nullptr || block_tables == nullptr || batch == 0) return KV_ERR_INVALID_ARG;
    if ((v_new == nullptr) != (pool->mla != 0)) return KV_ERR_INVALID_ARG;   // latent pools: no V
    if (token_pos == nullptr && context_lens == nullptr) return KV_ERR_INVALID_ARG;
    if (token_seq == nullptr && num_tokens > batch) return KV_ERR_INVALID_ARG;
    if (!aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(block_tables, 4) ||
        !aligned(token_seq, 4) || !aligned(token_pos, 4) || !aligned(context_lens, 4))
        return KV_ERR_INVALID_ARG;
    kv_status st = check_device(pool);
    if (st != KV_OK) return st;
    kvp::AppendParams p;
    p.k_new = static_cast<const uint16_t*>(k_new);
    p.v_new = static_cast<const uint16_t*>(v_new);
    p.token_seq = token_seq;
    p.token_pos = token_pos;
    p.tables = block_tables;
    p.ctx = context_lens;
    p.k_pool = pool->k;
    p.v_pool = pool->v;
    p.k_scale = pool->k_scale;
    p.v_scale = pool->v_scale;
    p.err = pool->err;
    p.num_tokens = num_tokens;
    p.batch = batch;
    p.max_blocks = max_blocks;
    p.num_blocks = pool->num_blocks;
    p.block_size = pool->block_size;
    p.kv_heads = pool->kv_heads;
    p.head_dim = pool->head_dim;
    p.fp8 = pool->dtype == KV_DTYPE_FP8_E4M3;
    p.q_len = 1;
    return kvp::launch_append(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? KV_OK
                                                                                   : KV_ERR_CUDA;
}

kv_status paged_norm_rope_append(kv_pool* pool, const void* q, int64_t q_stride, const void* k,
                                 int64_t k_stride, const void* v, int64_t v_stride, int q_heads,
                                 int num_tokens, const float* q_weight, const float* k_weight,
                                 float eps, const float* rope, int rope_positions, int rope_dim,
                                 kv_rope_style style, const int32_t* token_seq,
                                 const int32_t* token_pos, const int32_t* block_tables,
                                 int max_blocks, const int32_t* context_lens, int batch, int q_len,
                                 void* q_out, void* stream)
{
    if (pool == nullptr || pool->mla || num_tokens < 0 || batch < 0 || max_blocks <= 0 || q_heads <= 0 ||
        q_len <= 0)
        return KV_ERR_INVALID_ARG;
    if (static_cast<long long>(max_blocks) * pool->block_size > std::numeric_limits<int>::max())
        return KV_ERR_INVALID_ARG;                  // positions are 32-bit
    if (num_tokens == 0) return KV_OK;
    if (q == nullptr || k == nullptr || v == nullptr || q_out == nullptr || block_tables == nullptr || batch == 0)
        return KV_ERR_INVALID_ARG;
    if ((token_seq != nullptr || token_pos != nullptr) && q_len != 1) return KV_ERR_INVALID_ARG;
    if (token_pos == nullptr && context_lens == nullptr) return KV_ERR_INVALID_ARG;
    if (token_seq == nullptr && num_tokens > static_cast<long long>(batch) * q_len) return KV_ERR_INVALID_ARG;
    if (num_tokens % q_len != 0) return KV_ERR_INVALID_ARG;      // q_out holds whole sequences' tokens
    if ((q_weight == nullptr) != (k_weight == nullptr)) return KV_ERR_INVALID_ARG;
    if (q_weight != nullptr && !(std::isfinite(eps) && eps >= 0.f)) return KV_ERR_INVALID_ARG;
    if (rope != nullptr && (rope_positions <= 0 || rope_dim <= 0 || rope_dim % 16 != 0 || rope_dim > pool->head_dim))
        return KV_ERR_INVALID_ARG;
    if (style != KV_ROPE_HALF && style != KV_ROPE_INTERLEAVED) return KV_ERR_INVALID_ARG;
    const int64_t d = pool->head_dim;
    if (q_stride % 8 != 0 || k_stride % 8 != 0 || v_stride % 8 != 0 || q_stride < q_heads * d ||
        k_stride < pool->kv_heads * d || v_stride < pool->kv_heads * d)
        return KV_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(q_out, 16) || !aligned(q_weight, 16) ||
        !aligned(k_weight, 16) || !aligned(rope, 16) || !aligned(block_tables, 4) || !aligned(token_seq, 4) ||
        !aligned(token_pos, 4) || !aligned(context_lens, 4))
        return KV_ERR_INVALID_ARG;
    // one lane group per row at most, in 32 bits with room for the last CTA's groups
    if (static_cast<long long>(num_tokens) * (static_cast<long long>(q_heads) + 2 * pool->kv_heads) >
        std::numeric_limits<int>::max() - 64)
        return KV_ERR_UNSUPPORTED;
    kv_status st = check_device(pool);
    if (st != KV_OK) return st;
    kvp::NormRopeParams p;
    p.q = static_cast<const uint16_t*>(q);
    p.k = static_cast<const uint16_t*>(k);
    p.v = static_cast<const uint16_t*>(v);
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.q_weight = q_weight;
    p.k_weight = k_weight;
    p.rope = rope;
    p.rope_positions = rope_positions;
    p.rope_dim = rope != nullptr ? rope_dim : 0;
    p.interleaved = style == KV_ROPE_INTERLEAVED;
    p.eps = eps;
    p.token_seq = token_seq;
    p.token_pos = token_pos;
    p.tables = block_tables;
    p.ctx = context_lens;
    p.k_pool = pool->k;
    p.v_pool = pool->v;
    p.k_scale = pool->k_scale;
    p.v_scale = pool->v_scale;
    p.q_out = static_cast<uint16_t*>(q_out);
    p.err = pool->err;
    p.num_tokens = num_tokens;
    p.batch = batch;
    p.q_heads = q_heads;
    p.kv_heads = pool->kv_heads;
    p.max_blocks = max_blocks;
    p.num_blocks = pool->num_blocks;
    p.block_size = pool->block_size;
    p.q_len = q_len;
    p.chunks = 0;
    p.stop_stage = g_stop_stage.load(std::memory_order_relaxed);
    p.consumer_wait_ns = g_consumer_wait_ns.load(std::memory_order_relaxed);
    return kvp::launch_norm_rope_append(p, pool->head_dim, pool->dtype == KV_DTYPE_FP8_E4M3, pool->num_sms,
                                        static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? KV_OK
               : KV_ERR_CUDA;
}

kv_status kv_copy_blocks(kv_pool* pool, const kv_block_copy* copies, int n, void* stream)
{
    if (pool == nullptr || n < 0) return KV_ERR_INVALID_ARG;
    if (n == 0) return KV_OK;
    if (copies == nullptr || !aligned(copies, 4)) return KV_ERR_INVALID_ARG;
    if (n > (1 << 30)) return KV_ERR_UNSUPPORTED;
    kv_status st = check_device(pool);
    if (st != KV_OK) return st;
    const size_t block_bytes = static_cast<size_t>(pool->block_size) * pool->kv_heads *
                               pool->head_dim * pool->elem;
    return kvp::launch_copy_blocks(copies, n, pool->k, pool->v, block_bytes, pool->num_blocks,
                                   pool->err, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? KV_OK
               : KV_ERR_CUDA;
}

kv_status paged_decode_plan(const kv_pool* pool, int batch, int q_heads, int max_blocks,
                            int kv_split_tokens, int* split_tokens, int* max_splits)
{
    Plan p;
    kv_status st = make_plan(pool, batch, q_heads, 1, max_blocks, kv_split_tokens, &p);
    if (st != KV_OK) return st;
    if (split_tokens) *split_tokens = p.split_blocks * pool->block_size;
    if (max_splits) *max_splits = p.max_splits;
    return KV_OK;
}

kv_status kv_debug_decode_stall(int stop_stage, unsigned long long consumer_wait_ns)
{
    if (stop_stage < -1) return KV_ERR_INVALID_ARG;
    g_stop_stage.store(stop_stage, std::memory_order_relaxed);
    g_consumer_wait_ns.store(consumer_wait_ns, std::memory_order_relaxed);
    return KV_OK;
}

kv_status paged_decode_cta_heads(const kv_pool* pool, int batch, int q_heads, int q_len,
                                 int max_blocks, int kv_split_tokens, int* cta_heads)
{
    if (cta_heads == nullptr) return KV_ERR_INVALID_ARG;
    Plan p;
    kv_status st = make_plan(pool, batch, q_heads, q_len, max_blocks, kv_split_tokens, &p);
    if (st != KV_OK) return st;
    *cta_heads = p.cta_heads;
    return KV_OK;
}

kv_status paged_multi_query_workspace_size(const kv_pool* pool, int batch, int q_heads,
                                           int q_len, int max_blocks, int kv_split_tokens,
                                           size_t* bytes)
{
    if (bytes == nullptr) return KV_ERR_INVALID_ARG;
    Plan p;
    kv_status st = make_plan(pool, batch, q_heads, q_len, max_blocks, kv_split_tokens, &p);
    if (st != KV_OK) return st;
    *bytes = workspace_bytes_for(pool, batch, p);
    return KV_OK;
}

kv_status paged_decode_workspace_size(const kv_pool* pool, int batch, int q_heads,
                                      int max_blocks, int kv_split_tokens, size_t* bytes)
{
    return paged_multi_query_workspace_size(pool, batch, q_heads, 1, max_blocks, kv_split_tokens,
                                            bytes);
}

}  // extern "C"

namespace {

// Validates a decode call and fills its kernel parameters and grid (nothing launched).
kv_status make_decode_launch(const kv_pool* pool, const void* q, int q_heads, int q_len,
                             const int32_t* block_tables, int max_blocks,
                             const int32_t* context_lens, int batch, float scale,
                             int kv_split_tokens, void* workspace, size_t workspace_bytes,
                             void* out, float* lse_out, Plan* plan_out, kvp::DecodeParams* pp,
                             dim3* grid)
{
    Plan plan;
    kv_status st = make_plan(pool, batch, q_heads, q_len, max_blocks, kv_split_tokens, &plan);
    if (st != KV_OK) return st;
    if (pool->mla) return KV_ERR_INVALID_ARG;        // latent pools: paged_mla_decode_attention
    if (batch == 0) return KV_OK;
    if (q == nullptr || block_tables == nullptr || context_lens == nullptr || out == nullptr)
        return KV_ERR_INVALID_ARG;
    if (!std::isfinite(scale)) return KV_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(block_tables, 4) ||
        !aligned(context_lens, 4) || !aligned(lse_out, 4) || !aligned(workspace, 16))
        return KV_ERR_INVALID_ARG;
    if (batch > 65535 || static_cast<long long>(pool->kv_heads) * plan.head_groups > 65535)
        return KV_ERR_UNSUPPORTED;                  // grid x / y limits
    const size_t need = workspace_bytes_for(pool, batch, plan);
    if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return KV_ERR_INVALID_ARG;
    st = check_device(pool);
    if (st != KV_OK) return st;

    const WorkspaceLayout wl = workspace_layout(pool, batch, plan);
    kvp::DecodeParams& p = *pp;
    p.q = static_cast<const uint16_t*>(q);
    p.tables = block_tables;
    p.ctx = context_lens;
    p.k_scale = pool->k_scale;
    p.v_scale = pool->v_scale;
    p.out = static_cast<uint16_t*>(out);
    p.lse = lse_out;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    p.part_o = need > 0 ? reinterpret_cast<float*>(ws + wl.part_o) : nullptr;
    p.part_ml = need > 0 ? reinterpret_cast<float*>(ws + wl.part_ml) : nullptr;
    p.tickets = need > 0 ? reinterpret_cast<int*>(ws + wl.tickets) : nullptr;
    p.err = pool->err;
    p.batch = batch;
    p.q_heads = q_heads;
    p.kv_heads = pool->kv_heads;
    p.group = plan.group;
    p.head_groups = plan.head_groups;
    p.q_len = q_len;
    p.rows = plan.rows;
    p.max_blocks = max_blocks;
    p.num_blocks = pool->num_blocks;
    p.split_blocks = plan.split_blocks;
    p.max_splits = plan.max_splits;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.k_new = nullptr;
    p.v_new = nullptr;
    p.k_pool = nullptr;
    p.v_pool = nullptr;
    p.merge_kernel = 0;
    p.stop_stage = g_stop_stage.load(std::memory_order_relaxed);
    p.consumer_wait_ns = g_consumer_wait_ns.load(std::memory_order_relaxed);
    // chunk-major grid: x = (kv head group, row tile), y = sequence, z = chunk
    *grid = dim3(static_cast<unsigned>(pool->kv_heads / plan.cta_heads * plan.head_groups),
                 static_cast<unsigned>(batch), static_cast<unsigned>(plan.max_splits));
    *plan_out = plan;
    return KV_OK;
}

kv_status launch_decode(const kv_pool* pool, const Plan& plan, dim3 grid, const kvp::DecodeParams& p,
                        void* stream)
{
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (plan.cta_heads > 1) {
        return kvp::launch_decode_heads(pool->dtype == KV_DTYPE_FP8_E4M3, pool->head_dim,
                                        pool->block_size, plan.head_tile, plan.cta_heads,
                                        plan.cta_per_sm, grid, pool->tmk, pool->tmv, p, s) == cudaSuccess
                   ? KV_OK
                   : KV_ERR_CUDA;
    }
    cudaError_t e = pool->dtype == KV_DTYPE_BF16
                        ? kvp::launch_decode_bf16(pool->head_dim, pool->block_size, plan.head_tile,
                                                  grid, pool->tmk, pool->tmv, p, s)
                        : kvp::launch_decode_fp8(pool->head_dim, pool->block_size, plan.head_tile,
                                                 grid, pool->tmk, pool->tmv, p, s);
    return e == cudaSuccess ? KV_OK : KV_ERR_CUDA;
}

constexpr float kLog2e = 1.4426950408889634f;

// Validates a call of the span kernel and fills its decode parameters (nothing launched).
// extra: workspace bytes the call needs behind the kernel's own.
kv_status make_span_launch(const kv_pool* pool, const SpanPlan& plan, const void* q, int q_heads, int q_len,
                           const int32_t* block_tables, int max_blocks, const int32_t* context_lens, int batch,
                           float scale, void* workspace, size_t workspace_bytes, size_t extra, void* out,
                           float* lse_out, kvp::SpanParams* sp)
{
    if (!std::isfinite(scale * kLog2e)) return KV_ERR_INVALID_ARG;      // scores are kept in log2 units
    if (batch == 0) return KV_OK;
    if (q == nullptr || block_tables == nullptr || context_lens == nullptr || out == nullptr || workspace == nullptr)
        return KV_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(block_tables, 4) || !aligned(context_lens, 4) ||
        !aligned(lse_out, 4) || !aligned(workspace, 16))
        return KV_ERR_INVALID_ARG;
    const SpanLayout wl = span_layout(pool, plan);
    if (workspace_bytes < wl.total + extra) return KV_ERR_INVALID_ARG;
    kv_status st = check_device(pool);
    if (st != KV_OK) return st;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    kvp::DecodeParams& p = sp->d;
    p = {};
    p.q = static_cast<const uint16_t*>(q);
    p.tables = block_tables;
    p.ctx = context_lens;
    p.k_scale = pool->k_scale;
    p.v_scale = pool->v_scale;
    p.out = static_cast<uint16_t*>(out);
    p.lse = lse_out;
    p.tickets = reinterpret_cast<int*>(ws);
    p.part_ml = reinterpret_cast<float*>(ws + wl.part_ml);
    p.part_o = reinterpret_cast<float*>(ws + wl.part_o);
    p.err = pool->err;
    p.batch = batch;
    p.q_heads = q_heads;
    p.kv_heads = pool->kv_heads;
    p.group = q_heads / pool->kv_heads;
    p.head_groups = plan.head_groups;
    p.q_len = q_len;
    p.rows = plan.rows;
    p.max_blocks = max_blocks;
    p.num_blocks = pool->num_blocks;
    p.scale_log2 = scale * kLog2e;
    p.stop_stage = g_stop_stage.load(std::memory_order_relaxed);
    p.consumer_wait_ns = g_consumer_wait_ns.load(std::memory_order_relaxed);
    sp->block_size = pool->block_size;
    sp->least = plan.least;
    return KV_OK;
}

kv_status launch_span(const kv_pool* pool, const SpanPlan& plan, kvp::SpanRule rule, const kvp::SpanParams& p,
                      void* stream)
{
    const auto launch = pool->dtype == KV_DTYPE_BF16 ? kvp::launch_span_bf16 : kvp::launch_span_fp8;
    const int map = plan.heads / 2;                  // 1, 2, 4 heads
    return launch(rule, pool->head_dim, plan.head_tile, plan.heads, plan.ctas, pool->tmsk[map], pool->tmsv[map], p,
                  static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? KV_OK
               : KV_ERR_CUDA;
}

}  // namespace

extern "C" {

kv_status paged_attention_multi_query(const kv_pool* pool, const void* q, int q_heads, int q_len,
                                      const int32_t* block_tables, int max_blocks,
                                      const int32_t* context_lens, int batch, float scale,
                                      int kv_split_tokens, void* workspace,
                                      size_t workspace_bytes, void* out, float* lse_out,
                                      void* stream)
{
    Plan plan;
    kvp::DecodeParams p;
    dim3 grid;
    const kv_status st = make_decode_launch(pool, q, q_heads, q_len, block_tables, max_blocks,
                                            context_lens, batch, scale, kv_split_tokens, workspace,
                                            workspace_bytes, out, lse_out, &plan, &p, &grid);
    if (st != KV_OK || batch == 0) return st;
    return launch_decode(pool, plan, grid, p, stream);
}

kv_status paged_attention_masked_workspace_size(const kv_pool* pool, int batch, int q_heads,
                                                int q_len, int max_blocks, int window,
                                                int kv_split_tokens, size_t* bytes)
{
    if (bytes == nullptr) return KV_ERR_INVALID_ARG;
    SpanPlan p;
    kv_status st = make_masked_plan(pool, batch, q_heads, q_len, max_blocks, window, kv_split_tokens, &p);
    if (st == KV_OK) *bytes = span_layout(pool, p).total;
    return st;
}

kv_status paged_attention_masked(const kv_pool* pool, const void* q, int q_heads, int q_len,
                                 const int32_t* block_tables, int max_blocks,
                                 const int32_t* context_lens, int batch, float scale,
                                 const kv_attention_mask* mask, int kv_split_tokens,
                                 void* workspace, size_t workspace_bytes, void* out,
                                 float* lse_out, void* stream)
{
    kv_attention_mask m = {};
    if (mask != nullptr) m = *mask;
    if (!(m.softcap >= 0.f) || !std::isfinite(m.softcap * kLog2e) || (m.softcap > 0.f && !std::isfinite(2.f / m.softcap)))
        return KV_ERR_INVALID_ARG;
    if (!aligned(m.alibi_slopes, 4) || !aligned(m.first_keys, 4) || !aligned(m.prefix_lens, 4))
        return KV_ERR_INVALID_ARG;
    SpanPlan plan;
    kv_status st = make_masked_plan(pool, batch, q_heads, q_len, max_blocks, m.window, kv_split_tokens, &plan);
    if (st != KV_OK) return st;
    kvp::SpanParams p = {};
    st = make_span_launch(pool, plan, q, q_heads, q_len, block_tables, max_blocks, context_lens, batch, scale,
                          workspace, workspace_bytes, 0, out, lse_out, &p);
    if (st != KV_OK || batch == 0) return st;
    p.window = effective_window(pool, m.window, max_blocks);
    p.cap_log2 = m.softcap * kLog2e;
    p.cap_in = m.softcap > 0.f ? 2.f / m.softcap : 0.f;
    p.slopes = m.alibi_slopes;
    p.first_keys = m.first_keys;
    p.prefix_lens = m.prefix_lens;
    const int rule = (m.softcap > 0.f ? kvp::SPAN_CAP : 0) | (m.alibi_slopes != nullptr ? kvp::SPAN_BIAS : 0);
    return launch_span(pool, plan, static_cast<kvp::SpanRule>(rule), p, stream);
}

kv_status paged_shared_prefix_workspace_size(const kv_pool* pool, int batch, int q_heads, int q_len,
                                             int max_blocks, int n_groups, int kv_split_tokens,
                                             size_t* bytes)
{
    if (bytes == nullptr || n_groups < 0) return KV_ERR_INVALID_ARG;
    SpanPlan p;
    kv_status st = make_span_plan(pool, batch, q_heads, q_len, max_blocks, max_blocks, kv_split_tokens, &p);
    if (st != KV_OK) return st;
    const PrefixLayout l = prefix_layout(pool, batch, p, n_groups);
    if (l.pieces > (1 << 30)) return KV_ERR_UNSUPPORTED;
    *bytes = span_layout(pool, p).total + l.total;
    return KV_OK;
}

kv_status paged_shared_prefix_attention(const kv_pool* pool, const void* q, int q_heads, int q_len,
                                        const int32_t* block_tables, int max_blocks,
                                        const int32_t* context_lens, int batch,
                                        const int32_t* group_offsets, const int32_t* group_blocks,
                                        int n_groups, float scale, int kv_split_tokens,
                                        void* workspace, size_t workspace_bytes, void* out,
                                        float* lse_out, void* stream)
{
    if (n_groups < 0 || (n_groups > 0 && (group_offsets == nullptr || group_blocks == nullptr)) ||
        !aligned(group_offsets, 4) || !aligned(group_blocks, 4))
        return KV_ERR_INVALID_ARG;
    SpanPlan plan;
    kv_status st = make_span_plan(pool, batch, q_heads, q_len, max_blocks, max_blocks, kv_split_tokens, &plan);
    if (st != KV_OK) return st;
    const PrefixLayout l = prefix_layout(pool, batch, plan, n_groups);
    if (l.pieces > (1 << 30)) return KV_ERR_UNSUPPORTED;
    kvp::SpanParams p = {};
    st = make_span_launch(pool, plan, q, q_heads, q_len, block_tables, max_blocks, context_lens, batch, scale,
                          workspace, workspace_bytes, l.total, out, lse_out, &p);
    if (st != KV_OK || batch == 0) return st;
    if (l.total == 0) return launch_span(pool, plan, kvp::SPAN_MASK, p, stream);   // nobody to share with
    kvp::PrefixParams& s = p.shared;
    uint8_t* ws = static_cast<uint8_t*>(workspace) + span_layout(pool, plan).total;
    s.q = p.d.q;
    s.tables = block_tables;
    s.ctx = context_lens;
    s.group_offsets = group_offsets;
    s.group_blocks = group_blocks;
    s.k_scale = pool->k_scale;
    s.runs = reinterpret_cast<int2*>(ws + l.runs);
    s.piece_lse = reinterpret_cast<float4*>(ws + l.piece_lse);
    s.piece_o = reinterpret_cast<float*>(ws + l.piece_o);
    s.err = pool->err;
    s.batch = batch;
    s.kv_heads = pool->kv_heads;
    s.q_len = q_len;
    s.rows = plan.rows;
    s.max_blocks = max_blocks;
    s.num_blocks = pool->num_blocks;
    s.n_groups = n_groups;
    s.share_least = (kShareTokens + pool->block_size - 1) / pool->block_size;
    s.pieces = static_cast<int>(l.pieces);
    s.scale_log2 = p.d.scale_log2;
    s.stop_stage = p.d.stop_stage;
    if (kvp::launch_prefix(pool->dtype == KV_DTYPE_FP8_E4M3, pool->head_dim, pool->block_size, pool->num_sms, pool->tmpk,
                           pool->tmpv, s, static_cast<cudaStream_t>(stream)) != cudaSuccess)
        return KV_ERR_CUDA;
    return launch_span(pool, plan, kvp::SPAN_SUFFIX, p, stream);
}

kv_status paged_decode_step(kv_pool* pool, const void* k_new, const void* v_new, const void* q,
                            int q_heads, int q_len, const int32_t* block_tables, int max_blocks,
                            const int32_t* context_lens, int batch, float scale,
                            int kv_split_tokens, void* workspace, size_t workspace_bytes,
                            void* out, float* lse_out, void* stream)
{
    if (pool == nullptr || q_len < 1) return KV_ERR_INVALID_ARG;
    // everything is checked before anything is launched
    Plan plan;
    kvp::DecodeParams p;
    dim3 grid;
    kv_status st = make_decode_launch(pool, q, q_heads, q_len, block_tables, max_blocks,
                                      context_lens, batch, scale, kv_split_tokens, workspace,
                                      workspace_bytes, out, lse_out, &plan, &p, &grid);
    if (st != KV_OK || batch == 0) return st;
    if (k_new == nullptr || v_new == nullptr || !aligned(k_new, 16) || !aligned(v_new, 16))
        return KV_ERR_INVALID_ARG;
    if (static_cast<long long>(batch) * q_len > std::numeric_limits<int>::max())
        return KV_ERR_UNSUPPORTED;
    if (plan.head_tile == 8) {
        // One kernel: the CTA that reads a block holding one of the step's new tokens writes
        // that token's rows of its kv heads into the pool first (the append's arithmetic, the
        // same bytes), so no append kernel has to finish before the attention starts.
        p.k_new = static_cast<const uint16_t*>(k_new);
        p.v_new = static_cast<const uint16_t*>(v_new);
        p.k_pool = pool->k;
        p.v_pool = pool->v;
        return launch_decode(pool, plan, grid, p, stream);
    }
    // 16-row tiles: the append kernel, then the attention (the kernel's step form is not
    // built for them)
    kvp::AppendParams a;
    a.k_new = static_cast<const uint16_t*>(k_new);
    a.v_new = static_cast<const uint16_t*>(v_new);
    a.token_seq = nullptr;
    a.token_pos = nullptr;
    a.tables = block_tables;
    a.ctx = context_lens;
    a.k_pool = pool->k;
    a.v_pool = pool->v;
    a.k_scale = pool->k_scale;
    a.v_scale = pool->v_scale;
    a.err = pool->err;
    a.num_tokens = batch * q_len;
    a.batch = batch;
    a.max_blocks = max_blocks;
    a.num_blocks = pool->num_blocks;
    a.block_size = pool->block_size;
    a.kv_heads = pool->kv_heads;
    a.head_dim = pool->head_dim;
    a.fp8 = pool->dtype == KV_DTYPE_FP8_E4M3;
    a.q_len = q_len;
    if (kvp::launch_append(a, static_cast<cudaStream_t>(stream)) != cudaSuccess) return KV_ERR_CUDA;
    return launch_decode(pool, plan, grid, p, stream);
}

kv_status paged_decode_attention(const kv_pool* pool, const void* q, int q_heads,
                                 const int32_t* block_tables, int max_blocks,
                                 const int32_t* context_lens, int batch, float scale,
                                 int kv_split_tokens, void* workspace, size_t workspace_bytes,
                                 void* out, float* lse_out, void* stream)
{
    return paged_attention_multi_query(pool, q, q_heads, 1, block_tables, max_blocks,
                                       context_lens, batch, scale, kv_split_tokens, workspace,
                                       workspace_bytes, out, lse_out, stream);
}

kv_status paged_merge_attention_states(const void* outs, const float* lses, int n_src, long long rows,
                                       int head_dim, void* out, float* lse_out, void* stream)
{
    if (n_src < 1 || rows < 0 || head_dim < 8 || head_dim > 1024 || head_dim % 8 != 0)
        return KV_ERR_INVALID_ARG;
    if (rows == 0) return KV_OK;
    if (outs == nullptr || lses == nullptr || out == nullptr) return KV_ERR_INVALID_ARG;
    if (!aligned(outs, 16) || !aligned(out, 16) || !aligned(lses, 4) || !aligned(lse_out, 4))
        return KV_ERR_INVALID_ARG;
    return kvp::launch_merge_attention_states(
               static_cast<const uint16_t*>(outs), lses, n_src, rows, head_dim,
               static_cast<uint16_t*>(out), lse_out, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? KV_OK
               : KV_ERR_CUDA;
}

kv_status paged_decode_attention_split_merge(const kv_pool* pool, const void* q, int q_heads,
                                             const int32_t* block_tables, int max_blocks,
                                             const int32_t* context_lens, int batch, float scale,
                                             int kv_split_tokens, void* workspace,
                                             size_t workspace_bytes, void* out, float* lse_out,
                                             void* stream)
{
    Plan plan;
    kvp::DecodeParams p;
    dim3 grid;
    const kv_status st = make_decode_launch(pool, q, q_heads, 1, block_tables, max_blocks,
                                            context_lens, batch, scale, kv_split_tokens, workspace,
                                            workspace_bytes, out, lse_out, &plan, &p, &grid);
    if (st != KV_OK || batch == 0) return st;
    p.merge_kernel = plan.max_splits > 1;
    kv_status r = launch_decode(pool, plan, grid, p, stream);
    if (r != KV_OK || !p.merge_kernel) return r;
    return kvp::launch_decode_merge(p, pool->head_dim, pool->block_size,
                                    static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? KV_OK
               : KV_ERR_CUDA;
}

}  // extern "C"

// ---------------------------------------------------------------------------
// Multi-head latent attention (absorbed form) over a latent pool.
// ---------------------------------------------------------------------------
namespace {

constexpr int kMlaHeadTile = 16;

// The three forms of the latent decode.
enum MlaForm {
    kMlaMma = 0,            // mma.sync, head tiles of 16, a CTA per (tile, sequence, chunk)
    kMlaWide = 1,           // tcgen05, head tiles of 128, two latent halves each
    kMlaNarrow = 2,         // tcgen05, head tiles of 16
};

struct MlaPlan {
    int head_tiles, split_blocks, max_splits;
    int form;               // MlaForm
};

// Blocks of 64 tokens take a tcgen05 form: the wide one for at least 64 heads (tiles of
// 128 rows), the narrow one below that.
int mla_form(const kv_pool* pl, int q_heads)
{
    if (!pl->has_tc) return kMlaMma;
    return q_heads >= 64 ? kMlaWide : kMlaNarrow;
}

// Automatic chunk: about eight chunks per SM over the worst case, kept between
// 768 and 2048 tokens.  Measured on GB300 (DeepSeek-shaped layer, contexts
// uniform in [512, 4096]): 16 heads are fastest with 768-token chunks (about
// 2.5 CTAs per SM), 128 heads with ~1700 (chunks of 512 pay too many merges).
kv_status make_mla_plan(const kv_pool* pl, int batch, int q_heads, int max_blocks,
                        int split_tokens, MlaPlan* out)
{
    if (pl == nullptr || !pl->mla || batch < 0 || q_heads <= 0 || max_blocks <= 0 ||
        split_tokens < 0)
        return KV_ERR_INVALID_ARG;
    if (split_tokens % pl->block_size != 0) return KV_ERR_INVALID_ARG;
    if (static_cast<long long>(max_blocks) * pl->block_size > std::numeric_limits<int>::max())
        return KV_ERR_INVALID_ARG;
    MlaPlan p;
    p.form = mla_form(pl, q_heads);
    const int tile = p.form == kMlaWide ? kvp::MLA_TC_HEADS : kMlaHeadTile;
    p.head_tiles = (q_heads + tile - 1) / tile;
    if (p.form != kMlaMma) {
        // the units ((latent half,) head tile, sequence, block) are cut into one contiguous
        // range per CTA; split_blocks is the least a range holds (the chunk argument, or
        // automatically about half the worst-case share of an SM, 4..16 blocks), so a
        // sequence of max_blocks blocks is cut into at most ceil((max_blocks - 1) /
        // split_blocks) + 1 pieces, each merged from its own partial
        const int outer = p.head_tiles * (p.form == kMlaWide ? 2 : 1);
        if (split_tokens > 0) {
            p.split_blocks = split_tokens / pl->block_size;
        } else {
            const long long units = static_cast<long long>(batch > 0 ? batch : 1) * outer * max_blocks;
            const long long share = units / (2LL * (pl->num_sms > 0 ? pl->num_sms : 148));
            p.split_blocks = static_cast<int>(share < 4 ? 4 : (share > 16 ? 16 : share));
        }
        if (p.split_blocks > max_blocks) p.split_blocks = max_blocks;
        p.max_splits = (max_blocks - 1 + p.split_blocks - 1) / p.split_blocks + 1;
        if (p.max_splits > max_blocks) p.max_splits = max_blocks;
        // the partition's arithmetic: units x CTAs must stay far inside 64 bits
        const long long units_max = static_cast<long long>(batch) * outer * max_blocks;
        if (units_max > (1LL << 40)) return KV_ERR_UNSUPPORTED;
        if (p.max_splits > 65535 || p.head_tiles > 32767 || batch > 65535) return KV_ERR_UNSUPPORTED;
        *out = p;
        return KV_OK;
    }
    if (split_tokens > 0) {
        p.split_blocks = split_tokens / pl->block_size;
    } else {
        const long long units = static_cast<long long>(batch > 0 ? batch : 1) * p.head_tiles;
        const long long work = units * max_blocks * pl->block_size;
        const long long target = static_cast<long long>(pl->num_sms > 0 ? pl->num_sms : 148) * 8;
        long long tok = (work + target - 1) / target;
        if (tok < 768) tok = 768;
        if (tok > 2048) tok = 2048;
        p.split_blocks = static_cast<int>((tok + pl->block_size - 1) / pl->block_size);
    }
    if (p.split_blocks > max_blocks) p.split_blocks = max_blocks;
    p.max_splits = (max_blocks + p.split_blocks - 1) / p.split_blocks;
    if (p.max_splits > 65535 || p.head_tiles > 65535 || batch > 65535) return KV_ERR_UNSUPPORTED;
    *out = p;
    return KV_OK;
}

// partial outputs [batch, q_heads, max_splits, 512], (max, sum) pairs, then one ticket
// per (sequence, head tile); the tensor-core form lays its pieces out per (sequence,
// head tile, latent half, split) instead.
WorkspaceLayout mla_workspace_layout(int batch, int q_heads, const MlaPlan& p)
{
    WorkspaceLayout w{0, 0, 0, 0, 0};
    if (p.max_splits > 1 && p.form == kMlaNarrow) {
        // pieces (sequence, head tile, split): fp16 partials of 16 heads x 512 latent
        // numbers, fp32 (max, sum) per head, then the piece count of each (sequence, head tile)
        const size_t pieces = static_cast<size_t>(batch) * p.head_tiles * p.max_splits;
        w.part_ml = round_up(pieces * kvp::MLA_TCN_HEADS * kvp::MLA_DV * 2, kAlign);
        w.tickets = w.part_ml + round_up(pieces * kvp::MLA_TCN_HEADS * 2 * sizeof(float), kAlign);
        w.ticket_bytes = static_cast<size_t>(batch) * p.head_tiles * sizeof(int);
        w.total = w.tickets + w.ticket_bytes;
    } else if (p.max_splits > 1 && p.form == kMlaWide) {
        // pieces (sequence, head tile, latent half, split): fp16 partials of 128 heads x
        // 256 latent numbers, fp32 (max, sum) per head, then the piece count of each
        // (sequence, head tile, half) -- read by the merge kernel
        const size_t pieces = static_cast<size_t>(batch) * p.head_tiles * 2 * p.max_splits;
        w.part_ml = round_up(pieces * kvp::MLA_TC_HEADS * (kvp::MLA_DV / 2) * 2, kAlign);
        w.tickets = w.part_ml + round_up(pieces * kvp::MLA_TC_HEADS * 2 * sizeof(float), kAlign);
        w.ticket_bytes = static_cast<size_t>(batch) * p.head_tiles * 2 * sizeof(int);
        w.total = w.tickets + w.ticket_bytes;
    } else if (p.max_splits > 1) {
        const size_t n = static_cast<size_t>(batch) * q_heads * p.max_splits;
        w.part_ml = round_up(n * kvp::MLA_DV * sizeof(float), kAlign);
        w.tickets = w.part_ml + round_up(n * 2 * sizeof(float), kAlign);
        w.ticket_bytes = static_cast<size_t>(batch) * p.head_tiles * sizeof(int);
        w.total = w.tickets + w.ticket_bytes;
    }
    return w;
}

}  // namespace

extern "C" {

kv_status kv_mla_pool_create(int num_blocks, int block_size, int latent_dim, int rope_dim,
                             int device, kv_pool** out)
{
    if (out == nullptr) return KV_ERR_INVALID_ARG;
    *out = nullptr;
    if (num_blocks <= 0 || block_size <= 0 || latent_dim <= 0 || rope_dim < 0 || device < 0)
        return KV_ERR_INVALID_ARG;
    if (latent_dim != kvp::MLA_DV || rope_dim != kvp::MLA_DR) return KV_ERR_UNSUPPORTED;
    if (kvp::mla_stage_tokens(block_size, true) == 0) return KV_ERR_UNSUPPORTED;
    const long double bytes = static_cast<long double>(num_blocks) * block_size * kvp::MLA_DK * 2;
    if (bytes >= static_cast<long double>(1ull << 40)) return KV_ERR_UNSUPPORTED;

    int ndev = 0;
    if (cudaGetDeviceCount(&ndev) != cudaSuccess || device >= ndev) return KV_ERR_CUDA;
    DeviceGuard guard(device);
    if (!guard.ok) return KV_ERR_CUDA;

    kv_pool* p = new (std::nothrow) kv_pool();
    if (p == nullptr) return KV_ERR_OUT_OF_MEMORY;
    p->num_blocks = num_blocks;
    p->block_size = block_size;
    p->kv_heads = 1;
    p->head_dim = kvp::MLA_DK;
    p->device = device;
    p->dtype = KV_DTYPE_BF16;
    p->elem = 2;
    p->mla = 1;
    p->pool_bytes = static_cast<size_t>(bytes);
    const size_t half = round_up(p->pool_bytes, kAlign);
    const size_t scales = round_up(sizeof(float), kAlign);
    const size_t total = half + 2 * scales + kAlign;
    if (cudaMalloc(&p->base, total) != cudaSuccess) {
        cudaGetLastError();
        delete p;
        return KV_ERR_OUT_OF_MEMORY;
    }
    uint8_t* b = static_cast<uint8_t*>(p->base);
    p->k = b;
    p->v = nullptr;
    p->k_scale = reinterpret_cast<float*>(b + half);
    p->v_scale = reinterpret_cast<float*>(b + half + scales);
    p->err = reinterpret_cast<uint32_t*>(b + half + 2 * scales);
    kv_status st = KV_OK;
    if (cudaMemset(p->base, 0, total) != cudaSuccess) st = KV_ERR_CUDA;
    if (st == KV_OK && cudaDeviceGetAttribute(&p->num_sms, cudaDevAttrMultiProcessorCount, device) !=
                           cudaSuccess)
        st = KV_ERR_CUDA;
    if (st == KV_OK)
        st = encode_pool_map(p, p->k, &p->tmk, kvp::mla_stage_tokens(block_size, true));
    if (st == KV_OK)
        st = encode_pool_map(p, p->k, &p->tmv, kvp::mla_stage_tokens(block_size, false));
    if (st == KV_OK && block_size == kvp::MLA_TC_BLOCK) {
        st = encode_pool_map(p, p->k, &p->tmt, block_size, 1);
        if (st == KV_OK) st = encode_pool_map(p, p->k, &p->tmh, kvp::MLA_TCN_STAGE_TOKENS, 1);
        if (st == KV_OK && kvp::prepare_mla_decode_tc() != cudaSuccess) st = KV_ERR_CUDA;
        if (st == KV_OK && kvp::prepare_mla_decode_tcn() != cudaSuccess) st = KV_ERR_CUDA;
        p->has_tc = 1;
    }
    if (st == KV_OK && kvp::prepare_mla_decode(block_size) != cudaSuccess) st = KV_ERR_CUDA;
    if (st == KV_OK && cudaDeviceSynchronize() != cudaSuccess) st = KV_ERR_CUDA;
    if (st != KV_OK) {
        cudaGetLastError();
        cudaFree(p->base);
        delete p;
        return st;
    }
    *out = p;
    return KV_OK;
}

kv_status paged_mla_decode_plan(const kv_pool* pool, int batch, int q_heads, int max_blocks,
                                int kv_split_tokens, int* split_tokens, int* max_splits)
{
    MlaPlan p;
    kv_status st = make_mla_plan(pool, batch, q_heads, max_blocks, kv_split_tokens, &p);
    if (st != KV_OK) return st;
    if (split_tokens) *split_tokens = p.split_blocks * pool->block_size;
    if (max_splits) *max_splits = p.max_splits;
    return KV_OK;
}

kv_status paged_mla_workspace_size(const kv_pool* pool, int batch, int q_heads, int max_blocks,
                                   int kv_split_tokens, size_t* bytes)
{
    if (bytes == nullptr) return KV_ERR_INVALID_ARG;
    MlaPlan p;
    kv_status st = make_mla_plan(pool, batch, q_heads, max_blocks, kv_split_tokens, &p);
    if (st != KV_OK) return st;
    *bytes = mla_workspace_layout(batch, q_heads, p).total;
    return KV_OK;
}

}  // extern "C"

namespace {

// Everything paged_mla_decode_attention checks and sets up before its launch.
kv_status make_mla_launch(const kv_pool* pool, const void* q, int q_heads, const int32_t* block_tables,
                          int max_blocks, const int32_t* context_lens, int batch, float scale,
                          int kv_split_tokens, void* workspace, size_t workspace_bytes, void* out,
                          float* lse_out, MlaPlan* plan_out, kvp::MlaParams* params)
{
    MlaPlan plan;
    kv_status st = make_mla_plan(pool, batch, q_heads, max_blocks, kv_split_tokens, &plan);
    if (st != KV_OK) return st;
    if (batch == 0) return KV_OK;
    if (q == nullptr || block_tables == nullptr || context_lens == nullptr || out == nullptr)
        return KV_ERR_INVALID_ARG;
    if (!std::isfinite(scale)) return KV_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(block_tables, 4) ||
        !aligned(context_lens, 4) || !aligned(lse_out, 4) || !aligned(workspace, 16))
        return KV_ERR_INVALID_ARG;
    const WorkspaceLayout wl = mla_workspace_layout(batch, q_heads, plan);
    if (wl.total > 0 && (workspace == nullptr || workspace_bytes < wl.total))
        return KV_ERR_INVALID_ARG;
    st = check_device(pool);
    if (st != KV_OK) return st;

    kvp::MlaParams& p = *params;
    p.q = static_cast<const uint16_t*>(q);
    p.tables = block_tables;
    p.ctx = context_lens;
    p.out = static_cast<uint16_t*>(out);
    p.lse = lse_out;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    p.part_o = wl.total > 0 ? reinterpret_cast<float*>(ws + wl.part_o) : nullptr;
    p.part_ml = wl.total > 0 ? reinterpret_cast<float*>(ws + wl.part_ml) : nullptr;
    p.tickets = wl.total > 0 ? reinterpret_cast<int*>(ws + wl.tickets) : nullptr;
    p.err = pool->err;
    p.batch = batch;
    p.q_heads = q_heads;
    p.head_tiles = plan.head_tiles;
    p.max_blocks = max_blocks;
    p.num_blocks = pool->num_blocks;
    p.split_blocks = plan.split_blocks;
    p.max_splits = plan.max_splits;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.kv_new = nullptr;
    p.pool = nullptr;
    *plan_out = plan;
    return KV_OK;
}

kv_status launch_mla(const kv_pool* pool, const MlaPlan& plan, const kvp::MlaParams& p, void* stream)
{
    if (plan.form != kMlaMma) {
        // persistent: one CTA per SM, each taking a contiguous range of the units
        // ((latent half,) head tile, sequence, block); no more CTAs than ranges of
        // split_blocks units the longest batch could have
        const int outer = plan.head_tiles * (plan.form == kMlaWide ? 2 : 1);
        const long long units_max = static_cast<long long>(outer) * p.batch * p.max_blocks;
        const long long ranges = units_max / plan.split_blocks > 0 ? units_max / plan.split_blocks : 1;
        const int sms = pool->num_sms > 0 ? pool->num_sms : 148;
        const dim3 grid(static_cast<unsigned>(ranges < sms ? ranges : sms));
        if (plan.form == kMlaWide)
            return kvp::launch_mla_decode_tc(grid, pool->tmt, p, static_cast<cudaStream_t>(stream)) == cudaSuccess
                       ? KV_OK
                       : KV_ERR_CUDA;
        CUtensorMap tq;
        const kv_status st = encode_query_map(p.q, p.q_heads, p.batch, &tq);
        if (st != KV_OK) return st;
        return kvp::launch_mla_decode_tcn(grid, pool->tmh, tq, p, static_cast<cudaStream_t>(stream)) == cudaSuccess
                   ? KV_OK
                   : KV_ERR_CUDA;
    }
    // chunk-major grid: x = head tile, y = sequence, z = chunk.  Grids of up to
    // three CTAs per SM run the producer-warp variant (32-token stages, two CTAs
    // per SM), larger ones the three-CTAs-per-SM variant (16-token stages).
    const dim3 grid(static_cast<unsigned>(plan.head_tiles), static_cast<unsigned>(p.batch),
                    static_cast<unsigned>(plan.max_splits));
    const long long ctas = static_cast<long long>(plan.head_tiles) * p.batch * plan.max_splits;
    const bool prod = ctas <= 3LL * (pool->num_sms > 0 ? pool->num_sms : 148);
    return kvp::launch_mla_decode(pool->block_size, prod, grid, prod ? pool->tmk : pool->tmv, p,
                                  static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? KV_OK
               : KV_ERR_CUDA;
}

}  // namespace

extern "C" {

kv_status paged_mla_decode_attention(const kv_pool* pool, const void* q, int q_heads,
                                     const int32_t* block_tables, int max_blocks,
                                     const int32_t* context_lens, int batch, float scale,
                                     int kv_split_tokens, void* workspace, size_t workspace_bytes,
                                     void* out, float* lse_out, void* stream)
{
    MlaPlan plan;
    kvp::MlaParams p;
    kv_status st = make_mla_launch(pool, q, q_heads, block_tables, max_blocks, context_lens, batch, scale,
                                   kv_split_tokens, workspace, workspace_bytes, out, lse_out, &plan, &p);
    if (st != KV_OK || batch == 0) return st;
    return launch_mla(pool, plan, p, stream);
}

kv_status paged_mla_decode_step(kv_pool* pool, const void* kv_new, const void* q, int q_heads,
                                const int32_t* block_tables, int max_blocks,
                                const int32_t* context_lens, int batch, float scale,
                                int kv_split_tokens, void* workspace, size_t workspace_bytes,
                                void* out, float* lse_out, void* stream)
{
    if (pool == nullptr) return KV_ERR_INVALID_ARG;
    // everything is checked before anything is launched
    MlaPlan plan;
    kvp::MlaParams p;
    kv_status st = make_mla_launch(pool, q, q_heads, block_tables, max_blocks, context_lens, batch, scale,
                                   kv_split_tokens, workspace, workspace_bytes, out, lse_out, &plan, &p);
    if (st != KV_OK || batch == 0) return st;
    if (kv_new == nullptr || !aligned(kv_new, 16)) return KV_ERR_INVALID_ARG;
    // One attention launch (plus the merge of cut sequences): the CTA that reads the block
    // holding a sequence's new vector writes it into the pool first (the append's bytes).
    p.kv_new = static_cast<const uint16_t*>(kv_new);
    p.pool = pool->k;
    return launch_mla(pool, plan, p, stream);
}

}  // extern "C"

// ---------------------------------------------------------------------------
// Allocation-free decode attention.
//
// For callers that cannot allocate device memory themselves: plug-in hosts
// that hand a kernel only its input and output buffers, engines whose own
// allocator has reserved the whole GPU up front, and latency-critical paths
// where cudaMalloc's implicit device-wide synchronisation would stall other
// streams.  The split-KV partials live in the fixed-size array below, which is
// part of the library's device image: every GPU that loads the library holds
// it until the process exits.
// ---------------------------------------------------------------------------
static __device__ __align__(256) unsigned char kv_noalloc_scratch[KV_NO_ALLOC_SCRATCH_BYTES];

namespace {

constexpr int kMaxScratchDevices = 64;
std::mutex g_scratch_mutex;
void* g_scratch_addr[kMaxScratchDevices] = {};

// Device address of the scratch array on `device` (which must be current).
// Looked up once per device; the lookup is the only set-up step.
kv_status scratch_address(int device, void** addr)
{
    if (device < 0 || device >= kMaxScratchDevices) return KV_ERR_UNSUPPORTED;
    std::lock_guard<std::mutex> lock(g_scratch_mutex);
    if (g_scratch_addr[device] == nullptr) {
        void* p = nullptr;
        if (cudaGetSymbolAddress(&p, kv_noalloc_scratch) != cudaSuccess || p == nullptr) {
            cudaGetLastError();
            return KV_ERR_CUDA;
        }
        g_scratch_addr[device] = p;
    }
    *addr = g_scratch_addr[device];
    return KV_OK;
}

}  // namespace

extern "C" kv_status paged_decode_attention_noalloc(const kv_pool* pool, const void* q, int q_heads,
                                                    const int32_t* block_tables, int max_blocks,
                                                    const int32_t* context_lens, int batch,
                                                    float scale, int kv_split_tokens, void* out,
                                                    float* lse_out, void* stream)
{
    Plan plan;
    kv_status st = make_plan(pool, batch, q_heads, 1, max_blocks, kv_split_tokens, &plan);
    if (st != KV_OK) return st;
    if (batch == 0) return KV_OK;
    const size_t need = workspace_bytes_for(pool, batch, plan);
    if (need > KV_NO_ALLOC_SCRATCH_BYTES) return KV_ERR_UNSUPPORTED;
    st = check_device(pool);
    if (st != KV_OK) return st;
    void* scratch = nullptr;
    if (need > 0) {
        st = scratch_address(pool->device, &scratch);
        if (st != KV_OK) return st;
    }
    // Every argument is checked before the shared array is touched: a call that is
    // rejected writes nothing to it and launches nothing.
    kvp::DecodeParams p;
    dim3 grid;
    st = make_decode_launch(pool, q, q_heads, 1, block_tables, max_blocks, context_lens, batch,
                            scale, kv_split_tokens, scratch, need, out, lse_out, &plan, &p, &grid);
    if (st != KV_OK) return st;
    if (need > 0) {
        // The per-unit chunk counts in the scratch must start at zero, whatever
        // an earlier (possibly failed) call left there.
        const WorkspaceLayout wl = workspace_layout(pool, batch, plan);
        if (wl.ticket_bytes > 0 &&
            cudaMemsetAsync(static_cast<uint8_t*>(scratch) + wl.tickets, 0, wl.ticket_bytes,
                            static_cast<cudaStream_t>(stream)) != cudaSuccess) {
            cudaGetLastError();
            return KV_ERR_CUDA;
        }
    }
    return launch_decode(pool, plan, grid, p, stream);
}
