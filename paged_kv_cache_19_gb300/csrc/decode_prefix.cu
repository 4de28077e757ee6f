// decode_prefix.cu -- the shared pass of paged_shared_prefix_attention on the 5th-generation
// tensor cores (tcgen05): attention of all query rows of a group of sequences over the cache
// blocks they share, each block read once for all of them.
//
//   o_r, m_r, l_r = online softmax of  scale q_r . K[t]  over the shared tokens t that row r sees
//
// for the rows r = (member, query head of the kv head, query token).  With n members, g heads
// and q tokens each that is a matrix product of n g q rows against the K and V rows of the
// prefix: 4 n g q head_dim operations per kv head and token for 2 head_dim numbers read, so from
// about a hundred rows on it is bound by the tensor cores and the exponentials instead of memory.
//
// Persistent, one CTA per SM; the units are (group, kv head, pair of 128-row tiles, 128-token
// tile) in that order, with PFX_PAD positions before each run for what starting one costs, and every
// CTA takes an equal contiguous range (prefix_groups.cuh), so a
// run -- one (group, kv head, pair) -- is cut at range borders and each cut leaves a normalised
// fp32 partial (a piece) that the suffix kernel merges by log-sum-exp.  Warps:
//   * 0-3 and 4-7: two softmax teams, one per slot (128 rows: thread = row = tensor-memory lane).
//     A pair of more than 128 rows has a row tile in each slot and both slots take every token
//     tile; a pair of fewer has the same rows in both and the slots take alternate tiles, so
//     that either way one slot's softmax runs while the tensor cores work for the other; then team
//     1 hands its state to team 0 through shared memory, which folds it into its own.  A row's
//     scores are one thread's: its maximum and sum need no exchange.  The outputs leave through
//     shared memory, so that a piece's rows are written whole.
//   * 8: loads.  It walks the CTA's range and hands every run on (PFX_ITEMS ahead), so that only one
//     warp reads the groups' arrays.  A 128-token tile is 128 / block_size blocks, one TMA box each
//     for K and for V:
//     8 slots x 128-byte pieces x octets of slots, so that the tile in shared memory is the
//     tensor cores' canonical 128-byte-swizzled layout with 8-token groups one after another.
//     K and V tiles go through one ring in the order the MMAs consume them.  Blocks past the
//     prefix and invalid ids are loaded from past the end of the pool: the copy fills zeros.
//   * 9: one thread issues the MMAs.  Scores S[128 rows x 128 tokens] = Q . K^T with Q in shared
//     memory; output O[128 x head_dim] += P . V with P in tensor memory over the scores it came
//     from.  Per slot the order S(i), softmax, O(i), S(i+1) is fixed by that overlay; the other
//     slot's two MMAs fill the time of the softmax.
//   * 10-13 (fp8 cache): convert each landed K or V tile of e4m3 codes to f16 (exact) into the
//     ring the MMAs read.  The rows are f16 then too: a row of q is scaled by a power of two to
//     below 2^15 first, undone in its score factor; probabilities are f16.
//     Codes as the operand of an 8-bit MMA would need 8-bit probabilities next to them, off by
//     2^-4; f16 ones are off by 2^-11, bf16 ones (bf16 cache, whose values f16 cannot hold) by 2^-8.
// The output is rescaled only when the running maximum grows by more than 2^8 (log2 units):
// until then the older maximum stays the reference, which is exact because the division at the
// end uses the sum taken against the same reference.
//
// Measured on a GB300: 128 sequences of 64 query heads over 8 kv heads (1,024 rows a kv head) behind
// one document of 16,384 tokens take the pass 62 us, 69 GFLOP a call = 1.1 PFLOP/s, the tensor cores
// busy in 47 % of the cycles: a unit of 256 rows x 128 tokens costs about 2,850 cycles of MMA (the
// score MMAs read Q and K from shared memory, 64 KB for 2 x 128 x 128 scores, and run at its
// rate) and 1,590 of softmax beside them; the beginning of a run costs about 3,600 (q), its end 5,500
// (8-bit: more, the rows of q are scaled to f16 in place first).  32 groups of 8 sequences (32 rows, 512 tokens)
// take about 22 us, bound by those.  Whether a group is worth a run is decided by prefix_shares.
//
// Every wait is bounded; a late barrier sets KV_DEVERR_TIMEOUT, every role leaves its loops, and
// the CTA waits for its copies and MMAs in flight and frees its tensor memory.
#include "decode_common.cuh"
#include "kernels.h"
#include "prefix_groups.cuh"
#include "tcgen05.cuh"

namespace kvp {

namespace {

constexpr float PFX_RESCALE_LOG2 = 8.f;
constexpr int PFX_MASKS = 16;                       // ring of per-tile block masks
// A CTA's range has sqrt(PFX_CUT x tiles of the longest run) positions at least: a longer range takes the
// pass longer, every further piece of a run its members' merge.  With 0 (every CTA works) / 0.25 / 0.5 /
// 1 / 2, few members behind long prefixes: 3 sequences behind 12,215 tokens 48 / 34 / 36 / 41 / 46 us,
// 5 behind 11,788 54 / 42 / 40 / 41 / 44, 14 behind 3,185 32 / 28 / 25 / 26 / 28; many runs do not care.
constexpr float PFX_CUT = 0.5f;

template <bool FP8, int D, int BS>
struct PfxCfg {
    static constexpr int PIECES = D * 2 / 128;                  // 128-byte pieces of a 16-bit row
    static constexpr int OCTET = PIECES * 1024;                 // 8 tokens of a tile in the MMA layout
    static constexpr int TILE = PFX_TILE * D * 2;               // K or V tile as the MMAs read it
    static constexpr int RAW = PFX_TILE * D;                    // the same as e4m3 codes
    static constexpr int NRING = FP8 ? 3 : 160 * 1024 / TILE;
    static constexpr int NRAW = FP8 ? 4 : 0;
    static constexpr int QTILE = PFX_TILE * D * 2;              // one slot's rows
    static constexpr int BLOCKS = PFX_TILE / BS;                // blocks of a tile
    static constexpr int BOX = FP8 ? BS * D : BS * D * 2;       // bytes of one block's box
    static constexpr int CTL = 2048;
    static constexpr int SMEM = 1024 + 2 * QTILE + NRING * TILE + NRAW * RAW + CTL;
    static constexpr int THREADS = FP8 ? 14 * 32 : 10 * 32;
    static constexpr uint32_t S0 = 0, O0 = 256;                 // tensor-memory columns of slot 0
    static constexpr uint32_t IDESC_S = FP8 ? tc_idesc_f16(128, PFX_TILE, 0, 0) : tc_idesc_bf16(128, PFX_TILE, 0, 0);
    static constexpr uint32_t IDESC_O = FP8 ? tc_idesc_f16(128, D, 0, 1) : tc_idesc_bf16(128, D, 0, 1);
    static_assert(SMEM <= 227 * 1024, "one CTA per SM");
    static_assert(!FP8 || D == 128, "fp8 path is laid out for head_dim 128");
};

constexpr int PFX_ITEMS = 4;                        // items handed on ahead

// A run of one CTA: tiles tile0 .. tile0 + n - 1 of (group, kv head, pair).
struct PfxItem {
    int off, rows;          // first member; rows of the pair (1 .. 256)
    int row0;               // group row of the pair's first row
    int kvh, blocks, tile0, n, run;
    int pieces;             // of the whole run (with tile 0)
    int both;               // the slots take alternate tiles of the same rows
};

struct PfxCtl {
    uint64_t full[16], empty[16];                   // the ring the MMAs read
    uint64_t raw_full[4], raw_empty[4];             // fp8: landed codes
    uint64_t q_ready[2], s_full[2], p_full[2], o_full[2], mma_done;
    uint64_t item_full[PFX_ITEMS], item_empty[PFX_ITEMS];
    PfxItem items[PFX_ITEMS];                       // n 0: no more
    uint32_t tmem_base;
    int abort_flag;
    uint32_t masks[PFX_MASKS];                      // valid blocks of a token tile
    long long lo, hi, units;                        // this CTA's range, all units
    long long base;                                 // first unit of group0
    int group0, ctas;                               // group that holds lo; CTAs with units
    long long scan[14];
    int longest[14];                                // tiles of the longest run, by warp
    uint64_t x_full, e_done[2];                     // team 1's state handed over; a team is done with an item
    float2 x_ml[PFX_TILE];                          // team 1's maxima and sums
};


// The CTA that holds unit u of `units` cut into ranges for n CTAs.
__device__ __forceinline__ int pfx_cta_of(long long u, long long units, int n)
{
    return static_cast<int>(div_small((u + 1) * n - 1, units));
}

// The items of a CTA's range.
struct PfxWalk {
    long long u, hi, base, units;
    int g, pairs, tiles;
    PrefixGroup gr;

    __device__ __forceinline__ void load(const PrefixParams& p, int block_size)
    {
        gr = load_prefix_group(p, g);
        pairs = prefix_pairs(p, gr);
        tiles = (gr.blocks * block_size + PFX_TILE - 1) / PFX_TILE;
        units = tiles > 0 ? static_cast<long long>(p.kv_heads) * pairs * (tiles + PFX_PAD) : 0;
    }
    __device__ __forceinline__ void init(const PrefixParams& p, const PfxCtl* ctl, int block_size)
    {
        u = ctl->lo;
        hi = ctl->hi;
        base = ctl->base;
        g = ctl->group0;
        if (u < hi) load(p, block_size);
    }
    __device__ __forceinline__ bool next(const PrefixParams& p, const PfxCtl* ctl, int block_size, PfxItem& it)
    {
        it.n = 0;
        int run, first;                             // the run at u; its tile there (< 0: padding)
        long long left;
        for (;;) {
            if (u >= hi) return false;
            while (u >= base + units) {             // hi is at most the last group's end
                base += units;
                ++g;
                load(p, block_size);
            }
            const long long rel = u - base;
            run = static_cast<int>(div_small(rel, tiles + PFX_PAD));
            first = static_cast<int>(rel - static_cast<long long>(run) * (tiles + PFX_PAD)) - PFX_PAD;
            if (first < 0) {
                u -= first;                         // over the padding
                first = 0;
            }
            left = hi - u;
            if (left > 0) break;
        }
        it.tile0 = first;
        it.n = left < tiles - it.tile0 ? static_cast<int>(left) : tiles - it.tile0;
        it.kvh = run / pairs;
        const int pair = run - it.kvh * pairs;
        it.off = gr.off;
        it.row0 = pair * PFX_PAIR;
        it.rows = min(PFX_PAIR, gr.n * p.rows - it.row0);
        it.both = it.rows <= PFX_TILE;
        it.blocks = gr.blocks;
        it.run = prefix_run_base(p, g, gr) + run;
        // the run's pieces: one per CTA from the one of its first tile to the one of its last
        it.pieces = it.tile0 == 0 ? pfx_cta_of(u + tiles - 1, ctl->units, ctl->ctas) - static_cast<int>(blockIdx.x) + 1 : 0;
        u += it.n;
        return true;
    }
};

__device__ __forceinline__ bool pfx_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag)
{
    if (mbar_try_wait(bar, parity)) return true;
    const unsigned long long t0 = global_timer_ns();
    for (uint32_t i = 1;; ++i) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((i & 63u) == 0 && (*abort_flag || global_timer_ns() - t0 > WAIT_LIMIT_NS)) return false;
    }
}

__device__ __forceinline__ float max3(float a, float b, float c)
{
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    float2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(reinterpret_cast<uint64_t&>(d))
        : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)), "l"(reinterpret_cast<uint64_t&>(c)));
    return d;
}

__device__ __forceinline__ float2 add2(float2 a, float2 b)
{
    float2 d;
    asm("add.rn.f32x2 %0, %1, %2;"
        : "=l"(reinterpret_cast<uint64_t&>(d))
        : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
    return d;
}

// Maximum of 32 scores and mx.
__device__ __forceinline__ float max_of(const uint32_t (&x)[32], float mx)
{
    float m[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) m[e] = fmaxf(__uint_as_float(x[e]), __uint_as_float(x[e + 4]));
#pragma unroll
    for (int j = 8; j < 32; j += 8)
#pragma unroll
        for (int e = 0; e < 4; ++e) m[e] = max3(m[e], __uint_as_float(x[j + e]), __uint_as_float(x[j + 4 + e]));
    return max3(max3(m[0], m[1], mx), m[2], m[3]);
}

// 32 scores -> probabilities 2^(score * mul + sub), packed in pairs, and added to the sums.
template <bool FP8>
__device__ __forceinline__ void probs(const uint32_t (&x)[32], float2 mul, float2 sub, float2 (&sum)[2], uint32_t (&pk)[16])
{
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        const float2 y = fma2(make_float2(__uint_as_float(x[2 * j]), __uint_as_float(x[2 * j + 1])), mul, sub);
        const float2 pr = make_float2(fast_exp2(y.x), fast_exp2(y.y));
        sum[j & 1] = add2(sum[j & 1], pr);
        pk[j] = FP8 ? pack_f16x2(pr.x, pr.y) : pack_bf16x2(pr.x, pr.y);
    }
}

__device__ __forceinline__ void pfx_give_up(const PrefixParams& p, volatile int* abort_flag)
{
    if (!*abort_flag) atomicOr(p.err, KV_DEVERR_TIMEOUT);
    *abort_flag = 1;
}

}  // namespace

template <bool FP8, int D, int BS>
__global__ void __launch_bounds__(PfxCfg<FP8, D, BS>::THREADS, 1)
paged_prefix_pass(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
                  const PrefixParams p)
{
    using C = PfxCfg<FP8, D, BS>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint8_t* qsm = smem;                            // two slots' rows
    uint8_t* ring = qsm + 2 * C::QTILE;
    uint8_t* raw = ring + C::NRING * C::TILE;
    PfxCtl* ctl = reinterpret_cast<PfxCtl*>(raw + C::NRAW * C::RAW);
    static_assert(sizeof(PfxCtl) <= C::CTL, "control block");

    const int tid = threadIdx.x;
    const int warp = tid >> 5;
    const int lane = tid & 31;
    volatile int* abort_flag = &ctl->abort_flag;

    if (tid == 0) {
        for (int i = 0; i < C::NRING; ++i) {
            mbar_init(smem_u32(&ctl->full[i]), FP8 ? 4 : 1);
            mbar_init(smem_u32(&ctl->empty[i]), 1);
        }
        for (int i = 0; i < C::NRAW; ++i) {
            mbar_init(smem_u32(&ctl->raw_full[i]), 1);
            mbar_init(smem_u32(&ctl->raw_empty[i]), 4);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(smem_u32(&ctl->q_ready[s]), 4);
            mbar_init(smem_u32(&ctl->s_full[s]), 1);
            mbar_init(smem_u32(&ctl->p_full[s]), 4);
            mbar_init(smem_u32(&ctl->o_full[s]), 1);
        }
        for (int i = 0; i < PFX_ITEMS; ++i) {
            mbar_init(smem_u32(&ctl->item_full[i]), 1);
            mbar_init(smem_u32(&ctl->item_empty[i]), FP8 ? 13 : 9);     // MMA thread, softmax and converter warps
        }
        mbar_init(smem_u32(&ctl->mma_done), 1);
        mbar_init(smem_u32(&ctl->x_full), 4);
        for (int s = 0; s < 2; ++s) mbar_init(smem_u32(&ctl->e_done[s]), 4);
        ctl->abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 9) tc_alloc(smem_u32(&ctl->tmem_base), 512);
    if (warp == 8 && lane == 0) {
        prefetch_tensormap(&tmk);
        prefetch_tensormap(&tmv);
    }
    grid_dependency_wait();                         // inputs of the preceding kernel are ready
    grid_dependents_launch();                       // the suffix kernel may start launching

    // ---- this CTA's range of units: every thread takes every THREADS-th group.  First the
    // total and the checks, then the group that holds the range's first unit.
    {
        long long sum = 0;
        int longest = 0;                            // tiles of a run
        bool ok = true, blocks_ok = true;
        for (int g = tid; g < p.n_groups; g += C::THREADS) {
            ok = ok && prefix_offsets_ok(p, g);
            const int blocks = __ldg(p.group_blocks + g);
            blocks_ok = blocks_ok && blocks >= 0 && blocks <= p.max_blocks;
            PfxWalk w;
            w.g = g;
            w.load(p, BS);
            sum += w.units;
            if (w.units > 0) longest = max(longest, w.tiles);
        }
        if ((!ok || !blocks_ok) && blockIdx.x == 0) atomicOr(p.err, KV_DEVERR_GROUP);
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(FULL_MASK, sum, o);
        longest = __reduce_max_sync(FULL_MASK, longest);
        if (lane == 0) {
            ctl->scan[warp] = sum;
            ctl->longest[warp] = longest;
        }
        const bool all = __syncthreads_and(ok);     // bad offsets: nothing is shared
        long long units = 0;
        for (int w = 0; w < C::THREADS / 32; ++w) {
            units += ctl->scan[w];
            longest = max(longest, ctl->longest[w]);
        }
        if (!all) units = 0;
        const long long least = max(1, static_cast<int>(sqrtf(PFX_CUT * static_cast<float>(longest))));
        const long long most = (units + least - 1) / least;
        const int ctas = most < gridDim.x ? static_cast<int>(most) : static_cast<int>(gridDim.x);
        const int c = blockIdx.x;
        const long long lo = c < ctas ? div_small(units * c, ctas) : 0;
        const long long hi = c < ctas ? div_small(units * (c + 1), ctas) : 0;
        if (tid == 0) {
            ctl->units = units;
            ctl->ctas = ctas;
            ctl->lo = lo;
            ctl->hi = hi;
        }
        long long before = 0;                       // units of the groups of earlier rounds
        for (int g0 = 0; lo < hi && g0 < p.n_groups && before <= lo; g0 += C::THREADS) {
            PfxWalk w;
            w.units = 0;
            w.g = g0 + tid;
            if (w.g < p.n_groups) w.load(p, BS);
            long long scan = w.units;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long x = __shfl_up_sync(FULL_MASK, scan, o);
                if (lane >= o) scan += x;
            }
            __syncthreads();                        // the sums before this round are read
            if (lane == 31) ctl->scan[warp] = scan;
            __syncthreads();
            long long base = before + scan - w.units;
            for (int v = 0; v < warp; ++v) base += ctl->scan[v];
            for (int v = 0; v < C::THREADS / 32; ++v) before += ctl->scan[v];
            if (base <= lo && lo < base + w.units) {
                ctl->group0 = w.g;
                ctl->base = base;
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = ctl->tmem_base;
    PfxItem it;
    // item k as the producer handed it on; false: no more, or the wait gave up (then failed is set)
    const auto take_item = [&](int k, bool leader, bool& failed) {
        const int slot = k % PFX_ITEMS;
        if (!pfx_wait(smem_u32(&ctl->item_full[slot]), static_cast<uint32_t>(k / PFX_ITEMS) & 1u, abort_flag)) {
            failed = true;
            return false;
        }
        it = ctl->items[slot];
        if (leader) mbar_arrive(smem_u32(&ctl->item_empty[slot]));
        return it.n > 0;
    };

    if (warp == 8) {
        // ------------------------------------------------------------ loads
        // Tile sequence of an item, as the MMAs consume it: K_0 [K_1], then V_i, K_i+L with
        // L = 1, or 2 where the slots alternate.  The block ids of 32 blocks at a time, one
        // batch ahead of V's (K is at most two tiles ahead of V).
        constexpr int TPB = 32 / C::BLOCKS;         // tiles per batch of ids
        static_assert(TPB >= 3, "K never needs a batch that V's progress has not fetched");
        constexpr int NSLOT = FP8 ? C::NRAW : C::NRING;
        const uint32_t slot0 = smem_u32(FP8 ? raw : ring);
        constexpr uint32_t SLOT = FP8 ? C::RAW : C::TILE;
        uint64_t* full = FP8 ? ctl->raw_full : ctl->full;
        uint64_t* empty = FP8 ? ctl->raw_empty : ctl->empty;
        const int past = p.num_blocks;              // first block outside the pool: zeros
        int n = 0;                                  // tiles of K and V issued
        int kt = 0;                                 // K tiles issued
        bool ok = true;
        PfxWalk walk;
        walk.init(p, ctl, BS);
        for (int k = 0; ok; ++k) {
            const bool more = walk.next(p, ctl, BS, it);
            const int slot = k % PFX_ITEMS;
            ok = all_ok(pfx_wait(smem_u32(&ctl->item_empty[slot]), (static_cast<uint32_t>(k / PFX_ITEMS) & 1u) ^ 1u, abort_flag));
            if (!ok) break;
            if (lane == 0) {
                ctl->items[slot] = it;
                mbar_arrive(smem_u32(&ctl->item_full[slot]));
            }
            __syncwarp();
            if (!more) break;
            const int32_t* trow = p.tables + static_cast<size_t>(it.off) * p.max_blocks;
            const int blk0 = it.tile0 * C::BLOCKS;
            const int nblk = min(it.n * C::BLOCKS, it.blocks - blk0);   // blocks of the prefix
            const auto fetch = [&](int batch) {
                const int j = batch * 32 + lane;
                int id = past;
                if (j < nblk) {
                    id = __ldg(trow + blk0 + j);
                    if (id < 0 || id >= p.num_blocks) {
                        atomicOr(p.err, KV_DEVERR_BLOCK_ID);
                        id = past;                  // skipped: never addressed
                    }
                }
                return id;
            };
            int ids[2] = {fetch(0), fetch(1)};
            const auto issue = [&](const CUtensorMap* map, int tile, bool is_k) {
                const int batch = tile / TPB;
                const int mine = (tile - batch * TPB) * C::BLOCKS + lane % C::BLOCKS;
                const int id = __shfl_sync(FULL_MASK, batch & 1 ? ids[1] : ids[0], mine);
                const int s = n % NSLOT;
                bool good = true;
                if (lane == 0)                      // (test hook: at stop_stage the wait runs out)
                    good = n != p.stop_stage &&
                           pfx_wait(smem_u32(empty + s), (static_cast<uint32_t>(n / NSLOT) & 1u) ^ 1u, abort_flag);
                if (!all_ok(good)) return false;
                const uint32_t bar = smem_u32(full + s);
                if (is_k) {
                    const uint32_t held = __ballot_sync(FULL_MASK, id < past) & ((1u << C::BLOCKS) - 1u);
                    if (lane == 0) ctl->masks[kt % PFX_MASKS] = held;
                    ++kt;
                }
                if (lane == 0) mbar_arrive_expect_tx(bar, SLOT);
                __syncwarp();
                if (lane < C::BLOCKS)
                    tma_load_5d(slot0 + s * SLOT + lane * C::BOX, map, 0, 0, 0, id * (BS / 8), it.kvh, bar);
                ++n;
                return true;
            };
            const int ahead = it.both ? 2 : 1;
            for (int i = 0; ok && i < min(ahead, it.n); ++i) ok = issue(&tmk, i, true);
            for (int i = 0; ok && i < it.n; ++i) {
                ok = issue(&tmv, i, false);
                if (i % TPB == 0 && i > 0) {        // V has entered batch i / TPB: fetch the next
                    if ((i / TPB) & 1)
                        ids[0] = fetch(i / TPB + 1);
                    else
                        ids[1] = fetch(i / TPB + 1);
                }
                if (ok && i + ahead < it.n) ok = issue(&tmk, i + ahead, true);
            }
        }
        if (!ok) pfx_give_up(p, abort_flag);
        // copies still in flight must land before the CTA exits
        if (lane == 0)
            for (int j = max(0, n - NSLOT); j < n; ++j)
                if (!mbar_wait_bounded(smem_u32(full + j % NSLOT), static_cast<uint32_t>(j / NSLOT) & 1u)) break;
    } else if (warp == 9) {
        // ------------------------------------------------------------ MMA issue
        if (lane == 0) {
            bool ok = true;
            int n = 0;                              // tiles of K and V consumed
            uint32_t done[2] = {0u, 0u};            // softmax tiles waited for, per slot
            const auto wait_tile = [&](int at) {
                const bool good = pfx_wait(smem_u32(&ctl->full[at % C::NRING]),
                                           static_cast<uint32_t>(at / C::NRING) & 1u, abort_flag);
                tc_fence_after();
                return good;
            };
            const auto scores = [&](int s, int at) {
                const uint64_t a = tc_smem_desc(smem_u32(qsm) + s * C::QTILE, 16, 1024);
                const uint64_t b = tc_smem_desc(smem_u32(ring) + at % C::NRING * C::TILE, 16, C::OCTET);
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks)
                    tc_mma_ss(tbase + C::S0 + s * PFX_TILE,
                              a + static_cast<uint64_t>(((ks >> 2) * (PFX_TILE * 128) + (ks & 3) * 32) >> 4),
                              b + static_cast<uint64_t>(((ks >> 2) * 1024 + (ks & 3) * 32) >> 4), C::IDESC_S, ks > 0);
                tc_commit(smem_u32(&ctl->s_full[s]));
            };
            const auto output = [&](int s, int at, bool first) {
                const uint64_t b = tc_smem_desc(smem_u32(ring) + at % C::NRING * C::TILE, 1024, C::OCTET);
#pragma unroll
                for (int kk = 0; kk < PFX_TILE / 16; ++kk)
                    tc_mma_ts(tbase + C::O0 + s * D, tbase + C::S0 + s * PFX_TILE + kk * 8,
                              b + static_cast<uint64_t>((kk * 2 * C::OCTET) >> 4), C::IDESC_O, !(first && kk == 0));
            };
            const auto release = [&](int at) { tc_commit(smem_u32(&ctl->empty[at % C::NRING])); };
            const auto wait_p = [&](int s) {
                const bool good = pfx_wait(smem_u32(&ctl->p_full[s]), done[s]++ & 1u, abort_flag);
                tc_fence_after();
                return good;
            };
            bool failed = false;
            for (int k = 0; ok && take_item(k, true, failed); ++k) {
                for (int s = 0; ok && s < 2; ++s)
                    ok = pfx_wait(smem_u32(&ctl->q_ready[s]), static_cast<uint32_t>(k) & 1u, abort_flag);
                tc_fence_after();
                if (!it.both) {
                    if (ok && (ok = wait_tile(n))) {
                        scores(0, n);
                        scores(1, n);
                        release(n++);
                    }
                    for (int i = 0; ok && i < it.n; ++i) {
                        const int v = n, kn = n + 1;
                        const bool more = i + 1 < it.n;
                        if (!(ok = wait_tile(v) && wait_p(0))) break;
                        output(0, v, i == 0);
                        if (more) {
                            if (!(ok = wait_tile(kn))) break;
                            scores(0, kn);
                        }
                        if (!(ok = wait_p(1))) break;
                        output(1, v, i == 0);
                        release(v);
                        ++n;
                        if (more) {
                            scores(1, kn);
                            release(kn);
                            ++n;
                        }
                    }
                } else {
                    for (int i = 0; ok && i < min(2, it.n); ++i)
                        if ((ok = wait_tile(n))) {
                            scores(i, n);
                            release(n++);
                        }
                    for (int i = 0; ok && i < it.n; ++i) {
                        const int s = i & 1;
                        if (!(ok = wait_tile(n) && wait_p(s))) break;
                        output(s, n, i < 2);
                        release(n++);
                        if (i + 2 < it.n) {
                            if (!(ok = wait_tile(n))) break;
                            scores(s, n);
                            release(n++);
                        }
                    }
                }
                tc_commit(smem_u32(&ctl->o_full[0]));
                tc_commit(smem_u32(&ctl->o_full[1]));
            }
            if (!ok || failed) pfx_give_up(p, abort_flag);
            // every MMA issued must be complete before the tensor memory is freed
            tc_commit(smem_u32(&ctl->mma_done));
            mbar_wait_bounded(smem_u32(&ctl->mma_done), 0);
        }
    } else if (warp < 8) {
        // ------------------------------------------------------------ softmax, epilogue
        const int s = warp >> 2;                    // slot
        const int w = warp & 3;
        const int row = w * 32 + lane;              // row of the slot = tensor-memory lane
        const uint32_t lrow = tbase + (static_cast<uint32_t>(w * 32) << 16);
        const uint32_t tm_s = lrow + C::S0 + s * PFX_TILE, tm_o = lrow + C::O0 + s * D;
        const uint32_t qs = smem_u32(qsm) + s * C::QTILE;
        bool ok = true;
        int kt = 0;                                 // K tiles of the items before
        uint32_t seen = 0;                          // score tiles of this slot waited for
        int swaps = 0;                              // items whose slots were merged
        bool last_handed = false;
        for (int k = 0;; ++k) {
            bool failed = false;
            const bool more = take_item(k, false, failed);
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&ctl->item_empty[k % PFX_ITEMS]));
            ok = all_ok(!failed);
            if (!ok || !more) break;
            // ---- this warp's 32 rows of q into shared memory (K-major, 128-byte swizzle).  The score
            // MMAs of the item before are complete (o_full); its epilogue, which goes through this
            // memory, must be over in every warp of the team, and in team 0's if it merged.
            if (k > 0) {
                const uint32_t ph = static_cast<uint32_t>(k - 1) & 1u;
                ok = pfx_wait(smem_u32(&ctl->e_done[s]), ph, abort_flag);
                if (ok && s == 1 && last_handed) ok = pfx_wait(smem_u32(&ctl->e_done[0]), ph, abort_flag);
                if (!all_ok(ok)) {
                    ok = false;
                    break;
                }
            }
            const int first = it.row0 + (it.both ? 0 : s * PFX_TILE);   // group row of slot row 0
            const int rows = it.both ? it.rows : min(PFX_TILE, it.rows - s * PFX_TILE);
            constexpr int CH = D / 8;               // 16-byte chunks of a row
            constexpr int RPI = 32 / CH;            // rows of a warp-wide load
            const int ch = lane % CH;
            int r = w * 32 + lane / CH;             // the lane's row, its member and row of the member
            int m = (first + r) / p.rows, rr = first + r - m * p.rows;
            const auto source = [&]() {
                return reinterpret_cast<const uint4*>(
                           p.q + ((static_cast<size_t>(it.off + m) * p.kv_heads + it.kvh) * p.rows + rr) * D) + ch;
            };
            const auto target = [&]() { return qs + (ch >> 3) * (PFX_TILE * 128) + r * 128 + (((ch & 7) ^ (r & 7)) << 4); };
            const auto step = [&]() {
                r += RPI;
                for (rr += RPI; rr >= p.rows; rr -= p.rows) ++m;
            };
            // (loops are kept rolled: a launch fetches its code once, and a tile or two per CTA is all
            // that a short prefix has to hide that behind)
#pragma unroll 2
            for (int j = 0; j < CH; ++j, step()) {
                if (r < rows)
                    cp_async16(target(), source());
                else
                    asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(target()), "r"(0u) : "memory");
            }
            cp_async_wait_all();
            float q_up = 1.f;                       // undoes the row's power-of-two scale
            if constexpr (FP8) {
                // Each lane its row, in place: the largest magnitude to [2^14, 2^15) by a power of two,
                // then f16.
                __syncwarp();
                const auto chunk = [&](int c) { return qs + (c >> 3) * (PFX_TILE * 128) + row * 128 + (((c & 7) ^ (row & 7)) << 4); };
                uint32_t top = 0;                   // magnitudes of bf16 pairs order like integers
#pragma unroll 4
                for (int c = 0; c < CH; ++c) {
                    const uint4 x = lds128(chunk(c));
                    top = __vmaxu2(__vmaxu2(top, __vmaxu2(x.x & 0x7fff7fffu, x.y & 0x7fff7fffu)),
                                   __vmaxu2(x.z & 0x7fff7fffu, x.w & 0x7fff7fffu));
                }
                const uint32_t big = max(top << 16, top & 0xffff0000u);
                const int ex = min(254, max(14, 268 - static_cast<int>(big >> 23)));      // of the factor
                q_up = __uint_as_float(static_cast<uint32_t>(254 - ex) << 23);
                const float down = __uint_as_float(static_cast<uint32_t>(ex) << 23);
#pragma unroll 2
                for (int c = 0; c < CH; ++c) {
                    const uint4 x = lds128(chunk(c));
                    uint32_t v[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        v[e] = pack_f16x2(__uint_as_float(v[e] << 16) * down, __uint_as_float(v[e] & 0xffff0000u) * down);
                    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(chunk(c)), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                                 "r"(v[3])
                                 : "memory");
                }
            }
            fence_proxy_async_smem();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&ctl->q_ready[s]));

            // ---- the row: its visible tokens of the prefix, its score factor
            float mult0 = p.scale_log2;
            if constexpr (FP8) mult0 *= q_up * __ldg(p.k_scale + it.kvh);
            int lim = 1 << 30;                      // a row of padding: never masked, never stored
            const bool idle = w * 32 >= rows;       // a warp of padding: its probabilities are left
            if (row < rows) {                       // as they are, they reach its own rows alone
                const int m = (first + row) / p.rows, rr = first + row - m * p.rows;
                int ctx = __ldg(p.ctx + it.off + m);
                ctx = max(0, min(ctx, p.max_blocks * BS));
                lim = max(0, min(it.blocks * BS, ctx - p.q_len + rr % p.q_len + 1));
            }
            float m_ref = -INFINITY, l = 0.f;
            for (int i = it.both ? s : 0; i < it.n; i += it.both ? 2 : 1) {
                ok = all_ok(pfx_wait(smem_u32(&ctl->s_full[s]), seen++ & 1u, abort_flag));
                if (!ok) break;
                if (idle) {
                    if (lane == 0) mbar_arrive(smem_u32(&ctl->p_full[s]));
                    continue;
                }
                tc_fence_after();
                const uint32_t held = ctl->masks[(kt + i) % PFX_MASKS];
                const int nvis = lim - (it.tile0 + i) * PFX_TILE;         // visible tokens of the tile
                float mult = mult0;
                // A tile with hidden tokens (or a factor that turns the order round) is scaled and
                // masked in place first, so that the loop below has one form.
                if (!__all_sync(FULL_MASK, nvis >= PFX_TILE && mult0 >= 0.f) || held != (1u << C::BLOCKS) - 1u) {
#pragma unroll 1
                    for (int c = 0; c < PFX_TILE; c += 32) {
                        uint32_t r[32];
                        tc_ld32(tm_s + c, r);
                        tc_wait_ld();
#pragma unroll
                        for (int j = 0; j < 32; ++j) {
                            const bool seen_by = c + j < nvis && (held >> ((c + j) / BS) & 1u);
                            r[j] = __float_as_uint(seen_by ? __uint_as_float(r[j]) * mult0 : -INFINITY);
                        }
                        tc_st32(tm_s + c, r);
                    }
                    tc_wait_st();
                    mult = 1.f;
                }
                // The maximum: 32 columns at a time, the next ones on their way meanwhile.
                float mx = -INFINITY;
                uint32_t a[32], b[32];
                tc_ld32(tm_s, a);
#pragma unroll
                for (int c = 0; c < PFX_TILE; c += 64) {
                    tc_wait_ld(a);
                    tc_ld32(tm_s + c + 32, b);
                    mx = max_of(a, mx);
                    tc_wait_ld(b);
                    if (c + 64 < PFX_TILE) tc_ld32(tm_s + c + 64, a);
                    mx = max_of(b, mx);
                }
                mx *= mult;
                float f = 1.f;
                if (m_ref == -INFINITY) {
                    m_ref = mx;                     // nothing accumulated yet
                } else if (mx > m_ref + PFX_RESCALE_LOG2) {
                    f = fast_exp2(m_ref - mx);
                    l *= f;
                    m_ref = mx;
                }
                if (__any_sync(FULL_MASK, f != 1.f)) {
                    // this slot's output MMAs so far are complete: its scores were issued after
                    // them and have been waited for
#pragma unroll 1
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t r[32];
                        tc_ld32(tm_o + c * 32, r);
                        tc_wait_ld();
#pragma unroll
                        for (int j = 0; j < 32; ++j) r[j] = __float_as_uint(__uint_as_float(r[j]) * f);
                        tc_st32(tm_o + c * 32, r);
                    }
                    tc_wait_st();
                }
                const float m_use = m_ref == -INFINITY ? 0.f : m_ref;
                const float2 mul2 = make_float2(mult, mult), sub2 = make_float2(-m_use, -m_use);
                float2 ls[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                // Probabilities over the scores they come from: 32 tokens become 16 columns, all of
                // which have been read by then.
                tc_ld32(tm_s, a);
#pragma unroll
                for (int c = 0; c < PFX_TILE; c += 64) {
                    uint32_t pk[16];
                    tc_wait_ld(a);
                    tc_ld32(tm_s + c + 32, b);
                    probs<FP8>(a, mul2, sub2, ls, pk);
                    tc_wait_ld(b);
                    tc_st16(tm_s + c / 2, pk);
                    if (c + 64 < PFX_TILE) tc_ld32(tm_s + c + 64, a);
                    probs<FP8>(b, mul2, sub2, ls, pk);
                    tc_st16(tm_s + c / 2 + 16, pk);
                }
                const float2 lt = add2(ls[0], ls[1]);
                l += lt.x + lt.y;
                tc_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&ctl->p_full[s]));
            }
            if (ok) ok = all_ok(pfx_wait(smem_u32(&ctl->o_full[s]), static_cast<uint32_t>(k) & 1u, abort_flag));
            if (!ok) break;
            tc_fence_after();

            // ---- epilogue: the pair's rows of the piece, normalised.  Where the slots took alternate
            // tiles of the same rows, team 1 hands its state over through the rows' shared memory
            // (idle: every score MMA of the item is complete), [number][row], and team 0 merges.
            float m_out = m_ref, l_out = l, keep = 1.f, add = 0.f;
            const bool handed = it.both && it.n > 1;
            float* xo = reinterpret_cast<float*>(qsm);
            if (handed) {
                const uint32_t ph = static_cast<uint32_t>(swaps) & 1u;
                ++swaps;
                ok = all_ok(pfx_wait(smem_u32(&ctl->o_full[s ^ 1]), static_cast<uint32_t>(k) & 1u, abort_flag));
                if (ok && s == 1 && !idle) {
#pragma unroll 1
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t r[32];
                        tc_ld32(tm_o + c * 32, r);
                        tc_wait_ld();
#pragma unroll
                        for (int j = 0; j < 32; ++j) xo[(c * 32 + j) * PFX_TILE + row] = __uint_as_float(r[j]);
                    }
                    ctl->x_ml[row] = make_float2(m_ref, l);
                }
                __syncwarp();
                if (ok && s == 1 && lane == 0) mbar_arrive(smem_u32(&ctl->x_full));
                if (ok && s == 0) ok = all_ok(pfx_wait(smem_u32(&ctl->x_full), ph, abort_flag));
                if (!ok) break;
                if (s == 0) {
                    const float2 o = ctl->x_ml[row];
                    m_out = o.y > 0.f ? (l > 0.f ? fmaxf(m_ref, o.x) : o.x) : m_ref;
                    keep = l > 0.f ? fast_exp2(m_ref - m_out) : 0.f;
                    add = o.y > 0.f ? fast_exp2(o.x - m_out) : 0.f;
                    l_out = l * keep + o.y * add;
                }
            }
            if (!idle && !(it.both && s == 1)) {
                const float inv = l_out > 0.f ? 1.f / l_out : 0.f;
                keep *= inv;
                add *= inv;
                const size_t at = (static_cast<size_t>(blockIdx.x) + it.run) * PFX_PAIR + s * PFX_TILE + row;
                if (row < rows)
                    p.piece_lse[at] = make_float4(l_out > 0.f ? m_out + __log2f(l_out) : -INFINITY, 0.f, 0.f, 0.f);
                // Through shared memory, half a row at a time, so that the warp's stores are whole
                // rows: its own 128 bytes of every 512-byte line of the slot's query rows (idle by
                // now; with a merge, the lines of the numbers it has just read), 16-byte chunk c of
                // row i in line 32 (c / 8) + i at c % 8 ^ i % 8.
                constexpr int HALF = D / 2;
                const uint32_t stage = smem_u32(qsm) + s * C::QTILE + w * 128;
                const auto chunk = [&](int i, int c) { return stage + ((c >> 3) * 32 + i) * 512 + (((c & 7) ^ (i & 7)) << 4); };
#pragma unroll 1
                for (int d0 = 0; d0 < D; d0 += HALF) {
#pragma unroll 1
                    for (int c = 0; c < HALF; c += 32) {
                        uint32_t x[32];
                        tc_ld32(tm_o + d0 + c, x);
                        tc_wait_ld(x);
#pragma unroll
                        for (int j = 0; j < 32; ++j) x[j] = __float_as_uint(__uint_as_float(x[j]) * keep);
                        if (add != 0.f) {
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                x[j] = __float_as_uint(__uint_as_float(x[j]) + xo[(d0 + c + j) * PFX_TILE + row] * add);
                        }
                        __syncwarp();               // (the lines of d0 + c .. are read by every lane)
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(chunk(lane, c / 4 + j)), "r"(x[4 * j]),
                                         "r"(x[4 * j + 1]), "r"(x[4 * j + 2]), "r"(x[4 * j + 3])
                                         : "memory");
                    }
                    __syncwarp();
                    constexpr int CPR = HALF / 4;   // chunks of a row's half
#pragma unroll 4
                    for (int e = lane; e < 32 * CPR; e += 32) {
                        const int i = e / CPR, c = e % CPR;
                        const uint4 v = lds128(chunk(i, c));
                        if (w * 32 + i < rows)
                            *reinterpret_cast<uint4*>(p.piece_o + (at - lane + i) * D + d0 + c * 4) = v;
                    }
                    __syncwarp();
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&ctl->e_done[s]));
            last_handed = handed;
            if (it.tile0 == 0 && tid == 0) p.runs[it.run] = make_int2(static_cast<int>(blockIdx.x) + it.run, it.pieces);
            tc_fence_before();
            kt += it.n;
        }
        if (!ok && lane == 0) pfx_give_up(p, abort_flag);
    } else {
        // ------------------------------------------------------------ fp8: codes to f16
        if constexpr (FP8) {
            const int t = tid - 10 * 32;            // token of the tile
            bool ok = true;
            int n = 0;
            bool failed = false;
            for (int k = 0; ok; ++k) {
                const bool more = take_item(k, false, failed);
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&ctl->item_empty[k % PFX_ITEMS]));
                ok = all_ok(!failed);
                if (!more) break;
                for (int i = 0; ok && i < 2 * it.n; ++i, ++n) {
                    const int rs = n % C::NRAW, s = n % C::NRING;
                    ok = all_ok(pfx_wait(smem_u32(&ctl->raw_full[rs]), static_cast<uint32_t>(n / C::NRAW) & 1u, abort_flag) &&
                                pfx_wait(smem_u32(&ctl->empty[s]), (static_cast<uint32_t>(n / C::NRING) & 1u) ^ 1u, abort_flag));
                    if (!ok) break;
                    const uint32_t src = smem_u32(raw) + rs * C::RAW + t * 128;
                    const uint32_t dst = smem_u32(ring) + s * C::TILE + (t >> 3) * C::OCTET + (t & 7) * 128;
#pragma unroll 2
                    for (int c = 0; c < 8; ++c) {   // 16 codes -> two 16-byte chunks
                        const uint4 v = lds128(src + ((c ^ (t & 7)) << 4));
                        const uint32_t q[4] = {v.x, v.y, v.z, v.w};
                        uint32_t h[8];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            h[2 * e] = e4m3x2_to_f16x2(q[e]);
                            h[2 * e + 1] = e4m3x2_to_f16x2(q[e] >> 16);
                        }
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int ch = 2 * c + e;
                            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                                             dst + (ch >> 3) * 1024 + (((ch & 7) ^ (t & 7)) << 4)),
                                         "r"(h[4 * e]), "r"(h[4 * e + 1]), "r"(h[4 * e + 2]), "r"(h[4 * e + 3])
                                         : "memory");
                        }
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(smem_u32(&ctl->full[s]));
                        mbar_arrive(smem_u32(&ctl->raw_empty[rs]));
                    }
                }
            }
            if (!ok && lane == 0) pfx_give_up(p, abort_flag);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 9) tc_dealloc(tbase, 512);
}

#define KVP_PREFIX_VARIANTS(X) X(false, 64, 16) X(false, 64, 32) X(false, 128, 16) X(false, 128, 32) X(true, 128, 16) X(true, 128, 32)

cudaError_t prepare_prefix(bool fp8, int head_dim, int block_size)
{
#define KVP_CASE(F_, D_, BS_) \
    if (fp8 == F_ && head_dim == D_ && block_size == BS_) \
        return cudaFuncSetAttribute(paged_prefix_pass<F_, D_, BS_>, cudaFuncAttributeMaxDynamicSharedMemorySize, \
                                    PfxCfg<F_, D_, BS_>::SMEM);
    KVP_PREFIX_VARIANTS(KVP_CASE)
#undef KVP_CASE
    return cudaErrorInvalidValue;
}

cudaError_t launch_prefix(bool fp8, int head_dim, int block_size, int ctas, const CUtensorMap& tk,
                          const CUtensorMap& tv, const PrefixParams& p, cudaStream_t s)
{
#define KVP_CASE(F_, D_, BS_) \
    if (fp8 == F_ && head_dim == D_ && block_size == BS_) \
        return launch_dependent(paged_prefix_pass<F_, D_, BS_>, dim3(static_cast<unsigned>(ctas)), \
                                dim3(PfxCfg<F_, D_, BS_>::THREADS), PfxCfg<F_, D_, BS_>::SMEM, s, tk, tv, p);
    KVP_PREFIX_VARIANTS(KVP_CASE)
#undef KVP_CASE
    return cudaErrorInvalidValue;
}

}  // namespace kvp
