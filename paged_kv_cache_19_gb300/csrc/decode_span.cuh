// decode_span.cuh -- paged attention over a span of each sequence's keys: every query row sees
// one contiguous interval of token positions, and only the blocks that the rows of a tile see
// are read.
//
// For query token i of a sequence (position p = ctx - q_len + i) and query head h:
//   keys   max(first, p - window + 1) <= t < max(p + 1, min(prefix, ctx))
//   score  x = scale q . K[t];  x <- cap tanh(x / cap);  x <- x - slope_h |p - t|
//   out = softmax over those keys of x, times V;  a row that sees no key gives 0 and lse = -inf
// (the sliding window, the cap, the distance bias, the document start and the visible prefix
// are each optional).  The suffix form (SPAN_SUFFIX, paged_shared_prefix_attention) starts a
// sequence's keys behind the blocks that its group shares and takes the pieces that the shared
// pass left for its rows (prefix_groups.cuh) into the merge.
//
// A unit is (sequence, group of HC kv heads, tile of query rows) with the 16-token sub-blocks its
// rows see.  Windows, document starts and shared parts make the units of a batch short and unequal,
// so the grid is persistent -- the CTAs that are resident together -- and the units' sub-blocks,
// each unit preceded by SPAN_PAD positions for what starting and finishing it costs, are cut into
// equal contiguous ranges, one per CTA.
//   * One producer warp walks the CTA's range, hands every unit on through a queue in shared memory
//     and streams what it needs through a ring of stages: the query rows, then its sub-blocks, HC
//     heads at a time (one 5-D TMA tensor load for their K tiles, one for V; a load per head and tile
//     took 8-bit caches 117 us instead of 111 for 64 x 4,096 tokens), then the pieces of the shared
//     pass (bulk copies).  It runs ahead over unit borders, so the consumers read nothing from global
//     memory themselves and find the next unit's lengths and data there.
//   * Four consumer warps, 4 / HC per kv head, fold their head's tile of a sub-block (every
//     (4 / HC)-th one) into an online-softmax state in registers (decode_common.cuh,
//     process_block_rows under the rule of SpanRows).  With four heads a warp owns its rows and
//     finishes a unit by itself.
// Several warps of one head hand their states to the first of them through shared memory.  The
// pieces of a unit cut by a range border go through global memory: each leaves its fp32 state in the
// accumulators' layout, and the warp that finishes last merges them in order (tickets by range and
// head, zero between calls); many pieces in two levels.
// Bound by the K/V bytes of the visible blocks where there are many, by the kernel's beginning and
// end where there are few, and with an 8-bit cache by the handing over of 16-token stages: half the
// bytes of bf16 for the same waits and arrivals (packed documents take 24 of their 28 us without any
// arithmetic on the blocks; the decode kernel of several heads streams the same codes in 32-token
// stages at 96 % of the copy rate).  Measured on a GB300, 32 query heads over 8 kv heads of 128 numbers unless said:
//   one sequence of 300 tokens, capped                                    10.1 us
//   64 sequences, window of 1,000 tokens, capped: 260 MB                  50.4 us (5.2 TB/s; about 4 us
//     to start and 5 at the end, where the last pieces are merged and ranges end unevenly)
//   8 sequences to 128 K tokens, 64 query heads, with a bias: 2.66 GB    387 us (6.9 TB/s)
//   33 sequences of packed documents, 7 new tokens, 32 kv heads, 8-bit: 77 MB  27.6 us (2.8 TB/s)
//   64 sequences of 4,096 tokens, 64 query heads: bf16 165 us (6.5 TB/s), 8-bit 104 us (5.1 TB/s)
//   one sequence of 65,536 tokens, 4 kv heads: 134 MB                     42 us
// Tried: one CTA per unit and chunk of tokens (9.6 / 59 / 433 / 38 us for the first four), a range per
// warp instead of per CTA (15 / 54 / 414 / 38); all pieces of a unit merged by one warp (137 us for
// the last).  The cap costs one ex2 and one reciprocal per
// score (capped_tanh), the bias one add and one multiply; both are template flags, so a plain
// mask pays for neither.  Every wait is bounded (WAIT_LIMIT_NS); a warp whose wait runs out sets
// KV_DEVERR_TIMEOUT and leaves, and the producer waits for its copies in flight.
#pragma once

#include "decode_common.cuh"
#include "prefix_groups.cuh"
#include "tcgen05.cuh"

namespace kvp {

// tanh(u) from y = 2 log2(e) u: 1 - 2 / (1 + 2^y), absolute error of a few 2^-24, and its Taylor
// series where |u| < 1/4, so that the relative error stays below 2^-20 and a large cap loses
// nothing of small scores (the hardware's tanh instruction is off by 2^-11).
__device__ __forceinline__ float capped_tanh(float y)
{
    const float u = y * 0.34657359027997264f;
    const float u2 = u * u;
    const float series = u + u * u2 * (-1.f / 3.f + u2 * (2.f / 15.f + u2 * (-17.f / 315.f)));
    const float full = 1.f - __fdividef(2.f, 1.f + fast_exp2(y));
    return u2 < 0.0625f ? series : full;
}

// The rule of the rows of a thread's accumulator columns, positions absolute.
template <int NTT, int RULE>
struct SpanRows {
    static constexpr bool CAP = RULE == SPAN_CAP || RULE == SPAN_CAP_BIAS;
    static constexpr bool BIAS = RULE == SPAN_BIAS || RULE == SPAN_CAP_BIAS;
    int lo[NTT][2], hi[NTT][2];       // keys [lo, hi)
    float slope[NTT][2];              // log2 units per token of distance
    int pos[NTT][2];
    float sl2, cap_in, cap_log2;      // tanh argument: score * sl2 * cap_in = 2 log2(e) x / cap
    int tile_lo, tile_hi;             // keys that some row of the tile sees
    int base;                         // position of the block's first token
    __device__ __forceinline__ float logit(float s, int tok, int nt, int j) const
    {
        const int t = base + tok;
        float x = s * sl2;
        if constexpr (CAP) x = cap_log2 * capped_tanh(x * cap_in);
        if constexpr (BIAS) x -= slope[nt][j] * static_cast<float>(abs(pos[nt][j] - t));
        return t >= lo[nt][j] && t < hi[nt][j] ? x : -INFINITY;
    }
    __device__ __forceinline__ int value_lo() const { return tile_lo - base; }
    __device__ __forceinline__ int value_hi() const { return tile_hi - base; }
};

constexpr int SPAN_TOK = 16;          // tokens of a sub-block

// The keys of one sequence.
template <int RULE>
struct SpanSeq {
    int ctx, first, visible, group;   // group: whose shared pass holds the keys before first, or -1
    // g: the group that holds the sequence (-1: none), its members and shared blocks (SPAN_SUFFIX)
    __device__ __forceinline__ void load(const SpanParams& sp, int b, bool flag, int g = -1, int members = 0, int blocks = 0)
    {
        const DecodeParams& p = sp.d;
        // (not through L1: the suffix kernel may start before the shared pass has completed)
        ctx = __ldcg(p.ctx + b);
        first = visible = 0;
        group = -1;
        if constexpr (RULE == SPAN_SUFFIX) {
            if (g >= 0 && prefix_shares(sp.shared, members, blocks)) {
                first = blocks * sp.block_size;
                group = g;
            }
        } else {
            if (sp.first_keys != nullptr) first = max(0, __ldg(sp.first_keys + b));
            if (sp.prefix_lens != nullptr) visible = __ldg(sp.prefix_lens + b);
        }
        const int cap = p.max_blocks * sp.block_size;
        if (ctx < 0 || ctx > cap || (ctx > 0 && ctx < p.q_len)) {
            // out of range (clamped), or fewer cached tokens than new queries (kept: the queries
            // at negative positions see nothing but the visible prefix)
            if (flag) atomicOr(p.err, KV_DEVERR_CONTEXT);
            ctx = ctx < 0 ? 0 : (ctx > cap ? cap : ctx);
        }
        visible = min(visible, ctx);
    }
    // keys of query token i: both ends grow with i
    __device__ __forceinline__ int key_lo(const SpanParams& sp, int i) const
    {
        if (RULE == SPAN_SUFFIX || sp.window <= 0) return first;
        return max(first, ctx - sp.d.q_len + i - sp.window + 1);
    }
    __device__ __forceinline__ int key_hi(const SpanParams& sp, int i) const
    {
        return max(ctx - sp.d.q_len + i + 1, visible);
    }
    // keys that some row of tile hg sees; the tile's tokens are a run, or all of them where it
    // spans two heads
    __device__ __forceinline__ void tile_keys(const SpanParams& sp, int hg, int nt, int& lo, int& hi) const
    {
        const DecodeParams& p = sp.d;
        const int i0 = (hg * nt) % p.q_len;
        const int nh = min(nt, p.rows - hg * nt);
        const bool wraps = i0 + nh > p.q_len;
        lo = key_lo(sp, wraps ? 0 : i0);
        hi = key_hi(sp, wraps ? p.q_len - 1 : i0 + nh - 1);
    }
    // its sub-blocks: [sub, sub + return value)
    __device__ __forceinline__ int tile_subs(const SpanParams& sp, int hg, int nt, int& sub) const
    {
        int lo, hi;
        tile_keys(sp, hg, nt, lo, hi);
        sub = lo / SPAN_TOK;
        return hi > lo ? (hi + SPAN_TOK - 1) / SPAN_TOK - sub : 0;
    }
};

// A CTA's range of positions [lo, hi), and where it begins.
template <int RULE>
struct SpanRange {
    long long lo, hi;
    long long base;                   // position of sequence b0's first unit
    int b0;
    int per;                          // positions of one of its groups of kv heads
    SpanSeq<RULE> seq;
    int g;                            // SPAN_SUFFIX: the group that holds b0, or the next one (the
                                      // number of groups: none); -1: nothing is shared
};

// Group of sequence b among n groups whose offsets are in order: -1 outside all of them.
__device__ __forceinline__ int find_group(const int* off, int n, int b)
{
    if (n == 0 || b < off[0] || b >= off[n]) return -1;
    int lo = 0, hi = n;                                 // off[lo] <= b < off[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        (off[mid] <= b ? lo : hi) = mid;
    }
    return lo;
}

// A run of sub-blocks of one unit.
template <int RULE>
struct SpanItem {
    SpanSeq<RULE> seq;
    int b, kg, hg;                    // sequence, group of kv heads, row tile; b -1: no more items
    int sub0, n;                      // sub-blocks [sub0, sub0 + n) of the sequence
    int split, nsplit;                // which of the unit's pieces this is
    int range0;                       // range of its first piece
};

// Walks the units of a CTA's range.
template <int RULE, int NT, int HC>
struct SpanWalk {
    SpanSeq<RULE> seq;
    long long lo, hi, total, at;      // at: position of the current unit
    int b, kg, hg, ranges;
    int g, g_end;                     // SPAN_SUFFIX: group of b, or the next one; first sequence behind it
    bool pending;                     // the sequence of the next unit is not loaded yet

    __device__ __forceinline__ void load_seq(const SpanParams& sp)
    {
        if constexpr (RULE == SPAN_SUFFIX) {
            const PrefixParams& s = sp.shared;
            if (g >= 0) {
                while (g < s.n_groups && g_end <= b) {
                    ++g;
                    if (g < s.n_groups) g_end = __ldcg(s.group_offsets + g + 1);
                }
                if (g < s.n_groups) {
                    const int start = __ldcg(s.group_offsets + g), blocks = __ldcg(s.group_blocks + g);
                    if (start <= b) {
                        seq.load(sp, b, false, g, g_end - start, blocks);
                        return;
                    }
                }
            }
        }
        seq.load(sp, b, false);
    }

    __device__ __forceinline__ void init(const SpanParams& sp, const SpanRange<RULE>& r, long long all, int n_ranges)
    {
        lo = r.lo;
        hi = r.hi;
        total = all;
        ranges = n_ranges;
        at = hi;                      // an empty range has no base and no first sequence
        b = kg = hg = 0;
        pending = false;
        if (lo >= hi) return;
        at = r.base;
        b = r.b0;
        g = r.g;
        g_end = RULE == SPAN_SUFFIX && g >= 0 && g < sp.shared.n_groups ? __ldcg(sp.shared.group_offsets + g + 1) : 0;
        seq = r.seq;
        // whole groups of kv heads before the range
        kg = static_cast<int>(div_small(lo - at, r.per));
        at += static_cast<long long>(kg) * r.per;
    }
    __device__ __forceinline__ int range_of(long long pos) const
    {
        return static_cast<int>(div_small((pos + 1) * ranges - 1, total));
    }
    __device__ __forceinline__ bool next(const SpanParams& sp, SpanItem<RULE>& it)
    {
        while (at < hi) {
            if (pending) {
                load_seq(sp);
                pending = false;
            }
            int sub;
            const int n = seq.tile_subs(sp, hg, NT, sub);
            const long long first = at + SPAN_PAD, end = first + n;
            const long long a = max(lo, first), z = min(hi, end);
            const bool mine = n > 0 ? a < z : at >= lo;
            if (mine) {
                it.seq = seq;
                it.b = b;
                it.kg = kg;
                it.hg = hg;
                it.split = 0;
                it.nsplit = 1;
                it.range0 = static_cast<int>(blockIdx.x);
                it.sub0 = sub;
                it.n = n;
                if (n > 0 && (first < lo || end > hi)) {
                    it.range0 = range_of(first);
                    it.nsplit = range_of(end - 1) - it.range0 + 1;
                    it.split = static_cast<int>(blockIdx.x) - it.range0;
                    it.sub0 = sub + static_cast<int>(a - first);
                    it.n = static_cast<int>(z - a);
                }
            }
            at = end;
            if (++hg == sp.d.head_groups) {
                hg = 0;
                if (++kg == sp.d.kv_heads / HC) {
                    kg = 0;
                    ++b;
                    pending = true;
                }
            }
            if (mine) return true;
        }
        return false;
    }
};

__device__ __forceinline__ int ticket_add(int* ticket)
{
    int old;
    asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], 1;" : "=r"(old) : "l"(ticket) : "memory");
    return old;
}

// The queries' MMA operand (load_q_frags) from rows in shared memory.  An 8-bit cache takes 32
// consecutive numbers of a row per thread: four vector loads instead of load_q_frags' 32 scalars.
template <bool FP8, int D, int NT>
__device__ __forceinline__ float load_q_staged(uint32_t (&qf)[D / 16][NT / 8][2], const uint8_t* rows, int nh, int lane,
                                               float scale_log2, const float* k_scale, int kvh)
{
    if constexpr (!FP8) {
        return load_q_frags<FP8, D, SPAN_TOK, NT>(qf, reinterpret_cast<const uint16_t*>(rows), nh, lane, scale_log2, k_scale, kvh);
    } else {
        // as in load_q_frags: a power-of-two scale keeps max|q| below 2^15, undone in the factor
        uint32_t x[NT / 8][16];
        uint32_t big = 0;
#pragma unroll
        for (int nt = 0; nt < NT / 8; ++nt) {
            const int hl = nt * 8 + (lane >> 2);
            const uint32_t at = smem_u32(rows) + hl * (D * 2) + (lane & 3) * 64;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint4 v = hl < nh ? lds128(at + i * 16) : make_uint4(0u, 0u, 0u, 0u);
                x[nt][4 * i] = v.x, x[nt][4 * i + 1] = v.y, x[nt][4 * i + 2] = v.z, x[nt][4 * i + 3] = v.w;
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) big = max(big, max((x[nt][i] & 0x7fffu) << 16, x[nt][i] & 0x7fff0000u));
        }
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) big = max(big, __shfl_xor_sync(FULL_MASK, big, o));
        const int shift = max(0, static_cast<int>(big >> 23) - 126 - 15);
        const float down = __uint_as_float(static_cast<uint32_t>(127 - shift) << 23);
        const float up = __uint_as_float(static_cast<uint32_t>(127 + shift) << 23);
#pragma unroll
        for (int nt = 0; nt < NT / 8; ++nt)
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const uint32_t v = x[nt][2 * ks + e];
                    qf[ks][nt][e] = pack_f16x2(__uint_as_float(v << 16) * down, __uint_as_float(v & 0xffff0000u) * down);
                }
        return scale_log2 * up * __ldg(k_scale + kvh);
    }
}

// Kinds of a stage, in the low bits of its tag.
constexpr int TAG_SKIP = 0;           // a sub-block of an invalid block: nothing landed
constexpr int TAG_KV = 1;             // a sub-block
constexpr int TAG_Q = 2;              // the unit's query rows
constexpr int TAG_PIECE = 3;          // rows [a, b) of a piece: a, b in bits 8 .., 16 ..; the heads that
constexpr int TAG_LAST = 4;           // have it in bits 24 ..
                                      // LAST: the unit ends with this stage

// Rows of a tile whose pieces lie next to each other: at most three segments, cut where the group's
// rows pass into another row tile of the shared pass and at the rows a stage holds.
template <int NT, int RPS>
struct PieceRows {
    int row0, nh;                     // the tile's first row in its group, its rows
    __device__ __forceinline__ int end(int a) const
    {
        return min(nh, min(a + RPS, PFX_TILE - (row0 + a) % PFX_TILE + a));
    }
};

// Another state's 8-row tile nt -- its rows' (max, sum) pairs a, b and its accumulators x(ms) --
// folded into st.
template <class C, class X>
__device__ __forceinline__ void fold_state(WarpState<C>& st, int nt, float2 a, float2 b, const X& x)
{
    float f[2], g[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const float2 w = j == 0 ? a : b;
        const float m = w.y > 0.f ? fmaxf(st.m[nt][j], w.x) : st.m[nt][j];
        f[j] = m > -INFINITY ? fast_exp2(st.m[nt][j] - m) : 1.f;
        g[j] = w.y > 0.f ? fast_exp2(w.x - m) : 0.f;
        st.m[nt][j] = m;
        st.l[nt][j] = st.l[nt][j] * f[j] + g[j] * w.y;
    }
#pragma unroll
    for (int ms = 0; ms < C::KS; ++ms) {
        const float4 y = x(ms);
        st.o[ms][nt][0] = st.o[ms][nt][0] * f[0] + y.x * g[0];
        st.o[ms][nt][1] = st.o[ms][nt][1] * f[1] + y.y * g[1];
        st.o[ms][nt][2] = st.o[ms][nt][2] * f[0] + y.z * g[0];
        st.o[ms][nt][3] = st.o[ms][nt][3] * f[1] + y.w * g[1];
    }
}

// Rows [a, b) of a piece -- normalised outputs o [row][D] and log-sum-exps (log2 units, 4 floats
// apart; -inf: the row saw nothing) in shared memory -- folded into the state as one more block.
template <bool FP8, int D, int NT>
__device__ __forceinline__ void fold_piece(const float* o, const float* lse, int a, int b,
                                           WarpState<DecodeCfg<FP8, D, SPAN_TOK, NT>>& st, int lane)
{
    using C = DecodeCfg<FP8, D, SPAN_TOK, NT>;
    const int r = lane >> 2;
#pragma unroll
    for (int nt = 0; nt < C::NTT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int row = nt * 8 + 2 * (lane & 3) + j;
            if (row < a || row >= b) continue;
            const float s = lse[(row - a) * 4];
            if (!(s > -INFINITY)) continue;
            const float m = fmaxf(st.m[nt][j], s);
            const float f = fast_exp2(st.m[nt][j] - m), w = fast_exp2(s - m);
            st.m[nt][j] = m;
            st.l[nt][j] = st.l[nt][j] * f + (r == 0 ? w : 0.f);     // the lanes' sums are added up at the end
            const float* x = o + (row - a) * D + (FP8 ? 16 * r : r);
#pragma unroll
            for (int ms = 0; ms < C::KS; ++ms)
#pragma unroll
                for (int hi = 0; hi < 2; ++hi) {
                    float& y = st.o[ms][nt][2 * hi + j];
                    y = y * f + w * x[FP8 ? 2 * ms + hi : 16 * ms + 8 * hi];
                }
        }
}

// Whether a warp takes two sub-blocks at a time: an 8-bit cache's 16 tokens are too little work between
// two waits, and the two tiles are independent.  One / two: 64 sequences of 4,096 tokens 111 / 104 us,
// packed documents 28.8 / 27.6; behind a shared prefix, whose own parts are short, 81 / 84.  (With
// bf16 the loads are what a warp waits for, and 16-row tiles lack the registers.)
template <bool FP8, int NT, int HC, int RULE>
constexpr bool span_pairs() { return FP8 && NT == 8 && HC == 4 && RULE != SPAN_SUFFIX; }

template <bool FP8, int D, int NT, int HC>
struct SpanCfg : DecodeCfg<FP8, D, SPAN_TOK, NT> {
    using C = DecodeCfg<FP8, D, SPAN_TOK, NT>;
    static constexpr int NCW = 4;                   // consumer warps
    static constexpr int WPH = NCW / HC;            // of one kv head
    static constexpr int THREADS = (NCW + 1) * 32;
    static constexpr int MINB = SPAN_CTAS;          // CTAs per SM
    static constexpr int HSTAGE = HC * C::STAGE;    // K tiles of the heads, then V tiles; or the query
                                                    // rows of the heads; or a piece's rows of each head
    static constexpr int RPS = C::STAGE / (D * 4) < NT ? C::STAGE / (D * 4) : NT;   // rows of a piece stage
    static constexpr int LSE = HC * RPS * 16;       // and their log-sum-exps, 16 bytes a row
    static constexpr int CTL = 2048;                // barriers, items
    static constexpr int REGS4 = C::KS * C::NTT;    // groups of four accumulators of a thread
    static constexpr int HAND = WPH > 1 ? (NCW - HC) * (REGS4 * 16 + C::NTT * 16) * 32 : 0;   // states handed over
    static constexpr int BUDGET = 228 * 1024 / MINB - 1024 /* reserved */ - 1024 /* alignment */ - CTL - HAND;
    static constexpr int NST = BUDGET / (HSTAGE + LSE) < 16 ? BUDGET / (HSTAGE + LSE) : 16;
    static constexpr int SMEM = 1024 + NST * (HSTAGE + LSE) + HAND + CTL;
    static constexpr int QUEUE = 8;                 // items handed on ahead
    // More pieces of a unit than this are merged in two levels, by groups of at least MERGE_LEAST: 48
    // pieces (one sequence of 4,096 tokens, 4 kv heads) 25.8 us in one level, 16.4 in two, 300 pieces
    // (65,536 tokens) 137 and 42; limits of 6, 12 and 20 give the same times, a few pieces are
    // merged soonest without a second ticket.
    static constexpr int MERGE_ONE = 12, MERGE_LEAST = 3;
    static_assert(NST >= 3 && SMEM <= 227 * 1024, "a ring of three stages at least");
};

template <bool FP8, int D, int NT, int HC, int RULE>
__global__ void __launch_bounds__(SpanCfg<FP8, D, NT, HC>::THREADS, SpanCfg<FP8, D, NT, HC>::MINB)
paged_decode_span(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
                  const SpanParams sp)
{
    using C = DecodeCfg<FP8, D, SPAN_TOK, NT>;
    using S = SpanCfg<FP8, D, NT, HC>;
    constexpr int NST = S::NST, THREADS = S::THREADS, NCW = S::NCW, WPH = S::WPH, QUEUE = S::QUEUE;
    constexpr bool SUFFIX = RULE == SPAN_SUFFIX;
    const DecodeParams& p = sp.d;
    struct Ctl {
        uint64_t full[NST], empty[NST];
        uint64_t item_full[QUEUE], item_empty[QUEUE];
        uint64_t hand_full[HC], hand_free[HC];       // a head's states handed over, read
        SpanRange<RULE> range;
        long long scan[THREADS / 32];
        int tag[NST];                                // what the stage holds
        SpanItem<RULE> queue[QUEUE];
    };
    static_assert(sizeof(Ctl) <= S::CTL, "control block");
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint8_t* lse_sm = smem + NST * S::HSTAGE;
    uint8_t* hand_sm = lse_sm + NST * S::LSE;
    Ctl* ctl = reinterpret_cast<Ctl*>(hand_sm + S::HAND);

    const int tid = threadIdx.x;
    const int warp = tid >> 5;
    const int lane = tid & 31;
    const int r = lane >> 2, c = lane & 3;           // accumulator row and column pair of the lane

    if (tid == 0) {
        for (int i = 0; i < NST; ++i) {
            mbar_init(smem_u32(&ctl->full[i]), 1);
            mbar_init(smem_u32(&ctl->empty[i]), NCW);
        }
        for (int i = 0; i < QUEUE; ++i) {
            mbar_init(smem_u32(&ctl->item_full[i]), 1);
            mbar_init(smem_u32(&ctl->item_empty[i]), NCW);
        }
        for (int i = 0; i < HC; ++i) {
            mbar_init(smem_u32(&ctl->hand_full[i]), WPH > 1 ? WPH - 1 : 1);
            mbar_init(smem_u32(&ctl->hand_free[i]), 1);
        }
        fence_mbar_init();
        prefetch_tensormap(&tmk);
        prefetch_tensormap(&tmv);
    }
    // Inputs of the preceding kernel are ready.  The suffix form's preceding kernel is the shared
    // pass, which has waited for the kernels before it when it lets this one launch: only the pieces
    // it leaves are waited for, before the first is read (and before this CTA ends).
    if (!SUFFIX) grid_dependency_wait();
    grid_dependents_launch();                        // this grid is resident: the next may launch

    // ---- the groups (suffix form), in the ring's memory until the loads begin
    const int* off = sp.shared.group_offsets;
    const int* blocks = sp.shared.group_blocks;
    bool grouped = false;                            // the offsets are in order
    if constexpr (SUFFIX) {
        const int n = sp.shared.n_groups;
        int* mine = reinterpret_cast<int*>(smem);
        const bool fits = (2 * static_cast<size_t>(n) + 1) * 4 <= static_cast<size_t>(NST) * S::HSTAGE;
        bool ok = true;
        for (int g = tid; g <= n; g += THREADS) {
            const int a = __ldcg(off + g);
            if (fits) mine[g] = a;
            if (g < n) {
                const int e = __ldcg(off + g + 1);
                ok = ok && 0 <= a && a <= e && e <= p.batch;
                if (fits) mine[n + 1 + g] = __ldcg(blocks + g);
            }
        }
        grouped = __syncthreads_and(ok);             // bad offsets: nothing is shared
        if (fits) {
            off = mine;
            blocks = mine + n + 1;
        }
    }

    // ---- this CTA's range: the positions of all sequences, then the one it begins in.  A round
    // takes one sequence per thread; more than THREADS of them are gone through twice.
    long long total = 0;
    int ranges;
    {
        SpanSeq<RULE> mine;                          // the thread's sequence of the round
        const auto positions = [&](int b) {          // of one of its groups of kv heads
            int w = 0;
            if (b < p.batch) {
                const int g = SUFFIX && grouped ? find_group(off, sp.shared.n_groups, b) : -1;
                if (SUFFIX && g >= 0)
                    mine.load(sp, b, blockIdx.x == 0, g, off[g + 1] - off[g], blocks[g]);
                else
                    mine.load(sp, b, blockIdx.x == 0);
                int sub;
                for (int t = 0; t < p.head_groups; ++t) w += mine.tile_subs(sp, t, NT, sub) + SPAN_PAD;
            }
            return w;
        };
        const int kgs = p.kv_heads / HC;
        int per = positions(tid);
        const auto scan = [&](long long x) {         // inclusive, in the warp; the warps' sums in ctl
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long y = __shfl_up_sync(FULL_MASK, x, o);
                if (lane >= o) x += y;
            }
            if (lane == 31) ctl->scan[warp] = x;
            return x;
        };
        // the whole batch's positions; where it is more than one round, the rounds are summed first
        const bool one = p.batch <= THREADS;
        long long x = static_cast<long long>(per) * kgs;
        if (!one)
            for (int b = tid + THREADS; b < p.batch; b += THREADS) x += static_cast<long long>(positions(b)) * kgs;
        x = scan(x);
        __syncthreads();
#pragma unroll
        for (int v = 0; v < THREADS / 32; ++v) total += ctl->scan[v];
        const long long most = div_small(total + sp.least - 1, sp.least);       // ranges of `least` positions or more
        ranges = most < gridDim.x ? static_cast<int>(most) : static_cast<int>(gridDim.x);
        const int k = blockIdx.x;
        const long long lo = k < ranges ? div_small(total * k, ranges) : total;
        const long long hi = k < ranges ? div_small(total * (k + 1), ranges) : total;
        long long before = 0;
        for (int b0 = 0; lo < hi && b0 < p.batch && before <= lo; b0 += THREADS) {
            if (!one) {
                per = positions(b0 + tid);
                __syncthreads();                     // the sums before this round are read
                x = scan(static_cast<long long>(per) * kgs);
                __syncthreads();
            }
            const long long w = static_cast<long long>(per) * kgs;
            long long base = before + x - w;
#pragma unroll
            for (int v = 0; v < THREADS / 32; ++v) {
                if (v < warp) base += ctl->scan[v];
                before += ctl->scan[v];
            }
            if (base <= lo && lo < base + w) {
                ctl->range.base = base;
                ctl->range.b0 = b0 + tid;
                ctl->range.per = per;
                ctl->range.seq = mine;
                if (SUFFIX) {
                    const int g = find_group(off, grouped ? sp.shared.n_groups : 0, b0 + tid);
                    ctl->range.g = !grouped ? -1 : g >= 0 ? g : b0 + tid < off[0] ? 0 : sp.shared.n_groups;
                }
            }
        }
        if (tid == 0) {
            ctl->range.lo = lo;
            ctl->range.hi = hi;
        }
        if (SUFFIX) fence_proxy_async_smem();        // the ring's memory goes to the copies
        __syncthreads();
    }

    // ------------------------------------------------------------ producer warp
    if (warp == NCW) {
        SpanWalk<RULE, NT, HC> walk;
        walk.init(sp, ctl->range, total, ranges);
        const int per_block = sp.block_size / SPAN_TOK;                 // 1 or 2
        // lane 0 loads the K tiles of the heads, lane 1 the V tiles
        const CUtensorMap* my_map = lane == 0 ? &tmk : &tmv;
        const uint32_t my_off = lane == 0 ? 0u : static_cast<uint32_t>(HC * C::TILE);
        int ids = -1, ids_b = -1, ids_at = 0;        // table entries ids_at .. ids_at + 31 of sequence ids_b
        int n = 0;                                   // stages issued
        bool ok = true;
        for (int k = 0; ok; ++k) {
            SpanItem<RULE> it;
            const bool more = walk.next(sp, it);
            if (!more) it.b = -1;
            const int slot = k % QUEUE;
            ok = all_ok(mbar_wait_bounded(smem_u32(&ctl->item_empty[slot]), (static_cast<uint32_t>(k / QUEUE) & 1u) ^ 1u));
            if (!ok) break;
            if (lane == 0) {
                ctl->queue[slot] = it;
                mbar_arrive(smem_u32(&ctl->item_full[slot]));
            }
            __syncwarp();
            if (!more) break;
            // arms the next stage (tag, bytes to land); false: no more stages
            const auto arm = [&](int tag, uint32_t bytes) {
                if (n == p.stop_stage) return false; // test hook: the rest never lands
                const int st = n % NST;
                if (!all_ok(mbar_wait_bounded(smem_u32(&ctl->empty[st]), (static_cast<uint32_t>(n / NST) & 1u) ^ 1u)))
                    return false;
                if (lane == 0) {
                    ctl->tag[st] = tag;
                    if (bytes > 0)
                        mbar_arrive_expect_tx(smem_u32(&ctl->full[st]), bytes);
                    else
                        mbar_arrive(smem_u32(&ctl->full[st]));
                }
                __syncwarp();                        // armed before any of the stage's bytes can land
                return true;
            };
            const auto stage = [&]() { return smem_u32(smem + n % NST * S::HSTAGE); };
            const auto bar = [&]() { return smem_u32(&ctl->full[n % NST]); };

            // the shared pass's pieces of the unit's rows: per segment, lane h of the first HC holds
            // the first piece and the count of head h; the unit's first CTA takes them
            constexpr int SEGS = 3;
            const int nh = min(NT, p.rows - it.hg * NT);
            PieceRows<NT, S::RPS> pr{0, 0};
            int2 run[SEGS];
            int pieces = 0;                          // stages of pieces
            const auto count = [&](int g) {          // stages of segment g: the most any head has
                int y = run[g].y;
#pragma unroll
                for (int o = HC / 2; o >= 1; o >>= 1) y = max(y, __shfl_xor_sync(FULL_MASK, y, o));
                return __shfl_sync(FULL_MASK, y, 0);
            };
            // Looked up as late as the last sub-block, which has to say whether pieces follow: the loads
            // before it need not wait for the shared pass.
            const auto count_pieces = [&]() {
                if (!SUFFIX || it.seq.group < 0 || it.split != 0) return;
                grid_dependency_wait();              // the pieces of the shared pass are there
                const PrefixGroup gr = load_prefix_group(sp.shared, it.seq.group);
                const int pairs = prefix_pairs(sp.shared, gr);
                const int base = prefix_run_base(sp.shared, it.seq.group, gr);
                pr = PieceRows<NT, S::RPS>{(it.b - gr.off) * p.rows + it.hg * NT, nh};
                int a = 0;
#pragma unroll
                for (int g = 0; g < SEGS; ++g) {
                    run[g] = make_int2(0, 0);
                    if (a < nh && lane < HC) {
                        run[g] = __ldcg(sp.shared.runs + base + (it.kg * HC + lane) * pairs + (pr.row0 + a) / PFX_PAIR);
                        // (a shared pass that gave up may have left this run's entry unwritten)
                        if (run[g].x < 0 || run[g].y < 0 || run[g].x > sp.shared.pieces - run[g].y) run[g].y = 0;
                    }
                    if (a < nh) a = pr.end(a);
                }
#pragma unroll
                for (int g = 0; g < SEGS; ++g) pieces += count(g);
            };

            // ---- the query rows
            if (it.n == 0) count_pieces();
            ok = arm(TAG_Q | (it.n == 0 && pieces == 0 ? TAG_LAST : 0), static_cast<uint32_t>(HC * nh * D * 2));
            if (!ok) break;
            if (lane < HC) {
                const size_t row = (static_cast<size_t>(it.b) * p.kv_heads + it.kg * HC + lane) * p.rows + it.hg * NT;
                bulk_load(stage() + lane * (NT * D * 2), p.q + row * D, static_cast<uint32_t>(nh * D * 2), bar());
            }
            ++n;
            // ---- the sub-blocks
            for (int i = 0; i < it.n; ++i) {
                const int sub = it.sub0 + i;
                const int entry = per_block == 2 ? sub >> 1 : sub;
                if (ids_b != it.b || entry < ids_at || entry >= ids_at + 32) {
                    ids_b = it.b;
                    ids_at = entry;
                    const int j = entry + lane;
                    ids = j < p.max_blocks ? __ldcg(p.tables + static_cast<size_t>(it.b) * p.max_blocks + j) : -1;
                }
                const int blk = __shfl_sync(FULL_MASK, ids, entry - ids_at);
                const bool good = blk >= 0 && blk < p.num_blocks;
                if (!good && lane == 0) atomicOr(p.err, KV_DEVERR_BLOCK_ID);    // skipped: never addressed
                if (i + 1 == it.n) count_pieces();
                ok = arm((good ? TAG_KV : TAG_SKIP) | (i + 1 == it.n && pieces == 0 ? TAG_LAST : 0),
                         good ? static_cast<uint32_t>(S::HSTAGE) : 0u);
                if (!ok) break;
                if (good && lane < 2)
                    tma_load_5d(stage() + my_off, my_map, 0, 0, per_block == 2 ? (sub & 1) * SPAN_TOK : 0,
                                it.kg * HC, blk, bar());
                ++n;
            }
            if (!ok || pieces == 0) continue;
            // ---- the pieces
            int a = 0, done = 0;
#pragma unroll
            for (int g = 0; g < SEGS; ++g) {
                if (a >= nh || !ok) continue;
                const int e1 = pr.end(a), most = count(g);
                const int slot_rows = (pr.row0 + a) % PFX_PAIR;
                for (int e = 0; e < most; ++e) {
                    const uint32_t have = __ballot_sync(FULL_MASK, lane < HC && e < run[g].y);
                    const uint32_t rows = static_cast<uint32_t>(e1 - a);
                    ok = arm(TAG_PIECE | (a << 8) | (e1 << 16) | static_cast<int>(have << 24) | (++done == pieces ? TAG_LAST : 0),
                             static_cast<uint32_t>(__popc(have)) * rows * (D * 4 + 16));
                    if (!ok) break;
                    if (have >> lane & 1u) {
                        const size_t at = static_cast<size_t>(run[g].x + e) * PFX_PAIR + slot_rows;
                        bulk_load(stage() + lane * C::STAGE, sp.shared.piece_o + at * D, rows * (D * 4), bar());
                        bulk_load(smem_u32(lse_sm + n % NST * S::LSE) + lane * (S::RPS * 16), sp.shared.piece_lse + at,
                                  rows * 16, bar());
                    }
                    ++n;
                }
                a = e1;
            }
        }
        if (!ok && lane == 0 && n != p.stop_stage) atomicOr(p.err, KV_DEVERR_TIMEOUT);
        if (SUFFIX) grid_dependency_wait();          // the grid ends behind the shared pass
        // Drain: the CTA must not exit while a copy into its shared memory is in flight.
        for (int i = max(0, n - NST); i < n; ++i)
            if (!mbar_wait_bounded(smem_u32(&ctl->full[i % NST]), static_cast<uint32_t>(i / NST) & 1u)) break;
        return;
    }

    // ------------------------------------------------------------ consumer warps
    const unsigned long long wait_ns = p.consumer_wait_ns ? p.consumer_wait_ns : WAIT_LIMIT_NS;
    const int h = warp / WPH;                        // head of the group
    int taken = 0;                                   // stages of the items before
    bool ok = true;
    for (int k = 0;; ++k) {
        ok = all_ok(mbar_wait_bounded(smem_u32(&ctl->item_full[k % QUEUE]), static_cast<uint32_t>(k / QUEUE) & 1u));
        if (!ok) break;
        const SpanItem<RULE> it = ctl->queue[k % QUEUE];
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&ctl->item_empty[k % QUEUE]));
        if (it.b < 0) break;
        const int b = it.b, kvh = it.kg * HC + h;
        const int nh = min(NT, p.rows - it.hg * NT);                    // real rows in this tile
        const size_t row0 = (static_cast<size_t>(b) * p.kv_heads + kvh) * p.rows + it.hg * NT;
        uint32_t qf[C::KS][C::NTT][2];
        SpanRows<C::NTT, RULE> rows;
        rows.cap_in = sp.cap_in;
        rows.cap_log2 = sp.cap_log2;
        it.seq.tile_keys(sp, it.hg, NT, rows.tile_lo, rows.tile_hi);
#pragma unroll
        for (int nt = 0; nt < C::NTT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int local = nt * 8 + 2 * c + j;
                const int rr = it.hg * NT + local;
                const int head = rr / p.q_len, i = rr - head * p.q_len;
                rows.lo[nt][j] = it.seq.key_lo(sp, i);
                rows.hi[nt][j] = local < nh ? it.seq.key_hi(sp, i) : 0;        // padding rows see nothing
                rows.pos[nt][j] = it.seq.ctx - p.q_len + i;
                rows.slope[nt][j] = rows.BIAS && local < nh
                                        ? __ldg(sp.slopes + kvh * p.group + head) * 1.4426950408889634f
                                        : 0.f;
            }
        WarpState<C> st;
        reset_state(st);
        // every warp waits for every stage in order, also for those that another warp of its head
        // folds: a wait by parity is only unambiguous for the next phase
        int sub = it.sub0, turn = 0;
        for (bool last = false; !last; ++taken) {
            const int s = taken % NST;
            ok = all_ok(mbar_wait_bounded(smem_u32(&ctl->full[s]), static_cast<uint32_t>(taken / NST) & 1u, wait_ns));
            if (!ok) break;
            const int tag = ctl->tag[s];
            const uint8_t* st_sm = smem + s * S::HSTAGE;
            last = tag & TAG_LAST;
            if ((tag & 3) == TAG_Q) {
                rows.sl2 = load_q_staged<FP8, D, NT>(qf, st_sm + h * (NT * D * 2), nh, lane, p.scale_log2, p.k_scale, kvh);
            } else {
                const bool mine = WPH == 1 || turn % WPH == warp % WPH;
                ++turn;
                if ((tag & 3) == TAG_KV && mine) {
                    const uint32_t tk = smem_u32(st_sm) + h * C::TILE;
                    rows.base = sub * SPAN_TOK;
                    if constexpr (span_pairs<FP8, NT, HC, RULE>()) {
                        static_assert(WPH == 1, "a warp takes every sub-block of its head");
                        // the next stage with this one, where it is the next sub-block
                        const int s2 = s + 1 == NST ? 0 : s + 1;
                        int tag2 = TAG_Q;
                        if (!last) {
                            ok = all_ok(mbar_wait_bounded(smem_u32(&ctl->full[s2]),
                                                          static_cast<uint32_t>((taken + 1) / NST) & 1u, wait_ns));
                            if (!ok) break;
                            tag2 = ctl->tag[s2];
                        }
                        if ((tag2 & 3) == TAG_KV) {
                            const uint32_t tk2 = smem_u32(smem + s2 * S::HSTAGE) + h * C::TILE;
                            constexpr uint32_t FIRST = C::TILE;         // (16 tokens of 128 bytes)
                            process_block_rows<FP8, D, 2 * SPAN_TOK, NT>(
                                BlockTiles(tk, tk2 - FIRST, tk + HC * C::TILE, tk2 + HC * C::TILE - FIRST), rows, qf, st, lane);
                            last = tag2 & TAG_LAST;
                            __syncwarp();
                            if (lane == 0) {
                                mbar_arrive(smem_u32(&ctl->empty[s]));
                                mbar_arrive(smem_u32(&ctl->empty[s2]));
                            }
                            sub += 2;
                            ++taken;
                            continue;
                        }
                    }
                    process_block_rows<FP8, D, SPAN_TOK, NT>(BlockTiles(tk, tk + HC * C::TILE), rows, qf, st, lane);
                }
                if (SUFFIX && (tag & 3) == TAG_PIECE && mine && (tag >> (24 + h) & 1))
                    fold_piece<FP8, D, NT>(reinterpret_cast<const float*>(st_sm + h * C::STAGE),
                                           reinterpret_cast<const float*>(lse_sm + s * S::LSE + h * (S::RPS * 16)),
                                           tag >> 8 & 0xff, tag >> 16 & 0xff, st, lane);
                ++sub;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&ctl->empty[s]));
        }
        if (!ok) break;

        // -------------------------------------------------------- the unit's end
        reduce_row_sums(st);
        if constexpr (WPH > 1) {
            // The head's other warps hand their states to the first, in the accumulators' layout.
            constexpr int STATE = (S::REGS4 + C::NTT) * 32;             // 16-byte vectors of a state
            const int w = warp % WPH;
            float4* state = reinterpret_cast<float4*>(hand_sm) + (h * (WPH - 1) + (w > 0 ? w - 1 : 0)) * STATE + lane;
            if (w > 0) {
                // (the states before have been read: hand_free has completed once per unit)
                ok = k == 0 || all_ok(mbar_wait_bounded(smem_u32(&ctl->hand_free[h]), static_cast<uint32_t>(k - 1) & 1u));
                if (!ok) break;
#pragma unroll
                for (int ms = 0; ms < C::KS; ++ms)
#pragma unroll
                    for (int nt = 0; nt < C::NTT; ++nt)
                        state[(ms * C::NTT + nt) * 32] =
                            make_float4(st.o[ms][nt][0], st.o[ms][nt][1], st.o[ms][nt][2], st.o[ms][nt][3]);
#pragma unroll
                for (int nt = 0; nt < C::NTT; ++nt)
                    state[(S::REGS4 + nt) * 32] = make_float4(st.m[nt][0], st.l[nt][0], st.m[nt][1], st.l[nt][1]);
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&ctl->hand_full[h]));
                continue;
            }
            ok = all_ok(mbar_wait_bounded(smem_u32(&ctl->hand_full[h]), static_cast<uint32_t>(k) & 1u));
            if (!ok) break;
#pragma unroll 1
            for (int e = 0; e < WPH - 1; ++e, state += STATE)
#pragma unroll
                for (int nt = 0; nt < C::NTT; ++nt) {
                    const float4 ml = state[(S::REGS4 + nt) * 32];
                    fold_state<C>(st, nt, make_float2(ml.x, ml.y), make_float2(ml.z, ml.w),
                                  [&](int ms) { return state[(ms * C::NTT + nt) * 32]; });
                }
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&ctl->hand_free[h]));
        }
        const int parts = it.nsplit;                 // CTAs that hold parts of these rows
        if (parts > 1) {
            // Piece e lies in range range0 + e.  A range holds one unit that goes on from the range
            // before and one that goes on into the next at most, which gives every piece and every
            // ticket its place by range.
            const auto slot = [&](int e) {
                return static_cast<size_t>(2 * (it.range0 + e) + (e == 0 ? 1 : 0)) * HC + h;
            };
            // Many pieces are merged in two levels: groups of about sqrt(parts) neighbours first, then
            // the groups.
            int size = parts;
            if (parts > S::MERGE_ONE)
                for (size = S::MERGE_LEAST; size * size < parts;) ++size;
            int e = it.split;                        // the piece this state stands for
            int first = e / size * size, step = 1, n = min(size, parts - first);
            bool top = size == parts, last = true;
            float2* ml = reinterpret_cast<float2*>(p.part_ml);
            for (;;) {
                const size_t own = slot(e);
                float4* mine = reinterpret_cast<float4*>(p.part_o) + own * (S::REGS4 * 32) + lane;
#pragma unroll
                for (int ms = 0; ms < C::KS; ++ms)
#pragma unroll
                    for (int nt = 0; nt < C::NTT; ++nt)
                        mine[(ms * C::NTT + nt) * 32] =
                            make_float4(st.o[ms][nt][0], st.o[ms][nt][1], st.o[ms][nt][2], st.o[ms][nt][3]);
                if (r == 0) {
#pragma unroll
                    for (int nt = 0; nt < C::NTT; ++nt)
#pragma unroll
                        for (int j = 0; j < 2; ++j)
                            ml[own * NT + nt * 8 + 2 * c + j] = make_float2(st.m[nt][j], st.l[nt][j]);
                }
                // One acquire-release add by lane 0: the other lanes' stores come before it
                // (__syncwarp), the loads of the last warp after it.
                __syncwarp();
                if (n > 1) {
                    if (lane == 0) {
                        int* ticket = p.tickets + ((top ? 0 : gridDim.x) + it.range0 + first) * HC + h;
                        last = ticket_add(ticket) == n - 1;
                        if (last) *ticket = 0;       // ready for the next call
                    }
                    last = __shfl_sync(FULL_MASK, last, 0);
                    if (!last) break;
                    __syncwarp();
                    // all pieces in order (this warp's own among them), so the bits do not depend
                    // on which warp is last
                    reset_state(st);
                    constexpr int UN = C::NTT == 1 ? 3 : 1;      // pieces in flight
#pragma unroll 1
                    for (int e0 = 0; e0 < n; e0 += UN) {
                        float2 v[UN][C::NTT][2];
                        float4 x[UN][C::KS][C::NTT];
#pragma unroll
                        for (int u = 0; u < UN; ++u) {
                            const size_t at = slot(first + min(e0 + u, n - 1) * step);
                            const float4* other = reinterpret_cast<const float4*>(p.part_o) + at * (S::REGS4 * 32) + lane;
#pragma unroll
                            for (int nt = 0; nt < C::NTT; ++nt) {
#pragma unroll
                                for (int j = 0; j < 2; ++j) v[u][nt][j] = __ldcg(ml + at * NT + nt * 8 + 2 * c + j);
#pragma unroll
                                for (int ms = 0; ms < C::KS; ++ms) x[u][ms][nt] = __ldcg(other + (ms * C::NTT + nt) * 32);
                            }
                        }
#pragma unroll
                        for (int u = 0; u < UN; ++u) {
                            if (e0 + u >= n) break;
#pragma unroll
                            for (int nt = 0; nt < C::NTT; ++nt)
                                fold_state<C>(st, nt, v[u][nt][0], v[u][nt][1], [&](int ms) { return x[u][ms][nt]; });
                        }
                    }
                }
                if (top) break;
                top = true;
                e = first;
                first = 0;
                step = size;
                n = (parts + size - 1) / size;
            }
            if (!last) continue;
        }
        // ---- normalise and store.  An 8-bit cache's values get their scale last: the sums of codes
        // times a large scale, or a small scale divided by the sum, could leave the range of fp32.
        const float vs = FP8 ? __ldg(p.v_scale + kvh) : 1.f;
#pragma unroll
        for (int nt = 0; nt < C::NTT; ++nt) {
            const float inv[2] = {st.l[nt][0] > 0.f ? 1.f / st.l[nt][0] : 0.f,
                                  st.l[nt][1] > 0.f ? 1.f / st.l[nt][1] : 0.f};
            const int mine = nt * 8 + 2 * c;         // the lane's two rows
            if constexpr (FP8) {
                // numbers 16 r .. 16 r + 15 of both rows
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    uint32_t w[8];
#pragma unroll
                    for (int ms = 0; ms < C::KS; ++ms)
                        w[ms] = pack_bf16x2(st.o[ms][nt][j] * inv[j] * vs, st.o[ms][nt][2 + j] * inv[j] * vs);
                    if (mine + j < nh) {
                        uint4* dst = reinterpret_cast<uint4*>(p.out + (row0 + mine + j) * D + 16 * r);
                        dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
                        dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
                    }
                }
            } else {
                // numbers 16 ms + r and 16 ms + r + 8 of both rows: lanes r and r ^ 1 exchange, so
                // that an even r holds a pair of the first row and an odd one of the second
                const int row = mine + (r & 1);
                uint32_t* dst = reinterpret_cast<uint32_t*>(p.out + (row0 + row) * D + (r & 6));
#pragma unroll
                for (int ms = 0; ms < C::KS; ++ms)
#pragma unroll
                    for (int hi = 0; hi < 2; ++hi) {
                        const float a = st.o[ms][nt][2 * hi] * inv[0], d = st.o[ms][nt][2 * hi + 1] * inv[1];
                        const float got = __shfl_xor_sync(FULL_MASK, r & 1 ? a : d, 4);
                        const uint32_t w = r & 1 ? pack_bf16x2(got, d) : pack_bf16x2(a, got);
                        if (row < nh) dst[ms * 8 + hi * 4] = w;
                    }
            }
            if (p.lse != nullptr && r == 0) {
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    if (mine + j < nh) p.lse[row0 + mine + j] = lse_from(st.m[nt][j], st.l[nt][j]);
            }
        }
    }
    if (!ok && lane == 0) atomicOr(p.err, KV_DEVERR_TIMEOUT);
}

template <bool FP8, int D, int NT, int HC>
cudaError_t prepare_span_variant()
{
    using S = SpanCfg<FP8, D, NT, HC>;
    const auto raise = [](auto kernel) {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM);
    };
    cudaError_t e = raise(paged_decode_span<FP8, D, NT, HC, SPAN_MASK>);
    if (e == cudaSuccess) e = raise(paged_decode_span<FP8, D, NT, HC, SPAN_CAP>);
    if (e == cudaSuccess) e = raise(paged_decode_span<FP8, D, NT, HC, SPAN_BIAS>);
    if (e == cudaSuccess) e = raise(paged_decode_span<FP8, D, NT, HC, SPAN_CAP_BIAS>);
    if (e == cudaSuccess) e = raise(paged_decode_span<FP8, D, NT, HC, SPAN_SUFFIX>);
    return e;
}

template <bool FP8, int D, int NT, int HC>
cudaError_t launch_span_variant(SpanRule rule, int ctas, const CUtensorMap& tk, const CUtensorMap& tv,
                                const SpanParams& p, cudaStream_t s)
{
    using S = SpanCfg<FP8, D, NT, HC>;
    const auto go = [&](auto kernel) {
        return launch_dependent(kernel, dim3(static_cast<unsigned>(ctas)), dim3(S::THREADS), S::SMEM, s, tk, tv, p);
    };
    switch (rule) {
    case SPAN_MASK: return go(paged_decode_span<FP8, D, NT, HC, SPAN_MASK>);
    case SPAN_CAP: return go(paged_decode_span<FP8, D, NT, HC, SPAN_CAP>);
    case SPAN_BIAS: return go(paged_decode_span<FP8, D, NT, HC, SPAN_BIAS>);
    case SPAN_CAP_BIAS: return go(paged_decode_span<FP8, D, NT, HC, SPAN_CAP_BIAS>);
    case SPAN_SUFFIX: return go(paged_decode_span<FP8, D, NT, HC, SPAN_SUFFIX>);
    }
    return cudaErrorInvalidValue;
}

}  // namespace kvp
