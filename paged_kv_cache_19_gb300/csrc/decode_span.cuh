// decode_span.cuh -- paged attention over a span of each sequence's keys: every query row sees
// one contiguous interval of token positions, and only the blocks that the rows of a tile see
// are read.
//
// For query token i of a sequence (position p = ctx - q_len + i) and query head h:
//   keys   max(first, p - window + 1) <= t < max(p + 1, min(prefix, ctx))
//   score  x = scale q . K[t];  x <- cap tanh(x / cap);  x <- x - slope_h |p - t|
//   out = softmax over those keys of x, times V;  a row that sees no key gives 0 and lse = -inf
// (the sliding window, the cap, the distance bias, the document start and the visible prefix
// are each optional).  It is the decode kernel's structure (decode_kernel.cuh: one producer
// warp, a ring of TMA stages, four consumer warps, chunks merged by the last CTA of a unit)
// with two differences: a tile of query rows starts at the first block that one of its rows
// sees -- chunk j covers blocks [first + j S, first + (j + 1) S) -- and the rule of a row
// (SpanRows) is applied to the raw scores before the softmax.
//
// The suffix form (SPAN_SUFFIX, paged_shared_prefix_attention) starts a sequence's keys behind
// the blocks that its group shares and takes the pieces that the shared pass left for its rows
// (prefix_groups.cuh) as further chunks of the merge.
//
// It stays bound by the K/V bytes of the visible blocks.  The cap costs one ex2 and one
// reciprocal per score (capped_tanh), the bias one add and one multiply; both are template
// flags, so a plain mask pays for neither.
#pragma once

#include "decode_common.cuh"
#include "prefix_groups.cuh"

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

// The pieces of a shared pass that hold query row `r` (of the `rows` of a kv head) of a sequence:
// entry e has its (max, sum) at ml(e) and its normalised output numbers d0 .. d0 + 3 at o(e, d0).
template <int D>
struct RowPieces {
    const float2* ml0;
    const float* o0;
    int n = 0;
    bool both = false;                // the two slots of a piece hold the same rows
    __device__ __forceinline__ void find(const PrefixParams& p, int g, int b, int kvh, int r)
    {
        const PrefixGroup gr = load_prefix_group(p, g);
        const int grow = (b - gr.off) * p.rows + r;
        const int pair = grow / PFX_PAIR, at = grow - pair * PFX_PAIR;
        const int pairs = prefix_pairs(p, gr);
        const int2 run = __ldcg(p.runs + prefix_run_base(p, g, gr) + kvh * pairs + pair);
        // (a shared pass that gave up may have left this run's entry unwritten)
        if (run.x < 0 || run.y < 0 || run.x > p.pieces - run.y) return;
        both = gr.n * p.rows - pair * PFX_PAIR <= PFX_TILE;
        const size_t slot = static_cast<size_t>(run.x) * 2 + at / PFX_TILE;
        ml0 = p.piece_ml + slot * PFX_TILE + at % PFX_TILE;
        o0 = p.piece_o + slot * (PFX_TILE * D) + at % PFX_TILE * 4;
        n = both ? 2 * run.y : run.y;
    }
    __device__ __forceinline__ size_t slot(int e) const { return both ? e : 2 * e; }
    __device__ __forceinline__ float2 ml(int e) const { return __ldcg(ml0 + slot(e) * PFX_TILE); }
    __device__ __forceinline__ float4 o(int e, int d0) const
    {
        return __ldcg(reinterpret_cast<const float4*>(o0 + slot(e) * (PFX_TILE * D) + d0 * PFX_TILE));
    }
};

// Adds the pieces of a row to acc (numbers d0 ..) and the weight W, against the maximum M.
template <class C, int D>
__device__ __forceinline__ void add_pieces(const RowPieces<D>& pc, int d0, float M, float (&acc)[C::E], float& W)
{
#pragma unroll 4
    for (int e = 0; e < pc.n; ++e) {
        const float2 v = pc.ml(e);
        if (!(v.y > 0.f)) continue;                  // a piece this row sees nothing of
        const float w = v.y * fast_exp2(v.x - M);
        W += w;
#pragma unroll
        for (int k = 0; k < C::E; k += 4) {
            const float4 x = pc.o(e, d0 + k);
            acc[k] += w * x.x;
            acc[k + 1] += w * x.y;
            acc[k + 2] += w * x.z;
            acc[k + 3] += w * x.w;
        }
    }
}

template <bool FP8, int D, int BS, int NT>
struct SpanCfg : DecodeCfg<FP8, D, BS, NT> {
    using C = DecodeCfg<FP8, D, BS, NT>;
    static constexpr int SMEM = 1024 + C::NSTAGE * C::STAGE + C::NSTAGE * (8 + 8 + 4) + 16;   // ring, barriers, ids, flags
    static constexpr int MINB = NT == 8 ? 3 : 2;    // CTAs per SM: 16-row tiles keep twice the state
    static_assert(C::RED_BYTES <= C::NSTAGE * C::STAGE, "epilogue buffer reuses the stages");
};

template <bool FP8, int D, int BS, int NT, int RULE>
__global__ void __launch_bounds__(DecodeCfg<FP8, D, BS, NT>::THREADS, SpanCfg<FP8, D, BS, NT>::MINB)
paged_decode_span(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
                  const SpanParams sp)
{
    using C = DecodeCfg<FP8, D, BS, NT>;
    const DecodeParams& p = sp.d;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::NSTAGE * C::STAGE);
    uint64_t* empty = full + C::NSTAGE;
    int* stage_blk = reinterpret_cast<int*>(empty + C::NSTAGE);
    int* merge_flag = stage_blk + C::NSTAGE;
    int* group_slot = merge_flag + 1;                  // the suffix form: the sequence's group
    constexpr bool SUFFIX = RULE == SPAN_SUFFIX;

    const int b = blockIdx.y;
    const int kvh = blockIdx.x / p.head_groups;
    const int hg = blockIdx.x - kvh * p.head_groups;
    const int split = blockIdx.z;
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int nh = min(NT, p.rows - hg * NT);          // real rows in this tile
    const size_t row0 = (static_cast<size_t>(b) * p.kv_heads + kvh) * p.rows + hg * NT;

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::NSTAGE; ++i) {
            mbar_init(smem_u32(full + i), 1);
            mbar_init(smem_u32(empty + i), 1);
        }
        fence_mbar_init();
        if constexpr (SUFFIX) *group_slot = -1;
    }
    grid_dependency_wait();                          // inputs of the preceding kernel are ready

    int ctx = __ldg(p.ctx + b);
    int first = 0, prefix = 0;
    int group = -1;                                  // the sequence's group, if it shares blocks
    if constexpr (SUFFIX) {
        __syncthreads();
        bool ok = true;
        for (int g = threadIdx.x; g < sp.shared.n_groups; g += C::THREADS) {
            ok = ok && prefix_offsets_ok(sp.shared, g);
            if (__ldg(sp.shared.group_offsets + g) <= b && b < __ldg(sp.shared.group_offsets + g + 1)) *group_slot = g;
        }
        if (__syncthreads_and(ok)) group = *group_slot;   // bad offsets: nothing is shared
        if (group >= 0) {
            first = load_prefix_group(sp.shared, group).blocks * BS;
            if (first == 0) group = -1;
        }
    } else {
        if (sp.first_keys != nullptr) first = max(0, __ldg(sp.first_keys + b));
        if (sp.prefix_lens != nullptr) prefix = __ldg(sp.prefix_lens + b);
    }
    uint32_t qf[C::KS][C::NTT][2];
    float sl2 = 0.f;
    if (warp < C::NCW)
        sl2 = load_q_frags<FP8, D, BS, NT>(qf, p.q + row0 * D, nh, lane, p.scale_log2, p.k_scale, kvh);
    const int cap = p.max_blocks * BS;
    if (ctx < 0 || ctx > cap || (ctx > 0 && ctx < p.q_len)) {
        // out of range (clamped), or fewer cached tokens than new queries (kept: the queries
        // at negative positions see nothing but the visible prefix)
        if (threadIdx.x == 0 && split == 0 && blockIdx.x == 0) atomicOr(p.err, KV_DEVERR_CONTEXT);
        ctx = ctx < 0 ? 0 : (ctx > cap ? cap : ctx);
    }
    // keys of query token i: both ends grow with i
    const int visible = min(prefix, ctx);
    const auto key_lo = [&](int i) {
        const int pos = ctx - p.q_len + i;
        return !SUFFIX && sp.window > 0 ? max(first, pos - sp.window + 1) : first;
    };
    const auto key_hi = [&](int i) { return max(ctx - p.q_len + i + 1, visible); };
    // tokens of the tile's rows: a run, or all of them where the tile spans two heads
    const int i0 = (hg * NT) % p.q_len;
    const bool wraps = i0 + nh > p.q_len;
    const int tile_lo = key_lo(wraps ? 0 : i0);
    const int tile_hi = key_hi(wraps ? p.q_len - 1 : i0 + nh - 1);
    const int blk_first = tile_lo / BS;
    const int nblk = tile_hi > tile_lo ? (tile_hi + BS - 1) / BS - blk_first : 0;
    const int nsplit = nblk > 0 ? (nblk + p.split_blocks - 1) / p.split_blocks : 1;
    const int blk0 = blk_first + split * p.split_blocks;
    const int nb = max(0, min(nblk - split * p.split_blocks, p.split_blocks));
    __syncthreads();                                 // barriers initialised
    if (split >= nsplit) {                           // this tile has fewer chunks
        grid_dependents_launch();
        return;
    }

    // ------------------------------------------------------------ producer warp
    if (warp == C::NCW) {
        if (lane == 0) {
            prefetch_tensormap(&tmk);
            prefetch_tensormap(&tmv);
        }
        const int32_t* trow = p.tables + static_cast<size_t>(b) * p.max_blocks + blk0;
        int issued = 0;
        bool ok = true;
        for (int base = 0; base < nb && ok; base += 32) {
            const int j = base + lane;
            int id = -1;
            if (j < nb) {
                id = __ldg(trow + j);
                if (id < 0 || id >= p.num_blocks) {
                    atomicOr(p.err, KV_DEVERR_BLOCK_ID);
                    id = -1;                          // skipped: never addressed
                }
            }
            const int cnt = min(32, nb - base);
            for (int k = 0; k < cnt; ++k) {
                const int blk = __shfl_sync(FULL_MASK, id, k);
                const int it = base + k;
                if (it == p.stop_stage) {                // test hook: the rest never lands
                    ok = false;
                    break;
                }
                const int st = it % C::NSTAGE;
                const uint32_t ph = static_cast<uint32_t>(it / C::NSTAGE) & 1u;
                int good = 1;
                if (lane == 0) {
                    if (!mbar_wait_bounded(smem_u32(empty + st), ph ^ 1u)) {
                        atomicOr(p.err, KV_DEVERR_TIMEOUT);
                        good = 0;
                    } else {
                        stage_blk[st] = blk;
                        const uint32_t fb = smem_u32(full + st);
                        if (blk >= 0) {
                            const uint32_t dst = smem_u32(smem + st * C::STAGE);
                            mbar_arrive_expect_tx(fb, C::STAGE);
                            tma_load_5d(dst, &tmk, 0, 0, kvh, 0, blk, fb);
                            tma_load_5d(dst + C::TILE, &tmv, 0, 0, kvh, 0, blk, fb);
                        } else {
                            mbar_arrive(fb);
                        }
                    }
                }
                good = __shfl_sync(FULL_MASK, good, 0);
                if (!good) {
                    ok = false;
                    break;
                }
                issued = it + 1;
            }
        }
        grid_dependents_launch();                    // every load of this CTA is issued
        // Drain: the CTA must not exit while a copy into its shared memory is in flight.
        if (lane == 0) {
            for (int it = max(0, issued - C::NSTAGE); it < issued; ++it) {
                if (!mbar_wait_bounded(smem_u32(full + (it % C::NSTAGE)),
                                       static_cast<uint32_t>(it / C::NSTAGE) & 1u)) {
                    atomicOr(p.err, KV_DEVERR_TIMEOUT);
                    break;
                }
            }
        }
        return;
    }

    // ------------------------------------------------------------ consumer warps
    SpanRows<C::NTT, RULE> rows;
    rows.sl2 = sl2;
    rows.cap_in = sp.cap_in;
    rows.cap_log2 = sp.cap_log2;
    rows.tile_lo = tile_lo;
    rows.tile_hi = tile_hi;
#pragma unroll
    for (int nt = 0; nt < C::NTT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int local = nt * 8 + 2 * (lane & 3) + j;
            const int r = hg * NT + local;
            const int head = r / p.q_len, i = r - head * p.q_len;
            rows.lo[nt][j] = key_lo(i);
            rows.hi[nt][j] = local < nh ? key_hi(i) : 0;      // padding rows see nothing
            rows.pos[nt][j] = ctx - p.q_len + i;
            rows.slope[nt][j] = rows.BIAS && local < nh
                                    ? __ldg(sp.slopes + kvh * p.group + head) * 1.4426950408889634f
                                    : 0.f;
        }
    WarpState<C> st;
    reset_state(st);
    const unsigned long long wait_ns = p.consumer_wait_ns ? p.consumer_wait_ns : WAIT_LIMIT_NS;
    for (int it = warp; it < nb; it += C::NCW) {
        const int s = it % C::NSTAGE;
        const uint32_t ph = static_cast<uint32_t>(it / C::NSTAGE) & 1u;
        const bool arrived = mbar_wait_bounded(smem_u32(full + s), ph, wait_ns);
        if (!__all_sync(FULL_MASK, arrived)) {
            if (lane == 0) atomicOr(p.err, KV_DEVERR_TIMEOUT);
            break;
        }
        const int blk = stage_blk[s];
        if (blk >= 0) {
            const uint32_t tk = smem_u32(smem + s * C::STAGE);
            rows.base = (blk0 + it) * BS;
            process_block_rows<FP8, D, BS, NT>(tk, tk + C::TILE, rows, qf, st, lane);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(empty + s));
    }

    // ------------------------------------------------------------ epilogue
    grid_dependents_launch();
    reduce_row_sums(st);
    named_barrier_sync(1, C::NCW * 32);     // every consumer is done with the stages
    float* red = reinterpret_cast<float*>(smem);
    stash_state<FP8>(red, st, warp, lane);
    named_barrier_sync(1, C::NCW * 32);

    const int t = threadIdx.x;
    const int head = (t * C::E) / D;
    const int d0 = (t * C::E) % D;
    const size_t bh = row0 + head;                   // global query row
    if (head < nh) {
        float acc[C::E], M, L;
        combine_warps<C>(red, head, d0, FP8 ? __ldg(p.v_scale + kvh) : 1.f, acc, M, L);
        if (nsplit == 1) {
            if constexpr (SUFFIX) {
                RowPieces<D> pc;
                if (group >= 0) pc.find(sp.shared, group, b, kvh, hg * NT + head);
                if (pc.n > 0) {
                    float top = L > 0.f ? M : -INFINITY;
                    for (int e = 0; e < pc.n; ++e) {
                        const float2 v = pc.ml(e);
                        if (v.y > 0.f) top = fmaxf(top, v.x);
                    }
                    float W = L > 0.f ? L * fast_exp2(M - top) : 0.f;
#pragma unroll
                    for (int e = 0; e < C::E; ++e) acc[e] *= W;
                    add_pieces<C, D>(pc, d0, top, acc, W);
                    const float inv = W > 0.f ? 1.f / W : 0.f;
#pragma unroll
                    for (int e = 0; e < C::E; ++e) acc[e] *= inv;
                    M = top;
                    L = W;
                }
            }
            uint32_t* dst = reinterpret_cast<uint32_t*>(p.out + bh * D + d0);
#pragma unroll
            for (int e = 0; e < C::E; e += 2) dst[e / 2] = pack_bf16x2(acc[e], acc[e + 1]);
            if (p.lse != nullptr && d0 == 0) p.lse[bh] = lse_from(M, L);
        } else {
            float* dst = p.part_o + (bh * p.max_splits + split) * D + d0;
#pragma unroll
            for (int e = 0; e < C::E; ++e) dst[e] = acc[e];
            if (d0 == 0) {
                p.part_ml[(bh * p.max_splits + split) * 2 + 0] = M;
                p.part_ml[(bh * p.max_splits + split) * 2 + 1] = L;
            }
            __threadfence();                        // partial visible before the ticket
        }
    }
    if (nsplit == 1) return;

    // ---- ticket: the last chunk of this unit to finish merges all chunks
    named_barrier_sync(1, C::NCW * 32);
    int* ticket = p.tickets + (static_cast<size_t>(b) * p.kv_heads + kvh) * p.head_groups + hg;
    if (t == 0) {
        const int last = atomicAdd(ticket, 1) == nsplit - 1;
        if (last) __threadfence();
        *merge_flag = last;
    }
    named_barrier_sync(1, C::NCW * 32);
    if (!*merge_flag) return;
    if (head < nh) {
        const float* ml = p.part_ml + bh * p.max_splits * 2;
        float M = -INFINITY;
        RowPieces<D> pc;
        if constexpr (SUFFIX) {
            if (group >= 0) pc.find(sp.shared, group, b, kvh, hg * NT + head);
            for (int e = 0; e < pc.n; ++e) {
                const float2 v = pc.ml(e);
                if (v.y > 0.f) M = fmaxf(M, v.x);
            }
        }
        for (int j = 0; j < nsplit; ++j) {
            if (__ldcg(ml + 2 * j + 1) > 0.f) M = fmaxf(M, __ldcg(ml + 2 * j));
        }
        float acc[C::E];
#pragma unroll
        for (int e = 0; e < C::E; ++e) acc[e] = 0.f;
        float W = 0.f;
        const float* ob = p.part_o + bh * p.max_splits * D + d0;
        for (int j = 0; j < nsplit; ++j) {
            const float lj = __ldcg(ml + 2 * j + 1);
            if (!(lj > 0.f)) continue;               // a chunk this row sees nothing of
            const float wj = lj * fast_exp2(__ldcg(ml + 2 * j) - M);
            W += wj;
            const float* oj = ob + static_cast<size_t>(j) * D;
#pragma unroll
            for (int e = 0; e < C::E; e += 4) {
                const float4 v = __ldcg(reinterpret_cast<const float4*>(oj + e));
                acc[e] += wj * v.x;
                acc[e + 1] += wj * v.y;
                acc[e + 2] += wj * v.z;
                acc[e + 3] += wj * v.w;
            }
        }
        if constexpr (SUFFIX) add_pieces<C, D>(pc, d0, M, acc, W);
        const float inv = W > 0.f ? 1.f / W : 0.f;
        uint32_t* dst = reinterpret_cast<uint32_t*>(p.out + bh * D + d0);
#pragma unroll
        for (int e = 0; e < C::E; e += 2) dst[e / 2] = pack_bf16x2(acc[e] * inv, acc[e + 1] * inv);
        if (p.lse != nullptr && d0 == 0) p.lse[bh] = lse_from(M, W);
    }
    if (t == 0) *ticket = 0;                        // ready for the next call
}

template <bool FP8, int D, int BS, int NT>
cudaError_t prepare_span_variant()
{
    const auto raise = [](auto kernel) {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    SpanCfg<FP8, D, BS, NT>::SMEM);
    };
    cudaError_t e = raise(paged_decode_span<FP8, D, BS, NT, SPAN_MASK>);
    if (e == cudaSuccess) e = raise(paged_decode_span<FP8, D, BS, NT, SPAN_CAP>);
    if (e == cudaSuccess) e = raise(paged_decode_span<FP8, D, BS, NT, SPAN_BIAS>);
    if (e == cudaSuccess) e = raise(paged_decode_span<FP8, D, BS, NT, SPAN_CAP_BIAS>);
    if (e == cudaSuccess) e = raise(paged_decode_span<FP8, D, BS, NT, SPAN_SUFFIX>);
    return e;
}

template <bool FP8, int D, int BS, int NT>
cudaError_t launch_span_variant(SpanRule rule, dim3 grid, const CUtensorMap& tk, const CUtensorMap& tv,
                                const SpanParams& p, cudaStream_t s)
{
    const auto go = [&](auto kernel) {
        return launch_dependent(kernel, grid, dim3(DecodeCfg<FP8, D, BS, NT>::THREADS),
                                SpanCfg<FP8, D, BS, NT>::SMEM, s, tk, tv, p);
    };
    switch (rule) {
    case SPAN_MASK: return go(paged_decode_span<FP8, D, BS, NT, SPAN_MASK>);
    case SPAN_CAP: return go(paged_decode_span<FP8, D, BS, NT, SPAN_CAP>);
    case SPAN_BIAS: return go(paged_decode_span<FP8, D, BS, NT, SPAN_BIAS>);
    case SPAN_CAP_BIAS: return go(paged_decode_span<FP8, D, BS, NT, SPAN_CAP_BIAS>);
    case SPAN_SUFFIX: return go(paged_decode_span<FP8, D, BS, NT, SPAN_SUFFIX>);
    }
    return cudaErrorInvalidValue;
}

}  // namespace kvp
