// norm_rope_append.cu -- per-head RMS norm of queries and keys, rotary rotation by position,
// and the paged append of keys and values, in one pass over the projections' output.
//
// For every token i (sequence s, position p) and every head row x of its queries and keys:
//   y = x / sqrt(mean(x^2) + eps) * w                      (w given; else y = x)
//   (y_a, y_b) <- (y_a cos - y_b sin, y_b cos + y_a sin)   for the pairs of the first rope_dim
//                                                          numbers, cos/sin from row p of a table
// Queries go to q_out, keys to block table entry p / block_size, slot p % block_size of the
// pool, values to the same place of the V half (xuewyang.github.io/posts/kv, "A toy vLLM",
// write_kv; brunomaga.github.io, PagedKVCache.append).  Everything is fp32 between the bf16
// input and one rounding at the store: bf16 to nearest even, or e4m3(y / scale) with the
// quotient rounded to binary32 first, as paged_kv_append does -- a key is rounded once here,
// where norm, rotation and append as separate passes round it two or three times.
//
// What it must move is each row once in and once out; there is little to do per byte, so a prompt is
// bound by memory as long as the instructions per row are few, and a decode step by latency.  A row
// of D numbers belongs to D / 8 lanes, and a lane holds the two groups of four numbers that rotate
// with each other (half-split pairs: groups rope_dim / 2 apart; interleaved pairs, and numbers that
// do not rotate: neighbours): the rotation needs no exchange between lanes, the sum of squares one
// shuffle reduction, and most arithmetic runs two numbers at a time.  Two forms, by the number of
// tokens (launch_nra_form):
//   * direct: a lane group takes RPT rows of one token, their loads in flight together, and looks
//     the token's place up itself;
//   * streaming (prompts): see paged_norm_rope_append_stream.
// Measured on a GB300 (32 query heads and 8 kv heads of 128 numbers, normalised and rotated):
//   1 token          2.0 us, 64 tokens 2.35 us: the latency of position -> table -> row and a launch
//   185 tokens of 96 rows, rotated by half, 8-bit cache   4.25 us
//   8,191 tokens    39.6 us for 206 MB (5.2 TB/s, 77 % of the copy rate; the schedulers issue in 64 %
//     of the cycles).  The direct form takes 62 us: it looks the place of every token up anew in each
//     of the token's lane groups.
#include "append_row.cuh"
#include "device_common.cuh"
#include "kernels.h"

namespace kvp {

namespace {

constexpr int NRA_THREADS = 256;
// Rows per SM up to which a lane group of the direct form takes one row, or two (else four): fewer
// rows per lane group start sooner, more of them pay a token's lookups once.  With 1 / 2 / 4 rows:
// 1 token of 48 rows 2.05 / 2.40 / 3.2 us, 64 tokens 2.36 / 2.54 / 3.3, 185 tokens of 96 rows (8-bit)
// 5.44 / 4.43 / 5.09 (before the codes came from products); with 2 / 4: 456 tokens of 48 rows 5.02 / 5.27, 700 tokens 5.74 / 5.38.
constexpr int NRA_ROWS_1 = 54, NRA_ROWS_2 = 160;
// Tokens per CTA from which the streaming form is taken.  Streaming / direct: 1,000 tokens 8.1 / 7.5 us,
// 1,400 tokens 10.9 / 10.7, 2,000 tokens 13.8 / 15.4, 8,191 tokens 39.9 / 62.
constexpr int NRA_STREAM_TOKENS = 3;

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 mul2(float2 a, float2 b)
{
    float2 d;
    asm("mul.rn.f32x2 %0, %1, %2;"
        : "=l"(reinterpret_cast<uint64_t&>(d))
        : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
    return d;
}

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    float2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(reinterpret_cast<uint64_t&>(d))
        : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)), "l"(reinterpret_cast<uint64_t&>(c)));
    return d;
}

__device__ __forceinline__ uint32_t e4m3x4(float2 a, float2 b)
{
    return (static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(a, __NV_SATFINITE, __NV_E4M3)) & 0xffffu) |
           (static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(b, __NV_SATFINITE, __NV_E4M3)) << 16);
}

// e4m3 codes of y / scale, low element first, the bits of e4m3_codes8 (the quotient rounded to
// binary32, then the code).  The product with the reciprocal is off from that quotient by three
// steps of binary32 at most (1.5 2^-23 relative: two roundings against one), and the codes change
// only where the low 19 bits of a number are zero (between two codes: four significant bits below
// the codes' own), so the product gives the same code unless it is within four steps of such a
// number; then, and for scales whose reciprocal could leave the normal range, the division decides.
// (8,192 tokens of 48 rows 42.0 us, 43.6 with divisions only; 185 tokens of 96 rows 4.25 and 4.42.)
__device__ __forceinline__ uint2 e4m3_codes(const float2 (&y)[4], float scale)
{
    const float inv = __frcp_rn(scale);
    const float2 inv2 = make_float2(inv, inv);
    float2 q[4];
    uint32_t near = ~0u;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        q[e] = mul2(y[e], inv2);
        near = min(near, min((__float_as_uint(q[e].x) + 4u) & 0x7ffffu, (__float_as_uint(q[e].y) + 4u) & 0x7ffffu));
    }
    const uint32_t bits = __float_as_uint(scale);
    const bool exact = (bits & 0x7fffffu) == 0;     // a power of two: the product is the quotient
    const bool normal = (bits >> 23) - 28u < 200u;  // positive, 2^-99 .. 2^100
    if (!normal || (near <= 8 && !exact)) {
#pragma unroll
        for (int e = 0; e < 4; ++e) q[e] = make_float2(__fdiv_rn(y[e].x, scale), __fdiv_rn(y[e].y, scale));
    }
    return make_uint2(e4m3x4(q[0], q[1]), e4m3x4(q[2], q[3]));
}

__device__ __forceinline__ float2 bf16x2_floats(uint32_t w)
{
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

// Where a token goes.
struct NraToken {
    long long q_row;                                // row of q_out of its head 0; < 0: the token writes nothing
    long long slot;                                 // first row of its slot in the pool; < 0: not cached
};

__device__ __forceinline__ NraToken nra_token(const NormRopeParams& p, uint32_t i, int pos, int blk)
{
    const uint32_t b = i / static_cast<uint32_t>(p.q_len), t = i - b * static_cast<uint32_t>(p.q_len);
    NraToken tok;
    tok.q_row = static_cast<long long>(b) * p.q_heads * p.q_len + t;
    tok.slot = blk >= 0 && blk < p.num_blocks
                   ? (static_cast<long long>(blk) * p.block_size + pos % p.block_size) * p.kv_heads
                   : -1;
    return tok;
}

// A lane's numbers of a row -- at[0] .. at[0] + 3 and at[1] .. at[1] + 3 -- and how they rotate.
struct NraLane {
    int at[2];
    int pair;                                       // first of its four pairs in the table's row
    bool turn;

    __device__ __forceinline__ void init(const NormRopeParams& p, int l)
    {
        turn = 8 * l < p.rope_dim;                  // rope_dim 0: no rotation
        const bool split = turn && !p.interleaved;
        at[0] = split ? 4 * l : 8 * l;
        at[1] = split ? 4 * l + p.rope_dim / 2 : 8 * l + 4;
        pair = 4 * l;
    }
};

// cos, sin and -sin of a lane's four pairs.
struct NraTurn {
    float2 c[2], s[2], n[2];
    __device__ __forceinline__ void load(const NormRopeParams& p, const float* row, const NraLane& ln)
    {
        const float4 a = *reinterpret_cast<const float4*>(row + ln.pair);
        const float4 b = *reinterpret_cast<const float4*>(row + p.rope_dim / 2 + ln.pair);
        c[0] = make_float2(a.x, a.y), c[1] = make_float2(a.z, a.w);
        s[0] = make_float2(b.x, b.y), s[1] = make_float2(b.z, b.w);
        n[0] = make_float2(-b.x, -b.y), n[1] = make_float2(-b.z, -b.w);
    }
};

// A lane's numbers: y[0], y[1] the first four, y[2], y[3] the others.
__device__ __forceinline__ void nra_unpack(uint2 x0, uint2 x1, float2 (&y)[4])
{
    y[0] = bf16x2_floats(x0.x), y[1] = bf16x2_floats(x0.y);
    y[2] = bf16x2_floats(x1.x), y[3] = bf16x2_floats(x1.y);
}

__device__ __forceinline__ void nra_weights(const float* weight, const NraLane& ln, float2 (&g)[4])
{
    const float4 g0 = __ldg(reinterpret_cast<const float4*>(weight + ln.at[0]));
    const float4 g1 = __ldg(reinterpret_cast<const float4*>(weight + ln.at[1]));
    g[0] = make_float2(g0.x, g0.y), g[1] = make_float2(g0.z, g0.w);
    g[2] = make_float2(g1.x, g1.y), g[3] = make_float2(g1.z, g1.w);
}

// The mean square of a row and eps, the same bits in every lane of the row.
template <int D>
__device__ __forceinline__ float nra_mean_square(const float2 (&y)[4], float eps, unsigned group_mask)
{
    const float2 sq = fma2(y[0], y[0], fma2(y[1], y[1], fma2(y[2], y[2], mul2(y[3], y[3]))));
    float ss = sq.x + sq.y;
#pragma unroll
    for (int o = D / 16; o >= 1; o >>= 1) ss += __shfl_xor_sync(group_mask, ss, o);
    return fmaf(ss, 1.f / D, eps);
}

__device__ __forceinline__ float nra_rsqrt(float x)
{
    float y;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void nra_times(float2 (&y)[4], float f)
{
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] = mul2(y[e], make_float2(f, f));
}

// Squares of numbers below 2^-63 or above 2^63 leave the range of normal fp32 numbers: the factor of
// such a row comes from the mean square of the numbers times 2^96 or 2^-96 (what that rounds away is
// nothing beside the sum, which then lies between 2^-81 and 2^106) and of eps times the square of
// that.  Two factors, to be multiplied by one after the other: nothing on the way leaves the range
// either.  (Not inlined: in place it costs the decode step of 64 sequences 0.15 us, 3.1 -> 3.3.)
template <int D>
__device__ __noinline__ float2 nra_far_factors(float2 y0, float2 y1, float2 y2, float2 y3, float eps, unsigned group_mask,
                                               bool small)
{
    float2 y[4] = {y0, y1, y2, y3};
    const float by = small ? 0x1p96f : 0x1p-96f;
    nra_times(y, by);
    const float inv = nra_rsqrt(nra_mean_square<D>(y, eps * by * by, group_mask));
    return small ? make_float2(by, inv) : make_float2(inv, by);
}

// y <- y / sqrt(mean(y^2) + eps) * g.
template <int D>
__device__ __forceinline__ void nra_norm(float2 (&y)[4], const float2 (&g)[4], float eps, unsigned group_mask)
{
    const float ms = nra_mean_square<D>(y, eps, group_mask);
    float inv = nra_rsqrt(ms);
    if (!(ms >= 0x1p-100f && ms <= 0x1p100f)) {
        const float2 f = nra_far_factors<D>(y[0], y[1], y[2], y[3], eps, group_mask, ms < 1.f);
        nra_times(y, f.x);
        inv = f.y;
    }
    const float2 inv2 = make_float2(inv, inv);
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] = mul2(mul2(y[e], inv2), g[e]);
}

__device__ __forceinline__ void nra_rotate(float2 (&y)[4], const NraTurn& w, bool interleaved)
{
    if (interleaved) {
        // pairs (y[0].x, y[0].y), ..: gathered into first and second numbers and back
        const float2 a0 = make_float2(y[0].x, y[1].x), b0 = make_float2(y[0].y, y[1].y);
        const float2 a1 = make_float2(y[2].x, y[3].x), b1 = make_float2(y[2].y, y[3].y);
        const float2 p0 = fma2(b0, w.n[0], mul2(a0, w.c[0])), q0 = fma2(a0, w.s[0], mul2(b0, w.c[0]));
        const float2 p1 = fma2(b1, w.n[1], mul2(a1, w.c[1])), q1 = fma2(a1, w.s[1], mul2(b1, w.c[1]));
        y[0] = make_float2(p0.x, q0.x), y[1] = make_float2(p0.y, q0.y);
        y[2] = make_float2(p1.x, q1.x), y[3] = make_float2(p1.y, q1.y);
    } else {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const float2 a = y[e], b = y[2 + e];
            y[e] = fma2(b, w.n[e], mul2(a, w.c[e]));
            y[2 + e] = fma2(a, w.s[e], mul2(b, w.c[e]));
        }
    }
}

__device__ __forceinline__ void nra_store(uint16_t* dst, const NraLane& ln, const float2 (&y)[4])
{
    *reinterpret_cast<uint2*>(dst + ln.at[0]) = make_uint2(pack_bf16x2(y[0].x, y[0].y), pack_bf16x2(y[1].x, y[1].y));
    *reinterpret_cast<uint2*>(dst + ln.at[1]) = make_uint2(pack_bf16x2(y[2].x, y[2].y), pack_bf16x2(y[3].x, y[3].y));
}

__device__ __forceinline__ void nra_store_codes(uint8_t* dst, const NraLane& ln, const float2 (&y)[4], float scale)
{
    const uint2 codes = e4m3_codes(y, scale);
    *reinterpret_cast<uint32_t*>(dst + ln.at[0]) = codes.x;
    *reinterpret_cast<uint32_t*>(dst + ln.at[1]) = codes.y;
}

// Key (r < kv_heads) or value row of a cached token whose slot's rows begin at row `slot` of the
// pool; g: the keys' weights (norm).  Uniform in the row's lanes.
template <int D, bool FP8>
__device__ __forceinline__ void nra_kv_row(const NormRopeParams& p, size_t slot, const NraLane& ln, const NraTurn& w, bool norm,
                                           const float2 (&g)[4], uint2 x0, uint2 x1, int r, unsigned group_mask)
{
    const bool is_v = r >= p.kv_heads;
    const int h = is_v ? r - p.kv_heads : r;
    uint8_t* pool = is_v ? p.v_pool : p.k_pool;
    if (is_v && !FP8) {
        uint16_t* dst = reinterpret_cast<uint16_t*>(pool) + (slot + h) * D;
        *reinterpret_cast<uint2*>(dst + ln.at[0]) = x0;
        *reinterpret_cast<uint2*>(dst + ln.at[1]) = x1;
        return;
    }
    float2 y[4];
    nra_unpack(x0, x1, y);
    if (!is_v) {
        if (norm) nra_norm<D>(y, g, p.eps, group_mask);
        if (ln.turn) nra_rotate(y, w, p.interleaved);
    }
    if constexpr (FP8)
        nra_store_codes(pool + (slot + h) * D, ln, y, __ldg((is_v ? p.v_scale : p.k_scale) + h));
    else
        nra_store(reinterpret_cast<uint16_t*>(pool) + (slot + h) * D, ln, y);
}

// Sequence and position of token i, checked; flag: this thread reports what is wrong.  False: the
// token writes nothing.
__device__ __forceinline__ bool nra_place(const NormRopeParams& p, uint32_t i, bool flag, int& seq, int& pos)
{
    seq = p.token_seq != nullptr ? __ldg(p.token_seq + i) : static_cast<int>(i / static_cast<uint32_t>(p.q_len));
    if (seq < 0 || seq >= p.batch) {
        if (flag) atomicOr(p.err, KV_DEVERR_SEQ);
        return false;
    }
    pos = p.token_pos != nullptr ? __ldg(p.token_pos + i)
                                 : __ldg(p.ctx + seq) - p.q_len + static_cast<int>(i % static_cast<uint32_t>(p.q_len));
    if (pos < 0 || pos / p.block_size >= p.max_blocks || (p.rope != nullptr && pos >= p.rope_positions)) {
        if (flag) atomicOr(p.err, KV_DEVERR_POSITION);
        return false;
    }
    return true;
}

template <int D, bool FP8, int RPT>
__global__ void __launch_bounds__(NRA_THREADS) paged_norm_rope_append_kernel(const NormRopeParams p)
{
    constexpr int LPR = D / 8;                      // lanes of a row
    static_assert(LPR == 8 || LPR == 16, "several rows per warp");
    constexpr int GPC = NRA_THREADS / LPR;          // lane groups per CTA
    grid_dependency_wait();                         // inputs of the preceding kernel are ready
    grid_dependents_launch();
    const int l = threadIdx.x % LPR;
    const uint32_t unit = blockIdx.x * GPC + threadIdx.x / LPR;
    const uint32_t i = unit / p.chunks;             // token
    const int r0 = static_cast<int>(unit - i * p.chunks) * RPT;
    // a whole lane group leaves together; its lanes never shuffle with another group's
    if (i >= static_cast<uint32_t>(p.num_tokens)) return;
    const unsigned group_mask = ((1u << LPR) - 1u) << (threadIdx.x % 32 / LPR * LPR);
    const int rows = p.q_heads + 2 * p.kv_heads;

    NraLane ln;
    ln.init(p, l);
    uint2 x0[RPT], x1[RPT];
#pragma unroll
    for (int j = 0; j < RPT; ++j) {
        const int r = r0 + j;
        x0[j] = x1[j] = make_uint2(0u, 0u);
        if (r < rows) {
            const uint16_t* src =
                r < p.q_heads ? p.q + i * p.q_stride + r * D
                : r < p.q_heads + p.kv_heads ? p.k + i * p.k_stride + (r - p.q_heads) * D
                                             : p.v + i * p.v_stride + (r - p.q_heads - p.kv_heads) * D;
            x0[j] = __ldg(reinterpret_cast<const uint2*>(src + ln.at[0]));
            x1[j] = __ldg(reinterpret_cast<const uint2*>(src + ln.at[1]));
        }
    }
    const bool flag = r0 == 0 && l == 0;            // one lane of the token reports
    int seq, pos;
    if (!nra_place(p, i, flag, seq, pos)) return;
    const int blk = __ldg(p.tables + static_cast<size_t>(seq) * p.max_blocks + pos / p.block_size);
    const NraToken tok = nra_token(p, i, pos, blk);
    if (tok.slot < 0 && flag) atomicOr(p.err, KV_DEVERR_BLOCK_ID);      // its query row is still computed
    NraTurn w;
    if (ln.turn && r0 < p.q_heads + p.kv_heads) w.load(p, p.rope + static_cast<size_t>(pos) * p.rope_dim, ln);
    const bool norm = p.q_weight != nullptr;
#pragma unroll
    for (int j = 0; j < RPT; ++j) {
        const int r = r0 + j;
        if (r >= rows) return;
        float2 g[4];
        if (r < p.q_heads) {
            float2 y[4];
            nra_unpack(x0[j], x1[j], y);
            if (norm) {
                nra_weights(p.q_weight, ln, g);
                nra_norm<D>(y, g, p.eps, group_mask);
            }
            if (ln.turn) nra_rotate(y, w, p.interleaved);
            nra_store(p.q_out + (tok.q_row + static_cast<long long>(r) * p.q_len) * D, ln, y);
        } else if (tok.slot >= 0) {
            if (norm && r < p.q_heads + p.kv_heads) nra_weights(p.k_weight, ln, g);
            nra_kv_row<D, FP8>(p, tok.slot, ln, w, norm, g, x0[j], x1[j], r - p.q_heads, group_mask);
        }
    }
}

// The streaming form, for prompts: persistent CTAs take equal runs of tokens; a producer warp looks
// up 32 tokens' places at a time and brings each token's rows and its cos/sin row into a ring of
// stages with bulk copies, so that the loads run far ahead of the arithmetic and the chain
// position -> table -> row is paid once per 32 tokens; eight warps take a token's rows from there.
constexpr int NRS_CW = 8;
constexpr int NRS_THREADS = (NRS_CW + 1) * 32;
constexpr int NRS_CTAS = 3;                         // per SM
constexpr int NRS_RING = 72 * 1024;
constexpr int NRS_STAGES = 16;                      // at most

struct NrsCtl {
    uint64_t full[NRS_STAGES], empty[NRS_STAGES];
    NraToken tok[NRS_STAGES];
};

template <int D, bool FP8>
__global__ void __launch_bounds__(NRS_THREADS, NRS_CTAS)
paged_norm_rope_append_stream(const NormRopeParams p, int stage_bytes, int stages)
{
    constexpr int LPR = D / 8;
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ NrsCtl ctl;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < stages; ++i) {
            mbar_init(smem_u32(&ctl.full[i]), 1);
            mbar_init(smem_u32(&ctl.empty[i]), NRS_CW);
        }
        fence_mbar_init();
    }
    grid_dependency_wait();                         // inputs of the preceding kernel are ready
    grid_dependents_launch();
    __syncthreads();
    const uint32_t lo = static_cast<uint32_t>(static_cast<unsigned long long>(p.num_tokens) * blockIdx.x / gridDim.x);
    const uint32_t hi = static_cast<uint32_t>(static_cast<unsigned long long>(p.num_tokens) * (blockIdx.x + 1) / gridDim.x);
    const uint32_t q_bytes = static_cast<uint32_t>(p.q_heads) * D * 2, kv_bytes = static_cast<uint32_t>(p.kv_heads) * D * 2;
    const uint32_t rope_bytes = p.rope != nullptr ? static_cast<uint32_t>(p.rope_dim) * 4 : 0u;

    if (warp == NRS_CW) {
        bool ok = true;
        int n = 0;                                  // tokens issued
        const auto place = [&](uint32_t i, int& seq, int& pos, int& blk) {
            seq = -1;
            if (i >= hi) return;
            if (nra_place(p, i, true, seq, pos)) {
                blk = __ldg(p.tables + static_cast<size_t>(seq) * p.max_blocks + pos / p.block_size);
                if (blk < 0 || blk >= p.num_blocks) {
                    atomicOr(p.err, KV_DEVERR_BLOCK_ID);                // its query row is still computed
                    blk = -1;
                }
            } else {
                seq = -1;
            }
        };
        int seq, pos = 0, blk = -1;
        place(lo + lane, seq, pos, blk);
        for (uint32_t base = lo; base < hi && ok; base += 32) {
            int seq2, pos2 = 0, blk2 = -1;          // the next 32 tokens
            place(base + 32 + lane, seq2, pos2, blk2);
            const int cnt = static_cast<int>(min(32u, hi - base));
            for (int k = 0; k < cnt; ++k, ++n) {
                const int s = n % stages;
                const int tseq = __shfl_sync(FULL_MASK, seq, k);
                const int tpos = __shfl_sync(FULL_MASK, pos, k);
                const int tblk = __shfl_sync(FULL_MASK, blk, k);
                ok = n != p.stop_stage;             // test hook: the rest never lands
                if (!ok) break;
                ok = all_ok(mbar_wait_bounded(smem_u32(&ctl.empty[s]), (static_cast<uint32_t>(n / stages) & 1u) ^ 1u));
                if (!ok) break;
                const uint32_t i = base + k;
                const uint32_t bar = smem_u32(&ctl.full[s]);
                if (lane == 0) {
                    NraToken tok = nra_token(p, i, tpos, tblk);
                    if (tseq < 0) tok.q_row = -1;
                    ctl.tok[s] = tok;
                    if (tseq >= 0)
                        mbar_arrive_expect_tx(bar, q_bytes + 2 * kv_bytes + rope_bytes);
                    else
                        mbar_arrive(bar);
                }
                __syncwarp();                       // armed before any byte can land
                if (tseq >= 0 && lane < 4) {
                    const uint32_t dst = smem_u32(ring + static_cast<size_t>(s) * stage_bytes);
                    const void* src = lane == 0   ? static_cast<const void*>(p.q + i * p.q_stride)
                                      : lane == 1 ? static_cast<const void*>(p.k + i * p.k_stride)
                                      : lane == 2 ? static_cast<const void*>(p.v + i * p.v_stride)
                                                  : static_cast<const void*>(p.rope + static_cast<size_t>(tpos) * p.rope_dim);
                    const uint32_t off = lane == 0 ? 0u : lane == 1 ? q_bytes : lane == 2 ? q_bytes + kv_bytes : q_bytes + 2 * kv_bytes;
                    const uint32_t bytes = lane == 0 ? q_bytes : lane < 3 ? kv_bytes : rope_bytes;
                    if (bytes > 0) bulk_load(dst + off, src, bytes, bar);
                }
            }
            seq = seq2;
            pos = pos2;
            blk = blk2;
        }
        if (!ok && lane == 0 && n != p.stop_stage) atomicOr(p.err, KV_DEVERR_TIMEOUT);
        // copies still in flight must land before the CTA exits
        for (int j = max(0, n - stages); j < n; ++j)
            if (!mbar_wait_bounded(smem_u32(&ctl.full[j % stages]), static_cast<uint32_t>(j / stages) & 1u)) break;
        return;
    }

    NraLane ln;
    ln.init(p, lane % LPR);
    const unsigned group_mask = ((1u << LPR) - 1u) << (lane / LPR * LPR);
    constexpr int GPC = NRS_CW * 32 / LPR;          // rows in hand at a time
    const int count = static_cast<int>(hi - lo);
    const int group = threadIdx.x / LPR;
    const bool norm = p.q_weight != nullptr;
    float2 gq[4], gk[4];
    if (norm) {
        nra_weights(p.q_weight, ln, gq);
        nra_weights(p.k_weight, ln, gk);
    }
    const long long q_step = static_cast<long long>(p.q_len) * D;
    const unsigned long long wait_ns = p.consumer_wait_ns ? p.consumer_wait_ns : WAIT_LIMIT_NS;
    for (int n = 0; n < count; ++n) {
        const int s = n % stages;
        if (!all_ok(mbar_wait_bounded(smem_u32(&ctl.full[s]), static_cast<uint32_t>(n / stages) & 1u, wait_ns))) {
            if (lane == 0) atomicOr(p.err, KV_DEVERR_TIMEOUT);
            break;
        }
        const NraToken tok = ctl.tok[s];
        if (tok.q_row >= 0) {
            const uint8_t* st = ring + static_cast<size_t>(s) * stage_bytes;
            NraTurn w;
            if (ln.turn) w.load(p, reinterpret_cast<const float*>(st + q_bytes + 2 * kv_bytes), ln);
            const uint16_t* x = reinterpret_cast<const uint16_t*>(st) + group * D;
            uint16_t* dst = p.q_out + tok.q_row * D + group * q_step;
            for (int r = group; r < p.q_heads; r += GPC, x += GPC * D, dst += GPC * q_step) {
                float2 y[4];
                nra_unpack(*reinterpret_cast<const uint2*>(x + ln.at[0]), *reinterpret_cast<const uint2*>(x + ln.at[1]), y);
                if (norm) nra_norm<D>(y, gq, p.eps, group_mask);
                if (ln.turn) nra_rotate(y, w, p.interleaved);
                nra_store(dst, ln, y);
            }
            if (tok.slot >= 0) {
                x = reinterpret_cast<const uint16_t*>(st + q_bytes) + group * D;
                for (int r = group; r < 2 * p.kv_heads; r += GPC, x += GPC * D)
                    nra_kv_row<D, FP8>(p, tok.slot, ln, w, norm, gk, *reinterpret_cast<const uint2*>(x + ln.at[0]),
                                       *reinterpret_cast<const uint2*>(x + ln.at[1]), r, group_mask);
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&ctl.empty[s]));
    }
}

template <int D, bool FP8, int RPT>
cudaError_t launch_nra(NormRopeParams p, cudaStream_t s)
{
    constexpr int GPC = NRA_THREADS / (D / 8);
    const int rows = p.q_heads + 2 * p.kv_heads;
    p.chunks = static_cast<uint32_t>((rows + RPT - 1) / RPT);
    const long long units = static_cast<long long>(p.num_tokens) * p.chunks;
    const long long ctas = (units + GPC - 1) / GPC;
    return launch_dependent(paged_norm_rope_append_kernel<D, FP8, RPT>, dim3(static_cast<unsigned>(ctas)),
                            dim3(NRA_THREADS), 0, s, p);
}

template <int D, bool FP8>
cudaError_t launch_nra_form(const NormRopeParams& p, int num_sms, cudaStream_t s)
{
    const long long bytes = (static_cast<long long>(p.q_heads) + 2 * p.kv_heads) * D * 2 + p.rope_dim * 4;
    const long long stage = (bytes + 127) / 128 * 128;
    const int ctas = num_sms * NRS_CTAS;
    if (p.num_tokens >= NRA_STREAM_TOKENS * ctas && stage * 3 <= NRS_RING) {
        const int stages = static_cast<int>(NRS_RING / stage < NRS_STAGES ? NRS_RING / stage : NRS_STAGES);
        return launch_dependent(paged_norm_rope_append_stream<D, FP8>, dim3(static_cast<unsigned>(ctas)), dim3(NRS_THREADS),
                                static_cast<size_t>(stages) * stage, s, p, static_cast<int>(stage), stages);
    }
    const long long rows = static_cast<long long>(p.num_tokens) * (p.q_heads + 2 * p.kv_heads);
    if (rows <= static_cast<long long>(NRA_ROWS_1) * num_sms) return launch_nra<D, FP8, 1>(p, s);
    if (rows <= static_cast<long long>(NRA_ROWS_2) * num_sms) return launch_nra<D, FP8, 2>(p, s);
    return launch_nra<D, FP8, 4>(p, s);
}

template <int D, bool FP8>
cudaError_t prepare_nra()
{
    return cudaFuncSetAttribute(paged_norm_rope_append_stream<D, FP8>, cudaFuncAttributeMaxDynamicSharedMemorySize, NRS_RING);
}

}  // namespace

cudaError_t prepare_norm_rope_append(int head_dim, bool fp8)
{
    if (head_dim == 128) return fp8 ? prepare_nra<128, true>() : prepare_nra<128, false>();
    if (head_dim == 64 && !fp8) return prepare_nra<64, false>();
    return cudaErrorInvalidValue;
}

cudaError_t launch_norm_rope_append(const NormRopeParams& p, int head_dim, bool fp8, int num_sms, cudaStream_t s)
{
    if (head_dim == 128)
        return fp8 ? launch_nra_form<128, true>(p, num_sms, s) : launch_nra_form<128, false>(p, num_sms, s);
    if (head_dim == 64 && !fp8) return launch_nra_form<64, false>(p, num_sms, s);
    return cudaErrorInvalidValue;
}

}  // namespace kvp
