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
// What it must move is each row once in and once out; there is nothing else to do per byte, so
// it is bound by memory for a prompt and by latency for a decode step.  A row of D numbers
// belongs to D / 8 lanes (one 16-byte vector each): the sum of squares is a shuffle reduction
// inside those lanes, and the partner of a rotated number sits in the same lane (interleaved
// pairs) or a fixed number of lanes away (half-split pairs).  A lane group takes RPT rows of one
// token: their loads are in flight together, and the token's position, table entry and
// cos/sin row are fetched once for all of them.
#include "append_row.cuh"
#include "device_common.cuh"
#include "kernels.h"

namespace kvp {

namespace {

constexpr int NRA_THREADS = 256;

// Four pairs of e4m3 codes of y / scale, low element first (the arithmetic of e4m3_codes8).
__device__ __forceinline__ uint2 e4m3_codes8f(const float (&y)[8], float scale)
{
    uint32_t c[2] = {0u, 0u};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float2 v = make_float2(__fdiv_rn(y[2 * e], scale), __fdiv_rn(y[2 * e + 1], scale));
        const uint32_t two = __nv_cvt_float2_to_fp8x2(v, __NV_SATFINITE, __NV_E4M3);
        c[e >> 1] |= (two & 0xffffu) << (16 * (e & 1));
    }
    return make_uint2(c[0], c[1]);
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

    uint4 x[RPT];
#pragma unroll
    for (int j = 0; j < RPT; ++j) {
        const int r = r0 + j;
        x[j] = make_uint4(0u, 0u, 0u, 0u);
        if (r < rows) {
            const uint16_t* src =
                r < p.q_heads ? p.q + i * p.q_stride + r * D
                : r < p.q_heads + p.kv_heads ? p.k + i * p.k_stride + (r - p.q_heads) * D
                                             : p.v + i * p.v_stride + (r - p.q_heads - p.kv_heads) * D;
            x[j] = __ldg(reinterpret_cast<const uint4*>(src) + l);
        }
    }

    const int t = static_cast<int>(i % static_cast<uint32_t>(p.q_len));
    const int b = static_cast<int>(i / static_cast<uint32_t>(p.q_len));
    const int seq = p.token_seq != nullptr ? __ldg(p.token_seq + i) : b;
    const bool flag = r0 == 0 && l == 0;            // one lane of the token reports
    if (seq < 0 || seq >= p.batch) {
        if (flag) atomicOr(p.err, KV_DEVERR_SEQ);
        return;
    }
    const int pos = p.token_pos != nullptr ? __ldg(p.token_pos + i) : __ldg(p.ctx + seq) - p.q_len + t;
    if (pos < 0 || pos / p.block_size >= p.max_blocks || (p.rope != nullptr && pos >= p.rope_positions)) {
        if (flag) atomicOr(p.err, KV_DEVERR_POSITION);
        return;
    }
    const int blk = __ldg(p.tables + static_cast<size_t>(seq) * p.max_blocks + pos / p.block_size);
    const bool cached = blk >= 0 && blk < p.num_blocks;
    if (!cached && flag) atomicOr(p.err, KV_DEVERR_BLOCK_ID);   // its query row is still computed
    const size_t slot = (static_cast<size_t>(cached ? blk : 0) * p.block_size + pos % p.block_size) * p.kv_heads;

    // cos / sin of this lane's numbers (half-split: number 8l + e pairs with the one rope_dim / 2
    // away and uses entry (8l + e) mod rope_dim / 2; interleaved: pair 4l + e / 2)
    const int half = p.rope_dim / 2;
    const bool turn = p.rope != nullptr && 8 * l < p.rope_dim && r0 < p.q_heads + p.kv_heads;
    const bool upper = 8 * l >= half;
    float cs[8], sn[8];
    if (turn) {
        const float* row = p.rope + static_cast<size_t>(pos) * p.rope_dim;
        if (p.interleaved) {
            const float4 c = __ldg(reinterpret_cast<const float4*>(row) + l);
            const float4 s = __ldg(reinterpret_cast<const float4*>(row + half) + l);
            cs[0] = c.x, cs[1] = c.y, cs[2] = c.z, cs[3] = c.w;
            sn[0] = s.x, sn[1] = s.y, sn[2] = s.z, sn[3] = s.w;
        } else {
            const float4* c = reinterpret_cast<const float4*>(row + (upper ? 8 * l - half : 8 * l));
            const float4* s = reinterpret_cast<const float4*>(row + half + (upper ? 8 * l - half : 8 * l));
            const float4 c0 = __ldg(c), c1 = __ldg(c + 1), s0 = __ldg(s), s1 = __ldg(s + 1);
            cs[0] = c0.x, cs[1] = c0.y, cs[2] = c0.z, cs[3] = c0.w;
            cs[4] = c1.x, cs[5] = c1.y, cs[6] = c1.z, cs[7] = c1.w;
            sn[0] = s0.x, sn[1] = s0.y, sn[2] = s0.z, sn[3] = s0.w;
            sn[4] = s1.x, sn[5] = s1.y, sn[6] = s1.z, sn[7] = s1.w;
        }
    }
    const int partner = upper ? l - half / 8 : l + half / 8;
    const int from = (threadIdx.x % 32 / LPR) * LPR + (turn && !p.interleaved ? partner : l);

#pragma unroll
    for (int j = 0; j < RPT; ++j) {
        const int r = r0 + j;
        if (r >= rows) return;
        const bool is_q = r < p.q_heads;
        const bool is_v = r >= p.q_heads + p.kv_heads;
        const int h = is_q ? r : is_v ? r - p.q_heads - p.kv_heads : r - p.q_heads;
        if (is_v) {
            if (!cached) return;
            if constexpr (FP8)
                reinterpret_cast<uint2*>(p.v_pool + (slot + h) * D)[l] = e4m3_codes8(x[j], __ldg(p.v_scale + h));
            else
                reinterpret_cast<uint4*>(p.v_pool + (slot + h) * D * 2)[l] = x[j];
            continue;
        }
        float y[8];
        const uint32_t w4[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            y[2 * e] = __uint_as_float(w4[e] << 16);
            y[2 * e + 1] = __uint_as_float(w4[e] & 0xffff0000u);
        }
        const float* weight = is_q ? p.q_weight : p.k_weight;
        if (weight != nullptr) {
            float ss = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) ss += y[e] * y[e];
#pragma unroll
            for (int o = LPR / 2; o >= 1; o >>= 1) ss += __shfl_xor_sync(group_mask, ss, o);
            const float inv = rsqrtf(ss * (1.f / D) + p.eps);
            const float4 g0 = __ldg(reinterpret_cast<const float4*>(weight) + 2 * l);
            const float4 g1 = __ldg(reinterpret_cast<const float4*>(weight) + 2 * l + 1);
            const float g[8] = {g0.x, g0.y, g0.z, g0.w, g1.x, g1.y, g1.z, g1.w};
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = y[e] * inv * g[e];
        }
        if (p.rope != nullptr) {
            if (p.interleaved) {
                if (turn) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float a = y[2 * e], c = y[2 * e + 1];
                        y[2 * e] = a * cs[e] - c * sn[e];
                        y[2 * e + 1] = c * cs[e] + a * sn[e];
                    }
                }
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float o = __shfl_sync(group_mask, y[e], from);
                    if (turn) y[e] = upper ? y[e] * cs[e] + o * sn[e] : y[e] * cs[e] - o * sn[e];
                }
            }
        }
        if (is_q || !FP8) {
            const uint4 o = make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]),
                                       pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7]));
            if (is_q) {
                const size_t row = (static_cast<size_t>(b) * p.q_heads + h) * p.q_len + t;
                reinterpret_cast<uint4*>(p.q_out + row * D)[l] = o;
            } else if (cached) {
                reinterpret_cast<uint4*>(p.k_pool + (slot + h) * D * 2)[l] = o;
            }
        } else if (cached) {
            reinterpret_cast<uint2*>(p.k_pool + (slot + h) * D)[l] = e4m3_codes8f(y, __ldg(p.k_scale + h));
        }
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
cudaError_t launch_nra_rows(const NormRopeParams& p, cudaStream_t s)
{
    return launch_nra<D, FP8, 4>(p, s);
}

}  // namespace

cudaError_t launch_norm_rope_append(const NormRopeParams& p, int head_dim, bool fp8, cudaStream_t s)
{
    if (head_dim == 128) return fp8 ? launch_nra_rows<128, true>(p, s) : launch_nra_rows<128, false>(p, s);
    if (head_dim == 64 && !fp8) return launch_nra_rows<64, false>(p, s);
    return cudaErrorInvalidValue;
}

}  // namespace kvp
