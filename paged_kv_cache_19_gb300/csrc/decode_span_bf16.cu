// decode_span_bf16.cu -- bf16-cache variants of the span attention kernel.
#include "decode_span.cuh"

namespace kvp {

#define KVP_SPAN_BF16_VARIANTS(X) \
    X(64, 16, 8) X(64, 16, 16) X(64, 32, 8) X(64, 32, 16) \
    X(128, 16, 8) X(128, 16, 16) X(128, 32, 8) X(128, 32, 16)

cudaError_t launch_span_bf16(SpanRule rule, int head_dim, int block_size, int head_tile, dim3 grid,
                             const CUtensorMap& tk, const CUtensorMap& tv, const SpanParams& p,
                             cudaStream_t s)
{
#define KVP_CASE(D_, BS_, NT_) \
    if (head_dim == D_ && block_size == BS_ && head_tile == NT_) \
        return launch_span_variant<false, D_, BS_, NT_>(rule, grid, tk, tv, p, s);
    KVP_SPAN_BF16_VARIANTS(KVP_CASE)
#undef KVP_CASE
    return cudaErrorInvalidValue;
}

cudaError_t prepare_span_bf16(int head_dim, int block_size, int head_tile)
{
#define KVP_CASE(D_, BS_, NT_) \
    if (head_dim == D_ && block_size == BS_ && head_tile == NT_) \
        return prepare_span_variant<false, D_, BS_, NT_>();
    KVP_SPAN_BF16_VARIANTS(KVP_CASE)
#undef KVP_CASE
    return cudaErrorInvalidValue;
}

}  // namespace kvp
