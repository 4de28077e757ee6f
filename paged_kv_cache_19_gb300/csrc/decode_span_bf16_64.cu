// decode_span_bf16_64.cu -- bf16-cache variants of the span attention kernel, head_dim 64.
#include "decode_span.cuh"

namespace kvp {

#define KVP_SPAN_BF16_VARIANTS(X) \
    X(64, 8, 1) X(64, 8, 2) X(64, 8, 4) X(64, 16, 1) X(64, 16, 2) X(64, 16, 4)

cudaError_t launch_span_bf16_64(SpanRule rule, int head_dim, int head_tile, int heads, int ctas, const CUtensorMap& tk,
                             const CUtensorMap& tv, const SpanParams& p, cudaStream_t s)
{
#define KVP_CASE(D_, NT_, HC_) \
    if (head_dim == D_ && head_tile == NT_ && heads == HC_) \
        return launch_span_variant<false, D_, NT_, HC_>(rule, ctas, tk, tv, p, s);
    KVP_SPAN_BF16_VARIANTS(KVP_CASE)
#undef KVP_CASE
    return cudaErrorInvalidValue;
}

cudaError_t prepare_span_bf16_64(int head_dim, int head_tile, int heads)
{
#define KVP_CASE(D_, NT_, HC_) \
    if (head_dim == D_ && head_tile == NT_ && heads == HC_) return prepare_span_variant<false, D_, NT_, HC_>();
    KVP_SPAN_BF16_VARIANTS(KVP_CASE)
#undef KVP_CASE
    return cudaErrorInvalidValue;
}

}  // namespace kvp
