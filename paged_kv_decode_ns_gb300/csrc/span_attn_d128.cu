// span_attn_d128.cu -- instantiations of the span attention (contiguous rows, head_dim 128).
#include "span_attn.cuh"

cudaError_t ns::launch_span_d128(bool bf16, const span::Maps &tm, const span::Params &P, int ctas,
                              cudaStream_t stream)
{
    return bf16 ? span::launch<BF16, 128, 0>(tm, P, ctas, stream) : span::launch<F16, 128, 0>(tm, P, ctas, stream);
}
