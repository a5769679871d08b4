// span_attn_q4_d128.cu -- instantiations of the span attention (q4_0 paged cache, head_dim 128).
#include "span_attn.cuh"

cudaError_t ns::launch_span_q4_d128(bool bf16, const span::Maps &tm, const span::Params &P, int ctas,
                              cudaStream_t stream)
{
    return bf16 ? span::launch<BF16, 128, 4>(tm, P, ctas, stream) : span::launch<F16, 128, 4>(tm, P, ctas, stream);
}
