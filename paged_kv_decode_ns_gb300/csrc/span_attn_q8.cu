// span_attn_q8.cu -- instantiations of the span attention (q8_0 paged cache).
#include "span_attn.cuh"

cudaError_t ns::launch_span_q8(bool bf16, const span::Maps &tm, const span::Params &P, int ctas,
                              cudaStream_t stream)
{
    return bf16 ? span::launch<BF16, 64, 8>(tm, P, ctas, stream) : span::launch<F16, 64, 8>(tm, P, ctas, stream);
}
