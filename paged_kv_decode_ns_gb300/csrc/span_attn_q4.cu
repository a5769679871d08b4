// span_attn_q4.cu -- instantiations of the span attention (q4_0 paged cache).
#include "span_attn.cuh"

cudaError_t ns::launch_span_q4(bool bf16, const span::Maps &tm, const span::Params &P, int ctas,
                              cudaStream_t stream)
{
    return bf16 ? span::launch<BF16, 64, 4>(tm, P, ctas, stream) : span::launch<F16, 64, 4>(tm, P, ctas, stream);
}
