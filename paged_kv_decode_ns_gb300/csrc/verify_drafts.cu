// verify_drafts.cu -- verification of drafted tokens (speculative sampling).
//
// Draft i is accepted when u_i q_i(x_i) < p_i(x_i) (the product of two floats
// is exact in fp64).  At the first rejection the next token is drawn from
// w = max(p - q, 0), with no rejection from w = p_n: the smallest v whose
// cumulative weight exceeds r * sum w.  Sums are fp64.
#include "ns_common.cuh"
#include "ns_internal.h"

namespace ns {

namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;

struct Weights {
    const float *p, *q;  // q: nullptr when only p counts
    int skip;            // token of weight 0 (certain draft), or -1
    __device__ __forceinline__ double operator()(int v) const
    {
        const float a = __ldg(p + v);
        double w = a;
        if (q != nullptr)
            w -= (double)__ldg(q + v);
        return (w > 0.0 && v != skip) ? w : 0.0;
    }
};

__global__ void __launch_bounds__(kThreads) verify_kernel(const VerifyArgs a)
{
    __shared__ int sh_state;      // 0: go on, 1: skip the sequence
    __shared__ int sh_accepted;
    __shared__ double sh_sum[kWarps];
    __shared__ int sh_last[kWarps];
    const int s = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int first = __ldg(a.start + s), end = __ldg(a.start + s + 1);
    const int n = end - first;
    if (first < 0 || end < first || end > a.total_drafts) {
        if (threadIdx.x == 0)
            raise_status(a.status, NS_DEV_BAD_QUERY_SPAN);
        return;
    }
    int32_t *out = a.out_tokens + first + s;
    if (warp == 0) {
        int accepted = n;
        bool bad = false;
        for (int i0 = 0; i0 < n; i0 += 32) {
            const int i = i0 + lane;
            bool ok = true, off = false;
            if (i < n) {
                const int x = __ldg(a.tokens + first + i);
                off = x < 0 || x >= a.vocab;
                if (!off) {
                    const double p = __ldg(a.target + (long long)(first + s + i) * a.target_stride + x);
                    const double q = a.draft ? (double)__ldg(a.draft + (long long)(first + i) * a.draft_stride + x) : 1.0;
                    ok = (double)__ldg(a.accept_u + first + i) * q < p;
                }
            }
            bad |= __any_sync(0xffffffffu, off);
            const unsigned no = __ballot_sync(0xffffffffu, !ok);
            if (no != 0 && accepted == n)
                accepted = i0 + __ffs(no) - 1;
        }
        for (int i = lane; i <= n; i += 32)
            out[i] = !bad && i < accepted ? __ldg(a.tokens + first + i) : -1;
        if (lane == 0) {
            sh_state = bad ? 1 : 0;
            sh_accepted = accepted;
            a.num_accepted[s] = bad ? -1 : accepted;
            if (bad)
                raise_status(a.status, NS_DEV_BAD_TOKEN);
        }
    }
    __syncthreads();
    if (sh_state != 0)
        return;
    const int acc = sh_accepted;
    const bool refused = acc < n;
    Weights w;
    w.p = a.target + (long long)(first + s + acc) * a.target_stride;
    w.q = refused && a.draft ? a.draft + (long long)(first + acc) * a.draft_stride : nullptr;
    w.skip = refused && !a.draft ? __ldg(a.tokens + first + acc) : -1;

    // each warp owns a contiguous run of the vocabulary
    const int per = (a.vocab + kWarps - 1) / kWarps;
    const int lo = min(a.vocab, warp * per), hi = min(a.vocab, lo + per);
    double total = 0.0;
    for (int pass = 0; pass < 2; ++pass) {
        double sum = 0.0;
        int last = -1;  // the last token with a positive weight
        for (int v = lo + lane; v < hi; v += 32) {
            const double x = w(v);
            sum += x;
            last = x > 0.0 ? v : last;
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            sum += __shfl_xor_sync(0xffffffffu, sum, o);
            last = max(last, __shfl_xor_sync(0xffffffffu, last, o));
        }
        if (lane == 0) {
            sh_sum[warp] = sum;
            sh_last[warp] = last;
        }
        __syncthreads();
        total = 0.0;
        for (int i = 0; i < kWarps; ++i)
            total += sh_sum[i];
        if (total > 0.0 || (w.q == nullptr && w.skip < 0))
            break;
        w.q = nullptr;  // nothing is left of p after the draft's distribution: draw from p
        w.skip = -1;
        __syncthreads();
    }
    const double goal = (double)__ldg(a.sample_u + s) * total;
    double before = 0.0;  // weight of the warps before this one
    int mine = -1, lastv = -1;
    for (int i = 0; i < kWarps; ++i) {
        if (mine < 0 && before + sh_sum[i] > goal)
            mine = i;
        if (mine < 0)
            before += sh_sum[i];
        lastv = max(lastv, sh_last[i]);
    }
    if (mine < 0) {  // no cumulative weight exceeds the goal: no positive weight at all
        if (threadIdx.x == 0)
            out[acc] = lastv;
        return;
    }
    if (warp != mine)
        return;
    for (int v0 = lo; v0 < hi; v0 += 32) {
        const double x = v0 + lane < hi ? w(v0 + lane) : 0.0;
        double cum = x;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const double y = __shfl_up_sync(0xffffffffu, cum, o);
            if (lane >= o)
                cum += y;
        }
        const unsigned over = __ballot_sync(0xffffffffu, x > 0.0 && before + cum > goal);
        if (over != 0) {
            if (lane == 0)
                out[acc] = v0 + __ffs(over) - 1;
            return;
        }
        before += __shfl_sync(0xffffffffu, cum, 31);
    }
    // the run's sum in this order fell short of the goal by its rounding
    if (lane == 0)
        out[acc] = sh_last[mine];
}

}  // namespace

cudaError_t launch_verify_drafts(const VerifyArgs &a, cudaStream_t stream)
{
    verify_kernel<<<a.num_seqs, kThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace ns
