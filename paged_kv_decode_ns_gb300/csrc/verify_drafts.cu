// verify_drafts.cu -- verification of drafted tokens (speculative sampling).
//
// Draft i is accepted when u_i q_i(x_i) < p_i(x_i) (the product of two floats
// is exact in fp64).  At the first rejection the next token is drawn from
// w = max(p - q, 0), with no rejection from w = p_n: the smallest v whose
// cumulative weight exceeds r * sum w.
//
// A CTA per sequence, a cluster of up to eight while sequences are few: every CTA
// finds the first rejection itself (a few gathers), then sums its contiguous slice of
// the one row that matters, a contiguous run per warp.  The run sums go to every CTA
// of the cluster through distributed shared memory; the CTA that owns the run the
// goal falls into reads that run again, a stretch a warp, and one warp narrows the
// stretch down to the token.  One pass over one row of p and one of q is all the
// memory traffic and bounds a large batch: 256 sequences of 151936 tokens (311 MB)
// 54.0 us, 5.8 TB/s.  Four sequences take 10.6 us, a chain of dependent reads.
//
// Precision: neighbouring cumulative weights differ by single probabilities, so
// fp32 sums would move the drawn token.  fp64 additions (about two a clock on an SM)
// would cost more than the memory pass (one CTA a sequence with fp64 sums: 798 us
// for 256 sequences of 151936 tokens); here w is split exactly into a float and its
// rounding error (0 <= q <= p, so (p - w) - q is exact) and sums are pairs of
// floats (a run's is off by 2^-45 of itself at 151936 tokens, 2^-40 at 2^23, by
// emulation).  fp64 joins the few sums that are compared.
#include "ns_common.cuh"
#include "ns_internal.h"
#include "tcgen05.cuh"

namespace ns {

namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kMaxCluster = 8, kCtasPerSm = 2;
constexpr int kBatch = 4;  // 16-byte loads of a row in flight a thread

// h + l, l the rounding error of h.
struct Pair {
    float h, l;
    __device__ __forceinline__ double value() const { return (double)h + (double)l; }
};

// The weight of a token, exactly max(p - q, 0).  NaN counts as 0 in either (fmaxf and
// fminf return the other operand); with q within [0, p] the difference needs no test.
__device__ __forceinline__ Pair weight(float p, float q)
{
    p = fmaxf(p, 0.f);
    q = fminf(fmaxf(q, 0.f), p);
    Pair w;
    w.h = p - q;
    w.l = (p - w.h) - q;
    return w;
}

// The two heads are added without error; what is small stays in l.
__device__ __forceinline__ Pair operator+(Pair a, Pair b)
{
    const float t = a.h + b.h, x = t - a.h;
    return {t, ((a.h - (t - x)) + (b.h - x)) + (a.l + b.l)};
}

__device__ __forceinline__ Pair shfl_xor(Pair a, int o)
{
    return {__shfl_xor_sync(0xffffffffu, a.h, o), __shfl_xor_sync(0xffffffffu, a.l, o)};
}

// The same two at a time, in packed instructions: half the instructions of the
// sums, which bound a large batch as much as memory does.
struct Pair2 {
    float2 h, l;
};

__device__ __forceinline__ float2 sub2(float2 a, float2 b)  // rounds once
{
    return ffma2(b, make_float2(-1.f, -1.f), a);
}

template <bool Q>
__device__ __forceinline__ Pair2 weight(float2 p, float2 q)
{
    p = make_float2(fmaxf(p.x, 0.f), fmaxf(p.y, 0.f));
    if (!Q)
        return {p, make_float2(0.f, 0.f)};
    q = make_float2(fminf(fmaxf(q.x, 0.f), p.x), fminf(fmaxf(q.y, 0.f), p.y));
    Pair2 w;
    w.h = sub2(p, q);
    w.l = sub2(sub2(p, w.h), q);
    return w;
}

__device__ __forceinline__ Pair2 operator+(Pair2 a, Pair2 b)
{
    const float2 t = fadd2(a.h, b.h), x = sub2(t, a.h);
    return {t, fadd2(fadd2(sub2(a.h, sub2(t, x)), sub2(b.h, x)), fadd2(a.l, b.l))};
}

struct Row {
    const float *p, *q;  // q: nullptr when only p counts
    int skip;            // token of weight 0 (certain draft), or -1
    __device__ __forceinline__ Pair at(int v) const
    {
        return weight(v == skip ? 0.f : p[v], q != nullptr ? q[v] : 0.f);
    }
};

// This thread's share of [lo, hi): elements 4 lane + 128 i .. + 3 when the rows are
// 16-byte aligned at lo, lane + 32 i otherwise.
template <bool Q>
__device__ Pair slice_sum(const Row &r, int lo, int hi, int lane, bool aligned)
{
    Pair2 sum[2] = {};
    int v = lo;
    if (aligned) {
        for (; v < hi; v += kBatch * 128) {  // hi is a multiple of 4 here
            float4 p[kBatch], q[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const bool on = v + i * 128 + 4 * lane < hi;
                p[i] = on ? reinterpret_cast<const float4 *>(r.p + v + i * 128)[lane] : make_float4(0.f, 0.f, 0.f, 0.f);
                q[i] = Q && on ? reinterpret_cast<const float4 *>(r.q + v + i * 128)[lane] : make_float4(0.f, 0.f, 0.f, 0.f);
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                if (!Q) {
                    const int e = r.skip - (v + i * 128 + 4 * lane);
                    p[i].x = e == 0 ? 0.f : p[i].x;
                    p[i].y = e == 1 ? 0.f : p[i].y;
                    p[i].z = e == 2 ? 0.f : p[i].z;
                    p[i].w = e == 3 ? 0.f : p[i].w;
                }
                sum[0] = sum[0] + weight<Q>(make_float2(p[i].x, p[i].y), make_float2(q[i].x, q[i].y));
                sum[1] = sum[1] + weight<Q>(make_float2(p[i].z, p[i].w), make_float2(q[i].z, q[i].w));
            }
        }
    } else {
        for (; v < hi; v += 4 * kBatch * 32) {
            float p[4 * kBatch], q[4 * kBatch];
#pragma unroll
            for (int i = 0; i < 4 * kBatch; ++i) {
                const int at = v + i * 32 + lane;
                p[i] = at < hi && at != r.skip ? r.p[at] : 0.f;
                q[i] = Q && at < hi ? r.q[at] : 0.f;
            }
#pragma unroll
            for (int i = 0; i < 4 * kBatch; i += 2)
                sum[(i >> 1) & 1] = sum[(i >> 1) & 1] + weight<Q>(make_float2(p[i], p[i + 1]), make_float2(q[i], q[i + 1]));
        }
    }
    const Pair2 both = sum[0] + sum[1];
    return Pair{both.h.x, both.l.x} + Pair{both.h.y, both.l.y};
}

__device__ __forceinline__ void st_cluster_pair(uint32_t addr, Pair a)
{
    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(addr), "f"(a.h), "f"(a.l) : "memory");
}

// One warp: the first of `count` <= 256 weights, in order, whose cumulative sum
// exceeds goal; -1 when none does.  before: what came before the first, then before
// the one found.
struct Place {
    int at;
    double before, total;
};
template <class Goal>
__device__ Place find(const Pair *w, int count, int lane, double before, Goal goal)
{
    const int each = (count + 31) / 32, i0 = lane * each;
    double x[8], mine = 0.0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        x[i] = i < each && i0 + i < count ? w[i0 + i].value() : 0.0;
        if (i < each)
            mine += x[i];
    }
    double incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const double y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o)
            incl += y;
    }
    Place r;
    r.total = __shfl_sync(0xffffffffu, incl, 31);
    const double g = goal(r.total);
    double c = before + (incl - mine);
    int at = -1;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < each && at < 0) {
            if (x[i] > 0.0 && c + x[i] > g)
                at = i0 + i;
            else
                c += x[i];
        }
    const unsigned who = __ballot_sync(0xffffffffu, at >= 0);
    const int src = who != 0 ? __ffs(who) - 1 : 0;
    r.at = who != 0 ? __shfl_sync(0xffffffffu, at, src) : -1;
    r.before = __shfl_sync(0xffffffffu, c, src);
    return r;
}

__global__ void __launch_bounds__(kThreads, kCtasPerSm) verify_kernel(const VerifyArgs a, int cluster)
{
    __shared__ int sh_state;  // 0: go on, 1: skip the sequence
    __shared__ int sh_accepted;
    __shared__ __align__(8) Pair sh_run[2][kMaxCluster * kWarps];  // run sums of the cluster, in order (one set a pass)
    __shared__ Pair sh_part[kWarps], sh_lane[kThreads];
    __shared__ Place sh_place;
    __shared__ double sh_goal;
    __shared__ int sh_last;
    grid_dependency_wait();
    grid_launch_dependents();
    const int s = blockIdx.x / cluster, rank = blockIdx.x % cluster;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int first = a.start[s], end = a.start[s + 1];
    const int n = end - first;
    if (first < 0 || end < first || end > a.total_drafts) {
        if (threadIdx.x == 0 && rank == 0)
            raise_status(a.status, NS_DEV_BAD_QUERY_SPAN);
        return;  // the whole cluster
    }
    int32_t *out = a.out_tokens + first + s;
    const double u = a.sample_u[s];
    if (warp == 0) {
        int accepted = n;
        bool bad = false;
        for (int i0 = 0; i0 < n; i0 += 32) {
            const int i = i0 + lane;
            bool ok = true, off = false;
            if (i < n) {
                const int x = a.tokens[first + i];
                off = x < 0 || x >= a.vocab;
                if (!off) {
                    const double p = a.target[(long long)(first + s + i) * a.target_stride + x];
                    const double q = a.draft ? (double)fmaxf(a.draft[(long long)(first + i) * a.draft_stride + x], 0.f) : 1.0;
                    ok = (double)a.accept_u[first + i] * q < p;
                }
            }
            bad |= __any_sync(0xffffffffu, off);
            const unsigned no = __ballot_sync(0xffffffffu, !ok);
            if (no != 0 && accepted == n)
                accepted = i0 + __ffs(no) - 1;
        }
        if (rank == 0)  // the place of the drawn token is left to the CTA that finds it
            for (int i = lane; i <= n; i += 32)
                if (bad || i != accepted)
                    out[i] = !bad && i < accepted ? a.tokens[first + i] : -1;
        if (lane == 0) {
            sh_state = bad ? 1 : 0;
            sh_accepted = accepted;
            sh_last = -1;
            if (rank == 0) {
                a.num_accepted[s] = bad ? -1 : accepted;
                if (bad)
                    raise_status(a.status, NS_DEV_BAD_TOKEN);
            }
        }
    }
    __syncthreads();
    if (sh_state != 0)
        return;  // the whole cluster
    // every CTA of the cluster has started before another one writes to it
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    const int acc = sh_accepted;
    const bool refused = acc < n;
    Row r;
    r.p = a.target + (long long)(first + s + acc) * a.target_stride;
    r.q = refused && a.draft ? a.draft + (long long)(first + acc) * a.draft_stride : nullptr;
    r.skip = refused && !a.draft ? a.tokens[first + acc] : -1;

    // contiguous runs, one for each warp of the cluster, of whole 128-byte lines
    const int runs = cluster * kWarps;
    const int per = ((a.vocab + runs - 1) / runs + 31) / 32 * 32;
    const int mine = rank * kWarps + warp;
    const int lo = (int)min((long long)a.vocab, (long long)mine * per), hi = (int)min((long long)a.vocab, (long long)lo + per);
    for (int pass = 0; pass < 2; ++pass) {
        const bool aligned = ((reinterpret_cast<uintptr_t>(r.p) | reinterpret_cast<uintptr_t>(r.q)) & 15u) == 0 && a.vocab % 4 == 0;
        Pair sum = r.q != nullptr ? slice_sum<true>(r, lo, hi, lane, aligned) : slice_sum<false>(r, lo, hi, lane, aligned);
#pragma unroll
        for (int o = 16; o; o >>= 1)
            sum = sum + shfl_xor(sum, o);
        if (pass == 0)
            asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
        if (lane < cluster)
            st_cluster_pair(tc::map_to_rank(&sh_run[pass][mine], lane), sum);
        tc::cluster_sync();
        if (warp == 0) {
            const Place at = find(sh_run[pass], runs, lane, 0.0, [&](double total) { return u * total; });
            if (lane == 0) {
                sh_place = at;
                sh_goal = u * at.total;
            }
        }
        __syncthreads();
        if (sh_place.total > 0.0 || (r.q == nullptr && r.skip < 0))
            break;
        r.q = nullptr;  // nothing is left of p after the draft's distribution: draw from p
        r.skip = -1;
        __syncthreads();
    }
    const int run = sh_place.at;
    if (run < 0) {  // no positive weight at all
        if (threadIdx.x == 0 && rank == 0)
            out[acc] = -1;
        return;
    }
    if (run / kWarps != rank)
        return;
    // ---- the run's owner: a warp a stretch of it, then the warp that the goal falls to
    const double before = sh_place.before, goal = sh_goal;
    const int r0 = (int)min((long long)a.vocab, (long long)run * per), r1 = (int)min((long long)a.vocab, (long long)r0 + per);
    const int each = (per + kWarps - 1) / kWarps;
    const int v0 = min(r1, r0 + warp * each), v1 = min(r1, v0 + each);
    int seg = (each + 31) / 32, s0 = min(v1, v0 + lane * seg), s1 = min(v1, s0 + seg);  // a lane's part of it
    Pair sum = {0.f, 0.f};
    int lastv = -1;
#pragma unroll 8
    for (int v = s0; v < s1; ++v) {
        const Pair w = r.at(v);
        sum = sum + w;
        lastv = w.h > 0.f ? v : lastv;
    }
    sh_lane[threadIdx.x] = sum;
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        sum = sum + shfl_xor(sum, o);
        lastv = max(lastv, __shfl_xor_sync(0xffffffffu, lastv, o));
    }
    if (lane == 0) {
        sh_part[warp] = sum;
        if (lastv >= 0)
            atomicMax(&sh_last, lastv);
    }
    __syncthreads();
    if (warp != 0)
        return;
    const Place part = find(sh_part, kWarps, lane, before, [&](double) { return goal; });
    int token = sh_last;  // the run's sum in this order may fall short of the goal by its rounding
    if (part.at >= 0) {
        // narrow the stretch down: the lanes' parts of it are summed already, then a lane
        // a token of that part (a warp that walked the stretch in steps of 32 took 8 us
        // at 600 tokens)
        double c = part.before;
        int a0 = min(r1, r0 + part.at * each), a1 = min(r1, a0 + each);
        bool last = false;  // short of the goal: the last token with a weight
        Pair w = sh_lane[part.at * 32 + lane];
        while (true) {
            s0 = min(a1, a0 + lane * seg);
            s1 = min(a1, s0 + seg);
            const double x = w.value();
            double incl = x;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const double y = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o)
                    incl += y;
            }
            const unsigned some = __ballot_sync(0xffffffffu, x > 0.0);
            const unsigned over = __ballot_sync(0xffffffffu, x > 0.0 && c + incl > goal);
            if (some == 0)
                break;
            last |= over == 0;
            const int at = last ? 31 - __clz(some) : __ffs(over) - 1;
            c += __shfl_sync(0xffffffffu, incl - x, at);
            a0 = __shfl_sync(0xffffffffu, s0, at);
            a1 = __shfl_sync(0xffffffffu, s1, at);
            if (seg <= 1) {
                token = a0;
                break;
            }
            seg = (a1 - a0 + 31) / 32;
            w = {0.f, 0.f};
            for (int v = a0 + lane * seg; v < min(a1, a0 + (lane + 1) * seg); ++v)
                w = w + r.at(v);
        }
    }
    if (lane == 0)
        out[acc] = token;
}

}  // namespace

cudaError_t launch_verify_drafts(const VerifyArgs &a, cudaStream_t stream)
{
    // CTAs for a sequence: as many as run at once, up to a cluster of eight.  256 sequences of 151936 tokens: one each 54 us, two 60, four 67;
    // 33 of 50257: eight 10.4 us, sixteen 6 us more.
    int sms = 0;
    const cudaError_t e = current_sms(&sms);
    if (e != cudaSuccess)
        return e;
    int cluster = kMaxCluster;
    while (cluster > 1 && (long long)a.num_seqs * cluster > kCtasPerSm * sms)
        cluster /= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)a.num_seqs * cluster);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    // its set-up overlaps the end of the kernel before, which it waits for
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, verify_kernel, a, cluster);
}

}  // namespace ns
