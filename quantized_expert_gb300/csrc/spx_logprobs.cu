// spx_logprobs.cu -- log probabilities of given tokens, entropy and the most
// likely alternatives of rows of logits.
#include "spx_latent.cuh"

#include <math.h>

namespace spx {

namespace {

struct LogprobParams {
    const void *logits;
    int64_t stride;
    int N, V, k;
    const int32_t *ids;
    float *logp, *entropy, *top_logp;
    int32_t *top_ids;
};

// Order of the alternatives as one 64-bit key: the value first (larger is
// larger, -0 = +0, NaN above all), then the lower index.
__device__ __forceinline__ uint32_t order32(float x) {
    if (x != x) return 0xFFFFFFFFu;
    const uint32_t u = __float_as_uint(x + 0.f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ uint64_t order64(float x, int v) {
    return ((uint64_t)order32(x) << 32) | (uint32_t)~v;
}

// One block per row: one pass for the statistics, one per alternative.
template <int DT>
__global__ void __launch_bounds__(1024) logprobs_kernel(LogprobParams p) {
    using E = Elem<DT>;
    const typename E::T *x = static_cast<const typename E::T *>(p.logits) + (int64_t)blockIdx.x * p.stride;
    __shared__ float sm[32], sz[32], sd[32];
    __shared__ uint64_t sk[32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float m = -INFINITY;
    bool nan = false;
    for (int v = threadIdx.x; v < p.V; v += 1024) {
        const float f = E::up(x[v]);
        nan |= f != f;
        m = fmaxf(m, f);
    }
    nan = __syncthreads_or(nan);
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (lane == 0) sm[warp] = m;
    __syncthreads();
    for (int w = 0; w < 32; ++w) m = fmaxf(m, sm[w]);
    const float ref = m == -INFINITY ? 0.f : m;
    float z = 0.f, d = 0.f;
    for (int v = threadIdx.x; v < p.V; v += 1024) {
        const float t = E::up(x[v]) - ref, e = expf(t);
        z += e;
        d += e > 0.f ? e * t : 0.f;
    }
    for (int o = 16; o; o >>= 1) {
        z += __shfl_xor_sync(0xffffffffu, z, o);
        d += __shfl_xor_sync(0xffffffffu, d, o);
    }
    if (lane == 0) {
        sz[warp] = z;
        sd[warp] = d;
    }
    __syncthreads();
    z = d = 0.f;
    for (int w = 0; w < 32; ++w) {
        z += sz[w];
        d += sd[w];
    }
    const bool none = m == -INFINITY && !nan;
    const float log_z = nan ? NAN : none ? 0.f : m == INFINITY ? m : m + logf(z);
    if (threadIdx.x == 0) {
        if (p.logp) {
            const int id = p.ids[blockIdx.x];
            p.logp[blockIdx.x] = id >= 0 && id < p.V ? E::up(x[id]) - log_z : NAN;
        }
        if (p.entropy) p.entropy[blockIdx.x] = nan ? NAN : none ? 0.f : logf(z) - d / z;
    }
    uint64_t last = ~0ull;
    for (int j = 0; j < p.k; ++j) {
        uint64_t best = 0;
        for (int v = threadIdx.x; v < p.V; v += 1024) {
            const uint64_t key = order64(E::up(x[v]), v);
            if (key < last && key > best) best = key;
        }
        for (int o = 16; o; o >>= 1) best = max(best, __shfl_xor_sync(0xffffffffu, best, o));
        __syncthreads();
        if (lane == 0) sk[warp] = best;
        __syncthreads();
        for (int w = 0; w < 32; ++w) best = max(best, sk[w]);
        last = best;
        if (threadIdx.x == 0) {
            const int v = (int)~(uint32_t)best;
            p.top_ids[(size_t)blockIdx.x * p.k + j] = v;
            p.top_logp[(size_t)blockIdx.x * p.k + j] = E::up(x[v]) - log_z;
        }
    }
}

}  // namespace

}  // namespace spx

using namespace spx;

extern "C" int spx_token_logprobs(const spx_logprobs_args *a, spx_stream_t stream) {
    if (!a || a->N < 0 || a->V < 1 || a->k < 0 || a->k > a->V) return SPX_ERR_INVALID_ARG;
    if (a->dtype != SPX_F16 && a->dtype != SPX_BF16 && a->dtype != SPX_F32) return SPX_ERR_UNSUPPORTED;
    if (a->k > 32) return SPX_ERR_UNSUPPORTED;
    if (a->N == 0) return SPX_OK;
    if (!a->logits || a->stride < a->V || !a->ids != !a->logp || (a->k > 0) != (a->top_ids != nullptr) ||
        (a->k > 0) != (a->top_logp != nullptr))
        return SPX_ERR_INVALID_ARG;
    const uintptr_t es = a->dtype == SPX_F32 ? 4 : 2;
    if (reinterpret_cast<uintptr_t>(a->logits) % es) return SPX_ERR_INVALID_ARG;
    LogprobParams p{a->logits, a->stride, a->N, a->V, a->k, a->ids, a->logp, a->entropy, a->top_logp, a->top_ids};
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (a->dtype == SPX_F16)
        logprobs_kernel<SPX_F16><<<a->N, 1024, 0, s>>>(p);
    else if (a->dtype == SPX_BF16)
        logprobs_kernel<SPX_BF16><<<a->N, 1024, 0, s>>>(p);
    else
        logprobs_kernel<SPX_F32><<<a->N, 1024, 0, s>>>(p);
    return record_launch(cudaGetLastError());
}
