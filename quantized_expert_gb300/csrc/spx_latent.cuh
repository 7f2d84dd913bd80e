// spx_latent.cuh -- what the latent-attention launches share: element types,
// the parameter block and the decoding of a request's rows and pages.
#pragma once

#include <cuda_bf16.h>

#include "spx_internal.cuh"

namespace spx {

// Element type by its spx_dtype: conversions to and from fp32, one rounding; of
// two packed values, a product and sum, and what replaces one that is not finite.
template <int DT>
struct Elem;
template <>
struct Elem<SPX_F16> {
    using T = __half;
    static __device__ __forceinline__ float up(T v) { return __half2float(v); }
    static __device__ __forceinline__ T down(float v) { return __float2half_rn(v); }
    static __device__ __forceinline__ float2 up2(uint32_t v) { return __half22float2(*reinterpret_cast<__half2 *>(&v)); }
    static __device__ __forceinline__ uint32_t down2(float a, float b) {
        __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<uint32_t *>(&h);
    }
    static __device__ __forceinline__ uint32_t fma2(uint32_t a, uint32_t b, uint32_t c) {
        uint32_t r;
        asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
        return r;
    }
    static __device__ __forceinline__ uint32_t finite2(uint32_t v, uint32_t other) {
        if ((v & 0x7C00u) == 0x7C00u) v = (v & 0xFFFF0000u) | (other & 0xFFFFu);
        if ((v & 0x7C000000u) == 0x7C000000u) v = (v & 0xFFFFu) | (other & 0xFFFF0000u);
        return v;
    }
};
template <>
struct Elem<SPX_BF16> {
    using T = __nv_bfloat16;
    static __device__ __forceinline__ float up(T v) { return __bfloat162float(v); }
    static __device__ __forceinline__ T down(float v) { return __float2bfloat16_rn(v); }
    static __device__ __forceinline__ float2 up2(uint32_t v) {
        return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
    }
    static __device__ __forceinline__ uint32_t down2(float a, float b) {
        __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<uint32_t *>(&h);
    }
    static __device__ __forceinline__ uint32_t fma2(uint32_t a, uint32_t b, uint32_t c) {
        uint32_t r;
        asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
        return r;
    }
    static __device__ __forceinline__ uint32_t finite2(uint32_t v, uint32_t other) {
        if ((v & 0x7F80u) == 0x7F80u) v = (v & 0xFFFF0000u) | (other & 0xFFFFu);
        if ((v & 0x7F800000u) == 0x7F800000u) v = (v & 0xFFFFu) | (other & 0xFFFF0000u);
        return v;
    }
};
template <>
struct Elem<SPX_F32> {
    using T = float;
    static __device__ __forceinline__ float up(T v) { return v; }
    static __device__ __forceinline__ T down(float v) { return v; }
};

// Quotients by a divisor known to the host: q = (hi(x m) + x) >> s, exact for
// 0 <= x < 2^31 (m = floor(2^32 (2^s - d) / d) + 1, 2^s the least power >= d).
struct FastDiv {
    uint32_t m, s;
    int d;
    void set(int div) {
        d = div;
        s = 0;
        while ((1ull << s) < (uint64_t)div) ++s;
        m = (uint32_t)((((1ull << s) - (uint64_t)div) << 32) / (uint64_t)div + 1);
    }
    __device__ __forceinline__ int operator()(int x) const { return (int)((__umulhi((uint32_t)x, m) + (uint32_t)x) >> s); }
};

// Two fp32 values in one 64-bit register and the instructions that take them.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

struct LatentParams {
    // cache
    const uint16_t *cache;
    int64_t page_stride, token_stride;
    int num_pages, page_size, R, P;
    const int32_t *table;
    int max_pages, B;
    const int32_t *lens;
    // call
    int N, heads, max_q, max_len, dn, dv, causal;  // max_len: within the block table too
    FastDiv by_heads, by_page;
    int64_t q_stride, out_stride;
    const int32_t *q_start;
    const uint16_t *q, *w_uk, *w_uv;
    uint16_t *out;
    float *lse;
    float scale, scale_log2;  // scale_log2 = scale * log2(e)
    // workspace
    WsHeader *hdr;
    uint64_t budget;
    uint16_t *q_lat;  // [N][heads][R + P]
    float *o_lat;     // [N][heads][R]: rows of units that one share holds whole
    int4 *units;      // [B][groups]: first and last block of its shares, first slot, whole
    float2 *ml;       // [slots][nr]: reference and weight of a partial sum
    float *part;      // [slots][nr][R]: partial sums; block c has slots 2c (its first unit) and 2c + 1 (its last)
    // geometry of the attention launch
    int nr, nr_log2, groups, box_tokens;
    int chained;      // a launch of this call precedes the attention launch
    // expanded form: keys, values [heads][B][kv_rows][128], rotated parts [B][kv_rows][64]
    uint16_t *k_x, *v_x, *rope_x;
    int kv_rows, head_group;  // rows of a request (whole tiles); heads per block of the expand launch
};

// A request's query rows and cached length, cut to the call's bounds, so that
// no content of q_start or lens leads out of a buffer.
struct LatentReq {
    int row0, T, len;
};
__device__ __forceinline__ LatentReq latent_req(const LatentParams &p, int b) {
    LatentReq r;
    const int s = __ldg(p.q_start + b), e = __ldg(p.q_start + b + 1);
    r.row0 = min(max(s, 0), p.N);
    r.T = min(min(max(e - r.row0, 0), p.max_q), p.N - r.row0);
    r.len = min(max(__ldg(p.lens + b), 0), p.max_len);
    return r;
}
// Positions that token t of the request sees: [0, limit).
__device__ __forceinline__ int latent_limit(const LatentParams &p, const LatentReq &r, int t) {
    return p.causal ? max(r.len - r.T + t + 1, 0) : r.len;
}

// Where a role of a block gave up, what is in flight is waited for, this long at
// most, before shared and tensor memory are given back: once every role has left
// its loops, as those that had nothing more to wait for may have issued copies
// and products all the same.
constexpr uint64_t kSettleNs = 100000000ull;

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.aligned;" ::: "memory"); }
// Without the order of what was stored before (which waits for global stores).
__device__ __forceinline__ void cluster_arrive_relaxed() {
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.aligned;" ::: "memory"); }

// -------------------------------------------------------------------- host --
inline cudaLaunchConfig_t latent_config(dim3 grid, int threads, size_t smem, cudaStream_t s, cudaLaunchAttribute *attr,
                                        int cluster) {
    cudaLaunchConfig_t c = {};
    c.gridDim = grid;
    c.blockDim = dim3(threads);
    c.dynamicSmemBytes = smem;
    c.stream = s;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    c.attrs = attr;
    c.numAttrs = cluster > 1 ? 2 : 1;
    return c;
}

// The most dynamic shared memory that a kernel's launches ask for, set once per
// device and thread.
template <auto kernel>
int set_smem(size_t bytes) {
    static thread_local int done_dev = -1;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return record_launch(e);
    if (done_dev == dev) return SPX_OK;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e != cudaSuccess) return record_launch(e);
    done_dev = dev;
    return SPX_OK;
}

// spx_latent_prompt.cu: the expanded form's launches.
int launch_expanded(LatentParams &p, int dt, cudaStream_t s);

}  // namespace spx
