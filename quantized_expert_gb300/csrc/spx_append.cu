// spx_append.cu -- new tokens to the paged latent cache: norm, rotation and
// scatter in one launch, the queries' rotation with it.
//
// Elementwise but for one mean square over R <= 512 values, which a warp holds
// in registers: every input is read once and every output written once, so the
// launch is bound by memory (8192 tokens of 16 heads in bf16: 122 MB in 25 us,
// 4.9 TB/s, five sixths of it the queries, in order) or by its latency (17 tokens:
// 3.6 us in a stream of calls, 2.7 replayed from a graph).
#include "spx_latent.cuh"

namespace spx {

int latent_cache_check(const spx_latent_cache *c);

namespace {

struct AppendParams {
    uint16_t *cache;
    int64_t page_stride, token_stride;
    int num_pages, page_size, R, P, max_pages, B;
    const int32_t *table;
    int N;
    const uint16_t *kv, *w_norm, *q;
    uint16_t *q_out;
    int64_t kv_stride, q_stride, q_out_stride;
    const int32_t *req, *pos;
    float eps;
    const float *cos, *sin;
    int max_pos, interleaved, heads, q_width;
    int kv_blocks, copy_blocks;
    int64_t copies;              // units of all queries to copy (none in place)
    FastDiv by_units, by_heads;  // units to copy per head, heads
};

// Rotation of 16 values of a 64-wide part, its units of 8 values u and u + 4
// (u < 4), in place: both hold whole pairs in either order of the pairs.
__device__ __forceinline__ void rotate16(float (&x)[8], float (&y)[8], int u, bool interleaved, const float *cs,
                                         const float *sn) {
    const int i0 = interleaved ? 4 * u : 8 * u, i1 = interleaved ? 16 + 4 * u : 8 * u + 4;
    const float4 c0 = __ldg(reinterpret_cast<const float4 *>(cs + i0)), c1 = __ldg(reinterpret_cast<const float4 *>(cs + i1));
    const float4 s0 = __ldg(reinterpret_cast<const float4 *>(sn + i0)), s1 = __ldg(reinterpret_cast<const float4 *>(sn + i1));
    const float c[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
    const float s[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
    if (interleaved) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float a = x[2 * j], b = x[2 * j + 1], d = y[2 * j], e = y[2 * j + 1];
            x[2 * j] = a * c[j] - b * s[j];
            x[2 * j + 1] = b * c[j] + a * s[j];
            y[2 * j] = d * c[4 + j] - e * s[4 + j];
            y[2 * j + 1] = e * c[4 + j] + d * s[4 + j];
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float a = x[j], b = y[j];
            x[j] = a * c[j] - b * s[j];
            y[j] = b * c[j] + a * s[j];
        }
    }
}

template <int DT>
__device__ __forceinline__ void load8(float (&x)[8], const uint16_t *p) {
    const uint4 v = *reinterpret_cast<const uint4 *>(p);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 f = Elem<DT>::up2(w[j]);
        x[2 * j] = f.x;
        x[2 * j + 1] = f.y;
    }
}
template <int DT>
__device__ __forceinline__ void store8(uint16_t *p, const float (&x)[8]) {
    *reinterpret_cast<uint4 *>(p) = make_uint4(Elem<DT>::down2(x[0], x[1]), Elem<DT>::down2(x[2], x[3]),
                                               Elem<DT>::down2(x[4], x[5]), Elem<DT>::down2(x[6], x[7]));
}

// Blocks below kv_blocks: a warp per cache row (lane l holds the values 8l on
// and, for R > 256, 256 + 8l on; lanes 0-3 also the rotated part).  Then the
// queries in units of 8 values: blocks that copy, four units a thread, and
// blocks that rotate, two units (u and u + 4 of a head's rotated part).  A warp
// per head moved 384 bytes at a time and was bound by its instructions (8192
// tokens 67 us); copies and rotations in one warp took turns (31 us).
constexpr int kUnitsPerThread = 4;
template <int DT>
__global__ void __launch_bounds__(256) latent_append_kernel(const __grid_constant__ AppendParams p) {
    const int lane = threadIdx.x & 31;
    griddep_wait();
    griddep_launch_dependents();
    if ((int)blockIdx.x < p.kv_blocks) {
        const int n = (int)blockIdx.x * 8 + (threadIdx.x >> 5);
        if (n >= p.N) return;
        const int pos = __ldg(p.pos + n), b = __ldg(p.req + n), pi = pos / p.page_size;
        if (pos < 0 || (p.cos && pos >= p.max_pos) || b < 0 || b >= p.B || pi >= p.max_pages) return;
        const int pg = __ldg(p.table + (size_t)b * p.max_pages + pi);
        if (pg < 0 || pg >= p.num_pages) return;
        const uint16_t *src = p.kv + (int64_t)n * p.kv_stride;
        uint16_t *dst = p.cache + (int64_t)pg * p.page_stride + (int64_t)(pos - pi * p.page_size) * p.token_stride;
        float x[2][8], r0[8], r1[8], ss = 0.f;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int c0 = 256 * i + 8 * lane;
            if (c0 < p.R) {
                load8<DT>(x[i], src + c0);
#pragma unroll
                for (int j = 0; j < 8; ++j) ss = fmaf(x[i][j], x[i][j], ss);
            }
        }
        if (lane < 4) {
            load8<DT>(r0, src + p.R + 8 * lane);
            load8<DT>(r1, src + p.R + 32 + 8 * lane);
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const float inv = p.w_norm ? rsqrtf(ss / (float)p.R + p.eps) : 1.f;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int c0 = 256 * i + 8 * lane;
            if (c0 < p.R) {
                if (p.w_norm) {
                    float w[8];
                    load8<DT>(w, p.w_norm + c0);
#pragma unroll
                    for (int j = 0; j < 8; ++j) x[i][j] = x[i][j] * inv * w[j];
                }
                store8<DT>(dst + c0, x[i]);
            }
        }
        if (lane < 4) {
            if (p.cos) rotate16(r0, r1, lane, p.interleaved, p.cos + (size_t)pos * 32, p.sin + (size_t)pos * 32);
            store8<DT>(dst + p.R + 8 * lane, r0);
            store8<DT>(dst + p.R + 32 + 8 * lane, r1);
        }
        return;
    }
    if (blockIdx.x < (unsigned)(p.kv_blocks + p.copy_blocks)) {  // copies: q_width / 8 - 8 units a head
        const int64_t first = (int64_t)(blockIdx.x - p.kv_blocks) * (256 * kUnitsPerThread) + threadIdx.x;
        uint4 v[kUnitsPerThread];
        uint4 *dst[kUnitsPerThread];
#pragma unroll
        for (int k = 0; k < kUnitsPerThread; ++k) {
            const int64_t i = first + 256 * k;
            dst[k] = nullptr;
            if (i >= p.copies) continue;
            const int head = p.by_units((int)i), n = p.by_heads(head), h = head - n * p.heads;  // of all heads; token
            const int at = 8 * ((int)i - head * p.by_units.d), pos = __ldg(p.pos + n);
            if (pos < 0 || (p.cos && pos >= p.max_pos)) continue;
            dst[k] = reinterpret_cast<uint4 *>(p.q_out + (int64_t)n * p.q_out_stride + (int64_t)h * p.q_width + at);
            v[k] = *reinterpret_cast<const uint4 *>(p.q + (int64_t)n * p.q_stride + (int64_t)h * p.q_width + at);
        }
#pragma unroll
        for (int k = 0; k < kUnitsPerThread; ++k)
            if (dst[k]) *dst[k] = v[k];
        return;
    }
    // rotations: 4 a head
    const int64_t i = (int64_t)(blockIdx.x - p.kv_blocks - p.copy_blocks) * 256 + threadIdx.x;
    const int head = (int)(i >> 2), u = (int)i & 3, n = p.by_heads(head), h = head - n * p.heads;
    if (n >= p.N) return;
    const int pos = __ldg(p.pos + n);
    if (pos < 0 || (p.cos && pos >= p.max_pos)) return;
    const int at = p.q_width - 64 + 8 * u;
    const uint16_t *src = p.q + (int64_t)n * p.q_stride + (int64_t)h * p.q_width + at;
    uint16_t *dst = p.q_out + (int64_t)n * p.q_out_stride + (int64_t)h * p.q_width + at;
    float x[8], y[8];
    load8<DT>(x, src);
    load8<DT>(y, src + 32);
    if (p.cos) rotate16(x, y, u, p.interleaved, p.cos + (size_t)pos * 32, p.sin + (size_t)pos * 32);
    store8<DT>(dst, x);
    store8<DT>(dst + 32, y);
}

bool al16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

}  // namespace

}  // namespace spx

using namespace spx;

extern "C" int spx_latent_append(const spx_latent_append_args *a, spx_stream_t stream) {
    if (!a) return SPX_ERR_INVALID_ARG;
    int st = latent_cache_check(a->cache);
    if (st) return st;
    const spx_latent_cache &c = *a->cache;
    if (a->N < 0 || !a->cos != !a->sin) return SPX_ERR_INVALID_ARG;
    if (a->N == 0) return SPX_OK;
    if (!a->kv || !a->req || !a->pos) return SPX_ERR_INVALID_ARG;
    if (a->kv_stride < c.R + c.P || a->kv_stride % 8 || !al16(a->kv) || !al16(a->w_norm)) return SPX_ERR_INVALID_ARG;
    if (a->cos && (a->max_pos < 1 || !al16(a->cos) || !al16(a->sin))) return SPX_ERR_INVALID_ARG;
    if (!a->q != !a->q_out) return SPX_ERR_INVALID_ARG;
    if (a->q) {
        const int64_t w = (int64_t)a->heads * a->q_width;
        if (a->heads < 1 || a->q_width < c.P || a->q_width % 8 || a->q_stride < w || a->q_out_stride < w ||
            a->q_stride % 8 || a->q_out_stride % 8 || !al16(a->q) || !al16(a->q_out))
            return SPX_ERR_INVALID_ARG;
        if (a->q == a->q_out && a->q_stride != a->q_out_stride) return SPX_ERR_INVALID_ARG;
    }
    // in place only the rotated parts move
    const int per_head = a->q && a->q != a->q_out ? (a->q_width - c.P) / 8 : 0;
    const long long heads = a->q ? (long long)a->N * a->heads : 0, copies = heads * per_head;
    if (copies > 0x7ffffffell || heads > 0x1fffffffll) return SPX_ERR_UNSUPPORTED;
    const long long kv_blocks = ((long long)a->N + 7) / 8;
    const long long copy_blocks = (copies + 256 * kUnitsPerThread - 1) / (256 * kUnitsPerThread);
    const long long blocks = kv_blocks + copy_blocks + (4 * heads + 255) / 256;
    AppendParams p{};
    p.cache = static_cast<uint16_t *>(c.cache);
    p.page_stride = c.page_stride;
    p.token_stride = c.token_stride;
    p.num_pages = c.num_pages;
    p.page_size = c.page_size;
    p.R = c.R;
    p.P = c.P;
    p.max_pages = c.max_pages;
    p.B = c.B;
    p.table = c.block_table;
    p.N = a->N;
    p.kv = static_cast<const uint16_t *>(a->kv);
    p.w_norm = static_cast<const uint16_t *>(a->w_norm);
    p.q = static_cast<const uint16_t *>(a->q);
    p.q_out = static_cast<uint16_t *>(a->q_out);
    p.kv_stride = a->kv_stride;
    p.q_stride = a->q_stride;
    p.q_out_stride = a->q_out_stride;
    p.req = a->req;
    p.pos = a->pos;
    p.eps = a->eps;
    p.cos = a->cos;
    p.sin = a->sin;
    p.max_pos = a->max_pos;
    p.interleaved = a->interleaved;
    p.heads = a->heads;
    p.q_width = a->q_width;
    p.kv_blocks = (int)kv_blocks;
    p.copy_blocks = (int)copy_blocks;
    p.copies = copies;
    p.by_units.set(per_head ? per_head : 1);
    p.by_heads.set(a->q ? a->heads : 1);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = latent_config(dim3((unsigned)blocks), 256, 0, s, attr, 1);
    return record_launch(c.dtype == SPX_F16 ? cudaLaunchKernelEx(&cfg, latent_append_kernel<SPX_F16>, p)
                                            : cudaLaunchKernelEx(&cfg, latent_append_kernel<SPX_BF16>, p));
}
