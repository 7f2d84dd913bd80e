// spx_append.cu -- new tokens to the paged latent cache: norm, rotation and
// scatter in one launch, the queries' rotation with it.
//
// Elementwise but for one mean square over R <= 512 values, which a warp holds
// in registers: every input is read once and every output written once, so the
// launch is bound by memory (prompts) or by its latency (a verify pass).
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
};

// Rotation of the pairs held in 8 consecutive values x[i0 .. i0 + 8) of a
// P-wide part; `o` are the values at the partner half when not interleaved.
__device__ __forceinline__ void rotate8(float (&x)[8], const float (&o)[8], int i0, int P, bool inter, const float *cs,
                                        const float *sn) {
    if (inter) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float c = __ldg(cs + i0 / 2 + j), s = __ldg(sn + i0 / 2 + j);
            const float a = x[2 * j], b = x[2 * j + 1];
            x[2 * j] = a * c - b * s;
            x[2 * j + 1] = b * c + a * s;
        }
    } else {
        const bool second = i0 >= P / 2;
        const int k = second ? i0 - P / 2 : i0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float c = __ldg(cs + k + j), s = __ldg(sn + k + j);
            x[j] = second ? x[j] * c + o[j] * s : x[j] * c - o[j] * s;
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

// One warp per task: task n < N is the cache row of token n (lane l holds the
// values 8l and, for R > 256, 256 + 8l on; lanes 0-7 then take the rotated
// part); the others are one head of a token's queries each.
template <int DT>
__global__ void __launch_bounds__(256) latent_append_kernel(AppendParams p) {
    const long long task = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    const long long ntask = p.N + (p.q ? (long long)p.N * p.heads : 0);
    if (task >= ntask) return;
    const int n = (int)(task < p.N ? task : (task - p.N) / p.heads);
    const int pos = __ldg(p.pos + n);
    if (pos < 0 || (p.cos && pos >= p.max_pos)) return;
    const float *cs = p.cos ? p.cos + (size_t)pos * (p.P / 2) : nullptr;
    const float *sn = p.cos ? p.sin + (size_t)pos * (p.P / 2) : nullptr;
    if (task < p.N) {
        const int b = __ldg(p.req + n), pi = pos / p.page_size;
        if (b < 0 || b >= p.B || pi >= p.max_pages) return;
        const int pg = __ldg(p.table + (size_t)b * p.max_pages + pi);
        if (pg < 0 || pg >= p.num_pages) return;
        const uint16_t *src = p.kv + (int64_t)n * p.kv_stride;
        uint16_t *dst = p.cache + (int64_t)pg * p.page_stride + (int64_t)(pos - pi * p.page_size) * p.token_stride;
        float x[2][8], rot[8], oth[8], ss = 0.f;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int c0 = 256 * i + 8 * lane;
            if (c0 < p.R) {
                load8<DT>(x[i], src + c0);
#pragma unroll
                for (int j = 0; j < 8; ++j) ss = fmaf(x[i][j], x[i][j], ss);
            }
        }
        if (lane < p.P / 8) {
            load8<DT>(rot, src + p.R + 8 * lane);
            load8<DT>(oth, src + p.R + (8 * lane + p.P / 2) % p.P);
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
        if (lane < p.P / 8) {
            if (cs) rotate8(rot, oth, 8 * lane, p.P, p.interleaved, cs, sn);
            store8<DT>(dst + p.R + 8 * lane, rot);
        }
        return;
    }
    const int h = (int)((task - p.N) % p.heads);
    const uint16_t *src = p.q + (int64_t)n * p.q_stride + (int64_t)h * p.q_width;
    uint16_t *dst = p.q_out + (int64_t)n * p.q_out_stride + (int64_t)h * p.q_width;
    const int r0 = p.q_width - p.P;
    if (src != dst)
        for (int c0 = 8 * lane; c0 < r0; c0 += 256) *reinterpret_cast<uint4 *>(dst + c0) = *reinterpret_cast<const uint4 *>(src + c0);
    float x[8], oth[8];
    if (lane < p.P / 8) {
        load8<DT>(x, src + r0 + 8 * lane);
        load8<DT>(oth, src + r0 + (8 * lane + p.P / 2) % p.P);
    }
    __syncwarp();  // in place: every lane's loads before any lane's store
    if (lane < p.P / 8) {
        if (cs) rotate8(x, oth, 8 * lane, p.P, p.interleaved, cs, sn);
        store8<DT>(dst + r0 + 8 * lane, x);
    }
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
    const long long tasks = (long long)a->N * (a->q ? 1 + a->heads : 1), blocks = (tasks + 7) / 8;
    if (blocks > 0x7fffffffll) return SPX_ERR_UNSUPPORTED;
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
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (c.dtype == SPX_F16)
        latent_append_kernel<SPX_F16><<<(unsigned)blocks, 256, 0, s>>>(p);
    else
        latent_append_kernel<SPX_BF16><<<(unsigned)blocks, 256, 0, s>>>(p);
    return record_launch(cudaGetLastError());
}
