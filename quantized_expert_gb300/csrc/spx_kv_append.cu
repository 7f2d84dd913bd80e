// spx_kv_append.cu -- new tokens to the paged cache of keys and values: norm per
// head, rotation and scatter in one launch, the queries' norm and rotation with it.
//
// Elementwise but for a mean square over a head's D values, which 4 or 8 lanes
// hold in registers: bound by memory or, for few tokens, by the launch's own
// latency.  8192 tokens of 32 query and 8 key heads of 128 in bf16, norms and
// rotation: 206 MB in 37 us, 5.6 TB/s; 17 tokens 2.2 us replayed from a graph.
#include "spx_kv.cuh"

namespace spx {

namespace {

struct KvAppendParams {
    uint16_t *ck, *cv;
    int64_t page_stride, token_stride, head_stride;
    int num_pages, page_size, kv_heads, D, max_pages, B;
    const int32_t *table;
    int N, heads;  // heads: 0 without queries
    const uint16_t *k, *v, *q, *q_norm, *k_norm;
    uint16_t *q_out;
    int64_t k_stride, v_stride, q_stride, q_out_stride;
    const int32_t *req, *slot, *pos;
    float eps;
    const float *cos, *sin;
    int max_pos, P, interleaved;
    FastDiv by_page, by_sets;  // sets of heads of a row
};

template <int DT>
__device__ __forceinline__ void unpack8(float (&x)[8], uint4 v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 f = Elem<DT>::up2(w[j]);
        x[2 * j] = f.x;
        x[2 * j + 1] = f.y;
    }
}
template <int DT>
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
    return make_uint4(Elem<DT>::down2(x[0], x[1]), Elem<DT>::down2(x[2], x[3]), Elem<DT>::down2(x[4], x[5]),
                      Elem<DT>::down2(x[6], x[7]));
}

// D / 16 lanes hold a head, each two units of 8 values: of the rotated part
// units u and u + P / 16 (which hold whole pairs in either order of the pairs),
// of the rest two neighbouring ones.  They take kSet heads of a row together
// (queries, then keys, then values), so that the row's sines are read once for
// all of them.  Many tokens, more than L2 keeps for the attention that follows,
// are read and written past it (kSet = 2; the 206 MB above, us: 48.1, reads alone
// past it 48.1, writes alone 46.3, both 38.9, and in blocks of 128 threads, whose
// warps wait for fewer others at their ends, 37.0; four heads a thread 42.5, one 51.8).
constexpr int kThreads = 128;
__device__ __forceinline__ uint4 load16(const uint16_t *p, bool once) {
    return once ? __ldcs(reinterpret_cast<const uint4 *>(p)) : *reinterpret_cast<const uint4 *>(p);
}
__device__ __forceinline__ void store16(uint16_t *p, uint4 v, bool once) {
    if (once)
        __stcs(reinterpret_cast<uint4 *>(p), v);
    else
        *reinterpret_cast<uint4 *>(p) = v;
}
template <int DT, int D, int kSet>
__global__ void __launch_bounds__(kThreads, 8) kv_append_kernel(const __grid_constant__ KvAppendParams p) {
    constexpr int kLanes = D / 16;
    griddep_wait();
    griddep_launch_dependents();
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int u = threadIdx.x % kLanes, all = (int)(i / kLanes);
    const int n = p.by_sets(all), h0 = (all - n * p.by_sets.d) * kSet;
    const bool in = n < p.N;
    const int half = p.P / 16;
    const int c0 = 8 * (u < half ? u : 2 * u), c1 = u < half ? c0 + 8 * half : c0 + 8;
    // The values first, whether or not they will be wanted: where they go takes three reads one after the other.
    uint4 raw[kSet][2];
#pragma unroll
    for (int s = 0; s < kSet; ++s) {
        const int h = h0 + s, hk = h - p.heads, hv = hk - p.kv_heads;
        raw[s][0] = raw[s][1] = make_uint4(0, 0, 0, 0);
        if (!in || hv >= p.kv_heads) continue;
        const uint16_t *src = hk < 0   ? p.q + (int64_t)n * p.q_stride + (int64_t)h * D
                              : hv < 0 ? p.k + (int64_t)n * p.k_stride + (int64_t)hk * D
                                       : p.v + (int64_t)n * p.v_stride + (int64_t)hv * D;
        raw[s][0] = load16(src + c0, kSet > 1);
        raw[s][1] = load16(src + c1, kSet > 1);
    }
    const int slot = in ? __ldg(p.slot + n) : -1, pos = in ? (p.pos ? __ldg(p.pos + n) : slot) : -1;
    const bool live = slot >= 0 && pos >= 0 && !(p.cos && pos >= p.max_pos);
    // (no lane leaves: those of a head sum up its squares together)
    const bool turns = p.cos && u < half;
    int64_t place = -1;  // of the token in the cache
    if (live && h0 + kSet > p.heads) {
        const int b = __ldg(p.req + n), pi = p.by_page(slot);
        if (b >= 0 && b < p.B && pi < p.max_pages) {
            const int pg = __ldg(p.table + (size_t)b * p.max_pages + pi);
            if (pg >= 0 && pg < p.num_pages)
                place = (int64_t)pg * p.page_stride + (int64_t)(slot - pi * p.page_size) * p.token_stride;
        }
    }
    float cs[8], sn[8];
    if (turns && live) {
        // interleaved: the pairs of unit c are 4c .. 4c + 3; else those of units u and u + half are 8u .. 8u + 7
        const int a = p.interleaved ? c0 / 2 : c0, b = p.interleaved ? c1 / 2 : c0 + 4;
        const float *cr = p.cos + (int64_t)pos * (p.P / 2), *sr = p.sin + (int64_t)pos * (p.P / 2);
        const float4 x0 = __ldg(reinterpret_cast<const float4 *>(cr + a)), x1 = __ldg(reinterpret_cast<const float4 *>(cr + b));
        const float4 y0 = __ldg(reinterpret_cast<const float4 *>(sr + a)), y1 = __ldg(reinterpret_cast<const float4 *>(sr + b));
        cs[0] = x0.x; cs[1] = x0.y; cs[2] = x0.z; cs[3] = x0.w; cs[4] = x1.x; cs[5] = x1.y; cs[6] = x1.z; cs[7] = x1.w;
        sn[0] = y0.x; sn[1] = y0.y; sn[2] = y0.z; sn[3] = y0.w; sn[4] = y1.x; sn[5] = y1.y; sn[6] = y1.z; sn[7] = y1.w;
    }
#pragma unroll
    for (int s = 0; s < kSet; ++s) {
        const int h = h0 + s, hk = h - p.heads;
        const bool value = hk >= p.kv_heads;
        const uint16_t *w = value ? nullptr : hk < 0 ? p.q_norm : p.k_norm;
        float x[8], y[8];
        unpack8<DT>(x, raw[s][0]);
        unpack8<DT>(y, raw[s][1]);
        // (heads differ from lane group to lane group of a warp: the sum is made whether or not it is wanted)
        if (p.q_norm || p.k_norm) {
            float ss = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) ss = fmaf(x[j], x[j], fmaf(y[j], y[j], ss));
#pragma unroll
            for (int o = kLanes / 2; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            if (w) {
                const float inv = rsqrtf(ss / (float)D + p.eps);
                float a[8], b[8];
                unpack8<DT>(a, __ldg(reinterpret_cast<const uint4 *>(w + c0)));
                unpack8<DT>(b, __ldg(reinterpret_cast<const uint4 *>(w + c1)));
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    x[j] = x[j] * inv * a[j];
                    y[j] = y[j] * inv * b[j];
                }
            }
        }
        const int hv = hk - p.kv_heads;
        if (!live || hv >= p.kv_heads || (hk >= 0 && place < 0)) continue;
        uint16_t *dst = hk < 0   ? p.q_out + (int64_t)n * p.q_out_stride + (int64_t)h * D
                        : hv < 0 ? p.ck + place + (int64_t)hk * p.head_stride
                                 : p.cv + place + (int64_t)hv * p.head_stride;
        if (turns && !value) {
            if (p.interleaved) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float a = x[2 * j], b = x[2 * j + 1], d = y[2 * j], e = y[2 * j + 1];
                    x[2 * j] = a * cs[j] - b * sn[j];
                    x[2 * j + 1] = b * cs[j] + a * sn[j];
                    y[2 * j] = d * cs[4 + j] - e * sn[4 + j];
                    y[2 * j + 1] = e * cs[4 + j] + d * sn[4 + j];
                }
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float a = x[j], b = y[j];
                    x[j] = a * cs[j] - b * sn[j];
                    y[j] = b * cs[j] + a * sn[j];
                }
            }
        }
        // (what is neither normalised nor turned goes as it came: a NaN keeps its bits)
        const bool same = value || (!w && !turns);
        store16(dst + c0, same ? raw[s][0] : pack8<DT>(x), kSet > 1);
        store16(dst + c1, same ? raw[s][1] : pack8<DT>(y), kSet > 1);
    }
}

// Two heads a thread from what L2 keeps on (half of its 126 MB, read and
// written); below, one, for more threads and results that stay.
constexpr long long kLargeBytes = 64ll << 20;

template <int DT, int D, int kSet>
int launch_sets(KvAppendParams &p, cudaStream_t s) {
    const int sets = (p.heads + 2 * p.kv_heads + kSet - 1) / kSet;
    p.by_sets.set(sets);
    const int64_t blocks = ((int64_t)p.N * sets * (D / 16) + kThreads - 1) / kThreads;
    if (blocks * kThreads / (D / 16) > 0x7fffffffll) return SPX_ERR_UNSUPPORTED;
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = latent_config(dim3((unsigned)blocks), kThreads, 0, s, attr, 1);
    return record_launch(cudaLaunchKernelEx(&cfg, kv_append_kernel<DT, D, kSet>, p));
}
template <int DT, int D>
int launch(KvAppendParams &p, cudaStream_t s) {
    return 4ll * p.N * (p.heads + 2 * p.kv_heads) * D >= kLargeBytes ? launch_sets<DT, D, 2>(p, s) : launch_sets<DT, D, 1>(p, s);
}

}  // namespace

}  // namespace spx

using namespace spx;

extern "C" int spx_kv_append(const spx_kv_append_args *a, spx_stream_t stream) {
    if (!a) return SPX_ERR_INVALID_ARG;
    const int st = kv_cache_check(a->cache);
    if (st) return st;
    const spx_kv_cache &c = *a->cache;
    if (c.k == c.v || a->N < 0 || !a->cos != !a->sin || !a->q != !a->q_out || (a->q_norm && !a->q)) return SPX_ERR_INVALID_ARG;
    if (a->cos && (a->max_pos < 1 || !al16(a->cos) || !al16(a->sin))) return SPX_ERR_INVALID_ARG;
    if (a->cos && (a->P < 16 || a->P > c.D || a->P % 16)) return SPX_ERR_UNSUPPORTED;
    if ((a->q_norm || a->k_norm) && !(a->eps >= 0.f)) return SPX_ERR_INVALID_ARG;
    const int64_t kw = (int64_t)c.kv_heads * c.D;
    if (!al16(a->k) || !al16(a->v) || !al16(a->q_norm) || !al16(a->k_norm) || a->k_stride < kw || a->v_stride < kw ||
        a->k_stride % 8 || a->v_stride % 8)
        return SPX_ERR_INVALID_ARG;
    if (a->q) {
        const int64_t w = (int64_t)a->heads * c.D;
        if (a->heads < 1 || a->q_stride < w || a->q_out_stride < w || a->q_stride % 8 || a->q_out_stride % 8 ||
            !al16(a->q) || !al16(a->q_out) || (a->q == a->q_out && a->q_stride != a->q_out_stride))
            return SPX_ERR_INVALID_ARG;
        if (a->heads > 1024) return SPX_ERR_UNSUPPORTED;
    }
    if (a->N == 0) return SPX_OK;
    if (!a->k || !a->v || !a->req || !a->slot) return SPX_ERR_INVALID_ARG;
    KvAppendParams p{};
    p.ck = static_cast<uint16_t *>(c.k);
    p.cv = static_cast<uint16_t *>(c.v);
    p.page_stride = c.page_stride;
    p.token_stride = c.token_stride;
    p.head_stride = c.head_stride;
    p.num_pages = c.num_pages;
    p.page_size = c.page_size;
    p.kv_heads = c.kv_heads;
    p.D = c.D;
    p.max_pages = c.max_pages;
    p.B = c.B;
    p.table = c.block_table;
    p.N = a->N;
    p.heads = a->q ? a->heads : 0;
    p.k = static_cast<const uint16_t *>(a->k);
    p.v = static_cast<const uint16_t *>(a->v);
    p.q = static_cast<const uint16_t *>(a->q);
    p.q_norm = static_cast<const uint16_t *>(a->q_norm);
    p.k_norm = static_cast<const uint16_t *>(a->k_norm);
    p.q_out = static_cast<uint16_t *>(a->q_out);
    p.k_stride = a->k_stride;
    p.v_stride = a->v_stride;
    p.q_stride = a->q_stride;
    p.q_out_stride = a->q_out_stride;
    p.req = a->req;
    p.slot = a->slot;
    p.pos = a->pos;
    p.eps = a->eps;
    p.cos = a->cos;
    p.sin = a->sin;
    p.max_pos = a->max_pos;
    p.P = a->cos ? a->P : 0;
    p.interleaved = a->interleaved;
    p.by_page.set(c.page_size);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (c.D == 128) return c.dtype == SPX_F16 ? launch<SPX_F16, 128>(p, s) : launch<SPX_BF16, 128>(p, s);
    return c.dtype == SPX_F16 ? launch<SPX_F16, 64>(p, s) : launch<SPX_BF16, 64>(p, s);
}
