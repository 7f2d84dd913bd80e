// spx_latent.cu -- attention over the paged latent cache, absorbed form.
//
// With k[h] = (W_uk[h] c, r) and v[h] = W_uv[h] c the products with the
// up-projections move out of the sum over the cache:
//   q_nope . (W_uk c) = (q_nope W_uk) . c,   sum_p w_p W_uv c_p = W_uv sum_p w_p c_p,
// so the cached (c, r) is read once for all heads.  Three launches: queries to
// latent space, attention there, results through W_uv.
#include "spx_latent.cuh"

#include <math.h>

namespace spx {

namespace {

constexpr int kRows = 4;  // (token, head) rows of one block

template <int DT>
__global__ void __launch_bounds__(128) latent_q_kernel(LatentParams p) {
    using E = Elem<DT>;
    using T = typename E::T;
    const size_t row = blockIdx.x;
    const int h = (int)(row % p.heads);
    const T *q = reinterpret_cast<const T *>(p.q) + (row / p.heads) * p.q_stride + (size_t)h * (p.dn + p.P);
    T *dst = reinterpret_cast<T *>(p.q_lat) + row * (p.R + p.P);
    const T *w = reinterpret_cast<const T *>(p.w_uk) + (size_t)h * p.dn * p.R;
    for (int r = threadIdx.x; r < p.R; r += blockDim.x) {
        float s = 0.f;
        for (int d = 0; d < p.dn; ++d) s = fmaf(E::up(q[d]), E::up(w[(size_t)d * p.R + r]), s);
        dst[r] = E::down(s);
    }
    for (int i = threadIdx.x; i < p.P; i += blockDim.x) dst[p.R + i] = q[p.dn + i];
}

// One block: kRows rows of one request, a warp per cached token, online
// softmax per warp, the warps' sums joined at the end.
template <int DT>
__global__ void __launch_bounds__(256) latent_rows_kernel(LatentParams p) {
    using E = Elem<DT>;
    using T = typename E::T;
    const LatentReq rq = latent_req(p, blockIdx.y);
    const int nrows = rq.T * p.heads, r0 = blockIdx.x * kRows;
    if (r0 >= nrows) return;
    __shared__ float qs[kRows][576];
    __shared__ float ml[8][kRows][2];
    __shared__ float os[8][512];
    const int D = p.R + p.P, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const T *ql = p.w_uk ? reinterpret_cast<const T *>(p.q_lat) : reinterpret_cast<const T *>(p.q);
    int lim[kRows], most = 0;
    for (int i = 0; i < kRows; ++i) {
        const int r = min(r0 + i, nrows - 1), t = r / p.heads, h = r - t * p.heads;
        lim[i] = latent_limit(p, rq, t);
        most = max(most, lim[i]);
        const size_t n = rq.row0 + t;
        const T *src = p.w_uk ? ql + (n * p.heads + h) * D : ql + n * p.q_stride + (size_t)h * D;
        for (int d = threadIdx.x; d < D; d += blockDim.x) qs[i][d] = E::up(src[d]) * p.scale_log2;
    }
    __syncthreads();
    float m[kRows], l[kRows], o[kRows][16];
    for (int i = 0; i < kRows; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.f;
        for (int d = 0; d < 16; ++d) o[i][d] = 0.f;
    }
    for (int j = warp; j < most; j += 8) {
        const int pg = __ldg(p.table + (size_t)blockIdx.y * p.max_pages + j / p.page_size);
        float kv[18];
        const bool ok = pg >= 0 && pg < p.num_pages;
        const T *src = reinterpret_cast<const T *>(p.cache) + (int64_t)(ok ? pg : 0) * p.page_stride +
                       (int64_t)(j % p.page_size) * p.token_stride;
#pragma unroll
        for (int d = 0; d < 18; ++d) kv[d] = (ok && 32 * d + lane < D) ? E::up(src[32 * d + lane]) : 0.f;
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            if (j >= lim[i]) continue;
            float s = 0.f;
#pragma unroll
            for (int d = 0; d < 18; ++d)
                if (32 * d + lane < D) s = fmaf(qs[i][32 * d + lane], kv[d], s);
#pragma unroll
            for (int off = 16; off; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
            const float mn = fmaxf(m[i], s), ref = mn == -INFINITY ? 0.f : mn;
            const float c = exp2f(m[i] - ref), w = exp2f(s - ref);
            l[i] = l[i] * c + w;
#pragma unroll
            for (int d = 0; d < 16; ++d) o[i][d] = o[i][d] * c + w * kv[d];
            m[i] = mn;
        }
    }
    for (int i = 0; i < kRows; ++i) {
        if (lane == 0) {
            ml[warp][i][0] = m[i];
            ml[warp][i][1] = l[i];
        }
    }
    for (int i = 0; i < kRows; ++i) {
        __syncthreads();
        for (int d = 0; d < 16; ++d) os[warp][32 * d + lane] = o[i][d];
        __syncthreads();
        if (r0 + i >= nrows) continue;
        float mx = -INFINITY, L = 0.f;
        for (int w = 0; w < 8; ++w) mx = fmaxf(mx, ml[w][i][0]);
        const float ref = mx == -INFINITY ? 0.f : mx;
        for (int w = 0; w < 8; ++w) L += ml[w][i][1] * exp2f(ml[w][i][0] - ref);
        const int r = r0 + i, t = r / p.heads, h = r - t * p.heads;
        const size_t row = (size_t)(rq.row0 + t) * p.heads + h;
        const bool none = lim[i] <= 0;
        for (int d = threadIdx.x; d < p.R; d += blockDim.x) {
            float a = 0.f;
            for (int w = 0; w < 8; ++w) a += ml[w][i][1] == 0.f ? 0.f : os[w][d] * exp2f(ml[w][i][0] - ref);
            a = none ? 0.f : a / L;
            if (p.w_uv)
                p.o_lat[row * p.R + d] = a;
            else
                reinterpret_cast<T *>(p.out)[(rq.row0 + t) * p.out_stride + (size_t)h * p.R + d] = E::down(a);
        }
        if (p.lse && threadIdx.x == 0) p.lse[row] = none ? -INFINITY : (mx + log2f(L)) * 0.693147180559945f;
    }
}

template <int DT>
__global__ void __launch_bounds__(128) latent_out_kernel(LatentParams p) {
    using E = Elem<DT>;
    using T = typename E::T;
    const size_t row = blockIdx.x;
    const int h = (int)(row % p.heads);
    const float *o = p.o_lat + row * p.R;
    for (int v = threadIdx.x; v < p.dv; v += blockDim.x) {
        const T *w = reinterpret_cast<const T *>(p.w_uv) + ((size_t)h * p.dv + v) * p.R;
        float s = 0.f;
        for (int r = 0; r < p.R; ++r) s = fmaf(o[r], E::up(w[r]), s);
        reinterpret_cast<T *>(p.out)[(row / p.heads) * p.out_stride + (size_t)h * p.dv + v] = E::down(s);
    }
}

template <int DT>
int launch(const LatentParams &p, cudaStream_t s) {
    int st = SPX_OK;
    if (p.w_uk) {
        latent_q_kernel<DT><<<p.N * p.heads, 128, 0, s>>>(p);
        if ((st = record_launch(cudaGetLastError()))) return st;
    }
    const long long gx = ((long long)p.max_q * p.heads + kRows - 1) / kRows;
    latent_rows_kernel<DT><<<dim3((unsigned)gx, p.B), 256, 0, s>>>(p);
    if ((st = record_launch(cudaGetLastError()))) return st;
    if (p.w_uv) {
        latent_out_kernel<DT><<<p.N * p.heads, 128, 0, s>>>(p);
        st = record_launch(cudaGetLastError());
    }
    return st;
}

constexpr size_t kHdr = 256;
size_t up256(size_t n) { return (n + 255) / 256 * 256; }
bool al16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

}  // namespace

// Checks of a cache's description that need no device.
int latent_cache_check(const spx_latent_cache *c) {
    if (!c || !c->cache || !c->block_table || !c->lens) return SPX_ERR_INVALID_ARG;
    if (c->num_pages < 1 || c->page_size < 1 || c->max_pages < 1 || c->B < 1) return SPX_ERR_INVALID_ARG;
    if (c->dtype != SPX_F16 && c->dtype != SPX_BF16) return SPX_ERR_UNSUPPORTED;
    if (c->R < 128 || c->R > 512 || c->R % 128 || c->P != 64 || c->page_size % 16) return SPX_ERR_UNSUPPORTED;
    if (!al16(c->cache) || c->token_stride < c->R + c->P || c->token_stride % 8 || c->page_stride % 8)
        return SPX_ERR_INVALID_ARG;
    if (c->num_pages > 1 && c->page_stride < (int64_t)(c->page_size - 1) * c->token_stride + c->R + c->P)
        return SPX_ERR_INVALID_ARG;
    return SPX_OK;
}

}  // namespace spx

using namespace spx;

extern "C" size_t spx_latent_workspace_size(int B, int N, int max_q, int max_len, int heads, int R, int P, int dn,
                                            int dv, int form) {
    if (B < 1 || N < 0 || max_q < 0 || max_len < 0 || heads < 1 || form < 0 || form > 2) return 0;
    if (R < 128 || R > 512 || R % 128 || P != 64 || heads > 1024 || B > 65535) return 0;
    if ((dn != 0) != (dv != 0) || (dn && dn != 64 && dn != 128) || (dv && dv != 64 && dv != 128)) return 0;
    if (form == SPX_LATENT_EXPANDED) return 0;
    size_t n = kHdr;
    if (dn) n += up256((size_t)N * heads * (R + P) * 2) + up256((size_t)N * heads * R * 4);
    return n;
}

extern "C" int spx_latent_attention(const spx_latent_args *a, spx_stream_t stream) {
    if (!a) return SPX_ERR_INVALID_ARG;
    int st = latent_cache_check(a->cache);
    if (st) return st;
    const spx_latent_cache &c = *a->cache;
    if (!a->q_start || a->N < 0 || a->heads < 1 || a->max_q < 0 || a->max_len < 0) return SPX_ERR_INVALID_ARG;
    if (a->N > 0 && (!a->q || !a->out)) return SPX_ERR_INVALID_ARG;
    if (!a->w_uk != !a->w_uv || (!a->w_uk && (a->dn || a->dv))) return SPX_ERR_INVALID_ARG;
    if (a->form < 0 || a->form > 2 || !al16(a->q) || !al16(a->out) || !al16(a->w_uk) || !al16(a->w_uv))
        return SPX_ERR_INVALID_ARG;
    const int64_t qw = (int64_t)a->heads * (a->w_uk ? a->dn + c.P : c.R + c.P);
    const int64_t ow = (int64_t)a->heads * (a->w_uk ? a->dv : c.R);
    if (a->q_stride < qw || a->out_stride < ow || a->q_stride % 8 || a->out_stride % 8) return SPX_ERR_INVALID_ARG;
    const size_t need = spx_latent_workspace_size(c.B, a->N, a->max_q, a->max_len, a->heads, c.R, c.P, a->dn, a->dv,
                                                  a->form);
    if (!need) return SPX_ERR_UNSUPPORTED;
    if (!a->ws || a->ws_bytes < need || !al16(a->ws)) return SPX_ERR_WORKSPACE;
    if (a->N == 0 || a->max_q == 0) return SPX_OK;
    LatentParams p{};
    p.cache = static_cast<const uint16_t *>(c.cache);
    p.page_stride = c.page_stride;
    p.token_stride = c.token_stride;
    p.num_pages = c.num_pages;
    p.page_size = c.page_size;
    p.R = c.R;
    p.P = c.P;
    p.table = c.block_table;
    p.max_pages = c.max_pages;
    p.B = c.B;
    p.lens = c.lens;
    p.N = a->N;
    p.heads = a->heads;
    p.max_q = a->max_q < a->N ? a->max_q : a->N;
    p.max_len = a->max_len;
    p.dn = a->dn;
    p.dv = a->dv;
    p.causal = a->causal != 0;
    p.q_stride = a->q_stride;
    p.out_stride = a->out_stride;
    p.q_start = a->q_start;
    p.q = static_cast<const uint16_t *>(a->q);
    p.w_uk = static_cast<const uint16_t *>(a->w_uk);
    p.w_uv = static_cast<const uint16_t *>(a->w_uv);
    p.out = static_cast<uint16_t *>(a->out);
    p.lse = a->lse;
    p.scale = a->scale;
    p.scale_log2 = a->scale * 1.4426950408889634f;
    uint8_t *ws = static_cast<uint8_t *>(a->ws);
    p.hdr = reinterpret_cast<WsHeader *>(ws);
    p.q_lat = reinterpret_cast<uint16_t *>(ws + kHdr);
    p.o_lat = reinterpret_cast<float *>(ws + kHdr + up256((size_t)a->N * a->heads * (c.R + c.P) * 2));
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return c.dtype == SPX_F16 ? launch<SPX_F16>(p, s) : launch<SPX_BF16>(p, s);
}
