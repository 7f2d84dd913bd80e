// spx_kv_attention.cu -- attention over the paged cache of keys and values.
#include <math.h>

#include "spx_kv.cuh"

namespace spx {

namespace {

// A warp per (row, head), a token at a time.
template <int DT, int D>
__global__ void __launch_bounds__(256) kv_plain_kernel(const __grid_constant__ KvParams p) {
    constexpr int kPer = D / 32;
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31, at = (int)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int n = at / p.heads, h = at - n * p.heads;
    if (n >= p.N) return;
    for (int b = 0; b < p.B; ++b) {
        const KvReq r = kv_req(p, b);
        if (n < r.row0 || n >= r.row0 + r.T) continue;
        const KvSeen seen = kv_seen(p, r, n - r.row0);
        const int64_t head = (int64_t)(h / p.group) * p.head_stride;
        using T = typename Elem<DT>::T;
        float q[kPer], o[kPer] = {}, m = -INFINITY, l = 0.f;
        for (int j = 0; j < kPer; ++j)
            q[j] = Elem<DT>::up(reinterpret_cast<const T *>(p.q)[(int64_t)n * p.q_stride + (int64_t)h * D + kPer * lane + j]);
        for (int x = 0; x < r.len; ++x) {
            if (!(seen.word(x) & 1)) continue;
            const int pi = p.by_page(x), pg = __ldg(p.table + (size_t)b * p.max_pages + pi);
            const bool ok = pg >= 0 && pg < p.num_pages;
            const int64_t row = (int64_t)pg * p.page_stride + (int64_t)(x - pi * p.page_size) * p.token_stride + head;
            float s = 0.f, v[kPer];
            for (int j = 0; j < kPer; ++j) {
                s += ok ? q[j] * Elem<DT>::up(reinterpret_cast<const T *>(p.k)[row + kPer * lane + j]) : 0.f;
                v[j] = ok ? Elem<DT>::up(reinterpret_cast<const T *>(p.v)[row + kPer * lane + j]) : 0.f;
            }
            for (int i = 16; i; i >>= 1) s += __shfl_xor_sync(0xffffffffu, s, i);
            s *= p.scale_log2;
            const float mn = fmaxf(m, s), f = mn == m ? 1.f : exp2f(m - mn), w = mn == -INFINITY ? 0.f : exp2f(s - mn);
            m = mn;
            l = l * f + w;
            for (int j = 0; j < kPer; ++j) o[j] = o[j] * f + w * v[j];
        }
        for (int j = 0; j < kPer; ++j)
            reinterpret_cast<T *>(p.out)[(int64_t)n * p.out_stride + (int64_t)h * D + kPer * lane + j] =
                Elem<DT>::down(l == 0.f ? 0.f : o[j] / l);
        if (p.lse && lane == 0) p.lse[(int64_t)n * p.heads + h] = (m + log2f(l)) * 0.6931471805599453f;
    }
}

bool al16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

}  // namespace

// Checks of a cache's description that need no device.
int kv_cache_check(const spx_kv_cache *c) {
    if (!c || !c->k || !c->v || !c->block_table || !c->lens) return SPX_ERR_INVALID_ARG;
    if (c->num_pages < 1 || c->page_size < 1 || c->max_pages < 1 || c->B < 1 || c->kv_heads < 1) return SPX_ERR_INVALID_ARG;
    if (c->dtype != SPX_F16 && c->dtype != SPX_BF16) return SPX_ERR_UNSUPPORTED;
    if ((c->D != 64 && c->D != 128) || c->page_size % 16 || c->kv_heads > 1024 || c->B > 65535) return SPX_ERR_UNSUPPORTED;
    if (!al16(c->k) || !al16(c->v)) return SPX_ERR_INVALID_ARG;
    // from the dimension whose steps are shortest on, each step passes over all of those before
    int64_t n[3] = {c->page_size, c->kv_heads, c->num_pages}, st[3] = {c->token_stride, c->head_stride, c->page_stride};
    for (int i = 0; i < 3; ++i)
        if (st[i] % 8 || (n[i] > 1 && st[i] < c->D)) return SPX_ERR_INVALID_ARG;
    int64_t span = c->D;
    bool done[3] = {n[0] == 1, n[1] == 1, n[2] == 1};
    while (true) {
        int next = -1;
        for (int i = 0; i < 3; ++i)
            if (!done[i] && (next < 0 || st[i] < st[next])) next = i;
        if (next < 0) break;
        if (st[next] < span) return SPX_ERR_INVALID_ARG;
        if (st[next] >= (int64_t)1 << 38) return SPX_ERR_UNSUPPORTED;
        span += (n[next] - 1) * st[next];
        done[next] = true;
    }
    return SPX_OK;
}

}  // namespace spx

using namespace spx;

extern "C" size_t spx_kv_workspace_size(int B, int N, int max_q, int max_len, int heads, int kv_heads, int D) {
    if (B < 1 || N < 0 || max_q < 0 || max_len < 0 || heads < 1 || kv_heads < 1 || heads % kv_heads) return 0;
    if ((D != 64 && D != 128) || heads / kv_heads > kKvMaxGroup || kv_heads > 1024 || B > 65535) return 0;
    // rows of (token, head) and cached tokens are counted in 31 bits, and so are the tiles of the call
    if ((long long)N * heads > 1 << 30 || (long long)max_q * heads > 1 << 30) return 0;
    const long long rows = max_q < N ? max_q : N;
    if ((double)B * kv_heads * (rows * (heads / kv_heads) / 64 + 1) * (max_len / kKvTile + 1) > 2e9) return 0;
    return SPX_KV_WORKSPACE_ZERO;
}

extern "C" int spx_kv_attention(const spx_kv_attention_args *a, spx_stream_t stream) {
    if (!a) return SPX_ERR_INVALID_ARG;
    const int st = kv_cache_check(a->cache);
    if (st) return st;
    const spx_kv_cache &c = *a->cache;
    if (!a->q_start || a->N < 0 || a->heads < 1 || a->max_q < 0 || a->max_len < 0 || a->heads % c.kv_heads)
        return SPX_ERR_INVALID_ARG;
    if (!(a->scale > 0.f) || !(a->scale < INFINITY)) return SPX_ERR_INVALID_ARG;
    if (a->N > 0 && (!a->q || !a->out)) return SPX_ERR_INVALID_ARG;
    const int64_t w = (int64_t)a->heads * c.D;
    if (!al16(a->q) || !al16(a->out) || a->q_stride < w || a->out_stride < w || a->q_stride % 8 || a->out_stride % 8)
        return SPX_ERR_INVALID_ARG;
    if (a->tree && a->max_q > kKvMaxTree) return SPX_ERR_UNSUPPORTED;
    const size_t need = spx_kv_workspace_size(c.B, a->N, a->max_q, a->max_len, a->heads, c.kv_heads, c.D);
    if (!need) return SPX_ERR_UNSUPPORTED;
    if (!a->ws || a->ws_bytes < need || !al16(a->ws)) return SPX_ERR_WORKSPACE;
    if (a->N == 0 || a->max_q == 0) return SPX_OK;
    KvParams p{};
    p.k = static_cast<const uint16_t *>(c.k);
    p.v = static_cast<const uint16_t *>(c.v);
    p.page_stride = c.page_stride;
    p.token_stride = c.token_stride;
    p.head_stride = c.head_stride;
    p.num_pages = c.num_pages;
    p.page_size = c.page_size;
    p.kv_heads = c.kv_heads;
    p.D = c.D;
    p.table = c.block_table;
    p.max_pages = c.max_pages;
    p.B = c.B;
    p.lens = c.lens;
    p.N = a->N;
    p.heads = a->heads;
    p.group = a->heads / c.kv_heads;
    p.max_q = a->max_q;
    const long long held = (long long)c.max_pages * c.page_size;
    p.max_len = a->max_len < held ? a->max_len : (int)held;
    p.causal = a->causal != 0;
    p.by_group.set(p.group);
    p.by_page.set(c.page_size);
    p.q_stride = a->q_stride;
    p.out_stride = a->out_stride;
    p.q_start = a->q_start;
    p.tree = a->tree;
    p.q = static_cast<const uint16_t *>(a->q);
    p.out = static_cast<uint16_t *>(a->out);
    p.lse = a->lse;
    p.scale_log2 = a->scale * 1.4426950408889634f;
    p.hdr = static_cast<WsHeader *>(a->ws);
    p.budget = a->wait_budget_ns ? a->wait_budget_ns : 2000000000ull;
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = latent_config(dim3((unsigned)(((long long)a->N * a->heads + 7) / 8)), 256, 0,
                                           reinterpret_cast<cudaStream_t>(stream), attr, 1);
    const bool f16 = c.dtype == SPX_F16;
    return record_launch(c.D == 128 ? (f16 ? cudaLaunchKernelEx(&cfg, kv_plain_kernel<SPX_F16, 128>, p)
                                           : cudaLaunchKernelEx(&cfg, kv_plain_kernel<SPX_BF16, 128>, p))
                                    : (f16 ? cudaLaunchKernelEx(&cfg, kv_plain_kernel<SPX_F16, 64>, p)
                                           : cudaLaunchKernelEx(&cfg, kv_plain_kernel<SPX_BF16, 64>, p)));
}
