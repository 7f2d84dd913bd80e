// spx_kv.cuh -- what the launches over a paged cache of keys and values share:
// the parameter block, a request's rows, what a row sees, and the dealing out
// of the call's key tiles to blocks.
#pragma once

#include "spx_latent.cuh"

namespace spx {

constexpr int kKvMaxTree = 64;    // rows of a tree: the bits of a mask
constexpr int kKvMaxGroup = 64;   // query heads to a key head
constexpr int kKvTile = 128;      // cached tokens of a tile
constexpr int kKvMaxBlocks = 152; // blocks of an attention launch: one per SM at most

struct KvParams {
    // cache
    const uint16_t *k, *v;
    int64_t page_stride, token_stride, head_stride;
    int num_pages, page_size, kv_heads, D;
    const int32_t *table;
    int max_pages, B;
    const int32_t *lens;
    // call
    int N, heads, group, max_q, max_len, causal;  // group: query heads to a key head; max_len: within the block table too
    FastDiv by_group, by_page;
    int64_t q_stride, out_stride;
    const int32_t *q_start;
    const uint64_t *tree;
    const uint16_t *q;
    uint16_t *out;
    float *lse;
    float scale_log2;  // scale * log2(e)
    // workspace
    WsHeader *hdr;
    uint64_t budget;
};

// A request's rows and cached length, cut to the call's bounds, so that no
// content of q_start or lens leads out of a buffer.
struct KvReq {
    int row0, T, len;
};
__device__ __forceinline__ KvReq kv_req(const int32_t *q_start, const int32_t *lens, int b, int N, int max_q, int max_len) {
    KvReq r;
    const int s = __ldg(q_start + b), e = __ldg(q_start + b + 1);
    r.row0 = min(max(s, 0), N);
    r.T = (int)min(min((int64_t)max(e, r.row0) - r.row0, (int64_t)max_q), (int64_t)(N - r.row0));
    r.len = min(max(__ldg(lens + b), 0), max_len);
    return r;
}
__device__ __forceinline__ KvReq kv_req(const KvParams &p, int b) {
    return kv_req(p.q_start, p.lens, b, p.N, p.max_q, p.max_len);
}

// What row t of a request sees: the positions below `lim`, and base + j for the
// bits j of `bits` (a tree's).
struct KvSeen {
    int lim, base;
    uint64_t bits;
    // the positions p0 + 32 w .. p0 + 32 w + 31, one a bit
    __device__ __forceinline__ uint32_t word(int p0) const {
        const int n = lim - p0, s = base - p0;
        uint32_t v = n >= 32 ? 0xFFFFFFFFu : n > 0 ? (1u << n) - 1 : 0u;
        if (s >= 0) {
            if (s < 32) v |= (uint32_t)(bits << s);
        } else if (s > -64) {
            v |= (uint32_t)(bits >> -s);
        }
        return v;
    }
};
__device__ __forceinline__ KvSeen kv_seen(const KvParams &p, const KvReq &r, int t) {
    KvSeen s;
    s.base = r.len - r.T;
    s.bits = 0;
    if (t >= r.T) {
        s.lim = 0;
    } else if (p.tree) {
        s.lim = max(s.base, 0);
        const uint64_t own = r.T < 64 ? (1ull << r.T) - 1 : ~0ull;
        s.bits = __ldg(reinterpret_cast<const unsigned long long *>(p.tree) + r.row0 + t) & own;
    } else {
        s.lim = p.causal ? max(s.base + t + 1, 0) : r.len;
    }
    return s;
}
// Positions that every row of the request from t on sees.
__device__ __forceinline__ int kv_all_see(const KvParams &p, const KvReq &r, int t) {
    const int base = r.len - r.T;
    return p.tree ? max(base, 0) : p.causal ? max(base + t + 1, 0) : r.len;
}
// Positions beyond which no row up to t sees anything.
__device__ __forceinline__ int kv_none_see(const KvParams &p, const KvReq &r, int t) {
    return p.tree || !p.causal ? r.len : max(r.len - r.T + t + 1, 0);
}

// -------------------------------------------------------------------- host --
// spx_kv.cu
int kv_cache_check(const spx_kv_cache *c);

}  // namespace spx
