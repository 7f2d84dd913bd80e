// spx_tree.cu -- trees of drafted tokens: what each row sees and where it goes,
// and the path that the target agrees with.
#include "spx_kv.cuh"

namespace spx {

namespace {

// -------------------------------------------------------------------- layout --
struct LayoutParams {
    int N, max_q, clear_rest;
    const int32_t *q_start, *lens, *parent;
    int32_t *req, *slot, *pos;
    uint64_t *mask;
};

constexpr int kLayoutThreads = kKvMaxTree;

// Block (request, 64 rows of it), a row a thread.  A row's mask is its own bit
// and its parent's mask: after round r a row holds its nearest 2^r ancestors
// and knows the next one, so six rounds do for 64 rows (a walk up the tree
// takes as many dependent reads as the tree is deep).  One launch of a few dozen
// bytes a row: bound by its own latency (1.5 us for 17 rows, 1.65 for 64 trees of
// 64, replayed from a graph).
__global__ void __launch_bounds__(kLayoutThreads) tree_layout_kernel(const __grid_constant__ LayoutParams p) {
    __shared__ uint64_t seen[2][kKvMaxTree];
    __shared__ int up[2][kKvMaxTree];
    griddep_wait();
    griddep_launch_dependents();
    const int b = blockIdx.x, j = threadIdx.x, i = (int)blockIdx.y * kLayoutThreads + j;
    const KvReq r = kv_req(p.q_start, p.lens, b, p.N, p.max_q, 0x7fffffff);
    if (p.clear_rest) {  // the rows between this request's and the next one's, or behind the last one's
        const int end = b + 1 < (int)gridDim.x ? min(__ldg(p.q_start + b + 1), p.N) : p.N;
        for (int64_t row = (int64_t)r.row0 + r.T + i; row < end; row += (int)gridDim.y * kLayoutThreads) {
            if (p.req) p.req[row] = -1;
            if (p.slot) p.slot[row] = -1;
            if (p.pos) p.pos[row] = -1;
            if (p.mask) p.mask[row] = 0;
        }
    }
    if ((int)blockIdx.y * kLayoutThreads >= r.T) return;
    int above = i;
    uint64_t m = i < 64 ? (2ull << i) - 1 : 0;
    if (p.parent) {  // (one block a request)
        const int q = i < r.T ? __ldg(p.parent + r.row0 + i) : -1;
        m = 1ull << j;
        int a = q >= 0 && q < i ? q : -1;
        seen[0][j] = m;
        up[0][j] = a;
        __syncthreads();
#pragma unroll
        for (int x = 0; x < 6; ++x) {
            if (a >= 0) {
                m |= seen[x & 1][a];
                a = up[x & 1][a];
            }
            seen[x & 1 ^ 1][j] = m;
            up[x & 1 ^ 1][j] = a;
            __syncthreads();
        }
        above = __popcll(m) - 1;
    }
    if (i >= r.T) return;
    const int row = r.row0 + i, base = r.len - r.T;
    if (p.req) p.req[row] = b;
    if (p.slot) p.slot[row] = base + i;
    if (p.pos) p.pos[row] = base + above;
    if (p.mask) p.mask[row] = m;
}

// -------------------------------------------------------------------- accept --
constexpr int kMaxLayers = 128;
constexpr int kAcceptThreads = 128;
static_assert(kAcceptThreads >= 32 + kKvMaxTree, "a warp for the path, a thread for each row's place");
template <int M>  // room for the buffers of M / 2 layers
struct AcceptParams {
    int64_t page_stride, token_stride, head_stride;
    int num_pages, page_size, kv_heads, units, max_pages;  // units of 8 values of a head
    const int32_t *table, *lens;
    int N, max_q, columns;  // columns: units of all layers
    FastDiv by_page, by_units, by_heads;
    const int32_t *q_start, *parent, *token, *target;
    int32_t *n_kept, *path, *next, *lens_out;
    void *kv[M];  // of layer l: keys 2l, values 2l + 1
};

// Block (request, 128 columns): its first warp walks down the tree, two rows a
// lane in registers, a vote a step, while others look up where the rows are; then
// a thread moves one unit of 16 bytes of the path's rows, which ascend, so that a
// row is read before it is written over.  Every block of a request takes the same
// walk rather than wait for one.  24 layers of one request's 8 rows 2.9 us, its
// latency (walk, rows; 3.1 with the table read behind the walk); 32 layers of 16
// requests, 50 MB moved, 8.7 us from L2, 12.5 from DRAM (8 rows at a time for 16,
// 1.1 more; blocks of 256 threads 0.5; the table behind the walk 0.4).
template <int M>
__global__ void __launch_bounds__(kAcceptThreads) tree_accept_kernel(const __grid_constant__ AcceptParams<M> p) {
    __shared__ int way[kKvMaxTree], count, last_target;
    __shared__ int64_t place[kKvMaxTree];  // of the request's rows in the cache, -1: nowhere
    __shared__ int64_t from[kKvMaxTree], to[kKvMaxTree];
    griddep_wait();
    griddep_launch_dependents();
    const int b = blockIdx.x, lane = threadIdx.x & 31;
    const KvReq r = kv_req(p.q_start, p.lens, b, p.N, p.max_q, 0x7fffffff);
    const int base = r.len - r.T;
    if (threadIdx.x < 32) {
        int par[2], tok[2], tgt[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int i = lane + 32 * x;
            const bool in = i < r.T;
            par[x] = in && i > 0 ? __ldg(p.parent + r.row0 + i) : -1;
            if (par[x] >= i) par[x] = -1;
            tok[x] = in ? __ldg(p.token + r.row0 + i) : 0;
            tgt[x] = in ? __ldg(p.target + r.row0 + i) : -1;
        }
        int cur = 0, n = r.T > 0 ? 1 : 0, want = __shfl_sync(0xffffffffu, tgt[0], 0);
        if (lane == 0) way[0] = 0;
        while (n > 0) {  // (a row lies behind its parent: 64 rounds at most)
            const uint32_t lo = __ballot_sync(0xffffffffu, par[0] == cur && tok[0] == want);
            const uint32_t hi = __ballot_sync(0xffffffffu, par[1] == cur && tok[1] == want);
            if (!(lo | hi)) break;
            cur = lo ? __ffs(lo) - 1 : 31 + __ffs(hi);
            const int a = __shfl_sync(0xffffffffu, tgt[0], cur & 31), c = __shfl_sync(0xffffffffu, tgt[1], cur & 31);
            want = cur < 32 ? a : c;
            if (lane == 0) way[n] = cur;
            ++n;
        }
        if (lane == 0) {
            count = n;
            last_target = want;
        }
    } else if (threadIdx.x >= kAcceptThreads - kKvMaxTree) {  // meanwhile
        const int d = threadIdx.x - (kAcceptThreads - kKvMaxTree), at = base + d, pi = p.by_page(max(at, 0));
        int64_t to = -1;
        if (d < r.T && at >= 0 && pi < p.max_pages) {
            const int pg = __ldg(p.table + (size_t)b * p.max_pages + pi);
            if (pg >= 0 && pg < p.num_pages)
                to = (int64_t)pg * p.page_stride + (int64_t)(at - pi * p.page_size) * p.token_stride;
        }
        place[d] = to;
    }
    __syncthreads();
    const int n = count;
    if (blockIdx.y == 0) {
        if (threadIdx.x < r.T) p.path[r.row0 + threadIdx.x] = (int)threadIdx.x < n ? way[threadIdx.x] : -1;
        if (threadIdx.x == 0) {
            p.n_kept[b] = n;
            p.next[b] = n ? last_target : -1;
            p.lens_out[b] = base + n;
        }
    }
    // A row without a page reads as zeros, and as zeros it is moved: what stood at its destination is another row's.
    bool blank = false;
    if (threadIdx.x < kKvMaxTree) {
        const int d = threadIdx.x, i = d < n ? way[d] : d;
        from[d] = i == d || place[d] < 0 ? -1 : place[i];
        to[d] = place[d];
        blank = i != d && place[d] >= 0 && place[i] < 0;
    }
    const bool blanks = __syncthreads_or(blank);
    const int c = (int)blockIdx.y * kAcceptThreads + threadIdx.x;
    if (c >= p.columns) return;
    const int head = p.by_units(c), unit = c - head * p.units, x = p.by_heads(head), h = head - x * p.kv_heads;
    uint16_t *buf = static_cast<uint16_t *>(p.kv[x]) + (int64_t)h * p.head_stride + 8 * unit;
    constexpr int kAhead = 16;
    for (int d0 = 1; d0 < n; d0 += kAhead) {
        uint4 v[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            if (d0 + k < n && from[d0 + k] >= 0) v[k] = *reinterpret_cast<const uint4 *>(buf + from[d0 + k]);
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            if (d0 + k < n && from[d0 + k] >= 0) *reinterpret_cast<uint4 *>(buf + to[d0 + k]) = v[k];
    }
    if (blanks)  // (behind the moves: nothing is read any more)
        for (int d = 1; d < n; ++d)
            if (way[d] != d && from[d] < 0 && to[d] >= 0) *reinterpret_cast<uint4 *>(buf + to[d]) = make_uint4(0, 0, 0, 0);
}

// Buffers that one block reads while another writes must lie apart.
struct Span {
    const void *at;
    size_t bytes;
};
bool overlap(const Span &a, const Span &b) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.at), y = reinterpret_cast<uintptr_t>(b.at);
    return a.at && b.at && x < y + b.bytes && y < x + a.bytes;
}
template <int I, int O>
bool any_overlap(const Span (&in)[I], const Span (&out)[O]) {
    for (int o = 0; o < O; ++o) {
        for (int i = 0; i < I; ++i)
            if (overlap(in[i], out[o])) return true;
        for (int i = 0; i < o; ++i)
            if (overlap(out[i], out[o])) return true;
    }
    return false;
}

// Whether no pointer is there twice (none is null): a table of twice as many
// places, probed from where a pointer's bits lead.  (Every pair of 256, compared,
// would take as long as the launch.)
bool distinct(void *const *at, int n) {
    constexpr int kBits = 9;
    static_assert(1 << kBits >= 4 * kMaxLayers, "half of the places stay empty");
    void *seen[1 << kBits] = {};
    for (int i = 0; i < n; ++i) {
        uint32_t h = (uint32_t)(reinterpret_cast<uintptr_t>(at[i]) * 0x9E3779B97F4A7C15ull >> (64 - kBits));
        for (; seen[h]; h = (h + 1) & ((1 << kBits) - 1))
            if (seen[h] == at[i]) return false;
        seen[h] = at[i];
    }
    return true;
}

template <int M>
int launch_accept(const spx_tree_accept_args &a, const spx_kv_cache &c, cudaStream_t s) {
    AcceptParams<M> p{};
    for (int i = 0; i < 2 * a.n_layers; ++i) p.kv[i] = i & 1 ? a.layer_v[i >> 1] : a.layer_k[i >> 1];
    if (!distinct(p.kv, 2 * a.n_layers)) return SPX_ERR_INVALID_ARG;  // moved twice, it would be read after it was written
    p.page_stride = c.page_stride;
    p.token_stride = c.token_stride;
    p.head_stride = c.head_stride;
    p.num_pages = c.num_pages;
    p.page_size = c.page_size;
    p.kv_heads = c.kv_heads;
    p.units = c.D / 8;
    p.max_pages = c.max_pages;
    p.table = c.block_table;
    p.lens = c.lens;
    p.N = a.N;
    p.max_q = a.max_q;
    p.by_page.set(c.page_size);
    p.by_units.set(p.units);
    p.by_heads.set(c.kv_heads);
    p.q_start = a.q_start;
    p.parent = a.parent;
    p.token = a.token;
    p.target = a.target;
    p.n_kept = a.n_kept;
    p.path = a.path;
    p.next = a.next;
    p.lens_out = a.lens_out;
    const long long columns = 2ll * a.n_layers * c.kv_heads * p.units;
    const long long groups = columns ? (columns + kAcceptThreads - 1) / kAcceptThreads : 1;
    if (groups > 65535) return SPX_ERR_UNSUPPORTED;
    p.columns = (int)columns;
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = latent_config(dim3((unsigned)c.B, (unsigned)groups), kAcceptThreads, 0,
                                           s, attr, 1);
    return record_launch(cudaLaunchKernelEx(&cfg, tree_accept_kernel<M>, p));
}

}  // namespace

}  // namespace spx

using namespace spx;

extern "C" int spx_tree_layout(const spx_tree_layout_args *a, spx_stream_t stream) {
    if (!a || !a->q_start || !a->lens || a->B < 1 || a->N < 0 || a->max_q < 0) return SPX_ERR_INVALID_ARG;
    const size_t nb = (size_t)a->B * 4, nn = (size_t)a->N * 4;
    const Span in[] = {{a->q_start, nb + 4}, {a->lens, nb}, {a->parent, nn}};
    const Span out[] = {{a->req, nn}, {a->slot, nn}, {a->pos, nn}, {a->mask, 2 * nn}};
    if (any_overlap(in, out)) return SPX_ERR_INVALID_ARG;
    if (a->max_q > kKvMaxTree && (a->parent || a->mask)) return SPX_ERR_UNSUPPORTED;
    if (a->N == 0 || (a->max_q == 0 && !a->clear_rest)) return SPX_OK;
    const int rows = a->max_q < a->N ? a->max_q : a->N, groups = rows ? (rows + kLayoutThreads - 1) / kLayoutThreads : 1;
    if (groups > 65535) return SPX_ERR_UNSUPPORTED;
    LayoutParams p{a->N, a->max_q, a->clear_rest, a->q_start, a->lens, a->parent, a->req, a->slot, a->pos, a->mask};
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = latent_config(dim3((unsigned)a->B, (unsigned)groups), kLayoutThreads, 0,
                                           reinterpret_cast<cudaStream_t>(stream), attr, 1);
    return record_launch(cudaLaunchKernelEx(&cfg, tree_layout_kernel, p));
}

extern "C" int spx_tree_accept(const spx_tree_accept_args *a, spx_stream_t stream) {
    if (!a || !a->cache) return SPX_ERR_INVALID_ARG;
    spx_kv_cache c = *a->cache;
    if (a->n_layers < 0 || (a->n_layers > 0 && (!a->layer_k || !a->layer_v))) return SPX_ERR_INVALID_ARG;
    if (a->n_layers > kMaxLayers) return SPX_ERR_UNSUPPORTED;
    c.k = c.v = reinterpret_cast<void *>(uintptr_t(16));  // stands for a buffer: the layers' own are checked below
    const int st = kv_cache_check(&c);
    if (st) return st;
    for (int i = 0; i < 2 * a->n_layers; ++i) {
        const void *const buf = i & 1 ? a->layer_v[i >> 1] : a->layer_k[i >> 1];
        if (!buf || (reinterpret_cast<uintptr_t>(buf) & 15)) return SPX_ERR_INVALID_ARG;
    }
    if (!a->q_start || !a->n_kept || !a->next || !a->lens_out || a->N < 0 || a->max_q < 0) return SPX_ERR_INVALID_ARG;
    if (a->N > 0 && (!a->parent || !a->token || !a->target || !a->path)) return SPX_ERR_INVALID_ARG;
    const size_t nb = (size_t)c.B * 4, nn = (size_t)a->N * 4;
    const Span in[] = {{c.lens, nb}, {c.block_table, nb * c.max_pages}, {a->q_start, nb + 4}, {a->parent, nn}, {a->token, nn},
                       {a->target, nn}};
    const Span out[] = {{a->n_kept, nb}, {a->path, nn}, {a->next, nb}, {a->lens_out, nb}};
    if (any_overlap(in, out)) return SPX_ERR_INVALID_ARG;
    if (a->max_q > kKvMaxTree) return SPX_ERR_UNSUPPORTED;
    // (kernel parameters are copied with every launch: room for as many layers as usual, or for the most)
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return a->n_layers <= 32 ? launch_accept<64>(*a, c, s) : launch_accept<2 * kMaxLayers>(*a, c, s);
}
