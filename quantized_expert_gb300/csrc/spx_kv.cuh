// spx_kv.cuh -- what the launches over a paged cache of keys and values share:
// the parameter block, a request's rows, what a row sees, and the dealing out
// of the call's key tiles to blocks.
#pragma once

#include "spx_latent.cuh"

namespace spx {

constexpr int kKvMaxTree = 64;    // rows of a tree: the bits of a mask
constexpr int kKvMaxGroup = 64;   // query heads to a key head
constexpr int kKvTile = 128;      // cached tokens of a tile
constexpr int kKvMostCost = 4;    // of a unit beside its tiles, in tiles, in any launch
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
    FastDiv by_group, by_page, by_blocks;  // blocks of the attention launch
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
    uint32_t *done;    // [blocks] parts of the unit that begins in a block and ends in a later one; zero between calls
    float2 *ml;        // [2 blocks][rows] reference and weight of a partial sum's row
    float *part;       // [2 blocks][rows][D] partial sums
    int4 *seams;       // of a unit that crosses from block to block: its first row, its rows, key head, and its first block
                       // << 16 | its last (the same block: it does not)
    int seam_groups;   // above 0: one for each unit, this many to a request and key head; 0: one for each block
    int span;          // rows (tokens) of a unit
    int unit_cost;     // of a unit beside its tiles, in tiles
    int tile_tokens;   // rows (tokens) of a product of 128 (token, head) rows
    int q_tokens;      // of them, those that the copy of a unit's queries brings
    int box_tokens;    // cached tokens of one copy: the largest power of two that divides a page, 128 at most
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

// One warp, before the launches in front of this one have ended: what is read
// one after the other behind them comes as near as L2, where they may still
// write it (a tree's call 12.3 to 12.2 us from a graph, prompts of 4096 122 to 121).
__device__ __forceinline__ void kv_prefetch(const KvParams &p, int lane) {
    const auto fetch = [](const int32_t *at) { asm volatile("prefetch.global.L2 [%0];" ::"l"(at) : "memory"); };
    if (32 * lane <= p.B) fetch(p.q_start + 32 * lane);
    if (32 * lane < p.B) fetch(p.lens + 32 * lane);
    if (p.B == 1 && 32 * lane < p.max_pages) fetch(p.table + 32 * lane);
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

// ------------------------------------------------------------------ shares --
// A unit of work is a key head's query heads on up to `span` consecutive rows of
// a request; its tiles are the key tiles that any of these rows sees, one at
// least, so that a row which sees nothing is written too.  The tiles of all
// units, in the order request, key head, rows, are dealt out in equal
// contiguous shares, one a block: a long request and a ragged batch both fill
// the machine, and a block meets at most two units that are not its own alone.
// What a unit costs beside its tiles counts as `unit_cost` tiles in front of
// them that nobody works on, or a block with many short units would be late.
// A share that begins or ends inside a unit leaves a partial sum in the
// workspace: block c has place 2c for the unit in which its share begins,
// 2c + 1 for one that begins in its share and ends in a later block's.
__device__ __forceinline__ int kv_groups(int T, int span) { return (T + span - 1) / span; }
__device__ __forceinline__ int kv_tiles(const KvParams &p, const KvReq &r, int g, int span) {
    return max((kv_none_see(p, r, min((g + 1) * span, r.T) - 1) + kKvTile - 1) / kKvTile, 1);
}
// Tiles of all of a key head's units, with what a unit costs beside them.
__device__ __forceinline__ int kv_head_tiles(const KvParams &p, const KvReq &r, int span) {
    const int groups = kv_groups(r.T, span);
    if (groups <= 1 || p.tree || !p.causal) return groups ? groups * (kv_tiles(p, r, 0, span) + p.unit_cost) : 0;
    // (kv_tiles of all but the last unit in three instructions each, as a long prompt has many)
    int n = kv_tiles(p, r, groups - 1, span) + groups * p.unit_cost, a = r.len - r.T + span + kKvTile - 1;
    for (int g = 1; g < groups; ++g, a += span) n += max(a / kKvTile, 1);
    return n;
}

// Where a block's share begins, the same for all its threads.
struct KvShare {
    int b, h, g, off;  // unit, and the first tile of it
    int flat, left;    // index of that tile among the call's; tiles of the share from it on
    int share;         // tiles of a whole share
    KvReq rq;
};

// Tiles of a unit with what it costs beside them, 0 past the request's last one.
__device__ __forceinline__ int kv_unit_tiles(const KvParams &p, const KvReq &r, int g, int span, int groups) {
    return g < groups ? kv_tiles(p, r, g, span) + p.unit_cost : 0;
}
__device__ __forceinline__ int warp_upto(int n, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, n, o);
        if (lane >= o) n += v;
    }
    return n;
}

// One warp: every lane gets the block's share.  Requests a lane each (the last
// 32 stay in registers, which is all of a small batch); a single request's
// units a lane each, as a long prompt has many.  This is what a short call
// waits for, so divisors that the host knows are multiplied by.
__device__ __forceinline__ KvShare kv_find_share(const KvParams &p, int span, int lane) {
    KvShare w{};
    int total = 0, n = 0;  // tiles of a key head
    KvReq r{};
    if (p.B == 1) {
        r = kv_req(p, 0);
        if (r.T <= span) {
            n = r.T > 0 ? kv_tiles(p, r, 0, span) + p.unit_cost : 0;
        } else {
            const int groups = kv_groups(r.T, span);
            for (int g = lane; g < groups; g += 32) n += kv_unit_tiles(p, r, g, span, groups);
            n = __reduce_add_sync(0xffffffffu, n);
        }
        total = n;
    } else {
        for (int b0 = 0; b0 < p.B; b0 += 32) {
            n = 0;
            if (b0 + lane < p.B) {
                r = kv_req(p, b0 + lane);
                n = kv_head_tiles(p, r, span);
            }
            total += __reduce_add_sync(0xffffffffu, n);
        }
    }
    total *= p.kv_heads;
    w.share = max(p.by_blocks(total + p.by_blocks.d - 1), 1);
    w.flat = (int)min((int64_t)w.share * blockIdx.x, (int64_t)total);
    w.left = min(w.share, total - w.flat);
    if (w.left <= 0) return w;
    w.off = w.flat;
    if (p.B > 1) {
        int before = 0;
        for (int b0 = 0;; b0 += 32) {
            if (b0 >= p.B) {  // (not reached)
                w.left = 0;
                return w;
            }
            if (p.B > 32) {
                n = 0;
                if (b0 + lane < p.B) {
                    r = kv_req(p, b0 + lane);
                    n = kv_head_tiles(p, r, span);
                }
            }
            const int own = n * p.kv_heads, upto = warp_upto(own, lane), off = w.flat - (before + upto - own);
            const uint32_t mine = __ballot_sync(0xffffffffu, off >= 0 && off < own);
            if (mine) {
                const int l = __ffs(mine) - 1;
                w.b = b0 + l;
                w.off = __shfl_sync(0xffffffffu, off, l);
                r.row0 = __shfl_sync(0xffffffffu, r.row0, l);
                r.T = __shfl_sync(0xffffffffu, r.T, l);
                r.len = __shfl_sync(0xffffffffu, r.len, l);
                n = __shfl_sync(0xffffffffu, n, l);
                break;
            }
            before += __shfl_sync(0xffffffffu, upto, 31);
        }
    }
    w.rq = r;
    w.h = (int)((uint32_t)w.off / (uint32_t)n);
    w.off -= w.h * n;
    if (r.T > span) {
        const int groups = kv_groups(r.T, span);
        for (int g0 = 0; g0 < groups; g0 += 32) {
            const int t = kv_unit_tiles(p, r, g0 + lane, span, groups), upto = warp_upto(t, lane);
            const uint32_t mine = __ballot_sync(0xffffffffu, w.off >= upto - t && w.off < upto);
            if (mine) {
                const int l = __ffs(mine) - 1;
                w.g = g0 + l;
                w.off -= __shfl_sync(0xffffffffu, upto - t, l);
                break;
            }
            w.off -= __shfl_sync(0xffffffffu, upto, 31);
        }
    }
    w.off -= p.unit_cost;
    if (w.off < 0) {  // the share begins with what a unit costs
        w.flat -= w.off;
        w.left += w.off;
        w.off = 0;
    }
    return w;
}

// A walk over a share, unit by unit; the same in every role of a block.
struct KvWalk {
    int b, h, g, nt;    // unit, its tiles
    int tile, end;      // tiles of the unit in this share, one at least
    int flat, left;     // index of `tile` among the call's tiles; tiles of the share from `tile` on
    KvReq rq;
    __device__ __forceinline__ void begin(const KvParams &p, const KvShare &w, int span) {
        b = w.b;
        h = w.h;
        g = w.g;
        flat = w.flat;
        left = w.left;
        rq = w.rq;
        if (left <= 0) return;
        nt = kv_tiles(p, rq, g, span);
        tile = w.off;
        end = min(nt, tile + left);
    }
    __device__ __forceinline__ bool whole() const { return tile == 0 && end == nt; }
    __device__ __forceinline__ void next(const KvParams &p, int span) {
        left -= end - tile + p.unit_cost;
        flat += end - tile + p.unit_cost;
        if (left <= 0) return;
        if (++g == kv_groups(rq.T, span)) {
            g = 0;
            if (++h == p.kv_heads) {
                h = 0;
                do {
                    if (++b >= p.B) {  // (does not happen while tiles are left)
                        left = 0;
                        return;
                    }
                    rq = kv_req(p, b);
                } while (rq.T == 0);
            }
        }
        nt = kv_tiles(p, rq, g, span);
        tile = 0;
        end = min(nt, left);
    }
};

// ------------------------------------------------------------------- results --
constexpr float kKvLn2 = 0.6931471805599453f;
// The reference of a row moves only when a score is 2^kKvSlack above it, and
// weights are scaled by 2^kKvShift: they stay below fp16's largest value (2^16)
// and most of what is worth adding above its subnormals (2^-14).
constexpr float kKvSlack = 8.f, kKvShift = 5.f;
// References are held as scores are, without the scale.  The exponent of a weight
// is score * scale_log2 + kv_ref, rounded once, which is exact enough while a step
// of the reference's product with the scale is below 1; from there on (kv_far) the
// difference of score and reference is taken first, or a row's best weight might
// be 2^(half a step), infinite or nothing.
constexpr float kKvFar = 8388608.f;  // 2^23
__device__ __forceinline__ float kv_ref(float m, float scale_log2) { return m == -INFINITY ? 0.f : kKvShift - m * scale_log2; }
__device__ __forceinline__ bool kv_far(float m, float scale_log2) {
    return m != -INFINITY && fabsf(m * scale_log2) >= kKvFar;
}

// Log of a row's sum of exponentials from its reference and weight.
__device__ __forceinline__ float kv_lse(float m, float l) {
    return l == 0.f ? -INFINITY : (m + log2f(l) - kKvShift) * kKvLn2;
}
// The factor of a part with reference m under a common reference (0 without
// any, unless no part has one).
__device__ __forceinline__ float kv_factor(float m, float common) {
    return m == -INFINITY ? (common == -INFINITY ? 1.f : 0.f) : ex2(m - common);
}
// A result before its rounding.  The rounded weights may sum to more than their
// sum, by 2^-11 of it, and carry a mean of values at fp16's largest, 65504, past
// what fp16 holds; an infinity or a NaN stays.  (bf16 ends where fp32 does: sums of
// such values overflow before.)
template <int DT>
__device__ __forceinline__ float kv_held(float v) {
    return DT == SPX_F16 && fabsf(v) < 65536.f ? fminf(fmaxf(v, -65504.f), 65504.f) : v;
}
template <int DT>
__device__ __forceinline__ uint32_t kv_down2(float a, float b) {
    return Elem<DT>::down2(kv_held<DT>(a), kv_held<DT>(b));
}
// One warp: a row's sum over the parts `first`, first + step and so on of the
// blocks c0 .. c1, in their order, under the reference of them all.  r: row of a
// place, of which there are `rows`.  Sums are read kAhead parts at a time (a
// divisor of 32), the first ones with the references and weights (a part a lane,
// 32 at a time) and not behind them: what a row costs is the time of one read
// after the other.
template <int D>
struct KvSum {
    static constexpr int kPer = D / 32;
    float m, l, v[kPer];  // v: the lane's values
};
template <int D, int kAhead = 8>
__device__ __forceinline__ KvSum<D> kv_sum_parts(const KvParams &p, int c0, int c1, int first, int step, int rows, int r, int lane) {
    constexpr int kPer = D / 32;
    KvSum<D> s;
    const auto place = [&](int k) { return (size_t)(2 * k + (k == c0)) * rows + r; };
    const int n = (c1 - c0 - first) / step + 1;  // (first <= c1 - c0)
    uint32_t x[kAhead][kPer];
    const auto fetch = [&](int i0) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            if (i0 + i >= n) continue;
            const float *src = p.part + place(c0 + first + step * (i0 + i)) * D + kPer * lane;
            if (kPer == 4) {
                const uint4 v = __ldcg(reinterpret_cast<const uint4 *>(src));
                x[i][0] = v.x;
                x[i][1] = v.y;
                x[i][kPer - 2] = v.z;
                x[i][kPer - 1] = v.w;
            } else {
                const uint2 v = __ldcg(reinterpret_cast<const uint2 *>(src));
                x[i][0] = v.x;
                x[i][1] = v.y;
            }
        }
    };
    fetch(0);
    s.m = -INFINITY;
    s.l = 0.f;
#pragma unroll
    for (int j = 0; j < kPer; ++j) s.v[j] = 0.f;
    for (int k = c0 + lane; k <= c1; k += 32) s.m = fmaxf(s.m, __ldcg(&p.ml[place(k)]).x);
    const auto weights = [&](int i) {
        return i < n ? __ldcg(&p.ml[place(c0 + first + step * i)]) : make_float2(-INFINITY, 0.f);
    };
    float2 a = weights(lane);
#pragma unroll
    for (int o = 16; o; o >>= 1) s.m = fmaxf(s.m, __shfl_xor_sync(0xffffffffu, s.m, o));
    for (int i0 = 0; i0 < n; i0 += kAhead) {
        const int at = i0 & 31;
        if (i0 > 0) {
            fetch(i0);
            if (at == 0) a = weights(i0 + lane);
        }
        const float f = kv_factor(a.x, s.m), w = a.y * f;
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const float g = __shfl_sync(0xffffffffu, f, at + i), h = __shfl_sync(0xffffffffu, w, at + i);
            if (i0 + i >= n) continue;
            s.l += h;
#pragma unroll
            for (int j = 0; j < kPer; ++j) s.v[j] = fmaf(__uint_as_float(x[i][j]), g, s.v[j]);
        }
    }
    return s;
}
// One warp: a row's sum to the output.
template <int DT, int D>
__device__ __forceinline__ void kv_write_row(const KvParams &p, const KvSum<D> &s, int row, int head, int lane) {
    constexpr int kPer = D / 32;
    const float inv = s.l == 0.f ? 0.f : 1.f / s.l;
    uint32_t *dst = reinterpret_cast<uint32_t *>(p.out + (int64_t)row * p.out_stride + (int64_t)head * D + kPer * lane);
    const uint32_t lo = kv_down2<DT>(s.v[0] * inv, s.v[1] * inv);
    if (kPer == 4)
        *reinterpret_cast<uint2 *>(dst) = make_uint2(lo, kv_down2<DT>(s.v[kPer - 2] * inv, s.v[kPer - 1] * inv));
    else
        *dst = lo;
    if (p.lse && lane == 0) p.lse[(int64_t)row * p.heads + head] = kv_lse(s.m, s.l);
}

// -------------------------------------------------------------------- host --
// spx_kv_attention.cu
int kv_cache_check(const spx_kv_cache *c);
// spx_kv_tiles.cu: calls of more rows, on `blocks` blocks.
constexpr int kKvTileRows = 128;  // rows of one product
inline int kv_tile_tokens(int group) { return kKvTileRows / group; }
int launch_kv_tiles(KvParams &p, int dt, int blocks, cudaStream_t s);

}  // namespace spx
