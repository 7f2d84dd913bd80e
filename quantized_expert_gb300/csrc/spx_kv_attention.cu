// spx_kv_attention.cu -- attention over the paged cache of keys and values:
// entry point, and the launch for few rows.
//
//   out = sum_p w_p v_p / sum_p w_p,  w_p = exp(scale q . k_p - m),
//
// m a running reference of the row.  A unit of at most 16 (token, head) rows
// that share a key head (one token of a grouped model, a short chain) is bound
// by reading its keys and values once: 4 D bytes a token and key head against
// 4 D products a row, 16 of which the mma.sync tensor-core path does in a
// quarter of the time that the bytes take.  With two such tiles, 17 to 32 rows,
// it is no longer so (8 tokens of 4 heads, 16 requests of 4096 tokens: 75.9 us,
// and 55.9 in the launch for more rows; one request of 1000 tokens 11.9, 11.8).
#include <math.h>

#include "spx_kv.cuh"

namespace spx {

namespace {

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at)
                 : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at)
                 : "memory");
}
template <int DT>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if (DT == SPX_F16) {
        mma_16816(d, a, b0, b1);
    } else {
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
            "{%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    }
}
// 16 bytes from global to shared memory, or zeros.
__device__ __forceinline__ void cp_async16_or_zero(uint32_t dst, const void *src, bool real) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(real ? 16 : 0) : "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Block: a share of tiles, 8 warps.  Each warp takes 16 tokens of every tile of
// 128 on its own, from copies of its own that run kStages - 1 tiles ahead, into
// the units behind as well, so that a block's warps meet only at the end of a
// unit, where their sums are joined; 16 tokens lie in one page.  A block of 16
// tokens of keys (rows of D values, the 16-byte units of a row permuted by the
// row's last three bits) is the B operand of S = Q K^T, of values transposed
// that of O = P V; P passes from one product to the other in registers.
//
// Or (CLUSTER) the blocks of a cluster have the tiles of one unit, in equal
// parts: nothing is searched for, and the parts are joined from the blocks'
// shared memories instead of by way of the workspace and a counter.
//
// Measured, replayed from a graph: 65536 tokens of 8 key heads 47.6 us, 5.6 TB/s,
// 5 of them the launch's beginning (search, table, first copies) and 4 its end
// (sums of warps, of blocks); 32 requests of up to 4096 tokens and 16 key heads
// 91.7 us, 6.1 TB/s; 517 tokens of 16 heads 6.7 us, a chain of dependent reads
// (lengths, table, keys) and of barriers.  DRAM reads are the cache's bytes, once.
constexpr int kFewRows = 16;  // (token, head) rows of a unit at most
constexpr int kWarps = 8;
constexpr int kFewUnitCost = 1;  // of a unit beside its tiles, in tiles (65536 tokens of 8 units, us: 0 51.4, 1 47.6, 2 51.6; 32 requests of 16 units 92.7, 91.2, 92.0)
constexpr int kMostRanks = 8;  // blocks of a cluster
template <int D>
struct FewRows {
    static constexpr int kRows = kFewRows;
    static constexpr int kBlk = 16 * D * 2;  // keys or values of 16 tokens
    static constexpr int kStages = 3 * (128 / D);
    static constexpr int kRing = kWarps * kStages * 2 * kBlk;
    static constexpr int kSums = 4 * kRows * D * 4;  // sums of four warps
    static constexpr int kBytes = kRing + kSums + (kWarps + 1) * kRows * 8 + 64;
    static_assert(kBytes <= kSmemLimit, "shared memory of one block");
};

// The block that brings the last part of a unit joins them all.  A row's parts
// are dealt out to as many warps as there are for it; their sums are added in
// the order of the warps.  (A call of its own, for the registers of the loop.)
template <int DT, int D, int kRows>
__device__ __noinline__ void kv_join_unit(const KvParams &p, float *room, int c0, int c1, int rows, int row0, int head0) {
    constexpr int kPer = D / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // warps a row: one for every eight parts, which it reads together
    const int per = rows >= kWarps ? 1 : min(kWarps / rows, (c1 - c0) / 8 + 1);
    for (int i = warp; i < rows * per; i += kWarps) {  // (more than one round: per is 1)
        const int r = i / per, w = i - r * per, t = p.by_group(r), head = head0 + r - t * p.group;
        const KvSum<D> s = kv_sum_parts<D>(p, c0, c1, w, per, kRows, r, lane);
        if (per == 1) {
            kv_write_row<DT, D>(p, s, row0 + t, head, lane);
        } else {
#pragma unroll
            for (int j = 0; j < kPer; ++j) room[(i * kPer + j) * 32 + lane] = s.v[j];
            if (lane == 0) room[kWarps * D + 2 * i] = s.m, room[kWarps * D + 2 * i + 1] = s.l;
        }
    }
    if (per == 1) return;
    __syncthreads();
    if (warp < rows) {
        const int r = warp, t = p.by_group(r);
        KvSum<D> s;
        s.m = room[kWarps * D + 2 * r * per];
        s.l = 0.f;
#pragma unroll
        for (int j = 0; j < kPer; ++j) s.v[j] = 0.f;
        for (int w = 0; w < per; ++w) {
            s.l += room[kWarps * D + 2 * (r * per + w) + 1];
#pragma unroll
            for (int j = 0; j < kPer; ++j) s.v[j] += room[((r * per + w) * kPer + j) * 32 + lane];
        }
        kv_write_row<DT, D>(p, s, row0 + t, head0 + r - t * p.group, lane);
    }
}

__device__ __forceinline__ float2 ld_cluster2(uint32_t at) {
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t at) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(at)
                 : "memory");
    return v;
}
__device__ __forceinline__ uint32_t map_rank(uint32_t at, int rank) {
    uint32_t a;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(at), "r"(rank));
    return a;
}

template <int DT, int D, bool CLUSTER>
__global__ void __launch_bounds__(32 * kWarps, 1) kv_few_rows_kernel(const __grid_constant__ KvParams p) {
    using C = FewRows<D>;
    constexpr int kUnits = D / 8;  // 16-byte units of a row
    extern __shared__ __align__(1024) uint8_t smem[];
    float *sums = reinterpret_cast<float *>(smem + C::kRing);
    float2 *mls = reinterpret_cast<float2 *>(smem + C::kRing + C::kSums);  // [warp][row]
    float2 *own_ml = mls + kWarps * C::kRows;  // CLUSTER: [row] of the block
    int *last_part = reinterpret_cast<int *>(own_ml + C::kRows);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, quad = lane >> 2, pair = lane & 3;
    const uint32_t ring = smem_u32(smem) + warp * (C::kStages * 2 * C::kBlk);
    if (warp == 0) kv_prefetch(p, lane);
    griddep_wait();
    griddep_launch_dependents();
    KvShare share{};
    if (CLUSTER) {
        const int unit = (int)blockIdx.x / p.by_blocks.d, rank = (int)blockIdx.x - unit * p.by_blocks.d;
        share.b = unit / p.kv_heads;
        share.h = unit - share.b * p.kv_heads;
        share.rq = kv_req(p, share.b);
        // (a part without tiles, or of a request without rows, takes part in the join all the same)
        const int nt = share.rq.T > 0 ? kv_tiles(p, share.rq, 0, p.span) : 0, per = p.by_blocks(nt + p.by_blocks.d - 1);
        share.off = min(rank * per, nt);
        share.left = min(per, nt - share.off);
    } else {
        share = kv_find_share(p, p.span, lane);
        if (share.left <= 0) return;
    }

    // ---- copies
    KvWalk ahead;
    ahead.begin(p, share, p.span);
    int at = ahead.tile, page = 0;  // tile to copy next and its page
    const auto look_up = [&]() {
        if (ahead.left <= 0) return;
        const int p0 = kKvTile * at + 16 * warp;
        page = p0 < ahead.rq.len ? __ldg(p.table + (size_t)ahead.b * p.max_pages + p.by_page(p0)) : -1;
    };
    look_up();
    const auto copy = [&](int stage) {
        if (ahead.left > 0) {
            const int p0 = kKvTile * at + 16 * warp, n = min(ahead.rq.len - p0, 16);
            if (n > 0) {
                const bool ok = page >= 0 && page < p.num_pages;
                const int64_t place = (int64_t)(ok ? page : 0) * p.page_stride +
                                      (int64_t)(p0 - p.by_page(p0) * p.page_size) * p.token_stride +
                                      (int64_t)ahead.h * p.head_stride;
                const uint32_t dst = ring + stage * (2 * C::kBlk);
#pragma unroll
                for (int i = 0; i < kUnits / 2; ++i) {
                    const int t = i * (32 / kUnits) + lane / kUnits, u = lane % kUnits;
                    const bool real = ok && t < n;  // zeros past the length: their weight 0 times garbage might be a NaN
                    const int64_t from = place + (real ? (int64_t)t * p.token_stride + 8 * u : 0);
                    const uint32_t to = dst + t * (2 * D) + ((u ^ (t & 7)) << 4);
                    cp_async16_or_zero(to, p.k + from, real);
                    cp_async16_or_zero(to + C::kBlk, p.v + from, real);
                }
            }
            if (++at == ahead.end) {
                ahead.next(p, p.span);
                at = ahead.tile;
            }
            look_up();
        }
        cp_async_commit();
    };
#pragma unroll
    for (int s = 0; s < C::kStages - 1; ++s) copy(s);

    // ---- products
    KvWalk w;
    w.begin(p, share, p.span);
    if (CLUSTER) {
        if (share.rq.T == 0) return;  // (the cluster's blocks alike)
        w.tile = share.off;
        w.end = share.off + share.left;
    }
    int stage = 0;
#pragma unroll 1
    for (; CLUSTER || w.left > 0; w.next(p, p.span)) {
        const int rows = w.rq.T * p.group;
        // the queries, A operand: row quad (+ 8), values 16 ks + 2 pair (+ 8)
        uint32_t qa[D / 16][4];
        KvSeen seen[2];
        float m[2], l[2], o[D / 8][4];
#pragma unroll
        for (int y = 0; y < 2; ++y) {
            const int r = 8 * y + quad, t = p.by_group(r), j = r - t * p.group;
            const bool live = r < rows;
            const uint32_t *src = reinterpret_cast<const uint32_t *>(
                p.q + (int64_t)(w.rq.row0 + (live ? t : 0)) * p.q_stride + (int64_t)(w.h * p.group + (live ? j : 0)) * D);
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                qa[k][y] = live ? __ldg(src + 8 * k + pair) : 0u;
                qa[k][y + 2] = live ? __ldg(src + 8 * k + 4 + pair) : 0u;
            }
            seen[y] = kv_seen(p, w.rq, t);
            m[y] = -INFINITY;
            l[y] = 0.f;
        }
#pragma unroll
        for (int n = 0; n < D / 8; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[n][i] = 0.f;
        const int all = kv_all_see(p, w.rq, 0);
#pragma unroll 1
        for (int tile = w.tile; tile < w.end; ++tile) {
            copy(stage == 0 ? C::kStages - 1 : stage - 1);
            cp_async_wait<C::kStages - 1>();
            __syncwarp();
            const uint32_t ks = ring + stage * (2 * C::kBlk), vs = ks + C::kBlk;
            if (++stage == C::kStages) stage = 0;
            const int p0 = kKvTile * tile + 16 * warp;
            if (p0 >= w.rq.len) continue;
            float s[2][4];
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) s[n][i] = 0.f;
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                // tokens 0-7 and 8-15, units 2k and 2k + 1
                const int t = (lane & 7) + ((lane & 16) >> 1), u = 2 * k + ((lane >> 3) & 1);
                uint32_t b[4];
                ldsm4(b, ks + t * (2 * D) + ((u ^ (t & 7)) << 4));
                mma<DT>(s[0], qa[k], b[0], b[1]);
                mma<DT>(s[1], qa[k], b[2], b[3]);
            }
            if (p0 + 16 > all) {
                // what is not seen by every row: masks, and values that are not finite, whose weight 0 does not make
                // them 0.  A token with one is taken out of the product, and the rows that see it become NaNs.
                uint32_t bad = 0;
                {
                    const int t = lane >> 1;
#pragma unroll
                    for (int i = 0; i < kUnits / 2; ++i) {
                        const int u = i + (lane & 1) * (kUnits / 2);
                        const uint4 v = lds128(smem + (vs - smem_u32(smem)) + t * (2 * D) + ((u ^ (t & 7)) << 4));
                        uint32_t z = Elem<DT>::fma2(v.x, 0u, 0u);
                        z = Elem<DT>::fma2(v.y, 0u, z);
                        z = Elem<DT>::fma2(v.z, 0u, z);
                        z = Elem<DT>::fma2(v.w, 0u, z);
                        bad |= z & 0x7FFF7FFFu;
                    }
                    bad |= __shfl_xor_sync(0xffffffffu, bad, 1);
                    uint32_t mine = __ballot_sync(0xffffffffu, bad != 0);
                    bad = 0;
                    for (; mine; mine &= mine - 1) bad |= 1u << ((__ffs(mine) - 1) >> 1);
                    for (uint32_t left = bad; left; left &= left - 1) {
                        const int x = __ffs(left) - 1;
                        if (lane < kUnits)
                            *reinterpret_cast<uint4 *>(smem + (vs - smem_u32(smem)) + x * (2 * D) + (lane << 4)) =
                                make_uint4(0, 0, 0, 0);
                    }
                    __syncwarp();
                }
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const uint32_t word = seen[y].word(p0) & (p0 + 16 > w.rq.len ? (1u << (w.rq.len - p0)) - 1 : 0xFFFFu);
#pragma unroll
                    for (int n = 0; n < 2; ++n)
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            if (!(word >> (8 * n + 2 * pair + i) & 1)) s[n][2 * y + i] = -INFINITY;
                    if (word & bad)
#pragma unroll
                        for (int n = 0; n < D / 8; ++n) o[n][2 * y] = o[n][2 * y + 1] = NAN;
                }
            }
            float top[2], fac[2];
            bool rise = false;
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                float t = fmaxf(fmaxf(s[0][2 * y], s[0][2 * y + 1]), fmaxf(s[1][2 * y], s[1][2 * y + 1]));
                t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 1));
                t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 2));
                top[y] = t;
                rise |= (t - m[y]) * p.scale_log2 > kKvSlack;  // (scale > 0; not if both are -inf)
            }
            if (__any_sync(0xffffffffu, rise)) {
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const float mn = (top[y] - m[y]) * p.scale_log2 > kKvSlack ? top[y] : m[y];
                    fac[y] = mn == m[y] ? 1.f : ex2((m[y] - mn) * p.scale_log2);
                    m[y] = mn;
                    l[y] *= fac[y];
                }
#pragma unroll
                for (int n = 0; n < D / 8; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[n][i] *= fac[i >> 1];
            }
            float ref[2] = {kv_ref(m[0], p.scale_log2), kv_ref(m[1], p.scale_log2)};
            if (__any_sync(0xffffffffu, kv_far(m[0], p.scale_log2) || kv_far(m[1], p.scale_log2))) {
#pragma unroll
                for (int y = 0; y < 2; ++y)
                    if (kv_far(m[y], p.scale_log2)) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) s[i >> 1][2 * y + (i & 1)] -= m[y];
                        ref[y] = kKvShift;
                    }
            }
            uint32_t pa[4];
#pragma unroll
            for (int y = 0; y < 2; ++y) {
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    const float a = ex2(fmaf(s[n][2 * y], p.scale_log2, ref[y]));
                    const float b = ex2(fmaf(s[n][2 * y + 1], p.scale_log2, ref[y]));
                    l[y] += a + b;
                    pa[2 * n + y] = Elem<DT>::down2(a, b);  // rounded for the tensor cores; the weight's own sum is not
                }
            }
#pragma unroll
            for (int n = 0; n < D / 16; ++n) {
                // tokens 0-7 and 8-15 of unit 2n, then of unit 2n + 1
                const int t = lane & 15, u = 2 * n + (lane >> 4);
                uint32_t b[4];
                ldsm4_t(b, vs + t * (2 * D) + ((u ^ (t & 7)) << 4));
                mma<DT>(o[2 * n], pa, b[0], b[1]);
                mma<DT>(o[2 * n + 1], pa, b[2], b[3]);
            }
            __syncwarp();  // the stage may be copied into again
        }
        // ---- the warps' sums joined, in a fixed order
#pragma unroll
        for (int y = 0; y < 2; ++y) {
            m[y] *= p.scale_log2;  // from here on with the scale
            l[y] += __shfl_xor_sync(0xffffffffu, l[y], 1);
            l[y] += __shfl_xor_sync(0xffffffffu, l[y], 2);
            if (pair == 0) mls[warp * C::kRows + 8 * y + quad] = make_float2(m[y], l[y]);
        }
        __syncthreads();
        float top[2];
#pragma unroll
        for (int y = 0; y < 2; ++y) {
            float t = -INFINITY;
#pragma unroll
            for (int i = 0; i < kWarps; ++i) t = fmaxf(t, mls[i * C::kRows + 8 * y + quad].x);
            top[y] = t;
            const float f = kv_factor(m[y], t);
#pragma unroll
            for (int n = 0; n < D / 8; ++n) {
                o[n][2 * y] *= f;
                o[n][2 * y + 1] *= f;
            }
        }
        // warps 4-7 first, then warps 0-3 on top of them
#pragma unroll
        for (int half = 1; half >= 0; --half) {
            if (warp >> 2 == half)
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const int r = 8 * y + quad;
                    if (r >= rows) continue;
                    float2 *dst = reinterpret_cast<float2 *>(sums + ((warp & 3) * C::kRows + r) * D);
#pragma unroll
                    for (int n = 0; n < D / 8; ++n) {
                        const int u = (4 * n + pair) ^ (4 * (r & 3));  // spread over the banks
                        float2 v = make_float2(o[n][2 * y], o[n][2 * y + 1]);
                        if (half == 0) {
                            const float2 was = dst[u];
                            v.x += was.x;
                            v.y += was.y;
                        }
                        dst[u] = v;
                    }
                }
            __syncthreads();
        }
        const bool whole = CLUSTER || w.whole();
        const int place = 2 * blockIdx.x + (w.tile == 0);  // of a partial sum
        for (int i = threadIdx.x; i < rows * (D / 4); i += 32 * kWarps) {
            const int r = i / (D / 4), c = i % (D / 4), t = p.by_group(r), j = r - t * p.group;
            float mm = -INFINITY, ll = 0.f;
#pragma unroll
            for (int k = 0; k < kWarps; ++k) mm = fmaxf(mm, mls[k * C::kRows + r].x);
#pragma unroll
            for (int k = 0; k < kWarps; ++k) {
                // (a warp without tokens brings 0, one whose scores are all NaN no reference and a NaN, which stays)
                const float2 v = mls[k * C::kRows + r];
                ll += v.y * kv_factor(v.x, mm);
            }
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float4 a = *reinterpret_cast<const float4 *>(sums + (k * C::kRows + r) * D + ((4 * c) ^ (8 * (r & 3))));
                v.x += a.x;
                v.y += a.y;
                v.z += a.z;
                v.w += a.w;
            }
            if (CLUSTER) {
                *reinterpret_cast<float4 *>(sums + r * D + ((4 * c) ^ (8 * (r & 3)))) = v;
                if (c == 0) own_ml[r] = make_float2(mm, ll);
            } else if (whole) {
                const float inv = ll == 0.f ? 0.f : 1.f / ll;
                const int row = w.rq.row0 + t, head = w.h * p.group + j;
                *reinterpret_cast<uint2 *>(p.out + (int64_t)row * p.out_stride + (int64_t)head * D + 4 * c) =
                    make_uint2(kv_down2<DT>(v.x * inv, v.y * inv), kv_down2<DT>(v.z * inv, v.w * inv));
                if (p.lse && c == 0)
                    p.lse[(int64_t)row * p.heads + head] = kv_lse(mm, ll);
            } else {
                *reinterpret_cast<float4 *>(p.part + ((size_t)place * C::kRows + r) * D + 4 * c) = v;
                if (c == 0) p.ml[(size_t)place * C::kRows + r] = make_float2(mm, ll);
            }
        }
        if (CLUSTER) {
            // ---- the blocks' sums joined, in their order; a block writes a part of the results
            cluster_arrive();
            cluster_wait();
            const int ranks = p.by_blocks.d, rank = (int)cluster_rank();
            for (int i = rank * 32 * kWarps + threadIdx.x; i < rows * (D / 4); i += ranks * 32 * kWarps) {
                const int r = i / (D / 4), c = i % (D / 4), t = p.by_group(r), j = r - t * p.group;
                float2 a[kMostRanks];
                float4 x[kMostRanks];
                float mm = -INFINITY, ll = 0.f;
#pragma unroll
                for (int k = 0; k < kMostRanks; ++k) {
                    if (k >= ranks) continue;
                    a[k] = ld_cluster2(map_rank(smem_u32(own_ml + r), k));
                    x[k] = ld_cluster4(map_rank(smem_u32(sums + r * D + ((4 * c) ^ (8 * (r & 3)))), k));
                }
#pragma unroll
                for (int k = 0; k < kMostRanks; ++k)
                    if (k < ranks) mm = fmaxf(mm, a[k].x);
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int k = 0; k < kMostRanks; ++k) {
                    if (k >= ranks) continue;
                    const float f = kv_factor(a[k].x, mm);
                    ll += a[k].y * f;
                    v.x = fmaf(x[k].x, f, v.x);
                    v.y = fmaf(x[k].y, f, v.y);
                    v.z = fmaf(x[k].z, f, v.z);
                    v.w = fmaf(x[k].w, f, v.w);
                }
                const float inv = ll == 0.f ? 0.f : 1.f / ll;
                const int row = w.rq.row0 + t, head = w.h * p.group + j;
                *reinterpret_cast<uint2 *>(p.out + (int64_t)row * p.out_stride + (int64_t)head * D + 4 * c) =
                    make_uint2(kv_down2<DT>(v.x * inv, v.y * inv), kv_down2<DT>(v.z * inv, v.w * inv));
                if (p.lse && c == 0) p.lse[(int64_t)row * p.heads + head] = kv_lse(mm, ll);
            }
            cluster_arrive();  // no block leaves while its memory is read
            cluster_wait();
            break;
        }
        if (!whole) {
            const int c0 = w.tile == 0 ? (int)blockIdx.x : (w.flat - w.tile) / share.share;
            const int c1 = w.end == w.nt ? (int)blockIdx.x : (w.flat - w.tile + w.nt - 1) / share.share;
            __threadfence();
            __syncthreads();
            if (threadIdx.x == 0) {
                *last_part = atomicAdd(p.done + c0, 1u) == (uint32_t)(c1 - c0);
                if (*last_part) p.done[c0] = 0;
            }
            __syncthreads();
            if (*last_part) {
                __threadfence();
                kv_join_unit<DT, D, C::kRows>(p, sums, c0, c1, rows, w.rq.row0, w.h * p.group);
            }
        }
        __syncthreads();
    }
    cp_async_wait_all();
}

// Rows of a partial sum's place in the workspace: (token, head) rows of a unit
// of the launch that takes a call of `tokens` rows at most.
int place_rows(long long tokens, int group) {
    return tokens * group <= kFewRows ? kFewRows : tokens <= kv_tile_tokens(group) ? kKvTileRows : 2 * kKvTileRows;
}

// Tokens of a request at most: positions rounded up to a tile behind the rows of a unit are counted in 31 bits too.
constexpr int kMostLen = 0x7fff0000;

constexpr size_t up256(size_t n) { return (n + 255) / 256 * 256; }
constexpr size_t kDoneOffset = sizeof(WsHeader);
static_assert(kDoneOffset + kKvMaxBlocks * 4 <= SPX_KV_WORKSPACE_ZERO, "what must start at zero");
struct KvLayout {
    size_t seams, ml, part, bytes;
};
KvLayout kv_layout(int rows, int D) {
    KvLayout l;
    l.seams = SPX_KV_WORKSPACE_ZERO;
    l.ml = l.seams + up256((size_t)kKvMaxBlocks * 16);
    l.part = l.ml + up256((size_t)2 * kKvMaxBlocks * rows * 8);
    l.bytes = l.part + (size_t)2 * kKvMaxBlocks * rows * D * 4;
    return l;
}

template <int DT, int D, bool CLUSTER>
int launch_few(const KvParams &p, int blocks, cudaStream_t s) {
    const int st = set_smem<kv_few_rows_kernel<DT, D, CLUSTER>>(FewRows<D>::kBytes);
    if (st) return st;
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = latent_config(dim3((unsigned)blocks), 32 * kWarps, FewRows<D>::kBytes, s, attr,
                                           CLUSTER ? p.by_blocks.d : 1);
    return record_launch(cudaLaunchKernelEx(&cfg, kv_few_rows_kernel<DT, D, CLUSTER>, p));
}

// Clusters of 2, 4 and 8 blocks that the device runs at a time (0: not known).
template <int DT, int D>
const int *active_clusters() {
    static thread_local int done_dev = -1, active[3];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) dev = -1;
    if (dev < 0 || done_dev != dev) {
        for (int i = 0; i < 3; ++i) {
            cudaLaunchAttribute attr[2];
            cudaLaunchConfig_t cfg = latent_config(dim3(1024), 32 * kWarps, FewRows<D>::kBytes, nullptr, attr, 2 << i);
            active[i] = 0;
            if (dev < 0 || set_smem<kv_few_rows_kernel<DT, D, true>>(FewRows<D>::kBytes)) continue;
            if (cudaOccupancyMaxActiveClusters(&active[i], kv_few_rows_kernel<DT, D, true>, &cfg) != cudaSuccess) {
                cudaGetLastError();
                active[i] = 0;
            }
        }
        done_dev = dev;
    }
    return active;
}

// Blocks of a cluster for a call of few rows, or 0 for equal shares.  Clusters
// of S blocks take ceil(tiles / S) tiles' time, if the device runs all at once
// (8 of 8 blocks, 32 of 4); shares go by the number of all tiles, and their
// search and join cost two tiles more and a sixteenth for every part of a unit.
// Both, us, one token: 16 units of 512 tokens 6.6 and 8.5, of 2048 9.9 and 9.9;
// 8 units of 4096 tokens 9.4 and 10.3, of 8192 12.7 and 12.0; 1 unit of 4096
// tokens 9.6 and 11.7, of 8192 15.0 and 15.0; 128 units of 512 tokens (clusters
// in rounds) 13.6 and 8.6.
template <int DT, int D>
int cluster_ranks(long long units, int max_len, int blocks) {
    const long long tiles = (max_len + kKvTile - 1) / kKvTile;
    if (tiles <= 1 || units * tiles >= (1 << 20)) return 0;  // nothing to join; far from worth it
    const long long parts = blocks / units < tiles ? blocks / units : tiles;
    long long best = (units * tiles + blocks - 1) / blocks + 2 + parts / 16;
    const int *active = active_clusters<DT, D>();
    int ranks = 0;
    for (int i = 0; i < 3; ++i) {
        const int s = 2 << i;
        const long long cost = (tiles + s - 1) / s;
        if (units <= active[i] && cost < best) {
            best = cost;
            ranks = s;
        }
    }
    return ranks;
}

template <int DT, int D>
int launch_few_rows(KvParams &p, int sms, cudaStream_t s) {
    const long long units = (long long)p.B * p.kv_heads, tiles = units * ((p.max_len + kKvTile - 1) / kKvTile + (p.max_len == 0));
    const int ranks = cluster_ranks<DT, D>(units, p.max_len, sms);
    const int blocks = ranks ? (int)units * ranks : (int)(tiles < sms ? tiles : sms);  // no more blocks than tiles
    p.by_blocks.set(ranks ? ranks : blocks);
    return ranks ? launch_few<DT, D, true>(p, blocks, s) : launch_few<DT, D, false>(p, blocks, s);
}

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
        // (2^47 bytes, more than any device holds: sums of these stay within 64 bits, and strides within a tensor map's)
        if (st[next] >= (int64_t)1 << 38 || n[next] > ((int64_t)1 << 46) / st[next]) return SPX_ERR_UNSUPPORTED;
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
    // rows of (token, head) and cached tokens are counted in 31 bits, and so are the call's tiles with what units cost
    if ((long long)N * heads > 1 << 30 || (long long)max_q * heads > 1 << 30) return 0;
    const long long rows = max_q < N ? max_q : N;
    if ((double)B * kv_heads * (rows * (heads / kv_heads) / 64 + 1) * (max_len / kKvTile + 1 + kKvMostCost) > 2e9) return 0;
    return kv_layout(place_rows(rows, heads / kv_heads), D).bytes;
}

extern "C" int spx_kv_attention(const spx_kv_attention_args *a, spx_stream_t stream) {
    if (!a) return SPX_ERR_INVALID_ARG;
    const int st = kv_cache_check(a->cache);
    if (st) return st;
    const spx_kv_cache &c = *a->cache;
    if (!a->q_start || a->N < 0 || a->heads < 1 || a->max_q < 0 || a->max_len < 0 || a->heads % c.kv_heads)
        return SPX_ERR_INVALID_ARG;
    const float scale_log2 = a->scale * 1.4426950408889634f;
    if (!(a->scale > 0.f) || !(scale_log2 < INFINITY)) return SPX_ERR_INVALID_ARG;
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
    if (p.max_len > kMostLen) return SPX_ERR_UNSUPPORTED;
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
    p.scale_log2 = scale_log2;
    p.hdr = static_cast<WsHeader *>(a->ws);
    p.budget = a->wait_budget_ns ? a->wait_budget_ns : 2000000000ull;
    const int tokens = a->max_q < a->N ? a->max_q : a->N;
    const long long rows = (long long)tokens * p.group;
    uint8_t *ws = static_cast<uint8_t *>(a->ws);
    const KvLayout l = kv_layout(place_rows(tokens, p.group), c.D);
    p.done = reinterpret_cast<uint32_t *>(ws + kDoneOffset);
    p.ml = reinterpret_cast<float2 *>(ws + l.ml);
    p.part = reinterpret_cast<float *>(ws + l.part);
    const int sms = device_sm_count();
    if (sms < 1) return SPX_ERR_CUDA;
    const bool f16 = c.dtype == SPX_F16;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (rows <= kFewRows) {
        const int most = sms < kKvMaxBlocks ? sms : kKvMaxBlocks;
        p.span = a->max_q;
        p.unit_cost = kFewUnitCost;
        return c.D == 128 ? (f16 ? launch_few_rows<SPX_F16, 128>(p, most, s) : launch_few_rows<SPX_BF16, 128>(p, most, s))
                          : (f16 ? launch_few_rows<SPX_F16, 64>(p, most, s) : launch_few_rows<SPX_BF16, 64>(p, most, s));
    }
    p.seams = reinterpret_cast<int4 *>(ws + l.seams);
    return launch_kv_tiles(p, c.dtype, sms < kKvMaxBlocks ? sms : kKvMaxBlocks, s);
}
