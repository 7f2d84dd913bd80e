// spx_kv_attention.cu -- attention over the paged cache of keys and values:
// entry point, and the launch for few rows.
//
//   out = sum_p w_p v_p / sum_p w_p,  w_p = exp(scale q . k_p - m),
//
// m a running reference of the row.  A unit of at most 32 (token, head) rows
// that share a key head (one token of a grouped model, a short chain or tree) is
// bound by reading its keys and values once: 4 D bytes a token and key head
// against 4 D products a row, 16 of which the mma.sync tensor-core path does in
// a quarter of the time that the bytes take.
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
constexpr int kWarps = 8;
template <int D, int RT>
struct FewRows {
    static constexpr int kRows = 16 * RT;
    static constexpr int kBlk = 16 * D * 2;  // keys or values of 16 tokens
    static constexpr int kStages = (RT == 1 ? 3 : 2) * (128 / D);
    static constexpr int kRing = kWarps * kStages * 2 * kBlk;
    static constexpr int kSums = 4 * kRows * D * 4;  // sums of four warps
    static constexpr int kBytes = kRing + kSums + kWarps * kRows * 8 + 64;
    static_assert(kBytes <= kSmemLimit, "shared memory of one block");
};

template <int DT, int D, int RT>
__global__ void __launch_bounds__(32 * kWarps, 1) kv_few_rows_kernel(const __grid_constant__ KvParams p) {
    using C = FewRows<D, RT>;
    constexpr int kUnits = D / 8;  // 16-byte units of a row
    extern __shared__ __align__(1024) uint8_t smem[];
    float *sums = reinterpret_cast<float *>(smem + C::kRing);
    float2 *mls = reinterpret_cast<float2 *>(smem + C::kRing + C::kSums);  // [warp][row]
    int *last_part = reinterpret_cast<int *>(mls + kWarps * C::kRows);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, quad = lane >> 2, pair = lane & 3;
    const uint32_t ring = smem_u32(smem) + warp * (C::kStages * 2 * C::kBlk);
    griddep_wait();
    griddep_launch_dependents();
    const KvShare share = kv_find_share(p, p.span, lane);
    if (share.left <= 0) return;

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
    int stage = 0;
#pragma unroll 1
    for (; w.left > 0; w.next(p, p.span)) {
        const int rows = w.rq.T * p.group;
        // the queries, A operand: row quad (+ 8), values 16 ks + 2 pair (+ 8)
        uint32_t qa[RT][D / 16][4];
        KvSeen seen[RT][2];
        float m[RT][2], l[RT][2], o[RT][D / 8][4];
#pragma unroll
        for (int x = 0; x < RT; ++x)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                const int r = 16 * x + 8 * y + quad, t = p.by_group(r), j = r - t * p.group;
                const bool live = r < rows;
                const uint32_t *src = reinterpret_cast<const uint32_t *>(
                    p.q + (int64_t)(w.rq.row0 + (live ? t : 0)) * p.q_stride + (int64_t)(w.h * p.group + (live ? j : 0)) * D);
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    qa[x][k][y] = live ? __ldg(src + 8 * k + pair) : 0u;
                    qa[x][k][y + 2] = live ? __ldg(src + 8 * k + 4 + pair) : 0u;
                }
                seen[x][y] = kv_seen(p, w.rq, t);
                m[x][y] = -INFINITY;
                l[x][y] = 0.f;
            }
#pragma unroll
        for (int x = 0; x < RT; ++x)
#pragma unroll
            for (int n = 0; n < D / 8; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[x][n][i] = 0.f;
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
            float s[RT][2][4];
#pragma unroll
            for (int x = 0; x < RT; ++x)
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) s[x][n][i] = 0.f;
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                // tokens 0-7 and 8-15, units 2k and 2k + 1
                const int t = (lane & 7) + ((lane & 16) >> 1), u = 2 * k + ((lane >> 3) & 1);
                uint32_t b[4];
                ldsm4(b, ks + t * (2 * D) + ((u ^ (t & 7)) << 4));
#pragma unroll
                for (int x = 0; x < RT; ++x) {
                    mma<DT>(s[x][0], qa[x][k], b[0], b[1]);
                    mma<DT>(s[x][1], qa[x][k], b[2], b[3]);
                }
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
                for (int x = 0; x < RT; ++x)
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const uint32_t word = seen[x][y].word(p0) & (p0 + 16 > w.rq.len ? (1u << (w.rq.len - p0)) - 1 : 0xFFFFu);
#pragma unroll
                        for (int n = 0; n < 2; ++n)
#pragma unroll
                            for (int i = 0; i < 2; ++i)
                                if (!(word >> (8 * n + 2 * pair + i) & 1)) s[x][n][2 * y + i] = -INFINITY;
                        if (word & bad)
#pragma unroll
                            for (int n = 0; n < D / 8; ++n) o[x][n][2 * y] = o[x][n][2 * y + 1] = NAN;
                    }
            }
#pragma unroll
            for (int x = 0; x < RT; ++x) {
                float top[2], fac[2];
                bool rise = false;
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    float t = fmaxf(fmaxf(s[x][0][2 * y], s[x][0][2 * y + 1]), fmaxf(s[x][1][2 * y], s[x][1][2 * y + 1]));
                    t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 1));
                    t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 2));
                    top[y] = t * p.scale_log2;  // (scale > 0)
                    rise |= top[y] > m[x][y] + kKvSlack;
                }
                if (__any_sync(0xffffffffu, rise)) {
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const float mn = top[y] > m[x][y] + kKvSlack ? top[y] : m[x][y];
                        fac[y] = mn == m[x][y] ? 1.f : kv_ex2(m[x][y] - mn);
                        m[x][y] = mn;
                        l[x][y] *= fac[y];
                    }
#pragma unroll
                    for (int n = 0; n < D / 8; ++n)
#pragma unroll
                        for (int i = 0; i < 4; ++i) o[x][n][i] *= fac[i >> 1];
                }
                uint32_t pa[4];
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const float ref = m[x][y] == -INFINITY ? 0.f : kKvShift - m[x][y];
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        const float a = kv_ex2(fmaf(s[x][n][2 * y], p.scale_log2, ref));
                        const float b = kv_ex2(fmaf(s[x][n][2 * y + 1], p.scale_log2, ref));
                        l[x][y] += a + b;
                        pa[2 * n + y] = Elem<DT>::down2(a, b);  // rounded for the tensor cores; the weight's own sum is not
                    }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) *reinterpret_cast<uint32_t *>(&s[x][0][i]) = pa[i];
            }
#pragma unroll
            for (int n = 0; n < D / 16; ++n) {
                // tokens 0-7 and 8-15 of unit 2n, then of unit 2n + 1
                const int t = lane & 15, u = 2 * n + (lane >> 4);
                uint32_t b[4];
                ldsm4_t(b, vs + t * (2 * D) + ((u ^ (t & 7)) << 4));
#pragma unroll
                for (int x = 0; x < RT; ++x) {
                    const uint32_t pa[4] = {__float_as_uint(s[x][0][0]), __float_as_uint(s[x][0][1]),
                                            __float_as_uint(s[x][0][2]), __float_as_uint(s[x][0][3])};
                    mma<DT>(o[x][2 * n], pa, b[0], b[1]);
                    mma<DT>(o[x][2 * n + 1], pa, b[2], b[3]);
                }
            }
            __syncwarp();  // the stage may be copied into again
        }
        // ---- the warps' sums joined, in a fixed order
#pragma unroll
        for (int x = 0; x < RT; ++x)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                l[x][y] += __shfl_xor_sync(0xffffffffu, l[x][y], 1);
                l[x][y] += __shfl_xor_sync(0xffffffffu, l[x][y], 2);
                if (pair == 0) mls[warp * C::kRows + 16 * x + 8 * y + quad] = make_float2(m[x][y], l[x][y]);
            }
        __syncthreads();
        float top[RT][2];
#pragma unroll
        for (int x = 0; x < RT; ++x)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                float t = -INFINITY;
#pragma unroll
                for (int i = 0; i < kWarps; ++i) t = fmaxf(t, mls[i * C::kRows + 16 * x + 8 * y + quad].x);
                top[x][y] = t;
                const float f = kv_factor(m[x][y], t);
#pragma unroll
                for (int n = 0; n < D / 8; ++n) {
                    o[x][n][2 * y] *= f;
                    o[x][n][2 * y + 1] *= f;
                }
            }
        // warps 4-7 first, then warps 0-3 on top of them
#pragma unroll
        for (int half = 1; half >= 0; --half) {
            if (warp >> 2 == half)
#pragma unroll
                for (int x = 0; x < RT; ++x)
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const int r = 16 * x + 8 * y + quad;
                        if (r >= rows) continue;
                        float2 *dst = reinterpret_cast<float2 *>(sums + ((warp & 3) * C::kRows + r) * D);
#pragma unroll
                        for (int n = 0; n < D / 8; ++n) {
                            const int u = (4 * n + pair) ^ (4 * (r & 3));  // spread over the banks
                            float2 v = make_float2(o[x][n][2 * y], o[x][n][2 * y + 1]);
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
        const bool whole = w.whole();
        const int place = 2 * blockIdx.x + (w.tile == 0);  // of a partial sum
        for (int i = threadIdx.x; i < rows * (D / 4); i += 32 * kWarps) {
            const int r = i / (D / 4), c = i % (D / 4), t = p.by_group(r), j = r - t * p.group;
            float mm = -INFINITY, ll = 0.f;
#pragma unroll
            for (int k = 0; k < kWarps; ++k) mm = fmaxf(mm, mls[k * C::kRows + r].x);
#pragma unroll
            for (int k = 0; k < kWarps; ++k) {
                const float2 v = mls[k * C::kRows + r];
                if (v.x != -INFINITY) ll += v.y * kv_ex2(v.x - mm);
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
            if (whole) {
                const float inv = ll == 0.f ? 0.f : 1.f / ll;
                const int row = w.rq.row0 + t, head = w.h * p.group + j;
                *reinterpret_cast<uint2 *>(p.out + (int64_t)row * p.out_stride + (int64_t)head * D + 4 * c) =
                    make_uint2(Elem<DT>::down2(v.x * inv, v.y * inv), Elem<DT>::down2(v.z * inv, v.w * inv));
                if (p.lse && c == 0)
                    p.lse[(int64_t)row * p.heads + head] = kv_lse(mm, ll);
            } else {
                *reinterpret_cast<float4 *>(p.part + ((size_t)place * C::kRows + r) * D + 4 * c) = v;
                if (c == 0) p.ml[(size_t)place * C::kRows + r] = make_float2(mm, ll);
            }
        }
        if (!whole) {
            // ---- the block that brings the last part of a unit joins them all, in their order
            const int c0 = (w.flat - w.tile) / share.share, c1 = (w.flat - w.tile + w.nt - 1) / share.share;
            __threadfence();
            __syncthreads();
            if (threadIdx.x == 0) {
                *last_part = atomicAdd(p.done + c0, 1u) == (uint32_t)(c1 - c0);
                if (*last_part) p.done[c0] = 0;
            }
            __syncthreads();
            if (*last_part) {
                __threadfence();
                for (int r = warp; r < rows; r += kWarps) {
                    const int t = p.by_group(r), j = r - t * p.group;
                    kv_join_row<DT, D>(p, c0, c1, C::kRows, r, w.rq.row0 + t, w.h * p.group + j, lane);
                }
            }
        }
        __syncthreads();
    }
    cp_async_wait_all();
}

bool al16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// Rows of a partial sum's place in the workspace: (token, head) rows of a unit
// of the launch that takes a call of `tokens` rows at most.
constexpr int kFewRows = 32;
int place_rows(long long tokens, int group) {
    return tokens * group <= kFewRows ? kFewRows : tokens <= kv_tile_tokens(group) ? kKvTileRows : 2 * kKvTileRows;
}

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

template <int DT, int D, int RT>
int launch_few(const KvParams &p, int blocks, cudaStream_t s) {
    const int st = set_smem<kv_few_rows_kernel<DT, D, RT>>(FewRows<D, RT>::kBytes);
    if (st) return st;
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = latent_config(dim3((unsigned)blocks), 32 * kWarps, FewRows<D, RT>::kBytes, s, attr, 1);
    return record_launch(cudaLaunchKernelEx(&cfg, kv_few_rows_kernel<DT, D, RT>, p));
}
template <int DT, int D>
int launch_few_rt(const KvParams &p, int blocks, long long rows, cudaStream_t s) {
    return rows <= 16 ? launch_few<DT, D, 1>(p, blocks, s) : launch_few<DT, D, 2>(p, blocks, s);
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
    return kv_layout(place_rows(rows, heads / kv_heads), D).bytes;
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
        // no more blocks than tiles
        const long long most = (long long)c.B * c.kv_heads * ((p.max_len + kKvTile - 1) / kKvTile + (p.max_len == 0));
        const int blocks = (int)(most < sms && most < kKvMaxBlocks ? most : sms < kKvMaxBlocks ? sms : kKvMaxBlocks);
        p.span = a->max_q;
        p.unit_cost = 0;
        return c.D == 128 ? (f16 ? launch_few_rt<SPX_F16, 128>(p, blocks, rows, s) : launch_few_rt<SPX_BF16, 128>(p, blocks, rows, s))
                          : (f16 ? launch_few_rt<SPX_F16, 64>(p, blocks, rows, s) : launch_few_rt<SPX_BF16, 64>(p, blocks, rows, s));
    }
    p.seams = reinterpret_cast<int4 *>(ws + l.seams);
    return launch_kv_tiles(p, c.dtype, sms < kKvMaxBlocks ? sms : kKvMaxBlocks, s);
}
