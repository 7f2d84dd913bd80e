// spx_latent_prompt.cu -- attention over the paged latent cache, expanded form.
//
// A prompt has so many query rows that every head's keys and values are worth
// writing out: a query-key pair then costs dn + P + dv = 320 products instead
// of R + P + R = 1088.  Two launches:
//
//   expand launch     k[h] = W_uk[h] c, v[h] = W_uv[h] c for every cached token
//                     of the call's requests, rounded to the type, and the
//                     rotated parts side by side;
//   attention launch  softmax(scale (q_nope . k + q_rope . r)) v per head, a
//                     running maximum and sum per row.
//
// The second is a programmatic dependent of the first.
#include <math.h>
#include <string.h>

#include "spx_latent.cuh"
#include "spx_tcgen05.cuh"

namespace spx {

namespace {

constexpr int kPTile = 128;                 // tokens of a tile: rows of one product
constexpr int kPiece = kPTile * 128;        // 128 rows x 64 values, 16 KB

struct PromptMaps {
    CUtensorMap cache;       // [page][piece][token][64], boxes of 1 piece x box_tokens
    CUtensorMap w_uk, w_uv;  // [piece][head * 128 + row][64], boxes of 1 piece x 128 rows
    CUtensorMap q;           // [head][piece][token][64], boxes of 3 pieces x 128 tokens
};

// Keys and values are written as the attention launch reads them, in core
// matrices (units of 8 values, 16 bytes, of consecutive tokens side by side):
// per head, request and tile of 128 tokens 32 KB each, keys [unit 16][token
// 128][8], values [half 2][unit 16][token 64][8]; the rotated parts [unit
// 8][token 128][8] per request and tile.  A warp of tokens then stores 512
// bytes in a row (rows of 256 bytes a token cost four times the store
// transactions and held up the products), and a piece is one plain copy.
__device__ __forceinline__ size_t key_unit(int tile, int t, int unit) {
    return (size_t)tile * (2 * kPiece / 2) + (size_t)unit * (kPTile * 8) + (size_t)(t & (kPTile - 1)) * 8;
}
__device__ __forceinline__ size_t value_unit(int tile, int t, int unit) {
    return (size_t)tile * (2 * kPiece / 2) + (size_t)(t >> 6 & 1) * (kPiece / 2) + (size_t)unit * (64 * 8) +
           (size_t)(t & 63) * 8;
}

// ----------------------------------------------------------- expand launch --
// Block (token tile, group of heads, request): the tile's latent vectors stay
// in shared memory (A, R / 64 pieces of 128 tokens) while the heads' weights
// stream past in stages of 64 latent columns, W_uk[h] and W_uv[h] as the 256
// rows of B: D[128 tokens x 256] = keys and values of one head, in one of two
// accumulators.  A product of 256 columns takes 512 cycles a stage, in which an
// SM would have to fetch 32 KB from L2, 64 bytes a cycle and more than it gets:
// two blocks of neighbouring token tiles form one product of 256 tokens, for
// which each holds one of the two matrices, 32 bytes a cycle (each fetching one
// for both by multicast: 154 us for four prompt chunks replayed from a graph,
// halved 147; now 140, and 143 in a stream of calls).  A head's
// 8 stages take 4430 cycles while nothing else moves and 5000 beside the stores
// of the head before: 4096 tokens and 16 heads 15 us, 1.15 PFLOP/s.  Keys and
// values are rounded to the type once, as a cache of them would be.
constexpr int kExStages = 6;
constexpr int kExStage = kPiece;  // this block's half of B
constexpr int kExThreads = 384;  // copies of W, products, 2 warps' copies of A, 8 epilogue warps
struct ExMisc {
    uint64_t afull[8], wfull[kExStages], wempty[kExStages], dfull[2], dempty[2], fin;
    uint32_t tmem;
    int abort;
};
constexpr size_t kExSmem = 8 * (size_t)kPiece + kExStages * (size_t)kExStage + 1024;
static_assert(kExSmem <= (size_t)kSmemLimit && sizeof(ExMisc) <= 1024, "shared memory of one block");

template <int DT>
__global__ void __launch_bounds__(kExThreads, 1)
    latent_expand_kernel(const __grid_constant__ LatentParams p, const __grid_constant__ PromptMaps maps) {
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t *as = smem, *ws = as + 8 * kPiece;
    ExMisc &m = *reinterpret_cast<ExMisc *>(ws + kExStages * kExStage);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int b = blockIdx.z, t0 = kPTile * blockIdx.x, h0 = p.head_group * blockIdx.y;
    const int nh = min(p.head_group, p.heads - h0), nc = p.R / 64;
    const uint32_t rank = cluster_rank();
    if (threadIdx.x == 0) {
        for (int c = 0; c < nc; ++c) mbar_init(&m.afull[c], 2);
        for (int s = 0; s < kExStages; ++s) {
            mbar_init(&m.wfull[s], 1);
            mbar_init(&m.wempty[s], 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&m.dfull[s], 1);
            mbar_init(&m.dempty[s], 16);  // the epilogue warps of both blocks
        }
        mbar_init(&m.fin, 1);
        m.abort = 0;
        fence_mbar_init();
    }
    griddep_wait();
    griddep_launch_dependents();
    const LatentReq rq = latent_req(p, b);
    if (t0 - kPTile * (int)rank >= rq.len || rq.T == 0) return;  // both blocks of the cluster alike
    if (warp == 1) pair_tmem_alloc(&m.tmem, 512);
    tc_fence_before();
    __syncthreads();
    cluster_arrive();  // the other block's barriers exist
    cluster_wait();
    tc_fence_after();
    const uint32_t tmem = m.tmem;
    const WaitCtl ctl{&m.abort, &p.hdr->status, p.budget, SITE_LATENT};
    uint32_t lost = 0;  // heads (of the block's) in which this lane's token has a value that is not finite

    if (warp == 2 || warp == 3) {
        // ---- the latent vectors of 64 tokens
        const uint64_t pol = policy_evict_normal();
        const int bt = p.box_tokens, nb = 64 / bt, half = warp - 2;
        const int pos = t0 + 64 * half + bt * (lane & 3), pi = p.by_page(pos), my_at = pos - pi * p.page_size;
        int my_page = pos < rq.len ? __ldg(p.table + (size_t)b * p.max_pages + pi) : p.num_pages;
        if (my_page < 0 || my_page >= p.num_pages) my_page = p.num_pages;
        // (both blocks' copies count on rank 0's barriers, where the products are issued)
        for (int c = 0; c < nc; ++c) {
            const uint32_t afull = smem_of_rank(&m.afull[c], 0);
            if (rank == 0 && elect_one()) mbar_arrive_expect_tx(&m.afull[c], kPiece);
            __syncwarp();
            for (int j = 0; j < nb; ++j) {
                const int at = __shfl_sync(0xffffffffu, my_at, j), page = __shfl_sync(0xffffffffu, my_page, j);
                if (elect_one())
                    pair_load_4d(as + c * kPiece + half * (kPiece / 2) + j * bt * 128, &maps.cache, 0, at, c, page,
                                 afull, pol);
                __syncwarp();
            }
        }
        // ---- their rotated parts (once for all heads), a token a lane
        if (h0 == 0 && t0 < rq.len)
            for (int t = t0 + 64 * half + lane; t < t0 + 64 * half + 64; t += 32) {
                const int pg_i = p.by_page(t), pg = t < rq.len ? __ldg(p.table + (size_t)b * p.max_pages + pg_i) : -1;
                const bool ok = pg >= 0 && pg < p.num_pages;
                const uint16_t *src = p.cache + (int64_t)(ok ? pg : 0) * p.page_stride +
                                      (int64_t)(t - pg_i * p.page_size) * p.token_stride + p.R;
                uint16_t *dst = p.rope_x + ((size_t)b * (p.kv_rows / kPTile) + blockIdx.x) * (kPiece / 2) +
                                (size_t)(t & (kPTile - 1)) * 8;
#pragma unroll
                for (int u = 0; u < 8; ++u)
                    *reinterpret_cast<uint4 *>(dst + u * (kPTile * 8)) =
                        ok ? *reinterpret_cast<const uint4 *>(src + 8 * u) : make_uint4(0, 0, 0, 0);
            }
    } else if (warp == 0) {
        // ---- the weights
        const uint64_t pol = policy_evict_last();
        uint32_t it = 0;
        bool ok = true;
        for (int h = h0; ok && h < h0 + nh; ++h)
            for (int c = 0; c < nc; ++c, ++it) {
                const uint32_t s = it % kExStages;
                if (!(ok = ctl_wait(&m.wempty[s], ((it / kExStages) & 1) ^ 1, ctl))) break;
                if (elect_one()) {
                    if (rank == 0) mbar_arrive_expect_tx(&m.wfull[s], 2 * kExStage);
                    pair_load_3d(ws + s * kExStage, rank ? &maps.w_uv : &maps.w_uk, 0, 128 * h, c,
                                 smem_of_rank(&m.wfull[s], 0), pol);
                }
                __syncwarp();
            }
    } else if (warp == 1) {
        if (rank == 0) {
            // ---- products
            const uint32_t id = idesc_f16_f32(256, 256) | (DT == SPX_BF16 ? kIdescBf16 : 0u);
            const uint64_t ad = sw128_desc(smem_u32(as)), wd = sw128_desc(smem_u32(ws));
            uint32_t it = 0;
            bool ok = true;
            for (int i = 0; ok && i < nh; ++i) {
                const uint32_t d = tmem + (i & 1) * 256;
                if (!(ok = ctl_wait(&m.dempty[i & 1], ((i >> 1) & 1) ^ 1, ctl))) break;
                for (int c = 0; c < nc; ++c, ++it) {
                    const uint32_t s = it % kExStages;
                    if (i == 0 && !(ok = ctl_wait(&m.afull[c], 0, ctl))) break;
                    if (!(ok = ctl_wait(&m.wfull[s], (it / kExStages) & 1, ctl))) break;
                    tc_fence_after();
                    if (elect_one()) {
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            pair_umma_f16(d, ad + c * (kPiece / 16) + 2 * j, wd + s * (kExStage / 16) + 2 * j, id,
                                          (c | j) != 0);
                        pair_commit(&m.wempty[s]);
                        if (c == nc - 1) pair_commit(&m.dfull[i & 1]);
                    }
                    __syncwarp();
                }
            }
        }
    } else {
        // ---- epilogue: a token a lane, its keys (warps 4-7) or its values (warps 8-11)
        const int q = warp & 3, t = t0 + 32 * q + lane;
        const bool live = t < rq.len, values = warp >= 8;
        for (int i = 0; i < nh; ++i) {
            ctl_wait(&m.dfull[i & 1], (i >> 1) & 1, ctl);
            tc_fence_after();
            const size_t of_head = ((size_t)(h0 + i) * p.B + b) * p.kv_rows * 128;
            uint16_t *dst = values ? p.v_x + of_head + value_unit(blockIdx.x, t, 0) : p.k_x + of_head + key_unit(blockIdx.x, t, 0);
            const int step = values ? 64 * 8 : kPTile * 8;  // from unit to unit
#pragma unroll 1
            for (int x = 0; x < 128 && t0 < rq.len; x += 32) {
                uint32_t r[32];
                tmem_ld32(tmem + ((uint32_t)(32 * q) << 16) + (i & 1) * 256 + (values ? 128 : 0) + x, r);
                tmem_wait_ld();
                uint32_t o[16];
#pragma unroll
                for (int k = 0; k < 16; ++k)  // past the length: zeros
                    o[k] = live ? Elem<DT>::down2(__uint_as_float(r[2 * k]), __uint_as_float(r[2 * k + 1])) : 0u;
                // A value that is not finite, or that the type cannot hold, becomes 0, as its weight 0 in the rows
                // that do not see it times it would not be 0; a NaN in its key shows it to those that do.  Such a
                // key becomes a NaN (an infinity's score could be -inf, which only leaves the token out).  (0 times
                // all of them, summed, is a NaN if one is not finite.)
                uint32_t test = 0;
#pragma unroll
                for (int k = 0; k < 16; ++k) test = Elem<DT>::fma2(o[k], 0u, test);
                if (test & 0x7FFF7FFFu) {
#pragma unroll
                    for (int k = 0; k < 16; ++k)
                        o[k] = values ? Elem<DT>::finite2(o[k], 0u) : Elem<DT>::finite2(o[k], 0x7FFF7FFFu);
                    if (values) lost |= 1u << i;
                }
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    *reinterpret_cast<uint4 *>(dst + (x / 8 + k) * step) =
                        make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_remote(smem_of_rank(&m.dempty[i & 1], 0));
        }
    }
    tc_fence_before();
    __syncthreads();
    for (; lost; lost &= lost - 1) {  // behind the key's own stores
        const size_t of_head = ((size_t)(h0 + __ffs(lost) - 1) * p.B + b) * p.kv_rows * 128;
        p.k_x[of_head + key_unit(blockIdx.x, t0 + 32 * (warp & 3) + lane, 0)] = 0x7FFF;
    }
    __syncwarp();
    if (m.abort) {
        // (A block that has not given up has seen its last product, and with it every copy of both blocks; one
        // that has holds both back at the barrier below.)
        if (warp == 0) ctl_settle(kSettleNs);
        if (warp == 1 && rank == 0) {
            if (elect_one()) pair_commit(&m.fin);
            ctl_drain(&m.fin, 0, kSettleNs);
        }
        __syncwarp();
    }
    cluster_arrive_relaxed();  // both are done with the other's memories and barriers
    cluster_wait();
    if (warp == 1) {
        tc_fence_after();
        pair_tmem_dealloc(tmem, 512);
    }
    cluster_arrive_relaxed();
    cluster_wait();
}

// -------------------------------------------------------- attention launch --
// Block (two adjacent tiles of 128 query rows of a request, head).  Per tile X
// and key tile j:  S_X = Q_X K_j^T (128 x 128, 192 deep), softmax in registers
// (a row a thread), P_X back into S_X's tensor memory as the A operand of
// O_X += P_X V_j.  The two tiles share every key and value tile and take
// turns: while one's softmax runs, the other's products do.  Each has a warp of
// its own to issue them (O_X(j), then S_X(j + 1)): the waits for barriers that
// are long complete cost 150 cycles each, and with one issuing warp for both
// they left the tensor cores idle half the time.  The two pass a turn to each
// other, for otherwise they fall into step, both softmaxes at once and then
// both products (3900 cycles per key tile instead of 3100).  Tensor memory:
// S_0, S_1, O_0, O_1, 128 columns each.  Shared memory: Q 96 KB, keys in a
// ring of 5 pieces (128 tokens x 64), values in one of 3 halves (64 tokens x
// 128).
//
// Per key tile 2 (768 + 512) cycles of products against 2 x 16384 exponentials;
// the keys and values of a tile, 80 KB, come once per 256 rows (26 bytes a
// cycle and SM).  3100 cycles: a softmax takes 1250 from S to the last of P, and
// a slot of either ring is free too late for the copy into it to be there when
// it is wanted (both launches for 4096 tokens, replayed from a graph: 6 + 2 pieces
// 78 us, 4 + 4 85, 5 + 3 75; half pieces 78, for twice the copies and commits).
// 4096 tokens, 16 heads: 58 us; the call 79 in a stream of calls, 74 replayed.
// P is rounded to the type, scaled by 2^kFaShift off the subnormals of fp16.
constexpr int kFaThreads = 384;  // copies of Q and K, two issuers of products, copies of V; 4 softmax warps per tile
constexpr int kKRing = 5, kVRing = 3;
struct FaMisc {
    uint64_t qfull[2], kfull[2], rfull[2], vfull[2][2];  // by tiles, of which two are under way; rfull: the rotated part, vfull: by halves
    uint64_t kempty[kKRing], vempty[kVRing];     // both issuers are done with a piece
    uint64_t sfull[2], pfull[2][2], odone[2], fin[2];  // pfull: by halves of the keys
    uint64_t turn[2];                            // the other issuer has handed in its products
    uint32_t tmem;
    int abort;
};
constexpr size_t kFaSmem = 6 * (size_t)kPiece + kKRing * (size_t)kPiece + kVRing * (size_t)kPiece + 1024;
static_assert(kFaSmem <= (size_t)kSmemLimit && sizeof(FaMisc) <= 1024, "shared memory of one block");
constexpr float kFaSlack = 8.f, kFaShift = 5.f;  // as in the absorbed form

template <int N>
struct Ring {
    uint32_t i = 0, phase = 0;
    __device__ __forceinline__ void next() {
        if (++i == N) {
            i = 0;
            phase ^= 1;
        }
    }
};

template <int DT>
__global__ void __launch_bounds__(kFaThreads, 1)
    latent_prompt_kernel(const __grid_constant__ LatentParams p, const __grid_constant__ PromptMaps maps) {
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t *qs = smem, *ks = qs + 6 * kPiece, *vs = ks + kKRing * kPiece;
    FaMisc &m = *reinterpret_cast<FaMisc *>(vs + kVRing * kPiece);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // the longest rows first, as their blocks take longest
    const int b = blockIdx.y, h = blockIdx.x % p.heads, qt = (int)(gridDim.x / p.heads) - 1 - (int)(blockIdx.x / p.heads);
    const LatentReq rq = latent_req(p, b);
    const int r0 = 2 * kPTile * qt;
    if (r0 >= rq.T) {
        griddep_wait();
        return;
    }
    // key tiles of each query tile (0: no rows, or none that sees anything)
    int n[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        const int last = min(r0 + kPTile * (x + 1), rq.T) - 1;
        n[x] = last < r0 + kPTile * x ? 0 : (latent_limit(p, rq, last) + kPTile - 1) / kPTile;
    }
    const int most = max(n[0], n[1]);
    if (threadIdx.x == 0) {
        for (int i = 0; i < kKRing; ++i) mbar_init(&m.kempty[i], 2);
        for (int i = 0; i < kVRing; ++i) mbar_init(&m.vempty[i], 2);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&m.qfull[i], 1);
            mbar_init(&m.kfull[i], 1);
            mbar_init(&m.rfull[i], 1);
            mbar_init(&m.vfull[i][0], 1);
            mbar_init(&m.vfull[i][1], 1);
            mbar_init(&m.sfull[i], 1);
            mbar_init(&m.pfull[i][0], 4);
            mbar_init(&m.pfull[i][1], 4);
            mbar_init(&m.odone[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&m.fin[i], 1);
            mbar_init(&m.turn[i], 1);
        }
        m.abort = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(&m.tmem, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = m.tmem;
    const WaitCtl ctl{&m.abort, &p.hdr->status, p.budget, SITE_LATENT};

    if (warp == 0) {
        // ---- copies of Q and K
        const uint64_t pol = policy_evict_normal();
        for (int x = 0; x < 2; ++x)
            if (n[x] && elect_one()) {
                mbar_arrive_expect_tx(&m.qfull[x], 3 * kPiece);
                tma_load_4d(qs + 3 * x * kPiece, &maps.q, 0, rq.row0 + r0 + kPTile * x, 0, h, &m.qfull[x], pol);
            }
        __syncwarp();
        griddep_wait();
        Ring<kKRing> kr;
        bool ok = true;
        for (int j = 0; ok && j < most; ++j)
            for (int c = 0; c < 3; ++c, kr.next()) {
                if (!(ok = ctl_wait(&m.kempty[kr.i], kr.phase ^ 1, ctl))) break;
                if (elect_one()) {
                    uint64_t *full = c < 2 ? &m.kfull[j & 1] : &m.rfull[j & 1];
                    if (c != 1) mbar_arrive_expect_tx(full, c ? kPiece : 2 * kPiece);
                    const uint16_t *src = c < 2 ? p.k_x + ((size_t)h * p.B + b) * p.kv_rows * 128 + key_unit(j, 0, 8 * c)
                                                : p.rope_x + ((size_t)b * (p.kv_rows / kPTile) + j) * (kPiece / 2);
                    bulk_g2s(ks + kr.i * kPiece, src, kPiece, full, pol);
                }
                __syncwarp();
            }
    } else if (warp == 3) {
        // ---- copies of V: apart from those of K, which would wait behind them for room
        const uint64_t pol = policy_evict_normal();
        griddep_wait();
        Ring<kVRing> vr;
        bool ok = true;
        for (int j = 0; ok && j < most; ++j)
            for (int c = 0; c < 2; ++c, vr.next()) {
                if (!(ok = ctl_wait(&m.vempty[vr.i], vr.phase ^ 1, ctl))) break;
                if (elect_one()) {
                    mbar_arrive_expect_tx(&m.vfull[j & 1][c], kPiece);
                    bulk_g2s(vs + vr.i * kPiece,
                             p.v_x + ((size_t)h * p.B + b) * p.kv_rows * 128 + value_unit(j, 64 * c, 0), kPiece,
                             &m.vfull[j & 1][c], pol);
                }
                __syncwarp();
            }
    } else if (warp < 3) {
        // ---- products of one query tile
        const int x = warp - 1;
        const uint32_t fmt = DT == SPX_BF16 ? kIdescBf16 : 0u;
        const uint32_t id_s = idesc_f16_f32(128, 128) | fmt, id_o = idesc_f16_f32(128, 128) | fmt | kIdescBMn;
        const uint64_t qd = sw128_desc(smem_u32(qs) + 3 * x * kPiece), kd = plain_desc(smem_u32(ks), kPTile * 16, 128);
        const uint64_t vd = plain_desc(smem_u32(vs), 128, 64 * 16);  // a k-step: two units of K, 16 tokens of V
        const uint32_t st = tmem + 128 * x, ot = tmem + 256 + 128 * x;
        const int nx = n[x];
        Ring<kKRing> kr;
        Ring<kVRing> vr;
        bool ok = !nx || ctl_wait(&m.qfull[x], 0, ctl);
        // O_x(j - 1), then S_x(j), in one stretch behind everything that they wait for; past the tile's last
        // key both only pass the pieces on.  The rotated part of the keys, whose slot comes free last, has a
        // wait of its own behind the rest.
#pragma unroll 1
        for (int j = 0; ok && j <= most; ++j) {
            const bool has_o = j > 0 && j <= nx, has_s = j < nx;
            ok = (j == most || ctl_wait(&m.kfull[j & 1], (j >> 1) & 1, ctl)) &&
                 (j == 0 || ctl_wait(&m.vfull[(j - 1) & 1][0], ((j - 1) >> 1) & 1, ctl)) &&
                 // tile 1 goes behind tile 0's products of the same j, tile 0 behind tile 1's of the last
                 (x ? ctl_wait(&m.turn[1], j & 1, ctl) : j == 0 || ctl_wait(&m.turn[0], (j - 1) & 1, ctl)) &&
                 (!has_o || ctl_wait(&m.pfull[x][0], (j - 1) & 1, ctl));
            if (!ok) break;
            tc_fence_after();
            if (j > 0) {  // the first half while the softmax is at the second
                if (elect_one()) {
                    if (has_o) {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            umma_f16_ta(ot, st + 8 * i, vd + vr.i * (kPiece / 16) + 16 * i, id_o, (j != 1) | i);
                        umma_commit(&m.vempty[vr.i]);
                    } else {
                        mbar_arrive(&m.vempty[vr.i]);
                    }
                }
                __syncwarp();
                vr.next();
                ok = ctl_wait(&m.vfull[(j - 1) & 1][1], ((j - 1) >> 1) & 1, ctl) &&
                     (!has_o || ctl_wait(&m.pfull[x][1], (j - 1) & 1, ctl));
                if (!ok) break;
                tc_fence_after();
            }
            if (elect_one()) {
                if (has_o) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        umma_f16_ta(ot, st + 32 + 8 * i, vd + vr.i * (kPiece / 16) + 16 * i, id_o, 1);
                    umma_commit(&m.vempty[vr.i]);
                    if (j == nx) umma_commit(&m.odone[x]);
                } else if (j > 0) {
                    mbar_arrive(&m.vempty[vr.i]);
                }
                Ring<kKRing> k = kr;
                if (j < most)
#pragma unroll 1
                    for (int c = 0; c < 2; ++c, k.next()) {
                        if (has_s) {
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                umma_f16(st, qd + c * (kPiece / 16) + 2 * i, kd + k.i * (kPiece / 16) + 2 * kPTile * i, id_s, c | i);
                            umma_commit(&m.kempty[k.i]);
                        } else {
                            mbar_arrive(&m.kempty[k.i]);
                        }
                    }
                mbar_arrive(&m.turn[x ^ 1]);  // before the last piece, to hide the other's waking
            }
            __syncwarp();
            if (j > 0) vr.next();
            if (j == most) break;
            for (int c = 0; c < 2; ++c) kr.next();
            if (!(ok = ctl_wait(&m.rfull[j & 1], (j >> 1) & 1, ctl))) break;
            tc_fence_after();
            if (elect_one()) {
                if (has_s) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        umma_f16(st, qd + 2 * (kPiece / 16) + 2 * i, kd + kr.i * (kPiece / 16) + 2 * kPTile * i, id_s, 1);
                    umma_commit(&m.kempty[kr.i]);
                    umma_commit(&m.sfull[x]);
                } else {
                    mbar_arrive(&m.kempty[kr.i]);
                }
            }
            __syncwarp();
            kr.next();
        }
    } else if (warp >= 4) {
        // ---- softmax and results: a row a thread
        const int x = (warp - 4) >> 2, q = warp & 3, t = r0 + kPTile * x + 32 * q + lane;
        const uint32_t quarter = (uint32_t)(32 * q) << 16;
        const uint32_t st = tmem + quarter + 128 * x, ot = tmem + quarter + 256 + 128 * x;
        const bool live = t < rq.T;
        const int lim = live ? latent_limit(p, rq, t) : 0;
        const int lim_lo = latent_limit(p, rq, r0 + kPTile * x + 32 * q);  // the warp's first row sees least
        float mr = -INFINITY, l = 0.f;
#pragma unroll 1
        for (int j = 0; j < n[x]; ++j) {
            ctl_wait(&m.sfull[x], j & 1, ctl);
            tc_fence_after();
            const int p0 = kPTile * j;
            const bool masked = p0 + kPTile > lim_lo || !live;
            const int left = lim - p0;  // columns of this tile that the row sees
            uint32_t r[128];
#pragma unroll
            for (int c = 0; c < 4; ++c) tmem_ld32(st + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(r + 32 * c));
            tmem_wait_ld();
            if (__any_sync(0xffffffffu, masked))
#pragma unroll
                for (int k = 0; k < 128; ++k)
                    if (k >= left) r[k] = 0xFF800000u;
            float mx[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) mx[k] = __uint_as_float(r[k]);
#pragma unroll
            for (int k = 8; k < 128; ++k) mx[k & 7] = fmaxf(mx[k & 7], __uint_as_float(r[k]));
#pragma unroll
            for (int o = 4; o; o >>= 1)
#pragma unroll
                for (int k = 0; k < o; ++k) mx[k] = fmaxf(mx[k], mx[k + o]);
            const float top = mx[0] * p.scale_log2;  // (scale > 0)
            const bool rise = top > mr + kFaSlack;
            if (__any_sync(0xffffffffu, rise)) {
                const float mn = rise ? top : mr, f = mn == mr ? 1.f : ex2(mr - mn);
                mr = mn;
                l *= f;
                if (j > 0) {
                    // (O_x(j - 1) is done: S_x(j) came behind it)
#pragma unroll 1
                    for (int c = 0; c < 128; c += 16) {
                        uint32_t o[16];
                        tmem_ld16(ot + c, o);
#pragma unroll
                        for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                        tmem_st16(ot + c, o);
                    }
                }
            }
            const float ref = mr == -INFINITY ? 0.f : kFaShift - mr;
            const uint64_t sc2 = pack2(p.scale_log2, p.scale_log2), ref2 = pack2(ref, ref);
            uint64_t l2[2] = {0, 0};
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                uint32_t o[16];
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                    const float2 t = unpack2(fma2(pack2(__uint_as_float(r[32 * c + 2 * k]), __uint_as_float(r[32 * c + 2 * k + 1])),
                                                  sc2, ref2));
                    const float u = ex2(t.x), v = ex2(t.y);
                    l2[k & 1] = add2(l2[k & 1], pack2(u, v));
                    o[k] = Elem<DT>::down2(u, v);
                }
                tmem_st16(st + 16 * c, o);  // over S, which is in registers
                if (c & 1) {
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&m.pfull[x][c >> 1]);
                }
            }
            const float2 la = unpack2(add2(l2[0], l2[1]));
            l += la.x + la.y;
        }
        if (live) {
            if (p.lse)
                p.lse[(size_t)(rq.row0 + t) * p.heads + h] = n[x] ? (mr + log2f(l) - kFaShift) * 0.6931471805599453f : -INFINITY;
        }
        if (n[x]) ctl_wait(&m.odone[x], 0, ctl);
        tc_fence_after();
        const float inv = l == 0.f ? 0.f : 1.f / l;
        typename Elem<DT>::T *out = reinterpret_cast<typename Elem<DT>::T *>(p.out) +
                                    (int64_t)(rq.row0 + (live ? t : r0)) * p.out_stride + (size_t)h * 128;
#pragma unroll 1
        for (int c = 0; c < 128; c += 16) {
            uint32_t o[16];
            if (n[x]) {
                tmem_ld16(ot + c, o);
            } else {
#pragma unroll
                for (int k = 0; k < 16; ++k) o[k] = 0u;
            }
            uint32_t w[8];
#pragma unroll
            for (int k = 0; k < 8; ++k)
                w[k] = Elem<DT>::down2(__uint_as_float(o[2 * k]) * inv, __uint_as_float(o[2 * k + 1]) * inv);
            if (live) {
                uint4 *d = reinterpret_cast<uint4 *>(out + c);
                d[0] = make_uint4(w[0], w[1], w[2], w[3]);
                d[1] = make_uint4(w[4], w[5], w[6], w[7]);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (m.abort) {
        if (warp == 0) ctl_settle(kSettleNs);
        if (warp == 1 || warp == 2) {
            if (elect_one()) umma_commit(&m.fin[warp - 1]);
            ctl_drain(&m.fin[warp - 1], 0, kSettleNs);
        }
        __syncthreads();
    }
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// -------------------------------------------------------------------- host --
bool prompt_maps(const LatentParams &p, int dt, PromptMaps *m) {
    memset(m, 0, sizeof(*m));
    const uint64_t tok = (uint64_t)p.token_stride * 2;
    const uint64_t cd[4] = {64, (uint64_t)p.page_size, (uint64_t)(p.R + p.P) / 64, (uint64_t)p.num_pages};
    const uint64_t cs[3] = {tok, 128, p.num_pages > 1 ? (uint64_t)p.page_stride * 2 : tok * p.page_size};
    const uint32_t cb[4] = {64, (uint32_t)p.box_tokens, 1, 1};
    const uint64_t wd[3] = {64, (uint64_t)p.heads * 128, (uint64_t)p.R / 64}, wst[2] = {(uint64_t)p.R * 2, 128};
    const uint32_t wb[3] = {64, 128, 1};
    const uint64_t qd[4] = {64, (uint64_t)p.N, 3, (uint64_t)p.heads}, qst[3] = {(uint64_t)p.q_stride * 2, 128, 192 * 2};
    const uint32_t qb[4] = {64, 128, 3, 1};
    return map_rows64(&m->cache, dt, p.cache, 4, cd, cs, cb) && map_rows64(&m->w_uk, dt, p.w_uk, 3, wd, wst, wb) &&
           map_rows64(&m->w_uv, dt, p.w_uv, 3, wd, wst, wb) && map_rows64(&m->q, dt, p.q, 4, qd, qst, qb);
}

template <int DT>
int launch_expanded_dt(const LatentParams &p, int dt, cudaStream_t s) {
    PromptMaps maps;
    if (!prompt_maps(p, dt, &maps)) return SPX_ERR_UNSUPPORTED;
    int st = set_smem<latent_expand_kernel<DT>>(kExSmem);
    if (!st) st = set_smem<latent_prompt_kernel<DT>>(kFaSmem);
    if (st) return st;
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t c = latent_config(
        dim3((p.kv_rows / kPTile + 1) / 2 * 2, (p.heads + p.head_group - 1) / p.head_group, p.B), kExThreads, kExSmem, s,
        attr, 2);
    if ((st = record_launch(cudaLaunchKernelEx(&c, latent_expand_kernel<DT>, p, maps)))) return st;
    const int pairs = (p.max_q + 2 * kPTile - 1) / (2 * kPTile);
    c = latent_config(dim3(pairs * p.heads, p.B), kFaThreads, kFaSmem, s, attr, 1);
    return record_launch(cudaLaunchKernelEx(&c, latent_prompt_kernel<DT>, p, maps));
}

}  // namespace

int launch_expanded(LatentParams &p, int dt, cudaStream_t s) {
    // Heads per block of the expand launch: whole rounds over the SMs, a block's own cost taken as that of a head
    // (its latent vectors are two heads' bytes of weights, fetched beside the first head's).
    const long long tiles = (long long)p.B * ((p.kv_rows / kPTile + 1) / 2 * 2), sms = device_sm_count();
    if (sms < 1) return SPX_ERR_CUDA;
    long long best = 0;
    for (int g = 1; g <= 8 && g <= p.heads; ++g) {
        const long long blocks = tiles * ((p.heads + g - 1) / g), cost = (blocks + sms - 1) / sms * (g + 1);
        if (!best || cost < best) {
            best = cost;
            p.head_group = g;
        }
    }
    return dt == SPX_F16 ? launch_expanded_dt<SPX_F16>(p, dt, s) : launch_expanded_dt<SPX_BF16>(p, dt, s);
}

}  // namespace spx
