// spx_latent.cu -- attention over the paged latent cache, absorbed form.
//
// With k[h] = (W_uk[h] c, r) and v[h] = W_uv[h] c the products with the
// up-projections move out of the sum over the cache:
//   q_nope . (W_uk c) = (q_nope W_uk) . c,   sum_p w_p W_uv c_p = W_uv sum_p w_p c_p,
// so the cached (c, r) is read once for all heads.  Launches:
//
//   query launch      q_lat = (q_nope W_uk, q_rope), rounded to the type;
//   attention launch  softmax(scale q_lat . (c, r)) c in latent space, the
//                     cache cut into equal shares over the SMs, partial sums
//                     (with their maximum and weight) where a cut falls;
//   result launch     partial sums joined, times W_uv (or, with folded
//                     weights, a launch that only joins).
//
// Every launch is a programmatic dependent of the one before it.  What bounds a
// call: one request's draft step is a chain of three launches (517 cached tokens
// 15 us, 65536 28 us); many requests' is the cache (64 of up to 8192 tokens, 370
// MB: 83 us, of which the attention launch 68 at 5.4 TB/s); with 64 rows a unit
// half of the attention launch is the ring of tiles (see there).
#include <math.h>
#include <string.h>

#include "spx_latent.cuh"
#include "spx_tcgen05.cuh"

namespace spx {

namespace {

// --------------------------------------------------- small tensor products --
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], const void *p) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(smem_u32(p)));
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], const void *p) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(smem_u32(p)));
}
template <int DT>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
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

// ------------------------------------------------------------ query launch --
// Block (s, h, g): 16 * MT tokens' queries of head h times columns 64 s .. + 63
// of W_uk[h]; block s = 0 also copies the rotated part.  A block reads its
// slice of the weights once for all its tokens; the whole of W_uk is 2 MB for
// 16 heads, so the launch is bound by latency up to some hundred tokens (64
// tokens: 8.6 us alone, from DRAM; in a call the attention launch's set-up runs
// beside it).  q_lat is rounded to the type, as the tensor cores take it.
template <int DT, int MT>
__global__ void __launch_bounds__(128) latent_q_kernel(const __grid_constant__ LatentParams p) {
    extern __shared__ __align__(128) uint8_t lq_smem[];
    const int ldq = p.dn + 8;
    uint16_t *qs = reinterpret_cast<uint16_t *>(lq_smem);  // [16 MT][dn + 8]
    uint16_t *ws = qs + 16 * MT * ldq;                     // [dn][72]
    const int s = blockIdx.x, h = blockIdx.y, n0 = blockIdx.z * 16 * MT;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rows = min(16 * MT, p.N - n0);
    griddep_wait();
    griddep_launch_dependents();
    const uint16_t *wsrc = p.w_uk + (size_t)h * p.dn * p.R + 64 * s;
    for (int i = threadIdx.x; i < p.dn * 8; i += 128)
        cp_async16(ws + (i >> 3) * 72 + 8 * (i & 7), wsrc + (size_t)(i >> 3) * p.R + 8 * (i & 7));
    const int qv = p.dn / 8;
    for (int i = threadIdx.x; i < 16 * MT * qv; i += 128) {
        const int r = i / qv, c = i - r * qv;
        if (r < rows)
            cp_async16(qs + r * ldq + 8 * c, p.q + (n0 + r) * p.q_stride + (size_t)h * (p.dn + p.P) + 8 * c);
        else
            *reinterpret_cast<uint4 *>(qs + r * ldq + 8 * c) = make_uint4(0, 0, 0, 0);
    }
    cp_async_wait_all();
    __syncthreads();
    float acc[MT][2][4] = {};
    for (int k = 0; k < p.dn; k += 16) {
        uint32_t b[4];
        ldsm4t(b, ws + (k + (lane & 15)) * 72 + 16 * warp + 8 * (lane >> 4));
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            uint32_t a[4];
            ldsm4(a, qs + (16 * m + (lane & 15)) * ldq + k + 8 * (lane >> 4));
            mma16816<DT>(acc[m][0], a, b[0], b[1]);
            mma16816<DT>(acc[m][1], a, b[2], b[3]);
        }
    }
    const int D = p.R + p.P;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int r = 16 * m + (lane >> 2) + 8 * (j & 1);
            // o + 0 o: one that the type cannot hold becomes a NaN, as an infinity's scores could be -inf, which only
            // leave their tokens out
            const uint32_t o = Elem<DT>::down2(acc[m][j >> 1][2 * (j & 1)], acc[m][j >> 1][2 * (j & 1) + 1]);
            if (r < rows)
                *reinterpret_cast<uint32_t *>(p.q_lat + ((size_t)(n0 + r) * p.heads + h) * D + 64 * s + 16 * warp +
                                              8 * (j >> 1) + 2 * (lane & 3)) = Elem<DT>::fma2(o, 0u, o);
        }
    if (s == 0)
        for (int i = threadIdx.x; i < rows * (p.P / 8); i += 128) {
            const int r = i / (p.P / 8), c = i - r * (p.P / 8);
            *reinterpret_cast<uint4 *>(p.q_lat + ((size_t)(n0 + r) * p.heads + h) * D + p.R + 8 * c) =
                *reinterpret_cast<const uint4 *>(p.q + (n0 + r) * p.q_stride + (size_t)h * (p.dn + p.P) + p.dn + 8 * c);
        }
}

// Folded queries whose tokens are not contiguous, packed for the attention launch.
__global__ void __launch_bounds__(128) latent_pack_kernel(const __grid_constant__ LatentParams p) {
    griddep_wait();
    griddep_launch_dependents();
    const int per = p.heads * (p.R + p.P) / 8;
    const uint4 *src = reinterpret_cast<const uint4 *>(p.q + blockIdx.x * p.q_stride);
    uint4 *dst = reinterpret_cast<uint4 *>(p.q_lat) + (size_t)blockIdx.x * per;
    for (int i = threadIdx.x; i < per; i += 128) dst[i] = src[i];
}

// -------------------------------------------------------- attention launch --
// A unit is a request's rows NR g .. NR g + NR - 1 in (token, head) order; its
// cache, in tiles of 64 tokens, is one stretch of the call's tiles, which are
// dealt out in equal contiguous shares, one per block.
//
// The products are transposed, so that few rows leave no tensor-core lane
// idle and one copy of a tile in shared memory serves both:
//   S^T [64 tokens x rows] = C [64 x (R + P)] . Q^T        (A = the tile, k-major)
//   O^T [R x rows]        += V^T [R x 64 tokens] . P^T     (A = the tile, m-major)
// with Q and P as the B operands (N = rows) and O^T in tensor memory (R / 128
// accumulators of 128 lanes).  S^T has M = 64 (16 lanes of each quarter).
//
// The products of a tile read shared memory at its rate: 36 of 64 x 64 x 16 (32
// cycles each) and 16 of 128 x 64 x 16 (48), 1920 cycles on 64 rows, 1200 on
// 16.  Units of 16 rows wait for DRAM all the same.  Units of 64 rows leave room
// for two tiles, whose slots are taken from the copy's start to the last
// product: 2840 cycles a tile.  That is half of the launch (16 requests of 9 x 16
// rows over up to 8191 tokens: 16 tiles a share, 22 of 41 us; 32 of 2 x 64 rows
// over up to 4096: 23 of 47).  The other half is the wait for the query launch
// (7 us in the first, none in the second) and, not told apart by measurement,
// the units that begin inside a share, whose queries and first O wait for the
// unit before, and the partial sums.
//
// Softmax runs in base 2 with one reference per row; the sums are rescaled
// only when a maximum rises by more than 2^kSlack over it, which fp32 sums and
// fp16 weights of at most 2^(kSlack + kShift) bear.  kShift moves the weights
// away from the subnormals of fp16.
constexpr int kTile = 64;
constexpr float kSlack = 8.f, kShift = 5.f;
constexpr int kPairBytes = kTile * 256;  // 64 tokens x 128 latent values, as two 64-value halves
constexpr int kMaxBlocks = 160;  // blocks of the attention launch: one per SM, at most this many
constexpr int kRopeBytes = kTile * 128;
// Copies are issued by one warp per pair of a tile: a warp takes 250 to 300
// cycles for each, and one warp's nine of a tile were slower than the products.
// One more takes the queries, which wait for the launch that writes them.
constexpr int kCopyWarps = 4, kQueryWarp = kCopyWarps, kIssueWarp = kCopyWarps + 1;

// Ring depths by rows per unit: 2.25, 2.5 and 2 tiles.  Shared memory would allow
// 2.75 for 16 rows, but then no block starts beside one of the query launch.
// A tile's rotated part is not needed once its S^T is there, so its slot then
// takes the tile's softmax weights, P^T [64 tokens x 64 rows].
template <int NR>
struct AttnGeo {
    static constexpr int kPairs = NR <= 16 ? 9 : NR <= 32 ? 10 : 8;
    static constexpr int kRopes = 3;
    // Softmax warps: four (one per quarter of tensor memory) for each share of
    // the rows: one warp a scheduler cannot keep up with the products on 64 rows.
    static constexpr int kShares = NR <= 16 ? 1 : 2;
    static constexpr int kThreads = 32 * (kIssueWarp + 1) + 128 * kShares;
    static constexpr int kQBytes = 9 * NR * 128;
    static constexpr int kMisc = 3072;
    static constexpr int kSmem = kQBytes + kPairs * kPairBytes + kRopes * kRopeBytes + kMisc;
    static constexpr uint32_t kTmem = NR <= 16 ? 128 : NR <= 32 ? 256 : 512;  // >= 6 NR, a power of two
    static_assert(kSmem <= kSmemLimit, "shared memory of one block");
    static_assert(kPairs <= 12 && kRopes <= 4, "a landing barrier and a release for each slot");
};

struct AttnMisc {
    uint64_t pfull[12], rfull[4];    // copies have landed, by slots: pairs, rotated parts
    uint64_t pempty[12], rempty[4];  // slots free: pairs, rotated parts
    uint64_t qfull, qempty;       // the unit's queries landed / read for the last time
    uint64_t sfull[2];            // S^T of a tile is in tensor memory
    uint64_t wfull[2];            // a tile's weights are in shared memory (all softmax warps)
    uint64_t odone;               // O^T has taken a tile
    uint64_t udone;               // O^T has taken the last tile of a unit
    uint64_t ofree;               // O^T of the unit has been read out (all softmax warps)
    uint64_t fin;                 // products drained (abort path)
    uint32_t tmem;
    int abort;
    int b, g, off, flat, left, share;  // tiles of a share, and where this block's begins
    LatentReq rq;                      // the request b
    int odd;                           // the unit: a latent value that only some rows see is not finite
    int lim[64];                  // positions that each row sees
    float fac[64];
    float red[2][4][64];
};
static_assert(sizeof(AttnMisc) <= 3072, "the misc area holds it");

// A place in a ring of N slots and the parity of its use.
template <int N>
struct Slot {
    uint32_t i = 0, phase = 0;
    __device__ __forceinline__ void next() {
        if (++i == N) {
            i = 0;
            phase ^= 1;
        }
    }
    __device__ __forceinline__ void advance(int n) {  // n <= N
        i += n;
        if (i >= N) {
            i -= N;
            phase ^= 1;
        }
    }
};

// Tensor maps in pieces of 64 values (one swizzled row of 128 bytes).
struct AttnMaps {
    CUtensorMap pair;  // cache as [page][piece][token][64]: boxes of 2 pieces x 64 tokens, or 1 x gcd(page_size, 64)
    CUtensorMap rope;  // the same, boxes of 1 piece
    CUtensorMap q;     // queries as [piece][row][64], a box is all of a unit's
};

template <int NR>
__device__ __forceinline__ int unit_tiles(const LatentParams &p, const LatentReq &r, int g) {
    const int rows = r.T * p.heads;
    if (g * NR >= rows) return 0;
    const int last = p.by_heads(min((g + 1) * NR, rows) - 1);
    return (latent_limit(p, r, last) + kTile - 1) / kTile;
}

// A block's walk over its share, unit by unit; the same in every role.
template <int NR>
struct Walk {
    int b, g, nt;        // unit, its tiles
    int tile, end;       // tiles of the unit in this share
    int flat, left;      // index of `tile` among the call's tiles; tiles left from `tile` on
    bool first;          // the share begins inside or with this unit
    LatentReq rq;
    __device__ __forceinline__ void begin(const LatentParams &p, const AttnMisc &m) {
        b = m.b;
        g = m.g;
        flat = m.flat;
        left = m.left;
        first = true;
        if (left <= 0) return;
        rq = m.rq;
        nt = unit_tiles<NR>(p, rq, g);
        tile = m.off;
        end = min(nt, tile + left);
    }
    __device__ __forceinline__ void next(const LatentParams &p) {
        left -= end - tile;
        flat += end - tile;
        first = false;
        if (left <= 0) return;
        ++g;
        while (true) {
            nt = unit_tiles<NR>(p, rq, g);
            if (nt > 0) break;
            if ((g + 1) * NR < rq.T * p.heads) {
                ++g;
                continue;
            }
            if (++b >= p.B) {  // does not happen while tiles are left
                left = 0;
                return;
            }
            rq = latent_req(p, b);
            g = 0;
        }
        tile = 0;
        end = min(nt, left);
    }
};

// One warp: all tiles of the call, this block's share, and where it begins.
template <int NR>
__device__ __forceinline__ void find_share(const LatentParams &p, AttnMisc &m, int lane) {
    if (p.B == 1) {  // (the same without the scans, which a single short call would wait for)
        const LatentReq r = latent_req(p, 0);
        int total = 0;
        for (int g = 0; g * NR < r.T * p.heads; ++g) total += unit_tiles<NR>(p, r, g);
        const int share = max((total + (int)gridDim.x - 1) / (int)gridDim.x, 1), from = share * (int)blockIdx.x;
        int off = from, g = 0;
        if (from < total)
            for (int u; off >= (u = unit_tiles<NR>(p, r, g)); ++g) off -= u;
        if (lane == 0) {
            m.left = min(share, total - from);
            m.flat = from;
            m.share = share;
            m.b = 0;
            m.g = g;
            m.off = off;
            m.rq = r;
        }
        return;
    }
    LatentReq r{0, 0, 0};
    int n = 0, total = 0, share = 0, from = 0;
    bool found = false;
#pragma unroll 1
    for (int pass = 0; pass < 2 && !found; ++pass) {
        int before = 0;
#pragma unroll 1
        for (int b0 = 0; b0 < p.B && !found; b0 += 32) {
            if (pass == 0 || p.B > 32) {
                n = 0;
                if (b0 + lane < p.B) {
                    r = latent_req(p, b0 + lane);
                    for (int g = 0; g * NR < r.T * p.heads; ++g) n += unit_tiles<NR>(p, r, g);
                }
            }
            int incl = n;
#pragma unroll 1
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += v;
            }
            if (pass) {
                int off = from - (before + incl - n);
                const bool mine = off >= 0 && off < n;
                if (mine) {
                    int g = 0;
                    for (int u; off >= (u = unit_tiles<NR>(p, r, g)); ++g) off -= u;
                    m.b = b0 + lane;
                    m.g = g;
                    m.off = off;
                    m.rq = r;
                }
                found = __any_sync(0xffffffffu, mine);
            }
            before += __shfl_sync(0xffffffffu, incl, 31);
        }
        if (pass) break;
        total = before;
        share = max((total + (int)gridDim.x - 1) / (int)gridDim.x, 1);
        from = share * (int)blockIdx.x;
        if (lane == 0) {
            m.left = min(share, total - from);
            m.flat = from;
            m.share = share;
        }
        found = from >= total;
    }
}

template <int DT, int NR>
__global__ void __launch_bounds__(AttnGeo<NR>::kThreads, 1)
    latent_attn_kernel(const __grid_constant__ LatentParams p, const __grid_constant__ AttnMaps maps) {
    using G = AttnGeo<NR>;
    constexpr int PR = G::kPairs, RR = G::kRopes;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t *qs = smem, *pairs = qs + G::kQBytes, *ropes = pairs + PR * kPairBytes;
    AttnMisc &m = *reinterpret_cast<AttnMisc *>(ropes + RR * kRopeBytes);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int np = p.R / 128;  // pairs of a tile

    if (!p.chained) griddep_wait();
    if (warp == 0) {
        find_share<NR>(p, m, lane);
    } else if (warp == kIssueWarp) {
        tmem_alloc(&m.tmem, G::kTmem);
        tmem_relinquish();
    } else if (warp == kQueryWarp) {
        // the words from pfull to fin are all barriers
        uint64_t *bars = m.pfull;
        constexpr int kBars = 12 + 4 + 12 + 4 + 2 + 2 + 2 + 4;
        for (int i = lane; i < kBars; i += 32)
            mbar_init(&bars[i], &bars[i] == m.wfull || &bars[i] == m.wfull + 1 || &bars[i] == &m.ofree ? 4 * G::kShares : 1);
        if (lane == 0) m.abort = 0;
        fence_mbar_init();
        if (lane == 0) {
            prefetch_tmap(&maps.pair);
            prefetch_tmap(&maps.rope);
            prefetch_tmap(&maps.q);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    griddep_launch_dependents();
    const uint32_t tmem = m.tmem;
    const uint32_t s_col = (uint32_t)(np * NR);  // S^T buffers after the R / 128 parts of O^T
    const WaitCtl ctl{&m.abort, &p.hdr->status, p.budget, SITE_LATENT};
    Walk<NR> w;

    if (warp < kCopyWarps) {
        // ---- copies: warp c takes pair c of every tile, warp 0 the rotated part too
        const uint64_t pol = p.groups > 1 ? policy_evict_normal() : policy_evict_first();
        const int bt = p.box_tokens, nb = kTile / bt;  // boxes do not cross a page
        Slot<PR> ps;
        Slot<RR> rs;
        ps.i = warp;
        bool ok = true;
        for (w.begin(p, m); ok && warp < np && w.left > 0; w.next(p)) {
            const int32_t *tab = p.table + (size_t)w.b * p.max_pages;
            int box = 32, my_page = 0, my_at = 0;  // this lane's box of the 32 looked up together
#pragma unroll 1
            for (int i = w.tile; i < w.end; ++i, box += nb) {
                if (box >= 32) {
                    const int pos = kTile * i + bt * lane, pi = p.by_page(pos);
                    my_at = pos - pi * p.page_size;
                    // positions past the length come as zeros (a page out of range)
                    my_page = pos < w.rq.len ? __ldg(tab + pi) : p.num_pages;
                    if (my_page < 0 || my_page >= p.num_pages) my_page = p.num_pages;
                    box = 0;
                }
                uint64_t *full = &m.pfull[ps.i], *rfull = &m.rfull[rs.i];
                if (!(ok = (warp || ctl_wait(&m.rempty[rs.i], rs.phase ^ 1, ctl)) &&
                           ctl_wait(&m.pempty[ps.i], ps.phase ^ 1, ctl)))
                    break;
                uint8_t *dst = pairs + ps.i * kPairBytes, *rope = ropes + rs.i * kRopeBytes;
                const bool lead = elect_one();
                if (lead) {
                    mbar_arrive_expect_tx(full, kPairBytes);
                    if (warp == 0) mbar_arrive_expect_tx(rfull, kRopeBytes);
                }
#pragma unroll 1
                for (int j = 0; j < nb; ++j) {
                    const int at = __shfl_sync(0xffffffffu, my_at, box + j);
                    const int page = __shfl_sync(0xffffffffu, my_page, box + j);
                    if (lead) {
                        tma_load_4d(dst + j * bt * 128, &maps.pair, 0, at, 2 * warp, page, full, pol);
                        if (nb > 1)
                            tma_load_4d(dst + kPairBytes / 2 + j * bt * 128, &maps.pair, 0, at, 2 * warp + 1, page, full,
                                        pol);
                        if (warp == 0) tma_load_4d(rope + j * bt * 128, &maps.rope, 0, at, 2 * np, page, rfull, pol);
                    }
                }
                __syncwarp();
                ps.advance(np);
                rs.next();
            }
        }
    } else if (warp == kQueryWarp) {
        // ---- the units' queries, each once the last unit's have been read
        const uint64_t pol = policy_evict_normal();
        uint32_t seg = 0;
        bool ok = true;
        if (p.chained) griddep_wait();
        for (w.begin(p, m); ok && w.left > 0; w.next(p), ++seg) {
            if (!(ok = ctl_wait(&m.qempty, (seg & 1) ^ 1, ctl))) break;
            if (elect_one()) {
                mbar_arrive_expect_tx(&m.qfull, (uint32_t)(2 * np + 1) * NR * 128);
                tma_load_3d(qs, &maps.q, 0, w.rq.row0 * p.heads + NR * w.g, 0, &m.qfull, pol);
            }
            __syncwarp();
        }
    } else if (warp == kIssueWarp) {
        // ---- products: whichever is ready, the oldest tile's O first; S at most two tiles ahead of O
        const uint32_t fmt = DT == SPX_BF16 ? kIdescBf16 : 0u;
        const uint64_t qd = sw128_desc(smem_u32(qs)), kd = sw128_desc(smem_u32(pairs)), rd = sw128_desc(smem_u32(ropes));
        const uint64_t vd = sw128_desc_mn(smem_u32(pairs), kPairBytes / 2), pd = sw128_desc_mn(smem_u32(ropes), 0);
        uint32_t ts = 0, to = 0, seg = 0;  // next tile for S and for O
        Slot<PR> sp, op;                   // their first pairs
        Slot<RR> sr, orp;                  // and rotated parts / weights
        bool ok = true;
        for (w.begin(p, m); ok && w.left > 0; w.next(p), ++seg) {
            const int n16 = (min(NR, w.rq.T * p.heads - NR * w.g) + 15) & ~15;
            const uint32_t idS = idesc_f16_f32(64, n16) | fmt;
            const uint32_t idO = idesc_f16_f32(128, n16) | fmt | kIdescAMn | kIdescBMn;
            const uint32_t t0 = ts, t1 = ts + (uint32_t)(w.end - w.tile);
            if (!(ok = ctl_wait(&m.qfull, seg & 1, ctl))) break;
            uint64_t since = 0;
#pragma unroll 1
            while (to < t1) {
                const bool room = ts < t1 && ts - to < 2;
                if (to < ts && mbar_test(&m.wfull[to & 1], (to >> 1) & 1) && (to != t0 || mbar_test(&m.ofree, (seg & 1) ^ 1))) {
                    tc_fence_after();
                    if (elect_one()) {
                        Slot<PR> k = op;
#pragma unroll 1
                        for (int c = 0; c < np; ++c) {
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                umma_f16(tmem + c * NR, vd + k.i * (kPairBytes / 16) + 128 * j,
                                         pd + orp.i * (kRopeBytes / 16) + 128 * j, idO, to != t0 || j != 0);
                            umma_commit(&m.pempty[k.i]);
                            k.next();
                        }
                        umma_commit(&m.rempty[orp.i]);
                        umma_commit(&m.odone);
                        if (to + 1 == t1) umma_commit(&m.udone);
                    }
                    __syncwarp();
                    op.advance(np);
                    orp.next();
                    ++to;
                    since = 0;
                } else if (room && mbar_test(&m.pfull[sp.i], sp.phase)) {
                    // begun with the first pair: the others follow within its products, mostly
                    bool landed = true;
                    tc_fence_after();
                    const uint32_t sd = tmem + s_col + (ts & 1) * NR;
                    if (elect_one()) {
                        // descriptors count in 16 bytes: 32 bytes a k-step, half a pair, a chunk of Q
                        Slot<PR> k = sp;
                        uint64_t q = qd;
#pragma unroll 1
                        for (int c = 0; c < np; ++c) {
                            if (c && !mbar_test(&m.pfull[k.i], k.phase) && !(landed = ctl_wait(&m.pfull[k.i], k.phase, ctl)))
                                break;
                            const uint64_t a = kd + k.i * (kPairBytes / 16);
#pragma unroll
                            for (int j = 0; j < 8; ++j)
                                umma_f16(sd, a + (j >> 2) * (kPairBytes / 32) + 2 * (j & 3),
                                         q + (j >> 2) * (NR * 8) + 2 * (j & 3), idS, (c | j) != 0);
                            q += 2 * NR * 8;
                            k.next();
                        }
                        if (landed) landed = mbar_test(&m.rfull[sr.i], sr.phase) || ctl_wait(&m.rfull[sr.i], sr.phase, ctl);
                        if (landed) {
                            const uint64_t a = rd + sr.i * (kRopeBytes / 16);
#pragma unroll
                            for (int j = 0; j < 4; ++j) umma_f16(sd, a + 2 * j, q + 2 * j, idS, 1);
                            umma_commit(&m.sfull[ts & 1]);
                            if (ts + 1 == t1) umma_commit(&m.qempty);
                        }
                    }
                    if (!(ok = __all_sync(0xffffffffu, landed))) break;
                    sp.advance(np);
                    sr.next();
                    ++ts;
                    since = 0;
                } else if (*ctl.abort) {
                    ok = false;
                    break;
                } else if (!since) {
                    since = global_timer_ns();
                } else if (global_timer_ns() - since > ctl.budget) {
                    record_timeout(ctl.status, ctl.site);
                    *ctl.abort = 1;
                    ok = false;
                    break;
                }
            }
        }
    } else {
        // ---- softmax, rescaling, results
        constexpr int SH = G::kShares, NC = NR / SH, NB = NC / 8;  // rows of a share, in blocks of 8
        const int q = warp & 3;                                    // tensor-memory quarter
        const int sh = (warp - kIssueWarp - 1) >> 2, c0 = NC * sh;              // this warp's share of the rows: c0 ..
        const int tid = 32 * q + lane, all = 128 * sh + tid;       // index within the share's warps, among all
        const uint32_t quarter = tmem + ((uint32_t)(32 * q) << 16);
        const int cl = c0 + 2 * (lane & 3);    // this lane's rows: 8x + cl, 8x + cl + 1
        const int tok = 16 * q + (lane >> 2);  // its tokens: tok, tok + 8
        uint32_t tc = 0, seg = 0;  // tiles so far, parity of the units
        Slot<RR> rs;
        Slot<PR> ps;
        // (after a wait that gave up the loop runs on, as every warp has to meet the barriers)
        for (w.begin(p, m); w.left > 0; w.next(p), seg ^= 1) {
            const int rows = min(NR, w.rq.T * p.heads - NR * w.g), n16 = (rows + 15) & ~15;
            const int row0 = NR * w.g;
            bar_sync(7, 128 * SH);  // the last unit's limits and sums are read
            if (all == 0) m.odd = 0;
            if (all < NR) m.lim[all] = all < rows ? latent_limit(p, w.rq, p.by_heads(row0 + all)) : 0;
            bar_sync(7, 128 * SH);
            const int lim_lo = m.lim[0], lim_hi = m.lim[rows - 1];
            // References less kShift, and sums of weights, of this lane's rows (in pairs).  A row that has seen
            // nothing has a reference below every score.
            constexpr float kNone = -3e38f;
            float ref[2 * NB];
            uint64_t l2[NB];
#pragma unroll
            for (int c = 0; c < 2 * NB; ++c) ref[c] = kNone;
#pragma unroll
            for (int x = 0; x < NB; ++x) l2[x] = 0;
#pragma unroll 1
            for (int i = w.tile; i < w.end; ++i, ++tc, rs.next(), ps.advance(np)) {
                ctl_wait(&m.sfull[tc & 1], (tc >> 1) & 1, ctl);
                tc_fence_after();
                uint32_t r[4 * NB];
#pragma unroll
                for (int x = 0; x < NB; x += 2)
                    tmem_ld_16x256b_x2(quarter + s_col + (tc & 1) * NR + c0 + 8 * x, r + 4 * x);
                tmem_wait_ld();
                const int p0 = kTile * i;
                const bool masked = p0 + kTile > lim_lo;
                // exponents of the weights by the present references
                uint64_t w2[2 * NB];
                const uint64_t scale2 = pack2(p.scale_log2, p.scale_log2);
                auto exponents = [&]() {
#pragma unroll
                    for (int x = 0; x < NB; ++x) {
                        const uint64_t minus = pack2(-ref[2 * x], -ref[2 * x + 1]);
#pragma unroll
                        for (int k = 0; k < 2; ++k)
                            w2[2 * x + k] = fma2(pack2(__uint_as_float(r[4 * x + 2 * k]), __uint_as_float(r[4 * x + 2 * k + 1])),
                                                 scale2, minus);
                        if (masked || c0 + NC > n16) {
                            const int2 lim = *reinterpret_cast<const int2 *>(&m.lim[8 * x + cl]);
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                float2 v = unpack2(w2[2 * x + k]);
                                if (p0 + tok + 8 * k >= lim.x) v.x = -INFINITY;
                                if (p0 + tok + 8 * k >= lim.y) v.y = -INFINITY;
                                w2[2 * x + k] = pack2(v.x, v.y);
                            }
                        }
                    }
                };
                exponents();
                float most = -INFINITY;
#pragma unroll
                for (int x = 0; x < 2 * NB; ++x) {
                    const float2 v = unpack2(w2[x]);
                    most = fmaxf(most, fmaxf(v.x, v.y));
                }
                // A barrier that carries one bit: the products keep shared memory busy, and an exchange of the
                // maxima through it took longer than all the rest.  Only a rise beyond the slack needs one.
                if (bar_any(1 + sh, 128, most > kSlack + kShift)) {
                    float(*red)[64] = m.red[tc & 1];
                    float mx[2 * NB];
#pragma unroll
                    for (int x = 0; x < NB; ++x) {
                        const float2 u = unpack2(w2[2 * x]), v = unpack2(w2[2 * x + 1]);
                        // the larger of the two scores that the row sees
                        const float a0 = u.x == -INFINITY ? -INFINITY : __uint_as_float(r[4 * x]) * p.scale_log2;
                        const float a1 = u.y == -INFINITY ? -INFINITY : __uint_as_float(r[4 * x + 1]) * p.scale_log2;
                        const float b0 = v.x == -INFINITY ? -INFINITY : __uint_as_float(r[4 * x + 2]) * p.scale_log2;
                        const float b1 = v.y == -INFINITY ? -INFINITY : __uint_as_float(r[4 * x + 3]) * p.scale_log2;
                        mx[2 * x] = fmaxf(a0, b0);
                        mx[2 * x + 1] = fmaxf(a1, b1);
                    }
#pragma unroll
                    for (int o = 4; o < 32; o <<= 1)
#pragma unroll
                        for (int c = 0; c < 2 * NB; ++c) mx[c] = fmaxf(mx[c], __shfl_xor_sync(0xffffffffu, mx[c], o));
                    if (lane < 4)
#pragma unroll
                        for (int x = 0; x < NB; ++x)
                            *reinterpret_cast<float2 *>(&red[q][8 * x + cl]) = make_float2(mx[2 * x], mx[2 * x + 1]);
                    bar_sync(1 + sh, 128);
#pragma unroll
                    for (int x = 0; x < NB; ++x) {
                        float f[2];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const float2 v = *reinterpret_cast<const float2 *>(&red[k][8 * x + cl]);
                            mx[2 * x] = fmaxf(mx[2 * x], v.x);
                            mx[2 * x + 1] = fmaxf(mx[2 * x + 1], v.y);
                        }
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const float now = mx[2 * x + k] - kShift;
                            f[k] = 1.f;
                            if (now > ref[2 * x + k] + kSlack) {
                                f[k] = ex2(ref[2 * x + k] - now);
                                ref[2 * x + k] = now;
                            }
                        }
                        l2[x] = mul2(l2[x], pack2(f[0], f[1]));
                        if (q == 0 && lane < 4) *reinterpret_cast<float2 *>(&m.fac[8 * x + cl]) = make_float2(f[0], f[1]);
                    }
                    if (i > w.tile) {
                        bar_sync(1 + sh, 128);
                        // (O of tile tc - 2 is done, as S of this tile was issued behind it, and O of this one waits
                        // for this warp's weights: the barrier is in the phase of tc - 1 or just past it)
                        ctl_wait(&m.odone, (tc - 1) & 1, ctl);
                        tc_fence_after();
#pragma unroll 1
                        for (int c = 0; c < np; ++c)
#pragma unroll 1
                            for (int x = c0; x < min(c0 + NC, n16); x += 16) {
                                uint32_t o[16];
                                tmem_ld16(quarter + c * NR + x, o);
#pragma unroll
                                for (int k = 0; k < 16; ++k)
                                    o[k] = __float_as_uint(__uint_as_float(o[k]) * m.fac[x + k]);
                                tmem_st16(quarter + c * NR + x, o);
                            }
                        tmem_wait_st();
                        tc_fence_before();
                    }
                    exponents();
                }
#pragma unroll
                for (int x = 0; x < 2 * NB; ++x) {
                    const float2 v = unpack2(w2[x]);
                    w2[x] = pack2(ex2(v.x), ex2(v.y));
                    l2[x >> 1] = add2(l2[x >> 1], w2[x]);
                }
                uint8_t *wt = ropes + rs.i * kRopeBytes;
#pragma unroll
                for (int x = 0; x < NB; ++x)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const int t = tok + 8 * k;
                        const float2 v = unpack2(w2[2 * x + k]);
                        *reinterpret_cast<uint32_t *>(wt + t * 128 + 16 * ((x + c0 / 8) ^ (t & 7)) + 4 * (lane & 3)) =
                            Elem<DT>::down2(v.x, v.y);
                    }
                if (masked) {
                    // What some row may not see has weight 0 there, and 0 times an infinity or a NaN would
                    // still reach it: rows of the tile that nobody sees become 0, and in those that only
                    // some see every value that is not finite (those who see it get theirs with the results).
                    const int t0 = max(lim_lo - p0, 0);
                    Slot<PR> k0 = ps;
#pragma unroll 1
                    for (int c = 0; c < np; ++c, k0.next()) {
                        uint8_t *base = pairs + k0.i * kPairBytes;
#pragma unroll 1
                        for (int e = all; e < (kTile - t0) * 16; e += 128 * SH) {
                            const int t = t0 + (e >> 4), k = e & 15;
                            uint4 *at = reinterpret_cast<uint4 *>(base + (k >> 3) * (kPairBytes / 2) + t * 128 +
                                                                  16 * (k & 7));
                            uint4 v = make_uint4(0, 0, 0, 0);
                            if (p0 + t < lim_hi) {
                                v = *at;
                                // (0 times all eight, summed, is a NaN if one is not finite)
                                uint32_t test = Elem<DT>::fma2(v.x, 0u, Elem<DT>::fma2(v.y, 0u, 0u));
                                test = Elem<DT>::fma2(v.z, 0u, Elem<DT>::fma2(v.w, 0u, test));
                                if (test & 0x7FFF7FFFu) {
                                    v = make_uint4(Elem<DT>::finite2(v.x, 0u), Elem<DT>::finite2(v.y, 0u),
                                                   Elem<DT>::finite2(v.z, 0u), Elem<DT>::finite2(v.w, 0u));
                                    m.odd = 1;
                                }
                            }
                            *at = v;
                        }
                    }
                }
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&m.wfull[tc & 1]);
            }
            // ---- results of the unit, or of its part in this share
            // (odone may be one or two phases on by now; the next of udone waits for this unit's results)
            ctl_wait(&m.udone, seg, ctl);
            tc_fence_after();
            const bool whole = w.tile == 0 && w.end == w.nt;
            const int slot = 2 * (int)blockIdx.x + (w.first ? 0 : 1);
            if (all == 0 && w.tile == 0)
                p.units[(size_t)w.b * p.groups + w.g] =
                    make_int4((int)blockIdx.x, (w.flat + w.nt - 1) / m.share, slot, whole);
            float(*red)[64] = m.red[tc & 1];
            long long *at = reinterpret_cast<long long *>(m.red[(tc & 1) ^ 1]);
            float l[2 * NB];
#pragma unroll
            for (int x = 0; x < NB; ++x) {
                const float2 v = unpack2(l2[x]);
                l[2 * x] = v.x;
                l[2 * x + 1] = v.y;
            }
#pragma unroll
            for (int o = 4; o < 32; o <<= 1)
#pragma unroll
                for (int c = 0; c < 2 * NB; ++c) l[c] += __shfl_xor_sync(0xffffffffu, l[c], o);
            if (lane < 4)
#pragma unroll
                for (int c = 0; c < 2 * NB; ++c) {
                    const int col = 8 * (c >> 1) + cl + (c & 1);
                    red[q][col] = l[c];
                    if (q == 0) m.fac[col] = ref[c] == kNone ? -INFINITY : ref[c] + kShift;
                }
            bar_sync(7, 128 * SH);
            const bool direct = whole && !p.w_uv;
            const long long first_row = (long long)w.rq.row0 * p.heads + row0;
            if (all < rows) {
                const float L = red[0][all] + red[1][all] + red[2][all] + red[3][all], M = m.fac[all];
                const long long row = first_row + all;
                if (whole) {
                    m.fac[all] = M == -INFINITY && L == 0.f ? 0.f : 1.f / L;
                    if (p.lse) p.lse[row] = (M + log2f(L) - kShift) * 0.6931471805599453f;
                } else {
                    m.fac[all] = 1.f;
                    p.ml[(size_t)slot * NR + all] = make_float2(M, L);
                }
                if (direct) at[all] = row / p.heads * p.out_stride + row % p.heads * p.R;
            }
            bar_sync(7, 128 * SH);
            float *dst = whole ? p.o_lat + first_row * p.R : p.part + (size_t)slot * NR * p.R;
#pragma unroll 1
            for (int x = c0; x < min(c0 + NC, n16); x += 16) {
                float f[16];
#pragma unroll
                for (int k = 0; k < 16; ++k) f[k] = m.fac[x + k];
                const int left = rows - x;  // rows of these 16
#pragma unroll 1
                for (int c = 0; c < np; ++c) {
                    const int d = 128 * c + tid;
                    uint32_t o[16];
                    tmem_ld16(quarter + c * NR + x, o);
                    if (direct) {
#pragma unroll
                        for (int k = 0; k < 16; ++k)
                            if (k < left)
                                reinterpret_cast<typename Elem<DT>::T *>(p.out)[at[x + k] + d] =
                                    Elem<DT>::down(__uint_as_float(o[k]) * f[k]);
                    } else {
                        float *to = dst + (size_t)x * p.R + d;
#pragma unroll
                        for (int k = 0; k < 16; ++k, to += p.R)
                            if (k < left) __stcg(to, __uint_as_float(o[k]) * f[k]);
                    }
                }
            }
            // A latent value that is not finite makes a NaN of its column in the rows that see it, whatever their
            // weight; where all rows of a tile see it the products have done so.  (Behind this thread's own stores.)
            if (m.odd)
#pragma unroll 1
                for (int t = max(lim_lo, kTile * w.tile); t < min(lim_hi, kTile * w.end); ++t) {
                    const int pi = p.by_page(t), pg = __ldg(p.table + (size_t)w.b * p.max_pages + pi);
                    if (pg < 0 || pg >= p.num_pages) continue;
                    const uint16_t *src = p.cache + (int64_t)pg * p.page_stride + (int64_t)(t - pi * p.page_size) * p.token_stride;
#pragma unroll 1
                    for (int d = tid; d < p.R; d += 128) {
                        if (Elem<DT>::finite2(src[d], 0u) == src[d]) continue;
#pragma unroll 1
                        for (int x = c0; x < min(c0 + NC, rows); ++x) {
                            if (m.lim[x] <= t) continue;
                            if (direct)
                                p.out[at[x] + d] = 0x7FFFu;
                            else
                                __stcg(dst + (size_t)x * p.R + d, NAN);
                        }
                    }
                }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&m.ofree);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (m.abort) {
        if (warp == 0) ctl_settle(kSettleNs);
        if (warp == kIssueWarp) {
            if (elect_one()) umma_commit(&m.fin);
            ctl_drain(&m.fin, 0, kSettleNs);
        }
    }
    if (warp == kIssueWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, G::kTmem);
    }
}

// ----------------------------------------------------------- result launch --
// What became of a row of the call: its unit's shares, or nothing.  A warp
// looks up RW rows together and issues each kind of load for all of them, and
// for all shares, before it uses the first: the launch is a chain of four
// dependent reads (requests, units, weights, sums), which one after another
// for four rows and 150 shares cost over 10 us.
template <int RW>
struct RowSums {
    int first[RW], n[RW], slot[RW], col[RW];  // first block, shares, first slot, row within the unit
    bool whole[RW], owned[RW];
    float f[RW][kMaxBlocks / 32];             // factor of the share first + 32 q + lane
    float lse[RW];
    __device__ __forceinline__ int slot_of(int i, int k) const { return k == 0 ? slot[i] : 2 * (first[i] + k); }
};
constexpr int kShareChunks = kMaxBlocks / 32;

// Warp-wide: rows (n[i], head h); n[i] < 0 = none.
template <int RW>
__device__ __forceinline__ void find_rows(const LatentParams &p, const int (&n)[RW], int h, int lane, RowSums<RW> &r) {
    int unit[RW];
#pragma unroll
    for (int i = 0; i < RW; ++i) {
        unit[i] = -1;
        r.owned[i] = r.whole[i] = false;
        r.first[i] = r.n[i] = r.slot[i] = r.col[i] = 0;
    }
#pragma unroll 1
    for (int b0 = 0; b0 < p.B; b0 += 32) {
        LatentReq rq{0, 0, 0};
        if (b0 + lane < p.B) rq = latent_req(p, b0 + lane);
#pragma unroll
        for (int i = 0; i < RW; ++i) {
            const uint32_t hit = __ballot_sync(0xffffffffu, n[i] >= rq.row0 && n[i] < rq.row0 + rq.T);
            if (!hit || r.owned[i]) continue;
            const int src = __ffs(hit) - 1;
            const LatentReq o{__shfl_sync(0xffffffffu, rq.row0, src), __shfl_sync(0xffffffffu, rq.T, src),
                              __shfl_sync(0xffffffffu, rq.len, src)};
            r.owned[i] = true;
            const int row = (n[i] - o.row0) * p.heads + h, g = row >> p.nr_log2;
            r.col[i] = row & (p.nr - 1);
            const int last = p.by_heads(min((g + 1) << p.nr_log2, o.T * p.heads) - 1);
            if (latent_limit(p, o, last) > 0) unit[i] = (b0 + src) * p.groups + g;  // else a unit without tiles
        }
    }
    int4 u[RW];
#pragma unroll
    for (int i = 0; i < RW; ++i) u[i] = unit[i] >= 0 ? __ldcg(p.units + unit[i]) : make_int4(0, -1, 0, 0);
#pragma unroll
    for (int i = 0; i < RW; ++i) {
        r.first[i] = u[i].x;
        r.whole[i] = u[i].w != 0;
        r.n[i] = r.whole[i] ? 0 : u[i].y - u[i].x + 1;
        r.slot[i] = u[i].z;
    }
    float2 v[RW][kShareChunks];
#pragma unroll
    for (int i = 0; i < RW; ++i)
#pragma unroll
        for (int q = 0; q < kShareChunks; ++q) {
            const int k = 32 * q + lane;
            v[i][q] = make_float2(-INFINITY, 0.f);
            if (k < r.n[i]) v[i][q] = __ldcg(p.ml + (size_t)r.slot_of(i, k) * p.nr + r.col[i]);
        }
#pragma unroll
    for (int i = 0; i < RW; ++i) {
        float M = -INFINITY, L = 0.f;
#pragma unroll
        for (int q = 0; q < kShareChunks; ++q) M = fmaxf(M, v[i][q].x);
#pragma unroll
        for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
#pragma unroll
        for (int q = 0; q < kShareChunks; ++q) {
            r.f[i][q] = v[i][q].x == -INFINITY ? 0.f : ex2(v[i][q].x - M);
            L += v[i][q].x == -INFINITY ? v[i][q].y : v[i][q].y * r.f[i][q];
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
        const float inv = L == 0.f ? 0.f : 1.f / L;
#pragma unroll
        for (int q = 0; q < kShareChunks; ++q) r.f[i][q] *= inv;
        r.lse[i] = (M + log2f(L) - kShift) * 0.6931471805599453f;
    }
}
// The same for one row, handed by the warp that looked it up to the others of
// its block (each of them asking for itself made every block's 16 warps queue
// for the same few lines of L2: 10 us with 150 shares).
struct RowCard {
    int first, n, slot, col, whole, owned;
    float f[kMaxBlocks];
    __device__ __forceinline__ void put(const RowSums<1> &r, int lane) {
        if (lane == 0) {
            first = r.first[0];
            n = r.n[0];
            slot = r.slot[0];
            col = r.col[0];
            whole = r.whole[0];
            owned = r.owned[0];
        }
        for (int q = 0; q < kShareChunks; ++q) f[32 * q + lane] = r.f[0][q];
    }
    __device__ __forceinline__ void get(RowSums<1> &r, int lane) const {
        r.first[0] = first;
        r.n[0] = n;
        r.slot[0] = slot;
        r.col[0] = col;
        r.whole[0] = whole;
        r.owned[0] = owned;
#pragma unroll
        for (int q = 0; q < kShareChunks; ++q) r.f[0][q] = f[32 * q + lane];
    }
};
// Warp-wide: columns d4 .. d4 + 3 of the rows' joined sums over the shares k0,
// k0 + step and so on (step at most 32).
template <int RW>
__device__ __forceinline__ void join_sums(const LatentParams &p, const RowSums<RW> &r, int k0, int step, int d4,
                                          float4 (&a)[RW]) {
    int most = 0;
#pragma unroll
    for (int i = 0; i < RW; ++i) most = max(most, r.n[i]);
#pragma unroll
    for (int q = 0; q < kShareChunks; ++q) {
        if (32 * q >= most) break;
#pragma unroll 2
        for (int k = 0; k < min(most - 32 * q, 32); k += step) {
            float4 v[RW];
            float g[RW];
#pragma unroll
            for (int i = 0; i < RW; ++i) {
                const int c = 32 * q + k + k0;
                const bool in = k + k0 < 32 && c < r.n[i];
                g[i] = __shfl_sync(0xffffffffu, r.f[i][q], (k + k0) & 31);
                if (!in) g[i] = 0.f;
                v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (in)
                    v[i] = __ldcg(reinterpret_cast<const float4 *>(
                        p.part + ((size_t)r.slot_of(i, c) * p.nr + r.col[i]) * p.R + d4));
            }
#pragma unroll
            for (int i = 0; i < RW; ++i) {
                a[i].x = fmaf(g[i], v[i].x, a[i].x);
                a[i].y = fmaf(g[i], v[i].y, a[i].y);
                a[i].z = fmaf(g[i], v[i].z, a[i].z);
                a[i].w = fmaf(g[i], v[i].w, a[i].w);
            }
        }
    }
}
// Another block's shared memory (between two cluster barriers, so that the
// loads need no order among themselves).
__device__ __forceinline__ float2 cluster_ld2(const void *p, uint32_t rank) {
    uint32_t a;
    float2 v;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(a));
    return v;
}

// Cluster of R / 64 blocks per (head h, 16 MT tokens): block s multiplies the
// joined sums of latent columns 64 s .. + 63 by that slice of W_uv[h] and the
// cluster adds the slices up.  The joined sums enter the product as two values
// of the type (v and what its rounding left), which costs nothing here and
// saves a rounding.  With JOIN (few tokens, MT = 1) the block joins them
// itself, else they are in o_lat.  Bound by the chain of reads before its short
// product (144 tokens of 16 heads: 10.7 us alone).
template <int DT, int MT, bool JOIN>
__global__ void __launch_bounds__(JOIN ? 512 : 256, JOIN ? 1 : 3) latent_out_kernel(const __grid_constant__ LatentParams p) {
    static_assert(!JOIN || MT == 1, "a row per warp at least");
    constexpr int kThreads = JOIN ? 512 : 256;
    extern __shared__ __align__(128) uint8_t lo_smem[];
    uint16_t *wv = reinterpret_cast<uint16_t *>(lo_smem);          // [dv][72]
    uint16_t *hi = wv + p.dv * 72, *lo = hi + 16 * MT * 72;        // [16 MT][72] each
    float *part = reinterpret_cast<float *>(lo + 16 * MT * 72);    // [16 MT][dv]
    const int s = blockIdx.x, h = blockIdx.y, n0 = blockIdx.z * 16 * MT;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rows = min(16 * MT, p.N - n0);
    griddep_wait();
    griddep_launch_dependents();
    const uint16_t *wsrc = p.w_uv + (size_t)h * p.dv * p.R + 64 * s;
    for (int i = threadIdx.x; i < p.dv * 8; i += kThreads)
        cp_async16(wv + (i >> 3) * 72 + 8 * (i & 7), wsrc + (size_t)(i >> 3) * p.R + 8 * (i & 7));
    for (int i = rows * 9 + threadIdx.x; i < 16 * MT * 9; i += kThreads)  // rows past the last token
        reinterpret_cast<uint4 *>(hi)[i] = reinterpret_cast<uint4 *>(lo)[i] = make_uint4(0, 0, 0, 0);
    const int half = lane >> 4, d4 = 4 * (lane & 15);
    auto put = [&](int r, const float4 &a) {
        const uint2 v = make_uint2(Elem<DT>::down2(a.x, a.y), Elem<DT>::down2(a.z, a.w));
        const float2 y = Elem<DT>::up2(v.x), z = Elem<DT>::up2(v.y);
        *reinterpret_cast<uint2 *>(hi + r * 72 + d4) = v;
        *reinterpret_cast<uint2 *>(lo + r * 72 + d4) =
            make_uint2(Elem<DT>::down2(a.x - y.x, a.y - y.y), Elem<DT>::down2(a.z - z.x, a.w - z.y));
    };
    if constexpr (JOIN) {
        __shared__ float4 spread[16][16];
        __shared__ RowCard cards[16];
        // 16 warps: a row each, or with few rows several warps (and always both halves) for one
        const int wp = rows > 8 ? 1 : rows > 4 ? 2 : rows > 2 ? 4 : rows > 1 ? 8 : 16;
        const int sub = warp % wp, r = warp / wp;
        RowSums<1> rs;
        if (warp < rows) {
            const int n[1] = {n0 + warp};
            find_rows<1>(p, n, h, lane, rs);
            cards[warp].put(rs, lane);
            if (rs.owned[0] && !rs.whole[0] && s == 0 && lane == 0 && p.lse) p.lse[(size_t)n[0] * p.heads + h] = rs.lse[0];
        }
        __syncthreads();
        cards[min(r, rows - 1)].get(rs, lane);
        if (r >= rows) rs.n[0] = rs.whole[0] = 0;
        float4 sum[1] = {make_float4(0.f, 0.f, 0.f, 0.f)};
        if (rs.whole[0] && sub == 0 && half == 0)
            sum[0] = __ldcg(reinterpret_cast<const float4 *>(p.o_lat + ((size_t)(n0 + r) * p.heads + h) * p.R + 64 * s + d4));
        join_sums<1>(p, rs, 2 * sub + half, 2 * wp, 64 * s + d4, sum);
        float4 a = sum[0];
        a.x += __shfl_xor_sync(0xffffffffu, a.x, 16);
        a.y += __shfl_xor_sync(0xffffffffu, a.y, 16);
        a.z += __shfl_xor_sync(0xffffffffu, a.z, 16);
        a.w += __shfl_xor_sync(0xffffffffu, a.w, 16);
        if (wp > 1) {
            if (half == 0) spread[warp][lane] = a;
            __syncthreads();
            if (sub == 0 && half == 0)
                for (int k = 1; k < wp; ++k) {
                    const float4 v = spread[warp + k][lane];
                    a.x += v.x;
                    a.y += v.y;
                    a.z += v.z;
                    a.w += v.w;
                }
        }
        if (sub == 0 && half == 0 && r < rows) put(r, a);
    } else {
        float4 a[MT];
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            const int r = 16 * i + 2 * warp + half;
            a[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r < rows)
                a[i] = __ldcg(reinterpret_cast<const float4 *>(p.o_lat + ((size_t)(n0 + r) * p.heads + h) * p.R + 64 * s + d4));
        }
#pragma unroll
        for (int i = 0; i < MT; ++i)
            if (16 * i + 2 * warp + half < rows) put(16 * i + 2 * warp + half, a[i]);
    }
    cp_async_wait_all();
    __syncthreads();
    const int v0 = 16 * warp;
    if (v0 < p.dv) {
        float acc[MT][2][4] = {};
#pragma unroll
        for (int k = 0; k < 64; k += 16) {
            uint32_t b[4];
            ldsm4(b, wv + (v0 + (lane & 7) + 8 * (lane >> 4)) * 72 + k + 8 * ((lane >> 3) & 1));
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                uint32_t a[4];
                ldsm4(a, hi + (16 * m + (lane & 15)) * 72 + k + 8 * (lane >> 4));
                mma16816<DT>(acc[m][0], a, b[0], b[1]);
                mma16816<DT>(acc[m][1], a, b[2], b[3]);
                ldsm4(a, lo + (16 * m + (lane & 15)) * 72 + k + 8 * (lane >> 4));
                mma16816<DT>(acc[m][0], a, b[0], b[1]);
                mma16816<DT>(acc[m][1], a, b[2], b[3]);
            }
        }
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                *reinterpret_cast<float2 *>(part + (16 * m + (lane >> 2) + 8 * (j & 1)) * p.dv + v0 + 8 * (j >> 1) +
                                            2 * (lane & 3)) =
                    make_float2(acc[m][j >> 1][2 * (j & 1)], acc[m][j >> 1][2 * (j & 1) + 1]);
    }
    cluster_arrive();
    cluster_wait();
    const int ns = p.R / 64, dv_log2 = p.dv == 128 ? 7 : 6, pairs = rows << (dv_log2 - 1);
    for (int i = (int)cluster_rank() * kThreads + threadIdx.x; i < pairs; i += ns * kThreads) {
        float2 v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = k < ns ? cluster_ld2(part + 2 * i, (uint32_t)k) : make_float2(0.f, 0.f);
        float2 a = v[0];
#pragma unroll
        for (int k = 1; k < 8; ++k) {
            a.x += v[k].x;
            a.y += v[k].y;
        }
        const int r = 2 * i >> dv_log2, d = 2 * i & (p.dv - 1);
        *reinterpret_cast<uint32_t *>(p.out + (n0 + r) * p.out_stride + (size_t)h * p.dv + d) =
            Elem<DT>::down2(a.x, a.y);
    }
    cluster_arrive_relaxed();  // the others have read this block's sums
    cluster_wait();
}

// Folded weights, and many tokens: one block per row joins its partial sums, 4
// columns a thread and SUB threads a column, into out or (fp32, for the product
// that follows) o_lat; rows of whole units are there already.  SUB = 4
// shortens the sums of few rows, 1 leaves room for more blocks (4096 rows of 3
// shares: 25 us with 4, 13 with 1, from DRAM).  Bound by latency: two look-ups,
// then the sums.
template <int DT, int SUB>
__global__ void __launch_bounds__(128 * SUB) latent_join_kernel(const __grid_constant__ LatentParams p) {
    __shared__ float4 spread[SUB][128];
    __shared__ RowCard card;
    griddep_wait();
    griddep_launch_dependents();
    const int row = blockIdx.x, n[1] = {p.by_heads(row)}, h = row - n[0] * p.heads, lane = threadIdx.x & 31;
    const int sub = threadIdx.x >> 7, col = threadIdx.x & 127, d4 = 4 * col;
    RowSums<1> rs;
    if (threadIdx.x < 32) {
        find_rows<1>(p, n, h, lane, rs);
        card.put(rs, lane);
    }
    __syncthreads();
    if (card.whole || (!card.owned && !p.w_uv)) return;
    card.get(rs, lane);
    float4 a[1] = {make_float4(0.f, 0.f, 0.f, 0.f)};
    if (d4 < p.R) join_sums<1>(p, rs, sub, SUB, d4, a);
    if (SUB > 1) {
        spread[sub][col] = a[0];
        __syncthreads();
        if (sub) return;
        for (int k = 1; k < SUB; ++k) {
            const float4 v = spread[k][col];
            a[0].x += v.x;
            a[0].y += v.y;
            a[0].z += v.z;
            a[0].w += v.w;
        }
    }
    if (d4 < p.R) {
        if (p.w_uv)
            *reinterpret_cast<float4 *>(p.o_lat + (size_t)row * p.R + d4) = a[0];
        else
            *reinterpret_cast<uint2 *>(p.out + n[0] * p.out_stride + (size_t)h * p.R + d4) =
                make_uint2(Elem<DT>::down2(a[0].x, a[0].y), Elem<DT>::down2(a[0].z, a[0].w));
    }
    if (threadIdx.x == 0 && p.lse && rs.owned[0]) p.lse[row] = rs.lse[0];
}

// -------------------------------------------------------------------- host --
bool attn_maps(const LatentParams &p, int dt, const void *q, AttnMaps *maps) {
    const uint64_t tok = (uint64_t)p.token_stride * 2, pieces = (uint64_t)(p.R + p.P) / 64;
    const uint64_t dims[4] = {64, (uint64_t)p.page_size, pieces, (uint64_t)p.num_pages};
    const uint64_t strides[3] = {tok, 128, p.num_pages > 1 ? (uint64_t)p.page_stride * 2 : tok * p.page_size};
    const uint32_t pair[4] = {64, (uint32_t)p.box_tokens, p.box_tokens == kTile ? 2u : 1u, 1};
    const uint32_t rope[4] = {64, (uint32_t)p.box_tokens, 1, 1};
    const uint64_t qd[3] = {64, (uint64_t)p.N * p.heads, pieces}, qs[2] = {(uint64_t)(p.R + p.P) * 2, 128};
    const uint32_t qb[3] = {64, (uint32_t)p.nr, (uint32_t)pieces};
    return map_rows64(&maps->pair, dt, p.cache, 4, dims, strides, pair) &&
           map_rows64(&maps->rope, dt, p.cache, 4, dims, strides, rope) && map_rows64(&maps->q, dt, q, 3, qd, qs, qb);
}

template <int DT, int NR>
int launch_attn(const LatentParams &p, const AttnMaps &maps, int blocks, cudaStream_t s) {
    int st = set_smem<latent_attn_kernel<DT, NR>>(AttnGeo<NR>::kSmem);
    if (st) return st;
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t c = latent_config(dim3(blocks), AttnGeo<NR>::kThreads, AttnGeo<NR>::kSmem, s, attr, 1);
    return record_launch(cudaLaunchKernelEx(&c, latent_attn_kernel<DT, NR>, p, maps));
}

// Tokens per block of the products with the up-projections, in sixteens: 64 once
// there are enough of them to fill the SMs (heads x R / 64 blocks per group).
int token_tiles(int N) { return N > 32 ? 4 : 1; }

template <int DT>
int launch_q(const LatentParams &p, cudaStream_t s) {
    cudaLaunchAttribute attr[2];
    if (!p.w_uk) {
        cudaLaunchConfig_t c = latent_config(dim3(p.N), 128, 0, s, attr, 1);
        return record_launch(cudaLaunchKernelEx(&c, latent_pack_kernel, p));
    }
    const int mt = token_tiles(p.N);
    const size_t smem = (size_t)(16 * mt * (p.dn + 8) + p.dn * 72) * 2;
    cudaLaunchConfig_t c = latent_config(dim3(p.R / 64, p.heads, (p.N + 16 * mt - 1) / (16 * mt)), 128, smem, s, attr, 1);
    return record_launch(mt == 1 ? cudaLaunchKernelEx(&c, latent_q_kernel<DT, 1>, p)
                                 : cudaLaunchKernelEx(&c, latent_q_kernel<DT, 4>, p));
}

template <int DT, int MT, bool JOIN>
int launch_out(const LatentParams &p, cudaStream_t s) {
    const size_t smem = (size_t)(p.dv * 72 + 2 * 16 * MT * 72) * 2 + (size_t)16 * MT * p.dv * 4;
    const int st = set_smem<latent_out_kernel<DT, MT, JOIN>>((size_t)(128 * 72 + 2 * 16 * MT * 72) * 2 + (size_t)16 * MT * 512);
    if (st) return st;
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t c = latent_config(dim3(p.R / 64, p.heads, (p.N + 16 * MT - 1) / (16 * MT)), JOIN ? 512 : 256, smem, s,
                                         attr, p.R / 64);
    return record_launch(cudaLaunchKernelEx(&c, latent_out_kernel<DT, MT, JOIN>, p));
}

template <int DT>
int launch_absorbed(LatentParams &p, int dtype, bool packed, cudaStream_t s) {
    int st;
    p.chained = p.w_uk || !packed;
    const void *q = p.chained ? p.q_lat : p.q;
    AttnMaps maps;
    memset(&maps, 0, sizeof(maps));
    if (!attn_maps(p, dtype, q, &maps)) return SPX_ERR_UNSUPPORTED;
    const int sms = device_sm_count();
    if (sms < 1) return SPX_ERR_CUDA;
    const int blocks = sms < kMaxBlocks ? sms : kMaxBlocks;
    if (p.chained && (st = launch_q<DT>(p, s))) return st;
    st = p.nr == 16 ? launch_attn<DT, 16>(p, maps, blocks, s)
         : p.nr == 32 ? launch_attn<DT, 32>(p, maps, blocks, s)
                      : launch_attn<DT, 64>(p, maps, blocks, s);
    if (st) return st;
    // Many tokens: their rows are joined once, not by each of the R / 64 blocks that multiply them.
    if (p.w_uv && token_tiles(p.N) == 1) return launch_out<DT, 1, true>(p, s);
    cudaLaunchAttribute attr[2];
    const int sub = p.N * p.heads <= 4 * sms ? 4 : 1;
    cudaLaunchConfig_t c = latent_config(dim3(p.N * p.heads), 128 * sub, 0, s, attr, 1);
    st = record_launch(sub == 4 ? cudaLaunchKernelEx(&c, latent_join_kernel<DT, 4>, p)
                                : cudaLaunchKernelEx(&c, latent_join_kernel<DT, 1>, p));
    return st || !p.w_uv ? st : launch_out<DT, 4, false>(p, s);
}

// Rows per unit: the call's largest request in one unit where 16 or 32 rows
// hold it (least padding), else 64, the most that shared memory leaves room for.
int rows_per_unit(int max_q, int heads) {
    const long long rows = (long long)max_q * heads;
    return rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
}

constexpr size_t kHdr = 256;
size_t up256(size_t n) { return (n + 255) / 256 * 256; }
// The workspace of the absorbed form.
struct AbsorbedLayout {
    size_t units, ml, part, q_lat, o_lat, bytes;
};
AbsorbedLayout absorbed_layout(int B, int N, int max_q, int heads, int R, int P, bool weights) {
    const int nr = rows_per_unit(max_q, heads);
    const size_t groups = ((size_t)max_q * heads + nr - 1) / nr;
    AbsorbedLayout l;
    l.units = kHdr;
    l.ml = l.units + up256((size_t)B * groups * 16);
    l.part = l.ml + up256((size_t)2 * kMaxBlocks * 64 * 8);
    l.q_lat = l.part + up256((size_t)2 * kMaxBlocks * nr * R * 4);
    l.o_lat = l.q_lat + up256((size_t)N * heads * (R + P) * 2);
    l.bytes = l.o_lat + (weights ? up256((size_t)N * heads * R * 4) : 0);
    return l;
}
// The workspace of the expanded form.
struct ExpandedLayout {
    size_t k, v, rope, bytes;
    int rows;
};
ExpandedLayout expanded_layout(int B, int max_len, int heads) {
    ExpandedLayout l;
    l.rows = max_len <= 128 ? 128 : (int)(((long long)max_len + 127) / 128 * 128);
    const size_t one = (size_t)heads * B * l.rows * 256;
    l.k = kHdr;
    l.v = l.k + one;
    l.rope = l.v + one;
    l.bytes = l.rope + (size_t)B * l.rows * 128;
    return l;
}
// The form that a call takes: the one whose estimate is smaller, in us on 152
// SMs.  Absorbed: 1.55 per tile of 64 tokens and 64 rows and SM, 4 ns per (token,
// head) row of the joined results.  Expanded: 3.4 per key tile of 128 tokens,
// head and SM to write keys and values, 2.2 per key tile in which a block attends
// (blocks of 256 rows; few of them leave SMs idle).  Measured, absorbed /
// expanded: 16 heads, 4 x 4096 cached, 64 rows 81 / 114, 256 rows 249 / 118; 1 x
// 16384, 256 rows 197 / 269; 1 x 600, 32 rows 25 / 20; 32 heads, 4 x 4096, 96
// rows 197 / 176.
int latent_form(int form, int B, int max_q, int max_len, int heads, int dn, int dv) {
    if (form != SPX_LATENT_AUTO) return form;
    if (dn != 128 || dv != 128) return SPX_LATENT_ABSORBED;
    const double sms = 152, rows = (double)max_q * heads, tiles = ceil(max_len / 128.0);
    const double seen = ceil((max_len - (max_q < max_len ? max_q : max_len) / 2.0) / 128.0);  // causal
    const double blocks = (double)B * heads * ceil(max_q / 256.0);
    const double absorbed = 14 + 1.55 * ceil(B * ceil(rows / 64) * ceil(max_len / 64.0) / sms) + 0.004 * B * rows;
    const double expanded = 8 + 3.4 * ceil(B * tiles * heads / sms) + 2.2 * seen * (blocks > sms ? blocks / sms : 1);
    return expanded < absorbed ? SPX_LATENT_EXPANDED : SPX_LATENT_ABSORBED;
}

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
    // (token, head) rows and cached rows are counted in 31 bits
    if ((long long)N * heads > 1 << 30 || (long long)max_q * heads > 1 << 30 || (long long)B * max_len > 1 << 30) return 0;
    if ((dn != 0) != (dv != 0) || (dn && dn != 64 && dn != 128) || (dv && dv != 64 && dv != 128)) return 0;
    const int used = latent_form(form, B, max_q, max_len, heads, dn, dv);
    if (used == SPX_LATENT_EXPANDED) return dn == 128 && dv == 128 ? expanded_layout(B, max_len, heads).bytes : 0;
    // So are the tiles of all units, whatever q_start and lens hold; and the grid of the products with the
    // up-projections ends at 65535 blocks of 64 tokens.
    const long long nr = rows_per_unit(max_q, heads), rows = (long long)(max_q < N ? max_q : N) * heads;
    if ((double)B * ((rows + nr - 1) / nr) * ((max_len + 63) / 64) > 2e9 || (dn && N > 64 * 65535)) return 0;
    return absorbed_layout(B, N, max_q, heads, R, P, dn != 0).bytes;
}

extern "C" int spx_latent_attention(const spx_latent_args *a, spx_stream_t stream) {
    if (!a) return SPX_ERR_INVALID_ARG;
    int st = latent_cache_check(a->cache);
    if (st) return st;
    const spx_latent_cache &c = *a->cache;
    if (!a->q_start || a->N < 0 || a->heads < 1 || a->max_q < 0 || a->max_len < 0) return SPX_ERR_INVALID_ARG;
    if (a->N > 0 && (!a->q || !a->out)) return SPX_ERR_INVALID_ARG;
    // weights and widths together or neither: the workspace's size goes by the widths, the launches by the weights
    if (!a->w_uk != !a->w_uv || !a->w_uk != !a->dn || !a->w_uv != !a->dv) return SPX_ERR_INVALID_ARG;
    if (!(a->scale > 0.f) || !(a->scale < INFINITY)) return SPX_ERR_INVALID_ARG;
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
    p.max_q = a->max_q;
    const long long cap = (long long)c.max_pages * c.page_size;
    p.max_len = a->max_len < cap ? a->max_len : (int)cap;
    p.by_heads.set(a->heads);
    p.by_page.set(c.page_size);
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
    p.budget = a->wait_budget_ns ? a->wait_budget_ns : 2000000000ull;
    p.box_tokens = c.page_size % 64 == 0 ? 64 : c.page_size % 32 == 0 ? 32 : 16;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (latent_form(a->form, c.B, a->max_q, a->max_len, a->heads, a->dn, a->dv) == SPX_LATENT_EXPANDED) {
        const ExpandedLayout l = expanded_layout(c.B, a->max_len, a->heads);
        p.k_x = reinterpret_cast<uint16_t *>(ws + l.k);
        p.v_x = reinterpret_cast<uint16_t *>(ws + l.v);
        p.rope_x = reinterpret_cast<uint16_t *>(ws + l.rope);
        p.kv_rows = l.rows;
        return launch_expanded(p, c.dtype, s);
    }
    const AbsorbedLayout l = absorbed_layout(c.B, a->N, a->max_q, a->heads, c.R, c.P, p.w_uk != nullptr);
    p.nr = rows_per_unit(a->max_q, a->heads);
    p.nr_log2 = p.nr == 16 ? 4 : p.nr == 32 ? 5 : 6;
    p.groups = (int)(((long long)a->max_q * a->heads + p.nr - 1) / p.nr);
    p.units = reinterpret_cast<int4 *>(ws + l.units);
    p.ml = reinterpret_cast<float2 *>(ws + l.ml);
    p.part = reinterpret_cast<float *>(ws + l.part);
    p.q_lat = reinterpret_cast<uint16_t *>(ws + l.q_lat);
    p.o_lat = reinterpret_cast<float *>(ws + l.o_lat);
    const bool packed = a->q_stride == qw || a->N == 1;
    return c.dtype == SPX_F16 ? launch_absorbed<SPX_F16>(p, c.dtype, packed, s)
                              : launch_absorbed<SPX_BF16>(p, c.dtype, packed, s);
}
