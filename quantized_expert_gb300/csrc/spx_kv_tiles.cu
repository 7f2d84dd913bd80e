// spx_kv_tiles.cu -- attention over the paged cache of keys and values, calls
// of more than 16 (token, head) rows a key head: trees, verify passes, prompts.
//
// Rows that share a key head (the tokens of a request times the query heads of
// the group) are the 128 rows of a product:  S = Q K^T (128 rows x 128 cached
// tokens), softmax in registers, a row a thread, P back into S's tensor memory
// as the A operand of O += P V.  Keys and values come from the cache's pages as
// they lie, by tensor copies of whole runs of a page's tokens.
//
//   attention launch  shares of key tiles, one block an SM; partial sums of the
//                     units that cross from block to block
//   join launch       their sums, weighed and added in the order of the blocks
//
// The unit of a tree or a verify pass is bound by reading its keys and values,
// that of a prompt by the chain of one product, softmax and product: per tile of
// 256 rows and 128 keys 2 x (512 + 512) cycles of products, at the chip's rate,
// of 2600 to 2700 measured.  16384 tokens, 32 heads: 1.5 to 1.57 PFLOP/s.  A unit's
// beginning and end, 8000 cycles, leave the tensor cores idle, so that shorter
// prompts run at less (4096 tokens 120 us, 1.14 PFLOP/s; four chunks of up to 1021
// tokens behind up to 6007, pages of 16, 146 us, of which 73 tiles a block are
// 100).  Trees of 64 rows, 16 requests of up to 3001 tokens and 16 heads: 53.9 us,
// 4.7 TB/s; 17 rows, one request of 4113 tokens and 8 key heads: 12.6 us.
#include <math.h>
#include <string.h>

#include "spx_kv.cuh"
#include "spx_tcgen05.cuh"

namespace spx {

namespace {

constexpr int kThreads = 384;  // copies of K and V, two warps for products, copies of Q; 2 x 4 softmax warps
constexpr int kPiece = kKvTile * 128;  // 128 rows of 64 values, 16 KB

// What a unit costs beside its tiles (its first copies, the last product, the
// results), in tiles; us for 2, 3, 4: prompt of 4096 tokens 138, 126.5, 122, three
// of 2048 126, 120, 111, chunks as above 152.6, 150.1, 148.9, trees as above 56.4,
// 56.2, 56.2.  (5 and more are not measured: no minimum is known.)
constexpr int kUnitCost = 4;
static_assert(kUnitCost <= kKvMostCost, "what the workspace's size is checked for");
constexpr int kMiscBytes = 3 << 10;  // of a block's shared memory, behind the tiles

struct KvMaps {
    CUtensorMap k;     // [page][head][token][D], boxes of 64 values x box_tokens
    CUtensorMap v;     // [page][head][D / 64][token][64], boxes of all a token's values x box_tokens
    CUtensorMap q;     // [row][head][D], boxes of 64 values x a group's heads x q_tokens
};

// Two products are under way at a time, X = 0 and 1, and take turns: while one's
// softmax runs, the other's products do.  TALL: two tiles of 128 rows of a unit,
// on the same key tiles.  Otherwise a unit is one tile of rows, and X takes
// every second key tile; the two sums are joined at the unit's end.
template <int D, bool TALL>
struct Tiles {
    static constexpr int kPieces = D / 64;
    static constexpr int kSlot = kPieces * kPiece;  // keys or values of a tile
    static constexpr int kQTiles = TALL ? 2 : 1;
    // Slots, keys and values of a tile in turn; an even number where two warps fill them, so that each has its own.
    static constexpr int kRing = (14 - kQTiles * kPieces) / kPieces & (TALL ? ~0 : ~1);
    static constexpr int kSmem = (kQTiles * kPieces + kRing * kPieces) * kPiece + kMiscBytes;
    static constexpr int kRows = kQTiles * kKvTileRows;  // rows of a unit
    static_assert(kSmem <= kSmemLimit && kRing >= 5, "shared memory of one block");
};
// A unit's part in a block's share, as the fourth warp hands it to the others.
struct Unit {
    int end;             // tiles tile .. end - 1 of the unit; 0: no more units
    int tile, whole;     // whole: these are all of them
    int row0, T, len;    // the request
    int t0, h;           // first row (of the request), key head
    int n[2];            // tiles of X
    int b;
    int before;          // tiles of the block before it
    int tiles[2], units[2]; // of X before it: its tiles, units in which it has any
};
constexpr int kUnitRing = 4;
struct Misc {
    uint64_t ufull[kUnitRing], uempty[kUnitRing];
    uint64_t qfull, qempty;              // by units
    uint64_t full[14], empty[14];        // by slots
    uint64_t sfull[2], pfull[2][2];      // by tiles of X; pfull: by halves of the keys
    uint64_t odone[2], oempty[2];        // by units in which X has tiles
    uint64_t turn[2], fin[2];
    uint32_t tmem;
    int abort;
    Unit unit[kUnitRing];
    alignas(16) uint32_t bad[2][4][4];   // tokens with values that are not finite, in the last four tiles of a unit
    float2 ml[2][kKvTileRows];           // X's references and weights
};
static_assert(sizeof(Misc) <= kMiscBytes, "the misc area holds it");

// A place in the ring and the parity of its use.
template <int N>
struct Place {
    uint32_t i = 0, phase = 0;
    __device__ __forceinline__ void advance(uint32_t n) {  // n <= N
        i += n;
        if (i >= N) {
            i -= N;
            phase ^= 1;
        }
    }
    __device__ __forceinline__ void jump(uint32_t n) {
        i += n;
        phase ^= (i / N) & 1;
        i %= N;
    }
};

// Where the 64 values c of a tile's token t lie in a slot of values: a copy's
// tokens, 64 values each, then the next 64 of the same tokens.  (Keys lie 64
// values of all the tile's tokens after the other, as a K-major operand wants
// its groups of 8 rows at one distance; an MN-major one has no such wish, so
// that one copy brings whole rows, and pages of 16 tokens half the copies.)
template <int kPieces>
__device__ __forceinline__ int v_row(int box_tokens, int t, int c) {
    return (t & -box_tokens) * (128 * kPieces) + c * box_tokens * 128 + (t & (box_tokens - 1)) * 128;
}

// A softmax row takes 128 scores in registers: 168 a thread, what 384 threads
// share out evenly, are too few, so the first four warps give up some (4 x 32 x
// 72 + 8 x 32 x 208 <= 384 x 168; trees of 16 requests 55.2 us, with it 53.5, of
// one 15.7, 15.05; prompts within 1%).
__device__ __forceinline__ void fewer_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 72;"); }
__device__ __forceinline__ void more_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 208;"); }

// ctl_wait by a whole warp, which goes on or gives up as one: elections, loads of
// tensor memory and barriers take a warp together, and nothing else says that
// lanes do not leave the wait apart.  (One tree of 17 rows 13.1 us, with the votes
// 13.24; four chunks as above 149.7 and 150.2.)
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, const WaitCtl &c) {
    return __all_sync(0xffffffffu, ctl_wait(bar, parity, c));
}

// The same for the next unit.  A thread that waits is suspended for as long as the
// hardware likes, some microseconds, in which a shorter limit is lost; here one is
// kept to by asking without (in every wait it costs 1 to 2%), so that a call with a
// limit below a microsecond is sure to give up.
constexpr uint64_t kBriefNs = 1000;
__device__ __forceinline__ bool unit_wait(uint64_t *bar, uint32_t parity, const WaitCtl &c) {
    if (c.budget >= kBriefNs) return warp_wait(bar, parity, c);
    const uint64_t t0 = global_timer_ns();
    while (!__all_sync(0xffffffffu, mbar_test(bar, parity))) {
        if (__any_sync(0xffffffffu, *c.abort)) return false;
        if (__any_sync(0xffffffffu, global_timer_ns() - t0 > c.budget)) {
            record_timeout(c.status, c.site);
            *c.abort = 1;
            return false;
        }
    }
    return true;
}

// (four chunks as above 147.2 us, with it 146.6)
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// Values loaded from tensor memory are used behind this only: nothing else keeps
// arithmetic on them behind the wait.
template <int N>
__device__ __forceinline__ void hold(uint32_t (&r)[N]) {
#pragma unroll
    for (int i = 0; i < N; i += 8)
        asm volatile("" : "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), "+r"(r[i + 4]), "+r"(r[i + 5]),
                          "+r"(r[i + 6]), "+r"(r[i + 7]));
}

template <int DT, int D, bool TALL>
__global__ void __launch_bounds__(kThreads, 1)
    kv_tiles_kernel(const __grid_constant__ KvParams p, const __grid_constant__ KvMaps maps) {
    using C = Tiles<D, TALL>;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t *qs = smem, *ring = smem + C::kQTiles * C::kSlot;
    Misc &m = *reinterpret_cast<Misc *>(ring + C::kRing * C::kSlot);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kUnitRing; ++i) {
            mbar_init(&m.ufull[i], 1);
            mbar_init(&m.uempty[i], 11);  // copies, issuers, softmax warps
        }
        mbar_init(&m.qfull, 1);
        mbar_init(&m.qempty, TALL ? 2 : 1);
        for (int i = 0; i < C::kRing; ++i) {
            mbar_init(&m.full[i], 1);
            mbar_init(&m.empty[i], TALL ? 2 : 1);
        }
        for (int x = 0; x < 2; ++x) {
            mbar_init(&m.sfull[x], 1);
            mbar_init(&m.pfull[x][0], 4);
            mbar_init(&m.pfull[x][1], 4);
            mbar_init(&m.odone[x], 1);
            mbar_init(&m.oempty[x], TALL ? 4 : 8);
            mbar_init(&m.turn[x], 1);
            mbar_init(&m.fin[x], 1);
        }
        m.abort = 0;
        fence_mbar_init();
    }
    if (warp == 2) (&m.bad[0][0][0])[lane] = 0;
    if (p.q_tokens * p.group < kKvTileRows) {  // rows that no copy brings
        for (int i = threadIdx.x; i < C::kQTiles * C::kSlot / 16; i += kThreads)
            reinterpret_cast<uint4 *>(qs)[i] = make_uint4(0, 0, 0, 0);
        fence_proxy_async_smem();
    }
    if (warp == 0 && elect_one()) {
        prefetch_tmap(&maps.k);
        prefetch_tmap(&maps.v);
        prefetch_tmap(&maps.q);
    }
    if (warp == 1) {
        tmem_alloc(&m.tmem, 512);
        tmem_relinquish();
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = m.tmem;
    const WaitCtl ctl{&m.abort, &p.hdr->status, p.budget, SITE_KV};
    if (warp == 3) kv_prefetch(p, lane);
    griddep_wait();
    griddep_launch_dependents();

    if (warp < 4) {
        fewer_registers();
        if (warp == 3) {
            // ---- the share's units, one ahead of the copies of their queries but the first's; the unit that begins in this
            // share and ends in a later one, for the join launch
            const uint64_t pol = policy_evict_normal();
            const KvShare share = kv_find_share(p, p.span, lane);
            KvWalk w;
            w.begin(p, share, p.span);
            int4 seam = make_int4(0, 0, 0, 0);  // where there is one for each block
            int q_row = 0, q_head = 0;  // of the unit whose queries are to be copied next
            int before = 0, tiles[2] = {0, 0}, units[2] = {0, 0};
            bool ok = true;
            const auto copy_queries = [&]() {
                if (elect_one()) {
                    mbar_arrive_expect_tx(&m.qfull, C::kQTiles * C::kPieces * 128 * p.group * p.q_tokens);
                    for (int x = 0; x < C::kQTiles; ++x)
                        for (int c = 0; c < C::kPieces; ++c)
                            tma_load_3d(qs + (x * C::kPieces + c) * kPiece, &maps.q, 64 * c, q_head, q_row + x * p.tile_tokens,
                                        &m.qfull, pol);
                }
                __syncwarp();
            };
            for (uint32_t u = 0; ok; ++u) {
                const bool more = w.left > 0;
                if (!(ok = warp_wait(&m.uempty[u % kUnitRing], ((u / kUnitRing) & 1) ^ 1, ctl))) break;
                const int row = w.rq.row0 + w.g * p.span, head = w.h * p.group;
                if (more) {
                    if (u == 0) {  // nothing to wait for
                        q_row = row;
                        q_head = head;
                        copy_queries();
                    }
                    // Key tiles of X in the unit's part: TALL, those of its rows; else every second one.
                    const int parts = w.end - w.tile, t0 = w.g * p.span;
                    int n[2];
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const int first = t0 + x * p.tile_tokens, last = min(first + p.tile_tokens, w.rq.T) - 1;
                        const int all = last < first ? 0 : (kv_none_see(p, w.rq, last) + kKvTile - 1) / kKvTile;
                        n[x] = TALL ? min(max(all - w.tile, 0), parts) : (parts - x + 1) / 2;
                    }
                    if (lane == 0) {
                        m.unit[u % kUnitRing] = Unit{w.end, w.tile, w.whole(), w.rq.row0, w.rq.T, w.rq.len, t0, w.h, {n[0], n[1]},
                                                     w.b, before, {tiles[0], tiles[1]}, {units[0], units[1]}};
                        mbar_arrive(&m.ufull[u % kUnitRing]);
                    }
                    before += parts;
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        tiles[x] += n[x];
                        units[x] += n[x] > 0;
                    }
                    if (w.tile == 0) {
                        const bool cut = w.end < w.nt;
                        const int4 s = make_int4(row, min(w.rq.T - t0, p.span), w.h,
                                                 cut ? (int)blockIdx.x << 16 | (w.flat + w.nt - 1) / share.share : 0);
                        if (cut) seam = s;
                        if (p.seam_groups && lane == 0) p.seams[(w.b * p.kv_heads + w.h) * p.seam_groups + w.g] = s;
                    }
                    w.next(p, p.span);
                } else if (lane == 0) {
                    m.unit[u % kUnitRing].end = 0;
                    mbar_arrive(&m.ufull[u % kUnitRing]);
                }
                __syncwarp();
                if (u > 1) {
                    if (!(ok = warp_wait(&m.qempty, (u & 1), ctl))) break;  // of the unit before the last
                    copy_queries();
                }
                q_row = row;
                q_head = head;
                if (!more) break;
            }
            if (!p.seam_groups && lane == 0) p.seams[blockIdx.x] = seam;
        } else if (warp == 0 || (!TALL && warp == 2)) {
            // ---- copies: keys and values of the tiles in turn; where a warp is to spare, the values by that one, as a
            // short call waits for both
            const uint64_t pol = policy_evict_normal();
            // (a lane a copy: keys lane % boxes, 64 values lane / boxes; values lane)
            const int bt = p.box_tokens, boxes = kKvTile / bt, box = lane % boxes, piece = lane / boxes;
            // (a single request's table comes nearer while its share is looked for)
            if (p.B == 1 && 32 * lane < p.max_pages)
                asm volatile("prefetch.global.L1 [%0];" ::"l"(p.table + 32 * lane) : "memory");
            Place<C::kRing> r;
            const int kv0 = TALL ? 0 : warp >> 1, kv1 = TALL ? 2 : kv0 + 1;
            r.advance(kv0);
            bool ok = true;
            for (uint32_t u = 0; ok; ++u) {
                if (!(ok = warp_wait(&m.ufull[u % kUnitRing], (u / kUnitRing) & 1, ctl))) break;
                const Unit &d = m.unit[u % kUnitRing];
                const int end = d.end, first = d.tile, len = d.len, h = d.h;
                const int32_t *table = p.table + (size_t)d.b * p.max_pages;
                __syncwarp();
                if (lane == 0) mbar_arrive(&m.uempty[u % kUnitRing]);
                if (end == 0) break;
                int next = -1;  // the page of the lane's box, looked up a tile ahead
                const auto look_up = [&](int tile) {
                    const int p0 = kKvTile * tile + bt * box;
                    next = p0 < len ? __ldg(table + p.by_page(p0)) : -1;
                };
                look_up(first);
                for (int j = first; ok && j < end; ++j) {
                    const int p0 = kKvTile * j + bt * box, at = p0 - p.by_page(p0) * p.page_size;
                    const int page = next < 0 || next >= p.num_pages ? p.num_pages : next;  // (past the last one: zeros)
                    if (j + 1 < end) look_up(j + 1);
#pragma unroll 1
                    for (int kv = kv0; kv < kv1; ++kv, r.advance(TALL ? 1 : 2)) {
                        // (a converged warp asks one barrier, one word and one clock here; with a vote four chunks take
                        // 154 us for 149)
                        if (!(ok = ctl_wait(&m.empty[r.i], r.phase ^ 1, ctl))) break;
                        if (elect_one()) mbar_arrive_expect_tx(&m.full[r.i], C::kSlot);
                        __syncwarp();
                        uint8_t *dst = ring + r.i * C::kSlot;
                        if (kv) {
                            if (lane < boxes)
                                tma_load_5d(dst + box * bt * 128 * C::kPieces, &maps.v, 0, at, 0, h, page, &m.full[r.i], pol);
                        } else if (lane < boxes * C::kPieces) {
                            tma_load_4d(dst + piece * kPiece + box * bt * 128, &maps.k, 64 * piece, at, h, page, &m.full[r.i], pol);
                        }
                        __syncwarp();
                    }
                }
            }
        } else {
            // ---- products: O_X of X's last tile, then S_X of its next one, in one stretch behind everything that they
            // wait for.  TALL: a warp for each X, which pass a turn to each other and both see every slot.  Else the first
            // for both: a warp that saw only every second tile could wait for a slot before its last use, by the other,
            // had landed, and take the use before that, of the same parity, for the one that it waits for.
            const uint32_t fmt = DT == SPX_BF16 ? kIdescBf16 : 0u;
            const uint32_t id_s = idesc_f16_f32(128, 128) | fmt, id_o = idesc_f16_f32(128, D) | fmt | kIdescBMn;
            const uint64_t qd = sw128_desc(smem_u32(qs)), kd = sw128_desc(smem_u32(ring));
            const uint64_t vd = sw128_desc_mn(smem_u32(ring), p.box_tokens * 128);
            uint32_t vk[kKvTile / 16];  // of 16 tokens' values in a slot, in the descriptor's units
#pragma unroll
            for (int i = 0; i < kKvTile / 16; ++i) vk[i] = v_row<C::kPieces>(p.box_tokens, 16 * i, 0) / 16;
            const auto scores = [&](int x, uint32_t slot) {
                const uint64_t q = qd + (TALL ? x * (C::kSlot / 16) : 0), k = kd + slot * (C::kSlot / 16);
#pragma unroll
                for (int c = 0; c < C::kPieces; ++c)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        umma_f16(tmem + 128 * x, q + c * (kPiece / 16) + 2 * i, k + c * (kPiece / 16) + 2 * i, id_s, c | i);
            };
            const auto sums = [&](int x, uint32_t slot, int half, bool first) {
#pragma unroll
                for (int i = 4 * half; i < 4 * half + 4; ++i)
                    umma_f16_ta(tmem + 256 + 128 * x, tmem + 128 * x + 8 * i, vd + slot * (C::kSlot / 16) + vk[i], id_o,
                                !first || i);
            };
            Place<C::kRing> at;  // of the keys of the unit's first tile
            uint32_t tile0 = 0, tile1 = 0, unit0 = 0, unit1 = 0, step = 0;  // tiles and units of X before this one, turns
            bool ok = true;
            for (uint32_t u = 0; ok; ++u) {
                if (!(ok = warp_wait(&m.ufull[u % kUnitRing], (u / kUnitRing) & 1, ctl))) break;
                const Unit &d = m.unit[u % kUnitRing];
                const int end = d.end, all = end - d.tile, n0 = d.n[0], n1 = d.n[1];
                __syncwarp();
                if (lane == 0) mbar_arrive(&m.uempty[u % kUnitRing]);
                if (end == 0) break;
                Place<C::kRing> kr = at, vr = at;
                vr.advance(1);
                ok = warp_wait(&m.qfull, u & 1, ctl);
                // Step j: S of tile j, and O of the tile before (TALL; X's own, on the same tiles), or of the one before
                // that (tiles belong to X = 0 and 1 in turn).
                constexpr int kLag = TALL ? 1 : 2;
#pragma unroll 1
                for (int j = 0; ok && j < all + kLag; ++j) {
                    const int x = TALL ? warp - 1 : j & 1, t = j - kLag, n = TALL ? (x ? n1 : n0) : all;
                    const bool has_o = t >= 0 && t < n, has_s = j < n;
                    const uint32_t parity = ((x ? tile1 : tile0) + (TALL ? t : t >> 1)) & 1;  // of O's weights
                    const bool first = TALL ? t == 0 : t < 2, last = TALL ? t == n - 1 : t >= all - 2;  // O of X in the unit
                    // the slots of the unit's last tile are room for its results, and given back by the softmax warps
                    const bool last_k = TALL && j == all - 1, last_v = t == all - 1;
                    ok = (j >= all || ctl_wait(&m.full[kr.i], kr.phase, ctl)) && (t < 0 || ctl_wait(&m.full[vr.i], vr.phase, ctl)) &&
                         // tile 1 goes behind tile 0's products of the same step, tile 0 behind tile 1's of the last
                         // one, or they fall into step, both softmaxes at once and then both products
                         (!TALL || (x ? ctl_wait(&m.turn[1], step & 1, ctl) : step == 0 || ctl_wait(&m.turn[0], (step - 1) & 1, ctl))) &&
                         (!has_o || !first || ctl_wait(&m.oempty[x], ((x ? unit1 : unit0) & 1) ^ 1, ctl)) &&
                         (!has_o || ctl_wait(&m.pfull[x][0], parity, ctl));
                    if (!(ok = __all_sync(0xffffffffu, ok))) break;
                    tc_fence_after();
                    if (has_o) {  // the first half while the softmax is at the second
                        if (elect_one()) sums(x, vr.i, 0, first);
                        __syncwarp();
                        if (!(ok = warp_wait(&m.pfull[x][1], parity, ctl))) break;
                        tc_fence_after();
                    }
                    if (elect_one()) {
                        if (has_o) {
                            sums(x, vr.i, 1, false);
                            if (!last_v) umma_commit(&m.empty[vr.i]);
                            if (last) umma_commit(&m.odone[x]);
                        } else if (t >= 0 && !last_v) {
                            mbar_arrive(&m.empty[vr.i]);
                        }
                        if (has_s) {
                            scores(x, kr.i);
                            if (!last_k) umma_commit(&m.empty[kr.i]);
                            umma_commit(&m.sfull[x]);
                            if (j == n - 1) umma_commit(&m.qempty);
                        } else if (j < all && !last_k) {
                            mbar_arrive(&m.empty[kr.i]);
                        }
                        if (n == 0 && j == 0) mbar_arrive(&m.qempty);
                        if (TALL) mbar_arrive(&m.turn[x ^ 1]);
                    }
                    __syncwarp();
                    if (t >= 0) vr.advance(2);
                    kr.advance(2);
                    ++step;
                }
                tile0 += n0;
                tile1 += n1;
                unit0 += n0 > 0;
                unit1 += n1 > 0;
                at.jump(2 * all);
            }
        }
    } else {
        more_registers();
        // ---- softmax and results: a row a thread
        const int x = (warp - 4) >> 2, q = warp & 3, r = 32 * q + lane;
        const uint32_t quarter = (uint32_t)(32 * q) << 16;
        const uint32_t st = tmem + quarter + 128 * x, ot = tmem + quarter + 256;
        // (What a unit's end needs is read from its description there, and not held in registers beside a row's scores.)
        // (Warps that meet at barriers leave together: where one gave up, all hear of it.)
        bool ok = unit_wait(&m.ufull[0], 0, ctl);
        if (bar_any(2, 256, !ok)) ok = false;
#pragma unroll 1
        for (uint32_t u = 0; ok; ++u) {
            const Unit &d = m.unit[u % kUnitRing];
            if (d.end == 0) break;
            const auto row_of = [&](int &t) {  // the thread's row of the request, and whether there is one
                const int t_of = p.by_group(r);
                t = d.t0 + (TALL ? x * p.tile_tokens : 0) + t_of;
                return t_of < p.tile_tokens && t < d.T;
            };
            const int n = d.n[x], first = d.tile;
            KvSeen seen;
            int all;
            bool warp_live;
            {
                int t;
                const bool live = row_of(t);
                const KvReq rq{d.row0, d.T, d.len};
                warp_live = __any_sync(0xffffffffu, live);
                seen = kv_seen(p, rq, live ? t : rq.T);
                all = kv_all_see(p, rq, d.t0);
            }
            float mr = -INFINITY, l = 0.f;
            bool fine = true;  // no wait of the unit has given up
            const uint32_t tile = d.tiles[x];
#pragma unroll 1
            for (int i = 0; i < n; ++i) {
                const int li = TALL ? i : 2 * i + x, j = first + li, p0 = kKvTile * j;
                const bool masked = p0 + kKvTile > all;
                if (!(fine = warp_wait(&m.sfull[x], (tile + i) & 1, ctl))) break;
                tc_fence_after();
                if (masked) {
                    // Of a tile that not every row sees whole, the values of tokens past the length, and of those that
                    // hold one which is not finite, become zeros, as a weight of 0 does not make them so; the rows
                    // that see such a token become NaNs at the end.  A token a thread.  (Not before the scores are there: only
                    // then is the slot's last use known to be over, and the wait's parity that of this use.)
                    const uint32_t item = 2 * (d.before + li) + 1, slot = item % C::kRing;
                    if (!(fine = warp_wait(&m.full[slot], (item / C::kRing) & 1, ctl))) break;
                    uint8_t *row = ring + slot * C::kSlot + v_row<C::kPieces>(p.box_tokens, r, 0);
                    const int piece = p.box_tokens * 128;  // to the row's next 64 values
                    bool zero = p0 + r >= d.len;
                    if (!zero) {
                        uint32_t z = 0;
#pragma unroll
                        for (int k = 0; k < 8 * C::kPieces; ++k) {
                            const uint4 v = lds128(row + (k >> 3) * piece + (((k ^ r) & 7) << 4));
                            z = Elem<DT>::fma2(v.x, 0u, z);
                            z = Elem<DT>::fma2(v.y, 0u, z);
                            z = Elem<DT>::fma2(v.z, 0u, z);
                            z = Elem<DT>::fma2(v.w, 0u, z);
                        }
                        if (z & 0x7FFF7FFFu) {
                            zero = true;
                            atomicOr(&m.bad[u & 1][j & 3][r >> 5], 1u << (r & 31));
                        }
                    }
                    if (zero)
#pragma unroll
                        for (int k = 0; k < 8 * C::kPieces; ++k)
                            *reinterpret_cast<uint4 *>(row + (k >> 3) * piece + (((k ^ r) & 7) << 4)) = make_uint4(0, 0, 0, 0);
                    fence_proxy_async_smem();
                    __syncwarp();  // the lane that tells of the warp's weights tells of these zeros too, and a warp without rows
                                   // has nothing else to meet at
                }
                if (warp_live) {
                    uint32_t s[128];
#pragma unroll
                    for (int c = 0; c < 4; ++c) tmem_ld32(st + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(s + 32 * c));
                    tmem_wait_ld();
                    hold(s);
                    if (masked) {
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            const uint32_t word = seen.word(p0 + 32 * c);
#pragma unroll
                            for (int k = 0; k < 32; ++k)
                                if (!(word >> k & 1)) s[32 * c + k] = 0xFF800000u;
                        }
                    }
                    float mx[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) mx[k] = fmaxf(__uint_as_float(s[k]), __uint_as_float(s[k + 8]));
#pragma unroll
                    for (int k = 16; k < 128; k += 16)
#pragma unroll
                        for (int y = 0; y < 8; ++y) mx[y] = max3(mx[y], __uint_as_float(s[k + y]), __uint_as_float(s[k + y + 8]));
                    const float top = max3(max3(mx[0], mx[1], mx[2]), max3(mx[3], mx[4], mx[5]), fmaxf(mx[6], mx[7]));
                    const bool rise = (top - mr) * p.scale_log2 > kKvSlack;  // (scale > 0; not if both are -inf)
                    if (__any_sync(0xffffffffu, rise)) {
                        const float mn = rise ? top : mr, f = mn == mr ? 1.f : ex2((mr - mn) * p.scale_log2);
                        mr = mn;
                        l *= f;
                        if (i > 0) {
                            // (O_X of the last tile is done: this tile's S_X came behind it)
#pragma unroll 1
                            for (int c = 0; c < D; c += 16) {
                                uint32_t o[16];
                                tmem_ld16(ot + 128 * x + c, o);
#pragma unroll
                                for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                                tmem_st16(ot + 128 * x + c, o);
                            }
                        }
                    }
                    float ref = kv_ref(mr, p.scale_log2);
                    const bool far = kv_far(mr, p.scale_log2);
                    if (__any_sync(0xffffffffu, far)) {
                        const float from = far ? mr : 0.f;
#pragma unroll
                        for (int k = 0; k < 128; ++k) s[k] = __float_as_uint(__uint_as_float(s[k]) - from);
                        if (far) ref = kKvShift;
                    }
                    const uint64_t sc2 = pack2(p.scale_log2, p.scale_log2), ref2 = pack2(ref, ref);
                    uint64_t l2[2] = {0, 0};
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        uint32_t o[16];
#pragma unroll
                        for (int k = 0; k < 16; ++k) {
                            const float2 v = unpack2(fma2(pack2(__uint_as_float(s[32 * c + 2 * k]), __uint_as_float(s[32 * c + 2 * k + 1])),
                                                          sc2, ref2));
                            const float a = ex2(v.x), b = ex2(v.y);
                            l2[k & 1] = add2(l2[k & 1], pack2(a, b));
                            o[k] = Elem<DT>::down2(a, b);  // rounded for the tensor cores; the weights' own sum is not
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
                } else if (lane == 0) {
                    mbar_arrive(&m.pfull[x][0]);
                    mbar_arrive(&m.pfull[x][1]);
                }
            }
            // ---- the unit's end
            mr *= p.scale_log2;  // from here on with the scale
            const int parts = d.end - first, other = d.n[x ^ 1];
            fine = fine && (n == 0 || warp_wait(&m.odone[x], d.units[x] & 1, ctl)) &&
                   (other == 0 || warp_wait(&m.odone[x ^ 1], d.units[x ^ 1] & 1, ctl));
            tc_fence_after();
            if (!TALL) m.ml[x][r] = make_float2(mr, l);
            __syncwarp();
            // References, weights and lists of bad tokens are there.  Where a wait gave up all leave, and give no slot back: a
            // copy into it may be in flight, and the next one's bytes would count on the same phase of its barrier.
            if (bar_any(1, 256, !fine)) break;
            float f[2] = {1.f, 1.f};
            if (!TALL) {
                const float2 a = m.ml[0][r], b = m.ml[1][r];
                mr = fmaxf(a.x, b.x);
                f[0] = kv_factor(a.x, mr);
                f[1] = kv_factor(b.x, mr);
                l = a.y * f[0] + b.y * f[1];
            }
            // Whether the row sees a token with a value that is not finite: hardly ever is there one at all.
            bool poison = false;
            {
                const uint4 *lists = reinterpret_cast<const uint4 *>(&m.bad[u & 1][0][0]);
                uint4 any = lists[0];
#pragma unroll
                for (int i = 1; i < 4; ++i) any = make_uint4(any.x | lists[i].x, any.y | lists[i].y, any.z | lists[i].z, any.w | lists[i].w);
                if (any.x | any.y | any.z | any.w)
                    for (int j = max(first, all / kKvTile); j < first + parts; ++j)
                        for (int c = 0; c < 4; ++c)
                            if (m.bad[u & 1][j & 3][c] & seen.word(kKvTile * j + 32 * c)) poison = true;
            }
            const bool whole = d.whole;
            const float inv = !whole ? 1.f : l == 0.f ? 0.f : 1.f / l;
            f[0] = poison ? NAN : f[0] * inv;
            f[1] = poison ? NAN : f[1] * inv;
            // Results pass through the slots of the unit's last tile (TALL: of its keys for X = 0, of its values for
            // X = 1; else of its values), a warp's rows in a place of their own, so that stores are of whole rows and
            // not of 16 bytes of 32 rows.  Units of 16 bytes are permuted by the row.
            constexpr int kCols = TALL ? D : D / 2, kRow = kCols * 2, kU = kRow / 16;  // a warp's columns (else halves of D), bytes of a row
            const uint32_t item = 2 * (d.before + parts - 1), k_slot = item % C::kRing, v_slot = (item + 1) % C::kRing;
            const int c0 = TALL ? 0 : x * kCols;
            const size_t place = (size_t)(2 * blockIdx.x + (first == 0)) * C::kRows + (TALL ? 128 * x : 0) + 32 * q;
            if (warp_live) {
                int t;
                const bool live = row_of(t);
                const KvReq rq{d.row0, d.T, d.len};
                // (TALL; else it may hold another unit's by now)
                fine = (!TALL || warp_wait(&m.full[k_slot], (item / C::kRing) & 1, ctl)) &&
                       warp_wait(&m.full[v_slot], ((item + 1) / C::kRing) & 1, ctl);
                uint8_t *stage = ring + (TALL && x == 0 ? k_slot : v_slot) * C::kSlot + ((TALL ? 0 : 4 * x) + q) * 32 * kRow;
                // unit k of row i of the warp's 32
                const auto staged = [&](int i, int k) {
                    return reinterpret_cast<uint4 *>(stage + i * kRow + ((k ^ (i & (kU - 1))) << 4));
                };
                const bool has[2] = {TALL ? n > 0 : (x ? other : n) > 0, !TALL && (x ? n : other) > 0};
                // A half of the warp's columns at a time, scaled.
                constexpr int kHalf = kCols / 2, kLd = kHalf < 32 ? 16 : 32;
                const auto half_of = [&](int half, uint32_t (&o)[kHalf]) {
                    const uint32_t at = ot + c0 + half * kHalf;
#pragma unroll
                    for (int y = 0; y < (TALL ? 1 : 2); ++y) {
                        if (!has[y]) {
                            if (y == 0)
#pragma unroll
                                for (int k = 0; k < kHalf; ++k) o[k] = 0;
                            continue;
                        }
                        uint32_t v[kHalf];
#pragma unroll
                        for (int c = 0; c < kHalf; c += kLd) {
                            if (kLd == 32)
                                tmem_ld32(at + 128 * (TALL ? x : y) + c, *reinterpret_cast<uint32_t(*)[32]>(&v[c]));
                            else
                                tmem_ld16(at + 128 * (TALL ? x : y) + c, *reinterpret_cast<uint32_t(*)[16]>(&v[c]));
                        }
                        tmem_wait_ld();
                        hold(v);
#pragma unroll
                        for (int k = 0; k < kHalf; ++k)
                            o[k] = __float_as_uint(y == 0 ? __uint_as_float(v[k]) * f[0]
                                                          : fmaf(__uint_as_float(v[k]), f[1], __uint_as_float(o[k])));
                    }
                };
                if (whole) {
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        uint32_t o[kHalf];
                        half_of(half, o);
                        uint32_t over = 0;  // not zero: one is not finite
#pragma unroll
                        for (int k = 0; k < kU / 2; ++k) {
                            uint32_t v[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                v[i] = Elem<DT>::down2(__uint_as_float(o[8 * k + 2 * i]), __uint_as_float(o[8 * k + 2 * i + 1]));
                                if (DT == SPX_F16) over = Elem<DT>::fma2(v[i], 0u, over);
                            }
                            *staged(lane, half * (kU / 2) + k) = make_uint4(v[0], v[1], v[2], v[3]);
                        }
                        if (DT == SPX_F16 && (over & 0x7FFF7FFFu))  // (hardly ever: kv_held for all would cost what they do)
#pragma unroll
                            for (int k = 0; k < kU / 2; ++k) {
                                uint32_t v[4];
#pragma unroll
                                for (int i = 0; i < 4; ++i)
                                    v[i] = kv_down2<DT>(__uint_as_float(o[8 * k + 2 * i]), __uint_as_float(o[8 * k + 2 * i + 1]));
                                *staged(lane, half * (kU / 2) + k) = make_uint4(v[0], v[1], v[2], v[3]);
                            }
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    const int row0 = d.t0 + (TALL ? x * p.tile_tokens : 0), head0 = d.h * p.group;
                    // 16-byte unit k of the rows lane / kU + kStep i of the warp's 32, (row, head) by (row, head)
                    constexpr int kStep = 32 / kU;
                    const int k = lane % kU, step_t = kStep / p.group, step_j = kStep - step_t * p.group;
                    int i = lane / kU, tt = p.by_group(32 * q + i), jj = 32 * q + i - tt * p.group;
                    const int most = min(p.tile_tokens, rq.T - row0);
                    uint16_t *out = p.out + (int64_t)(rq.row0 + row0 + tt) * p.out_stride + (int64_t)(head0 + jj) * D + c0 + 8 * k;
                    const int64_t step = (int64_t)step_t * p.out_stride + step_j * D, wrap = p.out_stride - (int64_t)p.group * D;
#pragma unroll
                    for (int n8 = 0; n8 < kU; n8 += 8) {
                        uint4 v[8];
#pragma unroll
                        for (int y = 0; y < 8; ++y)
                            if (n8 + y < kU) v[y] = *staged(i + kStep * (n8 + y), k);
#pragma unroll
                        for (int y = 0; y < 8; ++y) {
                            if (n8 + y >= kU) continue;
                            if (tt < most) *reinterpret_cast<uint4 *>(out) = v[y];
                            tt += step_t;
                            jj += step_j;
                            out += step;
                            if (jj >= p.group) {
                                jj -= p.group;
                                ++tt;
                                out += wrap;
                            }
                        }
                    }
                    if (live && p.lse && (TALL || x == 0))
                        p.lse[(int64_t)(rq.row0 + t) * p.heads + head0 + r - p.by_group(r) * p.group] = kv_lse(mr, l);
                } else {
                    float *dst = p.part + place * D + c0;
#pragma unroll 1
                    for (int half = 0; half < 2; ++half) {  // 32 bits a value
                        uint32_t o[kHalf];
                        half_of(half, o);
#pragma unroll
                        for (int k = 0; k < kU; ++k) *staged(lane, k) = make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
                        fence_proxy_async_smem();
                        __syncwarp();
#pragma unroll 8
                        for (int i = 0; i < kU; ++i) {
                            const int row = i * (32 / kU) + lane / kU, k = lane % kU;
                            *reinterpret_cast<uint4 *>(dst + row * D + half * kHalf + 4 * k) = *staged(row, k);
                        }
                        __syncwarp();
                    }
                    if (live && (TALL || x == 0)) p.ml[place + lane] = make_float2(mr, l);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (n) mbar_arrive(&m.oempty[x]);
                if (!TALL && other) mbar_arrive(&m.oempty[x ^ 1]);
                mbar_arrive(&m.uempty[u % kUnitRing]);
            }
            if (warp == 4 && lane < 16) (&m.bad[(u & 1) ^ 1][0][0])[lane] = 0;
            ok = fine && unit_wait(&m.ufull[(u + 1) % kUnitRing], ((u + 1) / kUnitRing) & 1, ctl);
            if (bar_any(2, 256, !ok)) ok = false;  // and everyone has read what the next unit writes
            if (ok && q == 0 && lane == 0 && (TALL || x == 0)) {
                if (TALL) mbar_arrive(&m.empty[k_slot]);
                mbar_arrive(&m.empty[v_slot]);
            }
        }
    }
    __syncwarp();
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

// ------------------------------------------------------------------- join --
// Block (8 rows, unit), a row a warp: dependent reads (seam, parts), and at a
// prompt's end the bytes.  The unit is the one that begins in block y of the
// attention launch and ends in a later one, or (kByUnits) where units are half as
// many as blocks or fewer, unit y: few blocks without work, and if it has many
// parts they are read 16 or 32 at a time (not if it has few: 256 rows behind 5120
// tokens, 32 units, 32.6 us, 16 at a time, with half the warps, 39.1).  By units
// and by blocks, us: one tree of 17 rows over 4113 tokens, 8 units, 12.6 and 15.1;
// four trees of 64, 32 units, 32.4 and 35.2; 16 trees of 32 over 700, 128 units,
// 26.1 and 25.0.  At 8 a time four blocks fit an SM (four chunks as above 145.2 us,
// three 152.9).
constexpr int kJoinRows = 8;
template <int DT, int D, int kAhead, bool kByUnits>
__global__ void __launch_bounds__(32 * kJoinRows, kAhead == 8 ? 4 : 1) kv_join_kernel(const __grid_constant__ KvParams p, int unit_rows) {
    const int lane = threadIdx.x & 31;
    const int r = (int)blockIdx.x * kJoinRows + (threadIdx.x >> 5), in = r % kKvTileRows;
    const int t_of = p.by_group(in), t = r / kKvTileRows * p.tile_tokens + t_of;
    const int groups = kByUnits ? p.seam_groups : 1, y = blockIdx.y, g = y % groups, b = y / (groups * p.kv_heads);
    griddep_wait();
    griddep_launch_dependents();
    int4 seam = __ldcg(p.seams + y);
    if (kByUnits) {
        // (a unit of a request that has fewer has no entry, and none is sure to be there where a wait gave up)
        const KvReq rq = kv_req(p, b);
        seam.x = rq.row0 + g * p.span;
        seam.y = min(max(rq.T - g * p.span, 0), p.span);
        seam.z = (y - g) / groups - b * p.kv_heads;
    }
    const int c1 = min(seam.w & 0xFFFF, p.by_blocks.d - 1), c0 = seam.w >> 16 & 0xFFFF;
    if (c0 >= c1 || t_of >= p.tile_tokens || t >= seam.y) return;
    kv_write_row<DT, D>(p, kv_sum_parts<D, kAhead>(p, c0, c1, 0, 1, unit_rows, r, lane), seam.x + t,
                        seam.z * p.group + in - t_of * p.group, lane);
}

// -------------------------------------------------------------------- host --
bool kv_maps(const KvParams &p, int dt, KvMaps *m) {
    memset(m, 0, sizeof(*m));
    // (a stride of a dimension of one is not used, but has to pass for one)
    const uint64_t row = (uint64_t)p.D * 2;
    const uint64_t cd[4] = {(uint64_t)p.D, (uint64_t)p.page_size, (uint64_t)p.kv_heads, (uint64_t)p.num_pages};
    const uint64_t cs[3] = {(uint64_t)p.token_stride * 2, p.kv_heads > 1 ? (uint64_t)p.head_stride * 2 : row,
                            p.num_pages > 1 ? (uint64_t)p.page_stride * 2 : row};
    const uint32_t cb[4] = {64, (uint32_t)p.box_tokens, 1, 1};
    const uint64_t vd[5] = {64, cd[1], (uint64_t)p.D / 64, cd[2], cd[3]}, vs[4] = {cs[0], 128, cs[1], cs[2]};
    const uint32_t vb[5] = {64, (uint32_t)p.box_tokens, (uint32_t)p.D / 64, 1, 1};
    const uint64_t qd[3] = {(uint64_t)p.D, (uint64_t)p.heads, (uint64_t)p.N};
    const uint64_t qst[2] = {row, p.N > 1 ? (uint64_t)p.q_stride * 2 : row};
    const uint32_t qb[3] = {64, (uint32_t)p.group, (uint32_t)p.q_tokens};
    return map_rows64(&m->k, dt, p.k, 4, cd, cs, cb) && map_rows64(&m->v, dt, p.v, 5, vd, vs, vb) &&
           map_rows64(&m->q, dt, p.q, 3, qd, qst, qb);
}

template <int DT, int D, bool TALL>
int launch_dt(const KvParams &p, const KvMaps &maps, int blocks, cudaStream_t s) {
    using C = Tiles<D, TALL>;
    int st = set_smem<kv_tiles_kernel<DT, D, TALL>>(C::kSmem);
    if (st) return st;
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t c = latent_config(dim3((unsigned)blocks), kThreads, C::kSmem, s, attr, 1);
    if ((st = record_launch(cudaLaunchKernelEx(&c, kv_tiles_kernel<DT, D, TALL>, p, maps)))) return st;
    const int tokens = p.max_q < p.N ? p.max_q : p.N;  // rows of the largest unit
    const int rows = TALL ? C::kRows : tokens * p.group;
    const int units = p.seam_groups ? p.B * p.kv_heads * p.seam_groups : blocks, parts = blocks / units;
    c = latent_config(dim3((unsigned)((rows + kJoinRows - 1) / kJoinRows), (unsigned)units), 32 * kJoinRows, 0, s, attr, 1);
    return record_launch(!p.seam_groups ? cudaLaunchKernelEx(&c, kv_join_kernel<DT, D, 8, false>, p, C::kRows)
                         : parts <= 8   ? cudaLaunchKernelEx(&c, kv_join_kernel<DT, D, 8, true>, p, C::kRows)
                         : parts <= 16  ? cudaLaunchKernelEx(&c, kv_join_kernel<DT, D, 16, true>, p, C::kRows)
                                        : cudaLaunchKernelEx(&c, kv_join_kernel<DT, D, 32, true>, p, C::kRows));
}
template <int DT>
int launch_d(const KvParams &p, const KvMaps &maps, int blocks, bool tall, cudaStream_t s) {
    if (p.D == 128) return tall ? launch_dt<DT, 128, true>(p, maps, blocks, s) : launch_dt<DT, 128, false>(p, maps, blocks, s);
    return tall ? launch_dt<DT, 64, true>(p, maps, blocks, s) : launch_dt<DT, 64, false>(p, maps, blocks, s);
}

}  // namespace

int launch_kv_tiles(KvParams &p, int dt, int blocks, cudaStream_t s) {
    p.tile_tokens = kv_tile_tokens(p.group);
    const int tokens = p.max_q < p.N ? p.max_q : p.N;  // of a request at most
    const bool tall = tokens > p.tile_tokens;
    p.span = tall ? 2 * p.tile_tokens : p.tile_tokens;
    // (no more rows than a request may have: a copy takes long over rows past the last of all.  One tree of 17 rows over
    // 4113 tokens, 16 heads of their own: boxes of 128 rows 16.1 us, of 17 13.5)
    p.q_tokens = tokens < p.tile_tokens ? tokens : p.tile_tokens;
    p.unit_cost = kUnitCost;
    p.by_blocks.set(blocks);
    const long long groups = (tokens + p.span - 1) / p.span, units = groups * p.B * p.kv_heads;
    p.seam_groups = 2 * units <= blocks ? (int)groups : 0;
    p.box_tokens = 16;
    while (p.box_tokens < kKvTile && p.page_size % (2 * p.box_tokens) == 0) p.box_tokens *= 2;
    KvMaps maps;
    if (!kv_maps(p, dt, &maps)) return SPX_ERR_UNSUPPORTED;
    return dt == SPX_F16 ? launch_d<SPX_F16>(p, maps, blocks, tall, s) : launch_d<SPX_BF16>(p, maps, blocks, tall, s);
}

}  // namespace spx
