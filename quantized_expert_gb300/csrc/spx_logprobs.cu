// spx_logprobs.cu -- log probabilities of given tokens, entropy and the most
// likely alternatives of rows of logits, in one pass over memory.
//
// With a reference r (in base 2) and t_v = x_v log2(e) - r a row needs z = sum
// 2^t_v and d = sum t_v 2^t_v:  log p_v = ln(2) t_v - ln z,  entropy = ln z - ln(2)
// d / z.  Every thread keeps a reference of its own (near its running maximum), its
// z and d, and the threads' triples are joined at the end, as are those of the
// blocks that share a row (a cluster).  References are kept as they were rounded:
// then t_v is one rounding of its exact value, whatever the size of x_v, and what
// log2(e) itself lacks is 1e-8 of x_v - x_w between any two.
//
// Alternatives: each thread also remembers where its maximum lies.  A bound
// that between k and 2k of the threads' maxima reach (found by bisection) is
// one that at least k elements reach.  Long rows get such a bound from the first
// eighth of their elements, and the chunks that reach it are noted from there on;
// at the end only these, and the first eighth of the few threads whose maximum
// reaches the last bound, are read again (from L2), and the elements that reach
// it are ranked by counting.  (1088 rows of 102400 in bf16 with 20 alternatives:
// 52.5 us; all the chunks of such threads read again, 7 us more; without
// alternatives 39.6.)
//
// What bounds it: 4.25 TB/s of logits, where a copy runs at 6.8: 60% of the issue
// slots are taken, and 1088 rows are 1.8 waves of blocks (608 rows, one wave: 29
// us; fp32, 544 rows: 5.5 TB/s).
#include "spx_latent.cuh"

#include <math.h>

namespace spx {

namespace {

struct LogprobParams {
    const void *logits;
    int64_t stride;
    int N, V, k;
    const int32_t *ids;
    float *logp, *entropy, *top_logp;
    int32_t *top_ids;
};

// Order of the alternatives as one 64-bit key: the value first (larger is
// larger, -0 = +0, NaN above all), then the lower index.  0 is below every key.
__device__ __forceinline__ uint32_t order32(float x) {
    if (x != x) return 0xFFFFFFFFu;
    const uint32_t u = __float_as_uint(x + 0.f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ uint64_t order64(float x, int v) { return ((uint64_t)order32(x) << 32) | (uint32_t)~v; }

constexpr int kThreadsLp = 256, kWarpsLp = kThreadsLp / 32;
constexpr int kMaxCluster = 8, kMaxTop = 32;
constexpr int kCandidates = 2048;
constexpr int kHigh = 1024;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// Reference (in base 2), sum, and sum weighted by the exponent.
struct Stat {
    float m, z, d;
};
__device__ __forceinline__ Stat join(const Stat &a, const Stat &b) {
    Stat r;
    r.m = fmaxf(a.m, b.m);
    r.z = r.d = 0.f;
    if (a.z != 0.f) {  // (a NaN is not 0)
        const float t = a.m - r.m, f = ex2(t);
        r.z += a.z * f;
        r.d += (a.d + t * a.z) * f;
    }
    if (b.z != 0.f) {
        const float t = b.m - r.m, f = ex2(t);
        r.z += b.z * f;
        r.d += (b.d + t * b.z) * f;
    }
    return r;
}

// Two packed 16-bit values at a time: the larger of each pair (a NaN loses), and
// the pair with nothing below `low` (a NaN stays).
template <int DT>
__device__ __forceinline__ uint32_t max_pair(uint32_t a, uint32_t b) {
    uint32_t r;
    if (DT == SPX_F16)
        asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else
        asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
template <int DT>
__device__ __forceinline__ uint32_t floor_pair(uint32_t a, uint32_t low) {
    uint32_t r;
    if (DT == SPX_F16)
        asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(low));
    else
        asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(low));
    return r;
}
__device__ __forceinline__ float floor_nan(float a, float low) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(low));
    return r;
}

// 32 bytes of a row: kN elements from index v0 on, those outside [0, V) as -inf.
struct Raw {
    uint32_t w[8];
};
template <int DT>
struct Chunk {
    using T = typename Elem<DT>::T;
    static constexpr int kN = 32 / (int)sizeof(T);
    static constexpr int kDT = DT == SPX_F32 ? SPX_F16 : DT;
    static __device__ __forceinline__ Raw load(const T *x) {
        Raw r;
        asm volatile("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3]), "=r"(r.w[4]), "=r"(r.w[5]), "=r"(r.w[6]),
                       "=r"(r.w[7])
                     : "l"(x));
        return r;
    }
    static __device__ __forceinline__ Raw load(const T *x, int v0, int V) {
        if (v0 >= 0 && v0 + kN <= V) return load(x + v0);
        Raw r;
        T *e = reinterpret_cast<T *>(&r);
#pragma unroll
        for (int i = 0; i < kN; ++i) e[i] = v0 + i >= 0 && v0 + i < V ? x[v0 + i] : Elem<DT>::down(-INFINITY);
        return r;
    }
    static __device__ __forceinline__ void unpack(const Raw &r, float (&f)[kN]) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (DT == SPX_F32) {
                f[i] = __uint_as_float(r.w[i]);
            } else {
                const float2 p = Elem<kDT>::up2(r.w[i]);
                f[kN == 8 ? i : 2 * i] = p.x;
                f[kN == 8 ? i : 2 * i + 1] = p.y;
            }
        }
    }
    // the largest (a NaN loses; NaN if all are)
    static __device__ __forceinline__ float largest(const Raw &r) {
        if (DT == SPX_F32) {
            float m = __uint_as_float(r.w[0]);
#pragma unroll
            for (int i = 1; i < 8; ++i) m = fmaxf(m, __uint_as_float(r.w[i]));
            return m;
        }
        uint32_t m[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) m[i] = max_pair<kDT>(r.w[i], r.w[i + 4]);
        const float2 p = Elem<kDT>::up2(max_pair<kDT>(max_pair<kDT>(m[0], m[1]), max_pair<kDT>(m[2], m[3])));
        return fmaxf(p.x, p.y);
    }
    // What the lowest values count as: a -inf has weight 0 and must not meet an
    // infinite exponent in d.
    static constexpr float kFloor = DT == SPX_F16 ? -65504.f : -16777216.f;
    static __device__ __forceinline__ Raw floored(const Raw &r) {
        constexpr uint32_t low = DT == SPX_F16 ? 0xFBFFFBFFu : 0xCB80CB80u;  // kFloor
        Raw o;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            o.w[i] = DT == SPX_F32 ? __float_as_uint(floor_nan(__uint_as_float(r.w[i]), kFloor)) : floor_pair<kDT>(r.w[i], low);
        return o;
    }
};
// A maximum above kLarge sends its row through passes with differences first: a
// reference is its maximum's to 2^-24 of it, and 2^t could overflow for a much larger
// one.  So does a row's maximum that is not above kLow, from
// which the floor is not far enough.  (fp16's next value above its lowest is 32
// higher: what is floored weighs e^-32 at most there.)
constexpr float kLarge = 1e6f;
template <int DT>
constexpr float kLow = DT == SPX_F16 ? -65504.f : -kLarge;

// One thread's running sums over the elements of its chunks (two of each kind).
// Their reference follows the maximum only once that is kSlack above it: with a
// reference that moves at every new maximum some thread of a warp moves at most
// chunks.  e^kSlack stays small, since the entropy is a difference of ln z and d/z.
constexpr float kSlack = 4.f;
template <int DT>
struct Running {
    float m = -INFINITY, ref = -INFINITY;
    float rc = 0.f;                       // ref log2(e), rounded: what the exponents refer to
    uint64_t minus_rc = 0, z = 0, d = 0;
    int at;  // chunk of the first maximum
    __device__ __forceinline__ float take(const Raw &raw, int c) {
        using C = Chunk<DT>;
        const float mx = C::largest(raw);
        at = mx > m ? c : at;
        m = fmaxf(m, mx);
        if (mx > ref + kSlack) {
            const float to = fmaxf(mx, C::kFloor), to_rc = __fmul_rn(to, kLog2e);  // (not contracted with what follows)
            if (ref > -INFINITY) {
                const float t = rc - to_rc, g = ex2(t);
                d = mul2(fma2(pack2(t, t), z, d), pack2(g, g));
                z = mul2(z, pack2(g, g));
            }
            ref = to;
            rc = to_rc;
            minus_rc = pack2(-rc, -rc);
        }
        float f[C::kN];
        C::unpack(C::floored(raw), f);
#pragma unroll
        for (int i = 0; i < C::kN; i += 2) {
            const uint64_t t2 = fma2(pack2(f[i], f[i + 1]), pack2(kLog2e, kLog2e), minus_rc);
            const float2 t = unpack2(t2);
            const uint64_t e = pack2(ex2(t.x), ex2(t.y));
            z = add2(z, e);
            d = fma2(e, t2, d);
        }
        return mx;
    }
};

struct LogprobSmem {
    uint64_t key[kWarpsLp];              // scratch
    uint64_t cand[kCandidates];
    uint64_t top[kMaxCluster][kMaxTop];  // block 0: every block's alternatives
    Stat part[kMaxCluster];              // block 0: every block's sums
    Stat warp[kWarpsLp];
    uint32_t lo[kWarpsLp], hi[kWarpsLp];
    int n_cand, n_slices, slices[kThreadsLp];
    int n_high, high[kHigh];
    uint64_t few[2 * kMaxTop];
    int slow;
};

__device__ __forceinline__ uint32_t cluster_addr(const void *p, uint32_t rank) {
    uint32_t a;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a)
        : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(p))), "r"(rank));
    return a;
}
__device__ __forceinline__ void cluster_st(uint32_t a, float v) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(a), "f"(v) : "memory");
}
__device__ __forceinline__ void cluster_st(uint32_t a, uint64_t v) {
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(a), "l"(v) : "memory");
}

// The value of a key's upper half.
__device__ __forceinline__ float value_of(uint32_t o) {
    return o == 0xFFFFFFFFu ? NAN : __uint_as_float(o & 0x80000000u ? o & 0x7FFFFFFFu : ~o);
}

// The k largest keys of a row, one pass over it for each: rows with a
// NaN or a maximum above kLarge, and more candidates than the buffer holds.
template <int DT>
__device__ void top_by_passes(const typename Elem<DT>::T *x, int lo, int hi, int k, uint64_t *top, uint64_t *scratch) {
    uint64_t last = 0;
    for (int j = 0; j < k; ++j) {
        uint64_t best = 0;
        for (int v = lo + threadIdx.x; v < hi; v += kThreadsLp) {
            const uint64_t key = order64(Elem<DT>::up(x[v]), v);
            if ((j == 0 || key < last) && key > best) best = key;  // (a NaN at index 0 is the largest key there is)
        }
        for (int o = 16; o; o >>= 1) best = max(best, __shfl_xor_sync(0xffffffffu, best, o));
        __syncthreads();
        if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = best;
        __syncthreads();
        for (int w = 0; w < kWarpsLp; ++w) best = max(best, scratch[w]);
        last = best;
        if (threadIdx.x == 0) top[j] = best;
    }
    __syncthreads();
}

// A value that at least k of the block's threads' values (as order32 has them)
// reach, and no more than 2k if twelve halvings find such a one.
__device__ __forceinline__ uint32_t reached_by(uint32_t val, int k, LogprobSmem &s) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t lo = __reduce_min_sync(0xffffffffu, val), hi = __reduce_max_sync(0xffffffffu, val);
    if (lane == 0) {
        s.lo[warp] = lo;
        s.hi[warp] = hi;
    }
    __syncthreads();
    lo = __reduce_min_sync(0xffffffffu, s.lo[lane & (kWarpsLp - 1)]);
    hi = __reduce_max_sync(0xffffffffu, s.hi[lane & (kWarpsLp - 1)]);
    int reach = kThreadsLp;
    for (int i = 0; i < 12 && reach > 2 * k && hi - lo > 1; ++i) {
        const uint32_t mid = lo + (hi - lo) / 2;
        const int n = __syncthreads_count(val >= mid);
        if (n >= k) {
            lo = mid;
            reach = n;
        } else {
            hi = mid;
        }
    }
    __syncthreads();  // (s.lo and s.hi are written again)
    return lo;
}

// One cluster per row, its blocks taking equal stretches of it.  Four blocks an
// SM, for the registers of the loads in flight (five: 56 us for 52.5).
template <int DT>
__global__ void __launch_bounds__(kThreadsLp, 4) logprobs_kernel(const __grid_constant__ LogprobParams p) {
    using E = Elem<DT>;
    using T = typename E::T;
    using C = Chunk<DT>;
    constexpr int N = C::kN;
    __shared__ LogprobSmem s;
    const int nb = gridDim.x, row = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = cluster_rank();
    const T *x = static_cast<const T *>(p.logits) + (int64_t)row * p.stride;
    // chunk c holds the elements N c - shift on, so that its 32 bytes are aligned
    const int shift = (int)((reinterpret_cast<uintptr_t>(x) & 31) / sizeof(T));
    const int chunks = (p.V + shift + N - 1) / N, share = (chunks + nb - 1) / nb;
    const int c0 = (int)rank * share, c1 = min(chunks, c0 + share);

    griddep_wait();
    griddep_launch_dependents();
    cluster_arrive_relaxed();  // (awaited before the first store to block 0, which has begun by then)
    float given = NAN;  // the given token's logit
    if (rank == 0 && tid == 0 && p.logp) {
        const int id = p.ids[row];
        if (id >= 0 && id < p.V) given = E::up(x[id]);
    }
    Running<DT> run;
    run.at = c0 + tid;
    constexpr int kAhead = 3;  // loads in flight per thread
    const int whole = min(c1, (p.V + shift) / N);  // chunks that do not reach past the row
    // After the first chunks of each thread (an eighth) comes a first bound for the
    // alternatives, and the chunks that reach it are noted from there on.
    const int per = (c1 - c0 + kThreadsLp - 1) / kThreadsLp;
    const bool noting = p.k > 0 && per >= 4 * kAhead;
    const int first = noting ? (per / 8 + kAhead - 1) / kAhead * kAhead : per;
    float bound = INFINITY;
    if (tid == 0) s.n_cand = s.n_slices = s.n_high = 0;
    const auto take = [&](const Raw &raw, int c) {
        if (run.take(raw, c) >= bound) {
            const int n = atomicAdd(&s.n_high, 1);
            if (n < kHigh) s.high[n] = c;
        }
    };
    int c = c0 + tid;
#pragma unroll 1
    for (; c + (kAhead - 1) * kThreadsLp < whole; c += kAhead * kThreadsLp) {
        Raw raw[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int v0 = N * (c + u * kThreadsLp) - shift;
            raw[u] = u == 0 && v0 < 0 ? C::load(x, v0, p.V) : C::load(x + v0);
        }
        if (noting && c - tid == c0 + first * kThreadsLp) {
            const uint32_t o = reached_by(order32(run.m), p.k, s);
            if (o > order32(-INFINITY)) bound = value_of(o);
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) take(raw[u], c + u * kThreadsLp);
    }
#pragma unroll 1
    for (; c < c1; c += kAhead * kThreadsLp) {
        Raw raw[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
            if (c + u * kThreadsLp < c1) raw[u] = C::load(x, N * (c + u * kThreadsLp) - shift, p.V);
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
            if (c + u * kThreadsLp < c1) take(raw[u], c + u * kThreadsLp);
    }
    Stat a;
    {
        const float2 z = unpack2(run.z), d = unpack2(run.d);
        a = Stat{run.ref > -INFINITY ? run.rc : -INFINITY, z.x + z.y, d.x + d.y};
        if (run.ref == -INFINITY) a.d = 0.f;  // (nothing but -inf: no weight)
    }
    const int at = run.at;
    const bool bad = run.m > kLarge || a.z != a.z;
    const float own_m = run.m;
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        Stat b;
        b.m = __shfl_xor_sync(0xffffffffu, a.m, o);
        b.z = __shfl_xor_sync(0xffffffffu, a.z, o);
        b.d = __shfl_xor_sync(0xffffffffu, a.d, o);
        a = join(a, b);
    }
    if (lane == 0) s.warp[warp] = a;
    const bool any = c0 + tid < c1;
    const uint32_t val = any ? order32(own_m) : 0;
    {
        const uint32_t lo = __reduce_min_sync(0xffffffffu, val), hi = __reduce_max_sync(0xffffffffu, val);
        if (lane == 0) {
            s.lo[warp] = lo;
            s.hi[warp] = hi;
        }
    }
    const bool block_bad = __syncthreads_or(bad);
    cluster_wait();

    if (p.k > 0 && !block_bad) {
        // Upper and lower end of the keys that this thread's maximum may have.
        const uint64_t hi_key = any ? (uint64_t)val << 32 | (uint32_t)~max(N * at - shift, 0) : 0;
        const uint64_t key = any ? (uint64_t)val << 32 | (uint32_t)~(N * at - shift + N - 1) : 0;
        uint32_t lo32 = s.lo[lane & (kWarpsLp - 1)], hi32 = s.hi[lane & (kWarpsLp - 1)];
        lo32 = __reduce_min_sync(0xffffffffu, lo32);
        hi32 = __reduce_max_sync(0xffffffffu, hi32);
        // at least k keys reach tau (at first all of them, or those of the first bound), fewer reach hi
        if (bound < INFINITY) lo32 = max(lo32, order32(bound));
        uint64_t tau = (uint64_t)lo32 << 32, hi = ((uint64_t)hi32 << 32) + 0xffffffffull;
        int reach = kThreadsLp;
        while (reach > 2 * p.k && hi - tau > 1) {
            const uint64_t mid = tau + (hi - tau) / 2;
            const int n = __syncthreads_count(key >= mid);
            if (n >= p.k) {
                tau = mid;
                reach = n;
            } else {
                hi = mid;
            }
        }
        if (any && hi_key >= tau) s.slices[atomicAdd(&s.n_slices, 1)] = tid;
        __syncthreads();
        // their chunks up to the first bound and those noted after it (if there are
        // too many, all the chunks of theirs), dealt out over the block
        const int high = s.n_high, each = bound < INFINITY && high <= kHigh ? first : per;
        const int slices = s.n_slices * each, items = slices + (high > kHigh ? 0 : high);
        const uint32_t tau32 = (uint32_t)(tau >> 32);
        const float tau_value = tau32 > order32(-INFINITY) ? value_of(tau32) : -INFINITY;
#pragma unroll 1
        for (int i = tid; i < items; i += kThreadsLp) {
            const int slice = i / each;
            const int c = i < slices ? c0 + s.slices[slice] + (i - slice * each) * kThreadsLp : s.high[i - slices];
            if (c >= c1) continue;
            const Raw raw = C::load(x, N * c - shift, p.V);
            if (!(C::largest(raw) >= tau_value)) continue;
            float f[N];
            C::unpack(raw, f);
#pragma unroll
            for (int e = 0; e < N; ++e) {
                const int v = N * c - shift + e;
                const uint64_t kk = order64(f[e], v);
                if (kk >= tau && v >= 0 && v < p.V) {
                    const int n = atomicAdd(&s.n_cand, 1);
                    if (n < kCandidates) s.cand[n] = kk;
                }
            }
        }
        __syncthreads();
        if (s.n_cand > kCandidates) {
            top_by_passes<DT>(x, max(N * c0 - shift, 0), min(N * c1 - shift, p.V), p.k, s.cand, s.key);
            if (tid == 0) s.n_cand = p.k;
            __syncthreads();
        }
        int n = s.n_cand;
        const uint64_t *list = s.cand;
        // Ties leave many (all of a chunk's elements next to the one that counted):
        // a higher bound among them, found as the first, before they are ranked.
        if (n > kThreadsLp) {
            uint64_t lo = tau, end = ((uint64_t)hi32 << 32) + 0xffffffffull;
            int over = n;
            while (over > 2 * p.k && end - lo > 1) {
                const uint64_t mid = lo + (end - lo) / 2;
                int c = 0;
                for (int i = 0; i < n; i += kThreadsLp) c += __syncthreads_count(i + tid < n && s.cand[i + tid] >= mid);
                if (c >= p.k) {
                    lo = mid;
                    over = c;
                } else {
                    end = mid;
                }
            }
            if (tid == 0) s.n_slices = 0;
            __syncthreads();
            for (int i = tid; i < n; i += kThreadsLp)
                if (s.cand[i] >= lo) s.few[atomicAdd(&s.n_slices, 1)] = s.cand[i];
            __syncthreads();
            list = s.few;
            n = s.n_slices;
        }
        // the block's alternatives, to block 0
        for (int i = tid; i < n; i += kThreadsLp) {
            const uint64_t kk = list[i];
            int r = 0;
#pragma unroll 8
            for (int j = 0; j < n; ++j) r += list[j] > kk;
            // (a pass over too short a stretch leaves zeros)
            if (r < p.k && kk) cluster_st(cluster_addr(&s.top[rank][r], 0), kk);
        }
        for (int i = n + tid; i < p.k; i += kThreadsLp) cluster_st(cluster_addr(&s.top[rank][i], 0), (uint64_t)0);
    }
    if (warp == 0) {
        a = lane < kWarpsLp ? s.warp[lane] : Stat{-INFINITY, 0.f, 0.f};
#pragma unroll
        for (int o = kWarpsLp / 2; o; o >>= 1) {
            Stat b;
            b.m = __shfl_xor_sync(0xffffffffu, a.m, o);
            b.z = __shfl_xor_sync(0xffffffffu, a.z, o);
            b.d = __shfl_xor_sync(0xffffffffu, a.d, o);
            a = join(a, b);
        }
        if (lane == 0) {
            const uint32_t to = cluster_addr(&s.part[rank], 0);
            cluster_st(to, a.m);
            cluster_st(to + 4, block_bad ? NAN : a.z);
            cluster_st(to + 8, a.d);
        }
    }
    cluster_arrive();
    cluster_wait();
    if (rank != 0) return;

    // ---- block 0: the row
    a = s.part[0];
    bool slow = a.z != a.z, nan = false;  // (block_bad)
    for (int b = 1; b < nb; ++b) {
        slow |= s.part[b].z != s.part[b].z;
        a = join(a, s.part[b]);
    }
    const bool differences = slow || (a.m > -INFINITY && a.m <= kLow<DT> * kLog2e);
    if (differences) {  // two passes; the reference is the maximum itself from here on
        bool n = false;
        float m = -INFINITY;
        for (int v = tid; v < p.V; v += kThreadsLp) {
            const float f = E::up(x[v]);
            n |= f != f;
            m = fmaxf(m, f);
        }
        nan = __syncthreads_or(n);
#pragma unroll
        for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (lane == 0) s.warp[warp].m = m;
        __syncthreads();
        for (int w = 0; w < kWarpsLp; ++w) m = fmaxf(m, s.warp[w].m);
        a = Stat{m, 0.f, 0.f};
        if (!nan && m < INFINITY && m > -INFINITY) {
            for (int v = tid; v < p.V; v += kThreadsLp) {
                const float t = (E::up(x[v]) - m) * kLog2e, e = ex2(t);
                a.z += e;
                a.d = fmaf(e, fmaxf(t, -200.f), a.d);
            }
#pragma unroll
            for (int o = 16; o; o >>= 1) {
                a.z += __shfl_xor_sync(0xffffffffu, a.z, o);
                a.d += __shfl_xor_sync(0xffffffffu, a.d, o);
            }
            __syncthreads();
            if (lane == 0) s.warp[warp] = a;
            __syncthreads();
            a.z = a.d = 0.f;
            for (int w = 0; w < kWarpsLp; ++w) {
                a.z += s.warp[w].z;
                a.d += s.warp[w].d;
            }
        }
    }
    // without a distribution: a NaN, an infinity
    const bool no = slow && (nan || a.m == INFINITY);
    const bool none = !no && a.m == -INFINITY;
    const float ln_z = no || none ? 0.f : logf(a.z);
    const auto log_p = [&](float f) {
        if (no) return nan ? NAN : f - INFINITY;
        if (none) return f;
        if (differences) return (f - a.m) - ln_z;
        // (far below the others the product could overflow, and nothing is lost by the plain difference)
        return f < -2.f * kLarge ? f - fmaf(a.m, kLn2, ln_z) : fmaf(fmaf(f, kLog2e, -a.m), kLn2, -ln_z);
    };
    if (tid == 0) {
        if (p.logp) p.logp[row] = log_p(given);
        if (p.entropy) p.entropy[row] = no ? NAN : none ? 0.f : fmaxf(ln_z - kLn2 * a.d / a.z, 0.f);
    }
    if (p.k > 0) {
        if (slow) top_by_passes<DT>(x, 0, p.V, p.k, s.cand, s.key);
        const int n = slow ? p.k : nb * p.k;
        for (int i = tid; i < n; i += kThreadsLp) {
            const uint64_t kk = slow ? s.cand[i] : s.top[i / p.k][i % p.k];
            if (!kk) continue;
            int r = i;
            if (!slow && nb > 1) {
                r = 0;
                for (int b = 0; b < nb; ++b)
#pragma unroll 8
                    for (int j = 0; j < p.k; ++j) r += s.top[b][j] > kk;
            }
            if (r < p.k) {
                const int v = (int)~(uint32_t)kk;
                p.top_ids[(size_t)row * p.k + r] = v;
                p.top_logp[(size_t)row * p.k + r] = log_p(value_of((uint32_t)(kk >> 32)));
            }
        }
    }
}

// Blocks per row: doubled while there are fewer than 256 of them (1.7 an SM),
// to a portable cluster at most, and while each keeps 16 KB of the row; a block
// costs some 5 us of its own.  Measured with 102400 logits a row, blocks 1, 2,
// 4, 8 (us): 17 rows fp32 14.0, 10.5, 8.5, 8.0; 64 rows bf16 13.6, 10.7, 10.9,
// 13.6; 152 rows 14.2, 12.6, 17.9, 25.6; 608 rows 29.3, 36.6, 53.5, 83.7; 17
// rows of 32000 8.0, 7.3, 7.6, 9.9.
int blocks_per_row(int N, int64_t bytes) {
    int nb = 1;
    while (nb < kMaxCluster && (int64_t)N * nb < 256 && bytes / (2 * nb) >= 16000) nb *= 2;
    return nb;
}

template <int DT>
int launch(const LogprobParams &p, cudaStream_t s) {
    const int nb = blocks_per_row(p.N, (int64_t)p.V * (int64_t)sizeof(typename Elem<DT>::T));
    LogprobParams q = p;
    for (int r0 = 0; r0 < p.N; r0 += 65535) {  // the grid's second dimension
        q.logits = static_cast<const typename Elem<DT>::T *>(p.logits) + (int64_t)r0 * p.stride;
        q.N = p.N - r0 < 65535 ? p.N - r0 : 65535;
        q.ids = p.ids ? p.ids + r0 : nullptr;
        q.logp = p.logp ? p.logp + r0 : nullptr;
        q.entropy = p.entropy ? p.entropy + r0 : nullptr;
        q.top_ids = p.top_ids ? p.top_ids + (size_t)r0 * p.k : nullptr;
        q.top_logp = p.top_logp ? p.top_logp + (size_t)r0 * p.k : nullptr;
        cudaLaunchAttribute attr[2];
        cudaLaunchConfig_t c = latent_config(dim3(nb, q.N), kThreadsLp, 0, s, attr, nb);
        const int st = record_launch(cudaLaunchKernelEx(&c, logprobs_kernel<DT>, q));
        if (st) return st;
    }
    return SPX_OK;
}

}  // namespace

}  // namespace spx

using namespace spx;

extern "C" int spx_token_logprobs(const spx_logprobs_args *a, spx_stream_t stream) {
    if (!a || a->N < 0 || a->V < 1 || a->k < 0 || a->k > a->V) return SPX_ERR_INVALID_ARG;
    if (a->dtype != SPX_F16 && a->dtype != SPX_BF16 && a->dtype != SPX_F32) return SPX_ERR_UNSUPPORTED;
    if (a->k > kMaxTop || a->V > 1 << 30) return SPX_ERR_UNSUPPORTED;
    if (a->N == 0) return SPX_OK;
    if (!a->logits || a->stride < a->V || !a->ids != !a->logp || (a->k > 0) != (a->top_ids != nullptr) ||
        (a->k > 0) != (a->top_logp != nullptr))
        return SPX_ERR_INVALID_ARG;
    const uintptr_t es = a->dtype == SPX_F32 ? 4 : 2;
    if (reinterpret_cast<uintptr_t>(a->logits) % es) return SPX_ERR_INVALID_ARG;
    LogprobParams p{a->logits, a->stride, a->N, a->V, a->k, a->ids, a->logp, a->entropy, a->top_logp, a->top_ids};
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return a->dtype == SPX_F16 ? launch<SPX_F16>(p, s) : a->dtype == SPX_BF16 ? launch<SPX_BF16>(p, s)
                                                                                : launch<SPX_F32>(p, s);
}
