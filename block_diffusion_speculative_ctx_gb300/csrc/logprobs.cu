// Log probabilities of given tokens with entropy, ranks and the likeliest
// alternatives (dflash_token_logprobs), and their gradient by the logits
// (dflash_token_logprobs_grad); include/dflash.h.
//
// Forward, one pass over a row: with a running maximum m,
//   l = sum 2^y, t = sum 2^y y, y = (x - m) log2(e) / T
// give lse = m / T + ln l and the entropy ln l - ln 2 * t / l; a new maximum m' turns
// (l, t) into a (l, t + l d), d = (m - m') log2(e) / T, a = 2^d.  The difference comes
// before the scale, so logits of the type's lowest value stay what they are.
// Ranks: a token's are counted as the tiles go by (x >= the token's logit for ids
// before it, x >= the next value above for ids behind it), four tokens at a time; a
// warp's tile that lies below all of several tokens is passed over (512 fp32 rows, eight
// tokens of the 50 likeliest, 5 alternatives: 67 us; eight of the best 64th: 109; with one token
// the test costs more than it saves, 63 us for 60).
// Alternatives: elements that reach tau, a lower bound of the k-th best, go to a list
// of ids in shared memory.  The first tile gives tau: of the maxima of groups of four
// threads the k-th largest is a bound that k elements reach.  Now and then tau becomes the k-th best of
// the list.  A list that overflows (rows that rise along the vocabulary, rows of one value) is made again
// by a form that holds for any order (candidates_again).  Keys are (logit, lowest
// id), all different.  The tiles go by without a barrier.
// A row is split over the CTAs of a cluster, which push their results into the shared
// memory of its first one: no workspace, no second launch.
// Bound by the issue of instructions: 19 a logit with a rank and alternatives, 11 for
// the sums alone.  Measured (calls in a row): 512 fp32 rows of 151936, one token, 5
// alternatives 60.7 us (76 % of a measured copy's rate; 50.5 us without rank and
// alternatives); one row with 20 alternatives 7.9 us; 64 bf16 rows of 128256 with 8
// tokens and 8 alternatives 19.1 us (the chain of a CTA's four tiles, bootstrap, list, cluster and
// join).  Measured and not kept: ranks counted in integers (comparisons and integer adds share a pipe of half
// rate: 512 rows with eight tokens 149 us); a barrier and a count of candidates a tile (118 us
// for 65), a candidate's logit picked from registers (70 with 20 alternatives for
// 63), sums that clamp only where a tile holds -inf (60 us for the sums alone: registers), three
// CTAs an SM without spills (69).
//
// Backward: one pass, out_v = (sum g_i [t_i = v] - p_v (G + h (z_v + H))) / T with z = x / T - lse; a
// thread's four vectors are under way before the row's tokens are known, which are looked for in the
// CTA's chunk alone.  Bound by HBM: 89.5 us for 512 rows of 151936 in fp32 (102 % of a measured
// copy), 7.1 us for 64 bf16 rows of 128256 (launch and one trip).
#include <math.h>

#include "ops.h"
#include "tcgen05.cuh"

namespace dfl {

namespace {

using tc::add2, tc::ex2, tc::fma2, tc::mul2, tc::pack2, tc::unpack2;

constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;
constexpr float MIN_INVERSE = 1.f / (1 << 20), MAX_INVERSE = 1 << 20;  // of a temperature
constexpr int MAXT = DFLASH_LOGPROBS_MAX_TOKENS, MAXK = DFLASH_LOGPROBS_MAX_TOP;

// max(x, y), NaN where one is.
__device__ __forceinline__ float max_nan(float x, float y) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
    return r;
}
// The G elements of a 16-byte vector.
template <typename T>
__device__ __forceinline__ void widen(const uint4& r, float* x) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (sizeof(T) == 4) {
            x[i] = __uint_as_float(w[i]);
        } else {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
}

// ------------------------------------------------------------------------------ forward
constexpr int E = 16;  // elements of a thread in a tile
constexpr int MAXC = 8;
constexpr int LIST = 512;            // candidates of the list
constexpr int NOWHERE = 0x60000000;  // id of an element that is none
constexpr uint64_t ABOVE_NOTHING = 0x0080000000000000ull;  // the smallest key of a token above -inf
constexpr int CAP = 4096;  // of the list of a slice that overflows the short one: candidates,
constexpr int MANY = 128;  // threads of a tile that may add to it

struct Part {  // what a CTA hands to the cluster's first
    float3 sums;  // m, l, t
    int ahead[MAXT];
    uint64_t best[MAXK];
};
template <int NT>
struct Shared {
    Part part, in[MAXC];
    float xt[MAXT];
    int id[MAXT];
    float3 red[NT / 32];
    int n_cand, n_keep, below;
    float tau_v;
    uint64_t tau;
    alignas(16) uint64_t group[NT / 4];
    uint64_t keep[MAXK];
};
constexpr size_t LIST_BYTES = (CAP + 8) * 8;  // dynamic shared memory of the kernels with alternatives

__device__ __forceinline__ uint64_t key_of(float x, int id) { return argmax_key(x + 0.f, (uint32_t)id); }  // (-0 is 0)
__device__ __forceinline__ float key_value(uint64_t k) {
    const uint32_t u = (uint32_t)(k >> 32);
    return __uint_as_float(u & 0x80000000u ? u & 0x7FFFFFFFu : ~u);
}
// The next value above x of T's (-0 is 0; NaN above +inf).
template <typename T>
__device__ __forceinline__ float next_above(float x) {
    constexpr int STEP = sizeof(T) == 4 ? 1 : 1 << 16;
    const int u = __float_as_int(x + 0.f);
    return __int_as_float(u >= 0 ? u + STEP : u - STEP);
}
__device__ __forceinline__ float one_if_ge(float x, float y) {  // x >= y ? 1 : 0
    float r;
    asm("set.ge.f32.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
    return r;
}
// Keys of list[0 .. n) above `mine`; list is 16-byte aligned and list[n] is 0 where n is odd.
__device__ __forceinline__ int count_above(const uint64_t* list, int n, uint64_t mine) {
    int c = 0;
#pragma unroll 4
    for (int j = 0; j < n; j += 2) {
        const ulonglong2 y = *reinterpret_cast<const ulonglong2*>(list + j);
        c += (y.x > mine) + (y.y > mine);
    }
    return c;
}
// The same by four neighbouring threads, to each of them; list[n .. n + 8) is 0.
__device__ __forceinline__ int count_above4(const uint64_t* list, int n, uint64_t mine) {
    int c = 0;
#pragma unroll 2
    for (int j = 2 * (threadIdx.x & 3); j < n; j += 8) {
        const ulonglong2 y = *reinterpret_cast<const ulonglong2*>(list + j);
        c += (y.x > mine) + (y.y > mine);
    }
    c += __shfl_xor_sync(0xffffffffu, c, 1);
    return c + __shfl_xor_sync(0xffffffffu, c, 2);
}
__device__ __forceinline__ void st_first(uint32_t* local, uint32_t v) {  // to the same place in the cluster's first CTA
    uint32_t remote;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(remote) : "r"(tc::smem_u32(local)));
    asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(remote), "r"(v) : "memory");
}

// A CTA's part of a row: tokens before the first aligned vector and behind the last one are an extra tile of the last CTA's.
template <typename T, int NT>
struct Slice {
    static constexpr int G = 16 / (int)sizeof(T), NV = E / G;
    const T* X;
    int head, vecs, left, v0, v1, whole, full, tiles;
    __device__ __forceinline__ Slice(const T* row, int vocab, int rank, int parts) : X(row) {
        head = min(vocab, (int)((16 - ((uintptr_t)X & 15)) & 15) / (int)sizeof(T));
        vecs = (vocab - head) / G;
        left = vocab - vecs * G;
        const int per = (vecs + parts - 1) / parts;
        v0 = min(vecs, rank * per);
        v1 = min(vecs, v0 + per);
        whole = (v1 - v0) / (NT * NV);
        full = (v1 - v0 + NT * NV - 1) / (NT * NV);
        tiles = full + (rank == parts - 1 && left > 0);
    }
    // this thread's elements of tile `it` (-inf where there are none)
    __device__ __forceinline__ void load(int it, uint4 (&r)[NV]) const {
        const int tid = threadIdx.x, at = v0 + it * NV * NT + tid;
        const uint4* p = reinterpret_cast<const uint4*>(X + head) + at;
        if (it < whole) {
#pragma unroll
            for (int i = 0; i < NV; ++i) r[i] = __ldcs(p + i * NT);
            return;
        }
        const uint32_t NONE = sizeof(T) == 4 ? 0xFF800000u : 0xFF80FF80u;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            r[i] = make_uint4(NONE, NONE, NONE, NONE);
            if (it < full && at + i * NT < v1) r[i] = __ldcs(p + i * NT);
        }
        if (it == full && it < tiles && tid < left) {
            const T x = X[tid < head ? tid : tid + vecs * G];
            if constexpr (sizeof(T) == 4) r[0].x = __float_as_uint(to_f32(x));
            else r[0].x = 0xFF800000u | __float_as_uint(to_f32(x)) >> 16;
        }
    }
    __device__ __forceinline__ int first_id(int it) const { return head + (v0 + it * NV * NT) * G; }
    // id of element e of tile `it`
    __device__ __forceinline__ int id(int it, int e) const {
        const int tid = threadIdx.x;
        if (it == full) return e == 0 && tid < left ? (tid < head ? tid : tid + vecs * G) : NOWHERE;
        return first_id(it) + ((e / G) * NT + tid) * G + e % G;
    }
};

// The list's k best keys alone (n > k of them are in it), its k-th best as the new tau.  By all threads; the k-th key is
// found bit by bit.
template <int NT>
__device__ __noinline__ void keep_best(Shared<NT>& S, uint64_t* cand, int n, int k) {
    const int tid = threadIdx.x;
    uint64_t kth = 0;
#pragma unroll 1
    for (int bit = 63; bit >= 0; --bit) {
        const uint64_t at = kth | 1ull << bit;
        if (tid == 0) S.below = 0;
        __syncthreads();
        int c = 0;
        for (int i = tid; i < n; i += NT) c += cand[i] >= at;
        c = __reduce_add_sync(0xffffffffu, c);
        if ((tid & 31) == 0 && c) atomicAdd(&S.below, c);
        __syncthreads();
        if (S.below >= k) kth = at;
        __syncthreads();
    }
    if (tid == 0) S.n_keep = 0;
    __syncthreads();
    for (int i = tid; i < n; i += NT)
        if (cand[i] >= kth) S.keep[atomicAdd(&S.n_keep, 1)] = cand[i];
    __syncthreads();
    if (tid < k) cand[tid] = S.keep[tid];
    if (tid == 0) {
        S.n_cand = k;
        S.tau = kth;
    }
    __syncthreads();
}

// The candidates of a slice that has overflowed the short list, from its beginning, into the long one: its k best keys (or
// all that it has), S.n_cand of them.  Before a tile could fill the list tau, now a key, is raised (where more than MANY threads
// of a tile reach it: to the k-th largest of the maxima of groups of four threads, which at most 4 k threads reach) and the list
// cut to the k best; keys are all different, so rows in any order and of any ties fit.  For rows whose logits rise along the
// vocabulary, or are all alike.
template <typename T, int NT>
__device__ __noinline__ void candidates_again(Shared<NT>& S, uint64_t* cand, const Slice<T, NT>& sl, int k) {
    const int tid = threadIdx.x;
    __syncthreads();
    if (tid == 0) {
        S.n_cand = 0;
        S.tau = ABOVE_NOTHING;
    }
    __syncthreads();
    uint64_t tau = ABOVE_NOTHING;
    float tau_v = key_value(tau);
    int room = CAP;  // entries that are surely free
#pragma unroll 1
    for (int it = 0; it < sl.tiles; ++it) {
        uint4 r[Slice<T, NT>::NV];
        float x[E];
        sl.load(it, r);
#pragma unroll
        for (int i = 0; i < Slice<T, NT>::NV; ++i) widen<T>(r[i], x + i * Slice<T, NT>::G);
        float tm = x[0];
#pragma unroll
        for (int e = 1; e < E; ++e) tm = fmaxf(tm, x[e]);
        int n = __syncthreads_count(tm >= tau_v);
        if (n > MANY) {
            uint64_t key = 0;
            if (tm >= tau_v) {
                int at = 0;
#pragma unroll
                for (int e = E - 1; e >= 0; --e)
                    if (x[e] == tm) at = e;
                key = key_of(tm, sl.id(it, at));
            }
#pragma unroll
            for (int o = 1; o < 4; o <<= 1) {
                const uint64_t y = __shfl_xor_sync(0xffffffffu, key, o);
                key = y > key ? y : key;
            }
            if (tid % 4 == 0) S.group[tid / 4] = key;
            __syncthreads();
            if (tid < NT / 4) {
                const uint64_t mine = S.group[tid];
                if (mine > tau && count_above(S.group, NT / 4, mine) == k - 1) S.tau = mine;
            }
            __syncthreads();
            tau = S.tau;
            tau_v = key_value(tau);
            n = MANY;
        }
        if (tm >= tau_v) {
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (x[e] >= tau_v) {
                    const uint64_t key = key_of(x[e], sl.id(it, e));
                    if (key >= tau) {
                        const int at = atomicAdd(&S.n_cand, 1);
                        if (at < CAP) cand[at] = key;
                    }
                }
        }
        room -= E * n;
        if (room < E * MANY) {
            __syncthreads();
            const int have = min(S.n_cand, CAP);
            __syncthreads();
            room = CAP - have;
            if (room < CAP / 2) {
                keep_best<NT>(S, cand, have, k);
                tau = S.tau;
                tau_v = key_value(tau);
                room = CAP - k;
            }
        }
    }
    __syncthreads();
    const int have = min(S.n_cand, CAP);
    __syncthreads();
    if (have > k) keep_best<NT>(S, cand, have, k);
}

template <typename T, bool TOP, int NT>
__global__ void __launch_bounds__(NT, 1024 / NT) logprobs_kernel(dflash_logprobs_args a, int parts) {
    constexpr int G = 16 / (int)sizeof(T), NV = E / G, WARPS = NT / 32, GROUPS = NT / 4;
    __shared__ Shared<NT> S;
    extern __shared__ __align__(16) uint64_t list[];  // (TOP) keys of the list,
    int* ids = reinterpret_cast<int*>(list + LIST + 8);  // and their ids
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const long long row = blockIdx.x;
    const int rank = parts > 1 ? (int)tc::cluster_rank() : 0;
    // (its end: the first CTA's shared memory is there to be written to)
    if (parts > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    const Slice<T, NT> sl(reinterpret_cast<const T*>(a.logits) + row * a.ld_logits, a.vocab, rank, parts);
    pdl_wait();
    pdl_trigger();
    uint4 next[NV];
    sl.load(0, next);

    // (seen by all behind the first tile's barrier)
    if (tid < MAXT) {
        int t = -1;
        float x = 0.f;
        if (tid < a.n) {
            t = a.tokens[row * a.n + tid];
            if (t < 0 || t >= a.vocab) t = -1;
            else x = to_f32(sl.X[t]);
        }
        S.id[tid] = t;
        S.xt[tid] = x;
        S.part.ahead[tid] = 0;
        S.part.best[tid] = 0;
    }
    static_assert(MAXT == MAXK, "one thread for both");
    if (tid == 0) {
        S.n_cand = 0;
        S.tau_v = -INFINITY;
    }

    const float c = a.inv_temperature * LOG2E;
    const uint64_t c2 = pack2(c, c);
    float m = -INFINITY, l = 0.f, t = 0.f;
    int my_id = -1, my_ahead = 0;  // lane's token, the warp's elements ahead of it (of one token: the lane's), and its logit
    float my_xt = 0.f, lowest = INFINITY;  // (the lowest of the tokens' logits: a warp's elements below it are ahead of none)
    float tau_v = -INFINITY;  // candidates are as large (-inf: not known yet)
    int refresh = 2;
    // f(its key, the keys above it) for each of the list's n keys, by all threads, four a key; ends without a barrier
    auto rank_list = [&](int n, auto&& f) {
        for (int i0 = 0; i0 + 8 * warp < n; i0 += NT / 4) {
            const uint64_t mine = list[min(i0 + tid / 4, n)];
            const int above = count_above4(list, n, mine);
            if (mine && (tid & 3) == 0) f(mine, above);
        }
    };
    int keyed = 0;  // of the list, keys; from there on, ids
    auto make_keys = [&](int n) {
        for (int i = keyed + tid; i < n; i += NT) list[i] = key_of(to_f32(sl.X[ids[i]]), ids[i]);
        if (tid < 8) list[n + tid] = 0;
        keyed = n;
    };
#pragma unroll 1
    for (int it = 0; it < sl.tiles; ++it) {
        float x[E];
        uint4 raw[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            raw[i] = next[i];
            widen<T>(next[i], x + i * G);
        }
        sl.load(it + 1, next);

        // ---- statistics
        float tm = fmaxf(x[0], x[1]);
#pragma unroll
        for (int e = 2; e < E; e += 2) tm = fmaxf(fmaxf(tm, x[e]), x[e + 1]);
        if (tm > m) {
            const float d = (m - tm) * c, al = ex2(d);
            t = m == -INFINITY ? 0.f : al * fmaf(l, max_nan(d, -1000.f), t);
            l *= al;
            m = tm;
        }
        const float ref = m == -INFINITY ? 0.f : -m;
        const uint64_t ref2 = pack2(ref, ref);
        {
            uint64_t l2[2] = {0ull, 0ull}, t2[2] = {0ull, 0ull};
#pragma unroll
            for (int e = 0; e < E; e += 2) {
                float y0, y1;
                unpack2(mul2(add2(pack2(x[e], x[e + 1]), ref2), c2), y0, y1);
                y0 = max_nan(y0, -1000.f);  // (2^y y = 0 for a token at -inf)
                y1 = max_nan(y1, -1000.f);
                const uint64_t p2 = pack2(ex2(y0), ex2(y1));
                l2[(e >> 1) & 1] = add2(l2[(e >> 1) & 1], p2);
                t2[(e >> 1) & 1] = fma2(p2, pack2(y0, y1), t2[(e >> 1) & 1]);
            }
            float s0, s1;
            unpack2(add2(l2[0], l2[1]), s0, s1);
            l += s0 + s1;
            unpack2(add2(t2[0], t2[1]), s0, s1);
            t += s0 + s1;
        }

        // ---- a first tau, from the first tile that holds enough tokens (tau_v is the CTA's): among the maxima of the groups of
        // four threads the k-th largest, which k elements reach
        if (TOP && tau_v == -INFINITY) {
            float* group = reinterpret_cast<float*>(S.group);
            float g = fmaxf(tm, __shfl_xor_sync(0xffffffffu, tm, 1));
            g = fmaxf(g, __shfl_xor_sync(0xffffffffu, g, 2));
            if (tid % 4 == 0) group[tid / 4] = g;
            __syncthreads();
            int n = 0;  // groups above, and 2^16 times those as large
#pragma unroll 4
            for (int j = 4 * (tid & 3); j < GROUPS; j += 16) {
                const float4 y = *reinterpret_cast<const float4*>(group + j);
                n += (y.x > g) + (y.y > g) + (y.z > g) + (y.w > g);
                n += ((y.x == g) + (y.y == g) + (y.z == g) + (y.w == g)) << 16;
            }
            n += __shfl_xor_sync(0xffffffffu, n, 1);
            n += __shfl_xor_sync(0xffffffffu, n, 2);
            const int above = n & 0xFFFF;
            if (tid % 4 == 0 && above < a.k && above + (n >> 16) >= a.k) S.tau_v = g;  // (the same value from each that writes)
            __syncthreads();
            tau_v = S.tau_v;
        } else if (!TOP && it == 0) {
            __syncthreads();
        }

        // ---- ranks: of the ids behind the token's those of a larger logit count, of the ids before it also those of the same
        if (a.ranks && it == 0) {
            if (lane < a.n || a.n == 1) {
                my_id = S.id[a.n == 1 ? 0 : lane];
                my_xt = S.xt[a.n == 1 ? 0 : lane];
            }
            lowest = -warp_max(my_id < 0 ? -INFINITY : -my_xt);
        }
        if (a.ranks && (a.n == 1 || __any_sync(0xffffffffu, tm >= lowest))) {
            const int first = sl.first_id(it);
            // lane i's count of ahead += the warp's
            auto credit = [&](int i, int n) { my_ahead += lane == i ? n : 0; };
            // this thread's elements as large as least(j), j their vector (counted in floating point: comparisons have their pipe to
            // themselves)
            auto as_large = [&](auto&& least) {
                if constexpr (sizeof(T) == 4) {
                    uint64_t n2[2] = {0ull, 0ull};
#pragma unroll
                    for (int j = 0; j < NV; ++j) {
                        const float y = least(j);
#pragma unroll
                        for (int e = 0; e < G; e += 2)
                            n2[e >> 1] = add2(n2[e >> 1], pack2(one_if_ge(x[j * G + e], y), one_if_ge(x[j * G + e + 1], y)));
                    }
                    float lo, hi;
                    unpack2(add2(n2[0], n2[1]), lo, hi);
                    return __float2int_rn(lo + hi);
                } else {
                    // (0 or 1 in bf16: sums up to 256 are exact)
                    __nv_bfloat162 n2[2] = {__float2bfloat162_rn(0.f), __float2bfloat162_rn(0.f)};
#pragma unroll
                    for (int j = 0; j < NV; ++j) {
                        const __nv_bfloat162 y = __float2bfloat162_rn(least(j));
                        const uint32_t w[4] = {raw[j].x, raw[j].y, raw[j].z, raw[j].w};
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            n2[k & 1] = __hadd2(n2[k & 1], __hge2(*reinterpret_cast<const __nv_bfloat162*>(&w[k]), y));
                    }
                    n2[0] = __hadd2(n2[0], n2[1]);
                    return __float2int_rn(__low2float(n2[0]) + __high2float(n2[0]));
                }
            };
            if (it == sl.full) {  // single tokens: ids on both sides of any
                const int id = sl.id(it, 0);
                for (int i = 0; i < a.n; ++i) {
                    const float xt = __shfl_sync(0xffffffffu, my_xt, i);
                    const int at = __shfl_sync(0xffffffffu, my_id, i);
                    credit(i, __popc(__ballot_sync(0xffffffffu, x[0] > xt || (x[0] == xt && id < at))));
                }
            } else {
                const bool before = my_id >= first + NT * E;  // lane's token lies behind the tile
                // A token in the tile has ids on both sides; and elements that are none, -inf, are not as large as a token at -inf
                // behind them.
                const bool mixed = (unsigned)(my_id - first) < (unsigned)(NT * E) || (before && it >= sl.whole && my_xt == -INFINITY);
                const float my_least = before ? my_xt : next_above<T>(my_xt);
                // the same of the token at `at` by vectors: each lies before it, behind it or holds it
                auto of_mixed = [&](int at, float xt) {
                    constexpr int STEP = NT * G;  // ids from a thread's vector to its next
                    const float above = next_above<T>(xt);
                    const int t = at - first - tid * G;
                    int n = as_large([&](int j) { return t >= j * STEP + G ? xt : above; });
                    if ((t & (STEP - 1)) < G && (unsigned)t < NV * STEP) {
#pragma unroll
                        for (int j = 0; j < NV; ++j)
#pragma unroll
                            for (int e = 0; e < G; ++e) n += t > j * STEP + e && t < j * STEP + G && x[j * G + e] == xt;
                    }
                    if (it >= sl.whole && xt == -INFINITY) {
#pragma unroll
                        for (int j = 0; j < NV; ++j)
                            if (sl.v0 + (it * NV + j) * NT + tid >= sl.v1) n -= min(max(t - j * STEP, 0), G);
                    }
                    return n;
                };
                if (a.n == 1) {  // (every lane holds the one token; its counts are joined at the end)
                    my_ahead += mixed ? of_mixed(my_id, my_xt) : as_large([&](int) { return my_least; });
                } else {
                    const uint32_t some = __ballot_sync(0xffffffffu, mixed);
#pragma unroll 1
                    for (int q = 0; q < a.n;) {
                        if (q + 4 > a.n || some >> q & 15u) {
                            const int n = of_mixed(__shfl_sync(0xffffffffu, my_id, q), __shfl_sync(0xffffffffu, my_xt, q));
                            credit(q, __reduce_add_sync(0xffffffffu, n));
                            ++q;
                            continue;
                        }
                        uint32_t n[2] = {0u, 0u};  // two tokens' counts each
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float least = __shfl_sync(0xffffffffu, my_least, q + i);
                            n[i / 2] += (uint32_t)as_large([&](int) { return least; }) << 16 * (i & 1);
                        }
#pragma unroll
                        for (int i = 0; i < 2; ++i) n[i] = __reduce_add_sync(0xffffffffu, n[i]);
#pragma unroll
                        for (int i = 0; i < 4; ++i) credit(q + i, (int)(n[i / 2] >> 16 * (i & 1) & 0xFFFFu));
                        q += 4;
                    }
                }
            }
        }

        // ---- candidates; tau becomes the k-th best of the list now and then
        if (TOP) {
            const float least_v = fmaxf(tau_v, -3.402823466e38f);  // (-inf is none)
            if (tm >= least_v) {
                uint32_t on = 0;
#pragma unroll
                for (int e = 0; e < E; ++e)
                    if (x[e] >= least_v) on |= 1u << e;
                int at = atomicAdd(&S.n_cand, __popc(on));
                for (; on; on &= on - 1, ++at) {
                    if (at < LIST) ids[at] = sl.id(it, __ffs(on) - 1);
                }
            }
            if (it == refresh && 3 * it < sl.tiles) {  // (behind 3, 9, 33 .. tiles of at least 7, 25, 97 ..)
                refresh *= 4;
                __syncthreads();
                const int n = S.n_cand;
                if (n >= a.k && n <= LIST) {
                    make_keys(n);
                    __syncthreads();
                    rank_list(n, [&](uint64_t key, int above) {
                        if (above == a.k - 1) S.tau_v = key_value(key);
                    });
                }
                __syncthreads();
                tau_v = S.tau_v;
            }
        }
    }

    if (a.ranks) {
        if (a.n == 1) {
            my_ahead = __reduce_add_sync(0xffffffffu, my_ahead);
            if (lane) my_ahead = 0;
        }
        if (my_ahead) atomicAdd(&S.part.ahead[lane], my_ahead);
    }

    // ---- the CTA's results (the list's logits come while the warps join their sums)
    int n = 0;
    if (TOP) {
        __syncthreads();
        n = S.n_cand;
        if (n <= LIST) make_keys(n);
    }
    {
        const float M = warp_max(m);
        const float al = m == -INFINITY ? 0.f : ex2((m - M) * c);
        t = m == -INFINITY ? 0.f : al * fmaf(l, max_nan((m - M) * c, -1000.f), t);
        l = warp_sum(l * al);
        t = warp_sum(t);
        if (lane == 0) S.red[warp] = make_float3(M, l, t);
    }
    __syncthreads();
    // sums of `count` places, the same in every thread
    auto join = [&](int count, auto&& at) {
        float3 y[MAXC];
        float M = -INFINITY, L = 0.f, Z = 0.f;
#pragma unroll
        for (int i0 = 0; i0 < NT / 32; i0 += MAXC) {
            if (i0 >= count) break;
            const float before = M;
#pragma unroll
            for (int i = 0; i < MAXC; ++i) {
                y[i] = i0 + i < count ? at(i0 + i) : make_float3(-INFINITY, 0.f, 0.f);
                M = fmaxf(M, y[i].x);
            }
            auto add = [&](float m0, float l0, float t0) {
                const float d = (m0 - M) * c, al = m0 == -INFINITY ? 0.f : ex2(d);
                L = fmaf(l0, al, L);
                if (m0 != -INFINITY) Z = fmaf(al, fmaf(l0, max_nan(d, -1000.f), t0), Z);
            };
            const float l0 = L, z0 = Z;
            L = Z = 0.f;
            add(before, l0, z0);
#pragma unroll
            for (int i = 0; i < MAXC; ++i) add(y[i].x, y[i].y, y[i].z);
        }
        return make_float3(M, L, Z);
    };
    if (tid == NT - 1) S.part.sums = join(WARPS, [&](int i) { return S.red[i]; });
    if (TOP) {
        if (n > LIST) {
            candidates_again<T, NT>(S, list, sl, a.k);
            n = S.n_cand;
            if (tid < 8) list[n + tid] = 0;
            __syncthreads();
        }
        rank_list(n, [&](uint64_t key, int above) {
            if (above < a.k) S.part.best[above] = key;
        });
    }
    __syncthreads();
    constexpr int WORDS = sizeof(Part) / 4;
    static_assert(WORDS <= NT, "a thread a word");
    if (parts > 1) {
        asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
        if (tid < WORDS) st_first(reinterpret_cast<uint32_t*>(&S.in[rank]) + tid, reinterpret_cast<const uint32_t*>(&S.part)[tid]);
        __syncwarp();
        tc::cluster_sync();
        if (rank != 0) return;
    }
    const Part* in = parts > 1 ? S.in : &S.part;

    // ---- the row's
    const float3 sums = join(parts, [&](int i) { return in[i].sums; });
    m = sums.x;
    const bool bad = isnan(sums.y) || m == INFINITY, none = sums.y == 0.f;
    const float ln_l = logf(sums.y);
    auto logprob = [&](float x) { return bad ? NAN : x == -INFINITY ? -INFINITY : (x - m) * a.inv_temperature - ln_l; };
    if (tid == NT - 1) {
        if (a.lse) a.lse[row] = bad ? NAN : none ? -INFINITY : fmaf(m, a.inv_temperature, ln_l);
        if (a.lse_parts) *reinterpret_cast<float2*>(a.lse_parts + 2 * row) = bad ? make_float2(NAN, NAN) : make_float2(m, ln_l);
        if (a.entropy) a.entropy[row] = bad ? NAN : none ? 0.f : ln_l - LN2 * (sums.z / sums.y);
    }
    if (tid < a.n) {
        const int at = S.id[tid];
        int ahead = 0;
        for (int q = 0; q < parts; ++q) ahead += in[q].ahead[tid];
        if (a.logprobs) a.logprobs[row * a.n + tid] = at < 0 ? 0.f : logprob(S.xt[tid]);
        if (a.ranks) a.ranks[row * a.n + tid] = at < 0 || bad ? -1 : ahead;
    }
    if (TOP) {
        // The lists are sorted (0 behind): an alternative's place is the number of keys above it in each of them.
        const int q = tid / MAXK, i = tid % MAXK;
        const uint64_t mine = q < parts && i < a.k ? in[q].best[i] : 0;
        int found = 0;  // alternatives of the row (k or more, or, where it has fewer tokens, all)
        for (int s = 0; s < parts; ++s) found += __popc(__ballot_sync(0xffffffffu, in[s].best[lane] != 0));
        if (tid < a.k && (bad || tid >= found)) {
            if (a.top_ids) a.top_ids[row * a.k + tid] = -1;
            if (a.top_logprobs) a.top_logprobs[row * a.k + tid] = bad ? NAN : -INFINITY;
        }
        if (mine && !bad) {
            int above = 0;
#pragma unroll
            for (int s = 0; s < MAXC; ++s) {
                const uint64_t* y = in[min(s, parts - 1)].best;
                int at = 0;
#pragma unroll
                for (int step = MAXK / 2; step; step >>= 1) at += y[at + step - 1] > mine ? step : 0;
                at += y[at] > mine;
                above += s < parts ? at : 0;
            }
            if (above < a.k) {
                if (a.top_ids) a.top_ids[row * a.k + above] = (int)argmax_key_index(mine);
                if (a.top_logprobs) a.top_logprobs[row * a.k + above] = logprob(key_value(mine));
            }
        }
    }
}

template <typename T, int NT>
void forward(const Launch& L, const dflash_logprobs_args& a, int parts) {
    static_assert(MAXC * MAXK <= NT, "a thread for every part's every alternative");
    const bool top = a.k > 0 && (a.top_ids || a.top_logprobs);
    if (top) launch_k(L, logprobs_kernel<T, true, NT>, dim3(a.rows, 1, parts), dim3(NT), LIST_BYTES, parts, a, parts);
    else launch_k(L, logprobs_kernel<T, false, NT>, dim3(a.rows, 1, parts), dim3(NT), 0, parts, a, parts);
}
// A row goes to so many CTAs that there are four an SM, if its tiles last, and to wider ones where every CTA has an SM of its own
// (one row with 20 alternatives: 7.8 us, with 256 threads 9.7; without any 5.1 and 5.2).  Measured (graph replay, us; * the rule's),
// one token and five alternatives of fp32 rows of 151936 but where said, in
//                       one    two    four   eight parts
//   one row, 20         30     19.3   13.8   9.7 (wide: 7.8 *)
//   32 rows             27.6   17.7   11.7   9.5 *
//   128 rows            28.6   22.1   21.0   25.4 *
//   256 rows            37.6   34.4   40.2 * 46.8
//   304 rows            39.7   36.1 * 47.1   54.4
//   512 rows            57.6   60.7 * 70.2   86.0
//   512, eight tokens   118    109 *  121    138
//   1024 rows           111 *  114    129
//   64 bf16 rows of 128256, eight tokens and alternatives
//                       40.7   24.6   19.0   19.1 *
// so four an SM suit few rows and several tokens; where rows * parts comes out just below 608 (128, 256 and 512 rows here) half the
// parts would take 5 to 17 % less for one token.
template <typename T>
void forward(const Launch& L, const dflash_logprobs_args& a) {
    const long long tiles = ((long long)a.vocab + 256 * E - 1) / (256 * E);
    int parts = 1;
    while (parts < MAXC && 2 * parts <= tiles && (long long)a.rows * parts < 608) parts *= 2;
    if ((long long)a.rows * parts <= 152 && tiles >= 2 * parts) forward<T, 512>(L, a, parts);
    else forward<T, 256>(L, a, parts);
}

// ----------------------------------------------------------------------------- backward
constexpr int NB = 256, VB = 4;  // threads, 16-byte vectors a thread

template <typename T, bool VECTORS>
__global__ void __launch_bounds__(NB) logprobs_grad_kernel(dflash_logprobs_grad_args a, int chunks) {
    constexpr int G = 16 / (int)sizeof(T);
    const int tid = threadIdx.x, lane = tid & 31;
    const long long row = blockIdx.x / chunks;
    const int chunk = blockIdx.x - (int)row * chunks;
    const T* X = reinterpret_cast<const T*>(a.logits) + row * a.ld_logits;
    T* Y = reinterpret_cast<T*>(a.out) + row * a.ld_out;
    pdl_wait();
    pdl_trigger();
    const int head = VECTORS ? min(a.vocab, (int)((16 - ((uintptr_t)X & 15)) & 15) / (int)sizeof(T)) : 0;
    const int vecs = VECTORS ? (a.vocab - head) / G : 0, left = a.vocab - vecs * G;
    const int v0 = chunk * NB * VB;
    uint4 r[VB];
#pragma unroll
    for (int i = 0; i < VB; ++i) {
        const int v = v0 + i * NB + tid;
        r[i] = make_uint4(0u, 0u, 0u, 0u);
        if (VECTORS && v < vecs) r[i] = __ldcs(reinterpret_cast<const uint4*>(X + head) + v);
    }
    // lane i: the row's i-th token and its gradient
    int t = -1;
    float g = 0.f;
    if (lane < a.n) {
        t = a.tokens[row * a.n + lane];
        if (t < 0 || t >= a.vocab) t = -1;
        else g = a.grad_logprobs[row * a.n + lane];
    }
    const float h = a.grad_entropy ? a.grad_entropy[row] : 0.f, H = a.entropy ? a.entropy[row] : 0.f;
    const float sum = warp_sum(g);
    const bool zero = !__any_sync(0xffffffffu, g != 0.f) && h == 0.f;
    float lse, best = 0.f;  // x / T - lse, or with its two parts (x - best) / T - lse
    if (a.lse_parts) {
        const float2 two = *reinterpret_cast<const float2*>(a.lse_parts + 2 * row);
        best = two.x == -INFINITY ? 0.f : two.x;
        lse = two.y;
    } else {
        lse = a.lse[row];
    }
    if (lse == -INFINITY) lse = INFINITY;  // (a row of -inf alone: p = 0)
    // -p (G + h (ln p + H)); ln p below any p that is not 0
    auto slope = [&](float x) {
        const float z = max_nan(fmaf(x - best, a.inv_temperature, -lse), -1000.f);
        return -ex2(z * LOG2E) * fmaf(h, z + H, sum);
    };
    if (VECTORS) {
        const int lo = head + v0 * G, hi = lo + NB * VB * G;
        const uint32_t mine = __ballot_sync(0xffffffffu, t >= lo && t < hi);  // tokens of this chunk
#pragma unroll
        for (int i = 0; i < VB; ++i) {
            const int v = v0 + i * NB + tid;
            float x[G];
            widen<T>(r[i], x);
#pragma unroll
            for (int e = 0; e < G; ++e) x[e] = zero ? 0.f : slope(x[e]);
            for (uint32_t w = mine; w; w &= w - 1) {
                const int src = __ffs(w) - 1, at = __shfl_sync(0xffffffffu, t, src) - (head + v * G);
                const float gi = __shfl_sync(0xffffffffu, g, src);
#pragma unroll
                for (int e = 0; e < G; ++e)
                    if (at == e) x[e] += gi;
            }
            uint32_t o[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                if (sizeof(T) == 4) o[q] = __float_as_uint(x[q] * a.inv_temperature);
                else o[q] = tc::pack2_bf16(x[2 * q] * a.inv_temperature, x[2 * q + 1] * a.inv_temperature);
            }
            if (v < vecs) __stcs(reinterpret_cast<uint4*>(Y + head) + v, make_uint4(o[0], o[1], o[2], o[3]));
        }
    }
    // single tokens: those before the first vector and behind the last (with VECTORS of the last chunk's first warp)
    const int begin = VECTORS ? (chunk == chunks - 1 && tid < 32 ? 0 : left) : chunk * NB * VB,
              end = VECTORS ? left : min(left, begin + NB * VB);
    for (int k0 = begin; k0 < end; k0 += VECTORS ? 32 : NB) {
        const int k = k0 + (VECTORS ? lane : tid);
        const int id = k < end ? (VECTORS && k >= head ? k + vecs * G : k) : -2;
        float x = id >= 0 && !zero ? slope(to_f32(X[id])) : 0.f;
        for (int i = 0; i < a.n; ++i) {
            const int at = __shfl_sync(0xffffffffu, t, i);
            const float gi = __shfl_sync(0xffffffffu, g, i);
            if (at == id) x += gi;
        }
        if (id >= 0) Y[id] = from_f32<T>(x * a.inv_temperature);
    }
}

template <typename T>
void backward(const Launch& L, const dflash_logprobs_grad_args& a) {
    const int G = 16 / (int)sizeof(T);
    // vectors where logits and gradient lie alike in every row
    const bool alike = ((uintptr_t)a.logits - (uintptr_t)a.out) % 16 == 0 && (a.rows == 1 || (a.ld_logits - a.ld_out) % G == 0);
    const int step = NB * VB * (alike ? G : 1), chunks = (a.vocab + step - 1) / step;
    const dim3 grid((unsigned)((long long)a.rows * chunks));
    if (alike) launch_k(L, logprobs_grad_kernel<T, true>, grid, dim3(NB), 0, 1, a, chunks);
    else launch_k(L, logprobs_grad_kernel<T, false>, grid, dim3(NB), 0, 1, a, chunks);
}

}  // namespace

}  // namespace dfl

using namespace dfl;

extern "C" dflash_status dflash_token_logprobs(const dflash_logprobs_args* p, void* cuda_stream) {
    if (!p) return refuse("token_logprobs: args is NULL");
    const dflash_logprobs_args& a = *p;
    if (a.dtype != DFLASH_DTYPE_F32 && a.dtype != DFLASH_DTYPE_BF16) return refuse("token_logprobs: dtype must be F32 or BF16");
    if (a.rows < 0 || a.rows > (1 << 20)) return refuse("token_logprobs: rows outside [0, 2^20]");
    if (a.vocab < 1 || a.vocab > (1 << 30)) return refuse("token_logprobs: vocab outside [1, 2^30]");
    if (a.n < 0 || a.n > MAXT) return refuse("token_logprobs: n outside [0, 32]");
    if (a.k < 0 || a.k > MAXK) return refuse("token_logprobs: k outside [0, 32]");
    if (!(a.inv_temperature >= MIN_INVERSE && a.inv_temperature <= MAX_INVERSE))
        return refuse("token_logprobs: inv_temperature outside [2^-20, 2^20]");
    if ((a.rows > 0 && !a.logits) || (a.rows > 0 && a.n > 0 && !a.tokens)) return refuse("token_logprobs: NULL argument");
    if ((uintptr_t)a.logits % (a.dtype == DFLASH_DTYPE_BF16 ? 2 : 4)) return refuse("token_logprobs: logits is not aligned to its type");
    if ((uintptr_t)a.lse_parts % 8) return refuse("token_logprobs: lse_parts is not aligned to 8 bytes");
    if (a.ld_logits < a.vocab) return refuse("token_logprobs: the row stride is smaller than vocab");
    if (a.rows == 0) return DFLASH_OK;
    return queue(cuda_stream, "token_logprobs: launch failed", [&](const Launch& L) {
        if (a.dtype == DFLASH_DTYPE_BF16) forward<bf16>(L, a);
        else forward<float>(L, a);
    });
}

extern "C" dflash_status dflash_token_logprobs_grad(const dflash_logprobs_grad_args* p, void* cuda_stream) {
    if (!p) return refuse("token_logprobs_grad: args is NULL");
    const dflash_logprobs_grad_args& a = *p;
    if (a.dtype != DFLASH_DTYPE_F32 && a.dtype != DFLASH_DTYPE_BF16)
        return refuse("token_logprobs_grad: dtype must be F32 or BF16");
    if (a.rows < 0 || a.rows > (1 << 20)) return refuse("token_logprobs_grad: rows outside [0, 2^20]");
    if (a.vocab < 1 || a.vocab > (1 << 30)) return refuse("token_logprobs_grad: vocab outside [1, 2^30]");
    if (a.n < 0 || a.n > MAXT) return refuse("token_logprobs_grad: n outside [0, 32]");
    if (!(a.inv_temperature >= MIN_INVERSE && a.inv_temperature <= MAX_INVERSE))
        return refuse("token_logprobs_grad: inv_temperature outside [2^-20, 2^20]");
    if (a.reserved != 0) return refuse("token_logprobs_grad: reserved must be 0");
    if (a.rows > 0 && (!a.logits || !a.out || (!a.lse && !a.lse_parts) || (a.n > 0 && (!a.tokens || !a.grad_logprobs)) || (a.grad_entropy && !a.entropy)))
        return refuse("token_logprobs_grad: NULL argument");
    const uintptr_t es = a.dtype == DFLASH_DTYPE_BF16 ? 2 : 4;
    if (((uintptr_t)a.logits | (uintptr_t)a.out) % es) return refuse("token_logprobs_grad: logits or out is not aligned to its type");
    if ((uintptr_t)a.lse_parts % 8) return refuse("token_logprobs_grad: lse_parts is not aligned to 8 bytes");
    if (a.ld_logits < a.vocab || a.ld_out < a.vocab) return refuse("token_logprobs_grad: a row stride is smaller than vocab");
    if (a.out == a.logits && a.ld_out != a.ld_logits && a.rows > 1) return refuse("token_logprobs_grad: in place needs one row stride");
    const long long chunk = NB * VB;
    if ((long long)a.rows * ((a.vocab + chunk - 1) / chunk) >= (1ll << 31)) return refuse("token_logprobs_grad: rows * vocab is too large");
    if (a.rows == 0) return DFLASH_OK;
    return queue(cuda_stream, "token_logprobs_grad: launch failed", [&](const Launch& L) {
        if (a.dtype == DFLASH_DTYPE_BF16) backward<bf16>(L, a);
        else backward<float>(L, a);
    });
}
