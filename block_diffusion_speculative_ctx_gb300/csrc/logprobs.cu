// Log probabilities of given tokens with entropy, ranks and the likeliest
// alternatives (dflash_token_logprobs), and their gradient by the logits
// (dflash_token_logprobs_grad); include/dflash.h.
//
// Forward, one pass over a row: with a running maximum m,
//   l = sum 2^y, t = sum 2^y y, y = (x - m) log2(e) / T
// give lse = m / T + ln l and the entropy ln l - ln 2 * t / l; a new maximum m' turns
// (l, t) into a (l, t + l d), d = (m - m') log2(e) / T, a = 2^d.  The difference comes
// before the scale, so logits of the type's lowest value stay what they are.  A token's
// rank is counted on the way, in warps that hold a logit as large as its own.
// Alternatives: a tile's elements that reach tau, a lower bound of the k-th best
// so far, go to a list in shared memory.  tau is raised where more than 128 of a
// tile's threads reach it, as in the first tile: among the maxima of 64 groups of four threads the
// k-th largest is a bound that k elements reach, and at most 4 k threads with it.  Keys
// are (logit, lowest id), all different, so ties need no care and rows in any order
// fit the list.
// A row is split over the CTAs of a cluster, whose first one joins their results
// through distributed shared memory: no workspace, no second launch.
// Backward: one pass, out_v = (sum g_i [t_i = v] - p_v (G + h (z_v + H))) / T with z = x / T - lse.
// Bytes: the logits once; the gradient once more.
#include <math.h>

#include "ops.h"
#include "tcgen05.cuh"

namespace dfl {

namespace {

constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;
constexpr int MAXT = DFLASH_LOGPROBS_MAX_TOKENS, MAXK = DFLASH_LOGPROBS_MAX_TOP;

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
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
constexpr int NT = 256, WARPS = NT / 32, E = 16;  // threads; elements of a thread in a tile
constexpr int MAXC = 8;
constexpr int CAP = 4096;      // candidates in the list
constexpr int MANY = 128;      // threads of a tile that may add to it
constexpr int GROUPS = 64;
constexpr int NOWHERE = 0x60000000;  // id of an element that is none
constexpr uint64_t ABOVE_NOTHING = 0x0080000000000000ull;  // the smallest key of a token above -inf

struct Part {  // of a CTA, read by the cluster's first
    float m, l, t;
    int ahead[MAXT];
    uint64_t best[MAXK];
};
struct Shared {
    Part part;
    float xt[MAXT];
    int id[MAXT];
    float red[3][WARPS];
    int n_cand, n_keep, below;
    uint64_t tau;
    uint64_t group[GROUPS];
    uint64_t all[MAXC * MAXK];
};

__device__ __forceinline__ uint64_t key_of(float x, int id) { return argmax_key(x + 0.f, (uint32_t)id); }  // (-0 is 0)
__device__ __forceinline__ float key_value(uint64_t k) {
    const uint32_t u = (uint32_t)(k >> 32);
    return __uint_as_float(u & 0x80000000u ? u & 0x7FFFFFFFu : ~u);
}
template <typename V>
__device__ __forceinline__ V ld_part(const V* local, int rank, int parts) {
    if (parts == 1) return *local;
    uint32_t remote;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(tc::smem_u32(local)), "r"(rank));
    V v;
    if constexpr (sizeof(V) == 8) {
        asm volatile("ld.shared::cluster.b64 %0, [%1];" : "=l"(v) : "r"(remote) : "memory");
    } else {
        uint32_t w;
        asm volatile("ld.shared::cluster.b32 %0, [%1];" : "=r"(w) : "r"(remote) : "memory");
        v = *reinterpret_cast<V*>(&w);
    }
    return v;
}

// The list's k best keys alone (n > k of them are in it), its k-th best as the new tau.  By all threads; the k-th key is
// found bit by bit.  Lists that need it come from rows whose logits rise along the vocabulary.
__device__ __noinline__ void keep_best(Shared& S, uint64_t* cand, int n, int k) {
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
        if (cand[i] >= kth) S.all[atomicAdd(&S.n_keep, 1)] = cand[i];
    __syncthreads();
    if (tid < k) cand[tid] = S.all[tid];
    if (tid == 0) {
        S.n_cand = k;
        S.tau = kth;
    }
    __syncthreads();
}

template <typename T, bool TOP>
__global__ void __launch_bounds__(NT) logprobs_kernel(dflash_logprobs_args a, int parts) {
    constexpr int G = 16 / (int)sizeof(T), NV = E / G;
    __shared__ Shared S;
    extern __shared__ __align__(16) uint64_t cand[];  // [CAP] (TOP)
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const long long row = blockIdx.x;
    const int rank = parts > 1 ? (int)tc::cluster_rank() : 0;
    const T* X = reinterpret_cast<const T*>(a.logits) + row * a.ld_logits;
    pdl_wait();
    pdl_trigger();

    // tokens before the first aligned vector and behind the last one go to an extra tile of the last CTA
    const int head = min(a.vocab, (int)((16 - ((uintptr_t)X & 15)) & 15) / (int)sizeof(T));
    const int vecs = (a.vocab - head) / G, left = a.vocab - vecs * G;
    const int per = (vecs + parts - 1) / parts, v0 = min(vecs, rank * per), v1 = min(vecs, v0 + per);
    const int full = (v1 - v0 + NT * NV - 1) / (NT * NV), tiles = full + (rank == parts - 1 && left > 0);
    const uint32_t NONE = sizeof(T) == 4 ? 0xFF800000u : 0xFF80FF80u;  // -inf
    auto load = [&](int it, uint4 (&r)[NV]) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            r[i] = make_uint4(NONE, NONE, NONE, NONE);
            const int v = v0 + (it * NV + i) * NT + tid;
            if (it < full && v < v1) r[i] = __ldcs(reinterpret_cast<const uint4*>(X + head) + v);
        }
        if (it == full && it < tiles && tid < left) {
            const T x = X[tid < head ? tid : tid + vecs * G];
            if constexpr (sizeof(T) == 4) r[0].x = __float_as_uint(to_f32(x));
            else r[0].x = 0xFF800000u | __float_as_uint(to_f32(x)) >> 16;
        }
    };
    uint4 next[NV];
    load(0, next);

    if (tid < MAXT) {
        int t = -1;
        float x = 0.f;
        if (tid < a.n) {
            t = a.tokens[row * a.n + tid];
            if (t < 0 || t >= a.vocab) t = -1;
            else x = to_f32(X[t]);
        }
        S.id[tid] = t;
        S.xt[tid] = x;
        S.part.ahead[tid] = 0;
        S.part.best[tid] = 0;
    }
    static_assert(MAXT == MAXK, "one thread for both");
    if (tid == 0) {
        S.n_cand = 0;
        S.tau = ABOVE_NOTHING;
    }
    __syncthreads();

    const float c = a.inv_temperature * LOG2E;
    float m = -INFINITY, l = 0.f, t = 0.f;
    uint64_t tau = ABOVE_NOTHING;
    float tau_v = key_value(tau);
    int room = CAP;  // entries that are surely free
#pragma unroll 1
    for (int it = 0; it < tiles; ++it) {
        float x[E];
#pragma unroll
        for (int i = 0; i < NV; ++i) widen<T>(next[i], x + i * G);
        load(it + 1, next);
        const bool single = it == full;  // (one element a thread)
        int id[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int v = v0 + (it * NV + i) * NT + tid;
            id[i] = v < v1 ? head + v * G : NOWHERE;
        }
        if (single) id[0] = tid < left ? (tid < head ? tid : tid + vecs * G) : NOWHERE;

        // ---- statistics
        float tm = fmaxf(x[0], x[1]);
#pragma unroll
        for (int e = 2; e < E; e += 2) tm = fmaxf(tm, fmaxf(x[e], x[e + 1]));
        if (tm > m) {
            const float d = (m - tm) * c, al = ex2(d);
            t = m == -INFINITY ? 0.f : al * fmaf(l, max_nan(d, -1000.f), t);
            l *= al;
            m = tm;
        }
        const float ref = m == -INFINITY ? 0.f : m;
        if (a.entropy) {
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float y = max_nan((x[e] - ref) * c, -1000.f), p = ex2(y);
                l += p;
                t = fmaf(p, y, t);
            }
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e) l += ex2((x[e] - ref) * c);
        }

        // ---- ranks
        if (a.ranks)
#pragma unroll 1
            for (int q = 0; q < a.n; ++q) {
                const float xt = S.xt[q];
                const int at = S.id[q];
                if (at < 0 || !__any_sync(0xffffffffu, tm >= xt)) continue;
                int ahead = 0;
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    if (single) {
                        if (i == 0) ahead += x[0] > xt || (x[0] == xt && id[0] < at);
                    } else if (id[i] > at) {
#pragma unroll
                        for (int e = 0; e < G; ++e) ahead += x[i * G + e] > xt;
                    } else {
#pragma unroll
                        for (int e = 0; e < G; ++e) ahead += x[i * G + e] > xt || (x[i * G + e] == xt && id[i] + e < at);
                    }
                }
                ahead = __reduce_add_sync(0xffffffffu, ahead);
                if (lane == 0 && ahead) atomicAdd(&S.part.ahead[q], ahead);
            }

        // ---- candidates
        if (TOP) {
            bool may = tm >= tau_v;
            int n = __syncthreads_count(may);
            if (n > MANY) {
                uint64_t key = 0;
                if (may) {
#pragma unroll
                    for (int e = E - 1; e >= 0; --e)
                        if (x[e] == tm) key = key_of(tm, id[e / G] + e % G);
                }
#pragma unroll
                for (int o = 1; o < NT / GROUPS; o <<= 1) {
                    const uint64_t y = __shfl_xor_sync(0xffffffffu, key, o);
                    key = y > key ? y : key;
                }
                if (tid % (NT / GROUPS) == 0) S.group[tid / (NT / GROUPS)] = key;
                __syncthreads();
                if (tid < GROUPS) {
                    const uint64_t mine = S.group[tid];
                    int above = 0;
#pragma unroll 8
                    for (int j = 0; j < GROUPS; ++j) above += S.group[j] > mine;
                    if (above == a.k - 1 && mine > tau) S.tau = mine;
                }
                __syncthreads();
                tau = S.tau;
                tau_v = key_value(tau);
                may = tm >= tau_v;
                n = MANY;
            }
            if (may) {
#pragma unroll
                for (int e = 0; e < E; ++e)
                    if (x[e] >= tau_v) {
                        const uint64_t key = key_of(x[e], id[e / G] + e % G);
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
                    keep_best(S, cand, have, a.k);
                    tau = S.tau;
                    tau_v = key_value(tau);
                    room = CAP - a.k;
                }
            }
        }
    }

    // ---- the CTA's results
    {
        float M = warp_max(m);
        const float al = m == -INFINITY ? 0.f : ex2((m - M) * c);
        t = m == -INFINITY ? 0.f : al * fmaf(l, max_nan((m - M) * c, -1000.f), t);
        l = warp_sum(l * al);
        t = warp_sum(t);
        if (lane == 0) {
            S.red[0][warp] = M;
            S.red[1][warp] = l;
            S.red[2][warp] = t;
        }
    }
    __syncthreads();
    if (TOP) {
        int n = min(S.n_cand, CAP);
        if (n > 512) {
            __syncthreads();
            keep_best(S, cand, n, a.k);
            n = a.k;
        }
        for (int i = tid; i < n; i += NT) {
            const uint64_t mine = cand[i];
            int above = 0;
            for (int j = 0; j < n; ++j) above += cand[j] > mine;
            if (above < a.k) S.part.best[above] = mine;
        }
    }
    // (M, l, t) of lanes 0 .. n-1 joined in all of them
    auto join = [&](int n) {
        const float M = warp_max(lane < n ? m : -INFINITY);
        const float al = m == -INFINITY ? 0.f : ex2((m - M) * c);
        t = lane >= n || m == -INFINITY ? 0.f : al * fmaf(l, max_nan((m - M) * c, -1000.f), t);
        l = warp_sum(lane < n ? l * al : 0.f);
        t = warp_sum(t);
        m = M;
    };
    if (warp == 0) {
        if (lane < WARPS) {
            m = S.red[0][lane];
            l = S.red[1][lane];
            t = S.red[2][lane];
        }
        join(WARPS);
        if (lane == 0) {
            S.part.m = m;
            S.part.l = l;
            S.part.t = t;
        }
    }
    __syncwarp();
    if (parts > 1) tc::cluster_sync();
    else __syncthreads();
    if (rank == 0) {
        // ---- the row's: every warp joins the parts
        const int r = min(lane, parts - 1);
        m = ld_part(&S.part.m, r, parts);
        l = ld_part(&S.part.l, r, parts);
        t = ld_part(&S.part.t, r, parts);
        join(parts);
        const bool bad = isnan(l) || m == INFINITY, none = l == 0.f;
        const float ln_l = logf(l);
        auto logprob = [&](float x) { return bad ? NAN : x == -INFINITY ? -INFINITY : (x - m) * a.inv_temperature - ln_l; };
        if (tid == 0) {
            if (a.lse) a.lse[row] = bad ? NAN : none ? -INFINITY : fmaf(m, a.inv_temperature, ln_l);
            if (a.entropy) a.entropy[row] = bad ? NAN : none ? 0.f : ln_l - LN2 * (t / l);
        }
        if (tid < a.n) {
            const int at = S.id[tid];
            int ahead = 0;
            for (int q = 0; q < parts; ++q) ahead += ld_part(&S.part.ahead[tid], q, parts);
            if (a.logprobs) a.logprobs[row * a.n + tid] = at < 0 ? 0.f : logprob(S.xt[tid]);
            if (a.ranks) a.ranks[row * a.n + tid] = at < 0 || bad ? -1 : ahead;
        }
        if (TOP) {
            const int q = tid / MAXK, i = tid % MAXK;
            const uint64_t mine = q < parts ? ld_part(&S.part.best[i], q, parts) : 0;
            if (q < parts) S.all[tid] = mine;
            if (tid < a.k) {  // (what a row of few tokens leaves)
                if (a.top_ids) a.top_ids[row * a.k + tid] = -1;
                if (a.top_logprobs) a.top_logprobs[row * a.k + tid] = bad ? NAN : -INFINITY;
            }
            __syncthreads();
            if (mine && !bad) {
                int above = 0;
                for (int s = 0; s < parts; ++s)
                    for (int j = 0; j < a.k; ++j) above += S.all[s * MAXK + j] > mine;
                if (above < a.k) {
                    if (a.top_ids) a.top_ids[row * a.k + above] = (int)argmax_key_index(mine);
                    if (a.top_logprobs) a.top_logprobs[row * a.k + above] = logprob(key_value(mine));
                }
            }
        }
    }
    __syncwarp();
    if (parts > 1) tc::cluster_sync();  // (no CTA leaves while its results are read)
}
static_assert(MAXC * MAXK == NT, "a thread for every part's every alternative");

template <typename T>
void forward(const Launch& L, const dflash_logprobs_args& a) {
    const int G = 16 / (int)sizeof(T);
    const long long tiles = ((long long)a.vocab / G + NT * (E / G) - 1) / (NT * (E / G));
    int parts = 1;
    while (parts < MAXC && 2 * parts <= tiles && (long long)a.rows * parts < 152 * 16) parts *= 2;
    const bool top = a.k > 0 && (a.top_ids || a.top_logprobs);
    if (top) launch_k(L, logprobs_kernel<T, true>, dim3(a.rows, 1, parts), dim3(NT), CAP * 8, parts, a, parts);
    else launch_k(L, logprobs_kernel<T, false>, dim3(a.rows, 1, parts), dim3(NT), 0, parts, a, parts);
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
    float lse = a.lse[row];
    if (lse == -INFINITY) lse = INFINITY;  // (a row of -inf alone: p = 0)
    // -p (G + h (ln p + H)); ln p below any p that is not 0
    auto slope = [&](float x) {
        const float z = max_nan(fmaf(x, a.inv_temperature, -lse), -1000.f);
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

dflash_status fail(const char* msg) {
    set_global_error(msg);
    return DFLASH_E_INVAL;
}

template <typename F>
dflash_status queue(void* cuda_stream, const char* failed_text, F&& f) {
    bool failed = false;
    Launch L{(cudaStream_t)cuda_stream, nullptr};
    L.pdl = true;  // (each kernel waits for what runs before it ahead of its first read)
    L.failed = &failed;
    f(L);
    const cudaError_t e = cudaGetLastError();
    if (failed || e != cudaSuccess) {
        set_global_error(e != cudaSuccess ? cudaGetErrorString(e) : failed_text);
        return DFLASH_E_CUDA;
    }
    return DFLASH_OK;
}

}  // namespace

}  // namespace dfl

using namespace dfl;

extern "C" dflash_status dflash_token_logprobs(const dflash_logprobs_args* p, void* cuda_stream) {
    if (!p) return fail("token_logprobs: args is NULL");
    const dflash_logprobs_args& a = *p;
    if (a.dtype != DFLASH_DTYPE_F32 && a.dtype != DFLASH_DTYPE_BF16) return fail("token_logprobs: dtype must be F32 or BF16");
    if (a.rows < 0 || a.rows > (1 << 20)) return fail("token_logprobs: rows outside [0, 2^20]");
    if (a.vocab < 1 || a.vocab > (1 << 30)) return fail("token_logprobs: vocab outside [1, 2^30]");
    if (a.n < 0 || a.n > MAXT) return fail("token_logprobs: n outside [0, 32]");
    if (a.k < 0 || a.k > MAXK) return fail("token_logprobs: k outside [0, 32]");
    if (!(a.inv_temperature > 0.f) || a.inv_temperature > 3e38f)
        return fail("token_logprobs: inv_temperature must be positive and finite");
    if ((a.rows > 0 && !a.logits) || (a.rows > 0 && a.n > 0 && !a.tokens)) return fail("token_logprobs: NULL argument");
    if ((uintptr_t)a.logits % (a.dtype == DFLASH_DTYPE_BF16 ? 2 : 4)) return fail("token_logprobs: logits is not aligned to its type");
    if (a.ld_logits < a.vocab) return fail("token_logprobs: the row stride is smaller than vocab");
    if (a.rows == 0) return DFLASH_OK;
    return queue(cuda_stream, "token_logprobs: launch failed", [&](const Launch& L) {
        if (a.dtype == DFLASH_DTYPE_BF16) forward<bf16>(L, a);
        else forward<float>(L, a);
    });
}

extern "C" dflash_status dflash_token_logprobs_grad(const dflash_logprobs_grad_args* p, void* cuda_stream) {
    if (!p) return fail("token_logprobs_grad: args is NULL");
    const dflash_logprobs_grad_args& a = *p;
    if (a.dtype != DFLASH_DTYPE_F32 && a.dtype != DFLASH_DTYPE_BF16)
        return fail("token_logprobs_grad: dtype must be F32 or BF16");
    if (a.rows < 0 || a.rows > (1 << 20)) return fail("token_logprobs_grad: rows outside [0, 2^20]");
    if (a.vocab < 1 || a.vocab > (1 << 30)) return fail("token_logprobs_grad: vocab outside [1, 2^30]");
    if (a.n < 0 || a.n > MAXT) return fail("token_logprobs_grad: n outside [0, 32]");
    if (!(a.inv_temperature > 0.f) || a.inv_temperature > 3e38f)
        return fail("token_logprobs_grad: inv_temperature must be positive and finite");
    if (a.reserved != 0) return fail("token_logprobs_grad: reserved must be 0");
    if (a.rows > 0 && (!a.logits || !a.out || !a.lse || (a.n > 0 && (!a.tokens || !a.grad_logprobs)) || (a.grad_entropy && !a.entropy)))
        return fail("token_logprobs_grad: NULL argument");
    const uintptr_t es = a.dtype == DFLASH_DTYPE_BF16 ? 2 : 4;
    if (((uintptr_t)a.logits | (uintptr_t)a.out) % es) return fail("token_logprobs_grad: logits or out is not aligned to its type");
    if (a.ld_logits < a.vocab || a.ld_out < a.vocab) return fail("token_logprobs_grad: a row stride is smaller than vocab");
    if (a.out == a.logits && a.ld_out != a.ld_logits && a.rows > 1) return fail("token_logprobs_grad: in place needs one row stride");
    const long long chunk = NB * VB;
    if ((long long)a.rows * ((a.vocab + chunk - 1) / chunk) >= (1ll << 31)) return fail("token_logprobs_grad: rows * vocab is too large");
    if (a.rows == 0) return DFLASH_OK;
    return queue(cuda_stream, "token_logprobs_grad: launch failed", [&](const Launch& L) {
        if (a.dtype == DFLASH_DTYPE_BF16) backward<bf16>(L, a);
        else backward<float>(L, a);
    });
}
