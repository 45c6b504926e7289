// Attention of a batch that shares a prefix (dflash_shared_prefix_attention in
// include/dflash.h).
//
// Simplest form: one warp per (row, query head) walks the row's keys, prefix
// then own, with an online softmax in fp32 (base 2); lane l holds head
// dimensions l, l + 32, ...  Every key is read once per query vector.
#include <math.h>

#include <algorithm>

#include "shared_plan.cuh"
#include "tcgen05.cuh"

namespace dfl {

namespace {

template <typename T, int HD>
__global__ void __launch_bounds__(128) shared_simple_kernel(dflash_shared_prefix_args a) {
    pdl_wait();
    pdl_trigger();
    constexpr int PER = HD / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int r = blockIdx.x, h = blockIdx.y * 4 + warp;
    if (h >= a.n_heads) return;
    // the row's sequence: the last s with q_start[s] <= r
    int lo = 0, hi = a.batch;
    if (r < a.q_start[0] || r >= a.q_start[a.batch]) return;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a.q_start[mid] <= r) lo = mid;
        else hi = mid;
    }
    const int s = lo, start = a.q_start[s], m = a.q_start[s + 1] - start;
    const int own = a.kv_lens[s];
    bool bad = start < 0 || m <= 0 || start + m > a.rows || own < 0 || (long long)own > 64ll * a.width;
    const int lim = bad ? 0 : (a.causal ? max(own - m + (r - start) + 1, 0) : own);
    const int kvh = h / (a.n_heads / a.n_kv_heads);
    const T* q = reinterpret_cast<const T*>(a.q) + (long long)r * a.ld_q + (long long)h * HD;
    float qv[PER], o[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        qv[i] = to_f32(q[lane + 32 * i]);
        o[i] = 0.f;
    }
    const float sl = a.scale * 1.4426950408889634f;
    float mx = -INFINITY, l = 0.f;
    auto walk = [&](const int* pages, int n) {
        for (int k = 0; k < n; ++k) {
            const int page = pages[k >> 6];
            if (page < 0 || page >= a.n_pages) {
                bad = true;
                return;
            }
            const long long off = (((long long)page * a.n_kv_heads + kvh) * 64 + (k & 63)) * HD;
            const T* K = reinterpret_cast<const T*>(a.k_cache) + off;
            const T* V = reinterpret_cast<const T*>(a.v_cache) + off;
            float d = 0.f;
#pragma unroll
            for (int i = 0; i < PER; ++i) d += qv[i] * to_f32(K[lane + 32 * i]);
            d = warp_sum(d) * sl;
            const float mn = fmaxf(mx, d);
            const float al = mx == -INFINITY ? 0.f : exp2f(mx - mn), p = exp2f(d - mn);
            l = l * al + p;
#pragma unroll
            for (int i = 0; i < PER; ++i) o[i] = o[i] * al + p * to_f32(V[lane + 32 * i]);
            mx = mn;
        }
    };
    if (!bad) walk(a.prefix_pages, a.prefix_len);
    if (!bad) walk(a.table + (long long)s * a.ld_table, lim);
    const float inv = bad ? NAN : l > 0.f ? 1.f / l : 0.f;
    T* out = reinterpret_cast<T*>(a.out) + (long long)r * a.ld_out + (long long)h * HD;
#pragma unroll
    for (int i = 0; i < PER; ++i) out[lane + 32 * i] = from_f32<T>(bad ? NAN : o[i] * inv);
    if (a.lse && lane == 0)
        a.lse[(long long)r * a.n_heads + h] = bad ? NAN : l > 0.f ? (mx + log2f(l)) * 0.6931471805599453f : -INFINITY;
}


// Merge of the partial results: out = sum_i 2^(m_i - M) o_i / sum_i 2^(m_i - M) l_i over the segments that
// hold the row's query vectors, prefix and own, in plan order (one fixed order: the same bits every run).
// A CTA takes one row and one KV head, so its chain of dependent loads is: lengths -> (max, sum) of every
// segment, one a thread -> outputs, read by groups of threads that take every G-th segment, a thread 8 head
// dimensions of one query vector (whole 32-byte sectors).  Bytes: 4 hd + 8 per vector and segment, from L2.
struct MergeArgs {
    sp::Shape P;
    sp::Work W;
    void* out;
    float* lse;
    long long ld_out;
};

constexpr int MNT = 256;
constexpr int MSEG = 3 * 160;  // segments of one row: at most one per worker of line 0 and of line 1
constexpr int MHEADS = 8;      // query heads at a time

template <typename T>
__device__ __forceinline__ void store8(T* d, const float (&x)[8]);
template <>
__device__ __forceinline__ void store8<float>(float* d, const float (&x)[8]) {
    *reinterpret_cast<float4*>(d) = make_float4(x[0], x[1], x[2], x[3]);
    *reinterpret_cast<float4*>(d + 4) = make_float4(x[4], x[5], x[6], x[7]);
}
template <>
__device__ __forceinline__ void store8<bf16>(bf16* d, const float (&x)[8]) {
    *reinterpret_cast<uint4*>(d) =
        make_uint4(tc::pack2_bf16(x[0], x[1]), tc::pack2_bf16(x[2], x[3]), tc::pack2_bf16(x[4], x[5]), tc::pack2_bf16(x[6], x[7]));
}

template <typename T>
__global__ void __launch_bounds__(MNT) merge_kernel(MergeArgs a) {
    using namespace sp;
    __shared__ int seq_s, bad_s, n_s;
    __shared__ uint32_t blk_s[MSEG];               // block and stream of each segment
    __shared__ float wgt_s[MHEADS][MSEG];          // its weight 2^(m - M) for each query head
    __shared__ float inv_s[MHEADS];
    __shared__ float acc_s[MNT][8];
    const Shape& P = a.P;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int r = blockIdx.x, kvh = blockIdx.y;
    if (tid == 0) {
        seq_s = -1;
        bad_s = 0;
    }
    __syncthreads();
    pdl_wait();
    pdl_trigger();
    const Head h = *a.W.head;
    for (int c = tid; c < P.n_cta; c += MNT)
        if (a.W.err[c]) bad_s = 1;
    for (int s = tid; s < P.batch; s += MNT)
        if (P.q_start[s] <= r && r < P.q_start[s + 1]) seq_s = s;
    __syncthreads();
    bool bad = h.bad || bad_s;
    const int seq = seq_s;
    if (!bad && seq < 0) return;  // a row of no sequence
    // the row's items: [0] prefix, [1] own
    int line[2] = {0, 0}, n[2] = {0, 0}, n_eff[2] = {0, 0}, id[2] = {0, 0}, c0[2] = {0, 0}, nc[2] = {0, 0}, rl[2] = {0, 0};
    uint32_t at[2] = {0u, 0u};
    if (!bad) {
        const int start = P.q_start[seq];
        const Seq q = seq_of(P, start, P.q_start[seq + 1], P.kv_lens[seq]);
        if (q.kv < 0 || q.kv > (long long)64 * P.width) bad = true;
        if (P.npt) {
            const int RT = P.row_tile(h.pl), rt = (r - h.r_begin) / RT;
            line[0] = h.pl;
            n[0] = n_eff[0] = P.npt;
            id[0] = kvh * h.nqt + rt;
            at[0] = (uint32_t)id[0] * (P.lead[h.pl] + (uint32_t)P.npt * P.w);
            rl[0] = (r - h.r_begin) - rt * RT;
        }
        if (q.tiles && !bad) {
            const int RT = P.row_tile(q.line), j = r - start, gi = j / RT, k = kvh * q.groups + gi;
            line[1] = q.line;
            n[1] = q.tiles;
            n_eff[1] = seen_tiles(P, q, min(q.m, (gi + 1) * RT));
            id[1] = (h.pl == q.line ? h.n_prefix : 0) + (int)a.W.ibase[seq] + k;
            at[1] = a.W.base[seq] + (uint32_t)k * (P.lead[q.line] + (uint32_t)q.tiles * P.w);
            rl[1] = j - gi * RT;
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (n_eff[i]) {
                const uint32_t W = h.W[line[i]], t0 = at[i] + P.lead[line[i]];
                c0[i] = owner(W, t0, P.workers(line[i]));
                nc[i] = owner(W, t0 + (uint32_t)(n_eff[i] - 1) * P.w, P.workers(line[i])) - c0[i] + 1;
            }
    }
    const int cand = nc[0] + nc[1];  // workers that may hold a segment, in plan order
    auto vec = [&](int i) { return rl[i] % P.RH * P.g; };  // first of the row's vectors in its stream
    if (tid == 0) n_s = cand;
    for (int k = tid; k < cand; k += MNT) {
        const int i = k < nc[0] ? 0 : 1, c = i ? c0[1] + k - nc[0] : c0[0] + k;
        const uint32_t W = h.W[line[i]];
        int t0, t1;
        cut(max(at[i], part_begin(W, c, P.workers(line[i]))), part_begin(W, c + 1, P.workers(line[i])), at[i],
            P.lead[line[i]], P.w, n[i], t0, t1);
        uint32_t blk = 0xFFFFFFFFu;  // no tile of the item in this worker's part
        if (t0 < min(t1, n_eff[i])) {
            blk = block_of(P, h, line[i], id[i], c) + (uint32_t)(rl[i] / P.RH);
            if (a.W.block_bad[blk]) bad_s = 1;
        }
        blk_s[k] = blk;
    }
    __syncthreads();
    bad = bad || bad_s;

    const int chunks = P.hd / 8;
    for (int h0 = 0; h0 < P.g; h0 += MHEADS) {
        const int nh = min(MHEADS, P.g - h0);
        // weights: a warp takes a head
        for (int hh = warp; hh < nh; hh += MNT / 32) {
            float M = -INFINITY;
            for (int k = lane; k < cand; k += 32) {
                float m = -INFINITY;
                if (blk_s[k] != 0xFFFFFFFFu) m = a.W.ml[(size_t)blk_s[k] * P.VT + vec(k < nc[0] ? 0 : 1) + h0 + hh].x;
                wgt_s[hh][k] = m;
                M = fmaxf(M, m);
            }
            M = warp_max(M);
            float l = 0.f;
            for (int k = lane; k < cand; k += 32) {
                const float m = wgt_s[hh][k], w = m == -INFINITY ? 0.f : exp2f(m - M);
                if (w != 0.f) l += w * a.W.ml[(size_t)blk_s[k] * P.VT + vec(k < nc[0] ? 0 : 1) + h0 + hh].y;
                wgt_s[hh][k] = w;
            }
            l = warp_sum(l);
            if (lane == 0) {
                inv_s[hh] = bad ? NAN : l > 0.f ? 1.f / l : 0.f;
                if (a.lse)
                    a.lse[(long long)r * P.H + kvh * P.g + h0 + hh] =
                        bad ? NAN : l > 0.f ? (M + log2f(l)) * 0.6931471805599453f : -INFINITY;
            }
        }
        __syncthreads();
        const int part = nh * chunks, G = MNT / part, grp = tid / part, e = tid - grp * part;
        const int hh = e / chunks, c8 = e - hh * chunks;
        float o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (grp < G) {
#pragma unroll 4
            for (int k = grp; k < cand; k += G) {
                const float w = wgt_s[hh][k];
                if (w != 0.f) {
                    const float* src = a.W.o + (size_t)blk_s[k] * P.VT * P.hd +
                                       ((size_t)c8 * P.VT + vec(k < nc[0] ? 0 : 1) + h0 + hh) * 8;
                    const float4 x = *reinterpret_cast<const float4*>(src), y = *reinterpret_cast<const float4*>(src + 4);
                    o[0] += w * x.x;
                    o[1] += w * x.y;
                    o[2] += w * x.z;
                    o[3] += w * x.w;
                    o[4] += w * y.x;
                    o[5] += w * y.y;
                    o[6] += w * y.z;
                    o[7] += w * y.w;
                }
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) acc_s[tid][i] = o[i];
        }
        __syncthreads();
        if (grp == 0) {
            for (int q = 1; q < G; ++q)
#pragma unroll
                for (int i = 0; i < 8; ++i) o[i] += acc_s[tid + q * part][i];
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = bad ? NAN : o[i] * inv_s[hh];
            store8<T>(reinterpret_cast<T*>(a.out) + (long long)r * a.ld_out + (long long)(kvh * P.g + h0 + hh) * P.hd + c8 * 8, o);
        }
        __syncthreads();
    }
}

}  // namespace

bool shared_attention_tc(const Launch& L, const sp::Shape& P, const sp::Work& W, const dflash_shared_prefix_args& a);

namespace {

constexpr int CTAS = 152;  // one per SM

// The sizes alone (what the workspace depends on).
sp::Shape sizes_of(int H, int Hkv, int hd, int batch, int rows) {
    sp::Shape P = {};
    P.H = H;
    P.Hkv = Hkv;
    P.g = H / Hkv;
    P.hd = hd;
    P.VT = 128;
    P.RH = P.VT / P.g;
    P.KT = 64;
    P.batch = batch;
    P.rows = rows;
    P.n_cta = CTAS;
    // an item's fixed cost: two tiles on line 0, three on line 1
    P.w = 1;
    P.lead[0] = 2;
    P.lead[1] = 3;
    return P;
}

}  // namespace

bool shared_prefix_attention(const Launch& L, const dflash_shared_prefix_args& a) {
    if (a.dtype == DFLASH_DTYPE_F32) {
        const dim3 grid(a.rows, (a.n_heads + 3) / 4);
        if (a.head_dim == 128) launch_k(L, shared_simple_kernel<float, 128>, grid, dim3(128), 0, 1, a);
        else launch_k(L, shared_simple_kernel<float, 64>, grid, dim3(128), 0, 1, a);
        return true;
    }
    MergeArgs m;
    sp::Shape& P = m.P;
    P = sizes_of(a.n_heads, a.n_kv_heads, a.head_dim, a.batch, a.rows);
    P.width = a.width;
    P.prefix_len = a.prefix_len;
    P.causal = a.causal != 0;
    P.n_pages = a.n_pages;
    P.npt = (a.prefix_len + P.KT - 1) / P.KT;
    P.ld_table = a.ld_table;
    P.prefix_pages = a.prefix_pages;
    P.table = a.table;
    P.kv_lens = a.kv_lens;
    P.q_start = a.q_start;
    sp::layout((char*)a.workspace, P, &m.W);
    m.out = a.out;
    m.lse = a.lse;
    m.ld_out = a.ld_out;
    if (!shared_attention_tc(L, P, m.W, a)) return false;
    // the merge starts as the main kernel's CTAs leave
    Launch after = L;
    after.pdl = true;
    launch_k(after, merge_kernel<bf16>, dim3(a.rows, a.n_kv_heads), dim3(MNT), 0, 1, m);
    return true;
}

dflash_status check_shared_prefix(const dflash_shared_prefix_args& a, const char** why) {
    auto bad = [&](const char* m) {
        *why = m;
        return DFLASH_E_INVAL;
    };
    if (a.dtype != DFLASH_DTYPE_F32 && a.dtype != DFLASH_DTYPE_BF16)
        return bad("shared_prefix_attention: dtype must be F32 or BF16");
    if (a.head_dim != 64 && a.head_dim != 128) return bad("shared_prefix_attention: head_dim must be 64 or 128");
    if (a.n_heads < 1 || a.n_kv_heads < 1 || a.n_heads % a.n_kv_heads || a.n_heads / a.n_kv_heads > 64)
        return bad("shared_prefix_attention: n_heads must be a multiple of n_kv_heads, at most 64 times it");
    if (a.n_heads > 1024) return bad("shared_prefix_attention: more than 1024 heads");
    if (a.batch < 1 || a.batch > DFLASH_OPS_MAX_BATCH) return bad("shared_prefix_attention: batch outside [1, 2048]");
    if (a.rows < 0 || a.rows > (1 << 20)) return bad("shared_prefix_attention: rows outside [0, 2^20]");
    // rows of the caches as one matrix [pages * H_kv * 64, hd]: TMA coordinates are 32-bit
    if (a.n_pages < 1 || (long long)a.n_pages * a.n_kv_heads * 64 >= (1ll << 31))
        return bad("shared_prefix_attention: n_pages < 1, or n_pages * n_kv_heads * 64 reaches 2^31");
    if (a.prefix_len < 0 || a.prefix_len > (1 << 28)) return bad("shared_prefix_attention: prefix_len outside [0, 2^28]");
    if (a.width < 0 || a.width > (1 << 22)) return bad("shared_prefix_attention: width outside [0, 2^22]");
    if (!(a.scale > 0.f) || a.scale > 3e38f) return bad("shared_prefix_attention: scale must be positive and finite");
    if (!a.k_cache || !a.v_cache || !a.kv_lens || !a.q_start || (a.width > 0 && !a.table) ||
        (a.prefix_len > 0 && !a.prefix_pages) || (a.rows > 0 && (!a.q || !a.out)))
        return bad("shared_prefix_attention: NULL argument");
    const long long es = a.dtype == DFLASH_DTYPE_BF16 ? 2 : 4, width = (long long)a.n_heads * a.head_dim;
    if (((uintptr_t)a.q | (uintptr_t)a.k_cache | (uintptr_t)a.v_cache | (uintptr_t)a.out | (uintptr_t)a.workspace) & 15u)
        return bad("shared_prefix_attention: q, the caches, out and workspace must be 16-byte aligned");
    if (a.ld_q < width || a.ld_out < width || (a.ld_q * es) % 16 || (a.ld_out * es) % 16 || a.ld_q >= (1ll << 32) ||
        a.ld_out >= (1ll << 32))
        return bad("shared_prefix_attention: ld_q and ld_out must be at least H * hd and multiples of 16 bytes");
    if (a.ld_table < a.width) return bad("shared_prefix_attention: ld_table is smaller than width");
    if (a.workspace_bytes < dflash_shared_prefix_workspace(a.dtype, a.n_heads, a.n_kv_heads, a.head_dim, a.batch, a.rows) ||
        (a.rows > 0 && !a.workspace))
        return bad("shared_prefix_attention: workspace is smaller than dflash_shared_prefix_workspace()");
    return DFLASH_OK;
}

}  // namespace dfl

using namespace dfl;

extern "C" size_t dflash_shared_prefix_workspace(int32_t dtype, int32_t n_heads, int32_t n_kv_heads, int32_t head_dim,
                                                 int32_t batch, int32_t rows) {
    if (n_heads < 1 || n_kv_heads < 1 || n_heads % n_kv_heads || n_heads / n_kv_heads > 64 || batch < 1 ||
        batch > DFLASH_OPS_MAX_BATCH || rows < 0 || rows > (1 << 20) || (head_dim != 64 && head_dim != 128) ||
        (dtype != DFLASH_DTYPE_F32 && dtype != DFLASH_DTYPE_BF16))
        return 0;
    return sp::layout(nullptr, sizes_of(n_heads, n_kv_heads, head_dim, batch, rows), nullptr);
}

extern "C" dflash_status dflash_shared_prefix_attention(const dflash_shared_prefix_args* p, void* cuda_stream) {
    const char* why = "shared_prefix_attention: args is NULL";
    if (!p || check_shared_prefix(*p, &why) != DFLASH_OK) {
        set_global_error(why);
        return DFLASH_E_INVAL;
    }
    if (p->rows == 0) return DFLASH_OK;
    bool failed = false;
    Launch L{(cudaStream_t)cuda_stream, nullptr};
    L.failed = &failed;
    const bool ok = shared_prefix_attention(L, *p);
    const cudaError_t e = cudaGetLastError();
    if (!ok || failed || e != cudaSuccess) {
        set_global_error(e != cudaSuccess ? cudaGetErrorString(e)
                                          : "shared_prefix_attention: a kernel could not be prepared");
        return DFLASH_E_CUDA;
    }
    return DFLASH_OK;
}
