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
// A CTA takes one row and `kper` KV heads; a thread takes 8 head dimensions of one query vector, so each
// partial is read in whole 32-byte sectors.  Bytes: 4 hd + 8 per vector and segment (in L2), out written
// once.
struct MergeArgs {
    sp::Shape P;
    sp::Work W;
    void* out;
    float* lse;
    long long ld_out;
    int kper;
};

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
__global__ void __launch_bounds__(256) merge_kernel(MergeArgs a) {
    using namespace sp;
    __shared__ int seq_s, bad_s;
    const Shape& P = a.P;
    const int tid = threadIdx.x, r = blockIdx.x;
    if (tid == 0) {
        seq_s = -1;
        bad_s = 0;
    }
    __syncthreads();
    pdl_wait();
    pdl_trigger();
    const Head h = *a.W.head;
    for (int c = tid; c < P.n_cta; c += blockDim.x)
        if (a.W.err[c]) bad_s = 1;
    for (int s = tid; s < P.batch; s += blockDim.x)
        if (P.q_start[s] <= r && r < P.q_start[s + 1]) seq_s = s;
    __syncthreads();
    bool bad = h.bad || bad_s;
    const int seq = seq_s;
    if (!bad && seq < 0) return;  // a row of no sequence
    Seq q = {};
    int j = 0, start = 0;
    if (!bad) {
        start = P.q_start[seq];
        q = seq_of(P, start, P.q_start[seq + 1], P.kv_lens[seq]);
        j = r - start;
        if (q.kv < 0 || q.kv > (long long)64 * P.width) bad = true;
    }
    const int chunks = P.hd / 8;
    for (int i = tid; i < a.kper * P.g * chunks; i += blockDim.x) {
        const int c8 = i % chunks, hh = i / chunks % P.g, kvh = blockIdx.y * a.kper + i / (chunks * P.g);
        if (kvh >= P.Hkv) break;
        float M = -INFINITY, l = 0.f, o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        uint32_t slot_bad = 0;
        // the segments of the item whose line starts at b: n tiles of weight w, of which the first n_eff count
        auto item = [&](uint32_t b, uint32_t w, int n, int n_eff, int id, int nrows, int rl) {
            const bool pair = nrows > P.RH;
            const int x0 = pair ? rl / P.RH : 0, x1 = pair ? x0 : 1;
            const int v = (pair ? rl % P.RH : rl) * P.g + hh;
            const int c1 = owner(h.W, b + (uint32_t)(n - 1) * w, P.n_cta);
            for (int c = owner(h.W, b, P.n_cta); c <= c1; ++c) {
                const uint32_t lo = max(b, part_begin(h.W, c, P.n_cta)), hi = part_begin(h.W, c + 1, P.n_cta);
                const int t0 = (int)((lo - b + w - 1) / w);
                const int t1 = min((int)min((uint32_t)n, (hi - b + w - 1) / w), n_eff);
                if (t0 >= t1) continue;
                slot_bad |= a.W.slot_bad[id + c];
                for (int x = x0; x <= x1; ++x) {
                    if (x == 1 && !pair && t1 - t0 < 2) break;  // stream B had no tile
                    const size_t slot = (size_t)(id + c) * 2 + x;
                    const float2 ml = a.W.ml[slot * P.VT + v];
                    const float* src = a.W.o + slot * P.VT * P.hd + ((size_t)c8 * P.VT + v) * 8;
                    const float4 s0 = *reinterpret_cast<const float4*>(src), s1 = *reinterpret_cast<const float4*>(src + 4);
                    const float mn = fmaxf(M, ml.x);
                    const float e0 = M == -INFINITY ? 0.f : exp2f(M - mn), e1 = ml.x == -INFINITY ? 0.f : exp2f(ml.x - mn);
                    M = mn;
                    l = l * e0 + ml.y * e1;
                    const float y[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
#pragma unroll
                    for (int e = 0; e < 8; ++e) o[e] = o[e] * e0 + (e1 == 0.f ? 0.f : y[e] * e1);
                }
            }
        };
        if (!bad && P.npt) {
            const int rt = (r - h.r_begin) / P.RT, id = kvh * h.nqt + rt;
            item((uint32_t)id * P.npt * h.wp, h.wp, P.npt, P.npt, id, min(P.RT, h.r_end - h.r_begin - rt * P.RT),
                 (r - h.r_begin) % P.RT);
        }
        if (!bad && q.tiles) {
            const int gi = j / P.RT, k = kvh * q.groups + gi, nrows = min(P.RT, q.m - gi * P.RT);
            const int n_eff = P.causal ? min(q.tiles, cdiv(max(q.kv - q.m + gi * P.RT + nrows, 0), P.KT)) : q.tiles;
            item(a.W.base[seq] + (uint32_t)k * q.tiles * q.w, q.w, q.tiles, n_eff, (int)(h.n_prefix + a.W.ibase[seq]) + k, nrows,
                 j % P.RT);
        }
        const bool nan = bad || slot_bad;
        const float inv = l > 0.f ? 1.f / l : 0.f;
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = nan ? NAN : o[e] * inv;
        const int head = kvh * P.g + hh;
        store8<T>(reinterpret_cast<T*>(a.out) + (long long)r * a.ld_out + (long long)head * P.hd + c8 * 8, y);
        if (a.lse && c8 == 0)
            a.lse[(long long)r * P.H + head] = nan ? NAN : l > 0.f ? (M + log2f(l)) * 0.6931471805599453f : -INFINITY;
    }
}

}  // namespace

bool shared_attention_tc(const Launch& L, const sp::Shape& P, const sp::Work& W, const dflash_shared_prefix_args& a);

namespace {

constexpr int CTAS = 152;  // one per SM

sp::Shape shape_of(const dflash_shared_prefix_args& a) {
    sp::Shape P = {};
    P.H = a.n_heads;
    P.Hkv = a.n_kv_heads;
    P.g = a.n_heads / a.n_kv_heads;
    P.hd = a.head_dim;
    P.VT = 128;
    P.RH = P.VT / P.g;
    P.RT = 2 * P.RH;
    P.KT = 128;
    P.batch = a.batch;
    P.rows = a.rows;
    P.width = a.width;
    P.prefix_len = a.prefix_len;
    P.causal = a.causal != 0;
    P.n_pages = a.n_pages;
    P.npt = (a.prefix_len + P.KT - 1) / P.KT;
    P.n_cta = CTAS;
    P.ld_table = a.ld_table;
    P.prefix_pages = a.prefix_pages;
    P.table = a.table;
    P.kv_lens = a.kv_lens;
    P.q_start = a.q_start;
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
    m.P = shape_of(a);
    sp::layout((char*)a.workspace, a.head_dim, m.P.VT, a.batch, m.P.n_cta,
               sp::max_slots(a.n_kv_heads, m.P.RT, a.batch, a.rows, m.P.n_cta), &m.W);
    m.out = a.out;
    m.lse = a.lse;
    m.ld_out = a.ld_out;
    if (!shared_attention_tc(L, m.P, m.W, a)) return false;
    // the merge starts as the main kernel's CTAs leave
    Launch after = L;
    after.pdl = true;
    const int per = m.P.g * a.head_dim / 8;
    m.kper = std::max(1, 256 / per);
    launch_k(after, merge_kernel<bf16>, dim3(a.rows, (a.n_kv_heads + m.kper - 1) / m.kper), dim3(256), 0, 1, m);
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
    if (a.batch < 1 || a.batch > DFLASH_OPS_MAX_BATCH) return bad("shared_prefix_attention: batch outside [1, 4096]");
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
    const int RT = 2 * (128 / (n_heads / n_kv_heads));
    return sp::layout(nullptr, head_dim, 128, batch, CTAS, sp::max_slots(n_kv_heads, RT, batch, rows, CTAS), nullptr);
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
