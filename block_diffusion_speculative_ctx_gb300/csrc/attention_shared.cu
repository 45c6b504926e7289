// Attention of a batch that shares a prefix (dflash_shared_prefix_attention in
// include/dflash.h).
//
// Simplest form: one warp per (row, query head) walks the row's keys, prefix
// then own, with an online softmax in fp32 (base 2); lane l holds head
// dimensions l, l + 32, ...  Every key is read once per query vector.
#include <math.h>

#include "ops.h"

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

}  // namespace

bool shared_prefix_attention(const Launch& L, const dflash_shared_prefix_args& a) {
    const dim3 grid(a.rows, (a.n_heads + 3) / 4);
    if (a.dtype == DFLASH_DTYPE_BF16) {
        if (a.head_dim == 128) launch_k(L, shared_simple_kernel<bf16, 128>, grid, dim3(128), 0, 1, a);
        else launch_k(L, shared_simple_kernel<bf16, 64>, grid, dim3(128), 0, 1, a);
    } else {
        if (a.head_dim == 128) launch_k(L, shared_simple_kernel<float, 128>, grid, dim3(128), 0, 1, a);
        else launch_k(L, shared_simple_kernel<float, 64>, grid, dim3(128), 0, 1, a);
    }
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

extern "C" size_t dflash_shared_prefix_workspace(int32_t, int32_t, int32_t, int32_t, int32_t, int32_t) { return 16; }

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
