// A tree of drafted tokens around its verify pass: masks and positions before it
// (dflash_tree_masks), acceptance (dflash_tree_accept) and the cache behind it
// (dflash_kv_compact); include/dflash.h.
//
// Masks: node j sees itself and its chain of parents.  A thread a node walks the
// chain in shared memory; a parent has a lower number, so the mask's words come out
// from the last to the first, each written once.  A tree of drafts is some 16 links
// deep; a chain of 1024 nodes takes its 1024 steps.
// Acceptance: with next(p) = the lowest child of p that holds posterior[p] (an
// atomic minimum a node, whatever the order), the path is next applied from the
// root on: m independent steps and one chain of as many reads as tokens accepted.
// Both are bound by latency (a launch, two dependent reads of a few KB): some 2 us
// each in a graph.
// Compaction: path[j] >= j rises, so moves in the order of j never overwrite a row
// that is still to be read; a thread owns 16 bytes of a row of one head and has
// eight moves' loads in flight before their stores.  Bytes: twice the moved rows.
// Measured (graph replay, the three calls together): 5.8 us for one tree of 16 nodes
// over 5 layers, 10.5 us for 32 trees of up to 64 nodes over 36 layers (35 MB moved,
// 5.2 us at a measured copy's rate).
#include "ops.h"

namespace dfl {

namespace {

constexpr int MAXN = DFLASH_TREE_MAX_NODES;
enum : int { BAD_TREE = 1, BAD_SIZE = 2, BAD_ROWS = 4, BAD_LENGTH = 8, BAD_PAGE = 16 };

// A sequence's rows, or BAD_ROWS.
__device__ __forceinline__ int rows_of(const int* q_start, int s, int rows, int& start, int& m) {
    start = q_start[s];
    const int end = q_start[s + 1];
    m = end - start;
    return start < 0 || end < start || end > rows ? BAD_ROWS : 0;
}

constexpr int NT_MASK = 128;

__global__ void __launch_bounds__(NT_MASK) tree_masks_kernel(dflash_tree_masks_args a) {
    __shared__ int parent[MAXN];
    const int s = blockIdx.x, tid = threadIdx.x;
    pdl_wait();
    pdl_trigger();
    int start, m;
    int status = rows_of(a.q_start, s, a.rows, start, m);
    if (status == 0 && (m > MAXN || m > (long long)32 * a.words)) status = BAD_SIZE;
    int bad = 0;
    if (status == 0)
        for (int j = tid; j < m; j += NT_MASK) {
            const int p = a.parents[start + j];
            parent[j] = p;
            bad |= p < -1 || p >= j;
        }
    if (__syncthreads_or(bad)) status |= BAD_TREE;
    // the root's position, and the largest that m nodes can have
    const int kv = a.row_pos ? a.kv_lens[s] : m;
    const long long base = (long long)a.base_pos + kv - m;
    const bool placed = kv >= 0 && base >= 0 && base + m <= 1ll << 31;
    if (tid == 0) a.status[s] = status & BAD_ROWS || placed ? status : status | BAD_LENGTH;
    if (status & BAD_ROWS) return;
    for (int j = tid; j < m; j += NT_MASK) {
        uint32_t* out = a.masks + (long long)(start + j) * a.ld_mask;
        int at = a.words - 1, depth = -1;  // word that is written next
        uint32_t w = 0;
        if (status == 0) {
            for (int i = j; i >= 0; i = parent[i]) {
                for (; at > i >> 5; --at) {
                    out[at] = w;
                    w = 0;
                }
                w |= 1u << (i & 31);
                ++depth;
            }
        }
        for (; at >= 0; --at) {
            out[at] = w;
            w = 0;
        }
        if (a.depth) a.depth[start + j] = depth;
        if (a.row_pos) a.row_pos[start + j] = depth < 0 || !placed ? -1 : (int)(base + depth);
    }
}

__global__ void __launch_bounds__(NT_MASK) tree_accept_kernel(dflash_tree_accept_args a) {
    __shared__ int next[MAXN], path[MAXN];
    __shared__ int kept_s;
    const int s = blockIdx.x, tid = threadIdx.x;
    pdl_wait();
    pdl_trigger();
    int start, m;
    int status = rows_of(a.q_start, s, a.rows, start, m);
    if (status == 0 && m > MAXN) status = BAD_SIZE;
    const int nodes = status == 0 ? m : 0;
    for (int j = tid; j < nodes; j += NT_MASK) next[j] = MAXN;
    __syncthreads();
    int bad = 0;
    for (int j = tid; j < nodes; j += NT_MASK) {
        const int p = a.parents[start + j], token = a.tokens[start + j];
        if (p < -1 || p >= j) bad = 1;
        else if (p >= 0 && token == a.posterior[start + p])
            atomicMin(&next[p], j);
    }
    if (__syncthreads_or(bad)) status |= BAD_TREE;
    if (tid == 0) {
        int kept = 0;
        if (status == 0 && m > 0)
            for (int at = 0; at < MAXN && kept < a.width; at = next[at]) path[kept++] = at;
        kept_s = kept;
        a.status[s] = status;
        a.accepted[s] = kept - 1;
        a.bonus[s] = kept ? a.posterior[start + path[kept - 1]] : -1;
    }
    __syncthreads();
    for (int j = tid; j < a.width; j += NT_MASK) a.path[(long long)s * a.width + j] = j < kept_s ? path[j] : -1;
}

constexpr int NT_MOVE = 128, DEEP = 8;

// CTA (s, l): layer l / 2 of sequence s, keys or values.
__global__ void __launch_bounds__(NT_MOVE) kv_compact_kernel(dflash_kv_compact_args a, int vecs) {
    __shared__ int2 move[MAXN];  // token slots (64 * page + token) from and to, of the nodes that move
    __shared__ int count;
    const int s = blockIdx.x, tid = threadIdx.x;
    pdl_wait();
    pdl_trigger();
    int start, m;
    int status = rows_of(a.q_start, s, 0x7fffffff, start, m);
    const int kv = a.kv_lens[s], acc = a.accepted[s];
    if (status == 0 && (kv < m || kv > (long long)64 * a.width_table)) status = BAD_LENGTH;
    if (status == 0 && (acc < -1 || acc >= a.width)) status = BAD_TREE;
    const int kept = status == 0 ? acc + 1 : 0, first = kv - m;
    const int* path = a.path + (long long)s * a.width;
    const int* table = a.table + (long long)s * a.ld_table;
    int bad = 0;
    for (int j = tid; j < kept; j += NT_MOVE) {
        const int i = path[j], before = j ? path[j - 1] : -1;
        if (i <= before || i >= m || i < 0) {
            bad |= BAD_TREE;
        } else {
            int2 to = make_int2(-1, -1);
            if (i != j) {
                const int from_page = table[(first + i) >> 6], to_page = table[(first + j) >> 6];
                if (from_page < 0 || from_page >= a.n_pages || to_page < 0 || to_page >= a.n_pages) bad |= BAD_PAGE;
                to = make_int2(from_page * 64 + ((first + i) & 63), to_page * 64 + ((first + j) & 63));
            }
            move[j] = to;
        }
    }
    status |= __syncthreads_or(bad & BAD_TREE) ? BAD_TREE : 0;
    status |= __syncthreads_or(bad & BAD_PAGE) ? BAD_PAGE : 0;
    if (blockIdx.y == 0 && tid == 0) {
        a.status[s] = status;
        a.kv_out[s] = status ? kv : first + kept;
    }
    if (status) return;
    // the nodes that move are the last ones of the path: nodes in place are its first
    int still = 0;
    if (tid == 0) {
        while (still < kept && move[still].x < 0) ++still;
        count = still;
    }
    __syncthreads();
    still = count;
    char* cache = (char*)(blockIdx.y & 1 ? a.v_cache : a.k_cache) +
                  (long long)(blockIdx.y >> 1) * a.ld_layer * (a.dtype == DFLASH_DTYPE_BF16 ? 2 : 4);
    const long long row = (long long)vecs * 16;  // bytes of a head's token
    for (int u = tid; u < a.n_kv_heads * vecs; u += NT_MOVE) {
        const int h = u / vecs, c = u - h * vecs;
        auto at = [&](int slot) {
            return reinterpret_cast<uint4*>(cache + (((long long)(slot >> 6) * a.n_kv_heads + h) * 64 + (slot & 63)) * row) + c;
        };
        for (int j0 = still; j0 < kept; j0 += DEEP) {
            uint4 x[DEEP];
#pragma unroll
            for (int i = 0; i < DEEP; ++i)
                if (j0 + i < kept) x[i] = *at(move[j0 + i].x);
#pragma unroll
            for (int i = 0; i < DEEP; ++i)
                if (j0 + i < kept) *at(move[j0 + i].y) = x[i];
        }
    }
}

}  // namespace

}  // namespace dfl

using namespace dfl;

extern "C" dflash_status dflash_tree_masks(const dflash_tree_masks_args* p, void* cuda_stream) {
    if (!p) return refuse("tree_masks: args is NULL");
    const dflash_tree_masks_args& a = *p;
    if (a.batch < 1 || a.batch > DFLASH_OPS_MAX_BATCH) return refuse("tree_masks: batch outside [1, 2048]");
    if (a.rows < 0 || a.rows > (1 << 20)) return refuse("tree_masks: rows outside [0, 2^20]");
    if (a.words < 1 || a.words > (1 << 20) || a.ld_mask < a.words)
        return refuse("tree_masks: words outside [1, 2^20], or ld_mask smaller");
    if (a.base_pos < 0 || a.base_pos > (1 << 30)) return refuse("tree_masks: base_pos outside [0, 2^30]");
    if (!a.q_start || !a.status || (a.rows > 0 && (!a.parents || !a.masks)) || (a.row_pos && !a.kv_lens))
        return refuse("tree_masks: NULL argument");
    return queue(cuda_stream, "tree_masks: launch failed",
                 [&](const Launch& L) { launch_k(L, tree_masks_kernel, dim3(a.batch), dim3(NT_MASK), 0, 1, a); });
}

extern "C" dflash_status dflash_tree_accept(const dflash_tree_accept_args* p, void* cuda_stream) {
    if (!p) return refuse("tree_accept: args is NULL");
    const dflash_tree_accept_args& a = *p;
    if (a.batch < 1 || a.batch > DFLASH_OPS_MAX_BATCH) return refuse("tree_accept: batch outside [1, 2048]");
    if (a.rows < 0 || a.rows > (1 << 20)) return refuse("tree_accept: rows outside [0, 2^20]");
    if (a.width < 1 || a.width > MAXN) return refuse("tree_accept: width outside [1, 1024]");
    if (a.reserved != 0) return refuse("tree_accept: reserved must be 0");
    if (!a.q_start || !a.path || !a.accepted || !a.bonus || !a.status ||
        (a.rows > 0 && (!a.parents || !a.tokens || !a.posterior)))
        return refuse("tree_accept: NULL argument");
    return queue(cuda_stream, "tree_accept: launch failed",
                 [&](const Launch& L) { launch_k(L, tree_accept_kernel, dim3(a.batch), dim3(NT_MASK), 0, 1, a); });
}

extern "C" dflash_status dflash_kv_compact(const dflash_kv_compact_args* p, void* cuda_stream) {
    if (!p) return refuse("kv_compact: args is NULL");
    const dflash_kv_compact_args& a = *p;
    if (const char* why = bad_caches(a, "kv_compact: dtype must be F32 or BF16", "kv_compact: layers outside [1, 1024]",
                                     "kv_compact: n_pages, n_kv_heads or head_dim out of range (a head's row is a multiple of 16 bytes)",
                                     "kv_compact: the caches must be 16-byte aligned, ld_layer a multiple of 16 bytes and no smaller than a layer"))
        return refuse(why);
    // (their tokens would be moved twice)
    if (a.k_cache == a.v_cache) return refuse("kv_compact: v_cache may not be k_cache");
    if (caches_overlap(a)) return refuse("kv_compact: k_cache and v_cache overlap");
    if (a.batch < 1 || a.batch > DFLASH_OPS_MAX_BATCH) return refuse("kv_compact: batch outside [1, 2048]");
    if (a.width < 1 || a.width > MAXN) return refuse("kv_compact: width outside [1, 1024]");
    if (a.width_table < 0 || a.width_table > (1 << 22) || a.ld_table < a.width_table)
        return refuse("kv_compact: width_table outside [0, 2^22], or ld_table smaller");
    if (!a.kv_lens || !a.q_start || !a.path || !a.accepted || !a.kv_out || !a.status || (a.width_table > 0 && !a.table))
        return refuse("kv_compact: NULL argument");
    if (a.kv_out == a.kv_lens) return refuse("kv_compact: kv_out may not be kv_lens");
    const int vecs = a.head_dim * (a.dtype == DFLASH_DTYPE_BF16 ? 2 : 4) / 16;
    return queue(cuda_stream, "kv_compact: launch failed", [&](const Launch& L) {
        launch_k(L, kv_compact_kernel, dim3(a.batch, 2 * a.layers), dim3(NT_MOVE), 0, 1, a, vecs);
    });
}
