// Attention of a batch that shares a prefix (dflash_shared_prefix_attention in
// include/dflash.h) and of trees of drafted tokens (dflash_tree_attention): the
// entries, their checks, and the merge of the partial results
// that the main kernels (attention_shared_tc.cu for bf16, attention_shared_f32.cu)
// leave per segment of the plan (shared_plan.cuh).
//
// What a call cannot do without: the prefix's keys and values once per call (not
// once per sequence: 2 * H_kv * hd * prefix_len elements), each sequence's own
// keys and values once, q and out once, and 4 * hd operations per query vector
// and key.
#include <math.h>
#include <stdio.h>
#include <string.h>

#include <algorithm>

#include "shared_plan.cuh"
#include "tcgen05.cuh"

namespace dfl {

namespace {

// Merge of the partial results: out = sum_i 2^(m_i - M) o_i / sum_i 2^(m_i - M) l_i over the segments that
// hold the row's query vectors, prefix and own, in plan order (one fixed order: the same bits every run).
// A warp takes one row and one KV head (or 32 elements of them), whose blocks the main kernel has written down
// (Dir); lanes take 8 head dimensions of one query vector each (whole 32-byte sectors) and stream the segments through,
// four in flight.  NW > 1: the warps of a CTA share one (row, KV head), by elements and by segments, for calls of few rows
// (whose prefix is split the most).  Bytes: 4 hd + 8 per vector and segment, from L2; a small call
// waits for its chain of loads and, as much, for the code itself to come from L2 (hence rolled loops).  Consecutive
// lanes take the heads of a row, then the next 8 dimensions: a load of 32 lanes then takes whole 128-byte lines of
// the partials (32 prompts of 5 .. 130 rows: the call 127 -> 121 us).  Measured under a profiler: 12 us for 512 rows of
// 32 heads, 25 us for 2160.
struct MergeArgs {
    sp::Shape P;
    sp::Work W;
    void* out;
    float* lse;
    long long ld_out;
    uint32_t* report;  // the session's error word, or null
    int warps;         // NW == 1: warps per (row, KV head), by elements
};

constexpr int MWARPS = 8;

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

// (M, l, o) of two disjoint sets of keys joined into the first.
struct Part {
    float M = -INFINITY, l = 0.f, o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    __device__ __forceinline__ void join(float m, float s, const float4& x, const float4& y) {
        const float mn = fmaxf(M, m);
        const float e0 = M == -INFINITY ? 0.f : exp2f(M - mn), e1 = m == -INFINITY ? 0.f : exp2f(m - mn);
        M = mn;
        l = l * e0 + s * e1;
        const float v[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = o[e] * e0 + v[e] * e1;
    }
};

template <typename T, int NW>
__global__ void __launch_bounds__(32 * MWARPS, 3) merge_kernel(MergeArgs a) {
    using namespace sp;
    const Shape& P = a.P;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int unit = blockIdx.x * MWARPS + warp;
    const int r = NW > 1 ? blockIdx.x : unit / a.warps, kvh = blockIdx.y;
    __shared__ Part part_s[NW > 1 ? NW : 1][32];
    if (r >= P.rows) return;  // (NW > 1: the whole CTA)
    pdl_wait();
    pdl_trigger();
    const Dir d = a.W.dir[(size_t)r * P.Hkv + kvh];
    uint32_t err = 0;
#pragma unroll
    for (int i = 0; i < 5; ++i)
        if (lane + 32 * i < P.n_cta) err |= a.W.err[lane + 32 * i];
    if (d.pre_count == -1) return;  // a row of no sequence
    const bool late = __any_sync(0xffffffffu, err != 0), bad = late || d.pre_count == -2;
    if (late && a.report && lane == 0) atomicOr(a.report, ERR_TIMEOUT);
    const int count = bad ? 0 : d.pre_count + d.own_count;
    const int chunks = P.hd / 8, elems = P.g * chunks;
    // Warp we of `shares` takes every shares-th 32 elements; NW > 1: of the CTA's warps, warp w0 of each such group every
    // splits-th segment from w0 on.
    const int shares = NW > 1 ? min(cdiv(elems, 32), NW) : a.warps, splits = NW > 1 ? NW / shares : 1;
    const int w0 = NW > 1 ? warp / shares : 0, we = NW > 1 ? warp - w0 * shares : unit - r * a.warps;
#pragma unroll 1
    for (int eb = 0; eb < elems; eb += 32 * shares) {
        const int e0 = eb + 32 * we;
        if (NW == 1 && e0 >= elems) break;
        const int e = min(e0 + lane, elems - 1), c8 = e / P.g, hh = e - c8 * P.g;
        Part acc;
        uint32_t bb = 0;
#pragma unroll 1
        for (int k0 = w0; k0 < (w0 < splits ? count : 0); k0 += 4 * splits) {
            float2 ml[4];
            float4 x[4], y[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int k = k0 + i * splits;
                ml[i] = make_float2(-INFINITY, 0.f);
                x[i] = y[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (k < count) {
                    const bool p = k < d.pre_count;
                    const size_t blk = p ? d.pre_block + k * d.pre_step : d.own_block + (k - d.pre_count) * d.own_step;
                    const int v = (p ? d.pre_v : d.own_v) + hh;
                    ml[i] = a.W.ml[blk * P.VT + v];
                    const float* src = a.W.o + ((blk * chunks + c8) * P.VT + v) * 8;
                    x[i] = *reinterpret_cast<const float4*>(src);
                    y[i] = *reinterpret_cast<const float4*>(src + 4);
                    bb |= a.W.block_bad[blk];
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) acc.join(ml[i].x, ml[i].y, x[i], y[i]);
        }
        if (bb) acc.M = NAN;  // (a NaN maximum makes the whole row NaN below)
        if (NW > 1) {
            part_s[warp][lane] = acc;
            __syncthreads();
            if (w0 == 0)
#pragma unroll 1
                for (int q = 1; q < splits; ++q) {
                    const Part p = part_s[warp + q * shares][lane];
                    if (isnan(p.M) || isnan(acc.M)) acc.M = NAN;
                    else
                        acc.join(p.M, p.l, make_float4(p.o[0], p.o[1], p.o[2], p.o[3]),
                                 make_float4(p.o[4], p.o[5], p.o[6], p.o[7]));
                }
        }
        if (w0 == 0 && e0 + lane < elems) {
            const int head = kvh * P.g + hh;
            const bool nan = bad || isnan(acc.M);
            const float inv = acc.l == 0.f ? 0.f : 1.f / acc.l;  // (no key: 0; a NaN sum stays NaN)
#pragma unroll
            for (int i = 0; i < 8; ++i) acc.o[i] = nan ? NAN : acc.o[i] * inv;
            store8<T>(reinterpret_cast<T*>(a.out) + (long long)r * a.ld_out + (long long)head * P.hd + c8 * 8, acc.o);
            if (a.lse && c8 == 0)
                a.lse[(long long)r * P.H + head] =
                    nan ? NAN : acc.l == 0.f ? -INFINITY : (acc.M + log2f(acc.l)) * 0.6931471805599453f;
        }
        if (NW > 1) __syncthreads();
    }
}

}  // namespace

bool shared_attention_tc(const Launch& L, const sp::Shape& P, const sp::Work& W, const dflash_shared_prefix_args& a);
bool shared_attention_f32(const Launch& L, const sp::Shape& P, const sp::Work& W, const dflash_shared_prefix_args& a);

namespace {

constexpr int CTAS = 152;  // one per SM

// Query vectors of a worker (fp32: figures in attention_shared_f32.cu).
int vectors_of(bool f32, int g, int batch, int rows) { return !f32 ? 128 : (long long)rows * g > 32ll * batch ? 64 : 32; }

// The sizes alone (what the workspace depends on).
sp::Shape sizes_of(bool f32, int VT, int H, int Hkv, int hd, int batch, int rows) {
    sp::Shape P = {};
    P.H = H;
    P.g = H / Hkv;
    P.VT = VT;
    P.parts = 1;
    while (P.g % P.parts || P.g / P.parts > P.VT) ++P.parts;
    P.Hkv = Hkv * P.parts;
    P.g /= P.parts;
    P.hd = hd;
    P.RH = P.VT / P.g;
    P.KT = f32 ? 32 : 64;
    P.one_line = f32;
    P.batch = batch;
    P.rows = rows;
    P.n_cta = CTAS;
    // an item's fixed cost: four tiles on line 0, three on line 1 (32 prompts of 5 .. 130 rows behind 2100 keys: 114 us
    // with these, 130 with two on line 1, 112 with three on line 0, where blocks of 16 then take 22.6 instead of 21.5 us)
    P.lead[0] = 4;
    P.lead[1] = f32 ? 1 : 3;
    return P;
}

template <typename T>
void merge(const Launch& L, const MergeArgs& m) {
    // the merge starts as the main kernel's CTAs leave
    Launch after = L;
    after.pdl = true;
    // Rows of one stream: the prefix is split over nearly every worker of its line, else over a few.  (One token of four
    // sequences behind 512 keys: 10.3 us with eight warps, 11.0 with a warp per 32 elements, fp32 blocks of four 9.8 and
    // 12.0; verify blocks 32 x 16: 110 and 95 us.)
    if (m.P.rows <= m.P.RH) {
        launch_k(after, merge_kernel<T, MWARPS>, dim3(m.P.rows, m.P.Hkv), dim3(32 * MWARPS), 0, 1, m);
        return;
    }
    // A warp per 32 elements while that is at most seven CTAs an SM, else one per (row, KV head).  (Blocks of 16 of 8
    // sequences behind 1000 keys: 17.0 and 19.4 us; 32 prompts of 5 .. 130 rows behind 2100: 114.4 and 111.0.)
    MergeArgs a = m;
    const int shares = (m.P.g * m.P.hd / 8 + 31) / 32;
    auto ctas = [&](int w) { return (int)(((long long)m.P.rows * w + MWARPS - 1) / MWARPS); };
    if ((long long)ctas(shares) * m.P.Hkv <= 7 * CTAS) a.warps = shares;
    launch_k(after, merge_kernel<T, 1>, dim3(ctas(a.warps), m.P.Hkv), dim3(32 * MWARPS), 0, 1, a);
}

}  // namespace

bool shared_prefix_attention(const Launch& L, const dflash_shared_prefix_args& a, const TreeMasks* tree) {
    const bool f32 = a.dtype == DFLASH_DTYPE_F32;
    MergeArgs m;
    sp::Shape& P = m.P;
    P = sizes_of(f32, vectors_of(f32, a.n_heads / a.n_kv_heads, a.batch, a.rows), a.n_heads, a.n_kv_heads, a.head_dim, a.batch, a.rows);
    P.width = a.width;
    P.prefix_len = a.prefix_len;
    P.causal = a.causal != 0 && !tree;
    P.n_pages = a.n_pages;
    P.npt = (a.prefix_len + P.KT - 1) / P.KT;
    P.ld_table = a.ld_table;
    P.prefix_pages = a.prefix_pages;
    P.table = a.table;
    P.kv_lens = a.kv_lens;
    P.q_start = a.q_start;
    if (tree) {
        P.masks = tree->masks;
        P.ld_mask = tree->ld_mask;
        P.words = tree->words;
    }
    sp::layout((char*)a.workspace, P, &m.W);
    m.out = a.out;
    m.lse = a.lse;
    m.ld_out = a.ld_out;
    m.report = L.err;
    m.warps = 1;
    if (!(f32 ? shared_attention_f32(L, P, m.W, a) : shared_attention_tc(L, P, m.W, a))) return false;
    if (f32) merge<float>(L, m);
    else merge<bf16>(L, m);
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
    if (a.flags & ~DFLASH_ATTENTION_WEIGHT_PAIRS) return bad("shared_prefix_attention: flags holds an unknown one");
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
    // (the larger of fp32's two forms: no call with fewer rows or sequences needs more)
    auto bytes = [&](bool f32, int VT) {
        return sp::layout(nullptr, sizes_of(f32, VT, n_heads, n_kv_heads, head_dim, batch, rows), nullptr);
    };
    return dtype == DFLASH_DTYPE_F32 ? std::max(bytes(true, 32), bytes(true, 64)) : bytes(false, 128);
}

namespace {

dflash_status attend(const dflash_shared_prefix_args& a, const TreeMasks* tree, void* cuda_stream, const char* unprepared) {
    if (a.rows == 0) return DFLASH_OK;
    return queue(cuda_stream, unprepared, [&](const Launch& L) {
        if (!shared_prefix_attention(L, a, tree)) L.fail();
    });
}

}  // namespace

extern "C" dflash_status dflash_shared_prefix_attention(const dflash_shared_prefix_args* p, void* cuda_stream) {
    const char* why = "shared_prefix_attention: args is NULL";
    if (!p || check_shared_prefix(*p, &why) != DFLASH_OK) return refuse(why);
    return attend(*p, nullptr, cuda_stream, "shared_prefix_attention: a kernel could not be prepared");
}

extern "C" dflash_status dflash_tree_attention(const dflash_tree_attention_args* p, void* cuda_stream) {
    if (!p) return refuse("tree_attention: args is NULL");
    const char* why = "";
    if (check_shared_prefix(p->attn, &why) != DFLASH_OK) {
        // the same checks, in this call's name
        char text[256];
        const char* at = strchr(why, ':');
        snprintf(text, sizeof text, "tree_attention%s", at ? at : "");
        return refuse(text);
    }
    if (p->words < 1 || p->words > (1 << 20)) return refuse("tree_attention: words outside [1, 2^20]");
    if (p->reserved != 0) return refuse("tree_attention: reserved must be 0");
    if (p->attn.rows > 0 && !p->masks) return refuse("tree_attention: masks is NULL");
    if (p->ld_mask < p->words) return refuse("tree_attention: ld_mask is smaller than words");
    const TreeMasks tree = {p->masks, p->ld_mask, p->words};
    return attend(p->attn, &tree, cuda_stream, "tree_attention: a kernel could not be prepared");
}
