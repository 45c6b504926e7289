// How the shared-prefix attention divides its work: the arithmetic that the
// attention kernels and the merge kernel have in common.
//
// An item is one KV head's query vectors of a few rows (g heads each) against
// one key list: the prefix items (a row tile of the whole batch x KV head,
// against the prefix) and the own items (a row tile of one sequence x KV head,
// against the sequence's own keys).  A worker has VT vectors per stream; items
// of more than one stream's rows (RH) go on line 0, whose workers are the CTAs
// with both streams in step over the same tiles, the others on line 1, whose
// workers are the single streams.  A line strings its items up, prefix first,
// each with one weight w per tile of KT keys after a lead weight for its fixed
// cost (queries in, partial result out).  The line [0, W) is cut into equal
// parts, one per worker: a tile belongs to the worker in whose part its first
// unit lies.  So every worker gets the same work whatever the lengths are, and
// an item is split over no more workers than its weight takes.  A worker's run
// of tiles inside one item is a segment; its partial result (per vector:
// maximum, sum, unnormalised output) goes to a block of the workspace numbered
// by item + worker: along a line neither ever falls and one of them rises at
// each segment, so blocks are unique.
#pragma once

#include "ops.h"

namespace dfl {
namespace sp {

constexpr int MAX_BATCH = DFLASH_OPS_MAX_BATCH;

struct Shape {
    int H, Hkv, g, hd;
    int VT;        // query vectors per stream
    int RH;        // rows per stream: VT / g
    int KT;        // keys per tile
    int batch, rows, width, prefix_len, causal, n_pages;
    int npt;       // prefix tiles
    int n_cta;
    int w, lead[2];  // weights of a tile and of an item's fixed cost (per line)
    long long ld_table;
    const int *prefix_pages, *table, *kv_lens, *q_start;
    __host__ __device__ int row_tile(int line) const { return line == 0 ? 2 * RH : RH; }
    __host__ __device__ int workers(int line) const { return line == 0 ? n_cta : 2 * n_cta; }
};

// Cut of the lines, written by CTA 0 for the merge kernel.
struct Head {
    uint32_t W[2];     // total weights
    uint32_t CP;       // weight of the prefix items, at the start of line pl
    uint32_t items0;   // items on line 0
    int pl;            // line of the prefix items
    int n_prefix;      // prefix items
    int r_begin, r_end;
    int nqt;           // row tiles of the batch on line pl
    int bad;           // q_start is not a list of rows, or a line is too long
};

struct Work {
    Head* head;
    uint32_t* err;        // [n_cta]: a bounded wait ran out
    uint32_t* base;       // [batch]: first unit of the sequence's own items on its line
    uint32_t* ibase;      // [batch]: first of the sequence's own items on its line
    uint32_t* block_bad;  // [blocks]: a page of the segment lies outside the cache
    float2* ml;           // [blocks][VT]
    float* o;             // [blocks][hd / 8][VT][8]
};

// Blocks: line 0 takes two per (item, worker), line 1 one.
inline long long max_blocks(const Shape& P) {
    const long long RT = 2 * P.RH;
    // prefix row tiles; own items: every sequence adds at most one partial row tile to the full ones
    const long long items = P.Hkv * ((P.rows + RT - 1) / RT + P.rows / RT + (P.batch < P.rows ? P.batch : P.rows));
    return 2 * (items + P.n_cta) + 2 * P.n_cta;
}

inline size_t layout(char* p, const Shape& P, Work* w) {
    size_t at = 0;
    auto take = [&](size_t bytes) {
        char* q = p + at;
        at += (bytes + 255) / 256 * 256;
        return q;
    };
    const size_t blocks = (size_t)max_blocks(P);
    Work x;
    x.head = (Head*)take(sizeof(Head));
    x.err = (uint32_t*)take((size_t)P.n_cta * 4);
    x.base = (uint32_t*)take((size_t)P.batch * 4);
    x.ibase = (uint32_t*)take((size_t)P.batch * 4);
    x.block_bad = (uint32_t*)take(blocks * 4);
    x.ml = (float2*)take(blocks * P.VT * 8);
    x.o = (float*)take(blocks * P.VT * P.hd * 4);
    if (w) *w = x;
    return at;
}

__device__ __forceinline__ uint32_t part_begin(uint32_t W, int c, int n) {
    return (uint32_t)((unsigned long long)W * (unsigned)c / (unsigned)n);
}
// The worker whose part holds unit x < W: the last c with floor(c W / n) <= x.
__device__ __forceinline__ int owner(uint32_t W, uint32_t x, int n) {
    return (int)((((unsigned long long)x + 1) * (unsigned)n + W - 1) / W) - 1;
}
__device__ __forceinline__ int cdiv(int a, int b) { return (a + b - 1) / b; }
// Tiles [t0, t1) of an item of n tiles at unit b that lie in the part [lo, hi), lo >= b.
__device__ __forceinline__ void cut(uint32_t lo, uint32_t hi, uint32_t b, uint32_t lead, uint32_t w, int n, int& t0, int& t1) {
    const uint32_t x = lo - b, y = hi > b ? hi - b : 0u;
    t0 = x <= lead ? 0 : (int)((x - lead + w - 1) / w);
    t1 = y <= lead ? 0 : (int)min((uint32_t)n, (y - lead + w - 1) / w);
}
// First block of worker c's segment of item `id`.
__device__ __forceinline__ uint32_t block_of(const Shape& P, const Head& h, int line, int id, int c) {
    return line == 0 ? 2u * (uint32_t)(id + c) : 2u * (h.items0 + (uint32_t)P.n_cta) + (uint32_t)(id + c);
}

// A sequence's own items: m rows, kv keys (0 tiles for lengths out of range).
struct Seq {
    int m, kv, tiles, groups, line;
};
__device__ __forceinline__ Seq seq_of(const Shape& P, int start, int end, int kv) {
    Seq q;
    q.m = end - start;
    q.kv = kv;
    q.line = q.m > P.RH ? 0 : 1;
    const bool ok = q.m > 0 && kv > 0 && kv <= (long long)64 * P.width;
    q.tiles = ok ? cdiv(kv, P.KT) : 0;
    q.groups = q.tiles ? cdiv(q.m, P.row_tile(q.line)) : 0;
    return q;
}
// Own tiles that the rows [.., r1) of a sequence of m rows see.
__device__ __forceinline__ int seen_tiles(const Shape& P, const Seq& q, int r1) {
    return P.causal ? min(q.tiles, cdiv(max(q.kv - q.m + r1, 0), P.KT)) : q.tiles;
}

struct Seg {
    int seq;          // -1: prefix
    int kvh;
    int row0, nrows;  // rows of q
    int t0, t1;       // tiles
    int keys;         // keys of the list (prefix_len or kv)
    int lim0;         // keys seen by row row0 (causal own keys: one more per row)
    bool causal;
    uint32_t block;
};

// Walks the segments of worker `c` on a line.  base / ibase: see make_plan.
struct Walk {
    uint32_t p, p1;
    int line, c;
    __device__ __forceinline__ Walk(const Shape& P, const Head& h, int ln, int worker)
        : p(part_begin(h.W[ln], worker, P.workers(ln))), p1(part_begin(h.W[ln], worker + 1, P.workers(ln))), line(ln), c(worker) {}

    __device__ __forceinline__ bool next(const Shape& P, const Head& h, const uint32_t* base, const uint32_t* ibase, Seg& s) {
        const uint32_t w = P.w, lead = P.lead[line];
        const int RT = P.row_tile(line);
        base += line * MAX_BATCH;
        while (p < p1) {
            uint32_t b;
            int n, n_eff, id;
            if (h.pl == line && p < h.CP) {
                const uint32_t per = lead + (uint32_t)P.npt * w;
                id = (int)(p / per);
                b = (uint32_t)id * per;
                n = n_eff = P.npt;
                s.seq = -1;
                s.kvh = id / h.nqt;
                s.row0 = h.r_begin + id % h.nqt * RT;
                s.nrows = min(RT, h.r_end - s.row0);
                s.keys = s.lim0 = P.prefix_len;
                s.causal = false;
            } else {
                int lo = 0, hi = P.batch;  // the last sequence with base <= p has items here (base rises over it alone)
                while (hi - lo > 1) {
                    const int mid = (lo + hi) >> 1;
                    if (base[mid] <= p) lo = mid;
                    else hi = mid;
                }
                const int start = P.q_start[lo];
                const Seq q = seq_of(P, start, P.q_start[lo + 1], P.kv_lens[lo]);
                const uint32_t per = lead + (uint32_t)q.tiles * w;
                const int k = (int)((p - base[lo]) / per);
                b = base[lo] + (uint32_t)k * per;
                n = q.tiles;
                const int gi = k % q.groups;
                id = (h.pl == line ? h.n_prefix : 0) + (int)ibase[lo] + k;
                s.seq = lo;
                s.kvh = k / q.groups;
                s.row0 = start + gi * RT;
                s.nrows = min(RT, q.m - gi * RT);
                s.keys = q.kv;
                s.causal = P.causal != 0;
                s.lim0 = P.causal ? q.kv - q.m + gi * RT + 1 : q.kv;
                n_eff = seen_tiles(P, q, gi * RT + s.nrows);
            }
            int t1;
            cut(p, p1, b, lead, w, n, s.t0, t1);
            s.t1 = min(t1, n_eff);
            s.block = block_of(P, h, line, id, c);
            p = min(p1, b + lead + (uint32_t)n * w);
            if (s.t0 < s.t1) return true;
        }
        return false;
    }
};

// Scan of the batch by every thread of the CTA (NTHR threads, all call it): fills base ([2][MAX_BATCH]:
// per line, the exclusive sums of the own items' weights, from the prefix items' end), ibase ([batch]: of
// the counts on the sequence's line) and the head.  ws: 4 * NTHR / 32 words, flag: one word (shared
// memory).  Ends with a barrier.
template <int NTHR>
__device__ void make_plan(const Shape& P, uint32_t* base, uint32_t* ibase, uint32_t* ws, int* flag, Head& h) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    constexpr unsigned long long MOST = 1ull << 31;  // sums saturate here: the call is bad then
    if (tid == 0) *flag = 0;
    __syncthreads();
    h.r_begin = P.q_start[0];
    h.r_end = P.q_start[P.batch];
    int bad = 0;
    if (h.r_begin < 0 || h.r_end < h.r_begin || h.r_end > P.rows) {
        bad = 1;
        h.r_begin = h.r_end = 0;
    }
    const int live = h.r_end - h.r_begin;
    h.pl = live > P.RH ? 0 : 1;
    h.nqt = cdiv(live, P.row_tile(h.pl));
    h.n_prefix = P.npt ? h.nqt * P.Hkv : 0;
    unsigned long long cp = (unsigned long long)h.n_prefix * (P.lead[h.pl] + (unsigned long long)P.npt * P.w);
    if (cp >= MOST) {
        bad = 1;
        cp = 0;
    }
    h.CP = (uint32_t)cp;
    unsigned long long carry[2] = {h.pl == 0 ? cp : 0ull, h.pl == 1 ? cp : 0ull};
    uint32_t icarry[2] = {0u, 0u};
    for (int s0 = 0; s0 < P.batch; s0 += NTHR) {
        const int s = s0 + tid;
        unsigned long long c[2] = {0ull, 0ull};
        uint32_t it[2] = {0u, 0u};
        int line = 0;
        if (s < P.batch) {
            const int a = P.q_start[s], b = P.q_start[s + 1];
            if (a < 0 || b < a || b > P.rows) {
                bad = 1;
            } else {
                const Seq q = seq_of(P, a, b, P.kv_lens[s]);
                line = q.line;
                const uint32_t items = (uint32_t)(q.groups * P.Hkv);
                const unsigned long long cost = (unsigned long long)items * (P.lead[line] + (unsigned long long)q.tiles * P.w);
                if (cost >= MOST) bad = 1;
                else {
                    c[line] = cost;
                    it[line] = items;
                }
            }
        }
        unsigned long long ci[2];
        uint32_t ii[2];
#pragma unroll
        for (int l = 0; l < 2; ++l) {
            ci[l] = c[l];
            ii[l] = it[l];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const unsigned long long x = __shfl_up_sync(0xffffffffu, ci[l], o);
                const uint32_t y = __shfl_up_sync(0xffffffffu, ii[l], o);
                if (lane >= o) {
                    ci[l] = min(ci[l] + x, MOST);
                    ii[l] += y;
                }
            }
            if (lane == 31) {
                ws[4 * warp + 2 * l] = (uint32_t)ci[l];
                ws[4 * warp + 2 * l + 1] = ii[l];
            }
        }
        __syncthreads();
        unsigned long long before[2] = {0ull, 0ull};
        uint32_t ibefore[2] = {0u, 0u};
        for (int w = 0; w < NTHR / 32; ++w)
#pragma unroll
            for (int l = 0; l < 2; ++l) {
                if (w == warp) {
                    before[l] = carry[l];
                    ibefore[l] = icarry[l];
                }
                carry[l] = min(carry[l] + ws[4 * w + 2 * l], MOST);
                icarry[l] += ws[4 * w + 2 * l + 1];
            }
        if (s < P.batch) {
#pragma unroll
            for (int l = 0; l < 2; ++l) base[l * MAX_BATCH + s] = (uint32_t)min(before[l] + ci[l] - c[l], MOST);
            ibase[s] = line == 0 ? ibefore[0] + ii[0] - it[0] : ibefore[1] + ii[1] - it[1];
        }
        __syncthreads();
    }
    if (carry[0] >= MOST || carry[1] >= MOST) bad = 1;
    if (bad) *flag = 1;
    __syncthreads();
    h.bad = *flag;
    h.W[0] = h.bad ? 0u : (uint32_t)carry[0];
    h.W[1] = h.bad ? 0u : (uint32_t)carry[1];
    h.items0 = icarry[0] + (h.pl == 0 ? (uint32_t)h.n_prefix : 0u);
}

}  // namespace sp
}  // namespace dfl
