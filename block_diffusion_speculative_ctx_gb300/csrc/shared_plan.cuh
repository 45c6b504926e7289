// How the shared-prefix attention divides its work: the arithmetic that the
// attention kernels and the merge kernel have in common.
//
// An item is one KV head's query vectors of a few rows (g heads each) against
// one key list: the prefix items (a row tile of the whole batch x KV head,
// against the prefix) and the own items (a row tile of one sequence x KV head,
// against the sequence's own keys).  A worker has VT vectors per stream; items
// of more than one stream's rows (RH) go on line 0, whose workers are the CTAs
// with both streams in step over the same tiles, the others on line 1, whose
// workers are the single streams.  A line strings its items up, prefix first:
// an item takes a lead (its fixed cost: queries in, partial result out) and one
// unit per tile of KT keys that it has.  The line is cut into parts of equal
// length, one per worker, so every worker gets the same work whatever the
// lengths are, and an item is split over no more workers than its length takes.
// A worker's run of tiles inside one item is a segment; its partial result (per
// vector: maximum, sum, unnormalised output) goes to a block of the workspace
// numbered by item + worker: along a line neither ever falls and one of them
// rises at each segment, so blocks are unique, and an item's are consecutive.
#pragma once

#include "ops.h"

namespace dfl {
namespace sp {

struct Shape {
    int H, Hkv, g, hd;
    int VT;        // query vectors per stream
    int RH;        // rows per stream: VT / g
    int KT;        // keys per tile
    int batch, rows, width, prefix_len, causal, n_pages;
    int npt;       // prefix tiles
    int n_cta;
    int lead[2];   // an item's fixed cost in tiles (per line)
    int one_line;  // every item on line 1, row tiles of one stream
    int parts;     // KV heads here per KV head of the caches (more query heads than VT are split)
    long long ld_table;
    const int *prefix_pages, *table, *kv_lens, *q_start;
    __host__ __device__ int row_tile(int line) const { return line == 0 ? 2 * RH : RH; }
};

// Cut of the lines.
struct Head {
    uint32_t W[2];     // length
    uint32_t part[2];  // length of a worker's part: ceil(W / workers)
    int n1;            // CTAs on line 1 (two workers each); the others are on line 0
    uint32_t CP;       // length of the prefix items, at the start of line pl
    uint32_t items0;   // items on line 0
    int pl;            // line of the prefix items
    int n_prefix;      // prefix items
    int r_begin, r_end;
    int nqt;           // row tiles of the batch on line pl
    int bad;           // q_start is not a list of rows, or a line is too long
};

// Where the partial results of one row and KV head lie: blocks (first, count, step) and the row's first
// vector in them, of its prefix item and its own.  pre_count -1: a row of no sequence; -2: NaN.
struct Dir {
    int pre_block, pre_count, own_block, own_count;
    int pre_v, own_v, pre_step, own_step;
};

struct Work {
    uint32_t* err;        // [n_cta]: a bounded wait ran out
    Dir* dir;             // [rows][Hkv]
    uint32_t* block_bad;  // [blocks]: a page of the segment lies outside the cache
    float2* ml;           // [blocks][VT]
    float* o;             // [blocks][hd / 8][VT][8]
};

// Blocks: line 0 takes two per (item, worker), line 1 one.
inline long long max_blocks(const Shape& P) {
    const long long RT = P.row_tile(P.one_line);
    // prefix row tiles; own items: every sequence adds at most one partial row tile to the full ones
    const long long items = P.Hkv * ((P.rows + RT - 1) / RT + P.rows / RT + (P.batch < P.rows ? P.batch : P.rows));
    return (P.one_line ? items + 2 * P.n_cta : 2 * (items + P.n_cta)) + 2 * P.n_cta;
}

// Its sections begin on multiples of 256 bytes wherever the workspace itself begins (partial results are stored 32 bytes
// at a time); the size has room for that.
constexpr size_t ALIGN = 256;
inline size_t layout(char* p, const Shape& P, Work* w) {
    p = (char*)(((uintptr_t)p + ALIGN - 1) / ALIGN * ALIGN);
    size_t at = 0;
    auto take = [&](size_t bytes) {
        char* q = p + at;
        at += (bytes + ALIGN - 1) / ALIGN * ALIGN;
        return q;
    };
    const size_t blocks = (size_t)max_blocks(P);
    Work x;
    x.err = (uint32_t*)take((size_t)P.n_cta * 4);
    x.dir = (Dir*)take((size_t)P.rows * P.Hkv * sizeof(Dir));
    x.block_bad = (uint32_t*)take(blocks * 4);
    x.ml = (float2*)take(blocks * P.VT * 8);
    x.o = (float*)take(blocks * P.VT * P.hd * 4);
    if (w) *w = x;
    return at + ALIGN;
}

__device__ __forceinline__ int cdiv(int a, int b) { return (a + b - 1) / b; }
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
    q.line = q.m > P.RH && !P.one_line ? 0 : 1;
    const bool ok = q.m > 0 && kv > 0 && kv <= (long long)64 * P.width;
    q.tiles = ok ? cdiv(kv, P.KT) : 0;
    q.groups = q.tiles ? cdiv(q.m, P.row_tile(q.line)) : 0;
    return q;
}
// Own tiles that the rows [.., r1) of a sequence of m rows see.
__device__ __forceinline__ int seen_tiles(const Shape& P, const Seq& q, int r1) {
    return P.causal ? min(q.tiles, cdiv(max(q.kv - q.m + r1, 0), P.KT)) : q.tiles;
}

// What the roles need to know of a segment; n == 0: no more.
struct Seg {
    int n;            // tiles
    int t0;           // the first of them
    int keys;         // keys of the list (prefix_len or kv)
    int lim0;         // keys seen by the item's first row
    int step;         // and by each row more (causal own keys: 1, else 0)
    int nrows;        // rows of the item
    uint32_t block;
};

// Walks the segments of worker `c` on a line.  base / ibase: see make_plan.
struct Walk {
    uint32_t p, p1;
    int line, c;
    __device__ __forceinline__ Walk(const Shape& P, const Head& h, int ln, int worker)
        : p(min(h.W[ln], (uint32_t)worker * h.part[ln])), p1(min(h.W[ln], p + h.part[ln])), line(ln), c(worker) {}

    // The next segment, its KV head, first row of q and sequence (-1: prefix).
    __device__ __forceinline__ bool next(const Shape& P, const Head& h, const uint32_t* base, const uint32_t* ibase, Seg& s,
                                         int& kvh, int& row0, int& seq) {
        const uint32_t lead = P.lead[line];
        const int RT = P.row_tile(line);
        base += line * P.batch;
#pragma unroll 1
        while (p < p1) {
            uint32_t b;
            int n, n_eff, id;
            s.step = 0;
            if (h.pl == line && p < h.CP) {
                const uint32_t per = lead + (uint32_t)P.npt;
                id = (int)(p / per);
                b = (uint32_t)id * per;
                n = n_eff = P.npt;
                seq = -1;
                kvh = id / h.nqt;
                row0 = h.r_begin + (id - kvh * h.nqt) * RT;
                s.nrows = min(RT, h.r_end - row0);
                s.keys = s.lim0 = P.prefix_len;
            } else {
                int lo = 0, hi = P.batch;  // the last sequence with base <= p has items here (base rises over it alone)
#pragma unroll 1
                while (hi - lo > 1) {
                    const int mid = (lo + hi) >> 1;
                    if (base[mid] <= p) lo = mid;
                    else hi = mid;
                }
                const int start = P.q_start[lo];
                const Seq q = seq_of(P, start, P.q_start[lo + 1], P.kv_lens[lo]);
                const uint32_t per = lead + (uint32_t)q.tiles;
                const int k = (int)((p - base[lo]) / per);
                b = base[lo] + (uint32_t)k * per;
                n = q.tiles;
                id = (h.pl == line ? h.n_prefix : 0) + (int)ibase[lo] + k;
                seq = lo;
                kvh = k / q.groups;
                const int r = (k - kvh * q.groups) * RT;
                row0 = start + r;
                s.nrows = min(RT, q.m - r);
                s.keys = s.lim0 = q.kv;
                if (P.causal) {
                    s.lim0 = q.kv - q.m + r + 1;
                    s.step = 1;
                }
                n_eff = seen_tiles(P, q, r + s.nrows);
            }
            // tile t is unit b + lead + t
            s.t0 = max((int)(p - b) - (int)lead, 0);
            s.n = min(n_eff, (int)min(p1 - b, lead + (uint32_t)n) - (int)lead) - s.t0;
            s.block = block_of(P, h, line, id, c);
            p = min(p1, b + lead + (uint32_t)n);
            if (s.n > 0) return true;
        }
        return false;
    }
};

// Scan of the batch by every thread of the CTA (NTHR threads, all call it): fills base ([2][batch]:
// per line, the exclusive sums of the own items' lengths, from the prefix items' end), ibase ([batch]: of
// the counts on the sequence's line) and the head.  Ends with a barrier.  (Up to 32 sequences without one in
// between: the plan is 2 us of a small call's chain, most of it code that comes from L2.)
template <int NTHR>
struct PlanMem {
    uint32_t ws[NTHR / 32][4];
    unsigned long long sum[2];  // in 64 bits: a line of 2^31 units or more is refused
    int bad;
};
template <int NTHR>
__device__ __forceinline__ void make_plan(const Shape& P, uint32_t* base, uint32_t* ibase, PlanMem<NTHR>* m, Head& h) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int bad = 0;
    auto rows_ok = [&](int a, int b) { return a >= 0 && b >= a && b <= P.rows; };
    auto prefix = [&]() -> unsigned long long {  // the prefix items, from r_begin and r_end
        if (!rows_ok(h.r_begin, h.r_end)) {
            bad = 1;
            h.r_begin = h.r_end = 0;
        }
        const int live = h.r_end - h.r_begin;
        h.pl = live > P.RH && !P.one_line ? 0 : 1;
        h.nqt = cdiv(live, P.row_tile(h.pl));
        h.n_prefix = P.npt ? h.nqt * P.Hkv : 0;
        const unsigned long long cp = (unsigned long long)h.n_prefix * (unsigned)(P.lead[h.pl] + P.npt);
        h.CP = (uint32_t)cp;
        return cp;
    };
    // a sequence's own items: their line, number and length
    auto own_items = [&](int a, int b, int kv, int& line, uint32_t& items) -> unsigned long long {
        const Seq q = seq_of(P, a, b, kv);
        line = q.line;
        items = (uint32_t)(q.groups * P.Hkv);
        return (unsigned long long)items * (uint32_t)(P.lead[line] + q.tiles);
    };
    uint32_t total[4];  // per line: length, own items
    if (P.batch <= 32) {
        // every warp scans the whole batch, a sequence a lane: one round of loads and one barrier
        const int a = P.q_start[min(lane, P.batch)], b = P.q_start[min(lane + 1, P.batch)];
        const int kv = lane < P.batch ? P.kv_lens[lane] : 0;
        h.r_begin = __shfl_sync(0xffffffffu, a, 0);
        h.r_end = __shfl_sync(0xffffffffu, b, 31);
        const unsigned long long cp = prefix();
        int line = 0, len31 = cp >> 31 != 0;
        uint32_t items = 0, len = 0;
        if (rows_ok(a, b)) {
            const unsigned long long l = own_items(a, b, kv, line, items);
            len31 |= l >> 31 != 0;
            len = (uint32_t)l;
        } else {
            bad = 1;
        }
        // (per line, in units of 256: 2^31 is past what is left of 32 bits)
        const uint32_t sum0 = __reduce_add_sync(0xffffffffu, (line == 0 ? len >> 8 : 0u) + (lane == 0 && h.pl == 0 ? h.CP >> 8 : 0u));
        const uint32_t sum1 = __reduce_add_sync(0xffffffffu, (line == 1 ? len >> 8 : 0u) + (lane == 0 && h.pl == 1 ? h.CP >> 8 : 0u));
        h.bad = __any_sync(0xffffffffu, bad | len31) || sum0 >> 23 || sum1 >> 23;
        uint32_t v[4] = {line ? 0u : len, line ? len : 0u, line ? 0u : items, line ? items : 0u};
        const uint32_t own[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll 1
        for (int o = 1; o < 32; o <<= 1)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t y = __shfl_up_sync(0xffffffffu, v[i], o);
                if (lane >= o) v[i] += y;
            }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t before = i == h.pl ? h.CP : 0u;
            total[i] = __shfl_sync(0xffffffffu, v[i], 31) + before;
            v[i] += before - own[i];
        }
        if (warp == 0 && lane < P.batch) {
            base[lane] = v[0];
            base[P.batch + lane] = v[1];
            ibase[lane] = line ? v[3] : v[2];
        }
    } else {
        if (tid == 0) {
            m->bad = 0;
            m->sum[0] = m->sum[1] = 0;
        }
        h.r_begin = P.q_start[0];
        h.r_end = P.q_start[P.batch];
        const unsigned long long cp = prefix();
        total[0] = h.pl == 0 ? h.CP : 0u;
        total[1] = h.pl == 1 ? h.CP : 0u;
        total[2] = total[3] = 0u;
        __syncthreads();
        if (tid == 0) atomicAdd(&m->sum[h.pl], cp);
#pragma unroll 1
        for (int s0 = 0; s0 < P.batch; s0 += NTHR) {
            const int s = s0 + tid;
            uint32_t v[4] = {0u, 0u, 0u, 0u};
            int line = 0;
            if (s < P.batch) {
                const int a = P.q_start[s], b = P.q_start[s + 1];
                if (!rows_ok(a, b)) {
                    bad = 1;
                } else {
                    uint32_t items;
                    const unsigned long long l = own_items(a, b, P.kv_lens[s], line, items);
                    if (items) atomicAdd(&m->sum[line], l);
                    if (line) {
                        v[1] = (uint32_t)l;
                        v[3] = items;
                    } else {
                        v[0] = (uint32_t)l;
                        v[2] = items;
                    }
                }
            }
            uint32_t own[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll 1
            for (int o = 1; o < 32; o <<= 1)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t y = __shfl_up_sync(0xffffffffu, v[i], o);
                    if (lane >= o) v[i] += y;
                }
            if (lane == 31)
#pragma unroll
                for (int i = 0; i < 4; ++i) m->ws[warp][i] = v[i];
            __syncthreads();
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] -= own[i];
#pragma unroll 1
            for (int w = 0; w < NTHR / 32; ++w)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (w == warp) v[i] += total[i];
                    total[i] += m->ws[w][i];
                }
            if (s < P.batch) {
                base[s] = v[0];
                base[P.batch + s] = v[1];
                ibase[s] = line ? v[3] : v[2];
            }
            __syncthreads();
        }
        if (bad) m->bad = 1;
        __syncthreads();
        h.bad = m->bad || m->sum[0] >> 31 || m->sum[1] >> 31;
    }
    h.W[0] = h.bad ? 0u : total[0];
    h.W[1] = h.bad ? 0u : total[1];
    h.items0 = total[2] + (h.pl == 0 ? (uint32_t)h.n_prefix : 0u);
    // CTAs by the lines' work: a tile of line 1 takes a CTA 0.55 of the time of one of line 0 (at 0.48 / 0.55 / 0.62 the
    // verify blocks of 32 x 16 rows behind 8192 keys take 109 / 101 / 103 us; with every CTA on both lines in turn 116)
    const float c0 = (float)h.W[0], c1 = 0.55f * (float)h.W[1];
    h.n1 = h.W[0] == 0 ? P.n_cta : h.W[1] == 0 ? 0 : min(max(__float2int_rn(P.n_cta * (c1 / (c0 + c1))), 1), P.n_cta - 1);
    const uint32_t w0 = max(P.n_cta - h.n1, 1), w1 = max(2 * h.n1, 1);
    h.part[0] = max(1u, (h.W[0] + w0 - 1) / w0);
    h.part[1] = max(1u, (h.W[1] + w1 - 1) / w1);
    __syncthreads();
}

// The blocks of a row's item on its line: first unit `at`, number `id`, n_eff tiles seen, place rl in it.
__device__ __forceinline__ void dir_item(const Shape& P, const Head& h, int line, uint32_t at, int id, int n_eff, int rl,
                                         int& block, int& count, int& v, int& step) {
    const uint32_t part = h.part[line], t0 = at + (uint32_t)P.lead[line];
    const int c0 = (int)(t0 / part), x = rl >= P.RH ? 1 : 0;
    count = (int)((t0 + (uint32_t)n_eff - 1u) / part) - c0 + 1;
    step = line == 0 ? 2 : 1;
    block = (int)block_of(P, h, line, id, c0) + x;
    v = (rl - x * P.RH) * P.g;
}

// The directory for the merge kernel, by `warps` warps of which this is number `w`: a lane takes a (row, KV head)
// pair at a time.  Pairs are numbered through the rows of q (at most 2^20 of them, times 1024 heads), and the row's
// sequence is searched in the row starts: the work is the rows', whatever the longest sequence is.  (Chunks of 32 pairs of one
// sequence, as many for each as the longest one needs: 1024 sequences, one of 1024 rows and the others of one, 304 us instead
// of 235; fp32 blocks of four 9.7 instead of 8.7.)
__device__ __forceinline__ void write_dir(const Shape& P, const Head& h, const Work& W, const uint32_t* base,
                                          const uint32_t* ibase, int w, int warps, int lane) {
    const int pairs = P.rows * P.Hkv;
#pragma unroll 1
    for (int i = w * 32 + lane; i < pairs; i += warps * 32) {
        const int r = i / P.Hkv, kvh = i - r * P.Hkv;
        if (h.bad || r < h.r_begin || r >= h.r_end) {  // a call that went wrong, or a row of no sequence
            W.dir[i].pre_count = h.bad ? -2 : -1;
            continue;
        }
        int s = 0, hi = P.batch;  // the last sequence that begins at or before r (empty ones share their start with it)
#pragma unroll 1
        while (hi - s > 1) {
            const int mid = (s + hi) >> 1;
            if (P.q_start[mid] <= r) s = mid;
            else hi = mid;
        }
        const int start = P.q_start[s], m = P.q_start[s + 1] - start, j = r - start;
        const Seq q = seq_of(P, start, start + m, P.kv_lens[s]);
        Dir d = {0, 0, 0, 0, 0, 0, 1, 1};
        if (q.kv < 0 || q.kv > (long long)64 * P.width) {
            d.pre_count = -2;
        } else {
            if (P.npt) {
                const int RT = P.row_tile(h.pl), rt = (r - h.r_begin) / RT, id = kvh * h.nqt + rt;
                dir_item(P, h, h.pl, (uint32_t)id * (uint32_t)(P.lead[h.pl] + P.npt), id, P.npt, r - h.r_begin - rt * RT,
                         d.pre_block, d.pre_count, d.pre_v, d.pre_step);
            }
            if (q.tiles) {
                const int RT = P.row_tile(q.line), gi = j / RT, k = kvh * q.groups + gi;
                const int n_eff = seen_tiles(P, q, min(m, (gi + 1) * RT));
                if (n_eff)
                    dir_item(P, h, q.line, base[q.line * P.batch + s] + (uint32_t)k * (uint32_t)(P.lead[q.line] + q.tiles),
                             (h.pl == q.line ? h.n_prefix : 0) + (int)ibase[s] + k, n_eff, j - gi * RT, d.own_block, d.own_count,
                             d.own_v, d.own_step);
            }
        }
        W.dir[i] = d;
    }
}

}  // namespace sp
}  // namespace dfl
