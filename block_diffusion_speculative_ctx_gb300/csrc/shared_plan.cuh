// How the shared-prefix attention divides its work: the arithmetic that the
// attention kernels and the merge kernel have in common.
//
// Work is a line of tiles.  An item is one KV head's query vectors of up to RT
// rows (g heads each) against one key list: first the prefix items (every row
// tile of the batch x KV head, against the prefix), then per sequence its own
// items (KV head x row tile of the sequence, against its own keys).  An item
// has one tile per KT keys, each of a weight (its cost relative to the others).
// The line of weights [0, W) is cut into N equal parts, one per CTA: a tile
// belongs to the CTA whose part its first unit lies in.  So every CTA gets the
// same work whatever the lengths are, and an item is split over as few CTAs as
// its weight takes.  A CTA's run of tiles inside one item is a segment; its
// partial result (per vector: maximum, sum, unnormalised output) goes to slot
// item + cta of the workspace: along the line neither index ever falls and one
// of them rises at each segment, so slots are unique.
#pragma once

#include "ops.h"

namespace dfl {
namespace sp {

struct Shape {
    int H, Hkv, g, hd;
    int VT;        // query vectors per stream
    int RH;        // rows per stream: VT / g
    int RT;        // rows per item: two streams
    int KT;        // keys per tile
    int batch, rows, width, prefix_len, causal, n_pages;
    int npt;       // prefix tiles
    int n_cta;
    long long ld_table;
    const int *prefix_pages, *table, *kv_lens, *q_start;
};

// Cut of the line, written by CTA 0 for the merge kernel.
struct Head {
    uint32_t W;        // total weight
    uint32_t CP;       // weight of the prefix items
    uint32_t n_prefix; // prefix items
    uint32_t wp;       // weight of a prefix tile
    int r_begin, r_end;
    int bad;           // q_start is not a list of rows, or the line is too long
    int nqt;           // row tiles of the batch
};

// Workspace: Head, per-CTA error words, per-sequence first weight and first item,
// per-slot error words, per-slot (max, sum), per-slot outputs.
struct Work {
    Head* head;
    uint32_t* err;      // [n_cta]
    uint32_t* base;     // [batch]
    uint32_t* ibase;    // [batch]
    uint32_t* slot_bad; // [slots]
    float2* ml;         // [slots][2][VT]
    float* o;           // [slots][2][hd / 8][VT][8]
};

inline long long max_slots(int Hkv, int RT, int batch, int rows, int n_cta) {
    const long long tiles = (rows + RT - 1) / RT;
    // own items: every sequence adds at most one partial row tile to the full ones
    return Hkv * (tiles + rows / RT + (batch < rows ? batch : rows)) + n_cta;
}

inline size_t layout(char* p, int hd, int VT, int batch, int n_cta, long long slots, Work* w) {
    size_t at = 0;
    auto take = [&](size_t bytes) {
        char* q = p + at;
        at += (bytes + 255) / 256 * 256;
        return q;
    };
    Work x;
    x.head = (Head*)take(sizeof(Head));
    x.err = (uint32_t*)take((size_t)n_cta * 4);
    x.base = (uint32_t*)take((size_t)batch * 4);
    x.ibase = (uint32_t*)take((size_t)batch * 4);
    x.slot_bad = (uint32_t*)take((size_t)slots * 4);
    x.ml = (float2*)take((size_t)slots * 2 * VT * 8);
    x.o = (float*)take((size_t)slots * 2 * VT * hd * 4);
    if (w) *w = x;
    return at;
}

// Weight of a tile whose rows fill both streams / one stream (the keys are read and the
// scores computed once either way, the second stream's products come on top).
constexpr uint32_t W_PAIR = 3, W_ONE = 2;

__host__ __device__ __forceinline__ uint32_t part_begin(uint32_t W, int c, int n) {
    return (uint32_t)((unsigned long long)W * (unsigned)c / (unsigned)n);
}
// The CTA whose part holds unit x < W: the last c with floor(c W / n) <= x.
__device__ __forceinline__ int owner(uint32_t W, uint32_t x, int n) {
    return (int)((((unsigned long long)x + 1) * (unsigned)n + W - 1) / W) - 1;
}

__device__ __forceinline__ int cdiv(int a, int b) { return (a + b - 1) / b; }

// A sequence's own items: m rows, kv keys (0 tiles for lengths out of range).
struct Seq {
    int m, kv, tiles, groups;
    uint32_t w;
};
__device__ __forceinline__ Seq seq_of(const Shape& P, int start, int end, int kv) {
    Seq q;
    q.m = end - start;
    q.kv = kv;
    const bool ok = q.m > 0 && kv > 0 && kv <= (long long)64 * P.width;
    q.tiles = ok ? cdiv(kv, P.KT) : 0;
    q.groups = q.m > 0 ? cdiv(q.m, P.RT) : 0;
    q.w = q.m > P.RH ? W_PAIR : W_ONE;
    return q;
}

struct Seg {
    int seq;          // -1: prefix
    int kvh;
    int row0, nrows;  // rows of q
    int t0, t1;       // tiles
    int keys;         // keys of the list (prefix_len or kv)
    int lim0;         // own keys seen by row row0 (causal: one more per row); non-causal and prefix: keys
    int slot;
    bool pair;        // both streams hold rows (else both hold the same rows and share the tiles)
};

// Walks the segments of CTA `cta`.  base / ibase: exclusive prefix sums over the sequences of the
// own items' weights (from CP) and counts, in shared memory.
struct Walk {
    uint32_t p, p1;
    int cta;
    __device__ __forceinline__ Walk(const Head& h, int c, int n) : p(part_begin(h.W, c, n)), p1(part_begin(h.W, c + 1, n)), cta(c) {}

    __device__ __forceinline__ bool next(const Shape& P, const Head& h, const uint32_t* base, const uint32_t* ibase, Seg& s) {
        while (p < p1) {
            uint32_t b, w;
            int n, n_eff;
            if (p < h.CP) {
                const uint32_t per = (uint32_t)P.npt * h.wp, item = p / per;
                b = item * per;
                w = h.wp;
                n = n_eff = P.npt;
                s.seq = -1;
                s.kvh = (int)(item / h.nqt);
                s.row0 = h.r_begin + (int)(item % h.nqt) * P.RT;
                s.nrows = min(P.RT, h.r_end - s.row0);
                s.keys = s.lim0 = P.prefix_len;
                s.slot = (int)item + cta;
            } else {
                int lo = 0, hi = P.batch;  // the last sequence with base <= p has tiles (base strictly rises over it)
                while (hi - lo > 1) {
                    const int mid = (lo + hi) >> 1;
                    if (base[mid] <= p) lo = mid;
                    else hi = mid;
                }
                const int start = P.q_start[lo];
                const Seq q = seq_of(P, start, P.q_start[lo + 1], P.kv_lens[lo]);
                const uint32_t per = (uint32_t)q.tiles * q.w, k = (p - base[lo]) / per;
                b = base[lo] + k * per;
                w = q.w;
                n = q.tiles;
                const int gi = (int)(k % q.groups);
                s.seq = lo;
                s.kvh = (int)(k / q.groups);
                s.row0 = start + gi * P.RT;
                s.nrows = min(P.RT, q.m - gi * P.RT);
                s.keys = q.kv;
                s.lim0 = P.causal ? q.kv - q.m + gi * P.RT + 1 : q.kv;
                // causal: the tile's last row sees the most keys
                n_eff = P.causal ? min(n, cdiv(max(s.lim0 + s.nrows - 1, 0), P.KT)) : n;
                s.slot = (int)(h.n_prefix + ibase[lo] + k) + cta;
            }
            s.pair = s.nrows > P.RH;
            s.t0 = (int)((p - b + w - 1) / w);
            const int t1 = (int)min((uint32_t)n, (p1 - b + w - 1) / w);
            p = t1 == n ? b + (uint32_t)n * w : p1;
            s.t1 = min(t1, n_eff);
            if (s.t0 < s.t1) return true;
        }
        return false;
    }
};

// Scan of the batch by every thread of the CTA (NTHR threads, all call it): fills base / ibase and the
// head.  ws: 2 * NTHR / 32 words, flag: one word (shared memory).  Ends with a barrier.
template <int NTHR>
__device__ void make_plan(const Shape& P, uint32_t* base, uint32_t* ibase, uint32_t* ws, int* flag, Head& h) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
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
    h.nqt = cdiv(live, P.RT);
    h.wp = live > P.RH ? W_PAIR : W_ONE;
    h.n_prefix = P.npt ? (uint32_t)(h.nqt * P.Hkv) : 0u;
    unsigned long long cp = (unsigned long long)h.n_prefix * P.npt * h.wp;
    constexpr unsigned long long MOST = 1ull << 31;
    if (cp >= MOST) {
        bad = 1;
        cp = 0;
    }
    h.CP = (uint32_t)cp;
    unsigned long long carry = cp;
    uint32_t icarry = 0;
    for (int s0 = 0; s0 < P.batch; s0 += NTHR) {
        const int s = s0 + tid;
        unsigned long long c = 0;
        uint32_t it = 0;
        if (s < P.batch) {
            const int a = P.q_start[s], b = P.q_start[s + 1];
            if (a < 0 || b < a || b > P.rows) {
                bad = 1;
            } else {
                const Seq q = seq_of(P, a, b, P.kv_lens[s]);
                it = (uint32_t)(q.groups * P.Hkv);
                c = (unsigned long long)it * (uint32_t)q.tiles * q.w;
                if (c >= MOST) {
                    bad = 1;
                    c = 0;
                }
            }
        }
        // inclusive warp scans (32-bit sums saturate at MOST: the call is bad then)
        unsigned long long ci = c;
        uint32_t ii = it;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned long long x = __shfl_up_sync(0xffffffffu, ci, o);
            const uint32_t y = __shfl_up_sync(0xffffffffu, ii, o);
            if (lane >= o) {
                ci = min(ci + x, MOST);
                ii += y;
            }
        }
        if (lane == 31) {
            ws[2 * warp] = (uint32_t)ci;
            ws[2 * warp + 1] = ii;
        }
        __syncthreads();
        unsigned long long before = carry;
        uint32_t ibefore = icarry;
        for (int w = 0; w < NTHR / 32; ++w) {
            if (w == warp) {
                before = carry;
                ibefore = icarry;
            }
            carry = min(carry + ws[2 * w], MOST);
            icarry += ws[2 * w + 1];
        }
        if (s < P.batch) {
            base[s] = (uint32_t)min(before + ci - c, MOST);
            ibase[s] = ibefore + ii - it;
        }
        __syncthreads();
    }
    if (carry >= MOST) bad = 1;
    if (bad) *flag = 1;
    __syncthreads();
    h.bad = *flag;
    h.W = h.bad ? 0u : (uint32_t)carry;
}

}  // namespace sp
}  // namespace dfl
