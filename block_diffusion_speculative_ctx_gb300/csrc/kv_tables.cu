// Page tables and slot maps of a batch from its request lengths
// (dflash_kv_tables in include/dflash.h).
//
// Request s takes a_s = ceil((kv + new) / 64) - ceil(kv / 64) pages.  With A and
// Q the exclusive prefix sums of a and of the new lengths, its j-th new page is
// free_pages[used + A_s + j] and its rows start at Q_s.  Bytes: the table read and
// written, 16 B a row; at the largest session (1024 requests) that is 1.6 MB, far
// below a launch's latency, so the kernel is bound by its chain of dependent
// steps: lengths -> scan -> entries.  Hence one launch in which every CTA scans the
// whole batch itself (at most 2048 lengths, from L2) and then writes its share of
// the table (a warp per request) and of the rows: an exchange of the scan between
// CTAs, or a second launch, would cost more than the repeated scan.  In place
// (used_out is used) the count may change only when every CTA has read it: small
// calls run in one CTA, larger ones leave it to a second launch of one CTA.
// Measured (graph replay): 4.1 us for 32 requests of 16 new tokens, 5.0 us for
// 1024 requests of 16 (a launch alone is some 2 us).
#include <algorithm>

#include "ops.h"

namespace dfl {

namespace {

constexpr int NT = 512;
constexpr int PER = DFLASH_OPS_MAX_BATCH / NT;  // requests per thread of the scan
constexpr int CTAS = 152;

enum Part { ALL, ENTRIES, COUNT };  // what a launch writes: everything, all but used_out, used_out alone

__global__ void __launch_bounds__(NT) kv_tables_kernel(dflash_kv_tables_args a, Part what) {
    pdl_wait();
    pdl_trigger();
    __shared__ int qs[DFLASH_OPS_MAX_BATCH + 1];  // first row of each request
    __shared__ int pa[DFLASH_OPS_MAX_BATCH + 1];  // pages taken before each request
    __shared__ int kv_s[DFLASH_OPS_MAX_BATCH];
    __shared__ int2 wsum[NT / 32];
    __shared__ int bad_s;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) bad_s = 0;
    __syncthreads();

    // thread t owns the `per` consecutive requests from per * t (per as small as the batch allows)
    const int per = (a.batch + NT - 1) / NT, s0 = per * tid;
    int bad = 0;
    long long rows = 0, pages = 0;  // sums in 64 bits: lengths are the caller's
    int nw[PER], ad[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        nw[i] = ad[i] = 0;
        if (i < per && s0 + i < a.batch) {
            const int kv = a.kv_lens[s0 + i], n = a.new_lens[s0 + i];
            kv_s[s0 + i] = kv;
            if (kv < 0 || n < 0) {
                bad |= 8;
            } else {
                const long long need = ((long long)kv + n + 63) >> 6;
                nw[i] = n;
                ad[i] = (int)(need - (((long long)kv + 63) >> 6));
                if (need > a.width) bad |= 2;
            }
        }
        rows += nw[i];
        pages += ad[i];
    }
    const int used = a.free_pages ? *a.used : 0;
    if (used < 0) bad |= 8;
    // the sums saturate: past 2^30 the call fails its row or page check anyway
    constexpr long long SAT = 1ll << 30;
    int2 mine = make_int2((int)min(rows, SAT), (int)min(pages, SAT));
    int2 inc = mine;
    auto add = [](int x, int y) { return (int)min((long long)x + y, 1ll << 30); };
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, inc.x, o), y = __shfl_up_sync(0xffffffffu, inc.y, o);
        if (lane >= o) inc = make_int2(add(inc.x, x), add(inc.y, y));
    }
    if (lane == 31) wsum[warp] = inc;
    if (bad) atomicOr(&bad_s, bad);
    __syncthreads();
    int2 before = make_int2(0, 0), total = make_int2(0, 0);
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) {
        if (w == warp) before = total;
        total = make_int2(add(total.x, wsum[w].x), add(total.y, wsum[w].y));
    }
    // exclusive: the inclusive warp scan of the lane before, plus the warps before
    int2 ex = make_int2(__shfl_up_sync(0xffffffffu, inc.x, 1), __shfl_up_sync(0xffffffffu, inc.y, 1));
    if (lane == 0) ex = make_int2(0, 0);
    ex = make_int2(add(ex.x, before.x), add(ex.y, before.y));
#pragma unroll
    for (int i = 0; i < PER; ++i)
        if (i < per && s0 + i < a.batch) {
            qs[s0 + i] = ex.x;
            pa[s0 + i] = ex.y;
            ex = make_int2(add(ex.x, nw[i]), add(ex.y, ad[i]));
        }
    if (tid == 0) {
        qs[a.batch] = total.x;
        pa[a.batch] = total.y;
    }
    int status = bad_s;
    if (a.free_pages && (long long)max(used, 0) + total.y > a.n_free) status |= 1;
    if (total.x > a.rows) status |= 4;
    __syncthreads();
    const bool ok = status == 0;

    if (blockIdx.x == 0 && tid == 0 && what != ENTRIES && a.used_out)
        *a.used_out = ok ? used + (a.free_pages ? total.y : 0) : used;
    if (what == COUNT) return;
    if (blockIdx.x == 0 && tid == 0) *a.status = status;

    const int gt = blockIdx.x * NT + tid, gn = gridDim.x * NT;
    // table: the old entries copied (unless in place), the request's new pages, then scratch
    if (ok && a.table_out) {
        const bool copy = a.table_out != a.table;
        for (int s = gt >> 5; s < a.batch; s += gn >> 5) {
            const int old = (kv_s[s] + 63) >> 6, taken = pa[s + 1] - pa[s];
            const int* src = a.table + (long long)s * a.ld_table;
            const int* fresh = a.free_pages ? a.free_pages + used + pa[s] - old : src;
            int* dst = a.table_out + (long long)s * a.ld_out;
            for (int j = (copy ? 0 : old & ~31) + lane; j < a.width; j += 32)
                if (copy || j >= old) dst[j] = j < old ? src[j] : j < old + taken ? fresh[j] : a.scratch_page;
        }
    }
    // rows: the request of row r is the last s with qs[s] <= r (requests without rows share
    // their start with the next one)
    for (int r = gt; r < a.rows; r += gn) {
        int seq = -1, pos = -1;
        long long slot = -1;
        if (ok && r < total.x) {
            int lo = 0, hi = a.batch;  // qs[lo] <= r < qs[hi]
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (qs[mid] <= r) lo = mid;
                else hi = mid;
            }
            seq = lo;
            const int kv = kv_s[seq], i = kv + r - qs[seq];
            pos = a.base_pos + i;
            const int j = i >> 6, old = (kv + 63) >> 6;
            const int page = (j < old || !a.free_pages) ? a.table[(long long)seq * a.ld_table + j]
                                                        : a.free_pages[used + pa[seq] + j - old];
            slot = (long long)page * 64 + (i & 63);
        }
        if (a.row_seq) a.row_seq[r] = seq;
        if (a.row_pos) a.row_pos[r] = pos;
        if (a.slots) a.slots[r] = slot;
    }
    for (int s = gt; s <= a.batch; s += gn) a.q_start[s] = ok ? qs[s] : 0;
}

dflash_status fail(const char* msg) {
    set_global_error(msg);
    return DFLASH_E_INVAL;
}

}  // namespace

void kv_tables(const Launch& L, const dflash_kv_tables_args& a) {
    // A warp per request, a thread per row (1024 requests in one CTA: 71 us instead of 5.0).  In place up to 2048
    // entries and rows take one CTA: 32 requests whose pool is used up take 3.3 us, with the second launch 5.7.  What is
    // not in place is spread out whatever its size (32 requests of 16 tokens: 4.1 us, in one CTA 4.4).
    const long long rows = (a.rows + NT - 1) / NT, reqs = (a.batch + NT / 32 - 1) / (NT / 32);
    int c = (int)std::min<long long>(CTAS, std::max(rows, reqs));
    const bool inplace = a.used_out && a.used_out == a.used;
    if (inplace && (long long)a.batch * a.width + a.rows <= 2048) c = 1;
    const bool split = c > 1 && inplace;
    launch_k(L, kv_tables_kernel, dim3(c), dim3(NT), 0, 1, a, split ? ENTRIES : ALL);
    if (split) {
        Launch after = L;
        after.pdl = true;
        launch_k(after, kv_tables_kernel, dim3(1), dim3(NT), 0, 1, a, COUNT);
    }
}

}  // namespace dfl

using namespace dfl;

extern "C" dflash_status dflash_kv_tables(const dflash_kv_tables_args* p, void* cuda_stream) {
    if (!p) return fail("kv_tables: args is NULL");
    const dflash_kv_tables_args& a = *p;
    if (a.batch < 1 || a.batch > DFLASH_OPS_MAX_BATCH) return fail("kv_tables: batch outside [1, 2048]");
    if (a.width < 0 || a.rows < 0 || a.rows >= (1 << 30) || a.n_free < 0)
        return fail("kv_tables: width, rows and n_free must not be negative (rows below 2^30)");
    if (a.width > (1 << 24) || a.base_pos < 0 || a.base_pos > (1 << 30))
        return fail("kv_tables: width above 2^24 or base_pos outside [0, 2^30]");
    if (!a.kv_lens || !a.new_lens || !a.q_start || !a.status) return fail("kv_tables: NULL argument");
    if (a.width > 0 && !a.table) return fail("kv_tables: table is NULL");
    if (a.ld_table < a.width || (a.table_out && a.ld_out < a.width))
        return fail("kv_tables: a table row stride is smaller than width");
    if (a.free_pages && (!a.used || !a.used_out || (a.width > 0 && !a.table_out)))
        return fail("kv_tables: taking pages needs used, used_out and table_out");
    if (a.table_out == a.table && a.table && a.ld_out != a.ld_table)
        return fail("kv_tables: in place needs one row stride");
    bool failed = false;
    Launch L{(cudaStream_t)cuda_stream, nullptr};
    L.pdl = true;  // (each kernel waits for what runs before it ahead of its first read)
    L.failed = &failed;
    kv_tables(L, a);
    const cudaError_t e = cudaGetLastError();
    if (failed || e != cudaSuccess) {
        set_global_error(e != cudaSuccess ? cudaGetErrorString(e) : "kv_tables: launch failed");
        return DFLASH_E_CUDA;
    }
    return DFLASH_OK;
}
