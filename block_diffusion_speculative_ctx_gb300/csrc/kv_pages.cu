// Pages that several sequences hold (dflash_kv_fork and dflash_kv_release in
// include/dflash.h).
//
// Fork: two launches.  The first reads the children's lengths in every CTA (at
// most 2048 from L2, as the page tables do) and shares the work on the tables and
// the counts, a warp per child; the second copies the pages that end inside, a CTA
// per child, layer and cache, each head's tokens being one run of the page, of which a
// warp takes 4 KB at a time (by vectors of the whole page in turn: 64 children over
// 36 layers, with their release, 80 us instead of 69).  Bytes: the parents' last tokens once (their other
// children find them in L2) and each child's copy; nothing for the shared pages.
// Measured (graph replay): 4.9 us for four children over 5 layers; with the release
// 71 us for 64 children of 8 parents over 36 layers (340 MB: 50 us at a measured copy's rate).
//
// Release: one launch of one cluster, whose barriers separate the steps.
//   1  every page named is looked at (range, count);
//   2  its count falls by one for each mention: a page without a holder ends at -1
//      (below: it was returned too often, and the counts go back); with cuts, the counts
//      left on the pages that they end in tell whether another holder stays;
//   3  of a page's mentions the first takes it: an atomic minimum over the
//      mentions' numbers, kept in the count itself as INT_MIN + number (left out
//      where no page named had a second holder);
//   4  each warp counts the pages that its mentions took; with the counts of the
//      warps before it, it knows their places in the free list.
// Mentions are numbered (place in seqs, table entry) and a warp owns consecutive
// ones, so the list's order does not depend on the order of the atomics.  Bound by
// latency: seven to nine dependent trips to L2 and as many barriers; 6.1 us for four
// sequences of nine pages (with cuts a barrier and a trip more).
#include <algorithm>

#include "ops.h"
#include "tcgen05.cuh"

namespace dfl {

namespace {

constexpr int MAXB = DFLASH_OPS_MAX_BATCH;
enum : int { SHORT_POOL = 1, BAD_WIDTH = 2, BAD_LENGTH = 8, BAD_PAGE = 16, BAD_COUNT = 32, SHARED_CUT = 64 };

// ------------------------------------------------------------------------------ fork
constexpr int NT = 512, PER = MAXB / NT;

__global__ void __launch_bounds__(NT) fork_tables_kernel(dflash_kv_fork_args a) {
    pdl_wait();
    pdl_trigger();
    __shared__ int len_s[MAXB], taken_s[MAXB];
    __shared__ int wsum[NT / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // thread t owns the `per` consecutive children from per * t
    const int per = (a.children + NT - 1) / NT, c0 = per * tid;
    int bad = 0, mine = 0, takes[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        takes[i] = 0;
        if (i < per && c0 + i < a.children) {
            const int parent = a.parents[c0 + i];
            int n = 0;
            if (parent < 0 || parent >= a.batch) bad |= BAD_LENGTH;
            else {
                n = a.kv_lens[parent];
                if (n < 0) bad |= BAD_LENGTH;
                else if (n > (long long)64 * a.width) bad |= BAD_WIDTH;
                else takes[i] = (n & 63) != 0;
            }
            len_s[c0 + i] = n;
        }
        mine += takes[i];
    }
    const int used = *a.used;
    if (used < 0) bad |= BAD_LENGTH;
    int inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += x;
    }
    if (lane == 31) wsum[warp] = inc;
    int status = __syncthreads_or(bad & BAD_LENGTH) ? BAD_LENGTH : 0;
    status |= __syncthreads_or(bad & BAD_WIDTH) ? BAD_WIDTH : 0;
    int before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) {
        if (w == warp) before = total;
        total += wsum[w];
    }
    int at = before + inc - mine;
#pragma unroll
    for (int i = 0; i < PER; ++i)
        if (i < per && c0 + i < a.children) {
            taken_s[c0 + i] = at;
            at += takes[i];
        }
    if ((long long)max(used, 0) + total > a.n_free) status |= SHORT_POOL;
    __syncthreads();
    if (blockIdx.x == 0 && tid == 0) *a.status = status;
    const int gt = blockIdx.x * NT + tid, gn = gridDim.x * NT;
    for (int c = gt; c < a.children; c += gn) a.lens_out[c] = status ? 0 : len_s[c];
    if (status) return;
    for (int c = gt >> 5; c < a.children; c += gn >> 5) {
        const int n = len_s[c], full = n >> 6, fresh = n & 63 ? full : -1;
        const int* src = a.table + (long long)a.parents[c] * a.ld_table;
        int* dst = a.table_out + (long long)c * a.ld_out;
        for (int j = lane; j < a.width; j += 32) {
            int page = a.scratch_page;
            if (j < full) {
                page = src[j];
                if (page >= 0 && page < a.n_pages) atomicAdd(&a.refs[page], 1);
            } else if (j == fresh) {
                page = a.free_pages[used + taken_s[c]];
            }
            dst[j] = page;
        }
    }
}

constexpr int NT_COPY = 256, DEEP = 8;

// CTA (c, l): child c, layer l / 2, keys or values.
__global__ void __launch_bounds__(NT_COPY) fork_copy_kernel(dflash_kv_fork_args a, int vecs) {
    pdl_wait();
    pdl_trigger();
    const int c = blockIdx.x, tid = threadIdx.x;
    const bool ok = (*a.status & ~BAD_PAGE) == 0;
    if (c == 0 && blockIdx.y == 0) {  // the taken pages' number (no other CTA reads used any more)
        __shared__ int total;
        if (tid == 0) total = 0;
        __syncthreads();
        int mine = 0;
        if (ok)
            for (int i = tid; i < a.children; i += NT_COPY) mine += (a.lens_out[i] & 63) != 0;
        if (mine) atomicAdd(&total, mine);
        __syncthreads();
        if (tid == 0) *a.used_out = *a.used + total;
    }
    if (!ok) return;
    const int n = a.lens_out[c], full = n >> 6, tail = n & 63;
    const int* src_row = a.table + (long long)a.parents[c] * a.ld_table;
    const int* dst_row = a.table_out + (long long)c * a.ld_out;
    auto in = [&](int page) { return page >= 0 && page < a.n_pages; };
    if (blockIdx.y == 0) {
        bool bad = false;
        for (int j = tid; j < full + (tail != 0); j += NT_COPY) bad |= !in(src_row[j]) || !in(dst_row[j]);
        if (bad) atomicOr(a.status, BAD_PAGE);
    }
    if (tail == 0) return;
    const int from = src_row[full], to = dst_row[full];
    if (!in(from) || !in(to)) return;
    uint4* cache = reinterpret_cast<uint4*>((char*)(blockIdx.y & 1 ? a.v_cache : a.k_cache) +
                                            (long long)(blockIdx.y >> 1) * a.ld_layer * (a.dtype == DFLASH_DTYPE_BF16 ? 2 : 4));
    const int run = tail * vecs, page = 64 * vecs;  // vectors of a head that are copied, and that it has in a page
    const uint4* src = cache + (long long)from * a.n_kv_heads * page;
    uint4* dst = cache + (long long)to * a.n_kv_heads * page;
    // a warp takes DEEP vectors a lane of one head's run at a time
    constexpr int PIECE = 32 * DEEP;
    const int lane = tid & 31, pieces = (run + PIECE - 1) / PIECE;
    for (int u = tid >> 5; u < pieces * a.n_kv_heads; u += NT_COPY / 32) {
        const int h = u / pieces, i0 = (u - h * pieces) * PIECE + lane, at = h * page + i0, left = run - i0;
        uint4 x[DEEP];
#pragma unroll
        for (int i = 0; i < DEEP; ++i)
            if (32 * i < left) x[i] = src[at + 32 * i];
#pragma unroll
        for (int i = 0; i < DEEP; ++i)
            if (32 * i < left) dst[at + 32 * i] = x[i];
    }
}

// --------------------------------------------------------------------------- release
constexpr int NR = 1024, WARPS = NR / 32, MAXC = 8;
constexpr int UNIT = 256;        // table entries of one sequence that a warp takes at a time
constexpr int MAX_WIDTH = 1 << 18;  // a mention's number is its place in seqs times this, plus its table entry

__device__ __forceinline__ int ld_count(const int* p) {  // (past the SM's own cache: other SMs change the counts)
    int v;
    asm volatile("ld.relaxed.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ int ld_peer_int(const int* local, uint32_t rank) {
    uint32_t remote;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(tc::smem_u32(local)), "r"(rank));
    int v;
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(remote) : "memory");
    return v;
}

__global__ void __launch_bounds__(NR) kv_release_kernel(dflash_kv_release_args a, int n_cta) {
    __shared__ int units_s[MAXB + 1];  // units of the sequences before
    __shared__ int seq_s[MAXB], first_s[MAXB], pages_s[MAXB];  // its table entries first_s .. pages_s - 1 are named
    __shared__ uint32_t named[MAXB / 32];
    __shared__ int wsum[WARPS], counts[WARPS];
    __shared__ int flag_s[2];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = n_cta > 1 ? (int)tc::cluster_rank() : 0;
    pdl_wait();
    pdl_trigger();
    if (tid < MAXB / 32) named[tid] = 0;
    if (tid < 2) flag_s[tid] = 0;
    __syncthreads();

    // ---- the sequences, by every CTA: thread t owns 2 t and 2 t + 1
    int bad = 0, mine[2], cut[2];  // (cut: the page that a cut ends inside)
    bool out = false;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int k = 2 * tid + i;
        mine[i] = 0;
        cut[i] = -1;
        if (k < a.n) {
            const int s = a.seqs[k];
            int pages = 0, first = 0;
            if (s < 0 || s >= a.batch || atomicOr(&named[s >> 5], 1u << (s & 31)) >> (s & 31) & 1u) {
                bad |= BAD_LENGTH;
            } else {
                const int kv = a.kv_lens[s], keep = a.keep_lens ? a.keep_lens[s] : 0;
                if (kv < 0 || keep < 0 || keep > kv) bad |= BAD_LENGTH;
                else if (kv > (long long)64 * a.width) bad |= BAD_WIDTH;
                else {
                    pages = (kv + 63) >> 6, first = (keep + 63) >> 6;
                    if (rank == 0 && keep < kv && keep & 63) {
                        cut[i] = a.table[(long long)s * a.ld_table + (keep >> 6)];
                        out |= cut[i] < 0 || cut[i] >= a.n_pages || ld_count(&a.refs[cut[i]]) < 0;
                    }
                }
            }
            seq_s[k] = s;
            first_s[k] = first;
            pages_s[k] = pages;
            mine[i] = (pages - first + UNIT - 1) / UNIT;
        }
    }
    const int used = *a.used;
    if (used < 0 || used > a.n_free) bad |= BAD_LENGTH;
    int inc = mine[0] + mine[1];
    const int both = inc;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += x;
    }
    if (lane == 31) wsum[warp] = inc;
    int status = __syncthreads_or(bad & BAD_LENGTH) ? BAD_LENGTH : 0;
    status |= __syncthreads_or(bad & BAD_WIDTH) ? BAD_WIDTH : 0;
    const int sums = wsum[lane];  // (a lane a warp)
    const int total = __reduce_add_sync(0xffffffffu, sums);
    int before = __reduce_add_sync(0xffffffffu, lane < warp ? sums : 0);
    before += inc - both;
    if (2 * tid < a.n) units_s[2 * tid] = before;
    if (2 * tid + 1 < a.n) units_s[2 * tid + 1] = before + mine[0];
    if (tid == 0) units_s[a.n] = total;
    __syncthreads();

    // a warp's mentions: f(page, number, live) for its consecutive units, 32 at a time, in order; lanes behind the
    // sequence's last page are not live
    const int warps = n_cta * WARPS, share = (total + warps - 1) / warps;
    const int u0 = min(total, (rank * WARPS + warp) * share), u1 = min(total, u0 + share);
    int k0 = 0;  // the first unit's sequence: units_s[k0] <= u0 < units_s[k0 + 1]
    if (u0 < u1) {
        int hi = a.n;
        while (hi - k0 > 1) {
            const int mid = (k0 + hi) >> 1;
            if (units_s[mid] <= u0) k0 = mid;
            else hi = mid;
        }
    }
    auto mentions = [&](auto&& f) {
        int k = k0;
        for (int u = u0; u < u1; ++u) {
            while (units_s[k + 1] <= u) ++k;
            const int* row = a.table + (long long)seq_s[k] * a.ld_table;
            const int j0 = first_s[k] + (u - units_s[k]) * UNIT;
            int page[UNIT / 32];
#pragma unroll
            for (int i = 0; i < UNIT / 32; ++i) {
                const int j = j0 + 32 * i + lane;
                page[i] = j < pages_s[k] ? row[j] : -1;
            }
#pragma unroll
            for (int i = 0; i < UNIT / 32; ++i)
                if (j0 + 32 * i < pages_s[k]) f(page[i], k * MAX_WIDTH + j0 + 32 * i + lane, j0 + 32 * i + lane < pages_s[k]);
        }
    };
    auto meet = [&] {
        __syncwarp();
        if (n_cta > 1) tc::cluster_sync();
        else __syncthreads();
    };
    // the cluster's barrier, and the flags that some thread called it with
    int round = 0;
    auto any = [&](int x) {
        x = __reduce_or_sync(0xffffffffu, x);
        if (lane == 0 && x) atomicOr(&flag_s[round & 1], x);
        meet();
        int on = 0;
        for (int r = 0; r < n_cta; ++r) on |= n_cta > 1 ? ld_peer_int(&flag_s[round & 1], r) : flag_s[round & 1];
        ++round;
        return on;
    };

    int freed = 0;
    if (status == 0) {  // (every CTA found the same)
        mentions([&](int page, int, bool live) { out |= live && (page < 0 || page >= a.n_pages || ld_count(&a.refs[page]) < 0); });
        if (any(out)) status = BAD_PAGE;
    }
    if (status == 0) {
        enum { OVER = 1, SHARED = 2, CUT = 4 };  // a count below what its page had; a page that several mentions free; a cut's with others
        int seen = 0;
        mentions([&](int page, int, bool live) {
            if (!live) return;
            const int before = atomicSub(&a.refs[page], 1);
            if (before < 0) seen |= OVER;
            if (before > 0) seen |= SHARED;  // (it may yet be freed by others)
        });
        seen = any(seen);
        if (a.keep_lens && !(seen & OVER)) {  // (a cut's own sequence stays, so its page's count may not fall below 0 either)
            int left = 0;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int c = cut[i] < 0 ? 0 : ld_count(&a.refs[cut[i]]);
                left |= c < 0 ? OVER : c > 0 ? CUT : 0;
            }
            seen |= any(left);
        }
        if (seen & (OVER | CUT)) {
            status = seen & OVER ? BAD_COUNT : SHARED_CUT;
        } else {
            // which of a page's mentions takes it (a page that had no other holder has one)
            if (seen & SHARED) {
                mentions([&](int page, int number, bool live) {
                    if (live && ld_count(&a.refs[page]) < 0) atomicMin(&a.refs[page], INT32_MIN + number);
                });
                meet();
            }
            auto takes = [&](int page, int number, bool live) {
                if (!live) return false;
                const int c = ld_count(&a.refs[page]);
                return seen & SHARED ? c == INT32_MIN + number : c < 0;
            };
            int mine_taken = 0;
            mentions([&](int page, int number, bool live) {
                mine_taken += __popc(__ballot_sync(0xffffffffu, takes(page, number, live)));
            });
            if (lane == 0) counts[warp] = mine_taken;
            meet();
            int ahead = 0;
            for (int w = lane; w < warps; w += 32) {
                const int x = n_cta > 1 ? ld_peer_int(&counts[w % WARPS], w / WARPS) : counts[w];
                freed += x;
                if (w < rank * WARPS + warp) ahead += x;
            }
            freed = __reduce_add_sync(0xffffffffu, freed);
            ahead = __reduce_add_sync(0xffffffffu, ahead);
            if (freed > used) status = SHORT_POOL;
            int at = used - freed + ahead;
            mentions([&](int page, int number, bool live) {
                const bool mine = takes(page, number, live);
                const uint32_t took = __ballot_sync(0xffffffffu, mine);
                if (mine) {
                    if (status == 0) a.free_pages[at + __popc(took & ((1u << lane) - 1u))] = page;
                    atomicExch(&a.refs[page], status == 0 ? 0 : -1);
                }
                at += __popc(took);
            });
        }
        meet();
        if (status != 0)  // as it was
            mentions([&](int page, int, bool live) {
                if (live) atomicAdd(&a.refs[page], 1);
            });
    }
    if (rank == 0 && tid == 0) {
        *a.status = status;
        *a.used_out = status == 0 ? used - freed : used;
    }
    meet();  // (no CTA leaves while another may read its flags; every CTA has read *used)
}

}  // namespace

}  // namespace dfl

using namespace dfl;

extern "C" dflash_status dflash_kv_fork(const dflash_kv_fork_args* p, void* cuda_stream) {
    if (!p) return refuse("kv_fork: args is NULL");
    const dflash_kv_fork_args& a = *p;
    if (const char* why = bad_caches(a, "kv_fork: dtype must be F32 or BF16", "kv_fork: layers outside [1, 1024]",
                                     "kv_fork: n_pages, n_kv_heads or head_dim out of range (a head's row is a multiple of 16 bytes)",
                                     "kv_fork: the caches must be 16-byte aligned, ld_layer a multiple of 16 bytes and no smaller than a layer"))
        return refuse(why);
    // (one cache for both is copied twice alike)
    if (a.k_cache != a.v_cache && caches_overlap(a)) return refuse("kv_fork: k_cache and v_cache overlap");
    if (a.batch < 1 || a.batch > MAXB) return refuse("kv_fork: batch outside [1, 2048]");
    if (a.children < 1 || a.children > MAXB) return refuse("kv_fork: children outside [1, 2048]");
    if (a.width < 1 || a.width > (1 << 22) || a.ld_table < a.width || a.ld_out < a.width)
        return refuse("kv_fork: width outside [1, 2^22], or a table row stride is smaller");
    if (a.n_free < 0) return refuse("kv_fork: n_free must not be negative");
    if (!a.parents || !a.kv_lens || !a.table || !a.free_pages || !a.used || !a.refs || !a.table_out || !a.lens_out ||
        !a.used_out || !a.status)
        return refuse("kv_fork: NULL argument");
    if (a.table_out == a.table || a.lens_out == a.kv_lens)
        return refuse("kv_fork: the children's tables and lengths may not be the parents'");
    const int ctas = std::min(152, (a.children + NT / 32 - 1) / (NT / 32));
    const int vecs = a.head_dim * (a.dtype == DFLASH_DTYPE_BF16 ? 2 : 4) / 16;
    return queue(cuda_stream, "kv_fork: launch failed", [&](const Launch& L) {
        launch_k(L, fork_tables_kernel, dim3(ctas), dim3(NT), 0, 1, a);
        launch_k(L, fork_copy_kernel, dim3(a.children, 2 * a.layers), dim3(NT_COPY), 0, 1, a, vecs);
    });
}

extern "C" dflash_status dflash_kv_release(const dflash_kv_release_args* p, void* cuda_stream) {
    if (!p) return refuse("kv_release: args is NULL");
    const dflash_kv_release_args& a = *p;
    if (a.batch < 1 || a.batch > MAXB) return refuse("kv_release: batch outside [1, 2048]");
    if (a.n < 1 || a.n > MAXB) return refuse("kv_release: n outside [1, 2048]");
    if (a.width < 1 || a.width > MAX_WIDTH || a.ld_table < a.width)
        return refuse("kv_release: width outside [1, 2^18], or ld_table smaller");
    if (a.n_free < 0 || a.n_pages < 1) return refuse("kv_release: n_free < 0 or n_pages < 1");
    if (a.reserved != 0) return refuse("kv_release: reserved must be 0");
    if (!a.seqs || !a.kv_lens || !a.table || !a.free_pages || !a.used || !a.refs || !a.used_out || !a.status)
        return refuse("kv_release: NULL argument");
    // a warp per unit while they last
    const long long units = (long long)a.n * ((a.width + UNIT - 1) / UNIT);
    int ctas = 1;
    while (ctas < MAXC && units > (long long)ctas * WARPS) ctas *= 2;
    return queue(cuda_stream, "kv_release: launch failed",
                 [&](const Launch& L) { launch_k(L, kv_release_kernel, dim3(1, 1, ctas), dim3(NR), 0, ctas, a, ctas); });
}
