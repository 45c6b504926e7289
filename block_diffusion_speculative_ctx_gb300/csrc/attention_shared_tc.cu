// bf16 shared-prefix attention on the 5th-generation tensor cores (the main
// kernel of dflash_shared_prefix_attention; the partial results are merged by
// attention_shared.cu).
//
// Mathematics: per query vector, running maximum m (base 2, moved only when a
// score exceeds it by more than 8, so that weights stay below 2^8), running sum
// l = sum 2^(s - m) and O = sum 2^(s - m) v, one pass over the keys; fp32
// throughout, the weights rounded once to bf16 for the product with V (the sum
// takes the unrounded ones), or held as bf16 pairs (PAIR: hi, and lo = what hi's
// rounding left, in the other half of the S buffer; O += hi V + lo V).
//
// One CTA per SM holds two streams A, B of 128 query vectors each (TMEM lanes)
// and walks its part of one of the two lines of the plan (shared_plan.cuh):
//   line 0: A and B hold different rows of one item and share every K/V tile,
//           which halves the shared-memory fill per product (tensor-bound);
//   line 1: A and B walk segments of their own with half of the ring each
//           (few query vectors, so bound by the K/V bytes).
// The CTAs of the two lines run side by side, so the bytes of one line stream
// while the other line's products run on the neighbours, and each CTA has one
// start-up.
// Roles (warps): 0-3 softmax of A, 4-7 softmax of B (a thread is one query
// vector), 8 and 9 issue the tcgen05.mma of A and of B, 10 and 11 load (on line 0
// K and V, on line 1 the tiles of A and of B; a wait costs some 190 cycles even
// when its phase is long over, so two warps share them).
//   TMEM: per stream two S buffers of 64 columns (P overwrites its S as bf16 and
//   is the A operand of P V from there) and O.  S of tile j + 1 is there before
//   the softmax of tile j ends, so the softmax never waits for a product chain.
//   Shared memory: Q_A, Q_B, a ring of K or V tiles (64 keys: one cache page),
//   all 128-byte swizzled by TMA; page numbers come 32 at a time, one a lane.
// An MMA warp issues S0, S1, then batches of P V of tile j and S of tile j + 2,
// back to back: the tensor cores execute one thread's products in order, so P V
// has read P before the next S overwrites it.  Each batch has one commit (a
// commit holds the issue up by 100 cycles and more): it tells the softmax that S
// has come and O is up to date, and the loads that the batch's V and K stages
// are free.
//
// What bounds it.  Tensor cores: 64 keys of both streams are 1260 cycles (S is fed
// from shared memory at 48 cycles an M128 N64 K16 product, P V takes 64).  Measured
// on line 0: 1750 to 1780 cycles, 1200 TFLOP/s (32 x 16 rows of 32 heads against 32768
// keys: 229 us with the merge).  That is the chain of a softmax warp, which has one tile
// at a time; by clocks read between the dependent steps of one warp a stream: wait for the
// scores 370 cycles, scores out of TMEM 140, maximum and rescue test 315, exponentials with
// the sum and the rounding 630 (two warps share a scheduler), P into TMEM 65, hand-over 70,
// loop 160; with PAIR 710, 170, 310, 855, 75, 80, 160 (2350).  Trees differ by the wait
// alone (480, with PAIR 765: 1800 and 2320 a tile).  Measured and not kept: two warps per 32 rows, half of the keys each (279 us where this took 241);
// the streams' products in turn, half a tile apart (288: one stream's products alone
// wait for their own accumulator, 69 cycles each); the next scores loaded while P is
// stored (267); hand-over by a flag in shared memory (243).
// Line 1 is bound by bytes: 6.3 TB/s of K and V on 8192 own keys of 32 sequences.  The
// small calls are a chain: lengths, plan (2200 cycles), pages, first tile (4500), its
// softmax and product (1900), partial result, merge (10.3 us for one token of four
// sequences behind 512 keys).
//
// Pairs cost 5 % where bytes or the chain of a small call bound it (32 single rows
// behind 8192 keys 43.4 -> 46.9 us) and a fifth to a quarter where the softmax does
// (32 x 16 rows behind 8192 96 -> 119 us).  Sessions take them: their other attention
// holds its weights so, and a bf16 model's verify logits behind 1024 shared keys are
// 20 % farther from 64 bits without them (rms 5.1e-3 instead of 4.2e-3).
//
// Every wait is bounded; one that runs out sets the CTA's error word (the merge
// writes NaN), every role leaves, copies in flight are awaited (bounded).
#include <math.h>

#include "shared_plan.cuh"
#include "tcgen05.cuh"

namespace dfl {

namespace {

using namespace tc;
using namespace sp;

constexpr int VT = 128, KT = 64;
constexpr int NTHR = 384;

template <int HD>
struct Cfg {
    static constexpr int HALVES = HD / 64;            // 64-dim halves: one 128-byte swizzled row each
    static constexpr int Q_REG = VT * 128, Q_TILE = HALVES * Q_REG;
    static constexpr int KV_REG = KT * 128, TILE = HALVES * KV_REG;
    static constexpr int STAGES = HD == 128 ? 8 : 16;  // 128 KB
    static constexpr int RING_AT = 2 * Q_TILE;
    static constexpr int SMEM_TILES = RING_AT + STAGES * TILE;
};

constexpr int SEGS = 4;
// A wait for batch i must not begin once batch i + DONE can have completed (the barrier's parity would be
// that of before i).  The load warps wait the latest: a stage comes round after at most 16 ring positions, and
// the shortest segments (one tile: two positions, three batches) put 24 batches on those.
constexpr int DONE = 32;
struct LineBars {
    uint64_t kv_full[2][DONE];  // per load warp: V and K of its i-th batch have landed, on barrier i % DONE
    uint64_t q_full[2], q_empty[2];
    uint64_t p_full[2][2];     // per stream and S buffer
    uint64_t done[2][DONE];    // per stream: its i-th batch of products, on barrier i % DONE
    uint64_t o_empty[2];
    uint64_t drain[2];
    uint64_t seg_full[2][SEGS], seg_empty[2][SEGS];
};
struct Bars {
    LineBars line[2];
    Seg seg[2][SEGS];  // segments handed from a load warp to the other roles
    uint32_t rel[2][16];  // per load warp: the batch that frees a stage
    uint32_t tmem;
    PlanMem<NTHR> plan;
};

struct TcArgs {
    Shape P;
    Work W;
    float scale_log2;
};

// ---- PTX
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, uint64_t* bar, int c0, int c1, int c2) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(
            dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
}
// D (TMEM) (+)= A (TMEM, bf16 pairs) . B (smem)
__device__ __forceinline__ void umma_bf16_ts(uint32_t d, uint32_t a, uint64_t b_desc, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
        "r"(a), "l"(b_desc), "r"(idesc), "r"(acc));
}
__device__ __forceinline__ void tmem_ld32_issue(uint32_t taddr, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}
// The wait names the destination registers, so that no use of them moves above it.
__device__ __forceinline__ void tmem_ld32_wait(uint32_t* r) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                   "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]),
                   "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                   "+r"(r[30]), "+r"(r[31])
                 :
                 : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// One 32-byte store (two of 16 bytes touch every sector twice: 121 us instead of 113 for the 32 prompts of 5 .. 130
// rows behind 2100 keys).
__device__ __forceinline__ void st_global8(float* p, const uint32_t* r) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(r[0]), "r"(r[1]), "r"(r[2]),
                 "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}

// Ring positions of a segment of n tiles, in the order the MMA warps consume them: K0 K1 V0 K2 V1 K3 ...
__device__ __forceinline__ uint32_t k_seq(int j) { return (uint32_t)(j + max(0, j - 1)); }
__device__ __forceinline__ uint32_t v_seq(int j, int n) { return (uint32_t)(j + min(n, j + 2)); }

// The bounded waits of one thread: after one has run out, the later ones return at once.
struct Waiter {
    uint32_t* err;
    bool ok = true;
    __device__ __forceinline__ bool operator()(uint64_t* bar, uint32_t parity) {
        if (!mbar_try_wait(bar, parity) && ok && !late(bar, parity)) {
            ok = false;
            atomicOr(err, ERR_TIMEOUT);
        }
        return ok;
    }
    // about a second
    static __device__ __noinline__ bool late(uint64_t* bar, uint32_t parity, uint32_t limit = 1u << 23) {
        for (uint32_t i = 0; i < limit; ++i) {
            if (mbar_try_wait(bar, parity)) return true;
            if (i >= 1024) __nanosleep(128);
        }
        return false;
    }
};

// PAIR: the weights of P V as bf16 pairs.  TREE: rows see the own keys that their masks name; the tiles that hold nodes of
// the tree take 64 mask bits a row (two to three words from L2, asked for before the scores are waited for) and zero the rows
// of V that no row of the item sees.  Measured (graph replay): 230 us for 32 trees of 33 .. 64 nodes behind 8192 shared keys and
// 256 .. 2048 own (1030 TFLOP/s over the call, merge 22 us: the chain above); 10.6 us for 16 nodes behind 512 keys.  With PAIR 297
// and 11.2 us.  One bf16 a weight is what a call gets that does not ask for pairs, as in the causal form, whose bits a chain's
// tree has: its output is 2.1e-3 .. 2.4e-3 (rms, relative) from 64 bits, with pairs 1.7e-3, which the output's own rounding
// makes.  Measured and not kept: sixteen softmax warps, two a vector that take its tiles in turn and pass m and l on (264 us, 12.3 for the 16 nodes: each
// has a score buffer of its own, whose next scores come behind its own product, so its loop is chain and products in a row).
template <int HD, bool PAIR, bool TREE>
__global__ void __launch_bounds__(NTHR, 1)
    shared_tc_kernel(const __grid_constant__ TcArgs a, const __grid_constant__ CUtensorMap mq,
                     const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv) {
    using C = Cfg<HD>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    uint8_t* sm = smem_raw + (((raw + 1023u) & ~1023u) - raw);
    const uint32_t sb = smem_u32(sm);
    const uint32_t q_at = sb, ring_at = sb + C::RING_AT;
    Bars* bars = reinterpret_cast<Bars*>(sm + C::SMEM_TILES);
    uint32_t* base = reinterpret_cast<uint32_t*>(bars + 1);  // [2][batch], then [batch]
    uint32_t* ibase = base + 2 * a.P.batch;

    const Shape& P = a.P;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int cta = blockIdx.x;

    if (warp == 8) {
        tmem_alloc(&bars->tmem, 512);
        tmem_relinquish();
    }
    if (warp == 9) {  // (a barrier of each ring per lane)
#pragma unroll 1
        for (int i = 0; i < 4; ++i) {
            LineBars* B = &bars->line[i >> 1];
            mbar_init(&B->done[i & 1][lane], 1);
            mbar_init(&B->kv_full[i & 1][lane], i < 2 ? 2 : 1);  // load warps that fill the batch
        }
        mbar_fence_init();
    }
    static_assert(DONE == 32, "a lane each");
    if (tid == 0) {
        for (int line = 0; line < 2; ++line) {
            LineBars* B = &bars->line[line];
            for (int x = 0; x < 2; ++x) {
                mbar_init(&B->q_full[x], 1);
                mbar_init(&B->q_empty[x], 1);
                for (int b = 0; b < 2; ++b) mbar_init(&B->p_full[x][b], 4);
                mbar_init(&B->o_empty[x], 4);
                mbar_init(&B->drain[x], 1);
                for (int i = 0; i < SEGS; ++i) {
                    mbar_init(&B->seg_full[x][i], 1);
                    mbar_init(&B->seg_empty[x][i], line == 0 ? 10 : 5);  // MMA and softmax warps that read it
                }
            }
        }
        mbar_fence_init();
    }
    if (tid == 32 * 10) {
        prefetch_tmap(&mq);
        prefetch_tmap(&mk);
        prefetch_tmap(&mv);
    }
    pdl_wait();
    if (tid == 0) a.W.err[cta] = 0u;
    Head h;
    fence_before();
    make_plan<NTHR>(P, base, ibase, &bars->plan, h);  // (its barriers order the setup above)
    fence_after();
    const uint32_t tmem = bars->tmem;
    // for the merge kernel, by the warps that have nothing to do until the first scores
    if (warp < 8) write_dir(P, h, a.W, base, ibase, warp * P.n_cta + cta, 8 * P.n_cta, lane);
    uint32_t* err = &a.W.err[cta];
    Waiter wait{err};

    // line 1's CTAs are spread evenly between line 0's
    const int before = cta * h.n1 / P.n_cta, line = (cta + 1) * h.n1 / P.n_cta - before;
    const bool pair = line == 0;
    LineBars* B = &bars->line[line];
    // ring of a stream: all stages, in step with the other stream (line 0), or half of them (line 1)
    const uint32_t depth = pair ? C::STAGES : C::STAGES / 2;
    auto stage_of = [&](uint32_t pos) { return pos & (depth - 1); };
    // the tiles of the i-th batch of stream x have landed
    auto landed = [&](int x, uint32_t i) { return wait(&B->kv_full[pair ? 0 : x][i % DONE], (i / DONE) & 1); };
    // the i-th batch of stream x has completed (i counts through the line)
    auto batch_done = [&](int x, uint32_t i) { return wait(&B->done[x][i % DONE], (i / DONE) & 1); };
    auto worker = [&](int x) { return pair ? cta - before : 2 * before + x; };
    auto first_stage = [&](int x) { return pair ? 0u : (uint32_t)x * (C::STAGES / 2); };
    uint32_t ring = 0;  // ring position of the segment's first tile
    // the i-th segment, read by a whole warp (or its one issuing lane)
    auto take = [&](int x, uint32_t i, bool all, Seg& s) {
        const int rx = pair ? 0 : x, slot = i % SEGS;
        s.n = 0;
        if (!wait(&B->seg_full[rx][slot], (i / SEGS) & 1)) return false;
        s = bars->seg[rx][slot];
        if (all) __syncwarp();
        if (!all || lane == 0) mbar_arrive(&B->seg_empty[rx][slot]);
        return s.n > 0;
    };

    if (warp >= 10) {
        // ------------------------------------------------------------ loads
        // line 0: warp 10 (x = 0) hands out the segments and loads Q and K, warp 11 V; line 1: stream x's all
        const int x = warp - 10, rx = pair ? 0 : x;
        Walk walk(P, h, line, worker(x));
        uint32_t nseg = 0, armed = 0, nb = 0;  // nb: batches before this segment
        uint32_t* rel = bars->rel[x];
        int kvh, row0, seq;
        Seg s;
#pragma unroll 1
        while (wait.ok) {
            if (!walk.next<TREE>(P, h, base, ibase, s, kvh, row0, seq)) s.n = 0;
            if (lane == 0 && rx == x) {
                const int slot = nseg % SEGS;
                if (wait(&B->seg_empty[x][slot], ((nseg / SEGS) & 1) ^ 1)) {
                    bars->seg[x][slot] = s;
                    mbar_arrive(&B->seg_full[x][slot]);
                }
            }
            const int n = s.n;
            if (n == 0) break;
            const int* pages = seq < 0 ? P.prefix_pages : P.table + (long long)seq * P.ld_table;
            const int n_pages = (s.keys + 63) >> 6;  // valid entries of `pages`
            const int oob = P.n_pages * P.Hkv * 64;  // a row behind the cache: reads as zeros
            // page numbers 32 at a time, one a lane (K tiles run up to two ahead of V tiles: a window each); past
            // the list and outside the cache: zeros
            int bad = 0, w0[2] = {-64, -64}, pg[2] = {0, 0};
            auto tile = [&](int kv, int j, uint32_t i) {
                const int first = s.t0 + j;
                if (first >= w0[kv] + 32) {
                    w0[kv] = first;
                    pg[kv] = -1;
                    if (first + lane < n_pages) {
                        pg[kv] = pages[first + lane];
                        if (pg[kv] < 0 || pg[kv] >= P.n_pages) {
                            pg[kv] = -1;
                            bad |= first + lane < s.t0 + n;
                        }
                    }
                }
                const int p = __shfl_sync(0xffffffffu, pg[kv], first - w0[kv]);
                if (lane == 0) {
                    const uint32_t pos = ring + (kv ? v_seq(j, n) : k_seq(j)), st = first_stage(x) + stage_of(pos);
                    if (pos < depth || (batch_done(rx, rel[st]) && (!pair || batch_done(1, rel[st]))))
                        tma_load_3d(ring_at + st * C::TILE, kv ? &mv : &mk, &B->kv_full[rx][i % DONE], 0,
                                    p < 0 ? oob : (p * P.Hkv + kvh) * 64, 0);
                }
            };
            auto load_q = [&]() {
                if (lane || rx != x) return;
#pragma unroll 1
                for (int y = x; y < (pair ? 2 : x + 1); ++y) {
                    if (!wait(&B->q_empty[y], (nseg & 1) ^ 1)) break;
                    mbar_arrive_expect_tx(&B->q_full[y], C::HALVES * 128 * P.g * P.RH);
#pragma unroll
                    for (int c = 0; c < C::HALVES; ++c)
                        tma_load_3d(q_at + y * C::Q_TILE + c * C::Q_REG, &mq, &B->q_full[y], 64 * c, kvh * P.g,
                                    row0 + (pair ? y * P.RH : 0));
                }
            };
#pragma unroll 1
            for (int j = -2; j < n; ++j) {
                // batch: V of tile j, K of tile j + 2
                const uint32_t i = nb + j + 2;
                const bool has_v = j >= 0, has_k = j + 2 < n;
                const bool my_v = has_v && (!pair || x == 1), my_k = has_k && (!pair || x == 0);
                if (lane == 0) {
                    uint64_t* bar = &B->kv_full[rx][i % DONE];
                    if (my_v || my_k) mbar_arrive_expect_tx(bar, (my_v + my_k) * C::TILE);
                    else mbar_arrive(bar);  // (a batch without my tiles has its phase too)
                }
                if (j == -2 && nseg == 0) load_q();  // (nothing before them: while the page numbers come)
                if (my_v) tile(1, j, i);
                if (my_k) tile(0, j + 2, i);
                if (lane == 0) {
                    if (has_v) rel[first_stage(x) + stage_of(ring + v_seq(j, n))] = i;
                    if (has_k) rel[first_stage(x) + stage_of(ring + k_seq(j + 2))] = i;
                }
                armed = i + 1;
                // (behind the first tile, whose stage waits for the segment before alone)
                if (j == -2 && nseg > 0) load_q();
                wait.ok = __shfl_sync(0xffffffffu, (int)wait.ok, 0);
                if (!wait.ok) break;
            }
            ++nseg;
            bad = __any_sync(0xffffffffu, bad);
            if (lane == 0) {
                // (on line 0 warp 10's K tiles speak for the pages)
                if (rx == x) a.W.block_bad[s.block] = bad;
                if (pair && rx == x) a.W.block_bad[s.block + 1] = bad;
            }
            ring += 2 * n;
            nb += n + 2;
        }
        if (lane == 0 && wait.ok && rx == x) {
            // the last commits have arrived: nothing is under way to this line's barriers any more
            for (int y = x; y < (pair ? 2 : x + 1); ++y)
                if (nseg) {
                    for (uint32_t i = nb > DONE ? nb - DONE : 0; i < nb; ++i) batch_done(y, i);
                    wait(&B->q_empty[y], (nseg - 1) & 1);
                }
        }
        // a wait ran out: the copies in flight must land before the CTA leaves its shared memory
        if (lane == 0 && !wait.ok) {
            for (uint32_t i = armed > DONE ? armed - DONE : 0; i < armed; ++i)
                Waiter::late(&B->kv_full[rx][i % DONE], (i / DONE) & 1, 1u << 16);
            for (int y = x; y < (pair ? 2 : x + 1); ++y)
                if (nseg) Waiter::late(&B->q_full[y], (nseg - 1) & 1, 1u << 16);
        }
    } else if (warp >= 8) {
        // ------------------------------------------------------------ MMA
        const int x = warp - 8;
        if (lane == 0) {
            constexpr uint32_t ID_S = idesc_bf16(VT, KT), ID_O = idesc_bf16(VT, HD, true);
            const uint32_t tS = tmem + 128 * x, tO = tmem + 256 + HD * x;
            const uint64_t q_desc = sw128_desc(q_at + x * C::Q_TILE);
            const uint64_t k_desc = sw128_desc(ring_at), v_desc = sw128_desc(ring_at, C::KV_REG, 1024);
            uint32_t nseg = 0, nt = 0, nb = 0;  // segments, tiles and batches before this one
            Seg s;
#pragma unroll 1
            while (take(x, nseg, false, s)) {
                const int n = s.n;
                if (!wait(&B->q_full[x], nseg & 1)) break;
#pragma unroll 1
                for (int j = -2; j < n; ++j) {
                    // batch: P V of tile j, S of tile j + 2
                    const uint32_t vst = first_stage(x) + stage_of(ring + v_seq(max(j, 0), n));
                    const uint32_t kst = first_stage(x) + stage_of(ring + k_seq(j + 2));
                    const uint32_t d = tS + 64 * ((nt + j) & 1);  // S buffer of both tiles
                    if (j >= 0 || j + 2 < n) landed(x, nb + j + 2);
                    if (j >= 0) {
                        if (j == 0) wait(&B->o_empty[x], (nseg & 1) ^ 1);  // the segment before has been read out
                        wait(&B->p_full[x][(nt + j) & 1], ((nt + j) >> 1) & 1);
                    }
                    if (!wait.ok) break;
                    fence_after();
                    if (j >= 0) {
                        const uint64_t vd = v_desc + vst * (C::TILE >> 4);
#pragma unroll
                        for (int kk = 0; kk < KT / 16; ++kk)
                            umma_bf16_ts(tO, d + 8 * kk, vd + ((kk * 2048) >> 4), ID_O, (j > 0 || kk > 0) ? 1u : 0u);
                        if constexpr (PAIR)
#pragma unroll
                            for (int kk = 0; kk < KT / 16; ++kk)
                                umma_bf16_ts(tO, d + 32 + 8 * kk, vd + ((kk * 2048) >> 4), ID_O, 1u);
                    }
                    if (j + 2 < n) {
                        const uint64_t kd = k_desc + kst * (C::TILE >> 4);
#pragma unroll
                        for (int kk = 0; kk < HD / 16; ++kk)
                            umma_bf16(d, q_desc + (((kk >> 2) * C::Q_REG + (kk & 3) * 32) >> 4),
                                      kd + (((kk >> 2) * C::KV_REG + (kk & 3) * 32) >> 4), ID_S, kk > 0 ? 1u : 0u);
                    }
                    umma_commit(&B->done[x][(nb + j + 2) % DONE]);
                    if (j + 3 == n) umma_commit(&B->q_empty[x]);
                }
                nb += n + 2;
                ++nseg;
                nt += n;
                ring += 2 * n;
            }
            if (!wait.ok) {  // products that were issued must have ended before their accumulators are freed
                umma_commit(&B->drain[x]);
                Waiter::late(&B->drain[x], 0);
            }
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ softmax
        const int x = warp >> 2, v = tid & 127, quad = warp & 3;
        const uint32_t tl = tmem + ((uint32_t)(32 * quad) << 16);
        const uint32_t tO = tl + 256 + HD * x;
        const uint64_t scale2 = pack2(a.scale_log2, a.scale_log2);
        uint32_t nt = 0, nb = 0;  // tiles and batches before this segment
        uint32_t nseg = 0;
        Seg s;
#pragma unroll 1
        while (take(x, nseg, true, s)) {
            ++nseg;
            const int n = s.n;
            const int r0 = pair ? x * P.RH : 0;  // this stream's rows of the item
            const int nv = min(P.RH, s.nrows - r0) * P.g;
            int lim = 0x7fffffff;  // (a lane of no query vector: anything)
            if (!TREE && v < nv) lim = max(s.lim0 + s.step * (r0 + v / P.g), 0);
            const bool live_warp = 32 * quad < nv;
            const int lim_warp = __reduce_min_sync(0xffffffffu, lim);
            float m_run = -INFINITY, l_run = 0.f;
#pragma unroll 1
            for (int j = 0; j < n; ++j) {
                const int k0 = (s.t0 + j) * KT;
                const uint32_t buf = (nt + j) & 1;
                const uint32_t tS = tl + 128 * x + 64 * buf;
                const bool tree_tile = TREE && k0 + KT > s.lim0;
                uint64_t sees = ~0ull, seen = ~0ull;  // keys that this vector's row sees, that some row of the item sees
                if (TREE && tree_tile) {
                    if (v < nv) sees = tree_sees64(P, s, s.row0 + r0 + v / P.g, k0);
                    uint64_t any = 0;
                    for (int r = lane; r < s.nrows; r += 32) any |= tree_sees64(P, s, s.row0 + r, k0);
                    seen = (uint64_t)__reduce_or_sync(0xffffffffu, (uint32_t)(any >> 32)) << 32 |
                           __reduce_or_sync(0xffffffffu, (uint32_t)any);
                }
                if (!batch_done(x, nb + j)) break;
                fence_after();
                if (TREE ? seen != ~0ull : k0 + KT > s.keys) {
                    // the list ends inside this tile: zero the rows of V behind it (a page's unused slots may
                    // hold anything, and 0 * NaN is NaN); on line 0 both streams do, each before its own P V
                    const uint32_t st = first_stage(x) + stage_of(ring + v_seq(j, n));
                    if (!landed(x, nb + j + 2)) break;
                    uint8_t* V = sm + C::RING_AT + st * C::TILE;
                    for (int i = (TREE ? 0 : (s.keys - k0) * 8) + v; i < KT * 8; i += 128)
                        if (!TREE || !(seen >> (i >> 3) & 1u))
#pragma unroll
                        for (int c = 0; c < C::HALVES; ++c)
                            *reinterpret_cast<uint4*>(V + c * C::KV_REG + i * 16) = make_uint4(0u, 0u, 0u, 0u);
                    fence_proxy_async();
                }
                if (live_warp) {
                    uint32_t sr[KT];
                    tmem_ld32_issue(tS, sr);
                    tmem_ld32_issue(tS + 32, sr + 32);
                    tmem_ld32_wait(sr);
                    tmem_ld32_wait(sr + 32);
                    if (TREE) {
                        if (tree_tile) {
                            const uint32_t w[2] = {(uint32_t)sees, (uint32_t)(sees >> 32)};
#pragma unroll
                            for (int c = 0; c < KT; ++c)
                                if (!(w[c >> 5] >> (c & 31) & 1u)) sr[c] = 0xFF800000u;
                        }
                    } else if (k0 + KT > lim_warp) {
                        const int left = lim - k0;
#pragma unroll
                        for (int c = 0; c < KT; ++c)
                            if (c >= left) sr[c] = 0xFF800000u;  // -inf
                    }
                    float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int c = 0; c < KT; c += 2)
                        mx4[(c >> 1) & 3] =
                            fmaxf(fmaxf(mx4[(c >> 1) & 3], __uint_as_float(sr[c])), __uint_as_float(sr[c + 1]));
                    const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])) * a.scale_log2;
                    const float m_new = v < nv && mx > m_run + 8.f ? mx : m_run;
                    if (j > 0 && __any_sync(0xffffffffu, m_new != m_run)) {
                        // O holds the tiles before this one once the product of the last of them has completed
                        if (!batch_done(x, nb + j + 1)) break;
                        fence_after();
                        const float alpha = m_run == -INFINITY ? 0.f : ex2(m_run - m_new);
                        l_run *= alpha;
#pragma unroll 1
                        for (int c = 0; c < HD; c += 32) {
                            uint32_t o[32];
                            tmem_ld32_issue(tO + c, o);
                            tmem_ld32_wait(o);
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                            tmem_st32(tO + c, o);
                        }
                    }
                    m_run = m_new;
                    const float neg = m_run == -INFINITY ? 0.f : -m_run;
                    const uint64_t neg2 = pack2(neg, neg);
                    uint64_t sum2[2] = {0ull, 0ull};
                    uint32_t pk[KT / 2], pl[PAIR ? KT / 2 : 1];  // weights, and what their rounding left
#pragma unroll
                    for (int e = 0; e < KT / 2; ++e) {
                        float x0, x1;
                        unpack2(fma2(pack2(__uint_as_float(sr[2 * e]), __uint_as_float(sr[2 * e + 1])), scale2, neg2), x0, x1);
                        x0 = ex2(x0);
                        x1 = ex2(x1);
                        sum2[e & 1] = add2(sum2[e & 1], pack2(x0, x1));
                        pk[e] = pack2_bf16(x0, x1);
                        if constexpr (PAIR)
                            pl[e] = pack2_bf16(x0 - __uint_as_float(pk[e] << 16), x1 - __uint_as_float(pk[e] & 0xFFFF0000u));
                    }
                    tmem_st32(tS, pk);
                    if constexpr (PAIR) tmem_st32(tS + 32, pl);
                    float s0, s1;
                    unpack2(add2(sum2[0], sum2[1]), s0, s1);
                    l_run += s0 + s1;
                    tmem_st_wait();
                }
                fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&B->p_full[x][buf]);
            }
            if (!batch_done(x, nb + n + 1)) break;
            fence_after();
            if (live_warp) {
                const size_t blk = s.block + (pair ? x : 0);
                if (v < nv) a.W.ml[blk * VT + v] = make_float2(m_run, l_run);
                float* o = a.W.o + blk * VT * HD + (size_t)v * 8;
#pragma unroll 1
                for (int c = 0; c < HD; c += 32) {
                    uint32_t r[32];
                    tmem_ld32_issue(tO + c, r);
                    tmem_ld32_wait(r);
                    if (v < nv)
#pragma unroll
                        for (int e = 0; e < 4; ++e) st_global8(o + (size_t)(c / 8 + e) * VT * 8, r + 8 * e);
                }
            }
            fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&B->o_empty[x]);
            nt += n;
            nb += n + 2;
            ring += 2 * n;
        }
    }
    __syncwarp();
    // (not earlier: the merge's CTAs would gather on the SMs that are free first)
    pdl_trigger();
    fence_before();
    __syncthreads();
    if (warp == 8) {
        fence_after();
        tmem_dealloc(tmem, 512);
    }
}

typedef CUresult (*EncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                             const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                             CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
    static EncodeFn fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess)
            p = nullptr;
        return (EncodeFn)p;
    }();
    return fn;
}

bool encode(CUtensorMap* m, int rank, const void* ptr, const cuuint64_t* dims, const cuuint64_t* strides,
            const cuuint32_t* box) {
    const EncodeFn fn = encode_fn();
    if (!fn) return false;
    const cuuint32_t es[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(ptr), dims, strides, box, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int HD, bool PAIR, bool TREE>
bool run(const Launch& L, const Shape& P, const Work& W, const dflash_shared_prefix_args& a) {
    using C = Cfg<HD>;
    TcArgs t;
    t.P = P;
    t.W = W;
    t.scale_log2 = (float)((double)a.scale * 1.4426950408889634);
    CUtensorMap mq, mk, mv;
    {
        const cuuint64_t dims[3] = {(cuuint64_t)HD, (cuuint64_t)P.H, (cuuint64_t)P.rows};
        const cuuint64_t strides[2] = {(cuuint64_t)HD * 2, (cuuint64_t)a.ld_q * 2};
        const cuuint32_t box[3] = {64, (cuuint32_t)P.g, (cuuint32_t)P.RH};
        if (!encode(&mq, 3, a.q, dims, strides, box)) return false;
    }
    {
        // the caches as [halves of a row][rows][64]: one copy brings a page's keys of one KV head as 64-dim halves
        const cuuint64_t dims[3] = {64, (cuuint64_t)P.n_pages * P.Hkv * 64, (cuuint64_t)HD / 64};
        const cuuint64_t strides[2] = {(cuuint64_t)HD * 2, 128};
        const cuuint32_t box[3] = {64, 64, (cuuint32_t)HD / 64};
        if (!encode(&mk, 3, a.k_cache, dims, strides, box) || !encode(&mv, 3, a.v_cache, dims, strides, box)) return false;
    }
    const size_t smem = C::SMEM_TILES + sizeof(Bars) + 3 * P.batch * 4 + 1024;
    if (cudaFuncSetAttribute(shared_tc_kernel<HD, PAIR, TREE>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
        return false;
    launch_k(L, shared_tc_kernel<HD, PAIR, TREE>, dim3(P.n_cta), dim3(NTHR), smem, 1, t, mq, mk, mv);
    return true;
}

}  // namespace

namespace {

template <bool TREE>
bool pick(const Launch& L, const sp::Shape& P, const sp::Work& W, const dflash_shared_prefix_args& a) {
    if (a.flags & DFLASH_ATTENTION_WEIGHT_PAIRS)
        return P.hd == 128 ? run<128, true, TREE>(L, P, W, a) : run<64, true, TREE>(L, P, W, a);
    return P.hd == 128 ? run<128, false, TREE>(L, P, W, a) : run<64, false, TREE>(L, P, W, a);
}

}  // namespace

bool shared_attention_tc(const Launch& L, const sp::Shape& P, const sp::Work& W, const dflash_shared_prefix_args& a) {
    return P.masks ? pick<true>(L, P, W, a) : pick<false>(L, P, W, a);
}

}  // namespace dfl
