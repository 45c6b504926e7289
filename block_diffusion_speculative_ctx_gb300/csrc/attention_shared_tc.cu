// bf16 shared-prefix attention on the 5th-generation tensor cores (the main
// kernel of dflash_shared_prefix_attention; the partial results are merged by
// attention_shared.cu).
//
// Mathematics: per query vector, running maximum m (base 2, moved only when a
// score exceeds it by more than 8, so that weights stay below 2^8), running sum
// l = sum 2^(s - m) and O = sum 2^(s - m) v, one pass over the keys; fp32
// throughout, the weights rounded once to bf16 for the product with V (the sum
// takes the unrounded ones).
//
// One CTA per SM walks its segments of the plan (shared_plan.cuh).  A segment
// holds up to two streams A, B of 128 query vectors (TMEM lanes):
//   pair: A and B hold different rows and share every K/V tile, which halves
//         the shared-memory fill per product;
//   one:  A and B hold the same rows, A takes the even tiles and B the odd ones.
// Roles (warps): 0-3 softmax of A, 4-7 softmax of B (a thread is one query
// vector), 8 issues every tcgen05.mma, 9 loads.  While the tensor cores work on
// one stream's P V and next Q K^T, the other stream's softmax runs.
//   TMEM: S_A, S_B (128 columns each; P overwrites its S as bf16 and is the A
//   operand of P V from there), O_A, O_B.
//   Shared memory: Q_A, Q_B, a ring of 128-key K or V tiles (two cache pages),
//   all 128-byte swizzled by TMA; page numbers come 32 at a time, one a lane.
// Order of the MMA warp within a step: P V of A, Q K^T of A's next tile, then
// B's: the tensor cores execute in order, so P V has read P before the next S
// overwrites it, and a completed S implies that the P V before it has completed.
//
// Every wait is bounded; one that runs out sets the CTA's error word (the merge
// writes NaN), every role leaves, copies in flight are awaited (bounded).
#include <math.h>
#include <stdio.h>

#include "shared_plan.cuh"
#include "tcgen05.cuh"

namespace dfl {

namespace {

using namespace tc;
using namespace sp;

constexpr int VT = 128, KT = 128;
constexpr int NTHR = 320;

template <int HD>
struct Cfg {
    static constexpr int HALVES = HD / 64;
    static constexpr int REG = 128 * 128;             // 128 rows of 64 elements
    static constexpr int TILE = HALVES * REG;         // Q, K or V tile
    static constexpr int STAGES = HD == 128 ? 4 : 8;
    static constexpr int SMEM_TILES = (2 + STAGES) * TILE;
};

struct Bars {
    uint64_t kv_full[8], kv_empty[8];
    uint64_t q_full, q_empty;
    uint64_t s_full[2], p_full[2], o_full[2], o_empty[2];
    uint32_t tmem;
    int flag;
    int fail;
    uint32_t ws[2 * NTHR / 32];
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
__device__ __forceinline__ void tma_load_2d_u(uint32_t dst, const CUtensorMap* map, uint64_t* bar, int c0, int c1) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1)
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
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Ring positions of a segment of n tiles, in the order the MMA warp consumes them.
// pair: K0 V0 K1 V1 ...; one: K0 K1 V0 K2 V1 K3 ...
__device__ __forceinline__ uint32_t k_seq(bool pair, int j) { return pair ? 2u * j : (uint32_t)(j + max(0, j - 1)); }
__device__ __forceinline__ uint32_t v_seq(bool pair, int j, int n) {
    return pair ? 2u * j + 1u : (uint32_t)(j + min(n, j + 2));
}

template <int HD>
__global__ void __launch_bounds__(NTHR, 1)
    shared_tc_kernel(const __grid_constant__ TcArgs a, const __grid_constant__ CUtensorMap mq,
                     const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv) {
    using C = Cfg<HD>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    uint8_t* sm = smem_raw + (((raw + 1023u) & ~1023u) - raw);
    const uint32_t sb = smem_u32(sm);
    const uint32_t q_at = sb, ring_at = sb + 2 * C::TILE;
    Bars* B = reinterpret_cast<Bars*>(sm + C::SMEM_TILES);
    uint32_t* base = reinterpret_cast<uint32_t*>(B + 1);
    uint32_t* ibase = base + a.P.batch;

    const Shape& P = a.P;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int cta = blockIdx.x;

    if (warp == 8) {
        tmem_alloc(&B->tmem, 512);
        tmem_relinquish();
    }
    if (tid == 0) {
        for (int i = 0; i < C::STAGES; ++i) {
            mbar_init(&B->kv_full[i], 1);
            mbar_init(&B->kv_empty[i], 1);
        }
        mbar_init(&B->q_full, 1);
        mbar_init(&B->q_empty, 1);
        for (int x = 0; x < 2; ++x) {
            mbar_init(&B->s_full[x], 1);
            mbar_init(&B->p_full[x], 4);
            mbar_init(&B->o_full[x], 1);
            mbar_init(&B->o_empty[x], 4);
        }
        mbar_fence_init();
        B->fail = 0;
    }
    if (tid == 32 * 9) {
        prefetch_tmap(&mq);
        prefetch_tmap(&mk);
        prefetch_tmap(&mv);
    }
    pdl_wait();
    pdl_trigger();
    if (tid == 0) a.W.err[cta] = 0u;
    Head h;
    fence_before();
    make_plan<NTHR>(P, base, ibase, B->ws, &B->flag, h);  // (its barriers order the setup above)
    fence_after();
    const uint32_t tmem = B->tmem;
    if (cta == 0) {
        if (tid == 0) *a.W.head = h;
        for (int s = tid; s < P.batch; s += NTHR) {
            a.W.base[s] = base[s];
            a.W.ibase[s] = ibase[s];
        }
    }
    uint32_t* err = &a.W.err[cta];
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (ok && !mbar_wait(bar, parity, err)) {
            ok = false;
            *(volatile int*)&B->fail = 1;
        }
        return ok;
    };

    Walk walk(h, cta, P.n_cta);
    Seg s;
    uint32_t ring = 0;  // ring position of the segment's first tile
    uint32_t issued = 0;
    if (warp == 9) {
        // ------------------------------------------------------------ loads
        uint32_t nseg = 0;
        while (ok && walk.next(P, h, base, ibase, s)) {
            const int n = s.t1 - s.t0;
            const int* pages = s.seq < 0 ? P.prefix_pages : P.table + (long long)s.seq * P.ld_table;
            const int n_pages = (s.keys + 63) >> 6;  // valid entries of `pages`
            const uint32_t oob = (uint32_t)P.n_pages * P.Hkv * 64;
            uint32_t bad = 0;
            // windows of 32 page numbers, one a lane, for the K and the V tiles
            int kw = -64, vw = -64, kpg = 0, vpg = 0;
            auto tile = [&](bool is_v, int j) {
                int& w0 = is_v ? vw : kw;
                int& pg = is_v ? vpg : kpg;
                const int first = 2 * (s.t0 + j);
                if (first >= w0 + 32 || first < w0) {
                    w0 = first;
                    pg = first + lane < n_pages ? pages[first + lane] : -2;
                    // past the list: zeros; outside the cache: zeros, and the segment is bad
                    if (pg != -2 || first + lane < n_pages) {
                        if (pg < 0 || pg >= P.n_pages) {
                            pg = -1;
                        }
                    }
                }
                const int p0 = __shfl_sync(0xffffffffu, pg, first - w0), p1 = __shfl_sync(0xffffffffu, pg, first - w0 + 1);
                if (p0 == -1 || p1 == -1) bad = 1;
                const uint32_t pos = ring + (is_v ? v_seq(s.pair, j, n) : k_seq(s.pair, j));
                const int st = pos % C::STAGES;
                if (lane == 0) {
                    if (wait(&B->kv_empty[st], ((pos / C::STAGES) & 1) ^ 1)) {
                        mbar_arrive_expect_tx(&B->kv_full[st], C::TILE);
                        const uint32_t dst = ring_at + st * C::TILE;
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int pgi = i ? p1 : p0;
                            const int row = pgi < 0 ? (int)oob : (pgi * P.Hkv + s.kvh) * 64;
#pragma unroll
                            for (int c = 0; c < C::HALVES; ++c)
                                tma_load_2d_u(dst + c * C::REG + i * 64 * 128, is_v ? &mv : &mk, &B->kv_full[st], 64 * c, row);
                        }
                        issued = pos + 1;
                    }
                }
                ok = __shfl_sync(0xffffffffu, (int)ok, 0);
            };
            auto load_q = [&]() {
                if (lane == 0) {
                    if (wait(&B->q_empty, (nseg & 1) ^ 1)) {
                        mbar_arrive_expect_tx(&B->q_full, (s.pair ? 2 : 1) * C::HALVES * 128 * P.g * P.RH);
                        for (int x = 0; x < (s.pair ? 2 : 1); ++x)
#pragma unroll
                            for (int c = 0; c < C::HALVES; ++c)
                                tma_load_3d(q_at + x * C::TILE + c * C::REG, &mq, &B->q_full, 64 * c, s.kvh * P.g,
                                            s.row0 + x * P.RH);
                        ++nseg;
                    }
                }
                ok = __shfl_sync(0xffffffffu, (int)ok, 0);
            };
            // the queries after the first two tiles: those wait for stages of the segment before only
            if (s.pair) {
                for (int j = 0; j < n && ok; ++j) {
                    tile(false, j);
                    tile(true, j);
                    if (j == 0) load_q();
                }
            } else {
                tile(false, 0);
                if (n > 1) tile(false, 1);
                if (n == 1) tile(true, 0);
                load_q();
                for (int j = n == 1 ? 1 : 0; j < n && ok; ++j) {
                    tile(true, j);
                    if (j + 2 < n) tile(false, j + 2);
                }
            }
            if (lane == 0) a.W.slot_bad[s.slot] = bad;
            ring += 2 * n;
        }
        // a wait ran out: the copies in flight must land before the CTA leaves its shared memory
        if (lane == 0 && !ok) {
            const uint32_t lo = issued > C::STAGES ? issued - C::STAGES : 0;
            for (uint32_t pos = lo; pos < issued; ++pos) mbar_wait(&B->kv_full[pos % C::STAGES], (pos / C::STAGES) & 1, err);
            if (nseg) mbar_wait(&B->q_full, (nseg - 1) & 1, err);
        }
    } else if (warp == 8) {
        // ------------------------------------------------------------ MMA
        if (lane == 0) {
            constexpr uint32_t ID_S = idesc_bf16(VT, KT), ID_O = idesc_bf16(VT, HD, true);
            uint32_t nseg = 0, np[2] = {0, 0}, no[2] = {0, 0};
            while (ok && walk.next(P, h, base, ibase, s)) {
                const int n = s.t1 - s.t0;
                const int nx[2] = {s.pair ? n : (n + 1) / 2, s.pair ? n : n / 2};
                int s_left = nx[0] + nx[1];
                auto issue_s = [&](int x, int k) {
                    const uint32_t pos = ring + k_seq(s.pair, s.pair ? k : 2 * k + x);
                    const int st = pos % C::STAGES;
                    if (!wait(&B->kv_full[st], (pos / C::STAGES) & 1)) return;
                    fence_after();
                    const uint32_t qa = q_at + (s.pair ? x : 0) * C::TILE, kb = ring_at + st * C::TILE;
                    const uint32_t d = tmem + 128 * x;
#pragma unroll
                    for (int kk = 0; kk < HD / 16; ++kk)
                        umma_bf16(d, sw128_desc(qa + (kk >> 2) * C::REG + (kk & 3) * 32),
                                  sw128_desc(kb + (kk >> 2) * C::REG + (kk & 3) * 32), ID_S, kk > 0 ? 1u : 0u);
                    umma_commit(&B->s_full[x]);
                    if (!s.pair || x == 1) umma_commit(&B->kv_empty[st]);
                    if (--s_left == 0) umma_commit(&B->q_empty);
                };
                wait(&B->q_full, nseg & 1);
                ++nseg;
                for (int x = 0; x < 2; ++x)
                    if (ok && nx[x] > 0) issue_s(x, 0);
                for (int k = 0; k < nx[0] && ok; ++k)
                    for (int x = 0; x < 2; ++x) {
                        if (!ok || k >= nx[x]) continue;
                        if (k == 0) {
                            wait(&B->o_empty[x], (no[x] & 1) ^ 1);  // the segment before has been read out
                            ++no[x];
                        }
                        wait(&B->p_full[x], np[x] & 1);
                        ++np[x];
                        const uint32_t pos = ring + v_seq(s.pair, s.pair ? k : 2 * k + x, n);
                        const int st = pos % C::STAGES;
                        wait(&B->kv_full[st], (pos / C::STAGES) & 1);
                        if (!ok) break;
                        fence_after();
                        const uint32_t vb = ring_at + st * C::TILE;
                        const uint32_t d = tmem + 256 + HD * x, pa = tmem + 128 * x;
#pragma unroll
                        for (int kk = 0; kk < KT / 16; ++kk)
                            umma_bf16_ts(d, pa + 8 * kk, sw128_desc(vb + kk * 2048, C::REG, 1024), ID_O,
                                         (k > 0 || kk > 0) ? 1u : 0u);
                        if (!s.pair || x == 1) umma_commit(&B->kv_empty[st]);
                        if (k == nx[x] - 1) umma_commit(&B->o_full[x]);
                        else issue_s(x, k + 1);
                    }
                ring += 2 * n;
            }
        }
    } else {
        // ------------------------------------------------------------ softmax
        const int x = warp >> 2, v = tid & 127, quad = warp & 3;
        const uint32_t tl = tmem + ((uint32_t)(32 * quad) << 16);
        const uint32_t tS = tl + 128 * x, tO = tl + 256 + HD * x;
        uint32_t ns = 0, no = 0;
        while (ok && walk.next(P, h, base, ibase, s)) {
            const int n = s.t1 - s.t0;
            const int nx = s.pair ? n : (n + 1 - x) / 2;
            const int r0 = s.pair ? x * P.RH : 0;  // this stream's rows of the item
            const int nv = min(P.RH, s.nrows - r0) * P.g;
            int lim = 0;
            if (v < nv) lim = (s.seq >= 0 && P.causal) ? max(s.lim0 + r0 + v / P.g, 0) : s.keys;
            const bool live_warp = 32 * quad < nv;
            float m_run = -INFINITY, l_run = 0.f;
            for (int k = 0; k < nx; ++k) {
                const int j = s.pair ? k : 2 * k + x, k0 = (s.t0 + j) * KT;
                if (!wait(&B->s_full[x], ns & 1)) break;
                ++ns;
                fence_after();
                if (k0 + KT > s.keys && (!s.pair || x == 0)) {
                    // the list ends inside this tile: zero the rows of V behind it (a page's unused slots
                    // may hold anything, and 0 * NaN is NaN).  In a pair A's P V comes first.
                    const uint32_t pos = ring + v_seq(s.pair, j, n);
                    const int st = pos % C::STAGES;
                    if (!wait(&B->kv_full[st], (pos / C::STAGES) & 1)) break;
                    const int first = s.keys - k0;
                    uint8_t* V = sm + 2 * C::TILE + st * C::TILE;
                    for (int i = first * 8 + v; i < KT * 8; i += 128)
#pragma unroll
                        for (int c = 0; c < C::HALVES; ++c)
                            *reinterpret_cast<uint4*>(V + c * C::REG + i * 16) = make_uint4(0u, 0u, 0u, 0u);
                    fence_proxy_async();
                }
                if (live_warp) {
                    uint32_t sr[128];
#pragma unroll
                    for (int c = 0; c < 4; ++c) tmem_ld32_issue(tS + 32 * c, sr + 32 * c);
#pragma unroll
                    for (int c = 0; c < 4; ++c) tmem_ld32_wait(sr + 32 * c);
                    if (__any_sync(0xffffffffu, k0 + KT > lim)) {
                        const int left = lim - k0;
#pragma unroll
                        for (int c = 0; c < 128; ++c)
                            if (c >= left) sr[c] = 0xFF800000u;  // -inf
                    }
                    float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int c = 0; c < 128; ++c) mx4[c & 3] = fmaxf(mx4[c & 3], __uint_as_float(sr[c]));
                    const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])) * a.scale_log2;
                    const float m_new = mx > m_run + 8.f ? mx : m_run;
                    if (k > 0 && __any_sync(0xffffffffu, m_new != m_run)) {
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
                    float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        uint32_t pk[32];
#pragma unroll
                        for (int e = 0; e < 32; ++e) {
                            const float p0 = ex2(fmaf(__uint_as_float(sr[64 * c + 2 * e]), a.scale_log2, neg));
                            const float p1 = ex2(fmaf(__uint_as_float(sr[64 * c + 2 * e + 1]), a.scale_log2, neg));
                            sum[(2 * e) & 3] += p0;
                            sum[(2 * e + 1) & 3] += p1;
                            pk[e] = pack2_bf16(p0, p1);
                        }
                        tmem_st32(tS + 32 * c, pk);
                    }
                    l_run += (sum[0] + sum[1]) + (sum[2] + sum[3]);
                    tmem_st_wait();
                }
                fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&B->p_full[x]);
            }
            if (nx > 0 && wait(&B->o_full[x], no & 1)) {
                ++no;
                fence_after();
                if (live_warp) {
                    const size_t slot = (size_t)s.slot * 2 + x;
                    if (v < nv) a.W.ml[slot * VT + v] = make_float2(m_run, l_run);
                    float* o = a.W.o + slot * VT * HD + (size_t)v * 8;
#pragma unroll 1
                    for (int c = 0; c < HD; c += 32) {
                        uint32_t r[32];
                        tmem_ld32_issue(tO + c, r);
                        tmem_ld32_wait(r);
                        if (v < nv)
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                float* d = o + (size_t)(c / 8 + e) * VT * 8;
                                *reinterpret_cast<uint4*>(d) = make_uint4(r[8 * e], r[8 * e + 1], r[8 * e + 2], r[8 * e + 3]);
                                *reinterpret_cast<uint4*>(d + 4) =
                                    make_uint4(r[8 * e + 4], r[8 * e + 5], r[8 * e + 6], r[8 * e + 7]);
                            }
                    }
                }
                fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&B->o_empty[x]);
            }
            ring += 2 * n;
        }
    }
    __syncwarp();
    fence_before();
    __syncthreads();
    if (warp == 8) {
        fence_after();
        if (B->fail) {
            // products that were issued must have ended before their accumulators are freed
            if (lane == 0) {
                mbar_init(&B->q_full, 1);
                mbar_fence_init();
                umma_commit(&B->q_full);
                mbar_wait(&B->q_full, 0, err);
            }
            __syncwarp();
        }
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

template <int HD>
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
        const cuuint64_t dims[2] = {(cuuint64_t)HD, (cuuint64_t)P.n_pages * P.Hkv * 64};
        const cuuint64_t strides[1] = {(cuuint64_t)HD * 2};
        const cuuint32_t box[2] = {64, 64};
        if (!encode(&mk, 2, a.k_cache, dims, strides, box) || !encode(&mv, 2, a.v_cache, dims, strides, box)) return false;
    }
    const size_t smem = C::SMEM_TILES + sizeof(Bars) + (size_t)P.batch * 8 + 1024;
    if (cudaFuncSetAttribute(shared_tc_kernel<HD>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
        return false;
    launch_k(L, shared_tc_kernel<HD>, dim3(P.n_cta), dim3(NTHR), smem, 1, t, mq, mk, mv);
    return true;
}

}  // namespace

bool shared_attention_tc(const Launch& L, const sp::Shape& P, const sp::Work& W, const dflash_shared_prefix_args& a) {
    return P.hd == 128 ? run<128>(L, P, W, a) : run<64>(L, P, W, a);
}

}  // namespace dfl
