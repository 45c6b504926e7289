// fp32 shared-prefix attention on the CUDA cores (the main kernel of
// dflash_shared_prefix_attention for F32; attention_shared.cu merges).
//
// The same plan as the bf16 kernel with one line of work (shared_plan.cuh): a
// worker is a CTA of 128 threads with 32 or 64 query vectors, an item one KV
// head's vectors of that many / g rows, a tile 32 keys (half a page).  Per tile
//   S = Q K^T   a thread has 2 or 4 vectors x 4 keys: 32 or 64 FMAs per 6 or 8
//               vector loads from shared memory;
//   softmax     online in fp32 (base 2); a vector's 32 scores lie in 8 lanes;
//   O += P V    a thread has 2 or 4 vectors x hd / 8 dimensions.
// K and V of the next tile land (cp.async, double-buffered) meanwhile; keys behind
// the list's end are filled with zeros, so what a page's unused slots hold never
// matters.  Bound by the FMA pipes and shared memory for long work, by the chain
// lengths -> pages -> tile for the short calls that fp32 models make: 8.7 us (merge
// included, graph replay) for 3 blocks of 4 rows behind 500 keys, whose bytes take
// 0.1 us; the tiles of a plain fp32 kernel without the plan took 184 us.  64 vectors
// a worker where a sequence has more than 32 per KV head on average: 16 rows of 8
// sequences behind 4096 keys take 226 us (39 TFLOP/s) at 32 heads of 128 and 68 us at
// 16 heads of 64, with 32 vectors 339 and 116 us; sequences that fit 32 would compute
// in vain on their own keys (16 x 1 row, 2000 own keys: 216 us with 64, 164 with 32).
#include <math.h>

#include "shared_plan.cuh"

namespace dfl {

namespace {

using namespace sp;

constexpr int NT = 128, KT = 32;

template <int HD, int VT>
struct Smem {
    static constexpr int LD = HD + 4;  // rows 16 bytes apart in the banks
    float q[VT][LD];
    float k[2][KT][LD];
    float v[2][KT][LD];
    float p[VT][KT + 4];
    PlanMem<NT> plan;
    uint32_t base[1];  // [2][batch], then ibase [batch]
};

struct F32Args {
    Shape P;
    Work W;
    const float *q, *k, *v;
    long long ld_q;
    float scale_log2;
};

__device__ __forceinline__ void cp16(float* dst, const float* src, bool full) {
    const uint32_t d = (uint32_t)__cvta_generic_to_shared(dst);
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d), "l"(src), "r"(full ? 16 : 0) : "memory");
}

// UV query vectors a thread.
template <int HD, int UV>
__global__ void __launch_bounds__(NT, 2) shared_f32_kernel(F32Args a) {
    extern __shared__ __align__(16) uint8_t raw[];
    constexpr int VT = 16 * UV;
    Smem<HD, VT>& S = *reinterpret_cast<Smem<HD, VT>*>(raw);
    constexpr int C4 = HD / 4, DPT = HD / 32;  // float4 per row; float4 of O per thread and vector
    const Shape& P = a.P;
    const int tid = threadIdx.x, lane = tid & 31, cta = blockIdx.x;
    const int tv = tid >> 3, td = tid & 7;  // vectors UV tv ..; keys td + 8 i, dimensions 4 td + 32 i
    pdl_wait();
    Head h;
    uint32_t *base = S.base, *ibase = base + 2 * P.batch;
    make_plan<NT>(P, base, ibase, &S.plan, h);
    if (cta < P.n_cta && tid == 0) a.W.err[cta] = 0u;
    write_dir(P, h, a.W, base, ibase, (tid >> 5) * gridDim.x + cta, gridDim.x * (NT / 32), lane);

    Walk walk(P, h, 1, cta);
    Seg s;
    int kvh, row0, seq;
#pragma unroll 1
    while (walk.next(P, h, base, ibase, s, kvh, row0, seq)) {
        const int* pages = seq < 0 ? P.prefix_pages : P.table + (long long)seq * P.ld_table;
        const int nv = s.nrows * P.g;
        int bad = 0;
        auto load = [&](int j) {
            const int k0 = (s.t0 + j) * KT, page = pages[k0 >> 6];
            const bool in = page >= 0 && page < P.n_pages;
            bad |= !in;
            const long long off = (((long long)(in ? page : 0) * (P.Hkv / P.parts) + kvh / P.parts) * 64 + (k0 & 63)) * HD;
#pragma unroll 4
            for (int i = tid; i < KT * C4; i += NT) {
                const int r = i / C4, c = i - r * C4;
                const bool full = in && k0 + r < s.keys;
                cp16(&S.k[j & 1][r][4 * c], a.k + off + r * HD + 4 * c, full);
                cp16(&S.v[j & 1][r][4 * c], a.v + off + r * HD + 4 * c, full);
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        load(0);
        for (int i = tid; i < VT * C4; i += NT) {
            const int v = i / C4, c = i - v * C4;
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (v < nv) {
                const int r = v / P.g, hh = v - r * P.g;
                x = *reinterpret_cast<const float4*>(a.q + (long long)(row0 + r) * a.ld_q + (long long)(kvh * P.g + hh) * HD + 4 * c);
            }
            *reinterpret_cast<float4*>(&S.q[v][4 * c]) = x;
        }
        int lim[UV];
        float m[UV], l[UV];
        float4 o[UV][DPT];
#pragma unroll
        for (int u = 0; u < UV; ++u) {
            const int v = UV * tv + u;
            m[u] = -INFINITY;
            l[u] = 0.f;
            lim[u] = v < nv ? max(s.lim0 + s.step * (v / P.g), 0) : 0;
#pragma unroll
            for (int i = 0; i < DPT; ++i) o[u][i] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll 1
        for (int j = 0; j < s.n; ++j) {
            asm volatile("cp.async.wait_group 0;" ::: "memory");
            __syncthreads();  // the tile has come; the other buffer and P are free
            if (j + 1 < s.n) load(j + 1);
            const int b = j & 1, k0 = (s.t0 + j) * KT;
            float sc[UV][4];
#pragma unroll
            for (int u = 0; u < UV; ++u)
#pragma unroll
                for (int i = 0; i < 4; ++i) sc[u][i] = 0.f;
#pragma unroll 4
            for (int c = 0; c < HD; c += 4) {
                float4 q[UV];
#pragma unroll
                for (int u = 0; u < UV; ++u) q[u] = *reinterpret_cast<const float4*>(&S.q[UV * tv + u][c]);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float4 k = *reinterpret_cast<const float4*>(&S.k[b][td + 8 * i][c]);
#pragma unroll
                    for (int u = 0; u < UV; ++u)
                        sc[u][i] = fmaf(q[u].w, k.w, fmaf(q[u].z, k.z, fmaf(q[u].y, k.y, fmaf(q[u].x, k.x, sc[u][i]))));
                }
            }
#pragma unroll
            for (int u = 0; u < UV; ++u) {
                float mx = -INFINITY;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    sc[u][i] = k0 + td + 8 * i < lim[u] ? sc[u][i] * a.scale_log2 : -INFINITY;
                    mx = fmaxf(mx, sc[u][i]);
                }
#pragma unroll
                for (int x = 1; x < 8; x <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
                const float mn = fmaxf(m[u], mx), ref = mn == -INFINITY ? 0.f : mn;
                const float al = exp2f(m[u] - ref);  // (0 while there was no key)
                m[u] = mn;
                float sum = 0.f;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    sc[u][i] = exp2f(sc[u][i] - ref);
                    sum += sc[u][i];
                    S.p[UV * tv + u][td + 8 * i] = sc[u][i];
                }
#pragma unroll
                for (int x = 1; x < 8; x <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
                l[u] = l[u] * al + sum;
#pragma unroll
                for (int i = 0; i < DPT; ++i) {
                    o[u][i].x *= al;
                    o[u][i].y *= al;
                    o[u][i].z *= al;
                    o[u][i].w *= al;
                }
            }
            __syncwarp();  // a vector's weights were written by its own eight lanes
#pragma unroll 2
            for (int k = 0; k < KT; k += 4) {
                float p[UV][4];
#pragma unroll
                for (int u = 0; u < UV; ++u) {
                    const float4 x = *reinterpret_cast<const float4*>(&S.p[UV * tv + u][k]);
                    p[u][0] = x.x;
                    p[u][1] = x.y;
                    p[u][2] = x.z;
                    p[u][3] = x.w;
                }
#pragma unroll
                for (int e = 0; e < 4; ++e)
#pragma unroll
                    for (int i = 0; i < DPT; ++i) {
                        const float4 x = *reinterpret_cast<const float4*>(&S.v[b][k + e][4 * td + 32 * i]);
#pragma unroll
                        for (int u = 0; u < UV; ++u) {
                            o[u][i].x = fmaf(p[u][e], x.x, o[u][i].x);
                            o[u][i].y = fmaf(p[u][e], x.y, o[u][i].y);
                            o[u][i].z = fmaf(p[u][e], x.z, o[u][i].z);
                            o[u][i].w = fmaf(p[u][e], x.w, o[u][i].w);
                        }
                    }
            }
        }
        if (tid == 0) a.W.block_bad[s.block] = bad;
#pragma unroll
        for (int u = 0; u < UV; ++u) {
            const int v = UV * tv + u;
            if (v >= nv) continue;
            if (td == 0) a.W.ml[(size_t)s.block * VT + v] = make_float2(m[u], l[u]);
#pragma unroll
            for (int i = 0; i < DPT; ++i) {
                const int d = 4 * td + 32 * i;
                *reinterpret_cast<float4*>(a.W.o + ((size_t)s.block * (HD / 8) + d / 8) * VT * 8 + v * 8 + d % 8) = o[u][i];
            }
        }
        __syncthreads();  // Q, K, V and P are free for the next segment
    }
    pdl_trigger();
}

template <int HD, int UV>
bool run(const Launch& L, const F32Args& f) {
    const size_t smem = sizeof(Smem<HD, 16 * UV>) + 3 * f.P.batch * 4;
    if (cudaFuncSetAttribute(shared_f32_kernel<HD, UV>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
        return false;
    launch_k(L, shared_f32_kernel<HD, UV>, dim3(2 * f.P.n_cta), dim3(NT), smem, 1, f);
    return true;
}

}  // namespace

bool shared_attention_f32(const Launch& L, const sp::Shape& P, const sp::Work& W, const dflash_shared_prefix_args& a) {
    F32Args f;
    f.P = P;
    f.W = W;
    f.q = (const float*)a.q;
    f.k = (const float*)a.k_cache;
    f.v = (const float*)a.v_cache;
    f.ld_q = a.ld_q;
    f.scale_log2 = (float)((double)a.scale * 1.4426950408889634);
    if (P.VT == 64) return P.hd == 128 ? run<128, 4>(L, f) : run<64, 4>(L, f);
    return P.hd == 128 ? run<128, 2>(L, f) : run<64, 2>(L, f);
}

}  // namespace dfl
