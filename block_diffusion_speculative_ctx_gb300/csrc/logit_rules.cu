// Penalties for repeated tokens, biases and grammar masks on logits
// (dflash_process_logits in include/dflash.h).
//
// Per row this is one read and one write of the logits (HBM bound: 2 * vocab *
// element bytes a row, 622 MB for a 512-row verify pass at the Qwen3 vocabulary);
// the difficulty is that the history is a list of ids while the logits stream by
// vocabulary.  A CTA owns one chunk of the vocabulary for (a group of rows of) one
// sequence.  It first turns the sequence's history and biases into one or two
// words per token of its chunk in shared memory (counts by integer atomics, so the
// order is immaterial): the history is read once per chunk instead of once per
// row, from L2.  Then 16-byte vectors stream by, a row ahead of the stores (copied
// asynchronously into shared memory, each thread its own), with the mask words of
// the row after that under way, so no load waits for another; a vector that its
// mask closes entirely is not read, and a flag byte per vector says whether its
// words are looked up at all.  (Collecting the touched tokens in a list
// for a pass of their own took 147 us where this takes 110 us at 512 rows of 151936: frequent ids sit
// together, so the CTAs of the first chunk had nearly all of that pass to do.)
// Drafts stay a list of at most 31 ids: a token that is a draft carries a bit, and
// only such tokens count the drafts before their row.
// Measured (graph replay): 107 us for 512 rows of 151936 in fp32 (5.8 TB/s of the bytes above, 86 % of a measured copy;
// 122 us for rows of 151937, 261 us token by token); 18 us for 64 bf16 rows of 128256 and 9.6 us for 16 rows of one
// sequence behind up to 8448 tokens, where the lists' chain of loads counts; 3.5 us for a single row.
#include <math.h>

#include <algorithm>

#include "ops.h"

namespace dfl {

namespace {

constexpr int NT = 256, DEPTH = 2;
constexpr uint32_t IN_PROMPT = 0x80000000u, IS_DRAFT = 0x40000000u, COUNT = 0x3FFFFFFFu;

// A sequence's penalties; x / repetition is x times the rounded reciprocal (one rounding more, and the reciprocal has to be
// a normal number).  By an fp32 division a token 64 bf16 rows of 128256 take 22.1 us (so 18.1) and 512 rows of 151936 112 (so
// 106); the product corrected by its remainder, twice, 19.2 and 110; with a power of two for any penalty 18.7 and 108.5.
struct Rules {
    float rep, inv, pres, freq;
    const float* bias;  // the sequence's bias_values
    const int* draft;   // [31] tokens of the chunk, -1: none there
};
// The rule of token t (word w, bias entry b - 1) in the j-th row of the sequence.
__device__ __forceinline__ float apply(float x, uint32_t w, int b, int t, int j, const Rules& r) {
    uint32_t c = w & COUNT;
    if (w & IS_DRAFT)
#pragma unroll 1
        for (int i = 0; i < j; ++i) c += r.draft[i] == t;
    if (c || (w & IN_PROMPT)) x *= x > 0.f ? r.inv : r.rep;
    if (c) x = x - r.freq * (float)c - r.pres;
    if (b) x += r.bias[b - 1];
    return x;
}

__device__ __forceinline__ void cp16(void* dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src) : "memory");
}

struct Plan {
    int chunk;   // tokens per CTA
    int rows;    // rows per CTA
    int groups;  // row groups per sequence
};

// How rows lie: every row starts on 16 bytes; a row starts anywhere, in logits and out alike (its vectors begin with
// its first aligned token, the few before and behind them go one by one); logits and out lie differently (single
// tokens throughout).
enum Lie { ALIGNED, SHIFTED, SINGLE };

// T logits; NV vectors per thread and row (chunk = NT * NV * 16 / sizeof(T) tokens).
template <typename T, int NV, Lie LIE>
__global__ void __launch_bounds__(NT) logit_rules_kernel(dflash_logits_args a, Plan pl) {
    constexpr int G = 16 / (int)sizeof(T);  // tokens of a vector
    constexpr int CH = NT * NV * G;
    __shared__ __align__(16) uint32_t count[CH];       // occurrences after the prompt | IN_PROMPT | IS_DRAFT
    __shared__ __align__(16) uint32_t flag4[CH / G / 4];  // a byte per vector: a rule touches it
    __shared__ int draft[32], midx[32];
    extern __shared__ __align__(16) int bias[];        // [CH] 1 + last bias entry of the token, 0: none (bias_ids given)
    uint8_t* flag = reinterpret_cast<uint8_t*>(flag4);
    const int tid = threadIdx.x;
    const int c0 = blockIdx.x * CH, s = blockIdx.y / pl.groups, j0 = (blockIdx.y - s * pl.groups) * pl.rows;
    const int rows = min(pl.rows, a.rows_per_seq - j0);
    const long long row0 = (long long)s * a.rows_per_seq + j0;
    const int n = min(CH, a.vocab - c0);
    const bool inplace = a.out == a.logits, rules = a.history || a.bias_ids;
    const T* X = reinterpret_cast<const T*>(a.logits) + row0 * a.ld_logits + c0;
    T* Y = reinterpret_cast<T*>(a.out) + row0 * a.ld_out + c0;
    pdl_wait();
    pdl_trigger();

    // ---- the first row's mask words and vectors, under way while the words are made
    constexpr uint32_t ALL = (1u << G) - 1u;
    // tokens of row j before its first vector, and its vectors
    const int mis0 = (int)((uintptr_t)X / sizeof(T)) & (G - 1), mis_ld = (int)a.ld_logits & (G - 1);
    auto head = [&](int j) { return LIE == SHIFTED ? -(mis0 + j * mis_ld) & (G - 1) : 0; };
    auto vecs = [&](int j) { return LIE == SINGLE ? 0 : max(n - head(j), 0) / G; };
    // Rows on their way: each thread's vectors of DEPTH rows in shared memory, its own alone (no barrier).  512 rows of
    // 151936: 107 us with two rows, 112 with four, 166 with eight (fewer CTAs an SM); 112 with the row ahead in registers.
    uint4* ring = reinterpret_cast<uint4*>(bias + (a.bias_ids ? CH : 0)) + tid;
    uint32_t bits[DEPTH - 1][NV], next[NV];  // mask bits of the rows on their way, and of the row after them
    auto mask_bits = [&](int j, int m, uint32_t (&b)[NV]) {
        const int h = head(j);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int t = h + (tid + i * NT) * G;
            b[i] = ALL;
            if (m >= 0 && t < n) {
                const uint32_t* w = a.masks + (long long)m * a.ld_mask + ((c0 + t) >> 5);
                b[i] = w[0] >> (t & 31);
                if (LIE == SHIFTED && (t & 31) > 32 - G && ((c0 + t) | 31) + 1 < a.vocab) b[i] |= w[1] << (32 - (t & 31));
                b[i] &= ALL;
            }
        }
    };
    auto load_mask = [&](int j, uint32_t (&b)[NV]) { mask_bits(j, j < rows ? midx[j] : -1, b); };
    // (a shifted vector lies in two groups of G tokens)
    auto touched_vec = [&](int v, int h) { return flag[v] || (h && flag[v + 1]); };
    // in place, only vectors that a rule or the mask changes are touched
    auto live = [&](int i, uint32_t b, int j) {
        const int v = tid + i * NT;
        return v < vecs(j) && (!inplace || b != ALL || touched_vec(v, head(j)));
    };
    auto load = [&](int j, const uint32_t (&b)[NV]) {
        if (j < rows)
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (live(i, b[i], j) && b[i])
                    cp16(ring + ((j & (DEPTH - 1)) * NV + i) * NT, X + j * a.ld_logits + head(j) + (tid + i * NT) * G);
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    if (LIE != SINGLE) {
#pragma unroll
        for (int r = 0; r < DEPTH - 1; ++r) {
            const int m = a.masks && r < rows ? a.mask_index[row0 + r] : -1;
            mask_bits(r, m < a.n_masks ? m : -1, bits[r]);
        }
        if (!inplace)
#pragma unroll
            for (int r = 0; r < DEPTH - 1; ++r) load(r, bits[r]);
    }

    // ---- the chunk's words: the first reads of the lists go out before the barrier
    int len = 0, prompt = 0, lead = 0, quads = 0, bias_id = -1;
    const int* h = nullptr;
    int4 first = make_int4(-1, -1, -1, -1);
    if (a.history) {
        len = min(max(a.hist_lens[s], 0), a.hist_width);
        prompt = min(max(a.prompt_lens[s], 0), len);
        h = a.history + (long long)s * a.ld_hist;
        lead = min(len, (int)((16 - ((uintptr_t)h & 15)) & 15) / 4);
        quads = (len - lead) / 4;
        if (tid < quads) first = *reinterpret_cast<const int4*>(h + lead + 4 * tid);
    }
    if (a.bias_ids && tid < a.bias_width) bias_id = a.bias_ids[(long long)s * a.bias_width + tid];
    if (tid < rows) {
        const int m = a.masks ? a.mask_index[row0 + tid] : -1;
        midx[tid] = m < a.n_masks ? m : -1;
    }
    if (rules) {
        uint4* z = reinterpret_cast<uint4*>(count);
#pragma unroll
        for (int i = 0; i < CH / 4 / NT; ++i) z[tid + i * NT] = make_uint4(0u, 0u, 0u, 0u);
        if (a.bias_ids) {
            z = reinterpret_cast<uint4*>(bias);
#pragma unroll
            for (int i = 0; i < CH / 4 / NT; ++i) z[tid + i * NT] = make_uint4(0u, 0u, 0u, 0u);
        }
    }
    for (int i = tid; i < CH / G / 4; i += NT) flag4[i] = 0u;
    __syncthreads();
    Rules rule = {1.f, 1.f, 0.f, 0.f, a.bias_values + (long long)s * a.bias_width, draft};
    if (a.history) {
        if (a.repetition) rule.rep = a.repetition[s];
        if (a.presence) rule.pres = a.presence[s];
        if (a.frequency) rule.freq = a.frequency[s];
        rule.inv = 1.f / rule.rep;
        auto mark = [&](int id, int i) {
            const unsigned t = (unsigned)id - (unsigned)c0;
            if (id >= 0 && t < (unsigned)n) {
                if (i < prompt) atomicOr(&count[t], IN_PROMPT);
                else atomicAdd(&count[t], 1u);
                flag[t / G] = 1;
            }
        };
        if (tid < lead) mark(h[tid], tid);
#pragma unroll 1
        for (int q = tid; q < quads; q += NT) {
            const int4 v = first;
            if (q + NT < quads) first = *reinterpret_cast<const int4*>(h + lead + 4 * (q + NT));
            const int i = lead + 4 * q;
            mark(v.x, i);
            mark(v.y, i + 1);
            mark(v.z, i + 2);
            mark(v.w, i + 3);
        }
        const int rest = lead + 4 * quads + tid;
        if (rest < len) mark(h[rest], rest);
        if (tid < 32) {
            int t = -1;
            if (a.drafts && tid < a.rows_per_seq - 1) {
                const int id = a.drafts[(long long)s * (a.rows_per_seq - 1) + tid];
                if (id >= c0 && id - c0 < n) {
                    t = id - c0;
                    atomicOr(&count[t], IS_DRAFT);
                    flag[t / G] = 1;
                }
            }
            draft[tid] = t;
        }
    }
    if (a.bias_ids)
        for (int i = tid; i < a.bias_width; i += NT) {
            const int id = i == tid ? bias_id : a.bias_ids[(long long)s * a.bias_width + i];
            if (id >= c0 && id - c0 < n) {
                atomicMax(&bias[id - c0], i + 1);
                flag[(id - c0) / G] = 1;
            }
        }
    __syncthreads();

    // ---- the stream
    if (LIE != SINGLE) {
        load_mask(DEPTH - 1, next);
        if (inplace)  // (which vectors change is known only now)
#pragma unroll
            for (int r = 0; r < DEPTH - 1; ++r) load(r, bits[r]);
#pragma unroll 1
        for (int j = 0; j < rows; ++j) {
            load(j + DEPTH - 1, next);
            uint32_t b[NV];
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                b[i] = bits[0][i];
#pragma unroll
                for (int r = 0; r < DEPTH - 2; ++r) bits[r][i] = bits[r + 1][i];
                bits[DEPTH - 2][i] = next[i];
            }
            load_mask(j + DEPTH, next);
            asm volatile("cp.async.wait_group %0;" ::"n"(DEPTH - 1) : "memory");
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (live(i, b[i], j)) {
                    const int h = head(j);
                    const uint4 y = ring[((j & (DEPTH - 1)) * NV + i) * NT];
                    uint32_t w[4] = {y.x, y.y, y.z, y.w};
                    const int v = tid + i * NT;
                    if (b[i] && touched_vec(v, h)) {
#pragma unroll
                        for (int q = 0; q < G / 4; ++q) {  // four tokens at a time
                            const int t = h + v * G + 4 * q;
                            alignas(16) uint32_t c4[4];
                            alignas(16) int b4[4] = {0, 0, 0, 0};
                            if (LIE == ALIGNED) {
                                *reinterpret_cast<uint4*>(c4) = *reinterpret_cast<const uint4*>(count + t);
                                if (a.bias_ids) *reinterpret_cast<int4*>(b4) = *reinterpret_cast<const int4*>(bias + t);
                            } else {
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    c4[e] = count[t + e];
                                    if (a.bias_ids) b4[e] = bias[t + e];
                                }
                            }
                            float l[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                if (sizeof(T) == 4) l[e] = __uint_as_float(w[e]);
                                else l[e] = __uint_as_float(e & 1 ? w[2 * q + e / 2] & 0xFFFF0000u : w[2 * q + e / 2] << 16);
                                l[e] = apply(l[e], c4[e], b4[e], t + e, j0 + j, rule);
                            }
                            if (sizeof(T) == 4) {
#pragma unroll
                                for (int e = 0; e < 4; ++e) w[e] = __float_as_uint(l[e]);
                            } else {
                                const __nv_bfloat162 p0 = __floats2bfloat162_rn(l[0], l[1]), p1 = __floats2bfloat162_rn(l[2], l[3]);
                                w[(2 * q) & 3] = *reinterpret_cast<const uint32_t*>(&p0);
                                w[(2 * q + 1) & 3] = *reinterpret_cast<const uint32_t*>(&p1);
                            }
                        }
                    }
                    if (b[i] != ALL) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            if (sizeof(T) == 4) {
                                if (!(b[i] >> e & 1u)) w[e] = 0xFF800000u;
                            } else {
                                if (!(b[i] >> (2 * e) & 1u)) w[e] = (w[e] & 0xFFFF0000u) | 0xFF80u;
                                if (!(b[i] >> (2 * e + 1) & 1u)) w[e] = (w[e] & 0xFFFFu) | 0xFF800000u;
                            }
                        }
                    }
                    *reinterpret_cast<uint4*>(Y + j * a.ld_out + h + (tid + i * NT) * G) = make_uint4(w[0], w[1], w[2], w[3]);
                }
        }
    }

    // ---- single tokens: those of a row before its first vector and behind its last (SINGLE: all)
    const int slots = LIE == ALIGNED ? n % G : LIE == SHIFTED ? 2 * G : n, left = slots * rows;
#pragma unroll (LIE == SINGLE ? 4 : 1)
    for (int i = tid; i < left; i += NT) {
        const int j = i / slots, k = i - j * slots, h = head(j);
        const int t = k < h ? k : k + vecs(j) * G;
        if (t >= n) continue;
        const int m = midx[j];
        const bool on = m < 0 || (a.masks[(long long)m * a.ld_mask + ((c0 + t) >> 5)] >> ((c0 + t) & 31) & 1u);
        const bool touched = rules && flag[t / G];
        if (inplace && on && !touched) continue;
        float l = -INFINITY;
        if (on) {
            l = to_f32(X[j * a.ld_logits + t]);
            if (touched) l = apply(l, count[t], a.bias_ids ? bias[t] : 0, t, j0 + j, rule);
        }
        Y[j * a.ld_out + t] = from_f32<T>(l);
    }
}

template <typename T, int NV>
void run(const Launch& L, const dflash_logits_args& a) {
    Plan pl;
    pl.chunk = NT * NV * 16 / (int)sizeof(T);
    const int chunks = (a.vocab + pl.chunk - 1) / pl.chunk;
    // few CTAs (short batch): the rows of a sequence go to several, each of which reads the history again; 608 CTAs, four
    // an SM (16 rows of 151936 behind up to 8448 tokens: 11.3 us with 304, 10.3 with 608, 11.5 with 1216, one vector a thread)
    pl.groups = (int)std::min<long long>(a.rows_per_seq, std::max(1ll, 608ll / ((long long)chunks * a.batch)));
    pl.rows = (a.rows_per_seq + pl.groups - 1) / pl.groups;
    pl.groups = (a.rows_per_seq + pl.rows - 1) / pl.rows;
    const long long g = 16 / (int)sizeof(T);
    const bool base = ((uintptr_t)a.logits - (uintptr_t)a.out) % 16 == 0 && (a.ld_logits - a.ld_out) % g == 0;
    const Lie lie = base && (uintptr_t)a.logits % 16 == 0 && a.ld_logits % g == 0 ? ALIGNED : base ? SHIFTED : SINGLE;
    const size_t smem = (a.bias_ids ? (size_t)pl.chunk * 4 : 0) +
                        (lie == SINGLE ? 0 : (size_t)std::min(pl.rows, DEPTH) * NV * NT * 16);
    auto* k = lie == ALIGNED   ? logit_rules_kernel<T, NV, ALIGNED>
              : lie == SHIFTED ? logit_rules_kernel<T, NV, SHIFTED>
                               : logit_rules_kernel<T, NV, SINGLE>;
    // (static shared memory: at most 17.2 KB of the 48 that need no leave)
    if (smem > 30u << 10 && cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess) {
        L.fail();
        return;
    }
    launch_k(L, k, dim3(chunks, (unsigned)(a.batch * pl.groups)), dim3(NT), smem, 1, a, pl);
}

// Vectors per thread: two (with a row ahead in registers, 512 rows of 151936 took 111 us, with one vector 123; 64 bf16
// rows of 128256 20 and 23 us), unless the rows, split one a CTA, would leave fewer than two CTAs an SM (one row of
// 151936: 3.6 us with two, 3.4 with one).
template <typename T>
void run(const Launch& L, const dflash_logits_args& a) {
    const int chunk2 = NT * 2 * 16 / (int)sizeof(T);
    if ((long long)a.batch * a.rows_per_seq * ((a.vocab + chunk2 - 1) / chunk2) >= 304) run<T, 2>(L, a);
    else run<T, 1>(L, a);
}

}  // namespace

void process_logits(const Launch& L, const dflash_logits_args& a) {
    if (a.dtype == DFLASH_DTYPE_BF16) run<bf16>(L, a);
    else run<float>(L, a);
}

dflash_status check_logits(const dflash_logits_args& a, const char** why) {
    auto bad = [&](const char* m) {
        *why = m;
        return DFLASH_E_INVAL;
    };
    if (a.dtype != DFLASH_DTYPE_F32 && a.dtype != DFLASH_DTYPE_BF16) return bad("process_logits: dtype must be F32 or BF16");
    if (a.batch < 1 || a.batch > DFLASH_OPS_MAX_BATCH) return bad("process_logits: batch outside [1, 2048]");
    if (a.rows_per_seq < 1 || a.rows_per_seq > 32) return bad("process_logits: rows_per_seq outside [1, 32]");
    if (a.vocab < 1 || a.vocab > (1 << 30)) return bad("process_logits: vocab outside [1, 2^30]");
    if (!a.logits || !a.out) return bad("process_logits: logits or out is NULL");
    const uintptr_t esz = a.dtype == DFLASH_DTYPE_BF16 ? 2 : 4;
    if (((uintptr_t)a.logits | (uintptr_t)a.out) % esz) return bad("process_logits: logits or out is not aligned to its type");
    if (a.ld_logits < a.vocab || a.ld_out < a.vocab) return bad("process_logits: a row stride is smaller than vocab");
    if (a.out == a.logits && a.ld_out != a.ld_logits) return bad("process_logits: in place needs one row stride");
    if (a.history && (!a.hist_lens || !a.prompt_lens || a.hist_width < 0 || a.ld_hist < a.hist_width))
        return bad("process_logits: history needs hist_lens, prompt_lens and a row stride of at least hist_width");
    if (a.hist_width > (1 << 29) || a.bias_width > (1 << 29))
        return bad("process_logits: hist_width or bias_width above 2^29");
    if (!a.history && (a.drafts || a.repetition || a.presence || a.frequency))
        return bad("process_logits: penalties and drafts need a history");
    if (a.bias_ids && (!a.bias_values || a.bias_width < 0)) return bad("process_logits: bias_ids needs bias_values");
    if (a.masks && (!a.mask_index || a.n_masks < 0 || a.ld_mask < (a.vocab + 31) / 32))
        return bad("process_logits: masks need mask_index and at least ceil(vocab / 32) words a mask");
    return DFLASH_OK;
}

}  // namespace dfl

using namespace dfl;

extern "C" dflash_status dflash_process_logits(const dflash_logits_args* p, void* cuda_stream) {
    const char* why = "process_logits: args is NULL";
    if (!p || check_logits(*p, &why) != DFLASH_OK) {
        set_global_error(why);
        return DFLASH_E_INVAL;
    }
    bool failed = false;
    Launch L{(cudaStream_t)cuda_stream, nullptr};
    L.pdl = true;  // (each kernel waits for what runs before it ahead of its first read)
    L.failed = &failed;
    process_logits(L, *p);
    const cudaError_t e = cudaGetLastError();
    if (failed || e != cudaSuccess) {
        set_global_error(e != cudaSuccess ? cudaGetErrorString(e) : "process_logits: launch failed");
        return DFLASH_E_CUDA;
    }
    return DFLASH_OK;
}
