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
// row, from L2.  Then
//   - the stream: 16-byte vectors without a touched token are copied under the
//     row's mask, a row ahead of the stores; the mask words of the row after that
//     are under way, so no load waits for another.  A vector that its mask closes
//     entirely is not read;
//   - the touched vectors, collected in a list, a thread per token: they are few,
//     but sit together (frequent ids), so spreading them over the CTA keeps one
//     warp from doing them all, and the rule's code exists once.
// Drafts stay a list of at most 31 ids: a token that is a draft carries a bit, and
// only such tokens count the drafts before their row.
#include <math.h>

#include <algorithm>

#include "ops.h"

namespace dfl {

namespace {

constexpr int NT = 256;
constexpr uint32_t IN_PROMPT = 0x80000000u, IS_DRAFT = 0x40000000u, COUNT = 0x3FFFFFFFu;

struct Plan {
    int chunk;   // tokens per CTA
    int rows;    // rows per CTA
    int groups;  // row groups per sequence
};

// T logits; NV vectors per thread and row (chunk = NT * NV * 16 / sizeof(T) tokens); VEC: base pointers and
// row strides are multiples of 16 bytes (else the stream moves single elements).
template <typename T, int NV, bool VEC>
__global__ void __launch_bounds__(NT) logit_rules_kernel(dflash_logits_args a, Plan pl) {
    constexpr int G = 16 / (int)sizeof(T);  // tokens of a vector
    constexpr int CH = NT * NV * G;
    __shared__ __align__(16) uint32_t count[CH];       // occurrences after the prompt | IN_PROMPT | IS_DRAFT
    __shared__ __align__(16) uint32_t flag4[CH / G / 4];  // a byte per vector: a rule touches it
    __shared__ uint16_t list[CH / G];                  // the touched vectors
    __shared__ int n_list, draft[32], midx[32];
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

    // ---- the chunk's words
    if (tid < rows) {
        const int m = a.masks ? a.mask_index[row0 + tid] : -1;
        midx[tid] = m < a.n_masks ? m : -1;
    }
    if (tid == 0) n_list = 0;
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
    float rep = 1.f, pres = 0.f, freq = 0.f;
    if (a.history) {
        if (a.repetition) rep = a.repetition[s];
        if (a.presence) pres = a.presence[s];
        if (a.frequency) freq = a.frequency[s];
        const int len = min(max(a.hist_lens[s], 0), a.hist_width);
        const int prompt = min(max(a.prompt_lens[s], 0), len);
        const int* h = a.history + (long long)s * a.ld_hist;
        auto mark = [&](int id, int i) {
            const unsigned t = (unsigned)id - (unsigned)c0;
            if (id >= 0 && t < (unsigned)n) {
                if (i < prompt) atomicOr(&count[t], IN_PROMPT);
                else atomicAdd(&count[t], 1u);
                flag[t / G] = 1;
            }
        };
        const int lead = min(len, (int)((16 - ((uintptr_t)h & 15)) & 15) / 4), quads = (len - lead) / 4;
        if (tid < lead) mark(h[tid], tid);
#pragma unroll 2
        for (int q = tid; q < quads; q += NT) {
            const int4 v = *reinterpret_cast<const int4*>(h + lead + 4 * q);
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
            const int id = a.bias_ids[(long long)s * a.bias_width + i];
            if (id >= c0 && id - c0 < n) {
                atomicMax(&bias[id - c0], i + 1);
                flag[(id - c0) / G] = 1;
            }
        }
    __syncthreads();
    if (rules) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (flag[tid + i * NT]) list[atomicAdd(&n_list, 1)] = (uint16_t)(tid + i * NT);
        __syncthreads();
    }

    // ---- the stream: vectors without a touched token
    const int nvec = VEC ? n / G : 0;
    if (VEC) {
        constexpr uint32_t ALL = (1u << G) - 1u;
        auto mask_of = [&](int j) -> const uint32_t* {
            return j < rows && midx[j] >= 0 ? a.masks + (long long)midx[j] * a.ld_mask + (c0 >> 5) : nullptr;
        };
        uint32_t bits[NV], next[NV];  // mask bits of the row whose logits are loaded next, and of the row after
        uint4 x[NV];
        auto load_mask = [&](int j, uint32_t (&b)[NV]) {
            const uint32_t* m = mask_of(j);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int t = (tid + i * NT) * G;
                b[i] = m && t < n ? m[t >> 5] >> (t & 31) & ALL : ALL;
            }
        };
        // in place, only vectors that the mask changes are touched
        auto live = [&](int i, uint32_t b) {
            const int v = tid + i * NT;
            return v < nvec && !flag[v] && !(inplace && b == ALL);
        };
        auto load = [&](int j, const uint32_t (&b)[NV]) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (live(i, b[i]) && b[i]) x[i] = *reinterpret_cast<const uint4*>(X + j * a.ld_logits + (tid + i * NT) * G);
        };
        load_mask(0, bits);
        load_mask(1, next);
        load(0, bits);
#pragma unroll 1
        for (int j = 0; j < rows; ++j) {
            uint4 y[NV];
            uint32_t b[NV];
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                y[i] = x[i];
                b[i] = bits[i];
                bits[i] = next[i];
            }
            load_mask(j + 2, next);
            if (j + 1 < rows) load(j + 1, bits);
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (live(i, b[i])) {
                    uint32_t w[4] = {y[i].x, y[i].y, y[i].z, y[i].w};
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
                    *reinterpret_cast<uint4*>(Y + j * a.ld_out + (tid + i * NT) * G) = make_uint4(w[0], w[1], w[2], w[3]);
                }
        }
    }

    // ---- single tokens: the touched vectors, and what the stream's vectors do not cover (the last vocab % G
    // tokens, or everything when rows are not aligned)
    const float* bv = a.bias_values + (long long)s * a.bias_width;
    auto token = [&](int j, int t, bool touched) {
        const int m = midx[j];
        const bool on = m < 0 || (a.masks[(long long)m * a.ld_mask + ((c0 + t) >> 5)] >> ((c0 + t) & 31) & 1u);
        if (inplace && on && !touched) return;
        float l = -INFINITY;
        if (on) {
            l = to_f32(X[j * a.ld_logits + t]);
            if (touched) {
                const uint32_t w = count[t];
                uint32_t c = w & COUNT;
                if (w & IS_DRAFT)
#pragma unroll 1
                    for (int i = 0; i < j0 + j; ++i) c += draft[i] == t;
                if (c || (w & IN_PROMPT)) l = l > 0.f ? l / rep : l * rep;
                l -= freq * (float)c;
                if (c) l -= pres;
                if (a.bias_ids && bias[t]) l += bv[bias[t] - 1];
            }
        }
        Y[j * a.ld_out + t] = from_f32<T>(l);
    };
    const int per = rules ? n_list * G : 0, total = per * rows;
#pragma unroll 2
    for (int i = tid; i < total; i += NT) {
        const int j = i / per, k = i - j * per, t = list[k / G] * G + k % G;
        if (t < n) token(j, t, true);
    }
    const int from = nvec * G, left = (n - from) * rows;
#pragma unroll 4
    for (int i = tid; i < left; i += NT) {
        const int j = i / (n - from), t = from + i - j * (n - from);
        if (!(rules && flag[t / G])) token(j, t, false);
    }
}

template <typename T, int NV>
void run(const Launch& L, const dflash_logits_args& a) {
    Plan pl;
    pl.chunk = NT * NV * 16 / (int)sizeof(T);
    const int chunks = (a.vocab + pl.chunk - 1) / pl.chunk;
    // few CTAs (short batch): the rows of a sequence go to several, each of which reads the history again
    pl.groups = (int)std::min<long long>(a.rows_per_seq, std::max(1ll, 608ll / ((long long)chunks * a.batch)));
    pl.rows = (a.rows_per_seq + pl.groups - 1) / pl.groups;
    pl.groups = (a.rows_per_seq + pl.rows - 1) / pl.rows;
    const bool vec = (((uintptr_t)a.logits | (uintptr_t)a.out) % 16) == 0 && a.ld_logits % (16 / (int)sizeof(T)) == 0 &&
                     a.ld_out % (16 / (int)sizeof(T)) == 0;
    const size_t smem = a.bias_ids ? (size_t)pl.chunk * 4 : 0;
    launch_k(L, vec ? logit_rules_kernel<T, NV, true> : logit_rules_kernel<T, NV, false>,
             dim3(chunks, (unsigned)(a.batch * pl.groups)), dim3(NT), smem, 1, a, pl);
}

// Vectors per thread: two, unless that leaves fewer than two CTAs an SM.
template <typename T>
void run(const Launch& L, const dflash_logits_args& a) {
    const int chunk2 = NT * 2 * 16 / (int)sizeof(T);
    if ((long long)a.batch * ((a.vocab + chunk2 - 1) / chunk2) >= 304) run<T, 2>(L, a);
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
    L.failed = &failed;
    process_logits(L, *p);
    const cudaError_t e = cudaGetLastError();
    if (failed || e != cudaSuccess) {
        set_global_error(e != cudaSuccess ? cudaGetErrorString(e) : "process_logits: launch failed");
        return DFLASH_E_CUDA;
    }
    return DFLASH_OK;
}
