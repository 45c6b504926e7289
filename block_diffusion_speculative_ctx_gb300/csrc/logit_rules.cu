// Penalties for repeated tokens, biases and grammar masks on logits
// (dflash_process_logits in include/dflash.h).
//
// Per row this is one read and one write of the logits (HBM bound: 2 * vocab *
// element bytes a row, 622 MB for a 512-row verify pass at the Qwen3 vocabulary);
// the difficulty is that the history is a list of ids while the logits stream by
// vocabulary.  A CTA owns one chunk of the vocabulary for one sequence: it first
// turns the sequence's history, drafts and biases into per-token words for its
// chunk in shared memory (counts by integer atomics, so the order is immaterial),
// then streams its chunk of every row of the sequence.  The history is read once
// per (sequence, chunk) instead of once per row, from L2.  Drafts are kept as one
// bit per draft position and token, so that row j counts the drafts before it
// (popc of the bits below j) without a barrier between rows.  A flag byte per
// group of four tokens says whether any rule but a mask touches the group: nearly
// all groups take the short path (mask only).
#include <math.h>

#include "ops.h"

namespace dfl {

namespace {

constexpr int NT = 256;
constexpr uint32_t IN_PROMPT = 0x80000000u;

template <typename T>
struct Vec4;
template <>
struct Vec4<float> {
    float4 v;
    __device__ __forceinline__ void get(float (&x)[4]) const { x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w; }
    __device__ __forceinline__ void set(const float (&x)[4]) { v = make_float4(x[0], x[1], x[2], x[3]); }
};
template <>
struct Vec4<bf16> {
    uint2 v;
    __device__ __forceinline__ void get(float (&x)[4]) const {
        x[0] = __uint_as_float(v.x << 16);
        x[1] = __uint_as_float(v.x & 0xFFFF0000u);
        x[2] = __uint_as_float(v.y << 16);
        x[3] = __uint_as_float(v.y & 0xFFFF0000u);
    }
    __device__ __forceinline__ void set(const float (&x)[4]) {
        const __nv_bfloat162 a = __floats2bfloat162_rn(x[0], x[1]), b = __floats2bfloat162_rn(x[2], x[3]);
        v = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
    }
};

struct Rules {
    float rep, pres, freq;
};

// One token's rule: `word` its count after the prompt with IN_PROMPT, `extra` the drafts of it
// before this row.
__device__ __forceinline__ float apply(float x, uint32_t word, int extra, const Rules& r) {
    const uint32_t count = (word & ~IN_PROMPT) + (uint32_t)extra;
    if (count || (word & IN_PROMPT)) x = x > 0.f ? x / r.rep : x * r.rep;
    x -= r.freq * (float)count;
    if (count) x -= r.pres;
    return x;
}

// VEC: base pointers and row strides allow 4-token vectors.
template <typename T, bool VEC>
__global__ void __launch_bounds__(NT) logit_rules_kernel(dflash_logits_args a, int chunk) {
    pdl_wait();
    pdl_trigger();
    extern __shared__ uint32_t sm[];
    uint32_t* count = sm;                    // [chunk] occurrences after the prompt | IN_PROMPT
    uint32_t* draft = count + chunk;         // [chunk] bit i: draft i is this token
    int* bias = (int*)(draft + chunk);       // [chunk] 1 + last bias entry of this token (0: none)
    uint32_t* flag32 = (uint32_t*)(bias + chunk);
    uint8_t* flag = (uint8_t*)flag32;        // [chunk / 4]: a rule touches one of the four tokens
    const int tid = threadIdx.x;
    const int c0 = blockIdx.x * chunk, s = blockIdx.y;
    const int n = min(chunk, a.vocab - c0);
    const bool inplace = a.out == a.logits;

    for (int i = tid; i < 3 * chunk + chunk / 16; i += NT) sm[i] = 0u;
    __syncthreads();
    Rules rule{1.f, 0.f, 0.f};
    if (a.history) {
        if (a.repetition) rule.rep = a.repetition[s];
        if (a.presence) rule.pres = a.presence[s];
        if (a.frequency) rule.freq = a.frequency[s];
        const int len = min(max(a.hist_lens[s], 0), a.hist_width);
        const int prompt = min(max(a.prompt_lens[s], 0), len);
        const int* h = a.history + (long long)s * a.ld_hist;
        for (int i = tid; i < len; i += NT) {
            const unsigned t = (unsigned)(h[i] - c0);
            if (h[i] >= 0 && t < (unsigned)n) {
                if (i < prompt) atomicOr(&count[t], IN_PROMPT);
                else atomicAdd(&count[t], 1u);
                flag[t >> 2] = 1;
            }
        }
        if (a.drafts && tid < a.rows_per_seq - 1) {
            const int id = a.drafts[(long long)s * (a.rows_per_seq - 1) + tid];
            const unsigned t = (unsigned)(id - c0);
            if (id >= 0 && t < (unsigned)n) {
                atomicOr(&draft[t], 1u << tid);
                flag[t >> 2] = 1;
            }
        }
    }
    if (a.bias_ids) {
        for (int i = tid; i < a.bias_width; i += NT) {
            const int id = a.bias_ids[(long long)s * a.bias_width + i];
            const unsigned t = (unsigned)(id - c0);
            if (id >= 0 && t < (unsigned)n) {
                atomicMax(&bias[t], i + 1);
                flag[t >> 2] = 1;
            }
        }
    }
    __syncthreads();

    const float* bv = a.bias_values + (long long)s * a.bias_width;
    for (int j = 0; j < a.rows_per_seq; ++j) {
        const long long row = (long long)s * a.rows_per_seq + j;
        const T* x = reinterpret_cast<const T*>(a.logits) + row * a.ld_logits + c0;
        T* y = reinterpret_cast<T*>(a.out) + row * a.ld_out + c0;
        const uint32_t* mask = nullptr;
        if (a.masks) {
            const int m = a.mask_index[row];
            if (m >= 0 && m < a.n_masks) mask = a.masks + (long long)m * a.ld_mask + (c0 >> 5);
        }
        const uint32_t before = (1u << j) - 1u;  // drafts 0 .. j-1
        if (VEC) {
#pragma unroll 4
            for (int g = tid; g < n / 4; g += NT) {
                const int t = 4 * g;
                const uint32_t bits = mask ? (mask[t >> 5] >> (t & 31)) & 15u : 15u;
                const bool touched = flag[g] != 0;
                if (inplace && !touched && bits == 15u) continue;
                float v[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                Vec4<T> io;
                if (bits) {
                    io = *reinterpret_cast<const Vec4<T>*>(x + t);
                    if (bits != 15u || touched) {
                        float l[4];
                        io.get(l);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            if (touched) {
                                l[e] = apply(l[e], count[t + e], __popc(draft[t + e] & before), rule);
                                if (bias[t + e]) l[e] += bv[bias[t + e] - 1];
                            }
                            if ((bits >> e) & 1u) v[e] = l[e];
                        }
                        io.set(v);
                    }
                } else {
                    io.set(v);
                }
                *reinterpret_cast<Vec4<T>*>(y + t) = io;
            }
        }
        // scalar: rows that are not aligned, and the last vocab % 4 tokens
        for (int t = (VEC ? (n & ~3) : 0) + tid; t < n; t += NT) {
            const bool on = mask ? (mask[t >> 5] >> (t & 31)) & 1u : true;
            const bool touched = flag[t >> 2] != 0;
            if (inplace && !touched && on) continue;
            float l = -INFINITY;
            if (on) {
                l = to_f32(x[t]);
                if (touched) {
                    l = apply(l, count[t], __popc(draft[t] & before), rule);
                    if (bias[t]) l += bv[bias[t] - 1];
                }
            }
            y[t] = from_f32<T>(l);
        }
    }
}

template <typename T>
void run(const Launch& L, const dflash_logits_args& a) {
    // chunk: the largest of 4096 .. 1024 tokens that still gives about two CTAs an SM
    int chunk = 4096;
    while (chunk > 1024 && (long long)a.batch * ((a.vocab + chunk - 1) / chunk) < 2 * 152) chunk /= 2;
    const size_t smem = (size_t)chunk * 12 + chunk / 4;
    const size_t al = 4 * sizeof(T);
    const bool vec = (((uintptr_t)a.logits | (uintptr_t)a.out) % al) == 0 && a.ld_logits % 4 == 0 && a.ld_out % 4 == 0;
    const dim3 grid((a.vocab + chunk - 1) / chunk, a.batch);
    auto k = vec ? logit_rules_kernel<T, true> : logit_rules_kernel<T, false>;
    if (smem > 48 * 1024 &&
        cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
        L.fail();
    launch_k(L, k, grid, dim3(NT), smem, 1, a, chunk);
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
