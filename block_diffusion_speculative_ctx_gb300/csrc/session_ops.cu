// Small kernels by which the session's passes feed the serving operators: lengths
// behind the shared pages, the token history of the logit rules, the last rows of a
// ragged prefill.  All are latency-bound (a few words a sequence).
#include <math.h>

#include "ops.h"

namespace dfl {

namespace {

__global__ void own_lengths_kernel(int batch, const int* __restrict__ a, const int* __restrict__ b, int add,
                                   int* __restrict__ out, int* __restrict__ start, int block) {
    pdl_wait();
    pdl_trigger();
    for (int s = threadIdx.x; s <= batch; s += blockDim.x) {
        if (s < batch) out[s] = a[s] + (b ? b[s] : 0) + add;
        if (start) start[s] = s * block;
    }
}

__global__ void gather_last_rows_kernel(const float* __restrict__ x, int d, const int* __restrict__ start, int s0,
                                        float* __restrict__ dst) {
    pdl_wait();
    pdl_trigger();
    const float* src = x + (size_t)(start[s0 + blockIdx.x + 1] - 1) * d;
    for (int c = threadIdx.x; c < d; c += blockDim.x) dst[(size_t)blockIdx.x * d + c] = src[c];
}

__global__ void history_append_kernel(int batch, int B, int ld, const int* __restrict__ n, const int* __restrict__ anchor,
                                      const int* __restrict__ accepted, const int* __restrict__ proposal,
                                      int* __restrict__ history) {
    pdl_wait();
    pdl_trigger();
    const int s = blockIdx.x, a = accepted ? accepted[s] : 0, len = n[s];
    int* h = history + (size_t)s * ld;
    if ((int)threadIdx.x < a) h[len - a + threadIdx.x] = proposal[(size_t)s * (B - 1) + threadIdx.x];
    if (threadIdx.x == 0 && len < ld) h[len] = anchor[s];
}

__global__ void drop_indices_kernel(int* __restrict__ index, int rows, int n) {
    pdl_wait();
    pdl_trigger();
    const int r = blockIdx.x * blockDim.x + threadIdx.x;
    if (r < rows && index[r] >= n) index[r] = -1;
}

__global__ void check_rows_kernel(float* __restrict__ logits, long long ld, int rows, const int* __restrict__ best,
                                  uint32_t* __restrict__ err) {
    pdl_wait();
    pdl_trigger();
    const int r = blockIdx.x * blockDim.x + threadIdx.x;
    if (r >= rows || logits[r * ld + best[r]] != -INFINITY) return;
    atomicOr(err, ERR_NO_TOKEN);
    logits[r * ld] = 0.f;
}

}  // namespace

void own_lengths(const Launch& L, int batch, const int* a, const int* b, int add, int* out, int* start, const int* block) {
    launch_k(L, own_lengths_kernel, dim3(1), dim3(256), 0, 1, batch, a, b, add, out, start, block ? *block : 0);
}

void gather_last_rows(const Launch& L, const float* x, int d, const int* start, int s0, int n, float* dst) {
    if (n > 0) launch_k(L, gather_last_rows_kernel, dim3(n), dim3(256), 0, 1, x, d, start, s0, dst);
}

void history_append(const Launch& L, int batch, int B, int ld, const int* n, const int* anchor, const int* accepted,
                    const int* proposal, int* history) {
    launch_k(L, history_append_kernel, dim3(batch), dim3(32), 0, 1, batch, B, ld, n, anchor, accepted, proposal, history);
}

void drop_indices(const Launch& L, int* index, int rows, int n) {
    launch_k(L, drop_indices_kernel, dim3((rows + 127) / 128), dim3(128), 0, 1, index, rows, n);
}

void check_rows(const Launch& L, float* logits, long long ld, int rows, const int* best, uint32_t* err) {
    launch_k(L, check_rows_kernel, dim3((rows + 127) / 128), dim3(128), 0, 1, logits, ld, rows, best, err);
}

}  // namespace dfl
