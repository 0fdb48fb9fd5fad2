// Gradient of the indexer's scores from the 8-bit codes that the forward kept
// (its activation checkpoints). With G[t,j] the gradient of s[t,j] summed over
// the slots that select block j (0 where nothing does or j is no candidate),
// and m[t,h,j] = 1 where <q8[t,h], k8[j]> > 0 (relu's derivative, exact since
// the products of codes are whole numbers):
//
//   dq[t,h,:] = w[t,h] sum_j m G[t,j] ks[j] k8[j,:]
//   dk[j,:]   = sum_{t,h} m G[t,j] w[t,h] qs[t,h] q8[t,h,:]
//   dw[t,h]   = qs[t,h] sum_j G[t,j] ks[j] relu(<q8[t,h], k8[j]>)
//
// the gradients with respect to the values that the codes stand for. An entry
// with G = 0 contributes nothing, whatever its scale holds.
//
// Three launches: G written out densely, dq and dw by token, dk by block.
#include <cuda_bf16.h>

#include "indexer_q8.h"
#include "sai_device.cuh"

namespace sai {
namespace {

__device__ __forceinline__ bool candidate(const ScoresBwdArgs &a, int64_t row, int t, int j)
{
    const int64_t pos = (int64_t)a.t_begin + t;
    int64_t d0 = a.doc_start ? __ldg(a.doc_start + row) : 0;
    d0 = d0 < 0 ? 0 : (d0 > pos ? pos : d0);
    return (int64_t)(j + 1) * a.cr - 1 <= pos && (int64_t)j * a.cr >= d0;
}

// One block per token. Slots that name the same block are added in slot order
// by the one thread that owns the block, so the sum does not depend on timing.
__global__ void __launch_bounds__(256) bwd_scatter_kernel(const ScoresBwdArgs a, float *G)
{
    const int64_t row = blockIdx.x;
    const int t = (int)(row % a.S);
    float *g = G + row * a.P;
    for (int j = threadIdx.x; j < a.P; j += 256)
        g[j] = a.idx ? 0.f : (candidate(a, row, t, j) ? a.dscores[row * a.P + j] : 0.f);
    if (!a.idx)
        return;
    __syncthreads();
    for (int k = 0; k < a.K; ++k) {
        const int j = __ldg(a.idx + row * a.K + k);
        if (j < -1 || j >= a.P) {
            if (threadIdx.x == 0 && a.err)
                atomicExch(a.err, kErrIndex);
        } else if (j >= 0 && (j & 255) == (int)threadIdx.x && candidate(a, row, t, j)) {
            g[j] += a.dscores[row * a.K + k];
        }
    }
}

__device__ __forceinline__ int dot_codes(const int8_t *x, const int8_t *y, int D)
{
    int dot = 0;
    for (int i = 0; i < D / 16; ++i) {
        const int4 p = reinterpret_cast<const int4 *>(x)[i], q = reinterpret_cast<const int4 *>(y)[i];
        dot = __dp4a(p.x, q.x, dot);
        dot = __dp4a(p.y, q.y, dot);
        dot = __dp4a(p.z, q.z, dot);
        dot = __dp4a(p.w, q.w, dot);
    }
    return dot;
}

// One block per (token, head): thread d owns dq[d]; 128 keys at a time.
__global__ void __launch_bounds__(128) bwd_q_kernel(const ScoresBwdArgs a, const float *G)
{
    __shared__ float m[128];
    __shared__ float part[4];
    const int64_t rh = blockIdx.x;
    const int64_t row = rh / a.H;
    const int b = (int)(row / a.S);
    const int8_t *q = a.q8 + rh * a.D;
    const int8_t *kb = a.k8 + (int64_t)b * a.P * a.D;
    float acc = 0.f, dw = 0.f;
    for (int j0 = 0; j0 < a.P; j0 += 128) {
        const int j = j0 + threadIdx.x;
        float v = 0.f;
        if (j < a.P) {
            const float g = G[row * a.P + j];
            if (g != 0.f) {
                const float gk = g * a.k_scale[(int64_t)b * a.P + j];
                const int dot = dot_codes(q, kb + (int64_t)j * a.D, a.D);
                dw += gk * (float)max(dot, 0);
                v = dot > 0 ? gk : 0.f;
            }
        }
        m[threadIdx.x] = v;
        __syncthreads();
        if ((int)threadIdx.x < a.D)
            for (int i = 0; i < min(128, a.P - j0); ++i)
                if (m[i] != 0.f)
                    acc += m[i] * (float)kb[(int64_t)(j0 + i) * a.D + threadIdx.x];
        __syncthreads();
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1)
        dw += __shfl_xor_sync(0xffffffffu, dw, o);
    if ((threadIdx.x & 31) == 0)
        part[threadIdx.x >> 5] = dw;
    __syncthreads();
    if (threadIdx.x == 0)
        a.dw[rh] = (part[0] + part[1] + part[2] + part[3]) * a.q_scale[rh];
    if ((int)threadIdx.x < a.D)
        reinterpret_cast<__nv_bfloat16 *>(a.dq)[rh * a.D + threadIdx.x] = __float2bfloat16_rn(acc * a.w[rh]);
}

// One block per key: thread d owns dk[d]; 128 (token, head) rows at a time.
__global__ void __launch_bounds__(128) bwd_k_kernel(const ScoresBwdArgs a, const float *G)
{
    __shared__ float m[128];
    const int b = blockIdx.x / a.P;
    const int j = blockIdx.x - b * a.P;
    const int8_t *k = a.k8 + (int64_t)blockIdx.x * a.D;
    const int64_t r0 = (int64_t)b * a.S * a.H;
    float acc = 0.f;
    for (int i0 = 0; i0 < a.S * a.H; i0 += 128) {
        const int i = i0 + threadIdx.x;
        float v = 0.f;
        if (i < a.S * a.H) {
            const float g = G[((int64_t)b * a.S + i / a.H) * a.P + j];
            if (g != 0.f && dot_codes(a.q8 + (r0 + i) * a.D, k, a.D) > 0)
                v = g * (a.w[r0 + i] * a.q_scale[r0 + i]);
        }
        m[threadIdx.x] = v;
        if (!__syncthreads_or(v != 0.f))
            continue;
        if ((int)threadIdx.x < a.D)
            for (int e = 0; e < min(128, a.S * a.H - i0); ++e)
                if (m[e] != 0.f)
                    acc += m[e] * (float)a.q8[(r0 + i0 + e) * a.D + threadIdx.x];
        __syncthreads();
    }
    if ((int)threadIdx.x < a.D)
        reinterpret_cast<__nv_bfloat16 *>(a.dk)[(int64_t)blockIdx.x * a.D + threadIdx.x] = __float2bfloat16_rn(acc);
}

}  // namespace

size_t indexer_scores_bwd_ws_bytes(int B, int S, int H, int D, int P)
{
    (void)H;
    (void)D;
    return (size_t)B * S * P * 4;
}

cudaError_t launch_indexer_scores_bwd(const ScoresBwdArgs &a, void *ws, cudaStream_t stream)
{
    float *G = static_cast<float *>(ws);
    bwd_scatter_kernel<<<a.B * a.S, 256, 0, stream>>>(a, G);
    bwd_q_kernel<<<a.B * a.S * a.H, 128, 0, stream>>>(a, G);
    bwd_k_kernel<<<a.B * a.P, 128, 0, stream>>>(a, G);
    return cudaGetLastError();
}

}  // namespace sai
