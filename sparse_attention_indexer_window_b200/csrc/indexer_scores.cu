// The lightning indexer's scores from 8-bit queries and 8-bit cached keys:
//
//   s[b,t,j] = ks[b,j] * sum_h w[b,t,h] qs[b,t,h] relu(<q8[b,t,h,:], k8[b,j,:]>)
//
// for the candidates j of token t, -inf elsewhere. The products of the codes
// are whole numbers below 2^24, so they are exact; the sum over heads is in
// fp32. (Scales are not negative, so they leave relu's argument's sign alone.)
//
// One thread per key, one block per token and 128 keys: the key's codes stay
// in registers, the token's queries are read from shared memory.
#include <math.h>

#include "indexer_q8.h"
#include "sai_device.cuh"

namespace sai {
namespace {

template <int D>
__global__ void __launch_bounds__(128) scores_kernel(const ScoresArgs a)
{
    extern __shared__ int4 sq[];                       // [H][D/16] codes, then [H] weights
    float *sw = reinterpret_cast<float *>(sq + a.H * (D / 16));
    const int64_t row = blockIdx.x;
    const int b = (int)(row / a.S);
    const int t = (int)(row - (int64_t)b * a.S);
    const int j = blockIdx.y * 128 + threadIdx.x;
    const int4 *qg = reinterpret_cast<const int4 *>(a.q8 + row * a.H * D);
    for (int i = threadIdx.x; i < a.H * (D / 16); i += 128)
        sq[i] = __ldg(qg + i);
    for (int h = threadIdx.x; h < a.H; h += 128)
        sw[h] = a.w[row * a.H + h] * a.q_scale[row * a.H + h];
    __syncthreads();
    if (j >= a.P)
        return;
    const int64_t pos = (int64_t)(a.q_start ? __ldg(a.q_start + b) : 0) + t;
    int64_t d0 = a.doc_start ? __ldg(a.doc_start + row) : 0;
    d0 = d0 < 0 ? 0 : (d0 > pos ? pos : d0);
    bool see = (int64_t)(j + 1) * a.cr - 1 <= pos && (int64_t)j * a.cr >= d0 &&
               (!a.k_len || j < __ldg(a.k_len + b));
    float s = -INFINITY;
    if (see) {
        const int64_t kr = page_row(a.map, b, j);
        if (kr >= 0) {
            int4 k[D / 16];
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
                k[i] = __ldg(reinterpret_cast<const int4 *>(a.cache + kr * D) + i);
            float acc = 0.f;
            for (int h = 0; h < a.H; ++h) {
                int dot = 0;
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    const int4 q = sq[h * (D / 16) + i];
                    dot = __dp4a(q.x, k[i].x, dot);
                    dot = __dp4a(q.y, k[i].y, dot);
                    dot = __dp4a(q.z, k[i].z, dot);
                    dot = __dp4a(q.w, k[i].w, dot);
                }
                acc = fmaf(sw[h], (float)max(dot, 0), acc);
            }
            s = acc * __ldg(a.k_scale + kr);
        } else if (a.err) {
            atomicExch(a.err, kErrIndex);
        }
    }
    a.out[row * a.P + j] = s;
}

}  // namespace

cudaError_t launch_indexer_scores(const ScoresArgs &a, cudaStream_t stream)
{
    const dim3 grid((unsigned)(a.B * a.S), (unsigned)((a.P + 127) / 128));
    const size_t smem = (size_t)a.H * a.D + (size_t)a.H * 4;
    if (a.D == 32)
        scores_kernel<32><<<grid, 128, smem, stream>>>(a);
    else if (a.D == 64)
        scores_kernel<64><<<grid, 128, smem, stream>>>(a);
    else
        scores_kernel<128><<<grid, 128, smem, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace sai
