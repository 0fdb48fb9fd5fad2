// Rows quantised to 8 bits as they are written into a (paged) cache, and read
// back. The 8-bit formats are the ones the source pages name for the indexer's
// products (page "Docker Build for DeepSeek-v4": FP8 recipes; here also 8-bit
// integers); the arithmetic is this library's own:
//
//   a group of `group` consecutive values with largest magnitude amax becomes
//     int8:  code = rint(127 x / amax),  scale = amax / 127
//     e4m3:  code = e4m3(448 x / amax),  scale = amax / 448
//   (ties to even; amax = 0: codes 0, scale 0; a NaN or infinity in the group:
//   codes 0, scale NaN), and is read back as code * scale, formed in fp32 and then
//   rounded to the rows' type.
//
// The codes are those of the formula in exact arithmetic. For 16-bit inputs
// one correctly rounded quotient is enough: lim * x is exact in fp32, and a
// quotient of a 15- or 18-bit by an 11-bit integer that is no tie is further
// from any tie than fp32's rounding. For fp32 inputs quotients next to a tie
// are decided again in 64 bits. The quotient comes from the group's correctly
// rounded reciprocal y by Markstein's theorem (IBM J. Res. Dev. 34, 1990): with
// q0 = n y and the exact remainder r = n - d q0, q0 + r y is n / d correctly
// rounded. Three instructions a value; a full division for each value bound
// the kernel (52 us for 8 x 8192 rows of 512 against 15 us of HBM time).
//
// Bound: each value is read and each code written once (15 us of HBM for 8 x 8192
// rows of 512); the write takes 31 us of it, bound by its instructions (issue 0.75 a
// scheduler: about 25 a value), the read 20, bound by its loads' latency; a few
// rows the launch. One group is held by group/8 lanes, 8 values (one or two 16-byte
// loads) each, its maximum found by shuffles, so that a row is read once.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <math.h>
#include <type_traits>

#include "indexer_q8.h"
#include "sai_device.cuh"
#include "sai_host.h"

namespace sai {
namespace {

constexpr int kQ8Threads = 256;

template <class T>
__device__ __forceinline__ float to_f32(T x);
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }
template <>
__device__ __forceinline__ float to_f32<__half>(__half x) { return __half2float(x); }

template <class T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
template <>
__device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }

// Eight values as they lie in memory.
template <class T>
struct Raw {
    uint32_t w[2 * sizeof(T)];
};

// Eight values starting at p: 16-byte loads when the rows allow them (VEC),
// element loads otherwise.
template <class T, bool VEC>
__device__ __forceinline__ Raw<T> load8(const T *p)
{
    Raw<T> r;
    if constexpr (VEC) {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) {
            const uint4 v = __ldg(reinterpret_cast<const uint4 *>(p) + i);
            r.w[4 * i] = v.x;
            r.w[4 * i + 1] = v.y;
            r.w[4 * i + 2] = v.z;
            r.w[4 * i + 3] = v.w;
        }
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            r.w[i] = __float_as_uint(p[i]);
    } else {
        const uint16_t *h = reinterpret_cast<const uint16_t *>(p);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            r.w[i] = (uint32_t)h[2 * i] | ((uint32_t)h[2 * i + 1] << 16);
    }
    return r;
}

template <class T>
__device__ __forceinline__ float value(const Raw<T> &r, int i)
{
    if constexpr (sizeof(T) == 4) {
        return __uint_as_float(r.w[i]);
    } else {
        const uint16_t h = (uint16_t)(r.w[i >> 1] >> (16 * (i & 1)));
        return to_f32<T>(*reinterpret_cast<const T *>(&h));
    }
}

// The largest magnitude of the eight, as the type's bits (ordered as the values
// are, infinities and NaN above every number); and such bits as an fp32 number.
template <class T>
__device__ __forceinline__ uint32_t top_bits(const Raw<T> &r)
{
    if constexpr (sizeof(T) == 4) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            m = max(m, r.w[i] & 0x7fffffffu);
        return m;
    } else {
        constexpr uint32_t abs2 = 0x7fff7fffu;
        const uint32_t m = __vimax3_u16x2(__vimax3_u16x2(r.w[0] & abs2, r.w[1] & abs2, r.w[2] & abs2), r.w[3] & abs2, 0u);
        return max(m & 0xffffu, m >> 16);
    }
}
template <class T>
__device__ __forceinline__ float from_bits(uint32_t b)
{
    if constexpr (sizeof(T) == 4) {
        return __uint_as_float(b);
    } else {
        const uint16_t h = (uint16_t)b;
        return to_f32<T>(*reinterpret_cast<const T *>(&h));
    }
}

template <int CODE>
__device__ __forceinline__ constexpr float code_limit()
{
    return CODE == 0 ? 127.f : 448.f;
}

// fp32 inputs only: v = lim*x/amax in fp32 lies on a tie between two codes, or
// is too near one to tell; decide it in 64 bits and return a value on the
// right side (or on the tie itself, when it is one).
template <int CODE>
__device__ __forceinline__ float settle_tie(float v, float x, float amax)
{
    float tie;
    if (CODE == 0) {
        tie = truncf(v) + copysignf(0.5f, v);
    } else {
        // the e4m3 grid around v: 8 steps per binade, 2^-9 below 2^-6
        int e;
        frexpf(v, &e);                                  // |v| in [2^(e-1), 2^e)
        const float step = ldexpf(1.f, max(e - 1, -6) - 3);
        tie = (truncf(v / step) + copysignf(0.5f, v)) * step;
    }
    if (fabsf(v - tie) > fabsf(tie) * 1e-6f)
        return v;
    const double r = (double)code_limit<CODE>() * (double)x / (double)amax;
    if (r == (double)tie)
        return tie;
    return nextafterf(tie, r > (double)tie ? INFINITY : -INFINITY);
}

// Two codes (low byte first) of two values of a group with maximum d > 0 and
// y = 1 / d, both in the middle of fp32's range.
template <int CODE, bool TIES>
__device__ __forceinline__ uint32_t codes2(float x0, float x1, float d, float y)
{
    constexpr float lim = code_limit<CODE>();
    const float n0 = lim * x0, n1 = lim * x1;
    float v0 = n0 * y, v1 = n1 * y;
    v0 = fmaf(fmaf(-d, v0, n0), y, v0);
    v1 = fmaf(fmaf(-d, v1, n1), y, v1);
    if (TIES) {
        v0 = settle_tie<CODE>(v0, x0, d);
        v1 = settle_tie<CODE>(v1, x1, d);
    }
    if constexpr (CODE == 0)
        return (uint32_t)(__float2int_rn(v0) & 0xff) | ((uint32_t)(__float2int_rn(v1) & 0xff) << 8);
    else
        return __nv_cvt_float2_to_fp8x2(make_float2(v0, v1), __NV_SATFINITE, __NV_E4M3);
}

// amax / lim, correctly rounded (the same theorem; below 2^-90, where a remainder
// may be subnormal, by a division).
template <int CODE>
__device__ __forceinline__ float scale_of(float amax)
{
    constexpr float lim = code_limit<CODE>(), y = 1.f / lim;
    if (amax < 0x1p-90f)
        return __fdiv_rn(amax, lim);
    const float q = amax * y;
    return fmaf(fmaf(-lim, q, amax), y, q);
}

// The rows of one warp: lane l finds out where row l goes (or comes from), all of
// them at once; the rows are then walked `RP = 32 / lanes of a row` at a time,
// U such passes with their loads in flight together. (Found row by row, the
// divisions by n and the page size cost more than the row.)
struct RowWalk {
    uint32_t n_rows;     // B n
    int per_warp;        // rows of a warp, at most 32
    int vecs;            // vectors of a row
    int lane_log;        // lanes of a row, as a power of two
};

// LPG lanes hold one group of LPG * 8 * NCH values.
template <class T, int CODE, bool VEC, int LPG, int NCH, int U>
__global__ void __launch_bounds__(kQ8Threads) q8_write_kernel(const Q8WriteArgs a, const RowWalk w)
{
    const int lane = threadIdx.x & 31;
    const uint32_t base = (blockIdx.x * (kQ8Threads / 32) + (threadIdx.x >> 5)) * (uint32_t)w.per_warp;
    int64_t my_dst = -1, my_src = 0;
    if (lane < w.per_warp && base + lane < w.n_rows) {
        const uint32_t row = base + lane;
        const int b = (int)(row / (uint32_t)a.n);
        const int i = (int)(row - (uint32_t)b * (uint32_t)a.n);
        if (i < (a.n_new ? __ldg(a.n_new + b) : a.n)) {
            my_dst = page_row(a.map, b, (int64_t)(a.start ? __ldg(a.start + b) : 0) + i);
            if (my_dst < 0 && a.err)
                atomicExch(a.err, kErrIndex);
            my_src = (int64_t)b * a.stride_b + (int64_t)i * a.stride_n;
        }
    }
    const int RP = 32 >> w.lane_log, l = lane & ((1 << w.lane_log) - 1), gpr = a.D / a.group;
    for (int r0 = 0; r0 < w.per_warp; r0 += U * RP) {
        int64_t dst[U], src[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int r = r0 + u * RP + (lane >> w.lane_log);
            dst[u] = __shfl_sync(0xffffffffu, my_dst, r & 31);
            src[u] = __shfl_sync(0xffffffffu, my_src, r & 31);
            if (r >= w.per_warp)
                dst[u] = -1;
        }
        for (int v0 = 0; v0 < w.vecs; v0 += 32 * NCH) {
            Raw<T> f[U][NCH];
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int c = 0; c < NCH; ++c) {
                    const int v = v0 + c * 32 + l;
                    if (dst[u] >= 0 && v < w.vecs) {
                        f[u][c] = load8<T, VEC>(static_cast<const T *>(a.x) + src[u] + v * 8);
                    } else {
                        f[u][c] = Raw<T>{};
                    }
                }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                uint32_t top = 0;
#pragma unroll
                for (int c = 0; c < NCH; ++c)
                    top = max(top, top_bits<T>(f[u][c]));
#pragma unroll
                for (int o = LPG / 2; o >= 1; o >>= 1)
                    top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
                if (dst[u] < 0 || v0 + l >= w.vecs)
                    continue;
                const float amax = from_bits<T>(top);
                const bool finite = __float_as_uint(amax) < 0x7f800000u;
                // Very large and very small groups are moved, exactly, to where neither
                // lim * x nor the remainders of quotients that matter (codes 2^-10 up) leave
                // fp32's normal range; values that become subnormal on the way have code 0.
                const float shift = amax >= 0x1p60f ? 0x1p-64f : (amax < 0x1p-60f ? 0x1p64f : 1.f);
                const float den = amax * shift;
                const float inv = __frcp_rn(den);
                uint8_t *out = a.cache + dst[u] * a.D;
#pragma unroll
                for (int c = 0; c < NCH; ++c) {
                    uint32_t q[2] = {0u, 0u};
                    if (finite && top != 0u) {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            q[i >> 1] |= codes2<CODE, sizeof(T) == 4>(value(f[u][c], 2 * i) * shift,
                                                                      value(f[u][c], 2 * i + 1) * shift, den, inv)
                                         << (16 * (i & 1));
                    }
                    *reinterpret_cast<uint2 *>(out + (v0 + c * 32 + l) * 8) = make_uint2(q[0], q[1]);
                }
                if ((l & (LPG - 1)) == 0)
                    a.scales[dst[u] * gpr + (v0 + l) / (LPG * NCH)] =
                        finite ? scale_of<CODE>(amax) : __int_as_float(0x7fc00000);
            }
        }
    }
}

// Sixteen codes a lane: one 16-byte load, two (fp32: four) 16-byte stores.
template <class T, int CODE, int U>
__global__ void __launch_bounds__(kQ8Threads) q8_read_kernel(const Q8ReadArgs a, const RowWalk w)
{
    const int lane = threadIdx.x & 31;
    const uint32_t base = (blockIdx.x * (kQ8Threads / 32) + (threadIdx.x >> 5)) * (uint32_t)w.per_warp;
    int64_t my_src = -1;
    if (lane < w.per_warp && base + lane < w.n_rows) {
        const uint32_t row = base + lane;
        const int b = (int)(row / (uint32_t)a.n);
        const int i = (int)(row - (uint32_t)b * (uint32_t)a.n);
        int64_t pos;
        bool want = true, bad = false;
        if (a.idx) {
            pos = __ldg(a.idx + row);
            want = pos != -1;
            bad = pos < -1;
        } else {
            pos = (int64_t)(a.start ? __ldg(a.start + b) : 0) + i;
            bad = pos < 0;
        }
        if (want && !bad && a.lens)
            want = pos < __ldg(a.lens + b);
        if (want && !bad) {
            my_src = page_row(a.map, b, pos);
            bad = my_src < 0;
        }
        if (bad && a.err)
            atomicExch(a.err, kErrIndex);
    }
    const int RP = 32 >> w.lane_log, l = lane & ((1 << w.lane_log) - 1), gpr = a.D / a.group;
    for (int r0 = 0; r0 < w.per_warp; r0 += U * RP) {
        int64_t src[U];
        bool live[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int r = r0 + u * RP + (lane >> w.lane_log);
            src[u] = __shfl_sync(0xffffffffu, my_src, r & 31);
            live[u] = r < w.per_warp && base + r < w.n_rows;
        }
        for (int v = l; v < w.vecs; v += 32) {
            uint4 q[U];
            float sc[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                q[u] = make_uint4(0u, 0u, 0u, 0u);      // code 0 and scale 0: a row of zeros
                sc[u] = 0.f;
                if (live[u] && src[u] >= 0) {
                    q[u] = __ldg(reinterpret_cast<const uint4 *>(a.cache + src[u] * a.D) + v);
                    sc[u] = __ldg(a.scales + src[u] * gpr + (uint32_t)v * 16u / (uint32_t)a.group);
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (!live[u])
                    continue;
                alignas(16) T o[16];
                const uint32_t c[4] = {q[u].x, q[u].y, q[u].z, q[u].w};
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const uint32_t two = (c[e >> 1] >> (16 * (e & 1))) & 0xffffu;
                    float c0, c1;
                    if constexpr (CODE == 0) {
                        c0 = (float)(int8_t)(two & 0xffu);
                        c1 = (float)(int8_t)(two >> 8);
                    } else {
                        const __half2 h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3);
                        c0 = __low2float(h);
                        c1 = __high2float(h);
                    }
                    o[2 * e] = from_f32<T>(c0 * sc[u]);
                    o[2 * e + 1] = from_f32<T>(c1 * sc[u]);
                }
                const int64_t row = (int64_t)base + r0 + u * RP + (lane >> w.lane_log);
                uint4 *dst = reinterpret_cast<uint4 *>(static_cast<T *>(a.out) + row * a.D + v * 16);
#pragma unroll
                for (int e = 0; e < (int)sizeof(T); ++e)
                    dst[e] = reinterpret_cast<const uint4 *>(o)[e];
            }
        }
    }
}

// Rows of `vecs` vectors. Few rows: one pass a warp, for the latency; where
// that still gives 32 warps an SM, four passes a warp, two at a time.
RowWalk plan_rows(int64_t n_rows, int vecs, bool &deep, unsigned &blocks)
{
    RowWalk w;
    w.n_rows = (uint32_t)n_rows;
    w.vecs = vecs;
    w.lane_log = 0;
    while (w.lane_log < 5 && (1 << w.lane_log) < vecs)
        ++w.lane_log;
    const int rp = 32 >> w.lane_log;
    deep = rp <= 8 && n_rows / (4 * rp) >= 32LL * sm_count();
    w.per_warp = deep ? 4 * rp : rp;
    const int64_t per_block = (int64_t)w.per_warp * (kQ8Threads / 32);
    blocks = (unsigned)((n_rows + per_block - 1) / per_block);
    return w;
}

template <class T, int CODE, bool VEC, int LPG, int NCH>
cudaError_t run_write(const Q8WriteArgs &a, cudaStream_t st)
{
    bool deep;
    unsigned blocks;
    const RowWalk w = plan_rows((int64_t)a.B * a.n, a.D / 8, deep, blocks);
    if (deep)
        q8_write_kernel<T, CODE, VEC, LPG, NCH, 2><<<blocks, kQ8Threads, 0, st>>>(a, w);
    else
        q8_write_kernel<T, CODE, VEC, LPG, NCH, 1><<<blocks, kQ8Threads, 0, st>>>(a, w);
    return cudaGetLastError();
}

template <class T, int CODE, bool VEC>
cudaError_t write_group(const Q8WriteArgs &a, cudaStream_t st)
{
    switch (a.group) {
    case 32: return run_write<T, CODE, VEC, 4, 1>(a, st);
    case 64: return run_write<T, CODE, VEC, 8, 1>(a, st);
    case 128: return run_write<T, CODE, VEC, 16, 1>(a, st);
    case 256: return run_write<T, CODE, VEC, 32, 1>(a, st);
    default: return run_write<T, CODE, VEC, 32, 2>(a, st);
    }
}

template <class T>
cudaError_t write_type(const Q8WriteArgs &a, int code, cudaStream_t st)
{
    const bool vec = ((reinterpret_cast<uintptr_t>(a.x) | (uintptr_t)(a.stride_b * (int64_t)sizeof(T)) |
                       (uintptr_t)(a.stride_n * (int64_t)sizeof(T))) & 15u) == 0;
    if (code == 0)
        return vec ? write_group<T, 0, true>(a, st) : write_group<T, 0, false>(a, st);
    return vec ? write_group<T, 1, true>(a, st) : write_group<T, 1, false>(a, st);
}

template <class T>
cudaError_t read_type(const Q8ReadArgs &a, int code, cudaStream_t st)
{
    bool deep;
    unsigned blocks;
    const RowWalk w = plan_rows((int64_t)a.B * a.n, a.D / 16, deep, blocks);
    if (code == 0) {
        if (deep)
            q8_read_kernel<T, 0, 2><<<blocks, kQ8Threads, 0, st>>>(a, w);
        else
            q8_read_kernel<T, 0, 1><<<blocks, kQ8Threads, 0, st>>>(a, w);
    } else {
        if (deep)
            q8_read_kernel<T, 1, 2><<<blocks, kQ8Threads, 0, st>>>(a, w);
        else
            q8_read_kernel<T, 1, 1><<<blocks, kQ8Threads, 0, st>>>(a, w);
    }
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_q8_write(const Q8WriteArgs &a, int type, int code, cudaStream_t stream)
{
    if (type == 0)
        return write_type<__nv_bfloat16>(a, code, stream);
    return type == 1 ? write_type<__half>(a, code, stream) : write_type<float>(a, code, stream);
}

cudaError_t launch_q8_read(const Q8ReadArgs &a, int type, int code, cudaStream_t stream)
{
    if (type == 0)
        return read_type<__nv_bfloat16>(a, code, stream);
    return type == 1 ? read_type<__half>(a, code, stream) : read_type<float>(a, code, stream);
}

}  // namespace sai
