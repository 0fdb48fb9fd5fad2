// Rows quantised to 8 bits as they are written into a (paged) cache, and read
// back. The 8-bit formats are the ones the source pages name for the indexer's
// products (page "Docker Build for DeepSeek-v4": FP8 recipes; here also 8-bit
// integers); the arithmetic is this library's own:
//
//   a group of `group` consecutive values with largest magnitude amax becomes
//     int8:  code = rint(127 x / amax),  scale = amax / 127
//     e4m3:  code = e4m3(448 x / amax),  scale = amax / 448
//   (ties to even; amax = 0: codes 0, scale 0; a NaN or infinity in the group:
//   codes 0, scale NaN), and is read back as code * scale.
//
// The codes are those of the formula in exact arithmetic. For 16-bit inputs
// one correctly rounded division is enough: lim * x is exact in fp32, and a
// quotient of a 15- or 18-bit by an 11-bit integer that is no tie is further
// from any tie than fp32's rounding. For fp32 inputs quotients next to a tie
// are decided again in 64 bits.
//
// Bound: HBM (each value is read and each code written once); at a few rows,
// the launch. One group is held by group/8 lanes, 8 values (one or two 16-byte
// loads) each, its maximum found by shuffles, so that a row is read once.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <math.h>
#include <type_traits>

#include "indexer_q8.h"
#include "sai_device.cuh"

namespace sai {
namespace {

constexpr int kQ8Threads = 256;

template <class T>
__device__ __forceinline__ float to_f32(T x);
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }
template <>
__device__ __forceinline__ float to_f32<__half>(__half x) { return __half2float(x); }
template <>
__device__ __forceinline__ float to_f32<float>(float x) { return x; }

template <class T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
template <>
__device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }

// Eight values starting at p: 16-byte loads when the rows allow them (VEC),
// element loads otherwise.
template <class T, bool VEC>
__device__ __forceinline__ void load8(const T *p, float (&f)[8])
{
    alignas(16) T t[8];
    if constexpr (VEC) {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i)
            reinterpret_cast<uint4 *>(t)[i] = __ldg(reinterpret_cast<const uint4 *>(p) + i);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            t[i] = p[i];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        f[i] = to_f32<T>(t[i]);
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

// Two codes (low byte first) of two values of a group with maximum amax > 0.
template <int CODE, bool TIES>
__device__ __forceinline__ uint32_t codes2(float x0, float x1, float amax)
{
    constexpr float lim = code_limit<CODE>();
    float v0 = __fdiv_rn(lim * x0, amax), v1 = __fdiv_rn(lim * x1, amax);
    if (TIES) {
        v0 = settle_tie<CODE>(v0, x0, amax);
        v1 = settle_tie<CODE>(v1, x1, amax);
    }
    if constexpr (CODE == 0)
        return (uint32_t)(__float2int_rn(v0) & 0xff) | ((uint32_t)(__float2int_rn(v1) & 0xff) << 8);
    else
        return __nv_cvt_float2_to_fp8x2(make_float2(v0, v1), __NV_SATFINITE, __NV_E4M3);
}

// LPG lanes hold one group of LPG * 8 * NCH values.
template <class T, int CODE, bool VEC, int LPG, int NCH>
__global__ void __launch_bounds__(kQ8Threads) q8_write_kernel(const Q8WriteArgs a, uint32_t groups_per_row,
                                                              uint32_t n_units)
{
    const uint32_t unit = blockIdx.x * (kQ8Threads / LPG) + threadIdx.x / LPG;
    const int l = threadIdx.x % LPG;
    const uint32_t row = unit / groups_per_row;
    const uint32_t gi = unit - row * groups_per_row;
    int64_t dst = -1;
    const T *src = nullptr;
    if (unit < n_units) {
        const int b = (int)(row / (uint32_t)a.n);
        const int i = (int)(row - (uint32_t)b * (uint32_t)a.n);
        if (i < (a.n_new ? __ldg(a.n_new + b) : a.n)) {
            const int64_t pos = (int64_t)(a.start ? __ldg(a.start + b) : 0) + i;
            dst = page_row(a.map, b, pos);
            if (dst < 0 && a.err && l == 0)
                atomicExch(a.err, kErrIndex);
            src = static_cast<const T *>(a.x) + (int64_t)b * a.stride_b + (int64_t)i * a.stride_n +
                  (int64_t)gi * (LPG * 8 * NCH);
        }
    }
    float f[NCH][8];
    uint32_t top = 0;    // |x| as bits: ordered as the values are, infinities and NaN above every number
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
        if (dst >= 0) {
            load8<T, VEC>(src + c * (LPG * 8) + l * 8, f[c]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                f[c][i] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
            top = max(top, __float_as_uint(f[c][i]) & 0x7fffffffu);
    }
#pragma unroll
    for (int o = LPG / 2; o >= 1; o >>= 1)
        top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (dst < 0)
        return;
    const bool finite = top < 0x7f800000u;
    const float amax = __uint_as_float(top);
    // lim * x must not pass fp32's range: large groups are scaled down exactly
    const float shrink = (sizeof(T) == 2 && !std::is_same<T, __nv_bfloat16>::value) || amax < 0x1p118f ? 1.f : 0x1p-16f;
    const float den = amax * shrink;
    uint8_t *out = a.cache + dst * a.D + (int64_t)gi * (LPG * 8 * NCH);
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
        uint32_t w[2] = {0u, 0u};
        if (finite && top != 0u) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                w[i >> 1] |= codes2<CODE, sizeof(T) == 4>(f[c][2 * i] * shrink, f[c][2 * i + 1] * shrink, den)
                             << (16 * (i & 1));
        }
        *reinterpret_cast<uint2 *>(out + c * (LPG * 8) + l * 8) = make_uint2(w[0], w[1]);
    }
    if (l == 0)
        a.scales[dst * groups_per_row + gi] =
            finite ? __fdiv_rn(amax, code_limit<CODE>()) : __int_as_float(0x7fc00000);
}

// Sixteen codes a thread: one 16-byte load, two (fp32: four) 16-byte stores.
template <class T, int CODE>
__global__ void __launch_bounds__(kQ8Threads) q8_read_kernel(const Q8ReadArgs a, uint32_t parts_per_row,
                                                             uint64_t n_parts)
{
    const uint64_t part = (uint64_t)blockIdx.x * kQ8Threads + threadIdx.x;
    if (part >= n_parts)
        return;
    const uint32_t row = (uint32_t)(part / parts_per_row);
    const uint32_t p = (uint32_t)(part - (uint64_t)row * parts_per_row);
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
    int64_t src = -1;
    if (want && !bad) {
        src = page_row(a.map, b, pos);
        bad = src < 0;
    }
    if (bad && a.err)
        atomicExch(a.err, kErrIndex);
    alignas(16) T o[16];
    if (src >= 0) {
        const uint4 q = __ldg(reinterpret_cast<const uint4 *>(a.cache + src * a.D) + p);
        const float sc = __ldg(a.scales + src * (a.D / a.group) + (p * 16u) / (uint32_t)a.group);
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint32_t two = (w[e >> 1] >> (16 * (e & 1))) & 0xffffu;
            float c0, c1;
            if constexpr (CODE == 0) {
                c0 = (float)(int8_t)(two & 0xffu);
                c1 = (float)(int8_t)(two >> 8);
            } else {
                const __half2 h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3);
                c0 = __low2float(h);
                c1 = __high2float(h);
            }
            o[2 * e] = from_f32<T>(c0 * sc);
            o[2 * e + 1] = from_f32<T>(c1 * sc);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 16; ++e)
            o[e] = from_f32<T>(0.f);
    }
    uint4 *dst = reinterpret_cast<uint4 *>(static_cast<T *>(a.out) + (int64_t)row * a.D + p * 16);
#pragma unroll
    for (int e = 0; e < (int)sizeof(T); ++e)
        dst[e] = reinterpret_cast<const uint4 *>(o)[e];
}

template <class T, int CODE, bool VEC>
cudaError_t write_group(const Q8WriteArgs &a, cudaStream_t st)
{
    const uint32_t gpr = (uint32_t)(a.D / a.group);
    const uint32_t units = (uint32_t)a.B * (uint32_t)a.n * gpr;
    auto blocks = [&](int lpg) { return (unsigned)(((uint64_t)units * lpg + kQ8Threads - 1) / kQ8Threads); };
    switch (a.group) {
    case 32: q8_write_kernel<T, CODE, VEC, 4, 1><<<blocks(4), kQ8Threads, 0, st>>>(a, gpr, units); break;
    case 64: q8_write_kernel<T, CODE, VEC, 8, 1><<<blocks(8), kQ8Threads, 0, st>>>(a, gpr, units); break;
    case 128: q8_write_kernel<T, CODE, VEC, 16, 1><<<blocks(16), kQ8Threads, 0, st>>>(a, gpr, units); break;
    case 256: q8_write_kernel<T, CODE, VEC, 32, 1><<<blocks(32), kQ8Threads, 0, st>>>(a, gpr, units); break;
    default: q8_write_kernel<T, CODE, VEC, 32, 2><<<blocks(32), kQ8Threads, 0, st>>>(a, gpr, units); break;
    }
    return cudaGetLastError();
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
    const uint32_t ppr = (uint32_t)(a.D / 16);
    const uint64_t parts = (uint64_t)a.B * (uint64_t)a.n * ppr;
    const unsigned blocks = (unsigned)((parts + kQ8Threads - 1) / kQ8Threads);
    if (code == 0)
        q8_read_kernel<T, 0><<<blocks, kQ8Threads, 0, st>>>(a, ppr, parts);
    else
        q8_read_kernel<T, 1><<<blocks, kQ8Threads, 0, st>>>(a, ppr, parts);
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
