// Gradient of the indexer's scores from the 8-bit codes that the forward kept
// (its activation checkpoints), on tcgen05 tensor cores (sm_100a). With G[t,j]
// the gradient of s[t,j] summed over the slots that select block j (0 where
// nothing does or j is no candidate), and m[t,h,j] = 1 where <q8[t,h], k8[j]> > 0
// (relu's derivative, exact since the products of codes are whole numbers):
//
//   dq[t,h,:] = w[t,h] sum_j m G[t,j] ks[j] k8[j,:]
//   dk[j,:]   = sum_{t,h} m G[t,j] w[t,h] qs[t,h] q8[t,h,:]
//   dw[t,h]   = qs[t,h] sum_j G[t,j] ks[j] relu(<q8[t,h], k8[j]>)
//
// the gradients with respect to the values that the codes stand for.
//
// Launches: bwd_prep_kernel writes G densely (slots of one block added in slot
// order) with each token's and each key's largest magnitudes; bwd_tc_kernel<dq> and <dk>; and
// bwd_reduce_kernel adds dk's partial sums in a fixed order. Nothing depends on
// timing: the same inputs give the same bits.
//
// Both tensor-core kernels have one form. Two stationary 128-row tiles A (query
// rows for dq, keys for dk) meet a stream of 128-row tiles B (keys; query
// rows). Each step forms S = A B^T in 8-bit integers (kind::i8, exact), the
// epilogue turns S in place into M, fp16, the masked gradient of each product,
// and M, read from tensor memory as the A operand, multiplies B's codes in fp16
// (whole numbers up to 127 are exact there) into an fp32 accumulator:
//
//   dq: lanes are (t,h) rows; M = m gk, gk[t,j] = G[t,j] ks[j]; B2 = k8. The
//       fp32 sum for dw runs beside it. gk comes from shared memory, the same
//       for all heads of a token.
//   dk: lanes are keys; M = m G[t,j], one value a lane and token; B2 =
//       w qs q8, scaled by row as the codes are turned into fp16.
//
// fp16's 11 bits (a rounding of 2^-11 of each term, below the bf16 outputs'
// 2^-8) hold the operands after a power of two brings the largest to the top of
// its range; what falls out at the other end is below 2^-39 of it. gk has a power of
// two for each token, w qs one for each token, and G, times that one's inverse, one for
// each key: with one for the batch, a token's dq and a key's dk were lost where their
// gradients were 2^-35 of others'.
//
// Bound: the chain of products, M and products through tensor memory. Per 128 x 128
// tile of D = 128 the tensor pipe has 256 cycles of kind::i8 and 512 of kind::f16, and is
// busy for a third of dq's time and two fifths of dk's. In dq an item's end adds to it,
// where the accumulator is read before M is handed over: 80 us at S = 4096 are about 4,900
// cycles a step of two tiles, 0.80 ms at S = 16384, whose items are longer, about 3,450.
// The two stationary tiles alternate: while one's M is formed the other's products
// run. Tiles are walked whatever is selected in them, up to the last that the tokens can
// see: the cost does not fall with K or with documents that end earlier. Warp roles: warp 0 TMA, warps 1 and 2
// issue the MMAs of one tile each (one warp for both left the tensor pipe idle
// through its waits), warps 4..11 and 12..19 the epilogues of the two tiles (two
// warps for each 32 lanes, 64 columns each). The halves are four chains of
// products, M, second products and the next products in the same place, so that
// some are with the tensor pipe while others form M. dk: warps 20..27 turn B's
// codes into scaled fp16; dq takes the keys in fp16 as bwd_prep_kernel wrote them
// (turned into fp16 tile by tile they cost dq a sixth of its instructions), and
// warps 20..23 stage gk. Every wait is bounded; on timeout the kernel records
// SAI_ERR_TIMEOUT and unwinds, and bwd_reduce_kernel makes the call's outputs NaN.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>

#include "indexer_q8.h"
#include "sai_device.cuh"
#include "sai_host.h"

namespace sai {
namespace {

constexpr int bw_threads(bool dq) { return dq ? 768 : 896; }
constexpr int kBwRing = 3;              // code tiles B in flight
// Floats between two tokens' staged gk: four more than a tile where a warp's lanes
// span few tokens, so that they use other banks (with 16 tokens a tile the shared
// memory has no room for it).
constexpr int gk_row(int hp) { return hp == 8 ? 128 : 132; }
constexpr int kPrepThreads = 128;
constexpr int kPrepCols = 4096;         // columns of G gathered at once, at most
// Each key's largest magnitude is kept by so many groups of tokens apart (every
// eighth token): the first blocks all raise every word, and at one word a key their
// atomics took as long as the rest of the kernel (S = 4096: 26 us, 14 with eight).
constexpr int kKeyGroups = 8;

struct BwPlan {
    int tt_log;            // tokens a 128-row tile, as a power of two
    int n_steps_seq;       // dk: token tiles a sequence
    int n_pairs;           // dk: 256-key pairs a sequence; dq: token pairs (2 tt tokens) a sequence
    int per_seq;           // dk: steps of one sequence
    int share, rest;       // dk: steps of a CTA; the first `rest` CTAs take one more
    const float *G;        // [B,S,P]
    const uint32_t *key;   // [kKeyGroups,B,P] the key's largest |G| times the token's power of two for
                           // w qs, as bits
    const float2 *row;     // [B,S] scale of the token's gk, the power of two above its |w qs|; 0, 0 where
                           // it has no gradient
    float *part;           // dk: [grid + B n_pairs][256][D]
    uint32_t *gave_up;     // not 0 where a wait gave up
};

// The power of two that brings a largest magnitude (bits) below 2^top, at
// least half way; 1 when there is none or it is not finite.
__device__ __forceinline__ float range_scale(uint32_t bits, int top)
{
    if (bits == 0u || bits >= 0x7f800000u)
        return 1.f;
    int e;
    frexpf(__uint_as_float(bits), &e);            // magnitude in [2^(e-1), 2^e)
    return ldexpf(1.f, max(-120, min(120, top - e)));
}

// 1 / f of a power of two of at least 2^-126, at most 2^126.
__device__ __forceinline__ float inverse_pow2(float f) { return __uint_as_float((254u << 23) - __float_as_uint(f)); }

// dk's factors are scaled by token and by key: with u the power of two above the
// token's largest |w qs| (kept where 256 / u is a normal number), B2 is w qs q8 256 / u,
// below 2^15 (2^16 in the last binade, still fp16), and M is G u f, f the power of two that
// brings the key's largest |G| u below 2^15.
__device__ __forceinline__ float weight_pow2(uint32_t bits)
{
    return __uint_as_float(max(8u, min(254u, (bits >> 23) + 1u)) << 23);
}
__device__ __forceinline__ float weight_scale(float u) { return __uint_as_float((262u << 23) - __float_as_uint(u)); }
__device__ __forceinline__ float key_scale(uint32_t bits)
{
    return __uint_as_float(min(253u, 268u - (bits >> 23)) << 23);
}

// Candidates [lo, hi) of the token at local index t (its position fits 31 bits:
// checked on the host).
__device__ __forceinline__ void token_range(const ScoresBwdArgs &a, int b, int t, int &lo, int &hi)
{
    const uint32_t pos = (uint32_t)a.t_begin + (uint32_t)t;
    hi = (int)min((uint32_t)a.P, (pos + 1u) / (uint32_t)a.cr);
    lo = 0;
    if (a.doc_start) {
        const int d = __ldg(a.doc_start + (int64_t)b * a.S + t);
        const uint32_t d0 = d < 0 ? 0u : min((uint32_t)d, pos);
        lo = (int)min((uint32_t)hi, (d0 + (uint32_t)a.cr - 1u) / (uint32_t)a.cr);
    }
}

// Sixteen codes as fp16 pairs: a byte x as x + 128 under the exponent of 1024 is
// 1152 + x in fp16, exactly.
__device__ __forceinline__ void codes_to_f16(const uint4 &v, uint32_t (&o)[8])
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    const __half2 off = __floats2half2_rn(-1152.f, -1152.f);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const uint32_t u = w[e] ^ 0x80808080u;
        const uint32_t p01 = __byte_perm(u, 0x64646464u, 0x4140), p23 = __byte_perm(u, 0x64646464u, 0x4342);
        const __half2 h01 = __hadd2(*reinterpret_cast<const __half2 *>(&p01), off);
        const __half2 h23 = __hadd2(*reinterpret_cast<const __half2 *>(&p23), off);
        o[2 * e] = *reinterpret_cast<const uint32_t *>(&h01);
        o[2 * e + 1] = *reinterpret_cast<const uint32_t *>(&h23);
    }
}

// One block a token, then blocks that write the keys' codes in fp16 (exact) for
// dq, 16 a thread. With idx: the token's G, gathered in shared memory
// kPrepCols columns at a time and written out where it has candidates. A
// block named by one slot (the selection's case) is a plain store, claimed by a
// bit; if any block is claimed twice, the columns are gathered again by one
// thread a block in slot order, so that the sum does not depend on timing.
__global__ void __launch_bounds__(kPrepThreads)
    bwd_prep_kernel(const ScoresBwdArgs a, float *G, uint32_t *key_max, float2 *row_scale, uint4 *k16, bool vec, int cols)
{
    if ((int64_t)blockIdx.x >= (int64_t)a.B * a.S) {
        const int64_t i = ((int64_t)blockIdx.x - (int64_t)a.B * a.S) * kPrepThreads + threadIdx.x;
        if (i >= (int64_t)a.B * a.P * (a.D / 16))
            return;
        uint32_t o[8];
        codes_to_f16(__ldg(reinterpret_cast<const uint4 *>(a.k8) + i), o);
        k16[2 * i] = make_uint4(o[0], o[1], o[2], o[3]);
        k16[2 * i + 1] = make_uint4(o[4], o[5], o[6], o[7]);
        return;
    }
    extern __shared__ float4 prep_smem[];            // [cols] G, [cols / 32] claims
    float *g = reinterpret_cast<float *>(prep_smem);
    uint32_t *claimed = reinterpret_cast<uint32_t *>(g + cols);
    __shared__ uint32_t buf[3][kPrepThreads / 32];    // largest |w qs|, |G ks|; any gradient at all
    const int64_t row = blockIdx.x;
    const int b = (int)(row / a.S);
    const int t = (int)(row - (int64_t)b * a.S);
    int lo, hi;
    token_range(a, b, t, lo, hi);
    // the largest finite magnitudes: one NaN or infinity does not unscale the others
    auto finite = [](float v) {
        const uint32_t u = __float_as_uint(v) & 0x7fffffffu;
        return u < 0x7f800000u ? u : 0u;
    };
    const float *ks = a.k_scale + (int64_t)b * a.P;
    const float *ds = a.dscores + row * a.K;
    const int32_t *idx = a.idx ? a.idx + row * a.K : nullptr;
    // the first slots, on their way while the weights are looked at
    int4 id0 = make_int4(-1, -1, -1, -1);
    float4 v0 = make_float4(0.f, 0.f, 0.f, 0.f);
    const bool first = vec && (int)threadIdx.x < a.K / 4;
    if (first) {
        id0 = __ldg(reinterpret_cast<const int4 *>(idx) + threadIdx.x);
        v0 = __ldg(reinterpret_cast<const float4 *>(ds) + threadIdx.x);
    }
    // (H <= 128: one value a thread)
    const bool has_h = (int)threadIdx.x < a.H;
    const float wv = has_h ? __ldg(a.w + row * a.H + threadIdx.x) : 0.f;
    const float qv = has_h ? __ldg(a.q_scale + row * a.H + threadIdx.x) : 0.f;
    const uint32_t top_w = __reduce_max_sync(0xffffffffu, finite(wv * qv));
    if ((threadIdx.x & 31) == 0)
        buf[0][threadIdx.x >> 5] = top_w;
    __syncthreads();
    uint32_t w_bits = 0;
#pragma unroll
    for (int i = 0; i < kPrepThreads / 32; ++i)
        w_bits = max(w_bits, buf[0][i]);
    const float u = weight_pow2(w_bits);
    uint32_t top_gk = 0u, any = 0u;
    uint32_t *km = key_max + ((int64_t)(t & (kKeyGroups - 1)) * a.B + b) * a.P;
    auto seen = [&](float v, float scale) {
        if (v != 0.f) {
            any = 1u;
            top_gk = max(top_gk, finite(v * scale));
        }
    };
    // Largest of the keys [j0, j1), of which key j has the gradient of(j): only a
    // largest value's binade is used, so a word is written where the binade rises (a
    // stale word only means one more atomic). Four words a thread on their way at once.
    auto keys_seen = [&](int j0, int j1, auto of) {
        for (int j = j0 + threadIdx.x; j < j1; j += 4 * kPrepThreads) {
            uint32_t had[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                had[e] = j + e * kPrepThreads < j1 ? __ldcg(km + j + e * kPrepThreads) : 0u;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (j + e * kPrepThreads < j1) {
                    const uint32_t most = finite(of(j + e * kPrepThreads) * u);
                    if ((most >> 23) > (had[e] >> 23))
                        atomicMax(km + j + e * kPrepThreads, most);
                }
        }
    };
    if (!a.idx) {
        for (int j = lo + threadIdx.x; j < hi; j += kPrepThreads)
            seen(__ldg(ds + j), __ldg(ks + j));
        keys_seen(lo, hi, [&](int j) { return __ldg(ds + j); });
    } else {
        for (int c0 = lo & ~31; c0 < hi || c0 == (lo & ~31); c0 += cols) {
            const int n = max(0, min(cols, hi - c0));
            for (int j = threadIdx.x; j < n; j += kPrepThreads)
                g[j] = 0.f;
            for (int j = threadIdx.x; j < (n + 31) / 32; j += kPrepThreads)
                claimed[j] = 0u;
            __syncthreads();
            bool twice = false;
            auto slot = [&](int id, float v) {
                const int j = id - c0;
                if ((id < -1 || id >= a.P) && a.err)
                    atomicExch(a.err, kErrIndex);
                if (id < lo || id >= hi || j < 0 || j >= n)
                    return;
                if (atomicOr(&claimed[j >> 5], 1u << (j & 31)) & (1u << (j & 31)))
                    twice = true;
                else
                    g[j] = v;
            };
            if (vec) {
                if (first) {
                    slot(id0.x, v0.x);
                    slot(id0.y, v0.y);
                    slot(id0.z, v0.z);
                    slot(id0.w, v0.w);
                }
                for (int k = threadIdx.x + kPrepThreads; k < a.K / 4; k += kPrepThreads) {
                    const int4 id = __ldg(reinterpret_cast<const int4 *>(idx) + k);
                    const float4 v = __ldg(reinterpret_cast<const float4 *>(ds) + k);
                    slot(id.x, v.x);
                    slot(id.y, v.y);
                    slot(id.z, v.z);
                    slot(id.w, v.w);
                }
            } else {
                for (int k = threadIdx.x; k < a.K; k += kPrepThreads) {
                    const int id = __ldg(idx + k);
                    const float v = __ldg(ds + k);
                    slot(id, v);
                }
            }
            if (__syncthreads_or(twice)) {
                for (int j = threadIdx.x; j < n; j += kPrepThreads)
                    g[j] = 0.f;
                __syncthreads();
                for (int k = 0; k < a.K; ++k) {
                    const int id = __ldg(idx + k), j = id - c0;
                    if (id >= lo && id < hi && j >= 0 && j < n && (j & (kPrepThreads - 1)) == (int)threadIdx.x)
                        g[j] += __ldg(ds + k);
                }
                __syncthreads();
            }
            if (vec) {
                // (whole quadruples: what lies past the candidates is written, not read)
                for (int j = threadIdx.x * 4; j < n; j += kPrepThreads * 4) {
                    const float4 v = *reinterpret_cast<const float4 *>(g + j);
                    const float4 k4 = __ldg(reinterpret_cast<const float4 *>(ks + c0 + j));
                    *reinterpret_cast<float4 *>(G + row * a.P + c0 + j) = v;
                    const float vv[4] = {v.x, v.y, v.z, v.w}, kk[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (j + e < n)
                            seen(vv[e], kk[e]);
                }
            } else {
                for (int j = threadIdx.x; j < n; j += kPrepThreads) {
                    const float v = g[j];
                    if (c0 + j >= lo)
                        G[row * a.P + c0 + j] = v;
                    seen(v, __ldg(ks + c0 + j));
                }
            }
            // (a warp's atomics fall on 32 neighbouring words, however G is written)
            keys_seen(c0, c0 + n, [&](int j) { return g[j - c0]; });
            __syncthreads();
        }
    }
    top_gk = __reduce_max_sync(0xffffffffu, top_gk);
    any = __reduce_max_sync(0xffffffffu, any);
    if ((threadIdx.x & 31) == 0) {
        buf[1][threadIdx.x >> 5] = top_gk;
        buf[2][threadIdx.x >> 5] = any;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
#pragma unroll
        for (int i = 1; i < kPrepThreads / 32; ++i) {
            top_gk = max(top_gk, buf[1][i]);
            any |= buf[2][i];
        }
        row_scale[row] = any ? make_float2(range_scale(top_gk, 15), u) : make_float2(0.f, 0.f);
    }
}

// ------------------------------------------------------------ the walk
// dk: first step of CTA x's share of the batch's steps.
__device__ __forceinline__ int share_start(const BwPlan &p, int x) { return x * p.share + min(x, p.rest); }

// The steps of one CTA, the same for every role: dq walks one item (2 tt tokens,
// late tokens, which have the most key tiles, first) of every gridDim.x, there and
// back: the CTA with the longest item of one round takes the shortest of the next
// (always from the same end, the first CTA had 35 steps at S = 4096 where the mean
// is 31, and the whole call takes 178 us against 176). dk walks a contiguous share
// of all steps of the batch (a pair of key tiles times the token tiles that see
// it), so its share may end inside a pair.
template <int MODE>
struct Walk {
    int b, a0;          // sequence; the stationary rows' first token (dq) or key (dk)
    int s, s_end;       // the streamed tile and the end of the item's
    bool first;         // the item's first step
    int pair;           // dk: pair of the batch
    // position
    int item, hop;      // dq: the item, and how far on the next one is
    int at, end;        // dk

    __device__ __forceinline__ bool set(const ScoresBwdArgs &a, const BwPlan &p);
    __device__ __forceinline__ bool begin(const ScoresBwdArgs &a, const BwPlan &p)
    {
        item = (int)blockIdx.x;
        hop = 2 * ((int)gridDim.x - item) - 1;
        at = share_start(p, (int)blockIdx.x);
        end = share_start(p, (int)blockIdx.x + 1);
        return set(a, p);
    }
    __device__ __forceinline__ bool next(const ScoresBwdArgs &a, const BwPlan &p)
    {
        first = false;
        if (++s < s_end)
            return true;
        if (MODE == 0)
            hop_on();
        return set(a, p);
    }
    __device__ __forceinline__ void hop_on()
    {
        item += hop;
        hop = 2 * (int)gridDim.x - hop;
    }
    __device__ __forceinline__ bool last() const { return s == s_end - 1; }
};

// First token tile that sees a key of pair kp.
__device__ __forceinline__ int first_step(const ScoresBwdArgs &a, const BwPlan &p, int kp)
{
    const int64_t t = (int64_t)(256 * (int64_t)kp + 1) * a.cr - 1 - a.t_begin;
    return t <= 0 ? 0 : (int)min((int64_t)p.n_steps_seq, t >> p.tt_log);
}

template <>
__device__ __forceinline__ bool Walk<0>::set(const ScoresBwdArgs &a, const BwPlan &p)
{
    for (; item < a.B * p.n_pairs; hop_on()) {
        b = item % a.B;
        a0 = (p.n_pairs - 1 - item / a.B) << (p.tt_log + 1);
        const uint32_t seen = (uint32_t)a.t_begin + (uint32_t)min(a.S, a0 + (2 << p.tt_log));
        s = 0;
        s_end = (int)((min((uint32_t)a.P, seen / (uint32_t)a.cr) + 127u) / 128u);
        first = true;
        if (s_end > 0)
            return true;
        // no candidate: the epilogue writes the zeros before its walk
    }
    return false;
}

template <>
__device__ __forceinline__ bool Walk<1>::set(const ScoresBwdArgs &a, const BwPlan &p)
{
    if (at >= end)
        return false;
    b = at / p.per_seq;
    int r = at - b * p.per_seq;
    int kp = 0, f = first_step(a, p, 0);
    while (r >= p.n_steps_seq - f) {
        r -= p.n_steps_seq - f;
        f = first_step(a, p, ++kp);
    }
    s = f + r;
    const int n = min(p.n_steps_seq - s, end - at);
    s_end = s + n;
    at += n;
    a0 = kp * 256;
    pair = b * p.n_pairs + kp;
    first = true;
    return true;
}

struct BwSmem {
    uint64_t a_full[2], a_empty[2];
    uint64_t b_full[kBwRing], b_empty[kBwRing];
    uint64_t c_full[2], c_empty[2];      // fp16 tiles: loaded (dq); read
    uint64_t s_full[2][2];               // per stationary tile and half: products there
    uint64_t m_full[2][2][2];            // per tile and half, even and odd steps: M and B2 there
    uint64_t acc_full[2], acc_empty[2];  // per tile: an item's accumulator there; read by both halves
    uint64_t g_full[2], g_empty[2];      // dq: gk staged, read
    uint64_t dw_full[2];                 // dq, per tile: the second half's part of dw
    float dw[2][128];
    uint64_t drain[2];
    uint32_t tmem_base;
    int abort_flag;
};

// dq: gk of two steps, both tiles; and 1 KB of output for each epilogue warp.
constexpr size_t gk_bytes(int hp) { return (size_t)2 * 2 * (128 / hp) * gk_row(hp) * 4; }

template <int D>
constexpr size_t bw_smem_bytes(bool dq, int hp)
{
    return 1024 + 4 * 128 * D + (size_t)kBwRing * 128 * D + 2 * 128 * D * 2 + (dq ? gk_bytes(hp) + 16 * 1024 : 0) +
           sizeof(BwSmem);
}
static_assert(bw_smem_bytes<128>(true, 8) <= 232448, "shared memory of a block");

// Offset of 16-byte chunk c of row r in a tile of ROW_BYTES rows stored with
// the swizzle of that span (rows of 32, 64 or 128 bytes; the 16-byte chunks
// of a row are permuted by the row's place in its 8-row atom).
template <int ROW_BYTES>
__device__ __forceinline__ uint32_t swz(uint32_t r, uint32_t c)
{
    if (ROW_BYTES == 128)
        c ^= r & 7u;
    else if (ROW_BYTES == 64)
        c ^= (r >> 1) & 3u;
    else
        c ^= (r >> 2) & 1u;
    return r * ROW_BYTES + c * 16;
}

template <int MODE, int D, int HP>
__global__ void __launch_bounds__(bw_threads(MODE == 0), 1)
    bwd_tc_kernel(const __grid_constant__ CUtensorMap mapA, const __grid_constant__ CUtensorMap mapB,
                  const __grid_constant__ CUtensorMap mapC, const ScoresBwdArgs a, const BwPlan p)
{
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    constexpr int TT = 128 / HP;                       // tokens of a 128-row tile
    constexpr int kBwRow = gk_row(HP);
    constexpr uint32_t tile8 = 128 * D, tile16 = 256 * D;
    constexpr int kC = D * 2 > 128 ? 128 : D * 2;      // bytes of a row block of the fp16 tile
    uint8_t *sa = base;                                // [2 items][2 tiles]
    uint8_t *sb = sa + 4 * tile8;                      // [ring]
    uint8_t *sc = sb + kBwRing * tile8;                // [2] fp16
    float *sg = reinterpret_cast<float *>(sc + 2 * tile16);   // dq: [2][2 TT][kBwRow] gk,
                                                              // then 1 KB of output a warp
    BwSmem *sm = reinterpret_cast<BwSmem *>(reinterpret_cast<uint8_t *>(sg) +
                                            (MODE == 0 ? gk_bytes(HP) + 16 * 1024 : 0));
    constexpr int kConv = MODE == 0 ? 0 : 8;           // converting warps
    const int warp = uniform_warp();
    const int lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm->a_full[i], 1);
            mbar_init(&sm->a_empty[i], 2);          // each tile's last products
            mbar_init(&sm->c_full[i], 1);
            mbar_init(&sm->c_empty[i], 4);
            for (int h = 0; h < 2; ++h) {
                mbar_init(&sm->s_full[i][h], 1);
                mbar_init(&sm->m_full[i][h][0], 4 + kConv);    // the epilogue's warps and the converters
                mbar_init(&sm->m_full[i][h][1], 4 + kConv);
            }
            mbar_init(&sm->acc_full[i], 1);
            mbar_init(&sm->acc_empty[i], 8);
            mbar_init(&sm->g_full[i], 4);
            mbar_init(&sm->g_empty[i], 16);
            mbar_init(&sm->dw_full[i], 4);
            mbar_init(&sm->drain[i], 1);
        }
        for (int i = 0; i < kBwRing; ++i) {
            mbar_init(&sm->b_full[i], 1);
            mbar_init(&sm->b_empty[i], 4 + kConv);  // all products done (passed on by warps); converted
        }
        sm->abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 0) {
        tmem_alloc(&sm->tmem_base, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm->tmem_base;               // S/M of the two tiles, then their accumulators
    volatile int *abort_flag = &sm->abort_flag;
    Walk<MODE> wk;

    if (warp == 0) {
        // ------------------------------------------------ TMA producer
        if (lane == 0) {
            tma_prefetch_desc(&mapA);
            tma_prefetch_desc(&mapB);
        }
        int stage = 0, item = -1, n = 0;
        uint32_t phase = 0, a_used = 0, b_used = 0, b_parity = 0;
        bool ok = true;
        for (bool go = wk.begin(a, p); go; go = wk.next(a, p)) {
            if (wk.first) {
                ++item;
                const int ab = item & 1;
                if (!warp_mbar_wait_short(&sm->a_empty[ab], ((item >> 1) & 1) ^ 1u, abort_flag, a.err)) {
                    ok = false;
                    break;
                }
                if (lane == 0) {
                    mbar_arrive_expect_tx(&sm->a_full[ab], 2 * tile8);
                    for (int i = 0; i < 2; ++i) {
                        uint8_t *dst = sa + (2 * ab + i) * tile8;
                        if (MODE == 0)
                            tma_load_3d(dst, &mapA, &sm->a_full[ab], 0, 0, wk.b * a.S + wk.a0 + i * TT);
                        else
                            tma_load_3d(dst, &mapA, &sm->a_full[ab], 0, wk.a0 + i * 128, wk.b);
                    }
                }
                __syncwarp();
                a_used |= 1u << ab;
            }
            if (!warp_mbar_wait_short(&sm->b_empty[stage], phase ^ 1u, abort_flag, a.err)) {
                ok = false;
                break;
            }
            if (lane == 0) {
                mbar_arrive_expect_tx(&sm->b_full[stage], tile8);
                if (MODE == 0)
                    tma_load_3d(sb + stage * tile8, &mapB, &sm->b_full[stage], 0, wk.s * 128, wk.b);
                else
                    tma_load_3d(sb + stage * tile8, &mapB, &sm->b_full[stage], 0, 0, wk.b * a.S + wk.s * TT);
            }
            __syncwarp();
            b_used |= 1u << stage;
            b_parity = (b_parity & ~(1u << stage)) | (phase << stage);
            if (++stage == kBwRing) {
                stage = 0;
                phase ^= 1u;
            }
            if (MODE == 0) {
                // the same keys in fp16
                const int cb = n & 1;
                if (!warp_mbar_wait_short(&sm->c_empty[cb], ((n >> 1) & 1) ^ 1u, abort_flag, a.err)) {
                    ok = false;
                    break;
                }
                if (lane == 0) {
                    mbar_arrive_expect_tx(&sm->c_full[cb], tile16);
                    for (int blk = 0; blk < D * 2 / kC; ++blk)
                        tma_load_3d(sc + cb * tile16 + blk * (128 * kC), &mapC, &sm->c_full[cb], blk * (kC / 2),
                                    wk.s * 128, wk.b);
                }
                __syncwarp();
            }
            ++n;
        }
        if (!ok && lane == 0) {
            // let the copies in flight land before the CTA goes
            for (int i = 0; i < kBwRing; ++i)
                if (b_used & (1u << i))
                    mbar_drain(&sm->b_full[i], (b_parity >> i) & 1u);
            if (MODE == 0)
                for (int i = 0; i < 2; ++i)
                    if (n > i)
                        mbar_drain(&sm->c_full[i], (uint32_t)((n - 1 - i) / 2) & 1u);
            for (int i = 0; i < 2; ++i)
                if (a_used & (1u << i)) {
                    const int uses = (item - i + 2) / 2;       // loads asked for into buffer i, or one more
                    mbar_drain(&sm->a_full[i], (uint32_t)(uses - 1) & 1u);
                }
        }
        __syncwarp();
    } else if (warp == 1 || warp == 2) {
        // ------------------------------------------------ MMA issuer of tile i
        // A wait or a commit costs a warp about 100 cycles, so a step has two
        // waits and one commit; everything else that must be known done (code tiles
        // read, fp16 tiles read) follows from the products of the next step and
        // is passed on by the warps that wait for those. The halves are added in order.
        // A half's second products (kind::f16) read M from tensor memory, and the next
        // kind::i8 products are issued behind them, without a wait between, into the columns
        // that M lies in. This takes it that one thread's tcgen05.mma run in the order of
        // their issue. The PTX manual promises that for one accumulator and shape, and here
        // both differ; repeated runs of long lists of items have always given the same bits.
        const int i = warp - 1;
        constexpr uint32_t id_s = idesc_i8_s32(128, 64);
        constexpr uint32_t id_acc = idesc_f16_f32_bmn(128, D);
        const uint64_t a_desc = sdesc_k_rows<D>(smem_u32(sa + i * tile8));
        const uint64_t b_desc = sdesc_k_rows<D>(smem_u32(sb));
        const uint64_t c_desc = sdesc_mn_rows<kC>(smem_u32(sc), 128 * kC);
        const uint32_t t_s = tmem + i * 128, t_acc = tmem + 256 + i * D;
        int stage = 0, item = -1, n = 0, items = 0;
        uint32_t phase = 0;
        bool issued = false;
        // S = A B^T of the walk's step, for the 64 rows of B that half `hf` names
        auto products = [&](int hf) {
            const uint64_t da = a_desc + 2 * (item & 1) * (tile8 / 16);
            const uint64_t db = b_desc + stage * (tile8 / 16) + hf * (tile8 / 32);
            if (elect_one()) {
#pragma unroll
                for (int kk = 0; kk < D / 32; ++kk)
                    umma_i8(t_s + hf * 64, da + 2 * kk, db + 2 * kk, id_s, kk != 0);
                umma_commit(&sm->s_full[i][hf]);
                if (hf == 1 && wk.last())
                    umma_commit(&sm->a_empty[item & 1]);
            }
            __syncwarp();
            issued = true;
            if (hf == 1 && ++stage == kBwRing) {
                stage = 0;
                phase ^= 1u;
            }
        };
        // the walk's step: its tiles are in place
        auto arrive_step = [&]() -> bool {
            if (wk.first) {
                ++item;
                if (!warp_mbar_wait_short(&sm->a_full[item & 1], (item >> 1) & 1, abort_flag, a.err))
                    return false;
            }
            return warp_mbar_wait_short(&sm->b_full[stage], phase, abort_flag, a.err);
        };
        bool go = wk.begin(a, p);
        bool ok = go && arrive_step();
        if (ok) {
            tc_fence_after();
            products(0);
            products(1);
        }
        while (go && ok) {
            const bool fresh = wk.first, closes = wk.last();
            const uint64_t dc = c_desc + (n & 1) * (tile16 / 16);
            go = wk.next(a, p);                  // the walk is now one step ahead
            ok = !go || arrive_step();
#pragma unroll
            for (int hf = 0; hf < 2 && ok; ++hf) {
                ok = MODE == 0 && hf == 0
                         ? warp_mbar_wait_both(&sm->m_full[i][hf][n & 1], (n >> 1) & 1, &sm->c_full[n & 1], (n >> 1) & 1,
                                               abort_flag, a.err)
                         : warp_mbar_wait_short(&sm->m_full[i][hf][n & 1], (n >> 1) & 1, abort_flag, a.err);
                // an item's first products overwrite the accumulator: the last item's must
                // have been read (the first half is there before the second has read it)
                if (ok && hf == 0 && fresh) {
                    ok = warp_mbar_wait_short(&sm->acc_empty[i], (items & 1) ^ 1u, abort_flag, a.err);
                    ++items;
                }
                if (!ok)
                    break;
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        umma_f16_ta(t_acc, t_s + hf * 64 + kk * 8, dc + (hf * 4 + kk) * kC, id_acc,
                                    hf == 0 && kk == 0 && fresh ? 0u : 1u);
                    if (hf == 1 && closes)
                        umma_commit(&sm->acc_full[i]);
                }
                __syncwarp();
                if (go)
                    products(hf);
            }
            ++n;
        }
        if (*abort_flag && issued && lane == 0) {
            umma_commit(&sm->drain[i]);
            mbar_drain(&sm->drain[i], 0);
        }
        __syncwarp();
    } else if (MODE == 1 && warp >= 20) {
        // ------------------------------------------------ codes to fp16
        const int r = (threadIdx.x - 640) & 127;       // row of the tile; two threads a row
        constexpr int kChunks = D / 32;                // 16-code chunks a thread
        const int chunk0 = ((threadIdx.x - 640) >> 7) * kChunks;
        // this row's scale; its parts are loaded a step ahead and put together when used
        float rw = 0.f, rs = 0.f, ru = 0.f;
        auto fetch = [&]() {
            const int tt = r / HP, h = r % HP;
            const int t = wk.s * TT + tt;
            rw = rs = ru = 0.f;
            if (t < a.S && h < a.H) {
                const int64_t row = (int64_t)wk.b * a.S + t;
                ru = __ldg(&p.row[row].y);
                rw = __ldg(a.w + row * a.H + h);
                rs = __ldg(a.q_scale + row * a.H + h);
            }
        };
        int stage = 0, n = 0;
        uint32_t phase = 0;
        bool go = wk.begin(a, p);
        if (go)
            fetch();
        while (go) {
            // (a token without a gradient adds nothing, whatever its weights hold)
            const float scale = ru != 0.f ? rw * rs * weight_scale(ru) : 0.f;
            go = wk.next(a, p);
            if (go)
                fetch();
            const int cb = n & 1;
            if (!warp_mbar_wait_both(&sm->b_full[stage], phase, &sm->c_empty[cb], ((n >> 1) & 1) ^ 1u, abort_flag,
                                     a.err))
                break;
            const uint8_t *src = sb + stage * tile8;
            uint8_t *dst = sc + cb * tile16;
            // scale as an fp16 pair whose sum has 22 bits: x * scale is rounded once
            const __half hi = __float2half_rn(scale);
            const __half lo = __float2half_rn(scale - __half2float(hi));
            const __half2 hi2 = __half2half2(hi), lo2 = __half2half2(lo);
#pragma unroll
            for (int k = 0; k < kChunks; ++k) {
                const int c = chunk0 + k;
                const uint4 v = *reinterpret_cast<const uint4 *>(src + swz<D>(r, c));
                uint32_t o[8];
                codes_to_f16(v, o);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const __half2 h = *reinterpret_cast<const __half2 *>(&o[e]);
                    const __half2 y = __hfma2(h, hi2, __hmul2(h, lo2));
                    o[e] = *reinterpret_cast<const uint32_t *>(&y);
                }
                // 16 values are two 16-byte chunks of the row's fp16 block
                const uint32_t ch = 2 * c, blk = ch / (kC / 16), cc = ch % (kC / 16);
                uint8_t *d = dst + blk * (128 * kC);
                *reinterpret_cast<uint4 *>(d + swz<kC>(r, cc)) = make_uint4(o[0], o[1], o[2], o[3]);
                *reinterpret_cast<uint4 *>(d + swz<kC>(r, cc + 1)) = make_uint4(o[4], o[5], o[6], o[7]);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                for (int i = 0; i < 4; ++i)
                    mbar_arrive(&sm->m_full[i >> 1][i & 1][cb]);
                mbar_arrive(&sm->b_empty[stage]);
            }
            ++n;
            if (++stage == kBwRing) {
                stage = 0;
                phase ^= 1u;
            }
        }
    } else if (MODE == 0 && warp >= 20) {
        // ------------------------------------------------ dq: gk staged
        // gk of the step's 128 keys and both tiles' tokens: thread = key, one value
        // a token, read from G a step ahead; lane e holds token e's candidates and scale.
        constexpr int NT = 2 * TT;
        const int r = threadIdx.x - 640;
        float g[NT], ksv = 0.f, f = 0.f;
        int lo = 0, hi = 0;
        auto fetch = [&]() {
            if (wk.first) {
                const int t = wk.a0 + lane;
                lo = hi = 0;
                if (lane < NT && t < a.S) {
                    token_range(a, wk.b, t, lo, hi);
                    f = __ldg(&p.row[(int64_t)wk.b * a.S + t].x);
                }
            }
            const int j = wk.s * 128 + r;
            ksv = j < a.P ? __ldg(a.k_scale + (int64_t)wk.b * a.P + j) : 0.f;
            const float *src = p.G + ((int64_t)wk.b * a.S + wk.a0) * a.P + j;
#pragma unroll
            for (int e = 0; e < NT; ++e, src += a.P) {
                const int l = __shfl_sync(0xffffffffu, lo, e), u = __shfl_sync(0xffffffffu, hi, e);
                g[e] = j >= l && j < u ? __ldg(src) : 0.f;
            }
        };
        int n = 0;
        bool go = wk.begin(a, p);
        if (go)
            fetch();
        while (go) {
            if (!warp_mbar_wait_short(&sm->g_empty[n & 1], ((n >> 1) & 1) ^ 1u, abort_flag, a.err))
                break;
            float *dst = sg + (n & 1) * NT * kBwRow + r;
#pragma unroll
            for (int e = 0; e < NT; ++e) {
                const float fe = __shfl_sync(0xffffffffu, f, e);
                dst[e * kBwRow] = g[e] != 0.f ? g[e] * ksv * fe : 0.f;
            }
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&sm->g_full[n & 1]);
            ++n;
            go = wk.next(a, p);
            if (go)
                fetch();
        }
    } else if (warp >= 4) {
        // ------------------------------------------------ epilogue of tile i, 64 columns a warp
        const int i = (warp - 4) >> 3, half = ((warp - 4) >> 2) & 1;
        const int q = warp & 3;
        const int r = q * 32 + lane;                   // tile row
        // S columns [64 half, 64 half + 64); M takes the first 32 of them
        const uint32_t ts = tmem + i * 128 + half * 64 + ((uint32_t)(q * 32) << 16);
        // the accumulator's columns that this warp reads
        const uint32_t ta = tmem + 256 + i * D + half * (D / 2) + ((uint32_t)(q * 32) << 16);
        // One warp passes on what its tile's products of step n imply: it has read
        // step n's code tile and step n-1's fp16 tile.
        int ring = 0;
        auto pass_on = [&](int n) {
            if (q == 0 && lane == 0) {
                mbar_arrive(&sm->b_empty[ring]);
                if (n > 0)
                    mbar_arrive(&sm->c_empty[(n - 1) & 1]);
            }
            if (++ring == kBwRing)
                ring = 0;
        };
        int n = 0, items = 0;
        if constexpr (MODE == 0) {
            const int tt = r / HP, h = r % HP;
            uint4 *out = reinterpret_cast<uint4 *>(sg + 4 * TT * kBwRow) + (warp - 4) * 64;
            // Items without a candidate never reach the walk: their gradients are zero.
            for (int it = (int)blockIdx.x; it < a.B * p.n_pairs; it += gridDim.x) {
                const int b = it % a.B, a0 = (p.n_pairs - 1 - it / a.B) * 2 * TT, t = a0 + i * TT + tt;
                if (((uint32_t)a.t_begin + (uint32_t)min(a.S, a0 + 2 * TT)) / (uint32_t)a.cr > 0 || t >= a.S || h >= a.H || half)
                    continue;
                const int64_t row = ((int64_t)b * a.S + t) * a.H + h;
                a.dw[row] = 0.f;
                for (int c = 0; c < D / 8; ++c)
                    reinterpret_cast<uint4 *>(a.dq + row * D)[c] = make_uint4(0u, 0u, 0u, 0u);
            }
            // The thread's row of the current item, and of a finished one whose
            // accumulator is still to be read: that is done after the next item's
            // first M is formed (its products were under way), just before M is
            // handed over, from when on the accumulator may be overwritten.
            constexpr uint32_t kNone = 0xffffffffu;
            uint32_t row = kNone, old_row = kNone;      // B S H fits 31 bits
            float wq = 0.f, qs = 0.f, old_wq = 0.f, old_dw = 0.f;
            bool any = false, pending = false;
            uint64_t dw[2] = {0u, 0u};                  // two fp32 sums each
            auto finish = [&]() -> bool {
                if (!warp_mbar_wait_short(&sm->acc_full[i], items & 1, abort_flag, a.err))
                    return false;
                // (the item's accumulator is complete only after the first half has been
                // through its previous finish(): its word of that item has been read)
                if (half) {
                    sm->dw[i][r] = old_dw;
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(&sm->dw_full[i]);
                } else if (!warp_mbar_wait_short(&sm->dw_full[i], items & 1, abort_flag, a.err)) {
                    return false;
                }
                ++items;
                pending = false;
                tc_fence_after();
                if (!half && old_row != kNone)
                    a.dw[old_row] = old_dw + sm->dw[i][r];
                // 16 values of the warp's 32 rows at a time, through shared memory: two
                // lanes store one row's 32 bytes, not 32 lanes 16 bytes of 32 rows
                uint4 *dst[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const uint32_t to = __shfl_sync(0xffffffffu, old_row, e * 16 + (lane >> 1));
                    dst[e] = to == kNone ? nullptr
                                         : reinterpret_cast<uint4 *>(a.dq + (int64_t)to * D + half * (D / 2)) + (lane & 1);
                }
                uint4 *put0 = out + lane * 2 + ((lane >> 2) & 1), *put1 = out + lane * 2 + (((lane >> 2) & 1) ^ 1);
                const int l0 = lane >> 1, u = (lane & 1) ^ ((l0 >> 2) & 1);
                const uint4 *get0 = out + l0 * 2 + u, *get1 = get0 + 32;
                constexpr int kCh = D / 2 / 16;          // 16-column pieces
                uint32_t v[2][16];
                tmem_ld16(ta, v[0]);
#pragma unroll
                for (int k = 0; k < kCh; ++k) {
                    tmem_ld_wait();
                    if (k + 1 < kCh)
                        tmem_ld16(ta + (k + 1) * 16, v[(k + 1) & 1]);
                    uint32_t o[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const __nv_bfloat162 y = __floats2bfloat162_rn(__uint_as_float(v[k & 1][2 * e]) * old_wq,
                                                                       __uint_as_float(v[k & 1][2 * e + 1]) * old_wq);
                        o[e] = *reinterpret_cast<const uint32_t *>(&y);
                    }
                    __syncwarp();
                    *put0 = make_uint4(o[0], o[1], o[2], o[3]);
                    *put1 = make_uint4(o[4], o[5], o[6], o[7]);
                    __syncwarp();
                    const uint4 r0 = *get0, r1 = *get1;
                    if (dst[0])
                        dst[0][k * 2] = r0;
                    if (dst[1])
                        dst[1][k * 2] = r1;
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&sm->acc_empty[i]);
                return true;
            };
            bool go = wk.begin(a, p), ok = true;
            while (go) {
                if (wk.first) {
                    const int t = wk.a0 + i * TT + tt;
                    row = t < a.S && h < a.H ? (uint32_t)(((int64_t)wk.b * a.S + t) * a.H + h) : kNone;
                    const float f = row != kNone ? __ldg(&p.row[(int64_t)wk.b * a.S + t].x) : 0.f;
                    any = f != 0.f;
                    const float inv = any ? inverse_pow2(f) : 0.f;
                    wq = row != kNone ? __ldg(a.w + row) * inv : 0.f;
                    qs = row != kNone ? __ldg(a.q_scale + row) * inv : 0.f;
                }
                const bool closes = wk.last();
                go = wk.next(a, p);
                if (!warp_mbar_wait_both(&sm->g_full[n & 1], (n >> 1) & 1, &sm->s_full[i][half], n & 1, abort_flag,
                                         a.err)) {
                    ok = false;
                    break;
                }
                pass_on(n);
                tc_fence_after();
                const float *gk = sg + ((n & 1) * 2 * TT + i * TT + tt) * kBwRow + half * 64;
                uint32_t x[2][16];
                tmem_ld16(ts, x[0]);
#pragma unroll
                for (int c = 0; c < 64; c += 16) {
                    const uint32_t(&v)[16] = x[(c / 16) & 1];
                    tmem_ld_wait();
                    if (c + 16 < 64)
                        tmem_ld16(ts + c + 16, x[(c / 16 + 1) & 1]);
                    uint32_t m[8];
#pragma unroll
                    for (int e = 0; e < 16; e += 4) {
                        const float4 w = *reinterpret_cast<const float4 *>(gk + c + e);
                        // relu and conversion in one: max(x + M, M), M the bits of 2^23
                        float y[4];
#pragma unroll
                        for (int u = 0; u < 4; ++u)
                            y[u] = __int_as_float(__viaddmax_s32((int)v[e + u], 0x4B000000, 0x4B000000));
                        const uint64_t y01 = add2(pack2(y[0], y[1]), pack2(-8388608.f, -8388608.f));
                        const uint64_t y23 = add2(pack2(y[2], y[3]), pack2(-8388608.f, -8388608.f));
                        dw[0] = fma2(y01, pack2(w.x, w.y), dw[0]);
                        dw[1] = fma2(y23, pack2(w.z, w.w), dw[1]);
                        unpack2(y01, y[0], y[1]);
                        unpack2(y23, y[2], y[3]);
                        // M = m gk, m = min(y, 1) (y is 0 or at least 1)
                        const __half2 one = __half2half2(__ushort_as_half(0x3C00));
                        const __half2 m01 = __hmul2(__floats2half2_rn(w.x, w.y),
                                                    __hmul2_sat(__floats2half2_rn(y[0], y[1]), one));
                        const __half2 m23 = __hmul2(__floats2half2_rn(w.z, w.w),
                                                    __hmul2_sat(__floats2half2_rn(y[2], y[3]), one));
                        m[e / 2] = *reinterpret_cast<const uint32_t *>(&m01);
                        m[e / 2 + 1] = *reinterpret_cast<const uint32_t *>(&m23);
                    }
                    tmem_st8(ts + c / 2, m);            // these columns have been read
                }
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&sm->g_empty[n & 1]);
                if (pending && !finish()) {
                    ok = false;
                    break;
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&sm->m_full[i][half][n & 1]);
                ++n;
                if (closes) {
                    pending = true;
                    old_row = row;
                    old_wq = any ? wq : 0.f;     // (without a gradient the accumulator is 0, and stays 0)
                    float d0, d1;
                    unpack2(add2(dw[0], dw[1]), d0, d1);
                    old_dw = any ? (d0 + d1) * qs : 0.f;
                    dw[0] = dw[1] = 0u;
                }
            }
            if (pending && ok)
                ok = finish();
            if (!ok && lane == 0)
                *p.gave_up = 1u;
        } else {
            // this key's gradients of the tokens of the warp's columns, read a step
            // ahead; lane e holds token e's power of two for its weights and its candidates,
            // [0, hi) kept up by counting
            constexpr int NT = HP > 64 ? 1 : TT / 2;    // tokens of 64 columns
            const int e0 = HP > 64 ? 0 : half * NT;
            float raw[NT], u_tok = 0.f, f = 0.f;        // f: the key's scale
            int lo = 0, hi = 0, rem = 0;
            const int up = TT / a.cr, up_rem = TT - up * a.cr;
            auto fetch = [&]() {
                const int j = wk.a0 + i * 128 + r;
                const int t = wk.s * TT + lane;
                if (wk.first) {
                    uint32_t most = 0u;
#pragma unroll
                    for (int e = 0; e < kKeyGroups; ++e)
                        if (j < a.P)
                            most = max(most, __ldg(p.key + ((int64_t)e * a.B + wk.b) * a.P + j));
                    f = key_scale(most);
                    const uint32_t ends = (uint32_t)a.t_begin + (uint32_t)t + 1u;
                    hi = (int)(ends / (uint32_t)a.cr);
                    rem = (int)(ends - (uint32_t)hi * (uint32_t)a.cr);
                } else {
                    hi += up;
                    rem += up_rem;
                    if (rem >= a.cr) {
                        rem -= a.cr;
                        ++hi;
                    }
                }
                const float *src = p.G + ((int64_t)wk.b * a.S + wk.s * TT + e0) * a.P + j;
                const int end = t < a.S ? min(a.P, hi) : 0;
                u_tok = lane < TT && t < a.S ? __ldg(&p.row[(int64_t)wk.b * a.S + t].y) : 0.f;
                if (a.doc_start) {
                    int l, u;
                    lo = 0;
                    if (lane < TT && t < a.S) {
                        token_range(a, wk.b, t, l, u);
                        lo = l;
                    }
                }
#pragma unroll
                for (int e = 0; e < NT; ++e, src += a.P) {
                    const int u = __shfl_sync(0xffffffffu, end, e0 + e), l = __shfl_sync(0xffffffffu, lo, e0 + e);
                    raw[e] = j >= l && j < u ? __ldg(src) : 0.f;
                }
            };
            bool go = wk.begin(a, p), ok = true;
            if (go)
                fetch();
            while (go) {
                uint32_t g[NT];
#pragma unroll
                for (int e = 0; e < NT; ++e)
                    g[e] = __half_as_ushort(__float2half_rn(raw[e] * __shfl_sync(0xffffffffu, u_tok, e0 + e) * f));
                const float inv = inverse_pow2(f);
                const int pair = wk.pair;
                const bool closes = wk.last();
                go = wk.next(a, p);
                if (go)
                    fetch();
                ok = warp_mbar_wait_short(&sm->s_full[i][half], n & 1, abort_flag, a.err);
                if (!ok)
                    break;
                pass_on(n);
                tc_fence_after();
                // 16 columns at a time; the next 16 are loaded while these are masked
                uint32_t x[2][16];
                tmem_ld16(ts, x[0]);
#pragma unroll
                for (int c = 0; c < 64; c += 16) {
                    const uint32_t(&v)[16] = x[(c / 16) & 1];
                    tmem_ld_wait();
                    if (c + 16 < 64)
                        tmem_ld16(ts + c + 16, x[(c / 16 + 1) & 1]);
                    uint32_t m[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        // (1 or 0, 1 or 0) times the token's 16 bits
                        const uint32_t on = (uint32_t)__vimin_s32_relu((int)v[2 * e], 1) +
                                            ((uint32_t)__vimin_s32_relu((int)v[2 * e + 1], 1) << 16);
                        m[e] = on * g[HP > 64 ? 0 : (c + 2 * e) / HP];
                    }
                    tmem_st8(ts + c / 2, m);            // these columns have been read
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&sm->m_full[i][half][n & 1]);
                ++n;
                if (closes) {
                    ok = warp_mbar_wait_short(&sm->acc_full[i], items & 1, abort_flag, a.err);
                    if (!ok)
                        break;
                    ++items;
                    tc_fence_after();
                    // segment of pair `pair` in this CTA's share: both count up, their sum names it
                    float *o = p.part + ((int64_t)((int)blockIdx.x + pair) * 256 + i * 128 + r) * D + half * (D / 2);
#pragma unroll
                    for (int c = 0; c < D / 2; c += 16) {
                        uint32_t v[16];
                        tmem_ld16(ta + c, v);
                        tmem_ld_wait();
#pragma unroll
                        for (int e = 0; e < 16; e += 4)
                            *reinterpret_cast<float4 *>(o + c + e) =
                                make_float4(__uint_as_float(v[e]) * 0x1p-8f * inv, __uint_as_float(v[e + 1]) * 0x1p-8f * inv,
                                            __uint_as_float(v[e + 2]) * 0x1p-8f * inv,
                                            __uint_as_float(v[e + 3]) * 0x1p-8f * inv);
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(&sm->acc_empty[i]);
                }
            }
            if (!ok && lane == 0)
                *p.gave_up = 1u;
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// dk: the partial sums of a pair's segments, added in a fixed order. One block a
// key; the segments are cut into 1024 / D runs of neighbours, whose sums are
// added in order, so that the loads of a long list are in flight together.
__global__ void __launch_bounds__(256) bwd_reduce_kernel(const ScoresBwdArgs a, const BwPlan p)
{
    __shared__ float4 run[256];
    const bool gave_up = __ldg(p.gave_up) != 0u;
    const int b = (int)(blockIdx.x / (unsigned)a.P), j = (int)(blockIdx.x - (unsigned)b * (unsigned)a.P);
    const int kp = j >> 8, pair = b * p.n_pairs + kp;
    const int per_row = a.D / 4, runs = 256 / per_row;
    const int c = (threadIdx.x % per_row) * 4, me = threadIdx.x / per_row;
    int begin = p.per_seq * b;
    for (int k = 0; k < kp; ++k)
        begin += p.n_steps_seq - first_step(a, p, k);
    const int end = begin + p.n_steps_seq - first_step(a, p, kp);
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (begin < end) {
        // the shares that hold steps `begin` and `end - 1`
        const int longer = p.rest * (p.share + 1);
        auto share_of = [&](int at) {
            return at < longer ? at / (p.share + 1) : p.rest + (at - longer) / p.share;
        };
        const int x0 = share_of(begin), n = share_of(end - 1) - x0 + 1;
        const float *src = p.part + ((int64_t)(x0 + pair) * 256 + (j & 255)) * a.D + c;
        const int per = (n + runs - 1) / runs;
        const int i1 = min(n, (me + 1) * per);
#pragma unroll 4
        for (int i = me * per; i < i1; ++i) {
            const float4 v = *reinterpret_cast<const float4 *>(src + (int64_t)i * 256 * a.D);
            s.x += v.x;
            s.y += v.y;
            s.z += v.z;
            s.w += v.w;
        }
    }
    // a wait gave up, so that rows and partial sums are missing: no output is given out
    if (gave_up) {
        const int64_t rows = (int64_t)a.B * a.S * a.H, step = (int64_t)gridDim.x * blockDim.x;
        for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < rows; i += step) {
            a.dw[i] = __int_as_float(0x7fc00000);
            for (int c = 0; c < a.D / 8; ++c)
                reinterpret_cast<uint4 *>(a.dq + i * a.D)[c] = make_uint4(0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u);
        }
    }
    run[threadIdx.x] = s;
    __syncthreads();
    if (me)
        return;
    for (int i = 1; i < runs; ++i) {
        const float4 v = run[i * per_row + threadIdx.x];
        s.x += v.x;
        s.y += v.y;
        s.z += v.z;
        s.w += v.w;
    }
    if (gave_up)
        s.x = s.y = s.z = s.w = __int_as_float(0x7fc00000);
    const __nv_bfloat162 lo = __floats2bfloat162_rn(s.x, s.y), hi = __floats2bfloat162_rn(s.z, s.w);
    *reinterpret_cast<uint2 *>(a.dk + (int64_t)blockIdx.x * a.D + c) =
        make_uint2(*reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi));
}

size_t up16(size_t n) { return (n + 15) & ~size_t(15); }

// fp16 rows [B][P][D], 128 rows a box, in blocks of their swizzle span.
bool make_map_f16(CUtensorMap *m, const void *ptr, int D, int P, int B)
{
    PFN_cuTensorMapEncodeTiled_v12000 enc = encode_fn();
    if (!enc)
        return false;
    cuuint64_t gdim[3] = {(cuuint64_t)D, (cuuint64_t)P, (cuuint64_t)B};
    cuuint64_t gstride[2] = {(cuuint64_t)D * 2, (cuuint64_t)D * 2 * P};
    cuuint32_t box[3] = {(cuuint32_t)(D < 64 ? D : 64), 128, 1};
    cuuint32_t estride[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void *>(ptr), gdim, gstride, box, estride,
               CU_TENSOR_MAP_INTERLEAVE_NONE, D < 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int HP>
cudaError_t run_bwd(const ScoresBwdArgs &a, const void *k16, const BwPlan &pq, const BwPlan &pk, int grid_q, int grid_k,
                    cudaStream_t st)
{
    CUtensorMap rows, keys, keys16;    // query rows (HP heads of TT tokens) and keys, 128 rows a box
    if (!make_map_f16(&keys16, k16, D, a.P, a.B) ||
        !make_map_q8(&rows, a.q8, D, a.H, (uint64_t)a.B * a.S, HP, 128 / HP) ||
        !make_map_q8(&keys, a.k8, D, a.P, a.B, 128, 1))
        return cudaErrorUnknown;
    cudaError_t e = cudaFuncSetAttribute(bwd_tc_kernel<0, D, HP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)bw_smem_bytes<D>(true, HP));
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(bwd_tc_kernel<1, D, HP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)bw_smem_bytes<D>(false, HP));
    if (e != cudaSuccess)
        return e;
    bwd_tc_kernel<0, D, HP><<<grid_q, bw_threads(true), bw_smem_bytes<D>(true, HP), st>>>(rows, keys, keys16, a, pq);
    if (grid_k > 0)
        bwd_tc_kernel<1, D, HP><<<grid_k, bw_threads(false), bw_smem_bytes<D>(false, HP), st>>>(keys, rows, keys16, a, pk);
    bwd_reduce_kernel<<<(unsigned)(a.B * a.P), 256, 0, st>>>(a, pk);
    return cudaGetLastError();
}

template <int D>
cudaError_t run_bwd_heads(int hp, const ScoresBwdArgs &a, const void *k16, const BwPlan &pq, const BwPlan &pk, int grid_q, int grid_k,
                          cudaStream_t st)
{
    switch (hp) {
    case 8: return run_bwd<D, 8>(a, k16, pq, pk, grid_q, grid_k, st);
    case 16: return run_bwd<D, 16>(a, k16, pq, pk, grid_q, grid_k, st);
    case 32: return run_bwd<D, 32>(a, k16, pq, pk, grid_q, grid_k, st);
    case 64: return run_bwd<D, 64>(a, k16, pq, pk, grid_q, grid_k, st);
    default: return run_bwd<D, 128>(a, k16, pq, pk, grid_q, grid_k, st);
    }
}

// CTAs of the dk kernel: no more than there are steps if every pair saw every
// token tile.
int dk_shares(int B, int S, int H, int P)
{
    const int tt = 128 / padded_heads(H);
    const long long most = (long long)B * ((P + 255) / 256) * ((S + tt - 1) / tt);
    const int sms = sm_count();
    return (int)(most < sms ? most : sms);
}

}  // namespace

// Workspace: four words (the first: a wait gave up), each key's largest magnitude, two
// words a token, dk's partial sums, the keys in fp16, and G.
constexpr size_t kStatusBytes = 16;
size_t indexer_scores_bwd_ws_bytes(int B, int S, int H, int D, int P)
{
    const size_t slots = (size_t)dk_shares(B, S, H, P) + (size_t)B * ((P + 255) / 256);
    return kStatusBytes + up16((size_t)kKeyGroups * B * P * 4) + up16((size_t)B * S * 8) + slots * 256 * D * 4 + (size_t)B * P * D * 2 + (size_t)B * S * P * 4;
}

cudaError_t launch_indexer_scores_bwd(const ScoresBwdArgs &a, void *ws, cudaStream_t stream)
{
    const int sms = sm_count();
    if (sms <= 0)
        return cudaErrorUnknown;
    const int hp = padded_heads(a.H);
    const int tt = 128 / hp;
    int shares = dk_shares(a.B, a.S, a.H, a.P);
    uint8_t *w = static_cast<uint8_t *>(ws);
    uint32_t *gave_up = reinterpret_cast<uint32_t *>(w);
    uint32_t *key_max = reinterpret_cast<uint32_t *>(w + kStatusBytes);
    const size_t key_bytes = kStatusBytes + up16((size_t)kKeyGroups * a.B * a.P * 4);
    float2 *row_scale = reinterpret_cast<float2 *>(w + key_bytes);
    float *part = reinterpret_cast<float *>(w + key_bytes + up16((size_t)a.B * a.S * 8));
    BwPlan pk;
    pk.tt_log = 0;
    while ((1 << pk.tt_log) < tt)
        ++pk.tt_log;
    pk.n_steps_seq = (a.S + tt - 1) / tt;
    pk.n_pairs = (a.P + 255) / 256;
    uint4 *k16 = reinterpret_cast<uint4 *>(part + ((size_t)shares + (size_t)a.B * pk.n_pairs) * 256 * a.D);
    float *G = reinterpret_cast<float *>(reinterpret_cast<uint8_t *>(k16) + (size_t)a.B * a.P * a.D * 2);
    pk.G = a.idx ? G : a.dscores;
    pk.key = key_max;
    pk.gave_up = gave_up;
    pk.row = row_scale;
    pk.part = part;
    long long per_seq = 0;
    for (int kp = 0; kp < pk.n_pairs; ++kp) {
        const long long t = (256LL * kp + 1) * a.cr - 1 - a.t_begin;
        const long long f = t <= 0 ? 0 : t / tt;
        per_seq += pk.n_steps_seq - (f < pk.n_steps_seq ? f : pk.n_steps_seq);
    }
    const long long total = per_seq * a.B;       // fits 31 bits (checked on the host)
    if (total < shares)
        shares = (int)total;                     // no empty share
    pk.per_seq = (int)per_seq;
    pk.share = shares ? (int)(total / shares) : 0;
    pk.rest = shares ? (int)(total % shares) : 0;
    BwPlan pq = pk;
    pq.n_pairs = (a.S + 2 * tt - 1) / (2 * tt);
    const long long items = (long long)a.B * pq.n_pairs;
    const int grid_q = (int)(items < sms ? items : sms);
    cudaError_t e = cudaMemsetAsync(w, 0, key_bytes, stream);
    if (e != cudaSuccess)
        return e;
    // rows of idx, dscores, G and k_scale on 16-byte boundaries
    const bool vec = a.idx && a.K % 4 == 0 && a.P % 4 == 0 && al16(a.idx) && al16(a.dscores) && al16(a.k_scale);
    const int cols = a.idx ? (a.P < kPrepCols ? (a.P + 31) / 32 * 32 : kPrepCols) : 32;
    const int64_t key_blocks = ((int64_t)a.B * a.P * (a.D / 16) + kPrepThreads - 1) / kPrepThreads;
    bwd_prep_kernel<<<(unsigned)((int64_t)a.B * a.S + key_blocks), kPrepThreads, (size_t)cols * 4 + cols / 8, stream>>>(
        a, G, key_max, row_scale, k16, vec, cols);
    if (a.D == 32)
        return run_bwd_heads<32>(hp, a, k16, pq, pk, grid_q, shares, stream);
    if (a.D == 64)
        return run_bwd_heads<64>(hp, a, k16, pq, pk, grid_q, shares, stream);
    return run_bwd_heads<128>(hp, a, k16, pq, pk, grid_q, shares, stream);
}

}  // namespace sai
