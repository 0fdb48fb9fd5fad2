// The lightning indexer's scores from 8-bit queries and 8-bit cached keys on
// tcgen05 tensor cores (sm_100a):
//
//   s[b,t,j] = ks[b,j] * sum_h w[b,t,h] qs[b,t,h] relu(<q8[b,t,h,:], k8[b,j,:]>)
//
// for the candidates j of token t, -inf elsewhere. (Scales are not negative,
// so they leave relu's argument's sign alone.)
//
// The products of the codes are whole numbers below 2^22, exact in the tensor
// core's 32-bit integer accumulator and in fp32; the sum over heads is fp32.
//
// Tile: A = 128 keys (the accumulator's lanes), B = TT tokens x HP heads (up to
// 256 columns; HP is H rounded up to a power of two, the heads above H are
// zero-filled by the TMA box). With the keys on the lanes the sum over heads is
// a sum along each thread's own row, without shuffles, and a warp's 32 scores
// of one token are 32 consecutive outputs.
//
// Bound: the epilogue. A 128 x 256 tile of D = 128 is 512 cycles of MMA, but its
// 32,768 products each take an integer instruction (relu and conversion in one)
// and half of a packed subtraction and of a packed fma: about 800 cycles with the
// tensor-memory loads on the four schedulers (measured alone); 0.41 ms at S = 16384
// are about 1,800 cycles a tile, the rest of which is the chain of a tile's loads,
// barriers and hand-overs. Taken from there: the column weights are held in registers
// over an item's tiles (as broadcasts from shared memory they fill 1,024 cycles a
// tile with register bytes: 0.56 ms against 0.46 when that was tried), and a tile's two
// barriers are tested together. At few tokens a sequence a tile has few columns, and
// the producers' instructions and the keys' arrival bind.
//
// One CTA per SM walks work items (sequence, TT tokens, a range of key tiles).
// Warp roles (384 threads): warp 0 brings key tiles into a ring (TMA; a tile of
// a paged cache page by page) with their scales (bulk copies, or cp.async where
// rows have no 16-byte boundary, completing on the same barrier), warp 1 issues the
// MMAs, warps 2 and 3 prepare alternate items ahead of the others (bounds, query
// tile by TMA, the columns' weights) and fill their outputs that have no candidate
// with -inf (where the keys are split, warp 2 prepares every item and warp 3 brings
// every other key tile), warps 4..7 and 8..11 are
// two epilogue groups taking alternate tiles, each with its own 256-column
// accumulator. Nothing in the epilogue waits for global memory: at one 0.3 us
// tile every load there would cost more than the tile. Tiles without a
// candidate are never multiplied. Every wait is bounded; on timeout the kernel
// records SAI_ERR_TIMEOUT and unwinds, and what its CTA had not written is NaN.
#include <math.h>

#include "indexer_q8.h"
#include "sai_device.cuh"
#include "sai_host.h"

namespace sai {
namespace {

constexpr int kScEpiWarps = 8;
constexpr int kScThreads = 128 + 32 * kScEpiWarps;
constexpr int kScCols = 256;        // accumulator columns of a tile, at most
constexpr int kScMaxTok = 32;       // tokens a tile (HP = 8)
constexpr int kScRing = 6;          // key tiles in flight (even: each belongs to one of two producers)
static_assert(kScRing % 2 == 0, "a stage belongs to one producer");
constexpr int kScItems = 3;         // items prepared ahead (a query tile each)

struct ScPlan {
    int tt;             // tokens a tile
    int n_tt;           // token tiles a sequence
    int n_kt;           // key tiles a sequence
    int chunk;          // key tiles an item
    int producers;      // warps that bring key tiles: 1, or 2 (of alternate tiles)
    int n_items;
    int groups;         // epilogue groups a tile (128 columns each)
    int box_rows;       // rows of a key load
    int loads;          // loads a key tile
    int bulk;           // scales come in whole 16-byte pieces (else word by word)
};

// One item: TT tokens of a sequence and the key tiles [c_lo, c_hi); those in
// [k_lo, k_hi) hold a candidate of at least one of the tokens.
struct ScItem {
    int b, t0, ntok;
    int c_lo, c_hi, k_lo, k_hi;
    int n_keys;                     // entries the sequence's cache holds, at most P
    int jlo[kScMaxTok], jhi[kScMaxTok];   // each token's candidates
    alignas(16) float ww[kScCols];  // w * q_scale of each column
};

struct ScSmem {
    ScItem item[kScItems];
    alignas(16) float ks[kScRing][128];   // scales of a key tile
    uint32_t have[kScRing];         // which of its loads exist
    uint64_t i_full[kScItems], i_empty[kScItems];   // the item and its query tile
    uint64_t k_full[kScRing], k_empty[kScRing];
    uint64_t acc_full[4], acc_empty[4];
    uint64_t drain;
    uint32_t tmem_base;
    int abort_flag;
};

// Readers of an item's slot, beside the key producers: the MMA's completion and the
// epilogue warps.
constexpr int kScItemReaders = 1 + kScEpiWarps;

// Adds the products of four accumulator words and their weights to four partial
// sums; where a token ends, hands the sums over and clears them.
template <class End>
__device__ __forceinline__ void add_heads(const uint32_t *x, uint64_t w0, uint64_t w1, uint64_t (&s)[2], bool ends,
                                          End end)
{
    // max(x + M, M) with M the bits of 2^23 is the fp32 number 2^23 + relu(x), and
    // 2^23 comes off exactly
    constexpr int M = 0x4B000000;
    const uint64_t off = pack2(-8388608.f, -8388608.f);
    float y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        y[i] = __int_as_float(__viaddmax_s32((int)x[i], M, M));
    s[0] = fma2(add2(pack2(y[0], y[1]), off), w0, s[0]);
    s[1] = fma2(add2(pack2(y[2], y[3]), off), w1, s[1]);
    if (ends) {
        float a, b;
        unpack2(add2(s[0], s[1]), a, b);
        end(a + b);
        s[0] = s[1] = 0u;
    }
}

template <int D, int HP>
__global__ void __launch_bounds__(kScThreads, 1)
    scores_tc_kernel(const __grid_constant__ CUtensorMap mapQ, const __grid_constant__ CUtensorMap mapK,
                     const ScoresArgs a, const ScPlan p)
{
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    constexpr uint32_t q_bytes = kScCols * D, k_bytes = 128 * D;
    uint8_t *sq = base, *sk = base + kScItems * q_bytes;
    ScSmem *sm = reinterpret_cast<ScSmem *>(sk + kScRing * k_bytes);
    const int warp = uniform_warp();
    const int lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kScItems; ++i) {
            mbar_init(&sm->i_full[i], 1);
            mbar_init(&sm->i_empty[i], kScItemReaders + p.producers);
        }
        for (int s = 0; s < kScRing; ++s) {
            mbar_init(&sm->k_full[s], p.bulk ? 1 : 1 + 32);   // the tile's bytes; each lane's scales
            mbar_init(&sm->k_empty[s], 4 * p.groups);  // the tile's epilogue warps: its products are done then
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(&sm->acc_full[i], 1);
            mbar_init(&sm->acc_empty[i], 4 * p.groups);
        }
        mbar_init(&sm->drain, 1);
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
    const uint32_t tmem = sm->tmem_base;
    volatile int *abort_flag = &sm->abort_flag;
    const int cols = p.tt * HP;
    // accumulators in turn: two of 256 columns, or four of 128
    const int acc_log = cols > 128 ? 1 : 2;
    const uint32_t acc_cols = 512u >> acc_log;
    // One item of every gridDim.x. Whole token tiles come longest first and are taken
    // there and back: the CTA with the longest of one round takes the shortest of the
    // next (always from the same end, the first CTA had 35 key tiles at S = 4096 where
    // the mean is 31: 40.9 us against 39.0). Split ones have no such order (a decoding
    // batch takes 36.1 us as it is, 37.2 there and back).
    const int rounds = p.n_items / (int)gridDim.x, back = p.chunk == p.n_kt;
    auto item_of = [&](int n) {
        return n * (int)gridDim.x + ((n & back) ? (int)gridDim.x - 1 - (int)blockIdx.x : (int)blockIdx.x);
    };
    const int n_mine = rounds + (item_of(rounds) < p.n_items ? 1 : 0);
    // An item's chunk of key tiles, sequence and first token: chunks outermost, later
    // tokens (more candidates) first, so that the items of one CTA are spread over
    // tokens, sequences and chunks.
    auto place_of = [&](int n, int &c, int &b, int &t0) {
        const int i = item_of(n), tiles = a.B * p.n_tt;
        c = i / tiles;
        b = (i - c * tiles) % a.B;
        t0 = (p.n_tt - 1 - (i - c * tiles) / a.B) * p.tt;
    };

    if (warp < 4) {
    regs_dec<80>();
    if (warp == 0 || (warp == 3 && p.producers == 2)) {
        // ------------------------------------------------ key producer(s)
        if (lane == 0)
            tma_prefetch_desc(&mapK);
        const int mine = warp ? 1 : 0, step = p.producers;
        int stage = mine, slot = 0, n_tiles = 0;
        uint32_t phase = 0, iphase = 0, k_used = 0, k_parity = 0;
        bool ok = true;
        // tile row i*32 + lane comes with load from[i], as its row off[i] (several loads a tile)
        int from[4], off[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            from[i] = min((i * 32 + lane) / p.box_rows, 31);
            off[i] = i * 32 + lane - from[i] * p.box_rows;
        }
        for (int n = 0; n < n_mine && ok; ++n) {
            if (!warp_mbar_wait_short(&sm->i_full[slot], iphase, abort_flag, a.err)) {
                ok = false;
                break;
            }
            const ScItem &it = sm->item[slot];
            const int b = it.b, k_lo = it.k_lo, k_hi = it.k_hi, n_keys = it.n_keys;
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&sm->i_empty[slot]);
            if (++slot == kScItems) {
                slot = 0;
                iphase ^= 1u;
            }
            // The pages of 32 / loads tiles at a time, one a lane, read from the table a
            // batch ahead (read tile by tile, the table's latency bound a paged walk)
            const int per = 32 / p.loads, sub = lane % p.loads;
            int ahead = -1, ahead_row = 0, batch = -1, batch_row = 0;
            auto find = [&](int kb) {
                const int k = kb + step * (lane / p.loads), j0 = k * 128 + sub * p.box_rows;
                ahead = -1;
                ahead_row = 0;
                if (k >= k_hi || j0 >= n_keys || lane >= per * p.loads)
                    return;
                ahead = b;
                ahead_row = j0;
                if (a.map.table) {
                    const uint32_t pi = (uint32_t)j0 / (uint32_t)a.map.page;
                    ahead_row = j0 - (int)pi * a.map.page;
                    ahead = __ldg(a.map.table + (int64_t)b * a.map.max_pages + pi);
                }
            };
            // (of two producers each takes every other tile of all items' tiles)
            const int first_k = k_lo + ((n_tiles ^ mine) & (step - 1));
            n_tiles += k_hi - k_lo;
            find(first_k);
            int in = per;                             // tile within the batch
            for (int k = first_k; k < k_hi; k += step) {
                if (in == per) {
                    batch = ahead;
                    batch_row = ahead_row;
                    find(k + step * per);
                    in = 0;
                }
                const int at = in * p.loads + (lane < p.loads ? lane : 0);
                int page = __shfl_sync(0xffffffffu, batch, at);
                const int row = __shfl_sync(0xffffffffu, batch_row, at);
                ++in;
                if (lane >= p.loads || page >= a.map.n_pages)     // the epilogue reports pages outside the cache
                    page = -1;
                const uint32_t have = __ballot_sync(0xffffffffu, page >= 0);
                if (!warp_mbar_wait_short(&sm->k_empty[stage], phase ^ 1u, abort_flag, a.err)) {
                    ok = false;
                    break;
                }
                const float *first = a.k_scale + (int64_t)page * a.map.page + row;   // scale of this load's first row
                uint32_t bytes = page >= 0 ? (uint32_t)(p.box_rows * D) : 0u, sbytes = 0;
                if (p.bulk && page >= 0)
                    sbytes = (uint32_t)min(p.box_rows, a.map.page - row) * 4u;
                const uint32_t total = __reduce_add_sync(0xffffffffu, bytes + sbytes);
                if (lane == 0) {
                    sm->have[stage] = have;
                    mbar_arrive_expect_tx(&sm->k_full[stage], total);
                }
                __syncwarp();
                if (page >= 0) {
                    tma_load_3d(sk + stage * k_bytes + lane * p.box_rows * D, &mapK, &sm->k_full[stage], 0, row,
                                page);
                    if (p.bulk)
                        bulk_load(smem_u32(&sm->ks[stage][lane * p.box_rows]), first, sbytes, &sm->k_full[stage]);
                }
                __syncwarp();
                if (!p.bulk) {
                    const uint32_t to = smem_u32(&sm->ks[stage][lane]);
                    const int left = n_keys - k * 128;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float *f = reinterpret_cast<const float *>(
                            __shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(first), from[i]));
                        if (((have >> from[i]) & 1u) && i * 32 + lane < left)
                            cp_async4(to + i * 128, f + off[i]);
                    }
                    cp_async_arrive(&sm->k_full[stage]);
                }
                k_used |= 1u << stage;
                k_parity = (k_parity & ~(1u << stage)) | (phase << stage);
                if ((stage += step) >= kScRing) {
                    stage = mine;
                    phase ^= 1u;
                }
            }
        }
        if (!ok && lane == 0) {
            // let the copies in flight land before the CTA goes
            for (int s = 0; s < kScRing; ++s)
                if (k_used & (1u << s))
                    mbar_drain(&sm->k_full[s], (k_parity >> s) & 1u);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------ MMA issuer
        const uint32_t idesc = idesc_i8_s32(128, cols);
        const uint64_t q_desc = sdesc_k_rows<D>(smem_u32(sq)), k_desc = sdesc_k_rows<D>(smem_u32(sk));
        int stage = 0, slot = 0, n_tiles = 0;
        uint32_t phase = 0, iphase = 0;
        bool ok = true, issued = false;
        for (int n = 0; n < n_mine && ok; ++n) {
            if (!warp_mbar_wait_short(&sm->i_full[slot], iphase, abort_flag, a.err)) {
                ok = false;
                break;
            }
            const int n_live = sm->item[slot].k_hi - sm->item[slot].k_lo;
            const uint64_t db = q_desc + slot * (q_bytes / 16);
            for (int k = 0; k < n_live; ++k, ++n_tiles) {
                const int buf = n_tiles & ((1 << acc_log) - 1);
                if (!warp_mbar_wait_short(&sm->acc_empty[buf], ((n_tiles >> acc_log) & 1) ^ 1u, abort_flag, a.err) ||
                    !warp_mbar_wait_short(&sm->k_full[stage], phase, abort_flag, a.err)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint64_t da = k_desc + stage * (k_bytes / 16);
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < D / 32; ++kk)
                        umma_i8(tmem + buf * acc_cols, da + 2 * kk, db + 2 * kk, idesc, kk != 0);
                    umma_commit(&sm->acc_full[buf]);
                }
                issued = true;
                __syncwarp();
                if (++stage == kScRing) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
            if (!ok)
                break;
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&sm->i_empty[slot]);
            if (++slot == kScItems) {
                slot = 0;
                iphase ^= 1u;
            }
        }
        if (!ok && lane == 0 && issued) {
            umma_commit(&sm->drain);
            mbar_drain(&sm->drain, 0);
        }
        __syncwarp();
    } else {
        // ------------------------------------------------ items ahead
        if (lane == 0)
            tma_prefetch_desc(&mapQ);
        uint32_t q_used = 0, q_parity = 0;
        bool ok = true;
        for (int n = warp - 2; n < n_mine && ok; n += 3 - p.producers) {
            const int slot = n % kScItems;
            const uint32_t iphase = (uint32_t)(n / kScItems) & 1u;
            int c, b, t0;
            place_of(n, c, b, t0);
            const int ntok = min(p.tt, a.S - t0);
            const int c_lo = c * p.chunk, c_hi = min(p.n_kt, c_lo + p.chunk);
            const int64_t pos = (int64_t)(a.q_start ? __ldg(a.q_start + b) : 0) + t0 + lane;
            const int n_keys = a.k_len ? max(0, min(a.P, __ldg(a.k_len + b))) : a.P;
            const int64_t row0 = (int64_t)b * a.S + t0;
            float v[kScCols / 32];
#pragma unroll
            for (int e = 0; e < kScCols / 32; ++e) {
                const int col = e * 32 + lane, tt = col / HP, h = col % HP;
                v[e] = 0.f;
                if (col < cols && tt < ntok && h < a.H) {
                    const int64_t r = (row0 + tt) * a.H + h;
                    v[e] = __ldg(a.w + r) * __ldg(a.q_scale + r);
                }
            }
            int lo = 0, hi = 0;
            if (lane < ntok) {
                int64_t d0 = a.doc_start ? (int64_t)__ldg(a.doc_start + row0 + lane) : 0;
                d0 = d0 < 0 ? 0 : (d0 > pos ? pos : d0);
                // P * cr fits 31 bits (checked on the host), so both bounds do after the clamps
                const uint32_t ends = (uint32_t)(pos < 0 ? 0 : (pos + 1 > INT32_MAX ? (int64_t)INT32_MAX : pos + 1));
                hi = min(n_keys, (int)(ends / (uint32_t)a.cr));
                lo = pos < 0 ? 0 : (int)min((int64_t)hi, (d0 + a.cr - 1) / a.cr);
            }
            const bool any = lane < ntok && lo < hi;
            const int jlo = __reduce_min_sync(0xffffffffu, any ? lo : INT32_MAX);
            const int jhi = __reduce_max_sync(0xffffffffu, any ? hi : 0);
            int k_lo = c_lo, k_hi = c_lo;
            if (jhi > 0) {
                k_lo = max(c_lo, jlo >> 7);
                k_hi = min(c_hi, (jhi + 127) >> 7);
                if (k_hi <= k_lo)
                    k_lo = k_hi = c_lo;
            }
            if (!warp_mbar_wait_short(&sm->i_empty[slot], iphase ^ 1u, abort_flag, a.err)) {
                ok = false;
                break;
            }
            ScItem &it = sm->item[slot];
            if (lane == 0) {
                it.b = b;
                it.t0 = t0;
                it.ntok = ntok;
                it.c_lo = c_lo;
                it.c_hi = c_hi;
                it.k_lo = k_lo;
                it.k_hi = k_hi;
                it.n_keys = n_keys;
            }
            it.jlo[lane] = lo;
            it.jhi[lane] = hi;
#pragma unroll
            for (int e = 0; e < kScCols / 32; ++e)
                it.ww[e * 32 + lane] = v[e];
            __syncwarp();
            if (lane == 0) {
                if (k_lo < k_hi) {
                    mbar_arrive_expect_tx(&sm->i_full[slot], (uint32_t)cols * D);
                    tma_load_3d(sq + slot * q_bytes, &mapQ, &sm->i_full[slot], 0, 0, (int)row0);
                    q_used |= 1u << slot;
                    q_parity = (q_parity & ~(1u << slot)) | (iphase << slot);
                } else {
                    mbar_arrive(&sm->i_full[slot]);
                }
            }
            __syncwarp();
            // outputs without a candidate
            const int f0 = c_lo * 128, f1 = k_lo * 128, f2 = min(a.P, k_hi * 128), f3 = min(a.P, c_hi * 128);
            if (f0 < f1 || f2 < f3)
                for (int tt = 0; tt < ntok; ++tt) {
                    float *o = a.out + (row0 + tt) * a.P;
                    for (int j = f0 + lane; j < f1; j += 32)
                        o[j] = -INFINITY;
                    for (int j = f2 + lane; j < f3; j += 32)
                        o[j] = -INFINITY;
                }
        }
        if (!ok && lane == 0) {
            for (int s = 0; s < kScItems; ++s)
                if (q_used & (1u << s))
                    mbar_drain(&sm->i_full[s], (q_parity >> s) & 1u);
        }
        __syncwarp();
    }
    } else {
        // ------------------------------------------------ epilogue
        regs_inc<208>();      // 128 * 80 + 256 * 208 = 63488, of 384 * 168 = 64512
        constexpr int GC = 128;                 // columns of a group
        const int g = (warp - 4) >> 2;
        const int n_par = 2 / p.groups;         // groups of different tiles
        const int cg = g % p.groups, par = g / p.groups;
        const int n_cols = min(cols, GC);
        const int q = warp & 3;                 // TMEM lane quarter of this warp
        const int r = q * 32 + lane;            // tile row: the thread's key
        const int col0 = cg * GC;
        const int my_bit = min(r / p.box_rows, 31);
        constexpr int T = GC / HP;              // tokens of a group
        constexpr bool kRegBounds = T <= 4;     // their bounds are kept in registers
        const uint32_t acc_mask = (1u << acc_log) - 1;
        int n_tiles = 0, slot = 0, n = 0;
        uint32_t iphase = 0;
        bool ok = true;
        for (; n < n_mine; ++n) {
            if (!warp_mbar_wait_short(&sm->i_full[slot], iphase, abort_flag, a.err)) {
                ok = false;
                break;
            }
            const ScItem &it = sm->item[slot];
            const int n_live = it.k_hi - it.k_lo;
            const int nt = it.ntok - cg * T;     // tokens from the group's first on
            const int first = (par - n_tiles) & (n_par - 1);
            // the group's column weights stay in registers over the item's tiles
            // (a broadcast from shared memory costs as many cycles as the
            // register bytes it fills: 1024 a tile, twice the MMA)
            uint64_t w[GC / 2];                  // pairs
            int lo[kRegBounds ? T : 1], hi[kRegBounds ? T : 1], end[kRegBounds ? T : 1];
            if (first < n_live) {
#pragma unroll
                for (int c = 0; c < GC; c += 4) {
                    const ulonglong2 v = *reinterpret_cast<const ulonglong2 *>(it.ww + col0 + c);
                    w[c / 2] = v.x;
                    w[c / 2 + 1] = v.y;
                }
                if (kRegBounds) {
#pragma unroll
                    for (int e = 0; e < T; ++e) {
                        lo[e] = it.jlo[cg * T + e];
                        hi[e] = it.jhi[cg * T + e];
                        end[e] = e < nt ? a.P : 0;
                    }
                }
            }
            int j = (it.k_lo + first) * 128 + r;
            float *o = a.out + ((int64_t)it.b * a.S + it.t0 + cg * T) * a.P + j;
            for (int k = first; k < n_live; k += n_par, j += 128 * n_par, o += 128 * n_par) {
                const uint32_t use = (uint32_t)(n_tiles + k);
                const int stage = (int)(use % kScRing);
                const int buf = (int)(use & acc_mask);
                // (the scales landed before the products were formed: the second test only orders the reads)
                if (!warp_mbar_wait_both(&sm->acc_full[buf], (use >> acc_log) & 1u, &sm->k_full[stage],
                                         (use / kScRing) & 1u, abort_flag, a.err)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t taddr = tmem + buf * acc_cols + col0 + ((uint32_t)(q * 32) << 16);
                // 16 columns at a time; the next 16 are loaded while these are added
                uint32_t x[2][16];
                tmem_ld16(taddr, x[0]);
                const float ks = sm->ks[stage][r];
                const bool there = (sm->have[stage] >> my_bit) & 1u;
                // no branches: one comparison and a predicated store a token
                auto put = [&](int e, float sum) {
                    const int from = kRegBounds ? lo[kRegBounds ? e : 0] : it.jlo[cg * T + e];
                    const int to = kRegBounds ? hi[kRegBounds ? e : 0] : it.jhi[cg * T + e];
                    const float v = (j >= from) & (j < to) & there ? sum * ks : -INFINITY;
                    if (j < (kRegBounds ? end[kRegBounds ? e : 0] : (e < nt ? a.P : 0)))
                        o[(int64_t)e * a.P] = v;
                };
                uint64_t s[2] = {0u, 0u};            // four partial sums
#pragma unroll
                for (int c = 0; c < GC; c += 16) {
                    if (c >= n_cols)
                        break;
                    const uint32_t(&v)[16] = x[(c / 16) & 1];
                    tmem_ld_wait();
                    if (c + 16 < n_cols) {
                        tmem_ld16(taddr + c + 16, x[(c / 16 + 1) & 1]);
                    } else {
                        // the accumulator and the scales are free before the last columns are added
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) {
                            mbar_arrive(&sm->acc_empty[buf]);
                            mbar_arrive(&sm->k_empty[stage]);
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 16; e += 4)
                        add_heads(v + e, w[(c + e) / 2], w[(c + e) / 2 + 1], s, (c + e + 4) % HP == 0,
                                  [&](float sum) { put((c + e) / HP, sum); });
                }
                if (!there && a.err)
                    for (int e = 0; e < min(nt, T); ++e)
                        if (j >= it.jlo[cg * T + e] && j < it.jhi[cg * T + e])
                            atomicExch(a.err, kErrIndex);
            }
            if (!ok)
                break;
            n_tiles += n_live;
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&sm->i_empty[slot]);
            if (++slot == kScItems) {
                slot = 0;
                iphase ^= 1u;
            }
        }
        // A wait gave up: NaN for the item it was for and those behind it. (Another warp
        // may still write a finished tile's scores, or -inf where no candidate is, to them.)
        for (; !ok && n < n_mine; ++n) {
            int c, b, t0;
            place_of(n, c, b, t0);
            const int ntok = min(p.tt, a.S - t0), j1 = min(a.P, min(p.n_kt, (c + 1) * p.chunk) * 128);
            for (int tt = 0; tt < ntok; ++tt)
                for (int j = c * p.chunk * 128 + lane; j < j1; j += 32)
                    a.out[((int64_t)b * a.S + t0 + tt) * a.P + j] = __int_as_float(0x7fc00000);
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <int D>
size_t scores_smem()
{
    return 1024 + kScItems * (size_t)kScCols * D + (size_t)kScRing * 128 * D + sizeof(ScSmem);
}

template <int D, int HP>
cudaError_t run_scores(const CUtensorMap &mq, const CUtensorMap &mk, const ScoresArgs &a, const ScPlan &p, int grid,
                       cudaStream_t st)
{
    const size_t smem = scores_smem<D>();
    cudaError_t e = cudaFuncSetAttribute(scores_tc_kernel<D, HP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)smem);
    if (e != cudaSuccess)
        return e;
    scores_tc_kernel<D, HP><<<grid, kScThreads, smem, st>>>(mq, mk, a, p);
    return cudaGetLastError();
}

template <int D>
cudaError_t run_heads(int hp, const CUtensorMap &mq, const CUtensorMap &mk, const ScoresArgs &a, const ScPlan &p,
                      int grid, cudaStream_t st)
{
    switch (hp) {
    case 8: return run_scores<D, 8>(mq, mk, a, p, grid, st);
    case 16: return run_scores<D, 16>(mq, mk, a, p, grid, st);
    case 32: return run_scores<D, 32>(mq, mk, a, p, grid, st);
    case 64: return run_scores<D, 64>(mq, mk, a, p, grid, st);
    default: return run_scores<D, 128>(mq, mk, a, p, grid, st);
    }
}

}  // namespace

bool make_map_q8(CUtensorMap *m, const void *ptr, uint64_t d0, uint64_t d1, uint64_t d2, uint32_t box1, uint32_t box2)
{
    PFN_cuTensorMapEncodeTiled_v12000 enc = encode_fn();
    if (!enc)
        return false;
    cuuint64_t gdim[3] = {d0, d1, d2};
    cuuint64_t gstride[2] = {d0, d0 * d1};
    cuuint32_t box[3] = {(cuuint32_t)d0, box1, box2};
    cuuint32_t estride[3] = {1, 1, 1};
    const CUtensorMapSwizzle sw = d0 == 128 ? CU_TENSOR_MAP_SWIZZLE_128B
                                            : (d0 == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_32B);
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void *>(ptr), gdim, gstride, box, estride,
               CU_TENSOR_MAP_INTERLEAVE_NONE, sw, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int padded_heads(int H)
{
    int hp = 8;
    while (hp < H)
        hp *= 2;
    return hp;
}

cudaError_t launch_indexer_scores(const ScoresArgs &a, cudaStream_t stream)
{
    const int sms = sm_count();
    if (sms <= 0)
        return cudaErrorUnknown;
    const int hp = padded_heads(a.H);
    ScPlan p;
    // as many tokens a tile as fill 256 columns, but no more than there are;
    // at least 16 columns (the narrowest accumulator of 128 lanes)
    p.tt = kScCols / hp;
    while (p.tt > 1 && p.tt / 2 >= a.S && p.tt / 2 * hp >= 16)
        p.tt /= 2;
    p.n_tt = (a.S + p.tt - 1) / p.tt;
    p.n_kt = (a.P + 127) / 128;
    // Few token tiles (decoding): the keys are split too, into about eight items
    // an SM, but an item has four key tiles where that leaves two an SM (at one tile an
    // item the items' preparation bound: 32 x 2 tokens over 8192 entries take 20.8 us, 14.7
    // with four). With four token tiles an SM or more their unequal lengths even out
    // over the CTAs, and an item's query tile is best read once.
    const long long rows = (long long)a.B * p.n_tt;
    const long long two = rows * p.n_kt / (2LL * sms), least = two < 4 ? two : 4;
    long long chunk = rows >= 4LL * sms ? p.n_kt : rows * p.n_kt / (8LL * sms);
    if (chunk < least)
        chunk = least;
    p.chunk = (int)(chunk < 1 ? 1 : (chunk > p.n_kt ? p.n_kt : chunk));
    const long long items = rows * ((p.n_kt + p.chunk - 1) / p.chunk);
    if (items > INT32_MAX - 65536)
        return cudaErrorInvalidValue;
    p.n_items = (int)items;
    // Split items have few columns a tile, so that one producer's 1,150 cycles a tile
    // bound them (32 x 2 tokens over 16 to 33 thousand entries: 44.5 us, 36.1 with two);
    // whole ones are better served by two warps that prepare items (a packed batch:
    // 26.4 us, 31.2 with one).
    p.producers = p.chunk < p.n_kt && p.chunk >= 2 ? 2 : 1;
    p.box_rows = a.map.page < 128 ? a.map.page : 128;
    p.loads = a.map.max_pages > 1 && a.map.page < 128 ? 128 / a.map.page : 1;
    p.groups = p.tt * hp > 128 ? 2 : 1;
    p.bulk = a.map.page % 4 == 0 && al16(a.k_scale) ? 1 : 0;
    CUtensorMap mq, mk;
    if (!make_map_q8(&mq, a.q8, a.D, a.H, (uint64_t)a.B * a.S, hp, p.tt) ||
        !make_map_q8(&mk, a.cache, a.D, a.map.page, a.map.n_pages, p.box_rows, 1))
        return cudaErrorUnknown;
    const int grid = (int)(p.n_items < sms ? p.n_items : sms);
    if (a.D == 32)
        return run_heads<32>(hp, mq, mk, a, p, grid, stream);
    if (a.D == 64)
        return run_heads<64>(hp, mq, mk, a, p, grid, stream);
    return run_heads<128>(hp, mq, mk, a, p, grid, stream);
}

}  // namespace sai
