// fa8_pages.cu -- per-page key bounds (fa8_page_bounds) and the choice of pages for each query
// (fa8_select_pages).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <string.h>

#include <algorithm>
#include <type_traits>

#include "fa8.h"
#include "fa8_host.h"
#include "fa8_kernel.cuh"
#include "fa8_pages.cuh"

namespace fa8 {

// ------------------------------------------------------------------------------ page bounds
struct BoundsParams {
    const uint8_t *k;
    long long k_s[3];  // page, row, head
    uint8_t *bounds;
    long long b_s[2];  // page, head
    const int *cu_q;   // may be null
    int new_tokens;    // without cu_q; < 0: all
    int D, chunks, groups, npg, blocks_per_req, num_pages;
    host::Table tab;
    unsigned int *status;
};

constexpr int kBoundsThreads = 128;

__device__ __forceinline__ uint32_t hmin2_nan(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("min.NaN.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t hmax2_nan(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// A warp takes 128 bytes (eight 16-channel pieces, a whole line of every row) of one page: lane l holds
// piece l mod 8 of rows l / 8, l / 8 + 4, ..; then the four row parts meet by shuffles.  E4M3 -> f16 is
// exact, so the packed f16 minimum and maximum (NaN-propagating) are, and so is the way back.
// Bound: HBM, one read of the pages' K; short of it no unit alone (cold: DRAM 59 %, ALU pipe 64 %, 27 warps an SM
// that wait for loads).  Measured from a graph's replays, 2048 pages of 64 keys x 8 heads of 128 (137 MB): 25 us,
// 5.4 TB/s, 0.80 of the copy rate, as called 27 us (a thread per 16 channels walking all rows: 32 us); as many
// keys in pages of 16 and 8, where joining the row parts weighs more: 40 and 57 us (eight loads a lane whatever
// the page: 45 and 80); the one new page of 64 requests: 2.9 us (4.6).  With cu_seqlens_q a warp is launched for
// every column of the table, with or without work.
template <int U>
__global__ void __launch_bounds__(kBoundsThreads) page_bounds_kernel(const __grid_constant__ BoundsParams p) {
    const int b = blockIdx.x / p.blocks_per_req;
    const int lane = threadIdx.x & 31;
    const int item = (blockIdx.x - b * p.blocks_per_req) * (kBoundsThreads / 32) + (threadIdx.x >> 5);
    const int slot = item / p.groups;
    if (slot >= p.npg) return;
    const int ps = p.tab.page_size;
    // the chain is lengths -> page -> rows; with all pages asked for, the page does not wait for the lengths
    const int *bt = p.tab.bt + (long long)b * p.tab.bt_stride;
    const bool all = !p.cu_q && p.new_tokens < 0;
    int page = all ? __ldg(bt + slot) : -1;
    const int Lk = __ldg(p.tab.cu_k + b + 1) - __ldg(p.tab.cu_k + b);
    if (Lk < 0 || (long long)Lk > (long long)p.tab.max_pages * ps) {
        if (lane == 0) atomicOr(p.status, kStatusBounds);
        return;
    }
    int pi = slot;
    if (!all) {
        const int m = p.cu_q ? p.cu_q[b + 1] - p.cu_q[b] : p.new_tokens;
        if (m <= 0) return;
        pi += max(0, Lk - m) / ps;
    }
    if ((long long)pi * ps >= Lk) return;
    if (!all) page = bt[pi];
    if (page < 0 || page >= p.num_pages) {
        if (lane == 0) atomicOr(p.status, kStatusBounds);
        return;
    }
    const int rows = min(ps, Lk - pi * ps), part = lane >> 3;
    const int chunk = (item - slot * p.groups) * 8 + (lane & 7);
    const bool on = chunk < p.chunks;
    const int per = p.D >> 4, h = on ? chunk / per : 0, c = on ? chunk - h * per : 0;
    const uint8_t *src = p.k + (long long)page * p.k_s[0] + (long long)h * p.k_s[2] + 16 * c;
    uint32_t lo[8], hi[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {  // infinities: a part may have no row of its own
        lo[i] = 0x7C007C00u;
        hi[i] = 0xFC00FC00u;
    }
    auto take = [&](const Bytes<16> &v) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t a, d;
            e4m3x4_to_h2(v.w[i], a, d);
            lo[2 * i] = hmin2_nan(lo[2 * i], a);
            hi[2 * i] = hmax2_nan(hi[2 * i], a);
            lo[2 * i + 1] = hmin2_nan(lo[2 * i + 1], d);
            hi[2 * i + 1] = hmax2_nan(hi[2 * i + 1], d);
        }
    };
    for (int r = part; r < rows; r += 4 * U) {  // U loads in flight
        Bytes<16> v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) v[u] = ld_stream(src + (long long)min(r + 4 * u, rows - 1) * p.k_s[1]);
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (r + 4 * u < rows) take(v[u]);
    }
    // the four parts meet and divide the result: parts 0 and 1 keep the minima, 2 and 3 the maxima (as minima
    // of the negatives), then even parts the lower half of the channels, odd ones the upper
    uint32_t m[8], x[4];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t neg = hi[i] ^ 0x80008000u;
        m[i] = hmin2_nan(part & 2 ? neg : lo[i], __shfl_xor_sync(0xffffffffu, part & 2 ? lo[i] : neg, 16));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[i] = hmin2_nan(part & 1 ? m[4 + i] : m[i], __shfl_xor_sync(0xffffffffu, part & 1 ? m[i] : m[4 + i], 8));
        if (part & 2) x[i] ^= 0x80008000u;
    }
    if (!on) return;
    uint8_t *dst = p.bounds + (long long)page * p.b_s[0] + (long long)h * p.b_s[1] + 16 * c + (part >> 1) * p.D + 8 * (part & 1);
    *reinterpret_cast<uint2 *>(dst) = make_uint2(ptx::prmt_lo16(ptx::cvt_e4m3x2_h2(x[0]), ptx::cvt_e4m3x2_h2(x[1])),
                                                 ptx::prmt_lo16(ptx::cvt_e4m3x2_h2(x[2]), ptx::cvt_e4m3x2_h2(x[3])));
}

// ------------------------------------------------------------------------------ page selection
struct SelectParams {
    const uint8_t *q;
    long long q_s[3];  // request, token, head
    const uint8_t *bounds;
    long long b_s[2];  // page, head
    int *pages;
    long long o_s[3];  // request, token, head
    const int *cu_q;
    int T, B, Sq, Hkv, G, K, causal, keep_first, keep_last, num_pages, cluster;
    host::Table tab;
    unsigned int *status;
};

constexpr int kSelWarps = 4, kSelThreads = kSelWarps * 32;
constexpr int kSelMaxTable = 16384;  // block_table columns
constexpr int kSelMaxTable4 = 2048;  // of the kernel that takes four tokens at once
constexpr int kSelMaxCluster = 16;
constexpr int kSelList = 256;  // undecided pages that are ranked directly
constexpr int kSelHeld = 16;   // scores that a thread keeps in registers while it chooses

// TB tokens of one request per CTA.  TB = 1: the q-heads in groups of 8 NT rows, all four warps choose.
// TB = 4: each token's q-heads padded to GP = 2, 4 or 8 rows, so that the four tokens are the 4 GP
// columns of one pass over the bounds; then a warp chooses for each token.
template <int D, int NT, int TB>
struct SelCfg {
    static constexpr int GP = 2 * NT;        // TB = 4: rows per token
    static constexpr int ROW = 2 * D;        // bytes of a page's bounds
    // piece ch of row r of a buffer: rows a multiple of 128 bytes long alternate their halves, so that two
    // rows' lanes meet different banks
    static __device__ __forceinline__ int at(int r, int ch) { return r * ROW + 16 * (ROW % 128 == 0 ? ch ^ ((r & 1) << 2) : ch); }
    static constexpr int NV = ROW / 64;      // 16-byte vectors of a row per lane
    static constexpr int STEPS = ROW / 16;   // MMA k-steps
    static constexpr int BUF = 16 * ROW;   // 16 pages
    static constexpr int RING = kSelWarps * BUF;
    static constexpr int QR = TB == 1 ? 8 * NT : TB * GP;  // query rows of one pass
    static constexpr int Q_BYTES = NT * STEPS * 32 * 8 + QR * D;  // as MMA fragments, and as they are
    static constexpr int W = kSelWarps / TB;  // warps that choose for a token
    static_assert(W * TB == kSelWarps, "every warp belongs to one team, whose barrier counts its threads");
    // per token after the ring: fp32 scores, list, scratch, two bit masks; the keys of undecided pages take
    // the ring's place: 64 bits each of kSelList, or the upper 16 bits of every page's 48
    static __host__ __device__ int words(int table) { return (table + 31) / 32; }
    static __host__ __device__ int token_bytes(int table) { return words(table) * (32 * 4 + 8) + kSelList * 4 + 64; }
    static __host__ __device__ int key_bytes(int table) { return words(table) * 64 > kSelList * 8 ? words(table) * 64 : kSelList * 8; }
    static __host__ __device__ int front(int table) {
        const int keys = TB * key_bytes(table);
        return Q_BYTES + (keys > RING ? keys : RING);
    }
    static int smem(int table) { return 128 + front(table) + TB * ((token_bytes(table) + 15) & ~15); }
};

__device__ __forceinline__ unsigned int order_f32(float v) {
    const unsigned int u = __float_as_uint(v + 0.f);  // -0 counts as 0
    return u ^ ((u >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ float unorder_f32(unsigned int u) {
    return __uint_as_float(u ^ ((u >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}
// E4M3 code as a whole number of 2^-9 (NaN not handled)
__device__ __forceinline__ int fixed_e4m3(unsigned int code) {
    const int e = (code >> 3) & 15, m = code & 7;
    const int v = e == 0 ? m : (8 + m) << (e - 1);
    return (code & 0x80u) ? -v : v;
}

// The threads that choose for one token: W warps with their own barrier.  Most of what they run, they
// run once: short loops, because fetching unrolled code costs more than it saves.
template <int W>
struct Team {
    int t, id;            // thread of the team, team of the CTA
    unsigned int *words;  // 16 words of scratch
    __device__ __forceinline__ void sync() const {
        if constexpr (W == 1) __syncwarp();
        else ptx::named_bar_sync(1 + id, 32 * W);
    }
    // f over [0, n), each index by one thread
    template <typename F>
    __device__ __forceinline__ void each(int n, F f) const {
#pragma unroll 1
        for (int i = t; i < n; i += 32 * W) f(i);
    }
    // sum over the team of one value a thread; its maximum (MAX)
    template <bool MAX>
    __device__ __forceinline__ unsigned int reduce(unsigned int v) const {
        v = MAX ? __reduce_max_sync(0xffffffffu, v) : __reduce_add_sync(0xffffffffu, v);
        if constexpr (W > 1) {
            sync();  // the words have been read
            if ((t & 31) == 0) words[t >> 5] = v;
            sync();
            v = words[0];
#pragma unroll
            for (int i = 1; i < W; ++i) v = MAX ? max(v, words[i]) : v + words[i];
        }
        return v;
    }
    // The rank-th largest (rank >= 1) of scores [0, n), as ordered integers: bisection by counting, done
    // when exactly `rank` scores lie in the upper part (after about as many steps as n has bits).  A thread
    // keeps HELD scores in registers; one warp takes twice as many of a longer list (1024 pages: 76 us
    // for 512 tokens x 8 heads against 84; 2048: 173 against 185), four warps gain nothing by it.
    template <int HELD>
    __device__ __forceinline__ unsigned int kth_score(const float *scores, int n, unsigned int rank) const {
        unsigned int v[HELD], hi = 0, nlo = 0;
#pragma unroll
        for (int j = 0; j < HELD; ++j) {
            const int i = t + 32 * W * j;
            v[j] = i < n ? order_f32(scores[i]) : 0u;  // no score is 0: that is a NaN's place
        }
#pragma unroll
        for (int j = 0; j < HELD; ++j) {
            hi = max(hi, v[j]);
            if (v[j]) nlo = max(nlo, ~v[j]);
        }
        // the scores behind them, eight loads at once
        auto rest = [&](auto f) {
#pragma unroll 1
            for (int i = t + 32 * W * HELD; i < n; i += 8 * 32 * W) {
                unsigned int u[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) u[k] = i + 32 * W * k < n ? order_f32(scores[i + 32 * W * k]) : 0u;
#pragma unroll
                for (int k = 0; k < 8; ++k) f(u[k]);
            }
        };
        rest([&](unsigned int u) {
            hi = max(hi, u);
            if (u) nlo = max(nlo, ~u);
        });
        hi = reduce<true>(hi);
        unsigned int lo = ~reduce<true>(nlo);
#pragma unroll 1
        while (lo < hi) {
            const unsigned int mid = lo + (hi - lo + 1) / 2;
            unsigned int c = 0, low = 0;  // scores from mid up: how many, and the complement of the least
#pragma unroll
            for (int j = 0; j < HELD; ++j) c += v[j] >= mid;
            rest([&](unsigned int u) { c += u >= mid; });
            c = reduce<false>(c);
            if (c < rank) {
                hi = mid - 1;
                continue;
            }
            lo = mid;
            if (c > rank) continue;
#pragma unroll
            for (int j = 0; j < HELD; ++j)
                if (v[j] >= mid) low = max(low, ~v[j]);
            rest([&](unsigned int u) {
                if (u >= mid) low = max(low, ~u);
            });
            return ~reduce<true>(low);
        }
        return lo;
    }
    // The largest 48-bit key that at least `rank` (>= 1) of key(0 .. n - 1) reach.  Keys of 0 are none.
    template <typename F>
    __device__ __forceinline__ unsigned long long kth_key(F key, int n, unsigned int rank) const {
        unsigned long long lo = 0, hi = (1ull << 48) - 1;
#pragma unroll 1
        while (lo < hi) {
            const unsigned long long mid = lo + (hi - lo) / 2 + 1;
            unsigned int c = 0;
            each(n, [&](int i) { c += key(i) >= mid; });
            if (reduce<false>(c) >= rank) lo = mid;
            else hi = mid - 1;
        }
        return lo;
    }
};

// Exact score of one page for q-heads [first, end) of a token, by a warp: sum_c max(q_c lo_c, q_c hi_c) in
// units of 2^-18, the largest of the heads; a NaN ranks above all.  Order-preserving key of 48 bits:
// 2^45 + score, which is below 2^44 in magnitude ((448 2^9)^2 times 256 channels), or 2^48 - 1; never 0.
template <int D>
__device__ __forceinline__ unsigned long long exact_key(const uint8_t *src, const uint8_t *q, long long q_sh, int first, int end, int lane) {
    constexpr int NW = (D / 4 + 31) / 32;  // words of four channels per lane
    auto has_nan = [](uint32_t w) { return (((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) != 0; };
    int lo[NW][4], hi[NW][4];
    bool nan = false;
#pragma unroll
    for (int i = 0; i < NW; ++i) {
        const int wd = lane + 32 * i;
        const uint32_t l = wd < D / 4 ? *reinterpret_cast<const uint32_t *>(src + 4 * wd) : 0u;
        const uint32_t h = wd < D / 4 ? *reinterpret_cast<const uint32_t *>(src + D + 4 * wd) : 0u;
        nan |= has_nan(l) || has_nan(h);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            lo[i][e] = fixed_e4m3(l >> (8 * e) & 0xFFu);
            hi[i][e] = fixed_e4m3(h >> (8 * e) & 0xFFu);
        }
    }
    long long best = LLONG_MIN;
#pragma unroll 1
    for (int h = first; h < end; ++h) {
        long long s = 0;
        bool bad = nan;
#pragma unroll
        for (int i = 0; i < NW; ++i) {
            const uint32_t w = lane + 32 * i < D / 4 ? *reinterpret_cast<const uint32_t *>(q + h * q_sh + 4 * (lane + 32 * i)) : 0u;
            bad |= has_nan(w);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int x = fixed_e4m3(w >> (8 * e) & 0xFFu);
                s += (long long)x * (x < 0 ? lo[i][e] : hi[i][e]);
            }
        }
        // |s| < 2^40 in a lane: 20 low bits and the rest are summed apart
        const unsigned int low = __reduce_add_sync(0xffffffffu, (unsigned int)s & 0xFFFFFu);
        const int high = __reduce_add_sync(0xffffffffu, (int)(s >> 20));
        const long long sum = ((long long)high << 20) + low;
        best = max(best, __any_sync(0xffffffffu, bad) ? LLONG_MAX : sum);
    }
    return best == LLONG_MAX ? (1ull << 48) - 1 : (unsigned long long)(best + (1ll << 45));
}

// Every CTA scores its pages with f16 MMAs (pages on M, query rows on N; the contraction runs over
// [lo | hi] against [min(q,0) | max(q,0)], which is sum_c max(q_c lo_c, q_c hi_c)); a page's 2 D bytes
// arrive by asynchronous copies, 16 pages a buffer.  With few rows a cluster of CTAs
// shares a token's pages and rank 0 chooses.
//
// Exact choice from fp32 scores: E4M3 products are exact, and an MMA adds 16 of them to the running sum.  It cuts
// each of these 17 addends below 2^-25 of the largest one's leading bit and the result to fp32's 24 bits (what
// this GPU does, held by a probe: at most half of the bound over 87 kinds of data, among them equal products of
// one sign behind a large one, whose cut parts add up).  No magnitude that passes through is above
// A = max_h |q_h|_1 * max|bound|, and of a page's 2 D products at most D are not zero, as a q_c has one sign.  So
// with 2 D / 16 MMAs a score is off by at most eps = (D + 5 * 2 D / 16) 2^-25 A.  With t the k-th largest fp32
// score, pages above t + 2 eps are in and pages below t - 2 eps out whatever the true scores; the few between
// are scored again in 64-bit integers (E4M3 is a whole number of 2^-9) and ranked by (score, lower index).
//
// Bound: for many pages HBM (2 D bytes per page and kv-head) and the ALU pipe that widens them; else the
// chain of a CTA: 4 us to its first score, 5 us to choose.  Measured, d = 128: 64 x 8 pairs of 64 .. 2048
// pages (140 MB): 48 us, 2.9 TB/s, 0.43 of the copy rate (a token's pages in one CTA with two buffers:
// 51; per-lane bulk copies: 65; fragments straight to registers: 73); 512 tokens x 8 heads over 512 pages:
// 43 us (a token at a time: 164), over 2048 pages 174 us (282 with 64-bit keys of every page in shared memory
// and one load at a time behind the held scores); one pair of 2048 pages, d = 256, a cluster of 16 CTAs: 13 us
// (one CTA: 42); 8 of 16384, d = 128: 76 us, most of it the choice.  With an eps that counts on fp32's 24 bits
// alone, (D + 2 * 2 D / 16) 2^-23 A: 52, 47, 183, 16 and 79 us, for the pages that are scored again; with |x| + |y| of
// two pages as their maximum, an instruction less: 48, 45, 177, 13 and 76 us.
template <int D, int NT, int TB>
__global__ void __launch_bounds__(kSelThreads, D > 128 ? 4 : (TB == 1 && NT == 1 ? 7 : 5)) select_pages_kernel(const __grid_constant__ SelectParams p) {
    using C = SelCfg<D, NT, TB>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~static_cast<uintptr_t>(127));
    __shared__ float s_l1[kSelWarps][TB], s_kmax[kSelMaxCluster], s_kw[kSelWarps];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int CS = TB == 1 ? p.cluster : 1;
    const int rank = CS > 1 ? (int)cluster_rank() : 0;
    const int row = blockIdx.x / CS;
    const int kvh = row % p.Hkv, unit = row / p.Hkv;
    const int ps = p.tab.page_size;
    // ---- tokens tok0 .. tok0 + ntok - 1: the i0-th of request b's Lq new ones on
    int b, i0, Lq, tok0, ntok = 1;
    if constexpr (TB == 1) {
        tok0 = unit;
        if (!locate_token(p.cu_q, p.B, p.Sq, tok0, &b, &i0, &Lq)) return;
    } else {
        int blk;
        if (!p.cu_q) {
            const int per = (p.Sq + TB - 1) / TB;
            b = unit / per;
            blk = unit - b * per;
            Lq = p.Sq;
            tok0 = b * p.Sq;
        } else {  // request b's blocks start at slot cu_q[b] / TB + b
            int lo = 0, hi = p.B - 1;
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (p.cu_q[mid] / TB + mid <= unit) lo = mid;
                else hi = mid - 1;
            }
            b = lo;
            tok0 = p.cu_q[b];
            Lq = p.cu_q[b + 1] - tok0;
            blk = unit - (tok0 / TB + b);
        }
        i0 = blk * TB;
        tok0 += i0;
        ntok = min(TB, Lq - i0);
        if (blk < 0 || ntok <= 0 || tok0 < 0 || (long long)tok0 + ntok > p.T) return;
    }
    const long long bb = p.cu_q ? 0 : b;
    const long long t0 = p.cu_q ? tok0 : i0;
    const int *bt = p.tab.bt + (long long)b * p.tab.bt_stride;
    const uint8_t *q = p.q + bb * p.q_s[0] + t0 * p.q_s[1] + (long long)kvh * p.G * p.q_s[2];
    // the loads that the first scores wait for go out together: the query rows, the first pages (as far as
    // the table goes: the lengths are still on their way), the lengths.  Padding query rows repeat a real
    // one: the maximum does not see them.
    constexpr int QN = (C::QR * (D / 16) + kSelThreads - 1) / kSelThreads;
    uint4 qv[QN];
    auto load_q = [&](int g0) {
#pragma unroll
        for (int k = 0; k < QN; ++k) {
            const int x = tid + k * kSelThreads, r = x / (D / 16), ch = x - r * (D / 16);
            const int tk = TB == 1 ? 0 : min(r / C::GP, ntok - 1);
            const int h = TB == 1 ? (g0 + r < p.G ? g0 + r : g0) : (r % C::GP < p.G ? r % C::GP : 0);
            if (r < C::QR) qv[k] = __ldg(reinterpret_cast<const uint4 *>(q + tk * p.q_s[1] + h * p.q_s[2] + 16 * ch));
        }
    };
    load_q(0);
    const int p0 = p.keep_first + 16 * (warp * CS + rank), stride = 16 * kSelWarps * CS;
    auto id_at = [&](int it) { return lane < 16 && (long long)p0 + it * stride + lane < p.tab.max_pages ? __ldg(bt + p0 + it * stride + lane) : -1; };
    const int id_0 = id_at(0), id_1 = id_at(1);
    const int Lk = p.tab.cu_k[b + 1] - p.tab.cu_k[b];
    bool bad = Lk < 0 || (long long)Lk > (long long)p.tab.max_pages * ps;
    if (bad && tid == 0) atomicOr(p.status, kStatusBounds);
    // pages with a key that the i-th token sees
    auto pages_of = [&](int i) {
        const int vis = bad ? 0 : (p.causal ? min(Lk, Lk - Lq + i + 1) : Lk);
        return vis > 0 ? (vis - 1) / ps + 1 : 0;
    };
    const int n_last = pages_of(i0 + ntok - 1);  // the most of the CTA's tokens
    // ---- this thread's team chooses for one token
    Team<C::W> team;
    team.id = tid / (32 * C::W);
    team.t = tid % (32 * C::W);
    const int words = C::words(p.tab.max_pages);
    uint8_t *mine = smem + C::front(p.tab.max_pages) + team.id * ((C::token_bytes(p.tab.max_pages) + 15) & ~15);
    float *scores = reinterpret_cast<float *>(mine);
    int *list = reinterpret_cast<int *>(mine + words * 128);
    team.words = reinterpret_cast<unsigned int *>(list + kSelList);
    unsigned int *sel = team.words + 16, *amb = sel + words;
    uint8_t *key_mem = smem + C::Q_BYTES + team.id * C::key_bytes(p.tab.max_pages);
    const int n = team.id < ntok ? pages_of(i0 + team.id) : 0;
    int *out = p.pages + bb * p.o_s[0] + (t0 + team.id) * p.o_s[1] + kvh * p.o_s[2];
    if (team.id < ntok && n <= p.K && rank == 0) team.each(p.K, [&](int j) { out[j] = j < n ? j : -1; });
    if (n_last <= p.K) return;
    if (CS > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");

    const uint8_t *bounds = p.bounds + (long long)kvh * p.b_s[1];
    const unsigned int b_stride = (unsigned int)p.b_s[0];
    const int from = p.keep_first, to = n_last - p.keep_last;  // pages that go by score

    // ---- scores of this CTA's pages: chunk it is pages from + 16 ((warp + 4 it) CS + rank) ..
    uint2 *qf = reinterpret_cast<uint2 *>(smem);
    const uint32_t ring = ptx::smem_u32(smem + C::Q_BYTES) + warp * C::BUF;
    const int chunks = to > p0 ? (to - p0 + stride - 1) / stride : 0;
    uint32_t kmax2[4] = {0, 0, 0, 0};
    float l1[TB];
#pragma unroll
    for (int t = 0; t < TB; ++t) l1[t] = 0.f;
    for (int g0 = 0; g0 < (TB == 1 ? p.G : 1); g0 += 8 * NT) {
        if (g0) {
            __syncthreads();  // the last group's rows have been read
            load_q(g0);
        }
        // lane i < 16 holds the i-th page of the chunk that is fetched next; eight consecutive lanes copy
        // 128 consecutive bytes
        auto id_of = [&](int it) { return lane < 16 && it < chunks && p0 + it * stride + lane < to ? __ldg(bt + p0 + it * stride + lane) : -1; };
        int id = p0 + lane < to ? id_0 : -1, id2 = p0 + stride + lane < to ? id_1 : -1;
        unsigned int ok = 0;  // bit i: page i of the buffer is there
        constexpr int RP = C::ROW / 16;  // 16-byte pieces of a row
        auto fetch = [&](int it) {
            const bool good = id >= 0 && id < p.num_pages;
            if (!good && lane < 16 && p0 + it * stride + lane < to) atomicOr(p.status, kStatusBounds);
            const unsigned int m = __ballot_sync(0xffffffffu, good), page = good ? id : 0;
            auto copy = [&](auto all) {  // all: no page is missing
#pragma unroll
                for (int u = 0; u < RP / 2; ++u) {
                    const int r = 32 % RP == 0 ? (32 / RP) * u + lane / RP : (32 * u + lane) / RP;
                    const int ch = 32 % RP == 0 ? lane % RP : (32 * u + lane) % RP;
                    const uint8_t *src = bounds + 16 * ch + (unsigned long long)__shfl_sync(0xffffffffu, page, r) * b_stride;
                    const uint32_t dst = ring + C::at(r, ch);
                    if constexpr (decltype(all)::value) cp_async16(dst, src, 16);
                    else cp_async16(dst, m >> r & 1u ? src : p.bounds, m >> r & 1u ? 16 : 0);
                }
            };
            if (m == 0xFFFFu) copy(std::true_type());
            else copy(std::false_type());
            ok = m;
            id = id2;
            id2 = id_of(it + 2);
        };
        if (chunks > 0) fetch(0);
        cp_async_commit();
        uint8_t *qraw = smem + NT * C::STEPS * 32 * 8;
#pragma unroll
        for (int k = 0; k < QN; ++k)
            if (tid + k * kSelThreads < C::QR * (D / 16)) *reinterpret_cast<uint4 *>(qraw + 16 * (tid + k * kSelThreads)) = qv[k];
        __syncthreads();
#pragma unroll 2
        for (int x = tid; x < NT * C::STEPS * 32; x += kSelThreads) {
            const int ln = x & 31, st = (x >> 5) % C::STEPS, col = 8 * (x / (32 * C::STEPS)) + (ln >> 2);
            const int pos = 64 * (st >> 2) + 16 * (ln & 3) + 4 * (st & 3);
            const bool low = pos < D;
            const uint32_t w = *reinterpret_cast<const uint32_t *>(qraw + col * D + (low ? pos : pos - D));
            const uint32_t neg = ((w >> 7) & 0x01010101u) * 0xFFu;  // bytes with the sign bit
            uint32_t lo, hi;
            e4m3x4_to_h2(low ? (w & neg) : (w & ~neg), lo, hi);
            qf[x] = make_uint2(lo, hi);
        }
        // sums of |q|: eight lanes a row
#pragma unroll
        for (int r0 = 0; r0 < C::QR; r0 += 4 * kSelWarps) {
            const int r = r0 + 4 * warp + (lane >> 3);
            float s = 0.f;
            if (r < C::QR) {
#pragma unroll
                for (int c = 0; c < D; c += 32) {
                    uint32_t lo, hi;
                    float x0, x1, x2, x3;
                    e4m3x4_to_h2(*reinterpret_cast<const uint32_t *>(qraw + r * D + c + 4 * (lane & 7)), lo, hi);
                    ptx::h2_to_f32(lo, x0, x1);
                    ptx::h2_to_f32(hi, x2, x3);
                    s += (fabsf(x0) + fabsf(x1)) + (fabsf(x2) + fabsf(x3));
                }
            }
#pragma unroll
            for (int o = 4; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
#pragma unroll
            for (int t = 0; t < TB; ++t)
                if (TB == 1 || r / C::GP == t) l1[t] = fmaxf(l1[t], s);
        }
        __syncthreads();
#pragma unroll 1
        for (int it = 0; it < chunks; ++it) {
            cp_async_wait<0>();
            __syncwarp();
            float acc[NT][4];
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[t][e] = 0.f;
#pragma unroll
            for (int v = 0; v < C::NV; ++v) {
                const Bytes<16> x = ld_shared<16>(ring + C::at(lane >> 2, 4 * v + (lane & 3))), y = ld_shared<16>(ring + C::at(8 + (lane >> 2), 4 * v + (lane & 3)));
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    uint32_t a[4];
                    e4m3x4_to_h2(x.w[s], a[0], a[2]);
                    e4m3x4_to_h2(y.w[s], a[1], a[3]);
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        const uint2 bf = qf[(t * C::STEPS + 4 * v + s) * 32 + lane];
                        mma_f16(acc[t], a[0], a[1], a[2], a[3], bf.x, bf.y);
                    }
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const __half2 x = __habs2(*reinterpret_cast<__half2 *>(&a[2 * e])), y = __habs2(*reinterpret_cast<__half2 *>(&a[2 * e + 1]));
                        const uint32_t z = hmax2_nan(*reinterpret_cast<const uint32_t *>(&x), *reinterpret_cast<const uint32_t *>(&y));
                        kmax2[2 * (s & 1) + e] = hmax2_nan(z, kmax2[2 * (s & 1) + e]);
                    }
                }
            }
            const unsigned int there = ok;
            __syncwarp();  // the buffer has been read
            if (it + 1 < chunks) fetch(it + 1);
            cp_async_commit();
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int pl = 8 * half + (lane >> 2), pg = p0 + it * stride + pl, c = lane & 3;
                auto put = [&](int token, float s) {
                    float *dst = reinterpret_cast<float *>(reinterpret_cast<uint8_t *>(scores) +
                                                           (TB == 1 ? 0 : (token - team.id) * ((C::token_bytes(p.tab.max_pages) + 15) & ~15)));
                    if (pg >= to) return;
                    if (s != s) s = INFINITY;  // a NaN ranks above all
                    if (!(there >> pl & 1u)) s = -INFINITY;
                    if (TB == 1 && g0) s = fmaxf(s, dst[pg]);
                    dst[pg] = s;
                };
                auto top = [&](int t) { return max_nan(acc[t][2 * half], acc[t][2 * half + 1]); };
                if constexpr (TB == 1) {
                    float s = top(0);
#pragma unroll
                    for (int t = 1; t < NT; ++t) s = max_nan(s, top(t));
                    s = max_nan(s, __shfl_xor_sync(0xffffffffu, s, 1));
                    s = max_nan(s, __shfl_xor_sync(0xffffffffu, s, 2));
                    if (c == 0) put(0, s);
                } else if constexpr (C::GP == 8) {
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        float s = top(t);
                        s = max_nan(s, __shfl_xor_sync(0xffffffffu, s, 1));
                        s = max_nan(s, __shfl_xor_sync(0xffffffffu, s, 2));
                        if (c == t) put(t, s);
                    }
                } else if constexpr (C::GP == 4) {
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        float s = top(t);
                        s = max_nan(s, __shfl_xor_sync(0xffffffffu, s, 1));
                        if ((c & 1) == t) put(2 * t + (c >> 1), s);
                    }
                } else {
                    put(c, top(0));
                }
            }
        }
        cp_async_wait<0>();
    }
    {
        float k = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const __half2 x = *reinterpret_cast<__half2 *>(&kmax2[e]);
            k = max_nan(k, max_nan(__low2float(x), __high2float(x)));
        }
        if (k != k) k = 448.f;  // a NaN may have hidden the page beside it: the largest E4M3 value
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) k = fmaxf(k, __shfl_xor_sync(0xffffffffu, k, o));
#pragma unroll
        for (int t = 0; t < TB; ++t)
#pragma unroll
            for (int o = 16; o > 4; o >>= 1) l1[t] = fmaxf(l1[t], __shfl_xor_sync(0xffffffffu, l1[t], o));
        if (lane == 0) {
            s_kw[warp] = k;
#pragma unroll
            for (int t = 0; t < TB; ++t) s_l1[warp][t] = l1[t];
        }
    }
    __syncthreads();
    if (CS > 1) {
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
        if (rank > 0) {  // hand the scores over to rank 0
            const uint32_t dst = map_rank(ptx::smem_u32(scores), 0);
            for (int t = tid;; t += kSelThreads) {
                const int base = from + ((t >> 4) * CS + rank) * 16, pg = base + (t & 15);
                if (base >= to) break;
                if (pg < to) st_cluster_f32(dst + 4u * (uint32_t)pg, scores[pg]);
            }
        }
        if (tid == 0) {
            float k = s_kw[0];
            for (int w = 1; w < kSelWarps; ++w) k = fmaxf(k, s_kw[w]);
            st_cluster_f32(map_rank(ptx::smem_u32(s_kmax + rank), 0), k);
        }
        cluster_sync();
        if (rank > 0) return;
    }
    if (team.id >= ntok || n <= p.K) return;

    // ---- the choice
    const int last = n - p.keep_last, want = p.K - p.keep_first - p.keep_last;
    float a_l1 = 0.f, a_k = 0.f;
    for (int w = 0; w < kSelWarps; ++w) {
        a_l1 = fmaxf(a_l1, s_l1[w][TB == 1 ? 0 : team.id]);
        a_k = fmaxf(a_k, s_kw[w]);
    }
    for (int r = 0; CS > 1 && r < CS; ++r) a_k = fmaxf(a_k, s_kmax[r]);
    const float eps2 = 2.002f * (D + 5 * C::STEPS) * 0x1p-25f * a_l1 * a_k;  // 2 eps; 0.002 for A's own roundings
    float t_hi = INFINITY, t_lo = INFINITY;
    if (want > 0) {
        unsigned int kth;
        if (C::W > 1 || last - from <= 32 * kSelHeld) kth = team.template kth_score<kSelHeld>(scores + from, last - from, want);
        else kth = team.template kth_score<2 * kSelHeld>(scores + from, last - from, want);
        const float t = unorder_f32(kth);
        t_hi = __fadd_ru(t, eps2);
        t_lo = __fsub_rd(t, eps2);
    }
    const int nw = (n + 31) >> 5, tw = team.t >> 5;
    int n_in = 0;  // the same in every lane of a warp
    unsigned int *n_list = team.words + 14;
    if (team.t == 0) *n_list = 0;
    team.sync();
#pragma unroll 2
    for (int w = tw; w < nw; w += C::W) {
        const int pg = 32 * w + lane;
        const bool scored = pg >= from && pg < last;
        bool in = false, maybe = false;
        if (scored && want > 0) {
            const float s = scores[pg];
            in = s > t_hi;
            maybe = !in && s >= t_lo;
        }
        const unsigned int bs = __ballot_sync(0xffffffffu, in), bm = __ballot_sync(0xffffffffu, maybe);
        const unsigned int bf = __ballot_sync(0xffffffffu, pg < n && !scored);
        n_in += __popc(bs);
        if (maybe) {
            const unsigned int at = atomicAdd(n_list, 1u);
            if (at < kSelList) list[at] = pg;
        }
        if (lane == 0) {
            sel[w] = bs | bf;
            amb[w] = bm;
        }
    }
    if constexpr (C::W > 1) {
        if (lane == 0) team.words[tw] = (unsigned)n_in;
        team.sync();
        n_in = 0;
#pragma unroll
        for (int w = 0; w < C::W; ++w) n_in += (int)team.words[w];
    }
    team.sync();
    const int n_amb = (int)*n_list;
    const int places = want - n_in;  // for the undecided pages
    if (n_amb == places) {
        team.each(nw, [&](int w) { sel[w] |= amb[w]; });
    } else if (places > 0 && n_amb > 0) {
        // Keys that order the undecided pages exactly.  All-zero queries or bounds leave exact zeros.
        const bool exact = !(eps2 > 0.f);
        auto key_of = [&](int pg, int hs, int he) {
            if (exact) return (unsigned long long)order_f32(scores[pg]);
            const int id = bt[pg];
            if (id < 0 || id >= p.num_pages || hs >= he) return 0ull;
            return exact_key<D>(bounds + (long long)id * p.b_s[0], q + (TB == 1 ? 0 : team.id) * p.q_s[1], p.q_s[2], hs, he, lane);
        };
        if (n_amb <= kSelList) {
            unsigned long long *keys = reinterpret_cast<unsigned long long *>(key_mem);
            // by rank among the undecided; every warp scores a part of each page's heads
            team.each(n_amb, [&](int i) { keys[i] = 0; });
            team.sync();
#pragma unroll 1
            for (int i = 0; i < n_amb; ++i) {
                const unsigned long long key = key_of(list[i], tw * p.G / C::W, (tw + 1) * p.G / C::W);
                if (lane == 0) atomicMax(&keys[i], key);
            }
            team.sync();
            team.each(n_amb, [&](int i) {
                const int pg = list[i];
                const unsigned long long key = keys[i];
                int ahead = 0;
#pragma unroll 2
                for (int j = 0; j < n_amb; ++j) ahead += keys[j] > key || (keys[j] == key && list[j] < pg);
                if (ahead < places) atomicOr(&sel[pg >> 5], 1u << (pg & 31));
            });
        } else {
            // many (equal or nearly equal pages): a warp per page, then bisection over the keys, whose lower
            // 32 bits take the scores' place
            unsigned int *key_lo = reinterpret_cast<unsigned int *>(scores);
            unsigned short *key_hi = reinterpret_cast<unsigned short *>(key_mem);
            auto key_at = [&](int i) { return (unsigned long long)key_hi[i] << 32 | key_lo[i]; };
#pragma unroll 1
            for (int w = tw; w < nw; w += C::W) {
                if (!(amb[w] >> lane & 1u)) key_lo[32 * w + lane] = 0, key_hi[32 * w + lane] = 0;
#pragma unroll 1
                for (unsigned int bits = amb[w]; bits; bits &= bits - 1) {
                    const int pg = 32 * w + __ffs(bits) - 1;
                    const unsigned long long key = key_of(pg, 0, p.G);
                    __syncwarp();  // the page's score has been read
                    if (lane == 0) key_lo[pg] = (unsigned int)key, key_hi[pg] = (unsigned short)(key >> 32);
                }
            }
            team.sync();
            const unsigned long long t = team.kth_key(key_at, n, places);
            unsigned int c = 0;
            team.each(n, [&](int i) { c += key_at(i) > t; });
            int left = places - (int)team.template reduce<false>(c);  // of the keys equal to t
            if (tw == 0) {  // ties at the threshold in index order
                for (int w = 0; w < nw; ++w) {
                    const bool on = amb[w] >> lane & 1u;
                    const unsigned long long key = on ? key_at(32 * w + lane) : 0;
                    unsigned int take = __ballot_sync(0xffffffffu, on && key > t);
                    unsigned int tie = __ballot_sync(0xffffffffu, on && key == t);
                    while (tie && left > 0) {
                        take |= tie & -tie;
                        tie &= tie - 1;
                        --left;
                    }
                    if (lane == 0) sel[w] |= take;
                }
            }
        }
    }
    team.sync();
    // ---- the chosen pages in ascending order: thread t lists words [t per, (t + 1) per)
    const int per = (nw + 32 * C::W - 1) / (32 * C::W);
    int cnt = 0;
    for (int w = team.t * per; w < min(nw, (team.t + 1) * per); ++w) cnt += __popc(sel[w]);
    int incl = cnt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
    }
    int at = incl - cnt;
    if constexpr (C::W > 1) {
        if (lane == 31) team.words[tw] = (unsigned)incl;
        team.sync();
        for (int w = 0; w < tw; ++w) at += (int)team.words[w];
    }
    for (int w = team.t * per; w < min(nw, (team.t + 1) * per); ++w)
        for (unsigned int bits = sel[w]; bits; bits &= bits - 1)
            if (at < p.K) out[at++] = 32 * w + __ffs(bits) - 1;
}

template <int D, int NT, int TB>
cudaError_t launch_select(SelectParams &p, unsigned int rows, int dev, cudaStream_t s) {
    static host::SmemOptIn opt_in;
    static host::Cluster16 cluster16;
    const int smem = SelCfg<D, NT, TB>::smem(p.tab.max_pages);
    const cudaError_t e = opt_in(select_pages_kernel<D, NT, TB>, smem, dev);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(rows * p.cluster);
    cfg.blockDim = dim3(kSelThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = p.cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.cluster > 1 ? 1 : 0;
    if (p.cluster > 8 && !cluster16(select_pages_kernel<D, NT, TB>, cfg, dev)) {
        p.cluster = attr[0].val.clusterDim.x = 8;
        cfg.gridDim = dim3(rows * 8);
    }
    return cudaLaunchKernelEx(&cfg, select_pages_kernel<D, NT, TB>, p);
}

template <int D>
cudaError_t launch_select_dim(SelectParams &p, unsigned int rows, bool four, int dev, cudaStream_t s) {
    if (four) return p.G <= 2 ? launch_select<D, 1, 4>(p, rows, dev, s) : (p.G <= 4 ? launch_select<D, 2, 4>(p, rows, dev, s) : launch_select<D, 4, 4>(p, rows, dev, s));
    return p.G <= 8 ? launch_select<D, 1, 1>(p, rows, dev, s) : launch_select<D, 2, 1>(p, rows, dev, s);
}

}  // namespace fa8

namespace {

using namespace fa8::host;

// bounds (num_pages, Hkv, 2, D), E4M3
fa8_status check_bounds(const fa8_tensor *t, long long Hkv, long long D) {
    if (t->dtype != FA8_DTYPE_E4M3) return fail(FA8_ERR_UNSUPPORTED, "bounds must be E4M3");
    if (t->ndim != 4 || t->shape[1] != Hkv || t->shape[2] != 2 || t->shape[3] != D)
        return fail(FA8_ERR_INVALID_ARG, "bounds must be (num_pages, Hkv=%lld, 2, D=%lld)", Hkv, D);
    if (t->stride[3] != 1 || t->stride[2] != D) return fail(FA8_ERR_INVALID_ARG, "bounds: the last two dims must be contiguous");
    for (int i = 0; i < 2; ++i)
        if (t->stride[i] < 0 || t->stride[i] % 16 != 0) return fail(FA8_ERR_INVALID_ARG, "bounds: strides must be multiples of 16 bytes");
    if (t->stride[0] > 0x7fffffffLL) return fail(FA8_ERR_UNSUPPORTED, "bounds: a page's stride must be below 2^31 bytes");
    if (!aligned16(t->data)) return fail(FA8_ERR_INVALID_ARG, "bounds: data must be 16-byte aligned");
    if (t->shape[0] < 0 || t->shape[0] > 0x7fffffffLL) return fail(FA8_ERR_UNSUPPORTED, "too many pages");
    if (t->shape[0] > 0 && !t->data) return fail(FA8_ERR_INVALID_ARG, "bounds has a null data pointer");
    return FA8_SUCCESS;
}

}  // namespace

extern "C" {

fa8_status fa8_page_bounds(const fa8_tensor *k, fa8_tensor *bounds, const fa8_tensor *cu_seqlens_q,
                           const fa8_tensor *cu_seqlens_k, const fa8_tensor *block_table, int page_size, int new_tokens,
                           void *stream) {
    clear_error();
    if (!k || !bounds) return fail(FA8_ERR_INVALID_ARG, "k and bounds are required");
    if (k->dtype != FA8_DTYPE_E4M3) return fail(FA8_ERR_UNSUPPORTED, "k must be E4M3");
    fa8_status st = check_payload(k, "k");
    if (st) return st;
    if (k->ndim != 4) return fail(FA8_ERR_INVALID_ARG, "k must be paged (num_pages, page_size, Hkv, d)");
    const long long Hkv = k->shape[2], D = k->shape[3];
    if (D < 16 || D > 256 || D % 16 != 0) return fail(FA8_ERR_UNSUPPORTED, "d = %lld is not a multiple of 16 up to 256", D);
    if (Hkv <= 0 || Hkv > 65536) return fail(FA8_ERR_INVALID_ARG, "k needs kv heads");
    if ((st = check_bounds(bounds, Hkv, D))) return st;
    if ((st = check_written(bounds, "bounds"))) return st;
    if (bounds->shape[0] != k->shape[0]) return fail(FA8_ERR_INVALID_ARG, "bounds and k must have the same pages");
    if (k->shape[0] > 0 && !k->data) return fail(FA8_ERR_INVALID_ARG, "k has a null data pointer");
    if (!block_table || block_table->ndim != 2) return fail(FA8_ERR_INVALID_ARG, "block_table must be a 2-D int32 tensor");
    const long long B = block_table->shape[0];
    if (B <= 0 || B > 0x7fffffffLL - 1) return fail(FA8_ERR_INVALID_ARG, "batch must be >= 1");
    fa8::BoundsParams p;
    memset(&p, 0, sizeof(p));
    if ((st = check_table(cu_seqlens_k, block_table, page_size, (int)B, &p.tab))) return st;
    if (page_size != k->shape[1]) return fail(FA8_ERR_INVALID_ARG, "page_size (%d) != k.shape[1] (%lld)", page_size, (long long)k->shape[1]);
    if (cu_seqlens_q) {
        if ((st = check_int_vec(cu_seqlens_q, "cu_seqlens_q", B + 1))) return st;
        p.cu_q = static_cast<const int *>(cu_seqlens_q->data);
    }
    p.new_tokens = new_tokens;
    p.k = static_cast<const uint8_t *>(k->data);
    p.bounds = static_cast<uint8_t *>(bounds->data);
    for (int i = 0; i < 3; ++i) p.k_s[i] = k->stride[i];
    for (int i = 0; i < 2; ++i) p.b_s[i] = bounds->stride[i];
    p.D = (int)D;
    p.chunks = (int)(Hkv * D / 16);
    p.num_pages = (int)k->shape[0];
    p.npg = p.tab.max_pages;
    if (!cu_seqlens_q && new_tokens >= 0) {
        if (new_tokens == 0) return FA8_SUCCESS;
        p.npg = (int)std::min<long long>(p.npg, ((long long)new_tokens - 1 + page_size - 1) / page_size + 1);
    }
    p.groups = (p.chunks + 7) / 8;
    const long long items = (long long)p.npg * p.groups, warps = fa8::kBoundsThreads / 32;
    const long long per_req = (items + warps - 1) / warps;
    if (items > 0x7fffffffLL - warps || per_req * B > 0x7fffffffLL)
        return fail(FA8_ERR_UNSUPPORTED, "problem too large for the grid");
    p.blocks_per_req = (int)per_req;
    DeviceState *ds = nullptr;
    if ((st = device_state(&ds))) return st;
    p.status = ds->status;
    // as many loads in flight as a lane group has rows of a page, eight at most
    auto kernel = page_size <= 8 ? fa8::page_bounds_kernel<2> : (page_size <= 16 ? fa8::page_bounds_kernel<4> : fa8::page_bounds_kernel<8>);
    kernel<<<(unsigned)(per_req * B), fa8::kBoundsThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_fail(e, "page bounds kernel launch");
    return FA8_SUCCESS;
}

fa8_status fa8_select_pages(const fa8_tensor *q, const fa8_tensor *bounds, fa8_tensor *pages,
                            const fa8_tensor *cu_seqlens_q, const fa8_tensor *cu_seqlens_k, const fa8_tensor *block_table,
                            int page_size, int causal, int keep_first, int keep_last, void *stream) {
    clear_error();
    if (!q || !bounds || !pages) return fail(FA8_ERR_INVALID_ARG, "q, bounds and pages are required");
    if (q->dtype != FA8_DTYPE_E4M3) return fail(FA8_ERR_UNSUPPORTED, "q must be E4M3");
    fa8::SelectParams p;
    memset(&p, 0, sizeof(p));
    fa8_status st = check_payload(q, "q");
    if (st) return st;
    Queries qs;
    if ((st = check_queries(q, cu_seqlens_q, &qs))) return st;
    if (qs.D != 64 && qs.D != 96 && qs.D != 128 && qs.D != 192 && qs.D != 256)
        return fail(FA8_ERR_UNSUPPORTED, "d = %d is not supported", qs.D);
    if (bounds->ndim != 4) return fail(FA8_ERR_INVALID_ARG, "bounds must be (num_pages, Hkv, 2, D)");
    const long long Hkv = bounds->shape[1];
    if ((st = check_bounds(bounds, Hkv, qs.D))) return st;
    if ((st = check_groups(qs.Hq, Hkv, &p.G))) return st;
    if ((st = check_table(cu_seqlens_k, block_table, page_size, qs.B, &p.tab))) return st;
    if (p.tab.max_pages > fa8::kSelMaxTable)
        return fail(FA8_ERR_UNSUPPORTED, "block_table has %d columns, at most %d are supported", p.tab.max_pages, fa8::kSelMaxTable);
    if ((st = check_page_lists(pages, qs, (int)Hkv, p.o_s, &p.K))) return st;
    if ((st = check_written(pages, "pages"))) return st;
    if (p.K < 1) return fail(FA8_ERR_INVALID_ARG, "top_k must be at least 1");
    if (causal != 0 && causal != 1) return fail(FA8_ERR_INVALID_ARG, "causal must be 0 or 1");
    if (keep_first < 0 || keep_last < 0 || (long long)keep_first + keep_last > p.K)
        return fail(FA8_ERR_INVALID_ARG, "keep_first and keep_last must be >= 0 and sum to at most top_k (%d)", p.K);
    const long long rows = (long long)qs.T * Hkv;
    if (rows * fa8::kSelMaxCluster > 0x7fffffffLL) return fail(FA8_ERR_UNSUPPORTED, "problem too large for the grid");
    if (rows == 0) return FA8_SUCCESS;
    if (!q->data || !pages->data) return fail(FA8_ERR_INVALID_ARG, "q and pages need data");
    DeviceState *ds = nullptr;
    if ((st = device_state(&ds))) return st;
    p.q = static_cast<const uint8_t *>(q->data);
    for (int i = 0; i < 3; ++i) p.q_s[i] = qs.stride[i];
    p.bounds = static_cast<const uint8_t *>(bounds->data);
    p.b_s[0] = bounds->stride[0];
    p.b_s[1] = bounds->stride[1];
    p.pages = static_cast<int *>(pages->data);
    p.cu_q = qs.cu_q;
    p.T = qs.T;
    p.B = qs.B;
    p.Sq = qs.Sq;
    p.Hkv = (int)Hkv;
    p.causal = causal;
    p.keep_first = keep_first;
    p.keep_last = keep_last;
    p.num_pages = (int)bounds->shape[0];
    p.status = ds->status;
    // Several tokens per request and enough of them to fill the GPU in blocks of four: one pass over
    // the bounds serves four tokens.  Else a token at a time, and where there are few (token, kv-head)
    // pairs a cluster of CTAs shares each pair's pages, 128 or more a CTA, up to the seven CTAs that fit an
    // SM (512 ragged pairs of up to 2048 pages: 48 us in clusters of two, 55 without).  Clusters of 16 only
    // while every CTA may have an SM (one pair of 2048 pages, d = 256: 12.7 us against 14.8 in eight and 42 in one
    // CTA; 64 pairs: 33 against 29 in eight).
    const long long blocks = p.cu_q ? (long long)qs.T / 4 + qs.B : (long long)qs.B * ((qs.Sq + 3) / 4);
    const bool four = p.G <= 8 && (long long)qs.T >= 4LL * qs.B && blocks * Hkv >= 2LL * ds->sm_count &&
                      p.tab.max_pages <= fa8::kSelMaxTable4;
    p.cluster = 1;
    if (!four)
        while (p.cluster < fa8::kSelMaxCluster && rows * p.cluster * 2 <= (p.cluster < 8 ? 7LL : 1LL) * ds->sm_count && p.tab.max_pages >= 128 * p.cluster * 2)
            p.cluster *= 2;
    if (blocks * Hkv > 0x7fffffffLL) return fail(FA8_ERR_UNSUPPORTED, "problem too large for the grid");
    const unsigned grid = (unsigned)(four ? blocks * Hkv : rows);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e = cudaErrorInvalidValue;
    switch (qs.D) {
        case 64: e = fa8::launch_select_dim<64>(p, grid, four, ds->ordinal, s); break;
        case 96: e = fa8::launch_select_dim<96>(p, grid, four, ds->ordinal, s); break;
        case 128: e = fa8::launch_select_dim<128>(p, grid, four, ds->ordinal, s); break;
        case 192: e = fa8::launch_select_dim<192>(p, grid, four, ds->ordinal, s); break;
        case 256: e = fa8::launch_select_dim<256>(p, grid, four, ds->ordinal, s); break;
    }
    if (e != cudaSuccess) return cuda_fail(e, "page selection kernel launch");
    return FA8_SUCCESS;
}

}  // extern "C"
