// fa8_pages.cu -- per-page key bounds (fa8_page_bounds) and the choice of pages for each query
// (fa8_select_pages).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <string.h>

#include <algorithm>

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
    int D, chunks, npg, blocks_per_req, num_pages;
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

// A thread owns 16 channels of one kv-head of one page and walks the page's rows.  E4M3 -> f16 is
// exact, so the packed f16 minimum and maximum (NaN-propagating) are, and so is the way back.
// Bound: HBM, one read of the pages' K.
__global__ void __launch_bounds__(kBoundsThreads) page_bounds_kernel(const __grid_constant__ BoundsParams p) {
    const int b = blockIdx.x / p.blocks_per_req;
    const int item = (blockIdx.x - b * p.blocks_per_req) * kBoundsThreads + threadIdx.x;
    const int slot = item / p.chunks;
    if (slot >= p.npg) return;
    const int ps = p.tab.page_size;
    const int Lk = p.tab.cu_k[b + 1] - p.tab.cu_k[b];
    if (Lk < 0 || (long long)Lk > (long long)p.tab.max_pages * ps) {
        atomicOr(p.status, kStatusBounds);
        return;
    }
    int first = 0;
    const int m = p.cu_q ? p.cu_q[b + 1] - p.cu_q[b] : p.new_tokens;
    if (m >= 0) {
        if (m == 0) return;
        first = max(0, Lk - m) / ps;
    }
    const int pi = first + slot;
    if ((long long)pi * ps >= Lk) return;
    const int page = p.tab.bt[(long long)b * p.tab.bt_stride + pi];
    if (page < 0 || page >= p.num_pages) {
        atomicOr(p.status, kStatusBounds);
        return;
    }
    const int chunk = item - slot * p.chunks;
    const int per = p.D >> 4, h = chunk / per, c = chunk - h * per;
    const int rows = min(ps, Lk - pi * ps);
    const uint8_t *src = p.k + (long long)page * p.k_s[0] + (long long)h * p.k_s[2] + 16 * c;
    uint32_t lo[8], hi[8];
    {
        const Bytes<16> v = ld_stream<16>(src);
#pragma unroll
        for (int i = 0; i < 4; ++i) e4m3x4_to_h2(v.w[i], lo[2 * i], lo[2 * i + 1]);
#pragma unroll
        for (int i = 0; i < 8; ++i) hi[i] = lo[i];
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
    int r = 1;
    for (; r + 8 <= rows; r += 8) {  // eight loads in flight
        Bytes<16> v[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) v[u] = ld_stream<16>(src + (long long)(r + u) * p.k_s[1]);
#pragma unroll
        for (int u = 0; u < 8; ++u) take(v[u]);
    }
    for (; r < rows; ++r) take(ld_stream<16>(src + (long long)r * p.k_s[1]));
    uint32_t wl[4], wh[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        wl[i] = ptx::prmt_lo16(ptx::cvt_e4m3x2_h2(lo[2 * i]), ptx::cvt_e4m3x2_h2(lo[2 * i + 1]));
        wh[i] = ptx::prmt_lo16(ptx::cvt_e4m3x2_h2(hi[2 * i]), ptx::cvt_e4m3x2_h2(hi[2 * i + 1]));
    }
    uint8_t *dst = p.bounds + (long long)page * p.b_s[0] + (long long)h * p.b_s[1] + 16 * c;
    *reinterpret_cast<uint4 *>(dst) = make_uint4(wl[0], wl[1], wl[2], wl[3]);
    *reinterpret_cast<uint4 *>(dst + p.D) = make_uint4(wh[0], wh[1], wh[2], wh[3]);
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

constexpr int kSelThreads = 256, kSelWarps = kSelThreads / 32;
constexpr int kSelMaxTable = 16384;
constexpr int kSelMaxCluster = 8;

// Shared memory, by table width: the q operand of one group of rows; 8 bytes a page (fp32 scores,
// later the 64-bit keys of the undecided pages); two bit masks over the pages.
template <int D, int NT>
struct SelCfg {
    static constexpr int NV = 2 * D / 64;      // 16-byte vectors of a bounds row per lane
    static constexpr int STEPS = 2 * D / 16;   // MMA k-steps
    static constexpr int MT = D <= 128 ? 2 : 1;  // 16-page tiles in flight per warp (registers)
    static constexpr int Q_BYTES = NT * STEPS * 32 * 8;
    static int words(int table) { return (table + 31) / 32; }
    static int smem(int table) { return Q_BYTES + words(table) * 32 * 8 + 2 * words(table) * 4; }
};

__device__ __forceinline__ unsigned int order_f32(float v) {
    const unsigned int u = __float_as_uint(v);
    return u ^ ((u >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ float unorder_f32(unsigned int u) {
    return __uint_as_float(u ^ ((u >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}
// E4M3 code as a whole number of 2^-9 (NaN not handled)
__device__ __forceinline__ int fixed_e4m3(unsigned int code) {
    const int e = (code >> 3) & 15, m = code & 7;
    const int v = e == 0 ? m : (8 + m) << (e - 1);
    return (code & 0x80u) ? -v : v;
}

// The rank-th largest (rank >= 1) of `count` ordered integers of BITS bits, key(i) for i in
// [0, count) where on(i): 8 bits a pass, by histogram.  `left` returns how many equal to the
// result are among the rank largest.  Called by all threads.
template <int BITS, typename U, typename F>
__device__ __forceinline__ U kth_largest(int count, int rank, unsigned int *hist, unsigned int *res, int *left, F key) {
    U prefix = 0;
    for (int shift = BITS - 8; shift >= 0; shift -= 8) {
        for (int i = threadIdx.x; i < 256; i += kSelThreads) hist[i] = 0;
        __syncthreads();
        const U mask = shift + 8 >= BITS ? 0 : ~(U)0 << (shift + 8);
        for (int i = threadIdx.x; i < count; i += kSelThreads) {
            U u;
            if (key(i, &u) && (u & mask) == prefix) atomicAdd(&hist[(unsigned int)(u >> shift) & 255u], 1u);
        }
        __syncthreads();
        if (threadIdx.x < 32) {  // lane l: bins 255 - 8 l downwards
            const int lane = threadIdx.x;
            int own = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) own += (int)hist[255 - 8 * lane - j];
            int incl = own;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int x = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += x;
            }
            int above = incl - own;
            if (above < rank && rank <= incl) {
#pragma unroll 1
                for (int j = 0; j < 8; ++j) {
                    const int c = (int)hist[255 - 8 * lane - j];
                    if (above + c >= rank) {
                        res[0] = 255 - 8 * lane - j;
                        res[1] = (unsigned int)(rank - above);
                        break;
                    }
                    above += c;
                }
            }
        }
        __syncthreads();
        prefix |= (U)res[0] << shift;
        rank = (int)res[1];
        __syncthreads();
    }
    *left = rank;
    return prefix;
}

// A cluster of CTAs per (token, kv-head).  Every CTA scores a share of the pages with f16 MMAs
// (pages on M, q-heads on N; the contraction runs over [lo | hi] against [min(q,0) | max(q,0)],
// which is sum_c max(q_c lo_c, q_c hi_c)), and rank 0 chooses.
//
// Exact choice from fp32 scores: E4M3 products are exact, an MMA adds 16 of them to the running
// sum, and what it drops is below 2^-22 of the largest magnitude passing through, itself at most
// A = max_h |q_h|_1 * max|bound|.  So a score is off by at most eps = 2^-16 A (2 D / 16 <= 32
// steps, and a factor two to spare).  With t the k-th largest fp32 score, pages above t + 2 eps
// are in and pages below t - 2 eps out whatever the true scores; the few between are scored again
// in 64-bit integers (E4M3 is a whole number of 2^-9) and ranked by (score, lower index).
// Bound: HBM/L2, 2 D bytes per page and kv-head, for long requests; launch and chain latency for
// short ones.
template <int D, int NT>
__global__ void __launch_bounds__(kSelThreads) select_pages_kernel(const __grid_constant__ SelectParams p) {
    using C = SelCfg<D, NT>;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ unsigned int hist[256];
    __shared__ unsigned int res[2];
    __shared__ float s_l1[kSelWarps], s_kmax[kSelMaxCluster], s_kw[kSelWarps];
    __shared__ int s_in, s_amb, s_list[256], s_cnt, s_scan[kSelWarps];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int CS = p.cluster;
    const int rank = CS > 1 ? (int)cluster_rank() : 0;
    const int row = blockIdx.x / CS;
    const int kvh = row % p.Hkv, tok = row / p.Hkv;
    const int ps = p.tab.page_size;
    int b, i, Lq;
    if (!locate_token(p.cu_q, p.B, p.Sq, tok, &b, &i, &Lq)) return;
    const int Lk = p.tab.cu_k[b + 1] - p.tab.cu_k[b];
    int vis = p.causal ? min(Lk, Lk - Lq + i + 1) : Lk;
    if (Lk < 0 || (long long)Lk > (long long)p.tab.max_pages * ps) {
        if (tid == 0) atomicOr(p.status, kStatusBounds);
        vis = 0;
    }
    const int n = vis > 0 ? (vis - 1) / ps + 1 : 0;
    const long long bb = p.cu_q ? 0 : b, tt = p.cu_q ? tok : i;
    int *out = p.pages + bb * p.o_s[0] + tt * p.o_s[1] + kvh * p.o_s[2];
    if (n <= p.K) {
        if (rank == 0)
            for (int j = tid; j < p.K; j += kSelThreads) out[j] = j < n ? j : -1;
        return;
    }
    if (CS > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");

    uint2 *qf = reinterpret_cast<uint2 *>(smem);
    const int words = (p.tab.max_pages + 31) >> 5;
    float *scores = reinterpret_cast<float *>(smem + C::Q_BYTES);
    unsigned long long *keys = reinterpret_cast<unsigned long long *>(smem + C::Q_BYTES);
    unsigned int *sel = reinterpret_cast<unsigned int *>(smem + C::Q_BYTES + (size_t)words * 32 * 8);
    unsigned int *amb = sel + words;
    const int *bt = p.tab.bt + (long long)b * p.tab.bt_stride;
    const uint8_t *q = p.q + bb * p.q_s[0] + tt * p.q_s[1] + (long long)kvh * p.G * p.q_s[2];
    const uint8_t *bounds = p.bounds + (long long)kvh * p.b_s[1];
    const int from = p.keep_first, to = n - p.keep_last;  // pages that go by score

    // ---- scores of this CTA's pages
    uint32_t kmax2 = 0;
    float l1 = 0.f;
    for (int g0 = 0; g0 < p.G; g0 += 8 * NT) {
        if (g0) __syncthreads();
        for (int x = tid; x < NT * C::STEPS * 32; x += kSelThreads) {
            const int ln = x & 31, st = (x >> 5) % C::STEPS, nt = x / (32 * C::STEPS);
            // padding rows repeat row g0: the maximum over rows does not see them
            const int hr = g0 + nt * 8 + (ln >> 2) < p.G ? g0 + nt * 8 + (ln >> 2) : g0;
            const int pos = 64 * (st >> 2) + 16 * (ln & 3) + 4 * (st & 3);
            const bool low = pos < D;
            const uint32_t w = *reinterpret_cast<const uint32_t *>(q + hr * p.q_s[2] + (low ? pos : pos - D));
            const uint32_t neg = ((w >> 7) & 0x01010101u) * 0xFFu;  // bytes with the sign bit
            const uint32_t part = low ? (w & neg) : (w & ~neg);
            uint32_t lo, hi;
            e4m3x4_to_h2(part, lo, hi);
            qf[x] = make_uint2(lo, hi);
        }
        for (int r = warp; r < min(8 * NT, p.G - g0); r += kSelWarps) {
            float s = 0.f;
            for (int c = lane * 2; c < D; c += 64) {
                float x0, x1;
                ptx::e4m3x2_to_f32(*reinterpret_cast<const uint16_t *>(q + (g0 + r) * p.q_s[2] + c), x0, x1);
                s += fabsf(x0) + fabsf(x1);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
            l1 = fmaxf(l1, s);
        }
        __syncthreads();
        constexpr int PP = 16 * C::MT;  // pages per warp step
        for (int p0 = from + (warp * CS + rank) * PP; p0 < to; p0 += PP * CS * kSelWarps) {
            int id = -1;
            if (lane < PP && p0 + lane < to) {
                id = bt[p0 + lane];
                if (id < 0 || id >= p.num_pages) {
                    id = -1;
                    atomicOr(p.status, kStatusBounds);
                }
            }
            Bytes<16> raw[2 * C::MT][C::NV];
#pragma unroll
            for (int m = 0; m < 2 * C::MT; ++m) {
                const int pg = __shfl_sync(0xffffffffu, id, 8 * m + (lane >> 2));
                const uint8_t *src = bounds + (long long)max(pg, 0) * p.b_s[0] + 16 * (lane & 3);
#pragma unroll
                for (int v = 0; v < C::NV; ++v) {
                    if (pg >= 0) raw[m][v] = ld_stream<16>(src + 64 * v);
                    else raw[m][v] = Bytes<16>{};
                }
            }
            float acc[C::MT][NT][4];
#pragma unroll
            for (int m = 0; m < C::MT; ++m)
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[m][t][e] = 0.f;
#pragma unroll
            for (int v = 0; v < C::NV; ++v)
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    uint2 bf[NT];
#pragma unroll
                    for (int t = 0; t < NT; ++t) bf[t] = qf[(t * C::STEPS + 4 * v + s) * 32 + lane];
#pragma unroll
                    for (int m = 0; m < C::MT; ++m) {
                        uint32_t a0, a1, a2, a3;
                        e4m3x4_to_h2(raw[2 * m][v].w[s], a0, a2);
                        e4m3x4_to_h2(raw[2 * m + 1][v].w[s], a1, a3);
#pragma unroll
                        for (int t = 0; t < NT; ++t) mma_f16(acc[m][t], a0, a1, a2, a3, bf[t].x, bf[t].y);
                        const __half2 x = __hmax2(__hmax2(__habs2(*reinterpret_cast<__half2 *>(&a0)), __habs2(*reinterpret_cast<__half2 *>(&a1))),
                                                  __hmax2(__habs2(*reinterpret_cast<__half2 *>(&a2)), __habs2(*reinterpret_cast<__half2 *>(&a3))));
                        const __half2 y = __hmax2(x, *reinterpret_cast<__half2 *>(&kmax2));
                        kmax2 = *reinterpret_cast<const uint32_t *>(&y);
                    }
                }
#pragma unroll
            for (int m = 0; m < C::MT; ++m)
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    float s = -INFINITY;
                    bool nan = false;
#pragma unroll
                    for (int t = 0; t < NT; ++t)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float x = acc[m][t][2 * half + e];
                            nan |= x != x;
                            s = fmaxf(s, x);
                        }
                    if (nan) s = INFINITY;
                    s = fmaxf(s, __shfl_xor_sync(0xffffffffu, s, 1));
                    s = fmaxf(s, __shfl_xor_sync(0xffffffffu, s, 2));
                    const int pl = 16 * m + 8 * half + (lane >> 2);
                    const int pg = __shfl_sync(0xffffffffu, id, pl);
                    if ((lane & 3) == 0 && p0 + pl < to) {
                        if (pg < 0) s = -INFINITY;
                        if (g0) s = fmaxf(s, scores[p0 + pl]);
                        scores[p0 + pl] = s;
                    }
                }
        }
    }
    {
        float k = fmaxf(__low2float(*reinterpret_cast<__half2 *>(&kmax2)), __high2float(*reinterpret_cast<__half2 *>(&kmax2)));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) k = fmaxf(k, __shfl_xor_sync(0xffffffffu, k, o));
        if (lane == 0) {
            s_kw[warp] = k;
            s_l1[warp] = l1;
        }
    }
    if (tid == 0) s_in = s_amb = s_cnt = 0;
    __syncthreads();
    if (CS > 1) {
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
        if (rank > 0) {  // hand the scores over to rank 0
            constexpr int PP = 16 * C::MT;
            const uint32_t dst = map_rank(ptx::smem_u32(scores), 0);
            for (int t = tid; ; t += kSelThreads) {
                const int pg = from + ((t / PP) * CS + rank) * PP + t % PP;
                if (pg >= to) {
                    if (from + ((t / PP) * CS + rank) * PP >= to) break;
                    continue;
                }
                st_cluster_f32(dst + 4u * (uint32_t)pg, scores[pg]);
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

    // ---- the choice
    float a_l1 = s_l1[0], a_k = s_kw[0];
    for (int w = 1; w < kSelWarps; ++w) {
        a_l1 = fmaxf(a_l1, s_l1[w]);
        a_k = fmaxf(a_k, s_kw[w]);
    }
    for (int r = 0; CS > 1 && r < CS; ++r) a_k = fmaxf(a_k, s_kmax[r]);
    float eps2 = 2.f * 0x1p-16f * a_l1 * a_k;
    if (!(eps2 < INFINITY)) eps2 = 0.f;  // a NaN query: every score is NaN, decided by index
    const int m = to - from, want = p.K - p.keep_first - p.keep_last;
    float t_hi = INFINITY, t_lo = INFINITY;
    if (want > 0) {
        int left;
        const unsigned int u = kth_largest<32, unsigned int>(m, want, hist, res, &left, [&](int j, unsigned int *v) {
            *v = order_f32(scores[from + j]);
            return true;
        });
        const float t = unorder_f32(u);
        t_hi = __fadd_ru(t, eps2);
        t_lo = __fsub_rd(t, eps2);
    }
    const int nw = (n + 31) >> 5;
    for (int w = warp; w < nw; w += kSelWarps) {
        const int pg = 32 * w + lane;
        bool in = pg < n && (pg < from || pg >= to), maybe = false;
        if (pg >= from && pg < to && want > 0) {
            const float s = scores[pg];
            in = s > t_hi;
            maybe = !in && s >= t_lo;
        }
        const unsigned int bi = __ballot_sync(0xffffffffu, in), bm = __ballot_sync(0xffffffffu, maybe);
        const unsigned int bs = __ballot_sync(0xffffffffu, in && pg >= from && pg < to);
        if (lane == 0) {
            sel[w] = bi;
            amb[w] = bm;
            atomicAdd(&s_in, __popc(bs));
            atomicAdd(&s_amb, __popc(bm));
        }
    }
    __syncthreads();
    const int slots = want - s_in;  // places for the undecided pages
    if (s_amb == slots) {
        for (int w = tid; w < nw; w += kSelThreads) sel[w] |= amb[w];
    } else if (slots > 0) {
        // 64-bit scores of the undecided pages, a warp per page; keys overwrite the fp32 scores
        for (int w = warp; w < nw; w += kSelWarps) {
            for (unsigned int bits = amb[w]; bits; bits &= bits - 1) {
                const int pg = 32 * w + __ffs(bits) - 1;
                const int id = bt[pg];
                unsigned long long key = 0;
                if (id >= 0 && id < p.num_pages) {
                    const uint8_t *src = bounds + (long long)id * p.b_s[0];
                    long long best = LLONG_MIN;
                    for (int h = 0; h < p.G; ++h) {
                        long long s = 0;
                        bool nan = false;
                        for (int c = lane; c < D; c += 32) {
                            const unsigned int qc = q[h * p.q_s[2] + c];
                            const unsigned int lc = src[c], hc = src[D + c];
                            const unsigned int bc = (qc & 0x80u) ? lc : hc;
                            nan |= (qc & 0x7Fu) == 0x7Fu || (lc & 0x7Fu) == 0x7Fu || (hc & 0x7Fu) == 0x7Fu;
                            s += (long long)fixed_e4m3(qc) * fixed_e4m3(bc);
                        }
#pragma unroll
                        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
                        if (__any_sync(0xffffffffu, nan)) s = LLONG_MAX;
                        best = max(best, s);
                    }
                    key = (unsigned long long)best ^ 0x8000000000000000ull;
                }
                if (lane == 0) keys[pg] = key;
            }
        }
        __syncthreads();
        if (s_amb <= 256) {
            // by rank among the undecided
            for (int w = tid; w < nw; w += kSelThreads)
                for (unsigned int bits = amb[w]; bits; bits &= bits - 1) s_list[atomicAdd(&s_cnt, 1)] = 32 * w + __ffs(bits) - 1;
            __syncthreads();
            if (tid < s_amb) {
                const int pg = s_list[tid];
                const unsigned long long key = keys[pg];
                int ahead = 0;
                for (int j = 0; j < s_amb; ++j) {
                    const int o = s_list[j];
                    ahead += keys[o] > key || (keys[o] == key && o < pg);
                }
                if (ahead < slots) atomicOr(&sel[pg >> 5], 1u << (pg & 31));
            }
        } else {
            int left;
            const unsigned long long t = kth_largest<64, unsigned long long>(n, slots, hist, res, &left, [&](int j, unsigned long long *v) {
                if (!(amb[j >> 5] >> (j & 31) & 1u)) return false;
                *v = keys[j];
                return true;
            });
            if (warp == 0) {  // ties at the threshold in index order
                for (int w = 0; w < nw; ++w) {
                    const bool on = amb[w] >> lane & 1u;
                    const unsigned long long key = on ? keys[32 * w + lane] : 0;
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
    __syncthreads();
    // ---- the chosen pages in ascending order: thread t lists words [t per, (t + 1) per)
    const int per = (nw + kSelThreads - 1) / kSelThreads;
    int cnt = 0;
    for (int w = tid * per; w < min(nw, (tid + 1) * per); ++w) cnt += __popc(sel[w]);
    int incl = cnt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
    }
    if (lane == 31) s_scan[warp] = incl;
    __syncthreads();
    int at = incl - cnt;
    for (int w = 0; w < warp; ++w) at += s_scan[w];
    for (int w = tid * per; w < min(nw, (tid + 1) * per); ++w)
        for (unsigned int bits = sel[w]; bits; bits &= bits - 1)
            if (at < p.K) out[at++] = 32 * w + __ffs(bits) - 1;
}

template <int D, int NT>
cudaError_t launch_select(const SelectParams &p, unsigned int rows, cudaStream_t s) {
    const int smem = SelCfg<D, NT>::smem(p.tab.max_pages);
    cudaError_t e = cudaFuncSetAttribute(select_pages_kernel<D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
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
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, select_pages_kernel<D, NT>, p);
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
    const long long items = (long long)p.npg * p.chunks;
    const long long per_req = (items + fa8::kBoundsThreads - 1) / fa8::kBoundsThreads;
    if (items > 0x7fffffffLL - fa8::kBoundsThreads || per_req * B > 0x7fffffffLL)
        return fail(FA8_ERR_UNSUPPORTED, "problem too large for the grid");
    p.blocks_per_req = (int)per_req;
    DeviceState *ds = nullptr;
    if ((st = device_state(&ds))) return st;
    p.status = ds->status;
    fa8::page_bounds_kernel<<<(unsigned)(per_req * B), fa8::kBoundsThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
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
    // Few (token, kv-head) pairs: a cluster of CTAs shares each pair's pages, as long as every CTA
    // keeps two steps of its eight warps (512 pages) and the clusters fit the GPU at once.
    p.cluster = 1;
    while (p.cluster < fa8::kSelMaxCluster && rows * p.cluster * 2 <= ds->sm_count && p.tab.max_pages >= 256 * p.cluster * 2)
        p.cluster *= 2;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e = cudaErrorInvalidValue;
#define FA8_SELECT(D_)                                                                   \
    case D_:                                                                             \
        e = p.G <= 8 ? fa8::launch_select<D_, 1>(p, (unsigned)rows, s) : fa8::launch_select<D_, 2>(p, (unsigned)rows, s); \
        break;
    switch (qs.D) {
        FA8_SELECT(64)
        FA8_SELECT(96)
        FA8_SELECT(128)
        FA8_SELECT(192)
        FA8_SELECT(256)
    }
#undef FA8_SELECT
    if (e != cudaSuccess) return cuda_fail(e, "page selection kernel launch");
    return FA8_SUCCESS;
}

}  // extern "C"
