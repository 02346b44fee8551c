// fa8_scored.cuh -- what the kernels of fa8_fwd_scored and fa8_fwd_tree share: parameters, which keys a
// token sees, and what becomes of a score before the softmax.
//
//   z = softmax_scale dq dk q.k;   z = cap tanh(z / cap);   z = z - slope |pos - j|,   pos = i + Lk - Lq
//
// All of it in log2 units (times log2 e), so that weights are 2^(z - m).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "fa8.h"
#include "fa8_kernel.cuh"
#include "fa8_pages.cuh"

namespace fa8 {

struct ScoredParams {
    int B, Hq, Hkv, G, Sq, total_q;  // Sq: tokens per request (batched q)
    const int *cu_q;                 // null: batched
    int kv_mode;                     // 0 batched, 1 varlen, 2 paged
    int Sk, total_k;
    const int *cu_k, *bt;
    long long bt_stride;
    int max_pages, page_size, num_pages;
    int has_kv;                      // K and V hold anything (their maps are valid)
    const uint8_t *q, *v;
    long long q_s[3];                // request, token, head
    long long v_s[3];                // request or page, row, head
    const float *dq, *dk, *dv;
    long long dq_s[2], dk_s[2], dv_s[2];
    const float *sink, *slopes;
    float scale_log2;                // softmax_scale log2 e
    float cap_log2;                  // cap log2 e; 0: none
    int causal, window_left;
    const int *ranges;
    long long r_s[2];                // request, token
    const int *masks;                // the tree's, or null
    long long m_s[2];
    int words;                       // of a mask
    void *o;
    long long o_s[3];
    int out_fp16;
    float *lse;
    long long lse_s[3];              // request, token, head
    unsigned long long timeout_ns;
    unsigned int *status;
    // many rows
    int P;                           // positions of a unit's 128 rows
    int units, blocks;               // units (not split); tiles of positions per request (batched)
    int steal;                       // a CTA per unit: those that run take over the others'
    int split, min_tiles;            // even shares of all tiles over the CTAs, at least so many each
    float *part;                     // split (whole units; few rows: [cluster][row][column], then (m, l)): [slot][column / 4][row] float4, then [slot][row] float2 (m, l), [CTA] int4 (a cut)
    int box_n, boxes, box_v;         // keys of one TMA box of K, its boxes for two tiles; keys of one of V's
    int step_e, step_r;              // two tiles further: so many pages, so many rows
    // few rows
    int parts;                       // clusters that share a request's keys
    int cluster, box_shift;
};

// What one request holds.
struct ScReq {
    int Lq, Lk, q0, k0;  // q0, k0: first token and key in the packed tensors (0: batched, paged)
};
// Bit 0: its tokens do not lie in the tensors; bit 1: its keys do not, it counts as having none.
__device__ __forceinline__ int sc_lengths(const ScoredParams &p, int b, ScReq *r) {
    r->q0 = p.cu_q ? p.cu_q[b] : 0;
    r->Lq = p.cu_q ? p.cu_q[b + 1] - r->q0 : p.Sq;
    r->k0 = 0;
    r->Lk = p.Sk;
    if (p.kv_mode != 0) {
        const int a = p.cu_k[b];
        r->Lk = p.cu_k[b + 1] - a;
        if (p.kv_mode == 1) r->k0 = a;
    }
    const bool bad_q = p.cu_q && (r->Lq < 0 || r->q0 < 0 || (long long)r->q0 + r->Lq > p.total_q);
    const bool bad_k = r->Lk < 0 || (r->Lk > 0 && !p.has_kv) ||
                       (p.kv_mode == 1 && (r->k0 < 0 || (long long)r->k0 + r->Lk > p.total_k)) ||
                       (p.kv_mode == 2 && r->Lk > (long long)p.max_pages * p.page_size);
    if (bad_k) r->Lk = r->k0 = 0;
    return (bad_q ? 1 : 0) | (bad_k ? 2 : 0);
}
// The same, with a status bit for the bad; false where its tokens are.
__device__ __forceinline__ bool sc_request(const ScoredParams &p, int b, ScReq *r) {
    const int bad = sc_lengths(p, b, r);
    if (bad && (threadIdx.x & 31) == 0) atomicOr(p.status, kStatusBounds);
    return !(bad & 1);
}

// The keys that token i of a request sees lie in [lo, hi); of those from `lp` on (a tree's drafted
// tokens) the ones whose bit is set.
struct ScRow {
    int lo, hi, lp;
    const int *words;
};
__device__ __forceinline__ ScRow sc_row(const ScoredParams &p, int b, const ScReq &rq, int i) {
    ScRow r;
    const int pos = i + rq.Lk - rq.Lq;
    r.lo = p.window_left >= 0 ? max(0, pos - p.window_left) : 0;
    r.hi = p.causal ? min(rq.Lk, pos + 1) : rq.Lk;
    r.lp = 0x7fffffff;
    r.words = nullptr;
    const long long bb = p.cu_q ? 0 : b, tt = p.cu_q ? rq.q0 + i : i;
    if (p.ranges) {
        const int *g = p.ranges + bb * p.r_s[0] + tt * p.r_s[1];
        r.lo = max(r.lo, g[0]);
        r.hi = min(r.hi, g[1]);
    }
    if (p.masks) {
        r.lp = rq.Lk - rq.Lq;
        r.words = p.masks + bb * p.m_s[0] + tt * p.m_s[1];
    }
    if (r.hi <= r.lo) r.lo = r.hi = 0;
    return r;
}
// Whether the row sees key j.
__device__ __forceinline__ bool sc_sees(const ScRow &r, int words, int j) {
    if (j < r.lo || j >= r.hi) return false;
    if (j < r.lp) return true;
    const int d = j - r.lp;
    return (d >> 5) < words && (r.words[d >> 5] >> (d & 31) & 1);
}
// The low n bits (n may be out of 0..32).
__device__ __forceinline__ uint32_t sc_low(int n) { return n <= 0 ? 0u : (n >= 32 ? 0xffffffffu : (1u << n) - 1u); }
// Bit e: whether the row sees key k + e.
__device__ __forceinline__ uint32_t sc_see32(const ScRow &r, int words, int k) {
    uint32_t m = sc_low(r.hi - k) & ~sc_low(r.lo - k);
    if (r.words && k + 32 > r.lp) {
        const int d = k - r.lp;  // above -32
        const int w = d >> 5, sh = d & 31;
        const uint32_t a = w >= 0 ? (w < words ? (uint32_t)r.words[w] : 0u) : 0xffffffffu;
        const uint32_t c = w + 1 < words ? (uint32_t)r.words[w + 1] : 0u;
        m &= __funnelshift_r(a, c, sh);
    }
    return m;
}

__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// 2 log2(e) c / cap, finite for the least caps too: a score of zero stays zero.
__device__ __forceinline__ float sc_k2(float c, float cap) { return fminf(fmaxf(2.f * kLog2e * c / cap, -0x1p100f), 0x1p100f); }
// cap tanh(z / cap) of z = s c, with k2 = 2 log2(e) c / cap.  With t = 2^(-|s k2|), tanh |x| = (1 - t) / (1 + t), to 2^-22
// absolutely: of a cap far above the scores that is more than the scores' own rounding.
__device__ __forceinline__ float sc_cap_near(float s, float k2, float cap) {
    const float x = s * k2, t = ptx::ex2(-fabsf(x));
    return copysignf(cap, x) * ((1.f - t) * rcp(1.f + t));
}
// Caps above 128, in log2 units, need more than that (sc_cap).
constexpr float kFarCap = 128.01f * kLog2e;
// To 2^-20 of itself: below a quarter of the cap 1 - t would cancel, and z is multiplied by the series of tanh(x) / x,
// 1 - x^2 / 3 + 2 x^4 / 15 - 17 x^6 / 315 + 62 x^8 / 2835, whose next term is under 2^-26 there.
constexpr float kCapSeries = 0.25f * 2.f * kLog2e;  // |s k2| up to which
__device__ __forceinline__ float sc_cap_series(float s, float c, float k2) {
    const float x = s * k2, w = x * x * (0.25f * kLn2 * kLn2);
    return s * c * fmaf(w, fmaf(w, fmaf(w, fmaf(w, 62.f / 2835.f, -17.f / 315.f), 2.f / 15.f), -1.f / 3.f), 1.f);
}
__device__ __forceinline__ float sc_cap(float s, float c, float k2, float cap) {
    return fabsf(s * k2) < kCapSeries ? sc_cap_series(s, c, k2) : sc_cap_near(s, k2, cap);
}

// The row's bias is -slope |pos - j|.  Seen from pc = pos moved into [lo, hi), which keeps its products
// small, it is -slope |pc - j| - slope |pos - pc|: the second part goes to the LSE alone.
struct ScBias {
    float slope, off;  // log2 units
    int pc;
};
__device__ __forceinline__ ScBias sc_bias(const ScoredParams &p, const ScRow &r, int pos, int hq) {
    ScBias b;
    b.slope = p.slopes[hq] * kLog2e;
    b.pc = min(max(pos, r.lo), max(r.hi - 1, r.lo));
    b.off = -b.slope * fabsf((float)(pos - b.pc));
    return b;
}

// Output factor and LSE of a row whose weights 2^(z - m) sum to l (m and l include the bias's offset).  The unit's
// reciprocal and logarithm are within 2^-22, the first relatively, and a tenth of the code that a division and log2f take,
// which the kernel's products wait for.
__device__ __forceinline__ float sc_top(float m, float l, const float *sink, float *sum, float *sc) {
    const float ref = m == -INFINITY ? 0.f : m;
    *sum = l;
    *sc = 1.f;
    if (!sink) return ref;
    const float sl = *sink * kLog2e, top = fmaxf(ref, sl);
    *sc = ptx::ex2(ref - top);
    *sum = l * *sc + ptx::ex2(sl - top);
    return top;
}
__device__ __forceinline__ float sc_factor(float m, float l, const float *sink, float dv) {
    float sum, sc;
    sc_top(m, l, sink, &sum, &sc);
    return m == -INFINITY && l == 0.f ? 0.f : sc * dv * rcp(sum);  // (no visible key)
}
__device__ __forceinline__ float sc_lse(float m, float l, const float *sink) {
    if (m == -INFINITY && l == 0.f) return sink ? *sink : -INFINITY;
    float sum, sc, y;
    const float top = sc_top(m, l, sink, &sum, &sc);
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(sum));
    return (y + top) * kLn2;
}
__device__ __forceinline__ void sc_finish(float m, float l, const float *sink, float dv, float *f, float *lse) {
    *f = sc_factor(m, l, sink, dv);
    *lse = sc_lse(m, l, sink);
}

// Address of a key's V row.
__device__ __forceinline__ const uint8_t *sc_v_row(const ScoredParams &p, int b, const ScReq &rq, int kvh, int j) {
    long long page = b, row = j;
    if (p.kv_mode == 1) {
        page = 0;
        row = (long long)rq.k0 + j;
    } else if (p.kv_mode == 2) {
        const int e = p.bt[b * p.bt_stride + j / p.page_size];
        if (e < 0 || e >= p.num_pages) return nullptr;  // reads as zeros
        page = e;
        row = j % p.page_size;
    }
    return p.v + page * p.v_s[0] + row * p.v_s[1] + kvh * p.v_s[2];
}
// NaNs of V in tiles that some rows see and others do not go into the products as zeros there: a masked weight of zero would not
// silence them.  The rows that see them get them at the end.
// 16 bytes of V: bit c, whether channel c holds a NaN.
__device__ __forceinline__ uint32_t sc_nans(const uint32_t (&w)[4]) {
    uint32_t bits = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const uint32_t n = ((w[e] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
        bits |= ((n >> 7 & 1u) | (n >> 14 & 2u) | (n >> 21 & 4u) | (n >> 28 & 8u)) << (4 * e);
    }
    return bits;
}

template <int D, int DV>
fa8_status launch_scored_many(ScoredParams &p, const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv, int grid, int dev,
                              cudaStream_t s);
template <int D, int DV>
fa8_status launch_scored_few(ScoredParams &p, const fa8_tensor *k, const fa8_tensor *v, int tiles, long long max_keys, int sm_count, int dev,
                             cudaStream_t s);

}  // namespace fa8
