// fa8_rope.cu -- rotary positions, E4M3 rounding and the append to the K/V cache in one pass
// (fa8_rope_append), and the rotary frequencies of long contexts (fa8_rope_inv_freq, host).
//
//   (y0, y1) = rot_scale * (x0 cos a - x1 sin a, x0 sin a + x1 cos a),  a = pos * w_i
//   out      = e4m3(y / descale), saturating at +-448
//
// Angles: w_i / 2pi is held as a 64-bit fixed-point fraction of a turn, so pos * w_i modulo one
// turn is the low 64 bits of an integer product: exact at every position (an fp32 angle is off
// by 2^-24 of itself, 0.06 rad at position 2^20), and no range reduction follows.
//
// Bound: HBM, 2 bytes read and 1 written per element; short of it, latency: 17 warps an SM wait for their loads
// (issue slots 51 % used).  A thread
// keeps the same 16 dims of a head over the heads of one token, so its 8 pairs of sines serve all of
// them, arithmetic goes two values an instruction, and no barrier follows the loads.  Measured from a graph's
// replays, 8192 tokens of 32 + 2 x 8 heads of 128 dims (151 MB): 29 us, 5.2 TB/s, 0.77 of the copy rate (as
// called, inputs changing: 33; with the rounded reciprocal alone, which moves values halfway between two: 28);
// sines through shared memory, four tokens a CTA: 57 us; sincospif per pair and heads by select: 46 us; one decode
// token: 3.1 us.
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

struct RopeParams {
    const void *q, *k, *v;  // 16-bit inputs; strides in elements {request, token, head}
    long long q_s[3], k_s[3], v_s[3];
    uint8_t *qo, *ko, *vo;  // E4M3 outputs; K/V: {request or page, row, head}
    long long qo_s[3], ko_s[3], vo_s[3];
    const void *inv_freq;
    int freq_f64;
    const int *pos;  // may be null
    long long pos_s[2];
    float rot_scale;
    int rot, rot_off;
    const float *dq, *dk, *dv;
    long long dq_s[2], dk_s[2], dv_s[2];
    int T, B, Sq, Hq, Hkv, G, D, DV;
    unsigned int g_magic;  // ceil(2^32 / G): q-head -> kv-head
    const int *cu_q, *cu_k;  // null: batched
    int kv_mode, Sk, total_k, num_pages;
    host::Table tab;
    unsigned int *status;
};

constexpr int kRopeThreads = 128;
constexpr int kRopeMaxPairs = 128;

// w / 2pi modulo 1 in units of 2^-64 turns, from the bits of w = M 2^(e - 63): the high word of
// M * (2^66 / 2pi) carries e - 1 binary places.  Integers, because fp64 arithmetic is slow here.
__device__ __forceinline__ unsigned long long turns_of(const void *freq, int f64, int i) {
    unsigned long long M;
    int e;
    bool neg;
    if (f64) {
        const unsigned long long u = static_cast<const unsigned long long *>(freq)[i];
        e = (int)(u >> 52) & 2047;
        M = e ? (u << 11) | 0x8000000000000000ull : 0;
        e -= 1023;
        neg = u >> 63;
    } else {
        const unsigned int u = static_cast<const unsigned int *>(freq)[i];
        e = (int)(u >> 23) & 255;
        M = e ? ((unsigned long long)u << 40) | 0x8000000000000000ull : 0;
        e -= 127;
        neg = u >> 31;
    }
    const unsigned long long hi = __umul64hi(M, 0xA2F9836E4E44152Aull);  // 2^66 / 2pi
    const unsigned long long t = e <= 1 ? (1 - e < 64 ? hi >> (1 - e) : 0) : (e - 1 < 64 ? hi << (e - 1) : 0);
    return neg ? 0 - t : t;
}

__device__ __forceinline__ uint64_t fmul2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// Cosine and sine of two angles given in 2^-32 turns.  The nearest quarter turn is split off as an
// integer; the rest, at most pi / 4, goes through the Taylor series to x^9 and x^8 (truncated below
// 2e-9 and 3e-8), two angles per packed instruction.
__device__ __forceinline__ void cossin2(unsigned int ph0, unsigned int ph1, uint64_t &co, uint64_t &si) {
    const unsigned int q0 = (ph0 + 0x20000000u) >> 30, q1 = (ph1 + 0x20000000u) >> 30;
    constexpr float kUnit = 1.4629180792671596e-9f;  // 2 pi / 2^32
    const uint64_t x = fmul2(ptx::f2pack((float)(int)(ph0 - (q0 << 30)), (float)(int)(ph1 - (q1 << 30))), ptx::f2pack(kUnit, kUnit));
    const uint64_t z = fmul2(x, x);
    auto both = [](float v) { return ptx::f2pack(v, v); };
    uint64_t s = ptx::ffma2(z, both(1.f / 362880.f), both(-1.f / 5040.f));
    s = ptx::ffma2(z, s, both(1.f / 120.f));
    s = ptx::ffma2(z, s, both(-1.f / 6.f));
    s = ptx::ffma2(fmul2(x, z), s, x);
    uint64_t c = ptx::ffma2(z, both(1.f / 40320.f), both(-1.f / 720.f));
    c = ptx::ffma2(z, c, both(1.f / 24.f));
    c = ptx::ffma2(z, c, both(-0.5f));
    c = ptx::ffma2(z, c, both(1.f));
    float s0, s1, c0, c1;
    ptx::f2unpack(s, s0, s1);
    ptx::f2unpack(c, c0, c1);
    // quarter turns: odd ones swap the two, the sine is negative in 2 and 3, the cosine in 1 and 2
    auto flip = [](float v, unsigned int q) { return __uint_as_float(__float_as_uint(v) ^ ((q & 2u) << 30)); };
    co = ptx::f2pack(flip(q0 & 1 ? s0 : c0, q0 + 1), flip(q1 & 1 ? s1 : c1, q1 + 1));
    si = ptx::f2pack(flip(q0 & 1 ? c0 : s0, q0), flip(q1 & 1 ? c1 : s1, q1));
}

// A 16-bit pair as two fp32 in one 64-bit register (the low half first).
__device__ __forceinline__ uint64_t widen2(uint32_t x, __nv_bfloat16) {
    return ptx::f2pack(__uint_as_float(x << 16), __uint_as_float(x & 0xFFFF0000u));
}
__device__ __forceinline__ uint64_t widen2(uint32_t x, __half) {
    float lo, hi;
    ptx::h2_to_f32(x, lo, hi);
    return ptx::f2pack(lo, hi);
}
// Division by one descale, as x hi + x lo with one rounding: hi + lo is 1 / d to 2^-40 (while d is below 2^100 and
// lo not subnormal), so that a quotient halfway between two E4M3 values stays there.  hi is below 1 / d, so lo is
// positive and an infinity meets one of its own sign.
struct Divisor {
    uint64_t hi, lo;
    __device__ __forceinline__ explicit Divisor(float d) {
        const float h = 0.25f * __fdividef(1.f - 0x1p-21f, 0.25f * d);  // defined from 2^-126 to 2^126
        const float l = fmaxf(h * fmaf(-h, d, 1.f), 0x1p-149f);
        hi = ptx::f2pack(h, h);
        lo = ptx::f2pack(l, l);
    }
    __device__ __forceinline__ uint64_t operator()(uint64_t x) const { return ptx::ffma2(x, hi, fmul2(x, lo)); }
};
// four fp32 (two pairs) -> four E4M3 bytes
__device__ __forceinline__ uint32_t round4(uint64_t a, uint64_t b) {
    float a0, a1, b0, b1;
    ptx::f2unpack(a, a0, a1);
    ptx::f2unpack(b, b0, b1);
    return ptx::prmt_lo16(ptx::cvt_e4m3x2(a1, a0), ptx::cvt_e4m3x2(b1, b0));
}

// Rotates (ROT: where `on`), divides and rounds one thread's 16 dims: two groups of 8, `gap` apart.  A warp
// holds rotated dims and others, so both go through the rotation and the others drop it: exactly, also
// beside an infinity.
template <typename T, bool INTER, bool ROT>
__device__ __forceinline__ void rope_store(uint8_t *dst, int gap, const uint4 &ra, const uint4 &rb, const Divisor &div, bool on,
                                           const uint64_t (&cc)[INTER ? 8 : 4], const uint64_t (&ss)[INTER ? 8 : 4],
                                           const uint64_t (&ns)[INTER ? 1 : 4]) {
    const uint32_t wa[4] = {ra.x, ra.y, ra.z, ra.w}, wb[4] = {rb.x, rb.y, rb.z, rb.w};
    uint64_t a[4], c[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        a[e] = widen2(wa[e], T());
        c[e] = widen2(wb[e], T());
        if constexpr (ROT && INTER) {  // (x0, x1) {c, c} + (x1, x0) {-s, s}
            float x0, x1;
            ptx::f2unpack(a[e], x0, x1);
            const uint64_t y = ptx::ffma2(a[e], cc[e], fmul2(ptx::f2pack(x1, x0), ss[e]));
            a[e] = on ? y : a[e];
            ptx::f2unpack(c[e], x0, x1);
            const uint64_t z = ptx::ffma2(c[e], cc[4 + e], fmul2(ptx::f2pack(x1, x0), ss[4 + e]));
            c[e] = on ? z : c[e];
        } else if constexpr (ROT) {
            const uint64_t y = ptx::ffma2(a[e], cc[e], fmul2(c[e], ns[e]));
            const uint64_t z = ptx::ffma2(a[e], ss[e], fmul2(c[e], cc[e]));
            a[e] = on ? y : a[e];
            c[e] = on ? z : c[e];
        }
        a[e] = div(a[e]);
        c[e] = div(c[e]);
    }
    *reinterpret_cast<uint2 *>(dst) = make_uint2(round4(a[0], a[1]), round4(a[2], a[3]));
    *reinterpret_cast<uint2 *>(dst + gap) = make_uint2(round4(c[0], c[1]), round4(c[2], c[3]));
}

// A thread: 16 dims (x) of every blockDim.y-th head of one token.  blockDim = (D / 16, head lanes,
// tokens).  ALL: every dim is rotated.  The loads of its first K and V head and of a batch of NB q-heads go
// out first; the angles of its 8 pairs, shared by all heads, and the cache slot are computed while they are in
// flight.
template <typename T, bool INTER, int NB, bool ALL>
__global__ void __launch_bounds__(kRopeThreads, 5) rope_append_kernel(const __grid_constant__ RopeParams p) {
    __shared__ __align__(16) unsigned long long turn[kRopeMaxPairs];
    const int x = threadIdx.x, Y = blockDim.y * gridDim.y;
    const int y = blockIdx.y * blockDim.y + threadIdx.y;
    const int tid = (threadIdx.z * blockDim.y + threadIdx.y) * blockDim.x + x;
    const long long tok = (long long)blockIdx.x * blockDim.z + threadIdx.z;

    // ---- this thread's two groups of 8 dims: both halves of 8 pairs, or 16 dims that pass through
    int da, gap;
    const bool rotated = x < (p.rot >> 4);
    if (rotated) {
        da = p.rot_off + (INTER ? 16 : 8) * x;
        gap = INTER ? 8 : p.rot >> 1;
    } else {
        const int g = 2 * (x - (p.rot >> 4)), first = p.rot_off >> 3;  // 8-dim groups ahead of the rotated ones
        da = 8 * g + (g < first ? 0 : p.rot);
        gap = 8 * (g + 1) + (g + 1 < first ? 0 : p.rot) - da;
    }
    int b = 0, i = 0, Lq = 0;
    const bool live = tok < p.T && locate_token(p.cu_q, p.B, p.Sq, (int)tok, &b, &i, &Lq);
    const long long bb = p.cu_q ? 0 : b, tt = p.cu_q ? tok : i;
    auto load = [](const T *s, int gap, uint4 &a, uint4 &b) {
        a = __ldcs(reinterpret_cast<const uint4 *>(s));
        b = __ldcs(reinterpret_cast<const uint4 *>(s + gap));
    };
    const T *sq = static_cast<const T *>(p.q) + bb * p.q_s[0] + tt * p.q_s[1] + y * p.q_s[2] + da;
    const T *sk = static_cast<const T *>(p.k) + bb * p.k_s[0] + tt * p.k_s[1] + y * p.k_s[2] + da;
    const T *sv = static_cast<const T *>(p.v) + bb * p.v_s[0] + tt * p.v_s[1] + y * p.v_s[2] + 16 * x;
    const long long step_q = Y * p.q_s[2];
    uint4 ka, kb, va, vb, qa[NB], qb[NB];
    float kd = 1.f, vd = 1.f, qd[NB];
    auto descale = [&](const float *d, const long long *s, int h) { return d ? __ldg(d + b * s[0] + h * s[1]) : 1.f; };
    auto group = [&](int h) { return p.G == 1 ? h : (int)__umulhi((unsigned)h, p.g_magic); };
    const bool has_v = 16 * x < p.DV;
    if (live) {
        if (y < p.Hkv) {
            load(sk, gap, ka, kb);
            kd = descale(p.dk, p.dk_s, y);
            if (has_v) load(sv, 8, va, vb);
            vd = descale(p.dv, p.dv_s, y);
        }
#pragma unroll
        for (int k = 0; k < NB; ++k)
            if (y + k * Y < p.Hq) {
                load(sq + k * step_q, gap, qa[k], qb[k]);
                qd[k] = descale(p.dq, p.dq_s, group(y + k * Y));
            }
    }
    for (int k = tid; k < (p.rot >> 1); k += blockDim.x * blockDim.y * blockDim.z) turn[k] = turns_of(p.inv_freq, p.freq_f64, k);
    __syncthreads();
    if (!live) return;
    // ---- cache slot and position
    int kstart = 0, Lk = p.Sk;
    if (p.kv_mode != 0) {
        kstart = p.cu_k[b];
        Lk = p.cu_k[b + 1] - kstart;
    }
    const int j = Lk - Lq + i;  // key index of this token
    const bool none = j < 0 && Lk >= 0;  // more new tokens than keys (a padded slot): nothing to append
    bool ok = j >= 0 && Lk >= 0;
    long long outer = b, row = j;
    if (ok && p.kv_mode == 2) {
        const int pi = j / p.tab.page_size;
        int page = -1;
        if (pi < p.tab.max_pages) page = p.tab.bt[(long long)b * p.tab.bt_stride + pi];
        ok = page >= 0 && page < p.num_pages;
        outer = page;
        row = j - pi * p.tab.page_size;
    } else if (p.kv_mode == 1) {
        outer = 0;
        row = (long long)kstart + j;
        ok = ok && kstart >= 0 && row < p.total_k;
    }
    if (!ok && !none && x == 0 && y == 0) atomicOr(p.status, kStatusBounds);
    // ---- cosines and sines of its 8 pairs, packed as rope_store takes them
    uint64_t cc[INTER ? 8 : 4] = {}, ss[INTER ? 8 : 4] = {}, ns[INTER ? 1 : 4] = {};
    if (rotated) {
        const int pos = p.pos ? p.pos[bb * p.pos_s[0] + tt * p.pos_s[1]] : j;
        const uint64_t rs = ptx::f2pack(p.rot_scale, p.rot_scale);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            unsigned int ph[2];
#pragma unroll
            for (int f = 0; f < 2; ++f) {  // position * turn, the upper half of its fraction
                const unsigned long long w = turn[8 * x + 2 * e + f];
                ph[f] = __umulhi((unsigned)pos, (unsigned)w) + (unsigned)pos * (unsigned)(w >> 32);
                if (pos < 0) ph[f] -= (unsigned)w;
            }
            uint64_t co, si;
            cossin2(ph[0], ph[1], co, si);
            co = fmul2(co, rs);
            si = fmul2(si, rs);
            float s0, s1, c0, c1;
            ptx::f2unpack(si, s0, s1);
            ptx::f2unpack(co, c0, c1);
            if constexpr (INTER) {
                cc[2 * e] = ptx::f2pack(c0, c0);
                cc[2 * e + 1] = ptx::f2pack(c1, c1);
                ss[2 * e] = ptx::f2pack(-s0, s0);
                ss[2 * e + 1] = ptx::f2pack(-s1, s1);
            } else {
                cc[e] = co;
                ss[e] = si;
                ns[e] = ptx::f2pack(-s0, -s1);
            }
        }
    }
    auto store = [&](uint8_t *dst, const uint4 &a, const uint4 &c, float d) {
        rope_store<T, INTER, true>(dst, gap, a, c, Divisor(d), ALL || rotated, cc, ss, ns);
    };
    if (ok) {
        uint8_t *dk = p.ko + outer * p.ko_s[0] + row * p.ko_s[1] + da;
        uint8_t *dv = p.vo + outer * p.vo_s[0] + row * p.vo_s[1] + 16 * x;
        for (int h = y; h < p.Hkv; h += Y) {
            store(dk + h * p.ko_s[2], ka, kb, kd);
            if (has_v) rope_store<T, INTER, false>(dv + h * p.vo_s[2], 8, va, vb, Divisor(vd), false, cc, ss, ns);
            if (h + Y < p.Hkv) {
                sk += Y * p.k_s[2];
                sv += Y * p.v_s[2];
                load(sk, gap, ka, kb);
                kd = descale(p.dk, p.dk_s, h + Y);
                if (has_v) load(sv, 8, va, vb);
                vd = descale(p.dv, p.dv_s, h + Y);
            }
        }
    }
    uint8_t *dq = p.qo + bb * p.qo_s[0] + tt * p.qo_s[1] + y * p.qo_s[2] + da;
    const long long step_o = Y * p.qo_s[2];
    for (int h = y; h < p.Hq; h += NB * Y) {
#pragma unroll
        for (int k = 0; k < NB; ++k) {
            if (h + k * Y < p.Hq) {
                store(dq, qa[k], qb[k], qd[k]);
                if (h + (k + NB) * Y < p.Hq) {
                    load(sq + (k + NB) * step_q, gap, qa[k], qb[k]);
                    qd[k] = descale(p.dq, p.dq_s, group(h + (k + NB) * Y));
                }
            }
            dq += step_o;
        }
        sq += NB * step_q;
    }
}

template <typename T, bool INTER, int NB>
cudaError_t launch_rope_batch(const RopeParams &p, int lanes, int spread, cudaStream_t s) {
    const int xs = p.D / 16;
    const int ys = std::max(1, std::min(lanes, kRopeThreads / xs)), zs = kRopeThreads / (xs * ys);
    const dim3 grid((unsigned)(((long long)p.T + zs - 1) / zs), (unsigned)((spread + ys - 1) / ys));
    if (p.rot == p.D) rope_append_kernel<T, INTER, NB, true><<<grid, dim3(xs, ys, zs), 0, s>>>(p);
    else rope_append_kernel<T, INTER, NB, false><<<grid, dim3(xs, ys, zs), 0, s>>>(p);
    return cudaGetLastError();
}

template <typename T, bool INTER>
cudaError_t launch_rope(const RopeParams &p, int sm_count, cudaStream_t s) {
    // Enough tokens for two CTAs per SM: half as many head lanes as kv-heads, four at most, so that a
    // thread's heads share its angles (8192 tokens of 32 + 2 x 8 heads, d = 128: 29 us with four lanes,
    // 31 with eight, 32 with two).  Fewer: a lane per q-head, and the heads over several CTAs, to shorten
    // the chain.
    const int lanes = std::max(1, std::min(p.Hkv / 2, 4));
    if ((long long)p.T * lanes * (p.D / 16) >= 2LL * sm_count * kRopeThreads) return launch_rope_batch<T, INTER, 2>(p, lanes, 1, s);
    return launch_rope_batch<T, INTER, 1>(p, p.Hq, p.Hq, s);
}

}  // namespace fa8

namespace {

using namespace fa8::host;

// 16-bit input (B, Sq, H, d) or (total, H, d): last dim contiguous, 16-byte base and strides.
fa8_status check_input(const fa8_tensor *t, const char *name, int dtype, int ndim, long long s[3]) {
    if (t->dtype != dtype) return fail(FA8_ERR_INVALID_ARG, "q, k and v must have one dtype (bf16 or fp16): %s differs", name);
    if (t->ndim != ndim) return fail(FA8_ERR_INVALID_ARG, "%s must have q's rank", name);
    if (t->shape[ndim - 1] > 1 && t->stride[ndim - 1] != 1)
        return fail(FA8_ERR_INVALID_ARG, "%s: last dim must be contiguous", name);
    for (int i = 0; i < ndim - 1; ++i) {
        if (t->shape[i] < 0) return fail(FA8_ERR_INVALID_ARG, "%s: negative extent", name);
        if (t->shape[i] > 1 && (t->stride[i] % 8 != 0 || t->stride[i] < 0))
            return fail(FA8_ERR_INVALID_ARG, "%s: stride[%d]=%lld must be a non-negative multiple of 8 elements", name, i,
                        (long long)t->stride[i]);
    }
    if (!aligned16(t->data)) return fail(FA8_ERR_INVALID_ARG, "%s: data must be 16-byte aligned", name);
    s[0] = ndim == 4 && t->shape[0] > 1 ? t->stride[0] : 0;
    s[1] = t->shape[ndim - 3] > 1 ? t->stride[ndim - 3] : 0;
    s[2] = t->shape[ndim - 2] > 1 ? t->stride[ndim - 2] : 0;
    return FA8_SUCCESS;
}

}  // namespace

extern "C" {

fa8_status fa8_rope_inv_freq(int rotary_dim, double base, int scaling, double factor, double original_len,
                             double low, double high, double *inv_freq) {
    clear_error();
    if (!inv_freq) return fail(FA8_ERR_INVALID_ARG, "inv_freq is required");
    if (rotary_dim <= 0 || rotary_dim % 2 != 0 || rotary_dim > 65536)
        return fail(FA8_ERR_INVALID_ARG, "rotary_dim must be a positive even number");
    if (!(base > 1.0) || !std::isfinite(base)) return fail(FA8_ERR_INVALID_ARG, "base must be finite and above 1");
    if (scaling < FA8_ROPE_PLAIN || scaling > FA8_ROPE_BANDS) return fail(FA8_ERR_INVALID_ARG, "unknown rotary scaling %d", scaling);
    if (scaling != FA8_ROPE_PLAIN && (!(factor >= 1.0) || !std::isfinite(factor)))
        return fail(FA8_ERR_INVALID_ARG, "factor must be finite and at least 1");
    if (scaling == FA8_ROPE_YARN || scaling == FA8_ROPE_BANDS) {
        if (!(original_len > 0.0) || !std::isfinite(original_len))
            return fail(FA8_ERR_INVALID_ARG, "original_len must be positive");
        if (!(low > 0.0) || !(high > low) || !std::isfinite(high))
            return fail(FA8_ERR_INVALID_ARG, "0 < low < high is required");
    }
    if (scaling == FA8_ROPE_NTK && rotary_dim <= 2) return fail(FA8_ERR_INVALID_ARG, "NTK scaling needs rotary_dim > 2");
    const double two_pi = 6.283185307179586476925;
    const int half = rotary_dim / 2;
    if (scaling == FA8_ROPE_NTK) base *= std::pow(factor, (double)rotary_dim / (rotary_dim - 2));
    double from = 0.0, to = 1.0;
    if (scaling == FA8_ROPE_YARN) {
        // pair index at which a frequency makes n turns over the original length
        auto pair_of = [&](double n) { return rotary_dim * std::log(original_len / (n * two_pi)) / (2.0 * std::log(base)); };
        from = std::max(std::floor(pair_of(high)), 0.0);
        to = std::min(std::ceil(pair_of(low)), (double)rotary_dim - 1.0);
        if (!(to > from)) to = from + 0.001;
    }
    for (int i = 0; i < half; ++i) {
        const double w = std::pow(base, -2.0 * i / rotary_dim);
        double keep = 1.0;  // the part of w that stays; the rest is divided by factor
        if (scaling == FA8_ROPE_LINEAR) keep = 0.0;
        else if (scaling == FA8_ROPE_YARN) keep = 1.0 - std::min(1.0, std::max(0.0, (i - from) / (to - from)));
        else if (scaling == FA8_ROPE_BANDS) keep = std::min(1.0, std::max(0.0, (original_len * w / two_pi - low) / (high - low)));
        inv_freq[i] = scaling == FA8_ROPE_PLAIN || scaling == FA8_ROPE_NTK ? w : w * keep + w / factor * (1.0 - keep);
    }
    return FA8_SUCCESS;
}

fa8_status fa8_rope_append(const fa8_tensor *q, const fa8_tensor *k, const fa8_tensor *v, const fa8_tensor *inv_freq,
                           const fa8_tensor *positions, int interleaved, int rotary_offset, float rot_scale,
                           const fa8_tensor *descale_q, const fa8_tensor *descale_k, const fa8_tensor *descale_v,
                           fa8_tensor *q_out, fa8_tensor *k_out, fa8_tensor *v_out, const fa8_tensor *cu_seqlens_q,
                           const fa8_tensor *cu_seqlens_k, const fa8_tensor *block_table, int page_size, void *stream) {
    clear_error();
    if (!q || !k || !v || !inv_freq || !q_out || !k_out || !v_out)
        return fail(FA8_ERR_INVALID_ARG, "q, k, v, inv_freq, q_out, k_out and v_out are required");
    if (q->dtype != FA8_DTYPE_BF16 && q->dtype != FA8_DTYPE_F16) return fail(FA8_ERR_UNSUPPORTED, "q, k and v must be bf16 or fp16");
    if (q->ndim != 3 && q->ndim != 4) return fail(FA8_ERR_INVALID_ARG, "q must have 3 or 4 dims");
    fa8::RopeParams p;
    memset(&p, 0, sizeof(p));
    fa8_status st;
    const int nd = q->ndim;
    if ((st = check_input(q, "q", q->dtype, nd, p.q_s)) || (st = check_input(k, "k", q->dtype, nd, p.k_s)) ||
        (st = check_input(v, "v", q->dtype, nd, p.v_s)))
        return st;
    for (int i = 0; i < nd - 2; ++i)
        if (k->shape[i] != q->shape[i] || v->shape[i] != q->shape[i])
            return fail(FA8_ERR_INVALID_ARG, "q, k and v must hold the same tokens (dim %d differs)", i);
    const long long D = q->shape[nd - 1], DV = v->shape[nd - 1], Hq = q->shape[nd - 2], Hkv = k->shape[nd - 2];
    if (k->shape[nd - 1] != D) return fail(FA8_ERR_INVALID_ARG, "k head dim %lld != q head dim %lld", (long long)k->shape[nd - 1], D);
    if (D > 1024 || DV > 1024 || !supported_dims((int)D, (int)DV))
        return fail(FA8_ERR_UNSUPPORTED, "(d, dv) = (%lld, %lld) is not supported", D, DV);
    if (v->shape[nd - 2] != Hkv) return fail(FA8_ERR_INVALID_ARG, "k and v must have the same heads");
    if (Hkv <= 0 || Hq <= 0 || Hq % Hkv != 0 || Hq > 65536)
        return fail(FA8_ERR_INVALID_ARG, "q heads (%lld) must be a positive multiple of kv heads (%lld)", Hq, Hkv);
    // ---- tokens
    long long B, T;
    if (nd == 4) {
        if (cu_seqlens_q) return fail(FA8_ERR_INVALID_ARG, "cu_seqlens_q is only valid with a 3-D (varlen) q");
        B = q->shape[0];
        T = B * q->shape[1];
        p.Sq = (int)q->shape[1];
    } else {
        if (!cu_seqlens_q) return fail(FA8_ERR_INVALID_ARG, "a 3-D (varlen) q needs cu_seqlens_q");
        if (cu_seqlens_q->ndim != 1 || cu_seqlens_q->shape[0] < 2)
            return fail(FA8_ERR_INVALID_ARG, "cu_seqlens_q must have B+1 >= 2 entries");
        B = cu_seqlens_q->shape[0] - 1;
        T = q->shape[0];
        if ((st = check_int_vec(cu_seqlens_q, "cu_seqlens_q", B + 1))) return st;
        p.cu_q = static_cast<const int *>(cu_seqlens_q->data);
    }
    if (B <= 0 || B > 0x7fffffffLL - 1) return fail(FA8_ERR_INVALID_ARG, "batch must be >= 1");
    if (T > 0x7fffffffLL - 4) return fail(FA8_ERR_UNSUPPORTED, "too many tokens");
    p.B = (int)B;
    p.T = (int)T;
    p.Hq = (int)Hq;
    p.Hkv = (int)Hkv;
    p.G = (int)(Hq / Hkv);
    p.g_magic = p.G > 1 ? (unsigned)((0x100000000ull + p.G - 1) / p.G) : 0u;
    p.D = (int)D;
    p.DV = (int)DV;
    // ---- rotation
    if (inv_freq->dtype != FA8_DTYPE_F64 && inv_freq->dtype != FA8_DTYPE_F32)
        return fail(FA8_ERR_INVALID_ARG, "inv_freq must be fp64 or fp32");
    if (inv_freq->ndim != 1 || inv_freq->shape[0] < 1 || (inv_freq->shape[0] > 1 && inv_freq->stride[0] != 1) || !inv_freq->data)
        return fail(FA8_ERR_INVALID_ARG, "inv_freq must be a contiguous 1-D tensor of rotary_dim / 2 entries");
    const long long rot = 2 * inv_freq->shape[0];
    if (rot % 16 != 0) return fail(FA8_ERR_UNSUPPORTED, "rotary_dim (%lld) must be a multiple of 16", rot);
    if (rotary_offset < 0 || rotary_offset % 8 != 0)
        return fail(FA8_ERR_UNSUPPORTED, "rotary_offset must be a non-negative multiple of 8");
    if (rot + rotary_offset > D)
        return fail(FA8_ERR_INVALID_ARG, "rotary_offset %d + rotary_dim %lld is past the head dim %lld", rotary_offset, rot, D);
    if (interleaved != 0 && interleaved != 1) return fail(FA8_ERR_INVALID_ARG, "interleaved must be 0 or 1");
    if (!std::isfinite(rot_scale)) return fail(FA8_ERR_INVALID_ARG, "rot_scale must be finite");
    p.inv_freq = inv_freq->data;
    p.freq_f64 = inv_freq->dtype == FA8_DTYPE_F64;
    p.rot = (int)rot;
    p.rot_off = rotary_offset;
    p.rot_scale = rot_scale;
    if (positions) {
        if (positions->dtype != FA8_DTYPE_I32 || positions->ndim != nd - 2 || !positions->data)
            return fail(FA8_ERR_INVALID_ARG, "positions must be int32 with one entry per token");
        for (int i = 0; i < nd - 2; ++i)
            if (positions->shape[i] != q->shape[i]) return fail(FA8_ERR_INVALID_ARG, "positions must be int32 with one entry per token");
        p.pos = static_cast<const int *>(positions->data);
        p.pos_s[0] = nd == 4 ? positions->stride[0] : 0;
        p.pos_s[1] = positions->stride[nd - 3];
    }
    if ((st = check_descale(descale_q, "descale_q", p.B, p.Hkv, &p.dq, &p.dq_s[0], &p.dq_s[1])) ||
        (st = check_descale(descale_k, "descale_k", p.B, p.Hkv, &p.dk, &p.dk_s[0], &p.dk_s[1])) ||
        (st = check_descale(descale_v, "descale_v", p.B, p.Hkv, &p.dv, &p.dv_s[0], &p.dv_s[1])))
        return st;
    // ---- outputs
    for (const fa8_tensor *t : {q_out, k_out, v_out})
        if (t->dtype != FA8_DTYPE_E4M3) return fail(FA8_ERR_UNSUPPORTED, "q_out, k_out and v_out must be E4M3");
    if ((st = check_payload(q_out, "q_out")) || (st = check_payload(k_out, "k_out")) || (st = check_payload(v_out, "v_out"))) return st;
    if (q_out->ndim != nd) return fail(FA8_ERR_INVALID_ARG, "q_out must have q's shape");
    for (int i = 0; i < nd; ++i)
        if (q_out->shape[i] != q->shape[i]) return fail(FA8_ERR_INVALID_ARG, "q_out must have q's shape");
    if (k_out->ndim != v_out->ndim) return fail(FA8_ERR_INVALID_ARG, "k_out and v_out must have the same rank");
    const int kn = k_out->ndim;
    for (int i = 0; i < kn - 2; ++i)
        if (k_out->shape[i] != v_out->shape[i]) return fail(FA8_ERR_INVALID_ARG, "k_out and v_out leading shapes differ at dim %d", i);
    if (k_out->shape[kn - 1] != D || v_out->shape[kn - 1] != DV || k_out->shape[kn - 2] != Hkv || v_out->shape[kn - 2] != Hkv)
        return fail(FA8_ERR_INVALID_ARG, "k_out and v_out must end in (Hkv, d) and (Hkv, dv) of k and v");
    if (block_table) {
        if (kn != 4) return fail(FA8_ERR_INVALID_ARG, "paged k_out must be (num_pages, page_size, Hkv, d)");
        if ((st = check_table(cu_seqlens_k, block_table, page_size, p.B, &p.tab))) return st;
        if (page_size != k_out->shape[1]) return fail(FA8_ERR_INVALID_ARG, "page_size (%d) != k_out.shape[1] (%lld)", page_size, (long long)k_out->shape[1]);
        if (k_out->shape[0] > 0x7fffffffLL) return fail(FA8_ERR_UNSUPPORTED, "too many pages");
        p.kv_mode = 2;
        p.num_pages = (int)k_out->shape[0];
        p.cu_k = p.tab.cu_k;
    } else if (kn == 4) {
        if (cu_seqlens_k) return fail(FA8_ERR_INVALID_ARG, "cu_seqlens_k is only valid with varlen (3-D) or paged k_out");
        if (k_out->shape[0] != B) return fail(FA8_ERR_INVALID_ARG, "k_out batch (%lld) != q batch (%lld)", (long long)k_out->shape[0], B);
        if (k_out->shape[1] > 0x7fffffffLL) return fail(FA8_ERR_UNSUPPORTED, "too many keys");
        p.Sk = (int)k_out->shape[1];
    } else {
        if (!cu_seqlens_k) return fail(FA8_ERR_INVALID_ARG, "a 3-D (varlen) k_out needs cu_seqlens_k");
        if ((st = check_int_vec(cu_seqlens_k, "cu_seqlens_k", B + 1))) return st;
        if (k_out->shape[0] > 0x7fffffffLL) return fail(FA8_ERR_UNSUPPORTED, "too many keys");
        p.kv_mode = 1;
        p.total_k = (int)k_out->shape[0];
        p.cu_k = static_cast<const int *>(cu_seqlens_k->data);
    }
    if (T == 0) return FA8_SUCCESS;
    for (const fa8_tensor *t : {q, k, v, (const fa8_tensor *)q_out, (const fa8_tensor *)k_out, (const fa8_tensor *)v_out})
        if (!t->data && !(t != q_out && t->ndim == kn && t->shape[0] == 0))
            return fail(FA8_ERR_INVALID_ARG, "q, k, v, q_out, k_out and v_out need data");
    DeviceState *ds = nullptr;
    if ((st = device_state(&ds))) return st;
    p.q = q->data;
    p.k = k->data;
    p.v = v->data;
    p.qo = static_cast<uint8_t *>(q_out->data);
    p.ko = static_cast<uint8_t *>(k_out->data);
    p.vo = static_cast<uint8_t *>(v_out->data);
    for (int i = 0; i < 3; ++i) {
        p.qo_s[i] = nd == 4 ? q_out->stride[i] : (i ? q_out->stride[i - 1] : 0);
        p.ko_s[i] = kn == 4 ? k_out->stride[i] : (i ? k_out->stride[i - 1] : 0);
        p.vo_s[i] = kn == 4 ? v_out->stride[i] : (i ? v_out->stride[i - 1] : 0);
    }
    p.status = ds->status;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (q->dtype == FA8_DTYPE_BF16)
        e = interleaved ? fa8::launch_rope<__nv_bfloat16, true>(p, ds->sm_count, s) : fa8::launch_rope<__nv_bfloat16, false>(p, ds->sm_count, s);
    else
        e = interleaved ? fa8::launch_rope<__half, true>(p, ds->sm_count, s) : fa8::launch_rope<__half, false>(p, ds->sm_count, s);
    if (e != cudaSuccess) return cuda_fail(e, "rope append kernel launch");
    return FA8_SUCCESS;
}

}  // extern "C"
