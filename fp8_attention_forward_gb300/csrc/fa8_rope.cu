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
// Bound: HBM, 2 bytes read and 1 written per element.  A thread keeps the same 16 dims of a head
// over all heads of its tokens and loads two 16-byte groups (both halves of 8 pairs) of up to four
// tokens before it computes; the sines of a token are computed once, into shared memory, for all
// its heads.
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
    const int *cu_q, *cu_k;  // null: batched
    int kv_mode, Sk, total_k, num_pages;
    host::Table tab;
    unsigned int *status;
};

constexpr int kRopeThreads = 256;
constexpr int kRopeMaxPairs = 128;

__device__ __forceinline__ float2 unpack2(uint32_t x, __nv_bfloat16) {
    return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xFFFF0000u));
}
__device__ __forceinline__ float2 unpack2(uint32_t x, __half) {
    float lo, hi;
    ptx::h2_to_f32(x, lo, hi);
    return make_float2(lo, hi);
}

// One CTA: TB consecutive tokens.  blockDim = (D / 16, 256 / (D / 16)): x = 16 dims of a head, y
// (with grid y) = head among Hq q-heads, Hkv k-heads, Hkv v-heads.
template <typename T, bool INTER, int TB>
__global__ void __launch_bounds__(kRopeThreads) rope_append_kernel(const __grid_constant__ RopeParams p) {
    __shared__ unsigned long long turn[kRopeMaxPairs];  // w / 2pi, 2^-64 turns
    __shared__ float2 cs[TB][kRopeMaxPairs];
    __shared__ long long s_q[TB], s_k[TB], s_v[TB], s_qo[TB], s_ko[TB], s_vo[TB];
    __shared__ int s_pos[TB], s_b[TB];
    const int tid = threadIdx.y * blockDim.x + threadIdx.x;
    const int nthreads = blockDim.x * blockDim.y;
    const int pairs = p.rot >> 1;
    for (int i = tid; i < pairs; i += nthreads) {
        double f = p.freq_f64 ? static_cast<const double *>(p.inv_freq)[i]
                              : (double)static_cast<const float *>(p.inv_freq)[i];
        f *= 0.15915494309189533577;
        f -= floor(f);  // positions are whole numbers: whole turns per position drop out
        turn[i] = (unsigned long long)(f * 18446744073709551616.0);
    }
    if (tid < TB) {
        const long long tok = (long long)blockIdx.x * TB + tid;
        int b = -1, i = 0, Lq = 0, kstart = 0, Lk = 0, pos = 0;
        long long ko = -1, vo = -1;
        if (tok < p.T && locate_token(p.cu_q, p.B, p.Sq, (int)tok, &b, &i, &Lq)) {
            if (p.kv_mode == 0) {
                Lk = p.Sk;
            } else {
                kstart = p.cu_k[b];
                Lk = p.cu_k[b + 1] - kstart;
            }
            const int j = Lk - Lq + i;  // key index of this token
            bool ok = j >= 0;
            long long outer = 0, row = 0;
            if (ok) {
                if (p.kv_mode == 2) {
                    const int pi = j / p.tab.page_size;
                    int page = -1;
                    if (pi < p.tab.max_pages) page = p.tab.bt[(long long)b * p.tab.bt_stride + pi];
                    ok = page >= 0 && page < p.num_pages;
                    outer = page;
                    row = j - pi * p.tab.page_size;
                } else if (p.kv_mode == 1) {
                    row = (long long)kstart + j;
                    ok = kstart >= 0 && row < p.total_k;
                } else {
                    outer = b;
                    row = j;
                }
            }
            if (ok) {
                ko = outer * p.ko_s[0] + row * p.ko_s[1];
                vo = outer * p.vo_s[0] + row * p.vo_s[1];
            } else {
                atomicOr(p.status, kStatusBounds);
            }
            const long long bb = p.cu_q ? 0 : b, tt = p.cu_q ? tok : i;
            s_q[tid] = bb * p.q_s[0] + tt * p.q_s[1];
            s_k[tid] = bb * p.k_s[0] + tt * p.k_s[1];
            s_v[tid] = bb * p.v_s[0] + tt * p.v_s[1];
            s_qo[tid] = bb * p.qo_s[0] + tt * p.qo_s[1];
            pos = p.pos ? p.pos[bb * p.pos_s[0] + tt * p.pos_s[1]] : j;
        } else {
            b = -1;
        }
        s_ko[tid] = ko;
        s_vo[tid] = vo;
        s_pos[tid] = pos;
        s_b[tid] = b;
    }
    __syncthreads();
    for (int i = tid; i < TB * pairs; i += nthreads) {
        const int t = TB == 1 ? 0 : i / pairs, pr = TB == 1 ? i : i - t * pairs;
        const unsigned long long ph = (unsigned long long)(long long)s_pos[t] * turn[pr];
        float sn, cn;
        sincospif((float)(int)(ph >> 32) * 0x1p-31f, &sn, &cn);
        cs[t][pr] = make_float2(cn * p.rot_scale, sn * p.rot_scale);
    }
    __syncthreads();

    const int x = threadIdx.x;
    // this thread's two groups of 8 dims: both halves of 8 pairs, or 16 dims that pass through
    int da, db, pr = -1;
    const int ritems = p.rot >> 4;
    const int first = p.rot_off >> 3;  // 8-dim groups ahead of the rotated ones
    if (x < ritems) {
        if (INTER) {
            da = p.rot_off + 16 * x;
            db = da + 8;
        } else {
            da = p.rot_off + 8 * x;
            db = da + (p.rot >> 1);
        }
        pr = 8 * x;
    } else {
        const int g = 2 * (x - ritems);
        da = 8 * g + (g < first ? 0 : p.rot);
        db = 8 * (g + 1) + (g + 1 < first ? 0 : p.rot);
    }
    const int heads = p.Hq + 2 * p.Hkv;
    for (int h = blockIdx.y * blockDim.y + threadIdx.y; h < heads; h += gridDim.y * blockDim.y) {
        const int kind = h < p.Hq ? 0 : (h < p.Hq + p.Hkv ? 1 : 2);
        const int hh = kind == 0 ? h : (kind == 1 ? h - p.Hq : h - p.Hq - p.Hkv);
        if (kind == 2 && 16 * x >= p.DV) continue;
        const int a0 = kind == 2 ? 16 * x : da, b0 = kind == 2 ? a0 + 8 : db;
        const T *src = static_cast<const T *>(kind == 0 ? p.q : (kind == 1 ? p.k : p.v)) +
                       hh * (kind == 0 ? p.q_s[2] : (kind == 1 ? p.k_s[2] : p.v_s[2]));
        uint8_t *dst = kind == 0 ? p.qo + hh * p.qo_s[2] : (kind == 1 ? p.ko + hh * p.ko_s[2] : p.vo + hh * p.vo_s[2]);
        const float *ds = kind == 0 ? p.dq : (kind == 1 ? p.dk : p.dv);
        const long long *ds_s = kind == 0 ? p.dq_s : (kind == 1 ? p.dk_s : p.dv_s);
        const int g = kind == 0 ? hh / p.G : hh;
        const long long *from = kind == 0 ? s_q : (kind == 1 ? s_k : s_v);
        const long long *to = kind == 0 ? s_qo : (kind == 1 ? s_ko : s_vo);
        uint4 ra[TB], rb[TB];
        float inv[TB];
#pragma unroll
        for (int t = 0; t < TB; ++t) {
            const int b = s_b[t];
            if (b < 0) continue;
            ra[t] = __ldg(reinterpret_cast<const uint4 *>(src + from[t] + a0));
            rb[t] = __ldg(reinterpret_cast<const uint4 *>(src + from[t] + b0));
            inv[t] = ds ? 1.f / ds[b * ds_s[0] + g * ds_s[1]] : 1.f;
        }
#pragma unroll
        for (int t = 0; t < TB; ++t) {
            if (s_b[t] < 0 || to[t] < 0) continue;
            const uint32_t wa[4] = {ra[t].x, ra[t].y, ra[t].z, ra[t].w};
            const uint32_t wb[4] = {rb[t].x, rb[t].y, rb[t].z, rb[t].w};
            float a[8], b[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 u = unpack2(wa[e], T()), w = unpack2(wb[e], T());
                a[2 * e] = u.x;
                a[2 * e + 1] = u.y;
                b[2 * e] = w.x;
                b[2 * e + 1] = w.y;
            }
            if (kind != 2 && pr >= 0) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float2 c = cs[t][pr + e];
                    float &x0 = INTER ? (e < 4 ? a[2 * e] : b[2 * e - 8]) : a[e];
                    float &x1 = INTER ? (e < 4 ? a[2 * e + 1] : b[2 * e - 7]) : b[e];
                    const float y0 = x0 * c.x - x1 * c.y, y1 = x0 * c.y + x1 * c.x;
                    x0 = y0;
                    x1 = y1;
                }
            }
            uint32_t oa[2], ob[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                oa[e] = ptx::prmt_lo16(ptx::cvt_e4m3x2(a[4 * e + 1] * inv[t], a[4 * e] * inv[t]),
                                       ptx::cvt_e4m3x2(a[4 * e + 3] * inv[t], a[4 * e + 2] * inv[t]));
                ob[e] = ptx::prmt_lo16(ptx::cvt_e4m3x2(b[4 * e + 1] * inv[t], b[4 * e] * inv[t]),
                                       ptx::cvt_e4m3x2(b[4 * e + 3] * inv[t], b[4 * e + 2] * inv[t]));
            }
            *reinterpret_cast<uint2 *>(dst + to[t] + a0) = make_uint2(oa[0], oa[1]);
            *reinterpret_cast<uint2 *>(dst + to[t] + b0) = make_uint2(ob[0], ob[1]);
        }
    }
}

template <typename T, bool INTER>
cudaError_t launch_rope(const RopeParams &p, int sm_count, cudaStream_t s) {
    const int ipt = p.D / 16;
    const dim3 block(ipt, kRopeThreads / ipt);
    const int heads = p.Hq + 2 * p.Hkv;
    // Few tokens: one per CTA and the heads split over CTAs, so that a decode step's loads are all
    // in flight at once.  Many: four per CTA share the fixed-point frequencies.
    if (p.T <= 4 * sm_count) {
        const dim3 grid(p.T, (heads + block.y - 1) / block.y);
        rope_append_kernel<T, INTER, 1><<<grid, block, 0, s>>>(p);
    } else {
        rope_append_kernel<T, INTER, 4><<<dim3((p.T + 3) / 4, 1), block, 0, s>>>(p);
    }
    return cudaGetLastError();
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
