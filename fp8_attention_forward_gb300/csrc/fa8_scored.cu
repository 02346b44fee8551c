// fa8_scored.cu -- host side of fa8_fwd_scored and fa8_fwd_tree: argument checks, the choice of the kernel
// and of its launch (from shapes and the SM count only), the workspace of split launches.
#include <cuda.h>
#include <cuda_runtime.h>
#include <string.h>

#include <algorithm>
#include <cmath>
#include <numeric>

#include "fa8.h"
#include "fa8_host.h"
#include "fa8_scored.cuh"

using namespace fa8::host;

namespace {

constexpr long long kMax32 = 0x7fffffffLL;
constexpr long long kFewSplitKeys = 8192, kFewPartKeys = 2048;
constexpr int kTile = 64;  // keys of a tile of the kernel for many rows

// What the launch of a call looks like; strides and pointers go into `p`.
struct Launch {
    fa8::ScoredParams p;
    Queries qs;
    int DV = 0;
    bool few = false;     // at most 16 rows per kv-head
    int grid = 0;         // CTAs of the kernel for many rows
    long long max_keys = 0;
    size_t bytes = 0;     // of the workspace
    fa8_tensor k4, v4;    // K and V as 4-D tensors (varlen: one page)
};

fa8_status check_shapes(const fa8_tensor *q, const fa8_tensor *k, const fa8_tensor *v, const fa8_tensor *cu_q, const fa8_tensor *cu_k,
                        const fa8_tensor *bt, int page_size, Launch *L) {
    if (!q || !k || !v) return fail(FA8_ERR_INVALID_ARG, "q, k and v are required");
    for (const fa8_tensor *t : {q, k, v})
        if (t->dtype != FA8_DTYPE_E4M3) return fail(FA8_ERR_UNSUPPORTED, "q/k/v must be E4M3");
    fa8_status st;
    if ((st = check_payload(q, "q")) || (st = check_payload(k, "k")) || (st = check_payload(v, "v"))) return st;
    Queries &qs = L->qs;
    if ((st = check_queries(q, cu_q, &qs))) return st;
    fa8::ScoredParams &p = L->p;
    if (k->ndim != v->ndim) return fail(FA8_ERR_INVALID_ARG, "k and v must have the same rank");
    const int nd = k->ndim;
    for (int i = 0; i < nd - 1; ++i)
        if (k->shape[i] != v->shape[i]) return fail(FA8_ERR_INVALID_ARG, "k and v leading shapes differ at dim %d", i);
    if (k->shape[nd - 1] != qs.D) return fail(FA8_ERR_INVALID_ARG, "k head dim %lld != q head dim %d", (long long)k->shape[nd - 1], qs.D);
    if (v->shape[nd - 1] > 1024 || !supported_dims(qs.D, (int)v->shape[nd - 1]))
        return fail(FA8_ERR_UNSUPPORTED, "(d, dv) = (%d, %lld) is not supported", qs.D, (long long)v->shape[nd - 1]);
    L->DV = (int)v->shape[nd - 1];
    if ((st = check_groups(qs.Hq, k->shape[nd - 2], &p.G))) return st;
    p.Hkv = (int)k->shape[nd - 2];
    if (k->shape[0] > kMax32 || (nd == 4 && k->shape[1] > kMax32)) return fail(FA8_ERR_UNSUPPORTED, "too many keys");
    if (bt) {
        Table tab;
        if (nd != 4) return fail(FA8_ERR_INVALID_ARG, "paged k must be (num_pages, page_size, Hkv, d)");
        if ((st = check_table(cu_k, bt, page_size, qs.B, &tab))) return st;
        if (page_size != k->shape[1]) return fail(FA8_ERR_INVALID_ARG, "page_size (%d) != k.shape[1] (%lld)", page_size, (long long)k->shape[1]);
        p.kv_mode = 2;
        p.cu_k = tab.cu_k;
        p.bt = tab.bt;
        p.bt_stride = tab.bt_stride;
        p.max_pages = tab.max_pages;
        p.page_size = page_size;
        p.num_pages = (int)k->shape[0];
        L->max_keys = (long long)tab.max_pages * page_size;
    } else if (nd == 4) {
        if (cu_k) return fail(FA8_ERR_INVALID_ARG, "cu_seqlens_k is only valid with varlen (3-D) or paged k");
        if (k->shape[0] != qs.B) return fail(FA8_ERR_INVALID_ARG, "k batch (%lld) != q batch (%d)", (long long)k->shape[0], qs.B);
        p.kv_mode = 0;
        p.Sk = (int)k->shape[1];
        L->max_keys = p.Sk;
    } else {
        if (!cu_k) return fail(FA8_ERR_INVALID_ARG, "a 3-D (varlen) k needs cu_seqlens_k");
        if ((st = check_int_vec(cu_k, "cu_seqlens_k", (long long)qs.B + 1))) return st;
        p.kv_mode = 1;
        p.cu_k = static_cast<const int *>(cu_k->data);
        p.total_k = (int)k->shape[0];
        L->max_keys = p.total_k;
    }
    L->k4 = *k;
    L->v4 = *v;
    for (fa8_tensor *t : {&L->k4, &L->v4}) {
        if (nd == 4) continue;
        for (int i = 3; i > 0; --i) {
            t->shape[i] = t->shape[i - 1];
            t->stride[i] = t->stride[i - 1];
        }
        t->ndim = 4;
        t->stride[0] = t->stride[1] * std::max<int64_t>(1, t->shape[1]);
        t->shape[0] = 1;
    }
    p.has_kv = k->shape[0] > 0 && (nd == 3 || k->shape[1] > 0);
    p.B = qs.B;
    p.Hq = qs.Hq;
    p.Sq = qs.Sq;
    p.total_q = qs.T;
    p.cu_q = qs.cu_q;
    return FA8_SUCCESS;
}

// The launch on `sms` SMs.  ranges: what the tokens see is not known from the lengths.
fa8_status plan(Launch *L, bool ranges, int sms) {
    fa8::ScoredParams &p = L->p;
    const Queries &qs = L->qs;
    L->bytes = 0;
    // At most 16 rows per kv-head go to the kernel whose warps work alone, but with more than 8 of them and long keys its
    // MMAs of 8 rows take more than the memory (64 requests of 1024 .. 16384 keys, 16 rows, d = 128: 281 us, in units of 128
    // rows 247; 512 keys each: 20 and 30; d = 64, 4096 keys each: 49 and 70; 1 of 32768 keys and 4 kv-heads, in clusters of
    // 16: 23 and 27).
    const long long rows = (long long)qs.Sq * p.G;
    const bool units = rows > 8 && qs.D + L->DV >= 256 && L->max_keys >= 4096 && (long long)qs.B * p.Hkv * 32 > sms;
    if (!qs.cu_q && rows <= 16 && !units) {
        L->few = true;
        p.split = 0;
        // Long keys and few heads: several clusters of eight share a request's keys, as many as run at once (seven eighths of
        // the places: clusters do not fill all of them) while each keeps 2048 keys; a second kernel joins them.  (One request
        // of 131072 keys, d = 256, one kv-head: one cluster of 16 90 us, 32 of 8 25; d = 128, 8 kv-heads: 85 and 52; two of
        // 8192 keys: 18 and 14, of 4096: 13 either way.)
        const long long tiles = (long long)qs.B * p.Hkv, room = (rows > 8 && qs.D + L->DV > 256 ? 2 : 4) * 7LL * sms / 8;
        p.parts = L->max_keys < kFewSplitKeys ? 1 : (int)std::max(1LL, std::min(room / (8 * std::max(1LL, tiles)), L->max_keys / kFewPartKeys));
        if (p.parts > 1) L->bytes = (size_t)(tiles * p.parts * rows * (L->DV + 2)) * sizeof(float);
        if ((long long)qs.B * p.Hkv * 8 > kMax32) return fail(FA8_ERR_UNSUPPORTED, "problem too large for the grid");
        return FA8_SUCCESS;
    }
    p.P = 128 / p.G;
    long long slots;
    if (qs.cu_q) {
        slots = ((long long)qs.T + p.P - 1) / p.P + qs.B;
    } else {
        p.blocks = (qs.Sq + p.P - 1) / p.P;
        slots = (long long)qs.B * p.blocks;
    }
    const long long total = slots * p.Hkv;
    if (total > kMax32) return fail(FA8_ERR_UNSUPPORTED, "problem too large for the unit list");
    // Few units, or ragged ones: all their tiles in even shares over the CTAs, units that a cut goes through joined by a
    // second kernel, which takes about 3 us: so a share has at least eight tiles, about as long, or a whole unit where that
    // is less (14 trees of 31 of 36 keys, d = 256, 56 units in shares of eight: 45 us), and past six units an SM whole ones
    // even out by themselves.  Ranges may leave units little of their keys, which the shares do not know of: then only
    // with less than a unit an SM (two requests of 2011 tokens in documents, 252 units: 54 us in shares, 40 whole; two of 446
    // and 8438 keys, 5 tokens, 4 units: 25 and 116).
    const long long tiles = ((L->max_keys + kTile - 1) / kTile + 8) * total;
    p.min_tiles = 8;
    p.split = !qs.cu_q && p.has_kv && total < (ranges ? 1LL : 6LL) * sms && tiles < kMax32 / 2;
    if (p.split) {
        L->grid = (int)std::max(1LL, std::min<long long>(sms, std::max(total, (tiles + p.min_tiles - 1) / p.min_tiles)));
        if (L->grid == 1) p.split = 0;
    }
    // Whole units: with at least four an SM the CTAs take them as they come (two prompts of 4096, 2048 units, heads of unequal
    // cost: 376 us in fixed turns, 335), with fewer the last ones that a CTA has asked for ahead would wait (four chunks of
    // 1021, 256 units: 150 and 194).
    p.units = (int)total;
    p.steal = total >= 4LL * sms;
    if (!p.split) L->grid = (int)(p.steal ? total : std::min<long long>(sms, total));
    if (p.split) L->bytes = (size_t)L->grid * (2 * 128 * (L->DV + 2) + 4) * sizeof(float);
    return FA8_SUCCESS;
}

fa8_status check_outputs(const fa8_tensor *q, fa8_tensor *out, fa8_tensor *lse, Launch *L) {
    const int nd = q->ndim;
    const Queries &qs = L->qs;
    fa8::ScoredParams &p = L->p;
    fa8_status st;
    if (!out) return fail(FA8_ERR_INVALID_ARG, "out is required");
    if (out->dtype != FA8_DTYPE_BF16 && out->dtype != FA8_DTYPE_F16) return fail(FA8_ERR_INVALID_ARG, "out must be bf16 or fp16");
    if (out->ndim != nd) return fail(FA8_ERR_INVALID_ARG, "out must have q's rank");
    for (int i = 0; i < nd - 1; ++i) {
        if (out->shape[i] != q->shape[i]) return fail(FA8_ERR_INVALID_ARG, "out shape differs from q at dim %d", i);
        if (out->stride[i] % 8 != 0) return fail(FA8_ERR_INVALID_ARG, "out strides must be multiples of 8 elements");
    }
    if (out->shape[nd - 1] != L->DV) return fail(FA8_ERR_INVALID_ARG, "out last dim must be dv=%d", L->DV);
    if (out->stride[nd - 1] != 1) return fail(FA8_ERR_INVALID_ARG, "out: last dim must be contiguous");
    if (!aligned16(out->data)) return fail(FA8_ERR_INVALID_ARG, "out must be 16-byte aligned");
    if ((st = check_written(out, "out"))) return st;
    for (int i = 0; i < 3; ++i) p.o_s[i] = nd == 4 ? out->stride[i] : (i ? out->stride[i - 1] : 0);
    p.o = out->data;
    p.out_fp16 = out->dtype == FA8_DTYPE_F16;
    if (!lse) return FA8_SUCCESS;
    if (lse->dtype != FA8_DTYPE_F32) return fail(FA8_ERR_INVALID_ARG, "lse must be fp32");
    if (qs.cu_q) {
        if (lse->ndim != 2 || lse->shape[0] != qs.Hq || lse->shape[1] != qs.T) return fail(FA8_ERR_INVALID_ARG, "varlen lse must be (Hq, total_q)");
        p.lse_s[1] = lse->stride[1];
        p.lse_s[2] = lse->stride[0];
    } else {
        if (lse->ndim != 3 || lse->shape[0] != qs.B || lse->shape[1] != qs.Hq || lse->shape[2] != qs.Sq)
            return fail(FA8_ERR_INVALID_ARG, "lse must be (B, Hq, Sq)");
        p.lse_s[0] = lse->stride[0];
        p.lse_s[1] = lse->stride[2];
        p.lse_s[2] = lse->stride[1];
    }
    p.lse = static_cast<float *>(lse->data);
    return check_written(lse, "lse");
}

// (q's tokens, n) int32, last dim contiguous; strides {request, token}.
fa8_status check_per_token(const fa8_tensor *t, const char *name, const Queries &qs, long long n, long long stride[2]) {
    if (t->dtype != FA8_DTYPE_I32) return fail(FA8_ERR_INVALID_ARG, "%s must be int32", name);
    const int nd = qs.cu_q ? 2 : 3;
    const bool same = t->ndim == nd && (qs.cu_q ? t->shape[0] == qs.T : (t->shape[0] == qs.B && t->shape[1] == qs.Sq));
    if (!same || (n >= 0 && t->shape[nd - 1] != n)) return fail(FA8_ERR_INVALID_ARG, "%s must be (q's tokens, %s)", name, n == 2 ? "2" : "words");
    if (t->shape[nd - 1] > 1 && t->stride[nd - 1] != 1) return fail(FA8_ERR_INVALID_ARG, "%s: last dim must be contiguous", name);
    stride[0] = qs.cu_q ? 0 : t->stride[0];
    stride[1] = t->stride[nd - 2];
    return FA8_SUCCESS;
}

// All that the two entry points have in common, after their own arguments are in L->p.
fa8_status forward(Launch *L, const fa8_tensor *q, const fa8_tensor *k, const fa8_tensor *v, const fa8_tensor *descale_q,
                   const fa8_tensor *descale_k, const fa8_tensor *descale_v, fa8_tensor *out, fa8_tensor *lse, const fa8_tensor *sink,
                   float softcap, float softmax_scale, void *workspace, size_t workspace_bytes, void *stream) {
    fa8::ScoredParams &p = L->p;
    const Queries &qs = L->qs;
    fa8_status st;
    if ((st = check_outputs(q, out, lse, L))) return st;
    if ((st = check_descale(descale_q, "descale_q", qs.B, p.Hkv, &p.dq, &p.dq_s[0], &p.dq_s[1])) ||
        (st = check_descale(descale_k, "descale_k", qs.B, p.Hkv, &p.dk, &p.dk_s[0], &p.dk_s[1])) ||
        (st = check_descale(descale_v, "descale_v", qs.B, p.Hkv, &p.dv, &p.dv_s[0], &p.dv_s[1])))
        return st;
    if (sink) {
        if (sink->dtype != FA8_DTYPE_F32 || sink->ndim != 1 || sink->shape[0] != qs.Hq || (qs.Hq > 1 && sink->stride[0] != 1) || !sink->data)
            return fail(FA8_ERR_INVALID_ARG, "sink must be a contiguous fp32 (Hq,) tensor");
        p.sink = static_cast<const float *>(sink->data);
    }
    if (!std::isfinite(softcap) || softcap < 0.f) return fail(FA8_ERR_INVALID_ARG, "softcap must be finite and not negative");
    if (!std::isfinite(softmax_scale)) return fail(FA8_ERR_INVALID_ARG, "softmax_scale must be finite");
    if (softmax_scale <= 0.f) softmax_scale = 1.0f / std::sqrt((float)qs.D);
    p.scale_log2 = softmax_scale * 1.4426950408889634f;
    p.cap_log2 = softcap * 1.4426950408889634f;
    if (softcap > 0.f && p.cap_log2 < 0x1p-100f) return fail(FA8_ERR_UNSUPPORTED, "softcap is out of range");
    if ((st = plan(L, p.ranges != nullptr, 1))) return st;  // refuses what no device takes
    if (qs.T == 0) return FA8_SUCCESS;
    if (!q->data || !out->data || (lse && !lse->data) || (p.has_kv && (!k->data || !v->data)))
        return fail(FA8_ERR_INVALID_ARG, "q, k, v, out and lse need data");
    DeviceState *ds = nullptr;
    if ((st = device_state(&ds))) return st;
    if ((st = plan(L, p.ranges != nullptr, ds->sm_count))) return st;
    if (L->bytes) {
        if (!workspace || workspace_bytes < L->bytes)
            return fail(FA8_ERR_WORKSPACE, "this call needs %zu bytes of workspace, got %zu", L->bytes, workspace ? workspace_bytes : (size_t)0);
        if (!aligned16(workspace)) return fail(FA8_ERR_WORKSPACE, "workspace must be 16-byte aligned");
        p.part = static_cast<float *>(workspace);
    }
    p.q = static_cast<const uint8_t *>(q->data);
    p.v = static_cast<const uint8_t *>(v->data);
    for (int i = 0; i < 3; ++i) {
        p.q_s[i] = qs.stride[i];
        p.v_s[i] = L->v4.stride[i];
    }
    p.status = ds->status;
    p.timeout_ns = wait_timeout_ns();
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int dims = qs.D * 1000 + L->DV;
#define FA8_EACH(X) X(64, 64) X(96, 96) X(128, 128) X(192, 128) X(192, 192) X(256, 256)
    if (L->few) {
#define FA8_FEW(D_, DV_) \
    if (dims == D_ * 1000 + DV_) return fa8::launch_scored_few<D_, DV_>(p, &L->k4, &L->v4, qs.B * p.Hkv, L->max_keys, ds->sm_count, ds->ordinal, s);
        FA8_EACH(FA8_FEW)
    } else {
        const int cw = qs.D % 128 == 0 ? 128 : (qs.D % 64 == 0 ? 64 : 32);
        CUtensorMap tq, tk, tv;
        memset(&tk, 0, sizeof(tk));
        memset(&tv, 0, sizeof(tv));
        if ((st = encode_q(&tq, q, cw, p.G, p.P))) return st;
        // K comes two tiles at a time, V too where dv <= 128; boxes do not cross a page, and a unit may start with any tile
        const int step = 2 * kTile;
        p.box_n = p.kv_mode == 2 ? std::gcd(p.page_size, kTile) : step;
        p.boxes = step / p.box_n;
        p.box_v = L->DV <= 128 ? p.box_n : std::min(p.box_n, kTile);
        if (p.kv_mode == 2) {
            p.step_e = step / p.page_size;
            p.step_r = step % p.page_size;
        }
        if (p.has_kv) {
            if ((st = encode_kv(&tk, &L->k4, cw, p.box_n)) || (st = encode_kv(&tv, &L->v4, L->DV, p.box_v, false))) return st;
        }
#define FA8_MANY(D_, DV_) \
    if (dims == D_ * 1000 + DV_) return fa8::launch_scored_many<D_, DV_>(p, tq, tk, tv, L->grid, ds->ordinal, s);
        FA8_EACH(FA8_MANY)
    }
    return fail(FA8_ERR_UNSUPPORTED, "no kernel for (%d, %d)", qs.D, L->DV);
}

}  // namespace

extern "C" fa8_status fa8_fwd_scored_workspace_size(const fa8_tensor *q, const fa8_tensor *k, const fa8_tensor *v, const fa8_tensor *cu_seqlens_q,
                                                    const fa8_tensor *cu_seqlens_k, const fa8_tensor *block_table, int page_size,
                                                    const fa8_tensor *ranges, size_t *bytes_out) {
    clear_error();
    Launch L;
    memset(&L.p, 0, sizeof(L.p));
    fa8_status st;
    if ((st = check_shapes(q, k, v, cu_seqlens_q, cu_seqlens_k, block_table, page_size, &L))) return st;
    if ((st = plan(&L, ranges != nullptr, 1))) return st;
    size_t bytes = 0;
    if (L.qs.T > 0) {
        DeviceState *ds = nullptr;
        if ((st = device_state(&ds))) return st;
        if ((st = plan(&L, ranges != nullptr, ds->sm_count))) return st;
        bytes = L.bytes;
    }
    if (bytes_out) *bytes_out = bytes;
    return FA8_SUCCESS;
}

extern "C" fa8_status fa8_fwd_scored(const fa8_tensor *q, const fa8_tensor *k, const fa8_tensor *v, const fa8_tensor *descale_q,
                                     const fa8_tensor *descale_k, const fa8_tensor *descale_v, fa8_tensor *out, fa8_tensor *lse,
                                     const fa8_tensor *cu_seqlens_q, const fa8_tensor *cu_seqlens_k, const fa8_tensor *block_table,
                                     int page_size, int causal, int window_left, const fa8_tensor *ranges, const fa8_tensor *slopes,
                                     float softcap, const fa8_tensor *sink, float softmax_scale, void *workspace, size_t workspace_bytes,
                                     void *stream) {
    clear_error();
    Launch L;
    memset(&L.p, 0, sizeof(L.p));
    fa8_status st;
    if ((st = check_shapes(q, k, v, cu_seqlens_q, cu_seqlens_k, block_table, page_size, &L))) return st;
    if (causal != 0 && causal != 1) return fail(FA8_ERR_INVALID_ARG, "causal must be 0 or 1");
    if (window_left < -1) return fail(FA8_ERR_INVALID_ARG, "window_left must be -1 or >= 0");
    L.p.causal = causal;
    L.p.window_left = window_of(window_left, L.max_keys, L.qs.cu_q ? L.qs.T : L.qs.Sq);
    if (ranges) {
        if ((st = check_per_token(ranges, "ranges", L.qs, 2, L.p.r_s))) return st;
        if (!ranges->data && L.qs.T > 0) return fail(FA8_ERR_INVALID_ARG, "ranges needs data");
        L.p.ranges = static_cast<const int *>(ranges->data);
    }
    if (slopes) {
        if (slopes->dtype != FA8_DTYPE_F32 || slopes->ndim != 1 || slopes->shape[0] != L.qs.Hq || (L.qs.Hq > 1 && slopes->stride[0] != 1) ||
            !slopes->data)
            return fail(FA8_ERR_INVALID_ARG, "slopes must be a contiguous fp32 (Hq,) tensor");
        L.p.slopes = static_cast<const float *>(slopes->data);
    }
    return forward(&L, q, k, v, descale_q, descale_k, descale_v, out, lse, sink, softcap, softmax_scale, workspace, workspace_bytes, stream);
}

extern "C" fa8_status fa8_fwd_tree(const fa8_tensor *q, const fa8_tensor *k, const fa8_tensor *v, const fa8_tensor *masks,
                                   const fa8_tensor *descale_q, const fa8_tensor *descale_k, const fa8_tensor *descale_v, fa8_tensor *out,
                                   fa8_tensor *lse, const fa8_tensor *cu_seqlens_q, const fa8_tensor *cu_seqlens_k,
                                   const fa8_tensor *block_table, int page_size, float softcap, const fa8_tensor *sink, float softmax_scale,
                                   void *workspace, size_t workspace_bytes, void *stream) {
    clear_error();
    Launch L;
    memset(&L.p, 0, sizeof(L.p));
    fa8_status st;
    if ((st = check_shapes(q, k, v, cu_seqlens_q, cu_seqlens_k, block_table, page_size, &L))) return st;
    if (!masks) return fail(FA8_ERR_INVALID_ARG, "masks is required");
    if ((st = check_per_token(masks, "masks", L.qs, -1, L.p.m_s))) return st;
    const long long words = masks->shape[masks->ndim - 1];
    if (words > 4096) return fail(FA8_ERR_UNSUPPORTED, "%lld words per mask, at most 4096 are supported", words);
    if (!L.qs.cu_q && words * 32 < L.qs.Sq) return fail(FA8_ERR_INVALID_ARG, "masks of %lld words do not hold %d tokens", words, L.qs.Sq);
    if (!masks->data && L.qs.T > 0) return fail(FA8_ERR_INVALID_ARG, "masks needs data");
    L.p.words = (int)words;
    L.p.masks = static_cast<const int *>(masks->data);
    L.p.window_left = -1;
    return forward(&L, q, k, v, descale_q, descale_k, descale_v, out, lse, sink, softcap, softmax_scale, workspace, workspace_bytes, stream);
}
