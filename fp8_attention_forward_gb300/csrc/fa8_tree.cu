// fa8_tree.cu -- what a tree of drafted tokens needs beside its attention: the tokens' masks and positions
// from their parents (fa8_tree_masks), and the accepted tokens' keys and values moved to the front of the
// drafted ones in the cache (fa8_keep_tokens).
//
//   mask(i) = {i} + mask(parent(i)),   position(i) = Lk - Lq + |mask(i)| - 1
//   K, V of slot s  <-  those of drafted token kept(s), as if all were read before any is written
//
// Both move a few hundred bytes to a few MB: their time is a launch and a chain of dependent loads.
#include <cuda_runtime.h>
#include <string.h>

#include <algorithm>

#include "fa8.h"
#include "fa8_host.h"
#include "fa8_kernel.cuh"
#include "fa8_pages.cuh"

namespace fa8 {

constexpr int kMaxTreeWords = 128;
constexpr int kTreeThreads = 256;

struct TreeParams {
    const int *parents;
    long long p_s[2];  // request, token
    int *masks;
    long long m_s[2];
    int words;
    int *pos;          // may be null
    long long o_s[2];
    const int *cu_q, *cu_k;  // null: batched; positions from 0
    int Sq, total_q;
    unsigned int *status;
};

// A thread takes one word of one token's mask: it walks up from the token and notes the ancestors of its
// word; parents come before their children, so it is done below the word.  Word 0 sees all ancestors and
// counts them.  (A doubling of the links would take log2(depth) barriers; the walk is depth loads of
// shared memory.)
__global__ void __launch_bounds__(kTreeThreads) tree_masks_kernel(const __grid_constant__ TreeParams p) {
    __shared__ int up[32 * kMaxTreeWords];
    const int b = blockIdx.x, tid = threadIdx.x;
    const int q0 = p.cu_q ? p.cu_q[b] : 0, Lq = p.cu_q ? p.cu_q[b + 1] - q0 : p.Sq;
    if (p.cu_q && (q0 < 0 || Lq < 0 || (long long)q0 + Lq > p.total_q)) {
        if (tid == 0 && blockIdx.y == 0) atomicOr(p.status, kStatusBounds);
        return;
    }
    const long long bb = p.cu_q ? 0 : b;
    const int held = min(Lq, 32 * p.words);
    if (tid == 0 && blockIdx.y == 0 && held < Lq) atomicOr(p.status, kStatusBounds);
    const int first = p.cu_k ? p.cu_k[b + 1] - p.cu_k[b] - Lq : 0;
    const long long items = (long long)Lq * p.words;
    if ((long long)blockIdx.y * kTreeThreads >= items) return;
    for (int i = tid; i < held; i += kTreeThreads) {
        int x = p.parents[bb * p.p_s[0] + ((long long)q0 + i) * p.p_s[1]];
        if (x >= i) {
            atomicOr(p.status, kStatusBounds);
            x = -1;
        }
        up[i] = x;
    }
    __syncthreads();
    for (long long it = (long long)blockIdx.y * kTreeThreads + tid; it < items; it += (long long)gridDim.y * kTreeThreads) {
        const int i = (int)(it / p.words), w = (int)(it - (long long)i * p.words);
        uint32_t m = 0;
        int depth = -1;
        if (i < held) {
            for (int x = i; x >= 32 * w && x >= 0; x = up[x]) {
                if (x < 32 * w + 32) m |= 1u << (x & 31);
                ++depth;
            }
        }
        p.masks[bb * p.m_s[0] + ((long long)q0 + i) * p.m_s[1] + w] = (int)m;
        if (w == 0 && p.pos) p.pos[bb * p.o_s[0] + ((long long)q0 + i) * p.o_s[1]] = max(0, first + max(depth, 0));
    }
}

constexpr int kMaxKept = 1024;
constexpr int kKeepThreads = 256;

struct KeepParams {
    uint8_t *k, *v;
    long long k_s[3], v_s[3];  // request or page, row, head
    int kp, vp;                // 16-byte pieces of a head's row
    int Hkv, kv_mode, Sk, total_k;
    const int *kept;
    long long t_s;             // request
    int N, new_tokens;
    const int *cu_q, *cu_k, *bt;
    long long bt_stride;
    int max_pages, page_size, num_pages;
    unsigned int *status;
};

// A CTA takes CB 16-byte columns of a request's rows: reads them of every kept token into shared memory, then
// writes them to the slots.
template <int CB>
__global__ void __launch_bounds__(kKeepThreads) keep_tokens_kernel(const __grid_constant__ KeepParams p) {
    extern __shared__ __align__(16) uint4 s_rows[];  // [slot][column]
    const int b = blockIdx.x, tid = threadIdx.x;
    const int Lq = p.cu_q ? p.cu_q[b + 1] - p.cu_q[b] : p.new_tokens;
    int Lk = p.Sk, k0 = 0;
    if (p.kv_mode != 0) {
        const int a = p.cu_k[b];
        Lk = p.cu_k[b + 1] - a;
        if (p.kv_mode == 1) k0 = a;
    }
    const bool bad = Lq < 0 || Lk < 0 || (p.kv_mode == 1 && (k0 < 0 || (long long)k0 + Lk > p.total_k)) ||
                     (p.kv_mode == 2 && Lk > (long long)p.max_pages * p.page_size);
    const bool tell = tid == 0 && blockIdx.y == 0;
    if (bad) {
        if (tell) atomicOr(p.status, kStatusBounds);
        return;
    }
    const int first = Lk - Lq;
    const int col = blockIdx.y * CB + tid % CB, heads_k = p.Hkv * p.kp;
    const bool in = col < heads_k + p.Hkv * p.vp, of_v = col >= heads_k;
    const int pieces = of_v ? p.vp : p.kp, rel = of_v ? col - heads_k : col;
    uint8_t *base = of_v ? p.v : p.k;
    const long long sp = of_v ? p.v_s[0] : p.k_s[0], sr = of_v ? p.v_s[1] : p.k_s[1];
    if (in) base += (rel / pieces) * (of_v ? p.v_s[2] : p.k_s[2]) + 16 * (rel % pieces);
    // address of the column in the row of drafted token i; null where it has none
    auto at = [&](int i) -> uint8_t * {
        const int j = first + i;
        if (j < 0) return nullptr;  // a padded slot's token without a key
        if (p.kv_mode != 2) return base + (p.kv_mode == 0 ? b * sp : 0) + ((long long)k0 + j) * sr;
        const int e = p.bt[b * p.bt_stride + j / p.page_size];
        if (e < 0 || e >= p.num_pages) {
            atomicOr(p.status, kStatusBounds);
            return nullptr;
        }
        return base + e * sp + (long long)(j % p.page_size) * sr;
    };
    const int *kept = p.kept + b * p.t_s;
    constexpr int ROWS = kKeepThreads / CB;
    auto taken = [&](int s) -> int {  // the token for slot s, or -1
        const int i = kept[s];
        if (i < 0) return -1;
        if (i >= Lq || s >= Lq) {
            if (tid % CB == 0) atomicOr(p.status, kStatusBounds);
            return -1;
        }
        return i == s ? -1 : i;
    };
    for (int s = tid / CB; s < p.N; s += ROWS) {
        const int i = taken(s);
        if (i < 0 || !in) continue;
        const uint8_t *src = at(i);
        if (src && at(s)) s_rows[s * CB + tid % CB] = *reinterpret_cast<const uint4 *>(src);
    }
    __syncthreads();
    for (int s = tid / CB; s < p.N; s += ROWS) {
        const int i = taken(s);
        if (i < 0 || !in) continue;
        const uint8_t *src = at(i);
        uint8_t *dst = at(s);
        if (src && dst) *reinterpret_cast<uint4 *>(dst) = s_rows[s * CB + tid % CB];
    }
}

}  // namespace fa8

using namespace fa8::host;

namespace {

// int32 (B, Sq, ..) or packed (T, ..) with cu_q; `last`: one more dim, contiguous.
fa8_status check_tokens(const fa8_tensor *t, const char *name, int B, int Sq, int T, const fa8_tensor *cu_q, bool last, long long stride[2]) {
    if (t->dtype != FA8_DTYPE_I32) return fail(FA8_ERR_INVALID_ARG, "%s must be int32", name);
    const int nd = (cu_q ? 1 : 2) + (last ? 1 : 0);
    const bool same = t->ndim == nd && (cu_q ? t->shape[0] == T : (t->shape[0] == B && t->shape[1] == Sq));
    if (!same) return fail(FA8_ERR_INVALID_ARG, "%s must have the parents' shape%s", name, last ? " and words" : "");
    if (last && t->shape[nd - 1] > 1 && t->stride[nd - 1] != 1) return fail(FA8_ERR_INVALID_ARG, "%s: last dim must be contiguous", name);
    stride[0] = cu_q ? 0 : t->stride[0];
    stride[1] = t->stride[cu_q ? 0 : 1];
    return FA8_SUCCESS;
}

}  // namespace

extern "C" fa8_status fa8_tree_masks(const fa8_tensor *parents, fa8_tensor *masks, fa8_tensor *positions, const fa8_tensor *cu_seqlens_q,
                                     const fa8_tensor *cu_seqlens_k, void *stream) {
    clear_error();
    if (!parents || !masks) return fail(FA8_ERR_INVALID_ARG, "parents and masks are required");
    fa8_status st;
    if (parents->ndim != (cu_seqlens_q ? 1 : 2)) return fail(FA8_ERR_INVALID_ARG, "parents must be (B, Sq), or (total_q) with cu_seqlens_q");
    for (int i = 0; i < parents->ndim; ++i)
        if (parents->shape[i] < 0 || parents->shape[i] > 0x7fffffffLL) return fail(FA8_ERR_UNSUPPORTED, "too many tokens");
    fa8::TreeParams p;
    memset(&p, 0, sizeof(p));
    long long B = parents->shape[0], T = parents->shape[0];
    if (cu_seqlens_q) {
        if (cu_seqlens_q->ndim != 1 || cu_seqlens_q->shape[0] < 2 || cu_seqlens_q->shape[0] > 0x7fffffffLL)
            return fail(FA8_ERR_INVALID_ARG, "cu_seqlens_q must have B+1 >= 2 entries");
        B = cu_seqlens_q->shape[0] - 1;
        if ((st = check_int_vec(cu_seqlens_q, "cu_seqlens_q", B + 1))) return st;
        p.cu_q = static_cast<const int *>(cu_seqlens_q->data);
    } else {
        p.Sq = (int)parents->shape[1];
        T = B * p.Sq;
    }
    if (T > 0x7fffffffLL) return fail(FA8_ERR_UNSUPPORTED, "too many tokens");
    p.total_q = (int)T;
    if ((st = check_tokens(parents, "parents", (int)B, p.Sq, (int)T, cu_seqlens_q, false, p.p_s)) ||
        (st = check_tokens(masks, "masks", (int)B, p.Sq, (int)T, cu_seqlens_q, true, p.m_s)) || (st = check_written(masks, "masks")))
        return st;
    const long long words = masks->shape[masks->ndim - 1];
    if (words > fa8::kMaxTreeWords) return fail(FA8_ERR_UNSUPPORTED, "%lld words per mask, at most %d are supported", words, fa8::kMaxTreeWords);
    if ((!cu_seqlens_q && words * 32 < p.Sq) || (words == 0 && T > 0))
        return fail(FA8_ERR_INVALID_ARG, "masks of %lld words do not hold %lld tokens", words, cu_seqlens_q ? T : p.Sq);
    if (positions) {
        if ((st = check_tokens(positions, "positions", (int)B, p.Sq, (int)T, cu_seqlens_q, false, p.o_s)) || (st = check_written(positions, "positions")))
            return st;
        p.pos = static_cast<int *>(positions->data);
    }
    if (cu_seqlens_k) {
        if ((st = check_int_vec(cu_seqlens_k, "cu_seqlens_k", B + 1))) return st;
        p.cu_k = static_cast<const int *>(cu_seqlens_k->data);
    }
    if (T == 0) return FA8_SUCCESS;
    if (!parents->data || !masks->data || (positions && !positions->data)) return fail(FA8_ERR_INVALID_ARG, "parents, masks and positions need data");
    DeviceState *ds = nullptr;
    if ((st = device_state(&ds))) return st;
    p.parents = static_cast<const int *>(parents->data);
    p.masks = static_cast<int *>(masks->data);
    p.words = (int)words;
    p.status = ds->status;
    // blocks of a request: one item a thread where that keeps the grid small
    const long long most = (p.cu_q ? std::min<long long>(T, 32 * words) : p.Sq) * words;
    const unsigned y = (unsigned)std::min<long long>((most + fa8::kTreeThreads - 1) / fa8::kTreeThreads, 64);
    fa8::tree_masks_kernel<<<dim3((unsigned)B, y), fa8::kTreeThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? FA8_SUCCESS : cuda_fail(e, "tree masks kernel launch");
}

extern "C" fa8_status fa8_keep_tokens(fa8_tensor *k, fa8_tensor *v, const fa8_tensor *kept, const fa8_tensor *cu_seqlens_q,
                                      const fa8_tensor *cu_seqlens_k, const fa8_tensor *block_table, int page_size, int new_tokens,
                                      void *stream) {
    static SmemOptIn opt_wide, opt_narrow;
    clear_error();
    if (!k || !v || !kept) return fail(FA8_ERR_INVALID_ARG, "k, v and kept are required");
    fa8_status st;
    for (fa8_tensor *t : {k, v}) {
        const char *name = t == k ? "k" : "v";
        if (t->dtype != FA8_DTYPE_E4M3) return fail(FA8_ERR_UNSUPPORTED, "%s must be E4M3", name);
        if ((st = check_payload(t, name)) || (st = check_written(t, name))) return st;
        const long long d = t->shape[t->ndim - 1];
        if (d <= 0 || d % 16 != 0 || d > 1024) return fail(FA8_ERR_UNSUPPORTED, "%s: head dim %lld is not a multiple of 16 up to 1024", name, d);
    }
    if (k->ndim != v->ndim) return fail(FA8_ERR_INVALID_ARG, "k and v must have the same rank");
    const int nd = k->ndim;
    for (int i = 0; i < nd - 1; ++i)
        if (k->shape[i] != v->shape[i]) return fail(FA8_ERR_INVALID_ARG, "k and v leading shapes differ at dim %d", i);
    if (k->shape[0] > 0x7fffffffLL || (nd == 4 && k->shape[1] > 0x7fffffffLL) || k->shape[nd - 2] > 65536)
        return fail(FA8_ERR_UNSUPPORTED, "k is too large");
    if (kept->dtype != FA8_DTYPE_I32 || kept->ndim != 2 || (kept->shape[1] > 1 && kept->stride[1] != 1))
        return fail(FA8_ERR_INVALID_ARG, "kept must be int32 (B, N) with contiguous rows");
    const long long B = kept->shape[0], N = kept->shape[1];
    if (B < 1 || B > 0x7fffffffLL - 1) return fail(FA8_ERR_INVALID_ARG, "batch must be >= 1");
    if (N < 0) return fail(FA8_ERR_INVALID_ARG, "kept: negative extent");
    if (N > fa8::kMaxKept) return fail(FA8_ERR_UNSUPPORTED, "%lld kept tokens, at most %d are supported", N, fa8::kMaxKept);
    fa8::KeepParams p;
    memset(&p, 0, sizeof(p));
    if (cu_seqlens_q) {
        if ((st = check_int_vec(cu_seqlens_q, "cu_seqlens_q", B + 1))) return st;
        p.cu_q = static_cast<const int *>(cu_seqlens_q->data);
    } else if (new_tokens < 0) {
        return fail(FA8_ERR_INVALID_ARG, "new_tokens must not be negative");
    }
    p.new_tokens = new_tokens;
    if (block_table) {
        Table tab;
        if (nd != 4) return fail(FA8_ERR_INVALID_ARG, "paged k must be (num_pages, page_size, Hkv, d)");
        if ((st = check_table(cu_seqlens_k, block_table, page_size, (int)B, &tab))) return st;
        if (page_size != k->shape[1]) return fail(FA8_ERR_INVALID_ARG, "page_size (%d) != k.shape[1] (%lld)", page_size, (long long)k->shape[1]);
        p.kv_mode = 2;
        p.cu_k = tab.cu_k;
        p.bt = tab.bt;
        p.bt_stride = tab.bt_stride;
        p.max_pages = tab.max_pages;
        p.page_size = page_size;
        p.num_pages = (int)k->shape[0];
    } else if (nd == 4) {
        if (cu_seqlens_k) return fail(FA8_ERR_INVALID_ARG, "cu_seqlens_k is only valid with varlen (3-D) or paged k");
        if (k->shape[0] != B) return fail(FA8_ERR_INVALID_ARG, "k batch (%lld) != kept's (%lld)", (long long)k->shape[0], B);
        p.Sk = (int)k->shape[1];
    } else {
        if (!cu_seqlens_k) return fail(FA8_ERR_INVALID_ARG, "a 3-D (varlen) k needs cu_seqlens_k");
        if ((st = check_int_vec(cu_seqlens_k, "cu_seqlens_k", B + 1))) return st;
        p.kv_mode = 1;
        p.cu_k = static_cast<const int *>(cu_seqlens_k->data);
        p.total_k = (int)k->shape[0];
    }
    p.Hkv = (int)k->shape[nd - 2];
    if (N == 0 || p.Hkv == 0 || k->shape[0] == 0 || (nd == 4 && k->shape[1] == 0)) return FA8_SUCCESS;
    if (!k->data || !v->data || !kept->data) return fail(FA8_ERR_INVALID_ARG, "k, v and kept need data");
    DeviceState *ds = nullptr;
    if ((st = device_state(&ds))) return st;
    p.k = static_cast<uint8_t *>(k->data);
    p.v = static_cast<uint8_t *>(v->data);
    for (int i = 0; i < 3; ++i) {
        p.k_s[i] = nd == 4 ? k->stride[i] : (i ? k->stride[i - 1] : 0);
        p.v_s[i] = nd == 4 ? v->stride[i] : (i ? v->stride[i - 1] : 0);
    }
    p.kp = (int)(k->shape[nd - 1] / 16);
    p.vp = (int)(v->shape[nd - 1] / 16);
    p.kept = static_cast<const int *>(kept->data);
    p.t_s = kept->stride[0];
    p.N = (int)N;
    p.status = ds->status;
    // 512 bytes of a row a CTA while all slots' fit shared memory well, else 128
    const bool wide = N <= 128;
    const int cb = wide ? 32 : 8;
    const int smem = (int)N * cb * 16;
    const long long y = ((long long)p.Hkv * (p.kp + p.vp) + cb - 1) / cb;
    if (y > 65535) return fail(FA8_ERR_UNSUPPORTED, "k and v rows are too long");
    const cudaError_t o = wide ? opt_wide(fa8::keep_tokens_kernel<32>, smem, ds->ordinal) : opt_narrow(fa8::keep_tokens_kernel<8>, smem, ds->ordinal);
    if (o != cudaSuccess) return cuda_fail(o, "keep tokens shared memory");
    const dim3 grid((unsigned)B, (unsigned)y);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (wide) fa8::keep_tokens_kernel<32><<<grid, fa8::kKeepThreads, smem, s>>>(p);
    else fa8::keep_tokens_kernel<8><<<grid, fa8::kKeepThreads, smem, s>>>(p);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? FA8_SUCCESS : cuda_fail(e, "keep tokens kernel launch");
}
