// fa8_host.h -- internal: host-side pieces that every C entry point shares (the error text of
// the calling thread, per-device state, argument checks).  Defined in fa8_api.cu.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>
#include <mutex>

#include "fa8.h"

namespace fa8 {
namespace host {

// Sets the calling thread's fa8_last_error() and returns `s`.
fa8_status fail(fa8_status s, const char *fmt, ...);
fa8_status cuda_fail(cudaError_t e, const char *what);
void clear_error();

struct DeviceState {
    bool ready = false;
    int ordinal = 0;
    int sm_count = 0;
    unsigned int *status = nullptr;
};
// State of the current device, looked up on the first call for it.
fa8_status device_state(DeviceState **out);

// Opts a kernel in to `bytes` of dynamic shared memory on a device, once per size: what each device has
// been given for this kernel so far.  Setting is under a lock: a smaller size must not land after a larger.
struct SmemOptIn {
    std::atomic<int> given[64] = {};
    std::mutex mu;
    template <typename K>
    cudaError_t operator()(K *kernel, int bytes, int ordinal) {
        if (given[ordinal].load(std::memory_order_acquire) >= bytes) return cudaSuccess;
        std::lock_guard<std::mutex> lock(mu);
        if (given[ordinal].load(std::memory_order_relaxed) >= bytes) return cudaSuccess;
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e == cudaSuccess) given[ordinal].store(bytes, std::memory_order_release);
        return e;
    }
};

// Whether a launch in clusters of 16, past the portable 8, fits the device: asked once per kernel, device
// and shared-memory size.
struct Cluster16 {
    std::atomic<int> fits[64] = {}, not_from[64] = {};  // bytes + 1 up to which it fits, from which it does not
    template <typename K>
    bool operator()(K *kernel, const cudaLaunchConfig_t &cfg, int ordinal) {
        const int bytes = (int)cfg.dynamicSmemBytes + 1, no = not_from[ordinal].load(std::memory_order_relaxed);
        if (fits[ordinal].load(std::memory_order_relaxed) >= bytes) return true;
        if (no && bytes >= no) return false;
        int n = 0;
        const bool ok = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess &&
                        cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) == cudaSuccess && n > 0;
        if (!ok) cudaGetLastError();  // a refusal is an answer
        (ok ? fits : not_from)[ordinal].store(bytes, std::memory_order_relaxed);
        return ok;
    }
};

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool supported_dims(int d, int dv);
// The window that kernels get: one that no token's first key is behind is none (-1), since a position below zero less it
// could pass 32 bits.  max_keys, tokens: the most of a request.
inline int window_of(int window, long long max_keys, long long tokens) {
    return window >= max_keys || window + tokens > 0x7fffffffLL ? -1 : window;
}
// A contiguous 1-D int32 tensor of n entries.
fa8_status check_int_vec(const fa8_tensor *t, const char *name, long long n);
// E4M3 payload: last dim contiguous, other strides positive multiples of 16 bytes, 16-byte base.
fa8_status check_payload(const fa8_tensor *t, const char *name);
// A tensor that a call writes: refuses one whose entries share memory (an expanded dim).
fa8_status check_written(const fa8_tensor *t, const char *name);
// fp32, 0-d or (B, Hkv); NULL gives a null pointer (1.0).
fa8_status check_descale(const fa8_tensor *t, const char *name, int B, int Hkv, const float **ptr, long long *sb,
                         long long *sh);

// The paged cache's index side: block_table (B, max_pages), cu_seqlens_k (B+1) and, when the new
// tokens are packed, cu_seqlens_q (B+1).
struct Table {
    const int *cu_k = nullptr;
    const int *bt = nullptr;
    long long bt_stride = 0;
    int B = 0, max_pages = 0, page_size = 0;
};
fa8_status check_table(const fa8_tensor *cu_k, const fa8_tensor *bt, int page_size, int B, Table *out);

// TMA map of a paged K or V pool {d, head, row, page} whose boxes are `width` bytes of one head by
// `rows` rows, with the swizzle of that width (128, 64 or 32; none for others).
fa8_status encode_kv(CUtensorMap *m, const fa8_tensor *t, int width, int rows, bool swizzled = true);
// TMA map of Q {d, head, token, request}, boxes of `width` bytes of `heads` x `tokens`
// (packed Q: one request).
fa8_status encode_q(CUtensorMap *m, const fa8_tensor *t, int width, int heads, int tokens);
// The bound on every in-kernel wait (fa8_set_wait_timeout_ns).
unsigned long long wait_timeout_ns();

// Queries (B, Sq, Hq, D) or packed (T, Hq, D) with cu_seqlens_q; strides {request, token, head}.
struct Queries {
    int B = 0, Sq = 0, T = 0, Hq = 0, D = 0;
    const int *cu_q = nullptr;
    long long stride[3] = {0, 0, 0};
};
fa8_status check_queries(const fa8_tensor *q, const fa8_tensor *cu_q, Queries *out);
// q-heads per kv-head, 1 to 128.
fa8_status check_groups(long long Hq, long long Hkv, int *G);
// Page lists (B, Sq, Hkv, K) or (T, Hkv, K), int32, K <= kMaxPageList; strides {request, token, head}.
constexpr int kMaxPageList = 4096;
fa8_status check_page_lists(const fa8_tensor *t, const Queries &q, int Hkv, long long stride[3], int *K);

}  // namespace host
}  // namespace fa8
