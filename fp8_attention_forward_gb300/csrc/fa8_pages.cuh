// fa8_pages.cuh -- device pieces shared by the paged-cache operators: the token's request, the
// warp-level f16 MMA on E4M3 operands, and cluster addressing.
//
// Why warp MMAs here and not tcgen05: these kernels stream a cache past at most 16 query rows, so HBM
// or L2 is the bound and an MMA tile is mostly padding; what costs is the hand-off per tile.  With the
// keys (or pages) on M and the query rows on N = 8, a warp runs its chunks alone, from its own buffer,
// with no barrier or TMEM round trip between warps.  (64 x 8 lists of 2048 keys, d = dv = 128: 48 us; the
// tcgen05 decode kernel of fa8_fwd over as many contiguous keys: 66 us.)  A lane reads 8 or 16 contiguous
// bytes of a row, and because the order of a contraction is free, those bytes serve as its k elements of
// consecutive MMAs.  E4M3 is exact in f16 and products of two are exact in fp32.
#pragma once

#include <stdint.h>

#include "fa8_ptx.cuh"

namespace fa8 {

// Request b, index i within its Lq new tokens, of flat token `tok`; false for rows outside the
// packed sequences.  cu_q null: batched, Sq tokens each.
__device__ __forceinline__ bool locate_token(const int *cu_q, int B, int Sq, int tok, int *b, int *i, int *Lq) {
    if (!cu_q) {
        *b = tok / Sq;
        *i = tok - *b * Sq;
        *Lq = Sq;
        return true;
    }
    int lo = 0, hi = B - 1;  // last request whose first token is <= tok
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (cu_q[mid] <= tok) lo = mid;
        else hi = mid - 1;
    }
    const int start = cu_q[lo], end = cu_q[lo + 1];
    *b = lo;
    *i = tok - start;
    *Lq = end - start;
    return tok >= start && tok < end;
}

// D (16x8 fp32) += A (16x16 f16, row) B (16x8 f16, col)
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// transpose of an 8x8 matrix of 16-bit elements held in MMA fragment layout
__device__ __forceinline__ uint32_t trans8x8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
// four E4M3 bytes -> two f16 pairs (bytes 0, 1 and 2, 3)
__device__ __forceinline__ void e4m3x4_to_h2(uint32_t w, uint32_t &lo, uint32_t &hi) {
    lo = ptx::e4m3x2_to_h2(w);
    hi = ptx::e4m3x2_to_h2(w >> 16);
}
// {hi, lo} -> f16x2 (lo in the low half), round to nearest even, saturating; NaN stays
__device__ __forceinline__ uint32_t cvt_f16x2_sat(float hi, float lo) {
    uint32_t d;
    asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}
// two 16 x 16 byte tiles transposed, rows at the addresses of lanes 0 .. 15 and 16 .. 31: lane (r, c) gets
// column r of rows 4c .. 4c + 3 and column r + 8 of them, of either tile
__device__ __forceinline__ void ld_trans_b8(uint32_t (&d)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0, %1, %2, %3}, [%4];"
                 : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void st_shared_zero16(uint32_t addr) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(addr), "r"(0) : "memory");
}

template <int N>
struct Bytes {
    uint32_t w[N / 4];
};
// read-once global load of 16 bytes (no L1 allocation)
__device__ __forceinline__ Bytes<16> ld_stream(const uint8_t *p) {
    Bytes<16> r;
    asm volatile("ld.global.nc.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3])
                 : "l"(p));
    return r;
}
// N bytes of shared memory, aligned to N (12: to 4)
template <int N>
__device__ __forceinline__ Bytes<N> ld_shared(uint32_t addr) {
    Bytes<N> r;
    if constexpr (N == 16) {
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3]) : "r"(addr) : "memory");
    } else if constexpr (N == 8) {
        asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(r.w[0]), "=r"(r.w[1]) : "r"(addr) : "memory");
    } else {
#pragma unroll
        for (int i = 0; i < N / 4; ++i) asm volatile("ld.shared.b32 %0, [%1];" : "=r"(r.w[i]) : "r"(addr + 4 * i) : "memory");
    }
    return r;
}

// ---------------------------------------------------------------- asynchronous copies
// 16 bytes past L1; `bytes` = 0 reads nothing and writes zeros
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// waits until at most N of this thread's groups are pending
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// ---------------------------------------------------------------- clusters
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// every thread of every CTA of the cluster: writes before are visible after
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// address of a shared-memory word in CTA `rank` of the cluster
__device__ __forceinline__ uint32_t map_rank(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ float2 ld_cluster_f2(uint32_t addr) {
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void st_cluster_f32(uint32_t addr, float v) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

}  // namespace fa8
