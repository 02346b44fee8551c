// fa8_scored_few.cuh -- attention with capped, biased or masked scores for at most 16 query rows per kv-head
// (decode steps, small trees of drafted tokens): bound by the one read of K and V.
//
//   S^T (16 keys x 8 rows) = K . Q^T,  O^T (16 dv x 8 rows) += V^T . P^T      f16 MMAs on exactly widened E4M3
//
// As in the attention over listed pages, a warp works alone: every (warps x cluster)-th chunk of 16, 32 or 64 keys,
// its own running maximum, sum and O^T in registers, one K and one V buffer that TMA fills, merged at
// the end over the warps and, through distributed shared memory, the CTAs of a cluster.  The rows
// are the request's tokens x the q-heads of one kv-head, so a chunk can be visible to some of them
// alone: chunks inside every row's range take no mask.
//
// Measured (us; capped, d = 128, 16-key pages): 64 requests of 1024 .. 32768 keys, 64 q-heads on 8 362 to 375, from run to run
// (2.2 GB, 5.9 to 6.1 TB/s of 6.8 that a copy gets), 32 of 4096 keys 58, one of 4096 11 (a chain of dependent loads: lengths,
// table, keys, then the merge), of 131072 52.  From 9 rows on each K and V fragment feeds two MMAs, and from 2 x 8 rows the MMAs and
// conversions, not the memory, bound it.
#pragma once

#include <math.h>
#include <string.h>

#include <algorithm>
#include <numeric>

#include "fa8_host.h"
#include "fa8_scored.cuh"

namespace fa8 {

constexpr int kFewMaxCluster = 16;
// P is taken against 2^kFewBias below the row's maximum, which moves only for scores 2^kFewSlack above it: p <= 2^15 stays in
// f16's range, and a weight down to 2^-32 of the largest still counts in P V (of the kernel for many rows, whose slack is
// wider since it pays more for a move, 2^-28), every one in the sum.
constexpr float kFewBias = 7.f, kFewSlack = 8.f;

template <int D, int DV, int NT, int PW>
struct FewCfg {
    static constexpr int ROWS = 8 * NT;
    // 16-key tiles per chunk
    static constexpr int MT = D + DV <= 192 && NT == 1 ? 4 : (D + DV <= 256 ? 2 : 1);
    static constexpr int KC = 16 * MT, NG = 2 * MT;  // keys, 8-key groups
    // rows arrive as blocks of CW bytes, each block KC rows deep with the swizzle of its width
    static constexpr int CW = D % 128 == 0 ? 128 : (D % 64 == 0 ? 64 : 96), NCK = D / CW;
    static constexpr int CWV = DV % 128 == 0 ? 128 : (DV % 64 == 0 ? 64 : 96), NCV = DV / CWV;
    static constexpr int VK = CW == 96 ? 8 : 16;  // bytes of one K fragment load
    static constexpr int NKV = D / (4 * VK);      // K fragment loads per key and lane
    static constexpr int STEPS = D / 16;
    static constexpr bool HELD = NT * STEPS <= 8;  // Q's fragments in registers
    static constexpr int DT = DV / 16;
    static constexpr int OPITCH = DV + 4;
    static constexpr int K_STAGE = KC * D, V_STAGE = KC * DV, STAGE = K_STAGE + V_STAGE;
    static constexpr int Q_BYTES = NT * STEPS * 32 * 8;
    static constexpr int MERGE_BYTES = PW * ROWS * (OPITCH + 2) * 4;
    static constexpr int OFF_Q = PW * STAGE;
    static constexpr int SMEM_BYTES = 1024 + (OFF_Q + Q_BYTES > MERGE_BYTES ? OFF_Q + Q_BYTES : MERGE_BYTES);
    // CTAs per SM that registers are cut to
    static constexpr int CTAS = PW > 4 ? 1 : (NT == 2 && D + DV > 256 ? 2 : 4);
    static __device__ __forceinline__ int k_dim(int v, int c) {
        return CW == 128 ? (v >> 1) * 128 + 16 * (2 * c + (v & 1)) : 4 * VK * v + VK * c;
    }
    template <int W>
    static __device__ __forceinline__ int at(int row, int x) {
        const int piece = (x % W) >> 4, sw = W == 128 ? row & 7 : (W == 64 ? (row >> 1) & 3 : 0);
        return (x / W) * KC * W + row * W + 16 * (piece ^ sw) + (x & 15);
    }
};

// Notes, for each row that sees one, the channels of the NaNs in V's chunks of kc keys that are marked (modulo 32): chunk it
// begins at key k0 + it * step.  A lane looks through a key.  Whole warp.
template <int DV>
static __device__ __noinline__ void few_nans(const ScoredParams &p, int b, int kvh, int k0, int step, int kc, int chunks, const uint8_t *marked,
                                             uint32_t *s_bad) {
    const int lane = threadIdx.x & 31;
    ScReq rq;
    sc_lengths(p, b, &rq);
    for (int it = 0; it < chunks; ++it) {
        if (!marked[it & 31]) continue;
        for (int h = lane; h < kc; h += 32) {
            const int j = k0 + it * step + h;
            const uint8_t *v = j < rq.Lk ? sc_v_row(p, b, rq, kvh, j) : nullptr;
            if (!v) continue;
            uint32_t bits[DV / 32], any = 0;
#pragma unroll
            for (int w = 0; w < DV / 32; ++w) {
                const uint4 x = *reinterpret_cast<const uint4 *>(v + 32 * w), y = *reinterpret_cast<const uint4 *>(v + 32 * w + 16);
                any |= bits[w] = sc_nans({x.x, x.y, x.z, x.w}) | sc_nans({y.x, y.y, y.z, y.w}) << 16;
            }
            for (int i = 0; any && i < p.Sq; ++i) {
                if (!sc_sees(sc_row(p, b, rq, i), p.words, j)) continue;
                for (int rw = i * p.G; rw < (i + 1) * p.G; ++rw)
#pragma unroll
                    for (int w = 0; w < DV / 32; ++w)
                        if (bits[w] & ~*reinterpret_cast<volatile uint32_t *>(s_bad + rw * (DV / 32) + w)) atomicOr(s_bad + rw * (DV / 32) + w, bits[w]);
            }
        }
    }
}

template <int D, int DV, int NT, int PW>
__global__ void __launch_bounds__(32 * PW, FewCfg<D, DV, NT, PW>::CTAS)
    scored_few_kernel(const __grid_constant__ ScoredParams p, const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v) {
    using C = FewCfg<D, DV, NT, PW>;
    constexpr int kThreads = 32 * PW;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    __shared__ __align__(8) uint64_t s_bar[PW][2];
    __shared__ int s_abort, s_nan;
    __shared__ __align__(4) uint8_t s_noted[32 * PW];  // each warp's chunks with NaNs, modulo 32
    __shared__ float s_m[C::ROWS], s_l[C::ROWS];
    __shared__ uint32_t s_bad[C::ROWS * (DV / 32)];  // channels of the rows' outputs that are NaN
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int r = lane >> 2, c = lane & 3;
    const int CS = p.cluster;
    const int rank = CS > 1 ? (int)cluster_rank() : 0;
    const int tile = blockIdx.x / (CS * p.parts), piece = blockIdx.x / CS % p.parts, kvh = tile % p.Hkv, b = tile / p.Hkv;
    if (p.parts > 1) ptx::griddep_launch_dependents();  // the joining kernel waits for all of this one
    const int rows = p.Sq * p.G;
    const int h0 = kvh * p.G;
    ScReq rq;
    sc_request(p, b, &rq);
    const float dqv = p.dq ? __ldg(p.dq + b * p.dq_s[0] + kvh * p.dq_s[1]) : 1.f;
    const float dkv = p.dk ? __ldg(p.dk + b * p.dk_s[0] + kvh * p.dk_s[1]) : 1.f;
    if (tid == 0) {
        s_abort = s_nan = 0;
        if (p.has_kv) {
            ptx::prefetch_tmap(&tm_k);
            ptx::prefetch_tmap(&tm_v);
        }
    }
    if (tid < C::ROWS * (DV / 32)) s_bad[tid] = 0;
    static_assert(C::ROWS * (DV / 32) <= kThreads, "one each");
    s_noted[tid] = 0;
    const uint32_t bar_k = ptx::smem_u32(s_bar[warp]), bar_v = bar_k + 8;
    if (lane == 0) {
        ptx::mbar_init(bar_k, 1);
        ptx::mbar_init(bar_v, 1);
        ptx::fence_mbar_init();
        ptx::fence_proxy_async_smem();
    }
    // what this lane's rows 2c, 2c + 1 (and 8 more) see; rows that are not there see everything
    ScRow row[NT][2];
    int flo = 0, fhi = 0x7fffffff, slo = 0x7fffffff, shi = 0;  // seen by all rows, by some
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int rw = 8 * t + 2 * c + e;
            ScRow &x = row[t][e];
            x.lo = 0;
            x.hi = x.lp = 0x7fffffff;
            x.words = nullptr;
            if (rw < rows) {
                x = sc_row(p, b, rq, rw / p.G);
                flo = max(flo, x.lo);
                fhi = min(fhi, min(x.hi, max(0, x.lp)));
                if (x.hi > x.lo) {
                    slo = min(slo, x.lo);
                    shi = max(shi, x.hi);
                }
            }
        }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
        flo = max(flo, __shfl_xor_sync(0xffffffffu, flo, o));
        fhi = min(fhi, __shfl_xor_sync(0xffffffffu, fhi, o));
        slo = min(slo, __shfl_xor_sync(0xffffffffu, slo, o));
        shi = max(shi, __shfl_xor_sync(0xffffffffu, shi, o));
    }
    const int c0 = shi > slo ? slo / C::KC : 0;                                  // first chunk
    const int all = shi > slo ? (shi + C::KC - 1) / C::KC - c0 : 0;
    uint2 *qf = reinterpret_cast<uint2 *>(smem + C::OFF_Q);
    {
        const uint8_t *q = p.q + (long long)b * p.q_s[0] + (long long)h0 * p.q_s[2];
        for (int x = tid; x < NT * C::STEPS * 32; x += kThreads) {
            const int ln = x & 31, st = (x >> 5) % C::STEPS, nt = x / (32 * C::STEPS);
            const int qr = nt * 8 + (ln >> 2);
            constexpr int SPV = C::VK / 4;  // k-steps fed by one fragment load
            const int at = C::k_dim(st / SPV, ln & 3) + 4 * (st % SPV);
            uint32_t lo = 0, hi = 0;
            if (qr < rows) e4m3x4_to_h2(*reinterpret_cast<const uint32_t *>(q + (qr / p.G) * p.q_s[1] + (qr % p.G) * p.q_s[2] + at), lo, hi);
            qf[x] = make_uint2(lo, hi);
        }
    }
    __syncthreads();
    float cs = p.scale_log2 * dqv * dkv;
    if (cs == 0.f) cs = 0x1p-126f;  // below fp32: a masked -inf must stay one
    const float cap = p.cap_log2, k2 = cap > 0.f ? sc_k2(cs, cap) : 0.f;
    float slope[NT][2];
    int pc[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int rw = 8 * t + 2 * c + e;
            slope[t][e] = 0.f;
            pc[t][e] = 0;
            if (p.slopes && rw < rows) {
                const ScBias bs = sc_bias(p, row[t][e], rw / p.G + rq.Lk - rq.Lq, h0 + rw % p.G);
                slope[t][e] = bs.slope;
                pc[t][e] = bs.pc;
            }
        }

    // ---- the warp's chunk buffers, as chunk first + it * stride of the range; a lane's box of it: page, row
    const int first = (warp * p.parts + piece) * CS + rank, stride = CS * p.parts * PW;
    const uint32_t ks = ptx::smem_u32(smem) + warp * C::STAGE, vs = ks + C::K_STAGE;
    const int vrow = 2 * ((lane >> 2) & 3) + (lane & 1) + 8 * ((lane >> 1) & 1);
    const int nb = 1 << p.box_shift, mine = lane & (nb - 1), part = lane >> p.box_shift;
    const int chunks = all > first ? (all - first + stride - 1) / stride : 0;
    constexpr int kNoEntry = -0x7fffffff;
    const int *bt = p.bt + (long long)b * p.bt_stride;
    auto entry = [&](int it) -> int {  // table entry of this lane's box of chunk it
        const int j = (c0 + first + it * stride) * C::KC + mine * p.box_n;
        return it < chunks && j < rq.Lk ? bt[j / p.page_size] : kNoEntry;
    };
    int page = 0, prow = 0, ahead = kNoEntry;
    auto locate = [&](int it) {
        const int j = (c0 + first + it * stride) * C::KC + mine * p.box_n;
        if (p.kv_mode == 2) {
            page = ahead;
            if (page < 0 || page >= p.num_pages) {
                if (page != kNoEntry) atomicOr(p.status, kStatusBounds);
                page = p.num_pages;  // out of range: TMA fills zeros
            }
            prow = j % p.page_size;
            ahead = entry(it + 1);
        } else {
            page = p.kv_mode == 1 ? 0 : b;
            prow = rq.k0 + j;
        }
    };
    auto fetch_k = [&]() {
        if (lane == 0) ptx::mbar_arrive_expect_tx(bar_k, (uint32_t)C::K_STAGE);
        __syncwarp();
        if (part < C::NCK) ptx::tma_load_4d(ks + part * C::KC * C::CW + mine * p.box_n * C::CW, &tm_k, bar_k, part * C::CW, kvh, prow, page);
    };
    auto fetch_v = [&]() {
        if (lane == 0) ptx::mbar_arrive_expect_tx(bar_v, (uint32_t)C::V_STAGE);
        __syncwarp();
        if (part < C::NCV) ptx::tma_load_4d(vs + part * C::KC * C::CWV + mine * p.box_n * C::CWV, &tm_v, bar_v, part * C::CWV, kvh, prow, page);
    };
    const Waiter W{&s_abort, p.timeout_ns, p.status};
    if (chunks > 0) {
        if (p.kv_mode == 2) ahead = entry(0);
        locate(0);
        fetch_k();
        fetch_v();
    }
    float m[NT][2], l[NT][2];
    float o[C::DT][NT][4];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            m[t][e] = -INFINITY;
            l[t][e] = 0.f;
        }
#pragma unroll
    for (int d = 0; d < C::DT; ++d)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[d][t][e] = 0.f;
    uint2 qh[C::HELD ? NT * C::STEPS : 1];
    if constexpr (C::HELD) {
#pragma unroll
        for (int i = 0; i < NT * C::STEPS; ++i) qh[i] = qf[i * 32 + lane];
    }

    for (int it = 0; it < chunks; ++it) {
        const int k0 = (c0 + first + it * stride) * C::KC;
        const bool more = it + 1 < chunks;
        if (!W.wait_warp(bar_k, it & 1)) {  // another warp may have given up: this one's copies are still on their way
            W.drain(bar_k, it & 1);
            W.drain(bar_v, it & 1);
            break;
        }
        // ---- S^T
        float s[C::MT][NT][4];
#pragma unroll
        for (int x = 0; x < C::MT; ++x)
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[x][t][e] = 0.f;
#pragma unroll
        for (int j = 0; j < C::NKV; ++j) {
            Bytes<C::VK> kr[C::NG];
#pragma unroll
            for (int i = 0; i < C::NG; ++i) kr[i] = ld_shared<C::VK>(ks + C::template at<C::CW>(8 * i + r, C::k_dim(j, c)));
#pragma unroll
            for (int w = 0; w < C::VK / 4; ++w) {
                uint2 bf[NT];
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    const int i = t * C::STEPS + j * (C::VK / 4) + w;
                    if constexpr (C::HELD) bf[t] = qh[i];
                    else bf[t] = qf[i * 32 + lane];
                }
#pragma unroll
                for (int x = 0; x < C::MT; ++x) {
                    uint32_t a0, a1, a2, a3;
                    e4m3x4_to_h2(kr[2 * x].w[w], a0, a2);
                    e4m3x4_to_h2(kr[2 * x + 1].w[w], a1, a3);
#pragma unroll
                    for (int t = 0; t < NT; ++t) mma_f16(s[x][t], a0, a1, a2, a3, bf[t].x, bf[t].y);
                }
            }
        }
        __syncwarp();  // every lane has read the K buffer
        if (more) {
            locate(it + 1);
            fetch_k();
        }
        // ---- scores in log2 units: element [x][t][2 h + e] is key 16 x + 8 h + r, row 8 t + 2 c + e
        if (cap > kFarCap) {
#pragma unroll
            for (int x = 0; x < C::MT; ++x)
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[x][t][e] = sc_cap(s[x][t][e], cs, k2, cap);
        } else if (cap > 0.f) {
#pragma unroll
            for (int x = 0; x < C::MT; ++x)
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[x][t][e] = sc_cap_near(s[x][t][e], k2, cap);
        } else {
#pragma unroll
            for (int x = 0; x < C::MT; ++x)
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[x][t][e] *= cs;
        }
        if (p.slopes) {
#pragma unroll
            for (int x = 0; x < C::MT; ++x)
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        s[x][t][e] = fmaf(-slope[t][e & 1], fabsf((float)(pc[t][e & 1] - (k0 + 16 * x + 8 * (e >> 1) + r))), s[x][t][e]);
        }
        const bool partial = k0 < flo || k0 + C::KC > fhi;
        uint32_t any[(C::KC + 31) / 32], every[(C::KC + 31) / 32];  // keys that some row, that every row sees
        if (partial) {
#pragma unroll
            for (int w = 0; w < (C::KC + 31) / 32; ++w) {
                any[w] = 0;
                every[w] = 0xffffffffu;
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const uint32_t see = sc_see32(row[t][e], p.words, k0 + 32 * w);
                        if (8 * t + 2 * c + e < rows) {
                            any[w] |= see;
                            every[w] &= see;
                        }
#pragma unroll
                        for (int x = 2 * w; x < 2 * w + 2 && x < C::MT; ++x)
#pragma unroll
                            for (int h = 0; h < 2; ++h)
                                if (!(see >> (16 * (x - 2 * w) + 8 * h + r) & 1u)) s[x][t][2 * h + e] = -INFINITY;
                    }
#pragma unroll
                for (int sh = 1; sh < 4; sh <<= 1) {
                    any[w] |= __shfl_xor_sync(0xffffffffu, any[w], sh);
                    every[w] &= __shfl_xor_sync(0xffffffffu, every[w], sh);
                }
            }
        }
        // ---- softmax: the maximum that P is taken against moves only for scores 2^kFewSlack above it
        uint32_t pb[C::MT][NT][2];
        float mx[NT][2];
        bool moved = false;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float y = -INFINITY;
#pragma unroll
                for (int x = 0; x < C::MT; ++x) y = fmaxf(y, fmaxf(s[x][t][e], s[x][t][2 + e]));
                mx[t][e] = y;
                moved |= y > m[t][e] + (kFewBias + kFewSlack);
            }
        if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float mn = mx[t][e];
#pragma unroll
                    for (int sh = 4; sh < 32; sh <<= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, sh));
                    mn = fmaxf(m[t][e], mn - kFewBias);
                    const float alpha = mn == -INFINITY ? 1.f : ptx::ex2(m[t][e] - mn);  // 0 while nothing has been seen
                    m[t][e] = mn;
                    l[t][e] *= alpha;
#pragma unroll
                    for (int d = 0; d < C::DT; ++d) {
                        o[d][t][e] *= alpha;
                        o[d][t][2 + e] *= alpha;
                    }
                }
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const float r0 = m[t][0] == -INFINITY ? 0.f : m[t][0], r1 = m[t][1] == -INFINITY ? 0.f : m[t][1];
#pragma unroll
            for (int x = 0; x < C::MT; ++x)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float p0 = ptx::ex2(s[x][t][2 * h] - r0), p1 = ptx::ex2(s[x][t][2 * h + 1] - r1);
                    l[t][0] += p0;
                    l[t][1] += p1;
                    pb[x][t][h] = trans8x8(cvt_f16x2_sat(p1, p0));
                }
        }
        // ---- O^T
        if (!W.wait_warp(bar_v, it & 1)) {
            W.drain(bar_v, it & 1);
            if (more) W.drain(bar_k, (it + 1) & 1);
            break;
        }
        if (partial) {
            // rows of V that no row sees may hold anything: they become zeros; of those that some rows see the
            // NaNs do, and go into those rows' outputs at the end
#pragma unroll
            for (int i = 0; i < (C::KC + 31) / 32; ++i) {
                const bool none = !(any[i] >> lane & 1u), some = !(every[i] >> lane & 1u);
                if (lane + 32 * i < C::KC && (none || some)) {
#pragma unroll 1
                    for (int d = 0; d < DV; d += 16) {
                        const uint32_t a = vs + C::template at<C::CWV>(lane + 32 * i, d);
                        if (none) {
                            st_shared_zero16(a);
                            continue;
                        }
                        Bytes<16> w = ld_shared<16>(a);
                        uint32_t bad = 0;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const uint32_t n = ((w.w[e] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
                            bad |= n;
                            w.w[e] &= ~((n >> 7) * 0xffu);
                        }
                        if (bad) {
                            s_noted[32 * warp + (it & 31)] = 1;
                            ptx::st_shared_v4(a, w.w[0], w.w[1], w.w[2], w.w[3]);
                        }
                    }
                }
            }
            ptx::fence_proxy_async_smem();
            __syncwarp();
        }
#pragma unroll
        for (int x = 0; x < C::MT; ++x) {
#pragma unroll
            for (int w = 0; w < DV / 32; ++w) {
                uint32_t z[4], a0, a1, a2, a3;
                ld_trans_b8(z, vs + C::template at<C::CWV>(16 * x + vrow, 32 * w + 16 * (lane >> 4)));
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    e4m3x4_to_h2(z[2 * h], a0, a2);
                    e4m3x4_to_h2(z[2 * h + 1], a1, a3);
#pragma unroll
                    for (int t = 0; t < NT; ++t) mma_f16(o[2 * w + h][t], a0, a1, a2, a3, pb[x][t][0], pb[x][t][1]);
                }
            }
        }
        __syncwarp();  // and the V buffer
        if (more) fetch_v();
    }

    // ---- merge: warps through shared memory, CTAs through distributed shared memory
    __syncthreads();  // the buffers and Q are done with
    float *wo = reinterpret_cast<float *>(smem);                         // [warp][row][OPITCH]
    float *wm = wo + PW * C::ROWS * C::OPITCH, *wl = wm + PW * C::ROWS;  // [warp][row]
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float x = l[t][e];
#pragma unroll
            for (int sh = 4; sh < 32; sh <<= 1) x += __shfl_xor_sync(0xffffffffu, x, sh);
            const int rw = 8 * t + 2 * c + e;
            if (r == 0) {
                wm[warp * C::ROWS + rw] = m[t][e];
                wl[warp * C::ROWS + rw] = x;
            }
#pragma unroll
            for (int d = 0; d < C::DT; ++d)
#pragma unroll
                for (int h = 0; h < 2; ++h) wo[(warp * C::ROWS + rw) * C::OPITCH + 16 * d + 8 * h + r] = o[d][t][2 * h + e];
        }
    if (__any_sync(0xffffffffu, s_noted[32 * warp + lane])) {
        s_nan = 1;
        few_nans<DV>(p, b, kvh, (c0 + first) * C::KC, stride * C::KC, C::KC, chunks, s_noted + 32 * warp, s_bad);
    }
    __syncthreads();
    for (int x = tid; x < rows * (DV / 2); x += kThreads) {
        const int rw = x / (DV / 2), d = 2 * (x - rw * (DV / 2));
        float M = wm[rw];
#pragma unroll
        for (int w = 1; w < PW; ++w) M = fmaxf(M, wm[w * C::ROWS + rw]);
        const float ref = M == -INFINITY ? 0.f : M;
        float a0 = 0.f, a1 = 0.f, L = 0.f;
#pragma unroll
        for (int w = 0; w < PW; ++w) {
            const float f = ptx::ex2(wm[w * C::ROWS + rw] - ref);
            const float2 y = *reinterpret_cast<const float2 *>(wo + (w * C::ROWS + rw) * C::OPITCH + d);
            a0 = fmaf(f, y.x, a0);
            a1 = fmaf(f, y.y, a1);
            L = fmaf(f, wl[w * C::ROWS + rw], L);
        }
        *reinterpret_cast<float2 *>(wo + rw * C::OPITCH + d) = make_float2(a0, a1);
        if (d == 0) {
            s_m[rw] = M;
            s_l[rw] = L;
        }
    }
    if (CS > 1) cluster_sync();
    else __syncthreads();
    const float dvv = p.dv ? p.dv[b * p.dv_s[0] + kvh * p.dv_s[1]] : 1.f;
    const uint32_t a_m = ptx::smem_u32(s_m), a_l = ptx::smem_u32(s_l), a_o = ptx::smem_u32(wo), a_n = ptx::smem_u32(&s_nan);
    bool nan = false;
    if (CS > 1) {
        for (int k = 0; k < CS; ++k) nan |= __float_as_int(ld_cluster_f32(map_rank(a_n, k))) != 0;
    } else {
        nan = s_nan != 0;
    }
    const int total = rows * (DV / 2), share = (total + CS - 1) / CS;
    for (int x = rank * share + tid; x < min(total, (rank + 1) * share); x += kThreads) {
        const int rw = x / (DV / 2), d = 2 * (x - rw * (DV / 2));
        float M, L, a0, a1;
        if (CS > 1) {
            float mr[kFewMaxCluster];
            M = -INFINITY;
            for (int k = 0; k < CS; ++k) M = fmaxf(M, mr[k] = ld_cluster_f32(map_rank(a_m + 4u * rw, k)));
            const float ref = M == -INFINITY ? 0.f : M;
            L = a0 = a1 = 0.f;
            for (int k = 0; k < CS; ++k) {
                const float f = ptx::ex2(mr[k] - ref);
                const float2 y = ld_cluster_f2(map_rank(a_o + 4u * (uint32_t)(rw * C::OPITCH + d), k));
                a0 = fmaf(f, y.x, a0);
                a1 = fmaf(f, y.y, a1);
                L = fmaf(f, ld_cluster_f32(map_rank(a_l + 4u * rw, k)), L);
            }
        } else {
            M = s_m[rw];
            L = s_l[rw];
            a0 = wo[rw * C::OPITCH + d];
            a1 = wo[rw * C::OPITCH + d + 1];
        }
        const int i = rw / p.G, hq = h0 + rw % p.G;
        if (p.slopes) M += sc_bias(p, sc_row(p, b, rq, i), i + rq.Lk - rq.Lq, hq).off;
        if (nan) {
            const int word = rw * (DV / 32) + d / 32;
            uint32_t bad = s_bad[word];
            for (int k = 0; CS > 1 && k < CS; ++k) bad |= __float_as_uint(ld_cluster_f32(map_rank(ptx::smem_u32(s_bad + word), k)));
            if (bad >> (d & 31) & 1u) a0 = NAN;
            if (bad >> (d & 31) & 2u) a1 = NAN;
        }
        if (p.parts > 1) {
            const long long at = (long long)(blockIdx.x / CS) * rows + rw;
            *reinterpret_cast<float2 *>(p.part + at * DV + d) = make_float2(a0, a1);
            if (d == 0) reinterpret_cast<float2 *>(p.part + (long long)(gridDim.x / CS) * rows * DV)[at] = make_float2(M, L);
            continue;
        }
        float f, lse;
        sc_finish(M, L, p.sink ? p.sink + hq : nullptr, dvv, &f, &lse);
        uint8_t *dst = reinterpret_cast<uint8_t *>(p.o) + 2 * ((long long)b * p.o_s[0] + i * p.o_s[1] + (long long)hq * p.o_s[2] + d);
        if (p.out_fp16) *reinterpret_cast<__half2 *>(dst) = __floats2half2_rn(a0 * f, a1 * f);
        else *reinterpret_cast<__nv_bfloat162 *>(dst) = __floats2bfloat162_rn(a0 * f, a1 * f);
        if (d == 0 && p.lse) p.lse[(long long)b * p.lse_s[0] + i * p.lse_s[1] + (long long)hq * p.lse_s[2]] = lse;
    }
    if (CS > 1) cluster_sync();  // no CTA leaves while its shared memory is still read
}

// The parts of long requests, joined by their maxima: CTA = row, thread = two columns.
template <int DV>
__global__ void __launch_bounds__(DV / 2) scored_few_merge_kernel(const __grid_constant__ ScoredParams p, int tiles) {
    const int rows = p.Sq * p.G, tile = blockIdx.x / rows, rw = blockIdx.x - tile * rows, kvh = tile % p.Hkv, b = tile / p.Hkv;
    const int i = rw / p.G, hq = kvh * p.G + rw % p.G, d = 2 * threadIdx.x;
    const float sink = p.sink ? p.sink[hq] : 0.f, dv = p.dv ? p.dv[b * p.dv_s[0] + kvh * p.dv_s[1]] : 1.f;
    const float *po = p.part + ((long long)tile * p.parts * rows + rw) * DV + d;
    const float2 *pm = reinterpret_cast<const float2 *>(p.part + (long long)tiles * p.parts * rows * DV) + (long long)tile * p.parts * rows + rw;
    ptx::griddep_wait();
    constexpr int NB = 8;  // parts in flight
    float M = -INFINITY, L = 0.f, a0 = 0.f, a1 = 0.f;
    for (int k0 = 0; k0 < p.parts; k0 += NB) {
        float2 ml[NB], y[NB];
#pragma unroll
        for (int k = 0; k < NB; ++k) {
            const bool in = k0 + k < p.parts;
            ml[k] = in ? pm[(long long)(k0 + k) * rows] : make_float2(-INFINITY, 0.f);
            y[k] = in ? *reinterpret_cast<const float2 *>(po + (long long)(k0 + k) * rows * DV) : make_float2(0.f, 0.f);
        }
        float top = M;
#pragma unroll
        for (int k = 0; k < NB; ++k) top = fmaxf(top, ml[k].x);
        const float ref = top == -INFINITY ? 0.f : top, a = ptx::ex2(M - ref);
        L *= a;
        a0 *= a;
        a1 *= a;
#pragma unroll
        for (int k = 0; k < NB; ++k) {
            const float f = ptx::ex2(ml[k].x - ref);
            L = fmaf(f, ml[k].y, L);
            a0 = fmaf(f, y[k].x, a0);
            a1 = fmaf(f, y[k].y, a1);
        }
        M = top;
    }
    float f, lse;
    sc_finish(M, L, p.sink ? &sink : nullptr, dv, &f, &lse);
    uint8_t *dst = reinterpret_cast<uint8_t *>(p.o) + 2 * ((long long)b * p.o_s[0] + i * p.o_s[1] + (long long)hq * p.o_s[2] + d);
    if (p.out_fp16) *reinterpret_cast<__half2 *>(dst) = __floats2half2_rn(a0 * f, a1 * f);
    else *reinterpret_cast<__nv_bfloat162 *>(dst) = __floats2bfloat162_rn(a0 * f, a1 * f);
    if (d == 0 && p.lse) p.lse[(long long)b * p.lse_s[0] + i * p.lse_s[1] + (long long)hq * p.lse_s[2]] = lse;
}

template <int D, int DV, int NT, int PW>
fa8_status launch_few(ScoredParams &p, const fa8_tensor *k, const fa8_tensor *v, int tiles, int dev, cudaStream_t s) {
    static host::SmemOptIn opt_in;
    using C = FewCfg<D, DV, NT, PW>;
    p.box_n = p.kv_mode == 2 ? std::gcd(p.page_size, C::KC) : C::KC;
    p.box_shift = 0;
    while (p.box_n << p.box_shift < C::KC) ++p.box_shift;
    CUtensorMap tk, tv;
    memset(&tk, 0, sizeof(tk));
    memset(&tv, 0, sizeof(tv));
    if (p.has_kv) {
        fa8_status st;
        if ((st = host::encode_kv(&tk, k, C::CW, p.box_n)) || (st = host::encode_kv(&tv, v, C::CWV, p.box_n))) return st;
    }
    cudaError_t e = opt_in(scored_few_kernel<D, DV, NT, PW>, C::SMEM_BYTES, dev);
    if (e != cudaSuccess) return host::cuda_fail(e, "scored attention shared memory");
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)tiles * (unsigned)p.parts * (unsigned)p.cluster);
    cfg.blockDim = dim3(32 * PW);
    cfg.dynamicSmemBytes = C::SMEM_BYTES;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = p.cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    static host::Cluster16 cluster16;
    if (p.cluster > 8 && !cluster16(scored_few_kernel<D, DV, NT, PW>, cfg, dev)) {
        p.cluster = attr[0].val.clusterDim.x = 8;
        cfg.gridDim = dim3((unsigned)tiles * (unsigned)p.parts * 8u);
    }
    e = cudaLaunchKernelEx(&cfg, scored_few_kernel<D, DV, NT, PW>, p, tk, tv);
    if (e == cudaSuccess && p.parts > 1) {
        cfg.gridDim = dim3((unsigned)tiles * (unsigned)(p.Sq * p.G));
        cfg.blockDim = dim3(DV / 2);
        cfg.dynamicSmemBytes = 0;
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        e = cudaLaunchKernelEx(&cfg, scored_few_merge_kernel<DV>, p, tiles);
    }
    return e == cudaSuccess ? FA8_SUCCESS : host::cuda_fail(e, "scored attention kernel launch");
}

// Clusters share a request's keys while all of them run at once and every warp keeps at least two chunks, and
// further while a CTA keeps 1024 keys, so that long requests of a ragged batch do not end alone; where
// clusters of the most CTAs leave a quarter of the SMs empty, CTAs have eight warps.  The most is 16 where those fill no
// more than half of the SMs, else eight: a cluster takes its SMs from one of the eight groups that the chip is made of, and
// where another user's SMs or the group's size leave it fewer than 16, clusters wait for each other (one request of
// 131072 keys, d = 256, one kv-head: 170 us in a cluster of 8, 90 of 16; of 4096 keys and 8 kv-heads: 10.5 and 12).
template <int D, int DV>
fa8_status launch_few_rows(ScoredParams &p, const fa8_tensor *k, const fa8_tensor *v, int tiles, long long max_keys, int sm_count, int dev,
                           cudaStream_t s) {
    const int nt = p.Sq * p.G <= 8 ? 1 : 2;
    const long long keys = p.window_left >= 0 ? std::min<long long>(max_keys, (long long)p.window_left + p.Sq) : max_keys;
    const int kc = nt == 1 ? FewCfg<D, DV, 1, 4>::KC : FewCfg<D, DV, 2, 4>::KC, per_sm = nt == 1 ? FewCfg<D, DV, 1, 4>::CTAS : FewCfg<D, DV, 2, 4>::CTAS;
    const int most = p.parts == 1 && (long long)tiles * kFewMaxCluster * 2 <= sm_count ? kFewMaxCluster : 8;
    p.cluster = 1;
    while (p.cluster < most &&
           ((long long)tiles * p.cluster * 2 <= (long long)per_sm * sm_count ? keys >= 2LL * kc * 4 * p.cluster * 2 : keys >= 1024LL * p.cluster * 2))
        p.cluster *= 2;
    if (p.cluster < 8 || p.window_left >= 0) p.parts = 1;  // (too few keys for it)
    const bool wide = p.parts == 1 && p.cluster == most && (long long)tiles * p.cluster * 4 <= 3LL * sm_count && keys >= 2LL * kc * 8 * p.cluster;
    if (nt == 1) return wide ? launch_few<D, DV, 1, 8>(p, k, v, tiles, dev, s) : launch_few<D, DV, 1, 4>(p, k, v, tiles, dev, s);
    return wide ? launch_few<D, DV, 2, 8>(p, k, v, tiles, dev, s) : launch_few<D, DV, 2, 4>(p, k, v, tiles, dev, s);
}

#define FA8_DEFINE_SCORED_FEW(D_, DV_)                                                                                             \
    template <>                                                                                                                    \
    fa8_status launch_scored_few<D_, DV_>(ScoredParams & p, const fa8_tensor *k, const fa8_tensor *v, int tiles,                   \
                                          long long max_keys, int sm_count, int dev, cudaStream_t s) {                             \
        return launch_few_rows<D_, DV_>(p, k, v, tiles, max_keys, sm_count, dev, s);                                               \
    }

}  // namespace fa8
