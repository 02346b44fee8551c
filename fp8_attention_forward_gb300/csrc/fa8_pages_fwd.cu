// fa8_pages_fwd.cu -- attention over listed pages of an FP8 paged cache (fa8_fwd_pages).
//
// Each (token, kv-head) has its own list of pages, so a tile has at most the G q-heads of one
// kv-head as rows and no two tiles share keys by construction: the work is a gather of K and V
// rows, bound by HBM (decode) or by L2 (many tokens of one request).
//
//   S^T (16 keys x 8 rows)  = K (M = keys, k = d) . Q^T        f16 MMAs on exactly widened E4M3
//   O^T (16 dv x 8 rows)   += V^T (M = dv, k = keys) . P^T
//
// A warp works alone: it takes every (warps x cluster)-th chunk of 16, 32 or 64 keys of the list, keeps
// its own running maximum, sum and O^T in registers, and has one K and one V buffer that TMA fills
// (boxes of one head's rows of a page, swizzled): the next K while this chunk goes through softmax and
// PV, the next V during PV and the next S^T.  V's 16 x 16 byte tiles are transposed as they are loaded.  P is
// rounded to f16 (2^-11 relative down to 2^-21 of the row's maximum, and by 2^-32 of it below), not to E4M3 as in
// fa8_fwd: V widens to f16 anyway.  The warps, then the CTAs of the cluster through distributed shared memory,
// merge by their maxima: no workspace, no second kernel.
//
// Measured from a graph's replays (d = dv = 128, 64 x 8 lists of 2048 keys, 267 MB): 47 to 51 us by the GPU, 5.2 to
// 5.7 TB/s, 0.77 to 0.84 of the copy rate; as called, inputs changing, 53 us.  Many tokens of one request (512 x 8
// lists of 2048 keys, 2.1 GB through L2): 158 us, 13.6 TB/s, with shared memory at 65 %, L2 at 55 %, the ALU pipe,
// which widens E4M3 to f16, at 52 % and issue slots at 51 %; in chunks of 32 keys 168 us, of which the copies and
// the softmax without the products take 122.  Tried: V's fragments by 16-byte
// loads whose bytes are paired by permutes, 52 and 210 us; both operands straight to registers, 63 and 303;
// by 16-byte asynchronous copies, 61 and 258 (L2 is asked for every sector twice); QK by the E4M3 warp MMA,
// 3 % slower (it widens too); a second K or V buffer, 3 to 5 % slower.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <string.h>

#include <algorithm>
#include <numeric>

#include "fa8.h"
#include "fa8_host.h"
#include "fa8_kernel.cuh"
#include "fa8_pages.cuh"

namespace fa8 {

struct PagesParams {
    const uint8_t *q, *k, *v;
    long long q_s[3];            // request, token, head
    long long k_s[3], v_s[3];    // page, row, head
    const int *list;
    long long l_s[3];            // request, token, head
    const int *cu_q;
    const float *dq, *dk, *dv;
    long long dq_s[2], dk_s[2], dv_s[2];
    const float *sink;
    float scale_log2;
    void *o;
    long long o_s[3];
    int out_fp16;
    float *lse;
    long long lse_s[3];          // request, token, head
    int T, B, Sq, Hkv, G, K, causal, num_pages, cluster, row_blocks;
    int box;                     // keys of one TMA box: gcd(page_size, keys per chunk)
    int box_shift;               // log2 of the boxes per chunk
    unsigned int box_magic;      // ceil(2^32 / (page_size / box)): box -> list entry
    unsigned long long timeout_ns;
    host::Table tab;
    unsigned int *status;
};

constexpr int kPgMaxCluster = 8;
// P is taken against 2^kPgBias below a row's maximum, and that maximum moves only for scores 2^kPgSlack above it:
// p <= 2^15 stays in f16's range, and p of 2^-31 of the maximum is still more than zero.  (Scores past 2^24, where
// an fp32 step is a factor of two or more, saturate.)
constexpr float kPgBias = 7.f, kPgSlack = 8.f;

// MANY: many tokens per request, whose lists L2 serves: longer chunks, fewer CTAs.
template <int D, int DV, int NT, int PW, bool MANY>
struct PgCfg {
    static constexpr int ROWS = 8 * NT;
    // 16-key tiles per chunk (d = dv = 64, 512 tokens x 8 lists of 2048 keys: 97 us with four, 124 with two;
    // d = dv = 96: 124 and 146)
    static constexpr int MT = (D + DV <= 192 && NT == 1) || MANY ? 4 : (D + DV <= 256 ? 2 : 1);
    static constexpr int KC_LOG = MT == 4 ? 6 : (MT == 2 ? 5 : 4);
    static constexpr int KC = 16 * MT;                // keys per chunk
    static constexpr int NG = 2 * MT;                 // 8-key groups per chunk
    // rows arrive as blocks of CW bytes, each block KC rows deep with the swizzle of its width (rows of
    // 96 bytes in one block without one: four of them cover all banks once)
    static constexpr int CW = D % 128 == 0 ? 128 : (D % 64 == 0 ? 64 : 96), NCK = D / CW;
    static constexpr int CWV = DV % 128 == 0 ? 128 : (DV % 64 == 0 ? 64 : 96), NCV = DV / CWV;
    static_assert(NCK * CW == D && NCV * CWV == DV, "head dims");
    static constexpr int VK = CW == 96 ? 8 : 16;      // bytes of one K fragment load
    static constexpr int NKV = D / (4 * VK);          // K fragment loads per key and lane
    static constexpr int STEPS = D / 16;
    // Q's fragments stay in registers while they take 16 (chunk of tokens, d = 128: 168 us against 171; with
    // 32, 16 rows of d = 128: 23.2 against 21.6)
    static constexpr bool HELD = NT * STEPS <= 8;
    static constexpr int DT = DV / 16;                // 16-row tiles of O^T
    static constexpr int OPITCH = DV + 4;             // floats per row of a merge buffer
    static constexpr int K_STAGE = KC * D, V_STAGE = KC * DV, STAGE = K_STAGE + V_STAGE;
    static constexpr int Q_BYTES = NT * STEPS * 32 * 8;
    static constexpr int MERGE_BYTES = PW * ROWS * (OPITCH + 2) * 4;
    static constexpr int OFF_Q = PW * STAGE, OFF_ENT = OFF_Q + Q_BYTES;
    static int smem(int K) { return 1024 + std::max(OFF_ENT + ((K * 8 + 15) & ~15), MERGE_BYTES); }
    // CTAs per SM that registers are cut to: four of four warps, but where 16 rows of wide heads would
    // spill (d = dv = 192, 60 lists of 960 keys x 8 heads: 37.6 us against 54.7 uncut; 16 rows, d = dv =
    // 128: 24.8 against 31.7; 16 rows, d = dv = 256: 52.9 cut against 32)
    static constexpr int CTAS = PW > 4 ? 1 : (NT == 2 && D + DV > 256 ? 2 : (MANY ? 3 : 4));
    // first of the VK channels that lane column c takes with fragment load v (rows of 128 bytes: the
    // pieces 2c and 2c + 1 of a block, so that two rows' lanes meet different banks)
    static __device__ __forceinline__ int k_dim(int v, int c) {
        return CW == 128 ? (v >> 1) * 128 + 16 * (2 * c + (v & 1)) : 4 * VK * v + VK * c;
    }
    // byte offset in a stage of byte x of a row of width-W blocks (TMA swizzle of W bytes)
    template <int W>
    static __device__ __forceinline__ int at(int row, int x) {
        const int piece = (x % W) >> 4, sw = W == 128 ? row & 7 : (W == 64 ? (row >> 1) & 3 : 0);
        return (x / W) * KC * W + row * W + 16 * (piece ^ sw) + (x & 15);
    }
};

template <int D, int DV, int NT, int PW, bool MANY>
__global__ void __launch_bounds__(32 * PW, PgCfg<D, DV, NT, PW, MANY>::CTAS) fwd_pages_kernel(
    const __grid_constant__ PagesParams p, const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v) {
    using C = PgCfg<D, DV, NT, PW, MANY>;
    constexpr int kThreads = 32 * PW;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    __shared__ __align__(8) uint64_t s_bar[PW][2];
    __shared__ int s_abort;
    __shared__ int s_used;
    __shared__ float s_m[C::ROWS], s_l[C::ROWS];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int r = lane >> 2, c = lane & 3;
    const int CS = p.cluster;
    const int rank = CS > 1 ? (int)cluster_rank() : 0;
    int row = blockIdx.x / CS;
    const int rb = row % p.row_blocks;
    row /= p.row_blocks;
    const int kvh = row % p.Hkv, tok = row / p.Hkv;
    const int ps = p.tab.page_size;
    int b, ti, Lq;
    if (!locate_token(p.cu_q, p.B, p.Sq, tok, &b, &ti, &Lq)) return;
    const long long bb = p.cu_q ? 0 : b, tt = p.cu_q ? tok : ti;
    // the chain to the first copy is list -> block table -> page: its first link goes out at once
    const int *list = p.list + bb * p.l_s[0] + tt * p.l_s[1] + kvh * p.l_s[2];
    const int lp0 = tid < p.K ? __ldg(list + tid) : -1;
    const float dqv = p.dq ? __ldg(p.dq + b * p.dq_s[0] + kvh * p.dq_s[1]) : 1.f;
    const float dkv = p.dk ? __ldg(p.dk + b * p.dk_s[0] + kvh * p.dk_s[1]) : 1.f;
    const int Lk = p.tab.cu_k[b + 1] - p.tab.cu_k[b];
    int vis = p.causal ? min(Lk, Lk - Lq + ti + 1) : Lk;
    if (Lk < 0 || (long long)Lk > (long long)p.tab.max_pages * ps) {
        if (tid == 0) atomicOr(p.status, kStatusBounds);
        vis = 0;
    }
    const int h0 = kvh * p.G + rb * C::ROWS;            // first q-head of the tile
    const int rows = min(C::ROWS, p.G - rb * C::ROWS);  // real rows

    // ---- the list: page and first key of every entry (page -1: nothing visible in it)
    uint2 *qf = reinterpret_cast<uint2 *>(smem + C::OFF_Q);
    int2 *ent = reinterpret_cast<int2 *>(smem + C::OFF_ENT);
    if (tid == 0) {
        s_used = 0;
        s_abort = 0;
        if (p.num_pages > 0) {
            ptx::prefetch_tmap(&tm_k);
            ptx::prefetch_tmap(&tm_v);
        }
    }
    const uint32_t bar_k = ptx::smem_u32(s_bar[warp]), bar_v = bar_k + 8;
    if (lane == 0) {
        ptx::mbar_init(bar_k, 1);
        ptx::mbar_init(bar_v, 1);
        ptx::fence_mbar_init();
        ptx::fence_proxy_async_smem();
    }
    __syncthreads();
    {
        const int *bt = p.tab.bt + (long long)b * p.tab.bt_stride;
        int used = 0;
        for (int e = tid; e < p.K; e += kThreads) {
            const int lp = e == tid ? lp0 : list[e];
            int page = -1, key0 = 0;
            if (lp >= p.tab.max_pages) {
                atomicOr(p.status, kStatusBounds);
            } else if (lp >= 0 && (long long)lp * ps < vis) {
                page = bt[lp];
                if (page < 0 || page >= p.num_pages) {
                    page = -1;
                    atomicOr(p.status, kStatusBounds);
                } else {
                    used = e + 1;
                    key0 = lp * ps;
                }
            }
            ent[e] = make_int2(page, key0);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) used = max(used, __shfl_xor_sync(0xffffffffu, used, o));
        if (lane == 0 && used) atomicMax(&s_used, used);
        const uint8_t *q = p.q + bb * p.q_s[0] + tt * p.q_s[1] + (long long)h0 * p.q_s[2];
        for (int x = tid; x < NT * C::STEPS * 32; x += kThreads) {
            const int ln = x & 31, st = (x >> 5) % C::STEPS, nt = x / (32 * C::STEPS);
            const int qr = nt * 8 + (ln >> 2);
            constexpr int SPV = C::VK / 4;  // k-steps fed by one fragment load
            const int pos = C::k_dim(st / SPV, ln & 3) + 4 * (st % SPV);
            uint32_t lo = 0, hi = 0;
            if (qr < rows) e4m3x4_to_h2(*reinterpret_cast<const uint32_t *>(q + qr * p.q_s[2] + pos), lo, hi);
            qf[x] = make_uint2(lo, hi);
        }
    }
    __syncthreads();
    const int bpp = ps / p.box;            // boxes per page
    const int boxes = s_used * bpp;        // boxes of the list
    float cs = p.scale_log2 * dqv * dkv;
    if (cs == 0.f) cs = 0x1p-126f;  // below fp32: a masked -inf must stay one

    // ---- the warp's chunk buffer, one of K and one of V: chunk it is boxes (first + it * stride) <<
    // box_shift ..; K is fetched while the chunk before goes through softmax and PV, V during PV and S^T
    const int first = warp * CS + rank, stride = CS * PW;
    const uint32_t ks = ptx::smem_u32(smem) + warp * C::STAGE, vs = ks + C::K_STAGE;
    // the row of V's 16 x 16 byte tiles that this lane addresses: a lane of the transpose receives keys 2c,
    // 2c + 1, 2c + 8 and 2c + 9, as P^T's fragments have them
    const int vrow = 2 * ((lane >> 2) & 3) + (lane & 1) + 8 * ((lane >> 1) & 1);
    const int nb = 1 << p.box_shift, mine = lane & (nb - 1), part = lane >> p.box_shift;
    // this lane's box of the chunk: page, first row, and how many of its keys are visible
    int page, prow, lim;
    bool full;  // every key of the chunk
    auto locate = [&](int it) {
        const int bx = ((first + it * stride) << p.box_shift) + mine;
        page = p.num_pages;  // out of range: TMA fills zeros
        prow = 0;
        lim = 0;
        if (bx < boxes) {
            const int e = bpp == 1 ? bx : (int)__umulhi((unsigned)bx, p.box_magic);
            const int2 en = ent[e];
            if (en.x >= 0) {
                prow = (bx - e * bpp) * p.box;
                lim = vis - en.y - prow;
                if (lim > 0) page = en.x;
            }
        }
        full = __all_sync(0xffffffffu, lim >= p.box);
    };
    // visible keys of 8-key group i (of all lanes)
    auto group_lim = [&](int i) {
        const int sh = C::KC_LOG - p.box_shift, b0 = i * 8 >> sh;  // a box is 2^sh keys
        return __shfl_sync(0xffffffffu, lim, b0) - (i * 8 - (b0 << sh));
    };
    auto fetch_k = [&]() {
        if (lane == 0) ptx::mbar_arrive_expect_tx(bar_k, (uint32_t)C::K_STAGE);
        __syncwarp();
        if (part < C::NCK)
            ptx::tma_load_4d(ks + part * C::KC * C::CW + mine * p.box * C::CW, &tm_k, bar_k, part * C::CW, kvh, prow, page);
    };
    auto fetch_v = [&]() {
        if (lane == 0) ptx::mbar_arrive_expect_tx(bar_v, (uint32_t)C::V_STAGE);
        __syncwarp();
        if (part < C::NCV)
            ptx::tma_load_4d(vs + part * C::KC * C::CWV + mine * p.box * C::CWV, &tm_v, bar_v, part * C::CWV, kvh, prow, page);
    };
    const int all = (boxes + nb - 1) >> p.box_shift;
    const int chunks = all > first ? (all - first + stride - 1) / stride : 0;
    const Waiter W{&s_abort, p.timeout_ns, p.status};
    if (chunks > 0) {
        locate(0);
        fetch_k();
        fetch_v();
    }

    // running maximum less kPgBias (log2 units) and this lane's share of the sum, rows 2c, 2c + 1
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
            for (int i = 0; i < C::NG; ++i) {
                kr[i] = ld_shared<C::VK>(ks + C::template at<C::CW>(8 * i + r, C::k_dim(j, c)));
            }
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
        // ---- softmax in log2 units of the scaled score: mask, running maximum per row (over the
        // lanes of equal c), and O^T rescaled only when some row's maximum moved
        if (!full) {
#pragma unroll
            for (int x = 0; x < C::MT; ++x)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const bool off = r >= group_lim(2 * x + h);
#pragma unroll
                    for (int t = 0; t < NT; ++t)
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            if (off) s[x][t][2 * h + e] = -INFINITY;
                }
        }
        const bool partial = !full;
        int vlim[(C::KC + 31) / 32];  // above 0 where row 32 i + lane is visible
#pragma unroll
        for (int i = 0; i < (C::KC + 31) / 32; ++i) vlim[i] = partial ? group_lim((lane >> 3) + 4 * i) - (lane & 7) : 1;
        const bool more = it + 1 < chunks;
        __syncwarp();  // every lane has read the K buffer
        if (more) {
            locate(it + 1);
            fetch_k();
        }
        uint32_t pb[C::MT][NT][2];
        // The maximum that P is taken against moves only when some score is 2^kPgSlack above it (sums are fp32
        // anyway): most chunks need no maximum over lanes and no rescaling.
        float mx[NT][2];
        bool moved = false;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float y = -INFINITY;
#pragma unroll
                for (int x = 0; x < C::MT; ++x) y = fmaxf(y, fmaxf(s[x][t][e], s[x][t][2 + e]));
                mx[t][e] = y * cs;
                moved |= mx[t][e] > m[t][e] + (kPgBias + kPgSlack);
            }
        if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float mn = mx[t][e];
#pragma unroll
                    for (int sh = 4; sh < 32; sh <<= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, sh));
                    mn = fmaxf(m[t][e], mn - kPgBias);
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
            const float r0 = m[t][0] == -INFINITY ? 0.f : -m[t][0], r1 = m[t][1] == -INFINITY ? 0.f : -m[t][1];
#pragma unroll
            for (int x = 0; x < C::MT; ++x)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float p0 = ptx::ex2(fmaf(s[x][t][2 * h], cs, r0)), p1 = ptx::ex2(fmaf(s[x][t][2 * h + 1], cs, r1));
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
        if (partial) {  // rows that are not visible may hold anything: they become zeros
#pragma unroll
            for (int i = 0; i < (C::KC + 31) / 32; ++i)
                if (lane + 32 * i < C::KC && vlim[i] <= 0)
#pragma unroll
                    for (int d = 0; d < DV; d += 16) st_shared_zero16(vs + C::template at<C::CWV>(lane + 32 * i, d));
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
    __syncthreads();  // the buffers, the list and Q are done with
    float *wo = reinterpret_cast<float *>(smem);                       // [warp][row][OPITCH]
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
                for (int h = 0; h < 2; ++h)
                    wo[(warp * C::ROWS + rw) * C::OPITCH + 16 * d + 8 * h + r] = o[d][t][2 * h + e];
        }
    __syncthreads();
    // warp buffers -> buffer of warp 0 (relative to the CTA's maximum), and the CTA's m and l
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
    const uint32_t a_m = ptx::smem_u32(s_m), a_l = ptx::smem_u32(s_l), a_o = ptx::smem_u32(wo);
    // the cluster's CTAs share the tile's output: pair x of columns belongs to rank x mod CS's stretch
    const int total = rows * (DV / 2), share = (total + CS - 1) / CS;
    for (int x = rank * share + tid; x < min(total, (rank + 1) * share); x += kThreads) {
        const int rw = x / (DV / 2), d = 2 * (x - rw * (DV / 2));
        float M, L, a0, a1;
        if (CS > 1) {
            float mr[kPgMaxCluster];
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
        const int hq = h0 + rw;
        float lse, f;
        if (M == -INFINITY && L == 0.f) {  // no visible key
            f = 0.f;
            lse = p.sink ? p.sink[hq] : -INFINITY;
        } else {
            const float ref = M == -INFINITY ? 0.f : M;
            float top = ref, sum = L, sc = 1.f;
            if (p.sink) {
                const float sl = p.sink[hq] * kLog2e;
                top = fmaxf(ref, sl);
                sc = ptx::ex2(ref - top);
                sum = L * sc + ptx::ex2(sl - top);
            }
            f = sc * dvv / sum;
            lse = (log2f(sum) + top) * kLn2;
        }
        uint8_t *dst = reinterpret_cast<uint8_t *>(p.o) + 2 * (bb * p.o_s[0] + tt * p.o_s[1] + (long long)hq * p.o_s[2] + d);
        if (p.out_fp16) *reinterpret_cast<__half2 *>(dst) = __floats2half2_rn(a0 * f, a1 * f);
        else *reinterpret_cast<__nv_bfloat162 *>(dst) = __floats2bfloat162_rn(a0 * f, a1 * f);
        if (d == 0 && p.lse) p.lse[bb * p.lse_s[0] + tt * p.lse_s[1] + (long long)hq * p.lse_s[2]] = lse;
    }
    if (CS > 1) cluster_sync();  // no CTA leaves while its shared memory is still read
}

template <int D, int DV, int NT, int PW, bool MANY = false>
fa8_status launch_pages(PagesParams &p, const fa8_tensor *k, const fa8_tensor *v, unsigned int tiles, int dev, cudaStream_t s) {
    static host::SmemOptIn opt_in;
    using C = PgCfg<D, DV, NT, PW, MANY>;
    const int ps = p.tab.page_size;
    p.box = std::gcd(ps, C::KC);
    p.box_shift = 0;
    while (p.box << p.box_shift < C::KC) ++p.box_shift;
    p.box_magic = ps > p.box ? (unsigned)((0x100000000ull + ps / p.box - 1) / (ps / p.box)) : 0u;
    CUtensorMap tk, tv;
    memset(&tk, 0, sizeof(tk));
    memset(&tv, 0, sizeof(tv));
    if (p.num_pages > 0) {
        fa8_status st;
        if ((st = host::encode_kv(&tk, k, C::CW, p.box)) || (st = host::encode_kv(&tv, v, C::CWV, p.box))) return st;
    }
    const int smem = C::smem(p.K);
    cudaError_t e = opt_in(fwd_pages_kernel<D, DV, NT, PW, MANY>, smem, dev);
    if (e != cudaSuccess) return host::cuda_fail(e, "page attention shared memory");
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(tiles * p.cluster);
    cfg.blockDim = dim3(32 * PW);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = p.cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, fwd_pages_kernel<D, DV, NT, PW, MANY>, p, tk, tv);
    return e == cudaSuccess ? FA8_SUCCESS : host::cuda_fail(e, "page attention kernel launch");
}

}  // namespace fa8

using namespace fa8::host;

extern "C" fa8_status fa8_fwd_pages(const fa8_tensor *q, const fa8_tensor *k, const fa8_tensor *v, const fa8_tensor *pages,
                                    const fa8_tensor *descale_q, const fa8_tensor *descale_k, const fa8_tensor *descale_v,
                                    fa8_tensor *out, fa8_tensor *lse, const fa8_tensor *cu_seqlens_q,
                                    const fa8_tensor *cu_seqlens_k, const fa8_tensor *block_table, int page_size, int causal,
                                    const fa8_tensor *sink, float softmax_scale, void *stream) {
    clear_error();
    if (!q || !k || !v || !pages || !out) return fail(FA8_ERR_INVALID_ARG, "q, k, v, pages and out are required");
    for (const fa8_tensor *t : {q, k, v})
        if (t->dtype != FA8_DTYPE_E4M3) return fail(FA8_ERR_UNSUPPORTED, "q/k/v must be E4M3");
    fa8::PagesParams p;
    memset(&p, 0, sizeof(p));
    fa8_status st;
    if ((st = check_payload(q, "q")) || (st = check_payload(k, "k")) || (st = check_payload(v, "v"))) return st;
    Queries qs;
    if ((st = check_queries(q, cu_seqlens_q, &qs))) return st;
    if (k->ndim != 4 || v->ndim != 4) return fail(FA8_ERR_INVALID_ARG, "k and v must be paged (num_pages, page_size, Hkv, d)");
    for (int i = 0; i < 3; ++i)
        if (k->shape[i] != v->shape[i]) return fail(FA8_ERR_INVALID_ARG, "k and v leading shapes differ at dim %d", i);
    if (k->shape[3] != qs.D) return fail(FA8_ERR_INVALID_ARG, "k head dim %lld != q head dim %d", (long long)k->shape[3], qs.D);
    if (v->shape[3] > 1024 || !supported_dims(qs.D, (int)v->shape[3]))
        return fail(FA8_ERR_UNSUPPORTED, "(d, dv) = (%d, %lld) is not supported", qs.D, (long long)v->shape[3]);
    const int DV = (int)v->shape[3];
    const long long Hkv = k->shape[2];
    if ((st = check_groups(qs.Hq, Hkv, &p.G))) return st;
    if ((st = check_table(cu_seqlens_k, block_table, page_size, qs.B, &p.tab))) return st;
    if (page_size != k->shape[1]) return fail(FA8_ERR_INVALID_ARG, "page_size (%d) != k.shape[1] (%lld)", page_size, (long long)k->shape[1]);
    if (page_size > 4096) return fail(FA8_ERR_UNSUPPORTED, "page_size %d is above 4096", page_size);
    if (k->shape[0] > 0x7fffffffLL) return fail(FA8_ERR_UNSUPPORTED, "too many pages");
    if (k->shape[0] > 0 && (!k->data || !v->data)) return fail(FA8_ERR_INVALID_ARG, "k and v need data");
    if ((st = check_page_lists(pages, qs, (int)Hkv, p.l_s, &p.K))) return st;
    // ---- outputs
    const int nd = q->ndim;
    if (out->dtype != FA8_DTYPE_BF16 && out->dtype != FA8_DTYPE_F16) return fail(FA8_ERR_INVALID_ARG, "out must be bf16 or fp16");
    if (out->ndim != nd) return fail(FA8_ERR_INVALID_ARG, "out must have q's rank");
    for (int i = 0; i < nd - 1; ++i) {
        if (out->shape[i] != q->shape[i]) return fail(FA8_ERR_INVALID_ARG, "out shape differs from q at dim %d", i);
        if (out->stride[i] % 8 != 0) return fail(FA8_ERR_INVALID_ARG, "out strides must be multiples of 8 elements");
    }
    if (out->shape[nd - 1] != DV) return fail(FA8_ERR_INVALID_ARG, "out last dim must be dv=%d", DV);
    if (out->stride[nd - 1] != 1) return fail(FA8_ERR_INVALID_ARG, "out: last dim must be contiguous");
    if (!aligned16(out->data)) return fail(FA8_ERR_INVALID_ARG, "out must be 16-byte aligned");
    if ((st = check_written(out, "out"))) return st;
    if (lse) {
        if (lse->dtype != FA8_DTYPE_F32) return fail(FA8_ERR_INVALID_ARG, "lse must be fp32");
        if (qs.cu_q) {
            if (lse->ndim != 2 || lse->shape[0] != qs.Hq || lse->shape[1] != qs.T)
                return fail(FA8_ERR_INVALID_ARG, "varlen lse must be (Hq, total_q)");
            p.lse_s[1] = lse->stride[1];
            p.lse_s[2] = lse->stride[0];
        } else {
            if (lse->ndim != 3 || lse->shape[0] != qs.B || lse->shape[1] != qs.Hq || lse->shape[2] != qs.Sq)
                return fail(FA8_ERR_INVALID_ARG, "lse must be (B, Hq, Sq)");
            p.lse_s[0] = lse->stride[0];
            p.lse_s[1] = lse->stride[2];
            p.lse_s[2] = lse->stride[1];
        }
    }
    if (lse && (st = check_written(lse, "lse"))) return st;
    if ((st = check_descale(descale_q, "descale_q", qs.B, (int)Hkv, &p.dq, &p.dq_s[0], &p.dq_s[1])) ||
        (st = check_descale(descale_k, "descale_k", qs.B, (int)Hkv, &p.dk, &p.dk_s[0], &p.dk_s[1])) ||
        (st = check_descale(descale_v, "descale_v", qs.B, (int)Hkv, &p.dv, &p.dv_s[0], &p.dv_s[1])))
        return st;
    if (sink) {
        if (sink->dtype != FA8_DTYPE_F32 || sink->ndim != 1 || sink->shape[0] != qs.Hq || (qs.Hq > 1 && sink->stride[0] != 1) || !sink->data)
            return fail(FA8_ERR_INVALID_ARG, "sink must be a contiguous fp32 (Hq,) tensor");
        p.sink = static_cast<const float *>(sink->data);
    }
    if (causal != 0 && causal != 1) return fail(FA8_ERR_INVALID_ARG, "causal must be 0 or 1");
    if (!std::isfinite(softmax_scale)) return fail(FA8_ERR_INVALID_ARG, "softmax_scale must be finite");
    if (softmax_scale <= 0.f) softmax_scale = 1.0f / std::sqrt((float)qs.D);
    const int nt = p.G <= 8 ? 1 : 2;
    p.row_blocks = (p.G + 8 * nt - 1) / (8 * nt);
    const long long tiles = (long long)qs.T * Hkv * p.row_blocks;
    if (tiles * fa8::kPgMaxCluster > 0x7fffffffLL) return fail(FA8_ERR_UNSUPPORTED, "problem too large for the grid");
    if (tiles == 0) return FA8_SUCCESS;
    if (!q->data || !out->data || (lse && !lse->data) || (p.K > 0 && !pages->data))
        return fail(FA8_ERR_INVALID_ARG, "q, pages, out and lse need data");
    DeviceState *ds = nullptr;
    if ((st = device_state(&ds))) return st;
    p.q = static_cast<const uint8_t *>(q->data);
    p.k = static_cast<const uint8_t *>(k->data);
    p.v = static_cast<const uint8_t *>(v->data);
    for (int i = 0; i < 3; ++i) {
        p.q_s[i] = qs.stride[i];
        p.k_s[i] = k->stride[i];
        p.v_s[i] = v->stride[i];
        p.o_s[i] = nd == 4 ? out->stride[i] : (i ? out->stride[i - 1] : 0);
    }
    p.list = static_cast<const int *>(pages->data);
    p.cu_q = qs.cu_q;
    p.scale_log2 = softmax_scale * 1.4426950408889634f;
    p.o = out->data;
    p.out_fp16 = out->dtype == FA8_DTYPE_F16;
    p.lse = lse ? static_cast<float *>(lse->data) : nullptr;
    p.T = qs.T;
    p.B = qs.B;
    p.Sq = qs.Sq;
    p.Hkv = (int)Hkv;
    p.causal = causal;
    p.num_pages = (int)k->shape[0];
    p.status = ds->status;
    p.timeout_ns = wait_timeout_ns();
    // Clusters split a list over CTAs while all of them run at once and every warp keeps at least two
    // chunks (one of 64 keys); where clusters of eight still leave a quarter of the SMs empty, CTAs of eight
    // warps, one per SM, split it once more (8 lists of 4096 keys, d = dv = 256: 12.0 us against 15.5 with four
    // warps; 14 lists 13.0 against 16.9; 16 lists, whose clusters no longer fit at once, 23.8 against 17.9).
    const long long keys = (long long)p.K * page_size;
    const int kc = qs.D + DV <= 256 ? 32 : 16, per_sm = nt == 2 && qs.D + DV > 256 ? 2 : 4;
    p.cluster = 1;
    while (p.cluster < fa8::kPgMaxCluster && tiles * p.cluster * 2 <= (long long)per_sm * ds->sm_count && keys >= 2LL * kc * 4 * p.cluster * 2)
        p.cluster *= 2;
    const bool wide = p.cluster == fa8::kPgMaxCluster && tiles * p.cluster * 4 <= 3LL * ds->sm_count && keys >= 2LL * kc * 8 * p.cluster;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
#define FA8_PAGES(D_, DV_)                                                                               \
    case D_ * 1000 + DV_:                                                                                \
        return nt == 1 ? (wide ? fa8::launch_pages<D_, DV_, 1, 8>(p, k, v, (unsigned)tiles, ds->ordinal, s)           \
                               : fa8::launch_pages<D_, DV_, 1, 4>(p, k, v, (unsigned)tiles, ds->ordinal, s))          \
                       : (wide ? fa8::launch_pages<D_, DV_, 2, 8>(p, k, v, (unsigned)tiles, ds->ordinal, s)           \
                               : fa8::launch_pages<D_, DV_, 2, 4>(p, k, v, (unsigned)tiles, ds->ordinal, s));
    // Chunks of 64 keys for d = dv = 128 where L2 serves the lists of many tokens of a request (512 tokens x 8
    // lists of 2048 keys: 157 us against 168), not where HBM does (64 x 8 lists of one token each: 61
    // against 51: fewer copies in flight).
    if (qs.D == 128 && DV == 128 && nt == 1 && p.cluster == 1 && (long long)qs.T >= 16LL * qs.B)
        return fa8::launch_pages<128, 128, 1, 4, true>(p, k, v, (unsigned)tiles, ds->ordinal, s);
    switch (qs.D * 1000 + DV) {
        FA8_PAGES(64, 64)
        FA8_PAGES(96, 96)
        FA8_PAGES(128, 128)
        FA8_PAGES(192, 128)
        FA8_PAGES(192, 192)
        FA8_PAGES(256, 256)
    }
#undef FA8_PAGES
    return fail(FA8_ERR_UNSUPPORTED, "no page attention kernel for (%d, %d)", qs.D, DV);
}
