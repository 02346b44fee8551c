// fa8_scored_many.cuh -- attention with capped, biased or masked scores for many query rows per kv-head
// (prompts, chunks of them, trees of drafted tokens).
//
//   S = Q K^T (E4M3 MMAs);  z = score(S);  P = 2^(z - m) in f16;  O += P V (f16 MMAs, V widened exactly)
//
// One CTA per SM walks a list of units of 128 rows (positions x q-heads of a kv-head), in tiles of 64 keys, the last keys
// first (where distances weigh, those with the largest scores: the maximum then moves once).  What bounds a tile is
// the chain S -> maximum -> P -> O -> next S, thousands of cycles long, not a pipe: so the tiles go round four
// warpgroups of softmax, between which a row's running maximum passes in a word of shared memory, and S has four to six
// buffers in TMEM; P takes the place of its S.  O stays in TMEM over a whole unit and is scaled only when a row's
// maximum has moved by more than 2^kScSlack, so that no fold is paid per tile; P in f16 (2^-11 relative) needs no second
// term as one of E4M3 does, at the price of V widened to f16 in shared memory.
//
// Everything that runs per tile is kept in small rolled loops (16 columns of a tile at a time), the units are worked
// out by one warp and reach the others through shared memory, and one lane issues pairs of tiles: the 28 warps run eight
// different programs, and an SM's instruction caches are what they share (weights of 32 columns unrolled: capped prompt
// 372 us, of 16 302).
//
// Measured (us; two causal prompts of 4096, 32 q-heads on 8, d = 128, 275 GFLOP): no change of scores 207 (1330 TFLOP/s;
// fa8_fwd 298), capped 293, sloped 225, both 284; d = 64 185, sloped 193; 16 on 4, d = 192 / 128 127, 256 194.  At 207 the
// tensor pipe is busy 41 % of the time, the issue slots 64 %, the exponentials' unit 28 %; capped, that unit 45 %.
//
// Warpgroups (896 threads):
//   0-3   softmax, thread = row: tiles 0, 1, 2, 3 (mod 4)
//   4     output, thread = row: a unit's O from TMEM, scaled and stored, while the softmax is at the next unit
//   5     widen V: E4M3 rows from the TMA ring -> f16 in the MN-major swizzled layout of the MMA
//   6     control: a warp each for the units and TMA of Q (it owns the TMEM, too), the MMAs of S, those of O, TMA
//         of K and V (a warp each for these: 64 requests with pages of 16 256 -> 239 us, the prompts 2 .. 8 % longer)
// TMEM (512 columns): the buffers of S from 0 on, 64 columns each, then O.
#pragma once

#include "fa8_host.h"
#include "fa8_scored.cuh"

namespace fa8 {

// P is taken against 2^kScBias below the row's maximum, which moves only for scores 2^kScSlack above it: p <= 2^15
// stays in f16's range (scores past 2^24 saturate), and a weight down to 2^-28 of the largest still counts in P V, every
// one in the sum.  A slack of 8 kept three more bits there, but with scores of ten and more around zero O was scaled often
// (capped prompt with descales up to 6: 452 us, with 12 370).
constexpr float kScBias = 3.f, kScSlack = 12.f;

constexpr int kScTile = 64;  // keys of a tile; K is loaded, and S made, for two at a time
constexpr int kScUnits = 3;  // units between the warp that works them out and the ones that are done with them

constexpr int kScGroups = 4;             // warpgroups of softmax
constexpr int kScOut = 4 * kScGroups, kScConv = kScOut + 4, kScCtl = kScConv + 4, kScThreads = 32 * (kScCtl + 4);  // first warps
// registers per thread: at launch, then of the softmax, output, widening and control warpgroups (d = 256
// spills 8 to 12 bytes, 192 with slopes 8, the others nothing)
constexpr int kScRegs = 72, kScRegsS = 72, kScRegsO = 96, kScRegsV = 56, kScRegsC = 64;
static_assert(kScGroups * kScRegsS + kScRegsO + kScRegsV + kScRegsC <= (kScGroups + 3) * kScRegs && kScThreads * kScRegs <= 65536, "registers");
static_assert(kScRegsS == kScRegs && kScRegsO >= kScRegs && kScRegsV <= kScRegs && kScRegsC <= kScRegs, "taken or given");

template <int D, int DV>
struct ScCfg {
    static constexpr int NSB = DV <= 128 ? 6 : 4;     // buffers of S
    static constexpr uint32_t TM_O = NSB * kScTile;
    static_assert(TM_O + DV <= 512, "TMEM");
    static constexpr int CW = (D % 128 == 0) ? 128 : ((D % 64 == 0) ? 64 : 32);
    static constexpr int NCK = D / CW;
    static constexpr int CHUNK_Q = 128 * CW, CHUNK_K = 2 * kScTile * CW;
    static constexpr int CF = (DV % 64 == 0) ? 128 : 64;  // bytes of a row's chunk of f16 V
    static constexpr int NCF = DV * 2 / CF;
    static constexpr int CHUNK_F = kScTile * CF;
    // K and V share the stages of a ring while shared memory takes both for two tiles, else V comes a tile at a time.  The
    // widening warps take four tiles at a time, or pairs of them two: a stage is always widened by the same
    // warps, so that its barriers are at most one phase behind what they wait for.
    static constexpr bool ONE = DV <= 128;
    static constexpr int Q_BYTES = 128 * D, K_BYTES = 2 * kScTile * D, V_TILE = kScTile * DV, V_BYTES = ONE ? 2 * V_TILE : V_TILE,
                         VF_BYTES = kScTile * DV * 2;
    static constexpr int WIDE = ONE ? 4 : 2, STF = DV == 256 ? 2 : 4;  // stages of V in f16
    static constexpr int MISC_BYTES = 14336, LIMIT = 232448 - 1024;
    static constexpr int FIT = (LIMIT - MISC_BYTES - Q_BYTES - STF * VF_BYTES) / (K_BYTES + V_BYTES);
    static constexpr int ST = ONE && FIT >= 4 ? 4 : 2, STV = ST;       // stages of K and of V
    static_assert(STF % WIDE == 0, "phases");
    static constexpr int OFF_Q = 0, OFF_K = Q_BYTES, OFF_V = OFF_K + ST * K_BYTES, OFF_F = OFF_V + STV * V_BYTES;
    static constexpr int OFF_MISC = OFF_F + STF * VF_BYTES;
    static constexpr int SMEM_BYTES = OFF_MISC + MISC_BYTES + 1024;
    static_assert(SMEM_BYTES <= 232448, "shared memory");
    static_assert(Q_BYTES % 1024 == 0 && K_BYTES % 1024 == 0 && V_TILE % 1024 == 0 && VF_BYTES % 1024 == 0, "swizzle alignment");
    // barriers
    static constexpr int B_QF = 0, B_QE = 1, B_KF = 2, B_KE = B_KF + ST, B_VF = B_KE + ST, B_VE = B_VF + STV, B_FF = B_VE + STV,
                         B_SF = B_FF + STF, B_PF = B_SF + NSB / 2, B_OD = B_PF + NSB,  // S of two tiles, P, O of a tile done
                         B_LD = B_OD + NSB,           // a unit's sums are out [parity], have been read [parity]
                         B_LE = B_LD + 2,
                         B_EO = B_LE + 2,             // a unit's O has been read
                         B_DONE = B_EO + 1,
                         B_CL = B_DONE + 2,           // another CTA's unit
                         B_UF = B_CL + 1, B_UE = B_UF + kScUnits, NUM_BARS = B_UE + kScUnits;
    static constexpr int OFF_M = 512;                 // (tiles done, running maximum) [128]
    static constexpr int OFF_L = OFF_M + 1024;        // (maximum, sum) [unit parity][group][128]
    static constexpr int OFF_UNIT = OFF_L + 2048 * kScGroups;  // [kScUnits]: the unit, what its positions see [128] (lo, hi)
    static constexpr int OFF_ROWS = OFF_UNIT + 64 * kScUnits;
    static constexpr int OFF_NAN = OFF_ROWS + 1024 * kScUnits;  // [kScUnits][widening warp]: tiles with NaNs, modulo 64
    static constexpr int OFF_CL = OFF_NAN + 32 * kScUnits, OFF_SLOT = OFF_CL + 16, OFF_ABORT = OFF_SLOT + 4;
    static_assert(OFF_UNIT % 16 == 0 && OFF_CL % 16 == 0 && NUM_BARS * 8 <= OFF_M && OFF_ABORT + 4 <= MISC_BYTES, "misc area");
};

// ---------------------------------------------------------------- units
struct __align__(16) ScUnit {
    int b, kvh, pos0;   // first position
    int slot;           // of the workspace, -1: the unit is whole
    ScReq rq;
    int t0, t1;         // tiles of kScTile keys
    int end;            // no unit: the list is done
    float scale;        // of its scores, to log2 units
    int flo, fhi, slo, shi;  // keys that every row sees, that some row sees
};
static_assert(sizeof(ScUnit) == 64, "units are passed as four 16-byte words");
// Request and block of positions of slot x of packed sequences, their last blocks first.  Whole warp.
__device__ __forceinline__ bool sc_slot(const int *cu_q, int B, int P, int x, int *b, int *mb) {
    const int lane = threadIdx.x & 31;
    int base = 0;
    for (int s0 = 0; s0 < B; s0 += 32) {
        const int s = s0 + lane;
        int cnt = 0;
        if (s < B) {
            const int len = cu_q[s + 1] - cu_q[s];
            cnt = len > 0 ? (len - 1) / P + 1 : 0;
        }
        int inc = cnt;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += y;
        }
        const unsigned m = __ballot_sync(0xffffffffu, s < B && x < base + inc);
        if (m) {
            const int l = __ffs(m) - 1;
            const int ci = __shfl_sync(0xffffffffu, base + inc, l), cn = __shfl_sync(0xffffffffu, cnt, l);
            *b = s0 + l;
            *mb = cn - 1 - (x - (ci - cn));
            return true;
        }
        base += __shfl_sync(0xffffffffu, inc, 31);
    }
    return false;
}

// Split: every unit of a request counts all the request's visible tiles (the last token's; at least one), of which a
// share goes through those that its positions see, after sc_unit_cost that stand for what a unit costs besides (Q, the first
// scores, O: two requests of 247 and 5250 keys, 155 tokens, without them: 74 us, those with the short one's units last).
// One request's units are all alike: no cost, and cuts that fall on whole tiles of eight.
__device__ __forceinline__ int sc_unit_cost(const ScoredParams &p) { return p.B > 1 ? 6 : 0; }
__device__ __forceinline__ void sc_tiles(const ScoredParams &p, int Lk, int *first, int *n) {
    const int beg = p.window_left >= 0 ? max(0, Lk - p.Sq - p.window_left) : 0;
    *first = min(beg, max(0, Lk - 1)) / kScTile;
    *n = max(1, (Lk + kScTile - 1) / kScTile - *first) + sc_unit_cost(p);
}
// Where the list of all units' tiles is cut: share `per` of each CTA, and the request that holds position x
// with the position where it begins.  Whole warp.
struct ScCut {
    int total, per;
};
__device__ __forceinline__ int sc_scan(const ScoredParams &p, int nu, int x, int *base) {
    const int lane = threadIdx.x & 31;
    int sum = 0;
    for (int s0 = 0; s0 < p.B; s0 += 32) {
        const int s = s0 + lane;
        int cnt = 0;
        if (s < p.B) {
            ScReq rq;
            int f;
            sc_lengths(p, s, &rq);
            sc_tiles(p, rq.Lk, &f, &cnt);
            cnt *= nu;
        }
        int inc = cnt;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += y;
        }
        const unsigned m = __ballot_sync(0xffffffffu, s < p.B && x >= 0 && x < sum + inc);
        if (m) {
            const int l = __ffs(m) - 1;
            *base = sum + __shfl_sync(0xffffffffu, inc - cnt, l);
            return s0 + l;
        }
        sum += __shfl_sync(0xffffffffu, inc, 31);
    }
    *base = sum;  // past the end: all of it
    return p.B;
}
__device__ __forceinline__ ScCut sc_cut(const ScoredParams &p, int nu, int ctas) {
    ScCut c;
    sc_scan(p, nu, -1, &c.total);
    // a share has at least min_tiles, but where units are shorter than that no more than they have on average: a unit
    // that is not cut needs no joining
    const int units = nu * p.B;
    c.per = max(min(p.min_tiles, (c.total + units - 1) / units), (c.total + ctas - 1) / ctas);
    return c;
}

// Where the cuts are noted, behind the parts.
template <int DV>
__device__ __forceinline__ int4 *sc_cuts(const ScoredParams &p, int ctas) {
    return reinterpret_cast<int4 *>(p.part + (long long)ctas * 2 * 128 * (DV + 2));
}

struct ScIter {
    int k;                  // whole units: how many have been taken
    int pos, end, b, base;  // split
    int rank;               // whole units of up to 32 requests, fewer new tokens than their keys differ by: request `lane`'s place
                            // among them, the longest first; else -1
    // cuts: for the joining kernel, (request, unit of it, CTA of its last tile) of the unit that begins before this CTA's share
    // in the share just before; request -1 where there is none.
    __device__ __forceinline__ void init(const ScoredParams &p, int4 *cuts) {
        k = 0;
        if (!p.split) {
            rank = -1;
            if (p.cu_q || p.kv_mode == 0 || p.B > 32) return;
            const int lane = threadIdx.x & 31;
            ScReq rq;
            rq.Lk = 0;
            if (lane < p.B) sc_lengths(p, lane, &rq);
            const int keys = lane < p.B ? rq.Lk : -1;
            const int most = __reduce_max_sync(0xffffffffu, keys), least = __reduce_min_sync(0xffffffffu, lane < p.B ? keys : 0x7fffffff);
            if (most - least <= p.Sq) return;
            rank = 0;
            for (int x = 0; x < p.B; ++x) {
                const int y = __shfl_sync(0xffffffffu, keys, x);
                if (y > keys || (y == keys && x < lane)) ++rank;
            }
            return;
        }
        const int nu = p.blocks * p.Hkv;
        const ScCut c = sc_cut(p, nu, gridDim.x);
        pos = min(c.total, (int)blockIdx.x * c.per);
        end = min(c.total, pos + c.per);
        int4 cut = make_int4(-1, 0, 0, 0);
        if (pos < end) {
            b = sc_scan(p, nu, pos, &base);
            ScReq rq;
            int first, n;
            sc_lengths(p, b, &rq);
            sc_tiles(p, rq.Lk, &first, &n);
            const int y = (pos - base) / n, t = pos - base - y * n, start = pos - t;
            if (t > 0 && start / c.per + 1 == (int)blockIdx.x) cut = make_int4(b, y, (start + n - 1) / c.per, 0);
        }
        if ((threadIdx.x & 31) == 0) cuts[blockIdx.x] = cut;
    }
    // The next unit of this CTA.  Whole units are either one per CTA of the grid, and the first ones that run take the others'
    // over (steal), or there are many units less CTAs, and these take them in turn, back and forth.  Whole warp.
    // Keys that some position of the unit sees lie in [lo, hi).
    __device__ __forceinline__ void seen(const ScoredParams &p, int npos, const ScUnit *u, int &lo, int &hi) {
        const int last = min(u->pos0 + npos, u->rq.Lq) - 1;
        if (p.ranges) {
            lo = 0x7fffffff, hi = 0;
            for (int i = u->pos0 + (threadIdx.x & 31); i <= last; i += 32) {
                const ScRow r = sc_row(p, u->b, u->rq, i);
                if (r.hi > r.lo) {
                    lo = min(lo, r.lo);
                    hi = max(hi, r.hi);
                }
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                lo = min(lo, __shfl_xor_sync(0xffffffffu, lo, o));
                hi = max(hi, __shfl_xor_sync(0xffffffffu, hi, o));
            }
        } else {
            lo = p.window_left >= 0 ? max(0, u->pos0 + u->rq.Lk - u->rq.Lq - p.window_left) : 0;
            hi = sc_row(p, u->b, u->rq, last).hi;
        }
    }
    template <typename F>
    __device__ __forceinline__ bool next(const ScoredParams &p, int npos, ScUnit *u, const F &steal) {
        if (p.split) {
            if (pos >= end) return false;
            const int nu = p.blocks * p.Hkv;
            sc_request(p, b, &u->rq);
            int first, n;
            sc_tiles(p, u->rq.Lk, &first, &n);
            const int at = pos - base, y = at / n, t = at - y * n;
            const int take = min(n - t, end - pos);
            u->b = b;
            u->kvh = y % p.Hkv;
            u->pos0 = (y / p.Hkv) * npos;
            u->t0 = first + max(0, t - sc_unit_cost(p));
            u->t1 = first + max(0, t + take - sc_unit_cost(p));
            u->slot = take == n ? -1 : 2 * (int)blockIdx.x + (t == 0 ? 1 : 0);
            int lo, hi;
            seen(p, npos, u, lo, hi);
            u->t0 = max(u->t0, lo / kScTile);
            u->t1 = hi > lo ? min(u->t1, (hi - 1) / kScTile + 1) : 0;
            if (u->t1 <= u->t0) u->t0 = u->t1 = 0;
            pos += take;
            if (pos - base == nu * n) {
                base = pos;
                ++b;
            }
            return true;
        }
        while (true) {
            int x = (int)blockIdx.x;
            if (p.steal) {
                if (k > 0 && !steal(&x)) return false;
            } else {
                const int g = (int)gridDim.x;
                if ((long long)k * g >= p.units) return false;
                x = k * g + (k & 1 ? g - 1 - x : x);
            }
            ++k;
            if (x >= p.units) continue;
            const int slot = x / p.Hkv;
            int mb;
            u->kvh = x - slot * p.Hkv;
            if (!p.cu_q) {
                // the heaviest first: the last blocks, or the longest requests (four chunks, 256 units: 135 us, in the requests'
                // own order 135 to 167, as it falls)
                const unsigned at = __ballot_sync(0xffffffffu, rank == slot / p.blocks);
                u->b = at ? __ffs(at) - 1 : slot % p.B;
                mb = p.blocks - 1 - (at ? slot % p.blocks : slot / p.B);
            } else if (!sc_slot(p.cu_q, p.B, npos, slot, &u->b, &mb)) {
                continue;
            }
            if (!sc_request(p, u->b, &u->rq)) continue;
            u->pos0 = mb * npos;
            u->slot = -1;
            int lo, hi;
            seen(p, npos, u, lo, hi);
            u->t0 = hi > lo ? lo / kScTile : 0;
            u->t1 = hi > lo ? (hi - 1) / kScTile + 1 : 0;
            return true;
        }
    }
};

// ---------------------------------------------------------------- softmax pieces
__device__ __forceinline__ uint64_t sc_pair(const uint32_t *u) { return ptx::f2pack(u2f(u[0]), u2f(u[1])); }
__device__ __forceinline__ void sc_split(uint64_t y, uint32_t *u) {
    float a, b;
    ptx::f2unpack(y, a, b);
    u[0] = __float_as_uint(a);
    u[1] = __float_as_uint(b);
}
// 1 / (1 + e^(2 x)) of four scores, x = s k / cap as in sc_cap_near: tanh x = 1 - 2 / (1 + e^(2 x)) to 2^-22 absolutely.  They
// share one reciprocal, which e^(2 x) of at most 2^30 keeps in range (CUT: larger ones are cut there); a NaN
// reaches all four.
template <bool CUT>
__device__ __forceinline__ void sc_inv4(const uint32_t *u, float k2, uint64_t &ia, uint64_t &ib) {
    const uint64_t one = ptx::f2pack(1.f, 1.f), kk = ptx::f2pack(k2, k2);
    float x[4];
    ptx::f2unpack(ptx::fmul2(sc_pair(u), kk), x[0], x[1]);
    ptx::f2unpack(ptx::fmul2(sc_pair(u + 2), kk), x[2], x[3]);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if (CUT) asm("min.NaN.f32 %0, %0, %1;" : "+f"(x[e]) : "f"(30.f));
        x[e] = ptx::ex2(x[e]);
    }
    const uint64_t da = ptx::fadd2(one, ptx::f2pack(x[0], x[1])), db = ptx::fadd2(one, ptx::f2pack(x[2], x[3]));
    float pa, pb;
    ptx::f2unpack(ptx::fmul2(da, db), pa, pb);  // d0 d2, d1 d3
    const float r = rcp(pa * pb);
    const uint64_t rr = ptx::f2pack(r * pb, r * pa);
    ia = ptx::fmul2(db, rr);
    ib = ptx::fmul2(da, rr);
}
// The largest; NaN if there is one.
__device__ __forceinline__ float sc_max3(float a, float b, float c) {
    float y;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}
__device__ __forceinline__ float sc_max16(float m, const uint32_t (&u)[16]) {
    float m1 = -INFINITY;
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
        m = sc_max3(m, u2f(u[i]), u2f(u[i + 1]));
        m1 = sc_max3(m1, u2f(u[i + 2]), u2f(u[i + 3]));
    }
    return sc_max3(m, m1, m1);
}
// How a tile's scores become weights 2^z: z = u c + ref; with the cap; u + ref of scores changed in place; and
// the first two with a bias that grows by `slope` per key.
enum { kScNoCap, kScNearCap, kScFarCap };  // of the kernels: up to kFarCap, above
enum { kScPlain, kScCap, kScDone, kScBiased, kScCapBiased };
// P of 16 keys: 8 columns of f16 pairs, the unrounded weights into two sums.  r: what every two keys add; bias2:
// its growth over four.
template <int HOW>
__device__ __forceinline__ void sc_p16(const uint32_t (&u)[16], uint64_t c2, uint64_t ra, uint64_t rb, uint64_t bias2, float k2, uint64_t &acc0,
                                       uint64_t &acc1, uint32_t (&w)[8]) {
#pragma unroll
    for (int e = 0; e < 16; e += 4) {
        uint64_t ya, yb;
        if constexpr (HOW == kScCap || HOW == kScCapBiased) {
            uint64_t ia, ib;
            sc_inv4<false>(u + e, k2, ia, ib);
            ya = ptx::ffma2(ia, c2, ra);
            yb = ptx::ffma2(ib, c2, rb);
        } else if constexpr (HOW == kScDone) {
            ya = ptx::fadd2(sc_pair(u + e), ra);
            yb = ptx::fadd2(sc_pair(u + e + 2), rb);
        } else {
            ya = ptx::ffma2(sc_pair(u + e), c2, ra);
            yb = ptx::ffma2(sc_pair(u + e + 2), c2, rb);
        }
        if (HOW >= kScBiased && e < 12) {
            ra = ptx::fadd2(ra, bias2);
            rb = ptx::fadd2(rb, bias2);
        }
        float y0, y1, y2, y3;
        ptx::f2unpack(ya, y0, y1);
        ptx::f2unpack(yb, y2, y3);
        const float e0 = ptx::ex2(y0), e1 = ptx::ex2(y1), e2 = ptx::ex2(y2), e3 = ptx::ex2(y3);
        acc0 = ptx::fadd2(acc0, ptx::f2pack(e0, e1));
        acc1 = ptx::fadd2(acc1, ptx::f2pack(e2, e3));
        w[e / 2] = cvt_f16x2_sat(e1, e0);
        w[e / 2 + 1] = cvt_f16x2_sat(e3, e2);
    }
}
// The tile's P over its scores, 16 columns at a time, each loaded when the ones before are done with: a rolled loop, whose code
// stays small (instruction fetch is what a longer one waits for).  d: the first key less the one whose bias is zero.
template <int HOW>
__device__ __forceinline__ void sc_p64(uint32_t scol, float c, float ref, float k2, float cap, float slope, int d, uint64_t &l2) {
    constexpr bool kCap = HOW == kScCap || HOW == kScCapBiased, kBias = HOW >= kScBiased;
    const float cc = kCap ? -2.f * cap : c, rr = kCap ? cap + ref : ref;
    const uint64_t c2 = ptx::f2pack(cc, cc), bias2 = ptx::f2pack(4.f * slope, 4.f * slope);
    uint64_t acc0 = l2, acc1 = ptx::f2pack(0.f, 0.f);
    uint64_t ra = ptx::f2pack(rr, rr), rb = ra;
    auto bias = [&](int k) {
        if (!kBias) return;
        const float f = (float)(d + k);
        ra = ptx::f2pack(fmaf(slope, f, rr), fmaf(slope, f + 1.f, rr));
        rb = ptx::f2pack(fmaf(slope, f + 2.f, rr), fmaf(slope, f + 3.f, rr));
    };
    uint32_t ua[16], w[8];
#pragma unroll 1
    for (int q = 0; q < 4; ++q) {
        ptx::tmem_ld16(scol + 16 * q, ua);
        bias(16 * q);
        ptx::tmem_wait_ld();
        ptx::reg_fence16(ua);
        sc_p16<HOW>(ua, c2, ra, rb, bias2, k2, acc0, acc1, w);
        ptx::tmem_st8(scol + 8 * q, w);
    }
    l2 = ptx::fadd2(acc0, acc1);
}

// The tile's scores, in log2 units and capped in place, to 2^-20 of themselves.  Two exponentials and a shared reciprocal are
// good to 2^-20 of the cap, at 128 half of the weights' rounding; caps above that (kFarCap) take this pass of their own and go
// on as scores without one (two causal prompts of 4096, a cap of 1000: 412 us, of 50 338).
__device__ __forceinline__ void sc_cap64(uint32_t scol, float c, float k2, float cap) {
#pragma unroll 1
    for (int h = 0; h < kScTile; h += 8) {
        uint32_t v[8];
        ptx::tmem_ld8(scol + h, v);
        ptx::tmem_wait_ld();
        ptx::reg_fence8(v);
        float s[8], x = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            s[e] = u2f(v[e]);
            x = sc_max3(x, fabsf(s[e] * k2), x);
            v[e] = __float_as_uint(sc_cap_series(s[e], c, k2));
        }
        if (!__all_sync(0xffffffffu, x < kCapSeries)) {  // (rare under a cap of this size)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (!(fabsf(s[e] * k2) < kCapSeries)) v[e] = __float_as_uint(sc_cap_near(s[e], k2, cap));
        }
        ptx::tmem_st8(scol + h, v);
    }
    ptx::tmem_wait_st();
}

// NaNs of V in the noted tiles of unit un, into the outputs of those of the warp's rows (r) that see them, or into their parts, after
// these have been written: the next unit's products do not wait for it.  A lane looks through a key.  Whole warp.
template <typename C, int DV>
static __device__ __noinline__ void sc_put_nans(const ScoredParams &p, const uint8_t *misc, uint32_t un, int r) {
    constexpr int W = DV / 32;
    const ScUnit &u = *reinterpret_cast<const ScUnit *>(misc + C::OFF_UNIT + 64 * (un % kScUnits));
    const unsigned long long *noted = reinterpret_cast<const unsigned long long *>(misc + C::OFF_NAN) + 4 * (un % kScUnits);
    const int lane = threadIdx.x & 31, nt = u.t1 - u.t0, i = u.pos0 + r / p.G;
    const bool row_ok = r < p.P * p.G && i < u.rq.Lq;
    ScRow row = {0, 0, 0, nullptr};
    if (row_ok) row = sc_row(p, u.b, u.rq, i);
    uint32_t bad[W] = {};
    if (!__any_sync(0xffffffffu, row_ok)) return;
    for (unsigned long long tiles = noted[0] | noted[1] | noted[2] | noted[3]; tiles; tiles &= tiles - 1) {
        for (int t = __ffsll((long long)tiles) - 1; t < nt; t += 64) {
            for (int h = 0; h < kScTile; h += 32) {
                const int k = (u.t1 - 1 - t) * kScTile + h;
                const uint8_t *v = k + lane < u.rq.Lk ? sc_v_row(p, u.b, u.rq, u.kvh, k + lane) : nullptr;
                uint32_t bits[W], any = 0;
#pragma unroll
                for (int w = 0; w < W; ++w) {
                    bits[w] = 0;
                    if (v) {
                        const uint4 x = *reinterpret_cast<const uint4 *>(v + 32 * w), y = *reinterpret_cast<const uint4 *>(v + 32 * w + 16);
                        bits[w] = sc_nans({x.x, x.y, x.z, x.w}) | sc_nans({y.x, y.y, y.z, y.w}) << 16;
                    }
                    any |= bits[w];
                }
                for (uint32_t m = __ballot_sync(0xffffffffu, any != 0); m; m &= m - 1) {
                    const int l = __ffs(m) - 1;
                    const bool sees = sc_sees(row, p.words, k + l);
#pragma unroll
                    for (int w = 0; w < W; ++w) {
                        const uint32_t x = __shfl_sync(0xffffffffu, bits[w], l);
                        if (sees) bad[w] |= x;
                    }
                }
            }
        }
    }
    if (!row_ok) return;
    const int hq = u.kvh * p.G + r % p.G;
    uint16_t *out = static_cast<uint16_t *>(p.o) + (p.cu_q ? 0 : u.b) * p.o_s[0] + ((long long)u.rq.q0 + i) * p.o_s[1] + (long long)hq * p.o_s[2];
    float *part = u.slot >= 0 ? p.part + ((long long)u.slot * 128 * (DV / 4) + r) * 4 : nullptr;
#pragma unroll
    for (int w = 0; w < W; ++w)
        for (uint32_t m = bad[w]; m; m &= m - 1) {
            const int c = 32 * w + __ffs(m) - 1;
            if (part) part[(c / 4) * 128 * 4 + c % 4] = NAN;
            else out[c] = 0x7fff;  // of bf16 and of fp16
        }
}

// A bounded wait.  The timer is asked once in 256 tries: reading it takes longer than most waits.
__device__ __forceinline__ bool sc_wait_lane(uint32_t bar, uint32_t parity, uint32_t abort_saddr, unsigned long long timeout,
                                             unsigned int *status) {
    unsigned long long t0 = 0;
#pragma unroll 1
    for (unsigned int n = 1; !ptx::mbar_try_wait(bar, parity); ++n) {
        if (n & 255u) continue;
        const unsigned long long now = ptx::globaltimer();
        int ab;
        asm volatile("ld.volatile.shared.b32 %0, [%1];" : "=r"(ab) : "r"(abort_saddr));
        if (t0 == 0) t0 = now;
        if (!ab && now - t0 > timeout) {
            ab = 1;
            asm volatile("st.volatile.shared.b32 [%0], %1;" ::"r"(abort_saddr), "r"(1));
            atomicOr(status, kStatusTimeout);
        }
        if (ab) return false;
    }
    return true;
}
__device__ __forceinline__ bool sc_wait(uint32_t bar, uint32_t parity, uint32_t abort_saddr, unsigned long long timeout, unsigned int *status) {
    return __all_sync(0xffffffffu, sc_wait_lane(bar, parity, abort_saddr, timeout, status));
}

// The running maximum that the word at `saddr` holds after n tiles.
__device__ __forceinline__ bool sc_take(uint32_t saddr, uint32_t n, float *m, uint32_t abort_saddr, unsigned long long timeout, unsigned int *status) {
    unsigned long long t0 = 0, w;
    bool ok = true;
#pragma unroll 1
    for (unsigned int k = 1;; ++k) {
        asm volatile("ld.volatile.shared.b64 %0, [%1];" : "=l"(w) : "r"(saddr) : "memory");
        if ((uint32_t)w == n) break;
        if (k & 1023u) continue;
        const unsigned long long now = ptx::globaltimer();
        int ab;
        asm volatile("ld.volatile.shared.b32 %0, [%1];" : "=r"(ab) : "r"(abort_saddr));
        if (t0 == 0) t0 = now;
        if (!ab && now - t0 > timeout) {
            ab = 1;
            asm volatile("st.volatile.shared.b32 [%0], %1;" ::"r"(abort_saddr), "r"(1));
            atomicOr(status, kStatusTimeout);
        }
        if (ab) {
            ok = false;
            break;
        }
    }
    *m = u2f((uint32_t)(w >> 32));
    return __all_sync(0xffffffffu, ok);
}

// CAPS, BIAS: kernels of their own (slopes in the other kernels' code: d = 64 with slopes 239 us; far caps in the near ones':
// capped prompt 350 beside 337)
template <int D, int DV, int CAPS, bool BIAS>
__global__ void __launch_bounds__(kScThreads, 1)
    scored_kernel(const __grid_constant__ ScoredParams p, const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                  const __grid_constant__ CUtensorMap tm_v) {
    using C = ScCfg<D, DV>;
    constexpr bool CAP = CAPS == kScNearCap, FAR = CAPS == kScFarCap;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint8_t *misc = smem + C::OFF_MISC;
    const uint32_t bar0 = ptx::smem_u32(misc);
    auto BAR = [&](int i) -> uint32_t { return bar0 + 8u * (uint32_t)i; };
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(misc + C::OFF_SLOT);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(misc + C::OFF_ABORT);
    volatile unsigned long long *nan_tiles = reinterpret_cast<volatile unsigned long long *>(misc + C::OFF_NAN);
    const uint32_t sQ = ptx::smem_u32(smem + C::OFF_Q), sK = ptx::smem_u32(smem + C::OFF_K), sV = ptx::smem_u32(smem + C::OFF_V),
                   sF = ptx::smem_u32(smem + C::OFF_F);
    if (tid < 128) reinterpret_cast<unsigned long long *>(misc + C::OFF_M)[tid] = 0;
    if (tid == 0) {
        ptx::mbar_init(BAR(C::B_QF), 1);
        ptx::mbar_init(BAR(C::B_QE), 1);
        ptx::mbar_init(BAR(C::B_EO), 4);
        ptx::mbar_init(BAR(C::B_CL), 1);
        ptx::mbar_init(BAR(C::B_DONE), 1);
        ptx::mbar_init(BAR(C::B_DONE + 1), 1);
        for (int x = 0; x < C::NSB; ++x) {
            if (x % 2 == 0) ptx::mbar_init(BAR(C::B_SF + x / 2), 1);
            ptx::mbar_init(BAR(C::B_PF + x), 4);
            ptx::mbar_init(BAR(C::B_OD + x), 1);
        }
        for (int x = 0; x < 2; ++x) {
            ptx::mbar_init(BAR(C::B_LD + x), 4 * kScGroups);
            ptx::mbar_init(BAR(C::B_LE + x), 4);
        }
        for (int i = 0; i < C::ST; ++i) {
            ptx::mbar_init(BAR(C::B_KF + i), 1);
            ptx::mbar_init(BAR(C::B_KE + i), C::ONE ? 3 : 1);
        }
        for (int i = 0; i < C::STV; ++i) {
            ptx::mbar_init(BAR(C::B_VF + i), 1);
            ptx::mbar_init(BAR(C::B_VE + i), 4 / C::WIDE);
        }
        for (int i = 0; i < C::STF; ++i) ptx::mbar_init(BAR(C::B_FF + i), 4 / C::WIDE);
        for (int x = 0; x < kScUnits; ++x) {
            ptx::mbar_init(BAR(C::B_UF + x), 1);
            ptx::mbar_init(BAR(C::B_UE + x), kScCtl + 3);  // all warps but the one that writes them
        }
        *abort_flag = 0;
        ptx::fence_mbar_init();
        ptx::fence_proxy_async_smem();
    }
    if (warp == kScCtl) {
        if (lane == 0) {
            ptx::prefetch_tmap(&tm_q);
            if (p.has_kv) {
                ptx::prefetch_tmap(&tm_k);
                ptx::prefetch_tmap(&tm_v);
            }
        }
        ptx::tmem_alloc(ptx::smem_u32(tmem_slot), 512);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    if (p.split) ptx::griddep_launch_dependents();  // the joining kernel waits for all of this one
    const uint32_t tmem = *tmem_slot;
    const Waiter W{abort_flag, p.timeout_ns, p.status};
    const uint32_t abort_saddr = ptx::smem_u32(misc + C::OFF_ABORT);
    auto wait = [&](uint32_t bar, uint32_t parity) -> bool { return sc_wait(bar, parity, abort_saddr, p.timeout_ns, p.status); };
    auto wait_lane = [&](uint32_t bar, uint32_t parity) -> bool { return sc_wait_lane(bar, parity, abort_saddr, p.timeout_ns, p.status); };
    // The units go through shared memory from the one warp that works them out: copies of that code in every role
    // would drive what runs per tile out of the instruction cache.
    ScUnit u;
    uint32_t un = 0;  // units so far
    const uint32_t units_saddr = ptx::smem_u32(misc + C::OFF_UNIT);
    auto read_unit = [&](uint32_t n) {
        int4 *w = reinterpret_cast<int4 *>(&u);
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = ptx::ld_shared_v4_volatile(units_saddr + 64 * (n % kScUnits) + 16 * i);
    };
    auto release_unit = [&](uint32_t n) {
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(BAR(C::B_UE + n % kScUnits));
    };
    auto next_unit = [&]() -> bool {  // reads and releases it
        if (!wait(BAR(C::B_UF + un % kScUnits), un / kScUnits & 1u)) return false;
        read_unit(un);
        release_unit(un);
        ++un;
        return !u.end;
    };

    // what row r of the unit sees
    auto row_of = [&](int r, bool row_ok) -> ScRow {
        ScRow y;
        y.lo = 0;
        y.hi = y.lp = 0x7fffffff;
        y.words = nullptr;
        if (row_ok) {
            const volatile int *w = reinterpret_cast<const volatile int *>(misc + C::OFF_ROWS + 1024 * (un % kScUnits)) + 2 * (r / p.G);
            y.lo = w[0];
            y.hi = w[1];
            if (p.masks) {
                y.lp = u.rq.Lk - u.rq.Lq;
                y.words = p.masks + (p.cu_q ? 0 : u.b) * p.m_s[0] + ((long long)u.rq.q0 + u.pos0 + r / p.G) * p.m_s[1];
            }
        }
        return y;
    };

    if (warp >= kScCtl) {
        ptx::setmaxnreg_dec<kScRegsC>();
        const bool paged = p.kv_mode == 2;
        // One tile's TMA boxes: a lane each.  A box's table entry is asked for two steps ahead: its latency would be paid
        // per step.
        struct Boxes {
            int j, e, row;  // key, table column and row of the box two steps ahead
            int2 e0, e1;    // entry and row of the next two
        } x = {};
        constexpr int kNoEntry = -0x7fffffff;
        auto entry = [&]() -> int2 {
            const bool any = lane < p.boxes && x.j >= u.t0 * kScTile && x.j < u.rq.Lk;
            const int2 y = make_int2(any ? p.bt[u.b * p.bt_stride + x.e] : kNoEntry, any ? x.row : 0);
            x.j -= 2 * kScTile;
            x.e -= p.step_e;
            x.row -= p.step_r;
            if (x.row < 0) {
                x.row += p.page_size;
                --x.e;
            }
            return y;
        };
        auto boxes_of = [&]() {  // from the unit's last two tiles on
            x.row = u.rq.k0 + (u.t1 - 2) * kScTile;
            if (!paged) return;
            x.j = (u.t1 - 2) * kScTile + lane * p.box_n;
            x.e = x.j / p.page_size;  // (a key before the first has no entry, and none follows it)
            x.row = x.j - x.e * p.page_size;
            x.e0 = entry();
            x.e1 = entry();
        };
        auto next_box = [&](int &page, int &row) {
            page = p.kv_mode == 1 ? 0 : u.b;
            row = x.row;
            if (!paged) {
                x.row -= 2 * kScTile;
                return;
            }
            page = x.e0.x;
            row = x.e0.y;
            if (page < 0 || page >= p.num_pages) {
                if (page != kNoEntry) atomicOr(p.status, kStatusBounds);
                page = p.num_pages;  // out of range: TMA fills zeros
            }
            x.e0 = x.e1;
            x.e1 = entry();
        };
        const bool in = lane < (paged ? p.boxes : 1);
        bool ok = true;
        if (warp == kScCtl) {
            // ======================================================== units and Q
            int qf = 0;  // loads issued
            ScIter it;
            it.init(p, sc_cuts<DV>(p, gridDim.x));
            uint32_t cl = 0;  // phase of the answers
            auto steal = [&](int *x) -> bool {
                if (lane == 0) {
                    ptx::fence_proxy_async_smem();  // the answer before has been read
                    ptx::mbar_arrive_expect_tx(BAR(C::B_CL), 16);
                    ptx::cancel_cta(ptx::smem_u32(misc + C::OFF_CL), BAR(C::B_CL));
                }
                __syncwarp();
                if (!W.drain(BAR(C::B_CL), cl)) {  // (bounded, and not given up halfway: the answer is written to shared memory)
                    *abort_flag = 1;
                    return false;
                }
                cl ^= 1u;
                const bool mine = ptx::canceled_cta(ptx::smem_u32(misc + C::OFF_CL), x);
                __syncwarp();
                return mine;
            };
            while (ok) {
                const bool any = it.next(p, p.P, &u, steal);
                u.end = any ? 0 : 1;
                float dqv = 1.f, dkv = 1.f;
                if (any) {
                    if (p.dq) dqv = p.dq[u.b * p.dq_s[0] + u.kvh * p.dq_s[1]];
                    if (p.dk) dkv = p.dk[u.b * p.dk_s[0] + u.kvh * p.dk_s[1]];
                    const int e = paged && u.rq.Lk > 0 ? (min(u.t1 * kScTile, u.rq.Lk) - 1) / p.page_size - 32 * lane : -1;
                    if (e >= 0 && lane < 4) asm volatile("prefetch.global.L2 [%0];" ::"l"(p.bt + u.b * p.bt_stride + e));  // for the loader
                }
                const uint32_t ux = un % kScUnits;
                if (!wait(BAR(C::B_UE + ux), (un / kScUnits & 1u) ^ 1u)) { ok = false; break; }
                if (any) {
                    int flo = 0, fhi = 0x7fffffff, slo = 0x7fffffff, shi = 0;
                    for (int i = lane; i < p.P; i += 32) {
                        if (u.pos0 + i >= u.rq.Lq) break;
                        const ScRow r = sc_row(p, u.b, u.rq, u.pos0 + i);
                        reinterpret_cast<int2 *>(misc + C::OFF_ROWS + 1024 * ux)[i] = make_int2(r.lo, r.hi);
                        flo = max(flo, r.lo);
                        fhi = min(fhi, min(r.hi, max(0, r.lp)));
                        slo = min(slo, r.lo);
                        shi = max(shi, r.hi);
                    }
                    __syncwarp();
                    u.scale = p.scale_log2 * dqv * dkv;
                    if (u.scale == 0.f) u.scale = 0x1p-126f;  // below fp32: a masked -inf must stay one
                    u.flo = __reduce_max_sync(0xffffffffu, flo);
                    u.fhi = __reduce_min_sync(0xffffffffu, fhi);
                    u.slo = __reduce_min_sync(0xffffffffu, slo);
                    u.shi = __reduce_max_sync(0xffffffffu, shi);
                }
                if (lane == 0) {
                    const int4 *w = reinterpret_cast<const int4 *>(&u);
#pragma unroll
                    for (int i = 0; i < 4; ++i) ptx::st_shared_v4(units_saddr + 64 * ux + 16 * i, w[i].x, w[i].y, w[i].z, w[i].w);
                    ptx::mbar_arrive(BAR(C::B_UF + ux));
                }
                __syncwarp();
                ++un;
                if (!any) break;
                if (u.t1 <= u.t0) continue;
                if (!wait(BAR(C::B_QE), ((uint32_t)qf & 1u) ^ 1u)) { ok = false; break; }
                if (lane == 0) {
                    ptx::mbar_arrive_expect_tx(BAR(C::B_QF), (uint32_t)(D * p.P * p.G));
#pragma unroll
                    for (int c = 0; c < C::NCK; ++c)
                        ptx::tma_load_4d(sQ + c * C::CHUNK_Q, &tm_q, BAR(C::B_QF), c * C::CW, u.kvh * p.G, (p.cu_q ? u.rq.q0 : 0) + u.pos0,
                                         p.cu_q ? 0 : u.b);
                }
                __syncwarp();
                ++qf;
            }
            if (*abort_flag && qf > 0) W.drain(BAR(C::B_QF), (uint32_t)(qf - 1) & 1u);  // loads must land before shared memory is released
            __syncwarp();
        } else if (warp == kScCtl + 3) {
            // ======================================================== K and V, two tiles a step
            int s = 0, kf = 0, vf = 0;  // stage; loads issued
            uint32_t ph = 1;
            while (ok && next_unit()) {
                if (u.t1 <= u.t0) continue;
                boxes_of();
                for (int t = u.t0; ok && t < u.t1; t += 2) {
                    int page, row;
                    next_box(page, row);
                    if (!wait(BAR(C::B_KE + s), ph)) { ok = false; break; }
                    if (lane == 0) {
                        ptx::mbar_arrive_expect_tx(BAR(C::B_KF + s), (uint32_t)C::K_BYTES);
                        if (C::ONE) ptx::mbar_arrive_expect_tx(BAR(C::B_VF + s), (uint32_t)C::V_BYTES);
                    }
                    __syncwarp();
                    if (in) {
#pragma unroll
                        for (int c = 0; c < C::NCK; ++c)
                            ptx::tma_load_4d(sK + s * C::K_BYTES + c * C::CHUNK_K + lane * p.box_n * C::CW, &tm_k, BAR(C::B_KF + s),
                                             c * C::CW, u.kvh, row, page);
                        if (C::ONE) ptx::tma_load_4d(sV + s * C::V_BYTES + lane * p.box_n * DV, &tm_v, BAR(C::B_VF + s), 0, u.kvh, row, page);
                    }
                    ++kf;
                    if constexpr (!C::ONE) {
                        // a tile's V each: half of the boxes (all of its rows in one where K's two tiles are one box)
                        const int half = p.boxes > 1 ? p.boxes / 2 : 1;
                        for (int h = 0; h < 2; ++h) {
                            const int sv = vf % C::STV;
                            if (!wait(BAR(C::B_VE + sv), ((uint32_t)(vf / C::STV) & 1u) ^ 1u)) { ok = false; break; }
                            if (lane == 0) ptx::mbar_arrive_expect_tx(BAR(C::B_VF + sv), (uint32_t)C::V_BYTES);
                            __syncwarp();
                            const int y = p.boxes > 1 ? lane - (1 - h) * half : lane;
                            if (y >= 0 && y < half)
                                ptx::tma_load_4d(sV + sv * C::V_BYTES + y * p.box_v * DV, &tm_v, BAR(C::B_VF + sv), 0, u.kvh,
                                                 p.boxes > 1 ? row : row + (1 - h) * kScTile, page);
                            ++vf;
                        }
                    } else {
                        ++vf;
                    }
                    if (++s == C::ST) s = 0, ph ^= 1u;
                }
            }
            if (*abort_flag) {
                for (int i = max(0, kf - C::ST); i < kf; ++i) W.drain(BAR(C::B_KF + i % C::ST), (uint32_t)(i / C::ST) & 1u);
                for (int i = max(0, vf - C::STV); i < vf; ++i) W.drain(BAR(C::B_VF + i % C::STV), (uint32_t)(i / C::STV) & 1u);
            }
            __syncwarp();
        } else {
            // ======================================================== MMA issuers: one lane each
            const bool leader = ptx::elect_one();
            int buf = 0, stage = 0;  // of S and P; of K or of f16 V
            uint32_t sph = 0, ph = 0, uph = 0;
            if (warp == kScCtl + 1) {
                // S = Q K^T of two tiles, over the P of NSB tiles before, whose products must be complete
                constexpr uint32_t kIdesc = idesc_e4m3(128, 2 * kScTile, false);
                const uint64_t dk0 = sdesc(sK, 16, 8 * C::CW, swz_layout(C::CW)), dq = sdesc(sQ, 16, 8 * C::CW, swz_layout(C::CW));
                while (ok && next_unit()) {
                    const int nt = u.t1 - u.t0;
                    if (nt <= 0) continue;
                    if (leader) ok = wait_lane(BAR(C::B_QF), uph);
                    uph ^= 1u;
                    for (int t = 0; leader && ok && t < nt; t += 2) {
                        if (!(ok = wait_lane(BAR(C::B_OD + buf + 1), sph ^ 1u) && wait_lane(BAR(C::B_KF + stage), ph))) break;
                        ptx::tc_fence_after();
                        const uint64_t dk = dk0 + (uint64_t)((stage * C::K_BYTES) >> 4);
#pragma unroll
                        for (int kk = 0; kk < D / 32; ++kk) {
                            const int c = (kk * 32) / C::CW, y = (kk * 32) % C::CW;
                            ptx::mma_f8_ss(tmem + (uint32_t)(buf * kScTile), dq + (uint32_t)((c * C::CHUNK_Q + y) >> 4),
                                           dk + (uint32_t)((c * C::CHUNK_K + y) >> 4), kIdesc, kk > 0 ? 1u : 0u);
                        }
                        ptx::tc_commit(BAR(C::B_SF + buf / 2));
                        ptx::tc_commit(BAR(C::B_KE + stage));
                        if (t + 2 >= nt) ptx::tc_commit(BAR(C::B_QE));
                        if (++stage == C::ST) stage = 0, ph ^= 1u;
                        if ((buf += 2) == C::NSB) buf = 0, sph ^= 1u;
                    }
                    ok = __all_sync(0xffffffffu, ok);
                }
            } else {
                // O += P V.  (An odd unit's last pair has one tile: the other's barriers go on without a product.)
                constexpr uint32_t kIdesc = idesc_e4m3(128, DV, true);  // the same bits, of kind::f16: f16 x f16
                const uint64_t df0 = sdesc(sF, C::CHUNK_F, 8 * C::CF, swz_layout(C::CF));
                while (ok && next_unit()) {
                    const int nt = u.t1 - u.t0;
                    if (nt <= 0) continue;
                    if (leader) ok = wait_lane(BAR(C::B_EO), uph ^ 1u);  // the last unit's O has been read
                    uph ^= 1u;
                    for (int t = 0; leader && ok && t < nt; t += 2) {
                        const uint64_t df = df0 + (uint64_t)((stage * C::VF_BYTES) >> 4);
#pragma unroll
                        for (int h = 0; h < 2; ++h) {  // the upper tile first
                            if (!(ok = wait_lane(BAR(C::B_FF + stage + h), ph) && wait_lane(BAR(C::B_PF + buf + 1 - h), sph))) break;
                            ptx::tc_fence_after();
                            if (h == 0 || t + 1 < nt) {
#pragma unroll
                                for (int kk = 0; kk < kScTile / 16; ++kk)
                                    ptx::mma_f16_ts(tmem + C::TM_O, tmem + (uint32_t)((buf + 1 - h) * kScTile + kk * 8),
                                                    df + (uint64_t)((h * C::VF_BYTES + kk * 16 * C::CF) >> 4), kIdesc, h + kk > 0 || t > 0 ? 1u : 0u);
                            }
                            ptx::tc_commit(BAR(C::B_OD + buf + h));
                        }
                        if ((stage += 2) == C::STF) stage = 0, ph ^= 1u;
                        if ((buf += 2) == C::NSB) buf = 0, sph ^= 1u;
                    }
                    ok = __all_sync(0xffffffffu, ok);
                }
            }
            const uint32_t done = BAR(C::B_DONE + warp - kScCtl - 1);  // this issuer's MMAs must finish before TMEM is released
            if (leader) ptx::tc_commit(done);
            __syncwarp();
            W.drain(done, 0);
            __syncwarp();
        }
    } else if (warp >= kScConv) {
        // ======================================================== V to f16
        ptx::setmaxnreg_dec<kScRegsV>();
        // each warp takes every fourth tile (pairs every second), so that a tile's waits overlap the others' work
        const int wid = warp - kScConv, part = wid / C::WIDE;
        int g = 0;  // tiles of the CTA before the unit
        bool ok = true;
        while (ok && next_unit()) {
            const int nt = max(0, u.t1 - u.t0), even = nt + 1 & ~1;
            const uint32_t nx = un - 1;  // (the unit that had this word has written its output: its place is free)
            if (lane == 0) nan_tiles[(nx % kScUnits) * 4 + wid] = 0;
            __syncwarp();
            for (int t = (wid - g) & (C::WIDE - 1); t < even; t += C::WIDE) {
                const int at = g + t, fs = at % C::STF, k = (u.t1 - 1 - t) * kScTile;
                const int load = C::ONE ? at / 2 : at, vs = load % C::STV, last = at - C::STF;  // last: whose place this takes
                if (!wait(BAR(C::B_VF + vs), (uint32_t)(load / C::STV) & 1u)) { ok = false; break; }
                if (last >= 0 && !wait(BAR(C::B_OD + last % C::NSB), (uint32_t)(last / C::NSB) & 1u)) { ok = false; break; }
                const uint32_t src = sV + vs * C::V_BYTES + (C::ONE ? (~at & 1) * C::V_TILE : 0), dst = sF + fs * C::VF_BYTES;
                // keys that some rows see and others do not: their NaNs go in as zeros (a masked weight of zero
                // would not silence them) and are put into the rows that see them with the output
                const bool partial = k < u.flo || k + kScTile > u.fhi;
                constexpr int NP = C::CF / 32;  // 16-byte pieces of V's rows per chunk
                constexpr int KP = 32 / NP;     // keys per pass
                const int piece = lane % NP, key0 = lane / NP;
                const int sw = C::CF == 128 ? key0 & 7 : (key0 >> 1) & 3;  // KP is a multiple of 8
                static_assert(KP % 8 == 0 && kScTile % KP == 0, "passes");
                bool found = false;
#pragma unroll 1
                for (int key = t < nt ? key0 + part * KP : kScTile; key < kScTile; key += KP * (4 / C::WIDE)) {
                    // lanes of odd keys take the chunks in another order where that spreads the banks
                    Bytes<16> w[C::NCF];
#pragma unroll
                    for (int x = 0; x < C::NCF; ++x) {
                        const int chunk = C::NCF % 2 == 0 ? x ^ (key0 & 1) : x;
                        w[x] = ld_shared<16>(src + key * DV + chunk * (C::CF / 2) + piece * 16);
                    }
                    if (partial) {
                        uint32_t any = 0;
#pragma unroll
                        for (int x = 0; x < C::NCF; ++x)
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const uint32_t bad = ((w[x].w[e] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
                                any |= bad;
                                w[x].w[e] &= ~((bad >> 7) * 0xffu);
                            }
                        found |= any && k + key >= u.slo && k + key < u.shi;
                    }
#pragma unroll
                    for (int x = 0; x < C::NCF; ++x) {
                        const int chunk = C::NCF % 2 == 0 ? x ^ (key0 & 1) : x;
                        uint32_t h[8];
#pragma unroll
                        for (int e = 0; e < 4; ++e) e4m3x4_to_h2(w[x].w[e], h[2 * e], h[2 * e + 1]);
                        const uint32_t row = dst + chunk * C::CHUNK_F + key * C::CF;
                        ptx::st_shared_v4(row + (((2 * piece) ^ sw) << 4), h[0], h[1], h[2], h[3]);
                        ptx::st_shared_v4(row + (((2 * piece + 1) ^ sw) << 4), h[4], h[5], h[6], h[7]);
                    }
                }
                if (partial && __any_sync(0xffffffffu, found) && lane == 0) nan_tiles[(nx % kScUnits) * 4 + wid] |= 1ull << (t & 63);
                ptx::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    ptx::mbar_arrive(BAR(C::B_FF + fs));
                    ptx::mbar_arrive(BAR((C::ONE ? C::B_KE : C::B_VE) + vs));
                }
            }
            g += even;
        }
    } else if (warp >= kScOut) {
        // ======================================================== output
        ptx::setmaxnreg_inc<kScRegsO>();
        const int r = tid - 32 * kScOut;
        const uint32_t tm_o = tmem + ((uint32_t)((warp & 3) * 32) << 16) + C::TM_O;
        int i0 = 0, n = 0;  // tiles of the CTA, units with tiles
        while (wait(BAR(C::B_UF + un % kScUnits), un / kScUnits & 1u)) {
            read_unit(un);
            if (u.end) break;
            const bool any = u.t1 > u.t0;
            // all that the output needs beside O comes first: the next unit's products wait while O is read
            const int rp = u.pos0 + r / p.G, hq = u.kvh * p.G + r % p.G;
            const bool row_ok = r < p.P * p.G && rp < u.rq.Lq;
            const long long bb = p.cu_q ? 0 : u.b, tt = (long long)u.rq.q0 + rp;
            const float dv = p.dv ? p.dv[u.b * p.dv_s[0] + u.kvh * p.dv_s[1]] : 1.f;
            const ScRow row = row_of(r, row_ok);
            float off = 0.f;
            if (BIAS && row_ok) off = sc_bias(p, row, rp + u.rq.Lk - u.rq.Lq, hq).off;
            float m = -INFINITY, l = 0.f;
            if (any) {
                const int first = i0;  // its group's share comes first: the same sum whatever the CTA did before
                i0 += u.t1 - u.t0 + 1 & ~1;
                if (!wait(BAR(C::B_LD + (n & 1)), (uint32_t)(n >> 1) & 1u)) break;
                const float2 *x = reinterpret_cast<const float2 *>(misc + C::OFF_L) + 128 * kScGroups * (n & 1) + r;
                float2 ml[kScGroups];
#pragma unroll
                for (int y = 0; y < kScGroups; ++y) {
                    ml[y] = x[128 * (first + y & (kScGroups - 1))];
                    m = fmaxf(m, ml[y].x);
                }
                const float ref = m == -INFINITY ? 0.f : m;
#pragma unroll
                for (int y = 0; y < kScGroups; ++y) l = fmaf(ptx::ex2(ml[y].x - ref), ml[y].y, l);
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(BAR(C::B_LE + (n & 1)));
                ++n;
            }
            if (BIAS) m += off;
            const float *sink = p.sink && row_ok ? p.sink + hq : nullptr;
            const float f = sc_factor(m, l, sink, dv);
            uint8_t *dst = reinterpret_cast<uint8_t *>(p.o) + 2 * (bb * p.o_s[0] + tt * p.o_s[1] + (long long)hq * p.o_s[2]);
            if (any) {
                const int i = i0 - 1;  // the unit's last product
                if (!wait(BAR(C::B_OD + i % C::NSB), (uint32_t)(i / C::NSB) & 1u)) break;
                ptx::tc_fence_after();
            }
            bool nan = false;
#pragma unroll
            for (int w = 0; w < 4; ++w) nan |= nan_tiles[(un % kScUnits) * 4 + w] != 0;
            auto read = [&]() {  // O has been read: the next unit's products may go on
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(BAR(C::B_EO));
            };
            float4 *part = nullptr;
            if (u.slot >= 0) part = reinterpret_cast<float4 *>(p.part) + (long long)u.slot * 128 * (DV / 4) + r;
            // small loops: code that runs once a unit is fetched anew each time (64 columns unrolled, a division and log2f before:
            // 7200 cycles from the last product to the end of O's read, for which the next unit's products wait)
            const bool plain = any && !part;
            if (plain) {
#pragma unroll 1
                for (int x = 0; x < DV; x += 32) {
                    uint32_t v[32], w[16];
                    ptx::tmem_ld32(tm_o + x, v);
                    ptx::tmem_wait_ld();
                    ptx::reg_fence32(v);
                    if (x + 32 == DV) read();
                    const uint64_t f2 = ptx::f2pack(f, f);
#pragma unroll
                    for (int e = 0; e < 32; e += 2) sc_split(ptx::fmul2(sc_pair(v + e), f2), v + e);
                    if (p.out_fp16) {
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const __half2 h = __floats2half2_rn(u2f(v[2 * e]), u2f(v[2 * e + 1]));
                            w[e] = *reinterpret_cast<const uint32_t *>(&h);
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const __nv_bfloat162 h = __floats2bfloat162_rn(u2f(v[2 * e]), u2f(v[2 * e + 1]));
                            w[e] = *reinterpret_cast<const uint32_t *>(&h);
                        }
                    }
                    if (row_ok) {
#pragma unroll
                        for (int e = 0; e < 16; e += 4)
                            *reinterpret_cast<uint4 *>(dst + 2 * x + 4 * e) = make_uint4(w[e], w[e + 1], w[e + 2], w[e + 3]);
                    }
                    __syncwarp();
                }
            }
            if (part) reinterpret_cast<float2 *>(p.part + (long long)gridDim.x * 2 * 128 * DV)[(long long)u.slot * 128 + r] = make_float2(m, l);
            else if (row_ok && p.lse) p.lse[bb * p.lse_s[0] + tt * p.lse_s[1] + hq * p.lse_s[2]] = sc_lse(m, l, sink);
#pragma unroll 1
            for (int x = plain ? DV : 0; x < DV; x += 16) {
                uint32_t v[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) v[e] = 0u;
                if (any) {
                    ptx::tmem_ld16(tm_o + x, v);
                    ptx::tmem_wait_ld();
                    ptx::reg_fence16(v);
                    if (x + 16 == DV) read();
                }
                if (part && row_ok) {
#pragma unroll
                    for (int e = 0; e < 16; e += 4)
                        part[(long long)(x + e) / 4 * 128] = make_float4(u2f(v[e]), u2f(v[e + 1]), u2f(v[e + 2]), u2f(v[e + 3]));
                } else if (row_ok) {
                    float y[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) y[e] = u2f(v[e]) * f;
                    store8(dst + 2 * x, y, p.out_fp16);
                    store8(dst + 2 * x + 16, y + 8, p.out_fp16);
                }
                __syncwarp();
            }
            if (any && nan) sc_put_nans<C, DV>(p, misc, un, r);
            release_unit(un);
            ++un;
        }
    } else {
        // ======================================================== softmax
        const int grp = warp >> 2, r = tid & 127;  // which of the tiles, row
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t tm_o = tmem + lanes + C::TM_O;
        // A row's running maximum goes from tile to tile in one 8-byte word with the tile's number: no barrier, which
        // would cost the chain of all tiles two or three hundred cycles each.
        const uint32_t m_saddr = ptx::smem_u32(misc + C::OFF_M) + 8u * (uint32_t)r;
        auto take_m = [&](int i, float *m) -> bool { return sc_take(m_saddr, (uint32_t)i, m, abort_saddr, p.timeout_ns, p.status); };
        auto pass_m = [&](int i, float m) {
            asm volatile("st.volatile.shared.b64 [%0], %1;" ::"r"(m_saddr), "l"((unsigned long long)__float_as_uint(m) << 32 | (uint32_t)(i + 1)) : "memory");
        };
        int i0 = 0, n = 0;  // tiles of the CTA before the unit; units with tiles
        bool ok = true;
        while (ok && wait(BAR(C::B_UF + un % kScUnits), un / kScUnits & 1u)) {
            read_unit(un);
            if (u.end) break;
            const int nt = u.t1 - u.t0, t1 = u.t1;
            const bool row_ok = r < p.P * p.G && u.pos0 + r / p.G < u.rq.Lq;
            const ScRow row = row_of(r, row_ok);
            const bool idle = !__any_sync(0xffffffffu, row_ok);  // none of the warp's rows exists
            release_unit(un);
            ++un;
            if (nt <= 0) continue;
            float slope = 0.f;
            int pc = 0x7fffffff;
            if (BIAS && row_ok) {
                const ScBias x = sc_bias(p, row, u.pos0 + r / p.G + u.rq.Lk - u.rq.Lq, u.kvh * p.G + r % p.G);
                slope = x.slope;
                pc = x.pc;
            }
            const float c = FAR ? 1.f : u.scale, cap = p.cap_log2, k2 = CAPS != kScNoCap ? sc_k2(u.scale, cap) : 0.f;
            // tiles in [flo, fhi) need no mask in this warp; those that end before `left` lie left of all its positions
            const int flo = __reduce_max_sync(0xffffffffu, row.lo), fhi = __reduce_min_sync(0xffffffffu, min(row.hi, max(0, row.lp)));
            // (a negative scale, whose largest score is not the largest product's, has every tile's changed first)
            int left = BIAS ? __reduce_min_sync(0xffffffffu, pc == 0x7fffffff ? pc : pc + 1) : 0x7fffffff;
            if (c < 0.f) left = -1;
            float m = -INFINITY;  // running maximum less kScBias
            uint64_t l2 = ptx::f2pack(0.f, 0.f);  // this warp's share of the sum, in two parts
            const int even = nt + 1 & ~1;
            int k = (grp - i0) & (kScGroups - 1);
            for (; k < nt && !idle; k += kScGroups) {
                const int i = i0 + k, k0 = (t1 - 1 - k) * kScTile, bar = i % C::NSB ^ 1;  // (of a pair the upper tile goes first)
                const uint32_t scol = tmem + lanes + (uint32_t)(bar * kScTile);
                const bool partial = k0 < flo || k0 + kScTile > fhi;
                uint32_t sees0 = 0xffffffffu, sees1 = 0xffffffffu;  // (before the wait: masks come from memory)
                if (partial) {
                    sees0 = sc_see32(row, p.words, k0);
                    sees1 = sc_see32(row, p.words, k0 + 32);
                }
                bool prep = partial || k0 + kScTile > left;  // scores are changed in place first
                if (!wait(BAR(C::B_SF + bar / 2), (uint32_t)(i / C::NSB) & 1u)) { ok = false; break; }
                ptx::tc_fence_after();
                if (FAR) sc_cap64(scol, u.scale, k2, cap);
                // Rows that do not exist (heads that do not divide 128, positions past the request's) have scores of whatever
                // lies in their place of Q: their maximum is -inf, so that the votes below, and with them the other rows'
                // weights, do not depend on it.
                float mx = -INFINITY;
                if (!prep) {  // (the bias counts as the largest of the tile's)
#pragma unroll 1
                    for (int h = 0; h < kScTile; h += 16) {
                        uint32_t v[16];
                        ptx::tmem_ld16(scol + h, v);
                        ptx::tmem_wait_ld();
                        ptx::reg_fence16(v);
                        mx = sc_max16(mx, v);
                    }
                    prep = CAP && !__all_sync(0xffffffffu, mx * k2 <= 30.f || !row_ok);
                    mx = CAP ? sc_cap_near(mx, k2, cap) : mx * c;
                    if (BIAS) mx += slope * (float)(k0 + (slope > 0.f ? kScTile - 1 : 0) - pc);
                }
                if (prep) {
                    mx = -INFINITY;
                // to log2 units with all that belongs to them, masked ones to -inf
#pragma unroll 1
                    for (int h = 0; h < kScTile; h += 16) {
                        const int kh = k0 + h;
                        uint32_t v[16];
                        ptx::tmem_ld16(scol + h, v);
                        const uint32_t see = (h < 32 ? sees0 : sees1) >> (h & 16);
                        ptx::tmem_wait_ld();
                        ptx::reg_fence16(v);
                        if (CAP && partial) {
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                if (!(see >> e & 1u)) v[e] = 0u;  // a NaN would reach those that share its reciprocal
                        }
                        if (CAP) {
                            const uint64_t a2 = ptx::f2pack(cap, cap), b2 = ptx::f2pack(-2.f * cap, -2.f * cap);
#pragma unroll
                            for (int e = 0; e < 16; e += 4) {
                                uint64_t ia, ib;
                                sc_inv4<true>(v + e, k2, ia, ib);
                                sc_split(ptx::ffma2(ia, b2, a2), v + e);
                                sc_split(ptx::ffma2(ib, b2, a2), v + e + 2);
                            }
                        }
                        if constexpr (BIAS) {
                            const float cc = CAP ? 1.f : c;
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                v[e] = __float_as_uint(fmaf(-slope, fabsf((float)(pc - (kh + e))), u2f(v[e]) * cc));
                        }
                        if (!CAP && !BIAS) {
#pragma unroll
                            for (int e = 0; e < 16; ++e) v[e] = __float_as_uint(u2f(v[e]) * c);
                        }
                        if (partial) {
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                if (!(see >> e & 1u)) v[e] = 0xff800000u;  // -inf
                        }
                        mx = sc_max16(mx, v);
                        ptx::tmem_st16(scol + h, v);
                    }
                    ptx::tmem_wait_st();
                }

                if (!row_ok) mx = -INFINITY;

                // the maximum moves only when some row's score is 2^kScSlack above it; then O is scaled in TMEM
                float now;
                if (!take_m(i, &now)) { ok = false; break; }
                if (k > 0 && now != m) {  // another warp of these rows has moved it
                    const float a = ptx::ex2(m - now);
                    l2 = ptx::fmul2(l2, ptx::f2pack(a, a));
                    m = now;
                }
                bool moved = __any_sync(0xffffffffu, mx > m + (kScBias + kScSlack));
                if (BIAS && !prep && (moved || k == 0)) {  // the bound is not enough: the largest with each key's bias
                    mx = -INFINITY;
                    constexpr int N = CAP ? 8 : 16;  // columns a time (the prompts, 16 with a cap: 332 us beside 308; 8 without: 231 beside 224)
#pragma unroll 1
                    for (int h = 0; h < kScTile; h += N) {
                        uint32_t v[N];
                        if constexpr (CAP) ptx::tmem_ld8(scol + h, v);
                        else ptx::tmem_ld16(scol + h, v);
                        ptx::tmem_wait_ld();
                        if constexpr (CAP) ptx::reg_fence8(v);
                        else ptx::reg_fence16(v);
#pragma unroll
                        for (int e = 0; e < N; ++e) {
                            const float z = CAP ? sc_cap_near(u2f(v[e]), k2, cap) : u2f(v[e]) * c;
                            mx = fmaxf(mx, fmaf(slope, (float)(k0 + h + e - pc), z));
                        }
                    }
                    if (!row_ok) mx = -INFINITY;
                    moved = __any_sync(0xffffffffu, mx > m + (kScBias + kScSlack));
                }
                float alpha = 1.f;
                if (moved || k == 0) {
                    const float mn = fmaxf(m, mx - kScBias);
                    if (mn != -INFINITY) alpha = ptx::ex2(m - mn);
                    m = mn;
                    l2 = ptx::fmul2(l2, ptx::f2pack(alpha, alpha));
                }
                pass_m(i, m);
                if (moved && k > 0) {  // O is scaled once the product of the tile before is in it
                    if (!wait(BAR(C::B_OD + (i - 1) % C::NSB), (uint32_t)((i - 1) / C::NSB) & 1u)) { ok = false; break; }
                    ptx::tc_fence_after();
#pragma unroll 1
                    for (int x = 0; x < DV / 16; ++x) {
                        uint32_t y[16];
                        ptx::tmem_ld16(tm_o + 16 * x, y);
                        ptx::tmem_wait_ld();
                        ptx::reg_fence16(y);
#pragma unroll
                        for (int e = 0; e < 16; ++e) y[e] = __float_as_uint(u2f(y[e]) * alpha);
                        ptx::tmem_st16(tm_o + 16 * x, y);
                    }
                }
                // ---- P = 2^(z - m), over the scores
                const float ref = m == -INFINITY ? 0.f : -m;
                if (BIAS && __all_sync(0xffffffffu, mx < m - 40.f || !row_ok)) {  // all too small for f16, and 2^-47 of the largest in the sum
                    const uint32_t w[16] = {};
                    ptx::tmem_st16(scol, w);
                    ptx::tmem_st16(scol + 16, w);
                } else if ((CAP || BIAS) && prep) {
                    sc_p64<kScDone>(scol, 0.f, ref, 0.f, 0.f, 0.f, 0, l2);
                } else if (!CAP && !BIAS) {
                    sc_p64<kScPlain>(scol, prep ? 1.f : c, ref, 0.f, 0.f, 0.f, 0, l2);
                } else if (!BIAS) {
                    sc_p64<kScCap>(scol, 0.f, ref, k2, cap, 0.f, 0, l2);
                } else if (CAP) {
                    sc_p64<kScCapBiased>(scol, 0.f, ref, k2, cap, slope, k0 - pc, l2);
                } else {
                    sc_p64<kScBiased>(scol, c, ref, 0.f, 0.f, slope, k0 - pc, l2);
                }
                ptx::tmem_wait_st();
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(BAR(C::B_PF + bar));
            }
            for (; ok && k < even; k += kScGroups) {  // no rows, or no tile: the barriers alone
                const int i = i0 + k, bar = i % C::NSB ^ 1;
                float now;
                ok = wait(BAR(C::B_SF + bar / 2), (uint32_t)(i / C::NSB) & 1u) && take_m(i, &now);
                if (!ok) break;
                pass_m(i, now);
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(BAR(C::B_PF + bar));
            }
            if (!ok) break;
            i0 += even;
            // the share and what it is against, for the warps that write the output
            if (!wait(BAR(C::B_LE + (n & 1)), ((uint32_t)(n >> 1) & 1u) ^ 1u)) break;
            float la, lb;
            ptx::f2unpack(l2, la, lb);
            reinterpret_cast<float2 *>(misc + C::OFF_L)[128 * (kScGroups * (n & 1) + grp) + r] = make_float2(m, la + lb);
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(BAR(C::B_LD + (n & 1)));
            ++n;
        }
    }
    // ------------------------------------------------------------ teardown
    ptx::tc_fence_before();
    __syncthreads();
    if (warp == kScCtl) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, 512);
    }
}

// Units that the cuts went through: their parts, joined by their maxima.  CTA x takes the unit whose first cut is cut
// x + 1; y 8 columns (all of them have to be in flight: the parts come from L2); thread = row.  (32 columns to a CTA of 512
// threads: the tree of one request 20 us instead of 17.5; 32 to a thread: 28.)
constexpr int kScMergeCols = 8;
template <int DV>
__global__ void __launch_bounds__(128) scored_merge_kernel(const __grid_constant__ ScoredParams p, int ctas) {
    constexpr int rows = 128;
    const int c = blockIdx.x + 1, r = threadIdx.x;
    ptx::griddep_wait();  // the parts are written
    const int4 cut = sc_cuts<DV>(p, ctas)[c];
    const int b = cut.x, last = cut.z;
    if (b < 0) return;
    const int kvh = cut.y % p.Hkv, rp = (cut.y / p.Hkv) * p.P + r / p.G, hq = kvh * p.G + r % p.G;
    if (r >= p.P * p.G || rp >= p.Sq) return;
    const float2 *pm = reinterpret_cast<const float2 *>(p.part + (long long)ctas * 2 * rows * DV) + r;
    const float4 *po = reinterpret_cast<const float4 *>(p.part) + (long long)(kScMergeCols / 4) * blockIdx.y * rows + r;
    const float sink = p.sink ? p.sink[hq] : 0.f, dv = p.dv ? p.dv[b * p.dv_s[0] + kvh * p.dv_s[1]] : 1.f;
    float M = -INFINITY, L = 0.f, o[kScMergeCols];
#pragma unroll
    for (int e = 0; e < kScMergeCols; ++e) o[e] = 0.f;
    constexpr int NB = 8;  // parts in flight
    for (int i0 = c - 1; i0 <= last; i0 += NB) {
        float2 ml[NB];
        float4 v[NB][kScMergeCols / 4];
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            const long long slot = 2 * (i0 + i) + (i0 + i == c - 1 ? 1 : 0);
            const bool in = i0 + i <= last;
            ml[i] = in ? pm[slot * rows] : make_float2(-INFINITY, 0.f);
#pragma unroll
            for (int e = 0; e < kScMergeCols / 4; ++e)
                v[i][e] = in ? po[(slot * (DV / 4) + e) * rows] : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        float top = M;
#pragma unroll
        for (int i = 0; i < NB; ++i) top = fmaxf(top, ml[i].x);
        const float ref = top == -INFINITY ? 0.f : top, a = ptx::ex2(M - ref);
        L *= a;
#pragma unroll
        for (int e = 0; e < kScMergeCols; ++e) o[e] *= a;
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            const float f = ptx::ex2(ml[i].x - ref);
            L = fmaf(f, ml[i].y, L);
#pragma unroll
            for (int e = 0; e < kScMergeCols / 4; ++e) {
                o[4 * e] = fmaf(f, v[i][e].x, o[4 * e]);
                o[4 * e + 1] = fmaf(f, v[i][e].y, o[4 * e + 1]);
                o[4 * e + 2] = fmaf(f, v[i][e].z, o[4 * e + 2]);
                o[4 * e + 3] = fmaf(f, v[i][e].w, o[4 * e + 3]);
            }
        }
        M = top;
    }
    float f, lse;
    sc_finish(M, L, p.sink ? &sink : nullptr, dv, &f, &lse);
    if (p.lse && blockIdx.y == 0) p.lse[b * p.lse_s[0] + rp * p.lse_s[1] + hq * p.lse_s[2]] = lse;
    uint8_t *dst = reinterpret_cast<uint8_t *>(p.o) + 2 * (b * p.o_s[0] + rp * p.o_s[1] + (long long)hq * p.o_s[2] + kScMergeCols * blockIdx.y);
#pragma unroll
    for (int e = 0; e < kScMergeCols; ++e) o[e] *= f;
    store8(dst, o, p.out_fp16);
}

template <int D, int DV, int CAPS, bool BIAS>
fa8_status launch_scored_mode(const ScoredParams &p, const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv, int grid, int dev,
                              cudaStream_t s) {
    using C = ScCfg<D, DV>;
    static host::SmemOptIn opt_in;
    static std::atomic<int> regs{-1};
    // setmaxnreg draws on the registers of the launch: a count that the split was not planned for would wait forever
    if (regs < 0) {
        cudaFuncAttributes a;
        const cudaError_t e = cudaFuncGetAttributes(&a, scored_kernel<D, DV, CAPS, BIAS>);
        if (e != cudaSuccess) return host::cuda_fail(e, "scored attention kernel");
        regs = a.numRegs;
    }
    if (regs != kScRegs) return host::fail(FA8_ERR_CUDA, "scored attention kernel compiled to %d registers, %d planned", regs.load(), kScRegs);
    cudaError_t e = opt_in(scored_kernel<D, DV, CAPS, BIAS>, C::SMEM_BYTES, dev);
    if (e != cudaSuccess) return host::cuda_fail(e, "scored attention shared memory");
    scored_kernel<D, DV, CAPS, BIAS><<<grid, kScThreads, C::SMEM_BYTES, s>>>(p, tq, tk, tv);
    e = cudaGetLastError();
    if (e == cudaSuccess && p.split && grid > 1) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(grid - 1, DV / kScMergeCols);
        cfg.blockDim = dim3(128);
        cfg.stream = s;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        e = cudaLaunchKernelEx(&cfg, scored_merge_kernel<DV>, p, grid);
    }
    return e == cudaSuccess ? FA8_SUCCESS : host::cuda_fail(e, "scored attention kernel launch");
}

#define FA8_DEFINE_SCORED_MANY(D_, DV_)                                                                                            \
    template <>                                                                                                                    \
    fa8_status launch_scored_many<D_, DV_>(ScoredParams & p, const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv,  \
                                           int grid, int dev, cudaStream_t s) {                                                    \
        const int caps = p.cap_log2 > kFarCap ? kScFarCap : (p.cap_log2 > 0.f ? kScNearCap : kScNoCap);                            \
        if (p.slopes && caps == kScFarCap) return launch_scored_mode<D_, DV_, kScFarCap, true>(p, tq, tk, tv, grid, dev, s);       \
        if (p.slopes && caps == kScNearCap) return launch_scored_mode<D_, DV_, kScNearCap, true>(p, tq, tk, tv, grid, dev, s);     \
        if (p.slopes) return launch_scored_mode<D_, DV_, kScNoCap, true>(p, tq, tk, tv, grid, dev, s);                             \
        if (caps == kScFarCap) return launch_scored_mode<D_, DV_, kScFarCap, false>(p, tq, tk, tv, grid, dev, s);                  \
        if (caps == kScNearCap) return launch_scored_mode<D_, DV_, kScNearCap, false>(p, tq, tk, tv, grid, dev, s);                \
        return launch_scored_mode<D_, DV_, kScNoCap, false>(p, tq, tk, tv, grid, dev, s);                                          \
    }

}  // namespace fa8
