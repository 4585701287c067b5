// linear_tc.cu — linear attention with one decay per head on the tensor cores
// (bf16 data; steps 1 and 3 of linear.cu).
//
// k_linear_tc walks one segment of one head in chunks of 128 rows.  Per chunk
// (a, b, c: queries, keys, values; M: the incoming state, rows d_c, columns d_b;
// all products 128 x 128 x 128, fp32 accumulators in TMEM):
//   Sc = a b^T                    -> P_ij = s lambda^|i-j| Sc_ij on the causal side, bf16
//   O1 = a M^T,  O2 = P c         -> out_i = lambda^(i+1) O1_i + O2_i
//   Mu = c^T (w b)                -> M <- lambda^n M + Mu,  w_j = lambda^(n-1-j)
// O1 and O2 keep accumulators of their own because their rows decay
// differently, and a power of lambda below 1 cannot be divided out of a row.
// The state lives in fp32 registers of the state warps; only its copy as an
// operand of O1 is rounded to bf16.  w b is split into two bf16 parts, hi + lo,
// and Mu takes a product with each (c is exact in bf16): the update then
// carries 2^-17 per term instead of 2^-9, which the fp32 state is returned
// with.  P goes back to TMEM (A operand), over Sc.
//
// Bound: the tensor pipe needs five products (1.9 us at 11 TFLOP/s per SM) and
// the 128 KB in and out 3.0 us per chunk at 1/148 of the copy bandwidth, so the
// aim is to stream.  One CTA per SM, 18 warps, one thread each for TMA and MMA:
//   warps 0-7   P from Sc, outputs from O1 and O2 (row = TMEM lane, half the columns)
//   warps 8-15  hi + lo from b, the state
//   warp 16     TMA: b, a, c of each chunk into a ring of five 32 KB tiles
//   warp 17     MMA: Sc, O1, O2, Mu in this order, so that the next chunk's Sc
//               follows Mu while this chunk's outputs and state are drained
// hi overwrites b's tile (Sc has read it), lo and the bf16 state have a tile
// each: 7 x 32 KB.  Every wait is bounded (2 s): on expiry the status word is
// set and all roles leave.
//
// k_linear_state_tc is step 1: Mu alone over a whole segment, with
// w_j = lambda^(rows to the segment's end), accumulated in TMEM.
#include <cstring>

#include "linear.h"
#include "tc_ptx.cuh"

namespace gdn {
namespace tcg {

constexpr int kLtTile = kRows * kD * 2;                // one bf16 [2][128][64] operand: 32 KB
constexpr int kLtRing = 5;
constexpr int kLtThreads = 18 * 32;

struct LinTcArgs {
    CUtensorMap map[4];                                // the call's distinct tensors
    int8_t ia[kLinProblems], ib[kLinProblems], ic[kLinProblems];
    LinArgs a;
};

struct __align__(8) LtCtrl {
    uint64_t full[kLtRing], empty[kLtRing];
    uint64_t sc, p, split, o, drained, mu, state, drain;
    float pw[kRows];                                   // s_intra lambda^n
    float step[32];                                    // lambda^(31 - n), lambda^n if reverse
    uint32_t tmem;
    int abort;
};
constexpr int kLtSmem = 7 * kLtTile + (int)sizeof(LtCtrl);
static_assert(kLtSmem <= 232448, "shared memory budget");

// eight bf16 of one 16-byte group times w, as hi + lo
__device__ __forceinline__ void split8(const uint4& u, float w, uint4& hi, uint4& lo) {
    const uint32_t x[4] = {u.x, u.y, u.z, u.w};
    uint32_t h[4], l[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float a = __uint_as_float(x[i] << 16) * w;
        const float b = __uint_as_float(x[i] & 0xffff0000u) * w;
        h[i] = pack_b2(a, b);
        l[i] = pack_b2(a - __uint_as_float(h[i] << 16), b - __uint_as_float(h[i] & 0xffff0000u));
    }
    hi = make_uint4(h[0], h[1], h[2], h[3]);
    lo = make_uint4(l[0], l[1], l[2], l[3]);
}
// 32 values -> 16 TMEM columns of bf16 pairs
__device__ __forceinline__ void tmem_st_b16(uint32_t taddr, const float (&v)[32]) {
    uint32_t w[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = pack_b2(v[2 * i], v[2 * i + 1]);
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
        "%11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7]),
        "r"(w[8]), "r"(w[9]), "r"(w[10]), "r"(w[11]), "r"(w[12]), "r"(w[13]), "r"(w[14]),
        "r"(w[15])
        : "memory");
}
// 32 bytes, one whole sector
__device__ __forceinline__ void st_global32(void* p, const uint32_t (&w)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]),
                 "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}
__device__ __forceinline__ uint32_t lt_op_kmajor(uint32_t base, int kk) {
    return base + (kk >> 2) * (kRows * 128) + (kk & 3) * 32;
}

// rows n .. 127 of a tile become zero (this thread's row r, column half h)
__device__ __forceinline__ void zero_row(uint32_t tile, int r, int h) {
#pragma unroll
    for (int q = 0; q < 8; ++q) sts128(tile + op_off(r, 8 * h + q), make_uint4(0, 0, 0, 0));
}
// b's row r (column half h) times w into hi (in place) and lo; zero if off
__device__ __forceinline__ void split_row(uint32_t tile, uint32_t lo_tile, int r, int h, float w,
                                          bool on) {
#pragma unroll
    for (int q = 0; q < 8; ++q) {
        const uint32_t at = op_off(r, 8 * h + q);
        uint4 hi = make_uint4(0, 0, 0, 0), lo = hi;
        if (on) split8(lds128(tile + at), w, hi, lo);
        sts128(tile + at, hi);
        sts128(lo_tile + at, lo);
    }
}

__device__ __forceinline__ int lt_row0(const LinArgs& p, const LinSeg& g, int hv, int group) {
    const int64_t H = p.Hv / group;
    return (int)((g.b * H + hv / group) * p.T + g.t0);
}

// The bounded waits of one CTA.
struct LtWait {
    LtCtrl* c;
    int* status;
    __device__ bool live() const { return *(const volatile int*)&c->abort == 0; }
    __device__ bool operator()(uint64_t* b, uint32_t parity) const {
        if (!live()) return false;
        if (mbar_wait(b, parity)) return true;
        atomicExch(&c->abort, 1);
        raise_status(status, kStatusTimeout);
        return false;
    }
};

template <bool REV>
__device__ void lt_segment(const LinTcArgs& k, const LinProblem& q, const LinSeg& g, int hv,
                           uint8_t* smem, LtCtrl* ctrl) {
    const LinArgs& p = k.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const LtWait wait{ctrl, p.status};
    const int nch = (int)((g.n + kRows - 1) / kRows);
    const uint32_t tm = ctrl->tmem;
    const uint32_t tSc = tm, tO1 = tm + 128, tO2 = tm + 256, tMu = tm + 384;
    const uint32_t tiles = su32(smem), lo_tile = tiles + 5 * kLtTile, m_tile = tiles + 6 * kLtTile;
    const double lg = lin_log2(p.loggate, hv);
    // chunk number ci of the walk: its first row in the segment, its rows
    auto first_row = [&](int ci) { return (REV ? nch - 1 - ci : ci) * kRows; };
    auto rows_of = [&](int r0) { return (int)(g.n - r0 < kRows ? g.n - r0 : kRows); };
    // tile number 3 ci + {0: b, 1: a, 2: c} of the ring
    auto slot = [](int t) { return t % kLtRing; };
    auto phase = [](int t) { return (uint32_t)(t / kLtRing) & 1; };

    if (warp == 16) {
        if (lane == 0) {
            const int z = blockIdx.z;
            const CUtensorMap* mp[3] = {&k.map[k.ib[z]], &k.map[k.ia[z]], &k.map[k.ic[z]]};
            const int row[3] = {lt_row0(p, g, hv, q.gb), lt_row0(p, g, hv, q.ga),
                                lt_row0(p, g, hv, q.gc)};
            int t = 0;
            for (; t < 3 * nch; ++t) {
                const int s = slot(t), m = t % 3, y = row[m] + first_row(t / 3);
                if (t >= kLtRing && !wait(&ctrl->empty[s], phase(t) ^ 1)) break;
                if (!wait.live()) break;
                mbar_expect_tx(&ctrl->full[s], kLtTile);
                tma_load_2d(smem + s * kLtTile, mp[m], 0, y, &ctrl->full[s]);
                tma_load_2d(smem + s * kLtTile + kRows * 128, mp[m], 64, y, &ctrl->full[s]);
            }
            // whatever stopped the walk, copies in flight land before the CTA ends
            for (int i = t > kLtRing ? t - kLtRing : 0; i < t; ++i)
                mbar_wait(&ctrl->full[slot(i)], phase(i));
        }
    } else if (warp == 17) {
        if (lane == 0) {
            constexpr uint32_t idKK = idesc_f16(1, 0, 0, 128, 128);
            constexpr uint32_t idKM = idesc_f16(1, 0, 1, 128, 128);
            constexpr uint32_t idMM = idesc_f16(1, 1, 1, 128, 128);
            bool ok = true;
            for (int ci = 0; ci < nch && ok; ++ci) {
                const uint32_t par = ci & 1;
                const int tb = 3 * ci, ta = tb + 1, tc = tb + 2;
                const uint32_t sb = tiles + slot(tb) * kLtTile, sa = tiles + slot(ta) * kLtTile,
                               sv = tiles + slot(tc) * kLtTile;
                ok = wait(&ctrl->full[slot(tb)], phase(tb)) &&
                     wait(&ctrl->full[slot(ta)], phase(ta)) &&
                     (ci == 0 || wait(&ctrl->o, par ^ 1));         // P of the last chunk is read
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < 8; ++kk)
                    mma_ss(tSc, sdesc(lt_op_kmajor(sa, kk), 16, 1024),
                           sdesc(lt_op_kmajor(sb, kk), 16, 1024), idKK, kk > 0);
                mma_commit(&ctrl->sc);
                ok = wait(&ctrl->state, par) && (ci == 0 || wait(&ctrl->drained, par ^ 1));
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < 8; ++kk)
                    mma_ss(tO1, sdesc(lt_op_kmajor(sa, kk), 16, 1024),
                           sdesc(lt_op_kmajor(m_tile, kk), 16, 1024), idKK, kk > 0);
                mma_commit(&ctrl->empty[slot(ta)]);
                ok = wait(&ctrl->full[slot(tc)], phase(tc)) && wait(&ctrl->split, par) &&
                     wait(&ctrl->p, par);
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < 8; ++kk)
                    mma_ts(tO2, tSc + (kk >> 2) * 64 + (kk & 3) * 8,
                           sdesc(sv + kk * 2048, kRows * 128, 1024), idKM, kk > 0);
                mma_commit(&ctrl->o);
#pragma unroll
                for (int kk = 0; kk < 8; ++kk)
                    mma_ss(tMu, sdesc(sv + kk * 2048, kRows * 128, 1024),
                           sdesc(sb + kk * 2048, kRows * 128, 1024), idMM, kk > 0);
#pragma unroll
                for (int kk = 0; kk < 8; ++kk)
                    mma_ss(tMu, sdesc(sv + kk * 2048, kRows * 128, 1024),
                           sdesc(lo_tile + kk * 2048, kRows * 128, 1024), idMM, 1);
                mma_commit(&ctrl->mu);
                mma_commit(&ctrl->empty[slot(tb)]);
                mma_commit(&ctrl->empty[slot(tc)]);
            }
            mma_commit(&ctrl->drain);                  // nothing in flight when TMEM is freed
            mbar_wait(&ctrl->drain, 0);
        }
    } else if (warp < 8) {
        const int h = warp >> 2, quarter = warp & 3, r = quarter * 32 + lane;
        const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
        const int64_t orow = (g.b * p.Hv + hv) * p.T + g.t0;
        float din = REV ? 0.f : q.s_inter * lin_pow(lg, r + 1);
        int n_of_din = 0;
        for (int ci = 0; ci < nch; ++ci) {
            const uint32_t par = ci & 1;
            const int r0 = first_row(ci), n = rows_of(r0);
            if (!wait(&ctrl->sc, par)) break;
            tc_fence_after();
#pragma unroll
            for (int pc = 0; pc < 2; ++pc) {
                const int piece = 2 * h + pc, j0 = 32 * piece;
                const bool off = REV ? piece < quarter : piece > quarter;
                float v[32];
                if (off) {
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] = 0.f;
                } else {
                    tmem_ld32(tSc + lanes + j0, v);
                    if (piece == quarter || n < kRows) {           // the border: element by element
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            const int j = j0 + i, dist = REV ? j - r : r - j;
                            v[i] = dist >= 0 && j < n ? v[i] * ctrl->pw[dist & 127] : 0.f;
                        }
                    } else {
                        const float f = ctrl->pw[REV ? j0 - r : r - j0 - 31];
#pragma unroll
                        for (int i = 0; i < 32; i += 4) {
                            const float4 s = *reinterpret_cast<const float4*>(&ctrl->step[i]);
                            v[i] *= f * s.x;
                            v[i + 1] *= f * s.y;
                            v[i + 2] *= f * s.z;
                            v[i + 3] *= f * s.w;
                        }
                    }
                }
                tmem_st_b16(tSc + lanes + 64 * h + 16 * pc, v);
            }
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(&ctrl->p);
            if (REV && n != n_of_din) {
                din = r < n ? q.s_inter * lin_pow(lg, n - 1 - r) : 0.f;
                n_of_din = n;
            }
            if (!wait(&ctrl->o, par)) break;
            tc_fence_after();
            const int64_t at = (orow + r0 + r) * kD + 64 * h;
            if (q.out_f32) {
#pragma unroll
                for (int pc = 0; pc < 2; ++pc) {
                    float x[32], y[32];
                    tmem_ld2(tO1 + lanes + 64 * h + 32 * pc, x, tO2 + lanes + 64 * h + 32 * pc, y);
                    if (r < n)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            uint32_t w[8];
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                w[i] = __float_as_uint(fmaf(din, x[8 * e + i], y[8 * e + i]));
                            st_global32((float*)q.out + at + 32 * pc + 8 * e, w);
                        }
                }
                tc_fence_before();
                mbar_arrive(&ctrl->drained);
            } else {
                uint32_t w[4][8];
#pragma unroll
                for (int pc = 0; pc < 2; ++pc) {
                    float x[32], y[32];
                    tmem_ld2(tO1 + lanes + 64 * h + 32 * pc, x, tO2 + lanes + 64 * h + 32 * pc, y);
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        w[2 * pc + i / 8][i % 8] = pack_b2(fmaf(din, x[2 * i], y[2 * i]),
                                                           fmaf(din, x[2 * i + 1], y[2 * i + 1]));
                }
                tc_fence_before();
                mbar_arrive(&ctrl->drained);
                if (r < n)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        st_global32((__nv_bfloat16*)q.out + at + 16 * e, w[e]);
            }
        }
    } else {
        const int h = (warp - 8) >> 2, quarter = warp & 3, r = quarter * 32 + lane;
        const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
        float m[64];
        {   // the incoming state: this thread's row, 64 columns
            const bool first = REV ? g.k == g.m - 1 : g.k == 0;
            const float* src = nullptr;
            int rs = kD, cs = 1;
            if (!first) {
                src = q.ws + ((g.slot0 + (REV ? g.k : g.k - 1)) * p.Hv + hv) * kLinState;
            } else if (q.m0) {
                src = q.m0 + (g.seq * p.Hv + hv) * kLinState;
                if (q.m0_t) { rs = 1; cs = kD; }
            }
            if (!src) {
#pragma unroll
                for (int i = 0; i < 64; ++i) m[i] = 0.f;
            } else if (cs == 1) {
#pragma unroll
                for (int i = 0; i < 64; i += 4) {
                    const float4 f = *reinterpret_cast<const float4*>(src + r * rs + 64 * h + i);
                    m[i] = f.x; m[i + 1] = f.y; m[i + 2] = f.z; m[i + 3] = f.w;
                }
            } else {
#pragma unroll
                for (int i = 0; i < 64; ++i) m[i] = src[(64 * h + i) * kD + r];
            }
        }
        float w = 0.f, an = 0.f;
        int n_of_w = 0;
        bool ok = true;
        for (int ci = 0; ci <= nch; ++ci) {
            // the state as an operand (read by O1 of chunk ci; O1 of ci - 1 is done)
            if (ci < nch) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const uint4 u = make_uint4(pack_b2(m[8 * e], m[8 * e + 1]),
                                               pack_b2(m[8 * e + 2], m[8 * e + 3]),
                                               pack_b2(m[8 * e + 4], m[8 * e + 5]),
                                               pack_b2(m[8 * e + 6], m[8 * e + 7]));
                    sts128(m_tile + op_off(r, 8 * h + e), u);
                }
                fence_async_smem();
                tc_fence_before();
                mbar_arrive(&ctrl->state);
            }
            if (ci == nch) break;
            const uint32_t par = ci & 1;
            const int n = rows_of(first_row(ci));
            if (n != n_of_w) {
                w = q.s_state * lin_pow(lg, REV ? r + 1 : (r < n ? n - 1 - r : 0));
                an = lin_pow(lg, n);
                n_of_w = n;
            }
            const int tb = 3 * ci, tc = tb + 2;
            ok = wait(&ctrl->full[slot(tb)], phase(tb)) &&
                 wait(&ctrl->sc, par);                 // Sc has read b; Mu of ci - 1 has read lo
            if (!ok) break;
            split_row(tiles + slot(tb) * kLtTile, lo_tile, r, h, w, r < n);
            if (n < kRows) {                           // rows of others may hold NaN
                ok = wait(&ctrl->full[slot(tc)], phase(tc));
                if (!ok) break;
                if (r >= n) zero_row(tiles + slot(tc) * kLtTile, r, h);
            }
            fence_async_smem();
            mbar_arrive(&ctrl->split);
            ok = wait(&ctrl->mu, par);
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int pc = 0; pc < 2; ++pc) {
                float u[32];
                tmem_ld32(tMu + lanes + 64 * h + 32 * pc, u);
#pragma unroll
                for (int i = 0; i < 32; ++i) m[32 * pc + i] = fmaf(an, m[32 * pc + i], u[i]);
            }
        }
        if (ok && q.mout && (REV ? g.k == 0 : g.k == g.m - 1)) {
            float* dst = q.mout + (g.seq * p.Hv + hv) * kLinState + r * kD + 64 * h;
#pragma unroll
            for (int i = 0; i < 64; i += 4)
                *reinterpret_cast<float4*>(dst + i) = make_float4(m[i], m[i + 1], m[i + 2], m[i + 3]);
        }
    }
}

// grid: (segments, Hv, problems)
__global__ void __launch_bounds__(kLtThreads, 1) k_linear_tc(const __grid_constant__ LinTcArgs k) {
    extern __shared__ __align__(1024) uint8_t smem[];
    const LinArgs& p = k.a;
    if ((su32(smem) & 1023u) != 0) {
        if (threadIdx.x == 0) raise_status(p.status, kStatusSmemAlign);
        return;
    }
    const LinProblem& q = p.pr[blockIdx.z];
    const LinSeg g = lin_find(p, blockIdx.x, 0);
    if (!g.ok) return;
    const int hv = blockIdx.y, warp = threadIdx.x >> 5;
    LtCtrl* ctrl = reinterpret_cast<LtCtrl*>(smem + 7 * kLtTile);
    if (threadIdx.x == 0) {
        for (int i = 0; i < kLtRing; ++i) {
            mbar_init(&ctrl->full[i], 1);
            mbar_init(&ctrl->empty[i], 1);
        }
        mbar_init(&ctrl->sc, 1);
        mbar_init(&ctrl->p, 256);
        mbar_init(&ctrl->split, 256);
        mbar_init(&ctrl->o, 1);
        mbar_init(&ctrl->drained, 256);
        mbar_init(&ctrl->mu, 1);
        mbar_init(&ctrl->state, 256);
        mbar_init(&ctrl->drain, 1);
        ctrl->abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 17) tmem_alloc(&ctrl->tmem, 512);
    if (threadIdx.x < kRows + 32) {
        const double lg = lin_log2(p.loggate, hv);
        const int i = threadIdx.x;
        if (i < kRows) ctrl->pw[i] = q.s_intra * lin_pow(lg, i);
        else ctrl->step[i - kRows] = lin_pow(lg, q.reverse ? i - kRows : 31 - (i - kRows));
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (q.reverse) lt_segment<true>(k, q, g, hv, smem, ctrl);
    else lt_segment<false>(k, q, g, hv, smem, ctrl);
    tc_fence_before();
    __syncthreads();
    if (warp == 17) {
        tc_fence_after();
        tmem_dealloc(ctrl->tmem, 512);
    }
}

// ---- step 1: what a segment adds to the state ----
// Warps 0-7 split b, warp 8 loads, warp 9 multiplies.  Five ring tiles, two lo
// tiles, so that a chunk is split while the one before it is multiplied.
constexpr int kLsThreads = 10 * 32;
struct __align__(8) LsCtrl {
    uint64_t full[kLtRing], empty[kLtRing];
    uint64_t split[2], mu[2], drain;
    uint32_t tmem;
    int abort;
};
constexpr int kLsSmem = 7 * kLtTile + (int)sizeof(LsCtrl);

struct LsWait {
    LsCtrl* c;
    int* status;
    __device__ bool live() const { return *(const volatile int*)&c->abort == 0; }
    __device__ bool operator()(uint64_t* b, uint32_t parity) const {
        if (!live()) return false;
        if (mbar_wait(b, parity)) return true;
        atomicExch(&c->abort, 1);
        raise_status(status, kStatusTimeout);
        return false;
    }
};

// grid: (boundaries, Hv, problems)
__global__ void __launch_bounds__(kLsThreads, 1)
k_linear_state_tc(const __grid_constant__ LinTcArgs k) {
    extern __shared__ __align__(1024) uint8_t smem[];
    const LinArgs& p = k.a;
    if ((su32(smem) & 1023u) != 0) {
        if (threadIdx.x == 0) raise_status(p.status, kStatusSmemAlign);
        return;
    }
    const LinProblem& q = p.pr[blockIdx.z];
    LinSeg g = lin_find(p, blockIdx.x, 1);
    if (!g.ok) return;
    if (q.reverse) {                                   // boundary k: what segment k + 1 adds
        g.k += 1;
        g.t0 = g.seq_t0 + g.k * p.seg_len;
        g.n = g.seq_n - g.k * p.seg_len < p.seg_len ? g.seq_n - g.k * p.seg_len : p.seg_len;
    }
    const int hv = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    LsCtrl* ctrl = reinterpret_cast<LsCtrl*>(smem + 7 * kLtTile);
    if (threadIdx.x == 0) {
        for (int i = 0; i < kLtRing; ++i) {
            mbar_init(&ctrl->full[i], 1);
            mbar_init(&ctrl->empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&ctrl->split[i], 256);
            mbar_init(&ctrl->mu[i], 1);
        }
        mbar_init(&ctrl->drain, 1);
        ctrl->abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 9) tmem_alloc(&ctrl->tmem, 128);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = ctrl->tmem, tiles = su32(smem), lo_tile = tiles + 5 * kLtTile;
    const LsWait wait{ctrl, p.status};
    const int nch = (int)((g.n + kRows - 1) / kRows);
    auto slot = [](int t) { return t % kLtRing; };
    auto phase = [](int t) { return (uint32_t)(t / kLtRing) & 1; };
    if (warp == 8) {
        if (lane == 0) {
            const int z = blockIdx.z;
            const CUtensorMap* mp[2] = {&k.map[k.ib[z]], &k.map[k.ic[z]]};
            const int row[2] = {lt_row0(p, g, hv, q.gb), lt_row0(p, g, hv, q.gc)};
            int t = 0;
            for (; t < 2 * nch; ++t) {
                const int s = slot(t), y = row[t & 1] + (t >> 1) * kRows;
                if (t >= kLtRing && !wait(&ctrl->empty[s], phase(t) ^ 1)) break;
                if (!wait.live()) break;
                mbar_expect_tx(&ctrl->full[s], kLtTile);
                tma_load_2d(smem + s * kLtTile, mp[t & 1], 0, y, &ctrl->full[s]);
                tma_load_2d(smem + s * kLtTile + kRows * 128, mp[t & 1], 64, y, &ctrl->full[s]);
            }
            for (int i = t > kLtRing ? t - kLtRing : 0; i < t; ++i)
                mbar_wait(&ctrl->full[slot(i)], phase(i));
        }
    } else if (warp == 9) {
        if (lane == 0) {
            constexpr uint32_t idMM = idesc_f16(1, 1, 1, 128, 128);
            for (int ci = 0; ci < nch; ++ci) {
                const int tb = 2 * ci, tc = tb + 1;
                if (!wait(&ctrl->full[slot(tc)], phase(tc)) ||
                    !wait(&ctrl->split[ci & 1], (ci >> 1) & 1))
                    break;
                tc_fence_after();
                const uint32_t sb = tiles + slot(tb) * kLtTile, sv = tiles + slot(tc) * kLtTile,
                               sl = lo_tile + (ci & 1) * kLtTile;
#pragma unroll
                for (int kk = 0; kk < 8; ++kk)
                    mma_ss(tm, sdesc(sv + kk * 2048, kRows * 128, 1024),
                           sdesc(sb + kk * 2048, kRows * 128, 1024), idMM, ci > 0 || kk > 0);
#pragma unroll
                for (int kk = 0; kk < 8; ++kk)
                    mma_ss(tm, sdesc(sv + kk * 2048, kRows * 128, 1024),
                           sdesc(sl + kk * 2048, kRows * 128, 1024), idMM, 1);
                mma_commit(&ctrl->mu[ci & 1]);
                mma_commit(&ctrl->empty[slot(tb)]);
                mma_commit(&ctrl->empty[slot(tc)]);
            }
            mma_commit(&ctrl->drain);
            mbar_wait(&ctrl->drain, 0);
        }
    } else {
        const int h = warp >> 2, quarter = warp & 3, r = quarter * 32 + lane;
        const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
        const double lg = lin_log2(p.loggate, hv);
        bool ok = true;
        for (int ci = 0; ci < nch; ++ci) {
            const int tb = 2 * ci, tc = tb + 1, row = ci * kRows + r;
            const int n = (int)(g.n - ci * kRows < kRows ? g.n - ci * kRows : kRows);
            const float w =
                r < n ? q.s_state * lin_pow(lg, q.reverse ? row + 1 : g.n - 1 - row) : 0.f;
            ok = wait(&ctrl->full[slot(tb)], phase(tb)) &&
                 (ci < 2 || wait(&ctrl->mu[ci & 1], ((ci >> 1) & 1) ^ 1));
            if (!ok) break;
            split_row(tiles + slot(tb) * kLtTile, lo_tile + (ci & 1) * kLtTile, r, h, w, r < n);
            if (n < kRows) {
                ok = wait(&ctrl->full[slot(tc)], phase(tc));
                if (!ok) break;
                if (r >= n) zero_row(tiles + slot(tc) * kLtTile, r, h);
            }
            fence_async_smem();
            mbar_arrive(&ctrl->split[ci & 1]);
        }
        if (ok) ok = wait(&ctrl->mu[(nch - 1) & 1], ((nch - 1) >> 1) & 1);
        if (ok) {
            tc_fence_after();
            float* dst = q.ws + ((g.slot0 + (q.reverse ? g.k - 1 : g.k)) * p.Hv + hv) * kLinState +
                         r * kD + 64 * h;
#pragma unroll
            for (int pc = 0; pc < 2; ++pc) {
                float u[32];
                tmem_ld32(tm + lanes + 64 * h + 32 * pc, u);
#pragma unroll
                for (int i = 0; i < 32; i += 8) {
                    uint32_t x[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] = __float_as_uint(u[i + e]);
                    st_global32(dst + 32 * pc + i, x);
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tm, 128);
    }
}

}  // namespace tcg

// the distinct tensors of the call's problems, by pointer and heads
cudaError_t launch_linear_tc(const LinArgs& a, int nprob, const LinPlan& pl, bool states,
                             cudaStream_t st) {
    tcg::LinTcArgs k;
    memset(&k, 0, sizeof k);
    k.a = a;
    const void* seen[4] = {nullptr, nullptr, nullptr, nullptr};
    int group_of[4] = {0, 0, 0, 0}, count = 0;
    auto map_of = [&](const void* t, int group) -> int {
        for (int i = 0; i < count; ++i)
            if (seen[i] == t && group_of[i] == group) return i;
        if (count == 4 ||
            !tcg::map_kd(&k.map[count], t, a.B * (a.Hv / group) * (a.T > 0 ? a.T : 1)))
            return -1;
        seen[count] = t;
        group_of[count] = group;
        return count++;
    };
    if (a.T > 0)
        for (int i = 0; i < nprob; ++i) {
            const LinProblem& q = a.pr[i];
            const int ma = map_of(q.a, q.ga), mb = map_of(q.b, q.gb), mc = map_of(q.c, q.gc);
            if (ma < 0 || mb < 0 || mc < 0) return cudaErrorInvalidValue;
            k.ia[i] = (int8_t)ma;
            k.ib[i] = (int8_t)mb;
            k.ic[i] = (int8_t)mc;
        }
    cudaError_t e;
    if (states) {
        e = cudaFuncSetAttribute(tcg::k_linear_state_tc,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, tcg::kLsSmem);
        if (e != cudaSuccess) return e;
        tcg::k_linear_state_tc<<<dim3((unsigned)pl.bounds, (unsigned)a.Hv, nprob),
                                 tcg::kLsThreads, tcg::kLsSmem, st>>>(k);
    } else {
        e = cudaFuncSetAttribute(tcg::k_linear_tc, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 tcg::kLtSmem);
        if (e != cudaSuccess) return e;
        tcg::k_linear_tc<<<dim3((unsigned)pl.segs, (unsigned)a.Hv, nprob), tcg::kLtThreads,
                           tcg::kLtSmem, st>>>(k);
    }
    return cudaGetLastError();
}

}  // namespace gdn
