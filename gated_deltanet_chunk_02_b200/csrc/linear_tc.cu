// linear_tc.cu — linear attention with one decay per head on the tensor cores
// (bf16 data; steps 1 and 3 of linear.cu).
//
// k_linear_tc walks one segment of one head in chunks of 128 rows.  Per chunk
// (a, b, c: queries, keys, values; M: the incoming state, rows d_c, columns d_b;
// all products 128 x 128 x 128, fp32 accumulators in TMEM):
//   Sc = a b^T              -> P_ij = s lambda^|i-j| Sc_ij / d_i on the causal side, bf16
//   O  = a M^T + P c        -> out_i = s_out d_i O_i,  d_i = lambda^(i+1)
//   Mu = (w c)^T b          -> M <- lambda^n M + Mu,   w_j = lambda^(n-1-j)
// Both terms of an output share one accumulator: the row's decay d_i is taken
// out of its weights.  d_i stops at 2^-60, so that the weights stay in range;
// the state then reaches rows it should reach with less than 2^-60 with 2^-60,
// far below the rounding of anything it could matter to.
//
// The state lives in fp32 registers; only its copy as an operand of O is
// rounded to bf16, and so is P (each term of an output passes one rounding).
// b is exact in bf16 and w c is split into bf16 parts with a product each,
// smallest first: two parts (2^-16) where the state is only an operand later,
// three (exact) where it is returned or starts other segments.  Mu is added to
// the state in fp32 after every chunk: accumulation in TMEM rounds towards
// zero, and over a segment that alone would cost 1e-5.
//
// Bound: five products (2600 cycles of the tensor pipe) and 128 KB in and out
// per chunk (5600 cycles at 1/148 of the copy bandwidth), so the aim is to
// stream.  One CTA per SM, 19 warps:
//   warps 0-7   P from Sc, the parts of w c, the last chunk's outputs
//   warps 8-15  the state (lane = row, half the columns)
//   warp 16     TMA: b, a, c of each chunk into a ring of two chunks' tiles
//   warp 17     MMA: Sc, a M^T, P c, Mu
//   warp 18     TMA: outputs, staged in the tile of c
// P (over Sc) and the parts are A operands in TMEM, so shared memory holds the
// ring and the bf16 state alone and is read for B only.  The parts are made by
// ldmatrix, which transposes c on the way: a thread gets pairs of tokens of one
// column of c, a 32-bit column of A's row in TMEM (16x128b stores).  A third
// part lies in the columns of Sc that P leaves.
// What ruined first versions, at 8600 to 11000 cycles a chunk: unrolled loops
// (80 KB of code a chunk run at the rate it can be fetched), spilled registers
// (a reload is an L2 access, as shared memory leaves L1 no room), and products
// issued by a walk of one lane.  Every wait is bounded (2 s): on expiry the
// status word is set and all roles leave.
//
// k_linear_state_tc is step 1: the state part alone, always with three parts.
//
// One B200, bf16, graph replay: 65536 tokens of 16 heads in 9 segments a head:
// state pass 110 us (4.9 TB/s), outputs 197 us (5.4 TB/s), 315 us together
// (371 us in calls without a pause, where the power limit takes the clock from
// 1965 to 1560 MHz); batch 4 of 16 heads x 4096 tokens backward 199 us (223).
#include <cstddef>
#include <cstring>

#include "linear.h"
#include "tc_ptx.cuh"

namespace gdn {
namespace tcg {

constexpr int kLtTile = kRows * kD * 2;                // one bf16 [2][128][64] operand: 32 KB
constexpr int kLtRing = 6;
constexpr int kLtPart = 64;                            // TMEM columns of a part
constexpr int kLtThreads = 19 * 32;

struct LinTcArgs {
    CUtensorMap map[4];                                // the call's distinct inputs
    CUtensorMap out[kLinProblems];                     // bf16 outputs
    int8_t ia[kLinProblems], ib[kLinProblems], ic[kLinProblems];
    LinArgs a;
    unsigned long long limit_ns;                       // of a wait
    int withhold;                                      // tests: this block's last tile never comes
};

// A block's end without its work done: who has given up, and when to.
struct LtStop {
    unsigned long long limit_ns;
    int abort;
};

struct __align__(16) LtCtrl {
    uint64_t full[kLtRing], empty[kLtRing];
    uint64_t sc, p, parts, o, drained, mu, lo, state, staged[2], stored[2], drain;
    __align__(16) float pw[kRows];                     // s lambda^n
    __align__(16) float step[32];                      // lambda^(31 - n), lambda^n if reverse
    // by row, for whole chunks [0] and for the segment's last rows [1]: the
    // weight of c; and lambda^n as a sum of two floats
    float w[2][kRows];
    float d[kRows];                                    // of a whole chunk
    float an[2], an_lo[2], lambda;
    uint32_t tmem;
    LtStop stop;
    int odd;                                           // a state row ended as NaN
    __align__(16) int odd_from[kRows];                 // by column of c: lt_scan
};
constexpr int kLtSmem = (kLtRing + 1) * kLtTile + (int)sizeof(LtCtrl);
static_assert(kLtSmem <= 232448, "shared memory budget");
static_assert(offsetof(LtCtrl, step) % 16 == 0 && offsetof(LtCtrl, odd_from) % 16 == 0,
              "read 16 bytes at a time");

// Bounded wait; false once it ran out or another role's did.  The loop is a
// function of its own: a dozen copies of it would not leave the roles' code in
// the instruction cache.
__device__ __noinline__ bool lt_wait_long(uint64_t* b, uint32_t parity, LtStop* stop, int* status) {
    unsigned long long t0 = 0;
    for (int i = 0;; ++i) {
        if (mbar_try(b, parity)) return true;
        if ((i & 63) == 63) {
            if (*(volatile int*)&stop->abort) return false;
            const unsigned long long t = gtime();
            if (!t0) t0 = t;
            if (t - t0 > stop->limit_ns) break;
        }
    }
    atomicExch(&stop->abort, 1);
    raise_status(status, kStatusTimeout);
    return false;
}
// is the phase over? (mbar_try may hold the thread for a microsecond)
__device__ __forceinline__ bool mbar_test(uint64_t* b, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n"
        " selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok) : "r"(su32(b)), "r"(parity) : "memory");
    return ok != 0;
}
__device__ __forceinline__ bool lt_wait(uint64_t* b, uint32_t parity, LtStop* stop, int* status) {
    return mbar_try(b, parity) || lt_wait_long(b, parity, stop, status);
}
// the same for a whole warp, with one answer
__device__ __forceinline__ bool warp_wait(uint64_t* b, uint32_t parity, LtStop* stop, int* status) {
    return __all_sync(0xffffffffu, lt_wait(b, parity, stop, status));
}

// The upper 16 bits of both (truncated to bf16) as a pair, and what is left.
__device__ __forceinline__ uint32_t take_upper(F2& x) {
    float a, b;
    x.get(a, b);
    const uint32_t ua = __float_as_uint(a), ub = __float_as_uint(b);
    x = sub2(x, F2(__uint_as_float(ua & 0xffff0000u), __uint_as_float(ub & 0xffff0000u)));
    return __byte_perm(ua, ub, 0x7632);
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
// 16 lanes x 8 columns; thread t: lanes t / 4 (a0, b0) and t / 4 + 8 (a1, b1),
// columns t % 4 (a) and 4 + t % 4 (b)
__device__ __forceinline__ void tmem_st_16x128b(uint32_t taddr, uint32_t a0, uint32_t a1,
                                                uint32_t b0, uint32_t b1) {
    asm volatile("tcgen05.st.sync.aligned.16x128b.x2.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr),
                 "r"(a0), "r"(a1), "r"(b0), "r"(b1)
                 : "memory");
}
// One warp's share of the parts of w c: 32 columns of c (lanes of A) and the 64
// tokens from tok0 (32 columns of each part).  Truncation leaves 16, then 8
// bits, so that three parts are exact.  Tokens from n on are not the segment's
// and may hold anything: zero.
template <int PARTS>
__device__ __forceinline__ void split_c(uint32_t tile, int quarter, int tok0, int n,
                                        const float* w, uint32_t at_hi, uint32_t at_mid,
                                        uint32_t at_lo) {
    const int lane = threadIdx.x & 31;
#pragma unroll 1
    for (int t = 0; t < 64; t += 16) {
        uint32_t part[PARTS][2][4];                    // [part][eight tokens][eight columns of c]
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            uint32_t x[4];
            ldmatrix_x4_trans(
                tile + op_off(tok0 + t + 8 * j + (lane & 7), 4 * quarter + (lane >> 3)), x);
            const int tok = tok0 + t + 8 * j + 2 * (lane & 3);
            if (n < kRows) {
                const uint32_t keep = tok + 1 < n ? 0xffffffffu : (tok < n ? 0xffffu : 0u);
#pragma unroll
                for (int i = 0; i < 4; ++i) x[i] &= keep;
            }
            const float2 wt = *reinterpret_cast<const float2*>(w + tok);
            const F2 w2(wt.x, wt.y);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                F2 y = mul2(F2(__uint_as_float(x[i] << 16), __uint_as_float(x[i] & 0xffff0000u)),
                            w2);
#pragma unroll
                for (int e = 0; e < PARTS - 1; ++e) part[e][j][i] = take_upper(y);
                float a, b;
                y.get(a, b);
                part[PARTS - 1][j][i] = pack_b2(a, b);
            }
        }
#pragma unroll
        for (int e = 0; e < PARTS; ++e) {
            const uint32_t at = (e == 0 ? at_hi : (e == 1 ? at_mid : at_lo)) + t / 2;
            tmem_st_16x128b(at, part[e][0][0], part[e][0][1], part[e][1][0], part[e][1][1]);
            tmem_st_16x128b(at + (16u << 16), part[e][0][2], part[e][0][3], part[e][1][2],
                            part[e][1][3]);
        }
    }
}
// rows that are not the segment's, as an operand: zero (row r, columns 64 h ..)
__device__ __forceinline__ void zero_row(uint32_t tile, int r, int h) {
#pragma unroll 1
    for (int q = 0; q < 8; ++q) sts128(tile + op_off(r, 8 * h + q), make_uint4(0, 0, 0, 0));
}
// 32 columns as 16 TMEM columns of bf16 pairs
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&w)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
        "%11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7]),
        "r"(w[8]), "r"(w[9]), "r"(w[10]), "r"(w[11]), "r"(w[12]), "r"(w[13]), "r"(w[14]),
        "r"(w[15])
        : "memory");
}
// 32 bytes: one whole sector where the tensor starts on one (all of its rows
// then do), two stores of 16 where it has the 16 bytes of alignment that a call
// asks for and no more (128 packed sequences of 64 rows, 16 heads: 192 and 208 us)
__device__ __forceinline__ void st_global32(void* p, const uint32_t* w) {
    if ((reinterpret_cast<uintptr_t>(p) & 31) == 0) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p),
                     "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]),
                     "r"(w[7])
                     : "memory");
    } else {
        uint4* const q = reinterpret_cast<uint4*>(p);
        q[0] = make_uint4(w[0], w[1], w[2], w[3]);
        q[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
}
// one lane of a converged warp
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile(
        "{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(p));
    return p != 0;
}
// one arrival for the warp, behind what all its lanes did
__device__ __forceinline__ void warp_arrive(uint64_t* b, int lane) {
    __syncwarp();
    if (lane == 0) mbar_arrive(b);
}
// D (+)= A B over 128: both K-major in shared memory, or A in TMEM with B MN-major.
// A step of 16 is 32 bytes on in a K-major operand (64 columns to a half) and
// 2048 in an MN-major one.
__device__ __forceinline__ void mma_kk(uint32_t d, uint32_t a, uint32_t b) {
    const uint64_t da = sdesc(a, 16, 1024), db = sdesc(b, 16, 1024);
#pragma unroll
    for (int kk = 0; kk < 8; ++kk) {
        const uint32_t o = ((kk >> 2) * (kRows * 128) + (kk & 3) * 32) >> 4;
        mma_ss(d, da + o, db + o, idesc_f16(1, 0, 0, 128, 128), kk > 0);
    }
}
// D (+)= A B over 128 tokens, A in TMEM at a, its second half `half` columns on
__device__ __forceinline__ void mma_tm(uint32_t d, uint32_t a, uint32_t half, uint32_t b,
                                       bool fresh) {
    const uint64_t db = sdesc(b, kRows * 128, 1024);
#pragma unroll
    for (int kk = 0; kk < 8; ++kk)
        mma_ts(d, a + (kk >> 2) * half + (kk & 3) * 8, db + kk * 128, idesc_f16(1, 0, 1, 128, 128),
               !fresh || kk > 0);
}

__device__ __forceinline__ int lt_row0(const LinArgs& p, const LinSeg& g, int hv, int group) {
    const int64_t H = p.Hv / group;
    return (int)((g.b * H + hv / group) * p.T + g.t0);
}
// A place in the ring: counted on, as a division per tile costs a single
// thread more than the tile's products take to issue.
template <int N>
struct Ring {
    int slot = 0;
    uint32_t phase = 0;
    __device__ void next() {
        if (++slot == N) { slot = 0; phase ^= 1; }
    }
    __device__ uint32_t tile(uint32_t tiles) const { return tiles + slot * kLtTile; }
};
// Whatever stopped a walk after t tiles, copies in flight land before the CTA ends.
template <int N>
__device__ __forceinline__ void land(uint64_t* full, int t) {
    for (int i = t > N ? t - N : 0; i < t; ++i) mbar_wait(&full[i % N], (uint32_t)(i / N) & 1);
}

// row r (columns 64 h ..) of a state
__device__ __forceinline__ void store_state(float* dst, int r, int h, const float (&m)[64]) {
#pragma unroll
    for (int i = 0; i < 64; i += 8) {
        uint32_t w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = __float_as_uint(m[i + e]);
        st_global32(dst + r * kD + 64 * h + i, w);
    }
}
// M <- (a + a_lo) M + Mu: a's own rounding would add up over the chunks that a
// slow decay remembers
__device__ __forceinline__ void take_update(uint32_t mu, float a, float a_lo, float (&m)[64]) {
    const F2 a2(a, a), l2(a_lo, a_lo);
#pragma unroll
    for (int pc = 0; pc < 4; ++pc) {
        float u[16];
        tmem_ld16(mu + 16 * pc, u);
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
            float& x = m[16 * pc + i];
            float& y = m[16 * pc + i + 1];
            const F2 v(x, y);
            fma2(a2, v, fma2(l2, v, F2(u[i], u[i + 1]))).get(x, y);
        }
    }
}

// ---- the roles of k_linear_tc ----
struct LtWalk {                                        // chunks of a segment, in walking order
    int n, nch;
    bool rev;
    bool exact;                                        // the state is returned: three parts
    __device__ int first(int ci) const { return (rev ? nch - 1 - ci : ci) * kRows; }
    __device__ int rows(int r0) const { return n - r0 < kRows ? n - r0 : kRows; }
    // a row's place in walking order (rows that are not there have places too)
    __device__ int place(int ci, int r) const { return ci * kRows + (rev ? kRows - 1 - r : r); }
};

__device__ void lt_load(const LinTcArgs& k, const LinProblem& q, const LinSeg& g, int hv,
                        const LtWalk& wk, uint8_t* smem, LtCtrl* c) {
    const int z = g.z;
    const CUtensorMap *mb = &k.map[k.ib[z]], *ma = &k.map[k.ia[z]], *mc = &k.map[k.ic[z]];
    const int yb = lt_row0(k.a, g, hv, q.gb), ya = lt_row0(k.a, g, hv, q.ga),
              yc = lt_row0(k.a, g, hv, q.gc);
    const int tiles = 3 * wk.nch - (blockIdx.x == (unsigned)k.withhold);
    Ring<kLtRing> at;
    int t = 0, m = 0, r0 = wk.first(0);
    for (; t < tiles; ++t) {
        const int s = at.slot;
        if (t >= kLtRing && !lt_wait(&c->empty[s], at.phase ^ 1, &c->stop, k.a.status)) break;
        // c comes where the c of two chunks ago was, and after that chunk's outputs
        if (m == 2 && t >= kLtRing &&
            !lt_wait(&c->stored[t / 3 & 1], ((t / 3 - 2) >> 1) & 1, &c->stop, k.a.status))
            break;
        const CUtensorMap* mp = m == 0 ? mb : (m == 1 ? ma : mc);
        const int y = r0 + (m == 0 ? yb : (m == 1 ? ya : yc));
        mbar_expect_tx(&c->full[s], kLtTile);
        tma_load_2d(smem + s * kLtTile, mp, 0, y, &c->full[s]);
        tma_load_2d(smem + s * kLtTile + kRows * 128, mp, 64, y, &c->full[s]);
        at.next();
        if (++m == 3) { m = 0; r0 += wk.rev ? -kRows : kRows; }
    }
    land<kLtRing>(c->full, t);
}

// The whole warp walks and one lane issues: descriptors and addresses are then
// uniform values; in a walk of one lane each of them is moved to a uniform
// register first, and the eight steps of a product took 1500 cycles to issue.
__device__ void lt_multiply(const LtWalk& wk, uint32_t tiles, LtCtrl* c, int* status) {
    const uint32_t tSc = __shfl_sync(0xffffffffu, c->tmem, 0), tO = tSc + 128, tMu = tSc + 256;
    const uint32_t tPart = tSc + 384, m_tile = tiles + kLtRing * kLtTile;
    LtStop* const ab = &c->stop;
    const bool lead = elect_one();
    bool ahead = false;
    Ring<kLtRing> at;
#pragma unroll 1
    for (int ci = 0; ci < wk.nch; ++ci) {
        const uint32_t par = ci & 1;
        const Ring<kLtRing> b = at;
        at.next();
        const Ring<kLtRing> a = at;
        at.next();
        const Ring<kLtRing> v = at;
        at.next();
        const uint32_t sb = b.tile(tiles), sa = a.tile(tiles), sv = v.tile(tiles);
        if (!ahead) {
            if (!warp_wait(&c->full[b.slot], b.phase, ab, status) ||
                !warp_wait(&c->full[a.slot], a.phase, ab, status) ||
                // P of the last chunk has been read, and the third part beside it
                (ci > 0 && !warp_wait(wk.exact ? &c->mu : &c->o, par ^ 1, ab, status)))
                break;
            tc_fence_after();
            if (lead) {
                mma_kk(tSc, sa, sb);
                mma_commit(&c->sc);
            }
            __syncwarp();
        }
        if (!warp_wait(&c->state, par, ab, status) ||
            (ci > 0 && !warp_wait(&c->drained, par ^ 1, ab, status)))
            break;
        tc_fence_after();
        if (lead) {
            mma_kk(tO, sa, m_tile);
            mma_commit(&c->empty[a.slot]);
        }
        __syncwarp();
        // c's rows that are not the segment's are zero with the parts
        if (!warp_wait(&c->full[v.slot], v.phase, ab, status) ||
            !warp_wait(&c->p, par, ab, status) ||
            (wk.rows(wk.first(ci)) < kRows && !warp_wait(&c->parts, par, ab, status)))
            break;
        tc_fence_after();
        if (lead) {
            mma_tm(tO, tSc, 64, sv, false);
            mma_commit(&c->o);
        }
        __syncwarp();
        // the next Sc, if its tiles come while the parts are still made: the rows'
        // next work waits for it
        ahead = false;
        if (!wk.exact && ci + 1 < wk.nch) {
            Ring<kLtRing> a1 = at;
            a1.next();
            // (a look takes 50 cycles or more; after a million of them, 30 ms, the
            // wait for the parts below decides)
            for (int look = 0; look < (1 << 20) && !ahead &&
                               !__all_sync(0xffffffffu, mbar_test(&c->parts, par)); ++look) {
                ahead = __all_sync(0xffffffffu, mbar_test(&c->full[at.slot], at.phase) &&
                                                    mbar_test(&c->full[a1.slot], a1.phase) &&
                                                    mbar_test(&c->o, par));
                // another role's wait ran out
                if (__any_sync(0xffffffffu, *(volatile int*)&ab->abort)) break;
            }
            if (ahead) {
                tc_fence_after();
                if (lead) {
                    mma_kk(tSc, a1.tile(tiles), at.tile(tiles));
                    mma_commit(&c->sc);
                }
            }
            __syncwarp();
        }
        if (!warp_wait(&c->parts, par, ab, status)) break;
        tc_fence_after();
        if (wk.exact) {
            if (lead) {
                mma_tm(tMu, tSc + 32, 64, sb, true);   // lo
                mma_commit(&c->lo);
            }
            __syncwarp();
        }
        if (wk.exact && ci + 1 < wk.nch) {
            // the next Sc behind lo, which lies in its columns, if its tiles have
            // come (a sequence of 32 chunks: 114 us; behind hi 119, behind Mu 124)
            Ring<kLtRing> a1 = at;
            a1.next();
            ahead = __all_sync(0xffffffffu, mbar_test(&c->full[at.slot], at.phase) &&
                                                mbar_test(&c->full[a1.slot], a1.phase));
            if (ahead) {
                if (!warp_wait(&c->lo, par, ab, status)) break;
                tc_fence_after();
                if (lead) {
                    mma_kk(tSc, a1.tile(tiles), at.tile(tiles));
                    mma_commit(&c->sc);
                }
            }
            __syncwarp();
        }
        if (lead) {
            mma_tm(tMu, tPart + kLtPart, 32, sb, !wk.exact);       // mid
            mma_tm(tMu, tPart, 32, sb, false);                     // hi
            mma_commit(&c->mu);
            mma_commit(&c->empty[b.slot]);
            mma_commit(&c->empty[v.slot]);
        }
        __syncwarp();
    }
    if (lead) {
        mma_commit(&c->drain);                         // nothing in flight when TMEM is freed
        mbar_wait(&c->drain, 0);
    }
    __syncwarp();
}

// Half of one row's outputs from its accumulator: to the tile of c (which has
// been read; a's and b's are needed sooner), for the store warp; straight to memory where rows of the
// chunk are not the segment's, or in float32.  Direct stores of whole rows take
// the shared-memory pipe for 1000 cycles a chunk.
template <bool CAREFUL>
__device__ __forceinline__ void lt_output(uint32_t to, float d, int n, int r, int h, int64_t row,
                                          const LinProblem& q, uint32_t c_tile, LtCtrl* c,
                                          int chunk, int place) {
    const int lane = threadIdx.x & 31;
    uint32_t x[2][32];
    tmem_ld32_async(to, x[0]);
    tmem_ld32_async(to + 32, x[1]);
    tmem_wait_ld();
    tc_fence_before();
    warp_arrive(&c->drained, lane);
    if (CAREFUL) {
#pragma unroll
        for (int i = 0; i < 64; i += 4) {
            const int4 from = *reinterpret_cast<const int4*>(&c->odd_from[64 * h + i]);
            const int f[4] = {from.x, from.y, from.z, from.w};
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (place >= f[e]) x[(i + e) >> 5][(i + e) & 31] = 0x7fffffffu;
        }
    }
    const bool by_tma = n == kRows && !q.out_f32;
    const int64_t at = (row + r) * kD + 64 * h;
#pragma unroll
    for (int pc = 0; pc < 2; ++pc) {
#pragma unroll
        for (int i = 0; i < 32; ++i) x[pc][i] = __float_as_uint(d * __uint_as_float(x[pc][i]));
        if (q.out_f32) {
            if (r < n)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    st_global32((float*)q.out + at + 32 * pc + 8 * e, &x[pc][8 * e]);
            continue;
        }
        uint32_t w[16];
#pragma unroll
        for (int i = 0; i < 16; ++i)
            w[i] = pack_b2(__uint_as_float(x[pc][2 * i]), __uint_as_float(x[pc][2 * i + 1]));
        if (by_tma) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                sts128(c_tile + op_off(r, 8 * h + 4 * pc + e),
                       make_uint4(w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]));
        } else if (r < n) {
            st_global32((__nv_bfloat16*)q.out + at + 32 * pc, w);
            st_global32((__nv_bfloat16*)q.out + at + 32 * pc + 16, w + 8);
        }
    }
    fence_async_smem();
    warp_arrive(&c->staged[chunk & 1], lane);
}

// The store warp's lane: a chunk's staged outputs to memory; then c may come
// into their tile.
__device__ void lt_store(const LtWalk& wk, const LinProblem& q, const CUtensorMap* map, int row,
                         uint8_t* smem, LtCtrl* c, int* status) {
    Ring<kLtRing> at;
    for (int ci = 0; ci < wk.nch; ++ci) {
        at.next();
        at.next();
        const uint8_t* tile = smem + at.slot * kLtTile;
        at.next();
        const int r0 = wk.first(ci);
        if (!lt_wait(&c->staged[ci & 1], (ci >> 1) & 1, &c->stop, status)) break;
        if (wk.rows(r0) == kRows && !q.out_f32) {
            tma_store_2d(map, 0, row + r0, tile);
            tma_store_2d(map, 64, row + r0, tile + kRows * 128);
            bulk_commit();
            bulk_wait_read();
        }
        mbar_arrive(&c->stored[ci & 1]);
    }
    bulk_wait_all();
}

// An infinite or NaN value of c makes its column not a number from its row on,
// in walking order; rows before it do not see it.  But their weights for it,
// which are zero, would make NaN of it in P c.  So such values are zero for the
// product, and the places from which on their columns are lost are kept for the
// outputs and the state.  (An infinity is a NaN from here on: the split into
// parts makes one of it.)  Walks do so on their second turn only: a value that
// is not finite leaves NaN in its row of the state up to the end of a walk, which
// then is made again.  That the second turn is there costs ordinary data 2 %
// (packed 111 -> 113 us, backward 195 -> 199); scans of c in every walk, by the
// state's warps or by a warp of their own, cost 6 to 10 % (118 and 120, 215 and
// 213), as did tests for a second turn inside the roles.
__device__ __noinline__ void lt_scan(uint32_t tile, int r, int h, int place, LtCtrl* c) {
#pragma unroll 1
    for (int e = 8 * h; e < 8 * h + 8; ++e) {
        const uint4 u = lds128(tile + op_off(r, e));
        uint32_t w[4] = {u.x, u.y, u.z, u.w};
        bool found = false;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t half = i & 1 ? 0xffff0000u : 0xffffu, ones = half & 0x7f807f80u;
            if ((w[i >> 1] & ones) != ones) continue;
            w[i >> 1] &= ~half;
            found = true;
            atomicMin(&c->odd_from[8 * e + i], place);
        }
        if (found) sts128(tile + op_off(r, e), make_uint4(w[0], w[1], w[2], w[3]));
    }
    fence_async_smem();
}

template <bool CAREFUL>
__device__ __forceinline__ void lt_rows(const LinArgs& p, const LinProblem& q, const LinSeg& g, int hv,
                        const LtWalk& wk, uint32_t tiles, LtCtrl* c) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, h = warp >> 2, quarter = warp & 3;
    const int r = quarter * 32 + lane;
    const bool rev = wk.rev;
    const uint32_t tSc = c->tmem + ((uint32_t)(quarter * 32) << 16) + 64 * h, tO = tSc + 128;
    const int64_t orow = (g.b * p.Hv + hv) * p.T + g.t0;
    const float lam = c->lambda;
    float d = 0.f;
    const uint32_t tPart = c->tmem + ((uint32_t)(quarter * 32) << 16) + 384 + 32 * h;
    Ring<kLtRing> at;
    uint32_t c_tile = 0;
#pragma unroll 1
    for (int ci = 0; ci <= wk.nch; ++ci) {
        if (ci > 0) {                                  // the last chunk's outputs, while Mu is formed
            const int r0 = wk.first(ci - 1);
            // parts: the other warps have read c too
            if (!warp_wait(&c->parts, (ci - 1) & 1, &c->stop, p.status) ||
                !warp_wait(&c->o, (ci - 1) & 1, &c->stop, p.status))
                break;
            tc_fence_after();
            lt_output<CAREFUL>(tO, q.s_out * d, wk.rows(r0), r, h, orow + r0, q, c_tile, c,
                               ci - 1, wk.place(ci - 1, r));
        }
        if (ci < wk.nch) {
            const int n = wk.rows(wk.first(ci));
            d = c->d[rev ? min(r + kRows - n, kRows - 1) : r];
            const float inv = 1.f / d;
            if (!warp_wait(&c->sc, ci & 1, &c->stop, p.status)) break;
            tc_fence_after();
#pragma unroll 1
            for (int pc = 0; pc < 2; ++pc) {
                const int piece = 2 * h + pc, j0 = 32 * piece;
                uint32_t w[16];
                if (rev ? piece < quarter : piece > quarter) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) w[i] = 0;
                } else {
                    uint32_t v[32];
                    tmem_ld32_async(tSc + 32 * pc, v);
                    if (piece == quarter) {
                        // the border: 1, lambda, lambda^2, .. away from the diagonal
                        float t = 0.f;
                        const float one = q.s_weight * inv;
                        tmem_wait_ld();
                        if (!rev) {
#pragma unroll
                            for (int i = 31; i >= 0; --i) {
                                t = i == lane ? one : t * lam;
                                v[i] = i <= lane ? __float_as_uint(__uint_as_float(v[i]) * t) : 0u;
                            }
                        } else {
#pragma unroll
                            for (int i = 0; i < 32; ++i) {
                                t = i == lane ? one : t * lam;
                                v[i] = i >= lane && j0 + i < n
                                           ? __float_as_uint(__uint_as_float(v[i]) * t) : 0u;
                            }
                        }
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            w[i] = pack_b2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
                    } else {
                        const float f = c->pw[rev ? j0 - r : r - j0 - 31] * inv;
                        const F2 f2(f, f);
                        F2 s[16];
#pragma unroll
                        for (int i = 0; i < 16; i += 2) {
                            const float4 t = *reinterpret_cast<const float4*>(&c->step[2 * i]);
                            s[i] = mul2(F2(t.x, t.y), f2);
                            s[i + 1] = mul2(F2(t.z, t.w), f2);
                        }
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            float x, y;
                            mul2(F2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])), s[i])
                                .get(x, y);
                            v[2 * i] = __float_as_uint(x);
                            v[2 * i + 1] = __float_as_uint(y);
                        }
                        if (rev && n < kRows) {        // columns that are not the segment's rows
#pragma unroll
                            for (int i = 0; i < 32; ++i) v[i] = j0 + i < n ? v[i] : 0u;
                        }
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            w[i] = pack_b2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
                    }
                }
                tmem_st16(tSc + 16 * pc, w);           // behind the columns still to be read
            }
            tmem_wait_st();
            const Ring<kLtRing> b = at;
            at.next();
            at.next();
            const Ring<kLtRing> v = at;
            at.next();
            c_tile = v.tile(tiles);
            if (CAREFUL) {
                if (!warp_wait(&c->full[v.slot], v.phase, &c->stop, p.status)) break;
                if (r < n) lt_scan(c_tile, r, h, wk.place(ci, r), c);
            }
            tc_fence_before();
            warp_arrive(&c->p, lane);
            // the parts of w c, once the last chunk's have been read
            if (!warp_wait(&c->full[v.slot], v.phase, &c->stop, p.status) ||
                (ci > 0 && !warp_wait(&c->mu, (ci - 1) & 1, &c->stop, p.status)))
                break;
            tc_fence_after();
            const float* w = c->w[n < kRows];
            if (wk.exact)
                split_c<3>(v.tile(tiles), quarter, 64 * h, n, w, tPart, tPart + kLtPart, tSc + 32);
            else
                split_c<2>(v.tile(tiles), quarter, 64 * h, n, w, tPart, tPart + kLtPart, 0);
            if (n < kRows) {                           // rows of others may hold NaN
                if (!warp_wait(&c->full[b.slot], b.phase, &c->stop, p.status)) break;
                if (r >= n) {
                    zero_row(b.tile(tiles), r, h);
                    zero_row(v.tile(tiles), r, h);
                }
                fence_async_smem();
            }
            tmem_wait_st();
            tc_fence_before();
            warp_arrive(&c->parts, lane);
        }
    }
}

template <bool CAREFUL>
__device__ __forceinline__ void lt_state(const LinArgs& p, const LinProblem& q, const LinSeg& g, int hv,
                         const LtWalk& wk, uint32_t tiles, LtCtrl* c) {
    const int warp = (threadIdx.x >> 5) - 8, lane = threadIdx.x & 31, h = warp >> 2;
    const int r = (warp & 3) * 32 + lane;
    const uint32_t tMu = c->tmem + ((uint32_t)((warp & 3) * 32) << 16) + 256 + 64 * h;
    const uint32_t m_row = tiles + kLtRing * kLtTile + op_off(r, 8 * h);
    float m[64];
    {   // the incoming state
        const bool first = wk.rev ? g.k == g.m - 1 : g.k == 0;
        const float* src = nullptr;
        bool across = false;
        if (!first) {
            src = lin_boundary(q, g, wk.rev ? g.k : g.k - 1);
            across = q.ws_t != 0;
        } else if (q.m0) {
            src = q.m0 + (g.seq * p.Hv + hv) * kLinState;
            across = q.m0_t != 0;
        }
        if (!src) {
#pragma unroll
            for (int i = 0; i < 64; ++i) m[i] = 0.f;
        } else if (across) {
#pragma unroll
            for (int i = 0; i < 64; ++i) m[i] = src[(64 * h + i) * kD + r];
        } else {
#pragma unroll
            for (int i = 0; i < 64; i += 4) {
                const float4 f = *reinterpret_cast<const float4*>(src + r * kD + 64 * h + i);
                m[i] = f.x; m[i + 1] = f.y; m[i + 2] = f.z; m[i + 3] = f.w;
            }
        }
    }
#pragma unroll 1
    for (int ci = 0; ci < wk.nch; ++ci) {
        // the state as an operand of chunk ci; the last one has been read
#pragma unroll
        for (int e = 0; e < 8; ++e)
            sts128(m_row ^ (e << 4),
                   make_uint4(pack_b2(m[8 * e], m[8 * e + 1]), pack_b2(m[8 * e + 2], m[8 * e + 3]),
                              pack_b2(m[8 * e + 4], m[8 * e + 5]),
                              pack_b2(m[8 * e + 6], m[8 * e + 7])));
        fence_async_smem();
        tc_fence_before();
        warp_arrive(&c->state, lane);
        if (!warp_wait(&c->mu, ci & 1, &c->stop, p.status)) return;
        tc_fence_after();
        const int part = wk.rows(wk.first(ci)) < kRows;
        take_update(tMu, c->an[part], c->an_lo[part], m);
        if (CAREFUL && c->odd_from[r] < (ci + 1) * kRows)
#pragma unroll
            for (int i = 0; i < 64; ++i) m[i] = __uint_as_float(0x7fffffffu);
    }
    if (isnan(m[0])) c->odd = 1;
    if (wk.exact && q.mout)
        store_state(q.mout + (g.seq * p.Hv + hv) * kLinState, r, h, m);
}

// ---- short sequences ----
// Up to kLtShort rows go token by token on the CUDA cores, as in decoding: the
// state in registers (thread: state row v, every fourth group of four columns),
// everything in fp32.  32 heads: 6.6 us for one row, 12.4 for 8, 16.1 for 12; a
// chunk on the tensor cores takes 14.4 whatever its rows.
constexpr int kLtShort = 8;

__device__ __forceinline__ void ld4(const __nv_bfloat16* p, float (&x)[4]) {
    const uint2 u = __ldg(reinterpret_cast<const uint2*>(p));
    x[0] = __uint_as_float(u.x << 16); x[1] = __uint_as_float(u.x & 0xffff0000u);
    x[2] = __uint_as_float(u.y << 16); x[3] = __uint_as_float(u.y & 0xffff0000u);
}

__device__ void lt_short(const LinArgs& p, const LinProblem& q, const LinSeg& g, int hv) {
    if (threadIdx.x >= 512) return;                    // 16 whole warps
    const int v = threadIdx.x >> 2, sub = threadIdx.x & 3, n = (int)g.n;
    const bool rev = q.reverse != 0;
    const float lg = p.loggate[hv];
    float m[8][4];
    {
        const float* src = q.m0 ? q.m0 + (g.seq * p.Hv + hv) * kLinState : nullptr;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int c0 = 16 * e + 4 * sub;
            if (!src) {
#pragma unroll
                for (int i = 0; i < 4; ++i) m[e][i] = 0.f;
            } else if (q.m0_t) {
#pragma unroll
                for (int i = 0; i < 4; ++i) m[e][i] = src[(c0 + i) * kD + v];
            } else {
                const float4 f = *reinterpret_cast<const float4*>(src + v * kD + c0);
                m[e][0] = f.x; m[e][1] = f.y; m[e][2] = f.z; m[e][3] = f.w;
            }
        }
    }
    const __nv_bfloat16* a =
        (const __nv_bfloat16*)q.a + (int64_t)lt_row0(p, g, hv, q.ga) * kD + 4 * sub;
    const __nv_bfloat16* b =
        (const __nv_bfloat16*)q.b + (int64_t)lt_row0(p, g, hv, q.gb) * kD + 4 * sub;
    const __nv_bfloat16* c = (const __nv_bfloat16*)q.c + (int64_t)lt_row0(p, g, hv, q.gc) * kD + v;
    const int64_t out = ((g.b * p.Hv + hv) * p.T + g.t0) * kD + v;
    float lam, lam_lo;
    lin_decay(lg, lam, lam_lo);
    const float before = rev ? 1.f : lam, before_lo = rev ? 0.f : lam_lo;
    for (int t = 0; t < n; ++t) {
        const int64_t at = (int64_t)(rev ? n - 1 - t : t) * kD;
        const float w = q.s_state * __bfloat162float(c[at]);
        float o = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float x[4], y[4];
            ld4(a + at + 16 * e, x);
            ld4(b + at + 16 * e, y);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                m[e][i] = fmaf(before, m[e][i], fmaf(before_lo, m[e][i], w * y[i]));
                o = fmaf(m[e][i], x[i], o);
                if (rev) m[e][i] = fmaf(lam, m[e][i], lam_lo * m[e][i]);
            }
        }
        o += __shfl_xor_sync(0xffffffffu, o, 1);
        o += __shfl_xor_sync(0xffffffffu, o, 2);
        if (sub == 0) {
            if (q.out_f32) static_cast<float*>(q.out)[out + at] = q.s_out * o;
            else st_elem(static_cast<__nv_bfloat16*>(q.out), out + at, q.s_out * o);
        }
    }
    if (q.mout) {
        float* dst = q.mout + (g.seq * p.Hv + hv) * kLinState + v * kD + 4 * sub;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            *reinterpret_cast<float4*>(dst + 16 * e) =
                make_float4(m[e][0], m[e][1], m[e][2], m[e][3]);
    }
}

__device__ __forceinline__ void lt_barriers(LtCtrl* c) {
    for (int i = 0; i < kLtRing; ++i) {
        mbar_init(&c->full[i], 1);
        mbar_init(&c->empty[i], 1);
    }
    mbar_init(&c->sc, 1);
    mbar_init(&c->p, 8);
    mbar_init(&c->parts, 8);
    mbar_init(&c->o, 1);
    mbar_init(&c->drained, 8);
    mbar_init(&c->mu, 1);
    mbar_init(&c->lo, 1);
    mbar_init(&c->state, 8);
    for (int i = 0; i < 2; ++i) {
        mbar_init(&c->staged[i], 8);
        mbar_init(&c->stored[i], 1);
    }
    mbar_init(&c->drain, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}

// one walk of the segment by all roles
template <bool CAREFUL>
__device__ __forceinline__ void lt_turn(const LinTcArgs& k, const LinProblem& q, const LinSeg& g,
                                        const LtWalk& wk, uint8_t* smem, LtCtrl* c) {
    const LinArgs& p = k.a;
    const uint32_t tiles = su32(smem);
    const int hv = g.hv, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (warp < 8) {
        lt_rows<CAREFUL>(p, q, g, hv, wk, tiles, c);
    } else if (warp < 16) {
        lt_state<CAREFUL>(p, q, g, hv, wk, tiles, c);
    } else if (warp == 16) {
        if (lane == 0) lt_load(k, q, g, hv, wk, smem, c);
    } else if (warp == 17) {
        lt_multiply(wk, tiles, c, p.status);
    } else if (lane == 0) {
        lt_store(wk, q, &k.out[g.z], (int)((g.b * p.Hv + hv) * p.T + g.t0), smem, c, p.status);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
}

__device__ __forceinline__ LtWalk lt_walk(const LinSeg& g, const LinProblem& q) {
    return {(int)g.n, (int)((g.n + kRows - 1) / kRows), q.reverse != 0,
            // a sequence of several segments has its outgoing state from steps 1
            // and 2; whether one is asked for changes no output
            g.m == 1 && q.has_state};
}

// The walk's second turn (see lt_scan), behind all copies, products and arrivals
// of the first.  It finds its segment again: anything that the first turn kept
// for it would be spilled there (backward 203 us).  TMEM is still held, as a CTA
// allocates once, and freed here.
__device__ __noinline__ void lt_again(const LinTcArgs& k) {
    extern __shared__ __align__(1024) uint8_t smem[];
    LtCtrl* c = reinterpret_cast<LtCtrl*>(smem + (kLtRing + 1) * kLtTile);
    const LinSeg g = lin_find(k.a, blockIdx.x, kAllSegments,
                              *reinterpret_cast<LinFound*>(smem + kLtRing * kLtTile));
    const LinProblem& q = k.a.pr[g.z];
    const LtWalk wk = lt_walk(g, q);
    if (threadIdx.x == 0) {
        land<kLtRing>(c->empty, 3 * wk.nch);
        if (wk.exact) mbar_wait(&c->lo, (wk.nch - 1) & 1);
        for (uint64_t* b = c->full; b <= &c->drain; ++b)
            asm volatile("mbarrier.inval.shared::cta.b64 [%0];" ::"r"(su32(b)) : "memory");
        lt_barriers(c);
    }
    __syncthreads();
    tc_fence_after();
    lt_turn<true>(k, q, g, wk, smem, c);
    if (threadIdx.x >> 5 == 17) {
        tc_fence_after();
        tmem_dealloc(c->tmem, 512);
    }
}

// one block for each of lin_find's
__global__ void __launch_bounds__(kLtThreads, 1) k_linear_tc(const __grid_constant__ LinTcArgs k) {
    extern __shared__ __align__(1024) uint8_t smem[];
    const LinArgs& p = k.a;
    if ((su32(smem) & 1023u) != 0) {
        if (threadIdx.x == 0) raise_status(p.status, kStatusSmemAlign);
        return;
    }
    LtCtrl* c = reinterpret_cast<LtCtrl*>(smem + (kLtRing + 1) * kLtTile);
    // (its place is the state's tile, which no copy writes)
    const LinSeg g = lin_find(p, blockIdx.x, kAllSegments,
                              *reinterpret_cast<LinFound*>(smem + kLtRing * kLtTile));
    if (!g.ok) return;
    const LinProblem& q = p.pr[g.z];
    if (g.m == 1 && g.n <= kLtShort) {
        lt_short(p, q, g, g.hv);
        return;
    }
    const int hv = g.hv, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        lt_barriers(c);
        c->stop = {k.limit_ns, 0};
        c->odd = 0;
    }
    if (warp == 17) tmem_alloc(&c->tmem, 512);
    const LtWalk wk = lt_walk(g, q);
    {
        const double lg = lin_log2(p.loggate, hv);
        const int t = threadIdx.x, i = t % kRows, n1 = wk.n - (wk.nch - 1) * kRows;
        if (t < 2 * kRows) {
            const int n = t < kRows ? kRows : n1;
            c->w[t / kRows][i] = i < n ? q.s_state * lin_pow(lg, wk.rev ? i + 1 : n - 1 - i) : 0.f;
        } else if (t < 3 * kRows) {
            const float d = lin_pow(lg, wk.rev ? kRows - 1 - i : i + 1);
            c->d[i] = d < 0x1p-60f ? 0x1p-60f : d;     // NaN stays
        } else if (t < 4 * kRows) {
            c->odd_from[i] = 0x7fffffff;               // never
        } else if (i < 32) {
            c->step[i] = lin_pow(lg, wk.rev ? i : 31 - i);
        } else if (i < 34) {
            lin_pow2(lg, i == 32 ? kRows : n1, c->an[i - 32], c->an_lo[i - 32]);
        } else if (i == 34) {
            c->lambda = lin_pow(lg, 1);
        }
        if (t < kRows) c->pw[t] = q.s_weight * lin_pow(lg, t);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    lt_turn<false>(k, q, g, wk, smem, c);
    if (c->odd && !c->stop.abort) {
        lt_again(k);
        return;
    }
    if (warp == 17) {
        tc_fence_after();
        tmem_dealloc(c->tmem, 512);
    }
}

// ---- step 1: what a segment adds to the state ----
// As in k_linear_tc without rows, so that all seven tiles are the ring's and the
// parts have two buffers.  With the parts (of b) in shared memory a chunk's had
// to wait for the last chunk's products: 5000 cycles a chunk.
//   warps 0-7   the parts of c (32 rows of A, half the tokens), two buffers
//   warps 8-15  the state, in registers
//   warp 16     TMA: b, c of each chunk;   warp 17  MMA
constexpr int kLsThreads = 18 * 32;
constexpr int kLsRing = 7;
struct __align__(16) LsCtrl {
    uint64_t full[kLsRing], empty[kLsRing];
    uint64_t parts[2], read[2], mu, taken, drain;
    __align__(16) float w[2][kRows];                   // as in LtCtrl
    float an[2], an_lo[2];
    LinFound found;
    uint32_t tmem;
    LtStop stop;
};
constexpr int kLsSmem = kLsRing * kLtTile + (int)sizeof(LsCtrl);
static_assert(kLsSmem <= 232448, "shared memory budget");

// one block for each of lin_find's, of the sequences that are cut
__global__ void __launch_bounds__(kLsThreads, 1)
k_linear_state_tc(const __grid_constant__ LinTcArgs k) {
    extern __shared__ __align__(1024) uint8_t smem[];
    const LinArgs& p = k.a;
    if ((su32(smem) & 1023u) != 0) {
        if (threadIdx.x == 0) raise_status(p.status, kStatusSmemAlign);
        return;
    }
    LsCtrl* c = reinterpret_cast<LsCtrl*>(smem + kLsRing * kLtTile);
    const LinSeg g = lin_find(p, blockIdx.x, kCutSegments, c->found);
    if (!g.ok) return;
    const LinProblem& q = p.pr[g.z];
    if (q.ws_t) return;
    const int hv = g.hv, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float* const dst = lin_added(p, q, g);
    if (!dst) return;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kLsRing; ++i) {
            mbar_init(&c->full[i], 1);
            mbar_init(&c->empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&c->parts[i], 8);
            mbar_init(&c->read[i], 1);
        }
        mbar_init(&c->mu, 1);
        mbar_init(&c->taken, 8);
        mbar_init(&c->drain, 1);
        c->stop = {k.limit_ns, 0};
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 17) tmem_alloc(&c->tmem, 512);
    const LtWalk wk{(int)g.n, (int)((g.n + kRows - 1) / kRows), q.reverse != 0, true};
    {
        const double lg = lin_log2(p.loggate, hv);
        const int t = threadIdx.x, i = t % kRows, n1 = wk.n - (wk.nch - 1) * kRows;
        if (t < 2 * kRows) {
            const int n = t < kRows ? kRows : n1;
            c->w[t / kRows][i] = i < n ? q.s_state * lin_pow(lg, wk.rev ? i + 1 : n - 1 - i) : 0.f;
        } else if (t < 2 * kRows + 2) {
            lin_pow2(lg, i == 0 ? kRows : n1, c->an[i], c->an_lo[i]);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // TMEM: Mu, then two sets of hi, mid, lo
    const uint32_t tm = c->tmem, tiles = su32(smem), tPart = tm + 128;
    LtStop* const ab = &c->stop;
    if (warp == 16) {
        if (lane == 0) {
            const int z = g.z;
            const CUtensorMap *mb = &k.map[k.ib[z]], *mc = &k.map[k.ic[z]];
            const int yb = lt_row0(p, g, hv, q.gb), yc = lt_row0(p, g, hv, q.gc);
            Ring<kLsRing> at;
            int t = 0, r0 = wk.first(0);
            const int tiles = 2 * wk.nch - (blockIdx.x == (unsigned)k.withhold);
            for (; t < tiles; ++t) {              // c first: its parts are made of it
                const int s = at.slot, y = r0 + (t & 1 ? yb : yc);
                if (t >= kLsRing && !lt_wait(&c->empty[s], at.phase ^ 1, ab, p.status)) break;
                mbar_expect_tx(&c->full[s], kLtTile);
                tma_load_2d(smem + s * kLtTile, t & 1 ? mb : mc, 0, y, &c->full[s]);
                tma_load_2d(smem + s * kLtTile + kRows * 128, t & 1 ? mb : mc, 64, y, &c->full[s]);
                at.next();
                if (t & 1) r0 += wk.rev ? -kRows : kRows;
            }
            land<kLsRing>(c->full, t);
        }
    } else if (warp == 17) {
        const bool lead = elect_one();
        const uint32_t td = __shfl_sync(0xffffffffu, tm, 0);
        Ring<kLsRing> at;
#pragma unroll 1
        for (int ci = 0; ci < wk.nch; ++ci) {
            const Ring<kLsRing> v = at;
            at.next();
            const Ring<kLsRing> b = at;
            at.next();
            if (!warp_wait(&c->full[b.slot], b.phase, ab, p.status) ||
                !warp_wait(&c->parts[ci & 1], (ci >> 1) & 1, ab, p.status) ||
                (ci > 0 && !warp_wait(&c->taken, (ci - 1) & 1, ab, p.status)))
                break;
            tc_fence_after();
            const uint32_t sb = b.tile(tiles), pt = td + 128 + (ci & 1) * 3 * kLtPart;
            if (lead) {
                mma_tm(td, pt + 2 * kLtPart, 32, sb, true);        // lo
                mma_tm(td, pt + kLtPart, 32, sb, false);
                mma_tm(td, pt, 32, sb, false);                     // hi
                mma_commit(&c->mu);
                mma_commit(&c->read[ci & 1]);
                mma_commit(&c->empty[v.slot]);
                mma_commit(&c->empty[b.slot]);
            }
            __syncwarp();
        }
        if (lead) {
            mma_commit(&c->drain);
            mbar_wait(&c->drain, 0);
        }
    } else if (warp < 8) {
        const int quarter = warp & 3, tok0 = 64 * (warp >> 2);
        Ring<kLsRing> at;
#pragma unroll 1
        for (int ci = 0; ci < wk.nch; ++ci) {
            const int n = wk.rows(wk.first(ci));
            const Ring<kLsRing> v = at;
            at.next();
            const Ring<kLsRing> b = at;
            at.next();
            if (!warp_wait(&c->full[v.slot], v.phase, ab, p.status) ||
                (ci > 1 && !warp_wait(&c->read[ci & 1], ((ci >> 1) & 1) ^ 1, ab, p.status)))
                break;
            tc_fence_after();
            const uint32_t pt = tPart + (ci & 1) * 3 * kLtPart + ((uint32_t)(quarter * 32) << 16) +
                                tok0 / 2;
            split_c<3>(v.tile(tiles), quarter, tok0, n, c->w[n < kRows], pt, pt + kLtPart,
                       pt + 2 * kLtPart);
            if (n < kRows) {
                const int r = (warp & 3) * 32 + lane;
                if (!warp_wait(&c->full[b.slot], b.phase, ab, p.status)) break;
                if (r >= n) zero_row(b.tile(tiles), r, warp >> 2);
                fence_async_smem();
            }
            tmem_wait_st();
            tc_fence_before();
            warp_arrive(&c->parts[ci & 1], lane);
        }
    } else {
        const int h = (warp - 8) >> 2, r = (warp & 3) * 32 + lane;
        const uint32_t tMu = tm + ((uint32_t)((warp & 3) * 32) << 16) + 64 * h;
        float m[64];
#pragma unroll
        for (int i = 0; i < 64; ++i) m[i] = 0.f;
        bool ok = true;
#pragma unroll 1
        for (int ci = 0; ci < wk.nch && ok; ++ci) {
            const int part = wk.rows(wk.first(ci)) < kRows;
            ok = warp_wait(&c->mu, ci & 1, ab, p.status);
            if (!ok) break;
            tc_fence_after();
            take_update(tMu, c->an[part], c->an_lo[part], m);
            tc_fence_before();
            warp_arrive(&c->taken, lane);
        }
        if (ok) store_state(dst, r, h, m);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 17) {
        tc_fence_after();
        tmem_dealloc(tm, 512);
    }
}

}  // namespace tcg

// tests of the bounded waits (gdn_debug_arm_linear_expiry): the next launch of
// one kernel on this thread withholds a block's last tile
static thread_local int t_withhold = -1;
static thread_local bool t_withhold_states = false;
static thread_local unsigned long long t_withhold_ns = 0;

void arm_linear_expiry(int block, bool states, unsigned long long limit_ns) {
    t_withhold = block;
    t_withhold_states = states;
    t_withhold_ns = limit_ns;
}

// the distinct tensors of the call's problems, by pointer and heads
cudaError_t launch_linear_tc(const LinArgs& a, int nprob, const LinPlan& pl, bool states,
                             cudaStream_t st) {
    tcg::LinTcArgs k;
    memset(&k, 0, sizeof k);
    k.a = a;
    k.limit_ns = tcg::kTimeoutNs;
    k.withhold = -1;
    if (t_withhold >= 0 && t_withhold_states == states) {
        k.withhold = t_withhold;
        k.limit_ns = t_withhold_ns;
        t_withhold = -1;
    }
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
    if (a.T > 0 && !states)
        for (int i = 0; i < nprob; ++i)
            if (!a.pr[i].out_f32 && !tcg::map_kd(&k.out[i], a.pr[i].out, a.B * a.Hv * a.T))
                return cudaErrorInvalidValue;
    cudaError_t e;
    if (states) {
        e = cudaFuncSetAttribute(tcg::k_linear_state_tc,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, tcg::kLsSmem);
        if (e != cudaSuccess) return e;
        tcg::k_linear_state_tc<<<(unsigned)pl.cut_blocks,
                                 tcg::kLsThreads, tcg::kLsSmem, st>>>(k);
    } else {
        e = cudaFuncSetAttribute(tcg::k_linear_tc, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 tcg::kLtSmem);
        if (e != cudaSuccess) return e;
        tcg::k_linear_tc<<<(unsigned)pl.blocks, tcg::kLtThreads,
                           tcg::kLtSmem, st>>>(k);
    }
    return cudaGetLastError();
}

}  // namespace gdn
