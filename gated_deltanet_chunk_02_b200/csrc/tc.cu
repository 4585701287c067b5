// tc.cu — tcgen05 tensor-core kernels of libgdn (sm_100a).
//
// One persistent kernel template serves the bf16 chunk pipeline in seven
// modes: the fused inverse + WY step (on prepared inputs, or with the key
// normalisation and gate sums in front), A alone, WY alone, and three
// standalone inverses (the Neumann series with its residual, the sequential
// correction, the block decomposition).  Design:
//
// * A "tile" is 128 consecutive rows of the flattened [B*H*T, d] arrays, i.e.
//   128/KB blocks of KB tokens (KB = 64 or 128; chunks of k = 32 run as 64-token
//   blocks holding two chunks block-diagonally).  Every k x k product of the
//   method is ONE M=128 tcgen05.mma over the tile: the left operand stacks the
//   tile's blocks along M, the right operand places them side by side along N,
//   and each row reads only its own diagonal block of the 128 x 128 fp32
//   accumulator in tensor memory (TMEM).
// * Each "slot" of 8 warps owns one tile at a time.  Its elected thread issues
//   the tile's TMA loads (K with beta and g on one barrier, V on another, so
//   the K K^T product starts before V lands; in the standalone inverse, A one
//   tile ahead), its MMAs and its TMA stores.  Its 256 threads run the
//   epilogues (TMEM -> registers -> mask / accumulate / convert -> TMEM or
//   swizzled shared-memory operand).  Thread (r, h) owns row r of the tile
//   (its TMEM lane; the lane quarter is warp % 4) and the column half h.  The
//   series runs in Horner form with the left operand in TMEM; T0 sits in TMEM
//   at KB = 64 and in registers at KB = 128.  Two slots per CTA keep the
//   tensor pipe busy while the other slot runs an epilogue.
// * The residual sum uses Horner with stride 2 (Q_{m+2} = F + Q_m E^2) in the
//   fused step and doubling in the standalone inverse (at KB = 64 one product
//   per block and round: V_a stacked over E^a times E^a).
// * WY is computed transposed, W^T = K^T (T diag(beta))^T, a full-rate M=128
//   (= d) product; its epilogue transposes through the (now free) operand and
//   V tiles with stmatrix .trans and leaves with TMA bulk stores.
// * Every wait is bounded (2 s).  On expiry the kernel sets the status word,
//   stops issuing work, waits (bounded) for its own copies and MMAs and frees
//   TMEM before returning.
#include <cuda.h>

#include "common.cuh"
#include "tc.h"
#include "tc_ptx.cuh"

namespace gdn {
namespace tcg {

constexpr int kBandMax = 4;                      // widest band the fused step's band path takes

enum Mode { kFused = 0, kBuildA = 1, kNeumann = 2, kWY = 3, kNewton = 4, kFusedRaw = 5,
            kBlockInv = 6, kFusedBand = 7, kFusedRawBand = 8 };

// the fused step, on prepared inputs or with the prologue (raw K, per-token log-gates)
__host__ __device__ constexpr bool is_fused(int m) {
    return m == kFused || m == kFusedRaw || m == kFusedBand || m == kFusedRawBand;
}
// the fused step with the prologue in front
__host__ __device__ constexpr bool is_raw(int m) { return m == kFusedRaw || m == kFusedRawBand; }
// the fused step's band path (k = 64, mask on, N <= kBandMax; chosen at launch)
__host__ __device__ constexpr bool is_band(int m) { return m == kFusedBand || m == kFusedRawBand; }
__host__ __device__ constexpr bool uses_K(int m) { return is_fused(m) || m == kBuildA || m == kWY; }
__host__ __device__ constexpr bool uses_V(int m) { return is_fused(m) || m == kWY; }
// the standalone inverses: A in by TMA (staged a tile ahead), T out by TMA
__host__ __device__ constexpr bool inv_only(int m) {
    return m == kNeumann || m == kNewton || m == kBlockInv;
}
__host__ __device__ constexpr int block_of(int kc) { return kc < 64 ? 64 : kc; }

// Per-slot shared-memory layout (bytes).  The 1024-byte aligned operand
// regions of all slots come first, then each slot's beta/g, then control.
template <int KB, int MODE>
struct SlotLayout {
    static constexpr int kK = uses_K(MODE) ? kRows * kD * 2 : 0;        // bf16 [2][128][64]
    static constexpr int kV = uses_V(MODE) ? kRows * kD * 2 : 0;
    static constexpr int kAop = (is_fused(MODE) || inv_only(MODE)) ? kRows * KB * 2 : 0;
    static constexpr int kXY = (MODE == kBuildA) ? 0 : kRows * KB * 2;  // 16-bit [KB/64][128][64]
    static constexpr int offK = 0;
    static constexpr int offV = offK + kK;
    static constexpr int offX = offV + kV;
    static constexpr int offAop = offX + kXY;
    static constexpr int offY = offAop + kAop;
    // the standalone inverse stages the next tile's A (fp32, 128-byte swizzled
    // boxes of 32 columns x 128 rows) while it works on the current one
    static constexpr int kStage = inv_only(MODE) ? kRows * KB * 4 : 0;
    static constexpr int offStage = offY + kXY;
    static constexpr int bytes = offStage + kStage;
    static constexpr int bg_bytes = uses_K(MODE) ? 2 * kRows * 4 : 0;  // beta[128], g[128]
};

struct Params {
    int64_t rows;        // B*H*T
    int ntiles;
    int N, mask, S, gated;
    const float* Ain;    // kNeumann, kNewton
    const float* Tin;    // kWY
    float* Aout;         // kBuildA
    float* Tout;         // kFused (optional), kNeumann, kNewton
    int M;               // kNewton: sequential correction steps
    __nv_bfloat16* Kout; // kFusedRaw (optional): the L2-normalised K
    float* gout;         // kFusedRaw (optional): the chunk-local cumulative log-gates
    int* status;
    unsigned long long timeout_ns;   // bound of every wait (2 s)
    int withhold_tile;   // tests of the bounded waits: a load of this tile is never issued (-1: none)
    int withhold_v;      // ... that load is V (1) or K, beta and g (0)
};

struct __align__(8) Ctrl {
    uint64_t fullK[2];   // K tile, beta, g landed
    uint64_t fullV[2];   // V tile landed
    uint64_t mma[2];     // the slot's MMAs completed
    uint64_t wdone[2];   // the slot's W^T products completed (K no longer read)
    uint64_t mmac[2][2]; // per-chunk products of the chain rounds (slot, 64-row block)
    uint64_t drain[2][2];// after an expired wait: the issuing threads' products are done
    unsigned long long timeout_ns;   // the launch's bound of every wait
    uint32_t tmem;
    int abort;
};

template <int KC, int MODE, int NS>
struct KernelShape {
    static constexpr int KB = block_of(KC);
    using L = SlotLayout<KB, MODE>;
    static constexpr int threads = 256 * NS;
    static constexpr int smem = NS * L::bytes + NS * L::bg_bytes + (int)sizeof(Ctrl);
};

// ------------------------------------------------------------------------- //
// the kernel
// ------------------------------------------------------------------------- //
template <int KC, int MODE, int NS, int SN, int SS, int SG>
__global__ void __launch_bounds__(256 * NS, 1)
k_chunk_tc(const __grid_constant__ CUtensorMap mK, const __grid_constant__ CUtensorMap mV,
           const __grid_constant__ CUtensorMap mW, const __grid_constant__ CUtensorMap mU,
           const __grid_constant__ CUtensorMap mB, const __grid_constant__ CUtensorMap mG,
           const Params p) {
    constexpr int KB = block_of(KC);
    constexpr bool SUB = KC < KB;                  // two 32-token chunks per 64 block
    using L = SlotLayout<KB, MODE>;
    constexpr int NP = KB / 32;                    // 32-column pieces per block row
    constexpr int PPT = NP / 2;                    // pieces per thread (two threads per row)
    constexpr int NCH = kRows / KB;                // blocks per tile
    constexpr uint32_t kTmemCols = NS == 2 ? 512 : 256;

    extern __shared__ __align__(1024) uint8_t smem[];
    if ((su32(smem) & 1023u) != 0) {              // swizzled operands need 1024-byte alignment
        if (threadIdx.x == 0) raise_status(p.status, kStatusSmemAlign);
        return;
    }
    uint8_t* bg_base = smem + NS * L::bytes;
    Ctrl* ctrl = reinterpret_cast<Ctrl*>(bg_base + NS * L::bg_bytes);

    // The series order, the residual steps and whether W is gated: the call's,
    // or fixed at compile time in an instance specialised for one setting
    // (SN > 0, SS >= 0, SG >= 0), where every loop and branch on them folds away.
    const int pN = SN > 0 ? SN : p.N;
    const int pS = SS >= 0 ? SS : p.S;
    const int pG = SG >= 0 ? SG : p.gated;
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < NS; ++s) {
            mbar_init(&ctrl->fullK[s], 1);
            mbar_init(&ctrl->fullV[s], 1);
            mbar_init(&ctrl->mma[s], 1);
            mbar_init(&ctrl->wdone[s], 1);
            mbar_init(&ctrl->mmac[s][0], 1);
            mbar_init(&ctrl->mmac[s][1], 1);
            mbar_init(&ctrl->drain[s][0], 1);
            mbar_init(&ctrl->drain[s][1], 1);
        }
        ctrl->abort = 0;
        ctrl->timeout_ns = p.timeout_ns;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 0) tmem_alloc(&ctrl->tmem, kTmemCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = ctrl->tmem;

    // ------------------------------ slot s ------------------------------
    // Slot s = warps [8s, 8s + 8).  Thread (r, h) owns tile row r (= its TMEM
    // lane) and the column half h of that row's block; T0 / T of its half row
    // lives in its registers.
    const int s = warp / 8;
    const int h = (warp % 8) / 4;
    const int r = ((warp & 3) << 5) | lane;
    const int blk = r / KB;                        // block of this row in the tile
    const int i = r % KB;                          // row inside the block
    const int cl = SUB ? (i / KC) * KC : 0;        // first column of this row's chunk
    const int ch = cl + KC;                        // one past its last column
    const int jmin = (is_band(MODE) || p.mask) ? i - pN : -KB;   // band mask keeps columns j >= jmin
    uint8_t* base = smem + s * L::bytes;
    uint8_t* sK = base + L::offK;
    uint8_t* sV = base + L::offV;
    uint8_t* sAop = base + L::offAop;
    uint8_t* sX = base + L::offX;
    uint8_t* sY = base + L::offY;
    uint8_t* sStage = base + L::offStage;
    float* sb = reinterpret_cast<float*>(bg_base + s * L::bg_bytes);
    float* sg = sb + kRows;
    const uint32_t tm = tmem_base + (uint32_t)(s * 256);
    const uint32_t tl = tm + ((uint32_t)((warp & 3) * 32) << 16);   // this warp's lanes
    const uint32_t tD = tl + blk * KB;            // this row's diagonal block of D
    const bool leader = (warp % 8) == 0 && lane == 0;
    const int bar_id = 1 + s;
    const int pc0 = h * PPT;
    uint32_t mma_phase = 0;
    bool ok = true;
    // Once a wait has run out anywhere in the CTA, every thread still walks
    // the rest of its tile's barrier sequence (nobody leaves a slot between
    // two barriers), but waits entered from then on return at once (one
    // already under way runs to its bound) and no product, copy or store is
    // started; the slot leaves together at the next tile's first barrier.
    const volatile int* const abortp = &ctrl->abort;
    auto live = [&]() { return *abortp == 0; };

    auto fail_wait = [&]() {
        atomicExch(&ctrl->abort, 1);
        raise_status(p.status, kStatusTimeout);
    };
    auto wait_mma = [&]() -> bool {
        bool good = live() && mbar_wait(&ctrl->mma[s], mma_phase, &ctrl->timeout_ns);
        mma_phase ^= 1;
        if (!good) fail_wait();
        tc_fence_after();
        return good;
    };
    // hand the operands written by this slot to the tensor pipe
    // smem: generic shared-memory stores since the last publish feed the MMA
    auto publish = [&](bool smem) {
        tmem_wait_st();
        if (smem) fence_async_smem();
        tc_fence_before();
        bar_sync(bar_id, 256);
        tc_fence_after();
    };
    // k x k chain product D = a_buf[128 x KB] * b_buf[KB x 128] (b: MN-major)
    auto mma_chain = [&](const uint8_t* a_buf, const uint8_t* b_buf) {
        if (leader && live()) {
            constexpr uint32_t id = idesc_f16(0, 0, 1, 128, 128);
            const uint32_t ab = su32(a_buf), bb = su32(b_buf);
#pragma unroll 1
            for (int kk = 0; kk < KB / 16; ++kk) {
                uint64_t a = sdesc(ab + (kk >> 2) * (kRows * 128) + (kk & 3) * 32, 16, 1024);
                uint64_t b = sdesc(bb + kk * 2048, KB * 128, 1024);
                mma_ss(tm, a, b, id, kk > 0);
            }
            mma_commit(&ctrl->mma[s]);
        }
    };
    // k x k chain product D = Aop[128 x KB] (TMEM, fp16 pairs) * b_buf[KB x 128] (MN-major)
    auto mma_chain_t = [&](const uint8_t* b_buf) {
        if (leader && live()) {
            constexpr uint32_t id = idesc_f16(0, 0, 1, 128, 128);
            const uint32_t bb = su32(b_buf);
#pragma unroll 1
            for (int kk = 0; kk < KB / 16; ++kk) {
                uint64_t b = sdesc(bb + kk * 2048, KB * 128, 1024);
                mma_ts(tm, tm + 128 + kk * 8, b, id, kk > 0);
            }
            mma_commit(&ctrl->mma[s]);
        }
    };
    // Chain rounds (the series and the Horner residual) run per 64-row block
    // when a tile holds two: each block's 4 warps have their own barrier, MMA
    // barrier and issuing thread, and their products are M = 128, N = 64 (the
    // other block's rows come out as unused values), so the two blocks' rounds
    // interleave on the SM instead of waiting for each other.
    constexpr bool kSplit = (NCH == 2) && (is_fused(MODE) || inv_only(MODE));
    const int cg = kSplit ? blk : 0;
    const bool cleader = kSplit ? (lane == 0 && (warp % 8) == 2 * cg) : leader;
    const int cbar = kSplit ? 3 + 2 * s + cg : bar_id;
    uint32_t cphase = 0;
    uint64_t* const cmbar = kSplit ? &ctrl->mmac[s][cg] : &ctrl->mma[s];
    auto cpublish = [&](bool smem) {
        tmem_wait_st();
        if (smem) fence_async_smem();
        tc_fence_before();
        bar_sync(cbar, kSplit ? 128 : 256);
        tc_fence_after();
    };
    auto cwait = [&]() -> bool {
        if (!kSplit) return wait_mma();
        const bool good = live() && mbar_wait(cmbar, cphase, &ctrl->timeout_ns);
        cphase ^= 1;
        if (!good) fail_wait();
        tc_fence_after();
        return good;
    };
    constexpr int kCN = kSplit ? 64 : 128;                  // N of a chain product
    const uint32_t cd = tm + (kSplit ? 64 * cg : 0);        // its accumulator columns
    const uint32_t cbo = kSplit ? (uint32_t)(cg * 64 * 128) : 0u;   // its B rows
    auto cchain = [&](const uint8_t* a_buf, const uint8_t* b_buf) {
        if (cleader && live()) {
            constexpr uint32_t id = idesc_f16(0, 0, 1, kCN, 128);
            const uint32_t ab = su32(a_buf), bb = su32(b_buf) + cbo;
#pragma unroll 1
            for (int kk = 0; kk < KB / 16; ++kk) {
                uint64_t a = sdesc(ab + (kk >> 2) * (kRows * 128) + (kk & 3) * 32, 16, 1024);
                uint64_t b = sdesc(bb + kk * 2048, KB * 128, 1024);
                mma_ss(cd, a, b, id, kk > 0);
            }
            mma_commit(cmbar);
        }
    };
    auto cchain_t = [&](const uint8_t* b_buf) {
        if (cleader && live()) {
            constexpr uint32_t id = idesc_f16(0, 0, 1, kCN, 128);
            const uint32_t bb = su32(b_buf) + cbo;
#pragma unroll 1
            for (int kk = 0; kk < KB / 16; ++kk) {
                uint64_t b = sdesc(bb + kk * 2048, KB * 128, 1024);
                mma_ts(cd, tm + 128 + kk * 8, b, id, kk > 0);
            }
            mma_commit(cmbar);
        }
    };
    const uint32_t tA = tl + 128;                 // this row's A operand (fp16 pairs)
    // T0 / T: in TMEM columns [160, 224) at KB = 64 (two threads per row, 32
    // columns each), in registers at KB = 128.
    constexpr bool kT0Tmem = (KB == 64);
    const uint32_t tT = tl + 160;
    const uint32_t tF = tl + (KB == 64 ? 224 : 192);  // F = E + E^2 of the residual (fp16 pairs)
    // Band path of the fused step (k = 64, mask on, N <= kBandMax).  With the
    // mask, T0 = M.(sum_{n<=N} A^n) is zero below its N-th sub-diagonal, so the
    // series' products are needed only on the N + 1 diagonals the mask keeps,
    // and the two products with T0 as a factor, A T0 (for the residual E) and
    // T0 Q_S (for T), take at most N + 1 terms per entry.  These run on the
    // CUDA cores; the dense products (K K^T, the powers of E, WY) stay on the
    // tensor cores.  Storage:
    //   X (fp16)       A - I, for the band entries other rows read;
    //   TMEM           A - I in fp32, then T, in the block's own accumulator
    //                  columns (no other block's product writes them);
    //   Aop            bT[d-1][c] = T0[c+d][c], T0's band by column (zero past
    //                  the chunk);
    //   Y (fp16)       I + Q_S, whose rows the T0 (I + Q_S) product reads.
    constexpr bool kBandable = is_band(MODE) && KC == 64;
    constexpr bool band = kBandable;
    float* const bT = reinterpret_cast<float*>(sAop);
    float tb[kBandMax + 1];                        // tb[d] = T0[i][i-d], zero past N
    auto band_row = [&]() {                        // row i's band of T0 back from bT
        tb[0] = 1.f;
#pragma unroll
        for (int d = 1; d <= kBandMax; ++d)
            tb[d] = (d <= pN && i - d >= 0) ? bT[(d - 1) * kRows + blk * KB + i - d] : 0.f;
    };
    // the slot's leader loads its own tiles: K, beta, g on fullK, V on fullV
    int k_issued = 0, v_issued = 0;               // loads issued by this slot's leader
    auto issue_k = [&](int n) {
        const int tile = blockIdx.x + n * gridDim.x;
        if (!(uses_K(MODE) || inv_only(MODE)) || tile >= p.ntiles || !live()) return;
        if (tile == p.withhold_tile && !p.withhold_v) return;   // tests: the wait must run out
        ++k_issued;
        const int y = tile * kRows;
        if (inv_only(MODE)) {                          // A: KC / 32 boxes of 16 KB
            mbar_expect_tx(&ctrl->fullK[s], (KC / 32) * 16384);
#pragma unroll 1
            for (int b = 0; b < KC / 32; ++b)
                tma_load_2d(sStage + b * 16384, &mK, 32 * b, y, &ctrl->fullK[s]);
            return;
        }
        mbar_expect_tx(&ctrl->fullK[s], kRows * kD * 2 + 2 * kRows * 4);
        tma_load_2d(sK, &mK, 0, y, &ctrl->fullK[s]);
        tma_load_2d(sK + kRows * 128, &mK, 64, y, &ctrl->fullK[s]);
        tma_load_1d(sb, &mB, y, &ctrl->fullK[s]);
        tma_load_1d(sg, &mG, y, &ctrl->fullK[s]);
    };
    auto issue_v = [&](int n) {
        const int tile = blockIdx.x + n * gridDim.x;
        if (!uses_V(MODE) || tile >= p.ntiles || !live()) return;
        if (tile == p.withhold_tile && p.withhold_v) return;    // tests: the wait must run out
        ++v_issued;
        const int y = tile * kRows;
        mbar_expect_tx(&ctrl->fullV[s], kRows * kD * 2);
        tma_load_2d(sV, &mV, 0, y, &ctrl->fullV[s]);
        tma_load_2d(sV + kRows * 128, &mV, 64, y, &ctrl->fullV[s]);
    };
    // W leaves through the operand buffers (free once the WY products are done),
    // U through the V tile; K is reloaded for the next tile meanwhile.
    uint8_t* sWst = (MODE == kWY) ? sX : sAop;   // followed by Y: 32 KB at KB = 64
    bool staged_free = true;                       // previous tile's stores have read Aop/Y/V
    // The previous tile's W/U stores read Aop+Y and V; before this tile first
    // writes Y (or V is reloaded) the leader waits for those reads to finish.
    auto release_staging = [&](int n) {
        if (staged_free) return;
        if (leader) {
            bulk_wait_read();
            issue_v(n);
        }
        bar_sync(bar_id, 256);
        staged_free = true;
    };
    auto in_chunk = [&](int j) { return SUB ? (j >= cl && j < ch) : true; };
    // read / write this thread's 32-column piece pp of T0
    auto t0_get = [&](int pp, float (&t)[32], float* T0r) {
        if (kT0Tmem) {
            tmem_ld32((band ? tD : tT) + (pc0 + pp) * 32, t);
        } else {
#pragma unroll
            for (int jj = 0; jj < 32; ++jj) t[jj] = T0r[pp * 32 + jj];
        }
    };
    auto t0_put = [&](int pp, const float (&t)[32], float* T0r) {
        if (kT0Tmem) {
            tmem_st32((band ? tD : tT) + (pc0 + pp) * 32, t);
        } else {
#pragma unroll
            for (int jj = 0; jj < 32; ++jj) T0r[pp * 32 + jj] = t[jj];
        }
    };
    auto eye = [&](int j) { return i == j ? 1.f : 0.f; };
    auto piece_in_chunk = [&](int pc) { return !SUB || (pc * 32 >= cl && pc * 32 < ch); };

    // 8 fp16 values of row rr, columns 8q .. 8q + 7, of an operand buffer
    auto ld_h8 = [&](const uint8_t* buf, int rr, int q, float (&o)[8]) {
        uint4 u;
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
                     : "r"(su32(buf) + op_off(rr, q)));
        const uint32_t w4[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w4[c]));
            o[2 * c] = f.x;
            o[2 * c + 1] = f.y;
        }
    };
    if (leader) {
        issue_k(s);
        issue_v(s);
    }

    for (int n = s;; n += NS) {
        const int tile = blockIdx.x + n * gridDim.x;
        if (tile >= p.ntiles) break;
        const uint32_t use_par = (uint32_t)((n / NS) & 1);
        const int64_t row0 = (int64_t)tile * kRows;
        const int64_t grow = row0 + r;
        const bool valid = grow < p.rows;
        const int64_t cidx = grow / KC;                  // chunk of this row
        const int64_t rin = grow % KC;                   // row inside the chunk
        float T0[kT0Tmem ? 1 : PPT * 32];                // this thread's part of row r of T0 / T

        if ((uses_K(MODE) || inv_only(MODE)) && !(live() && mbar_wait(&ctrl->fullK[s], use_par, &ctrl->timeout_ns)))
            fail_wait();
        // the slot decides together whether to stop (an OR over its threads'
        // view of the abort flag, so no thread can read it differently)
        if (bar_sync_or(bar_id, 256, !live())) { ok = false; break; }

        if (is_fused(MODE) || MODE == kBuildA) {
            if constexpr (is_raw(MODE)) {
                // ---- prologue: K rows to unit L2 norm (in place, bf16) and the
                // per-token log-gates to chunk-local cumulative sums ----
                // Here lane l of the slot's warp w takes row 16 w + l / 2, panel
                // (64 columns) l % 2: its 64 values stay in registers, the two
                // halves' sums of squares (fp32) meet by one shuffle, and the
                // panel is rescaled in place; an all-zero row (past the end of
                // the data) stays zero.
                {
                    const int pr = 16 * (warp & 7) + (lane >> 1), pn = lane & 1;
                    const uint32_t rb = su32(sK) + pn * (kRows * 128) + pr * 128;
                    uint32_t w[32];
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        const uint4 u = lds128(rb + ((c ^ (pr & 7)) << 4));
                        w[4 * c] = u.x; w[4 * c + 1] = u.y; w[4 * c + 2] = u.z; w[4 * c + 3] = u.w;
                    }
                    float ss = 0.f;
#pragma unroll
                    for (int e = 0; e < 32; ++e) {                 // bf16 pair -> two floats
                        const float lo = __uint_as_float(w[e] << 16);
                        const float hi = __uint_as_float(w[e] & 0xffff0000u);
                        ss = fmaf(lo, lo, ss);
                        ss = fmaf(hi, hi, ss);
                    }
                    ss += __shfl_xor_sync(0xffffffffu, ss, 1);
                    const float inv = ss > 0.f ? rsqrtf(ss) : 0.f;
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        w[e] = pack_b2(__uint_as_float(w[e] << 16) * inv,
                                       __uint_as_float(w[e] & 0xffff0000u) * inv);
                    const int64_t gr = row0 + pr;
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        const uint4 u = make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
                        sts128(rb + ((c ^ (pr & 7)) << 4), u);
                        if (p.Kout && gr < p.rows)
                            *reinterpret_cast<uint4*>(p.Kout + gr * kD + pn * 64 + c * 8) = u;
                    }
                }
                // warp 0 of the slot: inclusive sums of the log-gates, restarted
                // every KC rows (lane l owns rows 4l .. 4l + 3)
                if ((warp & 7) == 0) {
                    const float4 x = *reinterpret_cast<const float4*>(sg + 4 * lane);
                    float y0 = x.x, y1 = y0 + x.y, y2 = y1 + x.z, y3 = y2 + x.w;
                    constexpr int seg = KC / 4;            // lanes per chunk
                    float run = y3;
#pragma unroll
                    for (int o = 1; o < seg; o <<= 1) {
                        const float up = __shfl_up_sync(0xffffffffu, run, o);
                        if ((lane % seg) >= o) run += up;
                    }
                    const float before = run - y3;        // this chunk's lanes before lane
                    y0 += before; y1 += before; y2 += before; y3 += before;
                    *reinterpret_cast<float4*>(sg + 4 * lane) = make_float4(y0, y1, y2, y3);
                    if (p.gout && row0 + 4 * lane < p.rows)
                        *reinterpret_cast<float4*>(p.gout + row0 + 4 * lane) =
                            make_float4(y0, y1, y2, y3);
                }
                fence_async_smem();                       // the rescaled K feeds the MMAs
                bar_sync(bar_id, 256);
            }
            // ---- G = K K^T over the tile, then A = -beta_i G_ij exp(g_i - g_j) ----
            if (leader && live()) {
                tc_fence_after();
                constexpr uint32_t id = idesc_f16(1, 0, 0, 128, 128);
                const uint32_t kbase = su32(sK);
#pragma unroll 1
                for (int kk = 0; kk < kD / 16; ++kk) {
                    uint64_t a = sdesc(kbase + (kk >> 2) * (kRows * 128) + (kk & 3) * 32, 16, 1024);
                    mma_ss(tm, a, a, id, kk > 0);
                }
                mma_commit(&ctrl->mma[s]);
            }
            if (!wait_mma()) ok = false;
            if (band) release_staging(n);             // the band tables take Aop
            const float bi = sb[r], gi = sg[r];
            const float* gcol = sg + blk * KB;
            float lbi = 0.f;                              // band path: log2(beta_i)
            if constexpr (band) asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(lbi) : "f"(bi));
#pragma unroll
            for (int pp = 0; pp < PPT; ++pp) {
                const int pc = pc0 + pp;
                float v[32];
                // pieces above the diagonal or in another chunk for the whole warp
                if (pc * 32 > (i | 31) || !piece_in_chunk(pc)) {
#pragma unroll
                    for (int jj = 0; jj < 32; ++jj) v[jj] = 0.f;
                } else {
                    tmem_ld32(tD + pc * 32, v);
#pragma unroll
                    for (int jj = 0; jj < 32; ++jj) {
                        const int j = pc * 32 + jj;
                        const bool in = in_chunk(j) && j < i;
                        if constexpr (band) {             // beta_i e^(g_i - g_j) = 2^((g_i - g_j) log2 e + log2 beta_i)
                            float e2;
                            asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e2)
                                : "f"(fmaf(gi - gcol[j], 1.4426950408889634f, lbi)));
                            v[jj] = in ? -v[jj] * e2 : 0.f;
                        } else {
                            v[jj] = in ? -bi * v[jj] * exp_e(gi - gcol[j]) : 0.f;
                        }
                    }
                }
                if (MODE == kBuildA) {
                    if (valid && piece_in_chunk(pc)) {
                        float* dst = p.Aout + cidx * KC * KC + rin * KC + (pc * 32 - cl);
#pragma unroll
                        for (int q = 0; q < 8; ++q)
                            reinterpret_cast<float4*>(dst)[q] =
                                make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
                    }
                } else if (kBandable && band) {
                    // A - I: fp16 to X, fp32 to the T0 columns of TMEM
                    if (pc == (i >> 5)) {
#pragma unroll
                        for (int jj = 0; jj < 32; ++jj)
                            if (pc * 32 + jj == i) v[jj] = -1.f;
                    }
                    st_op32<false>(sX, r, pc, v);
                    tmem_st32(tD + pc * 32, v);
                } else {
                    st_op32<false>(sX, r, pc, v);             // A (chain's right operand)
                    float t[32];
#pragma unroll
                    for (int jj = 0; jj < 32; ++jj) {
                        const int j = pc * 32 + jj;
                        t[jj] = eye(j) + (j >= jmin ? v[jj] : 0.f);   // X_1 = I + M.A
                    }
                    if (pN == 1) t0_put(pp, t, T0);
                    else tmem_st_h16(tA + pc * 16, t);
                }
            }
            if (MODE == kBuildA) {
                tc_fence_before();
                bar_sync(bar_id, 256);                 // beta/g and the accumulator are read
                if (leader) issue_k(n + NS);
                continue;
            }
        } else if (inv_only(MODE)) {
            // ---- A rows from the staged tile ----
            float av[32];                                  // kBlockInv: this thread's A piece
#pragma unroll
            for (int pp = 0; pp < PPT; ++pp) {
                const int pc = pc0 + pp;
                float v[32];
                if (piece_in_chunk(pc)) {                 // rows past the end were zero-filled
                    const uint32_t rb =
                        su32(sStage) + (uint32_t)(((pc * 32 - cl) >> 5) * 16384 + r * 128);
#pragma unroll
                    for (int c4 = 0; c4 < 8; ++c4) {
                        uint32_t u0, u1, u2, u3;
                        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                                     : "=r"(u0), "=r"(u1), "=r"(u2), "=r"(u3)
                                     : "r"(rb + ((c4 ^ (r & 7)) << 4)));
                        v[4 * c4] = __uint_as_float(u0);
                        v[4 * c4 + 1] = __uint_as_float(u1);
                        v[4 * c4 + 2] = __uint_as_float(u2);
                        v[4 * c4 + 3] = __uint_as_float(u3);
                    }
                } else {
#pragma unroll
                    for (int jj = 0; jj < 32; ++jj) v[jj] = 0.f;
                }
                if constexpr (MODE == kBlockInv) {
#pragma unroll
                    for (int jj = 0; jj < 32; ++jj) av[jj] = v[jj];
                } else {
                    st_op32<false>(sX, r, pc, v);
                    float t[32];
#pragma unroll
                    for (int jj = 0; jj < 32; ++jj) {
                        const int j = pc * 32 + jj;
                        t[jj] = eye(j) + (j >= jmin ? v[jj] : 0.f);       // X_1 = I + M.A
                    }
                    if (pN == 1) t0_put(pp, t, T0);
                    else tmem_st_h16(tA + pc * 16, t);
                }
            }
            // the stage is read: it takes the slot's next tile; the previous
            // tile's T store has read the Aop / Y staging before it is reused
            fence_async_smem();
            if (leader) bulk_wait_read();
            bar_sync(bar_id, 256);
            if (leader) issue_k(n + NS);
            if constexpr (MODE == kBlockInv && KB == 64) {
                // ---- exact inverse by 2 x 2 block decomposition: the 16 x 16
                // diagonal blocks by substitution, then per doubling level
                // T <- T + T (A_L T), A_L = A on that level's off-diagonal
                // blocks.  Row i's diagonal block b = i / 16 lies in piece
                // b / 2 (warp-uniform); its 16 rows are 16 lanes of one warp.
                const int b16 = i >> 4;
                const bool diag = (b16 >> 1) == h;
                float d[16];
#pragma unroll
                for (int cc = 0; cc < 16; ++cc) d[cc] = cc == (i & 15) ? 1.f : 0.f;
                if (diag) {
                    // T = I + A T inside the block, row j final before it is used;
                    // rows l <= j add A[l][j] = 0
                    const int base = lane & 16;
#pragma unroll
                    for (int j = 0; j < 15; ++j) {
                        const float aij = (b16 & 1) ? av[16 + j] : av[j];
#pragma unroll
                        for (int cc = 0; cc < 16; ++cc)
                            d[cc] = fmaf(aij, __shfl_sync(0xffffffffu, d[cc], base + j), d[cc]);
                    }
                }
                float b1[32], a1[32], a2[32];
#pragma unroll
                for (int jj = 0; jj < 32; ++jj) {
                    const float dj = (b16 & 1) ? (jj >= 16 ? d[jj & 15] : 0.f) : (jj < 16 ? d[jj & 15] : 0.f);
                    b1[jj] = diag ? dj : 0.f;
                    a1[jj] = (diag && (b16 & 1) && jj < 16) ? av[jj] : 0.f;   // block (2p+1, 2p)
                    a2[jj] = (KC == 64 && i >= 32 && h == 0) ? av[jj] : 0.f;  // block (1, 0) of 32s
                }
                st_op32<false>(sX, r, pc0, a1);
                st_op32<false>(sY, r, pc0, b1);
                st_op32<false>(sAop, r, pc0, a2);
                t0_put(0, b1, T0);
            }
        } else {
            // ---- kWY: T row from global memory ----
            release_staging(n);
#pragma unroll
            for (int pp = 0; pp < PPT; ++pp) {
                const int pc = pc0 + pp;
                float t[32];
                if (valid && piece_in_chunk(pc)) {
                    const float4* src = reinterpret_cast<const float4*>(
                        p.Tin + cidx * KC * KC + rin * KC + (pc * 32 - cl));
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        float4 a = __ldg(src + q);
                        t[4 * q] = a.x; t[4 * q + 1] = a.y; t[4 * q + 2] = a.z; t[4 * q + 3] = a.w;
                    }
                } else {
#pragma unroll
                    for (int jj = 0; jj < 32; ++jj) t[jj] = 0.f;
                }
                t0_put(pp, t, T0);
            }
        }

        if (is_fused(MODE)) release_staging(n);
        if (is_fused(MODE) || inv_only(MODE)) {
            // ---- truncated Neumann series in Horner form ----
            // X_1 = I + M.A, X_n = I + M.(X_{n-1} A), T0 = X_N: inside the band
            // X_{n-1} A reads only in-band entries of X_{n-1}, so masking every
            // step gives M.(sum_{n<=N} A^n) exactly.
            for (int pw = 2; !band && pw <= pN; ++pw) {
                cpublish(pw == 2);
                cchain_t(sX);                                           // X_{n-1} A
                if (!cwait()) ok = false;
#pragma unroll
                for (int pp = 0; pp < PPT; ++pp) {
                    const int pc = pc0 + pp;
                    float v[32];
                    tmem_ld32(tD + pc * 32, v);
#pragma unroll
                    for (int jj = 0; jj < 32; ++jj) {
                        const int j = pc * 32 + jj;
                        v[jj] = eye(j) + ((in_chunk(j) && j >= jmin) ? v[jj] : 0.f);
                    }
                    if (pw == pN) t0_put(pp, v, T0);
                    else tmem_st_h16(tA + pc * 16, v);
                }
            }
            if (kBandable && band) {
                // ---- the series on its band: X_1 = I + M.A, X_n = I + M.(X_{n-1} A)
                // evaluated on the N + 1 diagonals the mask keeps, row by row:
                // X_n[i][i-d] = [d = 0] + sum_{m<d} X_{n-1}[i][i-m] A[i-m][i-d].
                // Entries before the chunk's first column do not exist (zero).
                tmem_wait_st();
                tc_fence_before();
                bar_sync(cbar, 128);                              // A - I in X and TMEM
                tc_fence_after();
                // A[i-m][i-d] (m < d) from X, zero where the entry is not in the chunk
                auto wA = [&](int m, int d) {
                    const bool in = d <= pN && i - d >= 0;
                    const int row = in ? r - m : r, col = in ? i - d : 0;
                    uint16_t u;
                    asm volatile("ld.shared.u16 %0, [%1];"
                                 : "=h"(u)
                                 : "r"(su32(sX) + op_off(row, col >> 3) + 2 * (col & 7)));
                    return in ? __half2float(__ushort_as_half(u)) : 0.f;
                };
                tb[0] = 1.f;
#pragma unroll
                for (int d = 1; d <= kBandMax; ++d) tb[d] = wA(0, d);
#pragma unroll
                for (int nn = 2; nn <= kBandMax; ++nn) {
                    if (nn > pN) break;
                    float y[kBandMax + 1];
#pragma unroll
                    for (int d = 1; d <= kBandMax; ++d) {
                        float acc = wA(0, d);
#pragma unroll
                        for (int m = 1; m < d; ++m) acc = fmaf(tb[m], wA(m, d), acc);
                        y[d] = acc;
                    }
#pragma unroll
                    for (int d = 1; d <= kBandMax; ++d) tb[d] = y[d];
                }
                if (pS == 0) {
                    // T = T0: the band, zero elsewhere
                    float t[32];
#pragma unroll
                    for (int jj = 0; jj < 32; ++jj) {
                        const int dd = i - (pc0 * 32 + jj);
                        float x = 0.f;
#pragma unroll
                        for (int d = 0; d <= kBandMax; ++d) x = dd == d ? tb[d] : x;
                        t[jj] = x;
                    }
                    t0_put(0, t, T0);
                } else {
                    // T0 by column for A T0: column c of row c + d, zero past the chunk
                    if (h == 0) {
#pragma unroll
                        for (int d = 1; d <= kBandMax; ++d) {
                            if (d > pN) break;
                            if (i - d >= 0) bT[(d - 1) * kRows + blk * KB + i - d] = tb[d];
                            if (i + d >= KB) bT[(d - 1) * kRows + blk * KB + i] = 0.f;
                        }
                    }
                    bar_sync(cbar, 128);                          // bT written
                }
            }
            // ---- parallel residual correction: T = T0 G, G = sum_{s<=S} E^s ----
            // Two schedules.  Horner keeps Q_m in TMEM as the left operand
            // (stride 2 below: one product per round, in 64-row blocks that do
            // not wait for each other) and T0 in fp32; it serves the fused step,
            // k = 128 and every S the doubling does not.  The standalone inverse
            // at KB = 64 doubles when S + 1 is 2^m or 2^m + 1 (stacked, below).
            // In the fused step the stacked form measured slower at S <= 8 (its
            // lockstep rounds and wider epilogues cost more than the two rounds
            // it saves); at k = 128 a doubling with two products per round lost
            // to Horner, its extra k^3 products outweighing the rounds.
            if constexpr (MODE == kBlockInv && KB == 64) {
                // level 1 (16 -> 32): A1 in X, T in Y; level 2 (32 -> 64): A2 in Aop
                for (int lv = 0; lv < (KC == 64 ? 2 : 1); ++lv) {
                    cpublish(true);
                    cchain(lv == 0 ? sX : sAop, sY);                     // P = A_L T
                    if (!cwait()) ok = false;
                    {
                        float v[32];
                        tmem_ld32(tD + pc0 * 32, v);
                        st_op32<false>(sX, r, pc0, v);
                    }
                    cpublish(true);
                    cchain(sY, sX);                                      // T P
                    if (!cwait()) ok = false;
                    {
                        float v[32], t[32];
                        tmem_ld32(tD + pc0 * 32, v);
                        t0_get(0, t, T0);
#pragma unroll
                        for (int jj = 0; jj < 32; ++jj) t[jj] += v[jj];
                        t0_put(0, t, T0);
                        if (lv == 0) st_op32<false>(sY, r, pc0, t);
                    }
                }
            } else if constexpr (MODE == kNewton) {
                // Sequential correction, the form the method's parallel residual
                // replaces: R_m = I - (I - A) T_m = I - T_m + A T_m and
                // T_{m+1} = T_m + T_m R_m, two dependent products per step.
                // T_m stays fp32 (T0 columns / registers); its fp16 copy goes
                // to Y (right operand of A T_m) and to TMEM (left operand of
                // T_m R_m), and R_m to Y.
                for (int it = 0; it < p.M; ++it) {
#pragma unroll
                    for (int pp = 0; pp < PPT; ++pp) {
                        float t[32];
                        t0_get(pp, t, T0);
                        st_op32<false>(sY, r, pc0 + pp, t);                // T_m
                    }
                    cpublish(true);
                    cchain(sX, sY);                                      // A T_m
                    if (!cwait()) ok = false;
#pragma unroll
                    for (int pp = 0; pp < PPT; ++pp) {
                        const int pc = pc0 + pp;
                        float v[32], t[32];
                        tmem_ld32(tD + pc * 32, v);
                        t0_get(pp, t, T0);
#pragma unroll
                        for (int jj = 0; jj < 32; ++jj) {
                            const int j = pc * 32 + jj;
                            v[jj] = in_chunk(j) ? eye(j) - t[jj] + v[jj] : 0.f;   // R_m
                        }
                        st_op32<false>(sY, r, pc, v);
                        tmem_st_h16(tA + pc * 16, t);                      // T_m, left operand
                    }
                    cpublish(true);
                    cchain_t(sY);                                        // T_m R_m
                    if (!cwait()) ok = false;
#pragma unroll
                    for (int pp = 0; pp < PPT; ++pp) {
                        const int pc = pc0 + pp;
                        float v[32], t[32];
                        tmem_ld32(tD + pc * 32, v);
                        t0_get(pp, t, T0);
#pragma unroll
                        for (int jj = 0; jj < 32; ++jj)
                            if (in_chunk(pc * 32 + jj)) t[jj] += v[jj];      // T_{m+1}
                        t0_put(pp, t, T0);
                    }
                }
            } else if (pS > 0) {
                const int S = pS;
                int K2 = 0;
                while ((2 << K2) <= S + 1) ++K2;
                const bool p2p1 = (1 << K2) + 1 == S + 1;
                const bool dbl = (1 << K2) == S + 1 || p2p1;
                // Stacked doubling (64-row blocks, S + 1 = 2^J or 2^J + 1).
                // With U_a = sum_{s<a} E^s and V_a = T0 U_a: V_2a = V_a + V_a E^a
                // and E^2a = E^a E^a share the right operand E^a, so ONE M = 128
                // product per block gives both when its left operand stacks V_a
                // over E^a.  Block 0 stacks [V_0; E_0] (the X buffer), block 1
                // [E_1; V_1] (the Aop buffer): each block's V rows land on its
                // own TMEM lanes, where V_a stays in fp32 (the T0 columns), and
                // its E rows on the other block's lanes, whose threads write
                // them back.  Every thread therefore writes row r of X and of
                // Aop.  T0 (fp16) waits in Y for the last product T0 E^(2^J)
                // when S = 2^J.  S = 8 takes 5 dependent rounds (Horner: 7).
                bool stacked = false;
                if constexpr (KB == 64 && MODE == kNeumann) stacked = dbl;
                if (stacked) {
                    // this row's V_a; the other block's E^a row r; the other block's columns
                    auto sVr = [&]() { return blk == 0 ? sX : sAop; };
                    auto sEr = [&]() { return blk == 0 ? sAop : sX; };
                    auto tE = [&]() { return tl + (uint32_t)((1 - blk) * 64); };
                    // block 0's product into columns [0, 64), block 1's into [64, 128)
                    auto mma_blocks = [&](const uint8_t* a0, const uint8_t* b0, const uint8_t* a1,
                                          const uint8_t* b1) {
                        if (leader && live()) {
                            constexpr uint32_t id = idesc_f16(0, 0, 1, 64, 128);
                            const uint32_t x0 = su32(a0), y0 = su32(b0);
                            const uint32_t x1 = su32(a1), y1 = su32(b1);
#pragma unroll 1
                            for (int kk = 0; kk < 4; ++kk) {
                                mma_ss(tm, sdesc(x0 + kk * 32, 16, 1024),
                                       sdesc(y0 + kk * 2048, 64 * 128, 1024), id, kk > 0);
                                mma_ss(tm + 64, sdesc(x1 + kk * 32, 16, 1024),
                                       sdesc(y1 + kk * 2048, 64 * 128, 1024), id, kk > 0);
                            }
                            mma_commit(&ctrl->mma[s]);
                        }
                    };
#pragma unroll
                    for (int pp = 0; pp < PPT; ++pp) {
                        float t[32];
                        t0_get(pp, t, T0);
                        st_op32<false>(sY, r, pc0 + pp, t);                // T0
                    }
                    publish(true);
                    mma_blocks(sX, sY, sX, sY + 64 * 128);                  // A T0
                    if (!wait_mma()) ok = false;
#pragma unroll
                    for (int pp = 0; pp < PPT; ++pp) {
                        const int pc = pc0 + pp;
                        float v[32], t[32];
                        tmem_ld2(tD + pc * 32, v, tT + pc * 32, t);
#pragma unroll
                        for (int jj = 0; jj < 32; ++jj) {
                            const int j = pc * 32 + jj;
                            v[jj] = in_chunk(j) ? eye(j) - t[jj] + v[jj] : 0.f;   // E
                        }
                        st_op32<false>(sVr(), r, pc, t);                   // V_1 = T0
                        st_op32<false>(sVr(), r ^ 64, pc, v);              // E of this block
                    }
                    for (int rd = 1; rd <= K2; ++rd) {
                        const bool last = rd == K2;
                        publish(true);
                        mma_blocks(sX, sX + 64 * 128, sAop, sAop);          // [V; E] E, [E; V] E
                        if (!wait_mma()) ok = false;
#pragma unroll
                        for (int pp = 0; pp < PPT; ++pp) {
                            const int pc = pc0 + pp;
                            if (!last || p2p1) {
                                float e[32];
                                tmem_ld32(tE() + pc * 32, e);
#pragma unroll
                                for (int jj = 0; jj < 32; ++jj)
                                    if (!in_chunk(pc * 32 + jj)) e[jj] = 0.f;
                                st_op32<false>(sEr(), r, pc, e);           // E^2a
                            }
                            float d[32], v[32];
                            tmem_ld2(tD + pc * 32, d, tT + pc * 32, v);
#pragma unroll
                            for (int jj = 0; jj < 32; ++jj)
                                v[jj] = in_chunk(pc * 32 + jj) ? v[jj] + d[jj] : 0.f;   // V_2a
                            t0_put(pp, v, T0);
                            if (!last) st_op32<false>(sVr(), r, pc, v);
                        }
                    }
                    if (p2p1) {
                        publish(true);
                        mma_blocks(sY, sX + 64 * 128, sY, sAop);            // T0 E^(2^J)
                        if (!wait_mma()) ok = false;
#pragma unroll
                        for (int pp = 0; pp < PPT; ++pp) {
                            const int pc = pc0 + pp;
                            float d[32], v[32];
                            tmem_ld2(tD + pc * 32, d, tT + pc * 32, v);
#pragma unroll
                            for (int jj = 0; jj < 32; ++jj)
                                if (in_chunk(pc * 32 + jj)) v[jj] += d[jj];      // T
                            t0_put(pp, v, T0);
                        }
                    }
                } else {
                    // Horner with stride 2: Q_1 = E, E^2 = E E, F = E + E^2 = Q_2,
                    // Q_{m+2} = F + Q_m E^2, from Q_2 when S is even and from Q_1
                    // when it is odd, so no single step is left over (S = 8
                    // takes E^2, Q_4, Q_6, Q_8); Q_m (no identity) is the left
                    // operand in TMEM, E in X, E^2 then Q_S in Y, F in TMEM as
                    // fp16.
                    if (kBandable && band) {
                        // E = I + (A - I) T0 on this thread's columns j:
                        // (A - I) T0 [i][j] = sum_{d<=N} (A - I)[i][j+d] T0[j+d][j]
                        // (T0[j][j] = 1); the -I term takes T0's band off
                        float a[32], ed[4], v[32];
                        tmem_ld32(tD + pc0 * 32, a);
                        if (h == 0) {
                            tmem_ld4(tD + 32, ed);                  // the partner's first columns
                        } else {
#pragma unroll
                            for (int e = 0; e < 4; ++e) ed[e] = 0.f;   // past the chunk
                        }
#pragma unroll
                        for (int jj = 0; jj < 32; ++jj) v[jj] = a[jj];              // d = 0
#pragma unroll
                        for (int d = 1; d <= kBandMax; ++d) {
                            if (d > pN) break;
                            const float* tc = bT + (d - 1) * kRows + blk * KB + pc0 * 32;
#pragma unroll
                            for (int q = 0; q < 8; ++q) {
                                const float4 t4 = *reinterpret_cast<const float4*>(tc + 4 * q);
                                const float tt[4] = {t4.x, t4.y, t4.z, t4.w};
#pragma unroll
                                for (int c = 0; c < 4; ++c) {
                                    const int jj = 4 * q + c;
                                    const float ad = jj + d < 32 ? a[(jj + d) & 31] : ed[(jj + d) & 3];
                                    v[jj] = fmaf(ad, tt[c], v[jj]);
                                }
                            }
                        }
                        // the diagonal of the sum is -1 exactly: E[i][i] = 0, and
                        // (I + E)[i][i] = 1 for S = 1, where Q_1 = E is final
                        if (pc0 == (i >> 5)) {
#pragma unroll
                            for (int jj = 0; jj < 32; ++jj)
                                if (pc0 * 32 + jj == i) v[jj] = pS == 1 ? 1.f : 0.f;
                        }
                        if (pS == 1) {
                            st_op32<false>(sY, r, pc0, v);                // I + Q_1
                        } else {
                            st_op32<false>(sX, r, pc0, v);                  // E
                            tmem_st_h16(tA + pc0 * 16, v);                // Q_1 = E
                        }
                    } else {
#pragma unroll
                    for (int pp = 0; pp < PPT; ++pp) {
                        float t[32];
                        t0_get(pp, t, T0);
                        st_op32<false>(sY, r, pc0 + pp, t);                // T0
                    }
                    cpublish(true);
                    cchain(sX, sY);                                      // A T0
                    if (!cwait()) ok = false;
#pragma unroll
                    for (int pp = 0; pp < PPT; ++pp) {
                        const int pc = pc0 + pp;
                        float v[32], t[32];
                        tmem_ld32(tD + pc * 32, v);
                        t0_get(pp, t, T0);
#pragma unroll
                        for (int jj = 0; jj < 32; ++jj) {
                            const int j = pc * 32 + jj;
                            v[jj] = in_chunk(j) ? eye(j) - t[jj] + v[jj] : 0.f;   // E
                        }
                        if (pS == 1) {
                            st_op32<false>(sY, r, pc, v);                   // Q_1 = E
                            tmem_st_h16(tA + pc * 16, t);                 // T0
                        } else {
                            st_op32<false>(sX, r, pc, v);                   // E
                            tmem_st_h16(tA + pc * 16, v);                 // Q_1 = E
                        }
                    }
                    }
                    // this row's E from X, 8 columns at a time
                    auto e_row = [&](int pc, float (&e)[32]) {
#pragma unroll
                        for (int g = 0; g < 4; ++g) {
                            float h8[8];
                            ld_h8(sX, r, 4 * pc + g, h8);
#pragma unroll
                            for (int c = 0; c < 8; ++c) e[8 * g + c] = h8[c];
                        }
                    };
                    // Q_S is final: Q_S -> Y (right operand), T0 -> TMEM (left;
                    // the band path reads Q_S's rows from Y instead)
                    auto finish_q = [&](int pp, float (&q)[32]) {
                        const int pc = pc0 + pp;
#pragma unroll
                        for (int jj = 0; jj < 32; ++jj)
                            if (!in_chunk(pc * 32 + jj)) q[jj] = 0.f;
                        if (kBandable && band) {
                            if (pc == (i >> 5)) {
#pragma unroll
                                for (int jj = 0; jj < 32; ++jj)
                                    if (pc * 32 + jj == i) q[jj] = 1.f;        // I + Q_S
                            }
                            st_op32<false>(sY, r, pc, q);
                            return;
                        }
                        st_op32<false>(sY, r, pc, q);
                        float t[32];
                        t0_get(pp, t, T0);
                        tmem_st_h16(tA + pc * 16, t);
                    };
                    if (pS >= 2) {
                        cpublish(true);
                        cchain_t(sX);                                    // E E
                        if (!cwait()) ok = false;
#pragma unroll
                        for (int pp = 0; pp < PPT; ++pp) {
                            const int pc = pc0 + pp;
                            float v[32], e[32];
                            tmem_ld32(tD + pc * 32, v);
                            e_row(pc, e);
#pragma unroll
                            for (int jj = 0; jj < 32; ++jj) e[jj] += v[jj];     // F
                            if (pS == 2) {
                                finish_q(pp, e);                            // Q_2 = F
                            } else {
#pragma unroll
                                for (int jj = 0; jj < 32; ++jj)
                                    if (!in_chunk(pc * 32 + jj)) v[jj] = e[jj] = 0.f;
                                st_op32<false>(sY, r, pc, v);               // E^2
                                tmem_st_h16(tF + pc * 16, e);             // F
                                if (pS % 2 == 0) tmem_st_h16(tA + pc * 16, e);   // Q_2
                            }
                        }
                        int m = pS % 2 == 0 ? 2 : 1;
                        bool first = true;
                        while (pS >= 3 && m + 2 <= pS) {
                            cpublish(first);
                            first = false;
                            cchain_t(sY);                                // Q_m E^2
                            if (!cwait()) ok = false;
                            m += 2;
#pragma unroll
                            for (int pp = 0; pp < PPT; ++pp) {
                                const int pc = pc0 + pp;
                                float v[32], f[32];
                                tmem_ld32(tD + pc * 32, v);
                                tmem_ld_h16(tF + pc * 16, f);
#pragma unroll
                                for (int jj = 0; jj < 32; ++jj) v[jj] += f[jj];     // Q_m
                                if (m == pS) {
                                    finish_q(pp, v);
                                } else {
#pragma unroll
                                    for (int jj = 0; jj < 32; ++jj)
                                        if (!in_chunk(pc * 32 + jj)) v[jj] = 0.f;
                                    tmem_st_h16(tA + pc * 16, v);
                                }
                            }
                        }
                    }
                    if (kBandable && band) {
                        // T = T0 (I + Q_S): T[i][j] = sum_{e<=N} T0[i][i-e] (I + Q_S)[i-e][j],
                        // the rows of I + Q_S (fp16) from Y and row
                        // i's band of T0 back from bT
                        bar_sync(cbar, 128);                              // I + Q_S written
                        band_row();
                        float t[32];
#pragma unroll
                        for (int jj = 0; jj < 32; ++jj) t[jj] = 0.f;
#pragma unroll
                        for (int e = 0; e <= kBandMax; ++e) {
                            if (e > pN) break;
                            if (i - e < 0) continue;
#pragma unroll
                            for (int g = 0; g < 4; ++g) {
                                float h8[8];
                                ld_h8(sY, r - e, 4 * pc0 + g, h8);
#pragma unroll
                                for (int c = 0; c < 8; ++c) t[8 * g + c] = fmaf(tb[e], h8[c], t[8 * g + c]);
                            }
                        }
                        if (pG) {
                            t0_put(0, t, T0);
                        } else {                                  // WY's operand T diag(beta), bf16
                            if (p.Tout && valid) {
                                float* dst = p.Tout + cidx * KC * KC + rin * KC + pc0 * 32;
#pragma unroll
                                for (int q = 0; q < 8; ++q)
                                    reinterpret_cast<float4*>(dst)[q] =
                                        make_float4(t[4 * q], t[4 * q + 1], t[4 * q + 2], t[4 * q + 3]);
                            }
                            const float* bcol = sb + blk * KB + pc0 * 32;
#pragma unroll
                            for (int jj = 0; jj < 32; ++jj) t[jj] *= bcol[jj];
                            st_op32<true>(sX, r, pc0, t);
                        }
                    } else {
                    cpublish(true);
                    cchain_t(sY);                                        // T0 Q_S
                    if (!cwait()) ok = false;
#pragma unroll
                    for (int pp = 0; pp < PPT; ++pp) {
                        const int pc = pc0 + pp;
                        float v[32], t[32];
                        tmem_ld32(tD + pc * 32, v);
                        t0_get(pp, t, T0);
#pragma unroll
                        for (int jj = 0; jj < 32; ++jj)
                            if (in_chunk(pc * 32 + jj)) t[jj] += v[jj];          // T = T0 + T0 Q
                        t0_put(pp, t, T0);
                    }
                    }
                }
            }
            // ---- T out ----
            if (inv_only(MODE)) {
                // through the Aop | Y buffers as fp32 128-byte swizzled boxes, TMA store
                bar_sync(bar_id, 256);                 // this tile's Aop / Y operands are read
                const uint32_t st0 = su32(sAop);
#pragma unroll
                for (int pp = 0; pp < PPT; ++pp) {
                    const int pc = pc0 + pp;
                    if (piece_in_chunk(pc)) {
                        float t[32];
                        t0_get(pp, t, T0);
                        const uint32_t rb = st0 + (uint32_t)(((pc * 32 - cl) >> 5) * 16384 + r * 128);
#pragma unroll
                        for (int c4 = 0; c4 < 8; ++c4)
                            sts128(rb + ((c4 ^ (r & 7)) << 4),
                                   make_uint4(__float_as_uint(t[4 * c4]), __float_as_uint(t[4 * c4 + 1]),
                                              __float_as_uint(t[4 * c4 + 2]),
                                              __float_as_uint(t[4 * c4 + 3])));
                    }
                }
                fence_async_smem();
                tc_fence_before();
                bar_sync(bar_id, 256);
                if (leader && live()) {
#pragma unroll 1
                    for (int b = 0; b < KC / 32; ++b)
                        tma_store_2d(&mW, 32 * b, (int)row0, sAop + b * 16384);
                    bulk_commit();
                }
            } else if (p.Tout && !(band && pS > 0 && !pG)) {
#pragma unroll
                for (int pp = 0; pp < PPT; ++pp) {
                    const int pc = pc0 + pp;
                    if (valid && piece_in_chunk(pc)) {
                        float t[32];
                        t0_get(pp, t, T0);
                        float* dst = p.Tout + cidx * KC * KC + rin * KC + (pc * 32 - cl);
#pragma unroll
                        for (int q = 0; q < 8; ++q)
                            reinterpret_cast<float4*>(dst)[q] =
                                make_float4(t[4 * q], t[4 * q + 1], t[4 * q + 2], t[4 * q + 3]);
                    }
                }
            }
        }

        if (is_fused(MODE) || MODE == kWY) {
            // ---- WY: T diag(beta [exp g]) -> X (bf16), T diag(beta) -> Y ----
            release_staging(n);
            const float* bcol = sb + blk * KB;
            const float* gcol = sg + blk * KB;
#pragma unroll
            for (int pp = 0; pp < PPT; ++pp) {
                if (band && pS > 0 && !pG) break;    // written by the band product
                const int pc = pc0 + pp;
                float v[32], t[32];
                t0_get(pp, t, T0);
#pragma unroll
                for (int jj = 0; jj < 32; ++jj) {
                    const int j = pc * 32 + jj;
                    const float b = bcol[j];
                    v[jj] = t[jj] * (pG ? b * exp_e(gcol[j]) : b);
                }
                st_op32<true>(sX, r, pc, v);
                if (pG) {
#pragma unroll
                    for (int jj = 0; jj < 32; ++jj) v[jj] = t[jj] * bcol[pc * 32 + jj];
                    st_op32<true>(sY, r, pc, v);
                }
            }
            if (uses_V(MODE) && !(live() && mbar_wait(&ctrl->fullV[s], use_par, &ctrl->timeout_ns))) fail_wait();
            publish(true);
            if (leader && live()) {
                constexpr uint32_t id = idesc_f16(1, 1, 0, KB, 128);
                const uint32_t kb0 = su32(sK), vb0 = su32(sV), xb0 = su32(sX);
                const uint32_t ub0 = su32(pG ? sY : sX);
                // W^T first, with its own commit: the slot's next K tile can
                // start loading while the U^T products still run
#pragma unroll 1
                for (int c = 0; c < NCH; ++c) {
#pragma unroll 1
                    for (int kk = 0; kk < KB / 16; ++kk) {
                        const uint32_t ao = (c * KB + kk * 16) * 128;
                        const uint32_t bo = (c * KB) * 128 + (kk >> 2) * (kRows * 128) +
                                            (kk & 3) * 32;
                        mma_ss(tm + c * KB, sdesc(kb0 + ao, kRows * 128, 1024),
                               sdesc(xb0 + bo, 16, 1024), id, kk > 0);
                    }
                }
                mma_commit(&ctrl->wdone[s]);
#pragma unroll 1
                for (int c = 0; c < NCH; ++c) {
#pragma unroll 1
                    for (int kk = 0; kk < KB / 16; ++kk) {
                        const uint32_t ao = (c * KB + kk * 16) * 128;
                        const uint32_t bo = (c * KB) * 128 + (kk >> 2) * (kRows * 128) +
                                            (kk & 3) * 32;
                        mma_ss(tm + 128 + c * KB, sdesc(vb0 + ao, kRows * 128, 1024),
                               sdesc(ub0 + bo, 16, 1024), id, kk > 0);
                    }
                }
                mma_commit(&ctrl->mma[s]);
                if (live() && mbar_wait(&ctrl->wdone[s], use_par, &ctrl->timeout_ns)) issue_k(n + NS);   // K is free
                else fail_wait();
            }
            if (!wait_mma()) ok = false;
            // Lane d of the W^T / U^T accumulators is head-dim column d and
            // accumulator column x is tile row x.  Warp (quarter q, half h)
            // moves d in [32q, 32q + 32) x rows [64h, 64h + 64): 16x256b TMEM
            // loads give each thread (d, x..x+1) pairs of 8 x 8 blocks, and
            // stmatrix .trans writes the blocks transposed, one 16-byte row
            // segment (8 d of one tile row) per address, into the W staging
            // tile and the V tile in the TMA layout.
            {
                const uint32_t wst = su32(sWst), vst = su32(sV);
                const int mq = lane >> 3, mr = lane & 7;   // stmatrix: matrix, row of this address
                auto pk = [](uint32_t lo, uint32_t hi) {
                    return pack_b2(__uint_as_float(lo), __uint_as_float(hi));
                };
#pragma unroll 1
                for (int it2 = 0; it2 < 4; ++it2) {       // two 16-lane halves per TMEM wait
                    const int x0 = h * 64 + it2 * 16;
                    uint32_t wa[2][4], wb[2][4], ua[2][4], ub[2][4];
#pragma unroll
                    for (int hb = 0; hb < 2; ++hb) {
                        const uint32_t ta = tl + ((uint32_t)(16 * hb) << 16) + x0;
                        tmem_ld_16x256b(ta, wa[hb]);
                        tmem_ld_16x256b(ta + 8, wb[hb]);
                        tmem_ld_16x256b(ta + 128, ua[hb]);
                        tmem_ld_16x256b(ta + 136, ub[hb]);
                    }
                    tmem_wait_ld();
#pragma unroll
                    for (int hb = 0; hb < 2; ++hb) {
                        const int db = (warp & 3) * 32 + 16 * hb;
                        const int x = x0 + 8 * (mq >> 1) + mr, d = db + 8 * (mq & 1);
                        const uint32_t off = (uint32_t)((d >> 6) * (kRows * 128) + x * 128 +
                                                        ((((d & 63) >> 3) ^ (x & 7)) << 4));
                        stmatrix_x4_trans(wst + off, pk(wa[hb][0], wa[hb][1]), pk(wa[hb][2], wa[hb][3]),
                                          pk(wb[hb][0], wb[hb][1]), pk(wb[hb][2], wb[hb][3]));
                        stmatrix_x4_trans(vst + off, pk(ua[hb][0], ua[hb][1]), pk(ua[hb][2], ua[hb][3]),
                                          pk(ub[hb][0], ub[hb][1]), pk(ub[hb][2], ub[hb][3]));
                    }
                }
            }
            fence_async_smem();
            tc_fence_before();
            bar_sync(bar_id, 256);
            if (leader && live()) {
                const int y = (int)row0;
                tma_store_2d(&mW, 0, y, sWst);
                tma_store_2d(&mW, 64, y, sWst + kRows * 128);
                tma_store_2d(&mU, 0, y, sV);
                tma_store_2d(&mU, 64, y, sV + kRows * 128);
                bulk_commit();
            }
            staged_free = false;
            continue;
        }
        tc_fence_before();
        bar_sync(bar_id, 256);                 // accumulators free for the next tile
    }
    if (!ok || !live()) {
        // Drain (bounded, deaf to the abort flag): one more commit by each
        // issuing thread tracks every product it started, so TMEM is not freed
        // under one; the loads the leader started land before the CTA's shared
        // memory goes away.
        if (leader || cleader) {
            uint64_t* dm = &ctrl->drain[s][leader ? 0 : 1];
            mma_commit(dm);
            mbar_wait(dm, 0, &ctrl->timeout_ns);
        }
        if (leader) {
            if (k_issued > 0) mbar_wait(&ctrl->fullK[s], (uint32_t)((k_issued - 1) & 1), &ctrl->timeout_ns);
            if (v_issued > 0) mbar_wait(&ctrl->fullV[s], (uint32_t)((v_issued - 1) & 1), &ctrl->timeout_ns);
        }
    }
    if (leader) bulk_wait_all();                   // W, U stores complete
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem_base, kTmemCols);
    }
}

// ------------------------------------------------------------------------- //
// The chunk-wise forward's output pass on the tensor cores (k = 64, bf16 data)
// ------------------------------------------------------------------------- //
// O = s (diag(gamma) Q S_c^T + (Q K^T (.) Gamma (.) L) V~) per chunk, with
// gamma_i = e^{g_i}, Gamma_ij = e^{g_i - g_j}, L the lower triangle including the
// diagonal, S_c the chunk's start state (fp16, from the state recurrence), V~
// the corrected values (fp16) and s = 1 / ||q_i|| when the queries come raw
// (normalised here, since s scales a whole row of O), else 1.  A tile is two
// chunks (128 token rows) and one CTA of 8 warps per SM works through tiles:
//   G  = Q K^T                (bf16; M = N = 128, K = d)     -> TMEM [0, 128)
//   epilogue: A2 = G (.) Gamma (.) L on the row's own chunk block and 0 on the
//             other (fp16, into K's buffer); Q to fp16 in place
//   P0 = Q S_0^T, P1 = Q S_1^T (fp16; one product per chunk's start state)
//                                                            -> [128, 256), [256, 384)
//   Oi = A2 V~                (fp16; K = the tile's 128 tokens) -> [0, 128)
//   epilogue: O = s (gamma P_c + Oi) in bf16 through V~'s buffer, TMA store.
// Thread (r, h) owns tile row r (its TMEM lane) and column half h.  Waits are
// bounded as in the chunk kernel: after one runs out nobody leaves the tile
// early, no work is started, and the CTA stops together at the next tile.
struct ParamsOut {
    int64_t rows;        // B*H*T
    int64_t nchunks;     // B*H*T / 64
    int ntiles;
    int normalize_q;
    int* status;
};
constexpr int kOutThreads = 256;
constexpr int kOutOp = kRows * kD * 2;               // one [2][128][64] 16-bit operand: 32 KB
// Q | K, then A2 | V~, then O | S_0 | S_1 | g | the row norms' halves | control
constexpr int kOutSmem = 5 * kOutOp + kRows * 4 + 2 * kRows * 4;

struct __align__(8) CtrlOut {
    uint64_t full;       // Q, K, S_0, S_1, g of the tile landed
    uint64_t fullV;      // V~ landed
    uint64_t mma;        // the products completed
    uint64_t drain;      // after an expired wait: the leader's products are done
    uint32_t tmem;
    int abort;
};

__global__ void __launch_bounds__(kOutThreads, 1)
k_output_tc(const __grid_constant__ CUtensorMap mQ, const __grid_constant__ CUtensorMap mK,
         const __grid_constant__ CUtensorMap mVt, const __grid_constant__ CUtensorMap mS,
         const __grid_constant__ CUtensorMap mG, const __grid_constant__ CUtensorMap mO,
         const ParamsOut p) {
    extern __shared__ __align__(1024) uint8_t smem[];
    if ((su32(smem) & 1023u) != 0) {
        if (threadIdx.x == 0) raise_status(p.status, kStatusSmemAlign);
        return;
    }
    uint8_t* sQ = smem;
    uint8_t* sK = smem + kOutOp;                     // K, then A2
    uint8_t* sV = smem + 2 * kOutOp;                 // V~, then O
    uint8_t* sS0 = smem + 3 * kOutOp;
    uint8_t* sS1 = smem + 4 * kOutOp;
    float* sg = reinterpret_cast<float*>(smem + 5 * kOutOp);
    float* sqs = sg + kRows;                          // [2][128] halves of ||q||^2
    CtrlOut* ctrl = reinterpret_cast<CtrlOut*>(smem + kOutSmem);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int h = warp >> 2;
    const int r = ((warp & 3) << 5) | lane;
    const int c = r >> 6, i = r & 63;                 // chunk of the row in the tile, row in it
    const bool leader = threadIdx.x == 0;
    if (leader) {
        mbar_init(&ctrl->full, 1);
        mbar_init(&ctrl->fullV, 1);
        mbar_init(&ctrl->mma, 1);
        mbar_init(&ctrl->drain, 1);
        ctrl->abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 0) tmem_alloc(&ctrl->tmem, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = ctrl->tmem;
    const uint32_t tl = tm + ((uint32_t)((warp & 3) * 32) << 16);
    const volatile int* const abortp = &ctrl->abort;
    auto live = [&]() { return *abortp == 0; };
    auto fail_wait = [&]() {
        atomicExch(&ctrl->abort, 1);
        raise_status(p.status, kStatusTimeout);
    };
    uint32_t mma_phase = 0;
    auto wait_mma = [&]() {
        if (!(live() && mbar_wait(&ctrl->mma, mma_phase))) fail_wait();
        mma_phase ^= 1;
        tc_fence_after();
    };
    int main_issued = 0, v_issued = 0;
    auto issue_main = [&](int tile) {
        if (tile >= p.ntiles || !live()) return;
        ++main_issued;
        const int y = tile * kRows;
        const int ys = 2 * tile * kRows;              // S rows of the tile's first chunk
        mbar_expect_tx(&ctrl->full, 4 * kOutOp + kRows * 4);
        tma_load_2d(sQ, &mQ, 0, y, &ctrl->full);
        tma_load_2d(sQ + kRows * 128, &mQ, 64, y, &ctrl->full);
        tma_load_2d(sK, &mK, 0, y, &ctrl->full);
        tma_load_2d(sK + kRows * 128, &mK, 64, y, &ctrl->full);
        tma_load_2d(sS0, &mS, 0, ys, &ctrl->full);
        tma_load_2d(sS0 + kRows * 128, &mS, 64, ys, &ctrl->full);
        tma_load_2d(sS1, &mS, 0, ys + kRows, &ctrl->full);
        tma_load_2d(sS1 + kRows * 128, &mS, 64, ys + kRows, &ctrl->full);
        tma_load_1d(sg, &mG, y, &ctrl->full);
    };
    auto issue_v = [&](int tile) {
        if (tile >= p.ntiles || !live()) return;
        ++v_issued;
        const int y = tile * kRows;
        mbar_expect_tx(&ctrl->fullV, kOutOp);
        tma_load_2d(sV, &mVt, 0, y, &ctrl->fullV);
        tma_load_2d(sV + kRows * 128, &mVt, 64, y, &ctrl->fullV);
    };
    if (leader) {
        issue_main(blockIdx.x);
        issue_v(blockIdx.x);
    }
    bool ok = true, stored = false;
    for (int n = 0;; ++n) {
        const int tile = blockIdx.x + n * gridDim.x;
        if (tile >= p.ntiles) break;
        const uint32_t par = (uint32_t)(n & 1);
        if (!(live() && mbar_wait(&ctrl->full, par))) fail_wait();
        if (bar_sync_or(1, kOutThreads, !live())) { ok = false; break; }
        if (leader && live()) {
            if (stored) {                              // the last O store has read V~'s buffer
                bulk_wait_read();
                issue_v(tile);
            }
            tc_fence_after();
            constexpr uint32_t id = idesc_f16(1, 0, 0, 128, 128);     // bf16, both K-major
            const uint32_t qb = su32(sQ), kb = su32(sK);
#pragma unroll 1
            for (int kk = 0; kk < kD / 16; ++kk) {
                const uint32_t o = (kk >> 2) * (kRows * 128) + (kk & 3) * 32;
                mma_ss(tm, sdesc(qb + o, 16, 1024), sdesc(kb + o, 16, 1024), id, kk > 0);
            }
            mma_commit(&ctrl->mma);
        }
        wait_mma();
        // ---- A2 = G (.) Gamma (.) L (fp16) into K's buffer; Q to fp16 in place ----
        const float gi = sg[r];
        {
            const float* gcol = sg + 64 * c + 32 * h;
            float v[32];
            if (32 * h > i) {                          // the whole piece lies above the diagonal
#pragma unroll
                for (int jj = 0; jj < 32; ++jj) v[jj] = 0.f;
            } else {
                tmem_ld32(tl + 64 * c + 32 * h, v);
#pragma unroll
                for (int jj = 0; jj < 32; ++jj)
                    v[jj] = 32 * h + jj <= i ? v[jj] * exp_e(gi - gcol[jj]) : 0.f;
            }
            st_op32<false>(sK, r, 2 * c + h, v);
#pragma unroll
            for (int jj = 0; jj < 32; ++jj) v[jj] = 0.f;
            st_op32<false>(sK, r, 2 * (1 - c) + h, v);   // the other chunk's keys: zero
        }
        {
            float ss = 0.f;
            const uint32_t qb = su32(sQ);
#pragma unroll
            for (int q = 8 * h; q < 8 * h + 8; ++q) {
                const uint32_t a = qb + op_off(r, q);
                const uint4 u = lds128(a);
                const uint32_t w4[4] = {u.x, u.y, u.z, u.w};
                uint32_t o4[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float lo = __uint_as_float(w4[e] << 16);
                    const float hi = __uint_as_float(w4[e] & 0xffff0000u);
                    ss = fmaf(lo, lo, fmaf(hi, hi, ss));
                    o4[e] = pack_h2(lo, hi);
                }
                sts128(a, make_uint4(o4[0], o4[1], o4[2], o4[3]));
            }
            sqs[h * kRows + r] = ss;
        }
        fence_async_smem();
        tc_fence_before();
        bar_sync(1, kOutThreads);
        tc_fence_after();
        if (leader && live()) {
            if (!(mbar_wait(&ctrl->fullV, (uint32_t)((v_issued - 1) & 1)))) fail_wait();
            if (live()) {
                constexpr uint32_t idk = idesc_f16(0, 0, 0, 128, 128);   // fp16, both K-major
                constexpr uint32_t idm = idesc_f16(0, 0, 1, 128, 128);   // fp16, B MN-major
                const uint32_t qb = su32(sQ), ab = su32(sK), vb = su32(sV);
                const uint32_t s0 = su32(sS0), s1 = su32(sS1);
#pragma unroll 1
                for (int kk = 0; kk < kD / 16; ++kk) {
                    const uint32_t o = (kk >> 2) * (kRows * 128) + (kk & 3) * 32;
                    const uint64_t a = sdesc(qb + o, 16, 1024);
                    mma_ss(tm + 128, a, sdesc(s0 + o, 16, 1024), idk, kk > 0);
                    mma_ss(tm + 256, a, sdesc(s1 + o, 16, 1024), idk, kk > 0);
                    mma_ss(tm, sdesc(ab + o, 16, 1024), sdesc(vb + kk * 2048, kRows * 128, 1024),
                           idm, kk > 0);
                }
                mma_commit(&ctrl->mma);
            }
        }
        wait_mma();
        if (leader) issue_main(tile + gridDim.x);      // Q, K, S, g are read
        // ---- O = s (gamma P_c + Oi), bf16, into V~'s buffer ----
        {
            const float ss = sqs[r] + sqs[kRows + r];
            const float sc = p.normalize_q ? (ss > 0.f ? rsqrtf(ss) : 0.f) : 1.f;
            const float gam = exp_e(gi);
#pragma unroll
            for (int pc = 0; pc < 2; ++pc) {
                const int col = 64 * h + 32 * pc;
                float pv[32], ov[32];
                tmem_ld32(tl + 128 + 128 * c + col, pv);
                tmem_ld32(tl + col, ov);
#pragma unroll
                for (int jj = 0; jj < 32; ++jj) ov[jj] = sc * fmaf(gam, pv[jj], ov[jj]);
                st_op32<true>(sV, r, 2 * h + pc, ov);
            }
        }
        fence_async_smem();
        tc_fence_before();
        bar_sync(1, kOutThreads);
        if (leader && live()) {
            tma_store_2d(&mO, 0, tile * kRows, sV);
            tma_store_2d(&mO, 64, tile * kRows, sV + kRows * 128);
            bulk_commit();
        }
        stored = true;
    }
    if (!ok || !live()) {                              // drain, bounded, deaf to the flag
        if (leader) {
            mma_commit(&ctrl->drain);
            mbar_wait(&ctrl->drain, 0);
            if (main_issued > 0) mbar_wait(&ctrl->full, (uint32_t)((main_issued - 1) & 1));
            if (v_issued > 0) mbar_wait(&ctrl->fullV, (uint32_t)((v_issued - 1) & 1));
        }
    }
    if (leader) bulk_wait_all();
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tm, 512);
    }
}

// ------------------------------------------------------------------------- //
// INT8 truncated Neumann series on the tensor cores (k = 64)
// ------------------------------------------------------------------------- //
// Same tile / slot structure as k_chunk_tc: a tile stacks two 64-token chunks,
// acc_n = q_{n-1} q_1 is one M=128, N=128, K=64 tcgen05.mma of kind::i8
// (s8 x s8 -> s32 in TMEM), and each row reads its chunk's diagonal block.  The
// per-chunk maxima are reduced across the 4 warps that hold a chunk through
// shared memory.  Every float32 operation is the IEEE-rounded one of the scheme
// in gdn.h, in that order, so codes, accumulators, scales and T are bit-exact.
__host__ __device__ constexpr uint32_t idesc_i8(int N, int M) {
    // D s32 (2), A and B signed 8-bit (1), A K-major, B MN-major
    return (2u << 4) | (1u << 7) | (1u << 10) | (0u << 15) | (1u << 16) |
           ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
__device__ __forceinline__ void mma_i8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       uint32_t acc) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
// clamp(rint(x * r), +-127): one conversion with round to nearest even (it
// saturates, so the integer clamp gives what a clamp in float would).  With
// r = 0 (a zero maximum: every x is zero) the code is 0.
__device__ __forceinline__ int quant_i8(float x, float r) {
    const int q = __float2int_rn(__fmul_rn(x, r));
    return min(max(q, -127), 127);
}
// The same code with no conversion instruction, also as a float (qf): y is
// clamped to +-127 first (rounding then clamping gives the same code), and
// adding 1.5 * 2^23 rounds it to an integer with ties to even, the sum's
// low mantissa bits being the code.  The two forms differ only where x * r
// is NaN: a zero entry of a chunk whose maximum is below 127 / FLT_MAX
// (~3.7e-37), where r = 127 / max overflows (quant_i8 gives 0, this +-127).
__device__ __forceinline__ int quant_i8f(float x, float r, float& qf) {
    const float y = fminf(fmaxf(__fmul_rn(x, r), -127.f), 127.f);
    const float t = __fadd_rn(y, 12582912.f);
    qf = __fsub_rn(t, 12582912.f);
    return __float_as_int(t) - 0x4B400000;
}
// float(a) for |a| < 2^22 without a conversion instruction: the bit pattern
// of 1.5 * 2^23 plus a is the float 1.5 * 2^23 + a
__device__ __forceinline__ float i2f_small(int a) {
    return __fsub_rn(__int_as_float(a + 0x4B400000), 12582912.f);
}
// 32 int8 codes -> two 16-byte groups of a 128-byte swizzled row
__device__ __forceinline__ void st_i8x32(uint8_t* buf, int row, int q0, const int (&c)[32]) {
#pragma unroll
    for (int g = 0; g < 2; ++g) {
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int b = 16 * g + 4 * k;
            w[k] = (uint32_t)(c[b] & 0xff) | ((uint32_t)(c[b + 1] & 0xff) << 8) |
                   ((uint32_t)(c[b + 2] & 0xff) << 16) | ((uint32_t)(c[b + 3] & 0xff) << 24);
        }
        const int q = q0 + g;
        *reinterpret_cast<uint4*>(buf + row * 128 + (((q & 7) ^ (row & 7)) << 4)) =
            make_uint4(w[0], w[1], w[2], w[3]);
    }
}

struct ParamsI8 {
    int64_t rows;
    int ntiles;
    int N, mask;
    int S;               // residual steps (the RES instance)
    const float* A;
    float* T;
    int8_t* q;
    int32_t* acc;
    float* scale;
    int* status;
};

constexpr int kI8Slots = 2;
constexpr int kI8OpBytes = kRows * 128;            // 16 KB, rows at a 128-byte pitch
constexpr int kI8BBytes = 64 * 128;                // 8 KB: K = 64 rows of 128 codes
constexpr int kI8Stage = kRows * 64 * 4;           // 32 KB: the next tile's A (fp32, swizzled)
constexpr int kI8SlotBytes = kI8OpBytes + kI8BBytes + kI8Stage;

// RES: the residual correction in int8 products follows the series (S >= 1)
template <bool RES, int SN, int SS>
__global__ void __launch_bounds__(256 * kI8Slots, 1)
k_neumann_i8_tc(const __grid_constant__ CUtensorMap mA, const ParamsI8 p) {
    constexpr int KC = 64;
    extern __shared__ __align__(1024) uint8_t smem[];
    if ((su32(smem) & 1023u) != 0) {
        if (threadIdx.x == 0) raise_status(p.status, kStatusSmemAlign);
        return;
    }
    struct __align__(8) CtrlI8 {
        uint64_t mma[kI8Slots];
        uint64_t full[kI8Slots];                   // the slot's staged A landed
        uint64_t drain[kI8Slots];                  // after an expired wait: the slot's products are done
        uint32_t tmem;
        int abort;
        float red_f[kI8Slots][2][4];
        int red_i[kI8Slots][2][4];
    };
    CtrlI8* ctrl = reinterpret_cast<CtrlI8*>(smem + kI8Slots * kI8SlotBytes);
    // the series order and the residual steps: the call's, or fixed at compile
    // time in an instance specialised for one setting (SN > 0, SS >= 0)
    const int pN = SN > 0 ? SN : p.N;
    const int pS = SS >= 0 ? SS : p.S;
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kI8Slots; ++s) {
            mbar_init(&ctrl->mma[s], 1);
            mbar_init(&ctrl->full[s], 1);
            mbar_init(&ctrl->drain[s], 1);
        }
        ctrl->abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 0) tmem_alloc(&ctrl->tmem, 256);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = ctrl->tmem;

    const int s = warp / 8;
    const int h = (warp % 8) / 4;
    const int r = ((warp & 3) << 5) | lane;
    const int c = r / KC;                          // chunk of this row in the tile
    const int i = r % KC;
    const int wq = ((warp & 3) & 1) * 2 + h;       // this warp's slot among its chunk's 4 warps
    const int jmin = p.mask ? i - pN : -KC;
    uint8_t* sA = smem + s * kI8SlotBytes;
    uint8_t* sB = sA + kI8OpBytes;
    uint8_t* sStage = sB + kI8BBytes;
    const uint32_t tm = tmem_base + (uint32_t)(s * 128);
    const uint32_t tD = tm + ((uint32_t)((warp & 3) * 32) << 16) + c * KC + 32 * h;
    const bool leader = (warp % 8) == 0 && lane == 0;
    const int bar_id = 1 + s;
    uint32_t mma_phase = 0;
    bool ok = true;

    // maximum over the chunk held by this row's 4 warps
    auto chunk_max_f = [&](float v) {
        for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
        if (lane == 0) ctrl->red_f[s][c][wq] = v;
        bar_sync(bar_id, 256);
        const float m = fmaxf(fmaxf(ctrl->red_f[s][c][0], ctrl->red_f[s][c][1]),
                              fmaxf(ctrl->red_f[s][c][2], ctrl->red_f[s][c][3]));
        return m;
    };
    auto chunk_max_i = [&](int v) {
        for (int o = 16; o; o >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, o));
        if (lane == 0) ctrl->red_i[s][c][wq] = v;
        bar_sync(bar_id, 256);
        return max(max(ctrl->red_i[s][c][0], ctrl->red_i[s][c][1]),
                   max(ctrl->red_i[s][c][2], ctrl->red_i[s][c][3]));
    };
    // the same, with the slot's decision to stop taken at its barrier (an OR
    // over the threads' view of the abort flag)
    auto chunk_max_i_stop = [&](int v, bool& stop) {
        for (int o = 16; o; o >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, o));
        if (lane == 0) ctrl->red_i[s][c][wq] = v;
        stop = bar_sync_or(bar_id, 256, *(volatile int*)&ctrl->abort != 0);
        return max(max(ctrl->red_i[s][c][0], ctrl->red_i[s][c][1]),
                   max(ctrl->red_i[s][c][2], ctrl->red_i[s][c][3]));
    };

    // the slot's leader stages A of the slot's tile n: two 32-column boxes
    int a_issued = 0;
    auto issue_a = [&](int n) {
        const int tile = blockIdx.x + n * gridDim.x;
        if (tile >= p.ntiles) return;
        ++a_issued;
        mbar_expect_tx(&ctrl->full[s], kI8Stage);
        tma_load_2d(sStage, &mA, 0, tile * kRows, &ctrl->full[s]);
        tma_load_2d(sStage + 16384, &mA, 32, tile * kRows, &ctrl->full[s]);
    };
    if (leader) issue_a(s);

    for (int n = s;; n += kI8Slots) {
        const int tile = blockIdx.x + n * gridDim.x;
        if (tile >= p.ntiles) break;
        const int64_t grow = (int64_t)tile * kRows + r;
        const bool valid = grow < p.rows;
        const int64_t cidx = grow / KC, rin = grow % KC;
        if (!mbar_wait(&ctrl->full[s], (uint32_t)((n / kI8Slots) & 1))) {
            atomicExch(&ctrl->abort, 1);
            raise_status(p.status, kStatusTimeout);
        }
        float a[32];                                // rows past the end were zero-filled
        {
            const uint32_t rb = su32(sStage) + (uint32_t)(h * 16384 + r * 128);
#pragma unroll
            for (int c4 = 0; c4 < 8; ++c4) {
                uint32_t u0, u1, u2, u3;
                asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(u0), "=r"(u1), "=r"(u2), "=r"(u3)
                             : "r"(rb + ((c4 ^ (r & 7)) << 4)));
                a[4 * c4] = __uint_as_float(u0);
                a[4 * c4 + 1] = __uint_as_float(u1);
                a[4 * c4 + 2] = __uint_as_float(u2);
                a[4 * c4 + 3] = __uint_as_float(u3);
            }
        }
        fence_async_smem();
        // previous tile's reads of sA, sB, red and the stage done; the slot
        // decides together whether to stop (an OR over its threads' view of
        // the CTA's abort flag, which the other slot may raise at any time)
        if (bar_sync_or(bar_id, 256, *(volatile int*)&ctrl->abort != 0)) { ok = false; break; }
        if (leader) issue_a(n + kI8Slots);
        float amax = 0.f;
#pragma unroll
        for (int jj = 0; jj < 32; ++jj) {
            const int j = 32 * h + jj;
            if constexpr (!RES) {
                if (j < jmin) a[jj] = 0.f;             // P_1 = M . A
            }
            amax = fmaxf(amax, fabsf(j < jmin ? 0.f : a[jj]));
        }
        amax = chunk_max_f(amax);
        const float r1 = amax > 0.f ? __fdiv_rn(127.f, amax) : 0.f;
        const float s1 = amax > 0.f ? __fdiv_rn(amax, 127.f) : 0.f;
        int q[32];
        float t[32];
#pragma unroll
        for (int jj = 0; jj < 32; ++jj) {
            const int j = 32 * h + jj;
            float qf;
            q[jj] = quant_i8f(j < jmin ? 0.f : a[jj], r1, qf);
            t[jj] = __fadd_rn(i == j ? 1.f : 0.f, __fmul_rn(s1, qf));
        }
        st_i8x32(sA, r, 2 * h, q);                     // q_1 as the left operand
        st_i8x32(sB, i, 4 * c + 2 * h, q);             // q_1 as the right operand
        if (valid) {
            const int64_t base = (cidx * pN * KC + rin) * KC + 32 * h;
            if (p.q) {
#pragma unroll
                for (int jj = 0; jj < 32; jj += 4)
                    *reinterpret_cast<char4*>(p.q + base + jj) =
                        make_char4((signed char)q[jj], (signed char)q[jj + 1],
                                   (signed char)q[jj + 2], (signed char)q[jj + 3]);
            }
            if (p.acc) {
#pragma unroll
                for (int jj = 0; jj < 32; jj += 4)
                    *reinterpret_cast<int4*>(p.acc + base + jj) = make_int4(0, 0, 0, 0);
            }
            if (p.scale && rin == 0 && h == 0) p.scale[cidx * pN] = s1;
        }
        float sprev = s1;
        for (int pw = 1; pw < pN; ++pw) {
            fence_async_smem();
            tc_fence_before();
            bar_sync(bar_id, 256);
            tc_fence_after();
            if (leader) {
                constexpr uint32_t id = idesc_i8(128, 128);
#pragma unroll
                for (int kk = 0; kk < KC / 32; ++kk) {
                    const uint64_t ad = sdesc(su32(sA) + kk * 32, 16, 1024);
                    const uint64_t bd = sdesc(su32(sB) + kk * 32 * 128, 16, 1024);
                    mma_i8(tm, ad, bd, id, kk > 0);
                }
                mma_commit(&ctrl->mma[s]);
            }
            bool good = mbar_wait(&ctrl->mma[s], mma_phase);
            mma_phase ^= 1;
            if (!good) {
                atomicExch(&ctrl->abort, 1);
                raise_status(p.status, kStatusTimeout);
            }
            tc_fence_after();
            uint32_t raw[32];
            tmem_ld32_async(tD, raw);
            tmem_wait_ld();
            int accv[32];
            int m = 0;
#pragma unroll
            for (int jj = 0; jj < 32; ++jj) {
                const int j = 32 * h + jj;
                accv[jj] = (j < jmin) ? 0 : (int)raw[jj];
                m = max(m, abs(accv[jj]));
            }
            bool stop;
            m = chunk_max_i_stop(m, stop);
            if (stop) { ok = false; break; }
            const float mf = (float)m;
            const float rn = m > 0 ? __fdiv_rn(127.f, mf) : 0.f;
            const float sn = m > 0 ? __fmul_rn(__fmul_rn(sprev, s1), __fdiv_rn(mf, 127.f)) : 0.f;
#pragma unroll
            for (int jj = 0; jj < 32; ++jj) {
                float qf;
                q[jj] = quant_i8f(i2f_small(accv[jj]), rn, qf);
                t[jj] = __fadd_rn(t[jj], __fmul_rn(sn, qf));
            }
            if (pw + 1 < pN) st_i8x32(sA, r, 2 * h, q);
            if (valid) {
                const int64_t base = ((cidx * pN + pw) * KC + rin) * KC + 32 * h;
                if (p.q) {
#pragma unroll
                    for (int jj = 0; jj < 32; jj += 4)
                        *reinterpret_cast<char4*>(p.q + base + jj) =
                            make_char4((signed char)q[jj], (signed char)q[jj + 1],
                                       (signed char)q[jj + 2], (signed char)q[jj + 3]);
                }
                if (p.acc) {
#pragma unroll
                    for (int jj = 0; jj < 32; jj += 4)
                        *reinterpret_cast<int4*>(p.acc + base + jj) =
                            make_int4(accv[jj], accv[jj + 1], accv[jj + 2], accv[jj + 3]);
                }
                if (p.scale && rin == 0 && h == 0) p.scale[cidx * pN + pw] = sn;
            }
            sprev = sn;
        }
        if (!ok) break;
        if constexpr (RES) {
            // ---- residual correction, every product in int8 codes ----
            // X = T0 - I; E = (A - X) + s_A s_X (q_A q_X); E's powers as A's;
            // Gm = sum s_E,s q_E,s; T = (T0 + Gm) + s_X s_G (q_X q_G).
            auto product = [&](uint32_t (&raw)[32]) -> bool {   // codes in sA, sB -> TMEM
                fence_async_smem();
                tc_fence_before();
                bar_sync(bar_id, 256);
                tc_fence_after();
                if (leader) {
                    constexpr uint32_t id = idesc_i8(128, 128);
#pragma unroll
                    for (int kk = 0; kk < KC / 32; ++kk)
                        mma_i8(tm, sdesc(su32(sA) + kk * 32, 16, 1024),
                               sdesc(su32(sB) + kk * 32 * 128, 16, 1024), id, kk > 0);
                    mma_commit(&ctrl->mma[s]);
                }
                const bool good = mbar_wait(&ctrl->mma[s], mma_phase);
                mma_phase ^= 1;
                if (!good) {
                    atomicExch(&ctrl->abort, 1);
                    raise_status(p.status, kStatusTimeout);
                }
                tc_fence_after();
                tmem_ld32_async(tD, raw);
                tmem_wait_ld();
                return !bar_sync_or(bar_id, 256, *(volatile int*)&ctrl->abort != 0);
            };
            auto eye_f = [&](int jj) { return i == 32 * h + jj ? 1.f : 0.f; };
            // codes of the whole A and of X
            float ma = 0.f, mx = 0.f;
#pragma unroll
            for (int jj = 0; jj < 32; ++jj) {
                ma = fmaxf(ma, fabsf(a[jj]));
                mx = fmaxf(mx, fabsf(__fsub_rn(t[jj], eye_f(jj))));
            }
            // with N = 1 no product separates A's maximum from this one: every
            // warp must have read A's partials before they are overwritten
            if (pN == 1) bar_sync(bar_id, 256);
            ma = chunk_max_f(ma);
            bar_sync(bar_id, 256);                       // every warp has read ma's partials
            mx = chunk_max_f(mx);
            const float rA = ma > 0.f ? __fdiv_rn(127.f, ma) : 0.f;
            const float sA_ = ma > 0.f ? __fdiv_rn(ma, 127.f) : 0.f;
            const float rX = mx > 0.f ? __fdiv_rn(127.f, mx) : 0.f;
            const float sX_ = mx > 0.f ? __fdiv_rn(mx, 127.f) : 0.f;
#pragma unroll
            for (int jj = 0; jj < 32; ++jj) {
                float qf;
                q[jj] = quant_i8f(a[jj], rA, qf);
            }
            st_i8x32(sA, r, 2 * h, q);                              // q_A (left)
#pragma unroll
            for (int jj = 0; jj < 32; ++jj) {
                float qf;
                q[jj] = quant_i8f(__fsub_rn(t[jj], eye_f(jj)), rX, qf);
            }
            st_i8x32(sB, i, 4 * c + 2 * h, q);                      // q_X (right)
            uint32_t raw[32];
            if (!product(raw)) { ok = false; break; }
            // E, then its codes
            const float sAX = __fmul_rn(sA_, sX_);
            float me = 0.f;
#pragma unroll
            for (int jj = 0; jj < 32; ++jj) {
                a[jj] = __fadd_rn(__fsub_rn(a[jj], __fsub_rn(t[jj], eye_f(jj))),
                                  __fmul_rn(sAX, i2f_small((int)raw[jj])));  // E over A
                me = fmaxf(me, fabsf(a[jj]));
            }
            me = chunk_max_f(me);
            const float rE = me > 0.f ? __fdiv_rn(127.f, me) : 0.f;
            const float sE1 = me > 0.f ? __fdiv_rn(me, 127.f) : 0.f;
            float gm[32];
#pragma unroll
            for (int jj = 0; jj < 32; ++jj) {
                float qf;
                q[jj] = quant_i8f(a[jj], rE, qf);
                gm[jj] = __fmul_rn(sE1, qf);
            }
            float sprevE = sE1;
            for (int sp = 2; sp <= pS; ++sp) {
                tc_fence_before();
                bar_sync(bar_id, 256);                              // the last product's reads
                st_i8x32(sA, r, 2 * h, q);                          // q_E,s-1 (left)
                if (sp == 2) st_i8x32(sB, i, 4 * c + 2 * h, q);     // q_E1 (right)
                if (!product(raw)) { ok = false; break; }
                int m = 0;
#pragma unroll
                for (int jj = 0; jj < 32; ++jj) m = max(m, abs((int)raw[jj]));
                m = chunk_max_i(m);
                const float mf = (float)m;
                const float rn = m > 0 ? __fdiv_rn(127.f, mf) : 0.f;
                const float sn = m > 0 ? __fmul_rn(__fmul_rn(sprevE, sE1), __fdiv_rn(mf, 127.f)) : 0.f;
#pragma unroll
                for (int jj = 0; jj < 32; ++jj) {
                    float qf;
                    q[jj] = quant_i8f(i2f_small((int)raw[jj]), rn, qf);
                    gm[jj] = __fadd_rn(gm[jj], __fmul_rn(sn, qf));
                }
                sprevE = sn;
            }
            if (!ok) break;
            // codes of Gm; T = (T0 + Gm) + s_X s_G (q_X q_G)
            float mg = 0.f;
#pragma unroll
            for (int jj = 0; jj < 32; ++jj) mg = fmaxf(mg, fabsf(gm[jj]));
            bar_sync(bar_id, 256);                       // every warp has read me's partials
            mg = chunk_max_f(mg);
            const float rG = mg > 0.f ? __fdiv_rn(127.f, mg) : 0.f;
            const float sG = mg > 0.f ? __fdiv_rn(mg, 127.f) : 0.f;
            tc_fence_before();
            bar_sync(bar_id, 256);                                  // the last product's reads
#pragma unroll
            for (int jj = 0; jj < 32; ++jj) {
                float qf;
                q[jj] = quant_i8f(__fsub_rn(t[jj], eye_f(jj)), rX, qf);
            }
            st_i8x32(sA, r, 2 * h, q);                              // q_X (left)
#pragma unroll
            for (int jj = 0; jj < 32; ++jj) {
                float qf;
                q[jj] = quant_i8f(gm[jj], rG, qf);
            }
            st_i8x32(sB, i, 4 * c + 2 * h, q);                      // q_G (right)
            if (!product(raw)) { ok = false; break; }
            const float sXG = __fmul_rn(sX_, sG);
#pragma unroll
            for (int jj = 0; jj < 32; ++jj)
                t[jj] = __fadd_rn(__fadd_rn(t[jj], gm[jj]), __fmul_rn(sXG, i2f_small((int)raw[jj])));
        }
        if (valid) {
            float* dst = p.T + cidx * KC * KC + rin * KC + 32 * h;
#pragma unroll
            for (int q4 = 0; q4 < 8; ++q4)
                reinterpret_cast<float4*>(dst)[q4] =
                    make_float4(t[4 * q4], t[4 * q4 + 1], t[4 * q4 + 2], t[4 * q4 + 3]);
        }
        tc_fence_before();
    }
    if (!ok && leader) {
        // bounded: one more commit tracks every product the slot's issuing
        // thread started, so TMEM is not freed under one; its last load lands
        // before the shared memory goes away
        mma_commit(&ctrl->drain[s]);
        mbar_wait(&ctrl->drain[s], 0);
        if (a_issued > 0) mbar_wait(&ctrl->full[s], (uint32_t)((a_issued - 1) & 1));
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem_base, 256);
    }
}

// ------------------------------------------------------------------------- //
// INT16 truncated Neumann series (k = 64): int16 codes through 8-bit products
// ------------------------------------------------------------------------- //
// The INT16 scheme of gdn.h: codes in [-32767, 32767], accumulators exact in
// int64, every scale operation in IEEE binary64.  The tensor cores multiply
// 8-bit codes, so each product of two code matrices is assembled from bytes.
// With the offset code q' = q + 32768 = 256 h + l (h, l unsigned bytes),
//   sum_l q'_a q'_b = 65536 HH + 256 (HL + LH) + LL
// takes three accumulators of unsigned x unsigned kind::i8 products (HL and
// LH share one), and
//   sum_l q_a q_b = sum_l q'_a q'_b - 32768 (R_a + C_b) + 64 * 32768^2
// with R_a the row sums of q'_a and C_b the column sums of q'_b (64 terms per
// chunk).  Every intermediate is an exact integer, so codes, accumulators,
// scales and T match the oracle bit for bit.  One slot of 8 warps per CTA
// (the three accumulators take 384 of the SM's 512 TMEM columns), A staged
// by TMA one tile ahead.  The RES instance follows the series with the
// parallel residual correction, every product again of int16 codes.
struct ParamsI16 {
    int64_t rows;
    int ntiles;
    int N, mask;
    int S;               // residual steps (the RES instance)
    const float* A;
    float* T;
    int16_t* q;
    int64_t* acc;
    double* scale;
    int* status;
};

constexpr int kI16Op = kRows * 128;                  // 16 KB: 128 rows x 64 byte codes
constexpr int kI16B = 64 * 128;                      // 8 KB: 64 rows x 128 byte codes
constexpr int kI16Stage = kRows * 64 * 4;            // 32 KB: the next tile's A
constexpr int kI16Smem = 2 * kI16Op + 2 * kI16B + kI16Stage;
constexpr int kI16Ctrl = 2048;                       // the control block after the operands
constexpr int kI16T0 = 32 * 256 * 8;                 // RES: T0 in binary64, [column][thread]

// 32 byte codes -> two 16-byte groups of a 128-byte swizzled row
__device__ __forceinline__ void st_u8x32(uint8_t* buf, int row, int q0, const uint32_t (&b)[32]) {
#pragma unroll
    for (int g = 0; g < 2; ++g) {
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int e = 16 * g + 4 * k;
            w[k] = b[e] | (b[e + 1] << 8) | (b[e + 2] << 16) | (b[e + 3] << 24);
        }
        const int q = q0 + g;
        *reinterpret_cast<uint4*>(buf + row * 128 + (((q & 7) ^ (row & 7)) << 4)) =
            make_uint4(w[0], w[1], w[2], w[3]);
    }
}
// clamp(rint(x * r), +-32767) in binary64, as quant_i8 (r = 0 gives 0)
__device__ __forceinline__ int quant_i16(double x, double r) {
    const int q = __double2int_rn(__dmul_rn(x, r));
    return min(max(q, -32767), 32767);
}

template <bool RES, int SN, int SS>
__global__ void __launch_bounds__(256, 1)
k_neumann_i16_tc(const __grid_constant__ CUtensorMap mA, const ParamsI16 p) {
    constexpr int KC = 64;
    extern __shared__ __align__(1024) uint8_t smem[];
    if ((su32(smem) & 1023u) != 0) {
        if (threadIdx.x == 0) raise_status(p.status, kStatusSmemAlign);
        return;
    }
    struct __align__(8) CtrlI16 {
        uint64_t mma;
        uint64_t full;                             // the staged A landed
        uint64_t drain;                            // after an expired wait: the products are done
        uint32_t tmem;
        int abort;
        float red_f[2][4];
        long long red_l[2][4];
        double red_d[2][4];
        int rsum[kRows][2];                        // row sums of the left operand's q'
        int csum[2][64];                           // column sums of q'_1 (the right operand), per chunk
    };
    static_assert(sizeof(CtrlI16) <= kI16Ctrl, "control block");
    uint8_t* sAh = smem;
    uint8_t* sAl = sAh + kI16Op;
    uint8_t* sBh = sAl + kI16Op;
    uint8_t* sBl = sBh + kI16B;
    uint8_t* sStage = sBl + kI16B;
    CtrlI16* ctrl = reinterpret_cast<CtrlI16*>(smem + kI16Smem);
    // the series order and the residual steps, as in the INT8 kernel
    const int pN = SN > 0 ? SN : p.N;
    const int pS = SS >= 0 ? SS : p.S;
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        mbar_init(&ctrl->mma, 1);
        mbar_init(&ctrl->full, 1);
        mbar_init(&ctrl->drain, 1);
        ctrl->abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 0) tmem_alloc(&ctrl->tmem, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = ctrl->tmem;

    const int h = warp / 4;
    const int r = ((warp & 3) << 5) | lane;
    const int c = r / KC;                          // chunk of this row in the tile
    const int i = r % KC;
    const int wq = ((warp & 3) & 1) * 2 + h;       // this warp's slot among its chunk's 4 warps
    const int jmin = p.mask ? i - pN : -KC;
    const uint32_t tD = tm + ((uint32_t)((warp & 3) * 32) << 16) + c * KC + 32 * h;
    const bool leader = warp == 0 && lane == 0;
    uint32_t mma_phase = 0;
    bool ok = true;

    auto chunk_max_f = [&](float v) {
        for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
        if (lane == 0) ctrl->red_f[c][wq] = v;
        __syncthreads();
        return fmaxf(fmaxf(ctrl->red_f[c][0], ctrl->red_f[c][1]),
                     fmaxf(ctrl->red_f[c][2], ctrl->red_f[c][3]));
    };
    auto chunk_max_l = [&](long long v) {
        for (int o = 16; o; o >>= 1) {
            const long long w = __shfl_xor_sync(0xffffffffu, v, o);
            v = v > w ? v : w;
        }
        if (lane == 0) ctrl->red_l[c][wq] = v;
        __syncthreads();
        long long m = ctrl->red_l[c][0];
#pragma unroll
        for (int k = 1; k < 4; ++k) m = m > ctrl->red_l[c][k] ? m : ctrl->red_l[c][k];
        return m;
    };
    auto chunk_max_d = [&](double v) {
        for (int o = 16; o; o >>= 1) v = fmax(v, __shfl_xor_sync(0xffffffffu, v, o));
        if (lane == 0) ctrl->red_d[c][wq] = v;
        __syncthreads();
        return fmax(fmax(ctrl->red_d[c][0], ctrl->red_d[c][1]), fmax(ctrl->red_d[c][2], ctrl->red_d[c][3]));
    };
    // offset codes q' = q + 32768 as high and low bytes; row sum of this half-row
    auto split = [&](const int (&q)[32], uint32_t (&hb)[32], uint32_t (&lb)[32]) {
        int sum = 0;
#pragma unroll
        for (int jj = 0; jj < 32; ++jj) {
            const uint32_t o = (uint32_t)(q[jj] + 32768);
            hb[jj] = o >> 8;
            lb[jj] = o & 0xffu;
            sum += (int)o;
        }
        return sum;
    };
    int a_issued = 0;
    auto issue_a = [&](int n) {
        const int tile = blockIdx.x + n * gridDim.x;
        if (tile >= p.ntiles) return;
        ++a_issued;
        mbar_expect_tx(&ctrl->full, kI16Stage);
        tma_load_2d(sStage, &mA, 0, tile * kRows, &ctrl->full);
        tma_load_2d(sStage + 16384, &mA, 32, tile * kRows, &ctrl->full);
    };
    if (leader) issue_a(0);

    for (int n = 0;; ++n) {
        const int tile = blockIdx.x + n * gridDim.x;
        if (tile >= p.ntiles) break;
        const int64_t grow = (int64_t)tile * kRows + r;
        const bool valid = grow < p.rows;
        const int64_t cidx = grow / KC, rin = grow % KC;
        if (!mbar_wait(&ctrl->full, (uint32_t)(n & 1))) {
            atomicExch(&ctrl->abort, 1);
            raise_status(p.status, kStatusTimeout);
        }
        float a[32];                                // rows past the end were zero-filled
        {
            const uint32_t rb = su32(sStage) + (uint32_t)(h * 16384 + r * 128);
#pragma unroll
            for (int c4 = 0; c4 < 8; ++c4) {
                const uint4 u = lds128(rb + ((c4 ^ (r & 7)) << 4));
                a[4 * c4] = __uint_as_float(u.x);
                a[4 * c4 + 1] = __uint_as_float(u.y);
                a[4 * c4 + 2] = __uint_as_float(u.z);
                a[4 * c4 + 3] = __uint_as_float(u.w);
            }
        }
        fence_async_smem();
        __syncthreads();                           // the previous tile's operand reads are done
        if (*(volatile int*)&ctrl->abort) { ok = false; break; }
        if (leader) issue_a(n + 1);
        float amax = 0.f;
#pragma unroll
        for (int jj = 0; jj < 32; ++jj) {
            if (32 * h + jj < jmin) a[jj] = 0.f;   // P_1 = M . A
            amax = fmaxf(amax, fabsf(a[jj]));
        }
        amax = chunk_max_f(amax);
        const double r1 = amax > 0.f ? __ddiv_rn(32767.0, (double)amax) : 0.0;
        const double s1 = amax > 0.f ? __ddiv_rn((double)amax, 32767.0) : 0.0;
        int q[32];
        double t[32];
#pragma unroll
        for (int jj = 0; jj < 32; ++jj) {
            q[jj] = quant_i16((double)a[jj], r1);
            t[jj] = __dadd_rn(i == 32 * h + jj ? 1.0 : 0.0, __dmul_rn(s1, (double)q[jj]));
        }
        {
            uint32_t hb[32], lb[32];
            ctrl->rsum[r][h] = split(q, hb, lb);
            st_u8x32(sAh, r, 2 * h, hb);           // q'_1 as the left operand
            st_u8x32(sAl, r, 2 * h, lb);
            st_u8x32(sBh, i, 4 * c + 2 * h, hb);   // and as the right operand
            st_u8x32(sBl, i, 4 * c + 2 * h, lb);
            // column sums of q'_1 over the chunk's 64 rows: the two warps of
            // this chunk and half reduce 32 columns each by recursive halving
            int v[32];
#pragma unroll
            for (int jj = 0; jj < 32; ++jj) v[jj] = q[jj] + 32768;
#pragma unroll
            for (int sh = 16; sh >= 1; sh >>= 1) {
                const bool up = (lane & sh) != 0;
#pragma unroll
                for (int k = 0; k < sh; ++k) {
                    const int send = up ? v[k] : v[k + sh];
                    const int keep = up ? v[k + sh] : v[k];
                    v[k] = keep + __shfl_xor_sync(0xffffffffu, send, sh);
                }
            }
            // lane holds column 32 h + lane summed over this warp's 32 rows
            if ((warp & 1) == 0) ctrl->csum[c][32 * h + lane] = v[0];
            __syncthreads();
            if ((warp & 1) == 1) ctrl->csum[c][32 * h + lane] += v[0];
        }
        if (valid) {
            const int64_t base = (cidx * pN * KC + rin) * KC + 32 * h;
            if (p.q) {
#pragma unroll
                for (int jj = 0; jj < 32; jj += 4)
                    *reinterpret_cast<short4*>(p.q + base + jj) =
                        make_short4((short)q[jj], (short)q[jj + 1], (short)q[jj + 2], (short)q[jj + 3]);
            }
            if (p.acc) {
#pragma unroll
                for (int jj = 0; jj < 32; jj += 2)
                    *reinterpret_cast<longlong2*>(p.acc + base + jj) = make_longlong2(0, 0);
            }
            if (p.scale && rin == 0 && h == 0) p.scale[cidx * pN] = s1;
        }
        double sprev = s1;
        for (int pw = 1; pw < pN; ++pw) {
            fence_async_smem();
            tc_fence_before();
            __syncthreads();                       // operands, row and column sums written
            tc_fence_after();
            if (leader) {
                constexpr uint32_t id = (2u << 4) | (0u << 7) | (0u << 10) | (0u << 15) | (1u << 16) |
                                        ((uint32_t)(128 >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
#pragma unroll
                for (int kk = 0; kk < KC / 32; ++kk) {
                    const uint64_t ah = sdesc(su32(sAh) + kk * 32, 16, 1024);
                    const uint64_t al = sdesc(su32(sAl) + kk * 32, 16, 1024);
                    const uint64_t bh = sdesc(su32(sBh) + kk * 32 * 128, 16, 1024);
                    const uint64_t bl = sdesc(su32(sBl) + kk * 32 * 128, 16, 1024);
                    mma_i8(tm, ah, bh, id, kk > 0);                 // HH
                    mma_i8(tm + 128, ah, bl, id, kk > 0);           // HL
                    mma_i8(tm + 128, al, bh, id, 1);                // + LH
                    mma_i8(tm + 256, al, bl, id, kk > 0);           // LL
                }
                mma_commit(&ctrl->mma);
            }
            bool good = mbar_wait(&ctrl->mma, mma_phase);
            mma_phase ^= 1;
            if (!good) {
                atomicExch(&ctrl->abort, 1);
                raise_status(p.status, kStatusTimeout);
            }
            tc_fence_after();
            uint32_t hh[32], mm[32], ll[32];
            tmem_ld32_async(tD, hh);
            tmem_ld32_async(tD + 128, mm);
            tmem_ld32_async(tD + 256, ll);
            tmem_wait_ld();
            const long long ra = (long long)ctrl->rsum[r][0] + ctrl->rsum[r][1];
            long long accv[32];
            long long m = 0;
#pragma unroll
            for (int jj = 0; jj < 32; ++jj) {
                const long long full = 65536LL * (int)hh[jj] + 256LL * (int)mm[jj] + (long long)(int)ll[jj]
                                       - 32768LL * (ra + ctrl->csum[c][32 * h + jj]) +
                                       (long long)KC * 32768LL * 32768LL;
                accv[jj] = (32 * h + jj < jmin) ? 0 : full;
                const long long ab = accv[jj] < 0 ? -accv[jj] : accv[jj];
                m = m > ab ? m : ab;
            }
            m = chunk_max_l(m);
            if (*(volatile int*)&ctrl->abort) { ok = false; break; }
            const double mf = (double)m;
            const double rn = m > 0 ? __ddiv_rn(32767.0, mf) : 0.0;
            const double sn = m > 0 ? __dmul_rn(__dmul_rn(sprev, s1), __ddiv_rn(mf, 32767.0)) : 0.0;
#pragma unroll
            for (int jj = 0; jj < 32; ++jj) {
                q[jj] = quant_i16((double)accv[jj], rn);
                t[jj] = __dadd_rn(t[jj], __dmul_rn(sn, (double)q[jj]));
            }
            if (pw + 1 < pN) {
                uint32_t hb[32], lb[32];
                const int sum = split(q, hb, lb);
                tc_fence_before();
                __syncthreads();                   // every row sum of q'_{n-1} has been read
                ctrl->rsum[r][h] = sum;
                st_u8x32(sAh, r, 2 * h, hb);
                st_u8x32(sAl, r, 2 * h, lb);
            }
            if (valid) {
                const int64_t base = ((cidx * pN + pw) * KC + rin) * KC + 32 * h;
                if (p.q) {
#pragma unroll
                    for (int jj = 0; jj < 32; jj += 4)
                        *reinterpret_cast<short4*>(p.q + base + jj) =
                            make_short4((short)q[jj], (short)q[jj + 1], (short)q[jj + 2], (short)q[jj + 3]);
                }
                if (p.acc) {
#pragma unroll
                    for (int jj = 0; jj < 32; jj += 2)
                        *reinterpret_cast<longlong2*>(p.acc + base + jj) =
                            make_longlong2(accv[jj], accv[jj + 1]);
                }
                if (p.scale && rin == 0 && h == 0) p.scale[cidx * pN + pw] = sn;
            }
            sprev = sn;
        }
        if (!ok) break;
        if constexpr (RES) {
            // ---- residual correction, every product of int16 codes ----
            // X = T0 - I; E = (A - X) + (s_A s_X) (q_A q_X) over the whole A;
            // E's powers requantised as A's; Gm = sum_s s_E,s q_E,s;
            // T = (T0 + Gm) + (s_X s_G) (q_X q_G); every scale and sum in
            // binary64, T rounded once to float32.  T0 waits in shared memory.
            double* const sT0 = reinterpret_cast<double*>(smem + kI16Smem + kI16Ctrl);
            const int tid = threadIdx.x;
            auto t0 = [&](int jj) { return sT0[jj * 256 + tid]; };
            auto xv = [&](int jj) { return __dsub_rn(t0(jj), i == 32 * h + jj ? 1.0 : 0.0); };
#pragma unroll
            for (int jj = 0; jj < 32; ++jj) sT0[jj * 256 + tid] = t[jj];
            // the operands of one product: the left codes with their row sums,
            // the right codes with their column sums (both as offset bytes)
            auto set_left = [&](const int (&qq)[32]) {
                uint32_t hb[32], lb[32];
                ctrl->rsum[r][h] = split(qq, hb, lb);
                st_u8x32(sAh, r, 2 * h, hb);
                st_u8x32(sAl, r, 2 * h, lb);
            };
            auto set_right = [&](const int (&qq)[32]) {
                {
                    uint32_t hb[32], lb[32];
                    split(qq, hb, lb);
                    st_u8x32(sBh, i, 4 * c + 2 * h, hb);
                    st_u8x32(sBl, i, 4 * c + 2 * h, lb);
                }
                int v[32];
#pragma unroll
                for (int jj = 0; jj < 32; ++jj) v[jj] = qq[jj] + 32768;
#pragma unroll
                for (int sh = 16; sh >= 1; sh >>= 1) {
                    const bool up = (lane & sh) != 0;
#pragma unroll
                    for (int k = 0; k < sh; ++k) {
                        const int send = up ? v[k] : v[k + sh];
                        const int keep = up ? v[k + sh] : v[k];
                        v[k] = keep + __shfl_xor_sync(0xffffffffu, send, sh);
                    }
                }
                if ((warp & 1) == 0) ctrl->csum[c][32 * h + lane] = v[0];
                __syncthreads();
                if ((warp & 1) == 1) ctrl->csum[c][32 * h + lane] += v[0];
            };
            // every thread must be done with the last product's accumulators
            // and sums before the next operands are written
            auto begin_operands = [&]() {
                tc_fence_before();
                __syncthreads();
            };
            // left x right as int64, assembled from the three byte products
            auto product = [&](long long (&accv)[32]) {
                fence_async_smem();
                tc_fence_before();
                __syncthreads();                           // operands and sums written
                tc_fence_after();
                if (leader) {
                    constexpr uint32_t id = (2u << 4) | (0u << 7) | (0u << 10) | (0u << 15) | (1u << 16) |
                                            ((uint32_t)(128 >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
#pragma unroll
                    for (int kk = 0; kk < KC / 32; ++kk) {
                        const uint64_t ah = sdesc(su32(sAh) + kk * 32, 16, 1024);
                        const uint64_t al = sdesc(su32(sAl) + kk * 32, 16, 1024);
                        const uint64_t bh = sdesc(su32(sBh) + kk * 32 * 128, 16, 1024);
                        const uint64_t bl = sdesc(su32(sBl) + kk * 32 * 128, 16, 1024);
                        mma_i8(tm, ah, bh, id, kk > 0);                 // HH
                        mma_i8(tm + 128, ah, bl, id, kk > 0);           // HL
                        mma_i8(tm + 128, al, bh, id, 1);                // + LH
                        mma_i8(tm + 256, al, bl, id, kk > 0);           // LL
                    }
                    mma_commit(&ctrl->mma);
                }
                const bool good = mbar_wait(&ctrl->mma, mma_phase);
                mma_phase ^= 1;
                if (!good) {
                    atomicExch(&ctrl->abort, 1);
                    raise_status(p.status, kStatusTimeout);
                }
                tc_fence_after();
                uint32_t hh[32], mm[32], ll[32];
                tmem_ld32_async(tD, hh);
                tmem_ld32_async(tD + 128, mm);
                tmem_ld32_async(tD + 256, ll);
                tmem_wait_ld();
                const long long ra = (long long)ctrl->rsum[r][0] + ctrl->rsum[r][1];
#pragma unroll
                for (int jj = 0; jj < 32; ++jj)
                    accv[jj] = 65536LL * (int)hh[jj] + 256LL * (int)mm[jj] + (long long)(int)ll[jj] -
                               32768LL * (ra + ctrl->csum[c][32 * h + jj]) +
                               (long long)KC * 32768LL * 32768LL;
            };
            // codes of the whole A (reloaded: the stage already holds the next
            // tile) and of X
            float av[32];
            if (valid) {
                const float4* src = reinterpret_cast<const float4*>(p.A + (cidx * KC + rin) * KC + 32 * h);
#pragma unroll
                for (int q4 = 0; q4 < 8; ++q4) {
                    const float4 u = src[q4];
                    av[4 * q4] = u.x;
                    av[4 * q4 + 1] = u.y;
                    av[4 * q4 + 2] = u.z;
                    av[4 * q4 + 3] = u.w;
                }
            } else {
#pragma unroll
                for (int jj = 0; jj < 32; ++jj) av[jj] = 0.f;   // rows past the end: A = 0
            }
            float ma = 0.f;
            double mx = 0.0;
#pragma unroll
            for (int jj = 0; jj < 32; ++jj) {
                ma = fmaxf(ma, fabsf(av[jj]));
                mx = fmax(mx, fabs(xv(jj)));
            }
            ma = chunk_max_f(ma);
            mx = chunk_max_d(mx);
            const double rA = ma > 0.f ? __ddiv_rn(32767.0, (double)ma) : 0.0;
            const double sA = ma > 0.f ? __ddiv_rn((double)ma, 32767.0) : 0.0;
            const double rX = mx > 0.0 ? __ddiv_rn(32767.0, mx) : 0.0;
            const double sX = mx > 0.0 ? __ddiv_rn(mx, 32767.0) : 0.0;
            begin_operands();
#pragma unroll
            for (int jj = 0; jj < 32; ++jj) q[jj] = quant_i16((double)av[jj], rA);
            set_left(q);                                            // q_A
#pragma unroll
            for (int jj = 0; jj < 32; ++jj) q[jj] = quant_i16(xv(jj), rX);
            set_right(q);                                           // q_X
            long long accv[32];
            product(accv);
            // E and its codes
            const double sAX = __dmul_rn(sA, sX);
            double e[32];
            double me = 0.0;
#pragma unroll
            for (int jj = 0; jj < 32; ++jj) {
                e[jj] = __dadd_rn(__dsub_rn((double)av[jj], xv(jj)), __dmul_rn(sAX, (double)accv[jj]));
                me = fmax(me, fabs(e[jj]));
            }
            me = chunk_max_d(me);
            if (*(volatile int*)&ctrl->abort) { ok = false; break; }
            const double rE = me > 0.0 ? __ddiv_rn(32767.0, me) : 0.0;
            const double sE1 = me > 0.0 ? __ddiv_rn(me, 32767.0) : 0.0;
            double gm[32];
#pragma unroll
            for (int jj = 0; jj < 32; ++jj) {
                q[jj] = quant_i16(e[jj], rE);
                gm[jj] = __dmul_rn(sE1, (double)q[jj]);
            }
            double sprevE = sE1;
            for (int sp = 2; sp <= pS; ++sp) {
                begin_operands();
                set_left(q);                                        // q_E,s-1
                if (sp == 2) set_right(q);                          // q_E1
                product(accv);
                long long m = 0;
#pragma unroll
                for (int jj = 0; jj < 32; ++jj) {
                    const long long ab = accv[jj] < 0 ? -accv[jj] : accv[jj];
                    m = m > ab ? m : ab;
                }
                m = chunk_max_l(m);
                if (*(volatile int*)&ctrl->abort) { ok = false; break; }
                const double mf = (double)m;
                const double rn = m > 0 ? __ddiv_rn(32767.0, mf) : 0.0;
                const double sn = m > 0 ? __dmul_rn(__dmul_rn(sprevE, sE1), __ddiv_rn(mf, 32767.0)) : 0.0;
#pragma unroll
                for (int jj = 0; jj < 32; ++jj) {
                    q[jj] = quant_i16((double)accv[jj], rn);
                    gm[jj] = __dadd_rn(gm[jj], __dmul_rn(sn, (double)q[jj]));
                }
                sprevE = sn;
            }
            if (!ok) break;
            // codes of Gm; T = (T0 + Gm) + s_X s_G (q_X q_G)
            double mg = 0.0;
#pragma unroll
            for (int jj = 0; jj < 32; ++jj) mg = fmax(mg, fabs(gm[jj]));
            __syncthreads();                                        // every thread has read me's partials
            mg = chunk_max_d(mg);
            const double rG = mg > 0.0 ? __ddiv_rn(32767.0, mg) : 0.0;
            const double sG = mg > 0.0 ? __ddiv_rn(mg, 32767.0) : 0.0;
            begin_operands();
#pragma unroll
            for (int jj = 0; jj < 32; ++jj) q[jj] = quant_i16(xv(jj), rX);
            set_left(q);                                            // q_X
#pragma unroll
            for (int jj = 0; jj < 32; ++jj) q[jj] = quant_i16(gm[jj], rG);
            set_right(q);                                           // q_G
            product(accv);
            const double sXG = __dmul_rn(sX, sG);
#pragma unroll
            for (int jj = 0; jj < 32; ++jj)
                t[jj] = __dadd_rn(__dadd_rn(t0(jj), gm[jj]), __dmul_rn(sXG, (double)accv[jj]));
        }
        if (valid) {
            float* dst = p.T + cidx * KC * KC + rin * KC + 32 * h;
#pragma unroll
            for (int q4 = 0; q4 < 8; ++q4)
                reinterpret_cast<float4*>(dst)[q4] =
                    make_float4(__double2float_rn(t[4 * q4]), __double2float_rn(t[4 * q4 + 1]),
                                __double2float_rn(t[4 * q4 + 2]), __double2float_rn(t[4 * q4 + 3]));
        }
        tc_fence_before();
    }
    // the flag is raised only before a __syncthreads and read only after one,
    // so every thread takes the same decision; this last look covers a wait
    // that ran out in the tile's final product
    tc_fence_before();
    __syncthreads();
    if (*(volatile int*)&ctrl->abort) ok = false;
    if (!ok && leader) {
        // bounded: one more commit tracks every product started, so TMEM is
        // not freed under one; the last load lands before shared memory goes
        mma_commit(&ctrl->drain);
        mbar_wait(&ctrl->drain, 0);
        if (a_issued > 0) mbar_wait(&ctrl->full, (uint32_t)((a_issued - 1) & 1));
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tm, 512);
    }
}

// ------------------------------------------------------------------------- //
// k = 256: the truncated Neumann series on the tensor cores, S = 0
// ------------------------------------------------------------------------- //
// The chunk is a 2 x 2 block matrix of 128 x 128 blocks (the upper-right block
// of a strictly lower-triangular A is zero).  The series is summed in Horner
// form, X_1 = I + M.A and X_m = I + M.(X_{m-1} A), so that X_N = M.(sum of
// A^n, n = 0..N).  Keeping only the band of X_{m-1} changes nothing inside the
// band: entry (i, j) of X A reads X only at (i, l) with j < l <= i, and
// i - l < i - j.  One step is four 128 x 128 x 128 products:
//   D00 = X00 A00,  D10 = X10 A00 + X11 A10,  D11 = X11 A11
// with the X blocks as K-major left operands, the A blocks as MN-major right
// operands (both fp16 in shared memory, row-major with the 128-byte swizzle)
// and the three accumulators in TMEM columns [0, 384).  Warp group q (warps
// 4q .. 4q + 3) owns block q of {D00, D10, D11}: thread row = its TMEM lane.
// One chunk per CTA at a time (persistent grid); the 192 KB of operands leave
// no room for a second chunk.
struct Params256 {
    int64_t nc;
    int N;
    int mask;
    int S;
    const float* A;
    float* T;
    int* status;
};

constexpr int k256Threads = 384;
constexpr int k256Blk = kRows * 128 * 2;            // one 128 x 128 fp16 operand block
constexpr int k256Smem = 6 * k256Blk + 64;

// Byte offset of element (r, c) of a 128 x 128 fp16 operand block.
__device__ __forceinline__ uint32_t el_off256(int r, int c) {
    return op_off(r, c >> 3) + (uint32_t)((c & 7) * 2);
}

// T entries of the 32 x 32 tile (rows 32 rg .., columns c0 ..) that are zero
// whatever A holds: above the diagonal, or outside the band.
__device__ __forceinline__ bool zero_tile256(int rg, int c0, int mask, int N) {
    return c0 > 32 * rg + 31 || (mask && c0 + 31 < 32 * rg - N);
}

__global__ void __launch_bounds__(k256Threads, 1)
k_neumann256_tc(const Params256 p) {
    constexpr int KC = 256;
    extern __shared__ __align__(1024) uint8_t smem[];
    if ((su32(smem) & 1023u) != 0) {
        if (threadIdx.x == 0) raise_status(p.status, kStatusSmemAlign);
        return;
    }
    // right operands A00, A10, A11; left operands X00, X10, X11
    auto sA = [&](int b) { return smem + b * k256Blk; };
    auto sX = [&](int b) { return smem + (3 + b) * k256Blk; };
    uint64_t* mbar = reinterpret_cast<uint64_t*>(smem + 6 * k256Blk);
    uint32_t* tslot = reinterpret_cast<uint32_t*>(smem + 6 * k256Blk + 8);
    int* abort_flag = reinterpret_cast<int*>(smem + 6 * k256Blk + 16);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        mbar_init(mbar, 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 0) tmem_alloc(tslot, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = *tslot;

    const int gq = warp >> 2;                        // 0: D00, 1: D10, 2: D11
    const int rr = ((warp & 3) << 5) | lane;         // row inside the block = TMEM lane
    const int row = (gq ? 128 : 0) + rr;             // row inside the chunk
    const int col0 = gq == 2 ? 128 : 0;              // first column of the block
    const int rg = row >> 5;                         // this warp's 32-row group
    const uint32_t tD = tm + ((uint32_t)((warp & 3) * 32) << 16) + 128 * gq;
    const bool leader = threadIdx.x == 0;
    const int N = p.N, mask = p.mask;
    const int jmin = mask ? row - N : -KC;           // band: columns j >= jmin
    uint32_t phase = 0;
    bool ok = true, timed_out = false;

    // one step's products, issued by one thread
    auto issue = [&]() {
        constexpr uint32_t id = idesc_f16(0, 0, 1, 128, 128);
        auto blk = [&](uint32_t dcol, const uint8_t* xa, const uint8_t* ab, bool acc) {
            const uint32_t xb = su32(xa), bb = su32(ab);
#pragma unroll 1
            for (int kk = 0; kk < 8; ++kk)
                mma_ss(tm + dcol, sdesc(xb + (kk >> 2) * (kRows * 128) + (kk & 3) * 32, 16, 1024),
                       sdesc(bb + kk * 2048, kRows * 128, 1024), id, (acc || kk > 0) ? 1u : 0u);
        };
        blk(0, sX(0), sA(0), false);
        blk(128, sX(1), sA(0), false);
        blk(128, sX(2), sA(1), true);
        blk(256, sX(2), sA(2), false);
        mma_commit(mbar);
    };
    auto publish = [&]() {
        fence_async_smem();
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
    };

    for (int64_t c = blockIdx.x; c < p.nc; c += gridDim.x) {
        const float* Ac = p.A + c * KC * KC;
        float* Tc = p.T + c * KC * KC;
        // ---- A -> operands, X_1 = I + M.A; rows read whole by one warp (coalesced).
        // T entries that stay zero are written here; at N = 1 all of T is.
#pragma unroll 1
        for (int r0 = warp; r0 < KC; r0 += 4 * 12) {
            float4 a[4][2];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int rw = r0 + 12 * u;
                if (rw < KC) {
                    const float4* src = reinterpret_cast<const float4*>(Ac + (int64_t)rw * KC);
                    a[u][0] = __ldg(src + lane);
                    a[u][1] = __ldg(src + 32 + lane);
                }
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int rw = r0 + 12 * u;
                if (rw >= KC) continue;
                const int jm = mask ? rw - N : -KC;
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    const int j0 = 128 * hf + 4 * lane;
                    const float av[4] = {a[u][hf].x, a[u][hf].y, a[u][hf].z, a[u][hf].w};
                    float x[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        x[e] = (j0 + e == rw ? 1.f : 0.f) + (j0 + e >= jm ? av[e] : 0.f);
                    const bool upper = hf == 1 && rw < 128;
                    if (!upper) {
                        const int b = (rw >= 128) + hf;          // 0: (0,0), 1: (1,0), 2: (1,1)
                        const uint32_t off = el_off256(rw & 127, j0 & 127);
                        asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(su32(sA(b)) + off),
                                     "r"(pack_h2(av[0], av[1])), "r"(pack_h2(av[2], av[3]))
                                     : "memory");
                        asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(su32(sX(b)) + off),
                                     "r"(pack_h2(x[0], x[1])), "r"(pack_h2(x[2], x[3]))
                                     : "memory");
                    }
                    float4* dst = reinterpret_cast<float4*>(Tc + (int64_t)rw * KC + j0);
                    if (N == 1 && !upper)
                        *dst = make_float4(x[0], x[1], x[2], x[3]);
                    else if (upper || zero_tile256(rw >> 5, j0 & ~31, mask, N))
                        *dst = make_float4(0.f, 0.f, 0.f, 0.f);
                }
            }
        }
        publish();
        if (*(volatile int*)abort_flag) { ok = false; break; }
        // ---- steps 2 .. N
        for (int m = 2; m <= N; ++m) {
            if (leader) issue();
            if (mbar_wait(mbar, phase)) {
                phase ^= 1;
            } else {                                 // the products are still in flight
                timed_out = true;
                atomicExch(abort_flag, 1);
                raise_status(p.status, kStatusTimeout);
            }
            tc_fence_after();
#pragma unroll 1
            for (int pc = 0; pc < 4; ++pc) {
                const int c0 = col0 + 32 * pc;
                if (zero_tile256(rg, c0, mask, N)) continue;   // warp-uniform
                float v[32];
                tmem_ld32(tD + 32 * pc, v);
#pragma unroll
                for (int jj = 0; jj < 32; ++jj) {
                    const int j = c0 + jj;
                    v[jj] = (j == row ? 1.f : 0.f) + (j >= jmin ? v[jj] : 0.f);
                }
                if (m < N || p.S > 0) st_op32<false>(sX(gq), rr, pc, v);   // X_m; T0 for the residual
                if (m == N) {
                    float4* dst = reinterpret_cast<float4*>(Tc + (int64_t)row * KC + c0);
#pragma unroll
                    for (int q = 0; q < 8; ++q)
                        dst[q] = make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
                }
            }
            publish();
            if (*(volatile int*)abort_flag) { ok = false; break; }
        }
        if (!ok) break;
        // ---- residual (S > 0): E = I - T0 + A T0, Q_{m+1} = (I + Q_m) E,
        // T = T0 + T0 Q_S.  T0 (fp32) waits in the output T and is re-read from
        // there (each thread its own row pieces); the six operand blocks are
        // reused: A's blocks take E, then Q_S; the X blocks hold T0, then
        // I + Q_m, then T0 again for the last product.
        if (p.S > 0) {
            auto wait_products = [&]() {
                if (mbar_wait(mbar, phase)) {
                    phase ^= 1;
                } else {
                    timed_out = true;
                    atomicExch(abort_flag, 1);
                    raise_status(p.status, kStatusTimeout);
                }
                tc_fence_after();
            };
            auto t0_row = [&](int c0, float (&t)[32]) {
                const float4* src = reinterpret_cast<const float4*>(Tc + (int64_t)row * KC + c0);
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    const float4 x = src[q];
                    t[4 * q] = x.x; t[4 * q + 1] = x.y; t[4 * q + 2] = x.z; t[4 * q + 3] = x.w;
                }
            };
            // A T0: left A blocks, right T0 blocks
            if (leader) {
                constexpr uint32_t id = idesc_f16(0, 0, 1, 128, 128);
                auto blk = [&](uint32_t dcol, const uint8_t* xa, const uint8_t* ab, bool acc) {
                    const uint32_t xb = su32(xa), bb = su32(ab);
#pragma unroll 1
                    for (int kk = 0; kk < 8; ++kk)
                        mma_ss(tm + dcol, sdesc(xb + (kk >> 2) * (kRows * 128) + (kk & 3) * 32, 16, 1024),
                               sdesc(bb + kk * 2048, kRows * 128, 1024), id, (acc || kk > 0) ? 1u : 0u);
                };
                blk(0, sA(0), sX(0), false);
                blk(128, sA(1), sX(0), false);
                blk(128, sA(2), sX(1), true);
                blk(256, sA(2), sX(2), false);
                mma_commit(mbar);
            }
            wait_products();
#pragma unroll 1
            for (int pc = 0; pc < 4; ++pc) {
                const int c0 = col0 + 32 * pc;
                if (c0 > 32 * rg + 31) continue;        // above the diagonal for the whole warp
                float v[32], t[32];
                tmem_ld32(tD + 32 * pc, v);
                t0_row(c0, t);
#pragma unroll
                for (int jj = 0; jj < 32; ++jj) v[jj] += (c0 + jj == row ? 1.f : 0.f) - t[jj];   // E
                st_op32<false>(sA(gq), rr, pc, v);
                if (p.S > 1) {
#pragma unroll
                    for (int jj = 0; jj < 32; ++jj) v[jj] += (c0 + jj == row ? 1.f : 0.f);
                    st_op32<false>(sX(gq), rr, pc, v);                          // I + Q_1
                }
            }
            publish();
            if (*(volatile int*)abort_flag) { ok = false; break; }
            for (int m = 1; m < p.S; ++m) {                                     // (I + Q_m) E
                if (leader) issue();
                wait_products();
                const bool last = (m == p.S - 1);
#pragma unroll 1
                for (int pc = 0; pc < 4; ++pc) {
                    const int c0 = col0 + 32 * pc;
                    if (c0 > 32 * rg + 31) continue;
                    float v[32];
                    tmem_ld32(tD + 32 * pc, v);
                    if (last) {
                        st_op32<false>(sA(gq), rr, pc, v);                      // Q_S
                        float t[32];
                        t0_row(c0, t);
                        st_op32<false>(sX(gq), rr, pc, t);                      // T0
                    } else {
#pragma unroll
                        for (int jj = 0; jj < 32; ++jj) v[jj] += (c0 + jj == row ? 1.f : 0.f);
                        st_op32<false>(sX(gq), rr, pc, v);                      // I + Q_{m+1}
                    }
                }
                publish();
                if (*(volatile int*)abort_flag) { ok = false; break; }
            }
            if (!ok) break;
            if (leader) issue();                                                // T0 Q_S
            wait_products();
#pragma unroll 1
            for (int pc = 0; pc < 4; ++pc) {
                const int c0 = col0 + 32 * pc;
                if (c0 > 32 * rg + 31) continue;
                float v[32], t[32];
                tmem_ld32(tD + 32 * pc, v);
                t0_row(c0, t);
                float4* dst = reinterpret_cast<float4*>(Tc + (int64_t)row * KC + c0);
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    dst[q] = make_float4(t[4 * q] + v[4 * q], t[4 * q + 1] + v[4 * q + 1],
                                         t[4 * q + 2] + v[4 * q + 2], t[4 * q + 3] + v[4 * q + 3]);
            }
            publish();
            if (*(volatile int*)abort_flag) { ok = false; break; }
        }
    }
    if (timed_out) mbar_wait(mbar, phase);          // bounded: let the products finish
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tm, 512);
    }
}

// ------------------------------------------------------------------------- //
// A for k = 256 chunks: G = K K^T as three 128 x 128 blocks (G00, G10, G11;
// G01 is never needed), A_ij = -beta_i G_ij e^{g_i - g_j} for j < i.  One chunk
// per CTA at a time; the chunk's K arrives by TMA as two 128-row tiles (bf16,
// 128-byte swizzle) and the next chunk's K is loaded while this one's epilogue
// writes A.  Warp group q (warps 4q .. 4q + 3) owns block q of {G00, G10, G11}.
// ------------------------------------------------------------------------- //
struct ParamsA256 {
    int64_t nc;
    const float* beta;
    const float* g;
    float* A;
    int* status;
};

constexpr int kA256Smem = 2 * 2 * kRows * kD * 2 + 64;     // two stages of 2 K tiles, control

__global__ void __launch_bounds__(384, 1)
k_build_A256_tc(const __grid_constant__ CUtensorMap mK, const ParamsA256 p) {
    constexpr int KC = 256;
    extern __shared__ __align__(1024) uint8_t smem[];
    if ((su32(smem) & 1023u) != 0) {
        if (threadIdx.x == 0) raise_status(p.status, kStatusSmemAlign);
        return;
    }
    constexpr int kTile = kRows * kD * 2;                   // 32 KB: 128 rows of K
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + 4 * kTile);     // [2] stage landed
    uint64_t* mbar = full + 2;                                          // products done
    uint32_t* tslot = reinterpret_cast<uint32_t*>(mbar + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        mbar_init(&full[0], 1);
        mbar_init(&full[1], 1);
        mbar_init(mbar, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 0) tmem_alloc(tslot, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = *tslot;
    const int gq = warp >> 2;
    const int rr = ((warp & 3) << 5) | lane;
    const int row = (gq ? 128 : 0) + rr;
    const int col0 = gq == 2 ? 128 : 0;
    const uint32_t tD = tm + ((uint32_t)((warp & 3) * 32) << 16) + 128 * gq;
    const bool leader = threadIdx.x == 0;
    bool ok = true, timed_out = false;
    uint32_t phase = 0;
    int issued = 0;
    auto issue = [&](int64_t c, int st) {
        if (c >= p.nc) return;
        ++issued;
        uint8_t* base = smem + st * 2 * kTile;
        mbar_expect_tx(&full[st], 2 * kTile);
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const int y = (int)(c * KC + 128 * b);
            tma_load_2d(base + b * kTile, &mK, 0, y, &full[st]);
            tma_load_2d(base + b * kTile + kRows * 128, &mK, 64, y, &full[st]);
        }
    };
    if (leader) issue(blockIdx.x, 0);
    int it = 0;
    for (int64_t c = blockIdx.x; c < p.nc; c += gridDim.x, ++it) {
        const int st = it & 1;
        uint8_t* k0 = smem + st * 2 * kTile;
        uint8_t* k1 = k0 + kTile;
        if (!mbar_wait(&full[st], (uint32_t)((it >> 1) & 1))) {
            raise_status(p.status, kStatusTimeout);
            ok = false;
        }
        // the other stage is free (its products completed last iteration)
        if (leader) issue(c + gridDim.x, st ^ 1);
        tc_fence_after();
        if (leader && ok) {
            constexpr uint32_t id = idesc_f16(1, 0, 0, 128, 128);
            auto blk = [&](uint32_t dcol, const uint8_t* xa, const uint8_t* xb) {
                const uint32_t a0 = su32(xa), b0 = su32(xb);
#pragma unroll 1
                for (int kk = 0; kk < kD / 16; ++kk) {
                    const uint32_t ko = (kk >> 2) * (kRows * 128) + (kk & 3) * 32;
                    mma_ss(tm + dcol, sdesc(a0 + ko, 16, 1024), sdesc(b0 + ko, 16, 1024), id, kk > 0);
                }
            };
            blk(0, k0, k0);                                 // G00
            blk(128, k1, k0);                               // G10
            blk(256, k1, k1);                               // G11
            mma_commit(mbar);
        }
        __syncwarp();
        // (all threads) products done
        if (ok && !mbar_wait(mbar, phase)) {
            timed_out = true;
            raise_status(p.status, kStatusTimeout);
            ok = false;
        }
        if (ok) phase ^= 1;
        tc_fence_after();
        if (__syncthreads_or(!ok)) break;
        const int64_t grow = c * KC + row;
        const float bi = p.beta[grow], gi = p.g[grow];
        const float* gcol = p.g + c * KC + col0;
        float* Ar = p.A + (c * KC + row) * (int64_t)KC;
#pragma unroll 1
        for (int pc = 0; pc < 4; ++pc) {
            const int c0 = col0 + 32 * pc;
            float v[32];
            if (c0 > (row | 31)) {                          // above the diagonal for the warp
#pragma unroll
                for (int jj = 0; jj < 32; ++jj) v[jj] = 0.f;
            } else {
                tmem_ld32(tD + 32 * pc, v);
#pragma unroll
                for (int jj = 0; jj < 32; ++jj) {
                    const int j = c0 + jj;
                    v[jj] = j < row ? -bi * v[jj] * exp_e(gi - gcol[32 * pc + jj]) : 0.f;
                }
            }
            float4* dst = reinterpret_cast<float4*>(Ar + c0);
#pragma unroll
            for (int q = 0; q < 8; ++q) dst[q] = make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
        }
        if (gq == 0) {                                      // the upper-right block is zero
            float4* dst = reinterpret_cast<float4*>(Ar + 128);
#pragma unroll 4
            for (int q = 0; q < 32; ++q) dst[q] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        tc_fence_before();
        __syncthreads();                                    // accumulators free
    }
    if (timed_out) mbar_wait(mbar, phase);
    if (leader && issued > 0) mbar_wait(&full[(issued - 1) & 1], (uint32_t)(((issued - 1) >> 1) & 1));
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tm, 512);
    }
}

// ------------------------------------------------------------------------- //
// host side
// ------------------------------------------------------------------------- //
// [rows, cols] fp32, box 32 columns x 128 rows, 128-byte swizzle
static bool map_f32(CUtensorMap* m, const void* base, int64_t rows, int cols) {
    EncodeTiledFn f = encode_fn();
    if (!f) return false;
    cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)cols * 4};
    cuuint32_t box[2] = {32, (cuuint32_t)kRows};
    cuuint32_t es[2] = {1, 1};
    return f(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, const_cast<void*>(base), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// [rows] fp32, box 128 (rows past the end read as zero)
static bool map_vec(CUtensorMap* m, const void* base, int64_t rows) {
    EncodeTiledFn f = encode_fn();
    if (!f) return false;
    cuuint64_t dims[1] = {(cuuint64_t)rows};
    cuuint64_t strides[1] = {4};
    cuuint32_t box[1] = {(cuuint32_t)kRows};
    cuuint32_t es[1] = {1};
    return f(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 1, const_cast<void*>(base), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
             CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

static int num_sms() {
    int dev = 0, n = 148;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    return n;
}

struct IO {
    const void* K = nullptr;
    const void* V = nullptr;
    const float* beta = nullptr;
    const float* g = nullptr;
    void* W = nullptr;
    void* U = nullptr;
};

template <int KC, int MODE, int NS, int SN = 0, int SS = -1, int SG = -1>
static cudaError_t launch(const IO& io, const Params& p0, cudaStream_t st) {
    // the band path at N = 3, S = 8 (the method's setting for 64 x 64 chunks)
    // runs an instance with the orders and the gating fixed at compile time:
    // 8 % faster on 4096 chunks than the same kernel reading them from the
    // parameters
    if constexpr ((MODE == kFusedBand || MODE == kFusedRawBand) && SN == 0 && SS < 0)
        if (p0.N == 3 && p0.S == 8)
            return p0.gated ? launch<KC, MODE, NS, 3, 8, 1>(io, p0, st)
                            : launch<KC, MODE, NS, 3, 8, 0>(io, p0, st);
    // the standalone inverse at N = 3 with S = 0 (the chunk-size sweep's
    // setting, every k) and, at k = 64, S = 8 (the pages' setting), likewise
    if constexpr (MODE == kNeumann && SN == 0 && SS < 0) {
        if (p0.N == 3 && p0.S == 0) return launch<KC, MODE, NS, 3, 0>(io, p0, st);
        if constexpr (KC == 64)
            if (p0.N == 3 && p0.S == 8) return launch<KC, MODE, NS, 3, 8>(io, p0, st);
    }
    using KS = KernelShape<KC, MODE, NS>;
    static_assert(KS::smem <= 232448, "shared memory budget");
    CUtensorMap mK, mV, mW, mU, mB, mG;
    memset(&mK, 0, sizeof mK);
    memset(&mV, 0, sizeof mV);
    memset(&mW, 0, sizeof mW);
    memset(&mU, 0, sizeof mU);
    memset(&mB, 0, sizeof mB);
    memset(&mG, 0, sizeof mG);
    if (uses_K(MODE)) {
        if (!map_kd(&mK, io.K, p0.rows) || !map_vec(&mB, io.beta, p0.rows) ||
            !map_vec(&mG, io.g ? io.g : io.beta, p0.rows))
            return cudaErrorInvalidValue;
    }
    if (uses_V(MODE)) {
        if (!map_kd(&mV, io.V, p0.rows) || !map_kd(&mW, io.W, p0.rows) ||
            !map_kd(&mU, io.U, p0.rows))
            return cudaErrorInvalidValue;
    }
    if (inv_only(MODE)) {                          // A in through mK, T out through mW
        if (!map_f32(&mK, p0.Ain, p0.rows, KC) || !map_f32(&mW, p0.Tout, p0.rows, KC))
            return cudaErrorInvalidValue;
    }
    Params p = p0;
    p.status = status_ptr();
    size_t smem = KS::smem;
    if (smem < 120 * 1024) smem = 120 * 1024;     // one CTA per SM: it owns the SM's TMEM
    cudaError_t e = cudaFuncSetAttribute(k_chunk_tc<KC, MODE, NS, SN, SS, SG>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    const int grid = p.ntiles < num_sms() ? p.ntiles : num_sms();
    k_chunk_tc<KC, MODE, NS, SN, SS, SG><<<grid, KS::threads, smem, st>>>(mK, mV, mW, mU, mB, mG, p);
    return cudaGetLastError();
}

static Params base_params(int64_t nc, int k) {
    Params p;
    memset(&p, 0, sizeof p);
    p.rows = nc * k;
    p.ntiles = (int)((p.rows + kRows - 1) / kRows);
    p.timeout_ns = kTimeoutNs;
    p.withhold_tile = -1;
    return p;
}

// chunk size -> kernel instance; NS128 = slots per CTA at k = 128
template <int MODE, int NS128>
static cudaError_t dispatch(int k, const IO& io, const Params& p, cudaStream_t st) {
    switch (k) {
        case 32: return launch<32, MODE, 2>(io, p, st);
        case 64: return launch<64, MODE, 2>(io, p, st);
        case 128: return launch<128, MODE, NS128>(io, p, st);
        default: return cudaErrorNotSupported;
    }
}

}  // namespace tcg

bool tc_available() { return true; }
bool tc_i8_available() { return true; }

cudaError_t launch_build_A_tc(const void* K, const float* beta, const float* g, float* A,
                              int64_t nc, int k, cudaStream_t st) {
    tcg::Params p = tcg::base_params(nc, k);
    p.Aout = A;
    tcg::IO io;
    io.K = K;
    io.beta = beta;
    io.g = g;
    return tcg::dispatch<tcg::kBuildA, 2>(k, io, p, st);
}

cudaError_t launch_build_A256_tc(const void* K, const float* beta, const float* g, float* A,
                                 int64_t nc, cudaStream_t st) {
    CUtensorMap mK;
    memset(&mK, 0, sizeof mK);
    if (!tcg::map_kd(&mK, K, nc * 256)) return cudaErrorInvalidValue;
    tcg::ParamsA256 p;
    p.nc = nc;
    p.beta = beta;
    p.g = g;
    p.A = A;
    p.status = status_ptr();
    cudaError_t e = cudaFuncSetAttribute(tcg::k_build_A256_tc,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, tcg::kA256Smem);
    if (e != cudaSuccess) return e;
    const int sms = tcg::num_sms();
    const int grid = nc < sms ? (int)nc : sms;
    tcg::k_build_A256_tc<<<grid, 384, tcg::kA256Smem, st>>>(mK, p);
    return cudaGetLastError();
}

cudaError_t launch_neumann_tc(const float* A, float* T, int64_t nc, int k, int N, int mask, int S,
                              cudaStream_t st) {
    tcg::Params p = tcg::base_params(nc, k);
    p.Ain = A;
    p.Tout = T;
    p.N = N;
    p.mask = mask;
    p.S = S;
    return tcg::dispatch<tcg::kNeumann, 1>(k, tcg::IO(), p, st);
}

cudaError_t launch_blockinv_tc(const float* A, float* T, int64_t nc, int k, cudaStream_t st) {
    tcg::Params p = tcg::base_params(nc, k);
    p.Ain = A;
    p.Tout = T;
    p.N = 1;
    switch (k) {
        case 32: return tcg::launch<32, tcg::kBlockInv, 2>(tcg::IO(), p, st);
        case 64: return tcg::launch<64, tcg::kBlockInv, 2>(tcg::IO(), p, st);
        default: return cudaErrorNotSupported;
    }
}

cudaError_t launch_newton_tc(const float* A, float* T, int64_t nc, int k, int N, int mask, int M,
                             cudaStream_t st) {
    tcg::Params p = tcg::base_params(nc, k);
    p.Ain = A;
    p.Tout = T;
    p.N = N;
    p.mask = mask;
    p.M = M;
    return tcg::dispatch<tcg::kNewton, 1>(k, tcg::IO(), p, st);
}

cudaError_t launch_wy_tc(const float* T, const void* K, const void* V, const float* beta,
                         const float* g, void* W, void* U, int64_t nc, int k, cudaStream_t st) {
    tcg::Params p = tcg::base_params(nc, k);
    p.Tin = T;
    p.gated = g != nullptr;
    tcg::IO io;
    io.K = K;
    io.V = V;
    io.beta = beta;
    io.g = g;
    io.W = W;
    io.U = U;
    return tcg::dispatch<tcg::kWY, 1>(k, io, p, st);
}

// one instance of the integer kernels: shared-memory attribute, then the launch
template <bool RES, int SN, int SS>
static cudaError_t run_i8(const CUtensorMap& mA, const tcg::ParamsI8& p, int grid, size_t smem,
                          cudaStream_t st) {
    cudaError_t e = cudaFuncSetAttribute(tcg::k_neumann_i8_tc<RES, SN, SS>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    tcg::k_neumann_i8_tc<RES, SN, SS><<<grid, 256 * tcg::kI8Slots, smem, st>>>(mA, p);
    return cudaGetLastError();
}
template <bool RES, int SN, int SS>
static cudaError_t run_i16(const CUtensorMap& mA, const tcg::ParamsI16& p, int grid, size_t smem,
                           cudaStream_t st) {
    cudaError_t e = cudaFuncSetAttribute(tcg::k_neumann_i16_tc<RES, SN, SS>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    tcg::k_neumann_i16_tc<RES, SN, SS><<<grid, 256, smem, st>>>(mA, p);
    return cudaGetLastError();
}

cudaError_t launch_neumann_i8_tc(const float* A, float* T, int N, int mask, int8_t* q,
                                 int32_t* acc, float* sc, int64_t nc, cudaStream_t st, int S) {
    tcg::ParamsI8 p;
    memset(&p, 0, sizeof p);
    p.S = S;
    p.rows = nc * 64;
    p.ntiles = (int)((p.rows + tcg::kRows - 1) / tcg::kRows);
    p.N = N;
    p.mask = mask;
    p.A = A;
    p.T = T;
    p.q = q;
    p.acc = acc;
    p.scale = sc;
    p.status = status_ptr();
    CUtensorMap mA;
    memset(&mA, 0, sizeof mA);
    if (!tcg::map_f32(&mA, A, p.rows, 64)) return cudaErrorInvalidValue;
    // two CTAs per SM at most: each holds 256 of the SM's 512 TMEM columns
    const size_t smem = tcg::kI8Slots * tcg::kI8SlotBytes + 512;
    const int cap = 2 * tcg::num_sms();
    const int grid = p.ntiles < cap ? p.ntiles : cap;
    // N = 3 (with S = 8 for the residual), the method's setting for the
    // quantised paths, runs instances with the orders fixed at compile time
    if (p.S > 0)
        return (p.N == 3 && p.S == 8) ? run_i8<true, 3, 8>(mA, p, grid, smem, st)
                                      : run_i8<true, 0, -1>(mA, p, grid, smem, st);
    return p.N == 3 ? run_i8<false, 3, -1>(mA, p, grid, smem, st)
                    : run_i8<false, 0, -1>(mA, p, grid, smem, st);
}

cudaError_t launch_neumann_i16_tc(const float* A, float* T, int N, int mask, int16_t* q,
                                  int64_t* acc, double* sc, int64_t nc, cudaStream_t st, int S) {
    tcg::ParamsI16 p;
    memset(&p, 0, sizeof p);
    p.S = S;
    p.rows = nc * 64;
    p.ntiles = (int)((p.rows + tcg::kRows - 1) / tcg::kRows);
    p.N = N;
    p.mask = mask;
    p.A = A;
    p.T = T;
    p.q = q;
    p.acc = acc;
    p.scale = sc;
    p.status = status_ptr();
    CUtensorMap mA;
    memset(&mA, 0, sizeof mA);
    if (!tcg::map_f32(&mA, A, p.rows, 64)) return cudaErrorInvalidValue;
    // one CTA per SM: it takes all 512 TMEM columns (the shared-memory request
    // keeps a second CTA off the SM)
    size_t smem = tcg::kI16Smem + tcg::kI16Ctrl + (S > 0 ? tcg::kI16T0 : 0);
    if (smem < 120 * 1024) smem = 120 * 1024;
    const int sms = tcg::num_sms();
    const int grid = p.ntiles < sms ? p.ntiles : sms;
    if (S > 0)
        return (N == 3 && S == 8) ? run_i16<true, 3, 8>(mA, p, grid, smem, st)
                                  : run_i16<true, 0, -1>(mA, p, grid, smem, st);
    return N == 3 ? run_i16<false, 3, -1>(mA, p, grid, smem, st)
                  : run_i16<false, 0, -1>(mA, p, grid, smem, st);
}

cudaError_t launch_neumann256_tc(const float* A, float* T, int64_t nc, int N, int mask, int S,
                                cudaStream_t st) {
    tcg::Params256 p;
    p.nc = nc;
    p.N = N;
    p.mask = mask;
    p.S = S;
    p.A = A;
    p.T = T;
    p.status = status_ptr();
    cudaError_t e = cudaFuncSetAttribute(tcg::k_neumann256_tc,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         tcg::k256Smem);
    if (e != cudaSuccess) return e;
    const int sms = tcg::num_sms();
    const int grid = nc < sms ? (int)nc : sms;
    tcg::k_neumann256_tc<<<grid, tcg::k256Threads, tcg::k256Smem, st>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_output_tc(const void* Q, const void* K, const void* Vt, const float* g,
                             const void* Sst, void* O, int64_t nchunks, bool normalize_q,
                             cudaStream_t st) {
    using namespace tcg;
    const int64_t rows = nchunks * 64;
    CUtensorMap mQ, mK, mV, mS, mG, mO;
    if (!map_kd(&mQ, Q, rows) || !map_kd(&mK, K, rows) || !map_kd(&mV, Vt, rows) ||
        !map_kd(&mS, Sst, nchunks * kD) || !map_vec(&mG, g, rows) || !map_kd(&mO, O, rows))
        return cudaErrorInvalidValue;
    ParamsOut p;
    memset(&p, 0, sizeof p);
    p.rows = rows;
    p.nchunks = nchunks;
    p.ntiles = (int)((rows + kRows - 1) / kRows);
    p.normalize_q = normalize_q ? 1 : 0;
    p.status = status_ptr();
    const int smem = kOutSmem + (int)sizeof(CtrlOut);
    cudaError_t e =
        cudaFuncSetAttribute(k_output_tc, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    const int grid = p.ntiles < num_sms() ? p.ntiles : num_sms();
    k_output_tc<<<grid, kOutThreads, smem, st>>>(mQ, mK, mV, mS, mG, mO, p);
    return cudaGetLastError();
}

static thread_local int t_withhold_tile = -1;
static thread_local int t_withhold_v = 0;
static thread_local unsigned long long t_expiry_ns = 0;

void arm_wait_expiry(int tile, int v, unsigned long long timeout_ns) {
    t_withhold_tile = tile;
    t_withhold_v = v;
    t_expiry_ns = timeout_ns;
}

cudaError_t launch_fused_tc(const void* K, const void* V, const float* beta, const float* g,
                            int N, int mask, int S, int gated, void* W, void* U, float* Tout,
                            int64_t nc, int k, cudaStream_t st) {
    tcg::Params p = tcg::base_params(nc, k);
    if (t_withhold_tile >= 0) {                 // armed once by gdn_debug_arm_wait_expiry
        p.withhold_tile = t_withhold_tile;
        p.withhold_v = t_withhold_v;
        p.timeout_ns = t_expiry_ns;
        t_withhold_tile = -1;
    }
    p.N = N;
    p.mask = mask;
    p.S = S;
    p.gated = gated;
    p.Tout = Tout;
    tcg::IO io;
    io.K = K;
    io.V = V;
    io.beta = beta;
    io.g = g;
    io.W = W;
    io.U = U;
    if (k == 64 && mask && N <= tcg::kBandMax) return tcg::launch<64, tcg::kFusedBand, 2>(io, p, st);
    return tcg::dispatch<tcg::kFused, 1>(k, io, p, st);
}

cudaError_t launch_fused_raw_tc(const void* K, const void* V, const float* beta,
                                const float* loggate, int N, int mask, int S, int gated, void* W,
                                void* U, float* Tout, void* Kout, float* gout, int64_t nc, int k,
                                cudaStream_t st) {
    tcg::Params p = tcg::base_params(nc, k);
    p.N = N;
    p.mask = mask;
    p.S = S;
    p.gated = gated;
    p.Tout = Tout;
    p.Kout = static_cast<__nv_bfloat16*>(Kout);
    p.gout = gout;
    tcg::IO io;
    io.K = K;
    io.V = V;
    io.beta = beta;
    io.g = loggate;
    io.W = W;
    io.U = U;
    if (k == 64 && mask && N <= tcg::kBandMax)
        return tcg::launch<64, tcg::kFusedRawBand, 2>(io, p, st);
    return tcg::dispatch<tcg::kFusedRaw, 1>(k, io, p, st);
}

}  // namespace gdn
