// linear.h — internal structures of linear attention with a decay per head
// (linear.cu: host side and CUDA-core kernels; linear_tc.cu: tcgen05 kernels).
#pragma once

#include "common.cuh"
#include "kernels.h"

namespace gdn {

constexpr int kLinD = 128;                             // head dim
constexpr int kLinState = kLinD * kLinD;               // floats of one state

// One decayed linear attention.  With queries a, keys b, values c of one head
// and lambda = exp(loggate):
//   forward:  out_i = s_out [ s_weight sum_{j<=i} lambda^(i-j) (a_i.b_j) c_j + lambda^(i+1) M a_i ]
//             M'    = lambda^n M + s_state sum_j lambda^(n-1-j) c_j b_j^T
//   reverse:  out_i = s_out [ s_weight sum_{j>=i} lambda^(j-i) (a_i.b_j) c_j + lambda^(n-1-i) M a_i ]
//             M'    = lambda^n M + s_state sum_j lambda^(j+1) c_j b_j^T
// over n rows whose incoming state is M (entering at the first row, or at the
// last one if reverse).  The forward pass is (a, b, c) = (q, k, v); the
// gradients are three more: dq from (do, v, k), and in reverse dk from
// (v, do, q) and dv from (k, q, do).
struct LinProblem {
    const void* a; const void* b; const void* c;
    void* out;
    int ga, gb, gc;            // value heads per head of a, b, c
    int reverse;
    int out_f32;               // out is float32 whatever the data type
    const float* m0; int m0_t; // incoming state of each sequence (or null); transposed
    float* mout;               // outgoing state of each sequence (or null)
    int has_state;             // the call has an outgoing state here, wanted or not
    float s_out, s_weight, s_state;
    int ws_t;                  // the boundary states are another problem's, transposed
    float* ws;                 // states at the segment boundaries [boundary][128][128]
};
constexpr int kLinProblems = 3;

// Sequences are cut into segments of seg_len rows that run in parallel, each
// from the state at its boundary.
struct LinArgs {
    LinProblem pr[kLinProblems];
    const float* loggate;      // [Hv]
    const int32_t* cu;         // packed: [nseq + 1], else null
    int64_t nseq;              // sequences
    int64_t B, Hv, T;
    int nprob;
    int64_t seg_len;           // a multiple of 128
    int64_t whole;             // sequences x heads, the first ones, that stay whole (not packed)
    int64_t bounds;            // states in a problem's ws
    int* status;
};

// A block's work: problem z, head hv, rows [t0, t0 + n) of batch row b, which are
// segment number k of m of their sequence.  The state at the sequence's boundary
// i (between segments i and i + 1) is number st0 + i st_step in ws.
struct LinSeg {
    int z, hv;
    int64_t seq, b, t0, n;
    int k, m;
    int64_t st0, st_step;
    int64_t seq_t0, seq_n;
    bool ok;
};

__device__ __forceinline__ int64_t lin_segments(int64_t n, int64_t seg_len) {
    return n <= seg_len ? 1 : (n + seg_len - 1) / seg_len;
}
__device__ __forceinline__ void lin_bounds(const LinArgs& p, int64_t s, int64_t& t0, int64_t& n) {
    const int64_t lo = p.cu[s], hi = p.cu[s + 1];
    if (lo < 0 || hi < lo || hi > p.T) {               // bad bounds: no rows, and the status word
        raise_status(p.status, kStatusIndex);
        t0 = 0;
        n = 0;
    } else {
        t0 = lo;
        n = hi - lo;
    }
}
// Packed sequences come in classes by their share of all rows, so that the long
// ones start first whatever their places: class 0 has above a half, class 4 up
// to a 16th.  32 heads, 73 chunks, 32 of them one sequence's: 153 us in the
// order of the sequences, 125 us so (114 with the next chunk's scores early);
// backward in float32 231 and 172 us.
constexpr int kLinClasses = 5;
__device__ __forceinline__ int lin_class(int64_t n, int64_t rows) {
    return (2 * n <= rows) + (4 * n <= rows) + (8 * n <= rows) + (16 * n <= rows);
}
// g's own rows, from its sequence's
__device__ __forceinline__ void lin_rows(const LinArgs& p, LinSeg& g) {
    g.t0 = g.seq_t0 + g.k * p.seg_len;
    g.n = g.seq_n - g.k * p.seg_len;                   // one of one may be longer than a segment
    if (g.m > 1 && g.n > p.seg_len) g.n = p.seg_len;
    g.ok = true;
}
// What lin_find counts: every segment (one at least per sequence), or the
// segments of the sequences that have several.
enum : int { kAllSegments = 0, kCutSegments = 1 };
__device__ __forceinline__ int lin_counted(int m, int which) {
    return which == kCutSegments && m < 2 ? 0 : m;
}
struct LinFound {                                      // of a block, in shared memory
    LinSeg seg;
    uint32_t count[32][kLinClasses + 1];               // by warp: of each class; boundaries
};
// The work of a block, by the first `warps` of its warps.  Problems and heads
// come first, as those of one segment share inputs.  Each warp counts a stretch
// of the packed sequences, 32 at a time.
__device__ __forceinline__ void lin_search(const LinArgs& p, uint32_t block, int which, int warps,
                                           LinFound& f) {
    LinSeg g;
    g.ok = false;
    if (threadIdx.x == 0) f.seg = g;
    g.z = (int)(block % (uint32_t)p.nprob);
    uint32_t idx = block / (uint32_t)p.nprob;
    if (!p.cu) {
        // the whole ones (sequence, head), then the cut ones' segments
        const uint32_t units = (uint32_t)(p.nseq * p.Hv), whole = (uint32_t)p.whole;
        uint32_t u = idx;
        g.k = 0;
        g.m = 1;
        g.st0 = 0;
        if (which == kCutSegments || idx >= whole) {
            if (which == kAllSegments) idx -= whole;
            const uint32_t cut = units - whole;
            g.m = (int)lin_segments(p.T, p.seg_len);
            if (cut == 0 || idx >= cut * (uint64_t)g.m) return;
            g.k = (int)(idx / cut);
            u = idx - g.k * cut;
            g.st0 = (int64_t)u * (g.m - 1);
            u += whole;
        }
        g.st_step = 1;
        g.seq = u / (uint32_t)p.Hv;
        g.hv = (int)(u - (uint32_t)g.seq * (uint32_t)p.Hv);
        g.b = g.seq;
        g.seq_t0 = 0;
        g.seq_n = p.T;
        if (g.m > 1 && g.st0 + g.m - 1 > p.bounds) return;
        lin_rows(p, g);
        if (threadIdx.x == 0) f.seg = g;
        return;
    }
    g.hv = (int)(idx % (uint32_t)p.Hv);
    idx /= (uint32_t)p.Hv;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t per = (p.nseq + 32 * warps - 1) / (32 * warps) * 32;
    const int64_t lo = warp * per, hi = lo + per < p.nseq ? lo + per : p.nseq;
    int64_t t0 = 0, n = 0;
    int m = 0, cls = -1;
    auto read = [&](int64_t s) {
        t0 = n = 0;
        m = 0;
        cls = -1;
        if (s >= hi) return;
        lin_bounds(p, s, t0, n);
        m = (int)lin_segments(n, p.seg_len);
        cls = lin_class(n, p.T);
    };
    uint32_t count[kLinClasses + 1] = {};
    for (int64_t s0 = lo; s0 < hi; s0 += 32) {
        read(s0 + lane);
#pragma unroll
        for (int c = 0; c < kLinClasses; ++c)
            count[c] += __reduce_add_sync(0xffffffffu, cls == c ? lin_counted(m, which) : 0);
        count[kLinClasses] += __reduce_add_sync(0xffffffffu, m > 1 ? m - 1 : 0);
    }
    if (lane == 0)
#pragma unroll
        for (int c = 0; c <= kLinClasses; ++c) f.count[warp][c] = count[c];
    if (warps > 1) __syncthreads();
    else __syncwarp();
    // the class, and the warp whose stretch has it
    int want = 0;
#pragma unroll
    for (int c = 0; c < kLinClasses; ++c) {
        const uint32_t all =
            __reduce_add_sync(0xffffffffu, lane < warps ? f.count[lane][c] : 0);
        if (want == c && idx >= all) {
            idx -= all;
            ++want;
        }
    }
    if (want == kLinClasses) return;
    uint32_t inc = lane < warps ? f.count[lane][want] : 0;
    const uint32_t own = inc;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t a = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += a;
    }
    const int owner = __ffs(__ballot_sync(0xffffffffu, idx >= inc - own && idx < inc)) - 1;
    uint32_t before = __shfl_sync(0xffffffffu, inc - own, owner);
    int64_t slots = __reduce_add_sync(0xffffffffu, lane < owner ? f.count[lane][kLinClasses] : 0);
    if (warp != owner) return;
    bool found = false;
    for (int64_t s0 = lo; s0 < hi && !found; s0 += 32) {
        if (per > 32) read(s0 + lane);
        const int mine = cls == want ? lin_counted(m, which) : 0;
        int sum = mine, sinc = m ? m - 1 : 0;          // inclusive sums over the lanes
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int a = __shfl_up_sync(0xffffffffu, sum, o);
            const int b = __shfl_up_sync(0xffffffffu, sinc, o);
            if (lane >= o) { sum += a; sinc += b; }
        }
        found = mine > 0 && idx < before + sum && idx >= before + sum - mine;
        if (found) {                                   // one lane
            g.seq = s0 + lane;
            g.k = (int)(idx - before) - (sum - mine);
            g.m = m;
            g.seq_t0 = t0;
            g.seq_n = n;
            slots += sinc - (m - 1);
            g.b = 0;
            g.st0 = slots * p.Hv + g.hv;
            g.st_step = p.Hv;
            if ((slots + m - 1) * p.Hv > p.bounds)     // only sequences that overlap need more
                raise_status(p.status, kStatusIndex);
            else
                lin_rows(p, g);
            f.seg = g;
        }
        found = __any_sync(0xffffffffu, found);
        slots += __shfl_sync(0xffffffffu, sinc, 31);
        before += __shfl_sync(0xffffffffu, sum, 31);
    }
}
// The same, for all threads of a block.  One warp finds it where one count of 32
// will do: with all warps at it the start of every block was 5 us later.  Of
// 1000 sequences of 4 rows and 8 heads: one warp 1650 us, all of them 830 us.
__device__ __forceinline__ LinSeg lin_find(const LinArgs& p, uint32_t block, int which,
                                           LinFound& f) {
    const int warps = p.cu && p.nseq > 32 ? (int)(blockDim.x >> 5) : 1;
    if ((int)(threadIdx.x >> 5) < warps) lin_search(p, block, which, warps, f);
    __syncthreads();
    return f.seg;
}

// How a call is cut: the same for its workspace size and its launches.
struct LinPlan {
    int64_t seg_len, whole, bounds;
    int64_t blocks, cut_blocks;                        // of lin_find; upper bounds if packed
    int64_t units;                                     // sequences x heads that may be cut
    int64_t state_bytes;                               // boundary states of one problem
};
LinPlan linear_plan(const gdn_linear_shape& s, int nprob, bool bf16);
// ws: nprob * state_bytes; *launches counts the kernels
cudaError_t launch_linear(const LinArgs& a, int nprob, const LinPlan& pl, bool bf16, void* ws,
                          int* launches, cudaStream_t st);
// one of the two tensor-core kernels (linear_tc.cu): the boundary states, or the outputs
cudaError_t launch_linear_tc(const LinArgs& a, int nprob, const LinPlan& pl, bool states,
                             cudaStream_t st);
// the next launch of one of them: block `block` waits for a tile that never comes
void arm_linear_expiry(int block, bool states, unsigned long long limit_ns);
// out[b, h] = sum of part[b, h * group + g] over g, float32 -> the data type
cudaError_t launch_linear_group_sum(const LinArgs& a, const float* part, void* out, int group,
                                    bool bf16, cudaStream_t st);

__device__ __forceinline__ float* lin_boundary(const LinProblem& q, const LinSeg& g, int64_t i) {
    return q.ws + (g.st0 + i * g.st_step) * kLinState;
}
// Where step 1 leaves what segment k adds to the state: the slot of the
// boundary that it ends at in walking order; the walk's last segment ends at
// none, its place is the outgoing state itself (null if that is not wanted).
__device__ __forceinline__ float* lin_added(const LinArgs& p, const LinProblem& q, const LinSeg& g) {
    const bool last = q.reverse ? g.k == 0 : g.k == g.m - 1;
    if (last) return q.mout ? q.mout + (g.seq * p.Hv + g.hv) * kLinState : nullptr;
    return lin_boundary(q, g, q.reverse ? g.k - 1 : g.k);
}

// log2 of the decay; -inf (no memory at all) becomes a finite number whose
// product with a distance of zero is zero.  A NaN stays one here and below.
__device__ __forceinline__ double lin_log2(const float* loggate, int hv) {
    const double x = (double)loggate[hv] * 1.4426950408889634;
    return x < -1e30 ? -1e30 : x;
}
// an exponent of two, as far as floats and doubles care (the identity for NaN,
// which fmin and fmax are not)
__device__ __forceinline__ double lin_clamp(double x) {
    return x < -1000.0 ? -1000.0 : (x > 1000.0 ? 1000.0 : x);
}
// lambda^n, 1 for n = 0 whatever lambda: the exponent in binary64 and its
// fraction alone to exp2f, so that the error stays at exp2f's two units however
// far n reaches
__device__ __forceinline__ float lin_pow(double lg, int64_t n) {
    if (n == 0) return 1.f;
    const double x = lg * (double)n, i = rint(x);
    return ldexpf(exp2f((float)(x - i)), (int)lin_clamp(i));
}
// the same as a sum of two floats
__device__ __forceinline__ void lin_pow2(double lg, int64_t n, float& hi, float& lo) {
    const double x = n == 0 ? 1.0 : exp2(lin_clamp(lg * (double)n));
    hi = (float)x;
    lo = (float)(x - (double)hi);
}

// lambda itself as a sum of two floats, for walks token by token: the rounding
// of one comes back at every token, 3e-4 of the state over 16384 of them.  Near
// one the distance from one has float32's relative accuracy, which 1 / loggate
// tokens turn into 2^-23 in all; a decay of e^-0.5 or faster forgets its rounding.
__device__ __forceinline__ void lin_decay(float loggate, float& hi, float& lo) {
    if (fabsf(loggate) < 0.5f) {
        const float d = expm1f(loggate);
        hi = 1.f + d;
        lo = d - (hi - 1.f);
    } else {
        hi = expf(loggate);
        lo = 0.f;
    }
}

}  // namespace gdn
