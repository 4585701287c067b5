// linear.cu — linear attention with one decay per head: host side, the states
// at segment boundaries, shared-head gradients, and the float32 kernel
// (gdn_linear_forward, gdn_linear_backward).
//
// S_t = lambda_h S_{t-1} + v_t k_t^T, o_t = scale S_t q_t.  Within a chunk the
// products are dense (queries with keys, weights with values); between chunks
// only the 128 x 128 state is carried, so the work is linear in the length.
// A sequence's recurrence is cut into segments that run in parallel:
//   1. the states that segments add, each from zero (the state kernels);
//   2. k_lin_combine: the states at the boundaries and the outgoing one, in order;
//   3. every segment's outputs from its incoming state.
// One segment per sequence needs step 3 alone.  Step 1 reads keys and values
// once more, so the cut is made only where sequences times heads leave SMs
// idle (pick_segment).  The gradients are three recurrences of the same form
// (linear.h) and go through the same kernels, three problems to a launch.
#include "linear.h"

namespace gdn {
namespace {

// ---- step 2: boundary states ----
// Slot k of a sequence holds what segment k (k + 1 if reverse) adds from zero;
// it is replaced by the state that crosses that boundary.
constexpr int kCombineThreads = 256;
__global__ void __launch_bounds__(kCombineThreads) k_lin_combine(const LinArgs p) {
    const LinProblem& q = p.pr[blockIdx.z];
    if (q.ws_t) return;
    // blockIdx.x: (sequence, head), past those that are whole
    const int64_t seq = (p.whole + blockIdx.x) / p.Hv;
    const int hv = (int)(p.whole + blockIdx.x - seq * p.Hv);
    LinSeg g;
    if (p.cu) {
        // the sequence's first boundary: those of the sequences before it
        const int lane = threadIdx.x & 31;
        int64_t slots = 0, t0, n;
        lin_bounds(p, seq, t0, n);
        if (n <= p.seg_len) return;
        for (int64_t s = lane; s < seq; s += 32) {
            lin_bounds(p, s, t0, n);
            slots += lin_segments(n, p.seg_len) - 1;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) slots += __shfl_xor_sync(0xffffffffu, slots, o);
        lin_bounds(p, seq, t0, n);
        g.st0 = slots * p.Hv + hv;
        g.st_step = p.Hv;
        g.seq_n = n;
        g.m = (int)lin_segments(n, p.seg_len);
        if ((slots + g.m - 1) * p.Hv > p.bounds) return;
    } else {
        g.seq_n = p.T;
        g.m = (int)lin_segments(p.T, p.seg_len);
        g.st0 = blockIdx.x * (int64_t)(g.m - 1);
        g.st_step = 1;
        if (g.st0 + g.m - 1 > p.bounds) return;
    }
    if (g.m < 2) return;
    const double lg = lin_log2(p.loggate, hv);
    float full, full_lo, last, last_lo;                // a decay's own rounding would add up
    lin_pow2(lg, p.seg_len, full, full_lo);
    lin_pow2(lg, g.seq_n - (g.m - 1) * p.seg_len, last, last_lo);
    const auto decayed = [&](const float4& m, bool whole, const float4& u) {
        const float a = whole ? full : last, l = whole ? full_lo : last_lo;
        return make_float4(fmaf(a, m.x, fmaf(l, m.x, u.x)), fmaf(a, m.y, fmaf(l, m.y, u.y)),
                           fmaf(a, m.z, fmaf(l, m.z, u.z)), fmaf(a, m.w, fmaf(l, m.w, u.w)));
    };
    // a share of the state's elements, four to a thread at a time
    const int share = kLinState / gridDim.y;
    for (int e = blockIdx.y * share + 4 * threadIdx.x; e < (blockIdx.y + 1) * share;
         e += 4 * kCombineThreads) {
        float4 m = make_float4(0.f, 0.f, 0.f, 0.f);
        if (q.m0) {
            const float* s = q.m0 + (seq * p.Hv + hv) * kLinState;
            if (!q.m0_t) {
                m = *reinterpret_cast<const float4*>(s + e);
            } else {
                const int r = e / kLinD, c = e % kLinD;
                m = make_float4(s[c * kLinD + r], s[(c + 1) * kLinD + r], s[(c + 2) * kLinD + r],
                                s[(c + 3) * kLinD + r]);
            }
        }
        float4* const base = reinterpret_cast<float4*>(lin_boundary(q, g, 0) + e);
        const int64_t step = g.st_step * kLinState / 4;
        constexpr int kAhead = 8;                      // loads in flight
        for (int i0 = 0; i0 < g.m - 1; i0 += kAhead) {
            float4 u[kAhead];
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                const int i = i0 + j;
                if (i < g.m - 1) u[j] = base[(q.reverse ? g.m - 2 - i : i) * step];
            }
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                const int i = i0 + j;
                if (i >= g.m - 1) break;
                m = decayed(m, !(q.reverse && i == 0), u[j]);
                base[(q.reverse ? g.m - 2 - i : i) * step] = m;
            }
        }
        if (q.mout) {                                  // the walk's last segment left its part here
            float4* const out =
                reinterpret_cast<float4*>(q.mout + (seq * p.Hv + hv) * kLinState + e);
            *out = decayed(m, q.reverse, *out);
        }
    }
}

// ---- gradients of shared heads: the sum over the value heads of a group ----
// Is row t one of a sequence's?  By the whole warp, 32 starts at a look: the last
// that is not behind t has it if all bounds are in order.  A row not found there
// is of no sequence, or the bounds of others are bad and left out: all are tried.
__device__ __forceinline__ bool lin_has_row(const LinArgs& p, int64_t t) {
    const int lane = threadIdx.x & 31;
    const auto has = [&](int64_t s) {
        const int64_t lo = p.cu[s], hi = p.cu[s + 1];
        return lo >= 0 && lo <= t && t < hi && hi <= p.T;
    };
    int64_t s = 0;
    for (int64_t n = p.nseq; n > 1;) {
        const int64_t step = (n + 31) / 32, at = lane * step;
        const uint32_t before = __ballot_sync(0xffffffffu, at < n && p.cu[s + at] <= t);
        const int64_t skip = before ? (31 - __clz(before)) * step : 0;
        s += skip;
        n = n - skip < step ? n - skip : step;
    }
    if (has(s)) return true;
    bool found = false;
#pragma unroll 4
    for (int64_t i = lane; i < p.nseq; i += 32) found |= has(i);
    return __any_sync(0xffffffffu, found);
}
template <typename T>
__global__ void __launch_bounds__(256)
k_lin_group_sum(const LinArgs p, const float* part, T* out, int group) {
    const int64_t Hk = p.Hv / group;
    const int64_t v = (int64_t)blockIdx.x * 256 + threadIdx.x, row = v >> 5;   // a warp to a row
    const int64_t bh = row / p.T, t = row - bh * p.T, b = bh / Hk, h = bh - b * Hk;
    const int c = 4 * (int)(v & 31);
    if (bh >= p.B * Hk || (p.cu && !lin_has_row(p, t))) return;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int g = 0; g < group; ++g) {
        const float4 f = *reinterpret_cast<const float4*>(
            part + ((b * p.Hv + h * group + g) * p.T + t) * kLinD + c);
        s.x += f.x; s.y += f.y; s.z += f.z; s.w += f.w;
    }
    T* o = out + (bh * p.T + t) * kLinD + c;
    st_elem(o, 0, s.x); st_elem(o, 1, s.y); st_elem(o, 2, s.z); st_elem(o, 3, s.w);
}

// ---- steps 1 and 3 on CUDA cores ----
constexpr int kSimtThreads = 256;
constexpr int kSimtC = 64;                             // rows of a chunk
constexpr int kSimtDV = 32;                            // state rows (columns of c) per CTA
constexpr int kPitchD = kLinD + 4;                     // an odd number of 16-byte groups
constexpr int kPitchC = kSimtC + 4;

struct SimtSmem {
    float a[kSimtC][kPitchD];
    float b[kSimtC][kPitchD];
    float ct[kSimtDV][kPitchC];                        // values, transposed
    float m[kSimtDV][kPitchD];                         // the state slice
    float pm[kSimtC][kPitchC];                         // weights of the chunk
    float dec[kSimtC + 1];                             // lambda^0 .. lambda^64
    float an[2], an_lo[2];                             // lambda^n, a whole chunk's and the last one's
    int odd;                                           // a value was infinite or NaN
    LinFound found;
};

// The rows of a chunk split over 16 x 16 threads (scores) and 32 x 8 (outputs);
// each CTA carries 32 rows of the state, so four share a head and form the
// chunk's scores again, which costs less than passing them on: the float32
// peak of the CUDA cores is the bound either way.
template <bool STATE_ONLY, bool REV>
__device__ void simt_segment(const LinArgs& p, const LinProblem& q, const LinSeg& g, int hv,
                             int v0, SimtSmem& s) {
    const int tid = threadIdx.x;
    const double lg = lin_log2(p.loggate, hv);
    if (tid <= kSimtC) s.dec[tid] = lin_pow(lg, tid);
    if (tid == 0) s.odd = 0;
    const int last = (int)((g.n - 1) % kSimtC + 1);    // rows of the last chunk
    if (tid < 2) lin_pow2(lg, tid ? last : kSimtC, s.an[tid], s.an_lo[tid]);
    // incoming state
    for (int e = tid; e < kSimtDV * kLinD; e += kSimtThreads) {
        const int r = e / kLinD, c = e % kLinD;
        float m = 0.f;
        if (!STATE_ONLY) {
            const bool first = REV ? g.k == g.m - 1 : g.k == 0;
            if (!first) {
                const float* src = lin_boundary(q, g, REV ? g.k : g.k - 1);
                m = q.ws_t ? src[c * kLinD + v0 + r] : src[(v0 + r) * kLinD + c];
            } else if (q.m0) {
                const float* src = q.m0 + (g.seq * p.Hv + hv) * kLinState;
                m = q.m0_t ? src[c * kLinD + v0 + r] : src[(v0 + r) * kLinD + c];
            }
        }
        s.m[r][c] = m;
    }
    auto base = [&](int group) {
        const int64_t H = p.Hv / group;
        return ((g.b * H + hv / group) * p.T + g.t0) * kLinD;
    };
    const float* ga = (const float*)q.a + base(q.ga);
    const float* gb = (const float*)q.b + base(q.gb);
    const float* gc = (const float*)q.c + base(q.gc) + v0;
    const int64_t ob = ((g.b * p.Hv + hv) * p.T + g.t0) * kLinD + v0;
    const int64_t nch = (g.n + kSimtC - 1) / kSimtC;
    for (int64_t ci = 0; ci < nch; ++ci) {
        const int64_t r0 = (REV ? nch - 1 - ci : ci) * kSimtC;
        const int n = (int)(g.n - r0 < kSimtC ? g.n - r0 : kSimtC);
        __syncthreads();
        for (int e = tid; e < kSimtC * (kLinD / 4); e += kSimtThreads) {
            const int r = e / (kLinD / 4), c = 4 * (e % (kLinD / 4));
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
            if (r < n) {
                const int64_t o = (r0 + r) * kLinD + c;
                if (!STATE_ONLY) x = *reinterpret_cast<const float4*>(ga + o);
                y = *reinterpret_cast<const float4*>(gb + o);
            }
            if (!STATE_ONLY) *reinterpret_cast<float4*>(&s.a[r][c]) = x;
            *reinterpret_cast<float4*>(&s.b[r][c]) = y;
        }
        for (int e = tid; e < kSimtC * kSimtDV; e += kSimtThreads) {
            const int r = e / kSimtDV, c = e % kSimtDV;
            const float x = r < n ? gc[(r0 + r) * kLinD + c] : 0.f;
            if (!STATE_ONLY && !isfinite(x)) s.odd = 1;
            s.ct[c][r] = x;
        }
        __syncthreads();
        if (!STATE_ONLY) {
            {   // weights: rows ti + 16 u, columns tj + 16 w; blocks off the causal side are zero
                const int ti = tid >> 4, tj = tid & 15;
                float acc[4][4];
#pragma unroll
                for (int u = 0; u < 4; ++u)
#pragma unroll
                    for (int w = 0; w < 4; ++w) acc[u][w] = 0.f;
#pragma unroll 2
                for (int k = 0; k < kLinD; k += 4) {
                    float4 x[4], y[4];
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        x[u] = *reinterpret_cast<const float4*>(&s.a[ti + 16 * u][k]);
                        y[u] = *reinterpret_cast<const float4*>(&s.b[tj + 16 * u][k]);
                    }
#pragma unroll
                    for (int u = 0; u < 4; ++u)
#pragma unroll
                        for (int w = 0; w < 4; ++w)
                            if (REV ? w >= u : w <= u) {
                                acc[u][w] = fmaf(x[u].x, y[w].x, acc[u][w]);
                                acc[u][w] = fmaf(x[u].y, y[w].y, acc[u][w]);
                                acc[u][w] = fmaf(x[u].z, y[w].z, acc[u][w]);
                                acc[u][w] = fmaf(x[u].w, y[w].w, acc[u][w]);
                            }
                }
#pragma unroll
                for (int u = 0; u < 4; ++u)
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        const int i = ti + 16 * u, j = tj + 16 * w, dist = REV ? j - i : i - j;
                        s.pm[i][j] =
                            dist >= 0 && j < n ? q.s_weight * s.dec[dist] * acc[u][w] : 0.f;
                    }
            }
            __syncthreads();
            {   // outputs: rows ri, ri + 32, columns cj + 8 w
                const int ri = tid >> 3, cj = tid & 7;
                float in[2][4], st[2][4];
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int w = 0; w < 4; ++w) in[u][w] = st[u][w] = 0.f;
#pragma unroll 2
                for (int k = 0; k < kLinD; k += 4) {
                    float4 x[2], y[4];
#pragma unroll
                    for (int u = 0; u < 2; ++u)
                        x[u] = *reinterpret_cast<const float4*>(&s.a[ri + 32 * u][k]);
#pragma unroll
                    for (int w = 0; w < 4; ++w)
                        y[w] = *reinterpret_cast<const float4*>(&s.m[cj + 8 * w][k]);
#pragma unroll
                    for (int u = 0; u < 2; ++u)
#pragma unroll
                        for (int w = 0; w < 4; ++w) {
                            st[u][w] = fmaf(x[u].x, y[w].x, st[u][w]);
                            st[u][w] = fmaf(x[u].y, y[w].y, st[u][w]);
                            st[u][w] = fmaf(x[u].z, y[w].z, st[u][w]);
                            st[u][w] = fmaf(x[u].w, y[w].w, st[u][w]);
                        }
                }
                if (!s.odd) {
#pragma unroll 2
                    for (int k = 0; k < kSimtC; k += 4) {
                        float4 x[2], y[4];
#pragma unroll
                        for (int u = 0; u < 2; ++u)
                            x[u] = *reinterpret_cast<const float4*>(&s.pm[ri + 32 * u][k]);
#pragma unroll
                        for (int w = 0; w < 4; ++w)
                            y[w] = *reinterpret_cast<const float4*>(&s.ct[cj + 8 * w][k]);
#pragma unroll
                        for (int u = 0; u < 2; ++u)
#pragma unroll
                            for (int w = 0; w < 4; ++w) {
                                in[u][w] = fmaf(x[u].x, y[w].x, in[u][w]);
                                in[u][w] = fmaf(x[u].y, y[w].y, in[u][w]);
                                in[u][w] = fmaf(x[u].z, y[w].z, in[u][w]);
                                in[u][w] = fmaf(x[u].w, y[w].w, in[u][w]);
                            }
                    }
                } else {
                    // a weight of zero would make NaN of an infinite or NaN value,
                    // and the row is not to see what lies on its other side
#pragma unroll 1
                    for (int k = 0; k < kSimtC; ++k)
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            const int i = ri + 32 * u;
                            if (REV ? k < i : k > i) continue;
#pragma unroll
                            for (int w = 0; w < 4; ++w)
                                in[u][w] = fmaf(s.pm[i][k], s.ct[cj + 8 * w][k], in[u][w]);
                        }
                }
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int i = ri + 32 * u;
                    if (i >= n) continue;
                    const float d = REV ? s.dec[n - 1 - i] : s.dec[i + 1];
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        static_cast<float*>(q.out)[ob + (r0 + i) * kLinD + cj + 8 * w] =
                            q.s_out * fmaf(d, st[u][w], in[u][w]);
                    }
                }
            }
            __syncthreads();
        }
        {   // state: rows cr + 8 u (values), columns 4 kc .. 4 kc + 3 (keys)
            const int cr = tid >> 5, kc = 4 * (tid & 31);
            float4 acc[4];
            // as two floats: one's rounding is every chunk's and would add up
            const float an = s.an[n < kSimtC], al = s.an_lo[n < kSimtC];
#pragma unroll
            for (int u = 0; u < 4; ++u) acc[u] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
            for (int j = 0; j < kSimtC; j += 4) {
                float4 x[4], y[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    x[u] = *reinterpret_cast<const float4*>(&s.ct[cr + 8 * u][j]);
                    y[u] = *reinterpret_cast<const float4*>(&s.b[j + u][kc]);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int jj = j + e;
                    const float w = jj < n ? q.s_state * (REV ? s.dec[jj + 1] : s.dec[n - 1 - jj])
                                           : 0.f;
                    y[e].x *= w; y[e].y *= w; y[e].z *= w; y[e].w *= w;
                }
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const float xe[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        acc[u].x = fmaf(xe[e], y[e].x, acc[u].x);
                        acc[u].y = fmaf(xe[e], y[e].y, acc[u].y);
                        acc[u].z = fmaf(xe[e], y[e].z, acc[u].z);
                        acc[u].w = fmaf(xe[e], y[e].w, acc[u].w);
                    }
                }
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                float4* m = reinterpret_cast<float4*>(&s.m[cr + 8 * u][kc]);
                const float4 o = *m;
                *m = make_float4(fmaf(an, o.x, fmaf(al, o.x, acc[u].x)),
                                 fmaf(an, o.y, fmaf(al, o.y, acc[u].y)),
                                 fmaf(an, o.z, fmaf(al, o.z, acc[u].z)),
                                 fmaf(an, o.w, fmaf(al, o.w, acc[u].w)));
            }
        }
    }
    __syncthreads();
    // a sequence of several segments has its outgoing state from steps 1 and 2
    float* dst = nullptr;
    if (STATE_ONLY) dst = lin_added(p, q, g);
    else if (q.mout && g.m == 1) dst = q.mout + (g.seq * p.Hv + hv) * kLinState;
    if (dst)
        for (int e = tid; e < kSimtDV * kLinD; e += kSimtThreads)
            dst[v0 * kLinD + e] = s.m[e / kLinD][e % kLinD];
}

// four blocks, of 32 state rows each, for every one of lin_find's
template <bool STATE_ONLY>
__global__ void __launch_bounds__(kSimtThreads) k_linear_simt(const LinArgs p) {
    extern __shared__ __align__(16) uint8_t raw[];
    SimtSmem& s = *reinterpret_cast<SimtSmem*>(raw);
    const LinSeg g = lin_find(p, blockIdx.x >> 2,
                              STATE_ONLY ? kCutSegments : kAllSegments, s.found);
    if (!g.ok) return;
    const LinProblem& q = p.pr[g.z];
    if (STATE_ONLY && (q.ws_t || !lin_added(p, q, g))) return;
    const int hv = g.hv, v0 = (blockIdx.x & 3) * kSimtDV;
    if (q.reverse) simt_segment<STATE_ONLY, true>(p, q, g, hv, v0, s);
    else simt_segment<STATE_ONLY, false>(p, q, g, hv, v0, s);
}

cudaError_t run_simt(const LinArgs& a, int64_t blocks, bool states, cudaStream_t st) {
    const int smem = (int)sizeof(SimtSmem);
    const auto kernel = states ? k_linear_simt<true> : k_linear_simt<false>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    kernel<<<(unsigned)(4 * blocks), kSimtThreads, smem, st>>>(a);
    return cudaGetLastError();
}

// Segment length (a multiple of 128).  Costs are in units of half an output
// step (a chunk of 128 rows on one SM): a chunk of the state pass takes one, a
// CTA's start two in step 3 and one in step 1, the state at a boundary moves as
// much as two output steps, and two more launches cost eight.
// Sequences of one length are taken in waves: either all are cut alike (or not
// at all), or as many as fill whole waves stay whole, and the others' pieces
// follow as SMs come free.  64 heads x 4096 tokens backward (bf16) are 192
// lines on 148 SMs: 223 us in two waves, 198 us with 45 of them cut at 8 chunks,
// 215 us with all of them cut at 16.
struct LinCut {
    int64_t len, whole;
};
LinCut pick_segment(int64_t nprob, int64_t units, int64_t rows, int ctas_per_head) {
    const int64_t chunks = (rows + 127) / 128, sms = sm_count(), unit = nprob * ctas_per_head;
    const int64_t full = units * unit / sms;
    LinCut best{chunks, units};
    int64_t cost = (units * unit + sms - 1) / sms * (2 * chunks + 2);
    for (int64_t w = 0; w <= full; w += full > 0 ? full : 1) {
        const int64_t whole = w * sms / unit, cut = units - whole;
        for (int64_t m = 2; m <= chunks && m <= 128 && cut > 0; ++m) {
            const int64_t len = (chunks + m - 1) / m;
            if ((chunks + len - 1) / len != m) continue;  // as with fewer pieces
            const int64_t pieces = cut * unit * m, each = 3 * len + 3;
            const int64_t run = w > 0 ? w * (2 * chunks + 2) + pieces * each / sms + 3 * len / 2
                                      : (pieces + sms - 1) / sms * each;
            const int64_t c = run + 4 * cut * unit * (m - 1) / sms + 8;
            if (c < cost) { cost = c; best = {len, whole}; }
        }
    }
    return {best.len < 1 ? 128 : 128 * best.len, best.whole};
}
// Packed sequences have lengths that the host does not know.  Cut: all chunks
// spread over the SMs, half of a last segment behind them.  Not cut: that, or
// the longest sequence, taken to be half of the rows if there are several; its
// one piece returns a state, which takes a product more per chunk, hence 9/8 (73
// chunks of 32 heads, the longest 32: 114 us not cut, 127 to 141 us cut at 16
// to 8, 173 us at 4).
int64_t pick_segment_packed(int64_t nprob, int64_t nseq, int64_t Hv, int64_t rows,
                            int ctas_per_head) {
    const int64_t chunks = (rows + 127) / 128, sms = sm_count();
    const int64_t heads = nprob * Hv * ctas_per_head;
    const int64_t longest = nseq > 1 ? (chunks + 1) / 2 : chunks;
    const int64_t work = 2 * heads * (chunks + nseq) / sms;
    int64_t best = chunks;
    int64_t cost = (work > 2 * longest ? work : 2 * longest) * 9 / 8 + 2 * heads * nseq / sms;
    for (int64_t len = 1; len < longest; len += len < 16 ? 1 : len / 8) {
        const int64_t m = (chunks + len - 1) / len;    // segments of the cut ones
        const int64_t c = work + len + 2 * heads * (m + nseq) / sms + heads * (chunks + m) / sms +
                          len / 2 + 4 * nprob * Hv * m / sms + 8;
        if (c < cost) { cost = c; best = len; }
    }
    return best < 1 ? 128 : 128 * best;
}

}  // namespace

LinPlan linear_plan(const gdn_linear_shape& s, int nprob, bool bf16) {
    LinPlan pl;
    // on CUDA cores four CTAs share a head, two to an SM
    const int per = bf16 ? 1 : 2;
    if (s.nseq > 0) {
        pl.seg_len = pick_segment_packed(nprob, s.nseq, s.Hv, s.T, per);
        // a sequence of n rows has at most n / seg_len boundaries, and a segment more
        const int64_t m = s.T <= pl.seg_len ? 0 : s.T / pl.seg_len;
        pl.whole = 0;
        pl.units = s.nseq * s.Hv;
        pl.bounds = m * s.Hv;
        pl.blocks = (s.nseq + m) * s.Hv * nprob;
        pl.cut_blocks = (m + (s.nseq < m ? s.nseq : m)) * s.Hv * nprob;
    } else {
        const LinCut cut = pick_segment(nprob, s.B * s.Hv, s.T, per);
        pl.seg_len = cut.len;
        pl.whole = cut.whole;
        pl.units = s.B * s.Hv - cut.whole;
        const int64_t m = s.T <= pl.seg_len ? 1 : (s.T + pl.seg_len - 1) / pl.seg_len;
        pl.bounds = pl.units * (m - 1);
        pl.cut_blocks = m > 1 ? pl.units * m * nprob : 0;
        pl.blocks = (pl.whole + pl.units * m) * nprob;
    }
    pl.state_bytes = pl.bounds * kLinState * 4;
    return pl;
}

cudaError_t launch_linear(const LinArgs& a0, int nprob, const LinPlan& pl, bool bf16, void* ws,
                          int* launches, cudaStream_t st) {
    LinArgs a = a0;
    a.nprob = nprob;
    a.seg_len = pl.seg_len;
    a.whole = pl.whole;
    a.bounds = pl.bounds;
    a.status = status_ptr();
    uint8_t* at = (uint8_t*)ws;
    for (int i = nprob - 1; i >= 0; --i) {             // a sharing problem uses the one behind it
        if (a.pr[i].ws_t) {
            a.pr[i].ws = a.pr[i + 1].ws;
            continue;
        }
        a.pr[i].ws = (float*)at;
        at += pl.state_bytes;
    }
    cudaError_t e;
    if (pl.bounds > 0) {
        e = bf16 ? launch_linear_tc(a, nprob, pl, true, st)
                 : run_simt(a, pl.cut_blocks, true, st);
        if (e != cudaSuccess) return e;
        // blocks for four to an SM: of packed sequences many have nothing to do here
        int parts = 16;
        while (parts > 1 && pl.units * parts > 4LL * sm_count()) parts /= 2;
        k_lin_combine<<<dim3((unsigned)pl.units, parts, nprob), kCombineThreads, 0, st>>>(a);
        e = cudaGetLastError();
        if (e != cudaSuccess) return e;
        *launches += 2;
    }
    e = bf16 ? launch_linear_tc(a, nprob, pl, false, st)
             : run_simt(a, pl.blocks, false, st);
    if (e == cudaSuccess) ++*launches;
    return e;
}

cudaError_t launch_linear_group_sum(const LinArgs& a, const float* part, void* out, int group,
                                    bool bf16, cudaStream_t st) {
    const unsigned grid = (unsigned)((a.B * (a.Hv / group) * a.T * (kLinD / 4) + 255) / 256);
    if (bf16)
        k_lin_group_sum<<<grid, 256, 0, st>>>(a, part, (__nv_bfloat16*)out, group);
    else
        k_lin_group_sum<<<grid, 256, 0, st>>>(a, part, (float*)out, group);
    return cudaGetLastError();
}

}  // namespace gdn
