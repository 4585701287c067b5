// rotary.cu — rotary positions on queries and keys (gdn_rotary).
//
// Pair p of a head's first `rot` columns turns by the angle pos * f_p:
//   a' = m (a cos - b sin),   b' = m (a sin + b cos)
// with (a, b) = columns (p, p + rot/2) in the half layout and (2p, 2p + 1) in
// the interleaved one; the inverse turns by the negative angle, which is also
// the gradient (the matrix is m times orthogonal).  Columns from rot on are
// copied.
//
// The angle is reduced in binary64, pos * f_p and 1 / 2 pi as sums of two: one
// product of one each would lose 2^-53 of the turns, 2e-4 rad at position 10^12
// (a float32 product 0.06 rad at 10^6).  Only the fraction of a turn goes on to
// float32.
//
// GPU mapping.  Bound by moving the rows: 16 lanes hold one row of 128 columns
// (8 each), a CTA 16 tokens.  The angles of a token are the same for every
// head, so a lane forms its 8 (4 if interleaved) sines and cosines once and
// walks the heads with them, four rows in flight (64 registers, so that four
// CTAs share an SM: 1 GB of bf16 in 194 us, 202 at three); heads are split over CTAs
// only when the tokens alone do not fill the GPU (one token per request).
// The partner columns of the half layout come by shuffle from the lane that
// holds them when rot is a multiple of 16, else by loads of the elements.
#include "common.cuh"
#include "kernels.h"

namespace gdn {
namespace {

constexpr int kRotTokens = 16;                         // tokens per CTA
constexpr int kRotAhead = 4;                           // rows in flight per lane

enum RotMode { kInterleaved = 0, kHalf = 1, kHalfOdd = 2 };

template <typename T>
struct Row8;                                           // this lane's 8 columns, as loaded
template <>
struct Row8<__nv_bfloat16> {
    uint4 u;
    __device__ void load(const __nv_bfloat16* p) { u = *reinterpret_cast<const uint4*>(p); }
    __device__ void get(float (&x)[8]) const {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    __device__ void set(const float (&x)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        u = make_uint4(w[0], w[1], w[2], w[3]);
    }
    __device__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint4*>(p) = u; }
    __device__ Row8 from(int lane) const {
        Row8 r;
        r.u.x = __shfl_sync(0xffffffffu, u.x, lane, 16);
        r.u.y = __shfl_sync(0xffffffffu, u.y, lane, 16);
        r.u.z = __shfl_sync(0xffffffffu, u.z, lane, 16);
        r.u.w = __shfl_sync(0xffffffffu, u.w, lane, 16);
        return r;
    }
};
template <>
struct Row8<float> {
    float4 a, b;
    __device__ void load(const float* p) {
        a = *reinterpret_cast<const float4*>(p);
        b = *reinterpret_cast<const float4*>(p + 4);
    }
    __device__ void get(float (&x)[8]) const {
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
        x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    }
    __device__ void set(const float (&x)[8]) {
        a = make_float4(x[0], x[1], x[2], x[3]);
        b = make_float4(x[4], x[5], x[6], x[7]);
    }
    __device__ void store(float* p) const {
        *reinterpret_cast<float4*>(p) = a;
        *reinterpret_cast<float4*>(p + 4) = b;
    }
    __device__ Row8 from(int lane) const {
        float x[8];
        get(x);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = __shfl_sync(0xffffffffu, x[i], lane, 16);
        Row8 r;
        r.set(x);
        return r;
    }
};

// the fraction of a turn, within half of one, that pos * f radians leave
__device__ __forceinline__ float turn_fraction(double pos, double f) {
    constexpr double hi = 0.15915494309189535, lo = -9.839338337591243e-18;   // 1 / 2 pi
    const double a = pos * f, b = fma(pos, f, -a);
    const double t = a * hi, u = fma(a, hi, -t) + fma(a, lo, b * hi);
    return (float)((t - rint(t)) + u);
}

template <typename T, int MODE>
__global__ void __launch_bounds__(kRotTokens * 16, sizeof(T) == 2 && MODE != kHalfOdd ? 4 : 1)
k_rotary(const RotaryArgs p) {
    const int lane = threadIdx.x & 15;
    const int64_t n = (int64_t)blockIdx.x * kRotTokens + (threadIdx.x >> 4);
    const bool in = n < p.B * p.T;
    const int64_t b = in ? n / p.T : 0, t = in ? n % p.T : 0;
    const int c0 = 8 * lane, half = p.rot / 2;

    // x'_c = x_c cs[c] + x_partner(c) sn[c]; columns from rot on: cs = 1, no partner
    float cs[8], sn[8];
    const double pos = in ? (double)p.positions[n] : 0.0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (MODE == kInterleaved && (i & 1)) continue;
        const int c = c0 + i;
        float co = 1.f, si = 0.f;
        if (c < p.rot) {
            const int pr = MODE == kInterleaved ? c / 2 : (c < half ? c : c - half);
            sincospif(2.f * turn_fraction(pos, (double)p.inv_freq[pr]), &si, &co);
            co *= p.mscale;
            si *= p.inverse ? -p.mscale : p.mscale;
        }
        cs[i] = co;
        if (MODE == kInterleaved) {
            cs[i + 1] = co;
            sn[i] = -si;
            sn[i + 1] = si;
        } else {
            sn[i] = c < half ? -si : si;
        }
    }
    // half layout: the lane that holds this lane's partner columns
    const int from = MODE == kHalf ? (c0 < half ? lane + half / 8
                                                : (c0 < p.rot ? lane - half / 8 : lane))
                                   : 0;
    const int heads = (int)(p.Hq + p.Hk);
    const int h0 = blockIdx.y * p.heads_per_cta;
    const int h1 = min(heads, h0 + p.heads_per_cta);
    for (int hb = h0; hb < h1; hb += kRotAhead) {
        Row8<T> x[kRotAhead];
        const T* src[kRotAhead];
        T* dst[kRotAhead];
#pragma unroll
        for (int u = 0; u < kRotAhead; ++u) {
            const int h = min(hb + u, h1 - 1);         // the last rows again, not stored again
            const bool isq = h < p.Hq;
            const gdn_strides& xs = isq ? p.qs : p.ks;
            const gdn_strides& ys = isq ? p.qos : p.kos;
            const int64_t hh = isq ? h : h - p.Hq;
            src[u] = (const T*)(isq ? p.Q : p.K) + b * xs.b + hh * xs.h + t * xs.t;
            dst[u] = (T*)(isq ? p.Qo : p.Ko) + b * ys.b + hh * ys.h + t * ys.t + c0;
            if (in) x[u].load(src[u] + c0);
        }
        float o[MODE == kHalfOdd ? kRotAhead : 1][8];  // kHalfOdd: partners, read one by one
        if (MODE == kHalfOdd) {
#pragma unroll
            for (int u = 0; u < kRotAhead; ++u)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int c = c0 + i;
                    o[u][i] = in && c < p.rot ? ld_elem(src[u], c < half ? c + half : c - half)
                                              : 0.f;
                }
            __syncwarp();                              // in place: the row is read before it is written
        }
#pragma unroll
        for (int u = 0; u < kRotAhead; ++u) {
            float v[8], w[8];
            x[u].get(v);
            if (MODE == kInterleaved) {
#pragma unroll
                for (int i = 0; i < 8; ++i) w[i] = v[i ^ 1];
            } else if (MODE == kHalf) {
                x[u].from(from).get(w);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) w[i] = o[u][i];
            }
            float y[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                y[i] = c0 + i < p.rot ? fmaf(w[i], sn[i], v[i] * cs[i]) : v[i];
            x[u].set(y);
            if (in && hb + u < h1) x[u].store(dst[u]);
        }
    }
}

template <typename T>
void run_rotary(const RotaryArgs& a, dim3 grid, cudaStream_t st) {
    const int threads = kRotTokens * 16;
    if (a.interleaved) k_rotary<T, kInterleaved><<<grid, threads, 0, st>>>(a);
    else if (a.rot % 16 == 0) k_rotary<T, kHalf><<<grid, threads, 0, st>>>(a);
    else k_rotary<T, kHalfOdd><<<grid, threads, 0, st>>>(a);
}

}  // namespace

cudaError_t launch_rotary(RotaryArgs a, bool bf16, cudaStream_t st) {
    const int64_t blocks = (a.B * a.T + kRotTokens - 1) / kRotTokens;
    const int heads = (int)(a.Hq + a.Hk);
    // four CTAs per SM want work; a split costs each CTA its angles again
    int64_t split = (4LL * sm_count() + blocks - 1) / blocks;
    const int64_t most = (heads + kRotAhead - 1) / kRotAhead;
    split = split < 1 ? 1 : (split > most ? most : split);
    a.heads_per_cta = (int)((heads + split - 1) / split);
    const dim3 grid((unsigned)blocks,
                    (unsigned)((heads + a.heads_per_cta - 1) / a.heads_per_cta));
    if (bf16) run_rotary<__nv_bfloat16>(a, grid, st);
    else run_rotary<float>(a, grid, st);
    return cudaGetLastError();
}

}  // namespace gdn
