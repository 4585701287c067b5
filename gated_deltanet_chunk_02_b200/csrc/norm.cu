// norm.cu — the norms before and after a block with its gate and residual
// scale (gdn_block_norm) and their gradients (gdn_block_norm_backward).
//
// For a row of W = H d channels, y the block's output, r the residual stream:
//   yh = y / rms_d(y),  n = w_post yh          (rms over each head's d channels)
//   u  = act(z) n,      x = r + s u            (the new residual stream)
//   xh = x / rms_W(x),  N = w_pre xh           (the next block's input)
// with rms(v) = sqrt(mean(v^2) + eps); every part but y may be absent.
// Backward, for dX and dN:
//   dx = dX + (1/rms_W(x)) (g - xh mean(g xh)),  g = w_pre dN;   dR = dx
//   dz = s dx n act'(z);  dn = s dx act(z);  dw_pre += dN xh;  dw_post += dn yh
//   dy = (1/rms_d(y)) (e - yh mean_d(e yh)),  e = w_post dn
// The row is recomputed from y, z, r in float32, so nothing is saved in the
// forward pass and dx does not see X's rounding.
//
// GPU mapping.  Bound by moving the rows and, close behind, by instructions.  A
// row lives in the registers of `tpr` threads as V 16-byte vectors per thread
// and input, all loaded before anything is reduced.  V is 2 where rows are many
// (16384 x 2048 bf16, forward: 61 us, V = 4 69, V = 8 88; backward: 156 us, 204
// at V = 4 and 197 at V = 1), 1 where they are too few to fill the GPU, and more
// only where a row would take over 512 threads.  Weights are read again for
// each row (from L1).  A row's sums go by shuffle inside a warp and through
// shared memory across warps, in a fixed order.  Backward, CTAs stay, fetch a
// row ahead into shared memory and keep the weight gradients of their rows in
// registers; the CTAs' sums (float32) are added by a second kernel in CTA
// order, so results do not depend on scheduling.
//
// One B200, 16384 rows of 2048 bf16 channels with everything present: forward
// 61 us (336 MB in and out, 5.5 TB/s; instruction issue 74 %), backward 156 us
// (537 MB, 3.4 TB/s; issue 58 %, one row's chain of sums the rest).
#include "common.cuh"
#include "kernels.h"

namespace gdn {
namespace {

template <typename T>
constexpr int kE = 16 / (int)sizeof(T);                // channels of a vector

// Channels are handled in pairs (F2): one at a time the instructions, not the
// bytes, were the bound (forward 110 us, backward 243 us at 16384 x 2048 bf16).
__device__ __forceinline__ void unpack(const uint4& u, F2 (&x)[4]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        x[i] = F2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
}
__device__ __forceinline__ void unpack(const uint4& u, F2 (&x)[2]) {
    x[0] = F2(__uint_as_float(u.x), __uint_as_float(u.y));
    x[1] = F2(__uint_as_float(u.z), __uint_as_float(u.w));
}
__device__ __forceinline__ uint4 pack(const F2 (&x)[4]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float a, b;
        x[i].get(a, b);
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ uint4 pack(const F2 (&x)[2]) {
    float a, b, c, d;
    x[0].get(a, b);
    x[1].get(c, d);
    return make_uint4(__float_as_uint(a), __float_as_uint(b), __float_as_uint(c),
                      __float_as_uint(d));
}
__device__ __forceinline__ F2 both(float x) { return F2(x, x); }
__device__ __forceinline__ float sum2(F2 x) {
    float a, b;
    x.get(a, b);
    return a + b;
}
// weights of the channels from `at` on (ones without any)
template <int P>
__device__ __forceinline__ void weights(const float* w, int at, F2 (&x)[P]) {
    if (w) {
#pragma unroll
        for (int i = 0; i < P; i += 2) {
            const float4 f = __ldg(reinterpret_cast<const float4*>(w + at + 2 * i));
            x[i] = F2(f.x, f.y);
            x[i + 1] = F2(f.z, f.w);
        }
    } else {
#pragma unroll
        for (int i = 0; i < P; ++i) x[i] = both(1.f);
    }
}

// t = e^-z and s = 1 / (1 + t), two at a time, by the base-2 exponential (the
// product -z log2(e) costs |z| 2^-24).  z stops at -87, where t is still finite:
// 1 - s = t s then keeps its digits where s is near one.  The caller's z stops
// there too: z s is then at most 1.5e-36 however low the gate, where the type's
// lowest value times the s of -87 would be -5.6.  A NaN stays one.
__device__ __forceinline__ void logistic2(F2& z, F2& t, F2& s) {
    float x, y;
    z.get(x, y);
    asm("max.NaN.f32 %0, %0, 0fC2AE0000;" : "+f"(x));  // -87
    asm("max.NaN.f32 %0, %0, 0fC2AE0000;" : "+f"(y));
    z = F2(x, y);
    mul2(z, both(-1.442695041f)).get(x, y);
    asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(x));
    asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(y));
    t = F2(x, y);
    add2(t, both(1.f)).get(x, y);
    asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(x));
    asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(y));
    s = F2(x, y);
}
// x *= act(z), a vector's channels (z is used up)
template <int P>
__device__ __forceinline__ void apply_gate(F2 (&z)[P], int act, F2 (&x)[P]) {
    F2 t, s;
    if (act == GDN_ACT_SILU) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
            logistic2(z[i], t, s);
            x[i] = mul2(x[i], mul2(z[i], s));
        }
    } else {
#pragma unroll
        for (int i = 0; i < P; ++i) {
            logistic2(z[i], t, s);
            x[i] = mul2(x[i], s);
        }
    }
}
// du, n -> dn = du act(z) (in du) and dz = du n act'(z) (in z)
template <int P>
__device__ __forceinline__ void gate_gradient(F2 (&z)[P], int act, const F2 (&n)[P], F2 (&du)[P]) {
    F2 t, s;
    if (act == GDN_ACT_SILU) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
            logistic2(z[i], t, s);
            const F2 a = mul2(du[i], s);               // act' = s (1 + z (1 - s))
            du[i] = mul2(a, z[i]);
            z[i] = mul2(mul2(a, n[i]), fma2(z[i], mul2(t, s), both(1.f)));
        }
    } else {
#pragma unroll
        for (int i = 0; i < P; ++i) {
            logistic2(z[i], t, s);
            du[i] = mul2(du[i], s);                    // act' = s (1 - s)
            z[i] = mul2(mul2(du[i], n[i]), mul2(t, s));
        }
    }
}

// Sum of N values over the threads of a row (tpr of them, a multiple of 32),
// the same for all of them; `red` is used once per barrier-free stretch.
template <int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float* red, int tpr) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    const int warps = tpr >> 5;
    if (warps == 1) return;
    float* mine = red + threadIdx.y * warps * N;
    if ((threadIdx.x & 31) == 0)
#pragma unroll
        for (int i = 0; i < N; ++i) mine[(threadIdx.x >> 5) * N + i] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = 0.f;
    for (int k = 0; k < warps; ++k)
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += mine[k * N + i];
}
// the same over the lanes that hold one head of 128 channels (16 of bf16, 32)
template <int E>
__device__ __forceinline__ float head_sum(float x) {
#pragma unroll
    for (int o = 64 / E; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// offset of a row of y (rows are below 2^31), and of its channel e in the row
__device__ __forceinline__ int64_t y_row(const NormArgs& p, const gdn_strides& s, int64_t row) {
    const uint32_t T32 = (uint32_t)p.T, b = (uint32_t)row / T32, t = (uint32_t)row - b * T32;
    return b * s.b + t * s.t;
}
__device__ __forceinline__ int64_t y_in(const NormArgs& p, const gdn_strides& s, int e) {
    return p.H == 1 ? e : (e >> 7) * s.h + (e & 127);
}

// 1 / rms_d of y, by vector (H > 1) or for the row; 1 without a post norm
template <int V, int E>
__device__ __forceinline__ void post_scale(const NormArgs& p, const uint4 (&y)[V], float (&ry)[V],
                                           float* red, int tpr) {
#pragma unroll
    for (int k = 0; k < V; ++k) ry[k] = 1.f;
    if (!p.w_post) return;
    float q[V], all[1] = {0.f};
#pragma unroll
    for (int k = 0; k < V; ++k) {
        F2 v[E / 2], a = both(0.f);
        unpack(y[k], v);
#pragma unroll
        for (int i = 0; i < E / 2; ++i) a = fma2(v[i], v[i], a);
        q[k] = sum2(a);
        all[0] += q[k];
    }
    if (p.H == 1) {
        row_sums<1>(all, red, tpr);
        const float r = 1.f / sqrtf(all[0] / (float)p.d + p.eps);
#pragma unroll
        for (int k = 0; k < V; ++k) ry[k] = r;
    } else {
#pragma unroll
        for (int k = 0; k < V; ++k) ry[k] = 1.f / sqrtf(head_sum<E>(q[k]) * (1.f / 128.f) + p.eps);
    }
}

template <typename T, int V, int MAXT>
__global__ void __launch_bounds__(MAXT) k_block_norm(const NormArgs p) {
    constexpr int E = kE<T>;
    extern __shared__ float red[];
    const int tpr = blockDim.x, W = (int)(p.H * p.d);
    const int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y, rows = p.B * p.T;
    uint4 y[V], z[V], r[V];
    bool ok[V];
    const T* const yr = (const T*)p.Y + y_row(p, p.ys, row);
#pragma unroll
    for (int k = 0; k < V; ++k) {
        const int at = E * (threadIdx.x + k * tpr);
        ok[k] = at < W && row < rows;
        y[k] = z[k] = r[k] = make_uint4(0, 0, 0, 0);
        if (!ok[k]) continue;
        y[k] = *reinterpret_cast<const uint4*>(yr + y_in(p, p.ys, at));
        if (p.Z) z[k] = *reinterpret_cast<const uint4*>((const T*)p.Z + row * W + at);
        if (p.R) r[k] = *reinterpret_cast<const uint4*>((const T*)p.R + row * W + at);
    }
    float ry[V];
    post_scale<V, E>(p, y, ry, red, tpr);
    constexpr int P = E / 2;                           // pairs of a vector
    F2 x[V][P], xx = both(0.f);
#pragma unroll
    for (int k = 0; k < V; ++k) {
        const int at = E * (threadIdx.x + k * tpr);
        F2 w[P], yv[P], zv[P];
        weights(p.w_post, min(at, W - E), w);
        unpack(y[k], yv);
        unpack(r[k], x[k]);
        const F2 a = both(p.scale * ry[k]);
#pragma unroll
        for (int i = 0; i < P; ++i) yv[i] = mul2(mul2(yv[i], a), w[i]);
        if (p.Z) {
            unpack(z[k], zv);
            apply_gate(zv, p.act, yv);
        }
#pragma unroll
        for (int i = 0; i < P; ++i) {
            x[k][i] = add2(x[k][i], yv[i]);
            xx = fma2(x[k][i], x[k][i], xx);
        }
        if (p.X && ok[k])
            *reinterpret_cast<uint4*>((T*)p.X + row * W + at) = pack(x[k]);
    }
    if (!p.w_pre) return;
    float q[1] = {sum2(xx)};
    row_sums<1>(q, red + (tpr >> 5) * blockDim.y, tpr);
    const F2 ri = both(1.f / sqrtf(q[0] / (float)W + p.eps));
#pragma unroll
    for (int k = 0; k < V; ++k) {
        if (!ok[k]) continue;
        const int at = E * (threadIdx.x + k * tpr);
        F2 w[P];
        weights(p.w_pre, at, w);
#pragma unroll
        for (int i = 0; i < P; ++i) x[k][i] = mul2(mul2(x[k][i], ri), w[i]);
        *reinterpret_cast<uint4*>((T*)p.N + row * W + at) = pack(x[k]);
    }
}

template <typename T, int V, int MAXT, bool AHEAD>
__global__ void __launch_bounds__(MAXT) k_block_norm_backward(const NormArgs p) {
    constexpr int E = kE<T>;
    extern __shared__ __align__(16) float red[];
    const int tpr = blockDim.x, W = (int)(p.H * p.d), span = blockDim.y * (tpr >> 5) * 2;
    const int64_t rows = p.B * p.T, step = (int64_t)gridDim.x * blockDim.y;
    constexpr int P = E / 2;                           // pairs of a vector
    F2 dwo[V][P], dwi[V][P];
#pragma unroll
    for (int k = 0; k < V; ++k)
#pragma unroll
        for (int i = 0; i < P; ++i) dwo[k][i] = dwi[k][i] = both(0.f);
    // The next row's vectors come into shared memory (a thread's own places, so
    // no barrier) while a row is reduced; two sets in turn.
    uint4* const ahead =
        reinterpret_cast<uint4*>(red + ((3 * span + (blockDim.y - 1) * 2 * W + 3) & ~3));
    const int threads = tpr * blockDim.y, me = threadIdx.y * tpr + threadIdx.x;
    auto fetch = [&](int64_t row, int set) {
        const T* const yr = (const T*)p.Y + y_row(p, p.ys, row);
        const void* const src[5] = {p.Y, p.Z, p.R, p.dX, p.dN};
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int at = E * (threadIdx.x + k * tpr);
            const bool ok = at < W && row < rows;
#pragma unroll
            for (int j = 0; j < 5; ++j)
                if (src[j]) {
                    const T* g = (const T*)src[j];
                    if (ok) g = j == 0 ? yr + y_in(p, p.ys, at) : g + row * W + at;
                    const uint32_t to = (uint32_t)__cvta_generic_to_shared(
                        ahead + ((set * 5 + j) * V + k) * threads + me);
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(g),
                                 "r"(ok ? 16 : 0)
                                 : "memory");          // zeros where there is no channel
                }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    int set = 0;
    if (AHEAD) fetch((int64_t)blockIdx.x * blockDim.y + threadIdx.y, 0);
    for (int64_t base = (int64_t)blockIdx.x * blockDim.y; base < rows; base += step) {
        const int64_t row = base + threadIdx.y;        // every thread takes every barrier
        uint4 y[V], z[V], r[V], gx[V], gn[V];
        bool ok[V];
        if (AHEAD) {
            asm volatile("cp.async.wait_group 0;" ::: "memory");
            fetch(row + step, set ^ 1);
        }
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int at = E * (threadIdx.x + k * tpr);
            const int64_t e = row * W + at;
            ok[k] = at < W && row < rows;
            y[k] = z[k] = r[k] = gx[k] = gn[k] = make_uint4(0, 0, 0, 0);
            if (AHEAD) {
                const uint4* a = ahead + (set * 5 * V + k) * threads + me;
                y[k] = a[0];
                if (p.Z) z[k] = a[V * threads];
                if (p.R) r[k] = a[2 * V * threads];
                if (p.dX) gx[k] = a[3 * V * threads];
                if (p.dN) gn[k] = a[4 * V * threads];
            } else if (ok[k]) {
                y[k] = *reinterpret_cast<const uint4*>((const T*)p.Y + y_row(p, p.ys, row) +
                                                       y_in(p, p.ys, at));
                if (p.Z) z[k] = *reinterpret_cast<const uint4*>((const T*)p.Z + e);
                if (p.R) r[k] = *reinterpret_cast<const uint4*>((const T*)p.R + e);
                if (p.dX) gx[k] = *reinterpret_cast<const uint4*>((const T*)p.dX + e);
                if (p.dN) gn[k] = *reinterpret_cast<const uint4*>((const T*)p.dN + e);
            }
        }
        set ^= 1;
        float ry[V];
        post_scale<V, E>(p, y, ry, red, tpr);
        F2 x[V][P];                                    // x, then e
        float ri = 0.f, m = 0.f;
        // x, and its two sums: sum x^2, sum w_pre dN x (mean(g xh) = ri sum(g x) / W)
        F2 xx = both(0.f), gg = both(0.f);
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int at = min(E * (int)(threadIdx.x + k * tpr), W - E);
            F2 w[P], yv[P], zv[P], gv[P];
            weights(p.w_post, at, w);
            unpack(y[k], yv);
            unpack(r[k], x[k]);
            const F2 a = both(p.scale * ry[k]);
#pragma unroll
            for (int i = 0; i < P; ++i) yv[i] = mul2(mul2(yv[i], a), w[i]);
            if (p.Z) {
                unpack(z[k], zv);
                apply_gate(zv, p.act, yv);
            }
#pragma unroll
            for (int i = 0; i < P; ++i) x[k][i] = add2(x[k][i], yv[i]);
            if (p.w_pre) {
                weights(p.w_pre, at, w);
                unpack(gn[k], gv);
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    xx = fma2(x[k][i], x[k][i], xx);
                    gg = fma2(mul2(w[i], gv[i]), x[k][i], gg);
                }
            }
        }
        if (p.w_pre) {
            float q[2] = {sum2(xx), sum2(gg)};
            row_sums<2>(q, red + span, tpr);
            ri = 1.f / sqrtf(q[0] / (float)W + p.eps);
            m = ri * q[1] / (float)W;
        }
        float all[1] = {0.f}, eh[V];
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int at = E * (threadIdx.x + k * tpr), aw = min(at, W - E);
            const int64_t e = row * W + at;
            F2 w[P], yv[P], dx[P], gv[P];
            unpack(gx[k], dx);
            if (p.w_pre) {
                weights(p.w_pre, aw, w);
                unpack(gn[k], gv);
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    const F2 xh = mul2(x[k][i], both(ri));
                    dwi[k][i] = fma2(gv[i], xh, dwi[k][i]);
                    dx[i] = fma2(both(ri), fma2(xh, both(-m), mul2(w[i], gv[i])), dx[i]);
                }
            }
            if (p.dR && ok[k]) *reinterpret_cast<uint4*>((T*)p.dR + e) = pack(dx);
            weights(p.w_post, aw, w);
            unpack(y[k], yv);
#pragma unroll
            for (int i = 0; i < P; ++i) {
                yv[i] = mul2(yv[i], both(ry[k]));      // yh
                dx[i] = mul2(dx[i], both(p.scale));    // du
            }
            if (p.Z) {
                F2 zv[P], n[P];
                unpack(z[k], zv);
#pragma unroll
                for (int i = 0; i < P; ++i) n[i] = mul2(yv[i], w[i]);
                gate_gradient(zv, p.act, n, dx);       // dn
                if (ok[k]) *reinterpret_cast<uint4*>((T*)p.dZ + e) = pack(zv);
            }
            F2 s = both(0.f);
#pragma unroll
            for (int i = 0; i < P; ++i) {
                dwo[k][i] = fma2(dx[i], yv[i], dwo[k][i]);
                x[k][i] = mul2(dx[i], w[i]);
                s = fma2(x[k][i], yv[i], s);
            }
            eh[k] = sum2(s);
            all[0] += eh[k];
        }
        if (p.w_post && p.H == 1) row_sums<1>(all, red + 2 * span, tpr);
        T* const dyr = (T*)p.dY + y_row(p, p.dys, row);
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int at = E * (threadIdx.x + k * tpr);
            if (p.w_post) {
                F2 yv[P];
                unpack(y[k], yv);
                const float mk = p.H == 1 ? all[0] / (float)p.d : head_sum<E>(eh[k]) * (1.f / 128.f);
                const F2 a = both(ry[k]), b = both(-ry[k] * mk);
#pragma unroll
                for (int i = 0; i < P; ++i) x[k][i] = mul2(a, fma2(yv[i], b, x[k][i]));
            }
            if (ok[k]) *reinterpret_cast<uint4*>(dyr + y_in(p, p.dys, at)) = pack(x[k]);
        }
        // a sum's buffer is next written behind another sum's barrier when two
        // or three are present, else behind this one
        if (tpr > 32 && !(p.w_post && p.H == 1)) __syncthreads();
    }
    // the CTA's sums: its row groups in order, then to ws [CTA][2][W]
    F2* part = reinterpret_cast<F2*>(red + 3 * span);  // [blockDim.y - 1][2][W / 2]
    const int W2 = W / 2;
    if (blockDim.y > 1) {
        __syncthreads();
        if (threadIdx.y > 0)
#pragma unroll
            for (int k = 0; k < V; ++k) {
                const int at = P * (threadIdx.x + k * tpr);
                if (at < W2)
#pragma unroll
                    for (int i = 0; i < P; ++i) {
                        part[(threadIdx.y - 1) * 2 * W2 + at + i] = dwo[k][i];
                        part[((threadIdx.y - 1) * 2 + 1) * W2 + at + i] = dwi[k][i];
                    }
            }
        __syncthreads();
        if (threadIdx.y > 0) return;
    }
    F2* const to = reinterpret_cast<F2*>(p.ws) + (int64_t)blockIdx.x * 2 * W2;
#pragma unroll
    for (int k = 0; k < V; ++k) {
        const int at = P * (threadIdx.x + k * tpr);
        if (at >= W2) continue;
        for (int g = 0; g + 1 < blockDim.y; ++g)
#pragma unroll
            for (int i = 0; i < P; ++i) {
                dwo[k][i] = add2(dwo[k][i], part[g * 2 * W2 + at + i]);
                dwi[k][i] = add2(dwi[k][i], part[(g * 2 + 1) * W2 + at + i]);
            }
#pragma unroll
        for (int i = 0; i < P; ++i) {
            if (p.dw_post) to[at + i] = dwo[k][i];
            if (p.dw_pre) to[W2 + at + i] = dwi[k][i];
        }
    }
}

// dw[c] = sum over the CTAs, 32 strands each in order; blockIdx.y: post, pre
__global__ void __launch_bounds__(1024) k_norm_dw(const float* ws, float* dw_post, float* dw_pre,
                                                  int W, int ctas) {
    __shared__ float part[32][33];
    float* out = blockIdx.y ? dw_pre : dw_post;
    if (!out) return;
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    float a = 0.f;
    if (c < W)
#pragma unroll 8
        for (int g = w; g < ctas; g += 32) a += ws[((int64_t)g * 2 + blockIdx.y) * W + c];
    part[w][lane] = a;
    __syncthreads();
    if (w == 0 && c < W) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < 32; ++i) s += part[i][lane];
        out[c] = s;
    }
}

// vectors per thread, threads per row, rows per CTA
struct NormShape {
    int v, tpr, rpc;
};
// As many vectors a thread, `most` at the top, as leave 16 warps for every SM
// and the row a warp of its own; more where a row would take over 512 threads.
NormShape norm_shape(int64_t rows, int64_t W, int e, int most, int wide) {
    const int vecs = (int)(W / e);
    NormShape s;
    auto warps = [&](int v) { return (vecs + 32 * v - 1) / (32 * v); };
    s.v = 1;
    while ((warps(s.v) > 16 && s.v < wide) ||
           (s.v < most && vecs >= 64 * s.v && rows * warps(2 * s.v) >= 16LL * sm_count()))
        s.v *= 2;
    s.tpr = 32 * warps(s.v);
    s.rpc = s.tpr >= 128 ? 1 : 128 / s.tpr;
    return s;
}
constexpr int kForwardV = 2, kBackwardV = 2;           // where rows are many
constexpr int kForwardWide = 8, kBackwardWide = 4;     // where rows are wide

// CTAs of the backward pass, whatever the data type (the workspace's size goes by it)
int backward_ctas(int64_t rows) {
    const int64_t most = 4LL * sm_count();
    return (int)(rows < most ? rows : most);
}

template <typename T, int V, int MAXT>
void run_norm(const NormArgs& a, const NormShape& s, cudaStream_t st) {
    const int64_t ctas = (a.B * a.T + s.rpc - 1) / s.rpc;
    const int smem = 2 * s.rpc * (s.tpr / 32) * (int)sizeof(float);
    k_block_norm<T, V, MAXT><<<(unsigned)ctas, dim3(s.tpr, s.rpc), smem, st>>>(a);
}
template <typename T, int V, int MAXT>
cudaError_t run_norm_backward(const NormArgs& a, const NormShape& s, cudaStream_t st) {
    const int W = (int)(a.H * a.d), threads = s.tpr * s.rpc;
    int smem = (3 * 2 * s.rpc * (s.tpr / 32) + (s.rpc - 1) * 2 * W) * (int)sizeof(float);
    // rows ahead where three CTAs still share an SM's 227 KB (16384 x 2048 bf16:
    // 40 KB each); with wider rows those in registers are enough to load
    const int ahead = ((smem + 15) & ~15) + 2 * 5 * V * threads * 16;
    const dim3 grid((unsigned)backward_ctas(a.B * a.T)), block(s.tpr, s.rpc);
    if (ahead > 75 * 1024) {
        k_block_norm_backward<T, V, MAXT, false><<<grid, block, smem, st>>>(a);
        return cudaGetLastError();
    }
    cudaError_t e = cudaFuncSetAttribute(k_block_norm_backward<T, V, MAXT, true>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, 75 * 1024);
    if (e != cudaSuccess) return e;
    k_block_norm_backward<T, V, MAXT, true><<<grid, block, ahead, st>>>(a);
    return cudaGetLastError();
}
template <typename T>
void norm_forward(const NormArgs& a, cudaStream_t st) {
    const NormShape s = norm_shape(a.B * a.T, a.H * a.d, kE<T>, kForwardV, kForwardWide);
    if (s.v == 1) run_norm<T, 1, 512>(a, s, st);
    else if (s.v == 2) run_norm<T, 2, 512>(a, s, st);
    else if (s.v == 4) run_norm<T, 4, 512>(a, s, st);
    else run_norm<T, 8, 512>(a, s, st);
}
template <typename T>
cudaError_t norm_backward(const NormArgs& a, cudaStream_t st) {
    const NormShape s = norm_shape(a.B * a.T, a.H * a.d, kE<T>, kBackwardV, kBackwardWide);
    if (s.v == 1) return run_norm_backward<T, 1, 512>(a, s, st);
    if (s.v == 2) return run_norm_backward<T, 2, 512>(a, s, st);
    if (s.tpr <= 256) return run_norm_backward<T, 4, 256>(a, s, st);
    return run_norm_backward<T, 4, 1024>(a, s, st);
}

}  // namespace

int64_t block_norm_ws_bytes(int64_t rows, int64_t width) {
    return (int64_t)backward_ctas(rows) * 2 * width * 4;
}

cudaError_t launch_block_norm(const NormArgs& a, bool bf16, cudaStream_t st) {
    if (bf16) norm_forward<__nv_bfloat16>(a, st);
    else norm_forward<float>(a, st);
    return cudaGetLastError();
}

cudaError_t launch_block_norm_backward(const NormArgs& a, bool bf16, cudaStream_t st) {
    cudaError_t e = bf16 ? norm_backward<__nv_bfloat16>(a, st) : norm_backward<float>(a, st);
    if (e != cudaSuccess || !(a.dw_post || a.dw_pre)) return e;
    const int W = (int)(a.H * a.d);
    k_norm_dw<<<dim3((W + 31) / 32, 2), 1024, 0, st>>>(a.ws, a.dw_post, a.dw_pre, W,
                                                       backward_ctas(a.B * a.T));
    return cudaGetLastError();
}

}  // namespace gdn
