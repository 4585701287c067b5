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
// GPU mapping.  Bound by moving the rows.  A row lives in the registers of
// TPR threads, 8 channels per 16-byte (bf16) load and V such vectors per
// thread, so every input crosses once; CTAs are persistent, keep the weights
// in registers and load the next row while the current one is reduced.  A
// row's sums go by shuffle inside a warp and through shared memory across
// warps, in a fixed order.  Weight gradients stay in registers over all rows
// of a CTA; the CTAs' partial sums (float32) are added by a second kernel in
// CTA order, so results do not depend on scheduling.
#include "common.cuh"
#include "kernels.h"

namespace gdn {
namespace {

constexpr int kNormThreads = 256;                      // threads of a CTA with several rows
constexpr int kNormMaxRow = 512;                       // most threads on one row

// 8 consecutive channels
__device__ __forceinline__ void ld8(const __nv_bfloat16* p, float (&x)[8]) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void ld8(const float* p, float (&x)[8]) {
    const float4 a = *reinterpret_cast<const float4*>(p);
    const float4 b = *reinterpret_cast<const float4*>(p + 4);
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
__device__ __forceinline__ void st8(__nv_bfloat16* p, const float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void st8(float* p, const float (&x)[8]) {
    *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
}

// act(z) and its derivative.  Both tails of the logistic function come from
// e^-|z|, so 1 - s keeps its digits where s is near one.
__device__ __forceinline__ float gate_of(float z, int act, float& slope) {
    const float t = expf(-fabsf(z)), near1 = 1.f / (1.f + t), near0 = t * near1;
    const float s = z >= 0.f ? near1 : near0, s1 = z >= 0.f ? near0 : near1;
    if (act == GDN_ACT_SILU) {
        slope = s * fmaf(z, s1, 1.f);
        return z * s;
    }
    slope = s * s1;
    return s;
}

// Sum of N values over the threads of a row (TPR of them, a multiple of 32),
// the same for all of them.  `red` holds [rows of the CTA][TPR / 32][N] floats
// and is free again after the next call's first barrier: callers alternate two.
template <int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float* red, int tpr) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    const int warps = tpr >> 5;
    if (warps == 1) return;
    const int w = threadIdx.x >> 5;
    float* mine = red + threadIdx.y * warps * N;
    if ((threadIdx.x & 31) == 0)
#pragma unroll
        for (int i = 0; i < N; ++i) mine[w * N + i] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = 0.f;
    for (int k = 0; k < warps; ++k)
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += mine[k * N + i];
}
// the same over the 16 lanes that hold one head of 128 channels
__device__ __forceinline__ float head_sum(float x) {
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// One row's inputs for this thread: V vectors of 8 channels each.
template <typename T, int V>
struct RowIn {
    float y[V][8], z[V][8], r[V][8];
};

// offset of channel e of a row of y (rows are below 2^31)
__device__ __forceinline__ int64_t y_at(const NormArgs& p, const gdn_strides& s, int64_t row,
                                        int e) {
    const uint32_t T32 = (uint32_t)p.T, b = (uint32_t)row / T32, t = (uint32_t)row - b * T32;
    const int h = p.H == 1 ? 0 : e >> 7, c = p.H == 1 ? e : e & 127;
    return b * s.b + h * s.h + t * s.t + c;
}

// ---- the row up to x: yh, 1/rms(y) per vector, act, act', x ----
template <typename T, int V>
struct RowState {
    float y[V][8];        // yh (y itself without a post norm)
    float ry[V];          // 1 / rms of the vector's head
    float x[V][8];
    float g[V][8], dg[V][8];  // act(z), act'(z) (1, 0 without a gate)
};

template <typename T, int V, bool GRAD>
__device__ __forceinline__ void row_x(const NormArgs& p, const RowIn<T, V>& in,
                                      const float (&wo)[V][8], RowState<T, V>& s, float* red,
                                      int tpr, const bool (&has)[V]) {
#pragma unroll
    for (int k = 0; k < V; ++k) {
        s.ry[k] = 1.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) s.y[k][i] = in.y[k][i];
    }
    if (p.w_post) {
        if (p.H == 1) {
            float q[1] = {0.f};
#pragma unroll
            for (int k = 0; k < V; ++k)
#pragma unroll
                for (int i = 0; i < 8; ++i) q[0] = fmaf(s.y[k][i], s.y[k][i], q[0]);
            row_sums<1>(q, red, tpr);
            const float ri = 1.f / sqrtf(q[0] / (float)p.d + p.eps);
#pragma unroll
            for (int k = 0; k < V; ++k) s.ry[k] = ri;
        } else {
#pragma unroll
            for (int k = 0; k < V; ++k) {
                float q = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) q = fmaf(s.y[k][i], s.y[k][i], q);
                s.ry[k] = 1.f / sqrtf(head_sum(q) * (1.f / 128.f) + p.eps);
            }
        }
    }
#pragma unroll
    for (int k = 0; k < V; ++k) {
        if (!has[k]) s.ry[k] = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            s.y[k][i] *= s.ry[k];
            float n = s.y[k][i] * wo[k][i], sl = 0.f, g = 1.f;
            if (p.Z) g = gate_of(in.z[k][i], p.act, sl);
            if (GRAD) { s.g[k][i] = g; s.dg[k][i] = sl; }
            s.x[k][i] = fmaf(p.scale, n * g, in.r[k][i]);
            if (!has[k]) s.x[k][i] = 0.f;
        }
    }
}

template <typename T, int V>
__global__ void __launch_bounds__(kNormMaxRow)
k_block_norm(const NormArgs p) {
    extern __shared__ float red[];
    const int tpr = blockDim.x, W = (int)(p.H * p.d);
    const int64_t rows = p.B * p.T, step = (int64_t)gridDim.x * blockDim.y;
    int at[V];
    bool has[V];
    float wo[V][8], wi[V][8];
#pragma unroll
    for (int k = 0; k < V; ++k) {
        at[k] = 8 * (threadIdx.x + k * tpr);
        has[k] = at[k] < W;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            wo[k][i] = has[k] && p.w_post ? p.w_post[at[k] + i] : 1.f;
            wi[k][i] = has[k] && p.w_pre ? p.w_pre[at[k] + i] : 0.f;
        }
    }
    const int span = blockDim.y * (tpr >> 5);          // floats of one reduction buffer
    auto load = [&](int64_t row, RowIn<T, V>& in) {
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const bool ok = has[k] && row < rows;
            const int64_t e = row * W + at[k];
#pragma unroll
            for (int i = 0; i < 8; ++i) in.y[k][i] = in.z[k][i] = in.r[k][i] = 0.f;
            if (!ok) continue;
            ld8((const T*)p.Y + y_at(p, p.ys, row, at[k]), in.y[k]);
            if (p.Z) ld8((const T*)p.Z + e, in.z[k]);
            if (p.R) ld8((const T*)p.R + e, in.r[k]);
        }
    };
    for (int64_t base = (int64_t)blockIdx.x * blockDim.y; base < rows; base += step) {
        const int64_t row = base + threadIdx.y;        // every thread takes every barrier
        RowIn<T, V> in;
        load(row, in);
        RowState<T, V> s;
        row_x<T, V, false>(p, in, wo, s, red, tpr, has);
        float q[1] = {0.f};
        if (p.w_pre) {
#pragma unroll
            for (int k = 0; k < V; ++k)
#pragma unroll
                for (int i = 0; i < 8; ++i) q[0] = fmaf(s.x[k][i], s.x[k][i], q[0]);
            row_sums<1>(q, red + span, tpr);
        }
        const float ri = 1.f / sqrtf(q[0] / (float)W + p.eps);
#pragma unroll
        for (int k = 0; k < V; ++k) {
            if (!has[k] || row >= rows) continue;
            const int64_t e = row * W + at[k];
            if (p.X) st8((T*)p.X + e, s.x[k]);
            if (p.w_pre) {
#pragma unroll
                for (int i = 0; i < 8; ++i) s.x[k][i] = s.x[k][i] * ri * wi[k][i];
                st8((T*)p.N + e, s.x[k]);
            }
        }
        // red's two buffers are written in turn; with only one of the two
        // sums present the next row's would overtake its readers
        if (tpr > 32 && !(p.w_pre && p.w_post && p.H == 1)) __syncthreads();
    }
}

template <typename T, int V>
__global__ void __launch_bounds__(kNormMaxRow)
k_block_norm_backward(const NormArgs p) {
    extern __shared__ float red[];
    const int tpr = blockDim.x, W = (int)(p.H * p.d);
    const int64_t rows = p.B * p.T, step = (int64_t)gridDim.x * blockDim.y;
    int at[V];
    bool has[V];
    float wo[V][8], wi[V][8], dwo[V][8], dwi[V][8];
#pragma unroll
    for (int k = 0; k < V; ++k) {
        at[k] = 8 * (threadIdx.x + k * tpr);
        has[k] = at[k] < W;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            wo[k][i] = has[k] && p.w_post ? p.w_post[at[k] + i] : 1.f;
            wi[k][i] = has[k] && p.w_pre ? p.w_pre[at[k] + i] : 0.f;
            dwo[k][i] = dwi[k][i] = 0.f;
        }
    }
    const int span = blockDim.y * (tpr >> 5) * 2;
    for (int64_t base = (int64_t)blockIdx.x * blockDim.y; base < rows; base += step) {
        const int64_t row = base + threadIdx.y;
        RowIn<T, V> in;
        float dx[V][8], dn[V][8];
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const bool ok = has[k] && row < rows;
            const int64_t e = row * W + at[k];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                in.y[k][i] = in.z[k][i] = in.r[k][i] = dx[k][i] = dn[k][i] = 0.f;
            if (!ok) continue;
            ld8((const T*)p.Y + y_at(p, p.ys, row, at[k]), in.y[k]);
            if (p.Z) ld8((const T*)p.Z + e, in.z[k]);
            if (p.R) ld8((const T*)p.R + e, in.r[k]);
            if (p.dX) ld8((const T*)p.dX + e, dx[k]);
            if (p.dN) ld8((const T*)p.dN + e, dn[k]);
        }
        RowState<T, V> s;
        row_x<T, V, true>(p, in, wo, s, red, tpr, has);
        if (p.w_pre) {
            // sum x^2 and sum w_pre dN x together: mean(g xh) = ri sum(g x) / W
            float q[2] = {0.f, 0.f};
#pragma unroll
            for (int k = 0; k < V; ++k)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    q[0] = fmaf(s.x[k][i], s.x[k][i], q[0]);
                    q[1] = fmaf(wi[k][i] * dn[k][i], s.x[k][i], q[1]);
                }
            row_sums<2>(q, red + span, tpr);
            const float ri = 1.f / sqrtf(q[0] / (float)W + p.eps);
            const float m = ri * q[1] / (float)W;
#pragma unroll
            for (int k = 0; k < V; ++k)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float xh = s.x[k][i] * ri;
                    dwi[k][i] = fmaf(dn[k][i], xh, dwi[k][i]);
                    dx[k][i] = fmaf(ri, fmaf(-xh, m, wi[k][i] * dn[k][i]), dx[k][i]);
                }
        }
        float e1[1] = {0.f}, eh[V];
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int64_t e = row * W + at[k];
            const bool ok = has[k] && row < rows;
            if (p.dR && ok) st8((T*)p.dR + e, dx[k]);
            eh[k] = 0.f;
            float dz[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float du = p.scale * dx[k][i];
                dz[i] = du * (s.y[k][i] * wo[k][i]) * s.dg[k][i];
                const float d1 = du * s.g[k][i];       // dn
                dwo[k][i] = fmaf(d1, s.y[k][i], dwo[k][i]);
                dx[k][i] = d1 * wo[k][i];              // e
                eh[k] = fmaf(dx[k][i], s.y[k][i], eh[k]);
            }
            if (p.dZ && ok) st8((T*)p.dZ + e, dz);
            e1[0] += eh[k];
        }
        if (p.w_post) {
            float m = 0.f;
            if (p.H == 1) {
                row_sums<1>(e1, red + 2 * span, tpr);
                m = e1[0] / (float)p.d;
            }
#pragma unroll
            for (int k = 0; k < V; ++k) {
                const float mk = p.H == 1 ? m : head_sum(eh[k]) * (1.f / 128.f);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    dx[k][i] = s.ry[k] * fmaf(-s.y[k][i], mk, dx[k][i]);
            }
        }
#pragma unroll
        for (int k = 0; k < V; ++k)
            if (has[k] && row < rows)
                st8((T*)p.dY + y_at(p, p.dys, row, at[k]), dx[k]);
        // a sum's buffer is next written after at least one barrier of
        // another sum when two or three are present; with one, add one
        if (tpr > 32 && !(p.w_post && p.H == 1)) __syncthreads();
    }
    // partial sums of this CTA's row group: [group][2][W]
    const int64_t group = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
#pragma unroll
    for (int k = 0; k < V; ++k)
        if (has[k]) {
            if (p.dw_post) st8(p.ws + (group * 2) * W + at[k], dwo[k]);
            if (p.dw_pre) st8(p.ws + (group * 2 + 1) * W + at[k], dwi[k]);
        }
}

// dw[c] = sum over the groups in order, four strands; blockIdx.y: post, pre
__global__ void __launch_bounds__(256) k_norm_dw(const float* ws, float* dw_post, float* dw_pre,
                                                 int W, int groups) {
    __shared__ float part[8][32];
    float* out = blockIdx.y ? dw_pre : dw_post;
    if (!out) return;
    const int c = blockIdx.x * 32 + (threadIdx.x & 31), w = threadIdx.x >> 5;
    float a = 0.f;
    if (c < W)
        for (int g = w; g < groups; g += 8) a += ws[((int64_t)g * 2 + blockIdx.y) * W + c];
    part[w][threadIdx.x & 31] = a;
    __syncthreads();
    if (w == 0 && c < W) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) s += part[i][threadIdx.x];
        out[c] = s;
    }
}

// threads per row, vectors per thread and rows per CTA for a width
struct NormShape {
    int tpr, v, rpc;
};
NormShape norm_shape(int64_t W) {
    const int vecs = (int)(W / 8);
    NormShape s;
    s.v = vecs <= kNormMaxRow ? 1 : (vecs <= 2 * kNormMaxRow ? 2 : 4);
    s.tpr = ((vecs + s.v - 1) / s.v + 31) / 32 * 32;
    s.rpc = s.tpr >= kNormThreads ? 1 : kNormThreads / s.tpr;
    return s;
}

constexpr int kNormCtas = 4;                           // CTAs per SM of the backward pass

int backward_ctas(int64_t rows, const NormShape& s) {
    const int64_t need = (rows + s.rpc - 1) / s.rpc, most = (int64_t)kNormCtas * sm_count();
    return (int)(need < most ? need : most);
}

template <typename T, int V>
void run_norm(const NormArgs& a, const NormShape& s, cudaStream_t st) {
    const int64_t need = (a.B * a.T + s.rpc - 1) / s.rpc, most = 8LL * sm_count();
    const int smem = 2 * s.rpc * (s.tpr / 32) * (int)sizeof(float);
    k_block_norm<T, V><<<(unsigned)(need < most ? need : most), dim3(s.tpr, s.rpc), smem, st>>>(a);
}
template <typename T, int V>
void run_norm_backward(const NormArgs& a, const NormShape& s, cudaStream_t st) {
    const int smem = 3 * 2 * s.rpc * (s.tpr / 32) * (int)sizeof(float);
    k_block_norm_backward<T, V>
        <<<(unsigned)backward_ctas(a.B * a.T, s), dim3(s.tpr, s.rpc), smem, st>>>(a);
}

}  // namespace

int64_t block_norm_ws_bytes(int64_t rows, int64_t width) {
    const NormShape s = norm_shape(width);
    return (int64_t)backward_ctas(rows, s) * s.rpc * 2 * width * 4;
}

cudaError_t launch_block_norm(const NormArgs& a, bool bf16, cudaStream_t st) {
    const NormShape s = norm_shape(a.H * a.d);
    if (bf16) {
        if (s.v == 1) run_norm<__nv_bfloat16, 1>(a, s, st);
        else if (s.v == 2) run_norm<__nv_bfloat16, 2>(a, s, st);
        else run_norm<__nv_bfloat16, 4>(a, s, st);
    } else {
        if (s.v == 1) run_norm<float, 1>(a, s, st);
        else if (s.v == 2) run_norm<float, 2>(a, s, st);
        else run_norm<float, 4>(a, s, st);
    }
    return cudaGetLastError();
}

cudaError_t launch_block_norm_backward(const NormArgs& a, bool bf16, cudaStream_t st) {
    const NormShape s = norm_shape(a.H * a.d);
    if (bf16) {
        if (s.v == 1) run_norm_backward<__nv_bfloat16, 1>(a, s, st);
        else if (s.v == 2) run_norm_backward<__nv_bfloat16, 2>(a, s, st);
        else run_norm_backward<__nv_bfloat16, 4>(a, s, st);
    } else {
        if (s.v == 1) run_norm_backward<float, 1>(a, s, st);
        else if (s.v == 2) run_norm_backward<float, 2>(a, s, st);
        else run_norm_backward<float, 4>(a, s, st);
    }
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !(a.dw_post || a.dw_pre)) return e;
    const int W = (int)(a.H * a.d);
    k_norm_dw<<<dim3((W + 31) / 32, 2), 256, 0, st>>>(
        a.ws, a.dw_post, a.dw_pre, W, backward_ctas(a.B * a.T, s) * s.rpc);
    return cudaGetLastError();
}

}  // namespace gdn
