// kernels.h — internal launchers of libgdn (host side, not part of the C ABI).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/gdn.h"

namespace gdn {

int* status_ptr();     // device address of the status word (api.cu)
int sm_count();        // SMs of the current device (api.cu)

// CUDA-core kernels (simt.cu); k in {32, 64, 128} unless stated.
cudaError_t launch_build_A_simt(const void* K, const float* beta, const float* g, float* A,
                                int64_t nc, int k, bool bf16, cudaStream_t st);  // k <= 256
cudaError_t launch_neumann_simt(const float* A, float* T, int64_t nc, int k, int N, int mask,
                                int S, cudaStream_t st);
cudaError_t launch_wy_simt(const float* T, const void* K, const void* V, const float* beta,
                           const float* g, void* W, void* U, int64_t nc, int k, bool bf16,
                           cudaStream_t st);
cudaError_t launch_fused_simt(const void* K, const void* V, const float* beta, const float* g,
                              int N, int mask, int S, int gated, void* W, void* U, float* Tout,
                              int64_t nc, int k, bool bf16, cudaStream_t st);
cudaError_t launch_fwdsub(const float* A, float* T, int64_t nc, int k, cudaStream_t st);  // k <= 256
cudaError_t launch_neumann_i8_simt(const float* A, float* T, int N, int mask, int8_t* q,
                                   int32_t* acc, float* sc, int64_t nc, cudaStream_t st);

// Inter-chunk state scan of the forward (scan.cu); k = 64, d = 128.
// bf16: U is overwritten by V~ (fp16) and Sstates ([B*H*nchunk][d][d] fp16) by
// the chunks' start states; f32 uses neither.
// normalize_q (bf16): the query rows come raw and are L2-normalised in the output pass.
cudaError_t launch_scan(const void* Q, const void* K, const void* Wg, void* U, const float* g,
                        const float* S0, void* O, float* Sfin, void* Sstates, int64_t BH,
                        int64_t nchunk, bool bf16, cudaStream_t st, bool normalize_q = false);

// Decode steps (decode.cu); d = 128, S [B][Hv][d][d] fp32 updated in place.
cudaError_t launch_decode(const void* Q, const void* K, const void* V, const float* beta,
                          const float* loggate, float* S, void* O, int64_t B, int64_t Hk,
                          int64_t Hv, int64_t n, bool bf16, cudaStream_t st);
// the same without the delta term, states in a pool: row b's state is S[slots[b]]
cudaError_t launch_linear_decode(const void* Q, const void* K, const void* V,
                                 const float* loggate, float* S, const int32_t* slots,
                                 int64_t nslots, float scale, void* O, int64_t B, int64_t Hk,
                                 int64_t Hv, int64_t n, bool bf16, cudaStream_t st);

// Rotary positions (rotary.cu); d = 128.
struct RotaryArgs {
    const void* Q; gdn_strides qs; void* Qo; gdn_strides qos;
    const void* K; gdn_strides ks; void* Ko; gdn_strides kos;
    const int64_t* positions; const float* inv_freq;
    float mscale; int rot, interleaved, inverse;
    int64_t B, Hq, Hk, T;
    int heads_per_cta;     // set by the launcher
};
cudaError_t launch_rotary(RotaryArgs a, bool bf16, cudaStream_t st);

// The norms around a block (norm.cu): forward, and backward with the partial
// weight gradients in ws (block_norm_ws_bytes).
struct NormArgs {
    const void* Y; gdn_strides ys;
    const void* Z; const float* w_post; const void* R; const float* w_pre;
    float scale, eps; int act;
    void* X; void* N;                                  // forward
    const void* dX; const void* dN;                    // backward
    void* dY; gdn_strides dys; void* dZ; void* dR; float* dw_post; float* dw_pre; float* ws;
    int64_t B, T, H, d;
};
cudaError_t launch_block_norm(const NormArgs& a, bool bf16, cudaStream_t st);
cudaError_t launch_block_norm_backward(const NormArgs& a, bool bf16, cudaStream_t st);
int64_t block_norm_ws_bytes(int64_t rows, int64_t width);

}  // namespace gdn
