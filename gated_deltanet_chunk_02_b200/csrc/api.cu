// api.cu — the C ABI of libgdn: argument checks, dispatch, status word.
//
// Every entry point validates its arguments on the host before launching
// anything; on failure it returns a negative code, launches nothing and keeps
// a message for gdn_last_error().  Kernels report device-side failures by
// OR-ing bits into a per-device status word (never by trapping).
#include <cstdio>
#include <cmath>
#include <cstdarg>
#include <cstring>
#include <string>

#include "../../include/gdn.h"
#include "common.cuh"
#include "kernels.h"
#include "linear.h"
#include "tc.h"

namespace gdn {
__device__ int g_status = 0;
}  // namespace gdn

namespace {

thread_local std::string t_last_error;
thread_local int64_t t_launches = 0;

int fail(int code, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    t_last_error = buf;
    return code;
}

int cuda_fail(cudaError_t e, const char* what) {
    return fail(GDN_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Shape checks shared by all entry points; *nc receives the chunk count.
int check_shape(const gdn_shape& s, int64_t* nc) {
    if (s.B < 0 || s.H < 0 || s.T < 0) return fail(GDN_ERR_ARG, "negative B, H or T");
    if (s.k != 32 && s.k != 64 && s.k != 128 && s.k != 256)
        return fail(GDN_ERR_ARG, "chunk size k=%d not in {32, 64, 128, 256}", s.k);
    if (s.T % s.k) return fail(GDN_ERR_ARG, "T=%lld is not a multiple of k=%d", (long long)s.T, s.k);
    if (s.d != 128) return fail(GDN_ERR_UNSUPPORTED, "head dim d=%d (only 128 is built)", s.d);
    // each factor is below 2^31, so the products below cannot overflow int64
    if (s.B > 0x7fffffffLL || s.H > 0x7fffffffLL || s.T / s.k > 0x7fffffffLL)
        return fail(GDN_ERR_ARG, "too many chunks (B=%lld, H=%lld, T/k=%lld)", (long long)s.B,
                    (long long)s.H, (long long)(s.T / s.k));
    const int64_t bh = s.B * s.H;
    if (bh > 0x7fffffffLL) return fail(GDN_ERR_ARG, "too many chunks (B*H=%lld)", (long long)bh);
    const int64_t n = bh * (s.T / s.k);
    if (n > 0x7fffffffLL) return fail(GDN_ERR_ARG, "too many chunks (%lld)", (long long)n);
    *nc = n;
    return GDN_OK;
}

int check_ptrs(std::initializer_list<std::pair<const void*, const char*>> ps) {
    for (auto& p : ps) {
        if (!p.first) return fail(GDN_ERR_ARG, "%s is NULL", p.second);
        if (!aligned16(p.first)) return fail(GDN_ERR_ALIGN, "%s is not 16-byte aligned", p.second);
    }
    return GDN_OK;
}

int check_opt_ptr(const void* p, const char* name) {
    if (p && !aligned16(p)) return fail(GDN_ERR_ALIGN, "%s is not 16-byte aligned", name);
    return GDN_OK;
}

int check_dtype(gdn_dtype dt) {
    if (dt != GDN_F32 && dt != GDN_BF16) return fail(GDN_ERR_ARG, "unknown dtype %d", (int)dt);
    return GDN_OK;
}

int check_NS(int N, int mask, int S, int k) {
    if (N < 1 || N > k - 1) return fail(GDN_ERR_ARG, "Neumann order N=%d outside [1, k-1]", N);
    if (mask != 0 && mask != 1) return fail(GDN_ERR_ARG, "mask must be 0 or 1");
    if (S < 0 || S > 64) return fail(GDN_ERR_ARG, "residual steps S=%d outside [0, 64]", S);
    return GDN_OK;
}

int launched(cudaError_t e, const char* what, int kernels = 1) {
    if (e != cudaSuccess) return cuda_fail(e, what);
    t_launches += kernels;
    return GDN_OK;
}

// Small vectors (positions, lengths, slots, per-head scalars): element alignment.
int check_vec(const void* p, size_t size, const char* name, bool optional = false) {
    if (!p) return optional ? GDN_OK : fail(GDN_ERR_ARG, "%s is NULL", name);
    if (reinterpret_cast<uintptr_t>(p) % size)
        return fail(GDN_ERR_ALIGN, "%s is not aligned to its %d-byte elements", name, (int)size);
    return GDN_OK;
}

// Strides of rows that are read and written 16 bytes at a time.
int check_strides(const gdn_strides& s, gdn_dtype dt, const char* name) {
    const int64_t vec = dt == GDN_BF16 ? 8 : 4;
    if (s.b < 0 || s.h < 0 || s.t < 0) return fail(GDN_ERR_ARG, "%s has a negative stride", name);
    if (s.b % vec || s.h % vec || s.t % vec)
        return fail(GDN_ERR_ALIGN, "%s: strides are not multiples of 16 bytes", name);
    return GDN_OK;
}

// Rows of an output may not share memory: every stride that is walked is at
// least the extent of the dimensions inside it, in some order of the three.
int check_out_strides(const gdn_strides& s, int64_t B, int64_t H, int64_t T, int64_t d,
                      const char* name) {
    int64_t st[3] = {s.b, s.h, s.t}, n[3] = {B, H, T};
    int64_t extent = d;
    bool used[3] = {n[0] <= 1, n[1] <= 1, n[2] <= 1};
    for (int pass = 0; pass < 3; ++pass) {
        int best = -1;
        for (int i = 0; i < 3; ++i)
            if (!used[i] && (best < 0 || st[i] < st[best])) best = i;
        if (best < 0) break;
        if (st[best] < extent) return fail(GDN_ERR_ARG, "%s: rows overlap", name);
        used[best] = true;
        extent += (n[best] - 1) * st[best];
    }
    return GDN_OK;
}

constexpr int64_t kMaxRows = 0x7fffffffLL;             // tokens or rows of a call

int check_linear(const gdn_linear_shape& s, const int32_t* cu, gdn_dtype dtype) {
    if (int rc = check_dtype(dtype)) return rc;
    if (s.B < 0 || s.Hk < 0 || s.Hv < 0 || s.T < 0 || s.nseq < 0)
        return fail(GDN_ERR_ARG, "negative B, Hk, Hv, T or nseq");
    if (s.d != 128) return fail(GDN_ERR_UNSUPPORTED, "head dim d=%d (only 128 is built)", s.d);
    if (s.B == 0 || s.Hv == 0) return GDN_OK;
    if (s.Hk == 0 || s.Hv % s.Hk)
        return fail(GDN_ERR_ARG, "Hv=%lld is not a multiple of Hk=%lld", (long long)s.Hv,
                    (long long)s.Hk);
    if (s.Hv > 8192) return fail(GDN_ERR_ARG, "Hv=%lld above 8192", (long long)s.Hv);
    if (s.nseq > 0 && s.B != 1) return fail(GDN_ERR_ARG, "packed sequences need B=1");
    if (s.T > kMaxRows || s.B > kMaxRows || s.nseq > kMaxRows ||
        s.B * s.Hv > kMaxRows / 16 || s.nseq * s.Hv > kMaxRows / 16 ||   // 12 blocks each
        s.T * 32 > kMaxRows * 8 / s.Hv / s.B)
        return fail(GDN_ERR_ARG, "too many rows (B=%lld, Hv=%lld, T=%lld, nseq=%lld)",
                    (long long)s.B, (long long)s.Hv, (long long)s.T, (long long)s.nseq);
    if (s.nseq > 0) return check_vec(cu, 4, "cu_seqlens");
    if (cu) return fail(GDN_ERR_ARG, "cu_seqlens without nseq");
    return GDN_OK;
}

// bytes of a linear attention call's tensors
struct LinearBytes {
    int64_t k, v, state, decay, cu;
    LinearBytes(const gdn_linear_shape& s, gdn_dtype dt)
        : k(s.B * s.Hk * s.T * s.d * (dt == GDN_BF16 ? 2 : 4)),
          v(s.B * s.Hv * s.T * s.d * (dt == GDN_BF16 ? 2 : 4)),
          state((s.nseq > 0 ? s.nseq : s.B) * s.Hv * s.d * s.d * 4), decay(s.Hv * 4),
          cu((s.nseq + 1) * 4) {}
};

// Outputs that are an input (or one another) by pointer.
int check_apart(std::initializer_list<std::pair<const void*, const char*>> outs,
                std::initializer_list<std::pair<const void*, const char*>> ins) {
    for (auto o = outs.begin(); o != outs.end(); ++o) {
        if (!o->first) continue;
        for (auto& i : ins)
            if (o->first == i.first) return fail(GDN_ERR_ARG, "%s is %s", o->second, i.second);
        for (auto p = o + 1; p != outs.end(); ++p)
            if (o->first == p->first) return fail(GDN_ERR_ARG, "%s is %s", p->second, o->second);
    }
    return GDN_OK;
}

// Rows of bytes at up to three strides (of bytes): a tensor as it lies in memory.
struct Rows {
    const void* p;
    int64_t row, st[3], n[3];
    const char* name;
};
Rows flat(const void* p, int64_t bytes, const char* name) {
    return {p, bytes, {0, 0, 0}, {1, 1, 1}, name};
}
Rows strided(const void* p, const gdn_strides& s, int64_t B, int64_t H, int64_t T, int64_t d,
             int64_t elem, const char* name) {
    return {p, d * elem, {s.b * elem, s.h * elem, s.t * elem}, {B, H, T}, name};
}

// Does at + sum st_i x_i fall into [lo, hi] for some lo_i <= x_i <= hi_i?  Terms
// by stride, the largest first: what the others can still add leaves a nested
// layout one or two x to try at each.  One that leaves thousands counts as yes.
struct Term {
    __int128 st, lo, hi;
};
bool falls_in(const Term* t, int n, __int128 at, __int128 lo, __int128 hi, int& tries) {
    if (n == 0) return lo <= at && at <= hi;
    __int128 below = 0, above = 0;
    for (int i = 1; i < n; ++i) {
        below += t[i].st * t[i].lo;
        above += t[i].st * t[i].hi;
    }
    const auto floor_div = [](__int128 a, __int128 b) { return a >= 0 ? a / b : -((b - 1 - a) / b); };
    __int128 x0 = -floor_div(at + above - lo, t->st), x1 = floor_div(hi - at - below, t->st);
    if (x0 < t->lo) x0 = t->lo;
    if (x1 > t->hi) x1 = t->hi;
    for (__int128 x = x0; x <= x1; ++x)
        if (--tries < 0 || falls_in(t + 1, n - 1, at + t->st * x, lo, hi, tries)) return true;
    return false;
}
// Do two tensors have a byte in common?  A row of b starts at a distance of
// above -b.row and below a.row from one of a.
bool share_memory(const Rows& a, const Rows& b) {
    Term t[6];
    int n = 0;
    const auto add = [&](int64_t st, int64_t lo, int64_t hi) {
        if (st == 0 || (lo == 0 && hi == 0)) return;
        int i = 0;
        while (i < n && t[i].st > st) ++i;
        if (i < n && t[i].st == st) {
            t[i].lo += lo;
            t[i].hi += hi;
            return;
        }
        for (int j = n++; j > i; --j) t[j] = t[j - 1];
        t[i] = {st, lo, hi};
    };
    for (int i = 0; i < 3; ++i) {
        if (a.n[i] <= 0 || b.n[i] <= 0) return false;
        add(b.st[i], 0, b.n[i] - 1);
        add(a.st[i], 1 - a.n[i], 0);
    }
    if (!a.p || !b.p || a.row <= 0 || b.row <= 0) return false;
    int tries = 4096;
    return falls_in(t, n, (__int128)(intptr_t)b.p - (intptr_t)a.p, 1 - b.row, a.row - 1, tries);
}
// Outputs share no memory with inputs or one another (an input that may be an
// output in place is left out by the caller).
int check_memory(std::initializer_list<Rows> outs, std::initializer_list<Rows> ins) {
    for (auto o = outs.begin(); o != outs.end(); ++o) {
        for (auto& i : ins)
            if (share_memory(*o, i))
                return fail(GDN_ERR_ARG, "%s shares memory with %s", o->name, i.name);
        for (auto p = o + 1; p != outs.end(); ++p)
            if (share_memory(*o, *p))
                return fail(GDN_ERR_ARG, "%s shares memory with %s", p->name, o->name);
    }
    return GDN_OK;
}

// the packed or padded sequences of a call
gdn::LinArgs linear_args(const gdn_linear_shape& s, const float* loggate, const int32_t* cu) {
    gdn::LinArgs a;
    memset(&a, 0, sizeof a);
    a.loggate = loggate;
    a.cu = s.nseq > 0 ? cu : nullptr;
    a.nseq = s.nseq > 0 ? s.nseq : s.B;
    a.B = s.B;
    a.Hv = s.Hv;
    a.T = s.T;
    return a;
}

}  // namespace

#define GDN_TRY(x)                  \
    do {                            \
        int _rc = (x);              \
        if (_rc != GDN_OK) return _rc; \
    } while (0)

extern "C" {

int gdn_build_A(const void* K, const float* beta, const float* g, float* A, gdn_shape s,
                gdn_dtype dtype, void* stream) {
    int64_t nc;
    GDN_TRY(check_shape(s, &nc));
    GDN_TRY(check_dtype(dtype));
    if (nc == 0) return GDN_OK;
    GDN_TRY(check_ptrs({{K, "K"}, {beta, "beta"}, {g, "g"}, {A, "A"}}));
    cudaStream_t st = (cudaStream_t)stream;
    if (dtype == GDN_BF16 && gdn::tc_available() && s.k <= 128)
        return launched(gdn::launch_build_A_tc(K, beta, g, A, nc, s.k, st), "build_A (tcgen05)");
    if (dtype == GDN_BF16 && gdn::tc_available() && s.k == 256)
        return launched(gdn::launch_build_A256_tc(K, beta, g, A, nc, st), "build_A k=256 (tcgen05)");
    return launched(gdn::launch_build_A_simt(K, beta, g, A, nc, s.k, dtype == GDN_BF16, st),
                    "build_A");
}

int gdn_invert_neumann(const float* A, float* T, gdn_shape s, int N, int mask, int S,
                       gdn_prec prec, void* stream) {
    int64_t nc;
    GDN_TRY(check_shape(s, &nc));
    GDN_TRY(check_NS(N, mask, S, s.k));
    if (prec != GDN_PREC_F32 && prec != GDN_PREC_F16) return fail(GDN_ERR_ARG, "unknown precision");
    if (nc == 0) return GDN_OK;
    GDN_TRY(check_ptrs({{A, "A"}, {T, "T"}}));
    cudaStream_t st = (cudaStream_t)stream;
    if (prec == GDN_PREC_F16) {
        if (!gdn::tc_available()) return fail(GDN_ERR_UNSUPPORTED, "tensor-core path not built");
        if (s.k == 256)
            return launched(gdn::launch_neumann256_tc(A, T, nc, N, mask, S, st),
                            "neumann k=256 (tcgen05)");
        return launched(gdn::launch_neumann_tc(A, T, nc, s.k, N, mask, S, st), "neumann (tcgen05)");
    }
    if (s.k > 128) return fail(GDN_ERR_UNSUPPORTED, "float32 Neumann chain supports k <= 128");
    return launched(gdn::launch_neumann_simt(A, T, nc, s.k, N, mask, S, st), "neumann");
}

int gdn_invert_newton(const float* A, float* T, gdn_shape s, int N, int mask, int M,
                      void* stream) {
    int64_t nc;
    GDN_TRY(check_shape(s, &nc));
    GDN_TRY(check_NS(N, mask, 0, s.k));
    if (M < 0 || M > 6) return fail(GDN_ERR_ARG, "correction steps M=%d outside [0, 6]", M);
    if (s.k == 256) return fail(GDN_ERR_UNSUPPORTED, "sequential correction supports k <= 128");
    if (nc == 0) return GDN_OK;
    GDN_TRY(check_ptrs({{A, "A"}, {T, "T"}}));
    if (!gdn::tc_available()) return fail(GDN_ERR_UNSUPPORTED, "tensor-core path not built");
    return launched(gdn::launch_newton_tc(A, T, nc, s.k, N, mask, M, (cudaStream_t)stream),
                    "newton (tcgen05)");
}

int gdn_invert_blocked(const float* A, float* T, gdn_shape s, void* stream) {
    int64_t nc;
    GDN_TRY(check_shape(s, &nc));
    if (s.k > 64) return fail(GDN_ERR_UNSUPPORTED, "the block-decomposition inverse supports k <= 64");
    if (nc == 0) return GDN_OK;
    GDN_TRY(check_ptrs({{A, "A"}, {T, "T"}}));
    if (!gdn::tc_available()) return fail(GDN_ERR_UNSUPPORTED, "tensor-core path not built");
    return launched(gdn::launch_blockinv_tc(A, T, nc, s.k, (cudaStream_t)stream),
                    "blocked inverse (tcgen05)");
}

int gdn_invert_fwdsub(const float* A, float* T, gdn_shape s, void* stream) {
    int64_t nc;
    GDN_TRY(check_shape(s, &nc));
    if (nc == 0) return GDN_OK;
    GDN_TRY(check_ptrs({{A, "A"}, {T, "T"}}));
    return launched(gdn::launch_fwdsub(A, T, nc, s.k, (cudaStream_t)stream), "fwdsub");
}

int gdn_wy(const float* T, const void* K, const void* V, const float* beta, const float* g,
           void* W, void* U, gdn_shape s, gdn_dtype dtype, void* stream) {
    int64_t nc;
    GDN_TRY(check_shape(s, &nc));
    GDN_TRY(check_dtype(dtype));
    if (nc == 0) return GDN_OK;
    GDN_TRY(check_ptrs({{T, "T"}, {K, "K"}, {V, "V"}, {beta, "beta"}, {W, "W"}, {U, "U"}}));
    GDN_TRY(check_opt_ptr(g, "g"));
    cudaStream_t st = (cudaStream_t)stream;
    if (s.k > 128) return fail(GDN_ERR_UNSUPPORTED, "wy serves k <= 128");
    if (dtype == GDN_BF16 && gdn::tc_available())
        return launched(gdn::launch_wy_tc(T, K, V, beta, g, W, U, nc, s.k, st), "wy (tcgen05)");
    return launched(gdn::launch_wy_simt(T, K, V, beta, g, W, U, nc, s.k, dtype == GDN_BF16, st),
                    "wy");
}

int gdn_invert_neumann_i8(const float* A, float* T, int N, int mask, int8_t* q_dbg,
                          int32_t* acc_dbg, float* scale_dbg, gdn_shape s, void* stream) {
    int64_t nc;
    GDN_TRY(check_shape(s, &nc));
    if (s.k != 64) return fail(GDN_ERR_UNSUPPORTED, "INT8 path is built for k=64");
    if (N < 1 || N > 8) return fail(GDN_ERR_ARG, "INT8 path: N=%d outside [1, 8]", N);
    if (mask != 0 && mask != 1) return fail(GDN_ERR_ARG, "mask must be 0 or 1");
    if (nc == 0) return GDN_OK;
    GDN_TRY(check_ptrs({{A, "A"}, {T, "T"}}));
    GDN_TRY(check_opt_ptr(q_dbg, "q_dbg"));
    GDN_TRY(check_opt_ptr(acc_dbg, "acc_dbg"));
    GDN_TRY(check_opt_ptr(scale_dbg, "scale_dbg"));
    cudaStream_t st = (cudaStream_t)stream;
    if (gdn::tc_i8_available())
        return launched(gdn::launch_neumann_i8_tc(A, T, N, mask, q_dbg, acc_dbg, scale_dbg, nc, st),
                        "neumann_i8 (tcgen05)");
    return launched(gdn::launch_neumann_i8_simt(A, T, N, mask, q_dbg, acc_dbg, scale_dbg, nc, st),
                    "neumann_i8");
}

int gdn_invert_neumann_i8_residual(const float* A, float* T, int N, int mask, int S,
                                   gdn_shape s, void* stream) {
    int64_t nc;
    GDN_TRY(check_shape(s, &nc));
    if (s.k != 64) return fail(GDN_ERR_UNSUPPORTED, "INT8 path is built for k=64");
    if (N < 1 || N > 8) return fail(GDN_ERR_ARG, "INT8 path: N=%d outside [1, 8]", N);
    if (mask != 0 && mask != 1) return fail(GDN_ERR_ARG, "mask must be 0 or 1");
    if (S < 1 || S > 64) return fail(GDN_ERR_ARG, "residual steps S=%d outside [1, 64]", S);
    if (nc == 0) return GDN_OK;
    GDN_TRY(check_ptrs({{A, "A"}, {T, "T"}}));
    if (!gdn::tc_i8_available()) return fail(GDN_ERR_UNSUPPORTED, "integer tensor-core path not built");
    return launched(gdn::launch_neumann_i8_tc(A, T, N, mask, nullptr, nullptr, nullptr, nc,
                                              (cudaStream_t)stream, S),
                    "neumann_i8 with residual (tcgen05)");
}

int gdn_invert_neumann_i16(const float* A, float* T, int N, int mask, int16_t* q_dbg,
                           int64_t* acc_dbg, double* scale_dbg, gdn_shape s, void* stream) {
    int64_t nc;
    GDN_TRY(check_shape(s, &nc));
    if (s.k != 64) return fail(GDN_ERR_UNSUPPORTED, "the INT16 path is built for k = 64");
    if (N < 1 || N > 8) return fail(GDN_ERR_ARG, "INT16 Neumann order N=%d outside [1, 8]", N);
    if (mask != 0 && mask != 1) return fail(GDN_ERR_ARG, "mask must be 0 or 1");
    if (nc == 0) return GDN_OK;
    GDN_TRY(check_ptrs({{A, "A"}, {T, "T"}}));
    GDN_TRY(check_opt_ptr(q_dbg, "q"));
    GDN_TRY(check_opt_ptr(acc_dbg, "acc"));
    GDN_TRY(check_opt_ptr(scale_dbg, "scale"));
    if (!gdn::tc_i8_available()) return fail(GDN_ERR_UNSUPPORTED, "integer tensor-core path not built");
    return launched(gdn::launch_neumann_i16_tc(A, T, N, mask, q_dbg, acc_dbg, scale_dbg, nc,
                                               (cudaStream_t)stream),
                    "neumann int16 (tcgen05)");
}

int gdn_invert_neumann_i16_residual(const float* A, float* T, int N, int mask, int S,
                                    gdn_shape s, void* stream) {
    int64_t nc;
    GDN_TRY(check_shape(s, &nc));
    if (s.k != 64) return fail(GDN_ERR_UNSUPPORTED, "the INT16 path is built for k = 64");
    if (N < 1 || N > 8) return fail(GDN_ERR_ARG, "INT16 Neumann order N=%d outside [1, 8]", N);
    if (mask != 0 && mask != 1) return fail(GDN_ERR_ARG, "mask must be 0 or 1");
    if (S < 1 || S > 64) return fail(GDN_ERR_ARG, "residual steps S=%d outside [1, 64]", S);
    if (nc == 0) return GDN_OK;
    GDN_TRY(check_ptrs({{A, "A"}, {T, "T"}}));
    if (!gdn::tc_i8_available()) return fail(GDN_ERR_UNSUPPORTED, "integer tensor-core path not built");
    return launched(gdn::launch_neumann_i16_tc(A, T, N, mask, nullptr, nullptr, nullptr, nc,
                                               (cudaStream_t)stream, S),
                    "neumann int16 with residual (tcgen05)");
}

int gdn_chunk_wy_fused(const void* K, const void* V, const float* beta, const float* g, int N,
                       int mask, int S, int gated, void* W, void* U, float* T_out, gdn_shape s,
                       gdn_dtype dtype, void* stream) {
    int64_t nc;
    GDN_TRY(check_shape(s, &nc));
    GDN_TRY(check_dtype(dtype));
    GDN_TRY(check_NS(N, mask, S, s.k));
    if (gated != 0 && gated != 1) return fail(GDN_ERR_ARG, "gated must be 0 or 1");
    if (nc == 0) return GDN_OK;
    GDN_TRY(check_ptrs({{K, "K"}, {V, "V"}, {beta, "beta"}, {g, "g"}, {W, "W"}, {U, "U"}}));
    GDN_TRY(check_opt_ptr(T_out, "T_out"));
    cudaStream_t st = (cudaStream_t)stream;
    if (dtype == GDN_BF16 && gdn::tc_available()) {
        if (s.k > 128) return fail(GDN_ERR_UNSUPPORTED, "fused tensor-core path serves k <= 128");
        return launched(gdn::launch_fused_tc(K, V, beta, g, N, mask, S, gated, W, U, T_out, nc,
                                             s.k, st),
                        "chunk_wy_fused (tcgen05)");
    }
    if (s.k > 128) return fail(GDN_ERR_UNSUPPORTED, "fused CUDA-core path supports k <= 128");
    return launched(gdn::launch_fused_simt(K, V, beta, g, N, mask, S, gated, W, U, T_out, nc,
                                           s.k, dtype == GDN_BF16, st),
                    "chunk_wy_fused");
}

int gdn_chunk_wy_fused_raw(const void* K_raw, const void* V, const float* beta,
                           const float* loggate, int N, int mask, int S, int gated, void* W,
                           void* U, float* T_out, void* K_out, float* g_out, gdn_shape s,
                           gdn_dtype dtype, void* stream) {
    int64_t nc;
    GDN_TRY(check_shape(s, &nc));
    GDN_TRY(check_dtype(dtype));
    GDN_TRY(check_NS(N, mask, S, s.k));
    if (dtype != GDN_BF16) return fail(GDN_ERR_UNSUPPORTED, "the prologue is built for bf16 data");
    if (s.k == 256) return fail(GDN_ERR_UNSUPPORTED, "the fused step supports k <= 128");
    if (nc == 0) return GDN_OK;
    GDN_TRY(check_ptrs({{K_raw, "K_raw"}, {V, "V"}, {beta, "beta"}, {loggate, "loggate"},
                        {W, "W"}, {U, "U"}}));
    GDN_TRY(check_opt_ptr(T_out, "T_out"));
    GDN_TRY(check_opt_ptr(K_out, "K_out"));
    GDN_TRY(check_opt_ptr(g_out, "g_out"));
    if (!gdn::tc_available()) return fail(GDN_ERR_UNSUPPORTED, "tensor-core path not built");
    return launched(gdn::launch_fused_raw_tc(K_raw, V, beta, loggate, N, mask, S, gated, W, U,
                                             T_out, K_out, g_out, nc, s.k, (cudaStream_t)stream),
                    "fused with prologue (tcgen05)");
}

int64_t gdn_forward_workspace_bytes(gdn_shape s, gdn_dtype dtype) {
    int64_t nc;
    if (check_shape(s, &nc) != GDN_OK) return -1;
    if (dtype != GDN_F32 && dtype != GDN_BF16) return -1;
    const int64_t elem = dtype == GDN_BF16 ? 2 : 4;
    const int64_t rows = nc * s.k;
    // W_g and U for every chunk, then A and T (exact path)
    return 2 * rows * s.d * elem + 2 * nc * (int64_t)s.k * s.k * 4;
}

int gdn_forward(const void* Q, const void* K, const void* V, const float* beta, const float* g,
                const float* S0, int N, int mask, int S, int exact, void* O, float* S_final,
                void* workspace, int64_t workspace_bytes, gdn_shape s, gdn_dtype dtype,
                void* stream) {
    int64_t nc;
    GDN_TRY(check_shape(s, &nc));
    GDN_TRY(check_dtype(dtype));
    if (s.k != 64) return fail(GDN_ERR_UNSUPPORTED, "gdn_forward is built for k=64");
    if (exact != 0 && exact != 1) return fail(GDN_ERR_ARG, "exact must be 0 or 1");
    if (!exact) GDN_TRY(check_NS(N, mask, S, s.k));
    if (nc == 0) return GDN_OK;
    GDN_TRY(check_ptrs({{Q, "Q"}, {K, "K"}, {V, "V"}, {beta, "beta"}, {g, "g"}, {O, "O"},
                        {S_final, "S_final"}, {workspace, "workspace"}}));
    GDN_TRY(check_opt_ptr(S0, "S0"));
    const int64_t need = gdn_forward_workspace_bytes(s, dtype);
    if (workspace_bytes < need)
        return fail(GDN_ERR_ARG, "workspace of %lld bytes is below the %lld needed",
                    (long long)workspace_bytes, (long long)need);
    cudaStream_t st = (cudaStream_t)stream;
    const bool bf16 = dtype == GDN_BF16;
    const int64_t elem = bf16 ? 2 : 4;
    const int64_t rows = nc * s.k;
    uint8_t* ws = (uint8_t*)workspace;
    void* Wg = ws;
    void* U = ws + rows * s.d * elem;
    float* Abuf = (float*)(ws + 2 * rows * s.d * elem);
    float* Tbuf = Abuf + nc * (int64_t)s.k * s.k;
    if (exact) {
        GDN_TRY(gdn_build_A(K, beta, g, Abuf, s, dtype, stream));
        GDN_TRY(gdn_invert_fwdsub(Abuf, Tbuf, s, stream));
        GDN_TRY(gdn_wy(Tbuf, K, V, beta, g, Wg, U, s, dtype, stream));
    } else {
        GDN_TRY(gdn_chunk_wy_fused(K, V, beta, g, N, mask, S, 1, Wg, U, nullptr, s, dtype,
                                   stream));
    }
    // the A / T region (2 k^2 f32 per chunk = d^2 fp16 at k = 64) takes the
    // chunks' start states of the bf16 scan
    return launched(gdn::launch_scan(Q, K, Wg, U, g, S0, O, S_final, Abuf, s.B * s.H, s.T / s.k,
                                     bf16, st),
                    "forward scan");
}

int64_t gdn_forward_raw_workspace_bytes(gdn_shape s, gdn_dtype dtype) {
    int64_t nc;
    if (check_shape(s, &nc) != GDN_OK || dtype != GDN_BF16) return -1;
    const int64_t rows = nc * s.k;
    // gdn_forward's scratch, then the normalised keys (bf16) and the summed gates
    return gdn_forward_workspace_bytes(s, dtype) + rows * s.d * 2 + rows * 4;
}

int gdn_forward_raw(const void* Q_raw, const void* K_raw, const void* V, const float* beta,
                    const float* loggate, const float* S0, int N, int mask, int S, void* O,
                    float* S_final, void* workspace, int64_t workspace_bytes, gdn_shape s,
                    gdn_dtype dtype, void* stream) {
    int64_t nc;
    GDN_TRY(check_shape(s, &nc));
    GDN_TRY(check_dtype(dtype));
    if (dtype != GDN_BF16) return fail(GDN_ERR_UNSUPPORTED, "gdn_forward_raw is built for bf16 data");
    if (s.k != 64) return fail(GDN_ERR_UNSUPPORTED, "gdn_forward_raw is built for k=64");
    GDN_TRY(check_NS(N, mask, S, s.k));
    if (nc == 0) return GDN_OK;
    GDN_TRY(check_ptrs({{Q_raw, "Q_raw"}, {K_raw, "K_raw"}, {V, "V"}, {beta, "beta"},
                        {loggate, "loggate"}, {O, "O"}, {S_final, "S_final"},
                        {workspace, "workspace"}}));
    GDN_TRY(check_opt_ptr(S0, "S0"));
    if (!gdn::tc_available()) return fail(GDN_ERR_UNSUPPORTED, "tensor-core path not built");
    const int64_t need = gdn_forward_raw_workspace_bytes(s, dtype);
    if (workspace_bytes < need)
        return fail(GDN_ERR_ARG, "workspace of %lld bytes is below the %lld needed",
                    (long long)workspace_bytes, (long long)need);
    cudaStream_t st = (cudaStream_t)stream;
    const int64_t rows = nc * s.k;
    uint8_t* ws = (uint8_t*)workspace;
    void* Wg = ws;
    void* U = ws + rows * s.d * 2;
    float* Sstates = (float*)(ws + 2 * rows * s.d * 2);
    uint8_t* tail = ws + gdn_forward_workspace_bytes(s, dtype);
    void* Kn = tail;                                    // the normalised keys
    float* gsum = (float*)(tail + rows * s.d * 2);      // the chunk-local cumulative gates
    GDN_TRY(gdn_chunk_wy_fused_raw(K_raw, V, beta, loggate, N, mask, S, 1, Wg, U, nullptr, Kn,
                                   gsum, s, dtype, stream));
    return launched(gdn::launch_scan(Q_raw, Kn, Wg, U, gsum, S0, O, S_final, Sstates, s.B * s.H,
                                     s.T / s.k, true, st, true),
                    "forward scan (raw queries)");
}

int gdn_decode(const void* Q, const void* K, const void* V, const float* beta,
               const float* loggate, float* S, void* O, int64_t B, int64_t Hk, int64_t Hv,
               int64_t n, int32_t d, gdn_dtype dtype, void* stream) {
    GDN_TRY(check_dtype(dtype));
    if (B < 0 || Hk < 0 || Hv < 0 || n < 0) return fail(GDN_ERR_ARG, "negative B, Hk, Hv or n");
    if (d != 128) return fail(GDN_ERR_UNSUPPORTED, "head dim d=%d (only 128 is built)", d);
    if (B == 0 || Hv == 0 || n == 0) return GDN_OK;
    if (Hk == 0 || Hv % Hk)
        return fail(GDN_ERR_ARG, "Hv=%lld is not a multiple of Hk=%lld", (long long)Hv,
                    (long long)Hk);
    if (B > 65535 || Hv > (1LL << 28) || n > 0x7fffffffLL)
        return fail(GDN_ERR_ARG, "B, Hv or n too large");
    GDN_TRY(check_ptrs({{Q, "Q"}, {K, "K"}, {V, "V"}, {beta, "beta"}, {loggate, "loggate"},
                        {S, "S"}, {O, "O"}}));
    return launched(gdn::launch_decode(Q, K, V, beta, loggate, S, O, B, Hk, Hv, n,
                                       dtype == GDN_BF16, (cudaStream_t)stream),
                    "decode");
}

int gdn_rotary_frequencies(float* inv_freq, float* mscale, int rot, double base, int scaling,
                           double factor, int64_t original_length) {
    if (!inv_freq || !mscale) return fail(GDN_ERR_ARG, "inv_freq or mscale is NULL");
    if (rot < 2 || rot > 128 || rot % 2)
        return fail(GDN_ERR_ARG, "rot=%d is not an even number in [2, 128]", rot);
    if (!(base > 1.0) || !std::isfinite(base)) return fail(GDN_ERR_ARG, "base must be above 1");
    if (scaling < GDN_ROTARY_PLAIN || scaling > GDN_ROTARY_YARN)
        return fail(GDN_ERR_ARG, "unknown scaling %d", scaling);
    if (scaling != GDN_ROTARY_PLAIN && (!(factor >= 1.0) || !std::isfinite(factor)))
        return fail(GDN_ERR_ARG, "factor must be at least 1");
    if (scaling == GDN_ROTARY_YARN && original_length < 1)
        return fail(GDN_ERR_ARG, "original_length must be positive");
    if (scaling == GDN_ROTARY_NTK && rot > 2) base *= std::pow(factor, rot / (rot - 2.0));
    for (int i = 0; i < rot / 2; ++i) {
        double f = std::pow(base, -2.0 * i / rot);
        if (scaling == GDN_ROTARY_LINEAR) f /= factor;
        if (scaling == GDN_ROTARY_YARN) {
            const double turns = (double)original_length * f / 6.283185307179586;
            double keep = (turns - 1.0) / 31.0;
            keep = keep < 0.0 ? 0.0 : (keep > 1.0 ? 1.0 : keep);
            f *= keep + (1.0 - keep) / factor;
        }
        inv_freq[i] = (float)f;
    }
    *mscale = scaling == GDN_ROTARY_YARN ? (float)(0.1 * std::log(factor) + 1.0) : 1.f;
    return GDN_OK;
}

int gdn_rotary(const void* Q, gdn_strides qs, void* Q_out, gdn_strides qos, const void* K,
               gdn_strides ks, void* K_out, gdn_strides kos, const int64_t* positions,
               const float* inv_freq, float mscale, int rot, int interleaved, int inverse,
               int64_t B, int64_t Hq, int64_t Hk, int64_t T, int32_t d, gdn_dtype dtype,
               void* stream) {
    GDN_TRY(check_dtype(dtype));
    if (B < 0 || Hq < 0 || Hk < 0 || T < 0) return fail(GDN_ERR_ARG, "negative B, Hq, Hk or T");
    if (d != 128) return fail(GDN_ERR_UNSUPPORTED, "head dim d=%d (only 128 is built)", d);
    if (rot < 2 || rot > d || rot % 2)
        return fail(GDN_ERR_ARG, "rot=%d is not an even number in [2, %d]", rot, d);
    if ((interleaved != 0 && interleaved != 1) || (inverse != 0 && inverse != 1))
        return fail(GDN_ERR_ARG, "interleaved and inverse must be 0 or 1");
    if (B == 0 || T == 0 || Hq + Hk == 0) return GDN_OK;
    if (B > kMaxRows || T > kMaxRows || B * T > kMaxRows || Hq > 65536 || Hk > 65536)
        return fail(GDN_ERR_ARG, "too many tokens or heads");
    GDN_TRY(check_vec(positions, 8, "positions"));
    GDN_TRY(check_vec(inv_freq, 4, "inv_freq"));
    if (Hq > 0) {
        GDN_TRY(check_ptrs({{Q, "Q"}, {Q_out, "Q_out"}}));
        GDN_TRY(check_strides(qs, dtype, "Q"));
        GDN_TRY(check_strides(qos, dtype, "Q_out"));
        GDN_TRY(check_out_strides(qos, B, Hq, T, d, "Q_out"));
    }
    if (Hk > 0) {
        GDN_TRY(check_ptrs({{K, "K"}, {K_out, "K_out"}}));
        GDN_TRY(check_strides(ks, dtype, "K"));
        GDN_TRY(check_strides(kos, dtype, "K_out"));
        GDN_TRY(check_out_strides(kos, B, Hk, T, d, "K_out"));
    }
    // in place: the same rows; else apart
    const auto in_place = [&](const gdn_strides& i, const gdn_strides& o, int64_t H) {
        return (B == 1 || i.b == o.b) && (H == 1 || i.h == o.h) && (T == 1 || i.t == o.t);
    };
    if (Hq > 0 && Q == Q_out && !in_place(qs, qos, Hq))
        return fail(GDN_ERR_ARG, "Q_out is Q with other strides");
    if (Hk > 0 && K == K_out && !in_place(ks, kos, Hk))
        return fail(GDN_ERR_ARG, "K_out is K with other strides");
    if (Hq > 0 && Hk > 0) {
        GDN_TRY(check_apart({{Q_out, "Q_out"}, {K_out, "K_out"}}, {}));
        GDN_TRY(check_apart({{Q_out, "Q_out"}}, {{K, "K"}}));
        GDN_TRY(check_apart({{K_out, "K_out"}}, {{Q, "Q"}}));
    }
    const int64_t el = dtype == GDN_BF16 ? 2 : 4;
    const auto rows = [&](const void* p, const gdn_strides& s, int64_t H, const char* name) {
        return strided(H > 0 ? p : nullptr, s, B, H, T, d, el, name);
    };
    GDN_TRY(check_memory({rows(Q_out, qos, Hq, "Q_out"), rows(K_out, kos, Hk, "K_out")},
                         {rows(Q == Q_out ? nullptr : Q, qs, Hq, "Q"),
                          rows(K == K_out ? nullptr : K, ks, Hk, "K"),
                          flat(positions, B * T * 8, "positions"),
                          flat(inv_freq, rot / 2 * 4, "inv_freq")}));
    gdn::RotaryArgs a;
    memset(&a, 0, sizeof a);
    a.Q = Q; a.qs = qs; a.Qo = Q_out; a.qos = qos;
    a.K = K; a.ks = ks; a.Ko = K_out; a.kos = kos;
    a.positions = positions; a.inv_freq = inv_freq; a.mscale = mscale;
    a.rot = rot; a.interleaved = interleaved; a.inverse = inverse;
    a.B = B; a.Hq = Hq; a.Hk = Hk; a.T = T;
    return launched(gdn::launch_rotary(a, dtype == GDN_BF16, (cudaStream_t)stream), "rotary");
}

int64_t gdn_linear_forward_workspace_bytes(gdn_linear_shape s, gdn_dtype dtype) {
    static const int32_t some = 0;
    if (check_linear(s, s.nseq > 0 ? &some : nullptr, dtype) != GDN_OK) return -1;
    if (s.B == 0 || s.Hv == 0) return 0;
    return gdn::linear_plan(s, 1, dtype == GDN_BF16).state_bytes;
}

int gdn_linear_forward(const void* Q, const void* K, const void* V, const float* loggate,
                       const float* S0, const int32_t* cu_seqlens, float scale, void* O,
                       float* S_final, void* workspace, int64_t workspace_bytes,
                       gdn_linear_shape s, gdn_dtype dtype, void* stream) {
    GDN_TRY(check_linear(s, cu_seqlens, dtype));
    if (s.B == 0 || s.Hv == 0) return GDN_OK;
    if (s.T > 0) GDN_TRY(check_ptrs({{Q, "Q"}, {K, "K"}, {V, "V"}, {O, "O"}}));
    GDN_TRY(check_vec(loggate, 4, "loggate"));
    GDN_TRY(check_opt_ptr(S0, "S0"));
    GDN_TRY(check_opt_ptr(S_final, "S_final"));
    if (s.T > 0)
        GDN_TRY(check_apart({{O, "O"}, {S_final, "S_final"}},
                            {{Q, "Q"}, {K, "K"}, {V, "V"}, {S0, "S0"}}));
    const gdn::LinPlan pl = gdn::linear_plan(s, 1, dtype == GDN_BF16);
    if (workspace_bytes < pl.state_bytes)
        return fail(GDN_ERR_ARG, "workspace of %lld bytes is below the %lld needed",
                    (long long)workspace_bytes, (long long)pl.state_bytes);
    if (pl.state_bytes > 0) GDN_TRY(check_ptrs({{workspace, "workspace"}}));
    const LinearBytes n(s, dtype);
    GDN_TRY(check_memory({flat(O, n.v, "O"), flat(S_final, n.state, "S_final"),
                          flat(workspace, pl.state_bytes, "workspace")},
                         {flat(Q, n.k, "Q"), flat(K, n.k, "K"), flat(V, n.v, "V"),
                          flat(S0 == S_final ? nullptr : S0, n.state, "S0"),
                          flat(loggate, n.decay, "loggate"), flat(cu_seqlens, n.cu, "cu_seqlens")}));
    const int group = (int)(s.Hv / s.Hk);
    gdn::LinArgs a = linear_args(s, loggate, cu_seqlens);
    a.pr[0] = {Q, K, V, O, group, group, 1, 0, 0, S0, 0, S_final, 1, scale, 1.f, 1.f, 0, nullptr};
    int kernels = 0;
    return launched(gdn::launch_linear(a, 1, pl, dtype == GDN_BF16, workspace, &kernels,
                                       (cudaStream_t)stream),
                    "linear forward", kernels);
}

int64_t gdn_linear_backward_workspace_bytes(gdn_linear_shape s, gdn_dtype dtype) {
    static const int32_t some = 0;
    if (check_linear(s, s.nseq > 0 ? &some : nullptr, dtype) != GDN_OK) return -1;
    if (s.B == 0 || s.Hv == 0) return 0;
    const int64_t part = s.Hv == s.Hk ? 0 : s.B * s.Hv * s.T * (int64_t)s.d * 4;
    return 2 * gdn::linear_plan(s, 3, dtype == GDN_BF16).state_bytes + 2 * part;
}

int gdn_linear_backward(const void* Q, const void* K, const void* V, const float* loggate,
                        const float* S0, const void* dO, const float* dS_final,
                        const int32_t* cu_seqlens, float scale, void* dQ, void* dK, void* dV,
                        float* dS0, void* workspace, int64_t workspace_bytes, gdn_linear_shape s,
                        gdn_dtype dtype, void* stream) {
    GDN_TRY(check_linear(s, cu_seqlens, dtype));
    if (s.B > 0 && s.Hk > 0 && s.Hv == 0)              // dQ and dK would be sums over nothing
        return fail(GDN_ERR_ARG, "Hk=%lld without value heads", (long long)s.Hk);
    if (s.B == 0 || s.Hv == 0) return GDN_OK;
    if (s.T > 0)
        GDN_TRY(check_ptrs({{Q, "Q"}, {K, "K"}, {V, "V"}, {dO, "dO"}, {dQ, "dQ"}, {dK, "dK"},
                            {dV, "dV"}}));
    GDN_TRY(check_vec(loggate, 4, "loggate"));
    GDN_TRY(check_opt_ptr(S0, "S0"));
    GDN_TRY(check_opt_ptr(dS_final, "dS_final"));
    GDN_TRY(check_opt_ptr(dS0, "dS0"));
    if (s.T > 0)
        GDN_TRY(check_apart({{dQ, "dQ"}, {dK, "dK"}, {dV, "dV"}, {dS0, "dS0"}},
                            {{Q, "Q"}, {K, "K"}, {V, "V"}, {S0, "S0"}, {dO, "dO"},
                             {dS_final, "dS_final"}}));
    const int64_t need = gdn_linear_backward_workspace_bytes(s, dtype);
    if (workspace_bytes < need)
        return fail(GDN_ERR_ARG, "workspace of %lld bytes is below the %lld needed",
                    (long long)workspace_bytes, (long long)need);
    if (need > 0) GDN_TRY(check_ptrs({{workspace, "workspace"}}));
    const LinearBytes n(s, dtype);
    GDN_TRY(check_memory({flat(dQ, n.k, "dQ"), flat(dK, n.k, "dK"), flat(dV, n.v, "dV"),
                          flat(dS0, n.state, "dS0"), flat(workspace, need, "workspace")},
                         {flat(Q, n.k, "Q"), flat(K, n.k, "K"), flat(V, n.v, "V"),
                          flat(S0, n.state, "S0"), flat(dO, n.v, "dO"),
                          flat(dS_final == dS0 ? nullptr : dS_final, n.state, "dS_final"),
                          flat(loggate, n.decay, "loggate"), flat(cu_seqlens, n.cu, "cu_seqlens")}));
    const bool bf16 = dtype == GDN_BF16;
    const gdn::LinPlan pl = gdn::linear_plan(s, 3, bf16);
    const int group = (int)(s.Hv / s.Hk);
    const int64_t part = group == 1 ? 0 : s.B * s.Hv * s.T * (int64_t)s.d;
    float* pq = (float*)((uint8_t*)workspace + 2 * pl.state_bytes);
    float* pk = pq + part;
    const int f32 = group > 1;
    gdn::LinArgs a = linear_args(s, loggate, cu_seqlens);
    a.pr[0] = {dO, V, K, f32 ? (void*)pq : dQ, 1, 1, group, 0, f32, S0, 1, nullptr, 0,
               scale, 1.f, 1.f, 0, nullptr};
    // dk's states are dv's, transposed
    a.pr[1] = {V, dO, Q, f32 ? (void*)pk : dK, 1, 1, group, 1, f32, dS_final, 1, nullptr, 0,
               1.f, scale, scale, 1, nullptr};
    a.pr[2] = {K, Q, dO, dV, group, group, 1, 1, 0, dS_final, 0, dS0, 1, 1.f, scale, scale, 0,
               nullptr};
    cudaStream_t st = (cudaStream_t)stream;
    int kernels = 0;
    GDN_TRY(launched(gdn::launch_linear(a, 3, pl, bf16, workspace, &kernels, st),
                     "linear backward", kernels));
    if (group > 1 && s.T > 0) {
        GDN_TRY(launched(gdn::launch_linear_group_sum(a, pq, dQ, group, bf16, st), "dQ of a group"));
        GDN_TRY(launched(gdn::launch_linear_group_sum(a, pk, dK, group, bf16, st), "dK of a group"));
    }
    return GDN_OK;
}

int gdn_linear_decode(const void* Q, const void* K, const void* V, const float* loggate, float* S,
                      const int32_t* slots, int64_t nslots, float scale, void* O, int64_t B,
                      int64_t Hk, int64_t Hv, int64_t n, int32_t d, gdn_dtype dtype,
                      void* stream) {
    GDN_TRY(check_dtype(dtype));
    if (B < 0 || Hk < 0 || Hv < 0 || n < 0) return fail(GDN_ERR_ARG, "negative B, Hk, Hv or n");
    if (d != 128) return fail(GDN_ERR_UNSUPPORTED, "head dim d=%d (only 128 is built)", d);
    if (B == 0 || Hv == 0 || n == 0) return GDN_OK;
    if (Hk == 0 || Hv % Hk)
        return fail(GDN_ERR_ARG, "Hv=%lld is not a multiple of Hk=%lld", (long long)Hv,
                    (long long)Hk);
    if (B > 65535 || Hv > (1LL << 28) || n > 0x7fffffffLL)
        return fail(GDN_ERR_ARG, "B, Hv or n too large");
    if (nslots < (slots ? 0 : B))
        return fail(GDN_ERR_ARG, "nslots=%lld is below %lld", (long long)nslots,
                    (long long)(slots ? 0 : B));
    GDN_TRY(check_ptrs({{Q, "Q"}, {K, "K"}, {V, "V"}, {S, "S"}, {O, "O"}}));
    GDN_TRY(check_vec(loggate, 4, "loggate"));
    GDN_TRY(check_vec(slots, 4, "slots", true));
    GDN_TRY(check_apart({{O, "O"}, {S, "S"}}, {{Q, "Q"}, {K, "K"}, {V, "V"}}));
    const int64_t row = n * d * (dtype == GDN_BF16 ? 2 : 4);
    const auto all = [](int64_t a, int64_t b) {        // sizes have no bound of their own here
        return b != 0 && a > INT64_MAX / b ? INT64_MAX : a * b;
    };
    const int64_t k = all(B * Hk, row), v = all(B * Hv, row);
    GDN_TRY(check_memory({flat(O, v, "O"), flat(S, all(nslots, Hv * d * d * 4), "S")},
                         {flat(Q, k, "Q"), flat(K, k, "K"), flat(V, v, "V"),
                          flat(loggate, Hv * 4, "loggate"),
                          flat(slots, B * 4, "slots")}));
    return launched(gdn::launch_linear_decode(Q, K, V, loggate, S, slots, nslots, scale, O, B, Hk,
                                              Hv, n, dtype == GDN_BF16, (cudaStream_t)stream),
                    "linear decode");
}

static int check_norm(const void* Y, gdn_strides ys, const void* Z, const float* w_post,
                      const void* R, const float* w_pre, float eps, int act, int64_t B, int64_t T,
                      int64_t H, int64_t d, gdn_dtype dtype) {
    GDN_TRY(check_dtype(dtype));
    if (B < 0 || T < 0 || H < 0 || d < 0) return fail(GDN_ERR_ARG, "negative B, T, H or d");
    if (H > 1 && d != 128)
        return fail(GDN_ERR_UNSUPPORTED, "head dim d=%lld (only 128 is built for H > 1)",
                    (long long)d);
    if (d % 8) return fail(GDN_ERR_UNSUPPORTED, "width d=%lld is not a multiple of 8", (long long)d);
    if (H > 128 || d > 16384 || H * d > 16384)
        return fail(GDN_ERR_UNSUPPORTED, "rows of %lld x %lld channels (at most 16384)",
                    (long long)H, (long long)d);
    if (act != GDN_ACT_SIGMOID && act != GDN_ACT_SILU) return fail(GDN_ERR_ARG, "unknown act %d", act);
    if (!(eps > 0.f)) return fail(GDN_ERR_ARG, "eps must be positive");
    if (B > kMaxRows || T > kMaxRows || B * T > kMaxRows) return fail(GDN_ERR_ARG, "too many rows");
    if (B == 0 || T == 0 || H == 0 || d == 0) return GDN_OK;
    GDN_TRY(check_ptrs({{Y, "Y"}}));
    GDN_TRY(check_strides(ys, dtype, "Y"));
    GDN_TRY(check_opt_ptr(Z, "Z"));
    GDN_TRY(check_opt_ptr(w_post, "w_post"));
    GDN_TRY(check_opt_ptr(R, "R"));
    return check_opt_ptr(w_pre, "w_pre");
}

int gdn_block_norm(const void* Y, gdn_strides ys, const void* Z, const float* w_post,
                   const void* R, const float* w_pre, float scale, float eps, int act, void* X,
                   void* N, int64_t B, int64_t T, int64_t H, int64_t d, gdn_dtype dtype,
                   void* stream) {
    GDN_TRY(check_norm(Y, ys, Z, w_post, R, w_pre, eps, act, B, T, H, d, dtype));
    if (B == 0 || T == 0 || H == 0 || d == 0) return GDN_OK;
    if (!X && !N) return fail(GDN_ERR_ARG, "X and N are both NULL");
    if (!w_pre != !N) return fail(GDN_ERR_ARG, "w_pre and N go together");
    GDN_TRY(check_opt_ptr(X, "X"));
    GDN_TRY(check_opt_ptr(N, "N"));
    GDN_TRY(check_apart({{X, "X"}, {N, "N"}},
                        {{Y, "Y"}, {Z, "Z"}, {w_post, "w_post"}, {w_pre, "w_pre"}}));
    GDN_TRY(check_apart({{N, "N"}}, {{R, "R"}}));
    const int64_t el = dtype == GDN_BF16 ? 2 : 4, all = B * T * H * d * el;
    GDN_TRY(check_memory({flat(X, all, "X"), flat(N, all, "N")},
                         {strided(Y, ys, B, H, T, d, el, "Y"), flat(Z, all, "Z"),
                          flat(R == X ? nullptr : R, all, "R"), flat(w_post, H * d * 4, "w_post"),
                          flat(w_pre, H * d * 4, "w_pre")}));
    gdn::NormArgs a;
    memset(&a, 0, sizeof a);
    a.Y = Y; a.ys = ys; a.Z = Z; a.w_post = w_post; a.R = R; a.w_pre = w_pre;
    a.scale = scale; a.eps = eps; a.act = act; a.X = X; a.N = N;
    a.B = B; a.T = T; a.H = H; a.d = d;
    return launched(gdn::launch_block_norm(a, dtype == GDN_BF16, (cudaStream_t)stream),
                    "block norm");
}

int64_t gdn_block_norm_backward_workspace_bytes(int64_t B, int64_t T, int64_t H, int64_t d) {
    if (B < 0 || T < 0 || H < 0 || d < 0 || d % 8 || H > 128 || d > 16384 || H * d > 16384 ||
        B > kMaxRows || T > kMaxRows || B * T > kMaxRows)
        return -1;
    if (B * T == 0 || H * d == 0) return 0;
    return gdn::block_norm_ws_bytes(B * T, H * d);
}

int gdn_block_norm_backward(const void* Y, gdn_strides ys, const void* Z, const float* w_post,
                            const void* R, const float* w_pre, const void* dX, const void* dN,
                            float scale, float eps, int act, void* dY, gdn_strides dys, void* dZ,
                            void* dR, float* dw_post, float* dw_pre, void* workspace,
                            int64_t workspace_bytes, int64_t B, int64_t T, int64_t H, int64_t d,
                            gdn_dtype dtype, void* stream) {
    GDN_TRY(check_norm(Y, ys, Z, w_post, R, w_pre, eps, act, B, T, H, d, dtype));
    if (!Z != !dZ) return fail(GDN_ERR_ARG, "Z and dZ go together");
    if (!w_post != !dw_post) return fail(GDN_ERR_ARG, "w_post and dw_post go together");
    if (!w_pre != !dw_pre || !w_pre != !dN)
        return fail(GDN_ERR_ARG, "w_pre, dN and dw_pre go together");
    if (!R && dR) return fail(GDN_ERR_ARG, "dR without R");
    GDN_TRY(check_opt_ptr(dw_post, "dw_post"));
    GDN_TRY(check_opt_ptr(dw_pre, "dw_pre"));
    cudaStream_t st = (cudaStream_t)stream;
    if (B == 0 || T == 0 || H == 0 || d == 0) {        // no rows: the weights' gradients are zero
        const size_t bytes = (size_t)(H * d) * 4;
        for (float* w : {dw_post, dw_pre})
            if (w && bytes) {
                const cudaError_t e = cudaMemsetAsync(w, 0, bytes, st);
                if (e != cudaSuccess) return cuda_fail(e, "zero weight gradients");
            }
        return GDN_OK;
    }
    if (!dX && !dN) return fail(GDN_ERR_ARG, "dX and dN are both NULL");
    GDN_TRY(check_ptrs({{dY, "dY"}}));
    GDN_TRY(check_strides(dys, dtype, "dY"));
    GDN_TRY(check_out_strides(dys, B, H, T, d, "dY"));
    GDN_TRY(check_opt_ptr(dX, "dX"));
    GDN_TRY(check_opt_ptr(dN, "dN"));
    GDN_TRY(check_opt_ptr(dZ, "dZ"));
    GDN_TRY(check_opt_ptr(dR, "dR"));
    const int64_t need = w_post || w_pre ? gdn::block_norm_ws_bytes(B * T, H * d) : 0;
    if (workspace_bytes < need)
        return fail(GDN_ERR_ARG, "workspace of %lld bytes is below the %lld needed",
                    (long long)workspace_bytes, (long long)need);
    if (need > 0) GDN_TRY(check_ptrs({{workspace, "workspace"}}));
    GDN_TRY(check_apart({{dY, "dY"}, {dZ, "dZ"}, {dR, "dR"}, {dw_post, "dw_post"},
                         {dw_pre, "dw_pre"}},
                        {{Y, "Y"}, {Z, "Z"}, {w_post, "w_post"}, {R, "R"}, {w_pre, "w_pre"},
                         {dN, "dN"}}));
    GDN_TRY(check_apart({{dY, "dY"}, {dZ, "dZ"}}, {{dX, "dX"}}));
    const int64_t el = dtype == GDN_BF16 ? 2 : 4, all = B * T * H * d * el, w = H * d * 4;
    GDN_TRY(check_memory({strided(dY, dys, B, H, T, d, el, "dY"), flat(dZ, all, "dZ"),
                          flat(dR, all, "dR"), flat(dw_post, w, "dw_post"),
                          flat(dw_pre, w, "dw_pre"), flat(workspace, need, "workspace")},
                         {strided(Y, ys, B, H, T, d, el, "Y"), flat(Z, all, "Z"),
                          flat(w_post, w, "w_post"), flat(R, all, "R"), flat(w_pre, w, "w_pre"),
                          flat(dX == dR ? nullptr : dX, all, "dX"), flat(dN, all, "dN")}));
    gdn::NormArgs a;
    memset(&a, 0, sizeof a);
    a.Y = Y; a.ys = ys; a.Z = Z; a.w_post = w_post; a.R = R; a.w_pre = w_pre;
    a.scale = scale; a.eps = eps; a.act = act; a.dX = dX; a.dN = dN;
    a.dY = dY; a.dys = dys; a.dZ = dZ; a.dR = dR; a.dw_post = dw_post; a.dw_pre = dw_pre;
    a.ws = (float*)workspace;
    a.B = B; a.T = T; a.H = H; a.d = d;
    return launched(gdn::launch_block_norm_backward(a, dtype == GDN_BF16, st),
                    "block norm backward", w_post || w_pre ? 2 : 1);
}

int gdn_get_status(void* stream) {
    cudaStream_t st = (cudaStream_t)stream;
    cudaError_t e = cudaStreamSynchronize(st);
    if (e != cudaSuccess) return cuda_fail(e, "stream synchronise");
    int v = 0;
    e = cudaMemcpyFromSymbol(&v, gdn::g_status, sizeof(int));
    if (e != cudaSuccess) return cuda_fail(e, "read status");
    const int z = 0;
    e = cudaMemcpyToSymbol(gdn::g_status, &z, sizeof(int));
    if (e != cudaSuccess) return cuda_fail(e, "clear status");
    if (v & gdn::kStatusTimeout) return fail(GDN_ERR_TIMEOUT, "a bounded device wait ran out");
    if (v & gdn::kStatusIndex)
        return fail(GDN_ERR_ARG, "a slot or a sequence bound in device memory is out of range");
    if (v) return fail(GDN_ERR_CUDA, "device status bits 0x%x", v);
    return GDN_OK;
}

int gdn_debug_arm_wait_expiry(int tile, int load, double timeout_ms) {
    if (tile < 0) return fail(GDN_ERR_ARG, "tile=%d is negative", tile);
    if (load != 0 && load != 1) return fail(GDN_ERR_ARG, "load=%d is neither 0 (K) nor 1 (V)", load);
    if (!(timeout_ms > 0.0 && timeout_ms <= 2000.0))
        return fail(GDN_ERR_ARG, "timeout_ms=%g outside (0, 2000]", timeout_ms);
    if (!gdn::tc_available()) return fail(GDN_ERR_UNSUPPORTED, "tensor-core path not built");
    gdn::arm_wait_expiry(tile, load, (unsigned long long)(timeout_ms * 1e6));
    return GDN_OK;
}

int gdn_debug_arm_linear_expiry(int block, int kernel, double timeout_ms) {
    if (block < 0) return fail(GDN_ERR_ARG, "block=%d is negative", block);
    if (kernel != 0 && kernel != 1)
        return fail(GDN_ERR_ARG, "kernel=%d is neither 0 (outputs) nor 1 (states)", kernel);
    if (!(timeout_ms > 0.0 && timeout_ms <= 2000.0))
        return fail(GDN_ERR_ARG, "timeout_ms=%g outside (0, 2000]", timeout_ms);
    gdn::arm_linear_expiry(block, kernel == 1, (unsigned long long)(timeout_ms * 1e6));
    return GDN_OK;
}

const char* gdn_last_error(void) { return t_last_error.c_str(); }

int64_t gdn_launch_count(void) { return t_launches; }

}  // extern "C"

// Device address of the status word for kernels in other translation units.
namespace gdn {
void record_error(int code, const char* msg) {
    (void)code;
    t_last_error = msg;
}

int sm_count() {
    static int sms_of[64] = {0};                       // per device, looked up once
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
        (void)cudaGetLastError();
        return 148;
    }
    if (sms_of[dev]) return sms_of[dev];
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) {
        (void)cudaGetLastError();
        return 148;
    }
    return sms_of[dev] = n;
}

int* status_ptr() {
    static thread_local int dev = -1;
    static thread_local int* ptr = nullptr;
    int cur = 0;
    cudaGetDevice(&cur);
    if (cur != dev || !ptr) {
        void* p = nullptr;
        if (cudaGetSymbolAddress(&p, g_status) != cudaSuccess) return nullptr;
        ptr = (int*)p;
        dev = cur;
    }
    return ptr;
}
}  // namespace gdn
