// kd_glr.hip -- element-wise gated linear recurrence and its backward pass, gfx950.
//
// Per batch element b and channel c, with the state h in fp32:
//     h_t = f_t h_{t-1} + i_t x_t          (i_t = 1 without an input gate)
// and, for L = <dh, h> + <dhT, h_T>, walking back with m = dL/dh_t from the
// tokens after t:
//     g_t = dh_t + m;  dx_t = i_t g_t;  di_t = x_t g_t;  df_t = g_t h_{t-1};  m = f_t g_t
// and dh0 = the last m.
#include "kd_device.h"

namespace kd {

constexpr int GLR_CHUNK = 128;   // tokens between two kept states (KRON_DELTA_GLR_CHUNK)

// One thread per (b, channel), token by token.
template <class E, bool GATE>
__global__ __launch_bounds__(64) void kd_glr_fwd_kernel(const E* __restrict__ x, const E* __restrict__ f,
                                                        const E* __restrict__ gi, const float* __restrict__ h0,
                                                        E* __restrict__ h, float* __restrict__ hT,
                                                        float* __restrict__ hs, int T, int D)
{
    const int c = blockIdx.x * 64 + threadIdx.x, b = blockIdx.y;
    if (c >= D) return;
    const int nc = (T + GLR_CHUNK - 1) / GLR_CHUNK;
    float s = h0 ? h0[(size_t)b * D + c] : 0.f;
    for (int t = 0; t < T; ++t) {
        const size_t at = ((size_t)b * T + t) * D + c;
        if (hs && t % GLR_CHUNK == 0) hs[((size_t)b * nc + t / GLR_CHUNK) * D + c] = s;
        const float u = GATE ? (float)gi[at] * (float)x[at] : (float)x[at];
        s = fmaf((float)f[at], s, u);
        h[at] = (E)s;
    }
    if (hT) hT[(size_t)b * D + c] = s;
}

template <class E, bool GATE>
__global__ __launch_bounds__(64) void kd_glr_bwd_kernel(const E* __restrict__ x, const E* __restrict__ f,
                                                        const E* __restrict__ gi, const float* __restrict__ hs,
                                                        const E* __restrict__ dh, const float* __restrict__ dhT,
                                                        E* __restrict__ dx, E* __restrict__ df, E* __restrict__ di,
                                                        float* __restrict__ dh0, int T, int D)
{
    const int c = blockIdx.x * 64 + threadIdx.x, b = blockIdx.y;
    if (c >= D) return;
    const int nc = (T + GLR_CHUNK - 1) / GLR_CHUNK;
    float m = dhT ? dhT[(size_t)b * D + c] : 0.f;
    for (int k = nc - 1; k >= 0; --k) {
        const int t0 = k * GLR_CHUNK, n = min(GLR_CHUNK, T - t0);
        const size_t base = ((size_t)b * T + t0) * D + c;
        float hp[GLR_CHUNK];   // the state before each token of the chunk
        float s = hs[((size_t)b * nc + k) * D + c];
        for (int t = 0; t < n; ++t) {
            const size_t at = base + (size_t)t * D;
            hp[t] = s;
            s = fmaf((float)f[at], s, GATE ? (float)gi[at] * (float)x[at] : (float)x[at]);
        }
        for (int t = n - 1; t >= 0; --t) {
            const size_t at = base + (size_t)t * D;
            const float g = (float)dh[at] + m;
            if (GATE) {
                dx[at] = (E)((float)gi[at] * g);
                di[at] = (E)((float)x[at] * g);
            } else {
                dx[at] = (E)g;
            }
            df[at] = (E)(g * hp[t]);
            m = (float)f[at] * g;
        }
    }
    if (dh0) dh0[(size_t)b * D + c] = m;
}

// One token of every row: y = h' = f h + i x, with h' kept in fp32.
template <class E, bool GATE>
__global__ __launch_bounds__(256) void kd_glr_step_kernel(const E* __restrict__ x, const E* __restrict__ f,
                                                          const E* __restrict__ gi, const float* h_in,
                                                          E* __restrict__ y, float* h_out, int64_t n)
{
    const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (at >= n) return;
    const float u = GATE ? (float)gi[at] * (float)x[at] : (float)x[at];
    const float s = fmaf((float)f[at], h_in[at], u);
    y[at] = (E)s;
    h_out[at] = s;
}

template <class E>
static hipError_t glr_fwd(const void* x, const void* f, const void* gi, const float* h0, void* h, float* hT,
                          float* hs, int B, int T, int D, hipStream_t st)
{
    const dim3 grid((D + 63) / 64, B);
    if (gi)
        kd_glr_fwd_kernel<E, true><<<grid, 64, 0, st>>>((const E*)x, (const E*)f, (const E*)gi, h0, (E*)h, hT, hs, T, D);
    else
        kd_glr_fwd_kernel<E, false><<<grid, 64, 0, st>>>((const E*)x, (const E*)f, nullptr, h0, (E*)h, hT, hs, T, D);
    return hipGetLastError();
}

template <class E>
static hipError_t glr_bwd(const void* x, const void* f, const void* gi, const float* hs, const void* dh,
                          const float* dhT, void* dx, void* df, void* di, float* dh0, int B, int T, int D,
                          hipStream_t st)
{
    const dim3 grid((D + 63) / 64, B);
    if (gi)
        kd_glr_bwd_kernel<E, true><<<grid, 64, 0, st>>>((const E*)x, (const E*)f, (const E*)gi, hs, (const E*)dh, dhT,
                                                       (E*)dx, (E*)df, (E*)di, dh0, T, D);
    else
        kd_glr_bwd_kernel<E, false><<<grid, 64, 0, st>>>((const E*)x, (const E*)f, nullptr, hs, (const E*)dh, dhT,
                                                        (E*)dx, (E*)df, nullptr, dh0, T, D);
    return hipGetLastError();
}

template <class E>
static hipError_t glr_step(const void* x, const void* f, const void* gi, const float* h_in, void* y, float* h_out,
                           int64_t n, hipStream_t st)
{
    const unsigned grid = (unsigned)((n + 255) / 256);
    if (gi)
        kd_glr_step_kernel<E, true><<<grid, 256, 0, st>>>((const E*)x, (const E*)f, (const E*)gi, h_in, (E*)y, h_out, n);
    else
        kd_glr_step_kernel<E, false><<<grid, 256, 0, st>>>((const E*)x, (const E*)f, nullptr, h_in, (E*)y, h_out, n);
    return hipGetLastError();
}

size_t glr_workspace_bytes(int, int, int, int) { return 0; }

hipError_t launch_glr_fwd(int bf16, const void* x, const void* f, const void* gi, const float* h0, void* h, float* hT,
                          float* hs, void* ws, int B, int T, int D, hipStream_t st)
{
    (void)ws;
    return bf16 ? glr_fwd<__bf16>(x, f, gi, h0, h, hT, hs, B, T, D, st)
                : glr_fwd<float>(x, f, gi, h0, h, hT, hs, B, T, D, st);
}

hipError_t launch_glr_bwd(int bf16, const void* x, const void* f, const void* gi, const float* hs, const void* dh,
                          const float* dhT, void* dx, void* df, void* di, float* dh0, void* ws, int B, int T, int D,
                          hipStream_t st)
{
    (void)ws;
    return bf16 ? glr_bwd<__bf16>(x, f, gi, hs, dh, dhT, dx, df, di, dh0, B, T, D, st)
                : glr_bwd<float>(x, f, gi, hs, dh, dhT, dx, df, di, dh0, B, T, D, st);
}

hipError_t launch_glr_step(int bf16, const void* x, const void* f, const void* gi, const float* h_in, void* y,
                           float* h_out, int64_t n, hipStream_t st)
{
    return bf16 ? glr_step<__bf16>(x, f, gi, h_in, y, h_out, n, st) : glr_step<float>(x, f, gi, h_in, y, h_out, n, st);
}

}  // namespace kd
