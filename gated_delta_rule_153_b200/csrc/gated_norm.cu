// gated_norm.cu -- the layer's output norm and gate, forward and backward.
//
// Per token and head, over the d channels of the head (channels last):
//     c = x - mean (centred form) or x,  h = c / sqrt(mean(c^2) + eps),
//     y = w h s(z),   s(z) = z sigmoid(z).
// Backward, with e = dy w s(z):
//     dx = (e - h mean(e h) [- mean(e)]) / sqrt(mean(c^2) + eps),
//     dz = dy w h sigmoid(z) (1 + z (1 - sigmoid(z))),   dw = sum dy h s(z).
// Each tensor is read or written once, in 16-byte pieces: LPR lanes hold a row
// and reduce it with shuffles.  At 131,072 rows of 128 channels in bf16 the forward takes
// 21 us and the backward 32 us, 4.9 and 5.2 TB/s (75 and 80 % of the measured HBM rate), with
// half of the issue slots used: the rest is the start and the end of the one wave of CTAs
// and the latency of rows of which a warp has one turn on its way.  The sum of dw takes 7 us,
// a launch of few CTAs.
//
// The rows are dealt to `units` (groups of LPR lanes) in turn, unit u taking
// rows u, u + U, ... with U a multiple of the heads: neighbouring units read
// neighbouring rows, and a unit's head, and so its slice of w, never changes.  A
// unit therefore sums its dw in registers; a second kernel adds the units of a
// head (for a shared w, first within the CTA, then over the CTAs) in a fixed order.
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "checks.h"
#include "common.cuh"
#include "decay_tc.cuh"
#include "mma.cuh"

namespace gdn {
namespace {

using decay::add2f;
using decay::fma2;
using decay::mul2;

constexpr int NT = 256;

// 16 bytes of a row, as loaded and as fp32.
GDN_DEV void widen(float* v, const uint4& r, __nv_bfloat16) {
    const uint32_t x[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = unpack_bf16(x[i]);
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
    }
}
GDN_DEV void widen(float* v, const uint4& r, float) {
    v[0] = __uint_as_float(r.x); v[1] = __uint_as_float(r.y);
    v[2] = __uint_as_float(r.z); v[3] = __uint_as_float(r.w);
}
// 1 / (1 + e^-z).  For bf16 the fast exponential and quotient, whose error (2^-18 where
// the result is not small) is far below the rounding of the result.
GDN_DEV float sigmoid(float z, float) { return 1.f / (1.f + expf(-z)); }
GDN_DEV float sigmoid(float z, __nv_bfloat16) { return __fdividef(1.f, 1.f + __expf(-z)); }
GDN_DEV void store16(__nv_bfloat16* p, const float* v) {
    __stcs(reinterpret_cast<uint4*>(p), make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                                                   pack_bf16(v[6], v[7])));
}
GDN_DEV void store16(float* p, const float* v) {
    __stcs(reinterpret_cast<float4*>(p), make_float4(v[0], v[1], v[2], v[3]));
}

template <int LPR>
GDN_DEV float row_sum(float x) {
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// Shapes of a row: VEC channels per 16 bytes, LPR lanes, NV pieces per lane.
template <typename T, int D>
struct Row {
    static constexpr int VEC = 16 / sizeof(T), LPR = D / VEC < 32 ? D / VEC : 32, NV = D / (VEC * LPR), CPL = VEC * NV;
    static constexpr int UPC = NT / LPR;  // units per CTA
};

template <typename T, int D, bool CENTER, bool BWD>
__global__ void __launch_bounds__(NT, 4)
gated_norm_kernel(long long rows, int H, int wheads, long long U, float eps, const T* __restrict__ x,
                  const T* __restrict__ z, const float* __restrict__ w, const T* __restrict__ dy,
                  T* __restrict__ out, T* __restrict__ dz, float* __restrict__ part) {
    using R = Row<T, D>;
    const int sub = threadIdx.x % R::LPR;
    const long long unit = (long long)blockIdx.x * R::UPC + threadIdx.x / R::LPR;
    const int wh = wheads == 1 ? 0 : (int)(unit % H);
    float wr[R::CPL], dw[R::CPL];
#pragma unroll
    for (int j = 0; j < R::CPL; ++j) {
        wr[j] = w[wh * D + (j / R::VEC * R::LPR + sub) * R::VEC + j % R::VEC];
        dw[j] = 0.f;
    }
    uint4 nx[R::NV], nz[R::NV], ng[R::NV];
    auto fetch = [&](long long r) {
        const bool in = unit < U && r < rows;
#pragma unroll
        for (int p = 0; p < R::NV; ++p) {
            const size_t at = (size_t)(in ? r : 0) * D + (p * R::LPR + sub) * R::VEC;
            nx[p] = __ldcs(reinterpret_cast<const uint4*>(x + at));
            nz[p] = __ldcs(reinterpret_cast<const uint4*>(z + at));
            if constexpr (BWD) ng[p] = __ldcs(reinterpret_cast<const uint4*>(dy + at));
        }
    };
    // every lane of a warp runs the same number of turns: the shuffles need them all
    const long long first = (long long)blockIdx.x * R::UPC + (threadIdx.x / 32) * (32 / R::LPR);
    if (first < rows) fetch(unit);
    for (long long base = 0; base + first < rows; base += U) {
        const long long r = base + unit;
        const bool in = unit < U && r < rows;
        float xv[R::CPL], zv[R::CPL], g[R::CPL];
#pragma unroll
        for (int p = 0; p < R::NV; ++p) {
            widen(xv + p * R::VEC, nx[p], T());
            widen(zv + p * R::VEC, nz[p], T());
            if constexpr (BWD) widen(g + p * R::VEC, ng[p], T());
        }
        if (base + U + first < rows) fetch(r + U);  // the next turn's rows are on their way
        if constexpr (CENTER) {
            float mean = 0.f;
#pragma unroll
            for (int j = 0; j < R::CPL; ++j) mean += xv[j];
            mean = row_sum<R::LPR>(mean) * (-1.f / D);
#pragma unroll
            for (int j = 0; j < R::CPL; j += 2) add2f(xv[j], xv[j + 1], xv[j], xv[j + 1], mean, mean);
        }
        float s0 = 0.f, s1 = 0.f;
#pragma unroll
        for (int j = 0; j < R::CPL; j += 2) fma2(s0, s1, xv[j], xv[j + 1], xv[j], xv[j + 1], s0, s1);
        const float rs = rsqrtf(row_sum<R::LPR>(s0 + s1) * (1.f / D) + eps);
        float e0 = 0.f, e1 = 0.f, t0 = 0.f, t1 = 0.f;
#pragma unroll
        for (int j = 0; j < R::CPL; j += 2) {  // (pairs: two operations to an instruction)
            float h0, h1, a0, a1;
            const float g0 = sigmoid(zv[j], T()), g1 = sigmoid(zv[j + 1], T());
            mul2(h0, h1, xv[j], xv[j + 1], rs, rs);
            mul2(a0, a1, zv[j], zv[j + 1], g0, g1);
            if constexpr (BWD) {
                float w0, w1, p0, p1, q0, q1;
                mul2(w0, w1, g[j], g[j + 1], wr[j], wr[j + 1]);           // dy w
                mul2(p0, p1, g[j], g[j + 1], h0, h1);                     // dy h
                if (in) fma2(dw[j], dw[j + 1], p0, p1, a0, a1, dw[j], dw[j + 1]);
                // s'(z) = sigmoid + s (1 - sigmoid)
                fma2(q0, q1, a0, a1, -g0, -g1, a0, a1);
                add2f(q0, q1, q0, q1, g0, g1);
                mul2(p0, p1, w0, w1, h0, h1);
                mul2(zv[j], zv[j + 1], p0, p1, q0, q1);
                mul2(w0, w1, w0, w1, a0, a1);                             // e
                fma2(e0, e1, w0, w1, h0, h1, e0, e1);
                if constexpr (CENTER) add2f(t0, t1, t0, t1, w0, w1);
                xv[j] = h0; xv[j + 1] = h1;
                g[j] = w0; g[j + 1] = w1;
            } else {
                mul2(h0, h1, h0, h1, wr[j], wr[j + 1]);
                mul2(xv[j], xv[j + 1], h0, h1, a0, a1);
            }
        }
        if constexpr (BWD) {
            const float eh = row_sum<R::LPR>(e0 + e1) * (-1.f / D);
            const float es = CENTER ? row_sum<R::LPR>(t0 + t1) * (-1.f / D) : 0.f;
#pragma unroll
            for (int j = 0; j < R::CPL; j += 2) {
                fma2(xv[j], xv[j + 1], xv[j], xv[j + 1], eh, eh, g[j], g[j + 1]);
                if constexpr (CENTER) add2f(xv[j], xv[j + 1], xv[j], xv[j + 1], es, es);
                mul2(xv[j], xv[j + 1], xv[j], xv[j + 1], rs, rs);
            }
        }
        if (!in) continue;
#pragma unroll
        for (int p = 0; p < R::NV; ++p) {
            const size_t at = (size_t)r * D + (p * R::LPR + sub) * R::VEC;
            store16(out + at, xv + p * R::VEC);
            if constexpr (BWD) store16(dz + at, zv + p * R::VEC);
        }
    }
    if constexpr (BWD) {
        if (wheads == 1) {  // one sum per CTA, its units in order
            __shared__ float sum[R::UPC][D];
#pragma unroll
            for (int j = 0; j < R::CPL; ++j)
                sum[threadIdx.x / R::LPR][(j / R::VEC * R::LPR + sub) * R::VEC + j % R::VEC] = dw[j];
            __syncthreads();
            for (int c = threadIdx.x; c < D; c += NT) {
                float t = 0.f;
#pragma unroll 8
                for (int u = 0; u < R::UPC; ++u) t += sum[u][c];
                part[(size_t)blockIdx.x * D + c] = t;
            }
        } else if (unit < U) {
#pragma unroll
            for (int j = 0; j < R::CPL; ++j)
                part[unit * D + (j / R::VEC * R::LPR + sub) * R::VEC + j % R::VEC] = dw[j];
        }
    }
}

// dw[h] = sum of the parts u = h, h + heads, ... of U (per unit; for a shared w per CTA,
// heads = 1), 32 sums in parallel per channel, joined in a fixed order.
__global__ void __launch_bounds__(1024)
gated_norm_dw_kernel(long long U, int heads, int D, const float* __restrict__ part, float* __restrict__ dw) {
    __shared__ float s[32][33];
    const int c = blockIdx.y * 32 + threadIdx.x, h = blockIdx.x;
    float sum = 0.f;
#pragma unroll 4
    for (long long u = h + (long long)threadIdx.y * heads; u < U; u += 32ll * heads) sum += part[u * D + c];
    s[threadIdx.y][threadIdx.x] = sum;
    __syncthreads();
    const float t = warp_sum(s[threadIdx.x][threadIdx.y]);
    if (threadIdx.x == 0) dw[h * D + blockIdx.y * 32 + threadIdx.y] = t;
}

// Units of a call: four CTAs per SM, in whole turns of the heads, and no more than
// there are rows.
long long units(long long rows, int H, int lpr) {
    const long long fill = 148ll * 4 * (NT / lpr);
    return std::max<long long>(std::min(rows, fill) / H, 1) * H;
}

int lanes_per_row(gdn_dtype t, int d) { return std::min(32, d * (t == GDN_BF16 ? 2 : 4) / 16); }

template <bool BWD>
gdn_status run(long long rows, int H, int d, int wheads, gdn_dtype dtype, int center, float eps, const void* x,
               const void* z, const float* w, const void* dy, void* out, void* dz, float* part, cudaStream_t st) {
    auto go = [&](auto t, auto dd, auto cc) {
        using T = decltype(t);
        constexpr int D = decltype(dd)::value;
        constexpr bool C = decltype(cc)::value;
        using R = Row<T, D>;
        const long long U = units(rows, H, R::LPR);
        const unsigned grid = (unsigned)((U + R::UPC - 1) / R::UPC);
        GDN_LAUNCH(BWD ? "gated_norm_bwd" : "gated_norm_fwd", st, (gated_norm_kernel<T, D, C, BWD><<<grid, NT, 0, st>>>(
            rows, H, wheads, U, eps, (const T*)x, (const T*)z, w, (const T*)dy, (T*)out, (T*)dz, part)));
    };
    auto by_center = [&](auto t, auto dd) {
        if (center) go(t, dd, std::true_type{});
        else go(t, dd, std::false_type{});
    };
    auto by_dim = [&](auto t) {
        switch (d) {
            case 32: by_center(t, std::integral_constant<int, 32>{}); break;
            case 64: by_center(t, std::integral_constant<int, 64>{}); break;
            case 128: by_center(t, std::integral_constant<int, 128>{}); break;
            default: by_center(t, std::integral_constant<int, 256>{}); break;
        }
    };
    if (dtype == GDN_BF16) by_dim(__nv_bfloat16{});
    else by_dim(float{});
    return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

gdn_status check(long long rows, int H, int d, int wheads, gdn_dtype dtype, float eps) {
    if (rows < 1 || H < 1 || rows % H || (wheads != 1 && wheads != H)) return GDN_ERR_INVALID_ARG;
    if (rows > (1ll << 40) || H > (1 << 20)) return GDN_ERR_INVALID_ARG;
    if (dtype != GDN_BF16 && dtype != GDN_F32) return GDN_ERR_INVALID_ARG;
    if (!isfinite(eps) || eps < 0.f) return GDN_ERR_INVALID_ARG;
    if (d != 32 && d != 64 && d != 128 && d != 256) return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}

}  // namespace
}  // namespace gdn

using namespace gdn;

extern "C" {

gdn_status gdn_gated_norm_fwd(long long rows, int H, int d, int wheads, gdn_dtype dtype, int center, float eps,
                              const void* x, const void* z, const float* w, void* y, gdn_stream_t stream) {
    const gdn_status s = check(rows, H, d, wheads, dtype, eps);
    if (s != GDN_OK) return s;
    if (!x || !z || !w || !y) return GDN_ERR_INVALID_ARG;
    if (!all_aligned_to(16, {x, z, y}) || !aligned_to(w, 4)) return GDN_ERR_INVALID_ARG;
    const size_t n = (size_t)rows * d * (dtype == GDN_BF16 ? 2 : 4);
    if (outputs_overlap({{x, n}, {z, n}, {w, (size_t)wheads * d * 4}}, {{y, n}})) return GDN_ERR_INVALID_ARG;
    cudaGetLastError();
    return run<false>(rows, H, d, wheads, dtype, center, eps, x, z, w, nullptr, y, nullptr, nullptr,
                      (cudaStream_t)stream);
}

size_t gdn_gated_norm_bwd_workspace(long long rows, int H, int d, gdn_dtype dtype) {
    if (check(rows, H, d, 1, dtype, 0.f) != GDN_OK) return 0;
    return (size_t)units(rows, H, lanes_per_row(dtype, d)) * d * 4;
}

gdn_status gdn_gated_norm_bwd(long long rows, int H, int d, int wheads, gdn_dtype dtype, int center, float eps,
                              const void* x, const void* z, const float* w, const void* dy, void* dx, void* dz,
                              float* dw, void* ws, size_t ws_bytes, gdn_stream_t stream) {
    gdn_status s = check(rows, H, d, wheads, dtype, eps);
    if (s != GDN_OK) return s;
    if (!x || !z || !w || !dy || !dx || !dz || !dw) return GDN_ERR_INVALID_ARG;
    if (!all_aligned_to(16, {x, z, dy, dx, dz}) || !all_aligned_to(4, {w, dw})) return GDN_ERR_INVALID_ARG;
    const size_t need = gdn_gated_norm_bwd_workspace(rows, H, d, dtype);
    if (!ws || ws_bytes < need || !aligned_to(ws, 256)) return GDN_ERR_WORKSPACE;
    const size_t n = (size_t)rows * d * (dtype == GDN_BF16 ? 2 : 4), nw = (size_t)wheads * d * 4;
    if (outputs_overlap({{x, n}, {z, n}, {dy, n}, {w, nw}}, {{dx, n}, {dz, n}, {dw, nw}, {ws, need}}))
        return GDN_ERR_INVALID_ARG;
    cudaStream_t st = (cudaStream_t)stream;
    cudaGetLastError();
    s = run<true>(rows, H, d, wheads, dtype, center, eps, x, z, w, dy, dx, dz, (float*)ws, st);
    if (s != GDN_OK) return s;
    const int lpr = lanes_per_row(dtype, d), upc = NT / lpr;
    long long U = units(rows, H, lpr);
    if (wheads == 1) U = (U + upc - 1) / upc;
    GDN_LAUNCH("gated_norm_dw", st, (gated_norm_dw_kernel<<<dim3((unsigned)wheads, d / 32), dim3(32, 32), 0, st>>>(
        U, wheads, d, (const float*)ws, dw)));
    return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // extern "C"
