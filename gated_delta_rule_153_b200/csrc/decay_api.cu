// decay_api.cu -- host side of gdn_decay_*: argument checks, workspace sizes and
// the choice of kernels.
#include <math.h>

#include "checks.h"
#include "common.cuh"
#include "decay.h"

using namespace gdn;
using namespace gdn::decay;

namespace {

bool dim_ok(int d) { return d == 16 || d == 32 || d == 64 || d == 128; }

gdn_status check(const gdn_decay_dims* d, const int* cu, int nseq, Problem& p) {
    if (!d) return GDN_ERR_INVALID_ARG;
    if (d->B < 1 || d->T < 1 || d->H < 1 || d->Hk < 1 || d->H % d->Hk) return GDN_ERR_INVALID_ARG;
    if (d->dtype != GDN_BF16 && d->dtype != GDN_F32) return GDN_ERR_INVALID_ARG;
    if (!isfinite(d->scale)) return GDN_ERR_INVALID_ARG;
    if (nseq < 0 || (nseq == 0) != (cu == nullptr) || (nseq && d->B != 1)) return GDN_ERR_INVALID_ARG;
    if (!aligned_to(cu, 4)) return GDN_ERR_INVALID_ARG;
    // token, chain and chunk-slot numbers are 32-bit
    const long long rows = (long long)d->B * d->T, seqs = nseq ? nseq : d->B;
    if (rows > 0x7fffffffLL || seqs * d->H > 0x7fffffffLL || rows / 64 + seqs > 0x7fffffffLL / d->H)
        return GDN_ERR_INVALID_ARG;
    if (!dim_ok(d->dk) || !dim_ok(d->dv)) return GDN_ERR_UNSUPPORTED;
    p.seq = Seqs{cu, (int)seqs, d->T, (int)rows};
    p.H = d->H; p.Hk = d->Hk; p.dk = d->dk; p.dv = d->dv;
    p.dtype = d->dtype; p.scale = d->scale;
    return GDN_OK;
}

struct Bytes {
    size_t qk, v, g, state, cu;
};
Bytes bytes_of(const Problem& p) {
    const size_t e = p.dtype == GDN_BF16 ? 2 : 4, rows = p.seq.rows;
    return Bytes{rows * p.Hk * p.dk * e, rows * p.H * p.dv * e, rows * p.H * 4,
                 (size_t)p.seq.nseq * p.H * p.dk * p.dv * 4, p.seq.cu ? ((size_t)p.seq.nseq + 1) * 4 : 0};
}

gdn_status check_ws(const void* ws, size_t ws_bytes, size_t need) {
    return !ws || ws_bytes < need || !aligned_to(ws, 256) ? GDN_ERR_WORKSPACE : GDN_OK;
}

gdn_status launched() { return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA; }

size_t fwd_need(const Problem& p) { return tc_supported(p) ? tc_fwd_workspace(p) : simt_fwd_workspace(p); }
size_t bwd_need(const Problem& p) { return tc_supported(p) ? tc_bwd_workspace(p) : simt_bwd_workspace(p); }

// The workspace queries take no offsets: any non-null pointer stands for them.
const int* const kSomeOffsets = reinterpret_cast<const int*>(4);

}  // namespace

extern "C" {

size_t gdn_decay_fwd_workspace(const gdn_decay_dims* d, int nseq) {
    Problem p;
    return check(d, nseq > 0 ? kSomeOffsets : nullptr, nseq, p) == GDN_OK ? fwd_need(p) : 0;
}

size_t gdn_decay_bwd_workspace(const gdn_decay_dims* d, int nseq) {
    Problem p;
    return check(d, nseq > 0 ? kSomeOffsets : nullptr, nseq, p) == GDN_OK ? bwd_need(p) : 0;
}

gdn_status gdn_decay_fwd(const gdn_decay_dims* d, const int* cu_seqlens, int nseq, const void* q, const void* k,
                         const void* v, const float* g, const float* h0, void* o, float* hT, void* ws,
                         size_t ws_bytes, gdn_stream_t stream) {
    Problem p;
    gdn_status s = check(d, cu_seqlens, nseq, p);
    if (s != GDN_OK) return s;
    if (!q || !k || !v || !g || !o) return GDN_ERR_INVALID_ARG;
    if (!all_aligned_to(16, {q, k, v, g, h0, o, hT})) return GDN_ERR_INVALID_ARG;
    const size_t need = fwd_need(p);
    const Bytes b = bytes_of(p);
    if ((s = check_ws(ws, ws_bytes, need)) != GDN_OK) return s;
    if (outputs_overlap({{q, b.qk}, {k, b.qk}, {v, b.v}, {g, b.g}, {h0, b.state}, {cu_seqlens, b.cu}},
                        {{o, b.v}, {hT, b.state}, {ws, need}}))
        return GDN_ERR_INVALID_ARG;
    cudaStream_t st = (cudaStream_t)stream;
    cudaGetLastError();
    if (cudaMemsetAsync(ws, 0, sizeof(unsigned int), st) != cudaSuccess) return GDN_ERR_CUDA;
    if (tc_supported(p)) {
        if (!launch_tc_fwd(p, q, k, v, g, h0, o, hT, ws, st)) return GDN_ERR_CUDA;
    } else {
        launch_simt_fwd(p, q, k, v, g, h0, o, hT, ws, st);
    }
    return launched();
}

gdn_status gdn_decay_bwd(const gdn_decay_dims* d, const int* cu_seqlens, int nseq, const void* q, const void* k,
                         const void* v, const float* g, const float* h0, const void* dO, const float* dhT,
                         void* dq, void* dk, void* dv, float* dg, float* dh0, void* ws, size_t ws_bytes,
                         gdn_stream_t stream) {
    Problem p;
    gdn_status s = check(d, cu_seqlens, nseq, p);
    if (s != GDN_OK) return s;
    if (!q || !k || !v || !g || !dO || !dq || !dk || !dv || !dg) return GDN_ERR_INVALID_ARG;
    if ((h0 == nullptr) != (dh0 == nullptr)) return GDN_ERR_INVALID_ARG;
    if (!all_aligned_to(16, {q, k, v, g, h0, dO, dhT, dq, dk, dv, dg, dh0})) return GDN_ERR_INVALID_ARG;
    const size_t need = bwd_need(p);
    const Bytes b = bytes_of(p);
    if ((s = check_ws(ws, ws_bytes, need)) != GDN_OK) return s;
    if (outputs_overlap({{q, b.qk}, {k, b.qk}, {v, b.v}, {g, b.g}, {h0, b.state}, {dO, b.v}, {dhT, b.state},
                         {cu_seqlens, b.cu}},
                        {{dq, b.qk}, {dk, b.qk}, {dv, b.v}, {dg, b.g}, {dh0, b.state}, {ws, need}}))
        return GDN_ERR_INVALID_ARG;
    cudaStream_t st = (cudaStream_t)stream;
    cudaGetLastError();
    if (cudaMemsetAsync(ws, 0, sizeof(unsigned int), st) != cudaSuccess) return GDN_ERR_CUDA;
    if (tc_supported(p)) {
        if (!launch_tc_bwd(p, q, k, v, g, h0, dO, dhT, dq, dk, dv, dg, dh0, ws, st)) return GDN_ERR_CUDA;
    } else {
        launch_simt_bwd(p, q, k, v, g, h0, dO, dhT, dq, dk, dv, dg, dh0, ws, st);
    }
    return launched();
}

gdn_status gdn_decay_step(int N, int H, int Hk, int dk, int dv, gdn_dtype dtype, float scale, const void* q,
                          const void* k, const void* v, const float* g, float* state, void* o,
                          gdn_stream_t stream) {
    if (N < 1 || H < 1 || Hk < 1 || H % Hk || (long long)N * H > 0x7fffffffLL) return GDN_ERR_INVALID_ARG;
    if (dtype != GDN_BF16 && dtype != GDN_F32) return GDN_ERR_INVALID_ARG;
    if (!isfinite(scale)) return GDN_ERR_INVALID_ARG;
    if (!dim_ok(dk) || !dim_ok(dv)) return GDN_ERR_UNSUPPORTED;
    if (!q || !k || !v || !g || !state || !o) return GDN_ERR_INVALID_ARG;
    if (!all_aligned_to(16, {q, k, v, state, o}) || !aligned_to(g, 4)) return GDN_ERR_INVALID_ARG;
    const size_t e = dtype == GDN_BF16 ? 2 : 4, nh = (size_t)N * H;
    if (outputs_overlap({{q, (size_t)N * Hk * dk * e}, {k, (size_t)N * Hk * dk * e}, {v, nh * dv * e}, {g, nh * 4}},
                        {{state, nh * dv * dk * 4}, {o, nh * dv * e}}))
        return GDN_ERR_INVALID_ARG;
    cudaGetLastError();
    launch_decay_step(N, H, Hk, dk, dv, dtype, scale, q, k, v, g, state, o, (cudaStream_t)stream);
    return launched();
}

}  // extern "C"
