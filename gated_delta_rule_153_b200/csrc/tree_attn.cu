// tree_attn.cu -- softmax attention for a tree of drafted tokens over a paged
// cache, and the append of the accepted path to it: the softmax layers' side of
// draft-tree verification ("TreeWY: Speculative Verification for Gated DeltaNet
// Hybrids", the "Linked reviews" entry of the "Gated Delta Networks: Improving
// Mamba2 with Delta Rule" review page), beside gdn_tree_verify / gdn_tree_commit.
//
// Node i of sequence n stands at position len[n] + depth(i) and sees the cached
// positions p < len[n], its ancestors and itself; with a window w > 0 only
// those less than w positions back (itself always).  Per query head
//     o_i = sum_p softmax_p(scale q_i . k_p) v_p.
#include <math.h>

#include "checks.h"
#include "common.cuh"
#include "mma.cuh"

namespace gdn {
namespace {

constexpr int kMaxNodes = 64;

struct Cache {
    const __nv_bfloat16 *k, *v;  // [pages][page][Hkv][d]
    const int* table;            // [N][width]
    const int* len;              // [N]
    int pages, page, width;
};

// Cached tokens of sequence n; a length that the table cannot hold counts as none.
GDN_DEV int cached(const Cache& c, int n, unsigned int* status) {
    const int len = c.len[n];
    if (len < 0 || (long long)len > (long long)c.width * c.page) {
        if (status) atomicOr(status, 2u);
        return 0;
    }
    return len;
}

GDN_DEV int parent_of(const int* parent, int i, unsigned int* status) {
    const int p = parent[i];
    if (p < -1 || p >= i) {
        if (status) atomicOr(status, 2u);
        return -1;
    }
    return p;
}

// One warp per (sequence, node, query head); a lane holds D / 32 channels.
template <int D>
__global__ void __launch_bounds__(128)
tree_attn_kernel(int N, int M, int Hq, int Hkv, float scale, int window, const int* __restrict__ parent,
                 const __nv_bfloat16* __restrict__ q, const __nv_bfloat16* __restrict__ k,
                 const __nv_bfloat16* __restrict__ v, Cache c, __nv_bfloat16* __restrict__ o,
                 unsigned int* status) {
    constexpr int E = D / 32;
    const long long w = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
    if (w >= (long long)N * M * Hq) return;
    const int lane = threadIdx.x & 31;
    const int h = (int)(w % Hq), i = (int)(w / Hq % M), n = (int)(w / Hq / M), kh = h / (Hq / Hkv);
    float qr[E], acc[E], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        qr[e] = scale * __bfloat162float(q[(size_t)w * D + lane * E + e]);
        acc[e] = 0.f;
    }
    auto take = [&](const __nv_bfloat16* kr, const __nv_bfloat16* vr) {
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) s += qr[e] * __bfloat162float(kr[lane * E + e]);
        s = warp_sum(s);
        const float mn = fmaxf(m, s);
        const float a = m == -INFINITY ? 0.f : expf(m - mn), p = expf(s - mn);
        l = a * l + p;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = a * acc[e] + p * __bfloat162float(vr[lane * E + e]);
        m = mn;
    };
    const int* par = parent + (size_t)n * M;
    int depth = 0;
    for (int j = parent_of(par, i, status); j >= 0; j = parent_of(par, j, status)) ++depth;
    const int len = cached(c, n, status);
    const long long far = window > 0 ? (long long)len + depth - window + 1 : 0;
    for (int p = far > 0 ? (int)min(far, (long long)len) : 0; p < len; ++p) {
        const int pg = c.table[(size_t)n * c.width + p / c.page];
        if (pg < 0 || pg >= c.pages) {
            if (status) atomicOr(status, 2u);
            continue;
        }
        const size_t at = (((size_t)pg * c.page + p % c.page) * Hkv + kh) * D;
        take(c.k + at, c.v + at);
    }
    int back = 0;
    for (int j = i; j >= 0; j = parent_of(par, j, status), ++back) {
        if (window > 0 && back >= window) break;
        const size_t at = (((size_t)n * M + j) * Hkv + kh) * D;
        take(k + at, v + at);
    }
#pragma unroll
    for (int e = 0; e < E; ++e) o[(size_t)w * D + lane * E + e] = __float2bfloat16_rn(acc[e] / l);
}

// ---- append ------------------------------------------------------------------
// One CTA per sequence: the accepted node's root path, then its K and V rows to
// the cache positions after the last, in 16-byte pieces.
__global__ void __launch_bounds__(256)
tree_append_kernel(int M, int row16, const int* __restrict__ parent, const int* __restrict__ accepted,
                   const uint4* __restrict__ k, const uint4* __restrict__ v, uint4* __restrict__ kc,
                   uint4* __restrict__ vc, Cache c, int* __restrict__ new_len, unsigned int* status) {
    __shared__ int path[kMaxNodes], count, len;
    __shared__ long long dst[kMaxNodes];
    const int n = blockIdx.x, tid = threadIdx.x;
    if (tid == 0) {
        int a = accepted[n], d = 0;
        if (a < -1 || a >= M) {
            if (status) atomicOr(status, 2u);
            a = -1;
        }
        for (int j = a; j >= 0; j = parent_of(parent + (size_t)n * M, j, status)) path[d++] = j;  // leaf to root
        len = c.len[n];
        if (len < 0 || (long long)len + d > (long long)c.width * c.page) {
            if (status) atomicOr(status, 2u);
            d = 0;
        }
        count = d;
    }
    __syncthreads();
    const int d = count;
    bool bad = false;
    if (tid < d) {
        const int p = len + tid, pg = c.table[(size_t)n * c.width + p / c.page];
        bad = pg < 0 || pg >= c.pages;
        dst[tid] = (long long)pg * c.page + p % c.page;
    }
    if (__syncthreads_or(bad)) {  // a page that does not exist: this sequence stays as it is
        if (tid == 0) {
            if (status) atomicOr(status, 2u);
            new_len[n] = len;
        }
        return;
    }
    for (int e = tid; e < d * row16; e += 256) {
        const int t = e / row16, x = e % row16;
        const size_t src = ((size_t)n * M + path[d - 1 - t]) * row16 + x, to = (size_t)dst[t] * row16 + x;
        kc[to] = k[src];
        vc[to] = v[src];
    }
    if (tid == 0) new_len[n] = len + d;
}

gdn_status check(int N, int M, int Hq, int Hkv, int d, gdn_dtype dtype, int pages, int page, int width) {
    if (N < 1 || M < 1 || Hkv < 1 || Hq < 1 || Hq % Hkv || pages < 1 || width < 1) return GDN_ERR_INVALID_ARG;
    if (dtype != GDN_BF16 && dtype != GDN_F32) return GDN_ERR_INVALID_ARG;
    if ((long long)N * M * Hq > 0x7fffffffLL || (long long)pages * page > 0x7fffffffLL) return GDN_ERR_INVALID_ARG;
    if ((long long)width * page > 0x7fffffffLL - kMaxNodes) return GDN_ERR_INVALID_ARG;
    if (M > kMaxNodes || dtype != GDN_BF16 || (d != 64 && d != 128)) return GDN_ERR_UNSUPPORTED;
    if (page != 16 && page != 32 && page != 64 && page != 128) return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}

gdn_status launched() { return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA; }

}  // namespace
}  // namespace gdn

using namespace gdn;

extern "C" {

size_t gdn_tree_attn_workspace(int N, int M, int Hq, int Hkv, int d, gdn_dtype dtype, int page, int width) {
    if (check(N, M, Hq, Hkv, d, dtype, 1, page, width) != GDN_OK) return 0;
    return kStatusBytes;
}

gdn_status gdn_tree_attn(int N, int M, int Hq, int Hkv, int d, gdn_dtype dtype, float scale, int window,
                         const int* parent, const void* q, const void* k, const void* v, int pages, int page,
                         int width, const void* k_cache, const void* v_cache, const int* block_table,
                         const int* cache_len, void* o, void* ws, size_t ws_bytes, gdn_stream_t stream) {
    const gdn_status s = check(N, M, Hq, Hkv, d, dtype, pages, page, width);
    if (s != GDN_OK) return s;
    if (!isfinite(scale) || window < 0) return GDN_ERR_INVALID_ARG;
    if (!parent || !q || !k || !v || !k_cache || !v_cache || !block_table || !cache_len || !o)
        return GDN_ERR_INVALID_ARG;
    if (!all_aligned_to(16, {q, k, v, k_cache, v_cache, o}) || !all_aligned_to(4, {parent, block_table, cache_len}))
        return GDN_ERR_INVALID_ARG;
    const size_t need = gdn_tree_attn_workspace(N, M, Hq, Hkv, d, dtype, page, width);
    if (!ws || ws_bytes < need || !aligned_to(ws, 256)) return GDN_ERR_WORKSPACE;
    const size_t nm = (size_t)N * M, pool = (size_t)pages * page * Hkv * d * 2;
    if (outputs_overlap({{parent, nm * 4}, {q, nm * Hq * d * 2}, {k, nm * Hkv * d * 2}, {v, nm * Hkv * d * 2},
                         {k_cache, pool}, {v_cache, pool}, {block_table, (size_t)N * width * 4}, {cache_len, (size_t)N * 4}},
                        {{o, nm * Hq * d * 2}, {ws, need}}))
        return GDN_ERR_INVALID_ARG;
    cudaStream_t st = (cudaStream_t)stream;
    cudaGetLastError();
    if (cudaMemsetAsync(ws, 0, sizeof(unsigned int), st) != cudaSuccess) return GDN_ERR_CUDA;
    const Cache c{(const __nv_bfloat16*)k_cache, (const __nv_bfloat16*)v_cache, block_table, cache_len, pages, page, width};
    const unsigned grid = (unsigned)(((long long)N * M * Hq + 3) / 4);
    auto go = [&](auto dd) {
        GDN_LAUNCH("tree_attn", st, (tree_attn_kernel<decltype(dd)::value><<<grid, 128, 0, st>>>(
            N, M, Hq, Hkv, scale, window, parent, (const __nv_bfloat16*)q, (const __nv_bfloat16*)k,
            (const __nv_bfloat16*)v, c, (__nv_bfloat16*)o, (unsigned int*)ws)));
    };
    if (d == 64) go(std::integral_constant<int, 64>{});
    else go(std::integral_constant<int, 128>{});
    return launched();
}

gdn_status gdn_tree_append(int N, int M, int Hkv, int d, gdn_dtype dtype, const int* parent, const int* accepted,
                           const void* k, const void* v, int pages, int page, int width, void* k_cache,
                           void* v_cache, const int* block_table, const int* cache_len, int* new_len,
                           unsigned int* status, gdn_stream_t stream) {
    const gdn_status s = check(N, M, Hkv, Hkv, d, dtype, pages, page, width);
    if (s != GDN_OK) return s;
    if (!parent || !accepted || !k || !v || !k_cache || !v_cache || !block_table || !cache_len || !new_len)
        return GDN_ERR_INVALID_ARG;
    if (!all_aligned_to(16, {k, v, k_cache, v_cache}) ||
        !all_aligned_to(4, {parent, accepted, block_table, cache_len, new_len, status}))
        return GDN_ERR_INVALID_ARG;
    const size_t nm = (size_t)N * M, pool = (size_t)pages * page * Hkv * d * 2;
    // new_len may be cache_len itself: the length is read before it is written
    if (outputs_overlap({{parent, nm * 4}, {accepted, (size_t)N * 4}, {k, nm * Hkv * d * 2}, {v, nm * Hkv * d * 2},
                         {block_table, (size_t)N * width * 4}, {new_len == cache_len ? nullptr : cache_len, (size_t)N * 4}},
                        {{k_cache, pool}, {v_cache, pool}, {new_len, (size_t)N * 4}, {status, 4}}))
        return GDN_ERR_INVALID_ARG;
    cudaStream_t st = (cudaStream_t)stream;
    cudaGetLastError();
    const Cache c{(const __nv_bfloat16*)k_cache, (const __nv_bfloat16*)v_cache, block_table, cache_len, pages, page, width};
    GDN_LAUNCH("tree_append", st, (tree_append_kernel<<<(unsigned)N, 256, 0, st>>>(
        M, Hkv * d / 8, parent, accepted, (const uint4*)k, (const uint4*)v, (uint4*)k_cache, (uint4*)v_cache, c,
        new_len, status)));
    return launched();
}

}  // extern "C"
