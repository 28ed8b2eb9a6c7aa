// decay_tc.cuh -- pieces shared by the tensor-core kernels of linear attention
// with a decay per head: chunk positions, the gate vectors of a chunk, and the
// split of an fp32 value into bf16 terms.
#pragma once

#include "async.cuh"
#include "common.cuh"
#include "decay.h"
#include "tc5.cuh"
#include "tma.cuh"

namespace gdn {
namespace decay {

constexpr int CT = 128;  // tokens per chunk of the tensor-core kernels

// What the products of a chunk need of its gates.  G is the inclusive cumsum of
// log2(e) g over the chunk, formed in fp64 and kept as a pair of floats: the
// decay of a pair of tokens is then exact to fp32 however long the cumsum.
// Decays between 32-token blocks factor into one of the row and one of the
// column about the end of the block before the row's; both are at most 1.
struct alignas(16) Gates {
    float2 G[CT];        // high and low part
    float in[CT];        // scale e^{G_i}: from the state entering the chunk to token i
    float out[CT];       // e^{G_last - G_j}: from token j to the chunk's end (zero past its tokens)
    float row[CT];       // scale e^{G_i - G_b}, b = the last token before i's block (rows of block 0 unused)
    float col[3][96];    // [block - 1][j] e^{G_b - G_j}, j <= b
    float total;         // e^{G_last}
    double scratch[CT];
};

// One warp: the gates of a chunk of L <= 128 tokens; lane l holds tokens 4l ..
// 4l+3.  g points at the chunk's first token's gate, tokens `stride` apart.
GDN_DEV void load_gates(float (&x)[4], const float* g, size_t stride, int L) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int t = 4 * lane + j;
        x[j] = t < L ? g[(size_t)t * stride] : 0.f;
    }
}
GDN_DEV void form_gates(Gates& s, const float (&x)[4], int L, float scale, bool pairs) {
    const int lane = threadIdx.x & 31;
    double c[4], run = 0.0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        // e^g below 2^-400 is zero in fp32 as it is; -inf would not survive a difference
        const double y = (double)x[j] * 1.4426950408889634;
        run += y < -400.0 ? -400.0 : y;
        c[j] = run;
    }
    double before = run;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const double y = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += y;
    }
    const double last = __shfl_sync(0xffffffffu, before, 31);
    before -= run;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int t = 4 * lane + j;
        c[j] += before;
        const float hi = (float)c[j];
        s.G[t] = make_float2(hi, (float)(c[j] - (double)hi));
        s.in[t] = scale * exp2f((float)c[j]);
        s.out[t] = t < L ? exp2f((float)(last - c[j])) : 0.f;
        s.scratch[t] = c[j];
    }
    if (lane == 0) s.total = exp2f((float)last);
    __syncwarp();
    if (pairs) {
        const int b = lane / 8;  // this lane's tokens are all of block b
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (b > 0) s.row[4 * lane + j] = scale * exp2f((float)(c[j] - s.scratch[32 * b - 1]));
#pragma unroll
        for (int k = 1; k < 4; ++k) {
            const double base = s.scratch[32 * k - 1];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (b < k) s.col[k - 1][4 * lane + j] = exp2f((float)(base - c[j]));
        }
    }
}

// Decay between two tokens of one block, from their pairs.
GDN_DEV float pair_decay(float2 gi, float2 gj) { return exp2f((gi.x - gj.x) + (gi.y - gj.y)); }

// x and y as sums of TERMS bf16 values each (2 terms: to 2^-16, 3: to 2^-24),
// packed as (x, y) per term.
template <int TERMS>
GDN_DEV void split_bf16(uint32_t (&t)[TERMS], float x, float y) {
#pragma unroll
    for (int i = 0; i < TERMS; ++i) {
        t[i] = pack_bf16(x, y);
        if (i + 1 < TERMS) {
            const float2 f = unpack_bf16(t[i]);
            x -= f.x;
            y -= f.y;
        }
    }
}

// mbar_wait by a whole warp with one answer for all its lanes, whose next
// instructions (tensor-memory loads, shuffles) need them together.
GDN_DEV bool warp_wait(uint64_t* bar, uint32_t parity, unsigned int* status) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, status));
}

GDN_DEV unsigned char* align1k(unsigned char* p) {
    return reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(p) + 1023) & ~uintptr_t(1023));
}

}  // namespace decay
}  // namespace gdn
