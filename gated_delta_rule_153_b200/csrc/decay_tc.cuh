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

// Two fp32 operations in one instruction.
GDN_DEV void fma2(float& d0, float& d1, float a0, float a1, float b0, float b1, float c0, float c1) {
    asm("{\n .reg .b64 a, b, c;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n mov.b64 c, {%6, %7};\n"
        " fma.rn.f32x2 c, a, b, c;\n mov.b64 {%0, %1}, c;\n}\n"
        : "=f"(d0), "=f"(d1) : "f"(a0), "f"(a1), "f"(b0), "f"(b1), "f"(c0), "f"(c1));
}
GDN_DEV void mul2(float& d0, float& d1, float a0, float a1, float b0, float b1) {
    asm("{\n .reg .b64 a, b;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n"
        " mul.rn.f32x2 a, a, b;\n mov.b64 {%0, %1}, a;\n}\n"
        : "=f"(d0), "=f"(d1) : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}
GDN_DEV void add2f(float& d0, float& d1, float a0, float a1, float b0, float b1) {
    asm("{\n .reg .b64 a, b;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n"
        " add.rn.f32x2 a, a, b;\n mov.b64 {%0, %1}, a;\n}\n"
        : "=f"(d0), "=f"(d1) : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}

// 2^x; results below 2^-126 are zero.
GDN_DEV float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The gates of a chunk: the inclusive cumsum of log2(e) g over its tokens, as an
// unevaluated sum of two floats, so that the decay of a pair of tokens is exact to
// fp32 however long the cumsum.  Tokens past the sequence repeat the last value.
struct alignas(16) Gates {
    float2 G[CT];
};

// One warp: the gates of a chunk of L <= 128 tokens; lane l holds tokens 4l .. 4l+3.
// g points at the chunk's first token's gate, tokens `stride` apart.
GDN_DEV void load_gates(float (&x)[4], const float* g, size_t stride, int L) {
    const int t = 4 * (threadIdx.x & 31);
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = t + j < L ? g[(size_t)(t + j) * stride] : 0.f;
}
// (a, b) <- a + b in two floats each: the rounding error of the high parts' sum
// (exact, from the difference of what went in and what came out) joins the low.
GDN_DEV float2 add2(float2 a, float2 b) {
    const float s = a.x + b.x, v = s - a.x;
    const float e = ((a.x - (s - v)) + (b.x - v)) + (a.y + b.y);
    const float hi = s + e;
    return make_float2(hi, e - (hi - s));
}
GDN_DEV float diff2(float2 a, float2 b) { return (a.x - b.x) + (a.y - b.y); }

// From token j to token i of a chunk, j <= i.
GDN_DEV float pair_decay(float2 gi, float2 gj) { return ex2(diff2(gi, gj)); }
// From the chunk's start to token i.
GDN_DEV float start_decay(float2 gi) { return ex2(gi.x) * fmaf(gi.y, 0.693147182f, 1.f); }

GDN_DEV void form_gates(Gates& s, const float (&x)[4]) {
    const int lane = threadIdx.x & 31;
    float2 c[4];  // sums within the lane
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        // e^g below 2^-400 is zero in fp32 as it is; -inf would not survive a difference
        const float g = x[j] < -277.f ? -277.f : x[j];
        const float hi = g * 1.44269502f;
        c[j] = make_float2(hi, fmaf(g, 1.44269502f, -hi) + g * 1.92596299e-8f);
        if (j > 0) c[j] = add2(c[j], c[j - 1]);
    }
    float2 run = c[3];  // over this lane and those before it
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const float2 y = make_float2(__shfl_up_sync(0xffffffffu, run.x, o), __shfl_up_sync(0xffffffffu, run.y, o));
        if (lane >= o) run = add2(run, y);
    }
    float2 before = make_float2(__shfl_up_sync(0xffffffffu, run.x, 1), __shfl_up_sync(0xffffffffu, run.y, 1));
    if (lane == 0) before = make_float2(0.f, 0.f);
#pragma unroll
    for (int j = 0; j < 4; ++j) s.G[4 * lane + j] = add2(c[j], before);
}

// What packing left of x and y, packed.
GDN_DEV uint32_t rest_bf16(uint32_t packed, float x, float y) {
    const float2 f = unpack_bf16(packed);
    return pack_bf16(x - f.x, y - f.y);
}

// x and y as sums of TERMS bf16 values each (2 terms: to 2^-16, 3: to 2^-24),
// packed as (x, y) per term.
template <int TERMS>
GDN_DEV void split_bf16(uint32_t (&t)[TERMS], float x, float y) {
#pragma unroll
    for (int i = 0; i < TERMS; ++i) {
        t[i] = pack_bf16(x, y);
        if (i + 1 < TERMS) {
            const float2 f = unpack_bf16(t[i]);
            add2f(x, y, x, y, -f.x, -f.y);
        }
    }
}

// The upper halves of two fp32 values, packed, and their lower halves; and back.
GDN_DEV uint2 halves(float x, float y) {
    return make_uint2(__byte_perm(__float_as_uint(x), __float_as_uint(y), 0x7632),
                      __byte_perm(__float_as_uint(x), __float_as_uint(y), 0x5410));
}
GDN_DEV float2 join_halves(uint32_t up, uint32_t low) {
    return make_float2(__uint_as_float(__byte_perm(low, up, 0x5410)), __uint_as_float(__byte_perm(low, up, 0x7632)));
}
// What the upper halves, read as bf16 values, leave of the values: 16 bits, as two bf16
// terms, exactly.
GDN_DEV void split_rest(uint32_t& t2, uint32_t& t3, uint32_t up, uint32_t low) {
    const float2 x = join_halves(up, low), t1 = unpack_bf16(up);
    const float a = x.x - t1.x, b = x.y - t1.y;
    t2 = pack_bf16(a, b);
    const float2 f = unpack_bf16(t2);
    t3 = pack_bf16(a - f.x, b - f.y);
}

// Zeros of any sign while every bf16 of the x so far was finite, else NaN in one half or both.
GDN_DEV uint32_t seen_bf16(uint32_t x, uint32_t so_far) {
    asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(so_far) : "r"(x), "r"(0u));
    return so_far;
}
GDN_DEV bool all_finite(uint32_t seen) { return (seen & 0x7fff7fffu) == 0; }

// Where a chain's values first were not finite, per channel and for the earliest of them, in
// tokens from the chain's start as it is walked.  Such a value belongs to its own token's
// result and to later ones; in a product over all of a tile's tokens its zero weight
// would make the earlier ones NaN too, so it goes into the product as zero, and the
// results from its token on are made NaN (also where +-inf would be exact).
constexpr int kNever = 0x7fffffff;
constexpr uint32_t kNaN = 0x7fc00000u;
template <int N>
struct FirstBad {
    int at[N], any;
    GDN_DEV void none(int tid) {
        if (tid < N) at[tid] = kNever;
        if (tid == 0) any = kNever;
    }
    GDN_DEV void mark(int channel, int pos) {
        atomicMin(&at[channel], pos);
        atomicMin(&any, pos);
    }
};

// A bounded wait (1 s) in few instructions: these kernels run five roles' loops side by
// side, and their footprint in the instruction cache counts.  The caller reports a wait
// that gave up once, after its loop.
GDN_DEV bool wait_for(uint64_t* bar, uint32_t parity) {
    uint64_t t0 = 0;
    while (!mbar_try(bar, parity)) {
        const uint64_t t = globaltimer();
        if (!t0) t0 = t;
        if (t - t0 > kWaitNs) return false;
    }
    return true;
}

// One lane of a converged warp, chosen so that the compiler knows the branch to
// be the whole warp's: the products behind it take their operands from uniform
// registers (M = 128, N = 64: 48 cycles each against 56 behind lane == 0).
GDN_DEV bool elect_one() {
    uint32_t p;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
    return p != 0;
}

// wait_for by a whole warp with one answer for all its lanes, whose next
// instructions (tensor-memory loads, shuffles) need them together.
GDN_DEV bool warp_wait(uint64_t* bar, uint32_t parity) { return __all_sync(0xffffffffu, wait_for(bar, parity)); }

GDN_DEV unsigned char* align1k(unsigned char* p) {
    return reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(p) + 1023) & ~uintptr_t(1023));
}

}  // namespace decay
}  // namespace gdn
