// decay.cu -- linear attention with a decay per head in fp32 arithmetic on
// CUDA cores, by tiles of 32 tokens: the path of GDN_F32 and of the head dims the
// tensor-core kernels do not take; and the single-token step.
//
// The recurrence per (sequence, head), with a_t = e^{g_t}:
//     S_t = a_t S_{t-1} + v_t k_t^T,   o_t = S_t (scale q_t).
// The walk below is written for a general one,
//     R <- a R + y_t w_t^T,   out_t = c R x_t,
// because every gradient is another instance of it:
//     o : x = q,  w = k,  y = v    forwards,  from h0
//     dq: x = dO, w = v,  y = k    forwards,  from h0^T      (R = S^T)
//     dk: x = v,  w = dO, y = q    backwards, from dhT^T     (R = dS^T)
//     dv: x = k,  w = q,  y = dO   backwards, from dhT       (R = dS)
// Backwards, the decay between tokens t+1 and t is a_{t+1}.  scale goes with
// the out of the first two and with y of dk and w of dv.
//
// Gate gradient.  Let M_ji be what the pair of tokens j < i adds to <dO, o>
// (h0 counts as a token before the first, dhT as one after the last).  The
// decay of token t acts on the pairs j < t <= i, so within a chunk that ends
// after token e
//     dg_t = sum_{t <= i <= e} (q_i.dq'_i - k_i.dk'_i) + <S_e, dS_e>,
// where dq', dk' leave out the token's own pair.  The last term is taken from
// the states at each chunk's end, so the sums stay 64 tokens long: taken over
// a whole sequence instead, their rounding would grow with its length.
//
// Tiles of 32 tokens are taken at once.  With G the cumsum of the gates from the tile's
// start, D_ts the decay between tokens t and s, and R what enters the tile,
//     out_t = c (f_t R x_t + sum_s D_ts (w_s.x_t) y_s),   R <- e^{G_last} R + sum_s h_s y_s w_s^T
// over s <= t, with f = e^G and h = e^{G_last - G} forwards, and over s >= t, with the two
// exchanged, backwards.  All of it is small matrix products in fp32 on CUDA cores, from
// shared memory in register tiles (2 x 2 and 4 x 4 with 256 threads); a CTA holds
// 64 rows of R.  What bounds it is the issue of fp32 FMAs and, 1.5 to 2 times as long, the
// shared-memory loads that feed them (a 16-byte load takes four cycles of the SM's 128
// bytes per cycle, whatever its lanes share): about 6,700 of them per tile of 64 x 64 dims.
// Forward, 32 x 1024 tokens of 8 heads: 285 us at 64 x 64 dims, 1,017 us at 128 x 128.
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "decay.h"
#include "decay_tc.cuh"

namespace gdn {
namespace decay {
namespace {

constexpr int TT = 32;          // tokens per tile
constexpr int kRows = 64;       // rows of R per CTA at most
constexpr int AC = 64;          // tokens per chunk of the gate gradient

// A gate of -inf (or one so low that e^g is zero in fp32) is a reset.
GDN_DEV float decay_of(float g) { return expf(g); }

struct Operand {
    const void* p;
    int heads, rep, dim;  // heads of the tensor, value heads per head, channels
};
GDN_DEV size_t row_of(const Operand& a, long long tok, int h) {
    return ((size_t)tok * a.heads + h / a.rep) * a.dim;
}

struct Walk {
    Operand x, w, y, z;     // z (gate gradient): dotted with out
    const float* g;
    const float* init;      // [nseq, H, .., ..] or null
    bool init_t;            // init is stored [column][row]
    float* last;            // final state [row][column], or null
    void* out;              // [token][H][RD] in T, or in fp32 when out_f32
    bool out_f32;
    float c_out, c_y;
    Seqs seq;
    int H, RD;
    float* anchor;          // [slot][H][RD][CD] states at chunk ends: written forwards, read backwards
    float* dots;            // [row block][token][H]: sum over this CTA's rows of z . out' (own pair left out)
    float* cross;           // [row block][slot][H]: <S_e, dS_e> over this CTA's rows
    // Few chains are cut into runs of `len` tiles: first what each run adds to a zero R
    // and its decay (MAP), then all runs at once, each from what the ones before leave.
    int runs, len;
    bool wide;              // at most one CTA per SM: 256 threads
    float *runR, *runA;     // [item][H][RD][CD] and [item][H]
    unsigned int* status;
};

// Four consecutive values.
template <typename T>
struct Four;
template <>
struct Four<float> {
    using Raw = float4;
    GDN_DEV static float4 of(float4 v) { return v; }
};
template <>
struct Four<__nv_bfloat16> {
    using Raw = uint2;
    GDN_DEV static float4 of(uint2 v) {
        const float2 a = unpack_bf16(v.x), b = unpack_bf16(v.y);
        return make_float4(a.x, a.y, b.x, b.y);
    }
};
GDN_DEV void put4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
GDN_DEV void put4(__nv_bfloat16* p, float4 v) {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
}

template <int CD, int RB, int WT>
struct WalkSmem {  // rows padded by 16 bytes: eight rows of a column are in different banks
    float x[TT][CD + 4], w[TT][CD + 4], y[TT][RB + 4], z[TT][RB + 4], p[TT][TT + 4];
    float r[CD][RB + 4];
    float4 half[2][TT * RB / 4 / WT][WT == 256 && CD < 128 ? WT / 2 : 1];
    float2 g[TT];
    float f[TT], h[TT], own[TT], red[8];
    FirstBad<RB> bad;  // values of y that are not finite
};

// RB rows of R per CTA, WT threads.  16 and 32 rows in all have kernels of their own with
// 128 threads: lanes for 64 would idle (32 x 1024 tokens of 8 heads, 16 x 16 dims: 114 us
// against 175, 128 columns and 16 rows: 329 us against 507).  With 64 rows, 128
// threads have the larger register tiles, and so fewer loads from shared memory per
// product; 256 hide its latency better, with the next tile's rows on their way while this
// one is worked on.  128 columns: 256 where a CTA has an SM to itself (777 tokens of
// 4 heads: 71 us against 95), else 128 (32 x 1024 tokens of 8 heads: 1,010 us against
// 1,304).  Fewer columns: 256 throughout (within 2 % at that size, faster with few CTAs).
template <int CD, int RB, typename T, bool REV, bool MAP, int WT>
__global__ void __launch_bounds__(WT)
decay_walk_kernel(const Walk p) {
    extern __shared__ __align__(16) unsigned char raw[];
    WalkSmem<CD, RB, WT>& s = *reinterpret_cast<WalkSmem<CD, RB, WT>*>(raw);
    using F = Four<T>;
    constexpr int NX = TT * CD / 4 / WT > 0 ? TT * CD / 4 / WT : 1;  // groups of four per thread and tile
    constexpr int LR = RB / 4;                                       // lanes of a row of out
    constexpr int NC = CD * LR / WT > 0 ? CD * LR / WT : 1;          // columns of R per thread
    constexpr int NY = TT * LR / WT, NT = TT * LR / WT;              // rows of y, tokens of out per thread
    constexpr int NP = TT * 16 / WT;                                 // rows of p per thread
    static_assert(NT >= 1, "a thread has a token");
    // 256 threads: two halves of them take half of each sum over channels and tokens, in
    // 4 x 4 tiles, and each finishes half of the tokens (64 x 64 dims, 32 x 1024 tokens of
    // 8 heads: 281 us against 310 in 2 x 4 tiles; with 128 columns, 80 against 77 for 777
    // tokens of 4 heads, so not there)
    constexpr int KS = WT == 256 && CD < 128 ? 2 : 1;
    const int h = blockIdx.x % p.H, r0 = blockIdx.y * RB;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    long long tok0;
    int n, seq, run, first;
    if (!item_of(p.seq, p.runs, p.len * TT, MAP ? 1 : 0, blockIdx.x / p.H, seq, run, first)) return;
    if (!span_of(p.seq, seq, tok0, n)) {
        if (tid == 0) atomicOr(p.status, 2u);
        return;
    }
    const size_t sh = (size_t)seq * p.H + h;
    const long long slot0 = tok0 / AC + seq;
    const int tiles = (n + TT - 1) / TT;
    const int i0 = run * p.len, i1 = min(tiles, i0 + p.len);  // this run, in the order of the walk
    // the run that ends the chain (the first of an empty one) writes the last state
    const bool ends = i1 == tiles && (run == 0 || i0 < tiles);
    if (MAP ? i1 >= tiles : i0 >= tiles && !ends) return;
    // R, column-major; from run 1 on with what the runs before this one leave
#pragma unroll 8
    for (int e = tid; e < CD * RB; e += WT) {
        const int c = p.init_t ? e / RB : e % CD, r = p.init_t ? e % RB : e / CD, row = r0 + r;
        s.r[c][r] = MAP || !p.init || row >= p.RD ? 0.f : __ldg(p.init + (p.init_t ? (sh * CD + c) * p.RD + row : (sh * p.RD + row) * CD + c));
    }
    if (!MAP && run > 0) {
        __syncthreads();
        // R <- prod a_q R + sum_q (prod_{p > q} a_p) N_q
        float f = 1.f, mine[CD * RB / WT];
        const size_t next = (size_t)p.H * p.RD * CD;  // from a run to the next
        const float *a = p.runA + (size_t)first * p.H + h, *from = p.runR + ((size_t)first * p.H + h) * p.RD * CD + r0 * CD;
#pragma unroll
        for (int i = 0; i < CD * RB / WT; ++i) mine[i] = 0.f;
#pragma unroll 1
        for (int q = run - 1; q >= 0; --q, f *= __ldg(a + (size_t)(q + 1) * p.H)) {
#pragma unroll
            for (int i = 0; i < CD * RB / WT; ++i) {
                const int e = tid + WT * i;
                if (r0 + e / CD < p.RD) mine[i] = fmaf(f, __ldg(from + q * next + e), mine[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < CD * RB / WT; ++i) {
            const int e = tid + WT * i;
            s.r[e % CD][e / CD] = fmaf(f, s.r[e % CD][e / CD], mine[i]);
        }
    }
    if (!MAP) s.bad.none(tid);
    float all = 1.f;  // the decay of the run so far
    const bool has_z = !MAP && p.dots != nullptr;
    constexpr bool AHEAD = WT == 256 || (RB < kRows && CD < 128);
    const int r = 4 * (tid % LR), part = KS == 2 ? tid / (WT / KS) : 0;  // this thread's rows of R, and half
    typename F::Raw vx[NX], vw[NX], vy[NY], vz[NY];  // all on their way before any is put down
    float pg = 0.f;
    auto fetch = [&](int it) {
        const int tile = REV ? tiles - 1 - it : it, m = min(TT, n - tile * TT);
        const long long t0 = tok0 + (long long)tile * TT;
        const typename F::Raw zero{};
        auto get = [&](const Operand& o, int t, int c, bool in) {
            return in ? __ldg(reinterpret_cast<const typename F::Raw*>((const T*)o.p + row_of(o, t0 + t, h) + c)) : zero;
        };
        pg = warp == 0 && lane < m ? __ldg(p.g + (size_t)(t0 + lane) * p.H + h) : 0.f;
#pragma unroll
        for (int i = 0; i < NX; ++i) {
            const int e = 4 * (tid + WT * i), t = e / CD, c = e % CD;
            if (!MAP) vx[i] = get(p.x, t, c, t < m);
            vw[i] = get(p.w, t, c, t < m);
        }
#pragma unroll
        for (int i = 0; i < NY; ++i) {
            const int t = tid / LR + WT / LR * i;
            vy[i] = get(p.y, t, r0 + r, t < m && r0 + r < p.RD);
            if (has_z) vz[i] = get(p.z, t, r0 + r, t < m && r0 + r < p.RD);
        }
    };
    auto place = [&](int it, int t) { return (it - i0) * TT + (REV ? TT - 1 - t : t); };  // as the run is walked
    if (AHEAD && i0 < i1) fetch(i0);
    for (int it = i0; it < i1; ++it) {
        const int tile = REV ? tiles - 1 - it : it;
        const int m = min(TT, n - tile * TT);
        const long long t0 = tok0 + (long long)tile * TT;
        const int end = tile * TT + m;
        const bool border = end % AC == 0 || end == n;  // the tile ends a chunk
        const long long slot = slot0 + (end - 1) / AC;
        if (!AHEAD) fetch(it);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < NX; ++i) {
            const int e = 4 * (tid + WT * i), t = e / CD, c = e % CD;
            if (TT * CD / 4 < WT && t >= TT) break;
            if (!MAP) *reinterpret_cast<float4*>(&s.x[t][c]) = F::of(vx[i]);
            *reinterpret_cast<float4*>(&s.w[t][c]) = F::of(vw[i]);
        }
#pragma unroll
        for (int i = 0; i < NY; ++i) {
            const int t = tid / LR + WT / LR * i;
            const float4 v = F::of(vy[i]);
            float4 y = make_float4(p.c_y * v.x, p.c_y * v.y, p.c_y * v.z, p.c_y * v.w);
            if (!(0.f * y.x + 0.f * y.y + 0.f * y.z + 0.f * y.w == 0.f)) {
                float* const e[4] = {&y.x, &y.y, &y.z, &y.w};
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (!(fabsf(*e[j]) < INFINITY)) {
                        *e[j] = MAP ? __uint_as_float(kNaN) : 0.f;
                        if (!MAP) s.bad.mark(r + j, place(it, t));
                    }
            }
            *reinterpret_cast<float4*>(&s.y[t][r]) = y;
            if (has_z) *reinterpret_cast<float4*>(&s.z[t][r]) = F::of(vz[i]);
        }
        if (warp == 0) {  // the gates' cumsum, in two floats
            const float y = pg < -277.f ? -277.f : pg, hi = y * 1.44269502f;
            float2 c = make_float2(hi, fmaf(y, 1.44269502f, -hi) + y * 1.92596299e-8f);
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const float2 u = make_float2(__shfl_up_sync(0xffffffffu, c.x, o), __shfl_up_sync(0xffffffffu, c.y, o));
                if (lane >= o) c = add2(c, u);
            }
            const float2 last = make_float2(__shfl_sync(0xffffffffu, c.x, 31), __shfl_sync(0xffffffffu, c.y, 31));
            const float a = start_decay(c), b = pair_decay(last, c);
            s.g[lane] = c;
            s.f[lane] = REV ? b : a;
            s.h[lane] = REV ? a : b;
        }
        __syncthreads();
        if (AHEAD && it + 1 < i1) fetch(it + 1);
        const int bad = MAP ? kNever : s.bad.any;
        float sum[NT][4];
        auto add = [&](float (&o)[4], float q, const float4& v) {
            o[0] = fmaf(q, v.x, o[0]);
            o[1] = fmaf(q, v.y, o[1]);
            o[2] = fmaf(q, v.z, o[2]);
            o[3] = fmaf(q, v.w, o[3]);
        };
        if constexpr (!MAP) {
            {   // p[t][u] = D_tu (w_u . x_t) for t = tid / 16 + WT / 16 i, u = tid % 16 + 16 j (neighbouring
                // lanes read neighbouring rows, which are in different banks), its diagonal apart;
                // even and odd channels are added up apart
                const int ta = tid / 16, ua = tid % 16;
                float2 a[NP][2] = {};
#pragma unroll 2
                for (int c = 0; c < CD; c += 4) {
                    float4 xv[NP], wv[2];
#pragma unroll
                    for (int i = 0; i < NP; ++i) xv[i] = *reinterpret_cast<const float4*>(&s.x[ta + WT / 16 * i][c]);
#pragma unroll
                    for (int j = 0; j < 2; ++j) wv[j] = *reinterpret_cast<const float4*>(&s.w[ua + 16 * j][c]);
#pragma unroll
                    for (int i = 0; i < NP; ++i)
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            fma2(a[i][j].x, a[i][j].y, xv[i].x, xv[i].y, wv[j].x, wv[j].y, a[i][j].x, a[i][j].y);
                            fma2(a[i][j].x, a[i][j].y, xv[i].z, xv[i].w, wv[j].z, wv[j].w, a[i][j].x, a[i][j].y);
                        }
                }
#pragma unroll
                for (int i = 0; i < NP; ++i)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int t = ta + WT / 16 * i, u = ua + 16 * j;
                        const float d = a[i][j].x + a[i][j].y;
                        if (t == u) s.own[t] = d;
                        const bool in = REV ? u > t : u < t;
                        s.p[t][u] = in ? d * (REV ? pair_decay(s.g[u], s.g[t]) : pair_decay(s.g[t], s.g[u])) : 0.f;
                    }
            }
            __syncthreads();
            // out: KS NT tokens x 4 rows, over this half of the channels and of the tile's tokens
            const int tb = KS * NT * (tid % (WT / KS) / LR);
            float a[KS * NT][4] = {};
#pragma unroll 2
            for (int c = part * (CD / KS); c < (part + 1) * (CD / KS); c += 4) {
                float4 xv[KS * NT], rv[4];
#pragma unroll
                for (int i = 0; i < KS * NT; ++i) xv[i] = *reinterpret_cast<const float4*>(&s.x[tb + i][c]);
#pragma unroll
                for (int i = 0; i < 4; ++i) rv[i] = *reinterpret_cast<const float4*>(&s.r[c + i][r]);
#pragma unroll
                for (int i = 0; i < KS * NT; ++i) {
                    add(a[i], xv[i].x, rv[0]);
                    add(a[i], xv[i].y, rv[1]);
                    add(a[i], xv[i].z, rv[2]);
                    add(a[i], xv[i].w, rv[3]);
                }
            }
#pragma unroll
            for (int i = 0; i < KS * NT; ++i) {
                const float f = s.f[tb + i];
#pragma unroll
                for (int j = 0; j < 4; ++j) a[i][j] *= f;
            }
#pragma unroll 2
            for (int u = part * (TT / KS); u < (part + 1) * (TT / KS); u += 4) {
                float4 pv[KS * NT], yv[4];
#pragma unroll
                for (int i = 0; i < KS * NT; ++i) pv[i] = *reinterpret_cast<const float4*>(&s.p[tb + i][u]);
#pragma unroll
                for (int i = 0; i < 4; ++i) yv[i] = *reinterpret_cast<const float4*>(&s.y[u + i][r]);
#pragma unroll
                for (int i = 0; i < KS * NT; ++i) {
                    add(a[i], pv[i].x, yv[0]);
                    add(a[i], pv[i].y, yv[1]);
                    add(a[i], pv[i].z, yv[2]);
                    add(a[i], pv[i].w, yv[3]);
                }
            }
            // half of the tokens' sums go to the other half's threads, the other half come from them
#pragma unroll
            for (int i = 0; i < NT; ++i) {
#pragma unroll
                for (int j = 0; j < 4; ++j) sum[i][j] = KS == 2 && part ? a[(KS - 1) * NT + i][j] : a[i][j];
                if constexpr (KS == 2) {
                    const int g = (KS - 1) * NT + i;
                    s.half[part][i][tid % (WT / KS)] = part ? make_float4(a[i][0], a[i][1], a[i][2], a[i][3])
                                                            : make_float4(a[g][0], a[g][1], a[g][2], a[g][3]);
                }
            }
        }
        const int c0 = tid / LR * NC;  // this thread's columns of R
        const bool has_r = CD * LR >= WT || c0 < CD;
        if (!MAP && REV && p.cross && border) {
            // R is dS^T at the end of this chunk: dot it with the state there
            float d = 0.f;
            if (has_r && r0 + r < p.RD) {
                const float* A = p.anchor + (((size_t)slot * p.H + h) * p.RD + r0 + r) * CD + c0;
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int c = 0; c < NC; ++c) d += s.r[c0 + c][r + j] * A[(size_t)j * CD + c];
            }
            d = warp_sum(d);
            if (lane == 0) s.red[warp] = d;
        }
        if (!MAP) __syncthreads();
        if (!MAP && REV && p.cross && border && tid == 0) {
            float d = 0.f;
            for (int w = 0; w < WT / 32; ++w) d += s.red[w];
            p.cross[((size_t)blockIdx.y * chunk_slots(p.seq, AC) + slot) * p.H + h] = d;
        }
        if constexpr (!MAP) {
            const int t_out = KS * NT * (tid % (WT / KS) / LR) + part * NT;
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                const int t = t_out + i;
                if constexpr (KS == 2) {
                    const float4 v = s.half[1 - part][i][tid % (WT / KS)];
                    sum[i][0] += v.x; sum[i][1] += v.y; sum[i][2] += v.z; sum[i][3] += v.w;
                }
                if (bad <= place(it, t)) {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (s.bad.at[r + j] <= place(it, t)) sum[i][j] = __uint_as_float(kNaN);
                }
                const size_t row = (size_t)(t0 + t) * p.H + h;
                if (has_z) {
                    const float4 zv = *reinterpret_cast<const float4*>(&s.z[t][r]);
                    float d = zv.x * sum[i][0] + zv.y * sum[i][1] + zv.z * sum[i][2] + zv.w * sum[i][3];
#pragma unroll
                    for (int o = LR / 2; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
                    if (tid % LR == 0 && t < m) p.dots[(size_t)blockIdx.y * p.seq.rows * p.H + row] = p.c_out * d;
                }
                if (t < m && r0 + r < p.RD) {
                    add(sum[i], s.own[t], *reinterpret_cast<const float4*>(&s.y[t][r]));
                    const float4 v = make_float4(p.c_out * sum[i][0], p.c_out * sum[i][1], p.c_out * sum[i][2], p.c_out * sum[i][3]);
                    if (p.out_f32) put4((float*)p.out + row * p.RD + r0 + r, v);
                    else put4((T*)p.out + row * p.RD + r0 + r, v);
                }
            }
        }
        const float total = start_decay(s.g[TT - 1]);
        all *= total;
        if (has_r) {  // R; a thread: NC columns x 4 rows
            float a[NC][4];
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                const float4 v = *reinterpret_cast<const float4*>(&s.r[c0 + c][r]);
                a[c][0] = total * v.x; a[c][1] = total * v.y; a[c][2] = total * v.z; a[c][3] = total * v.w;
            }
#pragma unroll 4
            for (int u = 0; u < TT; ++u) {
                const float4 yv = *reinterpret_cast<const float4*>(&s.y[u][r]);
                const float f = s.h[u], q[4] = {f * yv.x, f * yv.y, f * yv.z, f * yv.w};
                float w[NC];
                if constexpr (NC >= 4) {
#pragma unroll
                    for (int c = 0; c < NC; c += 4) {
                        const float4 v = *reinterpret_cast<const float4*>(&s.w[u][c0 + c]);
                        w[c] = v.x; w[c + 1] = v.y; w[c + 2] = v.z; w[c + 3] = v.w;
                    }
                } else {
#pragma unroll
                    for (int c = 0; c < NC; ++c) w[c] = s.w[u][c0 + c];
                }
#pragma unroll
                for (int c = 0; c < NC; ++c)
#pragma unroll
                    for (int j = 0; j < 4; ++j) a[c][j] = fmaf(w[c], q[j], a[c][j]);
            }
            if (bad < (it - i0 + 1) * TT) {  // y went in without
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (s.bad.at[r + j] != kNever) {
#pragma unroll
                        for (int c = 0; c < NC; ++c) a[c][j] = __uint_as_float(kNaN);
                    }
            }
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                *reinterpret_cast<float4*>(&s.r[c0 + c][r]) = make_float4(a[c][0], a[c][1], a[c][2], a[c][3]);
                if (!MAP && !REV && p.anchor && border && r0 + r < p.RD) {
                    float* A = p.anchor + (((size_t)slot * p.H + h) * p.RD + r0 + r) * CD + c0 + c;
#pragma unroll
                    for (int j = 0; j < 4; ++j) A[(size_t)j * CD] = a[c][j];
                }
            }
        }
    }
    float* const to = MAP ? p.runR + ((size_t)(first + run) * p.H + h) * p.RD * CD : p.last && ends ? p.last + sh * p.RD * CD : nullptr;
    if (to) {
        __syncthreads();
        for (int e = tid; e < CD * RB; e += WT) {
            const int r = e / CD, c = e % CD;
            if (r0 + r < p.RD) to[(size_t)(r0 + r) * CD + c] = s.r[c][r];
        }
    }
    if (MAP && tid == 0 && blockIdx.y == 0) p.runA[(size_t)(first + run) * p.H + h] = all;
}

// dg of one chunk per warp: the suffix sums of q.dq' - k.dk' and the chunk end's <S, dS>.
__global__ void __launch_bounds__(128)
decay_gate_kernel(Seqs q, int H, int nb, const float* __restrict__ g, const float* __restrict__ dotq,
                  const float* __restrict__ dotk, const float* __restrict__ cross, float* __restrict__ dg) {
    const int s = blockIdx.x / H, h = blockIdx.x % H, lane = threadIdx.x & 31;
    long long tok0;
    int n;
    if (!span_of(q, s, tok0, n)) return;
    const long long slots = chunk_slots(q, AC);
    for (int c = blockIdx.y * 4 + (threadIdx.x >> 5); c * AC < n; c += gridDim.y * 4) {
        float x[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {  // lane: tokens 2 lane, 2 lane + 1 of the chunk
            const int pos = c * AC + 2 * lane + j;
            x[j] = 0.f;
            if (pos < n)
                for (int b = 0; b < nb; ++b) {
                    const size_t at = ((size_t)b * q.rows + tok0 + pos) * H + h;
                    x[j] += dotq[at] - dotk[at];
                }
        }
        float sum = x[0] + x[1], e = 0.f;
        float run = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {  // sums over this lane and those after it
            const float y = __shfl_down_sync(0xffffffffu, run, o);
            if (lane + o < 32) run += y;
        }
        for (int b = 0; b < nb; ++b) e += cross[((size_t)b * slots + tok0 / AC + s + c) * H + h];
        const int pos = c * AC + 2 * lane;
        const float after = run - sum + e;
        // past a reset nothing depends on the gate: zero, not the sums' rounding
        const size_t at = ((size_t)tok0 + pos) * H + h;
        if (pos + 1 < n) dg[at + H] = decay_of(g[at + H]) == 0.f ? 0.f : after + x[1];
        if (pos < n) dg[at] = decay_of(g[at]) == 0.f ? 0.f : after + x[1] + x[0];
    }
}

GDN_DEV void store8(float* to, const float (&x)[8]) {
    reinterpret_cast<float4*>(to)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(to)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
GDN_DEV void store8(__nv_bfloat16* to, const float (&x)[8]) {
    *reinterpret_cast<uint4*>(to) = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
}

// Gradients of shared key heads: the sum over a group's value heads, in order.  One
// thread per 8 channels of a row, dq and dk in one launch; bound by the reading of the
// fp32 parts.
template <typename T>
__global__ void __launch_bounds__(256)
decay_group_sum_kernel(Seqs q, int Hk, int rep, int d, const float* __restrict__ part_q, const float* __restrict__ part_k,
                       T* __restrict__ dq, T* __restrict__ dk) {
    long long tok0;
    int n;
    if (!span_of(q, blockIdx.x, tok0, n)) return;
    const float* part = blockIdx.z ? part_k : part_q;
    T* out = blockIdx.z ? dk : dq;
    const int sh = __ffs(d) - 4;  // d / 8 pieces per row, a power of two
    const size_t total = ((size_t)n * Hk) << sh;
    for (size_t e = (size_t)blockIdx.y * 256 + threadIdx.x; e < total; e += (size_t)gridDim.y * 256) {
        const size_t row = (size_t)tok0 * Hk + (e >> sh);  // token * Hk + key head
        const int c = 8 * (int)(e & ((1u << sh) - 1));
        const float4* src = reinterpret_cast<const float4*>(part + row * rep * d + c);
        float sum[8] = {};
#pragma unroll 2
        for (int r = 0; r < rep; ++r, src += d / 4) {
            const float4 x = __ldcs(src), y = __ldcs(src + 1);
            sum[0] += x.x; sum[1] += x.y; sum[2] += x.z; sum[3] += x.w;
            sum[4] += y.x; sum[5] += y.y; sum[6] += y.z; sum[7] += y.w;
        }
        store8(out + row * d + c, sum);
    }
}

template <int CD, int RB, typename T, bool REV, int WT>
void launch_walk_of(const Walk& w, cudaStream_t st) {
    const auto grid = [&](int runs) { return dim3((unsigned)(items(w.seq, runs, w.len * TT) * w.H), (w.RD + RB - 1) / RB); };
    const int smem = sizeof(WalkSmem<CD, RB, WT>);
    if (w.runs > 1) {
        auto* map = decay_walk_kernel<CD, RB, T, REV, true, WT>;
        cudaFuncSetAttribute(map, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        GDN_LAUNCH("decay_map", st, (map<<<w.seq.cu ? grid(w.runs) : grid(w.runs - 1), WT, smem, st>>>(w)));
    }
    auto* walk = decay_walk_kernel<CD, RB, T, REV, false, WT>;
    cudaFuncSetAttribute(walk, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    GDN_LAUNCH(REV ? "decay_walk_rev" : "decay_walk", st, (walk<<<grid(w.runs), WT, smem, st>>>(w)));
}

template <int CD, typename T, bool REV>
void launch_walk_rows(const Walk& w, cudaStream_t st) {
    if (w.RD == 16) launch_walk_of<CD, 16, T, REV, 128>(w, st);
    else if (w.RD == 32) launch_walk_of<CD, 32, T, REV, 128>(w, st);
    else if constexpr (CD < 128) launch_walk_of<CD, kRows, T, REV, 256>(w, st);
    else if (w.wide) launch_walk_of<CD, kRows, T, REV, 256>(w, st);
    else launch_walk_of<CD, kRows, T, REV, 128>(w, st);
}

template <typename T, bool REV>
void launch_walk(const Walk& w, int CD, cudaStream_t st) {
    switch (CD) {
        case 16: launch_walk_rows<16, T, REV>(w, st); break;
        case 32: launch_walk_rows<32, T, REV>(w, st); break;
        case 64: launch_walk_rows<64, T, REV>(w, st); break;
        default: launch_walk_rows<128, T, REV>(w, st);
    }
}

int row_blocks(int RD) { return (RD + kRows - 1) / kRows; }

// Runs per chain, of whole chunks: 1 when the chains fill the device.  Estimated in
// tiles on the critical path: a tile of the map costs a third of one of the walk, the
// second launch about four, and adding up what the runs before leave 0.1 each.  Packed
// sequences have rows / length + nseq runs together, however long the longest is.  (7
// packed sequences of up to 1002 tokens, 6 heads, 64 x 64: runs of 4 tiles 49 us, whole
// chains 197 us.)
struct Cut {
    int runs, len;
    long long ctas;  // with something to do
};
Cut cut(const Problem& p, int RD) {
    const int tiles = ((p.seq.cu ? p.seq.rows : p.seq.len) + TT - 1) / TT;
    const long long heads = (long long)p.H * row_blocks(RD);
    auto waves = [](long long n) { return (double)((n + 295) / 296); };  // two CTAs per SM
    Cut best{1, std::max(tiles, 1), heads * p.seq.nseq};
    double cost = ceil(longest(p.seq) / TT) * waves(heads * p.seq.nseq);
    for (int r = 2; r <= 64; ++r) {
        int len = (tiles + r - 1) / r;
        len += len % 2;  // whole chunks of the gate gradient
        const int runs = (tiles + len - 1) / len;
        if (runs < 2) break;
        const long long all = heads * items(p.seq, runs, len * TT);
        const double c = len * waves(all) * 4 / 3 + 4 + 0.1 * runs;
        if (c < 0.9 * cost) {
            cost = c;
            best = Cut{runs, len, all};
        }
    }
    return best;
}
size_t runs_bytes(const Problem& p, const Cut& c) {
    if (c.runs == 1) return 0;
    const size_t n = (size_t)items(p.seq, c.runs, c.len * TT) * p.H;
    return n * p.dk * p.dv * 4 + ((n * 4 + 255) & ~(size_t)255);
}
void set_runs(Walk& w, const Problem& p, const Cut& c, void* at) {
    w.runs = c.runs;
    w.len = c.len;
    w.wide = c.ctas <= 148;
    w.runR = (float*)at;
    w.runA = w.runR + (size_t)items(p.seq, c.runs, c.len * TT) * p.H * p.dk * p.dv;
}

struct BwdLayout {
    size_t runs, anchor, dotq, dotk, cross, dq, dk, end;
};
BwdLayout bwd_layout(const Problem& p) {
    BwdLayout l{};
    size_t o = kStatusBytes;
    auto take = [&](size_t bytes) { size_t r = o; o += (bytes + 255) & ~(size_t)255; return r; };
    const size_t slots = (size_t)chunk_slots(p.seq, AC), nb = row_blocks(p.dk), rows = p.seq.rows;
    l.runs = take(std::max(runs_bytes(p, cut(p, p.dk)), runs_bytes(p, cut(p, p.dv))));
    l.anchor = take(slots * p.H * p.dk * p.dv * 4);
    l.dotq = take(nb * rows * p.H * 4);
    l.dotk = take(nb * rows * p.H * 4);
    l.cross = take(nb * slots * p.H * 4);
    if (p.H != p.Hk) {
        l.dq = take(rows * p.H * p.dk * 4);
        l.dk = take(rows * p.H * p.dk * 4);
    }
    l.end = o;
    return l;
}

// Blocks along one sequence's tokens for the small kernels after the walks.
unsigned spread(const Problem& p, long long per_seq) {
    const long long want = (2048 + p.seq.nseq - 1) / p.seq.nseq;
    const long long n = per_seq < want ? per_seq : want;
    return (unsigned)(n < 1 ? 1 : n > 65535 ? 65535 : n);
}

template <typename T>
void run_bwd(const Problem& p, const void* q, const void* k, const void* v, const float* g, const float* h0,
             const void* dO, const float* dhT, void* dq, void* dk, void* dv, float* dg, float* dh0, void* ws,
             cudaStream_t st) {
    const BwdLayout l = bwd_layout(p);
    char* base = (char*)ws;
    const int rep = p.H / p.Hk;
    const Operand oq{q, p.Hk, rep, p.dk}, ok{k, p.Hk, rep, p.dk}, ov{v, p.H, 1, p.dv}, od{dO, p.H, 1, p.dv};
    Walk w{};
    w.g = g; w.seq = p.seq; w.H = p.H; w.status = (unsigned int*)ws;
    w.anchor = (float*)(base + l.anchor);
    w.out_f32 = rep > 1;
    set_runs(w, p, cut(p, p.dk), base + l.runs);
    // dq, with the states at the chunk ends kept
    w.x = od; w.w = ov; w.y = ok; w.z = oq;
    w.init = h0; w.init_t = true; w.c_out = p.scale; w.c_y = 1.f; w.RD = p.dk;
    w.out = rep > 1 ? (void*)(base + l.dq) : dq;
    w.dots = (float*)(base + l.dotq);
    launch_walk<T, false>(w, p.dv, st);
    // dk
    w.x = ov; w.w = od; w.y = oq; w.z = ok;
    w.init = dhT; w.c_out = 1.f; w.c_y = p.scale;
    w.out = rep > 1 ? (void*)(base + l.dk) : dk;
    w.dots = (float*)(base + l.dotk);
    w.cross = (float*)(base + l.cross);
    launch_walk<T, true>(w, p.dv, st);
    // dv and dh0: scale goes with w = q, which both the state and the read-out's own pair take
    Walk u{};
    u.g = g; u.seq = p.seq; u.H = p.H; u.status = (unsigned int*)ws;
    u.x = ok; u.w = oq; u.y = od;
    u.init = dhT; u.c_out = 1.f; u.c_y = p.scale; u.RD = p.dv;
    u.last = dh0;
    set_runs(u, p, cut(p, p.dv), base + l.runs);
    u.out = dv;
    launch_walk<T, true>(u, p.dk, st);
    const unsigned chunks = spread(p, (p.seq.cu ? p.seq.rows : p.seq.len) / (4 * AC) + 1);
    GDN_LAUNCH("decay_gate", st, (decay_gate_kernel<<<dim3((unsigned)((long long)p.seq.nseq * p.H), chunks), 128, 0, st>>>(
        p.seq, p.H, row_blocks(p.dk), g, (const float*)(base + l.dotq), (const float*)(base + l.dotk),
        (const float*)(base + l.cross), dg)));
    if (rep > 1) launch_group_sum(p, (const float*)(base + l.dq), (const float*)(base + l.dk), dq, dk, st);
}

template <typename T>
void run_fwd(const Problem& p, const void* q, const void* k, const void* v, const float* g, const float* h0,
             void* o, float* hT, void* ws, cudaStream_t st) {
    const int rep = p.H / p.Hk;
    Walk w{};
    w.g = g; w.seq = p.seq; w.H = p.H; w.status = (unsigned int*)ws;
    w.x = Operand{q, p.Hk, rep, p.dk}; w.w = Operand{k, p.Hk, rep, p.dk}; w.y = Operand{v, p.H, 1, p.dv};
    w.init = h0; w.last = hT; w.out = o; w.c_out = p.scale; w.c_y = 1.f; w.RD = p.dv;
    set_runs(w, p, cut(p, p.dv), (char*)ws + kStatusBytes);
    launch_walk<T, false>(w, p.dk, st);
}

// ---- the single-token step ---------------------------------------------------
// S <- a S + v k^T, o = S (scale q), in place: one 128-bit read and write per
// four state elements, which is what bounds it: 256 sequences of 16 heads, 128 x 128,
// in 93 us, 5.8 TB/s.  A row of DK floats is covered by DK/16 lanes holding 16 columns
// each (columns 4 (lane + L j) + e, whole 128-byte lines per warp instruction), two
// rows per thread; CTAs split the rows of a state as well, so that few streams still
// spread over the SMs.
constexpr int ST = 128;

template <int DK, typename T>
__global__ void __launch_bounds__(ST)
decay_step_kernel(int H, int Hk, int dv, float scale, const T* __restrict__ q, const T* __restrict__ k,
                  const T* __restrict__ v, const float* __restrict__ g, float* __restrict__ state,
                  T* __restrict__ o) {
    constexpr int L = DK / 16, RPW = 32 / L, RPB = (ST / 32) * RPW * 2;
    const int nh = blockIdx.x, n = nh / H, h = nh % H;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane % L, grp = lane / L;
    float* S = state + (size_t)nh * dv * DK;
    int row[2];
    float4 s[2][4];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        row[r] = blockIdx.y * RPB + (2 * warp + r) * RPW + grp;
        const float4* src = reinterpret_cast<const float4*>(S + (size_t)(row[r] < dv ? row[r] : 0) * DK);
#pragma unroll
        for (int j = 0; j < 4; ++j) s[r][j] = __ldcs(src + sub + L * j);
    }
    const size_t kh = ((size_t)n * Hk + h / (H / Hk)) * DK;
    float kr[16], qr[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        const int c = 4 * (sub + L * (j / 4)) + j % 4;
        kr[j] = to_f(k[kh + c]);
        qr[j] = to_f(q[kh + c]);
    }
    const float a = decay_of(g[nh]);
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const bool in = row[r] < dv;
        const float y = in ? to_f(v[(size_t)nh * dv + row[r]]) : 0.f;
        float acc = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float4& x = s[r][j];
            x.x = a * x.x + y * kr[4 * j]; x.y = a * x.y + y * kr[4 * j + 1];
            x.z = a * x.z + y * kr[4 * j + 2]; x.w = a * x.w + y * kr[4 * j + 3];
            acc += x.x * qr[4 * j] + x.y * qr[4 * j + 1] + x.z * qr[4 * j + 2] + x.w * qr[4 * j + 3];
        }
#pragma unroll
        for (int e = L / 2; e > 0; e >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, e);
        if (!in) continue;  // after the row's last shuffle
        float4* dst = reinterpret_cast<float4*>(S + (size_t)row[r] * DK);
#pragma unroll
        for (int j = 0; j < 4; ++j) __stcs(dst + sub + L * j, s[r][j]);
        if (sub == 0) o[(size_t)nh * dv + row[r]] = from_f<T>(scale * acc);
    }
}

template <typename T>
void run_step(int N, int H, int Hk, int dk, int dv, float scale, const void* q, const void* k, const void* v,
              const float* g, float* state, void* o, cudaStream_t st) {
    auto go = [&](auto cd) {
        constexpr int DK = decltype(cd)::value, RPB = (ST / 32) * (32 / (DK / 16)) * 2;
        GDN_LAUNCH("decay_step", st, (decay_step_kernel<DK, T><<<dim3((unsigned)((long long)N * H), (dv + RPB - 1) / RPB), ST, 0, st>>>(
            H, Hk, dv, scale, (const T*)q, (const T*)k, (const T*)v, g, state, (T*)o)));
    };
    switch (dk) {
        case 16: go(std::integral_constant<int, 16>{}); break;
        case 32: go(std::integral_constant<int, 32>{}); break;
        case 64: go(std::integral_constant<int, 64>{}); break;
        default: go(std::integral_constant<int, 128>{}); break;
    }
}

}  // namespace

void launch_group_sum(const Problem& p, const float* part_q, const float* part_k, void* dq, void* dk, cudaStream_t st) {
    const dim3 grid((unsigned)p.seq.nseq, spread(p, ((long long)(p.seq.cu ? p.seq.rows : p.seq.len) * p.Hk * p.dk) / 2048 + 1), 2);
    const int rep = p.H / p.Hk;
    if (p.dtype == GDN_BF16)
        GDN_LAUNCH("decay_group_sum", st, (decay_group_sum_kernel<<<grid, 256, 0, st>>>(p.seq, p.Hk, rep, p.dk, part_q, part_k, (__nv_bfloat16*)dq, (__nv_bfloat16*)dk)));
    else
        GDN_LAUNCH("decay_group_sum", st, (decay_group_sum_kernel<<<grid, 256, 0, st>>>(p.seq, p.Hk, rep, p.dk, part_q, part_k, (float*)dq, (float*)dk)));
}

size_t simt_fwd_workspace(const Problem& p) { return kStatusBytes + runs_bytes(p, cut(p, p.dv)); }

size_t simt_bwd_workspace(const Problem& p) { return bwd_layout(p).end; }

void launch_simt_fwd(const Problem& p, const void* q, const void* k, const void* v, const float* g,
                     const float* h0, void* o, float* hT, void* ws, cudaStream_t st) {
    if (p.dtype == GDN_BF16) run_fwd<__nv_bfloat16>(p, q, k, v, g, h0, o, hT, ws, st);
    else run_fwd<float>(p, q, k, v, g, h0, o, hT, ws, st);
}

void launch_simt_bwd(const Problem& p, const void* q, const void* k, const void* v, const float* g,
                     const float* h0, const void* dO, const float* dhT, void* dq, void* dk, void* dv,
                     float* dg, float* dh0, void* ws, cudaStream_t st) {
    if (p.dtype == GDN_BF16) run_bwd<__nv_bfloat16>(p, q, k, v, g, h0, dO, dhT, dq, dk, dv, dg, dh0, ws, st);
    else run_bwd<float>(p, q, k, v, g, h0, dO, dhT, dq, dk, dv, dg, dh0, ws, st);
}

void launch_decay_step(int N, int H, int Hk, int dk, int dv, gdn_dtype dtype, float scale, const void* q,
                       const void* k, const void* v, const float* g, float* state, void* o,
                       cudaStream_t st) {
    if (dtype == GDN_BF16) run_step<__nv_bfloat16>(N, H, Hk, dk, dv, scale, q, k, v, g, state, o, st);
    else run_step<float>(N, H, Hk, dk, dv, scale, q, k, v, g, state, o, st);
}

}  // namespace decay
}  // namespace gdn
