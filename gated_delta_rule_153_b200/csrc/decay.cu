// decay.cu -- linear attention with a decay per head in fp32 arithmetic on
// CUDA cores, one token at a time: the path of GDN_F32 and of the head dims the
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
// shared memory in 2 x 4 and 4 x 4 register tiles; a CTA holds 32 rows of R, and the next
// tile's values are on their way to registers meanwhile.  What bounds it is the issue of
// fp32 FMAs and their shared-memory loads, one tile after the other along a chain.
#include <math.h>

#include <type_traits>

#include "common.cuh"
#include "decay.h"
#include "decay_tc.cuh"

namespace gdn {
namespace decay {
namespace {

constexpr int TT = 32;          // tokens per tile
constexpr int WT = 128;         // threads per CTA
constexpr int RB = 32;          // rows of R per CTA
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

template <int CD>
struct WalkSmem {  // rows padded by 16 bytes: eight rows of a column are in different banks
    float x[TT][CD + 4], w[TT][CD + 4], y[TT][RB + 4], z[TT][RB + 4], p[TT][TT + 4];
    float r[CD][RB + 4];
    float2 g[TT];
    float f[TT], h[TT], own[TT], red[WT / 32];
};

template <int CD, typename T, bool REV>
__global__ void __launch_bounds__(WT)
decay_walk_kernel(const Walk p) {
    extern __shared__ __align__(16) unsigned char raw[];
    WalkSmem<CD>& s = *reinterpret_cast<WalkSmem<CD>*>(raw);
    using F = Four<T>;
    constexpr int NX = TT * CD / 4 / WT > 0 ? TT * CD / 4 / WT : 1;  // groups of four per thread and tile
    constexpr int NC = CD / 16;                                      // columns of R per thread
    const int seq = blockIdx.x / p.H, h = blockIdx.x % p.H, r0 = blockIdx.y * RB;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    long long tok0;
    int n;
    if (!span_of(p.seq, seq, tok0, n)) {
        if (tid == 0) atomicOr(p.status, 2u);
        return;
    }
    const size_t sh = (size_t)seq * p.H + h;
    const long long slot0 = tok0 / AC + seq;
    // R, column-major
    for (int e = tid; e < CD * RB; e += WT) {
        const int c = p.init_t ? e / RB : e % CD, r = p.init_t ? e % RB : e / CD, row = r0 + r;
        s.r[c][r] = !p.init || row >= p.RD ? 0.f : p.init_t ? p.init[(sh * CD + c) * p.RD + row] : p.init[(sh * p.RD + row) * CD + c];
    }
    const int tiles = (n + TT - 1) / TT;
    typename F::Raw px[NX], pw[NX], py[2], pz[2];
    float pg = 0.f;
    const bool has_z = p.dots != nullptr;
    auto fetch = [&](int tile) {
        const int m = min(TT, n - tile * TT);
        const long long t0 = tok0 + (long long)tile * TT;
        const typename F::Raw zero{};
#pragma unroll
        for (int i = 0; i < NX; ++i) {
            const int e = 4 * (tid + WT * i), t = e / CD, c = e % CD;
            const bool in = t < m;
            px[i] = in ? *reinterpret_cast<const typename F::Raw*>((const T*)p.x.p + row_of(p.x, t0 + t, h) + c) : zero;
            pw[i] = in ? *reinterpret_cast<const typename F::Raw*>((const T*)p.w.p + row_of(p.w, t0 + t, h) + c) : zero;
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int e = 4 * (tid + WT * i), t = e / RB, r = e % RB;
            const bool in = t < m && r0 + r < p.RD;
            py[i] = in ? *reinterpret_cast<const typename F::Raw*>((const T*)p.y.p + row_of(p.y, t0 + t, h) + r0 + r) : zero;
            pz[i] = in && has_z ? *reinterpret_cast<const typename F::Raw*>((const T*)p.z.p + row_of(p.z, t0 + t, h) + r0 + r) : zero;
        }
        if (warp == 0) pg = lane < m ? p.g[(size_t)(t0 + lane) * p.H + h] : 0.f;
    };
    if (tiles > 0) fetch(REV ? tiles - 1 : 0);
    for (int it = 0; it < tiles; ++it) {
        const int tile = REV ? tiles - 1 - it : it;
        const int m = min(TT, n - tile * TT);
        const long long t0 = tok0 + (long long)tile * TT;
        const int end = tile * TT + m;
        const bool border = end % AC == 0 || end == n;  // the tile ends a chunk
        const long long slot = slot0 + (end - 1) / AC;
        __syncthreads();
        if (TT * CD / 4 >= WT || tid < TT * CD / 4) {
#pragma unroll
            for (int i = 0; i < NX; ++i) {
                const int e = 4 * (tid + WT * i), t = e / CD, c = e % CD;
                *reinterpret_cast<float4*>(&s.x[t][c]) = F::of(px[i]);
                *reinterpret_cast<float4*>(&s.w[t][c]) = F::of(pw[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int e = 4 * (tid + WT * i), t = e / RB, r = e % RB;
            const float4 v = F::of(py[i]);
            *reinterpret_cast<float4*>(&s.y[t][r]) = make_float4(p.c_y * v.x, p.c_y * v.y, p.c_y * v.z, p.c_y * v.w);
            *reinterpret_cast<float4*>(&s.z[t][r]) = F::of(pz[i]);
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
        if (it + 1 < tiles) fetch(REV ? tile - 1 : tile + 1);
        {   // p[t][u] = D_tu (w_u . x_t), its diagonal apart; a thread: 2 x 4
            const int t = 2 * (tid / 8), u = 4 * (tid % 8);
            float a[2][4] = {};
#pragma unroll 4
            for (int c = 0; c < CD; c += 4) {
                float4 xv[2], wv[4];
#pragma unroll
                for (int i = 0; i < 2; ++i) xv[i] = *reinterpret_cast<const float4*>(&s.x[t + i][c]);
#pragma unroll
                for (int j = 0; j < 4; ++j) wv[j] = *reinterpret_cast<const float4*>(&s.w[u + j][c]);
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        a[i][j] += xv[i].x * wv[j].x + xv[i].y * wv[j].y + xv[i].z * wv[j].z + xv[i].w * wv[j].w;
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float4 v;
                float* q = &v.x;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int tt = t + i, uu = u + j;
                    if (tt == uu) s.own[tt] = a[i][j];
                    const bool in = REV ? uu > tt : uu < tt;
                    q[j] = in ? a[i][j] * (REV ? pair_decay(s.g[uu], s.g[tt]) : pair_decay(s.g[tt], s.g[uu])) : 0.f;
                }
                *reinterpret_cast<float4*>(&s.p[t + i][u]) = v;
            }
        }
        __syncthreads();
        {   // out; a thread: 2 tokens x 4 rows
            const int t = 2 * (tid / 8), r = 4 * (tid % 8);
            float a[2][4] = {};
#pragma unroll 2
            for (int c = 0; c < CD; c += 4) {
                float4 xv[2], rv[4];
#pragma unroll
                for (int i = 0; i < 2; ++i) xv[i] = *reinterpret_cast<const float4*>(&s.x[t + i][c]);
#pragma unroll
                for (int j = 0; j < 4; ++j) rv[j] = *reinterpret_cast<const float4*>(&s.r[c + j][r]);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float q[4] = {xv[i].x, xv[i].y, xv[i].z, xv[i].w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        a[i][0] += q[j] * rv[j].x; a[i][1] += q[j] * rv[j].y;
                        a[i][2] += q[j] * rv[j].z; a[i][3] += q[j] * rv[j].w;
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) a[i][j] *= s.f[t + i];
#pragma unroll 2
            for (int u = 0; u < TT; u += 4) {
                float4 pv[2], yv[4];
#pragma unroll
                for (int i = 0; i < 2; ++i) pv[i] = *reinterpret_cast<const float4*>(&s.p[t + i][u]);
#pragma unroll
                for (int j = 0; j < 4; ++j) yv[j] = *reinterpret_cast<const float4*>(&s.y[u + j][r]);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float q[4] = {pv[i].x, pv[i].y, pv[i].z, pv[i].w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        a[i][0] += q[j] * yv[j].x; a[i][1] += q[j] * yv[j].y;
                        a[i][2] += q[j] * yv[j].z; a[i][3] += q[j] * yv[j].w;
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int tt = t + i;
                const size_t row = (size_t)(t0 + tt) * p.H + h;
                if (has_z) {
                    const float4 zv = *reinterpret_cast<const float4*>(&s.z[tt][r]);
                    float d = zv.x * a[i][0] + zv.y * a[i][1] + zv.z * a[i][2] + zv.w * a[i][3];
#pragma unroll
                    for (int o = 4; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
                    if (tid % 8 == 0 && tt < m) p.dots[(size_t)blockIdx.y * p.seq.rows * p.H + row] = p.c_out * d;
                }
                if (tt < m && r0 + r < p.RD) {
                    const float4 yv = *reinterpret_cast<const float4*>(&s.y[tt][r]);
                    const float q = s.own[tt];
                    const float4 v = make_float4(p.c_out * (a[i][0] + q * yv.x), p.c_out * (a[i][1] + q * yv.y),
                                                 p.c_out * (a[i][2] + q * yv.z), p.c_out * (a[i][3] + q * yv.w));
                    if (p.out_f32) put4((float*)p.out + row * p.RD + r0 + r, v);
                    else put4((T*)p.out + row * p.RD + r0 + r, v);
                }
            }
        }
        const int c0 = tid / 8 * NC, r = 4 * (tid % 8);  // this thread's columns and rows of R
        if (REV && p.cross && border) {
            // R is dS^T at the end of this chunk: dot it with the state there
            float d = 0.f;
            if (r0 + r < p.RD) {
                const float* A = p.anchor + (((size_t)slot * p.H + h) * p.RD + r0 + r) * CD + c0;
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int c = 0; c < NC; ++c) d += s.r[c0 + c][r + j] * A[(size_t)j * CD + c];
            }
            d = warp_sum(d);
            if (lane == 0) s.red[warp] = d;
        }
        __syncthreads();
        if (REV && p.cross && border && tid == 0) {
            float d = 0.f;
            for (int w = 0; w < WT / 32; ++w) d += s.red[w];
            p.cross[((size_t)blockIdx.y * chunk_slots(p.seq, AC) + slot) * p.H + h] = d;
        }
        {   // R; a thread: NC columns x 4 rows
            const float total = start_decay(s.g[TT - 1]);
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
                    for (int j = 0; j < 4; ++j) a[c][j] += w[c] * q[j];
            }
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                *reinterpret_cast<float4*>(&s.r[c0 + c][r]) = make_float4(a[c][0], a[c][1], a[c][2], a[c][3]);
                if (!REV && p.anchor && border && r0 + r < p.RD) {
                    float* A = p.anchor + (((size_t)slot * p.H + h) * p.RD + r0 + r) * CD + c0 + c;
#pragma unroll
                    for (int j = 0; j < 4; ++j) A[(size_t)j * CD] = a[c][j];
                }
            }
        }
    }
    if (p.last) {
        __syncthreads();
        for (int e = tid; e < CD * RB; e += WT) {
            const int r = e / CD, c = e % CD;
            if (r0 + r < p.RD) p.last[(sh * p.RD + r0 + r) * CD + c] = s.r[c][r];
        }
    }
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

// Gradients of shared key heads: the sum over a group's value heads, in order.
template <typename T>
__global__ void __launch_bounds__(256)
decay_group_sum_kernel(Seqs q, int Hk, int rep, int d, const float* __restrict__ part, T* __restrict__ out) {
    long long tok0;
    int n;
    if (!span_of(q, blockIdx.x, tok0, n)) return;
    const size_t total = (size_t)n * Hk * d;
    for (size_t e = (size_t)blockIdx.y * 256 + threadIdx.x; e < total; e += (size_t)gridDim.y * 256) {
        const size_t row = e / d;  // token * Hk + key head
        const size_t c = e % d;
        const float* src = part + ((size_t)tok0 * Hk + row) * rep * d + c;
        float sum = 0.f;
        for (int r = 0; r < rep; ++r) sum += src[(size_t)r * d];
        out[((size_t)tok0 * Hk + row) * d + c] = from_f<T>(sum);
    }
}

template <typename T, bool REV>
void launch_walk(const Walk& w, int CD, cudaStream_t st) {
    auto go = [&](auto cd, const char* name) {
        constexpr int C = decltype(cd)::value;
        const dim3 grid((unsigned)((long long)w.seq.nseq * w.H), (w.RD + RB - 1) / RB);
        const int smem = sizeof(WalkSmem<C>);
        cudaFuncSetAttribute(decay_walk_kernel<C, T, REV>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        GDN_LAUNCH(name, st, (decay_walk_kernel<C, T, REV><<<grid, WT, smem, st>>>(w)));
    };
    const char* name = REV ? "decay_walk_rev" : "decay_walk";
    switch (CD) {
        case 16: go(std::integral_constant<int, 16>{}, name); break;
        case 32: go(std::integral_constant<int, 32>{}, name); break;
        case 64: go(std::integral_constant<int, 64>{}, name); break;
        default: go(std::integral_constant<int, 128>{}, name); break;
    }
}

int row_blocks(int RD) { return (RD + RB - 1) / RB; }

struct BwdLayout {
    size_t anchor, dotq, dotk, cross, dq, dk, end;
};
BwdLayout bwd_layout(const Problem& p) {
    BwdLayout l{};
    size_t o = kStatusBytes;
    auto take = [&](size_t bytes) { size_t r = o; o += (bytes + 255) & ~(size_t)255; return r; };
    const size_t slots = (size_t)chunk_slots(p.seq, AC), nb = row_blocks(p.dk), rows = p.seq.rows;
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
    u.out = dv;
    launch_walk<T, true>(u, p.dk, st);
    const unsigned chunks = spread(p, (p.seq.cu ? p.seq.rows : p.seq.len) / (4 * AC) + 1);
    GDN_LAUNCH("decay_gate", st, (decay_gate_kernel<<<dim3((unsigned)((long long)p.seq.nseq * p.H), chunks), 128, 0, st>>>(
        p.seq, p.H, row_blocks(p.dk), g, (const float*)(base + l.dotq), (const float*)(base + l.dotk),
        (const float*)(base + l.cross), dg)));
    if (rep > 1) {
        launch_group_sum(p, p.dk, (const float*)(base + l.dq), dq, st);
        launch_group_sum(p, p.dk, (const float*)(base + l.dk), dk, st);
    }
}

template <typename T>
void run_fwd(const Problem& p, const void* q, const void* k, const void* v, const float* g, const float* h0,
             void* o, float* hT, unsigned int* status, cudaStream_t st) {
    const int rep = p.H / p.Hk;
    Walk w{};
    w.g = g; w.seq = p.seq; w.H = p.H; w.status = status;
    w.x = Operand{q, p.Hk, rep, p.dk}; w.w = Operand{k, p.Hk, rep, p.dk}; w.y = Operand{v, p.H, 1, p.dv};
    w.init = h0; w.last = hT; w.out = o; w.c_out = p.scale; w.c_y = 1.f; w.RD = p.dv;
    launch_walk<T, false>(w, p.dk, st);
}

// ---- the single-token step ---------------------------------------------------
// S <- a S + v k^T, o = S (scale q), in place: one 128-bit read and write per
// four state elements.  A row of DK floats is covered by DK/16 lanes holding
// 16 columns each (columns 4 (lane + L j) + e, whole 128-byte lines per warp
// instruction), two rows per thread; CTAs split the rows of a state as well, so
// that few streams still spread over the SMs.
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

void launch_group_sum(const Problem& p, int d, const float* part, void* out, cudaStream_t st) {
    const dim3 grid((unsigned)p.seq.nseq, spread(p, ((long long)(p.seq.cu ? p.seq.rows : p.seq.len) * p.Hk * d) / 1024 + 1));
    if (p.dtype == GDN_BF16)
        GDN_LAUNCH("decay_group_sum", st, (decay_group_sum_kernel<<<grid, 256, 0, st>>>(p.seq, p.Hk, p.H / p.Hk, d, part, (__nv_bfloat16*)out)));
    else
        GDN_LAUNCH("decay_group_sum", st, (decay_group_sum_kernel<<<grid, 256, 0, st>>>(p.seq, p.Hk, p.H / p.Hk, d, part, (float*)out)));
}

size_t simt_bwd_workspace(const Problem& p) { return bwd_layout(p).end; }

void launch_simt_fwd(const Problem& p, const void* q, const void* k, const void* v, const float* g,
                     const float* h0, void* o, float* hT, unsigned int* status, cudaStream_t st) {
    if (p.dtype == GDN_BF16) run_fwd<__nv_bfloat16>(p, q, k, v, g, h0, o, hT, status, st);
    else run_fwd<float>(p, q, k, v, g, h0, o, hT, status, st);
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
