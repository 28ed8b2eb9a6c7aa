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
// A row of R is covered by L = CD/16 lanes of 16 columns each, one or
// two rows per thread, so R never leaves the registers; a tile of 32 tokens is staged in
// shared memory as fp32.  What bounds it is the fp32 FMA rate: 3 operations
// per state element and token (dk = dv = 128: 49 k per token-head and walk).
#include <math.h>

#include <type_traits>

#include "common.cuh"
#include "decay.h"

namespace gdn {
namespace decay {
namespace {

constexpr int TT = 32;          // tokens per staged tile
constexpr int WT = 128;         // threads per CTA
constexpr int AC = 64;          // tokens per chunk of the gate gradient

// A gate of -inf (or one so low that e^g is zero in fp32) is a reset.
GDN_DEV float decay_of(float g) { return expf(g); }

template <int CD>
constexpr int rows_per_thread() { return CD >= 64 ? 2 : 1; }
template <int CD>
constexpr int rows_per_cta() { return (WT / 32) * (32 / (CD / 16)) * rows_per_thread<CD>(); }

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

template <int CD, typename T, bool REV>
__global__ void __launch_bounds__(WT)
decay_walk_kernel(const Walk p) {
    constexpr int L = CD / 16, RPW = 32 / L, RPT = rows_per_thread<CD>(), RB = rows_per_cta<CD>(),
                  NW = WT / 32;
    __shared__ __align__(16) float sx[TT][CD], sw[TT][CD];
    __shared__ float sy[TT][RB], sz[TT][RB], sa[TT], sdot[NW][TT], sred[NW];
    const int s = blockIdx.x / p.H, h = blockIdx.x % p.H, r0 = blockIdx.y * RB;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int sub = lane % L, grp = lane / L;
    long long tok0;
    int n;
    if (!span_of(p.seq, s, tok0, n)) {
        if (tid == 0) atomicOr(p.status, 2u);
        return;
    }
    const size_t sh = (size_t)s * p.H + h;
    const long long slot0 = tok0 / AC + s;
    int row[RPT];
    float R[RPT][16];
#pragma unroll
    for (int q = 0; q < RPT; ++q) {
        row[q] = (warp * RPT + q) * RPW + grp;  // within the block
        const int r = r0 + row[q];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            const int c = 4 * (sub + L * (e / 4)) + e % 4;
            R[q][e] = 0.f;
            if (p.init && r < p.RD)
                R[q][e] = p.init_t ? p.init[(sh * CD + c) * p.RD + r] : p.init[(sh * p.RD + r) * CD + c];
        }
    }
    const int tiles = (n + TT - 1) / TT;
    for (int it = 0; it < tiles; ++it) {
        const int tile = REV ? tiles - 1 - it : it;
        const int m = min(TT, n - tile * TT);
        const long long t0 = tok0 + (long long)tile * TT;
        __syncthreads();
        for (int e = tid; e < m * CD; e += WT) {
            const int t = e / CD, c = e % CD;
            sx[t][c] = to_f(((const T*)p.x.p)[row_of(p.x, t0 + t, h) + c]);
            sw[t][c] = to_f(((const T*)p.w.p)[row_of(p.w, t0 + t, h) + c]);
        }
        for (int e = tid; e < m * RB; e += WT) {
            const int t = e / RB, r = e % RB;
            const bool in = r0 + r < p.RD;
            sy[t][r] = in ? p.c_y * to_f(((const T*)p.y.p)[row_of(p.y, t0 + t, h) + r0 + r]) : 0.f;
            if (p.dots) sz[t][r] = in ? to_f(((const T*)p.z.p)[row_of(p.z, t0 + t, h) + r0 + r]) : 0.f;
        }
        if (tid < m) {
            // backwards the decay applied before token t is that of token t + 1
            const long long t = t0 + tid + (REV ? 1 : 0);
            sa[tid] = t < tok0 + n ? decay_of(p.g[(size_t)t * p.H + h]) : 1.f;
        }
        __syncthreads();
        for (int i = 0; i < m; ++i) {
            const int t = REV ? m - 1 - i : i;
            const int pos = tile * TT + t;
            const float a = sa[t];
#pragma unroll
            for (int q = 0; q < RPT; ++q)
#pragma unroll
                for (int e = 0; e < 16; ++e) R[q][e] *= a;
            if (REV && p.cross && ((pos + 1) % AC == 0 || pos + 1 == n)) {
                // R is dS^T at the end of this chunk: dot it with the state there
                const long long slot = slot0 + pos / AC;
                float d = 0.f;
#pragma unroll
                for (int q = 0; q < RPT; ++q) {
                    const int r = r0 + row[q];
                    if (r >= p.RD) continue;
                    const float* A = p.anchor + (((size_t)slot * p.H + h) * p.RD + r) * CD;
#pragma unroll
                    for (int e = 0; e < 16; ++e) d += R[q][e] * A[4 * (sub + L * (e / 4)) + e % 4];
                }
                d = warp_sum(d);
                if (lane == 0) sred[warp] = d;
                __syncthreads();
                if (tid == 0) {
                    float all = 0.f;
                    for (int w = 0; w < NW; ++w) all += sred[w];
                    p.cross[((size_t)blockIdx.y * chunk_slots(p.seq, AC) + slot) * p.H + h] = all;
                }
                __syncthreads();
            }
            float acc[RPT], wx = 0.f, w[16];
#pragma unroll
            for (int q = 0; q < RPT; ++q) acc[q] = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float4 x4 = *reinterpret_cast<const float4*>(&sx[t][4 * (sub + L * j)]);
                const float4 w4 = *reinterpret_cast<const float4*>(&sw[t][4 * (sub + L * j)]);
                const float x[4] = {x4.x, x4.y, x4.z, x4.w};
                w[4 * j] = w4.x; w[4 * j + 1] = w4.y; w[4 * j + 2] = w4.z; w[4 * j + 3] = w4.w;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    wx += w[4 * j + e] * x[e];
#pragma unroll
                    for (int q = 0; q < RPT; ++q) acc[q] += R[q][4 * j + e] * x[e];
                }
            }
#pragma unroll
            for (int o = L / 2; o > 0; o >>= 1) {
                wx += __shfl_xor_sync(0xffffffffu, wx, o);
#pragma unroll
                for (int q = 0; q < RPT; ++q) acc[q] += __shfl_xor_sync(0xffffffffu, acc[q], o);
            }
            float dot = 0.f;
#pragma unroll
            for (int q = 0; q < RPT; ++q) {
                const float y = sy[t][row[q]];
                if (p.dots && sub == 0) dot += sz[t][row[q]] * acc[q];
                if (sub == 0 && r0 + row[q] < p.RD) {
                    const float v = p.c_out * (acc[q] + y * wx);
                    const size_t at = ((size_t)(t0 + t) * p.H + h) * p.RD + r0 + row[q];
                    if (p.out_f32) ((float*)p.out)[at] = v;
                    else ((T*)p.out)[at] = from_f<T>(v);
                }
#pragma unroll
                for (int e = 0; e < 16; ++e) R[q][e] += y * w[e];
            }
            if (p.dots) {
                dot = warp_sum(dot);
                if (lane == 0) sdot[warp][t] = p.c_out * dot;
            }
            if (!REV && p.anchor && ((pos + 1) % AC == 0 || pos + 1 == n)) {
                const long long slot = slot0 + pos / AC;
#pragma unroll
                for (int q = 0; q < RPT; ++q) {
                    const int r = r0 + row[q];
                    if (r >= p.RD) continue;
                    float* A = p.anchor + (((size_t)slot * p.H + h) * p.RD + r) * CD;
#pragma unroll
                    for (int e = 0; e < 16; ++e) A[4 * (sub + L * (e / 4)) + e % 4] = R[q][e];
                }
            }
        }
        if (p.dots) {
            __syncthreads();
            if (tid < m) {
                float d = 0.f;
                for (int w = 0; w < NW; ++w) d += sdot[w][tid];
                p.dots[((size_t)blockIdx.y * p.seq.rows + t0 + tid) * p.H + h] = d;
            }
        }
    }
    if (p.last) {
        const float a = REV && n > 0 ? decay_of(p.g[(size_t)tok0 * p.H + h]) : 1.f;
#pragma unroll
        for (int q = 0; q < RPT; ++q) {
            const int r = r0 + row[q];
            if (r >= p.RD) continue;
#pragma unroll
            for (int e = 0; e < 16; ++e)
                p.last[(sh * p.RD + r) * CD + 4 * (sub + L * (e / 4)) + e % 4] = a * R[q][e];
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
        const dim3 grid((unsigned)((long long)w.seq.nseq * w.H), (w.RD + rows_per_cta<C>() - 1) / rows_per_cta<C>());
        GDN_LAUNCH(name, st, (decay_walk_kernel<C, T, REV><<<grid, WT, 0, st>>>(w)));
    };
    const char* name = REV ? "decay_walk_rev" : "decay_walk";
    switch (CD) {
        case 16: go(std::integral_constant<int, 16>{}, name); break;
        case 32: go(std::integral_constant<int, 32>{}, name); break;
        case 64: go(std::integral_constant<int, 64>{}, name); break;
        default: go(std::integral_constant<int, 128>{}, name); break;
    }
}

int row_blocks(int RD, int CD) {
    const int rb = CD == 16 ? rows_per_cta<16>() : CD == 32 ? rows_per_cta<32>() : CD == 64 ? rows_per_cta<64>() : rows_per_cta<128>();
    return (RD + rb - 1) / rb;
}

struct BwdLayout {
    size_t anchor, dotq, dotk, cross, dq, dk, end;
};
BwdLayout bwd_layout(const Problem& p) {
    BwdLayout l{};
    size_t o = kStatusBytes;
    auto take = [&](size_t bytes) { size_t r = o; o += (bytes + 255) & ~(size_t)255; return r; };
    const size_t slots = (size_t)chunk_slots(p.seq, AC), nb = row_blocks(p.dk, p.dv), rows = p.seq.rows;
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
        p.seq, p.H, row_blocks(p.dk, p.dv), g, (const float*)(base + l.dotq), (const float*)(base + l.dotk),
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
