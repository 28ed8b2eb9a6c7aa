// decay_walk.cu -- linear attention with a decay per head on the fifth-generation
// tensor cores: the walk along a chain of 128-token chunks, with its state on
// chip from the first chunk to the last.
//
// One CTA walks one (sequence, head) for 64 of its dv value channels.  Per chunk,
// with S (key channels x value channels) entering it and D the pair decays:
//     A = Q K^T                        128 x 128 x dk     lane = query token
//     P = scale A .* D, causal         -> bf16 A operand in tensor memory
//     X = Q S                          128 x 64 x dk      lane = query token
//     Y = P V                          128 x 64 x 128
//     O = diag(scale e^G) X + Y
//     N = K^T (diag(e^{G_last - G}) V) dk x 64 x 128      lane = key channel
//     S <- e^{G_last} S + N            in fp32 registers
// Only the last line is sequential, and it is one multiply-add per element: N does
// not depend on S.  The products are issued in the order A X N Y, so that the tensor
// pipe has X and N to do while P is made from A, and Y and the next A while N goes
// into S.
//
// Rounding.  Products take bf16 operands and accumulate in fp32.  q, k, v are
// bf16 already.  P and, for X, the state are rounded to bf16 once: o itself is
// bf16, and the two errors are of the size of its own rounding.  Where a row of P has few
// entries, though, its rounding does not average out (o of few tokens was up to 1.8 times
// its type's rounding off): with SHORT, in a chunk of up to 64 tokens the other half of P
// holds what the rounding left, over the same V rows once more, for which the products take
// no longer.  The decayed V of
// the state is split into three bf16 terms (exact to fp32), because errors there
// would stay in the state, which is kept and returned in fp32.
//
// Roles: warps 0-7 make P of A (thread = query token), then the column factors of the
// next chunk's decays, then half of O; warps 8-15 own the state (thread = key channel,
// half of the value channels) and combine the other half of O; warp 16 issues the loads,
// warp 17 the products, warp 18 forms the gates' cumsum, two chunks ahead.  The decayed V
// is split by the last four warps and, a quarter of it, by the state's.  K and V tiles
// go through a two-stage ring; Q, which A and X are done with early in a chunk, has
// one place.
//
// MODE 2 walks K and V (backwards: Q and dO, with the gradient of the state) and
// writes the state entering each chunk, in fp32, for the backward's local products
// (decay_bwd.cu); warps 0-7 split V.
// MODE 1 walks K and V alone and writes the state a run of chunks adds to a zero
// state, with the run's decay.  With few chains, each is cut into runs: MODE 1 over
// all runs but the last, then MODE 0 or 2 over all runs at once, each starting from the
// sum of the runs before it.
//
// What bounds it, at 8 x 2048 tokens of 8 heads, dk = dv = 128 (128 CTAs of 16 chunks):
// MODE 0 takes 53 us, 2.6 TB/s of the bytes it cannot do without, 3.3 us a chunk: A, P (two
// warps per scheduler, latency), Y, O, each waiting for the one before, with X and N in
// between; the tensor pipe is busy for a third of it.  With O left to the warps of P alone
// it took 55 us, with O left to the state's 53 us.  MODE 2 takes 33 us forwards and 40 us
// backwards, 135 and 202 MB to and from HBM (K, V and the states out, backwards the forward
// states as well; the two CTAs of a head share K through L2): 4.1 and 5.0 TB/s, 62 and 77 %
// of the measured rate.
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "decay_tc.cuh"

namespace gdn {
namespace decay {
namespace {

constexpr int NB = 64;               // value channels per CTA
constexpr int PANEL = CT * 128;      // bytes of a 128-row, 64-channel tile
constexpr int kEpi = 8, kState = 8;  // warps that make P and O, and that own the state
// Warps that split V: four of their own in MODE 0, else the eight that P and O leave idle.
template <int MODE>
constexpr int kSplit = MODE == 0 ? 4 : kEpi;
// Whether the state's warps split a quarter of V: where they do not write images too.
template <int MODE>
constexpr bool kShare = MODE != 2;
template <int MODE>
constexpr int kThreads = 32 * (kEpi + kState + 3 + (MODE == 0 ? 4 : MODE == 2 ? 1 : 0));
constexpr int NST = 2;
constexpr int kShort = CT / 2;  // tokens of a chunk that has room for P in two terms
constexpr int TERMS = 3;  // bf16 terms of the decayed V: exact to fp32

template <int DK, int MODE>
struct alignas(1024) Smem {
    unsigned char Q[DK / 64][PANEL];  // MODE 2: the state's image on its way out
    struct Stage {
        unsigned char K[DK / 64][PANEL], V[PANEL];
    } st[NST];
    unsigned char Vt[3][PANEL];  // decayed V, three bf16 terms
    // MODE 0: the entering state in bf16, [key channel][64 value channels]; MODE 2 backwards:
    // the image of the forward state at the chunk's start
    unsigned char S[MODE == 2 ? 2 : 1][DK * 128];
    Gates gate[NST];
    float col[kEpi][CT];         // per warp of P: the column factors of its decays
    FirstBad<NB> bad;            // MODE 0: values that are not finite
    // of each stage, so that nobody who waits for one can fall two phases behind
    uint64_t full[NST], v_full[NST], v_free[NST], gfull[NST], gfree[NST], n_done[NST], o_done[NST];
    uint64_t img_ready, img_free, fwd_full, fwd_free, q_full, a_done, p_ready, vt_ready, s_ready[2], x_done, o_free, drain;
    uint32_t tmem;
};

struct Params {
    CUtensorMap qmap, kmap, vmap;
    Seqs seq;
    int H, rep, dv;
    float scale;
    const float *g, *h0;
    __nv_bfloat16* o;
    float* hT;
    int runs, len;        // runs per chain, chunks per run
    float *runS, *runG;   // [item][head][value block][DK][64] and [item][head] of MODE 1
    // MODE 2: the fp32 state entering each chunk, as its upper and its lower halves (the upper
    // ones are bf16 values): [slot][head][2][value block][DK][64] of 16 bits
    __nv_bfloat16* image;
    const __nv_bfloat16* other;  // backwards: the forward states, dotted into cross
    float* cross;                // [value block][slot][head]
    unsigned int* status;
};

// tensor-memory columns: A, P (bf16 pairs), X, Y, N (the terms of V apart)
constexpr uint32_t TA = 0, TP = 128, TX = 192, TY = 256, TN = 320, kCols = 512;
// N of chunk c: without the others it has two places
template <int MODE>
GDN_DEV uint32_t tn(int c) { return MODE == 0 ? TN : 3 * NB * (c & 1); }

template <int DK, int MODE, bool REV, bool SHORT>
__global__ void __launch_bounds__(kThreads<MODE>, 1)
decay_tc_walk_kernel(const __grid_constant__ Params p) {
    extern __shared__ __align__(1024) unsigned char raw[];
    Smem<DK, MODE>& s = *reinterpret_cast<Smem<DK, MODE>*>(align1k(raw));
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int vb = blockIdx.y, h = blockIdx.x % p.H;
    long long tok0;
    int n, seq, run, first;
    if (!item_of(p.seq, p.runs, p.len * CT, MODE == 1 ? 1 : 0, blockIdx.x / p.H, seq, run, first)) return;
    if (!span_of(p.seq, seq, tok0, n)) {
        if (tid == 0) atomicOr(p.status, 2u);
        return;
    }
    const int chunks = (n + CT - 1) / CT;
    const int c0 = run * p.len, c1 = min(chunks, c0 + p.len);
    // the run that ends the chain (the first of an empty one) writes hT; runs past the end do nothing
    const bool last = c1 == chunks && (run == 0 || c0 < chunks);
    if (MODE != 1 ? (c0 >= chunks && !last) : c1 >= chunks) return;
    const int nc = c1 - c0;
    const size_t chain = (size_t)seq * p.H + h;
    const size_t slab = (size_t)DK * NB;
    // chunk c of this run, in the order of the walk
    auto chunk_of = [&](int c) { return REV ? chunks - 1 - (c0 + c) : c0 + c; };
    const size_t slot0 = (size_t)(tok0 / CT) + seq;

    if (MODE == 0) s.bad.none(tid);
    if (tid == 0) {
        for (int i = 0; i < NST; ++i) {
            mbar_init(&s.full[i], 1);
            mbar_init(&s.v_full[i], 1);
            mbar_init(&s.v_free[i], kSplit<MODE> + (kShare<MODE> ? kState : 0));  // (MODE 0 has o_done for it)
            mbar_init(&s.n_done[i], 1);
            mbar_init(&s.o_done[i], 1);
            mbar_init(&s.gfull[i], 1);
            mbar_init(&s.gfree[i], (MODE == 0 ? kEpi : 0) + kState + kSplit<MODE>);
        }
        mbar_init(&s.q_full, 1);
        mbar_init(&s.img_ready, kState);
        mbar_init(&s.img_free, 1);
        mbar_init(&s.fwd_full, 1);
        mbar_init(&s.fwd_free, kState);
        mbar_init(&s.a_done, 1);
        mbar_init(&s.p_ready, kEpi);
        mbar_init(&s.vt_ready, kSplit<MODE> + (kShare<MODE> ? kState : 0));
        mbar_init(&s.s_ready[0], kState);
        mbar_init(&s.s_ready[1], kState);
        mbar_init(&s.x_done, 1);
        mbar_init(&s.o_free, kEpi + kState);
        mbar_init(&s.drain, 1);
        fence_mbar_init();
    }
    if (warp == kEpi + kState + 1) tc5::alloc(&s.tmem, kCols);
    tc5::fence_before();
    __syncthreads();
    tc5::fence_after();
    const uint32_t tm = __shfl_sync(0xffffffffu, s.tmem, 0);
    int done = 0;  // chunks this warp went through: fewer than nc after a wait that gave up
    const uint32_t trow = tm + ((uint32_t)(32 * (warp & 3)) << 16);

    // ---- V of a chunk, decayed, in bf16 terms: thread = token r, NP 16-byte pieces of its row ----
    // what token r adds decays, forwards to the chunk's end, backwards from its start
    auto weight = [&](int st, int r, int L) {
        const float2 ge = s.gate[st].G[CT - 1], gr = s.gate[st].G[r];
        return r < L ? (REV ? p.scale * start_decay(gr) : pair_decay(ge, gr)) : 0.f;
    };
    auto make = [&](auto& t, int c, int r, int q0, float wt, bool in) {
        constexpr int NP = sizeof(t) / sizeof(t[0]);
        const int st = c % NST;
        const int left = n - chunk_of(c) * CT;
        const bool again = SHORT && left <= kShort && r >= kShort && r - kShort < left;
        // of a short chunk, the piece kShort rows before the one at `at` (the swizzle is the same)
        auto twice = [&](uint32_t at) {
            uint4 v = *reinterpret_cast<const uint4*>(s.st[st].V + at - kShort * 128);
            uint32_t* const x[4] = {&v.x, &v.y, &v.z, &v.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if ((*x[e] & 0x7f80u) == 0x7f80u) *x[e] &= 0xffff0000u;
                if ((*x[e] & 0x7f800000u) == 0x7f800000u) *x[e] &= 0xffffu;
            }
            return v;
        };
        uint32_t seen = 0;
#pragma unroll
        for (int q = 0; q < NP; ++q) {
            const uint32_t at = 2 * swz<64>(r, 8 * (q0 + q));
            uint4 v = *reinterpret_cast<const uint4*>(s.st[st].V + at);
            if (!in) {  // rows past the chunk's tokens become zero, in V (for Y) and K too
                v = make_uint4(0, 0, 0, 0);
                if (MODE == 0) *reinterpret_cast<uint4*>(s.st[st].V + at) = again ? twice(at) : v;
            }
            const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float2 f = unpack_bf16(u[e]);
                if (MODE == 0) seen = seen_bf16(u[e], seen);
                mul2(f.x, f.y, f.x, f.y, wt, wt);
                uint32_t x[TERMS];
                split_bf16<TERMS>(x, f.x, f.y);
#pragma unroll
                for (int k = 0; k < TERMS; ++k) t[q][k][e] = x[k];
            }
        }
        if (MODE == 0 && !all_finite(seen)) {  // Y goes without; the state (t) does not
#pragma unroll 1
            for (int e = 0; e < 8 * NP; ++e) {
                uint16_t* v = reinterpret_cast<uint16_t*>(s.st[st].V + 2 * swz<64>(r, 8 * q0 + e));
                if ((*v & 0x7f80) == 0x7f80) {
                    *v = 0;
                    s.bad.mark(8 * q0 + e, c * CT + r);
                }
            }
        }
    };
    auto put = [&](auto& t, int r, int q0) {
        constexpr int NP = sizeof(t) / sizeof(t[0]);
#pragma unroll
        for (int q = 0; q < NP; ++q) {
            const uint32_t at = 2 * swz<64>(r, 8 * (q0 + q));
#pragma unroll
            for (int k = 0; k < TERMS; ++k)
                *reinterpret_cast<uint4*>(s.Vt[k] + at) = make_uint4(t[q][k][0], t[q][k][1], t[q][k][2], t[q][k][3]);
        }
    };
    // The warps of its own (with kShare pieces 0 .. 5 of 8, the others are the state warps'), w = 0 ..
    auto split = [&](int w) {
        constexpr int NP = kShare<MODE> ? 3 : 4;  // the first NP are made while the products still read the terms before
        const int r = 32 * (w & 3) + lane, part = w >> 2;
        for (int c = 0; c < nc; ++c) {
            const int st = c % NST, L = min(CT, n - chunk_of(c) * CT);
            if (!warp_wait(&s.gfull[st], (c / NST) & 1)) break;
            const float wt = weight(st, r, L);
            __syncwarp();
            if (lane == 0) mbar_arrive(&s.gfree[st]);
            if (!warp_wait(&s.v_full[st], (c / NST) & 1)) break;
            uint32_t t[NP][TERMS][4];
            make(t, c, r, NP * part, wt, r < L);
            if (MODE != 0) {
                __syncwarp();
                if (lane == 0) mbar_arrive(&s.v_free[st]);
            }
            if (c > 0 && !warp_wait(&s.n_done[(c - 1) % NST], ((c - 1) / NST) & 1)) break;
            put(t, r, NP * part);
            if (MODE == 0) {
                make(t, c, r, NP, wt, r < L);
                put(t, r, NP);
            }
            if (L < CT && !warp_wait(&s.full[st], (c / NST) & 1)) break;
            if (r >= L) {
#pragma unroll 1
                for (int q = part; q < DK / 8; q += kSplit<MODE> / 4)
                    *reinterpret_cast<uint4*>(s.st[st].K[q >> 3] + 2 * swz<64>(r, 8 * (q & 7))) = make_uint4(0, 0, 0, 0);
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&s.vt_ready);
            ++done;
        }
    };

    // 16 channels (from vc on) of O of chunk c: thread = query token r, as X and Y lie;
    // ein = scale e^{G_r}.  False after a wait that gave up.
    auto out = [&](int c, int r, int vc, float ein) {
        const int L = min(CT, n - chunk_of(c) * CT);
        if (!warp_wait(&s.o_done[c % NST], (c / NST) & 1)) return false;
        tc5::fence_after();
        const int bad = s.bad.any;
        float x[16], y[16];
        tc5::ld16(x, trow + TX + vc);
        tc5::ld16(y, trow + TY + vc);
        tc5::wait_ld();
        tc5::fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.o_free);
        uint32_t w[8], mine[4], got[4];
#pragma unroll
        for (int e = 0; e < 8; ++e) fma2(x[2 * e], x[2 * e + 1], ein, ein, x[2 * e], x[2 * e + 1], y[2 * e], y[2 * e + 1]);
        if (bad <= c * CT + r) {
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] = s.bad.at[vc + e] <= c * CT + r ? __uint_as_float(kNaN) : x[e];
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = pack_bf16(x[2 * e], x[2 * e + 1]);
        // lanes 2m, 2m+1 trade 16-byte pieces, so that each store instruction
        // writes whole 32-byte sectors: first row 2m, then row 2m + 1
        const bool odd = lane & 1;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            mine[e] = odd ? w[4 + e] : w[e];
            got[e] = __shfl_xor_sync(0xffffffffu, odd ? w[e] : w[4 + e], 1);
        }
        // even lanes now hold the first piece of both rows, odd lanes the second
        const uint4 a = make_uint4(mine[0], mine[1], mine[2], mine[3]);
        const uint4 b = make_uint4(got[0], got[1], got[2], got[3]);
        __nv_bfloat16* row = p.o + ((size_t)(tok0 + (long long)chunk_of(c) * CT + (r & ~1)) * p.H + h) * p.dv + vb * NB + vc + (odd ? 8 : 0);
        if ((r & ~1) < L) *reinterpret_cast<uint4*>(row) = odd ? b : a;
        if ((r | 1) < L) *reinterpret_cast<uint4*>(row + (size_t)p.H * p.dv) = odd ? a : b;
        return true;
    };

    if (warp < kEpi) {
        if constexpr (MODE == 0) {
            // ---- P: thread = query token, two warps per 32 tokens for the odd and even
            // 16-column pieces of A ------------------------------------------------
            const int blk = warp & 3, half = warp >> 2, i = 32 * blk + lane;
            float* const col = s.col[warp];
            float rf = 0.f, rd = 0.f, ein = 0.f;
            bool wide = false;
            float2 gi;
            // Decays factor about a base token b, e^{G_i - G_b} e^{G_b - G_j}: for the blocks
            // before this row's the end of the block before, so that both factors are at
            // most 1; for its own block the middle, where they stay within fp32 unless
            // half the block decays by more than 2^100.  The column factors are shared by
            // the warp's rows.
            auto factors = [&](int c) {
                const Gates& G = s.gate[c % NST];
                if (!warp_wait(&s.gfull[c % NST], (c / NST) & 1)) return false;
                gi = G.G[i];
                const float2 gm = G.G[32 * blk + 15];
                const float first = diff2(G.G[32 * blk], gm), last_ = diff2(gm, G.G[32 * blk + 31]);
                wide = !(first < 100.f && last_ < 100.f);  // the same for the whole warp
                __syncwarp();
                if (blk) {
                    const float2 gb = G.G[32 * blk - 1];
                    rf = p.scale * pair_decay(gi, gb);
#pragma unroll 1
                    for (int j = lane; j < 32 * blk; j += 32) col[j] = pair_decay(gb, G.G[j]);
                }
                rd = p.scale * ex2(diff2(gi, gm));
                col[32 * blk + lane] = ex2(diff2(gm, gi));
                __syncwarp();
                ein = p.scale * start_decay(gi);
                return true;
            };
            const uint32_t tp = trow + TP;
            if (nc > 0 && !factors(0)) done = -1;
            for (int c = 0; done == c && c < nc; ++c) {
                const int st = c % NST;
                const Gates& G = s.gate[st];
                const bool brief = SHORT && n - chunk_of(c) * CT <= kShort;
                if (!warp_wait(&s.a_done, c & 1)) break;
                tc5::fence_after();
#pragma unroll 1
                for (int J = half; J < 2 * blk + 2; J += 2) {  // 16 columns
                    float a[16];
                    uint32_t pk[8];
                    tc5::ld16(a, trow + TA + 16 * J);
                    tc5::wait_ld();
                    const bool diag = J >= 2 * blk;
                    const float f = diag ? rd : rf;
                    if (diag && wide) {  // pair by pair
#pragma unroll
                        for (int q = 0; q < 16; ++q) {
                            const float d = p.scale * pair_decay(gi, G.G[16 * J + q]);
                            a[q] = 16 * J + q <= i ? a[q] * d : 0.f;
                        }
                    } else {
                        const float4* cf = reinterpret_cast<const float4*>(col + 16 * J);
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            float4 w = cf[q];
                            mul2(w.x, w.y, w.x, w.y, f, f);
                            mul2(w.z, w.w, w.z, w.w, f, f);
                            mul2(a[4 * q], a[4 * q + 1], a[4 * q], a[4 * q + 1], w.x, w.y);
                            mul2(a[4 * q + 2], a[4 * q + 3], a[4 * q + 2], a[4 * q + 3], w.z, w.w);
                        }
                        if (diag) {
#pragma unroll
                            for (int q = 0; q < 16; ++q) a[q] = 16 * J + q <= i ? a[q] : 0.f;
                        }
                    }
#pragma unroll
                    for (int q = 0; q < 8; ++q) pk[q] = pack_bf16(a[2 * q], a[2 * q + 1]);
                    tc5::st8(tp + 8 * J, pk);
                    if (brief && J < 4) {
#pragma unroll
                        for (int q = 0; q < 8; ++q) pk[q] = rest_bf16(pk[q], a[2 * q], a[2 * q + 1]);
                        tc5::st8(tp + 8 * J + 32, pk);
                    }
                }
                {   // (of a short chunk, rows past its tokens may hold anything)
                    const uint32_t zero[8] = {};
#pragma unroll 1
                    for (int J = 2 * blk + 2 + half; J < 8; J += 2)
                        if (!brief || (J & 3) >= 2 * blk + 2) tc5::st8(tp + 8 * J, zero);
                }
                tc5::wait_st();
                tc5::fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&s.p_ready);
                    mbar_arrive(&s.gfree[st]);
                }
                const float e = ein;
                if (c + 1 < nc && !factors(c + 1)) break;  // while the products make Y
                if (!out(c, i, 32 * half + 16, e)) break;
                ++done;
            }
        }
        if constexpr (MODE != 0) split(warp);
    } else if (warp < kEpi + kState) {
        // ---- the state: thread = key channel r, value channels 32 half .. +31 ------
        // (and, to split V, thread = token r of the same channels)
        const int half = (warp - kEpi) >> 2, r = 32 * (warp & 3) + lane;
        const bool own = r < DK;
        float S[32];
        const float* h0 = MODE != 1 && p.h0 && own ? p.h0 + (chain * p.dv + vb * NB + 32 * half) * DK + r : nullptr;
#pragma unroll
        for (int e = 0; e < 32; ++e) S[e] = h0 ? h0[(size_t)e * DK] : 0.f;
        if (MODE != 1 && own) {
#pragma unroll 1
            for (int q = 0; q < run; ++q) {  // what the runs before this one leave
                const float a = p.runG[(size_t)(first + q) * p.H + h];
                const float* N = p.runS + (((size_t)(first + q) * p.H + h) * gridDim.y + vb) * slab + (size_t)(32 * half) * DK + r;
#pragma unroll
                for (int e = 0; e < 32; ++e) S[e] = a * S[e] + N[(size_t)e * DK];
            }
        }
        bool ok = true;
        float total = 1.f, decay = 1.f, ein = 0.f;
        auto add_n = [&](int c) {  // S <- e^{G_last} S + N(c), N in one accumulator per term of V
#pragma unroll 1
            for (int x = 0; x < TERMS; ++x) {
                float N[32];
                tc5::ld32(N, trow + tn<MODE>(c) + NB * x + 32 * half);
                tc5::wait_ld();
                const float a = x ? 1.f : total;
#pragma unroll
                for (int e = 0; e < 32; e += 2) fma2(S[e], S[e + 1], a, a, S[e], S[e + 1], N[e], N[e + 1]);
            }
            tc5::fence_before();
        };
        for (int c = 0; c < nc; ++c) {
            const int st = c % NST, L = min(CT, n - chunk_of(c) * CT);
            float next_ein = 0.f, next_total = 0.f;
            uint32_t t[1][TERMS][4];
            if constexpr (kShare<MODE>) {
                if (!(ok = warp_wait(&s.gfull[st], (c / NST) & 1))) break;
                if (MODE == 0) next_ein = p.scale * start_decay(s.gate[st].G[r]);
                next_total = start_decay(s.gate[st].G[CT - 1]);
                const float wt = weight(st, r, L);
                __syncwarp();
                if (lane == 0) mbar_arrive(&s.gfree[st]);
                if (!(ok = warp_wait(&s.v_full[st], (c / NST) & 1))) break;
                make(t, c, r, 6 + half, wt, r < L);
                if (MODE != 0) {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&s.v_free[st]);
                }
            }
            if (c > 0) {  // S entering chunk c; X(c-1), which read the last one, came before N(c-1)
                if (!(ok = warp_wait(&s.n_done[(c - 1) % NST], ((c - 1) / NST) & 1))) break;
                tc5::fence_after();
            }
            if constexpr (kShare<MODE>) {
                put(t, r, 6 + half);
                fence_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&s.vt_ready);
            }
            if (c > 0) add_n(c - 1);
            if constexpr (MODE == 0) {
                if (own) {
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        *reinterpret_cast<uint4*>(s.S[0] + 2 * swz<64>(r, 32 * half + 8 * q)) =
                            make_uint4(pack_bf16(S[8 * q], S[8 * q + 1]), pack_bf16(S[8 * q + 2], S[8 * q + 3]),
                                       pack_bf16(S[8 * q + 4], S[8 * q + 5]), pack_bf16(S[8 * q + 6], S[8 * q + 7]));
                }
                fence_async_smem();
            }
            // N(c-1) is in the registers (and, MODE 0, S where X finds it)
            __syncwarp();
            if (lane == 0) mbar_arrive(&s.s_ready[c & 1]);
            if (MODE == 0 && c > 0 && !(ok = out(c - 1, r, 32 * half, ein))) break;
            if constexpr (kShare<MODE>) {
                ein = next_ein;
                total = next_total;
                decay *= total;
            } else {
                if (!(ok = warp_wait(&s.gfull[st], (c / NST) & 1))) break;
                total = start_decay(s.gate[st].G[CT - 1]);
                __syncwarp();
                if (lane == 0) mbar_arrive(&s.gfree[st]);
            }
            if constexpr (MODE == 2) {
                if (REV) {
                    // <S, dS> of the chunk: this thread's part of both
                    float2 d2 = make_float2(0.f, 0.f);
                    if (!(ok = warp_wait(&s.fwd_full, c & 1))) break;
                    if (own) {
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const uint32_t at = 2 * swz<64>(r, 32 * half + 8 * q);
                            const uint4 a = *reinterpret_cast<const uint4*>(s.S[0] + at), b = *reinterpret_cast<const uint4*>(s.S[MODE == 2] + at);
                            const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const float2 f = join_halves(x[e], y[e]);
                                fma2(d2.x, d2.y, S[8 * q + 2 * e], S[8 * q + 2 * e + 1], f.x, f.y, d2.x, d2.y);
                            }
                        }
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&s.fwd_free);
                    float d = d2.x + d2.y;
                    d = warp_sum(d);
                    if (lane == 0) s.col[warp - kEpi][c & 1] = total * d;
                }
                if (c > 0 && !(ok = warp_wait(&s.img_free, (c - 1) & 1))) break;
                if (own) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        uint2 t[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) t[e] = halves(S[8 * q + 2 * e], S[8 * q + 2 * e + 1]);
                        unsigned char* at = (unsigned char*)s.Q + 2 * swz<64>(r, 32 * half + 8 * q);
                        *reinterpret_cast<uint4*>(at) = make_uint4(t[0].x, t[1].x, t[2].x, t[3].x);
                        *reinterpret_cast<uint4*>(at + DK * 128) = make_uint4(t[0].y, t[1].y, t[2].y, t[3].y);
                    }
                }
                fence_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&s.img_ready);
            }
            ++done;
        }
        if (ok && nc > 0) {
            if (MODE == 0 && !out(nc - 1, r, 32 * half, ein)) --done;
            if (warp_wait(&s.n_done[(nc - 1) % NST], ((nc - 1) / NST) & 1)) {
                tc5::fence_after();
                add_n(nc - 1);
            }
        }
        if (own) {
            float* to = nullptr;
            if (MODE == 1) to = p.runS + (((size_t)(first + run) * p.H + h) * gridDim.y + vb) * slab + (size_t)(32 * half) * DK + r;
            else if (last && p.hT) to = p.hT + (chain * p.dv + vb * NB + 32 * half) * DK + r;
            if (to) {
#pragma unroll
                for (int e = 0; e < 32; ++e) to[(size_t)e * DK] = S[e];
            }
        }
        if (MODE == 1 && vb == 0 && warp == kEpi && lane == 0) p.runG[(size_t)(first + run) * p.H + h] = decay;
    } else if (warp == kEpi + kState) {
        // ---- loads -----------------------------------------------------------
        if (lane == 0) {
            int nk = 0, nv = 0, nq = 0;  // copies begun
            for (int c = 0; c < nc; ++c) {
                // each operand goes in as soon as the products are done with the last in its place
                const int st = c % NST, ph = (c / NST - 1) & 1;
                auto& q = s.st[st];
                const int tok = (int)(tok0 + (long long)chunk_of(c) * CT), kh = h / p.rep;
                if (MODE != 0) {
                    if (c >= NST && !wait_for(&s.v_free[st], ph)) break;
                    mbar_arrive_expect(&s.v_full[st], PANEL);
                    tma_load_3d(q.V, &p.vmap, vb * NB, h, tok, &s.v_full[st]);
                    nv = c + 1;
                }
                if (c >= NST && !wait_for(&s.n_done[st], ph)) break;
                mbar_arrive_expect(&s.full[st], DK / 64 * PANEL);
#pragma unroll
                for (int x = 0; x < DK / 64; ++x) tma_load_3d(q.K[x], &p.kmap, 64 * x, kh, tok, &s.full[st]);
                nk = c + 1;
                if (MODE == 0) {
                    if (c >= NST && !wait_for(&s.o_done[st], ph)) break;
                    mbar_arrive_expect(&s.v_full[st], PANEL);
                    tma_load_3d(q.V, &p.vmap, vb * NB, h, tok, &s.v_full[st]);
                    nv = c + 1;
                }
                if constexpr (MODE == 2 && REV) {
                    if (c > 0 && !wait_for(&s.fwd_free, (c - 1) & 1)) break;
                    const size_t term = gridDim.y * (size_t)(DK * 128);
                    const unsigned char* from = reinterpret_cast<const unsigned char*>(p.other) +
                                                ((slot0 + chunk_of(c)) * p.H + h) * (2 * term) + vb * (size_t)(DK * 128);
                    mbar_arrive_expect(&s.fwd_full, 2 * DK * 128);
                    bulk_g2s(s.S[0], from, DK * 128, &s.fwd_full);
                    bulk_g2s(s.S[1], from + term, DK * 128, &s.fwd_full);
                    nq = c + 1;
                }
                if constexpr (MODE == 0) {
                    if (c > 0 && !wait_for(&s.x_done, (c - 1) & 1)) break;
                    mbar_arrive_expect(&s.q_full, DK / 64 * PANEL);
#pragma unroll
                    for (int x = 0; x < DK / 64; ++x) tma_load_3d(s.Q[x], &p.qmap, 64 * x, kh, tok, &s.q_full);
                    nq = c + 1;
                }
                ++done;
            }
            // no copy may be in flight when the CTA ends
            for (int d = max(0, nk - NST); d < nk; ++d) wait_for(&s.full[d % NST], (d / NST) & 1);
            for (int d = max(0, nv - NST); d < nv; ++d) wait_for(&s.v_full[d % NST], (d / NST) & 1);
            if (nq) wait_for(MODE == 0 ? &s.q_full : &s.fwd_full, (nq - 1) & 1);
        }
    } else if (warp == kEpi + kState + 1) {
        // ---- products: the warp stays together, one lane issues ----------------
        constexpr uint32_t ID_A = tc5::idesc_bf16(128, 128, false, false);
        constexpr uint32_t ID_X = tc5::idesc_bf16(128, NB, false, true);
        constexpr uint32_t ID_N = tc5::idesc_bf16(128, TERMS * NB, true, true);
        // descriptors of step 0; a K step is 32 bytes along 64-channel rows (then the
        // next panel), or 16 rows down a tile
        constexpr uint64_t KROWS = (16 * 128) >> 4, KCOLS = 32 >> 4, KPANEL = PANEL >> 4;
        const uint64_t dVt = tc5::mnmajor(smem_u32(s.Vt), 0, PANEL), dS = tc5::mnmajor(smem_u32(s.S), 0, PANEL);
        const uint64_t dQ = tc5::kmajor<CT>(smem_u32(s.Q), 0);
        for (int c = 0; c < nc; ++c) {
            const int st = c % NST;
            const uint64_t dK = tc5::kmajor<CT>(smem_u32(s.st[st].K), 0);
            const uint64_t dKt = tc5::mnmajor(smem_u32(s.st[st].K), 0, PANEL), dV = tc5::mnmajor(smem_u32(s.st[st].V), 0, PANEL);
            if constexpr (MODE == 0) {
                // A(c) goes where A(c-1) was, which P(c-1) is made of: p_ready came before Y(c-1)
                if (!warp_wait(&s.full[st], (c / NST) & 1)) break;
                if (!warp_wait(&s.q_full, c & 1)) break;
                tc5::fence_after();
                if (elect_one()) {
#pragma unroll 2
                    for (int k = 0; k < DK / 16; ++k) {
                        const uint64_t at = (k >> 2) * KPANEL + (k & 3) * KCOLS;
                        tc5::mma(tm + TA, dQ + at, dK + at, ID_A, k > 0);
                    }
                    tc5::commit(&s.a_done);
                }
                __syncwarp();
                if (!warp_wait(&s.s_ready[c & 1], (c >> 1) & 1)) break;
                if (c > 0 && !warp_wait(&s.o_free, (c - 1) & 1)) break;
                tc5::fence_after();
                if (elect_one()) {
#pragma unroll 2
                    for (int k = 0; k < DK / 16; ++k)
                        tc5::mma(tm + TX, dQ + (k >> 2) * KPANEL + (k & 3) * KCOLS, dS + k * KROWS, ID_X, k > 0);
                    tc5::commit(&s.x_done);
                }
                __syncwarp();
            }
            // N(c); with 64 key channels lanes 64-127 read the V tile behind K and are ignored
            // (MODE 1, 2: where N(c-2) was, which is in the registers once S entering c - 1 is)
            if (MODE != 0 && !warp_wait(&s.full[st], (c / NST) & 1)) break;
            if (MODE != 0 && c > 0 && !warp_wait(&s.s_ready[(c - 1) & 1], ((c - 1) >> 1) & 1)) break;
            if (!warp_wait(&s.vt_ready, c & 1)) break;
            tc5::fence_after();
            if (elect_one()) {
#pragma unroll 2
                for (int k = 0; k < CT / 16; ++k) tc5::mma(tm + tn<MODE>(c), dKt + k * KROWS, dVt + k * KROWS, ID_N, k > 0);
                tc5::commit(&s.n_done[st]);
            }
            __syncwarp();
            if constexpr (MODE == 0) {
                if (!warp_wait(&s.p_ready, c & 1)) break;
                tc5::fence_after();
                if (elect_one()) {
#pragma unroll 2
                    for (int k = 0; k < CT / 16; ++k) tc5::mma_ts(tm + TY, tm + TP + 8 * k, dV + k * KROWS, ID_X, k > 0);
                    tc5::commit(&s.o_done[st]);
                }
                __syncwarp();
            }
            ++done;
        }
        if (elect_one()) tc5::commit(&s.drain);  // no product may be in flight when the CTA ends
        warp_wait(&s.drain, 0);
    } else if (MODE == 0 && warp > kEpi + kState + 2) {
        split(warp - (kEpi + kState + 3));
    } else if (MODE == 2 && warp > kEpi + kState + 2) {
        // ---- the states' images to memory, and the sums of <S, dS> -------------------
        for (int c = 0; c < nc; ++c) {
            if (!warp_wait(&s.img_ready, c & 1)) break;
            if (REV) {
                float d = lane < kState ? s.col[lane][c & 1] : 0.f;
                d = warp_sum(d);
                if (lane == 0) p.cross[(vb * (size_t)chunk_slots(p.seq, CT) + slot0 + chunk_of(c)) * p.H + h] = d;
            }
            if (lane == 0) {
                unsigned char* to = reinterpret_cast<unsigned char*>(p.image) +
                                    ((slot0 + chunk_of(c)) * p.H + h) * (2 * gridDim.y * (size_t)(DK * 128)) + vb * (size_t)(DK * 128);
                bulk_s2g(to, s.Q, DK * 128);
                bulk_s2g(to + gridDim.y * (size_t)(DK * 128), (unsigned char*)s.Q + DK * 128, DK * 128);
                bulk_commit();
                bulk_wait_read<0>();
                mbar_arrive(&s.img_free);
            }
            __syncwarp();
            ++done;
        }
        if (lane == 0) bulk_wait<0>();
    } else {
        // ---- gates: the next two chunks' values are on their way while this one's wait ----
        float xa[4], xb[4];
        auto load = [&](float (&x)[4], int c) {
            if (c < nc) load_gates(x, p.g + (size_t)(tok0 + (long long)chunk_of(c) * CT) * p.H + h, p.H, min(CT, n - chunk_of(c) * CT));
        };
        auto form = [&](float (&x)[4], int c) {
            const int st = c % NST;
            if (c >= NST && !warp_wait(&s.gfree[st], ((c / NST) - 1) & 1)) return false;
            form_gates(s.gate[st], x);
            __syncwarp();
            if (lane == 0) mbar_arrive(&s.gfull[st]);
            load(x, c + 2);
            ++done;
            return true;
        };
        load(xa, 0);
        load(xb, 1);
        for (int c = 0; c < nc && form(xa, c) && (c + 1 == nc || form(xb, c + 1)); c += 2) {}
    }
    if (lane == 0 && done < nc) atomicOr(p.status, 1u);
    tc5::fence_before();
    __syncthreads();
    if (warp == kEpi + kState + 1) {
        tc5::fence_after();
        tc5::dealloc(tm, kCols);
    }
}

// Runs per chain: 1 when the chains fill the device; otherwise the number that
// gives the shortest estimated time, in chunk steps on the critical path.  A
// step of the walk costs about 1, one of the map (MODE 1) about 0.7, the second launch
// about 4, and adding up what the runs before leave 0.2 each.  Packed sequences have
// rows / length + nseq runs together, however long the longest is.  (16 heads of 8192
// tokens: 4 runs 81 us, 1 run 169 us.  9 packed sequences of up to 968 tokens, 8 heads:
// runs of 3 chunks 33 us, whole chains 29 us.)
struct Cut {
    int runs, len;
};
Cut cut_of(const Problem& p) {
    const int chunks = ((p.seq.cu ? p.seq.rows : p.seq.len) + CT - 1) / CT, nseq = p.seq.nseq;
    const long long heads = (long long)p.H * (p.dv / NB);
    Cut best{1, std::max(chunks, 1)};
    auto waves = [](long long n) { return (double)((n + 147) / 148); };
    double cost = ceil(longest(p.seq) / CT) * waves(heads * nseq);
    for (int r = 2; r <= 64 && r <= chunks; ++r) {
        const int len = (chunks + r - 1) / r, runs = (chunks + len - 1) / len;
        const long long all = heads * items(p.seq, runs, len * CT), maps = p.seq.cu ? all : all - heads * nseq;
        const double c = len * (waves(all) + 0.7 * waves(maps)) + 4 + 0.2 * runs;
        if (c < 0.9 * cost) {
            cost = c;
            best = Cut{runs, len};
        }
    }
    return best;
}

template <int MODE, bool REV, bool SHORT = false>
void launch(const Params& a, int dk, dim3 grid, cudaStream_t st) {
    auto go = [&](auto d) {
        constexpr int DK = decltype(d)::value;
        const int smem = sizeof(Smem<DK, MODE>) + 1024;
        cudaFuncSetAttribute(decay_tc_walk_kernel<DK, MODE, REV, SHORT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        GDN_LAUNCH(MODE == 0 ? "decay_tc_walk" : MODE == 1 ? "decay_tc_map" : "decay_tc_states", st,
                   (decay_tc_walk_kernel<DK, MODE, REV, SHORT><<<grid, kThreads<MODE>, smem, st>>>(a)));
    };
    if (dk == 64) go(std::integral_constant<int, 64>{});
    else go(std::integral_constant<int, 128>{});
}

// Workspace of the runs, after `base` bytes: their states and decays.
size_t runs_bytes(const Problem& p, const Cut& c) {
    if (c.runs == 1) return 0;
    const size_t n = (size_t)items(p.seq, c.runs, c.len * CT) * p.H;
    return n * p.dk * p.dv * 4 + ((n * 4 + 255) & ~(size_t)255);
}

Params params_of(const Problem& p, const Cut& c, const float* g, void* runs, void* ws) {
    Params a{};
    a.seq = p.seq; a.H = p.H; a.rep = p.H / p.Hk; a.dv = p.dv; a.scale = p.scale;
    a.g = g;
    a.runs = c.runs; a.len = c.len;
    a.status = (unsigned int*)ws;
    a.runS = (float*)runs;
    a.runG = a.runS + (size_t)items(p.seq, c.runs, c.len * CT) * p.H * p.dk * p.dv;
    return a;
}

// All runs of a call: with more than one, first what each leaves.
template <int MODE, bool REV>
void launch_runs(const Params& a, const Problem& p, cudaStream_t st) {
    const auto grid = [&](int runs) { return dim3((unsigned)(items(p.seq, runs, a.len * CT) * p.H), p.dv / NB); };
    if (a.runs > 1) launch<1, REV>(a, p.dk, p.seq.cu ? grid(a.runs) : grid(a.runs - 1), st);
    if (MODE == 0 && short_sequences(p)) launch<MODE, REV, MODE == 0>(a, p.dk, grid(a.runs), st);
    else launch<MODE, REV>(a, p.dk, grid(a.runs), st);
}

}  // namespace

// The dims that fill whole 64-channel panels; the products of smaller ones would be
// padding for the most part.  (16 heads of 8192 tokens, 128 x 128: 84 us here and 767 us
// on CUDA cores; the 350M-scale training step 258 us and 2.9 ms.  Of few tokens too: 4 tokens
// of 8 heads, 128 x 128, 21 us and 26 us, their backward 42 and 75; 64 x 64, 21 and 22.)
bool tc_supported(const Problem& p) {
    return p.dtype == GDN_BF16 && (p.dk == 64 || p.dk == 128) && (p.dv == 64 || p.dv == 128);
}

size_t tc_fwd_workspace(const Problem& p) { return kStatusBytes + runs_bytes(p, cut_of(p)); }

bool launch_tc_fwd(const Problem& p, const void* q, const void* k, const void* v, const float* g, const float* h0,
                   void* o, float* hT, void* ws, cudaStream_t st) {
    Params a = params_of(p, cut_of(p), g, (char*)ws + kStatusBytes, ws);
    if (!encode_head_map(&a.qmap, q, p.seq.rows, p.Hk, p.dk, CT) || !encode_head_map(&a.kmap, k, p.seq.rows, p.Hk, p.dk, CT) ||
        !encode_head_map(&a.vmap, v, p.seq.rows, p.H, p.dv, CT))
        return false;
    a.h0 = h0; a.o = (__nv_bfloat16*)o; a.hT = hT;
    launch_runs<0, false>(a, p, st);
    return true;
}

size_t tc_states_workspace(const Problem& p) { return runs_bytes(p, cut_of(p)); }

bool launch_tc_states(const Problem& p, const void* q, const void* k, const void* v, const float* g, const float* h0,
                      const void* dO, const float* dhT, float* dh0, void* S, void* dS, float* cross, void* runs, void* ws,
                      cudaStream_t st) {
    Params a = params_of(p, cut_of(p), g, runs, ws), b = a;
    if (!encode_head_map(&a.kmap, k, p.seq.rows, p.Hk, p.dk, CT) || !encode_head_map(&a.vmap, v, p.seq.rows, p.H, p.dv, CT) ||
        !encode_head_map(&b.kmap, q, p.seq.rows, p.Hk, p.dk, CT) || !encode_head_map(&b.vmap, dO, p.seq.rows, p.H, p.dv, CT))
        return false;
    a.h0 = h0; a.image = (__nv_bfloat16*)S;
    launch_runs<2, false>(a, p, st);
    b.h0 = dhT; b.hT = dh0; b.image = (__nv_bfloat16*)dS;
    b.other = (const __nv_bfloat16*)S; b.cross = cross;
    launch_runs<2, true>(b, p, st);
    return true;
}

}  // namespace decay
}  // namespace gdn
