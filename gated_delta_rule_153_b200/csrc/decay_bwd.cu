// decay_bwd.cu -- backward of linear attention with a decay per head on the
// fifth-generation tensor cores: the gradients of each 128-token chunk, given the
// state S entering it and the gradient dS of the state leaving it (decay_walk.cu).
//
// With D_ij = e^{G_i - G_j} (i >= j), per chunk and head:
//     dq = scale [ (D .* dO V^T) K + diag(e^G) dO S ]
//     dk = scale (D .* dO V^T)^T Q + diag(e^{G_last - G}) V dS
//     dv = scale (D .* Q K^T)^T dO + diag(e^{G_last - G}) K dS^T
// (S and dS as [key channel][value channel]).  The gate: M_ij = scale D_ij (q_i.k_j)
// (dO_i.v_j) is what the pair adds to <dO, o>; with r_i, c_j its row and column
// sums without the diagonal, a_i = q_i . (state part of dq_i) and b_j = k_j . (state
// part of dk_j),
//     dg_t = sum_{i >= t} (r_i - c_i) + sum_{i >= t} a_i + sum_{j < t} b_j + e^{G_last} <S, dS>:
// every pair of tokens before t and from t on, within the chunk, across its start,
// across its end, and over it.  dg is fp32, so M is taken from fp32 accumulators, and S
// and dS enter the products behind a and b as three bf16 terms, exact to fp32 (dv takes two
// of dS); D .* dO V^T and D .* Q K^T are rounded to bf16 once, as dq, dk and dv themselves
// are.  With SHORT, in a chunk of up to 64 tokens, where few roundings average out, the other
// half of these operands holds what the rounding left, over the same rows of K, Q and dO
// once more.
//
// One CTA per SM takes the chunk-heads in turn.  A chunk runs in two halves, the
// first with the query token on the tensor-memory lanes, the second with the key
// token, since each product wants its left operand's rows there:
//     Q K^T, dO V^T, dO S  -> dq, r, a        K Q^T, V dO^T, V dS, K dS^T  -> dk, dv, c, b
// The state parts are scaled in place and the other products accumulate onto them.
// Sixteen warps do the elementwise work (four per 32 tokens, a quarter of the columns
// each) and split the states; one issues loads and products; one forms the gates and sums
// dg.  Loads of the next chunk start as each operand is done with.
//
// What bounds it, at 8 x 2048 tokens of 8 heads, dk = dv = 128 (1,024 chunk-heads, seven
// per SM): 127 us, 18 us a chunk, 2.8 TB/s of DRAM traffic (361 MB, S and dS are 134 of
// them) with the tensor pipe busy for 28 %.  The four rounds of products and elementwise
// work of a chunk wait for one another, and shared memory (230 KB) and tensor memory
// (all 512 columns) hold one chunk.  With S and dS in two bf16 terms from memory it took 106
// us, dg off by 3e-6: of the 21 us the split is 9, its products 4, the two hand-offs 8.
// Splitting fp32 states from memory took 144 us, three terms from memory 134 us here and
// 40 us more in the walks.  Results leave by TMA from shared memory.
#include "decay_tc.cuh"

namespace gdn {
namespace decay {
namespace {

constexpr int PANEL = CT * 128;  // bytes of a 128-row, 64-channel tile
constexpr int kEpi = 16;
constexpr int kThreads = 32 * (kEpi + 2);

template <int DK, int DV>
struct alignas(1024) Smem {
    unsigned char Q[DK / 64][PANEL], K[DK / 64][PANEL], V[DV / 64][PANEL], Y[DV / 64][PANEL];  // Y = dO
    // S, then dS: the upper halves, which are the first bf16 term, and the lower halves.  Once
    // the first term is done with, the third and the second come in their places.
    unsigned char S[2][DV / 64][DK * 128];
    // Results on their way out: dq, then dk and dv, each once the store before it has read
    // its source.  At the largest dims they go by way of S: dq through the second place,
    // between its last use and the arrival of dS's, dk and dv through both, between dS and
    // the next chunk's S, which only the second products of that chunk need.
    static constexpr bool kOwnOut = DK + DV < 256;
    unsigned char O[kOwnOut ? (DK + DV) / 64 : 1][kOwnOut ? PANEL : 16];
    GDN_DEV unsigned char* out_q() { return kOwnOut ? O[0] : S[1][0]; }
    GDN_DEV unsigned char* out_k() { return kOwnOut ? O[0] : S[0][0]; }
    GDN_DEV unsigned char* out_v() { return out_k() + DK / 64 * PANEL; }
    Gates gate[2];
    float r[2][4][CT], c[2][4][CT], a[2][4][CT], b[2][4][CT];  // [chunk parity][column quarter][token]
    float col[kEpi][2][16];
    uint64_t t_full, kv_full, s_full[2], s_read, s_ready, gfull[2], zeroed, a_done, x_done, e1, q_done, e2, a2_done, x2_done, v_done, e3r,
        e3[2], o_done, e4, drain;
    uint32_t tmem;
};

struct Params {
    CUtensorMap qmap, kmap, vmap, ymap, dqmap, dkmap, dvmap;
    Seqs seq;
    int H, rep;
    float scale;
    const float* g;
    const unsigned char *S, *dS;
    const float* cross;
    void *dq, *dk;   // bf16, or fp32 parts per value head when rep > 1
    __nv_bfloat16* dv;
    float* dg;
    unsigned int* status;
};

// The chunk of slot x: its sequence is the last whose first slot is at most x.
struct Chunk {
    long long tok;
    int L;
};
GDN_DEV bool chunk_of_slot(const Seqs& q, long long slot, Chunk& c) {
    int lo = 0, hi = q.nseq - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        const long long first = (q.cu ? (long long)q.cu[mid] : (long long)mid * q.len) / CT + mid;
        if (first <= slot) lo = mid;
        else hi = mid - 1;
    }
    long long tok0;
    int n;
    if (!span_of(q, lo, tok0, n)) return false;
    const long long k = slot - (tok0 / CT + lo);
    if (k < 0 || k * CT >= n) return false;
    c.tok = tok0 + k * CT;
    c.L = (int)min((long long)CT, n - k * CT);
    return true;
}

// Columns c0 .. c0 + N - 1 of a row in the two-lane trade of decay_walk.cu: whole 32-byte
// sectors per store.  row0: the even row's address; w: this lane's packed row.
template <int NW>
GDN_DEV void store_rows(__nv_bfloat16* row0, size_t next, const uint32_t (&w)[NW], bool up, bool dn) {
    const bool odd = threadIdx.x & 1;
#pragma unroll
    for (int q = 0; q < NW / 8; ++q) {
        uint32_t mine[4], got[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            mine[e] = odd ? w[8 * q + 4 + e] : w[8 * q + e];
            got[e] = __shfl_xor_sync(0xffffffffu, odd ? w[8 * q + e] : w[8 * q + 4 + e], 1);
        }
        const uint4 a = make_uint4(mine[0], mine[1], mine[2], mine[3]);
        const uint4 b = make_uint4(got[0], got[1], got[2], got[3]);
        __nv_bfloat16* at = row0 + 16 * q + (odd ? 8 : 0);
        if (up) *reinterpret_cast<uint4*>(at) = odd ? b : a;
        if (dn) *reinterpret_cast<uint4*>(at + next) = odd ? a : b;
    }
}

// tensor-memory columns.  First half: Q K^T, dO V^T, dq, the bf16 operand of dq.  Second:
// K Q^T and V dO^T (their bf16 operands over them), dk, dv.
constexpr uint32_t TA = 0, TB = 128, TX = 256, TP = 384, TV = 384;

template <int DK, int DV, bool SHORT>
__global__ void __launch_bounds__(kThreads, 1)
decay_tc_bwd_kernel(const __grid_constant__ Params p) {
    extern __shared__ __align__(1024) unsigned char raw[];
    Smem<DK, DV>& s = *reinterpret_cast<Smem<DK, DV>*>(align1k(raw));
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const long long slots = chunk_slots(p.seq, CT), units = slots * p.H;
    if (tid == 0) {
        for (uint64_t* b : {&s.t_full, &s.kv_full, &s.s_full[0], &s.s_full[1], &s.s_read, &s.gfull[0], &s.gfull[1], &s.a_done, &s.x_done,
                            &s.q_done, &s.a2_done, &s.x2_done, &s.v_done, &s.o_done, &s.drain})
            mbar_init(b, 1);
        for (uint64_t* b : {&s.zeroed, &s.e1, &s.e2, &s.e3r, &s.e3[0], &s.e3[1], &s.e4, &s.s_ready}) mbar_init(b, kEpi);
        fence_mbar_init();
    }
    if (warp == kEpi) tc5::alloc(&s.tmem, 512);
    tc5::fence_before();
    __syncthreads();
    tc5::fence_after();
    const uint32_t tm = __shfl_sync(0xffffffffu, s.tmem, 0);
    bool ok = true;
    int x = 0;  // chunks so far
    Chunk ch;
    constexpr int QK = DK / 4, QV = DV / 4;  // columns of a quarter

    if (warp < kEpi) {
        const int blk = warp & 3, qt = warp >> 2, i = 32 * blk + lane;
        const uint32_t trow = tm + ((uint32_t)(32 * blk) << 16);
        // The second and third terms of a state (0: S, 1: dS), each where this thread reads
        auto split_state = [&](int which) {
            if (!warp_wait(&s.s_full[0], which) || !warp_wait(&s.s_full[1], which)) return false;
            if (!warp_wait(&s.s_read, which)) return false;  // the products are done with the first
#pragma unroll
            for (int q = 0; q < DK * DV / (8 * 32 * kEpi); ++q) {
                uint4 *up = reinterpret_cast<uint4*>(s.S[0]) + tid + 32 * kEpi * q, *low = reinterpret_cast<uint4*>(s.S[1]) + tid + 32 * kEpi * q;
                const uint4 a = *up, b = *low;
                uint4 t2, t3;
                split_rest(t2.x, t3.x, a.x, b.x);
                split_rest(t2.y, t3.y, a.y, b.y);
                split_rest(t2.z, t3.z, a.z, b.z);
                split_rest(t2.w, t3.w, a.w, b.w);
                *low = t2;
                *up = t3;
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&s.s_ready);
            return true;
        };
        for (long long u = blockIdx.x; ok && u < units; u += gridDim.x) {
            const int h = (int)(u % p.H);
            if (!chunk_of_slot(p.seq, u / p.H, ch)) continue;
            const int ph = x & 1, L = ch.L;
            const bool brief = SHORT && L <= CT / 2;
            const Gates& G = s.gate[ph];
            if (!(ok = warp_wait(&s.t_full, ph)) || !(ok = warp_wait(&s.kv_full, ph))) break;
            if (L < CT) {
                // rows past the chunk's tokens become zero: the products sum over tokens
                // (of a short chunk, K, Q and dO have a row again where its rest is: same swizzle)
                if (i >= L) {
                    const bool again = brief && i >= CT / 2 && i - CT / 2 < L;
                    const uint4 zero = make_uint4(0, 0, 0, 0);
                    auto fill = [&](unsigned char* row) {
                        *reinterpret_cast<uint4*>(row) = again ? *reinterpret_cast<const uint4*>(row - CT / 2 * 128) : zero;
                    };
#pragma unroll 1
                    for (int q = qt; q < DK / 8; q += 4) {
                        fill(s.Q[q >> 3] + 2 * swz<64>(i, 8 * (q & 7)));
                        fill(s.K[q >> 3] + 2 * swz<64>(i, 8 * (q & 7)));
                    }
#pragma unroll 1
                    for (int q = qt; q < DV / 8; q += 4) {
                        *reinterpret_cast<uint4*>(s.V[q >> 3] + 2 * swz<64>(i, 8 * (q & 7))) = zero;
                        fill(s.Y[q >> 3] + 2 * swz<64>(i, 8 * (q & 7)));
                    }
                }
                fence_async_smem();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&s.zeroed);
            if (!(ok = warp_wait(&s.gfull[ph], (x >> 1) & 1))) break;
            // ---- first half: lane = query token i ------------------------------------
            // (a piece: 16 columns; pieces qt and qt + 4 of the eight)
            const float2 gi = G.G[i];
            {
                float rf = 0.f;
                if (blk) {
                    const float2 gb = G.G[32 * blk - 1];
                    rf = p.scale * pair_decay(gi, gb);
                    const int j = 16 * (qt + 4 * (lane >> 4)) + (lane & 15);
                    s.col[warp][lane >> 4][lane & 15] = j < 32 * blk ? pair_decay(gb, G.G[j]) : 0.f;
                    __syncwarp();
                }
                if (!(ok = warp_wait(&s.a_done, ph))) break;
                // the operand goes where dv of the chunk before was
                if (x > 0 && !(ok = warp_wait(&s.e4, ph ^ 1))) break;
                tc5::fence_after();
                float rs = 0.f;
#pragma unroll 1
                for (int z = 0; z < (brief ? 1 : 2); ++z) {
                    const int J = qt + 4 * z, j0 = 16 * J;
                    uint32_t pk[8], rest[8] = {};
                    if (J < 2 * blk + 2) {
                        float A[16], B[16];
                        tc5::ld16(A, trow + TA + j0);
                        tc5::ld16(B, trow + TB + j0);
                        tc5::wait_ld();
                        if (J < 2 * blk) {
#pragma unroll
                            for (int e = 0; e < 16; ++e) {
                                B[e] *= rf * s.col[warp][z][e];
                                rs += A[e] * B[e];
                            }
                        } else {
#pragma unroll
                            for (int e = 0; e < 16; ++e) {
                                const int j = j0 + e;
                                B[e] = j <= i ? B[e] * (p.scale * pair_decay(gi, G.G[j])) : 0.f;
                                rs += j < i ? A[e] * B[e] : 0.f;
                            }
                        }
#pragma unroll
                        for (int e = 0; e < 8; ++e) pk[e] = pack_bf16(B[2 * e], B[2 * e + 1]);
                        if (brief) {
#pragma unroll
                            for (int e = 0; e < 8; ++e) rest[e] = rest_bf16(pk[e], B[2 * e], B[2 * e + 1]);
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; ++e) pk[e] = 0;
                    }
                    tc5::st8(trow + TP + 8 * J, pk);
                    if (brief) tc5::st8(trow + TP + 8 * J + CT / 4, rest);
                    if (z == 0 && !(ok = split_state(0))) break;  // its products run under the rest
                }
                if (!ok) break;
                s.r[ph][qt][i] = rs;
            }
            {   // the state part of dq, scaled in place; a_i = q_i . it
                const float f = p.scale * start_decay(gi);
                if (!(ok = warp_wait(&s.x_done, ph))) break;
                tc5::fence_after();
                float as = 0.f;
#pragma unroll 1
                for (int z = 0; z < QK / 16; ++z) {
                    const int c0 = qt * QK + 16 * z;
                    float X[16];
                    uint32_t w[16];
                    tc5::ld16(X, trow + TX + c0);
                    const uint4 q0 = *reinterpret_cast<const uint4*>(s.Q[c0 >> 6] + 2 * swz<64>(i, c0 & 63));
                    const uint4 q1 = *reinterpret_cast<const uint4*>(s.Q[c0 >> 6] + 2 * swz<64>(i, (c0 & 63) + 8));
                    const uint32_t qw[8] = {q0.x, q0.y, q0.z, q0.w, q1.x, q1.y, q1.z, q1.w};
                    tc5::wait_ld();
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float2 v = unpack_bf16(qw[e]);
                        X[2 * e] *= f;
                        X[2 * e + 1] *= f;
                        as += v.x * X[2 * e] + v.y * X[2 * e + 1];
                        w[2 * e] = __float_as_uint(X[2 * e]);
                        w[2 * e + 1] = __float_as_uint(X[2 * e + 1]);
                    }
                    tc5::st16(trow + TX + c0, w);
                }
                s.a[ph][qt][i] = as;
            }
            tc5::wait_st();
            tc5::fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&s.e1);
            const bool up = (i & ~1) < L, dn = (i | 1) < L;
            const size_t row = (size_t)(ch.tok + i) * p.H + h, row0 = (size_t)(ch.tok + (i & ~1)) * p.H + h;
            // A quarter of this lane's row of a result, n of its d columns: to the tile the
            // controller's TMA store takes (to == null: straight to memory, in fp32 for
            // the parts of shared key heads, or row by row for a short chunk)
            auto put = [&](unsigned char* to, void* out, uint32_t col, int n, int d) {
#pragma unroll 1
                for (int z = 0; z < n / 16; ++z) {
                    const int c0 = qt * n + 16 * z;
                    float v[16];
                    uint32_t w[8];
                    tc5::ld16(v, trow + col + c0);
                    tc5::wait_ld();
#pragma unroll
                    for (int e = 0; e < 8; ++e) w[e] = pack_bf16(v[2 * e], v[2 * e + 1]);
                    if (to) {
                        unsigned char* at = to + (c0 >> 6) * PANEL;
                        *reinterpret_cast<uint4*>(at + 2 * swz<64>(i, c0 & 63)) = make_uint4(w[0], w[1], w[2], w[3]);
                        *reinterpret_cast<uint4*>(at + 2 * swz<64>(i, (c0 & 63) + 8)) = make_uint4(w[4], w[5], w[6], w[7]);
                    } else if (p.rep > 1 && out != p.dv) {
                        float* at = (float*)out + row * d + c0;
                        if (i < L) {
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                *reinterpret_cast<float4*>(at + 4 * e) = make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
                        }
                    } else {
                        store_rows<8>((__nv_bfloat16*)out + row0 * d + c0, (size_t)p.H * d, w, up, dn);
                    }
                }
            };
            const bool whole = L == CT, tiles = whole && p.rep == 1;
            if (!(ok = warp_wait(&s.q_done, ph))) break;
            tc5::fence_after();
            put(tiles ? s.out_q() : nullptr, p.dq, TX, QK, DK);
            fence_async_smem();
            tc5::fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&s.e2);
            // ---- second half: lane = key token j = i ------------------------------------
            {
                const float2 gj = gi, gb = G.G[32 * blk + 31];
                const float rf = p.scale * pair_decay(gb, gj);
                const int t = 16 * (qt + 4 * (lane >> 4)) + (lane & 15);
                __syncwarp();
                s.col[warp][lane >> 4][lane & 15] = t >= 32 * blk + 32 ? pair_decay(G.G[t], gb) : 0.f;
                __syncwarp();
                if (!(ok = warp_wait(&s.a2_done, ph))) break;
                tc5::fence_after();
                float cs = 0.f;
                uint32_t pa[2][8], pb[2][8];
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                    const int J = qt + 4 * z, t0 = 16 * J;
                    if (brief && z) {
                        // (made with the first)
                    } else if (J >= 2 * blk) {
                        float A[16], B[16];
                        tc5::ld16(A, trow + TA + t0);
                        tc5::ld16(B, trow + TB + t0);
                        tc5::wait_ld();
                        if (J >= 2 * blk + 2) {
#pragma unroll
                            for (int e = 0; e < 16; ++e) {
                                const float d = rf * s.col[warp][z][e];
                                B[e] *= d;
                                cs += A[e] * B[e];
                                A[e] *= d;
                            }
                        } else {
#pragma unroll
                            for (int e = 0; e < 16; ++e) {
                                const float d = t0 + e >= i ? p.scale * pair_decay(G.G[t0 + e], gj) : 0.f;
                                B[e] = t0 + e >= i ? B[e] * d : 0.f;
                                cs += t0 + e > i ? A[e] * B[e] : 0.f;
                                A[e] = t0 + e >= i ? A[e] * d : 0.f;
                            }
                        }
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            pa[z][e] = pack_bf16(A[2 * e], A[2 * e + 1]);
                            pb[z][e] = pack_bf16(B[2 * e], B[2 * e + 1]);
                        }
                        if (z == 0 && brief) {
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                pa[1][e] = rest_bf16(pa[0][e], A[2 * e], A[2 * e + 1]);
                                pb[1][e] = rest_bf16(pb[0][e], B[2 * e], B[2 * e + 1]);
                            }
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            pa[z][e] = pb[z][e] = 0;
                            if (z == 0 && brief) pa[1][e] = pb[1][e] = 0;
                        }
                    }
                }
                s.c[ph][qt][i] = cs;
                // the operands go over the accumulators once every warp has read its part
                tc5::fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&s.e3r);
                if (!(ok = warp_wait(&s.e3r, ph))) break;
                tc5::fence_after();
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                    tc5::st8(trow + TA + 8 * (qt + 4 * z), pa[z]);
                    tc5::st8(trow + TB + 8 * (qt + 4 * z), pb[z]);
                }
            }
            if (!(ok = split_state(1))) break;
            {   // the state parts of dk and dv, scaled in place; b_j = k_j . dk's
                const float f = i < L ? pair_decay(G.G[CT - 1], gi) : 0.f;
                if (!(ok = warp_wait(&s.x2_done, ph))) break;
                tc5::fence_after();
                float bs = 0.f;
#pragma unroll 1
                for (int z = 0; z < QK / 16; ++z) {
                    const int c0 = qt * QK + 16 * z;
                    float X[16];
                    uint32_t w[16];
                    tc5::ld16(X, trow + TX + c0);
                    const uint4 q0 = *reinterpret_cast<const uint4*>(s.K[c0 >> 6] + 2 * swz<64>(i, c0 & 63));
                    const uint4 q1 = *reinterpret_cast<const uint4*>(s.K[c0 >> 6] + 2 * swz<64>(i, (c0 & 63) + 8));
                    const uint32_t qw[8] = {q0.x, q0.y, q0.z, q0.w, q1.x, q1.y, q1.z, q1.w};
                    tc5::wait_ld();
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float2 v = unpack_bf16(qw[e]);
                        X[2 * e] *= f;
                        X[2 * e + 1] *= f;
                        bs += v.x * X[2 * e] + v.y * X[2 * e + 1];
                        w[2 * e] = __float_as_uint(X[2 * e]);
                        w[2 * e + 1] = __float_as_uint(X[2 * e + 1]);
                    }
                    tc5::st16(trow + TX + c0, w);
                }
                s.b[ph][qt][i] = bs;
                if (!(ok = warp_wait(&s.v_done, ph))) break;
                tc5::fence_after();
#pragma unroll 1
                for (int z = 0; z < QV / 16; ++z) {
                    const uint32_t at = trow + TV + qt * QV + 16 * z;
                    float X[16];
                    uint32_t w[16];
                    tc5::ld16(X, at);
                    tc5::wait_ld();
#pragma unroll
                    for (int e = 0; e < 16; ++e) w[e] = __float_as_uint(X[e] * f);
                    tc5::st16(at, w);
                }
            }
            tc5::wait_st();
            tc5::fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&s.e3[ph]);
            if (!(ok = warp_wait(&s.o_done, ph))) break;
            tc5::fence_after();
            put(tiles ? s.out_k() : nullptr, p.dk, TX, QK, DK);
            put(whole ? s.out_v() : nullptr, p.dv, TV, QV, DV);
            fence_async_smem();
            tc5::fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&s.e4);
            ++x;
        }
    } else if (warp == kEpi) {
        // ---- loads and products ---------------------------------------------------
        constexpr uint32_t ID_TT = tc5::idesc_bf16(128, CT, false, false);  // token x token
        constexpr uint32_t ID_K = tc5::idesc_bf16(128, DK, false, false);   // x state, key channels
        constexpr uint32_t ID_VT = tc5::idesc_bf16(128, DV, false, true);   // state read along value channels; tokens x dO
        constexpr uint32_t ID_KT = tc5::idesc_bf16(128, DK, false, true);   // tokens x K or Q
        constexpr uint64_t KROWS = (16 * 128) >> 4, KCOLS = 32 >> 4, KPANEL = PANEL >> 4, SPANEL = (DK * 128) >> 4;
        constexpr uint64_t STERM = DV / 64 * SPANEL;
        const uint64_t dQ = tc5::kmajor<CT>(smem_u32(s.Q), 0), dK = tc5::kmajor<CT>(smem_u32(s.K), 0);
        const uint64_t dV = tc5::kmajor<CT>(smem_u32(s.V), 0), dY = tc5::kmajor<CT>(smem_u32(s.Y), 0);
        const uint64_t tQ = tc5::mnmajor(smem_u32(s.Q), 0, PANEL), tK = tc5::mnmajor(smem_u32(s.K), 0, PANEL);
        const uint64_t tY = tc5::mnmajor(smem_u32(s.Y), 0, PANEL);
        const uint64_t dS = tc5::kmajor<DK>(smem_u32(s.S), 0), tS = tc5::mnmajor(smem_u32(s.S), 0, DK * 128);
        constexpr uint32_t SB = 2 * DV * DK * 2;  // bytes of a state's image
        auto cols = [](int k, uint64_t panel) { return (uint64_t)(k >> 2) * panel + (uint64_t)(k & 3) * KCOLS; };
        auto next_unit = [&](long long u, Chunk& c) {
            while (u < units && !chunk_of_slot(p.seq, u / p.H, c)) u += gridDim.x;
            return u;
        };
        auto load_qy = [&](long long u, const Chunk& c) {
            if (elect_one()) {
                const int h = (int)(u % p.H), kh = h / p.rep, tok = (int)c.tok;
                mbar_arrive_expect(&s.t_full, (DK + DV) / 64 * PANEL);
#pragma unroll
                for (int y = 0; y < DK / 64; ++y) tma_load_3d(s.Q[y], &p.qmap, 64 * y, kh, tok, &s.t_full);
#pragma unroll
                for (int y = 0; y < DV / 64; ++y) tma_load_3d(s.Y[y], &p.ymap, 64 * y, h, tok, &s.t_full);
            }
            __syncwarp();
        };
        auto load_kv = [&](long long u, const Chunk& c) {
            if (elect_one()) {
                const int h = (int)(u % p.H), kh = h / p.rep, tok = (int)c.tok;
                mbar_arrive_expect(&s.kv_full, (DK + DV) / 64 * PANEL);
#pragma unroll
                for (int y = 0; y < DK / 64; ++y) tma_load_3d(s.K[y], &p.kmap, 64 * y, kh, tok, &s.kv_full);
#pragma unroll
                for (int y = 0; y < DV / 64; ++y) tma_load_3d(s.V[y], &p.vmap, 64 * y, h, tok, &s.kv_full);
            }
            __syncwarp();
        };
        auto load_s = [&](long long u, const unsigned char* from, int term) {
            if (elect_one()) {
                mbar_arrive_expect(&s.s_full[term], SB / 2);
                bulk_g2s(s.S[term], from + (size_t)u * SB + term * (SB / 2), SB / 2, &s.s_full[term]);
            }
            __syncwarp();
        };
        long long u = next_unit(blockIdx.x, ch);
        int nt = 0, nkv = 0, ns[2] = {0, 0};  // loads issued of each kind
        if (u < units) {
            load_qy(u, ch); ++nt;
            load_kv(u, ch); ++nkv;
            load_s(u, p.S, 0); ++ns[0];
            load_s(u, p.S, 1); ++ns[1];
        }
        Chunk nx;
        long long un = u < units ? next_unit(u + gridDim.x, nx) : units;
        for (; ok && u < units; ++x) {
            const int ph = x & 1;
            // first half
            if (!(ok = warp_wait(&s.t_full, ph)) || !(ok = warp_wait(&s.kv_full, ph)) || !(ok = warp_wait(&s.zeroed, ph))) break;
            tc5::fence_after();
            if (elect_one()) {
#pragma unroll 2
                for (int k = 0; k < DK / 16; ++k) tc5::mma(tm + TA, dQ + cols(k, KPANEL), dK + cols(k, KPANEL), ID_TT, k > 0);
#pragma unroll 2
                for (int k = 0; k < DV / 16; ++k) tc5::mma(tm + TB, dY + cols(k, KPANEL), dV + cols(k, KPANEL), ID_TT, k > 0);
                tc5::commit(&s.a_done);
            }
            __syncwarp();
            if (!s.kOwnOut && x > 0) {  // S, where dk and dv of the chunk before were
                if (lane == 0) bulk_wait_read<0>();
                __syncwarp();
                load_s(u, p.S, 0);
                load_s(u, p.S, 1);
                ++ns[0];
                ++ns[1];
            }
            // the next chunk's operands to L2 meanwhile: their places here come free late, and
            // all SMs would then wait for DRAM at once
            if (un < units && lane == 0) {
                const int hn = (int)(un % p.H), kn = hn / p.rep, tn = (int)nx.tok;
#pragma unroll 1
                for (int y = 0; y < DK / 64; ++y) {
                    tma_prefetch_3d(&p.qmap, 64 * y, kn, tn);
                    tma_prefetch_3d(&p.kmap, 64 * y, kn, tn);
                }
#pragma unroll 1
                for (int y = 0; y < DV / 64; ++y) {
                    tma_prefetch_3d(&p.vmap, 64 * y, hn, tn);
                    tma_prefetch_3d(&p.ymap, 64 * y, hn, tn);
                }
                bulk_prefetch_l2(p.S + (size_t)un * SB, SB);
                bulk_prefetch_l2(p.dS + (size_t)un * SB, SB);
            }
            __syncwarp();
            // (dO S goes where dk of the chunk before was: its e4 came before these loads)
            if (!(ok = warp_wait(&s.s_full[0], 0))) break;
            tc5::fence_after();
            if (elect_one()) {
#pragma unroll 2
                for (int k = 0; k < DV / 16; ++k) tc5::mma(tm + TX, dY + cols(k, KPANEL), dS + cols(k, SPANEL), ID_K, k > 0);
                tc5::commit(&s.s_read);
            }
            __syncwarp();
            if (!(ok = warp_wait(&s.s_ready, 0))) break;  // the other terms, in the places of the halves
            tc5::fence_after();
            if (elect_one()) {
#pragma unroll 1
                for (int t = 0; t < 2; ++t)
#pragma unroll 2
                    for (int k = 0; k < DV / 16; ++k)
                        tc5::mma(tm + TX, dY + cols(k, KPANEL), dS + t * STERM + cols(k, SPANEL), ID_K, true);
                tc5::commit(&s.x_done);
            }
            __syncwarp();
            if (!(ok = warp_wait(&s.x_done, ph))) break;
            load_s(u, p.dS, 0);
            ++ns[0];
            if (s.kOwnOut) {
                load_s(u, p.dS, 1);
                ++ns[1];
            }
            if (!(ok = warp_wait(&s.e1, ph))) break;
            tc5::fence_after();
            if (s.kOwnOut && lane == 0) bulk_wait_read<0>();  // dq goes where dk and dv of the chunk before were
            __syncwarp();
            if (elect_one()) {
#pragma unroll 2
                for (int k = 0; k < CT / 16; ++k) tc5::mma_ts(tm + TX, tm + TP + 8 * k, tK + k * KROWS, ID_KT, true);
                tc5::commit(&s.q_done);
                // second half
#pragma unroll 2
                for (int k = 0; k < DK / 16; ++k) tc5::mma(tm + TA, dK + cols(k, KPANEL), dQ + cols(k, KPANEL), ID_TT, k > 0);
#pragma unroll 2
                for (int k = 0; k < DV / 16; ++k) tc5::mma(tm + TB, dV + cols(k, KPANEL), dY + cols(k, KPANEL), ID_TT, k > 0);
                tc5::commit(&s.a2_done);
            }
            __syncwarp();
            // V dS goes where dq is read, K dS^T where its operand was
            if (!(ok = warp_wait(&s.e2, ph))) break;
            const int h = (int)(u % p.H), tok = (int)ch.tok;
            const bool whole = ch.L == CT, tiles = whole && p.rep == 1;
            if (lane == 0 && tiles) {
#pragma unroll
                for (int y = 0; y < DK / 64; ++y) tma_store_3d(&p.dqmap, 64 * y, h, tok, s.out_q() + y * PANEL);
                bulk_commit();
                if (!s.kOwnOut) bulk_wait_read<0>();
            }
            __syncwarp();
            if (!s.kOwnOut) {
                load_s(u, p.dS, 1);
                ++ns[1];
            }
            if (!(ok = warp_wait(&s.s_full[0], 1))) break;
            tc5::fence_after();
            if (elect_one()) {
#pragma unroll 2
                for (int k = 0; k < DV / 16; ++k) tc5::mma(tm + TX, dV + cols(k, KPANEL), dS + cols(k, SPANEL), ID_K, k > 0);
#pragma unroll 2
                for (int k = 0; k < DK / 16; ++k) tc5::mma(tm + TV, dK + cols(k, KPANEL), tS + k * KROWS, ID_VT, k > 0);
                tc5::commit(&s.s_read);
            }
            __syncwarp();
            if (!(ok = warp_wait(&s.s_ready, 1))) break;
            tc5::fence_after();
            if (elect_one()) {
#pragma unroll 1
                for (int t = 0; t < 2; ++t)
#pragma unroll 2
                    for (int k = 0; k < DV / 16; ++k)
                        tc5::mma(tm + TX, dV + cols(k, KPANEL), dS + t * STERM + cols(k, SPANEL), ID_K, true);
                tc5::commit(&s.x2_done);
#pragma unroll 2
                for (int k = 0; k < DK / 16; ++k) tc5::mma(tm + TV, dK + cols(k, KPANEL), tS + STERM + k * KROWS, ID_VT, true);
                tc5::commit(&s.v_done);
            }
            __syncwarp();
            if (!(ok = warp_wait(&s.v_done, ph))) break;
            if (s.kOwnOut && un < units) {
                load_s(un, p.S, 0);
                load_s(un, p.S, 1);
                ++ns[0];
                ++ns[1];
            }
            if (!(ok = warp_wait(&s.e3[ph], (x >> 1) & 1))) break;  // K's rows are read by then too
            tc5::fence_after();
            // dk, written after the products below, goes where the store of dq reads
            if (s.kOwnOut && lane == 0) bulk_wait_read<0>();
            __syncwarp();
            if (un < units) {
                load_kv(un, nx);
                ++nkv;
            }
            if (elect_one()) {
#pragma unroll 2
                for (int k = 0; k < CT / 16; ++k) tc5::mma_ts(tm + TX, tm + TB + 8 * k, tQ + k * KROWS, ID_KT, true);
#pragma unroll 2
                for (int k = 0; k < CT / 16; ++k) tc5::mma_ts(tm + TV, tm + TA + 8 * k, tY + k * KROWS, ID_VT, true);
                tc5::commit(&s.o_done);
            }
            __syncwarp();
            Chunk n2;
            const long long u2 = un < units ? next_unit(un + gridDim.x, n2) : units;
            if (!(ok = warp_wait(&s.o_done, ph))) break;
            if (un < units) {
                load_qy(un, nx);
                ++nt;
            }
            if (!(ok = warp_wait(&s.e4, ph))) break;
            if (lane == 0) {
                if (tiles) {
#pragma unroll
                    for (int y = 0; y < DK / 64; ++y) tma_store_3d(&p.dkmap, 64 * y, h, tok, s.out_k() + y * PANEL);
                }
                if (whole) {
#pragma unroll
                    for (int y = 0; y < DV / 64; ++y) tma_store_3d(&p.dvmap, 64 * y, h, tok, s.out_v() + y * PANEL);
                }
                bulk_commit();
            }
            __syncwarp();
            u = un;
            un = u2;
            ch = nx;
            nx = n2;
        }
        // no copy and no product may be in flight when the CTA ends
        if (nt) warp_wait(&s.t_full, (nt - 1) & 1);
        if (nkv) warp_wait(&s.kv_full, (nkv - 1) & 1);
        for (int t = 0; t < 2; ++t)
            if (ns[t]) warp_wait(&s.s_full[t], (ns[t] - 1) & 1);
        if (lane == 0) bulk_wait<0>();
        if (elect_one()) tc5::commit(&s.drain);
        warp_wait(&s.drain, 0);
    } else {
        // ---- gates of the next chunk, then dg of this one ---------------------------
        float g[4];
        auto next_unit = [&](long long u, Chunk& c) {
            while (u < units && !chunk_of_slot(p.seq, u / p.H, c)) u += gridDim.x;
            return u;
        };
        auto form = [&](long long u, const Chunk& c, int n) {
            load_gates(g, p.g + (size_t)c.tok * p.H + (int)(u % p.H), p.H, c.L);
            form_gates(s.gate[n & 1], g);
            __syncwarp();
            if (lane == 0) mbar_arrive(&s.gfull[n & 1]);
        };
        long long u = next_unit(blockIdx.x, ch);
        if (u < units) form(u, ch, 0);
        for (; ok && u < units; ++x) {
            const int ph = x & 1;
            Chunk nx;
            const long long un = next_unit(u + gridDim.x, nx);
            // the other gates are free once the chunk before is done with them (its e3)
            if (un < units) form(un, nx, x + 1);
            if (!(ok = warp_wait(&s.e3[ph], (x >> 1) & 1))) break;
            // dg: lane holds tokens 4 lane .. 4 lane + 3
            const int h = (int)(u % p.H);
            float y[4], b[4], sy = 0.f, sb = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int t = 4 * lane + j;
                y[j] = b[j] = 0.f;
                if (t < ch.L) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        y[j] += s.r[ph][q][t] - s.c[ph][q][t] + s.a[ph][q][t];
                        b[j] += s.b[ph][q][t];
                    }
                }
                sy += y[j];
                sb += b[j];
            }
            float after = sy, before = sb;  // sums over the lanes from this one on, and up to it
#pragma unroll 1
            for (int o = 1; o < 32; o <<= 1) {
                const float v = __shfl_down_sync(0xffffffffu, after, o), w = __shfl_up_sync(0xffffffffu, before, o);
                if (lane + o < 32) after += v;
                if (lane >= o) before += w;
            }
            float cross = 0.f;
            for (int v = 0; v < DV / 64; ++v) cross += p.cross[(size_t)v * units + u];
            float run = after - sy + cross + before - sb;  // at the end of this lane's tokens, from b before them
#pragma unroll
            for (int j = 0; j < 4; ++j) run += b[j];
#pragma unroll
            for (int j = 3; j >= 0; --j) {
                run += y[j];
                run -= b[j];
                const int t = 4 * lane + j;
                if (t < ch.L) {
                    const size_t at = (size_t)(ch.tok + t) * p.H + h;
                    p.dg[at] = p.g[at] < -104.f ? 0.f : run;  // past a reset nothing depends on the gate
                }
            }
            u = un;
            ch = nx;
        }
    }
    if (!ok && lane == 0) atomicOr(p.status, 1u);
    tc5::fence_before();
    __syncthreads();
    if (warp == kEpi) {
        tc5::fence_after();
        tc5::dealloc(tm, 512);
    }
}

struct Layout {
    size_t S, dS, cross, runs, dq, dk, end;
};
Layout layout(const Problem& p) {
    Layout l{};
    size_t o = kStatusBytes;
    auto take = [&](size_t bytes) { size_t r = o; o += (bytes + 255) & ~(size_t)255; return r; };
    const size_t slots = (size_t)chunk_slots(p.seq, CT), image = slots * p.H * 2 * p.dk * p.dv * 2;
    l.S = take(image);
    l.dS = take(image);
    l.cross = take(slots * p.H * (p.dv / 64) * 4);
    l.runs = take(tc_states_workspace(p));
    if (p.H != p.Hk) {
        l.dq = take((size_t)p.seq.rows * p.H * p.dk * 4);
        l.dk = take((size_t)p.seq.rows * p.H * p.dk * 4);
    }
    l.end = o;
    return l;
}

template <int DK, int DV>
void launch(const Params& a, const Problem& p, cudaStream_t st) {
    const int smem = sizeof(Smem<DK, DV>) + 1024;
    auto* kernel = short_sequences(p) ? decay_tc_bwd_kernel<DK, DV, true> : decay_tc_bwd_kernel<DK, DV, false>;
    cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    const long long units = chunk_slots(p.seq, CT) * p.H;
    GDN_LAUNCH("decay_tc_bwd", st, (kernel<<<(unsigned)(units < 148 ? units : 148), kThreads, smem, st>>>(a)));
}

}  // namespace

size_t tc_bwd_workspace(const Problem& p) { return layout(p).end; }

bool launch_tc_bwd(const Problem& p, const void* q, const void* k, const void* v, const float* g, const float* h0,
                   const void* dO, const float* dhT, void* dq, void* dk, void* dv, float* dg, float* dh0, void* ws,
                   cudaStream_t st) {
    const Layout l = layout(p);
    char* base = (char*)ws;
    Params a{};
    if (!encode_head_map(&a.qmap, q, p.seq.rows, p.Hk, p.dk, CT) || !encode_head_map(&a.kmap, k, p.seq.rows, p.Hk, p.dk, CT) ||
        !encode_head_map(&a.vmap, v, p.seq.rows, p.H, p.dv, CT) || !encode_head_map(&a.ymap, dO, p.seq.rows, p.H, p.dv, CT))
        return false;
    const bool parts = p.H != p.Hk;
    if (!encode_head_map(&a.dvmap, dv, p.seq.rows, p.H, p.dv, CT)) return false;
    if (!parts && (!encode_head_map(&a.dqmap, dq, p.seq.rows, p.H, p.dk, CT) || !encode_head_map(&a.dkmap, dk, p.seq.rows, p.H, p.dk, CT)))
        return false;
    a.seq = p.seq; a.H = p.H; a.rep = p.H / p.Hk; a.scale = p.scale; a.g = g;
    a.S = (unsigned char*)base + l.S; a.dS = (unsigned char*)base + l.dS; a.cross = (float*)(base + l.cross);
    a.dq = parts ? (void*)(base + l.dq) : dq;
    a.dk = parts ? (void*)(base + l.dk) : dk;
    a.dv = (__nv_bfloat16*)dv; a.dg = dg; a.status = (unsigned int*)ws;
    if (!launch_tc_states(p, q, k, v, g, h0, dO, dhT, dh0, base + l.S, base + l.dS, (float*)(base + l.cross), base + l.runs, ws, st))
        return false;
    if (p.dk == 64 && p.dv == 64) launch<64, 64>(a, p, st);
    else if (p.dk == 64) launch<64, 128>(a, p, st);
    else if (p.dv == 64) launch<128, 64>(a, p, st);
    else launch<128, 128>(a, p, st);
    if (parts) launch_group_sum(p, (const float*)(base + l.dq), (const float*)(base + l.dk), dq, dk, st);
    return true;
}

}  // namespace decay
}  // namespace gdn
