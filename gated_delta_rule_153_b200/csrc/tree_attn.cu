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
#include "decay_tc.cuh"
#include "mma.cuh"
#include "tc5.cuh"
#include "tma.cuh"

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

// ---- attention -----------------------------------------------------------------
// A unit is a (sequence, key head, 128 rows): the rows are the nodes' query heads of
// that key head, row = node * group + head in group.  Its keys come in tiles of
// 128, the cached ones first, the nodes themselves as the last.  Every key tile
// of every unit is one step of work, and the steps of the whole call, in order, are
// cut evenly over one CTA per SM, so that sequences of any lengths fill the
// device.  A CTA whose share starts or ends within a unit leaves a partial result
// (maximum, sum, weighted sum) in the workspace; the last CTA of a unit to do so,
// told by a counter, joins them, in the order of the steps whoever that is.  With units
// for less than half of the SMs, each unit instead gets a number of CTAs of its own:
// no CTA then works on two, which would be most of its time.
//
// Per tile:  S = Q K^T (tcgen05, 128 x 128 x d, lane = row),  P = e^{S - m} as a
// bf16 A operand over S in tensor memory,  O += P V.  Two groups of four softmax
// warps take the tiles in turn, each with its own m, l and O, so that one group's
// products run under the other's exponentials; they are joined at the segment's
// end.  O is rescaled only when the maximum grew by more than 2^8: until then
// the weights, and their sums, are just that much larger.  Keys and values arrive
// by TMA, page by page, through a three-stage ring.
// What bounds it is the HBM read of the cached keys and values: 32 sequences of up to
// 8192 tokens, 32 nodes, 16 query and 4 key heads of 128 channels take 90 us, 4.0 TB/s of
// the 360 MB, of which the steps are 63 us; the rest is the start, the last partial
// results and their joins.
constexpr int KT = 128;              // keys per tile
constexpr int PANEL = KT * 128;      // bytes of a 128-row, 64-channel tile
constexpr int NST = 3;
constexpr int kSoft = 8;             // softmax warps, two groups
constexpr int kThreads = 32 * (kSoft + 2);

template <int D>
struct alignas(1024) Smem {
    unsigned char Q[D / 64][PANEL];
    unsigned char K[NST][D / 64][PANEL], V[NST][D / 64][PANEL];
    float2 ml[128];                  // a segment's end: one group's maxima and sums, then both factors
    int parent[kMaxNodes];
    // By parity of the segment, values that are not finite where rows differ in what they see:
    // the nodes that hold one, and the last such cached position (-1: none)
    unsigned long long bad_nodes[2];
    int bad_pos[2];
    // 16-row pieces of a step's tile that hold cached rows; twice the stages, as the
    // loader may be that far ahead of the softmax warps
    uint32_t have[2 * NST];
    uint64_t k_full[NST], v_full[NST], k_free[NST], v_free[NST], s_ready[2], p_ready[2], o_done[2], q_full, seg_done, meet, drain;
    long long warp_sum[kSoft + 2];
    int n0;
    long long before, total;
    int last[2], b0[2], b1[2];  // the units left at the end: whether joined here, and their CTAs
    uint32_t tmem;
};

struct Params {
    CUtensorMap qmap, kmap, vmap, knode, vnode;
    Cache c;
    int N, M, Hq, Hkv, group, row_tiles, window;
    float scale;
    int q_tma;                       // Q rows by TMA: a tile is whole nodes, and the scale is positive
    const int* parent;
    const __nv_bfloat16* q;
    __nv_bfloat16* o;
    float* part;                     // [CTA][2][D / 4][rows][4] weighted sums, then [rows][2] m and l
    int part_rows, part_floats;      // rows of a part, and its size (whole 16-byte pieces)
    unsigned int* count;             // per unit: parts left so far
    int split;                       // CTAs per unit, or 0: the steps cut evenly over all CTAs
    unsigned int* status;
};

// The steps of sequence n: its first key tile that any node sees, the tiles from
// there, and the one of the nodes.
struct Span {
    int len, first, steps;
};
GDN_DEV Span span_of(const Params& p, int n) {
    Span s;
    s.len = cached(p.c, n, p.status);
    const int lo = p.window > 0 ? max(0, s.len - p.window + 1) : 0;
    s.first = lo / KT;
    s.steps = (s.len + KT - 1) / KT - s.first + 1;
    return s;
}

// A CTA's share of one unit: steps t0 .. t1 - 1 of its `span.steps`.
struct Segment {
    int n, kh, rt, t0, t1;
    Span span;
};

// Walks the segments of a CTA's share [at, end) of all steps.
struct Walk {
    long long at, end, base;  // base: steps before sequence n
    int n;
    Span span;
    GDN_DEV bool next(const Params& p, Segment& g) {
        if (at >= end) return false;
        const int units = p.Hkv * p.row_tiles;
        while (at >= base + (long long)span.steps * units) {
            base += (long long)span.steps * units;
            span = span_of(p, ++n);
        }
        const int u = (int)((at - base) / span.steps);
        g.n = n;
        g.kh = u / p.row_tiles;
        g.rt = u % p.row_tiles;
        g.span = span;
        g.t0 = (int)((at - base) % span.steps);
        g.t1 = (int)min((long long)span.steps, g.t0 + (end - at));
        at += g.t1 - g.t0;
        return true;
    }
};

// The shares of a call of `total` steps: at least two steps each.
GDN_DEV long long shares(long long total, int ctas) { return min((long long)ctas, (total + 1) / 2); }
GDN_DEV long long share_start(long long total, long long parts, long long b) { return total * b / parts; }

// All threads: total steps, and the sequence that holds step `at` with the steps
// before it (s.n0, s.before).  Every thread sums a run of sequences.
template <class S>
GDN_DEV void locate(S& s, const Params& p, int b, int ctas) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (p.N + kThreads - 1) / kThreads, a = min(p.N, tid * per), e = min(p.N, a + per);
    const int units = p.Hkv * p.row_tiles;
    long long mine = 0;
    for (int n = a; n < e; ++n) mine += span_of(p, n).steps;
    long long run = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, run, o);
        if (lane >= o) run += y;
    }
    if (lane == 31) s.warp_sum[warp] = run;
    __syncthreads();
    long long before = run - mine, all = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) before += s.warp_sum[w];
        all += s.warp_sum[w];
    }
    all *= units;
    before *= units;
    const long long at = share_start(all, shares(all, ctas), b);
    if (at >= before && at < before + mine * units) {
        int n = a;
        for (;; ++n) {
            const long long st = (long long)span_of(p, n).steps * units;
            if (at < before + st) break;
            before += st;
        }
        s.n0 = n;
        s.before = before;
    }
    if (tid == 0) s.total = all;
    __syncthreads();
}
// The share that holds step `at`.
GDN_DEV int owner_of(long long total, long long parts, long long at) {
    long long b = at * parts / total;
    while (share_start(total, parts, b + 1) <= at) ++b;
    while (share_start(total, parts, b) > at) --b;
    return (int)b;
}
// Sixteen values of a row in bf16.
GDN_DEV void put16(__nv_bfloat16* to, const float (&u)[16]) {
    uint32_t h[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) h[q] = pack_bf16(u[2 * q], u[2 * q + 1]);
    *reinterpret_cast<uint4*>(to) = make_uint4(h[0], h[1], h[2], h[3]);
    *reinterpret_cast<uint4*>(to + 8) = make_uint4(h[4], h[5], h[6], h[7]);
}

using decay::align1k;
using decay::all_finite;
using decay::elect_one;
using decay::ex2;
using decay::seen_bf16;
using decay::wait_for;
using decay::warp_wait;

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
tree_attn_kernel(const __grid_constant__ Params p) {
    extern __shared__ __align__(1024) unsigned char raw[];
    Smem<D>& s = *reinterpret_cast<Smem<D>*>(align1k(raw));
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int ctas = gridDim.x, b = blockIdx.x;
    if (tid == 0) {
        for (int i = 0; i < NST; ++i) {
            mbar_init(&s.k_full[i], 1);
            mbar_init(&s.v_full[i], 1);
            mbar_init(&s.k_free[i], 1);
            mbar_init(&s.v_free[i], 1);
        }
        for (int g = 0; g < 2; ++g) {
            mbar_init(&s.s_ready[g], 1);
            mbar_init(&s.p_ready[g], kSoft / 2);
            mbar_init(&s.o_done[g], 1);
        }
        mbar_init(&s.q_full, p.q_tma ? 1 : kSoft);
        mbar_init(&s.seg_done, kSoft);
        mbar_init(&s.meet, kSoft);
        mbar_init(&s.drain, 1);
        fence_mbar_init();
    }
    if (warp == kSoft + 1) tc5::alloc(&s.tmem, 512);
    if (!p.split) locate(s, p, b, ctas);
    tc5::fence_before();
    __syncthreads();
    tc5::fence_after();
    const uint32_t tm = __shfl_sync(0xffffffffu, s.tmem, 0);
    const long long parts = p.split ? 0 : shares(s.total, ctas);
    Walk w{0, 0, 0, 0, {}};
    int pieces = 0;  // split: CTAs that share this one's unit
    if (p.split) {
        const int unit = b / p.split, units = p.Hkv * p.row_tiles, q = b % p.split;
        w.n = unit / units;
        w.span = span_of(p, w.n);
        pieces = max(1, min(p.split, w.span.steps / 2));
        if (q < pieces) {
            w.at = (long long)(unit % units) * w.span.steps + share_start(w.span.steps, pieces, q);
            w.end = (long long)(unit % units) * w.span.steps + share_start(w.span.steps, pieces, q + 1);
        }
    } else if (b < parts) {
        w = Walk{share_start(s.total, parts, b), share_start(s.total, parts, b + 1), s.before, s.n0, {}};
        w.span = span_of(p, w.n);
    }
    // tensor-memory columns of a group: S (P over it, as bf16 pairs), O
    constexpr uint32_t TG = 256, TO = 128;
    int x = 0;      // steps so far: the group and the phases of its barriers follow from it
    int segs = 0;
    bool ok = true;
    Segment g;
    if (warp < kSoft) {
        const int grp = warp >> 2, r = 32 * (warp & 3) + lane;
        const uint32_t tg = tm + ((uint32_t)(32 * (warp & 3)) << 16) + TG * grp;
        const float sc = p.scale == 0.f ? 1.4426950408889634f : fabsf(p.scale) * 1.4426950408889634f;
        const int R = p.M * p.group;
        struct {
            Segment g;
            long long u0;  // the unit's first step
        } left[2];
        int lefts = 0, met = 0;
        auto meet = [&]() {  // the softmax warps come together (within the bounds of a wait)
            __syncwarp();
            if (lane == 0) mbar_arrive(&s.meet);
            return ok = warp_wait(&s.meet, met++ & 1);
        };
        while (ok && w.next(p, g)) {
            const int row = g.rt * 128 + r, node = row / p.group, head = g.kh * p.group + row % p.group;
            const bool live = row < R;
            const bool busy = g.rt * 128 + 32 * (warp & 3) < R;  // this warp has rows
            const size_t qrow = (((size_t)g.n * p.M + (live ? node : 0)) * p.Hq + (live ? head : 0)) * D;
            if (!p.q_tma) {
                // Q of the unit (its sign with the scale's; zero for a zero scale and past the rows):
                // D / 8 lanes to a row, all of a warp's 16 rows on their way at once.  Every S
                // of the Q before is done: this warp has waited for all of them.
                constexpr int LR = D / 8, RPI = 32 / LR;
                const uint32_t flip = p.scale < 0.f ? 0x80008000u : 0u;
                uint4 v[16 / RPI];
#pragma unroll
                for (int j = 0; j < 16 / RPI; ++j) {
                    const int y = g.rt * 128 + 16 * warp + RPI * j + lane / LR;
                    v[j] = make_uint4(0, 0, 0, 0);
                    if (y < R && p.scale != 0.f)
                        v[j] = __ldg(reinterpret_cast<const uint4*>(
                            p.q + (((size_t)g.n * p.M + y / p.group) * p.Hq + g.kh * p.group + y % p.group) * D + 8 * (lane % LR)));
                }
#pragma unroll
                for (int j = 0; j < 16 / RPI; ++j) {
                    const int y = 16 * warp + RPI * j + lane / LR, ch = lane % LR;
                    *reinterpret_cast<uint4*>(s.Q[ch >> 3] + 2 * swz<64>(y, 8 * (ch & 7))) =
                        make_uint4(v[j].x ^ flip, v[j].y ^ flip, v[j].z ^ flip, v[j].w ^ flip);
                }
                fence_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&s.q_full);
            }
            if (tid < p.M) s.parent[tid] = parent_of(p.parent + (size_t)g.n * p.M, tid, p.status);
            const int par = segs & 1;
            if (tid == 0) {
                s.bad_nodes[par] = 0;
                s.bad_pos[par] = -1;
            }
            if (!meet()) break;
            // what this row sees: cached positions from `lo`, nodes in `anc`
            unsigned long long anc = 0;
            int depth = 0;
            if (live) {
                for (int j = node, back = 0; j >= 0; j = s.parent[j], ++back) {
                    if (p.window == 0 || back < p.window) anc |= 1ull << j;
                    depth = back;
                }
            }
            const long long far = p.window > 0 ? (long long)g.span.len + depth - p.window + 1 : 0;
            const int lo = far > 0 ? (int)min(far, (long long)g.span.len) : 0;
            float m = -INFINITY, l = 0.f;
            bool any = false;  // this group had a step in this segment
            for (int t = g.t0; t < g.t1; ++t, ++x) {
                if ((x & 1) != grp) continue;
                const int st = x % NST, ph = (x >> 1) & 1;
                const bool tree = t == g.span.steps - 1;
                const int key0 = (g.span.first + t) * KT;
                if (!(ok = warp_wait(&s.s_ready[grp], ph))) break;
                tc5::fence_after();
                uint32_t have = 0xff;
                if (!tree) {
                    // the loader wrote `have` before it armed k_full, which the product waited for
                    have = s.have[x % (2 * NST)];
                }
                const bool partly = tree || have != 0xff || key0 + KT > g.span.len ||
                                    (p.window > 0 && key0 < g.span.len + p.M - p.window);
                if (partly) {
                    if (busy) {  // scores that this row does not see become -inf
#pragma unroll 1
                        for (int j = 0; j < 8; ++j) {
                            uint32_t seen;
                            if (tree) {
                                seen = j < 4 ? (uint32_t)(anc >> (16 * j)) & 0xffffu : 0u;
                            } else {
                                const int k0 = key0 + 16 * j, a = max(lo - k0, 0), e = min(g.span.len - k0, 16);
                                seen = e > 0 && a < 16 && (have >> j & 1) ? ((1u << e) - 1u) & ~((1u << a) - 1u) : 0u;
                            }
                            float v[16];
                            uint32_t u[16];
                            tc5::ld16(v, tg + 16 * j);
                            tc5::wait_ld();
#pragma unroll
                            for (int q = 0; q < 16; ++q) u[q] = (seen >> q) & 1 ? __float_as_uint(v[q]) : 0xff800000u;
                            tc5::st16(tg + 16 * j, u);
                        }
                        tc5::wait_st();
                    }
                    // and values that no row sees become zero: whatever the places hold, a
                    // zero weight times it must be zero
                    if (!(ok = warp_wait(&s.v_full[st], (x / NST) & 1))) break;
                    const bool dead = tree ? r >= p.M
                                           : key0 + r >= g.span.len || !(have >> (r >> 4) & 1) ||
                                                 (p.window > 0 && key0 + r <= g.span.len - p.window);
                    if (dead) {
#pragma unroll 1
                        for (int j = 0; j < D / 8; ++j)
                            *reinterpret_cast<uint4*>(s.V[st][j >> 3] + 2 * swz<64>(r, 8 * (j & 7))) = make_uint4(0, 0, 0, 0);
                    } else if (p.M > 1 && (tree || p.window > 0)) {
                        // a value that some rows see and others do not: one that is not finite
                        // goes in as zero, and the rows that see it are made NaN at the end
                        bool fine = true;
#pragma unroll 1
                        for (int j = 0; j < D / 8; ++j) {
                            uint4* at = reinterpret_cast<uint4*>(s.V[st][j >> 3] + 2 * swz<64>(r, 8 * (j & 7)));
                            const uint4 v = *at;
                            if (all_finite(seen_bf16(v.x, seen_bf16(v.y, seen_bf16(v.z, seen_bf16(v.w, 0u)))))) continue;
                            *at = make_uint4(0, 0, 0, 0);
                            fine = false;
                        }
                        if (!fine && tree) atomicOr(&s.bad_nodes[par], 1ull << r);
                        if (!fine && !tree) atomicMax(&s.bad_pos[par], key0 + r);
                    }
                    fence_async_smem();
                }
                if (busy) {
                    float mt = -INFINITY;
#pragma unroll 1
                    for (int j = 0; j < 4; ++j) {
                        float v[32];
                        tc5::ld32(v, tg + 32 * j);
                        tc5::wait_ld();
                        float a = v[0], c = v[1];
#pragma unroll
                        for (int q = 2; q < 32; q += 2) {
                            a = fmaxf(a, v[q]);
                            c = fmaxf(c, v[q + 1]);
                        }
                        mt = fmaxf(mt, fmaxf(a, c));
                    }
                    mt *= sc;
                    const bool grow = mt > m + 8.f;
                    if (__any_sync(0xffffffffu, grow)) {
                        const float mn = grow ? mt : m;
                        const float f = grow ? ex2(m - mn) : 1.f;
                        l *= f;
                        m = mn;
                        if (any) {
                            // O of the last step of this group must be in
                            if (!(ok = warp_wait(&s.o_done[grp], ph ^ 1))) break;
                            tc5::fence_after();
#pragma unroll 1
                            for (int j = 0; j < D / 16; ++j) {
                                float v[16];
                                uint32_t u[16];
                                tc5::ld16(v, tg + TO + 16 * j);
                                tc5::wait_ld();
#pragma unroll
                                for (int q = 0; q < 16; ++q) u[q] = __float_as_uint(f * v[q]);
                                tc5::st16(tg + TO + 16 * j, u);
                            }
                            tc5::wait_st();
                        }
                    }
                    const float off = m == -INFINITY ? 0.f : -m;
                    float l0 = 0.f, l1 = 0.f;
#pragma unroll 1
                    for (int j = 0; j < 4; ++j) {
                        float v[32];
                        uint32_t u[16];
                        tc5::ld32(v, tg + 32 * j);
                        tc5::wait_ld();
#pragma unroll
                        for (int q = 0; q < 16; ++q) {
                            const float a = ex2(fmaf(v[2 * q], sc, off)), c = ex2(fmaf(v[2 * q + 1], sc, off));
                            l0 += a;
                            l1 += c;
                            u[q] = pack_bf16(a, c);
                        }
                        tc5::st16(tg + 16 * j, u);
                    }
                    l += l0 + l1;
                    tc5::wait_st();
                }
                any = true;
                tc5::fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&s.p_ready[grp]);
            }
            if (!ok) break;
            // ---- the segment's result: both groups' O, each group half of the channels ----
            // (x is now past the segment; the last step of each group is the one of its parity)
            for (int q = 0; q < 2 && ok; ++q) {
                const int y = x - 1 - ((x - 1 - q) & 1);  // the last step of group q so far
                if (y >= x - (g.t1 - g.t0)) ok = warp_wait(&s.o_done[q], (y >> 1) & 1);
            }
            if (!ok) break;
            tc5::fence_after();
            // m and l of both groups; the factors of their sums (a group without a step has
            // nothing in its O)
            float mx = 0.f, lt = 0.f, f0, f1;
            const bool whole = g.t0 == 0 && g.t1 == g.span.steps;
            if (grp == 1) s.ml[r] = make_float2(m, any ? l : 0.f);
            if (!meet()) break;
            if (grp == 0) {
                const float2 o = s.ml[r];
                const float l0 = any ? l : 0.f;
                mx = fmaxf(m, o.x);
                f0 = l0 != 0.f ? ex2(m - mx) : 0.f;  // (a NaN goes on)
                f1 = o.y != 0.f ? ex2(o.x - mx) : 0.f;
                lt = l0 * f0 + o.y * f1;
                if ((s.bad_nodes[par] & anc) || s.bad_pos[par] >= lo) f0 = f1 = lt = __uint_as_float(decay::kNaN);
                if (whole) {
                    f0 *= 1.f / lt;
                    f1 *= 1.f / lt;
                }
                s.ml[r] = make_float2(f0, f1);
            }
            if (!meet()) break;
            if (grp == 1) {
                const float2 o = s.ml[r];
                f0 = o.x;
                f1 = o.y;
            }
            if (busy) {
                // a CTA that starts within the unit leaves its part in place 0, else in 1
                float* part = p.part + ((size_t)b * 2 + (g.t0 > 0 ? 0 : 1)) * p.part_floats;
                __nv_bfloat16* out = p.o + qrow;
                const uint32_t t0 = tg - TG * grp + TO, t1 = t0 + TG;
#pragma unroll 1
                for (int j = 0; j < D / 32; ++j) {
                    const int c0 = grp * (D / 2) + 16 * j;
                    float u[16], v[16];
                    tc5::ld16(u, t0 + c0);
                    tc5::ld16(v, t1 + c0);
                    tc5::wait_ld();
#pragma unroll
                    for (int q = 0; q < 16; ++q) u[q] = (f0 != 0.f ? f0 * u[q] : 0.f) + (f1 != 0.f ? f1 * v[q] : 0.f);
                    if (!live) continue;
                    if (whole) {
                        put16(out + c0, u);
                    } else {  // a warp's rows side by side
#pragma unroll
                        for (int q = 0; q < 16; q += 4)
                            *reinterpret_cast<float4*>(part + ((size_t)(c0 + q) / 4 * p.part_rows + r) * 4) =
                                make_float4(u[q], u[q + 1], u[q + 2], u[q + 3]);
                    }
                }
                if (!whole && live && grp == 0)
                    *reinterpret_cast<float2*>(part + (size_t)D * p.part_rows + 2 * r) = make_float2(mx, lt);
            }
            if (!whole) {  // to be told at the end
                left[lefts].g = g;
                left[lefts++].u0 = w.at - g.t1;
            }
            tc5::fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&s.seg_done);
            ++segs;
        }
        // ---- the units of which this CTA had a part: told, and joined if it was the last ----
        // (at the end, when the parts' stores have long been on their way)
        if (ok && lefts) {
            __threadfence();
            if (meet()) {
                if (tid < lefts) {
                    const Segment& y = left[tid].g;
                    const int b0 = p.split ? b / p.split * p.split : owner_of(s.total, parts, left[tid].u0);
                    const int b1 = p.split ? b0 + pieces - 1 : owner_of(s.total, parts, left[tid].u0 + y.span.steps - 1);
                    s.b0[tid] = b0;
                    s.b1[tid] = b1;
                    s.last[tid] = atomicAdd(p.count + ((size_t)y.n * p.Hkv + y.kh) * p.row_tiles + y.rt, 1u) == (unsigned)(b1 - b0);
                }
                meet();
            }
        }
        for (int i = 0; ok && i < lefts; ++i) {
            const Segment& y = left[i].g;
            const int row = y.rt * 128 + r;
            if (!s.last[i] || row >= R) continue;
            __threadfence();
            // half of the channels of each part in turn, all on their way at once
            float mj = -INFINITY, lj = 0.f, u[D / 2];
#pragma unroll
            for (int q = 0; q < D / 2; ++q) u[q] = 0.f;
#pragma unroll 1
            for (int c = s.b0[i]; c <= s.b1[i]; ++c) {
                // the first of a unit's CTAs left its part in place 1, the others in place 0
                const float* at = p.part + ((size_t)c * 2 + (c > s.b0[i] ? 0 : 1)) * p.part_floats;
                const float2 o = __ldcg(reinterpret_cast<const float2*>(at + (size_t)D * p.part_rows + 2 * r));
                at += ((size_t)(grp * (D / 8)) * p.part_rows + r) * 4;
                float4 v[D / 8];
#pragma unroll
                for (int q = 0; q < D / 8; ++q) v[q] = __ldcg(reinterpret_cast<const float4*>(at + (size_t)q * 4 * p.part_rows));
                if (o.y == 0.f) continue;  // (a part without a visible key has nothing in its sums)
                const float mn = fmaxf(mj, o.x), f = ex2(o.x - mn), e = lj != 0.f ? ex2(mj - mn) : 0.f;
                mj = mn;
                lj = e * lj + f * o.y;
#pragma unroll
                for (int q = 0; q < D / 8; ++q) {
                    u[4 * q] = e * u[4 * q] + f * v[q].x; u[4 * q + 1] = e * u[4 * q + 1] + f * v[q].y;
                    u[4 * q + 2] = e * u[4 * q + 2] + f * v[q].z; u[4 * q + 3] = e * u[4 * q + 3] + f * v[q].w;
                }
            }
            const float inv = 1.f / lj;
            __nv_bfloat16* out = p.o + (((size_t)y.n * p.M + row / p.group) * p.Hq + y.kh * p.group + row % p.group) * D + grp * (D / 2);
#pragma unroll
            for (int q = 0; q < D / 2; q += 16) {
                float w[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) w[e] = inv * u[q + e];
                put16(out + q, w);
            }
        }
    } else if (warp == kSoft) {
        // ---- loads: a lane per page -------------------------------------------------
        const int pages = KT / p.c.page;
        // Q follows the first step's keys and values, once the S before it are done
        auto load_q = [&]() {
            if (!p.q_tma) return true;
            if (x > 0 && !(ok = warp_wait(&s.k_free[(x - 1) % NST], ((x - 1) / NST) & 1))) return false;
            if (lane == 0) {
                mbar_arrive_expect(&s.q_full, D / 64 * PANEL);
#pragma unroll
                for (int y = 0; y < D / 64; ++y)
                    tma_load_3d(s.Q[y], &p.qmap, 64 * y, g.kh * p.group, g.n * p.M + g.rt * (128 / p.group), &s.q_full);
            }
            __syncwarp();
            ++segs;
            return true;
        };
        while (ok && w.next(p, g)) {
            for (int t = g.t0; t < g.t1; ++t, ++x) {
                const int st = x % NST, use = x / NST;
                if (t == g.span.steps - 1) {  // the nodes
                    if (use > 0 && !(ok = warp_wait(&s.k_free[st], (use - 1) & 1))) break;
                    if (lane == 0) {
                        mbar_arrive_expect(&s.k_full[st], D / 64 * PANEL / 2);
#pragma unroll
                        for (int y = 0; y < D / 64; ++y) tma_load_3d(s.K[st][y], &p.knode, 64 * y, g.kh, g.n * p.M, &s.k_full[st]);
                    }
                    if (use > 0 && !(ok = warp_wait(&s.v_free[st], (use - 1) & 1))) { ++x; break; }
                    if (lane == 0) {
                        mbar_arrive_expect(&s.v_full[st], D / 64 * PANEL / 2);
#pragma unroll
                        for (int y = 0; y < D / 64; ++y) tma_load_3d(s.V[st][y], &p.vnode, 64 * y, g.kh, g.n * p.M, &s.v_full[st]);
                    }
                    if (t == g.t0 && !load_q()) { ++x; break; }
                    continue;
                }
                const int pos = (g.span.first + t) * KT + lane * p.c.page;
                int pg = -1;
                // (a page wholly before the window may have been given back: its entry is not read)
                if (lane < pages && pos < g.span.len && (p.window == 0 || pos + p.c.page > g.span.len - p.window + 1)) {
                    pg = p.c.table[(size_t)g.n * p.c.width + pos / p.c.page];
                    if (pg < 0 || pg >= p.c.pages) {
                        atomicOr(p.status, 2u);
                        pg = -1;
                    }
                }
                const uint32_t got = __ballot_sync(0xffffffffu, pg >= 0);
                const uint32_t bytes = (uint32_t)__popc(got) * p.c.page * D * 2;
                const int at = lane * p.c.page * 128;
                if (use > 0 && !(ok = warp_wait(&s.k_free[st], (use - 1) & 1))) break;
                if (lane == 0) {
                    uint32_t have = 0;
                    for (int i = 0; i < pages; ++i)
                        if (got >> i & 1) have |= ((1u << (p.c.page / 16)) - 1u) << (i * (p.c.page / 16));
                    s.have[x % (2 * NST)] = have;
                    mbar_arrive_expect(&s.k_full[st], bytes);
                }
                __syncwarp();
                if (pg >= 0) {
#pragma unroll
                    for (int y = 0; y < D / 64; ++y) tma_load_3d(s.K[st][y] + at, &p.kmap, 64 * y, g.kh, pg * p.c.page, &s.k_full[st]);
                }
                __syncwarp();
                if (use > 0 && !(ok = warp_wait(&s.v_free[st], (use - 1) & 1))) { ++x; break; }
                if (lane == 0) mbar_arrive_expect(&s.v_full[st], bytes);
                __syncwarp();
                if (pg >= 0) {
#pragma unroll
                    for (int y = 0; y < D / 64; ++y) tma_load_3d(s.V[st][y] + at, &p.vmap, 64 * y, g.kh, pg * p.c.page, &s.v_full[st]);
                }
                __syncwarp();
                if (t == g.t0 && !load_q()) { ++x; break; }
            }
        }
        if (p.q_tma && segs) warp_wait(&s.q_full, (segs - 1) & 1);
        // no copy may be in flight when the CTA ends (a stage that a wait gave up on makes this
        // one give up as well: its copies are in by then)
        for (int y = max(0, x - NST); y < x; ++y) {
            warp_wait(&s.k_full[y % NST], (y / NST) & 1);
            warp_wait(&s.v_full[y % NST], (y / NST) & 1);
        }
    } else {
        // ---- products: S of step x, then O of the step before -------------------------
        constexpr uint32_t ID_S = tc5::idesc_bf16(128, KT, false, false), ID_O = tc5::idesc_bf16(128, D, false, true);
        constexpr uint64_t KROWS = (16 * 128) >> 4, KCOLS = 32 >> 4, KPANEL = PANEL >> 4;
        const uint64_t dQ = tc5::kmajor<KT>(smem_u32(s.Q), 0);
        while (ok && w.next(p, g)) {
            if (!(ok = warp_wait(&s.q_full, segs & 1))) break;
            const int x0 = x, x1 = x + (g.t1 - g.t0);
            for (; x <= x1; ++x) {
                if (x < x1) {
                    const int st = x % NST;
                    // S goes where P of two steps before was: its product must be done with it
                    if (x >= 2 && !(ok = warp_wait(&s.o_done[x & 1], ((x >> 1) & 1) ^ 1))) break;
                    if (!(ok = warp_wait(&s.k_full[st], (x / NST) & 1))) break;
                    tc5::fence_after();
                    if (elect_one()) {
                        const uint64_t dK = tc5::kmajor<KT>(smem_u32(s.K[st]), 0);
#pragma unroll 2
                        for (int k = 0; k < D / 16; ++k) {
                            const uint64_t at = (k >> 2) * KPANEL + (k & 3) * KCOLS;
                            tc5::mma(tm + TG * (x & 1), dQ + at, dK + at, ID_S, k > 0);
                        }
                        tc5::commit(&s.s_ready[x & 1]);
                        tc5::commit(&s.k_free[st]);
                    }
                    __syncwarp();
                }
                if (x > x0) {
                    const int y = x - 1, st = y % NST;
                    // the O of the segment before has been read
                    if (y == x0 && segs > 0 && !(ok = warp_wait(&s.seg_done, (segs - 1) & 1))) break;
                    if (!(ok = warp_wait(&s.v_full[st], (y / NST) & 1))) break;
                    if (!(ok = warp_wait(&s.p_ready[y & 1], (y >> 1) & 1))) break;
                    tc5::fence_after();
                    if (elect_one()) {
                        const uint64_t dV = tc5::mnmajor(smem_u32(s.V[st]), 0, PANEL);
                        const uint32_t tp = tm + TG * (y & 1);
#pragma unroll 2
                        for (int k = 0; k < KT / 16; ++k)
                            tc5::mma_ts(tp + TO, tp + 8 * k, dV + k * KROWS, ID_O, k > 0 || y - x0 >= 2);
                        tc5::commit(&s.o_done[y & 1]);
                        tc5::commit(&s.v_free[st]);
                    }
                    __syncwarp();
                }
            }
            if (!ok) break;
            x = x1;
            ++segs;
        }
        if (elect_one()) tc5::commit(&s.drain);  // no product may be in flight when the CTA ends
        warp_wait(&s.drain, 0);
    }
    if (!ok && lane == 0) atomicOr(p.status, 1u);
    tc5::fence_before();
    __syncthreads();
    if (warp == kSoft + 1) {
        tc5::fence_after();
        tc5::dealloc(tm, 512);
    }
}

constexpr int kCtas = 148;  // one per SM

// Workspace: the status word, the units' counters, the parts.
size_t count_bytes(int N, int M, int Hq, int Hkv) {
    return ((size_t)N * Hkv * ((M * (Hq / Hkv) + 127) / 128) * 4 + 255) & ~(size_t)255;
}
int part_rows(int M, int group) { return M * group < 128 ? M * group : 128; }
int part_floats(int M, int group, int d) { return (part_rows(M, group) * (d + 2) + 3) & ~3; }
size_t part_bytes(int M, int group, int d) { return (size_t)kCtas * 2 * part_floats(M, group, d) * 4; }

template <int D>
bool launch_attn(Params& a, const void* k, const void* v, cudaStream_t st) {
    const int box = a.c.page;
    if (!encode_head_map(&a.kmap, a.c.k, (long long)a.c.pages * a.c.page, a.Hkv, D, box) ||
        !encode_head_map(&a.vmap, a.c.v, (long long)a.c.pages * a.c.page, a.Hkv, D, box) ||
        !encode_head_map(&a.knode, k, (long long)a.N * a.M, a.Hkv, D, KT / 2) ||
        !encode_head_map(&a.vnode, v, (long long)a.N * a.M, a.Hkv, D, KT / 2))
        return false;
    a.q_tma = a.scale > 0.f && 128 % a.group == 0;
    if (a.q_tma && !encode_head_map(&a.qmap, a.q, (long long)a.N * a.M, a.Hq, D, 128 / a.group, a.group)) return false;
    const int smem = sizeof(Smem<D>) + 1024;
    cudaFuncSetAttribute(tree_attn_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    const long long units = (long long)a.N * a.Hkv * a.row_tiles;
    // (3 sequences of 8 heads and 512 visible tokens: 19 us, cut evenly 26 us)
    a.split = units * 2 <= kCtas ? (int)(kCtas / units) : 0;
    GDN_LAUNCH("tree_attn", st, (tree_attn_kernel<D><<<a.split ? (unsigned)(units * a.split) : kCtas, kThreads, smem, st>>>(a)));
    return true;
}

// ---- append ------------------------------------------------------------------
// One CTA per sequence: the accepted node's root path, then its K and V rows to
// the cache positions after the last, in 16-byte pieces.  Four dependent reads (node,
// parents, length and page, rows) and a launch are what it takes: 8.4 us for 256 sequences
// of up to 32 nodes, 7.4 us for 5.
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
    // positions, rounded up to whole key tiles and with the nodes behind them, are 32-bit
    if ((long long)width * page > 0x7fffffffLL - 2 * KT) return GDN_ERR_INVALID_ARG;
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
    return kStatusBytes + count_bytes(N, M, Hq, Hkv) + part_bytes(M, Hq / Hkv, d);
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
    const size_t counts = count_bytes(N, M, Hq, Hkv);
    if (cudaMemsetAsync(ws, 0, kStatusBytes + counts, st) != cudaSuccess) return GDN_ERR_CUDA;
    const Cache c{(const __nv_bfloat16*)k_cache, (const __nv_bfloat16*)v_cache, block_table, cache_len, pages, page, width};
    Params a{};
    a.c = c;
    a.N = N; a.M = M; a.Hq = Hq; a.Hkv = Hkv; a.group = Hq / Hkv;
    a.row_tiles = (M * a.group + 127) / 128;
    a.window = window; a.scale = scale; a.parent = parent;
    a.q = (const __nv_bfloat16*)q; a.o = (__nv_bfloat16*)o;
    a.count = (unsigned int*)((char*)ws + kStatusBytes);
    a.part = (float*)((char*)ws + kStatusBytes + counts);
    a.part_rows = part_rows(M, a.group);
    a.part_floats = part_floats(M, a.group, d);
    a.status = (unsigned int*)ws;
    const bool fine = d == 64 ? launch_attn<64>(a, k, v, st) : launch_attn<128>(a, k, v, st);
    if (!fine) return GDN_ERR_CUDA;
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
