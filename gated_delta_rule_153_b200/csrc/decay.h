// decay.h -- shapes and launchers of linear attention with a decay per head
// (gdn_decay_*), shared between its entry points and its kernels.
#pragma once

#include <cuda_runtime.h>
#include <math.h>
#include <stddef.h>

#include "../../include/gdn.h"

namespace gdn {
namespace decay {

// The sequences of a call: nseq sequences of one row of `rows` tokens.  cu is
// null for a batch (sequence s = tokens s*len .. s*len + len - 1).
struct Seqs {
    const int* cu;
    int nseq, len;
    int rows;  // tokens of the tensors in all
};

struct Problem {
    Seqs seq;
    int H, Hk, dk, dv;
    gdn_dtype dtype;
    float scale;
};

// Chunks of C tokens are cut from each sequence's own first token; chunk c of
// sequence s has slot (first token / C) + s + c.  Slots of different sequences
// never meet, whatever their lengths, so no prefix sum over them is needed.
__host__ __device__ inline long long chunk_slots(const Seqs& q, int C) { return q.rows / C + (long long)q.nseq; }

// Items of a grid (item_of), each with one CTA per head and block of value channels; what
// the runs leave is kept per item and head.
inline long long items(const Seqs& q, int runs, int run_len) {
    return q.cu && runs > 1 ? q.rows / run_len + (long long)q.nseq : (long long)q.nseq * runs;
}

// The longest sequence as far as the host can tell: a row cut at random into n sequences
// has a longest of rows (1 + 1/2 + .. + 1/n) / n on average, the sum being ln n + 0.577 + 1/2n.
inline double longest(const Seqs& q) {
    const double n = q.nseq;
    return q.cu && q.nseq > 1 ? q.rows * (log(n) + 0.577 + 0.5 / n) / n : q.len;
}

#ifdef __CUDACC__
// The token range of sequence s.  False if its offsets are not one: out of the
// row, decreasing, or below the offset before them (it would then share tokens
// with an earlier sequence); nothing of such a sequence is read or written.
__device__ __forceinline__ bool span_of(const Seqs& q, int s, long long& tok0, int& n) {
    tok0 = (long long)s * q.len;
    n = q.len;
    if (!q.cu) return true;
    const int a = q.cu[s], b = q.cu[s + 1];
    tok0 = a;
    n = b - a;
    return !(a < 0 || b < a || b > q.rows || (s > 0 && q.cu[s - 1] > a));
}

// Chains cut into runs of `run_len` tokens: the sequence and run of a CTA's item.  A batch
// has the items of run 0 first, then those of run 1; packed sequences have theirs one
// sequence after the other, so that the CTAs with something to do are neighbours and
// the device spreads them evenly: at most rows / run_len + nseq of them, all of a grid.
// `skip` (0 or 1) leaves out the last runs.  `first` is the place of the sequence's run 0
// in what the runs leave: its item among those without last runs.  Called by whole
// warps; false past the end.
__device__ __forceinline__ bool item_of(const Seqs& q, int runs, int run_len, int skip, int item, int& seq, int& run,
                                        int& first) {
    if (!q.cu || runs == 1) {
        seq = item % q.nseq;
        run = item / q.nseq;
        first = seq * runs;
        return true;
    }
    const int lane = threadIdx.x & 31, all = item;
    for (int s0 = 0; s0 < q.nseq; s0 += 32) {
        long long tok0;
        int n, mine = 0;
        if (s0 + lane < q.nseq)  // a sequence whose offsets are none has one, to say so
            mine = span_of(q, s0 + lane, tok0, n) && n > run_len ? (n + run_len - 1) / run_len - skip : 1 - skip;
        int upto = mine;
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += v;
        }
        const unsigned past = __ballot_sync(0xffffffffu, upto > item);
        if (past) {
            const int at = __ffs(past) - 1;
            seq = s0 + at;
            run = item - __shfl_sync(0xffffffffu, upto - mine, at);
            first = all - run - (skip ? 0 : seq);  // every sequence before has one last run
            return true;
        }
        item -= __shfl_sync(0xffffffffu, upto, 31);
    }
    return false;
}
#endif

// fp32 arithmetic on CUDA cores, any supported dims (decay.cu).
size_t simt_fwd_workspace(const Problem& p);
size_t simt_bwd_workspace(const Problem& p);
void launch_simt_fwd(const Problem& p, const void* q, const void* k, const void* v, const float* g,
                     const float* h0, void* o, float* hT, void* ws, cudaStream_t st);
void launch_decay_step(int N, int H, int Hk, int dk, int dv, gdn_dtype dtype, float scale, const void* q,
                       const void* k, const void* v, const float* g, float* state, void* o,
                       cudaStream_t st);
void launch_simt_bwd(const Problem& p, const void* q, const void* k, const void* v, const float* g,
                     const float* h0, const void* dO, const float* dhT, void* dq, void* dk, void* dv,
                     float* dg, float* dh0, void* ws, cudaStream_t st);

// dq or dk of shared key heads: [token][H][d] fp32 summed over each group into [token][Hk][d].
void launch_group_sum(const Problem& p, const float* part_q, const float* part_k, void* dq, void* dk, cudaStream_t st);

// Sequences of up to 64 tokens, packed ones on average: the tensor-core kernels then keep
// what rounding the pair products of such chunks leaves.  The code for it costs a long call
// (350M-scale forward 53 -> 61 us, local gradients 128 -> 138), a short one little (256
// sequences of 16 tokens, 8 heads, 128 x 128: 214 -> 227 us, their backward 559 -> 574).
inline bool short_sequences(const Problem& p) {
    return (p.seq.cu ? (long long)p.seq.rows : (long long)p.seq.len * p.seq.nseq) <= 64ll * p.seq.nseq;
}

// Tensor cores: bf16 with dk, dv in {64, 128} (decay_walk.cu).  The launchers return
// false if a tensor map could not be encoded (nothing launched).
bool tc_supported(const Problem& p);
size_t tc_fwd_workspace(const Problem& p);
// The backward (decay_bwd.cu).  launch_tc_states: the state entering each chunk of
// 128 tokens and the gradient of the one leaving it, in fp32 as images of their upper and
// lower halves, [slot][head][2][dv/64][dk][64], and cross [dv/64][slot][head] = e^{G_last} <S, dS>.
size_t tc_states_workspace(const Problem& p);
bool launch_tc_states(const Problem& p, const void* q, const void* k, const void* v, const float* g, const float* h0,
                      const void* dO, const float* dhT, float* dh0, void* S, void* dS, float* cross, void* runs, void* ws,
                      cudaStream_t st);
size_t tc_bwd_workspace(const Problem& p);
bool launch_tc_bwd(const Problem& p, const void* q, const void* k, const void* v, const float* g, const float* h0,
                   const void* dO, const float* dhT, void* dq, void* dk, void* dv, float* dg, float* dh0, void* ws,
                   cudaStream_t st);
bool launch_tc_fwd(const Problem& p, const void* q, const void* k, const void* v, const float* g, const float* h0,
                   void* o, float* hT, void* ws, cudaStream_t st);

}  // namespace decay
}  // namespace gdn
