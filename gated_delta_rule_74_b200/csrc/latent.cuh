// Shapes and device helpers shared by the latent-cache kernels (not part of the C ABI).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "kda_common.cuh"

namespace kda {

struct LatentAppendShape {
  long long tokens;                 // rows of kv: N * L, or the packed T
  int N, L, H, rank, rope;          // L = 0: packed (cu_seqlens)
  int num_pages, page_size, max_pages;
  long long page_stride, row_stride;       // cache, in elements
  long long kv_stride;                     // kv, elements between tokens
  long long q_tok, q_head, qo_tok, qo_head;
  float eps;
  int interleaved;
  int parts;                        // warps a token, set by the launcher: 1, or the row's and the heads'
};

cudaError_t launch_latent_append(const void* kv, const float* w, const float* inv_freq,
                                 const void* q_pe, void* q_out, void* cache,
                                 const int32_t* page_table, const int32_t* seq_lens,
                                 const int32_t* cu_seqlens, LatentAppendShape sh, int dtype,
                                 cudaStream_t stream);

cudaError_t launch_verify_tokens(const float* target, const float* draft,
                                 const int32_t* draft_tokens, const float* uniforms,
                                 const int32_t* draft_lens, int32_t* tokens, int32_t* accepted,
                                 int N, int L, int V, cudaStream_t stream);

// First row of sequence n in cu_seqlens, kept inside [0, T] whatever it holds.
__device__ __forceinline__ int cu_at(const int32_t* cu, int n, int T) {
  return min(max(__ldg(cu + n), 0), T);
}

// The sequence of token `tok`, its first token and its token count; false for a token of
// none.  Packed: the first sequence whose end lies behind the token, 32 ends a step over
// the lanes.  Warp-cooperative (`tok` uniform over the warp).
__device__ __forceinline__ bool token_sequence(long long tok, int N, int L, const int32_t* cu,
                                               int T, int lane, int* seq, int* first, int* count) {
  if (!cu) {
    *seq = (int)((uint32_t)tok / (uint32_t)L);          // tokens are fewer than 2^31
    *first = *seq * L;
    *count = L;
    return true;
  }
  int lo = 0, hi = N;                       // the answer lies in [lo, hi]; hi = N: none
  while (lo < hi) {
    const int step = (hi - lo + 31) / 32;
    const int n = lo + (lane + 1) * step - 1;          // last sequence of this lane's share
    const bool past = n >= hi || cu_at(cu, n + 1, T) > tok;
    const unsigned vote = __ballot_sync(0xffffffffu, past);
    const int share = vote ? __ffs(vote) - 1 : 32;
    lo += share * step;                                 // the shares before end at or before tok
    hi = min(hi, lo + step - 1);
  }
  if (lo >= N) return false;
  *seq = lo;
  *first = cu_at(cu, lo, T);
  *count = cu_at(cu, lo + 1, T) - *first;
  return tok >= *first && tok < *first + *count;
}

}  // namespace kda
