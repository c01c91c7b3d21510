// Verification of drafted tokens (kda_verify_tokens).
//
// Of a sequence with L drafted tokens x_i, target probabilities p_0 .. p_L and draft
// probabilities q_0 .. q_{L-1} (none: q_i(x_i) = 1 and 0 elsewhere), given u_0 .. u_L:
//     draft i stands while u_i q_i(x_i) < p_i(x_i);  a = the drafts before the first that falls
//     weights w = (p_a - q_a)_+ if a < L, else p_L;  token a = min {v : sum_{v' <= v} w > u_L sum w}
// so that the tokens are distributed as the target's own.  Products and sums are 64-bit
// (an fp32 product or difference is exact there, and the running sum is good to 1e-15).
//
// Bound by memory: of all the rows given, one target row and (after a rejection) one draft
// row a sequence are read.  A cluster of C CTAs shares a sequence, each warp summing
// four neighbouring stretches of the vocabulary; the stretches' sums meet in the first CTA's
// shared memory, whose first warp finds the stretch that the threshold falls into and reads
// that one again, 256 elements at a time and the last of them lane by lane.  No atomics:
// the same inputs give the same tokens.  C is the largest of 1, 2, 4, 8 whose CTAs are all
// resident at once (four an SM, for eight loads of each row in flight a lane) and whose
// stretches stay above 64 elements.  Apart from the rows' bytes a call costs four dependent
// trips to memory (drafts, their probabilities, the row, the stretch again).
#include <cooperative_groups.h>

#include "kda_common.cuh"
#include "latent.cuh"

namespace kda {
namespace {
namespace cg = cooperative_groups;

constexpr int kVT = 256;                 // threads of a CTA
constexpr int kVW = kVT / 32;
constexpr int kVPerSm = 4;               // resident CTAs of an SM
constexpr int kSub = 4;                  // stretches of a warp
constexpr int kMaxCluster = 8;
constexpr int kUnroll = 8, kBlock = 32 * kUnroll;

// Weight of an element: what the target has over the draft, never below zero; a NaN is none.
__device__ __forceinline__ double weight(float p, float q) {
  const bool over = p > q;
  return (double)(over ? p : 0.f) - (double)(over ? q : 0.f);
}

// This lane's share of the weights of [v0, v1).
template <bool kDraft>
__device__ __forceinline__ double lane_sum(const float* p, const float* q, int v0, int v1, int lane) {
  double sum = 0.0;
  for (int v = v0 + lane; v < v1; v += kBlock) {
    float pv[kUnroll], qv[kUnroll];
    const bool whole = v - lane + kBlock <= v1;
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const bool in = whole || v + 32 * i < v1;
      pv[i] = in ? __ldg(p + v + 32 * i) : 0.f;
      qv[i] = kDraft && in ? __ldg(q + v + 32 * i) : 0.f;
    }
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) sum += weight(pv[i], qv[i]);
  }
  return sum;
}

__global__ void __launch_bounds__(kVT, kVPerSm)
kda_verify_kernel(const float* __restrict__ target, const float* __restrict__ draft,
                  const int32_t* __restrict__ draft_tokens, const float* __restrict__ uniforms,
                  const int32_t* __restrict__ draft_lens, int32_t* __restrict__ tokens,
                  int32_t* __restrict__ accepted, int L, int V) {
  __shared__ double s_sum[kMaxCluster * kVW * kSub];   // the first CTA's: every stretch's sum
  __shared__ int s_acc;
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const long long n = blockIdx.x / C;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  cluster.barrier_arrive();                          // before the first remote store: all CTAs run

  const int Ln = draft_lens ? min(max(__ldg(draft_lens + n), 0), L) : L;
  const int32_t* xs = draft_tokens + n * L;
  const float* us = uniforms + n * (L + 1);
  if (warp == 0) {
    int a = Ln;
    for (int i0 = 0; i0 < Ln && a == Ln; i0 += 32) {
      const int i = i0 + lane;
      bool falls = false;
      if (i < Ln) {
        const int x = __ldg(xs + i);
        falls = true;                                // a token outside the vocabulary falls
        if (x >= 0 && x < V) {
          const float px = __ldg(target + (n * (L + 1) + i) * V + x);
          const float qx = draft ? __ldg(draft + (n * L + i) * V + x) : 1.0f;
          falls = !((double)__ldg(us + i) * (double)qx < (double)px);
        }
      }
      const unsigned vote = __ballot_sync(0xffffffffu, falls);
      if (vote) a = i0 + __ffs(vote) - 1;
    }
    if (lane == 0) s_acc = a;
  }
  __syncthreads();
  const int a = s_acc;
  const bool rejected = a < Ln;
  const float* p = target + (n * (L + 1) + a) * V;
  const float* q = rejected && draft ? draft + (n * L + a) * V : nullptr;
  const int xr = rejected ? __ldg(xs + a) : -1;      // without draft rows: its weight is zero
  const int cut = rejected && !draft ? xr : -1;

  // ---- this warp's stretches
  const int S = C * kVW * kSub;
  const int len = (V + S - 1) / S;
  const int st0 = (rank * kVW + warp) * kSub;
  double sum[kSub];
#pragma unroll
  for (int i = 0; i < kSub; ++i) {
    const int v0 = (int)min((long long)(st0 + i) * len, (long long)V);
    const int v1 = (int)min((long long)v0 + len, (long long)V);
    if (q) {
      sum[i] = lane_sum<true>(p, q, v0, v1, lane);
    } else if (cut >= v0 && cut < v1) {
      sum[i] = lane_sum<false>(p, q, v0, cut, lane) + lane_sum<false>(p, q, cut + 1, v1, lane);
    } else {
      sum[i] = lane_sum<false>(p, q, v0, v1, lane);
    }
  }
#pragma unroll
  for (int i = 0; i < kSub; ++i)
#pragma unroll
    for (int o = 16; o; o >>= 1) sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], o);
  cluster.barrier_wait();
  if (lane == 0) {
    double* d = cluster.map_shared_rank(&s_sum[st0], 0);
#pragma unroll
    for (int i = 0; i < kSub; ++i) d[i] = sum[i];
  }
  cluster.barrier_arrive();
  if (rank != 0) return;                             // nothing of this CTA is read by another
  cluster.barrier_wait();
  if (warp != 0) return;

  // ---- the first stretch whose running sum passes u * total (S <= 256: eight a lane)
  constexpr int P = kMaxCluster * kVW * kSub / 32;
  double part[P], mine = 0.0;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    part[i] = lane * P + i < S ? s_sum[lane * P + i] : 0.0;
    mine += part[i];
  }
  double run = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double up = __shfl_up_sync(0xffffffffu, run, o);
    if (lane >= o) run += up;
  }
  const double total = __shfl_sync(0xffffffffu, run, 31);
  const double thr = (double)__ldg(us + L) * total;
  run -= mine;                                       // what lies before this lane's stretches
  int hit = -1, last = -1;
  double before = 0.0;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    if (part[i] > 0.0) {
      last = lane * P + i;
      if (hit < 0 && run + part[i] > thr) {
        hit = last;
        before = run;
      }
    }
    run += part[i];
  }
  const unsigned hits = __ballot_sync(0xffffffffu, hit >= 0);
  const unsigned lasts = __ballot_sync(0xffffffffu, last >= 0);
  int tok = -1;
  if (lasts) {
    // rounding may leave the threshold behind every sum: then the last weight there is
    const int src = hits ? __ffs(hits) - 1 : 31 - __clz(lasts);
    const int st = __shfl_sync(0xffffffffu, hits ? hit : last, src);
    before = __shfl_sync(0xffffffffu, before, src);
    const int b0 = (int)min((long long)st * len, (long long)V);
    const int b1 = (int)min((long long)b0 + len, (long long)V);
    // its first block of 256 whose running sum passes (or the last with any weight)
    constexpr int kB = kUnroll;
    float pv[kB], qv[kB];
    auto load = [&](int v) {
#pragma unroll
      for (int i = 0; i < kB; ++i) {
        const int e = v + 32 * i + lane;
        const bool in = e < b1 && e != cut;
        pv[i] = in ? __ldg(p + e) : 0.f;
        qv[i] = in && q ? __ldg(q + e) : 0.f;
      }
    };
    int at = -1;
    double at_before = 0.0;
    bool passed = false;
    load(b0);
    for (int v = b0; v < b1 && !passed; v += kBlock) {
      double bs = 0.0;
#pragma unroll
      for (int i = 0; i < kB; ++i) bs += weight(pv[i], qv[i]);
      if (v + kBlock < b1) load(v + kBlock);
#pragma unroll
      for (int o = 16; o; o >>= 1) bs += __shfl_xor_sync(0xffffffffu, bs, o);
      if (bs > 0.0) {
        at = v;
        at_before = before;
        passed = hits && before + bs > thr;
      }
      before += bs;
    }
    if (at >= 0) {
      load(at);
      bool done = false;
#pragma unroll
      for (int i = 0; i < kB; ++i) {
        const double wv = weight(pv[i], qv[i]);
        double r = wv;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const double up = __shfl_up_sync(0xffffffffu, r, o);
          if (lane >= o) r += up;
        }
        const unsigned some = __ballot_sync(0xffffffffu, wv > 0.0);
        const unsigned over = __ballot_sync(0xffffffffu, wv > 0.0 && passed && at_before + r > thr);
        if (!done && some) tok = at + 32 * i + (over ? __ffs(over) - 1 : 31 - __clz(some));
        done = done || over;
        at_before += __shfl_sync(0xffffffffu, r, 31);
      }
    }
  } else if (rejected && xr >= 0 && xr < V) {
    tok = xr;                                        // p = q up to rounding: the draft is a draw of p
  }

  for (int i = lane; i <= L; i += 32) tokens[n * (L + 1) + i] = i < a ? __ldg(xs + i) : i == a ? tok : -1;
  if (lane == 0) accepted[n] = a;
}

}  // namespace

cudaError_t launch_verify_tokens(const float* target, const float* draft,
                                 const int32_t* draft_tokens, const float* uniforms,
                                 const int32_t* draft_lens, int32_t* tokens, int32_t* accepted,
                                 int N, int L, int V, cudaStream_t stream) {
  int sms = 0;
  if (!device_ctx(&sms, nullptr)) return cudaErrorInvalidDevice;
  int C = 1;
  while (C < kMaxCluster && 2LL * C * N <= (long long)kVPerSm * sms && V >= 2 * C * kVW * kSub * 64)
    C *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(N * C));
  cfg.blockDim = dim3(kVT);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim = {(unsigned)C, 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaSuccess;
  KDA_TIMED(KDA_KERNEL_VERIFY, stream,
            e = cudaLaunchKernelEx(&cfg, kda_verify_kernel, target, draft, draft_tokens, uniforms,
                                   draft_lens, tokens, accepted, L, V));
  note_launches(1);
  return e;
}

}  // namespace kda
