// Work division, partial results and launchers of the latent attention (not part of the
// C ABI).
//
// A sequence's rows (new token i, head h -> row i H + h, contiguous in q) are cut into
// blocks of `nr` rows; a block attends to the sequence's first `lim` tokens, lim the last
// of its rows' causal limits, in tiles of `kt` tokens.  All tiles of all blocks form one
// line, in order of sequence, block and tile, each block's behind `lead` empty places for
// what it costs besides (its start and its results), and CTA c of G takes the stretch
// [W c / G, W (c + 1) / G) of its W places: every CTA the same number to within one,
// whatever the lengths, with at most two blocks a CTA that others share.  A block that one
// CTA has whole is written straight to `out`; of the others each CTA leaves a partial
// result (normalised fp32 rows and their log-sums), which the join kernel adds up in the
// order of the CTAs.  Nothing is planned on the host, which does not know the lengths.
#pragma once

#include "latent.cuh"

namespace kda {

struct LatentAttnShape {
  int N, L, T, H, rank, rope;       // L = 0: packed, T tokens in all (cu_seqlens)
  int num_pages, page_size, max_pages;
  long long page_stride, row_stride;
  float scale;
};

// Workspace of one call: the CTAs' headers, then 2 G partial results of nr rows (slot 2 c:
// the block that CTA c's stretch begins inside of, 2 c + 1: the one that it ends inside of).
struct LatentPartials {
  int4* head;                       // [G] {first row, rows (0: nothing to join), last CTA, -}
  float* lse;                       // [2 G][nr], natural logarithm
  float* o;                         // [2 G][nr][rank]
};
constexpr int kLatentMaxCtas = 1024;
constexpr uint32_t kLatentPolls = 1u << 22;   // of a wait, before it gives up

inline size_t latent_scratch_bytes(int G, int nr, int rank) {
  return (size_t)kLatentMaxCtas * sizeof(int4) + (((size_t)2 * G * nr * 4 + 255) & ~(size_t)255) +
         (size_t)2 * G * nr * rank * 4;
}
inline LatentPartials latent_partials(void* ws, int G, int nr) {
  char* p = static_cast<char*>(ws);
  LatentPartials r;
  r.head = reinterpret_cast<int4*>(p);
  r.lse = reinterpret_cast<float*>(p + (size_t)kLatentMaxCtas * sizeof(int4));
  r.o = r.lse + ((((size_t)2 * G * nr * 4 + 255) & ~(size_t)255) >> 2);
  return r;
}

// Scratch bytes of one call; rows a sequence has (packed: on average) decide the block.
size_t latent_attn_scratch_bytes(int N, int L, int T, int H, int rank, int rope, int page_size,
                                 int dtype, int sms);
cudaError_t launch_latent_attn(const void* q, const void* cache, const int32_t* page_table,
                               const int32_t* seq_lens, const int32_t* cu_seqlens, void* out,
                               float* lse, const LatentAttnShape& sh, int dtype,
                               cudaStream_t stream, const Workspace* ws,
                               uint32_t polls = kLatentPolls);

// The tensor-core kernel (latent_attn_tc.cu): bf16, pages of a multiple of 8 rows.
bool latent_tc_supported(int dtype, int page_size);
size_t latent_tc_scratch_bytes(int N, int L, int T, int H, int rank, int sms);
cudaError_t launch_latent_tc(const void* q, const void* cache, const int32_t* page_table,
                             const int32_t* seq_lens, const int32_t* cu_seqlens, void* out,
                             float* lse, const LatentAttnShape& sh, int sms, void* buf,
                             cudaStream_t stream, uint32_t polls);
cudaError_t launch_latent_join(void* out, float* lse, const LatentPartials& pt, int G, int nr,
                               const LatentAttnShape& sh, int dtype, cudaStream_t stream);

// ------------------------------------------------------------------ device side
// sum_{i < n} floor((a i + b) / m), a, b >= 0, m > 0
__device__ inline long long floor_sum(long long n, long long m, long long a, long long b) {
  long long s = 0;
  while (n > 0) {
    if (a >= m) {
      s += (n - 1) * n / 2 * (a / m);
      a %= m;
    }
    if (b >= m) {
      s += n * (b / m);
      b %= m;
    }
    const long long y = a * n + b;
    if (y < m) break;
    n = y / m;
    b = y % m;
    const long long t = m;
    m = a;
    a = t;
  }
  return s;
}

// One sequence's blocks.
struct LatentSeq {
  int len, cnt, first;              // cached tokens, new tokens, first new token (row of q / H)
  int nb;                           // blocks
  int b1;                           // blocks before this one see no tile (one is counted)
  long long base;                   // see tiles()

  __device__ LatentSeq(const LatentAttnShape& sh, const int32_t* seq_lens, const int32_t* cu,
                       int n, int nr, int kt) {
    const long long cap = (long long)sh.max_pages * sh.page_size;
    len = (int)min((long long)max(__ldg(seq_lens + n), 0), min(cap, (long long)INT32_MAX - 4096));
    if (cu) {
      first = cu_at(cu, n, sh.T);
      cnt = max(cu_at(cu, n + 1, sh.T) - first, 0);
    } else {
      first = n * sh.L;
      cnt = sh.L;
    }
    nb = (int)(((long long)cnt * sh.H + nr - 1) / nr);
    const long long need = (long long)kt * sh.H;
    base = nr - 1 + (long long)(len - cnt + kt) * sh.H;
    b1 = base >= need ? 0 : (int)min((need - base + nr - 1) / nr, (long long)nb);
  }
  // Tiles of block b: its last row's limit is len - cnt + (b nr + nr - 1) / H + 1, so that
  // ceil(limit / kt) = floor((b nr + base) / (kt H)); one at least.
  __device__ int tiles(int b, const LatentAttnShape& sh, int nr, int kt) const {
    if (b == nb - 1) return max(1, (len + kt - 1) / kt);
    return b < b1 ? 1 : (int)(((long long)b * nr + base) / ((long long)kt * sh.H));
  }
  // Places of blocks [0, b), b < nb
  __device__ long long before(int b, const LatentAttnShape& sh, int nr, int kt, int lead) const {
    const long long n = (long long)b * lead;
    if (b <= b1) return n + b;
    return n + b1 + floor_sum(b - b1, (long long)kt * sh.H, nr, base + (long long)nr * b1);
  }
  __device__ long long total(const LatentAttnShape& sh, int nr, int kt, int lead) const {
    return nb == 0 ? 0 : before(nb - 1, sh, nr, kt, lead) + lead + tiles(nb - 1, sh, nr, kt);
  }
};

// A CTA's stretch: where it starts and how many places it has.
struct LatentStart {
  int n, b, at;                     // sequence, block, first place inside of the block
  long long places;                 // of the stretch (0: nothing to do)
  long long pos;                    // its first place in the line
  long long W;                      // places of the line
  int G;                            // CTAs that have a stretch
};

// All threads of the CTA (a multiple of 32, at most 1024); `sh_sum` 33 values.
__device__ inline void latent_find_start(const LatentAttnShape& sh, const int32_t* seq_lens,
                                         const int32_t* cu, int nr, int kt, int lead,
                                         LatentStart* st, long long* sh_sum) {
  const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 31, warp = tid >> 5;
  const int per = (sh.N + nt - 1) / nt;
  const int n0 = min(tid * per, sh.N), n1 = min(n0 + per, sh.N);
  long long mine = 0;
  for (int n = n0; n < n1; ++n) mine += LatentSeq(sh, seq_lens, cu, n, nr, kt).total(sh, nr, kt, lead);
  long long run = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long up = __shfl_up_sync(0xffffffffu, run, o);
    if (lane >= o) run += up;
  }
  if (lane == 31) sh_sum[warp] = run;
  __syncthreads();
  if (warp == 0) {
    long long w = lane < nt / 32 ? sh_sum[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long up = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += up;
    }
    __syncwarp();
    sh_sum[lane + 1] = w;
    if (lane == 0) sh_sum[0] = 0;
  }
  __syncthreads();
  const long long W = sh_sum[32];
  const int G = (int)min((long long)gridDim.x, W);
  const int c = blockIdx.x;
  long long from = 0, to = 0;
  if (c < G) {
    from = W * c / G;
    to = W * (c + 1) / G;
  }
  long long at = sh_sum[warp] + run - mine;             // places before this thread's sequences
  if (tid == 0) {
    st->places = to - from;
    st->pos = from;
    st->W = W;
    st->G = G;
  }
  if (to > from && at <= from && from < at + mine) {
    for (int n = n0; n < n1; ++n) {
      const LatentSeq q(sh, seq_lens, cu, n, nr, kt);
      const long long t = q.total(sh, nr, kt, lead);
      if (from < at + t) {
        int lo = 0, hi = q.nb - 1;                       // the last block that starts at or before
        while (lo < hi) {
          const int mid = (lo + hi + 1) / 2;
          if (at + q.before(mid, sh, nr, kt, lead) <= from) lo = mid;
          else hi = mid - 1;
        }
        st->n = n;
        st->b = lo;
        st->at = (int)(from - at - q.before(lo, sh, nr, kt, lead));
        break;
      }
      at += t;
    }
  }
  __syncthreads();
}

// The pieces of a stretch, one after the other; every role of a CTA walks it for itself.
struct LatentPiece {
  int n;                            // sequence
  int t0, t1, tiles;                // tiles [t0, t1) of the block's `tiles`
  int len, start;                   // cached tokens; position of the sequence's first new token
  long long row0;                   // first row of the block in q (tokens * H + heads)
  int row_in_seq, rows;             // the same inside of the sequence; rows of the block
  long long end;                    // the block's last place in the line
};

struct LatentWalk {
  int n, b, at;
  long long left, pos;
  __device__ explicit LatentWalk(const LatentStart& s)
      : n(s.n), b(s.b), at(s.at), left(s.places), pos(s.pos) {}
  __device__ bool next(const LatentAttnShape& sh, const int32_t* seq_lens, const int32_t* cu,
                       int nr, int kt, int lead, LatentPiece* p) {
    while (left > 0 && n < sh.N) {
      const LatentSeq q(sh, seq_lens, cu, n, nr, kt);
      if (b >= q.nb) {
        ++n;
        b = 0;
        continue;
      }
      p->n = n;
      p->tiles = q.tiles(b, sh, nr, kt);
      const int took = (int)min((long long)(lead + p->tiles - at), left);
      p->t0 = max(at - lead, 0);
      p->t1 = at + took - lead;
      p->len = q.len;
      p->start = q.len - q.cnt;
      p->row_in_seq = b * nr;
      p->rows = (int)min((long long)nr, (long long)q.cnt * sh.H - (long long)b * nr);
      p->row0 = (long long)q.first * sh.H + (long long)b * nr;
      p->end = pos - at + lead + p->tiles - 1;
      left -= took;
      pos += took;
      at = 0;
      ++b;
      if (p->t1 > 0) return true;                        // else the stretch ends in the empty places
    }
    return false;
  }
};

// The CTA whose stretch holds position x of the line.
__device__ __forceinline__ int latent_cta_of(long long x, long long W, int G) {
  return (int)(((x + 1) * G - 1) / W);
}

}  // namespace kda
