// Latent attention over a paged cache on the CUDA cores (kda_latent_attn, fp32 or pages
// that the tensor-core kernel's tiles do not divide), and the join of partial results.
//
// Row r (new token i, head h) with query q_r attends to the first lim_r = len - L + i + 1
// cached rows c_j [rank + rope]:
//     s_rj = scale q_r . c_j,    p = softmax over j < lim_r,    out_r = sum_j p_rj c_j[0, rank)
// in one pass over the cache with the running maximum and sum of the softmax.  A row that
// sees nothing gives zeros and a log-sum of -inf.
//
// One CTA holds 16 rows; tiles of 32 cached rows come by cp.async into two buffers, the next
// one under the arithmetic of this one, and each is used for both products by all 16 rows.
// Scores: each of the eight warps takes an eighth of the columns of all 16 x 32, a thread
// four rows by four tokens (eight 16-byte reads of shared memory for 64 FMAs); the eight
// partial sums meet in shared memory.  Output: a thread holds eight rows by four columns in
// registers (three 16-byte reads for 32 FMAs); with a rank below 512 the threads that
// remain take other tokens of the tile, and the sums meet at the end of a block.  Bound by
// these reads, not by the cache's bytes.  (A form on the tensor cores would have to split each
// operand in three bf16 or TF32 terms to keep fp32's accuracy; it has not been built.)
// Where there are more rows and shared memory holds but one such CTA an SM, a CTA holds 32 rows
// and tiles of 16 tokens instead: half a warp a sixteenth of the columns, eight rows by four
// tokens a thread (12 reads for 128 FMAs), 16 rows by four columns of the output (five for 64).
#include <type_traits>

#include "latent_attn.cuh"
#include "sm100.cuh"

namespace kda {
namespace {

constexpr int kNT = 256;
constexpr int kLead = 1;                 // tiles that a block costs besides its own
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// Four neighbouring elements as fp32.
__device__ __forceinline__ float4 four(const float* x) { return *reinterpret_cast<const float4*>(x); }
__device__ __forceinline__ float4 four(const __nv_bfloat16* x) {
  const uint2 u = *reinterpret_cast<const uint2*>(x);
  return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u),
                     __uint_as_float(u.y << 16), __uint_as_float(u.y & 0xffff0000u));
}
// Shared memory: Q [16][LD], two tiles [32][LD] (LD = D + 16 bytes: rows shift by four banks),
// the warps' partial scores.
template <typename T> __host__ __device__ constexpr int simt_ld(int D) { return D + 16 / (int)sizeof(T); }
// Cached rows of a tile, and floats of a warp's partial scores' row (32 rows: padded for the banks).
__host__ __device__ constexpr int simt_tile(int rows) { return 512 / rows; }
__host__ __device__ constexpr int simt_red_ld(int rows) { return rows == 16 ? 32 : 20; }
// Floats of the partial scores, in whose place the token groups' sums meet in the end.
__host__ __device__ constexpr int simt_red(int rows, int split) {
  return rows == 16 ? 4096 : split > 1 ? 8192 : 8 * 32 * simt_red_ld(32);
}
int simt_split(int rank) { return rank == 128 ? 4 : rank == 256 ? 2 : 1; }
template <typename T> int simt_smem(int D, int rank, int rows) {
  return (rows + 2 * simt_tile(rows)) * simt_ld<T>(D) * (int)sizeof(T) +
         simt_red(rows, simt_split(rank)) * 4;
}

// kSplit: groups of threads that share a tile's tokens in the value product, at most
// 512 / rank (384: one, which leaves two warps without columns).
template <typename T, int kRows, int kSplit>
__global__ void __launch_bounds__(kNT, kRows == 16 ? 2 : 1)
kda_latent_simt_kernel(const T* __restrict__ q, const T* __restrict__ cache,
                       const int32_t* __restrict__ page_table,
                       const int32_t* __restrict__ seq_lens,
                       const int32_t* __restrict__ cu_seqlens, T* __restrict__ out,
                       float* __restrict__ lse, LatentAttnShape sh, LatentPartials pt) {
  using namespace sm100;
  constexpr int kTile = simt_tile(kRows), kRL = simt_red_ld(kRows);
  extern __shared__ float4 smem4[];
  const int D = sh.rank + sh.rope, LD = simt_ld<T>(D);
  T* const sq = reinterpret_cast<T*>(smem4);
  T* const sk = sq + kRows * LD;
  float* const sred = reinterpret_cast<float*>(sk + 2 * kTile * LD);   // [8][kRows][kRL]
  __shared__ __align__(16) float sp[kTile][kRows + 4];
  __shared__ __align__(16) float s_alpha[kRows];
  __shared__ float s_inv[kRows];
  __shared__ LatentStart st;
  __shared__ long long s_sum[33];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  latent_find_start(sh, seq_lens, cu_seqlens, kRows, kTile, kLead, &st, s_sum);
  if (tid == 0) pt.head[blockIdx.x] = make_int4(0, 0, 0, 0);

  constexpr int E = 16 / sizeof(T);
  constexpr int kRT = kNT / kRows, kTG = kTile / 4;         // threads of a row; groups of tokens
  const int r = tid / kRT, j0 = tid % kRT;                  // softmax: row r, tokens j0, j0 + kRT
  // scores: rows rg + 4 a, tokens tg + kTG b of 4 kTG lanes; those share an equal part of the columns
  constexpr int kA = kRows / 4, kSl = kNT / (4 * kTG);
  const int rg = lane / kTG % 4, tg = lane % kTG, sl = tid / (4 * kTG), DS = D / kSl;
  // output: rows hr .., columns d0 .. of tokens [kTile / kSplit * part, ..)
  constexpr int kH = kRows / 2;
  const int per = sh.rank / 2, part = tid / per, hr = kH * (tid & 1), d0 = (tid - part * per) / 2 * 4;
  const bool has = part < kSplit;
  LatentWalk walk(st);
  LatentPiece p;
  while (walk.next(sh, seq_lens, cu_seqlens, kRows, kTile, kLead, &p)) {
    // tile t into buffer b; zeros where there is no row
    auto fetch = [&](int t, int b) {
      constexpr int kT = kNT / kTile;                       // threads of a row
      const int row = tid / kT, pos = t * kTile + row;
      const T* src = cache;
      uint32_t bytes = 0;
      if (pos < p.len) {
        const int pg = pos / sh.page_size;
        const int page = __ldg(page_table + (long long)p.n * sh.max_pages + pg);
        if (page >= 0 && page < sh.num_pages) {
          src = cache + page * sh.page_stride + (pos - pg * sh.page_size) * sh.row_stride;
          bytes = 16;
        }
      }
      for (int e = tid % kT * E; e < D; e += kT * E)
        cp_async16(sk + (b * kTile + row) * LD + e, src + (bytes ? e : 0), bytes);
      cp_async_commit();
    };
    __syncthreads();                                        // the block before is done with
    {
      const int from = r < p.rows ? r : 0;
      for (int e = j0 * E; e < D; e += kRT * E)
        cp_async16(sq + r * LD + e, q + (p.row0 + from) * D + e, r < p.rows ? 16 : 0);
    }
    fetch(p.t0, 0);
    float acc[kH][4];
#pragma unroll
    for (int i = 0; i < kH; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) acc[i][k] = 0.f;
    float m = -INFINITY, l = 0.f;
    const int lim = min(p.start + (p.row_in_seq + r) / sh.H + 1, p.len);
    const int low = p.start + p.row_in_seq / sh.H + 1;      // the block's first row's limit
    for (int t = p.t0; t < p.t1; ++t) {
      const int k0 = t * kTile, b = (t - p.t0) & 1;
      if (t + 1 < p.t1) {
        fetch(t + 1, b ^ 1);
        cp_async_wait_group<1>();
      } else {
        cp_async_wait_group<0>();
      }
      __syncthreads();                                      // this tile is there
      {
        float x[kA][4] = {};
        const T* a = sq + rg * LD + sl * DS;
        const T* y = sk + (b * kTile + tg) * LD + sl * DS;
#pragma unroll 2
        for (int d = 0; d < DS; d += 4) {
          float4 av[kA], yv[4];
#pragma unroll
          for (int i = 0; i < kA; ++i) av[i] = four(a + 4 * i * LD + d);
#pragma unroll
          for (int j = 0; j < 4; ++j) yv[j] = four(y + kTG * j * LD + d);
#pragma unroll
          for (int i = 0; i < kA; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
              x[i][j] = fmaf(av[i].x, yv[j].x, fmaf(av[i].y, yv[j].y,
                        fmaf(av[i].z, yv[j].z, fmaf(av[i].w, yv[j].w, x[i][j]))));
        }
        // of 32 rows a warp has two parts of the columns: each half keeps half of the rows
        const bool up = kA == 8 && lane >= 16;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float v = x[i][j];
            if constexpr (kA == 8) {
              const float w = x[i + 4][j], give = up ? v : w;
              v = (up ? w : v) + __shfl_xor_sync(0xffffffffu, give, 16);
            }
            sred[(warp * kRows + rg + 4 * i + (up ? 16 : 0)) * kRL + tg + kTG * j] = v;
          }
      }
      __syncthreads();
      float s0 = 0.f, s1 = 0.f;
#pragma unroll
      for (int w = 0; w < 8; ++w) {
        s0 += sred[(w * kRows + r) * kRL + j0];
        s1 += sred[(w * kRows + r) * kRL + j0 + kRT];
      }
      const float c = sh.scale * kLog2e;
      s0 = k0 + j0 < lim ? s0 * c : -INFINITY;
      s1 = k0 + j0 + kRT < lim ? s1 * c : -INFINITY;
      float mx = fmaxf(s0, s1);
#pragma unroll
      for (int o = kRT / 2; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      const float mn = fmaxf(m, mx), ms = mn == -INFINITY ? 0.f : mn;
      const float p0 = exp2f(s0 - ms), p1 = exp2f(s1 - ms);   // a NaN score gives a NaN weight
      float ls = p0 + p1;
#pragma unroll
      for (int o = kRT / 2; o; o >>= 1) ls += __shfl_xor_sync(0xffffffffu, ls, o);
      const float al = exp2f(m - ms);
      l = l * al + ls;
      m = mn;
      sp[j0][r] = p0;
      sp[j0 + kRT][r] = p1;
      if (j0 == 0) s_alpha[r] = al;
      __syncthreads();
      const bool mixed = k0 + kTile > low;                  // some row does not see some token
#pragma unroll
      for (int i = 0; i < kH; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[i][k] *= s_alpha[hr + i];
      const T* v0 = sk + b * kTile * LD + d0;
      auto add_values = [&](auto all) {                     // all: every row sees every token
        constexpr int n = kTile / kSplit;
#pragma unroll 4
        for (int j = n * part; j < n * (part + 1); ++j) {
          float w[kH];
          const float4 v4 = four(v0 + j * LD);
          const float v[4] = {v4.x, v4.y, v4.z, v4.w};
#pragma unroll
          for (int i = 0; i < kH; i += 4)
            *reinterpret_cast<float4*>(w + i) = *reinterpret_cast<const float4*>(&sp[j][hr + i]);
#pragma unroll
          for (int i = 0; i < kH; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k)                     // a weight of zero takes nothing, not 0 * inf
              acc[i][k] = !decltype(all)::value && w[i] == 0.f ? acc[i][k]
                                                               : fmaf(w[i], v[k], acc[i][k]);
        }
      };
      if (has) {
        if (mixed) add_values(std::false_type());
        else add_values(std::true_type());
      }
      __syncthreads();                                      // the tile and its weights are used
    }
    // ---- the token groups' sums, the upper half of the groups to the lower each time
#pragma unroll
    for (int h = kSplit / 2; h > 0; h /= 2) {               // h rank kRows floats: all of sred at most
      float* const x = sred + (part % h * kH * per + tid % per) * 4;
      if (part >= h && part < 2 * h) {
#pragma unroll
        for (int i = 0; i < kH; ++i)
          *reinterpret_cast<float4*>(x + i * per * 4) =
              make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
      }
      __syncthreads();
      if (part < h) {
#pragma unroll
        for (int i = 0; i < kH; ++i) {
          const float4 y = *reinterpret_cast<const float4*>(x + i * per * 4);
          acc[i][0] += y.x;
          acc[i][1] += y.y;
          acc[i][2] += y.z;
          acc[i][3] += y.w;
        }
      }
      __syncthreads();
    }
    // ---- results: whole blocks to the output, shared ones to a partial slot
    const bool first = p.t0 == 0, last = p.t1 == p.tiles;
    const int slot = first && last ? -1 : 2 * (int)blockIdx.x + (first ? 1 : 0);
    if (j0 == 0) {
      s_inv[r] = l == 0.f ? 0.f : 1.0f / l;
      const float z = l == 0.f ? -INFINITY : (m == -INFINITY ? 0.f : m) * kLn2 + logf(l);
      if (slot >= 0) pt.lse[slot * kRows + r] = z;
      else if (lse && r < p.rows) lse[p.row0 + r] = z;
    }
    if (slot >= 0 && first && tid == 0)
      pt.head[blockIdx.x] =
          make_int4((int)p.row0, p.rows, latent_cta_of(p.end, st.W, st.G), 0);
    __syncthreads();
    if (part == 0) {
#pragma unroll
      for (int i = 0; i < kH; ++i) {
        if (hr + i >= p.rows) break;
        const float inv = s_inv[hr + i];
        const float o[4] = {acc[i][0] * inv, acc[i][1] * inv, acc[i][2] * inv, acc[i][3] * inv};
        if (slot >= 0) {
          *reinterpret_cast<float4*>(pt.o + ((long long)slot * kRows + hr + i) * sh.rank + d0) =
              make_float4(o[0], o[1], o[2], o[3]);
        } else {
          T* y = out + (p.row0 + hr + i) * sh.rank + d0;
#pragma unroll
          for (int k = 0; k < 4; ++k) y[k] = from_f32<T>(o[k]);
        }
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Join: row = sum_c e^(lse_c - M) o_c / sum_c e^(lse_c - M) over the CTAs that share the
// row's block, in their order.  Bound by latency (the partial results are in L2).  Up to 8 CTAs
// a row: 128 threads take it, all loads at once; up to 64: a warp takes 128 of its columns,
// eight loads at a time; more: a block does, each of its 16 warps a sixteenth of the CTAs.
constexpr int kJT = 512;
constexpr int kFew = 8, kSome = 64;

// Partial slot of the i-th CTA of a shared block that starts in CTA c0.
__device__ __forceinline__ long long join_slot(int c0, int i) {
  return i == 0 ? 2 * c0 + 1 : 2 * (c0 + i);
}
template <typename T>
__device__ __forceinline__ void join_store(T* o, const float4& a) {
  o[0] = from_f32<T>(a.x);
  o[1] = from_f32<T>(a.y);
  o[2] = from_f32<T>(a.z);
  o[3] = from_f32<T>(a.w);
}
__device__ __forceinline__ void join_add(float4& a, float w, const float4& v) {
  if (w == 0.f) return;                              // nothing seen: nothing taken
  a.x = fmaf(w, v.x, a.x);
  a.y = fmaf(w, v.y, a.y);
  a.z = fmaf(w, v.z, a.z);
  a.w = fmaf(w, v.w, a.w);
}

// Many items: block (c, y) takes rows y, y + gridDim.y, .. (or fours of rows) of the shared block
// that starts in CTA c, if one does.  Few (kList): the blocks that there are get listed and
// their rows spread over the grid.  kEither: so, if a block of many CTAs has rows for more than two
// rounds of its y.
enum { kEach = 0, kList = 1, kEither = 2 };
template <typename T>
__global__ void __launch_bounds__(kJT)
kda_latent_join_kernel(T* __restrict__ out, float* __restrict__ lse, LatentPartials pt, int G,
                       int nr, int rank, int form) {
  __shared__ float s_w[kLatentMaxCtas];
  __shared__ float4 s_part[kJT / 32][32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = tid >> 7, d4 = tid & 127;
  __shared__ int s_list[kLatentMaxCtas], s_n;
  __shared__ uint32_t s_mask[kLatentMaxCtas / 32];
  int c0 = blockIdx.x;
  const int parts = rank / 128;                        // units of a row
  sm100::grid_dep_wait();
  bool list = form == kList;
  if (form == kEither) {
    bool far = false;
    for (int c = tid; c < G; c += kJT) {
      const int4 h = pt.head[c];
      far = far || (h.z - c >= kSome && h.y * parts > 2 * (int)gridDim.y);
    }
    list = __syncthreads_or(far);
  }
  if (list) {                                          // in the CTAs' order: every block's is the same
    for (int c = tid; c - lane < G; c += kJT) {
      const uint32_t some = __ballot_sync(0xffffffffu, c < G && pt.head[c].y > 0);
      if (lane == 0) s_mask[c >> 5] = some;
    }
    __syncthreads();
    for (int c = tid; c - lane < G; c += kJT) {
      const uint32_t some = s_mask[c >> 5];
      int at = __popc(some & ((1u << lane) - 1));
      for (int w = 0; w < c >> 5; ++w) at += __popc(s_mask[w]);
      if (some >> lane & 1) s_list[at] = c;
      if (c == G - 1) s_n = at + (int)(some >> lane & 1);
    }
    __syncthreads();
  }
  int4 hd = list ? make_int4(0, 0, 0, 0) : pt.head[c0];
  int k = hd.z - c0 + 1;
  if (!list && k <= kFew) {
    for (int r = 4 * blockIdx.y + g; r < hd.y; r += 4 * gridDim.y) {
      float w[kFew];
      float4 v[kFew];
#pragma unroll
      for (int i = 0; i < kFew; ++i) {
        w[i] = -INFINITY;
        if (i < k) {
          const long long at = join_slot(c0, i) * nr + r;
          w[i] = pt.lse[at];
          if (d4 * 4 < rank) v[i] = *reinterpret_cast<const float4*>(pt.o + at * rank + d4 * 4);
        }
      }
      float M = -INFINITY, z = 0.f;
#pragma unroll
      for (int i = 0; i < kFew; ++i) M = fmaxf(M, w[i]);
      const float Ms = M == -INFINITY ? 0.f : M;
#pragma unroll
      for (int i = 0; i < kFew; ++i) z += expf(w[i] - Ms);   // a NaN makes all of it one
      const float inv = z == 0.f ? 0.f : 1.0f / z;
      if (d4 == 0 && lse) lse[hd.x + r] = z == 0.f ? -INFINITY : Ms + logf(z);
      if (d4 * 4 < rank) {
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int i = 0; i < kFew; ++i)
          if (i < k) join_add(a, expf(w[i] - Ms) * inv, v[i]);
        join_store(out + (long long)(hd.x + r) * rank + d4 * 4, a);
      }
    }
    return;
  }
  if (!list && k <= kSome) {
    constexpr int kWarps = kJT / 32;
    for (int u = blockIdx.y * kWarps + warp; u < hd.y * parts; u += gridDim.y * kWarps) {
      const int r = u / parts, d = 128 * (u - r * parts) + 4 * lane;
      float w[2];                                      // of CTAs lane, lane + 32
#pragma unroll
      for (int j = 0; j < 2; ++j)
        w[j] = lane + 32 * j < k ? pt.lse[join_slot(c0, lane + 32 * j) * nr + r] : -INFINITY;
      float M = fmaxf(w[0], w[1]);
#pragma unroll
      for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
      const float Ms = M == -INFINITY ? 0.f : M;
      w[0] = expf(w[0] - Ms);                          // a NaN makes all of it one
      w[1] = expf(w[1] - Ms);
      float z = w[0] + w[1];
#pragma unroll
      for (int o = 16; o; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
      const float inv = z == 0.f ? 0.f : 1.0f / z;
      if (d == 0 && lse) lse[hd.x + r] = z == 0.f ? -INFINITY : Ms + logf(z);
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll 8
        for (int i = 32 * j; i < min(k, 32 * j + 32); ++i)
          join_add(a, __shfl_sync(0xffffffffu, w[j], i & 31) * inv,
                   *reinterpret_cast<const float4*>(pt.o + (join_slot(c0, i) * nr + r) * rank + d));
      join_store(out + (long long)(hd.x + r) * rank + d, a);
    }
    return;
  }
  const int u0 = list ? blockIdx.y * gridDim.x + blockIdx.x : blockIdx.y;
  const int du = list ? gridDim.x * gridDim.y : gridDim.y;
  const int units = (list ? s_n * nr : hd.y) * parts;
  for (int u = u0; u < units; u += du) {
    int r = u / parts;
    const int d = 128 * (u - r * parts) + 4 * lane;
    if (list) {
      c0 = s_list[r / nr];
      r %= nr;
      hd = pt.head[c0];
      k = hd.z - c0 + 1;
      if (r >= hd.y) continue;
    }
    __syncthreads();                                   // s_w and s_part of the unit before are read
    for (int i = tid; i < k; i += kJT) s_w[i] = pt.lse[join_slot(c0, i) * nr + r];
    __syncthreads();
    float M = -INFINITY;
    for (int i = lane; i < k; i += 32) M = fmaxf(M, s_w[i]);
#pragma unroll
    for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    const float Ms = M == -INFINITY ? 0.f : M;
    float z = 0.f;
    for (int i = lane; i < k; i += 32) z += expf(s_w[i] - Ms);   // a NaN makes all of it one
#pragma unroll
    for (int o = 16; o; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
    const float inv = z == 0.f ? 0.f : 1.0f / z;
    if (tid == 0 && d == 0 && lse) lse[hd.x + r] = z == 0.f ? -INFINITY : Ms + logf(z);
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int i = warp; i < k; i += kJT / 32)
      join_add(a, expf(s_w[i] - Ms) * inv,
               *reinterpret_cast<const float4*>(pt.o + (join_slot(c0, i) * nr + r) * rank + d));
    s_part[warp][lane] = a;
    __syncthreads();
    if (warp == 0) {
#pragma unroll
      for (int i = 1; i < kJT / 32; ++i) {
        const float4 v = s_part[i][lane];
        a.x += v.x;
        a.y += v.y;
        a.z += v.z;
        a.w += v.w;
      }
      join_store(out + (long long)(hd.x + r) * rank + d, a);
    }
  }
}

template <typename T>
using SimtKernel = void (*)(const T*, const T*, const int32_t*, const int32_t*, const int32_t*, T*,
                            float*, LatentAttnShape, LatentPartials);
template <typename T> SimtKernel<T> simt_kernel(int rank, int rows) {
  if constexpr (sizeof(T) == 4)
    if (rows == 32)
      return rank == 256 ? kda_latent_simt_kernel<T, 32, 2> : kda_latent_simt_kernel<T, 32, 1>;
  switch (simt_split(rank)) {
    case 4: return kda_latent_simt_kernel<T, 16, 4>;
    case 2: return kda_latent_simt_kernel<T, 16, 2>;
    default: return kda_latent_simt_kernel<T, 16, 1>;
  }
}
template <typename T> bool simt_setup() {
  for (int rank = 128; rank <= 512; rank += 128)
    for (int rows = 16; rows <= 32; rows += 16)
      if (cudaFuncSetAttribute(simt_kernel<T>(rank, rows), cudaFuncAttributeMaxDynamicSharedMemorySize,
                               simt_smem<T>(512 + 64, 512, 16)) != cudaSuccess)
        return false;
  return true;
}

// Whether two CTAs of 16 rows fit an SM (4 KB: the variables and what the system keeps).
bool simt_two(int D, int rank, int dtype) {
  const int smem =
      dtype == KDA_BF16 ? simt_smem<__nv_bfloat16>(D, rank, 16) : simt_smem<float>(D, rank, 16);
  return 2 * (smem + 4096) <= 228 * 1024;
}

// Rows of a block: 32 where two CTAs of 16 do not fit an SM (fp32 from 320 columns on) and few of
// the rows would be empty (2 x 200 tokens of 12 heads behind 3000, rank 512: 655 us against 814;
// rank 256 122 against 126).  Where two fit they are faster (4 x 16 tokens of 96 heads, bf16,
// 1315 against 1364; rank 128 141 against 148).  Packed: of a sequence's rows on average.
int simt_rows(int N, int L, int T, int H, int D, int rank, int dtype) {
  const long long rows = L > 0 ? (long long)L * H : (((long long)T + N - 1) / N) * H;
  return !simt_two(D, rank, dtype) && (rows > 96 || (rows + 15) / 16 % 2 == 0) ? 32 : 16;
}

// CTAs that are resident at once: more would go in two rounds, each with its start and results
// (fp32, rank 512, 12 heads, up to 4000 tokens: 4 sequences 28.5 us against 38.2, 8 44.2 against
// 54.5).  One CTA of 512 threads where two of 256 do not fit is slower (32 sequences of up to 8000
// tokens 259 us against 250): what bounds it is shared memory, not the warps there are.
int simt_ctas(int sms, int D, int rank, int dtype) {
  const int n = simt_two(D, rank, dtype) ? 2 * sms : sms;
  return n < kLatentMaxCtas ? n : kLatentMaxCtas;
}

template <typename T>
cudaError_t run_simt(const void* q, const void* cache, const int32_t* page_table,
                     const int32_t* seq_lens, const int32_t* cu, void* out, float* lse,
                     const LatentAttnShape& sh, int rows, int G, const LatentPartials& pt,
                     cudaStream_t stream) {
  const int smem = simt_smem<T>(sh.rank + sh.rope, sh.rank, rows);
  KDA_TIMED(KDA_KERNEL_LATENT_ATTN, stream,
            simt_kernel<T>(sh.rank, rows)<<<G, kNT, smem, stream>>>(
                static_cast<const T*>(q), static_cast<const T*>(cache), page_table, seq_lens, cu,
                static_cast<T*>(out), lse, sh, pt));
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  note_launches(1);
  return launch_latent_join(out, lse, pt, G, rows, sh, sizeof(T) == 2 ? KDA_BF16 : KDA_F32, stream);
}

}  // namespace

// Few blocks of rows, each over more than 16 CTAs, are listed and spread over the grid, two rounds at
// most of 2 us (8 sequences of 16 heads, rank 128: 15.7 us a call against 17.7); a warp for each 128
// columns of a row where some CTAs share it (16 sequences of 12 heads: 27.0 against 30.8 listed); else
// blocks of 8 rows, of which many find nothing to do.  A packed call's blocks are as many as its rows
// fill, or as its sequences with tokens.  Where one count is few and the other not, the kernel looks
// (on the device, by the first count alone 100 sequences of one head behind 500 tokens took 53 us,
// by the second 22, so 23; two of eight tokens behind 30000 among 62 empty slots 23, 57 and 24).
cudaError_t launch_latent_join(void* out, float* lse, const LatentPartials& pt, int G, int nr,
                               const LatentAttnShape& sh, int dtype, cudaStream_t stream) {
  const int rank = sh.rank, units = nr * (rank / 128);
  const bool packed = sh.L == 0;
  const long long tokens = packed ? sh.T : sh.L;             // uniform: of a sequence
  const long long full = (tokens * sh.H + nr - 1) / nr, each = tokens * ((sh.H + nr - 1) / nr);
  const long long items = packed ? full : sh.N * full;       // packed: at least
  const long long own = tokens * sh.H / nr + (sh.N < tokens ? sh.N : tokens);
  const long long at_most = !packed ? items : own < each ? own : each;
  const long long work = packed ? tokens * sh.H * (rank / 128) : items * units, most = 4LL * G;
  auto few = [&](long long n) { return work <= 8LL * G && n * 16 < G; };
  const int form = !few(items) ? kEach : few(at_most) ? kList : kEither;
  const int y = at_most * kFew <= 2LL * G ? (units + 15) / 16 : nr <= 32 ? 4 : (nr + 7) / 8;
  const dim3 grid = form == kList ? dim3((unsigned)(at_most * units < most ? at_most * units : most)) : dim3(G, y);
  cudaError_t e = cudaSuccess;
  if (dtype == KDA_BF16)
    KDA_TIMED(KDA_KERNEL_LATENT_ATTN, stream,
              e = launch_after(kda_latent_join_kernel<__nv_bfloat16>, grid, dim3(kJT), 0, stream,
                               static_cast<__nv_bfloat16*>(out), lse, pt, G, nr, rank, form));
  else
    KDA_TIMED(KDA_KERNEL_LATENT_ATTN, stream,
              e = launch_after(kda_latent_join_kernel<float>, grid, dim3(kJT), 0, stream,
                               static_cast<float*>(out), lse, pt, G, nr, rank, form));
  note_launches(1);
  return e;
}

size_t latent_attn_scratch_bytes(int N, int L, int T, int H, int rank, int rope, int page_size,
                                 int dtype, int sms) {
  if (latent_tc_supported(dtype, page_size))
    return latent_tc_scratch_bytes(N, L, T, H, rank, sms);
  return latent_scratch_bytes(simt_ctas(sms, rank + rope, rank, dtype),
                              simt_rows(N, L, T, H, rank + rope, rank, dtype), rank);
}

cudaError_t launch_latent_attn(const void* q, const void* cache, const int32_t* page_table,
                               const int32_t* seq_lens, const int32_t* cu_seqlens, void* out,
                               float* lse, const LatentAttnShape& sh, int dtype,
                               cudaStream_t stream, const Workspace* ws, uint32_t polls) {
  int sms = 0;
  cudaMemPool_t pool = nullptr;
  if (!device_ctx(&sms, ws ? nullptr : &pool)) return cudaErrorInvalidDevice;
  if (!once_per_device(kOnceLatentSimt,
                       []() { return simt_setup<float>() && simt_setup<__nv_bfloat16>(); }))
    return cudaErrorInvalidDevice;
  const size_t bytes =
      latent_attn_scratch_bytes(sh.N, sh.L, sh.T, sh.H, sh.rank, sh.rope, sh.page_size, dtype,
                                sms);
  void* buf = ws ? ws->ptr : nullptr;
  cudaError_t e;
  if (!ws) {
    if (!pool) return cudaErrorMemoryAllocation;
    e = cudaMallocFromPoolAsync(&buf, bytes, pool, stream);
    if (e != cudaSuccess) return e;
  }
  const int D = sh.rank + sh.rope, rows = simt_rows(sh.N, sh.L, sh.T, sh.H, D, sh.rank, dtype);
  const int G = simt_ctas(sms, D, sh.rank, dtype);
  const LatentPartials pt = latent_partials(buf, G, rows);
  if (latent_tc_supported(dtype, sh.page_size))
    e = launch_latent_tc(q, cache, page_table, seq_lens, cu_seqlens, out, lse, sh, sms, buf, stream,
                         polls);
  else
    e = dtype == KDA_BF16 ? run_simt<__nv_bfloat16>(q, cache, page_table, seq_lens, cu_seqlens, out,
                                                  lse, sh, rows, G, pt, stream)
                        : run_simt<float>(q, cache, page_table, seq_lens, cu_seqlens, out, lse, sh,
                                          rows, G, pt, stream);
  if (!ws) {
    const cudaError_t f = cudaFreeAsync(buf, stream);
    if (e == cudaSuccess) e = f;
  }
  return e;
}

}  // namespace kda
