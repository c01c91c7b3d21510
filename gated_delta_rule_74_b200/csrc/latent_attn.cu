// Latent attention over a paged cache on the CUDA cores (kda_latent_attn, fp32 or pages
// that the tensor-core kernel's tiles do not divide), and the join of partial results.
//
// Row r (new token i, head h) with query q_r attends to the first lim_r = len - L + i + 1
// cached rows c_j [rank + rope]:
//     s_rj = scale q_r . c_j,    p = softmax over j < lim_r,    out_r = sum_j p_rj c_j[0, rank)
// in one pass over the cache with the running maximum and sum of the softmax.  A row that
// sees nothing gives zeros and a log-sum of -inf.
//
// One CTA holds 16 rows; a tile of 32 cached rows is brought to shared memory as fp32 once
// and used for both products by all 16.  Scores: thread (r, j) takes row r against tokens
// j and j + 16.  Output: thread d holds columns d and d + 256 of all 16 rows in registers.
// Bound by shared-memory reads (each FMA's operands come from there), not by the cache's
// bytes; fp32 has no tensor-core form of fp32 accuracy.
#include "latent_attn.cuh"
#include "sm100.cuh"

namespace kda {
namespace {

constexpr int kNT = 256;
constexpr int kRows = 16;                // rows of a block
constexpr int kTile = 32;                // cached rows of a tile
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// One piece's results, straight to the output or to partial slot `slot` (>= 0).
template <typename T>
__device__ __forceinline__ void put(T* out, float* lse, const LatentPartials& pt, int slot,
                                    int rank, long long row, int r, int nr, int d, float v) {
  if (slot < 0) out[row * rank + d] = from_f32<T>(v);
  else pt.o[((long long)slot * nr + r) * rank + d] = v;
}

template <typename T>
__global__ void __launch_bounds__(kNT)
kda_latent_simt_kernel(const T* __restrict__ q, const T* __restrict__ cache,
                       const int32_t* __restrict__ page_table,
                       const int32_t* __restrict__ seq_lens,
                       const int32_t* __restrict__ cu_seqlens, T* __restrict__ out,
                       float* __restrict__ lse, LatentAttnShape sh, LatentPartials pt) {
  extern __shared__ float4 smem4[];
  const int D = sh.rank + sh.rope, LD = D + 4;
  float* const sq = reinterpret_cast<float*>(smem4);       // [16][LD]
  float* const sk = sq + kRows * LD;                       // [32][LD]
  __shared__ float sp[kTile][kRows];
  __shared__ float s_alpha[kRows], s_l[kRows];
  __shared__ LatentStart st;
  __shared__ long long s_sum[33];
  const int tid = threadIdx.x;
  latent_find_start(sh, seq_lens, cu_seqlens, kRows, kTile, &st, s_sum);
  if (tid == 0) pt.head[blockIdx.x] = make_int4(0, 0, 0, 0);

  const int r = tid >> 4, j0 = tid & 15;
  constexpr int E = 16 / sizeof(T);
  LatentWalk walk(st);
  LatentPiece p;
  while (walk.next(sh, seq_lens, cu_seqlens, kRows, kTile, &p)) {
    __syncthreads();
    for (int i = tid; i < kRows * (D / E); i += kNT) {
      const int row = i / (D / E), e = (i - row * (D / E)) * E;
      uint4 u = make_uint4(0, 0, 0, 0);
      if (row < p.rows) u = __ldg(reinterpret_cast<const uint4*>(q + (p.row0 + row) * D + e));
      const T* x = reinterpret_cast<const T*>(&u);
#pragma unroll
      for (int k = 0; k < E; ++k) sq[row * LD + e + k] = to_f32(x[k]);
    }
    float acc[2][kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) acc[0][i] = acc[1][i] = 0.f;
    float m = -INFINITY, l = 0.f;
    const int lim = min(p.start + (p.row_in_seq + r) / sh.H + 1, p.len);
    const int low = p.start + p.row_in_seq / sh.H + 1;      // the block's first row's limit
    for (int t = p.t0; t < p.t1; ++t) {
      const int k0 = t * kTile;
      __syncthreads();                                      // the tile before is consumed
      for (int i = tid; i < kTile * (D / E); i += kNT) {
        const int row = i / (D / E), e = (i - row * (D / E)) * E;
        const int pos = k0 + row;
        uint4 u = make_uint4(0, 0, 0, 0);
        if (pos < p.len) {
          const int page = __ldg(page_table + (long long)p.n * sh.max_pages + pos / sh.page_size);
          if (page >= 0 && page < sh.num_pages)
            u = __ldg(reinterpret_cast<const uint4*>(
                cache + page * sh.page_stride + (pos % sh.page_size) * sh.row_stride + e));
        }
        const T* x = reinterpret_cast<const T*>(&u);
#pragma unroll
        for (int k = 0; k < E; ++k) sk[row * LD + e + k] = to_f32(x[k]);
      }
      __syncthreads();
      float s0 = 0.f, s1 = 0.f;
      {
        const float4* a = reinterpret_cast<const float4*>(sq + r * LD);
        const float4* b0 = reinterpret_cast<const float4*>(sk + j0 * LD);
        const float4* b1 = reinterpret_cast<const float4*>(sk + (j0 + 16) * LD);
#pragma unroll 4
        for (int i = 0; i < D / 4; ++i) {
          const float4 x = a[i], y = b0[i], z = b1[i];
          s0 = fmaf(x.x, y.x, fmaf(x.y, y.y, fmaf(x.z, y.z, fmaf(x.w, y.w, s0))));
          s1 = fmaf(x.x, z.x, fmaf(x.y, z.y, fmaf(x.z, z.z, fmaf(x.w, z.w, s1))));
        }
      }
      const float c = sh.scale * kLog2e;
      s0 = k0 + j0 < lim ? s0 * c : -INFINITY;
      s1 = k0 + j0 + 16 < lim ? s1 * c : -INFINITY;
      float mx = fmaxf(s0, s1);
      bool nan = s0 != s0 || s1 != s1;                      // fmaxf drops a NaN: kept apart
#pragma unroll
      for (int o = 8; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o, 16));
      const float mn = fmaxf(m, mx), ms = mn == -INFINITY ? 0.f : mn;
      const float p0 = nan ? s0 + s1 : exp2f(s0 - ms), p1 = exp2f(s1 - ms);
      float ls = p0 + p1;
#pragma unroll
      for (int o = 8; o; o >>= 1) ls += __shfl_xor_sync(0xffffffffu, ls, o, 16);
      const float al = exp2f(m - ms);
      l = l * al + ls;
      m = mn;
      sp[j0][r] = p0;
      sp[j0 + 16][r] = p1;
      if (j0 == 0) s_alpha[r] = al;
      __syncthreads();
      const bool mixed = k0 + kTile > low;                  // some row does not see some token
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        acc[0][i] *= s_alpha[i];
        acc[1][i] *= s_alpha[i];
      }
#pragma unroll 2
      for (int j = 0; j < kTile; ++j) {
        float w[kRows];
#pragma unroll
        for (int i = 0; i < kRows; i += 4)
          *reinterpret_cast<float4*>(w + i) = *reinterpret_cast<const float4*>(&sp[j][i]);
        const float v0 = tid < sh.rank ? sk[j * LD + tid] : 0.f;
        const float v1 = tid + kNT < sh.rank ? sk[j * LD + tid + kNT] : 0.f;
        if (mixed) {                                        // a weight of zero takes nothing, not 0 * inf
#pragma unroll
          for (int i = 0; i < kRows; ++i) {
            acc[0][i] = w[i] == 0.f ? acc[0][i] : fmaf(w[i], v0, acc[0][i]);
            acc[1][i] = w[i] == 0.f ? acc[1][i] : fmaf(w[i], v1, acc[1][i]);
          }
        } else {
#pragma unroll
          for (int i = 0; i < kRows; ++i) {
            acc[0][i] = fmaf(w[i], v0, acc[0][i]);
            acc[1][i] = fmaf(w[i], v1, acc[1][i]);
          }
        }
      }
    }
    // ---- results: whole blocks to the output, shared ones to a partial slot
    const bool first = p.t0 == 0, last = p.t1 == p.tiles;
    const int slot = first && last ? -1 : 2 * (int)blockIdx.x + (first ? 1 : 0);
    if (j0 == 0) {
      s_l[r] = l;
      const float z = l == 0.f ? -INFINITY : (m == -INFINITY ? 0.f : m) * kLn2 + logf(l);
      if (slot >= 0) pt.lse[slot * kRows + r] = z;
      else if (lse && r < p.rows) lse[p.row0 + r] = z;
    }
    if (slot >= 0 && first && tid == 0)
      pt.head[blockIdx.x] =
          make_int4((int)p.row0, p.rows, latent_cta_of(p.pos + p.tiles - 1, st.W, st.G), 0);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      if (i >= p.rows) break;
      const float inv = s_l[i] == 0.f ? 0.f : 1.0f / s_l[i];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int d = tid + h * kNT;
        if (d < sh.rank)
          put(out, lse, pt, slot, sh.rank, p.row0 + i, i, kRows, d, acc[h][i] * inv);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Join: row = sum_c e^(lse_c - M) o_c / sum_c e^(lse_c - M) over the CTAs that share the
// row's block, in their order.  Bound by latency (the partial results are in L2): a block's
// four groups of 128 threads take a row each while few CTAs share it, all loads at once,
// and a quarter of the CTAs each where many do.
constexpr int kJT = 512;
constexpr int kFew = 8;

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

template <typename T>
__global__ void __launch_bounds__(kJT)
kda_latent_join_kernel(T* __restrict__ out, float* __restrict__ lse, LatentPartials pt, int G,
                       int nr, int rank) {
  __shared__ int s_off[kLatentMaxCtas + 1];
  __shared__ float s_w[kLatentMaxCtas];
  __shared__ float4 s_part[3][128];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = tid >> 7, d4 = tid & 127;
  sm100::grid_dep_wait();
  // units (rows, or four rows) of the CTAs' shared blocks before each CTA
  if (warp == 0) {
    int run = 0;
    for (int c0 = 0; c0 < G; c0 += 32) {
      const int c = c0 + lane;
      int v = 0;
      if (c < G) {
        const int4 hd = pt.head[c];
        v = hd.z - c + 1 <= kFew ? (hd.y + 3) / 4 : hd.y;
      }
      int s = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += up;
      }
      if (c < G) s_off[c] = run + s - v;
      run += __shfl_sync(0xffffffffu, s, 31);
    }
    if (lane == 0) s_off[G] = run;
  }
  __syncthreads();
  const int units = s_off[G];
  for (int u = blockIdx.x; u < units; u += gridDim.x) {
    int lo = 0, hi = G - 1;                            // the last CTA that starts at or before u
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (s_off[mid] <= u) lo = mid;
      else hi = mid - 1;
    }
    const int c0 = lo;
    const int4 hd = pt.head[c0];
    const int k = hd.z - c0 + 1;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    if (k <= kFew) {
      const int r = 4 * (u - s_off[c0]) + g;
      if (r >= hd.y) continue;
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
#pragma unroll
        for (int i = 0; i < kFew; ++i)
          if (i < k) join_add(a, expf(w[i] - Ms) * inv, v[i]);
        join_store(out + (long long)(hd.x + r) * rank + d4 * 4, a);
      }
      continue;
    }
    const int r = u - s_off[c0];
    __syncthreads();                                   // s_w and s_part of the row before are read
    for (int i = tid; i < k; i += kJT) s_w[i] = pt.lse[join_slot(c0, i) * nr + r];
    __syncthreads();
    float M = -INFINITY;
    for (int i = lane; i < k; i += 32) M = fmaxf(M, s_w[i]);
#pragma unroll
    for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    const float Ms = M == -INFINITY ? 0.f : M;
    float z = 0.f;
    for (int i = lane; i < k; i += 32) z += expf(s_w[i] - Ms);
#pragma unroll
    for (int o = 16; o; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
    const float inv = z == 0.f ? 0.f : 1.0f / z;
    if (tid == 0 && lse) lse[hd.x + r] = z == 0.f ? -INFINITY : Ms + logf(z);
    const int i0 = k * g / 4, i1 = k * (g + 1) / 4;
    if (d4 * 4 < rank) {
#pragma unroll 8
      for (int i = i0; i < i1; ++i)
        join_add(a, expf(s_w[i] - Ms) * inv,
                 *reinterpret_cast<const float4*>(pt.o + (join_slot(c0, i) * nr + r) * rank + d4 * 4));
    }
    if (g > 0) s_part[g - 1][d4] = a;
    __syncthreads();
    if (g == 0 && d4 * 4 < rank) {
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        const float4 v = s_part[i][d4];
        a.x += v.x;
        a.y += v.y;
        a.z += v.z;
        a.w += v.w;
      }
      join_store(out + (long long)(hd.x + r) * rank + d4 * 4, a);
    }
  }
}

int simt_smem(int D) { return (kRows + kTile) * (D + 4) * 4; }

template <typename T>
cudaError_t run_simt(const void* q, const void* cache, const int32_t* page_table,
                     const int32_t* seq_lens, const int32_t* cu, void* out, float* lse,
                     const LatentAttnShape& sh, int G, const LatentPartials& pt,
                     cudaStream_t stream) {
  KDA_TIMED(KDA_KERNEL_LATENT_ATTN, stream,
            kda_latent_simt_kernel<T><<<G, kNT, simt_smem(sh.rank + sh.rope), stream>>>(
                static_cast<const T*>(q), static_cast<const T*>(cache), page_table, seq_lens, cu,
                static_cast<T*>(out), lse, sh, pt));
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  note_launches(1);
  return launch_latent_join(out, lse, pt, G, kRows, sh.rank,
                            sizeof(T) == 2 ? KDA_BF16 : KDA_F32, stream);
}

int simt_ctas(int sms) { return 2 * sms < kLatentMaxCtas ? 2 * sms : kLatentMaxCtas; }

}  // namespace

// Four join blocks an SM are resident; more would only wait.
cudaError_t launch_latent_join(void* out, float* lse, const LatentPartials& pt, int G, int nr,
                               int rank, int dtype, cudaStream_t stream) {
  int sms = 0;
  if (!device_ctx(&sms, nullptr)) return cudaErrorInvalidDevice;
  cudaError_t e = cudaSuccess;
  if (dtype == KDA_BF16)
    KDA_TIMED(KDA_KERNEL_LATENT_ATTN, stream,
              e = launch_after(kda_latent_join_kernel<__nv_bfloat16>, dim3(4 * sms), dim3(kJT), 0,
                               stream, static_cast<__nv_bfloat16*>(out), lse, pt, G, nr, rank));
  else
    KDA_TIMED(KDA_KERNEL_LATENT_ATTN, stream,
              e = launch_after(kda_latent_join_kernel<float>, dim3(4 * sms), dim3(kJT), 0, stream,
                               static_cast<float*>(out), lse, pt, G, nr, rank));
  note_launches(1);
  return e;
}

size_t latent_attn_scratch_bytes(int N, int L, int T, int H, int rank, int page_size, int dtype,
                                 int sms) {
  if (latent_tc_supported(dtype, page_size))
    return latent_tc_scratch_bytes(N, L, T, H, rank, sms);
  return latent_scratch_bytes(simt_ctas(sms), kRows, rank);
}

cudaError_t launch_latent_attn(const void* q, const void* cache, const int32_t* page_table,
                               const int32_t* seq_lens, const int32_t* cu_seqlens, void* out,
                               float* lse, const LatentAttnShape& sh, int dtype,
                               cudaStream_t stream, const Workspace* ws) {
  int sms = 0;
  cudaMemPool_t pool = nullptr;
  if (!device_ctx(&sms, ws ? nullptr : &pool)) return cudaErrorInvalidDevice;
  if (!once_per_device(kOnceLatentSimt, []() {
        const int most = simt_smem(576);
        return cudaFuncSetAttribute(kda_latent_simt_kernel<float>,
                                    cudaFuncAttributeMaxDynamicSharedMemorySize, most) ==
                   cudaSuccess &&
               cudaFuncSetAttribute(kda_latent_simt_kernel<__nv_bfloat16>,
                                    cudaFuncAttributeMaxDynamicSharedMemorySize, most) ==
                   cudaSuccess;
      }))
    return cudaErrorInvalidDevice;
  const size_t bytes =
      latent_attn_scratch_bytes(sh.N, sh.L, sh.T, sh.H, sh.rank, sh.page_size, dtype, sms);
  void* buf = ws ? ws->ptr : nullptr;
  cudaError_t e;
  if (!ws) {
    if (!pool) return cudaErrorMemoryAllocation;
    e = cudaMallocFromPoolAsync(&buf, bytes, pool, stream);
    if (e != cudaSuccess) return e;
  }
  const int G = simt_ctas(sms);
  const LatentPartials pt = latent_partials(buf, G, kRows);
  if (latent_tc_supported(dtype, sh.page_size))
    e = launch_latent_tc(q, cache, page_table, seq_lens, cu_seqlens, out, lse, sh, sms, buf, stream);
  else
    e = dtype == KDA_BF16 ? run_simt<__nv_bfloat16>(q, cache, page_table, seq_lens, cu_seqlens, out,
                                                  lse, sh, G, pt, stream)
                        : run_simt<float>(q, cache, page_table, seq_lens, cu_seqlens, out, lse, sh,
                                          G, pt, stream);
  if (!ws) {
    const cudaError_t f = cudaFreeAsync(buf, stream);
    if (e == cudaSuccess) e = f;
  }
  return e;
}

}  // namespace kda
