// Appending latent rows to a paged cache (kda_latent_append).
//
// For new token i of a sequence with `len` cached tokens (the L new ones included),
// at position p = len - L + i:
//     y[0, rank)       = x[0, rank) * rsqrt(mean(x[0, rank)^2) + eps) * w      (w given)
//     y[rank, rank+64) = R(p) x[rank, rank+64)                             (inv_freq given)
//     cache[page_table[seq][p / page_size]][p % page_size] = y
// and the query heads' rotated parts q_pe_out = R(p) q_pe.  R(p) turns pair f by the
// angle p * inv_freq[f]; the product is taken and reduced to a fraction of a turn in 64
// bits (a far position has lost its angle in 32), the sine and cosine of the fraction in
// 32.  Sums and products are fp32, rounded once to the cache's type.
//
// Bound by memory: every byte is read and written once.  One warp per (token, part):
// part 0 is the token's own row (16 elements a lane, the norm a warp reduction), part
// j > 0 the 16 query heads [16 (j - 1), 16 j).  Two heads a step, 16 lanes a head, each
// lane two neighbouring pairs, so a warp reads whole 128-byte (bf16) runs; all of a
// part's loads are issued before the first is used.  A part recomputes its token's
// position and angles: a few dozen instructions against a wait for another warp.
#include "kda_common.cuh"
#include "latent.cuh"

namespace kda {
namespace {

constexpr int kRope = 64;               // rotated elements a row (or none)
constexpr int kHeadsPerPart = 16;
constexpr int kWarps = 4;

struct Turn2 { float c0, s0, c1, s1; bool on; };   // two frequencies' cosines and sines

template <typename T> struct Vec2;
template <> struct Vec2<float> { using type = float2; };
template <> struct Vec2<__nv_bfloat16> { using type = __nv_bfloat162; };

__device__ __forceinline__ float2 up2(float2 v) { return v; }
__device__ __forceinline__ float2 up2(__nv_bfloat162 v) { return __bfloat1622float2(v); }
template <typename T> __device__ __forceinline__ typename Vec2<T>::type down2(float x, float y);
template <> __device__ __forceinline__ float2 down2<float>(float x, float y) {
  return make_float2(x, y);
}
template <> __device__ __forceinline__ __nv_bfloat162 down2<__nv_bfloat16>(float x, float y) {
  return __floats2bfloat162_rn(x, y);
}

// The elements of pairs f, f + 1 (f = 2 j): (4j .. 4j+3) interleaved, else (2j, 2j+1) and
// (32 + 2j, 32 + 2j + 1).
template <typename T> struct Pairs { typename Vec2<T>::type u, w; };

template <typename T>
__device__ __forceinline__ Pairs<T> load_pairs(const T* x, int j, bool inter) {
  using V = typename Vec2<T>::type;
  return {*reinterpret_cast<const V*>(x + (inter ? 4 * j : 2 * j)),
          *reinterpret_cast<const V*>(x + (inter ? 4 * j + 2 : kRope / 2 + 2 * j))};
}
template <typename T>
__device__ __forceinline__ void store_turned(T* y, int j, bool inter, Pairs<T> p, const Turn2& t) {
  using V = typename Vec2<T>::type;
  if (t.on) {                                      // else a copy, bit for bit
    const float2 u = up2(p.u), w = up2(p.w);
    const float x0 = u.x, x1 = inter ? w.x : u.y, z0 = inter ? u.y : w.x, z1 = w.y;
    const float a0 = x0 * t.c0 - z0 * t.s0, b0 = x0 * t.s0 + z0 * t.c0;
    const float a1 = x1 * t.c1 - z1 * t.s1, b1 = x1 * t.s1 + z1 * t.c1;
    p.u = inter ? down2<T>(a0, b0) : down2<T>(a0, a1);
    p.w = inter ? down2<T>(a1, b1) : down2<T>(b0, b1);
  }
  *reinterpret_cast<V*>(y + (inter ? 4 * j : 2 * j)) = p.u;
  *reinterpret_cast<V*>(y + (inter ? 4 * j + 2 : kRope / 2 + 2 * j)) = p.w;
}

// cos and sin of pos * freq
__device__ __forceinline__ void turn(int pos, float freq, float* c, float* s) {
  double t = (double)pos * (double)freq * 0.15915494309189533577;   // turns: 1 / (2 pi)
  t -= rint(t);
  sincospif(2.0f * (float)t, s, c);
}

template <typename T>
__global__ void __launch_bounds__(32 * kWarps)
kda_latent_append_kernel(const T* __restrict__ kv, const float* __restrict__ w,
                         const float* __restrict__ inv_freq, const T* __restrict__ q_pe,
                         T* __restrict__ q_out, T* __restrict__ cache,
                         const int32_t* __restrict__ page_table,
                         const int32_t* __restrict__ seq_lens,
                         const int32_t* __restrict__ cu_seqlens, LatentAppendShape sh) {
  const int lane = threadIdx.x & 31;
  const long long unit = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const long long tok = unit / sh.parts;
  const int part = (int)(unit - tok * sh.parts);
  if (tok >= sh.tokens) return;

  // the token's own loads do not wait for its position
  constexpr int E = 16 / sizeof(T);                   // elements of a 16-byte load
  constexpr int NV = 16 / E;                          // loads of a lane: 16 elements at most
  uint4 xv[NV];
  if (part == 0) {
    const T* x = kv + tok * sh.kv_stride;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = (i * 32 + lane) * E;
      xv[i] = e < sh.rank ? __ldg(reinterpret_cast<const uint4*>(x + e)) : make_uint4(0, 0, 0, 0);
    }
  }
  int seq, i0, cnt;
  if (!token_sequence(tok, sh.N, sh.L, cu_seqlens, (int)sh.tokens, lane, &seq, &i0, &cnt)) return;
  const int pos = seq_lens[seq] - cnt + (int)(tok - i0);

  const int j = lane & 15;                            // pairs 2j, 2j + 1
  Turn2 t = {1.f, 0.f, 1.f, 0.f, false};
  if (sh.rope && inv_freq) {
    const float2 f = __ldg(reinterpret_cast<const float2*>(inv_freq) + j);
    turn(pos, f.x, &t.c0, &t.s0);
    turn(pos, f.y, &t.c1, &t.s1);
    t.on = true;
  }

  if (part > 0) {
    const int h0 = (part - 1) * kHeadsPerPart + (lane >> 4);
    Pairs<T> p[kHeadsPerPart / 2];
#pragma unroll
    for (int i = 0; i < kHeadsPerPart / 2; ++i)
      if (h0 + 2 * i < sh.H)
        p[i] = load_pairs(q_pe + tok * sh.q_tok + (h0 + 2 * i) * sh.q_head, j, sh.interleaved);
#pragma unroll
    for (int i = 0; i < kHeadsPerPart / 2; ++i)
      if (h0 + 2 * i < sh.H)
        store_turned(q_out + tok * sh.qo_tok + (h0 + 2 * i) * sh.qo_head, j, sh.interleaved, p[i],
                      t);
    return;
  }

  // the slot: outside the table or the cache, the row is not written
  if (pos < 0 || pos / sh.page_size >= sh.max_pages) return;
  const int page = __ldg(page_table + (long long)seq * sh.max_pages + pos / sh.page_size);
  if (page < 0 || page >= sh.num_pages) return;
  T* y = cache + page * sh.page_stride + (pos % sh.page_size) * sh.row_stride;

  if (w) {
    float x[16], ss = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const T* xe = reinterpret_cast<const T*>(&xv[i]);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        x[i * E + e] = to_f32(xe[e]);
        ss = fmaf(x[i * E + e], x[i * E + e], ss);
      }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const float r = rsqrtf(ss / (float)sh.rank + sh.eps);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e0 = (i * 32 + lane) * E;
      if (e0 >= sh.rank) continue;
      T* xe = reinterpret_cast<T*>(&xv[i]);
#pragma unroll
      for (int e4 = 0; e4 < E; e4 += 4) {
        const float4 g = __ldg(reinterpret_cast<const float4*>(w + e0 + e4));
        xe[e4] = from_f32<T>(x[i * E + e4] * r * g.x);
        xe[e4 + 1] = from_f32<T>(x[i * E + e4 + 1] * r * g.y);
        xe[e4 + 2] = from_f32<T>(x[i * E + e4 + 2] * r * g.z);
        xe[e4 + 3] = from_f32<T>(x[i * E + e4 + 3] * r * g.w);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = (i * 32 + lane) * E;
    if (e < sh.rank) *reinterpret_cast<uint4*>(y + e) = xv[i];
  }
  if (sh.rope && lane < 16) {
    const Pairs<T> p = load_pairs(kv + tok * sh.kv_stride + sh.rank, j, sh.interleaved);
    store_turned(y + sh.rank, j, sh.interleaved, p, t);
  }
}

}  // namespace

cudaError_t launch_latent_append(const void* kv, const float* w, const float* inv_freq,
                                 const void* q_pe, void* q_out, void* cache,
                                 const int32_t* page_table, const int32_t* seq_lens,
                                 const int32_t* cu_seqlens, LatentAppendShape sh, int dtype,
                                 cudaStream_t stream) {
  sh.parts = 1 + (q_pe ? (sh.H + kHeadsPerPart - 1) / kHeadsPerPart : 0);
  const long long units = sh.tokens * sh.parts;
  const unsigned grid = (unsigned)((units + kWarps - 1) / kWarps);
  if (dtype == KDA_BF16)
    KDA_TIMED(KDA_KERNEL_LATENT_APPEND, stream,
              kda_latent_append_kernel<<<grid, 32 * kWarps, 0, stream>>>(
                  static_cast<const __nv_bfloat16*>(kv), w, inv_freq,
                  static_cast<const __nv_bfloat16*>(q_pe), static_cast<__nv_bfloat16*>(q_out),
                  static_cast<__nv_bfloat16*>(cache), page_table, seq_lens, cu_seqlens, sh));
  else
    KDA_TIMED(KDA_KERNEL_LATENT_APPEND, stream,
              kda_latent_append_kernel<<<grid, 32 * kWarps, 0, stream>>>(
                  static_cast<const float*>(kv), w, inv_freq, static_cast<const float*>(q_pe),
                  static_cast<float*>(q_out), static_cast<float*>(cache), page_table, seq_lens,
                  cu_seqlens, sh));
  note_launches(1);
  return cudaGetLastError();
}

}  // namespace kda
