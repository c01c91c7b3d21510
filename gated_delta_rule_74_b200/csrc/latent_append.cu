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
// Every byte is read and written once; what bounds the kernel short of memory is
// instructions, so that a lane moves 16 bytes a load and store (a quarter of a bf16 head's
// pairs, an eighth of an fp32 head's) and forms one frequency's angle, which the others
// take from it.  With many tokens a warp does all of one, its row (16 elements a lane, the
// norm a warp reduction) and its query heads, eight (fp32: four) a step, two steps'
// loads ahead; with few (a decode step) a warp takes the row or 16 query heads, to wait
// for fewer loads in a row.
#include "kda_common.cuh"
#include "latent.cuh"

namespace kda {
namespace {

constexpr int kRope = 64;               // rotated elements a row (or none)
constexpr int kHeadsPerPart = 16;
constexpr int kWarps = 4;
constexpr uint32_t kAll = 0xffffffffu;

// E pairs of one lane (E: elements of 16 bytes): pairs [E j, E j + E), whose elements are
// x[2 E j, 2 E j + 2 E) interleaved, else x[E j, ..) and x[32 + E j, ..).
template <typename T> struct Pairs {
  static constexpr int E = 16 / sizeof(T);
  uint4 u, w;
  __device__ void load(const T* x, int j, bool inter) {
    u = *reinterpret_cast<const uint4*>(x + (inter ? 2 * E * j : E * j));
    w = *reinterpret_cast<const uint4*>(x + (inter ? 2 * E * j + E : kRope / 2 + E * j));
  }
  __device__ void store(T* x, int j, bool inter) const {
    *reinterpret_cast<uint4*>(x + (inter ? 2 * E * j : E * j)) = u;
    *reinterpret_cast<uint4*>(x + (inter ? 2 * E * j + E : kRope / 2 + E * j)) = w;
  }
  __device__ void turn(const float (&c)[E], const float (&s)[E], bool inter) {
    T a[E], b[E];                                     // the loads' elements
    *reinterpret_cast<uint4*>(a) = u;
    *reinterpret_cast<uint4*>(b) = w;
#pragma unroll
    for (int i = 0; i < E; ++i) {
      // interleaved: pair i is elements 2 i, 2 i + 1 of the two loads together
      T& p = inter ? (i < E / 2 ? a[(2 * i) % E] : b[(2 * i) % E]) : a[i];
      T& q = inter ? (i < E / 2 ? a[(2 * i + 1) % E] : b[(2 * i + 1) % E]) : b[i];
      const float x = to_f32(p), y = to_f32(q);
      p = from_f32<T>(x * c[i] - y * s[i]);
      q = from_f32<T>(x * s[i] + y * c[i]);
    }
    u = *reinterpret_cast<const uint4*>(a);
    w = *reinterpret_cast<const uint4*>(b);
  }
};

// cos and sin of pos * freq
__device__ __forceinline__ void turn(int pos, float freq, float* c, float* s) {
  double t = (double)pos * (double)freq * 0.15915494309189533577;   // turns: 1 / (2 pi)
  t -= rint(t);
  sincospif(2.0f * (float)t, s, c);
}

template <typename T, bool kInter>
__global__ void __launch_bounds__(32 * kWarps, 6)
kda_latent_append_kernel(const T* __restrict__ kv, const float* __restrict__ w,
                         const float* __restrict__ inv_freq, const T* q_pe, T* q_out,
                         T* __restrict__ cache, const int32_t* __restrict__ page_table,
                         const int32_t* __restrict__ seq_lens,
                         const int32_t* __restrict__ cu_seqlens, LatentAppendShape sh) {
  constexpr int E = 16 / sizeof(T);                   // elements of a 16-byte load
  constexpr int NV = 16 / E;                          // a row's loads of a lane
  constexpr int LH = 32 / E, HP = 32 / LH;            // lanes of a head, heads of a step
  const int lane = threadIdx.x & 31;
  const int tok = blockIdx.x * kWarps + (threadIdx.x >> 5), part = blockIdx.y;
  if (tok >= sh.tokens) return;

  // ---- query heads [h0, h1), two steps' loads ahead; the loads do not wait for the position
  const int j = lane % LH;
  // (the row's own part of several has none)
  const bool heads = q_pe && (sh.parts == 1 || part > 0);
  const int h0 = (part > 0 ? (part - 1) * kHeadsPerPart : 0) + lane / LH;
  const int h1 = !heads ? 0 : sh.parts == 1 ? sh.H : min(part * kHeadsPerPart, sh.H);
  Pairs<T> p0, p1;
  auto load_heads = [&](int h) {
    if (h < h1) p0.load(q_pe + tok * sh.q_tok + h * sh.q_head, j, kInter);
    if (h + HP < h1) p1.load(q_pe + tok * sh.q_tok + (h + HP) * sh.q_head, j, kInter);
  };
  load_heads(h0);
  const T* const x = kv + tok * sh.kv_stride;
  uint4 xv[NV];
  Pairs<T> rp;
  if (part == 0) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = (i * 32 + lane) * E;
      xv[i] = e < sh.rank ? __ldg(reinterpret_cast<const uint4*>(x + e)) : make_uint4(0, 0, 0, 0);
    }
    if (sh.rope && lane < LH) rp.load(x + sh.rank, lane, kInter);
  }
  int seq, first, cnt;
  if (!token_sequence(tok, sh.N, sh.L, cu_seqlens, (int)sh.tokens, lane, &seq, &first, &cnt)) return;
  const int pos = __ldg(seq_lens + seq) - cnt + (tok - first);

  // the row's slot (page -1: outside of the table or the cache, it is not written)
  int page = -1, row = 0;
  if (part == 0 && pos >= 0) {
    const int pg = pos / sh.page_size;
    row = pos - pg * sh.page_size;
    if (pg < sh.max_pages) page = __ldg(page_table + (long long)seq * sh.max_pages + pg);
  }
  const bool turned = sh.rope && inv_freq;
  float c[E], s[E];
  if (turned) {
    float cl, sl;                                     // of frequency `lane`
    turn(pos, __ldg(inv_freq + lane), &cl, &sl);
#pragma unroll
    for (int i = 0; i < E; ++i) {
      c[i] = __shfl_sync(kAll, cl, E * j + i);
      s[i] = __shfl_sync(kAll, sl, E * j + i);
    }
  }

  for (int h = h0; h < h1; h += 2 * HP) {
    if (turned) p0.turn(c, s, kInter);
    p0.store(q_out + tok * sh.qo_tok + h * sh.qo_head, j, kInter);
    if (h + HP < h1) {
      if (turned) p1.turn(c, s, kInter);
      p1.store(q_out + tok * sh.qo_tok + (h + HP) * sh.qo_head, j, kInter);
    }
    load_heads(h + 2 * HP);
  }
  if (page < 0 || page >= sh.num_pages) return;

  // ---- the row
  T* const y = cache + page * sh.page_stride + row * sh.row_stride;
  if (w) {
    float f[16], ss = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const T* xe = reinterpret_cast<const T*>(&xv[i]);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        f[i * E + e] = to_f32(xe[e]);
        ss = fmaf(f[i * E + e], f[i * E + e], ss);
      }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(kAll, ss, o);
    const float r = rsqrtf(ss / (float)sh.rank + sh.eps);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e0 = (i * 32 + lane) * E;
      if (e0 >= sh.rank) continue;
      T* xe = reinterpret_cast<T*>(&xv[i]);
#pragma unroll
      for (int e4 = 0; e4 < E; e4 += 4) {
        const float4 g = __ldg(reinterpret_cast<const float4*>(w + e0 + e4));
        xe[e4] = from_f32<T>(f[i * E + e4] * r * g.x);
        xe[e4 + 1] = from_f32<T>(f[i * E + e4 + 1] * r * g.y);
        xe[e4 + 2] = from_f32<T>(f[i * E + e4 + 2] * r * g.z);
        xe[e4 + 3] = from_f32<T>(f[i * E + e4 + 3] * r * g.w);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = (i * 32 + lane) * E;
    if (e < sh.rank) *reinterpret_cast<uint4*>(y + e) = xv[i];
  }
  if (sh.rope && lane < LH) {
    if (turned) rp.turn(c, s, kInter);
    rp.store(y + sh.rank, lane, kInter);
  }
}

template <typename T>
void run_append(const void* kv, const float* w, const float* inv_freq, const void* q_pe,
                void* q_out, void* cache, const int32_t* page_table, const int32_t* seq_lens,
                const int32_t* cu_seqlens, const LatentAppendShape& sh, cudaStream_t stream) {
  auto kern = sh.interleaved ? kda_latent_append_kernel<T, true> : kda_latent_append_kernel<T, false>;
  kern<<<dim3((unsigned)((sh.tokens + kWarps - 1) / kWarps), sh.parts), 32 * kWarps, 0, stream>>>(
      static_cast<const T*>(kv), w, inv_freq, static_cast<const T*>(q_pe), static_cast<T*>(q_out),
      static_cast<T*>(cache), page_table, seq_lens, cu_seqlens, sh);
}

}  // namespace

cudaError_t launch_latent_append(const void* kv, const float* w, const float* inv_freq,
                                 const void* q_pe, void* q_out, void* cache,
                                 const int32_t* page_table, const int32_t* seq_lens,
                                 const int32_t* cu_seqlens, LatentAppendShape sh, int dtype,
                                 cudaStream_t stream) {
  int sms = 0;
  if (!device_ctx(&sms, nullptr)) return cudaErrorInvalidDevice;
  // a warp a token once there are 16 warps an SM of them
  sh.parts = !q_pe || sh.tokens >= 16LL * sms ? 1 : 1 + (sh.H + kHeadsPerPart - 1) / kHeadsPerPart;
  auto run = dtype == KDA_BF16 ? run_append<__nv_bfloat16> : run_append<float>;
  KDA_TIMED(KDA_KERNEL_LATENT_APPEND, stream,
            run(kv, w, inv_freq, q_pe, q_out, cache, page_table, seq_lens, cu_seqlens, sh, stream));
  note_launches(1);
  return cudaGetLastError();
}

}  // namespace kda
