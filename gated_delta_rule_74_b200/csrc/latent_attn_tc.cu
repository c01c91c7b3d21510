// Latent attention over a paged cache on the tensor cores (kda_latent_attn, bf16).
//
// For a block of up to 96 query rows (new token, head) and a tile of 64 cached rows C
// [64][rank + rope], whose first `rank` columns are the values too:
//     S (128 x 64)      = Q C^T                      Q's rows on the TMEM lanes
//     P (rows x 64)     = 2^(scale log2e S - m)      to shared memory as bf16
//     O^T (rank x rows) += C[:, 0:rank]^T P^T        the value columns on the lanes
// with the running maximum m and sum of the softmax.  The tile is read from memory once and
// serves both products from one place in shared memory: K-major for the scores, the same
// bytes MN-major for the values.  O is held transposed because a row needs its 512 values
// beside S in 512 TMEM columns: O^T takes `rows` columns for each 128 of them, so that 96
// rows (all heads of a model at one token) fit with two score tiles; with Q's rows on the
// lanes O alone would take all 512 columns.
//
// Bound by the cache's bytes for few rows (12 heads: 24 FLOP a byte), near the balance of
// memory and tensor cores at 96 rows.  The MMAs stage A and B in shared memory; at N = 64
// reading them takes 48 of the 128-byte cycles that the 32 of the product would leave.
//
// One CTA an SM, its stretch of tiles as latent_attn.cuh lays it out.  Warp 0 brings the
// tiles by TMA into a ring of slots (128 columns x 64 rows, the rope columns apart), one box
// a run of rows inside of a page; warp 1 issues the MMAs; warps 4..7 do the softmax (thread =
// row), the rare rescaling of O^T and the results (thread = value column).  The maximum that
// the weights refer to moves only when a row's passes it by 2^8, so that O^T is rescaled a
// few times a sequence; the weights stay below 2^8, far inside of bf16 and fp32.
// The scores of tile t + 1 are issued while tile t's softmax runs, as far as slots allow
// (all of them up to 64 rows, the rope and half of the rank at 96); whichever of "the next slot is
// there" and "the weights are there" comes first goes first.
//
// Rows of the tile that some query row does not see (the causal edge, what lies behind the
// length in the last page) have weights of exactly zero; their infinities and NaN would
// still spoil the sum, so after the scores of such a tile are done those values are set to
// zero in shared memory.  Of a visible row they have reached the score already.
#include "latent_attn.cuh"
#include "sm100.cuh"
#include "tma.cuh"

namespace kda {

// Set when a bounded wait of the latent attention gives up (diagnostic).
__device__ int g_latent_timeout = 0;

namespace {
using namespace sm100;
using bf16 = __nv_bfloat16;

constexpr int kTcThreads = 256;
constexpr int kTcTile = 64;
constexpr int kTcMaxRows = 96;
constexpr uint32_t kChunk = 64 * 128;              // 64 cached rows x 64 columns
constexpr uint32_t kSlot = 2 * kChunk;
constexpr int kMaxSlots = 12;
constexpr uint32_t kTcSmem = 229376;               // Q, slots, P; + 1024 for the alignment
constexpr uint32_t kTmemCols = 512, kTmemS = 384;
constexpr uint32_t kWaitLimit = 1u << 22, kPollLimit = 1u << 26;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// How shared memory is divided, from the block's rows and the row's columns.
struct TcPlan {
  int nr;                           // rows of a block, a multiple of 16 up to 96
  int npair;                        // rank / 128
  int nq, np;                       // Q and P buffers
  int slots, rope_slots;
  uint32_t q_bytes, p_bytes;
  int box_rows, groups;             // rows of a TMA box; boxes for 64 rows of one chunk
};

// Q is buffered twice while it is small (a decode step changes blocks every few tiles), P
// while the slots then still hold two tiles.
TcPlan tc_plan(int nr, int rank, int rope, int page_size) {
  TcPlan p;
  p.nr = nr;
  p.npair = rank / 128;
  p.q_bytes = (uint32_t)nr * (rank + rope) * 2;
  p.p_bytes = (uint32_t)nr * 128;
  p.nq = nr <= 32 ? 2 : 1;
  p.np = nr <= 64 ? 2 : 1;
  const uint32_t left = kTcSmem - p.nq * p.q_bytes - p.np * p.p_bytes;
  p.rope_slots = rope ? 2 : 0;
  if (rope && (int)((left - 2 * kChunk) / kSlot) < 2 * p.npair) p.rope_slots = 1;
  p.slots = (int)((left - p.rope_slots * kChunk) / kSlot);
  if (p.slots > kMaxSlots) p.slots = kMaxSlots;
  p.box_rows = kTcTile;
  while (page_size % p.box_rows) p.box_rows /= 2;
  p.groups = kTcTile / p.box_rows;
  return p;
}

struct TcBars {
  uint64_t q_full[2], q_empty[2];
  uint64_t full[kMaxSlots], empty[kMaxSlots];
  uint64_t rope_full[2], rope_empty[2];
  uint64_t s_full[2], s_empty[2];
  uint64_t p_full[2], pv_done[2];
  uint64_t o_empty, drain;
};

__device__ __forceinline__ float ex2(float x) {      // 2^x; 0 below 2^-126
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t zero_bad(uint32_t w) {     // two bf16: inf, NaN -> 0
  if ((w & 0x7f80u) == 0x7f80u) w &= 0xffff0000u;
  if ((w & 0x7f800000u) == 0x7f800000u) w &= 0x0000ffffu;
  return w;
}

__global__ void __launch_bounds__(kTcThreads, 1)
kda_latent_tc_kernel(const __grid_constant__ CUtensorMap q_map,
                     const __grid_constant__ CUtensorMap c_map,
                     const int32_t* __restrict__ page_table,
                     const int32_t* __restrict__ seq_lens,
                     const int32_t* __restrict__ cu_seqlens, bf16* __restrict__ out,
                     float* __restrict__ lse, LatentAttnShape sh, TcPlan pl, LatentPartials pt) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ TcBars bar;
  __shared__ LatentStart st;
  __shared__ long long s_sum[33];
  __shared__ float s_row[kTcMaxRows];               // rescaling factors, then 1 / sum
  __shared__ uint32_t s_tmem;
  uint8_t* const sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                 ~uintptr_t(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int nr = pl.nr, npair = pl.npair;
  uint8_t* const sq = sm;
  uint8_t* const sslot = sq + pl.nq * pl.q_bytes;
  uint8_t* const srope = sslot + pl.slots * kSlot;
  uint8_t* const sp = srope + pl.rope_slots * kChunk;

  if (warp == 1) {
    tmem_alloc(&s_tmem, kTmemCols);
    tmem_relinquish();
  }
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar.q_full[i], 1);
      mbar_init(&bar.q_empty[i], 1);
      mbar_init(&bar.rope_full[i], 1);
      mbar_init(&bar.rope_empty[i], 1);
      mbar_init(&bar.s_full[i], 1);
      mbar_init(&bar.s_empty[i], 4);
      mbar_init(&bar.p_full[i], 4);
      mbar_init(&bar.pv_done[i], 1);
    }
    for (int i = 0; i < kMaxSlots; ++i) {
      mbar_init(&bar.full[i], 1);
      mbar_init(&bar.empty[i], 1);
    }
    mbar_init(&bar.o_empty, 4);
    mbar_init(&bar.drain, 1);
    fence_mbar_init();
    pt.head[blockIdx.x] = make_int4(0, 0, 0, 0);
  }
  latent_find_start(sh, seq_lens, cu_seqlens, nr, kTcTile, &st, s_sum);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tb = s_tmem;
  grid_dep_launch();                                // the join may be made ready
  const int qblocks = (sh.rank + sh.rope) / 64;
  const bool rope = sh.rope != 0;
  bool ok = true;

  if (warp == 0) {
    // ------------------------------------------------------------- tiles by TMA
    LatentWalk walk(st);
    LatentPiece p;
    uint32_t it = 0, slot = 0, slot_use = 0, rt = 0;     // blocks, pair slots, rope slots so far
    while (ok && walk.next(sh, seq_lens, cu_seqlens, nr, kTcTile, &p)) {
      const uint32_t qi = it % pl.nq, quse = it / pl.nq;
      ++it;
      if (quse > 0) ok = mbar_wait(&bar.q_empty[qi], (quse - 1) & 1, kWaitLimit);
      if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
      if (lane == 0) {
        mbar_arrive_expect_tx(&bar.q_full[qi], pl.q_bytes);
        for (int c = 0; c < qblocks; ++c)
          tma_load_3d(sq + qi * pl.q_bytes + c * nr * 128, &q_map, 64 * c, (int)p.row0, 0,
                      &bar.q_full[qi]);
      }
      __syncwarp();
      for (int t = p.t0; t < p.t1 && ok; ++t) {
        // this lane's box: rows [64 t + lane box_rows, ..) of the sequence; zeros where there
        // is no such page
        int page = sh.num_pages, row = 0;
        const int pos = t * kTcTile + lane * pl.box_rows;
        if (lane < pl.groups && pos < p.len) {
          const int id = __ldg(page_table + (long long)p.n * sh.max_pages + pos / sh.page_size);
          row = pos % sh.page_size;
          if (id >= 0 && id < sh.num_pages) page = id;
        }
        if (rope) {
          const uint32_t r = rt % pl.rope_slots, use = rt / pl.rope_slots;
          ++rt;
          if (use > 0) ok = mbar_wait(&bar.rope_empty[r], (use - 1) & 1, kWaitLimit);
          if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
          if (lane == 0) mbar_arrive_expect_tx(&bar.rope_full[r], kChunk);
          __syncwarp();
          if (lane < pl.groups)
            tma_load_3d(srope + r * kChunk + lane * pl.box_rows * 128, &c_map, sh.rank, row, page,
                        &bar.rope_full[r]);
        }
        for (int j = 0; j < npair; ++j) {
          if (slot_use > 0) ok = mbar_wait(&bar.empty[slot], (slot_use - 1) & 1, kWaitLimit);
          if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
          if (lane == 0) mbar_arrive_expect_tx(&bar.full[slot], kSlot);
          __syncwarp();
          if (lane < pl.groups) {
            uint8_t* d = sslot + slot * kSlot + lane * pl.box_rows * 128;
            tma_load_3d(d, &c_map, 128 * j, row, page, &bar.full[slot]);
            tma_load_3d(d + kChunk, &c_map, 128 * j + 64, row, page, &bar.full[slot]);
          }
          if (++slot == (uint32_t)pl.slots) {
            slot = 0;
            ++slot_use;
          }
        }
      }
    }
    if (!ok) {
      // let the copies in flight land before the memory goes away
      for (uint32_t i = 0; i < (uint32_t)pl.slots; ++i) {
        const uint32_t uses = slot_use + (i < slot ? 1 : 0);
        if (uses) mbar_wait(&bar.full[i], (uses - 1) & 1, kWaitLimit);
      }
      for (uint32_t r = 0; r < (uint32_t)pl.rope_slots; ++r) {
        const uint32_t uses = rt / pl.rope_slots + (r < rt % pl.rope_slots ? 1 : 0);
        if (uses > 1) mbar_wait(&bar.rope_full[r], (uses - 2) & 1, kWaitLimit);
      }
      for (uint32_t i = 0; i < (uint32_t)pl.nq; ++i) {
        const uint32_t uses = it / pl.nq + (i < it % pl.nq ? 1 : 0);
        if (uses > 1) mbar_wait(&bar.q_full[i], (uses - 2) & 1, kWaitLimit);
      }
    }
  } else if (warp == 1 && lane == 0) {
    // ------------------------------------------------------------- the MMAs
    const uint32_t id_qk = idesc_bf16(128, kTcTile, false, false);
    const uint32_t id_pv = idesc_bf16(128, nr, true, false);
    const uint32_t aslot = smem_u32(sslot), arope = smem_u32(srope), ap = smem_u32(sp);
    LatentWalk walk(st);
    LatentPiece p;
    uint32_t it = 0, g = 0, rt = 0;                      // blocks, tiles, rope slots
    uint32_t slot = 0, use = 0;                          // of the next scores' pair
    uint32_t vslot = 0;                                  // of the next values' pair
    // next pair (or, with k = -1, the rope columns) of the scores of tile `t`
    auto issue_qk = [&](int k, uint32_t t, uint32_t aq) {
      const uint32_t d = tb + kTmemS + (t & 1) * kTcTile;
      if (k < 0) {
        const uint32_t r = rt % pl.rope_slots;
        const uint32_t a = aq + (uint32_t)(2 * npair * nr * 128), b = arope + r * kChunk;
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          mma_ss(d, desc_kmajor_sw128(a, nr, kk), desc_kmajor_sw128(b, kTcTile, kk), id_qk, kk > 0);
        mma_commit(&bar.rope_empty[r]);
        ++rt;
        return;
      }
      const uint32_t a = aq + (uint32_t)(2 * k * nr * 128), b = aslot + slot * kSlot;
#pragma unroll
      for (int kk = 0; kk < 8; ++kk)
        mma_ss(d, desc_kmajor_sw128(a, nr, kk), desc_kmajor_sw128(b, kTcTile, kk), id_qk,
               rope || k > 0 || kk > 0);
      if (++slot == (uint32_t)pl.slots) {
        slot = 0;
        ++use;
      }
    };
    auto qk_bar = [&](int k) -> uint64_t* { return k < 0 ? &bar.rope_full[rt % pl.rope_slots] : &bar.full[slot]; };
    auto qk_par = [&](int k) -> uint32_t { return (k < 0 ? rt / pl.rope_slots : use) & 1; };

    while (ok && walk.next(sh, seq_lens, cu_seqlens, nr, kTcTile, &p)) {
      const uint32_t qi = it % pl.nq;
      const uint32_t aq = smem_u32(sq + qi * pl.q_bytes);
      const int nt = p.t1 - p.t0;
      ok = mbar_wait(&bar.q_full[qi], (it / pl.nq) & 1, kWaitLimit);
      const int k0 = rope ? -1 : 0;
      int k = k0;                                        // next part of the scores of tile i
      for (int i = 0; i <= nt && ok; ++i) {
        // scores of tile i (g + 1 for i > 0) and, between them, the values of tile i - 1
        const uint32_t ts = i == 0 ? g : g + 1;
        const bool scores = i < nt;
        if (scores && ts >= 2) ok = ok && mbar_wait(&bar.s_empty[ts & 1], ((ts >> 1) - 1) & 1, kWaitLimit);
        if (i > 0) {
          const uint32_t pb = g % pl.np;
          uint32_t polls = 0;
          while (ok && !mbar_test_wait(&bar.p_full[pb], (g / pl.np) & 1)) {
            if (scores && k < npair && mbar_test_wait(qk_bar(k), qk_par(k))) {
              tc_fence_after();
              issue_qk(k++, ts, aq);
              if (k == npair) mma_commit(&bar.s_full[ts & 1]);
            }
            if (++polls > kPollLimit) ok = false;
          }
          if (i == 1 && it > 0)                          // the block before has left O^T
            ok = ok && mbar_wait(&bar.o_empty, (it - 1) & 1, kWaitLimit);
          if (!ok) break;
          tc_fence_after();
          for (int j = 0; j < npair; ++j) {
            const uint32_t a = aslot + vslot * kSlot, b = ap + pb * pl.p_bytes;
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_ss(tb + j * nr, desc_mnmajor_sw128(a, kTcTile, kk), desc_kmajor_sw128(b, nr, kk),
                     id_pv, i > 1 || kk > 0);
            mma_commit(&bar.empty[vslot]);
            if (++vslot == (uint32_t)pl.slots) vslot = 0;
          }
          mma_commit(&bar.pv_done[pb]);
          ++g;
        }
        if (scores) {
          while (ok && k < npair) {
            ok = mbar_wait(qk_bar(k), qk_par(k), kWaitLimit);
            if (!ok) break;
            tc_fence_after();
            issue_qk(k++, ts, aq);
            if (k == npair) mma_commit(&bar.s_full[ts & 1]);
          }
          k = k0;
          if (i == nt - 1) mma_commit(&bar.q_empty[qi]);
        }
      }
      ++it;
    }
    if (!ok) {
      mma_commit(&bar.drain);
      mbar_wait(&bar.drain, 0, kWaitLimit);
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------- softmax and results
    const int wq = warp - 4, r = 32 * wq + lane, t128 = tid - 128;
    const uint32_t tl = tb + ((uint32_t)(32 * wq) << 16);
    const bool has_rows = 32 * wq < nr;
    const float c = sh.scale * kLog2e;
    LatentWalk walk(st);
    LatentPiece p;
    uint32_t g = 0;
    bool dead = false;
    while (!dead && walk.next(sh, seq_lens, cu_seqlens, nr, kTcTile, &p)) {
      const bool row = r < p.rows;
      const int lim = min(p.start + (p.row_in_seq + r) / sh.H + 1, p.len);
      const int low = p.start + p.row_in_seq / sh.H + 1;
      float m = -INFINITY, l = 0.f;
      for (int t = p.t0; t < p.t1; ++t, ++g) {
        ok = ok && mbar_wait(&bar.s_full[g & 1], (g >> 1) & 1, kWaitLimit);
        tc_fence_after();
        const int k0 = t * kTcTile;
        const bool mixed = k0 + kTcTile > low;
        uint32_t s[4][16];
        if (has_rows) {
#pragma unroll
          for (int i = 0; i < 4; ++i) tmem_ld16(tl + kTmemS + (g & 1) * kTcTile + 16 * i, s[i]);
          tmem_wait_ld();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.s_empty[g & 1]);
        bool need = false;
        float mt = -INFINITY;
        if (has_rows) {
          if (mixed) {
#pragma unroll
            for (int i = 0; i < 64; ++i)
              if (k0 + i >= lim) s[i >> 4][i & 15] = 0xff800000u;      // -inf
          }
#pragma unroll
          for (int i = 0; i < 64; ++i) mt = fmaxf(mt, __uint_as_float(s[i >> 4][i & 15]));
          mt = fmaxf(m, mt * c);                         // c > 0: the scaled maximum
          need = row && m != -INFINITY && mt > m + 8.f;
          if (m == -INFINITY) m = mt;
        }
        // rows that some query row does not see: nothing that 0 * would turn into a NaN
        if (mixed) {
          const int first = max(low - k0, 0), per = sh.rank / 8;
          for (int i = t128; i < (kTcTile - first) * per; i += 128) {
            const int tok = first + i / per, c8 = i % per;
            const uint32_t sl = (g * npair + (c8 >> 4)) % pl.slots;
            uint4* w = reinterpret_cast<uint4*>(sslot + sl * kSlot + ((c8 >> 3) & 1) * kChunk +
                                                tok * 128 + (c8 & 7) * 16);
            const uint4 a = *w;
            const uint4 b = make_uint4(zero_bad(a.x), zero_bad(a.y), zero_bad(a.z), zero_bad(a.w));
            if (a.x != b.x || a.y != b.y || a.z != b.z || a.w != b.w) *w = b;
          }
        }
        if (named_bar_or(1, 128, need || !ok)) {
          if (named_bar_or(1, 128, !ok)) { dead = true; break; }
          // rescale O^T to the maxima of now (tiles before this one have been added)
          float al = 1.f;
          if (has_rows && row && m != -INFINITY) {
            al = ex2(m - mt);
            l *= al;
            m = mt;
          }
          if (r < nr) s_row[r] = al;
          ok = ok && mbar_wait(&bar.pv_done[(g - 1) % pl.np], ((g - 1) / pl.np) & 1, kWaitLimit);
          named_bar(1, 128);
          tc_fence_after();
          for (int j = 0; j < npair; ++j)
            for (int i = 0; i < nr; i += 16) {
              uint32_t o[16];
              tmem_ld16(tl + j * nr + i, o);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * s_row[i + e]);
              tmem_st16(tl + j * nr + i, o);
            }
          tmem_wait_st();
          tc_fence_before();
        }
        if (has_rows) {
          const float ms = m == -INFINITY ? 0.f : m;
          if (g >= (uint32_t)pl.np)
            ok = ok && mbar_wait(&bar.pv_done[g % pl.np], (g / pl.np - 1) & 1, kWaitLimit);
          uint8_t* const pr = sp + (g % pl.np) * pl.p_bytes + r * 128;
#pragma unroll
          for (int c8 = 0; c8 < 8; ++c8) {
            float e[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              e[i] = row ? ex2(fmaf(__uint_as_float(s[c8 >> 1][8 * (c8 & 1) + i]), c, -ms)) : 0.f;
              l += e[i];
            }
            if (r < nr)
              *reinterpret_cast<uint4*>(pr + ((c8 ^ (r & 7)) << 4)) =
                  make_uint4(pack_bf16(e[0], e[1]), pack_bf16(e[2], e[3]), pack_bf16(e[4], e[5]),
                             pack_bf16(e[6], e[7]));
          }
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.p_full[g % pl.np]);
      }
      if (dead) break;
      // ---- results: whole blocks to the output, shared ones to a partial slot
      const bool first = p.t0 == 0, last = p.t1 == p.tiles;
      const int slot = first && last ? -1 : 2 * (int)blockIdx.x + (first ? 1 : 0);
      if (r < nr) {
        s_row[r] = l == 0.f ? 0.f : 1.0f / l;
        const float z = l == 0.f ? -INFINITY : (m == -INFINITY ? 0.f : m) * kLn2 + logf(l);
        if (slot >= 0) pt.lse[slot * nr + r] = z;
        else if (lse && row) lse[p.row0 + r] = z;
      }
      if (slot >= 0 && first && t128 == 0)
        pt.head[blockIdx.x] =
            make_int4((int)p.row0, p.rows, latent_cta_of(p.pos + p.tiles - 1, st.W, st.G), 0);
      ok = ok && mbar_wait(&bar.pv_done[(g - 1) % pl.np], ((g - 1) / pl.np) & 1, kWaitLimit);
      if (named_bar_or(1, 128, !ok)) break;
      tc_fence_after();
      for (int j = 0; j < npair; ++j) {
        const int d = 128 * j + r;
        for (int i = 0; i < p.rows; i += 16) {
          uint32_t o[16];
          tmem_ld16(tl + j * nr + i, o);
          tmem_wait_ld();
          if (slot < 0) {
#pragma unroll
            for (int e = 0; e < 16; ++e)
              if (i + e < p.rows)
                out[(p.row0 + i + e) * sh.rank + d] =
                    __float2bfloat16_rn(__uint_as_float(o[e]) * s_row[i + e]);
          } else {
#pragma unroll
            for (int e = 0; e < 16; ++e)
              if (i + e < p.rows)
                pt.o[((long long)slot * nr + i + e) * sh.rank + d] =
                    __uint_as_float(o[e]) * s_row[i + e];
          }
        }
      }
      tc_fence_before();
      named_bar(1, 128);                                 // s_row is free again
      if (lane == 0) mbar_arrive(&bar.o_empty);
    }
  }
  if (!ok) atomicExch(&g_latent_timeout, 1);
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tb, kTmemCols);
  }
}

// Rows of a block: all of a sequence's where they fit, else the size that cuts them into
// fewer blocks (each reads the cached rows again), the smaller one where both do.
int tc_rows(int N, int L, int T, int H) {
  const long long rows = L > 0 ? (long long)L * H : (((long long)T + N - 1) / N) * H;
  if (rows <= kTcMaxRows) return (int)((rows + 15) / 16 * 16);
  return (rows + 63) / 64 <= (rows + kTcMaxRows - 1) / kTcMaxRows ? 64 : kTcMaxRows;
}

}  // namespace

bool latent_tc_supported(int dtype, int page_size) { return dtype == KDA_BF16 && page_size % 8 == 0; }

int latent_tc_ctas(int sms) { return sms < kLatentMaxCtas ? sms : kLatentMaxCtas; }

size_t latent_tc_scratch_bytes(int N, int L, int T, int H, int rank, int sms) {
  return latent_scratch_bytes(latent_tc_ctas(sms), tc_rows(N, L, T, H), rank);
}

cudaError_t launch_latent_tc(const void* q, const void* cache, const int32_t* page_table,
                             const int32_t* seq_lens, const int32_t* cu_seqlens, void* out,
                             float* lse, const LatentAttnShape& sh, int sms, void* buf,
                             cudaStream_t stream) {
  if (!once_per_device(kOnceLatentTc, []() {
        return cudaFuncSetAttribute(kda_latent_tc_kernel,
                                    cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    (int)kTcSmem + 1024) == cudaSuccess;
      }))
    return cudaErrorInvalidDevice;
  const int nr = tc_rows(sh.N, sh.L, sh.T, sh.H), G = latent_tc_ctas(sms);
  const TcPlan pl = tc_plan(nr, sh.rank, sh.rope, sh.page_size);
  const LatentPartials pt = latent_partials(buf, G, nr);
  const uint64_t D = sh.rank + sh.rope;
  const uint64_t rows = (uint64_t)(sh.L > 0 ? (long long)sh.N * sh.L : sh.T) * sh.H;
  CUtensorMap q_map, c_map;
  if (!make_row_map_3d(&q_map, q, D, rows, 1, D * 2, D * 2, 64, (uint32_t)nr) ||
      !make_row_map_3d(&c_map, cache, D, sh.page_size, sh.num_pages, sh.row_stride * 2,
                       sh.page_stride * 2, 64, (uint32_t)pl.box_rows))
    return cudaErrorInvalidValue;
  KDA_TIMED(KDA_KERNEL_LATENT_ATTN, stream,
            kda_latent_tc_kernel<<<G, kTcThreads, kTcSmem + 1024, stream>>>(
                q_map, c_map, page_table, seq_lens, cu_seqlens, static_cast<bf16*>(out), lse, sh,
                pl, pt));
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  note_launches(1);
  return launch_latent_join(out, lse, pt, G, nr, sh.rank, KDA_BF16, stream);
}

// Reads (and with reset clears) g_latent_timeout; host side of kda_device_status.
cudaError_t take_latent_timeout(int* flag, bool reset) {
  int v = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_latent_timeout, sizeof(int));
  if (e == cudaSuccess && reset && v != 0) {
    const int zero = 0;
    e = cudaMemcpyToSymbol(g_latent_timeout, &zero, sizeof(int));
  }
  *flag = v;
  return e;
}

}  // namespace kda
