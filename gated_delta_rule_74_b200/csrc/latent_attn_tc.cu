// Latent attention over a paged cache on the tensor cores (kda_latent_attn, bf16).
//
// For a block of up to 96 query rows (new token, head) and a tile of 64 or 48 cached rows C
// [64][rank + rope], whose first `rank` columns are the values too:
//     S^T (64 x rows)   = C Q^T                      tokens on the TMEM lanes
//     P (64 x rows)     = 2^(scale log2e S - m)      to shared memory as bf16
//     O^T (rank x rows) += C[:, 0:rank]^T P          the value columns on the lanes
// with the running maximum m and sum of the softmax.  The tile is read from memory once and
// serves both products from one place in shared memory: K-major for the scores, the same
// bytes MN-major for the values.  Everything is held transposed.  O^T takes `rows` TMEM
// columns for each 128 of its values, so that 96 rows (all heads of a model at one token) fit
// beside the scores; with rows on the lanes, O alone would take all 512 columns.  S^T makes
// the tile the M side of both products, so that few rows (12 heads) cost the MMAs few
// operand bytes: 2.5 KB of shared memory an MMA of 64 x 16 against 6 KB of 128 x 64 (rows
// padded to the lanes), which held the decode step at 65% of the memory's rate.
//
// Bound by the cache's bytes for few rows (12 heads: 24 FLOP a byte), near the balance of
// memory and tensor cores at 96 rows.
//
// One CTA an SM, its stretch of tiles as latent_attn.cuh lays it out.  Warps 0 and 2 bring
// the tiles by TMA into a ring, eight tokens with all their columns a box (so that pages of any
// multiple of eight do), warp 3 Q; warp 1 issues the scores' MMAs, warp 12 the
// values'; warps 4..11 do the softmax (two warps a lane quarter of 16 tokens, half of the rows
// each; a thread holds two tokens and two of every eight rows), the rare rescaling of O^T and the
// results (thread = value column).  When a wait of one of them gives up, all of them meet at a
// barrier, and those with loads or MMAs in flight wait for these before the CTA leaves; rows that
// it had still to finish become NaN.
// The maximum that the weights refer to moves only when a score passes it by 2^8: a tile then
// needs one vote, no reduction over the tokens, O^T is rescaled a few times a sequence, and
// the weights stay below 2^8, far inside of bf16 and fp32.  Sums are kept by thread and
// joined at the end of a block; O^T is added up in fp32 in TMEM (against 64 bits 0.0019 of the
// output's norm, its own rounding and the weights', with 1M tokens a block, 0.004 with 4M, where
// what the tensor core cuts off at each of 2^18 additions shows).
// Scores and values are issued by two warps, each of which waits for its own operands alone: one
// warp for both puts the scores of tile t + 1 before the values of tile t, whose slot then comes
// free 1100 cycles later (when the second warp came, on the device: 1024-token chunk 563 -> 500 us,
// 256 sequences 216 -> 209, 43 of 96 heads 153 -> 145; now 521, 203 and 143, after tiles of 48
// tokens and the results' loop, which cost the chunk 7 us, and the meeting of the roles, which cost
// it 5).  The values' products run over 16 tokens at a time and hand those back to the producers
// at once.
// The weights are rounded to bf16 because both operands of an MMA are of one type, the cached rows'.
// The sum that divides adds them unrounded: it is the log-sum's too, which stays good to fp32 that
// way.  A second sum, of the rounded ones, brought the output's error from 0.0020-0.0021 of its norm to
// 0.0019-0.0020 (its own rounding is 0.0017 of that) and cost 96 heads 4.5% and the chunk 1.5%.
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

constexpr int kTcThreads = 416;
constexpr int kSoft = 256;                         // threads of warps 4..11
constexpr int kTcMaxRows = 96;
constexpr int kMaxTiles = 4;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kDrainLimit = 1u << 14;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kNone = -3e38f;                    // maximum of a row that has seen nothing

// Tokens of a tile.  64 fill the MMAs' M side, but there is room for more tiles of 48 beside Q at
// rank 512: three instead of two up to 48 rows (on the device 256 sequences of 12 heads 203 us against
// 207, 100 of 24 heads 96 against 98), two instead of one at 80 and 96 (60 of 80 heads 104 against
// 133).  Of either two fit at 64 rows.  Tiles of 32 at 16 rows cost more MMAs than they save (242 us).
__host__ __device__ constexpr int tc_tile(int nr) { return nr == 64 ? 64 : 48; }
// Dynamic shared memory: all but 3 KB of the 227 (2 KB at 96 rows) for the variables.
__host__ __device__ constexpr uint32_t tc_smem(int nr) { return nr > 80 ? 230400 : 229376; }

// How shared memory is divided, from the block's rows and the row's columns: a ring of tiles,
// Q, P.  A tile is groups of eight tokens, a group all of a row's 64-column chunks one after
// the other, a chunk [8][128 B] with the 128-byte swizzle; a group comes by one TMA box.
struct TcPlan {
  int npair, nch;                   // rank / 128; chunks of a row
  int ntile, nq, np;                // tiles of the ring; Q and P buffers
  uint32_t group, tile_bytes, q_bytes, p_bytes;
};

// Q is buffered twice while that costs no tile (a decode step changes blocks every few tiles), P
// where there is room beside the tiles.
TcPlan tc_plan(int nr, int rank, int rope) {
  TcPlan p;
  const int kt = tc_tile(nr);
  p.npair = rank / 128;
  p.nch = (rank + rope) / 64;
  p.group = (uint32_t)p.nch * 1024;
  p.tile_bytes = kt / 8 * p.group;
  p.q_bytes = (uint32_t)nr * p.nch * 128;
  p.p_bytes = (uint32_t)nr * kt * 2;
  p.nq = nr <= 16 ? 2 : 1;
  const uint32_t fixed = p.nq * p.q_bytes + p.p_bytes;
  p.ntile = (int)((tc_smem(nr) - fixed) / p.tile_bytes);
  if (p.ntile > kMaxTiles) p.ntile = kMaxTiles;
  p.np = fixed + p.ntile * p.tile_bytes + p.p_bytes <= tc_smem(nr) ? 2 : 1;
  return p;
}

struct TcBars {
  uint64_t q_full[2], q_empty[2];
  uint64_t full[kMaxTiles], empty[kMaxTiles][4];   // empty: by 16 tokens of the tile
  uint64_t s_full[2], s_empty[2];
  uint64_t p_full[2], pv_done[2];
  uint64_t o_empty, drain[2];
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

// TMEM: O^T, rank / 128 blocks of NR columns, then two buffers of S^T, or one at 96 rows.
template <int NR>
__global__ void __launch_bounds__(kTcThreads, 1)
kda_latent_tc_kernel(const __grid_constant__ CUtensorMap q_map,
                     const __grid_constant__ CUtensorMap c_map,
                     const int32_t* __restrict__ page_table,
                     const int32_t* __restrict__ seq_lens,
                     const int32_t* __restrict__ cu_seqlens, bf16* __restrict__ out,
                     float* __restrict__ lse, LatentAttnShape sh, TcPlan pl, LatentPartials pt,
                     uint32_t limit) {
  constexpr int nr = NR, KT = tc_tile(NR), KK = KT / 16, kSBuf = NR <= 80 ? 2 : 1;
  // tiles that a block costs besides its own (193 sequences of 3 blocks, rank 384: 122 us, 127 with 2
  // and 3; rank 128 92 and 96; rank 512 with position values 173 and 169)
  constexpr int kLead = NR <= 48 ? 3 : 5;
  constexpr uint32_t kTmemS = 4 * NR;
  // the alignment is part of the declaration: there is no room to round up
  extern __shared__ __align__(1024) uint8_t sm[];
  __shared__ TcBars bar;
  __shared__ LatentStart st;
  __shared__ float s_m[NR];                         // maxima the weights refer to, scaled
  __shared__ uint8_t s_more[NR];                    // tokens each row sees more than the first
  __shared__ __align__(16) float s_row[NR];         // rescaling factors, then 1 / sum
  // two lane quarters' maxima or sums at a time; before, the sums of latent_find_start
  __shared__ __align__(16) float s_red[2 * NR < 68 ? 68 : 2 * NR];
  __shared__ uint32_t s_tmem;
  __shared__ uint32_t s_units[2];                   // 16-token loads that warps 0 and 2 have started
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int npair = pl.npair;
  // the ring first: the MMAs' 64 rows of a 48-token tile reach 16 rows behind it, into Q
  uint8_t* const ring = sm;
  uint8_t* const sq = ring + pl.ntile * pl.tile_bytes;
  uint8_t* const sp = sq + pl.nq * pl.q_bytes;

  if (warp == 1) {
    tmem_alloc(&s_tmem, kTmemCols);
    tmem_relinquish();
  }
  {                                                 // a barrier a thread
    uint64_t* const mine = reinterpret_cast<uint64_t*>(&bar) + tid;
    if (tid < (int)(sizeof(bar) / sizeof(uint64_t))) {
      const bool soft = mine == &bar.o_empty || (mine >= bar.s_empty && mine < bar.s_empty + 2) ||
                        (mine >= bar.p_full && mine < bar.p_full + 2);
      const bool tile = mine >= bar.full && mine < bar.full + kMaxTiles;
      mbar_init(mine, soft ? kSoft / 32 : tile ? KK : 1);
      fence_mbar_init();
    }
  }
  if (tid == 96) pt.head[blockIdx.x] = make_int4(0, 0, 0, 0);
  latent_find_start(sh, seq_lens, cu_seqlens, nr, KT, kLead, &st,
                    reinterpret_cast<long long*>(s_red));
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tb = s_tmem;
  grid_dep_launch();                                // the join may be made ready
  bool ok = true;
  constexpr uint32_t kAll = 0xffffffffu;

  if (warp == 0 || warp == 2) {
    // ------------------------------------------------------------- tiles by TMA
    // 16 tokens (two groups) at a time, the two warps in turn: one warp's loop (wait, look up,
    // arm, copy; 400 to 600 cycles) alone holds the stream below 4 TB/s.
    LatentWalk walk(st);
    LatentPiece p;
    uint32_t slot = 0, use = 0, turn = 0, units = 0;
    while (ok && walk.next(sh, seq_lens, cu_seqlens, nr, KT, kLead, &p)) {
      // lane's group of tile t: its page (one past the cache, which reads as zeros, where there
      // is none)
      auto look = [&](int t) {
        const int pos = t * KT + 8 * lane;
        if (lane >= KT / 8 || t >= p.t1 || pos >= p.len) return sh.num_pages;
        const int id = __ldg(page_table + (long long)p.n * sh.max_pages + pos / sh.page_size);
        return id >= 0 && id < sh.num_pages ? id : sh.num_pages;
      };
      int next_page = look(p.t0);
      for (int t = p.t0; t < p.t1 && ok; ++t) {
        const int page = next_page, row = (t * KT + 8 * lane) % sh.page_size;
        next_page = look(t + 1);
        uint8_t* const d = ring + slot * pl.tile_bytes;
        for (int k = 0; k < KK; ++k, turn ^= 1) {
          if (turn != (uint32_t)(warp >> 1)) continue;
          if (use > 0) ok = __all_sync(kAll, mbar_wait(&bar.empty[slot][k], (use - 1) & 1, limit));
          if (!ok) break;
          const int pg0 = __shfl_sync(kAll, page, 2 * k), rw0 = __shfl_sync(kAll, row, 2 * k);
          const int pg1 = __shfl_sync(kAll, page, 2 * k + 1), rw1 = __shfl_sync(kAll, row, 2 * k + 1);
          if (elect_one()) {
            mbar_arrive_expect_tx(&bar.full[slot], 2 * pl.group);
            tma_load_4d(d + 2 * k * pl.group, &c_map, 0, rw0, 0, pg0, &bar.full[slot]);
            tma_load_4d(d + (2 * k + 1) * pl.group, &c_map, 0, rw1, 0, pg1, &bar.full[slot]);
          }
          ++units;
          __syncwarp();
        }
        if (++slot == (uint32_t)pl.ntile) {
          slot = 0;
          ++use;
        }
      }
    }
    if (lane == 0) s_units[warp >> 1] = units;
    if (named_bar_or(2, kTcThreads, !ok) && warp == 0) {
      // of the last tiles' loads those that were not started arrive without one, so that each
      // tile's barrier completes when what was started has landed
      uint32_t end = 2 * s_units[1];                     // loads in their order: warps 0, 2, 0, ..
      if (s_units[0] > 0) end = max(end, 2 * s_units[0] - 1);
      const uint32_t tiles = (end + KK - 1) / KK, n = (uint32_t)pl.ntile;
      for (uint32_t i = tiles > n ? tiles - n : 0; i < tiles; ++i) {
        for (uint32_t u = i * KK; u < (i + 1) * KK; ++u)
          if (u / 2 >= s_units[u & 1] && lane == 0) mbar_arrive(&bar.full[i % n]);
        __syncwarp();
        mbar_wait(&bar.full[i % n], (i / n) & 1, kDrainLimit);
      }
    }
  } else if (warp == 3) {
    // ------------------------------------------------------------- Q by TMA
    LatentWalk walk(st);
    LatentPiece p;
    uint32_t qi = 0, quse = 0;
    while (ok && walk.next(sh, seq_lens, cu_seqlens, nr, KT, kLead, &p)) {
      if (quse > 0) ok = __all_sync(kAll, mbar_wait(&bar.q_empty[qi], (quse - 1) & 1, limit));
      if (!ok) break;
      if (elect_one()) {
        mbar_arrive_expect_tx(&bar.q_full[qi], pl.q_bytes);
        tma_load_4d(sq + qi * pl.q_bytes, &q_map, 0, (int)p.row0, 0, 0, &bar.q_full[qi]);
      }
      __syncwarp();
      if (++qi == (uint32_t)pl.nq) {
        qi = 0;
        ++quse;
      }
    }
    const bool bad = named_bar_or(2, kTcThreads, !ok);
    for (uint32_t i = 0; bad && i < (uint32_t)pl.nq; ++i) {
      const uint32_t uses = quse + (i < qi ? 1 : 0);
      if (uses) mbar_wait(&bar.q_full[i], (uses - 1) & 1, kDrainLimit);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------- the scores' MMAs
    // The whole warp runs the loop, one lane issues (see elect_one).
    const uint32_t id_qk = idesc_bf16(64, nr, false, false);
    // first descriptors.  The tile's groups of eight tokens lie `group` bytes apart, as the
    // rows of this operand; a K step is 32 bytes further in a chunk
    const uint64_t dq = desc_kmajor_sw128(smem_u32(sq), nr, 0);
    const uint64_t dk = smem_desc(smem_u32(ring), 16, pl.group, kSw128);
    LatentWalk walk(st);
    LatentPiece p;
    uint32_t t = 0, slot = 0, use = 0;                   // tiles
    uint32_t qi = 0, quse = 0;
    while (ok && walk.next(sh, seq_lens, cu_seqlens, nr, KT, kLead, &p)) {
      const uint64_t q0 = dq + (uint64_t)(qi * (pl.q_bytes / 16));
      ok = __all_sync(kAll, mbar_wait(&bar.q_full[qi], quse & 1, limit));
      for (int i = p.t0; i < p.t1 && ok; ++i, ++t) {
        const uint32_t sb = t % kSBuf;
        bool go = mbar_wait(&bar.full[slot], use & 1, limit);
        if (t >= kSBuf) go = go && mbar_wait(&bar.s_empty[sb], (t / kSBuf - 1) & 1, limit);
        ok = __all_sync(kAll, go);
        if (!ok) break;
        tc_fence_after();
        const uint32_t d = tb + kTmemS + sb * nr;
        const uint64_t k0 = dk + (uint64_t)(slot * (pl.tile_bytes / 16));
        if (elect_one()) {
          for (int c = 0; c < pl.nch; ++c) {
            const uint64_t a = k0 + (uint64_t)(c * 64), b = q0 + (uint64_t)(c * nr * 8);
            mma_ss_all(d, a, b, id_qk, c > 0);
#pragma unroll
            for (int e = 1; e < 4; ++e) mma_ss_all(d, a + 2 * e, b + 2 * e, id_qk, 1);
          }
          mma_commit(&bar.s_full[sb]);
          if (i == p.t1 - 1) mma_commit(&bar.q_empty[qi]);
        }
        __syncwarp();
        if (++slot == (uint32_t)pl.ntile) {
          slot = 0;
          ++use;
        }
      }
      if (++qi == (uint32_t)pl.nq) {
        qi = 0;
        ++quse;
      }
    }
    if (named_bar_or(2, kTcThreads, !ok)) {
      if (elect_one()) mma_commit(&bar.drain[0]);
      __syncwarp();
      mbar_wait(&bar.drain[0], 0, kDrainLimit);
    }
  } else if (warp == 12) {
    // ------------------------------------------------------------- the values' MMAs
    const uint32_t id_pv = idesc_bf16(128, nr, true, true);
    // the groups of eight tokens are the K index of this operand, a K step two groups; of P
    // 512 bytes
    const uint64_t dv = smem_desc(smem_u32(ring), 1024, pl.group, kSw128);
    const uint64_t dp = desc_mnmajor_sw32(smem_u32(sp), KT, 0);
    LatentWalk walk(st);
    LatentPiece p;
    uint32_t it = 0, slot = 0;                           // blocks; tile of the ring
    uint32_t pb = 0, puse = 0;
    while (ok && walk.next(sh, seq_lens, cu_seqlens, nr, KT, kLead, &p)) {
      for (int i = p.t0; i < p.t1; ++i) {
        bool go = mbar_wait(&bar.p_full[pb], puse & 1, limit);
        if (i == p.t0 && it > 0)                         // the block before has left O^T
          go = go && mbar_wait(&bar.o_empty, (it - 1) & 1, limit);
        ok = __all_sync(kAll, go);
        if (!ok) break;
        tc_fence_after();
        const uint64_t a0 = dv + (uint64_t)(slot * (pl.tile_bytes / 16));
        const uint64_t b0 = dp + (uint64_t)(pb * (pl.p_bytes / 16));
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < KK; ++k) {
            const uint64_t a = a0 + (uint64_t)(2 * k * (pl.group / 16));
            for (int j = 0; j < npair; ++j)
              mma_ss_all(tb + j * nr, a + (uint64_t)(j * 128), b0 + 32 * k, id_pv, k > 0 || i > p.t0);
            mma_commit(&bar.empty[slot][k]);
          }
          mma_commit(&bar.pv_done[pb]);
        }
        __syncwarp();
        if (++slot == (uint32_t)pl.ntile) slot = 0;
        if (++pb == (uint32_t)pl.np) {
          pb = 0;
          ++puse;
        }
      }
      ++it;
    }
    if (named_bar_or(2, kTcThreads, !ok)) {
      if (elect_one()) mma_commit(&bar.drain[1]);
      __syncwarp();
      mbar_wait(&bar.drain[1], 0, kDrainLimit);
    }
  } else {
    // ------------------------------------------------------------- softmax and results
    constexpr int kG = NR / 16;                          // groups of eight rows of a half
    const int wq = warp & 3, half = (warp - 4) >> 2, ts = tid - 128;
    const int g0 = half * kG;
    const int tok = 16 * wq + (lane >> 2), c0 = 2 * (lane & 3);   // tokens tok, tok + 8
    const bool act = 16 * wq < KT;                       // the quarter has tokens
    const uint32_t tl = tb + ((uint32_t)(32 * wq) << 16);
    const float c = sh.scale * kLog2e;
    LatentWalk walk(st);
    LatentPiece p;
    uint32_t g = 0, pb = 0, puse = 0;                    // tiles; next P buffer
    bool dead = false;
    // PV of the tile `back` tiles ago is done
    auto pv_wait = [&](uint32_t back) {
      const uint32_t t = g - back;
      return mbar_wait(&bar.pv_done[pl.np == 2 ? t & 1 : 0], (pl.np == 2 ? t >> 1 : t) & 1, limit);
    };
    while (!dead && walk.next(sh, seq_lens, cu_seqlens, nr, KT, kLead, &p)) {
      const int low = p.start + p.row_in_seq / sh.H + 1; // the first row's limit, the least
      if (ts < nr) {                                     // rows behind the block: no weight at all
        s_m[ts] = ts < p.rows ? kNone : INFINITY;
        s_more[ts] = (uint8_t)((p.row_in_seq + ts) / sh.H - p.row_in_seq / sh.H);
      }
      float l[kG][2], m[kG][2];                          // of this thread's rows
      named_bar(1, kSoft);
#pragma unroll
      for (int i = 0; i < kG; ++i) {
        l[i][0] = l[i][1] = 0.f;
        m[i][0] = s_m[8 * (g0 + i) + c0];
        m[i][1] = s_m[8 * (g0 + i) + c0 + 1];
      }
      for (int t = p.t0; t < p.t1; ++t, ++g) {
        const uint32_t sb = kSBuf == 2 ? g & 1 : 0;
        ok = ok && mbar_wait(&bar.s_full[sb], (kSBuf == 2 ? g >> 1 : g) & 1, limit);
        tc_fence_after();
        const bool mixed = (t + 1) * KT > low;
        uint32_t s[kG][4];
        if (act) {
#pragma unroll
          for (int i = 0; i < kG; ++i) tmem_ld_16x256b(tl + kTmemS + sb * nr + 8 * (g0 + i), s[i]);
          tmem_wait_ld();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.s_empty[sb]);
        // whether some scaled score passes its row's maximum by 2^8
        float top = -INFINITY;
        if (act && mixed) {
#pragma unroll
          for (int i = 0; i < kG; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (t * KT + tok + 8 * (e >> 1) >= low + s_more[8 * (g0 + i) + c0 + (e & 1)])
                s[i][e] = 0xff800000u;                   // -inf
        }
        if (act) {
#pragma unroll
          for (int i = 0; i < kG; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              top = fmaxf(top, fmaf(__uint_as_float(s[i][e]), c, -m[i][e & 1]));
        }
        // rows that some query row does not see: nothing that 0 * would turn into a NaN
        if (mixed) {
          const int first = max(low - t * KT, 0), per = sh.rank / 8;
          uint8_t* const tile = ring + g % pl.ntile * pl.tile_bytes;
          for (int i = ts; i < (KT - first) * per; i += kSoft) {
            const int k = first + i / per, c8 = i % per;
            uint4* w = reinterpret_cast<uint4*>(tile + (k >> 3) * pl.group + (c8 >> 3) * 1024 +
                                                (k & 7) * 128 + (c8 & 7) * 16);
            const uint4 a = *w;
            const uint4 b = make_uint4(zero_bad(a.x), zero_bad(a.y), zero_bad(a.z), zero_bad(a.w));
            if (a.x != b.x || a.y != b.y || a.z != b.z || a.w != b.w) *w = b;
          }
        }
        if (named_bar_or(1, kSoft, top > 8.f || !ok)) {
          // a maximum that passed (the first tile's always): weights, sums and O^T go to the
          // maxima of now
          auto maxima = [&](bool with) {                 // with: those of another quarter
#pragma unroll
            for (int i = 0; i < kG; ++i) {
              float a = fmaxf(__uint_as_float(s[i][0]), __uint_as_float(s[i][2]));
              float b = fmaxf(__uint_as_float(s[i][1]), __uint_as_float(s[i][3]));
#pragma unroll
              for (int o = 4; o < 32; o <<= 1) {
                a = fmaxf(a, __shfl_xor_sync(kAll, a, o));
                b = fmaxf(b, __shfl_xor_sync(kAll, b, o));
              }
              float* d = s_red + (wq & 1) * nr + 8 * (g0 + i) + c0;
              if (lane < 4) {
                d[0] = with ? fmaxf(a, d[0]) : a;
                d[1] = with ? fmaxf(b, d[1]) : b;
              }
            }
          };
          if (wq < 2) maxima(false);
          named_bar(1, kSoft);
          if (wq >= 2 && act) maxima(true);
          named_bar(1, kSoft);
          if (ts < nr) {
            const float mo = s_m[ts];
            const float mn = fmaxf(mo, c * fmaxf(s_red[ts], s_red[nr + ts]));
            s_row[ts] = mo == mn ? 1.f : ex2(mo - mn);
            s_m[ts] = mn;
          }
          if (t > p.t0) ok = ok && pv_wait(1);           // the tiles before have been added
          if (named_bar_or(1, kSoft, !ok)) { dead = true; break; }
#pragma unroll
          for (int i = 0; i < kG; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              l[i][e] *= s_row[8 * (g0 + i) + c0 + e];
              m[i][e] = s_m[8 * (g0 + i) + c0 + e];
            }
          if (t > p.t0) {
            tc_fence_after();
            for (int j = half; j < npair; j += 2)
#pragma unroll 1
              for (int i = 0; i < nr; i += 16) {
                uint32_t o[16];
                tmem_ld16(tl + j * nr + i, o);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; ++e)
                  o[e] = __float_as_uint(__uint_as_float(o[e]) * s_row[i + e]);
                tmem_st16(tl + j * nr + i, o);
              }
            tmem_wait_st();
            tc_fence_before();
          }
        }
        if (puse > 0) ok = ok && pv_wait(pl.np);         // the buffer's last values are done
        if (act) {
          uint32_t pk[kG][2];                              // rows c0, c0 + 1 of tokens tok, tok + 8
#pragma unroll
          for (int i = 0; i < kG; ++i) {
            float x[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              x[e] = ex2(fmaf(__uint_as_float(s[i][e]), c, -m[i][e & 1]));
            l[i][0] += x[0] + x[2];
            l[i][1] += x[1] + x[3];
            pk[i][0] = pack_bf16(x[0], x[1]);
            pk[i][1] = pack_bf16(x[2], x[3]);
          }
          // to shared memory two groups of rows at once: lane 8 k + j addresses row j of matrix k,
          // tokens [8 (k % 2), + 8) of group i + k / 2
          const uint32_t pr = smem_u32(sp + pb * pl.p_bytes);
          const uint32_t at = 16 * wq + (lane & 15);
#pragma unroll
          for (int i = 0; i + 1 < kG; i += 2)
            stmatrix_x4(pr + chunk_mnmajor_sw32(g0 + i + (lane >> 4), at, KT), pk[i][0],
                        pk[i][1], pk[i + 1][0], pk[i + 1][1]);
          if (kG & 1)
            stmatrix_x2(pr + chunk_mnmajor_sw32(g0 + kG - 1, at, KT), pk[kG - 1][0],
                        pk[kG - 1][1]);
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.p_full[pb]);
        if (++pb == (uint32_t)pl.np) {
          pb = 0;
          ++puse;
        }
      }
      if (dead) break;
      // ---- results: whole blocks to the output, shared ones to a partial slot
      const bool first = p.t0 == 0, last = p.t1 == p.tiles;
      const int slot = first && last ? -1 : 2 * (int)blockIdx.x + (first ? 1 : 0);
      auto sums = [&](bool with) {
#pragma unroll
        for (int i = 0; i < kG; ++i) {
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) {
            l[i][0] += __shfl_xor_sync(kAll, l[i][0], o);
            l[i][1] += __shfl_xor_sync(kAll, l[i][1], o);
          }
          float* d = s_red + (wq & 1) * nr + 8 * (g0 + i) + c0;
          if (lane < 4) {
            d[0] = with ? l[i][0] + d[0] : l[i][0];
            d[1] = with ? l[i][1] + d[1] : l[i][1];
          }
        }
      };
      if (wq < 2) sums(false);
      named_bar(1, kSoft);
      if (wq >= 2 && act) sums(true);
      ok = ok && pv_wait(1);
      if (named_bar_or(1, kSoft, !ok)) { dead = true; break; }
      if (ts < nr) {
        const float z = s_red[ts] + s_red[nr + ts];
        s_row[ts] = z == 0.f ? 0.f : 1.0f / z;
        const float y = z == 0.f ? -INFINITY : s_m[ts] * kLn2 + logf(z);
        if (slot >= 0) pt.lse[slot * nr + ts] = y;
        else if (lse && ts < p.rows) lse[p.row0 + ts] = y;
      }
      if (slot >= 0 && first && ts == 0)
        pt.head[blockIdx.x] =
            make_int4((int)p.row0, p.rows, latent_cta_of(p.end, st.W, st.G), 0);
      named_bar(1, kSoft);
      tc_fence_after();
      // 16 rows a load, the next one's under the stores: each stores 32 columns of a row a warp
      uint32_t o[2][16];
      int fi = 0, fj = half, si = 0, sj = half;          // row and columns of the next load, store
      auto step = [&](int& i, int& j) {
        i += 16;
        if (i >= p.rows) {
          i = 0;
          j += 2;
        }
      };
      auto fetch = [&](uint32_t (&v)[16]) {
        if (fj < npair) tmem_ld16(tl + fj * nr + fi, v);
        step(fi, fj);
      };
      auto put = [&](const uint32_t (&v)[16]) {
        const int i = si, d = 128 * sj + 32 * wq + lane, rows = min(p.rows - i, 16);
        step(si, sj);
        float f[16];
#pragma unroll
        for (int e = 0; e < 16; e += 4) {
          const float4 w = *reinterpret_cast<const float4*>(s_row + i + e);
          f[e] = __uint_as_float(v[e]) * w.x;
          f[e + 1] = __uint_as_float(v[e + 1]) * w.y;
          f[e + 2] = __uint_as_float(v[e + 2]) * w.z;
          f[e + 3] = __uint_as_float(v[e + 3]) * w.w;
        }
        if (slot < 0) {
          bf16* y = out + (p.row0 + i) * sh.rank + d;
#pragma unroll
          for (int e = 0; e < 16; ++e, y += sh.rank)
            if (e < rows) *y = __float2bfloat16_rn(f[e]);
        } else {
          float* y = pt.o + ((long long)slot * nr + i) * sh.rank + d;
#pragma unroll
          for (int e = 0; e < 16; ++e, y += sh.rank)
            if (e < rows) *y = f[e];
        }
      };
      fetch(o[0]);
#pragma unroll 1
      while (sj < npair) {
        tmem_wait_ld();
        fetch(o[1]);
        put(o[0]);
        if (sj >= npair) break;
        tmem_wait_ld();
        fetch(o[0]);
        put(o[1]);
      }
      tc_fence_before();
      named_bar(1, kSoft);                               // the block's rows are done with
      if (lane == 0) mbar_arrive(&bar.o_empty);
    }
    // what is left undone when a wait has given up is NaN, not what the memory held before
    if (dead) {
      const float bad = __uint_as_float(0x7fffffffu);
      do {
        const bool first = p.t0 == 0;
        if (first && p.t1 == p.tiles) {
          if (lse && ts < p.rows) lse[p.row0 + ts] = bad;
          for (int i = ts; i < p.rows * sh.rank; i += kSoft)
            out[p.row0 * sh.rank + i] = __float2bfloat16_rn(bad);
        } else {                                           // by the join's weight of it
          if (ts < nr) pt.lse[(2 * (int)blockIdx.x + (first ? 1 : 0)) * nr + ts] = bad;
          if (first && ts == 0)
            pt.head[blockIdx.x] =
                make_int4((int)p.row0, p.rows, latent_cta_of(p.end, st.W, st.G), 0);
        }
      } while (walk.next(sh, seq_lens, cu_seqlens, nr, KT, kLead, &p));
    }
    named_bar_or(2, kTcThreads, !ok);
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

using TcKernel = void (*)(CUtensorMap, CUtensorMap, const int32_t*, const int32_t*,
                          const int32_t*, bf16*, float*, LatentAttnShape, TcPlan, LatentPartials,
                          uint32_t);
TcKernel tc_kernel(int nr) {
  switch (nr) {
    case 16: return kda_latent_tc_kernel<16>;
    case 32: return kda_latent_tc_kernel<32>;
    case 48: return kda_latent_tc_kernel<48>;
    case 64: return kda_latent_tc_kernel<64>;
    case 80: return kda_latent_tc_kernel<80>;
    default: return kda_latent_tc_kernel<96>;
  }
}

// Rows of a block: all of a sequence's up to 64, a multiple of 16.  Up to 96: all of them, or, of
// few sequences, two blocks of 48: the CTAs then share a sequence by many, and what they
// write and join counts for more than reading the cache twice (on the device, 96 heads, 4000 to 8192
// tokens: 4 sequences 35 us against 42, 16 58 against 63, 24 78 against 77; 43 of up to 16384 160
// against 143; of 400 tokens 4 sequences 21 against 25, 16 23 against 27, of 50 19 against 23 and 21
// against 25).  Of more rows, 64, whose tiles of 64 tokens cost the MMAs less a row and token than
// 96 or 48 with tiles of 48 (a 1024-token chunk of 12 heads behind 8192 to 32768 tokens: 521 us
// against 537 and 573).
// Packed, a sequence has so many on average, which says little when one has most of them: from 1024
// rows on that are more than a token for each sequence, at least 48 (512 slots, all empty but for
// a 1024-token chunk of 12 heads behind 16384: 32 rows 804 us, 48 594, 64 553; 256 sequences of two
// tokens behind 4000, which the host cannot tell from it: 220, 233, 276).  Fewer tokens than sequences are
// a decode batch with empty slots: 16 rows of 12 heads 210 us, 48 222.
constexpr int kTcSkewRows = 1024;
int tc_rows(int N, int L, int T, int H) {
  const long long rows = L > 0 ? (long long)L * H : (((long long)T + N - 1) / N) * H;
  if (rows > kTcMaxRows) return 64;
  if (rows > 64 && N <= 16) return 48;
  if (L == 0 && rows < 48 && ((long long)T - N + 1) * H >= kTcSkewRows) return 48;
  return (int)((rows + 15) / 16 * 16);
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
                             cudaStream_t stream, uint32_t polls) {
  if (!once_per_device(kOnceLatentTc, []() {
        for (int nr = 16; nr <= kTcMaxRows; nr += 16)
          if (cudaFuncSetAttribute(tc_kernel(nr), cudaFuncAttributeMaxDynamicSharedMemorySize,
                                   (int)tc_smem(nr)) != cudaSuccess)
            return false;
        return true;
      }))
    return cudaErrorInvalidDevice;
  const int nr = tc_rows(sh.N, sh.L, sh.T, sh.H), G = latent_tc_ctas(sms);
  const TcPlan pl = tc_plan(nr, sh.rank, sh.rope);
  const LatentPartials pt = latent_partials(buf, G, nr);
  const uint64_t D = sh.rank + sh.rope;
  const uint64_t rows = (uint64_t)(sh.L > 0 ? (long long)sh.N * sh.L : sh.T) * sh.H;
  CUtensorMap q_map, c_map;
  if (!make_chunk_map_4d(&q_map, q, rows, D / 64, 1, D * 2, D * 2, (uint32_t)nr,
                         (uint32_t)(D / 64)) ||
      !make_chunk_map_4d(&c_map, cache, sh.page_size, D / 64, sh.num_pages, sh.row_stride * 2,
                         sh.page_stride * 2, 8, (uint32_t)(D / 64)))
    return cudaErrorInvalidValue;
  KDA_TIMED(KDA_KERNEL_LATENT_ATTN, stream,
            tc_kernel(nr)<<<G, kTcThreads, tc_smem(nr), stream>>>(
                q_map, c_map, page_table, seq_lens, cu_seqlens, static_cast<bf16*>(out), lse, sh,
                pl, pt, polls));
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  note_launches(1);
  return launch_latent_join(out, lse, pt, G, nr, sh, KDA_BF16, stream);
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
