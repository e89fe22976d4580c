// mass.cuh -- the accepted drafts of every sequence into the cache, and their
// attention weight added to the positions' sums, on the tcgen05 tensor cores.
//
//   mass_out[s] = mass_in[s] (0 for the new rows)
//               + sum over the accepted tokens' query rows r that see s of
//                 exp(q_r.k_s / 8 - lse_r)
//
// The scores are taken transposed, S^T = K Q^T: 128 positions are the tensor
// memory's lanes and the query rows its columns. A position's sum then runs
// along one thread's registers, there is neither a maximum nor a second
// product, and what a position past the end holds stays in its own lane. All
// query rows of a (sequence, group) stay in shared memory (up to 1152 of 128
// bytes) beside the ring of K blocks.
//
// Bounds: 128 bytes of K and 8 of mass a position; one exponential a (row,
// position), 16 a clock and SM on the MUFU, so that past about 90 rows the
// exponentials bind; one pair in kMassPolyEvery is evaluated on the FMA pipe.
// Measured, 8 groups: 8 x 6 accepted (one row a token; in one of the sequences
// none) over 20001 to 32767 positions 41.9 us = 4.9 TB/s of 6.5 that a copy reaches;
// 2 x 128 (two rows) over 60000 to 65536 128 us against 63 of exponentials on the
// MUFU alone: issue and latency. Sixteen softmax warps took 118 us there, but 58-60 instead of 50
// for 8 x 1 over 32767.
// Work is cut as in tree_umma.cuh: ranges of equal weight over all positions of
// the sequences that accept anything, one block per SM; up to 90 rows the groups side by
// side, so that a position's contiguous G rows are read at about the same time (with
// G = 32 or 64 on a multiple of G blocks, 128), above that one after the other.
//
//   warp 0      K blocks: the cache's by TMA; the accepted rows, the last block of
//               a unit, gathered
//   warps 1, 2  lane 0 issues the products of the even (odd) blocks
//   warp 3      the accepted rows into the cache
//   warps 4..11 query rows and lse into shared memory at a unit's start; then
//               exponentials and sums, one thread a position (warps 4..7 the
//               even blocks, 8..11 the odd)
// TMEM columns: 128 t + 256 buf .. + 127: scores of tile t, buffer buf.
#pragma once

#include "cache.cuh"
#include "sm100.cuh"
#include "tree_umma.cuh"

namespace gqe {

constexpr int kMassThreads = 384;
constexpr int kMassMaxStages = 8;  // of K; an even number is used, so that a stage's blocks are all one tile's
constexpr int kMassMaxRows = kTreeMax * 9;  // T * (k + 1)
// The polynomial is off by 2.7e-6 at most, the MUFU by 2e-7; the exponent itself,
// a difference of numbers between 8 and 32 in fp32, puts either off by 1e-6.
constexpr int kMassPolyEvery = 4;

struct MassParams {
  CUtensorMap tmK;  // the cache as [B*cap][G][64], box (64, 1, 128)
  CommitParams c;
  int nchunk;       // chunks of 128 query rows that fit, for T tokens
  int nstage;
  int step;         // G: the groups side by side; 1: ranges over all groups
};
struct MassSmem {
  static constexpr int kLse = 0;                                // [1152] -lse, log2 units
  static constexpr int kTok = kLse + kMassMaxRows * 4;          // [1152] place of the row's token in the path, -1: no token
  static constexpr int kOld = kTok + kMassMaxRows * 2;          // [4][256] sums so far
  static constexpr int kPrefix = kOld + 4096;                   // [B + 1]
  static constexpr int kBar = kPrefix + (kTreeMaxB + 1) * 8;
  static constexpr int kQ = (kBar + 512 + 1023) / 1024 * 1024;  // chunks of 16 KB, then the ring's stages of 16 KB
};
inline int mass_smem(int nchunk, int nstage) { return MassSmem::kQ + (nchunk + nstage) * 16384 + 1024; }

// Weight of a block of 128 positions against so many rows: the bytes' time up
// to about 90 rows, then the exponentials'.
__device__ __forceinline__ int mass_weight(int rows) { return rows > 90 ? rows : 90; }

struct MassItem {
  int b, g, L, n, R, nblk, j0, j1;
};
struct MassCursor {
  long long x0, x1, base;
  int b, g, only;
  __device__ __forceinline__ bool next(const CommitParams& p, MassItem& it) {
    while (b < p.B && base < x1) {
      commit_lens(p, b, it.L, it.n);
      if (it.n <= 0) {  // (nothing accepted: no weight, no unit in any role; mass_keep)
        ++b;
        g = only >= 0 ? only : 0;
        continue;
      }
      it.b = b;
      it.g = g;
      it.R = it.n * (p.k + (g == 0 ? 1 : 0));
      it.nblk = (it.L + kTuBlock - 1) / kTuBlock + 1;
      const int w = only >= 0 ? 1 : mass_weight(it.R);
      const long long a = x0 - base, e = x1 - base;
      it.j0 = a <= 0 ? 0 : (int)min((long long)it.nblk, (a + w - 1) / w);
      it.j1 = (int)min((long long)it.nblk, (e + w - 1) / w);
      base += (long long)it.nblk * w;
      if (only >= 0) {
        ++b;
      } else if (++g == p.G) {
        g = 0;
        ++b;
      }
      if (it.j0 < it.j1) return true;
    }
    return false;
  }
};

// A position's weights from N query rows, added to eight sums; nlse = -lse. With
// kFresh the position is the accepted token at `place`, seen from there on. (As
// a condition in one function the places' loads and comparisons were issued for
// every position, 4 of 9.5 instructions a score.)
// A weight that is zero (a token that does not see the place, -lse = -infinity of
// a row that is none) adds nothing: the MUFU gives 0, the polynomial what fadd2_ftz
// takes as 0. So do weights below 2^-126, wherever their row falls.
template <int N, bool kFresh>
__device__ __forceinline__ void mass_add(const uint32_t (&a)[N], const float* nlse, const int16_t* tok, float sl2, int place,
                                         float (&sum)[8]) {
#pragma unroll
  for (int i = 0; i < N / 4; ++i) {
    const float4 l4 = reinterpret_cast<const float4*>(nlse)[i];
    float x[4], y[4];
    ffma2(x[0], x[1], __uint_as_float(a[4 * i]), __uint_as_float(a[4 * i + 1]), sl2, sl2, l4.x, l4.y);
    ffma2(x[2], x[3], __uint_as_float(a[4 * i + 2]), __uint_as_float(a[4 * i + 3]), sl2, sl2, l4.z, l4.w);
    if constexpr (kFresh) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (place > tok[4 * i + e]) x[e] = -INFINITY;
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      if (!kFresh && (2 * i + e) % kMassPolyEvery == kMassPolyEvery - 1) {
        exp2_poly4(y[2 * e], y[2 * e + 1], x[2 * e], x[2 * e + 1]);
      } else {
        y[2 * e] = ex2_approx(x[2 * e]);
        y[2 * e + 1] = ex2_approx(x[2 * e + 1]);
      }
    }
    const int s = (4 * i) & 7;
    fadd2_ftz(sum[s], sum[s + 1], sum[s], sum[s + 1], y[0], y[1]);
    fadd2_ftz(sum[s + 2], sum[s + 3], sum[s + 2], sum[s + 3], y[2], y[3]);
  }
}

// Sequences that accept nothing keep their sums: where those go to another
// buffer, all blocks of threads copy them, a piece of 1024 positions of one
// (sequence, group) at a time, by the 256 threads that would add. Nothing of such
// a sequence goes through the barriers: a unit without query rows would have its
// summing threads wait for no product, and run phases ahead of the threads that
// issue them.
__device__ __forceinline__ void mass_keep(const CommitParams& p, const long long* prefix, int wtid) {
  constexpr int kPiece = 1024;
  const int lane = wtid & 31;
  for (int b0 = 0; b0 < p.B; b0 += 32) {
    const int b = b0 + lane;
    int L = 0, n = -1;
    if (b < p.B && prefix[b + 1] == prefix[b]) commit_lens(p, b, L, n);
    const int pieces = n == 0 ? (L + kPiece - 1) / kPiece : 0;  // of each group
    int sum = pieces * p.G;                                     // below 2^31 over a warp: B * cap * G / 1024
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const int o = __shfl_up_sync(0xffffffffu, sum, d);
      if (lane >= d) sum += o;
    }
    const int total = __shfl_sync(0xffffffffu, sum, 31);
    for (int i = blockIdx.x; i < total; i += gridDim.x) {
      const int at = __popc(__ballot_sync(0xffffffffu, sum <= i));  // the lane whose sequence it is
      const int len = __shfl_sync(0xffffffffu, L, at), each = __shfl_sync(0xffffffffu, pieces, at);
      const int r = i - (__shfl_sync(0xffffffffu, sum, at) - each * p.G);
      const size_t row = ((size_t)(b0 + at) * p.G + r / each) * p.cap;
      const int s = r % each * kPiece + wtid;
      float v[kPiece / 256];
#pragma unroll
      for (int u = 0; u < kPiece / 256; ++u)
        if (s + u * 256 < len) v[u] = p.mass_in[row + s + u * 256];
#pragma unroll
      for (int u = 0; u < kPiece / 256; ++u)
        if (s + u * 256 < len) p.mass_out[row + s + u * 256] = v[u];
    }
  }
}

__global__ void __launch_bounds__(kMassThreads, 1) cache_mass_kernel(const __grid_constant__ MassParams P) {
  using S = MassSmem;
  const CommitParams& p = P.c;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + S::kBar);  // [kMassMaxStages]
  uint64_t* k_empty = k_full + kMassMaxStages;                     // [kMassMaxStages]
  uint64_t* q_full = k_empty + kMassMaxStages;                     // all rows and lse of a unit are there
  uint64_t* q_free = q_full + 1;                                   // both tiles are done with a unit
  uint64_t* q_tile = q_free + 1;                                   // [2] as q_full, of the units with a block of the tile
  uint64_t* s_full = q_tile + 2;                                   // [2 tiles][2 buffers]
  uint64_t* s_free = s_full + 4;                                   // [2][2]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(s_free + 4);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* s_nan = reinterpret_cast<int*>(tmem_slot + 2);              // [2] units: a row's weights are NaN
  float* s_nlse = reinterpret_cast<float*>(smem + S::kLse);
  float* s_old = reinterpret_cast<float*>(smem + S::kOld);
  int16_t* s_tok = reinterpret_cast<int16_t*>(smem + S::kTok);
  long long* prefix = reinterpret_cast<long long*>(smem + S::kPrefix);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int s = 0; s < kMassMaxStages; ++s) {
      mbar_init(&k_full[s], 1);
      mbar_init(&k_empty[s], 1);
    }
    mbar_init(q_full, 256);
    mbar_init(q_free, 256);
    mbar_init(&q_tile[0], 256);
    mbar_init(&q_tile[1], 256);
    for (int i = 0; i < 4; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_free[i], 128);
    }
    *abort_flag = 0;
    s_nan[0] = s_nan[1] = 0;
    fence_mbar_init();
    tma_prefetch_desc(&P.tmK);
  }
  if (warp == 1) tmem_alloc(tmem_slot, 512);
  pdl_wait();
  pdl_trigger();
  {
    if (tid == 0) prefix[0] = 0;
    for (int b = tid; b < p.B; b += kMassThreads) {
      int L, n;
      commit_lens(p, b, L, n);
      long long w = 0;
      if (n > 0) {
        w = (L + kTuBlock - 1) / kTuBlock + 1;
        if (P.step == 1) w *= mass_weight(n * (p.k + 1)) + (long long)(p.G - 1) * mass_weight(n * p.k);
      }
      prefix[b + 1] = w;
    }
    __syncthreads();
    scan_prefix<kMassThreads>(prefix, p.B);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const uint32_t sbase = smem_u32(smem);
  const long long total = prefix[p.B];
  const int ranges = gridDim.x / P.step, cta = blockIdx.x;
  const int range = min(cta / P.step, ranges);
  MassCursor cur;
  cur.x0 = tree_range(total, range, ranges);
  cur.x1 = tree_range(total, min(range + 1, ranges), ranges);
  cur.b = tree_first(prefix, p.B, cur.x0);
  cur.base = prefix[cur.b];
  cur.only = P.step > 1 ? cta % P.step : -1;
  cur.g = max(cur.only, 0);
  MassItem it = {};
  const uint32_t ring = S::kQ + P.nchunk * 16384;

  if (warp == 0) {
    // ---- K blocks, in order: the cache's by TMA, the accepted rows gathered ---------
    uint32_t kv = 0;
    bool ok = true;
    while (ok && cur.next(p, it)) {
      for (int j = it.j0; j < it.j1; ++j, ++kv) {
        const int s = kv % P.nstage;
        ok = mbar_wait(&k_empty[s], ((kv / P.nstage) & 1) ^ 1, abort_flag);
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        if (j < it.nblk - 1) {
          if (lane == 0) {
            mbar_arrive_expect_tx(&k_full[s], 16384);
            tma_load_3d(smem + ring + s * 16384, &P.tmK, &k_full[s], 0, it.g, it.b * p.cap + j * kTuBlock);
          }
          continue;
        }
        // eight lanes a row; rows past the last are left as they are (a lane of S^T
        // that is not stored)
        for (int i = lane >> 3; i < it.n; i += 4) {
          const int tok = commit_token(p, it.b, i);
          uint4 v = make_uint4(0u, 0u, 0u, 0u);
          if (tok >= 0) v = reinterpret_cast<const uint4*>(p.Kn + (((size_t)it.b * p.T + tok) * p.G + it.g) * 64)[lane & 7];
          *reinterpret_cast<uint4*>(smem + ring + s * 16384 + i * 128 + (((lane & 7) ^ (i & 7)) << 4)) = v;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&k_full[s]);
      }
    }
  } else if (warp <= 2) {
    if (lane == 0) {
      const int t = warp - 1;
      uint32_t kv = 0, q_cnt = 0, s_cnt = 0;
      bool ok = true;
      while (ok && cur.next(p, it)) {
        const int nj = it.j1 - it.j0;
        // block kv + jj belongs to tile (kv + jj) % 2, so that the tiles take
        // turns across units too. (q_tile counts the units that have a block of
        // the tile: in the others neither side waits for the other, and their
        // phases could drift apart.)
        if ((int)((kv & 1) ^ t) < nj) {
          if (!(ok = mbar_wait(&q_tile[t], q_cnt & 1, abort_flag))) break;
          ++q_cnt;
        }
        tc_fence_after();
        for (int jj = (kv & 1) ^ t; ok && jj < nj; jj += 2) {
          const uint32_t kvj = kv + jj;
          const int s = kvj % P.nstage;
          if (!(ok = mbar_wait(&k_full[s], (kvj / P.nstage) & 1, abort_flag))) break;
          tc_fence_after();
          const uint32_t ka = sbase + ring + s * 16384;
          for (int r0 = 0; r0 < it.R; r0 += 128, ++s_cnt) {
            const int buf = s_cnt & 1;
            if (!(ok = mbar_wait(&s_free[t * 2 + buf], ((s_cnt >> 1) & 1) ^ 1, abort_flag))) break;
            tc_fence_after();
            const int cols = min(128, (it.R - r0 + 15) & ~15);
            const uint32_t idesc = idesc_bf16(128, 16, false, false) + ((uint32_t)((cols >> 3) - 2) << 17);
            const uint32_t qa = sbase + S::kQ + (r0 >> 7) * 16384;
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              umma_ss(tmem_base + buf * 256 + t * 128, sdesc_sw128(ka + kk * 32, 16, 1024),
                      sdesc_sw128(qa + kk * 32, 16, 1024), idesc, kk != 0);
            umma_commit(&s_full[t * 2 + buf]);
          }
          umma_commit(&k_empty[s]);
        }
        kv += nj;
      }
    }
  } else if (warp == 3) {
    // ---- (sequence, place of the path) pairs, over all blocks -------------------------
    for (int i = cta; i < p.B * p.T; i += gridDim.x) {
      int L, n;
      const int b = i / p.T, j = i % p.T;
      commit_lens(p, b, L, n);
      commit_append_row(p, b, j, L, n, lane, 32);
    }
  } else {
    const int t = (warp - 4) >> 2, q = warp & 3;
    const int row = q * 32 + lane;      // position of the block
    const int wtid = tid - 128;         // of the 256
    const uint32_t tm = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + t * 128;
    uint32_t kv = 0, units = 0, s_cnt = 0;
    bool ok = true;
    while (ok && cur.next(p, it)) {
      // the unit's query rows, once neither tile multiplies by the ones before
      bool w_ok = units == 0 || mbar_wait(q_free, (units - 1) & 1, abort_flag);
      if (!__all_sync(0xffffffffu, w_ok)) { ok = false; break; }
      const int Rp = (it.R + 15) & ~15;
      for (int i = wtid; i < Rp * 8; i += 256) {
        const int r = i >> 3, ch = i & 7;
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        const int j = r < it.R ? tree_row_token(r, it.n, p.k) : -1;
        const int tok = j >= 0 ? commit_token(p, it.b, j) : -1;
        size_t qrow = 0;
        if (tok >= 0) {
          qrow = ((size_t)it.b * p.T + tok) * p.Ha + tree_row_slot(r, it.n, it.g, p.k, p.G);
          v = reinterpret_cast<const uint4*>(p.Q + qrow * 64)[ch];
        }
        *reinterpret_cast<uint4*>(smem + S::kQ + (r >> 7) * 16384 + (r & 127) * 128 + ((ch ^ (r & 7)) << 4)) = v;
        if (ch == 0) {
          const float ls = tok >= 0 ? p.lse[qrow] * -1.4426950408889634f : -INFINITY;  // (no row: every weight is 0)
          // NaN, or +infinity where all of the row's scores are -infinity: every
          // cached position's sum is NaN (the polynomial would lose it)
          if (!(ls < INFINITY)) s_nan[units & 1] = 1;
          s_nlse[r] = ls;
          s_tok[r] = (int16_t)(tok >= 0 ? j : -1);
        }
      }
      fence_proxy_async_smem();
      const int nj = it.j1 - it.j0;
      if ((int)(kv & 1) < nj) mbar_arrive(&q_tile[0]);
      if ((int)((kv & 1) ^ 1) < nj) mbar_arrive(&q_tile[1]);
      mbar_arrive(q_full);
      w_ok = mbar_wait(q_full, units & 1, abort_flag);  // lse of the other warps
      if (!__all_sync(0xffffffffu, w_ok)) { ok = false; break; }
      const float nan = s_nan[units & 1] ? __int_as_float(0x7fffffff) : 0.f;
      if (wtid == 0) s_nan[(units + 1) & 1] = 0;
      const size_t at = ((size_t)it.b * p.G + it.g) * p.cap;
      // a position's sum so far comes into shared memory three of the tile's blocks
      // ahead, each thread its own (in registers the move from one block's to the
      // next's waited for the load: 1200 of 2200 cycles a block)
      auto fetch_old = [&](int jj, uint32_t slot) {
        const int j = it.j0 + jj;
        const bool in = jj < nj && j < it.nblk - 1 && j * kTuBlock + row < it.L;
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(&s_old[(slot & 3) * 256 + wtid])),
                     "l"(p.mass_in + at + (in ? j * kTuBlock + row : 0)), "r"(in ? 4 : 0)
                     : "memory");
        asm volatile("cp.async.commit_group;" ::: "memory");
      };
      uint32_t slot = 0;
#pragma unroll
      for (int i = 0; i < 3; ++i) fetch_old((int)((kv & 1) ^ t) + 2 * i, i);
      for (int jj = (kv & 1) ^ t; jj < nj; jj += 2) {
        const int j = it.j0 + jj;
        const bool fresh = j == it.nblk - 1;  // the accepted rows
        const int s0 = fresh ? it.L : j * kTuBlock, valid = fresh ? it.n : min(kTuBlock, it.L - s0);
        fetch_old(jj + 6, slot + 3);
        asm volatile("cp.async.wait_group 3;" ::: "memory");
        const float old = s_old[(slot & 3) * 256 + wtid];
        ++slot;
        // (of the accepted rows only those that its token sees: MUFU, which keeps it)
        float sum[8] = {fresh ? 0.f : nan, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        for (int r0 = 0; r0 < it.R; r0 += 128, ++s_cnt) {
          const int buf = s_cnt & 1;
          w_ok = mbar_wait(&s_full[t * 2 + buf], (s_cnt >> 1) & 1, abort_flag);
          if (!__all_sync(0xffffffffu, w_ok)) { ok = false; break; }
          tc_fence_after();
          const int cols = min(128, Rp - r0);
          if (q * 32 < valid) {
            int c0 = 0;
            if (fresh) {
              for (; c0 < cols; c0 += 16) {
                uint32_t a[16];
                tmem_ld16(tm + buf * 256 + c0, a);
                mass_add<16, true>(a, s_nlse + r0 + c0, s_tok + r0 + c0, p.scale_log2, row, sum);
              }
            }
            for (; c0 + 64 <= cols; c0 += 64) {
              uint32_t a[64];
              tmem_ld64(tm + buf * 256 + c0, a);
              mass_add<64, false>(a, s_nlse + r0 + c0, nullptr, p.scale_log2, 0, sum);
            }
            for (; c0 < cols; c0 += 16) {
              uint32_t a[16];
              tmem_ld16(tm + buf * 256 + c0, a);
              mass_add<16, false>(a, s_nlse + r0 + c0, nullptr, p.scale_log2, 0, sum);
            }
          }
          tc_fence_before();
          mbar_arrive(&s_free[t * 2 + buf]);
        }
        if (!ok) break;
        if (row < valid) {
          float w = ((sum[0] + sum[1]) + (sum[2] + sum[3])) + ((sum[4] + sum[5]) + (sum[6] + sum[7]));
          // a place whose path index is out of range holds no token (its key here is zero)
          if (fresh && s_tok[row * p.k] < 0) w = 0.f;
          p.mass_out[at + s0 + row] = old + w;
        }
      }
      asm volatile("cp.async.wait_group 0;" ::: "memory");
      if (!ok) break;
      mbar_arrive(q_free);
      ++units;
      kv += nj;
    }
    if (ok && p.mass_out != p.mass_in) mass_keep(p, prefix, wtid);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (*abort_flag) {
    const unsigned long long t0n = globaltimer_ns();
    while (globaltimer_ns() - t0n < 100000ull) {}
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, 512);
  }
}

}  // namespace gqe
