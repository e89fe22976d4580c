// tree_umma.cuh -- attention of a tree of drafted tokens over a key/value cache
// on the tcgen05 tensor cores (the mathematics: tree.cuh).
//
// Units. The query rows of one (sequence, group) are cut into units of up to
// 256 rows, two tiles of 128. A unit's keys are its cached blocks of 128
// positions and one block of drafted tokens. All units' blocks, one after the
// other, are cut into gridDim.x ranges of equal weight, one persistent block of
// threads (one per SM) each: whatever the lengths and however few the
// sequences, every SM streams the same share. A unit that a range's end cuts is
// left as partial (m, l, O) rows for tree_umma_merge_kernel, at most two of
// them per range; the others are written at once.
//
// Inside a unit two tiles A and B run side by side, each with its MMA thread
// and its four softmax warps:
//   a unit of more than 128 rows   A and B hold its two row tiles, and every
//                                  K/V block serves both;
//   else                           A and B hold the same rows and take the
//                                  blocks in turn, A the even, B the odd ones,
//                                  and are added at the end.
// A pair block costs half again what a block of the second kind does (weights 3
// and 2): it is bound by exponentials, the other by the cache's bytes.
//
//   warp 0      TMA producer: K/V blocks through a ring of kTuStages
//   warps 1, 2  lane 0 issues the MMAs of tile A (warp 1, also the TMEM owner)
//               or B: S = Q K^T (SS, 128x128x64) and O += P V (TS, N = 64)
//   warp 3      for a unit's draft block: the ancestor masks, by pointer
//               doubling, and which drafted values are not finite
//   warps 4..11 softmax, one thread a row: Q into shared memory at the start of
//               a unit; then per block S from TMEM, the running maximum
//               (rescaled lazily) and sum, P as bf16 into TMEM
// What a masked row holds is kept out in three places: masked scores are
// replaced, not added to; value rows past the last valid one are zeroed before
// P V; drafted values that are not finite are zeroed too, and added at the end
// to the rows that see them.
// TMEM columns: S_A [0,128) S_B [128,256) O_A [256,320) O_B [320,384)
//               P_A [384,448) P_B [448,512).
#pragma once

#include "attn2.cuh"
#include "sm100.cuh"
#include "tree.cuh"

namespace gqe {

constexpr int kTuStages = 5;
constexpr int kTuThreads = 384;
constexpr int kTuRegsLow = 88, kTuRegsHigh = 208;  // 88*128 + 208*256 = 168*384
constexpr int kTuMaxB = 1024;                      // B * G * M <= 8192 and G * M >= 8
constexpr int kTuBlock = 128;                      // keys of a block
constexpr int kTuRows = 256;                       // rows of a unit
constexpr int kTuPolyEvery = 8;  // every n-th pair of exponentials on the FMA pipe (as in attn2.cuh)

struct TreeUmmaParams {
  CUtensorMap tmK, tmV;    // caches as [B*cap][G][64], box (64, 1, 128)
  CUtensorMap tmKn, tmVn;  // drafts as [B*T][G][64]
  TreeParams p;            // part_ml, part_o: [2 * gridDim.x][prow] rows
  int2* unit_cta;          // [units] first and last range that holds blocks of the unit
  int u0, u1;              // units of group 0 and of each other group, for T tokens
  int prow;                // rows a part holds, the most that a unit has
};

struct TuSmem {
  static constexpr int kQ = 0;                               // Q_A, Q_B
  static constexpr int kKV = 32768;                          // stages of K, V
  static constexpr int kMask = kKV + kTuStages * 32768;      // [2][128] ancestor masks
  static constexpr int kUp = kMask + 2 * kTreeMax * 16;      // [128] pointers of the doubling
  static constexpr int kBad = kUp + kTreeMax * 4;            // [2][4] drafts with values that are not finite
  static constexpr int kML = kBad + 32;                      // [2][128] m, l of the tiles
  static constexpr int kPrefix = kML + 2 * 128 * 8;          // [B + 1] weight before each sequence
  static constexpr int kBar = kPrefix + (kTuMaxB + 1) * 8;
  static constexpr int kBytes = kBar + 512 + 1024;
};

struct TuItem {
  int b, g, s;         // sequence, group, unit of the group
  int L, n, R;         // cached positions, drafted tokens, rows of the group
  int rows;            // rows of the unit
  bool pair;           // two row tiles
  int nblk, j0, j1;    // blocks of the unit; this range's
  int unit;
  __device__ __forceinline__ int tile_blocks(int t) const {
    if (pair) return j1 - j0;
    return (j1 - j0 + 1 - t) >> 1;
  }
  __device__ __forceinline__ bool owns(int t, int jj) const { return pair || (jj & 1) == t; }
  __device__ __forceinline__ int row_base(int t) const { return s * kTuRows + (pair ? t * 128 : 0); }
  __device__ __forceinline__ bool has_drafts() const { return j1 == nblk; }
  __device__ __forceinline__ bool whole() const { return j0 == 0 && j1 == nblk; }
};

__device__ __forceinline__ int tu_weight(int rows) {  // of one block of a unit of so many rows
  return rows > 128 ? 3 : 2;
}
__device__ __forceinline__ long long tu_group_weight(int R) {
  const int full = R / kTuRows, rest = R % kTuRows;
  return (long long)full * 3 + (rest ? tu_weight(rest) : 0);
}
__device__ __forceinline__ long long tu_seq_weight(int L, int n, int G, int k) {
  if (n == 0) return 0;
  const long long nblk = (L + kTuBlock - 1) / kTuBlock + 1;
  return nblk * (tu_group_weight(n * (k + 1)) + (long long)(G - 1) * tu_group_weight(n * k));
}
__device__ __forceinline__ long long tu_range(long long total, int c, int grid) { return total * c / grid; }
__device__ __forceinline__ int tu_range_of(long long total, int grid, long long x) {
  return (int)(((x + 1) * grid - 1) / total);
}

// The units that a range of weight [x0, x1) holds blocks of, in order. A block
// belongs to the range that its first weight falls into.
struct TuCursor {
  long long x0, x1, base;
  int b, g, s;
  __device__ __forceinline__ void start(const TreeParams& p, const long long* prefix, long long a, long long e) {
    x0 = a;
    x1 = e;
    int lo = 0, hi = p.B - 1;  // the last sequence that begins at or before x0
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (prefix[mid] <= x0) lo = mid; else hi = mid - 1;
    }
    b = lo;
    g = s = 0;
    base = prefix[lo];
    int L, n;
    tree_lens(p.cache_len, p.draft_len, b, p.cap, p.T, L, n);
    if (n > 0 && p.G > 1) {  // straight to the group
      const long long nblk = (L + kTuBlock - 1) / kTuBlock + 1;
      const long long w0 = nblk * tu_group_weight(n * (p.k + 1)), w1 = nblk * tu_group_weight(n * p.k);
      if (x0 - base >= w0) {
        const int skip = min((int)((x0 - base - w0) / w1), p.G - 2);
        g = 1 + skip;
        base += w0 + skip * w1;
      }
    }
  }
  __device__ __forceinline__ bool next(const TreeUmmaParams& P, TuItem& it) {
    const TreeParams& p = P.p;
    while (b < p.B && base < x1) {
      tree_lens(p.cache_len, p.draft_len, b, p.cap, p.T, it.L, it.n);
      it.R = it.n * (p.k + (g == 0 ? 1 : 0));
      it.rows = min(it.R - s * kTuRows, kTuRows);
      if (it.rows <= 0) {
        s = 0;
        if (it.n == 0 || ++g == p.G) {
          g = 0;
          ++b;
        }
        continue;
      }
      it.b = b;
      it.g = g;
      it.s = s;
      it.pair = it.rows > 128;
      it.nblk = (it.L + kTuBlock - 1) / kTuBlock + 1;
      it.unit = b * (P.u0 + (p.G - 1) * P.u1) + (g == 0 ? s : P.u0 + (g - 1) * P.u1 + s);
      const int w = tu_weight(it.rows);
      const long long a = x0 - base, e = x1 - base;
      it.j0 = a <= 0 ? 0 : (int)min((long long)it.nblk, (a + w - 1) / w);
      it.j1 = (int)min((long long)it.nblk, (e + w - 1) / w);
      base += (long long)it.nblk * w;
      ++s;
      if (it.j0 < it.j1) return true;
    }
    return false;
  }
};

// 2^x for a pair on the FMA pipe, to 4e-6: as exp2_poly2 of attn2.cuh with a
// polynomial of degree 4 (fit_exp2_poly.py), for the log-sum in fp32 beside O.
__device__ __forceinline__ void exp2_poly4(float& y0, float& y1, float x0, float x1) {
  constexpr float kShift = 12582912.0f;  // 1.5 * 2^23
  constexpr float c0 = 9.999992847e-01f, c1 = 6.931217909e-01f, c2 = 2.402474433e-01f, c3 = 5.591785908e-02f,
                  c4 = 9.570102207e-03f;
  x0 = fmaxf(x0, -125.0f);
  x1 = fmaxf(x1, -125.0f);
  float t0, t1, j0, j1, f0, f1, p0, p1;
  fadd2(t0, t1, x0, x1, kShift, kShift);
  fadd2(j0, j1, t0, t1, -kShift, -kShift);
  ffma2(f0, f1, j0, j1, -1.0f, -1.0f, x0, x1);
  ffma2(p0, p1, f0, f1, c4, c4, c3, c3);
  ffma2(p0, p1, p0, p1, f0, f1, c2, c2);
  ffma2(p0, p1, p0, p1, f0, f1, c1, c1);
  ffma2(p0, p1, p0, p1, f0, f1, c0, c0);
  y0 = __int_as_float(__float_as_int(p0) + (__float_as_int(t0) << 23));
  y1 = __int_as_float(__float_as_int(p1) + (__float_as_int(t1) << 23));
}

// Three-way maximum that keeps NaN.
__device__ __forceinline__ float fmax3_nan(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

__global__ void __launch_bounds__(kTuThreads, 1) tree_attn_umma_kernel(const __grid_constant__ TreeUmmaParams P) {
  using S = TuSmem;
  const TreeParams& p = P.p;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S::kBar);
  uint64_t* k_full = bars;                  // [kTuStages]
  uint64_t* v_full = k_full + kTuStages;    // [kTuStages]
  uint64_t* kv_empty = v_full + kTuStages;  // [kTuStages]
  uint64_t* q_full = kv_empty + kTuStages;  // [2] tiles
  uint64_t* s_full = q_full + 2;            // [2]
  uint64_t* s_free = s_full + 2;            // [2]
  uint64_t* p_full = s_free + 2;            // [2]
  uint64_t* pv_done = p_full + 2;           // [2]
  uint64_t* mask_full = pv_done + 2;        // [2] buffers
  uint64_t* mask_empty = mask_full + 2;     // [2]
  uint64_t* both = mask_empty + 2;          // [2] both tiles' softmax threads meet: m, l written; O read
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(both + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  long long* prefix = reinterpret_cast<long long*>(smem + S::kPrefix);
  uint4* s_mask = reinterpret_cast<uint4*>(smem + S::kMask);
  uint32_t* s_bad = reinterpret_cast<uint32_t*>(smem + S::kBad);
  float2* s_ml = reinterpret_cast<float2*>(smem + S::kML);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int s = 0; s < kTuStages; ++s) {
      mbar_init(&k_full[s], 1);
      mbar_init(&v_full[s], 1);
      mbar_init(&kv_empty[s], 2);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&q_full[t], 128);
      mbar_init(&s_full[t], 1);
      mbar_init(&s_free[t], 128);
      mbar_init(&p_full[t], 128);
      mbar_init(&pv_done[t], 1);
      mbar_init(&mask_full[t], 32);
      mbar_init(&mask_empty[t], 256);
      mbar_init(&both[t], 256);
    }
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&P.tmK);
    tma_prefetch_desc(&P.tmV);
    tma_prefetch_desc(&P.tmKn);
    tma_prefetch_desc(&P.tmVn);
  }
  if (warp == 1) tmem_alloc(tmem_slot, 512);
  pdl_wait();
  pdl_trigger();
  // weight before each sequence (inclusive sums, shifted by one)
  if (tid == 0) prefix[0] = 0;
  for (int b = tid; b < p.B; b += kTuThreads) {
    int L, n;
    tree_lens(p.cache_len, p.draft_len, b, p.cap, p.T, L, n);
    prefix[b + 1] = tu_seq_weight(L, n, p.G, p.k);
  }
  __syncthreads();
  for (int d = 1; d < p.B; d *= 2) {
    long long v[(kTuMaxB + kTuThreads - 1) / kTuThreads];
#pragma unroll
    for (int i = 0; i < (kTuMaxB + kTuThreads - 1) / kTuThreads; ++i) {
      const int b = tid + i * kTuThreads;
      if (b < p.B) v[i] = prefix[b + 1] + (b >= d ? prefix[b + 1 - d] : 0);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < (kTuMaxB + kTuThreads - 1) / kTuThreads; ++i) {
      const int b = tid + i * kTuThreads;
      if (b < p.B) prefix[b + 1] = v[i];
    }
    __syncthreads();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const uint32_t sbase = smem_u32(smem);
  // no range below the weight of a block, so that every range inside a unit
  // holds one
  const long long total = prefix[p.B];
  const int grid = (int)max(1ll, min((long long)gridDim.x, total / 3)), cta = blockIdx.x;
  TuCursor cur;
  cur.start(p, prefix, tu_range(total, min(cta, grid), grid), tu_range(total, min(cta + 1, grid), grid));
  TuItem it;

  if (warp < 4) {
    setmaxnreg_dec<kTuRegsLow>();
    if (warp == 0 && lane == 0) {
      // ---- producer ----------------------------------------------------------------
      uint32_t kv = 0;
      bool ok = true;
      while (ok && cur.next(P, it)) {
        for (int j = it.j0; j < it.j1; ++j, ++kv) {
          const int s = kv % kTuStages;
          if (!(ok = mbar_wait(&kv_empty[s], ((kv / kTuStages) & 1) ^ 1, abort_flag))) break;
          const bool drafts = j == it.nblk - 1;
          const int row = drafts ? it.b * p.T : it.b * p.cap + j * kTuBlock;
          uint8_t* to = smem + S::kKV + s * 32768;
          mbar_arrive_expect_tx(&k_full[s], 16384);
          tma_load_3d(to, drafts ? &P.tmKn : &P.tmK, &k_full[s], 0, it.g, row);
          mbar_arrive_expect_tx(&v_full[s], 16384);
          tma_load_3d(to + 16384, drafts ? &P.tmVn : &P.tmV, &v_full[s], 0, it.g, row);
        }
      }
    } else if ((warp == 1 || warp == 2) && lane == 0) {
      // ---- MMA issue: warp 1 drives tile A, warp 2 tile B -----------------------------
      const int t = warp - 1;
      constexpr uint32_t idesc_s = idesc_bf16(128, 128, false, false);
      constexpr uint32_t idesc_o = idesc_bf16(128, 64, false, true);
      uint32_t kv = 0, s_cnt = 0, pv_cnt = 0, q_cnt = 0;
      bool ok = true;
      const uint32_t qa = sbase + S::kQ + t * 16384;
      auto issue_s = [&](uint32_t kvi) -> bool {
        if (!mbar_wait(&k_full[kvi % kTuStages], (kvi / kTuStages) & 1, abort_flag)) return false;
        if (s_cnt > 0 && !mbar_wait(&s_free[t], (s_cnt - 1) & 1, abort_flag)) return false;
        tc_fence_after();
        const uint32_t ka = sbase + S::kKV + (kvi % kTuStages) * 32768;
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          umma_ss(tmem_base + t * 128, sdesc_sw128(qa + kk * 32, 16, 1024), sdesc_sw128(ka + kk * 32, 16, 1024), idesc_s,
                  kk != 0);
        umma_commit(&s_full[t]);
        ++s_cnt;
        return true;
      };
      while (ok && cur.next(P, it)) {
        const int nj = it.j1 - it.j0, mine = it.tile_blocks(t);
        const int stride = it.pair ? 1 : 2, first = it.pair ? 0 : t;
        if (!(ok = mbar_wait(&q_full[t], q_cnt & 1, abort_flag))) break;
        ++q_cnt;
        if (mine > 0 && !(ok = issue_s(kv + first))) break;
        for (int jj = 0; ok && jj < nj; ++jj) {
          const uint32_t kvj = kv + jj;
          if (it.owns(t, jj)) {
            if (jj + stride < nj && !(ok = issue_s(kvj + stride))) break;
            if (!(ok = mbar_wait(&v_full[kvj % kTuStages], (kvj / kTuStages) & 1, abort_flag))) break;
            if (!(ok = mbar_wait(&p_full[t], pv_cnt & 1, abort_flag))) break;
            tc_fence_after();
            const uint32_t va = sbase + S::kKV + (kvj % kTuStages) * 32768 + 16384;
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
              umma_ts(tmem_base + 256 + t * 64, tmem_base + 384 + t * 64 + kk * 8, sdesc_sw128(va + kk * 2048, 8192, 1024),
                      idesc_o, (jj != first || kk != 0) ? 1u : 0u);
            umma_commit(&pv_done[t]);
            ++pv_cnt;
            umma_commit(&kv_empty[kvj % kTuStages]);
          } else {
            // the other tile's block: released only after it has arrived (an
            // earlier arrival would count for the stage's previous block)
            if (!(ok = mbar_wait(&k_full[kvj % kTuStages], (kvj / kTuStages) & 1, abort_flag))) break;
            if (!(ok = mbar_wait(&v_full[kvj % kTuStages], (kvj / kTuStages) & 1, abort_flag))) break;
            mbar_arrive(&kv_empty[kvj % kTuStages]);
          }
        }
        kv += nj;
      }
    } else if (warp == 3) {
      // ---- ancestor masks of the units whose draft block is here ----------------------
      int* up = reinterpret_cast<int*>(smem + S::kUp);
      uint32_t cnt = 0;
      while (cur.next(P, it)) {
        if (!it.has_drafts()) continue;
        const int buf = cnt & 1;
        bool ok = mbar_wait(&mask_empty[buf], ((cnt >> 1) & 1) ^ 1, abort_flag);
        if (!__all_sync(0xffffffffu, ok)) break;
        uint4* mask = s_mask + buf * kTreeMax;
        for (int i = lane; i < kTreeMax; i += 32) {
          int u = -1;
          if (i < it.n) {
            u = p.parent ? p.parent[(size_t)it.b * p.T + i] : i - 1;
            if (u < -1 || u >= i) {
              flag_bounds_error();
              u = -1;
            }
          }
          uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (i >> 5 == j) w[j] = 1u << (i & 31);
          mask[i] = make_uint4(w[0], w[1], w[2], w[3]);
          up[i] = u;
        }
        __syncwarp();
        for (int span = 1; span < it.n; span *= 2) {
          uint4 m[4];
          int u[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int i = lane + 32 * q;
            u[q] = up[i];
            m[q] = mask[i];
            if (u[q] >= 0) {
              const uint4 a = mask[u[q]];
              m[q] = make_uint4(m[q].x | a.x, m[q].y | a.y, m[q].z | a.z, m[q].w | a.w);
              u[q] = up[u[q]];
            }
          }
          __syncwarp();
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            mask[lane + 32 * q] = m[q];
            up[lane + 32 * q] = u[q];
          }
          __syncwarp();
        }
        // drafted values that are not finite: eight lanes a row
        uint32_t bad[4] = {0u, 0u, 0u, 0u};
        const __nv_bfloat16* vn = p.Vn + ((size_t)it.b * p.T * p.G + it.g) * 64;
#pragma unroll 4
        for (int i0 = 0; i0 < kTreeMax; i0 += 4) {
          const int i = i0 + (lane >> 3);
          bool b0 = false;
          if (i < it.n) {
            const uint4 v = reinterpret_cast<const uint4*>(vn + (size_t)i * p.G * 64)[lane & 7];
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) b0 |= (w[e] & 0x7f80u) == 0x7f80u || (w[e] & 0x7f800000u) == 0x7f800000u;
          }
          const uint32_t hit = __ballot_sync(0xffffffffu, b0);
#pragma unroll
          for (int q = 0; q < 4; ++q)
            if (hit & (0xffu << (8 * q))) bad[(i0 + q) >> 5] |= 1u << ((i0 + q) & 31);
        }
        if (lane < 4) s_bad[buf * 4 + lane] = lane == 0 ? bad[0] : (lane == 1 ? bad[1] : (lane == 2 ? bad[2] : bad[3]));
        mbar_arrive(&mask_full[buf]);
        ++cnt;
      }
    }
  } else {
    setmaxnreg_inc<kTuRegsHigh>();
    // ---- softmax: warps 4..7 tile A, 8..11 tile B, one thread a row --------------------
    const int t = (warp - 4) >> 2;
    const int q = warp & 3;
    const int row = q * 32 + lane;  // of the tile
    const uint32_t lane_off = static_cast<uint32_t>(q * 32) << 16;
    const uint32_t tm_s = tmem_base + lane_off + t * 128;
    const uint32_t tm_o = tmem_base + lane_off + 256 + t * 64;
    const uint32_t tm_p = tmem_base + lane_off + 384 + t * 64;
    const float sl2 = p.scale_log2;
    uint32_t kv = 0;             // blocks of the range before this unit's
    uint32_t cnt = 0, other = 0; // blocks that this tile and the other have processed
    uint32_t masks = 0, meets = 0;
    bool ok = true;
    while (ok && cur.next(P, it)) {
      const int base = it.row_base(t), r = base + row;
      const int nrow = min(128, it.R - base);          // rows of this tile
      const bool warp_on = q * 32 < nrow;
      const int rc = min(r, it.R - 1);                 // (rows past the last repeat it and are not stored)
      const int tok = tree_row_token(rc, it.n, p.k), slot = tree_row_slot(rc, it.n, it.g, p.k, p.G);
      const size_t out = ((size_t)it.b * p.T + tok) * p.Ha + slot;
      {
        // this row of Q, swizzled as the MMA reads it. Every S of the unit
        // before has been read, so its Q is no longer in use.
        const uint4* src = reinterpret_cast<const uint4*>(p.Q + out * 64);
        uint8_t* qs = smem + S::kQ + t * 16384 + row * 128;
        uint4 v[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) v[c] = src[c];
#pragma unroll
        for (int c = 0; c < 8; ++c) *reinterpret_cast<uint4*>(qs + ((c ^ (row & 7)) << 4)) = v[c];
        fence_proxy_async_smem();
        mbar_arrive(&q_full[t]);
      }
      const int nj = it.j1 - it.j0;
      const int stride = it.pair ? 1 : 2, first = it.pair ? 0 : t;
      float m_run = -INFINITY, l_run = 0.f;
      for (int jj = first; jj < nj; jj += stride, ++cnt) {
        const int j = it.j0 + jj;
        const bool drafts = j == it.nblk - 1;
        const int valid = drafts ? it.n : min(kTuBlock, it.L - j * kTuBlock);
        bool w_ok = !drafts || mbar_wait(&mask_full[masks & 1], (masks >> 1) & 1, abort_flag);
        if (w_ok && (valid < kTuBlock || drafts)) {
          // this thread's value row: zeroed past the last valid one; without
          // the values that are not finite in a drafted row
          const uint32_t kvj = kv + jj;
          w_ok = mbar_wait(&v_full[kvj % kTuStages], (kvj / kTuStages) & 1, abort_flag);
          uint8_t* vs = smem + S::kKV + (kvj % kTuStages) * 32768 + 16384 + row * 128;
          if (w_ok && row >= valid) {
#pragma unroll
            for (int c = 0; c < 8; ++c) *reinterpret_cast<uint4*>(vs + 16 * c) = make_uint4(0u, 0u, 0u, 0u);
          } else if (w_ok && drafts && ((s_bad[(masks & 1) * 4 + (row >> 5)] >> (row & 31)) & 1u)) {
            for (int c = 0; c < 32; ++c) {
              uint32_t w = *reinterpret_cast<uint32_t*>(vs + 4 * c);
              if ((w & 0x7f80u) == 0x7f80u) w &= 0xffff0000u;
              if ((w & 0x7f800000u) == 0x7f800000u) w &= 0x0000ffffu;
              *reinterpret_cast<uint32_t*>(vs + 4 * c) = w;
            }
          }
          fence_proxy_async_smem();
        }
        w_ok = w_ok && mbar_wait(&s_full[t], cnt & 1, abort_flag);
        if (!__all_sync(0xffffffffu, w_ok)) { ok = false; break; }
        tc_fence_after();
        if (!warp_on) {
          // P of rows that are not stored may hold anything; the arrival must
          // not fall into the block before, though
          tc_fence_before();
          mbar_arrive(&s_free[t]);
          w_ok = jj == first || mbar_wait(&pv_done[t], (cnt - 1) & 1, abort_flag);
          if (!__all_sync(0xffffffffu, w_ok)) { ok = false; break; }
          mbar_arrive(&p_full[t]);
          continue;
        }
        float s[128];
        tmem_ld128f(tm_s, s);
        tc_fence_before();
        mbar_arrive(&s_free[t]);  // S may be overwritten by the next block's QK^T now
        if (drafts) {
          const uint4 mk = s_mask[(masks & 1) * kTreeMax + tok];
#pragma unroll
          for (int c = 0; c < 128; ++c)
            if (!((mask_word(mk, c >> 5) >> (c & 31)) & 1u)) s[c] = -INFINITY;
        } else if (valid < kTuBlock) {
#pragma unroll
          for (int c = 0; c < 128; ++c)
            if (c >= valid) s[c] = -INFINITY;
        }
        float m4[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
        for (int c = 4; c < 128; c += 8) {
          m4[0] = fmax3_nan(m4[0], s[c], s[c + 1]);
          m4[1] = fmax3_nan(m4[1], s[c + 2], s[c + 3]);
          if (c + 4 < 128) {
            m4[2] = fmax3_nan(m4[2], s[c + 4], s[c + 5]);
            m4[3] = fmax3_nan(m4[3], s[c + 6], s[c + 7]);
          }
        }
        const float mx = fmax3_nan(fmax3_nan(m4[0], m4[1], m4[1]), m4[2], m4[3]);
        const float m_new = fmaxf(m_run, mx * sl2);
        const float m_use = (m_new > m_run + kRescaleThreshold) ? m_new : m_run;
        const float mu = m_use == -INFINITY ? 0.f : m_use;
        const float alpha = ex2_approx(m_run - mu);
        const bool rescale = jj != first && m_use != m_run;
        m_run = m_use;
        float sm[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        uint32_t pk[64];
        if (drafts) {
          // (a masked place must be exactly zero here: MUFU only)
#pragma unroll
          for (int pi = 0; pi < 64; ++pi) {
            float x0, x1;
            ffma2(x0, x1, s[2 * pi], s[2 * pi + 1], sl2, sl2, -mu, -mu);
            const float y0 = ex2_approx(x0), y1 = ex2_approx(x1);
            fadd2(sm[2 * (pi & 3)], sm[2 * (pi & 3) + 1], sm[2 * (pi & 3)], sm[2 * (pi & 3) + 1], y0, y1);
            pk[pi] = pack_bf16x2(y0, y1);
          }
        } else {
#pragma unroll
          for (int pi = 0; pi < 64; ++pi) {
            float x0, x1, y0, y1;
            ffma2(x0, x1, s[2 * pi], s[2 * pi + 1], sl2, sl2, -mu, -mu);
            if ((pi % kTuPolyEvery) == kTuPolyEvery - 1) {
              exp2_poly4(y0, y1, x0, x1);
            } else {
              y0 = ex2_approx(x0);
              y1 = ex2_approx(x1);
            }
            fadd2(sm[2 * (pi & 3)], sm[2 * (pi & 3) + 1], sm[2 * (pi & 3)], sm[2 * (pi & 3) + 1], y0, y1);
            pk[pi] = pack_bf16x2(y0, y1);
          }
        }
        l_run = l_run * alpha + (((sm[0] + sm[1]) + (sm[2] + sm[3])) + ((sm[4] + sm[5]) + (sm[6] + sm[7])));
        if (!(mx < INFINITY)) l_run = __int_as_float(0x7fffffff);  // a score that is NaN or +inf: the row is NaN
        if (jj != first) {
          w_ok = mbar_wait(&pv_done[t], (cnt - 1) & 1, abort_flag);
          if (!__all_sync(0xffffffffu, w_ok)) { ok = false; break; }
          tc_fence_after();
          if (__any_sync(0xffffffffu, rescale)) {
#pragma unroll
            for (int h = 0; h < 4; ++h) {
              uint32_t o[16];
              tmem_ld16(tm_o + h * 16, o);
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
              tmem_st16(tm_o + h * 16, o);
            }
          }
        }
        tmem_st64(tm_p, pk);
        tc_fence_before();
        mbar_arrive(&p_full[t]);
      }
      if (!ok) break;
      const int nother = it.pair ? nj : (nj + t) >> 1;  // blocks of the other tile
      other += nother;
      const int mine = it.tile_blocks(t);
      // ---- the unit's end ------------------------------------------------------------
      bool w_ok = mine == 0 || mbar_wait(&pv_done[t], (cnt - 1) & 1, abort_flag);
      if (!__all_sync(0xffffffffu, w_ok)) { ok = false; break; }
      float f_own = 1.f, f_other = 0.f, M = m_run, l = l_run;
      if (!it.pair) {
        // the two tiles of the same rows: each row's (m, l) through shared
        // memory; then this tile takes half of the columns of both outputs
        s_ml[t * 128 + row] = make_float2(m_run, l_run);
        mbar_arrive(&both[0]);
        w_ok = mbar_wait(&both[0], meets & 1, abort_flag) &&
               (nother == 0 || mbar_wait(&pv_done[t ^ 1], (other - 1) & 1, abort_flag));
        if (!__all_sync(0xffffffffu, w_ok)) { ok = false; break; }
        const float2 o = s_ml[(t ^ 1) * 128 + row];
        M = fmaxf(m_run, o.x);
        const float Mu = M == -INFINITY ? 0.f : M;
        f_own = mine == 0 ? 0.f : ex2_approx(m_run - Mu);
        f_other = nother == 0 ? 0.f : ex2_approx(o.x - Mu);
        l = (mine == 0 ? 0.f : f_own * l_run) + (nother == 0 ? 0.f : f_other * o.y);
      }
      tc_fence_after();
      const bool whole = it.whole();
      const bool live = row < nrow;
      const float inv = whole ? 1.f / l : 1.f;
      const uint32_t part = (2 * cta + (it.j0 == 0 ? 1 : 0)) * P.prow + (it.pair ? t * 128 : 0) + row;
      uint4 mk = make_uint4(0u, 0u, 0u, 0u);
      bool any_bad = false;
      if (it.has_drafts()) {
        // (waited for already by the tile whose block it was)
        if (!mbar_wait(&mask_full[masks & 1], (masks >> 1) & 1, abort_flag)) { ok = false; }
        const uint4 bd = *reinterpret_cast<const uint4*>(s_bad + (masks & 1) * 4);
        mk = s_mask[(masks & 1) * kTreeMax + tok];
        mk = make_uint4(mk.x & bd.x, mk.y & bd.y, mk.z & bd.z, mk.w & bd.w);
        any_bad = (mk.x | mk.y | mk.z | mk.w) != 0u;
      }
      if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
      if (warp_on) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (!it.pair && h != t) continue;
          float o[32];
          {
            uint32_t a[32];
            if (mine > 0) {
              tmem_ld32(tm_o + h * 32, a);
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = __uint_as_float(a[i]) * f_own;
            } else {
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = 0.f;
            }
            if (!it.pair && nother > 0) {
              tmem_ld32(tmem_base + lane_off + 256 + (t ^ 1) * 64 + h * 32, a);
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = fmaf(__uint_as_float(a[i]), f_other, o[i]);
            }
          }
          if (any_bad && live) {
            for (int w = 0; w < 4; ++w)
              for (uint32_t bits = mask_word(mk, w); bits; bits &= bits - 1) {
                const __nv_bfloat16* v =
                    p.Vn + (((size_t)it.b * p.T + w * 32 + __ffs(bits) - 1) * p.G + it.g) * 64 + h * 32;
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                  const float x = __bfloat162float(v[i]);
                  if (!isfinite(x)) o[i] += x;
                }
              }
          }
          if (live && whole) {
            __nv_bfloat16* dst = p.O + out * 64 + h * 32;
#pragma unroll
            for (int i = 0; i < 4; ++i)
              st_global_v4(dst + i * 8, pack_bf16x2(o[8 * i] * inv, o[8 * i + 1] * inv),
                           pack_bf16x2(o[8 * i + 2] * inv, o[8 * i + 3] * inv),
                           pack_bf16x2(o[8 * i + 4] * inv, o[8 * i + 5] * inv),
                           pack_bf16x2(o[8 * i + 6] * inv, o[8 * i + 7] * inv));
          } else if (live) {
            float4* dst = reinterpret_cast<float4*>(p.part_o + (size_t)part * 64 + h * 32);
#pragma unroll
            for (int i = 0; i < 8; ++i) dst[i] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
          }
        }
      }
      if (live && (it.pair || t == 0)) {
        if (!whole)
          *reinterpret_cast<float2*>(p.part_ml + (size_t)part * 2) = make_float2(M, l);
        else if (p.lse)
          p.lse[out] = (M + log2f(l)) * 0.6931471805599453f;
      }
      if (t == 0 && row == 0 && it.j0 == 0) {
        // the ranges that hold blocks of this unit
        const long long ubase = cur.base - (long long)it.nblk * tu_weight(it.rows);
        P.unit_cta[it.unit] =
            make_int2(cta, tu_range_of(total, grid, ubase + (long long)(it.nblk - 1) * tu_weight(it.rows)));
      }
      tc_fence_before();
      if (it.has_drafts()) {
        mbar_arrive(&mask_empty[masks & 1]);
        ++masks;
      }
      if (!it.pair) {
        // neither tile's next O may overwrite what the other still reads
        mbar_arrive(&both[1]);
        w_ok = mbar_wait(&both[1], meets & 1, abort_flag);
        if (!__all_sync(0xffffffffu, w_ok)) { ok = false; break; }
        ++meets;
      }
      kv += nj;
    }
  }
  __syncwarp();  // lanes that skipped a single-lane role wait for it
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

// The parts of every row that was cut, added: `kParts` groups of 16 lanes a row,
// four dimensions a lane.
constexpr int kTuMergeThreads = 128;
template <int kParts>
__global__ void __launch_bounds__(kTuMergeThreads) tree_umma_merge_kernel(const TreeUmmaParams P) {
  static_assert(kParts == 2 || kParts == 8, "a warp or the block per row");
  const TreeParams& p = P.p;
  __shared__ float s_m[kTuMergeThreads / 16], s_l[kTuMergeThreads / 16];
  __shared__ float4 s_o[kTuMergeThreads];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, part = (tid >> 4) % kParts, d = tid & 15;
  constexpr int kRowsPer = kTuMergeThreads / 16 / kParts;
  const int sub = (tid >> 4) / kParts;
  const long long id = (long long)blockIdx.x * kRowsPer + sub;
  bool on = id < (long long)p.B * p.T * p.Ha;
  const long long cid = on ? id : 0;
  const int slot = (int)(cid % p.Ha), bt = (int)(cid / p.Ha), b = bt / p.T, tok = bt % p.T;
  int L, n;
  tree_lens(p.cache_len, p.draft_len, b, p.cap, p.T, L, n);
  on = on && tok < n;
  const bool shared = slot == p.G * p.k;
  const int g = shared ? 0 : slot / p.k;
  const int row = shared ? n * p.k + tok : tok * p.k + slot % p.k;
  const int s = row / kTuRows;
  int2 ctas = make_int2(0, 0);
  if (on) ctas = P.unit_cta[b * (P.u0 + (p.G - 1) * P.u1) + (g == 0 ? s : P.u0 + (g - 1) * P.u1 + s)];
  on = on && ctas.x != ctas.y;  // (else it was written at once)
  float m = -INFINITY, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  if (on) {
    for (int c = ctas.x + part; c <= ctas.y; c += kParts) {
      const size_t at = (size_t)(2 * c + (c == ctas.x ? 1 : 0)) * P.prow + row % kTuRows;
      const float2 ml = *reinterpret_cast<const float2*>(p.part_ml + at * 2);
      const float4 v = *reinterpret_cast<const float4*>(p.part_o + at * 64 + d * 4);
      const float M = fmaxf(m, ml.x), Mu = M == -INFINITY ? 0.f : M;
      const float f0 = ex2_approx(m - Mu), f1 = ex2_approx(ml.x - Mu);
      m = M;
      l = fmaf(l, f0, ml.y * f1);
      o.x = fmaf(o.x, f0, v.x * f1);
      o.y = fmaf(o.y, f0, v.y * f1);
      o.z = fmaf(o.z, f0, v.z * f1);
      o.w = fmaf(o.w, f0, v.w * f1);
    }
  }
  if (d == 0) {
    s_m[tid >> 4] = m;
    s_l[tid >> 4] = l;
  }
  s_o[tid] = o;
  __syncthreads();
  if (!on || part != 0) return;
  float M = -INFINITY;
#pragma unroll
  for (int q = 0; q < kParts; ++q) M = fmaxf(M, s_m[sub * kParts + q]);
  const float Mu = M == -INFINITY ? 0.f : M;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float sum = 0.f;
#pragma unroll
  for (int q = 0; q < kParts; ++q) {
    const float f = ex2_approx(s_m[sub * kParts + q] - Mu);
    const float4 v = s_o[(sub * kParts + q) * 16 + d];
    sum = fmaf(s_l[sub * kParts + q], f, sum);
    acc.x = fmaf(v.x, f, acc.x);
    acc.y = fmaf(v.y, f, acc.y);
    acc.z = fmaf(v.z, f, acc.z);
    acc.w = fmaf(v.w, f, acc.w);
  }
  const float inv = 1.f / sum;
  const size_t out = (size_t)bt * p.Ha + slot;
  *reinterpret_cast<uint2*>(p.O + out * 64 + d * 4) = make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
  if (p.lse && d == 0) p.lse[out] = (M + log2f(sum)) * 0.6931471805599453f;
}

}  // namespace gqe
