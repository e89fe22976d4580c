// tree.cuh -- attention of a tree of drafted tokens over a key/value cache.
//
// Sequence b has L = cache_len[b] cached positions and n = draft_len[b] drafted
// tokens, token i the child of parent[i] < i (-1: of the cached sequence).
// A query row of token i attends
//     every cached position s < L,  and  i itself and its ancestors,
//   O = sum_s p_s v_s / l,   p_s = exp(q.k_s / 8 - m),   l = sum_s p_s,
//   lse = m + log l.
// Work per (sequence, group): its R = n*k rows (and in group 0 the n shared
// rows) against L + n keys; 256 bytes of K and V a key, 256 flops a (row, key).
#pragma once

#include "decode.cuh"
#include "sm100.cuh"

namespace gqe {

constexpr int kTreeMax = 128;  // drafted tokens of a sequence

struct TreeParams {
  const __nv_bfloat16 *Q, *Kn, *Vn;  // [B*T, Ha, 64], [B*T, G, 64]
  const __nv_bfloat16 *Kc, *Vc;      // [B, cap, G, 64]
  const int32_t *cache_len, *draft_len, *parent;
  __nv_bfloat16* O;
  float* lse;
  int B, T, G, k, Ha, cap;
  float scale_log2;
  // The rows of a (sequence, group) are cut into units of `urows`: u0 of them in
  // group 0, u1 in each other group, for T tokens.
  int urows, u0, u1;
  // Units that a range of keys cut in pieces: two parts a block of threads, part
  // 2 c + 1 the one that starts the unit, 2 c the one that goes on with it
  float *part_ml, *part_o;  // [2 * gridDim.x][prow] {m, l}, [..][64]
  int prow;                 // rows of a part, the most that a unit has
  int2* unit_cta;           // [B * (u0 + (G - 1) * u1)] first and last block that holds keys of the unit
  int step;                 // from one of them to the next
};

// Rows of a group: the selected experts' (token-major), then in group 0 the
// shared head's.
__device__ __forceinline__ int tree_row_token(int r, int n, int k) { return r < n * k ? r / k : r - n * k; }
__device__ __forceinline__ int tree_row_slot(int r, int n, int g, int k, int G) {
  return r < n * k ? g * k + r % k : G * k;
}
// Cached positions and drafted tokens of sequence b; n = 0 where either is out
// of range (recorded; nothing of the sequence is read or written).
__device__ __forceinline__ void tree_lens(const int32_t* cache_len, const int32_t* draft_len, int b, int cap, int T,
                                          int& L, int& n) {
  L = cache_len[b];
  n = draft_len ? draft_len[b] : T;
  if (L < 0 || L > cap || n < 0 || n > T) {
    flag_bounds_error();
    L = 0;
    n = 0;
  }
}

// The keys of all sequences, one after the other and cut into blocks, are split
// into ranges of equal weight; prefix[b] is the weight before sequence b. Every
// thread of the block calls it, with w(b) the weight of sequence b.
constexpr int kTreeMaxB = 1024;  // B * G * M <= 8192 and G * M >= 8
// prefix[1 .. B] to its inclusive sums, by doubling; prefix[0] = 0 before.
template <int kThreads, typename I>
__device__ __forceinline__ void scan_prefix(I* prefix, int B) {
  constexpr int kEach = (kTreeMaxB + kThreads - 1) / kThreads;
  const int tid = threadIdx.x;
  for (int d = 1; d < B; d *= 2) {
    I v[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int b = tid + i * kThreads;
      if (b < B) v[i] = prefix[b + 1] + (b >= d ? prefix[b + 1 - d] : I(0));
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int b = tid + i * kThreads;
      if (b < B) prefix[b + 1] = v[i];
    }
    __syncthreads();
  }
}
template <int kThreads, typename I, typename F>
__device__ __forceinline__ void tree_prefix(const TreeParams& p, I* prefix, F w) {
  const int tid = threadIdx.x;
  if (tid == 0) prefix[0] = 0;
  for (int b = tid; b < p.B; b += kThreads) {
    int L, n;
    tree_lens(p.cache_len, p.draft_len, b, p.cap, p.T, L, n);
    prefix[b + 1] = n == 0 ? 0 : w(L, n);
  }
  __syncthreads();
  scan_prefix<kThreads>(prefix, p.B);
}
// The last sequence that begins at or before x.
template <typename I>
__device__ __forceinline__ int tree_first(const I* prefix, int B, long long x) {
  int lo = 0, hi = B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (prefix[mid] <= x) lo = mid; else hi = mid - 1;
  }
  return lo;
}
// Where range c begins, and the range that holds x.
__device__ __forceinline__ long long tree_range(long long total, int c, int ranges) { return total * c / ranges; }
__device__ __forceinline__ int tree_range_of(long long total, int ranges, long long x) {
  return (int)(((x + 1) * ranges - 1) / total);
}

// mask[i] = bits of token i and its ancestors, by pointer doubling: after round
// r a token's mask covers 2^r generations and up[] points 2^r up. All threads
// of the block call it.
__device__ __forceinline__ void tree_masks(const int32_t* parent, int n, uint4* mask, int* up) {
  const int tid = threadIdx.x;
  for (int i = tid; i < kTreeMax; i += blockDim.x) {
    int p = -1;
    if (i < n) {
      p = parent ? parent[i] : i - 1;
      if (p < -1 || p >= i) {
        flag_bounds_error();
        p = -1;
      }
    }
    uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (i >> 5 == j) w[j] = 1u << (i & 31);
    mask[i] = make_uint4(w[0], w[1], w[2], w[3]);
    up[i] = p;
  }
  __syncthreads();
  for (int span = 1; span < n; span *= 2) {
    uint4 m = make_uint4(0u, 0u, 0u, 0u);
    int u = -1;
    if (tid < n) {
      u = up[tid];
      m = mask[tid];
      if (u >= 0) {
        const uint4 a = mask[u];
        m = make_uint4(m.x | a.x, m.y | a.y, m.z | a.z, m.w | a.w);
        u = up[u];
      }
    }
    __syncthreads();
    if (tid < n) {
      mask[tid] = m;
      up[tid] = u;
    }
    __syncthreads();
  }
}
__device__ __forceinline__ uint32_t mask_word(const uint4& m, int w) {
  return w == 0 ? m.x : (w == 1 ? m.y : (w == 2 ? m.z : m.w));
}

// ---------------------------------------------------------------------------
// tree_attn_mma_kernel, for few rows: units of 16 * WR rows. Block c of four
// warps takes unit c % U of the U units of a sequence and, of every sequence
// that its range c / U of the keys touches, the key blocks in it. Neighbouring
// blocks so read the groups' rows of the same positions at about the same time
// (a position's G rows are contiguous: with the groups apart in time DRAM gave
// 10% less). Keys come in blocks of 64 through a ring of kTmStages stages
// (cp.async; K and V, 128-byte rows, 16-byte chunks swizzled). The warps are
// WR x (4 / WR): WR row tiles of 16 rows, and for each of them 4 / WR warps that
// take a share of every block's keys and are added at the end. Products on
// mma.sync m16n8k16 (bf16 in, fp32 accumulate), running maximum and sum per row
// in the log2 domain, P rounded to bf16 for P V (the tensor cores' operand type;
// l adds the unrounded p).
//
// Measured, 8 groups, one row a token: 8 x 16 tokens over 20001 to 32767
// positions 80-86 us = 5.0-5.4 TB/s of 6.5 that a copy reaches (433 MB read,
// issue slots 45% used, tensor pipe 17%): DRAM binds. One token over 4095: 11.1
// us with the merge, two kernels' latency.
// ---------------------------------------------------------------------------
constexpr int kTmKeys = 64;
constexpr int kTmStages = 3;
constexpr int kTmThreads = 128;
constexpr int kTmStageBytes = 2 * kTmKeys * 128;
constexpr int kTmSmem = kTmStages * kTmStageBytes + 1024;

template <int WR>
__global__ void __launch_bounds__(kTmThreads, WR == 4 ? 3 : 4) tree_attn_mma_kernel(const TreeParams p) {
  constexpr int WK = 4 / WR;          // warps that share a row tile
  constexpr int kRows = 16 * WR;      // rows of a unit
  constexpr int kWKeys = kTmKeys / WK;
  extern __shared__ uint8_t tm_raw[];
  __shared__ uint4 s_mask[kTreeMax];
  __shared__ int s_up[kTreeMax];
  __shared__ uint32_t s_bad[kTreeMax / 32];
  pdl_wait();
  pdl_trigger();
  uint8_t* ring = tm_raw + ((1024u - (smem_u32(tm_raw) & 1023u)) & 1023u);
  int* prefix = reinterpret_cast<int*>(ring + kTmStages * kTmStageBytes);  // [B + 1] blocks of keys: below 2^26
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int U = p.u0 + (p.G - 1) * p.u1, u = blockIdx.x % U;
  const int g = u < p.u0 ? 0 : 1 + (u - p.u0) / p.u1;
  const int row0 = (u < p.u0 ? u : (u - p.u0) % p.u1) * kRows;
  auto blocks = [](int L, int n) { return (L + kTmKeys - 1) / kTmKeys + (n + kTmKeys - 1) / kTmKeys; };
  tree_prefix<kTmThreads>(p, prefix, blocks);
  __syncthreads();
  // no range below four blocks of keys while that leaves a sequence sixteen of
  // them, which the merge takes in two steps (one sequence of 4095 positions,
  // one token: 15.9 us with a block of keys each, 11.1 so; 5 x 13 tokens over
  // 1500, 125 blocks: 16.2 either way, 19.8 with four blocks each)
  const long long total = prefix[p.B], most = max(total / 4, 16ll * p.B);
  const int ranges = (int)max(1ll, min((long long)(gridDim.x / U), min(total, most))), range = blockIdx.x / U;
  if (range >= ranges) return;
  const long long x0 = tree_range(total, range, ranges), x1 = tree_range(total, range + 1, ranges);
  for (int b = tree_first(prefix, p.B, x0); b < p.B && prefix[b] < x1; ++b) {
    int L, n;
    tree_lens(p.cache_len, p.draft_len, b, p.cap, p.T, L, n);
    const int R = n * (p.k + (g == 0 ? 1 : 0));
    if (row0 >= R) continue;
    const int ncb = (L + kTmKeys - 1) / kTmKeys;  // cached key blocks; then the drafted
    const int nblk = blocks(L, n);
    const int j0 = (int)max(0ll, x0 - prefix[b]), j1 = (int)min((long long)nblk, x1 - prefix[b]);
    if (j0 >= j1) continue;
    const bool whole = j0 == 0 && j1 == nblk;
    const size_t kstride = (size_t)p.G * 64;
    const __nv_bfloat16* kc = p.Kc + ((size_t)b * p.cap * p.G + g) * 64;
    const __nv_bfloat16* vc = p.Vc + ((size_t)b * p.cap * p.G + g) * 64;
    const __nv_bfloat16* kn = p.Kn + ((size_t)b * p.T * p.G + g) * 64;
    const __nv_bfloat16* vn = p.Vn + ((size_t)b * p.T * p.G + g) * 64;
    auto issue = [&](int j) {  // block j into its stage; rows past the valid keys are zero
      if (j < j1) {
        const bool cached = j < ncb;
        const int s0 = (cached ? j : j - ncb) * kTmKeys;
        const int nk = min(kTmKeys, (cached ? L : n) - s0);
        const __nv_bfloat16* ks = (cached ? kc : kn) + (size_t)s0 * kstride;
        const __nv_bfloat16* vs = (cached ? vc : vn) + (size_t)s0 * kstride;
        const uint32_t dst = smem_u32(ring) + ((j - j0) % kTmStages) * kTmStageBytes;
#pragma unroll
        for (int i = 0; i < kTmKeys * 8 / kTmThreads; ++i) {
          const int at = i * kTmThreads + tid, key = at >> 3, ch = at & 7;
          const uint32_t off = key * 128 + ((ch ^ (key & 7)) << 4);
          const int size = key < nk ? 16 : 0;  // 0: fill with zeros, nothing is read
          const size_t src = (size_t)(key < nk ? key : 0) * kstride + ch * 8;
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + off), "l"(ks + src), "r"(size)
                       : "memory");
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + kTmKeys * 128 + off), "l"(vs + src),
                       "r"(size)
                       : "memory");
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int i = 0; i < kTmStages - 1; ++i) issue(j0 + i);
    if (tid < kTreeMax / 32) s_bad[tid] = 0u;
    const bool drafts_here = j1 > ncb && j0 < j1;
    if (drafts_here) tree_masks(p.parent ? p.parent + (size_t)b * p.T : nullptr, n, s_mask, s_up);

    const int wr = warp / WK, wk = warp % WK;
    const int r = lane >> 2, c = lane & 3;
    const int mi = lane >> 3, mr = lane & 7;
    const int ra = row0 + wr * 16 + r, rb = ra + 8;  // this thread's two rows
    const bool warp_on = row0 + wr * 16 < R;
    uint32_t qa[4][4];
    {
      const int ta = min(ra, R - 1), tb = min(rb, R - 1);
      const __nv_bfloat16* q0 =
          p.Q + (((size_t)b * p.T + tree_row_token(ta, n, p.k)) * p.Ha + tree_row_slot(ta, n, g, p.k, p.G)) * 64;
      const __nv_bfloat16* q1 =
          p.Q + (((size_t)b * p.T + tree_row_token(tb, n, p.k)) * p.Ha + tree_row_slot(tb, n, g, p.k, p.G)) * 64;
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
        const int d0 = 16 * kk + 2 * c;
        qa[kk][0] = *reinterpret_cast<const uint32_t*>(q0 + d0);
        qa[kk][1] = *reinterpret_cast<const uint32_t*>(q1 + d0);
        qa[kk][2] = *reinterpret_cast<const uint32_t*>(q0 + d0 + 8);
        qa[kk][3] = *reinterpret_cast<const uint32_t*>(q1 + d0 + 8);
      }
    }
    float o[8][4];
#pragma unroll
    for (int dt = 0; dt < 8; ++dt)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[dt][e] = 0.f;
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
    for (int j = j0; j < j1; ++j) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kTmStages - 2) : "memory");
      __syncthreads();  // block j has landed for every thread, and block j - 1 is used up
      issue(j + kTmStages - 1);
      const bool cached = j < ncb;
      const int s0 = (cached ? j : j - ncb) * kTmKeys;
      const int nk = min(kTmKeys, (cached ? L : n) - s0);
      uint8_t* stage = ring + ((j - j0) % kTmStages) * kTmStageBytes;
      if (!cached) {
        // A drafted value that is not finite reaches its descendants only: it is
        // zeroed here (0 x NaN would reach every row) and added at the end.
        for (int i = tid; i < nk * 8; i += kTmThreads) {
          uint4* at = reinterpret_cast<uint4*>(stage + kTmKeys * 128 + (i >> 3) * 128 + (((i & 7) ^ ((i >> 3) & 7)) << 4));
          uint32_t w[4] = {at->x, at->y, at->z, at->w};
          bool bad = false;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if ((w[e] & 0x7f80u) == 0x7f80u) bad = true, w[e] &= 0xffff0000u;
            if ((w[e] & 0x7f800000u) == 0x7f800000u) bad = true, w[e] &= 0x0000ffffu;
          }
          if (bad) {
            *at = make_uint4(w[0], w[1], w[2], w[3]);
            const int key = s0 + (i >> 3);
            atomicOr(&s_bad[key >> 5], 1u << (key & 31));
          }
        }
        __syncthreads();
      }
      if (!warp_on) continue;
      const uint32_t kb = smem_u32(stage), vb = kb + kTmKeys * 128;
      float sc[kWKeys / 8][4];
#pragma unroll
      for (int nt = 0; nt < kWKeys / 8; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[nt][e] = 0.f;
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
#pragma unroll
        for (int np = 0; np < kWKeys / 16; ++np) {
          const int key = wk * kWKeys + np * 16 + (mi >> 1) * 8 + mr, ch = 2 * kk + (mi & 1);
          uint32_t b0, b1, b2, b3;
          ldsm_x4(kb + key * 128 + ((ch ^ (key & 7)) << 4), b0, b1, b2, b3);
          mma_bf16_16816(sc[2 * np], qa[kk], b0, b1);
          mma_bf16_16816(sc[2 * np + 1], qa[kk], b2, b3);
        }
      if (!cached) {
        const uint4 ma = s_mask[tree_row_token(min(ra, R - 1), n, p.k)], mb = s_mask[tree_row_token(min(rb, R - 1), n, p.k)];
#pragma unroll
        for (int nt = 0; nt < kWKeys / 8; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int key = s0 + wk * kWKeys + nt * 8 + 2 * c + e;
            const bool in = key < n;  // (bits past n are never set, word index stays in range)
            if (!in || !((mask_word(ma, (key >> 5) & 3) >> (key & 31)) & 1u)) sc[nt][e] = -INFINITY;
            if (!in || !((mask_word(mb, (key >> 5) & 3) >> (key & 31)) & 1u)) sc[nt][2 + e] = -INFINITY;
          }
      } else if (nk < kTmKeys) {
#pragma unroll
        for (int nt = 0; nt < kWKeys / 8; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            if (wk * kWKeys + nt * 8 + 2 * c + e >= nk) sc[nt][e] = sc[nt][2 + e] = -INFINITY;
      }
      float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
      for (int nt = 0; nt < kWKeys / 8; ++nt) {
        mx0 = fmaxf(mx0, fmaxf(sc[nt][0], sc[nt][1]));
        mx1 = fmaxf(mx1, fmaxf(sc[nt][2], sc[nt][3]));
      }
      mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, 1));
      mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, 2));
      mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, 1));
      mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, 2));
      const float mn0 = fmaxf(m0, mx0 * p.scale_log2), mn1 = fmaxf(m1, mx1 * p.scale_log2);
      // a row that has seen no key yet keeps m = -inf; its exponents use 0
      const float mu0 = mn0 == -INFINITY ? 0.f : mn0, mu1 = mn1 == -INFINITY ? 0.f : mn1;
      const float al0 = ex2_approx(m0 - mu0), al1 = ex2_approx(m1 - mu1);
      m0 = mn0;
      m1 = mn1;
      float ls0 = 0.f, ls1 = 0.f;
#pragma unroll
      for (int nt = 0; nt < kWKeys / 8; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          sc[nt][e] = ex2_approx(fmaf(sc[nt][e], p.scale_log2, -mu0));
          sc[nt][2 + e] = ex2_approx(fmaf(sc[nt][2 + e], p.scale_log2, -mu1));
          ls0 += sc[nt][e];
          ls1 += sc[nt][2 + e];
        }
      l0 = fmaf(l0, al0, ls0);
      l1 = fmaf(l1, al1, ls1);
#pragma unroll
      for (int dt = 0; dt < 8; ++dt) {
        o[dt][0] *= al0;
        o[dt][1] *= al0;
        o[dt][2] *= al1;
        o[dt][3] *= al1;
      }
#pragma unroll
      for (int ks = 0; ks < kWKeys / 16; ++ks) {
        const uint32_t pa[4] = {pack_bf16x2(sc[2 * ks][0], sc[2 * ks][1]), pack_bf16x2(sc[2 * ks][2], sc[2 * ks][3]),
                                pack_bf16x2(sc[2 * ks + 1][0], sc[2 * ks + 1][1]),
                                pack_bf16x2(sc[2 * ks + 1][2], sc[2 * ks + 1][3])};
#pragma unroll
        for (int dp = 0; dp < 4; ++dp) {
          const int key = wk * kWKeys + ks * 16 + (mi & 1) * 8 + mr, ch = 2 * dp + (mi >> 1);
          uint32_t b0, b1, b2, b3;
          ldsm_x4_t(vb + key * 128 + ((ch ^ (key & 7)) << 4), b0, b1, b2, b3);
          mma_bf16_16816(o[2 * dp], pa, b0, b1);
          mma_bf16_16816(o[2 * dp + 1], pa, b2, b3);
        }
      }
    }
    l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
    l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
    if constexpr (WK > 1) {
      // the warps of a row tile are added: maxima first, then each warp's sums
      // and outputs scaled to the common maximum
      asm volatile("cp.async.wait_group 0;" ::: "memory");
      __syncthreads();  // the ring is free
      float* s_m = reinterpret_cast<float*>(ring);            // [4][16]
      float* s_l = s_m + 64;                                  // [4][16]
      float* s_o = s_l + 64;                                  // [4][16][66]
      if (c == 0) {
        s_m[warp * 16 + r] = m0;
        s_m[warp * 16 + r + 8] = m1;
      }
      __syncthreads();
      float M0 = -INFINITY, M1 = -INFINITY;
#pragma unroll
      for (int w = 0; w < WK; ++w) {
        M0 = fmaxf(M0, s_m[(wr * WK + w) * 16 + r]);
        M1 = fmaxf(M1, s_m[(wr * WK + w) * 16 + r + 8]);
      }
      const float f0 = M0 == -INFINITY ? 0.f : ex2_approx(m0 - M0), f1 = M1 == -INFINITY ? 0.f : ex2_approx(m1 - M1);
      if (c == 0) {
        s_l[warp * 16 + r] = l0 * f0;
        s_l[warp * 16 + r + 8] = l1 * f1;
      }
#pragma unroll
      for (int dt = 0; dt < 8; ++dt) {
        *reinterpret_cast<float2*>(s_o + (warp * 16 + r) * 66 + dt * 8 + 2 * c) = make_float2(o[dt][0] * f0, o[dt][1] * f0);
        *reinterpret_cast<float2*>(s_o + (warp * 16 + r + 8) * 66 + dt * 8 + 2 * c) =
            make_float2(o[dt][2] * f1, o[dt][3] * f1);
      }
      m0 = M0;
      m1 = M1;
      __syncthreads();
      l0 = l1 = 0.f;
#pragma unroll
      for (int dt = 0; dt < 8; ++dt)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[dt][e] = 0.f;
#pragma unroll
      for (int w = 0; w < WK; ++w) {
        const int ww = wr * WK + w;
        l0 += s_l[ww * 16 + r];
        l1 += s_l[ww * 16 + r + 8];
#pragma unroll
        for (int dt = 0; dt < 8; ++dt) {
          const float2 a = *reinterpret_cast<const float2*>(s_o + (ww * 16 + r) * 66 + dt * 8 + 2 * c);
          const float2 d = *reinterpret_cast<const float2*>(s_o + (ww * 16 + r + 8) * 66 + dt * 8 + 2 * c);
          o[dt][0] += a.x;
          o[dt][1] += a.y;
          o[dt][2] += d.x;
          o[dt][3] += d.y;
        }
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int row = h ? rb : ra;
      if (row >= R || wk != 0) continue;
      const int tok = tree_row_token(row, n, p.k);
      if (drafts_here && (s_bad[0] | s_bad[1] | s_bad[2] | s_bad[3])) {
        const uint4 mk = s_mask[tok];
        for (int w = 0; w < 4; ++w)
          for (uint32_t bits = s_bad[w] & mask_word(mk, w); bits; bits &= bits - 1) {
            const __nv_bfloat16* v = vn + (size_t)(w * 32 + __ffs(bits) - 1) * kstride;
#pragma unroll
            for (int dt = 0; dt < 8; ++dt)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const float x = __bfloat162float(v[dt * 8 + 2 * c + e]);
                if (!isfinite(x)) o[dt][2 * h + e] += x;
              }
          }
      }
      const float m = h ? m1 : m0, l = h ? l1 : l0;
      if (whole) {
        const size_t at = ((size_t)b * p.T + tok) * p.Ha + tree_row_slot(row, n, g, p.k, p.G);
        const float inv = 1.f / l;
#pragma unroll
        for (int dt = 0; dt < 8; ++dt)
          *reinterpret_cast<uint32_t*>(p.O + at * 64 + dt * 8 + 2 * c) =
              pack_bf16x2(o[dt][2 * h] * inv, o[dt][2 * h + 1] * inv);
        if (p.lse && c == 0) p.lse[at] = (m + log2f(l)) * 0.6931471805599453f;
      } else {
        const size_t at = (size_t)(2 * blockIdx.x + (j0 == 0 ? 1 : 0)) * p.prow + (row - row0);
        if (c == 0) *reinterpret_cast<float2*>(p.part_ml + at * 2) = make_float2(m, l);
#pragma unroll
        for (int dt = 0; dt < 8; ++dt)
          *reinterpret_cast<float2*>(p.part_o + at * 64 + dt * 8 + 2 * c) = make_float2(o[dt][2 * h], o[dt][2 * h + 1]);
      }
    }
    if (j0 == 0 && tid == 0)
      p.unit_cta[b * U + u] = make_int2(blockIdx.x, tree_range_of(total, ranges, prefix[b] + nblk - 1) * U + u);
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();  // ring, masks and flags are free for the next sequence
  }
}

// The parts of every row that was cut, added: `kParts` groups of 16 lanes a row,
// four dimensions a lane.
constexpr int kTreeMergeThreads = 128;
template <int kParts>
__global__ void __launch_bounds__(kTreeMergeThreads) tree_merge_kernel(const TreeParams p) {
  static_assert(kParts == 2 || kParts == 8, "a warp or the block per row");
  __shared__ float s_m[kTreeMergeThreads / 16], s_l[kTreeMergeThreads / 16];
  __shared__ float4 s_o[kTreeMergeThreads];
  // (The lengths were there before the attention kernel began, and this one
  // begins when all of its blocks have: they are read before the wait for it.)
  const int tid = threadIdx.x, part = (tid >> 4) % kParts, d = tid & 15;
  constexpr int kRowsPer = kTreeMergeThreads / 16 / kParts;
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
  const int s = row / p.urows;
  pdl_wait();
  pdl_trigger();
  int2 ctas = make_int2(0, 0);
  if (on) ctas = p.unit_cta[b * (p.u0 + (p.G - 1) * p.u1) + (g == 0 ? s : p.u0 + (g - 1) * p.u1 + s)];
  on = on && ctas.x != ctas.y;  // (else it was written at once)
  float m = -INFINITY, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  if (on) {
#pragma unroll 4
    for (int c = ctas.x + part * p.step; c <= ctas.y; c += kParts * p.step) {
      const size_t at = (size_t)(2 * c + (c == ctas.x ? 1 : 0)) * p.prow + row % p.urows;
      const float2 ml = *reinterpret_cast<const float2*>(p.part_ml + at * 2);
      const float4 v = *reinterpret_cast<const float4*>(p.part_o + at * 64 + d * 4);
      // a score that is NaN leaves no maximum, and l NaN: it stays so
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
  *reinterpret_cast<uint2*>(p.O + out * 64 + d * 4) =
      make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
  if (p.lse && d == 0) p.lse[out] = (M + log2f(sum)) * 0.6931471805599453f;
}

}  // namespace gqe
