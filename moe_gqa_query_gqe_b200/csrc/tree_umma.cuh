// tree_umma.cuh -- attention of a tree of drafted tokens over a key/value cache
// on the tcgen05 tensor cores (the mathematics: tree.cuh).
//
// Units. The query rows of one (sequence, group) are cut into units of up to
// 256 rows, two tiles of 128. A unit's keys are its cached blocks of 128
// positions and one block of drafted tokens. All units' blocks, one after the
// other, are cut into gridDim.x ranges of equal weight, one persistent block of
// threads (one per SM) each: whatever the lengths and however few the
// sequences, every SM streams the same share. A unit that a range's end cuts is
// left as partial (m, l, O) rows for tree_merge_kernel, at most two of
// them per range; the others are written at once.
//
// Inside a unit two tiles A and B run side by side, each with its MMA thread
// and its four softmax warps:
//   a unit of more than 128 rows   A and B hold its two row tiles, and every
//                                  K/V block serves both;
//   else                           A and B hold the same rows and take the
//                                  range's blocks in turn.
//                                  With 64 rows or fewer a tile holds them
//                                  twice: each copy takes its half of the
//                                  block's keys (P is zero in the other), so
//                                  that all four warps share the exponentials.
//                                  Tiles and copies are added at the end.
// A pair block costs half again what a block of the second kind does (weights 3
// and 2): it is bound by exponentials, the other by the cache's bytes.
//
//   warp 0      TMA producer: K and V blocks, each through a ring of its own
//   warps 1, 2  lane 0 issues the MMAs of tile A (warp 1, also the TMEM owner)
//               or B: S = Q K^T (SS, 128x128x64) and O += P V (TS, N = 64)
//   warp 3      for a unit's draft block: the ancestor masks, by pointer
//               doubling, and which drafted values are not finite
//   warps 4..11 softmax, one thread a row: Q into shared memory at the start of
//               a unit; then per block S from TMEM, the running maximum
//               (rescaled lazily) and sum, P as bf16 into TMEM
// Bounds: one exponential a (row, position), 16 a clock and SM on the MUFU (one
// pair in kTuPolyEvery on the FMA pipe), against 256 flops: 4 x 128 tokens of two
// rows a group over 131072 positions of 8 groups take 253 us for the exponentials,
// 179 for the products and 164 for the bytes. Measured there: 531 us (550
// TFLOP/s) over several sets of inputs in turn, 476 on one set again and again. The
// two softmax warps of a scheduler wait for their own chains (issue slots 30-35%
// used, MUFU 54% of the time): a block's scores are read in three steps, and S is
// held until half of its exponentials are done. (attn2.cuh, with as many warps and
// registers, holds all 128 scores of a row and spills 8 bytes; here the loop's
// pointers and its masked forms take that room.) Sixteen warps, a row over four threads, took
// 821-855 us (96 registers a thread spill); the next scores loaded from tensor
// memory during a block's exponentials, in pieces of 32, 525 against 479 (88 bytes
// a thread spill).
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

// Stages of K and of V (held longer: until P V). Both even: outside pairs the
// tiles take turns at the blocks, and so a stage's blocks all belong to one
// tile, which sees its phases one by one.
constexpr int kTuKStages = 4, kTuVStages = 6;
constexpr int kTuThreads = 384;
constexpr int kTuRegsLow = 88, kTuRegsHigh = 208;  // 88*128 + 208*256 = 168*384
constexpr int kTuBlock = 128;                      // keys of a block
constexpr int kTuRows = 256;                       // rows of a unit
// Every n-th pair of exponentials on the FMA pipe (4 x 128 tokens of two rows a
// group over 131072 positions: 497 us with 16, 485 with 8 or 6, 476 with 4).
constexpr int kTuPolyEvery = 4;

struct TreeUmmaParams {
  CUtensorMap tmK, tmV;    // caches as [B*cap][G][64], box (64, 1, 128)
  CUtensorMap tmKn, tmVn;  // drafts as [B*T][G][64]
  TreeParams p;            // p.step = G: the groups side by side, range r of group g is block r * G + g; 1: range r is block r
};

struct TuSmem {
  static constexpr int kQ = 0;                               // Q_A, Q_B
  static constexpr int kSum = 0;                             // [256][32] fp32: half of both tiles' O, at a unit's end
  static constexpr int kK = 32768;                           // stages of K
  static constexpr int kV = kK + kTuKStages * 16384;         // stages of V
  static constexpr int kMask = kV + kTuVStages * 16384;      // [2][128] ancestor masks
  static constexpr int kUp = kMask + 2 * kTreeMax * 16;      // [128] pointers of the doubling
  static constexpr int kBad = kUp + kTreeMax * 4;            // [2][4] drafts with values that are not finite
  static constexpr int kML = kBad + 32;                      // [2][128] m, l of the tiles
  static constexpr int kWarp = kML + 2 * 128 * 8;            // [8] TuWarp of the softmax warps
  static constexpr int kPrefix = kWarp + 8 * 128;            // [B + 1] weight before each sequence
  static constexpr int kBar = kPrefix + (kTreeMaxB + 1) * 8;
  static constexpr int kBytes = kBar + 512 + 1024;
};

struct TuItem {
  int b, g, s;         // sequence, group, unit of the group
  int L, n, R;         // cached positions, drafted tokens, rows of the group
  int rows;            // rows of the unit
  int pair;            // two row tiles
  int nblk, j0, j1;    // blocks of the unit; this range's
  int unit;
  __device__ __forceinline__ int copies() const { return rows > 64 ? 1 : 2; }
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
__device__ __forceinline__ long long tu_seq_weight(int L, int n, int G, int k, bool aligned) {
  const long long nblk = (L + kTuBlock - 1) / kTuBlock + 1;
  if (aligned) return nblk * 2;
  return nblk * (tu_group_weight(n * (k + 1)) + (long long)(G - 1) * tu_group_weight(n * k));
}
// The units that a range of weight [x0, x1) holds blocks of, in order. A block
// belongs to the range that its first weight falls into.
struct TuCursor {
  long long x0, x1, base;
  int b, g, s;
  int only;  // the group that this block takes, or -1: all
  __device__ __forceinline__ void start(const TreeParams& p, const long long* prefix, long long a, long long e, int group) {
    x0 = a;
    x1 = e;
    b = tree_first(prefix, p.B, x0);
    g = s = 0;
    base = prefix[b];
    only = group;
    if (group >= 0) {
      g = group;
      return;
    }
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
        if (only >= 0) {
          ++b;
        } else if (it.n == 0 || ++g == p.G) {
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
      it.unit = b * (p.u0 + (p.G - 1) * p.u1) + (g == 0 ? s : p.u0 + (g - 1) * p.u1 + s);
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

// 2^x for a pair on the FMA pipe, to 2.7e-6 relative for -126 < x < 128: as
// exp2_poly2 of attn2.cuh with a polynomial of degree 4 (fit_exp2_poly.py), for
// the log-sum in fp32 beside O. From -126 down (-infinity too) the result is a
// subnormal number, 2^-126 / sqrt(2) at least: nothing to a softmax, whose largest term is
// near 1, and zero once added with fadd2_ftz. Not for x >= 128, nor for NaN.
__device__ __forceinline__ void exp2_poly4(float& y0, float& y1, float x0, float x1) {
  constexpr float kShift = 12582912.0f;  // 1.5 * 2^23
  constexpr float c0 = 9.999992847e-01f, c1 = 6.931217909e-01f, c2 = 2.402474433e-01f, c3 = 5.591785908e-02f,
                  c4 = 9.570102207e-03f;
  x0 = fmaxf(x0, -126.5f);  // (halfway to the even exponent -126, so that the bits below stay positive)
  x1 = fmaxf(x1, -126.5f);
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

// Sums of a pair; subnormal terms and sums are zero.
__device__ __forceinline__ void fadd2_ftz(float& d0, float& d1, float a0, float a1, float b0, float b1) {
  asm("{\n\t.reg .b64 ra, rb, rd;\n\t"
      "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
      "add.rn.ftz.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
      : "=f"(d0), "=f"(d1)
      : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}

constexpr int kTuPiece = 4;  // columns a thread finishes at a time
__device__ __forceinline__ void tmem_ld4(uint32_t taddr, uint32_t (&r)[4]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(taddr)
      : "memory");
}

// Three-way maximum that keeps NaN.
__device__ __forceinline__ float fmax3_nan(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// A softmax warp's place in its range, in shared memory: in registers it pushed
// the scores out of them.
struct TuWarp {
  TuCursor cur;
  TuItem it;
  int more;
};
static_assert(sizeof(TuWarp) <= 128, "its slot");
__device__ __forceinline__ TuItem tu_item(const TuWarp* w) {  // read anew at every call
  TuItem it;
  const volatile int* src = reinterpret_cast<const volatile int*>(&w->it);
  int* dst = reinterpret_cast<int*>(&it);
#pragma unroll
  for (int i = 0; i < (int)(sizeof(TuItem) / 4); ++i) dst[i] = src[i];
  return it;
}

// The sum of the values in a column of `rows` cached rows that are not finite;
// `none` where there are none. Rarely called; with numbers for arguments, since
// references to the caller's structures kept those in local memory (8 x 128 tokens
// over 32K 158 us instead of 151).
__device__ __noinline__ float tu_not_finite(const __nv_bfloat16* v, int rows, uint32_t stride, float none) {
  float sum = 0.f;
#pragma unroll 8
  for (int s = 0; s < rows; ++s, v += stride) {
    const float x = __bfloat162float(*v);
    if (!isfinite(x)) sum += x;
  }
  return sum == 0.f ? none : sum;
}

// The barriers and tensor-memory addresses of one tile's softmax warps.
struct TuTile {
  uint64_t *s_free, *pv_done, *p_full;
  volatile int* abort_flag;
  uint32_t tm_s, tm_o, tm_p;
  float sl2;
};

// Sixty-four columns of S in registers.
template <bool kMasked>
__device__ __forceinline__ void tu_scores(uint32_t taddr, uint32_t b0, uint32_t b1, float (&s)[64]) {
  uint32_t r[64];
  tmem_ld64(taddr, r);
#pragma unroll
  for (int i = 0; i < 64; ++i) {
    s[i] = __uint_as_float(r[i]);
    if constexpr (kMasked)
      if (!(((i < 32 ? b0 : b1) >> (i & 31)) & 1u)) s[i] = -INFINITY;
  }
}
__device__ __forceinline__ float tu_max(const float (&s)[64]) {
  float m4[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
  for (int c = 4; c < 64; c += 8) {
    m4[0] = fmax3_nan(m4[0], s[c], s[c + 1]);
    m4[1] = fmax3_nan(m4[1], s[c + 2], s[c + 3]);
    if (c + 4 < 64) {
      m4[2] = fmax3_nan(m4[2], s[c + 4], s[c + 5]);
      m4[3] = fmax3_nan(m4[3], s[c + 6], s[c + 7]);
    }
  }
  return fmax3_nan(fmax3_nan(m4[0], m4[1], m4[1]), m4[2], m4[3]);
}
// P of sixty-four columns, as bf16 pairs; their sum is returned.
template <bool kPoly>
__device__ __forceinline__ float tu_exp(const float (&s)[64], float sl2, float mu, uint32_t (&pk)[32]) {
  float sm[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int pi = 0; pi < 32; ++pi) {
    float x0, x1, y0, y1;
    ffma2(x0, x1, s[2 * pi], s[2 * pi + 1], sl2, sl2, -mu, -mu);
    if (kPoly && (pi % kTuPolyEvery) == kTuPolyEvery - 1) {
      exp2_poly4(y0, y1, x0, x1);
    } else {
      y0 = ex2_approx(x0);
      y1 = ex2_approx(x1);
    }
    fadd2(sm[2 * (pi & 3)], sm[2 * (pi & 3) + 1], sm[2 * (pi & 3)], sm[2 * (pi & 3) + 1], y0, y1);
    pk[pi] = pack_bf16x2(y0, y1);
  }
  return ((sm[0] + sm[1]) + (sm[2] + sm[3])) + ((sm[4] + sm[5]) + (sm[6] + sm[7]));
}
__device__ __forceinline__ void tu_store_p(uint32_t taddr, const uint32_t (&pk)[32]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t r[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) r[i] = pk[h * 16 + i];
    tmem_st16(taddr + h * 16, r);
  }
}

// One block of keys for a thread's row: its 128 / D scores (columns col0 on),
// softmax, P. With kMasked the row sees the keys of `mk` only (a function of its
// own: as a condition the comparisons were issued for every block). The scores
// are taken sixty-four at a time, the first half twice: all 128 in registers
// spill 116 bytes a thread and take a sixth longer (4 x 128 tokens of two rows
// a group over 131072 positions: 562 us against 478).
// First: the unit's first block of this tile.
template <int D, bool kMasked>
__device__ __forceinline__ bool tu_block(const TuTile& T, int col0, const uint4& mk, bool first, uint32_t cnt,
                                         float& m_run, float& l_run) {
  // (a masked place must be exactly zero: MUFU only; with copies the
  // exponentials bind nothing)
  constexpr bool kPoly = D == 1 && !kMasked;
  float s[64];
  float mx = -INFINITY;
  if constexpr (D == 1) {
    tu_scores<kMasked>(T.tm_s, mk.x, mk.y, s);
    mx = tu_max(s);
  }
  const bool low = D == 1 || col0 == 0;  // (D = 2: the copy's columns)
  tu_scores<kMasked>(T.tm_s + (D == 1 ? 64 : col0), D == 1 || !low ? mk.z : mk.x, D == 1 || !low ? mk.w : mk.y, s);
  if constexpr (D == 2) {
    tc_fence_before();
    mbar_arrive(T.s_free);  // S may be overwritten by the next block's QK^T now
  }
  {
    const float m2 = tu_max(s);
    mx = fmax3_nan(mx, m2, m2);
  }
  const float m_new = fmaxf(m_run, mx * T.sl2);
  const float m_use = (m_new > m_run + kRescaleThreshold) ? m_new : m_run;
  const float mu = m_use == -INFINITY ? 0.f : m_use;  // (nothing seen yet)
  const float alpha = ex2_approx(m_run - mu);
  const bool rescale = !first && m_use != m_run;
  m_run = m_use;
  uint32_t pk[32];
  l_run = l_run * alpha + tu_exp<kPoly>(s, T.sl2, mu, pk);
  if (!(mx < INFINITY)) l_run = __int_as_float(0x7fffffff);  // a score that is NaN or +inf: the row is NaN
  if (!first) {
    const bool w_ok = mbar_wait(T.pv_done, (cnt - 1) & 1, T.abort_flag);
    if (!__all_sync(0xffffffffu, w_ok)) return false;
    tc_fence_after();
    if (__any_sync(0xffffffffu, rescale)) {
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        uint32_t o[16];
        tmem_ld16(T.tm_o + h * 16, o);
#pragma unroll
        for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
        tmem_st16(T.tm_o + h * 16, o);
      }
    }
  }
  tu_store_p(T.tm_p + (D == 1 ? 32 : col0 / 2), pk);
  if constexpr (D == 1) {
    tu_scores<kMasked>(T.tm_s, mk.x, mk.y, s);
    tc_fence_before();
    mbar_arrive(T.s_free);
    l_run += tu_exp<kPoly>(s, T.sl2, mu, pk);
    tu_store_p(T.tm_p, pk);
  }
  tc_fence_before();
  mbar_arrive(T.p_full);
  return true;
}

// A tile's blocks of a unit, for one thread: all that the loop needs of the unit.
struct TuUnit {
  TuTile T;
  uint64_t *s_full, *mask_full, *v_full;
  uint8_t* v_row;       // this thread's row of V's first stage
  const uint4* mask;    // its token's ancestors
  const uint32_t* bad;  // the word of s_bad with its V row
  uint32_t mask_parity;
  int first, nj, stride;  // blocks first, first + stride, ... below nj
  int jdraft, left;       // the drafts' block; cached positions from the range's first block on
  int n, row, col0;
  bool warp_on;
  uint32_t kv, cnt;  // blocks before the unit: of the range, of the tile
  float m, l;
};
template <int D>
__device__ __forceinline__ bool tu_unit(TuUnit& u) {
  const TuTile T = u.T;
  float m_run = -INFINITY, l_run = 0.f;
  uint32_t cnt = u.cnt;
  const int first = u.first, nj = u.nj, stride = u.stride;
  bool ok = true;
  for (int jj = first; jj < nj; jj += stride, ++cnt) {
    const bool drafts = jj == u.jdraft;
    const int valid = drafts ? u.n : min(kTuBlock, u.left - jj * kTuBlock);
    bool w_ok = !drafts || mbar_wait(u.mask_full, u.mask_parity, T.abort_flag);
    if (w_ok && (valid < kTuBlock || drafts)) {
      // this thread's value row: zeroed past the last valid one; without the
      // values that are not finite in a drafted row
      const uint32_t kvj = u.kv + jj;
      w_ok = mbar_wait(&u.v_full[kvj % kTuVStages], (kvj / kTuVStages) & 1, T.abort_flag);
      uint8_t* vs = u.v_row + (kvj % kTuVStages) * 16384;
      if (w_ok && u.row >= valid) {
#pragma unroll
        for (int c = 0; c < 8; ++c) *reinterpret_cast<uint4*>(vs + 16 * c) = make_uint4(0u, 0u, 0u, 0u);
      } else if (w_ok && drafts && ((*u.bad >> (u.row & 31)) & 1u)) {
        for (int c = 0; c < 32; ++c) {
          uint32_t w = *reinterpret_cast<uint32_t*>(vs + 4 * c);
          if ((w & 0x7f80u) == 0x7f80u) w &= 0xffff0000u;
          if ((w & 0x7f800000u) == 0x7f800000u) w &= 0x0000ffffu;
          *reinterpret_cast<uint32_t*>(vs + 4 * c) = w;
        }
      }
      fence_proxy_async_smem();
    }
    w_ok = w_ok && mbar_wait(u.s_full, cnt & 1, T.abort_flag);
    if (!__all_sync(0xffffffffu, w_ok)) { ok = false; break; }
    tc_fence_after();
    if (!u.warp_on) {
      // P of rows that are not stored may hold anything; the arrival must not
      // fall into the block before, though
      tc_fence_before();
      mbar_arrive(T.s_free);
      w_ok = jj == first || mbar_wait(T.pv_done, (cnt - 1) & 1, T.abort_flag);
      if (!__all_sync(0xffffffffu, w_ok)) { ok = false; break; }
      mbar_arrive(T.p_full);
      continue;
    }
    if (drafts || valid < kTuBlock) {
      uint4 mk;
      if (drafts) {
        mk = *u.mask;
      } else {  // the first `valid` of the block
        auto word = [&](int w) { return valid >= 32 * w + 32 ? 0xffffffffu : (valid <= 32 * w ? 0u : (1u << (valid - 32 * w)) - 1u); };
        mk = make_uint4(word(0), word(1), word(2), word(3));
      }
      ok = tu_block<D, true>(T, u.col0, mk, jj == first, cnt, m_run, l_run);
    } else {
      ok = tu_block<D, false>(T, u.col0, make_uint4(0u, 0u, 0u, 0u), jj == first, cnt, m_run, l_run);
    }
    if (!ok) break;
  }
  u.cnt = cnt;
  u.m = m_run;
  u.l = l_run;
  return ok;
}

__global__ void __launch_bounds__(kTuThreads, 1) tree_attn_umma_kernel(const __grid_constant__ TreeUmmaParams P) {
  using S = TuSmem;
  const TreeParams& p = P.p;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S::kBar);
  uint64_t* k_full = bars;                   // [kTuKStages]
  uint64_t* v_full = k_full + kTuKStages;    // [kTuVStages]
  uint64_t* k_empty = v_full + kTuVStages;   // [kTuKStages] two arrivals: each tile's, or two of the tile whose block it is
  uint64_t* v_empty = k_empty + kTuKStages;  // [kTuVStages]
  uint64_t* q_full = v_empty + kTuVStages;   // [2] tiles
  uint64_t* s_full = q_full + 2;            // [2]
  uint64_t* s_free = s_full + 2;            // [2]
  uint64_t* p_full = s_free + 2;            // [2]
  uint64_t* pv_done = p_full + 2;           // [2]
  uint64_t* mask_full = pv_done + 2;        // [2] buffers
  uint64_t* mask_empty = mask_full + 2;     // [2]
  uint64_t* both = mask_empty + 2;          // both tiles' softmax threads meet
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(both + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  long long* prefix = reinterpret_cast<long long*>(smem + S::kPrefix);
  uint4* s_mask = reinterpret_cast<uint4*>(smem + S::kMask);
  uint32_t* s_bad = reinterpret_cast<uint32_t*>(smem + S::kBad);
  float2* s_ml = reinterpret_cast<float2*>(smem + S::kML);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int s = 0; s < kTuKStages; ++s) {
      mbar_init(&k_full[s], 1);
      mbar_init(&k_empty[s], 2);
    }
    for (int s = 0; s < kTuVStages; ++s) {
      mbar_init(&v_full[s], 1);
      mbar_init(&v_empty[s], 2);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&q_full[t], 128);
      mbar_init(&s_full[t], 1);
      mbar_init(&s_free[t], 128);
      mbar_init(&p_full[t], 128);
      mbar_init(&pv_done[t], 1);
      mbar_init(&mask_full[t], 32);
      mbar_init(&mask_empty[t], 256);
    }
    mbar_init(both, 256);
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
  tree_prefix<kTuThreads>(p, prefix, [&](int L, int n) { return tu_seq_weight(L, n, p.G, p.k, p.step > 1); });
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const uint32_t sbase = smem_u32(smem);
  // ranges: `step` blocks of threads (one a group, or one) take each; none is
  // below the weight of a block, so that every range inside a unit holds one
  const long long total = prefix[p.B];
  const int step = p.step, cta = blockIdx.x;
  const int grid = (int)max(1ll, min((long long)(gridDim.x / step), total / 3));
  const int range = min(cta / step, grid);
  TuCursor cur;
  cur.start(p, prefix, tree_range(total, range, grid), tree_range(total, min(range + 1, grid), grid), step > 1 ? cta % step : -1);
  TuItem it = {};

  if (warp < 4) {
    setmaxnreg_dec<kTuRegsLow>();
    if (warp == 0 && lane == 0) {
      // ---- producer: K and V each as soon as their own stage is free (K's is when
      // its scores are done, long before V's) ----------------------------------------
      struct Stream {
        TuCursor cur;
        TuItem it;
        int j;
        uint32_t n;
        bool done;
      };
      Stream str[2] = {{cur, it, 0, 0, false}, {cur, it, 0, 0, false}};
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        str[v].done = !str[v].cur.next(P, str[v].it);
        if (!str[v].done) str[v].j = str[v].it.j0;
      }
      unsigned long long idle = 0;  // since when neither could go on
      for (uint32_t spin = 0; !(str[0].done && str[1].done); ++spin) {
        bool moved = false;
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          Stream& a = str[v];
          const uint32_t stages = v ? kTuVStages : kTuKStages, s = a.n % stages;
          if (a.done || !mbar_test(v ? &v_empty[s] : &k_empty[s], ((a.n / stages) & 1) ^ 1)) continue;
          const bool drafts = a.j == a.it.nblk - 1;
          const int row = drafts ? a.it.b * p.T : a.it.b * p.cap + a.j * kTuBlock;
          uint64_t* full = v ? &v_full[s] : &k_full[s];
          mbar_arrive_expect_tx(full, 16384);
          tma_load_3d(smem + (v ? S::kV : S::kK) + s * 16384, v ? (drafts ? &P.tmVn : &P.tmV) : (drafts ? &P.tmKn : &P.tmK),
                      full, 0, a.it.g, row);
          ++a.n;
          moved = true;
          if (++a.j == a.it.j1) {
            a.done = !a.cur.next(P, a.it);
            if (!a.done) a.j = a.it.j0;
          }
        }
        if (moved) {
          idle = 0;
        } else if ((spin & 63u) == 0) {
          if (*abort_flag) break;
          const unsigned long long now = globaltimer_ns();
          if (idle == 0) idle = now;
          if (now - idle > kWaitTimeoutNs) {
            *abort_flag = 1;
            atomicExch(&g_error_word, kDevErrTimeout);
            break;
          }
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
      auto s_ready = [&](uint32_t kvi) {
        return mbar_test(&k_full[kvi % kTuKStages], (kvi / kTuKStages) & 1) &&
               (s_cnt == 0 || mbar_test(&s_free[t], (s_cnt - 1) & 1));
      };
      auto issue_s = [&](uint32_t kvi, bool alone) {  // (ready)
        tc_fence_after();
        const uint32_t ka = sbase + S::kK + (kvi % kTuKStages) * 16384;
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          umma_ss(tmem_base + t * 128, sdesc_sw128(qa + kk * 32, 16, 1024), sdesc_sw128(ka + kk * 32, 16, 1024), idesc_s,
                  kk != 0);
        umma_commit(&s_full[t]);
        umma_commit(&k_empty[kvi % kTuKStages]);
        if (alone) umma_commit(&k_empty[kvi % kTuKStages]);
        ++s_cnt;
      };
      auto wait_s = [&](uint32_t kvi) {
        return mbar_wait(&k_full[kvi % kTuKStages], (kvi / kTuKStages) & 1, abort_flag) &&
               (s_cnt == 0 || mbar_wait(&s_free[t], (s_cnt - 1) & 1, abort_flag));
      };
      while (ok && cur.next(P, it)) {
        const int nj = it.j1 - it.j0;
        const int stride = it.pair ? 1 : 2, first = it.pair ? 0 : (int)((kv & 1) ^ t);
        // (q_full counts the units that have a block of this tile: in the others
        // neither side waits for the other, and their phases could drift apart)
        if (first < nj) {
          if (!(ok = mbar_wait(&q_full[t], q_cnt & 1, abort_flag) && wait_s(kv + first))) break;
          ++q_cnt;
          issue_s(kv + first, !it.pair);
        }
        for (int jj = first; jj < nj; jj += stride) {
          const uint32_t kvj = kv + jj;
          // the next block's scores as soon as its K is there, but P V does not
          // wait for them: V's stage is what the loads behind it wait for
          bool ahead = jj + stride < nj;
          for (uint32_t i = 0; ahead && i < 100000000u && !mbar_test(&p_full[t], pv_cnt & 1); ++i) {
            if (s_ready(kvj + stride)) {
              issue_s(kvj + stride, !it.pair);
              ahead = false;
            } else if ((i & 1023u) == 1023u && *abort_flag) {
              break;
            }
          }
          if (!(ok = mbar_wait(&p_full[t], pv_cnt & 1, abort_flag))) break;
          if (!(ok = mbar_wait(&v_full[kvj % kTuVStages], (kvj / kTuVStages) & 1, abort_flag))) break;
          tc_fence_after();
          const uint32_t va = sbase + S::kV + (kvj % kTuVStages) * 16384;
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            umma_ts(tmem_base + 256 + t * 64, tmem_base + 384 + t * 64 + kk * 8, sdesc_sw128(va + kk * 2048, 8192, 1024),
                    idesc_o, (jj != first || kk != 0) ? 1u : 0u);
          umma_commit(&pv_done[t]);
          ++pv_cnt;
          umma_commit(&v_empty[kvj % kTuVStages]);
          if (!it.pair) umma_commit(&v_empty[kvj % kTuVStages]);
          if (ahead) {
            if (!(ok = wait_s(kvj + stride))) break;
            issue_s(kvj + stride, !it.pair);
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
    const TuTile T = {&s_free[t], &pv_done[t], &p_full[t], abort_flag, tmem_base + lane_off + t * 128,
                      tmem_base + lane_off + 256 + t * 64, tmem_base + lane_off + 384 + t * 64, p.scale_log2};
    float4* sums = reinterpret_cast<float4*>(smem + S::kSum);
    uint32_t kv = 0;   // blocks of the range before this unit's
    uint32_t cnt = 0;  // blocks that this tile has processed
    uint32_t masks = 0, meets = 0;
    bool ok = true;
    // all 256 softmax threads
    auto meet = [&]() -> bool {
      mbar_arrive(both);
      const bool w_ok = mbar_wait(both, meets & 1, abort_flag);
      ++meets;
      return __all_sync(0xffffffffu, w_ok);
    };
    TuWarp* place = reinterpret_cast<TuWarp*>(smem + S::kWarp + (warp - 4) * 128);
    if (lane == 0) place->cur = cur;
    while (ok) {
      if (lane == 0) place->more = place->cur.next(P, place->it);
      __syncwarp();
      if (!*reinterpret_cast<volatile int*>(&place->more)) break;
      TuItem it = tu_item(place);
      const int nj = it.j1 - it.j0;
      const int stride = it.pair ? 1 : 2, first = it.pair ? 0 : (int)((kv & 1) ^ t);
      const int D = it.copies(), width = 128 / D;      // rows a copy has room for
      const int copy = row / width;
      int base = it.row_base(t);
      int nrow = min(width, it.R - base);              // rows of this tile
      const bool warp_on = q * 32 % width < nrow;
      int rc = min(base + row % width, it.R - 1);      // (rows past the last repeat it and are not stored)
      int tok = tree_row_token(rc, it.n, p.k), slot = tree_row_slot(rc, it.n, it.g, p.k, p.G);
      size_t out = ((size_t)it.b * p.T + tok) * p.Ha + slot;
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
        if (D > 1) {
          // P of the keys that are other copies': zero for the whole unit
          const uint32_t z[16] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
#pragma unroll
          for (int h = 0; h < 4; ++h) tmem_st16(T.tm_p + h * 16, z);
        }
        if (first < nj) mbar_arrive(&q_full[t]);
      }
      TuUnit U;
      U.T = T;
      U.s_full = &s_full[t];
      U.mask_full = &mask_full[masks & 1];
      U.v_full = v_full;
      U.v_row = smem + S::kV + row * 128;
      U.mask = s_mask + (masks & 1) * kTreeMax + tok;
      U.bad = s_bad + (masks & 1) * 4 + (row >> 5);
      U.mask_parity = (masks >> 1) & 1;
      U.first = first;
      U.nj = nj;
      U.stride = stride;
      U.jdraft = it.nblk - 1 - it.j0;
      U.left = it.L - it.j0 * kTuBlock;
      U.n = it.n;
      U.row = row;
      U.col0 = copy * width;
      U.warp_on = warp_on;
      U.kv = kv;
      U.cnt = cnt;
      ok = D == 1 ? tu_unit<1>(U) : tu_unit<2>(U);
      cnt = U.cnt;
      const float m_run = U.m, l_run = U.l;
      if (!ok) break;
      it = tu_item(place);
      base = it.row_base(t);
      nrow = min(width, it.R - base);
      rc = min(base + row % width, it.R - 1);
      tok = tree_row_token(rc, it.n, p.k);
      slot = tree_row_slot(rc, it.n, it.g, p.k, p.G);
      out = ((size_t)it.b * p.T + tok) * p.Ha + slot;
      const int mine = first < nj ? 1 : 0;  // has blocks
      // ---- the unit's end ------------------------------------------------------------
      bool w_ok = mine == 0 || mbar_wait(&pv_done[t], (cnt - 1) & 1, abort_flag);
      // the drafts that are not finite and their masks (waited for already by
      // the tile whose block it was)
      const bool fix = it.has_drafts();
      w_ok = w_ok && (!fix || mbar_wait(&mask_full[masks & 1], (masks >> 1) & 1, abort_flag));
      if (!__all_sync(0xffffffffu, w_ok)) { ok = false; break; }
      tc_fence_after();
      const bool whole = it.whole();
      // what a thread writes: columns c0 .. c0 + nc - 1 of either half of row `wrow`
      int wrow = row, c0 = 0, nc = 32, wslot = slot, wtok = tok;
      size_t wout = out;
      float M = m_run, l = l_run, f = 1.f;
      if (!it.pair) {
        // tiles and copies are added through shared memory: (m, l) of each,
        // then each O scaled to the common maximum
        s_ml[t * 128 + row] = make_float2(m_run, l_run);
        if (!(ok = meet())) break;  // (Q of both tiles is no longer read, either)
        float Mx = -INFINITY;
        for (int i = row % width; i < 256; i += width) Mx = fmaxf(Mx, s_ml[i].x);
        f = mine == 0 ? 0.f : ex2_approx(m_run - (Mx == -INFINITY ? 0.f : Mx));
        // 256 threads over `width` rows: 256 / width threads a row
        const int tix = t * 128 + row, per = 256 / width;
        wrow = tix / per;
        nc = 32 / per;  // of each half
        c0 = (tix % per) * nc;
        M = -INFINITY;
        for (int i = wrow; i < 256; i += width) M = fmaxf(M, s_ml[i].x);
        l = 0.f;
        for (int i = wrow; i < 256; i += width) {
          const float2 ml = s_ml[i];
          // (a tile without blocks has m = -inf, l = 0)
          l += ml.y * (ml.y == 0.f ? 0.f : ex2_approx(ml.x - (M == -INFINITY ? 0.f : M)));
        }
        const int wc = min(base + wrow, it.R - 1);
        wtok = tree_row_token(wc, it.n, p.k);
        wslot = tree_row_slot(wc, it.n, it.g, p.k, p.G);
        wout = ((size_t)it.b * p.T + wtok) * p.Ha + wslot;
      }
      const bool live = wrow < nrow;
      const float inv = whole ? 1.f / l : 1.f;
      const uint32_t part = (2 * cta + (it.j0 == 0 ? 1 : 0)) * p.prow + (it.pair ? t * 128 : 0) + wrow;
      uint4 mk = make_uint4(0u, 0u, 0u, 0u);
      if (fix) {
        const uint4 bd = *reinterpret_cast<const uint4*>(s_bad + (masks & 1) * 4);
        mk = s_mask[(masks & 1) * kTreeMax + wtok];
        mk = make_uint4(mk.x & bd.x, mk.y & bd.y, mk.z & bd.z, mk.w & bd.w);
      }
      const bool any_bad = (mk.x | mk.y | mk.z | mk.w) != 0u;
      for (int h = 0; h < 2; ++h) {
        if (!it.pair) {
          // this half of the columns of every row, scaled
          if (h == 1 && !(ok = meet())) break;  // (the first half is read)
          if (warp_on) {
            uint32_t a[32];
            if (mine > 0) tmem_ld32(T.tm_o + h * 32, a);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
              if (mine > 0)
                v = make_float4(__uint_as_float(a[4 * i]) * f, __uint_as_float(a[4 * i + 1]) * f,
                                __uint_as_float(a[4 * i + 2]) * f, __uint_as_float(a[4 * i + 3]) * f);
              sums[(t * 128 + row) * 8 + (i ^ (row & 7))] = v;
            }
          }
          if (!(ok = meet())) break;
        }
        for (int c = h * 32 + c0; c < h * 32 + c0 + nc; c += kTuPiece) {
        float o[kTuPiece];
        if (it.pair) {
          if (!warp_on) break;
          __syncwarp();  // (whole again after the rows' own branches)
          uint32_t a[kTuPiece];
          tmem_ld4(T.tm_o + c, a);
#pragma unroll
          for (int i = 0; i < kTuPiece; ++i) o[i] = __uint_as_float(a[i]);
        } else {
#pragma unroll
          for (int i = 0; i < kTuPiece; ++i) o[i] = 0.f;
          for (int i = wrow; i < 256; i += width) {
            const float4 a = sums[i * 8 + (((c & 31) >> 2) ^ (i & 7))];
            o[0] += a.x;
            o[1] += a.y;
            o[2] += a.z;
            o[3] += a.w;
          }
          // With two copies a tile the zero weights of the other copy's keys times a
          // cached value that is infinite are NaN. A row whose sum is a number has only
          // numbers for weights, so that such values alone make its columns NaN or
          // infinite: their sum is the column.
          const float all = (o[0] + o[1]) + (o[2] + o[3]);
          if (all != all && l == l) {
#pragma unroll
            for (int i = 0; i < kTuPiece; ++i)
              if (o[i] != o[i])
                o[i] = tu_not_finite(p.Vc + (((size_t)it.b * p.cap + it.j0 * kTuBlock) * p.G + it.g) * 64 + c + i,
                                     min(it.L, it.j1 * kTuBlock) - it.j0 * kTuBlock, p.G * 64, o[i]);
          }
        }
        if (any_bad && live) {
          for (int w = 0; w < 4; ++w)
            for (uint32_t bits = mask_word(mk, w); bits; bits &= bits - 1) {
              const __nv_bfloat16* v = p.Vn + (((size_t)it.b * p.T + w * 32 + __ffs(bits) - 1) * p.G + it.g) * 64 + c;
#pragma unroll
              for (int i = 0; i < kTuPiece; ++i) {
                const float x = __bfloat162float(v[i]);
                if (!isfinite(x)) o[i] += x;
              }
            }
        }
        if (live && whole)
          *reinterpret_cast<uint2*>(p.O + wout * 64 + c) =
              make_uint2(pack_bf16x2(o[0] * inv, o[1] * inv), pack_bf16x2(o[2] * inv, o[3] * inv));
        else if (live)
          *reinterpret_cast<float4*>(p.part_o + (size_t)part * 64 + c) = make_float4(o[0], o[1], o[2], o[3]);
        }
      }
      if (!ok) break;
      if (live && c0 == 0) {
        if (!whole)
          *reinterpret_cast<float2*>(p.part_ml + (size_t)part * 2) = make_float2(M, l);
        else if (p.lse)
          p.lse[wout] = (M + log2f(l)) * 0.6931471805599453f;
      }
      if (t == 0 && row == 0 && it.j0 == 0) {
        // the ranges that hold blocks of this unit
        const long long ubase = place->cur.base - (long long)it.nblk * tu_weight(it.rows);
        p.unit_cta[it.unit] =
            make_int2(cta, tree_range_of(total, grid, ubase + (long long)(it.nblk - 1) * tu_weight(it.rows)) * step +
                               (step > 1 ? cta % step : 0));
      }
      tc_fence_before();
      if (fix) {
        mbar_arrive(&mask_empty[masks & 1]);
        ++masks;
      }
      // the sums are read: the next unit's Q may take their place
      if (!it.pair && !(ok = meet())) break;
      kv += it.j1 - it.j0;
      __syncwarp();
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

}  // namespace gqe
