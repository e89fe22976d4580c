// rope.cuh -- norms of the queries and keys of each head and the rotation by
// position, in one pass over Q and K.
//
//   y = x * rsqrt(mean(x^2) + eps) * w[head]          (x itself without weights)
//   (a, b) -> (a c - b s, b c + a s) for every pair i < rot/2 of the head,
//   c = scale * cos(pos * inv_freq[i]), s = scale * sin(pos * inv_freq[i])
//
// The query row of slot (g, j) takes the weight of the expert it belongs to,
// head g*M + sel[n, g, j]; the shared row takes the last. Everything between
// the bf16 input and the bf16 output is fp32: the result is rounded once.
//
// Angles: pos * inv_freq reaches 10^6 radians and more at far positions, where
// an fp32 product has lost the angle (spacing 0.06). The turns pos * inv_freq /
// 2 pi are taken in fp64, reduced to [-1/2, 1/2], and only then rounded to
// fp32 for sincospi: one fp64 multiply, one subtraction and one rounding for
// each (token, pair), shared by all heads of the token.
//
// Work: memory-bound, 256 bytes a head (read and written once). Four lanes hold
// a head, 16 elements (two 16-byte chunks) each, so that a rotation's partners
// are in one thread: with half = rot/2 a multiple of eight, lane l < half/8
// takes chunks l and l + half/8, and the other lanes the chunks that are not
// rotated, two by two; neighbouring pairs are in one chunk anyhow. Only other
// values of half go through shared memory. A block takes `tpb` tokens, whose
// cosines and sines it computes once into shared memory while its first loads
// are in flight.
#pragma once

#include "sm100.cuh"

namespace gqe {

constexpr int kRopeThreads = 256;
constexpr int kRopeBatch = 2;      // head rows a thread loads before it uses the first
constexpr int kRopeMaxTpb = 16;    // tokens a block takes at most

enum : int { kRopeInterleaved = 0, kRopeHalf8 = 1, kRopeHalfAny = 2 };

struct RopeParams {
  const __nv_bfloat16 *Q, *K;    // [N, Ha, 64], [N, G, 64]; null: that side is absent
  const __nv_bfloat16 *wq, *wk;  // [G*M + 1, 64], [G, 64]; null: no norm on that side
  const int32_t* sel;            // [N, G, k]
  const float* inv_freq;         // [rot/2]
  const int32_t* positions;      // [N], or null: t = n % T
  __nv_bfloat16 *Qo, *Ko;
  float eps, scale;
  int N, T, G, M, k, Ha, Hq, Hk;  // Hq = Ha or 0, Hk = G or 0
  int rot, tpb;
  int log2k;
  uint32_t inv_H;  // ceil(2^20 / (Hq + Hk)): row / H as a multiply, exact for rows < 2^20 / H
};

template <int kLayout>
__global__ void __launch_bounds__(kRopeThreads) qk_rope_kernel(const RopeParams p) {
  __shared__ float2 s_cs[kRopeMaxTpb][32];
  __shared__ float s_row[kLayout == kRopeHalfAny ? kRopeThreads * 16 : 1];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x;
  const int l4 = tid & 3, grp = tid >> 2;  // lane of the head, head row of the pass
  const int H = p.Hq + p.Hk;
  const int n0 = blockIdx.x * p.tpb;
  const int ntok = min(p.tpb, p.N - n0);
  const int rows = ntok * H;
  const int half = p.rot >> 1;
  constexpr int kPass = kRopeThreads / 4;
  // this lane's two chunks of eight elements
  int c0 = l4, c1 = l4 + 4;
  bool turns_here = true;  // (half layout) the chunks are each other's partners
  if constexpr (kLayout == kRopeHalf8) {
    const int hc = half >> 3;
    turns_here = l4 < hc;
    c0 = turns_here ? l4 : 2 * l4;
    c1 = turns_here ? l4 + hc : 2 * l4 + 1;
  }
  uint4 buf[kRopeBatch][2];
  auto load = [&](int base) {
#pragma unroll
    for (int u = 0; u < kRopeBatch; ++u) {
      const int r = base + u * kPass + grp;
      if (r < rows) {
        const int t = (int)(((uint32_t)r * p.inv_H) >> 20), h = r - t * H;
        const size_t n = (size_t)n0 + t;
        const __nv_bfloat16* src = h < p.Hq ? p.Q + (n * p.Ha + h) * 64 : p.K + (n * p.G + (h - p.Hq)) * 64;
        buf[u][0] = reinterpret_cast<const uint4*>(src)[c0];
        buf[u][1] = reinterpret_cast<const uint4*>(src)[c1];
      }
    }
  };
  load(0);
  for (int i = tid; i < ntok * 32; i += kRopeThreads) {
    const int t = i >> 5, f = i & 31;
    if (f < half) {
      const int n = n0 + t;
      const int pos = p.positions ? p.positions[n] : n % p.T;
      double turns = (double)pos * ((double)p.inv_freq[f] * 0.15915494309189533577);
      turns -= rint(turns);
      float s, c;
      sincospif((float)(2.0 * turns), &s, &c);
      s_cs[t][f] = make_float2(c * p.scale, s * p.scale);
    }
  }
  __syncthreads();
  for (int base = 0; base < rows; base += kPass * kRopeBatch) {
    uint4 cur[kRopeBatch][2];
#pragma unroll
    for (int u = 0; u < kRopeBatch; ++u) {
      cur[u][0] = buf[u][0];
      cur[u][1] = buf[u][1];
    }
    load(base + kPass * kRopeBatch);
#pragma unroll
    for (int u = 0; u < kRopeBatch; ++u) {
      const int r = base + u * kPass + grp;
      // a warp holds eight rows; shuffles need all of its lanes
      if (!__any_sync(0xffffffffu, r < rows)) break;
      const bool live = r < rows;
      const int rr = live ? r : rows - 1;
      const int t = (int)(((uint32_t)rr * p.inv_H) >> 20), h = rr - t * H;
      const size_t n = (size_t)n0 + t;
      const bool is_q = h < p.Hq;
      const __nv_bfloat16* wt = is_q ? p.wq : p.wk;
      uint4 wv[2];
      if (wt != nullptr) {
        int head = h - p.Hq;
        if (is_q) {
          head = p.G * p.M;
          if (h < p.G * p.k) {
            const int e = p.sel[n * (p.G * p.k) + h];
            if (e < 0 || e >= p.M) flag_bounds_error();
            head = (h >> p.log2k) * p.M + min(max(e, 0), p.M - 1);
          }
        }
        wv[0] = reinterpret_cast<const uint4*>(wt + (size_t)head * 64)[c0];
        wv[1] = reinterpret_cast<const uint4*>(wt + (size_t)head * 64)[c1];
      }
      float y[2][8];
      float ss = 0.f;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const uint32_t w32[4] = {cur[u][c].x, cur[u][c].y, cur[u][c].z, cur[u][c].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          y[c][2 * j] = bf16lo_to_f32(w32[j]);
          y[c][2 * j + 1] = bf16hi_to_f32(w32[j]);
          ss = fmaf(y[c][2 * j], y[c][2 * j], ss);
          ss = fmaf(y[c][2 * j + 1], y[c][2 * j + 1], ss);
        }
      }
      ss += __shfl_xor_sync(0xffffffffu, ss, 1);
      ss += __shfl_xor_sync(0xffffffffu, ss, 2);
      if (wt != nullptr) {
        const float rs = rsqrtf(fmaf(ss, 1.f / 64.f, p.eps));
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const uint32_t ww[4] = {wv[c].x, wv[c].y, wv[c].z, wv[c].w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            y[c][2 * j] *= rs * bf16lo_to_f32(ww[j]);
            y[c][2 * j + 1] *= rs * bf16hi_to_f32(ww[j]);
          }
        }
      }
      if constexpr (kLayout == kRopeInterleaved) {
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int f = 4 * (c ? c1 : c0) + j;
            if (f < half) {
              const float2 cs = s_cs[t][f];
              const float a = y[c][2 * j], b = y[c][2 * j + 1];
              y[c][2 * j] = fmaf(a, cs.x, -b * cs.y);
              y[c][2 * j + 1] = fmaf(b, cs.x, a * cs.y);
            }
          }
      } else if constexpr (kLayout == kRopeHalf8) {
        if (turns_here) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float2 cs = s_cs[t][c0 * 8 + j];
            const float a = y[0][j], b = y[1][j];
            y[0][j] = fmaf(a, cs.x, -b * cs.y);
            y[1][j] = fmaf(b, cs.x, a * cs.y);
          }
        }
      } else {
        float* row = s_row + grp * 64;
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int j = 0; j < 8; ++j) row[(c ? c1 : c0) * 8 + j] = y[c][j];
        __syncwarp();
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int e = (c ? c1 : c0) * 8 + j;
            if (e < half) {
              const float2 cs = s_cs[t][e];
              y[c][j] = fmaf(y[c][j], cs.x, -row[e + half] * cs.y);
            } else if (e < p.rot) {
              const float2 cs = s_cs[t][e - half];
              y[c][j] = fmaf(y[c][j], cs.x, row[e - half] * cs.y);
            }
          }
        __syncwarp();
      }
      if (live) {
        __nv_bfloat16* dst = is_q ? p.Qo + (n * p.Ha + h) * 64 : p.Ko + (n * p.G + (h - p.Hq)) * 64;
#pragma unroll
        for (int c = 0; c < 2; ++c)
          st_global_v4(dst + (c ? c1 : c0) * 8, pack_bf16x2(y[c][0], y[c][1]), pack_bf16x2(y[c][2], y[c][3]),
                       pack_bf16x2(y[c][4], y[c][5]), pack_bf16x2(y[c][6], y[c][7]));
      }
    }
  }
}

}  // namespace gqe
