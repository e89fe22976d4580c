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
// an fp32 product has lost the angle (spacing 0.06). inv_freq / 2 pi, in turns
// a position, is therefore held as a 64-bit fraction of a turn (from fp64, once
// a block): pos times that, modulo 2^64, is the angle modulo a turn, by three
// integer multiplies, exact but for the fraction's own rounding (relative
// 2^-53). As a signed number it is converted to fp32 once, so small angles keep
// their relative precision, and goes to sincospi.
//
// Work: memory-bound, 256 bytes a head (read and written once). A block walks
// over its tokens in chunks of `tpb`, whose rows of Q and of K are contiguous
// and come by bulk copies into a ring of kRopeStages chunks: loads stay in
// flight whatever the warps do, which is what the time hung on (4.0 TB/s at 60%
// of the issue slots with loads through registers one token ahead). Four lanes
// hold a head, 16 elements (two 16-byte chunks) each, and a rotation's partners
// are in one thread: with half = rot/2 a multiple of eight, lane l < half/8
// takes 16-byte chunks l and l + half/8, and the other lanes those that are not
// rotated, two by two; neighbouring pairs are in one chunk anyhow. Only other
// values of half go through shared memory. A thread keeps its head, so that
// addresses advance by a constant; cosines and sines are computed once a chunk,
// for the next one; products are packed in pairs (f32x2).
//
// Measured, Q and K of 8 groups: 1 x 131072 tokens of 25 heads 171-177 us =
// 4.8-5.0 TB/s of 6.5 that a copy reaches (265 us with loads through registers
// and each thread its own angles); 8 x 2048 of 17 heads 18.6 us: 14.8 at
// the long case's rate, the rest the start and the end of a short kernel; one
// token 2.3 us. In the interleaved layout a lane's two chunks are neighbours, so
// that each of its stores covers every second 16 bytes of the head.
#pragma once

#include "attn2.cuh"
#include "sm100.cuh"

namespace gqe {

constexpr int kRopeThreads = 256;      // at most, for up to 64 heads a token
constexpr int kRopeThreadsWide = 544;  // 129 heads (rounded up to whole warps) of one token
constexpr int kRopeMaxTpb = 16;    // tokens of a chunk at most
constexpr int kRopeStages = 3;

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
  int rot;
  int tp, tpb;  // tokens side by side in a block, tokens of a chunk (a multiple of tp)
  int span;     // tokens of a block (a multiple of tp)
  int log2k;
};

__device__ __forceinline__ void fmul2(float& d0, float& d1, float a0, float a1, float b0, float b1) {
  asm("{\n\t.reg .b64 ra, rb, rd;\n\t"
      "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
      "mul.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
      : "=f"(d0), "=f"(d1)
      : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}
// Two rotations: (a, b) -> (a c - b s, b c + a s).
__device__ __forceinline__ void turn2(float& a0, float& a1, float& b0, float& b1, float c0, float c1, float s0, float s1) {
  float x0, x1, y0, y1;
  fmul2(x0, x1, b0, b1, -s0, -s1);
  fmul2(y0, y1, a0, a1, s0, s1);
  ffma2(a0, a1, a0, a1, c0, c1, x0, x1);
  ffma2(b0, b1, b0, b1, c0, c1, y0, y1);
}

template <int kLayout, int kThreads>
__global__ void __launch_bounds__(kThreads) qk_rope_kernel(const RopeParams p) {
  __shared__ float4 s_cos[2][kRopeMaxTpb][8], s_sin[2][kRopeMaxTpb][8];
  extern __shared__ uint8_t rope_raw[];
  __shared__ unsigned long long s_turn[32];
  __shared__ uint64_t s_full[kRopeStages];
  __shared__ int s_abort;
  __shared__ float s_row[kLayout == kRopeHalfAny ? kThreads * 16 : 1];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x;
  const int l4 = tid & 3, grp = tid >> 2;  // lane of the head; head of this thread
  const int H = p.Hq + p.Hk;
  const int half = p.rot >> 1;
  const int tl = min(grp / H, p.tp - 1);  // (lanes past the last head repeat one and store nothing)
  const int h = min(grp - tl * H, H - 1);
  const bool mine = grp < p.tp * H;
  const bool is_q = h < p.Hq;
  // this lane's two chunks of eight elements
  int c0 = kLayout == kRopeInterleaved ? 2 * l4 : l4, cd = kLayout == kRopeInterleaved ? 1 : 4;  // c0 and c0 + cd
  bool turns_here = true;  // (half layout) the chunks are each other's partners
  if constexpr (kLayout == kRopeHalf8) {
    const int hc = half >> 3;
    turns_here = l4 < hc;
    c0 = turns_here ? l4 : 2 * l4;
    cd = turns_here ? hc : 1;
  }
  // the block's tokens are [n0, n1), this thread's n0 + tl, n0 + tl + tp, ...
  const int n0 = blockIdx.x * p.span, n1 = min(p.N, n0 + p.span);
  const int own = is_q ? p.Hq : p.Hk;  // rows a token on this thread's side
  const uint32_t step = (uint32_t)p.tp * own * 8;  // 16-byte chunks from one token to its next
  uint4* dst = reinterpret_cast<uint4*>(is_q ? p.Qo : p.Ko) +
               ((size_t)(n0 + tl) * own + (is_q ? h : h - p.Hq)) * 8 + c0;
  // its first row in a stage: the chunk's rows of Q, then those of K
  const uint32_t at0 = (tl * own + (is_q ? h : p.tpb * p.Hq + h - p.Hq)) * 8 + c0;
  uint8_t* ring = rope_raw + ((128u - (smem_u32(rope_raw) & 127u)) & 127u);
  const uint32_t stage_bytes = p.tpb * H * 128;
  auto copy = [&](int chunk, int s) {  // (one thread) a chunk's rows into stage s
    if (chunk >= n1) return;
    const uint32_t nt = min(p.tpb, n1 - chunk);
    uint8_t* to = ring + s * stage_bytes;
    mbar_arrive_expect_tx(&s_full[s], nt * H * 128);
    if (p.Hq) bulk_load(to, p.Q + (size_t)chunk * p.Hq * 64, nt * p.Hq * 128, &s_full[s]);
    if (p.Hk) bulk_load(to + p.tpb * p.Hq * 128, p.K + (size_t)chunk * p.Hk * 64, nt * p.Hk * 128, &s_full[s]);
  };
  const bool normed = (is_q ? p.wq : p.wk) != nullptr;
  const uint4* wt = reinterpret_cast<const uint4*>(is_q ? p.wq : p.wk) + c0;
  const bool routed = is_q && h < p.G * p.k && normed;  // its weight row depends on the token
  const int32_t* sel = p.sel + (size_t)(n0 + tl) * (p.G * p.k) + h;
  const int expert0 = (h >> p.log2k) * p.M;
  // the expert of this thread's next token is loaded one token ahead
  int e_next = 0;
  auto fetch = [&](int n) {
    if (routed && n < n1) {
      e_next = sel[0];
      sel += p.tp * (p.G * p.k);
    }
  };
  uint4 w0, w1;
  auto load_weights = [&](int head) {
    w0 = wt[head * 8];
    w1 = wt[head * 8 + cd];
  };
  auto angles = [&](int chunk, int buf) {
    for (int i = tid; i < p.tpb * 32; i += blockDim.x) {
      const int t = i >> 5, f = i & 31, n = chunk + t;
      if (f < half && n < n1) {
        const int pos = p.positions ? p.positions[n] : n % p.T;
        const long long turn = (long long)((unsigned long long)(long long)pos * s_turn[f]);
        float s, c;
        sincospif(__ll2float_rn(turn) * 0x1p-63f, &s, &c);
        reinterpret_cast<float*>(s_cos[buf][t])[f] = c * p.scale;
        reinterpret_cast<float*>(s_sin[buf][t])[f] = s * p.scale;
      }
    }
  };
  if (tid == 0) {
    for (int s = 0; s < kRopeStages; ++s) mbar_init(&s_full[s], 1);
    s_abort = 0;
    fence_mbar_init();
    for (int s = 0; s < kRopeStages; ++s) copy(n0 + s * p.tpb, s);
  }
  fetch(n0 + tl);
  if (normed && !routed) load_weights(is_q ? p.G * p.M : h - p.Hq);
  if (tid < half) {
    const double turns = (double)p.inv_freq[tid] * 0.15915494309189533577;
    s_turn[tid] = (unsigned long long)((turns - floor(turns)) * 0x1p64);
  }
  __syncthreads();
  angles(n0, 0);
  __syncthreads();
  int buf = 0, stage = 0;
  uint32_t parity = 0;
  bool ok = true;
  for (int chunk = n0; chunk < n1; chunk += p.tpb, buf ^= 1) {
    if (chunk + p.tpb < n1) angles(chunk + p.tpb, buf ^ 1);
    ok = mbar_wait(&s_full[stage], parity, &s_abort);
    const uint4* src = reinterpret_cast<const uint4*>(ring + stage * stage_bytes) + at0;
    for (int t = tl; t < p.tpb; t += p.tp, src += step) {
      const bool live = mine && chunk + t < n1;
      const uint4 b0 = src[0], b1 = src[cd];  // (past the last token: what the stage held)
      const uint32_t u[8] = {b0.x, b0.y, b0.z, b0.w, b1.x, b1.y, b1.z, b1.w};
      if (routed) {
        if (e_next < 0 || e_next >= p.M) flag_bounds_error();
        load_weights(expert0 + min(max(e_next, 0), p.M - 1));
      }
      fetch(chunk + t + p.tp);
      float y[16];  // chunk c0, then chunk c0 + cd
      float s0 = 0.f, s1 = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        y[2 * j] = bf16lo_to_f32(u[j]);
        y[2 * j + 1] = bf16hi_to_f32(u[j]);
        ffma2(s0, s1, y[2 * j], y[2 * j + 1], y[2 * j], y[2 * j + 1], s0, s1);
      }
      float ss = s0 + s1;
      ss += __shfl_xor_sync(0xffffffffu, ss, 1);
      ss += __shfl_xor_sync(0xffffffffu, ss, 2);
      if (normed) {
        const float rs = rsqrtf(fmaf(ss, 1.f / 64.f, p.eps));
        const uint32_t ww[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float a, b;
          fmul2(a, b, bf16lo_to_f32(ww[j]), bf16hi_to_f32(ww[j]), rs, rs);
          fmul2(y[2 * j], y[2 * j + 1], y[2 * j], y[2 * j + 1], a, b);
        }
      }
      if constexpr (kLayout == kRopeInterleaved) {
        // a chunk is four neighbouring pairs
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int at = c0 + c;
          const float4 cs = s_cos[buf][t][at], sn = s_sin[buf][t][at];
          float* v = y + 8 * c;
          if (4 * at + 4 <= half) {
            turn2(v[0], v[2], v[1], v[3], cs.x, cs.y, sn.x, sn.y);
            turn2(v[4], v[6], v[5], v[7], cs.z, cs.w, sn.z, sn.w);
          } else if (4 * at < half) {  // rot ends inside the chunk
            float z0 = 0.f, z1 = 0.f;
            turn2(v[0], z0, v[1], z1, cs.x, 0.f, sn.x, 0.f);
            if (4 * at + 1 < half) turn2(v[2], z0, v[3], z1, cs.y, 0.f, sn.y, 0.f);
            if (4 * at + 2 < half) turn2(v[4], z0, v[5], z1, cs.z, 0.f, sn.z, 0.f);
          }
        }
      } else if constexpr (kLayout == kRopeHalf8) {
        if (turns_here) {
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const float4 cs = s_cos[buf][t][2 * c0 + q], sn = s_sin[buf][t][2 * c0 + q];
            float *a = y + 4 * q, *b = y + 8 + 4 * q;
            turn2(a[0], a[1], b[0], b[1], cs.x, cs.y, sn.x, sn.y);
            turn2(a[2], a[3], b[2], b[3], cs.z, cs.w, sn.z, sn.w);
          }
        }
      } else {
        float* row = s_row + grp * 64;
#pragma unroll
        for (int j = 0; j < 16; ++j) row[(j < 8 ? c0 : c0 + cd) * 8 + (j & 7)] = y[j];
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const int e = (j < 8 ? c0 : c0 + cd) * 8 + (j & 7);
          if (e < p.rot) {
            const bool lo = e < half;
            const int f = lo ? e : e - half;
            const float c = reinterpret_cast<const float*>(s_cos[buf][t])[f], s = reinterpret_cast<const float*>(s_sin[buf][t])[f];
            y[j] = fmaf(y[j], c, (lo ? -row[e + half] : row[f]) * s);
          }
        }
        __syncwarp();
      }
      if (live) {
        dst[0] = make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7]));
        dst[cd] = make_uint4(pack_bf16x2(y[8], y[9]), pack_bf16x2(y[10], y[11]), pack_bf16x2(y[12], y[13]), pack_bf16x2(y[14], y[15]));
      }
      dst += step;
    }
    // the next chunk's angles are there; this one's and its stage are used up
    if (!(ok = __syncthreads_and(ok))) break;
    if (tid == 0) copy(chunk + kRopeStages * p.tpb, stage);
    if (++stage == kRopeStages) stage = 0, parity ^= 1;
  }
  if (!ok) {
    // a wait ran out: let the copies in flight land before the block exits
    const unsigned long long t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 100000ull) {}
  }
}

}  // namespace gqe
