// cache.cuh -- upkeep of a key/value cache: the accepted drafts appended, their
// attention weight added to every cached position's sum, and the positions
// with the least of it evicted.
#pragma once

#include "decode.cuh"
#include "sm100.cuh"
#include "tree.cuh"

namespace gqe {

struct CommitParams {
  const int32_t *path, *n_acc, *positions, *cache_len;
  const __nv_bfloat16 *Q, *Kn, *Vn;
  const float* lse;
  __nv_bfloat16 *Kc, *Vc;
  int32_t* pos;
  const float* mass_in;
  float* mass_out;
  int32_t* new_len;
  int B, T, G, k, Ha, cap;
  float scale_log2;
};

// Length and accepted tokens of sequence b; n = -1 where they are out of range
// (recorded; the sequence is left as it is).
__device__ __forceinline__ void commit_lens(const CommitParams& p, int b, int& L, int& n) {
  L = p.cache_len[b];
  n = p.n_acc ? p.n_acc[b] : p.T;
  if (L < 0 || L > p.cap || n < 0 || n > p.T || n > p.cap - L) {
    flag_bounds_error();
    n = -1;
  }
}
// Drafted token at place j of the accepted path; an index out of range is
// recorded and gives -1 (that row is skipped).
__device__ __forceinline__ int commit_token(const CommitParams& p, int b, int j) {
  const int i = p.path ? p.path[(size_t)b * p.T + j] : j;
  if (i < 0 || i >= p.T) {
    flag_bounds_error();
    return -1;
  }
  return i;
}

// Place j of sequence b's accepted path into the cache, by `threads` threads of
// which this is `i`: G*64 values of K and of V, and the G positions.
__device__ __forceinline__ void commit_append_row(const CommitParams& p, int b, int j, int L, int n, int i, int threads) {
  if (j == 0 && i == 0) p.new_len[b] = n < 0 ? p.cache_len[b] : L + n;
  if (j >= n) return;
  const int tok = commit_token(p, b, j);
  if (tok < 0) return;
  const size_t src = ((size_t)b * p.T + tok) * p.G * 64, dst = ((size_t)b * p.cap + L + j) * p.G * 64;
  for (int t = i; t < p.G * 16; t += threads) {
    const int at = (t >> 1) * 8;
    const __nv_bfloat16* s = (t & 1 ? p.Vn : p.Kn) + src + at;
    __nv_bfloat16* d = (t & 1 ? p.Vc : p.Kc) + dst + at;
    *reinterpret_cast<uint4*>(d) = *reinterpret_cast<const uint4*>(s);
  }
  if (p.pos != nullptr)
    for (int g = i; g < p.G; g += threads)
      p.pos[((size_t)b * p.G + g) * p.cap + L + j] = p.positions ? p.positions[(size_t)b * p.T + tok] : L + j;
}

// The commit without the sums: one block per (sequence, place of the path).
constexpr int kAppendThreads = 128;
__global__ void __launch_bounds__(kAppendThreads) commit_append_kernel(const CommitParams p) {
  pdl_wait();
  pdl_trigger();
  const int b = blockIdx.x / p.T, j = blockIdx.x % p.T;
  int L, n;
  commit_lens(p, b, L, n);
  commit_append_row(p, b, j, L, n, threadIdx.x, kAppendThreads);
}

// ---------------------------------------------------------------------------
// Eviction
// ---------------------------------------------------------------------------
struct EvictParams {
  const int32_t *cache_len, *next_pos;
  __nv_bfloat16 *Kc, *Vc;
  const float* mass_in;
  float* mass_out;
  const int32_t* pos_in;
  int32_t* pos_out;
  int32_t* new_len;
  int32_t *moves;  // [B*G] rows to move
  int32_t *holes, *late;  // [B*G][cap / 2 + 1] slots left empty below keep, rows kept past it
  int B, G, cap, keep, sink, recent, list;
};

// Order of the rows as unsigned numbers: a row that must stay above every
// mass, NaN below every mass, -0 and +0 equal.
__device__ __forceinline__ uint32_t evict_key(float m, int pos, int sink, long long recent_from) {
  if (pos < sink || (long long)pos >= recent_from) return 0xffffffffu;
  if (m != m) return 0u;
  const uint32_t u = __float_as_uint(m + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// One block per (sequence, group): the keep-th largest key by four 8-bit radix
// passes over the rows (mass and position, 8 bytes a row, from L2 after the
// first), then the rows in order: a row stays if its key is larger, or equal
// and among the first of the equal ones. Mass and position of the staying rows
// are written; the empty slots below keep and the staying rows past it go to
// the lists, in order.
constexpr int kEvictThreads = 1024;
__global__ void __launch_bounds__(kEvictThreads) evict_select_kernel(const EvictParams p) {
  __shared__ int s_hist[256];
  __shared__ int s_warp[3][32];
  __shared__ int s_pick[2];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int b = blockIdx.x / p.G;
  int n = p.cache_len[b];
  if (n < 0 || n > p.cap) {
    flag_bounds_error();
    if (tid == 0) p.moves[blockIdx.x] = -1;
    return;
  }
  const size_t at = (size_t)blockIdx.x * p.cap;
  const float* mass = p.mass_in + at;
  const int32_t* pos = p.pos_in + at;
  const long long recent_from = (long long)p.next_pos[b] - p.recent;
  if (n <= p.keep) {
    for (int i = tid; i < n; i += kEvictThreads) {
      p.mass_out[at + i] = mass[i];
      p.pos_out[at + i] = pos[i];
    }
    if (tid == 0) p.moves[blockIdx.x] = 0;
    return;
  }
  uint32_t prefix = 0;
  int need = p.keep;  // rows still to be found among those that share the prefix
  for (int shift = 24; shift >= 0; shift -= 8) {
    if (tid < 256) s_hist[tid] = 0;
    __syncthreads();
    for (int i = tid; i < n; i += kEvictThreads) {
      const uint32_t key = evict_key(mass[i], pos[i], p.sink, recent_from);
      if (shift == 24 || (key >> (shift + 8)) == prefix) atomicAdd(&s_hist[(key >> shift) & 255u], 1);
    }
    __syncthreads();
    if (warp == 0) {
      // lane l holds bins 8l .. 8l+7; suffix sums from the top
      int bins[8], sum = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) sum += bins[i] = s_hist[lane * 8 + i];
      int above = sum;
#pragma unroll
      for (int d = 1; d < 32; d *= 2) {
        const int o = __shfl_down_sync(0xffffffffu, above, d);
        if (lane + d < 32) above += o;
      }
      above -= sum;  // in the lanes above this one
      for (int i = 7; i >= 0; --i) {
        if (above < need && above + bins[i] >= need) {
          s_pick[0] = lane * 8 + i;
          s_pick[1] = need - above;
        }
        above += bins[i];
      }
    }
    __syncthreads();
    prefix = (prefix << 8) | (uint32_t)s_pick[0];
    need = s_pick[1];
    __syncthreads();
  }
  // the rows in order, 1024 at a time
  int eq_base = 0, hole_base = 0, late_base = 0;
  int32_t* holes = p.holes + (size_t)blockIdx.x * p.list;
  int32_t* late = p.late + (size_t)blockIdx.x * p.list;
  for (int i0 = 0; i0 < n; i0 += kEvictThreads) {
    const int i = i0 + tid;
    float m = 0.f;
    int ps = 0;
    uint32_t key = 0;
    if (i < n) {
      m = mass[i];
      ps = pos[i];
      key = evict_key(m, ps, p.sink, recent_from);
    }
    const uint32_t below = (1u << lane) - 1u;
    const uint32_t eq = __ballot_sync(0xffffffffu, i < n && key == prefix);
    if (lane == 0) s_warp[0][warp] = __popc(eq);
    __syncthreads();
    int rank = eq_base, eq_all = 0;
    for (int w = 0; w < 32; ++w) {
      const int v = s_warp[0][w];
      if (w < warp) rank += v;
      eq_all += v;
    }
    rank += __popc(eq & below);
    eq_base += eq_all;
    const bool stays = i < n && (key > prefix || (key == prefix && rank < need));
    const uint32_t hb = __ballot_sync(0xffffffffu, i < p.keep && !stays);
    const uint32_t lb = __ballot_sync(0xffffffffu, i >= p.keep && stays);
    if (lane == 0) {
      s_warp[1][warp] = __popc(hb);
      s_warp[2][warp] = __popc(lb);
    }
    __syncthreads();
    int ho = hole_base, la = late_base, h_all = 0, l_all = 0;
    for (int w = 0; w < 32; ++w) {
      const int v = s_warp[1][w], x = s_warp[2][w];
      if (w < warp) {
        ho += v;
        la += x;
      }
      h_all += v;
      l_all += x;
    }
    if (i < p.keep && !stays) holes[ho + __popc(hb & below)] = i;
    if (i >= p.keep && stays) late[la + __popc(lb & below)] = i;
    if (i < p.keep && stays) {
      p.mass_out[at + i] = m;
      p.pos_out[at + i] = ps;
    }
    hole_base += h_all;
    late_base += l_all;
    __syncthreads();
  }
  if (tid == 0) p.moves[blockIdx.x] = hole_base;
}

// Rows past keep into the holes: eight lanes a row, K and V.
constexpr int kMoveThreads = 256;
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const EvictParams p) {
  pdl_wait();
  pdl_trigger();
  const int bg = blockIdx.y, b = bg / p.G, g = bg % p.G;
  const int m = p.moves[bg];
  if (g == 0 && blockIdx.x == 0 && threadIdx.x == 0) p.new_len[b] = m < 0 ? p.cache_len[b] : min(p.cache_len[b], p.keep);
  const size_t at = (size_t)bg * p.cap;
  const int l8 = threadIdx.x & 7;
  for (int i = blockIdx.x * (kMoveThreads / 8) + (threadIdx.x >> 3); i < m; i += gridDim.x * (kMoveThreads / 8)) {
    const int to = p.holes[(size_t)bg * p.list + i], from = p.late[(size_t)bg * p.list + i];
    const size_t src = (((size_t)b * p.cap + from) * p.G + g) * 64, dst = (((size_t)b * p.cap + to) * p.G + g) * 64;
    const uint4 kv = reinterpret_cast<const uint4*>(p.Kc + src)[l8], vv = reinterpret_cast<const uint4*>(p.Vc + src)[l8];
    reinterpret_cast<uint4*>(p.Kc + dst)[l8] = kv;
    reinterpret_cast<uint4*>(p.Vc + dst)[l8] = vv;
    if (l8 == 0) p.mass_out[at + to] = p.mass_in[at + from];
    if (l8 == 1) p.pos_out[at + to] = p.pos_in[at + from];
  }
}

}  // namespace gqe
