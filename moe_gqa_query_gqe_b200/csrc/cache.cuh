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
  int32_t *holes, *late;  // [B*G][list] slots left empty below keep, rows kept past it
  uint32_t* bits;         // [B*G][words] a bit a row: it stays
  int B, G, cap, keep, sink, recent, list, words;
  int ncta;  // blocks of a cluster
  int held;  // keys a block can hold in shared memory
};

// Order of the rows as unsigned numbers: a row that must stay above every
// mass, NaN below every mass, -0 and +0 equal.
__device__ __forceinline__ uint32_t evict_key(float m, int pos, int sink, long long recent_from) {
  if (pos < sink || (long long)pos >= recent_from) return 0xffffffffu;
  if (m != m) return 0u;
  const uint32_t u = __float_as_uint(m + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ int ld_dsmem_s32(uint32_t cluster_addr) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(cluster_addr) : "memory");
  return v;
}

__device__ __forceinline__ int2 ld_dsmem_v2(uint32_t cluster_addr) {
  int2 v;
  asm volatile("ld.shared::cluster.v2.s32 {%0,%1}, [%2];"
               : "=r"(v.x), "=r"(v.y)
               : "r"(cluster_addr)
               : "memory");
  return v;
}
// Every thread of the cluster, whether its warp has reconverged or not; within
// one block the block's own barrier (a third of the time).
__device__ __forceinline__ void cluster_sync_any(int ncta) {
  if (ncta == 1) {
    __syncthreads();
  } else {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
  }
}

// One cluster of `ncta` blocks per (sequence, group). Each block takes a
// contiguous share of the rows, each warp a contiguous share of the block's, so
// that (block, warp, step, lane) is the rows' order.
//   1. Keys (mass and position, 8 bytes a row) are read once and held in shared
//      memory, as far as they fit.
//   2. The keep-th largest key by three radix passes of 11, 11 and 10 bits: a
//      histogram per block, added over the cluster through distributed shared
//      memory. (Masses lie within a few powers of two of one another: with 8
//      bits the first pass counted into a handful of bins.) The second pass
//      leaves its candidates in a list, which the third goes over.
//   3. A row stays if its key is larger, or equal and among the first of the
//      equal ones: a bit a row. The empty slots below keep and the staying rows
//      past it go to two lists, in order: ranks from the bits' counts, over lanes,
//      warps and blocks.
//   4. Row j of the one list moves into slot j of the other, eight lanes a row,
//      K and V, four rows of a lane in flight.
// Bound by the moved rows' bytes (K and V, 256 bytes read and 256 written a row, in
// pieces of 128), or, where few leave, by the instructions a row of the passes and
// the chain of barriers. Measured, 8 sequences of 8 groups: 30000 to 32768 rows to
// 4096 59 us, 25 of them before the first move (floor 21: 8 bytes a row and the
// moves at the copy's rate); 4100 to 4096 12.3 us.
constexpr int kEvictThreads = 1024;
constexpr int kEvictWarps = kEvictThreads / 32;  // 32: a lane holds a warp's count
constexpr int kEvictBins = 2048;
constexpr int kEvictCands = 128;  // of a warp
constexpr int kEvictBatch = 8;    // rows of a lane that are loaded together
struct EvictShared {
  int hist[kEvictBins];
  int total[2][kEvictBins];  // this block's histogram, of two passes in turn: read by the cluster
  uint32_t cand[kEvictWarps][kEvictCands];
  int counts[3];             // equal keys, holes, late rows of this block: read by the cluster
  int warp[3][kEvictWarps];
  int pick[3];
};
__global__ void __launch_bounds__(kEvictThreads, 1) cache_evict_kernel(const EvictParams p) {
  extern __shared__ uint32_t s_keys[];
  __shared__ EvictShared sh;
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int bg = blockIdx.x / p.ncta, rank = blockIdx.x % p.ncta, b = bg / p.G, g = bg % p.G;
  const int n = p.cache_len[b];
  const bool first = g == 0 && rank == 0 && tid == 0;
  if (n < 0 || n > p.cap) {
    flag_bounds_error();
    if (first) p.new_len[b] = n;
    return;
  }
  if (first) p.new_len[b] = min(n, p.keep);
  const size_t at = (size_t)bg * p.cap;
  const float* mass = p.mass_in + at;
  const int32_t* pos = p.pos_in + at;
  if (n <= p.keep) {
    for (int i = rank * kEvictThreads + tid; i < n; i += p.ncta * kEvictThreads) {
      p.mass_out[at + i] = mass[i];
      p.pos_out[at + i] = pos[i];
    }
    return;
  }
  const long long recent_from = (long long)p.next_pos[b] - p.recent;
  // this warp's rows: base .. base + len - 1, those below n
  const int len = ((n + p.ncta - 1) / p.ncta + kEvictThreads - 1) / kEvictThreads * 32;
  const int share = len * kEvictWarps;
  const int base = rank * share + warp * len;
  const bool held = share <= p.held;
  uint32_t* mine = s_keys + warp * len;
  auto key_at = [&](int i) -> uint32_t {  // row base + i
    return held ? mine[i] : evict_key(mass[base + i], pos[base + i], p.sink, recent_from);
  };
  const int steps = min(len, max(0, n - base));  // rows of this warp
  const uint32_t below = (1u << lane) - 1u;
  uint32_t prefix = 0;
  int need = p.keep;  // rows still to be found among those that share the prefix
  int same = 0;       // how many share it
  int ncand = 0;      // this warp's keys that share the first digit
  for (int pass = 0; pass < 3; ++pass) {
    for (int i = tid; i < kEvictBins; i += kEvictThreads) sh.hist[i] = 0;
    __syncthreads();
    if (pass == 0) {
      for (int i0 = 0; i0 < steps; i0 += 32 * kEvictBatch) {
        float m[kEvictBatch];
        int ps[kEvictBatch];
#pragma unroll
        for (int u = 0; u < kEvictBatch; ++u) {
          const int i = i0 + u * 32 + lane;
          if (i < steps) {
            m[u] = mass[base + i];
            ps[u] = pos[base + i];
          }
        }
#pragma unroll
        for (int u = 0; u < kEvictBatch; ++u) {
          const int i = i0 + u * 32 + lane;
          if (i >= steps) continue;
          const uint32_t key = evict_key(m[u], ps[u], p.sink, recent_from);
          if (held) mine[i] = key;
          if (base + i < p.keep) {  // (a slot that is left gets its row's at the end)
            p.mass_out[at + base + i] = m[u];
            p.pos_out[at + base + i] = ps[u];
          }
          atomicAdd(&sh.hist[key >> 21], 1);
        }
      }
    } else if (pass == 1 || ncand > kEvictCands) {
      const int cut = pass == 1 ? 21 : 10, shift = pass == 1 ? 10 : 0;
      const uint32_t digits = pass == 1 ? 2047u : 1023u;
      for (int i0 = 0; i0 < steps; i0 += 32 * kEvictBatch) {
        uint32_t key[kEvictBatch];
#pragma unroll
        for (int u = 0; u < kEvictBatch; ++u) {
          const int i = i0 + u * 32 + lane;
          key[u] = i < steps ? key_at(i) : 0u;
        }
#pragma unroll
        for (int u = 0; u < kEvictBatch; ++u) {
          const bool in = i0 + u * 32 + lane < steps && (key[u] >> cut) == prefix;
          if (in) atomicAdd(&sh.hist[(key[u] >> shift) & digits], 1);
          if (pass == 1) {
            const uint32_t all = __ballot_sync(0xffffffffu, in);
            const int to = ncand + __popc(all & below);
            if (in && to < kEvictCands) sh.cand[warp][to] = key[u];
            ncand += __popc(all);
          }
        }
      }
    } else {
      __syncwarp();
      for (int i = lane; i < ncand; i += 32) {
        const uint32_t key = sh.cand[warp][i];
        if ((key >> 10) == prefix) atomicAdd(&sh.hist[key & 1023u], 1);
      }
    }
    __syncthreads();
    int* total = sh.total[pass & 1];
    for (int i = tid; i < kEvictBins; i += kEvictThreads) total[i] = sh.hist[i];
    cluster_sync_any(p.ncta);
    // the highest bins first: thread t holds bins 2047 - 2 t and below; sums over
    // the threads before it. The cluster's histograms are loaded together: a load
    // from another block takes a thousand cycles here.
    static_assert(kEvictBins == 2 * kEvictThreads, "one 8-byte load a block");
    const int* mine2 = &total[kEvictBins - 2 - tid * 2];
    int bins[2] = {mine2[1], mine2[0]};
    if (p.ncta > 1) {
      int2 part[7];
#pragma unroll
      for (int c = 1; c < 8; ++c)
        if (c < p.ncta) part[c - 1] = ld_dsmem_v2(mapa_shared(smem_u32(mine2), (rank + c) & (p.ncta - 1)));
#pragma unroll
      for (int c = 1; c < 8; ++c)
        if (c < p.ncta) {
          bins[0] += part[c - 1].y;
          bins[1] += part[c - 1].x;
        }
    }
    const int sum = bins[0] + bins[1];
    int above = sum;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const int o = __shfl_up_sync(0xffffffffu, above, d);
      if (lane >= d) above += o;
    }
    if (lane == 31) sh.warp[0][warp] = above;
    __syncthreads();
    above += __reduce_add_sync(0xffffffffu, lane < warp ? sh.warp[0][lane] : 0) - sum;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (above < need && above + bins[i] >= need) {
        sh.pick[0] = kEvictBins - 1 - tid * 2 - i;
        sh.pick[1] = need - above;
        sh.pick[2] = bins[i];
      }
      above += bins[i];
    }
    __syncthreads();
    prefix = (prefix << (pass == 2 ? 10 : 11)) | (uint32_t)sh.pick[0];
    need = sh.pick[1];
    same = sh.pick[2];
  }
  // A count of each warp (warp[what]) and each block (counts[what]): the sum over
  // what comes before this warp, in the block and in the cluster's blocks before.
  auto before = [&](int what) {
    int v = lane < warp ? sh.warp[what][lane] : 0;
    if (p.ncta > 1 && lane < rank) v += ld_dsmem_s32(mapa_shared(smem_u32(&sh.counts[what]), lane));
    return __reduce_add_sync(0xffffffffu, v);
  };
  auto sum_warps = [&](int what) {  // (warp 0)
    const int v = __reduce_add_sync(0xffffffffu, sh.warp[what][lane]);
    if (lane == 0) sh.counts[what] = v;
  };
  // bits of the rows that stay, and how many holes and late rows they make
  uint32_t* bits = p.bits + (size_t)bg * p.words + base / 32;
  int holes = 0, late = 0;
  auto count = [&](int i0, uint32_t stay) {  // of rows base + i0 .. + 31
    const int left = min(32, steps - i0), under = min(max(p.keep - (base + i0), 0), 32);
    const uint32_t there = left == 32 ? 0xffffffffu : (1u << left) - 1u;
    const uint32_t low = under == 32 ? 0xffffffffu : (1u << under) - 1u;
    holes += __popc(~stay & there & low);
    late += __popc(stay & ~low);
    if (lane == 0) bits[i0 / 32] = stay;
  };
  if (need == same) {
    for (int i0 = 0; i0 < steps; i0 += 32 * kEvictBatch) {
      uint32_t key[kEvictBatch];
#pragma unroll
      for (int u = 0; u < kEvictBatch; ++u) {
        const int i = i0 + u * 32 + lane;
        key[u] = i < steps ? key_at(i) : 0u;
      }
#pragma unroll
      for (int u = 0; u < kEvictBatch; ++u) {
        const int i = i0 + u * 32;
        if (i < steps) count(i, __ballot_sync(0xffffffffu, i + lane < steps && key[u] >= prefix));
      }
    }
  } else {  // only the first of the equal keys' rows stay
    int eq = 0;
    __syncthreads();
    if (ncand <= kEvictCands) {
      for (int i = lane; i < ncand; i += 32) eq += sh.cand[warp][i] == prefix;
    } else {
      for (int i = lane; i < steps; i += 32) eq += key_at(i) == prefix;
    }
    eq = __reduce_add_sync(0xffffffffu, eq);
    if (lane == 0) sh.warp[0][warp] = eq;
    __syncthreads();
    if (warp == 0) sum_warps(0);
    cluster_sync_any(p.ncta);
    eq = before(0);
    for (int i0 = 0; i0 < steps; i0 += 32) {
      const bool in = i0 + lane < steps;
      const uint32_t key = in ? key_at(i0 + lane) : 0u;
      const uint32_t e = __ballot_sync(0xffffffffu, in && key == prefix);
      count(i0, __ballot_sync(0xffffffffu, in && (key > prefix || (key == prefix && eq + __popc(e & below) < need))));
      eq += __popc(e);
    }
  }
  if (lane == 0) {
    sh.warp[1][warp] = holes;
    sh.warp[2][warp] = late;
  }
  __syncthreads();
  if (warp == 0) {
    sum_warps(1);
    sum_warps(2);
  }
  cluster_sync_any(p.ncta);
  holes = before(1);
  late = before(2);
  int32_t* hole_list = p.holes + (size_t)bg * p.list;
  int32_t* late_list = p.late + (size_t)bg * p.list;
  __syncwarp();
  for (int i0 = 0; i0 < steps; i0 += 1024) {  // a lane, 32 rows
    const int r0 = i0 + lane * 32, left = min(32, steps - r0), under = min(max(p.keep - (base + r0), 0), 32);
    uint32_t h = 0, l = 0;
    if (left > 0) {
      const uint32_t stay = bits[r0 / 32];
      const uint32_t there = left == 32 ? 0xffffffffu : (1u << left) - 1u;
      const uint32_t low = under == 32 ? 0xffffffffu : (1u << under) - 1u;
      h = ~stay & there & low;
      l = stay & ~low;
    }
    const int hc = __popc(h), lc = __popc(l);
    int hs = hc, ls = lc;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const int x = __shfl_up_sync(0xffffffffu, hs, d), y = __shfl_up_sync(0xffffffffu, ls, d);
      if (lane >= d) {
        hs += x;
        ls += y;
      }
    }
    // (as many rows stay as the passes counted unless the masses change
    // meanwhile: nothing is then written or moved out of range)
    for (int to = holes + hs - hc; h && to < p.list; h &= h - 1) hole_list[to++] = base + r0 + __ffs(h) - 1;
    for (int to = late + ls - lc; l && to < p.list; l &= l - 1) late_list[to++] = base + r0 + __ffs(l) - 1;
    holes += __shfl_sync(0xffffffffu, hs, 31);
    late += __shfl_sync(0xffffffffu, ls, 31);
  }
  int moves = 0, others = 0;
  if (lane < p.ncta) {
    moves = ld_dsmem_s32(mapa_shared(smem_u32(&sh.counts[1]), lane));
    others = ld_dsmem_s32(mapa_shared(smem_u32(&sh.counts[2]), lane));
  }
  moves = __reduce_add_sync(0xffffffffu, moves);
  others = __reduce_add_sync(0xffffffffu, others);
  if (moves != others || moves > p.list) {
    flag_bounds_error();
    moves = 0;
  }
  __threadfence();
  cluster_sync_any(p.ncta);  // the lists are there; no block's shared memory is read from here on
  const int l8 = lane & 7;
  for (int i0 = (rank * kEvictWarps + warp) * 16; i0 < moves; i0 += p.ncta * kEvictWarps * 16) {
    int to[4], from[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int i = i0 + u * 4 + (lane >> 3);
      to[u] = i < moves ? __ldcg(hole_list + i) : -1;
      from[u] = i < moves ? __ldcg(late_list + i) : 0;
    }
    uint4 kv[4], vv[4];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (to[u] >= 0) {
        const size_t src = (((size_t)b * p.cap + from[u]) * p.G + g) * 64;
        kv[u] = reinterpret_cast<const uint4*>(p.Kc + src)[l8];
        vv[u] = reinterpret_cast<const uint4*>(p.Vc + src)[l8];
      }
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (to[u] >= 0) {
        const size_t dst = (((size_t)b * p.cap + to[u]) * p.G + g) * 64;
        reinterpret_cast<uint4*>(p.Kc + dst)[l8] = kv[u];
        reinterpret_cast<uint4*>(p.Vc + dst)[l8] = vv[u];
        if (l8 == 0) p.mass_out[at + to[u]] = mass[from[u]];
        if (l8 == 1) p.pos_out[at + to[u]] = pos[from[u]];
      }
  }
}

}  // namespace gqe
