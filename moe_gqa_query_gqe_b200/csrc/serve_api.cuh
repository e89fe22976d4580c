// serve_api.cuh -- C entry points of the operators around the key/value cache
// (declared in include/gqe.h): argument checks, workspace and launches. Part
// of gqe_api.cu's translation unit.
#pragma once

#include "cache.cuh"
#include "mass.cuh"
#include "rope.cuh"
#include "tree.cuh"
#include "tree_umma.cuh"

namespace {

int check_opt(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (p != nullptr && !aligned16(p)) return GQE_ERR_INVALID_ARG;
  return GQE_OK;
}

// [rows, G, 64] bf16 in boxes of one group's row at 128 positions. Rows of 128
// bytes are all that a box touches of a position's G: fetching 256 bytes into L2
// for each would read the neighbour's too.
int tmap_group(CUtensorMap* tm, const void* base, long long rows, int G) {
  return tmap_heads(tm, base, rows, G, 1, kTuBlock, CU_TENSOR_MAP_L2_PROMOTION_L2_128B);
}

// The tree attention's kernel. Both cut the keys of all sequences into equal
// ranges; the tensor-core kernel (tree_umma.cuh) has the higher rate and costs
// some 12 us before its first block, the other one (tree.cuh) half of that. By
// scores, the rows of a group times the positions that the caches can hold, with
// 8 groups and one row a token (us, tree.cuh / tree_umma.cuh):
//    32 rows   1 x 32000  27.2 / 23.5   4 x 32000  63.5 / 63.0   16 x 4000  46.2 / 48.7
//    64 rows   1 x 16000  26.6 / 25.7   4 x 16000  58.7 / 58.5   16 x 2000  47.9 / 47.3
//   128 rows   1 x 16000  36.9 / 42.1   4 x  8000  63.3 / 51.4   16 x 2000  68.7 / 59.3
//   128 rows   4 x 32000 187.8 / 97.0
bool tree_takes_umma(const gqe_dims* d, int cap) {
  const long long R = (long long)d->T * d->k;
  return R > 32 && R * d->G * d->B >= cdiv(20000000, cap);
}

// Units and grid of either kernel. Neither they nor the workspace depend on the
// cache's capacity.
struct TreePlan {
  int wr;          // row tiles of 16 a unit (tree.cuh)
  int urows, u0, u1, prow;
  int blocks, step;
  long long units;
};
constexpr int kTreeSms = 148;  // of a B200
TreePlan tree_plan(const gqe_dims* d, bool umma) {
  TreePlan t;
  const int R = d->T * d->k, R0 = R + d->T;
  t.wr = R <= 16 ? 1 : (R <= 32 ? 2 : 4);
  t.urows = umma ? kTuRows : 16 * t.wr;
  t.u0 = (int)cdiv(R0, t.urows);
  t.u1 = (int)cdiv(R, t.urows);
  t.prow = std::min(t.urows, R0);
  const int per_seq = t.u0 + (d->G - 1) * t.u1;
  t.units = (long long)d->B * per_seq;
  if (umma) {
    // the groups side by side where every group is one tile; else ranges over
    // all units, whose weights differ. (148 / G * G blocks: 128 with G = 32 or 64)
    t.step = R0 <= 128 ? d->G : 1;
    t.blocks = kTreeSms / t.step * t.step;
  } else {
    // as many ranges as four blocks an SM allow: one wave up to 32 rows. Of the
    // variant for more (wr = 4, 168 registers) an SM holds three blocks, and up to a
    // quarter of the ranges run after the others.
    t.step = per_seq;
    t.blocks = std::max(1, kTreeSms * 4 / per_seq) * per_seq;
  }
  return t;
}
size_t tree_carve(const gqe_dims* d, bool umma, TreeParams* p, uint8_t* ws) {
  const TreePlan t = tree_plan(d, umma);
  Carver c{ws};
  const size_t rows = (size_t)2 * t.blocks * t.prow;
  float* ml = c.take<float>(rows * 2);
  float* o = c.take<float>(rows * 64);
  int2* cta = c.take<int2>((size_t)t.units);
  if (p) {
    p->part_ml = ml;
    p->part_o = o;
    p->unit_cta = cta;
    p->urows = t.urows;
    p->u0 = t.u0;
    p->u1 = t.u1;
    p->prow = t.prow;
    p->step = t.step;
  }
  return c.off;
}
size_t tree_ws_bytes(const gqe_dims* d) {
  return std::max(tree_carve(d, false, nullptr, nullptr), tree_carve(d, true, nullptr, nullptr));
}

// Sequences, drafted tokens and capacity of the cache operators.
int check_tree_dims(const gqe_dims* d, int cap) {
  GQE_TRY(check_dims(d));
  if (cap < 1) return GQE_ERR_INVALID_ARG;
  if (d->T > kTreeMax || (long long)d->B * cap >= (1ll << 31)) return GQE_ERR_UNSUPPORTED;
  return GQE_OK;
}

int evict_list(const gqe_dims* d) { return d->T / 2 + 1; }
// words of a bit a row; a cluster's shares are whole blocks of rows
int evict_words(const gqe_dims* d) { return (int)cdiv(d->T, 32) + 8 * kEvictWarps; }
size_t evict_ws_bytes(const gqe_dims* d, EvictParams* p, uint8_t* ws) {
  Carver c{ws};
  const size_t bg = (size_t)d->B * d->G;
  int32_t* holes = c.take<int32_t>(bg * evict_list(d));
  int32_t* late = c.take<int32_t>(bg * evict_list(d));
  uint32_t* bits = c.take<uint32_t>(bg * evict_words(d));
  if (p) {
    p->bits = bits;
    p->holes = holes;
    p->late = late;
  }
  return c.off;
}

}  // namespace

extern "C" {

int gqe_qk_rope(const gqe_dims* d, int layout, int rot, float eps, float scale, const void* Q, const void* K,
                const void* wq, const void* wk, const int32_t* sel, const float* inv_freq, const int32_t* positions,
                void* Qo, void* Ko, void* stream) {
  GQE_TRY(check_dims(d));
  if (layout != GQE_ROPE_HALF && layout != GQE_ROPE_INTERLEAVED) return GQE_ERR_INVALID_ARG;
  if (rot < 0 || rot > 64 || (rot & 1) != 0 || !(eps >= 0.f)) return GQE_ERR_INVALID_ARG;
  if ((Q == nullptr) != (Qo == nullptr) || (K == nullptr) != (Ko == nullptr)) return GQE_ERR_INVALID_ARG;
  if (Q == nullptr && K == nullptr) return GQE_ERR_INVALID_ARG;
  if (Q != nullptr && wq != nullptr && sel == nullptr) return GQE_ERR_INVALID_ARG;
  if (rot > 0 && inv_freq == nullptr) return GQE_ERR_INVALID_ARG;
  GQE_TRY(check_opt({Q, K, wq, wk, sel, inv_freq, positions, Qo, Ko}));
  GQE_TRY(check_device());
  RopeParams p;
  memset(&p, 0, sizeof(p));
  p.Q = static_cast<const __nv_bfloat16*>(Q);
  p.K = static_cast<const __nv_bfloat16*>(K);
  p.wq = static_cast<const __nv_bfloat16*>(wq);
  p.wk = static_cast<const __nv_bfloat16*>(wk);
  p.sel = sel;
  p.inv_freq = inv_freq;
  p.positions = positions;
  p.Qo = static_cast<__nv_bfloat16*>(Qo);
  p.Ko = static_cast<__nv_bfloat16*>(Ko);
  p.eps = eps;
  p.scale = scale;
  p.N = d->B * d->T;
  p.T = d->T;
  p.G = d->G;
  p.M = d->M;
  p.k = d->k;
  p.Ha = d->G * d->k + 1;
  p.Hq = Q ? p.Ha : 0;
  p.Hk = K ? d->G : 0;
  p.rot = rot;
  for (p.log2k = 0; (1 << p.log2k) < d->k;) ++p.log2k;
  // a block: as many tokens side by side as 256 threads hold (one where a
  // token's heads alone are more); it walks over chunks of about 16 KB, smaller
  // ones while that leaves SMs without a block
  const int H = p.Hq + p.Hk;
  p.tp = std::min(kRopeMaxTpb, std::max(1, kRopeThreads / 4 / H));
  p.tpb = std::max(1, std::min(kRopeMaxTpb, 128 / H) / p.tp) * p.tp;
  while (p.tpb > p.tp && cdiv(p.N, p.tpb) < 4 * sm_count()) p.tpb -= p.tp;
  if (p.N < p.tp) p.tp = p.tpb = p.N;
  const int nchunk = (int)cdiv(p.N, p.tpb);
  const int smem = kRopeStages * p.tpb * H * 128 + 128;
  const dim3 block((unsigned)(cdiv(4 * H * p.tp, 32) * 32));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  auto run = [&](auto kern) -> int {
    GQE_TRY(set_smem(kern, smem));
    int per_sm = 1;  // blocks an SM holds; asked for only where there are more chunks than SMs
    if (nchunk > sm_count())
      GQE_TRY(cuda_status(cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, (int)block.x, smem)));
    const int most = std::min(nchunk, std::max(1, per_sm) * sm_count());
    p.span = (int)cdiv(cdiv(p.N, most), p.tp) * p.tp;
    return launch_pdl(kern, dim3((unsigned)cdiv(p.N, p.span)), block, smem, st, p);
  };
  const int lay = layout == GQE_ROPE_INTERLEAVED || rot == 0 ? kRopeInterleaved : (rot % 16 == 0 ? kRopeHalf8 : kRopeHalfAny);
  if (block.x > kRopeThreads)
    return lay == kRopeInterleaved ? run(qk_rope_kernel<kRopeInterleaved, kRopeThreadsWide>)
           : lay == kRopeHalf8     ? run(qk_rope_kernel<kRopeHalf8, kRopeThreadsWide>)
                                   : run(qk_rope_kernel<kRopeHalfAny, kRopeThreadsWide>);
  return lay == kRopeInterleaved ? run(qk_rope_kernel<kRopeInterleaved, kRopeThreads>)
         : lay == kRopeHalf8     ? run(qk_rope_kernel<kRopeHalf8, kRopeThreads>)
                                 : run(qk_rope_kernel<kRopeHalfAny, kRopeThreads>);
}

int gqe_tree_attn(const gqe_dims* d, int32_t cap, const void* Q, const void* K_new, const void* V_new,
                  const void* K_cache, const void* V_cache, const int32_t* cache_len, const int32_t* draft_len,
                  const int32_t* parent, void* O, float* lse, void* ws, size_t ws_bytes, void* stream) {
  GQE_TRY(check_tree_dims(d, cap));
  GQE_TRY(check_ptrs({Q, K_new, V_new, K_cache, V_cache, cache_len, O}));
  GQE_TRY(check_opt({draft_len, parent, lse}));
  if (O == Q) return GQE_ERR_INVALID_ARG;
  GQE_TRY(check_ws(ws, ws_bytes, gqe_workspace_bytes(d, GQE_OP_TREE_ATTN)));
  GQE_TRY(check_device());
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool umma = tree_takes_umma(d, cap);
  const TreePlan t = tree_plan(d, umma);
  TreeUmmaParams P;
  memset(&P, 0, sizeof(P));
  TreeParams& p = P.p;
  tree_carve(d, umma, &p, static_cast<uint8_t*>(ws));
  p.Q = static_cast<const __nv_bfloat16*>(Q);
  p.Kn = static_cast<const __nv_bfloat16*>(K_new);
  p.Vn = static_cast<const __nv_bfloat16*>(V_new);
  p.Kc = static_cast<const __nv_bfloat16*>(K_cache);
  p.Vc = static_cast<const __nv_bfloat16*>(V_cache);
  p.cache_len = cache_len;
  p.draft_len = draft_len;
  p.parent = parent;
  p.O = static_cast<__nv_bfloat16*>(O);
  p.lse = lse;
  p.B = d->B;
  p.T = d->T;
  p.G = d->G;
  p.k = d->k;
  p.Ha = d->G * d->k + 1;
  p.cap = cap;
  p.scale_log2 = 1.4426950408889634f / sqrtf(64.f);
  const dim3 grid((unsigned)t.blocks);
  if (umma) {
    GQE_TRY(tmap_group(&P.tmK, K_cache, (long long)d->B * cap, d->G));
    GQE_TRY(tmap_group(&P.tmV, V_cache, (long long)d->B * cap, d->G));
    GQE_TRY(tmap_group(&P.tmKn, K_new, (long long)d->B * d->T, d->G));
    GQE_TRY(tmap_group(&P.tmVn, V_new, (long long)d->B * d->T, d->G));
    GQE_TRY(set_smem(tree_attn_umma_kernel, TuSmem::kBytes));
    GQE_TRY(launch_pdl(tree_attn_umma_kernel, grid, dim3(kTuThreads), TuSmem::kBytes, st, P));
  } else {
    auto run = [&](auto kern) -> int {
      const int smem = kTmSmem + (d->B + 1) * 4;
      GQE_TRY(set_smem(kern, smem));
      return launch_pdl(kern, grid, dim3(kTmThreads), smem, st, p);
    };
    GQE_TRY(t.wr == 1   ? run(tree_attn_mma_kernel<1>)
            : t.wr == 2 ? run(tree_attn_mma_kernel<2>)
                        : run(tree_attn_mma_kernel<4>));
  }
  // the rows that were cut: a block of threads each where the units are few and
  // so cut into many parts, else a warp
  const long long rows = (long long)d->B * d->T * p.Ha;
  if (t.units * 4 < t.blocks)
    return launch_pdl(tree_merge_kernel<8>, dim3((unsigned)rows), dim3(kTreeMergeThreads), 0, st, p);
  return launch_pdl(tree_merge_kernel<2>, dim3((unsigned)cdiv(rows, 4)), dim3(kTreeMergeThreads), 0, st, p);
}

int gqe_tree_commit(const gqe_dims* d, int32_t cap, const int32_t* path, const int32_t* n_acc, const int32_t* positions,
                    const void* Q, const float* lse, const void* K_new, const void* V_new, const int32_t* cache_len,
                    void* K_cache, void* V_cache, int32_t* pos, const float* mass_in, float* mass_out, int32_t* new_len,
                    void* stream) {
  GQE_TRY(check_tree_dims(d, cap));
  GQE_TRY(check_ptrs({K_new, V_new, cache_len, K_cache, V_cache, new_len}));
  GQE_TRY(check_opt({path, n_acc, positions, Q, lse, pos, mass_in, mass_out}));
  if ((mass_in == nullptr) != (mass_out == nullptr)) return GQE_ERR_INVALID_ARG;
  if (mass_in != nullptr && (Q == nullptr || lse == nullptr)) return GQE_ERR_INVALID_ARG;
  if (new_len == cache_len || new_len == n_acc) return GQE_ERR_INVALID_ARG;
  GQE_TRY(check_device());
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  CommitParams p;
  memset(&p, 0, sizeof(p));
  p.path = path;
  p.n_acc = n_acc;
  p.positions = positions;
  p.cache_len = cache_len;
  p.Q = static_cast<const __nv_bfloat16*>(Q);
  p.lse = lse;
  p.Kn = static_cast<const __nv_bfloat16*>(K_new);
  p.Vn = static_cast<const __nv_bfloat16*>(V_new);
  p.Kc = static_cast<__nv_bfloat16*>(K_cache);
  p.Vc = static_cast<__nv_bfloat16*>(V_cache);
  p.pos = pos;
  p.mass_in = mass_in;
  p.mass_out = mass_out;
  p.new_len = new_len;
  p.B = d->B;
  p.T = d->T;
  p.G = d->G;
  p.k = d->k;
  p.Ha = d->G * d->k + 1;
  p.cap = cap;
  p.scale_log2 = 1.4426950408889634f / sqrtf(64.f);
  if (mass_in == nullptr)
    return launch_pdl(commit_append_kernel, dim3((unsigned)(d->B * d->T)), dim3(kAppendThreads), 0, st, p);
  MassParams P;
  memset(&P, 0, sizeof(P));
  P.c = p;
  GQE_TRY(tmap_group(&P.tmK, K_cache, (long long)d->B * cap, d->G));
  const int rows = d->T * (d->k + 1);
  P.nchunk = (int)cdiv(rows, 128);
  P.nstage = kMassMaxStages;
  while (mass_smem(P.nchunk, P.nstage) > 232448) P.nstage -= 2;
  P.step = rows <= 90 ? d->G : 1;
  const int smem = mass_smem(P.nchunk, P.nstage);
  GQE_TRY(set_smem(cache_mass_kernel, smem));
  return launch_pdl(cache_mass_kernel, dim3((unsigned)(kTreeSms / P.step * P.step)), dim3(kMassThreads), smem, st, P);
}

int gqe_cache_evict(const gqe_dims* d, int32_t keep, int32_t sink, int32_t recent, const int32_t* cache_len,
                    const int32_t* next_pos, void* K_cache, void* V_cache, const float* mass_in, float* mass_out,
                    const int32_t* pos_in, int32_t* pos_out, int32_t* new_len, void* ws, size_t ws_bytes,
                    void* stream) {
  GQE_TRY(check_dims(d));
  if (keep < 1 || sink < 0 || recent < 0 || (long long)sink + recent > keep) return GQE_ERR_INVALID_ARG;
  GQE_TRY(check_ptrs({cache_len, next_pos, K_cache, V_cache, mass_in, mass_out, pos_in, pos_out, new_len}));
  if (new_len == cache_len || new_len == next_pos) return GQE_ERR_INVALID_ARG;
  GQE_TRY(check_ws(ws, ws_bytes, gqe_workspace_bytes(d, GQE_OP_CACHE_EVICT)));
  GQE_TRY(check_device());
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  EvictParams p;
  memset(&p, 0, sizeof(p));
  evict_ws_bytes(d, &p, static_cast<uint8_t*>(ws));
  p.cache_len = cache_len;
  p.next_pos = next_pos;
  p.Kc = static_cast<__nv_bfloat16*>(K_cache);
  p.Vc = static_cast<__nv_bfloat16*>(V_cache);
  p.mass_in = mass_in;
  p.mass_out = mass_out;
  p.pos_in = pos_in;
  p.pos_out = pos_out;
  p.new_len = new_len;
  p.B = d->B;
  p.G = d->G;
  p.cap = d->T;
  p.keep = keep;
  p.sink = sink;
  p.recent = recent;
  p.list = evict_list(d);
  p.words = evict_words(d);
  // as many blocks a (sequence, group), up to a portable cluster, as there are SMs
  // for and as have 4096 rows each (8 sequences x 8 groups x 4100 rows: 12.4 us with one
  // block each, 20.6 with two of half as many threads); each holds its keys where
  // they are no more than 160 KB
  const long long bg = (long long)d->B * d->G;
  p.ncta = 1;
  while (p.ncta < 8 && bg * p.ncta * 2 <= kTreeSms && d->T >= 8192 * p.ncta) p.ncta *= 2;
  p.held = std::min((int)cdiv(cdiv(d->T, p.ncta), kEvictThreads) * kEvictThreads, 40960);
  GQE_TRY(set_smem(cache_evict_kernel, p.held * 4));
  return launch_pdl_cluster(cache_evict_kernel, dim3((unsigned)(bg * p.ncta)), dim3(kEvictThreads), p.held * 4, p.ncta, st, p);
}

}  // extern "C"
