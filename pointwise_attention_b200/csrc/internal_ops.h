// internal_ops.h -- declarations of the 8-bit projection and of scoring against
// the 4-bit cache, shared by the host API and their kernels.
#pragma once
#include "cand4_cut.h"
#include "internal.h"

namespace hstu {

// Check sites of the HSTU_DEBUG_BOUNDS build (bounds.cuh has the others').
constexpr int BS_CAND4_TS = 50, BS_CAND4_ROW = 51, BS_CAND4_KEY = 52, BS_CAND4_SUM = 53;

// Arguments of the UVQK projection of 8-bit rows.
struct Proj8Args {
  const float* x_scale;     // [T]
  const float* w_scale;     // [N]
  const float* bias;        // [N] or nullptr
  void* out0;               // u [T, Nu]
  void* out1;               // v [T, Nu]
  void* out2;               // q [T, Nq]
  void* out3;               // k [T, Nq]
  int* status;
  int T, E, Nu, Nq;
  int act;                  // 1 = SiLU after the bias
  int vec32;                // every output pointer is 32-byte aligned
};

// The outputs u, v, q, k as [T, columns] bf16, boxes of 32 columns x 32 rows
// with the 64-byte swizzle.
struct Proj8Outs {
  CUtensorMap map[4];
};

// Arguments of candidate scoring against histories in a 4-bit cache (kv4.cu
// has the cache's layout).
struct Cand4Args {
  const int32_t* offsets;        // history [B+1]
  const int32_t* cand_offsets;   // candidates [B+1]
  const int32_t* first_rows;     // [B] cache row of each history's first token, or nullptr: offsets
  const int64_t* timestamps;     // history [T] (with a time table)
  const int64_t* cand_ts;        // candidates [C] (with a time table)
  const float* rab_pos;          // [H, 2L-1] or nullptr
  const float* rab_time;         // [H, nb] or nullptr
  const uint8_t* k_codes;        // cache [R, H, 64]
  const uint16_t* k_scales;      // cache [R, H, 4] bf16
  const uint8_t* v_codes;
  const uint16_t* v_scales;
  const void* q;                 // candidates [C, H, 128] bf16
  const void* k;
  const void* v;
  const void* u;                 // candidates [C, H*128]
  void* y;                       // candidates [C, H*128]
  const float* ln_weight;        // [H*128] or nullptr
  const float* ln_bias;
  // workspace: sums over the history, [part_rows][H*128] fp32 (cand4_cut.h has
  // which row is whose)
  float* part;
  size_t part_rows;
  int sum_rows;                  // many candidates: rows of a split's sums
  // workspace (many candidates, with a time table): the time plan of every
  // candidate against every 32-key block of its user's history, a word each,
  // [blocks][C]; and, for the last kCand4Near blocks where the plan is TB_GEN32,
  // the bucket of every score, a byte each, [kCand4Near][C][32]
  uint32_t* plan;
  uint4* near;
  int* status;
  int B, T, C, H, R;
  int max_seq_len, max_cands;
  int L, nb, norm_len;
  int chunk, splits;             // history keys per CTA, CTAs along the longest history
  float eps;
  BucketTable bt;
};

// Kernel launchers (return cudaSuccess or the launch error).
cudaError_t launch_cand4_few(const Cand4Args& a, const Cand4Cut& cut, cudaStream_t stream);
cudaError_t launch_cand4_plans(const Cand4Args& a, cudaStream_t stream);
cudaError_t launch_cand4_sm100(const Cand4Args& a, const CUtensorMap& tq, cudaStream_t stream);
cudaError_t launch_cand4_finish(const Cand4Args& a, const Cand4Cut& cut, bool after_sums,
                                cudaStream_t stream);
int uvqk_fp8_cols(int T, int E, int N);   // columns of a tile of the 8-bit projection
cudaError_t launch_uvqk_fp8_sm100(const Proj8Args& a, const CUtensorMap& tx, const CUtensorMap& tw,
                                  const Proj8Outs& to, cudaStream_t stream);

}  // namespace hstu
