// proj8_sm100.cu -- the UVQK projection of 8-bit rows on sm_100a.
//
//   [U | V | Q | K] = act((X8 W8^T) sx_t sw_n + b_n)
//   X8 [T, E], W8 [H(2dv+2dqk), E] e4m3 with one fp32 scale per row
//
// ("HSTU (Generative Recommender)" model card, HSTUBlock.uvqk; the optional
// SiLU is the reproduction note's SiLU(Norm(X) W_UVQK).)  The scales of a row
// of X and of a row of W are constant over a sum, so they are applied to the
// fp32 accumulator; the outputs are rounded to bf16 once.
//
// Two kernels.  For E <= 1024 a CTA keeps one block of NT columns of W8 (all of
// its K) in shared memory and walks the row tiles, so that per 128 x NT outputs
// only 128 rows of X8 are brought in: reading both operands anew for every tile
// would move as many bytes out of L2 as the outputs move into HBM, which is
// what should bound the call.  Accumulators are double-buffered in TMEM: the
// epilogue of one tile runs under the MMAs of the next.  For wider rows a
// kernel that streams both operands.
// In both, warp 0 issues TMA loads of 128-byte-wide boxes with the 128-byte
// swizzle (columns past E and rows past T read as zeros), warp 1 allocates TMEM
// and issues 128 x NT x 32 MMAs, warps 2.. are the epilogue, one accumulator
// row per thread.  Every wait is bounded.
//
// Measured on a B200: 131072 x 512 by 2048 columns with SiLU, 605 MB, 275 GFLOP:
// 156 us = 1.76 PFLOP/s = 3.9 TB/s by itself, 164 us in a row of calls and 188 us
// where the GPU waits for the call's host side (bf16 operands: 0.40 ms).  Shared
// memory bounds it (operands, staged outputs, column scales: 84% busy), with HBM
// at 39% and the tensor cores at 40%; a plain fill of the 537 MB of outputs takes
// 141 us.
#include <cuda_bf16.h>

#include <atomic>

#include "bounds.cuh"
#include "internal_ops.h"
#include "ops.cuh"
#include "ptx.cuh"
#include "tile_math.cuh"

namespace hstu {
namespace {

constexpr int kBM = 128;                   // rows per tile
constexpr int kBK = 128;                   // K bytes per stage (one 128-byte swizzle row)
constexpr int kABytes = kBM * kBK;         // 16 KB

__device__ __forceinline__ bool wait_or_flag(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                             int* status) {
  const bool ok = mbar_wait(bar, parity, abort_flag);
  if (!ok) {
    if (status) atomicOr(status, kStatusTimeout);
    *abort_flag = 1;
  }
  return ok;
}

// SiLU(x) from h = x / 2: h (1 + tanh h), relative error of the tanh at most
// 2^-11; measured over -16 < x < 16 the result is off by |x| 2^-19 at most.
// (x / (1 + 2^(-x log2 e)) with the hardware's power and reciprocal, or with a
// reciprocal by a polynomial and a Newton step: 198 to 212 us where this takes
// 164 to 181, 131072 x 512 by 2048 columns in a row of calls.)
__device__ __forceinline__ uint64_t silu2(uint64_t h2) {
  const float2 h = unpack_f32x2(h2);
  return ffma2(h2, pack_f32x2(tanh_approx(h.x), tanh_approx(h.y)), h2);
}

// The output tensor and column that column n0 of the projection belongs to.
struct Dest {
  __nv_bfloat16* base;   // of column n0
  int ld, which, col;    // which output tensor, and the column in it
};
__device__ __forceinline__ Dest dest_of(const Proj8Args& a, int n0) {
  const int Nu = a.Nu, Nq = a.Nq;
  int which = 0, col = n0;
  if (col >= 2 * Nu) {
    col -= 2 * Nu;
    which = 2 + (col >= Nq);
    col -= which == 3 ? Nq : 0;
  } else if (col >= Nu) {
    col -= Nu;
    which = 1;
  }
  void* const out[4] = {a.out0, a.out1, a.out2, a.out3};
  return {static_cast<__nv_bfloat16*>(out[which]) + col, which < 2 ? Nu : Nq, which, col};
}

// 32 neighbouring outputs of a row from their accumulators: (acc sx) sw + b,
// SiLU, one rounding.  sw and bias: 32 values each, halved where act is set.
__device__ __forceinline__ void outputs32(const uint32_t (&v)[32], float sx, const float* sw,
                                          const float* bias, int act, uint32_t (&w)[16]) {
  const uint64_t sx2 = pack_f32x2(sx, sx);
#pragma unroll
  for (int g = 0; g < 8; ++g) {
    const float4 s4 = *reinterpret_cast<const float4*>(sw + 4 * g);
    const float4 b4 = *reinterpret_cast<const float4*>(bias + 4 * g);
    uint64_t p0 = fmul2(pack_f32x2(__uint_as_float(v[4 * g]), __uint_as_float(v[4 * g + 1])), sx2);
    uint64_t p1 = fmul2(pack_f32x2(__uint_as_float(v[4 * g + 2]), __uint_as_float(v[4 * g + 3])), sx2);
    p0 = ffma2(p0, pack_f32x2(s4.x, s4.y), pack_f32x2(b4.x, b4.y));
    p1 = ffma2(p1, pack_f32x2(s4.z, s4.w), pack_f32x2(b4.z, b4.w));
    if (act) {
      p0 = silu2(p0);
      p1 = silu2(p1);
    }
    const float2 f0 = unpack_f32x2(p0), f1 = unpack_f32x2(p1);
    w[2 * g] = pack_bf16x2(f0.x, f0.y);
    w[2 * g + 1] = pack_bf16x2(f1.x, f1.y);
  }
}

// 32 bf16 (64 bytes) of one row, as two 32-byte or four 16-byte stores.
__device__ __forceinline__ void store_row32(__nv_bfloat16* dst, const uint32_t (&w)[16], bool v32) {
  if (v32) {
    st_global_v8(dst, reinterpret_cast<const uint32_t(&)[8]>(w[0]));
    st_global_v8(dst + 16, reinterpret_cast<const uint32_t(&)[8]>(w[8]));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      reinterpret_cast<uint4*>(dst)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
  }
}

// The scales and biases of columns n0.. in shared memory.
template <int NT, int THREADS>
__device__ __forceinline__ void load_columns(const Proj8Args& a, int n0, float* sw, float* sb) {
  const float f = a.act ? 0.5f : 1.0f;
  for (int i = static_cast<int>(threadIdx.x); i < NT; i += THREADS) {
    sw[i] = f * __ldg(a.w_scale + n0 + i);
    sb[i] = a.bias ? f * __ldg(a.bias + n0 + i) : 0.f;
  }
}

// ------------------------------------------------------- W in shared memory
constexpr int kStagesX = 3;
constexpr int kMaxW = 131072;              // bytes of W8 kept: NT columns x (E up to 128s)

template <int NT>
struct Keep {
  // Epilogue warps per TMEM lane quarter: with two of them (eight warps) the
  // epilogue's latencies bound 131072 x 512 x 2048 at 177 us.
  static constexpr int S = NT >= 128 ? 4 : NT / 32;
  static constexpr int kThreads = 64 + 128 * S;
  static constexpr int kCols = NT / S;         // per epilogue thread
  static constexpr int kTmem = 2 * NT;         // two accumulators
  // barriers: X full, X empty, W full, accumulator full, accumulator empty
  static constexpr int B_XFULL = 0, B_XEMPTY = kStagesX, B_W = 2 * kStagesX, B_TFULL = B_W + 1,
                       B_TEMPTY = B_TFULL + 2, kNumBars = B_TEMPTY + 2;
  static constexpr int kOffX = 0;                           // stages of X
  // Outputs leave by TMA, 32 rows x 32 columns a warp at a time: stores of the
  // threads themselves (a row each) kept the load/store unit 91% busy.
  static constexpr int kOffOut = kStagesX * kABytes;        // 2 KB a warp
  static constexpr int kOffCols = kOffOut + 4 * S * 2048;   // float [2][NT]
  static constexpr int kOffBar = kOffCols + 8 * NT;
  static constexpr int kOffMisc = kOffBar + 8 * kNumBars;
  static constexpr int kOffW = (kOffMisc + 16 + 1023) / 1024 * 1024;
  static int smem(int nk) { return kOffW + nk * NT * kBK + 1024; }
};
static_assert(Keep<256>::kOffCols % 16 == 0 && Keep<32>::kOffCols % 16 == 0, "read as float4");
static_assert(Keep<256>::kOffW + kMaxW + 1024 <= 227 * 1024, "shared memory per CTA");

template <int NT>
__global__ void __launch_bounds__(Keep<NT>::kThreads, 1)
    uvqk_fp8_keep(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
                  const __grid_constant__ Proj8Outs tm_out, const __grid_constant__ Proj8Args a) {
  using C = Keep<NT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(smem);
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);
  const int lane = threadIdx.x & 31;
  auto bar = [&](int i) { return sbase + C::kOffBar + 8u * i; };
  uint32_t* misc = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + 1);
  float* s_sw = reinterpret_cast<float*>(smem + C::kOffCols);
  // CTA (column block, first row tile): row tiles every `step` from there
  const int blocks = (2 * a.Nu + 2 * a.Nq) / NT;
  const int n0 = static_cast<int>(blockIdx.x) % blocks * NT;
  const int first = static_cast<int>(blockIdx.x) / blocks, step = static_cast<int>(gridDim.x) / blocks;
  const int tiles = (a.T + kBM - 1) / kBM;
  const int nk = (a.E + kBK - 1) / kBK;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kNumBars; ++i) mbar_init(bar(i), i >= C::B_TEMPTY ? 4 * C::S : 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(sbase + C::kOffMisc, C::kTmem);
    tmem_relinquish();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tm_a);
    tma_prefetch_desc(&tm_b);
  }
  load_columns<NT, C::kThreads>(a, n0, s_sw, s_sw + NT);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = misc[0];

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0) {
      mbar_arrive_expect_tx(bar(C::B_W), static_cast<uint32_t>(nk * NT * kBK));
      for (int kb = 0; kb < nk; ++kb)
        tma_load_2d(sbase + C::kOffW + kb * NT * kBK, &tm_b, bar(C::B_W), kb * kBK, n0);
      bool ok = true;
      unsigned use = 0;
      for (int m = first; m < tiles && ok; m += step)
        for (int kb = 0; kb < nk; ++kb, ++use) {
          const unsigned st = use % kStagesX, turn = use / kStagesX;
          if (turn > 0) ok = wait_or_flag(bar(C::B_XEMPTY + st), (turn - 1) & 1u, abort_flag, a.status);
          if (!ok) break;
          mbar_arrive_expect_tx(bar(C::B_XFULL + st), kABytes);
          tma_load_2d(sbase + C::kOffX + st * kABytes, &tm_a, bar(C::B_XFULL + st), kb * kBK,
                      checked(a.status, m * kBM, a.T, BS_PROJ_TMA));
        }
      if (!ok) {   // let the copies already issued land before shared memory goes away
        mbar_wait(bar(C::B_W), 0, nullptr);
        for (unsigned u = use > kStagesX ? use - kStagesX : 0u; u < use; ++u)
          mbar_wait(bar(C::B_XFULL + u % kStagesX), (u / kStagesX) & 1u, nullptr);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    constexpr uint32_t idesc = idesc_e4m3_f32(128, NT);
    bool ok = true;
    auto wait = [&](int i, unsigned parity) {
      if (ok)
        ok = __all_sync(0xffffffffu, wait_or_flag(bar(i), parity & 1u, abort_flag, a.status));
    };
    wait(C::B_W, 0);
    unsigned use = 0, n = 0;
    for (int m = first; m < tiles && ok; m += step, ++n) {
      const unsigned acc = n & 1u;
      if (n >= 2) wait(C::B_TEMPTY + acc, n / 2 - 1);
      for (int kb = 0; kb < nk && ok; ++kb, ++use) {
        const unsigned st = use % kStagesX;
        wait(C::B_XFULL + st, use / kStagesX);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          const uint64_t ad = sw128_desc(sbase + C::kOffX + st * kABytes, 16, 1024);
          const uint64_t bd = sw128_desc(sbase + C::kOffW + kb * NT * kBK, 16, 1024);
#pragma unroll
          for (int ks = 0; ks < kBK / 32; ++ks)
            mma_ss_f8(tmem + acc * NT, ad + 2 * ks, bd + 2 * ks, idesc, (kb > 0 || ks > 0) ? 1u : 0u);
          mma_commit(bar(C::B_XEMPTY + st));
          if (kb == nk - 1) mma_commit(bar(C::B_TFULL + acc));
        }
        __syncwarp();
      }
    }
    // TMEM is released only after the MMAs issued here have finished writing
    // it: the last commit to each X stage covers them.
    for (unsigned u = use > kStagesX ? use - kStagesX : 0u; u < use; ++u)
      mbar_wait(bar(C::B_XEMPTY + u % kStagesX), (u / kStagesX) & 1u, nullptr);
  } else {
    // ------------------------------------------------------------ epilogue
    const int q4 = warp & 3, cs = (warp - 2) >> 2;
    const int c0 = cs * C::kCols;
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>(32 * q4) << 16) + c0;
    const Dest d = dest_of(a, n0);
    const int r = 32 * q4 + lane;
    auto scale_of = [&](int m) {
      const int t = m * kBM + r;
      return m < tiles && t < a.T ? __ldg(a.x_scale + t) : 0.f;
    };
    float sx = scale_of(first);
    bool ok = true;
    unsigned n = 0;
    for (int m = first; m < tiles && ok; m += step, ++n) {
      const unsigned acc = n & 1u;
      const float snext = scale_of(m + step);
      ok = wait_or_flag(bar(C::B_TFULL + acc), (n / 2) & 1u, abort_flag, a.status) && !*abort_flag;
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      const uint32_t out = sbase + C::kOffOut + static_cast<uint32_t>(warp - 2) * 2048u;
#pragma unroll 1
      for (int c = 0; c < C::kCols; c += 32) {
        uint32_t v[32], w[16];
        tmem_ld32_nowait(lane_addr + acc * NT + c, v);
        tmem_wait_ld_dep(v);
        if (c + 32 == C::kCols) {
          // the accumulator is in registers: the next tile but one may have it
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(C::B_TEMPTY + acc));
        }
        outputs32(v, sx, s_sw + c0 + c, s_sw + NT + c0 + c, a.act, w);
        if (lane == 0) bulk_wait_group_read0();   // the box before has been read
        __syncwarp();
        // a 64-byte row of the box (64-byte swizzle)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          st_shared_v4(out + lane * 64 + (i ^ ((lane >> 1) & 3)) * 16,
                       make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]));
        fence_proxy_async_smem();
        __syncwarp();
        // (rows past T inside the box are not written; a box past T is not sent)
        if (lane == 0 && m * kBM + 32 * q4 < a.T) {
          tma_store_2d(&tm_out.map[d.which], out, d.col + c0 + c, m * kBM + 32 * q4);
          bulk_commit_group();
        }
      }
      sx = snext;
    }
    if (lane == 0) bulk_wait_group0();
    tc_fence_before();
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmem);
  }
}

// ------------------------------------------------------- both streamed
template <int NT>
struct Cfg {
  static constexpr int S = NT >= 64 ? 2 : 1;   // epilogue warps per TMEM lane quarter
  static constexpr int kThreads = 64 + 128 * S;
  static constexpr int kCols = NT / S;         // per epilogue thread
  static constexpr int kBBytes = NT * kBK;
  static constexpr int kStage = kABytes + kBBytes;
  static constexpr int kStages = NT == 256 ? 2 : 4;
  static constexpr int kOffBar = kStages * kStage;
  static constexpr int kNumBars = 2 * kStages + 1;
  static constexpr int kOffMisc = kOffBar + kNumBars * 8;
  static constexpr int kOffCols = (kOffMisc + 16 + 15) / 16 * 16;   // float [2][NT]
  static constexpr int kSmem = kOffCols + 8 * NT + 1024;
};

template <int NT>
__global__ void __launch_bounds__(Cfg<NT>::kThreads, 2)
    uvqk_fp8_stream(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
                   const __grid_constant__ Proj8Args a) {
  using C = Cfg<NT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto bar = [&](int i) { return sbase + C::kOffBar + 8u * i; };
  const int B_FULL = 0, B_EMPTY = C::kStages, B_TFULL = 2 * C::kStages;
  uint32_t* misc = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + 1);
  // x = column block, y = row tile: CTAs resident together share one X tile
  // through L2 (W stays there)
  const int m0 = static_cast<int>(blockIdx.y) * kBM;
  const int n0 = static_cast<int>(blockIdx.x) * NT;
  const int nk = (a.E + kBK - 1) / kBK;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kNumBars; ++i) mbar_init(bar(i), 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(sbase + C::kOffMisc, NT);
    tmem_relinquish();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tm_a);
    tma_prefetch_desc(&tm_b);
  }
  float* s_sw = reinterpret_cast<float*>(smem + C::kOffCols);
  load_columns<NT, C::kThreads>(a, n0, s_sw, s_sw + NT);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = misc[0];

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0) {
      int last[C::kStages];
      for (int s = 0; s < C::kStages; ++s) last[s] = -1;
      bool ok = true;
      for (int kb = 0; kb < nk && ok; ++kb) {
        const int st = kb % C::kStages, use = kb / C::kStages;
        if (use > 0) ok = wait_or_flag(bar(B_EMPTY + st), (use - 1) & 1, abort_flag, a.status);
        if (!ok) break;
        const uint32_t dst = sbase + st * C::kStage;
        mbar_arrive_expect_tx(bar(B_FULL + st), C::kStage);
        tma_load_2d(dst, &tm_a, bar(B_FULL + st), kb * kBK, checked(a.status, m0, a.T, BS_PROJ_TMA));
        tma_load_2d(dst + kABytes, &tm_b, bar(B_FULL + st), kb * kBK, n0);
        last[st] = use;
      }
      if (!ok)   // let the copies already issued land before shared memory goes away
        for (int s = 0; s < C::kStages; ++s)
          if (last[s] >= 0) mbar_wait(bar(B_FULL + s), last[s] & 1, nullptr);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      constexpr uint32_t idesc = idesc_e4m3_f32(128, NT);
      bool ok = true;
      for (int kb = 0; kb < nk && ok; ++kb) {
        const int st = kb % C::kStages;
        ok = wait_or_flag(bar(B_FULL + st), (kb / C::kStages) & 1, abort_flag, a.status);
        if (!ok) break;
        tc_fence_after();
        const uint32_t sa = sbase + st * C::kStage, sb = sa + kABytes;
#pragma unroll
        for (int ks = 0; ks < kBK / 32; ++ks)
          mma_ss_f8(tmem, sw128_desc(sa + ks * 32, 16, 1024), sw128_desc(sb + ks * 32, 16, 1024),
                    idesc, (kb > 0 || ks > 0) ? 1u : 0u);
        mma_commit(bar(B_EMPTY + st));
      }
      mma_commit(bar(B_TFULL));   // every MMA issued has completed (or none was)
      // TMEM is released only after the MMAs issued here have finished writing it.
      mbar_wait(bar(B_TFULL), 0, nullptr);
    }
  } else {
    // ------------------------------------------------------------ epilogue
    const int q4 = warp & 3;                         // TMEM lane quarter of this warp
    const int cs = (warp - 2) >> 2;                  // column slice 0..S-1
    const int t = m0 + 32 * q4 + lane;               // row = TMEM lane
    const bool row_ok = t < a.T;
    const int c0 = cs * C::kCols;                    // first tile column of the slice
    const float sx = row_ok ? __ldg(a.x_scale + t) : 0.f;
    const uint32_t taddr = tmem + (static_cast<uint32_t>(32 * q4) << 16) + c0;
    bool ok = wait_or_flag(bar(B_TFULL), 0, abort_flag, a.status) && !*abort_flag;
    ok = __all_sync(0xffffffffu, ok);
    if (ok) {
      tc_fence_after();
      const Dest d = dest_of(a, n0);
      __nv_bfloat16* drow = d.base + static_cast<size_t>(t) * d.ld + c0;
#pragma unroll 1
      for (int c = 0; c < C::kCols; c += 32) {
        uint32_t v[32], w[16];
        tmem_ld32_nowait(taddr + c, v);
        tmem_wait_ld_dep(v);
        outputs32(v, sx, s_sw + c0 + c, s_sw + NT + c0 + c, a.act, w);
        if (row_ok) store_row32(drow + c, w, a.vec32);
      }
    }
    tc_fence_before();
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, NT);
  }
}

template <typename K>
cudaError_t configure(K kernel, int smem) {
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
}

template <int NT>
cudaError_t launch_keep(const Proj8Args& a, const CUtensorMap& tx, const CUtensorMap& tw,
                        const Proj8Outs& to, cudaStream_t stream) {
  static std::atomic<bool> configured[64];   // per device: shared-memory opt-in done
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev < 0 || dev >= 64 || !configured[dev].load(std::memory_order_acquire)) {
    err = configure(uvqk_fp8_keep<NT>, Keep<NT>::smem(kMaxW / (NT * kBK)));
    if (err != cudaSuccess) return err;
    if (dev >= 0 && dev < 64) configured[dev].store(true, std::memory_order_release);
  }
  // as many CTAs per column block as there are row tiles and SMs for
  const int blocks = (2 * a.Nu + 2 * a.Nq) / NT, tiles = (a.T + kBM - 1) / kBM;
  int per = 148 / blocks;
  per = per < 1 ? 1 : per > tiles ? tiles : per;
  const int nk = (a.E + kBK - 1) / kBK;
  uvqk_fp8_keep<NT><<<static_cast<unsigned>(blocks) * per, Keep<NT>::kThreads, Keep<NT>::smem(nk),
                      stream>>>(tx, tw, to, a);
  return cudaGetLastError();
}

cudaError_t launch_stream(const Proj8Args& a, const CUtensorMap& tx, const CUtensorMap& tw,
                          cudaStream_t stream) {
  using C = Cfg<256>;
  static std::atomic<bool> configured[64];   // per device: shared-memory opt-in done
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev < 0 || dev >= 64 || !configured[dev].load(std::memory_order_acquire)) {
    err = configure(uvqk_fp8_stream<256>, C::kSmem);
    if (err != cudaSuccess) return err;
    if (dev >= 0 && dev < 64) configured[dev].store(true, std::memory_order_release);
  }
  const dim3 grid(static_cast<unsigned>((2 * a.Nu + 2 * a.Nq) / 256),
                  static_cast<unsigned>((a.T + kBM - 1) / kBM));
  uvqk_fp8_stream<256><<<grid, C::kThreads, C::kSmem, stream>>>(tx, tw, a);
  return cudaGetLastError();
}

static_assert(Cfg<256>::kOffCols % 16 == 0, "read as float4");

}  // namespace

// Columns of a tile: 256 where that makes at least a tile per SM, fewer for
// fewer rows (17 rows by 4096 columns: 18 us with 256 columns a CTA, on 16 SMs),
// and where W's block would not fit shared memory.
int uvqk_fp8_cols(int T, int E, int N) {
  const int nk = (E + kBK - 1) / kBK;
  if (nk > kMaxW / (128 * kBK)) return 256;   // streamed
  const int64_t tiles = (static_cast<int64_t>(T) + kBM - 1) / kBM;
  int nt = 256;
  while (nt > 32 && (nk * nt * kBK > kMaxW || tiles * (N / nt) < 148)) nt /= 2;
  return nt;
}

cudaError_t launch_uvqk_fp8_sm100(const Proj8Args& a, const CUtensorMap& tx, const CUtensorMap& tw,
                                  const Proj8Outs& to, cudaStream_t stream) {
  if (a.T == 0) return cudaSuccess;
  if ((a.E + kBK - 1) / kBK > kMaxW / (128 * kBK)) return launch_stream(a, tx, tw, stream);
  switch (uvqk_fp8_cols(a.T, a.E, 2 * a.Nu + 2 * a.Nq)) {
    case 256: return launch_keep<256>(a, tx, tw, to, stream);
    case 128: return launch_keep<128>(a, tx, tw, to, stream);
    case 64: return launch_keep<64>(a, tx, tw, to, stream);
    default: return launch_keep<32>(a, tx, tw, to, stream);
  }
}

}  // namespace hstu
