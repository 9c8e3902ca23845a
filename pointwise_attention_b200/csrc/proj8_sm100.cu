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
// A CTA computes 128 rows x NT columns of one output tensor (every split point
// is a multiple of 256).  Warp 0 issues TMA loads of 128 x 128 (X8) and
// NT x 128 (W8) byte boxes with the 128-byte swizzle (columns past E and rows
// past T read as zeros), warp 1 allocates TMEM and issues 128 x NT x 32 MMAs,
// warps 2.. are the epilogue, one accumulator row per thread.  Every wait is
// bounded.
#include <cuda_bf16.h>

#include <atomic>

#include "bounds.cuh"
#include "internal.h"
#include "ptx.cuh"
#include "tile_math.cuh"

namespace hstu {
namespace {

constexpr int kBM = 128;                   // rows per tile
constexpr int kBK = 128;                   // K bytes per stage (one 128-byte swizzle row)
constexpr int kABytes = kBM * kBK;         // 16 KB

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
  static constexpr int kSmem = kOffMisc + 16 + 1024;
};

__device__ __forceinline__ bool wait_or_flag(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                             int* status) {
  const bool ok = mbar_wait(bar, parity, abort_flag);
  if (!ok) {
    if (status) atomicOr(status, kStatusTimeout);
    *abort_flag = 1;
  }
  return ok;
}

template <int NT>
__global__ void __launch_bounds__(Cfg<NT>::kThreads, 2)
    uvqk_fp8_sm100(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
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
      // the output tensor and column this tile starts at
      const int Nu = a.Nu, Nq = a.Nq;
      __nv_bfloat16* dst;
      int col, ld;
      if (n0 < Nu) { dst = static_cast<__nv_bfloat16*>(a.out0); col = n0; ld = Nu; }
      else if (n0 < 2 * Nu) { dst = static_cast<__nv_bfloat16*>(a.out1); col = n0 - Nu; ld = Nu; }
      else if (n0 < 2 * Nu + Nq) { dst = static_cast<__nv_bfloat16*>(a.out2); col = n0 - 2 * Nu; ld = Nq; }
      else { dst = static_cast<__nv_bfloat16*>(a.out3); col = n0 - 2 * Nu - Nq; ld = Nq; }
      __nv_bfloat16* drow = dst + static_cast<size_t>(t) * ld + col + c0;
#pragma unroll 1
      for (int c = 0; c < C::kCols / 32; ++c) {
        uint32_t v[32];
        tmem_ld32_nowait(taddr + 32u * c, v);
        tmem_wait_ld_dep(v);
        uint32_t w[16];
        const int n = n0 + c0 + 32 * c;
#pragma unroll
        for (int g = 0; g < 8; ++g) {
          const float4 sw = __ldg(reinterpret_cast<const float4*>(a.w_scale + n) + g);
          const float4 bb = a.bias ? __ldg(reinterpret_cast<const float4*>(a.bias + n) + g)
                                   : make_float4(0.f, 0.f, 0.f, 0.f);
          const float s4[4] = {sw.x, sw.y, sw.z, sw.w}, b4[4] = {bb.x, bb.y, bb.z, bb.w};
          float f[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            f[i] = fmaf(__uint_as_float(v[4 * g + i]) * sx, s4[i], b4[i]);
            if (a.act) f[i] = __fdividef(f[i], 1.0f + __expf(-f[i]));
          }
          w[2 * g] = pack_bf16x2(f[0], f[1]);
          w[2 * g + 1] = pack_bf16x2(f[2], f[3]);
        }
        if (row_ok) {
          if (a.vec32) {
            st_global_v8(drow + 32 * c, reinterpret_cast<const uint32_t(&)[8]>(w[0]));
            st_global_v8(drow + 32 * c + 16, reinterpret_cast<const uint32_t(&)[8]>(w[8]));
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              reinterpret_cast<uint4*>(drow + 32 * c)[i] =
                  make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
          }
        }
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

template <int NT>
cudaError_t launch(const Proj8Args& a, const CUtensorMap& tx, const CUtensorMap& tw,
                   cudaStream_t stream) {
  using C = Cfg<NT>;
  static std::atomic<bool> configured[64];   // per device: shared-memory opt-in done
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev < 0 || dev >= 64 || !configured[dev].load(std::memory_order_acquire)) {
    err = cudaFuncSetAttribute(uvqk_fp8_sm100<NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               C::kSmem);
    if (err != cudaSuccess) return err;
    if (dev >= 0 && dev < 64) configured[dev].store(true, std::memory_order_release);
  }
  const dim3 grid(static_cast<unsigned>((2 * a.Nu + 2 * a.Nq) / NT),
                  static_cast<unsigned>((a.T + kBM - 1) / kBM));
  uvqk_fp8_sm100<NT><<<grid, C::kThreads, C::kSmem, stream>>>(tx, tw, a);
  return cudaGetLastError();
}

}  // namespace

int uvqk_fp8_cols(int T, int N) { return 256; }

cudaError_t launch_uvqk_fp8_sm100(const Proj8Args& a, const CUtensorMap& tx, const CUtensorMap& tw,
                                  cudaStream_t stream) {
  if (a.T == 0) return cudaSuccess;
  return launch<256>(a, tx, tw, stream);
}

}  // namespace hstu
