// cand4_plans.cu -- what the many-candidate kernel needs of the timestamps,
// once for all heads: the time plan (tile_math.cuh) of every candidate against
// every 32-key block of its user's history, and the buckets themselves for the
// history's last four blocks.
//
// The blocks near a history's end span many buckets (the time differences are
// small beside their spread), so no plan fits them and each score would search
// its bucket: two random shared-memory reads per score, where a byte found
// here leaves one.  It matters for short histories, whose only tiles these are
// (32 users x 512 candidates x 8 heads, 128 keys each: 139 -> 131 us, a part of
// it from launching the scoring kernel beside this pass).
//
// CTA (micro-batch of 128 candidates, user; group of kBlocks history blocks);
// warp w takes candidates 128 mt + 32 w + lane, the rows of the scoring kernel's
// epilogue warps, so that the warp's common kind of plan is theirs.
#include "bounds.cuh"
#include "internal_ops.h"
#include "tile_math.cuh"

namespace hstu {
namespace {

constexpr int kThreads = 128;
constexpr int kBlocks = 8;

struct PlanTab {
  const uint4* oct_;
  const unsigned* thr32_;
  __device__ __forceinline__ const uint4* oct() const { return oct_; }
  __device__ __forceinline__ const unsigned* thr32() const { return thr32_; }
};

__global__ void __launch_bounds__(kThreads) hstu_cand4_plans(const __grid_constant__ Cand4Args a) {
  __shared__ uint4 s_oct[32];
  __shared__ unsigned s_thr32[kMaxBuckets];
  __shared__ uint32_t s_ts[kThreads / 32][32];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const unsigned tiles = (static_cast<unsigned>(a.max_cands) + 127u) / 128u;
  const int mt = static_cast<int>(blockIdx.x % tiles), b = static_cast<int>(blockIdx.x / tiles);
  const int c0 = __ldg(a.cand_offsets + b), cb = __ldg(a.cand_offsets + b + 1) - c0;
  const int s = __ldg(a.offsets + b), nb = __ldg(a.offsets + b + 1) - s;
  const int j0 = static_cast<int>(blockIdx.y) * kBlocks;
  // ranges that contradict the sizes are reported by the last kernel (a uniform
  // exit, before any barrier, as for groups of blocks past the history)
  if (c0 < 0 || cb <= 0 || cb > a.C - c0 || s < 0 || nb <= 0 || nb > a.T - s ||
      nb > a.max_seq_len || 128 * mt >= cb || 32 * j0 >= nb)
    return;
  for (int i = threadIdx.x; i < 32; i += kThreads) s_oct[i] = a.bt.oct[i];
  for (int i = threadIdx.x; i < kMaxBuckets; i += kThreads) s_thr32[i] = a.bt.thr32[i];
  __syncthreads();
  const int i = 128 * mt + 32 * warp + lane;         // this thread's candidate of the user
  const bool row_ok = i < cb;
  // candidates past the user's last repeat it, as in the scoring kernel
  const int cand = c0 + (row_ok ? i : cb - 1);
  const long long my_ts = __ldg(a.cand_ts + checked(a.status, cand, a.C, BS_CAND4_ROW));
  const uint32_t my32 = static_cast<uint32_t>(my_ts);
  const int blocks = (nb + 31) / 32, j1 = min(blocks, j0 + kBlocks);
  const PlanTab tab{s_oct, s_thr32};
  uint32_t* ts32 = s_ts[warp];
  // keys past the history repeat its last
  auto column_ts = [&](int jc) {
    return __ldg(a.timestamps + checked(a.status, s + min(32 * jc + lane, nb - 1), a.T, BS_CAND4_TS));
  };
  long long next = column_ts(j0);
  for (int jc = j0; jc < j1; ++jc) {
    const long long kt = next;
    if (jc + 1 < j1) next = column_ts(jc + 1);
    __syncwarp();
    ts32[lane] = static_cast<uint32_t>(kt);
    // the block's extremes: its ends where it ascends, else by reduction
    const long long after = __shfl_down_sync(0xffffffffu, kt, 1);
    const bool asc = !__any_sync(0xffffffffu, lane < 31 && after < kt);
    long long lo = kt, hi = kt;
    if (asc) {
      lo = __shfl_sync(0xffffffffu, kt, 0);
      hi = __shfl_sync(0xffffffffu, kt, 31);
    } else {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const long long x = __shfl_xor_sync(0xffffffffu, lo, o), y = __shfl_xor_sync(0xffffffffu, hi, o);
        lo = x < lo ? x : lo;
        hi = y > hi ? y : hi;
      }
    }
    __syncwarp();
    TimePlan p;
    const int tb = plan_shape_dn(p, my_ts, lo, hi, asc, ts32, tab);
    if (row_ok) a.plan[static_cast<size_t>(jc) * a.C + cand] = plan_word(p, tb);
    // (tb is the warp's: all 32-bit differences where it is TB_GEN32)
    if (blocks - 1 - jc < kCand4Near && tb == TB_GEN32) {
      uint32_t w[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        w[q] = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int d = static_cast<int>(my32 - ts32[4 * q + e]);
          w[q] |= static_cast<uint32_t>(bucket32(static_cast<uint32_t>(d < 0 ? -d : d), tab.oct())) << (8 * e);
        }
      }
      if (row_ok) {
        uint4* dst = a.near + (static_cast<size_t>(blocks - 1 - jc) * a.C + cand) * 2;
        dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
        dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
      }
    }
  }
}

}  // namespace

cudaError_t launch_cand4_plans(const Cand4Args& a, cudaStream_t stream) {
  // (user, micro-batch) in x, the group of history blocks in y
  const dim3 grid(static_cast<unsigned>(a.B) * ((static_cast<unsigned>(a.max_cands) + 127u) / 128u),
                  static_cast<unsigned>(((a.max_seq_len + 31) / 32 + kBlocks - 1) / kBlocks));
  hstu_cand4_plans<<<grid, kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace hstu
