// rab.cu -- the position-bias table of the attention from a short table of
// learned buckets, and its gradient.
//
//   rab_pos[h][L-1+d] = table[h][bucket(d)]   (d = i - j >= 0; entries of later
//                                              keys, d < 0, are 0)
//   d_table[h][k]     = sum over the distances d < L of bucket k of
//                       d_rab_pos[h][L-1+d]
//   bucket(d)         = number of thresholds at or below d
//
// The thresholds ascend, so a bucket is a range of neighbouring distances: the
// forward looks a quad's first bucket up by bisection and steps from there,
// the backward is a sum over ranges.  Both move 4 bytes per table entry and
// are bound by the launch up to some hundred thousand entries, then by HBM.
// Measured on a B200: table of 8 heads x 16383 entries from 32 buckets 6 us;
// gradient of 32 heads x 100003 distances 9 us (12.8 MB; half of it is the
// cluster's start, its barriers and the tables; walking runs of distances and
// segmenting at the borders took 17 us).
#include <cooperative_groups.h>
#include <nvtx3/nvToolsExt.h>

#include <cmath>
#include <cstdint>

#include "hstu.h"
#include "internal.h"

namespace hstu {
namespace {

namespace cg = cooperative_groups;

struct RabArgs {
  const float* in;    // forward: table [H, NB]; backward: d_rab_pos [H, 2L-1]
  float* out;         // forward: rab_pos [H, 2L-1]; backward: d_table [H, NB]
  int L, nb;
  int thr[kMaxBuckets];   // thr[k] = smallest distance of bucket k + 1; entries from nb - 1: INT_MAX
};

// Thresholds at or below d (entries past nb - 1 are INT_MAX, above every d).
__device__ __forceinline__ int find_bucket(const int* thr, int d) {
  int k = 0;
#pragma unroll
  for (int step = kMaxBuckets / 2; step > 0; step >>= 1)
    if (thr[k + step - 1] <= d) k += step;
  return k;
}

constexpr int kFwdThreads = 256;

// Four neighbouring entries per thread, cut so that whole quads are 16-byte
// aligned whatever the row's own alignment (2L - 1 is odd).
__global__ void __launch_bounds__(kFwdThreads) hstu_rab_fwd(const __grid_constant__ RabArgs a) {
  __shared__ float tab[kMaxBuckets];
  __shared__ int thr[kMaxBuckets];
  const int h = static_cast<int>(blockIdx.y);
  const int W = 2 * a.L - 1;
  for (int i = static_cast<int>(threadIdx.x); i < kMaxBuckets; i += kFwdThreads) {
    thr[i] = a.thr[i];
    tab[i] = i < a.nb ? __ldg(a.in + static_cast<size_t>(h) * a.nb + i) : 0.f;
  }
  __syncthreads();
  float* row = a.out + static_cast<size_t>(h) * W;
  const int skew = static_cast<int>((reinterpret_cast<uintptr_t>(row) >> 2) & 3u);
  const int64_t f0 = (static_cast<int64_t>(blockIdx.x) * kFwdThreads + threadIdx.x) * 4 - skew;
  if (f0 >= W) return;
  float v[4] = {0.f, 0.f, 0.f, 0.f};
  const int64_t d0 = f0 - (a.L - 1);
  if (d0 + 3 >= 0) {
    int d = static_cast<int>(d0 < 0 ? 0 : d0);
    int k = find_bucket(thr, d);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (d0 + e < 0) continue;
      while (k < kMaxBuckets - 1 && thr[k] <= d) ++k;
      v[e] = tab[k];
      ++d;
    }
  }
  if (f0 >= 0 && f0 + 3 < W) {
    *reinterpret_cast<float4*>(row + f0) = make_float4(v[0], v[1], v[2], v[3]);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (f0 + e >= 0 && f0 + e < W) row[f0 + e] = v[e];
  }
}

constexpr int kBwdWarps = 16;
constexpr int kPiece = 1024;   // distances of a piece: 32 loads a lane

// One cluster per head.  A bucket's distances are cut into pieces of kPiece, so
// that no piece crosses a border; the cluster's warps take pieces in turn and
// add each one's sum to their own sum of its bucket, in order.  Warps, then
// CTAs, are added in order too, so the result does not depend on timing.
__global__ void __launch_bounds__(32 * kBwdWarps) hstu_rab_bwd(const __grid_constant__ RabArgs a) {
  __shared__ int start[kMaxBuckets + 1];   // first distance of each bucket
  __shared__ int piece0[kMaxBuckets + 1];  // first piece of each bucket
  __shared__ float part[kBwdWarps][kMaxBuckets];
  __shared__ float total[kMaxBuckets];
  cg::cluster_group cluster = cg::this_cluster();
  const int ranks = static_cast<int>(cluster.num_blocks());
  const int rank = static_cast<int>(cluster.block_rank());
  const int h = static_cast<int>(blockIdx.y);
  const int warp = static_cast<int>(threadIdx.x >> 5), lane = static_cast<int>(threadIdx.x & 31);
  for (int i = static_cast<int>(threadIdx.x); i <= kMaxBuckets; i += 32 * kBwdWarps)
    start[i] = i == 0 ? 0 : i >= a.nb ? a.L : min(a.thr[i - 1], a.L);
  for (int i = static_cast<int>(threadIdx.x); i < kBwdWarps * kMaxBuckets; i += 32 * kBwdWarps)
    part[i / kMaxBuckets][i % kMaxBuckets] = 0.f;
  __syncthreads();
  if (warp == 0) {
    // running count of pieces: four buckets per lane, a scan over the lanes
    int n[4], own = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      n[e] = (start[4 * lane + e + 1] - start[4 * lane + e] + kPiece - 1) / kPiece;
      own += n[e];
    }
    int up = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, up, o);
      if (lane >= o) up += y;
    }
    int at = up - own;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      piece0[4 * lane + e] = at;
      at += n[e];
    }
    if (lane == 31) piece0[kMaxBuckets] = at;
  }
  __syncthreads();

  const float* g = a.in + static_cast<size_t>(h) * (2 * static_cast<size_t>(a.L) - 1) + (a.L - 1);
  const int pieces = piece0[kMaxBuckets];
  for (int p = rank + ranks * warp; p < pieces; p += ranks * kBwdWarps) {
    int k = 0;   // the last bucket whose first piece is at or before p
#pragma unroll
    for (int step = kMaxBuckets / 2; step > 0; step >>= 1)
      if (piece0[k + step] <= p) k += step;
    const int lo = start[k] + (p - piece0[k]) * kPiece, n = min(kPiece, start[k + 1] - lo);
    float sum = 0.f;
    if (n <= 256) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (32 * i + lane < n) sum += __ldg(g + lo + 32 * i + lane);
    } else {
      float v[kPiece / 32];
#pragma unroll
      for (int i = 0; i < kPiece / 32; ++i)
        v[i] = 32 * i + lane < n ? __ldg(g + lo + 32 * i + lane) : 0.f;
#pragma unroll
      for (int i = 0; i < kPiece / 32; ++i) sum += v[i];
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) part[warp][k] += sum;
  }
  __syncthreads();
  for (int k = static_cast<int>(threadIdx.x); k < a.nb; k += 32 * kBwdWarps) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kBwdWarps; ++w) s += part[w][k];
    total[k] = s;
  }
  if (ranks > 1) {
    cluster.sync();
    if (rank == 0)
      for (int k = static_cast<int>(threadIdx.x); k < a.nb; k += 32 * kBwdWarps) {
        float s = total[k];
        for (int r = 1; r < ranks; ++r) s += cluster.map_shared_rank(total, r)[k];
        a.out[static_cast<size_t>(h) * a.nb + k] = s;
      }
    cluster.sync();   // the sums stay until they are read
  } else {
    __syncthreads();
    for (int k = static_cast<int>(threadIdx.x); k < a.nb; k += 32 * kBwdWarps)
      a.out[static_cast<size_t>(h) * a.nb + k] = total[k];
  }
}

// ------------------------------------------------------------- host
// Whole numbers of up to 32 * kWords bits, for comparing powers.
struct Big {
  static constexpr int kWords = 128;   // 127 factors below 2^31 take 3937 bits
  uint32_t w[kWords];
  int n;
  Big() : w{1u}, n(1) {}
  void mul(uint32_t m) {
    uint64_t carry = 0;
    for (int i = 0; i < n; ++i) {
      carry += static_cast<uint64_t>(w[i]) * m;
      w[i] = static_cast<uint32_t>(carry);
      carry >>= 32;
    }
    if (carry) w[n++] = static_cast<uint32_t>(carry);
  }
  bool at_least(const Big& o) const {
    if (n != o.n) return n > o.n;
    for (int i = n - 1; i >= 0; --i)
      if (w[i] != o.w[i]) return w[i] > o.w[i];
    return true;
  }
};

hstu_status_t fill(RabArgs* a, int32_t H, int32_t L, int32_t nb, const int32_t* thresholds,
                   const float* in, float* out) {
  if (H < 0 || L < 1 || nb < 1 || nb > kMaxBuckets || (nb > 1 && !thresholds))
    return HSTU_ERR_INVALID_ARG;
  if (static_cast<int64_t>(L) * 2 - 1 > 0x7FFFFFFFll) return HSTU_ERR_INVALID_ARG;
  for (int k = 0; k + 1 < nb; ++k)
    if (thresholds[k] < 1 || (k > 0 && thresholds[k] < thresholds[k - 1])) return HSTU_ERR_INVALID_ARG;
  if (H > 0 && (!in || !out || reinterpret_cast<uintptr_t>(in) % 4 != 0 ||
                reinterpret_cast<uintptr_t>(out) % 4 != 0))
    return HSTU_ERR_INVALID_ARG;
  if (H > 65535) return HSTU_ERR_UNSUPPORTED;
  a->in = in;
  a->out = out;
  a->L = L;
  a->nb = nb;
  for (int k = 0; k < kMaxBuckets; ++k) a->thr[k] = k + 1 < nb ? thresholds[k] : 0x7FFFFFFF;
  return HSTU_OK;
}

struct RabRange {
  explicit RabRange(const char* name) { nvtxRangePushA(name); }
  ~RabRange() { nvtxRangePop(); }
};

}  // namespace
}  // namespace hstu

using namespace hstu;

extern "C" {

HSTU_API int32_t hstu_pos_bucket_thresholds(int32_t* out, int32_t num_buckets, int32_t max_exact,
                                            int32_t max_distance) {
  if (!out || num_buckets < 1 || num_buckets > kMaxBuckets || max_exact < 1 ||
      max_exact > num_buckets || (max_exact < num_buckets && max_distance <= max_exact))
    return -1;
  const int n = num_buckets - max_exact;
  for (int k = 1; k < num_buckets; ++k) {
    if (k <= max_exact) {
      out[k - 1] = k;
      continue;
    }
    // the smallest d with d^n >= max_exact^(n-j) max_distance^j, j = k - max_exact
    const int j = k - max_exact;
    Big bound;
    for (int i = 0; i < n - j; ++i) bound.mul(static_cast<uint32_t>(max_exact));
    for (int i = 0; i < j; ++i) bound.mul(static_cast<uint32_t>(max_distance));
    auto reaches = [&](int64_t d) {
      Big p;
      for (int i = 0; i < n; ++i) p.mul(static_cast<uint32_t>(d));
      return p.at_least(bound);
    };
    const long double guess =
        max_exact * std::pow(static_cast<long double>(max_distance) / max_exact,
                             static_cast<long double>(j) / n);
    int64_t d = static_cast<int64_t>(guess);
    if (d < max_exact) d = max_exact;
    if (d > max_distance) d = max_distance;
    while (!reaches(d)) ++d;                              // ends at max_distance at the latest
    while (d > max_exact && reaches(d - 1)) --d;
    out[k - 1] = static_cast<int32_t>(d);
  }
  return num_buckets - 1;
}

HSTU_API hstu_status_t hstu_rab_bucket_fwd(int32_t H, int32_t L, int32_t num_buckets,
                                           const int32_t* thresholds, const float* table,
                                           float* rab_pos, void* stream) {
  RabRange range("hstu_rab_bucket_fwd");
  RabArgs a;
  const hstu_status_t st = fill(&a, H, L, num_buckets, thresholds, table, rab_pos);
  if (st != HSTU_OK || H == 0) return st;
  const int64_t quads = (2 * static_cast<int64_t>(L) - 1 + 3 + 3) / 4;   // skew up to 3 entries
  const dim3 grid(static_cast<unsigned>((quads + kFwdThreads - 1) / kFwdThreads),
                  static_cast<unsigned>(H));
  hstu_rab_fwd<<<grid, kFwdThreads, 0, static_cast<cudaStream_t>(stream)>>>(a);
  return cudaGetLastError() == cudaSuccess ? HSTU_OK : HSTU_ERR_CUDA;
}

HSTU_API hstu_status_t hstu_rab_bucket_bwd(int32_t H, int32_t L, int32_t num_buckets,
                                           const int32_t* thresholds, const float* d_rab_pos,
                                           float* d_table, void* stream) {
  RabRange range("hstu_rab_bucket_bwd");
  RabArgs a;
  const hstu_status_t st = fill(&a, H, L, num_buckets, thresholds, d_rab_pos, d_table);
  if (st != HSTU_OK || H == 0) return st;
  // about one piece a warp: a CTA's 16 warps take their buckets' short pieces
  // and 4096 distances before a second CTA joins it
  unsigned ranks = 1;
  while (ranks < 8 && static_cast<int64_t>(ranks) * 4096 < L) ranks *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ranks, static_cast<unsigned>(H));
  cfg.blockDim = dim3(32 * kBwdWarps);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ranks;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, hstu_rab_bwd, a) == cudaSuccess ? HSTU_OK : HSTU_ERR_CUDA;
}

}  // extern "C"
