// kv4.cu -- keys and values of cached histories held in 4 bits: writing a
// cache's rows and reading them back.
//
// Each head's 128 values of a token form four groups of 32.  A group has one
// scale s, the smallest number of five significant bits at or above
// max|x| / 7 (kept as bf16), and per value a whole number
//   n = rint(x / s), -7 <= n <= 7, ties to even,   value = n s.
// Three significant bits times five are at most eight, so n s is a bf16
// number: what the attention multiplies is exactly what the cache stands for.
// Rounding s upwards keeps max|x| / s at or below 7 at the cost of at most
// 1/16 of a step.
//
// Layout: codes [rows, H, 64] bytes; eight values make one little-endian
// 32-bit word with value 2i in bits 4i.. and value 2i + 1 in bits 16 + 4i..,
// each as n + 8.  (word >> 4i) & 0x000F000F is then the pair (2i, 2i + 1) in
// the halves of a register, which the readers turn into bf16 pairs.
// Scales [rows, H, 4] bf16.
//
// Both directions move 2 * 256 B of bf16 and 2 * 72 B of cache per token and
// head, once: HBM bounds them.  Measured on a B200, 69637 tokens of 8 heads (365
// MB each way): 135 us for both, 5.4 TB/s (one word a thread, divisions and
// one-element arithmetic: 407 us; four words a thread: 168 us).
#include <cuda_bf16.h>
#include <nvtx3/nvToolsExt.h>

#include <cstdint>

#include "hstu.h"
#include "internal.h"
#include "kv4.cuh"
#include "ptx.cuh"

namespace hstu {
namespace {

constexpr int kThreads = 128;
// A thread takes pairs of words (16 values: 32 bytes of bf16, 8 of codes), so
// that its loads or stores fill whole sectors, P of them kThreads apart: that
// many loads are in flight.  With single words the reading back was bound by
// L1 (90% busy).  P is 8, or 1 where blocks of 8 would leave SMs without one
// (both ways, 8 heads, one kernel after the other in a graph: 32 tokens 2.8 us
// with P = 1 and 6.0 with 8, 2048 tokens 11.0 and 8.0, 69637 tokens 256 and
// 133; 4 and 16 pairs 141 and 145 there).
constexpr int kPairs = 8;
constexpr int kSms = 148;

struct Kv4Args {
  const void* src[2];    // pack: k, v bf16 [T, H, 128]; unpack: codes
  void* dst[2];          // pack: codes; unpack: k, v
  void* scales[2];       // written by pack, read by unpack
  const int32_t* rows;   // [T] cache row of each token, or null (token t: row t)
  int* status;
  int64_t units;         // T * H * 8 pairs of words
  int H, R;              // heads, cache rows
  int vec32;             // k and v are 32-byte aligned
};

// Pair i of the call: token i / (8 H), and the same pair of its cache row.
// Rows outside the cache: -1 marks a token that has none; others are reported.
__device__ __forceinline__ bool cache_pair(const Kv4Args& a, int64_t i, int64_t* at) {
  if (!a.rows) {
    *at = i;
    return true;
  }
  const int64_t per = 8ll * a.H, t = i / per;
  const int row = __ldg(a.rows + t);
  if (row < 0 || row >= a.R) {
    if (row != -1 && a.status) atomicOr(a.status, kStatusBadOffsets);
    return false;
  }
  *at = row * per + (i - t * per);
  return true;
}

// Two neighbouring lanes share a group of 32.
template <int P>
__global__ void __launch_bounds__(kThreads) hstu_kv4_pack_rows(const Kv4Args a) {
  const int which = static_cast<int>(blockIdx.y);
  const int64_t i0 = static_cast<int64_t>(blockIdx.x) * (kThreads * P) + threadIdx.x;
  const uint4* src = static_cast<const uint4*>(a.src[which]);
  uint32_t w[P][8];
#pragma unroll
  for (int j = 0; j < P; ++j) {
    const int64_t i = i0 + j * kThreads;   // units is a multiple of 8: whole groups of lanes
    if (i < a.units && a.vec32) {
      ld_global_nc_v8(src + 2 * i, w[j]);
    } else {
      const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
      const uint4 lo = i < a.units ? __ldg(src + 2 * i) : zero, hi = i < a.units ? __ldg(src + 2 * i + 1) : zero;
      w[j][0] = lo.x; w[j][1] = lo.y; w[j][2] = lo.z; w[j][3] = lo.w;
      w[j][4] = hi.x; w[j][5] = hi.y; w[j][6] = hi.z; w[j][7] = hi.w;
    }
  }
#pragma unroll
  for (int j = 0; j < P; ++j) {
    const int64_t i = i0 + j * kThreads;
    // |x| as bit patterns: ordered like the values, NaN above infinity; the
    // maximum of both halves of a word at once
    uint32_t m = w[j][0] & 0x7FFF7FFFu;
#pragma unroll
    for (int e = 1; e < 8; ++e) m = __vmaxu2(m, w[j][e] & 0x7FFF7FFFu);
    m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 1));
    const float s = kv4_scale(max(m >> 16, m & 0xFFFFu));
    const float inv = kv4_inverse(s);
    const uint64_t inv2 = pack_f32x2(inv, inv);
    uint32_t code[2] = {0u, 0u};
#pragma unroll
    for (int e = 0; e < 8; ++e)
      code[e >> 2] |= (kv4_codes(w[j][e], inv2) & 0x000F000Fu) << (4 * (e & 3));
    int64_t at;
    if (i >= a.units || !cache_pair(a, i, &at)) continue;
    static_cast<uint2*>(a.dst[which])[at] = make_uint2(code[0], code[1]);
    if ((at & 1) == 0)
      static_cast<__nv_bfloat16*>(a.scales[which])[at >> 1] = __float2bfloat16_rn(s);   // exact
  }
}

template <int P>
__global__ void __launch_bounds__(kThreads) hstu_kv4_unpack_rows(const Kv4Args a) {
  const int which = static_cast<int>(blockIdx.y);
  const int64_t i0 = static_cast<int64_t>(blockIdx.x) * (kThreads * P) + threadIdx.x;
  uint2 code[P];
  uint32_t scale[P];
  bool live[P];
#pragma unroll
  for (int j = 0; j < P; ++j) {
    const int64_t i = i0 + j * kThreads;
    int64_t at;
    live[j] = i < a.units && cache_pair(a, i, &at);
    if (live[j]) {
      code[j] = __ldg(static_cast<const uint2*>(a.src[which]) + at);
      scale[j] = __ldg(static_cast<const uint16_t*>(a.scales[which]) + (at >> 1));
    }
  }
#pragma unroll
  for (int j = 0; j < P; ++j) {
    if (!live[j]) continue;
    const uint32_t s2 = scale[j] | (scale[j] << 16);
    const uint32_t o[8] = {kv4_pair<0>(code[j].x, s2), kv4_pair<1>(code[j].x, s2),
                           kv4_pair<2>(code[j].x, s2), kv4_pair<3>(code[j].x, s2),
                           kv4_pair<0>(code[j].y, s2), kv4_pair<1>(code[j].y, s2),
                           kv4_pair<2>(code[j].y, s2), kv4_pair<3>(code[j].y, s2)};
    uint4* dst = static_cast<uint4*>(a.dst[which]) + 2 * (i0 + j * kThreads);
    if (a.vec32) {
      st_global_v8(dst, o);
    } else {
      dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
      dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
    }
  }
}

struct Kv4Range {
  explicit Kv4Range(const char* name) { nvtxRangePushA(name); }
  ~Kv4Range() { nvtxRangePop(); }
};

hstu_status_t run(bool pack, int32_t T, int32_t H, int32_t cache_rows, const int32_t* rows,
                  const void* k, const void* v, const void* kc, const void* ks, const void* vc,
                  const void* vs, void* workspace, size_t workspace_bytes, void* stream) {
  if (T < 0 || H < 1 || cache_rows < 0 || (!rows && cache_rows < T)) return HSTU_ERR_INVALID_ARG;
  if (T > 0) {
    const void* ptrs[] = {k, v, kc, ks, vc, vs};
    for (const void* p : ptrs)
      if (!p || reinterpret_cast<uintptr_t>(p) % 16 != 0) return HSTU_ERR_INVALID_ARG;
  }
  if (reinterpret_cast<uintptr_t>(rows) % 4 != 0) return HSTU_ERR_INVALID_ARG;
  // blocks of at least kThreads pairs of words in grid x
  const int64_t units = 8ll * T * H;
  if (H > 65536 || units > 0x7FFFFFFFll * kThreads) return HSTU_ERR_UNSUPPORTED;
  // only the cache rows given by index can be found wrong on the device
  if ((rows || workspace) && (!workspace || reinterpret_cast<uintptr_t>(workspace) % 256 != 0 ||
                              workspace_bytes < 256))
    return HSTU_ERR_WORKSPACE;
  if (T == 0) return HSTU_OK;
  Kv4Args a;
  a.src[0] = pack ? k : kc;
  a.src[1] = pack ? v : vc;
  a.dst[0] = const_cast<void*>(pack ? kc : k);
  a.dst[1] = const_cast<void*>(pack ? vc : v);
  a.scales[0] = const_cast<void*>(ks);
  a.scales[1] = const_cast<void*>(vs);
  a.rows = rows;
  a.status = static_cast<int*>(workspace);
  a.units = units;
  a.H = H;
  a.R = cache_rows;
  a.vec32 = reinterpret_cast<uintptr_t>(k) % 32 == 0 && reinterpret_cast<uintptr_t>(v) % 32 == 0;
  const int64_t many = (units + kThreads * kPairs - 1) / (kThreads * kPairs);
  const bool few = 2 * many < kSms;
  const dim3 grid(static_cast<unsigned>(few ? (units + kThreads - 1) / kThreads : many), 2);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const auto kernel = pack ? (few ? hstu_kv4_pack_rows<1> : hstu_kv4_pack_rows<kPairs>)
                           : (few ? hstu_kv4_unpack_rows<1> : hstu_kv4_unpack_rows<kPairs>);
  kernel<<<grid, kThreads, 0, s>>>(a);
  return cudaGetLastError() == cudaSuccess ? HSTU_OK : HSTU_ERR_CUDA;
}

}  // namespace
}  // namespace hstu

extern "C" {

HSTU_API hstu_status_t hstu_kv4_pack(int32_t T, int32_t H, const void* k, const void* v,
                                     const int32_t* rows, int32_t cache_rows, void* k_codes,
                                     void* k_scales, void* v_codes, void* v_scales,
                                     void* workspace, size_t workspace_bytes, void* stream) {
  hstu::Kv4Range range("hstu_kv4_pack");
  return hstu::run(true, T, H, cache_rows, rows, k, v, k_codes, k_scales, v_codes, v_scales,
                   workspace, workspace_bytes, stream);
}

HSTU_API hstu_status_t hstu_kv4_unpack(int32_t T, int32_t H, const void* k_codes,
                                       const void* k_scales, const void* v_codes,
                                       const void* v_scales, const int32_t* rows,
                                       int32_t cache_rows, void* k, void* v, void* workspace,
                                       size_t workspace_bytes, void* stream) {
  hstu::Kv4Range range("hstu_kv4_unpack");
  return hstu::run(false, T, H, cache_rows, rows, k, v, k_codes, k_scales, v_codes, v_scales,
                   workspace, workspace_bytes, stream);
}

}  // extern "C"
