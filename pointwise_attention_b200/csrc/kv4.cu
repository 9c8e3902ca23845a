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
// MB each way): 168 us for both, 4.4 TB/s (one word a thread, divisions and
// one-element arithmetic: 407 us).
#include <cuda_bf16.h>
#include <nvtx3/nvToolsExt.h>

#include <cstdint>

#include "hstu.h"
#include "internal.h"
#include "kv4.cuh"

namespace hstu {
namespace {

constexpr int kThreads = 256;
constexpr int kWords = 4;   // words of a thread, kThreads apart: that many loads in flight

struct Kv4Args {
  const void* src[2];    // pack: k, v bf16 [T, H, 128]; unpack: codes
  void* dst[2];          // pack: codes; unpack: k, v
  void* scales[2];       // written by pack, read by unpack
  const int32_t* rows;   // [T] cache row of each token, or null (token t: row t)
  int* status;
  int64_t units;         // T * H * 16 words of eight values
  int H, R;              // heads, cache rows
};

// Word i of the call: token i / (16 H), and the same word of its cache row.
// Rows outside the cache: -1 marks a token that has none; others are reported.
__device__ __forceinline__ bool cache_word(const Kv4Args& a, int64_t i, int64_t* at) {
  if (!a.rows) {
    *at = i;
    return true;
  }
  const int64_t per = 16ll * a.H, t = i / per;
  const int row = __ldg(a.rows + t);
  if (row < 0 || row >= a.R) {
    if (row != -1 && a.status) atomicOr(a.status, kStatusBadOffsets);
    return false;
  }
  *at = row * per + (i - t * per);
  return true;
}

// Four neighbouring lanes share a group of 32.
__global__ void __launch_bounds__(kThreads) hstu_kv4_pack_rows(const Kv4Args a) {
  const int which = static_cast<int>(blockIdx.y);
  const int64_t i0 = static_cast<int64_t>(blockIdx.x) * (kThreads * kWords) + threadIdx.x;
  uint4 raw[kWords];
#pragma unroll
  for (int j = 0; j < kWords; ++j) {
    const int64_t i = i0 + j * kThreads;   // units is a multiple of 16: whole groups of lanes
    raw[j] = i < a.units ? __ldg(static_cast<const uint4*>(a.src[which]) + i)
                         : make_uint4(0u, 0u, 0u, 0u);
  }
#pragma unroll
  for (int j = 0; j < kWords; ++j) {
    const int64_t i = i0 + j * kThreads;
    const uint32_t w[4] = {raw[j].x, raw[j].y, raw[j].z, raw[j].w};
    // |x| as bit patterns: ordered like the values, NaN above infinity; the
    // maximum of both halves of a word at once
    uint32_t m = w[0] & 0x7FFF7FFFu;
#pragma unroll
    for (int e = 1; e < 4; ++e) m = __vmaxu2(m, w[e] & 0x7FFF7FFFu);
    m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 2));
    const float s = kv4_scale(max(m >> 16, m & 0xFFFFu));
    const float inv = kv4_inverse(s);
    const uint64_t inv2 = pack_f32x2(inv, inv);
    uint32_t code = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) code |= (kv4_codes(w[e], inv2) & 0x000F000Fu) << (4 * e);
    int64_t at;
    if (i >= a.units || !cache_word(a, i, &at)) continue;
    static_cast<uint32_t*>(a.dst[which])[at] = code;
    if ((at & 3) == 0)
      static_cast<__nv_bfloat16*>(a.scales[which])[at >> 2] = __float2bfloat16_rn(s);   // exact
  }
}

__global__ void __launch_bounds__(kThreads) hstu_kv4_unpack_rows(const Kv4Args a) {
  const int which = static_cast<int>(blockIdx.y);
  const int64_t i0 = static_cast<int64_t>(blockIdx.x) * (kThreads * kWords) + threadIdx.x;
  uint32_t code[kWords], scale[kWords];
  bool live[kWords];
#pragma unroll
  for (int j = 0; j < kWords; ++j) {
    const int64_t i = i0 + j * kThreads;
    int64_t at;
    live[j] = i < a.units && cache_word(a, i, &at);
    if (live[j]) {
      code[j] = __ldg(static_cast<const uint32_t*>(a.src[which]) + at);
      scale[j] = __ldg(static_cast<const uint16_t*>(a.scales[which]) + (at >> 2));
    }
  }
#pragma unroll
  for (int j = 0; j < kWords; ++j) {
    if (!live[j]) continue;
    const uint32_t s2 = scale[j] | (scale[j] << 16);
    uint4 o;
    o.x = kv4_pair<0>(code[j], s2);
    o.y = kv4_pair<1>(code[j], s2);
    o.z = kv4_pair<2>(code[j], s2);
    o.w = kv4_pair<3>(code[j], s2);
    static_cast<uint4*>(a.dst[which])[i0 + j * kThreads] = o;
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
  // blocks of kThreads * kWords words in grid x
  const int64_t units = 16ll * T * H;
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
  constexpr int64_t kBlock = kThreads * kWords;
  const dim3 grid(static_cast<unsigned>((units + kBlock - 1) / kBlock), 2);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (pack)
    hstu_kv4_pack_rows<<<grid, kThreads, 0, s>>>(a);
  else
    hstu_kv4_unpack_rows<<<grid, kThreads, 0, s>>>(a);
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
