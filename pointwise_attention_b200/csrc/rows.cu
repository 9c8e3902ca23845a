// rows.cu -- row operators ahead of an HSTU layer's projection: the
// root-mean-square norm with the residual's addition (forward and backward)
// and the quantisation of rows to 8 bits (e4m3 with one scale per row).
//
//   h_te = round(x_te + res_te)                    (the residual stream's type)
//   r_t  = 1 / sqrt(mean_e h_te^2 + eps)
//   v_te = h_te r_t w_e
//   y    = round(v)   or   q8 = e4m3(v / s_t),  s_t = max(max_e |v_te|, 2^-100) / 448
//
//   g = w dy;  dx = dres + r (g - h r^2 mean_e(g h));  dw_e = sum_t dy_te h_te r_t
//
// Every operator is one pass over its rows: a row lives in the registers of
// the TPR threads that own it (NV vectors of VEC elements each), so that each
// input is read once and each output written once; what bounds them is HBM.
// Sums, statistics and products are fp32.  h is rounded to the stream's type
// before the norm because that is the value which the next layer and the
// backward read; y and q8 take v unrounded.
//
// Measured on a B200 (copies reach 6.56 TB/s): 131071 x 512 bf16 with a residual
// to h, 8 bits, scales and rstd, 471 MB: 78 us (6.0 TB/s; 90 us with the next
// row's loads in registers, 128 us with one-element arithmetic, whose 470
// instructions a row were what bounded it); backward of 32768 x 512 bf16 with
// d_residual, 134 MB: 27 us with the kernel of the weight's sums (5.0 TB/s; 31 us
// with three blocks an SM, whose 80 registers a thread spill; 45 us without the
// ring).  2^25 elements in rows of other lengths, before and after those lengths
// had shapes of their own, in us: bf16 forward 64 columns 115 -> 49, 333 125 ->
// 88, 8000 68 -> 50, 8001 176 -> 80; bf16 backward 64 columns 137 -> 50, 4096
// 75 -> 52, 8001 173 -> 92; fp32 backward 512 columns 98 -> 68, 8192 100 -> 76.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <nvtx3/nvToolsExt.h>

#include <atomic>
#include <cmath>
#include <cstdint>

#include "hstu.h"
#include "internal.h"
#include "ops.cuh"
#include "tile_math.cuh"

namespace hstu {
namespace {

constexpr int kMaxE = 16384;
constexpr int kMaxT = 0x7FFF0000;   // a row index plus the grid's stride stays in 32 bits
constexpr float kE4M3Max = 448.0f;
constexpr float kAmaxFloor = 7.8886090522101181e-31f;   // 2^-100: keeps 1 / scale finite

struct RowsArgs {
  const void* x;
  const void* res;       // or null
  const float* weight;   // [E] or null (ones)
  void* h;               // or null
  void* y;               // or null
  uint8_t* q8;           // or null (with scale)
  float* scale;
  float* rstd;           // or null
  int T, E;
  float eps;
};

struct RowsBwdArgs {
  const void* dy;
  const void* h;
  const float* weight;   // [E] or null (ones)
  const float* rstd;
  const void* dres;      // or null
  void* dx;
  float* partial;        // [gridDim.x][E], or null: no weight gradient
  int T, E;
};

template <typename T> struct Elem;
template <> struct Elem<float> {
  static __device__ __forceinline__ float get(float v) { return v; }
  static __device__ __forceinline__ float put(float v) { return v; }
};
template <> struct Elem<__nv_bfloat16> {
  static __device__ __forceinline__ float get(__nv_bfloat16 v) { return __bfloat162float(v); }
  static __device__ __forceinline__ __nv_bfloat16 put(float v) { return __float2bfloat16_rn(v); }
};

template <typename T, int VEC>
struct alignas(sizeof(T) * VEC) Pack {
  T v[VEC];
};

// The vectors of one row that this thread owns: vector i sits at column
// (i TPR + lane) VEC; columns at or past E read as zeros.
template <typename T, int VEC, int TPR, int NV>
__device__ __forceinline__ void load_row(const T* row, int lane, int E, Pack<T, VEC> (&p)[NV]) {
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * TPR + lane) * VEC;
    if (c < E) {
      p[i] = *reinterpret_cast<const Pack<T, VEC>*>(row + c);
    } else {
#pragma unroll
      for (int e = 0; e < VEC; ++e) p[i].v[e] = Elem<T>::put(0.f);
    }
  }
}

template <int VEC, int TPR, int NV>
__device__ __forceinline__ void load_weight(const float* w, int lane, int E, float (&r)[NV * VEC]) {
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * TPR + lane) * VEC;
#pragma unroll
    for (int e = 0; e < VEC; ++e) r[i * VEC + e] = 1.f;
    if (w && c < E) {
      if (VEC >= 4) {
#pragma unroll
        for (int e = 0; e < VEC; e += 4) {
          const float4 f = __ldg(reinterpret_cast<const float4*>(w + c + e));
          r[i * VEC + e] = f.x;
          r[i * VEC + e + 1] = f.y;
          r[i * VEC + e + 2] = f.z;
          r[i * VEC + e + 3] = f.w;
        }
      } else if (VEC == 2) {
        const float2 f = __ldg(reinterpret_cast<const float2*>(w + c));
        r[i * VEC] = f.x;
        r[i * VEC + VEC - 1] = f.y;
      } else {
        r[i * VEC] = __ldg(w + c);
      }
    }
  }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sum (or, for bit patterns of non-negative floats, maximum) over the TPR
// threads of a row.  TPR > 32: the block is the row.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* red) {
#pragma unroll
  for (int o = TPR < 32 ? TPR / 2 : 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (TPR > 32) {
    __syncthreads();   // red may still be read by the row before
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = red[0];
#pragma unroll
    for (int i = 1; i < TPR / 32; ++i) v += red[i];
  }
  return v;
}

template <int TPR>
__device__ __forceinline__ uint32_t row_umax(uint32_t v, uint32_t* red) {
  if (TPR < 32) {
#pragma unroll
    for (int o = TPR / 2; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, o));
  } else {
    v = __reduce_max_sync(0xffffffffu, v);
  }
  if (TPR > 32) {
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = red[0];
#pragma unroll
    for (int i = 1; i < TPR / 32; ++i) v = max(v, red[i]);
  }
  return v;
}

template <int TPR>
constexpr int block_threads() { return TPR <= 32 ? 256 : TPR; }

// Blocks of an SM that a kernel of N elements a thread is compiled for: up to 24
// warps, backward 16 where 24 would spill (32768 x 512 bf16: 27 against 31 us).
template <int TPR, int N>
constexpr int fwd_resident() { return N <= 16 ? 768 / block_threads<TPR>() : 1; }
template <int TPR, int N>
constexpr int bwd_resident() {
  constexpr int blocks = (N <= 8 ? 768 : N <= 16 ? 512 : 256) / block_threads<TPR>();
  return blocks > 0 ? blocks : 1;
}

// The arithmetic runs on pairs of neighbouring owned elements (fp32 pairs: one
// instruction for two), which halves the issue slots that bound these kernels
// beside HBM.
template <typename T, int VEC, int NV>
__device__ __forceinline__ uint64_t get_pair(const Pack<T, VEC> (&p)[NV], int i) {
  const int a = 2 * i, b = 2 * i + 1;
  return pack_f32x2(Elem<T>::get(p[a / VEC].v[a % VEC]), Elem<T>::get(p[b / VEC].v[b % VEC]));
}

template <typename T, int VEC, int NV>
__device__ __forceinline__ void put_pair(Pack<T, VEC> (&p)[NV], int i, uint64_t v) {
  const int a = 2 * i, b = 2 * i + 1;
  const float2 f = unpack_f32x2(v);
  if constexpr (sizeof(T) == 2 && VEC % 2 == 0) {
    *reinterpret_cast<uint32_t*>(&p[a / VEC].v[a % VEC]) = pack_bf16x2(f.x, f.y);
  } else {
    p[a / VEC].v[a % VEC] = Elem<T>::put(f.x);
    p[b / VEC].v[b % VEC] = Elem<T>::put(f.y);
  }
}

// Larger magnitude; a NaN on either side gives a NaN.
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(fabsf(b)));
  return d;
}

// Rows on their way from HBM: where they are taken in 16-byte vectors, a
// thread copies its part of the rows that it will come to asynchronously to
// shared memory, kDepth - 1 rows ahead: as many as BLOCKS blocks of an SM have
// room for.  Every thread copies what it reads itself, so its own wait for its
// copies is all that stands between the two.
template <typename T, int VEC, int TPR, int NV, int TENSORS, int BLOCKS>
struct Ring {
  static constexpr int kRows = block_threads<TPR>() / TPR;
  static constexpr int kStage = kRows * TENSORS * NV * TPR * 16;
  static constexpr int kRoom = 227 * 1024 / BLOCKS - 1536;   // beside a block's own kilobyte
  static constexpr int kDepth = NV <= 4 && 3 * kStage <= kRoom ? 3 : 2;
  // (forward: one row ahead is what its registers hold without the ring, and a
  // block per row is no faster with a ring of two: 2048 fp32 98 against 93 us)
  static constexpr bool on =
      sizeof(T) * VEC == 16 && kDepth * kStage <= kRoom && (TPR <= 32 || TENSORS == 3 || kDepth == 3);
  static constexpr int kBytes = on ? kDepth * kStage : 0;
  uint4* mine;   // of this thread: [stage][tensor][vector], TPR vectors apart
  int lane, stage;

  __device__ __forceinline__ Ring(void* smem, int sub, int lane_)
      : mine(static_cast<uint4*>(smem) + (sub * kDepth * TENSORS * NV) * TPR + lane_),
        lane(lane_), stage(0) {}
  __device__ __forceinline__ uint4* slot(int st, int tensor, int i) const {
    return mine + ((st * TENSORS + tensor) * NV + i) * TPR;
  }
  __device__ __forceinline__ void copy(int st, int tensor, const T* row, int E) const {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * TPR + lane) * VEC;
      if (c < E)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(static_cast<uint32_t>(
                         __cvta_generic_to_shared(slot(st, tensor, i)))),
                     "l"(row + c)
                     : "memory");
    }
  }
  __device__ __forceinline__ static void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
  __device__ __forceinline__ static void wait() {   // all but the newest kDepth - 2 groups
    asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 2) : "memory");
  }
  __device__ __forceinline__ void read(int tensor, Pack<T, VEC> (&p)[NV], int E) const {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if ((i * TPR + lane) * VEC < E) {
        *reinterpret_cast<uint4*>(&p[i]) = *slot(stage, tensor, i);
      } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e) p[i].v[e] = Elem<T>::put(0.f);
      }
    }
  }
};

// NORM: the norm; otherwise the rows as they are (quantisation alone).
template <typename T, int VEC, int TPR, int NV, bool NORM>
__global__ void __launch_bounds__(block_threads<TPR>(), fwd_resident<TPR, NV * VEC>())
    hstu_rows_fwd(const RowsArgs a) {
  constexpr int kRows = block_threads<TPR>() / TPR;   // rows of a block at a time
  constexpr int N = NV * VEC, P = N / 2;
  __shared__ float red[TPR > 32 ? TPR / 32 : 1];
  const int lane = static_cast<int>(threadIdx.x) % TPR;
  const int sub = static_cast<int>(threadIdx.x) / TPR;
  const T* x = static_cast<const T*>(a.x);
  const T* res = static_cast<const T*>(a.res);
  uint64_t w[P];
  if (NORM) {
    float f[N];
    load_weight<VEC, TPR, NV>(a.weight, lane, a.E, f);
#pragma unroll
    for (int i = 0; i < P; ++i) w[i] = pack_f32x2(f[2 * i], f[2 * i + 1]);
  }
  // The loop is uniform over a warp, and over the block where the block is the
  // row; rows past T of a warp with several read as zeros and are not written.
  // Without the ring the next row's loads are issued before this row's sums
  // are waited for.
  const int stride = static_cast<int>(gridDim.x) * kRows;
  int t = static_cast<int>(blockIdx.x) * kRows + sub;
  Pack<T, VEC> p[NV], q[NV];
  auto load = [&](int row) {
    const int E = row < a.T ? a.E : 0;
    load_row<T, VEC, TPR, NV>(x + static_cast<size_t>(row) * a.E, lane, E, p);
    if (NORM && res) load_row<T, VEC, TPR, NV>(res + static_cast<size_t>(row) * a.E, lane, E, q);
  };
  using R = Ring<T, VEC, TPR, NV, 2, fwd_resident<TPR, N>()>;
  extern __shared__ __align__(16) uint8_t s_dyn[];
  R ring(s_dyn, sub, lane);
  // rows past T are not copied; their group is empty (rows ahead may pass 31 bits)
  auto send = [&](uint32_t row, int st) {
    if (row < static_cast<uint32_t>(a.T)) {
      ring.copy(st, 0, x + static_cast<size_t>(row) * a.E, a.E);
      if (NORM && res) ring.copy(st, 1, res + static_cast<size_t>(row) * a.E, a.E);
    }
    R::commit();
  };
  if constexpr (R::on) {
#pragma unroll
    for (int i = 0; i < R::kDepth - 1; ++i) send(static_cast<uint32_t>(t) + i * stride, i);
  } else {
    if (TPR < 32 || t < a.T) load(t);
  }
  // the first row of the warp
  int tw = TPR < 32 ? t - sub % (TPR < 32 ? 32 / TPR : 1) : t;
  for (; tw < a.T; t += stride, tw += stride) {
    const bool live = TPR >= 32 || t < a.T;
    const int E = live ? a.E : 0;
    const size_t at = static_cast<size_t>(t) * a.E;
    if constexpr (R::on) {
      R::wait();
      ring.read(0, p, E);
      if (NORM && res) ring.read(1, q, E);
      // the stage of the row before is free
      send(static_cast<uint32_t>(t) + (R::kDepth - 1) * stride, ring.stage == 0 ? R::kDepth - 1 : ring.stage - 1);
      ring.stage = ring.stage == R::kDepth - 1 ? 0 : ring.stage + 1;
    }
    if (NORM && res) {
#pragma unroll
      for (int i = 0; i < P; ++i)
        put_pair<T, VEC, NV>(p, i, fadd2(get_pair<T, VEC, NV>(p, i), get_pair<T, VEC, NV>(q, i)));
      if (a.h) {
        T* h = static_cast<T*>(a.h) + at;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int c = (i * TPR + lane) * VEC;
          if (c < E) *reinterpret_cast<Pack<T, VEC>*>(h + c) = p[i];
        }
      }
    }
    uint64_t v[P];
#pragma unroll
    for (int i = 0; i < P; ++i) v[i] = get_pair<T, VEC, NV>(p, i);
    if (!R::on && tw < a.T - stride) load(t + stride);
    if (NORM) {
      uint64_t ss2 = 0ull;
#pragma unroll
      for (int i = 0; i < P; ++i) ss2 = ffma2(v[i], v[i], ss2);
      const float2 s2 = unpack_f32x2(ss2);
      const float ss = row_sum<TPR>(s2.x + s2.y, red);
      const float r = 1.0f / sqrtf(ss / static_cast<float>(a.E) + a.eps);
      if (a.rstd && lane == 0 && live) a.rstd[t] = r;
      const uint64_t r2 = pack_f32x2(r, r);
#pragma unroll
      for (int i = 0; i < P; ++i) v[i] = fmul2(fmul2(v[i], r2), w[i]);
      if (a.y) {
        T* y = static_cast<T*>(a.y) + at;
        Pack<T, VEC> o[NV];
#pragma unroll
        for (int i = 0; i < P; ++i) put_pair<T, VEC, NV>(o, i, v[i]);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int c = (i * TPR + lane) * VEC;
          if (c < E) *reinterpret_cast<Pack<T, VEC>*>(y + c) = o[i];
        }
      }
    }
    if (!NORM || a.q8) {
      // The threads' maxima meet as bit patterns: those of |v| are ordered
      // like the values, with NaN above infinity, so that a NaN reaches the
      // scale.
      float m = 0.f;
#pragma unroll
      for (int i = 0; i < P; ++i) {
        const float2 f = unpack_f32x2(v[i]);
        m = max_nan(max_nan(m, f.x), f.y);
      }
      const float top =
          __uint_as_float(row_umax<TPR>(__float_as_uint(m), reinterpret_cast<uint32_t*>(red)));
      const float s = (top < kAmaxFloor ? kAmaxFloor : top) / kE4M3Max;
      const float inv = 1.0f / s;
      if (lane == 0 && live) a.scale[t] = s;
      uint8_t* q8 = a.q8 + at;
      const uint64_t inv2 = pack_f32x2(inv, inv);
      Pack<uint8_t, VEC> o[NV];
#pragma unroll
      for (int i = 0; i < P; ++i) {
        const __nv_fp8x2_storage_t c =
            __nv_cvt_float2_to_fp8x2(unpack_f32x2(fmul2(v[i], inv2)), __NV_SATFINITE, __NV_E4M3);
        if constexpr (VEC % 2 == 0) {
          *reinterpret_cast<__nv_fp8x2_storage_t*>(&o[2 * i / VEC].v[2 * i % VEC]) = c;
        } else {
          o[2 * i].v[0] = static_cast<uint8_t>(c & 0xFFu);
          o[2 * i + 1].v[0] = static_cast<uint8_t>(c >> 8);
        }
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * TPR + lane) * VEC;
        if (c < E) *reinterpret_cast<Pack<uint8_t, VEC>*>(q8 + c) = o[i];
      }
    }
  }
}

template <typename T, int VEC, int TPR, int NV>
__global__ void __launch_bounds__(block_threads<TPR>(), bwd_resident<TPR, NV * VEC>())
    hstu_rows_bwd(const RowsBwdArgs a) {
  constexpr int kRows = block_threads<TPR>() / TPR;
  constexpr int N = NV * VEC, P = N / 2;
  __shared__ float red[TPR > 32 ? TPR / 32 : 1];
  // the rows' ring and, after the rows, their weight sums [kRows][TPR N]
  extern __shared__ __align__(16) uint8_t s_dyn[];
  using R = Ring<T, VEC, TPR, NV, 3, bwd_resident<TPR, N>()>;
  const int lane = static_cast<int>(threadIdx.x) % TPR;
  const int sub = static_cast<int>(threadIdx.x) / TPR;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  uint64_t w[P], dw2[P];
  {
    float f[N];
    load_weight<VEC, TPR, NV>(a.weight, lane, a.E, f);
#pragma unroll
    for (int i = 0; i < P; ++i) {
      w[i] = pack_f32x2(f[2 * i], f[2 * i + 1]);
      dw2[i] = 0ull;
    }
  }
  const int stride = static_cast<int>(gridDim.x) * kRows;
  int t = static_cast<int>(blockIdx.x) * kRows + sub;
  Pack<T, VEC> pd[NV], ph[NV], pr[NV];
  const T* dy = static_cast<const T*>(a.dy);
  const T* h = static_cast<const T*>(a.h);
  const T* dres = static_cast<const T*>(a.dres);
  R ring(s_dyn, sub, lane);
  // rows past T are not copied; their group is empty (rows ahead may pass 31 bits)
  auto send = [&](uint32_t row, int st) {
    if (row < static_cast<uint32_t>(a.T)) {
      const size_t at = static_cast<size_t>(row) * a.E;
      ring.copy(st, 0, dy + at, a.E);
      ring.copy(st, 1, h + at, a.E);
      if (dres) ring.copy(st, 2, dres + at, a.E);
    }
    R::commit();
  };
  float rn = t < a.T ? __ldg(a.rstd + t) : 0.f;
  if constexpr (R::on) {
#pragma unroll
    for (int i = 0; i < R::kDepth - 1; ++i) send(static_cast<uint32_t>(t) + i * stride, i);
  }
  // the first row of the warp
  int tw = TPR < 32 ? t - sub % (TPR < 32 ? 32 / TPR : 1) : t;
  for (; tw < a.T; t += stride, tw += stride) {
    const bool live = TPR >= 32 || t < a.T;
    const int E = live ? a.E : 0;
    const size_t at = static_cast<size_t>(t) * a.E;
    if constexpr (R::on) {
      R::wait();
      ring.read(0, pd, E);
      ring.read(1, ph, E);
      if (dres) ring.read(2, pr, E);
      // the stage of the row before is free
      send(static_cast<uint32_t>(t) + (R::kDepth - 1) * stride, ring.stage == 0 ? R::kDepth - 1 : ring.stage - 1);
      ring.stage = ring.stage == R::kDepth - 1 ? 0 : ring.stage + 1;
    } else {
      load_row<T, VEC, TPR, NV>(dy + at, lane, E, pd);
      load_row<T, VEC, TPR, NV>(h + at, lane, E, ph);
      if (dres) load_row<T, VEC, TPR, NV>(dres + at, lane, E, pr);
    }
    const float r = rn;
    rn = t < a.T - stride ? __ldg(a.rstd + t + stride) : 0.f;
    const uint64_t r2 = pack_f32x2(r, r);
    // g = w dy and z = h r: dx = r g - z (r mean(g z)), dw += dy z; g and z are
    // made twice, which leaves registers for more rows on an SM
    uint64_t dot2 = 0ull;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const uint64_t d = get_pair<T, VEC, NV>(pd, i);
      const uint64_t z = fmul2(get_pair<T, VEC, NV>(ph, i), r2);
      dot2 = ffma2(fmul2(d, w[i]), z, dot2);
      dw2[i] = ffma2(d, z, dw2[i]);
    }
    const float2 d2 = unpack_f32x2(dot2);
    const float dot = row_sum<TPR>(d2.x + d2.y, red);
    const float k = -r * (dot / static_cast<float>(a.E));
    const uint64_t k2 = pack_f32x2(k, k);
    T* dx = static_cast<T*>(a.dx) + at;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const uint64_t g = fmul2(get_pair<T, VEC, NV>(pd, i), w[i]);
      const uint64_t z = fmul2(get_pair<T, VEC, NV>(ph, i), r2);
      uint64_t x = ffma2(z, k2, fmul2(g, r2));
      if (dres) x = fadd2(x, get_pair<T, VEC, NV>(pr, i));
      put_pair<T, VEC, NV>(pd, i, x);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * TPR + lane) * VEC;
      if (c < E) *reinterpret_cast<Pack<T, VEC>*>(dx + c) = pd[i];
    }
  }
  float dw[N];
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const float2 f = unpack_f32x2(dw2[i]);
    dw[2 * i] = f.x;
    dw[2 * i + 1] = f.y;
  }
  if (!a.partial) return;
  float* part = a.partial + static_cast<size_t>(blockIdx.x) * a.E;
  if (TPR <= 32) {
    // the sums of the block's rows, added in their order, over the ring's room
    float* sdw = reinterpret_cast<float*>(s_dyn);
    if constexpr (R::on) asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) sdw[sub * TPR * N + (i / VEC * TPR + lane) * VEC + i % VEC] = dw[i];
    __syncthreads();
    for (int c = static_cast<int>(threadIdx.x); c < a.E; c += block_threads<TPR>()) {
      float s = 0.f;
#pragma unroll
      for (int g = 0; g < kRows; ++g) s += sdw[g * TPR * N + c];
      part[c] = s;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = (i / VEC * TPR + lane) * VEC + i % VEC;
      if (c < a.E) part[c] = dw[i];
    }
  }
}

// dw[c] = the blocks' partial sums added in a fixed order: 8 columns by 128
// strides of blocks per CTA, four loads in flight a thread.
__global__ void __launch_bounds__(1024) hstu_rows_dw(const float* partial, int blocks, int E,
                                                     float* dw) {
  __shared__ float red[8][129];
  const int cx = static_cast<int>(threadIdx.x & 7), gy = static_cast<int>(threadIdx.x >> 3);
  const int c = static_cast<int>(blockIdx.x) * 8 + cx;
  asm volatile("griddepcontrol.wait;" ::: "memory");   // launched while the rows' kernel runs
  float s = 0.f;
  if (c < E)
    for (int g = gy; g < blocks; g += 4 * 128) {
      float v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        v[i] = g + 128 * i < blocks ? partial[static_cast<size_t>(g + 128 * i) * E + c] : 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) s += v[i];
    }
  red[cx][gy] = s;
  __syncthreads();
  const int col = static_cast<int>(threadIdx.x >> 5), lane = static_cast<int>(threadIdx.x & 31);
  if (col >= 8) return;
  s = (red[col][lane] + red[col][lane + 32]) + (red[col][lane + 64] + red[col][lane + 96]);
  s = warp_sum(s);
  if (lane == 0 && static_cast<int>(blockIdx.x) * 8 + col < E) dw[blockIdx.x * 8 + col] = s;
}

bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// One row shape of the kernels: elements per vector, threads per row, vectors
// per thread.  The smallest that holds E columns is taken: a part of a warp per
// row for short rows, a warp up to 1024 columns (no barrier), 128 threads up to
// 4096, 512 up to 16384.  Rows whose columns or addresses do not divide into
// 16-byte vectors take one element at a time; bf16 in pairs where the columns
// are even and the addresses allow it, in the backward (2^25 elements, 334
// columns 73 -> 64 us, 1002 68 -> 58, 8002 92 -> 75) and in short rows (forward
// 50 columns 73 -> 60 us, 202 80 -> 71; 334 88 -> 98, so not there).
template <int VEC_, int TPR_, int NV_>
struct Shape {
  static constexpr int VEC = VEC_, TPR = TPR_, NV = NV_;
};

template <typename T, bool BWD, typename F>
cudaError_t pick_shape(bool vec, bool pairs, int E, F&& f) {
  if constexpr (sizeof(T) == 2) {
    if (vec) {
      if (E <= 32) return f(Shape<8, 4, 1>{});
      if (E <= 64) return f(Shape<8, 8, 1>{});
      if (E <= 128) return f(Shape<8, 8, 2>{});
      if (E <= 256) return f(Shape<8, 16, 2>{});
      if (E <= 512) return f(Shape<8, 32, 2>{});
      if (E <= 1024) return f(Shape<8, 32, 4>{});
      if (E <= 2048) return f(Shape<8, 128, 2>{});
      if (E <= 4096) return f(Shape<8, 128, 4>{});
      if (E <= 8192) return f(Shape<8, 512, 2>{});
      return f(Shape<8, 512, 4>{});
    }
    if (pairs && E <= 64) return f(Shape<2, 8, 4>{});
    if (pairs && E <= 128) return f(Shape<2, 16, 4>{});
    if (pairs && E <= 256) return f(Shape<2, 32, 4>{});
    if constexpr (BWD) {
      if (pairs) {
        if (E <= 512) return f(Shape<2, 32, 8>{});
        if (E <= 1024) return f(Shape<2, 32, 16>{});
        if (E <= 2048) return f(Shape<2, 128, 8>{});
        if (E <= 4096) return f(Shape<2, 128, 16>{});
        if (E <= 8192) return f(Shape<2, 512, 8>{});
        return f(Shape<2, 512, 16>{});
      }
    }
  } else {
    if (vec) {
      if (E <= 16) return f(Shape<4, 4, 1>{});
      if (E <= 32) return f(Shape<4, 8, 1>{});
      if (E <= 64) return f(Shape<4, 16, 1>{});
      if (E <= 128) return f(Shape<4, 16, 2>{});
      if (E <= 256) return f(Shape<4, 32, 2>{});
      if (E <= 512) return f(Shape<4, 32, 4>{});
      if (E <= 1024) return f(Shape<4, 32, 8>{});
      if (E <= 2048) return f(Shape<4, 128, 4>{});
      if (E <= 4096) return f(Shape<4, 128, 8>{});
      if (E <= 8192) return f(Shape<4, 512, 4>{});
      return f(Shape<4, 512, 8>{});
    }
  }
  if (E <= 64) return f(Shape<1, 8, 8>{});
  if (E <= 128) return f(Shape<1, 16, 8>{});
  if (E <= 256) return f(Shape<1, 32, 8>{});
  if (E <= 512) return f(Shape<1, 32, 16>{});
  if (E <= 1024) return f(Shape<1, 32, 32>{});
  if (E <= 2048) return f(Shape<1, 128, 16>{});
  if (E <= 4096) return f(Shape<1, 128, 32>{});
  if (E <= 8192) return f(Shape<1, 512, 16>{});
  return f(Shape<1, 512, 32>{});
}

// Opts a kernel in to its shared memory, once per device and kernel (S, T and
// KIND tell the kernels apart).
template <typename S, typename T, int KIND, typename K>
cudaError_t opt_in(K kernel, int smem) {
  if (smem <= 47 * 1024) return cudaSuccess;   // of 48, a little is static
  static std::atomic<bool> done[64];
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev < 0 || dev >= 64 || !done[dev].load(std::memory_order_acquire)) {
    err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (err != cudaSuccess) return err;
    if (dev >= 0 && dev < 64) done[dev].store(true, std::memory_order_release);
  }
  return cudaSuccess;
}

template <typename T, bool NORM>
cudaError_t launch_rows_fwd(const RowsArgs& a, cudaStream_t stream) {
  constexpr size_t V = 16;
  const bool vec = a.E % (V / sizeof(T)) == 0 && aligned(a.x, V) && aligned(a.res, V) &&
                   aligned(a.h, V) && aligned(a.y, V) && aligned(a.q8, V / sizeof(T)) &&
                   aligned(a.weight, V);
  const bool pairs = a.E % 2 == 0 && aligned(a.x, 4) && aligned(a.res, 4) && aligned(a.h, 4) &&
                     aligned(a.y, 4) && aligned(a.q8, 2) && aligned(a.weight, 8);
  return pick_shape<T, false>(vec, pairs, a.E, [&](auto s) {
    using S = decltype(s);
    constexpr int kRows = block_threads<S::TPR>() / S::TPR;
    // eight blocks per SM at most: each row's loads then run ahead of it
    const int64_t need = (static_cast<int64_t>(a.T) + kRows - 1) / kRows;
    // (and 2^16 rows: kMaxT)
    const int most = 8 * 148 * kRows < 0x10000 ? 8 * 148 : 0xFFFF / kRows;
    const int blocks = static_cast<int>(need < most ? need : most);
    constexpr int smem =
        Ring<T, S::VEC, S::TPR, S::NV, 2, fwd_resident<S::TPR, S::NV * S::VEC>()>::kBytes;
    auto kernel = hstu_rows_fwd<T, S::VEC, S::TPR, S::NV, NORM>;
    const cudaError_t err = opt_in<S, T, NORM ? 1 : 2>(kernel, smem);
    if (err != cudaSuccess) return err;
    kernel<<<blocks, block_threads<S::TPR>(), smem, stream>>>(a);
    return cudaGetLastError();
  });
}

// Blocks of the backward: as many as run at a time, so that each starts and
// adds its weight's sums once.  A function of the sizes alone (not of the device), so that
// the order of the sums is too.
int bwd_blocks(int T, int E) {
  const int rows = E <= 1024 ? 8 : 1;
  const int most =
      (E <= 64 ? 3 : E <= 512 ? 2 : E <= 1024 ? 1 : E <= 2048 ? 4 : E <= 4096 ? 2 : 1) * 148;
  const int64_t need = (static_cast<int64_t>(T) + rows - 1) / rows;
  return static_cast<int>(need < most ? need : most);
}

template <typename T>
cudaError_t launch_rows_bwd(const RowsBwdArgs& a, float* dw, cudaStream_t stream) {
  constexpr size_t V = 16;
  const bool vec = a.E % (V / sizeof(T)) == 0 && aligned(a.dy, V) && aligned(a.h, V) &&
                   aligned(a.dres, V) && aligned(a.dx, V) && aligned(a.weight, V);
  const bool pairs = a.E % 2 == 0 && aligned(a.dy, 4) && aligned(a.h, 4) && aligned(a.dres, 4) &&
                     aligned(a.dx, 4) && aligned(a.weight, 8);
  const int blocks = bwd_blocks(a.T, a.E);
  const cudaError_t err = pick_shape<T, true>(vec, pairs, a.E, [&](auto s) {
    using S = decltype(s);
    using R = Ring<T, S::VEC, S::TPR, S::NV, 3, bwd_resident<S::TPR, S::NV * S::VEC>()>;
    constexpr int sums = S::TPR <= 32 ? 256 * S::NV * S::VEC * 4 : 0;
    constexpr int smem = R::kBytes > sums ? R::kBytes : sums;
    auto kernel = hstu_rows_bwd<T, S::VEC, S::TPR, S::NV>;
    const cudaError_t e = opt_in<S, T, 0>(kernel, smem);
    if (e != cudaSuccess) return e;
    kernel<<<blocks, block_threads<S::TPR>(), smem, stream>>>(a);
    return cudaGetLastError();
  });
  if (err != cudaSuccess || !dw) return err;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((a.E + 7) / 8));
  cfg.blockDim = dim3(1024);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, hstu_rows_dw, static_cast<const float*>(a.partial), blocks, a.E, dw);
}

size_t elem_bytes(hstu_dtype_t d) { return d == HSTU_BF16 ? 2 : 4; }

hstu_status_t check_rows(hstu_dtype_t dtype, int32_t T, int32_t E) {
  if ((dtype != HSTU_F32 && dtype != HSTU_BF16) || T < 0 || E < 1) return HSTU_ERR_INVALID_ARG;
  return HSTU_OK;
}

struct RowsRange {
  explicit RowsRange(const char* name) { nvtxRangePushA(name); }
  ~RowsRange() { nvtxRangePop(); }
};

}  // namespace
}  // namespace hstu

using namespace hstu;

extern "C" {

HSTU_API hstu_status_t hstu_rmsnorm_fwd(hstu_dtype_t dtype, int32_t T, int32_t E, const void* x,
                                        const void* residual, const float* weight, float eps,
                                        void* h, void* y, uint8_t* q8, float* q8_scale,
                                        float* rstd, void* stream) {
  RowsRange range("hstu_rmsnorm_fwd");
  const hstu_status_t st = check_rows(dtype, T, E);
  if (st != HSTU_OK) return st;
  if (!(eps > 0.0f) || !std::isfinite(eps)) return HSTU_ERR_INVALID_ARG;
  if ((q8 == nullptr) != (q8_scale == nullptr)) return HSTU_ERR_INVALID_ARG;
  if (h && !residual) return HSTU_ERR_INVALID_ARG;
  if (T > 0) {
    if (!x || (!y && !q8)) return HSTU_ERR_INVALID_ARG;
    const size_t b = elem_bytes(dtype);
    if (!aligned(x, b) || !aligned(residual, b) || !aligned(h, b) || !aligned(y, b))
      return HSTU_ERR_INVALID_ARG;
  }
  if (!aligned(weight, 4) || !aligned(q8_scale, 4) || !aligned(rstd, 4))
    return HSTU_ERR_INVALID_ARG;
  if (E > kMaxE || T > kMaxT) return HSTU_ERR_UNSUPPORTED;
  if (T == 0) return HSTU_OK;
  const RowsArgs a{x, residual, weight, h, y, q8, q8_scale, rstd, T, E, eps};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t err = dtype == HSTU_BF16 ? launch_rows_fwd<__nv_bfloat16, true>(a, s)
                                             : launch_rows_fwd<float, true>(a, s);
  return err == cudaSuccess ? HSTU_OK : HSTU_ERR_CUDA;
}

HSTU_API hstu_status_t hstu_quant_rows(hstu_dtype_t dtype, int32_t T, int32_t E, const void* x,
                                       uint8_t* q8, float* q8_scale, void* stream) {
  RowsRange range("hstu_quant_rows");
  const hstu_status_t st = check_rows(dtype, T, E);
  if (st != HSTU_OK) return st;
  if (T > 0 && (!x || !q8 || !q8_scale || !aligned(x, elem_bytes(dtype)) || !aligned(q8_scale, 4)))
    return HSTU_ERR_INVALID_ARG;
  if (E > kMaxE || T > kMaxT) return HSTU_ERR_UNSUPPORTED;
  if (T == 0) return HSTU_OK;
  const RowsArgs a{x, nullptr, nullptr, nullptr, nullptr, q8, q8_scale, nullptr, T, E, 1.0f};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t err = dtype == HSTU_BF16 ? launch_rows_fwd<__nv_bfloat16, false>(a, s)
                                             : launch_rows_fwd<float, false>(a, s);
  return err == cudaSuccess ? HSTU_OK : HSTU_ERR_CUDA;
}

HSTU_API size_t hstu_rmsnorm_bwd_workspace_size(int32_t T, int32_t E) {
  if (T < 0 || T > kMaxT || E < 1 || E > kMaxE) return 0;
  // no less than smaller calls of any row length need
  size_t n = static_cast<size_t>(bwd_blocks(T, E)) * E * sizeof(float);
  for (int e = 64; e < E; e *= 2) {
    const size_t m = static_cast<size_t>(bwd_blocks(T, e)) * e * sizeof(float);
    if (m > n) n = m;
  }
  return n < 256 ? 256 : (n + 255) / 256 * 256;
}

HSTU_API hstu_status_t hstu_rmsnorm_bwd(hstu_dtype_t dtype, int32_t T, int32_t E, const void* dy,
                                        const void* h, const float* rstd, const float* weight,
                                        const void* d_residual, void* dx, float* d_weight,
                                        void* workspace, size_t workspace_bytes, void* stream) {
  RowsRange range("hstu_rmsnorm_bwd");
  const hstu_status_t st = check_rows(dtype, T, E);
  if (st != HSTU_OK) return st;
  if (T > 0) {
    const size_t b = elem_bytes(dtype);
    if (!dy || !h || !rstd || !dx || !aligned(dy, b) || !aligned(h, b) || !aligned(dx, b) ||
        !aligned(d_residual, b))
      return HSTU_ERR_INVALID_ARG;
  }
  if (!aligned(rstd, 4) || !aligned(weight, 4) || !aligned(d_weight, 4)) return HSTU_ERR_INVALID_ARG;
  if (E > kMaxE || T > kMaxT) return HSTU_ERR_UNSUPPORTED;
  if (d_weight && (!workspace || !aligned(workspace, 256) ||
                   workspace_bytes < hstu_rmsnorm_bwd_workspace_size(T, E)))
    return HSTU_ERR_WORKSPACE;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (T == 0) {
    // no rows: the weight's gradient is an empty sum
    if (d_weight && cudaMemsetAsync(d_weight, 0, sizeof(float) * E, s) != cudaSuccess)
      return HSTU_ERR_CUDA;
    return HSTU_OK;
  }
  const RowsBwdArgs a{dy, h, weight, rstd, d_residual, dx,
                      d_weight ? static_cast<float*>(workspace) : nullptr, T, E};
  const cudaError_t err = dtype == HSTU_BF16 ? launch_rows_bwd<__nv_bfloat16>(a, d_weight, s)
                                             : launch_rows_bwd<float>(a, d_weight, s);
  return err == cudaSuccess ? HSTU_OK : HSTU_ERR_CUDA;
}

}  // extern "C"
