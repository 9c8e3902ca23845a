// cand4_few.cu -- candidate scoring against histories in a 4-bit cache, the
// form that splits every history over many warps.
//
// The operation is hstu_cand_fwd's with keys and values n s of the cache in
// place of bf16 ones: candidate c of user b attends to every history token
// j < n_b and to itself, and
//   O_c = (sum_j SiLU(q_c . k_j + bias_cj) v_j + SiLU(q_c . k_c + bias_cc) v_c) / N,
//   y_c = (gamma LayerNorm(O_c over all heads) + beta) SiLU(u_c).
// There is no softmax, so sums over parts of a history simply add.
//
// A CTA takes (user, `chunk` keys, 8 NT candidates, up to 8 heads): a warp per
// head, or several warps per head where there are fewer heads.  All heads of
// a cache row are neighbours, so the CTA reads whole contiguous rows, once for
// its candidates.  Per 16 keys a warp computes S^T = K Q^T and O^T += V^T P^T
// with m16n8k16 MMAs whose A operand is decoded in registers straight from
// the codes (the order of the dimensions in an MMA is free as long as both
// operands share it, so a lane takes whole 16-byte runs of codes):
//   K: lane (g, t) holds dims 32t.. of keys g and g + 8 (one scale each);
//   V: lane (g, t) holds dims 16g.. of keys 2t, 2t+1, 2t+8, 2t+9.
// The candidates are the MMA's 8 columns: with few of them the tensor core's
// work is small beside the cache's bytes, which bound the kernel.
// P is rounded to bf16 for the second product; scores, SiLU and sums are fp32.
//
// The slices' sums go to the workspace in fp32; cand4_finish adds them in
// slice order (the result does not depend on timing), adds the self term and
// applies the LayerNorm and the gate.
#include <cuda_bf16.h>

#include <algorithm>

#include "bounds.cuh"
#include "internal.h"
#include "kv4.cuh"
#include "tile_math.cuh"

namespace hstu {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxChunk = 512;

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// SiLU in fp32; exp overflows to infinity for very negative x, the quotient to 0
__device__ __forceinline__ float silu_f(float x) { return __fdividef(x, 1.0f + __expf(-x)); }

__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 8 x 8 transpose of 16-bit elements over the warp (row g: lanes 4g..4g+3).
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ void grid_dependents() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// One 16-key block of a head as it sits in the cache.
struct Block {
  uint4 k[2];          // keys g, g + 8: codes of dims 32t..32t+31
  uint2 v[4];          // keys 2t, 2t+1, 2t+8, 2t+9: codes of dims 16g..16g+15
  uint32_t ks[2];      // their scales
  uint32_t vs[4];
  float pos[2];        // position bias of keys g, g + 8
};

struct User {
  int c0, cb, s, nb, r0;
  bool ok;
};

// A user's ranges, checked against the sizes.
__device__ __forceinline__ User user_ranges(const Cand4Args& a, int b) {
  User x;
  x.c0 = __ldg(a.cand_offsets + b);
  x.cb = __ldg(a.cand_offsets + b + 1) - x.c0;
  x.s = __ldg(a.offsets + b);
  x.nb = __ldg(a.offsets + b + 1) - x.s;
  x.r0 = a.first_rows ? __ldg(a.first_rows + b) : x.s;
  x.ok = x.c0 >= 0 && x.cb >= 0 && x.cb <= a.C - x.c0 && x.cb <= a.max_cands && x.s >= 0 &&
         x.nb >= 0 && x.nb <= a.T - x.s && x.nb <= a.max_seq_len && x.r0 >= 0 &&
         x.nb <= a.R - x.r0 && !(a.rab_pos && x.nb >= a.L);
  return x;
}

template <int NT, bool POS, bool TIME>
__global__ void __launch_bounds__(kThreads, NT == 1 ? 2 : 1)
    hstu_cand4_few(const __grid_constant__ Cand4Args a, const Cand4Cut cut) {
  constexpr int NC = 8 * NT;
  __shared__ float s_rabt[TIME ? kWarps : 1][TIME ? kMaxBuckets : 1];
  __shared__ long long s_thr[TIME ? kThrLen : 1];
  __shared__ signed char s_first[TIME ? 64 : 1];
  __shared__ __align__(16) uint8_t s_bk[TIME ? kMaxChunk * NC : 16];   // [key][candidate] bucket
  grid_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  unsigned x = blockIdx.x;
  const int hg = static_cast<int>(x % static_cast<unsigned>(cut.hgroups));
  x /= static_cast<unsigned>(cut.hgroups);
  const int split = static_cast<int>(x % static_cast<unsigned>(cut.splits));
  x /= static_cast<unsigned>(cut.splits);
  const int cg = static_cast<int>(x % static_cast<unsigned>(cut.cgroups));
  const int b = static_cast<int>(x / static_cast<unsigned>(cut.cgroups));
  const User us = user_ranges(a, b);
  if (!us.ok) {
    if (threadIdx.x == 0 && a.status) atomicOr(a.status, kStatusBadOffsets);
    return;
  }
  const int first = split * cut.chunk;                  // this CTA's keys: first..last-1
  const int last = min(us.nb, first + cut.chunk);
  const int cands = min(NC, us.cb - NC * cg);
  if (cands <= 0 || first >= last) return;
  const int cand0 = us.c0 + NC * cg;

  if (TIME) {
    for (int i = threadIdx.x; i < kThrLen; i += kThreads) s_thr[i] = a.bt.thr[i];
    for (int i = threadIdx.x; i < 64; i += kThreads) s_first[i] = a.bt.first_k[i];
    for (int i = threadIdx.x; i < cut.heads * kMaxBuckets; i += kThreads) {
      const int hh = 8 * hg + i / kMaxBuckets, k = i % kMaxBuckets;
      s_rabt[i / kMaxBuckets][k] = (hh < a.H && k < a.nb) ? __ldg(a.rab_time + hh * a.nb + k) : 0.f;
    }
    __syncthreads();
    // every (key, candidate) bucket once for all heads
    for (int i = threadIdx.x; i < (last - first) * NC; i += kThreads) {
      const int c = i % NC, j = first + i / NC;
      int k = 0;
      if (c < cands)
        k = time_bucket(__ldg(a.cand_ts + checked(a.status, cand0 + c, a.C, BS_CAND4_ROW)) -
                            __ldg(a.timestamps + checked(a.status, us.s + j, a.T, BS_CAND4_TS)),
                        s_thr, s_first);
      s_bk[i] = static_cast<uint8_t>(k);
    }
    __syncthreads();
  }

  const int h = 8 * hg + warp % cut.heads, part = warp / cut.heads;
  if (h >= a.H || part >= cut.parts) return;
  const int step = 16 * cut.parts;
  int j0 = first + 16 * part;
  if (j0 >= last) return;

  // Q as the B operand: candidate g (of each group of 8), dims 32t..32t+31;
  // candidates past the user's last read as zeros
  uint32_t qb[NT][16];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const bool live = 8 * n + g < cands;
    const uint4* src = reinterpret_cast<const uint4*>(
        static_cast<const __nv_bfloat16*>(a.q) +
        (static_cast<size_t>(checked(a.status, cand0 + (live ? 8 * n + g : 0), a.C, BS_CAND4_ROW)) * a.H + h) * 128 +
        32 * t);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint4 w = live ? __ldg(src + i) : make_uint4(0u, 0u, 0u, 0u);
      qb[n][4 * i] = w.x;
      qb[n][4 * i + 1] = w.y;
      qb[n][4 * i + 2] = w.z;
      qb[n][4 * i + 3] = w.w;
    }
  }
  float o[NT][8][4];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int m = 0; m < 8; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[n][m][i] = 0.f;

  const float* rpos = POS ? a.rab_pos + static_cast<size_t>(h) * (2 * static_cast<size_t>(a.L) - 1) + (a.L - 1)
                          : nullptr;
  // keys past the CTA's last repeat it (their P is 0)
  auto load = [&](int j, Block& x) {
    auto at = [&](int key) {
      return static_cast<size_t>(checked(a.status, us.r0 + min(key, last - 1), a.R, BS_CAND4_KEY)) * a.H + h;
    };
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const size_t r = at(j + g + 8 * i);
      x.k[i] = __ldg(reinterpret_cast<const uint4*>(a.k_codes + r * 64) + t);
      x.ks[i] = __ldg(a.k_scales + r * 4 + t);
      if (POS) x.pos[i] = __ldg(rpos + (us.nb - min(j + g + 8 * i, last - 1)));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const size_t r = at(j + 2 * t + (i & 1) + 8 * (i >> 1));
      x.v[i] = __ldg(reinterpret_cast<const uint2*>(a.v_codes + r * 64) + g);
      x.vs[i] = __ldg(a.v_scales + r * 4 + (g >> 1));
    }
  };
  Block cur, nxt;
  load(j0, cur);
  for (; j0 < last; j0 += step) {
    if (j0 + step < last) load(j0 + step, nxt);
    // S^T = K Q^T
    float s[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) s[n][i] = 0.f;
    {
      const uint32_t s0 = cur.ks[0] | (cur.ks[0] << 16), s1 = cur.ks[1] | (cur.ks[1] << 16);
      const uint32_t m0 = kv4_m24(s0), m1 = kv4_m24(s1);
      const uint32_t w0[4] = {cur.k[0].x, cur.k[0].y, cur.k[0].z, cur.k[0].w};
      const uint32_t w1[4] = {cur.k[1].x, cur.k[1].y, cur.k[1].z, cur.k[1].w};
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const uint32_t a0 = kv4_pair_fma<0>(w0[w], s0, m0), a1 = kv4_pair_fma<0>(w1[w], s1, m1);
        const uint32_t a2 = kv4_pair_fma<1>(w0[w], s0, m0), a3 = kv4_pair_fma<1>(w1[w], s1, m1);
        const uint32_t b0 = kv4_pair_fma<2>(w0[w], s0, m0), b1 = kv4_pair_fma<2>(w1[w], s1, m1);
        const uint32_t b2 = kv4_pair_fma<3>(w0[w], s0, m0), b3 = kv4_pair_fma<3>(w1[w], s1, m1);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          mma_16816(s[n], a0, a1, a2, a3, qb[n][4 * w], qb[n][4 * w + 1]);
          mma_16816(s[n], b0, b1, b2, b3, qb[n][4 * w + 2], qb[n][4 * w + 3]);
        }
      }
    }
    // P: keys g, g + 8 by candidates 2t, 2t+1, transposed into the B operand
    uint32_t pb[NT][2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int j = j0 + g + 8 * i;
      const bool live = j < last;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float x0 = s[n][2 * i], x1 = s[n][2 * i + 1];
        if (POS) {
          x0 += cur.pos[i];
          x1 += cur.pos[i];
        }
        if (TIME && live) {
          const uint32_t k2 = *reinterpret_cast<const uint16_t*>(
              s_bk + (j - first) * NC + 8 * n + 2 * t);
          const float* rt = s_rabt[warp % cut.heads];
          x0 += rt[k2 & 0xFFu];
          x1 += rt[k2 >> 8];
        }
        const uint32_t p2 = live ? pack_bf16x2(silu_f(x0), silu_f(x1)) : 0u;
        pb[n][i] = transpose8(p2);
      }
    }
    // O^T += V^T P^T
    {
      // scales of the keys that share a register: (2t, 2t+1), (2t+8, 2t+9)
      const uint32_t sa = cur.vs[0] | (cur.vs[1] << 16), sb = cur.vs[2] | (cur.vs[3] << 16);
      const uint32_t ma = kv4_m24(sa), mb = kv4_m24(sb);
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const uint32_t va = w ? cur.v[0].y : cur.v[0].x, vb = w ? cur.v[1].y : cur.v[1].x;
        const uint32_t vc = w ? cur.v[2].y : cur.v[2].x, vd = w ? cur.v[3].y : cur.v[3].x;
        // even and odd dims of two keys, a key per half
        const uint32_t ea = __byte_perm(va, vb, 0x5410), oa = __byte_perm(va, vb, 0x7632);
        const uint32_t eb = __byte_perm(vc, vd, 0x5410), ob = __byte_perm(vc, vd, 0x7632);
#define HSTU_PV(I)                                                                       \
  {                                                                                      \
    const uint32_t a0 = kv4_pair_fma<I>(ea, sa, ma), a1 = kv4_pair_fma<I>(oa, sa, ma);   \
    const uint32_t a2 = kv4_pair_fma<I>(eb, sb, mb), a3 = kv4_pair_fma<I>(ob, sb, mb);   \
    _Pragma("unroll") for (int n = 0; n < NT; ++n)                                       \
        mma_16816(o[n][4 * w + I], a0, a1, a2, a3, pb[n][0], pb[n][1]);                  \
  }
        HSTU_PV(0)
        HSTU_PV(1)
        HSTU_PV(2)
        HSTU_PV(3)
#undef HSTU_PV
      }
    }
    cur = nxt;
  }
  // lane (g, t): dims 16g..16g+15 of candidates 2t, 2t+1
  const int slice = split * cut.parts + part;
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      if (8 * n + 2 * t + c >= cands) continue;
      float4* dst = reinterpret_cast<float4*>(
          a.part + (static_cast<size_t>(slice) * a.C + cand0 + 8 * n + 2 * t + c) * (a.H * 128) + h * 128 + 16 * g);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        dst[i] = make_float4(o[n][2 * i][c], o[n][2 * i][c + 2], o[n][2 * i + 1][c], o[n][2 * i + 1][c + 2]);
    }
}

// Sum over a block of 32 H threads, the same in every thread.
__device__ __forceinline__ float block_sum(float v, float* red, int warps) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = red[0];
  for (int i = 1; i < warps; ++i) v += red[i];
  return v;
}

// A block per candidate, a warp per head, four dimensions per thread.
template <bool POS, bool TIME>
__global__ void __launch_bounds__(512) hstu_cand4_finish(const __grid_constant__ Cand4Args a,
                                                         const Cand4Cut cut) {
  __shared__ float red[16];
  const int b = static_cast<int>(blockIdx.x / static_cast<unsigned>(a.max_cands));
  const int i = static_cast<int>(blockIdx.x % static_cast<unsigned>(a.max_cands));
  const User us = user_ranges(a, b);
  if (!us.ok || i >= us.cb) return;   // reported by the first kernel
  const int D = a.H * 128;
  const size_t cand = checked(a.status, us.c0 + i, a.C, BS_CAND4_ROW);
  const int col = 4 * static_cast<int>(threadIdx.x);
  const int h = static_cast<int>(threadIdx.x >> 5);
  const size_t at = cand * D + col;
  auto row4 = [&](const void* p, float (&f)[4]) {
    const uint2 w = __ldg(reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p) + at));
    f[0] = bf16_lo(w.x);
    f[1] = bf16_hi(w.x);
    f[2] = bf16_lo(w.y);
    f[3] = bf16_hi(w.y);
  };
  float q[4], k[4], v[4], u[4];
  row4(a.q, q);
  row4(a.k, k);
  row4(a.v, v);
  row4(a.u, u);
  float x = fmaf(q[0], k[0], fmaf(q[1], k[1], fmaf(q[2], k[2], q[3] * k[3])));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  if (POS) x += __ldg(a.rab_pos + static_cast<size_t>(h) * (2 * static_cast<size_t>(a.L) - 1) + (a.L - 1));
  if (TIME) x += __ldg(a.rab_time + h * a.nb);   // time difference 0: bucket 0
  const float self = silu_f(x);
  const float inv_n = 1.0f / static_cast<float>(a.norm_len > 0 ? a.norm_len : us.nb + 1);
  grid_wait();
  float o[4] = {0.f, 0.f, 0.f, 0.f};
  // the slices that hold keys: part p of split s starts at key s chunk + 16 p
  const size_t stride = static_cast<size_t>(a.C) * D;
  for (int s = 0; s * cut.chunk < us.nb; ++s)
    for (int p = 0; p < cut.parts; ++p) {
      if (s * cut.chunk + 16 * p >= us.nb) break;
      const float4 f = *reinterpret_cast<const float4*>(
          a.part + static_cast<size_t>(s * cut.parts + p) * stride + at);
      o[0] += f.x;
      o[1] += f.y;
      o[2] += f.z;
      o[3] += f.w;
    }
  float sum = 0.f;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    o[e] = fmaf(self, v[e], o[e]) * inv_n;
    sum += o[e];
  }
  const float mean = block_sum(sum, red, a.H) / static_cast<float>(D);
  float sq = 0.f;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    o[e] -= mean;
    sq = fmaf(o[e], o[e], sq);
  }
  const float rstd = 1.0f / sqrtf(block_sum(sq, red, a.H) / static_cast<float>(D) + a.eps);
  float y[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float w = a.ln_weight ? __ldg(a.ln_weight + col + e) : 1.f;
    const float c = a.ln_bias ? __ldg(a.ln_bias + col + e) : 0.f;
    y[e] = fmaf(o[e] * rstd, w, c) * silu_f(u[e]);
  }
  *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.y) + at) =
      make_uint2(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]));
}

template <bool POS, bool TIME>
cudaError_t launch_finish(const Cand4Args& a, const Cand4Cut& cut, bool after_sums,
                          cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.B) * static_cast<unsigned>(a.max_cands));
  cfg.blockDim = dim3(32 * static_cast<unsigned>(a.H));
  cfg.stream = stream;
  // launched while the kernel of the sums runs; waits for it before reading
  // them (without one before it, an ordinary launch: what runs before is then
  // the caller's, and may still write the candidates)
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = after_sums ? 1 : 0;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, hstu_cand4_finish<POS, TIME>, a, cut);
}

template <bool POS, bool TIME>
cudaError_t launch_few(const Cand4Args& a, const Cand4Cut& cut, cudaStream_t stream) {
  const unsigned grid = static_cast<unsigned>(a.B) * cut.cgroups * cut.splits * cut.hgroups;
  if (cut.nt == 1)
    hstu_cand4_few<1, POS, TIME><<<grid, kThreads, 0, stream>>>(a, cut);
  else
    hstu_cand4_few<2, POS, TIME><<<grid, kThreads, 0, stream>>>(a, cut);
  return cudaGetLastError();
}

}  // namespace

// Keys per CTA: about four CTAs per SM over the whole problem, at least two
// 16-key blocks per warp, at most kMaxChunk.
constexpr int64_t kCtas = 4 * 148;

// More candidates per user than this take the tcgen05 kernel.
constexpr int kFewMax = 16;

Cand4Cut cand4_cut(int B, int H, int max_seq_len, int max_cands) {
  Cand4Cut c;
  c.many = max_cands > kFewMax;
  if (c.many) {
    c.heads = 1;
    c.parts = 1;
    c.hgroups = H;
    c.nt = 0;
    c.cgroups = static_cast<int>((static_cast<int64_t>(max_cands) + 255) / 256);
    // one CTA walks a whole history where there are CTAs enough; otherwise
    // histories are cut so that there are about two a SM
    const int64_t groups = static_cast<int64_t>(B) * H * c.cgroups;
    const int64_t want = groups > 2 * 148 ? 1 : (2 * 148 + groups - 1) / (groups > 0 ? groups : 1);
    int64_t chunk = ((max_seq_len + want - 1) / want + 127) / 128 * 128;
    if (chunk < 256) chunk = 256;
    c.chunk = static_cast<int>(chunk);
    c.splits = static_cast<int>((max_seq_len + chunk - 1) / chunk);
    return c;
  }
  c.heads = H < kWarps ? H : kWarps;
  c.parts = kWarps / c.heads;
  c.hgroups = (H + kWarps - 1) / kWarps;
  c.nt = max_cands <= 8 ? 1 : 2;
  c.cgroups = static_cast<int>((static_cast<int64_t>(max_cands) + 8 * c.nt - 1) / (8 * c.nt));
  const int64_t step = 16 * c.parts;
  const int64_t groups = static_cast<int64_t>(B) * c.hgroups * c.cgroups;
  int64_t chunk = groups > kCtas ? kMaxChunk : (groups * max_seq_len / kCtas + step - 1) / step * step;
  const int64_t most = kMaxChunk / step * step;
  chunk = chunk < 2 * step ? 2 * step : chunk > most ? most : chunk;
  c.chunk = static_cast<int>(chunk);
  c.splits = static_cast<int>((max_seq_len + chunk - 1) / chunk);
  return c;
}

// Few candidates: splits <= max_seq_len / (2 step) + 1 always, and splits <=
// kCtas / groups + 1 where the chunk is between its limits; C <= 16 groups /
// hgroups candidates then make at most 16 kCtas + C rows a part, and
// max_seq_len / most + 1 splits at the upper limit.  Many: splits <=
// max_seq_len / 256 + 1, and splits <= 296 / groups + 1 with C <= 256 groups / H.
size_t cand4_part_rows(int H, int max_seq_len, int C, int max_cands) {
  const int64_t parts = H < kWarps ? kWarps / H : 1;
  const int64_t step = 16 * parts, most = kMaxChunk / step * step;
  const int64_t c = C, n = max_seq_len;
  const int64_t few = parts * std::min(c * (n / (2 * step) + 1), 16 * kCtas + c * (n / most + 2));
  const int64_t many = std::min(c * (n / 256 + 1), c + 2 * 148 * 256 / H + 1);
  return static_cast<size_t>(max_cands > kFewMax ? std::max(few, many) : few);
}

size_t cand4_plan_bytes(int max_seq_len, int C, int max_cands) {
  return max_cands > kFewMax ? (static_cast<size_t>(max_seq_len) + 127) / 128 * 16 * C : 0;
}

cudaError_t launch_cand4_finish(const Cand4Args& a, const Cand4Cut& cut, bool after_sums,
                                cudaStream_t stream) {
  const bool pos = a.rab_pos != nullptr, time = a.rab_time != nullptr;
  if (pos && time) return launch_finish<true, true>(a, cut, after_sums, stream);
  if (pos) return launch_finish<true, false>(a, cut, after_sums, stream);
  if (time) return launch_finish<false, true>(a, cut, after_sums, stream);
  return launch_finish<false, false>(a, cut, after_sums, stream);
}

cudaError_t launch_cand4_few(const Cand4Args& a, const Cand4Cut& cut, cudaStream_t stream) {
  const bool pos = a.rab_pos != nullptr, time = a.rab_time != nullptr;
  if (pos && time) return launch_few<true, true>(a, cut, stream);
  if (pos) return launch_few<true, false>(a, cut, stream);
  if (time) return launch_few<false, true>(a, cut, stream);
  return launch_few<false, false>(a, cut, stream);
}

}  // namespace hstu
