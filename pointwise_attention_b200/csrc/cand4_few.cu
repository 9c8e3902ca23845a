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
// The histories, one after another as the offsets pack them, are cut into
// equal shares of tokens, one per CTA (two CTAs a SM, shares of at most
// kMaxShare tokens), whatever the histories' lengths; a CTA walks the pieces of
// the histories that its share covers.  A CTA takes up to 8 heads, a warp per
// head, or several warps per head where there are fewer heads.  All heads of a
// cache row are neighbours, so a CTA reads whole contiguous rows, once for a
// user's candidates (8 NT of them at most).  Per 16 keys a warp computes
// S^T = K Q^T and O^T += V^T P^T with m16n8k16 MMAs whose A operand is decoded
// in registers straight from the codes (the order of the dimensions in an MMA
// is free as long as both operands share it, so a lane takes whole 16-byte runs
// of codes):
//   K: lane (g, t) holds dims 32t.. of keys g and g + 8 (one scale each);
//   V: lane (g, t) holds dims 16g.. of keys 2t, 2t+1, 2t+8, 2t+9.
// The candidates are the MMA's 8 columns: with few of them the tensor core's
// work is small beside decoding and the cache's bytes, which bound the kernel.
// P enters the second product as the sum of two bf16 numbers (2^-16 of it is
// lost; one number would lose 2^-8, as much as the output's own rounding, to
// save eight of 24 MMAs that do not bound the kernel); scores, SiLU and sums
// are fp32.
//
// The pieces' sums go to the workspace in fp32; a second kernel adds them in
// order (the result does not depend on timing), adds the self term and applies
// the LayerNorm and the gate.
//
// Measured on a B200: one candidate for each of 32 users, 8 heads, histories of
// 256-4096 tokens (81 MB of cache): 46 us (the bytes alone take 12).  Latency
// bounds it: a warp's chain of decoding, MMA, SiLU, transpose and MMA, some 500
// instructions per 16 keys and head (200 of them decoding), leaves half of the
// issue slots empty at 14 warps an SM; 19 us are starts and the last kernel (a
// user's 16 keys).  A CTA per (user, run of keys) left SMs idle at the
// end (64 us); cp.async by the lanes cost 145 shared-memory wavefronts a block.
#include <cuda_bf16.h>

#include <atomic>

#include "bounds.cuh"
#include "internal_ops.h"
#include "kv4.cuh"
#include "ops.cuh"
#include "ptx.cuh"
#include "tile_math.cuh"

namespace hstu {
namespace {

constexpr int kWarps = kCand4FewWarps;
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxShare = kCand4MaxShare;

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// SiLU in fp32, x / (1 + 2^(-x log2 e)); for very negative x the power is
// infinite and the quotient 0
__device__ __forceinline__ float silu_f(float x) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
  return x * r;
}

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

// Before a thread of the last kernel leaves with nothing to do: the grid's first
// block stays until the kernels before are over, so that this kernel ends after
// them whatever the ranges are.  The next call on the workspace starts behind
// this kernel alone, and the pass over the timestamps may still be at work for
// users whose ranges this one reports.
__device__ __forceinline__ void leave_last() {
  if (blockIdx.x == 0) grid_wait();
}

// A round of a piece: 16 keys per part, brought to shared memory by bulk copies
// (whole cache rows, which need no address arithmetic of the threads), kStages
// - 1 rounds ahead.
constexpr int kStages = 4;
constexpr int kCodeBytes = 8192;                 // 16 keys x 8 heads x 64, whatever the heads
constexpr int kScaleBytes = 16 * 16 * 8 + 16;    // 16 keys x up to 16 heads x 8, and a lead
constexpr int kStageBytes = 2 * (kCodeBytes + kScaleBytes);
static_assert(kScaleBytes % 16 == 0, "bulk copies start on 16 bytes");

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

// Tokens of a CTA's share: whole rounds of 16-key blocks, at least two.
__device__ __forceinline__ int share_of(const Cand4Args& a, const Cand4Cut& cut) {
  const int step = 16 * cut.parts;
  const int64_t total = __ldg(a.offsets + a.B);
  const int64_t per = (total + cut.ctas - 1) / cut.ctas;
  const int64_t up = (per + step - 1) / step * step;
  // (offsets that contradict the sizes are reported; the share stays in its room)
  return static_cast<int>(up < 2 * step ? 2 * step : up > kMaxShare ? kMaxShare : up);
}

// Offsets that keep to the sizes end within the CTAs' shares.
__device__ __forceinline__ bool in_shares(const User& us, int share, const Cand4Cut& cut) {
  return static_cast<int64_t>(us.s) + us.nb <= static_cast<int64_t>(cut.ctas) * share;
}

template <int NT, bool POS, bool TIME>
__global__ void __launch_bounds__(kThreads, NT == 1 ? 2 : 1)
    hstu_cand4_few(const __grid_constant__ Cand4Args a, const Cand4Cut cut) {
  constexpr int NC = 8 * NT;
  __shared__ float s_rabt[TIME ? kWarps : 1][TIME ? kMaxBuckets : 1];
  __shared__ long long s_thr[TIME ? kThrLen : 1];
  __shared__ signed char s_first[TIME ? 64 : 1];
  __shared__ __align__(16) uint8_t s_bk[TIME ? (kMaxShare + 16 * kWarps) * NC : 16];   // [key][candidate] bucket
  extern __shared__ __align__(16) uint8_t s_dyn[];                     // the stages
  __shared__ __align__(8) uint64_t s_bar[2 * kStages];                 // full, empty
  __shared__ int s_abort;
  grid_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int hg = static_cast<int>(blockIdx.x) % cut.hgroups, cta = static_cast<int>(blockIdx.x) / cut.hgroups;
  const int share = share_of(a, cut);
  const int64_t begin = static_cast<int64_t>(cta) * share, end = begin + share;
  // The last user that starts at or before the share's first token: by
  // bisection down to 256 users, then all threads look at one each (a chain of
  // loads costs half a microsecond a link).
  int b = 0, among = a.B;
  while (among > kThreads) {
    const int half = among / 2;
    if (__ldg(a.offsets + b + half) <= begin) b += half;
    among -= half;
  }
  {
    const int i = static_cast<int>(threadIdx.x);
    const int n = __syncthreads_count(i > 0 && i < among && __ldg(a.offsets + b + i) <= begin);
    b += n;
  }
  const int h = 8 * hg + warp % cut.heads, part = warp / cut.heads;
  const int step = 16 * cut.parts;
  const bool works = h < a.H && part < cut.parts;
  const float* rpos = POS ? a.rab_pos + static_cast<size_t>(h) * (2 * static_cast<size_t>(a.L) - 1) + (a.L - 1)
                          : nullptr;
  const int hc = min(kWarps, a.H - 8 * hg);          // heads of this CTA
  const unsigned seg = static_cast<unsigned>(hc) * 64u;   // bytes of a row's codes in a stage
  auto full = [&](int st) { return smem_u32(s_bar + st); };
  auto empty = [&](int st) { return smem_u32(s_bar + kStages + st); };
  volatile int* abort_flag = &s_abort;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(full(i), 1);
      mbar_init(empty(i), static_cast<uint32_t>(hc * cut.parts));   // the warps that work
    }
    s_abort = 0;
    fence_mbar_init();
  }
  __syncthreads();
  // A wait that runs out is reported; then nothing is waited for or copied any more.
  auto wait = [&](uint32_t bar, unsigned use) {
    if (mbar_try_wait(bar, use & 1u) || *abort_flag) return;
    if (!mbar_wait(bar, use & 1u, abort_flag)) {
      if (a.status) atomicOr(a.status, kStatusTimeout);
      *abort_flag = 1;
    }
  };
  unsigned round0 = 0;    // rounds of the pieces before
  unsigned issued = 0;    // warp 0: rounds whose copies were issued
  if (TIME) {
    for (int i = threadIdx.x; i < kThrLen; i += kThreads) s_thr[i] = a.bt.thr[i];
    for (int i = threadIdx.x; i < 64; i += kThreads) s_first[i] = a.bt.first_k[i];
    for (int i = threadIdx.x; i < cut.heads * kMaxBuckets; i += kThreads) {
      const int hh = 8 * hg + i / kMaxBuckets, k = i % kMaxBuckets;
      s_rabt[i / kMaxBuckets][k] = (hh < a.H && k < a.nb) ? __ldg(a.rab_time + hh * a.nb + k) : 0.f;
    }
  }

  for (; b < a.B; ++b) {
    const User us = user_ranges(a, b);   // (one that is not ok is reported by the last kernel)
    if (us.s >= end) break;
    const int first = static_cast<int>(begin > us.s ? begin - us.s : 0);   // keys of this piece
    const int last = static_cast<int>(end - us.s < us.nb ? end - us.s : us.nb);
    if (!us.ok || !in_shares(us, share, cut) || first >= last || us.cb == 0) continue;
    const int cands = us.cb, cand0 = us.c0, n_keys = last - first;

    const int rounds = (n_keys + step - 1) / step;
    // warp 0 brings the rounds in order: codes of this CTA's heads, scales of
    // all heads (from the 16-byte boundary at or before the round's first)
    const size_t row0 = static_cast<size_t>(us.r0 + first);
    const unsigned lead = (a.H & 1) ? 8u * (static_cast<unsigned>(row0) & 1u) : 0u;   // steps are even
    const uint8_t* kc0 = a.k_codes + (row0 * a.H + 8 * hg) * 64;
    const uint8_t* vc0 = a.v_codes + (row0 * a.H + 8 * hg) * 64;
    const uint8_t* ks0 = reinterpret_cast<const uint8_t*>(a.k_scales) + (row0 * a.H * 8 - lead);
    const uint8_t* vs0 = reinterpret_cast<const uint8_t*>(a.v_scales) + (row0 * a.H * 8 - lead);
    int next = 0;
    auto bring = [&]() {
      const unsigned use = round0 + next;
      const int st = static_cast<int>(use % kStages);
      if (use >= kStages) wait(empty(st), use / kStages - 1);
      if (*abort_flag) return;
      issued = use + 1;
      const int rows = min(step, n_keys - next * step);
      checked(a.status, us.r0 + first + next * step, a.R, BS_CAND4_KEY);
      const uint32_t dst = smem_u32(s_dyn) + st * kStageBytes;
      // The scales' copy ends on 16 bytes too.  With an odd number of heads it
      // may be 8 bytes short of a boundary: it takes the next row's with it,
      // or, at the end of the cache, stops before and a thread brings the rest.
      uint32_t sbytes = lead + static_cast<uint32_t>(rows * a.H) * 8u;
      if (sbytes & 8u) {
        if (us.r0 + first + next * step + rows < a.R) {
          sbytes += 8u;
        } else {
          sbytes -= 8u;
          if (lane == 0) {
            uint8_t* at = s_dyn + st * kStageBytes + 2 * kCodeBytes + sbytes;
            *reinterpret_cast<uint2*>(at) = __ldg(reinterpret_cast<const uint2*>(ks0 + sbytes));
            *reinterpret_cast<uint2*>(at + kScaleBytes) =
                __ldg(reinterpret_cast<const uint2*>(vs0 + sbytes));
          }
        }
      }
      if (lane == 0) {
        mbar_arrive_expect_tx(full(st), 2u * (rows * seg + sbytes));
        if (sbytes > 0) {
          bulk_load(dst + 2 * kCodeBytes, ks0, sbytes, full(st));
          bulk_load(dst + 2 * kCodeBytes + kScaleBytes, vs0, sbytes, full(st));
        }
        if (cut.hgroups == 1) {   // whole rows: one run
          bulk_load(dst, kc0, rows * seg, full(st));
          bulk_load(dst + kCodeBytes, vc0, rows * seg, full(st));
        }
      }
      if (cut.hgroups > 1) {
        __syncwarp();
        if ((lane & 15) < rows)   // 16 rows of K, 16 of V
          bulk_load(dst + (lane >> 4) * kCodeBytes + (lane & 15) * seg,
                    (lane < 16 ? kc0 : vc0) + static_cast<unsigned>((lane & 15) * a.H * 64), seg, full(st));
      }
      const unsigned by = static_cast<unsigned>(step * a.H);
      kc0 += by * 64u;
      vc0 += by * 64u;
      ks0 += by * 8u;
      vs0 += by * 8u;
      ++next;
    };
    if (warp == 0)
      for (int r = 0; r < min(rounds, kStages - 1); ++r) bring();
    if (TIME) {
      __syncthreads();   // the piece before is done with its buckets
      // buckets of candidates that do not exist: 0, as good as any
      for (int i = threadIdx.x; i < n_keys * (NC / 8); i += kThreads)
        reinterpret_cast<uint2*>(s_bk)[i] = make_uint2(0u, 0u);
      __syncthreads();
      // every (key, candidate) bucket once for all heads
      for (int i = threadIdx.x; i < n_keys * cands; i += kThreads) {
        const int j = i / cands, c = i - j * cands;
        const int k =
            time_bucket(__ldg(a.cand_ts + checked(a.status, cand0 + c, a.C, BS_CAND4_ROW)) -
                            __ldg(a.timestamps + checked(a.status, us.s + first + j, a.T, BS_CAND4_TS)),
                        s_thr, s_first);
        s_bk[j * NC + c] = static_cast<uint8_t>(k);
      }
      __syncthreads();
    }
    if (!works) {
      round0 += rounds;
      continue;
    }

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

    // position bias of keys g, g + 8 of this warp's 16, a round ahead (keys
    // past the last take any entry)
    float pos[2] = {0.f, 0.f}, pnext[2] = {0.f, 0.f};
    int dist = us.nb - first - 16 * part - g;   // of key g of the next round
    auto load_pos = [&]() {
      pnext[0] = __ldg(rpos + max(dist, 0));
      pnext[1] = __ldg(rpos + max(dist - 8, 0));
      dist -= step;
    };
    if (POS) load_pos();
    // where this lane's codes and scales are in a stage
    const unsigned kb = (h - 8 * hg) * 64u, sb = 2 * kCodeBytes + lead + h * 8u, H8 = a.H * 8u;
    const int k0 = 16 * part + g, v0 = 16 * part + 2 * t;
    unsigned st = round0 % kStages, turn = round0 / kStages;
    int left = n_keys - 16 * part;             // keys from this warp's first of the round on
    const uint8_t* bk = s_bk + k0 * NC + 2 * t;   // buckets of key g, candidates 2t, 2t + 1
    for (int r = 0; r < rounds; ++r) {
      if (warp == 0 && next < rounds) bring();
      if (POS) {
        pos[0] = pnext[0];
        pos[1] = pnext[1];
        load_pos();
      }
      wait(full(st), turn);
      __syncwarp();
      const uint8_t* stage = s_dyn + st * kStageBytes;
      const uint32_t gone = empty(st);
      if (++st == kStages) {
        st = 0;
        ++turn;
      }
      uint4 kc[2];
      uint2 vc[4];
      uint32_t ks[2], vs[4];
      auto take = [&](auto row_of) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const unsigned w = row_of(k0 + 8 * i);
          kc[i] = *reinterpret_cast<const uint4*>(stage + (kb + 16 * t) + w * seg);
          ks[i] = *reinterpret_cast<const uint16_t*>(stage + (sb + 2 * t) + w * H8);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const unsigned w = row_of(v0 + (i & 1) + 8 * (i >> 1));
          vc[i] = *reinterpret_cast<const uint2*>(stage + (kCodeBytes + kb + 8 * g) + w * seg);
          vs[i] = *reinterpret_cast<const uint16_t*>(stage + (kScaleBytes + sb + (g & 6)) + w * H8);
        }
      };
      if (left >= 16) {
        take([](int w) { return static_cast<unsigned>(w); });
      } else if (left > 0) {
        // rows past the last repeat it (their P is 0)
        take([&](int w) { return static_cast<unsigned>(min(w, left + 16 * part - 1)); });
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(gone);        // all of it is in registers
      if (left <= 0) break;                    // (only in the last round)
      // S^T = K Q^T, two sums of four MMAs each
      float s[NT][4], s_[NT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[n][i] = s_[n][i] = 0.f;
      {
        const uint32_t s0 = __byte_perm(ks[0], 0u, 0x1010), s1 = __byte_perm(ks[1], 0u, 0x1010);
        const uint32_t m0 = kv4_m24(s0), m1 = kv4_m24(s1);
        const uint32_t w0[4] = {kc[0].x, kc[0].y, kc[0].z, kc[0].w};
        const uint32_t w1[4] = {kc[1].x, kc[1].y, kc[1].z, kc[1].w};
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const uint32_t a0 = kv4_pair_fma<0>(w0[w], s0, m0), a1 = kv4_pair_fma<0>(w1[w], s1, m1);
          const uint32_t a2 = kv4_pair_fma<1>(w0[w], s0, m0), a3 = kv4_pair_fma<1>(w1[w], s1, m1);
          const uint32_t b0 = kv4_pair_fma<2>(w0[w], s0, m0), b1 = kv4_pair_fma<2>(w1[w], s1, m1);
          const uint32_t b2 = kv4_pair_fma<3>(w0[w], s0, m0), b3 = kv4_pair_fma<3>(w1[w], s1, m1);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            mma_16816(s[n], a0, a1, a2, a3, qb[n][4 * w], qb[n][4 * w + 1]);
            mma_16816(s_[n], b0, b1, b2, b3, qb[n][4 * w + 2], qb[n][4 * w + 3]);
          }
        }
      }
      // P: keys g, g + 8 by candidates 2t, 2t+1, transposed into the B operand
      uint32_t pb[NT][2], pl[NT][2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float x0 = s[n][2 * i] + s_[n][2 * i], x1 = s[n][2 * i + 1] + s_[n][2 * i + 1];
          if (POS) {
            x0 += pos[i];
            x1 += pos[i];
          }
          if (TIME) {
            // (buckets of keys past the last are old ones or none: below 128 or cut there)
            const uint32_t k2 = *reinterpret_cast<const uint16_t*>(bk + 8 * i * NC + 8 * n);
            const float* rt = s_rabt[warp % cut.heads];
            x0 += rt[k2 & 0x7Fu];
            x1 += rt[(k2 >> 8) & 0x7Fu];
          }
          const bool in = g + 8 * i < left;
          const float p0 = in ? silu_f(x0) : 0.f, p1 = in ? silu_f(x1) : 0.f;
          const uint32_t hi = pack_bf16x2(p0, p1);
          pb[n][i] = transpose8(hi);
          pl[n][i] = transpose8(pack_bf16x2(p0 - bf16_lo(hi), p1 - bf16_hi(hi)));
        }
      }
      left -= step;
      bk += step * NC;
      // O^T += V^T P^T
      {
        // scales of the keys that share a register: (2t, 2t+1), (2t+8, 2t+9)
        const uint32_t sa = __byte_perm(vs[0], vs[1], 0x5410), sb = __byte_perm(vs[2], vs[3], 0x5410);
        const uint32_t ma = kv4_m24(sa), mb = kv4_m24(sb);
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          const uint32_t va = w ? vc[0].y : vc[0].x, vb = w ? vc[1].y : vc[1].x;
          const uint32_t vg = w ? vc[2].y : vc[2].x, vh = w ? vc[3].y : vc[3].x;
          // even and odd dims of two keys, a key per half
          const uint32_t ea = __byte_perm(va, vb, 0x5410), oa = __byte_perm(va, vb, 0x7632);
          const uint32_t eb = __byte_perm(vg, vh, 0x5410), ob = __byte_perm(vg, vh, 0x7632);
#define HSTU_PV(I)                                                                       \
    {                                                                                      \
      const uint32_t a0 = kv4_pair_fma<I>(ea, sa, ma), a1 = kv4_pair_fma<I>(oa, sa, ma);   \
      const uint32_t a2 = kv4_pair_fma<I>(eb, sb, mb), a3 = kv4_pair_fma<I>(ob, sb, mb);   \
      _Pragma("unroll") for (int n = 0; n < NT; ++n) {                                     \
        mma_16816(o[n][4 * w + I], a0, a1, a2, a3, pb[n][0], pb[n][1]);                    \
        mma_16816(o[n][4 * w + I], a0, a1, a2, a3, pl[n][0], pl[n][1]);                  \
    }                                                                                    \
    }
          HSTU_PV(0)
          HSTU_PV(1)
          HSTU_PV(2)
          HSTU_PV(3)
#undef HSTU_PV
        }
      }
    }
    round0 += rounds;
    if (16 * part >= n_keys) continue;
    // lane (g, t): dims 16g..16g+15 of candidates 2t, 2t+1
    const int piece = (cta + b) * cut.parts + part;   // pieces begin with a CTA or with a user
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        if (8 * n + 2 * t + c >= cands) continue;
        const size_t row = checked(a.status, static_cast<size_t>(piece) * a.max_cands + 8 * n + 2 * t + c,
                                   a.part_rows, BS_CAND4_SUM);
        float4* dst = reinterpret_cast<float4*>(a.part + row * (a.H * 128) + h * 128 + 16 * g);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          dst[i] = make_float4(o[n][2 * i][c], o[n][2 * i][c + 2], o[n][2 * i + 1][c], o[n][2 * i + 1][c + 2]);
      }
  }
  // copies still under way (after a wait that ran out) land before shared memory goes
  if (warp == 0 && *abort_flag)
    for (unsigned r = issued > kStages ? issued - kStages : 0u; r < issued; ++r)
      mbar_wait(full(static_cast<int>(r % kStages)), (r / kStages) & 1u, nullptr);
}

// Sum over the first 32 H threads of a block, the same in each of them.
__device__ __forceinline__ float heads_sum(float v, float* red, int H) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  named_bar_sync(1, 32 * H);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  named_bar_sync(1, 32 * H);
  v = red[0];
  for (int i = 1; i < H; ++i) v += red[i];
  return v;
}

// A block per candidate; a warp per head, four dimensions per thread, and
// `groups` such sets of warps that share the slices (the sums over parts of the
// history) between them.
template <bool POS, bool TIME>
__global__ void __launch_bounds__(1024) hstu_cand4_finish(const __grid_constant__ Cand4Args a,
                                                          const Cand4Cut cut, int groups) {
  __shared__ float red[16];
  __shared__ float4 sums[32][32];
  const int b = static_cast<int>(blockIdx.x / static_cast<unsigned>(a.max_cands));
  const int i = static_cast<int>(blockIdx.x % static_cast<unsigned>(a.max_cands));
  const User us = user_ranges(a, b);
  const int share = share_of(a, cut);
  if (!us.ok || !in_shares(us, share, cut)) {
    if (threadIdx.x == 0 && a.status) atomicOr(a.status, kStatusBadOffsets);
    return leave_last();
  }
  if (i >= us.cb) return leave_last();
  const int D = a.H * 128;
  const size_t cand = checked(a.status, us.c0 + i, a.C, BS_CAND4_ROW);
  const int warp = static_cast<int>(threadIdx.x >> 5), lane = static_cast<int>(threadIdx.x & 31);
  const int h = warp % a.H, set = warp / a.H;
  const int col = 128 * h + 4 * lane;
  const size_t at = cand * D + col;
  float self = 0.f, v[4] = {}, u[4] = {};
  if (set == 0) {
    auto row4 = [&](const void* p, float (&f)[4]) {
      const uint2 w = __ldg(reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p) + at));
      f[0] = bf16_lo(w.x);
      f[1] = bf16_hi(w.x);
      f[2] = bf16_lo(w.y);
      f[3] = bf16_hi(w.y);
    };
    float q[4], k[4];
    row4(a.q, q);
    row4(a.k, k);
    row4(a.v, v);
    row4(a.u, u);
    float x = fmaf(q[0], k[0], fmaf(q[1], k[1], fmaf(q[2], k[2], q[3] * k[3])));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    if (POS) x += __ldg(a.rab_pos + static_cast<size_t>(h) * (2 * static_cast<size_t>(a.L) - 1) + (a.L - 1));
    if (TIME) x += __ldg(a.rab_time + h * a.nb);   // time difference 0: bucket 0
    self = silu_f(x);
  }
  const float inv_n = 1.0f / static_cast<float>(a.norm_len > 0 ? a.norm_len : us.nb + 1);
  // where the slices are, how far apart and how many
  // (pieces of the CTAs whose shares cover the history; of a piece's parts
  // those that have a 16-key block)
  const int c0 = us.s / share, c1 = us.nb > 0 ? (us.s + us.nb - 1) / share : c0;
  const size_t stride = static_cast<size_t>(a.max_cands) * D;
  const float* src = a.part + ((static_cast<size_t>(c0) + b) * cut.parts * a.max_cands + i) * D + col;
  const int slices = us.nb > 0 ? (c1 - c0 + 1) * cut.parts : 0;
  // whether slice s was written
  auto written = [&](int s) {
    if (cut.parts == 1) return true;
    const int64_t lo = static_cast<int64_t>(us.s / share + s / cut.parts) * share;
    const int64_t first = lo > us.s ? lo : us.s;
    const int64_t last = lo + share < us.s + us.nb ? lo + share : us.s + us.nb;
    return 16 * (s % cut.parts) < last - first;
  };
  grid_wait();
  float o[4] = {0.f, 0.f, 0.f, 0.f};
  for (int s = set; s < slices; s += 4 * groups) {
    float4 f[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      f[e] = s + e * groups < slices && written(s + e * groups)
                 ? *reinterpret_cast<const float4*>(src + (s + e * groups) * stride)
                 : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      o[0] += f[e].x;
      o[1] += f[e].y;
      o[2] += f[e].z;
      o[3] += f[e].w;
    }
  }
  if (groups > 1) {
    sums[warp][lane] = make_float4(o[0], o[1], o[2], o[3]);
    __syncthreads();
    if (set > 0) return;
    for (int e = 1; e < groups; ++e) {
      const float4 f = sums[e * a.H + h][lane];
      o[0] += f.x;
      o[1] += f.y;
      o[2] += f.z;
      o[3] += f.w;
    }
  }
  float sum = 0.f;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    o[e] = fmaf(self, v[e], o[e]) * inv_n;
    sum += o[e];
  }
  const float mean = heads_sum(sum, red, a.H) / static_cast<float>(D);
  float sq = 0.f;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    o[e] -= mean;
    sq = fmaf(o[e], o[e], sq);
  }
  const float rstd = 1.0f / sqrtf(heads_sum(sq, red, a.H) / static_cast<float>(D) + a.eps);
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

// The same for many candidates: a warp per candidate, which keeps its whole row
// (NH >= H heads, four dimensions of each per lane) in registers.
template <int NH, bool POS, bool TIME>
__global__ void __launch_bounds__(256) hstu_cand4_finish_rows(const __grid_constant__ Cand4Args a,
                                                              const Cand4Cut cut) {
  const int blocks = (a.max_cands + 7) / 8;
  const int b = static_cast<int>(blockIdx.x / static_cast<unsigned>(blocks));
  const int i = 8 * static_cast<int>(blockIdx.x % static_cast<unsigned>(blocks)) +
                static_cast<int>(threadIdx.x >> 5);
  const int lane = static_cast<int>(threadIdx.x & 31);
  const User us = user_ranges(a, b);
  const int cfirst = __ldg(a.cand_offsets);
  if (!us.ok || !cand4_in_sums(us.c0, us.cb, cfirst, a.sum_rows)) {
    if (threadIdx.x == 0 && a.status) atomicOr(a.status, kStatusBadOffsets);
    return leave_last();
  }
  if (i >= us.cb) return leave_last();
  const int D = a.H * 128;
  const size_t cand = checked(a.status, us.c0 + i, a.C, BS_CAND4_ROW);
  const size_t at = cand * D + 4 * lane;     // head h: + 128 h
  // (heads past H read nothing and count as zeros: no branch stands between the
  // loads of different heads)
  auto row2 = [&](const void* p, int h) {
    return h < a.H ? __ldg(reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p) + at + 128 * h))
                   : make_uint2(0u, 0u);
  };
  float self[NH];
  {
    uint2 q[NH], k[NH];
#pragma unroll
    for (int h = 0; h < NH; ++h) {
      q[h] = row2(a.q, h);
      k[h] = row2(a.k, h);
    }
#pragma unroll
    for (int h = 0; h < NH; ++h) {
      float x = fmaf(bf16_lo(q[h].x), bf16_lo(k[h].x),
                     fmaf(bf16_hi(q[h].x), bf16_hi(k[h].x),
                          fmaf(bf16_lo(q[h].y), bf16_lo(k[h].y), bf16_hi(q[h].y) * bf16_hi(k[h].y))));
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
      if (POS && h < a.H)
        x += __ldg(a.rab_pos + static_cast<size_t>(h) * (2 * static_cast<size_t>(a.L) - 1) + (a.L - 1));
      if (TIME && h < a.H) x += __ldg(a.rab_time + h * a.nb);   // time difference 0: bucket 0
      self[h] = silu_f(x);
    }
  }
  const float inv_n = 1.0f / static_cast<float>(a.norm_len > 0 ? a.norm_len : us.nb + 1);
  const int slices = (us.nb + cut.chunk - 1) / cut.chunk;
  const size_t stride = static_cast<size_t>(a.sum_rows) * D;
  const size_t sum0 = static_cast<size_t>(us.c0 - cfirst + i) * D + 4 * lane;
  uint2 v[NH];
#pragma unroll
  for (int h = 0; h < NH; ++h) v[h] = row2(a.v, h);
  grid_wait();
  float4 o[NH];
#pragma unroll
  for (int h = 0; h < NH; ++h) o[h] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s = 0; s < slices; ++s) {
    const float* src = a.part + checked(a.status, s * stride + sum0, a.part_rows * D, BS_CAND4_SUM);
    float4 f[NH];
#pragma unroll
    for (int h = 0; h < NH; ++h)
      f[h] = h < a.H ? *reinterpret_cast<const float4*>(src + 128 * h) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int h = 0; h < NH; ++h) {
      o[h].x += f[h].x;
      o[h].y += f[h].y;
      o[h].z += f[h].z;
      o[h].w += f[h].w;
    }
  }
  float sum = 0.f;
#pragma unroll
  for (int h = 0; h < NH; ++h) {
    o[h].x = fmaf(self[h], bf16_lo(v[h].x), o[h].x) * inv_n;
    o[h].y = fmaf(self[h], bf16_hi(v[h].x), o[h].y) * inv_n;
    o[h].z = fmaf(self[h], bf16_lo(v[h].y), o[h].z) * inv_n;
    o[h].w = fmaf(self[h], bf16_hi(v[h].y), o[h].w) * inv_n;
    sum += (o[h].x + o[h].y) + (o[h].z + o[h].w);
  }
  uint2 u[NH];
#pragma unroll
  for (int h = 0; h < NH; ++h) u[h] = row2(a.u, h);
#pragma unroll
  for (int e = 16; e > 0; e >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, e);
  const float mean = sum / static_cast<float>(D);
  float sq = 0.f;
#pragma unroll
  for (int h = 0; h < NH; ++h) {
    o[h].x -= mean;
    o[h].y -= mean;
    o[h].z -= mean;
    o[h].w -= mean;
    const float q = fmaf(o[h].x, o[h].x, fmaf(o[h].y, o[h].y, fmaf(o[h].z, o[h].z, o[h].w * o[h].w)));
    sq += h < a.H ? q : 0.f;
  }
#pragma unroll
  for (int e = 16; e > 0; e >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, e);
  const float rstd = 1.0f / sqrtf(sq / static_cast<float>(D) + a.eps);
#pragma unroll
  for (int h = 0; h < NH; ++h) {
    if (h >= a.H) break;
    const float g[4] = {bf16_lo(u[h].x), bf16_hi(u[h].x), bf16_lo(u[h].y), bf16_hi(u[h].y)};
    const float z[4] = {o[h].x * rstd, o[h].y * rstd, o[h].z * rstd, o[h].w * rstd};
    const int col = 128 * h + 4 * lane;
    float y[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float w = a.ln_weight ? __ldg(a.ln_weight + col + e) : 1.f;
      const float c = a.ln_bias ? __ldg(a.ln_bias + col + e) : 0.f;
      y[e] = fmaf(z[e], w, c) * silu_f(g[e]);
    }
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.y) + at + 128 * h) =
        make_uint2(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]));
  }
}

template <bool POS, bool TIME>
cudaError_t launch_finish(const Cand4Args& a, const Cand4Cut& cut, bool after_sums,
                          cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.B) * static_cast<unsigned>(a.max_cands));
  // few candidates have many slices and the SMs to themselves
  const int groups = a.H <= 4 ? 8 : 32 / a.H;
  cfg.blockDim = dim3(32 * static_cast<unsigned>(a.H * groups));
  cfg.stream = stream;
  // launched while the kernel of the sums runs; waits for it before reading
  // them (without one before it, an ordinary launch: what runs before is then
  // the caller's, and may still write the candidates)
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = after_sums ? 1 : 0;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cut.many) {
    cfg.gridDim = dim3(static_cast<unsigned>(a.B) * ((static_cast<unsigned>(a.max_cands) + 7) / 8));
    cfg.blockDim = dim3(256);
    return a.H <= 8 ? cudaLaunchKernelEx(&cfg, hstu_cand4_finish_rows<8, POS, TIME>, a, cut)
                    : cudaLaunchKernelEx(&cfg, hstu_cand4_finish_rows<16, POS, TIME>, a, cut);
  }
  return cudaLaunchKernelEx(&cfg, hstu_cand4_finish<POS, TIME>, a, cut, groups);
}

template <bool POS, bool TIME>
cudaError_t launch_few(const Cand4Args& a, const Cand4Cut& cut, cudaStream_t stream) {
  const unsigned grid = static_cast<unsigned>(cut.ctas) * static_cast<unsigned>(cut.hgroups);
  constexpr int kRing = kStageBytes * kStages;
  auto kernel = cut.nt == 1 ? hstu_cand4_few<1, POS, TIME> : hstu_cand4_few<2, POS, TIME>;
  static std::atomic<bool> configured[2][64];   // per device: shared-memory opt-in done
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev < 0 || dev >= 64 || !configured[cut.nt - 1][dev].load(std::memory_order_acquire)) {
    err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRing);
    if (err != cudaSuccess) return err;
    if (dev >= 0 && dev < 64) configured[cut.nt - 1][dev].store(true, std::memory_order_release);
  }
  kernel<<<grid, kThreads, kRing, stream>>>(a, cut);
  return cudaGetLastError();
}

}  // namespace

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
