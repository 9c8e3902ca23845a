// cand4_sm100.cu -- candidate scoring against histories in a 4-bit cache, the
// form for many candidates: tcgen05 products over tiles decoded in shared
// memory.  cand4_few.cu states the operation; the sums that leave here are
// finished by the same last kernel.
//
// A CTA takes (user, 256 candidates, head, up to `chunk` keys): two tiles of
// 128 candidates share every decoded tile of 128 keys and values, which halves
// the decoding, and fill TMEM: S0, S1, O0, O1 at 128 columns each.
//   warps 0..3    decode: codes and scales from the cache (one tile ahead in
//                 registers) to bf16 in the 128-byte-swizzled layout of the
//                 MMA operands, two stages each of K and V; the keys' position
//                 bias and timestamps beside them
//   warps 4..19   epilogue, eight warps per candidate tile: half bias and SiLU
//                 in fp32, P (bf16, its one rounding) over S in TMEM; then O
//   warp 20       TMEM, the candidates' Q by TMA, and every MMA: while one
//                 tile's scores are in the epilogue, the tensor core works for
//                 the other
// SiLU(x) = h (1 + tanh h), h = x / 2, with tanh.approx.f32 (one special
// function per score, relative error at most 2^-11: at most |x| 2^-12 in P).
// Every wait is bounded; a wait that runs out sets the timeout bit of the
// status word and the CTA leaves through the same barriers.
#include <cuda_bf16.h>

#include <atomic>

#include "bounds.cuh"
#include "internal.h"
#include "kv4.cuh"
#include "ptx.cuh"
#include "tile_math.cuh"

namespace hstu {
namespace {

constexpr int kDecWarps = 4;
constexpr int kEpiWarps = 16;
constexpr int kThreads = 32 * (kDecWarps + kEpiWarps + 1);
constexpr int kHalf = 16384;               // 128 rows x 64 bf16
constexpr int kTile = 2 * kHalf;           // 128 x 128 bf16
constexpr int kRing = 4;                   // key metadata of this many tiles
constexpr int kMaxOrder = 512;             // users ranked by length, at most

constexpr int kOffQ = 0;                   // two candidate tiles
constexpr int kOffK = kOffQ + 2 * kTile;   // two stages
constexpr int kOffV = kOffK + 2 * kTile;
constexpr int kOffPos = kOffV + 2 * kTile;             // float [kRing][128]: half position bias
constexpr int kOffTs = kOffPos + kRing * 128 * 4;      // uint32 [kRing][128]: timestamps, low words
constexpr int kOffThr = kOffTs + kRing * 128 * 4;      // long long [kThrLen]
constexpr int kOffFirst = kOffThr + kThrLen * 8;       // signed char [64]
constexpr int kOffRabH = kOffFirst + 64;               // float [kMaxBuckets]: half time bias
constexpr int kOffOct = kOffRabH + kMaxBuckets * 4;    // uint4 [32]
constexpr int kOffThr32 = kOffOct + 32 * 16;           // unsigned [kMaxBuckets]
constexpr int kOffBar = kOffThr32 + kMaxBuckets * 4;
enum {
  B_QFULL = 0,     // + candidate tile
  B_KFULL = 2,     // + stage
  B_KEMPTY = 4,
  B_VFULL = 6,
  B_VEMPTY = 8,
  B_SFULL = 10,    // + candidate tile
  B_PFULL = 12,
  B_PVDONE = 14,
  B_OFULL = 16,
  B_META = 17,     // + ring slot
  kNumBars = B_META + kRing
};
constexpr int kOffMisc = kOffBar + kNumBars * 8;       // [0] TMEM base, [1] abort, [2] user
constexpr int kSmem = kOffMisc + 16 + 1024;
static_assert(kOffOct % 16 == 0 && kOffBar % 8 == 0 && kOffThr % 8 == 0, "table alignment");
static_assert(kMaxOrder * 4 <= kRing * 128 * 4, "lengths fit the ring");
static_assert(kSmem <= 227 * 1024, "shared memory per CTA");

constexpr uint32_t kIdescS = idesc_bf16_f32(128, 128, false, false);
constexpr uint32_t kIdescPV = idesc_bf16_f32(128, 128, false, true);
constexpr uint32_t kColO = 256;

struct Tab {
  const uint4* oct_;
  const unsigned* thr32_;
  const float* rabh_;
  __device__ __forceinline__ const uint4* oct() const { return oct_; }
  __device__ __forceinline__ const unsigned* thr32() const { return thr32_; }
  __device__ __forceinline__ const float* rabt() const { return rabh_; }
};

__device__ __forceinline__ bool flagged(bool ok, int* status) {
  if (!ok && status) atomicOr(status, kStatusTimeout);
  return ok;
}

// P pairs of one 32-key block from its scores: h = S / 2 + half bias, h + h tanh h.
template <bool POS, int TB>
__device__ __forceinline__ void p_block(const uint32_t (&sv)[32], const float* pos,
                                        const uint32_t* ts32, const float (&tv)[4], const int (&ts)[3],
                                        uint32_t my32, const Tab& tab, uint32_t (&packed)[16]) {
#pragma unroll
  for (int c4 = 0; c4 < 8; ++c4) {
    float4 p4 = make_float4(0.f, 0.f, 0.f, 0.f);
    if (POS) p4 = *reinterpret_cast<const float4*>(pos + 4 * c4);
    const float pv[4] = {p4.x, p4.y, p4.z, p4.w};
    float y[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int c = 4 * c4 + e;
      float h = __uint_as_float(sv[c]);
      if (TB == TB_CONST && !POS) {
        h = fmaf(h, 0.5f, tv[0]);
      } else {
        h = POS ? fmaf(h, 0.5f, pv[e]) : 0.5f * h;
        if (TB == TB_CONST) h += tv[0];
        if (TB == TB_SPLIT) h += c < ts[0] ? tv[0] : tv[1];
        if (TB == TB_MULTI) h += c >= ts[2] ? tv[3] : c >= ts[1] ? tv[2] : c >= ts[0] ? tv[1] : tv[0];
        if (TB == TB_GEN32) {
          const int d = static_cast<int>(ts32[c] - my32);
          h += tab.rabt()[bucket32(static_cast<uint32_t>(d < 0 ? -d : d), tab.oct())];
        }
      }
      y[e] = fmaf(h, tanh_approx(h), h);
    }
    packed[2 * c4] = pack_bf16x2(y[0], y[1]);
    packed[2 * c4 + 1] = pack_bf16x2(y[2], y[3]);
  }
}

// One 16-byte run of codes (a group of 32 dims) to its four 16-byte chunks of
// bf16 in the swizzled tile.  Lanes of the upper half of the head take their
// chunks in another order: eight lanes' stores then fall on distinct banks.
__device__ __forceinline__ void decode_group(uint32_t tile, int row, int t, uint4 code, uint32_t s) {
  const uint32_t s2 = s | (s << 16), m = kv4_m24(s2);
  const bool up = t >= 2;
  const uint32_t w[4] = {up ? code.z : code.x, up ? code.w : code.y, up ? code.x : code.z,
                         up ? code.y : code.w};
  const uint32_t base = tile + (t >> 1) * kHalf + row * 128;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t chunk = 4u * (t & 1) + (static_cast<uint32_t>(i) ^ (up ? 2u : 0u));
    uint4 o;
    o.x = kv4_pair_fma<0>(w[i], s2, m);
    o.y = kv4_pair_fma<1>(w[i], s2, m);
    o.z = kv4_pair_fma<2>(w[i], s2, m);
    o.w = kv4_pair_fma<3>(w[i], s2, m);
    st_shared_v4(base + ((chunk ^ (row & 7u)) << 4), o);
  }
}

}  // namespace

template <bool POS, bool TIME>
__global__ void __launch_bounds__(kThreads, 1)
    hstu_cand4_sm100(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ Cand4Args a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto bar = [&](int i) { return sbase + kOffBar + 8u * i; };
  uint32_t* misc = reinterpret_cast<uint32_t*>(smem + kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + 1);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // (candidate batch, split, head, rank of the user), batches fastest: the
  // batches of one (user, head) share its cache rows in L2; long histories first
  unsigned x = blockIdx.x;
  const unsigned batches = (static_cast<unsigned>(a.max_cands) + 255u) / 256u;
  const int mb = static_cast<int>(x % batches);
  x /= batches;
  const int split = static_cast<int>(x % static_cast<unsigned>(a.splits));
  x /= static_cast<unsigned>(a.splits);
  const int h = static_cast<int>(x % static_cast<unsigned>(a.H));
  const int rank = static_cast<int>(x / static_cast<unsigned>(a.H));
  int b = rank;
  if (a.B > 1 && a.B <= kMaxOrder) {
    // the user of this rank (ties by index): every thread ranks one user
    int* len = reinterpret_cast<int*>(smem + kOffPos);   // before its ring is in use
    for (int i = threadIdx.x; i < a.B; i += kThreads)
      len[i] = __ldg(a.offsets + i + 1) - __ldg(a.offsets + i);
    if (threadIdx.x == 0) misc[2] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < a.B; i += kThreads) {
      const int n = len[i];
      int r = 0;
      for (int o = 0; o < a.B; ++o) r += (len[o] > n || (len[o] == n && o < i)) ? 1 : 0;
      if (r == rank) misc[2] = static_cast<uint32_t>(i);
    }
    __syncthreads();
    b = static_cast<int>(misc[2]);
  }
  const int c0 = __ldg(a.cand_offsets + b);
  const int cb = __ldg(a.cand_offsets + b + 1) - c0;
  const int s = __ldg(a.offsets + b);
  const int nb = __ldg(a.offsets + b + 1) - s;
  const int r0 = a.first_rows ? __ldg(a.first_rows + b) : s;
  if (c0 < 0 || cb < 0 || cb > a.C - c0 || cb > a.max_cands || s < 0 || nb < 0 || nb > a.T - s ||
      nb > a.max_seq_len || r0 < 0 || nb > a.R - r0 || (POS && nb >= a.L)) {
    if (threadIdx.x == 0 && a.status) atomicOr(a.status, kStatusBadOffsets);
    return;
  }
  const int key0 = split * a.chunk;
  const int keys = min(nb - key0, a.chunk);              // this CTA's
  const int rows = min(cb - 256 * mb, 256);
  if (rows <= 0 || keys <= 0) return;
  const int cand0 = c0 + 256 * mb;
  const int nt = (keys + 127) / 128;
  const int tiles = rows > 128 ? 2 : 1;                  // candidate tiles

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(B_QFULL + i), 1);
      mbar_init(bar(B_KFULL + i), kDecWarps);
      mbar_init(bar(B_KEMPTY + i), 1);
      mbar_init(bar(B_VFULL + i), kDecWarps);
      mbar_init(bar(B_VEMPTY + i), 1);
      mbar_init(bar(B_SFULL + i), 1);
      mbar_init(bar(B_PFULL + i), kEpiWarps / 2);
      mbar_init(bar(B_PVDONE + i), 1);
    }
    mbar_init(bar(B_OFULL), 1);
    for (int i = 0; i < kRing; ++i) mbar_init(bar(B_META + i), kDecWarps);
    *abort_flag = 0;
    fence_mbar_init();
  }
  long long* s_thr = reinterpret_cast<long long*>(smem + kOffThr);
  signed char* s_first = reinterpret_cast<signed char*>(smem + kOffFirst);
  Tab tab;
  tab.oct_ = reinterpret_cast<const uint4*>(smem + kOffOct);
  tab.thr32_ = reinterpret_cast<const unsigned*>(smem + kOffThr32);
  tab.rabh_ = reinterpret_cast<const float*>(smem + kOffRabH);
  if (TIME) {
    for (int i = threadIdx.x; i < kThrLen; i += kThreads) s_thr[i] = a.bt.thr[i];
    for (int i = threadIdx.x; i < 64; i += kThreads) s_first[i] = a.bt.first_k[i];
    for (int i = threadIdx.x; i < kMaxBuckets; i += kThreads)
      reinterpret_cast<float*>(smem + kOffRabH)[i] =
          i < a.nb ? 0.5f * __ldg(a.rab_time + h * a.nb + i) : 0.f;
    for (int i = threadIdx.x; i < 32; i += kThreads)
      reinterpret_cast<uint4*>(smem + kOffOct)[i] = a.bt.oct[i];
    for (int i = threadIdx.x; i < kMaxBuckets; i += kThreads)
      reinterpret_cast<unsigned*>(smem + kOffThr32)[i] = a.bt.thr32[i];
  }
  if (warp == kDecWarps + kEpiWarps) {
    tmem_alloc(sbase + kOffMisc, 512);
    tmem_relinquish();
    if (lane == 0) tma_prefetch_desc(&tm_q);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = misc[0];

  if (warp < kDecWarps) {
    // ------------------------------------------------------------ decode
    // lane (row, t): the row's dims 32t..32t+31; rows warp 8 + 32 i + row
    const int t = lane & 3, row = 8 * warp + (lane >> 2);
    const float* rpos =
        POS ? a.rab_pos + static_cast<size_t>(h) * (2 * static_cast<size_t>(a.L) - 1) + (a.L - 1) : nullptr;
    struct Regs {
      uint4 c[4];
      uint32_t s[4];
    } k, v;
    float pos = 0.f;
    uint32_t ts = 0;
    auto load = [&](const uint8_t* codes, const uint16_t* scales, int n, Regs& r) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int key = 128 * n + 32 * i + row;
        r.c[i] = make_uint4(0u, 0u, 0u, 0u);      // keys past the CTA's decode to zeros
        r.s[i] = 0u;
        if (key < keys) {
          const size_t at =
              static_cast<size_t>(checked(a.status, r0 + key0 + key, a.R, BS_CAND4_KEY)) * a.H + h;
          r.c[i] = __ldg(reinterpret_cast<const uint4*>(codes + at * 64) + t);
          r.s[i] = __ldg(scales + at * 4 + t);
        }
      }
    };
    auto load_meta = [&](int n) {
      const int key = 128 * n + 32 * warp + lane;
      const bool in = key < keys;
      if (POS) pos = in ? 0.5f * __ldg(rpos + (nb - key0 - key)) : 0.f;
      if (TIME)
        ts = static_cast<uint32_t>(__ldg(
            a.timestamps + checked(a.status, s + key0 + min(key, keys - 1), a.T, BS_CAND4_TS)));
    };
    load(a.k_codes, a.k_scales, 0, k);
    load_meta(0);
    load(a.v_codes, a.v_scales, 0, v);
    bool ok = true;
    for (int n = 0; n < nt; ++n) {
      const int st = n & 1, use = n >> 1;
      if (use > 0) ok = flagged(mbar_wait(bar(B_KEMPTY + st), (use - 1) & 1, abort_flag), a.status);
      if (!__all_sync(0xffffffffu, ok)) break;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        decode_group(sbase + kOffK + st * kTile, row + 32 * i, t, k.c[i], k.s[i]);
      // this slot's last readers finished tile n - kRing before S of tile n - 2
      // could be issued, which the wait above saw completed
      if (POS) reinterpret_cast<float*>(smem + kOffPos)[(n & (kRing - 1)) * 128 + 32 * warp + lane] = pos;
      if (TIME) reinterpret_cast<uint32_t*>(smem + kOffTs)[(n & (kRing - 1)) * 128 + 32 * warp + lane] = ts;
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(bar(B_KFULL + st));
        mbar_arrive(bar(B_META + (n & (kRing - 1))));
      }
      if (n + 1 < nt) {
        load(a.k_codes, a.k_scales, n + 1, k);
        load_meta(n + 1);
      }
      if (use > 0) ok = flagged(mbar_wait(bar(B_VEMPTY + st), (use - 1) & 1, abort_flag), a.status);
      if (!__all_sync(0xffffffffu, ok)) break;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        decode_group(sbase + kOffV + st * kTile, row + 32 * i, t, v.c[i], v.s[i]);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(B_VFULL + st));
      if (n + 1 < nt) load(a.v_codes, a.v_scales, n + 1, v);
    }
    if (!ok) *abort_flag = 1;
  } else if (warp == kDecWarps + kEpiWarps) {
    // ------------------------------------------------------------ Q and the MMAs
    if (lane == 0) {
      for (int g = 0; g < tiles; ++g) {
        const int qrow = checked(a.status, cand0 + 128 * g, a.C, BS_CAND4_ROW);
        mbar_arrive_expect_tx(bar(B_QFULL + g), kTile);
        tma_load_3d(sbase + kOffQ + g * kTile, &tm_q, bar(B_QFULL + g), 0, h, qrow);
        tma_load_3d(sbase + kOffQ + g * kTile + kHalf, &tm_q, bar(B_QFULL + g), 64, h, qrow);
      }
      bool ok = true;
      auto wait = [&](int i, int parity) {
        ok = ok && flagged(mbar_wait(bar(i), parity & 1, abort_flag), a.status);
      };
      // S of candidate tile g and key tile n; its columns hold P of tile n - 1
      // until that tile's P V is done
      auto issue_s = [&](int g, int n) {
        const int st = n & 1;
        if (n == 0) wait(B_QFULL + g, 0);
        wait(B_KFULL + st, n >> 1);
        if (n > 0) wait(B_PVDONE + g, n - 1);
        if (!ok) return;
        tc_fence_after();
        const uint32_t qa = sbase + kOffQ + g * kTile, ka = sbase + kOffK + st * kTile;
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) {
          const uint32_t off = (ks >> 2) * kHalf + (ks & 3) * 32;
          mma_ss(tmem + 128u * g, sw128_desc(qa + off, 16, 1024), sw128_desc(ka + off, 16, 1024),
                 kIdescS, ks > 0 ? 1u : 0u);
        }
        if (g == tiles - 1) mma_commit(bar(B_KEMPTY + st));
        mma_commit(bar(B_SFULL + g));
      };
      for (int g = 0; g < tiles; ++g) issue_s(g, 0);
      for (int n = 0; n < nt && ok; ++n) {
        const int st = n & 1;
        for (int g = 0; g < tiles && ok; ++g) {
          wait(B_VFULL + st, n >> 1);
          wait(B_PFULL + g, n);
          if (!ok) break;
          tc_fence_after();
          const uint32_t va = sbase + kOffV + st * kTile;
#pragma unroll
          for (int ks = 0; ks < 8; ++ks)
            // keys 16ks..16ks+15: P of a 32-column block sits in its first 16 columns
            mma_ts(tmem + kColO + 128u * g, tmem + 128u * g + 32u * (ks >> 1) + 8u * (ks & 1),
                   sw128_desc(va + ks * 2048, kHalf, 1024), kIdescPV, (n > 0 || ks > 0) ? 1u : 0u);
          if (g == tiles - 1) mma_commit(bar(B_VEMPTY + st));
          mma_commit(bar(B_PVDONE + g));
          if (n + 1 < nt) issue_s(g, n + 1);
        }
      }
      if (!ok) {
        *abort_flag = 1;
        // the copies of Q land before shared memory is released
        for (int g = 0; g < tiles; ++g) mbar_wait(bar(B_QFULL + g), 0, nullptr);
      }
      mma_commit(bar(B_OFULL));
      // TMEM is released only after every MMA issued here has completed.
      mbar_wait(bar(B_OFULL), 0, nullptr);
    }
  } else {
    // ------------------------------------------------------------ epilogue
    const int e = warp - kDecWarps;
    const int g = e >> 3, half = (e >> 2) & 1, q4 = warp & 3;
    const int r = 128 * g + 32 * q4 + lane;
    const bool row_ok = r < rows;
    const bool live = 128 * g + 32 * q4 < rows;    // the warp has candidates
    // rows past the last candidate repeat it, so that a warp's plans are of one kind
    const int cand = cand0 + min(r, rows - 1);
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>(32 * q4) << 16);
    const uint32_t saddr = lane_addr + 128u * g + 64u * half;
    const long long my_ts =
        TIME ? __ldg(a.cand_ts + checked(a.status, cand, a.C, BS_CAND4_ROW)) : 0ll;
    const uint32_t* plan = TIME ? a.plan + static_cast<size_t>(key0 / 32 + 2 * half) * a.C + cand : nullptr;
    auto plan_of = [&](int n, int cc) {
      return (TIME && 128 * n + 64 * half + 32 * cc < keys)
                 ? __ldg(plan + static_cast<size_t>(4 * n + cc) * a.C) : 0u;
    };
    uint32_t pw[2] = {0u, 0u};
    if (live) {
      pw[0] = plan_of(0, 0);
      pw[1] = plan_of(0, 1);
    }
    bool ok = true;
    for (int n = 0; n < nt && g < tiles; ++n) {
      const int slot = n & (kRing - 1);
      ok = flagged(mbar_wait(bar(B_SFULL + g), n & 1, abort_flag), a.status) &&
           flagged(mbar_wait(bar(B_META + slot), (n / kRing) & 1, abort_flag), a.status);
      ok = __all_sync(0xffffffffu, ok);   // the TMEM accesses below are warp-collective
      if (!ok) break;
      tc_fence_after();
      if (live) {
        uint32_t nw[2] = {0u, 0u};
        if (n + 1 < nt) {
          nw[0] = plan_of(n + 1, 0);
          nw[1] = plan_of(n + 1, 1);
        }
#pragma unroll 1
        for (int cc = 0; cc < 2; ++cc) {
          uint32_t sv[32];
          tmem_ld32_nowait(saddr + 32u * cc, sv);
          const int col = 64 * half + 32 * cc;           // first column of the tile
          const int valid = keys - (128 * n + col);      // keys of this block
          const float* pos = reinterpret_cast<const float*>(smem + kOffPos) + slot * 128 + col;
          const uint32_t* ts32 = reinterpret_cast<const uint32_t*>(smem + kOffTs) + slot * 128 + col;
          TimePlan tp{};
          float tv[4] = {0.f, 0.f, 0.f, 0.f};
          int tb = TB_NONE;
          if (TIME && valid > 0) {
            tb = plan_unword(tp, cc ? pw[1] : pw[0]);
            if (tb >= TB_CONST && tb <= TB_MULTI) {
              const int last = tb == TB_CONST ? 0 : tb == TB_SPLIT ? 1 : 3;
#pragma unroll
              for (int i = 0; i < 4; ++i) tv[i] = tab.rabt()[max(tp.k_a - min(i, last), 0)];
            }
          }
          tmem_wait_ld_dep(sv);
          uint32_t packed[16];
          if (valid <= 0) {
#pragma unroll
            for (int i = 0; i < 16; ++i) packed[i] = 0u;
          } else {
            const uint32_t my32 = static_cast<uint32_t>(my_ts);
            if (!TIME || tb == TB_NONE) {
              p_block<POS, TB_NONE>(sv, pos, ts32, tv, tp.s, my32, tab, packed);
            } else if (tb == TB_CONST) {
              p_block<POS, TB_CONST>(sv, pos, ts32, tv, tp.s, my32, tab, packed);
            } else if (tb == TB_SPLIT) {
              p_block<POS, TB_SPLIT>(sv, pos, ts32, tv, tp.s, my32, tab, packed);
            } else if (tb == TB_MULTI) {
              p_block<POS, TB_MULTI>(sv, pos, ts32, tv, tp.s, my32, tab, packed);
            } else if (tb == TB_GEN32) {
              p_block<POS, TB_GEN32>(sv, pos, ts32, tv, tp.s, my32, tab, packed);
            } else {
              // time spans of 2^31 or more: the 64-bit bucket search per element
#pragma unroll
              for (int c = 0; c < 32; c += 2) {
                float y[2];
#pragma unroll
                for (int f = 0; f < 2; ++f) {
                  const int key = min(key0 + 128 * n + col + c + f, nb - 1);
                  const long long kt =
                      __ldg(a.timestamps + checked(a.status, s + key, a.T, BS_CAND4_TS));
                  float hx = POS ? fmaf(__uint_as_float(sv[c + f]), 0.5f, pos[c + f])
                                 : 0.5f * __uint_as_float(sv[c + f]);
                  hx += tab.rabt()[time_bucket(my_ts - kt, s_thr, s_first)];
                  y[f] = fmaf(hx, tanh_approx(hx), hx);
                }
                packed[c / 2] = pack_bf16x2(y[0], y[1]);
              }
            }
            if (valid < 32) {
              // keys past the CTA's last weigh exactly 0
#pragma unroll
              for (int i = 0; i < 16; ++i)
                packed[i] &= (2 * i < valid ? 0x0000FFFFu : 0u) | (2 * i + 1 < valid ? 0xFFFF0000u : 0u);
            }
          }
          tmem_st16(saddr + 32u * cc, packed);   // over this warp's own S columns, already read
        }
        pw[0] = nw[0];
        pw[1] = nw[1];
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(B_PFULL + g));
    }
    if (ok) ok = flagged(mbar_wait(bar(B_OFULL), 0, abort_flag), a.status);
    ok = __all_sync(0xffffffffu, ok) && !*abort_flag;
    if (!ok && lane == 0) *abort_flag = 1;
    if (ok && live) {
      tc_fence_after();
      const size_t D = static_cast<size_t>(a.H) * 128;
      float* dst = a.part + (static_cast<size_t>(split) * a.C + cand) * D + h * 128 + 64 * half;
#pragma unroll 1
      for (int cc = 0; cc < 2; ++cc) {
        uint32_t ov[32];
        tmem_ld32_nowait(lane_addr + kColO + 128u * g + 64u * half + 32u * cc, ov);
        tmem_wait_ld_dep(ov);
        if (row_ok) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            reinterpret_cast<float4*>(dst + 32 * cc)[i] =
                make_float4(__uint_as_float(ov[4 * i]), __uint_as_float(ov[4 * i + 1]),
                            __uint_as_float(ov[4 * i + 2]), __uint_as_float(ov[4 * i + 3]));
        }
      }
    }
    tc_fence_before();
  }
  __syncthreads();
  if (warp == kDecWarps + kEpiWarps) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <bool POS, bool TIME>
cudaError_t launch_t(const Cand4Args& a, const CUtensorMap& tq, cudaStream_t stream) {
  static std::atomic<bool> configured[64];   // per device: shared-memory opt-in done
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev < 0 || dev >= 64 || !configured[dev].load(std::memory_order_acquire)) {
    err = cudaFuncSetAttribute(hstu_cand4_sm100<POS, TIME>,
                               cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (err != cudaSuccess) return err;
    if (dev >= 0 && dev < 64) configured[dev].store(true, std::memory_order_release);
  }
  const unsigned grid = static_cast<unsigned>((a.max_cands + 255) / 256) *
                        static_cast<unsigned>(a.splits) * static_cast<unsigned>(a.H) *
                        static_cast<unsigned>(a.B);
  hstu_cand4_sm100<POS, TIME><<<grid, kThreads, kSmem, stream>>>(tq, a);
  return cudaGetLastError();
}

cudaError_t launch_cand4_sm100(const Cand4Args& a, const CUtensorMap& tq, cudaStream_t stream) {
  const bool pos = a.rab_pos != nullptr, time = a.rab_time != nullptr;
  if (pos && time) return launch_t<true, true>(a, tq, stream);
  if (pos) return launch_t<true, false>(a, tq, stream);
  if (time) return launch_t<false, true>(a, tq, stream);
  return launch_t<false, false>(a, tq, stream);
}

}  // namespace hstu
