// cand4_sm100.cu -- candidate scoring against histories in a 4-bit cache, the
// form for many candidates: tcgen05 products over tiles decoded in shared
// memory.  cand4_few.cu states the operation; the sums that leave here are
// finished by the same last kernel.
//
// A CTA takes (user, 256 candidates, head, up to `chunk` keys): two tiles of
// 128 candidates share every decoded tile of 128 keys and values, which halves
// the decoding, and fill TMEM: S0, S1, O0, O1 at 128 columns each.
//   warps 0..3    decode K (warps 4..7: V): codes and scales from the cache, a
//                 tile ahead in registers, to bf16 in the 128-byte-swizzled
//                 layout of the MMA operands, two stages each; the keys'
//                 position bias and timestamps beside K
//   warps 8..15   epilogue, four per candidate tile, a row (TMEM lane) per
//                 thread: half bias and SiLU in fp32, P (bf16, its one
//                 rounding) over S in TMEM; then O
//   warp 16       TMEM, the candidates' Q by TMA, and every MMA: while one
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

constexpr int kDecWarps = 4;               // of K, and as many of V
constexpr int kEpi0 = 2 * kDecWarps;       // first epilogue warp
constexpr int kEpiWarps = 8;
constexpr int kMmaWarp = kEpi0 + kEpiWarps;
constexpr int kThreads = 32 * (kMmaWarp + 1);
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
// tv, ts: the plan's half biases and split columns (tile_math.cuh).
template <bool POS, int TB>
__device__ __forceinline__ void p_block(const uint32_t (&sv)[32], const float* pos,
                                        const uint32_t* ts32, const float (&tv)[4], const int (&ts)[3],
                                        uint32_t my32, const Tab& tab, uint32_t (&packed)[16]) {
  const uint64_t half2 = pack_f32x2(0.5f, 0.5f), tc2 = pack_f32x2(tv[0], tv[0]);
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const uint64_t s2 = pack_f32x2(__uint_as_float(sv[2 * i]), __uint_as_float(sv[2 * i + 1]));
    uint64_t h2;
    if (POS) {
      h2 = ffma2(s2, half2, *reinterpret_cast<const uint64_t*>(pos + 2 * i));
      if (TB == TB_CONST) h2 = fadd2(h2, tc2);
    } else {
      h2 = ffma2(s2, half2, TB == TB_CONST ? tc2 : 0ull);
    }
    if (TB == TB_SPLIT || TB == TB_MULTI || TB == TB_GEN32) {
      float b[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int c = 2 * i + e;
        if (TB == TB_SPLIT) b[e] = c < ts[0] ? tv[0] : tv[1];
        if (TB == TB_MULTI) b[e] = c >= ts[2] ? tv[3] : c >= ts[1] ? tv[2] : c >= ts[0] ? tv[1] : tv[0];
        if (TB == TB_GEN32) {
          const int d = static_cast<int>(ts32[c] - my32);
          b[e] = tab.rabt()[bucket32(static_cast<uint32_t>(d < 0 ? -d : d), tab.oct())];
        }
      }
      h2 = fadd2(h2, pack_f32x2(b[0], b[1]));
    }
    const float2 h = unpack_f32x2(h2);
    const float2 y = unpack_f32x2(ffma2(h2, pack_f32x2(tanh_approx(h.x), tanh_approx(h.y)), h2));
    packed[i] = pack_bf16x2(y.x, y.y);
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
  // (broadcast, so that the compiler knows the roles' branches to be warp-uniform)
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);
  const int lane = threadIdx.x & 31;
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
      mbar_init(bar(B_PFULL + i), kEpiWarps / 2);   // the tile's epilogue warps
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
  if (warp == kMmaWarp) {
    tmem_alloc(sbase + kOffMisc, 512);
    tmem_relinquish();
    if (lane == 0) tma_prefetch_desc(&tm_q);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = misc[0];

  if (warp < kEpi0) {
    // ------------------------------------------------------------ decode
    // lane (row, t): the row's dims 32t..32t+31; rows 8 w + 32 i + row of the tile
    const bool is_k = warp < kDecWarps;
    const int w = warp & (kDecWarps - 1), t = lane & 3, row = 8 * w + (lane >> 2);
    const uint8_t* codes = is_k ? a.k_codes : a.v_codes;
    const uint16_t* scales = is_k ? a.k_scales : a.v_scales;
    const uint32_t dst = sbase + (is_k ? kOffK : kOffV);
    const int b_full = is_k ? B_KFULL : B_VFULL, b_empty = is_k ? B_KEMPTY : B_VEMPTY;
    const float* rpos =
        POS ? a.rab_pos + static_cast<size_t>(h) * (2 * static_cast<size_t>(a.L) - 1) + (a.L - 1) : nullptr;
    uint4 c[4];
    uint32_t sc[4];
    float pos = 0.f;
    uint32_t ts = 0;
    auto load = [&](int n) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int key = 128 * n + 32 * i + row;
        c[i] = make_uint4(0u, 0u, 0u, 0u);      // keys past the CTA's decode to zeros
        sc[i] = 0u;
        if (key < keys) {
          const size_t at =
              static_cast<size_t>(checked(a.status, r0 + key0 + key, a.R, BS_CAND4_KEY)) * a.H + h;
          c[i] = __ldg(reinterpret_cast<const uint4*>(codes + at * 64) + t);
          sc[i] = __ldg(scales + at * 4 + t);
        }
      }
      if (is_k) {
        const int key = 128 * n + 32 * w + lane;
        if (POS) pos = key < keys ? __ldg(rpos + (nb - key0 - key)) : 0.f;
        if (TIME)
          ts = static_cast<uint32_t>(__ldg(
              a.timestamps + checked(a.status, s + key0 + min(key, keys - 1), a.T, BS_CAND4_TS)));
      }
    };
    load(0);
    bool ok = true;
    for (int n = 0; n < nt; ++n) {
      const int st = n & 1, use = n >> 1, slot = n & (kRing - 1);
      if (use > 0) ok = flagged(mbar_wait(bar(b_empty + st), (use - 1) & 1, abort_flag), a.status);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
#pragma unroll
      for (int i = 0; i < 4; ++i) decode_group(dst + st * kTile, row + 32 * i, t, c[i], sc[i]);
      if (is_k) {
        // the slot's last readers finished tile n - kRing before S of tile n - 2
        // could be issued, which the wait above saw completed
        if (POS) reinterpret_cast<float*>(smem + kOffPos)[slot * 128 + 32 * w + lane] = 0.5f * pos;
        if (TIME) reinterpret_cast<uint32_t*>(smem + kOffTs)[slot * 128 + 32 * w + lane] = ts;
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(bar(b_full + st));
        if (is_k) mbar_arrive(bar(B_META + slot));
      }
      if (n + 1 < nt) load(n + 1);
    }
    if (!ok) *abort_flag = 1;
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ Q and the MMAs
    // the whole warp walks the schedule; one lane issues
    if (elect_one()) {
      for (int g = 0; g < tiles; ++g) {
        const int qrow = checked(a.status, cand0 + 128 * g, a.C, BS_CAND4_ROW);
        mbar_arrive_expect_tx(bar(B_QFULL + g), kTile);
        tma_load_3d(sbase + kOffQ + g * kTile, &tm_q, bar(B_QFULL + g), 0, h, qrow);
        tma_load_3d(sbase + kOffQ + g * kTile + kHalf, &tm_q, bar(B_QFULL + g), 64, h, qrow);
      }
    }
    __syncwarp();
    bool ok = true;
    auto wait = [&](int i, int parity) {
      if (ok)
        ok = __all_sync(0xffffffffu,
                        flagged(mbar_wait(bar(i), parity & 1, abort_flag), a.status));
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
      if (elect_one()) {
        const uint64_t qd = sw128_desc(sbase + kOffQ + g * kTile, 16, 1024);
        const uint64_t kd = sw128_desc(sbase + kOffK + st * kTile, 16, 1024);
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) {
          const uint32_t off = ((ks >> 2) * kHalf + (ks & 3) * 32) >> 4;
          mma_ss(tmem + 128u * g, qd + off, kd + off, kIdescS, ks > 0 ? 1u : 0u);
        }
        if (g == tiles - 1) mma_commit(bar(B_KEMPTY + st));
        mma_commit(bar(B_SFULL + g));
      }
      __syncwarp();
    };
    for (int g = 0; g < tiles; ++g) issue_s(g, 0);
    for (int n = 0; n < nt && ok; ++n) {
      const int st = n & 1;
      for (int g = 0; g < tiles && ok; ++g) {
        wait(B_VFULL + st, n >> 1);
        wait(B_PFULL + g, n);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          const uint64_t vd = sw128_desc(sbase + kOffV + st * kTile, kHalf, 1024);
#pragma unroll
          for (int ks = 0; ks < 8; ++ks)
            // keys 16ks..16ks+15: P of a 32-column block sits in its first 16 columns
            mma_ts(tmem + kColO + 128u * g, tmem + 128u * g + 32u * (ks >> 1) + 8u * (ks & 1),
                   vd + ks * (2048 >> 4), kIdescPV, (n > 0 || ks > 0) ? 1u : 0u);
          if (g == tiles - 1) mma_commit(bar(B_VEMPTY + st));
          mma_commit(bar(B_PVDONE + g));
        }
        __syncwarp();
        if (n + 1 < nt) issue_s(g, n + 1);
      }
    }
    if (!ok) {
      *abort_flag = 1;
      // the copies of Q land before shared memory is released
      for (int g = 0; g < tiles; ++g) mbar_wait(bar(B_QFULL + g), 0, nullptr);
    }
    if (elect_one()) mma_commit(bar(B_OFULL));
    __syncwarp();
    // TMEM is released only after every MMA issued here has completed.
    mbar_wait(bar(B_OFULL), 0, nullptr);
  } else {
    // ------------------------------------------------------------ epilogue
    const int g = (warp - kEpi0) >> 2, q4 = warp & 3;
    const int r = 128 * g + 32 * q4 + lane;
    const bool row_ok = r < rows;
    const bool live = 128 * g + 32 * q4 < rows;    // the warp has candidates
    // rows past the last candidate repeat it, so that a warp's plans are of one kind
    const int cand = cand0 + min(r, rows - 1);
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>(32 * q4) << 16);
    const uint32_t saddr = lane_addr + 128u * g;
    const long long my_ts =
        TIME ? __ldg(a.cand_ts + checked(a.status, cand, a.C, BS_CAND4_ROW)) : 0ll;
    // this candidate's time plans against tile n's four blocks, loaded a tile ahead
    uint32_t pw[4] = {0u, 0u, 0u, 0u};
    auto load_plans = [&](int n) {
      const uint32_t* p = a.plan + static_cast<size_t>(key0 / 32 + 4 * n) * a.C + cand;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (128 * n + 32 * i < keys) pw[i] = __ldg(p + static_cast<size_t>(i) * a.C);
    };
    if (TIME && live) load_plans(0);
    bool ok = true;
    for (int n = 0; n < nt && g < tiles; ++n) {
      const int slot = n & (kRing - 1);
      ok = flagged(mbar_wait(bar(B_SFULL + g), n & 1, abort_flag), a.status) &&
           flagged(mbar_wait(bar(B_META + slot), (n / kRing) & 1, abort_flag), a.status);
      ok = __all_sync(0xffffffffu, ok);   // the TMEM accesses below are warp-collective
      if (!ok) break;
      tc_fence_after();
      if (live) {
#pragma unroll 1
        for (int cc = 0; cc < 4; ++cc) {
          const int col = 32 * cc;                       // first column of the block
          const int valid = keys - (128 * n + col);      // its keys
          uint32_t packed[16];
          if (valid <= 0) {
#pragma unroll
            for (int i = 0; i < 16; ++i) packed[i] = 0u;
          } else {
            uint32_t sv[32];
            tmem_ld32_nowait(saddr + col, sv);
            const float* pos = reinterpret_cast<const float*>(smem + kOffPos) + slot * 128 + col;
            const uint32_t* ts32 = reinterpret_cast<const uint32_t*>(smem + kOffTs) + slot * 128 + col;
            TimePlan tp{};
            float tv[4] = {0.f, 0.f, 0.f, 0.f};
            int tb = TB_NONE;
            if (TIME) {
              tb = plan_unword(tp, pw[0]);
              // blocks come in order: the next one's word moves up
              pw[0] = pw[1];
              pw[1] = pw[2];
              pw[2] = pw[3];
              tv[0] = tab.rabt()[tp.k_a];
              tv[1] = tab.rabt()[max(tp.k_a - 1, 0)];
            }
            tmem_wait_ld_dep(sv);
            const uint32_t my32 = static_cast<uint32_t>(my_ts);
            if (!TIME || tb == TB_NONE) {
              p_block<POS, TB_NONE>(sv, pos, ts32, tv, tp.s, my32, tab, packed);
            } else if (tb == TB_CONST) {
              p_block<POS, TB_CONST>(sv, pos, ts32, tv, tp.s, my32, tab, packed);
            } else if (tb == TB_SPLIT) {
              p_block<POS, TB_SPLIT>(sv, pos, ts32, tv, tp.s, my32, tab, packed);
            } else if (tb == TB_MULTI) {
              tv[2] = tab.rabt()[max(tp.k_a - 2, 0)];
              tv[3] = tab.rabt()[max(tp.k_a - 3, 0)];
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
          tmem_st16(saddr + col, packed);   // over this row's own S columns, already read
        }
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(B_PFULL + g));
      if (TIME && live && n + 1 < nt) load_plans(n + 1);
    }
    if (ok) ok = flagged(mbar_wait(bar(B_OFULL), 0, abort_flag), a.status);
    ok = __all_sync(0xffffffffu, ok) && !*abort_flag;
    if (!ok && lane == 0) *abort_flag = 1;
    if (ok && live) {
      tc_fence_after();
      const size_t D = static_cast<size_t>(a.H) * 128;
      float* dst = a.part + (static_cast<size_t>(split) * a.C + cand) * D + h * 128;
#pragma unroll 1
      for (int cc = 0; cc < 4; ++cc) {
        uint32_t ov[32];
        tmem_ld32_nowait(lane_addr + kColO + 128u * g + 32u * cc, ov);
        tmem_wait_ld_dep(ov);
        if (row_ok) {
#pragma unroll
          for (int i = 0; i < 4; ++i)   // whole 32-byte sectors
            st_global_v8(dst + 32 * cc + 8 * i, reinterpret_cast<const uint32_t(&)[8]>(ov[8 * i]));
        }
      }
    }
    tc_fence_before();
  }
  __syncthreads();
  if (warp == kMmaWarp) {
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
