// cand4_sm100.cu -- candidate scoring against histories in a 4-bit cache, the
// form for many candidates: tcgen05 products over tiles decoded in shared
// memory.  cand4_few.cu states the operation; the sums that leave here are
// finished by the same last kernel.
//
// An item of work is (user, 256 candidates, head, up to `chunk` keys): two tiles
// of 128 candidates share every decoded tile of 128 keys and values, which
// halves the decoding, and fill TMEM: S0, S1, O0, O1 at 128 columns each.  A CTA
// per SM walks the items, longest histories first, rounds in alternating
// direction (so that each CTA's sum is about the same); the roles run on into
// the next item on their own, so that its first tiles are decoded and
// multiplied while the last one's sums are written (with a CTA per item a fifth
// of the time went to starts and ends).
//   warps 0..3    decode K (warps 4..6: V): codes and scales from the cache, a
//                 tile ahead in registers, to bf16 in the 128-byte-swizzled
//                 layout of the MMA operands, two stages each; the keys'
//                 position bias and timestamps beside K
//   warps 8..15   epilogue, four per candidate tile, a row (TMEM lane) per
//                 thread: half bias and SiLU in fp32, P (bf16, its one
//                 rounding) over S in TMEM; then O
//   warp 7        TMEM, the candidates' Q by TMA, and every MMA: while one
//                 tile's scores are in the epilogue, the tensor core works for
//                 the other
// SiLU(x) = h (1 + tanh h), h = x / 2, with tanh.approx.f32 (one special
// function per score, relative error at most 2^-11: at most |x| 2^-12 in P).
// Every wait is bounded; a wait that runs out sets the timeout bit of the
// status word and the CTA leaves through the same barriers.
//
// Measured on a B200: 512 candidates for each of 32 users, 8 heads, histories of
// 256-4096 tokens, position and time bias, 146 GFLOP: 311 us here; with the plan
// pass (15) and the last kernel (62), which start beside it, 332 to 385 us a call
// by the lengths drawn.  Latency bounds it: a key tile's chain of products, epilogue and
// barriers takes about 5300 cycles where the tensor core needs 2200 and tanh
// 2048.  Half tiles with barriers of their own (64 keys) did not help: their
// MMAs take as long to issue as whole ones.
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

// Sixteen warps, four to a scheduler: one more would cost every thread 32
// registers (a scheduler's share of the register file).
constexpr int kKWarps = 4, kVWarps = 3;    // that decode K and V
constexpr int kMmaWarp = kKWarps + kVWarps;
constexpr int kEpi0 = kMmaWarp + 1;        // first epilogue warp
constexpr int kEpiWarps = 8;
constexpr int kThreads = 32 * (kEpi0 + kEpiWarps);
constexpr int kRuns = 16;                  // a tile's rows in groups of eight
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
constexpr int kOffRabH = kOffFirst + 64;               // float [16][kMaxBuckets]: half time bias
constexpr int kOffOrder = kOffRabH + 16 * kMaxBuckets * 4;   // int [kMaxOrder]: users by length
constexpr int kOffOct = kOffOrder + kMaxOrder * 4;     // uint4 [32]
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
  B_OEMPTY = 17,
  B_END = 18,
  B_META = 19,     // + ring slot
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
template <bool POS, int TB>   // (TB_BYTES: ts32 are the scores' bucket bytes)
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
    if (TB == TB_SPLIT || TB == TB_MULTI || TB == TB_GEN32 || TB == TB_BYTES) {
      float b[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int c = 2 * i + e;
        if (TB == TB_SPLIT) b[e] = c < ts[0] ? tv[0] : tv[1];
        if (TB == TB_MULTI) b[e] = c >= ts[2] ? tv[3] : c >= ts[1] ? tv[2] : c >= ts[0] ? tv[1] : tv[0];
        if (TB == TB_BYTES) b[e] = tab.rabt()[(ts32[c >> 2] >> (8 * (c & 3))) & 0x7Fu];
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

  int* order = reinterpret_cast<int*>(smem + kOffOrder);
  const bool ordered = a.B > 1 && a.B <= kMaxOrder;
  if (ordered) {
    // the users by history length, longest first (ties by index)
    int* len = reinterpret_cast<int*>(smem + kOffPos);   // before its ring is in use
    for (int i = threadIdx.x; i < a.B; i += kThreads) {
      len[i] = __ldg(a.offsets + i + 1) - __ldg(a.offsets + i);
      order[i] = i;   // (in range whatever the offsets are)
    }
    __syncthreads();
    for (int i = threadIdx.x; i < a.B; i += kThreads) {
      const int n = len[i];
      int r = 0;
      for (int o = 0; o < a.B; ++o) r += (len[o] > n || (len[o] == n && o < i)) ? 1 : 0;
      order[r] = i;
    }
  }
  const unsigned batches = (static_cast<unsigned>(a.max_cands) + 255u) / 256u;
  const unsigned items = batches * static_cast<unsigned>(a.splits) * static_cast<unsigned>(a.H) *
                         static_cast<unsigned>(a.B);
  // The CTA's item of each round, and what it is: (candidate batch, split, head,
  // rank of the user), batches fastest: the batches of one (user, head) run at
  // the same time and share its cache rows in L2.
  struct Item {
    int h, c0, cand0, cfirst, rows, s, nb, r0, split, key0, keys, nt, tiles;
  };
  auto item_of = [&](unsigned round, Item& it) {   // false: nothing to do
    const unsigned base = round * gridDim.x;
    unsigned x = base + ((round & 1u) ? gridDim.x - 1u - blockIdx.x : blockIdx.x);
    if (x >= items) return false;
    const int mb = static_cast<int>(x % batches);
    x /= batches;
    it.split = static_cast<int>(x % static_cast<unsigned>(a.splits));
    x /= static_cast<unsigned>(a.splits);
    it.h = static_cast<int>(x % static_cast<unsigned>(a.H));
    const int rank = static_cast<int>(x / static_cast<unsigned>(a.H));
    const int b = ordered ? order[rank] : rank;
    it.cfirst = __ldg(a.cand_offsets);
    it.c0 = __ldg(a.cand_offsets + b);
    const int cb = __ldg(a.cand_offsets + b + 1) - it.c0;
    it.s = __ldg(a.offsets + b);
    it.nb = __ldg(a.offsets + b + 1) - it.s;
    it.r0 = a.first_rows ? __ldg(a.first_rows + b) : it.s;
    // ranges that contradict the sizes are reported by the last kernel
    if (it.c0 < 0 || cb < 0 || cb > a.C - it.c0 || cb > a.max_cands || it.s < 0 || it.nb < 0 ||
        it.nb > a.T - it.s || it.nb > a.max_seq_len || it.r0 < 0 || it.nb > a.R - it.r0 ||
        (POS && it.nb >= a.L) || !cand4_in_sums(it.c0, cb, it.cfirst, a.sum_rows))
      return false;
    it.key0 = it.split * a.chunk;
    it.keys = min(it.nb - it.key0, a.chunk);
    it.rows = min(cb - 256 * mb, 256);
    it.cand0 = it.c0 + 256 * mb;
    it.nt = (it.keys + 127) / 128;
    it.tiles = it.rows > 128 ? 2 : 1;                  // candidate tiles
    return it.rows > 0 && it.keys > 0;
  };
  const unsigned rounds = (items + gridDim.x - 1u) / gridDim.x;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(B_QFULL + i), 1);
      mbar_init(bar(B_KFULL + i), kKWarps);
      mbar_init(bar(B_KEMPTY + i), 1);
      mbar_init(bar(B_VFULL + i), kVWarps);
      mbar_init(bar(B_VEMPTY + i), 1);
      mbar_init(bar(B_SFULL + i), 1);
      mbar_init(bar(B_PFULL + i), kEpiWarps / 2);   // the tile's epilogue warps
      mbar_init(bar(B_PVDONE + i), 1);
    }
    mbar_init(bar(B_OFULL), 1);
    mbar_init(bar(B_OEMPTY), kEpiWarps);
    mbar_init(bar(B_END), 1);
    for (int i = 0; i < kRing; ++i) mbar_init(bar(B_META + i), kKWarps);
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
    for (int i = threadIdx.x; i < a.H * kMaxBuckets; i += kThreads) {
      const int h = i / kMaxBuckets, k = i % kMaxBuckets;
      reinterpret_cast<float*>(smem + kOffRabH)[i] = k < a.nb ? 0.5f * __ldg(a.rab_time + h * a.nb + k) : 0.f;
    }
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

  if (warp < kMmaWarp) {
    // ------------------------------------------------------------ decode
    // lane (row, t): the row's dims 32t..32t+31; rows 8 (w + warps i) + row of
    // the tile
    const bool is_k = warp < kKWarps;
    const int warps = is_k ? kKWarps : kVWarps;
    const int w = is_k ? warp : warp - kKWarps, t = lane & 3, row = 8 * w + (lane >> 2);
    constexpr int kMost = (kRuns + kVWarps - 1) / kVWarps;
    const uint8_t* codes = is_k ? a.k_codes : a.v_codes;
    const uint16_t* scales = is_k ? a.k_scales : a.v_scales;
    const uint32_t dst = sbase + (is_k ? kOffK : kOffV);
    const int b_full = is_k ? B_KFULL : B_VFULL, b_empty = is_k ? B_KEMPTY : B_VEMPTY;
    uint4 c[kMost];
    uint32_t sc[kMost];
    float pos = 0.f;
    uint32_t ts = 0;
    Item it;
    auto load = [&](int n) {
#pragma unroll
      for (int i = 0; i < kMost; ++i) {
        if (w + warps * i >= kRuns) break;
        const int key = 128 * n + 8 * warps * i + row;
        c[i] = make_uint4(0u, 0u, 0u, 0u);      // keys past the item's decode to zeros
        sc[i] = 0u;
        if (key < it.keys) {
          const size_t at =
              static_cast<size_t>(checked(a.status, it.r0 + it.key0 + key, a.R, BS_CAND4_KEY)) * a.H + it.h;
          c[i] = __ldg(reinterpret_cast<const uint4*>(codes + at * 64) + t);
          sc[i] = __ldg(scales + at * 4 + t);
        }
      }
      if (is_k) {
        const int key = 128 * n + 32 * w + lane;
        if (POS) {
          const float* rpos = a.rab_pos + static_cast<size_t>(it.h) * (2 * static_cast<size_t>(a.L) - 1) + (a.L - 1);
          pos = key < it.keys ? __ldg(rpos + (it.nb - it.key0 - key)) : 0.f;
        }
        if (TIME)
          ts = static_cast<uint32_t>(__ldg(
              a.timestamps + checked(a.status, it.s + it.key0 + min(key, it.keys - 1), a.T, BS_CAND4_TS)));
      }
    };
    bool ok = true;
    unsigned tn = 0;      // tiles of all items so far
    for (unsigned round = 0; round < rounds && ok; ++round) {
      if (!item_of(round, it)) continue;
      load(0);
      for (int n = 0; n < it.nt; ++n, ++tn) {
        const unsigned st = tn & 1u, use = tn >> 1, slot = tn & (kRing - 1);
        if (use > 0) ok = flagged(mbar_wait(bar(b_empty + st), (use - 1) & 1, abort_flag), a.status);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
#pragma unroll
        for (int i = 0; i < kMost; ++i) {
          if (w + warps * i >= kRuns) break;
          decode_group(dst + st * kTile, row + 8 * warps * i, t, c[i], sc[i]);
        }
        if (is_k) {
          // the slot's last readers finished tile tn - kRing before S of tile
          // tn - 2 could be issued, which the wait above saw completed
          if (POS) reinterpret_cast<float*>(smem + kOffPos)[slot * 128 + 32 * w + lane] = 0.5f * pos;
          if (TIME) reinterpret_cast<uint32_t*>(smem + kOffTs)[slot * 128 + 32 * w + lane] = ts;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bar(b_full + st));
          if (is_k) mbar_arrive(bar(B_META + slot));
        }
        if (n + 1 < it.nt) load(n + 1);
      }
    }
    if (!ok) *abort_flag = 1;
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ Q and the MMAs
    // the whole warp walks the schedule; one lane issues
    bool ok = true;
    auto wait = [&](int i, unsigned parity) {
      if (ok)
        ok = __all_sync(0xffffffffu,
                        flagged(mbar_wait(bar(i), parity & 1u, abort_flag), a.status));
    };
    // so far: tiles, items, and per candidate tile its Q tiles, S and P V products
    unsigned tn = 0, done = 0, qn[2] = {0u, 0u}, sn[2] = {0u, 0u}, pn[2] = {0u, 0u};
    Item it;
    // S of candidate tile g and the item's key tile n; its columns hold the P
    // of its tile before until that one's P V is done
    auto issue_s = [&](int g, int n) {
      const unsigned st = (tn + n) & 1u;
      if (n == 0) wait(B_QFULL + g, qn[g] - 1);
      wait(B_KFULL + st, (tn + n) >> 1);
      if (sn[g] > 0) wait(B_PVDONE + g, sn[g] - 1);
      if (!ok) return;
      ++sn[g];
      tc_fence_after();
      if (elect_one()) {
        const uint64_t qd = sw128_desc(sbase + kOffQ + g * kTile, 16, 1024);
        const uint64_t kd = sw128_desc(sbase + kOffK + st * kTile, 16, 1024);
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) {
          const uint32_t off = ((ks >> 2) * kHalf + (ks & 3) * 32) >> 4;
          mma_ss(tmem + 128u * g, qd + off, kd + off, kIdescS, ks > 0 ? 1u : 0u);
        }
        if (g == it.tiles - 1) mma_commit(bar(B_KEMPTY + st));
        mma_commit(bar(B_SFULL + g));
      }
      __syncwarp();
    };
    for (unsigned round = 0; round < rounds && ok; ++round) {
      if (!item_of(round, it)) continue;
      // the item before has no S left to compute from its Q
      if (tn > 0) wait(B_KEMPTY + ((tn - 1) & 1u), (tn - 1) >> 1);
      if (!ok) break;
      if (elect_one()) {
        for (int g = 0; g < it.tiles; ++g) {
          const int qrow = checked(a.status, it.cand0 + 128 * g, a.C, BS_CAND4_ROW);
          mbar_arrive_expect_tx(bar(B_QFULL + g), kTile);
          tma_load_3d(sbase + kOffQ + g * kTile, &tm_q, bar(B_QFULL + g), 0, it.h, qrow);
          tma_load_3d(sbase + kOffQ + g * kTile + kHalf, &tm_q, bar(B_QFULL + g), 64, it.h, qrow);
        }
      }
      __syncwarp();
      for (int g = 0; g < it.tiles; ++g) ++qn[g];
      for (int g = 0; g < it.tiles; ++g) issue_s(g, 0);
      for (int n = 0; n < it.nt && ok; ++n) {
        const unsigned st = (tn + n) & 1u;
        for (int g = 0; g < it.tiles && ok; ++g) {
          wait(B_VFULL + st, (tn + n) >> 1);
          wait(B_PFULL + g, pn[g]);
          if (n == 0 && g == 0 && done > 0) wait(B_OEMPTY, done - 1);   // O of the item before is read
          if (!ok) break;
          ++pn[g];
          tc_fence_after();
          if (elect_one()) {
            const uint64_t vd = sw128_desc(sbase + kOffV + st * kTile, kHalf, 1024);
#pragma unroll
            for (int ks = 0; ks < 8; ++ks)
              // keys 16ks..16ks+15: P of a 32-column block sits in its first 16 columns
              mma_ts(tmem + kColO + 128u * g, tmem + 128u * g + 32u * (ks >> 1) + 8u * (ks & 1),
                     vd + ks * (2048 >> 4), kIdescPV, (n > 0 || ks > 0) ? 1u : 0u);
            if (g == it.tiles - 1) mma_commit(bar(B_VEMPTY + st));
            mma_commit(bar(B_PVDONE + g));
            if (n == it.nt - 1 && g == it.tiles - 1) mma_commit(bar(B_OFULL));
          }
          __syncwarp();
          if (n + 1 < it.nt) issue_s(g, n + 1);
        }
      }
      tn += it.nt;
      ++done;
    }
    if (!ok) {
      *abort_flag = 1;
      // the copies of Q land before shared memory is released
      for (int g = 0; g < 2; ++g)
        if (qn[g] > 0) mbar_wait(bar(B_QFULL + g), (qn[g] - 1) & 1u, nullptr);
    }
    if (elect_one()) mma_commit(bar(B_END));
    __syncwarp();
    // TMEM is released only after every MMA issued here has completed.
    mbar_wait(bar(B_END), 0, nullptr);
  } else {
    // ------------------------------------------------------------ epilogue
    const int g = (warp - kEpi0) >> 2, q4 = warp & 3;
    const int r = 128 * g + 32 * q4 + lane;
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>(32 * q4) << 16);
    const uint32_t saddr = lane_addr + 128u * g;
    const size_t D = static_cast<size_t>(a.H) * 128;
    bool ok = true;
    bool round_first = true;
    unsigned tn = 0, done = 0, en = 0;   // tiles and items so far, this candidate tile's S
    for (unsigned round = 0; round < rounds; ++round) {
      // (what the tiles need of the item; the rest is looked up again, so that
      // it holds no registers meanwhile)
      int keys, nt, cand, rows, tiles, near0;
      const uint32_t* plan = nullptr;
      {
        Item it;
        if (!item_of(round, it)) continue;
        keys = it.keys;
        nt = it.nt;
        rows = it.rows;
        tiles = it.tiles;
        // rows past the last candidate repeat it, so that a warp's plans are of one kind
        cand = it.cand0 + min(r, it.rows - 1);
        if (TIME) plan = a.plan + static_cast<size_t>(it.key0 / 32) * a.C + cand;
        near0 = (it.nb - it.key0 + 31) / 32 - 1;   // blocks from the item's first to the history's last
        tab.rabh_ = reinterpret_cast<const float*>(smem + kOffRabH) + it.h * kMaxBuckets;
      }
      const bool live = 128 * g + 32 * q4 < rows;    // the warp has candidates
      const uint32_t my32 =
          TIME ? static_cast<uint32_t>(__ldg(a.cand_ts + checked(a.status, cand, a.C, BS_CAND4_ROW))) : 0u;
      // this candidate's time plans against tile n's four blocks, loaded a tile ahead
      uint32_t pw[4] = {0u, 0u, 0u, 0u};
      auto load_plans = [&](int n) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (128 * n + 32 * i < keys) pw[i] = ld_global_u32(plan + static_cast<size_t>(i) * a.C);
        plan += static_cast<size_t>(4) * a.C;
      };
      if (TIME && round_first) {
        // the plan pass, which this kernel is launched beside, is over
        asm volatile("griddepcontrol.wait;" ::: "memory");
        round_first = false;
      }
      if (TIME && live) load_plans(0);
      for (int n = 0; n < nt && g < tiles; ++n) {
        const unsigned slot = (tn + n) & (kRing - 1);
        ok = flagged(mbar_wait(bar(B_SFULL + g), en & 1u, abort_flag), a.status) &&
             flagged(mbar_wait(bar(B_META + slot), ((tn + n) / kRing) & 1u, abort_flag), a.status);
        ok = __all_sync(0xffffffffu, ok);   // the TMEM accesses below are warp-collective
        if (!ok) break;
        ++en;
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
              } else if (tb == TB_GEN32 && near0 - (4 * n + cc) < kCand4Near) {
                const uint4* src = a.near + (static_cast<size_t>(near0 - (4 * n + cc)) * a.C + cand) * 2;
                const uint4 lo = ld_global_v4(src), hi = ld_global_v4(src + 1);
                const uint32_t bytes[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
                p_block<POS, TB_BYTES>(sv, pos, bytes, tv, tp.s, my32, tab, packed);
              } else if (tb == TB_GEN32) {
                p_block<POS, TB_GEN32>(sv, pos, ts32, tv, tp.s, my32, tab, packed);
              } else {
                // time spans of 2^31 or more: the 64-bit bucket search per element
                Item it;
                item_of(round, it);
                const long long my_ts = __ldg(a.cand_ts + cand);
#pragma unroll
                for (int c = 0; c < 32; c += 2) {
                  float y[2];
#pragma unroll
                  for (int f = 0; f < 2; ++f) {
                    const int key = min(it.key0 + 128 * n + col + c + f, it.nb - 1);
                    const long long kt =
                        __ldg(a.timestamps + checked(a.status, it.s + key, a.T, BS_CAND4_TS));
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
      if (ok) ok = flagged(mbar_wait(bar(B_OFULL), done & 1u, abort_flag), a.status);
      ok = __all_sync(0xffffffffu, ok) && !*abort_flag;
      if (!ok) break;
      tn += nt;
      ++done;
      tc_fence_after();
      Item it;
      item_of(round, it);
      const size_t row = checked(a.status, static_cast<size_t>(it.split) * a.sum_rows + (cand - it.cfirst),
                                 a.part_rows, BS_CAND4_SUM);
      float* dst = a.part + row * D + it.h * 128;
#pragma unroll 1
      for (int cc = 0; cc < 4; ++cc) {
        uint32_t ov[32];
        if (live) {
          tmem_ld32_nowait(lane_addr + kColO + 128u * g + 32u * cc, ov);
          tmem_wait_ld_dep(ov);
        }
        if (cc == 3) {
          // O is in registers: the next item's P V may have its columns
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(B_OEMPTY));
        }
        if (live && r < rows) {
#pragma unroll
          for (int i = 0; i < 4; ++i)   // whole 32-byte sectors
            st_global_v8(dst + 32 * cc + 8 * i, reinterpret_cast<const uint32_t(&)[8]>(ov[8 * i]));
        }
      }
    }
    if (!ok && lane == 0) *abort_flag = 1;
    tc_fence_before();
  }
  // (also where a CTA had nothing to score: this kernel ends after the plan pass)
  if (TIME) asm volatile("griddepcontrol.wait;" ::: "memory");
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
  const unsigned items = static_cast<unsigned>((a.max_cands + 255) / 256) *
                         static_cast<unsigned>(a.splits) * static_cast<unsigned>(a.H) *
                         static_cast<unsigned>(a.B);
  const unsigned grid = items < 148u ? items : 148u;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = stream;
  // with a time table: beside the plan pass, which the epilogue waits for (what
  // else is read was there before the plan pass began)
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = TIME ? 1 : 0;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, hstu_cand4_sm100<POS, TIME>, tq, a);
}

cudaError_t launch_cand4_sm100(const Cand4Args& a, const CUtensorMap& tq, cudaStream_t stream) {
  const bool pos = a.rab_pos != nullptr, time = a.rab_time != nullptr;
  if (pos && time) return launch_t<true, true>(a, tq, stream);
  if (pos) return launch_t<true, false>(a, tq, stream);
  if (time) return launch_t<false, true>(a, tq, stream);
  return launch_t<false, false>(a, tq, stream);
}

}  // namespace hstu
