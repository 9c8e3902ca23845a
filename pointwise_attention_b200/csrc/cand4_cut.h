// cand4_cut.h -- how candidate scoring against the 4-bit cache is cut into CTAs,
// and the room and rows of its sums in the workspace.  Sizes alone decide; host
// code only, but for the check of a user's rows, and free of CUDA headers.
//
// The sums over (parts of) the histories are rows of H * 128 fp32:
//   few candidates   (piece, candidate i of the user): row piece * max_cands + i,
//                    pieces begin with a CTA's share or with a user;
//   many candidates  (split, candidate): row split * sum_rows + n, the batch's
//                    n-th candidate, counted from cand_offsets[0].  The rows of
//                    q that belong to no user have none, however many they are
//                    (a server's buffer of a fixed size): counted with them, the
//                    splits' rows would not fit the room below.
#pragma once
#include <algorithm>
#include <cstddef>
#include <cstdint>

#ifdef __CUDACC__
#define HSTU_HD __host__ __device__ __forceinline__
#else
#define HSTU_HD inline
#endif

namespace hstu {

constexpr int kCand4FewWarps = 8;     // few: warps of a CTA
constexpr int kCand4MaxShare = 512;   // few: tokens of a CTA's share at most
constexpr int kCand4Near = 4;         // many: key blocks at a history's end with bucket bytes

// More candidates per user than this take the tcgen05 kernel: for 32 users, 8
// heads and 2176 keys, up to 7 candidates take 43 us and up to 15 take 70 us
// with the other, and up to 23 take 150 us there, as much as two passes of the
// other would.
constexpr int kCand4FewMax = 16;

struct Cand4Cut {
  int many;      // the kernel for many candidates: 256 of them, a head a CTA
  int heads;     // few: heads of a CTA, one warp each, times
  int parts;     // few: warps that share a head's keys (many: 1)
  int hgroups;   // CTAs along the heads
  int nt;        // few: groups of 8 candidates of a CTA
  int ctas;      // few: shares of the tokens
  int cgroups;   // many: CTAs along a user's candidates
  int chunk, splits;   // many: history keys per CTA, CTAs along the longest history
};

inline Cand4Cut cand4_cut(int B, int H, int max_seq_len, int max_cands, int total_tokens) {
  Cand4Cut c{};
  c.many = max_cands > kCand4FewMax;
  if (c.many) {
    c.parts = 1;
    c.hgroups = H;
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
  c.heads = H < kCand4FewWarps ? H : kCand4FewWarps;
  c.parts = kCand4FewWarps / c.heads;
  c.hgroups = (H + kCand4FewWarps - 1) / kCand4FewWarps;
  c.nt = max_cands <= 8 ? 1 : 2;
  c.cgroups = 1;
  // two CTAs a SM, or as many as keep the shares at kCand4MaxShare tokens
  const int64_t most = std::min(static_cast<int64_t>(B) * max_seq_len,
                                static_cast<int64_t>(total_tokens));
  c.ctas = static_cast<int>(
      std::max<int64_t>(2 * 148 / c.hgroups, (most + kCand4MaxShare - 1) / kCand4MaxShare));
  return c;
}

// Many: rows of one split's sums, the most candidates that B users can have.
inline int cand4_sum_rows(int B, int C, int max_cands) {
  return static_cast<int>(std::min(static_cast<int64_t>(B) * max_cands, static_cast<int64_t>(C)));
}

// Many: whether a user's candidates c0 .. c0 + cb - 1 (0 <= c0, cb) are among
// those rows, cfirst = cand_offsets[0].  Offsets that keep to the sizes always
// are; others are reported.
HSTU_HD bool cand4_in_sums(int c0, int cb, int cfirst, int sum_rows) {
  return cfirst >= 0 && c0 >= cfirst && c0 - cfirst <= sum_rows - cb;
}

// Rows that hold the sums of every cut with H heads, at most B histories of
// max_seq_len and at most C candidates, max_cands a user; it grows with each of
// them.  Few: a row per candidate, part and piece.  Many: splits <=
// max_seq_len / 256 + 1, and splits < 296 / groups + 1 with sum_rows <=
// B * max_cands <= 256 groups / H.
inline size_t cand4_part_rows(int B, int H, int max_seq_len, int C, int max_cands) {
  const int64_t n = max_seq_len, c = cand4_sum_rows(B, C, max_cands);
  const Cand4Cut f = cand4_cut(B, H, max_seq_len, std::min(max_cands, kCand4FewMax), 0x7FFFFFFF);
  const int64_t few = (static_cast<int64_t>(f.ctas) + B) * f.parts * std::min(max_cands, kCand4FewMax);
  const int64_t many = std::min(c * (n / 256 + 1), c + 2 * 148 * 256 / H + 1);
  return static_cast<size_t>(max_cands > kCand4FewMax ? std::max(few, many) : few);
}

// Many, with a time table: Cand4Args::plan and, behind it, Cand4Args::near.
inline size_t cand4_near_offset(int max_seq_len, int C) {
  return ((static_cast<size_t>(max_seq_len) + 31) / 32 * 4 * C + 255) / 256 * 256;
}
inline size_t cand4_plan_bytes(int max_seq_len, int C, int max_cands) {
  return max_cands > kCand4FewMax
             ? cand4_near_offset(max_seq_len, C) + static_cast<size_t>(C) * 32 * kCand4Near
             : 0;
}

}  // namespace hstu
