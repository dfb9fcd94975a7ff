// kv_query.h -- what the kernels that take queries to the cache share (kv_attention.hip, kv_weigh.hip): a
// call's rows, keys and work as the device sees them, rotated queries as fp16 operands and codes
// converted to fp16 in the same order. Device code only; each translation unit gets its own copy.
#pragma once
#include "kv_common.h"

namespace convrot {
namespace {

using namespace kv;

__device__ __forceinline__ uint32_t add_h2(uint32_t a, float off) {
  const f16x2 d = {static_cast<_Float16>(off), static_cast<_Float16>(off)};
  return __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, a) + d);
}

// 4-bit codes of a dword as fp16: nibbles (0, 4), (1, 5), (2, 6), (3, 7). The nibble with its
// sign bit flipped, c + 8, goes into the mantissa of 1024 (low nibbles) or of 64 (high ones).
__device__ __forceinline__ void nibbles_f16(uint32_t x, uint32_t (&h)[4]) {
  h[0] = add_h2((x & 0x000F000Fu) ^ 0x64086408u, -1032.0f);
  h[1] = add_h2((x & 0x00F000F0u) ^ 0x54805480u, -72.0f);
  x >>= 8;
  h[2] = add_h2((x & 0x000F000Fu) ^ 0x64086408u, -1032.0f);
  h[3] = add_h2((x & 0x00F000F0u) ^ 0x54805480u, -72.0f);
}

// 8-bit codes of a dword as fp16: bytes (0, 2), (1, 3), as mantissas of 1024 + (c + 128).
__device__ __forceinline__ void bytes_f16(uint32_t x, uint32_t (&h)[2]) {
  x ^= 0x80808080u;
  h[0] = add_h2(__builtin_amdgcn_perm(0x64646464u, x, 0x04020400u), -1152.0f);
  h[1] = add_h2(__builtin_amdgcn_perm(0x64646464u, x, 0x04030401u), -1152.0f);
}

__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
  const f16x2 h = {static_cast<_Float16>(a), static_cast<_Float16>(b)};
  return __builtin_bit_cast(uint32_t, h);
}

// What the fp16 pair `h` leaves of (a, b), as fp16.
__device__ __forceinline__ uint32_t rest_f16(uint32_t h, float a, float b) {
  const f16x2 f = __builtin_bit_cast(f16x2, h);
  return pack_f16(a - static_cast<float>(f[0]), b - static_cast<float>(f[1]));
}

__device__ __forceinline__ f32x4 mfma(const u32x4& a, const u32x4& b, const f32x4& c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// The power of two for a query row whose largest rotated element is `top`: 2^(8 - exponent), the
// largest comes to lie in [256, 512). Rows of zeros, and largest elements below 2^-100, get 2^108.
__device__ __forceinline__ float query_scale(float top) {
  int e = static_cast<int>(__float_as_uint(top) >> 23) - 127;
  e = e < -100 ? -100 : e;
  return __uint_as_float(static_cast<uint32_t>(127 + 8 - e) << 23);
}

// 8 elements of a rotated query, times `up`, as fp16 pairs in the order in which nibbles_f16 /
// bytes_f16 give the codes; `rest`: what that rounding leaves, as fp16.
template <int BITS>
__device__ __forceinline__ void query_words(const float (&v)[8], float up, bool rest, uint32_t (&w)[4]) {
  constexpr int kA[4] = {0, 1, BITS == 4 ? 2 : 4, BITS == 4 ? 3 : 5};
  constexpr int kB = BITS == 4 ? 4 : 2;
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const float a = v[kA[i]] * up, b = v[kA[i] + kB] * up;
    w[i] = pack_f16(a, b);
    if (rest) w[i] = rest_f16(w[i], a, b);
  }
}

typedef const __attribute__((address_space(4))) int32_t* ConstTable;   // read through the scalar cache
__device__ __forceinline__ ConstTable const_table(const int32_t* p) { return (ConstTable)(uintptr_t)p; }

// Row n of a sequence's (token, head of the group) rows, n < 2^31: its token.
__device__ __forceinline__ int token_of(const KvAttentionArgs& a, int n) {
  return static_cast<int>((__umulhi(static_cast<uint32_t>(n), a.group_mul) + static_cast<uint32_t>(n)) >> a.group_shift);
}

// A sequence's rows and keys as the device sees them, whatever the tables hold: rows lie in
// [0, total_q), keys in the sequence's page table.
struct Seq {
  int q0, q_len, kv_len;
};
__device__ __forceinline__ int clamp(int x, int most) { return x < 0 ? 0 : x > most ? most : x; }
__device__ __forceinline__ Seq sequence(const KvAttentionArgs& a, int b) {
  Seq s;
  const int total = static_cast<int>(a.total_q);
  if (a.q_start) {
    const ConstTable t = const_table(a.q_start);
    s.q0 = clamp(t[b], total);
    const int q1 = clamp(t[b + 1], total);
    s.q_len = q1 < s.q0 ? 0 : q1 - s.q0;
  } else {
    s.q0 = b * a.even_q;
    s.q_len = a.even_q;
  }
  s.kv_len = clamp(const_table(a.kv_len)[b], a.max_pages << a.lps);
  return s;
}

// A workgroup's work. Workgroups go to the 8 XCDs in turn; a page's heads lie side by side in
// memory, and heads that walk the same pages at the same time on one XCD share its address
// translations. So the (sequence, split) pairs are dealt to the XCDs and a pair's heads (and row
// tiles) follow each other on its XCD. A short sequence's work lies in its first splits: from
// sequence to sequence the splits are turned by one, or some XCDs would have all of it.
struct Place {
  int split, head, tile, seq;   // seq >= a.seqs: nothing (pairs are padded to whole turns)
};
constexpr uint32_t kXcds = 8;
__device__ __forceinline__ Place place(const KvAttentionArgs& a) {
  const uint32_t inner = (uint32_t)a.heads * a.row_tiles, turn = blockIdx.x / kXcds;
  const uint32_t pair = turn / inner * kXcds + blockIdx.x % kXcds, in = turn % inner;
  Place p;
  p.tile = a.row_tiles == 1 ? 0 : in / a.heads;
  p.head = in - p.tile * a.heads;
  p.seq = a.splits == 1 ? pair : pair / a.splits;
  p.split = a.splits == 1 ? 0 : (pair - p.seq * a.splits + p.seq) % a.splits;
  return p;
}

// The keys [lo, hi) that row r of a sequence attends to.
__device__ __forceinline__ void key_range(const KvAttentionArgs& a, const Seq& s, int token, int& lo, int& hi) {
  hi = s.kv_len;
  lo = 0;
  if (a.causal) {
    const int pos = s.kv_len - s.q_len + token;   // the token's own position, below 0 if it has none
    hi = pos + 1 < 0 ? 0 : pos + 1;
    if (a.window > 0) lo = pos + 1 - a.window < 0 ? 0 : pos + 1 - a.window;
  }
}

template <int D, int BITS>
struct Geometry {
  using R = Row<D, BITS>;
  static constexpr int kLaneBytes = R::kBytes / 4;                           // K (or V) bytes a lane loads of a 16-token step
  static constexpr int kLoad = kLaneBytes < 16 ? kLaneBytes : 16;            // in loads of this many
  static constexpr int kLoads = kLaneBytes / kLoad;
  static constexpr int kWords = kLoad / 4;
  static constexpr int kOps = D / 32;                                        // matrix steps of a q . k
  static constexpr int kTilesD = D / 16;                                     // 16-wide tiles of the output
};

template <int N>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t (&w)[N]) {
  if constexpr (N == 4) {
    const u32x4 x = *reinterpret_cast<const u32x4*>(p);
#pragma unroll
    for (int i = 0; i < 4; i++) w[i] = x[i];
  } else {
    const u32x2 x = *reinterpret_cast<const u32x2*>(p);
    w[0] = x[0];
    w[1] = x[1];
  }
}

// The 8-element chunk of a row that K operand `op` of lane group g holds.
template <int D, int BITS>
__device__ __forceinline__ int operand_chunk(int op, int g) {
  using G = Geometry<D, BITS>;
  constexpr int kPer = G::kLoad / BITS;   // 8-element chunks a load brings to a lane
  return (op / kPer) * (4 * kPer) + g * kPer + op % kPer;
}

}  // namespace
}  // namespace convrot
