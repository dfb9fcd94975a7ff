// kv_attention.hip -- attention over a cache of rotated 8- or 4-bit keys and values
// (rq_kv_attention; layout and definition in convrot.h).
//
// Mathematics. With R the normalized block rotation, a held key is R^T (s_k c_k) for its codes
// c_k, so q . k = s_k (R q) . c_k: the query is rotated once and the keys are used as codes. The
// output sum_j p_j v_j = R^T (sum_j (p_j s_v,j) c_v,j) is rotated back once. Codes are integers of
// at most 7 bits and a sign, exact in fp16, so both products run on fp16 matrix instructions with
// fp32 sums. Two roundings remain: of R q to fp16 (scaled by a power of two a row so that its
// largest element lies in [256, 512)) and of the weights p_j s_v,j to fp16. For fp16 queries and
// outputs a second fp16 holds what the first leaves of both, and takes a second matrix
// instruction: one rounding to 11 bits beside the output's own would be felt. bf16 has 8.
//
// The running softmax keeps a reference b for each row, not the maximum: a key's logit t (base 2)
// gives p' = 2^(t - b), sums l = sum p', and the weight p' s_v. b is set so that the largest
// weight met is 2^7, whatever share of that is the value's size (a key that takes nearly all of l
// may have a value of next to nothing), and stays until a weight passes 2^15; then b moves and
// what was summed is scaled. So weights down to 2^-21 of the largest are normal fp16 numbers, and
// most tiles only compare. l may be far above 1.
#include "kv_common.h"

namespace convrot {
namespace {

using namespace kv;

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kTop = 7.0f;        // log2 of the largest weight when b is set
constexpr float kMost = 32768.0f;   // weights above this move b
constexpr float kMostExp = 90.0f;   // log2 of the p' that a moved b allows, and the sum that
constexpr float kMostSum = 0x1p120f;   // moves it
constexpr float kNoRef = -3.0e38f;  // b of a row that has met no key
constexpr int kMinChunk = 1024;     // keys
constexpr int kWaves = 4;
constexpr int kRows = 16;          // query rows of a tile: (token, head of the group) pairs

__device__ __forceinline__ float neg_inf() { return -__builtin_inff(); }

// Maximum / sum over the four lanes that hold the same query row (lane xor 16, 32).
__device__ __forceinline__ float quad_max(float x) {
  x = fmaxf(x, __shfl_xor(x, 16, 64));
  return fmaxf(x, __shfl_xor(x, 32, 64));
}
__device__ __forceinline__ float quad_sum(float x) {
  x += __shfl_xor(x, 16, 64);
  return x + __shfl_xor(x, 32, 64);
}

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

// A tile of keys as a wave holds it: STEPS times 16 tokens.
template <int D, int BITS, int STEPS>
struct Tile {
  using G = Geometry<D, BITS>;
  uint32_t k[STEPS][G::kLoads][G::kWords], v[STEPS][G::kLoads][G::kWords];
  float ks, vs;   // scales, spread over a row of 16 lanes: of token 16 (r / 4) + 4 g + r % 4
  uint32_t ok;    // bit j: step j's page is in the cache
};

// The value that lane N of the lane's row of 16 holds (an operand modifier, no instruction).
template <int N>
__device__ __forceinline__ float row_lane(float v) {
  return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0x150 + N, 0xF, 0xF, true));
}
// a[j][i] = b[j][i] times the scale of step j's token 4g + i.
template <int STEPS, int N = 0>
__device__ __forceinline__ void times_scale(float (&a)[STEPS][4], const float (&b)[STEPS][4], float scale) {
  if constexpr (N < 4 * STEPS) {
    a[N / 4][N % 4] = row_lane<N>(scale) * b[N / 4][N % 4];
    times_scale<STEPS, N + 1>(a, b, scale);
  }
}

// Page table entries of a tile's steps, read through the scalar cache. Steps past the table's end
// take its last entry (their tokens are masked: they lie behind kv_len).
template <int STEPS>
struct Pages {
  int at[STEPS];
};
template <int STEPS>
__device__ __forceinline__ Pages<STEPS> tile_pages(const KvAttentionArgs& a, ConstTable table, int tile) {
  Pages<STEPS> p;
#pragma unroll
  for (int j = 0; j < STEPS; j++) {
    const int at = (tile * STEPS + j) * 16 >> a.lps;
    p.at[j] = table[at < a.max_pages ? at : a.max_pages - 1];
  }
  return p;
}

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

// The codes and scales of a tile. Lane (r, g) = (lane % 16, lane / 16) loads, of each 16-token
// step, token r's K bytes (chunk g of every 4 * kLoad) and of the four tokens 4g .. 4g+3 the V
// columns kLoad / 4 * r ..: each load instruction of the wave reads 64 * kLoad contiguous bytes,
// and what arrives is the matrix operand but for the conversion: no exchange between lanes. A page
// index outside the cache loads from page 0; its tokens are masked.
template <int D, int BITS, int STEPS>
__device__ __forceinline__ void load_tile(const KvAttentionArgs& a, const Pages<STEPS>& pages, int head, int tile,
                                          int r, int g, Tile<D, BITS, STEPS>& t) {
  using G = Geometry<D, BITS>;
  using R = Row<D, BITS>;
  const int page = 1 << a.lps;
  const uint32_t k_lane = r * R::kBytes + g * G::kLoad, v_lane = g * (4 * R::kBytes) + r * G::kLoad;
  const int s_step = r >> 2 < STEPS ? r >> 2 : 0;   // with fewer than four steps some lanes repeat
  const uint8_t* s_at = nullptr;
  t.ok = 0;
#pragma unroll
  for (int j = 0; j < STEPS; j++) {
    const int pg = pages.at[j];
    const bool ok = pg >= 0 && pg < a.num_pages;
    t.ok |= ok ? 1u << j : 0u;
    const uint8_t* block = a.cache + ((int64_t)(ok ? pg : 0) * a.heads + head) * a.head_bytes;
    const int off = (tile * STEPS + j) * 16 & (page - 1);
    // One scalar base a step, 32-bit lane offsets.
    const uint32_t kp = off * R::kBytes + k_lane, vp = (page + off) * R::kBytes + v_lane;
    const uint8_t* sp = block + (2 * page * R::kBytes + off * 4);
    s_at = j == 0 || s_step == j ? sp : s_at;
#pragma unroll
    for (int l = 0; l < G::kLoads; l++) {
      load_words(block + (kp + l * 4 * G::kLoad), t.k[j][l]);
      load_words(block + (vp + l * 16 * G::kLoad), t.v[j][l]);
    }
  }
  const uint32_t token = 4 * g + (r & 3);
  t.ks = *reinterpret_cast<const float*>(s_at + token * 4);
  t.vs = *reinterpret_cast<const float*>(s_at + (page + token) * 4);
}

// The 8-element chunk of a row that K operand `op` of lane group g holds.
template <int D, int BITS>
__device__ __forceinline__ int operand_chunk(int op, int g) {
  using G = Geometry<D, BITS>;
  constexpr int kPer = G::kLoad / BITS;   // 8-element chunks a load brings to a lane
  return (op / kPer) * (4 * kPer) + g * kPer + op % kPer;
}

// Column (element) of the output row that accumulator `m`, register i of lane group g holds.
template <int D, int BITS>
__device__ __forceinline__ int output_column(int m, int i, int g) {
  using G = Geometry<D, BITS>;
  const int row = 4 * g + i;
  if constexpr (BITS == 4) {
    const int l = m / (2 * G::kWords), x = m / 2 % G::kWords, e = m % 2;
    return 2 * (l * 16 * G::kWords + G::kWords * row + x) + e;
  } else {
    return (m / G::kWords) * 16 * G::kWords + G::kWords * row + m % G::kWords;
  }
}

// A wave's running softmax over 16 query rows; lane (r, g) holds row r.
template <int D, int BITS>
struct State {
  using G = Geometry<D, BITS>;
  f32x4 o[G::kTilesD];
  float b;   // the row's reference
  float l;   // this lane's part of the row's sum of p'
};

template <int D, int BITS>
__device__ __forceinline__ void start(State<D, BITS>& s) {
#pragma unroll
  for (int m = 0; m < D / 16; m++) s.o[m] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  s.b = kNoRef;
  s.l = 0.0f;
}

template <int D, int BITS, int STEPS, bool SPLIT>
__device__ __forceinline__ void attend_tile(Tile<D, BITS, STEPS>& t, const u32x4 (&q)[D / 32], const u32x4 (&q2)[D / 32],
                                            float c, bool full, int r, int first, int lo, int hi, int kv_len, State<D, BITS>& s) {
  using G = Geometry<D, BITS>;
  float x[STEPS][4], p[STEPS][4], w[STEPS][4];
#pragma unroll
  for (int j = 0; j < STEPS; j++) {
    f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int op = 0; op < G::kOps; op++) {
      u32x4 kop;
      if constexpr (BITS == 4) {
        uint32_t h[4];
        nibbles_f16(t.k[j][op / G::kWords][op % G::kWords], h);
        kop = u32x4{h[0], h[1], h[2], h[3]};
      } else {
        uint32_t h0[2], h1[2];
        bytes_f16(t.k[j][op / 2][op % 2 * 2], h0);
        bytes_f16(t.k[j][op / 2][op % 2 * 2 + 1], h1);
        kop = u32x4{h0[0], h0[1], h1[0], h1[1]};
      }
      if constexpr (SPLIT) acc = mfma(kop, q2[op], acc);
      acc = mfma(kop, q[op], acc);
    }
#pragma unroll
    for (int i = 0; i < 4; i++) x[j][i] = acc[i];
  }
  times_scale<STEPS>(x, x, t.ks);
  if (!full) {   // the same in every lane
    const int mine = first + 16 * (r >> 2) + (r & 3);   // `first` includes 4 g
    const uint32_t step = r >> 2 < STEPS ? r >> 2 : 0;
    t.vs = mine < kv_len && (t.ok >> step & 1u) ? t.vs : 0.0f;
#pragma unroll
    for (int j = 0; j < STEPS; j++) {
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const int key = first + 16 * j + i;
        const int end = t.ok >> j & 1u ? kv_len : 0, own = hi < end ? hi : end;
        x[j][i] = static_cast<uint32_t>(key - lo) < static_cast<uint32_t>(own > lo ? own - lo : 0) ? x[j][i] : neg_inf();
      }
    }
  }
  // Weights for the present b; true if they fit: none above kMost, and no p' so large that l might
  // come near its range's end (a first key's is infinite: b is kNoRef).
  float l;
  auto weigh = [&]() {
    float wtop = 0.0f;
    l = s.l;
#pragma unroll
    for (int j = 0; j < STEPS; j++) {
#pragma unroll
      for (int i = 0; i < 4; i++) {
        p[j][i] = __builtin_amdgcn_exp2f(__builtin_fmaf(x[j][i], c, -s.b));
        l += p[j][i];
      }
    }
    times_scale<STEPS>(w, p, t.vs);
#pragma unroll
    for (int j = 0; j < STEPS; j++) {
#pragma unroll
      for (int i = 0; i < 4; i++) wtop = fmaxf(wtop, w[j][i]);
    }
    return wtop <= kMost && l < kMostSum;
  };
  if (!__all(weigh())) {
    // The logarithm of the tile's largest weight, and its largest logit, over the row's four lanes.
    const float lv = t.vs > 0.0f ? __builtin_amdgcn_logf(t.vs) : neg_inf();
    float one[STEPS][4], wl = neg_inf(), top = neg_inf();
#pragma unroll
    for (int j = 0; j < STEPS; j++) {
#pragma unroll
      for (int i = 0; i < 4; i++) one[j][i] = 1.0f;
    }
    times_scale<STEPS>(p, one, lv);
#pragma unroll
    for (int j = 0; j < STEPS; j++) {
#pragma unroll
      for (int i = 0; i < 4; i++) {
        top = fmaxf(top, x[j][i]);
        wl = fmaxf(wl, __builtin_fmaf(x[j][i], c, p[j][i]));
      }
    }
    wl = quad_max(wl);
    top = quad_max(top) * c;
    const bool moves = wl - s.b > 15.0f || top - s.b > kMostExp;
    const float b = moves ? fmaxf(wl - kTop, top - kMostExp) : s.b;
    const float alpha = __builtin_amdgcn_exp2f(s.b - b);   // 0 for a row that had no reference
    s.b = b;
    s.l *= alpha;
#pragma unroll
    for (int m = 0; m < G::kTilesD; m++) s.o[m] *= alpha;
    weigh();
  }
  s.l = l;
#pragma unroll
  for (int j = 0; j < STEPS; j += 2) {
    const u32x4 hi = {pack_f16(w[j][0], w[j][2]), pack_f16(w[j][1], w[j][3]),
                      pack_f16(w[j + 1][0], w[j + 1][2]), pack_f16(w[j + 1][1], w[j + 1][3])};
    u32x4 rest;
    if constexpr (SPLIT) {
#pragma unroll
      for (int k = 0; k < 2; k++) {
        rest[2 * k] = rest_f16(hi[2 * k], w[j + k][0], w[j + k][2]);
        rest[2 * k + 1] = rest_f16(hi[2 * k + 1], w[j + k][1], w[j + k][3]);
      }
    }
    auto add = [&](int m, const u32x4& vop) {
      if constexpr (SPLIT) s.o[m] = mfma(vop, rest, s.o[m]);
      s.o[m] = mfma(vop, hi, s.o[m]);
    };
#pragma unroll
    for (int l = 0; l < G::kLoads; l++) {
#pragma unroll
      for (int y = 0; y < G::kWords; y++) {
        if constexpr (BITS == 4) {
          uint32_t h0[4], h1[4];
          nibbles_f16(t.v[j][l][y], h0);
          nibbles_f16(t.v[j + 1][l][y], h1);
          const int m = (l * G::kWords + y) * 2;
          add(m, u32x4{h0[0], h0[2], h1[0], h1[2]});
          add(m + 1, u32x4{h0[1], h0[3], h1[1], h1[3]});
        } else {
          uint32_t h0[2], h1[2];
          bytes_f16(t.v[j][l][y], h0);
          bytes_f16(t.v[j + 1][l][y], h1);
          add(l * G::kWords + y, u32x4{h0[0], h0[1], h1[0], h1[1]});
        }
      }
    }
  }
}

// A row's output in the rotated domain, 8 elements a lane and block, rotated back and stored.
template <int D, int BITS>
__device__ __forceinline__ void store_row(uint8_t* p, int dt, float (&v)[Row<D, BITS>::kChunks][8], int c, bool ok) {
  using R = Row<D, BITS>;
#pragma unroll
  for (int b = 0; b < R::kChunks; b++) {
    const float f = wht_block<R::kLanes>(v[b], c) * R::kNorm;
#pragma unroll
    for (int i = 0; i < 8; i++) v[b][i] *= f;
    if (ok) store8(p + (b * 128 + c * 8) * 2, dt, v[b]);
  }
}

// One workgroup: a tile of 16 query rows of one key head and sequence, and one split of its keys.
// The four waves take the split's tiles of keys in turn, each with a softmax of its own; they are
// joined through LDS, and splits through the workspace (kv_join_kernel).
template <int D, int BITS, int STEPS, bool SPLIT>
__global__ __launch_bounds__(kWaves * 64, D == 256 ? 1 : 2) void kv_attend_kernel(KvAttentionArgs a) {
  using R = Row<D, BITS>;
  using G = Geometry<D, BITS>;
  constexpr int kOutPad = 4, kTile = 16 * STEPS;
  __shared__ __attribute__((aligned(16))) float lds_o[kWaves][kRows][D + kOutPad];
  __shared__ float lds_m[kWaves][kRows], lds_l[kWaves][kRows], lds_c[kRows];
  uint32_t* lds_q = reinterpret_cast<uint32_t*>(lds_o);   // [2][kRows][D / 2], before the first key

  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
  const Place at = place(a);
  if (at.seq >= a.seqs) return;
  const int split = at.split, head = at.head, b = at.seq;
  const Seq s = sequence(a, b);
  const int rows = (s.q_len < a.max_q ? s.q_len : a.max_q) * a.group;   // at most 2^30: checked on the host
  const ConstTable table = const_table(a.pages + (int64_t)b * a.max_pages);

  const int tile = at.tile;
  if (tile * kRows >= rows) return;
  // Keys of this tile's rows, and of this lane's row.
  const int row_first = tile * kRows, row_last = (row_first + kRows < rows ? row_first + kRows : rows) - 1;
  int lo, hi, t_lo, t_hi;
  const bool mine = row_first + r < rows;
  key_range(a, s, token_of(a, mine ? row_first + r : row_first), lo, hi);
  if (!mine) hi = lo = 0;
  int full_lo, full_hi;   // every row attends to [full_lo, full_hi)
  key_range(a, s, token_of(a, row_first), t_lo, full_hi);
  key_range(a, s, token_of(a, row_last), full_lo, t_hi);
  const bool whole = row_last - row_first == kRows - 1;
  const int tiles_lo = t_lo / kTile, tiles_hi = (t_hi + kTile - 1) / kTile;
  const int count = tiles_hi > tiles_lo ? tiles_hi - tiles_lo : 0;
  const int share = (count + a.splits - 1) / a.splits, chunk = share > a.chunk / kTile ? share : a.chunk / kTile;
  const int begin = tiles_lo + (split * (int64_t)chunk < count ? split * chunk : count);
  const int end = tiles_lo + (count - (begin - tiles_lo) < chunk ? count : begin - tiles_lo + chunk);
  if (begin >= end) {   // no keys
    const int n = row_first + threadIdx.x / kRows, token = token_of(a, n), qh = head * a.group + n - token * a.group;
    if (n <= row_last) {   // 16 threads a row
      const int64_t out_row = (int64_t)(s.q0 + token) * a.q_heads + qh;
      if (a.splits > 1) {   // all that the join needs to know
        if (r == 0) a.part_stat[(out_row * a.splits + split) * 2] = neg_inf();
      } else {
        uint8_t* p = a.out + ((s.q0 + token) * a.out_token + qh * a.out_head) * 2;
        for (int d = r * 8; d < D; d += 128) *reinterpret_cast<u32x4*>(p + d * 2) = u32x4{0u, 0u, 0u, 0u};
        if (r == 0 && a.lse) a.lse[out_row] = neg_inf();
      }
    }
    return;
  }
  // One tile is in flight while the other is worked on, and the page entries of the one after.
  // Past the end the last tile is loaded again: loads under a condition would have to be waited
  // for as soon as they are issued. The first tile is under way before the queries are.
  int i = begin + wave;
  auto next = [&](int at) { return at + kWaves < end ? at + kWaves : at; };
  // (A wave without tiles loads the last one too, and does not use it.)
  Tile<D, BITS, STEPS> t0, t1;
  Pages<STEPS> pages = tile_pages<STEPS>(a, table, i < end ? i : end - 1);
  load_tile<D, BITS, STEPS>(a, pages, head, i < end ? i : end - 1, r, g, t0);
  int n = next(i);
  pages = tile_pages<STEPS>(a, table, n < end ? n : end - 1);
  // Queries: rotated, scaled, to fp16, in the K operands' element order.
  {
    const int u = threadIdx.x % R::kLanes, chunk = chunk_of_lane(u), row = threadIdx.x / R::kLanes;
    const int n = tile * kRows + row;
    const bool ok = row < kRows && n < rows;
    const int token = ok ? token_of(a, n) : 0, qh = head * a.group + (ok ? n - token * a.group : 0);
    const uint8_t* x = a.q + ((s.q0 + token) * a.q_token + qh * a.q_head) * 2;
    float v[R::kChunks][8], sign = 1.0f, top = 0.0f;
#pragma unroll
    for (int k = 0; k < R::kChunks; k++) load8(x + (k * 128 + chunk * 8) * 2, a.dt, v[k]);
#pragma unroll
    for (int k = 0; k < R::kChunks; k++) {
      sign = wht_block<R::kLanes>(v[k], chunk);
#pragma unroll
      for (int i = 0; i < 8; i++) top = fmaxf(top, fabsf(v[k][i]));
    }
    top = row_max<R::kLanes>(top);
    // 2^(8 - exponent): the largest element comes to lie in [256, 512). Rows of zeros, and
    // largest elements below 2^-100, are scaled by 2^108.
    int e = static_cast<int>(__float_as_uint(top) >> 23) - 127;
    e = e < -100 ? -100 : e;
    const float up = __uint_as_float(static_cast<uint32_t>(127 + 8 - e) << 23);
    if (row < kRows) {
#pragma unroll
      for (int k = 0; k < R::kChunks; k++) {
        float y[8];
        uint32_t hi[8], lo[8];
#pragma unroll
        for (int i = 0; i < 8; i++) {
          y[i] = v[k][i] * (sign * up);
          const _Float16 h = static_cast<_Float16>(y[i]);
          hi[i] = __builtin_bit_cast(uint16_t, h);
          lo[i] = __builtin_bit_cast(uint16_t, static_cast<_Float16>(y[i] - static_cast<float>(h)));
        }
        // Pairs in the order in which nibbles_f16 / bytes_f16 give the codes.
        constexpr int kA[4] = {0, 1, BITS == 4 ? 2 : 4, BITS == 4 ? 3 : 5};
        constexpr int kB = BITS == 4 ? 4 : 2;
        uint32_t* p = lds_q + row * (D / 2) + (k * 16 + chunk) * 4;
#pragma unroll
        for (int i = 0; i < 4; i++) {
          p[i] = hi[kA[i]] | (hi[kA[i] + kB] << 16);
          if constexpr (SPLIT) p[kRows * (D / 2) + i] = lo[kA[i]] | (lo[kA[i] + kB] << 16);
        }
      }
      // Logits in base 2 are t * c, t = sum of fp16 query times code, times the key's scale.
      if (u == 0) lds_c[row] = a.scale * (kLog2e * R::kNorm) / up;
    }
    __syncthreads();
  }
  u32x4 q[G::kOps], q2[G::kOps];
#pragma unroll
  for (int op = 0; op < G::kOps; op++) {
    const uint32_t* p = lds_q + r * (D / 2) + operand_chunk<D, BITS>(op, g) * 4;
    q[op] = *reinterpret_cast<const u32x4*>(p);
    q2[op] = SPLIT ? *reinterpret_cast<const u32x4*>(p + kRows * (D / 2)) : q[op];
  }
  const float c = fmaxf(lds_c[r], 1.1754944e-38f);   // a positive factor keeps masked logits at -inf
  __syncthreads();   // lds_q is read: lds_o may be written

  State<D, BITS> st;
  start(st);
  if (i < end) {
    auto attend = [&](Tile<D, BITS, STEPS>& t, int at) {
      const int first = at * kTile;
      const bool full = whole && t.ok == (1u << STEPS) - 1 && first >= full_lo && first + kTile <= full_hi;
      attend_tile<D, BITS, STEPS, SPLIT>(t, q, q2, c, full, r, first + 4 * g, lo, hi, s.kv_len, st);
    };
    while (true) {
      load_tile<D, BITS, STEPS>(a, pages, head, n, r, g, t1);
      int m = next(n);
      pages = tile_pages<STEPS>(a, table, m);
      attend(t0, i);
      if (n == i) break;
      i = n;
      n = m;
      load_tile<D, BITS, STEPS>(a, pages, head, n, r, g, t0);
      m = next(n);
      pages = tile_pages<STEPS>(a, table, m);
      attend(t1, i);
      if (n == i) break;
      i = n;
      n = m;
    }
  }

  // Join the waves.
  st.l = quad_sum(st.l);
  if (g == 0) {
    lds_m[wave][r] = st.l > 0.0f ? st.b : neg_inf();
    lds_l[wave][r] = st.l;
  }
  __syncthreads();
  float top = lds_m[0][r];
#pragma unroll
  for (int w = 1; w < kWaves; w++) top = fmaxf(top, lds_m[w][r]);
  {
    const float m = lds_m[wave][r];
    const float f = m == neg_inf() ? 0.0f : __builtin_amdgcn_exp2f(m - top);
#pragma unroll
    for (int m16 = 0; m16 < G::kTilesD; m16++) {
#pragma unroll
      for (int i = 0; i < 4; i++) lds_o[wave][r][output_column<D, BITS>(m16, i, g)] = st.o[m16][i] * f;
    }
  }
  __syncthreads();
  {
    const int u = threadIdx.x % R::kLanes, chunk = chunk_of_lane(u), row = threadIdx.x / R::kLanes;
    const int n = tile * kRows + row, rc = row < kRows ? row : kRows - 1;
    const bool ok = row < kRows && n < rows;
    const int token = ok ? token_of(a, n) : 0, qh = head * a.group + (ok ? n - token * a.group : 0);
    float best = neg_inf(), sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kWaves; w++) best = fmaxf(best, lds_m[w][rc]);
#pragma unroll
    for (int w = 0; w < kWaves; w++)
      sum += lds_m[w][rc] == neg_inf() ? 0.0f : lds_l[w][rc] * __builtin_amdgcn_exp2f(lds_m[w][rc] - best);
    float v[R::kChunks][8];
#pragma unroll
    for (int k = 0; k < R::kChunks; k++) {
#pragma unroll
      for (int i = 0; i < 8; i++) {
        float y = 0.0f;
#pragma unroll
        for (int w = 0; w < kWaves; w++) y += lds_o[w][rc][k * 128 + chunk * 8 + i];
        v[k][i] = y;
      }
    }
    const int64_t out_row = (int64_t)(s.q0 + token) * a.q_heads + qh;
    if (a.splits > 1) {
      if (ok) {
        float* p = a.part_out + (out_row * a.splits + split) * D;
#pragma unroll
        for (int k = 0; k < R::kChunks; k++)
          if (best != neg_inf()) store8(reinterpret_cast<uint8_t*>(p + k * 128 + chunk * 8), kF32, v[k]);
        if (u == 0) {
          a.part_stat[(out_row * a.splits + split) * 2] = best;
          a.part_stat[(out_row * a.splits + split) * 2 + 1] = sum;
        }
      }
    } else {
      const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
#pragma unroll
      for (int k = 0; k < R::kChunks; k++) {
#pragma unroll
        for (int i = 0; i < 8; i++) v[k][i] *= inv;
      }
      if (ok && a.lse && u == 0) a.lse[out_row] = sum > 0.0f ? (best + __log2f(sum)) * kLn2 : neg_inf();
      store_row<D, BITS>(a.out + ((s.q0 + token) * a.out_token + qh * a.out_head) * 2, a.dt, v, chunk, ok);
    }
  }
}

// Joins the splits of a row. A workgroup takes one row: its 256 / kLanes groups of lanes take the
// splits in turn, each with a reference of its own, and are joined through LDS by the first.
template <int D, int BITS>
__global__ __launch_bounds__(256) void kv_join_kernel(KvAttentionArgs a) {
  using R = Row<D, BITS>;
  constexpr int kGroups = 256 / R::kLanes;
  __shared__ __attribute__((aligned(16))) float lds_o[kGroups][D + 4];
  __shared__ float lds_b[kGroups], lds_l[kGroups];
  const int u = threadIdx.x % R::kLanes, chunk = chunk_of_lane(u), group = threadIdx.x / R::kLanes;
  const Seq s = sequence(a, blockIdx.y);
  const int in = blockIdx.x / a.q_heads, head = blockIdx.x - in * a.q_heads;
  if (in >= s.q_len) return;
  const int64_t token = s.q0 + in, row = token * a.q_heads + head;
  const float* stat = a.part_stat + row * a.splits * 2;
  const float* part = a.part_out + row * a.splits * D;
  float best = neg_inf(), sum = 0.0f;
  float v[R::kChunks][8];
#pragma unroll
  for (int k = 0; k < R::kChunks; k++) {
#pragma unroll
    for (int i = 0; i < 8; i++) v[k][i] = 0.0f;
  }
  for (int i = group; i < a.splits; i += kGroups) best = fmaxf(best, stat[2 * i]);
  for (int i = group; i < a.splits; i += kGroups) {
    const float b = stat[2 * i];
    if (b == neg_inf()) continue;   // the split had no keys: its output was not written
    const float f = __builtin_amdgcn_exp2f(b - best);
    sum = __builtin_fmaf(stat[2 * i + 1], f, sum);
#pragma unroll
    for (int k = 0; k < R::kChunks; k++) {
      float x[8];
      load8(reinterpret_cast<const uint8_t*>(part + (int64_t)i * D + k * 128 + chunk * 8), kF32, x);
#pragma unroll
      for (int e = 0; e < 8; e++) v[k][e] = __builtin_fmaf(x[e], f, v[k][e]);
    }
  }
#pragma unroll
  for (int k = 0; k < R::kChunks; k++)
    store8(reinterpret_cast<uint8_t*>(&lds_o[group][k * 128 + chunk * 8]), kF32, v[k]);
  if (u == 0) {
    lds_b[group] = best;
    lds_l[group] = sum;
  }
  __syncthreads();
  if (threadIdx.x >= 64) return;   // the first wave: its first group's lanes store
  best = neg_inf();
  for (int i = 0; i < kGroups; i++) best = fmaxf(best, lds_b[i]);
  sum = 0.0f;
#pragma unroll
  for (int k = 0; k < R::kChunks; k++) {
#pragma unroll
    for (int e = 0; e < 8; e++) v[k][e] = 0.0f;
  }
  const int groups = a.splits < kGroups ? a.splits : kGroups;
  for (int i = 0; i < groups; i++) {
    const float f = lds_b[i] == neg_inf() ? 0.0f : __builtin_amdgcn_exp2f(lds_b[i] - best);
    sum = __builtin_fmaf(lds_l[i], f, sum);
#pragma unroll
    for (int k = 0; k < R::kChunks; k++) {
#pragma unroll
      for (int e = 0; e < 8; e++) v[k][e] = __builtin_fmaf(lds_o[i][k * 128 + chunk * 8 + e], f, v[k][e]);
    }
  }
  const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
#pragma unroll
  for (int k = 0; k < R::kChunks; k++) {
#pragma unroll
    for (int i = 0; i < 8; i++) v[k][i] *= inv;
  }
  const bool ok = group == 0;
  if (ok && a.lse && u == 0) a.lse[row] = sum > 0.0f ? (best + __log2f(sum)) * kLn2 : neg_inf();
  store_row<D, BITS>(a.out + (token * a.out_token + head * a.out_head) * 2, a.dt, v, chunk, ok);
}

template <int D, int BITS>
hipError_t launch(const KvAttentionArgs& a, hipStream_t stream) {
  const dim3 grid(((unsigned)a.splits * a.seqs + kXcds - 1) / kXcds * kXcds * a.row_tiles * a.heads);
  constexpr int kSteps = 2;
  if (a.dt == kF16)
    kv_attend_kernel<D, BITS, kSteps, true><<<grid, kWaves * 64, 0, stream>>>(a);
  else
    kv_attend_kernel<D, BITS, kSteps, false><<<grid, kWaves * 64, 0, stream>>>(a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.splits == 1) return e;
  kv_join_kernel<D, BITS><<<dim3((unsigned)a.max_q * a.q_heads, (unsigned)a.seqs), 256, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace

KvAttentionPlan plan_kv_attention(int64_t total_q, int seqs, int q_heads, int heads, int head_dim, int bits,
                                  int64_t max_q_len, int64_t max_kv_len, int window) {
  const int64_t group = q_heads / heads;
  KvAttentionPlan p;
  const int64_t tiles = (max_q_len * group + kRows - 1) / kRows;
  p.row_tiles = static_cast<int>(tiles < 1 ? 1 : tiles);
  // Enough workgroups for 256 compute units several times over, none with fewer than kMinChunk
  // keys. A split takes the same number of keys in every sequence, and at least kMinChunk: of a
  // long sequence beside short ones no workgroup has more than its share. Measured (64 sequences
  // up to 8192 tokens, 8 heads / 4 up to 131072, one of them most of the work): 768 workgroups 77 /
  // 66 us, 1024 77 / 80, 2048 76 / 59, 4096 81 / 80.
  int64_t span = max_kv_len;
  if (window > 0 && window + max_q_len < span) span = window + max_q_len;
  const int64_t groups = (int64_t)seqs * heads * p.row_tiles, want = (2048 + groups - 1) / groups;
  const int64_t most = (span + 511) / 512;
  const int64_t splits = want < most ? want : most;
  p.splits = static_cast<int>(splits < 1 ? 1 : splits > 256 ? 256 : splits);
  p.chunk = kMinChunk;
  p.workspace_bytes = p.splits > 1 ? (size_t)total_q * q_heads * p.splits * (head_dim + 2) * 4 : 0;
  return p;
}

hipError_t launch_kv_attention(const KvAttentionArgs& a, int head_dim, int bits, hipStream_t stream) {
  if (a.total_q == 0 || a.seqs == 0) return hipSuccess;
  switch (head_dim) {
    case 64: return bits == 8 ? launch<64, 8>(a, stream) : launch<64, 4>(a, stream);
    case 128: return bits == 8 ? launch<128, 8>(a, stream) : launch<128, 4>(a, stream);
    default: return bits == 8 ? launch<256, 8>(a, stream) : launch<256, 4>(a, stream);
  }
}

}  // namespace convrot
