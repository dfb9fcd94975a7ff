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
// most tiles only compare. l may be far above 1. Between logits beyond 2^22 binary32 has no such b
// (and a b half a step off at 2^30 would have p' off by 2^32): there b is the largest logit rounded to
// binary32, the others are rounded so too before b is taken off, and e, taken off after that, stands
// for the value's size. Tiles of rows with an e always go the longer way.
#include "kv_common.h"
#include "kv_query.h"

namespace convrot {
namespace {

using namespace kv;

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kTop = 7.0f;        // log2 of the largest weight when b is set
constexpr float kMost = 32768.0f;   // weights above this move b
// log2 of the p' that a moved b allows (beside a key of that p' whose value is zero, what others add is
// lost below 2^-115 of l), and the sum that moves b.
constexpr float kMostExp = 90.0f;
constexpr float kMostSum = 0x1p120f;
constexpr float kNoRef = -3.0e38f;  // b of a row that has met no key
constexpr int kMinChunk = 1024;     // keys
// More query rows of a sequence and key head than this go by blocks of 128. Measured at 8 heads of 128,
// stream / block: 16 sequences of 4096 tokens, 48 rows 54 / 71 us, 64 rows 61 / 67, 96 rows 82 / 73;
// 2 of 16384, 64 rows 37 / 46, 96 rows 54 / 49.
constexpr int kStreamRows = 64;
constexpr int kSteps = 2;          // 16-token steps of a stream tile
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

// A value's scale, 0 where it is no finite number. The writer makes no such scale, but a token that some
// rows of a tile do not attend to need never have been written, and its scale may read as anything:
// the weight of 0 that it has there, times infinity or NaN, would be NaN.
__device__ __forceinline__ float value_scale(float s) { return __builtin_fabsf(s) < __builtin_inff() ? s : 0.0f; }

// The reference of a row: p' = 2^(t - b), or, for large logits, 2^((t - b) - e) (e not 0).
struct Ref {
  float b, e;
};
constexpr float kLarge = 0x1p22f;   // logits: their steps are 1/4 here
__device__ __forceinline__ bool is_large(float logit) { return __builtin_fabsf(logit) >= kLarge && logit != kNoRef; }
// x c - b: one rounding, or for large logits two, x c first.
__device__ __forceinline__ float from_logit(float x, float c, float b, bool large) {
  return __builtin_fmaf(x, c, large ? 0.0f : -b) - (large ? b : 0.0f);
}
// The reference after a tile. `top`, `wl`: the largest logit (x c, rounded) and, counted from `near`,
// the largest logarithm of a weight; near: the larger of top and the reference there was.
__device__ __forceinline__ Ref moved(const Ref& r, float near, float top, float wl) {
  const float from = (near - r.b) - r.e;
  const bool moves = wl + from > 15.0f || (top - near) + from > kMostExp;
  const float off = fmaxf(wl - kTop, (top - near) - kMostExp);
  const bool large = is_large(near);
  const float e = off == 0.0f ? 0x1p-20f : off;
  Ref n = {moves ? large ? near : near + off : r.b, moves ? large ? e : 0.0f : r.e};
  asm volatile("" : "+v"(n.b));   // or the differences from r.b are kept for the case that it has not moved
  return n;
}

// A tile of keys as a wave holds it: kSteps times 16 tokens.
template <int D, int BITS>
struct Tile {
  using G = Geometry<D, BITS>;
  uint32_t k[kSteps][G::kLoads][G::kWords], v[kSteps][G::kLoads][G::kWords];
  float ks, vs;   // scales, spread over a row of 16 lanes: of token 16 (r / 4) + 4 g + r % 4
  uint32_t ok;    // bit j: step j's page is in the cache
};

// The value that lane N of the lane's row of 16 holds (an operand modifier, no instruction).
template <int N>
__device__ __forceinline__ float row_lane(float v) {
  return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0x150 + N, 0xF, 0xF, true));
}
// a[j][i] = b[j][i] times the scale of step j's token 4g + i.
template <int N = 0>
__device__ __forceinline__ void times_scale(float (&a)[kSteps][4], const float (&b)[kSteps][4], float scale) {
  if constexpr (N < 4 * kSteps) {
    a[N / 4][N % 4] = row_lane<N>(scale) * b[N / 4][N % 4];
    times_scale<N + 1>(a, b, scale);
  }
}

// The largest of x[n] c - near plus the value that lane FIRST + n of the row holds. LARGE: some row's
// logits are.
template <bool LARGE, int FIRST, int COUNT, int N = 0>
__device__ __forceinline__ float largest(const float (&x)[COUNT], float c, float near, float per_key, float so_far) {
  if constexpr (N < COUNT) {
    const float t = from_logit(x[N], c, near, LARGE && is_large(near));
    return largest<LARGE, FIRST, COUNT, N + 1>(x, c, near, per_key, fmaxf(so_far, row_lane<FIRST + N>(per_key) + t));
  } else {
    return so_far;
  }
}

// Page table entries of a tile's steps, read through the scalar cache. Steps past the table's end
// take its last entry (their tokens are masked: they lie behind kv_len).
struct Pages {
  int at[kSteps];
};
__device__ __forceinline__ Pages tile_pages(const KvAttentionArgs& a, ConstTable table, int tile) {
  Pages p;
#pragma unroll
  for (int j = 0; j < kSteps; j++) {
    const int at = (tile * kSteps + j) * 16 >> a.lps;
    p.at[j] = table[at < a.max_pages ? at : a.max_pages - 1];
  }
  return p;
}

// The codes and scales of a tile. Lane (r, g) = (lane % 16, lane / 16) loads, of each 16-token
// step, token r's K bytes (chunk g of every 4 * kLoad) and of the four tokens 4g .. 4g+3 the V
// columns kLoad / 4 * r ..: each load instruction of the wave reads 64 * kLoad contiguous bytes,
// and what arrives is the matrix operand but for the conversion: no exchange between lanes. A page
// index outside the cache loads from page 0; its tokens are masked.
template <int D, int BITS>
__device__ __forceinline__ void load_tile(const KvAttentionArgs& a, const Pages& pages, int head, int tile,
                                          int r, int g, Tile<D, BITS>& t) {
  using G = Geometry<D, BITS>;
  using R = Row<D, BITS>;
  const int page = 1 << a.lps;
  const uint32_t k_lane = r * R::kBytes + g * G::kLoad, v_lane = g * (4 * R::kBytes) + r * G::kLoad;
  const int s_step = r >> 2 < kSteps ? r >> 2 : 0;   // with fewer than four steps some lanes repeat
  const uint8_t* s_at = nullptr;
  t.ok = 0;
#pragma unroll
  for (int j = 0; j < kSteps; j++) {
    const int pg = pages.at[j];
    const bool ok = pg >= 0 && pg < a.num_pages;
    t.ok |= ok ? 1u << j : 0u;
    const uint8_t* block = a.cache + ((int64_t)(ok ? pg : 0) * a.heads + head) * a.head_bytes;
    const int off = (tile * kSteps + j) * 16 & (page - 1);
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
  Ref ref;   // the row's reference
  float l;   // this lane's part of the row's sum of p': 0 if it has met no key, and only then (a sum that
             // is no number is a result like any other, for the waves' and the splits' joins too)
};

template <int D, int BITS>
__device__ __forceinline__ void start(State<D, BITS>& s) {
#pragma unroll
  for (int m = 0; m < D / 16; m++) s.o[m] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  s.ref = {kNoRef, 0.0f};
  s.l = 0.0f;
}

template <int D, int BITS, bool SPLIT>
__device__ __forceinline__ void attend_tile(Tile<D, BITS>& t, const u32x4 (&q)[D / 32], const u32x4 (&q2)[D / 32],
                                            float c, bool full, int r, int first, int lo, int hi, int kv_len, State<D, BITS>& s) {
  using G = Geometry<D, BITS>;
  float x[kSteps][4], p[kSteps][4], w[kSteps][4];
#pragma unroll
  for (int j = 0; j < kSteps; j++) {
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
  // No branch between the products and the first use of what they give: where two ways meet, the compiler
  // (ROCm 7.2) counts the wait states after a matrix instruction along one of them only.
  times_scale(x, x, t.ks);
  t.vs = value_scale(t.vs);
  if (!full) {   // the same in every lane
    asm volatile("");   // a branch, not selects in every tile
    const int mine = first + 16 * (r >> 2) + (r & 3);   // `first` includes 4 g
    const uint32_t step = r >> 2 < kSteps ? r >> 2 : 0;
    t.vs = mine < kv_len && (t.ok >> step & 1u) ? t.vs : 0.0f;
#pragma unroll
    for (int j = 0; j < kSteps; j++) {
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const int key = first + 16 * j + i;
        const int end = t.ok >> j & 1u ? kv_len : 0, own = hi < end ? hi : end;
        x[j][i] = static_cast<uint32_t>(key - lo) < static_cast<uint32_t>(own > lo ? own - lo : 0) ? x[j][i] : neg_inf();
      }
    }
  }
  // Weights for the present reference; true if they fit: none above kMost, and no p' so large that l
  // might come near its range's end (a first key's is infinite: b is kNoRef).
  float l;
  auto weigh = [&](auto exponent_of) {
    float wtop = 0.0f;
    l = s.l;
#pragma unroll
    for (int j = 0; j < kSteps; j++) {
#pragma unroll
      for (int i = 0; i < 4; i++) {
        p[j][i] = __builtin_amdgcn_exp2f(exponent_of(x[j][i]));
        l += p[j][i];
      }
    }
    times_scale(w, p, t.vs);
#pragma unroll
    for (int j = 0; j < kSteps; j++) {
#pragma unroll
      for (int i = 0; i < 4; i++) wtop = fmaxf(wtop, w[j][i]);
    }
    return wtop <= kMost && l < kMostSum;
  };
  const bool fits = weigh([&](float y) { return __builtin_fmaf(y, c, -s.ref.b); });
  if (!__all(fits && s.ref.e == 0.0f)) {
    // The logarithm of the tile's largest weight, and its largest logit, over the row's four lanes.
    const float lv = t.vs > 0.0f ? __builtin_amdgcn_logf(t.vs) : neg_inf();
    float top = neg_inf();
#pragma unroll
    for (int j = 0; j < kSteps; j++) {
#pragma unroll
      for (int i = 0; i < 4; i++) top = fmaxf(top, x[j][i]);
    }
    top = quad_max(top) * c;
    const float near = fmaxf(top, s.ref.b);
    const bool large = __any(is_large(near));
    static_assert(kSteps == 2, "");
    float wl;
    if (large)
      wl = largest<true, 4>(x[1], c, near, lv, largest<true, 0>(x[0], c, near, lv, neg_inf()));
    else
      wl = largest<false, 4>(x[1], c, near, lv, largest<false, 0>(x[0], c, near, lv, neg_inf()));
    const Ref n = moved(s.ref, near, top, quad_max(wl));
    const float alpha = __builtin_amdgcn_exp2f((s.ref.b - n.b) + (s.ref.e - n.e));   // 0 for a row that had no reference
    s.ref = n;
    s.l *= alpha;
#pragma unroll
    for (int m = 0; m < G::kTilesD; m++) s.o[m] *= alpha;
    if (large)
      weigh([&](float y) { return from_logit(y, c, s.ref.b, s.ref.e != 0.0f) - s.ref.e; });
    else
      weigh([&](float y) { return __builtin_fmaf(y, c, -s.ref.b); });
  }
  s.l = l;
#pragma unroll
  for (int j = 0; j < kSteps; j += 2) {
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
// The waves take the split's tiles of keys in turn, each with a softmax of its own; they are joined
// through LDS, and splits through the workspace (kv_join_kernel).
template <int D, int BITS, bool SPLIT, int WAVES>
__global__ __launch_bounds__(WAVES * 64, D == 256 ? 1 : 2) void kv_attend_kernel(KvAttentionArgs a) {
  using R = Row<D, BITS>;
  using G = Geometry<D, BITS>;
  constexpr int kOutPad = 4, kTile = 16 * kSteps;
  __shared__ __attribute__((aligned(16))) float lds_o[WAVES][kRows][D + kOutPad];
  __shared__ float lds_m[WAVES][kRows], lds_l[WAVES][kRows], lds_c[kRows];
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
  auto next = [&](int at) { return at + WAVES < end ? at + WAVES : at; };
  // (A wave without tiles loads the last one too, and does not use it.)
  Tile<D, BITS> t0, t1;
  Pages pages = tile_pages(a, table, i < end ? i : end - 1);
  load_tile<D, BITS>(a, pages, head, i < end ? i : end - 1, r, g, t0);
  int n = next(i);
  pages = tile_pages(a, table, n < end ? n : end - 1);
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
    const float up = query_scale(top);
    if (row < kRows) {
#pragma unroll
      for (int k = 0; k < R::kChunks; k++) {
        uint32_t w[4];
        uint32_t* p = lds_q + row * (D / 2) + (k * 16 + chunk) * 4;
        query_words<BITS>(v[k], sign * up, false, w);
        *reinterpret_cast<u32x4*>(p) = u32x4{w[0], w[1], w[2], w[3]};
        if constexpr (SPLIT) {
          query_words<BITS>(v[k], sign * up, true, w);
          *reinterpret_cast<u32x4*>(p + kRows * (D / 2)) = u32x4{w[0], w[1], w[2], w[3]};
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
    auto attend = [&](Tile<D, BITS>& t, int at) {
      const int first = at * kTile;
      const bool full = whole && t.ok == (1u << kSteps) - 1 && first >= full_lo && first + kTile <= full_hi;
      attend_tile<D, BITS, SPLIT>(t, q, q2, c, full, r, first + 4 * g, lo, hi, s.kv_len, st);
    };
    while (true) {
      load_tile<D, BITS>(a, pages, head, n, r, g, t1);
      int m = next(n);
      pages = tile_pages(a, table, m);
      attend(t0, i);
      if (n == i) break;
      i = n;
      n = m;
      load_tile<D, BITS>(a, pages, head, n, r, g, t0);
      m = next(n);
      pages = tile_pages(a, table, m);
      attend(t1, i);
      if (n == i) break;
      i = n;
      n = m;
    }
  }

  // Join the waves.
  st.l = quad_sum(st.l) * __builtin_amdgcn_exp2f(st.ref.e);   // counted from b, as o will be
  if (g == 0) {
    lds_m[wave][r] = st.l == 0.0f ? neg_inf() : st.ref.b;
    lds_l[wave][r] = st.l;
  }
  __syncthreads();
  float top = lds_m[0][r];
#pragma unroll
  for (int w = 1; w < WAVES; w++) top = fmaxf(top, lds_m[w][r]);
  {
    const float m = lds_m[wave][r];
    const float f = m == neg_inf() ? 0.0f : __builtin_amdgcn_exp2f((m - top) + st.ref.e);
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
    for (int w = 0; w < WAVES; w++) best = fmaxf(best, lds_m[w][rc]);
#pragma unroll
    for (int w = 0; w < WAVES; w++)
      sum += lds_m[w][rc] == neg_inf() ? 0.0f : lds_l[w][rc] * __builtin_amdgcn_exp2f(lds_m[w][rc] - best);
    float v[R::kChunks][8];
#pragma unroll
    for (int k = 0; k < R::kChunks; k++) {
#pragma unroll
      for (int i = 0; i < 8; i++) {
        float y = 0.0f;
#pragma unroll
        for (int w = 0; w < WAVES; w++) y += lds_o[w][rc][k * 128 + chunk * 8 + i];
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
      const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
      for (int k = 0; k < R::kChunks; k++) {
#pragma unroll
        for (int i = 0; i < 8; i++) v[k][i] *= inv;
      }
      if (ok && a.lse && u == 0) a.lse[out_row] = sum == 0.0f ? neg_inf() : (best + __log2f(sum)) * kLn2;
      store_row<D, BITS>(a.out + ((s.q0 + token) * a.out_token + qh * a.out_head) * 2, a.dt, v, chunk, ok);
    }
  }
}

// ---- Many query rows: tiles of keys shared by a workgroup ----------------------------------
//
// One workgroup: 128 query rows of one key head and sequence, 32 a wave, and one split of the
// keys. The stream kernel above converts every code in every wave, 64 codes for a wave's 16 rows;
// here a tile of 64 keys is converted once for 128 rows and laid in LDS as fp16 operands of
// 32x32x16 matrix instructions:
//   K   [key][D], 16-byte chunks (8 elements) of a row exchanged by key & 7
//   V   [d][64 keys], chunk 2 s + h of a row: the keys that lane half h holds of 16-key step s,
//       16 s + 4 h + {0, 2, 1, 3} and 8 further; chunks exchanged by (d ^ d / 8) & 7
// so that eight neighbouring lanes always touch eight different 16-byte bank groups. As above the
// logits come out with a query row in each lane (two lanes a row), which is the operand of the
// second product. While one tile is worked on the next is converted into a second buffer, and the
// codes of the one after are on their way.
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kBlockRows = 128, kBlockKeys = 64;

__device__ __forceinline__ f32x16 mfma32(const u32x4& a, const u32x4& b, const f32x16& c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// Barrier for LDS: global loads under way stay so.
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

template <int N = 0>
__device__ __forceinline__ void times_scale16(float (&a)[16], const float (&b)[16], float scale) {
  if constexpr (N < 16) {
    a[N] = row_lane<N>(scale) * b[N];
    times_scale16<N + 1>(a, b, scale);
  }
}

// At head_dim 64 in bf16 three waves a SIMD: 168 registers, two of them spilled with 8-bit codes (2 x 4096 x 4096,
// 12 heads: 169 us; 188 with 170 registers and two waves). In fp16 the rests of queries and weights do not
// all fit: 57 registers are spilled at head_dim 256 with 8-bit codes, 46 with 4-bit ones, 2 at 128 with 8-bit
// ones (that shape in fp16 and bf16: 1141 and 698 us, 1071 and 666, 408 and 287).
template <int D, int BITS, bool SPLIT>
__global__ __launch_bounds__(256, D == 256 ? 1 : D == 64 && !SPLIT ? 3 : 2) void kv_attend_block_kernel(KvAttentionArgs a) {
  using R = Row<D, BITS>;
  constexpr int kUnits = R::kBytes / 32;        // 16-byte pieces of a tile's codes a thread loads
  constexpr int kPieces = 4 * R::kBytes;        // of K, and as many of V
  constexpr bool kTwoSteps = R::kBytes == 32;   // a wave's pieces lie in two 16-token steps
  constexpr int kOps = D / 16, kTilesD = D / 32;
  constexpr uint32_t kBuffer = kBlockKeys * D * 4;   // a tile of K and V; two of them in turn
  __shared__ __attribute__((aligned(16))) uint8_t lds[2 * kBuffer];
  __shared__ float lds_ks[2][kBlockKeys], lds_vs[2][kBlockKeys];
  __shared__ uint64_t lds_ok[2];
  __shared__ float lds_c[4][32];
  // A chunk's place in its K row: what loads and stages a row has its chunks of 64 elements in
  // different lanes, which the second term keeps apart.
  auto k_chunk = [](int chunk, int key) {
    return chunk ^ (key & 7) ^ (BITS == 8 ? chunk >> 3 & 1 : D == 128 ? (chunk >> 3 & 1) * 2 : chunk >> 3 & 3);
  };

  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, r = lane & 31, h = lane >> 5;
  // Heads first, then sequences; the tiles from the last to the first (with causal the last ones
  // have the most keys); splits last. From tile to tile the sequences are turned by one: workgroups
  // go to the XCDs and to the shader engines of one in turn, and of a ragged batch's tiles most
  // are the longest sequence's (chunks of 423 to 2048 rows, 8 heads: 1212 us with that sequence
  // always in the same place, 718 us so).
  uint32_t id = blockIdx.x;
  const int head = id % a.heads;
  id /= a.heads;
  const uint32_t turn = id / a.seqs;
  const int b = (id - turn * a.seqs + turn) % a.seqs;
  const int split = a.splits == 1 ? 0 : turn / a.row_tiles;
  const int tile = a.row_tiles - 1 - (turn - split * a.row_tiles);
  const Seq s = sequence(a, b);
  const int rows = (s.q_len < a.max_q ? s.q_len : a.max_q) * a.group;
  const int row_first = tile * kBlockRows;
  if (row_first >= rows) return;
  const int row_last = (row_first + kBlockRows < rows ? row_first + kBlockRows : rows) - 1;
  const ConstTable table = const_table(a.pages + (int64_t)b * a.max_pages);
  const int page = 1 << a.lps;

  // Keys: of the workgroup, of the wave, of the lane's row.
  int t_lo, t_hi, lo, hi, w_lo, w_hi, full_lo, full_hi;
  key_range(a, s, token_of(a, row_first), t_lo, hi);
  key_range(a, s, token_of(a, row_last), lo, t_hi);
  const int w_first = row_first + 32 * wave, w_last = w_first + 31 < rows ? w_first + 31 : rows - 1;
  w_lo = w_hi = full_lo = full_hi = 0;
  if (w_first < rows) {
    key_range(a, s, token_of(a, w_first), w_lo, full_hi);
    key_range(a, s, token_of(a, w_last), full_lo, w_hi);
    if (w_last != w_first + 31) full_hi = 0;
  }
  const bool mine = w_first + r < rows;
  key_range(a, s, token_of(a, mine ? w_first + r : row_first), lo, hi);
  if (!mine) lo = hi = 0;
  const int tiles_lo = t_lo / kBlockKeys, tiles_hi = (t_hi + kBlockKeys - 1) / kBlockKeys;
  const int count = tiles_hi > tiles_lo ? tiles_hi - tiles_lo : 0;
  const int share = (count + a.splits - 1) / a.splits, chunk = share > a.chunk / kBlockKeys ? share : a.chunk / kBlockKeys;
  const int begin = tiles_lo + (split * (int64_t)chunk < count ? split * chunk : count);
  const int end = tiles_lo + (count - (begin - tiles_lo) < chunk ? count : begin - tiles_lo + chunk);

  // Codes of a tile: piece p of K is 16 bytes of key p / (row_bytes / 16), piece p of V the 16
  // bytes at column 4 (p % (row_bytes / 4)) of token group p / (row_bytes / 4); consecutive lanes
  // read consecutive bytes of a page. The table entry of a wave's 16-token step comes through the
  // scalar cache one tile ahead; lane L of the first two waves loads key L's scale.
  u32x4 raw[kUnits];
  float raw_scale = 0.0f;
  bool raw_ok = false;
  int at_page[kUnits][kTwoSteps ? 2 : 1], scale_page = 0;
  // The token group of V's piece p. Of 16 neighbouring lanes 8 take groups whose tokens go into the
  // other half of a 16-byte chunk: their writes then meet in no bank.
  auto v_group = [](int p) {
    const int g = p / (R::kBytes / 4);
    if constexpr (R::kBytes == 64) return g ^ (p >> 3 & 1) * 2;
    if constexpr (R::kBytes == 32) return (g & ~3) | (g & 1) << 1 | (g >> 1 & 1);
    return g;
  };
  // The wave's n-th 64 pieces: V's (known when compiling where a round of the workgroup is all K's or
  // all V's), their first, and its 16-token step: 16 tokens are row_bytes pieces.
  auto is_v = [&](int n) { return kPieces >= 256 ? n * 256 >= kPieces : wave * 64 >= kPieces; };
  auto piece_of = [&](int n) { return n * 256 + wave * 64 - (is_v(n) ? kPieces : 0); };
  auto step_of = [&](int n) { return piece_of(n) / R::kBytes; };
  auto load_pages = [&](int at) {
#pragma unroll
    for (int n = 0; n < kUnits; n++) {
#pragma unroll
      for (int k = 0; k < (kTwoSteps ? 2 : 1); k++) {
        const int e = (at * kBlockKeys + (step_of(n) + k) * 16) >> a.lps;
        at_page[n][k] = table[e < a.max_pages ? e : a.max_pages - 1];
      }
    }
    if (wave < 2) {
      const int e = (at * kBlockKeys + lane) >> a.lps;
      scale_page = a.pages[(int64_t)b * a.max_pages + (e < a.max_pages ? e : a.max_pages - 1)];
    }
  };
  auto load_codes = [&](int at) {
#pragma unroll
    for (int n = 0; n < kUnits; n++) {
      const int p = piece_of(n) + lane, step = step_of(n);
      const bool values = is_v(n);
      const uint8_t* block[kTwoSteps ? 2 : 1];
#pragma unroll
      for (int k = 0; k < (kTwoSteps ? 2 : 1); k++) {
        const int pg = at_page[n][k];
        const bool ok = pg >= 0 && pg < a.num_pages;
        block[k] = a.cache + ((int64_t)(ok ? pg : 0) * a.heads + head) * a.head_bytes;
      }
      // The piece's bytes follow its step's first: 16 tokens' K (or V) codes are 16 row_bytes.
      const uint8_t* base = block[0];
      int off = (at * kBlockKeys + step * 16) & (page - 1);
      const int q = values ? v_group(p) * (R::kBytes / 4) + p % (R::kBytes / 4) : p;
      uint32_t in = (q - step * R::kBytes) * 16;
      if constexpr (kTwoSteps) {
        if (lane >= 32) {
          base = block[1];
          off = (at * kBlockKeys + (step + 1) * 16) & (page - 1);
          in -= 16 * R::kBytes;
        }
      }
      raw[n] = *reinterpret_cast<const u32x4*>(base + ((off + (values ? page : 0)) * R::kBytes + in));
    }
    if (wave < 2) {
      const int key = at * kBlockKeys + lane;
      const bool in = scale_page >= 0 && scale_page < a.num_pages;
      raw_ok = in && key < s.kv_len;
      const uint8_t* block = a.cache + ((int64_t)(in ? scale_page : 0) * a.heads + head) * a.head_bytes;
      raw_scale = reinterpret_cast<const float*>(block + 2 * page * R::kBytes)[(wave ? page : 0) + (key & (page - 1))];
    }
  };
  auto stage = [&](int half) {   // into buffer `half`
#pragma unroll
    for (int n = 0; n < kUnits; n++) {
      const int p = piece_of(n) + lane;
      if (!is_v(n)) {
        const int key = p / (R::kBytes / 16), first = p % (R::kBytes / 16) * (16 / BITS);   // the piece's first chunk
        uint32_t to = half * kBuffer + key * (D * 2) + k_chunk(first, key) * 16;
        asm volatile("" : "+v"(to));
#pragma unroll
        for (int w = 0; w < 4; w += BITS / 4) {
          u32x4 c;
          if constexpr (BITS == 4) {
            uint32_t x[4];
            nibbles_f16(raw[n][w], x);
            c = u32x4{x[0], x[1], x[2], x[3]};
          } else {
            uint32_t x[2], y[2];
            bytes_f16(raw[n][w], x);
            bytes_f16(raw[n][w + 1], y);
            c = u32x4{x[0], x[1], y[0], y[1]};
          }
          *reinterpret_cast<u32x4*>(lds + (to ^ (w * 4 / BITS) * 16)) = c;
        }
      } else {
        // Rows d = kRow col + y, y < 4 kRow <= 8: the chunk of row d is that of row kRow col, exchanged by y.
        const int group = v_group(p), col = p % (R::kBytes / 4) * 4;
        const int at = (group >> 2) * 2 + (group & 1);
        constexpr int kRow = 8 / BITS;
        const int d0 = kRow * col;
        uint32_t to = half * kBuffer + kBuffer / 2 + d0 * 128 + ((at ^ ((d0 ^ (d0 >> 3)) & 7)) * 16) + (group >> 1 & 1) * 8;
        asm volatile("" : "+v"(to));
        auto put = [&](int y, uint32_t a0, uint32_t a1) {
          *reinterpret_cast<u32x2*>(lds + (to ^ y * 16) + y * 128) = u32x2{a0, a1};
        };
#pragma unroll
        for (int w = 0; w < 4; w++) {
          if constexpr (BITS == 4) {
            uint32_t x[4];
            nibbles_f16(raw[n][w], x);
            put(2 * w, x[0], x[2]);
            put(2 * w + 1, x[1], x[3]);
          } else {
            uint32_t x[2];
            bytes_f16(raw[n][w], x);
            put(w, x[0], x[1]);
          }
        }
      }
    }
    if (wave == 0) {
      const uint64_t ok = __ballot(raw_ok);
      if (lane == 0) lds_ok[half] = ok;
      lds_ks[half][lane] = raw_scale;
    } else if (wave == 1) {
      lds_vs[half][lane] = raw_ok ? value_scale(raw_scale) : 0.0f;
    }
  };
  if (begin < end) {
    load_pages(begin);
    load_codes(begin);
    load_pages(begin + 1 < end ? begin + 1 : begin);
  }

  // Queries, a wave its own 32 rows: rotated, scaled, to fp16, in the K operands' element order.
  u32x4 q[kOps], q2[kOps];
  {
    constexpr int kAtOnce = 64 / R::kLanes;
    uint32_t* region = reinterpret_cast<uint32_t*>(lds) + wave * (16 * D);   // 32 rows of D / 2 words
    const int u = lane % R::kLanes, chunk = chunk_of_lane(u);
    for (int part = 0; part < (SPLIT ? 2 : 1); part++) {
      for (int k0 = 0; k0 < 32; k0 += kAtOnce) {
        const int row = k0 + lane / R::kLanes, n = w_first + row;
        const bool ok = n < rows;
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
        const float up = query_scale(row_max<R::kLanes>(top));
#pragma unroll
        for (int k = 0; k < R::kChunks; k++) {
          uint32_t w[4];
          query_words<BITS>(v[k], sign * up, part == 1, w);
          *reinterpret_cast<u32x4*>(region + row * (D / 2) + ((k * 16 + chunk) ^ (row & 7)) * 4) = u32x4{w[0], w[1], w[2], w[3]};
        }
        if (u == 0) lds_c[wave][row] = a.scale * (kLog2e * R::kNorm) / up;
      }
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int m = 0; m < kOps; m++) {
        const u32x4 w = *reinterpret_cast<const u32x4*>(region + r * (D / 2) + ((2 * m + h) ^ (r & 7)) * 4);
        if (part == 0) q[m] = w;
        if (SPLIT && part == 1) q2[m] = w;
      }
      __builtin_amdgcn_wave_barrier();
    }
  }
  const float c = fmaxf(lds_c[wave][r], 1.1754944e-38f);

  // Where the lane reads its operands: chunk 2 m + h of K row r, chunk 2 k + h of V row 32 t + r. All
  // others follow by exchanging bits of the address, which costs less than keeping them.
  uint32_t k_at = r * (D * 2) + k_chunk(h, r) * 16, v_at = kBuffer / 2 + r * 128 + (h ^ ((r ^ (r >> 3)) & 7)) * 16;

  f32x16 o[kTilesD];
#pragma unroll
  for (int t = 0; t < kTilesD; t++) {
#pragma unroll
    for (int i = 0; i < 16; i++) o[t][i] = 0.0f;
  }
  Ref ref = {kNoRef, 0.0f};
  float sum = 0.0f;

  lds_barrier();   // the queries' region has been read
  if (begin < end) {
    stage(0);
    load_codes(begin + 1 < end ? begin + 1 : begin);
    load_pages(begin + 2 < end ? begin + 2 : end - 1);
  }
  lds_barrier();
  for (int at = begin; at < end; at++) {
    // One buffer is read, the next tile goes into the other, the one after is on its way.
    const int half = (at - begin) & 1, first = at * kBlockKeys;
    auto next = [&]() {
      stage(half ^ 1);
      load_codes(at + 2 < end ? at + 2 : end - 1);
      load_pages(at + 3 < end ? at + 3 : end - 1);
    };
    if (first >= w_hi || first + kBlockKeys <= w_lo) {   // none of the wave's rows
      next();
      lds_barrier();
      k_at ^= kBuffer;
      v_at ^= kBuffer;
      continue;
    }
    const uint64_t there = lds_ok[half];
    asm volatile("" : "+v"(k_at), "+v"(v_at));   // not kept over the loop in all their forms
    // Both 32-key halves together: two chains of products.
    f32x16 acc[2];
#pragma unroll
    for (int sub = 0; sub < 2; sub++) {
#pragma unroll
      for (int i = 0; i < 16; i++) acc[sub][i] = 0.0f;
    }
#pragma unroll
    for (int m = 0; m < kOps; m++) {
#pragma unroll
      for (int sub = 0; sub < 2; sub++) {
        const u32x4 kop = *reinterpret_cast<const u32x4*>(lds + (k_at ^ k_chunk(2 * m, 0) * 16) + sub * 32 * (D * 2));
        if constexpr (SPLIT) acc[sub] = mfma32(kop, q2[m], acc[sub]);
        acc[sub] = mfma32(kop, q[m], acc[sub]);
      }
    }
    next();   // beside the products
    // Lane n of a row of 16 holds the scales of its half's n-th key: 8 (n / 4) + 4 h + n % 4.
    const int sk = 8 * ((lane & 15) >> 2) + 4 * h + (lane & 3);
    float x[2][16], p[2][16], vs[2];
#pragma unroll
    for (int sub = 0; sub < 2; sub++) {
      vs[sub] = lds_vs[half][sub * 32 + sk];
#pragma unroll
      for (int i = 0; i < 16; i++) x[sub][i] = acc[sub][i];
      times_scale16(x[sub], x[sub], lds_ks[half][sub * 32 + sk]);
    }
    if (!(there == ~0ull && first >= full_lo && first + kBlockKeys <= full_hi)) {
      asm volatile("");   // a branch, not 32 selects in every tile
      const uint32_t span = hi > lo ? hi - lo : 0;
#pragma unroll
      for (int sub = 0; sub < 2; sub++) {
        const uint32_t bits = static_cast<uint32_t>(there >> (sub * 32)) >> (4 * h);
        const uint32_t from = first + sub * 32 + 4 * h - lo;
#pragma unroll
        for (int i = 0; i < 16; i++) {
          const int n = 8 * (i / 4) + i % 4;
          x[sub][i] = from + n < span && (bits >> n & 1u) ? x[sub][i] : neg_inf();
        }
      }
    }
    float l, w[2][16];
    auto weigh = [&](auto exponent_of) {
      l = sum;
      float wtop = 0.0f;
#pragma unroll
      for (int sub = 0; sub < 2; sub++) {
#pragma unroll
        for (int i = 0; i < 16; i++) {
          p[sub][i] = __builtin_amdgcn_exp2f(exponent_of(x[sub][i]));
          l += p[sub][i];
        }
        times_scale16(w[sub], p[sub], vs[sub]);
#pragma unroll
        for (int i = 0; i < 16; i++) wtop = fmaxf(wtop, w[sub][i]);
      }
      return wtop <= kMost && l < kMostSum;
    };
    const bool fits = weigh([&](float y) { return __builtin_fmaf(y, c, -ref.b); });
    if (!__all(fits && ref.e == 0.0f)) {   // as in attend_tile
      float wl = neg_inf(), top = neg_inf();
#pragma unroll
      for (int sub = 0; sub < 2; sub++) {
#pragma unroll
        for (int i = 0; i < 16; i++) top = fmaxf(top, x[sub][i]);
      }
      top = fmaxf(top, __shfl_xor(top, 32, 64)) * c;
      const float near = fmaxf(top, ref.b);
      const bool large = __any(is_large(near));
#pragma unroll
      for (int sub = 0; sub < 2; sub++) {
        const float lv = vs[sub] > 0.0f ? __builtin_amdgcn_logf(vs[sub]) : neg_inf();
        if (large)
          wl = largest<true, 0>(x[sub], c, near, lv, wl);
        else
          wl = largest<false, 0>(x[sub], c, near, lv, wl);
      }
      const Ref n = moved(ref, near, top, fmaxf(wl, __shfl_xor(wl, 32, 64)));
      const float alpha = __builtin_amdgcn_exp2f((ref.b - n.b) + (ref.e - n.e));
      ref = n;
      sum *= alpha;
#pragma unroll
      for (int t = 0; t < kTilesD; t++) o[t] *= alpha;
      if (large)
        weigh([&](float y) { return from_logit(y, c, ref.b, ref.e != 0.0f) - ref.e; });
      else
        weigh([&](float y) { return __builtin_fmaf(y, c, -ref.b); });
    }
    sum = l;
#pragma unroll
    for (int k = 0; k < 4; k++) {
      const float* y = w[k / 2] + 8 * (k % 2);
      const u32x4 lead = {pack_f16(y[0], y[2]), pack_f16(y[1], y[3]), pack_f16(y[4], y[6]), pack_f16(y[5], y[7])};
      u32x4 rest;
      if constexpr (SPLIT)
        rest = u32x4{rest_f16(lead[0], y[0], y[2]), rest_f16(lead[1], y[1], y[3]), rest_f16(lead[2], y[4], y[6]),
                     rest_f16(lead[3], y[5], y[7])};
#pragma unroll
      for (int t = 0; t < kTilesD; t++) {
        const u32x4 vop = *reinterpret_cast<const u32x4*>(lds + (v_at ^ ((2 * k) ^ (t & 1) * 4) * 16) + t * 32 * 128);
        if constexpr (SPLIT) o[t] = mfma32(vop, rest, o[t]);
        o[t] = mfma32(vop, lead, o[t]);
      }
    }
    lds_barrier();
    k_at ^= kBuffer;
    v_at ^= kBuffer;
  }

  // Outputs, a wave its own rows, 16 at a time through its quarter of the LDS.
  sum += __shfl_xor(sum, 32, 64);
  const float back = __builtin_amdgcn_exp2f(ref.e);   // to what is counted from b
  float* region = reinterpret_cast<float*>(lds) + wave * (16 * D);
  const int u = lane % R::kLanes, cc = chunk_of_lane(u);
  for (int part = 0; part < 2; part++) {
    __builtin_amdgcn_wave_barrier();
    if ((r >> 4) == part) {
#pragma unroll
      for (int t = 0; t < kTilesD; t++) {
#pragma unroll
        for (int i = 0; i < 4; i++)
          *reinterpret_cast<f32x4*>(region + (r & 15) * D + ((t * 8 + 2 * i + h) ^ (r & 15)) * 4) =
              f32x4{o[t][4 * i], o[t][4 * i + 1], o[t][4 * i + 2], o[t][4 * i + 3]};
      }
    }
    __builtin_amdgcn_wave_barrier();
    for (int k0 = 0; k0 < 16; k0 += 64 / R::kLanes) {
      const int row = k0 + lane / R::kLanes, n = w_first + part * 16 + row;
      const bool ok = n < rows;
      const int token = ok ? token_of(a, n) : 0, qh = head * a.group + (ok ? n - token * a.group : 0);
      const float g = __shfl(back, part * 16 + row, 64);
      const float l = __shfl(sum, part * 16 + row, 64) * g, rb = __shfl(ref.b, part * 16 + row, 64);
      float v[R::kChunks][8];
#pragma unroll
      for (int k = 0; k < R::kChunks; k++) {
#pragma unroll
        for (int e = 0; e < 2; e++) {
          const f32x4 y = *reinterpret_cast<const f32x4*>(region + row * D + ((k * 32 + cc * 2 + e) ^ row) * 4);
#pragma unroll
          for (int i = 0; i < 4; i++) v[k][4 * e + i] = y[i] * g;
        }
      }
      const int64_t out_row = (int64_t)(s.q0 + token) * a.q_heads + qh;
      if (a.splits > 1) {
        if (!ok) continue;
        if (l != 0.0f) {
          float* to = a.part_out + (out_row * a.splits + split) * D;
#pragma unroll
          for (int k = 0; k < R::kChunks; k++) store8(reinterpret_cast<uint8_t*>(to + k * 128 + cc * 8), kF32, v[k]);
        }
        if (u == 0) {
          a.part_stat[(out_row * a.splits + split) * 2] = l == 0.0f ? neg_inf() : rb;
          a.part_stat[(out_row * a.splits + split) * 2 + 1] = l;
        }
      } else {
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
        for (int k = 0; k < R::kChunks; k++) {
#pragma unroll
          for (int i = 0; i < 8; i++) v[k][i] *= inv;
        }
        if (ok && a.lse && u == 0) a.lse[out_row] = l == 0.0f ? neg_inf() : (rb + __log2f(l)) * kLn2;
        store_row<D, BITS>(a.out + ((s.q0 + token) * a.out_token + qh * a.out_head) * 2, a.dt, v, cc, ok);
      }
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
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
  for (int k = 0; k < R::kChunks; k++) {
#pragma unroll
    for (int i = 0; i < 8; i++) v[k][i] *= inv;
  }
  const bool ok = group == 0;
  if (ok && a.lse && u == 0) a.lse[row] = sum == 0.0f ? neg_inf() : (best + __log2f(sum)) * kLn2;
  store_row<D, BITS>(a.out + (token * a.out_token + head * a.out_head) * 2, a.dt, v, chunk, ok);
}

template <int D, int BITS>
void launch_stream(const KvAttentionArgs& a, hipStream_t stream) {
  const dim3 grid(((unsigned)a.splits * a.seqs + kXcds - 1) / kXcds * kXcds * a.row_tiles * a.heads);
  // With a workgroup for each compute unit or fewer, eight waves share a split's keys: a wave's tiles
  // come one behind the other, each a trip to memory (one token over 2048, 2 key heads of 128, in a
  // graph: 19.9 us with four waves, 16.3 with eight; over 128 tokens 6.5 both). With more workgroups
  // four: the registers hold twelve waves a unit, and hold no eight of head_dim 256 at all.
  if constexpr (D < 256) {
    if (grid.x <= 256) {
      if (a.dt == kF16)
        kv_attend_kernel<D, BITS, true, 8><<<grid, 512, 0, stream>>>(a);
      else
        kv_attend_kernel<D, BITS, false, 8><<<grid, 512, 0, stream>>>(a);
      return;
    }
  }
  if (a.dt == kF16)
    kv_attend_kernel<D, BITS, true, 4><<<grid, 256, 0, stream>>>(a);
  else
    kv_attend_kernel<D, BITS, false, 4><<<grid, 256, 0, stream>>>(a);
}

template <int D, int BITS>
hipError_t launch(const KvAttentionArgs& a, hipStream_t stream) {
  if (a.block) {
    const dim3 grid((unsigned)a.splits * a.row_tiles * a.seqs * a.heads);
    if (a.dt == kF16)
      kv_attend_block_kernel<D, BITS, true><<<grid, 256, 0, stream>>>(a);
    else
      kv_attend_block_kernel<D, BITS, false><<<grid, 256, 0, stream>>>(a);
  } else {
    launch_stream<D, BITS>(a, stream);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.splits == 1) return e;
  kv_join_kernel<D, BITS><<<dim3((unsigned)a.max_q * a.q_heads, (unsigned)a.seqs), 256, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace

KvAttentionPlan plan_kv_attention(int64_t total_q, int seqs, int q_heads, int heads, int head_dim,
                                  int64_t max_q_len, int64_t max_kv_len, int window) {
  const int64_t group = q_heads / heads;
  KvAttentionPlan p;
  p.block = max_q_len * group > kStreamRows;
  const int tile_rows = p.block ? kBlockRows : kRows;
  const int64_t tiles = (max_q_len * group + tile_rows - 1) / tile_rows;
  p.row_tiles = static_cast<int>(tiles < 1 ? 1 : tiles);
  // Enough workgroups for 256 compute units several times over. A split takes the same number of
  // keys in every sequence, the longest's share and at most kMinChunk where that is less: of a long
  // sequence beside short ones no workgroup has more than its share, and the short ones' are few.
  // Stream kernel (64 sequences up to 8192 tokens, 8 heads / 4 up to 131072, one of them most of the
  // work): 768 workgroups 77 / 66 us, 1024 77 / 80, 2048 76 / 59, 4096 81 / 80. Block kernel: two a
  // compute unit. A join costs about 5 us and each row of it some more: splits have 512 keys at
  // least; 256 with few blocks (300 rows over 1500 keys, 8 heads: 45 us with 512, 34 with 256; 512
  // rows of 4 heads each over 512 keys, 8 key heads: 28 unsplit, 40 with 256), and 2048 with enough
  // groups already, where a split only spares the wait for the longest.
  int64_t span = max_kv_len;
  if (window > 0 && window + max_q_len < span) span = window + max_q_len;
  const int64_t groups = (int64_t)seqs * heads * p.row_tiles, want = p.block ? 512 / groups : (2048 + groups - 1) / groups;
  const int64_t most = span / (groups >= 1024 ? 2048 : p.block && groups < 96 ? 256 : 512);
  const int64_t splits = want < most ? want : most;
  p.splits = static_cast<int>(splits < 1 ? 1 : splits > 256 ? 256 : splits);
  const int64_t share = (span + p.splits - 1) / p.splits;
  p.chunk = static_cast<int>(share < kMinChunk ? (share + 127) / 128 * 128 : kMinChunk);
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
