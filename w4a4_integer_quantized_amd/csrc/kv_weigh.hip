// kv_weigh.hip -- attention weights added up for each cached token (rq_kv_attention_weights;
// definition in convrot.h):
//   weights[s, g, j] = keep * weights[s, g, j] + sum over query rows t and heads h of key head g of
//                      exp(softmax_scale * q_th . K_j - lse_th),  over the rows that attend to j.
//
// Mathematics. As in kv_attention.hip a logit is s_j (R q) . c_j for the held codes c_j and the rotated
// query. With lse given there is no softmax left to run: every weight is one exponential, and a sum over
// rows. So keys are what a lane owns: v_mfma_f32_16x16x32_f16 with A = 16 query rows and B = 16
// tokens puts a token in each lane, its scale a scalar of the lane, and 4 query rows in its registers; a
// token's sum stays in the lane over all rows, and no token's number ever meets another's.
// The sums are returned in binary32, so the logits have to be good to about 2^-20: queries are always
// taken as two fp16 (leading and remainder), scaled by a power of two a row. Codes are exact.
//
// A wave keeps KT times 16 tokens as fp16 operands, converted once, and walks over the query rows in tiles
// of 16, which the workgroup's four waves (four ranges of tokens) share through LDS.
//   Few rows (a decode step): bound by the K codes' bytes and the latency of reaching them through the page table.
//   The workgroup rotates the queries itself, once for all its ranges, and loads the next range's codes, and the sums
//   that were there before, ahead of its work on one; ranges in front of every row's window take no loads. 64 sequences
//   of 8192 tokens, 8 heads of 128, 4-bit codes: 62 us, 2.8 TB/s. 79 us with one range a workgroup, 65 with the sums
//   before read when they are needed, 68 with operands read four steps ahead and three waves a SIMD, 72 with KT = 4
//   (two waves), 67 with two ranges ahead. A wave's 32 tokens cost 220 vector instructions and 256 cycles of products, and
//   half the time is their issue.
//   Many: bound by the matrix instructions (two a product), and one exponential for each pair beside them. Queries are
//   rotated once, by weigh_query_kernel, into operand order. Chunks of 2048 rows over 9000 tokens, 32 heads over 8 of
//   128, four sequences: 470 us a call, 26 us of it the queries; the products, 504 GFLOP of fp16, take 403 us at the
//   rate of a large library product. Rows are shared out until there are 6000 workgroups (520 us with 3000): with 1152
//   of them, of which 768 run at once, the second turn leaves half the card without work, 636 us. Weights of one tile
//   computed between the next one's products, a barrier for two tiles, a higher priority while products run: no gain.
//   128 registers instead of 150, for a fourth workgroup on a CU, with operands read one step ahead: 512 us.
#include "kv_common.h"
#include "kv_query.h"

namespace convrot {
namespace {

using namespace kv;

constexpr float kLog2e = 1.44269504088896340736f;
constexpr int kRows = 16;      // query rows of a tile: (token, head of the group) pairs
constexpr int kWaves = 4;

// A tile of queries in memory or LDS: operand words [op][leading, rest][lane][16 B], then for each of the 16
// rows its log2-sum of exponentials (+inf: the row counts for nothing) and kCommon / (its power of two). Rows whose
// largest rotated element lies in [1/8, 1024) are scaled by kCommon, which leaves [2, 2^14) and a remainder's step
// of 2^-25 beside it; others each by a power of their own. A tile of the former only needs no factor a row.
constexpr float kCommon = 16.0f;
template <int D>
struct QueryTile {
  static constexpr int kWords = D / 32 * 2 * 1024;        // bytes of the operands
  static constexpr int kBytes = kWords + 256;             // [16 lse][16 factors], padded to one copy of 64 dwords
};

// Rotate, scale and split the rows n0 .. n0 + 15 of (sequence, key head) into `dst`; 256 threads. Rows from
// `rows` on, and rows whose lse or query is no finite number, become zeros that count for nothing.
template <int D, int BITS>
__device__ __forceinline__ void make_query_tile(const KvAttentionArgs& a, const Seq& s, int head, int n0, int rows, uint8_t* dst) {
  using R = Row<D, BITS>;
  using G = Geometry<D, BITS>;
  const int u = threadIdx.x % R::kLanes, chunk = chunk_of_lane(u), row = threadIdx.x / R::kLanes;
  const int n = n0 + row;
  const bool there = row < kRows && n < rows;
  float* const info = reinterpret_cast<float*>(dst + QueryTile<D>::kWords);
  if (__ballot(there) == 0) {   // none of this wave's rows
    if (row >= kRows) return;
#pragma unroll
    for (int k = 0; k < R::kChunks; k++) {
      constexpr int kPer = G::kLoad / BITS;
      const int ch = k * 16 + chunk, op = ch / (4 * kPer) * kPer + ch % kPer, g = ch % (4 * kPer) / kPer;
      uint8_t* p = dst + op * 2048 + (g * 16 + row) * 16;
      *reinterpret_cast<u32x4*>(p) = u32x4{0u, 0u, 0u, 0u};
      *reinterpret_cast<u32x4*>(p + 1024) = u32x4{0u, 0u, 0u, 0u};
    }
    if (u == 0) {
      info[row] = __builtin_inff();
      info[16 + row] = 1.0f;
    }
    return;
  }
  const int token = there ? token_of(a, n) : 0, qh = head * a.group + (there ? n - token * a.group : 0);
  const uint8_t* x = a.q + ((s.q0 + token) * a.q_token + qh * a.q_head) * 2;
  const float lse = there ? a.lse[(int64_t)(s.q0 + token) * a.q_heads + qh] : __builtin_inff();
  float v[R::kChunks][8], sign = 1.0f, top = 0.0f;
#pragma unroll
  for (int k = 0; k < R::kChunks; k++) {
    load8(x + (k * 128 + chunk * 8) * 2, a.dt, v[k]);
    sign = wht_block<R::kLanes>(v[k], chunk);
#pragma unroll
    for (int i = 0; i < 8; i++) {
      const float m = fabsf(v[k][i]);
      top = fmaxf(top, m < __builtin_inff() ? m : __builtin_inff());   // NaN too
    }
  }
  top = row_max<R::kLanes>(top);
  const bool ok = there && fabsf(lse) < __builtin_inff() && top < __builtin_inff();
  const float up = !ok || (top >= 0.125f && top < 1024.0f) ? kCommon : query_scale(top);
  if (row >= kRows) return;
#pragma unroll
  for (int k = 0; k < R::kChunks; k++) {
    if (!ok) {
#pragma unroll
      for (int i = 0; i < 8; i++) v[k][i] = 0.0f;
    }
    // Chunk ch of the row is the operand `op` of lane group g: operand_chunk(op, g) == ch.
    constexpr int kPer = G::kLoad / BITS;
    const int ch = k * 16 + chunk, op = ch / (4 * kPer) * kPer + ch % kPer, g = ch % (4 * kPer) / kPer;
    uint32_t w[4];
    uint8_t* p = dst + op * 2048 + (g * 16 + row) * 16;
    query_words<BITS>(v[k], sign * up, false, w);
    *reinterpret_cast<u32x4*>(p) = u32x4{w[0], w[1], w[2], w[3]};
    query_words<BITS>(v[k], sign * up, true, w);
    *reinterpret_cast<u32x4*>(p + 1024) = u32x4{w[0], w[1], w[2], w[3]};
  }
  if (u == 0) {
    info[row] = ok ? lse * kLog2e : __builtin_inff();
    info[16 + row] = kCommon / up;
  }
}

// Where the tiles of a sequence's rows begin: q0 * group / 16 + b leaves room for every sequence's last, not
// full one. Below query_tiles(), whatever q_start holds.
__device__ __forceinline__ int64_t first_tile(const KvAttentionArgs& a, const Seq& s, int b) {
  return (int64_t)s.q0 * a.group / kRows + b;
}
__device__ __forceinline__ int rows_of(const KvAttentionArgs& a, const Seq& s) {
  return (s.q_len < a.max_q ? s.q_len : a.max_q) * a.group;
}

// Query tiles of a whole call, in memory. Grid: (tile of a sequence, head, sequence).
template <int D, int BITS>
__global__ __launch_bounds__(256) void weigh_query_kernel(const KvWeighArgs w) {
  const KvAttentionArgs& a = w.a;
  const uint32_t per = (uint32_t)w.query_tiles_seq * a.heads;
  const int b = blockIdx.x / per, in = blockIdx.x - b * per;
  const int tile = in / a.heads, head = in - tile * a.heads;
  const Seq s = sequence(a, b);
  const int rows = rows_of(a, s);
  if (tile * kRows >= rows) return;
  make_query_tile<D, BITS>(a, s, head, tile * kRows, rows,
                           w.queries + ((first_tile(a, s, b) + tile) * a.heads + head) * QueryTile<D>::kBytes);
}

typedef __attribute__((address_space(3))) void lds_void;

// A wave's tokens as they come from memory.
template <int D, int BITS, int KT>
struct Raw {
  using G = Geometry<D, BITS>;
  uint32_t k[KT][G::kLoads][G::kWords];
  float scale[KT];
  uint32_t there;   // bit k: step k's page is in the cache and some of its tokens in the sequence
};

// Codes and scales of the tokens first .. first + 16 KT - 1. Lane (r, g): token r's bytes, chunk g of every 4 * kLoad.
template <int D, int BITS, int KT>
__device__ __forceinline__ void load_keys(const KvAttentionArgs& a, ConstTable table, int head, int kv_len, int first, int r, int g,
                                          Raw<D, BITS, KT>& t) {
  using R = Row<D, BITS>;
  using G = Geometry<D, BITS>;
  const int page = 1 << a.lps;
  t.there = 0;
#pragma unroll
  for (int k = 0; k < KT; k++) {
    const int j = (first + 16 * k) >> a.lps;      // past the table's end: its last entry, not used
    const int pg = table[j < a.max_pages ? j : a.max_pages - 1];
    const bool ok = pg >= 0 && pg < a.num_pages;
    t.there |= ok && first + 16 * k < kv_len ? 1u << k : 0u;
    const uint8_t* block = a.cache + ((int64_t)(ok ? pg : 0) * a.heads + head) * a.head_bytes;
    const int off = (first + 16 * k) & (page - 1);
#pragma unroll
    for (int l = 0; l < G::kLoads; l++) load_words(block + (off + r) * R::kBytes + g * G::kLoad + l * 4 * G::kLoad, t.k[k][l]);
    t.scale[k] = *reinterpret_cast<const float*>(block + 2 * page * R::kBytes + (off + r) * 4);
  }
}

// What takes a product to a logit in base 2: a token's scale, this, and kCommon / (the row's power of two).
template <int D, int BITS>
__device__ __forceinline__ float logit_factor(const KvAttentionArgs& a) { return a.scale * (kLog2e * Row<D, BITS>::kNorm / kCommon); }

// The same as operands: codes in fp16, each token's scale, and that times logit_factor().
template <int D, int BITS, int KT>
struct Keys {
  u32x4 op[KT][D / 32];
  float scale[KT], factor[KT];
};
template <int D, int BITS, int KT>
__device__ __forceinline__ void convert_keys(const KvAttentionArgs& a, const Raw<D, BITS, KT>& t, Keys<D, BITS, KT>& key) {
  using G = Geometry<D, BITS>;
#pragma unroll
  for (int k = 0; k < KT; k++) {
    // A scale that is no finite number belongs to a token that was never written.
    key.scale[k] = fabsf(t.scale[k]) < __builtin_inff() ? t.scale[k] : 0.0f;
    key.factor[k] = key.scale[k] * logit_factor<D, BITS>(a);
#pragma unroll
    for (int op = 0; op < G::kOps; op++) {
      if constexpr (BITS == 4) {
        uint32_t h[4];
        nibbles_f16(t.k[k][op / G::kWords][op % G::kWords], h);
        key.op[k][op] = u32x4{h[0], h[1], h[2], h[3]};
      } else {
        uint32_t h[2], i[2];
        bytes_f16(t.k[k][2 * op / G::kWords][2 * op % G::kWords], h);
        bytes_f16(t.k[k][(2 * op + 1) / G::kWords][(2 * op + 1) % G::kWords], i);
        key.op[k][op] = u32x4{h[0], h[1], i[0], i[1]};
      }
    }
  }
}

// The products of a tile of queries at `q` (LDS) with a wave's keys. Operands are read AHEAD steps at a time, ahead of
// the products: read one by one, each waits for LDS. (Few rows: 2, which leaves registers for a fourth wave a SIMD.)
template <int D, int BITS, int KT, int AHEAD>
__device__ __forceinline__ void multiply(const uint8_t* q, const Keys<D, BITS, KT>& key, int lane, f32x4 (&acc)[KT]) {
  constexpr int kAhead = D / 32 < AHEAD ? D / 32 : AHEAD;
#pragma unroll
  for (int k = 0; k < KT; k++) acc[k] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int o = 0; o < D / 32; o += kAhead) {
    u32x4 lead[kAhead], rest[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; i++) {
      lead[i] = *reinterpret_cast<const u32x4*>(q + (o + i) * 2048 + lane * 16);
      rest[i] = *reinterpret_cast<const u32x4*>(q + (o + i) * 2048 + 1024 + lane * 16);
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < kAhead; i++) {
#pragma unroll
      for (int k = 0; k < KT; k++) acc[k] = mfma(lead[i], key.op[k][o + i], acc[k]);
#pragma unroll
      for (int k = 0; k < KT; k++) acc[k] = mfma(rest[i], key.op[k][o + i], acc[k]);
    }
  }
}

// The rows' numbers of a tile that a lane needs: of rows 4 g .. 4 g + 3.
struct RowInfo {
  f32x4 lse, down;
};
template <int D>
__device__ __forceinline__ RowInfo row_info(const uint8_t* q, int g) {
  RowInfo i;
  i.lse = *reinterpret_cast<const f32x4*>(q + QueryTile<D>::kWords + g * 16);
  i.down = *reinterpret_cast<const f32x4*>(q + QueryTile<D>::kWords + 64 + g * 16);
  return i;
}

// Whether every row of a tile (those past the last add nothing anyway) attends to all of the tokens first .. last.
__device__ __forceinline__ int whole_tile(const KvAttentionArgs& a, int tile, int rows, int before, int first, int last) {
  int all = 1;
  if (a.causal) {
    const int n1 = tile * kRows + kRows < rows ? tile * kRows + kRows - 1 : rows - 1;
    all = before + token_of(a, tile * kRows) >= last && (a.window == 0 || before + token_of(a, n1) + 1 - a.window <= first);
  }
  return __builtin_amdgcn_readfirstlane(all);
}

// Whether all rows of a tile have the common scale.
__device__ __forceinline__ int common_scale(const RowInfo& i) {
  const bool own = i.down[0] != 1.0f || i.down[1] != 1.0f || i.down[2] != 1.0f || i.down[3] != 1.0f;
  return __builtin_amdgcn_readfirstlane(__ballot(own) == 0);
}

// A zero row's product is 0 and its lse +inf: a weight of 0 whatever the scale. Rows of another power of two may be anywhere in
// binary32 and the keys at its other end: there the product meets the token's scale first, then what is left, so that nothing
// in between is larger or smaller than both.
template <int D, int BITS, int KT>
__device__ __forceinline__ void weights_of(const KvAttentionArgs& a, f32x4 (&acc)[KT], const RowInfo& info, int common,
                                           const Keys<D, BITS, KT>& key, float (&p)[KT][4]) {
  // The wait that a read of the last product needs, before the branch: it is not added across one.
#pragma unroll
  for (int k = 0; k < KT; k++) asm volatile("" : "+v"(acc[k]));
  asm volatile("s_nop 7\n\ts_nop 3" : "+v"(acc[KT - 1]));
  if (!common) {
    const float c = logit_factor<D, BITS>(a);
#pragma unroll
    for (int k = 0; k < KT; k++)
#pragma unroll
      for (int i = 0; i < 4; i++)
        p[k][i] = __builtin_amdgcn_exp2f(__builtin_fmaf(acc[k][i] * key.scale[k], info.down[i] * c, -info.lse[i]));
    return;
  }
#pragma unroll
  for (int k = 0; k < KT; k++)
#pragma unroll
    for (int i = 0; i < 4; i++) p[k][i] = __builtin_amdgcn_exp2f(__builtin_fmaf(acc[k][i], key.factor[k], -info.lse[i]));
}

template <int KT>
__device__ __forceinline__ void add_weights(const KvAttentionArgs& a, const Seq& s, int tile, int all, int first, int r, int g,
                                            float (&p)[KT][4], float (&sum)[KT]) {
  if (!all) {
#pragma unroll
    for (int i = 0; i < 4; i++) {
      int lo, hi;
      key_range(a, s, token_of(a, tile * kRows + 4 * g + i), lo, hi);
#pragma unroll
      for (int k = 0; k < KT; k++) {
        const int j = first + 16 * k + r;
        p[k][i] = j >= lo && j < hi ? p[k][i] : 0.0f;
      }
    }
  }
#pragma unroll
  for (int k = 0; k < KT; k++) sum[k] += (p[k][0] + p[k][1]) + (p[k][2] + p[k][3]);
}

// What was there before for the token that a lane will write (see write_sums); zero where it does not count, as in a share of
// the rows (`shared`). (Loaded from somewhere in any case: a load under a condition is waited for at once.)
template <int KT>
__device__ __forceinline__ bool had_before(const KvWeighArgs& w, bool shared, const Seq& s, int first, int r, int g) {
  const int j = first + 16 * g + r;
  return !shared && w.keep != 0.0f && g < KT && j < s.kv_len && !(w.a.causal && j >= s.kv_len - s.q_len);
}
template <int KT>
__device__ __forceinline__ float load_before(const KvWeighArgs& w, bool shared, const Place& at, const Seq& s, int first, int r, int g) {
  const float* row = w.weights + ((int64_t)at.seq * w.a.heads + at.head) * ((int64_t)w.a.max_pages << w.a.lps);
  return row[had_before<KT>(w, shared, s, first, r, g) ? first + 16 * g + r : 0];
}

// Over the four lanes of a token; then lane (r, g) writes token r of step g.
template <int KT>
__device__ __forceinline__ void write_sums(const KvWeighArgs& w, bool shared, const Place& at, const Seq& s, int first, uint32_t there, int r, int g,
                                           float before, const float (&sum)[KT]) {
  const KvAttentionArgs& a = w.a;
  float mine = 0.0f;
#pragma unroll
  for (int k = 0; k < KT; k++) {
    float x = there >> k & 1 ? sum[k] : 0.0f;
    x += __shfl_xor(x, 16, 64);
    x += __shfl_xor(x, 32, 64);
    mine = g == k ? x : mine;
  }
  const int j = first + 16 * g + r;
  if (g < KT && j < s.kv_len) {
    const int64_t row = (int64_t)at.seq * a.heads + at.head, out = row * ((int64_t)a.max_pages << a.lps) + j;
    if (shared)
      w.parts[at.tile * w.part_stride + row * w.part_span + j] = mine;
    else
      w.weights[out] = had_before<KT>(w, shared, s, first, r, g) ? __builtin_fmaf(w.keep, before, mine) : mine;
  }
}

// Shares of the query rows: the most, and the fewest tiles of one. (One sequence of 2844 tokens, 16 heads over one: 198 us
// with 16 shares, 78 with 64; 4 or 16 tiles change calls of a few hundred rows by a tenth either way.)
constexpr int kMostShares = 64, kLeastTiles = 8;
constexpr int kFewTiles = 2;   // query tiles that a workgroup makes itself

// Few query rows: the workgroup makes the query tiles once and walks over its ranges of tokens (number `split`
// and every a.splits-th after), the next range's codes on their way meanwhile.
template <int D, int BITS, int KT>
__global__ __launch_bounds__(256, 2) void weigh_few_kernel(const KvWeighArgs w) {
  using Q = QueryTile<D>;
  constexpr int kKeys = kWaves * KT * 16;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[kFewTiles * Q::kBytes];
  const KvAttentionArgs& a = w.a;
  const Place at = place(a);
  if (at.seq >= a.seqs) return;
  const Seq s = sequence(a, at.seq);
  const int64_t step = (int64_t)a.splits * kKeys;
  int64_t base = (int64_t)at.split * kKeys;
  if (base >= s.kv_len) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int rows = rows_of(a, s), before = s.kv_len - s.q_len, tiles = (rows + kRows - 1) / kRows;   // at most kFewTiles
  const ConstTable table = const_table(a.pages) + (int64_t)at.seq * a.max_pages;
  // Tokens before lo are outside every row's window: ranges of them take no part but in what was there before.
  const int lo = a.causal && a.window > 0 && before + 1 - a.window > 0 ? before + 1 - a.window : 0;
  for (; base < s.kv_len && base + kKeys <= lo; base += step) {
    float none[KT] = {};
    const int first = static_cast<int>(base) + wave * (KT * 16);
    write_sums<KT>(w, false, at, s, first, 0, r, g, load_before<KT>(w, false, at, s, first, r, g), none);
  }
  if (base >= s.kv_len) return;
  // A range's codes and what was there before; past the last range the last again.
  Raw<D, BITS, KT> next;
  float next_was;
  auto load = [&](int64_t at_base) __attribute__((always_inline)) {
    const int first = static_cast<int>(at_base < s.kv_len ? at_base : base) + wave * (KT * 16);
    next_was = load_before<KT>(w, false, at, s, first, r, g);
    load_keys<D, BITS, KT>(a, table, at.head, s.kv_len, first, r, g, next);
  };
  load(base);
  for (int tile = 0; tile < tiles; tile++) make_query_tile<D, BITS>(a, s, at.head, tile * kRows, rows, lds + tile * Q::kBytes);
  __syncthreads();
  for (; base < s.kv_len; base += step) {
    const int first = static_cast<int>(base) + wave * (KT * 16);
    Keys<D, BITS, KT> key;
    convert_keys<D, BITS, KT>(a, next, key);
    const uint32_t there = next.there;
    const float was = next_was;
    load(base + step);
    float sum[KT];
#pragma unroll
    for (int k = 0; k < KT; k++) sum[k] = 0.0f;
    for (int tile = 0; tile < tiles; tile++) {
      int all = whole_tile(a, tile, rows, before, first, first + KT * 16 - 1);
      const uint8_t* q = lds + tile * Q::kBytes;
      const RowInfo info = row_info<D>(q, g);
      int common = common_scale(info);
      asm volatile("" : "+s"(all), "+s"(common));   // settled before the products
      f32x4 acc[KT];
      float p[KT][4];
      multiply<D, BITS, KT, 2>(q, key, lane, acc);
      weights_of<D, BITS, KT>(a, acc, info, common, key, p);
      add_weights<KT>(a, s, tile, all, first, r, g, p, sum);
    }
    write_sums<KT>(w, false, at, s, first, there, r, g, was, sum);
  }
}

// Many query rows: tiles come from memory, made by weigh_query_kernel, copied to a ring in LDS three ahead.
// a.row_tiles workgroups share a range's rows, up to token w.part_span; behind it, where the lengths that the plan was made for
// have ended, the first of them takes all.
template <int D, int BITS>
__global__ __launch_bounds__(256, 2) void weigh_many_kernel(const KvWeighArgs w) {
  using Q = QueryTile<D>;
  constexpr int KT = 4, kKeys = kWaves * KT * 16;
  constexpr int kRing = 4, kCopies = Q::kWords / 1024 / kWaves + 1;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[kRing * Q::kBytes];
  const KvAttentionArgs& a = w.a;
  const Place at = place(a);
  if (at.seq >= a.seqs) return;
  const Seq s = sequence(a, at.seq);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int rows = rows_of(a, s), before = s.kv_len - s.q_len;   // position of the first query row
  const ConstTable table = const_table(a.pages) + (int64_t)at.seq * a.max_pages;
  const uint8_t* const queries = w.queries + (first_tile(a, s, at.seq) * a.heads + at.head) * Q::kBytes;
  // (Buffer copies: the compiler takes the other kind for LDS accesses and waits for them before each read.)
  auto fetch = [&](int tile, int buffer) __attribute__((always_inline)) {
    const __amdgpu_buffer_rsrc_t src = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint8_t*>(queries + (int64_t)tile * a.heads * Q::kBytes), (short)0, Q::kBytes, 0x00020000);
    uint8_t* dst = lds + buffer * Q::kBytes;
#pragma unroll
    for (int i = 0; i < Q::kWords / 1024 / kWaves; i++) {
      const int c = wave * (Q::kWords / 1024 / kWaves) + i;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(src, (lds_void*)(dst + c * 1024), 16, lane * 16, c * 1024, 0, 0);
    }
    // Every wave copies the rows' numbers, to the same place.
    __builtin_amdgcn_raw_ptr_buffer_load_lds(src, (lds_void*)(dst + Q::kWords), 4, lane * 4, Q::kWords, 0, 0);
  };

  for (int64_t base = (int64_t)at.split * kKeys; base < s.kv_len; base += (int64_t)a.splits * kKeys) {
    const int key0 = static_cast<int>(base), first = key0 + wave * (KT * 16);   // the workgroup's, the wave's
    const bool shared = a.row_tiles > 1 && base < w.part_span;
    if (!shared && at.tile > 0) break;
    // The tiles of rows that attend to some token of the workgroup's range, and this workgroup's share.
    int t0 = 0, t1 = (rows + kRows - 1) / kRows;
    if (a.causal) {
      const int lo_token = key0 - before;             // rows before it end in front of the range
      if (lo_token > 0) {
        const int64_t n = (int64_t)lo_token * a.group / kRows;
        t0 = n < t1 ? static_cast<int>(n) : t1;
      }
      if (a.window > 0) {
        const int64_t hi_token = (int64_t)key0 + kKeys - 1 + a.window - before;   // the first whose window begins behind it
        const int64_t n = hi_token <= 0 ? 0 : (hi_token * a.group + kRows - 1) / kRows;
        t1 = n < t1 ? static_cast<int>(n) : t1;
      }
    }
    if (shared && t1 > t0) {
      const int share = (t1 - t0 + a.row_tiles - 1) / a.row_tiles;
      t0 += at.tile * share;
      t1 = t0 + share < t1 ? t0 + share : t1;
    }
    float sum[KT];
#pragma unroll
    for (int k = 0; k < KT; k++) sum[k] = 0.0f;
    if (t0 >= t1) {   // the same for the whole workgroup
      write_sums<KT>(w, shared, at, s, first, 0, r, g, load_before<KT>(w, shared, at, s, first, r, g), sum);
      continue;
    }
    Raw<D, BITS, KT> raw;
    load_keys<D, BITS, KT>(a, table, at.head, s.kv_len, first, r, g, raw);
#pragma unroll
    for (int i = 0; i < kRing - 1; i++)
      if (t0 + i < t1) fetch(t0 + i, i);
    Keys<D, BITS, KT> key;
    convert_keys<D, BITS, KT>(a, raw, key);
    for (int tile = t0; tile < t1; tile++) {
      const int buffer = (tile - t0) % kRing;
      // This wave's part of the tile is there (those of the next two may be under way), then everybody's, and
      // the buffer of the tile before is done with: its reads were waited for before their products.
      if (tile + 2 < t1) {
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"(2 * kCopies) : "memory");
      } else if (tile + 1 < t1) {
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"(kCopies) : "memory");
      } else {
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      __builtin_amdgcn_s_barrier();
      __builtin_amdgcn_sched_barrier(0);
      if (tile + kRing - 1 < t1) fetch(tile + kRing - 1, (buffer + kRing - 1) % kRing);
      const uint8_t* q = lds + buffer * Q::kBytes;
      const RowInfo info = row_info<D>(q, g);
      int all = whole_tile(a, tile, rows, before, first, first + KT * 16 - 1), common = common_scale(info);
      asm volatile("" : "+s"(all), "+s"(common));
      f32x4 acc[KT];
      float p[KT][4];
      multiply<D, BITS, KT, 4>(q, key, lane, acc);
      weights_of<D, BITS, KT>(a, acc, info, common, key, p);
      add_weights<KT>(a, s, tile, all, first, r, g, p, sum);
    }
    __syncthreads();   // the buffers are done with before the next range's first copy
    write_sums<KT>(w, shared, at, s, first, raw.there, r, g, load_before<KT>(w, shared, at, s, first, r, g), sum);
  }
}

// The shares of rows of each token added up, in order.
__global__ __launch_bounds__(256) void weigh_join_kernel(const KvWeighArgs w) {
  const KvAttentionArgs& a = w.a;
  const int64_t span = (int64_t)a.max_pages << a.lps;
  const int b = blockIdx.y / a.heads;
  const Seq s = sequence(a, b);
  const int before = s.kv_len - s.q_len;
  const int64_t end = s.kv_len < w.part_span ? s.kv_len : w.part_span;
  for (int64_t j = (int64_t)blockIdx.x * 256 + threadIdx.x; j < end; j += (int64_t)gridDim.x * 256) {
    const int64_t out = (int64_t)blockIdx.y * span + j, part = (int64_t)blockIdx.y * w.part_span + j;
    float sum = 0.0f;
#pragma unroll 8
    for (int t = 0; t < a.row_tiles; t++) sum += w.parts[t * w.part_stride + part];
    const bool had = w.keep != 0.0f && !(a.causal && j >= before);
    w.weights[out] = had ? __builtin_fmaf(w.keep, w.weights[out], sum) : sum;
  }
}

template <int D, int BITS>
hipError_t launch(const KvWeighArgs& w, int kt, bool many, hipStream_t st) {
  const KvAttentionArgs& a = w.a;
  if (many) {
    hipLaunchKernelGGL((weigh_query_kernel<D, BITS>), dim3((unsigned)((int64_t)a.seqs * w.query_tiles_seq * a.heads)), dim3(256), 0, st, w);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const int64_t pairs = ((int64_t)a.seqs * a.splits + kXcds - 1) / kXcds * kXcds;
  const dim3 grid((unsigned)(pairs * a.heads * a.row_tiles)), block(256);
  if (many)
    hipLaunchKernelGGL((weigh_many_kernel<D, BITS>), grid, block, 0, st, w);
  else if (kt == 1)
    hipLaunchKernelGGL((weigh_few_kernel<D, BITS, 1>), grid, block, 0, st, w);
  else
    hipLaunchKernelGGL((weigh_few_kernel<D, BITS, 2>), grid, block, 0, st, w);
  if (a.row_tiles > 1) {
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(weigh_join_kernel, dim3((unsigned)w.join_blocks, (unsigned)(a.seqs * a.heads)), dim3(256), 0, st, w);
  }
  return hipGetLastError();
}

}  // namespace

KvWeighPlan plan_kv_weigh(int64_t total_q, int seqs, int q_heads, int heads, int head_dim, int64_t max_q_len, int64_t max_kv_len) {
  KvWeighPlan p = {};
  const int64_t group = q_heads / heads;
  p.query_tiles_seq = (max_q_len * group + kRows - 1) / kRows;
  // Above 32 rows queries are rotated once for all. (Two tiles of them fit beside the codes; see the top for the rest.)
  p.many = p.query_tiles_seq > kFewTiles;
  p.kt = p.many ? 4 : 2;
  auto ranges = [&] { return (max_kv_len + kWaves * 16 * p.kt - 1) / (kWaves * 16 * p.kt); };
  if (!p.many)
    if (ranges() * seqs * heads < 1024) p.kt = 1;
  p.splits = ranges() < 1 ? 1 : ranges();
  if (!p.many) {
    const int64_t pairs = (int64_t)seqs * heads, want = (4096 + pairs - 1) / pairs;
    if (p.splits > want) p.splits = want;
  }
  p.row_splits = 1;
  if (p.many) {
    const int64_t groups = p.splits * seqs * heads, want = (6000 + groups - 1) / groups, most = p.query_tiles_seq / kLeastTiles;
    p.row_splits = want < most ? want : most;
    if (p.row_splits > kMostShares) p.row_splits = kMostShares;
    if (p.row_splits < 1) p.row_splits = 1;
    p.query_bytes = ((total_q * group / kRows + seqs + 1) * heads * (head_dim / 32 * 2048 + 256) + 255) / 256 * 256;
    // Sums of each share for the tokens of the plan's ranges: with the 6000 workgroups above 12 MB at most. (Not for the page
    // table's, which may be far wider than any sequence is long: 2048 rows over 2048 tokens, 32 heads over 8, take 82 to 88 us
    // with tables of 2048 to 2^20 tokens; unshared 394.)
    p.part_span = p.splits * (kWaves * 16 * p.kt);
    if (p.row_splits > 1) p.part_bytes = p.row_splits * seqs * heads * p.part_span * 4;
  }
  return p;
}

hipError_t launch_kv_weigh(const KvWeighArgs& w, int head_dim, int bits, int kt, bool many, hipStream_t stream) {
  switch (head_dim) {
    case 64: return bits == 8 ? launch<64, 8>(w, kt, many, stream) : launch<64, 4>(w, kt, many, stream);
    case 128: return bits == 8 ? launch<128, 8>(w, kt, many, stream) : launch<128, 4>(w, kt, many, stream);
    default: return bits == 8 ? launch<256, 8>(w, kt, many, stream) : launch<256, 4>(w, kt, many, stream);
  }
}

}  // namespace convrot
