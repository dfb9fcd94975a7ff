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
// of 16, which the workgroup's four waves (four ranges of tokens) share through LDS. Few rows (a
// decode step): bound by the K codes' bytes; the workgroup rotates the queries itself. Many: bound by the
// matrix instructions (two a product) and one exponential for each pair beside them; queries are rotated once, by
// weigh_query_kernel, into operand order, and tiles are copied to LDS one ahead.
#include "kv_common.h"
#include "kv_query.h"

namespace convrot {
namespace {

using namespace kv;

constexpr float kLog2e = 1.44269504088896340736f;
constexpr int kRows = 16;      // query rows of a tile: (token, head of the group) pairs
constexpr int kWaves = 4;

// A tile of queries in memory or LDS: operand words [op][leading, rest][lane][16 B], then for each of the 16
// rows its log2-sum of exponentials (+inf: the row counts for nothing) and 1 / (its power of two).
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
  const float up = ok ? query_scale(top) : 1.0f;
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
    float* info = reinterpret_cast<float*>(dst + QueryTile<D>::kWords);
    info[row] = ok ? lse * kLog2e : __builtin_inff();
    info[16 + row] = ok ? 1.0f / up : 0.0f;
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

// Tokens of the workgroup's range number `split` (and, past a hint that was too small, every a.splits-th after).
// PREP: query tiles come from memory; else the workgroup makes them.
template <int D, int BITS, int KT, bool PREP>
__global__ __launch_bounds__(256, 2) void weigh_kernel(const KvWeighArgs w) {
  using R = Row<D, BITS>;
  using G = Geometry<D, BITS>;
  using Q = QueryTile<D>;
  constexpr int kKeys = kWaves * KT * 16;
  constexpr int kBuffers = PREP ? 2 : 1;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[kBuffers * Q::kBytes];
  const KvAttentionArgs& a = w.a;
  const Place at = place(a);
  if (at.seq >= a.seqs) return;
  const Seq s = sequence(a, at.seq);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int rows = rows_of(a, s), before = s.kv_len - s.q_len;   // position of the first query row
  const int page = 1 << a.lps;
  const ConstTable table = const_table(a.pages) + (int64_t)at.seq * a.max_pages;

  for (int64_t base = (int64_t)at.split * kKeys; base < s.kv_len; base += (int64_t)a.splits * kKeys) {
    const int key0 = static_cast<int>(base), first = key0 + wave * (KT * 16);   // the workgroup's, the wave's
    // The codes and scales of this wave's tokens. Lane (r, g): token r's bytes, chunk g of every 4 * kLoad.
    uint32_t raw[KT][G::kLoads][G::kWords];
    float ks[KT];
    bool there[KT];
#pragma unroll
    for (int k = 0; k < KT; k++) {
      const int j = (first + 16 * k) >> a.lps;      // past the table's end: its last entry, not used
      const int pg = table[j < a.max_pages ? j : a.max_pages - 1];
      there[k] = pg >= 0 && pg < a.num_pages && first + 16 * k < s.kv_len;
      const uint8_t* block = a.cache + ((int64_t)(there[k] ? pg : 0) * a.heads + at.head) * a.head_bytes;
      const int off = (first + 16 * k) & (page - 1);
#pragma unroll
      for (int l = 0; l < G::kLoads; l++)
        load_words(block + (off + r) * R::kBytes + g * G::kLoad + l * 4 * G::kLoad, raw[k][l]);
      ks[k] = *reinterpret_cast<const float*>(block + 2 * page * R::kBytes + (off + r) * 4);
    }
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
    if (a.row_tiles > 1 && t1 > t0) {
      const int share = (t1 - t0 + a.row_tiles - 1) / a.row_tiles;
      t0 += at.tile * share;
      t1 = t0 + share < t1 ? t0 + share : t1;
    }
    const uint8_t* const queries = PREP ? w.queries + (first_tile(a, s, at.seq) * a.heads + at.head) * Q::kBytes : nullptr;
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
    if (PREP && t0 < t1) fetch(t0, 0);

    u32x4 key[KT][G::kOps];
    float factor[KT], sum[KT];
#pragma unroll
    for (int k = 0; k < KT; k++) {
      // A scale that is no finite number belongs to a token that was never written.
      factor[k] = fabsf(ks[k]) < __builtin_inff() ? ks[k] * (a.scale * (kLog2e * R::kNorm)) : 0.0f;
      sum[k] = 0.0f;
#pragma unroll
      for (int op = 0; op < G::kOps; op++) {
        if constexpr (BITS == 4) {
          uint32_t h[4];
          nibbles_f16(raw[k][op / G::kWords][op % G::kWords], h);
          key[k][op] = u32x4{h[0], h[1], h[2], h[3]};
        } else {
          uint32_t h[2], i[2];
          bytes_f16(raw[k][2 * op / G::kWords][2 * op % G::kWords], h);
          bytes_f16(raw[k][(2 * op + 1) / G::kWords][(2 * op + 1) % G::kWords], i);
          key[k][op] = u32x4{h[0], h[1], i[0], i[1]};
        }
      }
    }

    for (int tile = t0; tile < t1; tile++) {
      const int buffer = PREP ? (tile - t0) & 1 : 0;
      if constexpr (PREP) {
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // this wave's part of the tile is there,
        __syncthreads();                                    // and everybody's; the other buffer is done with
        if (tile + 1 < t1) fetch(tile + 1, buffer ^ 1);
      } else {
        __syncthreads();                                    // the tile before is done with
        make_query_tile<D, BITS>(a, s, at.head, tile * kRows, rows, lds);
        __syncthreads();
      }
      // Does every row of the tile (those past the last add nothing anyway) attend to all of the wave's tokens?
      int all = 1;
      if (a.causal) {
        const int n1 = tile * kRows + kRows < rows ? tile * kRows + kRows - 1 : rows - 1;
        all = before + token_of(a, tile * kRows) >= first + KT * 16 - 1 &&
              (a.window == 0 || before + token_of(a, n1) + 1 - a.window <= first);
      }
      all = __builtin_amdgcn_readfirstlane(all);
      asm volatile("" : "+s"(all));   // settled before the products: no branch between them and their first use
      const uint8_t* q = lds + buffer * Q::kBytes;
      f32x4 acc[KT];
#pragma unroll
      for (int k = 0; k < KT; k++) acc[k] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int op = 0; op < G::kOps; op++) {
        const u32x4 lead = *reinterpret_cast<const u32x4*>(q + op * 2048 + lane * 16);
        const u32x4 rest = *reinterpret_cast<const u32x4*>(q + op * 2048 + 1024 + lane * 16);
#pragma unroll
        for (int k = 0; k < KT; k++) acc[k] = mfma(lead, key[k][op], acc[k]);
#pragma unroll
        for (int k = 0; k < KT; k++) acc[k] = mfma(rest, key[k][op], acc[k]);
      }
      const f32x4 lse = *reinterpret_cast<const f32x4*>(q + Q::kWords + g * 16);
      const f32x4 down = *reinterpret_cast<const f32x4*>(q + Q::kWords + 64 + g * 16);
      float p[KT][4];
#pragma unroll
      for (int k = 0; k < KT; k++)
#pragma unroll
        for (int i = 0; i < 4; i++)
          p[k][i] = __builtin_amdgcn_exp2f(__builtin_fmaf(acc[k][i] * down[i], factor[k], -lse[i]));
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
    if constexpr (PREP) __syncthreads();   // both buffers are done with before the next range's first copy

    // Over the four lanes of a token; then lane (r, g) writes token r of step g.
    float mine = 0.0f;
#pragma unroll
    for (int k = 0; k < KT; k++) {
      float x = there[k] ? sum[k] : 0.0f;
      x += __shfl_xor(x, 16, 64);
      x += __shfl_xor(x, 32, 64);
      mine = g == k ? x : mine;
    }
    const int j = first + 16 * g + r;
    if (g < KT && j < s.kv_len) {
      const int64_t out = ((int64_t)at.seq * a.heads + at.head) * ((int64_t)a.max_pages << a.lps) + j;
      if (a.row_tiles > 1) {
        w.parts[at.tile * w.part_stride + out] = mine;
      } else {
        const bool had = w.keep != 0.0f && !(a.causal && j >= before);
        w.weights[out] = had ? __builtin_fmaf(w.keep, w.weights[out], mine) : mine;
      }
    }
  }
}

// The shares of rows of each token added up, in order.
__global__ __launch_bounds__(256) void weigh_join_kernel(const KvWeighArgs w) {
  const KvAttentionArgs& a = w.a;
  const int64_t span = (int64_t)a.max_pages << a.lps;
  const int b = blockIdx.y / a.heads;
  const Seq s = sequence(a, b);
  const int before = s.kv_len - s.q_len;
  for (int64_t j = (int64_t)blockIdx.x * 256 + threadIdx.x; j < s.kv_len; j += (int64_t)gridDim.x * 256) {
    const int64_t out = (int64_t)blockIdx.y * span + j;
    float sum = 0.0f;
    for (int t = 0; t < a.row_tiles; t++) sum += w.parts[t * w.part_stride + out];
    const bool had = w.keep != 0.0f && !(a.causal && j >= before);
    w.weights[out] = had ? __builtin_fmaf(w.keep, w.weights[out], sum) : sum;
  }
}

template <int D, int BITS, int KT, bool PREP>
hipError_t launch_kt(const KvWeighArgs& w, hipStream_t st) {
  const KvAttentionArgs& a = w.a;
  if constexpr (PREP) {
    hipLaunchKernelGGL((weigh_query_kernel<D, BITS>), dim3((unsigned)((int64_t)a.seqs * w.query_tiles_seq * a.heads)), dim3(256), 0, st, w);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const int64_t pairs = ((int64_t)a.seqs * a.splits + kXcds - 1) / kXcds * kXcds;
  hipLaunchKernelGGL((weigh_kernel<D, BITS, KT, PREP>), dim3((unsigned)(pairs * a.heads * a.row_tiles)), dim3(256), 0, st, w);
  if (a.row_tiles > 1) {
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(weigh_join_kernel, dim3((unsigned)w.join_blocks, (unsigned)(a.seqs * a.heads)), dim3(256), 0, st, w);
  }
  return hipGetLastError();
}

template <int D, int BITS>
hipError_t launch(const KvWeighArgs& w, int kt, bool prep, hipStream_t st) {
  if (prep) return launch_kt<D, BITS, 4, true>(w, st);
  return kt == 4 ? launch_kt<D, BITS, 4, false>(w, st) : kt == 2 ? launch_kt<D, BITS, 2, false>(w, st) : launch_kt<D, BITS, 1, false>(w, st);
}

}  // namespace

KvWeighPlan plan_kv_weigh(int64_t total_q, int seqs, int q_heads, int heads, int head_dim, int64_t max_q_len, int64_t max_kv_len,
                          int64_t span) {
  KvWeighPlan p = {};
  const int64_t group = q_heads / heads;
  p.query_tiles_seq = (max_q_len * group + kRows - 1) / kRows;
  // Above 32 rows queries are rotated once for all.
  p.prep = p.query_tiles_seq > 2;
  p.kt = 4;
  auto ranges = [&] { return (max_kv_len + kWaves * 16 * p.kt - 1) / (kWaves * 16 * p.kt); };
  if (!p.prep)
    while (p.kt > 1 && ranges() * seqs * heads < 1024) p.kt /= 2;
  p.splits = ranges() < 1 ? 1 : ranges();
  p.row_splits = 1;
  if (p.prep) {
    const int64_t groups = p.splits * seqs * heads, want = (512 + groups - 1) / groups, most = p.query_tiles_seq / 8;
    p.row_splits = want < most ? want : most;
    if (p.row_splits > 16) p.row_splits = 16;
    if (p.row_splits < 1) p.row_splits = 1;
    p.query_bytes = ((total_q * group / kRows + seqs + 1) * heads * (head_dim / 32 * 2048 + 256) + 255) / 256 * 256;
    // Sums of each share for the whole page table: not where that is much.
    if (p.row_splits > 1 && p.row_splits * seqs * heads * span > (int64_t(1) << 26)) p.row_splits = 1;
    if (p.row_splits > 1) p.part_bytes = p.row_splits * seqs * heads * span * 4;
  }
  return p;
}

hipError_t launch_kv_weigh(const KvWeighArgs& w, int head_dim, int bits, int kt, bool prep, hipStream_t stream) {
  switch (head_dim) {
    case 64: return bits == 8 ? launch<64, 8>(w, kt, prep, stream) : launch<64, 4>(w, kt, prep, stream);
    case 128: return bits == 8 ? launch<128, 8>(w, kt, prep, stream) : launch<128, 4>(w, kt, prep, stream);
    default: return bits == 8 ? launch<256, 8>(w, kt, prep, stream) : launch<256, 4>(w, kt, prep, stream);
  }
}

}  // namespace convrot
