// kv_evict.hip -- a cache brought down to a budget of tokens (rq_kv_evict; definition in convrot.h): for each
// sequence and key head the tokens that stay are chosen by their weights, and their codes and scales are
// written, in order, into new pages.
//
// evict_select_kernel: a workgroup a (sequence, key head). The weight of the last token that still fits
// is found digit by digit (11, 11 and 10 bits of the weights as ordered integers, a histogram of 2048 counters in LDS for
// each), then one pass in order writes the indices: everything above that weight, and of those beside it the
// first. Counters are integers: the same choice every time.
// evict_move_kernel: bound by memory. Bytes are moved as they are. K rows and scales are copied; V bytes lie four
// tokens side by side, so each four new tokens gather a byte from each of four old groups: a lone token
// that stays costs the reading of its whole group's V lines.
#include "kv_common.h"

namespace convrot {
namespace {

using namespace kv;

constexpr int kSelectThreads = 1024, kSelectWaves = kSelectThreads / 64;
constexpr int kBins = 2048;
constexpr int kMoveTokens = 64;   // new tokens of a move workgroup

typedef float f32x4u __attribute__((ext_vector_type(4)));

__device__ __forceinline__ int kv_length(const KvEvictArgs& a, int b) {
  const int n = a.kv_len[b], most = a.max_pages << a.lps;
  return n < 0 ? 0 : n > most ? most : n;
}

// Weights as integers of the same order; a NaN is below all, -0 is 0.
__device__ __forceinline__ uint32_t order_key(float w) {
  w += 0.0f;
  const uint32_t u = __float_as_uint(w);
  const uint32_t k = u & 0x80000000u ? ~u : u | 0x80000000u;
  return w == w ? k : 0u;
}

// Inclusive sum over a wave's lanes.
__device__ __forceinline__ uint32_t wave_scan(uint32_t x, int lane) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) {
    const uint32_t y = __shfl_up(x, m, 64);
    x += lane >= m ? y : 0u;
  }
  return x;
}

__global__ __launch_bounds__(kSelectThreads) void evict_select_kernel(const KvEvictArgs a) {
  __shared__ uint32_t bins[kBins];
  __shared__ uint32_t part[2][kSelectWaves];
  __shared__ uint32_t found[2];    // a digit, and how many are still wanted of those that have it
  const int b = blockIdx.x / a.heads, head = blockIdx.x - b * a.heads;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int n = kv_length(a, b);
  int32_t* const kept = a.kept + (int64_t)blockIdx.x * a.budget;
  const float* const weights = a.weights + (int64_t)blockIdx.x * ((int64_t)a.max_pages << a.lps);
  float* const out = a.new_weights ? a.new_weights + (int64_t)blockIdx.x * ((int64_t)a.new_max_pages << a.lps) : nullptr;
  if (head == 0 && tid == 0) a.new_kv_len[b] = n < a.budget ? n : a.budget;
  if (n <= a.budget) {
    for (int i = tid; i < a.budget; i += kSelectThreads) {
      kept[i] = i < n ? i : -1;
      if (out && i < n) out[i] = weights[i];
    }
    return;
  }
  // Tokens [lo, hi) are chosen from, `want` of them; those around stay. Rows begin at multiples of 16 floats.
  const int lo = a.first, hi = n - a.recent;
  uint32_t want = a.budget - a.first - a.recent;
  uint32_t prefix = 0, edge = 0;
  const bool choose = want > 0;     // the same for the whole workgroup
  if (choose) {
    for (int digit = 0; digit < 3; digit++) {
      const int shift = digit == 0 ? 21 : digit == 1 ? 10 : 0, bits = digit == 2 ? 10 : 11;
      for (int i = tid; i < kBins; i += kSelectThreads) bins[i] = 0;
      __syncthreads();
      for (int base = 0; base < hi; base += 4 * kSelectThreads) {
        const int j = base + 4 * tid;
        f32x4u w = {0.0f, 0.0f, 0.0f, 0.0f};
        if (j < hi) w = *reinterpret_cast<const f32x4u*>(weights + j);   // up to 3 past hi: within the row
#pragma unroll
        for (int e = 0; e < 4; e++) {
          const uint32_t key = order_key(w[e]);
          const bool in = j + e >= lo && j + e < hi && (digit == 0 || key >> (shift + bits) == prefix);
          const uint32_t bin = key >> shift & ((1u << bits) - 1);
          // Lanes that meet the first lane's counter add to it together: weights of one size, zeros above all.
          const uint64_t active = __ballot(in);
          if (active == 0) continue;
          const int leader = __builtin_ctzll(active);
          const uint32_t same = __shfl(bin, leader, 64);
          const uint64_t with = __ballot(in && bin == same);
          if (lane == leader) atomicAdd(&bins[same], (uint32_t)__builtin_popcountll(with));
          if (in && bin != same) atomicAdd(&bins[bin], 1u);
        }
      }
      __syncthreads();
      // The counter, from the top, in which the want-th lies: thread t has the counters 2047 - 2t and the next.
      const uint32_t c0 = bins[kBins - 1 - 2 * tid], c1 = bins[kBins - 2 - 2 * tid];
      const uint32_t incl = wave_scan(c0 + c1, lane);
      if (lane == 63) part[0][wave] = incl;
      __syncthreads();
      uint32_t before = incl - c0 - c1;
      for (int v = 0; v < wave; v++) before += part[0][v];
      if (before < want && before + c0 >= want) {
        found[0] = kBins - 1 - 2 * tid;
        found[1] = want - before;
      } else if (before + c0 < want && before + c0 + c1 >= want) {
        found[0] = kBins - 2 - 2 * tid;
        found[1] = want - before - c0;
      }
      __syncthreads();
      prefix = digit == 0 ? found[0] : prefix << bits | found[0];
      want = found[1];
      __syncthreads();
    }
    edge = prefix;
  }
  // In order: what lies around, what is above the edge, and the first `want` beside it.
  uint32_t above_so_far = 0, beside_so_far = 0;
  for (int base = 0; base < n; base += 4 * kSelectThreads) {
    const int j = base + 4 * tid;
    f32x4u w = {0.0f, 0.0f, 0.0f, 0.0f};
    if (j < n) w = *reinterpret_cast<const f32x4u*>(weights + j);
    uint32_t above = 0, beside = 0;    // a bit a token
#pragma unroll
    for (int e = 0; e < 4; e++) {
      const uint32_t key = order_key(w[e]);
      const bool around = j + e < lo || j + e >= hi;
      if (j + e < n && (around || (choose && key > edge))) above |= 1u << e;
      if (j + e < n && !around && choose && key == edge) beside |= 1u << e;
    }
    const uint32_t counts = (uint32_t)__builtin_popcount(above) | (uint32_t)__builtin_popcount(beside) << 16;
    const uint32_t incl = wave_scan(counts, lane);    // at most 256 in each half
    if (lane == 63) part[(base / (4 * kSelectThreads)) & 1][wave] = incl;
    __syncthreads();    // (the other half of `part` is read by nobody any more at the next write of this one)
    uint32_t total = 0, ahead = incl - counts;
    for (int v = 0; v < kSelectWaves; v++) {
      const uint32_t x = part[(base / (4 * kSelectThreads)) & 1][v];
      if (v < wave) ahead += x;
      total += x;        // at most 4096 in each half
    }
    uint32_t up = above_so_far + (ahead & 0xFFFFu), at_edge = beside_so_far + (ahead >> 16);
#pragma unroll
    for (int e = 0; e < 4; e++) {
      const bool is_above = above >> e & 1, is_beside = beside >> e & 1;
      if (is_above || (is_beside && at_edge < want)) {
        const uint32_t at = up + (at_edge < want ? at_edge : want);
        kept[at] = j + e;
        if (out) out[at] = w[e];
      }
      up += is_above;
      at_edge += is_beside;
    }
    above_so_far += total & 0xFFFFu;
    beside_so_far += total >> 16;
  }
}

// The head's block of a page of a table, or null.
__device__ __forceinline__ uint8_t* block_of(const KvEvictArgs& a, const int32_t* table, int token, int head) {
  const int pg = table[token >> a.lps];
  return pg >= 0 && pg < a.num_pages ? a.cache + ((int64_t)pg * a.heads + head) * a.head_bytes : nullptr;
}

// New tokens [64 c, 64 c + 64) of a (sequence, key head). RB: bytes of a row of codes.
template <int RB>
__global__ __launch_bounds__(256) void evict_move_kernel(const KvEvictArgs a) {
  const int tid = threadIdx.x, page = 1 << a.lps;
  const int head = blockIdx.x % a.heads, rest = blockIdx.x / a.heads, chunk = rest % a.chunks, b = rest / a.chunks;
  const int n = kv_length(a, b), count = n < a.budget ? n : a.budget, i0 = chunk * kMoveTokens;
  if (i0 >= count) return;
  const int32_t* const kept = a.kept + ((int64_t)b * a.heads + head) * a.budget;
  const int32_t* const from = a.pages + (int64_t)b * a.max_pages;
  const int32_t* const to = a.new_pages + (int64_t)b * a.new_max_pages;
  // K rows: 16 bytes a thread.
  constexpr int kPer = RB / 16;
#pragma unroll
  for (int job = tid; job < kMoveTokens * kPer; job += 256) {
    const int i = i0 + job / kPer, at = job % kPer * 16;
    if (i < count) {
      const int j = kept[i];
      const uint8_t* src = block_of(a, from, j, head);
      uint8_t* dst = block_of(a, to, i, head);
      u32x4 x = {0u, 0u, 0u, 0u};
      if (src) x = *reinterpret_cast<const u32x4*>(src + (j & (page - 1)) * RB + at);
      if (dst) *reinterpret_cast<u32x4*>(dst + (i & (page - 1)) * RB + at) = x;
    }
  }
  // V: four new tokens and four of their bytes a thread.
  constexpr int kQuads = RB / 4;
#pragma unroll
  for (int job = tid; job < kMoveTokens / 4 * kQuads; job += 256) {
    const int i = i0 + job / kQuads * 4, at = job % kQuads * 16;
    if (i < count) {
      uint8_t* dst = block_of(a, to, i, head);
      u32x4 x[4];
      uint32_t sel[4], keep = 0;
#pragma unroll
      for (int e = 0; e < 4; e++) {
        x[e] = u32x4{0u, 0u, 0u, 0u};
        sel[e] = 0;
        if (i + e < count) {
          const int j = kept[i + e], off = j & (page - 1);
          const uint8_t* src = block_of(a, from, j, head);
          if (src) x[e] = *reinterpret_cast<const u32x4*>(src + page * RB + (off >> 2) * (4 * RB) + at);
          sel[e] = off & 3;
        } else {
          keep |= 0xFFu << (8 * e);    // past the last token: what is there stays
        }
      }
      if (dst) {
        u32x4* const p = reinterpret_cast<u32x4*>(dst + page * RB + ((i & (page - 1)) >> 2) * (4 * RB) + at);
        u32x4 y, old = {0u, 0u, 0u, 0u};
        if (keep) old = *p;
#pragma unroll
        for (int c = 0; c < 4; c++) {
          uint32_t v = 0;
#pragma unroll
          for (int e = 0; e < 4; e++) {
            const uint32_t word = x[e][c];
            v |= (word >> (8 * sel[e]) & 0xFFu) << (8 * e);
          }
          const uint32_t was = old[c];
          y[c] = (v & ~keep) | (was & keep);
        }
        *p = y;
      }
    }
  }
  // Scales: K's and V's, 64 of each.
  if (tid < 2 * kMoveTokens) {
    const int i = i0 + (tid & (kMoveTokens - 1)), part = tid / kMoveTokens;
    if (i < count) {
      const int j = kept[i];
      const uint8_t* src = block_of(a, from, j, head);
      uint8_t* dst = block_of(a, to, i, head);
      uint32_t x = 0;
      if (src) x = *reinterpret_cast<const uint32_t*>(src + 2 * page * RB + (part * page + (j & (page - 1))) * 4);
      if (dst) *reinterpret_cast<uint32_t*>(dst + 2 * page * RB + (part * page + (i & (page - 1))) * 4) = x;
    }
  }
}

}  // namespace

int64_t kv_evict_chunks(int budget) { return (budget + kMoveTokens - 1) / kMoveTokens; }

hipError_t launch_kv_evict(const KvEvictArgs& a, int row_bytes, hipStream_t stream) {
  hipLaunchKernelGGL(evict_select_kernel, dim3((unsigned)(a.seqs * (int64_t)a.heads)), dim3(kSelectThreads), 0, stream, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const dim3 grid((unsigned)((int64_t)a.seqs * a.chunks * a.heads)), block(256);
  switch (row_bytes) {
    case 32: hipLaunchKernelGGL((evict_move_kernel<32>), grid, block, 0, stream, a); break;
    case 64: hipLaunchKernelGGL((evict_move_kernel<64>), grid, block, 0, stream, a); break;
    case 128: hipLaunchKernelGGL((evict_move_kernel<128>), grid, block, 0, stream, a); break;
    default: hipLaunchKernelGGL((evict_move_kernel<256>), grid, block, 0, stream, a); break;
  }
  return hipGetLastError();
}

}  // namespace convrot
