// kv_evict.hip -- a cache brought down to a budget of tokens (rq_kv_evict; definition in convrot.h): for each
// sequence and key head the tokens that stay are chosen by their weights, and their codes and scales are
// written, in order, into new pages.
//
// evict_select_kernel: a workgroup a (sequence, key head). The weight of the last token that still fits
// is found digit by digit (11, 11 and 10 bits of the weights as ordered integers, a histogram of 2048 counters in LDS for
// each), then one pass in order writes the indices: everything above that weight, and of those beside it the
// first. Counters are integers: the same choice every time. Bound by its vector instructions and its barriers: 22 us for
// 512 rows of 8192. Few long rows are cut into parts (evict_part_kernel), each pass of which is bound by reading.
// Weights kept in registers over the four passes: no gain (the instructions bound it, and there are fewer waves).
// evict_move_kernel: bound by memory. Bytes are moved as they are. K rows and scales are copied; V bytes lie four
// tokens side by side, so each four new tokens gather a byte from each of four old groups: a lone token
// that stays costs the reading of its whole group's V lines. 64 sequences of 8192 tokens to 2048, 8 heads of 128, 4-bit
// codes: 71 us, 221 MB read and 122 MB written by the counters, 4.8 TB/s, what a large copy reaches. (93 us with each kind
// loaded and stored before the next.)
#include "kv_common.h"

namespace convrot {
namespace {

using namespace kv;

constexpr int kSelectThreads = 1024, kSelectWaves = kSelectThreads / 64;
constexpr int kBins = 2048;
constexpr int kMoveTokens = 64;   // new tokens of a move workgroup
// A row's parts, and the workgroups that they come to. (32 rows of 131072 tokens: 137 us with one workgroup a row, whose
// CU's vector instructions bound it; 40 with 256 in all, 46 with 512 and 71 with 1024, as every part reads every part's
// counters. 512 rows of 8192: 22 us as they are, twice that in two parts each.)
constexpr int kPartTokens = 4096, kSelectGroups = 256;

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

// Bits of a wave's mask that lie before this lane.
__device__ __forceinline__ uint32_t below(uint64_t m) {
  return __builtin_amdgcn_mbcnt_hi((uint32_t)(m >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)m, 0));
}

// Sum over the wave's first 16 lanes, for all of it.
__device__ __forceinline__ uint32_t row16_sum(uint32_t x) {
  x += __builtin_amdgcn_mov_dpp((int)x, 0xB1, 0xF, 0xF, true);
  x += __builtin_amdgcn_mov_dpp((int)x, 0x4E, 0xF, 0xF, true);
  x += __builtin_amdgcn_mov_dpp((int)x, 0x141, 0xF, 0xF, true);
  x += __builtin_amdgcn_mov_dpp((int)x, 0x128, 0xF, 0xF, true);
  return __builtin_amdgcn_readfirstlane(x);
}

constexpr int digit_bits(int digit) { return digit == 2 ? 10 : 11; }
constexpr int digit_shift(int digit) { return digit == 0 ? 21 : digit == 1 ? 10 : 0; }

// What a (sequence, key head) is asked for: tokens [lo, hi) of n are chosen from, `want` of them; those around stay.
struct Choice {
  int b, head, n, lo, hi;
  uint32_t want;
  int32_t* kept;
  const float* weights;     // begins at a multiple of 16 floats
  float* out;               // new weights, or null
};
__device__ __forceinline__ Choice row_of(const KvEvictArgs& a, int row) {
  Choice r;
  r.b = row / a.heads;
  r.head = row - r.b * a.heads;
  r.n = kv_length(a, r.b);
  r.lo = a.first;
  r.hi = r.n - a.recent;
  r.want = a.budget - a.first - a.recent;
  r.kept = a.kept + (int64_t)row * a.budget;
  r.weights = a.weights + (int64_t)row * ((int64_t)a.max_pages << a.lps);
  r.out = a.new_weights ? a.new_weights + (int64_t)row * ((int64_t)a.new_max_pages << a.lps) : nullptr;
  return r;
}

// A row within the budget: everything stays. Places i0, i0 + step, ..
__device__ __forceinline__ void keep_all(const KvEvictArgs& a, const Choice& r, int i0, int step) {
  for (int i = i0; i < a.budget; i += step) {
    r.kept[i] = i < r.n ? i : -1;
    if (r.out && i < r.n) r.out[i] = r.weights[i];
  }
}

// Weights of the tokens j .. j + 3, zeros from `end` on in steps of four (within the row all the same).
__device__ __forceinline__ f32x4u four_weights(const Choice& r, int j, int end) {
  f32x4u w = {0.0f, 0.0f, 0.0f, 0.0f};
  if (j < end) w = *reinterpret_cast<const f32x4u*>(r.weights + j);
  return w;
}

// How many of the tokens [begin, end) (begin a multiple of 4) that are chosen from, and whose digits before are
// `prefix`, have each value of a digit. Ends with every counter written.
__device__ __forceinline__ void count_digit(const Choice& r, int begin, int end, int digit, uint32_t prefix, uint32_t* bins) {
  const int tid = threadIdx.x, lane = tid & 63;
  const int shift = digit_shift(digit), bits = digit_bits(digit);
  end = end < r.hi ? end : r.hi;
  f32x4u next = four_weights(r, begin + 4 * tid, end);
  for (int i = tid; i < kBins; i += kSelectThreads) bins[i] = 0;
  __syncthreads();
  for (int base = begin; base < end; base += 4 * kSelectThreads) {
    const int j = base + 4 * tid;
    const f32x4u w = next;
    next = four_weights(r, j + 4 * kSelectThreads, end);
    const bool inner = base >= r.lo && base + 4 * kSelectThreads <= end;   // all of them are chosen from
#pragma unroll
    for (int e = 0; e < 4; e++) {
      const uint32_t key = order_key(w[e]);
      bool in = digit == 0 || key >> (shift + bits) == prefix;
      if (!inner) in = in && j + e >= r.lo && j + e < end;
      const uint32_t bin = key >> shift & ((1u << bits) - 1);
      // Lanes that meet the first lane's counter add to it together: weights of one size, zeros above all.
      const uint64_t active = __ballot(in);
      if (active == 0) continue;
      const int leader = __builtin_ctzll(active);
      const uint32_t same = __builtin_amdgcn_readlane(bin, leader);
      const uint64_t with = __ballot(in && bin == same);
      if (lane == leader) atomicAdd(&bins[same], (uint32_t)__builtin_popcountll(with));
      if (in && bin != same) atomicAdd(&bins[bin], 1u);
    }
  }
  __syncthreads();
}

// The digit, from the top, in which the want-th token lies, and the count still wanted of it, into found[0 .. 1].
// Thread t has the counters c0 of 2047 - 2t and c1 of the next. Ends with found written.
__device__ __forceinline__ void find_digit(uint32_t c0, uint32_t c1, uint32_t want, uint32_t* part, uint32_t* found) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const uint32_t incl = wave_scan(c0 + c1, lane);
  if (lane == 63) part[wave] = incl;
  __syncthreads();
  uint32_t before = incl - c0 - c1;
  before += row16_sum(lane < wave && lane < kSelectWaves ? part[lane] : 0u);
  if (before < want && before + c0 >= want) {
    found[0] = kBins - 1 - 2 * tid;
    found[1] = want - before;
  } else if (before + c0 < want && before + c0 + c1 >= want) {
    found[0] = kBins - 2 - 2 * tid;
    found[1] = want - before - c0;
  }
  __syncthreads();
}

// The tokens [begin, end) that stay, in order: what lies around, what is above the edge, and the first `want` of the
// row beside it. `above` and `beside` tokens of each kind lie before them. part: 2 * kSelectWaves numbers.
__device__ __forceinline__ void write_kept(const Choice& r, int begin, int end, bool choose, uint32_t edge, uint32_t want, uint32_t above,
                                           uint32_t beside, uint32_t* part) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int turn = 0;
  f32x4u next = four_weights(r, begin + 4 * tid, end);
  for (int base = begin; base < end; base += 4 * kSelectThreads, turn ^= kSelectWaves) {
    const int j = base + 4 * tid;
    const f32x4u w = next;
    next = four_weights(r, j + 4 * kSelectThreads, end);
    // A bit a token; and how many of each kind lie before this lane's in the wave (below) and in all of it.
    uint32_t is_above = 0, is_beside = 0, up = above, at_edge = beside, wave_above = 0, wave_beside = 0;
#pragma unroll
    for (int e = 0; e < 4; e++) {
      const uint32_t key = order_key(w[e]);
      const bool around = j + e < r.lo || j + e >= r.hi;
      const bool has = j + e < end && (around || (choose && key > edge));
      const bool edges = j + e < end && !around && choose && key == edge;
      is_above |= has ? 1u << e : 0u;
      is_beside |= edges ? 1u << e : 0u;
      const uint64_t m = __ballot(has), n = __ballot(edges);
      up += below(m);
      wave_above += __builtin_popcountll(m);
      at_edge += below(n);
      wave_beside += __builtin_popcountll(n);
    }
    if (lane == 0) part[turn + wave] = wave_above | wave_beside << 16;      // at most 256 in each half
    __syncthreads();    // (the other half of `part` is read by nobody any more at the next write of this one)
    // Lane v holds wave v's numbers: sums over the waves before this one, and over all (at most 4096 in each half).
    const uint32_t x = lane < kSelectWaves ? part[turn + lane] : 0u;
    const uint32_t ahead = row16_sum(lane < wave ? x : 0u), total = row16_sum(x);
    up += ahead & 0xFFFFu;
    at_edge += ahead >> 16;
#pragma unroll
    for (int e = 0; e < 4; e++) {
      const bool has = is_above >> e & 1, edges = is_beside >> e & 1;
      if (has || (edges && at_edge < want)) {
        const uint32_t at = up + (at_edge < want ? at_edge : want);
        r.kept[at] = j + e;
        if (r.out) r.out[at] = w[e];
      }
      up += has;
      at_edge += edges;
    }
    above += total & 0xFFFFu;
    beside += total >> 16;
  }
}

__global__ __launch_bounds__(kSelectThreads) void evict_select_kernel(const KvEvictArgs a) {
  __shared__ uint32_t bins[kBins], part[2 * kSelectWaves], found[2];
  const int tid = threadIdx.x;
  const Choice r = row_of(a, blockIdx.x);
  if (r.head == 0 && tid == 0) a.new_kv_len[r.b] = r.n < a.budget ? r.n : a.budget;
  if (r.n <= a.budget) return keep_all(a, r, tid, kSelectThreads);
  uint32_t want = r.want, prefix = 0;
  const bool choose = want > 0;     // the same for the whole workgroup
  if (choose) {
    for (int digit = 0; digit < 3; digit++) {
      count_digit(r, 0, r.n, digit, prefix, bins);
      find_digit(bins[kBins - 1 - 2 * tid], bins[kBins - 2 - 2 * tid], want, part, found);
      prefix = digit == 0 ? found[0] : prefix << digit_bits(digit) | found[0];
      want = found[1];
      __syncthreads();
    }
  }
  write_kept(r, 0, r.n, choose, prefix, want, 0, 0, part);
}

// The same by a.parts workgroups a row and one launch for each of 0, 1, 2: counting a digit, and 3: writing. Each
// launch adds the parts' counters of the digit before up and finds it, every workgroup for itself. A row's scratch:
//   [2][2]          digits so far and count still wanted, after digit 0 and 1
//   [2][parts]      tokens of each part above those digits
//   [parts][2048], [parts][2048], [parts][1024]   counters
__host__ __device__ constexpr int64_t scratch_words(int parts) { return 4 + (int64_t)parts * (2 + 2 * kBins + kBins / 2); }

template <int STAGE>
__global__ __launch_bounds__(kSelectThreads) void evict_part_kernel(const KvEvictArgs a) {
  __shared__ uint32_t bins[kBins], part[2 * kSelectWaves], found[2], sums[kSelectWaves], edges;
  const int tid = threadIdx.x, parts = a.parts, row = blockIdx.x / parts, p = blockIdx.x - row * parts;
  const Choice r = row_of(a, row);
  if (STAGE == 3 && r.head == 0 && p == 0 && tid == 0) a.new_kv_len[r.b] = r.n < a.budget ? r.n : a.budget;
  if (r.n <= a.budget) {
    if (STAGE == 3) keep_all(a, r, p * kSelectThreads + tid, parts * kSelectThreads);
    return;
  }
  const int size = ((r.n + parts - 1) / parts + 3) / 4 * 4;
  const int64_t from = (int64_t)p * size;
  const int begin = from < r.n ? (int)from : r.n, end = begin + size < r.n ? begin + size : r.n;
  uint32_t* const scratch = a.scratch + row * scratch_words(parts);
  uint32_t *const state = scratch, *const tally = scratch + 4, *const counters = tally + 2 * parts;
  uint32_t want = r.want, prefix = 0, above = 0, beside = 0;
  const bool choose = want > 0;
  if (choose && STAGE > 0) {
    constexpr int kDigit = STAGE - 1, kSize = 1 << digit_bits(kDigit);
    if (kDigit > 0) {
      prefix = state[2 * (kDigit - 1)];
      want = state[2 * (kDigit - 1) + 1];
    }
    const uint32_t* const all = counters + (int64_t)kDigit * parts * kBins;
    const int at = kBins - 2 - 2 * tid;       // c[1] counts digit at + 1, c[0] digit at
    u32x2 c = {0u, 0u}, mine = {0u, 0u};      // mine: of this part; at the last digit of all before it
    if (at < kSize) {
#pragma unroll 8
      for (int q = 0; q < parts; q++) {
        const u32x2 x = *reinterpret_cast<const u32x2*>(all + q * kSize + at);
        c += x;
        if (STAGE == 3 ? q < p : q == p) mine += x;
      }
    }
    find_digit(c[1], c[0], want, part, found);
    const int digit = found[0];
    prefix = kDigit == 0 ? digit : prefix << digit_bits(kDigit) | digit;
    want = found[1];
    uint32_t mine_above = (at + 1 > digit ? mine[1] : 0u) + (at > digit ? mine[0] : 0u);
    if (STAGE == 3 && tid < p) mine_above += tally[parts + tid];       // (at most 32 parts)
#pragma unroll
    for (int m = 32; m > 0; m >>= 1) mine_above += __shfl_xor(mine_above, m, 64);
    if ((tid & 63) == 0) sums[tid >> 6] = mine_above;
    if (STAGE == 3 && (at == digit || at + 1 == digit)) edges = at == digit ? mine[0] : mine[1];
    __syncthreads();
    for (int v = 0; v < kSelectWaves; v++) above += sums[v];
    if (STAGE == 3) {
      beside = edges;
    } else if (tid == 0) {
      tally[kDigit * parts + p] = above + (kDigit > 0 ? tally[(kDigit - 1) * parts + p] : 0u);
      if (p == 0) {
        state[2 * kDigit] = prefix;
        state[2 * kDigit + 1] = want;
      }
    }
  }
  if constexpr (STAGE < 3) {
    if (!choose) return;
    constexpr int kSize = 1 << digit_bits(STAGE);
    count_digit(r, begin, end, STAGE, prefix, bins);
    uint32_t* const out = counters + (int64_t)STAGE * parts * kBins + p * kSize;
    for (int i = tid; i < kSize; i += kSelectThreads) out[i] = bins[i];
  } else {
    above += (begin < r.lo ? begin : r.lo) + (begin > r.hi ? begin - r.hi : 0);     // those around before this part
    write_kept(r, begin, end, choose, prefix, want, above, beside, part);
  }
}

// Where the head's block of a page of a table begins in the cache, in bytes; -1: the page is not in it.
__device__ __forceinline__ int64_t block_of(const KvEvictArgs& a, const int32_t* table, int token, int head) {
  const int pg = table[token >> a.lps];
  return pg >= 0 && pg < a.num_pages ? ((int64_t)pg * a.heads + head) * a.head_bytes : -1;
}

// New tokens [64 c, 64 c + 64) of a (sequence, key head). RB: bytes of a row of codes. The places are looked up once, then
// everything is loaded before anything is stored. (What comes from no page is loaded from the cache's first and replaced by
// zeros: a load under a condition would be waited for on its own.)
template <int RB>
__global__ __launch_bounds__(256) void evict_move_kernel(const KvEvictArgs a) {
  __shared__ int64_t from[kMoveTokens], to[kMoveTokens];   // blocks, or -1
  __shared__ int places[kMoveTokens];                       // in the old page
  const int tid = threadIdx.x, page = 1 << a.lps;
  const int head = blockIdx.x % a.heads, rest = blockIdx.x / a.heads, chunk = rest % a.chunks, b = rest / a.chunks;
  const int n = kv_length(a, b), count = n < a.budget ? n : a.budget, i0 = chunk * kMoveTokens;
  if (i0 >= count) return;
  if (tid < kMoveTokens) {
    const int i = i0 + tid;
    int64_t src = -1, dst = -1;
    int place = 0;
    if (i < count) {
      const int j = a.kept[((int64_t)b * a.heads + head) * a.budget + i];
      dst = block_of(a, a.new_pages + (int64_t)b * a.new_max_pages, i, head);
      src = block_of(a, a.pages + (int64_t)b * a.max_pages, j, head);
      place = j & (page - 1);
    }
    from[tid] = src;
    to[tid] = dst;
    places[tid] = place;
  }
  __syncthreads();
  const u32x4 zeros = {0u, 0u, 0u, 0u};
  // K rows: 16 bytes a thread. V: four new tokens and four of their bytes. Scales: K's and V's, 64 of each.
  constexpr int kPer = RB / 16, kQuads = RB / 4, kTurns = RB < 64 ? 1 : RB / 64;
  u32x4 k[kTurns], v[kTurns][4];
#pragma unroll
  for (int t = 0; t < kTurns; t++) {
    const int job = tid + 256 * t, i = job / kPer % kMoveTokens, at = job % kPer * 16;
    const int64_t src = from[i];
    k[t] = *reinterpret_cast<const u32x4*>(a.cache + (src < 0 ? 0 : src) + places[i] * RB + at);
  }
#pragma unroll
  for (int t = 0; t < kTurns; t++) {
    const int job = tid + 256 * t, i = job / kQuads * 4 % kMoveTokens, at = job % kQuads * 16;
#pragma unroll
    for (int e = 0; e < 4; e++) {
      const int64_t src = from[i + e];
      v[t][e] = *reinterpret_cast<const u32x4*>(a.cache + (src < 0 ? 0 : src) + page * RB + (places[i + e] >> 2) * (4 * RB) + at);
    }
  }
  const int si = tid & (kMoveTokens - 1), part = tid / kMoveTokens & 1;
  const int64_t scales = from[si];
  const uint32_t scale = *reinterpret_cast<const uint32_t*>(a.cache + (scales < 0 ? 0 : scales) + 2 * page * RB + (part * page + places[si]) * 4);
  asm volatile("" ::: "memory");   // the loads stay in front of it

#pragma unroll
  for (int t = 0; t < kTurns; t++) {
    const int job = tid + 256 * t, i = job / kPer, at = job % kPer * 16;
    if (i < kMoveTokens && to[i] >= 0)
      *reinterpret_cast<u32x4*>(a.cache + to[i] + ((i0 + i) & (page - 1)) * RB + at) = from[i] < 0 ? zeros : k[t];
  }
#pragma unroll
  for (int t = 0; t < kTurns; t++) {
    const int job = tid + 256 * t, i = job / kQuads * 4, at = job % kQuads * 16;
    if (i < kMoveTokens && to[i] >= 0) {
      u32x4* const p = reinterpret_cast<u32x4*>(a.cache + to[i] + page * RB + (((i0 + i) & (page - 1)) >> 2) * (4 * RB) + at);
      uint32_t keep = 0, sel[4], there[4];
#pragma unroll
      for (int e = 0; e < 4; e++) {
        sel[e] = places[i + e] & 3;
        there[e] = from[i + e] < 0 ? 0u : 0xFFu << (8 * e);
        if (i0 + i + e >= count) keep |= 0xFFu << (8 * e);    // past the last token: what is there stays
      }
      u32x4 y, old = zeros;
      if (keep) old = *p;
#pragma unroll
      for (int c = 0; c < 4; c++) {
        uint32_t x = old[c] & keep;
#pragma unroll
        for (int e = 0; e < 4; e++) {
          const uint32_t word = v[t][e][c];
          x |= (word >> (8 * sel[e]) & 0xFFu) << (8 * e) & there[e];
        }
        y[c] = x;
      }
      *p = y;
    }
  }
  if (tid < 2 * kMoveTokens && to[si] >= 0)
    *reinterpret_cast<uint32_t*>(a.cache + to[si] + 2 * page * RB + (part * page + ((i0 + si) & (page - 1))) * 4) = scales < 0 ? 0u : scale;
}

}  // namespace

int64_t kv_evict_chunks(int budget) { return (budget + kMoveTokens - 1) / kMoveTokens; }

KvEvictPlan plan_kv_evict(int64_t groups, int64_t span) {
  KvEvictPlan p = {1, 0};
  if (groups < 1) return p;
  const int64_t most = kSelectGroups / groups, all = (span + kPartTokens - 1) / kPartTokens;
  p.parts = (int)(most < all ? most : all);
  if (p.parts > 32) p.parts = 32;
  if (p.parts < 2) p.parts = 1;
  if (p.parts > 1) p.workspace_bytes = (size_t)(groups * scratch_words(p.parts) * 4);
  return p;
}

hipError_t launch_kv_evict(const KvEvictArgs& a, int row_bytes, hipStream_t stream) {
  const dim3 rows((unsigned)(a.seqs * (int64_t)a.heads * a.parts));
  if (a.parts == 1) {
    hipLaunchKernelGGL(evict_select_kernel, rows, dim3(kSelectThreads), 0, stream, a);
  } else {
    hipLaunchKernelGGL((evict_part_kernel<0>), rows, dim3(kSelectThreads), 0, stream, a);
    hipLaunchKernelGGL((evict_part_kernel<1>), rows, dim3(kSelectThreads), 0, stream, a);
    hipLaunchKernelGGL((evict_part_kernel<2>), rows, dim3(kSelectThreads), 0, stream, a);
    hipLaunchKernelGGL((evict_part_kernel<3>), rows, dim3(kSelectThreads), 0, stream, a);
  }
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
