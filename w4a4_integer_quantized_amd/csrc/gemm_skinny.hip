// gemm_skinny.hip -- the gated product for few tokens (decode steps, drafts): int8 / int4 codes, and FP6 tiles (below).
//
// With few tokens the product is bound by the weights' bytes, 2 N * Kb, each read once. So the work is laid
// out for bytes in flight, not for reuse: a workgroup takes one to four 32-row blocks of the weights (16 gate rows
// and the 16 up rows of the same outputs), its waves share out K by 128-byte lines, and each wave copies
// its lines straight to LDS a line or two ahead, waiting for nobody but itself. v_mfma_i32_16x16x64_i8 with A =
// 16 weight rows and B = 16 tokens: a lane gets 4 consecutive outputs of one token, gate and up alike. The
// waves' sums (int32, exact in any order) meet in LDS.
//
// Copies to LDS rather than loads into registers because of their order: a fragment has 16 rows of the weights,
// so a load of fragments touches 16 lines for every 16 lanes, while a copy may take 8 whole lines at once. N = 11264,
// K = 4096: one token, 8 bits 20.5 us (4.5 TB/s; into registers 24.4), 4 bits 10.4 (12.6); 64 tokens 24 us (34).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "gemm_common.h"
#include "internal.h"

namespace convrot {
namespace {

using namespace gemm;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void* base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)bytes, 0x00020000);
}

constexpr int kFp6 = 2, kUnit = 127;   // the matrix instruction's FP6 E2M3, and E8M0 of 2^0

// 16 bytes a lane from memory to LDS, lane l's at dst + 16 l.
__device__ __forceinline__ void copy16(__amdgpu_buffer_rsrc_t rs, uint32_t off, uint8_t* dst) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void*)dst, 16, off, 0, 0, 0);
}

// Four outputs of a token from the sums of their gate and up rows. scales, biases: of the block's rows (gate; up 16 on).
template <int OUT>
__device__ __forceinline__ void store_gated(const float (&gate)[4], const float (&up)[4], float xs, const float* scales, const float* biases,
                                            int act, uint16_t* dst) {
  auto finish = [&](auto tag) __attribute__((always_inline)) {
    constexpr int ACT = decltype(tag)::value;
    float y[4];
#pragma unroll
    for (int e = 0; e < 4; e++) {
      const float g = __builtin_fmaf(gate[e], __fmul_rn(scales[e], xs), biases[e]);
      const float u = __builtin_fmaf(up[e], __fmul_rn(scales[16 + e], xs), biases[16 + e]);
      y[e] = __fmul_rn(activate<ACT>(g), u);
    }
    uint2 o;
    o.x = pack2(y[0], y[1], OUT);
    o.y = pack2(y[2], y[3], OUT);
    *reinterpret_cast<uint2*>(dst) = o;
  };
  if (act == kActSilu) {
    finish(std::integral_constant<int, kActSilu>{});
  } else if (act == kActGeluErf) {
    finish(std::integral_constant<int, kActGeluErf>{});
  } else if (act == kActGeluTanh) {
    finish(std::integral_constant<int, kActGeluTanh>{});
  } else {
    finish(std::integral_constant<int, kActNone>{});
  }
}

// MT tiles of 16 tokens, RB blocks of 32 weight rows. The waves take the 128-byte lines of K in turn, each with a
// ring of SLOTS lines of its own: [32 RB rows][128 B] of weights and, for each of the line's two 64-byte
// k steps and each tile, [16 rows][64 B] of tokens. LDS positions are swizzled by row (16-byte chunk c of a
// 128-byte row at c ^ ((row >> 1) & 7), of a 64-byte row at c ^ ((row >> 1) & 3)), so that the 16 lanes of a
// fragment read's pass hit distinct banks. No barrier until the waves' sums meet: a wave waits for its
// own copies only.
template <int BITS, int OUT, bool XT, int MT, int RB, int WAVES, int SLOTS>
__global__ __launch_bounds__(64 * WAVES) void gemm_gated_skinny_kernel(
    const uint8_t* __restrict__ Xq, const float* __restrict__ sx, const uint8_t* __restrict__ Wq, const float* __restrict__ sw,
    const float* __restrict__ bias, uint16_t* __restrict__ Y, int M, int N, int Kb, int act) {
  static_assert(SLOTS <= 2, "the waits below know two lines");
  constexpr int kW = 32 * RB * 128, kSlot = kW + 2 * MT * 1024, kCopies = 4 * RB + 2 * MT;
  constexpr int kRed = WAVES * 2 * RB * MT * 1024, kRing = WAVES * SLOTS * kSlot;
  // One array: with several the compiler, telling them apart, waits for all copies before each read.
  constexpr int kScales = kRing > kRed ? kRing : kRed;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[kScales + (64 * RB + 16 * MT) * 4];
  float* const w_scales = reinterpret_cast<float*>(lds + kScales);   // w_scale, bias of the blocks' rows, x_scale
  float *const biases = w_scales + 32 * RB, *const x_scales = biases + 32 * RB;
  static_assert(WAVES * 64 >= 16 * MT && WAVES * 64 >= 32 * RB, "a thread for each of the epilogue's operands");
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int64_t row0 = (int64_t)blockIdx.x * (32 * RB);
  const int rows = 2 * N - row0 < 32 * RB ? (int)(2 * N - row0) : 32 * RB;
  const int nk = Kb >> 6, lines = (nk + 1) >> 1;

  // The epilogue's operands, asked for first.
  float my_w = 0.0f, my_b = 0.0f, my_x = 0.0f;
  if (tid < rows) {
    my_w = sw[row0 + tid];
    my_b = bias ? bias[row0 + tid] : 0.0f;
  }
  if (tid < MT * 16 && tid < M) my_x = sx[tid];

  const __amdgpu_buffer_rsrc_t wrs = rsrc(Wq + row0 * Kb, (uint32_t)rows * (uint32_t)Kb);
  const __amdgpu_buffer_rsrc_t xrs = XT ? rsrc(Xq, 256u * (uint32_t)Kb) : rsrc(Xq, (uint32_t)M * (uint32_t)Kb);
  uint8_t* const ring = lds + wave * (SLOTS * kSlot);
  uint32_t w_off[4 * RB], x_off[MT];   // this lane's 16 bytes of each copy, at line 0
#pragma unroll
  for (int j = 0; j < 4 * RB; j++) {
    const int row = 8 * j + (lane >> 3), c = (lane & 7) ^ ((row >> 1) & 7);
    w_off[j] = (uint32_t)(row * Kb + 16 * c);
  }
#pragma unroll
  for (int t = 0; t < MT; t++) {
    const int x = lane >> 2, c = (lane & 3) ^ ((x >> 1) & 3), row = 16 * t + x;
    x_off[t] = (uint32_t)(row * (XT ? 64 : Kb) + 16 * c);
  }
  auto copy = [&](int slot, int q) __attribute__((always_inline)) {
    uint8_t* const dst = ring + slot * kSlot;
#pragma unroll
    for (int j = 0; j < 4 * RB; j++) copy16(wrs, w_off[j] + 128 * q, dst + j * 1024);
#pragma unroll
    for (int i = 0; i < 2; i++)
#pragma unroll
      for (int t = 0; t < MT; t++)
        copy16(xrs, x_off[t] + (XT ? (uint32_t)(2 * q + i) << 14 : (uint32_t)(128 * q + 64 * i)), dst + kW + (i * MT + t) * 1024);
  };

  v4i acc[2 * RB][MT];
#pragma unroll
  for (int h = 0; h < 2 * RB; h++)
#pragma unroll
    for (int t = 0; t < MT; t++) acc[h][t] = v4i{0, 0, 0, 0};
  struct Frags {
    v4i w[2 * RB], x[MT];
  };
  auto read = [&](Frags& f, const uint8_t* src, int i) __attribute__((always_inline)) {
#pragma unroll
    for (int h = 0; h < 2 * RB; h++) {
      const int row = 16 * h + r;
      f.w[h] = *reinterpret_cast<const v4i*>(src + row * 128 + (((4 * i + g) ^ ((row >> 1) & 7)) << 4));
    }
#pragma unroll
    for (int t = 0; t < MT; t++)
      f.x[t] = *reinterpret_cast<const v4i*>(src + kW + (i * MT + t) * 1024 + r * 64 + ((g ^ ((r >> 1) & 3)) << 4));
  };
  auto multiply = [&](const Frags& f) __attribute__((always_inline)) {
    if constexpr (BITS == 8) {
#pragma unroll
      for (int h = 0; h < 2 * RB; h++)
#pragma unroll
        for (int t = 0; t < MT; t++) acc[h][t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(f.w[h], f.x[t], acc[h][t], 0, 0, 0);
    } else {   // even and odd codes as bytes of 16 times their value; the sum is 256 acc
      v4i xe[MT], xo[MT];
#pragma unroll
      for (int t = 0; t < MT; t++) {
        xe[t] = (f.x[t] << 4) & (int)0xF0F0F0F0;
        xo[t] = f.x[t] & (int)0xF0F0F0F0;
      }
#pragma unroll
      for (int h = 0; h < 2 * RB; h++) {
        const v4i we = (f.w[h] << 4) & (int)0xF0F0F0F0, wo = f.w[h] & (int)0xF0F0F0F0;
#pragma unroll
        for (int t = 0; t < MT; t++) {
          acc[h][t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(we, xe[t], acc[h][t], 0, 0, 0);
          acc[h][t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wo, xo[t], acc[h][t], 0, 0, 0);
        }
      }
    }
  };

#pragma unroll
  for (int i = 0; i < SLOTS; i++)
    if (wave + WAVES * i < lines) copy(i, wave + WAVES * i);
  int slot = 0;
  for (int q = wave; q < lines; q += WAVES) {
    // This line's copies have landed: those of the line behind it, where there is one, may be under way.
    if (SLOTS > 1 && q + WAVES < lines) {
      asm volatile("s_waitcnt vmcnt(%0)" ::"n"(kCopies) : "memory");
    } else {
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    }
    Frags f0, f1;
    read(f0, ring + slot * kSlot, 0);
    read(f1, ring + slot * kSlot, 1);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // the slot is free again
    if (q + WAVES * SLOTS < lines) copy(slot, q + WAVES * SLOTS);
    // K may end in the middle of a line. (No branch: the products stay in one block with what waits for them.)
    const int half = 2 * q + 1 < nk ? -1 : 0;
#pragma unroll
    for (int t = 0; t < MT; t++) f1.x[t] &= half;
    multiply(f0);
    multiply(f1);
    slot = slot + 1 == SLOTS ? 0 : slot + 1;
  }

  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // no copy is under way when the ring becomes the sums' place
  __syncthreads();
  int4* const red = reinterpret_cast<int4*>(lds);    // [WAVES][2 RB][MT][64]
#pragma unroll
  for (int h = 0; h < 2 * RB; h++)
#pragma unroll
    for (int t = 0; t < MT; t++) red[((wave * 2 * RB + h) * MT + t) * 64 + lane] = __builtin_bit_cast(int4, acc[h][t]);
  if (tid < 32 * RB) {
    w_scales[tid] = my_w;
    biases[tid] = my_b;
  }
  if (tid < MT * 16) x_scales[tid] = my_x;
  __syncthreads();
  // A wave finishes tiles of 16 tokens and 16 outputs.
  for (int tile = wave; tile < MT * RB; tile += WAVES) {
    const int t = tile % MT, rb = tile / MT, m = 16 * t + r;
    v4i sum[2] = {v4i{0, 0, 0, 0}, v4i{0, 0, 0, 0}};
#pragma unroll
    for (int w = 0; w < WAVES; w++)
#pragma unroll
      for (int h = 0; h < 2; h++)
        sum[h] += __builtin_bit_cast(v4i, red[((w * 2 * RB + 2 * rb + h) * MT + t) * 64 + lane]);
    if (32 * rb >= rows || m >= M) continue;
    float gate[4], up[4];
#pragma unroll
    for (int e = 0; e < 4; e++) {
      gate[e] = static_cast<float>(BITS == 4 ? sum[0][e] >> 8 : sum[0][e]);
      up[e] = static_cast<float>(BITS == 4 ? sum[1][e] >> 8 : sum[1][e]);
    }
    const int n = 32 * rb + 4 * g;
    store_gated<OUT>(gate, up, x_scales[m], w_scales + n, biases + n, act, Y + (int64_t)m * N + row0 / 2 + 16 * rb + 4 * g);
  }
}

// The same for FP6 tiles, with v_mfma_scale_f32_16x16x128_f8f6f4: lane (r, g) holds 32 codes of a row, the half g % 2 of
// slice 2 q + g / 2 of a step q of 128 (16 bytes of plane 1 and 8 of plane 2). A fragment's 16 rows lie side by side in
// the tiles, 512 and 256 bytes a slice, so loads go straight to registers, DEPTH steps ahead. Past K's end
// they give zeros. Sums are integers below 2^24: exact in binary32 in any order. N = 11264, K = 4096, a call with its
// rotation: 16.5 us for one token, 19.7 for 64, 23.4 for 96 (26 to 27 on the 256 x 128 tiles); N = 2048, K = 8192: 13 to
// 20 us up to 128 tokens, 40 on the tiles. Two blocks of rows a workgroup, or more steps ahead: 1 to 4 us slower.
template <int OUT, int MT, int DEPTH>
__global__ __launch_bounds__(256) void gemm_gated_skinny6_kernel(const uint8_t* __restrict__ Xt, const float* __restrict__ sx,
                                                                 const uint8_t* __restrict__ Wt, const float* __restrict__ sw,
                                                                 const float* __restrict__ bias, uint16_t* __restrict__ Y, int M, int N,
                                                                 int K, int act) {
  typedef int v8i __attribute__((ext_vector_type(8)));
  typedef int v2i __attribute__((ext_vector_type(2)));
  constexpr int WAVES = 4, kSliceX = 256 * 48, kSliceW = 128 * 48;
  __shared__ __attribute__((aligned(16))) float4 red[WAVES * 2 * MT * 64];
  __shared__ float w_scales[32], biases[32], x_scales[16 * MT];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int64_t row0 = (int64_t)blockIdx.x * 32;
  const int slices = K >> 6, steps = slices >> 1;
  if (tid < 32) {
    w_scales[tid] = sw[row0 + tid];
    biases[tid] = bias ? bias[row0 + tid] : 0.0f;
  }
  if (tid < 16 * MT) x_scales[tid] = tid < M ? sx[tid] : 0.0f;

  // A workgroup's 32 rows lie in one 128-row panel.
  const __amdgpu_buffer_rsrc_t wrs = rsrc(Wt + (row0 >> 7) * ((int64_t)slices * kSliceW), (uint32_t)slices * kSliceW);
  const __amdgpu_buffer_rsrc_t xrs = rsrc(Xt, (uint32_t)slices * kSliceX);
  auto place = [&](int row, int panel, uint32_t& one, uint32_t& two) __attribute__((always_inline)) {
    const uint32_t slice = (uint32_t)(g >> 1) * (panel * 48);
    one = slice + row * 32 + 16 * ((g & 1) ^ ((row >> 3) & 1));
    two = slice + panel * 32 + row * 16 + 8 * ((g & 1) ^ ((row >> 4) & 1));
  };
  uint32_t w1[2], w2[2], x1[MT], x2[MT];
#pragma unroll
  for (int h = 0; h < 2; h++) place((int)(row0 & 127) + 16 * h + r, 128, w1[h], w2[h]);
#pragma unroll
  for (int t = 0; t < MT; t++) place(16 * t + r, 256, x1[t], x2[t]);
  struct Step {
    v4i w1[2], x1[MT];
    v2i w2[2], x2[MT];
  } ring[DEPTH];
  auto load = [&](Step& s, int q) __attribute__((always_inline)) {
    const uint32_t wq = (uint32_t)q * (2 * kSliceW), xq = (uint32_t)q * (2 * kSliceX);
#pragma unroll
    for (int h = 0; h < 2; h++) {
      s.w1[h] = __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(wrs, w1[h] + wq, 0, 0));
      s.w2[h] = __builtin_bit_cast(v2i, __builtin_amdgcn_raw_buffer_load_b64(wrs, w2[h] + wq, 0, 0));
    }
#pragma unroll
    for (int t = 0; t < MT; t++) {
      s.x1[t] = __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(xrs, x1[t] + xq, 0, 0));
      s.x2[t] = __builtin_bit_cast(v2i, __builtin_amdgcn_raw_buffer_load_b64(xrs, x2[t] + xq, 0, 0));
    }
  };
  auto operand = [](const v4i& a, const v2i& b) __attribute__((always_inline)) {
    return v8i{a[0], a[1], a[2], a[3], b[0], b[1], 0, 0};
  };
  typedef float v4f __attribute__((ext_vector_type(4)));
  v4f acc[2][MT];
#pragma unroll
  for (int h = 0; h < 2; h++)
#pragma unroll
    for (int t = 0; t < MT; t++) acc[h][t] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int d = 0; d < DEPTH; d++) {
    load(ring[d], wave + WAVES * d);
    __builtin_amdgcn_sched_barrier(0);
  }
  for (int q = wave; q < steps; q += WAVES * DEPTH) {
#pragma unroll
    for (int d = 0; d < DEPTH; d++) {
#pragma unroll
      for (int h = 0; h < 2; h++)
#pragma unroll
        for (int t = 0; t < MT; t++)
          acc[h][t] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(operand(ring[d].w1[h], ring[d].w2[h]), operand(ring[d].x1[t], ring[d].x2[t]),
                                                                       acc[h][t], kFp6, kFp6, 0, kUnit, 0, kUnit);
      __builtin_amdgcn_sched_barrier(0);    // in order: else all steps' products wait for all steps' loads
      load(ring[d], q + WAVES * (DEPTH + d));
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  // The wait that a read of the last product needs: the loop's end lies between them.
  asm volatile("s_nop 7\n\ts_nop 7\n\ts_nop 7" ::: "memory");
#pragma unroll
  for (int h = 0; h < 2; h++)
#pragma unroll
    for (int t = 0; t < MT; t++) red[((wave * 2 + h) * MT + t) * 64 + lane] = __builtin_bit_cast(float4, acc[h][t]);
  __syncthreads();
  for (int t = wave; t < MT; t += WAVES) {
    const int m = 16 * t + r;
    v4f sum[2] = {v4f{0.0f, 0.0f, 0.0f, 0.0f}, v4f{0.0f, 0.0f, 0.0f, 0.0f}};
#pragma unroll
    for (int w = 0; w < WAVES; w++)
#pragma unroll
      for (int h = 0; h < 2; h++)
        sum[h] += __builtin_bit_cast(v4f, red[((w * 2 + h) * MT + t) * 64 + lane]);
    if (m >= M) continue;
    const float gate[4] = {sum[0][0], sum[0][1], sum[0][2], sum[0][3]}, up[4] = {sum[1][0], sum[1][1], sum[1][2], sum[1][3]};
    store_gated<OUT>(gate, up, x_scales[m], w_scales + 4 * g, biases + 4 * g, act, Y + (int64_t)m * N + row0 / 2 + 4 * g);
  }
}

struct SkinnyCall {
  const uint8_t* Xq;
  const float* sx;
  const uint8_t* Wq;
  const float *sw, *bias;
  uint16_t* Y;
  int M, N, Kb, act;
  hipStream_t st;
};

template <int BITS, int OUT, bool XT, int MT, int RB, int WAVES, int SLOTS>
hipError_t launch_waves(const SkinnyCall& c) {
  hipLaunchKernelGGL((gemm_gated_skinny_kernel<BITS, OUT, XT, MT, RB, WAVES, SLOTS>),
                     dim3((unsigned)((c.N + 16 * RB - 1) / (16 * RB))), dim3(64 * WAVES), 0, c.st, c.Xq, c.sx, c.Wq, c.sw, c.bias,
                     c.Y, c.M, c.N, c.Kb, c.act);
  return hipGetLastError();
}

// Blocks of weights a workgroup takes: the most that leave the fewest rounds of workgroups times blocks,
// `most` at most. (64 tokens, K = 4096, 8 bits: 704 blocks 30 us by ones, 29.6 by twos, 24 by threes; 512
// blocks 21, 18, 20; 256 blocks 11.7, 14, 17.) A workgroup of one block leaves room for a second only up to 16
// tokens, where more blocks do not pay: 20.5, 24, 23 us for 704.
int blocks_of(int64_t blocks, int most) {
  int best = 1;
  int64_t least = -1;
  for (int rb = 1; rb <= most; rb++) {
    const int64_t cost = ((blocks + rb - 1) / rb + kNumCUs - 1) / kNumCUs * rb;
    if (least < 0 || cost <= least) {
      least = cost;
      best = rb;
    }
  }
  return best;
}

template <int BITS, int OUT, bool XT, int MT>
hipError_t launch_blocks(const SkinnyCall& c) {
  constexpr int kMost = MT == 8 ? 2 : MT == 6 ? 3 : 4;    // what the sums' place in LDS allows
  const int rb = blocks_of(c.N / 16, kMost);
  if constexpr (kMost >= 4) {
    if (rb == 4) return launch_waves<BITS, OUT, XT, MT, 4, 4, 1>(c);
  }
  if constexpr (kMost >= 3) {
    if (rb == 3) return launch_waves<BITS, OUT, XT, MT, 3, 4, 1>(c);
  }
  if (rb == 2) return launch_waves<BITS, OUT, XT, MT, 2, 4, MT <= 4 ? 2 : 1>(c);
  return launch_waves<BITS, OUT, XT, MT, 1, 4, MT <= 4 ? 2 : 1>(c);
}

template <int BITS, int OUT, bool XT>
hipError_t launch_tokens(const SkinnyCall& c) {
  if (c.M <= 16) return launch_waves<BITS, OUT, XT, 1, 1, 4, 2>(c);
  if (c.M <= 32) return launch_blocks<BITS, OUT, XT, 2>(c);
  if (c.M <= 48) return launch_blocks<BITS, OUT, XT, 3>(c);
  if (c.M <= 64) return launch_blocks<BITS, OUT, XT, 4>(c);
  if (c.M <= 96) return launch_blocks<BITS, OUT, XT, 6>(c);
  return launch_blocks<BITS, OUT, XT, 8>(c);
}

}  // namespace

// Up to 96 tokens; up to 128 where two rounds of workgroups hold all blocks. Measured against the 256 x 128 tiles
// (K = 4096, 8 bits): 96 tokens, N = 11264 27.5 against 37 us; 128 tokens, N = 4096 15.9 against 32.6, N = 8192 22.9
// against 34.7, but N = 11264 42.3 against 37.3 (4 bits: 30.5 against 27.5). FP6 tiles: 128 tokens, N = 11264 28.2 against
// 26.5, N = 5120, K = 2048 15.0 against 17.7.
bool gated_skinny_supported(int64_t M, int64_t N) { return M <= 96 || (M <= 128 && N / 16 <= 2 * kNumCUs); }

hipError_t launch_gated_skinny(const void* Xq, const float* sx, const void* Wq, const float* sw, const float* bias, int64_t M,
                               int64_t N, int64_t Kb, int bits, bool x_tiled, void* Y, int out_dt, int act, hipStream_t st) {
  const SkinnyCall c = {static_cast<const uint8_t*>(Xq), sx, static_cast<const uint8_t*>(Wq), sw, bias,
                        static_cast<uint16_t*>(Y), (int)M, (int)N, (int)Kb, act, st};
  if (out_dt == kF16) {
    if (bits == 8) return x_tiled ? launch_tokens<8, kOutF16, true>(c) : launch_tokens<8, kOutF16, false>(c);
    return x_tiled ? launch_tokens<4, kOutF16, true>(c) : launch_tokens<4, kOutF16, false>(c);
  }
  if (bits == 8) return x_tiled ? launch_tokens<8, kOutBF16, true>(c) : launch_tokens<8, kOutBF16, false>(c);
  return x_tiled ? launch_tokens<4, kOutBF16, true>(c) : launch_tokens<4, kOutBF16, false>(c);
}


template <int OUT, int MT, int DEPTH>
hipError_t launch6(const SkinnyCall& c) {
  hipLaunchKernelGGL((gemm_gated_skinny6_kernel<OUT, MT, DEPTH>), dim3((unsigned)(c.N / 16)), dim3(256), 0, c.st, c.Xq, c.sx, c.Wq, c.sw,
                     c.bias, c.Y, c.M, c.N, c.Kb, c.act);
  return hipGetLastError();
}

template <int OUT>
hipError_t launch6_tokens(const SkinnyCall& c) {
  if (c.M <= 16) return launch6<OUT, 1, 4>(c);
  if (c.M <= 32) return launch6<OUT, 2, 2>(c);
  if (c.M <= 48) return launch6<OUT, 3, 2>(c);
  if (c.M <= 64) return launch6<OUT, 4, 2>(c);
  if (c.M <= 96) return launch6<OUT, 6, 2>(c);
  return launch6<OUT, 8, 1>(c);
}

hipError_t launch_gated_skinny6(const void* Xt, const float* sx, const void* Wt, const float* sw, const float* bias, int64_t M, int64_t N,
                                int64_t K, void* Y, int out_dt, int act, hipStream_t st) {
  const SkinnyCall c = {static_cast<const uint8_t*>(Xt), sx, static_cast<const uint8_t*>(Wt), sw, bias,
                        static_cast<uint16_t*>(Y), (int)M, (int)N, (int)K, act, st};
  return out_dt == kF16 ? launch6_tokens<kOutF16>(c) : launch6_tokens<kOutBF16>(c);
}

}  // namespace convrot
