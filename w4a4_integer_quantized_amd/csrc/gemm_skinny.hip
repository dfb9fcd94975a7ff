// gemm_skinny.hip -- the gated product for few tokens (decode steps, drafts): int8 / int4 codes.
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

// 16 bytes a lane from memory to LDS, lane l's at dst + 16 l.
__device__ __forceinline__ void copy16(__amdgpu_buffer_rsrc_t rs, uint32_t off, uint8_t* dst) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void*)dst, 16, off, 0, 0, 0);
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
  static_assert(SLOTS <= 4, "the waits below know four lines");
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
    // This line's copies have landed: those of the lines behind it, SLOTS - 1 or what is left, may be under way.
    if (SLOTS > 3 && q + 3 * WAVES < lines) {
      asm volatile("s_waitcnt vmcnt(%0)" ::"n"(kCopies * 3) : "memory");
    } else if (SLOTS > 2 && q + 2 * WAVES < lines) {
      asm volatile("s_waitcnt vmcnt(%0)" ::"n"(kCopies * 2) : "memory");
    } else if (SLOTS > 1 && q + WAVES < lines) {
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
    auto finish = [&](auto tag) __attribute__((always_inline)) {
      constexpr int ACT = decltype(tag)::value;
      const float xs = x_scales[m];
      float y[4];
#pragma unroll
      for (int e = 0; e < 4; e++) {
        const int n = 32 * rb + 4 * g + e;
        const int ig = BITS == 4 ? sum[0][e] >> 8 : sum[0][e], iu = BITS == 4 ? sum[1][e] >> 8 : sum[1][e];
        const float gate = __builtin_fmaf(static_cast<float>(ig), __fmul_rn(w_scales[n], xs), biases[n]);
        const float up = __builtin_fmaf(static_cast<float>(iu), __fmul_rn(w_scales[16 + n], xs), biases[16 + n]);
        y[e] = __fmul_rn(activate<ACT>(gate), up);
      }
      uint2 o;
      o.x = pack2(y[0], y[1], OUT);
      o.y = pack2(y[2], y[3], OUT);
      *reinterpret_cast<uint2*>(Y + (int64_t)m * N + row0 / 2 + 16 * rb + 4 * g) = o;
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
// against 34.7, but N = 11264 42.3 against 37.3 (4 bits: 30.5 against 27.5).
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

}  // namespace convrot
