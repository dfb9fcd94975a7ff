// kv_common.h -- what the cache kernels share (kv_cache.hip, kv_attention.hip): the page layout
// of convrot.h, the Walsh-Hadamard transform of a head row over a group of lanes, and the
// conversion of codes to fp16 matrix operands.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "internal.h"

namespace convrot {
namespace kv {

typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

// A head's block of a page, for `page` = 1 << lps tokens of row_bytes code bytes each:
//   K codes   [page][row_bytes]
//   V codes   [page / 4][row_bytes][4]   byte b of token t at ((t / 4) * row_bytes + b) * 4 + t % 4
//   K scales  float [page]
//   V scales  float [page]
template <int D, int BITS>
struct Row {
  static constexpr int kBytes = D * BITS / 8;            // code bytes of a head row
  static constexpr int kBlock = D < 128 ? D : 128;       // rotation block
  static constexpr int kLanes = kBlock / 8;              // lanes that hold a row, 8 elements a chunk
  static constexpr int kChunks = D / kBlock;             // chunks a lane holds
  static constexpr float kNorm = kBlock == 128 ? 0x1.6a09e6p-4f : 0.125f;   // fl(1 / sqrt(kBlock))
  static constexpr float kQmax = BITS == 8 ? 127.0f : 7.0f;
};

template <int DPP_CTRL>
__device__ __forceinline__ float dpp_f(float v) {
  return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), DPP_CTRL, 0xF, 0xF, true));
}

// The chunk (8 elements) of a rotation block that lane u of its group holds. With it, flipping
// chunk bit 0, 1, 2 or 3 is lane xor 1, 2, 7 or 8: one DPP exchange each.
__device__ __forceinline__ int chunk_of_lane(int u) { return u ^ (3 * ((u >> 2) & 1)); }

// The unnormalized Walsh-Hadamard transform of one block, stages h = 1, 2, 4, ... in this order,
// 8 elements a lane (chunk `c` of the block) over LANES lanes. Every lane of the wave takes part.
// In a cross-lane stage the upper lane of a pair computes mine - partner, the negated butterfly
// difference; the sign that a lane's values end up with is returned (fl is sign-symmetric, and
// later stages pair lanes of equal sign, so the magnitudes are exactly those of the transform).
template <int LANES>
__device__ __forceinline__ float wht_block(float (&v)[8], int c) {
#pragma unroll
  for (int h = 1; h < 8; h <<= 1) {
#pragma unroll
    for (int i = 0; i < 8; i++) {
      if ((i & h) == 0) {
        const float a = v[i], b = v[i + h];
        v[i] = __fadd_rn(a, b);
        v[i + h] = __fsub_rn(a, b);
      }
    }
  }
  const float m0 = (c & 1) ? -1.0f : 1.0f, m1 = (c & 2) ? -1.0f : 1.0f;
  const float m2 = (c & 4) ? -1.0f : 1.0f, m3 = (c & 8) ? -1.0f : 1.0f;
  // v = fma(partner's v, m, v), the exchange an operand modifier of the fma (the compiler moves the
  // value first). A lane exchange must not follow the write of what it reads by less than two
  // instructions: the nop stands for what came before, and eight values keep each other apart.
#define KV_EXCHANGE(CTRL, M)                                                                                    \
  asm volatile("s_nop 1\n\t"                                                                                             \
      "v_fmac_f32_dpp %0, %0, %8 " CTRL " row_mask:0xf bank_mask:0xf\n\t"                                       \
      "v_fmac_f32_dpp %1, %1, %8 " CTRL " row_mask:0xf bank_mask:0xf\n\t"                                       \
      "v_fmac_f32_dpp %2, %2, %8 " CTRL " row_mask:0xf bank_mask:0xf\n\t"                                       \
      "v_fmac_f32_dpp %3, %3, %8 " CTRL " row_mask:0xf bank_mask:0xf\n\t"                                       \
      "v_fmac_f32_dpp %4, %4, %8 " CTRL " row_mask:0xf bank_mask:0xf\n\t"                                       \
      "v_fmac_f32_dpp %5, %5, %8 " CTRL " row_mask:0xf bank_mask:0xf\n\t"                                       \
      "v_fmac_f32_dpp %6, %6, %8 " CTRL " row_mask:0xf bank_mask:0xf\n\t"                                       \
      "v_fmac_f32_dpp %7, %7, %8 " CTRL " row_mask:0xf bank_mask:0xf"                                           \
      : "+v"(v[0]), "+v"(v[1]), "+v"(v[2]), "+v"(v[3]), "+v"(v[4]), "+v"(v[5]), "+v"(v[6]), "+v"(v[7])            \
      : "v"(M))
  KV_EXCHANGE("quad_perm:[1,0,3,2]", m0);
  KV_EXCHANGE("quad_perm:[2,3,0,1]", m1);
  KV_EXCHANGE("row_half_mirror", m2);
  if constexpr (LANES == 16) KV_EXCHANGE("row_ror:8", m3);
#undef KV_EXCHANGE
  return (__builtin_popcount(c) & 1) ? -1.0f : 1.0f;
}

// Maximum over the LANES lanes that hold one row.
template <int LANES>
__device__ __forceinline__ float row_max(float a) {
  a = fmaxf(a, dpp_f<0xB1>(a));
  a = fmaxf(a, dpp_f<0x4E>(a));
  a = fmaxf(a, dpp_f<0x141>(a));
  if constexpr (LANES == 16) a = fmaxf(a, dpp_f<0x128>(a));
  return a;
}

// 8 consecutive elements at p -> fp32 (exact upcast); p is 16-byte aligned.
__device__ __forceinline__ void load8(const uint8_t* p, int dt, float (&v)[8]) {
  const u32x4 a = *reinterpret_cast<const u32x4*>(p);
  if (dt == kF32) {
    const u32x4 b = *reinterpret_cast<const u32x4*>(p + 16);
#pragma unroll
    for (int i = 0; i < 4; i++) {
      v[i] = __uint_as_float(a[i]);
      v[4 + i] = __uint_as_float(b[i]);
    }
  } else if (dt == kF16) {
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const uint32_t w = a[i];   // a copy: the cast of a vector's element takes its first
      const f16x2 h = __builtin_bit_cast(f16x2, w);
      v[2 * i] = static_cast<float>(h[0]);
      v[2 * i + 1] = static_cast<float>(h[1]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; i++) {
      v[2 * i] = __uint_as_float(a[i] << 16);
      v[2 * i + 1] = __uint_as_float(a[i] & 0xFFFF0000u);
    }
  }
}

// fp32 -> bf16 bits, round to nearest even (a NaN stays a NaN).
__device__ __forceinline__ uint32_t bf16_bits(float x) {
  return __builtin_bit_cast(uint16_t, static_cast<__bf16>(x));
}

template <bool STREAM>
__device__ __forceinline__ void store16(uint8_t* p, const u32x4& a) {
  if constexpr (STREAM)
    __builtin_nontemporal_store(a, reinterpret_cast<u32x4*>(p));
  else
    *reinterpret_cast<u32x4*>(p) = a;
}

// 8 consecutive values -> 8 elements of type dt at p (one rounding, to nearest even). STREAM: past
// the caches.
template <bool STREAM = false>
__device__ __forceinline__ void store8(uint8_t* p, int dt, const float (&v)[8]) {
  u32x4 a, b;
  if (dt == kF32) {
#pragma unroll
    for (int i = 0; i < 4; i++) {
      a[i] = __float_as_uint(v[i]);
      b[i] = __float_as_uint(v[4 + i]);
    }
    store16<STREAM>(p, a);
    store16<STREAM>(p + 16, b);
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; i++) {
    if (dt == kF16) {
      const f16x2 h = {static_cast<_Float16>(v[2 * i]), static_cast<_Float16>(v[2 * i + 1])};
      a[i] = __builtin_bit_cast(uint32_t, h);
    } else {
      a[i] = bf16_bits(v[2 * i]) | (bf16_bits(v[2 * i + 1]) << 16);
    }
  }
  store16<STREAM>(p, a);
}

__device__ __forceinline__ int elem_bytes(int dt) { return dt == kF32 ? 4 : 2; }

}  // namespace kv
}  // namespace convrot
