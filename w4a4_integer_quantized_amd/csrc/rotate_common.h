// rotate_common.h -- pieces shared by the kernels that rotate rows (block-128 Walsh-Hadamard) and
// quantize them: exact upcasts, butterfly stages in a lane and across lanes, the row's multiplier and
// scale, codes packed and stored in every layout. Device code only; each translation unit gets its own
// copy.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "internal.h"

namespace convrot {
namespace {

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

constexpr float kInvSqrtBlock = 0x1.6a09e6p-4f;  // binary32 nearest to 1/sqrt(128)
constexpr float kRoundMagic = 12582912.0f;       // 1.5 * 2^23

template <int DPP_CTRL>
__device__ __forceinline__ float dpp_f(float v) {
  return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), DPP_CTRL, 0xF, 0xF, true));
}

// 16 bytes at p.
__device__ __forceinline__ u32x4 load16(const void* p) { return *static_cast<const u32x4*>(p); }

// 8 consecutive elements -> fp32 (exact upcast).
template <int DT>
__device__ __forceinline__ void load8(const void* base, int64_t elem, float (&v)[8]) {
  if constexpr (DT == kF32) {
    const float* p = static_cast<const float*>(base) + elem;
    const u32x4 a = load16(p), b = load16(p + 4);
#pragma unroll
    for (int i = 0; i < 4; i++) {
      v[i] = __uint_as_float(a[i]);
      v[4 + i] = __uint_as_float(b[i]);
    }
  } else {
    const u32x4 a = load16(static_cast<const uint16_t*>(base) + elem);
    const uint32_t w[4] = {a[0], a[1], a[2], a[3]};
#pragma unroll
    for (int i = 0; i < 4; i++) {
      if constexpr (DT == kF16) {
        v[2 * i] = static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(w[i] & 0xFFFFu)));
        v[2 * i + 1] = static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(w[i] >> 16)));
      } else {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      }
    }
  }
}

// Butterfly stages h = 1, 2, 4 on 8 consecutive elements.
__device__ __forceinline__ void fwht8(float (&v)[8]) {
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
}

// Cross-lane stages h = 8, 16, 32, 64 (lane masks 1, 2, 7, 8), sign-tracked.
__device__ __forceinline__ void cross_stages(float (&v)[8], float m0, float m1, float m2, float m3) {
#pragma unroll
  for (int i = 0; i < 8; i++) v[i] = __builtin_fmaf(dpp_f<0xB1>(v[i]), m0, v[i]);   // quad_perm [1,0,3,2]
#pragma unroll
  for (int i = 0; i < 8; i++) v[i] = __builtin_fmaf(dpp_f<0x4E>(v[i]), m1, v[i]);   // quad_perm [2,3,0,1]
#pragma unroll
  for (int i = 0; i < 8; i++) v[i] = __builtin_fmaf(dpp_f<0x141>(v[i]), m2, v[i]);  // row_half_mirror
#pragma unroll
  for (int i = 0; i < 8; i++) v[i] = __builtin_fmaf(dpp_f<0x128>(v[i]), m3, v[i]);  // row_ror:8
}

__device__ __forceinline__ uint32_t code_bits(float u, float tinv) {
  return __float_as_uint(__fadd_rn(__fmul_rn(u, tinv), kRoundMagic));
}

// Byte offset of code byte kb (of Kb per row) of row `row`: row-major, or the tiled layout of
// convrot.h ([256-row panel][64-byte k step][256 rows][64 B]; Kb is a multiple of 64).
__device__ __forceinline__ int64_t code_offset(int64_t row, int64_t kb, int64_t Kb, bool tiled) {
  if (!tiled) return row * Kb + kb;
  return (((row >> 8) * (Kb >> 6) + (kb >> 6)) << 14) + ((row & 255) << 6) + (kb & 63);
}

// Quantize + store one piece (8 codes) at `dst` (their bytes are contiguous in both layouts).
template <int BITS>
__device__ __forceinline__ void store_piece(uint8_t* dst, const float (&v)[8], float tinv) {
  uint32_t y[8];
#pragma unroll
  for (int i = 0; i < 8; i++) y[i] = code_bits(v[i], tinv);
  if constexpr (BITS == 8) {
    uint2 o;
    o.x = (y[0] & 0xFFu) | ((y[1] & 0xFFu) << 8) | ((y[2] & 0xFFu) << 16) | (y[3] << 24);
    o.y = (y[4] & 0xFFu) | ((y[5] & 0xFFu) << 8) | ((y[6] & 0xFFu) << 16) | (y[7] << 24);
    *reinterpret_cast<uint2*>(dst) = o;
  } else {
    uint32_t o = 0;
#pragma unroll
    for (int i = 0; i < 8; i++) o |= (y[i] & 0xFu) << (4 * i);
    *reinterpret_cast<uint32_t*>(dst) = o;
  }
}

__device__ __forceinline__ float wave_max(float a, int width) {
  for (int off = 1; off < width; off <<= 1) a = fmaxf(a, __shfl_xor(a, off, 64));
  return a;
}

// The row's multiplier and scale. A row whose absmax is zero, or too small for fl(q_max / a)
// to be finite, is quantized as a zero row: multiplier 0 (every code 0) and scale 0.
__device__ __forceinline__ void row_scalars(float a, float qmax, int j, float& tinv, float& scale) {
  float inv = (a > 0.0f) ? __fdiv_rn(qmax, a) : 0.0f;
  if (__builtin_isinf(inv)) inv = 0.0f;
  scale = inv != 0.0f ? __fdiv_rn(__fmul_rn(a, kInvSqrtBlock), qmax) : 0.0f;
  tinv = (__builtin_popcount(j) & 1) ? -inv : inv;
}

// Butterfly on the two fp16 halves a (low) and b (high) of a dword, fused with the exact
// upcast: v_fma_mix_f32 takes fp16 operands exactly and rounds a*(+-1) + b once to fp32, i.e.
// fl(a + b) and fl(a - b). (Written out because the compiler turns fma(x, 1, y) into an add
// and then needs separate conversions.)
__device__ __forceinline__ void bfly_f16(uint32_t w, float& lo, float& hi) {
  asm("v_fma_mix_f32 %0, %2, 1.0, %2 op_sel:[0,0,1] op_sel_hi:[1,0,1]\n\t"
      "v_fma_mix_f32 %1, %2, -1.0, %2 op_sel:[1,0,0] op_sel_hi:[1,0,1]"
      : "=&v"(lo), "=v"(hi)
      : "v"(w));
}

// Load piece (8 elements) and apply butterfly stage h = 1 (with the upcast).
template <int DT>
__device__ __forceinline__ void load_stage1(const void* base, int64_t elem, float (&v)[8]) {
  if constexpr (DT == kF16) {
    const u32x4 a = load16(static_cast<const uint16_t*>(base) + elem);
    bfly_f16(a[0], v[0], v[1]);
    bfly_f16(a[1], v[2], v[3]);
    bfly_f16(a[2], v[4], v[5]);
    bfly_f16(a[3], v[6], v[7]);
  } else {
    load8<DT>(base, elem, v);
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      const float a = v[i], b = v[i + 1];
      v[i] = __fadd_rn(a, b);
      v[i + 1] = __fsub_rn(a, b);
    }
  }
}

// Stages h = 2, 4 inside a piece.
__device__ __forceinline__ void stages_2_4(float (&v)[8]) {
#pragma unroll
  for (int h = 2; h < 8; h <<= 1) {
#pragma unroll
    for (int i = 0; i < 8; i++) {
      if ((i & h) == 0) {
        const float a = v[i], b = v[i + h];
        v[i] = __fadd_rn(a, b);
        v[i + h] = __fsub_rn(a, b);
      }
    }
  }
}

__device__ __forceinline__ void bfly_pieces(float (&x)[8], float (&y)[8]) {
#pragma unroll
  for (int r = 0; r < 8; r++) {
    const float a = x[r], b = y[r];
    x[r] = __fadd_rn(a, b);
    y[r] = __fsub_rn(a, b);
  }
}

// Code bytes of 8 quantized values -> int8 pair of dwords or one int4 dword.
__device__ __forceinline__ uint32_t pack4_i8(uint32_t y0, uint32_t y1, uint32_t y2, uint32_t y3) {
  const uint32_t lo = __builtin_amdgcn_perm(y1, y0, 0x0c0c0400u);   // [y0.b0, y1.b0, 0, 0]
  const uint32_t hi = __builtin_amdgcn_perm(y3, y2, 0x04000c0cu);   // [0, 0, y2.b0, y3.b0]
  return lo | hi;
}

// Quantize + store the 32 consecutive codes of v[0..3] at `dst` (32 or 16 contiguous bytes in
// both layouts: a lane's run never crosses a 64-byte k step).
template <int BITS>
__device__ __forceinline__ void quant_store32(uint8_t* dst, const float (&v)[4][8], float tinv) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 4; i++) {
    uint32_t y[8];
#pragma unroll
    for (int r = 0; r < 8; r++) y[r] = code_bits(v[i][r], tinv);
    if constexpr (BITS == 8) {
      w[2 * i] = pack4_i8(y[0], y[1], y[2], y[3]);
      w[2 * i + 1] = pack4_i8(y[4], y[5], y[6], y[7]);
    } else {
      uint32_t o = 0;
#pragma unroll
      for (int r = 0; r < 8; r++) o |= (y[r] & 0xFu) << (4 * r);
      w[i] = o;
    }
  }
  if constexpr (BITS == 8) {
    uint4* p = reinterpret_cast<uint4*>(dst);
    p[0] = make_uint4(w[0], w[1], w[2], w[3]);
    p[1] = make_uint4(w[4], w[5], w[6], w[7]);
  } else {
    *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// ---- FP6 tiles (4-bit codes stored as FP6 E2M3 for the FP6 matrix cores; see convrot.h) ----
// Byte `b` (0..23) of the 24-byte operand string of row `row`, 64-element slice `s`, half `h`,
// in panels of P rows: plane 1 (bytes 0..15, 32 B per row) then plane 2 (bytes 16..23, 16 B per
// row), each with its two halves swapped on row bit 3 (plane 1) or bit 4 (plane 2).
__device__ __forceinline__ int64_t fp6_offset(int64_t row, int s, int h, int b, int P, int nsl) {
  const int64_t base = ((row / P) * nsl + s) * (int64_t)(P * 48);
  const int rr = (int)(row % P);
  if (b < 16) return base + rr * 32 + 16 * (h ^ ((rr >> 3) & 1)) + b;
  return base + P * 32 + rr * 16 + 8 * (h ^ ((rr >> 4) & 1)) + (b - 16);
}

// FP6 E2M3 bytes of four codes given as two's-complement bytes in [-7, 7]: byte permutes look
// the low three bits up in {0, 8, 16, 20, 24, 26, 28, 30} (0, 1.0, 2.0, 1.5 * 2, 4.0,
// 1.25 * 4, 1.5 * 4, 1.75 * 4) for non-negative codes and in the patterns of -(8 - j) (sign bit
// 32 set) for negative ones, and a bytewise select by the sign picks one.
__device__ __forceinline__ uint32_t fp6_bytes(uint32_t d) {
  const uint32_t j = d & 0x07070707u;
  const uint32_t pos = __builtin_amdgcn_perm(0x1E1C1A18u, 0x14100800u, j);
  const uint32_t neg = __builtin_amdgcn_perm(0x28303438u, 0x3A3C3E00u, j);
  const uint32_t s = ((d >> 7) & 0x01010101u) * 0xFFu;   // 0xFF in the bytes of negative codes
  return (neg & s) | (pos & ~s);
}

// Four 6-bit codes (the low six bits of each byte of c) -> one 24-bit field, code i at bit 6i.
__device__ __forceinline__ uint32_t pack6x4(uint32_t c) {
  uint32_t g = (c & 0x3Fu) | ((c >> 2) & ~0x3Fu);
  g = (g & 0xFFFu) | ((c >> 4) & ~0xFFFu);
  return (g & 0x3FFFFu) | ((c >> 6) & ~0x3FFFFu);
}

// Quantize the 32 consecutive values of v[0..3] (one lane's operand string: half h of slice s)
// and store them as FP6 tiles.
__device__ __forceinline__ void quant_store32_fp6(uint8_t* Q, int64_t row, int s, int h, int P, int nsl,
                                                  const float (&v)[4][8], float tinv) {
  uint32_t g[8];
#pragma unroll
  for (int i = 0; i < 4; i++) {
#pragma unroll
    for (int q = 0; q < 2; q++) {
      uint32_t y[4];
#pragma unroll
      for (int r = 0; r < 4; r++) y[r] = code_bits(v[i][4 * q + r], tinv);
      g[2 * i + q] = pack6x4(fp6_bytes(pack4_i8(y[0], y[1], y[2], y[3])));
    }
  }
  const uint4 lo = make_uint4(g[0] | (g[1] << 24), (g[1] >> 8) | (g[2] << 16), (g[2] >> 16) | (g[3] << 8),
                              g[4] | (g[5] << 24));
  const uint2 hi = make_uint2((g[5] >> 8) | (g[6] << 16), (g[6] >> 16) | (g[7] << 8));
  *reinterpret_cast<uint4*>(Q + fp6_offset(row, s, h, 0, P, nsl)) = lo;
  *reinterpret_cast<uint2*>(Q + fp6_offset(row, s, h, 16, P, nsl)) = hi;
}

// The same for one piece of 8 consecutive values (elements 8q .. 8q+7 of the string, 6 bytes at
// byte 6q), written as three 16-bit words (each lies within one plane).
__device__ __forceinline__ void store_piece_fp6(uint8_t* Q, int64_t row, int s, int h, int q, int P, int nsl,
                                                const float (&v)[8], float tinv) {
  uint32_t g[2];
#pragma unroll
  for (int k = 0; k < 2; k++) {
    uint32_t y[4];
#pragma unroll
    for (int r = 0; r < 4; r++) y[r] = code_bits(v[4 * k + r], tinv);
    g[k] = pack6x4(fp6_bytes(pack4_i8(y[0], y[1], y[2], y[3])));
  }
  const uint16_t w[3] = {static_cast<uint16_t>(g[0] & 0xFFFFu),
                         static_cast<uint16_t>((g[0] >> 16) | ((g[1] & 0xFFu) << 8)),
                         static_cast<uint16_t>(g[1] >> 8)};
#pragma unroll
  for (int k = 0; k < 3; k++) *reinterpret_cast<uint16_t*>(Q + fp6_offset(row, s, h, 6 * q + 2 * k, P, nsl)) = w[k];
}

// v[r] = partner(v[r]) * m + v[r] on 8 registers, the partner read through DPP (CTRL): one
// v_fmac_f32 with a DPP source per value, i.e. the single rounding of v +- partner. Each
// instruction reads only the register it writes, so only the first can follow the VALU write of
// its source; the leading s_nop covers the DPP read-after-write (and exec-write) wait states.
#define RQ_FMAC_DPP8(CTRL)                                                                        \
  asm volatile("s_nop 4\n\t"                                                                      \
               "v_fmac_f32_dpp %0, %0, %8 " CTRL " row_mask:0xf bank_mask:0xf\n\t"                \
               "v_fmac_f32_dpp %1, %1, %8 " CTRL " row_mask:0xf bank_mask:0xf\n\t"                \
               "v_fmac_f32_dpp %2, %2, %8 " CTRL " row_mask:0xf bank_mask:0xf\n\t"                \
               "v_fmac_f32_dpp %3, %3, %8 " CTRL " row_mask:0xf bank_mask:0xf\n\t"                \
               "v_fmac_f32_dpp %4, %4, %8 " CTRL " row_mask:0xf bank_mask:0xf\n\t"                \
               "v_fmac_f32_dpp %5, %5, %8 " CTRL " row_mask:0xf bank_mask:0xf\n\t"                \
               "v_fmac_f32_dpp %6, %6, %8 " CTRL " row_mask:0xf bank_mask:0xf\n\t"                \
               "v_fmac_f32_dpp %7, %7, %8 " CTRL " row_mask:0xf bank_mask:0xf"                    \
               : "+v"(v[0]), "+v"(v[1]), "+v"(v[2]), "+v"(v[3]), "+v"(v[4]), "+v"(v[5]),         \
                 "+v"(v[6]), "+v"(v[7])                                                           \
               : "v"(m))

// Cross-lane stages h = 8, 16, 32, 64 on a chunk held by lane u of a 16-lane group with chunk
// index c(u) = u ^ (3 * ((u >> 2) & 1)): flipping bit k of c is lane xor 1, 2, 7, 8, i.e.
// quad_perm [1,0,3,2], quad_perm [2,3,0,1], row_half_mirror and row_ror:8. Sign-tracked with
// m_k = -1 on the lane whose bit k of c is set, as in the quad scheme above.
__device__ __forceinline__ void stage_h8(float (&v)[8], float m) { RQ_FMAC_DPP8("quad_perm:[1,0,3,2]"); }
__device__ __forceinline__ void stage_h16(float (&v)[8], float m) { RQ_FMAC_DPP8("quad_perm:[2,3,0,1]"); }
__device__ __forceinline__ void stage_h32(float (&v)[8], float m) { RQ_FMAC_DPP8("row_half_mirror"); }
__device__ __forceinline__ void stage_h64(float (&v)[8], float m) { RQ_FMAC_DPP8("row_ror:8"); }
#undef RQ_FMAC_DPP8

// max(a, |x|, |y|) in one instruction.
__device__ __forceinline__ float max_abs2(float a, float x, float y) {
  float r;
  asm("v_max3_f32 %0, |%1|, |%2|, %3" : "=v"(r) : "v"(x), "v"(y), "v"(a));
  return r;
}

// Max over the 16 lanes of a DPP row (the same four exchanges as the stages), each step one
// v_max_f32 with a DPP source (s_nop 1: the wait states of a DPP read after a VALU write).
__device__ __forceinline__ float row16_max(float a) {
  asm volatile("s_nop 1\n\t"
               "v_max_f32_dpp %0, %0, %0 quad_perm:[1,0,3,2] row_mask:0xf bank_mask:0xf\n\t"
               "s_nop 1\n\t"
               "v_max_f32_dpp %0, %0, %0 quad_perm:[2,3,0,1] row_mask:0xf bank_mask:0xf\n\t"
               "s_nop 1\n\t"
               "v_max_f32_dpp %0, %0, %0 row_half_mirror row_mask:0xf bank_mask:0xf\n\t"
               "s_nop 1\n\t"
               "v_max_f32_dpp %0, %0, %0 row_ror:8 row_mask:0xf bank_mask:0xf"
               : "+v"(a));
  return a;
}

typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));

// The int8 codes of 8 values as two dwords: p = fl(u * tinv), then fl(p + 1.5 * 2^23), whose low
// byte is the code, written straight into byte i of the dword by the add itself (SDWA
// dst_sel:BYTE_i, the other bytes kept).
__device__ __forceinline__ u32x2 quant8_i8(const float (&v)[8], float tinv) {
  const float magic = kRoundMagic;
  uint32_t d[2];
#pragma unroll
  for (int h = 0; h < 2; h++) {
    const float p0 = __fmul_rn(v[4 * h], tinv), p1 = __fmul_rn(v[4 * h + 1], tinv);
    const float p2 = __fmul_rn(v[4 * h + 2], tinv), p3 = __fmul_rn(v[4 * h + 3], tinv);
    uint32_t w;
    asm("v_add_f32_sdwa %0, %1, %2 dst_sel:BYTE_0 dst_unused:UNUSED_PAD src0_sel:DWORD src1_sel:DWORD"
        : "=v"(w) : "v"(p0), "v"(magic));
    asm("v_add_f32_sdwa %0, %1, %2 dst_sel:BYTE_1 dst_unused:UNUSED_PRESERVE src0_sel:DWORD src1_sel:DWORD"
        : "+v"(w) : "v"(p1), "v"(magic));
    asm("v_add_f32_sdwa %0, %1, %2 dst_sel:BYTE_2 dst_unused:UNUSED_PRESERVE src0_sel:DWORD src1_sel:DWORD"
        : "+v"(w) : "v"(p2), "v"(magic));
    asm("v_add_f32_sdwa %0, %1, %2 dst_sel:BYTE_3 dst_unused:UNUSED_PRESERVE src0_sel:DWORD src1_sel:DWORD"
        : "+v"(w) : "v"(p3), "v"(magic));
    d[h] = w;
  }
  return u32x2{d[0], d[1]};
}

// The int4 codes of 8 values, code i in bits 4i .. 4i+3.
__device__ __forceinline__ uint32_t quant8_i4(const float (&v)[8], float tinv) {
  uint32_t o = 0;
#pragma unroll
  for (int i = 0; i < 8; i++) o |= (code_bits(v[i], tinv) & 0xFu) << (4 * i);
  return o;
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rq_rsrc(const void* base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)bytes, 0x00020000);
}

constexpr int kNt = 2;   // buffer-load cache policy: nontemporal (X is streamed once)

}  // namespace
}  // namespace convrot
