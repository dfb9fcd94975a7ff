// norm_quant.hip -- root-mean-square norm with the residual's addition, rotated and quantized:
//   h = x + residual (rounded to the rows' type, kept),  v_k = fl(h_k * w_k),
//   codes and scale of v as in rotate_quant.hip, the scale times r = 1 / sqrt(mean(h^2) + eps).
//
// The norm's factor r is one positive number a row. The quantizer divides by the row's own
// maximum, so r cancels out of the codes: they come from v alone, bit for bit whatever the order
// of the sum of squares, and r enters only the row's scale. So one pass does: while a row is
// rotated its squares are summed, and both of the row's reductions (maximum, sum) run together.
//
// Bound by memory: a row is read once (and the residual), h and the codes are written once. Lanes
// are laid out as in the coalesced kernel of rotate_quant.hip (a 16-lane group holds a
// 128-block, lane u the 8-element chunk c(u); a row of nb blocks takes G groups of NI blocks each),
// but blocks past nb are left out by buffer offsets beyond the resource (loads give zeros, stores
// are dropped), so any nb <= 128 fits. Rows past 128 blocks (K > 16384) take a second kernel that reads
// them twice.
//
// 41472 rows of 1024, fp16, with residual and h: 49 us for 297 MB, 6.1 TB/s (a plain copy of 2 GiB reaches 4.9: part of
// the writes is still on its way in the last cache when the kernel ends). 16384 rows of 4096: 81 us for 470 MB, 5.8 TB/s.
// 64 rows of 4096: 3.4 us, a launch's latency.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "internal.h"
#include "rotate_common.h"

namespace convrot {
namespace {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// Past the end of any resource here (all are below 2^31 bytes, see launch_norm_quant): a load
// there gives zeros, a store does nothing.
constexpr uint32_t kNowhere = 0x80000000u;

// The 16-byte words of 8 elements.
template <int DT>
struct Chunk {
  u32x4 w[DT == kF32 ? 2 : 1];
};

template <int DT, int POLICY>
__device__ __forceinline__ Chunk<DT> load_chunk(__amdgpu_buffer_rsrc_t rs, uint32_t off) {
  Chunk<DT> c;
  c.w[0] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, off, 0, POLICY));
  if constexpr (DT == kF32)
    c.w[1] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, off + 16, 0, POLICY));
  return c;
}

template <int DT>
__device__ __forceinline__ void store_chunk(__amdgpu_buffer_rsrc_t rs, uint32_t off, const Chunk<DT>& c) {
  __builtin_amdgcn_raw_buffer_store_b128(c.w[0], rs, off, 0, 0);
  if constexpr (DT == kF32) __builtin_amdgcn_raw_buffer_store_b128(c.w[1], rs, off + 16, 0, 0);
}

template <int DT>
__device__ __forceinline__ void unpack(const Chunk<DT>& c, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; i++) {
    if constexpr (DT == kF32) {
      v[i] = __uint_as_float(c.w[0][i]);
      v[4 + i] = __uint_as_float(c.w[1][i]);
    } else if constexpr (DT == kF16) {
      const uint32_t both = c.w[0][i];   // (a bit cast of the vector's element itself takes the first)
      const f16x2 p = __builtin_bit_cast(f16x2, both);
      v[2 * i] = static_cast<float>(p[0]);
      v[2 * i + 1] = static_cast<float>(p[1]);
    } else {
      v[2 * i] = __uint_as_float(c.w[0][i] << 16);
      v[2 * i + 1] = __uint_as_float(c.w[0][i] & 0xFFFF0000u);
    }
  }
}

// x + r in the rows' type. The binary32 sum of two 16-bit values rounded again to 16 bits is the
// sum rounded once (24 bits hold twice 11, and twice 8, and two more).
template <int DT>
__device__ __forceinline__ Chunk<DT> add_chunks(const Chunk<DT>& x, const Chunk<DT>& r) {
  float a[8], b[8];
  unpack<DT>(x, a);
  unpack<DT>(r, b);
  Chunk<DT> h;
#pragma unroll
  for (int i = 0; i < 4; i++) {
    if constexpr (DT == kF32) {
      h.w[0][i] = __float_as_uint(__fadd_rn(a[i], b[i]));
      h.w[1][i] = __float_as_uint(__fadd_rn(a[4 + i], b[4 + i]));
    } else {
      const f32x2 s = {__fadd_rn(a[2 * i], b[2 * i]), __fadd_rn(a[2 * i + 1], b[2 * i + 1])};
      if constexpr (DT == kF16)
        h.w[0][i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(s, f16x2));
      else
        h.w[0][i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(s, bf16x2));
    }
  }
  return h;
}

// The norm's weights of a chunk: binary32 (W32), or the rows' 16-bit type; none at all (uniform): not touched.
template <int DT, bool W32>
using Weights = Chunk<(W32 || DT == kF32) ? kF32 : DT>;

template <int DT, bool W32>
__device__ __forceinline__ Weights<DT, W32> load_weights(const NormQuantArgs& a, __amdgpu_buffer_rsrc_t rs, uint32_t elem,
                                                         bool there) {
  Weights<DT, W32> w = {};
  if (a.weight) w = load_chunk<(W32 || DT == kF32) ? kF32 : DT, 0>(rs, there ? elem * (W32 || DT == kF32 ? 4 : 2) : kNowhere);
  return w;
}
template <int DT, bool W32>
__device__ __forceinline__ void apply_weights(const NormQuantArgs& a, float (&v)[8], const Weights<DT, W32>& w) {
  if (!a.weight) return;
  float f[8];
  unpack<(W32 || DT == kF32) ? kF32 : DT>(w, f);
#pragma unroll
  for (int i = 0; i < 8; i++) v[i] = __fmul_rn(v[i], f[i]);
}

__device__ __forceinline__ float sum_squares(float ss, const float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; i++) ss = __builtin_fmaf(v[i], v[i], ss);
  return ss;
}

// Sum over the 16 lanes of a DPP row; every lane gets the same bits (each step adds the same two).
__device__ __forceinline__ float row16_sum(float a) {
  a += dpp_f<0xB1>(a);
  a += dpp_f<0x4E>(a);
  a += dpp_f<0x141>(a);
  a += dpp_f<0x128>(a);
  return a;
}

// Whether squares may have left binary32's range: above (bf16 and binary32 rows beyond about
// 1e18), or below it where eps does not outweigh what was lost. 2^-85: squares below 2^-126 add up to less than
// 2^-109 over 2^17 elements, 2^-24 of it.
__device__ __forceinline__ bool squares_lost(float ss, float eps) {
  return !(ss < __builtin_inff()) || (ss < 0x1p-85f && eps < 0x1p-85f);
}

// The row's scale: `scale` is the quantizer's.
__device__ __forceinline__ float norm_scale(float scale, float ss, float K, float eps) {
  const float mean = __fadd_rn(__fdiv_rn(ss, K), eps);
  return __fmul_rn(scale, __fdiv_rn(1.0f, __fsqrt_rn(mean)));
}
__device__ __forceinline__ float norm_scale64(float scale, double ss, int K, float eps) {
  return scale == 0.0f ? 0.0f : static_cast<float>(scale / sqrt(ss / K + eps));
}

// Where codes go: a resource from the workgroup's first row (its panel in the tiled layouts) and
// a row's byte offset in it. All of a workgroup's rows lie in one 256-row panel.
struct CodeDst {
  __amdgpu_buffer_rsrc_t rs;
  uint32_t row;     // of the tiled layouts: within the panel
};
template <int BITS>
__device__ __forceinline__ CodeDst code_dst(const NormQuantArgs& a, int64_t row0, int64_t row, int rows_here) {
  CodeDst d;
  if constexpr (BITS == 6) {
    const int64_t panel = (int64_t)256 * 48 * (a.K >> 6);
    d.rs = rq_rsrc(a.codes + (row0 >> 8) * panel, (uint32_t)panel);
    d.row = (uint32_t)(row & 255);
  } else {
    const int Kb = a.K * BITS / 8;
    if (a.layout == kCodeTiled) {
      d.rs = rq_rsrc(a.codes + (row0 >> 8) * 256 * (int64_t)Kb, 256u * (uint32_t)Kb);
      d.row = (uint32_t)(row & 255) << 6;
    } else {
      d.rs = rq_rsrc(a.codes + row0 * (int64_t)Kb, (uint32_t)(rows_here * Kb));
      d.row = (uint32_t)((row - row0) * Kb);
    }
  }
  return d;
}

// Quantize the chunk of elements elem .. elem + 7 of a row and store its codes (dropped unless `there`).
// FP6 tiles: the four lanes of a quad hold one 24-byte operand string of 32 codes (6 bytes each,
// chunk elem / 8 % 4 of it), six dwords in which the second and the fifth are shared by two lanes:
// the even chunk's lane takes the 16 bits from its partner and stores it.
template <int BITS>
__device__ __forceinline__ void store_codes(const NormQuantArgs& a, const CodeDst& d, uint32_t elem, const float (&v)[8],
                                            float tinv, bool there) {
  if constexpr (BITS == 6) {
    uint32_t g[2];
#pragma unroll
    for (int k = 0; k < 2; k++) {
      uint32_t y[4];
#pragma unroll
      for (int r = 0; r < 4; r++) y[r] = code_bits(v[4 * k + r], tinv);
      g[k] = pack6x4(fp6_bytes(pack4_i8(y[0], y[1], y[2], y[3])));
    }
    const uint32_t low = g[0] | (g[1] << 24), high = g[1] >> 8;          // the chunk's 48 bits
    const uint32_t next = __builtin_amdgcn_mov_dpp((int)low, 0xB1, 0xF, 0xF, true);   // the partner's low 32
    const uint32_t q = (elem >> 3) & 3, h = (elem >> 5) & 1;
    const uint32_t slice = (elem >> 6) * (256 * 48);
    // Bytes 0..15 of the string in plane 1, 16..23 in plane 2 (halves swapped on row bits 3 and 4).
    const uint32_t p1 = slice + d.row * 32 + 16 * (h ^ ((d.row >> 3) & 1));
    const uint32_t p2 = slice + 256 * 32 + d.row * 16 + 8 * (h ^ ((d.row >> 4) & 1));
    // Chunk 0: dwords 0 and 1; 1: dword 2; 2: dwords 3 and 4; 3: dword 5.
    const uint32_t first = (q & 1) ? (low >> 16) | (high << 16) : low;
    const uint32_t at = q == 0 ? p1 : q == 1 ? p1 + 8 : q == 2 ? p1 + 12 : p2 + 4;
    __builtin_amdgcn_raw_buffer_store_b32(first, d.rs, there ? at : kNowhere, 0, 0);
    const uint32_t at2 = q == 0 ? p1 + 4 : p2;
    __builtin_amdgcn_raw_buffer_store_b32(high | (next << 16), d.rs, there && !(q & 1) ? at2 : kNowhere, 0, 0);
  } else {
    uint32_t off = elem * BITS / 8;
    if (a.layout == kCodeTiled) off = ((off >> 6) << 14) + (off & 63);   // 64-byte k steps of 256 rows
    off = there ? off + d.row : kNowhere;
    if constexpr (BITS == 8) {
      uint32_t y[8];
#pragma unroll
      for (int i = 0; i < 8; i++) y[i] = code_bits(v[i], tinv);
      const u32x2 o = {pack4_i8(y[0], y[1], y[2], y[3]), pack4_i8(y[4], y[5], y[6], y[7])};
      __builtin_amdgcn_raw_buffer_store_b64(o, d.rs, off, 0, 0);
    } else {
      __builtin_amdgcn_raw_buffer_store_b32(quant8_i4(v, tinv), d.rs, off, 0, 0);
    }
  }
}

// Stages h = 1 .. 64 of a chunk; the lane's sign factor goes to the multiplier (row_scalars).
__device__ __forceinline__ void rotate_chunk(float (&v)[8], int c) {
  fwht8(v);
  stage_h8(v, (c & 1) ? -1.0f : 1.0f);
  stage_h16(v, (c & 2) ? -1.0f : 1.0f);
  stage_h32(v, (c & 4) ? -1.0f : 1.0f);
  stage_h64(v, (c & 8) ? -1.0f : 1.0f);
}

__device__ __forceinline__ float max_abs8(float m, const float (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 8; j += 2) m = max_abs2(m, v[j], v[j + 1]);
  return m;
}

// The squares of one chunk of a row in 64 bits, from memory: h where it was stored (x or the residual may
// lie under it; a lane stored this chunk itself), else the sum again.
template <int DT, bool RES, typename Rows>
__device__ __forceinline__ double squares64(const NormQuantArgs& a, Rows rows, __amdgpu_buffer_rsrc_t xrs,
                                            __amdgpu_buffer_rsrc_t rrs, int slot, uint32_t elem, bool there) {
  constexpr int kEs = DT == kF32 ? 4 : 2;
  Chunk<DT> h;
  if (a.h) {
    h = load_chunk<DT, 0>(rows(a.h, a.h_stride), there ? (uint32_t)(slot * a.h_stride) + elem * kEs : kNowhere);
  } else {
    h = load_chunk<DT, 0>(xrs, there ? (uint32_t)(slot * a.x_stride) + elem * kEs : kNowhere);
    if constexpr (RES)
      h = add_chunks<DT>(h, load_chunk<DT, 0>(rrs, there ? (uint32_t)(slot * a.res_stride) + elem * kEs : kNowhere));
  }
  float f[8];
  unpack<DT>(h, f);
  double sum = 0.0;
#pragma unroll
  for (int i = 0; i < 8; i++) sum += (double)f[i] * f[i];
  return sum;
}

// One pass: a row of nb <= NI * G blocks in S = 16 * G lanes, 256 / S rows a workgroup of 256
// threads, or one row of S = 128, 256 or 512 threads whose waves join through LDS.
template <int DT, int BITS, int NI, bool RES, bool W32>
__global__ __launch_bounds__(512) void norm_quant_kernel(const NormQuantArgs a) {
  constexpr int kEs = DT == kF32 ? 4 : 2;
  __shared__ float red[2][8];
  const int tid = threadIdx.x, S = a.lanes;
  const bool multi = S > 64;
  const int lg = __builtin_ctz(multi ? 64 : S);
  const int R = multi ? 1 : 256 >> lg;
  const int t = multi ? tid : (tid & (S - 1));
  const int64_t row0 = (int64_t)blockIdx.x * R;
  const int slot = multi ? 0 : tid >> lg;
  const int64_t row = row0 + slot;
  const bool active = row < a.M;
  const int rows_here = (int)(a.M - row0 < R ? a.M - row0 : R);
  const int G = S >> 4, g = t >> 4, u = t & 15;
  const int c = u ^ (3 * ((u >> 2) & 1));
  const int nb = a.K >> 7;

  auto rows = [&](const uint8_t* p, int64_t stride) {
    return rq_rsrc(p + row0 * stride, (uint32_t)((rows_here - 1) * stride + a.K * kEs));
  };
  const __amdgpu_buffer_rsrc_t xrs = rows(a.x, a.x_stride), rrs = rows(RES ? a.res : a.x, RES ? a.res_stride : a.x_stride);
  const __amdgpu_buffer_rsrc_t wrs = rq_rsrc(a.weight, (uint32_t)a.K * (W32 || DT == kF32 ? 4 : 2));
  auto elem = [&](int i) { return (uint32_t)((g + i * G) * 128 + 8 * c); };
  auto there = [&](int i) { return active && g + i * G < nb; };

  Chunk<DT> h[NI], add[NI];
  Weights<DT, W32> w[NI];
#pragma unroll
  for (int i = 0; i < NI; i++)
    h[i] = load_chunk<DT, kNt>(xrs, there(i) ? (uint32_t)(slot * a.x_stride) + elem(i) * kEs : kNowhere);
  if constexpr (RES) {
#pragma unroll
    for (int i = 0; i < NI; i++)
      add[i] = load_chunk<DT, kNt>(rrs, there(i) ? (uint32_t)(slot * a.res_stride) + elem(i) * kEs : kNowhere);
  }
#pragma unroll
  for (int i = 0; i < NI; i++) w[i] = load_weights<DT, W32>(a, wrs, elem(i), there(i));

  float v[NI][8], ss = 0.0f, amax = 0.0f;
#pragma unroll
  for (int i = 0; i < NI; i++) {
    if constexpr (RES) h[i] = add_chunks<DT>(h[i], add[i]);
    unpack<DT>(h[i], v[i]);
    ss = sum_squares(ss, v[i]);
  }
  if (a.h) {
    const __amdgpu_buffer_rsrc_t hrs = rows(a.h, a.h_stride);
#pragma unroll
    for (int i = 0; i < NI; i++)
      store_chunk<DT>(hrs, there(i) ? (uint32_t)(slot * a.h_stride) + elem(i) * kEs : kNowhere, h[i]);
  }
#pragma unroll
  for (int i = 0; i < NI; i++) apply_weights<DT, W32>(a, v[i], w[i]);
#pragma unroll
  for (int i = 0; i < NI; i++) rotate_chunk(v[i], c);
#pragma unroll
  for (int i = 0; i < NI; i++) amax = max_abs8(amax, v[i]);

  amax = row16_max(amax);
  ss = row16_sum(ss);
  if (S >= 32) {
    amax = fmaxf(amax, __shfl_xor(amax, 16, 64));
    ss += __shfl_xor(ss, 16, 64);
  }
  if (S >= 64) {
    amax = fmaxf(amax, __shfl_xor(amax, 32, 64));
    ss += __shfl_xor(ss, 32, 64);
  }
  if (multi) {
    if ((tid & 63) == 0) {
      red[0][tid >> 6] = amax;
      red[1][tid >> 6] = ss;
    }
    __syncthreads();
    amax = red[0][0];
    ss = red[1][0];
    for (int k = 1; k < (S >> 6); k++) {
      amax = fmaxf(amax, red[0][k]);
      ss += red[1][k];
    }
  }
  float tinv, scale;
  row_scalars(amax, BITS == 8 ? 127.0f : 7.0f, c, tinv, scale);
  const CodeDst dst = code_dst<BITS>(a, row0, row, rows_here);
#pragma unroll
  for (int i = 0; i < NI; i++) store_codes<BITS>(a, dst, elem(i), v[i], tinv, there(i));
  if (squares_lost(ss, a.eps)) {   // rare; the same for all lanes of a row
    double sum = 0.0;
    for (int i = 0; i < NI; i++) sum += squares64<DT, RES>(a, rows, xrs, rrs, slot, elem(i), there(i));
    for (int m = 1; m < (multi ? 64 : S); m <<= 1) sum += __shfl_xor(sum, m, 64);
    if (multi) {
      __shared__ double red64[8];
      if ((tid & 63) == 0) red64[tid >> 6] = sum;
      __syncthreads();
      sum = red64[0];
      for (int k = 1; k < (S >> 6); k++) sum += red64[k];
    }
    scale = norm_scale64(scale, sum, a.K, a.eps);
  } else {
    scale = norm_scale(scale, ss, (float)a.K, a.eps);
  }
  if (active && t == 0) a.scales[row] = scale;
}

// Rows of more than 128 blocks: a workgroup a row, read twice. The first pass adds, stores h, sums the
// squares and finds the maximum, the second rotates again and quantizes. Each lane reads back only
// what it stored itself.
template <int DT, int BITS, bool RES, bool W32>
__global__ __launch_bounds__(256) void norm_quant_long_kernel(const NormQuantArgs a) {
  constexpr int kEs = DT == kF32 ? 4 : 2;
  __shared__ float red[2][4];
  __shared__ double red64[4];
  const int tid = threadIdx.x;
  const int64_t row0 = blockIdx.x;
  const int g = tid >> 4, u = tid & 15;
  const int c = u ^ (3 * ((u >> 2) & 1));
  const int nb = a.K >> 7;
  auto rows = [&](const uint8_t* p, int64_t stride) { return rq_rsrc(p + row0 * stride, (uint32_t)(a.K * kEs)); };
  const __amdgpu_buffer_rsrc_t xrs = rows(a.x, a.x_stride), rrs = rows(RES ? a.res : a.x, RES ? a.res_stride : a.x_stride);
  const __amdgpu_buffer_rsrc_t hrs = rows(a.h ? a.h : a.x, a.h ? a.h_stride : a.x_stride);
  const __amdgpu_buffer_rsrc_t wrs = rq_rsrc(a.weight, (uint32_t)a.K * (W32 || DT == kF32 ? 4 : 2));
  auto row_chunk = [&](uint32_t e, bool there) {
    const uint32_t off = there ? e * kEs : kNowhere;
    Chunk<DT> h = load_chunk<DT, 0>(xrs, off);
    if constexpr (RES) h = add_chunks<DT>(h, load_chunk<DT, 0>(rrs, off));
    return h;
  };
  float ss = 0.0f, amax = 0.0f;
  for (int b = g; b < nb + g; b += 16) {   // nb rounded up to 16: all lanes stay for the exchanges
    const bool there = b < nb;
    const uint32_t e = (uint32_t)(b * 128 + 8 * c);
    const Chunk<DT> h = row_chunk(e, there);
    float v[8];
    unpack<DT>(h, v);
    if (a.h) store_chunk<DT>(hrs, there ? e * kEs : kNowhere, h);
    ss = sum_squares(ss, v);
    apply_weights<DT, W32>(a, v, load_weights<DT, W32>(a, wrs, e, there));
    rotate_chunk(v, c);
    amax = max_abs8(amax, v);
  }
  amax = wave_max(row16_max(amax), 64);
  ss = row16_sum(ss);
  ss += __shfl_xor(ss, 16, 64);
  ss += __shfl_xor(ss, 32, 64);
  if ((tid & 63) == 0) {
    red[0][tid >> 6] = amax;
    red[1][tid >> 6] = ss;
  }
  __syncthreads();
  amax = fmaxf(fmaxf(red[0][0], red[0][1]), fmaxf(red[0][2], red[0][3]));
  ss = (red[1][0] + red[1][1]) + (red[1][2] + red[1][3]);
  float tinv, scale;
  row_scalars(amax, BITS == 8 ? 127.0f : 7.0f, c, tinv, scale);
  const CodeDst dst = code_dst<BITS>(a, row0, row0, 1);
  const bool lost = squares_lost(ss, a.eps);
  double sum = 0.0;
  for (int b = g; b < nb + g; b += 16) {
    const bool there = b < nb;
    const uint32_t e = (uint32_t)(b * 128 + 8 * c);
    const Chunk<DT> h = a.h ? load_chunk<DT, 0>(hrs, there ? e * kEs : kNowhere) : row_chunk(e, there);
    float v[8];
    unpack<DT>(h, v);
    if (lost)
      for (int i = 0; i < 8; i++) sum += (double)v[i] * v[i];
    apply_weights<DT, W32>(a, v, load_weights<DT, W32>(a, wrs, e, there));
    rotate_chunk(v, c);
    store_codes<BITS>(a, dst, e, v, tinv, there);
  }
  if (lost) {   // the same for the whole workgroup
    for (int m = 1; m < 64; m <<= 1) sum += __shfl_xor(sum, m, 64);
    if ((tid & 63) == 0) red64[tid >> 6] = sum;
    __syncthreads();
    scale = norm_scale64(scale, (red64[0] + red64[1]) + (red64[2] + red64[3]), a.K, a.eps);
  } else {
    scale = norm_scale(scale, ss, (float)a.K, a.eps);
  }
  if (tid == 0) a.scales[row0] = scale;
}

// Groups of a row of nb <= 128 blocks (16 lanes each). Below 24 blocks the fewest that leave at most four
// blocks a group, above it as many as hold nb in four, as in choose_coalesced().
int choose_groups(int64_t nb) {
  if (nb > 64) return 32;
  if (nb >= 24) return 16;
  int G = 1;
  while ((nb + G - 1) / G > 4) G *= 2;
  return G;
}

template <int DT, int BITS, bool RES, bool W32>
hipError_t launch_kernel(const NormQuantArgs& args, hipStream_t st) {
  NormQuantArgs a = args;
  const int64_t nb = a.K / 128;
  if (nb > 128) {
    hipLaunchKernelGGL((norm_quant_long_kernel<DT, BITS, RES, W32>), dim3((unsigned)a.M), dim3(256), 0, st, a);
    return hipGetLastError();
  }
  const int G = choose_groups(nb);
  a.lanes = 16 * G;
  const int threads = a.lanes <= 64 ? 256 : a.lanes, R = threads / a.lanes;
  const dim3 grid((unsigned)((a.M + R - 1) / R)), block(threads);
  switch ((nb + G - 1) / G) {
    case 1: hipLaunchKernelGGL((norm_quant_kernel<DT, BITS, 1, RES, W32>), grid, block, 0, st, a); break;
    case 2: hipLaunchKernelGGL((norm_quant_kernel<DT, BITS, 2, RES, W32>), grid, block, 0, st, a); break;
    case 3: hipLaunchKernelGGL((norm_quant_kernel<DT, BITS, 3, RES, W32>), grid, block, 0, st, a); break;
    default: hipLaunchKernelGGL((norm_quant_kernel<DT, BITS, 4, RES, W32>), grid, block, 0, st, a); break;
  }
  return hipGetLastError();
}

template <int DT, int BITS>
hipError_t launch_bits(const NormQuantArgs& a, hipStream_t st) {
  if constexpr (DT != kF32) {   // rows of binary32 have weights of binary32: one kernel
    if (a.weight_f32) return a.res ? launch_kernel<DT, BITS, true, true>(a, st) : launch_kernel<DT, BITS, false, true>(a, st);
  }
  return a.res ? launch_kernel<DT, BITS, true, false>(a, st) : launch_kernel<DT, BITS, false, false>(a, st);
}

template <int DT>
hipError_t launch_dt(const NormQuantArgs& a, int bits, hipStream_t st) {
  if (a.layout == kCodeFp6X) return launch_bits<DT, 6>(a, st);
  return bits == 8 ? launch_bits<DT, 8>(a, st) : launch_bits<DT, 4>(a, st);
}

}  // namespace

int64_t norm_quant_threads(int64_t M, int64_t K) {
  const int lanes = K / 128 > 128 ? 256 : 16 * choose_groups(K / 128), threads = lanes <= 64 ? 256 : lanes;
  const int64_t R = threads / lanes;
  return (M + R - 1) / R * threads;
}

hipError_t launch_norm_quant(const NormQuantArgs& a, int dt, int bits, hipStream_t stream) {
  if (a.M == 0) return hipSuccess;
  switch (dt) {
    case kF32: return launch_dt<kF32>(a, bits, stream);
    case kF16: return launch_dt<kF16>(a, bits, stream);
    default: return launch_dt<kBF16>(a, bits, stream);
  }
}

}  // namespace convrot
