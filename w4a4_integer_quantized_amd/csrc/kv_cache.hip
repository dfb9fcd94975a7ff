// kv_cache.hip -- keys and values rotated and quantized into a paged cache as they are written,
// and read back (rq_kv_cache_write, rq_kv_cache_read; layout and arithmetic in convrot.h).
//
// Both are one pass over their data and bound by memory. A head row of D elements takes
// min(D, 128) / 8 lanes, 8 consecutive elements (16 bytes of fp16 / bf16) a lane and block, so
// that its transform is seven (six) butterfly stages of which three stay in the lane and the
// others are DPP exchanges; a 256-element row is two blocks in the same lanes. A wave holds the
// same head of 4 (D = 64: 8) consecutive tokens. Lanes are never masked off inside the transform:
// rows past the end load the last row and store nothing.
#include "kv_common.h"

namespace convrot {
namespace {

using namespace kv;

constexpr int kThreads = 256;
// Rows read back beyond this are stored past the caches: they would not stay in them (the L2s hold
// 32 MiB) until they are used. 65536 tokens, 8 heads of 128 (268 MB): 118 us through the caches,
// 78 us past them; 5184 tokens, 16 heads of 64 (21 MB): 9.4 us either way.
constexpr int64_t kStreamBytes = int64_t(32) << 20;
constexpr float kRoundMagic = 12582912.0f;   // 1.5 * 2^23: its low mantissa bits hold the code

// Where a lane's token is. Its row among the workgroup's is clamped to the last token's; an address is
// a base that the workgroup shares and one product of a 32-bit and a 64-bit factor.
struct Token {
  int64_t first;    // the workgroup's first token
  uint32_t row;     // this lane's, counted from it
  bool there;       // it is one of the call's
};
template <int ROWS>
__device__ __forceinline__ Token token_of(const KvCacheArgs& a, int lanes) {
  Token t;
  t.first = (int64_t)blockIdx.x * ROWS;
  const int64_t left = a.tokens - t.first;
  const uint32_t row = threadIdx.x / lanes, last = left < ROWS ? static_cast<uint32_t>(left) - 1 : ROWS - 1;
  t.there = row <= last;
  t.row = t.there ? row : last;
  return t;
}
__device__ __forceinline__ int64_t row_offset(const Token& t, int head, int64_t token_stride, int64_t head_stride, int es) {
  const int64_t base = (t.first * token_stride + head * head_stride) * es;
  return base + static_cast<int64_t>(t.row * static_cast<uint64_t>(token_stride * es));
}

// The block of (page, head) that holds a slot, and the token's place in it. False if the slot lies
// outside the cache.
struct Place {
  uint8_t* block;
  int off;
};
__device__ __forceinline__ bool find(const KvCacheArgs& a, int64_t slot, int head, Place& p) {
  const bool in = slot >= 0 && slot < a.num_pages << a.lps;
  const uint32_t page = in ? static_cast<uint32_t>(slot >> a.lps) : 0u;
  p.block = a.cache + head * a.head_bytes + page * static_cast<uint64_t>(a.head_bytes * a.heads);
  p.off = in ? static_cast<int>(slot & ((1 << a.lps) - 1)) : 0;
  return in;
}

// The low bytes of four values.
__device__ __forceinline__ uint32_t low_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  const uint32_t lo = __builtin_amdgcn_perm(b, a, 0x0c0c0400u), hi = __builtin_amdgcn_perm(d, c, 0x04000c0cu);
  return lo | hi;
}

// The row's codes: rounded half to even by adding 1.5 * 2^23 (|u * inv| <= q_max < 2^22). `inv`
// carries the lane's sign.
template <int BITS>
__device__ __forceinline__ void codes8(const float (&v)[8], float inv, uint32_t& lo, uint32_t& hi) {
  uint32_t y[8];
#pragma unroll
  for (int i = 0; i < 8; i++) y[i] = __float_as_uint(__fadd_rn(__fmul_rn(v[i], inv), kRoundMagic));
  if constexpr (BITS == 8) {
    lo = low_bytes(y[0], y[1], y[2], y[3]);
    hi = low_bytes(y[4], y[5], y[6], y[7]);
  } else {
    const uint32_t even = low_bytes(y[0], y[2], y[4], y[6]), odd = low_bytes(y[1], y[3], y[5], y[7]);
    lo = (even & 0x0F0F0F0Fu) | ((odd << 4) & 0xF0F0F0F0u);
    hi = 0;
  }
}

// One workgroup: kThreads / kLanes rows, i.e. that many consecutive tokens of one head; gridDim.y
// is the heads. The keys' row and the values' row of a token are the same lanes' work, both loaded
// before either is worked on. Its instructions show beside its traffic, so the two rows' divisions
// are one: lanes whose bit 2 is set divide for the values' row, the others for the keys', and the
// halves exchange the quotients. A write and its read-back, with addresses from one product a lane
// and codes gathered by byte permutes as well: 143 us against 146 with a division for each row, at
// 65536 tokens of 8 heads of 128; 16.7 against 17.2 at 5184 tokens of 16 heads of 64.
template <int D, int BITS>
__global__ __launch_bounds__(kThreads) void kv_write_kernel(KvCacheArgs a) {
  using R = Row<D, BITS>;
  const int u = threadIdx.x % R::kLanes, c = chunk_of_lane(u);
  const Token t = token_of<kThreads / R::kLanes>(a, R::kLanes);
  const int head = blockIdx.y;
  const int es = elem_bytes(a.dt);
  float v[2][R::kChunks][8];
#pragma unroll
  for (int part = 0; part < 2; part++) {   // keys, values
    const uint8_t* x = part ? a.v + row_offset(t, head, a.v_token, a.v_head, es)
                            : a.k + row_offset(t, head, a.k_token, a.k_head, es);
#pragma unroll
    for (int b = 0; b < R::kChunks; b++) load8(x + (b * 128 + c * 8) * es, a.dt, v[part][b]);
  }
  Place p;
  const bool in = find(a, a.slots[t.first + t.row], head, p) && t.there;
  const int page = 1 << a.lps;
  float sign = 1.0f, m[2];
#pragma unroll
  for (int part = 0; part < 2; part++) {
    m[part] = 0.0f;
#pragma unroll
    for (int b = 0; b < R::kChunks; b++) {
      sign = wht_block<R::kLanes>(v[part][b], c);
#pragma unroll
      for (int i = 0; i < 8; i++) m[part] = fmaxf(m[part], fabsf(v[part][b][i]));
    }
    m[part] = row_max<R::kLanes>(m[part]);
  }
  // A row whose absmax is zero, or too small for fl(q_max / a) to be finite, is a zero row.
  const bool values = u & 4;
  const float top = values ? m[1] : m[0];
  float mine = top > 0.0f ? __fdiv_rn(R::kQmax, top) : 0.0f;
  if (__builtin_isinf(mine)) mine = 0.0f;
  const float scale = mine != 0.0f ? __fdiv_rn(__fmul_rn(top, R::kNorm), R::kQmax) : 0.0f;
  const float other = dpp_f<0x141>(mine);   // row_half_mirror: a lane of the other four
  if (!in) return;   // no exchange follows
  const float inv[2] = {(values ? other : mine) * sign, (values ? mine : other) * sign};
  if ((u & ~4) == 0) reinterpret_cast<float*>(p.block + 2 * (size_t)page * R::kBytes)[(values ? page : 0) + p.off] = scale;
#pragma unroll
  for (int part = 0; part < 2; part++) {
#pragma unroll
    for (int b = 0; b < R::kChunks; b++) {
      uint32_t lo, hi;
      codes8<BITS>(v[part][b], inv[part], lo, hi);
      const int at = b * (16 * BITS) + c * BITS;   // the chunk's first byte in its row
      if (part == 0) {
        uint8_t* q = p.block + (p.off * R::kBytes + at);
        if constexpr (BITS == 8)
          *reinterpret_cast<u32x2*>(q) = u32x2{lo, hi};
        else
          *reinterpret_cast<uint32_t*>(q) = lo;
      } else {
        uint8_t* q = p.block + (page * R::kBytes + ((p.off >> 2) * R::kBytes + at) * 4 + (p.off & 3));
#pragma unroll
        for (int i = 0; i < BITS; i++) q[4 * i] = static_cast<uint8_t>((i < 4 ? lo : hi) >> (8 * (i & 3)));
      }
    }
  }
}

// The same rows back: x = fl(fl(scale * c) * WHT(codes)), the transform of the codes exact in
// binary32, rounded once to the output type. A slot outside the cache gives a row of zeros.
// STREAM: the outputs go past the caches (kStreamBytes).
template <int D, int BITS, bool STREAM>
__global__ __launch_bounds__(kThreads) void kv_read_kernel(KvCacheArgs a) {
  using R = Row<D, BITS>;
  const int u = threadIdx.x % R::kLanes, c = chunk_of_lane(u);
  const Token t = token_of<kThreads / R::kLanes>(a, R::kLanes);
  const int head = blockIdx.y;
  Place p;
  const bool in = find(a, a.slots[t.first + t.row], head, p);
  const int es = elem_bytes(a.dt), page = 1 << a.lps;
  const float* scales = reinterpret_cast<const float*>(p.block + 2 * (size_t)page * R::kBytes) + p.off;
  const float scale[2] = {scales[0], scales[page]};
  uint32_t w[2][R::kChunks][2];
  u32x4 y[R::kChunks][BITS / 4];
#pragma unroll
  for (int b = 0; b < R::kChunks; b++) {
    const int at = b * (16 * BITS) + c * BITS;
    const uint8_t* q = p.block + (p.off * R::kBytes + at);
    w[0][b][0] = *reinterpret_cast<const uint32_t*>(q);
    if constexpr (BITS == 8) w[0][b][1] = *reinterpret_cast<const uint32_t*>(q + 4);
    // Four tokens' V bytes come with each 4-byte column; the neighbouring rows of the wave load
    // the same 16 bytes, so the lines are read once.
    q = p.block + (page * R::kBytes + ((p.off >> 2) * R::kBytes + at) * 4);
#pragma unroll
    for (int i = 0; i < BITS / 4; i++) y[b][i] = *reinterpret_cast<const u32x4*>(q + 16 * i);
  }
  const uint32_t shift = 8 * (p.off & 3);
#pragma unroll
  for (int b = 0; b < R::kChunks; b++) {
#pragma unroll
    for (int i = 0; i < BITS / 4; i++)
      w[1][b][i] = ((y[b][i][0] >> shift) & 0xFFu) | (((y[b][i][1] >> shift) & 0xFFu) << 8) |
                   (((y[b][i][2] >> shift) & 0xFFu) << 16) | ((y[b][i][3] >> shift) << 24);
  }
#pragma unroll
  for (int part = 0; part < 2; part++) {
    const float s = __fmul_rn(scale[part], R::kNorm);
    uint8_t* x = part ? a.v_out + row_offset(t, head, a.v_token, a.v_head, es)
                      : a.k_out + row_offset(t, head, a.k_token, a.k_head, es);
#pragma unroll
    for (int b = 0; b < R::kChunks; b++) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; i++) {
        if constexpr (BITS == 8)
          v[i] = static_cast<float>(static_cast<int32_t>(w[part][b][i / 4] << (24 - 8 * (i & 3))) >> 24);
        else
          v[i] = static_cast<float>(static_cast<int32_t>(w[part][b][0] << (28 - 4 * i)) >> 28);
      }
      const float sign = wht_block<R::kLanes>(v, c), f = in ? s * sign : 0.0f;
#pragma unroll
      for (int i = 0; i < 8; i++) v[i] = __fmul_rn(f, v[i]);
      if (t.there) store8<STREAM>(x + (b * 128 + c * 8) * es, a.dt, v);
    }
  }
}

// A grid has fewer than 2^32 threads along an axis, 16 of them a token at most: one launch takes
// 2^27 tokens.
constexpr int64_t kLaunchTokens = int64_t(1) << 27;

template <int D, int BITS>
hipError_t launch(const KvCacheArgs& call, bool write, hipStream_t stream) {
  constexpr int kRows = kThreads / Row<D, BITS>::kLanes;
  const int es = call.dt == kF32 ? 4 : 2;
  const bool past = 2 * call.tokens * call.heads * D * es > kStreamBytes;
  hipError_t e = hipSuccess;
  for (int64_t first = 0; e == hipSuccess && first < call.tokens; first += kLaunchTokens) {
    KvCacheArgs a = call;
    a.tokens = call.tokens - first < kLaunchTokens ? call.tokens - first : kLaunchTokens;
    a.slots += first;
    const int64_t k = first * a.k_token * es, v = first * a.v_token * es;
    const dim3 grid(static_cast<unsigned>((a.tokens + kRows - 1) / kRows), static_cast<unsigned>(a.heads));
    if (write) {
      a.k += k;
      a.v += v;
      kv_write_kernel<D, BITS><<<grid, kThreads, 0, stream>>>(a);
    } else {
      a.k_out += k;
      a.v_out += v;
      if (past)
        kv_read_kernel<D, BITS, true><<<grid, kThreads, 0, stream>>>(a);
      else
        kv_read_kernel<D, BITS, false><<<grid, kThreads, 0, stream>>>(a);
    }
    e = hipGetLastError();
  }
  return e;
}

}  // namespace

hipError_t launch_kv_cache(const KvCacheArgs& a, int head_dim, int bits, bool write, hipStream_t stream) {
  if (a.tokens == 0) return hipSuccess;
  switch (head_dim) {
    case 64: return bits == 8 ? launch<64, 8>(a, write, stream) : launch<64, 4>(a, write, stream);
    case 128: return bits == 8 ? launch<128, 8>(a, write, stream) : launch<128, 4>(a, write, stream);
    default: return bits == 8 ? launch<256, 8>(a, write, stream) : launch<256, 4>(a, write, stream);
  }
}

}  // namespace convrot
