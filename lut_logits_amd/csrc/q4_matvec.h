// q4_matvec.h -- what the two kernels of the 4-bit matrix products share (q4_matvec.hip, q4_batch.hip).
#pragma once

#include "rq_internal.h"

namespace rq {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float floatx4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

struct Q4Args {
  const u32x4* codes;        // [RT][KT][64]
  const void* scales;        // [RT][KT][16][128 / group]
  const void* offsets;       // the same, or null
  const uint16_t* levels;    // 16 bf16, or null: code - 8
  const void* x;             // [B][D]
  const float* x2;           // [B][D], or null
  float* y;                  // [B][rows]
  int64_t rows;
  int D, B, x_dtype, scale_dtype;
  int RT, KT;                // blocks of 16 rows, blocks of 128 columns
  int RG;                    // groups of row blocks that a wave takes together
  int src;                   // Q4Source
  int wk;                    // waves of a workgroup that share a row group and split its columns
};

// ---- decoding: the 8 codes of a word as 8 bf16 values, in the order of the columns

// By table: v_perm_b32 takes 4 bytes at a time from an 8-byte table; the two halves of the table are told apart by the code's
// top bit, which v_perm's sign selectors spread over a byte. Once for the levels' low bytes and once for the high ones: 24 vector
// operations for 8 weights.
// As numbers: v_cvt_off_f32_i4 makes a two's-complement nibble t / 16, so a code with its top bit flipped gives
// (code - 8) / 16, exactly: 14 operations. The sums are then a sixteenth (kUnit) until the end.
template <bool LEV>
struct Q4Decoder;

template <>
struct Q4Decoder<true> {
  static constexpr float kUnit = 1.0f;
  uint32_t lo[4], hi[4];   // low and high bytes of the 16 levels
  __device__ __forceinline__ explicit Q4Decoder(const uint16_t* levels) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      lo[i] = hi[i] = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t v = levels[4 * i + j];
        lo[i] |= (v & 0xffu) << (8 * j);
        hi[i] |= (v >> 8) << (8 * j);
      }
    }
  }
  __device__ __forceinline__ bf16x8 operator()(uint32_t w) const {
    const uint32_t se = w & 0x07070707u;          // even nibbles: columns 0..3
    const uint32_t so = (w >> 4) & 0x07070707u;   // odd nibbles: columns 4..7
    // a byte of ones where the code's top bit is set (sign selectors: bytes 1, 3, 5, 7)
    const uint32_t me = __builtin_amdgcn_perm(w << 4, w << 12, 0x0b090a08u);
    const uint32_t mo = __builtin_amdgcn_perm(w, w << 8, 0x0b090a08u);
    auto pick = [](uint32_t m, uint32_t a, uint32_t b) { return (m & a) | (~m & b); };
    const uint32_t el = pick(me, __builtin_amdgcn_perm(lo[3], lo[2], se), __builtin_amdgcn_perm(lo[1], lo[0], se));
    const uint32_t eh = pick(me, __builtin_amdgcn_perm(hi[3], hi[2], se), __builtin_amdgcn_perm(hi[1], hi[0], se));
    const uint32_t ol = pick(mo, __builtin_amdgcn_perm(lo[3], lo[2], so), __builtin_amdgcn_perm(lo[1], lo[0], so));
    const uint32_t oh = pick(mo, __builtin_amdgcn_perm(hi[3], hi[2], so), __builtin_amdgcn_perm(hi[1], hi[0], so));
    u32x4 r;
    r.x = __builtin_amdgcn_perm(eh, el, 0x05010400u);
    r.y = __builtin_amdgcn_perm(eh, el, 0x07030602u);
    r.z = __builtin_amdgcn_perm(oh, ol, 0x05010400u);
    r.w = __builtin_amdgcn_perm(oh, ol, 0x07030602u);
    return __builtin_bit_cast(bf16x8, r);
  }
};

template <>
struct Q4Decoder<false> {
  static constexpr float kUnit = 16.0f;
  __device__ __forceinline__ explicit Q4Decoder(const uint16_t*) {}
  static __device__ __forceinline__ uint32_t two(uint32_t a, uint32_t b) {
    typedef float f2 __attribute__((ext_vector_type(2)));
    typedef __bf16 b2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f2{__builtin_amdgcn_cvt_off_f32_i4((int)a), __builtin_amdgcn_cvt_off_f32_i4((int)b)}, b2));
  }
  __device__ __forceinline__ bf16x8 operator()(uint32_t w) const {
    w ^= 0x88888888u;
    uint32_t v = w >> 4;
    asm("" : "+v"(v));   // the bytes are selected by the conversions themselves; folding the shifts into them would undo that
    auto byte = [](uint32_t u, int i) { return (u >> (8 * i)) & 0xffu; };
    const u32x4 r = {two(byte(w, 0), byte(w, 1)), two(byte(w, 2), byte(w, 3)), two(byte(v, 0), byte(v, 1)), two(byte(v, 2), byte(v, 3))};
    return __builtin_bit_cast(bf16x8, r);
  }
};

// ---- activations

// The bits of v's leading bf16 part (truncated; NaN stays NaN) and what is left (0 where v is not finite).
__device__ __forceinline__ uint32_t cut_bf16(float& v) {
  const uint32_t u = __float_as_uint(v);
  const bool finite = (u & 0x7f800000u) != 0x7f800000u;
  v = finite ? v - __uint_as_float(u & 0xffff0000u) : 0.0f;
  return (u >> 16) | (!finite && (u & 0x007fffffu) ? 0x40u : 0u);
}

// What the activations are made of, and the parts that takes.
enum Q4Source { kQ4F32, kQ4Gelu, kQ4BF16, kQ4F16 };   // (a product of two factors is an fp32 number)
constexpr int q4_parts(int src) { return src == kQ4BF16 ? 1 : src == kQ4F16 ? 2 : 3; }

// N activations of vector b from column k on, loaded (their bits; no use of them, so that the loads of many are under way together) and
// then made numbers, zeros behind the last column. Loads are clamped, not guarded.
template <int SRC, int N>
struct Q4Acts {
  uint32_t x[N], x2[SRC == kQ4Gelu ? N : 1];
  __device__ __forceinline__ void load(const Q4Args& a, int b, int k) {
    const int64_t row = (int64_t)b * a.D;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int64_t i = row + min(k + j, a.D - 1);
      if constexpr (SRC == kQ4F32 || SRC == kQ4Gelu) x[j] = static_cast<const uint32_t*>(a.x)[i];
      else x[j] = static_cast<const uint16_t*>(a.x)[i];
      if constexpr (SRC == kQ4Gelu) x2[j] = reinterpret_cast<const uint32_t*>(a.x2)[i];
    }
  }
  // The same by 16 bytes at a time, whatever their alignment, where all N are there.
  __device__ __forceinline__ void load_wide(const Q4Args& a, int b, int k) {
    typedef unsigned int word4 __attribute__((ext_vector_type(4), aligned(2)));
    if (k + N > a.D) return load(a, b, k);
    const int64_t i = (int64_t)b * a.D + k;
    if constexpr (SRC == kQ4F32 || SRC == kQ4Gelu) {
#pragma unroll
      for (int j = 0; j < N; j += 4) {
        const u32x4 w = *reinterpret_cast<const word4*>(static_cast<const uint32_t*>(a.x) + i + j);
#pragma unroll
        for (int e = 0; e < 4; ++e) x[j + e] = w[e];
        if constexpr (SRC == kQ4Gelu) {
          const u32x4 w2 = *reinterpret_cast<const word4*>(a.x2 + i + j);
#pragma unroll
          for (int e = 0; e < 4; ++e) x2[j + e] = w2[e];
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < N; j += 8) {
        const u32x4 w = *reinterpret_cast<const word4*>(static_cast<const uint16_t*>(a.x) + i + j);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[j + e] = (w[e / 2] >> (16 * (e & 1))) & 0xffffu;
      }
    }
  }
  __device__ __forceinline__ void values(const Q4Args& a, int k, float (&v)[N]) const {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      float f = __uint_as_float(x[j]);
      if constexpr (SRC == kQ4BF16) f = bf16_to_f32(x[j]);
      if constexpr (SRC == kQ4F16) f = (float)__builtin_bit_cast(_Float16, (uint16_t)x[j]);
      if constexpr (SRC == kQ4Gelu) f = gelu_tanh(f) * __uint_as_float(x2[j]);
      v[j] = k + j < a.D ? f : 0.0f;
    }
  }
};

// ---- scales of one row of one block: GPT values of fp32, or of 16 bits, as they lie in memory until they are used

template <int GPT, bool WIDE>
struct Q4Scales {
  static constexpr int N = WIDE ? GPT : (GPT + 1) / 2;
  uint32_t w[N];
  __device__ __forceinline__ void load(const void* p, int64_t row) {   // row: block * 16 + row in it
    if constexpr (!WIDE && GPT == 1) w[0] = static_cast<const uint16_t*>(p)[row];
    else {
#pragma unroll
      for (int i = 0; i < N; ++i) w[i] = static_cast<const uint32_t*>(p)[row * N + i];
    }
  }
  __device__ __forceinline__ float get(int g, int dtype) const {
    if constexpr (WIDE) return __uint_as_float(w[g]);
    const uint32_t h = GPT == 1 ? w[0] : (w[g / 2] >> (16 * (g & 1))) & 0xffffu;
    const float half = (float)__builtin_bit_cast(_Float16, (uint16_t)h), brain = bf16_to_f32(h);
    return dtype == RQ_BF16 ? brain : half;   // selected, not branched: the loops stay whole
  }
};

// Launches of the two kernels. ws: q4_batch_ws_bytes.
size_t q4_batch_ws_bytes(Q4Args a, int gpt);
hipError_t launch_q4_batch(Q4Args a, int gpt, void* ws, hipStream_t stream);

}  // namespace rq
