// q4_matvec.hip -- products with matrices kept in 4 bits with a scale per group of columns.
//
//     y[b][r] = sum_g s[r][g] sum_{k in g} v(c[r][k]) a[b][k]  +  o[r][g] sum_{k in g} a[b][k]
// v(c) = c - 8 or a table of 16 bf16 values; a = x or gelu_tanh(x) * x2.
//
// Bound: HBM (0.5 byte a weight and the scales) while there are few vectors. The
// weights become bf16 in registers and meet a on the matrix cores, which makes
// one vector and sixteen cost the same and leaves the vector unit to the decoding alone.
//
// Exactness: every level is a bf16 value, and fp32 activations are cut into three bf16
// parts (24 bits: 8 + 8 + 8, by truncation, so that nothing overflows), fp16 ones into
// two; every product is then exact and the sums are fp32. The parts are further columns of
// the same matrix-core product: slot PS*b + p holds part p of vector b (PS = 1, 2 or 4), which
// puts all parts of a vector into one lane's accumulators.
//
// Layout of the codes: blocks of 16 rows x 128 columns, 1 KB: lane (i16, kg) of a wave
// loads 16 bytes, the codes of row i16 at columns 32w + 8kg + j (word w = one step of 32
// columns). Column j sits in nibble 2j (j < 4) or 2(j-4)+1: the even nibbles of a word are
// then columns 0..3 and the odd ones 4..7, so that the byte-wise table lookup below yields
// the pairs (0,1), (2,3), (4,5), (6,7) in the operand's order.
//
// Lookup: v_perm_b32 takes 4 bytes at a time from an 8-byte table; two halves of the table,
// selected by the code's top bit (spread over a byte by v_perm's sign selectors), for the low
// and the high bytes of the levels: 24 vector operations for 8 weights.
//
// Work split: a workgroup of 8 waves stages a (its parts) in LDS; WK of its waves share a
// group of T row blocks and split the columns, 8 / WK groups run side by side. Many rows: WK = 1, workgroups
// stay and walk over the rows. Few rows: WK = 8, so that every CU has loads in flight; the waves' sums meet in LDS in wave order
// (no atomics: the same call gives the same bits).
#include "rq_internal.h"

namespace rq {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float floatx4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

constexpr int kQ4Threads = 512;
constexpr int kQ4Waves = kQ4Threads / 64;

struct Q4Args {
  const u32x4* codes;        // [RT][KT][64]
  const void* scales;        // [RT][KT][16][128 / group]
  const void* offsets;       // the same, or null
  const uint16_t* levels;    // 16 bf16, or null: code - 8
  const void* x;             // [B][D]
  const float* x2;           // [B][D], or null
  float* y;                  // [B][rows]
  int64_t rows;
  int D, B, x_dtype, scale_f16;
  int RT, KT;                // blocks of 16 rows, blocks of 128 columns
  int RG;                    // groups of T row blocks
  int parts, ps, bt;         // parts and slots of a vector, vectors of a batch tile
  int wk;                    // waves that share a row group
  int kc;                    // column blocks staged at a time
  int red_at_start;          // one round: the waves' sums take the place of the staged activations
  const uint16_t* xp;        // activations cut into parts beforehand: [B * parts][KT * 128], or null
  const float* xpsum;        // and their group sums: [batch tile][KT * GPT][16 NT]
};

// The 8 codes of a word as 8 bf16 levels. lo/hi: the low and high bytes of the 16 levels.
struct Levels {
  uint32_t lo[4], hi[4];
};
__device__ __forceinline__ bf16x8 decode8(uint32_t w, const Levels& t) {
  const uint32_t se = w & 0x07070707u;          // even nibbles: columns 0..3
  const uint32_t so = (w >> 4) & 0x07070707u;   // odd nibbles: columns 4..7
  // a byte of ones where the code's top bit is set (sign selectors of v_perm: bytes 1, 3, 5, 7)
  const uint32_t me = __builtin_amdgcn_perm(w << 4, w << 12, 0x0b090a08u);
  const uint32_t mo = __builtin_amdgcn_perm(w, w << 8, 0x0b090a08u);
  auto pick = [](uint32_t m, uint32_t a, uint32_t b) { return (m & a) | (~m & b); };
  const uint32_t el = pick(me, __builtin_amdgcn_perm(t.lo[3], t.lo[2], se), __builtin_amdgcn_perm(t.lo[1], t.lo[0], se));
  const uint32_t eh = pick(me, __builtin_amdgcn_perm(t.hi[3], t.hi[2], se), __builtin_amdgcn_perm(t.hi[1], t.hi[0], se));
  const uint32_t ol = pick(mo, __builtin_amdgcn_perm(t.lo[3], t.lo[2], so), __builtin_amdgcn_perm(t.lo[1], t.lo[0], so));
  const uint32_t oh = pick(mo, __builtin_amdgcn_perm(t.hi[3], t.hi[2], so), __builtin_amdgcn_perm(t.hi[1], t.hi[0], so));
  u32x4 r;
  r.x = __builtin_amdgcn_perm(eh, el, 0x05010400u);
  r.y = __builtin_amdgcn_perm(eh, el, 0x07030602u);
  r.z = __builtin_amdgcn_perm(oh, ol, 0x05010400u);
  r.w = __builtin_amdgcn_perm(oh, ol, 0x07030602u);
  return __builtin_bit_cast(bf16x8, r);
}

// The bits of v's leading bf16 part (truncated; NaN stays NaN) and what is left (0 where v is not finite).
__device__ __forceinline__ uint32_t cut_bf16(float& v) {
  const uint32_t u = __float_as_uint(v);
  if ((u & 0x7f800000u) == 0x7f800000u) {
    v = 0.0f;
    return (u >> 16) | ((u & 0x007fffffu) ? 0x40u : 0u);
  }
  v -= __uint_as_float(u & 0xffff0000u);
  return u >> 16;
}

__device__ __forceinline__ float load_act(const Q4Args& a, int64_t b, int k) {
  if (k >= a.D) return 0.0f;
  const int64_t i = b * a.D + k;
  float v;
  if (a.x_dtype == RQ_F32) v = static_cast<const float*>(a.x)[i];
  else if (a.x_dtype == RQ_BF16) v = bf16_to_f32(static_cast<const uint16_t*>(a.x)[i]);
  else v = (float)static_cast<const _Float16*>(a.x)[i];
  return a.x2 ? gelu_tanh(v) * a.x2[i] : v;
}

// Scale words of one row of one block: GPT values of SB bytes.
template <int GPT, int SB>
struct ScaleWords {
  static constexpr int N = GPT * SB / 4 > 0 ? GPT * SB / 4 : 1;
  uint32_t w[N];
  __device__ __forceinline__ void load(const void* p, int64_t row) {   // row: (block * 16 + row in it)
    if constexpr (GPT * SB == 2) w[0] = static_cast<const uint16_t*>(p)[row];
    else {
#pragma unroll
      for (int i = 0; i < N; ++i) w[i] = static_cast<const uint32_t*>(p)[row * N + i];
    }
  }
  __device__ __forceinline__ float get(int g, int f16) const {
    if constexpr (SB == 4) return __uint_as_float(w[g]);
    const uint32_t h = (w[g >> 1] >> (16 * (g & 1))) & 0xffffu;
    if (f16) return (float)__builtin_bit_cast(_Float16, (uint16_t)h);
    return bf16_to_f32(h);
  }
};

template <int NT, int T, int GPT, int SB, bool OFF>
__global__ __launch_bounds__(kQ4Threads) __attribute__((amdgpu_waves_per_eu(2, 8))) void q4_matvec_kernel(Q4Args a) {
  constexpr int U = T == 1 ? 3 : 1;    // column blocks whose loads are issued together
  constexpr int STEPS = 4 / GPT;       // steps of 32 columns in a group
  extern __shared__ __align__(16) unsigned char smem[];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);   // (uniform)
  const int i16 = lane & 15, kg = lane >> 4;
  const int wk = a.wk, wr = kQ4Waves / wk;
  const int kpart = wave % wk, rpart = wave / wk;
  const int b0 = blockIdx.y * a.bt;
  const int nb = min(a.bt, a.B - b0);                       // vectors of this batch tile
  const int staged = nb * a.parts;
  const int ld = a.kc * 128 + 8;                            // row stride of a part: 16 bytes past a whole bank turn
  uint16_t* xs = reinterpret_cast<uint16_t*>(smem);         // [staged][ld]
  float* xsum = reinterpret_cast<float*>(smem + (((size_t)min(a.bt, a.B) * a.parts * ld * 2 + 15) & ~(size_t)15));   // [kc * GPT][16 NT]
  float* red = a.red_at_start ? reinterpret_cast<float*>(smem) : xsum + (OFF ? a.kc * GPT * 16 * NT : 0);   // [wr][wk - 1][T * NT * 4][64]

  Levels lv;
  if (a.levels) {   // (uniform)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t l = 0, h = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t v = a.levels[4 * i + j];
        l |= (v & 0xffu) << (8 * j);
        h |= (v >> 8) << (8 * j);
      }
      lv.lo[i] = l;
      lv.hi[i] = h;
    }
  } else {          // -8 .. 7
    lv = Levels{{0xa0c0e000u, 0x80004080u, 0x40008000u, 0xe0c0a080u}, {0xc0c0c0c1u, 0xbfc0c0c0u, 0x40403f00u, 0x40404040u}};
  }

  // LDS row of this lane's slot in each column tile (slots without a part repeat one: their sums are not used)
  int xrow[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int slot = 16 * n + i16;
    const int b = min(slot / a.ps, nb - 1), p = min(slot % a.ps, a.parts - 1);
    xrow[n] = (b * a.parts + p) * ld + 8 * kg;
  }

  struct Stage {
    u32x4 c[U][T];
    ScaleWords<GPT, SB> s[U][T], o[OFF ? U : 1][OFF ? T : 1];
  };
  const int nchunks = (a.KT + a.kc - 1) / a.kc;
  // loads of U column blocks from kt on (stride wk), clamped to the matrix
  auto load = [&](Stage& st, int rg, int kt) {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int t = 0; t < T; ++t) {
        const int64_t blk = (int64_t)min(rg * T + t, a.RT - 1) * a.KT + min(kt + u * wk, a.KT - 1);
        st.c[u][t] = a.codes[blk * 64 + lane];
        st.s[u][t].load(a.scales, blk * 16 + i16);
        if constexpr (OFF) st.o[u][t].load(a.offsets, blk * 16 + i16);
      }
  };
  floatx4 tot[T][NT];
  auto compute = [&](const Stage& st, int kt, int k_lo, int k_hi) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (kt + u * wk >= k_hi) break;   // (uniform)
      const int col = (kt + u * wk - k_lo) * 128;
#pragma unroll
      for (int g = 0; g < GPT; ++g) {
        floatx4 acc[T][NT];
#pragma unroll
        for (int w = g * STEPS; w < (g + 1) * STEPS; ++w) {
          bf16x8 xf[NT];
#pragma unroll
          for (int n = 0; n < NT; ++n) xf[n] = *reinterpret_cast<const bf16x8*>(xs + xrow[n] + col + 32 * w);
#pragma unroll
          for (int t = 0; t < T; ++t) {
            const bf16x8 wv = decode8(st.c[u][t][w], lv);
#pragma unroll
            for (int n = 0; n < NT; ++n)
              acc[t][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xf[n], wv, w == g * STEPS ? floatx4{0.f, 0.f, 0.f, 0.f} : acc[t][n], 0, 0, 0);
          }
        }
#pragma unroll
        for (int t = 0; t < T; ++t) {
          const float s = st.s[u][t].get(g, a.scale_f16);
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) tot[t][n][e] = fmaf(s, acc[t][n][e], tot[t][n][e]);
        }
        if constexpr (OFF) {
          floatx4 xv[NT];
          const float* xp = xsum + (col / 128 * GPT + g) * 16 * NT + 4 * kg;
#pragma unroll
          for (int n = 0; n < NT; ++n) xv[n] = *reinterpret_cast<const floatx4*>(xp + 16 * n);
#pragma unroll
          for (int t = 0; t < T; ++t) {
            const float o = st.o[u][t].get(g, a.scale_f16);
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int e = 0; e < 4; ++e) tot[t][n][e] = fmaf(o, xv[n][e], tot[t][n][e]);
          }
        }
      }
    }
  };
  // activations of column blocks [k_lo, k_hi) as bf16 parts, two columns a thread and step; group sums of the parts
  auto stage = [&](int k_lo, int k_hi) {
    if (a.xp) {   // (uniform) cut beforehand: 16-byte copies
      const int n16 = (k_hi - k_lo) * 16;
      const uint16_t* src = a.xp + ((size_t)b0 * a.parts * a.KT + k_lo) * 128;
#pragma unroll 4
      for (int i = tid; i < staged * n16; i += kQ4Threads) {
        const int r = i / n16, j = i - r * n16;
        *reinterpret_cast<u32x4*>(xs + r * ld + 8 * j) = *reinterpret_cast<const u32x4*>(src + (size_t)r * a.KT * 128 + 8 * j);
      }
      if constexpr (OFF) {
        const int n = (k_hi - k_lo) * GPT * 16 * NT;
        const float* q = a.xpsum + ((size_t)blockIdx.y * a.KT + k_lo) * GPT * 16 * NT;
        for (int i = tid; i < n; i += kQ4Threads) xsum[i] = q[i];
      }
      return;
    }
    const int pairs = (k_hi - k_lo) * 64;
    for (int b = 0; b < nb; ++b) {
#pragma unroll 4
      for (int i = tid; i < pairs; i += kQ4Threads) {
        float v0 = load_act(a, b0 + b, k_lo * 128 + 2 * i), v1 = load_act(a, b0 + b, k_lo * 128 + 2 * i + 1);
        for (int p = 0; p < a.parts; ++p) {   // (uniform)
          const uint32_t lo = cut_bf16(v0), hi = cut_bf16(v1);
          *reinterpret_cast<uint32_t*>(xs + (b * a.parts + p) * ld + 2 * i) = lo | (hi << 16);
        }
      }
    }
    if constexpr (OFF) {
      __syncthreads();
      constexpr int GC = 128 / GPT;   // columns of a group
      const int groups = (k_hi - k_lo) * GPT;
      for (int i = tid; i < groups * 16 * NT; i += kQ4Threads) {
        const int slot = i % (16 * NT), g = i / (16 * NT);
        const int b = slot / a.ps, p = slot % a.ps;
        float s = 0.0f;
        if (b < nb && p < a.parts) {
          const uint16_t* q = xs + (b * a.parts + p) * ld + g * GC;
          for (int j = 0; j < GC; j += 2) {
            const uint32_t two = *reinterpret_cast<const uint32_t*>(q + j);
            s += __uint_as_float(two << 16) + __uint_as_float(two & 0xffff0000u);
          }
        }
        xsum[i] = s;
      }
    }
  };

  const int stride = (int)gridDim.x * wr;
  const int rounds = (a.RG + stride - 1) / stride;   // the same for every workgroup: barriers inside
  int rg = blockIdx.x * wr + rpart;
  Stage s0, s1;
  load(s0, rg, kpart);
  for (int round = 0; round < rounds; ++round, rg += stride) {
#pragma unroll
    for (int t = 0; t < T; ++t)
#pragma unroll
      for (int n = 0; n < NT; ++n) tot[t][n] = floatx4{0.f, 0.f, 0.f, 0.f};
    for (int c = 0; c < nchunks; ++c) {
      const int k_lo = c * a.kc, k_hi = min(a.KT, k_lo + a.kc);
      if (nchunks > 1 || round == 0) {   // (uniform)
        if (c > 0 || round > 0) __syncthreads();   // the last chunk has been read
        stage(k_lo, k_hi);
        __syncthreads();
      }
      // this wave's blocks: k_lo + kpart + i * wk; the stage behind a chunk's or a row group's last is the next one's first
      for (int kt = k_lo + kpart; kt < k_hi; kt += U * wk) {
        const bool more = kt + U * wk < k_hi;
        const bool last = c + 1 == nchunks;
        load(s1, more || !last ? rg : rg + stride, more ? kt + U * wk : (last ? kpart : k_hi + kpart));
        compute(s0, kt, k_lo, k_hi);
        s0 = s1;
      }
    }
    if (wk > 1 && a.red_at_start) __syncthreads();   // (uniform) the activations have been read
    if (wk > 1) {   // (uniform) sums of the waves of a row group, in wave order
      float* r = red + (size_t)rpart * (wk - 1) * (T * NT * 4) * 64 + lane;
      if (kpart > 0) {
#pragma unroll
        for (int t = 0; t < T; ++t)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) r[(((size_t)(kpart - 1) * T + t) * NT + n) * 256 + e * 64] = tot[t][n][e];
      }
      __syncthreads();
      if (kpart == 0) {
        for (int p = 0; p + 1 < wk; ++p)
#pragma unroll
          for (int t = 0; t < T; ++t)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int e = 0; e < 4; ++e) tot[t][n][e] += r[(((size_t)p * T + t) * NT + n) * 256 + e * 64];
      }
      if (round + 1 < rounds) __syncthreads();   // read before the next round writes
    }
    if (kpart == 0 && rg < a.RG) {
#pragma unroll
      for (int t = 0; t < T; ++t) {
        const int64_t r = ((int64_t)rg * T + t) * 16 + i16;
        if (r >= a.rows) continue;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const floatx4 v = tot[t][n];
          auto put = [&](int b, float f) {
            if (b < nb) a.y[(int64_t)(b0 + b) * a.rows + r] = f;
          };
          if (a.ps == 4) put(4 * n + kg, v[0] + (v[1] + v[2]));   // (uniform)
          else if (a.ps == 2) {
            put(8 * n + 2 * kg, v[0] + v[1]);
            put(8 * n + 2 * kg + 1, v[2] + v[3]);
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) put(16 * n + 4 * kg + e, v[e]);
          }
        }
      }
    }
  }
}

// The parts of 8 columns of one vector a thread (and of both factors' product), and the sums of the parts
// over each group of columns: a group is 4, 8 or 16 neighbouring threads.
__global__ __launch_bounds__(256) void q4_cut_kernel(Q4Args a, int gpt, int nt, uint16_t* __restrict__ xp, float* __restrict__ xpsum) {
  const int n8 = a.KT * 16;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const bool in = i < (int64_t)a.B * n8;   // whole blocks of 16 threads (n8 is a multiple of 16)
  const int b = in ? (int)(i / n8) : 0, c = in ? (int)(i - (int64_t)b * n8) : 0;
  float v[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = in ? load_act(a, b, c * 8 + j) : 0.0f;
  for (int p = 0; p < a.parts; ++p) {
    uint32_t u[8];
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      u[j] = cut_bf16(v[j]);
      s += __uint_as_float(u[j] << 16);
    }
    if (in)
      *reinterpret_cast<u32x4*>(xp + (((int64_t)b * a.parts + p) * n8 + c) * 8) =
          u32x4{u[0] | (u[1] << 16), u[2] | (u[3] << 16), u[4] | (u[5] << 16), u[6] | (u[7] << 16)};
    if (!xpsum) continue;
    const int threads = 16 / gpt;
    for (int m = 1; m < threads; m <<= 1) s += __shfl_xor(s, m, 64);
    if (in && c % threads == 0) {
      const int tile = b / a.bt, slot = (b - tile * a.bt) * a.ps + p;
      xpsum[((int64_t)tile * a.KT * gpt + c / threads) * 16 * nt + slot] = s;
    }
  }
}

// One thread for the 8 codes of a word of the block layout; columns past D and rows past the matrix are code 0.
__global__ void pack_q4_codes_kernel(const uint8_t* __restrict__ src, int64_t rows, int D, int KT, uint32_t* __restrict__ dst,
                                     int64_t words) {
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= words) return;
  const int64_t blk = i >> 8;
  const int in = (int)(i & 255), w = in & 3, i16 = (in >> 2) & 15, kg = in >> 6;
  const int64_t r = (blk / KT) * 16 + i16;
  const int k0 = (int)(blk % KT) * 128 + 32 * w + 8 * kg;
  uint32_t out = 0;
  if (r < rows) {
    const int64_t row = r * ((D + 1) / 2);
    for (int j = 0; j < 8; ++j) {
      const int k = k0 + j;
      if (k >= D) break;
      const uint32_t byte = src[row + k / 2];
      const uint32_t code = (k & 1) ? byte >> 4 : byte & 15u;
      out |= code << (4 * (j < 4 ? 2 * j : 2 * (j - 4) + 1));
    }
  }
  dst[i] = out;
}

template <typename E>
__global__ void pack_q4_scales_kernel(const E* __restrict__ src, int64_t rows, int G, int KT, int gpt, E* __restrict__ dst,
                                      int64_t n) {
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= n) return;
  const int g = (int)(i % gpt);
  const int64_t row = i / gpt;   // block * 16 + row in it
  const int64_t blk = row / 16;
  const int64_t r = (blk / KT) * 16 + row % 16;
  const int64_t group = (blk % KT) * gpt + g;
  dst[i] = (r < rows && group < G) ? src[r * G + group] : (E)0;
}

struct Q4Plan {
  int NT, T;
  size_t lds, xp, total;   // LDS; workspace: bytes of the parts, and with their group sums (0: cut while staging)
  unsigned gx, gy;
};

size_t staged_bytes(const Q4Args& a, int NT, int gpt, bool off) {
  const size_t xs = ((size_t)std::min(a.bt, a.B) * a.parts * (a.kc * 128 + 8) * 2 + 15) & ~(size_t)15;
  return xs + (off ? (size_t)a.kc * gpt * 16 * NT * 4 : 0);
}

// Activation parts by type (an activation made of two factors is an fp32 number whatever x is).
int q4_parts(int x_dtype, bool x2) { return x2 || x_dtype == RQ_F32 ? 3 : x_dtype == RQ_F16 ? 2 : 1; }

Q4Plan plan_q4(Q4Args& a, int x_dtype, bool x2, int gpt, bool off) {
  Q4Plan p;
  a.parts = q4_parts(x_dtype, x2);
  a.ps = a.parts == 3 ? 4 : a.parts;
  const int slots = a.B * a.ps;   // B <= 65535, ps <= 4
  p.NT = slots <= 16 ? 1 : slots <= 32 ? 2 : slots <= 64 ? 4 : 8;
  p.T = p.NT == 1 ? 1 : 2;
  a.bt = 16 * p.NT / a.ps;
  a.RG = (a.RT + p.T - 1) / p.T;
  // waves of a row group: enough that every CU holds about 16 waves, with the column blocks to feed them
  a.wk = 1;
  while (a.wk < kQ4Waves && a.wk * 2 <= a.KT && (int64_t)a.RG * a.wk < 16 * kCUs) a.wk *= 2;
  const int wr = kQ4Waves / a.wk;
  const size_t red = a.wk > 1 ? (size_t)wr * (a.wk - 1) * p.T * p.NT * 1024 : 0;
  int64_t wgs = (a.RG + wr - 1) / wr;
  a.kc = a.KT;
  const size_t whole = staged_bytes(a, p.NT, gpt, off);
  const size_t half = (size_t)kLdsBudget / 2;
  int64_t stay = kCUs * (whole + red <= half ? 2 : 1);
  if (whole + (wgs <= stay ? 0 : red) <= (size_t)kLdsBudget) {
    // staged once, by workgroups that stay where there are more row groups than fit the chip at once
    a.red_at_start = wgs <= stay;
    p.lds = a.red_at_start ? std::max(whole, red) : whole + red;
    wgs = std::min(wgs, stay);
  } else {
    // in chunks, of whole rounds of the waves, that leave room for two workgroups a CU; one round
    while (a.kc > 1 && staged_bytes(a, p.NT, gpt, off) > half) --a.kc;
    if (a.kc > a.wk) a.kc = a.kc / a.wk * a.wk;
    a.red_at_start = 1;
    p.lds = std::max(staged_bytes(a, p.NT, gpt, off), red);
  }
  p.gx = (unsigned)wgs;
  p.gy = (unsigned)((a.B + a.bt - 1) / a.bt);
  p.xp = p.total = 0;
  if (a.B > 4 || (x2 && a.B > 1)) {
    p.xp = (size_t)a.B * a.parts * a.KT * 256;
    p.total = p.xp + (off ? (size_t)p.gy * a.KT * gpt * 16 * p.NT * 4 : 0);
  }
  return p;
}

template <int NT, int T, int GPT, int SB, bool OFF>
hipError_t launch_one(const Q4Args& a, const Q4Plan& p, hipStream_t stream) {
  auto kern = q4_matvec_kernel<NT, T, GPT, SB, OFF>;
  if (p.lds > 64 * 1024) {
    hipError_t e = hipFuncSetAttribute((const void*)kern, hipFuncAttributeMaxDynamicSharedMemorySize, (int)p.lds);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(kern, dim3(p.gx, p.gy), dim3(kQ4Threads), p.lds, stream, a);
  return hipGetLastError();
}

template <int GPT, int SB, bool OFF>
hipError_t launch_nt(const Q4Args& a, const Q4Plan& p, hipStream_t stream) {
  switch (p.NT) {
    case 1: return launch_one<1, 1, GPT, SB, OFF>(a, p, stream);
    case 2: return launch_one<2, 2, GPT, SB, OFF>(a, p, stream);
    case 4: return launch_one<4, 2, GPT, SB, OFF>(a, p, stream);
    default: return launch_one<8, 2, GPT, SB, OFF>(a, p, stream);
  }
}

template <int GPT>
hipError_t launch_gpt(const Q4Args& a, const Q4Plan& p, int sb, hipStream_t stream) {
  if (sb == 4) return a.offsets ? launch_nt<GPT, 4, true>(a, p, stream) : launch_nt<GPT, 4, false>(a, p, stream);
  return a.offsets ? launch_nt<GPT, 2, true>(a, p, stream) : launch_nt<GPT, 2, false>(a, p, stream);
}

}  // namespace

static int64_t q4_blocks(int64_t rows, int D) { return ((rows + 15) / 16) * (int64_t)((D + 127) / 128); }
size_t q4_codes_bytes(int64_t rows, int D) { return (size_t)q4_blocks(rows, D) * 1024; }
size_t q4_scale_count(int64_t rows, int D, int group) { return (size_t)q4_blocks(rows, D) * 16 * (128 / group); }

hipError_t launch_pack_q4_codes(const uint8_t* src, int64_t rows, int D, void* dst, hipStream_t stream) {
  const int64_t words = q4_blocks(rows, D) * 256;
  hipLaunchKernelGGL(pack_q4_codes_kernel, dim3((unsigned)((words + 255) / 256)), dim3(256), 0, stream, src, rows, D,
                     (D + 127) / 128, static_cast<uint32_t*>(dst), words);
  return hipGetLastError();
}

hipError_t launch_pack_q4_scales(const void* src, int64_t rows, int D, int group, int elem_bytes, void* dst,
                                 hipStream_t stream) {
  const int64_t n = (int64_t)q4_scale_count(rows, D, group);
  const int G = (D + group - 1) / group, KT = (D + 127) / 128, gpt = 128 / group;
  const dim3 grid((unsigned)((n + 255) / 256));
  if (elem_bytes == 4)
    hipLaunchKernelGGL(pack_q4_scales_kernel<uint32_t>, grid, dim3(256), 0, stream, static_cast<const uint32_t*>(src), rows, G,
                       KT, gpt, static_cast<uint32_t*>(dst), n);
  else
    hipLaunchKernelGGL(pack_q4_scales_kernel<uint16_t>, grid, dim3(256), 0, stream, static_cast<const uint16_t*>(src), rows, G,
                       KT, gpt, static_cast<uint16_t*>(dst), n);
  return hipGetLastError();
}

static Q4Args q4_args(const rq_q4_matrix* W, int B) {
  Q4Args a = {};
  a.codes = static_cast<const u32x4*>(W->codes);
  a.scales = W->scales;
  a.offsets = W->offsets;
  a.levels = W->levels;
  a.rows = W->rows;
  a.D = W->D;
  a.B = B;
  a.scale_f16 = W->scale_dtype == RQ_F16;
  a.RT = (int)((W->rows + 15) / 16);
  a.KT = (W->D + 127) / 128;
  return a;
}

size_t q4_matvec_ws_bytes(const rq_q4_matrix* W, int x_dtype, bool x2, int B) {
  Q4Args a = q4_args(W, B);
  return plan_q4(a, x_dtype, x2, 128 / W->group, W->offsets != nullptr).total;
}

hipError_t launch_q4_matvec(const rq_q4_matrix* W, const void* x, int x_dtype, const float* x2, int B, float* y, void* ws,
                            hipStream_t stream) {
  Q4Args a = q4_args(W, B);
  const int gpt = 128 / W->group, sb = W->scale_dtype == RQ_F32 ? 4 : 2;
  const Q4Plan p = plan_q4(a, x_dtype, x2 != nullptr, gpt, W->offsets != nullptr);
  a.x = x;
  a.x_dtype = x_dtype;
  a.x2 = x2;
  a.y = y;
  if (p.total) {
    uint16_t* xp = static_cast<uint16_t*>(ws);
    float* sums = W->offsets ? reinterpret_cast<float*>(static_cast<char*>(ws) + p.xp) : nullptr;
    const int64_t n = (int64_t)B * a.KT * 16;
    hipLaunchKernelGGL(q4_cut_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, stream, a, gpt, p.NT, xp, sums);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    a.xp = xp;
    a.xpsum = sums;
  }
  if (gpt == 4) return launch_gpt<4>(a, p, sb, stream);
  if (gpt == 2) return launch_gpt<2>(a, p, sb, stream);
  return launch_gpt<1>(a, p, sb, stream);
}

}  // namespace rq
