// rope.hip -- rotary positions, alone or together with the write of keys and values into the paged cache.
//
// Pair i of a head turns by the angle a = position * freqs[i]:
//     (x1, x2) -> m * (x1 cos a - x2 sin a, x2 cos a + x1 sin a)
// with pairs (i, i + rot/2) in the half layout and (2i, 2i + 1) in the interleaved one; the values from rot on
// pass unchanged. The inverse turns by -a, which is also the gradient (the rotation is orthogonal up to m).
//
// Angles: position * freqs[i] in 64 bits, as turns, reduced to half a turn before the fp32 sine and cosine:
// at position 10^6 a 32-bit product would already be off by a tenth of a radian.
//
// Bound: HBM; every value is read and written once. A workgroup takes up to 16
// tokens, computes their cosines and sines once into LDS for all heads, then walks over (token, head, 8 values)
// with 16-byte accesses. The cache keeps V transposed inside a page ([head size][page size], the layout that attention's matrix product
// reads without a transpose): a tile of 16 positions is aligned to 16, so it lies in one page, and a thread
// gathers one column's 16 values (reads are coalesced over the columns) into 16-byte stores.
// The grid's second axis splits a tile's items where there are few tiles.
#include "rq_internal.h"

namespace rq {
namespace {

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

constexpr int kRopeThreads = 256;
constexpr int kRopeTile = 16;   // positions of a tile; page sizes are multiples of it

struct RopeArgs {
  const void *q, *k, *v;          // [tokens][heads][size], token strides below; k, v only with a cache
  int64_t q_stride, k_stride, v_stride, o_stride;
  int in_dtype, out_dtype;
  int tokens, heads, kv_heads, size, half;
  int inverse;
  const int32_t* positions;       // [tokens], or null with a cache: the place in it
  const double* freqs;            // [half]
  float mscale;
  void* out;
  rq_seq_batch batch;
  rq_kv_cache cache;
  int32_t* bad;
};

__device__ __forceinline__ float load1(const void* p, int dtype, int64_t i) {
  if (dtype == RQ_F32) return static_cast<const float*>(p)[i];
  if (dtype == RQ_BF16) return bf16_to_f32(static_cast<const uint16_t*>(p)[i]);
  return (float)static_cast<const _Float16*>(p)[i];
}
__device__ __forceinline__ uint16_t pack1(float v, int dtype) {
  return dtype == RQ_BF16 ? f32_to_bf16(v) : __builtin_bit_cast(uint16_t, (_Float16)v);
}
__device__ __forceinline__ void store1(void* p, int dtype, int64_t i, float v) {
  if (dtype == RQ_F32) static_cast<float*>(p)[i] = v;
  else static_cast<uint16_t*>(p)[i] = pack1(v, dtype);
}
template <int VEC>
__device__ __forceinline__ void load_vec(const void* p, int dtype, int64_t i, float (&v)[VEC]) {
  if constexpr (VEC == 1) {
    v[0] = load1(p, dtype, i);
  } else if (dtype == RQ_F32) {
    const u32x4* s = reinterpret_cast<const u32x4*>(static_cast<const float*>(p) + i);
    const u32x4 a = s[0], b = s[1];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[j] = __uint_as_float(a[j]);
      v[4 + j] = __uint_as_float(b[j]);
    }
  } else {
    const u32x4 a = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(p) + i);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t lo = a[j] & 0xffffu, hi = a[j] >> 16;
      v[2 * j] = dtype == RQ_BF16 ? bf16_to_f32(lo) : (float)__builtin_bit_cast(_Float16, (uint16_t)lo);
      v[2 * j + 1] = dtype == RQ_BF16 ? bf16_to_f32(hi) : (float)__builtin_bit_cast(_Float16, (uint16_t)hi);
    }
  }
}
template <int VEC>
__device__ __forceinline__ void store_vec(void* p, int dtype, int64_t i, const float (&v)[VEC]) {
  if constexpr (VEC == 1) {
    store1(p, dtype, i, v[0]);
  } else if (dtype == RQ_F32) {
    u32x4* d = reinterpret_cast<u32x4*>(static_cast<float*>(p) + i);
    d[0] = u32x4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])};
    d[1] = u32x4{__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7])};
  } else {
    u32x4 a;
#pragma unroll
    for (int j = 0; j < 4; ++j) a[j] = pack1(v[2 * j], dtype) | ((uint32_t)pack1(v[2 * j + 1], dtype) << 16);
    *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(p) + i) = a;
  }
}

// VEC values a thread and access: 8 (16-byte accesses of 16-bit types) or 1.
template <int VEC, bool INTERLEAVED>
__global__ __launch_bounds__(kRopeThreads) void rope_kernel(RopeArgs a, int append) {
  extern __shared__ __align__(16) float2 turn[];   // [tokens of the tile][half]
  __shared__ int tile_pos[kRopeTile];              // place in the sequence
  const int tid = threadIdx.x;
  // this tile's tokens: [t0, t0 + n), all of one sequence, in one page, with a cache
  int t0, n, place0 = 0, page = -1;
  if (append) {   // (uniform)
    const SeqTile st = find_tile(a.batch, kRopeTile, 2, (int)blockIdx.x);
    if (st.seq < 0) return;
    const int new0 = st.len - st.n;                                       // place of the sequence's first new token (may be < 0)
    const int lo = (floor_div(new0, kRopeTile) + st.tile) * kRopeTile;    // the tile's places: lo .. lo + 15
    const int first = max(lo, new0), end = min(lo + kRopeTile, st.len);
    if (first >= end) return;
    t0 = st.t0 + (first - new0);
    n = end - first;
    place0 = first;
    const int pi = lo >= 0 ? lo / a.cache.page_size : -1;
    if (pi >= 0 && pi < a.batch.max_pages) page = a.batch.table[(int64_t)st.seq * a.batch.max_pages + pi];
    if ((unsigned)page >= (unsigned)a.cache.pages) {
      page = -1;
      if (a.bad && tid == 0 && blockIdx.y == 0) atomicAdd(a.bad, n);
    }
  } else {
    t0 = (int)blockIdx.x * kRopeTile;
    n = min(kRopeTile, a.tokens - t0);
  }
  if (tid < n) tile_pos[tid] = a.positions ? a.positions[t0 + tid] : place0 + tid;
  __syncthreads();
  for (int i = tid; i < n * a.half; i += kRopeThreads) {
    const int t = i / a.half;
    double turns = (double)tile_pos[t] * (a.freqs[i - t * a.half] * 0.15915494309189533577);   // 1 / (2 pi)
    turns -= rint(turns);
    float s, c;
    sincospif((float)(2.0 * turns), &s, &c);
    turn[i] = make_float2(c * a.mscale, (a.inverse ? -s : s) * a.mscale);
  }
  __syncthreads();

  const int rot = 2 * a.half;
  const int turned = INTERLEAVED ? rot / (VEC == 1 ? 2 : VEC) : a.half / VEC;   // rotated items of a head
  const int per_head = turned + (a.size - rot) / VEC;                           // and those that pass
  const int hk = append ? a.kv_heads : 0;
  const int items = n * (a.heads + hk) * per_head;
  const int vitems = hk * a.size;                                               // columns of V
  const int share = (items + vitems + (int)gridDim.y - 1) / (int)gridDim.y;
  const int it0 = (int)blockIdx.y * share, it1 = min(items + vitems, it0 + share);
  const int place_in_page = page >= 0 ? place0 % a.cache.page_size : 0;
  for (int it = it0 + tid; it < it1; it += kRopeThreads) {
    if (it < items) {
      const int c = it % per_head, th = it / per_head;
      const int h = th % (a.heads + hk), t = th / (a.heads + hk);
      const bool is_k = h >= a.heads;
      const void* src = is_k ? a.k : a.q;
      const int64_t from = (int64_t)(t0 + t) * (is_k ? a.k_stride : a.q_stride) + (int64_t)(is_k ? h - a.heads : h) * a.size;
      void* dst = is_k ? a.cache.k : a.out;
      int64_t to = (int64_t)(t0 + t) * a.o_stride + (int64_t)h * a.size;
      if (is_k) {
        if (page < 0) continue;
        to = (((int64_t)page * hk + (h - a.heads)) * a.cache.page_size + place_in_page + t) * a.size;
      }
      const float2* tr = turn + t * a.half;
      if (c >= turned) {
        const int i = rot + (c - turned) * VEC;
        float x[VEC];
        load_vec<VEC>(src, a.in_dtype, from + i, x);
        store_vec<VEC>(dst, a.out_dtype, to + i, x);
      } else if constexpr (!INTERLEAVED) {
        const int i = c * VEC;
        float x1[VEC], x2[VEC], y1[VEC], y2[VEC];
        load_vec<VEC>(src, a.in_dtype, from + i, x1);
        load_vec<VEC>(src, a.in_dtype, from + a.half + i, x2);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const float2 cs = tr[i + j];
          y1[j] = x1[j] * cs.x - x2[j] * cs.y;
          y2[j] = x2[j] * cs.x + x1[j] * cs.y;
        }
        store_vec<VEC>(dst, a.out_dtype, to + i, y1);
        store_vec<VEC>(dst, a.out_dtype, to + a.half + i, y2);
      } else if constexpr (VEC == 1) {
        const float x1 = load1(src, a.in_dtype, from + 2 * c), x2 = load1(src, a.in_dtype, from + 2 * c + 1);
        const float2 cs = tr[c];
        store1(dst, a.out_dtype, to + 2 * c, x1 * cs.x - x2 * cs.y);
        store1(dst, a.out_dtype, to + 2 * c + 1, x2 * cs.x + x1 * cs.y);
      } else {
        const int i = c * VEC;
        float x[VEC], y[VEC];
        load_vec<VEC>(src, a.in_dtype, from + i, x);
#pragma unroll
        for (int j = 0; j < VEC; j += 2) {
          const float2 cs = tr[(i + j) / 2];
          y[j] = x[j] * cs.x - x[j + 1] * cs.y;
          y[j + 1] = x[j + 1] * cs.x + x[j] * cs.y;
        }
        store_vec<VEC>(dst, a.out_dtype, to + i, y);
      }
    } else if (page >= 0) {
      const int d = it - items;   // column of V: (head, place in the head)
      const int h = d / a.size, e = d - h * a.size;
      const int64_t from = (int64_t)t0 * a.v_stride + d;
      uint16_t* dst = static_cast<uint16_t*>(a.cache.v) + (((int64_t)page * hk + h) * a.size + e) * a.cache.page_size + place_in_page;
      if (n == kRopeTile) {
        uint32_t w[kRopeTile / 2];
#pragma unroll
        for (int t = 0; t < kRopeTile; t += 2)
          w[t / 2] = pack1(load1(a.v, a.in_dtype, from + t * a.v_stride), a.out_dtype) |
                     ((uint32_t)pack1(load1(a.v, a.in_dtype, from + (t + 1) * a.v_stride), a.out_dtype) << 16);
        reinterpret_cast<u32x4*>(dst)[0] = u32x4{w[0], w[1], w[2], w[3]};
        reinterpret_cast<u32x4*>(dst)[1] = u32x4{w[4], w[5], w[6], w[7]};
      } else {
        for (int t = 0; t < n; ++t) dst[t] = pack1(load1(a.v, a.in_dtype, from + t * a.v_stride), a.out_dtype);
      }
    }
  }
}

bool aligned16(const void* p) { return (uintptr_t)p % 16 == 0; }

hipError_t launch(const RopeArgs& a, bool interleaved, int append, int tiles, hipStream_t stream) {
  const int ib = a.in_dtype == RQ_F32 ? 4 : 2, ob = a.out_dtype == RQ_F32 ? 4 : 2;
  // 16-byte accesses where every row and every half begins at 16 bytes and holds whole 8s
  bool vec = a.size % 8 == 0 && (interleaved ? 2 * a.half : a.half) % 8 == 0 && aligned16(a.q) && aligned16(a.out) &&
             a.q_stride * ib % 16 == 0 && a.o_stride * ob % 16 == 0;
  if (append) vec = vec && aligned16(a.k) && a.k_stride * ib % 16 == 0;
  // enough workgroups for the chip where there are few tiles: at least 256 items each
  const int64_t items = (int64_t)(a.heads + (append ? 2 * a.kv_heads : 0)) * a.size / (vec ? 8 : 1) *
                        std::min(kRopeTile, std::max(1, a.tokens / std::max(1, append ? a.batch.seqs : 1)));
  const int64_t want = (4 * kCUs + tiles - 1) / tiles;
  const int parts = (int)std::max<int64_t>(1, std::min(want, items / kRopeThreads));
  const size_t lds = (size_t)kRopeTile * a.half * sizeof(float2);
  const dim3 grid((unsigned)tiles, (unsigned)parts), block(kRopeThreads);
  if (interleaved) {
    if (vec) hipLaunchKernelGGL((rope_kernel<8, true>), grid, block, lds, stream, a, append);
    else hipLaunchKernelGGL((rope_kernel<1, true>), grid, block, lds, stream, a, append);
  } else {
    if (vec) hipLaunchKernelGGL((rope_kernel<8, false>), grid, block, lds, stream, a, append);
    else hipLaunchKernelGGL((rope_kernel<1, false>), grid, block, lds, stream, a, append);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_rope(const void* x, int x_dtype, int tokens, int heads, int size, int64_t x_stride, const int32_t* positions,
                       const double* freqs, int rot, int layout, float mscale, int inverse, void* out, int out_dtype,
                       int64_t out_stride, hipStream_t stream) {
  RopeArgs a = {};
  a.q = x;
  a.q_stride = x_stride;
  a.o_stride = out_stride;
  a.in_dtype = x_dtype;
  a.out_dtype = out_dtype;
  a.tokens = tokens;
  a.heads = heads;
  a.size = size;
  a.half = rot / 2;
  a.inverse = inverse;
  a.positions = positions;
  a.freqs = freqs;
  a.mscale = mscale;
  a.out = out;
  return launch(a, layout == RQ_ROPE_INTERLEAVED, 0, (tokens + kRopeTile - 1) / kRopeTile, stream);
}

hipError_t launch_rope_append(const rq_seq_batch* batch, const rq_kv_cache* cache, const void* q, const void* k, const void* v,
                              int in_dtype, int64_t q_stride, int64_t k_stride, int64_t v_stride, int heads,
                              const int32_t* positions, const double* freqs, int rot, int layout, float mscale, void* q_out,
                              int32_t* bad, hipStream_t stream) {
  RopeArgs a = {};
  a.q = q;
  a.k = k;
  a.v = v;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.o_stride = (int64_t)heads * cache->head_dim;
  a.in_dtype = in_dtype;
  a.out_dtype = cache->dtype;
  a.tokens = batch->tokens;
  a.heads = heads;
  a.kv_heads = cache->kv_heads;
  a.size = cache->head_dim;
  a.half = rot / 2;
  a.positions = positions;
  a.freqs = freqs;
  a.mscale = mscale;
  a.out = q_out;
  a.batch = *batch;
  a.cache = *cache;
  a.bad = bad;
  return launch(a, layout == RQ_ROPE_INTERLEAVED, 1, batch->tokens / kRopeTile + 2 * batch->seqs, stream);
}

}  // namespace rq
