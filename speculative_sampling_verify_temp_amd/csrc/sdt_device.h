// What the tree-drafting kernels share on gfx950: the cache's addressing, the
// per-request checks, element conversions and the host checks of the cache
// descriptor.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <math.h>

#include "sd_tree.h"
#include "sdv_device.h"

namespace sdt {

using sdv::WAVE;

// The cache as the kernels see it.
struct Cache {
  char* k;
  char* v;
  int64_t page_stride, head_stride, slot_stride;   // bytes
  const int32_t* table;
  int64_t ld_table;
  const int32_t* lens;
  int B, H, page_shift, page_mask, num_pages, cap;
};

// Nodes of one request; T = 0 and a status bit where the offsets are wrong.
struct Nodes {
  int first, T;
  uint32_t st;
};

__device__ __forceinline__ Nodes request_nodes(const int32_t* off, int b, int N, int max_nodes) {
  const int a = off[b], e = off[b + 1];
  Nodes n{a, e - a, 0u};
  if (a < 0 || e < a || e > N || e - a > max_nodes) n = Nodes{0, 0, SD_ST_BAD_NODES};
  return n;
}

// Slots of request b in use; 0 and a status bit where the length is wrong.
__device__ __forceinline__ int request_ctx(const Cache& c, int b, uint32_t& st) {
  const int n = c.lens[b];
  if (n >= 0 && n <= c.cap) return n;
  st |= SD_ST_BAD_LEN;
  return 0;
}

// Byte offset of (slot, head) in k and in v, -1 on a bad page.  Page indexes
// times strides pass 32 bits in a large pool: 64-bit arithmetic.
__device__ __forceinline__ int64_t slot_offset(const Cache& c, const int32_t* row, int slot, int h) {
  const int p = row[slot >> c.page_shift];
  if ((unsigned)p >= (unsigned)c.num_pages) return -1;
  return p * c.page_stride + h * c.head_stride + (slot & c.page_mask) * c.slot_stride;
}

__device__ __forceinline__ const int32_t* table_row(const Cache& c, int b) {
  return c.table + b * c.ld_table;
}

// A 16-bit element as fp32.
template <int DT>
__device__ __forceinline__ float to_f32(uint16_t u) {
  if constexpr (DT == SD_BF16) return __uint_as_float((uint32_t)u << 16);
  _Float16 h;
  __builtin_memcpy(&h, &u, 2);
  return (float)h;
}

// fp32 rounded to a 16-bit element (to nearest, ties to even).
template <int DT>
__device__ __forceinline__ uint16_t from_f32(float x) {
  uint16_t u;
  if constexpr (DT == SD_BF16) {
    const __bf16 h = (__bf16)x;
    __builtin_memcpy(&u, &h, 2);
  } else {
    const _Float16 h = (_Float16)x;
    __builtin_memcpy(&u, &h, 2);
  }
  return u;
}

// ---- rows of logits ----

template <int DT>
__device__ __forceinline__ float to_float(const char* row, int i) {
  if constexpr (DT == SD_BF16) return __uint_as_float((uint32_t)((const uint16_t*)row)[i] << 16);
  return ((const float*)row)[i];
}

__device__ __forceinline__ uint64_t wave_max_u64(uint64_t x) {
#pragma unroll
  for (int o = WAVE / 2; o > 0; o >>= 1) {
    const uint64_t y = __shfl_xor(x, o);
    x = y > x ? y : x;
  }
  return x;
}

// Running extremes of raw words, packed 16-bit halves (bf16) or whole (fp32):
// 3 integer operations a word.  As signed numbers the bits order the values that
// are not negative and put a positive NaN above +inf; as unsigned ones they order
// the negative ones downwards and put a negative NaN above -inf.
template <int DT>
struct Extremes {
  typedef short s16x2 __attribute__((ext_vector_type(2)));
  typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
  uint32_t smax, umax, umin;
  __device__ void clear() {
    constexpr uint32_t NINF = DT == SD_BF16 ? 0xFF80FF80u : 0xFF800000u;
    smax = umax = umin = NINF;
  }
  __device__ void add(uint32_t w) {
    if constexpr (DT == SD_BF16) {
      const s16x2 s = __builtin_elementwise_max(__builtin_bit_cast(s16x2, smax), __builtin_bit_cast(s16x2, w));
      const u16x2 u = __builtin_elementwise_max(__builtin_bit_cast(u16x2, umax), __builtin_bit_cast(u16x2, w));
      const u16x2 v = __builtin_elementwise_min(__builtin_bit_cast(u16x2, umin), __builtin_bit_cast(u16x2, w));
      smax = __builtin_bit_cast(uint32_t, s);
      umax = __builtin_bit_cast(uint32_t, u);
      umin = __builtin_bit_cast(uint32_t, v);
    } else {
      smax = (uint32_t)max((int)smax, (int)w);
      umax = max(umax, w);
      umin = min(umin, w);
    }
  }
  // Largest value, and whether a NaN was seen.
  __device__ float value(bool& nan) const {
    if constexpr (DT == SD_BF16) {
      const int s = max((int)(short)(smax & 0xFFFF), (int)(short)(smax >> 16));
      const uint32_t u = max(umax & 0xFFFFu, umax >> 16), v = min(umin & 0xFFFFu, umin >> 16);
      nan |= s > 0x7F80 || u > 0xFF80u;
      return __uint_as_float((s >= 0 ? (uint32_t)s : v) << 16);
    } else {
      nan |= (int)smax > 0x7F800000 || umax > 0xFF800000u;
      return __uint_as_float((int)smax >= 0 ? smax : umin);
    }
  }
};

// ---- MFMA 16x16x32 ----

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(1))) u32x4 global_u32x4;
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

template <int DT>
__device__ __forceinline__ f32x4 mfma(const s16x8& a, const s16x8& b, const f32x4& c) {
  if constexpr (DT == SD_BF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// Over the lanes l, l ^ 16, l ^ 32, l ^ 48: the four that share a column of a
// 16x16 result.
__device__ __forceinline__ float quad_max(float x) {
  auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
  r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float quad_sum(float x) {
  auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// Swizzle of a row's chunks: 16 rows at one chunk position cover all banks.
template <int D>
__device__ __forceinline__ int swz(int row) {
  return D == 128 ? row & 15 : (row >> 1) & 7;
}

// ---- host side ----

inline bool aligned16(const void* p) { return ((uintptr_t)p % 16) == 0; }

// SD_OK or the code of the first defect of a cache descriptor.
inline int check_cache(const sd_kv_cache_t& c) {
  if (!c.k || !c.v || !c.page_table || !c.context_lens || !aligned16(c.k) || !aligned16(c.v))
    return SD_EINVAL;
  if (c.dtype != SD_BF16 && c.dtype != SD_F16) return SD_EINVAL;
  if (c.B < 1 || c.H_kv < 1 || c.D < 1 || c.page_size < 1 || c.num_pages < 1 || c.max_pages < 1 ||
      c.ld_table < c.max_pages)
    return SD_EINVAL;
  if (c.page_stride < 0 || c.head_stride < 0 || c.slot_stride < c.D || c.page_stride % 8 ||
      c.head_stride % 8 || c.slot_stride % 8)
    return SD_EINVAL;
  if (c.D != 64 && c.D != 128) return SD_EUNSUPPORTED;
  if ((c.page_size & (c.page_size - 1)) || c.page_size > SD_MAX_PAGE_SIZE) return SD_EUNSUPPORTED;
  if ((int64_t)c.max_pages * c.page_size > (1 << 30)) return SD_EUNSUPPORTED;
  if (c.B > 65535 || c.H_kv > 65535) return SD_EUNSUPPORTED;
  return SD_OK;
}

inline Cache device_cache(const sd_kv_cache_t& c) {
  Cache d;
  d.k = static_cast<char*>(c.k);
  d.v = static_cast<char*>(c.v);
  d.page_stride = c.page_stride * 2;
  d.head_stride = c.head_stride * 2;
  d.slot_stride = c.slot_stride * 2;
  d.table = c.page_table;
  d.ld_table = c.ld_table;
  d.lens = c.context_lens;
  d.B = c.B;
  d.H = c.H_kv;
  d.page_shift = __builtin_ctz((unsigned)c.page_size);
  d.page_mask = c.page_size - 1;
  d.num_pages = c.num_pages;
  d.cap = c.max_pages * c.page_size;
  return d;
}

// Strides of packed node rows: 16-byte aligned rows.
inline bool rows_ok(const void* p, int64_t node, int64_t head) {
  return p && aligned16(p) && node >= 0 && head >= 0 && node % 8 == 0 && head % 8 == 0;
}

}  // namespace sdt
