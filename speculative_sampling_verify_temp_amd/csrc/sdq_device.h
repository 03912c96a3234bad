// What the kernels of the 8-bit cache share on gfx950: its addressing and the
// host checks of its descriptor.
#pragma once
#include "sd_serve.h"
#include "sdt_device.h"

namespace sdq {

using sdv::WAVE;

constexpr float MIN_SCALE = 0x1p-50f, MAX_SCALE = 0x1p50f;

// The cache as the kernels see it; strides of k and v in bytes, of scales in
// entries.
struct QuantCache {
  char *k, *v;
  float *ks, *vs;
  int64_t page_stride, head_stride, slot_stride, scale_page, scale_head;
  const int32_t* table;
  int64_t ld_table;
  const int32_t* lens;
  int B, H, page_shift, page_mask, block_shift, num_pages, cap;
};

__device__ __forceinline__ int request_ctx(const QuantCache& c, int b, uint32_t& st) {
  const int n = c.lens[b];
  if (n >= 0 && n <= c.cap) return n;
  st |= SD_ST_BAD_LEN;
  return 0;
}

// 0, or within the range that a scale may have.
__device__ __forceinline__ bool scale_ok(float s) { return s == 0.0f || (s >= MIN_SCALE && s <= MAX_SCALE); }

// SD_OK or the code of the first defect of a cache descriptor.
inline int check_cache(const sd_quant_cache_t& c) {
  using sdt::aligned16;
  if (!c.k || !c.v || !c.k_scale || !c.v_scale || !c.page_table || !c.context_lens || !aligned16(c.k) ||
      !aligned16(c.v) || (uintptr_t)c.k_scale % 4 || (uintptr_t)c.v_scale % 4)
    return SD_EINVAL;
  if (c.code != SD_I8 && c.code != SD_E4M3) return SD_EINVAL;
  if (c.B < 1 || c.H_kv < 1 || c.D < 1 || c.page_size < 1 || c.block < 1 || c.num_pages < 1 || c.max_pages < 1 ||
      c.ld_table < c.max_pages)
    return SD_EINVAL;
  if (c.page_stride < 0 || c.head_stride < 0 || c.slot_stride < c.D || c.page_stride % 16 || c.head_stride % 16 ||
      c.slot_stride % 16 || c.scale_page < 0 || c.scale_head < 0)
    return SD_EINVAL;
  if (c.D != 64 && c.D != 128) return SD_EUNSUPPORTED;
  if ((c.page_size & (c.page_size - 1)) || c.page_size > SD_MAX_PAGE_SIZE || (c.block & (c.block - 1)) ||
      c.block < SD_MIN_BLOCK || c.block > c.page_size)
    return SD_EUNSUPPORTED;
  if ((int64_t)c.max_pages * c.page_size > (1 << 30)) return SD_EUNSUPPORTED;
  if (c.B > 65535 || c.H_kv > 32767) return SD_EUNSUPPORTED;
  // offsets within a page are 32 bits wide
  if (c.slot_stride > (1 << 20)) return SD_EUNSUPPORTED;
  return SD_OK;
}

inline QuantCache device_cache(const sd_quant_cache_t& c) {
  QuantCache d;
  d.k = static_cast<char*>(c.k), d.v = static_cast<char*>(c.v);
  d.ks = c.k_scale, d.vs = c.v_scale;
  d.page_stride = c.page_stride, d.head_stride = c.head_stride, d.slot_stride = c.slot_stride;
  d.scale_page = c.scale_page, d.scale_head = c.scale_head;
  d.table = c.page_table, d.ld_table = c.ld_table, d.lens = c.context_lens;
  d.B = c.B, d.H = c.H_kv;
  d.page_shift = __builtin_ctz((unsigned)c.page_size), d.page_mask = c.page_size - 1;
  d.block_shift = __builtin_ctz((unsigned)c.block);
  d.num_pages = c.num_pages, d.cap = c.max_pages * c.page_size;
  return d;
}

}  // namespace sdq
