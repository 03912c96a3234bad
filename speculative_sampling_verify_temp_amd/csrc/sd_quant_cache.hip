// Append to a paged key/value cache held in 8 bits on gfx950.
//
// A workgroup takes one block of slots of one head, of keys or of values: the
// largest magnitude of its new rows gives the scale, then the rows' codes are
// written.  Bound by HBM for prompts (2 bytes read, 1 written an element), by
// latency for the few rows that a verify keeps.
//
// The new rows of a block are read once, into registers, where they fit (blocks
// of up to 64 slots); larger blocks read them again for the codes.  Scales are
// inverted once a block, so an element costs a product, a rounding and the
// packing.  Nothing is used twice, so loads and stores pass the caches by: prompts
// of 4099 tokens, 8 heads of 128, 8 requests, blocks of 64, go from 47.8 to 43.0 us,
// 4.7 TB/s of the 5.15 that a copy reaches (workgroups of 512 threads: 48, heads
// side by side in the grid: 49).  6 kept tokens of 32 requests, 4 heads: 4.4 us.
#include <algorithm>
#include <type_traits>

#include "sdq_device.h"

using namespace sdv;
using namespace sdt;
using namespace sdq;

namespace {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

struct AppendArgs {
  QuantCache c;
  const char *kn, *vn;
  int64_t k_node, k_head, v_node, v_head;   // bytes
  const int32_t* off;
  const int32_t* path;
  int64_t ld_path;
  const int32_t* path_lens;
  int N, max_new;
  int32_t* out_ctx;
  uint32_t* status;
};

struct New {
  int ctx, m, first;
  uint32_t st;
};

// The request's new rows; m = 0 where anything about it is wrong.  Called by
// whole waves: every lane gets the same answer.
__device__ __forceinline__ New request_new(const AppendArgs& a, int b) {
  const Nodes nd = request_nodes(a.off, b, a.N, a.max_new);
  New r{0, nd.T, nd.first, nd.st};
  r.ctx = request_ctx(a.c, b, r.st);
  if (a.path) {
    r.m = a.path_lens[b];
    const int l = threadIdx.x % WAVE;
    bool bad = r.m < 0 || r.m > nd.T;
    if (!bad && l < r.m) {      // (at most 64 of them)
      const int p = a.path[b * a.ld_path + l];
      bad = p < 0 || p >= nd.T;
    }
    if (__any(bad)) r.st |= SD_ST_BAD_PATH;
  }
  if (!r.st && (int64_t)r.ctx + r.m > a.c.cap) r.st |= SD_ST_BAD_LEN;
  if (r.st) r.m = 0;
  return r;
}

// Status, one wave per request, ahead of the rows, which add to it.
__global__ __launch_bounds__(WAVE) void k_append_status(AppendArgs a) {
  const int b = blockIdx.x, l = threadIdx.x;
  const New r = request_new(a, b);
  const int32_t* tab = a.c.table + b * a.c.ld_table;
  bool bad = false;
  if (r.m > 0)
    for (int p = (r.ctx >> a.c.page_shift) + l; p <= (r.ctx + r.m - 1) >> a.c.page_shift; p += WAVE)
      bad |= (unsigned)tab[p] >= (unsigned)a.c.num_pages;
  const uint32_t st = r.st | (__any(bad) ? SD_ST_BAD_PAGE : 0u);
  if (l == 0) a.status[b] = st;
}

template <int CODE>
constexpr float top() { return CODE == SD_I8 ? 127.0f : 448.0f; }

// Four values times inv as codes; STRANGE: some may not be finite.
template <int CODE, bool STRANGE>
__device__ __forceinline__ uint32_t codes4(const float* x, float inv) {
  constexpr float T = top<CODE>();
  float y[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    y[i] = __builtin_amdgcn_fmed3f(x[i] * inv, -T, T);
    if constexpr (STRANGE) {
      if (x[i] != x[i]) y[i] = 0.0f;
      else if (!(fabsf(x[i]) < INFINITY)) y[i] = copysignf(T, x[i]);
    }
  }
  if constexpr (CODE == SD_I8) {
    uint32_t u = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) u |= ((uint32_t)(int)rintf(y[i]) & 255u) << (8 * i);
    return u;
  } else {
    int u = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], 0, false);
    u = __builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], u, true);
    return (uint32_t)u;
  }
}

// Four codes as values, without their scale.
template <int CODE>
__device__ __forceinline__ void values4(uint32_t u, float (&x)[4]) {
  if constexpr (CODE == SD_I8) {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = (float)(int8_t)(u >> (8 * i));
  } else {
    x[0] = __builtin_amdgcn_cvt_f32_fp8((int)u, 0);
    x[1] = __builtin_amdgcn_cvt_f32_fp8((int)u, 1);
    x[2] = __builtin_amdgcn_cvt_f32_fp8((int)u, 2);
    x[3] = __builtin_amdgcn_cvt_f32_fp8((int)u, 3);
  }
}

template <int DT>
__device__ __forceinline__ void unpack8(const uint4& v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = to_f32<DT>((uint16_t)w[i]);
    x[2 * i + 1] = to_f32<DT>((uint16_t)(w[i] >> 16));
  }
}

// grid (blocks that max_new rows may touch, 2 H, B).  A thread holds up to UA
// vectors of 8 elements of the block's new rows at a time.
constexpr int UA = 4;

template <int DT, int CODE, int D, int NT>
__global__ __launch_bounds__(NT) void k_append(AppendArgs a) {
  constexpr int VPR = D / 8;       // vectors of a row
  __shared__ float part[NT / WAVE];
  const int b = blockIdx.z, tid = threadIdx.x;
  const bool value = blockIdx.y & 1;
  const int h = blockIdx.y >> 1;
  const New nw = request_new(a, b);
  if (blockIdx.x == 0 && blockIdx.y == 0 && tid == 0)
    a.out_ctx[b] = (nw.st & SD_ST_BAD_LEN) ? a.c.lens[b] : nw.ctx + nw.m;
  const int block = 1 << a.c.block_shift;
  if (nw.m <= 0 || (int)blockIdx.x > ((nw.m - 1) >> a.c.block_shift) + 1) return;      // past what the rows can touch
  const int start = (nw.ctx & -block) + blockIdx.x * block;
  const int lo = max(nw.ctx, start) - start, hi = min(nw.ctx + nw.m - start, block);      // the block's new slots
  if (lo >= hi) return;
  const int page = a.c.table[b * a.c.ld_table + (start >> a.c.page_shift)];
  if ((unsigned)page >= (unsigned)a.c.num_pages) return;
  const int place = start & a.c.page_mask;
  char* const out = (value ? a.c.v : a.c.k) + page * a.c.page_stride + h * a.c.head_stride + place * a.c.slot_stride;
  float* const scale_at = (value ? a.c.vs : a.c.ks) + page * a.c.scale_page + h * a.c.scale_head +
                          (place >> a.c.block_shift);
  const char* const in = (value ? a.vn : a.kn) + h * (value ? a.v_head : a.k_head);
  const int64_t in_node = value ? a.v_node : a.k_node;
  float old = lo > 0 ? *scale_at : 0.0f;
  if (!scale_ok(old)) old = 0.0f;

  const int n = (hi - lo) * VPR;      // vectors of the new rows
  auto load = [&](int v) {
    const int i = start + lo + v / VPR - nw.ctx;
    const int64_t row = nw.first + (a.path ? a.path[b * a.ld_path + i] : i);
    return __builtin_bit_cast(uint4, __builtin_nontemporal_load((const u32x4*)(in + row * in_node + (v % VPR) * 16)));
  };
  uint4 w[UA];
  auto load_round = [&](int v0) {
#pragma unroll
    for (int u = 0; u < UA; ++u) {
      const int v = v0 + u * NT + tid;
      w[u] = v < n ? load(v) : make_uint4(0, 0, 0, 0);
    }
  };
  // Magnitudes order as their bits do, two elements to a packed maximum; what
  // is not finite lies above the rest and is looked at only where there is some.
  typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
  constexpr uint32_t INF = DT == SD_BF16 ? 0x7F80u : 0x7C00u;
  u16x2 bits = {0, 0};
  for (int v0 = 0; v0 < n; v0 += NT * UA) {
    load_round(v0);
#pragma unroll
    for (int u = 0; u < UA; ++u) {
      const uint32_t q[4] = {w[u].x, w[u].y, w[u].z, w[u].w};
#pragma unroll
      for (int i = 0; i < 4; ++i)
        bits = __builtin_elementwise_max(bits, __builtin_bit_cast(u16x2, q[i] & 0x7FFF7FFFu));
    }
  }
  const uint16_t most = bits[0] > bits[1] ? bits[0] : bits[1];
  float amax = to_f32<DT>(most);
  const bool strange = __any(most >= INF);
  if (strange) {
    amax = 0.0f;
    for (int v0 = 0; v0 < n; v0 += NT * UA) {
      if (n > NT * UA) load_round(v0);
#pragma unroll
      for (int u = 0; u < UA; ++u) {
        float x[8];
        unpack8<DT>(w[u], x);
#pragma unroll
        for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(x[i]) < INFINITY ? fabsf(x[i]) : 0.0f);
      }
    }
  }
  amax = wave_max(amax);
  if constexpr (NT > WAVE) {
    if (tid % WAVE == 0) part[tid / WAVE] = amax;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NT / WAVE; ++i) amax = fmaxf(amax, part[i]);
  }
  float fresh = amax > 0.0f ? fminf(fmaxf(amax / top<CODE>(), MIN_SCALE), MAX_SCALE) : 0.0f;
  const float scale = fmaxf(old, fresh);
  const float inv = scale > 0.0f ? 1.0f / scale : 0.0f;
  if (tid == 0) *scale_at = scale;

  for (int v0 = 0; v0 < n; v0 += NT * UA) {
#pragma unroll
    for (int u = 0; u < UA; ++u) {
      const int v = v0 + u * NT + tid;
      if (v >= n) break;
      if (n > NT * UA) w[u] = load(v);
      float x[8];
      unpack8<DT>(w[u], x);
      u32x2 c;
      if (strange) c = u32x2{codes4<CODE, true>(x, inv), codes4<CODE, true>(x + 4, inv)};
      else c = u32x2{codes4<CODE, false>(x, inv), codes4<CODE, false>(x + 4, inv)};
      __builtin_nontemporal_store(c, (u32x2*)(out + (lo + v / VPR) * a.c.slot_stride + (v % VPR) * 8));
    }
  }
  // the codes of slots that were there, where their scale has grown
  if (lo > 0 && scale > old) {
    for (int v = tid; v < lo * VPR; v += NT) {
      uint2* const at = (uint2*)(out + (v / VPR) * a.c.slot_stride + (v % VPR) * 8);
      const uint2 c = *at;
      float x[4], y[4];
      values4<CODE>(c.x, x);
      values4<CODE>(c.y, y);
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] *= old, y[i] *= old;
      *at = make_uint2(codes4<CODE, true>(x, inv), codes4<CODE, true>(y, inv));
    }
  }
  if (a.status && strange && tid % WAVE == 0) atomicOr(&a.status[b], (uint32_t)SD_ST_NONFINITE);
}

int check(const sd_quant_append_args_t* p) {
  if (!p) return SD_EINVAL;
  const int rc = check_cache(p->cache);
  if (rc) return rc;
  if (p->dtype != SD_BF16 && p->dtype != SD_F16) return SD_EINVAL;
  if (!rows_ok(p->k_new, p->k_node, p->k_head) || !rows_ok(p->v_new, p->v_node, p->v_head) || !p->node_offsets ||
      p->N < 1 || p->max_new < 1)
    return SD_EINVAL;
  if (p->path && (!p->path_lens || p->ld_path < p->max_new)) return SD_EINVAL;
  if (p->path && p->max_new > SD_MAX_NODES) return SD_EUNSUPPORTED;
  // rows and scales of pages and heads are their own
  const sd_quant_cache_t& c = p->cache;
  if ((c.num_pages > 1 && (!c.page_stride || !c.scale_page)) || (c.H_kv > 1 && (!c.head_stride || !c.scale_head)))
    return SD_EINVAL;
  if (c.k == c.v || c.k_scale == c.v_scale) return SD_EINVAL;
  return SD_OK;
}

// One wave a block where its rows fit the registers of one.
template <int DT, int CODE, int D>
void launch(const AppendArgs& a, unsigned blocks, hipStream_t st) {
  const int block = 1 << a.c.block_shift;
  const dim3 grid(blocks, 2 * a.c.H, a.c.B);
  if (block * (D / 8) <= WAVE * UA)
    hipLaunchKernelGGL((k_append<DT, CODE, D, WAVE>), grid, dim3(WAVE), 0, st, a);
  else
    hipLaunchKernelGGL((k_append<DT, CODE, D, 256>), grid, dim3(256), 0, st, a);
}

}  // namespace

extern "C" int sd_quant_append(const sd_quant_append_args_t* p, int32_t* out_context,
                               uint32_t* out_status, void* stream) {
  const int rc = check(p);
  if (rc) return rc;
  if (!out_context || (const void*)out_status == out_context) return SD_EINVAL;
  for (const int32_t* in : {p->cache.context_lens, p->cache.page_table, p->node_offsets, p->path, p->path_lens})
    if (out_context == in || (out_status && out_status == (const uint32_t*)in)) return SD_EINVAL;
  AppendArgs a;
  a.c = device_cache(p->cache);
  a.kn = static_cast<const char*>(p->k_new), a.vn = static_cast<const char*>(p->v_new);
  a.k_node = p->k_node * 2, a.k_head = p->k_head * 2, a.v_node = p->v_node * 2, a.v_head = p->v_head * 2;
  a.off = p->node_offsets;
  a.path = p->path, a.ld_path = p->ld_path, a.path_lens = p->path_lens;
  a.N = p->N, a.max_new = p->max_new;
  a.out_ctx = out_context, a.status = out_status;
  // a grid dimension holds less than 2^32 threads
  const int blocks = ((std::min(a.max_new, a.c.cap) - 1) >> a.c.block_shift) + 2;
  if (blocks >= 1 << 24) return SD_EUNSUPPORTED;
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (out_status) {
    hipLaunchKernelGGL(k_append_status, dim3(a.c.B), dim3(WAVE), 0, st, a);
    if (hipGetLastError() != hipSuccess) return SD_EHIP;
  }
  auto go = [&](auto dt, auto code) {
    if (p->cache.D == 64) launch<decltype(dt)::value, decltype(code)::value, 64>(a, (unsigned)blocks, st);
    else launch<decltype(dt)::value, decltype(code)::value, 128>(a, (unsigned)blocks, st);
  };
  using BF = std::integral_constant<int, SD_BF16>;
  using HF = std::integral_constant<int, SD_F16>;
  using I8 = std::integral_constant<int, SD_I8>;
  using E4 = std::integral_constant<int, SD_E4M3>;
  if (p->cache.code == SD_I8) p->dtype == SD_BF16 ? go(BF{}, I8{}) : go(HF{}, I8{});
  else p->dtype == SD_BF16 ? go(BF{}, E4{}) : go(HF{}, E4{});
  return hipGetLastError() == hipSuccess ? SD_OK : SD_EHIP;
}
