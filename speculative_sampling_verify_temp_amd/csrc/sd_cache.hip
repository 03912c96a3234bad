// Append to and eviction from a paged key/value cache on gfx950.
//
// sd_cache_commit:
//   k_commit_append  one workgroup per request: the branch's keys, values and
//                    positions into the slots behind the context;
//   k_commit_mass    one thread per (slot, KV head): the slot's weight, a sum
//                    of exp(scale q . k - lse) over the branch's query rows.
// sd_cache_evict:
//   k_evict_select   one workgroup per (request, KV head): the budget-th
//                    largest key by a radix search, then the freed slots
//                    below the budget and the kept ones past it, in order;
//   k_evict_move     16 bytes a lane: each kept row past the budget into its
//                    freed slot.
#include <algorithm>

#include "sdt_device.h"

using namespace sdv;
using namespace sdt;

namespace {

struct CommitArgs {
  Cache c;
  const char *kn, *vn;
  int64_t k_node, k_head, v_node, v_head;   // bytes
  const int32_t* off;
  const int32_t* path;
  int64_t ld_path;
  const int32_t* path_lens;
  int N, max_nodes;
  const char* q;
  int64_t q_node, q_head;
  const float* lse;
  int Hq, G;
  float scale, decay;
  const float* mass_in;
  float* mass_out;
  int64_t ld_mass;
  int32_t* positions;
  const int32_t* seen;
  int32_t* out_ctx;
  uint32_t* status;
};

struct Branch {
  int ctx, m, first;
  uint32_t st;
};

// The request's branch; m = 0 where anything about it is wrong.  Called by
// whole waves: every lane gets the same answer.
__device__ __forceinline__ Branch request_branch(const CommitArgs& a, int b) {
  const Nodes nd = request_nodes(a.off, b, a.N, a.max_nodes);
  Branch r{0, 0, nd.first, nd.st};
  r.ctx = request_ctx(a.c, b, r.st);
  const int m = a.path_lens[b];
  const int l = threadIdx.x % WAVE;
  bool bad = m < 0 || m > nd.T;
  if (!bad && l < m) {
    const int p = a.path[b * a.ld_path + l];
    bad = p < 0 || p >= nd.T;
  }
  if (__any(bad)) r.st |= SD_ST_BAD_PATH;
  else {
    const int64_t end = (int64_t)r.ctx + m;
    if (end > a.c.cap || ((a.mass_out || a.positions) && end > a.ld_mass)) r.st |= SD_ST_BAD_LEN;
  }
  r.m = r.st ? 0 : m;
  return r;
}

template <int D>
__global__ __launch_bounds__(256) void k_commit_append(CommitArgs a) {
  constexpr int LPR = D / 8;   // lanes of one row
  const int b = blockIdx.x, tid = threadIdx.x;
  const Branch r = request_branch(a, b);
  const int32_t* tab = table_row(a.c, b);
  for (int u = tid / LPR; u < r.m * a.c.H; u += 256 / LPR) {
    const int i = u / a.c.H, h = u % a.c.H, d = (tid % LPR) * 16;
    const int64_t at = slot_offset(a.c, tab, r.ctx + i, h);
    const int64_t row = r.first + a.path[b * a.ld_path + i];
    if (at >= 0) {
      *(uint4*)(a.c.k + at + d) = *(const uint4*)(a.kn + row * a.k_node + h * a.k_head + d);
      *(uint4*)(a.c.v + at + d) = *(const uint4*)(a.vn + row * a.v_node + h * a.v_head + d);
    }
    if (a.positions && d == 0)
      a.positions[((int64_t)b * a.c.H + h) * a.ld_mass + r.ctx + i] = a.seen[b] + i;
  }
  if (tid >= WAVE) return;
  if (tid == 0) a.out_ctx[b] = (r.st & SD_ST_BAD_LEN) ? a.c.lens[b] : r.ctx + r.m;
  if (!a.status) return;
  bool bad_page = false;
  for (int p = tid; p < (r.ctx + r.m + a.c.page_mask) >> a.c.page_shift; p += WAVE)
    bad_page |= (unsigned)tab[p] >= (unsigned)a.c.num_pages;
  const uint32_t st = r.st | (__any(bad_page) ? SD_ST_BAD_PAGE : 0u);
  if (tid == 0) a.status[b] = st;
}

template <int DT, int D>
__global__ __launch_bounds__(256) void k_commit_mass(CommitArgs a) {
  const int b = blockIdx.z, h = blockIdx.y;
  const Branch r = request_branch(a, b);
  if (r.st) return;
  const int32_t* tab = table_row(a.c, b);
  for (int t = blockIdx.x * 256 + threadIdx.x; t < r.ctx + r.m; t += gridDim.x * 256) {
    const bool fresh = t >= r.ctx;
    const char* k = nullptr;
    if (fresh) {
      const int64_t row = r.first + a.path[b * a.ld_path + t - r.ctx];
      k = a.kn + row * a.k_node + h * a.k_head;
    } else {
      const int64_t at = slot_offset(a.c, tab, t, h);
      if (at >= 0) k = a.c.k + at;
    }
    float w = 0.0f;
    for (int i = fresh ? t - r.ctx : 0; k && i < r.m; ++i) {
      const int64_t row = r.first + a.path[b * a.ld_path + i];
      for (int g = h * a.G; g < (h + 1) * a.G; ++g) {
        const uint16_t* q = (const uint16_t*)(a.q + row * a.q_node + g * a.q_head);
        float x = 0.0f;
        for (int d = 0; d < D; ++d) x = fmaf(to_f32<DT>(q[d]), to_f32<DT>(((const uint16_t*)k)[d]), x);
        w += expf(x * a.scale - a.lse[row * a.Hq + g]);
      }
    }
    const int64_t at = ((int64_t)b * a.c.H + h) * a.ld_mass + t;
    if (!fresh && a.decay != 0.0f) w += a.decay * a.mass_in[at];
    a.mass_out[at] = w;
  }
}

// ---- eviction ----

constexpr int NT_E = 1024;

struct EvictArgs {
  Cache c;
  const float* mass_in;
  float* mass_out;
  const int32_t* pos_in;
  int32_t* pos_out;
  int64_t ld;
  const int32_t* seen;
  int budget, recent, sinks;
  int moves;                 // most rows that one head can move
  int32_t *holes, *late, *count;   // [B * H][moves], [B * H]
  int32_t* out_ctx;
  uint32_t* status;
};

// Rank key of a slot: protected positions above every mass, NaN as -inf.
__device__ __forceinline__ uint32_t evict_key(const EvictArgs& a, int64_t row, int t, int recent_from) {
  if (a.pos_in) {
    const int p = a.pos_in[row + t];
    if (p < a.sinks || p >= recent_from) return 0xFFFFFFFFu;
  }
  const float m = a.mass_in[row + t];
  return ord_key(m != m ? -INFINITY : m);
}

__global__ __launch_bounds__(NT_E) void k_evict_select(EvictArgs a) {
  __shared__ int hist[256];
  __shared__ int scratch[NT_E / WAVE];
  __shared__ int sel[2];
  const int h = blockIdx.x, b = blockIdx.y, tid = threadIdx.x;
  uint32_t st = 0;
  const int n = request_ctx(a.c, b, st);
  const int bh = b * a.c.H + h;
  const int64_t row = (int64_t)bh * a.ld;
  if (st) {
    if (tid == 0) a.count[bh] = 0;
    return;
  }
  const int64_t from = a.pos_in && a.recent > 0 ? (int64_t)a.seen[b] - a.recent : 0x7FFFFFFF;
  const int recent_from = a.pos_in && a.recent > 0 ? (int)max(from, (int64_t)INT_MIN) : INT_MAX;
  // the budget-th largest key, eight bits at a time; `want` slots of the
  // keys equal to it are kept, the lowest
  uint32_t cut = 0;
  int want = a.budget;
  const bool all = n <= a.budget;
  for (int shift = 24; !all && shift >= 0; shift -= 8) {
    for (int i = tid; i < 256; i += NT_E) hist[i] = 0;
    __syncthreads();
    for (int t = tid; t < n; t += NT_E) {
      const uint32_t k = evict_key(a, row, t, recent_from);
      if (shift == 24 || (k >> (shift + 8)) == (cut >> (shift + 8))) atomicAdd(&hist[(k >> shift) & 255], 1);
    }
    __syncthreads();
    if (tid == 0) {
      int w = want, i = 255;
      while (i > 0 && hist[i] < w) w -= hist[i--];
      sel[0] = i, sel[1] = w;
    }
    __syncthreads();
    cut |= (uint32_t)sel[0] << shift;
    want = sel[1];
    __syncthreads();
  }
  int equal = 0, holes = 0, late = 0;
  for (int t0 = 0; t0 < n; t0 += NT_E) {
    const int t = t0 + tid;
    uint32_t k = 0;
    if (t < n) k = evict_key(a, row, t, recent_from);
    bool keep = t < n && all;
    if (!all) {
      int tot;
      const int e = t < n && k == cut;
      const int at = equal + block_excl_scan_int<NT_E>(e, scratch, &tot);
      equal += tot;
      keep = t < n && (k > cut || (e && at < want));
    }
    const bool hole = t < n && t < a.budget && !keep, move = keep && t >= a.budget;
    int tot;
    const int hp = holes + block_excl_scan_int<NT_E>(hole, scratch, &tot);
    holes += tot;
    const int lp = late + block_excl_scan_int<NT_E>(move, scratch, &tot);
    late += tot;
    if (hole) a.holes[(int64_t)bh * a.moves + hp] = t;
    if (move) a.late[(int64_t)bh * a.moves + lp] = t;
    if (keep && !move) {
      a.mass_out[row + t] = a.mass_in[row + t];
      if (a.pos_in) a.pos_out[row + t] = a.pos_in[row + t];
    }
  }
  if (tid == 0) a.count[bh] = late;
}

template <int D>
__global__ __launch_bounds__(256) void k_evict_move(EvictArgs a) {
  constexpr int LPR = D / 8;
  const int h = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
  const int bh = b * a.c.H + h, n = a.count[bh];
  const int64_t row = (int64_t)bh * a.ld, list = (int64_t)bh * a.moves;
  const int32_t* tab = table_row(a.c, b);
  const int d = (tid % LPR) * 16;
  for (int i = blockIdx.x * (256 / LPR) + tid / LPR; i < n; i += gridDim.x * (256 / LPR)) {
    const int src = a.late[list + i], dst = a.holes[list + i];
    const int64_t s = slot_offset(a.c, tab, src, h), t = slot_offset(a.c, tab, dst, h);
    if (s >= 0 && t >= 0) {
      *(uint4*)(a.c.k + t + d) = *(const uint4*)(a.c.k + s + d);
      *(uint4*)(a.c.v + t + d) = *(const uint4*)(a.c.v + s + d);
    }
    if (d == 0) {
      a.mass_out[row + dst] = a.mass_in[row + src];
      if (a.pos_in) a.pos_out[row + dst] = a.pos_in[row + src];
    }
  }
  if (h == 0 && blockIdx.x == 0 && tid < WAVE) {
    uint32_t st = 0;
    const int ctx = request_ctx(a.c, b, st);
    if (tid == 0) a.out_ctx[b] = st ? a.c.lens[b] : min(ctx, a.budget);
    if (!a.status) return;
    bool bad_page = false;
    for (int p = tid; p < (ctx + a.c.page_mask) >> a.c.page_shift; p += WAVE)
      bad_page |= (unsigned)tab[p] >= (unsigned)a.c.num_pages;
    if (__any(bad_page)) st |= SD_ST_BAD_PAGE;
    if (tid == 0) a.status[b] = st;
  }
}

int check(const sd_cache_commit_args_t* p) {
  if (!p) return SD_EINVAL;
  const int rc = check_cache(p->cache);
  if (rc) return rc;
  if (p->max_nodes > SD_MAX_NODES) return SD_EUNSUPPORTED;
  if (!rows_ok(p->k_new, p->k_node, p->k_head) || !rows_ok(p->v_new, p->v_node, p->v_head) ||
      !p->node_offsets || !p->path || !p->path_lens || p->N < 1 || p->max_nodes < 1 ||
      p->ld_path < p->max_nodes || !p->positions != !p->seen)
    return SD_EINVAL;
  if ((p->mass_out || p->positions) && p->ld_mass < 1) return SD_EINVAL;
  if (p->mass_out) {
    if (!rows_ok(p->q, p->q_node, p->q_head) || !p->lse || p->H_q < 1 || p->H_q % p->cache.H_kv ||
        !isfinite(p->scale) || !isfinite(p->decay) || (p->decay != 0.0f && !p->mass_in))
      return SD_EINVAL;
    if (p->H_q / p->cache.H_kv > SD_MAX_GROUP) return SD_EUNSUPPORTED;
  }
  return SD_OK;
}

int check(const sd_cache_evict_args_t* p) {
  if (!p) return SD_EINVAL;
  const int rc = check_cache(p->cache);
  if (rc) return rc;
  if (!p->mass_in || !p->mass_out || !p->positions_in != !p->positions_out || p->budget < 1 ||
      p->recent < 0 || p->sinks < 0 || (int64_t)p->recent + p->sinks > p->budget ||
      p->ld_mass < (int64_t)p->cache.max_pages * p->cache.page_size)
    return SD_EINVAL;
  if (p->positions_in ? !p->seen : (p->recent || p->sinks)) return SD_EINVAL;
  return SD_OK;
}

int most_moves(const sd_cache_evict_args_t* p) {
  const int cap = p->cache.max_pages * p->cache.page_size;
  return std::max(0, std::min(p->budget, cap - p->budget));
}

}  // namespace

extern "C" int sd_cache_commit(const sd_cache_commit_args_t* args, int32_t* out_context,
                               uint32_t* out_status, void* stream) {
  const int rc = check(args);
  if (rc) return rc;
  if (!out_context || out_context == args->cache.context_lens) return SD_EINVAL;
  CommitArgs a{};
  a.c = device_cache(args->cache);
  a.kn = static_cast<const char*>(args->k_new);
  a.vn = static_cast<const char*>(args->v_new);
  a.k_node = args->k_node * 2, a.k_head = args->k_head * 2;
  a.v_node = args->v_node * 2, a.v_head = args->v_head * 2;
  a.off = args->node_offsets;
  a.path = args->path, a.ld_path = args->ld_path, a.path_lens = args->path_lens;
  a.N = args->N, a.max_nodes = args->max_nodes;
  a.ld_mass = args->ld_mass;
  a.positions = args->positions, a.seen = args->seen;
  a.mass_out = args->mass_out;
  a.out_ctx = out_context;
  a.status = out_status;
  hipStream_t st = static_cast<hipStream_t>(stream);
  const int D = args->cache.D;
  if (a.mass_out) {
    a.q = static_cast<const char*>(args->q);
    a.q_node = args->q_node * 2, a.q_head = args->q_head * 2;
    a.lse = args->lse;
    a.Hq = args->H_q, a.G = args->H_q / a.c.H;
    a.scale = args->scale, a.decay = args->decay;
    a.mass_in = args->mass_in;
    const dim3 grid(std::min((a.c.cap + 255) / 256, 1024), a.c.H, a.c.B);
    if (args->cache.dtype == SD_BF16) {
      if (D == 64) hipLaunchKernelGGL((k_commit_mass<SD_BF16, 64>), grid, dim3(256), 0, st, a);
      else hipLaunchKernelGGL((k_commit_mass<SD_BF16, 128>), grid, dim3(256), 0, st, a);
    } else {
      if (D == 64) hipLaunchKernelGGL((k_commit_mass<SD_F16, 64>), grid, dim3(256), 0, st, a);
      else hipLaunchKernelGGL((k_commit_mass<SD_F16, 128>), grid, dim3(256), 0, st, a);
    }
    if (hipGetLastError() != hipSuccess) return SD_EHIP;
  }
  if (D == 64) hipLaunchKernelGGL(k_commit_append<64>, dim3(a.c.B), dim3(256), 0, st, a);
  else hipLaunchKernelGGL(k_commit_append<128>, dim3(a.c.B), dim3(256), 0, st, a);
  return hipGetLastError() == hipSuccess ? SD_OK : SD_EHIP;
}

extern "C" int sd_cache_evict_workspace_bytes(const sd_cache_evict_args_t* args, size_t* bytes) {
  if (!bytes) return SD_EINVAL;
  const int rc = check(args);
  if (rc) return rc;
  *bytes = (size_t)args->cache.B * args->cache.H_kv * (2 * (size_t)most_moves(args) + 1) * 4;
  return SD_OK;
}

extern "C" int sd_cache_evict(const sd_cache_evict_args_t* args, void* workspace,
                              size_t workspace_bytes, int32_t* out_context,
                              uint32_t* out_status, void* stream) {
  size_t need = 0;
  const int rc = sd_cache_evict_workspace_bytes(args, &need);
  if (rc) return rc;
  if (!out_context || out_context == args->cache.context_lens) return SD_EINVAL;
  if (!workspace || workspace_bytes < need || (uintptr_t)workspace % 4) return SD_EWORKSPACE;
  EvictArgs a;
  a.c = device_cache(args->cache);
  a.mass_in = args->mass_in, a.mass_out = args->mass_out;
  a.pos_in = args->positions_in, a.pos_out = args->positions_out;
  a.ld = args->ld_mass;
  a.seen = args->seen;
  a.budget = args->budget, a.recent = args->recent, a.sinks = args->sinks;
  a.moves = most_moves(args);
  const size_t bh = (size_t)a.c.B * a.c.H;
  a.holes = static_cast<int32_t*>(workspace);
  a.late = a.holes + bh * a.moves;
  a.count = a.late + bh * a.moves;
  a.out_ctx = out_context;
  a.status = out_status;
  hipStream_t st = static_cast<hipStream_t>(stream);
  hipLaunchKernelGGL(k_evict_select, dim3(a.c.H, a.c.B), dim3(NT_E), 0, st, a);
  if (hipGetLastError() != hipSuccess) return SD_EHIP;
  const int chunks = std::max(1, std::min((a.moves + 63) / 64, 256));
  const dim3 grid(chunks, a.c.H, a.c.B);
  if (args->cache.D == 64) hipLaunchKernelGGL(k_evict_move<64>, grid, dim3(256), 0, st, a);
  else hipLaunchKernelGGL(k_evict_move<128>, grid, dim3(256), 0, st, a);
  return hipGetLastError() == hipSuccess ? SD_OK : SD_EHIP;
}
