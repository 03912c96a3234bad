// Attention of a drafted tree over a paged cache on gfx950.
//
// Row (node i, query head g) of a request: s_j = scale q . k_j over the
// request's cache slots and the nodes that i sees, o = softmax(s) . v with a
// running maximum and sum, so the scores never leave the chip.
//
// k_tree_attention: one wave per row.  Lane l scores key 64 t + l of step t,
// then the lanes turn to the D output columns and walk the step's 64 keys.
#include "sdt_device.h"

using namespace sdv;
using namespace sdt;

namespace {

struct AttnArgs {
  Cache c;
  const char *q, *kn, *vn;
  int64_t q_node, q_head, k_node, k_head, v_node, v_head;   // bytes
  const int32_t* off;
  const int32_t* parents;
  const uint64_t* mask;
  int N, max_nodes, Hq, G;
  float scale;
  char* out;
  float* lse;
  uint32_t* status;
};

// The nodes that node i of the request sees, as bits.
__device__ __forceinline__ uint64_t sees(const AttnArgs& a, const Nodes& nd, int i) {
  const uint64_t own = nd.T == 64 ? ~0ull : (1ull << nd.T) - 1;
  if (a.mask) return a.mask[nd.first + i] & own;
  if (!a.parents) return (2ull << i) - 1;
  uint64_t m = 0;
  for (int j = i; j >= 0;) {
    m |= 1ull << j;
    const int p = a.parents[nd.first + j];
    j = p < j ? p : -1;      // p < -1 ends the walk too
  }
  return m;
}

template <int DT, int D>
__global__ __launch_bounds__(WAVE) void k_tree_attention(AttnArgs a) {
  __shared__ float sq[D];
  const int g = blockIdx.x, i = blockIdx.y, b = blockIdx.z, l = threadIdx.x;
  const Nodes nd = request_nodes(a.off, b, a.N, a.max_nodes);
  if (i >= nd.T) return;
  uint32_t st = 0;
  const int ctx = request_ctx(a.c, b, st);
  const int row = nd.first + i, h = g / a.G;
  const uint16_t* q = (const uint16_t*)(a.q + row * a.q_node + g * a.q_head);
  for (int d = l; d < D; d += WAVE) sq[d] = to_f32<DT>(q[d]);
  __syncthreads();
  const int32_t* tab = table_row(a.c, b);
  const uint64_t vis = st ? 0 : sees(a, nd, i);
  const int total = st ? 0 : ctx + nd.T;
  float m = -INFINITY, s = 0.0f, o[D / WAVE] = {};
  for (int t0 = 0; t0 < total; t0 += WAVE) {
    const int t = t0 + l;
    const uint16_t *k = nullptr, *v = nullptr;
    if (t < ctx) {
      const int64_t at = slot_offset(a.c, tab, t, h);
      if (at >= 0) k = (const uint16_t*)(a.c.k + at), v = (const uint16_t*)(a.c.v + at);
    } else if (t < total && (vis >> (t - ctx) & 1)) {
      const int64_t r = nd.first + t - ctx;
      k = (const uint16_t*)(a.kn + r * a.k_node + h * a.k_head);
      v = (const uint16_t*)(a.vn + r * a.v_node + h * a.v_head);
    }
    float x = -INFINITY;
    if (k) {
      x = 0.0f;
      for (int d = 0; d < D; ++d) x = fmaf(sq[d], to_f32<DT>(k[d]), x);
      x *= a.scale;
    }
    const float mn = fmaxf(m, wave_max(x));
    if (!(mn > -INFINITY) && !__any(x != x)) continue;
    const float p = k ? expf(x - mn) : 0.0f;
    const float f = expf(m - mn);
    s = s * f + p;
    m = mn;
#pragma unroll
    for (int u = 0; u < D / WAVE; ++u) o[u] *= f;
    for (int j = 0; j < WAVE; ++j) {
      const float pj = __shfl(p, j);
      const uint64_t vj = __shfl((uint64_t)v, j);
      if (!vj) continue;
#pragma unroll
      for (int u = 0; u < D / WAVE; ++u)
        o[u] = fmaf(pj, to_f32<DT>(((const uint16_t*)vj)[u * WAVE + l]), o[u]);
    }
  }
#pragma unroll
  for (int x = WAVE / 2; x > 0; x >>= 1) s += __shfl_xor(s, x);
  const bool none = s == 0.0f;
  uint16_t* out = (uint16_t*)a.out + ((int64_t)row * a.Hq + g) * D;
#pragma unroll
  for (int u = 0; u < D / WAVE; ++u) out[u * WAVE + l] = from_f32<DT>(none ? 0.0f : o[u] / s);
  if (a.lse && l == 0) a.lse[(int64_t)row * a.Hq + g] = none ? -INFINITY : m + logf(s);
}

// Status bits of one request per workgroup.
__global__ __launch_bounds__(WAVE) void k_tree_status(AttnArgs a) {
  const int b = blockIdx.x, l = threadIdx.x;
  const Nodes nd = request_nodes(a.off, b, a.N, a.max_nodes);
  uint32_t st = nd.st;
  const int ctx = request_ctx(a.c, b, st);
  const int32_t* tab = table_row(a.c, b);
  bool bad_page = false, bad_tree = false;
  for (int p = l; p < (ctx + a.c.page_mask) >> a.c.page_shift; p += WAVE)
    bad_page |= (unsigned)tab[p] >= (unsigned)a.c.num_pages;
  if (a.parents && !a.mask && l < nd.T) {
    const int p = a.parents[nd.first + l];
    bad_tree = p < -1 || p >= l;
  }
  if (__any(bad_page)) st |= SD_ST_BAD_PAGE;
  if (__any(bad_tree)) st |= SD_ST_BAD_TREE;
  if (l == 0) a.status[b] = st;
}

int check(const sd_tree_attention_args_t* p) {
  if (!p) return SD_EINVAL;
  const int rc = check_cache(p->cache);
  if (rc) return rc;
  if (!rows_ok(p->q, p->q_node, p->q_head) || !rows_ok(p->k_new, p->k_node, p->k_head) ||
      !rows_ok(p->v_new, p->v_node, p->v_head) || !p->node_offsets || p->N < 1 ||
      p->max_nodes < 1 || p->H_q < 1 || p->H_q % p->cache.H_kv || !isfinite(p->scale))
    return SD_EINVAL;
  if (p->max_nodes > SD_MAX_NODES || p->H_q / p->cache.H_kv > SD_MAX_GROUP || p->H_q > 65535)
    return SD_EUNSUPPORTED;
  return SD_OK;
}

AttnArgs device_args(const sd_tree_attention_args_t* p) {
  AttnArgs a;
  a.c = device_cache(p->cache);
  a.q = static_cast<const char*>(p->q);
  a.kn = static_cast<const char*>(p->k_new);
  a.vn = static_cast<const char*>(p->v_new);
  a.q_node = p->q_node * 2, a.q_head = p->q_head * 2;
  a.k_node = p->k_node * 2, a.k_head = p->k_head * 2;
  a.v_node = p->v_node * 2, a.v_head = p->v_head * 2;
  a.off = p->node_offsets;
  a.parents = p->parents;
  a.mask = p->tree_mask;
  a.N = p->N;
  a.max_nodes = p->max_nodes;
  a.Hq = p->H_q;
  a.G = p->H_q / p->cache.H_kv;
  a.scale = p->scale;
  return a;
}

template <int DT>
void launch(const AttnArgs& a, int D, hipStream_t st) {
  const dim3 grid(a.Hq, a.max_nodes, a.c.B);
  if (D == 64)
    hipLaunchKernelGGL((k_tree_attention<DT, 64>), grid, dim3(WAVE), 0, st, a);
  else
    hipLaunchKernelGGL((k_tree_attention<DT, 128>), grid, dim3(WAVE), 0, st, a);
}

}  // namespace

extern "C" int sd_tree_attention_workspace_bytes(const sd_tree_attention_args_t* args, size_t* bytes) {
  if (!bytes) return SD_EINVAL;
  const int rc = check(args);
  if (rc) return rc;
  *bytes = 0;
  return SD_OK;
}

extern "C" int sd_tree_attention(const sd_tree_attention_args_t* args, void* workspace,
                                 size_t workspace_bytes, void* out, float* out_lse,
                                 uint32_t* out_status, void* stream) {
  size_t need = 0;
  const int rc = sd_tree_attention_workspace_bytes(args, &need);
  if (rc) return rc;
  if (!out || !aligned16(out)) return SD_EINVAL;
  if (need && (!workspace || workspace_bytes < need)) return SD_EWORKSPACE;
  AttnArgs a = device_args(args);
  a.out = static_cast<char*>(out);
  a.lse = out_lse;
  a.status = out_status;
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (args->cache.dtype == SD_BF16)
    launch<SD_BF16>(a, args->cache.D, st);
  else
    launch<SD_F16>(a, args->cache.D, st);
  if (hipGetLastError() != hipSuccess) return SD_EHIP;
  if (out_status) {
    hipLaunchKernelGGL(k_tree_status, dim3(a.c.B), dim3(WAVE), 0, st, a);
    if (hipGetLastError() != hipSuccess) return SD_EHIP;
  }
  return SD_OK;
}
