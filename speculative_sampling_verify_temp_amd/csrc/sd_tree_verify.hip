// Greedy verify of a drafted tree on gfx950.
//
// Two launches on the caller's stream:
//   k_tree_argmax  one workgroup per (node row, slice of the vocabulary): the
//                  slice's maximum and its lowest id as one 64-bit key;
//   k_tree_walk    one wave per request: from the root, the row's maximum
//                  over the slices, then the first child with that token.
#include <algorithm>

#include "sdt_device.h"

using namespace sdv;
using namespace sdt;

namespace {

constexpr int NT_A = 256;

struct VerifyArgs {
  const char* logits;
  int64_t row_bytes;
  const int32_t *tokens, *parents, *off;
  int B, N, V, max_nodes;
  uint32_t flags;
  int slices, slice_vecs;   // 16-byte vectors of a slice
  uint64_t* part;           // [N][slices]
  int32_t *accepted, *path, *out_tokens;
  uint32_t* status;
};

// Larger logit, then lower id, as the larger key; a NaN above everything.
__device__ __forceinline__ uint64_t arg_key(float z, int id) {
  const uint32_t o = z != z ? 0xFFFFFFFFu : ord_key(z);
  return ((uint64_t)o << 32) | (uint32_t)~id;
}

__device__ __forceinline__ uint64_t wave_max_u64(uint64_t x) {
#pragma unroll
  for (int o = WAVE / 2; o > 0; o >>= 1) {
    const uint64_t y = __shfl_xor(x, o);
    x = y > x ? y : x;
  }
  return x;
}

template <int DT>
__global__ __launch_bounds__(NT_A) void k_tree_argmax(VerifyArgs a) {
  constexpr int E = DT == SD_BF16 ? 8 : 4;
  __shared__ uint64_t sm[NT_A / WAVE];
  const int row = blockIdx.x, sl = blockIdx.y, tid = threadIdx.x;
  const char* p = a.logits + row * a.row_bytes;
  const int nvec = (a.V + E - 1) / E;
  const int lo = sl * a.slice_vecs, hi = min(nvec, lo + a.slice_vecs);
  uint64_t best = 0;
  for (int k = lo + tid; k < hi; k += NT_A) {
    const uint4 w = reinterpret_cast<const uint4*>(p)[k];
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const float z = DT == SD_BF16 ? __uint_as_float(e & 1 ? u[e / 2] & 0xFFFF0000u : u[e / 2] << 16)
                                    : __uint_as_float(u[e]);
      const int id = k * E + e;
      if (id < a.V) {
        const uint64_t key = arg_key(z, id);
        best = key > best ? key : best;
      }
    }
  }
  best = wave_max_u64(best);
  if (tid % WAVE == 0) sm[tid / WAVE] = best;
  __syncthreads();
  if (tid == 0) {
    for (int w = 1; w < NT_A / WAVE; ++w) best = sm[w] > best ? sm[w] : best;
    a.part[(int64_t)row * a.slices + sl] = best;
  }
}

__global__ __launch_bounds__(WAVE) void k_tree_walk(VerifyArgs a) {
  const int b = blockIdx.x, l = threadIdx.x;
  const Nodes nd = request_nodes(a.off, b, a.N, a.max_nodes);
  uint32_t st = nd.T > 0 ? nd.st : SD_ST_BAD_NODES;
  const int tok = l < nd.T ? a.tokens[nd.first + l] : -1;
  int up = l < nd.T && l > 0 ? a.parents[nd.first + l] : -1;
  bool bad_tree = l < nd.T && (l > 0 ? up < -1 || up >= l : a.parents[nd.first] < -1 || a.parents[nd.first] >= 0);
  if (up < -1 || up >= l) up = -1;
  if (__any(bad_tree)) st |= SD_ST_BAD_TREE;
  if (__any(l > 0 && l < nd.T && (tok < 0 || tok >= a.V))) st |= SD_ST_BAD_DRAFT_ID;
  int cur = 0, count = 0, my_path = -1, my_tok = -1;
  if (!(st & SD_ST_TREE_INVALID_MASK)) {
    for (;;) {      // each step goes to a higher node: at most T steps
      const uint64_t kids = __ballot(up == cur);
      if (l == count) my_path = cur;
      if ((a.flags & SD_NO_BONUS) && kids == 0) break;
      uint64_t best = 0;
      for (int s = l; s < a.slices; s += WAVE) {
        const uint64_t k = a.part[(int64_t)(nd.first + cur) * a.slices + s];
        best = k > best ? k : best;
      }
      best = wave_max_u64(best);
      if ((uint32_t)(best >> 32) == 0xFFFFFFFFu) {
        st |= SD_ST_NONFINITE;
        break;
      }
      const int win = (int)~(uint32_t)best;
      if (l == count) my_tok = win;
      const uint64_t next = __ballot(up == cur && tok == win);
      if (next == 0) break;
      cur = __builtin_ctzll(next);
      ++count;
    }
  }
  const bool bad = st & SD_ST_TREE_INVALID_MASK;
  if (l < a.max_nodes) {
    a.path[(int64_t)b * a.max_nodes + l] = bad ? -1 : my_path;
    a.out_tokens[(int64_t)b * a.max_nodes + l] = bad ? -1 : my_tok;
  }
  if (l == 0) {
    a.accepted[b] = bad ? -1 : count;
    if (a.status) a.status[b] = st;
  }
}

int check(const sd_tree_verify_args_t* p) {
  if (!p || !p->logits || !aligned16(p->logits) || !p->tokens || !p->parents || !p->node_offsets)
    return SD_EINVAL;
  if (p->dtype != SD_F32 && p->dtype != SD_BF16) return SD_EINVAL;
  const int es = p->dtype == SD_BF16 ? 2 : 4;
  if (p->B < 1 || p->N < 1 || p->V < 1 || p->max_nodes < 1 || p->ld < p->V || (p->ld * es) % 16 ||
      (p->flags & ~(uint32_t)SD_NO_BONUS))
    return SD_EINVAL;
  if (p->max_nodes > SD_MAX_NODES || p->V >= (1 << 30) || p->N > (1 << 24)) return SD_EUNSUPPORTED;
  return SD_OK;
}

// Vocabulary slices of a row: enough workgroups for the chip, none below 512
// vectors.
int slice_count(int N, int nvec) {
  return std::max(1, std::min({(2048 + N - 1) / N, (nvec + 511) / 512, 64}));
}

}  // namespace

extern "C" int sd_tree_verify_workspace_bytes(const sd_tree_verify_args_t* args, size_t* bytes) {
  if (!bytes) return SD_EINVAL;
  const int rc = check(args);
  if (rc) return rc;
  const int E = args->dtype == SD_BF16 ? 8 : 4;
  *bytes = (size_t)args->N * slice_count(args->N, (args->V + E - 1) / E) * 8;
  return SD_OK;
}

extern "C" int sd_tree_verify_greedy(const sd_tree_verify_args_t* args, void* workspace,
                                     size_t workspace_bytes, int32_t* out_accepted,
                                     int32_t* out_path, int32_t* out_tokens,
                                     uint32_t* out_status, void* stream) {
  size_t need = 0;
  const int rc = sd_tree_verify_workspace_bytes(args, &need);
  if (rc) return rc;
  if (!out_accepted || !out_path || !out_tokens) return SD_EINVAL;
  if (!workspace || workspace_bytes < need || (uintptr_t)workspace % 8) return SD_EWORKSPACE;
  const int E = args->dtype == SD_BF16 ? 8 : 4, nvec = (args->V + E - 1) / E;
  VerifyArgs a;
  a.logits = static_cast<const char*>(args->logits);
  a.row_bytes = args->ld * (16 / E);
  a.tokens = args->tokens, a.parents = args->parents, a.off = args->node_offsets;
  a.B = args->B, a.N = args->N, a.V = args->V, a.max_nodes = args->max_nodes;
  a.flags = args->flags;
  a.slices = slice_count(a.N, nvec);
  a.slice_vecs = (nvec + a.slices - 1) / a.slices;
  a.part = static_cast<uint64_t*>(workspace);
  a.accepted = out_accepted, a.path = out_path, a.out_tokens = out_tokens, a.status = out_status;
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (args->dtype == SD_BF16)
    hipLaunchKernelGGL(k_tree_argmax<SD_BF16>, dim3(a.N, a.slices), dim3(NT_A), 0, st, a);
  else
    hipLaunchKernelGGL(k_tree_argmax<SD_F32>, dim3(a.N, a.slices), dim3(NT_A), 0, st, a);
  if (hipGetLastError() != hipSuccess) return SD_EHIP;
  hipLaunchKernelGGL(k_tree_walk, dim3(a.B), dim3(WAVE), 0, st, a);
  return hipGetLastError() == hipSuccess ? SD_OK : SD_EHIP;
}
