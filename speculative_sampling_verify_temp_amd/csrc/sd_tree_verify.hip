// Greedy verify of a drafted tree on gfx950.
//
// Bound by the bytes of logits read.  Which rows the walk visits is known one
// row at a time, so there are two ways (rule at walk_rows):
//   few rows in all    k_tree_argmax finds the maximum of every row, a
//                      workgroup per (row, slice of the vocabulary), and
//                      k_tree_walk, one wave per request, follows the tree;
//   many rows          k_tree_descend, one workgroup per request, reads only
//                      the rows that its walk visits, one after another.
//
// The scan of a row takes 1.5 operations a bf16 logit (Extremes).  A thread
// only keeps which group of its vectors holds its maximum; the token is looked
// up afterwards by the threads that hold the row's.
#include <algorithm>

#include "sdt_device.h"

using namespace sdv;
using namespace sdt;

namespace {

constexpr int NT_A = 256;    // threads of a (row, slice)
constexpr int NT_D = 1024;   // threads of a walk that reads its own rows
constexpr int UD = 19;       // vectors a thread of such a walk loads at once: 155648 bf16 logits

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

// Lowest id in the thread's UG vectors of a group at k0 whose logit is z, or -1.
template <int DT, int NT, int UG>
__device__ __forceinline__ int find_in(const uint4 (&w)[UG], int k0, int last, float z) {
  constexpr int E = DT == SD_BF16 ? 8 : 4;
  int id = -1;
#pragma unroll
  for (int u = UG - 1; u >= 0; --u) {
    const int k = min(k0 + u * NT + (int)threadIdx.x, last);
    const uint32_t q[4] = {w[u].x, w[u].y, w[u].z, w[u].w};
#pragma unroll
    for (int e = E - 1; e >= 0; --e) {
      const float y = DT == SD_BF16 ? __uint_as_float(e & 1 ? q[e / 2] & 0xFFFF0000u : q[e / 2] << 16)
                                    : __uint_as_float(q[e]);
      if (y == z) id = k * E + e;
    }
  }
  return id;
}

template <int NT, int UG>
__device__ __forceinline__ void load_group(const uint4* row, int k0, int last, uint4 (&w)[UG]) {
#pragma unroll
  for (int u = 0; u < UG; ++u) w[u] = row[min(k0 + u * NT + (int)threadIdx.x, last)];
}

// The maximum of the whole vectors [lo, hi) of a row, and of its last V % E
// logits if `tail`, with its lowest id, as arg_key, in every thread.  Threads
// past the end read the last vector again, which changes no maximum.
// sm: 2 NT / WAVE words.
template <int DT, int NT, int UG>
__device__ uint64_t row_best(const char* p, int lo, int hi, int V, bool tail, uint64_t* sm) {
  constexpr int E = DT == SD_BF16 ? 8 : 4;
  const uint4* const row = reinterpret_cast<const uint4*>(p);
  const int tid = threadIdx.x, last = hi - 1;
  float best = -INFINITY;
  int at = -1;                  // first vector of the group that holds it, -2: the tail
  bool nan = false;
  uint4 w[UG];
  for (int k0 = lo; k0 < hi; k0 += NT * UG) {
    load_group<NT, UG>(row, k0, last, w);
    Extremes<DT> x;
    x.clear();
#pragma unroll
    for (int u = 0; u < UG; ++u) {
      x.add(w[u].x);
      x.add(w[u].y);
      x.add(w[u].z);
      x.add(w[u].w);
    }
    const float z = x.value(nan);
    if (z > best || at < 0) best = z, at = k0;
  }
  if (tail && tid < V % E) {
    const float z = to_float<DT>(p, V - V % E + tid);
    nan |= z != z;
    if (z > best || at < 0) best = z, at = -2;
  }
  uint64_t key = at == -1 ? 0 : arg_key(nan ? __builtin_nanf("") : best, 0) & ~0xFFFFFFFFull;
  uint64_t top = wave_max_u64(key);
  if (tid % WAVE == 0) sm[tid / WAVE] = top;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < NT / WAVE; ++i) top = sm[i] > top ? sm[i] : top;
  // the holders of the maximum find its first place in their group, which is
  // still in registers if the row has only one
  key = key == top ? key : 0;
  if (key && !nan) {
    int id;
    if (at == -2) {
      id = V - V % E + tid;
    } else {
      if (hi - lo > NT * UG) load_group<NT, UG>(row, at, last, w);
      id = find_in<DT, NT, UG>(w, at, last, best);
    }
    key = top | (uint32_t)~id;
  }
  key = wave_max_u64(key);
  sm += NT / WAVE;
  if (tid % WAVE == 0) sm[tid / WAVE] = key;
  __syncthreads();
  key = 0;
#pragma unroll
  for (int i = 0; i < NT / WAVE; ++i) key = sm[i] > key ? sm[i] : key;
  return key;
}

template <int DT>
__global__ __launch_bounds__(NT_A) void k_tree_argmax(VerifyArgs a) {
  constexpr int E = DT == SD_BF16 ? 8 : 4;
  __shared__ uint64_t sm[2 * NT_A / WAVE];
  const int row = blockIdx.x, sl = blockIdx.y;
  const int lo = sl * a.slice_vecs, hi = min(a.V / E, lo + a.slice_vecs);
  const uint64_t best = row_best<DT, NT_A, 4>(a.logits + row * a.row_bytes, lo, hi, a.V, sl == a.slices - 1, sm);
  if (threadIdx.x == 0) a.part[(int64_t)row * a.slices + sl] = best;
}

// The tree of one request in the lanes of a wave: lane l holds node l.
struct Walk {
  Nodes nd;
  uint32_t st;
  int tok, up;
  int cur = 0, count = 0, my_path = -1, my_tok = -1;

  __device__ Walk(const VerifyArgs& a, int b) {
    const int l = threadIdx.x % WAVE;
    nd = request_nodes(a.off, b, a.N, a.max_nodes);
    st = nd.T > 0 ? nd.st : SD_ST_BAD_NODES;
    tok = l < nd.T ? a.tokens[nd.first + l] : -1;
    up = l < nd.T ? a.parents[nd.first + l] : -1;
    const bool bad = up < -1 || up >= l;
    if (bad || l == 0) up = -1;
    if (__any(bad && l < nd.T)) st |= SD_ST_BAD_TREE;
    if (__any(l > 0 && l < nd.T && (tok < 0 || tok >= a.V))) st |= SD_ST_BAD_DRAFT_ID;
  }
  __device__ bool valid() const { return !(st & SD_ST_TREE_INVALID_MASK); }
  // Enter the current node; false if its row is not needed.
  __device__ bool enter(uint32_t flags) {
    if ((int)(threadIdx.x % WAVE) == count) my_path = cur;
    return !((flags & SD_NO_BONUS) && __ballot(up == cur) == 0);
  }
  // Take its row's maximum; false at the walk's end.  Each step goes to a
  // higher node: at most T of them.
  __device__ bool step(uint64_t best) {
    if ((uint32_t)(best >> 32) == 0xFFFFFFFFu) {
      st |= SD_ST_NONFINITE;
      return false;
    }
    const int win = (int)~(uint32_t)best;
    if ((int)(threadIdx.x % WAVE) == count) my_tok = win;
    const uint64_t next = __ballot(up == cur && tok == win);
    if (next == 0) return false;
    cur = __builtin_ctzll(next);
    ++count;
    return true;
  }
  __device__ void write(const VerifyArgs& a, int b) const {
    const int l = threadIdx.x % WAVE;
    const bool bad = !valid();
    if (l < a.max_nodes) {
      a.path[(int64_t)b * a.max_nodes + l] = bad ? -1 : my_path;
      a.out_tokens[(int64_t)b * a.max_nodes + l] = bad ? -1 : my_tok;
    }
    if (l == 0) {
      a.accepted[b] = bad ? -1 : count;
      if (a.status) a.status[b] = st;
    }
  }
};

__global__ __launch_bounds__(WAVE) void k_tree_walk(VerifyArgs a) {
  const int b = blockIdx.x, l = threadIdx.x;
  Walk w(a, b);
  while (w.valid() && w.enter(a.flags)) {
    uint64_t best = 0;
    for (int s = l; s < a.slices; s += WAVE) {
      const uint64_t k = a.part[(int64_t)(w.nd.first + w.cur) * a.slices + s];
      best = k > best ? k : best;
    }
    if (!w.step(wave_max_u64(best))) break;
  }
  w.write(a, b);
}

template <int DT>
__global__ __launch_bounds__(NT_D) void k_tree_descend(VerifyArgs a) {
  constexpr int E = DT == SD_BF16 ? 8 : 4;
  __shared__ uint64_t sm[2 * NT_D / WAVE];
  const int b = blockIdx.x;
  Walk w(a, b);      // every wave walks along
  while (w.valid() && w.enter(a.flags)) {
    const char* row = a.logits + (int64_t)(w.nd.first + w.cur) * a.row_bytes;
    if (!w.step(row_best<DT, NT_D, UD>(row, 0, a.V / E, a.V, true, sm))) break;
  }
  if (threadIdx.x < WAVE) w.write(a, b);
}

int check(const sd_tree_verify_args_t* p) {
  if (!p || !p->logits || !aligned16(p->logits) || !p->tokens || !p->parents || !p->node_offsets)
    return SD_EINVAL;
  if (p->dtype != SD_F32 && p->dtype != SD_BF16) return SD_EINVAL;
  const int es = p->dtype == SD_BF16 ? 2 : 4;
  if (p->B < 1 || p->N < 1 || p->V < 1 || p->max_nodes < 1 || p->ld < p->V || (p->ld * es) % 16 ||
      (p->flags & ~(uint32_t)SD_NO_BONUS))
    return SD_EINVAL;
  if (p->max_nodes > SD_MAX_NODES || p->V >= (1 << 28) || p->N > (1 << 24)) return SD_EUNSUPPORTED;
  return SD_OK;
}

// Vocabulary slices of a row: enough workgroups for the chip, none below 512
// vectors.
int slice_count(int N, int nvec) {
  return std::max(1, std::min({(2048 + N - 1) / N, (nvec + 511) / 512, 64}));
}

// Whether to read only the rows that the walks visit.  One workgroup reads a
// row at about 70 GB/s, a full chip at about 4.5 TB/s, and a step of a walk
// costs about 2 us beside its bytes: reading all N rows takes longer than a walk
// of d + 1 rows when N > (d + 1) (64 + 9 MB / row).  Walks are rarely deeper than
// 16 (a deeper one costs at most four times what reading all rows would).
bool walk_rows(const sd_tree_verify_args_t* p) {
  const int64_t row = (int64_t)p->V * (p->dtype == SD_BF16 ? 2 : 4);
  return p->N * row > std::min(p->max_nodes, 16) * (64 * row + (9 << 20));
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
  if (walk_rows(args)) {
    if (args->dtype == SD_BF16)
      hipLaunchKernelGGL(k_tree_descend<SD_BF16>, dim3(a.B), dim3(NT_D), 0, st, a);
    else
      hipLaunchKernelGGL(k_tree_descend<SD_F32>, dim3(a.B), dim3(NT_D), 0, st, a);
    return hipGetLastError() == hipSuccess ? SD_OK : SD_EHIP;
  }
  if (args->dtype == SD_BF16)
    hipLaunchKernelGGL(k_tree_argmax<SD_BF16>, dim3(a.N, a.slices), dim3(NT_A), 0, st, a);
  else
    hipLaunchKernelGGL(k_tree_argmax<SD_F32>, dim3(a.N, a.slices), dim3(NT_A), 0, st, a);
  if (hipGetLastError() != hipSuccess) return SD_EHIP;
  hipLaunchKernelGGL(k_tree_walk, dim3(a.B), dim3(WAVE), 0, st, a);
  return hipGetLastError() == hipSuccess ? SD_OK : SD_EHIP;
}
