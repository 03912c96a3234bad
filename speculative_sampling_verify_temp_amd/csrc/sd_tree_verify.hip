// Greedy verify of a drafted tree on gfx950.
//
// Bound by the bytes of logits read.  Which rows the walk visits is known one
// row at a time, so there are two ways (rule at walk_rows):
//   few rows in all    (one tree of 16 rows of 151936 fp32 logits: 4.6 + 4.3
//                      us, latency) k_tree_argmax finds the maximum of every row, a
//                      workgroup per (row, slice of the vocabulary), and
//                      k_tree_walk, one wave per request, follows the tree;
//   many rows          k_tree_descend reads only the rows that the walks visit,
//                      one after another, each by a team of workgroups.
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
constexpr int NT_D = 512;    // threads of a workgroup of a team
constexpr int UD = 8;        // vectors a thread of a team loads at once

struct Team;

struct VerifyArgs {
  const char* logits;
  int64_t row_bytes;
  const int32_t *tokens, *parents, *off;
  int B, N, V, max_nodes;
  uint32_t flags;
  int slices, slice_vecs;   // 16-byte vectors of a slice
  int polls;                // looks at a row that is waited for
  uint64_t* part;           // [N][slices] ([B][slices] where walks read their rows)
  Team* team;               // [B], there
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

// ---- walks that read their own rows ----
//
// One workgroup reads a row from HBM at about 30 GB/s, so a team of `slices` of
// them shares each row of a request's walk.  They meet through tickets: ticket
// k of a request is slice k % slices of its row number k / slices.  A workgroup
// takes the next ticket, waits until that row is known, leaves its slice's
// maximum, and the last one of a row to do so takes the step and makes the
// next row known.  A ticket is only waited for by later ones, and whoever holds
// an earlier one is running, so every wait ends however few workgroups of a
// team the chip holds at a time.  (Calls that overlap on one workspace, which
// the interface forbids, could take each other's tickets: waits are bounded, and
// such a request keeps the -1 and SD_ST_UNFINISHED that its results begin with.)
//
// What the team shares is only touched by relaxed agent-scope atomics, which
// act where all of the chip's caches meet; a wait for the ones before stands
// where order matters.  (Acquire and release operations would also write back
// and invalidate whole L2 caches: 14 us a step instead of 6.)

struct Team {
  uint32_t ticket, left, row, pad;          // row: depth << 8 | node, or DONE
  uint64_t visited[SD_MAX_NODES];           // by depth: node << 32 | its row's best token
};
constexpr uint32_t DONE = 0xFFFFFFFFu;
constexpr int MAX_POLLS = 1 << 21;          // about two seconds; a wait takes microseconds

template <typename T>
__device__ __forceinline__ T shared_load(const T* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
template <typename T>
__device__ __forceinline__ void shared_store(T* p, T v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ uint32_t shared_add(uint32_t* p) {
  return __hip_atomic_fetch_add(p, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
// All memory operations of this wave before are done, and none after begun.
__device__ __forceinline__ void settle() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0);
  asm volatile("" ::: "memory");
}

// Results of a walk that has ended, by one wave; the entries of lane l.
__device__ __forceinline__ void finish(const VerifyArgs& a, int b, uint32_t st, int accepted, int path, int tok) {
  const int l = threadIdx.x % WAVE;
  const bool bad = st & SD_ST_TREE_INVALID_MASK;
  if (l < a.max_nodes) {
    a.path[(int64_t)b * a.max_nodes + l] = bad ? -1 : path;
    a.out_tokens[(int64_t)b * a.max_nodes + l] = bad ? -1 : tok;
  }
  if (l == 0) {
    a.accepted[b] = bad ? -1 : accepted;
    if (a.status) a.status[b] = st;
  }
}

// Requests as their walks begin, one wave each.
__global__ __launch_bounds__(WAVE) void k_tree_begin(VerifyArgs a) {
  const int b = blockIdx.x, l = threadIdx.x;
  Walk w(a, b);
  const bool go = w.valid() && w.enter(a.flags);
  finish(a, b, w.st | (go ? SD_ST_UNFINISHED : 0u), 0, w.my_path, -1);
  if (l == 0) {
    Team& t = a.team[b];
    t.ticket = t.left = 0;
    t.row = go ? 0 : DONE;
  }
}

template <int DT>
__global__ __launch_bounds__(NT_D) void k_tree_descend(VerifyArgs a) {
  constexpr int E = DT == SD_BF16 ? 8 : 4;
  __shared__ uint64_t sm[2 * NT_D / WAVE];
  __shared__ uint32_t ticket_sh, row_sh, last_sh;
  const int b = blockIdx.y, tid = threadIdx.x, l = tid % WAVE;
  Team& team = a.team[b];
  uint64_t* const part = a.part + (int64_t)b * a.slices;
  uint32_t next = tid == 0 ? shared_add(&team.ticket) : 0;
  Walk w(a, b);
  for (;;) {
    if (tid == 0) {
      const uint32_t depth = next / (uint32_t)a.slices;
      uint32_t r = DONE;
      for (int i = 0; i < a.polls; ++i) {
        r = shared_load(&team.row);
        if (r == DONE || (r >> 8) >= depth) break;
        r = DONE;
        __builtin_amdgcn_s_sleep(1);
      }
      ticket_sh = next, row_sh = r;
    }
    __syncthreads();
    if (row_sh == DONE) return;
    const int sl = (int)(ticket_sh % (uint32_t)a.slices), depth = (int)(row_sh >> 8) & 63, cur = min((int)(row_sh & 63u), w.nd.T - 1);
    if (tid == 0) next = shared_add(&team.ticket);      // on its way while the row is read
    const int lo = sl * a.slice_vecs, hi = min(a.V / E, lo + a.slice_vecs);
    const char* row = a.logits + (int64_t)(w.nd.first + cur) * a.row_bytes;
    const uint64_t mine = row_best<DT, NT_D, UD>(row, lo, hi, a.V, sl == a.slices - 1, sm);
    if (tid == 0) {
      shared_store(&part[sl], mine);
      settle();
      last_sh = shared_add(&team.left) == (uint32_t)((depth + 1) * a.slices - 1);
    }
    __syncthreads();
    if (last_sh && tid < WAVE) {
      settle();
      uint64_t best = 0;
      for (int s = l; s < a.slices; s += WAVE) {
        const uint64_t k = shared_load(&part[s]);
        best = k > best ? k : best;
      }
      best = wave_max_u64(best);
      if (l == 0) shared_store(&team.visited[depth], (uint64_t)cur << 32 | (uint32_t)~(uint32_t)best);
      w.cur = cur, w.count = depth;
      const bool on = w.step(best);
      const bool more = on && w.enter(a.flags);
      settle();
      if (!more) {
        // (a node entered last without its row has no entry there)
        const int rows = on ? w.count : depth + 1;
        const uint64_t v = l < rows ? shared_load(&team.visited[l]) : 0;
        finish(a, b, w.st, w.count, l < rows ? (int)(v >> 32) : l == w.count ? w.cur : -1, l < rows ? (int)(uint32_t)v : -1);
      }
      if (l == 0) shared_store(&team.row, more ? (uint32_t)w.count << 8 | (uint32_t)w.cur : DONE);
    }
    __syncthreads();
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
  if (p->max_nodes > SD_MAX_NODES || p->V >= (1 << 28) || p->B > 65535) return SD_EUNSUPPORTED;
  // a grid dimension holds less than 2^32 threads
  if ((int64_t)p->N * NT_A > UINT32_MAX) return SD_EUNSUPPORTED;
  return SD_OK;
}

// Whether to read only the rows that the walks visit.  A step of that takes
// about 5.5 us (64 requests, 152064 bf16 logits); reading every row, at about
// 4.5 TB/s, is the shorter way where it takes no longer than half of the steps of
// a walk of max_nodes, or of 16, which walks are rarely longer than: 12 MB a step.
// (64 trees of 64 nodes: 215 us for all rows, 41 us for walks of up to 7.)
bool walk_rows(const sd_tree_verify_args_t* p) {
  const int64_t row = (int64_t)p->V * (p->dtype == SD_BF16 ? 2 : 4);
  return p->N * row > std::min(p->max_nodes, 16) * (int64_t)(12 << 20);
}

// Workgroups a row is shared by, and the 16-byte vectors of each.
struct Slices {
  int count, vecs;
  bool walk;
};

Slices slices_of(const sd_tree_verify_args_t* p) {
  const int E = p->dtype == SD_BF16 ? 8 : 4, nvec = (p->V + E - 1) / E;
  Slices s;
  s.walk = walk_rows(p);
  // all rows: about 2048 workgroups; walks: about two a CU.  None below 512 vectors.
  const int rows = s.walk ? p->B : p->N, want = s.walk ? 512 : 2048;
  s.count = std::max(1, std::min({(want + rows - 1) / rows, (nvec + 511) / 512, 64}));
  s.vecs = (nvec + s.count - 1) / s.count;
  return s;
}

size_t parts_bytes(const sd_tree_verify_args_t* p, const Slices& s) {
  return ((size_t)(s.walk ? p->B : p->N) * s.count * 8 + 63) & ~(size_t)63;
}

}  // namespace

extern "C" int sd_tree_verify_workspace_bytes(const sd_tree_verify_args_t* args, size_t* bytes) {
  if (!bytes) return SD_EINVAL;
  const int rc = check(args);
  if (rc) return rc;
  const Slices s = slices_of(args);
  *bytes = parts_bytes(args, s) + (s.walk ? (size_t)args->B * sizeof(Team) : 0);
  return SD_OK;
}

extern "C" int sd_tree_verify_greedy(const sd_tree_verify_args_t* args, void* workspace,
                                     size_t workspace_bytes, int32_t* out_accepted,
                                     int32_t* out_path, int32_t* out_tokens,
                                     uint32_t* out_status, void* stream) {
  return sd_debug_tree_verify_polls(args, workspace, workspace_bytes, out_accepted, out_path, out_tokens,
                                    out_status, MAX_POLLS, stream);
}

extern "C" int sd_debug_tree_verify_polls(const sd_tree_verify_args_t* args, void* workspace,
                                          size_t workspace_bytes, int32_t* out_accepted,
                                          int32_t* out_path, int32_t* out_tokens,
                                          uint32_t* out_status, int32_t polls, void* stream) {
  size_t need = 0;
  const int rc = sd_tree_verify_workspace_bytes(args, &need);
  if (rc) return rc;
  if (!out_accepted || !out_path || !out_tokens) return SD_EINVAL;
  for (const int32_t* in : {args->tokens, args->parents, args->node_offsets})
    if (out_accepted == in || out_path == in || out_tokens == in) return SD_EINVAL;
  if (!workspace || workspace_bytes < need || (uintptr_t)workspace % 8) return SD_EWORKSPACE;
  const Slices s = slices_of(args);
  VerifyArgs a;
  a.logits = static_cast<const char*>(args->logits);
  a.row_bytes = args->ld * (args->dtype == SD_BF16 ? 2 : 4);
  a.tokens = args->tokens, a.parents = args->parents, a.off = args->node_offsets;
  a.B = args->B, a.N = args->N, a.V = args->V, a.max_nodes = args->max_nodes;
  a.flags = args->flags;
  a.slices = s.count, a.slice_vecs = s.vecs;
  a.polls = polls;
  a.part = static_cast<uint64_t*>(workspace);
  a.team = reinterpret_cast<Team*>(static_cast<char*>(workspace) + parts_bytes(args, s));
  a.accepted = out_accepted, a.path = out_path, a.out_tokens = out_tokens, a.status = out_status;
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (s.walk) {
    hipLaunchKernelGGL(k_tree_begin, dim3(a.B), dim3(WAVE), 0, st, a);
    if (hipGetLastError() != hipSuccess) return SD_EHIP;
    if (args->dtype == SD_BF16)
      hipLaunchKernelGGL(k_tree_descend<SD_BF16>, dim3(a.slices, a.B), dim3(NT_D), 0, st, a);
    else
      hipLaunchKernelGGL(k_tree_descend<SD_F32>, dim3(a.slices, a.B), dim3(NT_D), 0, st, a);
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
