// Verify of a drafted tree against probabilities on gfx950.
//
// The walk tests a node's children in order.  What a test needs, p and q of the
// child's token in its parent's rows, is known for every node before the walk
// begins: lane l of a wave loads those of node l, and accepted children cost
// nothing more.  Only a rejection needs whole rows: Z, the sum of max(p - cut q, 0),
// and after the last one the draw, whose total is the last Z.
//
// So a request makes one pass over the rows of a node for each rejection on its
// walk, and one for the draw where nothing was rejected at its last node.  Bound
// by those rows' bytes in large batches, by a pass's latency in small ones.
//
// k_sample_begin    one wave per request: the walk up to its first pass.
// k_sample_passes   teams of workgroups make the passes, one slice of the
//                   vocabulary each; every wave leaves the sum of its own
//                   stretch.  The last workgroup of a pass to do so goes on with
//                   the walk, and at its end finds the stretch and the token that
//                   the draw falls on.
//
// Teams meet through tickets: ticket k of a request is slice k % slices of its
// pass number k / slices.  A ticket is only waited for by later ones, and whoever
// holds an earlier one is running, so every wait ends however few workgroups of a
// team the chip holds at a time.  (Calls that overlap on one workspace, which the
// interface forbids, could take each other's tickets: waits are bounded, and such a
// request keeps the -1 and SD_ST_UNFINISHED that its results begin with.)  What a
// team shares is only touched by relaxed agent-scope atomics, with a wait for the
// ones before where order matters.
#include <algorithm>

#include "sd_serve.h"
#include "sdt_device.h"

using namespace sdv;
using namespace sdt;

namespace {

constexpr int NT = 512;               // threads of a workgroup
constexpr int WV = NT / WAVE;
constexpr int US = 4;                 // vectors of each row that a lane loads at once
constexpr uint32_t DONE = 0xFFFFFFFFu;
constexpr int MAX_POLLS = 1 << 21;    // about two seconds; a wait takes microseconds

// Where a walk stands, and what its next pass sums up.
struct Team {
  uint32_t ticket, left, pass, place;       // pass: its number, or DONE; place: count << 16 | next child << 8 | node
  double cut, Z, gone;
  uint32_t mode, st;
  uint8_t path[SD_MAX_NODES];
};
enum : uint32_t { RESIDUAL, PLAIN };        // max(p - cut q, 0), or p without the rejected tokens

struct SampleArgs {
  const float *p, *q;
  int64_t ld_p, ld_q;
  const int32_t *tokens, *parents, *off;
  const float *u, *v;
  int B, N, V, Vd, max_nodes;
  uint32_t flags;
  int slices, stretch;      // stretch: vectors of 4 that a wave sums up
  int polls;
  double* part;             // [B][slices * WV]
  Team* team;               // [B]
  int32_t *accepted, *path, *out_tokens;
  uint32_t* status;
};

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

__device__ __forceinline__ bool bad_prob(double x) { return !(x >= 0.0 && x < INFINITY); }

// A request's tree and walk in a wave: lane l holds node l.
struct Walk {
  Nodes nd;
  uint32_t st;
  int tok, up;
  double px, qx, u;      // of the lane's token in its parent's rows
  int cur = 0, child = 0, count = 0, my_path = -1;
  double cut = 0.0, Z = 1.0, gone = 0.0;
  uint32_t mode;

  // mine: whether this wave is the one that walks.
  __device__ Walk(const SampleArgs& a, int b, bool mine) {
    const int l = threadIdx.x % WAVE;
    nd = request_nodes(a.off, b, a.N, a.max_nodes);
    st = nd.T > 0 ? nd.st : SD_ST_BAD_NODES;
    tok = l < nd.T ? a.tokens[nd.first + l] : -1;
    up = l < nd.T ? a.parents[nd.first + l] : -1;
    const float uf = l < nd.T && l > 0 ? a.u[nd.first + l] : 0.0f;
    const bool bad = up < -1 || up >= l;
    if (bad || l == 0) up = -1;
    if (__any(bad && l < nd.T)) st |= SD_ST_BAD_TREE;
    if (__any(l > 0 && l < nd.T && (tok < 0 || tok >= a.V))) st |= SD_ST_BAD_DRAFT_ID;
    mode = a.q ? RESIDUAL : PLAIN;
    px = qx = 0.0;
    u = uf;
    if (mine && valid() && up >= 0) {
      const int64_t row = nd.first + up;
      px = a.p[row * a.ld_p + tok];
      if (a.q && tok < a.Vd) qx = a.q[row * a.ld_q + tok];
    }
    if (l == 0) my_path = 0;
  }
  __device__ bool valid() const { return !(st & SD_ST_TREE_INVALID_MASK); }

  // Tests children until a pass is needed (true) or the walk is over without one.
  // Each step takes or rejects a node past all before it: at most T of them.
  __device__ bool advance(const SampleArgs& a) {
    const int l = threadIdx.x % WAVE;
    for (;;) {
      const uint64_t kids = __ballot(up == cur && l >= child);
      if (!kids) {
        // the walk ends here; where nothing was rejected the row is still to be summed up
        if ((a.flags & SD_NO_BONUS) && __ballot(up == cur) == 0) return false;
        mode = PLAIN;
        return true;
      }
      const int i = __builtin_ctzll(kids);
      const double x = lane_read(px, i), y = lane_read(qx, i), r = lane_read(u, i);
      const int t = __builtin_amdgcn_readlane(tok, i);
      if (!(r >= 0.0 && r < 1.0)) st |= SD_ST_BAD_PARAM;
      if (bad_prob(x) || bad_prob(y)) st |= SD_ST_NONFINITE;
      if (!valid()) return false;
      bool take;
      double rate = 1.0;
      if (a.q) {
        const double left = 1.0 - gone;
        if (a.flags & SD_NO_REPLACEMENT) rate = left > 0.0 ? 1.0 / left : 0.0;
        if (y == 0.0) st |= SD_ST_Q_ZERO;
        take = r * (y * rate) * Z < fmax(x - cut * y, 0.0);
      } else {
        // a token that was rejected here before has p = 0
        const bool again = __any(up == cur && l < child && tok == t);
        take = !again && r * Z < x;
        if (!take && !again) Z -= x;
      }
      if (take) {
        cur = i, child = 0, ++count;
        cut = 0.0, Z = 1.0, gone = 0.0;
        if (l == count) my_path = i;
        continue;
      }
      child = i + 1;
      if (a.q) {
        gone += y;
        cut += Z * rate;
        mode = RESIDUAL;
        return true;
      }
    }
  }

  // Results: the path in the lanes, the token drawn (-1: none).
  __device__ void write(const SampleArgs& a, int b, int drawn) const {
    const int l = threadIdx.x % WAVE;
    const bool bad = !valid();
    // token of the node after this one on the path
    const int next = __shfl(my_path, min(l + 1, WAVE - 1));
    int t = __shfl(tok, max(next, 0));
    t = l < count ? t : l == count ? drawn : -1;
    if (l < a.max_nodes) {
      a.path[(int64_t)b * a.max_nodes + l] = bad || l > count ? -1 : my_path;
      a.out_tokens[(int64_t)b * a.max_nodes + l] = bad ? -1 : t;
    }
    if (l == 0) {
      a.accepted[b] = bad ? -1 : count;
      if (a.status) a.status[b] = st;
    }
  }

  // Into and out of what the team shares.
  __device__ void leave(Team& t, uint32_t pass) const {
    const int l = threadIdx.x % WAVE;
    shared_store(&t.path[l], (uint8_t)my_path);
    if (l == 0) {
      shared_store(&t.cut, cut), shared_store(&t.Z, Z), shared_store(&t.gone, gone);
      shared_store(&t.mode, mode), shared_store(&t.st, st);
      shared_store(&t.place, (uint32_t)(count << 16 | child << 8 | cur));
    }
    settle();
    if (l == 0) shared_store(&t.pass, pass);
  }
  __device__ void enter(const Team& t) {
    const int l = threadIdx.x % WAVE;
    const uint32_t p = shared_load(&t.place);
    cur = (int)(p & 63u), child = (int)(p >> 8 & 127u), count = (int)(p >> 16 & 63u);
    cut = shared_load(&t.cut), Z = shared_load(&t.Z), gone = shared_load(&t.gone);
    mode = shared_load(&t.mode) & 1u, st = shared_load(&t.st);
    const uint8_t m = shared_load(&t.path[l]);
    my_path = l <= count ? (int)(m & 63u) : -1;
  }
};

__global__ __launch_bounds__(WAVE) void k_sample_begin(SampleArgs a) {
  const int b = blockIdx.x, l = threadIdx.x;
  Walk w(a, b, true);
  const bool go = w.valid() && w.advance(a);
  Team& t = a.team[b];
  if (l == 0) t.ticket = t.left = 0;
  if (go) {
    Walk none = w;
    none.st |= SD_ST_UNFINISHED;
    none.write(a, b, -1);
  } else {
    w.write(a, b, -1);
  }
  w.leave(t, go ? 0 : DONE);
}

// Vector k of a row of n elements of which `full` vectors are whole.  Loads are
// unconditional: lanes past them read the last whole vector, and get zeros.
__device__ __forceinline__ float4 load4(const float* row, int k, int full) {
  if (full == 0) return make_float4(0, 0, 0, 0);
  const float4 v = *(const float4*)(row + 4 * (int64_t)min(k, full - 1));
  return k < full ? v : make_float4(0, 0, 0, 0);
}

// The elements of a row's last vector where that is not whole.
__device__ __forceinline__ void load_rest(const float* row, int k, int n, float4& v) {
  if (k != n / 4) return;
  if (n % 4 > 0) v.x = row[4 * (int64_t)k];
  if (n % 4 > 1) v.y = row[4 * (int64_t)k + 1];
  if (n % 4 > 2) v.z = row[4 * (int64_t)k + 2];
}

// What a pass sums up: the rows of a node and the weight of an element.
struct Rows {
  const float *p, *q;      // q is p where the weights are p alone
  int np, nq;              // elements
  double cut;
  bool pair;

  __device__ Rows(const SampleArgs& a, const Nodes& nd, uint32_t place, uint32_t mode, double c) {
    const int64_t row = nd.first + min((int)(place & 63u), nd.T - 1);
    pair = mode == RESIDUAL && a.q;
    p = a.p + row * a.ld_p;
    q = pair ? a.q + row * a.ld_q : p;
    np = a.V, nq = pair ? a.Vd : 0;
    cut = pair ? c : 0.0;
  }
  template <int U>
  __device__ void load(int k0, int step, int hi, float4 (&x)[U], float4 (&y)[U]) const {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = k0 + u * step;
      x[u] = load4(p, k, min(hi, np / 4));
      y[u] = pair ? load4(q, k, min(hi, nq / 4)) : make_float4(0, 0, 0, 0);
    }
  }
  // Elements of vectors that are not whole, if the vectors [first, last) hold any.
  template <int U>
  __device__ void rest(int first, int last, int k0, int step, int hi, float4 (&x)[U], float4 (&y)[U]) const {
    const int ep = np / 4, eq = nq / 4;
    if (!((ep >= first && ep < last) || (pair && eq >= first && eq < last))) return;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = k0 + u * step;
      if (k >= hi) continue;
      load_rest(p, k, np, x[u]);
      if (pair) load_rest(q, k, nq, y[u]);
    }
  }
  // The weights of the n tokens `gone` taken out of the vectors [first, last).
  template <int U>
  __device__ static void drop(const int* gone, int n, int first, int last, int k0, int step, float4 (&x)[U]) {
    for (int j = 0; j < n; ++j) {
      const int e = gone[j];
      if (e / 4 < first || e / 4 >= last) continue;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = e - 4 * (k0 + u * step);
        if (i == 0) x[u].x = 0.0f;
        if (i == 1) x[u].y = 0.0f;
        if (i == 2) x[u].z = 0.0f;
        if (i == 3) x[u].w = 0.0f;
      }
    }
  }
  __device__ double weight(float x, float y) const { return fmax(fma(-cut, (double)y, (double)x), 0.0); }
};

__device__ __forceinline__ float at(const float4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

__global__ __launch_bounds__(NT) void k_sample_passes(SampleArgs a) {
  __shared__ uint32_t ticket_sh, pass_sh, place_sh, mode_sh;
  __shared__ int last_sh, gone_n, gone_sh[SD_MAX_NODES], go_sh, piece_sh, token_sh, spare_sh;
  __shared__ double cut_sh, total_sh[WV], base_sh;
  const int b = blockIdx.y, tid = threadIdx.x, l = tid % WAVE;
  const int wv = __builtin_amdgcn_readfirstlane(tid / WAVE);
  Team& team = a.team[b];
  const int pieces = a.slices * WV;
  double* const part = a.part + (int64_t)b * pieces;
  uint32_t next = tid == 0 ? shared_add(&team.ticket) : 0;
  Walk w(a, b, wv == 0);      // (its loads are on their way while the first pass is waited for)
  const int nvec = (a.V + 3) / 4;

  for (;;) {
    if (tid == 0) {
      const uint32_t want = next / (uint32_t)a.slices;
      uint32_t r = DONE;
      for (int i = 0; i < a.polls; ++i) {
        r = shared_load(&team.pass);
        if (r == DONE || r >= want) break;
        r = DONE;
        __builtin_amdgcn_s_sleep(1);
      }
      settle();
      place_sh = shared_load(&team.place), mode_sh = shared_load(&team.mode), cut_sh = shared_load(&team.cut);
      ticket_sh = next, pass_sh = r;
    }
    __syncthreads();
    const uint32_t pass = pass_sh;
    if (pass == DONE) return;
    const int sl = (int)(ticket_sh % (uint32_t)a.slices);
    const Rows rows(a, w.nd, place_sh, mode_sh, cut_sh);
    if (tid < WAVE && !a.q) {
      // tokens that a draw without draft rows leaves out, each once
      const int cur = (int)(place_sh & 63u), child = (int)(place_sh >> 8 & 127u);
      bool no = w.up == cur && l < child;
      for (int i = 0; i < WAVE - 1; ++i) {
        const int t = __builtin_amdgcn_readlane(w.tok, i);
        if (__builtin_amdgcn_readlane((int)no, i) && l > i && w.tok == t) no = false;
      }
      const uint64_t m = __ballot(no);
      if (no) gone_sh[__popcll(m & ((1ull << l) - 1))] = w.tok;
      if (l == 0) gone_n = __popcll(m);
    }
    if (tid == 0) next = shared_add(&team.ticket);      // on its way while the rows are read
    if (!a.q) __syncthreads();
    const int out = a.q ? 0 : gone_n;

    const int lo = min(nvec, (sl * WV + wv) * a.stretch), hi = min(nvec, lo + a.stretch);
    double sum = 0.0;
    bool bad = false;
    for (int k0 = lo; k0 < hi; k0 += WAVE * US) {
      float4 x[US], y[US];
      rows.load<US>(k0 + l, WAVE, hi, x, y);
      rows.rest<US>(k0, k0 + WAVE * US, k0 + l, WAVE, hi, x, y);
      rows.drop<US>(gone_sh, out, k0, k0 + WAVE * US, k0 + l, WAVE, x);
#pragma unroll
      for (int u = 0; u < US; ++u) {
        const float lowest = fminf(fminf(fminf(x[u].x, x[u].y), fminf(x[u].z, x[u].w)),
                                   fminf(fminf(y[u].x, y[u].y), fminf(y[u].z, y[u].w)));
        const float all = (x[u].x + x[u].y) + (x[u].z + x[u].w) + ((y[u].x + y[u].y) + (y[u].z + y[u].w));
        bad |= !(lowest >= 0.0f) || !(all < INFINITY);
        sum += rows.weight(x[u].x, y[u].x);
        sum += rows.weight(x[u].y, y[u].y);
        sum += rows.weight(x[u].z, y[u].z);
        sum += rows.weight(x[u].w, y[u].w);
      }
    }
    sum = wave_sum(bad ? (double)NAN : sum);
    if (l == 0) shared_store(&part[sl * WV + wv], sum);
    settle();
    __syncthreads();
    if (tid == 0) last_sh = shared_add(&team.left) == (pass + 1) * (uint32_t)a.slices - 1;
    __syncthreads();
    if (!last_sh) continue;

    // The last of the pass.  Its total, in the order of the stretches.
    const double mine = tid < pieces ? shared_load(&part[tid]) : 0.0;
    const bool nan = __syncthreads_or(!(mine < INFINITY));
    const double incl = wave_incl_scan(mine);
    if (l == WAVE - 1) total_sh[wv] = incl;
    __syncthreads();
    double before = 0.0, total = 0.0;
#pragma unroll
    for (int i = 0; i < WV; ++i) {
      if (i < wv) before += total_sh[i];
      total += total_sh[i];
    }
    if (tid < WAVE) {
      w.enter(team);
      enum { STOP, DRAW, AGAIN } go = STOP;
      const double v = (double)a.v[b];
      if (nan) w.st |= SD_ST_NONFINITE;
      if (w.valid()) {
        if (w.mode == RESIDUAL && !(total > 0.0)) {
          // p = q but for rounding: the draw is from p, after one more pass
          w.st |= SD_ST_RESID_ZERO;
          w.mode = PLAIN, w.child = WAVE;
          go = AGAIN;
        } else if (w.mode == RESIDUAL && __ballot(w.up == w.cur && l >= w.child)) {
          w.Z = total;
          if (w.advance(a)) go = AGAIN;
        } else if (!(total > 0.0)) {
          w.st |= SD_ST_NONFINITE;
        } else {
          if (!(v >= 0.0 && v < 1.0)) w.st |= SD_ST_BAD_PARAM;
          else go = DRAW;
        }
      }
      if (go == AGAIN) w.leave(team, pass + 1);
      if (go == STOP) {
        w.write(a, b, -1);
        if (l == 0) shared_store(&team.pass, DONE);
      }
      if (l == 0) go_sh = go, piece_sh = INT_MAX, spare_sh = -1, token_sh = INT_MAX;
    }
    __syncthreads();
    if (go_sh == 2) continue;
    if (go_sh == 0) return;

    // The draw: the stretch whose part of the cumulative sum passes t first (the
    // last one with a weight, where rounding leaves t at the total) ...
    const double t = (double)a.v[b] * total;
    if (mine > 0.0) {
      if (before + incl > t) atomicMin(&piece_sh, tid);
      atomicMax(&spare_sh, tid);
    }
    __syncthreads();
    const int piece = piece_sh < INT_MAX ? piece_sh : spare_sh;
    __syncthreads();
    if (tid == piece) base_sh = before + incl - mine, spare_sh = -1;
    __syncthreads();
    // ... and its token, a vector a thread at a time
    double base = base_sh;
    const int end = min(nvec, (piece + 1) * a.stretch);
    for (int k0 = piece * a.stretch; k0 < end && token_sh == INT_MAX; k0 += NT) {
      float4 x[1], y[1];
      const int k = k0 + tid;
      rows.load<1>(k, 0, end, x, y);
      rows.rest<1>(k0, k0 + NT, k, 0, end, x, y);
      rows.drop<1>(gone_sh, out, k0, k0 + NT, k, 0, x);
      double g[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) g[i] = rows.weight(at(x[0], i), at(y[0], i));
      const double own = (g[0] + g[1]) + (g[2] + g[3]);
      const double run = wave_incl_scan(own);
      if (l == WAVE - 1) total_sh[wv] = run;
      __syncthreads();
      double c = base + run - own, all = 0.0;
#pragma unroll
      for (int i = 0; i < WV; ++i) {
        if (i < wv) c += total_sh[i];
        all += total_sh[i];
      }
      int pick = INT_MAX, some = -1;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        c += g[i];
        if (g[i] > 0.0) {
          some = 4 * k + i;
          if (c > t) pick = min(pick, some);
        }
      }
      if (pick < INT_MAX) atomicMin(&token_sh, pick);
      if (some >= 0) atomicMax(&spare_sh, some);
      base += all;
      __syncthreads();
    }
    if (tid < WAVE) {
      w.write(a, b, token_sh < INT_MAX ? token_sh : spare_sh);
      if (l == 0) shared_store(&team.pass, DONE);
    }
    return;
  }
}

int check(const sd_tree_sample_args_t* p) {
  if (!p || !p->target_probs || !aligned16(p->target_probs) || !aligned16(p->draft_probs) || !p->tokens ||
      !p->parents || !p->node_offsets || !p->accept_uniforms || !p->draw_uniforms)
    return SD_EINVAL;
  if (p->B < 1 || p->N < 1 || p->V < 1 || p->max_nodes < 1 || p->ld_target < p->V || p->ld_target % 4 ||
      (p->flags & ~(uint32_t)(SD_NO_BONUS | SD_NO_REPLACEMENT)))
    return SD_EINVAL;
  if (p->draft_probs && (p->V_draft < 1 || p->V_draft > p->V || p->ld_draft < p->V_draft || p->ld_draft % 4))
    return SD_EINVAL;
  if (p->max_nodes > SD_MAX_NODES || p->V >= (1 << 28) || p->B > 65535) return SD_EUNSUPPORTED;
  return SD_OK;
}

// Workgroups that share a request's rows: about two a CU in all, none with less
// than 64 vectors a wave, and a stretch for every thread of the last at most.
int slices_of(const sd_tree_sample_args_t* p) {
  const int nvec = (p->V + 3) / 4;
  return std::max(1, std::min({(512 + p->B - 1) / p->B, (nvec + NT - 1) / NT, NT / WV}));
}

size_t parts_bytes(const sd_tree_sample_args_t* p) { return (size_t)p->B * slices_of(p) * WV * sizeof(double); }

}  // namespace

extern "C" int sd_tree_sample_workspace_bytes(const sd_tree_sample_args_t* args, size_t* bytes) {
  if (!bytes) return SD_EINVAL;
  const int rc = check(args);
  if (rc) return rc;
  *bytes = parts_bytes(args) + (size_t)args->B * sizeof(Team);
  return SD_OK;
}

extern "C" int sd_tree_verify_sample(const sd_tree_sample_args_t* args, void* workspace,
                                     size_t workspace_bytes, int32_t* out_accepted,
                                     int32_t* out_path, int32_t* out_tokens,
                                     uint32_t* out_status, void* stream) {
  return sd_debug_tree_sample_polls(args, workspace, workspace_bytes, out_accepted, out_path, out_tokens,
                                    out_status, MAX_POLLS, stream);
}

extern "C" int sd_debug_tree_sample_polls(const sd_tree_sample_args_t* args, void* workspace,
                                          size_t workspace_bytes, int32_t* out_accepted,
                                          int32_t* out_path, int32_t* out_tokens,
                                          uint32_t* out_status, int32_t polls, void* stream) {
  size_t need = 0;
  const int rc = sd_tree_sample_workspace_bytes(args, &need);
  if (rc) return rc;
  if (!out_accepted || !out_path || !out_tokens) return SD_EINVAL;
  const void* outs[] = {out_accepted, out_path, out_tokens, out_status};
  const void* ins[] = {args->target_probs, args->draft_probs, args->tokens, args->parents, args->node_offsets,
                       args->accept_uniforms, args->draw_uniforms};
  for (int i = 0; i < 4; ++i) {
    for (const void* in : ins)
      if (outs[i] && outs[i] == in) return SD_EINVAL;
    for (int j = 0; j < i; ++j)
      if (outs[i] && outs[i] == outs[j]) return SD_EINVAL;
  }
  if (!workspace || workspace_bytes < need || (uintptr_t)workspace % 8) return SD_EWORKSPACE;
  SampleArgs a;
  a.p = args->target_probs, a.q = args->draft_probs;
  a.ld_p = args->ld_target, a.ld_q = args->ld_draft;
  a.tokens = args->tokens, a.parents = args->parents, a.off = args->node_offsets;
  a.u = args->accept_uniforms, a.v = args->draw_uniforms;
  a.B = args->B, a.N = args->N, a.V = args->V, a.Vd = args->V_draft, a.max_nodes = args->max_nodes;
  a.flags = args->flags;
  a.slices = slices_of(args);
  const int pieces = a.slices * WV;
  a.stretch = ((a.V + 3) / 4 + pieces - 1) / pieces;
  a.polls = polls;
  a.part = static_cast<double*>(workspace);
  a.team = reinterpret_cast<Team*>(static_cast<char*>(workspace) + parts_bytes(args));
  a.accepted = out_accepted, a.path = out_path, a.out_tokens = out_tokens, a.status = out_status;
  hipStream_t st = static_cast<hipStream_t>(stream);
  hipLaunchKernelGGL(k_sample_begin, dim3(a.B), dim3(WAVE), 0, st, a);
  if (hipGetLastError() != hipSuccess) return SD_EHIP;
  hipLaunchKernelGGL(k_sample_passes, dim3(a.slices, a.B), dim3(NT), 0, st, a);
  return hipGetLastError() == hipSuccess ? SD_OK : SD_EHIP;
}
