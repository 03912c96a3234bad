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
// by passes that follow each other: each reads its rows (again, where only cut has
// changed since the one before), and at its end what a wave sums up travels to the
// others and back, some 4 us; the longest walk of a batch has several.  Rows of 151936:
// 1 tree of 16 nodes 15 us; 64 trees of 20, draws without replacement, up to 4 passes,
// 40 us (the bytes of one pass: 15); 48 trees of a beam, one pass each, 18 us (6).
//
// k_sample_begin    clears what the teams share.
// k_sample_passes   teams of workgroups, one a slice of the vocabulary; each of their
//                   waves sums up a stretch of its own.  Every member leaves its
//                   slice's sum for the others, reads theirs, and follows the walk by
//                   itself, so a pass costs one store and one look at it.  A sum
//                   carries its pass in its 7 lowest bits, and the sums of two passes
//                   have places of their own: who writes the third has read the first.
//                   The member whose slice the draw falls on finds the token.
//
// A slice is claimed before its sum is left, by the workgroup that it belongs to or,
// when that does not come, by one that waits for it and has it from then on; who
// loses its last slice ends.  So every wait is for a workgroup that runs, however few
// of a team the chip holds at a time.  (Calls that overlap on one workspace, which the
// interface forbids, could take each other's slices: waits are bounded, and such a
// request keeps the -1 and SD_ST_UNFINISHED that its results begin with.)  What a
// team shares is only touched by relaxed agent-scope atomics, a value each.
#include <algorithm>

#include "sd_serve.h"
#include "sdt_device.h"

using namespace sdv;
using namespace sdt;

namespace {

constexpr int NT = 512;               // threads of a workgroup
constexpr int WV = NT / WAVE;
constexpr int US = 4;                 // vectors of each row that a lane loads at once (in the last two cases
                                      // above 2 take 1 us less and 1 more, 8 take 5 and 2 more)
constexpr int MAX_SLICES = WAVE;      // (a lane looks at each)
constexpr uint64_t TAG = 127;         // of a sum; passes are SD_MAX_NODES + 1 at most: every node's
                                      // rejection but the root's, a draw, one more after a total of 0
constexpr int MAX_POLLS = 1 << 21;    // about two seconds; a wait takes microseconds
constexpr int STEAL = 24;             // looks at a pass before its unclaimed slices are taken over, some 20 us

struct Team {
  uint64_t sums[2][MAX_SLICES];       // of the even passes and the odd ones; their tag is the pass + 1
  uint32_t claims[MAX_SLICES];        // passes for which a slice was claimed
};
enum Mode : uint32_t { RESIDUAL, PLAIN };      // weights max(p - cut q, 0), or p without the rejected tokens
enum Next { STOP, DRAW, PASS };

struct SampleArgs {
  const float *p, *q;
  int64_t ld_p, ld_q;
  const int32_t *tokens, *parents, *off;
  const float *u, *v;
  int B, N, V, Vd, max_nodes;
  uint32_t flags;
  int slices, stretch;      // stretch: vectors of 4 that a wave sums up
  int polls;
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
// Whether *p was `from`; it is `from + 1` then.
__device__ __forceinline__ bool shared_claim(uint32_t* p, uint32_t from) {
  return __hip_atomic_compare_exchange_strong(p, &from, from + 1, __ATOMIC_RELAXED, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ bool bad_prob(double x) { return !(x >= 0.0 && x < INFINITY); }

// A request's tree and walk in a wave: lane l holds node l.
struct Walk {
  Nodes nd;
  uint32_t st;
  int tok, up;
  double px, qx, u;      // of the lane's token in its parent's rows
  float v;
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
    v = a.v[b];
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

  // Goes on after a pass with this total.
  __device__ Next resume(const SampleArgs& a, double total) {
    const int l = threadIdx.x % WAVE;
    if (!(total < INFINITY)) {      // (NaN: an element that is no probability)
      st |= SD_ST_NONFINITE;
      return STOP;
    }
    const bool resid = mode == RESIDUAL;
    if (!(total > 0.0) && (resid || (!a.q && __any(up == cur && l < child)))) {
      // p = q but for rounding, or every token that p holds was given and rejected, since
      // its numbers sum to 1 only within rounding: the draw is from all of p, after
      // one more pass
      st |= SD_ST_RESID_ZERO;
      mode = PLAIN;
      child = resid ? WAVE : 0;      // (without draft rows the tokens before it are left out)
      return PASS;
    }
    if (resid && __ballot(up == cur && l >= child)) {
      Z = total;
      return advance(a) ? PASS : STOP;
    }
    if (!(total > 0.0)) st |= SD_ST_NONFINITE;
    else if (!(v >= 0.0f && v < 1.0f)) st |= SD_ST_BAD_PARAM;
    else return DRAW;
    return STOP;
  }
};

// Requests as they are until their walks end, one wave each.
__global__ __launch_bounds__(WAVE) void k_sample_begin(SampleArgs a) {
  const int b = blockIdx.x, l = threadIdx.x;
  Team& t = a.team[b];
  t.sums[0][l] = t.sums[1][l] = 0;
  t.claims[l] = 0;
  if (l < a.max_nodes) {
    a.path[(int64_t)b * a.max_nodes + l] = -1;
    a.out_tokens[(int64_t)b * a.max_nodes + l] = -1;
  }
  if (l == 0) {
    a.accepted[b] = -1;
    if (a.status) a.status[b] = SD_ST_UNFINISHED;
  }
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

  __device__ Rows(const SampleArgs& a, int64_t row, uint32_t mode, double c) {
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
    if (!n) return;
    const int l = threadIdx.x % WAVE, mine = l < n ? gone[l] : -1;
    for (uint64_t in = __ballot(mine >= 0 && mine / 4 >= first && mine / 4 < last); in; in &= in - 1) {
      const int e = __builtin_amdgcn_readlane(mine, __builtin_ctzll(in));
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

// The sum of a lane's weights, NaN where one of its elements is no probability.
template <int U>
__device__ __forceinline__ void add_up(const Rows& rows, const float4 (&x)[U], const float4 (&y)[U], double& sum, bool& bad) {
#pragma unroll
  for (int u = 0; u < U; ++u) {
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

__global__ __launch_bounds__(NT, 4) void k_sample_passes(SampleArgs a) {
  __shared__ uint32_t mode_sh;
  __shared__ int cur_sh, go_sh, got_sh, draw_sh, gone_n, gone_sh[SD_MAX_NODES], token_sh, spare_sh;
  __shared__ double cut_sh, t_sh, sums_sh[WV], run_sh[WV];
  __shared__ uint64_t missing_sh;
  const int b = blockIdx.y, own = blockIdx.x, tid = threadIdx.x, l = tid % WAVE;
  const int wv = __builtin_amdgcn_readfirstlane(tid / WAVE);
  Team& team = a.team[b];
  const int nvec = (a.V + 3) / 4;
  Walk w(a, b, wv == 0);      // wave 0 walks

  // Wave 0: how it goes on, for the others.
  auto tell = [&](Next go) {
    if (l == 0) go_sh = go;
    if (go != PASS) return;
    if (l == 0) mode_sh = w.mode, cur_sh = w.cur, cut_sh = w.cut;
    if (a.q) return;
    // tokens that a draw without draft rows leaves out, each once
    bool no = w.up == w.cur && l < w.child;
    for (uint64_t some = __ballot(no); some; some &= some - 1) {
      const int i = __builtin_ctzll(some);
      if (l > i && w.tok == __builtin_amdgcn_readlane(w.tok, i)) no = false;
    }
    const uint64_t m = __ballot(no);
    if (no) gone_sh[__popcll(m & ((1ull << l) - 1))] = w.tok;
    if (l == 0) gone_n = __popcll(m);
  };
  if (wv == 0) tell(w.valid() && w.advance(a) ? PASS : STOP);
  __syncthreads();
  if (go_sh == STOP) {
    if (own == 0 && wv == 0) w.write(a, b, -1);
    return;
  }

  uint64_t mine = 1ull << own;      // slices that this workgroup sums up
  for (uint32_t pass = 0;; ++pass) {
    const int out = a.q ? 0 : gone_n;
    const Rows rows(a, w.nd.first + cur_sh, mode_sh, cut_sh);
    const uint32_t tag = pass + 1;
    int held = -1;                  // the slice whose stretches' sums are in sums_sh

    // A slice's stretches, one a wave.
    auto sum_up = [&](int s) {
      const int lo = min(nvec, (s * WV + wv) * a.stretch), hi = min(nvec, lo + a.stretch);
      double sum = 0.0;
      bool bad = false;
      for (int k0 = lo; k0 < hi; k0 += WAVE * US) {
        float4 x[US], y[US];
        rows.load<US>(k0 + l, WAVE, hi, x, y);
        rows.rest<US>(k0, k0 + WAVE * US, k0 + l, WAVE, hi, x, y);
        rows.drop<US>(gone_sh, out, k0, k0 + WAVE * US, k0 + l, WAVE, x);
        add_up<US>(rows, x, y, sum, bad);
      }
      sum = wave_sum(bad ? (double)NAN : sum);
      if (l == 0) sums_sh[wv] = sum;
      held = s;
    };
    auto slice_sum = [&] {          // in every thread, with its tag
      double sum = 0.0;
#pragma unroll
      for (int i = 0; i < WV; ++i) sum += sums_sh[i];
      return (__builtin_bit_cast(uint64_t, sum) & ~TAG) | tag;
    };

    uint64_t want = mine;
    mine = 0;
    for (int looks = 0, most = min(STEAL, a.polls);;) {
      for (; want; want &= want - 1) {
        const int s = __builtin_ctzll(want);
        // the claim is under way while the slice is summed up
        bool got = true;
        if (tid == 0 && a.slices > 1) got = shared_claim(&team.claims[s], pass);
        sum_up(s);
        if (tid == 0) got_sh = got;
        __syncthreads();
        if (got_sh) {
          mine |= 1ull << s;
          if (tid == 0 && a.slices > 1) shared_store(&team.sums[pass % 2][s], slice_sum());
        }
        if (want & (want - 1)) __syncthreads();
      }
      if (!mine) return;
      if (wv == 0) {
        uint64_t bits = tag, missing = 0;
        bool late = false;
        for (;;) {
          if (a.slices == 1) bits = l == 0 ? slice_sum() : tag;
          else if (l < a.slices) bits = shared_load(&team.sums[pass % 2][l]);
          late = __any((bits & TAG) > tag);
          missing = __ballot((bits & TAG) != tag);
          if (!missing || late || ++looks > most) break;
          __builtin_amdgcn_s_sleep(1);
        }
        if (l == 0) missing_sh = missing;
        // (others have gone on without this one, or it has given up)
        if (late || (missing && most == a.polls)) {
          if (l == 0) missing_sh = 0, go_sh = STOP, draw_sh = -1;
        } else if (!missing) {
          const double x = __builtin_bit_cast(double, bits & ~TAG);
          const double incl = wave_incl_scan(x);
          const double total = lane_read(incl, WAVE - 1);
          const Next go = w.resume(a, __any(!(x < INFINITY)) ? (double)NAN : total);
          tell(go);
          // the draw: the slice whose sum takes the running one past t first (the
          // last one with a weight, where rounding leaves t at the total)
          int s = 0;
          if (go == DRAW) {
            const double t = (double)w.v * total;
            const uint64_t past = __ballot(x > 0.0 && incl > t), some = __ballot(x > 0.0);
            s = past ? __builtin_ctzll(past) : WAVE - 1 - __builtin_clzll(some);
            const double before = lane_read(incl - x, s);
            if (l == 0) t_sh = t - before, token_sh = INT_MAX, spare_sh = -1;
          }
          if (l == 0) draw_sh = s;
        }
      }
      __syncthreads();
      want = missing_sh;
      if (!want) break;
      most = a.polls;
      __syncthreads();
    }
    if (go_sh == PASS) continue;
    const int s = draw_sh;
    if (s < 0 || !(mine >> s & 1)) return;      // another one's to finish
    if (go_sh == STOP) {
      if (wv == 0) w.write(a, b, -1);
      return;
    }

    // The token: first its stretch ...
    if (held != s) sum_up(s);
    __syncthreads();
    const double t = t_sh;
    double base = 0.0, run = 0.0;
    int piece = 0;
#pragma unroll
    for (int i = 0; i < WV; ++i) {
      const double x = sums_sh[i];
      // (once the running sum is past t, the stretch is found)
      if (x > 0.0 && !(run > t)) base = run, piece = i;
      run += x;
    }
    // ... and in it a vector a thread at a time
    const int lo = min(nvec, (s * WV + piece) * a.stretch), hi = min(nvec, lo + a.stretch);
    for (int k0 = lo; k0 < hi && token_sh == INT_MAX; k0 += NT) {
      float4 x[1], y[1];
      const int k = k0 + tid;
      rows.load<1>(k, 0, hi, x, y);
      rows.rest<1>(k0, k0 + NT, k, 0, hi, x, y);
      rows.drop<1>(gone_sh, out, k0, k0 + NT, k, 0, x);
      double g[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) g[i] = rows.weight(at(x[0], i), at(y[0], i));
      const double sum = (g[0] + g[1]) + (g[2] + g[3]);
      const double incl = wave_incl_scan(sum);
      if (l == WAVE - 1) run_sh[wv] = incl;
      __syncthreads();
      double c = base + incl - sum, all = 0.0;
#pragma unroll
      for (int i = 0; i < WV; ++i) {
        if (i < wv) c += run_sh[i];
        all += run_sh[i];
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
    if (wv == 0) w.write(a, b, token_sh < INT_MAX ? token_sh : spare_sh);
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

// Workgroups that share a request's rows: two a CU in all (one: 45 instead of 40 us
// in the case of 64 trees); where they are several, none with less than 32 vectors a wave.
int slices_of(const sd_tree_sample_args_t* p) {
  const int nvec = (p->V + 3) / 4;
  return std::max(1, std::min({512 / p->B, (nvec + NT - 1) / NT, MAX_SLICES}));
}

}  // namespace

extern "C" int sd_tree_sample_workspace_bytes(const sd_tree_sample_args_t* args, size_t* bytes) {
  if (!bytes) return SD_EINVAL;
  const int rc = check(args);
  if (rc) return rc;
  *bytes = (size_t)args->B * sizeof(Team);
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
  a.polls = polls < 0 ? MAX_POLLS : polls;
  a.team = static_cast<Team*>(workspace);
  a.accepted = out_accepted, a.path = out_path, a.out_tokens = out_tokens, a.status = out_status;
  hipStream_t st = static_cast<hipStream_t>(stream);
  hipLaunchKernelGGL(k_sample_begin, dim3(a.B), dim3(WAVE), 0, st, a);
  if (hipGetLastError() != hipSuccess) return SD_EHIP;
  // (a negative bound: half of each team stays away, the others take its slices over)
  hipLaunchKernelGGL(k_sample_passes, dim3(polls < 0 ? (a.slices + 1) / 2 : a.slices, a.B), dim3(NT), 0, st, a);
  return hipGetLastError() == hipSuccess ? SD_OK : SD_EHIP;
}
