// Append to and eviction from a paged key/value cache on gfx950.
//
// sd_cache_commit:
//   k_commit       one workgroup per (run of slots, KV head, request): the
//                  slots' weights, sums of exp(scale q . k - lse) over the
//                  branch's query rows, by MFMA; the first run's also
//                  appends the branch's keys, values and positions.
// sd_cache_evict:
//   k_evict_select   one workgroup per (request, KV head): the budget-th
//                    largest key by a radix search, then the freed slots
//                    below the budget and the kept ones past it, in order;
//   k_evict_move     each kept row past the budget into its freed slot.
#include <algorithm>

#include "sdt_device.h"

using namespace sdv;
using namespace sdt;

namespace {

constexpr int NT_C = 256;   // threads of a commit workgroup: 64 keys a wave
constexpr int QB = 128;     // query rows in LDS

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

// Append of head h: keys, values and positions; the first head's workgroup
// also leaves the length and the status.
template <int D>
__device__ void append(const CommitArgs& a, const Branch& r, int b, int h) {
  constexpr int LPR = D / 8;   // lanes of one row
  const int tid = threadIdx.x, d = (tid % LPR) * 16;
  const int32_t* tab = table_row(a.c, b);
  for (int i = tid / LPR; i < r.m; i += NT_C / LPR) {
    const int64_t at = slot_offset(a.c, tab, r.ctx + i, h);
    const int64_t row = r.first + a.path[b * a.ld_path + i];
    if (at >= 0) {
      *(uint4*)(a.c.k + at + d) = *(const uint4*)(a.kn + row * a.k_node + h * a.k_head + d);
      *(uint4*)(a.c.v + at + d) = *(const uint4*)(a.vn + row * a.v_node + h * a.v_head + d);
    }
    if (a.positions && d == 0)
      a.positions[((int64_t)b * a.c.H + h) * a.ld_mass + r.ctx + i] = a.seen[b] + i;
  }
  if (h || tid >= WAVE) return;
  if (tid == 0) a.out_ctx[b] = (r.st & SD_ST_BAD_LEN) ? a.c.lens[b] : r.ctx + r.m;
  if (!a.status) return;
  bool bad_page = false;
  for (int p = tid; p < (r.ctx + r.m + a.c.page_mask) >> a.c.page_shift; p += WAVE)
    bad_page |= (unsigned)tab[p] >= (unsigned)a.c.num_pages;
  const uint32_t st = r.st | (__any(bad_page) ? SD_ST_BAD_PAGE : 0u);
  if (tid == 0) a.status[b] = st;
}

// grid (chunks of `chunk` slots, H, B).  A wave holds 64 keys in registers as
// MFMA operands straight from the cache and meets the branch's query rows, 16
// at a time from LDS: S = Q . K^T, so a lane holds 4 rows of one key and the
// sum over the rows is in its own registers but for two lane swaps at the end.
// The keys are read once; row blocks past the first are staged again for every
// tile.  Bound by HBM up to about 150 rows: 363 MB of keys and weights in 86 us
// (4.2 TB/s) for 32 requests of 5k to 16k slots, 4 KV heads and up to 42 rows.
template <int DT, int D>
__global__ __launch_bounds__(NT_C, 2) void k_commit(CommitArgs a, int chunk) {
  constexpr int KS = D / 32, CPR = D / 8;
  __shared__ __align__(16) char sq[QB * D * 2];
  __shared__ __align__(16) float se[QB];
  const int b = blockIdx.z, h = blockIdx.y, tid = threadIdx.x, l = tid % WAVE, w = tid / WAVE;
  const int n = l & 15, g4 = l >> 4;
  const Branch br = request_branch(a, b);
  if (blockIdx.x == 0) append<D>(a, br, b, h);
  const int end = br.ctx + br.m;
  int base = blockIdx.x * chunk;
  const int stop = base + min(chunk, max(0, end - base));
  if (!a.mass_out || br.st || base >= stop) return;
  const int32_t* tab = table_row(a.c, b);
  const int rows = br.m * a.G;
  const float c = a.scale * 1.4426950408889634f;

  auto stage = [&](int q0) {       // query rows q0 .. q0 + QB - 1, zeros past the last; e = +inf: not counted
    __syncthreads();
    for (int u = tid; u < QB * CPR; u += NT_C) {
      const int lr = u / CPR, col = u % CPR, r = q0 + lr;
      if (lr >= ((rows - q0 + 15) & ~15)) break;
      uint4 v = make_uint4(0, 0, 0, 0);
      if (r < rows) {
        const int64_t node = br.first + a.path[b * a.ld_path + r / a.G];
        v = *(const uint4*)(a.q + node * a.q_node + (h * a.G + r % a.G) * a.q_head + col * 16);
      }
      *(uint4*)(sq + lr * (D * 2) + ((col ^ swz<D>(lr)) * 16)) = v;
    }
    for (int lr = tid; lr < QB; lr += NT_C) {
      const int r = q0 + lr;
      float e = INFINITY;
      if (r < rows) {
        const int64_t node = br.first + a.path[b * a.ld_path + r / a.G];
        e = a.lse[node * a.Hq + h * a.G + r % a.G] * 1.4426950408889634f;
        if (e == -INFINITY) e = INFINITY;      // it saw nothing: no weight
      }
      se[lr] = e;
    }
    __syncthreads();
  };

  s16x8 k[4][KS];
  uint32_t on = 0;                  // bit s: this lane's key of subtile s is there
  auto load = [&](int from) {
    on = 0;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int t = from + w * 64 + s * 16 + n;
      const char* p = nullptr;
      if (t < br.ctx) {
        const int64_t at = slot_offset(a.c, tab, t, h);
        if (at >= 0) p = a.c.k + at;
      } else if (t < end) {
        p = a.kn + (int64_t)(br.first + a.path[b * a.ld_path + t - br.ctx]) * a.k_node + h * a.k_head;
      }
      on |= (p ? 1u : 0u) << s;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) k[s][ks] = p ? *(const s16x8*)(p + ks * 64 + g4 * 16) : s16x8{};
    }
  };

  const int64_t row = ((int64_t)b * a.c.H + h) * a.ld_mass;
  bool staged = false;
  for (; base < stop; base += NT_C) {
    load(base);
    float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    const bool fresh = base + w * 64 + 64 > br.ctx;
    for (int q0 = 0; q0 < rows; q0 += QB) {
      if (!staged) stage(q0);
      staged = rows <= QB;
      const int tiles = (min(rows - q0, QB) + 15) / 16;
      for (int rt = 0; rt < tiles; ++rt) {
        s16x8 q[KS];
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          const int lr = rt * 16 + n;
          q[ks] = *(const s16x8*)(sq + lr * (D * 2) + (((ks * 4 + g4) ^ swz<D>(lr)) * 16));
        }
        const f32x4 e = *(const f32x4*)(se + rt * 16 + g4 * 4);
        // Row i sees the slots in use and the appended ones 0 .. i.  Rows that do not
        // count have e = +inf.  Products with an infinite key may not be numbers, so
        // they are left out, not added: up[r] is the last appended slot whose key
        // row r counts for.
        const bool chosen = fresh || __any(fmaxf(fmaxf(e[0], e[1]), fmaxf(e[2], e[3])) == INFINITY);
        int up[4] = {};
        if (chosen) {
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            up[r] = fresh ? (q0 + rt * 16 + g4 * 4 + r) / a.G : INT_MAX;
            if (e[r] == INFINITY) up[r] = INT_MIN;
          }
        }
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          f32x4 x = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) x = mfma<DT>(q[ks], k[s][ks], x);
          if (chosen) {
            const int j = base + w * 64 + s * 16 + n - br.ctx;
#pragma unroll
            for (int r = 0; r < 4; ++r) sum[s] += j <= up[r] ? fast_exp2(fmaf(x[r], c, -e[r])) : 0.0f;
          } else {
#pragma unroll
            for (int r = 0; r < 4; ++r) sum[s] += fast_exp2(fmaf(x[r], c, -e[r]));
          }
        }
      }
    }
    // lane (n, g4) leaves key 16 g4 + n of the wave's 64
    float mine = 0.0f;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const float v = quad_sum(sum[s]);
      if (g4 == s) mine = (on >> s & 1) ? v : 0.0f;
    }
    const int t = base + w * 64 + l;
    if (t < stop) {
      if (t < br.ctx && a.decay != 0.0f) mine = fmaf(a.decay, a.mass_in[row + t], mine);
      a.mass_out[row + t] = mine;
    }
  }
}

// ---- eviction ----

constexpr int NT_E = 1024;     // threads of a selection
constexpr int WE = NT_E / WAVE;
constexpr int HB = 2048;        // digits of the histogram
constexpr int MV = 64;         // rows of a move workgroup's round

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
__device__ __forceinline__ uint32_t rank_key(const EvictArgs& a, float m, int p, int recent_from) {
  if (a.pos_in && (p < a.sinks || p >= recent_from)) return 0xFFFFFFFFu;
  return ord_key(m != m ? -INFINITY : m);
}

__device__ __forceinline__ uint32_t evict_key(const EvictArgs& a, int64_t row, int t, int recent_from) {
  return rank_key(a, a.mass_in[row + t], a.pos_in ? a.pos_in[row + t] : 0, recent_from);
}

// The digit at which the `want` largest keys of the histogram end, and how
// many keys of that digit belong to them; thread 0 has the highest digits.
__device__ __forceinline__ void find_digit(const int* hist, int want, int* scratch, int* digit, int* left) {
  const int top = HB - 1 - 2 * (int)threadIdx.x;
  const int c0 = hist[2 * top] + hist[2 * top + 1], c1 = hist[2 * top - 2] + hist[2 * top - 1];
  int total;
  const int above = block_excl_scan_int<NT_E>(c0 + c1, scratch, &total);
  if (above < want && want <= above + c0) *digit = top, *left = want - above;
  if (above + c0 < want && want <= above + c0 + c1) *digit = top - 1, *left = want - above - c0;
}

// One workgroup per (KV head, request).  The rank keys of up to LCAP slots are
// kept in LDS, so mass and positions are read once; longer contexts compute
// them again in each of the 5 or 6 passes.  Bound by what one CU reads (about
// 30 GB/s) and by the latencies of the passes over LDS.  Digits are 11 bits wide,
// as masses share few exponents, and two copies of the histogram keep
// neighbouring lanes apart.  39 us for 64 heads of 20k to 32k slots; 10 us for
// 2053 slots.
template <int LCAP>
__global__ __launch_bounds__(NT_E) void k_evict_select(EvictArgs a) {
  __shared__ uint32_t keys[LCAP];
  __shared__ int hist[2 * HB];
  __shared__ int sel[2];
  __shared__ int scratch[WE];
  __shared__ int counts[3][WE];
  // slots a thread loads at once, and steps of 64 slots a wave of the last
  // passes takes at once: more of them only where contexts are long
  constexpr int UE = LCAP > 4096 ? 16 : 4, UP = LCAP > 4096 ? 8 : 4;
  const int h = blockIdx.x, b = blockIdx.y, tid = threadIdx.x, l = tid % WAVE;
  const int w = __builtin_amdgcn_readfirstlane(tid / WAVE);
  uint32_t st = 0;
  const int n = request_ctx(a.c, b, st);
  const int bh = b * a.c.H + h;
  const int64_t row = (int64_t)bh * a.ld;
  if (st || n <= a.budget) {
    for (int t = tid; t < n; t += NT_E) {
      if (a.mass_out != a.mass_in) a.mass_out[row + t] = a.mass_in[row + t];
      if (a.pos_in && a.pos_out != a.pos_in) a.pos_out[row + t] = a.pos_in[row + t];
    }
    if (tid == 0) a.count[bh] = 0;
    return;
  }
  const int recent_from = a.pos_in ? (int)max((int64_t)a.seen[b] - a.recent, (int64_t)INT_MIN) : INT_MAX;
  const bool held = n <= LCAP;
  auto key = [&](int t) { return held ? keys[t] : evict_key(a, row, t, recent_from); };

  // the budget-th largest key, 11, 11 and 10 bits at a time; of the slots
  // equal to it the lowest `want` are kept
  uint32_t cut = 0;
  int want = a.budget;
  for (int digit = 0; digit < 3; ++digit) {
    const int shift = digit == 0 ? 21 : digit == 1 ? 10 : 0;
    const uint32_t mask = digit == 2 ? 1023u : 2047u;
    const int known = digit == 0 ? 31 : digit == 1 ? 21 : 10;      // bits below the digits found
    for (int i = tid; i < 2 * HB; i += NT_E) hist[i] = 0;
    __syncthreads();
    auto count = [&](uint32_t k) {
      if (digit == 0 || (k >> known) == (cut >> known)) atomicAdd(&hist[((k >> shift) & mask) * 2 + (l & 1)], 1);
    };
    if (digit > 0 && held) {
#pragma unroll 8
      for (int t = tid; t < n; t += NT_E) count(keys[t]);
    } else {
      for (int t0 = tid; t0 < n; t0 += NT_E * UE) {
        float m[UE];
        int p[UE];
#pragma unroll
        for (int u = 0; u < UE; ++u) {
          const int t = min(t0 + u * NT_E, n - 1);
          m[u] = a.mass_in[row + t];
          p[u] = a.pos_in ? a.pos_in[row + t] : 0;
        }
#pragma unroll
        for (int u = 0; u < UE; ++u) {
          const int t = t0 + u * NT_E;
          if (t >= n) break;
          const uint32_t k = rank_key(a, m[u], p[u], recent_from);
          if (held) keys[t] = k;
          count(k);
        }
      }
    }
    __syncthreads();
    find_digit(hist, want, scratch, &sel[0], &sel[1]);
    __syncthreads();
    cut |= (uint32_t)sel[0] << shift;
    want = sel[1];
  }
  const int at_cut = (int)(cut & 1023u) * 2;
  const int equal = hist[at_cut] + hist[at_cut + 1];

  // a contiguous run of slots per wave: ballots order the slots within it,
  // the waves' counts the runs
  const int len = ((n + WE - 1) / WE + WAVE - 1) / WAVE * WAVE;
  const int lo = min(n, w * len), hi = min(n, lo + len);
  auto before = [&](int which) {
    int s = 0;
    for (int i = 0; i < w; ++i) s += counts[which][i];
    return s;
  };
  auto first = [](int k) { return k >= WAVE ? ~0ull : k <= 0 ? 0ull : (1ull << k) - 1; };   // lanes 0 .. k - 1
  int eq = 0;
  if (equal != want) {
    for (int t0 = lo; t0 < hi; t0 += WAVE) eq += __popcll(__ballot(key(min(t0 + l, n - 1)) == cut) & first(hi - t0));
    if (l == 0) counts[0][w] = eq;
    __syncthreads();
    eq = before(0);
  }
  // first the waves' counts of freed and displaced slots, then the lists; a
  // step's 64 slots are masks in scalar registers
  int holes = 0, late = 0;
  for (int pass = 0; pass < 2; ++pass) {
    int e = eq, hp = holes, lp = late;
    const bool copy = pass && a.mass_out != a.mass_in, copy_pos = pass && a.pos_in && a.pos_out != a.pos_in;
    for (int t1 = lo; t1 < hi; t1 += WAVE * UP) {
      uint32_t k[UP];
      float m[UP] = {};
      int p[UP] = {};
      if (held) {
#pragma unroll
        for (int u = 0; u < UP; ++u) k[u] = keys[min(t1 + u * WAVE + l, n - 1)];
      } else {
#pragma unroll
        for (int u = 0; u < UP; ++u) k[u] = evict_key(a, row, min(t1 + u * WAVE + l, n - 1), recent_from);
      }
      if (copy && t1 < a.budget) {
#pragma unroll
        for (int u = 0; u < UP; ++u) m[u] = a.mass_in[row + min(t1 + u * WAVE + l, n - 1)];
      }
      if (copy_pos && t1 < a.budget) {
#pragma unroll
        for (int u = 0; u < UP; ++u) p[u] = a.pos_in[row + min(t1 + u * WAVE + l, n - 1)];
      }
#pragma unroll
      for (int u = 0; u < UP; ++u) {
        const int t0 = t1 + u * WAVE, t = t0 + l;
        const uint64_t in = first(hi - t0), low = first(a.budget - t0);
        uint64_t keep = __ballot(k[u] >= cut) & in;
        if (equal != want) {      // of the slots at the cut, the first `want` of the row
          const uint64_t same = __ballot(k[u] == cut) & in;
          const uint64_t early = __ballot(e + (int)__builtin_amdgcn_mbcnt_hi((uint32_t)(same >> 32),
                                          __builtin_amdgcn_mbcnt_lo((uint32_t)same, 0)) < want);
          keep &= ~same | early;
          e += __popcll(same);
        }
        const uint64_t hole = ~keep & in & low, move = keep & ~low;
        if (pass) {
          const int hat = hp + (int)__builtin_amdgcn_mbcnt_hi((uint32_t)(hole >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)hole, 0));
          const int lat = lp + (int)__builtin_amdgcn_mbcnt_hi((uint32_t)(move >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)move, 0));
          if (hole >> l & 1) a.holes[(int64_t)bh * a.moves + hat] = t;
          if (move >> l & 1) a.late[(int64_t)bh * a.moves + lat] = t;
          if ((keep & low) >> l & 1) {
            if (copy) a.mass_out[row + t] = m[u];
            if (copy_pos) a.pos_out[row + t] = p[u];
          }
        }
        hp += __popcll(hole);
        lp += __popcll(move);
      }
    }
    if (pass == 0) {
      if (l == 0) counts[1][w] = hp, counts[2][w] = lp;
      __syncthreads();
      holes = before(1), late = before(2);
    } else if (tid == NT_E - 1) {
      a.count[bh] = lp;
    }
  }
}

// Rows of up to MV moves a round: their addresses once into LDS, then all
// loads of a round before its stores.  Bound by HBM: each moved row is read and
// written once, 370 MB in 72 us (5.1 TB/s) for 64 heads that keep 8192 of 20k to
// 32k slots.
template <int D>
__global__ __launch_bounds__(256) void k_evict_move(EvictArgs a) {
  constexpr int LPR = D / 8, RPI = 256 / LPR, IT = MV / RPI;
  __shared__ int64_t from[MV], to[MV];
  const int h = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
  const int bh = b * a.c.H + h, n = min(a.count[bh], a.moves);
  const int64_t row = (int64_t)bh * a.ld, list = (int64_t)bh * a.moves;
  const int32_t* tab = table_row(a.c, b);
  const int d = (tid % LPR) * 16;
  for (int i0 = blockIdx.x * MV; i0 < n; i0 += gridDim.x * MV) {
    if (tid < MV) {
      int64_t s = -1, t = -1;
      if (i0 + tid < n) {
        const int src = min(max(a.late[list + i0 + tid], 0), a.c.cap - 1);
        const int dst = min(max(a.holes[list + i0 + tid], 0), a.c.cap - 1);
        s = slot_offset(a.c, tab, src, h);
        t = slot_offset(a.c, tab, dst, h);
        a.mass_out[row + dst] = a.mass_in[row + src];
        if (a.pos_in) a.pos_out[row + dst] = a.pos_in[row + src];
      }
      from[tid] = t < 0 ? -1 : s;
      to[tid] = t;
    }
    __syncthreads();
    uint4 k[IT], v[IT];
#pragma unroll
    for (int u = 0; u < IT; ++u) {
      const int64_t s = from[u * RPI + tid / LPR];
      k[u] = v[u] = make_uint4(0, 0, 0, 0);
      if (s >= 0) {
        k[u] = *(const uint4*)(a.c.k + s + d);
        v[u] = *(const uint4*)(a.c.v + s + d);
      }
    }
#pragma unroll
    for (int u = 0; u < IT; ++u) {
      const int64_t t = to[u * RPI + tid / LPR];
      if (from[u * RPI + tid / LPR] >= 0) {
        *(uint4*)(a.c.k + t + d) = k[u];
        *(uint4*)(a.c.v + t + d) = v[u];
      }
    }
    __syncthreads();
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
  // heads or pages that share their memory cannot be cut apart
  if ((p->cache.head_stride == 0 && p->cache.H_kv > 1) || (p->cache.page_stride == 0 && p->cache.num_pages > 1))
    return SD_EINVAL;
  if ((int64_t)p->cache.B * p->cache.H_kv > INT32_MAX) return SD_EUNSUPPORTED;      // heads are counted in 32 bits
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
  if (!out_context) return SD_EINVAL;
  for (const int32_t* in : {args->cache.context_lens, args->node_offsets, args->path, args->path_lens, args->seen})
    if (out_context == in) return SD_EINVAL;
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
  }
  // Slots of a workgroup: 256 (one tile) unless that makes more than about
  // 1024 workgroups, since each stages the query rows anew (32 requests of 5k to
  // 16k slots: 86 us, 3 % more with 2048, 13 % with 4096).  The lengths are not
  // known here, so the table's room is what is cut: where most of it is unused,
  // the slots in use lie in few workgroups (the same requests in tables of 32768
  // slots 227 us, of 131072 597 us).
  const int64_t tiles = (a.c.cap + NT_C - 1) / NT_C;
  const int64_t per = std::max<int64_t>(1, std::min(tiles, tiles * a.c.H * a.c.B / 1024));
  const int chunk = (int)per * NT_C;
  const dim3 grid(a.mass_out ? (unsigned)((tiles + per - 1) / per) : 1u, a.c.H, a.c.B);
  if (args->cache.dtype == SD_BF16) {
    if (D == 64) hipLaunchKernelGGL((k_commit<SD_BF16, 64>), grid, dim3(NT_C), 0, st, a, chunk);
    else hipLaunchKernelGGL((k_commit<SD_BF16, 128>), grid, dim3(NT_C), 0, st, a, chunk);
  } else {
    if (D == 64) hipLaunchKernelGGL((k_commit<SD_F16, 64>), grid, dim3(NT_C), 0, st, a, chunk);
    else hipLaunchKernelGGL((k_commit<SD_F16, 128>), grid, dim3(NT_C), 0, st, a, chunk);
  }
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
  // rank keys in LDS: 16 KB leave room for other workgroups, 136 KB do not
  if (a.c.cap <= 4096)
    hipLaunchKernelGGL(k_evict_select<4096>, dim3(a.c.H, a.c.B), dim3(NT_E), 0, st, a);
  else
    hipLaunchKernelGGL(k_evict_select<34816>, dim3(a.c.H, a.c.B), dim3(NT_E), 0, st, a);
  if (hipGetLastError() != hipSuccess) return SD_EHIP;
  const int chunks = std::max(1, std::min((a.moves + MV - 1) / MV, 1024));
  const dim3 grid(chunks, a.c.H, a.c.B);
  if (args->cache.D == 64) hipLaunchKernelGGL(k_evict_move<64>, grid, dim3(256), 0, st, a);
  else hipLaunchKernelGGL(k_evict_move<128>, grid, dim3(256), 0, st, a);
  return hipGetLastError() == hipSuccess ? SD_OK : SD_EHIP;
}
