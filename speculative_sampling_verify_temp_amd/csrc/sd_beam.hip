// Beam selection over a vocabulary and reordering of beam states on gfx950.
//
// k_beam_rows    one workgroup per (beam, slice of the vocabulary), the slice in
//                registers: its maximum, its sum of exponentials and its n_out
//                best logits in order (larger logit, then lower id);
// k_beam_merge   one workgroup per request: each beam's maximum and the logarithm
//                of its sum from its slices, the candidates' scores in 64 bits,
//                the n_out best.
//
// Both choose the n best of many in the same way: the n-th largest of 64 maxima,
// each of a 64th of the threads, bounds the n-th largest of all from below, so
// only the values not below it (about n, 300 at n = 64) are listed and ranked by
// counting the larger ones.  Where ties make that list overflow the best are
// taken one by one.
// k_beam_reorder one thread per 16-byte column of a state row: the column of
//                every source beam that another beam takes over is read
//                before any is written, so the rows permute in place.
#include <algorithm>

#include "sdt_device.h"

using namespace sdv;
using namespace sdt;

namespace {

constexpr int NT_B = 256;
constexpr int NT_M = 1024;       // threads of a merge
constexpr int NV = 4;            // 16-byte vectors of a thread's part of a slice
constexpr int LIST = 1024;       // places for the values not below the bound
constexpr int MAXO = SD_MAX_BEAMS;

struct BeamArgs {
  const char* logits;
  int64_t row_bytes;
  const float* scores;
  const uint8_t* ended;
  int B, W, V, n_out, eos, slices, slice_vecs;
  float* part_m;       // [B * W][slices] maximum, NaN where the slice holds a NaN or +inf
  double* part_s;      // sum of exp(z - maximum)
  uint64_t* part_best; // [B * W][slices][n_out]: ord_key(z) << 32 | ~id, descending; 0: none
  float* out_scores;
  int32_t *out_parents, *out_tokens;
  uint8_t* out_ended;
  uint32_t* status;
};

__device__ __forceinline__ bool examined(const BeamArgs& a, int bw) {
  return !(a.ended && a.ended[bw]) && a.scores[bw] > -INFINITY;
}

template <int NT>
__device__ __forceinline__ uint64_t block_max_u64(uint64_t x, uint64_t* scratch) {
  x = wave_max_u64(x);
  __syncthreads();
  if (threadIdx.x % WAVE == 0) scratch[threadIdx.x / WAVE] = x;
  __syncthreads();
  for (int w = 0; w < NT / WAVE; ++w) x = scratch[w] > x ? scratch[w] : x;
  return x;
}

template <int LANES, typename K>
__device__ __forceinline__ K lanes_max(K x) {
#pragma unroll
  for (int o = 1; o < LANES; o <<= 1) {
    const K y = __shfl_xor(x, o);
    x = y > x ? y : x;
  }
  return x;
}

// The n-th largest (n <= 64) of the 64 keys in LDS, in every thread: bit by bit
// from the top, the largest value that n of a wave's 64 lanes reach.  Bits below
// LOW are the same in all keys of one sign: n lanes that reach a value with them
// clear are enough of a bound.
template <int LOW, typename K>
__device__ __forceinline__ K nth_of_64(const K* keys, int n) {
  const K k = keys[threadIdx.x % WAVE];
  K edge = 0;
#pragma unroll
  for (int bit = (int)sizeof(K) * 8 - 1; bit >= LOW; --bit) {
    const K c = edge | (K)1 << bit;
    if (__popcll(__ballot(k >= c)) >= n) edge = c;
  }
  return edge;
}

// Logit e of a 16-byte vector.
template <int DT>
__device__ __forceinline__ float logit_of(const uint4& w, int e) {
  const uint32_t q[4] = {w.x, w.y, w.z, w.w};
  if constexpr (DT == SD_BF16) return __uint_as_float(e & 1 ? q[e / 2] & 0xFFFF0000u : q[e / 2] << 16);
  return __uint_as_float(q[e]);
}

// A logit is read once and its exponential costs about 8 issue slots; with the
// bound and the list, which every slice makes anew, the vector ALU is the limit:
// 26.6 us for 256 rows of 152064 bf16 logits, a fifth of them ended (62 MB, 2.3
// TB/s).  Slices of 4 vectors a
// thread beat 8 (34 against 36 us: more workgroups a CU hide the two
// synchronizations).
template <int DT>
__global__ __launch_bounds__(NT_B, 6) void k_beam_rows(BeamArgs a) {
  constexpr int E = DT == SD_BF16 ? 8 : 4;
  __shared__ float sf[NT_B / WAVE];
  __shared__ double sd[NT_B / WAVE];
  __shared__ uint64_t su[NT_B / WAVE];
  __shared__ __align__(16) uint32_t keys[WAVE];
  __shared__ uint64_t list[LIST];
  __shared__ int listed;
  const int bw = blockIdx.x, sl = blockIdx.y, tid = threadIdx.x;
  if (!examined(a, bw)) return;
  const int64_t out = (int64_t)bw * a.slices + sl;
  const uint4* const row = reinterpret_cast<const uint4*>(a.logits + bw * a.row_bytes);
  const int nvec = (a.V + E - 1) / E, lo = sl * a.slice_vecs, hi = min(nvec, lo + a.slice_vecs);
  const int mine = (hi - lo + NT_B - 1) / NT_B;      // vectors a thread takes
  if (tid == 0) listed = 0;
  uint4 w[NV];
#pragma unroll
  for (int u = 0; u < NV; ++u) {
    w[u] = make_uint4(0, 0, 0, 0);
    if (u < mine) w[u] = row[min(lo + u * NT_B + tid, hi - 1)];
  }
  // past the end: -inf, which is no candidate and adds nothing
  constexpr uint32_t NINF = DT == SD_BF16 ? 0xFF80FF80u : 0xFF800000u;
  const bool tail = hi == nvec && a.V % E != 0;
#pragma unroll
  for (int u = 0; u < NV; ++u) {
    const int k = lo + u * NT_B + tid;
    if (u >= mine || k >= hi) {
      w[u] = make_uint4(NINF, NINF, NINF, NINF);
    } else if (tail && k == nvec - 1) {
      uint32_t q[4] = {w[u].x, w[u].y, w[u].z, w[u].w};
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (k * E + e >= a.V) {
          if constexpr (DT == SD_BF16)
            q[e / 2] = e & 1 ? (q[e / 2] & 0xFFFFu) | 0xFF800000u : (q[e / 2] & 0xFFFF0000u) | 0xFF80u;
          else
            q[e] = NINF;
        }
      w[u] = make_uint4(q[0], q[1], q[2], q[3]);
    }
  }
  bool nan = false;
  float vtop[NV], top = -INFINITY;
#pragma unroll
  for (int u = 0; u < NV; ++u) {
    Extremes<DT> x;
    x.clear();
    x.add(w[u].x);
    x.add(w[u].y);
    x.add(w[u].z);
    x.add(w[u].w);
    vtop[u] = x.value(nan);
    top = fmaxf(top, vtop[u]);
  }
  if (nan) top = INFINITY;           // reported like one
  // exponentials against the thread's own maximum: at most 32 terms of at most
  // 1 in fp32; the threads' sums meet in 64 bits.  The maximum is taken off before
  // the scaling: the term of the maximum is exactly 1 whatever the logits' level,
  // and the lowest finite logits, as masks hold them, stay in range.
  constexpr float C = 1.4426950408889634f;
  float s = 0.0f;
  if (top > -INFINITY && top < INFINITY) {
#pragma unroll
    for (int u = 0; u < NV; ++u)
      if (u < mine) {
#pragma unroll
        for (int e = 0; e < E; ++e) s += fast_exp2((logit_of<DT>(w[u], e) - top) * C);
      }
  }
  const uint32_t o = ord_key(top), group = lanes_max<4>(o);
  const float wtop = wave_max(top);
  if (tid % 4 == 0) keys[tid / 4] = group;
  if (tid % WAVE == 0) sf[tid / WAVE] = wtop;
  __syncthreads();
  float m = sf[0];
#pragma unroll
  for (int i = 1; i < NT_B / WAVE; ++i) m = fmaxf(m, sf[i]);
  if (m == INFINITY) {
    if (tid == 0) a.part_m[out] = __builtin_nanf("");
    return;
  }
  const uint32_t floor = ord_key(-INFINITY);         // not a candidate
  const uint32_t edge = nth_of_64<DT == SD_BF16 ? 16 : 0>(keys, a.n_out);
  const double part = wave_sum(top > -INFINITY ? (double)s * (double)fast_exp2((top - m) * C) : 0.0);
  if (tid % WAVE == 0) sd[tid / WAVE] = part;
  uint64_t* const best = a.part_best + out * a.n_out;
#pragma unroll
  for (int u = 0; u < NV; ++u)
    if (ord_key(vtop[u]) >= edge && vtop[u] > -INFINITY) {
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const uint32_t k = ord_key(logit_of<DT>(w[u], e));
        if (k >= edge && k > floor) {
          const int at = atomicAdd(&listed, 1);
          if (at < LIST) list[at] = ((uint64_t)k << 32) | (uint32_t)~((lo + u * NT_B + tid) * E + e);
        }
      }
    }
  __syncthreads();
  if (tid == 0) {
    double total = 0.0;
    for (int i = 0; i < NT_B / WAVE; ++i) total += sd[i];
    a.part_m[out] = m, a.part_s[out] = total;
  }
  const int n = listed;
  if (n <= LIST) {
    for (int i = tid; i < n; i += NT_B) {
      const uint64_t k = list[i];
      int rank = 0;
      for (int j = 0; j < n; ++j) rank += list[j] > k;
      if (rank < a.n_out) best[rank] = k;
    }
    for (int j = n + tid; j < a.n_out; j += NT_B) best[j] = 0;
    return;
  }
  uint64_t last = ~0ull;
  for (int j = 0; j < a.n_out; ++j) {
    uint64_t b = 0;
#pragma unroll
    for (int u = 0; u < NV; ++u)
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const uint32_t o = ord_key(logit_of<DT>(w[u], e));
        const uint64_t k = ((uint64_t)o << 32) | (uint32_t)~((lo + u * NT_B + tid) * E + e);
        if (o > floor && k < last && k > b) b = k;
      }
    last = block_max_u64<NT_B>(b, su);
    if (tid == 0) best[j] = last;
  }
}

// A score as a key whose order is the score's.
__device__ __forceinline__ uint64_t ord64(double x) {
  const uint64_t u = (uint64_t)__double_as_longlong(x == 0.0 ? 0.0 : x);
  return (u >> 63) ? ~u : (u | (1ull << 63));
}

__device__ __forceinline__ double from_ord64(uint64_t o) {
  return __longlong_as_double((long long)((o >> 63) ? o & ~(1ull << 63) : ~o));
}

__device__ __forceinline__ float from_ord32(uint32_t o) {
  return __uint_as_float((o & 0x80000000u) ? o & 0x7FFFFFFFu : ~o);
}

// A candidate: its score as a key, and ~(beam << 32 | token), so that the better
// of two is the larger pair; s = 0: none.
struct Candidate {
  uint64_t s, i;
  __device__ bool over(const Candidate& o) const { return s > o.s || (s == o.s && i > o.i); }
};

// Latency: 8 us for 8 beams of 19 slices (14 us with 256 threads, which took the
// beams four at a time).
__global__ __launch_bounds__(NT_M) void k_beam_merge(BeamArgs a) {
  // log-sum-exp = top + rest, kept apart: where the logits are far from zero (a
  // row of nothing but masks) their sum would lose the rest, even in 64 bits
  __shared__ double rest[MAXO];
  __shared__ float top_of[MAXO];
  __shared__ uint8_t kind[MAXO];      // 0: no candidates, 1: its slices', 2: ended
  __shared__ uint32_t st_sh;
  __shared__ __align__(16) uint64_t keys[WAVE];
  __shared__ uint64_t su[NT_M / WAVE], list_s[LIST], list_i[LIST];
  __shared__ float score[MAXO];
  __shared__ int listed;
  const int b = blockIdx.x, tid = threadIdx.x, l = tid % WAVE;
  if (tid == 0) st_sh = 0, listed = 0;
  __syncthreads();
  for (int w = tid / WAVE; w < a.W; w += NT_M / WAVE) {
    const int bw = b * a.W + w;
    const float sc = a.scores[bw];
    uint32_t st = 0;
    float m = -INFINITY;
    double e = 0.0;
    const int kd = !(sc > -INFINITY) ? 0 : a.ended && a.ended[bw] ? 2 : 1;
    if (sc != sc || sc == INFINITY) st |= SD_ST_BAD_PARAM;
    if (kd == 1 && !st) {
      const float* pm = a.part_m + (int64_t)bw * a.slices;
      const double* ps = a.part_s + (int64_t)bw * a.slices;
      bool bad = false;
      for (int s = l; s < a.slices; s += WAVE) {
        bad |= pm[s] != pm[s];
        m = fmaxf(m, pm[s]);
      }
      m = wave_max(m);
      if (__any(bad) || !(m > -INFINITY)) st |= SD_ST_NONFINITE;
      else {
        double z = 0.0;
        for (int s = l; s < a.slices; s += WAVE)
          if (pm[s] > -INFINITY) z += ps[s] * exp((double)pm[s] - (double)m);
        e = log(wave_sum(z));
      }
    }
    if (l == 0) {
      rest[w] = e, top_of[w] = m, kind[w] = (uint8_t)kd, score[w] = sc;
      if (st) atomicOr(&st_sh, st);
    }
  }
  __syncthreads();
  const bool bad = st_sh != 0;
  const int per = a.slices * a.n_out, total = bad ? 0 : a.W * per;
  auto candidate = [&](int c) {
    const int w = c / per, r = c % per;
    Candidate x{0, 0};
    double sc = -INFINITY;
    int id = a.eos;
    if (kind[w] == 2) {
      if (r == 0) sc = score[w];
    } else if (kind[w] == 1) {
      const uint64_t k = a.part_best[(int64_t)b * a.W * per + c];
      if (k) {
        id = (int)~(uint32_t)k;
        sc = (double)score[w] + (((double)from_ord32((uint32_t)(k >> 32)) - (double)top_of[w]) - rest[w]);
      }
    }
    if (sc > -INFINITY) x.s = ord64(sc), x.i = ~((uint64_t)w << 32 | (uint32_t)id);
    return x;
  };
  auto put = [&](int j, const Candidate& x) {
    const int o = b * a.n_out + j;
    const int w = x.s ? (int)(~x.i >> 32) : -1, id = x.s ? (int)(uint32_t)~x.i : -1;
    a.out_scores[o] = x.s ? (float)from_ord64(x.s) : -INFINITY;
    a.out_parents[o] = w;
    a.out_tokens[o] = id;
    if (a.out_ended) a.out_ended[o] = x.s && (kind[w] == 2 || id == a.eos);
  };
  uint64_t top = 0;
  for (int c = tid; c < total; c += NT_M) top = max(top, candidate(c).s);
  const uint64_t group = lanes_max<NT_M / WAVE>(top);
  if (tid % (NT_M / WAVE) == 0) keys[tid / (NT_M / WAVE)] = group;
  __syncthreads();
  const uint64_t edge = nth_of_64<0>(keys, a.n_out);
  if (top >= edge && top) {
    for (int c = tid; c < total; c += NT_M) {
      const Candidate x = candidate(c);
      if (x.s >= edge && x.s) {
        const int at = atomicAdd(&listed, 1);
        if (at < LIST) list_s[at] = x.s, list_i[at] = x.i;
      }
    }
  }
  __syncthreads();
  const int n = listed;
  if (n <= LIST) {
    for (int i = tid; i < n; i += NT_M) {
      const Candidate x{list_s[i], list_i[i]};
      int rank = 0;
      for (int j = 0; j < n; ++j) rank += Candidate{list_s[j], list_i[j]}.over(x);
      if (rank < a.n_out) put(rank, x);
    }
    for (int j = n + tid; j < a.n_out; j += NT_M) put(j, Candidate{0, 0});
  } else {
    Candidate last{~0ull, ~0ull};
    for (int j = 0; j < a.n_out; ++j) {
      Candidate best{0, 0};
      for (int c = tid; c < total; c += NT_M) {
        const Candidate x = candidate(c);
        if (last.over(x) && x.over(best)) best = x;
      }
      const uint64_t s = block_max_u64<NT_M>(best.s, su);
      const uint64_t i = block_max_u64<NT_M>(best.s == s ? best.i : 0, su);
      last = Candidate{s, i};
      if (tid == 0) put(j, last);
    }
  }
  if (tid == 0 && a.status) a.status[b] = st_sh;
}

struct ReorderArgs {
  const char* in;
  char* out;
  int64_t in_layer, in_request, in_beam, in_seg, out_layer, out_request, out_beam, out_seg;
  const int32_t *parents, *lengths;
  int64_t unit;
  int layers, B, W_in, W_out, segs, max_units;
};

// One 16-byte column of all beams a thread, in registers between its loads and
// its stores; WM bounds the beams, so that they are registers.  Bound by HBM:
// beams that keep their place cost nothing, the rest are read and written once
// (32 requests of 8 beams, 4 layers, up to 512 units of 128 bytes: 36 us).
template <int WM>
__global__ __launch_bounds__(256) void k_beam_reorder(ReorderArgs a) {
  __shared__ int par[WM];
  const int b = blockIdx.y, ls = blockIdx.z, layer = ls / a.segs, seg = ls % a.segs;
  const bool same = a.in == a.out;
  if ((int)threadIdx.x < WM) {
    const int w = threadIdx.x, p = w < a.W_out ? a.parents[b * a.W_out + w] : -1;
    par[w] = p >= 0 && p < a.W_in && !(same && p == w) ? p : -1;     // -1: nothing to move
  }
  __syncthreads();
  const int len = a.lengths ? min(max(a.lengths[b], 0), a.max_units) : a.max_units;
  const int64_t cols = len * a.unit / 16;
  const char* src = a.in + layer * a.in_layer + b * a.in_request + seg * a.in_seg;
  char* dst = a.out + layer * a.out_layer + b * a.out_request + seg * a.out_seg;
  for (int64_t c = blockIdx.x * 256 + threadIdx.x; c < cols; c += gridDim.x * 256) {
    uint4 v[WM];
#pragma unroll
    for (int w = 0; w < WM; ++w) {
      const int p = __builtin_amdgcn_readfirstlane(par[w]);
      v[w] = make_uint4(0, 0, 0, 0);
      if (p >= 0) v[w] = *(const uint4*)(src + p * a.in_beam + c * 16);
    }
#pragma unroll
    for (int w = 0; w < WM; ++w) {
      const int p = __builtin_amdgcn_readfirstlane(par[w]);
      if (p >= 0) *(uint4*)(dst + w * a.out_beam + c * 16) = v[w];
    }
  }
}

int check(const sd_beam_select_args_t* p) {
  if (!p || !p->logits || !aligned16(p->logits) || !p->scores) return SD_EINVAL;
  if (p->dtype != SD_F32 && p->dtype != SD_BF16) return SD_EINVAL;
  const int es = p->dtype == SD_BF16 ? 2 : 4;
  if (p->B < 1 || p->W < 1 || p->V < 1 || p->n_out < 1 || p->ld < p->V || (p->ld * es) % 16)
    return SD_EINVAL;
  if (p->W > SD_MAX_BEAMS || p->n_out > SD_MAX_BEAMS || p->V >= (1 << 24) || p->B > (1 << 20))
    return SD_EUNSUPPORTED;
  // a grid dimension holds less than 2^32 threads
  if ((int64_t)p->B * p->W * NT_B > UINT32_MAX) return SD_EUNSUPPORTED;
  return SD_OK;
}

// Vectors of a slice: one per thread until that makes more than about 1024
// workgroups, at most NV.
int slice_vectors(int rows, int nvec) {
  const int64_t per = ((int64_t)rows * nvec / 1024 + NT_B - 1) / NT_B;
  return NT_B * (int)std::clamp<int64_t>(per, 1, NV);
}

struct BeamLayout {
  int slice_vecs, slices;
  size_t m, s, best, total;    // byte offsets
};

BeamLayout layout(const sd_beam_select_args_t* p) {
  const int E = p->dtype == SD_BF16 ? 8 : 4, nvec = (p->V + E - 1) / E, rows = p->B * p->W;
  BeamLayout L;
  L.slice_vecs = slice_vectors(rows, nvec);
  L.slices = (nvec + L.slice_vecs - 1) / L.slice_vecs;
  const size_t n = (size_t)rows * L.slices;
  L.best = 0;
  L.s = n * p->n_out * 8;
  L.m = L.s + n * 8;
  L.total = L.m + n * 4;
  return L;
}

}  // namespace

extern "C" int sd_beam_select_workspace_bytes(const sd_beam_select_args_t* args, size_t* bytes) {
  if (!bytes) return SD_EINVAL;
  const int rc = check(args);
  if (rc) return rc;
  *bytes = layout(args).total;
  return SD_OK;
}

extern "C" int sd_beam_select(const sd_beam_select_args_t* args, void* workspace,
                              size_t workspace_bytes, float* out_scores, int32_t* out_parents,
                              int32_t* out_tokens, uint8_t* out_ended, uint32_t* out_status,
                              void* stream) {
  size_t need = 0;
  const int rc = sd_beam_select_workspace_bytes(args, &need);
  if (rc) return rc;
  if (!out_scores || !out_parents || !out_tokens || out_scores == args->scores ||
      (out_ended && out_ended == args->ended))
    return SD_EINVAL;
  if (!workspace || workspace_bytes < need || (uintptr_t)workspace % 8) return SD_EWORKSPACE;
  const BeamLayout L = layout(args);
  char* const ws = static_cast<char*>(workspace);
  BeamArgs a;
  a.logits = static_cast<const char*>(args->logits);
  a.row_bytes = args->ld * (args->dtype == SD_BF16 ? 2 : 4);
  a.scores = args->scores, a.ended = args->ended;
  a.B = args->B, a.W = args->W, a.V = args->V, a.n_out = args->n_out, a.eos = args->eos_id;
  a.slices = L.slices, a.slice_vecs = L.slice_vecs;
  a.part_m = reinterpret_cast<float*>(ws + L.m);
  a.part_s = reinterpret_cast<double*>(ws + L.s);
  a.part_best = reinterpret_cast<uint64_t*>(ws + L.best);
  a.out_scores = out_scores, a.out_parents = out_parents, a.out_tokens = out_tokens;
  a.out_ended = out_ended, a.status = out_status;
  hipStream_t st = static_cast<hipStream_t>(stream);
  const dim3 grid(a.B * a.W, a.slices);
  if (args->dtype == SD_BF16) hipLaunchKernelGGL(k_beam_rows<SD_BF16>, grid, dim3(NT_B), 0, st, a);
  else hipLaunchKernelGGL(k_beam_rows<SD_F32>, grid, dim3(NT_B), 0, st, a);
  if (hipGetLastError() != hipSuccess) return SD_EHIP;
  hipLaunchKernelGGL(k_beam_merge, dim3(a.B), dim3(NT_M), 0, st, a);
  return hipGetLastError() == hipSuccess ? SD_OK : SD_EHIP;
}

extern "C" int sd_beam_reorder(const sd_beam_reorder_args_t* p, void* stream) {
  if (!p || !p->in || !p->out || !aligned16(p->in) || !aligned16(p->out) || !p->parents) return SD_EINVAL;
  if (p->layers < 1 || p->B < 1 || p->W_in < 1 || p->W_out < 1 || p->segs < 1 || p->max_units < 1 ||
      p->unit_bytes < 16)
    return SD_EINVAL;
  const int64_t strides[] = {p->in_layer, p->in_request, p->in_beam, p->in_seg, p->out_layer,
                             p->out_request, p->out_beam, p->out_seg, p->unit_bytes};
  for (int64_t s : strides)
    if (s < 0 || s % 16) return SD_EINVAL;
  // rows of out that share their memory
  if ((p->out_layer == 0 && p->layers > 1) || (p->out_request == 0 && p->B > 1) ||
      (p->out_beam == 0 && p->W_out > 1) || (p->out_seg == 0 && p->segs > 1))
    return SD_EINVAL;
  if (p->in == p->out && (p->W_in != p->W_out || p->in_layer != p->out_layer ||
                          p->in_request != p->out_request || p->in_beam != p->out_beam ||
                          p->in_seg != p->out_seg))
    return SD_EINVAL;
  if (p->W_in > SD_MAX_BEAMS || p->W_out > SD_MAX_BEAMS || p->B > 65535 ||
      (int64_t)p->layers * p->segs > 65535)
    return SD_EUNSUPPORTED;
  ReorderArgs a;
  a.in = static_cast<const char*>(p->in);
  a.out = static_cast<char*>(p->out);
  a.in_layer = p->in_layer, a.in_request = p->in_request, a.in_beam = p->in_beam, a.in_seg = p->in_seg;
  a.out_layer = p->out_layer, a.out_request = p->out_request, a.out_beam = p->out_beam, a.out_seg = p->out_seg;
  a.parents = p->parents, a.lengths = p->lengths;
  a.unit = p->unit_bytes;
  a.layers = p->layers, a.B = p->B, a.W_in = p->W_in, a.W_out = p->W_out, a.segs = p->segs;
  a.max_units = p->max_units;
  const int64_t cols = p->max_units * p->unit_bytes / 16;
  const dim3 grid((unsigned)std::min<int64_t>((cols + 255) / 256, 1024), a.B, a.layers * a.segs);
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (a.W_out <= 4) hipLaunchKernelGGL(k_beam_reorder<4>, grid, dim3(256), 0, st, a);
  else if (a.W_out <= 8) hipLaunchKernelGGL(k_beam_reorder<8>, grid, dim3(256), 0, st, a);
  else if (a.W_out <= 16) hipLaunchKernelGGL(k_beam_reorder<16>, grid, dim3(256), 0, st, a);
  else hipLaunchKernelGGL(k_beam_reorder<MAXO>, grid, dim3(256), 0, st, a);
  return hipGetLastError() == hipSuccess ? SD_OK : SD_EHIP;
}
