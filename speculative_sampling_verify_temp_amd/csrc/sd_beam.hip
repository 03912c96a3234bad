// Beam selection over a vocabulary and reordering of beam states on gfx950.
//
// k_beam_rows    one workgroup per (beam, slice of the vocabulary): the
//                slice's maximum, its sum of exponentials, and its n_out best
//                logits in order (larger logit, then lower id);
// k_beam_merge   one workgroup per request: each beam's log-sum-exp from its
//                slices, the candidates' scores in 64 bits, the n_out best;
// k_beam_reorder one thread per 16-byte column of a state row: the column of
//                every source beam that another beam takes over is read
//                before any is written, so the rows permute in place.
#include <algorithm>

#include "sdt_device.h"

using namespace sdv;
using namespace sdt;

namespace {

constexpr int NT_B = 256;
constexpr int MAXO = SD_MAX_BEAMS;

struct SliceOut {
  float m;        // maximum, NaN where the slice holds a NaN or +inf
  float pad;
  double s;       // sum of exp(z - m)
  uint64_t best[MAXO];   // ord_key(z) << 32 | ~id, descending; 0: none
};

struct BeamArgs {
  const char* logits;
  int64_t row_bytes;
  const float* scores;
  const uint8_t* ended;
  int B, W, V, n_out, eos, slices, slice_vecs;
  SliceOut* part;   // [B * W][slices]
  float* out_scores;
  int32_t *out_parents, *out_tokens;
  uint8_t* out_ended;
  uint32_t* status;
};

__device__ __forceinline__ bool examined(const BeamArgs& a, int bw) {
  return !(a.ended && a.ended[bw]) && a.scores[bw] > -INFINITY;
}

__device__ __forceinline__ uint64_t wave_max_u64(uint64_t x) {
#pragma unroll
  for (int o = WAVE / 2; o > 0; o >>= 1) {
    const uint64_t y = __shfl_xor(x, o);
    x = y > x ? y : x;
  }
  return x;
}

__device__ __forceinline__ uint64_t block_max_u64(uint64_t x, uint64_t* scratch) {
  x = wave_max_u64(x);
  __syncthreads();
  if (threadIdx.x % WAVE == 0) scratch[threadIdx.x / WAVE] = x;
  __syncthreads();
  for (int w = 0; w < NT_B / WAVE; ++w) x = scratch[w] > x ? scratch[w] : x;
  return x;
}

template <int DT>
__device__ __forceinline__ float logit(const char* row, int i) {
  if constexpr (DT == SD_BF16) return __uint_as_float((uint32_t)((const uint16_t*)row)[i] << 16);
  return ((const float*)row)[i];
}

template <int DT>
__global__ __launch_bounds__(NT_B) void k_beam_rows(BeamArgs a) {
  constexpr int E = DT == SD_BF16 ? 8 : 4;
  __shared__ float sf[NT_B / WAVE];
  __shared__ double sd[NT_B / WAVE];
  __shared__ int si[NT_B / WAVE];
  __shared__ uint64_t su[NT_B / WAVE];
  const int bw = blockIdx.x, sl = blockIdx.y, tid = threadIdx.x;
  if (!examined(a, bw)) return;
  const char* row = a.logits + bw * a.row_bytes;
  const int lo = sl * a.slice_vecs * E, hi = min(a.V, lo + a.slice_vecs * E);
  SliceOut& out = a.part[(int64_t)bw * a.slices + sl];
  float m = -INFINITY;
  int bad = 0;
  for (int i = lo + tid; i < hi; i += NT_B) {
    const float z = logit<DT>(row, i);
    bad |= nonfinite(z);
    m = fmaxf(m, z);
  }
  bad = block_or<NT_B>(bad, si);
  m = block_max<NT_B>(m, sf);
  double s = 0.0;
  if (!bad && m > -INFINITY)
    for (int i = lo + tid; i < hi; i += NT_B) s += (double)expf(logit<DT>(row, i) - m);
  s = block_sum<NT_B>(s, sd);
  if (tid == 0) out.m = bad ? __builtin_nanf("") : m, out.s = s;
  uint64_t last = ~0ull;
  for (int j = 0; j < a.n_out; ++j) {
    uint64_t best = 0;
    for (int i = lo + tid; !bad && i < hi; i += NT_B) {
      const float z = logit<DT>(row, i);
      const uint64_t k = z > -INFINITY ? ((uint64_t)ord_key(z) << 32) | (uint32_t)~i : 0;
      if (k < last && k > best) best = k;
    }
    last = block_max_u64(best, su);
    if (tid == 0) out.best[j] = last;
    if (last == 0) last = 1;   // nothing is below: the rest of the list is empty
  }
}

// A score as a key whose order is the score's.
__device__ __forceinline__ uint64_t ord64(double x) {
  const uint64_t u = (uint64_t)__double_as_longlong(x == 0.0 ? 0.0 : x);
  return (u >> 63) ? ~u : (u | (1ull << 63));
}

__device__ __forceinline__ float from_ord32(uint32_t o) {
  return __uint_as_float((o & 0x80000000u) ? o & 0x7FFFFFFFu : ~o);
}

__global__ __launch_bounds__(NT_B) void k_beam_merge(BeamArgs a) {
  __shared__ double lse[MAXO];
  __shared__ uint32_t st_sh;
  __shared__ uint64_t su[NT_B / WAVE];
  const int b = blockIdx.x, tid = threadIdx.x;
  if (tid == 0) st_sh = 0;
  __syncthreads();
  if (tid < a.W) {
    const int bw = b * a.W + tid;
    const float sc = a.scores[bw];
    uint32_t st = 0;
    double e = 0.0;
    if (sc != sc || sc == INFINITY) st |= SD_ST_BAD_PARAM;
    else if (examined(a, bw)) {
      const SliceOut* p = a.part + (int64_t)bw * a.slices;
      float m = -INFINITY;
      for (int s = 0; s < a.slices; ++s) {
        if (p[s].m != p[s].m) st |= SD_ST_NONFINITE;
        m = fmaxf(m, p[s].m);
      }
      if (!(m > -INFINITY)) st |= SD_ST_NONFINITE;
      double z = 0.0;
      for (int s = 0; s < a.slices; ++s)
        if (p[s].s > 0.0) z += p[s].s * exp((double)p[s].m - (double)m);
      e = (double)m + log(z);
    }
    lse[tid] = e;
    if (st) atomicOr(&st_sh, st);
  }
  __syncthreads();
  const bool bad = st_sh != 0;
  const int total = bad ? 0 : a.W * a.slices * a.n_out;
  uint64_t last_s = ~0ull, last_i = 0;   // the candidate chosen before, by score and then by place
  for (int j = 0; j < a.n_out; ++j) {
    uint64_t bs = 0, bi = 0;             // score key and ~place of the best below it
    double bx = -INFINITY;
    for (int c = tid; c < total; c += NT_B) {
      const int w = c / (a.slices * a.n_out), r = c % (a.slices * a.n_out), bw = b * a.W + w;
      double x;
      int id;
      if (a.ended && a.ended[bw]) {
        if (r) continue;
        x = a.scores[bw], id = a.eos;
      } else {
        if (!examined(a, bw)) continue;
        const uint64_t k = a.part[(int64_t)bw * a.slices + r / a.n_out].best[r % a.n_out];
        if (k == 0) continue;
        id = (int)~(uint32_t)k;
        x = (double)a.scores[bw] + ((double)from_ord32((uint32_t)(k >> 32)) - lse[w]);
      }
      if (!(x > -INFINITY)) continue;
      const uint64_t s = ord64(x), i = ~((uint64_t)w << 32 | (uint32_t)id);
      if (s > last_s || (s == last_s && i >= last_i)) continue;
      if (s > bs || (s == bs && i > bi)) bs = s, bi = i, bx = x;
    }
    const uint64_t s = block_max_u64(bs, su);
    const uint64_t i = block_max_u64(bs == s ? bi : 0, su);
    last_s = s, last_i = i;
    const int o = b * a.n_out + j;
    if (s == 0 ? tid == 0 : (bs == s && bi == i)) {
      const int w = s ? (int)(~i >> 32) : -1, id = s ? (int)(uint32_t)~i : -1;
      a.out_scores[o] = s ? (float)bx : -INFINITY;
      a.out_parents[o] = w;
      a.out_tokens[o] = id;
      if (a.out_ended) a.out_ended[o] = s && ((a.ended && a.ended[b * a.W + w]) || id == a.eos);
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

__global__ __launch_bounds__(256) void k_beam_reorder(ReorderArgs a) {
  __shared__ int par[MAXO];
  const int b = blockIdx.y, ls = blockIdx.z, layer = ls / a.segs, seg = ls % a.segs;
  if (threadIdx.x < a.W_out) {
    const int p = a.parents[b * a.W_out + threadIdx.x];
    par[threadIdx.x] = p >= 0 && p < a.W_in ? p : -1;
  }
  __syncthreads();
  const int len = a.lengths ? min(max(a.lengths[b], 0), a.max_units) : a.max_units;
  const int64_t cols = len * a.unit / 16;
  const bool same = a.in == a.out;
  const char* src = a.in + layer * a.in_layer + b * a.in_request + seg * a.in_seg;
  char* dst = a.out + layer * a.out_layer + b * a.out_request + seg * a.out_seg;
  for (int64_t c = blockIdx.x * 256 + threadIdx.x; c < cols; c += gridDim.x * 256) {
    uint4 v[MAXO];
    for (int w = 0; w < a.W_out; ++w)
      if (par[w] >= 0 && !(same && par[w] == w)) v[w] = *(const uint4*)(src + par[w] * a.in_beam + c * 16);
    for (int w = 0; w < a.W_out; ++w)
      if (par[w] >= 0 && !(same && par[w] == w)) *(uint4*)(dst + w * a.out_beam + c * 16) = v[w];
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
  return SD_OK;
}

int slice_count(int rows, int nvec) {
  return std::max(1, std::min({(1024 + rows - 1) / rows, (nvec + 511) / 512, 64}));
}

}  // namespace

extern "C" int sd_beam_select_workspace_bytes(const sd_beam_select_args_t* args, size_t* bytes) {
  if (!bytes) return SD_EINVAL;
  const int rc = check(args);
  if (rc) return rc;
  const int E = args->dtype == SD_BF16 ? 8 : 4, rows = args->B * args->W;
  *bytes = (size_t)rows * slice_count(rows, (args->V + E - 1) / E) * sizeof(SliceOut);
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
  const int E = args->dtype == SD_BF16 ? 8 : 4, nvec = (args->V + E - 1) / E;
  BeamArgs a;
  a.logits = static_cast<const char*>(args->logits);
  a.row_bytes = args->ld * (16 / E);
  a.scores = args->scores, a.ended = args->ended;
  a.B = args->B, a.W = args->W, a.V = args->V, a.n_out = args->n_out, a.eos = args->eos_id;
  a.slices = slice_count(a.B * a.W, nvec);
  a.slice_vecs = (nvec + a.slices - 1) / a.slices;
  a.part = static_cast<SliceOut*>(workspace);
  a.out_scores = out_scores, a.out_parents = out_parents, a.out_tokens = out_tokens;
  a.out_ended = out_ended, a.status = out_status;
  hipStream_t st = static_cast<hipStream_t>(stream);
  const dim3 grid(a.B * a.W, a.slices);
  if (args->dtype == SD_BF16) hipLaunchKernelGGL(k_beam_rows<SD_BF16>, grid, dim3(NT_B), 0, st, a);
  else hipLaunchKernelGGL(k_beam_rows<SD_F32>, grid, dim3(NT_B), 0, st, a);
  if (hipGetLastError() != hipSuccess) return SD_EHIP;
  hipLaunchKernelGGL(k_beam_merge, dim3(a.B), dim3(NT_B), 0, st, a);
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
  hipLaunchKernelGGL(k_beam_reorder, grid, dim3(256), 0, static_cast<hipStream_t>(stream), a);
  return hipGetLastError() == hipSuccess ? SD_OK : SD_EHIP;
}
