// Norms of queries and keys with the position rotation on gfx950.
//
// y = x / sqrt(mean(x^2) + eps) * w per head, then pairs of y are turned by
// position * inv_freq.  One read and one write of every element: bound by HBM
// for prompts, by latency for the nodes of a verify.
//
// A workgroup takes a few tokens with all their heads, so that a token's sines
// and cosines are computed once, into LDS, while the rows are on their way.
// D / 16 lanes share a row, 16 elements each: a lane's two vectors hold both
// elements of its pairs, so a row needs no exchange but the sum of squares.
// 16411 tokens of 28 + 4 heads of 128: 49 us, 5.5 TB/s; 288 tokens of 16 + 8 heads:
// 4.2 us; one token of 14 + 2 heads of 64: 2.4 us.
#include <algorithm>

#include "sd_serve.h"
#include "sdt_device.h"

using namespace sdv;
using namespace sdt;

namespace {

constexpr int NT_R = 256;
constexpr int MAX_TURNS = 1024;     // (token, frequency)s of a workgroup

struct RopeArgs {
  const char *q, *k;
  char *qo, *ko;
  int64_t q_node, q_head, k_node, k_head, qo_node, qo_head, ko_node, ko_head;   // bytes
  const char *wq, *wk;
  const int32_t* pos;
  const float* freq;
  int N, Hq, H, rot, tokens;      // H: heads of both; tokens of a workgroup
  float eps, inv_H;
};

// Sum over the LPR lanes that share a row, in each of them.
template <int LPR>
__device__ __forceinline__ float row_sum(float x) {
  x += dpp_f32<DPP_XOR1>(x);
  x += dpp_f32<DPP_XOR2>(x);
  if constexpr (LPR >= 8) x += dpp_f32<DPP_ROW_HALF_MIRROR>(x);
  if constexpr (LPR >= 16) x += dpp_f32<DPP_ROW_MIRROR>(x);
  return x;
}

template <int DT>
__device__ __forceinline__ void unpack(const uint4& v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = to_f32<DT>((uint16_t)w[i]);
    x[2 * i + 1] = to_f32<DT>((uint16_t)(w[i] >> 16));
  }
}

template <int DT>
__device__ __forceinline__ uint4 pack(const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = (uint32_t)from_f32<DT>(x[2 * i]) | (uint32_t)from_f32<DT>(x[2 * i + 1]) << 16;
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <int DT, int D, bool PAIRS>
__global__ __launch_bounds__(NT_R) void k_norm_rope(RopeArgs a) {
  constexpr int LPR = D / 16, RPP = NT_R / LPR;     // lanes of a row, rows of a pass
  __shared__ __align__(16) float turn[2 * MAX_TURNS];      // cos, sin by (token, frequency)
  const int tid = threadIdx.x, lane = tid % LPR;
  const int t0 = blockIdx.x * a.tokens, nt = min(a.tokens, a.N - t0), half = a.rot / 2;
  const bool turned = lane * 16 < a.rot;
  // first elements of the lane's two vectors
  const int e0 = turned && !PAIRS ? lane * 8 : lane * 16, e1 = turned && !PAIRS ? half + lane * 8 : lane * 16 + 8;

  const int rows = nt * a.H;
  uint4 v0, v1;
  int tok = 0, h = 0;
  auto load = [&](int r) {
    tok = (int)(((float)r + 0.5f) * a.inv_H);      // r < 2^20: exact
    h = r - tok * a.H;
    const char* p = h < a.Hq ? a.q + (int64_t)(t0 + tok) * a.q_node + h * a.q_head
                             : a.k + (int64_t)(t0 + tok) * a.k_node + (h - a.Hq) * a.k_head;
    v0 = *(const uint4*)(p + e0 * 2);
    v1 = *(const uint4*)(p + e1 * 2);
  };
  int r = tid / LPR;
  if (r < rows) load(r);

  // the angle in turns: two products and a constant, each rounded to 53 bits, so off
  // by at most 3 2^-53 of itself.  That is below fp32's own rounding of the fraction
  // that is left, 2^-26, for angles of up to 2^25 turns, and 2^-23 turns at the
  // farthest positions
  for (int i = tid; i < nt * half; i += NT_R) {
    const int t = i / half, j = i - t * half;
    const double turns = (double)a.pos[t0 + t] * (double)a.freq[j] * 0.15915494309189533577;
    const float f = (float)(turns - rint(turns));
    float s, c;
    sincospif(2.0f * f, &s, &c);
    turn[i] = c;
    turn[MAX_TURNS + i] = s;
  }
  __syncthreads();

  while (r < rows) {
    float x[8], y[8];
    unpack<DT>(v0, x);
    unpack<DT>(v1, y);
    const int tk = tok, hd = h;
    const bool query = hd < a.Hq;
    if (r + RPP < rows) load(r + RPP);
    const char* w = query ? a.wq : a.wk;
    if (w) {
      float ss = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], fmaf(y[i], y[i], ss));
      const float inv = 1.0f / sqrtf(row_sum<LPR>(ss) * (1.0f / D) + a.eps);
      float wx[8], wy[8];
      unpack<DT>(*(const uint4*)(w + e0 * 2), wx);
      unpack<DT>(*(const uint4*)(w + e1 * 2), wy);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] *= inv * wx[i], y[i] *= inv * wy[i];
    }
    if (turned) {
      const float* c = turn + tk * half + lane * 8;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float cs = c[i], sn = c[MAX_TURNS + i];
        float& p = PAIRS ? (i < 4 ? x[2 * i] : y[2 * i - 8]) : x[i];
        float& q = PAIRS ? (i < 4 ? x[2 * i + 1] : y[2 * i - 7]) : y[i];
        const float u = p, v = q;
        p = u * cs - v * sn;
        q = v * cs + u * sn;
      }
    }
    char* o = query ? a.qo + (int64_t)(t0 + tk) * a.qo_node + hd * a.qo_head
                    : a.ko + (int64_t)(t0 + tk) * a.ko_node + (hd - a.Hq) * a.ko_head;
    *(uint4*)(o + e0 * 2) = pack<DT>(x);
    *(uint4*)(o + e1 * 2) = pack<DT>(y);
    r += RPP;
  }
}

// Strides of an output of N nodes and H heads whose rows share no memory: the
// nodes' rows within a node's, or the other way round.
bool apart(int64_t node, int64_t head, int N, int H, int D) {
  if (N > 1 && H > 1)
    return (head >= D && node >= head * (H - 1) + D) || (node >= D && head >= node * (N - 1) + D);
  return (N == 1 || node >= D) && (H == 1 || head >= D);
}

int check(const sd_qk_norm_rope_args_t* p) {
  if (!p || p->N < 1 || p->H_q < 1 || p->H_k < 0 || p->D < 1 || !p->positions || !p->inv_freq) return SD_EINVAL;
  if (p->dtype != SD_BF16 && p->dtype != SD_F16) return SD_EINVAL;
  if (!rows_ok(p->q, p->q_node, p->q_head) || !rows_ok(p->q_out, p->q_out_node, p->q_out_head)) return SD_EINVAL;
  if (p->H_k && (!rows_ok(p->k, p->k_node, p->k_head) || !rows_ok(p->k_out, p->k_out_node, p->k_out_head)))
    return SD_EINVAL;
  if ((p->q_weight && !aligned16(p->q_weight)) || (p->k_weight && !aligned16(p->k_weight))) return SD_EINVAL;
  if (!(p->eps >= 0.0f) || !isfinite(p->eps) || p->rot < 16 || p->rot % 16 || p->rot > p->D) return SD_EINVAL;
  if (p->D != 64 && p->D != 128 && p->D != 256) return SD_EUNSUPPORTED;
  if ((int64_t)p->H_q + p->H_k > 65535) return SD_EUNSUPPORTED;
  if (!apart(p->q_out_node, p->q_out_head, p->N, p->H_q, p->D)) return SD_EINVAL;
  if (p->H_k && !apart(p->k_out_node, p->k_out_head, p->N, p->H_k, p->D)) return SD_EINVAL;
  // in place only where each row is its own result
  if (p->q_out == p->q && (p->q_out_node != p->q_node || p->q_out_head != p->q_head)) return SD_EINVAL;
  if (p->H_k) {
    if (p->k_out == p->k && (p->k_out_node != p->k_node || p->k_out_head != p->k_head)) return SD_EINVAL;
    if (p->q_out == p->k || p->k_out == p->q || p->q_out == p->k_out) return SD_EINVAL;
  }
  for (const void* o : {p->q_out, p->H_k ? p->k_out : nullptr})
    if (o && (o == p->q_weight || o == p->k_weight || o == p->positions || o == p->inv_freq)) return SD_EINVAL;
  return SD_OK;
}

template <int DT, int D>
void launch(const RopeArgs& a, bool pairs, hipStream_t st) {
  const dim3 grid((unsigned)((a.N + a.tokens - 1) / a.tokens));
  if (pairs) hipLaunchKernelGGL((k_norm_rope<DT, D, true>), grid, dim3(NT_R), 0, st, a);
  else hipLaunchKernelGGL((k_norm_rope<DT, D, false>), grid, dim3(NT_R), 0, st, a);
}

}  // namespace

extern "C" int sd_qk_norm_rope(const sd_qk_norm_rope_args_t* p, void* stream) {
  const int rc = check(p);
  if (rc) return rc;
  RopeArgs a;
  a.q = static_cast<const char*>(p->q), a.k = static_cast<const char*>(p->k);
  a.qo = static_cast<char*>(p->q_out), a.ko = static_cast<char*>(p->k_out);
  a.q_node = p->q_node * 2, a.q_head = p->q_head * 2, a.k_node = p->k_node * 2, a.k_head = p->k_head * 2;
  a.qo_node = p->q_out_node * 2, a.qo_head = p->q_out_head * 2;
  a.ko_node = p->k_out_node * 2, a.ko_head = p->k_out_head * 2;
  a.wq = static_cast<const char*>(p->q_weight), a.wk = static_cast<const char*>(p->k_weight);
  a.pos = p->positions, a.freq = p->inv_freq;
  a.N = p->N, a.Hq = p->H_q, a.H = p->H_q + p->H_k, a.rot = p->rot;
  a.eps = p->eps, a.inv_H = 1.0f / (float)a.H;
  // tokens of a workgroup: as many as give every lane a row, and no more turns
  // than the table holds
  const int rpp = NT_R / (p->D / 16);
  a.tokens = std::max(1, std::min(rpp / a.H, MAX_TURNS / (a.rot / 2)));
  // a grid dimension holds less than 2^32 threads
  if (p->N / a.tokens >= (1 << 24) - 1) return SD_EUNSUPPORTED;
  hipStream_t st = static_cast<hipStream_t>(stream);
  const bool bf = p->dtype == SD_BF16, pairs = p->interleaved != 0;
  if (p->D == 64) bf ? launch<SD_BF16, 64>(a, pairs, st) : launch<SD_F16, 64>(a, pairs, st);
  else if (p->D == 128) bf ? launch<SD_BF16, 128>(a, pairs, st) : launch<SD_F16, 128>(a, pairs, st);
  else bf ? launch<SD_BF16, 256>(a, pairs, st) : launch<SD_F16, 256>(a, pairs, st);
  return hipGetLastError() == hipSuccess ? SD_OK : SD_EHIP;
}
