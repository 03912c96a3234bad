// Attention of a drafted tree over a paged cache held in 8 bits on gfx950.
//
// Row (node i, query head g) of a request: s_j = scale q . k_j over the visible
// slots of the cache and the nodes that i sees, o = softmax(s) . v with a running
// maximum and sum.  A slot's key is ks * code, its value vs * code, with the scales
// of its block.
//
// The rows that share a KV head (nodes x heads of its group) are packed into one
// matrix.  A workgroup is four waves over the same 16 MT rows, each with keys of its
// own, 32 slots at a time straight from the cache into registers: nothing is staged,
// so the waves meet only at the end of a run.  Blocks and pages hold whole multiples
// of 16 slots, so what addresses 16 of them is in scalar registers.
//
//   S^T = K . Q^T   a lane loads 16 bytes of a key and makes two operands of them;
//                   the queries' columns are in the same order.
//   weights         with M the running maximum of x = s + log2(vs) (base 2),
//                   w = 2^(x - M) is the weight times vs: it meets the codes, and
//                   w / vs sums up the softmax.  So each scale costs an operand of
//                   an instruction that is there anyway, and w lies below 1 however
//                   far the scales lie apart.
//   O^T = V^T . W^T a lane loads D / 16 columns of each of its 8 keys and transposes
//                   bytes within its own registers; operand d holds columns
//                   d, D / 16 + d, ...
//
// Codes are exact in 16 bits.  The weights of cached tokens enter the product in
// fp16, whatever the queries' type: 11 bits, held at 2^7 of the running maximum, so
// that a long tail beside one dominating key keeps its precision down to 2^-21 of
// it.  Those of the nodes, whose values may pass fp16's range, are of the queries'
// type.  They are divided by their fp32 sum: the rounded ones' would miss tokens whose
// weight is large but whose w is not, beside values of a far larger scale.
//
// The (request, KV head, row tile, key tile) units form one list that is cut into
// equal runs, one per workgroup; parts are joined in a fixed order.  Through a
// window only the key tiles that it (or the sinks) touches are units.
#include <algorithm>
#include <type_traits>

#include "sdq_device.h"

using namespace sdv;
using namespace sdt;
using sdq::QuantCache;

namespace {

constexpr int WAVES = 4, KEYS = 32, KT = WAVES * KEYS;      // keys of a wave's step, of a unit
constexpr int NT_Q = WAVES * WAVE;
constexpr float LIFT = 7.0f;

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

struct QAttnArgs {
  QuantCache c;
  const char *q, *kn, *vn;
  int64_t q_node, q_head, k_node, k_head, v_node, v_head;   // bytes
  const int32_t* off;
  const int32_t* parents;
  int N, max_nodes, Hq, G, mts_max, window, sinks;
  bool whole;       // no row tile's keys are split
  float scale, inv_G;
  float* part;      // partial results, two slots a run
  char* out;
  float* lse;
  uint32_t* status;
};

// ---- the unit list ----

// What the lanes of a wave hold of up to 64 requests, one each: slots in use,
// nodes, row tiles, key tiles (the tree's is the last) and units, for all KV
// heads, up to and including the lane's own.  Key tile t is the cache's tile t
// below `head`, t + skip from there on.
struct Requests {
  int ctx, first, T, mts, nt, head, skip, incl;
  uint32_t st;
};

__device__ __forceinline__ int first_seen(int position, int window) { return window > position ? 0 : position - window + 1; }

template <int RT>
__device__ __forceinline__ Requests requests(const QAttnArgs& a, int b) {
  Requests r{0, 0, 0, 0, 0, 0, 0, 0, 0};
  if (b < a.c.B) {
    const Nodes nd = request_nodes(a.off, b, a.N, a.max_nodes);
    r.ctx = sdq::request_ctx(a.c, b, r.st);
    r.first = nd.first, r.T = nd.T;
    r.mts = (nd.T * a.G + RT - 1) / RT;
    const int tiles = (r.ctx + KT - 1) / KT;
    if (a.window) {
      // the root sees the earliest slot of all
      const int from = first_seen(r.ctx, a.window) / KT;
      r.head = min((min(a.sinks, r.ctx) + KT - 1) / KT, tiles);
      r.skip = max(0, min(from, tiles) - r.head);
    }
    r.nt = tiles - r.skip + 1;
  }
  r.incl = wave_incl_scan_int(r.mts * r.nt * a.c.H);
  return r;
}

__device__ __forceinline__ int lane_units(const Requests& r) { return lane_read(r.incl, WAVE - 1); }

__device__ __forceinline__ int wave_max_int(int x) {
  x = max(x, dpp_i32<DPP_XOR1>(x));
  x = max(x, dpp_i32<DPP_XOR2>(x));
  x = max(x, dpp_i32<DPP_ROW_HALF_MIRROR>(x));
  x = max(x, dpp_i32<DPP_ROW_MIRROR>(x));
  return max(max(lane_read(x, 0), lane_read(x, 16)), max(lane_read(x, 32), lane_read(x, 48)));
}

// All units, and the units of a run: equal shares, but no row tile in more than
// about 32 parts, which the join would take longer to add up than their runs
// save.  r: the first 64 requests.
struct Cut {
  int total, per;
};

template <int RT>
__device__ __forceinline__ Cut cut_units(const QAttnArgs& a, const Requests& r, int runs) {
  int total = lane_units(r), nt = r.nt;
  for (int b0 = WAVE; b0 < a.c.B; b0 += WAVE) {
    const Requests q = requests<RT>(a, b0 + (int)threadIdx.x % WAVE);
    total += lane_units(q);
    nt = max(nt, q.nt);
  }
  return Cut{total, max((int)(((unsigned)total + runs - 1) / (unsigned)runs), (wave_max_int(nt) + 31) / 32)};
}

// r / G for a packed row (exact: r < 2^11, G <= 32).
__device__ __forceinline__ int row_node(const QAttnArgs& a, int r) { return (int)(((float)r + 0.5f) * a.inv_G); }

// Lane j: itself and the ancestors of node j of the request, as bits, by pointer
// doubling (six steps reach the root of any tree of 64 nodes); its depth.
struct Seen {
  uint64_t nodes;
  int depth;
};

__device__ __forceinline__ Seen seen_by_lane(const QAttnArgs& a, int first, int T, int ctx) {
  const int j = threadIdx.x % WAVE;
  Seen s;
  if (!a.parents) {
    s.nodes = (2ull << j) - 1;
  } else {
    int up = j < T ? a.parents[first + j] : -1;
    if (up < -1 || up >= j) up = -1;
    s.nodes = 1ull << j;
#pragma unroll
    for (int i = 0; i < 6; ++i) {
      const int from = max(up, 0);
      const uint64_t mu = __shfl(s.nodes, from);
      const int uu = __shfl(up, from);
      if (up >= 0) s.nodes |= mu, up = uu;
    }
  }
  s.depth = __popcll(s.nodes) - 1;
  if (a.window && a.window < T) {
    const uint64_t all = s.nodes;
    for (int i = 0; i < T; ++i) {
      const int d = lane_read(s.depth, i);
      if (s.depth - d >= a.window && ctx + d >= a.sinks) s.nodes &= ~(1ull << i);
    }
    s.nodes &= all;
  }
  return s;
}

// ---- codes as operands ----

// 4 codes, as two pairs of 16-bit elements of type DT, without their scale.
template <int DT, int CODE>
__device__ __forceinline__ u32x2 widen(uint32_t u) {
  u32x2 r;
  if constexpr (CODE == SD_E4M3) {
    if constexpr (DT == SD_BF16) {
      r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(u, 1.0f, false));
      r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(u, 1.0f, true));
    } else {
      r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(u, 1.0f, false));
      r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(u, 1.0f, true));
    }
  } else if constexpr (DT == SD_BF16) {
    // whole numbers of 8 bits are exact in the upper half of an fp32
    float f[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = (float)(int8_t)(u >> (8 * i));
    r[0] = __builtin_amdgcn_perm(__float_as_uint(f[1]), __float_as_uint(f[0]), 0x07060302u);
    r[1] = __builtin_amdgcn_perm(__float_as_uint(f[3]), __float_as_uint(f[2]), 0x07060302u);
  } else {
    // 0x6480 ^ code is the fp16 number 1152 + code
    const f16x2 bias = {(_Float16)1152.0f, (_Float16)1152.0f};
    r[0] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(0u, u, 0x0C010C00u) ^ 0x64806480u) - bias);
    r[1] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(0u, u, 0x0C030C02u) ^ 0x64806480u) - bias);
  }
  return r;
}

// e4m3 codes that are not numbers as 0.
__device__ __forceinline__ uint32_t numbers(uint32_t u) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if ((u >> (8 * i) & 0x7Fu) == 0x7Fu) u &= ~(0xFFu << (8 * i));
  return u;
}

// Column `byte` of 8 keys as fp16 operand elements; w[s][r]: 4 columns of key
// 16 s + 4 g4 + r.
template <int CODE>
struct Columns {

  s16x8 col[4];
  __device__ Columns(const uint32_t (&w)[2][4]) {
    u32x4 c[4];
    if constexpr (CODE == SD_I8) {
      const f16x2 bias = {(_Float16)1152.0f, (_Float16)1152.0f};
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t x = __builtin_amdgcn_perm(w[s][2 * p + 1], w[s][2 * p], 0x0C040C00u + 0x00010001u * i);
            c[i][2 * s + p] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, x ^ 0x64806480u) - bias);
          }
    } else {
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          const u32x2 a = widen<SD_F16, CODE>(w[s][2 * p]), b = widen<SD_F16, CODE>(w[s][2 * p + 1]);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            c[2 * i][2 * s + p] = __builtin_amdgcn_perm(b[i], a[i], 0x05040100u);
            c[2 * i + 1][2 * s + p] = __builtin_amdgcn_perm(b[i], a[i], 0x07060302u);
          }
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) col[i] = __builtin_bit_cast(s16x8, c[i]);
  }
};

// Any of the 8 elements infinite or not a number, and the others.
template <int DT>
__device__ __forceinline__ uint32_t finite_or_zero(uint32_t u, bool& odd) {
  constexpr uint32_t E = DT == SD_BF16 ? 0x7F80u : 0x7C00u;
  if ((u & E) == E) u &= 0xFFFF0000u, odd = true;
  if (((u >> 16) & E) == E) u &= 0x0000FFFFu, odd = true;
  return u;
}

// A pointer whose loads go through the scalar cache (uniform addresses only, of
// memory that the kernel does not write).
template <typename T>
__device__ __forceinline__ T scalar_load(const T* p) {
  return *(const __attribute__((address_space(4))) T*)(uint64_t)p;
}

// 32 slots of one KV head as loaded, and what is uniform about each 16 of them.
template <int D>
struct Raw {
  static constexpr int KW = D / 64, VW = D / 64;      // 16-byte loads of a key; words of a key's columns
  u32x4 k[2][KW];
  uint32_t v[2][4][VW];
  float kscale[2], vscale[2];
  int n[2];      // slots that are there, if their scales are sound
};

template <int DT, int CODE, int D, int MT>
__global__ __launch_bounds__(NT_Q, MT == 4 ? 1 : 2) void k_quant_tiles(QAttnArgs a) {
  constexpr int RT = 16 * MT, KS = D / 32, CB = D / 16, KW = D / 64, VW = D / 64, JR = D + 4;
  constexpr int SLOT = RT * (D + 2);
  __shared__ __align__(16) float join[(WAVES - 1) * RT * JR];
  __shared__ int odd_value;      // a node's value is infinite or not a number
  const int tid = threadIdx.x, l = tid % WAVE, n = l & 15, g4 = l >> 4;
  const int w = __builtin_amdgcn_readfirstlane(tid / WAVE);
  const float c = a.scale * 1.4426950408889634f;      // scores in base 2

  Requests rq = requests<RT>(a, l);
  int run, u0, u1;
  if (a.whole) {
    run = 0, u0 = 0, u1 = 0;
  } else {
    // Workgroups of one XCD take neighbouring runs: row tiles of one KV head
    // find each other's keys in its L2.
    const int runs = gridDim.x;
    const auto [total, per] = cut_units<RT>(a, rq, runs);
    run = (int)(blockIdx.x % 8) * (runs / 8) + (int)(blockIdx.x / 8);      // runs is a multiple of 8
    if ((int64_t)run * per >= total) return;
    u0 = run * per, u1 = u0 + min(per, total - u0);
  }

  // the request (lane f of this 64) that holds unit u0, and its units before
  int b0 = 0, f, in;
  if (a.whole) {
    const int b = blockIdx.x / (a.c.H * a.mts_max), seg = blockIdx.x % (a.c.H * a.mts_max);
    b0 = b & ~(WAVE - 1), f = b & (WAVE - 1);
    if (b0) rq = requests<RT>(a, b0 + l);
    const int mts = lane_read(rq.mts, f), nt = lane_read(rq.nt, f);
    if (seg % a.mts_max >= mts) return;
    in = (seg / a.mts_max * mts + seg % a.mts_max) * nt;
    u1 = nt;
  } else {
    int left = u0;
    while (left >= lane_units(rq)) {
      left -= lane_units(rq);
      b0 += WAVE;
      rq = requests<RT>(a, b0 + l);
    }
    f = __builtin_ctzll(__ballot(left < rq.incl));
    in = left - (f ? lane_read(rq.incl, f - 1) : 0);
  }

  // offsets of a lane within 16 slots
  const uint32_t kat = (uint32_t)(n * (int)a.c.slot_stride + g4 * 16);
  const uint32_t vat = (uint32_t)(g4 * 4 * (int)a.c.slot_stride + n * CB);

  while (u0 < u1) {
    const int units = lane_read(rq.incl, f) - (f ? lane_read(rq.incl, f - 1) : 0);
    const int ctx = lane_read(rq.ctx, f), first = lane_read(rq.first, f), T = lane_read(rq.T, f);
    const int mts = lane_read(rq.mts, f), nt = lane_read(rq.nt, f);
    const int head = lane_read(rq.head, f), skip = lane_read(rq.skip, f);
    const uint32_t st = (uint32_t)lane_read((int)rq.st, f);
    const int32_t* const tab = a.c.table + (b0 + f) * a.c.ld_table;
    const int rows = T * a.G;
    const int stop = u0 + min(u1 - u0, units - in);
    while (u0 < stop) {
      const int seg = in / nt, t0 = in - seg * nt;
      const int h = seg / mts, mt = seg - h * mts;
      const int t1 = min(nt, t0 + (stop - u0));
      const int row0 = mt * RT;

      // queries as the B operand: lane (n, g4) holds of row n the columns that it
      // loads of a key, 64 (ks / 2) + 16 g4 + 8 (ks % 2) .. + 7
      s16x8 q[MT][KS];
      int node[MT], from[MT];
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const int r = row0 + 16 * m + n;
        const bool on = r < rows;
        node[m] = on ? row_node(a, r) : 0;
        const int hd = h * a.G + (on ? r - node[m] * a.G : 0);
        const char* qp = a.q + (int64_t)(first + node[m]) * a.q_node + hd * a.q_head;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
          q[m][ks] = on ? *(const s16x8*)(qp + (ks / 2 * 64 + g4 * 16 + ks % 2 * 8) * 2) : s16x8{};
      }
      // what the rows see of the tree, and the first slot that their windows show
      uint64_t vis[MT];
      if (t1 == nt || a.window) {
        const Seen seen = seen_by_lane(a, first, T, ctx);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          vis[m] = st ? 0 : __shfl(seen.nodes, node[m]);
          from[m] = a.window ? first_seen(ctx + __shfl(seen.depth, node[m]), a.window) : 0;
        }
      } else {
#pragma unroll
        for (int m = 0; m < MT; ++m) vis[m] = 0, from[m] = 0;
      }
      // slots below this one are past some row's window
      const int all_from = a.window ? first_seen(ctx + T - 1, a.window) : 0;

      if (tid == 0) odd_value = 0;
      __syncthreads();

      f32x4 o[MT][CB];
      float mx[MT], sum[MT];      // sums: of the lane's own keys

      auto page_of = [&](int t, int s) {
        const int slot = (t < head ? t : t + skip) * KT + w * KEYS + s * 16;
        return t < nt - 1 && slot < ctx ? scalar_load(tab + (slot >> a.c.page_shift)) : -1;
      };
      auto load = [&](int t, const int (&page)[2], Raw<D>& x) {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const int slot = (t < head ? t : t + skip) * KT + w * KEYS + s * 16;
          const bool there = (unsigned)page[s] < (unsigned)a.c.num_pages;
          // (what is not there reads the pool's first rows and is masked)
          const int p = there ? page[s] : 0, place = there ? slot & a.c.page_mask : 0;
          const int64_t at = p * a.c.page_stride + h * a.c.head_stride + place * a.c.slot_stride;
          const int64_t sc = p * a.c.scale_page + h * a.c.scale_head + (place >> a.c.block_shift);
          x.kscale[s] = scalar_load(a.c.ks + sc);
          x.vscale[s] = scalar_load(a.c.vs + sc);
          x.n[s] = there ? min(16, ctx - slot) : 0;
          const char* kb = a.c.k + at;
          const char* vb = a.c.v + at;
#pragma unroll
          for (int i = 0; i < KW; ++i) x.k[s][i] = *(const global_u32x4*)((uint64_t)kb + kat + i * 64);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const uint64_t va = (uint64_t)vb + vat + r * (uint32_t)a.c.slot_stride;
            if constexpr (VW == 2) {
              const u32x2 y = *(const __attribute__((address_space(1))) u32x2*)va;
              x.v[s][r][0] = y[0], x.v[s][r][1] = y[1];
            } else {
              x.v[s][r][0] = *(const __attribute__((address_space(1))) uint32_t*)va;
            }
          }
        }
      };

      // Scores to weights: x[s][m] becomes 2^(x ks + lv - M), packed as elements of
      // type PT; bit 16 s + j of on[m]: whether row m sees key j of the 16.
      auto weigh = [&](auto masked, auto type, f32x4 (&x)[2][MT], const float (&ks)[2], const float (&lv)[2],
                       const float (&iv)[2], const uint32_t (&on)[MT], s16x8 (&p)[MT]) {
        constexpr bool MASKED = decltype(masked)::value;
        constexpr int PT = decltype(type)::value;
        bool grown = false;
        float top[MT];
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          top[m] = -INFINITY;
#pragma unroll
          for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              float y = fmaf(x[s][m][r], ks[s], lv[s]);
              if constexpr (MASKED) y = (on[m] >> (g4 * 4) >> (s * 16 + r) & 1) ? y : -INFINITY;
              x[s][m][r] = y;
              top[m] = fmaxf(top[m], y);
            }
          // the sums are rescaled only when a maximum grows by more than 2^8: until
          // then weights up to 2^15 are as exact as those below
          grown |= top[m] - LIFT > mx[m] + 8.0f;
        }
        if (__any(grown)) {
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            const float mn = fmaxf(mx[m], quad_max(top[m]) - LIFT);
            const float fct = mn > -INFINITY ? fast_exp2(mx[m] - mn) : 1.0f;
            mx[m] = mn;
            sum[m] *= fct;
#pragma unroll
            for (int d = 0; d < CB; ++d) o[m][d] *= fct;
          }
        }
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const float ms = mx[m] > -INFINITY ? mx[m] : 0.0f;
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            float y[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              y[r] = fast_exp2(x[s][m][r] - ms);
              p[m][s * 4 + r] = (short)from_f32<PT>(y[r]);
            }
            sum[m] = fmaf((y[0] + y[1]) + (y[2] + y[3]), iv[s], sum[m]);
          }
        }
      };

      // 32 slots against this wave's rows.
      auto cached = [&](int t, Raw<D>& x, bool strict) {
        const int s0 = (t < head ? t : t + skip) * KT + w * KEYS;
        float ks[2], lv[2], iv[2];
        uint32_t valid = 0;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const bool sound = sdq::scale_ok(x.kscale[s]) && sdq::scale_ok(x.vscale[s]);
          const int m = sound ? max(x.n[s], 0) : 0;
          valid |= ((1u << m) - 1) << (16 * s);
          ks[s] = sound ? x.kscale[s] * c : 0.0f;
          const float v = sound && x.vscale[s] > 0.0f ? x.vscale[s] : sdq::MIN_SCALE;
          lv[s] = __log2f(v);
          iv[s] = 1.0f / v;
          if (m < 16 || x.vscale[s] == 0.0f) {
            // a weight of 0 times a code that is not a number would not be 0
#pragma unroll
            for (int r = 0; r < 4; ++r)
              if (g4 * 4 + r >= m || x.vscale[s] == 0.0f)
#pragma unroll
                for (int j = 0; j < VW; ++j) x.v[s][r][j] = 0;
          }
        }
        if (valid == 0) return;
        if (CODE == SD_E4M3 && strict) {
#pragma unroll
          for (int s = 0; s < 2; ++s) {
#pragma unroll
            for (int i = 0; i < KW; ++i)
#pragma unroll
              for (int j = 0; j < 4; ++j) x.k[s][i][j] = numbers(x.k[s][i][j]);
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
              for (int j = 0; j < VW; ++j) x.v[s][r][j] = numbers(x.v[s][r][j]);
          }
        }
        f32x4 y[2][MT];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
#pragma unroll
          for (int m = 0; m < MT; ++m) y[s][m] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int k2 = 0; k2 < KS; ++k2) {
            const u32x2 e = widen<DT, CODE>(x.k[s][k2 / 2][k2 % 2 * 2]), g = widen<DT, CODE>(x.k[s][k2 / 2][k2 % 2 * 2 + 1]);
            const s16x8 kf = __builtin_bit_cast(s16x8, u32x4{e[0], e[1], g[0], g[1]});
#pragma unroll
            for (int m = 0; m < MT; ++m) y[s][m] = mfma<DT>(kf, q[m][k2], y[s][m]);
          }
        }
        s16x8 p[MT];
        using F16 = std::integral_constant<int, SD_F16>;
        const bool edge = a.window && s0 < all_from && s0 + KEYS > a.sinks;
        if (valid == 0xFFFFFFFFu && !edge) {
          uint32_t on[MT] = {};
          weigh(std::false_type{}, F16{}, y, ks, lv, iv, on, p);
        } else {
          uint32_t on[MT];
          const int sn = min(max(a.sinks - s0, 0), 32);
          const uint32_t first_ones = sn >= 32 ? 0xFFFFFFFFu : (1u << sn) - 1;
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            const int skip_keys = min(max(from[m] - s0, 0), 32);
            const uint32_t near = skip_keys >= 32 ? 0u : 0xFFFFFFFFu << skip_keys;
            on[m] = valid & (a.window ? near | first_ones : 0xFFFFFFFFu);
          }
          weigh(std::true_type{}, F16{}, y, ks, lv, iv, on, p);
        }
#pragma unroll
        for (int j = 0; j < VW; ++j) {
          const uint32_t words[2][4] = {{x.v[0][0][j], x.v[0][1][j], x.v[0][2][j], x.v[0][3][j]},
                                        {x.v[1][0][j], x.v[1][1][j], x.v[1][2][j], x.v[1][3][j]}};
          const Columns<CODE> cols(words);
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int m = 0; m < MT; ++m) o[m][4 * j + i] = mfma<SD_F16>(cols.col[i], p[m], o[m][4 * j + i]);
        }
      };

      // Nodes 32 w .. + 31 of the tree, of the queries' type, against this wave's rows.
      auto nodes = [&]() {
        if (w * KEYS >= T) return;
        f32x4 y[2][MT];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const int j = min(w * KEYS + s * 16 + n, T - 1);
          const char* kp = a.kn + (int64_t)(first + j) * a.k_node + h * a.k_head;
#pragma unroll
          for (int m = 0; m < MT; ++m) y[s][m] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int k2 = 0; k2 < KS; ++k2) {
            const s16x8 kf = *(const s16x8*)(kp + (k2 / 2 * 64 + g4 * 16 + k2 % 2 * 8) * 2);
#pragma unroll
            for (int m = 0; m < MT; ++m) y[s][m] = mfma<DT>(kf, q[m][k2], y[s][m]);
          }
        }
        const float ks[2] = {c, c}, lv[2] = {0.0f, 0.0f}, iv[2] = {1.0f, 1.0f};
        uint32_t on[MT];
#pragma unroll
        for (int m = 0; m < MT; ++m) on[m] = (uint32_t)(vis[m] >> (w * KEYS));      // (waves past the tree have returned)
        s16x8 p[MT];
        weigh(std::true_type{}, std::integral_constant<int, DT>{}, y, ks, lv, iv, on, p);
        // columns 8 (or 4) n .. of the lane's 8 nodes
        uint32_t v[2][4][CB / 2];
        bool odd = false;
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int j = w * KEYS + s * 16 + g4 * 4 + r;
            const char* vp = a.vn + (int64_t)(first + min(j, T - 1)) * a.v_node + h * a.v_head + n * CB * 2;
#pragma unroll
            for (int i = 0; i < CB / 2; ++i)
              v[s][r][i] = j < T ? finite_or_zero<DT>(((const uint32_t*)vp)[i], odd) : 0u;
          }
        // 0 x infinity in the product would reach rows that do not see this node:
        // such values are added at the end instead
        if (odd) odd_value = 1;
#pragma unroll
        for (int i = 0; i < CB / 2; ++i) {
          u32x4 e, g;
#pragma unroll
          for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              e[2 * s + r] = __builtin_amdgcn_perm(v[s][2 * r + 1][i], v[s][2 * r][i], 0x05040100u);
              g[2 * s + r] = __builtin_amdgcn_perm(v[s][2 * r + 1][i], v[s][2 * r][i], 0x07060302u);
            }
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            o[m][2 * i] = mfma<DT>(__builtin_bit_cast(s16x8, e), p[m], o[m][2 * i]);
            o[m][2 * i + 1] = mfma<DT>(__builtin_bit_cast(s16x8, g), p[m], o[m][2 * i + 1]);
          }
        }
      };

      // The key tiles of this run.  An e4m3 code that is not a number counts as 0;
      // looking for them costs a tenth, so it is done only where a result came out as
      // none (the second pass).
      const int cached_end = min(t1, nt - 1);
      for (int strict = 0; strict < 2; ++strict) {
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          mx[m] = -INFINITY, sum[m] = 0.0f;
#pragma unroll
          for (int d = 0; d < CB; ++d) o[m][d] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        }
        Raw<D> x[2];
        int page[2] = {page_of(t0, 0), page_of(t0, 1)};
        if (t0 < cached_end) load(t0, page, x[0]);
        page[0] = page_of(t0 + 1, 0), page[1] = page_of(t0 + 1, 1);
        for (int t = t0; t < cached_end; t += 2) {
          if (t + 1 < cached_end) {
            load(t + 1, page, x[1]);
            page[0] = page_of(t + 2, 0), page[1] = page_of(t + 2, 1);
          }
          cached(t, x[0], strict);
          if (t + 1 >= cached_end) break;
          if (t + 2 < cached_end) {
            load(t + 2, page, x[0]);
            page[0] = page_of(t + 3, 0), page[1] = page_of(t + 3, 1);
          }
          cached(t + 1, x[1], strict);
        }
        if constexpr (CODE != SD_E4M3) break;
        bool nan = false;
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          nan |= sum[m] != sum[m];
#pragma unroll
          for (int d = 0; d < CB; ++d)
#pragma unroll
            for (int r = 0; r < 4; ++r) nan |= o[m][d][r] != o[m][d][r];
        }
        if (!__any(nan)) break;
      }
      if (t1 == nt) nodes();
#pragma unroll
      for (int m = 0; m < MT; ++m) sum[m] = quad_sum(sum[m]);

      // the waves' keys: the first one adds the others up
      if (w > 0) {
        float* const z = join + (w - 1) * RT * JR;
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          float* const zr = z + (16 * m + n) * JR;
#pragma unroll
          for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int d = 0; d < CB; d += 4)
              *(f32x4*)(zr + (g4 * 4 + r) * CB + d) = f32x4{o[m][d][r], o[m][d + 1][r], o[m][d + 2][r], o[m][d + 3][r]};
          if (g4 == 0) zr[D] = mx[m], zr[D + 1] = sum[m];
        }
      }
      __syncthreads();
      if (w == 0) {
        for (int k2 = 1; k2 < WAVES; ++k2) {
          const float* const z = join + (k2 - 1) * RT * JR;
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            const float* const zr = z + (16 * m + n) * JR;
            const float m2 = zr[D], mn = fmaxf(mx[m], m2), ms = mn > -INFINITY ? mn : 0.0f;
            const float f1 = fast_exp2(mx[m] - ms), f2 = fast_exp2(m2 - ms);
            mx[m] = mn;
            sum[m] = sum[m] * f1 + zr[D + 1] * f2;
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
              for (int d = 0; d < CB; d += 4) {
                const f32x4 y = *(const f32x4*)(zr + (g4 * 4 + r) * CB + d);
#pragma unroll
                for (int e = 0; e < 4; ++e) o[m][d + e][r] = o[m][d + e][r] * f1 + y[e] * f2;
              }
          }
        }
        if (t1 == nt && odd_value) {
#pragma unroll
          for (int m = 0; m < MT; ++m)
            for (int j = 0; j < T; ++j) {
              const uint16_t* v = (const uint16_t*)(a.vn + (int64_t)(first + j) * a.v_node + h * a.v_head);
#pragma unroll
              for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int d = 0; d < CB; ++d) {
                  const float y = to_f32<DT>(v[(g4 * 4 + r) * CB + d]);
                  if ((vis[m] >> j & 1) && !(fabsf(y) < INFINITY)) o[m][d][r] += y;
                }
            }
        }
        const bool whole = t0 == 0 && t1 == nt;
        float* const part = a.part + (int64_t)(run * 2 + (t0 == 0)) * SLOT;
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const int lr = 16 * m + n, r0 = row0 + lr;
          if (r0 >= rows) continue;
          if (whole) {
            const bool none = sum[m] == 0.0f;
            const float inv = none ? 0.0f : 1.0f / sum[m];
            const int64_t at = (int64_t)(first + node[m]) * a.Hq + h * a.G + (r0 - node[m] * a.G);
            char* const out = a.out + at * (D * 2) + g4 * 4 * CB * 2;
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
              for (int d = 0; d < CB; d += 4) {
                uint32_t u[2];
#pragma unroll
                for (int e = 0; e < 2; ++e)
                  u[e] = (uint32_t)from_f32<DT>(none ? 0.0f : o[m][d + 2 * e][r] * inv) |
                         (uint32_t)from_f32<DT>(none ? 0.0f : o[m][d + 2 * e + 1][r] * inv) << 16;
                *(uint2*)(out + (r * CB + d) * 2) = make_uint2(u[0], u[1]);
              }
            if (a.lse && g4 == 0) a.lse[at] = none ? -INFINITY : (mx[m] + __log2f(sum[m])) * 0.6931471805599453f;
          } else {
            float* const z = part + lr * D + g4 * 4 * CB;
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
              for (int d = 0; d < CB; d += 4)
                *(f32x4*)(z + r * CB + d) = f32x4{o[m][d][r], o[m][d + 1][r], o[m][d + 2][r], o[m][d + 3][r]};
            if (g4 == 0) {
              part[RT * D + lr] = mx[m];
              part[RT * D + RT + lr] = sum[m];
            }
          }
        }
      }
      __syncthreads();      // the join's LDS and odd_value are the next segment's
      u0 += t1 - t0;
      in += t1 - t0;
    }
    in = 0;
    if (++f == WAVE && u0 < u1) {
      f = 0, b0 += WAVE;
      rq = requests<RT>(a, b0 + l);
    }
  }
}

// Rows whose key tiles went to several runs: their parts in the order of the
// runs, JN at a time.  grid (4-column groups of a row tile / 256, H * row
// tiles, B).
template <int DT, int D, int MT>
__global__ __launch_bounds__(256) void k_quant_join(QAttnArgs a, int runs) {
  constexpr int RT = 16 * MT, GPR = D / 4, JN = 8, SLOT = RT * (D + 2);
  const int b = blockIdx.z, h = blockIdx.y / a.mts_max, mt = blockIdx.y % a.mts_max, l = threadIdx.x % WAVE;
  Requests rq = requests<RT>(a, l);
  const int per = cut_units<RT>(a, rq, runs).per;
  int before = 0;
  for (int b0 = 0; b0 + WAVE <= b; b0 += WAVE) {
    before += lane_units(rq);
    rq = requests<RT>(a, b0 + WAVE + l);
  }
  const int f = b % WAVE, nt = lane_read(rq.nt, f), mts = lane_read(rq.mts, f);
  if (mt >= mts) return;
  if (f) before += lane_read(rq.incl, f - 1);
  const int s = before + (h * mts + mt) * nt;
  const int w0 = (int)((unsigned)s / (unsigned)per), w1 = (int)((unsigned)(s + nt - 1) / (unsigned)per);
  const int lin = blockIdx.x * 256 + threadIdx.x, lr = lin / GPR, col = lin % GPR, r = mt * RT + lr;
  if (w0 == w1 || lr >= RT || r >= lane_read(rq.T, f) * a.G) return;
  float m = -INFINITY, sum = 0.0f;
  f32x4 o = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int w = w0; w <= w1; w += JN) {
    float pm[JN], ps[JN];
    f32x4 po[JN];
#pragma unroll
    for (int i = 0; i < JN; ++i) {
      const int wi = min(w + i, w1);
      const float* z = a.part + (int64_t)(wi * 2 + (wi == w0)) * SLOT;
      pm[i] = z[RT * D + lr];
      ps[i] = z[RT * D + RT + lr];
      po[i] = *(const f32x4*)(z + lr * D + col * 4);
    }
#pragma unroll
    for (int i = 0; i < JN; ++i) {
      if (w + i > w1) break;
      const float mn = fmaxf(m, pm[i]), ms = mn > -INFINITY ? mn : 0.0f;
      const float f1 = fast_exp2(m - ms), f2 = fast_exp2(pm[i] - ms);
      m = mn;
      sum = sum * f1 + ps[i] * f2;
      o = o * f1 + po[i] * f2;
    }
  }
  const bool none = sum == 0.0f;
  const float inv = none ? 0.0f : 1.0f / sum;
  const int node = row_node(a, r);
  const int64_t at = (int64_t)(lane_read(rq.first, f) + node) * a.Hq + h * a.G + (r - node * a.G);
  uint32_t u[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    u[i] = (uint32_t)from_f32<DT>(none ? 0.0f : o[2 * i] * inv) |
           (uint32_t)from_f32<DT>(none ? 0.0f : o[2 * i + 1] * inv) << 16;
  *(uint2*)(a.out + at * (D * 2) + col * 8) = make_uint2(u[0], u[1]);
  if (a.lse && col == 0) a.lse[at] = none ? -INFINITY : (m + __log2f(sum)) * 0.6931471805599453f;
}

// Status bits of one request per workgroup.
__global__ __launch_bounds__(WAVE) void k_quant_status(QAttnArgs a) {
  const int b = blockIdx.x, l = threadIdx.x;
  const Nodes nd = request_nodes(a.off, b, a.N, a.max_nodes);
  uint32_t st = nd.st;
  const int ctx = sdq::request_ctx(a.c, b, st);
  const int32_t* tab = a.c.table + b * a.c.ld_table;
  bool bad_page = false, bad_scale = false, bad_tree = false;
  const int last = first_seen(ctx, a.window ? a.window : INT_MAX);
  for (int p = l; p < (ctx + a.c.page_mask) >> a.c.page_shift; p += WAVE) {
    // pages that no row sees are not looked at
    if (a.window && (p << a.c.page_shift) >= a.sinks && ((p + 1) << a.c.page_shift) <= last) continue;
    const int page = tab[p];
    if ((unsigned)page >= (unsigned)a.c.num_pages) {
      bad_page = true;
      continue;
    }
    const int used = min(ctx - (p << a.c.page_shift), a.c.page_mask + 1);
    for (int h = 0; h < a.c.H; ++h)
      for (int k = 0; k << a.c.block_shift < used; ++k) {
        const int64_t at = page * a.c.scale_page + h * a.c.scale_head + k;
        bad_scale |= !sdq::scale_ok(a.c.ks[at]) || !sdq::scale_ok(a.c.vs[at]);
      }
  }
  if (a.parents && l < nd.T) {
    const int p = a.parents[nd.first + l];
    bad_tree = p < -1 || p >= l;
  }
  if (__any(bad_page)) st |= SD_ST_BAD_PAGE;
  if (__any(bad_scale)) st |= SD_ST_BAD_SCALE;
  if (__any(bad_tree)) st |= SD_ST_BAD_TREE;
  if (l == 0) a.status[b] = st;
}

int check(const sd_quant_attention_args_t* p) {
  if (!p) return SD_EINVAL;
  const int rc = sdq::check_cache(p->cache);
  if (rc) return rc;
  if (p->dtype != SD_BF16 && p->dtype != SD_F16) return SD_EINVAL;
  if (!rows_ok(p->q, p->q_node, p->q_head) || !rows_ok(p->k_new, p->k_node, p->k_head) ||
      !rows_ok(p->v_new, p->v_node, p->v_head) || !p->node_offsets || p->N < 1 ||
      p->max_nodes < 1 || p->H_q < 1 || p->H_q % p->cache.H_kv || !isfinite(p->scale))
    return SD_EINVAL;
  if (p->window < 0 || p->sinks < 0 || (p->sinks && !p->window)) return SD_EINVAL;
  if (p->max_nodes > SD_MAX_NODES || p->H_q / p->cache.H_kv > SD_MAX_GROUP || p->H_q > 65535)
    return SD_EUNSUPPORTED;
  return SD_OK;
}

QAttnArgs device_args(const sd_quant_attention_args_t* p) {
  QAttnArgs a;
  a.c = sdq::device_cache(p->cache);
  a.q = static_cast<const char*>(p->q);
  a.kn = static_cast<const char*>(p->k_new);
  a.vn = static_cast<const char*>(p->v_new);
  a.q_node = p->q_node * 2, a.q_head = p->q_head * 2;
  a.k_node = p->k_node * 2, a.k_head = p->k_head * 2;
  a.v_node = p->v_node * 2, a.v_head = p->v_head * 2;
  a.off = p->node_offsets;
  a.parents = p->parents;
  a.N = p->N;
  a.max_nodes = p->max_nodes;
  a.Hq = p->H_q;
  a.G = p->H_q / p->cache.H_kv;
  a.inv_G = 1.0f / (float)a.G;
  a.window = p->window, a.sinks = p->sinks;
  a.scale = p->scale;
  return a;
}

// Row tiles of 16 a wave for `rows` packed rows a KV head.
template <typename F>
auto with_rows(int rows, F&& f) {
  if (rows <= 16) return f(std::integral_constant<int, 1>{});
  if (rows <= 32) return f(std::integral_constant<int, 2>{});
  return f(std::integral_constant<int, 4>{});
}

// Workgroups that share the unit list: one a CU of those with 4 row tiles, else
// two.
constexpr int run_count(int mt) { return mt == 4 ? 256 : 512; }

// Where there are no more key tiles than this, splitting them and joining the
// parts in a second launch costs more than it saves.
constexpr int WHOLE_TILES = 8;

// How a call is cut up.
struct Plan {
  int mts_max;                // row tiles of a KV head
  int64_t segments, tiles;    // (request, KV head, row tile)s, and key tiles of one
  bool fits, whole;
};

Plan plan(const sd_quant_attention_args_t* p, int mt) {
  const sd_quant_cache_t& c = p->cache;
  const int rt = 16 * mt, rows = p->max_nodes * (p->H_q / c.H_kv);
  Plan r;
  r.mts_max = (rows + rt - 1) / rt;
  r.segments = (int64_t)c.B * c.H_kv * r.mts_max;
  r.tiles = ((int64_t)c.max_pages * c.page_size + KT - 1) / KT + 1;
  if (p->window) r.tiles = std::min(r.tiles, ((int64_t)p->sinks + KT - 1) / KT + ((int64_t)p->window + KT - 1) / KT + 2);
  r.fits = r.segments <= 0x7FFFFFFF / r.tiles;      // units are counted in 32 bits
  // (and a grid dimension holds less than 2^32 threads)
  r.whole = r.tiles <= WHOLE_TILES && r.segments * NT_Q <= UINT32_MAX;
  return r;
}

template <int DT, int CODE, int D>
int launch(QAttnArgs a, const sd_quant_attention_args_t* p, hipStream_t st) {
  return with_rows(a.max_nodes * a.G, [&](auto mt) {
    constexpr int MT = decltype(mt)::value, runs = run_count(MT);
    const Plan r = plan(p, MT);
    a.mts_max = r.mts_max;
    a.whole = r.whole;
    hipLaunchKernelGGL((k_quant_tiles<DT, CODE, D, MT>), dim3(a.whole ? (unsigned)r.segments : (unsigned)runs),
                       dim3(NT_Q), 0, st, a);
    if (hipGetLastError() != hipSuccess) return SD_EHIP;
    if (a.whole) return SD_OK;
    const dim3 grid((16 * MT * (D / 4) + 255) / 256, a.c.H * a.mts_max, a.c.B);
    hipLaunchKernelGGL((k_quant_join<DT, D, MT>), grid, dim3(256), 0, st, a, runs);
    return hipGetLastError() == hipSuccess ? SD_OK : SD_EHIP;
  });
}

}  // namespace

extern "C" int sd_quant_attention_workspace_bytes(const sd_quant_attention_args_t* args, size_t* bytes) {
  if (!bytes) return SD_EINVAL;
  const int rc = check(args);
  if (rc) return rc;
  return with_rows(args->max_nodes * (args->H_q / args->cache.H_kv), [&](auto mt) {
    constexpr int MT = decltype(mt)::value;
    const Plan p = plan(args, MT);
    *bytes = p.whole ? 0 : (size_t)run_count(MT) * 2 * (16 * MT) * (args->cache.D + 2) * sizeof(float);
    return p.fits ? SD_OK : SD_EUNSUPPORTED;
  });
}

extern "C" int sd_quant_attention(const sd_quant_attention_args_t* args, void* workspace,
                                  size_t workspace_bytes, void* out, float* out_lse,
                                  uint32_t* out_status, void* stream) {
  size_t need = 0;
  int rc = sd_quant_attention_workspace_bytes(args, &need);
  if (rc) return rc;
  if (!out || !aligned16(out)) return SD_EINVAL;
  if (out == args->k_new || out == args->v_new || out == args->cache.k || out == args->cache.v) return SD_EINVAL;
  // a query row is read by the workgroups of its own result alone, before they
  // write it or before the join does
  if (out == args->q && (args->q_head != args->cache.D || args->q_node != (int64_t)args->H_q * args->cache.D))
    return SD_EINVAL;
  if (need && (!workspace || workspace_bytes < need || !aligned16(workspace))) return SD_EWORKSPACE;
  QAttnArgs a = device_args(args);
  a.out = static_cast<char*>(out);
  a.lse = out_lse;
  a.status = out_status;
  a.part = static_cast<float*>(workspace);
  hipStream_t st = static_cast<hipStream_t>(stream);
  auto go = [&](auto dt, auto code) {
    constexpr int DT = decltype(dt)::value, CODE = decltype(code)::value;
    return args->cache.D == 64 ? launch<DT, CODE, 64>(a, args, st) : launch<DT, CODE, 128>(a, args, st);
  };
  using BF = std::integral_constant<int, SD_BF16>;
  using HF = std::integral_constant<int, SD_F16>;
  using I8 = std::integral_constant<int, SD_I8>;
  using E4 = std::integral_constant<int, SD_E4M3>;
  if (args->cache.code == SD_I8) rc = args->dtype == SD_BF16 ? go(BF{}, I8{}) : go(HF{}, I8{});
  else rc = args->dtype == SD_BF16 ? go(BF{}, E4{}) : go(HF{}, E4{});
  if (rc) return rc;
  if (out_status) {
    hipLaunchKernelGGL(k_quant_status, dim3(a.c.B), dim3(WAVE), 0, st, a);
    if (hipGetLastError() != hipSuccess) return SD_EHIP;
  }
  return SD_OK;
}
