// Attention of a drafted tree over a paged cache on gfx950.
//
// Row (node i, query head g) of a request: s_j = scale q . k_j over the
// request's cache slots and the nodes that i sees, o = softmax(s) . v with a
// running maximum and sum, so the scores never leave the chip.
//
// The rows that share a KV head (nodes x heads of its group) are packed into
// one matrix, so a key or value is read once for all of them.  Keys come in
// tiles of KT; the tree's own nodes are one more tile behind the cache's.  All
// (request, KV head, row tile, key tile) units form one list that is cut into
// equal runs, one per workgroup: ragged batches and single long contexts
// spread over the chip alike.  A workgroup that holds all key tiles of its
// rows writes them out; the others leave (maximum, sum, product) in the
// workspace and k_attn_join adds them up in a fixed order.
//
// k_attn_tiles   the wave's scores are S^T = K . Q^T on MFMA 16x16x32, so a
//                lane holds 8 keys of one row per step of 32 keys: the
//                running maximum takes two lane swaps, the weights P^T are
//                already in the layout that O^T = V^T . P^T wants, and V comes
//                out of LDS transposed (ds_read_b64_tr_b16).  Keys are staged
//                through registers into swizzled LDS rows, the next tile's
//                loads in flight behind the products.
//                Up to about 130 rows a KV head it is bound by the latencies of
//                a run's start and end, as long as 3 of its tiles: 3.2 TB/s over
//                32 chains of 9 nodes, 3.8 TB/s over longer contexts, where a
//                copy reaches 4.85.  Past that it is bound by the issue of
//                softmax and products, which overlap little: 16 trees of 64 nodes
//                over 16k to 32k slots take 476 us, 640 TFLOP/s, with the matrix
//                cores busy 37 %, the vector ALU 43 % and LDS 33 % of the time.
// k_attn_join    one thread per 4 output columns of a split row; latency, 6 to
//                12 us.
#include <type_traits>

#include "sdt_device.h"

using namespace sdv;
using namespace sdt;

namespace {

struct AttnArgs {
  Cache c;
  const char *q, *kn, *vn;
  int64_t q_node, q_head, k_node, k_head, v_node, v_head;   // bytes
  const int32_t* off;
  const int32_t* parents;
  const uint64_t* mask;
  int N, max_nodes, Hq, G, mts_max;
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
// heads, up to and including the lane's own.
struct Requests {
  int ctx, first, T, mts, nt, incl;
  uint32_t st;
};

template <int RT, int KT>
__device__ __forceinline__ Requests requests(const AttnArgs& a, int b) {
  Requests r{0, 0, 0, 0, 0, 0, 0};
  if (b < a.c.B) {
    const Nodes nd = request_nodes(a.off, b, a.N, a.max_nodes);
    r.ctx = request_ctx(a.c, b, r.st);
    r.first = nd.first, r.T = nd.T;
    r.mts = (nd.T * a.G + RT - 1) / RT;
    r.nt = (r.ctx + KT - 1) / KT + 1;
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

template <int RT, int KT>
__device__ __forceinline__ Cut cut_units(const AttnArgs& a, const Requests& r, int runs) {
  int total = lane_units(r), nt = r.nt;
  for (int b0 = WAVE; b0 < a.c.B; b0 += WAVE) {
    const Requests q = requests<RT, KT>(a, b0 + (int)threadIdx.x % WAVE);
    total += lane_units(q);
    nt = max(nt, q.nt);
  }
  return Cut{total, max((int)(((unsigned)total + runs - 1) / (unsigned)runs), (wave_max_int(nt) + 31) / 32)};
}

// r / G for a packed row (exact: r < 2^11, G <= 32).
__device__ __forceinline__ int row_node(const AttnArgs& a, int r) { return (int)(((float)r + 0.5f) * a.inv_G); }

// Lane j: the nodes that node j of the request sees, as bits.  Ancestors by
// pointer doubling: six steps reach the root of any tree of 64 nodes.
__device__ __forceinline__ uint64_t seen_by_lane(const AttnArgs& a, int first, int T) {
  const int j = threadIdx.x % WAVE;
  const bool in = j < T;
  if (a.mask) return in ? a.mask[first + j] & (T == 64 ? ~0ull : (1ull << T) - 1) : 0;
  if (!a.parents) return (2ull << j) - 1;
  int up = in ? a.parents[first + j] : -1;
  if (up < -1 || up >= j) up = -1;
  uint64_t m = 1ull << j;
#pragma unroll
  for (int s = 0; s < 6; ++s) {
    const int from = max(up, 0);
    const uint64_t mu = __shfl(m, from);
    const int uu = __shfl(up, from);
    if (up >= 0) m |= mu, up = uu;
  }
  return m;
}

// Any of the 8 elements infinite or not a number.
template <int DT>
__device__ __forceinline__ bool any_nonfinite(const u32x4& w) {
  constexpr uint32_t E = DT == SD_BF16 ? 0x7F80u : 0x7C00u;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    bad |= (w[i] & E) == E || ((w[i] >> 16) & E) == E;
  return bad;
}

template <int DT>
__device__ __forceinline__ uint32_t finite_or_zero(uint32_t u) {
  constexpr uint32_t E = DT == SD_BF16 ? 0x7F80u : 0x7C00u;
  if ((u & E) == E) u &= 0xFFFF0000u;
  if (((u >> 16) & E) == E) u &= 0x0000FFFFu;
  return u;
}

// MT tiles of 16 rows a wave, RG waves over the rows, KG groups of RG waves
// over the keys, NS steps of 32 keys a tile and group.
template <int D_, int MT_, int RG_, int KG_, int NS_>
struct Shape {
  static constexpr int D = D_, MT = MT_, RG = RG_, KG = KG_, NS = NS_;
  static constexpr int NT = WAVE * RG * KG;      // threads
  static constexpr int RT = 16 * MT * RG;        // rows of a workgroup
  static constexpr int KEYS = 32 * NS;           // keys of a group's tile
  static constexpr int KT = KEYS * KG;           // keys of a unit
  static constexpr int CPR = D / 8;              // 16-byte chunks of a row
  static constexpr int NCH = KEYS * CPR / (WAVE * RG);
  static constexpr int TILE = KEYS * D * 2;      // bytes of a group's K (or V) tile
  static constexpr int JR = D + 4;               // floats of a row in the join of the key groups
  static constexpr int JOIN = (KG - 1) * RT * JR * 4;
  static constexpr int LDS = 2 * KG * TILE > JOIN ? 2 * KG * TILE : JOIN;
  static constexpr int SLOT = RT * (D + 3);      // floats of a partial result
  static_assert(KT >= SD_MAX_NODES && KEYS <= 64, "the tree is one tile");
};

template <int DT, typename S>
__global__ __launch_bounds__(S::NT, 2) void k_attn_tiles(AttnArgs a) {
  constexpr int D = S::D, MT = S::MT, RG = S::RG, KG = S::KG, NS = S::NS, KS = D / 32, DTS = D / 16, VA = 2;      // VA: V operands read ahead
  __shared__ __align__(16) char lds[S::LDS];
  __shared__ int odd_value;      // a tree value is infinite or not a number
  const int tid = threadIdx.x, l = tid % WAVE, w = tid / WAVE, n = l & 15, g4 = l >> 4;
  const int rg = w % RG, kg = w / RG;
  char* const ldk = lds + kg * 2 * S::TILE;
  char* const ldv = ldk + S::TILE;
  // scores in base 2; a negative scale is in the queries' signs, and one of zero
  // stays above it so that a masked score times it is still -inf
  const float c = fmaxf(fabsf(a.scale) * 1.4426950408889634f, 1e-30f);
  // Weights are taken against a reference `LIFT` below the running maximum, which
  // may grow by 8 before it moves: fp16 weights lie below 2^15 and keep their
  // precision down to 2^-21 of the largest, something down to 2^-32 of it (a long
  // context's tail beside one dominating key).  bf16 has fp32's exponents.
  constexpr float LIFT = DT == SD_F16 ? 7.0f : 0.0f;

  Requests rq = requests<S::RT, S::KT>(a, l);
  int run, u0, u1;
  if (a.whole) {
    // one workgroup per (request, KV head, row tile): nothing is split
    run = 0, u0 = 0, u1 = 0;
  } else {
    // Workgroups of one XCD take neighbouring runs: row tiles of one KV head
    // find each other's keys in its L2.
    const int runs = gridDim.x;
    const auto [total, per] = cut_units<S::RT, S::KT>(a, rq, runs);
    run = (int)(blockIdx.x % 8) * (runs / 8) + (int)(blockIdx.x / 8);      // runs is a multiple of 8
    if ((int64_t)run * per >= total) return;
    u0 = run * per, u1 = u0 + min(per, total - u0);      // (u0 + per may pass 31 bits)
  }

  // the request (lane f of this 64) that holds unit u0, and its units before
  int b0 = 0, f, in;
  if (a.whole) {
    const int b = blockIdx.x / (a.c.H * a.mts_max), seg = blockIdx.x % (a.c.H * a.mts_max);
    b0 = b & ~(WAVE - 1), f = b & (WAVE - 1);
    if (b0) rq = requests<S::RT, S::KT>(a, b0 + l);
    const int mts = lane_read(rq.mts, f), nt = lane_read(rq.nt, f);
    if (seg % a.mts_max >= mts) return;
    in = (seg / a.mts_max * mts + seg % a.mts_max) * nt;
    u1 = nt;
  } else {
    int left = u0;
    while (left >= lane_units(rq)) {
      left -= lane_units(rq);
      b0 += WAVE;
      rq = requests<S::RT, S::KT>(a, b0 + l);
    }
    f = __builtin_ctzll(__ballot(left < rq.incl));
    in = left - (f ? lane_read(rq.incl, f - 1) : 0);
  }

  while (u0 < u1) {
    const int units = lane_read(rq.incl, f) - (f ? lane_read(rq.incl, f - 1) : 0);
    const int ctx = lane_read(rq.ctx, f), first = lane_read(rq.first, f), T = lane_read(rq.T, f);
    const int mts = lane_read(rq.mts, f), nt = lane_read(rq.nt, f);
    const uint32_t st = (uint32_t)lane_read((int)rq.st, f);
    const int32_t* const tab = table_row(a.c, b0 + f);
    const int rows = T * a.G;
    const int stop = u0 + min(u1 - u0, units - in);
    while (u0 < stop) {
      const int seg = in / nt, t0 = in - seg * nt;
      const int h = seg / mts, mt = seg - h * mts;
      const int t1 = min(nt, t0 + (stop - u0));
      const int row0 = mt * S::RT + rg * 16 * MT;

      // Lane l of a wave looks key l of its group's tile up; the page of the
      // tile after the next one is always on its way.
      auto page_of = [&](int t) {
        const int s = t * S::KT + kg * S::KEYS + l;
        return t < nt - 1 && l < S::KEYS && s < ctx ? tab[s >> a.c.page_shift] : -1;
      };
      const int page0 = page_of(t0);
      int page = page_of(t0 + 1);

      // this wave's queries, as the B operand: lane (n, g4) holds columns
      // 32 ks + 8 g4 .. + 7 of row n
      const s16x8 sign = s16x8{} + (short)(a.scale < 0.0f ? 0x8000 : 0);
      s16x8 q[MT][KS];
      int node[MT];
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const int r = row0 + 16 * m + n;
        const bool on = r < rows;
        node[m] = on ? row_node(a, r) : 0;
        const int head = h * a.G + (on ? r - node[m] * a.G : 0);
        const char* qp = a.q + (int64_t)(first + node[m]) * a.q_node + head * a.q_head;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
          q[m][ks] = on ? *(const s16x8*)(qp + (ks * 32 + g4 * 8) * 2) ^ sign : s16x8{};
      }
      f32x4 o[MT][DTS];
      // sum: of the weights, for the log-sum-exp; norm (any of its 4 equal
      // entries): of the weights as the product sees them, which it is divided by
      f32x4 norm[MT];
      float mx[MT], sum[MT];
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        mx[m] = -INFINITY, sum[m] = 0.0f;
        norm[m] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int d = 0; d < DTS; ++d) o[m][d] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      }
      if (tid == 0) odd_value = 0;

      // Loads are unconditional: a key that is not there reads the pool's first
      // row (or the tree's last) and is masked, its value zeroed on the way to
      // LDS.
      u32x4 rk[S::NCH], rv[S::NCH];
      uint64_t ok = 0;                 // keys of the loaded tile that are there
      auto load = [&](int t, int page) {
        uint64_t kp[S::NCH], vp[S::NCH];      // (as numbers: pointers that meet lose their address space)
        if (t < nt - 1) {
          const bool there = (unsigned)page < (unsigned)a.c.num_pages;
          ok = __ballot(there);
          const int s = t * S::KT + kg * S::KEYS + l;
          const int64_t at = there ? page * a.c.page_stride + h * a.c.head_stride + (s & a.c.page_mask) * a.c.slot_stride : 0;
#pragma unroll
          for (int i = 0; i < S::NCH; ++i) {
            const int lin = (i * RG + rg) * WAVE + l, col = lin % S::CPR;
            const int64_t x = __shfl(at, lin / S::CPR) + col * 16;
            kp[i] = (uint64_t)a.c.k + x;
            vp[i] = (uint64_t)a.c.v + x;
          }
        } else {
          // (opaque to the compiler, which would otherwise keep these addresses
          // in 40 registers throughout the loop)
          int from = first;
          asm volatile("" : "+s"(from));
          const int left = T - kg * S::KEYS;
          ok = left >= 64 ? ~0ull : left > 0 ? (1ull << left) - 1 : 0;
#pragma unroll
          for (int i = 0; i < S::NCH; ++i) {
            const int lin = (i * RG + rg) * WAVE + l, col = lin % S::CPR;
            const int64_t r = from + min(kg * S::KEYS + lin / S::CPR, T - 1);
            kp[i] = (uint64_t)a.kn + r * a.k_node + h * a.k_head + col * 16;
            vp[i] = (uint64_t)a.vn + r * a.v_node + h * a.v_head + col * 16;
          }
        }
        // (one set of loads for both: two would have to meet in copies, which
        // wait for them)
#pragma unroll
        for (int i = 0; i < S::NCH; ++i) {
          rk[i] = *(const global_u32x4*)kp[i];
          rv[i] = *(const global_u32x4*)vp[i];
        }
      };

      load(t0, page0);
      uint64_t vis[MT];
      if (t1 == nt) {
        const uint64_t seen = st ? 0 : seen_by_lane(a, first, T);
#pragma unroll
        for (int m = 0; m < MT; ++m) vis[m] = __shfl(seen, node[m]);
      } else {
#pragma unroll
        for (int m = 0; m < MT; ++m) vis[m] = 0;
      }
      // One tile in LDS against this wave's rows.  MASKED: bit j of on[m] says
      // whether row m sees the group's key j.
      auto tile = [&](auto masked, const uint64_t (&on)[MT]) {
        constexpr bool MASKED = decltype(masked)::value;
        // S^T: lane (n, g4) gets keys 16 s + 4 g4 + r of row n; the reads of 16
        // keys are issued ahead of the products of the 16 before
        auto keys = [&](int s, s16x8 (&kf)[KS]) {
          const int row = s * 16 + n;
#pragma unroll
          for (int ks = 0; ks < KS; ++ks)
            kf[ks] = *(const s16x8*)(ldk + row * (D * 2) + (((ks * 4 + g4) ^ swz<D>(row)) * 16));
        };
        // V^T of 16 columns by 32 keys, keys in the weights' order
        auto values = [&](int i) {
          const int ns = i / DTS, d = i % DTS;
          s16x8 v;
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            const int row = ns * 32 + s * 16 + g4 * 4 + (n >> 2);
            const int at = row * (D * 2) + (((d * 2 + ((n & 3) >> 1)) ^ swz<D>(row)) * 16) + (n & 1) * 8;
            const s16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(ldv + at));
            v[s * 4] = y[0], v[s * 4 + 1] = y[1], v[s * 4 + 2] = y[2], v[s * 4 + 3] = y[3];
          }
          return v;
        };
        f32x4 x[2 * NS][MT];
        s16x8 kf[2][KS], vf[VA];
        keys(0, kf[0]);
#pragma unroll
        for (int s = 0; s < 2 * NS; ++s) {
          if (s + 1 < 2 * NS) {
            keys(s + 1, kf[(s + 1) & 1]);
          } else {
#pragma unroll
            for (int i = 0; i < VA; ++i) vf[i] = values(i);
          }
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            x[s][m] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) x[s][m] = mfma<DT>(kf[s & 1][ks], q[m][ks], x[s][m]);
          }
        }
        float ms[MT];
        bool grown = false;
        float top[MT];
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          top[m] = -INFINITY;
          const uint64_t mine = on[m] >> (g4 * 4);      // bit 16 s + r: this lane's
#pragma unroll
          for (int s = 0; s < 2 * NS; ++s)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              if constexpr (MASKED)
                x[s][m][r] = (mine >> (s * 16 + r) & 1) ? x[s][m][r] : -INFINITY;
              top[m] = fmaxf(top[m], x[s][m][r]);
            }
          top[m] = quad_max(top[m]) * c - LIFT;
          // the sums are rescaled only when a maximum grows by more than 2^8:
          // until then weights up to 2^8 (2^15) are as exact as those below
          grown |= top[m] > mx[m] + 8.0f;
        }
        if (__any(grown)) {
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            const float mn = fmaxf(mx[m], top[m]);
            const float f = mn > -INFINITY ? fast_exp2(mx[m] - mn) : 1.0f;
            mx[m] = mn;
            sum[m] *= f;
            norm[m] *= f;
#pragma unroll
            for (int d = 0; d < DTS; ++d) o[m][d] *= f;
          }
        }
#pragma unroll
        for (int m = 0; m < MT; ++m) ms[m] = mx[m] > -INFINITY ? mx[m] : 0.0f;
#pragma unroll
        for (int ns = 0; ns < NS; ++ns) {
          s16x8 p[MT];
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
              for (int r = 0; r < 4; ++r) {
                const float y = fast_exp2(fmaf(x[ns * 2 + s][m][r], c, -ms[m]));
                sum[m] += y;
                // the weights enter the product in the element type, half a
                // step off each; dividing by the sum of the rounded ones takes
                // the rounding of a weight that dominates out again
                p[m][s * 4 + r] = (short)from_f32<DT>(y);
              }
          const s16x8 ones = s16x8{} + (short)(DT == SD_BF16 ? 0x3F80 : 0x3C00);
#pragma unroll
          for (int m = 0; m < MT; ++m) norm[m] = mfma<DT>(ones, p[m], norm[m]);
          // O^T
#pragma unroll
          for (int d = 0; d < DTS; ++d) {
            const int i = ns * DTS + d;
#pragma unroll
            for (int m = 0; m < MT; ++m) o[m][d] = mfma<DT>(vf[i % VA], p[m], o[m][d]);
            if (i + VA < NS * DTS) vf[i % VA] = values(i + VA);
          }
        }
      };

      for (int t = t0; t < t1; ++t) {
        if (RG > 1 || t == t0) __syncthreads();      // the tile before has been read
        const bool tree = t == nt - 1;
        const uint64_t valid = ok;
        constexpr uint64_t FULL = S::KEYS == 64 ? ~0ull : (1ull << (S::KEYS % 64)) - 1;
        if (tree || (valid & FULL) != FULL) {
#pragma unroll
          for (int i = 0; i < S::NCH; ++i) {
            const int row = ((i * RG + rg) * WAVE + l) / S::CPR;
            if (!(valid >> row & 1)) {
              rv[i] = u32x4{0, 0, 0, 0};
            } else if (tree && any_nonfinite<DT>(rv[i])) {
              // 0 x infinity in the product would reach rows that do not see
              // this node: such values are added at the end instead
              odd_value = 1;
#pragma unroll
              for (int j = 0; j < 4; ++j) rv[i][j] = finite_or_zero<DT>(rv[i][j]);
            }
          }
        }
#pragma unroll
        for (int i = 0; i < S::NCH; ++i) {
          const int lin = (i * RG + rg) * WAVE + l, row = lin / S::CPR, col = lin % S::CPR;
          const int at = row * (D * 2) + ((col ^ swz<D>(row)) * 16);
          *(u32x4*)(ldk + at) = rk[i];
          *(u32x4*)(ldv + at) = rv[i];
        }
        if (RG > 1) __syncthreads();
        else __builtin_amdgcn_wave_barrier();
        if (t + 1 < t1) {
          load(t + 1, page);
          page = page_of(t + 2);
        }
        if (!tree && (valid & FULL) == FULL) {
          tile(std::false_type{}, vis);
        } else {
          uint64_t on[MT];
#pragma unroll
          for (int m = 0; m < MT; ++m)      // (the tree's 64 nodes are in the first groups' keys)
            on[m] = !tree ? valid : S::KT <= 64 || kg * S::KEYS < 64 ? valid & vis[m] >> (kg * S::KEYS) : 0;
          tile(std::true_type{}, on);
        }
        if (RG == 1) __builtin_amdgcn_wave_barrier();
      }
#pragma unroll
      for (int m = 0; m < MT; ++m) sum[m] = quad_sum(sum[m]);

      // key groups: the first one adds the others up
      if (KG > 1) {
        float* const sh = (float*)lds;
        __syncthreads();
        if (kg > 0) {
          float* const z = sh + ((kg - 1) * RG + rg) * 16 * MT * S::JR;
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            float* const zr = z + (16 * m + n) * S::JR;
#pragma unroll
            for (int d = 0; d < DTS; ++d) *(f32x4*)(zr + d * 16 + g4 * 4) = o[m][d];
            if (g4 == 0) zr[D] = mx[m], zr[D + 1] = sum[m], zr[D + 2] = norm[m][0];
          }
        }
        __syncthreads();
        if (kg == 0) {
          for (int k2 = 1; k2 < KG; ++k2) {
            const float* const z = sh + ((k2 - 1) * RG + rg) * 16 * MT * S::JR;
#pragma unroll
            for (int m = 0; m < MT; ++m) {
              const float* const zr = z + (16 * m + n) * S::JR;
              const float m2 = zr[D], mn = fmaxf(mx[m], m2), ms = mn > -INFINITY ? mn : 0.0f;
              const float f1 = fast_exp2(mx[m] - ms), f2 = fast_exp2(m2 - ms);
              mx[m] = mn;
              sum[m] = sum[m] * f1 + zr[D + 1] * f2;
              norm[m][0] = norm[m][0] * f1 + zr[D + 2] * f2;
#pragma unroll
              for (int d = 0; d < DTS; ++d) o[m][d] = o[m][d] * f1 + *(const f32x4*)(zr + d * 16 + g4 * 4) * f2;
            }
          }
        }
      }
      if (RG > 1 && KG == 1) __syncthreads();      // odd_value
      if (kg == 0) {
        if (t1 == nt && odd_value) {
#pragma unroll
          for (int m = 0; m < MT; ++m)
            for (int j = 0; j < T; ++j) {
              const uint16_t* v = (const uint16_t*)(a.vn + (int64_t)(first + j) * a.v_node + h * a.v_head);
#pragma unroll
              for (int d = 0; d < DTS; ++d)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                  const float y = to_f32<DT>(v[d * 16 + g4 * 4 + r]);
                  if ((vis[m] >> j & 1) && !(fabsf(y) < INFINITY)) o[m][d][r] += y;
                }
            }
        }
        const bool whole = t0 == 0 && t1 == nt;
        float* const part = a.part + (int64_t)(run * 2 + (t0 == 0)) * S::SLOT;
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const int lr = rg * 16 * MT + 16 * m + n, r = mt * S::RT + lr;
          if (r >= rows) continue;
          if (whole) {
            const bool none = sum[m] == 0.0f;
            const float inv = none ? 0.0f : 1.0f / norm[m][0];
            const int64_t at = (int64_t)(first + node[m]) * a.Hq + h * a.G + (r - node[m] * a.G);
            char* const out = a.out + at * (D * 2);
#pragma unroll
            for (int d = 0; d < DTS; ++d) {
              uint32_t u[2];
#pragma unroll
              for (int r2 = 0; r2 < 2; ++r2)
                u[r2] = (uint32_t)from_f32<DT>(none ? 0.0f : o[m][d][2 * r2] * inv) |
                        (uint32_t)from_f32<DT>(none ? 0.0f : o[m][d][2 * r2 + 1] * inv) << 16;
              *(uint2*)(out + (d * 16 + g4 * 4) * 2) = make_uint2(u[0], u[1]);
            }
            if (a.lse && g4 == 0) a.lse[at] = none ? -INFINITY : (mx[m] + __log2f(sum[m])) * 0.6931471805599453f;
          } else {
            float* const z = part + lr * D;
#pragma unroll
            for (int d = 0; d < DTS; ++d) *(f32x4*)(z + d * 16 + g4 * 4) = o[m][d];
            if (g4 == 0) {
              part[S::RT * D + lr] = mx[m];
              part[S::RT * D + S::RT + lr] = sum[m];
              part[S::RT * D + 2 * S::RT + lr] = norm[m][0];
            }
          }
        }
      }
      __syncthreads();      // LDS is the next segment's
      u0 += t1 - t0;
      in += t1 - t0;
    }
    in = 0;
    if (++f == WAVE && u0 < u1) {
      f = 0, b0 += WAVE;
      rq = requests<S::RT, S::KT>(a, b0 + l);
    }
  }
}

// Rows whose key tiles went to several runs: their parts in the order of the
// runs, JN at a time.  grid (4-column groups of a row tile / 256, H * row
// tiles, B).
template <int DT, typename S>
__global__ __launch_bounds__(256) void k_attn_join(AttnArgs a, int runs) {
  constexpr int D = S::D, GPR = D / 4, JN = 8;
  const int b = blockIdx.z, h = blockIdx.y / a.mts_max, mt = blockIdx.y % a.mts_max, l = threadIdx.x % WAVE;
  Requests rq = requests<S::RT, S::KT>(a, l);
  const int per = cut_units<S::RT, S::KT>(a, rq, runs).per;
  int before = 0;
  for (int b0 = 0; b0 + WAVE <= b; b0 += WAVE) {
    before += lane_units(rq);
    rq = requests<S::RT, S::KT>(a, b0 + WAVE + l);
  }
  const int f = b % WAVE, nt = lane_read(rq.nt, f), mts = lane_read(rq.mts, f);
  if (mt >= mts) return;
  if (f) before += lane_read(rq.incl, f - 1);
  const int s = before + (h * mts + mt) * nt;
  const int w0 = (int)((unsigned)s / (unsigned)per), w1 = (int)((unsigned)(s + nt - 1) / (unsigned)per);
  const int lin = blockIdx.x * 256 + threadIdx.x, lr = lin / GPR, col = lin % GPR, r = mt * S::RT + lr;
  if (w0 == w1 || r >= lane_read(rq.T, f) * a.G) return;
  float m = -INFINITY, sum = 0.0f, norm = 0.0f;
  f32x4 o = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int w = w0; w <= w1; w += JN) {
    float pm[JN], ps[JN], pn[JN];
    f32x4 po[JN];
#pragma unroll
    for (int i = 0; i < JN; ++i) {
      const int wi = min(w + i, w1);
      const float* z = a.part + (int64_t)(wi * 2 + (wi == w0)) * S::SLOT;
      pm[i] = z[S::RT * D + lr];
      ps[i] = z[S::RT * D + S::RT + lr];
      pn[i] = z[S::RT * D + 2 * S::RT + lr];
      po[i] = *(const f32x4*)(z + lr * D + col * 4);
    }
#pragma unroll
    for (int i = 0; i < JN; ++i) {
      if (w + i > w1) break;
      const float mn = fmaxf(m, pm[i]), ms = mn > -INFINITY ? mn : 0.0f;
      const float f1 = fast_exp2(m - ms), f2 = fast_exp2(pm[i] - ms);
      m = mn;
      sum = sum * f1 + ps[i] * f2;
      norm = norm * f1 + pn[i] * f2;
      o = o * f1 + po[i] * f2;
    }
  }
  const bool none = sum == 0.0f;
  const float inv = none ? 0.0f : 1.0f / norm;
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
__global__ __launch_bounds__(WAVE) void k_tree_status(AttnArgs a) {
  const int b = blockIdx.x, l = threadIdx.x;
  const Nodes nd = request_nodes(a.off, b, a.N, a.max_nodes);
  uint32_t st = nd.st;
  const int ctx = request_ctx(a.c, b, st);
  const int32_t* tab = table_row(a.c, b);
  bool bad_page = false, bad_tree = false;
  for (int p = l; p < (ctx + a.c.page_mask) >> a.c.page_shift; p += WAVE)
    bad_page |= (unsigned)tab[p] >= (unsigned)a.c.num_pages;
  if (a.parents && !a.mask && l < nd.T) {
    const int p = a.parents[nd.first + l];
    bad_tree = p < -1 || p >= l;
  }
  if (__any(bad_page)) st |= SD_ST_BAD_PAGE;
  if (__any(bad_tree)) st |= SD_ST_BAD_TREE;
  if (l == 0) a.status[b] = st;
}

int check(const sd_tree_attention_args_t* p) {
  if (!p) return SD_EINVAL;
  const int rc = check_cache(p->cache);
  if (rc) return rc;
  if (!rows_ok(p->q, p->q_node, p->q_head) || !rows_ok(p->k_new, p->k_node, p->k_head) ||
      !rows_ok(p->v_new, p->v_node, p->v_head) || !p->node_offsets || p->N < 1 ||
      p->max_nodes < 1 || p->H_q < 1 || p->H_q % p->cache.H_kv || !isfinite(p->scale))
    return SD_EINVAL;
  if (p->max_nodes > SD_MAX_NODES || p->H_q / p->cache.H_kv > SD_MAX_GROUP || p->H_q > 65535)
    return SD_EUNSUPPORTED;
  return SD_OK;
}

AttnArgs device_args(const sd_tree_attention_args_t* p) {
  AttnArgs a;
  a.c = device_cache(p->cache);
  a.q = static_cast<const char*>(p->q);
  a.kn = static_cast<const char*>(p->k_new);
  a.vn = static_cast<const char*>(p->v_new);
  a.q_node = p->q_node * 2, a.q_head = p->q_head * 2;
  a.k_node = p->k_node * 2, a.k_head = p->k_head * 2;
  a.v_node = p->v_node * 2, a.v_head = p->v_head * 2;
  a.off = p->node_offsets;
  a.parents = p->parents;
  a.mask = p->tree_mask;
  a.N = p->N;
  a.max_nodes = p->max_nodes;
  a.Hq = p->H_q;
  a.G = p->H_q / p->cache.H_kv;
  a.inv_G = 1.0f / (float)a.G;
  a.scale = p->scale;
  return a;
}

// The shape for `rows` packed rows a KV head: fewer rows leave more waves to
// the keys.  16 rows a wave need no register spills and win up to 128 rows (63
// rows 49 us against 64 for 32 a wave, 28 rows 52 against 90, 112 rows 61 against
// 78); past that 32 a wave halve the LDS reads (448 rows 462 us against 600).
// f(Shape{}) is called with the one taken.
template <int D, typename F>
auto with_shape(int rows, F&& f) {
  if (rows <= 16) return f(Shape<D, 1, 1, 4, 1>{});
  if (rows <= 32) return f(Shape<D, 1, 2, 2, 1>{});
  if (rows <= 64) return f(Shape<D, 1, 4, 1, 2>{});
  if (rows <= 128) return f(Shape<D, 1, 8, 1, 2>{});
  return f(Shape<D, 2, 8, 1, 2>{});
}

// Workgroups that share the unit list: two per CU of 4 waves, one of 8.
template <typename S>
constexpr int run_count() {
  return S::NT == 512 ? 256 : 512;
}

// Where a table holds no more than this many key tiles, splitting them and
// joining the parts in a second launch costs more than it saves (517 slots of
// one request: 9 us in one launch, 6 + 5 us and a launch's host time in two).
constexpr int WHOLE_TILES = 8;

// How a call is cut up.
struct Plan {
  int mts_max;                // row tiles of a KV head
  int64_t segments, tiles;    // (request, KV head, row tile)s, and key tiles of one
  bool fits, whole;
};

template <typename S>
Plan plan(const sd_kv_cache_t& c, int rows) {
  Plan p;
  p.mts_max = (rows + S::RT - 1) / S::RT;
  p.segments = (int64_t)c.B * c.H_kv * p.mts_max;
  p.tiles = ((int64_t)c.max_pages * c.page_size + S::KT - 1) / S::KT + 1;
  p.fits = p.segments <= 0x7FFFFFFF / p.tiles;      // units are counted in 32 bits
  // (and a grid dimension holds less than 2^32 threads)
  p.whole = p.tiles <= WHOLE_TILES && p.segments * S::NT <= UINT32_MAX;
  return p;
}

template <int DT, int D>
int launch(AttnArgs a, const sd_kv_cache_t& c, int rows, hipStream_t st) {
  return with_shape<D>(rows, [&](auto s) {
    using S = decltype(s);
    constexpr int runs = run_count<S>();
    const Plan p = plan<S>(c, rows);
    const int64_t segments = p.segments;
    a.mts_max = p.mts_max;
    a.whole = p.whole;
    hipLaunchKernelGGL((k_attn_tiles<DT, S>), dim3(a.whole ? (unsigned)segments : (unsigned)runs), dim3(S::NT), 0, st, a);
    if (hipGetLastError() != hipSuccess) return SD_EHIP;
    if (a.whole) return SD_OK;
    const dim3 grid(S::RT * (D / 4) / 256, a.c.H * a.mts_max, a.c.B);
    hipLaunchKernelGGL((k_attn_join<DT, S>), grid, dim3(256), 0, st, a, runs);
    return hipGetLastError() == hipSuccess ? SD_OK : SD_EHIP;
  });
}

}  // namespace

extern "C" int sd_tree_attention_workspace_bytes(const sd_tree_attention_args_t* args, size_t* bytes) {
  if (!bytes) return SD_EINVAL;
  const int rc = check(args);
  if (rc) return rc;
  const int rows = args->max_nodes * (args->H_q / args->cache.H_kv);
  auto size = [&](auto s) {
    using S = decltype(s);
    const Plan p = plan<S>(args->cache, rows);
    *bytes = p.whole ? 0 : (size_t)run_count<S>() * 2 * S::SLOT * sizeof(float);
    return p.fits ? SD_OK : SD_EUNSUPPORTED;
  };
  return args->cache.D == 64 ? with_shape<64>(rows, size) : with_shape<128>(rows, size);
}

extern "C" int sd_tree_attention(const sd_tree_attention_args_t* args, void* workspace,
                                 size_t workspace_bytes, void* out, float* out_lse,
                                 uint32_t* out_status, void* stream) {
  size_t need = 0;
  int rc = sd_tree_attention_workspace_bytes(args, &need);
  if (rc) return rc;
  if (!out || !aligned16(out)) return SD_EINVAL;
  if (out == args->k_new || out == args->v_new || out == args->cache.k || out == args->cache.v) return SD_EINVAL;
  // a query row is read by the workgroups of its own result alone, before they
  // write it or before the join does
  if (out == args->q && (args->q_head != args->cache.D || args->q_node != (int64_t)args->H_q * args->cache.D))
    return SD_EINVAL;
  if (need && (!workspace || workspace_bytes < need || !aligned16(workspace))) return SD_EWORKSPACE;
  AttnArgs a = device_args(args);
  a.out = static_cast<char*>(out);
  a.lse = out_lse;
  a.status = out_status;
  hipStream_t st = static_cast<hipStream_t>(stream);
  a.part = static_cast<float*>(workspace);
  const int rows = a.max_nodes * a.G, D = args->cache.D;
  if (args->cache.dtype == SD_BF16)
    rc = D == 64 ? launch<SD_BF16, 64>(a, args->cache, rows, st) : launch<SD_BF16, 128>(a, args->cache, rows, st);
  else
    rc = D == 64 ? launch<SD_F16, 64>(a, args->cache, rows, st) : launch<SD_F16, 128>(a, args->cache, rows, st);
  if (rc) return rc;
  if (out_status) {
    hipLaunchKernelGGL(k_tree_status, dim3(a.c.B), dim3(WAVE), 0, st, a);
    if (hipGetLastError() != hipSuccess) return SD_EHIP;
  }
  return SD_OK;
}
