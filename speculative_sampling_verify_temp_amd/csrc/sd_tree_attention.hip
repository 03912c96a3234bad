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
// k_attn_join    one thread per 4 output columns of a split row.
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
  int N, max_nodes, Hq, G;
  float scale;
  float* part;      // partial results, two slots a run
  char* out;
  float* lse;
  uint32_t* status;
};

// The nodes that node i of the request sees, as bits.
__device__ __forceinline__ uint64_t sees(const AttnArgs& a, const Nodes& nd, int i) {
  const uint64_t own = nd.T == 64 ? ~0ull : (1ull << nd.T) - 1;
  if (a.mask) return a.mask[nd.first + i] & own;
  if (!a.parents) return (2ull << i) - 1;
  uint64_t m = 0;
  for (int j = i; j >= 0;) {
    m |= 1ull << j;
    const int p = a.parents[nd.first + j];
    j = p < j ? p : -1;      // p < -1 ends the walk too
  }
  return m;
}

// ---- the unit list ----

// Row tiles and key tiles of request b, and its units (all KV heads).
struct Extent {
  int rows, mts, nt;
  double units;
};

template <int RT, int KT>
__device__ __forceinline__ Extent request_extent(const AttnArgs& a, int b) {
  Extent e{0, 0, 0, 0.0};
  if (b >= a.c.B) return e;
  const Nodes nd = request_nodes(a.off, b, a.N, a.max_nodes);
  uint32_t st = 0;
  const int ctx = request_ctx(a.c, b, st);
  e.rows = nd.T * a.G;
  e.mts = (e.rows + RT - 1) / RT;
  e.nt = (ctx + KT - 1) / KT + 1;
  e.units = (double)e.mts * e.nt * a.c.H;     // exact: below 2^53
  return e;
}

// All units, by every wave alike.
template <int RT, int KT>
__device__ __forceinline__ double total_units(const AttnArgs& a) {
  double u = 0.0;
  for (int b0 = 0; b0 < a.c.B; b0 += WAVE)
    u += wave_sum(request_extent<RT, KT>(a, b0 + threadIdx.x % WAVE).units);
  return u;
}

__device__ __forceinline__ int64_t run_length(double units, int runs) {
  return ((int64_t)units + runs - 1) / runs;
}

// Any of the 8 elements infinite or not a number.
template <int DT>
__device__ __forceinline__ bool any_nonfinite(const uint4& w) {
  constexpr uint32_t E = DT == SD_BF16 ? 0x7F80u : 0x7C00u;
  bool bad = false;
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    bad |= (u[i] & E) == E || ((u[i] >> 16) & E) == E;
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
  static constexpr int JOIN = (KG - 1) * RT * (D + 2) * 4;
  static constexpr int LDS = 2 * KG * TILE > JOIN ? 2 * KG * TILE : JOIN;
  static constexpr int SLOT = RT * (D + 2);      // floats of a partial result
  static_assert(KT >= SD_MAX_NODES && KEYS <= 64, "the tree is one tile");
};

template <int DT, typename S>
__global__ __launch_bounds__(S::NT, 2) void k_attn_tiles(AttnArgs a) {
  constexpr int D = S::D, MT = S::MT, RG = S::RG, KG = S::KG, NS = S::NS, KS = D / 32, DTS = D / 16;
  __shared__ __align__(16) char lds[S::LDS];
  __shared__ int odd_value;      // a tree value is infinite or not a number
  const int tid = threadIdx.x, l = tid % WAVE, w = tid / WAVE, n = l & 15, g4 = l >> 4;
  const int rg = w % RG, kg = w / RG;
  char* const ldk = lds + kg * 2 * S::TILE;
  char* const ldv = ldk + S::TILE;
  const float c = a.scale * 1.4426950408889634f;

  // Workgroups of one XCD take neighbouring runs: row tiles of one KV head
  // find each other's keys in its L2.
  const int runs = gridDim.x, per_xcd = runs / 8;
  const int run = runs % 8 ? (int)blockIdx.x : (int)(blockIdx.x % 8) * per_xcd + (int)(blockIdx.x / 8);
  const int64_t total = (int64_t)total_units<S::RT, S::KT>(a);
  const int64_t per = run_length((double)total, runs);
  int64_t u0 = run * per, u1 = min(total, u0 + per);
  if (u0 >= u1) return;

  // the request that holds unit u0
  int b = 0;
  int64_t before = 0;
  for (int b0 = 0;; b0 += WAVE) {
    const double incl = wave_incl_scan(request_extent<S::RT, S::KT>(a, b0 + l).units);
    const uint64_t over = __ballot((double)(u0 - before) < incl);
    if (over) {
      const int f = __builtin_ctzll(over);
      b = b0 + f;
      if (f) before += (int64_t)lane_read(incl, f - 1);
      break;
    }
    before += (int64_t)lane_read(incl, WAVE - 1);
  }
  b = __builtin_amdgcn_readfirstlane(b);
  int64_t in = u0 - before;      // units of request b before ours

  for (; u0 < u1; ++b, in = 0) {
    const Extent e = request_extent<S::RT, S::KT>(a, b);
    const int64_t mine = (int64_t)e.units - in;
    if (mine <= 0) continue;
    const Nodes nd = request_nodes(a.off, b, a.N, a.max_nodes);
    uint32_t st = 0;
    const int ctx = request_ctx(a.c, b, st);
    const int32_t* tab = table_row(a.c, b);
    const int64_t stop = min(u1, u0 + mine);
    while (u0 < stop) {
      const int seg = (int)(in / e.nt), t0 = (int)(in % e.nt);
      const int h = seg / e.mts, mt = seg % e.mts;
      const int t1 = (int)min((int64_t)e.nt, t0 + (stop - u0));
      const int row0 = mt * S::RT + rg * 16 * MT;

      // this wave's queries, as the B operand: lane (n, g4) holds columns
      // 32 ks + 8 g4 .. + 7 of row n
      s16x8 q[MT][KS];
      uint64_t vis[MT];
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const int r = row0 + 16 * m + n;
        const bool on = r < e.rows;
        const int node = on ? r / a.G : 0, head = h * a.G + (on ? r % a.G : 0);
        const char* qp = a.q + (int64_t)(nd.first + node) * a.q_node + head * a.q_head;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          q[m][ks] = on ? *(const s16x8*)(qp + (ks * 32 + g4 * 8) * 2) : s16x8{};
        }
        vis[m] = on && !st && t1 == e.nt ? sees(a, nd, node) : 0;
      }
      f32x4 o[MT][DTS];
      float mx[MT], sum[MT];
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        mx[m] = -INFINITY, sum[m] = 0.0f;
#pragma unroll
        for (int d = 0; d < DTS; ++d) o[m][d] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      }
      if (tid == 0) odd_value = 0;

      // Lane l of a wave looks key l of its group's tile up; the page of the
      // tile after the next one is always on its way.
      auto page_of = [&](int t) {
        const int s = t * S::KT + kg * S::KEYS + l;
        return t < e.nt - 1 && l < S::KEYS && s < ctx ? tab[s >> a.c.page_shift] : -1;
      };
      uint4 rk[S::NCH], rv[S::NCH];
      uint64_t ok = 0;
      auto load = [&](int t, int page) {
        if (t == e.nt - 1) {
          const int left = nd.T - kg * S::KEYS;
          ok = left >= 64 ? ~0ull : left > 0 ? (1ull << left) - 1 : 0;
        } else {
          ok = __ballot((unsigned)page < (unsigned)a.c.num_pages);
        }
        const int s = t * S::KT + kg * S::KEYS + l;
        const int64_t at = page * a.c.page_stride + h * a.c.head_stride + (s & a.c.page_mask) * a.c.slot_stride;
#pragma unroll
        for (int i = 0; i < S::NCH; ++i) {
          const int lin = (i * RG + rg) * WAVE + l, row = lin / S::CPR, col = lin % S::CPR;
          rk[i] = rv[i] = make_uint4(0, 0, 0, 0);
          const char *kp, *vp;
          if (t == e.nt - 1) {
            const int64_t r = nd.first + kg * S::KEYS + row;
            kp = a.kn + r * a.k_node + h * a.k_head;
            vp = a.vn + r * a.v_node + h * a.v_head;
          } else {
            const int64_t x = __shfl(at, row);
            kp = a.c.k + x;
            vp = a.c.v + x;
          }
          if (ok >> row & 1) {
            rk[i] = *(const uint4*)(kp + col * 16);
            rv[i] = *(const uint4*)(vp + col * 16);
          }
        }
      };

      load(t0, page_of(t0));
      int page = page_of(t0 + 1);
      for (int t = t0; t < t1; ++t) {
        if (RG > 1 || t == t0) __syncthreads();      // the tile before has been read
        const bool tree = t == e.nt - 1;
#pragma unroll
        for (int i = 0; i < S::NCH; ++i) {
          const int lin = (i * RG + rg) * WAVE + l, row = lin / S::CPR, col = lin % S::CPR;
          const int at = row * (D * 2) + ((col ^ swz<D>(row)) * 16);
          if (tree && any_nonfinite<DT>(rv[i])) {
            // 0 x infinity in the product would reach rows that do not see
            // this node: such values are added at the end instead
            odd_value = 1;
            rv[i] = make_uint4(finite_or_zero<DT>(rv[i].x), finite_or_zero<DT>(rv[i].y),
                               finite_or_zero<DT>(rv[i].z), finite_or_zero<DT>(rv[i].w));
          }
          *(uint4*)(ldk + at) = rk[i];
          *(uint4*)(ldv + at) = rv[i];
        }
        const uint64_t valid = ok;
        if (RG > 1) __syncthreads();
        else __builtin_amdgcn_wave_barrier();
        if (t + 1 < t1) {
          load(t + 1, page);
          page = page_of(t + 2);
        }
#pragma unroll
        for (int ns = 0; ns < NS; ++ns) {
          // S^T: lane (n, g4) gets keys 16 s + 4 g4 + r of row n
          f32x4 x[2][MT];
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            const int row = ns * 32 + s * 16 + n;
#pragma unroll
            for (int m = 0; m < MT; ++m) x[s][m] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
              const s16x8 k = *(const s16x8*)(ldk + row * (D * 2) + (((ks * 4 + g4) ^ swz<D>(row)) * 16));
#pragma unroll
              for (int m = 0; m < MT; ++m) x[s][m] = mfma<DT>(k, q[m][ks], x[s][m]);
            }
          }
          const uint32_t some = (uint32_t)(valid >> (ns * 32));
          s16x8 p[MT];
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            float top = -INFINITY;
            const uint32_t on = tree ? some & (uint32_t)(vis[m] >> (kg * S::KEYS + ns * 32)) : some;
            if (tree || some != 0xFFFFFFFFu) {
#pragma unroll
              for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                  x[s][m][r] = (on >> (s * 16 + g4 * 4 + r) & 1) ? x[s][m][r] * c : -INFINITY;
            } else {
#pragma unroll
              for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int r = 0; r < 4; ++r) x[s][m][r] *= c;
            }
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
              for (int r = 0; r < 4; ++r) top = fmaxf(top, x[s][m][r]);
            top = quad_max(top);
            // the sums are rescaled only when a maximum grows by more than
            // 2^8: until then weights up to 2^8 are as exact as those below 1
            if (__any(top > mx[m] + 8.0f)) {
              const float mn = fmaxf(mx[m], top);
              const float f = mn > -INFINITY ? fast_exp2(mx[m] - mn) : 1.0f;
              mx[m] = mn;
              sum[m] *= f;
#pragma unroll
              for (int d = 0; d < DTS; ++d) o[m][d] *= f;
            }
            const float ms = mx[m] > -INFINITY ? mx[m] : 0.0f;
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
              for (int r = 0; r < 4; ++r) {
                const float y = fast_exp2(x[s][m][r] - ms);
                sum[m] += y;
                // the weights enter the product in the element type: half a
                // step each, and the sum keeps their fp32 values
                p[m][s * 4 + r] = (short)from_f32<DT>(y);
              }
          }
          // O^T: V^T of 16 columns by 32 keys, keys in the weights' order
#pragma unroll
          for (int d = 0; d < DTS; ++d) {
            s16x8 v;
#pragma unroll
            for (int s = 0; s < 2; ++s) {
              const int row = ns * 32 + s * 16 + g4 * 4 + (n >> 2);
              const int at = row * (D * 2) + (((d * 2 + ((n & 3) >> 1)) ^ swz<D>(row)) * 16) + (n & 1) * 8;
              const s16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(ldv + at));
              v[s * 4] = y[0], v[s * 4 + 1] = y[1], v[s * 4 + 2] = y[2], v[s * 4 + 3] = y[3];
            }
#pragma unroll
            for (int m = 0; m < MT; ++m) o[m][d] = mfma<DT>(v, p[m], o[m][d]);
          }
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
          float* const z = sh + ((kg - 1) * RG + rg) * 16 * MT * (D + 2);
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            float* const zr = z + (16 * m + n) * (D + 2);
#pragma unroll
            for (int d = 0; d < DTS; ++d)
#pragma unroll
              for (int r = 0; r < 4; ++r) zr[d * 16 + g4 * 4 + r] = o[m][d][r];
            if (g4 == 0) zr[D] = mx[m], zr[D + 1] = sum[m];
          }
        }
        __syncthreads();
        if (kg == 0) {
          for (int k2 = 1; k2 < KG; ++k2) {
            const float* const z = sh + ((k2 - 1) * RG + rg) * 16 * MT * (D + 2);
#pragma unroll
            for (int m = 0; m < MT; ++m) {
              const float* const zr = z + (16 * m + n) * (D + 2);
              const float m2 = zr[D], mn = fmaxf(mx[m], m2), ms = mn > -INFINITY ? mn : 0.0f;
              const float f1 = fast_exp2(mx[m] - ms), f2 = fast_exp2(m2 - ms);
              mx[m] = mn;
              sum[m] = sum[m] * f1 + zr[D + 1] * f2;
#pragma unroll
              for (int d = 0; d < DTS; ++d)
#pragma unroll
                for (int r = 0; r < 4; ++r) o[m][d][r] = o[m][d][r] * f1 + zr[d * 16 + g4 * 4 + r] * f2;
            }
          }
        }
      }
      if (RG > 1 && KG == 1) __syncthreads();      // odd_value
      if (kg == 0) {
        if (t1 == e.nt && odd_value) {
#pragma unroll
          for (int m = 0; m < MT; ++m)
            for (int j = 0; j < nd.T; ++j) {
              const uint16_t* v = (const uint16_t*)(a.vn + (int64_t)(nd.first + j) * a.v_node + h * a.v_head);
#pragma unroll
              for (int d = 0; d < DTS; ++d)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                  const float y = to_f32<DT>(v[d * 16 + g4 * 4 + r]);
                  if ((vis[m] >> j & 1) && !(fabsf(y) < INFINITY)) o[m][d][r] += y;
                }
            }
        }
        const bool whole = t0 == 0 && t1 == e.nt;
        float* const part = a.part + (int64_t)(run * 2 + (t0 == 0)) * S::SLOT;
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const int lr = rg * 16 * MT + 16 * m + n, r = mt * S::RT + lr;
          if (r >= e.rows) continue;
          if (whole) {
            const bool none = sum[m] == 0.0f;
            const float inv = none ? 0.0f : 1.0f / sum[m];
            const int64_t at = (int64_t)(nd.first + r / a.G) * a.Hq + h * a.G + r % a.G;
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
            }
          }
        }
      }
      __syncthreads();      // LDS is the next segment's
      u0 += t1 - t0;
      in += t1 - t0;
    }
  }
}

// Rows whose key tiles went to several runs: their parts in the order of the
// runs.  grid (4-column groups of a row tile / 256, H * row tiles, B).
template <int DT, typename S>
__global__ __launch_bounds__(256) void k_attn_join(AttnArgs a, int runs, int mts_max) {
  constexpr int D = S::D, GPR = D / 4;
  const int b = blockIdx.z, h = blockIdx.y / mts_max, mt = blockIdx.y % mts_max, l = threadIdx.x % WAVE;
  const Extent e = request_extent<S::RT, S::KT>(a, b);
  if (mt >= e.mts) return;
  const int lin = blockIdx.x * 256 + threadIdx.x, lr = lin / GPR, col = lin % GPR;
  const int64_t per = run_length(total_units<S::RT, S::KT>(a), runs);
  double before = 0.0;
  for (int b0 = 0; b0 < b; b0 += WAVE)
    before += wave_sum(b0 + l < b ? request_extent<S::RT, S::KT>(a, b0 + l).units : 0.0);
  const int64_t s = (int64_t)before + (int64_t)(h * e.mts + mt) * e.nt;
  const int64_t w0 = s / per, w1 = (s + e.nt - 1) / per;
  const int r = mt * S::RT + lr;
  if (w0 == w1 || lr >= S::RT || r >= e.rows) return;
  auto part = [&](int64_t w) { return a.part + (w * 2 + (w == w0)) * S::SLOT; };
  float m = -INFINITY;
  for (int64_t w = w0; w <= w1; ++w) m = fmaxf(m, part(w)[S::RT * D + lr]);
  const float ms = m > -INFINITY ? m : 0.0f;
  float sum = 0.0f;
  f32x4 o = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int64_t w = w0; w <= w1; ++w) {
    const float* z = part(w);
    const float f = fast_exp2(z[S::RT * D + lr] - ms);
    sum += z[S::RT * D + S::RT + lr] * f;
    o += *(const f32x4*)(z + lr * D + col * 4) * f;
  }
  const Nodes nd = request_nodes(a.off, b, a.N, a.max_nodes);
  const bool none = sum == 0.0f;
  const float inv = none ? 0.0f : 1.0f / sum;
  const int64_t at = (int64_t)(nd.first + r / a.G) * a.Hq + h * a.G + r % a.G;
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
  a.scale = p->scale;
  return a;
}

// The shape for `rows` packed rows a KV head: fewer rows leave more waves to
// the keys.  f(Shape{}) is called with the one taken.
template <int D, typename F>
auto with_shape(int rows, F&& f) {
  if (rows <= 16) return f(Shape<D, 1, 1, 4, 1>{});
  if (rows <= 32) return f(Shape<D, 2, 1, 4, 1>{});
  if (rows <= 64) return f(Shape<D, 2, 2, 2, 1>{});
  if (rows <= 128) return f(Shape<D, 2, 4, 1, 2>{});
  return f(Shape<D, 2, 8, 1, 2>{});
}

// Workgroups that share the unit list: two per CU of 4 waves, one of 8.
template <typename S>
constexpr int run_count() {
  return S::NT == 512 ? 256 : 512;
}

template <int DT, int D>
int launch(AttnArgs a, int rows, hipStream_t st) {
  return with_shape<D>(rows, [&](auto s) {
    using S = decltype(s);
    constexpr int runs = run_count<S>();
    hipLaunchKernelGGL((k_attn_tiles<DT, S>), dim3(runs), dim3(S::NT), 0, st, a);
    if (hipGetLastError() != hipSuccess) return SD_EHIP;
    const int mts = (rows + S::RT - 1) / S::RT;
    const dim3 grid(S::RT * (D / 4) / 256, a.c.H * mts, a.c.B);
    hipLaunchKernelGGL((k_attn_join<DT, S>), grid, dim3(256), 0, st, a, runs, mts);
    return hipGetLastError() == hipSuccess ? SD_OK : SD_EHIP;
  });
}

}  // namespace

extern "C" int sd_tree_attention_workspace_bytes(const sd_tree_attention_args_t* args, size_t* bytes) {
  if (!bytes) return SD_EINVAL;
  const int rc = check(args);
  if (rc) return rc;
  const int rows = args->max_nodes * (args->H_q / args->cache.H_kv);
  auto size = [](auto s) {
    using S = decltype(s);
    return (size_t)run_count<S>() * 2 * S::SLOT * sizeof(float);
  };
  *bytes = args->cache.D == 64 ? with_shape<64>(rows, size) : with_shape<128>(rows, size);
  return SD_OK;
}

extern "C" int sd_tree_attention(const sd_tree_attention_args_t* args, void* workspace,
                                 size_t workspace_bytes, void* out, float* out_lse,
                                 uint32_t* out_status, void* stream) {
  size_t need = 0;
  int rc = sd_tree_attention_workspace_bytes(args, &need);
  if (rc) return rc;
  if (!out || !aligned16(out)) return SD_EINVAL;
  if (!workspace || workspace_bytes < need || !aligned16(workspace)) return SD_EWORKSPACE;
  AttnArgs a = device_args(args);
  a.out = static_cast<char*>(out);
  a.lse = out_lse;
  a.status = out_status;
  hipStream_t st = static_cast<hipStream_t>(stream);
  a.part = static_cast<float*>(workspace);
  const int rows = a.max_nodes * a.G, D = args->cache.D;
  if (args->cache.dtype == SD_BF16)
    rc = D == 64 ? launch<SD_BF16, 64>(a, rows, st) : launch<SD_BF16, 128>(a, rows, st);
  else
    rc = D == 64 ? launch<SD_F16, 64>(a, rows, st) : launch<SD_F16, 128>(a, rows, st);
  if (rc) return rc;
  if (out_status) {
    hipLaunchKernelGGL(k_tree_status, dim3(a.c.B), dim3(WAVE), 0, st, a);
    if (hipGetLastError() != hipSuccess) return SD_EHIP;
  }
  return SD_OK;
}
