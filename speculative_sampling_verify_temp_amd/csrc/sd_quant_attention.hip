// Attention of a drafted tree over a paged cache held in 8 bits on gfx950.
//
// Row (node i, query head g) of a request: s_j = scale q . k_j over the visible
// slots of the cache and the nodes that i sees, o = softmax(s) . v with a running
// maximum and sum.  A slot's key is ks * code, its value vs * code, with the scales
// of its block.
//
// The rows that share a KV head (nodes x heads of its group) are packed into one
// matrix.  A workgroup is four waves, in groups: those of one share 16 MT rows, and
// each has keys of its own, 32 slots at a time straight from the cache into registers.
// Nothing is staged, so the waves meet only at the end of a run; two groups read the
// same keys at nearly the same time, one of them out of the L1.  Blocks and pages hold
// whole multiples of 16 slots, so what addresses 16 of them is in scalar registers.
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
// type, in two parts: one node often dominates its row.  They are divided by their
// fp32 sum: the rounded ones' would miss tokens whose weight is large but whose w is
// not, beside values of a far larger scale.
//
// The (request, KV head, row tile, key tile) units form one list that is cut into
// equal runs, one per workgroup; parts are joined in a fixed order.  Through a
// window only the key tiles that it (or the sinks) touches are units.
//
// A wave issues 320 instructions for 32 int8 keys of 32 rows: 96 widen codes (each once
// a wave), 80 are the softmax, 34 matrix products, 12 loads, the rest broadcasts, scalar
// work and waits; 400 for 48 rows, so rows are cheap where they share a widened key.  On
// long contexts the vector units issue 59% of the time and the matrix units work 36%, one
// after the other; the smaller cases wait besides, for loads and at the runs' ends
// (41% and 17%, 38% and 16%).  Medians of the trace, in us:
//   32 chains of 9, 28/4 heads of 128, e4m3, 500-16384 slots    85 + join 7   (bytes: 55)
//   23 trees of 21, 16/8 heads, int8, fp16, window 4099         60 + 6        (bytes: 35)
//   16 trees of 64, 28/4 heads, int8, 16384-32768 slots         440 + 11      (products: 251)
//   1 token, 14/2 heads of 64, 517 slots                        8.8, latency
// Registers: nothing is spilled by up to 64 rows a workgroup (one register by 32 fp16
// rows over e4m3 codes of 128 columns); the 96-row shape of 128 columns spills 84 to
// 103, outside the key loop but for one or two moves where slots are looked up.
// Tried without gain: three waves a SIMD (spills), four row tiles a wave (spills), two
// tiles on their way, keys widened once into LDS for both groups, the products of a tile
// under the softmax of the one before, loads that pass the caches by (98 instead of 82),
// 8 or 16 waves on one token.
#include <algorithm>
#include <type_traits>

#include "sdq_device.h"

using namespace sdv;
using namespace sdt;
using sdq::QuantCache;

namespace {

constexpr int KEYS = 32;      // keys of a wave's step
constexpr int TREE = 8;       // units that the tree of a row tile counts as
constexpr int RUNS = 512;     // workgroups that share the unit list: two a CU, a multiple of 8
constexpr float LIFT = 7.0f, LOG2E = 1.4426950408889634f;

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(1))) u32x2 global_u32x2;
typedef __attribute__((address_space(1))) s16x8 global_s16x8;

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
// nodes, row tiles, key tiles with the tree behind them, and units, for all KV
// heads, up to and including the lane's own.  Key tile t is the cache's tile t
// below `head`, t + skip from there on.  The tree, with what begins and ends a row
// tile's part, takes as long as TREE key tiles and counts as so many, the first
// of which stands for it.
struct Requests {
  int ctx, first, T, mts, nt, head, skip, incl;
  uint32_t st;
};

__device__ __forceinline__ int first_seen(int position, int window) { return window > position ? 0 : position - window + 1; }

template <int RT, int KT>
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
    r.nt = tiles - r.skip + TREE;
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
__device__ __forceinline__ Cut cut_units(const QAttnArgs& a, const Requests& r) {
  int total = lane_units(r), nt = r.nt;
  for (int b0 = WAVE; b0 < a.c.B; b0 += WAVE) {
    const Requests q = requests<RT, KT>(a, b0 + (int)threadIdx.x % WAVE);
    total += lane_units(q);
    nt = max(nt, q.nt);
  }
  return Cut{total, max((int)(((unsigned)total + RUNS - 1) / (unsigned)RUNS), (wave_max_int(nt) + 31) / 32)};
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
    for (int i = 0; i < T; ++i) {
      const int d = lane_read(s.depth, i);
      if (s.depth - d >= a.window && ctx + d >= a.sinks) s.nodes &= ~(1ull << i);
    }
  }
  return s;
}

// ---- codes as operands ----

// 4 codes as two pairs of fp16 numbers: e4m3 by value; int8 as (code + 128) 2^-24,
// which a byte with its sign turned is as the bits of an fp16 number.
template <int CODE>
__device__ __forceinline__ u32x2 widen(uint32_t u) {
  u32x2 r;
  if constexpr (CODE == SD_E4M3) {
    r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(u, 1.0f, false));
    r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(u, 1.0f, true));
  } else {
    u ^= 0x80808080u;
    r[0] = __builtin_amdgcn_perm(0u, u, 0x0C010C00u);
    r[1] = __builtin_amdgcn_perm(0u, u, 0x0C030C02u);
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

// 4 columns of 8 keys, a word a key, as operands: col[i] holds column i of the keys
// in their order.
template <int CODE>
__device__ __forceinline__ void columns(uint32_t w0, uint32_t w1, uint32_t w2, uint32_t w3, uint32_t w4, uint32_t w5,
                                        uint32_t w6, uint32_t w7, s16x8 (&col)[4]) {
  uint32_t w[8] = {w0, w1, w2, w3, w4, w5, w6, w7};
  u32x4 c[4];
  if constexpr (CODE == SD_I8) {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] ^= 0x80808080u;
  }
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    if constexpr (CODE == SD_I8) {
#pragma unroll
      for (int i = 0; i < 4; ++i) c[i][p] = __builtin_amdgcn_perm(w[2 * p + 1], w[2 * p], 0x0C040C00u + 0x00010001u * i);
    } else {
      const u32x2 a = widen<CODE>(w[2 * p]), b = widen<CODE>(w[2 * p + 1]);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        c[2 * i][p] = __builtin_amdgcn_perm(b[i], a[i], 0x05040100u);
        c[2 * i + 1][p] = __builtin_amdgcn_perm(b[i], a[i], 0x07060302u);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) col[i] = __builtin_bit_cast(s16x8, c[i]);
}

// Elements that are infinite or not a number as 0.
template <int DT>
__device__ __forceinline__ uint32_t finite_or_zero(uint32_t u, bool& odd) {
  constexpr uint32_t E = DT == SD_BF16 ? 0x7F80u : 0x7C00u;
  const bool lo = (u & E) == E, hi = (u & (E << 16)) == E << 16;
  odd = lo || hi;
  return u & (lo ? 0xFFFF0000u : 0xFFFFFFFFu) & (hi ? 0x0000FFFFu : 0xFFFFFFFFu);
}

// The kernel's arguments, read again where they are next needed: held over the loops
// they would not fit the scalar registers.
__device__ __forceinline__ const QAttnArgs& args_again() {
  uint64_t p = (uint64_t)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(p));
  return *(const QAttnArgs*)(const __attribute__((address_space(4))) QAttnArgs*)p;
}

// (fmaxf on numbers of unknown origin takes two instructions each)
__device__ __forceinline__ float max3(float x, float y, float z) {
  float r;
  asm("v_max3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(x), "v"(y), "v"(z));
  return r;
}

// MT row tiles of 16 a wave, RG groups of KG waves over the rows, each wave of a
// group with 32 keys of a unit's.  OCC waves a SIMD at least.
template <int D_, int MT_, int RG_, int KG_, int OCC_>
struct Shape {
  static constexpr int OCC = OCC_;
  static constexpr int D = D_, MT = MT_, RG = RG_, KG = KG_;
  static constexpr int WAVES = RG * KG, NT = WAVES * WAVE;
  static constexpr int RT = 16 * MT * RG;           // rows of a workgroup
  static constexpr int KT = KEYS * KG;              // keys of a unit
  static constexpr int JR = D + 4;                  // floats of a row in the join of the key groups
  static constexpr int SLOT = RT * (D + 2);         // floats of a partial result
  static_assert(KT >= SD_MAX_NODES, "the tree is one unit");
};

template <int DT, int CODE, typename S>
__global__ __launch_bounds__(S::NT, S::OCC) void k_quant_tiles(QAttnArgs a) {
  constexpr int D = S::D, MT = S::MT, RG = S::RG, KG = S::KG, RT = S::RT, KT = S::KT, JR = S::JR;
  constexpr int KS = D / 32, CB = D / 16, KW = D / 64, VW = D / 64;      // steps of a product, columns of a lane, words
  // int8 codes enter as (code + 128) 2^-24, the fp16 number whose bits they are
  // with the sign turned
  constexpr float UNIT = CODE == SD_I8 ? 0x1p24f : 1.0f, BIAS = CODE == SD_I8 ? 128.0f : 0.0f;
  // 3 row tiles' queries would not fit the registers: they lie in LDS, which the join
  // takes over
  constexpr bool QL = MT > 2;
  static_assert(!QL || RT * D / 2 <= (KG - 1) * RT * JR);
  __shared__ __align__(16) float join[(KG - 1) * RT * JR];
  __shared__ int odd_value;      // a node's value is infinite or not a number
  const int tid = threadIdx.x, lane = tid % WAVE;
  const int w = __builtin_amdgcn_readfirstlane(tid / WAVE), rg = w % RG, kg = w / RG;
  Requests rq = requests<RT, KT>(a, lane);
  int run, u0, u1;
  if (a.whole) {
    run = 0, u0 = 0, u1 = 0;
  } else {
    // Workgroups of one XCD take neighbouring runs: row tiles of one KV head
    // find each other's keys in its L2.
    const auto [total, per] = cut_units<RT, KT>(a, rq);
    run = (int)(blockIdx.x % 8) * (RUNS / 8) + (int)(blockIdx.x / 8);
    if ((int64_t)run * per >= total) return;
    u0 = run * per, u1 = u0 + min(per, total - u0);
  }

  // the request (lane f of this 64) that holds unit u0, and its units before
  int b0 = 0, f, in;
  if (a.whole) {
    const int b = blockIdx.x / (a.c.H * a.mts_max), seg = blockIdx.x % (a.c.H * a.mts_max);
    b0 = b & ~(WAVE - 1), f = b & (WAVE - 1);
    if (b0) rq = requests<RT, KT>(a, b0 + lane);
    const int mts = lane_read(rq.mts, f), nt = lane_read(rq.nt, f);
    if (seg % a.mts_max >= mts) return;
    in = (seg / a.mts_max * mts + seg % a.mts_max) * nt;
    u1 = nt;
  } else {
    int left = u0;
    while (left >= lane_units(rq)) {
      left -= lane_units(rq);
      b0 += WAVE;
      rq = requests<RT, KT>(a, b0 + lane);
    }
    f = __builtin_ctzll(__ballot(left < rq.incl));
    in = left - (f ? lane_read(rq.incl, f - 1) : 0);
  }

  while (u0 < u1) {
    const int units = lane_read(rq.incl, f) - (f ? lane_read(rq.incl, f - 1) : 0);
    const int ctx = lane_read(rq.ctx, f), first = lane_read(rq.first, f), T = lane_read(rq.T, f);
    const int mts = lane_read(rq.mts, f), nt = lane_read(rq.nt, f);
    const int head = lane_read(rq.head, f), skip = lane_read(rq.skip, f);
    const uint32_t st = (uint32_t)lane_read((int)rq.st, f);
    const int rows = T * a.G;
    const int stop = u0 + min(u1 - u0, units - in);
    while (u0 < stop) {
      const int seg = in / nt, t0 = in - seg * nt;
      const int h = seg / mts, mt = seg - h * mts;
      const int t1 = min(nt, t0 + (stop - u0));
      u0 += t1 - t0;
      in += t1 - t0;
      if (t0 > nt - TREE) continue;      // nothing but what the tree counts for
      const int cached = nt - TREE, cached_end = min(t1, cached);
      const bool tree = t1 > cached;
      const int row0 = mt * RT + rg * 16 * MT;
      const QAttnArgs& a = args_again();
      // (As if it were new: what follows from the lane alone would be kept over all
      // loops, in more registers than there are.)
      int l = lane;
      asm volatile("" : "+v"(l));
      const int n = l & 15, g4 = l >> 4;
      // offsets of a lane within 16 slots
      const uint32_t slot_stride = (uint32_t)a.c.slot_stride;
      const uint32_t kat = n * slot_stride + g4 * 16, vat = g4 * 4 * slot_stride + n * CB;

      // The wave's rows: their nodes; queries as the B operand, lane (n, g4) holding
      // of row n the columns that it loads of a key, 64 (ks / 2) + 16 g4 + 8 (ks % 2)
      // .. + 7.  bf16 queries become fp16 ones times a power of 2 that takes the row's
      // largest to 2^14: exact down to 2^-30 of it.
      int node[MT];
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const int r = row0 + 16 * m + n;
        node[m] = r < rows ? row_node(a, r) : 0;
      }
      // (loads are unconditional: rows that are not there read the first one's)
      auto queries = [&](const QAttnArgs& a, int m, s16x8 (&x)[KS]) {
        const int r = row0 + 16 * m + n;
        const int hd = h * a.G + (r < rows ? r - node[m] * a.G : 0);
        const uint64_t qp = (uint64_t)(a.q + (int64_t)(first + node[m]) * a.q_node + hd * a.q_head) + g4 * 32;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) x[ks] = *(const global_s16x8*)(qp + (ks / 2 * 64 + ks % 2 * 8) * 2);
        if (r >= rows) {
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) x[ks] = s16x8{};
        }
      };
      f32x4 o[MT][CB], norm[MT];            // norm: sums of the weights as the product sees them
      float ref[MT], sum[MT], limit[MT];    // weights are taken against ref, moved where one passes 2^limit

      const uint64_t kh = (uint64_t)(a.c.k + h * a.c.head_stride), vh = (uint64_t)(a.c.v + h * a.c.head_stride);
      auto slot_of = [&](int t) { return (t < head ? t : t + skip) * KT + kg * KEYS; };

      // What there is to know about the next 32 tiles' slots, 16 a lane: lane 2 i + s
      // has those of tile base + i, half s.
      int base;
      int at_lo, at_hi;              // byte offset in the head's keys and values
      int bytes, there;              // of the slots that are there; 256 more where their values are 0 altogether
      float key_scale, value_log, value_inv;
      const float *key_at, *value_at;
      auto look_up = [&](int t0) {
        const QAttnArgs& a = args_again();
        const int32_t* const tab = a.c.table + (b0 + f) * a.c.ld_table;
        base = t0;
        const int t = t0 + l / 2, slot = slot_of(t) + (l & 1) * 16;
        const int page = t < cached && slot < ctx ? tab[slot >> a.c.page_shift] : -1;
        const bool found = (unsigned)page < (unsigned)a.c.num_pages;
        const uint32_t p = found ? page : 0, place = found ? slot & a.c.page_mask : 0;
        const uint64_t at = p * (uint64_t)a.c.page_stride + place * (uint32_t)a.c.slot_stride;      // (a page's: below 2^30)
        at_lo = (int)(uint32_t)at, at_hi = (int)(uint32_t)(at >> 32);
        const int64_t sc = p * a.c.scale_page + h * a.c.scale_head + (place >> a.c.block_shift);
        there = found ? min(16, ctx - slot) : 0;
        bytes = there * (int)slot_stride;
        key_at = a.c.ks + sc, value_at = a.c.vs + sc;
      };
      auto look_up_scales = [&]() {
        // the key's scale with all that a product is times but the row's 1 / up, which passes
        // fp32's range beside 2^24 for queries near the largest of their type
        const float k = *key_at, v = *value_at, c = args_again().scale * LOG2E;
        const bool sound = sdq::scale_ok(k) && sdq::scale_ok(v), none = v == 0.0f;
        const float x = sound && !none ? v : sdq::MIN_SCALE;
        key_scale = sound ? k * UNIT * c : 0.0f;
        value_log = __builtin_amdgcn_logf(x);
        value_inv = __builtin_amdgcn_rcpf(x);
        there = (sound ? there : 0) | (none ? 256 : 0);
      };
      // Buffers over the 16 slots (those in use, none where they are not there): what
      // lies past them reads as zeros, without a memory access.
      struct Rows {
        uint64_t at;
        int bytes;
      };
      auto rows_of = [&](int t, int s) {
        const int i = 2 * (t - base) + s;
        return Rows{(uint64_t)(uint32_t)lane_read(at_hi, i) << 32 | (uint32_t)lane_read(at_lo, i), lane_read(bytes, i)};
      };
      auto buffer = [](uint64_t at, int bytes) {
        return __builtin_amdgcn_make_buffer_rsrc((void*)at, (short)0, bytes, 0x00020000);
      };
      u32x4 rk[2][KW];
      uint32_t rv[2][4][VW];
      auto load_k = [&](int s, const Rows& x) {
        const __amdgpu_buffer_rsrc_t rs = buffer(kh + x.at, x.bytes);
#pragma unroll
        for (int i = 0; i < KW; ++i) rk[s][i] = __builtin_amdgcn_raw_buffer_load_b128(rs, kat + i * 64, 0, 0);
      };
      auto load_v = [&](int s, const Rows& x) {
        const __amdgpu_buffer_rsrc_t rs = buffer(vh + x.at, x.bytes);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          if constexpr (VW == 2) {
            const u32x2 y = __builtin_amdgcn_raw_buffer_load_b64(rs, vat, r * slot_stride, 0);
            rv[s][r][0] = y[0], rv[s][r][1] = y[1];
          } else {
            rv[s][r][0] = __builtin_amdgcn_raw_buffer_load_b32(rs, vat, r * slot_stride, 0);
          }
        }
      };
      auto begin = [&]() {
#pragma unroll
        for (int s = 0; s < 2; ++s) load_k(s, rows_of(t0, s));
#pragma unroll
        for (int s = 0; s < 2; ++s) load_v(s, rows_of(t0, s));
      };

      // Everything that is first needed, on its way at once.
      if (t0 < cached_end) look_up(t0);
      s16x8 q[MT][KS];
#pragma unroll
      for (int m = 0; m < MT; ++m) queries(a, m, q[m]);
      if (t0 < cached_end) begin(), look_up_scales();
      // the first slot that the rows' windows show; slots below all_from are past some
      // row's
      int from[MT];
      uint64_t vis[MT];
      if (tree || a.window) {
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
      const int all_from = a.window ? first_seen(ctx + T - 1, a.window) : 0, sinks = a.sinks;
      if (tid == 0) odd_value = 0;

      s16x8* const lds_q = (s16x8*)join + rg * MT * KS * WAVE + l;
      float cr[MT], bias[MT];      // what a product is times beside the key's scale, and what it holds too much
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        float up = 1.0f;
        if constexpr (DT == SD_BF16) {
          float top = 0.0f;
#pragma unroll
          for (int ks = 0; ks < KS; ++ks)
#pragma unroll
            for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(to_f32<DT>((uint16_t)q[m][ks][i])));
          // (127 + 14) - the exponent, where the row is neither 0 nor infinite
          const int e = (int)(__float_as_uint(quad_max(top)) >> 23);
          up = e > 0 && e < 255 ? __uint_as_float((uint32_t)min(127 + 14 + 127 - e, 227) << 23) : 1.0f;
        }
        float sum = 0.0f;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float x = to_f32<DT>((uint16_t)q[m][ks][i]) * up;
            if constexpr (DT == SD_BF16) q[m][ks][i] = (short)from_f32<SD_F16>(x);
            if constexpr (CODE == SD_I8) sum += x;
          }
        if (QL && kg == m % KG) {
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) lds_q[(m * KS + ks) * WAVE] = q[m][ks];
        }
        cr[m] = 1.0f / up;
        bias[m] = CODE == SD_I8 ? quad_sum(sum) * (BIAS / UNIT) : 0.0f;
      }
      if constexpr (QL) __syncthreads();
      // Scores z, relative to ref, to weights 2^z as elements of type PT; z holds what the
      // rounding of them left.
      auto weigh = [&](auto type, f32x4 (&z)[2][MT], const float (&iv)[2], s16x8 (&p)[MT]) {
        constexpr int PT = decltype(type)::value;
        bool grown = false;
        float top[MT];
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          top[m] = max3(max3(z[0][m][0], z[0][m][1], z[0][m][2]), max3(z[0][m][3], z[1][m][0], z[1][m][1]),
                        max3(z[1][m][2], z[1][m][3], z[1][m][3]));
          // the sums are rescaled only when a maximum grows by more than 2^8: until
          // then weights up to 2^15 are as exact as those below
          grown |= top[m] > limit[m];
        }
        if (__any(grown)) {
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            const float rise = quad_max(top[m]) - LIFT;
            if (rise > limit[m] - (LIFT + 8.0f)) {      // > 0, or any rise at all where nothing was seen yet
              const float fct = limit[m] > 0.0f ? fast_exp2(-rise) : 0.0f;
              ref[m] += rise;
              limit[m] = LIFT + 8.0f;
              sum[m] *= fct;
              norm[m] *= fct;
#pragma unroll
              for (int d = 0; d < CB; ++d) o[m][d] *= fct;
#pragma unroll
              for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int r = 0; r < 4; ++r) z[s][m][r] -= rise;
            }
          }
        }
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            float y[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              y[r] = fast_exp2(z[s][m][r]);
              const uint16_t u = from_f32<PT>(y[r]);
              p[m][s * 4 + r] = (short)u;
              z[s][m][r] = y[r] - to_f32<PT>(u);
            }
            sum[m] = fmaf((y[0] + y[1]) + (y[2] + y[3]), iv[s], sum[m]);
          }
      };
      // Bit 16 s + j of on: whether the row sees key j of the 16.
      auto mask = [&](f32x4 (&z)[2][MT], int m, uint32_t on) {
        on >>= g4 * 4;
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
          for (int r = 0; r < 4; ++r) z[s][m][r] = (on >> (s * 16 + r) & 1) ? z[s][m][r] : -INFINITY;
      };

      // Nodes 32 kg .. + 31 of the tree, of the queries' type, against the wave's rows.
      auto nodes = [&]() {
        if (kg * KEYS >= T) return;
        const QAttnArgs& a = args_again();
        const float c = a.scale * LOG2E;
        // keys, and columns n CB .. of the lane's 8 nodes
        s16x8 kf[2][KS];
        uint32_t v[2][4][CB / 2];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const int j = min(kg * KEYS + s * 16 + n, T - 1);
          const uint64_t kp = (uint64_t)(a.kn + (int64_t)(first + j) * a.k_node + h * a.k_head) + g4 * 32;
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) kf[s][ks] = *(const global_s16x8*)(kp + (ks / 2 * 64 + ks % 2 * 8) * 2);
        }
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int j = min(kg * KEYS + s * 16 + g4 * 4 + r, T - 1);
            const uint64_t vp = (uint64_t)(a.vn + (int64_t)(first + j) * a.v_node + h * a.v_head) + n * CB * 2;
            if constexpr (CB == 8) {
              const u32x4 y = *(const global_u32x4*)vp;
#pragma unroll
              for (int i = 0; i < 4; ++i) v[s][r][i] = y[i];
            } else {
              const u32x2 y = *(const global_u32x2*)vp;
              v[s][r][0] = y[0], v[s][r][1] = y[1];
            }
          }
        f32x4 z[2][MT];
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          // (as they are, and read again: held over the key loop they would be spilled)
          s16x8 qf[KS];
          queries(a, m, qf);
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            z[s][m] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) z[s][m] = mfma<DT>(kf[s][ks], qf[ks], z[s][m]);
          }
        }
#pragma unroll
        for (int m = 0; m < MT; ++m) {
#pragma unroll
          for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int r = 0; r < 4; ++r) z[s][m][r] = fmaf(z[s][m][r], c, -ref[m]);
          mask(z, m, (uint32_t)(vis[m] >> (kg * KEYS)));
        }
        const float one[2] = {1.0f, 1.0f};
        s16x8 p[MT], rest[MT];
        weigh(std::integral_constant<int, DT>{}, z, one, p);
        // A node may dominate its row, and the sum that it is divided by holds its weight as
        // it is: the 8 bits of a bf16 weight would be half a step of the result.  So what
        // the rounding left enters too: weights of 16 bits, of 22 in fp16.
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int r = 0; r < 4; ++r) rest[m][s * 4 + r] = (short)from_f32<DT>(z[s][m][r]);
        // 0 x infinity in the product would reach rows that do not see this node:
        // such values are added at the end instead
        bool odd = false;
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const bool in = kg * KEYS + s * 16 + g4 * 4 + r < T;
#pragma unroll
            for (int i = 0; i < CB / 2; ++i) {
              bool strange = false;
              const uint32_t y = finite_or_zero<DT>(v[s][r][i], strange);
              v[s][r][i] = in ? y : 0u;
              odd |= in && strange;
            }
          }
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
            o[m][2 * i] = mfma<DT>(__builtin_bit_cast(s16x8, e), rest[m], o[m][2 * i]);
            o[m][2 * i + 1] = mfma<DT>(__builtin_bit_cast(s16x8, g), rest[m], o[m][2 * i + 1]);
          }
        }
        if (odd) odd_value = 1;
      };

      // The cache's key tiles of this run.  An e4m3 code that is not a number counts as
      // 0; looking for them costs a fifth, so it is done only where a result came out
      // as none (the second pass).
      for (int strict = 0;; ++strict) {
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          ref[m] = 0.0f, limit[m] = -INFINITY, sum[m] = 0.0f;
          norm[m] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int d = 0; d < CB; ++d) o[m][d] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        }
        // A tile's keys are loaded behind the products of the one before, its values
        // behind the weighted sums.  (Loads are not skipped behind the last tile: a wait
        // could not tell which are on their way.)
        for (int t = t0; t < cached_end; ++t) {
          f32x4 z[2][MT];
          if (CODE == SD_E4M3 && strict) {
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
              for (int i = 0; i < KW; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) rk[s][i][j] = numbers(rk[s][i][j]);
          }
#pragma unroll
          for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int m = 0; m < MT; ++m) z[s][m] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) {
            s16x8 kf[2];
#pragma unroll
            for (int s = 0; s < 2; ++s) {
              const u32x2 e = widen<CODE>(rk[s][ks / 2][ks % 2 * 2]), g = widen<CODE>(rk[s][ks / 2][ks % 2 * 2 + 1]);
              kf[s] = __builtin_bit_cast(s16x8, u32x4{e[0], e[1], g[0], g[1]});
            }
#pragma unroll
            for (int m = 0; m < MT; ++m) {
              const s16x8 x = QL ? lds_q[(m * KS + ks) * WAVE] : q[m][ks];
#pragma unroll
              for (int s = 0; s < 2; ++s) z[s][m] = mfma<SD_F16>(kf[s], x, z[s][m]);
            }
          }
          const int s0 = slot_of(t);
          uint32_t valid = 0, none = 0;
          float ks[2], lv[2], iv[2];
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            const int i = 2 * (t - base) + s, n16 = lane_read(there, i);
            valid |= ((1u << (n16 & 255)) - 1) << (16 * s);
            none |= (n16 >> 8) << s;
            ks[s] = lane_read(key_scale, i), lv[s] = lane_read(value_log, i), iv[s] = lane_read(value_inv, i);
          }
          if (t + 1 - base == 32) look_up(t + 1), look_up_scales();
          Rows next[2];
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            next[s] = rows_of(t + 1, s);
            load_k(s, next[s]);
          }
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int s = 0; s < 2; ++s) {
              const float k = ks[s] * cr[m], off = fmaf(-bias[m], k, lv[s] - ref[m]);
#pragma unroll
              for (int r = 0; r < 4; ++r) z[s][m][r] = fmaf(z[s][m][r], k, off);
            }
          if (valid != 0xFFFFFFFFu || (s0 < all_from && s0 + KEYS > sinks)) {
            const int sn = min(max(sinks - s0, 0), 32);
            const uint32_t first_ones = sn >= 32 ? 0xFFFFFFFFu : (1u << sn) - 1;
#pragma unroll
            for (int m = 0; m < MT; ++m) {
              const int past = min(max(from[m] - s0, 0), 32);
              const uint32_t near = past >= 32 ? 0u : 0xFFFFFFFFu << past;
              mask(z, m, valid & (near | first_ones));      // (without a window `near` is everything)
            }
          }
          s16x8 p[MT];
          weigh(std::integral_constant<int, SD_F16>{}, z, iv, p);
          if (none) {
#pragma unroll
            for (int s = 0; s < 2; ++s)
              if (none >> s & 1)
#pragma unroll
                for (int r = 0; r < 4; ++r)
#pragma unroll
                  for (int j = 0; j < VW; ++j) rv[s][r][j] = 0;
          }
          if (CODE == SD_E4M3 && strict) {
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
              for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int j = 0; j < VW; ++j) rv[s][r][j] = numbers(rv[s][r][j]);
          }
          if constexpr (CODE == SD_I8) {
            const s16x8 ones = s16x8{} + (short)0x3C00;
#pragma unroll
            for (int m = 0; m < MT; ++m) norm[m] = mfma<SD_F16>(ones, p[m], norm[m]);
          }
#pragma unroll
          for (int j = 0; j < VW; ++j) {
            s16x8 col[4];
            columns<CODE>(rv[0][0][j], rv[0][1][j], rv[0][2][j], rv[0][3][j], rv[1][0][j], rv[1][1][j], rv[1][2][j],
                          rv[1][3][j], col);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
              for (int m = 0; m < MT; ++m) o[m][4 * j + i] = mfma<SD_F16>(col[i], p[m], o[m][4 * j + i]);
          }
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            load_v(s, next[s]);
          }
        }
        if constexpr (CODE == SD_I8) {
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int d = 0; d < CB; ++d)
#pragma unroll
              for (int r = 0; r < 4; ++r) o[m][d][r] = fmaf(o[m][d][r], UNIT, -BIAS * norm[m][0]);
          break;
        } else {
          bool nan = false;
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            nan |= sum[m] != sum[m];
#pragma unroll
            for (int d = 0; d < CB; ++d)
#pragma unroll
              for (int r = 0; r < 4; ++r) nan |= o[m][d][r] != o[m][d][r];
          }
          if (strict || !__any(nan) || t0 >= cached_end) break;
          look_up(t0), begin(), look_up_scales();
        }
      }
      __syncthreads();      // odd_value; the join's LDS is free
      if (tree) nodes();
      float mx[MT];
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        sum[m] = quad_sum(sum[m]);
        mx[m] = limit[m] > 0.0f ? ref[m] : -INFINITY;
      }

      // the waves' keys: the first of a row group adds the others up
      if (kg > 0) {
        float* const z = join + ((kg - 1) * RG + rg) * 16 * MT * JR;
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
      if (kg == 0) {
        const QAttnArgs& a = args_again();
        for (int k2 = 1; k2 < KG; ++k2) {
          const float* const z = join + ((k2 - 1) * RG + rg) * 16 * MT * JR;
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
        if (tree && odd_value) {
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
        const bool whole = t0 == 0 && tree;
        float* const part = a.part + (int64_t)(run * 2 + (t0 == 0)) * S::SLOT;
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const int lr = rg * 16 * MT + 16 * m + n, r0 = mt * RT + lr;
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
    }
    in = 0;
    if (++f == WAVE && u0 < u1) {
      f = 0, b0 += WAVE;
      rq = requests<RT, KT>(a, b0 + lane);
    }
  }
}

// Rows whose key tiles went to several runs: their parts in the order of the
// runs, JN at a time.  grid (4-column groups of a row tile / 256, H * row
// tiles, B).
template <int DT, typename S>
__global__ __launch_bounds__(256) void k_quant_join(QAttnArgs a) {
  constexpr int D = S::D, RT = S::RT, KT = S::KT, GPR = D / 4, JN = 8, SLOT = S::SLOT;
  const int b = blockIdx.z, h = blockIdx.y / a.mts_max, mt = blockIdx.y % a.mts_max, l = threadIdx.x % WAVE;
  Requests rq = requests<RT, KT>(a, l);
  const int per = cut_units<RT, KT>(a, rq).per;
  int before = 0;
  for (int b0 = 0; b0 + WAVE <= b; b0 += WAVE) {
    before += lane_units(rq);
    rq = requests<RT, KT>(a, b0 + WAVE + l);
  }
  const int f = b % WAVE, nt = lane_read(rq.nt, f), mts = lane_read(rq.mts, f);
  if (mt >= mts) return;
  if (f) before += lane_read(rq.incl, f - 1);
  const int s = before + (h * mts + mt) * nt;
  const int w0 = (int)((unsigned)s / (unsigned)per), w1 = (int)((unsigned)(s + nt - TREE) / (unsigned)per);      // (the tree's)
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
  // slots that no row sees, between the sinks and what the root's window shows first, are
  // not looked at
  const int last = first_seen(ctx, a.window ? a.window : INT_MAX);
  auto hidden = [&](int slot, int shift) { return a.window && slot >= a.sinks && slot + (1 << shift) <= last; };
  for (int p = l; p < (ctx + a.c.page_mask) >> a.c.page_shift; p += WAVE) {
    if (hidden(p << a.c.page_shift, a.c.page_shift)) continue;
    const int page = tab[p];
    if ((unsigned)page >= (unsigned)a.c.num_pages) {
      bad_page = true;
      continue;
    }
    const int used = min(ctx - (p << a.c.page_shift), a.c.page_mask + 1);
    for (int h = 0; h < a.c.H; ++h)
      for (int k = 0; k << a.c.block_shift < used; ++k) {
        if (hidden((p << a.c.page_shift) + (k << a.c.block_shift), a.c.block_shift)) continue;
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

// The shape for `rows` packed rows a KV head: the fewest row tiles that hold them,
// the waves on different keys where they are few.  Above 64 rows 96 at a time take
// 1.25 times as long as 64.  us for contexts of 500-16384 slots, 28/4 heads of 128:
//   14 rows, 32 requests    55 (one token of 14/2 heads, 517 slots: 8.8), with 32-row tiles 58 (10.5)
//   28 rows, 32 requests    58, with 64-row tiles 75
//   42 rows, 24 requests    60, with 96-row tiles 77
//   84 rows, 16 requests    63, with 64-row tiles 68
//   126 rows, 16 requests   70, with 96-row tiles 89
template <int D, typename F>
auto with_shape(int rows, F&& f) {
  if (rows <= 16) return f(Shape<D, 1, 1, 4, 2>{});
  if (rows <= 32) return f(Shape<D, 2, 1, 4, 2>{});
  if ((rows + 95) / 96 * 5 > (rows + 63) / 64 * 4) return f(Shape<D, 2, 2, 2, 2>{});
  return f(Shape<D, 3, 2, 2, 2>{});
}

// Where there are no more key tiles than this, splitting them and joining the
// parts in a second launch costs more than it saves.  One token, tiles of 128 slots:
// 1000 slots 9.9 us whole and 10.4 split, 2000 slots 14.4 and 13.3; 64 requests of 4
// nodes and 500-900 slots 19 and 27.
constexpr int WHOLE_TILES = 11;

// How a call is cut up.
struct Plan {
  int mts_max;                // row tiles of a KV head
  int64_t segments, tiles;    // (request, KV head, row tile)s, and key tiles of one
  bool fits, whole;
};

template <typename S>
Plan plan(const sd_quant_attention_args_t* p) {
  const sd_quant_cache_t& c = p->cache;
  const int rows = p->max_nodes * (p->H_q / c.H_kv);
  Plan r;
  r.mts_max = (rows + S::RT - 1) / S::RT;
  r.segments = (int64_t)c.B * c.H_kv * r.mts_max;
  r.tiles = ((int64_t)c.max_pages * c.page_size + S::KT - 1) / S::KT + TREE;
  if (p->window)
    r.tiles = std::min(r.tiles, ((int64_t)p->sinks + S::KT - 1) / S::KT + ((int64_t)p->window + S::KT - 1) / S::KT + 1 + TREE);
  r.fits = r.segments <= 0x7FFFFFFF / r.tiles;      // units are counted in 32 bits
  // (and a grid dimension holds less than 2^32 threads)
  r.whole = r.tiles - TREE <= WHOLE_TILES && r.segments * S::NT <= UINT32_MAX;
  return r;
}

template <int DT, int CODE, int D>
int launch(QAttnArgs a, const sd_quant_attention_args_t* p, hipStream_t st) {
  return with_shape<D>(a.max_nodes * a.G, [&](auto s) {
    using S = decltype(s);
    const Plan r = plan<S>(p);
    a.mts_max = r.mts_max;
    a.whole = r.whole;
    hipLaunchKernelGGL((k_quant_tiles<DT, CODE, S>), dim3(a.whole ? (unsigned)r.segments : (unsigned)RUNS),
                       dim3(S::NT), 0, st, a);
    if (hipGetLastError() != hipSuccess) return SD_EHIP;
    if (a.whole) return SD_OK;
    const dim3 grid((S::RT * (D / 4) + 255) / 256, a.c.H * a.mts_max, a.c.B);
    hipLaunchKernelGGL((k_quant_join<DT, S>), grid, dim3(256), 0, st, a);
    return hipGetLastError() == hipSuccess ? SD_OK : SD_EHIP;
  });
}

}  // namespace

extern "C" int sd_quant_attention_workspace_bytes(const sd_quant_attention_args_t* args, size_t* bytes) {
  if (!bytes) return SD_EINVAL;
  const int rc = check(args);
  if (rc) return rc;
  const int rows = args->max_nodes * (args->H_q / args->cache.H_kv);
  auto size = [&](auto s) {
    using S = decltype(s);
    const Plan p = plan<S>(args);
    *bytes = p.whole ? 0 : (size_t)RUNS * 2 * S::SLOT * sizeof(float);
    return p.fits ? SD_OK : SD_EUNSUPPORTED;
  };
  return args->cache.D == 64 ? with_shape<64>(rows, size) : with_shape<128>(rows, size);
}

extern "C" int sd_quant_attention(const sd_quant_attention_args_t* args, void* workspace,
                                  size_t workspace_bytes, void* out, float* out_lse,
                                  uint32_t* out_status, void* stream) {
  size_t need = 0;
  int rc = sd_quant_attention_workspace_bytes(args, &need);
  if (rc) return rc;
  if (!out || !aligned16(out)) return SD_EINVAL;
  const sd_quant_cache_t& c = args->cache;
  const void* const outs[] = {out, out_lse, out_status};
  const void* const ins[] = {args->k_new, args->v_new, c.k, c.v, c.k_scale, c.v_scale, c.page_table, c.context_lens,
                             args->node_offsets, args->parents, need ? workspace : nullptr};
  for (int i = 0; i < 3; ++i) {
    if (!outs[i]) continue;
    for (const void* in : ins)
      if (outs[i] == in) return SD_EINVAL;
    if (i && outs[i] == args->q) return SD_EINVAL;
    for (int j = 0; j < i; ++j)
      if (outs[i] == outs[j]) return SD_EINVAL;
  }
  // a query row is read by the workgroups of its own result alone, before they
  // write it or before the join does
  if (out == args->q && ((args->H_q > 1 && args->q_head != args->cache.D) ||
                         (args->N > 1 && args->q_node != (int64_t)args->H_q * args->cache.D)))
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
