// Losses through the LM head, cross entropy and distillation from a teacher's
// top logits, with their gradients.
//
// Both have a target that is sparse over the vocabulary (one id with weight 1,
// or `top` ids with weights q), so they share every product:
//   forward   l = s r h W^T, per row the log of the sum of exponentials and
//             the few l at the target's ids; no l leaves the product's tile
//             but those (few tiles apart, whose K is split: k_head_part)
//   backward  per piece of the vocabulary l again, G = s r g exp(l - lse) in
//             bf16, its entries at the target's ids replaced by
//             s r g (p - q); then u += G W (dL/dz r) and d_W = G^T h.  One such
//             entry is as large as the rest of its row together, so its bf16
//             rounding (up to 2^-8) would show in the gradients as much as the
//             gradients' own.  What that rounding takes off is therefore added
//             to u (times the id's row of W) and to d_W (times the row of h),
//             both before they are rounded: the entries and the rest of G
//             cancel in a trained head's d_W, so nothing may be rounded between
// with r = 1 / sqrt(mean h^2 + eps), s the logit scale and g = dL/dloss.
// r s multiplies the fp32 accumulators: the products' operands are the bf16
// inputs themselves, and G is the one value that is rounded on the way.
// Above 256 tokens those that do not count are left out of the products: rows[]
// lists the others, which are gathered.
#include "common.h"
#include "kernels.h"

#include <type_traits>

namespace moe {

namespace {

constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.693147180559945309417f;

MOE_DEV float hl_sum64(float v) {
#pragma unroll
  for (int x = 32; x > 0; x >>= 1) v += shfl_xor(v, x);
  return v;
}
MOE_DEV float hl_max64(float v) {
#pragma unroll
  for (int x = 32; x > 0; x >>= 1) v = fmaxf(v, shfl_xor(v, x));
  return v;
}
MOE_DEV float hl_exp2(float v) { return __builtin_amdgcn_exp2f(v); }  // one instruction, 1 ulp
// Beyond this the rounding of y = l log2 e, up to 2^-24 |y|, is no longer small
// as an exponent (at 2^31 it is past fp32's): exponents are formed another way.
constexpr float kFarLogit = 1.0e6f;
MOE_DEV float hl_not_above_0(float v) { return v > 0.0f ? 0.0f : v; }  // NaN stays
MOE_DEV float hl_not_below_0(float v) { return v < 0.0f ? 0.0f : v; }
// Joins two (maximum, sum of 2^(y - maximum)) pairs; an empty one has sum 0.
MOE_DEV void hl_merge(float& m, float& s, float m2, float s2) {
  if (s2 == 0.0f) return;
  if (s == 0.0f) {
    m = m2;
    s = s2;
    return;
  }
  const float M = fmaxf(m, m2);
  float d, d2;
  {
#pragma clang fp contract(off)  // with a product behind m or m2 its rounding would stay in the difference
    d = m - M;
    d2 = m2 - M;
  }
  s = s * hl_exp2(d) + s2 * hl_exp2(d2);
  m = M;
}

}  // namespace

// G W (dL/dz) has few tiles for few rows or a narrow h, and a long K: its K is
// split over `splits` workgroups per tile, which add to separate slabs of u
// (added up in order by k_head_dh, so results do not depend on the order of
// execution).  The number follows from the rows that count, when they are
// known: the least
//   rounds of workgroups x (K steps each x step + over) + splits x (writing and
//   reading a slab at 5 MB per microsecond, and an eighth of one in k_head_dh)
// in microseconds, step and over being the tile's (HeadShape).
constexpr int HEAD_SPLITS = 64;  // one per lane of the wave that chooses
struct HeadSplit {
  int H, K, bm, bn;  // of the first piece, so every piece adds to the same slabs
  int slots, most;   // workgroups that run at a time; most workgroups
  float step, over;  // microseconds per K step, and per tile besides
};
MOE_DEV int head_splits(const HeadSplit& q, int n, int lane) {
  const int tiles = ((n + q.bm - 1) / q.bm) * ((q.H + q.bn - 1) / q.bn), steps = (q.K + 63) / 64, s = lane + 1;
  float cost = INFINITY;
  if (s == 1 || (tiles * s <= q.most && s <= steps))
    cost = (float)((tiles * s + q.slots - 1) / q.slots) * ((float)((steps + s - 1) / s) * q.step + q.over) +
           (float)s * ((float)n * (float)q.H * (8.0f / 5e6f) + 0.125f);
  const float least = -hl_max64(-cost);
  return __ffsll(__ballot(cost == least));  // the first of them
}

// ---- which tokens count -----------------------------------------------------

// Log of a teacher's probability before its normalisation, x - m times the
// scale: the difference first, and held above the lowest fp32 values, so that
// logits of -3.4e38 (a mask's) stay slots that are there, at probability 0 or,
// where all of a token's are, equal.
MOE_DEV float hl_teacher(float x, float m, float tscale) {
  const float y = (x - m) * tscale;
  return y < -3.0e38f ? -3.0e38f : y;  // NaN stays
}

// One wave, one token's slots: the log of the teacher's probabilities of slots
// lane, lane + 64, ... (-infinity for those that are not there); whether any is.
MOE_DEV bool head_teacher(const int32_t* __restrict__ ids, const float* __restrict__ tlogits, int V, int top,
                          float tscale, int lane, float (&lq)[4]) {
  float m = -INFINITY;
  bool any = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int j = i * 64 + lane;
    lq[i] = -INFINITY;
    if (j < top) {
      const int id = ids[j];
      if (id >= 0 && id < V) lq[i] = tlogits[j];
    }
    const bool have = !(lq[i] == -INFINITY);
    any |= have;
    if (have) m = fmaxf(m, lq[i]);
  }
  m = hl_max64(m);
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (!(lq[i] == -INFINITY)) {
      lq[i] = hl_teacher(lq[i], m, tscale);
      s += expf(lq[i]);
    }
  const float ls = logf(hl_sum64(s));
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (!(lq[i] == -INFINITY)) lq[i] -= ls;
  return __any(any);
}

// Distillation, more than HEAD_SAME tokens, one wave each: lq and flag.
__global__ __launch_bounds__(256) void k_head_teacher(const int32_t* __restrict__ ids, const float* __restrict__ tlogits,
                                                      int T, int V, int top, float tscale, float* __restrict__ lq,
                                                      uint8_t* __restrict__ flag) {
  const int t = blockIdx.x * 4 + (threadIdx.x >> 6), lane = threadIdx.x & 63;
  if (t >= T) return;
  float q[4];
  const bool counts =
      head_teacher(ids + (int64_t)t * top, tlogits + (int64_t)t * top, V, top, tscale, lane, q);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i * 64 + lane < top) lq[(int64_t)t * top + i * 64 + lane] = q[i];
  if (lane == 0) flag[t] = counts;
}

// The list of tokens that count, in order, and each token's place in it (-1).
// flag null: a token counts if its id is in [0, V).  One block, 8192 tokens at a
// time: a wave takes 512 in steps of 64 (one per lane).
__global__ __launch_bounds__(1024) void k_head_compact(const uint8_t* __restrict__ flag, const int32_t* __restrict__ ids,
                                                       int T, int V, HeadSplit q, int32_t* __restrict__ rows,
                                                       int32_t* __restrict__ cidx, int32_t* __restrict__ count) {
  __shared__ int wsum[16];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int base = 0;
  for (int t0 = 0; t0 < T; t0 += 8192) {
    const int t = t0 + wave * 512 + lane;
    int x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int u = min(t + i * 64, T - 1);
      x[i] = flag != nullptr ? (int)flag[u] - 1 : ids[u];  // counts: in [0, V)
    }
    uint64_t on[8];
    int k = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      on[i] = __ballot(t + i * 64 < T && x[i] >= 0 && x[i] < V);
      k += __popcll(on[i]);
    }
    __syncthreads();  // the previous round's sums have been read
    if (lane == 0) wsum[wave] = k;
    __syncthreads();
    int at = base;
#pragma unroll
    for (int w = 0; w < 16; ++w) {
      const int v = wsum[w];
      if (w < wave) at += v;
      base += v;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int u = t + i * 64, c = at + __popcll(on[i] & ((1ull << lane) - 1));
      const bool o = (on[i] >> lane) & 1;
      if (u < T) cidx[u] = o ? c : -1;
      if (o) rows[c] = u;
      at += __popcll(on[i]);
    }
  }
  if (wave == 0) {
    const int splits = head_splits(q, base, lane);
    if (lane == 0) {
      count[0] = base;
      count[1] = splits;
    }
  }
}

// What a product's epilogue needs of its row c (16 bytes, one load).
struct HeadRow {
  float f2;   // logit_scale / rms * log2 e
  float f;    // forward: logit_scale / rms; backward: that times dL/dloss
  float l2;   // backward: lse log2 e
  int tgt;    // cross entropy: the target's id
};

// How the rows that count are found: from k_head_compact's list; by every block
// itself among at most 1024 flags (block 0 writes the lists, no launch is spent
// on them); or, up to HEAD_SAME tokens, not at all: row c is token c, rows of
// tokens that do not count are zeros, and the teacher's probabilities are
// formed here too.  Up to there one tile row holds all tokens, whatever number of
// them counts, so leaving some out spares little.  Zeros against gathered, us: 250 x
// 2048 x 32000 with 16 slots forward 41.7 / 44.6 (half of them count 39.6 / 42.3),
// gradient 86 / 90 (80 / 82); gradient of 250 x 7168 x 32000 244 / 245, half 239 /
// 229, a fifth 235 / 217.
enum { HR_LIST, HR_FEW, HR_SAME };
constexpr int HEAD_FEW = 1024, HEAD_SAME = 256;

struct HeadRowsArgs {
  const uint16_t* h;
  int64_t h_stride;
  int T, H, Hp, V, top, bm;
  float eps, scale, tscale;
  const int32_t* ids;
  const float* tlogits;  // null: cross entropy
  const uint8_t* flag;   // distillation, HR_LIST and HR_FEW
  const float* loss;     // backward (cross entropy)
  const float* lse;      // backward
  const float* dloss;    // backward
  HeadSplit split;
  int32_t* rows;
  int32_t* cidx;
  int32_t* count;        // rows, splits of G W
  uint16_t* hc;
  float* r;
  HeadRow* info;
  int32_t* eid;          // backward, cross entropy: the row's target (-1: none) and G there
  float* ev;
  float* lq;
};

// The rows that count, one after the other, as the products read them: hc
// [..][Hp] with zeros in columns H..Hp (the K of the products goes in steps of
// 64) and in the rows up to the next multiple of a tile's bm rows, with
// r[c] = 1/rms of row c and its HeadRow (zeros behind the last row).  One block
// per row.  A copy that costs the products nothing to mask: 38 us for 8192 x 7168
// (235 MB, 6.2 TB/s), 4-6 us up to 1024 rows.
template <int MODE>
__global__ __launch_bounds__(256) void k_head_gather(HeadRowsArgs p) {
  __shared__ float part[4], part2[4];
  __shared__ int wsum[4], found;
  const int c = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int n, t = c;
  bool live;  // row c holds a token that counts
  if (MODE == HR_SAME) {
    n = p.T;
    if (p.tlogits == nullptr) {
      const int y = c < n ? p.ids[c] : -1;
      live = y >= 0 && y < p.V;
    } else {
      // thread j has slot j (top <= 256)
      float x = -INFINITY;
      if (c < n && tid < p.top) {
        const int id = p.ids[(int64_t)c * p.top + tid];
        if (id >= 0 && id < p.V) x = p.tlogits[(int64_t)c * p.top + tid];
      }
      const bool have = !(x == -INFINITY);
      const float m4 = hl_max64(have ? x : -INFINITY);
      const bool any4 = __any(have);
      if (lane == 0) {
        part[wave] = m4;
        wsum[wave] = any4;
      }
      __syncthreads();
      const float m = fmaxf(fmaxf(part[0], part[1]), fmaxf(part[2], part[3]));
      live = wsum[0] | wsum[1] | wsum[2] | wsum[3];
      x = hl_teacher(x, m, p.tscale);  // not used where there is no slot
      const float s4 = hl_sum64(have ? expf(x) : 0.0f);
      if (lane == 0) part2[wave] = s4;
      __syncthreads();
      const float ls = logf((part2[0] + part2[1]) + (part2[2] + part2[3]));
      if (c < n && tid < p.top) p.lq[(int64_t)c * p.top + tid] = have ? x - ls : -INFINITY;
    }
    if (c < n && tid == 0) {
      p.rows[c] = c;
      p.cidx[c] = live ? c : -1;
    }
  } else if (MODE == HR_FEW) {
    // thread i looks at tokens 4 i .. 4 i + 3
    int on[4], k = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int u = tid * 4 + i;
      on[i] = u < p.T && (p.flag != nullptr ? p.flag[u] != 0 : p.ids[u] >= 0 && p.ids[u] < p.V);
      k += on[i];
    }
    int before = k;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int v = __shfl_up(before, d, 64);
      if (lane >= d) before += v;
    }
    if (lane == 63) wsum[wave] = before;
    __syncthreads();
    before -= k;
#pragma unroll
    for (int w = 0; w < 4; ++w)
      if (w < wave) before += wsum[w];
    n = wsum[0] + wsum[1] + wsum[2] + wsum[3];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int u = tid * 4 + i;
      if (on[i] && before == c) found = u;
      if (c == 0 && u < p.T) {
        p.cidx[u] = on[i] ? before : -1;
        if (on[i]) p.rows[before] = u;
      }
      before += on[i];
    }
    __syncthreads();
    live = c < n;
    if (live) t = found;
  } else {
    n = p.count[0];
    live = c < n;
    if (live) t = p.rows[c];
  }
  if (MODE != HR_LIST && c == 0 && wave == 0) {
    const int splits = head_splits(p.split, n, lane);
    if (lane == 0) {
      p.count[0] = n;
      p.count[1] = splits;
    }
  }
  if (c >= (n + p.bm - 1) / p.bm * p.bm) return;
  uint16_t* o = p.hc + (int64_t)c * p.Hp;
  const uint16_t* row = p.h + (int64_t)t * p.h_stride;
  float ss = 0.0f;
  for (int i = tid; i < p.Hp / 8; i += 256) {
    u32x4 q = {0, 0, 0, 0};
    if (live && i < p.H / 8) q = *reinterpret_cast<const u32x4*>(row + i * 8);
    *reinterpret_cast<u32x4*>(o + i * 8) = q;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float a = bf16_bits_to_f32(q[j] & 0xFFFFu), b = bf16_bits_to_f32(q[j] >> 16);
      ss = fmaf(a, a, ss);
      ss = fmaf(b, b, ss);
    }
  }
  if (!live) {
    if (tid == 0) {
      p.info[c] = HeadRow{0.0f, 0.0f, 0.0f, -1};
      if (p.loss != nullptr && c < n) p.eid[c] = -1;
    }
    return;
  }
  ss = hl_sum64(ss);
  __syncthreads();  // part has been read
  if (lane == 0) part[wave] = ss;
  __syncthreads();
  if (tid == 0) {
    const float rr =
        p.eps > 0.0f ? 1.0f / sqrtf(((part[0] + part[1]) + (part[2] + part[3])) / (float)p.H + p.eps) : 1.0f;
    const float f = p.scale * rr;
    p.r[c] = rr;
    HeadRow w = {f * kLog2e, f, 0.0f, p.tlogits == nullptr ? p.ids[t] : -1};
    if (p.dloss != nullptr) {
      w.f = f * p.dloss[t];
      w.l2 = p.lse[t] * kLog2e;
      if (p.loss != nullptr) {
        p.eid[c] = w.tgt;
        p.ev[c] = w.f * expm1f(-p.loss[t]);  // p - 1 = exp(-loss) - 1
      }
    }
    p.info[c] = w;
  }
}

// ---- the products -----------------------------------------------------------
//
// C[m][n] = sum_k A[m][k] B[n][k] on 16x16x32 bf16 MFMAs, tiles of BM x BN by 8
// waves, K in steps of 64.  Each operand lies in memory either with K
// contiguous (rows m) or with m contiguous (rows k): the head's forward
// product, G W and G^T h need both kinds, and no transposed copy is made.
//
// Stages of 64 K go to an LDS ring by DMA; a wave reads its fragments of the
// next 32 K into registers while the MFMAs of the current 32 run (two MFMA
// rows per LDS read), so that only the barrier of every 64 K shows.
// K-contiguous rows (128 bytes per stage) keep 16-byte part p at slot
// p ^ ((row >> 1) & 7): the 16 rows of a fragment cover all banks once.
// m-contiguous rows (2 BM bytes) are read by the transposing 8-byte LDS read,
// 4 rows x 32 bytes per 16 lanes; 32-byte piece c of row k lies at
// c ^ (k & 3 | (k >> 1 & 4)), so the 8 rows that 32 lanes touch at once cover
// all banks.
//
// The accumulators are formed transposed (B's fragment first): a lane then
// holds 4 consecutive columns of one row.
//
// Large products are bound by the MFMAs at the clock that the power limit leaves:
// 8192 x 7168 x 32000 takes 2.52-2.62 ms for h W^T with G's epilogue and 5.34-5.66
// for both others, 1.3-1.5 PFLOP/s with the matrix cores busy 0.81 of the cycles.
// 256 x 256 tiles read each operand least, and eight waves of 128 x 64 of them
// hold two K halves of fragments beside 128 accumulators (four waves of 128 x 128:
// 8.9 against 8.5 ms for the whole gradient).  Few rows are bound by the stream
// of W: 64 rows of 7168 x 32000 79-85 us, 5.4-5.8 TB/s; one row of 2048 x 32000
// 33 us, 4.0 TB/s from memory (22 where the last-level cache holds W).

typedef short s16x4 __attribute__((ext_vector_type(4)));

// An operand tile: p its first element, ld bytes between rows, `mn` valid rows
// (K contiguous) or columns from there, `k` valid K.  Loads past either are
// redirected to the last valid piece: rows and columns past the end belong to
// outputs that are not kept, and past the end of K the other operand holds
// zeros.
struct HeadSrc {
  const char* p;
  uint32_t ld;
  int mn;
  int k;
  const int32_t* list = nullptr;  // rows taken through a list (HeadOperand's ROWS)
  int zero = 0;                   // a row of zeros
};

// global_load_lds with a uniform base and a 32-bit lane offset.
MOE_DEV void hl_dma(const char* base, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(lds), "v"(off), "s"(base) : "memory");
}

// The same with an address of each lane's own.
MOE_DEV void hl_dma_at(const char* addr, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(lds), "v"(addr) : "memory");
}

// One operand of a tile: R rows (or columns) by 64 K per stage.  ROWS (m
// contiguous): K row k is row list[k] of the matrix at p, a row of zeros past k.
template <int R, bool KM, int NW, bool ROWS = false>
struct HeadOperand {
  static constexpr int BYTES = R * 128;
  static constexpr int ND = R / 8 / NW;  // DMAs per wave and stage
  static constexpr int RB = KM ? R * 2 : 128;
  static constexpr int LPR = RB / 16;     // lanes per row of a DMA
  static_assert(R % (8 * NW) == 0 && (!KM || R >= 128) && (!ROWS || (KM && LPR == 32)), "tile");
  HeadSrc s;
  uint32_t off[ND];
  MOE_DEV static int row_of(int wave, int lane, int j) { return (wave * ND + j) * (64 / LPR) + lane / LPR; }
  MOE_DEV void init(const HeadSrc& src, int wave, int lane) {
    s = src;
#pragma unroll
    for (int j = 0; j < ND; ++j) {
      const int row = row_of(wave, lane, j), q = lane % LPR;
      if (KM) {
        const int f = (row & 3) | ((row >> 1) & 4);
        const int col = min((((q >> 1) ^ f) << 4) + (q & 1) * 8, s.mn - 8);
        off[j] = (ROWS ? 0 : (uint32_t)row * s.ld) + col * 2;
      } else {
        off[j] = (uint32_t)min(row, s.mn - 1) * s.ld + ((q ^ ((row >> 1) & 7)) << 4);
      }
    }
  }
  // DMA j of stage kt into the stage at LDS address lds.  LAST: the stage may
  // reach past the end of K.
  template <bool LAST>
  MOE_DEV void issue(int j, int kt, uint32_t lds, int wave, int lane) const {
    if constexpr (ROWS) {
      // the two K rows of this DMA, by scalar loads (the list has 64 more
      // entries behind it, whatever they hold)
      typedef const __attribute__((address_space(4))) int32_t* const_i32;
      const int k0 = __builtin_amdgcn_readfirstlane(kt * 64 + (wave * ND + j) * 2);
      const const_i32 l = (const_i32)(uintptr_t)(s.list + k0);
      const int a = k0 < s.k ? l[0] : s.zero, b = k0 + 1 < s.k ? l[1] : s.zero;
      hl_dma_at(s.p + (int64_t)(lane < 32 ? a : b) * s.ld + off[j],
                __builtin_amdgcn_readfirstlane(lds + (wave * ND + j) * 1024));
      return;
    }
    uint32_t o = off[j];
    const int over = kt * 64 + 64 - s.k;  // K past the end (uniform)
    if (LAST && over > 0) {
      const int row = row_of(wave, lane, j);
      if (KM) {
        const int last = 63 - over;
        if (row > last) o -= (uint32_t)(row - last) * s.ld;
      } else {
        const int k = ((lane % LPR) ^ ((row >> 1) & 7)) * 8, last = 56 - over;
        if (k > last) o -= (k - last) * 2;
      }
    }
    hl_dma(s.p + (KM ? (int64_t)kt * 64 * s.ld : (int64_t)kt * 128), o,
           __builtin_amdgcn_readfirstlane(lds + (wave * ND + j) * 1024));
  }
  // Fragment of rows r0 + 16 i .. (r0 a multiple of 16 i's range), K half s.
  // base: lane_base(r0, lane).
  MOE_DEV static int lane_base(int r0, int lane) {
    const int ln = lane & 15, lg = lane >> 4;
    if (KM) {
      const int f = (ln >> 2) | ((lg & 1) << 2);
      return (8 * lg + (ln >> 2)) * RB + (((r0 >> 4) ^ f) << 5) + (ln & 3) * 8;
    }
    return (r0 + ln) * 128 + ((lg ^ (ln >> 1)) << 4);
  }
  MOE_DEV static bf16x8 frag(const uint8_t* st, int base, int i, int half) {
    if (KM) {
      const uint8_t* a = st + (base ^ (i << 5)) + half * 32 * RB;
      typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
      const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)a);
      const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(a + 4 * RB));
      return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    }
    return *reinterpret_cast<const bf16x8*>(st + (base ^ (half << 6)) + i * 2048);
  }
};

// The tile of a workgroup: BM x BN, WM x WN waves, S stages; WPS waves per
// SIMD in flight (2 per resident workgroup).
template <int BM_, int BN_, int WM_, int WN_, int S_, int WPS_>
struct HeadTile {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, S = S_, WPS = WPS_;
  static constexpr int MI = BM / WM / 16, NJ = BN / WN / 16;  // 16-row and 16-column pieces per wave
  static constexpr int STAGE = (BM + BN) * 128;
  // Tiles with two stages keep a fifth half-stage buffer: A and B pieces of the
  // stages take turns in a ring of five, and A's of the stage after the next are
  // requested half a step before B's.
  static constexpr bool FIVE = S == 2;
  static_assert(!FIVE || BM == BN, "buffers of one size");
  static constexpr int SMEM = FIVE ? 5 * BM * 128 : S * STAGE;
  static constexpr int NW = WM * WN, NT = NW * 64;
  // what a last round of these tiles may be done with (head_tile_tail)
  using Half = std::conditional_t<FIVE, HeadTile<BM_ / 2, BN_, WM_, WN_, 3, WPS_>, HeadTile>;
};

// SQ (four threads per row of A): also sums into *ss the squares of the 16
// values that thread t sees per stage of row t / 4 of A.  ADD: adds to acc, and
// B's rows come through a list.
template <class C, bool KMA, bool KMB, bool SQ = false, bool ADD = false>
MOE_DEV void head_mm(const HeadSrc& sa, const HeadSrc& sb, int KT, f32x4 (&acc)[C::MI][C::NJ], uint8_t* smem,
                     float* ss = nullptr) {
  static_assert(!SQ || (!KMA && C::NT == 4 * C::BM && !C::FIVE), "rows per thread");
  using OA = HeadOperand<C::BM, KMA, C::NW>;
  using OB = HeadOperand<C::BN, KMB, C::NW, ADD>;
  constexpr int S = C::S, MI = C::MI, NJ = C::NJ, NPER = OA::ND + OB::ND;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  OA oa;
  OB ob;
  oa.init(sa, wave, lane);
  ob.init(sb, wave, lane);
  const uint32_t smem0 = lds_u32(smem);
  // a stage's place: its slot of the ring, or (FIVE) the buffer of its A piece,
  // B's piece in the next one
  auto off_a = [](int slot) { return C::FIVE ? slot * OA::BYTES : slot * C::STAGE; };
  auto off_b = [](int slot) {
    return C::FIVE ? (slot == 4 ? 0 : slot + 1) * OA::BYTES : slot * C::STAGE + OA::BYTES;
  };
  auto next = [](int slot) { return C::FIVE ? (slot >= 3 ? slot - 3 : slot + 2) : slot + 1 == S ? 0 : slot + 1; };
  auto issue1 = [&](auto last, int j, int kt, int slot) {
    constexpr bool LAST = decltype(last)::value;
    if (j < OA::ND) oa.template issue<LAST>(j, kt, smem0 + off_a(slot), wave, lane);
    else ob.template issue<LAST>(j - OA::ND, kt, smem0 + off_b(slot), wave, lane);
  };
  const int ba = OA::lane_base((wave / C::WN) * MI * 16, lane);
  const int bb = OB::lane_base((wave % C::WN) * NJ * 16, lane);
  if (!ADD)
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j) acc[i][j] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int s = 0; s < S; ++s)
    if (s < KT)
#pragma unroll
      for (int j = 0; j < NPER; ++j) issue1(std::true_type(), j, s, C::FIVE ? 2 * s : s);
  wait_stages<NPER>(min(S, KT) - 1);
  lds_barrier();
  // fragments of the current and of the next 32 K: B's, then A's
  bf16x8 f[2][NJ + MI];
  auto read = [&](int x, int slot, int i, int half) {
    f[x][i] = i < NJ ? OB::frag(smem + off_b(slot), bb, i, half) : OA::frag(smem + off_a(slot), ba, i - NJ, half);
  };
#pragma unroll
  for (int i = 0; i < NJ + MI; ++i) read(0, 0, i, 0);
  // The MFMAs of fragments f[x], with the reads of the next fragments into
  // f[1 - x] spread over the first three quarters of them (so that they have
  // arrived when they are wanted) and the parts dma(i) of a stage in between: a
  // wave's MFMAs then never wait behind a run of other instructions.
  constexpr int NR = NJ + MI, RM = MI * NJ * 3 / 4;  // fragments, MFMAs that lead their reads
  auto phase = [&](auto x, int rslot, int half, auto dma) {
    constexpr int X = decltype(x)::value;
#pragma unroll
    for (int m = 0; m < MI * NJ; ++m) {
      const int i = m / NJ, j = m % NJ;
      acc[i][j] = mfma_bf16_16x16x32(f[X][j], f[X][NJ + i], acc[i][j]);
      if (m < RM) {
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int r = m * NR / RM; r < (m + 1) * NR / RM; ++r) read(1 - X, rslot, r, half);
        __builtin_amdgcn_sched_barrier(0);
      }
      if (m % NJ == NJ / 2) {
        __builtin_amdgcn_sched_barrier(0);
        dma(i);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  };
  using X0 = std::integral_constant<int, 0>;
  using X1 = std::integral_constant<int, 1>;
  int slot = 0;
  float ss_low = 0.0f;
  // ISSUE: 0 no stage left to issue, 1 stage kt + S, 2 the same and it is the last
  auto step = [&](auto issue, int kt) {
    constexpr int ISSUE = decltype(issue)::value;
    const int nslot = next(slot);
    using Last = std::integral_constant<bool, ISSUE == 2>;
    if (SQ) {
      // a stage's 16 squares first, then one compensated addition: a plain sum
      // over the whole row would cost 1/rms, and so every logit, a few 1e-7
      const int row = threadIdx.x >> 2, part = (threadIdx.x & 3) * 2;
      float x[8];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const u32x4 q = *reinterpret_cast<const u32x4*>(smem + off_a(slot) + row * 128 +
                                                        (((part + j) ^ ((row >> 1) & 7)) << 4));
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float a = bf16_bits_to_f32(q[e] & 0xFFFFu), b = bf16_bits_to_f32(q[e] >> 16);
          x[j * 4 + e] = fmaf(a, a, b * b);
        }
      }
      const float y = (((x[0] + x[1]) + (x[2] + x[3])) + ((x[4] + x[5]) + (x[6] + x[7]))) - ss_low;
      const float sum = *ss + y;
      ss_low = (sum - *ss) - y;
      *ss = sum;
    }
    phase(X0(), slot, 1, [&](int i) {
      if (C::FIVE && ISSUE) {
#pragma unroll
        for (int j = i * OA::ND / MI; j < (i + 1) * OA::ND / MI; ++j) issue1(Last(), j, kt + S, next(nslot));
      }
    });
    // after the barrier every wave holds the rest of this stage in registers
    // (its place is free), and the next stage has landed
    if (ISSUE) wait_vmcnt_clamped<C::FIVE ? OA::ND : (S - 2) * NPER>();
    else if (kt + 1 < KT) wait_stages<NPER>(KT - 2 - kt);
    lds_barrier();
    phase(X1(), nslot, 0, [&](int i) {
      if (C::FIVE && ISSUE) {
#pragma unroll
        for (int j = i * 2 * OB::ND / MI; j < (i + 1) * 2 * OB::ND / MI && j < OB::ND; ++j)
          issue1(Last(), OA::ND + j, kt + S, next(nslot));
      } else if (ISSUE) {
#pragma unroll
        for (int j = i * NPER / MI; j < (i + 1) * NPER / MI; ++j) issue1(Last(), j, kt + S, slot);
      }
    });
    slot = nslot;
  };
  int kt = 0;
#pragma unroll 1
  for (; kt < KT - S - 1; ++kt) step(std::integral_constant<int, 1>(), kt);
  if (kt < KT - S) step(std::integral_constant<int, 2>(), kt++);
#pragma unroll 1
  for (; kt < KT; ++kt) step(std::integral_constant<int, 0>(), kt);
  lds_barrier();  // the stages are free
}

// Workgroup -> tile.  Workgroups go round the 8 XCDs; each XCD takes a
// contiguous range of tiles, ordered in bands of GM tile rows, so the tiles
// it works on at one time share few row and column panels in its L2.
constexpr int HEAD_GM = 4;
MOE_DEV void head_order(int idx, int nm, int nn, int& m, int& n) {
  const int band = idx / (HEAD_GM * nn), rem = idx - band * HEAD_GM * nn;
  const int gm = min(HEAD_GM, nm - band * HEAD_GM);
  n = rem / gm;
  m = band * HEAD_GM + rem - n * gm;
}
// Place of workgroup bid among `total` pieces of work, -1 past them.
MOE_DEV int head_place(int bid, int total) {
  const int per = (total + 7) >> 3, at = bid >> 3, idx = (bid & 7) * per + at;
  return at >= per || idx >= total ? -1 : idx;
}
MOE_DEV bool head_tile(int bid, int nm, int nn, int& m, int& n) {
  const int idx = head_place(bid, nm * nn);
  if (idx < 0) return false;
  head_order(idx, nm, nn, m, n);
  return true;
}
// The same where the last round of tiles would leave half of the CUs idle: its
// tiles are done as two halves of BM/2 rows each (2867 rows of 2048 x 50257:
// 523 -> 487 us; 3686 of 7168 x 32000: 1365 -> 1320).  Halves: `half` is 0 or 1;
// -1: a whole tile.
MOE_DEV bool head_tile_tail(int bid, int nm, int nn, int slots, int& m, int& n, int& half) {
  const int nt = nm * nn;
  int whole = nt / slots * slots & ~7;
  if ((nt - whole) * 2 > slots) whole = nt;
  half = -1;
  if (whole == nt) return head_tile(bid, nm, nn, m, n);
  int idx;
  if (bid < whole) {
    idx = head_place(bid, whole);
  } else {
    idx = head_place(bid - whole, (nt - whole) * 2);
    if (idx < 0) return false;
    half = idx & 1;
    idx = whole + (idx >> 1);
  }
  head_order(idx, nm, nn, m, n);
  return true;
}

struct HeadGemm {
  const uint16_t* h;      // direct forward: the rows as they are, T of them
  int64_t h_stride;
  int T;
  float eps;
  const uint16_t* hc;     // [..][Hp]
  const uint16_t* w;
  int64_t w_stride;
  int H, Hp, V, top;
  const int32_t* rows;
  const int32_t* count;   // rows, splits of G W
  const float* r;         // [count]
  int32_t* eid;           // [count][top] G's entries at the target's ids: id (-1: none),
  float* ev;              //   value (null: none are kept)
  bool exact;             // what rounding them takes off is added to u
  const int2* rtile;      // d_w: first row and rows of each 256 ids in rlist and rem
  const int32_t* rlist;   // rows of hc with an entry among those ids
  const uint16_t* rem;    // [..][256] what rounding took off those entries
  int zero_row;           // of hc
  const HeadRow* info;    // [..]
  float scale;
  const int32_t* ids;
  bool distill;
  float* stats;   // [count][nvb][2]
  float* zt;      // [count][top]
  uint16_t* g;    // [..][piece]
  float* u;       // [count][H]
  uint16_t* dw;   // [V][H]
  float* lp;      // [psplits][T][Vp] partial h W^T (K split), Vp a multiple of 4
  int psplits, Vp;
  bool direct;    // its rows are h's as they are
  int slots;      // CUs
  int v0, piece;
};

// Forward: per row and block of BN columns the maximum of y = l log2 e and the
// sum of 2^(y - maximum), and the logits at the target's ids (the tile goes
// through LDS for those).  DIRECT: for one tile row (up to 128) of a width that is
// a multiple of 64 the rows are read where they are and their 1/rms is formed
// from the staged pieces, so nothing has to be launched before this.
template <class C>
struct HeadStats {
  static constexpr int RED = C::WN * C::BM * 4;  // bytes of the rows' maxima, and of their sums
  // the tile of logits, or a part of it, and the rows' statistics behind it
  static constexpr int ZR = C::BM * C::BN * 4 + 2 * RED <= C::SMEM ? C::BM : C::BM / C::WM;
  static constexpr int ZB = ZR * C::BN * 4;
  static constexpr int SMEM = ZB + 2 * RED > C::SMEM ? ZB + 2 * RED : C::SMEM;
};
template <class C, bool DIRECT>
MOE_DEV void head_stats(const HeadGemm& p, int n, int m0, int nt, uint8_t* smem) {
  constexpr int RED = HeadStats<C>::RED, ZR = HeadStats<C>::ZR, ZB = HeadStats<C>::ZB;
  float(*rm)[C::BM] = reinterpret_cast<float(*)[C::BM]>(smem + ZB);
  float(*rs)[C::BM] = reinterpret_cast<float(*)[C::BM]>(smem + ZB + RED);
  const int n0 = nt * C::BN, nvb = (p.V + C::BN - 1) / C::BN;
  HeadSrc sa = {reinterpret_cast<const char*>(p.hc + (int64_t)m0 * p.Hp), (uint32_t)p.Hp * 2, C::BM, p.Hp};
  if (DIRECT) sa = HeadSrc{reinterpret_cast<const char*>(p.h), (uint32_t)p.h_stride * 2, n, p.H};
  const HeadSrc sb = {reinterpret_cast<const char*>(p.w + (int64_t)n0 * p.w_stride), (uint32_t)p.w_stride * 2,
                      p.V - n0, p.H};
  f32x4 acc[C::MI][C::NJ];
  float ss = 0.0f;
  head_mm<C, false, false, DIRECT>(sa, sb, p.Hp / 64, acc, smem, &ss);
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, ln = lane & 15, lg = lane >> 4;
  const int wm = wave / C::WN * C::MI * 16, wn = wave % C::WN * C::NJ * 16;
  const bool full = n0 + C::BN <= p.V;  // uniform: no column of the tile is past the vocabulary
  HeadRow info[C::MI];
  if (DIRECT) {
    ss += shfl_xor(ss, 1);
    ss += shfl_xor(ss, 2);
    float* rr = reinterpret_cast<float*>(smem);
    if ((threadIdx.x & 3) == 0) rr[threadIdx.x >> 2] = p.eps > 0.0f ? 1.0f / sqrtf(ss / (float)p.H + p.eps) : 1.0f;
    lds_barrier();
#pragma unroll
    for (int i = 0; i < C::MI; ++i) {
      const int row = wm + i * 16 + ln;
      const float f = p.scale * rr[row];
      info[i] = HeadRow{f * kLog2e, f, 0.0f, p.distill || row >= n ? -1 : p.ids[row]};
    }
    lds_barrier();
  } else {
#pragma unroll
    for (int i = 0; i < C::MI; ++i) info[i] = p.info[m0 + wm + i * 16 + ln];
  }
  auto rows_stats = [&](auto all) {
    constexpr bool ALL = decltype(all)::value;
#pragma unroll
    for (int i = 0; i < C::MI; ++i) {
      const int row = wm + i * 16 + ln;
      float mx = -INFINITY, s = 0.0f;
#pragma unroll
      for (int j = 0; j < C::NJ; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (ALL || n0 + wn + j * 16 + lg * 4 + e < p.V) mx = fmaxf(mx, acc[i][j][e]);
      mx = fmaxf(mx, shfl_xor(mx, 16));
      const float top = fmaxf(mx, shfl_xor(mx, 32));
      mx = top * info[i].f2;
      if (!__any(fabsf(mx) > kFarLogit)) {
#pragma unroll
        for (int j = 0; j < C::NJ; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (ALL || n0 + wn + j * 16 + lg * 4 + e < p.V) s += hl_exp2(fmaf(acc[i][j][e], info[i].f2, -mx));
      } else {
#pragma unroll
        for (int j = 0; j < C::NJ; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (ALL || n0 + wn + j * 16 + lg * 4 + e < p.V) s += hl_exp2((acc[i][j][e] - top) * info[i].f2);
      }
      s += shfl_xor(s, 16);
      s += shfl_xor(s, 32);
      if (lg == 0) {
        rm[wave % C::WN][row] = mx;
        rs[wave % C::WN][row] = s;
      }
    }
  };
  if (full) rows_stats(std::true_type());
  else rows_stats(std::false_type());
  if (!p.distill) {
    // the one lane that holds a row's target picks it out
#pragma unroll
    for (int i = 0; i < C::MI; ++i) {
      const int tc = info[i].tgt - n0 - wn;
      const bool hit = tc >= 0 && tc < C::NJ * 16 && ((tc >> 2) & 3) == lg;
      if (!__any(hit)) continue;
      float z = 0.0f;
#pragma unroll
      for (int j = 0; j < C::NJ; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) z = tc == j * 16 + lg * 4 + e ? acc[i][j][e] : z;
      if (hit) p.zt[m0 + wm + i * 16 + ln] = z * info[i].f;
    }
    lds_barrier();
  } else {
    // the logits go through LDS, ZR rows of the tile at a time, 16-byte piece q
    // of a row at q ^ (row & 15); NT / ZR threads look up a row's ids
#pragma unroll
    for (int z0 = 0; z0 < C::BM; z0 += ZR) {
      if (z0) lds_barrier();
      if (ZR == C::BM || wm == z0) {
#pragma unroll
        for (int i = 0; i < C::MI; ++i)
#pragma unroll
          for (int j = 0; j < C::NJ; ++j) {
            const int row = wm + i * 16 + ln, q = (wn + j * 16) / 4 + lg;
            *reinterpret_cast<f32x4*>(smem + (row - z0) * C::BN * 4 + ((q ^ (row & 15)) << 4)) = acc[i][j] * info[i].f;
          }
      }
      lds_barrier();
      constexpr int TPR = C::NT / ZR > 0 ? C::NT / ZR : 1;
      const int row = z0 + (int)threadIdx.x / TPR, c = m0 + row;
      if (threadIdx.x < ZR * TPR && c < n) {
        const int32_t* id = p.ids + (int64_t)(DIRECT ? c : p.rows[c]) * p.top;
        for (int k = threadIdx.x % TPR; k < p.top; k += TPR) {
          const int v = id[k] - n0;
          if (v >= 0 && v < C::BN && n0 + v < p.V)
            p.zt[(int64_t)c * p.top + k] = *reinterpret_cast<const float*>(
                smem + (row - z0) * C::BN * 4 + (((v >> 2) ^ (row & 15)) << 4) + (v & 3) * 4);
        }
      }
    }
  }
  for (int row = threadIdx.x; row < C::BM && m0 + row < n; row += C::NT) {
    float m = rm[0][row], s = rs[0][row];
#pragma unroll
    for (int w = 1; w < C::WN; ++w) hl_merge(m, s, rm[w][row], rs[w][row]);
    float* o = p.stats + ((int64_t)(m0 + row) * nvb + nt) * 2;
    o[0] = m;
    o[1] = s;
  }
}
template <class C, bool DIRECT>
__global__ __launch_bounds__(C::NT, C::WPS) void k_head_stats(HeadGemm p) {
  using Half = typename C::Half;
  constexpr int SMEM = HeadStats<C>::SMEM > HeadStats<Half>::SMEM ? HeadStats<C>::SMEM : HeadStats<Half>::SMEM;
  __shared__ __align__(16) uint8_t smem[SMEM];
  const int n = DIRECT ? p.T : *p.count, nm = (n + C::BM - 1) / C::BM, nvb = (p.V + C::BN - 1) / C::BN;
  int mt, nt, half = -1;
  if (std::is_same<C, Half>::value ? !head_tile(blockIdx.x, nm, nvb, mt, nt)
                                   : !head_tile_tail(blockIdx.x, nm, nvb, p.slots, mt, nt, half))
    return;
  if (half < 0) {
    head_stats<C, DIRECT>(p, n, mt * C::BM, nt, smem);
  } else {
    const int m0 = mt * C::BM + half * Half::BM;
    if (m0 < n) head_stats<Half, DIRECT>(p, n, m0, nt, smem);
  }
}

// The tile of a wave's accumulators as bf16 rows in LDS, for stores of whole
// rows: 8 bytes per lane straight to memory would leave 32-byte pieces of 16
// rows per instruction.
template <class C>
struct HeadOut {
  static constexpr int LS = C::BN * 2 + 16;  // LDS row stride
  static_assert(C::BM * LS <= C::SMEM, "the tile fits the stage buffers");
  MOE_DEV static uint8_t* at(uint8_t* smem, int row, int col) { return smem + row * LS + col * 2; }
  // Rows [0, nrows) and bytes [0, nb) of each (a multiple of 16) to g, gs bytes apart.
  MOE_DEV static void store(const uint8_t* smem, char* g, int64_t gs, int nrows, int nb) {
    constexpr int PPR = C::BN / 8, RPI = C::NT / PPR;  // 16-byte pieces per row, rows per step
    const int r0 = (int)threadIdx.x / PPR, x = (int)threadIdx.x % PPR * 16;
    if (x >= nb) return;
    constexpr int G = C::BM / RPI >= 4 ? 4 : 1;
#pragma unroll 1
    for (int r = r0; r < C::BM; r += G * RPI) {
      u32x4 v[G];
#pragma unroll
      for (int i = 0; i < G; ++i) v[i] = *reinterpret_cast<const u32x4*>(smem + (r + i * RPI) * LS + x);
#pragma unroll
      for (int i = 0; i < G; ++i)
        if (r + i * RPI < nrows) *reinterpret_cast<u32x4*>(g + (r + i * RPI) * gs + x) = v[i];
    }
  }
};

// Backward: G, columns [v0, v0 + piece), of every row of the tiles (zeros
// behind the last row and past the vocabulary).
template <class C>
MOE_DEV void head_grad(const HeadGemm& p, int m0, int nt, uint8_t* smem) {
  const int n0 = p.v0 + nt * C::BN;
  const HeadSrc sa = {reinterpret_cast<const char*>(p.hc + (int64_t)m0 * p.Hp), (uint32_t)p.Hp * 2, C::BM, p.Hp};
  // a piece's last tiles may lie past the vocabulary: they read its last row and write zeros
  const int nb = min(n0, p.V - 1);
  const HeadSrc sb = {reinterpret_cast<const char*>(p.w + (int64_t)nb * p.w_stride), (uint32_t)p.w_stride * 2,
                      p.V - nb, p.H};
  f32x4 acc[C::MI][C::NJ];
  head_mm<C, false, false>(sa, sb, p.Hp / 64, acc, smem);
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, ln = lane & 15, lg = lane >> 4;
  const int wm = wave / C::WN * C::MI * 16, wn = wave % C::WN * C::NJ * 16;
  const bool full = n0 + C::BN <= p.V;
  HeadRow info[C::MI];
#pragma unroll
  for (int i = 0; i < C::MI; ++i) info[i] = p.info[m0 + wm + i * 16 + ln];
  auto write = [&](auto all) {
    constexpr bool ALL = decltype(all)::value;
#pragma unroll
    for (int i = 0; i < C::MI; ++i) {
      uint8_t* o = HeadOut<C>::at(smem, wm + i * 16 + ln, wn + lg * 4);
      if (__any(fabsf(info[i].l2) > kFarLogit)) {  // p <= 1 whatever roundings of l and lse leave
#pragma unroll
        for (int j = 0; j < C::NJ; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            acc[i][j][e] = hl_not_above_0(fmaf(acc[i][j][e], info[i].f2, -info[i].l2));
        info[i].f2 = 1.0f;
        info[i].l2 = 0.0f;
      }
#pragma unroll
      for (int j = 0; j < C::NJ; ++j) {
        float x[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[e] = info[i].f * hl_exp2(fmaf(acc[i][j][e], info[i].f2, -info[i].l2));
          if (!ALL && n0 + wn + j * 16 + lg * 4 + e >= p.V) x[e] = 0.0f;
        }
        *reinterpret_cast<u32x2*>(o + j * 32) = (u32x2){bf16x2_bits(x[0], x[1]), bf16x2_bits(x[2], x[3])};
      }
    }
  };
  if (full) write(std::true_type());
  else write(std::false_type());
  if (!p.distill) {
    // the lane that wrote a row's target puts s r g (p - 1) over it
#pragma unroll
    for (int i = 0; i < C::MI; ++i) {
      const int tc = info[i].tgt - n0 - wn;
      if (tc >= 0 && tc < C::NJ * 16 && ((tc >> 2) & 3) == lg)
        *reinterpret_cast<uint16_t*>(HeadOut<C>::at(smem, wm + i * 16 + ln, wn + tc)) =
            (uint16_t)f32_to_bf16_bits(p.ev[m0 + wm + i * 16 + ln]);
    }
  }
  lds_barrier();
  HeadOut<C>::store(smem, reinterpret_cast<char*>(p.g + (int64_t)m0 * p.piece + (n0 - p.v0)), (int64_t)p.piece * 2,
                    C::BM, C::BN * 2);
}
template <class C>
__global__ __launch_bounds__(C::NT, C::WPS) void k_head_grad(HeadGemm p) {
  using Half = typename C::Half;
  __shared__ __align__(16) uint8_t smem[C::SMEM > Half::SMEM ? C::SMEM : Half::SMEM];
  const int nm = (*p.count + C::BM - 1) / C::BM, nn = p.piece / C::BN;
  int mt, nt, half = -1;
  if (std::is_same<C, Half>::value ? !head_tile(blockIdx.x, nm, nn, mt, nt)
                                   : !head_tile_tail(blockIdx.x, nm, nn, p.slots, mt, nt, half))
    return;
  // rows behind the last one get their zeros from either half
  if (half < 0) head_grad<C>(p, mt * C::BM, nt, smem);
  else head_grad<Half>(p, mt * C::BM + half * Half::BM, nt, smem);
}

// u (slab of this workgroup's share of K) += G W over a piece.
template <class C>
MOE_DEV void head_dz(const HeadGemm& p, int bid, uint8_t* smem) {
  const int n = *p.count, nm = (n + C::BM - 1) / C::BM, nn = (p.H + C::BN - 1) / C::BN;
  if (n == 0) return;
  const int splits = p.count[1];
  int mt, nt;
  if (!head_tile(bid, nm * splits, nn, mt, nt)) return;
  const int sp = mt / nm;
  mt -= sp * nm;
  const int Kp = min(p.piece, p.V - p.v0), steps = (Kp + 63) / 64;
  const int k0 = (int)((int64_t)steps * sp / splits) * 64, k1 = (int)((int64_t)steps * (sp + 1) / splits) * 64;
  const int m0 = mt * C::BM, n0 = nt * C::BN, K = min(k1, Kp) - k0;
  f32x4 acc[C::MI][C::NJ];
  if (K > 0) {
    const HeadSrc sa = {reinterpret_cast<const char*>(p.g + (int64_t)m0 * p.piece + k0), (uint32_t)p.piece * 2, C::BM,
                        p.piece - k0};
    const HeadSrc sb = {reinterpret_cast<const char*>(p.w + (int64_t)(p.v0 + k0) * p.w_stride + n0),
                        (uint32_t)p.w_stride * 2, p.H - n0, K};
    head_mm<C, false, true>(sa, sb, (K + 63) / 64, acc, smem);
  } else if (p.v0 != 0) {
    return;
  } else {
#pragma unroll
    for (int i = 0; i < C::MI; ++i)
#pragma unroll
      for (int j = 0; j < C::NJ; ++j) acc[i][j] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
  }
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, ln = lane & 15, lg = lane >> 4;
  const int wm = wave / C::WN * C::MI * 16, wn = wave % C::WN * C::NJ * 16;
#pragma unroll
  for (int i = 0; i < C::MI; ++i) {
    const int c = m0 + wm + i * 16 + ln;
    if (c >= n) continue;
#pragma unroll
    for (int j = 0; j < C::NJ; ++j) {
      const int col = n0 + wn + j * 16 + lg * 4;
      if (col >= p.H) continue;
      f32x4* o = reinterpret_cast<f32x4*>(p.u + ((int64_t)sp * n + c) * p.H + col);
      *o = p.v0 == 0 ? acc[i][j] : *o + acc[i][j];
    }
  }
}

// d_w rows [v0, v0 + piece) = G^T h, with rem^T h of the rows that have entries
// there in the same accumulators: d_w is rounded once.
template <class C>
MOE_DEV void head_dw(const HeadGemm& p, int bid, uint8_t* smem) {
  const int n = *p.count, M = min(p.piece, p.V - p.v0);
  int mt, nt;
  if (!head_tile(bid, (M + C::BM - 1) / C::BM, (p.H + C::BN - 1) / C::BN, mt, nt)) return;
  const int m0 = mt * C::BM, n0 = nt * C::BN, KT = (n + 63) / 64;
  const HeadSrc sa = {reinterpret_cast<const char*>(p.g + m0), (uint32_t)p.piece * 2, p.piece - m0, KT * 64};
  const HeadSrc sb = {reinterpret_cast<const char*>(p.hc + n0), (uint32_t)p.Hp * 2, p.Hp - n0, KT * 64};
  f32x4 acc[C::MI][C::NJ];
  if (KT > 0) {
    head_mm<C, true, true>(sa, sb, KT, acc, smem);
  } else {
#pragma unroll
    for (int i = 0; i < C::MI; ++i)
#pragma unroll
      for (int j = 0; j < C::NJ; ++j) acc[i][j] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
  }
  if (p.rtile != nullptr) {
    static_assert(C::BM == 256, "rem's width");
    const int2 r = p.rtile[(p.v0 + m0) / 256];
    const int first = __builtin_amdgcn_readfirstlane(r.x), k = __builtin_amdgcn_readfirstlane(r.y);
    if (k > 0) {
      const HeadSrc ra = {reinterpret_cast<const char*>(p.rem + (int64_t)first * 256), 512, 256, k};
      const HeadSrc rb = {reinterpret_cast<const char*>(p.hc + n0), (uint32_t)p.Hp * 2, p.Hp - n0, k, p.rlist + first,
                          p.zero_row};
      head_mm<C, true, true, false, true>(ra, rb, (k + 63) / 64, acc, smem);
    }
  }
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, ln = lane & 15, lg = lane >> 4;
  const int wm = wave / C::WN * C::MI * 16, wn = wave % C::WN * C::NJ * 16;
#pragma unroll
  for (int i = 0; i < C::MI; ++i)
#pragma unroll
    for (int j = 0; j < C::NJ; ++j)
      *reinterpret_cast<u32x2*>(HeadOut<C>::at(smem, wm + i * 16 + ln, wn + j * 16 + lg * 4)) =
          (u32x2){bf16x2_bits(acc[i][j][0], acc[i][j][1]), bf16x2_bits(acc[i][j][2], acc[i][j][3])};
  lds_barrier();
  HeadOut<C>::store(smem, reinterpret_cast<char*>(p.dw + (int64_t)(p.v0 + m0) * p.H + n0), (int64_t)p.H * 2, M - m0,
                    (p.H - n0) * 2);
}

template <class C>
__global__ __launch_bounds__(C::NT, C::WPS) void k_head_dz(HeadGemm p) {
  __shared__ __align__(16) uint8_t smem[C::SMEM];
  head_dz<C>(p, blockIdx.x, smem);
}
template <class C>
__global__ __launch_bounds__(C::NT, C::WPS) void k_head_dw(HeadGemm p) {
  __shared__ __align__(16) uint8_t smem[C::SMEM];
  head_dw<C>(p, blockIdx.x, smem);
}
// Both of a piece in one launch, the longer G W tiles first: the G^T h tiles
// fill the CUs that its last round leaves idle.
template <class C>
__global__ __launch_bounds__(C::NT, C::WPS) void k_head_dz_dw(HeadGemm p, int ndz) {
  __shared__ __align__(16) uint8_t smem[C::SMEM];
  if ((int)blockIdx.x < ndz) head_dz<C>(p, blockIdx.x, smem);
  else head_dw<C>(p, blockIdx.x - ndz, smem);
}

// Few tiles (a small vocabulary, few rows) leave CUs idle and, with each tile's
// own requests alone in flight, most of the memory's rate unused.  There K is
// split: partial h W^T go to slabs of fp32 (at most 64 MB), and what the
// epilogues above do is done from their sums.
template <class C>
__global__ __launch_bounds__(C::NT, C::WPS) void k_head_part(HeadGemm p) {
  __shared__ __align__(16) uint8_t smem[C::SMEM];
  const int n = p.direct ? p.T : *p.count, nm = (n + C::BM - 1) / C::BM;
  int mt, nt;
  if (n == 0 || !head_tile(blockIdx.x, nm * p.psplits, (p.V + C::BN - 1) / C::BN, mt, nt)) return;
  const int sp = mt / nm;
  mt -= sp * nm;
  const int steps = p.Hp / 64, s0 = steps * sp / p.psplits, s1 = steps * (sp + 1) / p.psplits;
  const int m0 = mt * C::BM, n0 = nt * C::BN, k0 = s0 * 64;
  HeadSrc sa = {reinterpret_cast<const char*>(p.hc + (int64_t)m0 * p.Hp + k0), (uint32_t)p.Hp * 2, C::BM, p.Hp - k0};
  if (p.direct)
    sa = HeadSrc{reinterpret_cast<const char*>(p.h + (int64_t)m0 * p.h_stride + k0), (uint32_t)p.h_stride * 2, n - m0,
                 p.H - k0};
  const HeadSrc sb = {reinterpret_cast<const char*>(p.w + (int64_t)n0 * p.w_stride + k0), (uint32_t)p.w_stride * 2,
                      p.V - n0, p.H - k0};
  f32x4 acc[C::MI][C::NJ];
  head_mm<C, false, false>(sa, sb, s1 - s0, acc, smem);
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, ln = lane & 15, lg = lane >> 4;
  const int wm = wave / C::WN * C::MI * 16, wn = wave % C::WN * C::NJ * 16;
#pragma unroll
  for (int i = 0; i < C::MI; ++i) {
    const int c = m0 + wm + i * 16 + ln;
    if (c >= n) continue;
#pragma unroll
    for (int j = 0; j < C::NJ; ++j) {
      const int col = n0 + wn + j * 16 + lg * 4;
      if (col < p.V) *reinterpret_cast<f32x4*>(p.lp + ((int64_t)sp * p.T + c) * p.Vp + col) = acc[i][j];
    }
  }
}
// Columns v .. v + 3 of row c: the slabs' sum, in order.
MOE_DEV f32x4 head_part4(const HeadGemm& p, int c, int v) {
  const float* o = p.lp + (int64_t)c * p.Vp + v;
  const int64_t slab = (int64_t)p.T * p.Vp;
  f32x4 z = *reinterpret_cast<const f32x4*>(o);
  int s = 1;
  for (; s + 3 < p.psplits; s += 3) {  // three slabs' loads in flight
    const f32x4 a = *reinterpret_cast<const f32x4*>(o + s * slab), b = *reinterpret_cast<const f32x4*>(o + (s + 1) * slab),
                c3 = *reinterpret_cast<const f32x4*>(o + (s + 2) * slab);
    z = ((z + a) + b) + c3;
  }
  for (; s < p.psplits; ++s) z += *reinterpret_cast<const f32x4*>(o + s * slab);
  return z;
}
MOE_DEV float head_part1(const HeadGemm& p, int c, int v) { return head_part4(p, c, v & ~3)[v & 3]; }

// G from the slabs: a block takes 2048 columns of a row, 8 per thread.
__global__ __launch_bounds__(256) void k_head_part_grad(HeadGemm p, int bm) {
  const int c = blockIdx.x, n = p.count[0], v = blockIdx.y * 2048 + (int)threadIdx.x * 8;
  if (c >= (n + bm - 1) / bm * bm || v >= p.piece) return;
  const HeadRow w = p.info[c];
  float x[8];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    f32x4 z = {0.0f, 0.0f, 0.0f, 0.0f};
    if (c < n && v + k * 4 < p.V) z = head_part4(p, c, v + k * 4);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int at = v + k * 4 + e;
      x[k * 4 + e] = c < n && at < p.V ? w.f * hl_exp2(hl_not_above_0(fmaf(z[e], w.f2, -w.l2))) : 0.0f;
      if (!p.distill && at == w.tgt && at < p.V) x[k * 4 + e] = p.ev[c];
    }
  }
  *reinterpret_cast<u32x4*>(p.g + (int64_t)c * p.piece + v) =
      (u32x4){bf16x2_bits(x[0], x[1]), bf16x2_bits(x[2], x[3]), bf16x2_bits(x[4], x[5]), bf16x2_bits(x[6], x[7])};
}

// Per token (one wave): joins its blocks' statistics and forms the outputs.
// Bound by the latency of a few dependent reads (4-6 us at 1 to 4096 tokens).
// DIRECT: row t is token t, and whether it counts and the teacher's
// probabilities are found here.
struct HeadFinish {
  const float* stats;
  const float* zt;
  const int32_t* cidx;
  const int32_t* ids;
  const float* lq;
  const float* tlogits;
  float tscale;
  int T, V, nvb, top;
  float* loss;
  float* lse;
  float* logp;  // null: cross entropy
};
template <bool DIRECT>
__global__ __launch_bounds__(256) void k_head_finish(HeadFinish p) {
  const int t = blockIdx.x * 4 + (threadIdx.x >> 6), lane = threadIdx.x & 63;
  if (t >= p.T) return;
  const bool distill = p.logp != nullptr;
  float lq[4];  // of slots lane, lane + 64, ...
  int c = t;
  if (DIRECT) {
    if (distill) {
      c = head_teacher(p.ids + (int64_t)t * p.top, p.tlogits + (int64_t)t * p.top, p.V, p.top, p.tscale, lane, lq) ? t
                                                                                                                  : -1;
    } else {
      const int y = p.ids[t];
      c = y >= 0 && y < p.V ? t : -1;
    }
  } else {
    c = p.cidx[t];
    if (distill)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        lq[i] = i * 64 + lane < p.top ? p.lq[(int64_t)t * p.top + i * 64 + lane] : -INFINITY;
  }
  if (c < 0) {
    if (distill)
      for (int j = lane; j < p.top; j += 64) p.logp[(int64_t)t * p.top + j] = 0.0f;
    if (lane == 0) {
      p.loss[t] = !distill && p.ids[t] >= p.V ? __builtin_nanf("") : 0.0f;
      p.lse[t] = 0.0f;
    }
    return;
  }
  float m = -INFINITY, s = 0.0f;
  for (int b = lane; b < p.nvb; b += 64) {
    const float* o = p.stats + ((int64_t)c * p.nvb + b) * 2;
    hl_merge(m, s, o[0], o[1]);
  }
#pragma unroll
  for (int x = 1; x < 64; x <<= 1) {
    const float m2 = shfl_xor(m, x), s2 = shfl_xor(s, x);
    hl_merge(m, s, m2, s2);
  }
  const float l = m * kLn2 + logf(s);
  float kl;
  if (distill) {
    kl = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int j = i * 64 + lane;
      if (j < p.top) {
        const bool have = !(lq[i] == -INFINITY);
        const float lp = have ? hl_not_above_0(p.zt[(int64_t)c * p.top + j] - l) : 0.0f;
        p.logp[(int64_t)t * p.top + j] = lp;
        if (have) kl = fmaf(expf(lq[i]), lq[i] - lp, kl);
      }
    }
    kl = hl_sum64(kl);
  } else {
    kl = hl_not_below_0(l - p.zt[c]);
  }
  if (lane == 0) {
    p.loss[t] = kl;
    p.lse[t] = l;
  }
}

// The same from slabs, one block per token.  p.direct: 1/rms is formed here too.
__global__ __launch_bounds__(256) void k_head_part_finish(HeadGemm g, HeadFinish p) {
  __shared__ float sm[4], ss[4];
  const int t = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const bool distill = p.logp != nullptr;
  float lq[4];
  int c = t;
  if (g.direct) {
    if (distill) {
      c = head_teacher(p.ids + (int64_t)t * p.top, p.tlogits + (int64_t)t * p.top, p.V, p.top, p.tscale, lane, lq) ? t
                                                                                                                  : -1;
    } else {
      const int y = p.ids[t];
      c = y >= 0 && y < p.V ? t : -1;
    }
  } else {
    c = p.cidx[t];
    if (distill)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        lq[i] = i * 64 + lane < p.top ? p.lq[(int64_t)t * p.top + i * 64 + lane] : -INFINITY;
  }
  if (c < 0) {
    if (distill)
      for (int j = tid; j < p.top; j += 256) p.logp[(int64_t)t * p.top + j] = 0.0f;
    if (tid == 0) {
      p.loss[t] = !distill && p.ids[t] >= p.V ? __builtin_nanf("") : 0.0f;
      p.lse[t] = 0.0f;
    }
    return;
  }
  float f;
  if (g.direct) {
    float r = 1.0f;
    if (g.eps > 0.0f) {
      float sq = 0.0f;
      const uint16_t* row = g.h + (int64_t)t * g.h_stride;
      for (int i = tid; i < g.H / 8; i += 256) {
        const u32x4 q = *reinterpret_cast<const u32x4*>(row + i * 8);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float a = bf16_bits_to_f32(q[j] & 0xFFFFu), b = bf16_bits_to_f32(q[j] >> 16);
          sq = fmaf(a, a, sq);
          sq = fmaf(b, b, sq);
        }
      }
      sq = hl_sum64(sq);
      if (lane == 0) ss[wave] = sq;
      __syncthreads();
      r = 1.0f / sqrtf(((ss[0] + ss[1]) + (ss[2] + ss[3])) / (float)g.H + g.eps);
      __syncthreads();
    }
    f = g.scale * r;
  } else {
    f = g.info[c].f;
  }
  const float f2 = f * kLog2e;
  float m = -INFINITY, s = 0.0f;
  for (int v = tid * 4; v < p.V; v += 1024) {
    const f32x4 z = head_part4(g, c, v);
    float y[4], mx = -INFINITY;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      y[e] = v + e < p.V ? z[e] : -INFINITY;
      mx = fmaxf(mx, y[e]);
    }
    float sum = 0.0f;
#pragma unroll
    for (int e = 0; e < 4; ++e) sum += hl_exp2((y[e] - mx) * f2);
    hl_merge(m, s, mx * f2, sum);
  }
#pragma unroll
  for (int x = 1; x < 64; x <<= 1) {
    const float m2 = shfl_xor(m, x), s2 = shfl_xor(s, x);
    hl_merge(m, s, m2, s2);
  }
  if (lane == 0) {
    sm[wave] = m;
    ss[wave] = s;
  }
  __syncthreads();
  if (wave != 0) return;
  m = sm[0];
  s = ss[0];
#pragma unroll
  for (int w = 1; w < 4; ++w) hl_merge(m, s, sm[w], ss[w]);
  const float l = m * kLn2 + logf(s);
  float kl;
  if (distill) {
    kl = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int j = i * 64 + lane;
      if (j < p.top) {
        const bool have = !(lq[i] == -INFINITY);
        const float lp = have ? hl_not_above_0(head_part1(g, c, p.ids[(int64_t)t * p.top + j]) * f - l) : 0.0f;
        p.logp[(int64_t)t * p.top + j] = lp;
        if (have) kl = fmaf(expf(lq[i]), lq[i] - lp, kl);
      }
    }
    kl = hl_sum64(kl);
  } else {
    kl = hl_not_below_0(l - head_part1(g, c, p.ids[t]) * f);
  }
  if (lane == 0) {
    p.loss[t] = kl;
    p.lse[t] = l;
  }
}

// Distillation's backward: the entries s r g (p - q) at the slots' ids, from
// the forward's log-probs, one wave per row, into G's columns [v0, v0 + piece).
// Slots that repeat an id add their q, and the first of them is the entry.  ev
// not null: with the first piece the entries go to ev too, their ids to eid.
// 8 us for 1500 rows of 33 slots: reads that wait for each other.
__global__ __launch_bounds__(256) void k_head_targets(const int32_t* __restrict__ rows, const int32_t* __restrict__ count,
                                                      const int32_t* __restrict__ ids, const float* __restrict__ lq,
                                                      const float* __restrict__ logp, const HeadRow* __restrict__ info,
                                                      int top, int v0, int piece, uint16_t* __restrict__ g,
                                                      int32_t* __restrict__ eid, float* __restrict__ ev) {
  __shared__ int sid[4][256];
  __shared__ float sq[4][256];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int c = blockIdx.x * 4 + wave;
  if (c >= *count) return;
  const int t = rows[c];
  const float cf = info[c].f;
  for (int j = lane; j < top; j += 64) {
    const float q = lq[(int64_t)t * top + j];
    const bool have = !(q == -INFINITY);
    sid[wave][j] = have ? ids[(int64_t)t * top + j] : -1;
    sq[wave][j] = have ? expf(q) : 0.0f;
  }
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");  // a wave reads only its own slots
  __builtin_amdgcn_wave_barrier();
  for (int j = lane; j < top; j += 64) {
    const int id = sid[wave][j], v = id - v0;
    const bool here = id >= 0 && v >= 0 && v < piece;
    if (!here && (ev == nullptr || v0 != 0)) continue;
    float q = 0.0f;
    bool first = id >= 0;
    for (int i = 0; i < top; ++i)
      if (sid[wave][i] == id) {
        q += sq[wave][i];
        if (i < j) first = false;
      }
    const float x = first ? cf * (expf(logp[(int64_t)t * top + j]) - q) : 0.0f;
    if (ev != nullptr && v0 == 0) {
      eid[(int64_t)c * top + j] = first ? id : -1;
      ev[(int64_t)c * top + j] = x;
    }
    if (here && first) g[(int64_t)c * piece + v] = (uint16_t)f32_to_bf16_bits(x);
  }
}

// What the rounding of an entry to bf16 took off (0 where that has no value).
MOE_DEV float head_rem(float x) {
  const float r = x - bf16_bits_to_f32(f32_to_bf16_bits(x));
  return fabsf(r) < INFINITY ? r : 0.0f;
}

// For d_w: the tokens that have entries among each 256 ids, in order, and what
// rounding took off those entries as rows of 256 bf16 (again rounded: 2^-16 of
// the entry is left), which head_dw multiplies by the tokens' rows of h.  The
// tokens of 256 ids lie behind the entries of all lower ids, so that one row per
// entry is room enough; places that stay free get tile -1.  Lists and rows are
// 9-10 and 5 us for 8192 targets of 32000 ids, 16-19 and 8-9 for 1500 x 33 of
// 50257, dependent reads; in head_dw they are 1-2 more K steps a tile (128 of
// tokens) and 4 (24).
struct HeadRem {
  const int32_t* eid;
  const float* ev;
  const int32_t* count;
  int top;
  int2* tile;         // first place, tokens
  int32_t* list;      // [places] token
  int32_t* own;       // [places] tile
  uint16_t* rem;      // [places][256]
  uint16_t* zero_row; // of hc
  int Hp;
};
// Row `at` by 32 lanes: token c's entries among ids lo .. lo + 255.
MOE_DEV void head_rem_row(const HeadRem& p, int at, int c, int lo, int l, uint16_t* buf) {
  const int32_t* id = p.eid + (int64_t)c * p.top;
  const float* ev = p.ev + (int64_t)c * p.top;
  *reinterpret_cast<u32x4*>(buf + l * 8) = (u32x4){0, 0, 0, 0};
  for (int j = l; j < p.top; j += 32) {
    const int v = id[j] - lo;
    const float x = ev[j];
    if (v >= 0 && v < 256) buf[v] = (uint16_t)f32_to_bf16_bits(head_rem(x));  // an id has one entry at most
  }
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");  // the lanes are of one wave
  __builtin_amdgcn_wave_barrier();
  *reinterpret_cast<u32x4*>(p.rem + (int64_t)at * 256 + l * 8) = *reinterpret_cast<const u32x4*>(buf + l * 8);
}
// One block per 256 ids finds its tokens; with `rows` it forms their rows too.
// That spares a launch, but one block forms the rows of a frequent id alone.
// Gradients of 512 x 8000 with d_w, rows here against a launch of their own:
// 128 tokens of uniform ids 38.6 / 40.2 us, of Zipf ids 40.9 / 41.9; 256 42.9 /
// 44.8 and 47.5 / 47.3; 1000 73.6 / 74.7 and 95.9 / 87.0.
constexpr int HEAD_REM_ROWS = 256;
__global__ __launch_bounds__(1024) void k_head_rem_list(HeadRem p, bool rows) {
  __shared__ __align__(16) uint16_t buf[32][256];
  __shared__ int wsum[2][16], wown[16];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int lo = blockIdx.x * 256, n = *p.count, total = n * p.top;
  if (blockIdx.x == 0)
    for (int i = tid; i < p.Hp / 8; i += 1024) *reinterpret_cast<u32x4*>(p.zero_row + i * 8) = (u32x4){0, 0, 0, 0};
  int below = 0, mine = 0;
#pragma unroll 8
  for (int e = tid; e < total; e += 1024) {
    const int id = p.eid[e];
    below += id >= 0 && id < lo;
    mine += (uint32_t)(id - lo) < 256u;
  }
#pragma unroll
  for (int x = 32; x > 0; x >>= 1) {
    below += shfl_xor(below, x);
    mine += shfl_xor(mine, x);
  }
  if (lane == 0) {
    wsum[0][wave] = below;
    wown[wave] = mine;
  }
  __syncthreads();
  int first = 0, places = 0;
#pragma unroll
  for (int w = 0; w < 16; ++w) {
    first += wsum[0][w];
    places += wown[w];
  }
  int k = 0;
  if (places > 0)
    for (int c0 = 0, b = 1; c0 < n; c0 += 1024, b ^= 1) {
      const int c = c0 + tid;
      bool on = false;
      if (c < n)
#pragma unroll 8
        for (int j = 0; j < p.top; ++j) on |= (uint32_t)(p.eid[(int64_t)c * p.top + j] - lo) < 256u;
      const uint64_t m = __ballot(on);
      if (lane == 0) wsum[b][wave] = __popcll(m);
      __syncthreads();  // the sums before are in the other half, so one barrier is enough
      int at = first + k + __popcll(m & ((1ull << lane) - 1));
#pragma unroll
      for (int w = 0; w < 16; ++w) {
        const int v = wsum[b][w];
        if (w < wave) at += v;
        k += v;
      }
      if (on) {
        p.list[at] = c;
        p.own[at] = blockIdx.x;
      }
    }
  if (tid == 0) p.tile[blockIdx.x] = make_int2(first, k);
  // the last block's end with the last place
  const int end = blockIdx.x + 1 < gridDim.x ? first + places : total;
  if (!rows) {
    for (int i = first + k + tid; i < end; i += 1024) p.own[i] = -1;
    return;
  }
  __syncthreads();
  for (int i = tid >> 5; i < k; i += 32) head_rem_row(p, first + i, p.list[first + i], lo, tid & 31, buf[tid >> 5]);
}
// The rows of all places, 32 lanes each.
__global__ __launch_bounds__(256) void k_head_rem_rows(HeadRem p) {
  __shared__ __align__(16) uint16_t buf[8][256];
  const int g = threadIdx.x >> 5, at = blockIdx.x * 8 + g;
  const int tile = at < *p.count * p.top ? p.own[at] : -1;
  if (tile >= 0) head_rem_row(p, at, p.list[at], tile * 256, threadIdx.x & 31, buf[g]);
}

// A row's entries as the u of its token takes them: ids (-1: none) and what
// rounding took off.
struct HeadEntries {
  int id[256];
  float rem[256];
};
// Row c's entries into LDS (a barrier has to follow).
MOE_DEV void head_load_entries(const HeadGemm& p, int c, HeadEntries& s) {
  const int j = threadIdx.x;
  if (j < p.top) {
    s.id[j] = p.eid[(int64_t)c * p.top + j];
    s.rem[j] = head_rem(p.ev[(int64_t)c * p.top + j]);
  }
}
// Adds entries [first, top) in steps of `step`, times their rows of W, 8 columns
// from col, to a and b; eight rows' loads in flight (four, and each iteration's
// ids read before them: 8 x 7168 x 2000 with 64 slots 75 us, 38 without entries).
MOE_DEV void head_add_entries(const HeadGemm& p, const HeadEntries& s, int first, int step, int col, f32x4& a,
                              f32x4& b) {
  for (int k = first; k < p.top; k += 8 * step) {
    u32x4 w[8];
    float x[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int at = k + j * step, v = at < p.top ? s.id[at] : -1;
      x[j] = v >= 0 ? s.rem[at] : 0.0f;
      w[j] = (u32x4){0, 0, 0, 0};
      if (v >= 0) w[j] = *reinterpret_cast<const u32x4*>(p.w + (int64_t)v * p.w_stride + col);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        a[2 * e] = fmaf(x[j], bf16_bits_to_f32(w[j][e] & 0xFFFFu), a[2 * e]);
        a[2 * e + 1] = fmaf(x[j], bf16_bits_to_f32(w[j][e] >> 16), a[2 * e + 1]);
        b[2 * e] = fmaf(x[j], bf16_bits_to_f32(w[j][e + 2] & 0xFFFFu), b[2 * e]);
        b[2 * e + 1] = fmaf(x[j], bf16_bits_to_f32(w[j][e + 2] >> 16), b[2 * e + 1]);
      }
  }
}

// d_h = u - r^2 h mean(h u), or u without a norm, u the sum of its slabs;
// zeros for tokens that do not count.  For H <= 2048, where u has the most
// slabs, and for H <= 8192 with at most two tokens per CU: one block per token,
// its NT threads in groups of P = the power of two at or above H / 8, each of
// which adds every (NT / P)-th slab; the groups' sums are added in order.  NT is
// 1024 where tokens are few and adding the groups is not the longer part.
// Bound by the slabs' reads: 12 us for 200 x 7168 in nine slabs, 1024 threads
// against 256: 3 x 1560 with 44 targets 21 -> 10.5 us, 107 x 4136 13.3 -> 9.1; with
// many targets by their rows of W: 1500 x 2048 with 33 39-50 us, 4-5 TB/s.
template <int NT>
__global__ __launch_bounds__(NT) void k_head_dh_narrow(HeadGemm p, const uint16_t* __restrict__ h, int64_t h_stride,
                                                        const int32_t* __restrict__ cidx, bool norm, int P,
                                                        uint16_t* __restrict__ dh) {
  __shared__ __align__(16) f32x4 sum[2][NT];
  __shared__ float part[NT / 64];
  __shared__ HeadEntries ent;
  const int t = blockIdx.x, c = cidx[t], H = p.H, np = H / 8, tid = threadIdx.x;
  const int i = tid & (P - 1), g = tid / P, groups = NT / P;
  uint16_t* o = dh + (int64_t)t * H + i * 8;
  if (c < 0) {
    if (g == 0 && i < np) *reinterpret_cast<u32x4*>(o) = (u32x4){0, 0, 0, 0};
    return;
  }
  if (p.exact) {
    head_load_entries(p, c, ent);
    __syncthreads();
  }
  const int splits = p.count[1];
  const int64_t slab = (int64_t)p.count[0] * H;
  const float* us = p.u + (int64_t)c * H + i * 8;
  u32x4 q = {0, 0, 0, 0};
  if (norm && i < np) q = *reinterpret_cast<const u32x4*>(h + (int64_t)t * h_stride + i * 8);
  f32x4 a = {0.0f, 0.0f, 0.0f, 0.0f}, b = a;
  if (i < np) {
    int s = g;
    for (; s + 3 * groups < splits; s += 4 * groups) {  // four slabs' loads in flight
      f32x4 x[4], y[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x[j] = *reinterpret_cast<const f32x4*>(us + (s + j * groups) * slab);
        y[j] = *reinterpret_cast<const f32x4*>(us + (s + j * groups) * slab + 4);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        a += x[j];
        b += y[j];
      }
    }
    for (; s < splits; s += groups) {
      a += *reinterpret_cast<const f32x4*>(us + s * slab);
      b += *reinterpret_cast<const f32x4*>(us + s * slab + 4);
    }
    if (p.exact) head_add_entries(p, ent, g, groups, i * 8, a, b);
  }
  if (groups > 1) {
    sum[0][tid] = a;
    sum[1][tid] = b;
    __syncthreads();
    for (int k = 1; k < groups; ++k) {
      a = k == 1 ? sum[0][i] + sum[0][P + i] : a + sum[0][k * P + i];
      b = k == 1 ? sum[1][i] + sum[1][P + i] : b + sum[1][k * P + i];
    }
  }
  float f = 0.0f;
  if (norm) {
    float dot = 0.0f;
    if (g == 0)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        dot = fmaf(j < 2 ? a[2 * j] : b[2 * j - 4], bf16_bits_to_f32(q[j] & 0xFFFFu), dot);
        dot = fmaf(j < 2 ? a[2 * j + 1] : b[2 * j - 3], bf16_bits_to_f32(q[j] >> 16), dot);
      }
    dot = hl_sum64(dot);
    if ((tid & 63) == 0) part[tid >> 6] = dot;
    __syncthreads();
    float all = 0.0f;
#pragma unroll
    for (int w = 0; w < NT / 64; ++w) all += part[w];
    f = p.r[c] * p.r[c] * all / (float)H;
  }
  if (g != 0 || i >= np) return;
  u32x4 x;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float lo = j < 2 ? a[2 * j] : b[2 * j - 4], hi = j < 2 ? a[2 * j + 1] : b[2 * j - 3];
    x[j] = bf16x2_bits(fmaf(-f, bf16_bits_to_f32(q[j] & 0xFFFFu), lo), fmaf(-f, bf16_bits_to_f32(q[j] >> 16), hi));
  }
  *reinterpret_cast<u32x4*>(o) = x;
}

// The same for wider h: one block per token, a thread keeps its
// NP pieces of 8 columns of u and h in registers between the sum and the
// result (NP = 4: H <= 8192, 16: any).
template <int NP>
__global__ __launch_bounds__(256) void k_head_dh(HeadGemm p, const uint16_t* __restrict__ h, int64_t h_stride,
                                                 const int32_t* __restrict__ cidx, bool norm,
                                                 uint16_t* __restrict__ dh) {
  __shared__ float part[4];
  __shared__ HeadEntries ent;
  const int t = blockIdx.x, c = cidx[t], H = p.H, np = H / 8;
  uint16_t* o = dh + (int64_t)t * H;
  if (c < 0) {
    for (int i = threadIdx.x; i < np; i += 256) *reinterpret_cast<u32x4*>(o + i * 8) = (u32x4){0, 0, 0, 0};
    return;
  }
  if (p.exact) {
    head_load_entries(p, c, ent);
    __syncthreads();
  }
  const int splits = p.count[1];
  const int64_t slab = (int64_t)p.count[0] * H;
  const float* ur = p.u + (int64_t)c * H;
  const uint16_t* hr = h + (int64_t)t * h_stride;
  f32x4 a[NP], b[NP];
  u32x4 q[NP];
#pragma unroll
  for (int k = 0; k < NP; ++k) {
    const int i = threadIdx.x + k * 256;
    a[k] = b[k] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
    q[k] = (u32x4){0, 0, 0, 0};
    if (i < np) {
      a[k] = *reinterpret_cast<const f32x4*>(ur + i * 8);
      b[k] = *reinterpret_cast<const f32x4*>(ur + i * 8 + 4);
      if (norm) q[k] = *reinterpret_cast<const u32x4*>(hr + i * 8);  // without a norm h is not read
    }
  }
#pragma unroll
  for (int k = 0; k < NP; ++k) {
    const int i = threadIdx.x + k * 256;
    if (i >= np) continue;
    const float* us = ur + i * 8;
    int s = 1;
    for (; s + 4 <= splits; s += 4) {  // four slabs' loads in flight
      f32x4 x[4], y[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x[j] = *reinterpret_cast<const f32x4*>(us + (s + j) * slab);
        y[j] = *reinterpret_cast<const f32x4*>(us + (s + j) * slab + 4);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        a[k] += x[j];
        b[k] += y[j];
      }
    }
    for (; s < splits; ++s) {
      a[k] += *reinterpret_cast<const f32x4*>(us + s * slab);
      b[k] += *reinterpret_cast<const f32x4*>(us + s * slab + 4);
    }
    if (p.exact) head_add_entries(p, ent, 0, 1, i * 8, a[k], b[k]);
  }
  float f = 0.0f;
  if (norm) {
    float dot = 0.0f;
#pragma unroll
    for (int k = 0; k < NP; ++k)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        dot = fmaf(j < 2 ? a[k][2 * j] : b[k][2 * j - 4], bf16_bits_to_f32(q[k][j] & 0xFFFFu), dot);
        dot = fmaf(j < 2 ? a[k][2 * j + 1] : b[k][2 * j - 3], bf16_bits_to_f32(q[k][j] >> 16), dot);
      }
    dot = hl_sum64(dot);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = dot;
    __syncthreads();
    f = p.r[c] * p.r[c] * ((part[0] + part[1]) + (part[2] + part[3])) / (float)H;
  }
#pragma unroll
  for (int k = 0; k < NP; ++k) {
    const int i = threadIdx.x + k * 256;
    u32x4 x;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float lo = j < 2 ? a[k][2 * j] : b[k][2 * j - 4], hi = j < 2 ? a[k][2 * j + 1] : b[k][2 * j - 3];
      x[j] = bf16x2_bits(fmaf(-f, bf16_bits_to_f32(q[k][j] & 0xFFFFu), lo),
                         fmaf(-f, bf16_bits_to_f32(q[k][j] >> 16), hi));
    }
    if (i < np) *reinterpret_cast<u32x4*>(o + i * 8) = x;
  }
}

namespace {
inline int cdiv(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }
// The tiles, and what each costs: microseconds per K step of 64 with every CU
// busy, and per tile besides (start, epilogue), measured from T = 16..1500 over
// five heads of 512 x 8000 to 7168 x 32000 and 2048 x 128000.
using HeadBig = HeadTile<256, 256, 2, 4, 2, 2>;
struct HeadShape {
  int bm, bn, per_cu;  // per_cu: workgroups a CU holds
  float step, over;
};
constexpr HeadShape kHeadShapes[] = {
    {256, 256, 1, 1.36f, 7.0f}, {256, 128, 1, 0.78f, 5.0f}, {128, 256, 1, 0.84f, 5.0f},
    {128, 128, 1, 0.54f, 4.0f}, {64, 128, 2, 0.60f, 3.5f}, {192, 128, 1, 0.72f, 4.5f},
};
constexpr int kHeadShapeCount = sizeof(kHeadShapes) / sizeof(kHeadShapes[0]);
template <typename F>
void head_dispatch(int shape, F f) {
  switch (shape) {
    case 0: f(HeadBig()); break;
    case 1: f(HeadTile<256, 128, 4, 2, 3, 2>()); break;
    case 2: f(HeadTile<128, 256, 2, 4, 3, 2>()); break;
    case 3: f(HeadTile<128, 128, 2, 4, 4, 2>()); break;
    case 5: f(HeadTile<192, 128, 4, 2, 3, 2>()); break;
    default: f(HeadTile<64, 128, 2, 2, 3, 2>()); break;
  }
}
// Microseconds of a product of M rows, N columns and K, its K split `splits`
// ways: rounds of workgroups, each step of which takes the longer of reading its
// rows of W at 5 MB per microsecond (`width`: times more for narrow tiles of a
// product that reads W in row pieces) and its MFMAs with a third of that.
float head_cost(const HeadShape& t, int M, int N, int K, int splits, int cus, float width) {
  const int64_t nm = (M + t.bm - 1) / t.bm, tiles = nm * ((N + t.bn - 1) / t.bn) * splits;
  const int64_t slots = (int64_t)cus * t.per_cu, rounds = (tiles + slots - 1) / slots;
  const int64_t steps = ((K + 63) / 64 + splits - 1) / splits, act = tiles < slots ? tiles : slots;
  const float mfma = act > cus || t.per_cu == 1 ? t.step : 0.6f * t.step;  // alone on its CU
  const float mem = (float)act / (float)nm * (float)(t.bn * 128) / 5e6f * (t.bn < 256 ? width : 1.0f);
  const float both = mfma + 0.35f * mem;
  return (float)rounds * ((float)steps * (both > mem ? both : mem) + t.over);
}
// The cheapest tile for h W^T.  Within 0.3% of the best tile of each of those
// shapes on average, 10% at most (always 256 x 256: 1.6 times the best at 16
// rows of 512 x 8000 and 1.7 at 64 rows of 7168 x 32000; always 64 x 128: 2
// times at 1500 rows).  The 192-row tile is for 129 to 192 rows and for such
// remainders: 190 rows of 7168 x 32000 129 -> 115 us (256 x 128), gradient of
// 180 rows of 2048 x 32000 83 -> 70.
// With K split (splits > 1) the slabs are written and read at about 8 MB per
// microsecond, the forward reads a row of them with one block and the backward
// has a launch more.  Against unsplit: forward of 2 x 6488 x 1118 45 -> 19 us,
// 42 x 5536 x 3619 39 -> 22, 256 x 4096 x 4096 30 -> 22; gradient of the second
// 55 -> 38; the same from 8000 columns at 64 rows of 2048 or 300 of 3264.
int head_tile_logits(int T, int H, int V, bool bwd, int cus, int* splits) {
  int best = 0;
  float least = -1.0f;
  for (int i = 0; i < kHeadShapeCount; ++i)
    for (int s = 1; s <= 16 && (s == 1 || (s <= (H + 63) / 64 && (int64_t)T * ((V + 3) & ~3) * s <= (16 << 20))); ++s) {
      float c = head_cost(kHeadShapes[i], T, V, H, s, cus, 1.0f);
      if (i == 0 && s == 1) {  // halves in the last round (head_tile_tail): those of shape 2
        const int tiles = cdiv(T, 256) * cdiv(V, 256), last = tiles % cus;
        if (last > 0 && last * 2 <= cus) c -= (float)((H + 63) / 64) * 0.52f + 2.0f;
      }
      if (s > 1) {
        const float bytes = (float)T * (float)V * (float)s * 8.0f;
        c += bytes / 8e6f + (bwd ? 6.0f : 1.0f + (float)V * (float)s * 2.5e-4f);
      }
      if (least < 0.0f || c < least) {
        least = c;
        best = i;
        *splits = s;
      }
    }
  return best;
}
// Most workgroups of the G W product: room for a second round's splits.
int head_dz_max(int T, int H, int bm, int bn) {
  const int64_t tiles = (int64_t)((T + bm - 1) / bm) * ((H + bn - 1) / bn);
  return (int)(tiles > 2048 ? tiles : tiles * 2 > 1024 ? tiles * 2 : 1024);
}
// The cheapest tile for G W with its best split (2% from the best on average).
int head_tile_dz(int T, int H, int K, int cus) {
  int best = 0;
  float least = -1.0f;
  for (int i = 0; i < kHeadShapeCount; ++i) {
    const HeadShape& t = kHeadShapes[i];
    const int64_t tiles = (int64_t)((T + t.bm - 1) / t.bm) * ((H + t.bn - 1) / t.bn);
    const int64_t most = head_dz_max(T, H, t.bm, t.bn);
    for (int s = 1; s <= HEAD_SPLITS && (s == 1 || (tiles * s <= most && s <= (K + 63) / 64)); ++s) {
      const float c = head_cost(t, T, H, K, s, cus, 1.25f) + (float)s * ((float)T * (float)H * (8.0f / 5e6f) + 0.125f);
      if (least < 0.0f || c < least) {
        least = c;
        best = i;
      }
    }
  }
  return best;
}
// Workgroups for nm x nn tiles (a multiple of the 8 XCDs); with `halves` of a
// last round besides.
int head_grid(int64_t nm, int64_t nn, int halves = 0) { return cdiv(nm * nn, 8) * 8 + cdiv(halves, 8) * 8; }
int head_cus() {
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess) dev = 0;
  return device_cus(dev);
}
}  // namespace

HeadPlan head_plan(int T, int H, int V, int top, bool distill, bool bwd) {
  HeadPlan p{};
  p.T = T;
  p.H = H;
  p.V = V;
  p.top = top;
  p.distill = distill;
  p.bwd = bwd;
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o = (o + bytes + 255) / 256 * 256;
    return at;
  };
  p.Hp = (H + 63) / 64 * 64;
  const int cus = head_cus();
  p.tile_l = head_tile_logits(T, H, V, bwd, cus, &p.psplits);
  p.bm = kHeadShapes[p.tile_l].bm;
  const size_t t = (size_t)T, r256 = (t + 255) / 256 * 256, r192 = (t + 191) / 192 * 192;
  const size_t rows = r256 > r192 ? r256 : r192;  // whole tiles of any shape
  if (bwd) {
    // columns of G per piece: 512 MB of G, at least 256 columns (256 MB, which
    // the last-level cache would hold: 2% slower at 8192 x 7168 x 32000 and 14%
    // at 8192 x 512 x 128000, where every piece reads and writes u again)
    const int64_t most = T > 0 ? ((int64_t)256 << 20) / (int64_t)rows / 256 * 256 : V;
    p.npieces = cdiv(V, most > 256 ? most : 256);
    p.piece = cdiv(cdiv(V, p.npieces), 256) * 256;
    p.npieces = cdiv(V, p.piece);
    if (p.npieces > 1) p.psplits = 1;
    p.tile_z = head_tile_dz(T, H, p.piece < V ? p.piece : V, cus);
    p.dz_max = head_dz_max(T, H, kHeadShapes[p.tile_z].bm, kHeadShapes[p.tile_z].bn);
  }
  p.r = take(rows * 4);
  p.info = take(rows * sizeof(HeadRow));
  // What rounding takes off G's entries at the target's ids is always added for
  // cross entropy (with d_w one place of 512 bytes per token).  A teacher's ids
  // cost a row of W each for u, and their tokens K steps of d_w: taken while they
  // are few, altogether or for the vocabulary.  Taken against not, us: 64 x 1024 x
  // 1000 with 16 ids 28 / 27 frozen, 43 / 33 with d_w; 1500 x 2048 x 50257 with 33
  // 549 / 524 and 907 / 798; 200 x 7168 x 32000 with 64 270 / 246 and 534 / 437.
  // Past the rule 4096 x 7168 x 32000 with 64 would be 3215 / 2727 and 5200 /
  // 3979, with 128 3737 / 2752 and 6151 / 4022: there the entries stay rounded,
  // which leaves 1.4 times the results' own rounding instead of 1.0.
  const int64_t entries = (int64_t)T * top;
  p.exact = bwd && (!distill || (int64_t)top * 900 <= V || entries <= (V > 2048 ? V / 2 : 1024));
  p.exact_w = p.exact && entries <= (1 << 20);
  p.eid = take(p.exact ? t * top * 4 : 0);
  p.ev = take(p.exact ? t * top * 4 : 0);
  p.rtile = take(p.exact_w ? (size_t)cdiv(V, 256) * 8 : 0);
  p.rlist = take(p.exact_w ? (t * top + 64) * 4 : 0);
  p.rown = take(p.exact_w ? t * top * 4 : 0);
  p.rem = take(p.exact_w ? t * top * 512 : 0);
  p.flag = take(distill ? t : 0);
  p.rows = take(t * 4);
  p.cidx = take(t * 4);
  p.count = take(8);
  p.hc = take((rows + p.exact_w) * p.Hp * 2);  // a row of zeros last
  p.zero_row = (int)rows;
  p.lq = take(distill ? t * top * 4 : 0);
  p.lp = take(p.psplits > 1 ? t * ((V + 3) / 4 * 4) * p.psplits * 4 : 0);
  if (!bwd) {
    p.zt = take(t * top * 4);
    p.stats = take(t * cdiv(V, kHeadShapes[p.tile_l].bn) * 8);
  } else {
    // slabs of u: the splits of a tile times the tiles stay below dz_max (or are 1)
    size_t u = (size_t)p.dz_max * kHeadShapes[p.tile_z].bm * kHeadShapes[p.tile_z].bn;
    if (u > t * H * HEAD_SPLITS) u = t * H * HEAD_SPLITS;
    if (u < t * H) u = t * H;
    p.u = take(u * 4);
    p.g = take(rows * p.piece * 2);
  }
  p.total = o;
  // a launch has fewer than 2^32 threads in a dimension
  if (!bwd && p.psplits == 1)
    head_dispatch(p.tile_l, [&](auto c) {
      using C = decltype(c);
      const int64_t blocks = (int64_t)((T + C::BM - 1) / C::BM) * ((V + C::BN - 1) / C::BN) + 2 * cus + 16;
      if (blocks * C::NT >= (1ll << 32)) p.total = 0;
    });
  return p;
}

static HeadGemm head_common(const HeadPlan& p, const HeadArgs& a, hipStream_t s) {
  char* ws = a.ws;
  uint8_t* flag = p.distill && p.T > HEAD_SAME ? reinterpret_cast<uint8_t*>(ws + p.flag) : nullptr;
  HeadRowsArgs q{};
  q.h = a.h;
  q.h_stride = a.h_stride;
  q.T = p.T;
  q.H = p.H;
  q.Hp = p.Hp;
  q.V = p.V;
  q.top = p.top;
  q.bm = p.bm;
  q.eps = a.eps;
  q.scale = a.scale;
  q.tscale = a.teacher_scale;
  q.ids = a.ids;
  q.tlogits = a.tlogits;
  q.flag = flag;
  if (p.bwd) {
    q.loss = p.distill ? nullptr : a.loss;
    q.lse = a.lse;
    q.dloss = a.dloss;
  }
  const HeadShape& z = kHeadShapes[p.tile_z];
  q.split = HeadSplit{p.H, p.bwd ? (p.piece < p.V ? p.piece : p.V) : 64, z.bm, z.bn, head_cus() * z.per_cu, p.dz_max,
                      z.step, z.over};
  q.rows = reinterpret_cast<int32_t*>(ws + p.rows);
  q.cidx = reinterpret_cast<int32_t*>(ws + p.cidx);
  q.count = reinterpret_cast<int32_t*>(ws + p.count);
  uint16_t* hc = q.hc = reinterpret_cast<uint16_t*>(ws + p.hc);
  q.r = reinterpret_cast<float*>(ws + p.r);
  q.info = reinterpret_cast<HeadRow*>(ws + p.info);
  q.eid = reinterpret_cast<int32_t*>(ws + p.eid);
  q.ev = reinterpret_cast<float*>(ws + p.ev);
  q.lq = reinterpret_cast<float*>(ws + p.lq);
  if (flag != nullptr)
    hipLaunchKernelGGL(k_head_teacher, dim3(cdiv(p.T, 4)), dim3(256), 0, s, a.ids, a.tlogits, p.T, p.V, p.top,
                       a.teacher_scale, q.lq, flag);
  const dim3 grid(cdiv(p.T, p.bm) * p.bm);
  if (p.T <= HEAD_SAME) {
    hipLaunchKernelGGL(k_head_gather<HR_SAME>, grid, dim3(256), 0, s, q);
  } else if (p.T <= HEAD_FEW) {
    hipLaunchKernelGGL(k_head_gather<HR_FEW>, grid, dim3(256), 0, s, q);
  } else {
    hipLaunchKernelGGL(k_head_compact, dim3(1), dim3(1024), 0, s, flag, a.ids, p.T, p.V, q.split, q.rows, q.cidx,
                       q.count);
    hipLaunchKernelGGL(k_head_gather<HR_LIST>, grid, dim3(256), 0, s, q);
  }
  HeadGemm g{};
  g.hc = hc;
  g.w = a.w;
  g.w_stride = a.w_stride;
  g.H = p.H;
  g.Hp = p.Hp;
  g.V = p.V;
  g.top = p.top;
  g.slots = head_cus();
  g.rows = q.rows;
  g.count = q.count;
  g.r = q.r;
  g.eid = q.eid;
  g.ev = p.distill && !p.exact ? nullptr : q.ev;
  g.exact = p.exact;
  g.info = q.info;
  g.distill = p.distill;
  g.scale = a.scale;
  g.ids = a.ids;
  g.dw = a.dw;
  return g;
}

// The partial products' launch.
static void launch_head_part(const HeadPlan& p, const HeadGemm& g, hipStream_t s) {
  head_dispatch(p.tile_l, [&](auto c) {
    using C = decltype(c);
    hipLaunchKernelGGL(k_head_part<C>, dim3(head_grid((int64_t)cdiv(p.T, C::BM) * p.psplits, cdiv(p.V, C::BN))),
                       dim3(C::NT), 0, s, g);
  });
}

void launch_head_loss(const HeadPlan& p, const HeadArgs& a, hipStream_t s) {
  const bool part = p.psplits > 1;
  const bool direct = p.H % 64 == 0 && (part ? p.T <= HEAD_SAME : p.T <= p.bm && p.tile_l >= 2 && p.tile_l <= 4);
  HeadGemm g = direct ? HeadGemm{} : head_common(p, a, s);
  g.h = a.h;
  g.h_stride = a.h_stride;
  g.T = p.T;
  g.eps = a.eps;
  g.w = a.w;
  g.w_stride = a.w_stride;
  g.H = p.H;
  g.Hp = p.Hp;
  g.V = p.V;
  g.top = p.top;
  g.scale = a.scale;
  g.ids = a.ids;
  g.distill = p.distill;
  g.stats = reinterpret_cast<float*>(a.ws + p.stats);
  g.zt = reinterpret_cast<float*>(a.ws + p.zt);
  HeadFinish f{g.stats,
               g.zt,
               reinterpret_cast<const int32_t*>(a.ws + p.cidx),
               a.ids,
               reinterpret_cast<const float*>(a.ws + p.lq),
               a.tlogits,
               a.teacher_scale,
               p.T,
               p.V,
               cdiv(p.V, kHeadShapes[p.tile_l].bn),
               p.top,
               a.loss,
               a.lse,
               a.logp};
  if (part) {
    g.lp = reinterpret_cast<float*>(a.ws + p.lp);
    g.psplits = p.psplits;
    g.Vp = (p.V + 3) / 4 * 4;
    g.direct = direct;
    launch_head_part(p, g, s);
    hipLaunchKernelGGL(k_head_part_finish, dim3(p.T), dim3(256), 0, s, g, f);
    return;
  }
  if (direct) {
    head_dispatch(p.tile_l, [&](auto c) {
      using C = decltype(c);
      if constexpr (C::NT == 4 * C::BM)
        hipLaunchKernelGGL((k_head_stats<C, true>), dim3(head_grid(1, f.nvb)), dim3(C::NT), 0, s, g);
    });
    hipLaunchKernelGGL(k_head_finish<true>, dim3(cdiv(p.T, 4)), dim3(256), 0, s, f);
    return;
  }
  head_dispatch(p.tile_l, [&](auto c) {
    using C = decltype(c);
    hipLaunchKernelGGL((k_head_stats<C, false>), dim3(head_grid(cdiv(p.T, C::BM), f.nvb, C::FIVE ? g.slots : 0)),
                       dim3(C::NT), 0, s, g);
  });
  hipLaunchKernelGGL(k_head_finish<false>, dim3(cdiv(p.T, 4)), dim3(256), 0, s, f);
}

void launch_head_loss_bwd(const HeadPlan& p, const HeadArgs& a, hipStream_t s) {
  HeadGemm g = head_common(p, a, s);
  g.u = reinterpret_cast<float*>(a.ws + p.u);
  g.g = reinterpret_cast<uint16_t*>(a.ws + p.g);
  g.lp = reinterpret_cast<float*>(a.ws + p.lp);
  g.T = p.T;
  g.psplits = p.psplits;
  g.Vp = (p.V + 3) / 4 * 4;
  g.piece = p.piece;
  const int ndz = head_grid(p.dz_max, 1), ndw = head_grid(cdiv(p.piece, HeadBig::BM), cdiv(p.H, HeadBig::BN));
  for (int i = 0; i < p.npieces; ++i) {
    g.v0 = i * p.piece;
    if (p.psplits > 1) {
      launch_head_part(p, g, s);
      hipLaunchKernelGGL(k_head_part_grad, dim3(cdiv(p.T, p.bm) * p.bm, cdiv(p.piece, 2048)), dim3(256), 0, s, g, p.bm);
    } else {
      head_dispatch(p.tile_l, [&](auto c) {
        using C = decltype(c);
        hipLaunchKernelGGL(k_head_grad<C>, dim3(head_grid(cdiv(p.T, C::BM), p.piece / C::BN, C::FIVE ? g.slots : 0)),
                           dim3(C::NT), 0, s, g);
      });
    }
    if (p.distill)
      hipLaunchKernelGGL(k_head_targets, dim3(cdiv(p.T, 4)), dim3(256), 0, s, g.rows, g.count, a.ids,
                         reinterpret_cast<const float*>(a.ws + p.lq), a.logp, g.info, p.top, g.v0, p.piece, g.g, g.eid,
                         g.ev);
    if (a.dw != nullptr && p.exact_w && i == 0) {
      HeadRem r{g.eid, g.ev, g.count, p.top};
      r.tile = reinterpret_cast<int2*>(a.ws + p.rtile);
      r.list = reinterpret_cast<int32_t*>(a.ws + p.rlist);
      r.own = reinterpret_cast<int32_t*>(a.ws + p.rown);
      r.rem = reinterpret_cast<uint16_t*>(a.ws + p.rem);
      r.zero_row = const_cast<uint16_t*>(g.hc) + (int64_t)p.zero_row * p.Hp;
      r.Hp = p.Hp;
      g.rtile = r.tile;
      g.rlist = r.list;
      g.rem = r.rem;
      g.zero_row = p.zero_row;
      hipLaunchKernelGGL(k_head_rem_list, dim3(cdiv(p.V, 256)), dim3(1024), 0, s, r, p.T <= HEAD_REM_ROWS);
      if (p.T > HEAD_REM_ROWS)
        hipLaunchKernelGGL(k_head_rem_rows, dim3(cdiv((int64_t)p.T * p.top, 8)), dim3(256), 0, s, r);
    }
    if (a.dw != nullptr && p.tile_z == 0) {
      hipLaunchKernelGGL(k_head_dz_dw<HeadBig>, dim3(ndz + ndw), dim3(HeadBig::NT), 0, s, g, ndz);
      continue;
    }
    head_dispatch(p.tile_z, [&](auto c) {
      using C = decltype(c);
      hipLaunchKernelGGL(k_head_dz<C>, dim3(ndz), dim3(C::NT), 0, s, g);
    });
    if (a.dw != nullptr) hipLaunchKernelGGL(k_head_dw<HeadBig>, dim3(ndw), dim3(HeadBig::NT), 0, s, g);
  }
  const int32_t* cidx = reinterpret_cast<const int32_t*>(a.ws + p.cidx);
  int P = 8;
  while (P < p.H / 8) P *= 2;
  if (p.H > 512 && p.H <= 8192 && p.T <= 2 * head_cus()) {
    hipLaunchKernelGGL(k_head_dh_narrow<1024>, dim3(p.T), dim3(1024), 0, s, g, a.h, a.h_stride, cidx, a.eps > 0.0f, P,
                       a.dh);
  } else if (p.H <= 2048) {
    hipLaunchKernelGGL(k_head_dh_narrow<256>, dim3(p.T), dim3(256), 0, s, g, a.h, a.h_stride, cidx, a.eps > 0.0f, P, a.dh);
  } else if (p.H <= 8192)
    hipLaunchKernelGGL(k_head_dh<4>, dim3(p.T), dim3(256), 0, s, g, a.h, a.h_stride, cidx, a.eps > 0.0f, a.dh);
  else
    hipLaunchKernelGGL(k_head_dh<16>, dim3(p.T), dim3(256), 0, s, g, a.h, a.h_stride, cidx, a.eps > 0.0f, a.dh);
}

}  // namespace moe
