// The gate: scores of the router's logits, a choice of experts with a balance
// bias and groups, and the gradient of the chosen weights.
//
// Per token, with an expert "out" where its logit or its bias is -infinity or
// NaN (s = 0, chosen only behind every expert that is in):
//   s_e = 1 / (1 + exp(-l_e))  or  softmax over the experts that are in
//   c_e = s_e + b_e            what the choice goes by
//   group value = the largest c of the group, or the sum of its two largest
//   chosen: the k largest c within the top_groups best groups; ties go to the
//   lowest group and the lowest id
//   w_j = scale s_j, or scale s_j / sum_i s_i
#include "common.h"
#include "kernels.h"

namespace moe {

namespace {

// Orders one wave's LDS accesses before and after it (no other wave waits).
MOE_DEV void gate_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
}

MOE_DEV bool gate_out(float v) { return v != v || v == -INFINITY; }

template <int LPT>
MOE_DEV float gate_max(float v) {
#pragma unroll
  for (int x = 1; x < LPT; x <<= 1) v = fmaxf(v, __shfl_xor(v, x, 64));
  return v;
}
template <int LPT, typename T>
MOE_DEV T gate_sum(T v) {
#pragma unroll
  for (int x = 1; x < LPT; x <<= 1) v += __shfl_xor(v, x, 64);
  return v;
}
template <int LPT>
MOE_DEV uint64_t gate_max_u64(uint64_t v) {
#pragma unroll
  for (int x = 1; x < LPT; x <<= 1) {
    const uint64_t o = __shfl_xor((unsigned long long)v, x, 64);
    v = o > v ? o : v;
  }
  return v;
}

// Order of the choice in one number: the 54 upper bits of c in 64 bits, made
// monotone (values closer than 2^-42 of their size count as equal), and the id
// below them, the lowest the largest.  1 << 10 | id: an expert that is out; 0:
// not to be chosen.
MOE_DEV uint64_t gate_key(double c, bool out, int e) {
  uint64_t b = __double_as_longlong(c + 0.0);
  b = (b >> 63) ? ~b : (b | 0x8000000000000000ull);
  return (out ? 1024ull : b & ~1023ull) | (uint64_t)(1023 - e);
}

}  // namespace

// One token by the whole wave, lane r with the experts r, r + 64, ...: SLOTS, E <=
// 64 SLOTS.  Scores are formed in 64 bits, since two neighbours' order decides
// which expert runs.  lds: E + GATE_MAX_GROUPS numbers.
template <int SLOTS>
MOE_DEV void gate_token(const GateArgs& p, int t, double* sc) {
  const int r = threadIdx.x & 63, E = p.E;
  const float* row = p.logits + (int64_t)t * E;
  double* gv = sc + E;
  float l[SLOTS], b[SLOTS];
  bool out[SLOTS];
#pragma unroll
  for (int i = 0; i < SLOTS; ++i) {
    const int e = r + 64 * i;
    l[i] = e < E ? row[e] : -INFINITY;
    b[i] = e < E && p.bias ? p.bias[e] : 0.0f;
    out[i] = gate_out(l[i]) || gate_out(b[i]);
  }
  double s[SLOTS];
  if (p.sigmoid) {
#pragma unroll
    for (int i = 0; i < SLOTS; ++i) s[i] = out[i] ? 0.0 : 1.0 / (1.0 + exp(-(double)l[i]));
  } else {
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < SLOTS; ++i) m = out[i] ? m : fmaxf(m, l[i]);
    m = gate_max<64>(m);
    double z = 0.0;
#pragma unroll
    for (int i = 0; i < SLOTS; ++i) {
      s[i] = out[i] ? 0.0 : l[i] == m ? 1.0 : exp((double)l[i] - (double)m);
      z += s[i];
    }
    z = gate_sum<64>(z);
#pragma unroll
    for (int i = 0; i < SLOTS; ++i) s[i] = z > 0.0 ? s[i] / z : 0.0;
  }
  uint64_t key[SLOTS];
#pragma unroll
  for (int i = 0; i < SLOTS; ++i) {
    const int e = r + 64 * i;
    const double c = s[i] + (double)b[i];
    key[i] = e < E ? gate_key(c, out[i], e) : 0ull;
    if (p.groups > 1 && e < E) sc[e] = out[i] ? -INFINITY : c;
  }
  if (p.groups > 1) {
    gate_sync();
    const int per = E / p.groups;
    double v = -INFINITY;
    if (r < p.groups) {
      double a = -INFINITY, a2 = -INFINITY;
#pragma unroll 4
      for (int i = 0; i < per; ++i) {
        const double x = sc[r * per + i];
        a2 = fmax(a2, fmin(a, x));
        a = fmax(a, x);
      }
      v = p.top2 && a2 > -INFINITY ? a + a2 : a;
      gv[r] = v;
    }
    gate_sync();
    int rank = 0;
    for (int j = 0; j < p.groups; ++j) rank += (gv[j] > v || (gv[j] == v && j < r)) ? 1 : 0;
    const uint64_t chosen = __ballot(r < p.groups && rank < p.top_groups);  // bit: group
#pragma unroll
    for (int i = 0; i < SLOTS; ++i) {
      const int e = r + 64 * i;
      if (e < E && !((chosen >> (e / per)) & 1)) key[i] = 0;
    }
    gate_sync();
  }
#pragma unroll
  for (int i = 0; i < SLOTS; ++i)
    if (r + 64 * i < E) sc[r + 64 * i] = s[i];
  int mine = 0;
  for (int j = 0; j < p.k; ++j) {
    uint64_t best = 0;
#pragma unroll
    for (int i = 0; i < SLOTS; ++i) best = key[i] > best ? key[i] : best;
    best = gate_max_u64<64>(best);
#pragma unroll
    for (int i = 0; i < SLOTS; ++i) key[i] = key[i] == best ? 0ull : key[i];
    if (r == j) mine = 1023 - (int)(best & 1023u);
  }
  gate_sync();
  const double sj = r < p.k ? sc[mine] : 0.0;
  const double tot = p.renorm ? gate_sum<16>(sj) : 1.0;
  if (r < p.k) {
    p.ids[(int64_t)t * p.k + r] = mine;
    p.w[(int64_t)t * p.k + r] = tot > 0.0 ? (float)((double)p.scale * sj / tot) : 0.0f;
  }
  gate_sync();  // the next token's
}

// The groups that k_gate does not take: other numbers than 1, 2, 4, 8 and 16, and
// any of an E that is not a multiple of 16.  VALU-bound: 64-bit exponentials, a 64-bit
// maximum over the wave for every choice, and a group's value by one lane, one expert
// after the other: 16384 x 264 in 8 groups 44 us, 380 in 4 53, 384 in 6 51 (256 in 8
// by k_gate on such logits 17).
template <int SLOTS>
__global__ __launch_bounds__(64) void k_gate_wave(GateArgs p) {
  extern __shared__ __align__(16) double gate_lds[];
  gate_token<SLOTS>(p, blockIdx.x, gate_lds);
}

MOE_DEV uint32_t gate_max16(uint32_t v) {
  v = max(v, (uint32_t)dpp_i32<0xB1>((int)v));   // quad_perm [1,0,3,2]
  v = max(v, (uint32_t)dpp_i32<0x4E>((int)v));   // quad_perm [2,3,0,1]
  v = max(v, (uint32_t)dpp_i32<0x124>((int)v));  // row_ror:4
  return max(v, (uint32_t)dpp_i32<0x128>((int)v));
}
template <int CTRL>
MOE_DEV float gate_dpp(float v) { return __int_as_float(dpp_i32<CTRL>(__float_as_int(v))); }
MOE_DEV float gate_max16(float v) {
  v = fmaxf(v, gate_dpp<0xB1>(v));
  v = fmaxf(v, gate_dpp<0x4E>(v));
  v = fmaxf(v, gate_dpp<0x124>(v));
  return fmaxf(v, gate_dpp<0x128>(v));
}
MOE_DEV float gate_sum16(float v) {
  v += gate_dpp<0xB1>(v);
  v += gate_dpp<0x4E>(v);
  v += gate_dpp<0x124>(v);
  return v + gate_dpp<0x128>(v);
}
// exp(x), x <= 0, to about an ulp: the product with log2 e in two parts.
MOE_DEV float gate_exp(float x) {
  x = fmaxf(x, -200.0f);  // 0 from -104 on
  const float t = x * 1.44269504f, lo = fmaf(x, 1.44269504f, -t) + x * 1.92596299e-8f;
  return fmaf(__builtin_amdgcn_exp2f(t) * lo, 0.693147181f, __builtin_amdgcn_exp2f(t));
}
// The two largest of two pairs.
template <int CTRL>
MOE_DEV void gate_top2(float& a, float& a2) {
  const float b = gate_dpp<CTRL>(a), b2 = gate_dpp<CTRL>(a2);
  a2 = fmaxf(fminf(a, b), fmaxf(a2, b2));
  a = fmaxf(a, b);
}

// The four largest of a lane's keys in falling order, of those below `last`.
template <int SL>
MOE_DEV void gate_largest4(const uint32_t (&key)[SL], uint32_t last, uint32_t (&t)[4]) {
#pragma unroll
  for (int q = 0; q < 4; ++q) t[q] = 0;
#pragma unroll
  for (int i = 0; i < SL; ++i) {
    uint32_t x = key[i] < last ? key[i] : 0u;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint32_t m = max(t[q], x);
      x = min(t[q], x);
      t[q] = m;
    }
  }
}

// Softmax's sum over a token's experts in 64 bits, for each of its 16 lanes n of them
// from e0 on; m: the largest logit, which is one of them.  exp(x) = 2^w exp(y), |y| <=
// ln 2 / 2, by the polynomial of degree 9 through exp at the Chebyshev points (0 and 1 as
// its first coefficients' errors): 3e-14.  Experts that are out count exp(-80), which is
// not seen beside the largest term's 1.  The row comes from the cache once more: held
// over the choice it would cost every gate registers (16384 x 1024 sigmoid 62 us, 47 so).
// VALU-bound, 15 operations of 64 bits per expert: 1.9 us of 12.9 at 5001 x 384, 15 of
// 63 at 16384 x 1024.
template <bool ALIGNED>
MOE_DEV double gate_sum64(const float* row, const float* bias, int e0, int n, float m) {
  // in scalar registers: as literals each would be moved to where the sum is formed
  double k[8] = {2.763265575933203e-06, 2.488447635159146e-05, 1.984119061583585e-04, 1.3888801714761622e-03,
                 8.333333367332009e-03, 4.1666667040776456e-02, 0.16666666666615607,  0.4999999999943814};
#pragma unroll
  for (int j = 0; j < 8; ++j) asm("" : "+s"(k[j]));
  const float low = m - 80.0f;
  const double md = m, whole = 6755399441055744.0;  // 1.5 2^52: a sum with it is rounded to an integer, its lower word
  double z = 0.0;
#pragma unroll 1
  for (int i = 0; i < n; i += 4) {
    float l[4];
    if constexpr (ALIGNED) {
      const f32x4 v = *reinterpret_cast<const f32x4*>(row + e0 + i);
#pragma unroll
      for (int q = 0; q < 4; ++q) l[q] = v[q];
      if (bias) {
        const f32x4 b = *reinterpret_cast<const f32x4*>(bias + e0 + i);
#pragma unroll
        for (int q = 0; q < 4; ++q) l[q] = gate_out(b[q]) ? -INFINITY : l[q];
      }
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        l[q] = i + q < n && !(bias && gate_out(bias[e0 + i + q])) ? row[e0 + i + q] : -INFINITY;
    }
    double y[4], w[4], e[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const double x = (double)fmaxf(l[q], low) - md;  // fmaxf: NaN as well
      w[q] = fma(x, 1.4426950408889634, whole);
      y[q] = fma(w[q] - whole, -0.69314718055994531, x);
      e[q] = k[0];
    }
#pragma unroll
    for (int j = 1; j < 10; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) e[q] = fma(e[q], y[q], j < 8 ? k[j] : 1.0);
#pragma unroll
    for (int q = 0; q < 4; ++q) z += __hiloint2double(__double2hiint(e[q]) + (__double2loint(w[q]) << 20), __double2loint(e[q]));
  }
  z = gate_sum<16>(z);
  if (fabsf(m) >= 0x1p30f) {  // infinite, or the next logit below is 64 off: as many terms of 1
    z = 0.0;
    for (int i = 0; i < n; ++i) z += row[e0 + i] == m && !(bias && gate_out(bias[e0 + i])) ? 1.0 : 0.0;
    z = gate_sum<16>(z);
  }
  return z;
}

// Four tokens per wave, 16 lanes each, lane r with the experts from r ceil(E / 16)
// on (SL at most); 1, 2, 4, 8 or 16 groups, with groups E a multiple of 16.
//
// The choice is made on fp32 scores as 22-bit steps below the largest c, down to
// what two experts of every lane reach; a lane keeps its four largest keys sorted,
// and a round takes the largest of 16 heads.  Where two values that the choice
// depends on lie within what fp32 may be off (about 1 token in 1000 of a trained
// router's), or it reaches an expert below the steps or out, the token is done
// again in 64 bits.  16384 x 256 in 8 groups: 31 us with 64-bit scores for all, 22
// with rounds over all keys, 13.5 now; 16 MB are 3.7 at a copy's rate, the rest is the
// choice (1070 VALU instructions per wave of four tokens).
template <int SL, int SLOTS, bool ALIGNED>
__global__ __launch_bounds__(64) void k_gate(GateArgs p) {
  extern __shared__ __align__(16) double gate_lds[];
  const int lane = threadIdx.x, r = lane & 15, E = p.E;
  const int t = blockIdx.x * 4 + (lane >> 4);
  const bool live = t < p.T;
  const float* row = p.logits + (int64_t)(live ? t : p.T - 1) * E;
  const int sl = ALIGNED ? SL : (E + 15) / 16, e0 = r * sl, n = min(sl, E - e0);  // n may be < 1
  auto load = [&](const float* v, float (&o)[SL]) {
    if constexpr (ALIGNED) {
#pragma unroll
      for (int i = 0; i < SL / 4; ++i) {
        const f32x4 q = *reinterpret_cast<const f32x4*>(v + e0 + 4 * i);
#pragma unroll
        for (int j = 0; j < 4; ++j) o[4 * i + j] = q[j];
      }
    } else {
#pragma unroll
      for (int i = 0; i < SL; ++i) o[i] = i < n ? v[e0 + i] : -INFINITY;
    }
  };
  float c[SL], b[SL];
  load(row, c);
#pragma unroll
  for (int i = 0; i < SL; ++i) b[i] = 0.0f;
  if (p.bias) load(p.bias, b);
  // an expert that is out gets -infinity for c (a quarter of each: no overflow)
  bool out[SL];
#pragma unroll
  for (int i = 0; i < SL; ++i) out[i] = !(fmaf(c[i], 0.25f, 0.25f * b[i]) > -INFINITY);
  // scores; tol: what two values of c may be off against each other.  Sigmoid: an
  // argument rounded by 2^-24 moves s by at most 0.23 of that, and three
  // operations follow; softmax: its terms, their sum of E and the quotient.
  float m = 0.0f, tol = 8e-7f;
  if (p.sigmoid) {
#pragma unroll
    for (int i = 0; i < SL; ++i)
      c[i] = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(c[i] * -1.44269504f));
  } else {
    m = -INFINITY;
#pragma unroll
    for (int i = 0; i < SL; ++i) m = out[i] ? m : fmaxf(m, c[i]);
    m = gate_max16(m);
    float z = 0.0f;
#pragma unroll
    for (int i = 0; i < SL; ++i) {
      c[i] = out[i] ? 0.0f : c[i] == m ? 1.0f : gate_exp(c[i] - m);
      z += c[i];
    }
    z = gate_sum16(z);
    const float iz = 1.0f / z;  // z >= 1 where an expert is in
    tol = 4e-6f * iz;
#pragma unroll
    for (int i = 0; i < SL; ++i) c[i] *= iz;
  }
  float a = -INFINITY, a2 = -INFINITY;  // this lane's largest, and the next
#pragma unroll
  for (int i = 0; i < SL; ++i) {
    c[i] = out[i] ? -INFINITY : c[i] + b[i];
    a2 = fmaxf(a2, fminf(a, c[i]));
    a = fmaxf(a, c[i]);
  }
  bool sure = true;
  bool mine_in = true;   // this lane's group is chosen
  if (p.groups > 1) {
    float ga = a, ga2 = a2;
    const int lanes = 16 / p.groups, g = r / lanes;
    if (lanes > 1) gate_top2<0xB1>(ga, ga2);
    if (lanes > 2) gate_top2<0x4E>(ga, ga2);
    if (lanes > 4) gate_top2<0x141>(ga, ga2);  // row_half_mirror
    if (lanes > 8) gate_top2<0x140>(ga, ga2);  // row_mirror
    const bool two = p.top2 && ga2 > -INFINITY;
    const float v = two ? ga + ga2 : ga;
    int rank = 0;
    for (int j = 1; j < p.groups; ++j) {
      const int og = (g + j) & (p.groups - 1);
      const float o = __shfl(v, (lane & 48) + og * lanes, 64);
      rank += (o > v || (o == v && og < g)) ? 1 : 0;
    }
    mine_in = rank < p.top_groups;
    // the least chosen group against the best of the others
    const float least = -gate_max16(mine_in ? -v : -INFINITY), other = gate_max16(mine_in ? -INFINITY : v);
    const float size = gate_max16(ga > -INFINITY ? fmaxf(fabsf(ga), two ? fabsf(ga2) : 0.0f) : 0.0f);
    sure = p.top_groups == p.groups || other == -INFINITY || least - other > 4.0f * tol + 1e-6f * size;
  }
  // steps from hi down to the least of the lanes' second largest (of the only one)
  const float hi = gate_max16(mine_in ? a : -INFINITY);
  const float low = mine_in ? (a2 > -INFINITY ? a2 : a > -INFINITY ? a : INFINITY) : INFINITY;
  const float range = hi + gate_max16(-low);
  // infinite or NaN (no range, infinite values): every key has step 1, nothing is sure
  const float unit = 4190000.0f / range;
  const uint32_t code = 1023u - e0;
  uint32_t key[SL], top[4];
#pragma unroll
  for (int i = 0; i < SL; ++i)
    key[i] = ((uint32_t)fmaxf(fmaf(c[i] - hi, unit, 4194302.0f), 1.0f) << 10) + code - i;
  gate_largest4<SL>(key, mine_in ? 0xFFFFFFFFu : 0u, top);
  tol += 2.4e-7f * fmaxf(fabsf(hi), fabsf(hi - range));
  const float gap = 2.0f * tol * unit + 3.0f;
  const uint32_t need = gap < 4.0e6f ? (uint32_t)gap : 4194303u;  // NaN: the latter
  bool more = SL > 4 && top[3] != 0u;  // there may be keys behind the four
  int mine = 0;
  uint32_t popped = 0;
  // takes the largest key away, for lane j's choice
  auto take = [&](int j, uint32_t best) {
    if (r == j) mine = 1023 - (int)(best & 1023u);
    if (top[0] == best) {
      popped = best;
#pragma unroll
      for (int q = 0; q < 3; ++q) top[q] = top[q + 1];
      top[3] = 0u;
    }
    if (SL > 4 && __any(more && top[0] == 0u)) {
      if (more && top[0] == 0u) {
        gate_largest4<SL>(key, popped, top);
        more = top[3] != 0u;
      }
    }
  };
  bool order = true;  // of the chosen among each other
  uint32_t before = 0;
  for (int j = 0; j < p.k; ++j) {
    const uint32_t best = gate_max16(top[0]);
    sure = sure && best >= 2048u;
    order = order && (j == 0 || (before >> 10) - (best >> 10) >= need);
    take(j, best);
    before = best;
  }
  int among = p.k;  // experts that the chosen are among
  uint32_t next = gate_max16(top[0]);
  if (__any(next != 0u && (before >> 10) - (next >> 10) < need)) {
    // the first that is not chosen is as near: it is looked at too, if the one behind it is not
    const bool near = next != 0u && (before >> 10) - (next >> 10) < need;
    take(p.k, next);
    const uint32_t then = gate_max16(top[0]);
    if (near) {
      among = p.k + 1;
      order = false;
      sure = sure && p.k < 16 && next >= 2048u && (then == 0u || (next >> 10) - (then >> 10) >= need);
    }
  }
  // their order in 64 bits (softmax without a bias: that of its terms)
  sure = sure && (order || p.sigmoid || !p.bias);
  if (__any(live && sure && !order)) {
    uint64_t k64 = 0;
    if (r < among && sure) {
      const float l = row[mine];
      const double s = p.sigmoid ? 1.0 / (1.0 + exp(-(double)l)) : l == m ? 1.0 : exp((double)l - (double)m);
      k64 = gate_key(p.bias ? s + (double)p.bias[mine] : s, false, mine);
    }
    int rank = 0, chosen = 0;
    for (int j = 0; j <= p.k; ++j)
      rank += __shfl((unsigned long long)k64, (lane & 48) + min(j, 15), 64) > k64 && j < among ? 1 : 0;
    for (int j = 0; j <= p.k; ++j) {
      const int from = (lane & 48) + min(j, 15), id = __shfl(mine, from, 64);
      if (__shfl(rank, from, 64) == r && j < among) chosen = id;
    }
    if (sure && !order) mine = chosen;
  }
  uint64_t again = __ballot(live && !sure);
  const double all = p.sigmoid || p.renorm ? 1.0 : gate_sum64<ALIGNED>(row, p.bias, e0, ALIGNED ? SL : n, m);
  if (live && sure) {
    // the weights of the chosen in 64 bits
    double s = 0.0;
    if (r < p.k) {
      const float l = row[mine];
      s = p.sigmoid ? 1.0 / (1.0 + exp(-(double)l)) : l == m ? 1.0 : exp((double)l - (double)m);
    }
    const double tot = p.renorm ? gate_sum<16>(s) : all;
    if (r < p.k) {
      p.ids[(int64_t)t * p.k + r] = mine;
      p.w[(int64_t)t * p.k + r] = tot > 0.0 ? (float)((double)p.scale * s / tot) : 0.0f;
    }
  }
  while (again) {
    const int w = __ffsll((unsigned long long)again) - 1;
    again &= ~(0xFFFFull << (w & 48));
    gate_token<SLOTS>(p, blockIdx.x * 4 + (w >> 4), gate_lds);
  }
}

// What the gradients of one token's weights (16 lanes, r < k with a slot) come to:
// with r_j = s_j / sum_i s_i and, where the weights sum to scale,
// ds_j s_j = (scale dw_j - sum_i scale dw_i r_i) r_j, else scale dw_j s_j,
//   sigmoid: dl_j = ds_j s_j (1 - s_j)
//   softmax: dl_e = s_e (ds_e - sum_j ds_j s_j); where the weights were
//            renormalised the last sum is 0.
// Sigmoids are formed in 64 bits by the forward's own operations, so r_j is the
// forward's also where every chosen score is below fp32's smallest number, and 0
// where they are 0 in 64 bits too (logits below -709).  Softmax terms are taken
// against the largest, their sum is 1 at least.
// Ids outside [0, E) are left out, an id that is there twice gets both.
struct GateSlot {
  int id;
  bool there, in;
  float l, dw;
};
MOE_DEV GateSlot gate_slot(const GateArgs& p, int64_t t, int r, const float* row) {
  GateSlot s;
  s.id = r < p.k ? p.ids[t * p.k + r] : -1;
  s.there = s.id >= 0 && s.id < p.E;
  s.l = s.there ? row[s.id] : -INFINITY;
  s.in = s.there && !gate_out(s.l) && !(p.bias && gate_out(p.bias[s.id]));
  s.dw = s.in ? p.dw[t * p.k + r] : 0.0f;  // of an absent slot whatever is there has no part
  return s;
}
// m, iz: softmax's maximum and the reciprocal of its sum (renormalised: of the
// chosen, and any).  `add`: of the slot's own logit, without softmax's common sum
// `dot`; sparse gradients are whole.  True: this lane writes for its id.
MOE_DEV bool gate_slot_grad(const GateArgs& p, const GateSlot& s, int r, float m, float iz, float& add, float& dot) {
  dot = 0.0f;
  if (p.sigmoid) {
    const double ex = exp(-(double)s.l), sj = s.in ? 1.0 / (1.0 + ex) : 0.0;
    const double rest = ex < INFINITY ? ex * sj : 1.0;  // 1 - s_j
    double g = (double)p.scale * (double)s.dw, part = sj;
    if (p.renorm) {
      const double tot = gate_sum<16>(sj);
      part = tot > 0.0 ? sj / tot : 0.0;
      g -= gate_sum<16>(s.in ? g * part : 0.0);
    }
    add = s.in ? (float)(g * part * rest) : 0.0f;
  } else {
    const float sj = s.in ? (s.l == m ? 1.0f : expf(s.l - m)) * iz : 0.0f;
    float g = p.scale * s.dw;
    if (p.renorm) {
      const float tot = gate_sum16(sj), it = tot > 0.0f ? 1.0f / tot : 0.0f;
      g = (g - gate_sum16(g * sj) * it) * it;
    }
    dot = gate_sum16(s.in ? g * sj : 0.0f);
    add = s.in ? g * sj : 0.0f;
  }
  // one lane per id: the first with it takes what the others add
  bool first = s.there;
  const int base = threadIdx.x & 48;
  for (int j = 0; j < p.k; ++j) {
    const int o = __shfl(s.id, base + j, 64);
    const float v = __shfl(add, base + j, 64);
    if (o == s.id && j < r) first = false;
    if (o == s.id && j > r) add += v;
  }
  return first;
}

// Four tokens per wave, lane r with the experts 4 (r + 16 i) .. + 3 (E a multiple
// of 4): a row is read once, if at all (softmax whose weights are not
// renormalised is the one gradient that every logit has a part in), and written
// once.  What the chosen get goes through LDS.  Memory bounds it: softmax 32768 x 256, 69
// MB, 15 us where they stay in the last-level cache from call to call, 17 (4.0 TB/s) where
// inputs and results of 800 MB take turns; 16384 x 1024 39 us.
template <int SL>
__global__ __launch_bounds__(64) void k_gate_bwd_rows(GateArgs p) {
  __shared__ __align__(16) float lds[4][64 * SL / 4];
  constexpr int N = SL / 4;
  const int lane = threadIdx.x, r = lane & 15, E = p.E;
  const int t = blockIdx.x * 4 + (lane >> 4);
  const bool live = t < p.T, dense = !p.sigmoid && !p.renorm;
  const int64_t tt = live ? t : p.T - 1;
  const float* row = p.logits + tt * E;
  float* out = p.dlogits + tt * E;
  float* ds = lds[lane >> 4];
  const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
  const GateSlot s = gate_slot(p, tt, r, row);
#pragma unroll
  for (int i = 0; i < N; ++i) *reinterpret_cast<f32x4*>(ds + 4 * (r + 16 * i)) = zero;
  f32x4 e[N];
  float m = -INFINITY, iz = 1.0f;
  if (dense) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int at = 4 * (r + 16 * i);
      e[i] = at < E ? *reinterpret_cast<const f32x4*>(row + at) : (f32x4){-INFINITY, -INFINITY, -INFINITY, -INFINITY};
      if (p.bias && at < E) {
        const f32x4 b = *reinterpret_cast<const f32x4*>(p.bias + at);
#pragma unroll
        for (int q = 0; q < 4; ++q) e[i][q] = gate_out(b[q]) ? -INFINITY : e[i][q];
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        e[i][q] = e[i][q] != e[i][q] ? -INFINITY : e[i][q];
        m = fmaxf(m, e[i][q]);
      }
    }
    m = gate_max16(m);
    float z = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float x = e[i][q];
        e[i][q] = x == -INFINITY ? 0.0f : x == m ? 1.0f : gate_exp(x - m);
        z += e[i][q];
      }
    z = gate_sum16(z);
    iz = z > 0.0f ? 1.0f / z : 0.0f;
  } else if (!p.sigmoid) {
    m = gate_max16(s.in ? s.l : -INFINITY);
  }
  float add, dot;
  const bool first = gate_slot_grad(p, s, r, m, iz, add, dot);
  if (p.accumulate && !dense) {
    if (live && first) out[s.id] += add;
    return;
  }
  gate_sync();
  if (first) ds[s.id] = add;
  gate_sync();
  if (!live) return;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int at = 4 * (r + 16 * i);
    if (at < E) {
      f32x4 v = *reinterpret_cast<const f32x4*>(ds + at);
      if (dense) {
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] = fmaf(-dot, e[i][q] * iz, v[q]);
      }
      if (p.accumulate) v += *reinterpret_cast<const f32x4*>(out + at);
      *reinterpret_cast<f32x4*>(out + at) = v;
    }
  }
}

// The same for any E, element by element.
__global__ __launch_bounds__(64) void k_gate_bwd(GateArgs p) {
  extern __shared__ __align__(16) float gate_bwd_lds[];
  const int lane = threadIdx.x, r = lane & 15, E = p.E;
  const int t = blockIdx.x * 4 + (lane >> 4);
  const bool live = t < p.T, dense = !p.sigmoid && !p.renorm;
  const int64_t tt = live ? t : p.T - 1;
  const float* row = p.logits + tt * E;
  float* out = p.dlogits + tt * E;
  float* ds = gate_bwd_lds + (lane >> 4) * E;
  const GateSlot s = gate_slot(p, tt, r, row);
  auto at = [&](int e) { return gate_out(row[e]) || (p.bias && gate_out(p.bias[e])) ? -INFINITY : row[e]; };
  float m = s.in ? s.l : -INFINITY, iz = 1.0f;
  if (dense)
    for (int e = r; e < E; e += 16) m = fmaxf(m, at(e));
  m = gate_max16(m);
  if (dense) {
    float z = 0.0f;
    for (int e = r; e < E; e += 16) {
      const float v = at(e);
      z += v == -INFINITY ? 0.0f : v == m ? 1.0f : gate_exp(v - m);
    }
    z = gate_sum16(z);
    iz = z > 0.0f ? 1.0f / z : 0.0f;
  }
  float add, dot;
  const bool first = gate_slot_grad(p, s, r, m, iz, add, dot);
  if (p.accumulate && !dense) {
    if (live && first) out[s.id] += add;
    return;
  }
  for (int e = r; e < E; e += 16) ds[e] = 0.0f;
  gate_sync();
  if (first) ds[s.id] = add;
  gate_sync();
  if (!live) return;
  for (int e = r; e < E; e += 16) {
    float v = ds[e];
    if (dense) {
      const float x = at(e);
      v = fmaf(-dot, (x == -INFINITY ? 0.0f : x == m ? 1.0f : gate_exp(x - m)) * iz, v);
    }
    if (p.accumulate) v += out[e];
    out[e] = v;
  }
}

// g[t][j] = <d_out_t, y_tj>: the sum of the row's parts (one per N block of the
// backward's first product), in their order.
__global__ __launch_bounds__(256) void k_pair_grad(const int32_t* __restrict__ row_of, const float* __restrict__ gpart,
                                                   int nparts, int R, float* __restrict__ g) {
  const int q = blockIdx.x * 256 + threadIdx.x;
  if (q >= R) return;
  const float* part = gpart + (int64_t)row_of[q] * nparts;
  float s = 0.0f;
  for (int i = 0; i < nparts; ++i) s += part[i];
  g[q] = s;
}

void launch_gate(const GateArgs& a, hipStream_t s) {
  if (a.T == 0) return;
  const size_t lds = (size_t)(a.E + GATE_MAX_GROUPS) * 8;
  const bool g16 = a.groups == 1 || (a.groups <= 16 && (a.groups & (a.groups - 1)) == 0 && a.E % 16 == 0);
  if (g16) {
    const dim3 g((a.T + 3) / 4), b(64);
#define GATE(SL, S)                                                                                        \
  do {                                                                                                     \
    if (a.E == 16 * SL) hipLaunchKernelGGL(HIP_KERNEL_NAME(k_gate<SL, S, true>), g, b, lds, s, a);         \
    else hipLaunchKernelGGL(HIP_KERNEL_NAME(k_gate<SL, S, false>), g, b, lds, s, a);                       \
  } while (0)
    if (a.E <= 64) GATE(4, 1);
    else if (a.E <= 128) GATE(8, 2);
    else if (a.E <= 256) GATE(16, 4);
    else if (a.E <= 384) GATE(24, 6);
    else if (a.E <= 512) GATE(32, 8);
    else GATE(64, 16);
#undef GATE
    return;
  }
  const dim3 g(a.T), b(64);
#define GATE(S) hipLaunchKernelGGL(HIP_KERNEL_NAME(k_gate_wave<S>), g, b, lds, s, a)
  if (a.E <= 128) GATE(2);
  else if (a.E <= 512) GATE(8);
  else GATE(16);
#undef GATE
}

void launch_gate_bwd(const GateArgs& a, hipStream_t s) {
  if (a.T == 0) return;
  const dim3 g((a.T + 3) / 4), b(64);
#define GATE(SL) hipLaunchKernelGGL(k_gate_bwd_rows<SL>, g, b, 0, s, a)
  if (a.E % 4 != 0) hipLaunchKernelGGL(k_gate_bwd, g, b, (size_t)a.E * 16, s, a);
  else if (a.E <= 64) GATE(4);
  else if (a.E <= 128) GATE(8);
  else if (a.E <= 256) GATE(16);
  else if (a.E <= 384) GATE(24);
  else if (a.E <= 512) GATE(32);
  else GATE(64);
#undef GATE
}

void launch_pair_grad(const int32_t* row_of, const float* gpart, int nparts, int R, float* g, hipStream_t s) {
  if (R == 0) return;
  hipLaunchKernelGGL(k_pair_grad, dim3((R + 255) / 256), dim3(256), 0, s, row_of, gpart, nparts, R, g);
}

}  // namespace moe
