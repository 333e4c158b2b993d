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

// LPT lanes per token (16: four tokens per wave; 64: one), lane r of them with
// the experts r, r + LPT, ...: SLOTS, E <= LPT SLOTS.  Scores are formed in 64
// bits, since two neighbours' order decides which expert runs.  LDS per token:
// the scores, the group values.
template <int LPT, int SLOTS>
__global__ __launch_bounds__(64) void k_gate(GateArgs p) {
  extern __shared__ __align__(16) double gate_lds[];
  constexpr int TPW = 64 / LPT;
  const int lane = threadIdx.x, r = lane % LPT, E = p.E;
  const int t = blockIdx.x * TPW + lane / LPT;
  const bool live = t < p.T;
  const float* row = p.logits + (int64_t)(live ? t : 0) * E;
  double* sc = gate_lds + (lane / LPT) * (E + GATE_MAX_GROUPS);
  double* gv = sc + E;

  float l[SLOTS], b[SLOTS];
  bool out[SLOTS];
#pragma unroll
  for (int i = 0; i < SLOTS; ++i) {
    const int e = r + LPT * i;
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
    m = gate_max<LPT>(m);
    double z = 0.0;
#pragma unroll
    for (int i = 0; i < SLOTS; ++i) {
      s[i] = out[i] ? 0.0 : l[i] == m ? 1.0 : exp((double)l[i] - (double)m);
      z += s[i];
    }
    z = gate_sum<LPT>(z);
#pragma unroll
    for (int i = 0; i < SLOTS; ++i) s[i] = z > 0.0 ? s[i] / z : 0.0;
  }
  uint64_t key[SLOTS];
#pragma unroll
  for (int i = 0; i < SLOTS; ++i) {
    const int e = r + LPT * i;
    const double c = s[i] + (double)b[i];
    key[i] = e < E ? gate_key(c, out[i], e) : 0ull;
    if (p.groups > 1 && e < E) sc[e] = out[i] ? -INFINITY : c;
  }
  if (p.groups > 1) {
    gate_sync();
    const int per = E / p.groups;
    for (int g = r; g < p.groups; g += LPT) {
      double a = -INFINITY, a2 = -INFINITY;
      for (int i = 0; i < per; ++i) {
        const double v = sc[g * per + i];
        a2 = fmax(a2, fmin(a, v));
        a = fmax(a, v);
      }
      gv[g] = p.top2 && a2 > -INFINITY ? a + a2 : a;
    }
    gate_sync();
    uint64_t chosen = 0;  // of this lane's groups r, r + LPT, ... (bit i)
    for (int g = r, i = 0; g < p.groups; g += LPT, ++i) {
      const double v = gv[g];
      int rank = 0;
      for (int j = 0; j < p.groups; ++j) rank += (gv[j] > v || (gv[j] == v && j < g)) ? 1 : 0;
      if (rank < p.top_groups) chosen |= 1ull << i;
    }
    gate_sync();
    for (int g = r, i = 0; g < p.groups; g += LPT, ++i) gv[g] = (chosen >> i) & 1 ? 1.0 : 0.0;
    gate_sync();
#pragma unroll
    for (int i = 0; i < SLOTS; ++i) {
      const int e = r + LPT * i;
      if (e < E && gv[e / per] == 0.0) key[i] = 0;
    }
    gate_sync();
  }
#pragma unroll
  for (int i = 0; i < SLOTS; ++i)
    if (r + LPT * i < E) sc[r + LPT * i] = s[i];
  int mine = 0;
  for (int j = 0; j < p.k; ++j) {
    uint64_t best = 0;
#pragma unroll
    for (int i = 0; i < SLOTS; ++i) best = key[i] > best ? key[i] : best;
    best = gate_max_u64<LPT>(best);
#pragma unroll
    for (int i = 0; i < SLOTS; ++i) key[i] = key[i] == best ? 0ull : key[i];
    if (r == j) mine = 1023 - (int)(best & 1023u);
  }
  gate_sync();
  const double sj = r < p.k ? sc[mine] : 0.0;
  const double tot = p.renorm ? gate_sum<LPT>(sj) : 1.0;
  if (!live || r >= p.k) return;
  p.ids[(int64_t)t * p.k + r] = mine;
  p.w[(int64_t)t * p.k + r] = tot > 0.0 ? (float)((double)p.scale * sj / tot) : 0.0f;
}

// d_logits of one token by 16 lanes: with ds_j = scale dw_j, or with weights
// that sum to scale, ds_j = (scale dw_j - sum_i dw_i w_i) / sum_i s_i,
//   sigmoid: dl_j = ds_j s_j (1 - s_j)
//   softmax: dl_e = s_e (ds_e - sum_j ds_j s_j); where the weights were
//            renormalised the last sum is 0.
// Ids outside [0, E) are left out, an id that is there twice gets both.
__global__ __launch_bounds__(64) void k_gate_bwd(GateArgs p) {
  extern __shared__ __align__(16) float gate_bwd_lds[];
  const int lane = threadIdx.x, r = lane & 15, E = p.E;
  const int t = blockIdx.x * 4 + (lane >> 4);
  const bool live = t < p.T;
  const int64_t tt = live ? t : 0;
  const float* row = p.logits + tt * E;
  float* ds = gate_bwd_lds + (lane >> 4) * E;
  const int id = r < p.k ? p.ids[tt * p.k + r] : -1;
  const bool there = id >= 0 && id < E;
  const float lj = there ? row[id] : -INFINITY;
  const bool in = there && !gate_out(lj) && !(p.bias && gate_out(p.bias[id]));
  const float dw = r < p.k ? p.dw[tt * p.k + r] : 0.0f;
  const bool dense = !p.sigmoid && !p.renorm;
  float m = 0.0f, iz = 1.0f;
  if (!p.sigmoid) {
    m = in ? lj : -INFINITY;
    if (dense)
      for (int e = r; e < E; e += 16) {
        const float v = row[e];
        if (!gate_out(v) && !(p.bias && gate_out(p.bias[e]))) m = fmaxf(m, v);
      }
    m = gate_max<16>(m);
    float z = 0.0f;
    if (dense) {
      for (int e = r; e < E; e += 16) {
        const float v = row[e];
        if (!gate_out(v) && !(p.bias && gate_out(p.bias[e]))) z += v == m ? 1.0f : expf(v - m);
      }
      z = gate_sum<16>(z);
    } else {
      z = 1.0f;  // any: only ratios of chosen scores are used
    }
    iz = z > 0.0f ? 1.0f / z : 0.0f;
  }
  float sj = 0.0f, sp = 0.0f;  // the score, and its derivative (softmax: by its own logit, but for the sum)
  if (in) {
    if (p.sigmoid) {
      const float e = expf(-fabsf(lj)), q = 1.0f / (1.0f + e);
      sj = lj >= 0.0f ? q : e * q;
      sp = e * q * q;
    } else {
      sj = (lj == m ? 1.0f : expf(lj - m)) * iz;
      sp = sj;
    }
  }
  float g = p.scale * dw;
  if (p.renorm) {
    const float tot = gate_sum<16>(sj), it = tot > 0.0f ? 1.0f / tot : 0.0f;
    g = (g - gate_sum<16>(g * sj) * it) * it;
  }
  const float dot = dense ? gate_sum<16>(in ? g * sj : 0.0f) : 0.0f;
  float add = in ? g * sp : 0.0f;
  // one lane per id: the first with it takes what the others add
  bool first = there;
  for (int j = 0; j < p.k; ++j) {
    const int o = __shfl(id, (lane & 48) + j, 64);
    const float v = __shfl(add, (lane & 48) + j, 64);
    if (o == id && j < r) first = false;
    if (o == id && j > r) add += v;
  }
  if (p.accumulate && !dense) {
    if (live && first) p.dlogits[tt * E + id] += add;
    return;
  }
  for (int e = r; e < E; e += 16) ds[e] = 0.0f;
  gate_sync();
  if (first) ds[id] = add;
  gate_sync();
  if (!live) return;
  for (int e = r; e < E; e += 16) {
    float v = ds[e];
    if (dense) {
      const float x = row[e];
      if (!gate_out(x) && !(p.bias && gate_out(p.bias[e]))) v -= dot * ((x == m ? 1.0f : expf(x - m)) * iz);
    }
    if (p.accumulate) v += p.dlogits[tt * E + e];
    p.dlogits[tt * E + e] = v;
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

template <int LPT>
static void launch_gate_lpt(const GateArgs& a, hipStream_t s) {
  const dim3 g((a.T + 64 / LPT - 1) / (64 / LPT)), b(64);
  const size_t lds = (size_t)(64 / LPT) * (a.E + GATE_MAX_GROUPS) * 8;
  const int n = (a.E + LPT - 1) / LPT;
#define GATE(S) hipLaunchKernelGGL(HIP_KERNEL_NAME(k_gate<LPT, S>), g, b, lds, s, a)
  if constexpr (LPT == 64) {
    if (n <= 2) GATE(2);
    else if (n <= 4) GATE(4);
    else if (n <= 6) GATE(6);
    else if (n <= 8) GATE(8);
    else GATE(16);
  } else {
    if (n <= 4) GATE(4);
    else if (n <= 8) GATE(8);
    else if (n <= 16) GATE(16);
    else if (n <= 24) GATE(24);
    else GATE(32);
  }
#undef GATE
}

void launch_gate(const GateArgs& a, hipStream_t s) {
  if (a.T == 0) return;
  if (a.T <= 1024 || a.E > 512) launch_gate_lpt<64>(a, s);
  else launch_gate_lpt<16>(a, s);
}

void launch_gate_bwd(const GateArgs& a, hipStream_t s) {
  if (a.T == 0) return;
  hipLaunchKernelGGL(k_gate_bwd, dim3((a.T + 3) / 4), dim3(64), (size_t)a.E * 16, s, a);
}

void launch_pair_grad(const int32_t* row_of, const float* gpart, int nparts, int R, float* g, hipStream_t s) {
  if (R == 0) return;
  hipLaunchKernelGGL(k_pair_grad, dim3((R + 255) / 256), dim3(256), 0, s, row_of, gpart, nparts, R, g);
}

}  // namespace moe
