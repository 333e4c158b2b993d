// Router balance loss, per-expert counts and their gradient.
//
// Per segment s of n counted tokens: P_e = mean p_t[e] with p_t = softmax over
// all E experts, c_e the routed slots, loss = E / (k n) sum_e c_e P_e;
// gradient p_t[e] (a_e - sum_i p_t[i] a_i), a_e = d_loss E c_e / (k n^2).
// One read of the logits each way (and one write of d_logits), so memory
// latency and bandwidth bound both.
//
// A token's row is held by 16 lanes (a DPP row: maxima and sums are four
// register-to-register steps), E/16 experts each in aligned fours, so a wave
// works on four tokens at once and every lane keeps the running sums of its
// own experts in registers over all its tokens.
#include "common.h"
#include "kernels.h"

#include <type_traits>

namespace moe {

namespace {

template <int CTRL>
MOE_DEV float bl_dpp(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, false));
}
// Maximum and sum over the 16 lanes of a DPP row, the same in every lane.
MOE_DEV float bl_max16(float v) {
  v = fmaxf(v, bl_dpp<0xB1>(v));
  v = fmaxf(v, bl_dpp<0x4E>(v));
  v = fmaxf(v, bl_dpp<0x124>(v));
  return fmaxf(v, bl_dpp<0x128>(v));
}
MOE_DEV float bl_sum16(float v) {
  v += bl_dpp<0xB1>(v);
  v += bl_dpp<0x4E>(v);
  v += bl_dpp<0x124>(v);
  return v + bl_dpp<0x128>(v);
}

// Expert of value j (0..3) of group i of lane ln of a row.
MOE_DEV int bl_expert(int i, int ln, int j) { return (i * 16 + ln) * 4 + j; }

// The row's logits; experts >= E read as -infinity.  VEC: E is a multiple of
// 4, so the rows are 16-byte aligned.
template <int NV, bool VEC>
MOE_DEV void bl_load(const float* __restrict__ row, int E, int ln, float (&v)[NV * 4]) {
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = bl_expert(i, ln, 0);
    if (VEC) {
      f32x4 q = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
      if (e < E) q = *reinterpret_cast<const f32x4*>(row + e);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[i * 4 + j] = q[j];
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) v[i * 4 + j] = e + j < E ? row[e + j] : -INFINITY;
    }
  }
}

// v <- softmax of the row; a row of -infinities gives zeros.
template <int N>
MOE_DEV void bl_softmax(float (&v)[N]) {
  float m = v[0];
#pragma unroll
  for (int i = 1; i < N; ++i) m = fmaxf(m, v[i]);
  m = bl_max16(m);
  if (m == -INFINITY) m = 0.0f;
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    v[i] = expf(v[i] - m);
    s += v[i];
  }
  s = bl_sum16(s);
  const float inv = s == 0.0f ? 0.0f : 1.0f / s;
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] *= inv;
}

// First index in [0, n) whose offset is above t, i.e. the number of offsets
// <= t among off[0..n) (non-decreasing).
MOE_DEV int bl_count_le(const int32_t* off, int n, int t) {
  int lo = 0, hi = n;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (off[mid] <= t) lo = mid + 1;
    else hi = mid;
  }
  return lo;
}

}  // namespace

// A block sums one slab of `slab` consecutive tokens.  Where segments meet
// inside a slab it leaves one partial sum per segment: slab b and segment s
// share slot b + s (both only grow along the tokens, so slots are distinct;
// at most slabs + S - 1 of them).
template <int NV, bool VEC>
__global__ __launch_bounds__(256) void k_balance_sums(const float* __restrict__ logits, const int32_t* __restrict__ ids,
                                                      const uint8_t* __restrict__ mask,
                                                      const int32_t* __restrict__ off, int S, int T, int E, int k,
                                                      int slab, float* __restrict__ psum, int32_t* __restrict__ csum,
                                                      int32_t* __restrict__ tsum) {
  constexpr int NE = NV * 64;
  __shared__ float red[16][NE];
  __shared__ int cnt[NE];
  __shared__ int ntok;
  const int tid = threadIdx.x, row = tid >> 4, ln = tid & 15;
  const int b = blockIdx.x;
  int t = b * slab;
  const int tend = min(T, t + slab);
  int s = 0;
  if (off != nullptr) {
    // the segment of t: the last one that starts at or before it
    s = bl_count_le(off, S, t) - 1;
    if (s < 0) {  // tokens before the first segment
      s = 0;
      t = max(t, off[0]);
    }
  }
  while (t < tend && s < S) {
    const int send = off != nullptr ? min(tend, max(off[s + 1], t)) : tend;
    if (send > t) {
      for (int e = tid; e < NE; e += 256) cnt[e] = 0;
      if (tid == 0) ntok = 0;
      __syncthreads();
      float acc[NV * 4];
#pragma unroll
      for (int i = 0; i < NV * 4; ++i) acc[i] = 0.0f;
      int mine = 0;
      for (int u = t + row; u < send; u += 16) {
        if (mask != nullptr && mask[u] == 0) continue;
        ++mine;
        float v[NV * 4];
        bl_load<NV, VEC>(logits + (int64_t)u * E, E, ln, v);
        bl_softmax(v);
#pragma unroll
        for (int i = 0; i < NV * 4; ++i) acc[i] += v[i];
        if (ln < k) {
          const int e = ids[(int64_t)u * k + ln];
          if (e >= 0 && e < E) atomicAdd(&cnt[e], 1);
        }
      }
      if (ln == 0 && mine) atomicAdd(&ntok, mine);
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) red[row][bl_expert(i, ln, j)] = acc[i * 4 + j];
      __syncthreads();
      const int64_t slot = b + s;
      for (int e = tid; e < E; e += 256) {
        float a = 0.0f;
#pragma unroll
        for (int r = 0; r < 16; ++r) a += red[r][e];
        psum[slot * E + e] = a;
        csum[slot * E + e] = cnt[e];
      }
      if (tid == 0) tsum[slot] = ntok;
      __syncthreads();
    }
    t = send;
    ++s;
  }
}

// One block per segment: adds its slots in order and forms the outputs.
__global__ __launch_bounds__(1024) void k_balance_finish(const float* __restrict__ psum,
                                                         const int32_t* __restrict__ csum,
                                                         const int32_t* __restrict__ tsum,
                                                         const int32_t* __restrict__ off, int T, int E, int k,
                                                         int slab, float* __restrict__ loss,
                                                         int32_t* __restrict__ counts, int32_t* __restrict__ tokens,
                                                         float* __restrict__ probs) {
  __shared__ float rp[1024];
  __shared__ int rc[1024];
  __shared__ float wsum[16];
  const int s = blockIdx.x, tid = threadIdx.x;
  const int t0 = off != nullptr ? min(max(off[s], 0), T) : 0;
  const int t1 = off != nullptr ? min(max(off[s + 1], t0), T) : T;
  const int b0 = t0 / slab, nb = t1 > t0 ? (t1 - 1) / slab - b0 + 1 : 0;
  // tokens of the segment
  int n = 0;
  for (int b = tid; b < nb; b += 1024) n += tsum[b0 + b + s];
  rc[tid] = n;
  __syncthreads();
  for (int d = 512; d > 0; d >>= 1) {
    if (tid < d) rc[tid] += rc[tid + d];
    __syncthreads();
  }
  n = rc[0];
  __syncthreads();
  const float inv = n > 0 ? 1.0f / (float)n : 0.0f;
  // G groups of threads share the slots of an expert (E <= 1024)
  const int W = (E + 63) / 64 * 64, G = 1024 / W;
  const int g = tid / W, e = tid - g * W;
  float a = 0.0f;
  int c = 0;
  if (g < G && e < E)
    for (int b = g; b < nb; b += G) {
      a += psum[(int64_t)(b0 + b + s) * E + e];
      c += csum[(int64_t)(b0 + b + s) * E + e];
    }
  rp[tid] = a;
  rc[tid] = c;
  __syncthreads();
  float part = 0.0f;
  if (tid < E) {
    for (int j = 1; j < G; ++j) {
      a += rp[j * W + tid];
      c += rc[j * W + tid];
    }
    const float p = a * inv;
    probs[(int64_t)s * E + tid] = p;
    counts[(int64_t)s * E + tid] = c;
    part = (float)c * p;
  }
#pragma unroll
  for (int x = 32; x > 0; x >>= 1) part += shfl_xor(part, x);
  if ((tid & 63) == 0) wsum[tid >> 6] = part;
  __syncthreads();
  if (tid == 0) {
    float l = 0.0f;
    for (int i = 0; i < 16; ++i) l += wsum[i];
    loss[s] = l * inv * ((float)E / (float)k);
    tokens[s] = n;
  }
}

// Gradient.  The mean count is taken off a first: it drops out of
// a_e - sum_i p_i a_i (sum p = 1) and would only cost digits there.
template <int NV, bool VEC>
__global__ __launch_bounds__(256) void k_balance_bwd(const float* __restrict__ logits,
                                                     const uint8_t* __restrict__ mask,
                                                     const int32_t* __restrict__ off, int S, int T, int E, int k,
                                                     const int32_t* __restrict__ counts,
                                                     const int32_t* __restrict__ tokens,
                                                     const float* __restrict__ dloss, int accumulate, int slab,
                                                     float* __restrict__ dlogits) {
  const int row = threadIdx.x >> 4, ln = threadIdx.x & 15;
  const int tend = min(T, ((int)blockIdx.x + 1) * slab);
  int shi = -1;  // end of the segment whose a is held
  float a[NV * 4];
  bool none = false;
  for (int t = blockIdx.x * slab + row; t < tend; t += 16) {
    if (t >= shi) {
      int s = 0;
      shi = T;
      if (off != nullptr) {
        s = bl_count_le(off, S + 1, t) - 1;  // -1 or S: no segment
        shi = s >= S ? T : off[s + 1];
      }
      none = s < 0 || s >= S || tokens[s] <= 0;
      if (!none) {
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int e = bl_expert(i, ln, j);
            a[i * 4 + j] = e < E ? (float)counts[(int64_t)s * E + e] : 0.0f;
            sum += a[i * 4 + j];
          }
        const float mean = bl_sum16(sum) / (float)E;
        const float inv = 1.0f / (float)tokens[s];
        const float f = dloss[s] * ((float)E / (float)k) * inv * inv;
#pragma unroll
        for (int i = 0; i < NV * 4; ++i) a[i] = (a[i] - mean) * f;
      }
    }
    const bool on = !none && !(mask != nullptr && mask[t] == 0);
    float v[NV * 4];
    if (on) {
      bl_load<NV, VEC>(logits + (int64_t)t * E, E, ln, v);
      bl_softmax(v);
      float dot = 0.0f;
#pragma unroll
      for (int i = 0; i < NV * 4; ++i) dot = fmaf(v[i], a[i], dot);
      dot = bl_sum16(dot);
#pragma unroll
      for (int i = 0; i < NV * 4; ++i) v[i] *= a[i] - dot;
    } else {
      if (accumulate) continue;
#pragma unroll
      for (int i = 0; i < NV * 4; ++i) v[i] = 0.0f;
    }
    float* o = dlogits + (int64_t)t * E;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = bl_expert(i, ln, 0);
      if (VEC) {
        if (e < E) {
          f32x4 q = {v[i * 4], v[i * 4 + 1], v[i * 4 + 2], v[i * 4 + 3]};
          if (accumulate) q += *reinterpret_cast<const f32x4*>(o + e);
          *reinterpret_cast<f32x4*>(o + e) = q;
        }
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (e + j < E) o[e + j] = accumulate ? o[e + j] + v[i * 4 + j] : v[i * 4 + j];
      }
    }
  }
}

// Tokens per block: 16 rows of lanes take them 16 at a time.
int balance_slab(int T) {
  int slab = 16;
  while (slab < 1024 && (T + slab - 1) / slab > 512) slab *= 2;
  return slab;
}
int64_t balance_slots(int T, int S) { return (T + balance_slab(T) - 1) / balance_slab(T) + (int64_t)S; }

// f(NV, VEC) with 64 NV >= E.
template <typename F>
static void balance_dispatch(int E, F f) {
  const bool vec = E % 4 == 0;
#define MOE_BL(NV)                                       \
  do {                                                   \
    if (vec) f(std::integral_constant<int, NV>(), std::true_type());  \
    else f(std::integral_constant<int, NV>(), std::false_type());     \
  } while (0)
  if (E <= 64) MOE_BL(1);
  else if (E <= 128) MOE_BL(2);
  else if (E <= 256) MOE_BL(4);
  else if (E <= 384) MOE_BL(6);
  else if (E <= 512) MOE_BL(8);
  else MOE_BL(16);
#undef MOE_BL
}

void launch_balance(const float* logits, const int32_t* ids, const uint8_t* mask, const int32_t* off, int S, int T,
                    int E, int k, float* psum, int32_t* csum, int32_t* tsum, float* loss, int32_t* counts,
                    int32_t* tokens, float* probs, hipStream_t s) {
  const int slab = balance_slab(T);
  if (T > 0)
    balance_dispatch(E, [&](auto nv, auto vec) {
      hipLaunchKernelGGL((k_balance_sums<decltype(nv)::value, decltype(vec)::value>), dim3((T + slab - 1) / slab),
                         dim3(256), 0, s, logits, ids, mask, off, S, T, E, k, slab, psum, csum, tsum);
    });
  hipLaunchKernelGGL(k_balance_finish, dim3(S), dim3(1024), 0, s, psum, csum, tsum, off, T, E, k, slab, loss, counts,
                     tokens, probs);
}

void launch_balance_bwd(const float* logits, const uint8_t* mask, const int32_t* off, int S, int T, int E, int k,
                        const int32_t* counts, const int32_t* tokens, const float* dloss, int accumulate,
                        float* dlogits, hipStream_t s) {
  if (T == 0) return;
  const int slab = balance_slab(T);
  balance_dispatch(E, [&](auto nv, auto vec) {
    hipLaunchKernelGGL((k_balance_bwd<decltype(nv)::value, decltype(vec)::value>), dim3((T + slab - 1) / slab),
                       dim3(256), 0, s, logits, mask, off, S, T, E, k, counts, tokens, dloss, accumulate, slab,
                       dlogits);
  });
}

}  // namespace moe
