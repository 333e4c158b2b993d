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
//
// 32768 x 384 in 40 segments, a fifth of the tokens masked: gradient 24-26 us for
// 91 MB (3.5-3.8 TB/s).  16384 x 256 in 13 segments: sums 7.4-8.8 us and finish
// 5.8-6.9, the second waiting for the first.  64 x 384 in one launch: 5.7-6.4 us.
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

// v <- softmax of the row; a row of -infinities gives zeros.  2^(x log2 e - c)
// in one fused operation: c's own rounding is the same for the whole row and
// drops out.  It is up to 2^-24 |c|, which for a row of a mask's values (-1e10) is
// past the exponents of fp32: far from 0 m is taken off first.
template <int N>
MOE_DEV void bl_softmax(float (&v)[N]) {
  constexpr float kLog2e = 1.44269504088896340736f;
  float m = v[0];
#pragma unroll
  for (int i = 1; i < N; ++i) m = fmaxf(m, v[i]);
  m = bl_max16(m);
  const float far = fabsf(m) > 65536.0f && m != -INFINITY ? m : 0.0f;
  const float c = m == -INFINITY ? 0.0f : (m - far) * kLog2e;
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    v[i] = __builtin_amdgcn_exp2f(fmaf(v[i] - far, kLog2e, -c));
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

// A thread's share of a run of tokens [t, tend): sums of softmax rows into acc
// (16 lanes per token, `stride` tokens apart), routed slots into the LDS
// counts, tokens into mine.
template <int NV, bool VEC>
MOE_DEV void bl_run(const float* __restrict__ logits, const int32_t* __restrict__ ids,
                    const uint8_t* __restrict__ mask, int t, int tend, int stride, int E, int k, int ln, int* cnt,
                    float (&acc)[NV * 4], int& mine) {
  for (int u = t; u < tend; u += stride) {
    if (mask != nullptr && mask[u] == 0) continue;
    ++mine;
    float v[NV * 4];
    bl_load<NV, VEC>(logits + (int64_t)u * E, E, ln, v);
    if (ln < k) {
      const int e = ids[(int64_t)u * k + ln];
      if (e >= 0 && e < E) atomicAdd(&cnt[e], 1);
    }
    bl_softmax(v);
#pragma unroll
    for (int i = 0; i < NV * 4; ++i) acc[i] += v[i];
  }
}

// Adds the four tokens' lanes of a wave and writes the wave's sums.
template <int NV>
MOE_DEV void bl_wave_sums(float (&acc)[NV * 4], int lane, float* out) {
#pragma unroll
  for (int i = 0; i < NV * 4; ++i) {
    acc[i] += shfl_xor(acc[i], 16);
    acc[i] += shfl_xor(acc[i], 32);
  }
  if (lane < 16)
#pragma unroll
    for (int i = 0; i < NV; ++i)
      *reinterpret_cast<f32x4*>(out + bl_expert(i, lane, 0)) =
          (f32x4){acc[i * 4], acc[i * 4 + 1], acc[i * 4 + 2], acc[i * 4 + 3]};
}

constexpr int BL_OFF = 1024;  // segment offsets that fit the LDS copy

}  // namespace

// A block sums one slab of `slab` consecutive tokens.  Where segments meet
// inside a slab it leaves one partial sum per segment: slab b and segment s
// share slot b + s (both only grow along the tokens, so slots are distinct;
// at most slabs + S - 1 of them).  Also clears the finish's tickets.
template <int NV, bool VEC>
__global__ __launch_bounds__(256) void k_balance_sums(const float* __restrict__ logits, const int32_t* __restrict__ ids,
                                                      const uint8_t* __restrict__ mask,
                                                      const int32_t* __restrict__ off, int S, int T, int E, int k,
                                                      int slab, float* __restrict__ psum, int32_t* __restrict__ csum,
                                                      int32_t* __restrict__ tsum, int32_t* __restrict__ ticket) {
  constexpr int NE = NV * 64;
  __shared__ __align__(16) float red[4][NE];
  __shared__ int cnt[NE], loff[BL_OFF];
  __shared__ int ntok;
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, row = tid >> 4, ln = tid & 15;
  const int b = blockIdx.x;
  for (int i = b * 256 + tid; i < S; i += gridDim.x * 256) ticket[i] = 0;
  int t = b * slab;
  const int tend = min(T, t + slab);
  int s = 0;
  if (off != nullptr) {
    if (S < BL_OFF) {  // the search's dependent reads go to LDS
      for (int i = tid; i <= S; i += 256) loff[i] = off[i];
      __syncthreads();
      s = bl_count_le(loff, S, t) - 1;
    } else {
      s = bl_count_le(off, S, t) - 1;
    }
    if (s < 0) {  // tokens before the first segment
      s = 0;
      t = max(t, off[0]);
    }
  }
  while (t < tend && s < S) {
    const int send = off != nullptr ? min(tend, max(S < BL_OFF ? loff[s + 1] : off[s + 1], t)) : tend;
    if (send > t) {
      for (int e = tid; e < NE; e += 256) cnt[e] = 0;
      if (tid == 0) ntok = 0;
      __syncthreads();
      float acc[NV * 4];
#pragma unroll
      for (int i = 0; i < NV * 4; ++i) acc[i] = 0.0f;
      int mine = 0;
      bl_run<NV, VEC>(logits, ids, mask, t + row, send, 16, E, k, ln, cnt, acc, mine);
      if (ln == 0 && mine) atomicAdd(&ntok, mine);
      bl_wave_sums<NV>(acc, lane, red[wave]);
      __syncthreads();
      const int64_t slot = b + s;
      for (int e = tid; e < E; e += 256) {
        psum[slot * E + e] = (red[0][e] + red[1][e]) + (red[2][e] + red[3][e]);
        csum[slot * E + e] = cnt[e];
      }
      if (tid == 0) tsum[slot] = ntok;
      __syncthreads();
    }
    t = send;
    ++s;
  }
}

// Block (s, j) adds the slots of segment s for experts 64 j .. 64 j + 63, 16
// groups of 64 threads each taking every 16th slot; the last block of the
// segment to arrive (a ticket) adds the loss's parts in the order of j, so
// results do not depend on which one it is.
__global__ __launch_bounds__(1024) void k_balance_finish(const float* __restrict__ psum,
                                                         const int32_t* __restrict__ csum,
                                                         const int32_t* __restrict__ tsum,
                                                         const int32_t* __restrict__ off, int T, int E, int k,
                                                         int slab, int32_t* __restrict__ ticket,
                                                         float* __restrict__ part, float* __restrict__ loss,
                                                         int32_t* __restrict__ counts, int32_t* __restrict__ tokens,
                                                         float* __restrict__ probs) {
  __shared__ float rp[16][64];
  __shared__ int rc[16][64], rn[16];
  const int s = blockIdx.x, tid = threadIdx.x, g = tid >> 6, lane = tid & 63, e = blockIdx.y * 64 + lane;
  const int t0 = off != nullptr ? min(max(off[s], 0), T) : 0;
  const int t1 = off != nullptr ? min(max(off[s + 1], t0), T) : T;
  const int b0 = t0 / slab, nb = t1 > t0 ? (t1 - 1) / slab - b0 + 1 : 0;
  const int64_t first = b0 + s;
  int n = 0;
  for (int b = tid; b < nb; b += 1024) n += tsum[first + b];
#pragma unroll
  for (int x = 32; x > 0; x >>= 1) n += shfl_xor(n, x);
  if (lane == 0) rn[g] = n;
  float a = 0.0f;
  int c = 0;
  if (e < E)
    for (int b = g; b < nb; b += 128) {
      // up to 8 slots' loads in flight
      float x[8];
      int y[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const bool in = b + i * 16 < nb;
        x[i] = in ? psum[(first + b + i * 16) * E + e] : 0.0f;
        y[i] = in ? csum[(first + b + i * 16) * E + e] : 0;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        a += x[i];
        c += y[i];
      }
    }
  rp[g][lane] = a;
  rc[g][lane] = c;
  __syncthreads();
  if (g != 0) return;
  n = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) n += rn[i];
#pragma unroll
  for (int i = 1; i < 16; ++i) {
    a += rp[i][lane];
    c += rc[i][lane];
  }
  const float inv = n > 0 ? 1.0f / (float)n : 0.0f;
  const float p = a * inv;
  if (e < E) {
    probs[(int64_t)s * E + e] = p;
    counts[(int64_t)s * E + e] = c;
  }
  float l = e < E ? (float)c * p : 0.0f;
#pragma unroll
  for (int x = 32; x > 0; x >>= 1) l += shfl_xor(l, x);
  if (lane == 0) {
    int last = 1;
    if (gridDim.y > 1) {
      // agent scope: other XCDs' parts are in memory before their ticket is
      __hip_atomic_store(&part[(int64_t)s * gridDim.y + blockIdx.y], l, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      last = __hip_atomic_fetch_add(&ticket[s], 1, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) == (int)gridDim.y - 1;
      if (last) {
        l = 0.0f;
        for (unsigned j = 0; j < gridDim.y; ++j)
          l += __hip_atomic_load(&part[(int64_t)s * gridDim.y + j], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      }
    }
    if (last) {
      loss[s] = l * inv * ((float)E / (float)k);
      tokens[s] = n;
    }
  }
}

// Up to BALANCE_ONE tokens: one launch, a block of 64 tokens' lanes per segment
// that forms the outputs itself.
template <int NV, bool VEC>
__global__ __launch_bounds__(1024) void k_balance_one(const float* __restrict__ logits, const int32_t* __restrict__ ids,
                                                      const uint8_t* __restrict__ mask,
                                                      const int32_t* __restrict__ off, int T, int E, int k,
                                                      float* __restrict__ loss, int32_t* __restrict__ counts,
                                                      int32_t* __restrict__ tokens, float* __restrict__ probs) {
  constexpr int NE = NV * 64;
  __shared__ __align__(16) float red[16][NE];
  __shared__ int cnt[NE];
  __shared__ float wsum[16];
  __shared__ int ntok;
  const int s = blockIdx.x, tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, row = tid >> 4, ln = tid & 15;
  const int t0 = off != nullptr ? min(max(off[s], 0), T) : 0;
  const int t1 = off != nullptr ? min(max(off[s + 1], t0), T) : T;
  if (tid < NE) cnt[tid] = 0;
  if (tid == 0) ntok = 0;
  __syncthreads();
  float acc[NV * 4];
#pragma unroll
  for (int i = 0; i < NV * 4; ++i) acc[i] = 0.0f;
  int mine = 0;
  bl_run<NV, VEC>(logits, ids, mask, t0 + row, t1, 64, E, k, ln, cnt, acc, mine);
  if (ln == 0 && mine) atomicAdd(&ntok, mine);
  bl_wave_sums<NV>(acc, lane, red[wave]);
  __syncthreads();
  const int n = ntok;
  const float inv = n > 0 ? 1.0f / (float)n : 0.0f;
  float l = 0.0f;
  if (tid < E) {
    float a = 0.0f;
#pragma unroll
    for (int w = 0; w < 16; ++w) a += red[w][tid];
    const float p = a * inv;
    const int c = cnt[tid];
    probs[(int64_t)s * E + tid] = p;
    counts[(int64_t)s * E + tid] = c;
    l = (float)c * p;
  }
#pragma unroll
  for (int x = 32; x > 0; x >>= 1) l += shfl_xor(l, x);
  if (lane == 0) wsum[wave] = l;
  __syncthreads();
  if (tid == 0) {
    l = 0.0f;
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
  __shared__ int loff[BL_OFF];
  const int row = threadIdx.x >> 4, ln = threadIdx.x & 15;
  const int tend = min(T, ((int)blockIdx.x + 1) * slab);
  if (off != nullptr && S < BL_OFF) {
    for (int i = threadIdx.x; i <= S; i += 256) loff[i] = off[i];
    __syncthreads();
  }
  int shi = -1;  // end of the segment whose a is held
  float a[NV * 4];
  bool none = false;
  for (int t = blockIdx.x * slab + row; t < tend; t += 16) {
    if (t >= shi) {
      int s = 0;
      shi = T;
      if (off != nullptr) {
        s = (S < BL_OFF ? bl_count_le(loff, S + 1, t) : bl_count_le(off, S + 1, t)) - 1;  // -1 or S: no segment
        shi = s >= S ? T : S < BL_OFF ? loff[s + 1] : off[s + 1];
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

constexpr int BALANCE_ONE = 1024;

// Tokens per block: 16 rows of lanes take them 16 at a time, and two blocks
// per CU hide the reads' latency.
int balance_slab(int T, int most = 512) {
  int slab = 16;
  while (slab < 1024 && (T + slab - 1) / slab > most) slab *= 2;
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
                    int E, int k, float* psum, int32_t* csum, int32_t* tsum, int32_t* ticket, float* part, float* loss,
                    int32_t* counts, int32_t* tokens, float* probs, hipStream_t s) {
  const int slab = balance_slab(T);
  if (T <= BALANCE_ONE) {
    balance_dispatch(E, [&](auto nv, auto vec) {
      hipLaunchKernelGGL((k_balance_one<decltype(nv)::value, decltype(vec)::value>), dim3(S), dim3(1024), 0, s, logits,
                         ids, mask, off, T, E, k, loss, counts, tokens, probs);
    });
    return;
  }
  balance_dispatch(E, [&](auto nv, auto vec) {
    hipLaunchKernelGGL((k_balance_sums<decltype(nv)::value, decltype(vec)::value>), dim3((T + slab - 1) / slab),
                       dim3(256), 0, s, logits, ids, mask, off, S, T, E, k, slab, psum, csum, tsum, ticket);
  });
  hipLaunchKernelGGL(k_balance_finish, dim3(S, (E + 63) / 64), dim3(1024), 0, s, psum, csum, tsum, off, T, E, k, slab,
                     ticket, part, loss, counts, tokens, probs);
}

void launch_balance_bwd(const float* logits, const uint8_t* mask, const int32_t* off, int S, int T, int E, int k,
                        const int32_t* counts, const int32_t* tokens, const float* dloss, int accumulate,
                        float* dlogits, hipStream_t s) {
  if (T == 0) return;
  const int slab = balance_slab(T, 1024);
  balance_dispatch(E, [&](auto nv, auto vec) {
    hipLaunchKernelGGL((k_balance_bwd<decltype(nv)::value, decltype(vec)::value>), dim3((T + slab - 1) / slab),
                       dim3(256), 0, s, logits, mask, off, S, T, E, k, counts, tokens, dloss, accumulate, slab,
                       dlogits);
  });
}

}  // namespace moe
