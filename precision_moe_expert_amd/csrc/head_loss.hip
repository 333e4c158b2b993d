// Losses through the LM head, cross entropy and distillation from a teacher's
// top logits, with their gradients.
//
// Both have a target that is sparse over the vocabulary (one id with weight 1,
// or `top` ids with weights q), so they share every product:
//   forward   l = s r h W^T, per row the log of the sum of exponentials and
//             the few l at the target's ids; no l leaves the product's tile
//             but those
//   backward  per piece of the vocabulary l again, G = s r g exp(l - lse) in
//             bf16, its entries at the target's ids replaced by
//             s r g (p - q); then u += G W (dL/dz r) and d_W = G^T h
// with r = 1 / sqrt(mean h^2 + eps), s the logit scale and g = dL/dloss.
// r s multiplies the fp32 accumulators: the products' operands are the bf16
// inputs themselves, and G is the one value that is rounded on the way.
// Tokens that do not count are left out of the products: rows[] lists the
// others, and operand rows are fetched through it.
#include "common.h"
#include "kernels.h"

namespace moe {

namespace {

constexpr int HB = 128;       // rows and columns of a product's tile
constexpr int HK = 32;        // K per step
constexpr int HS = HK + 8;    // LDS row stride of a staged operand (elements)

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
MOE_DEV void hl_merge(float& m, float& s, float m2, float s2) {
  if (s2 == 0.0f) return;  // an empty part changes nothing
  if (s == 0.0f) {
    m = m2;
    s = s2;
    return;
  }
  const float M = fmaxf(m, m2);
  s = s * expf(m - M) + s2 * expf(m2 - M);
  m = M;
}

}  // namespace

// Per token (one wave): whether it counts, 1/rms of its row, and for
// distillation the log of the teacher's probabilities (-infinity for slots
// that are not there).
__global__ __launch_bounds__(256) void k_head_rows(const uint16_t* __restrict__ h, int64_t h_stride, int T, int H, int V,
                                                   float eps, const int32_t* __restrict__ ids, int top,
                                                   const float* __restrict__ tlogits, float tscale,
                                                   float* __restrict__ r, uint8_t* __restrict__ flag,
                                                   float* __restrict__ lq) {
  const int t = blockIdx.x * 4 + (threadIdx.x >> 6), lane = threadIdx.x & 63;
  if (t >= T) return;
  bool counts;
  if (tlogits == nullptr) {
    const int y = ids[t];
    counts = y >= 0 && y < V;
  } else {
    float x[4], m = -INFINITY;
    bool have[4], any = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int j = i * 64 + lane;
      have[i] = false;
      x[i] = -INFINITY;
      if (j < top) {
        const int id = ids[(int64_t)t * top + j];
        if (id >= 0 && id < V) {
          x[i] = tlogits[(int64_t)t * top + j];
          have[i] = !(x[i] == -INFINITY);
          x[i] *= tscale;
        }
      }
      any |= have[i];
      if (have[i]) m = fmaxf(m, x[i]);
    }
    m = hl_max64(m);
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (have[i]) s += expf(x[i] - m);
    const float ls = logf(hl_sum64(s));
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i * 64 + lane < top) lq[(int64_t)t * top + i * 64 + lane] = have[i] ? x[i] - m - ls : -INFINITY;
    counts = __any(any);
  }
  float rr = 1.0f;
  if (counts && eps > 0.0f) {
    float ss = 0.0f;
    const uint16_t* row = h + (int64_t)t * h_stride;
    for (int c = lane; c < H / 8; c += 64) {
      const u32x4 q = *reinterpret_cast<const u32x4*>(row + c * 8);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float a = bf16_bits_to_f32(q[i] & 0xFFFFu), b = bf16_bits_to_f32(q[i] >> 16);
        ss = fmaf(a, a, ss);
        ss = fmaf(b, b, ss);
      }
    }
    rr = 1.0f / sqrtf(hl_sum64(ss) / (float)H + eps);
  }
  if (lane == 0) {
    r[t] = rr;
    flag[t] = counts;
  }
}

// The list of tokens that count, in order, and each token's place in it (-1).
__global__ __launch_bounds__(1024) void k_head_compact(const uint8_t* __restrict__ flag, int T,
                                                       int32_t* __restrict__ rows, int32_t* __restrict__ cidx,
                                                       int32_t* __restrict__ count) {
  __shared__ int part[1024];
  const int tid = threadIdx.x, per = (T + 1023) / 1024;
  const int t0 = min(T, tid * per), t1 = min(T, t0 + per);
  int n = 0;
  for (int t = t0; t < t1; ++t) n += flag[t];
  part[tid] = n;
  __syncthreads();
  for (int d = 1; d < 1024; d <<= 1) {
    const int v = tid >= d ? part[tid - d] : 0;
    __syncthreads();
    part[tid] += v;
    __syncthreads();
  }
  int c = part[tid] - n;
  for (int t = t0; t < t1; ++t) {
    if (flag[t]) {
      rows[c] = t;
      cidx[t] = c++;
    } else {
      cidx[t] = -1;
    }
  }
  if (tid == 1023) *count = part[1023];
}

// One product of the head; what its operands are and what becomes of the
// accumulators:
//   STATS  h W^T -> (max, sum of exponentials) per row and column block, and
//          the logits at the target's ids
//   GRAD   h W^T -> G, columns [v0, v0 + piece)
//   DZ     G W   -> u, added up over the pieces
//   DW     G^T h -> d_w rows [v0, v0 + piece)
enum { HP_STATS, HP_GRAD, HP_DZ, HP_DW };

struct HeadGemm {
  const uint16_t* h;
  const uint16_t* w;
  int64_t h_stride, w_stride;
  int H, V, top;
  const int32_t* rows;
  const int32_t* count;
  const float* r;
  const float* lse;
  const float* dloss;
  float scale;
  const int32_t* ids;
  float* stats;   // [count][nvb][2]
  float* zt;      // [T][top]
  uint16_t* g;    // [count][piece]
  float* u;       // [count][H]
  uint16_t* dw;   // [V][H]
  int v0, piece;
};

template <int MODE>
__global__ __launch_bounds__(256) void k_head_gemm(HeadGemm p) {
  __shared__ __align__(16) uint16_t sa[HB * HS], sb[HB * HS];
  __shared__ float zs[MODE == HP_STATS ? HB * (HB + 1) : 1];
  __shared__ float rm[2][HB], rs[2][HB];
  const int n = *p.count;
  const int m0 = blockIdx.y * HB, n0 = blockIdx.x * HB;
  const int M = MODE == HP_DW ? min(p.piece, p.V - p.v0) : n;
  if (m0 >= M) return;
  const int N = (MODE == HP_STATS || MODE == HP_GRAD) ? p.V : p.H;
  const int K = (MODE == HP_STATS || MODE == HP_GRAD) ? p.H : MODE == HP_DZ ? min(p.piece, p.V - p.v0) : n;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int ln = lane & 15, lg = lane >> 4;
  const int wm = (wave >> 1) * 64, wn = (wave & 1) * 64;
  f32x4 acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
  const u32x4 zero = {0, 0, 0, 0};
  for (int k0 = 0; k0 < K; k0 += HK) {
    __syncthreads();
    if (MODE == HP_STATS || MODE == HP_GRAD || MODE == HP_DZ) {  // A rows hold K contiguously
      for (int c = threadIdx.x; c < HB * HK / 8; c += 256) {
        const int m = m0 + c / (HK / 8), k = k0 + c % (HK / 8) * 8;
        u32x4 q = zero;
        if (m < M && k < K) {
          const uint16_t* src = MODE == HP_DZ ? p.g + (int64_t)m * p.piece + k
                                              : p.h + (int64_t)p.rows[m] * p.h_stride + k;
          q = *reinterpret_cast<const u32x4*>(src);
        }
        *reinterpret_cast<u32x4*>(sa + (c / (HK / 8)) * HS + c % (HK / 8) * 8) = q;
      }
    } else {
      for (int c = threadIdx.x; c < HB * HK / 8; c += 256) {
        const int k = c / (HB / 8), m = c % (HB / 8) * 8;
        u32x4 q = zero;
        if (k0 + k < K) q = *reinterpret_cast<const u32x4*>(p.g + (int64_t)(k0 + k) * p.piece + m0 + m);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          sa[(m + 2 * i) * HS + k] = (uint16_t)(q[i] & 0xFFFFu);
          sa[(m + 2 * i + 1) * HS + k] = (uint16_t)(q[i] >> 16);
        }
      }
    }
    if (MODE == HP_STATS || MODE == HP_GRAD) {
      for (int c = threadIdx.x; c < HB * HK / 8; c += 256) {
        const int v = p.v0 + n0 + c / (HK / 8), k = k0 + c % (HK / 8) * 8;
        u32x4 q = zero;
        if (v < N && k < K) q = *reinterpret_cast<const u32x4*>(p.w + (int64_t)v * p.w_stride + k);
        *reinterpret_cast<u32x4*>(sb + (c / (HK / 8)) * HS + c % (HK / 8) * 8) = q;
      }
    } else {
      for (int c = threadIdx.x; c < HB * HK / 8; c += 256) {
        const int k = c / (HB / 8), m = c % (HB / 8) * 8;
        u32x4 q = zero;
        if (k0 + k < K && n0 + m < N)
          q = *reinterpret_cast<const u32x4*>(
              (MODE == HP_DZ ? p.w + (int64_t)(p.v0 + k0 + k) * p.w_stride
                             : p.h + (int64_t)p.rows[k0 + k] * p.h_stride) + n0 + m);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          sb[(m + 2 * i) * HS + k] = (uint16_t)(q[i] & 0xFFFFu);
          sb[(m + 2 * i + 1) * HS + k] = (uint16_t)(q[i] >> 16);
        }
      }
    }
    __syncthreads();
    bf16x8 a[4], b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      a[i] = *reinterpret_cast<const bf16x8*>(sa + (wm + i * 16 + ln) * HS + lg * 8);
      b[i] = *reinterpret_cast<const bf16x8*>(sb + (wn + i * 16 + ln) * HS + lg * 8);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = mfma_bf16_16x16x32(a[i], b[j], acc[i][j]);
  }
  // accumulator [i][j][e]: row wm + 16 i + 4 lg + e, column wn + 16 j + ln
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int lr = wm + i * 16 + lg * 4 + e, c = m0 + lr;
      const bool in = c < M;
      if (MODE == HP_STATS) {
        const float f = in ? p.scale * p.r[p.rows[c]] : 0.0f;
        float z[4], mx = -INFINITY, s = 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          z[j] = n0 + wn + j * 16 + ln < N ? acc[i][j][e] * f : -INFINITY;
          zs[lr * (HB + 1) + wn + j * 16 + ln] = z[j];
          mx = fmaxf(mx, z[j]);
        }
#pragma unroll
        for (int x = 1; x < 16; x <<= 1) mx = fmaxf(mx, shfl_xor(mx, x));
#pragma unroll
        for (int j = 0; j < 4; ++j) s += n0 + wn + j * 16 + ln < N ? expf(z[j] - mx) : 0.0f;
#pragma unroll
        for (int x = 1; x < 16; x <<= 1) s += shfl_xor(s, x);
        if (ln == 0) {
          rm[wave & 1][lr] = mx;
          rs[wave & 1][lr] = s;
        }
      } else if (in) {
        if (MODE == HP_GRAD) {
          const int t = p.rows[c];
          const float f = p.scale * p.r[t], l = p.lse[t], cf = f * p.dloss[t];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int v = n0 + wn + j * 16 + ln;
            if (v < p.piece)
              p.g[(int64_t)c * p.piece + v] =
                  p.v0 + v < N ? (uint16_t)f32_to_bf16_bits(cf * expf(acc[i][j][e] * f - l)) : 0;
          }
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int v = n0 + wn + j * 16 + ln;
            if (v >= N) continue;
            if (MODE == HP_DZ) {
              float* o = p.u + (int64_t)c * p.H + v;
              *o = p.v0 == 0 ? acc[i][j][e] : *o + acc[i][j][e];
            } else {
              p.dw[(int64_t)(p.v0 + c) * p.H + v] = (uint16_t)f32_to_bf16_bits(acc[i][j][e]);
            }
          }
        }
      }
    }
  if (MODE == HP_STATS) {
    __syncthreads();
    if (threadIdx.x < HB && m0 + (int)threadIdx.x < M) {
      const int lr = threadIdx.x;
      float m = rm[0][lr], s = rs[0][lr];
      hl_merge(m, s, rm[1][lr], rs[1][lr]);
      float* o = p.stats + ((int64_t)(m0 + lr) * gridDim.x + blockIdx.x) * 2;
      o[0] = m;
      o[1] = s;
    }
    for (int q = threadIdx.x; q < HB * p.top; q += 256) {
      const int lr = q / p.top;
      if (m0 + lr >= M) break;
      const int64_t at = (int64_t)p.rows[m0 + lr] * p.top + q % p.top;
      const int v = p.ids[at] - n0;
      if (v >= 0 && v < HB && n0 + v < N) p.zt[at] = zs[lr * (HB + 1) + v];
    }
  }
}

// Per token (one wave): joins its blocks' statistics and forms the outputs.
__global__ __launch_bounds__(256) void k_head_finish(const float* __restrict__ stats, const float* __restrict__ zt,
                                                     const int32_t* __restrict__ cidx,
                                                     const int32_t* __restrict__ ids, const float* __restrict__ lq,
                                                     int T, int V, int nvb, int top, bool distill,
                                                     float* __restrict__ loss, float* __restrict__ lse,
                                                     float* __restrict__ logp) {
  const int t = blockIdx.x * 4 + (threadIdx.x >> 6), lane = threadIdx.x & 63;
  if (t >= T) return;
  const int c = cidx[t];
  if (c < 0) {
    if (distill)
      for (int j = lane; j < top; j += 64) logp[(int64_t)t * top + j] = 0.0f;
    if (lane == 0) {
      loss[t] = !distill && ids[t] >= V ? __builtin_nanf("") : 0.0f;
      lse[t] = 0.0f;
    }
    return;
  }
  float m = -INFINITY, s = 0.0f;
  for (int b = lane; b < nvb; b += 64) {
    const float* o = stats + ((int64_t)c * nvb + b) * 2;
    hl_merge(m, s, o[0], o[1]);
  }
#pragma unroll
  for (int x = 1; x < 64; x <<= 1) {
    const float m2 = shfl_xor(m, x), s2 = shfl_xor(s, x);
    hl_merge(m, s, m2, s2);
  }
  const float l = m + logf(s);
  float kl;
  if (distill) {
    kl = 0.0f;
    for (int j = lane; j < top; j += 64) {
      const int64_t at = (int64_t)t * top + j;
      const float q = lq[at];
      const bool have = !(q == -INFINITY);
      const float lp = have ? zt[at] - l : 0.0f;
      logp[at] = lp;
      if (have) kl = fmaf(expf(q), q - lp, kl);
    }
    kl = hl_sum64(kl);
  } else {
    kl = l - zt[t];
  }
  if (lane == 0) {
    loss[t] = kl;
    lse[t] = l;
  }
}

// Backward: G at the target's ids in [v0, v0 + piece), from the forward's
// log-probs: s r g (p - q), one wave per counted token.  Slots that repeat an
// id add their q, and the first of them writes.
__global__ __launch_bounds__(256) void k_head_targets(const int32_t* __restrict__ rows, const int32_t* __restrict__ count,
                                                      const int32_t* __restrict__ ids, const float* __restrict__ lq,
                                                      const float* __restrict__ logp, const float* __restrict__ loss,
                                                      const float* __restrict__ r, const float* __restrict__ dloss,
                                                      float scale, int V, int top, int v0, int piece,
                                                      uint16_t* __restrict__ g) {
  __shared__ int sid[4][256];
  __shared__ float sq[4][256];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int c = blockIdx.x * 4 + wave;
  if (c >= *count) return;
  const int t = rows[c];
  const float cf = scale * r[t] * dloss[t];
  if (lq == nullptr) {  // cross entropy: p - 1 = exp(-loss) - 1
    const int v = ids[t] - v0;
    if (lane == 0 && v >= 0 && v < piece)
      g[(int64_t)c * piece + v] = (uint16_t)f32_to_bf16_bits(cf * expm1f(-loss[t]));
    return;
  }
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
    if (id < 0 || v < 0 || v >= piece) continue;
    float q = 0.0f;
    bool first = true;
    for (int i = 0; i < top; ++i)
      if (sid[wave][i] == id) {
        q += sq[wave][i];
        if (i < j) first = false;
      }
    if (first) g[(int64_t)c * piece + v] = (uint16_t)f32_to_bf16_bits(cf * (expf(logp[(int64_t)t * top + j]) - q));
  }
}

// d_h = u - r^2 h mean(h u), or u without a norm; zeros for tokens that do
// not count.  One block per token.
__global__ __launch_bounds__(256) void k_head_dh(const float* __restrict__ u, const uint16_t* __restrict__ h,
                                                 int64_t h_stride, const int32_t* __restrict__ cidx,
                                                 const float* __restrict__ r, int H, bool norm,
                                                 uint16_t* __restrict__ dh) {
  __shared__ float part[4];
  const int t = blockIdx.x, c = cidx[t];
  uint16_t* o = dh + (int64_t)t * H;
  if (c < 0) {
    for (int i = threadIdx.x; i < H / 8; i += 256) *reinterpret_cast<u32x4*>(o + i * 8) = (u32x4){0, 0, 0, 0};
    return;
  }
  const float* ur = u + (int64_t)c * H;
  const uint16_t* hr = h + (int64_t)t * h_stride;
  float f = 0.0f;
  if (norm) {
    float dot = 0.0f;
    for (int i = threadIdx.x; i < H; i += 256) dot = fmaf(ur[i], bf16_bits_to_f32(hr[i]), dot);
    dot = hl_sum64(dot);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = dot;
    __syncthreads();
    f = r[t] * r[t] * ((part[0] + part[1]) + (part[2] + part[3])) / (float)H;
  }
  for (int i = threadIdx.x; i < H / 8; i += 256) {
    const f32x4 a = *reinterpret_cast<const f32x4*>(ur + i * 8), b = *reinterpret_cast<const f32x4*>(ur + i * 8 + 4);
    u32x4 q = {0, 0, 0, 0};
    if (norm) q = *reinterpret_cast<const u32x4*>(hr + i * 8);  // without a norm f = 0 and h is not read
    u32x4 x;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float lo = j < 2 ? a[2 * j] : b[2 * j - 4], hi = j < 2 ? a[2 * j + 1] : b[2 * j - 3];
      x[j] = bf16x2_bits(fmaf(-f, bf16_bits_to_f32(q[j] & 0xFFFFu), lo), fmaf(-f, bf16_bits_to_f32(q[j] >> 16), hi));
    }
    *reinterpret_cast<u32x4*>(o + i * 8) = x;
  }
}

namespace {
inline int cdiv(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }
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
  const size_t t = (size_t)T;
  p.r = take(t * 4);
  p.flag = take(t);
  p.rows = take(t * 4);
  p.cidx = take(t * 4);
  p.count = take(4);
  p.lq = take(distill ? t * top * 4 : 0);
  if (!bwd) {
    p.zt = take(t * top * 4);
    p.stats = take(t * cdiv(V, HB) * 8);
  } else {
    // columns of G per piece: 256 MB of G, at least 256 columns
    const int64_t most = T > 0 ? ((int64_t)128 << 20) / T / 256 * 256 : V;
    p.npieces = cdiv(V, most > 256 ? most : 256);
    p.piece = cdiv(cdiv(V, p.npieces), 256) * 256;
    p.npieces = cdiv(V, p.piece);
    p.u = take(t * H * 4);
    p.g = take(t * p.piece * 2);
  }
  p.total = o;
  return p;
}

static HeadGemm head_common(const HeadPlan& p, const HeadArgs& a, hipStream_t s) {
  char* ws = a.ws;
  float* r = reinterpret_cast<float*>(ws + p.r);
  uint8_t* flag = reinterpret_cast<uint8_t*>(ws + p.flag);
  int32_t* rows = reinterpret_cast<int32_t*>(ws + p.rows);
  int32_t* cidx = reinterpret_cast<int32_t*>(ws + p.cidx);
  int32_t* count = reinterpret_cast<int32_t*>(ws + p.count);
  float* lq = p.distill ? reinterpret_cast<float*>(ws + p.lq) : nullptr;
  hipLaunchKernelGGL(k_head_rows, dim3(cdiv(p.T, 4)), dim3(256), 0, s, a.h, a.h_stride, p.T, p.H, p.V, a.eps, a.ids,
                     p.top, a.tlogits, a.teacher_scale, r, flag, lq);
  hipLaunchKernelGGL(k_head_compact, dim3(1), dim3(1024), 0, s, flag, p.T, rows, cidx, count);
  HeadGemm g{};
  g.h = a.h;
  g.w = a.w;
  g.h_stride = a.h_stride;
  g.w_stride = a.w_stride;
  g.H = p.H;
  g.V = p.V;
  g.top = p.top;
  g.rows = rows;
  g.count = count;
  g.r = r;
  g.lse = a.lse;
  g.dloss = a.dloss;
  g.scale = a.scale;
  g.ids = a.ids;
  g.dw = a.dw;
  return g;
}

void launch_head_loss(const HeadPlan& p, const HeadArgs& a, hipStream_t s) {
  HeadGemm g = head_common(p, a, s);
  const int nvb = cdiv(p.V, HB);
  g.stats = reinterpret_cast<float*>(a.ws + p.stats);
  g.zt = reinterpret_cast<float*>(a.ws + p.zt);
  hipLaunchKernelGGL(k_head_gemm<HP_STATS>, dim3(nvb, cdiv(p.T, HB)), dim3(256), 0, s, g);
  hipLaunchKernelGGL(k_head_finish, dim3(cdiv(p.T, 4)), dim3(256), 0, s, g.stats, g.zt,
                     reinterpret_cast<const int32_t*>(a.ws + p.cidx), a.ids,
                     reinterpret_cast<const float*>(a.ws + p.lq), p.T, p.V, nvb, p.top, p.distill, a.loss, a.lse,
                     a.logp);
}

void launch_head_loss_bwd(const HeadPlan& p, const HeadArgs& a, hipStream_t s) {
  HeadGemm g = head_common(p, a, s);
  g.u = reinterpret_cast<float*>(a.ws + p.u);
  g.g = reinterpret_cast<uint16_t*>(a.ws + p.g);
  g.piece = p.piece;
  const int mb = cdiv(p.T, HB), hb = cdiv(p.H, HB);
  for (int i = 0; i < p.npieces; ++i) {
    g.v0 = i * p.piece;
    hipLaunchKernelGGL(k_head_gemm<HP_GRAD>, dim3(p.piece / HB, mb), dim3(256), 0, s, g);
    hipLaunchKernelGGL(k_head_targets, dim3(cdiv(p.T, 4)), dim3(256), 0, s, g.rows, g.count, a.ids,
                       p.distill ? reinterpret_cast<const float*>(a.ws + p.lq) : nullptr, a.logp, a.loss, g.r,
                       a.dloss, a.scale, p.V, p.top, g.v0, p.piece, g.g);
    hipLaunchKernelGGL(k_head_gemm<HP_DZ>, dim3(hb, mb), dim3(256), 0, s, g);
    if (a.dw != nullptr) hipLaunchKernelGGL(k_head_gemm<HP_DW>, dim3(hb, p.piece / HB), dim3(256), 0, s, g);
  }
  hipLaunchKernelGGL(k_head_dh, dim3(p.T), dim3(256), 0, s, g.u, a.h, a.h_stride,
                     reinterpret_cast<const int32_t*>(a.ws + p.cidx), g.r, p.H, a.eps > 0.0f, a.dh);
}

}  // namespace moe
