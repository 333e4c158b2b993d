// The global norm of a list of tensors and their clipping by it.
//
//   norm = sqrt(sum of g^2 over every element of every tensor)
//   out  = g max_norm / norm  where norm > max_norm (and finite), else g
//
// Squares are formed and added in 64 bits: in 32 they overflow from 1.8e19 on,
// vanish below 1e-23 and drift over long sums.  A launch takes a list of up to
// CLIP_TENSORS tensors as its argument, cut into chunks that the blocks share;
// which block adds what in which order is fixed by the sizes, so the norm is the
// same in every run.
//
// Memory bounds both passes, each of which reads everything, the second also
// writing it: 478 MB of fp32 and bf16 272 us, 299 at a large copy's rate (the end of
// the list stays in the last-level cache between the passes).  Few elements are
// bound by the call: 2 million 15.5 us, 4 + 6 on the GPU.
#include "common.h"
#include "kernels.h"
#include "moe_lp.h"

namespace moe {

namespace {

constexpr int CLIP_BYTES = 32768;  // of a chunk

MOE_DEV float f16_bits_to_f32(uint32_t b) { return (float)__builtin_bit_cast(_Float16, (uint16_t)b); }

// 16 bytes of a tensor as floats and back.
template <int DT>
struct ClipVec {
  static constexpr int N = DT == MOE_DTYPE_F32 ? 4 : 8, SIZE = DT == MOE_DTYPE_F32 ? 4 : 2;
  MOE_DEV static float get(const u32x4& v, int i) {
    if constexpr (DT == MOE_DTYPE_F32) return __uint_as_float(v[i]);
    const uint32_t h = (v[i >> 1] >> (16 * (i & 1))) & 0xFFFFu;
    return DT == MOE_DTYPE_BF16 ? bf16_bits_to_f32(h) : f16_bits_to_f32(h);
  }
  MOE_DEV static uint32_t bits(float f) {
    if constexpr (DT == MOE_DTYPE_F32) return __float_as_uint(f);
    else if constexpr (DT == MOE_DTYPE_BF16) return f32_to_bf16_bits(f);
    else return __builtin_bit_cast(uint16_t, (_Float16)f);
  }
  MOE_DEV static float load(const void* p, int64_t i) {
    if constexpr (DT == MOE_DTYPE_F32) return static_cast<const float*>(p)[i];
    const uint32_t h = static_cast<const uint16_t*>(p)[i];
    return DT == MOE_DTYPE_BF16 ? bf16_bits_to_f32(h) : f16_bits_to_f32(h);
  }
  MOE_DEV static void store(void* p, int64_t i, float f) {
    if constexpr (DT == MOE_DTYPE_F32) static_cast<float*>(p)[i] = f;
    else static_cast<uint16_t*>(p)[i] = (uint16_t)bits(f);
  }
  MOE_DEV static u32x4 scaled(const u32x4& v, float c) {
    u32x4 o;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (DT == MOE_DTYPE_F32) o[i] = bits(get(v, i) * c);
      else o[i] = bits(get(v, 2 * i) * c) | (bits(get(v, 2 * i + 1) * c) << 16);
    }
    return o;
  }
};

// Chunk `at` of the launch's list: its tensor, first element and length.
struct ClipChunk {
  int t;
  int64_t first;
  int n;
};
MOE_DEV ClipChunk clip_chunk(const ClipList& l, int at) {
  int lo = 0, hi = l.n - 1;  // last tensor whose first chunk is at or before `at`
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (l.t[mid].chunk0 <= at) lo = mid; else hi = mid - 1;
  }
  const int len = CLIP_BYTES / (l.t[lo].dtype == MOE_DTYPE_F32 ? 4 : 2);
  ClipChunk c;
  c.t = lo;
  c.first = (int64_t)(at - l.t[lo].chunk0) * len;
  c.n = (int)min((int64_t)len, l.t[lo].n - c.first);
  return c;
}

template <int DT>
MOE_DEV double clip_squares(const void* p, int64_t first, int n) {
  using V = ClipVec<DT>;
  double s = 0.0;
  const char* q = static_cast<const char*>(p) + first * V::SIZE;
  const int nv = ((uintptr_t)q & 15) == 0 ? n / V::N : 0;
  const u32x4* v = reinterpret_cast<const u32x4*>(q);
#pragma unroll 4
  for (int i = threadIdx.x; i < nv; i += 256) {
    const u32x4 x = v[i];
#pragma unroll
    for (int j = 0; j < V::N; ++j) {
      const double f = (double)V::get(x, j);
      s = fma(f, f, s);
    }
  }
  for (int i = nv * V::N + threadIdx.x; i < n; i += 256) {
    const double f = (double)V::load(q, i);
    s = fma(f, f, s);
  }
  return s;
}

template <int DT>
MOE_DEV void clip_scale(const void* p, void* out, int64_t first, int n, float c) {
  using V = ClipVec<DT>;
  const char* q = static_cast<const char*>(p) + first * V::SIZE;
  char* o = static_cast<char*>(out) + first * V::SIZE;
  const int nv = (((uintptr_t)q | (uintptr_t)o) & 15) == 0 ? n / V::N : 0;
  const u32x4* v = reinterpret_cast<const u32x4*>(q);
  u32x4* w = reinterpret_cast<u32x4*>(o);
#pragma unroll 4
  for (int i = threadIdx.x; i < nv; i += 256) w[i] = V::scaled(v[i], c);
  for (int i = nv * V::N + threadIdx.x; i < n; i += 256) V::store(o, i, V::load(q, i) * c);
}

// Sum over the block, in every thread.
MOE_DEV double clip_block_sum(double s, double* sh) {
#pragma unroll
  for (int x = 1; x < 64; x <<= 1) s += __shfl_xor(s, x, 64);
  if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = s;
  __syncthreads();
  s = (sh[0] + sh[1]) + (sh[2] + sh[3]);
  __syncthreads();
  return s;
}

MOE_DEV double clip_total(const double* parts, int nparts, double* sh) {
  double s = 0.0;
  for (int i = threadIdx.x; i < nparts; i += 256) s += parts[i];
  return clip_block_sum(s, sh);
}

}  // namespace

int64_t clip_chunks(int64_t elems, int dtype) {
  const int64_t len = CLIP_BYTES / (dtype == MOE_DTYPE_F32 ? 4 : 2);
  return (elems + len - 1) / len;
}

// Four 16-byte loads per thread ahead of the sums; 86-111 us for 478 MB.
__global__ __launch_bounds__(256) void k_norm_parts(ClipList l, double* __restrict__ parts) {
  __shared__ double sh[4];
  double s = 0.0;
  for (int at = blockIdx.x; at < l.chunks; at += gridDim.x) {
    const ClipChunk c = clip_chunk(l, at);
    const ClipTensor& t = l.t[c.t];
    if (t.dtype == MOE_DTYPE_F32) s += clip_squares<MOE_DTYPE_F32>(t.p, c.first, c.n);
    else if (t.dtype == MOE_DTYPE_BF16) s += clip_squares<MOE_DTYPE_BF16>(t.p, c.first, c.n);
    else s += clip_squares<MOE_DTYPE_F16>(t.p, c.first, c.n);
  }
  s = clip_block_sum(s, sh);
  if (threadIdx.x == 0) parts[blockIdx.x] = s;
}

__global__ __launch_bounds__(256) void k_norm_finish(const double* __restrict__ parts, int nparts,
                                                     float* __restrict__ norm) {
  __shared__ double sh[4];
  const double s = clip_total(parts, nparts, sh);
  if (threadIdx.x == 0) *norm = (float)sqrt(s);
}

// The chunks are taken last to first: the last ones read by the norm are those
// that the last-level cache still holds.  157 us for 478 MB read and written.
__global__ __launch_bounds__(256) void k_clip(ClipList l, const double* __restrict__ parts, int nparts, float* norm,
                                              int write, float max_norm) {
  __shared__ double sh[4];
  double n;
  if (nparts > 0) {
    n = sqrt(clip_total(parts, nparts, sh));
    if (write && blockIdx.x == 0 && threadIdx.x == 0) *norm = (float)n;
  } else {
    n = (double)*norm;
  }
  // not finite: also a norm past fp32's range, which the caller sees as infinite
  const bool clip = n > (double)max_norm && (float)n < INFINITY;
  const float c = clip ? (float)((double)max_norm / n) : 1.0f;
  for (int at = l.chunks - 1 - (int)blockIdx.x; at >= 0; at -= (int)gridDim.x) {
    const ClipChunk k = clip_chunk(l, at);
    const ClipTensor& t = l.t[k.t];
    if (!clip && t.p == t.out) continue;
    if (t.dtype == MOE_DTYPE_F32) clip_scale<MOE_DTYPE_F32>(t.p, t.out, k.first, k.n, c);
    else if (t.dtype == MOE_DTYPE_BF16) clip_scale<MOE_DTYPE_BF16>(t.p, t.out, k.first, k.n, c);
    else clip_scale<MOE_DTYPE_F16>(t.p, t.out, k.first, k.n, c);
  }
}

static int clip_grid(const ClipList& l) { return l.chunks < CLIP_BLOCKS ? l.chunks : CLIP_BLOCKS; }

int launch_norm_parts(const ClipList& l, double* parts, hipStream_t s) {
  hipLaunchKernelGGL(k_norm_parts, dim3(clip_grid(l)), dim3(256), 0, s, l, parts);
  return clip_grid(l);
}

void launch_norm_finish(const double* parts, int nparts, float* norm, hipStream_t s) {
  hipLaunchKernelGGL(k_norm_finish, dim3(1), dim3(256), 0, s, parts, nparts, norm);
}

void launch_clip(const ClipList& l, const double* parts, int nparts, float* norm, int write, float max_norm,
                 hipStream_t s) {
  hipLaunchKernelGGL(k_clip, dim3(clip_grid(l)), dim3(256), 0, s, l, parts, nparts, norm, write, max_norm);
}

}  // namespace moe
