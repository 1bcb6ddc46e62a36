// Root-mean-square norm of a residual stream, with the residual's addition and an output in the
// storage type or in 8 bits with scales, and its gradients.
//
//   r = x + res;  y = r / sqrt(mean(r^2) + eps) * weight
//   dx = s (w dy - r s^2 mean(w dy r)) + dres,   s = 1 / sqrt(mean(r^2) + eps);   dw = sum_rows dy r s
//
// Both directions are bound by HBM: a row is read once into registers (at most kElems values a
// thread), reduced, and written once.  A row belongs to TPR threads; a block of narrow rows
// takes several at once.  Sums, scales and the weight's gradient are fp32.
#include <cuda_fp8.h>

#include "common.cuh"
#include "kernels.h"

namespace mlstm {
namespace {

constexpr int kElems = 16;     // values of a row that a thread holds
constexpr int kMaxD = 16384;   // kElems * 1024 threads
constexpr int kThreads = 256;  // block size while rows are narrow

enum { kOut = 0, kE4m3 = 1, kInt8 = 2 };

// VEC consecutive values as fp32; VEC = 1 or 16 bytes of the storage type.
template <typename T, int VEC>
__device__ __forceinline__ void load_vec(const T* __restrict__ p, float (&x)[VEC]) {
  if constexpr (VEC == 1) {
    x[0] = io<T>::load(p, 0);
  } else if constexpr (sizeof(T) == 4) {
    const float4 v = __ldcs(reinterpret_cast<const float4*>(p));
    x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
  } else {
    const uint4 v = __ldcs(reinterpret_cast<const uint4*>(p));
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(u[i] << 16);
      x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
  }
}

template <typename T, int VEC>
__device__ __forceinline__ void store_vec(T* __restrict__ p, const float (&x)[VEC]) {
  if constexpr (VEC == 1) {
    io<T>::store(p, 0, x[0]);
  } else if constexpr (sizeof(T) == 4) {
    *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
  } else {
    __nv_bfloat162 b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) b[i] = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(b);
  }
}

template <int VEC>
__device__ __forceinline__ void load_w(const float* __restrict__ p, float (&x)[VEC]) {
  if constexpr (VEC == 1) {
    x[0] = __ldg(p);
  } else {
#pragma unroll
    for (int i = 0; i < VEC; i += 4) {
      const float4 v = __ldg(reinterpret_cast<const float4*>(p + i));
      x[i] = v.x, x[i + 1] = v.y, x[i + 2] = v.z, x[i + 3] = v.w;
    }
  }
}

// Sum over the TPR threads of a row, the same value in each; red: N values a warp.  Every thread
// of the block calls it.
template <typename F, int N>
__device__ __forceinline__ void row_sum(F (&v)[N], int tpr, F (*red)[N]) {
  for (int d = min(tpr, 32) / 2; d > 0; d /= 2)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], d);
  if (tpr > 32) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = tpr >> 5, base = warp / nw * nw;
    __syncthreads();  // red is read by the row before
    if (lane == 0)
#pragma unroll
      for (int i = 0; i < N; ++i) red[warp][i] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      F s = lane < nw ? red[base + lane][i] : F(0);
#pragma unroll
      for (int d = 16; d > 0; d /= 2) s += __shfl_xor_sync(0xffffffffu, s, d);
      v[i] = s;
    }
  }
}

// Whether fp32 held the sum of squares: ms = mean(r^2) + eps is neither so large that a square may
// have overflowed nor so small that the squares have vanished (nor NaN).
__device__ __forceinline__ bool in_range(float ms) { return ms > 1e-30f && ms < 1e34f; }

// The rows of the block for which fp32 did not: v becomes r / sqrt(mean(r^2) + eps) from sums in 64
// bits, which hold the squares of every fp32 value.  Every thread of the block calls it.
template <int NV, int VEC>
__device__ __noinline__ double normalise_wide(float (&v)[NV][VEC], float eps, int D, int tpr) {
  __shared__ double red[32][1];
  double s[1] = {0.0};
  for (int i = 0; i < NV; ++i)
    for (int e = 0; e < VEC; ++e) s[0] += (double)v[i][e] * v[i][e];
  row_sum<double, 1>(s, tpr, red);
  const double inv = 1.0 / sqrt(s[0] / D + eps);
  for (int i = 0; i < NV; ++i)
    for (int e = 0; e < VEC; ++e) v[i][e] = (float)(v[i][e] * inv);
  return inv;
}

// |x| as an unsigned integer: ordered like |x|, with NaN above infinity, so that a maximum keeps it.
__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// VEC values, already divided by their scale, in 8 bits.  NaN stays NaN in e4m3 and gives -127 as an
// integer (its scale is NaN).
template <int KIND, int VEC>
__device__ __forceinline__ void to8(const float (&z)[VEC], uint8_t (&q)[VEC]) {
  if constexpr (KIND == kInt8) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) q[e] = (uint8_t)(int8_t)__float2int_rn(fminf(fmaxf(z[e], -127.f), 127.f));
  } else if constexpr (VEC == 1) {
    q[0] = (uint8_t)__nv_cvt_float_to_fp8(z[0], __NV_SATFINITE, __NV_E4M3);
  } else {
#pragma unroll
    for (int e = 0; e < VEC; e += 2) {
      const uint16_t two = __nv_cvt_float2_to_fp8x2(make_float2(z[e], z[e + 1]), __NV_SATFINITE, __NV_E4M3);
      q[e] = (uint8_t)two, q[e + 1] = (uint8_t)(two >> 8);
    }
  }
}

// Grid: ceil(rows / rows a block).  group: channels that share a scale (D: the whole row).  A group
// of 128 is 128 / VEC neighbouring lanes of one warp; odd widths (VEC 1) meet in shared memory.
template <typename T, int VEC, int KIND, int BLOCK>
__global__ void __launch_bounds__(BLOCK) rms_norm_kernel(const T* x, const T* res, const float* __restrict__ weight,
                                                        float eps, T* r_out, void* y, float* __restrict__ scales,
                                                        long long rows, int D, int tpr, int group) {
  constexpr int NV = kElems / VEC;
  __shared__ float red[32][1];
  __shared__ uint32_t gmax[KIND == kOut ? 1 : 128];
  const int t = threadIdx.x % tpr, sub = threadIdx.x / tpr;
  const long long row = (long long)blockIdx.x * (blockDim.x / tpr) + sub;
  const bool live = row < rows;  // dead rows of the last block still take part in the shuffles
  const size_t base = live ? (size_t)row * D : 0;
  float v[NV][VEC];
  float s[1] = {0.f};
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * tpr + t) * VEC;
#pragma unroll
    for (int e = 0; e < VEC; ++e) v[i][e] = 0.f;
    if (live && c < D) load_vec<T, VEC>(x + base + c, v[i]);
  }
  if (res) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * tpr + t) * VEC;
      if (live && c < D) {
        float a[VEC];
        load_vec<T, VEC>(res + base + c, a);
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[i][e] += a[e];
        store_vec<T, VEC>(r_out + base + c, v[i]);  // this thread's own elements: r_out may be res
      }
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int e = 0; e < VEC; ++e) s[0] = fmaf(v[i][e], v[i][e], s[0]);
  row_sum<float, 1>(s, tpr, red);
  // the norm reads the sum before it is rounded to the storage type
  const float ms = s[0] / (float)D + eps;
  float inv = 1.f / sqrtf(ms);
  if (__syncthreads_or(!in_range(ms))) {  // a block's rows together: the wide sums meet at barriers
    normalise_wide<NV, VEC>(v, eps, D, tpr);
    inv = 1.f;
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * tpr + t) * VEC;
    if (live && c < D) {
      float w[VEC];
      if (weight) load_w<VEC>(weight + c, w);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        v[i][e] *= inv;
        if (weight) v[i][e] *= w[e];
      }
      if constexpr (KIND == kOut) store_vec<T, VEC>(reinterpret_cast<T*>(y) + base + c, v[i]);
    }
  }
  if constexpr (KIND != kOut) {
    constexpr float kTop = KIND == kE4m3 ? 448.f : 127.f;
    const int ngroups = (D + group - 1) / group;
    uint32_t m[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      m[i] = 0;
#pragma unroll
      for (int e = 0; e < VEC; ++e) m[i] = max(m[i], abs_bits(v[i][e]));
    }
    if (group == D) {  // one maximum for the row
#pragma unroll
      for (int i = 1; i < NV; ++i) m[0] = max(m[0], m[i]);
      for (int d = min(tpr, 32) / 2; d > 0; d /= 2) m[0] = max(m[0], __shfl_xor_sync(0xffffffffu, m[0], d));
      if (tpr > 32) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = tpr >> 5;
        if (lane == 0) gmax[warp] = m[0];
        __syncthreads();
        m[0] = __reduce_max_sync(0xffffffffu, lane < nw ? gmax[warp / nw * nw + lane] : 0u);
      }
#pragma unroll
      for (int i = 1; i < NV; ++i) m[i] = m[0];
    } else if constexpr (VEC > 1) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int d = 64 / VEC; d > 0; d /= 2) m[i] = max(m[i], __shfl_xor_sync(0xffffffffu, m[i], d));
    } else {  // one row a block: the launcher gives odd widths with groups tpr >= 64
      for (int i = threadIdx.x; i < ngroups; i += blockDim.x) gmax[i] = 0;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = i * tpr + t;
        if (live && c < D) atomicMax(&gmax[c / group], m[i]);  // a maximum: the order does not matter
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < NV; ++i) m[i] = i * tpr + t < D ? gmax[(i * tpr + t) / group] : 0;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * tpr + t) * VEC;
      if (live && c < D) {
        const float amax = __uint_as_float(m[i]);
        const float scale = m[i] == 0 ? 1.f : amax / kTop;
        if (c % group == 0) scales[(size_t)row * ngroups + c / group] = scale;
        // one reciprocal for the group; where it could leave fp32's range the quotient itself
        const float inv_scale = kTop / amax;
        const bool tiny = amax < 1e-30f;
        float z[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) z[e] = m[i] == 0 ? v[i][e] : tiny ? v[i][e] / scale : v[i][e] * inv_scale;
        uint8_t q[VEC];
        to8<KIND, VEC>(z, q);
        uint8_t* out = reinterpret_cast<uint8_t*>(y) + base + c;
        if constexpr (VEC == 8) {
          *reinterpret_cast<uint2*>(out) = *reinterpret_cast<const uint2*>(q);
        } else if constexpr (VEC == 4) {
          *reinterpret_cast<uint32_t*>(out) = *reinterpret_cast<const uint32_t*>(q);
        } else {
          out[0] = q[0];
        }
      }
    }
  }
}

// Gradients.  A block walks rows blockIdx.x, + gridDim.x, ... so that a thread meets the same
// channels every time and keeps their share of the weight's gradient in registers; part: one row
// of D sums a block, added up in order by rms_norm_dw_kernel.
template <typename T, int VEC, int BLOCK>
__global__ void __launch_bounds__(BLOCK) rms_norm_bwd_kernel(const T* dy, const T* __restrict__ r,
                                                            const float* __restrict__ weight, float eps, const T* dres,
                                                            T* dx, float* __restrict__ part, long long rows, int D,
                                                            int tpr) {
  constexpr int NV = kElems / VEC;
  extern __shared__ float sums[];  // [rows a block][D] when a block takes several rows
  __shared__ float red[32][2];
  const int t = threadIdx.x % tpr, sub = threadIdx.x / tpr, rpb = blockDim.x / tpr;
  float dw[NV][VEC];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int e = 0; e < VEC; ++e) dw[i][e] = 0.f;
  for (long long r0 = (long long)blockIdx.x * rpb; r0 < rows; r0 += (long long)gridDim.x * rpb) {
    const long long row = r0 + sub;
    const bool live = row < rows;
    const size_t base = live ? (size_t)row * D : 0;
    float a[NV][VEC], d[NV][VEC];
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * tpr + t) * VEC;
#pragma unroll
      for (int e = 0; e < VEC; ++e) a[i][e] = d[i][e] = 0.f;
      if (live && c < D) {
        load_vec<T, VEC>(r + base + c, a[i]);
        load_vec<T, VEC>(dy + base + c, d[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * tpr + t) * VEC;
      float w[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) w[e] = 1.f;
      if (weight && c < D) load_w<VEC>(weight + c, w);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        s[0] = fmaf(a[i][e], a[i][e], s[0]);
        s[1] = fmaf(a[i][e], d[i][e] * w[e], s[1]);
      }
    }
    row_sum<float, 2>(s, tpr, red);
    const float ms = s[0] / (float)D + eps;
    float inv = 1.f / sqrtf(ms), scale = inv;  // scale takes r to n = r s where a still holds r
    float along = s[1] / (float)D * inv;       // mean(w dy n)
    if (__syncthreads_or(!in_range(ms))) {
      inv = (float)normalise_wide<NV, VEC>(a, eps, D, tpr);
      scale = 1.f;
      s[1] = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * tpr + t) * VEC;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float w = weight && c < D ? weight[c + e] : 1.f;
          s[1] = fmaf(a[i][e], d[i][e] * w, s[1]);
        }
      }
      row_sum<float, 2>(s, tpr, red);
      along = s[1] / (float)D;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * tpr + t) * VEC;
      if (live && c < D) {
        float w[VEC], out[VEC], add[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) w[e] = 1.f, add[e] = 0.f;
        if (weight) load_w<VEC>(weight + c, w);
        if (dres) load_vec<T, VEC>(dres + base + c, add);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float n = a[i][e] * scale;
          out[e] = fmaf(inv, d[i][e] * w[e] - n * along, add[e]);
          dw[i][e] = fmaf(d[i][e], n, dw[i][e]);
        }
        store_vec<T, VEC>(dx + base + c, out);  // dx may be dy or dres: this thread's own elements
      }
    }
  }
  if (!part) return;
  float* mine = rpb > 1 ? sums + (size_t)sub * D : part + (size_t)blockIdx.x * D;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * tpr + t) * VEC;
    if (c < D)
#pragma unroll
      for (int e = 0; e < VEC; ++e) mine[c + e] = dw[i][e];
  }
  if (rpb > 1) {
    __syncthreads();
    for (int c = threadIdx.x; c < D; c += blockDim.x) {
      float v = 0.f;
      for (int i = 0; i < rpb; ++i) v += sums[(size_t)i * D + c];
      part[(size_t)blockIdx.x * D + c] = v;
    }
  }
}

// dw[c] = sum of n rows of part, in order: 32 channels a block, 32 partial sums each.
__global__ void __launch_bounds__(1024) rms_norm_dw_kernel(const float* __restrict__ part, int n, int D, float* dw) {
  __shared__ float s[32][33];
  const int c = blockIdx.x * 32 + threadIdx.x;
  float v = 0.f;
  if (c < D)
    for (int i = threadIdx.y; i < n; i += 32) v += part[(size_t)i * D + c];
  s[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  v = s[threadIdx.x][threadIdx.y];
#pragma unroll
  for (int d = 16; d > 0; d /= 2) v += __shfl_xor_sync(0xffffffffu, v, d);
  if (threadIdx.x == 0 && blockIdx.x * 32 + threadIdx.y < D) dw[blockIdx.x * 32 + threadIdx.y] = v;
}

int vec_of(int D, int dtype) {
  const int v = dtype ? 8 : 4;
  return D % v == 0 ? v : 1;
}
// Threads of a row: a power of two with at most kElems values each.  least: the fewest allowed.
int row_threads(int D, int least) {
  int t = least;
  while (t * kElems < D) t *= 2;
  return t;
}

// Two blocks for each of 148 SMs, whatever the device: the workspace's size follows from it.
int bwd_blocks(long long rows, int rpb) {
  const long long need = (rows + rpb - 1) / rpb;
  return (int)(need < 296 ? need : 296);
}

template <typename T, int VEC, int BLOCK>
cudaError_t fwd_block(const RmsArgs& a, int tpr, int block, cudaStream_t stream) {
  const long long rpb = block / tpr;
  const unsigned grid = (unsigned)((a.rows + rpb - 1) / rpb);
#define MLSTM_RMS(KIND)                                                                                        \
  rms_norm_kernel<T, VEC, KIND, BLOCK><<<grid, block, 0, stream>>>((const T*)a.x, (const T*)a.res, a.weight,   \
                                                                   a.eps, (T*)a.r_out, a.y, a.scales, a.rows, \
                                                                   a.D, tpr, a.group)
  if (a.kind == kOut)
    MLSTM_RMS(kOut);
  else if (a.kind == kE4m3)
    MLSTM_RMS(kE4m3);
  else
    MLSTM_RMS(kInt8);
#undef MLSTM_RMS
  return cudaGetLastError();
}

template <typename T, int VEC>
cudaError_t fwd_kind(const RmsArgs& a, cudaStream_t stream) {
  const bool odd_groups = VEC == 1 && a.kind != kOut && a.group < a.D;
  // groups of 128 channels lie inside one warp: 16 or 32 lanes of a row at least
  const int tpr = row_threads(a.D, odd_groups ? kThreads : 32);
  return tpr <= kThreads ? fwd_block<T, VEC, kThreads>(a, tpr, kThreads, stream)
                         : fwd_block<T, VEC, 1024>(a, tpr, tpr, stream);
}

template <typename T, int VEC, int BLOCK>
cudaError_t bwd_block(const RmsArgs& a, int tpr, int block, cudaStream_t stream) {
  const int rpb = block / tpr, grid = bwd_blocks(a.rows, rpb);
  const size_t smem = rpb > 1 && a.dweight ? sizeof(float) * rpb * a.D : 0;  // at most 8 rows of 512
  rms_norm_bwd_kernel<T, VEC, BLOCK><<<grid, block, smem, stream>>>(
      (const T*)a.dy, (const T*)a.x, a.weight, a.eps, (const T*)a.res, (T*)a.y, a.dweight ? a.part : nullptr, a.rows,
      a.D, tpr);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !a.dweight) return e;
  rms_norm_dw_kernel<<<(a.D + 31) / 32, dim3(32, 32), 0, stream>>>(a.part, grid, a.D, a.dweight);
  return cudaGetLastError();
}

template <typename T, int VEC>
cudaError_t bwd_kind(const RmsArgs& a, cudaStream_t stream) {
  const int tpr = row_threads(a.D, 32);
  return tpr <= kThreads ? bwd_block<T, VEC, kThreads>(a, tpr, kThreads, stream)
                         : bwd_block<T, VEC, 1024>(a, tpr, tpr, stream);
}

}  // namespace

bool rms_norm_supported(int D) { return D >= 1 && D <= kMaxD; }

size_t rms_norm_bwd_workspace_bytes(long long rows, int D) {
  const int tpr = row_threads(D, 32);
  return sizeof(float) * (size_t)bwd_blocks(rows, tpr < kThreads ? kThreads / tpr : 1) * D;
}

cudaError_t launch_rms_norm(const RmsArgs& a, cudaStream_t stream) {
  const int vec = vec_of(a.D, a.dtype);
  if (a.dtype) return vec > 1 ? fwd_kind<__nv_bfloat16, 8>(a, stream) : fwd_kind<__nv_bfloat16, 1>(a, stream);
  return vec > 1 ? fwd_kind<float, 4>(a, stream) : fwd_kind<float, 1>(a, stream);
}

cudaError_t launch_rms_norm_bwd(const RmsArgs& a, cudaStream_t stream) {
  const int vec = vec_of(a.D, a.dtype);
  if (a.dtype) return vec > 1 ? bwd_kind<__nv_bfloat16, 8>(a, stream) : bwd_kind<__nv_bfloat16, 1>(a, stream);
  return vec > 1 ? bwd_kind<float, 4>(a, stream) : bwd_kind<float, 1>(a, stream);
}

}  // namespace mlstm
