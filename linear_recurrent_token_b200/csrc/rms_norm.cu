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

// VEC consecutive values (VEC = 1, or 16 bytes of the storage type) at p, in device or shared memory, as fp32.
template <typename T, int VEC>
__device__ __forceinline__ void load_vec(const T* p, float (&x)[VEC]) {
  if constexpr (VEC == 1) {
    x[0] = io<T>::load(p, 0);
  } else {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 4) {
        x[i] = __uint_as_float(u[i]);
      } else {
        x[2 * i] = __uint_as_float(u[i] << 16);
        x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
      }
    }
  }
}

// The rows ahead of the one in work, on their way from HBM: every thread copies its own vectors of NT tensors
// into slots of shared memory that it alone reads, so that a wait for its own copies is all that a row costs
// and up to 100 KB an SM are in flight whatever the block does (less where a row leaves lanes or places empty: about
// 18 KB for bf16 rows of 64 channels).  Odd widths (VEC 1), and fp32 rows of more than 8192 channels, have no such
// copies and read from memory.
template <typename T, int VEC, int NT, int TPR>
struct Ring {
  static constexpr int NV = kElems / VEC, BLOCK = TPR > kThreads ? TPR : kThreads;
  static constexpr int stage = NT * NV * BLOCK * 16;
  static constexpr int all = NT == 2 ? 65536 : 98304;  // three blocks an SM forward, two backward
  static constexpr int stages = all / stage > 2 ? all / stage : 2;
  static constexpr bool direct = VEC == 1 || 2 * stage > 200 * 1024;  // the widest fp32 rows do not fit twice
  static constexpr int bytes = direct ? 0 : stages * stage;
  const T* src[NT];
  char* smem;
  long long rows, stride;
  int D, t;

  __device__ __forceinline__ char* slot(int turn, int k, int i) const {
    return smem + (((turn % stages) * NT + k) * NV + i) * BLOCK * 16 + threadIdx.x * 16;
  }
  // brings row `row` for turn `turn`
  __device__ __forceinline__ void fetch(int turn, long long row) const {
    if constexpr (!direct) {
      if (row < rows)
#pragma unroll
        for (int k = 0; k < NT; ++k)
#pragma unroll
          for (int i = 0; i < NV; ++i) {
            const int c = (i * TPR + t) * VEC;
            if (src[k] && c < D) {
              const uint32_t to = (uint32_t)__cvta_generic_to_shared(slot(turn, k, i));
              asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(src[k] + (size_t)row * D + c) : "memory");
            }
          }
      asm volatile("cp.async.commit_group;" ::: "memory");
    }
  }
  __device__ __forceinline__ void start(long long row) const {
    if constexpr (!direct)
#pragma unroll
      for (int s = 0; s < stages - 1; ++s) fetch(s, row + s * stride);
  }
  __device__ __forceinline__ void wait() const {
    if constexpr (!direct) asm volatile("cp.async.wait_group %0;" ::"n"(stages - 2) : "memory");
  }
  // vector i of tensor k; zeros behind the row's end
  __device__ __forceinline__ void read(int turn, long long row, int k, int i, float (&x)[VEC]) const {
    const int c = (i * TPR + t) * VEC;
    if (row < rows && c < D) {
      if constexpr (!direct)
        load_vec<T, VEC>(reinterpret_cast<const T*>(slot(turn, k, i)), x);
      else
        load_vec<T, VEC>(src[k] + (size_t)row * D + c, x);
    } else {
#pragma unroll
      for (int e = 0; e < VEC; ++e) x[e] = 0.f;
    }
  }
};

template <typename T, int VEC>
__device__ __forceinline__ void store_vec(T* p, const float (&x)[VEC]) {
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

// The TPR threads of a row meet (rows of one warp or less have no barrier).
template <int TPR>
__device__ __forceinline__ void row_barrier() {
  asm volatile("bar.sync %0, %1;" ::"r"(1 + (int)threadIdx.x / TPR), "n"(TPR) : "memory");
}

// Sums over the TPR threads of a row, the same in each; red: N values a warp, not in use by anyone.
template <int TPR, typename F, int N>
__device__ __forceinline__ void row_sum(F (&v)[N], F (*red)[N]) {
#pragma unroll
  for (int d = (TPR < 32 ? TPR : 32) / 2; d > 0; d /= 2)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], d);
  if constexpr (TPR > 32) {
    constexpr int NW = TPR / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (lane == 0)
#pragma unroll
      for (int i = 0; i < N; ++i) red[warp][i] = v[i];
    row_barrier<TPR>();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      v[i] = red[warp / NW * NW + lane % NW][i];
#pragma unroll
      for (int d = NW / 2; d > 0; d /= 2) v[i] += __shfl_xor_sync(0xffffffffu, v[i], d);
    }
  }
}

template <int NV, int VEC>
__device__ __forceinline__ void copy(float (&to)[NV][VEC], const float (&from)[NV][VEC]) {
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int e = 0; e < VEC; ++e) to[i][e] = from[i][e];
}

// Whether fp32 held the sum of squares: ms = mean(r^2) + eps is neither so large that a square may
// have overflowed nor so small that the squares have vanished (nor NaN).  The same in a row's threads.
__device__ __forceinline__ bool in_range(float ms) { return ms > 1e-30f && ms < 1e34f; }

// The row for which fp32 did not: v becomes r / sqrt(mean(r^2) + eps) from sums in 64 bits, which hold
// the squares of every fp32 value.
template <int TPR, int NV, int VEC>
__device__ __noinline__ double normalise_wide(float (&v)[NV][VEC], float eps, int D) {
  __shared__ double red[32][1];
  double s[1] = {0.0};
  for (int i = 0; i < NV; ++i)
    for (int e = 0; e < VEC; ++e) s[0] += (double)v[i][e] * v[i][e];
  if constexpr (TPR > 32) row_barrier<TPR>();
  row_sum<TPR, double, 1>(s, red);
  const double inv = 1.0 / sqrt(s[0] / D + eps);
  for (int i = 0; i < NV; ++i)
    for (int e = 0; e < VEC; ++e) v[i][e] = (float)(v[i][e] * inv);
  return inv;
}

// VEC values, already divided by their scale, in 8 bits.  NaN stays NaN in e4m3 and gives -127 as an
// integer (its scale is NaN).
__device__ __forceinline__ uint32_t as_int8(float z) { return (uint32_t)__float2int_rn(fminf(fmaxf(z, -127.f), 127.f)); }
template <int KIND, int VEC>
__device__ __forceinline__ void store8(uint8_t* out, const float (&z)[VEC]) {
  if constexpr (VEC == 1) {
    *out = KIND == kInt8 ? (uint8_t)as_int8(z[0]) : (uint8_t)__nv_cvt_float_to_fp8(z[0], __NV_SATFINITE, __NV_E4M3);
  } else {
    uint32_t q[VEC / 4];
#pragma unroll
    for (int e = 0; e < VEC / 4; ++e) {
      const float *x = z + 4 * e;
      if constexpr (KIND == kInt8) {
        q[e] = __byte_perm(__byte_perm(as_int8(x[0]), as_int8(x[1]), 0x0040), __byte_perm(as_int8(x[2]), as_int8(x[3]), 0x0040), 0x5410);
      } else {
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x[0], x[1]), __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x[2], x[3]), __NV_SATFINITE, __NV_E4M3);
        q[e] = lo | hi << 16;
      }
    }
    if constexpr (VEC == 8)
      *reinterpret_cast<uint2*>(out) = make_uint2(q[0], q[1]);
    else
      *reinterpret_cast<uint32_t*>(out) = q[0];
  }
}

// The larger magnitude, NaN where either is.
__device__ __forceinline__ float max_abs(float m, float x) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(m), "f"(fabsf(x)));
  return r;
}

// A block walks rows blockIdx.x, + gridDim.x, ...: a thread meets the same channels every time, keeps their
// weights, and has the next row's loads in flight while it reduces this one.  group: channels that share
// a scale (D: the whole row).  A group of 128 is 128 / VEC neighbouring lanes of one warp; odd widths
// (VEC 1) meet in shared memory.  16384 x 4096 bf16 with residual and e4m3 output: 82 us for 470 MB, 5.7 TB/s,
// 87 % of a copy's rate.
template <typename T, int VEC, int KIND, int TPR>
__global__ void __launch_bounds__(TPR > kThreads ? TPR : kThreads, TPR > kThreads ? 1 : 3)
    rms_norm_kernel(const T* x, const T* res, const float* __restrict__ weight, float eps, T* r_out, void* y,
                    float* __restrict__ scales, long long rows, int D, float inv_d, int group) {
  constexpr int NV = kElems / VEC, BLOCK = TPR > kThreads ? TPR : kThreads, RPB = BLOCK / TPR;
  __shared__ float red[2][32][1];
  __shared__ uint32_t gmax[2][KIND == kOut ? 1 : 128];
  const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR;
  extern __shared__ __align__(16) char smem[];
  float w[NV][VEC];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * TPR + t) * VEC;
#pragma unroll
    for (int e = 0; e < VEC; ++e) w[i][e] = 1.f;
    if (weight && c < D) load_w<VEC>(weight + c, w[i]);
  }
  using R = Ring<T, VEC, 2, TPR>;
  const R ring{{x, res}, smem, rows, (long long)gridDim.x * RPB, D, t};
  ring.start((long long)blockIdx.x * RPB + sub);
  int turn = 0;
  for (long long r0 = (long long)blockIdx.x * RPB; r0 < rows; r0 += ring.stride, ++turn) {
    const long long row = r0 + sub;
    const bool live = row < rows;  // dead rows of the last block still take part in the shuffles
    const size_t base = live ? (size_t)row * D : 0;
    float v[NV][VEC], s[1] = {0.f};
    ring.wait();
    // Read from memory, a row's loads all come before the first store, which may lie on one of them (bf16 with
    // residual, 33520 x 1001: 74 us, 316 vector by vector; 8186 x 4099: 146/517; four blocks an SM: 109, 144); read
    // from shared memory, vector by vector, which takes fewer registers.
    constexpr int AHEAD = R::direct ? NV : 1;
    float add[AHEAD][VEC];
    if constexpr (R::direct) {
#pragma unroll
      for (int i = 0; i < NV; ++i) ring.read(turn, row, 0, i, v[i]);
      if (res)
#pragma unroll
        for (int i = 0; i < NV; ++i) ring.read(turn, row, 1, i, add[i]);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * TPR + t) * VEC;
      if constexpr (!R::direct) {
        ring.read(turn, row, 0, i, v[i]);
        if (res) ring.read(turn, row, 1, i, add[0]);
      }
      if (res) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[i][e] += add[i % AHEAD][e];
        if (live && c < D) store_vec<T, VEC>(r_out + base + c, v[i]);  // this thread's own: r_out may be res or x
      }
#pragma unroll
      for (int e = 0; e < VEC; ++e) s[0] = fmaf(v[i][e], v[i][e], s[0]);
    }
    ring.fetch(turn + R::stages - 1, row + (R::stages - 1) * ring.stride);
    row_sum<TPR, float, 1>(s, red[turn & 1]);
    // the norm reads the sum before it is rounded to the storage type
    const float ms = s[0] * inv_d + eps;
    float inv = rsqrtf(ms);
    if (!in_range(ms)) {
      float wide[NV][VEC];  // a copy: v itself stays in registers
      copy(wide, v);
      normalise_wide<TPR, NV, VEC>(wide, eps, D);
      copy(v, wide);
      inv = 1.f;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * TPR + t) * VEC;
#pragma unroll
      for (int e = 0; e < VEC; ++e) v[i][e] = v[i][e] * inv * w[i][e];
      if constexpr (KIND == kOut)
        if (live && c < D) store_vec<T, VEC>(reinterpret_cast<T*>(y) + base + c, v[i]);
    }
    if constexpr (KIND != kOut) {
      constexpr float kTop = KIND == kE4m3 ? 448.f : 127.f;
      const int ngroups = group == D ? 1 : (D + 127) / 128;
      uint32_t m[NV];  // magnitudes as integers: in their order, with NaN above infinity
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float big = 0.f;
#pragma unroll
        for (int e = 0; e < VEC; ++e) big = (i * TPR + t) * VEC < D ? max_abs(big, v[i][e]) : 0.f;
        m[i] = __float_as_uint(big);
      }
      if (group == D) {  // one maximum for the row
#pragma unroll
        for (int i = 1; i < NV; ++i) m[0] = max(m[0], m[i]);
        m[0] = __reduce_max_sync(0xffffffffu, m[0]);
        if constexpr (TPR > 32) {
          constexpr int NW = TPR / 32;
          const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
          if (lane == 0) gmax[turn & 1][warp] = m[0];
          row_barrier<TPR>();
          m[0] = __reduce_max_sync(0xffffffffu, gmax[turn & 1][warp / NW * NW + lane % NW]);
        }
#pragma unroll
        for (int i = 1; i < NV; ++i) m[i] = m[0];
      } else if constexpr (VEC > 1) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int d = 64 / VEC; d > 0; d /= 2) m[i] = max(m[i], __shfl_xor_sync(0xffffffffu, m[i], d));
      } else {  // one row a block: the launcher gives odd widths with groups TPR >= 256
        for (int i = threadIdx.x; i < ngroups; i += BLOCK) gmax[turn & 1][i] = 0;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int c = i * TPR + t;  // a warp's 32 channels lie in one group (33520 x 1001: an atomic a lane 1136 us, a warp 341)
          const uint32_t most = __reduce_max_sync(0xffffffffu, live && c < D ? m[i] : 0u);
          if ((t & 31) == 0 && c < D) atomicMax(&gmax[turn & 1][c / 128], most);  // the order does not matter
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < NV; ++i) m[i] = i * TPR + t < D ? gmax[turn & 1][(i * TPR + t) / 128] : 0;
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * TPR + t) * VEC;
        const float amax = __uint_as_float(m[i]);
        // one quick division for the group (whose result is 0 above 2^126), of a maximum brought into its range
        const float up = amax < 1e-30f ? 0x1p100f : amax > 0x1p100f ? 0x1p-100f : 1.f;
        const float f = m[i] == 0 ? 0.f : __fdividef(kTop, amax * up);
        if (up != 1.f)
#pragma unroll
          for (int e = 0; e < VEC; ++e) v[i][e] *= up;
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[i][e] *= f;
        if (live && c < D) {
          store8<KIND, VEC>(reinterpret_cast<uint8_t*>(y) + base + c, v[i]);
          if (group == D ? c == 0 : c % 128 == 0)  // groups have 128 channels
            scales[(size_t)row * ngroups + (group == D ? 0 : c / 128)] = m[i] == 0 ? 1.f : amax * (1.f / kTop);
        }
      }
    }
  }
}

// Gradients.  A block walks rows blockIdx.x, + gridDim.x, ... so that a thread meets the same
// channels every time and keeps their share of the weight's gradient in registers; part: one row
// of D sums a block, added up in order by rms_norm_dw_kernel.  The next rows are on their way while this one
// is reduced.  8192 x 4096 bf16 with the residual's gradient: 47 us for 268 MB, 5.7 TB/s, 87 % of a copy's rate; the
// sum over the blocks after it 5 us, latency.
template <typename T, int VEC, int TPR>
__global__ void __launch_bounds__(TPR > kThreads ? TPR : kThreads, TPR > kThreads ? 1 : 2)
    rms_norm_bwd_kernel(const T* dy, const T* r, const float* __restrict__ weight, float eps, const T* dres, T* dx,
                        float* __restrict__ part, long long rows, int D, float inv_d) {
  constexpr int NV = kElems / VEC, BLOCK = TPR > kThreads ? TPR : kThreads, RPB = BLOCK / TPR;
  extern __shared__ __align__(16) char smem[];  // the ring; then [rows a block][D] sums where a block takes several rows
  __shared__ float red[2][32][2];
  const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR;
  float dw[NV][VEC], w[NV][VEC];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * TPR + t) * VEC;
#pragma unroll
    for (int e = 0; e < VEC; ++e) dw[i][e] = 0.f, w[i][e] = 1.f;
    if (weight && c < D) load_w<VEC>(weight + c, w[i]);
  }
  using R = Ring<T, VEC, 3, TPR>;
  const R ring{{r, dy, dres}, smem, rows, (long long)gridDim.x * RPB, D, t};
  ring.start((long long)blockIdx.x * RPB + sub);
  int turn = 0;
  for (long long r0 = (long long)blockIdx.x * RPB; r0 < rows; r0 += ring.stride, ++turn) {
    const long long row = r0 + sub;
    const bool live = row < rows;
    const size_t base = live ? (size_t)row * D : 0;
    float a[NV][VEC], d[NV][VEC], s[2] = {0.f, 0.f};
    ring.wait();
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      ring.read(turn, row, 0, i, a[i]);
      ring.read(turn, row, 1, i, d[i]);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        s[0] = fmaf(a[i][e], a[i][e], s[0]);
        s[1] = fmaf(a[i][e], d[i][e] * w[i][e], s[1]);
      }
    }
    row_sum<TPR, float, 2>(s, red[turn & 1]);
    const float ms = s[0] * inv_d + eps;
    float inv = rsqrtf(ms), scale = inv;  // scale takes r to n = r s where a still holds r
    float along = s[1] * inv_d * inv;     // mean(w dy n)
    if (!in_range(ms)) {
      float wide[NV][VEC];  // a copy: a itself stays in registers
      copy(wide, a);
      inv = (float)normalise_wide<TPR, NV, VEC>(wide, eps, D);
      copy(a, wide);
      scale = 1.f;
      s[0] = s[1] = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < VEC; ++e) s[1] = fmaf(a[i][e], d[i][e] * w[i][e], s[1]);
      if constexpr (TPR > 32) row_barrier<TPR>();  // red is still being read
      row_sum<TPR, float, 2>(s, red[turn & 1]);
      along = s[1] * inv_d;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * TPR + t) * VEC;
      if (live && c < D) {
        float out[VEC], more[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) more[e] = 0.f;
        if (dres) ring.read(turn, row, 2, i, more);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float n = a[i][e] * scale;
          out[e] = fmaf(inv, d[i][e] * w[i][e] - n * along, more[e]);
          dw[i][e] = fmaf(d[i][e], n, dw[i][e]);
        }
        store_vec<T, VEC>(dx + base + c, out);  // dx may be dy or dres: this thread's own elements, read above
      }
    }
    ring.fetch(turn + R::stages - 1, row + (R::stages - 1) * ring.stride);
  }
  if (!part) return;
  float* sums = reinterpret_cast<float*>(smem);
  if (RPB > 1) {
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
  }
  float* mine = RPB > 1 ? sums + (size_t)sub * D : part + (size_t)blockIdx.x * D;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * TPR + t) * VEC;
    if (c < D)
#pragma unroll
      for (int e = 0; e < VEC; ++e) mine[c + e] = dw[i][e];
  }
  if constexpr (RPB > 1) {
    __syncthreads();
    for (int c = threadIdx.x; c < D; c += BLOCK) {
      float v = 0.f;
      for (int i = 0; i < RPB; ++i) v += sums[(size_t)i * D + c];
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

template <typename T, int VEC, int TPR>
cudaError_t fwd_rows(const RmsArgs& a, cudaStream_t stream) {
  constexpr int block = TPR > kThreads ? TPR : kThreads;
  const long long blocks = (a.rows + block / TPR - 1) / (block / TPR);
  const unsigned grid = (unsigned)(blocks < 444 ? blocks : 444);  // three blocks for each of 148 SMs
  constexpr int smem = Ring<T, VEC, 2, TPR>::bytes;
#define MLSTM_RMS(KIND)                                                                                               \
  do {                                                                                                                \
    const auto kernel = rms_norm_kernel<T, VEC, KIND, TPR>;                                                           \
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);            \
    if (e != cudaSuccess) return e;                                                                                   \
    kernel<<<grid, block, smem, stream>>>((const T*)a.x, (const T*)a.res, a.weight, a.eps, (T*)a.r_out, a.y, a.scales, \
                                          a.rows, a.D, 1.f / a.D, a.group);                                           \
  } while (0)
  if (a.kind == kOut)
    MLSTM_RMS(kOut);
  else if (a.kind == kE4m3)
    MLSTM_RMS(kE4m3);
  else
    MLSTM_RMS(kInt8);
#undef MLSTM_RMS
  return cudaGetLastError();
}

template <typename T, int VEC, int TPR>
cudaError_t bwd_rows(const RmsArgs& a, cudaStream_t stream) {
  constexpr int block = TPR > kThreads ? TPR : kThreads, rpb = block / TPR;
  const int grid = bwd_blocks(a.rows, rpb);
  const int sums = rpb > 1 && a.dweight ? (int)sizeof(float) * rpb * a.D : 0;
  constexpr int ring = Ring<T, VEC, 3, TPR>::bytes, most_sums = rpb > 1 ? (int)sizeof(float) * rpb * TPR * kElems : 0;
  const int smem = sums > ring ? sums : ring;
  const auto kernel = rms_norm_bwd_kernel<T, VEC, TPR>;
  // the same limit from every call: it belongs to the function, and another thread may set it before this launch
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, ring > most_sums ? ring : most_sums);
  if (e != cudaSuccess) return e;
  kernel<<<grid, block, smem, stream>>>((const T*)a.dy, (const T*)a.x, a.weight, a.eps,
                                                                  (const T*)a.res, (T*)a.y,
                                                                  a.dweight ? a.part : nullptr, a.rows, a.D,
                                        1.f / a.D);
  e = cudaGetLastError();
  if (e != cudaSuccess || !a.dweight) return e;
  rms_norm_dw_kernel<<<(a.D + 31) / 32, dim3(32, 32), 0, stream>>>(a.part, grid, a.D, a.dweight);
  return cudaGetLastError();
}

template <typename T, int VEC>
cudaError_t by_rows(const RmsArgs& a, bool backward, cudaStream_t stream) {
  // groups of 128 channels lie inside one warp: 16 or 32 lanes of a row; odd widths with groups want
  // one row a block
  const bool odd_groups = !backward && VEC == 1 && a.kind != kOut && a.group < a.D;
  switch (row_threads(a.D, odd_groups ? kThreads : 32)) {
    case 32: return backward ? bwd_rows<T, VEC, 32>(a, stream) : fwd_rows<T, VEC, 32>(a, stream);
    case 64: return backward ? bwd_rows<T, VEC, 64>(a, stream) : fwd_rows<T, VEC, 64>(a, stream);
    case 128: return backward ? bwd_rows<T, VEC, 128>(a, stream) : fwd_rows<T, VEC, 128>(a, stream);
    case 256: return backward ? bwd_rows<T, VEC, 256>(a, stream) : fwd_rows<T, VEC, 256>(a, stream);
    case 512: return backward ? bwd_rows<T, VEC, 512>(a, stream) : fwd_rows<T, VEC, 512>(a, stream);
    default: return backward ? bwd_rows<T, VEC, 1024>(a, stream) : fwd_rows<T, VEC, 1024>(a, stream);
  }
}

cudaError_t launch(const RmsArgs& a, bool backward, cudaStream_t stream) {
  const int vec = vec_of(a.D, a.dtype);
  if (a.dtype)
    return vec > 1 ? by_rows<__nv_bfloat16, 8>(a, backward, stream) : by_rows<__nv_bfloat16, 1>(a, backward, stream);
  return vec > 1 ? by_rows<float, 4>(a, backward, stream) : by_rows<float, 1>(a, backward, stream);
}

}  // namespace

bool rms_norm_supported(int D) { return D >= 1 && D <= kMaxD; }

size_t rms_norm_bwd_workspace_bytes(long long rows, int D) {
  const int tpr = row_threads(D, 32);
  return sizeof(float) * (size_t)bwd_blocks(rows, tpr < kThreads ? kThreads / tpr : 1) * D;
}

cudaError_t launch_rms_norm(const RmsArgs& a, cudaStream_t stream) { return launch(a, false, stream); }

cudaError_t launch_rms_norm_bwd(const RmsArgs& a, cudaStream_t stream) { return launch(a, true, stream); }

}  // namespace mlstm
