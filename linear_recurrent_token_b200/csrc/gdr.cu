// Gated delta rule token by token: the recurrent prefill and the decode step.
//
//   S' = e^g S;  u = beta (v - S'^T k);  S = S' + k u^T;  o = S^T q            state S [K, V] fp32
//
// Both kernels read the state once a token for both products and never form S' on its own:
//   r0 = S^T k,  o0 = S^T q;  u = beta (v - e^g r0);  o = e^g o0 + (k . q) u;  S = e^g S + k u^T.
#include "common.cuh"
#include "kernels.h"

namespace mlstm {
namespace {

// Below this log decay e^g is zero in fp32 (and in fp64 sums of it nothing is lost); a token with
// g = -infinity forgets everything.  NaN stays NaN.
__device__ __forceinline__ float decay(float g) { return g < -200.f ? 0.f : expf(g); }

// ---------------------------------------------------------------------------------------------
// Recurrent prefill.  A block walks one sequence of one value head for 32 value columns: four
// lanes to a column, each with every fourth float4 of its KP key rows in registers, so that a row's
// k and q are broadcast reads of shared memory and the two products end in two shuffles.  A
// few tokens are staged at a time while those before them are computed.  What bounds it is the chain
// of a token (products, shuffles, update); columns and heads run beside one another: 128
// tokens of 128 x 128 bf16 take 67 us for 16 heads, 89 for 64, 504 for 512.
constexpr int kRecCols = 32, kRecThreads = 128;

template <typename T, int KP>
__global__ void __launch_bounds__(kRecThreads) gdr_recurrent_kernel(const GdrArgs a) {
  constexpr int R = KP / 4;                // rows a thread
  constexpr int kRecTok = KP > 128 ? 8 : 16;  // tokens staged at a time
  constexpr int TT = kRecThreads / kRecTok;   // threads a token in k . q
  __shared__ __align__(16) float sk[2][kRecTok][KP], sq[2][kRecTok][KP];
  __shared__ float sv[2][kRecTok][kRecCols], salpha[2][kRecTok], sbeta[2][kRecTok], skq[2][kRecTok];
  const int n = blockIdx.z, h = blockIdx.y, c0 = blockIdx.x * kRecCols;
  const int tid = threadIdx.x, part = tid & 3, col = tid >> 2, c = c0 + col;
  const int hk = h / (a.H / a.HK);
  long long lo = 0, len = a.T, b = n;
  if (a.packed) {  // offsets come from the device: bounded here to the tokens that there are
    lo = min(max((long long)a.offsets[n], 0LL), (long long)a.T);
    len = min(max((long long)a.offsets[n + 1], lo), (long long)a.T) - lo;
    b = 0;
  }
  const T* q = (const T*)a.q + b * a.sq.b + hk * a.sq.h + lo * a.sq.t;
  const T* k = (const T*)a.k + b * a.sk.b + hk * a.sk.h + lo * a.sk.t;
  const T* v = (const T*)a.v + b * a.sv.b + h * a.sv.h + lo * a.sv.t;
  const float* g = a.g + b * a.sg.b + h * a.sg.h + lo * a.sg.t;
  const float* be = a.beta + b * a.sb.b + h * a.sb.h + lo * a.sb.t;
  T* o = (T*)a.o + b * a.so.b + h * a.so.h + lo * a.so.t;

  const size_t state = ((size_t)n * a.H + h) * a.K * a.V;
  float S[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int row = (i >> 2) * 16 + part * 4 + (i & 3);
    S[i] = a.S0 && row < a.K && c < a.V ? a.S0[state + (size_t)row * a.V + c] : 0.f;
  }

  auto stage = [&](int buf, long long t0) {
    for (int e = tid; e < kRecTok * KP; e += kRecThreads) {
      const int t = e / KP, d = e % KP;
      const bool in = t0 + t < len && d < a.K;
      sk[buf][t][d] = in ? io<T>::load(k, (size_t)((t0 + t) * a.sk.t + d)) : 0.f;
      sq[buf][t][d] = in ? io<T>::load(q, (size_t)((t0 + t) * a.sq.t + d)) : 0.f;
    }
    for (int e = tid; e < kRecTok * kRecCols; e += kRecThreads) {
      const int t = e / kRecCols, d = e % kRecCols;
      sv[buf][t][d] = t0 + t < len && c0 + d < a.V ? io<T>::load(v, (size_t)((t0 + t) * a.sv.t + c0 + d)) : 0.f;
    }
    if (tid < kRecTok) {
      const bool in = t0 + tid < len;
      salpha[buf][tid] = in ? decay(g[(t0 + tid) * a.sg.t]) : 1.f;
      sbeta[buf][tid] = in ? be[(t0 + tid) * a.sb.t] : 0.f;
    }
  };
  auto keys_by_queries = [&](int buf) {
    const int t = tid / TT;
    float s = 0.f;
    for (int d = tid % TT; d < KP; d += TT) s = fmaf(sk[buf][t][d], sq[buf][t][d], s);
#pragma unroll
    for (int d = TT / 2; d > 0; d /= 2) s += __shfl_xor_sync(0xffffffffu, s, d);
    if (tid % TT == 0) skq[buf][t] = s;
  };

  int buf = 0;
  if (len > 0) stage(0, 0);
  __syncthreads();
  for (long long t0 = 0; t0 < len; t0 += kRecTok, buf ^= 1) {
    keys_by_queries(buf);
    if (t0 + kRecTok < len) stage(buf ^ 1, t0 + kRecTok);
    __syncthreads();
    const int m = (int)min((long long)kRecTok, len - t0);
    for (int t = 0; t < m; ++t) {
      float kk[R], r[4] = {0.f, 0.f, 0.f, 0.f}, w[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int j = 0; j < R / 4; ++j) {
        const float4 x = *reinterpret_cast<const float4*>(&sk[buf][t][j * 16 + part * 4]);
        const float4 y = *reinterpret_cast<const float4*>(&sq[buf][t][j * 16 + part * 4]);
        kk[4 * j] = x.x, kk[4 * j + 1] = x.y, kk[4 * j + 2] = x.z, kk[4 * j + 3] = x.w;
        r[0] = fmaf(S[4 * j], x.x, r[0]), w[0] = fmaf(S[4 * j], y.x, w[0]);
        r[1] = fmaf(S[4 * j + 1], x.y, r[1]), w[1] = fmaf(S[4 * j + 1], y.y, w[1]);
        r[2] = fmaf(S[4 * j + 2], x.z, r[2]), w[2] = fmaf(S[4 * j + 2], y.z, w[2]);
        r[3] = fmaf(S[4 * j + 3], x.w, r[3]), w[3] = fmaf(S[4 * j + 3], y.w, w[3]);
      }
      float r0 = (r[0] + r[1]) + (r[2] + r[3]), o0 = (w[0] + w[1]) + (w[2] + w[3]);
#pragma unroll
      for (int d = 1; d < 4; d *= 2) {
        r0 += __shfl_xor_sync(0xffffffffu, r0, d);
        o0 += __shfl_xor_sync(0xffffffffu, o0, d);
      }
      const float alpha = salpha[buf][t];
      const float u = sbeta[buf][t] * (sv[buf][t][col] - alpha * r0);
#pragma unroll
      for (int i = 0; i < R; ++i) S[i] = fmaf(kk[i], u, alpha * S[i]);
      if (part == 0 && c < a.V) io<T>::store(o, (size_t)((t0 + t) * a.so.t + c), fmaf(alpha, o0, skq[buf][t] * u));
    }
    __syncthreads();
  }
  if (a.S_out && c < a.V) {
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int row = (i >> 2) * 16 + part * 4 + (i & 3);
      if (row < a.K) a.S_out[state + (size_t)row * a.V + c] = S[i];
    }
  }
}

template <typename T>
cudaError_t launch_rec(const GdrArgs& a, cudaStream_t stream) {
  const dim3 grid((a.V + kRecCols - 1) / kRecCols, a.H, a.N);
  if (a.K <= 64)
    gdr_recurrent_kernel<T, 64><<<grid, kRecThreads, 0, stream>>>(a);
  else if (a.K <= 128)
    gdr_recurrent_kernel<T, 128><<<grid, kRecThreads, 0, stream>>>(a);
  else
    gdr_recurrent_kernel<T, 256><<<grid, kRecThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

// ---------------------------------------------------------------------------------------------
// Decode step.  CW lanes cover 4 CW neighbouring value columns of a state row with 16-byte
// accesses, 256 / CW rows at a time; every load of a thread (NR rows) is in flight before the first
// is used, and one pass over shared memory joins both products.  Bound by HBM: the state is read
// and written once, 8 K V bytes a head.  256 rows of 16 heads of 128 x 128, six of them padding, 529 MB: 94 us
// in a loop from Python, 5.6 TB/s, 85 % of a copy's rate, 88 in a graph; one row: 3.3 us, latency.  (The
// tile in shared memory, three blocks on an SM instead of two, took 10 us more.)
//
// Rows of the batch that name the same slot are taken one after the other in the batch's order by
// the block of the first of them; a slot outside 0 .. pool - 1 marks padding (o = 0).
constexpr int kStepThreads = 256;
// A block sends for the state of the head this many blocks behind it, as far as L2: that its own loads wait for
// its slot, and its stores for its sums, then leaves memory busy.  256 rows of 16 heads of 128 x 128, slots
// given: without 102 us, 148 ahead 92, 296 93, 592 93; no slots 94, 87, 88, 88.  Not for heads below 64 KB, more
// of which share an SM (4096 of 64 x 64: 27 without, 29 with; 2048 of 64 x 128: 21.4/22.4), nor beyond 256 KB,
// which fill memory's queues by themselves (4096 of 128 x 256, between the two: 175/168).
constexpr int kStepAhead = 148, kStepLeast = 16384, kStepMost = 65536;

template <typename T, int CW, int NR>
__global__ void __launch_bounds__(kStepThreads) gdr_step_kernel(const GdrStepArgs a) {
  constexpr int RP = kStepThreads / CW;  // state rows side by side
  __shared__ float4 red[2][RP][CW];
  __shared__ float sk[256], sq[256], skq[8];
  __shared__ int first, next;
  const int b0 = blockIdx.z, h = blockIdx.y, hk = h / (a.H / a.HK), tid = threadIdx.x;
  const int lane = tid % CW, rp = tid / CW, c = (blockIdx.x * CW + lane) * 4;
  const bool in = c < a.V;
  const T *q = (const T*)a.q, *k = (const T*)a.k, *v = (const T*)a.v;
  T* o = (T*)a.o;
  const long long slot = a.slots ? (long long)a.slots[b0] : b0;
  if (slot < 0 || slot >= a.pool) {
    if (in && rp == 0)
#pragma unroll
      for (int e = 0; e < 4; ++e) io<T>::store(o, (size_t)(b0 * a.so.b + h * a.so.h + c + e), 0.f);
    return;
  }
  float* state = a.S + ((size_t)slot * a.H + h) * a.K * a.V + c;
  float4 S[NR];
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    const int row = i * RP + rp;
    S[i] = in && row < a.K ? __ldcs(reinterpret_cast<const float4*>(state + (size_t)row * a.V))
                           : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  if (tid == kStepThreads - 1 && blockIdx.x == 0 && a.K * a.V >= kStepLeast && a.K * a.V <= kStepMost) {
    const long long ahead = (long long)b0 * a.H + h + max(1, kStepAhead / (int)gridDim.x), row = ahead / a.H;
    const long long at = row >= a.B ? -1 : a.slots ? (long long)a.slots[row] : row;
    if (at >= 0 && at < a.pool)
      asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(a.S + ((size_t)at * a.H + ahead % a.H) * a.K * a.V),
                   "r"(a.K * a.V * 4)
                   : "memory");
  }
  if (tid == 0) first = 1, next = a.B;
  for (int b = b0; b < a.B;) {
    if (b != b0) __syncthreads();  // the row before has read shared memory
    float kq = 0.f;
    if (tid < a.K) {
      sk[tid] = io<T>::load(k, (size_t)(b * a.sk.b + hk * a.sk.h + tid));
      sq[tid] = io<T>::load(q, (size_t)(b * a.sq.b + hk * a.sq.h + tid));
      kq = sk[tid] * sq[tid];
    }
#pragma unroll
    for (int d = 16; d > 0; d /= 2) kq += __shfl_xor_sync(0xffffffffu, kq, d);
    if ((tid & 31) == 0) skq[tid >> 5] = kq;
    const float alpha = decay(a.g[b * a.sg.b + h * a.sg.h]), beta = a.beta[b * a.sb.b + h * a.sb.h];
    float x[4] = {0.f, 0.f, 0.f, 0.f};
    if (in)
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = io<T>::load(v, (size_t)(b * a.sv.b + h * a.sv.h + c + e));
    __syncthreads();
    if (a.slots) {  // other rows of the batch on this slot: one before, and the next after this one
      bool before = false;
      int after = a.B;
      for (int i = tid; i < a.B; i += kStepThreads)
        if (a.slots[i] == (int)slot) {
          if (i < b0) before = true;
          if (i > b && i < after) after = i;
        }
      if (before) first = 0;
      if (after < a.B) atomicMin(&next, after);
    }
    float4 r = make_float4(0.f, 0.f, 0.f, 0.f), w = r;
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      const int row = i * RP + rp;
      const float y = row < a.K ? sk[row] : 0.f, z = row < a.K ? sq[row] : 0.f;
      r.x = fmaf(S[i].x, y, r.x), r.y = fmaf(S[i].y, y, r.y), r.z = fmaf(S[i].z, y, r.z), r.w = fmaf(S[i].w, y, r.w);
      w.x = fmaf(S[i].x, z, w.x), w.y = fmaf(S[i].y, z, w.y), w.z = fmaf(S[i].z, z, w.z), w.w = fmaf(S[i].w, z, w.w);
    }
#pragma unroll
    for (int d = CW; d < 32; d *= 2) {  // rows side by side in one warp
      r.x += __shfl_xor_sync(0xffffffffu, r.x, d), r.y += __shfl_xor_sync(0xffffffffu, r.y, d);
      r.z += __shfl_xor_sync(0xffffffffu, r.z, d), r.w += __shfl_xor_sync(0xffffffffu, r.w, d);
      w.x += __shfl_xor_sync(0xffffffffu, w.x, d), w.y += __shfl_xor_sync(0xffffffffu, w.y, d);
      w.z += __shfl_xor_sync(0xffffffffu, w.z, d), w.w += __shfl_xor_sync(0xffffffffu, w.w, d);
    }
    const int warp = tid >> 5;
    if ((tid & 31) < CW) red[0][warp][lane] = r, red[1][warp][lane] = w;
    __syncthreads();
    if (!first) return;
    const int following = next;
    r = w = make_float4(0.f, 0.f, 0.f, 0.f);
    kq = 0.f;
#pragma unroll
    for (int i = 0; i < kStepThreads / 32; ++i) {
      const float4 y = red[0][i][lane], z = red[1][i][lane];
      r.x += y.x, r.y += y.y, r.z += y.z, r.w += y.w;
      w.x += z.x, w.y += z.y, w.z += z.z, w.w += z.w;
      kq += skq[i];
    }
    const float4 u = make_float4(beta * (x[0] - alpha * r.x), beta * (x[1] - alpha * r.y), beta * (x[2] - alpha * r.z),
                                 beta * (x[3] - alpha * r.w));
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      const int row = i * RP + rp;
      const float y = row < a.K ? sk[row] : 0.f;
      S[i] = make_float4(fmaf(y, u.x, alpha * S[i].x), fmaf(y, u.y, alpha * S[i].y), fmaf(y, u.z, alpha * S[i].z),
                         fmaf(y, u.w, alpha * S[i].w));
    }
    if (in && rp == 0) {
      const size_t at = (size_t)(b * a.so.b + h * a.so.h + c);
      io<T>::store(o, at, fmaf(alpha, w.x, kq * u.x));
      io<T>::store(o, at + 1, fmaf(alpha, w.y, kq * u.y));
      io<T>::store(o, at + 2, fmaf(alpha, w.z, kq * u.z));
      io<T>::store(o, at + 3, fmaf(alpha, w.w, kq * u.w));
    }
    b = following;
    if (b < a.B) {
      __syncthreads();  // everyone has read `next`
      if (tid == 0) next = a.B;
    }
  }
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    const int row = i * RP + rp;
    if (in && row < a.K) __stcs(reinterpret_cast<float4*>(state + (size_t)row * a.V), S[i]);
  }
}

template <typename T, int CW>
void launch_step_cw(const GdrStepArgs& a, cudaStream_t stream) {
  constexpr int RP = kStepThreads / CW;
  const dim3 grid((a.V + 4 * CW - 1) / (4 * CW), a.H, a.B);
  const int nr = (a.K + RP - 1) / RP;
  if (nr <= 2) {
    gdr_step_kernel<T, CW, 2><<<grid, kStepThreads, 0, stream>>>(a);
  } else if (nr <= 4) {
    gdr_step_kernel<T, CW, 4><<<grid, kStepThreads, 0, stream>>>(a);
  } else if (nr <= 8) {
    gdr_step_kernel<T, CW, 8><<<grid, kStepThreads, 0, stream>>>(a);
  } else if constexpr (RP < 32) {  // K is at most 256
    if constexpr (RP < 16) {
      if (nr > 16) return gdr_step_kernel<T, CW, 32><<<grid, kStepThreads, 0, stream>>>(a);
    }
    gdr_step_kernel<T, CW, 16><<<grid, kStepThreads, 0, stream>>>(a);
  }
}

template <typename T>
cudaError_t launch_step_t(const GdrStepArgs& a, cudaStream_t stream) {
  const long long heads = (long long)a.B * a.H;
  // Few heads: narrower tiles, more blocks.  us, narrow / wide, by heads of 128 x 128: 64 4.1/4.8, 96 4.7/4.9,
  // 128 5.6/4.9, 288 9.4/7.3; of 64 x 64: 64 3.2/3.3, 128 3.8/3.3; of 128 x 256: 32 4.1/4.7, 64 5.6/4.9.
  if (a.V <= 32 || heads * ((a.V + 63) / 64) < 200)
    launch_step_cw<T, 8>(a, stream);
  else if (a.V <= 64)
    launch_step_cw<T, 16>(a, stream);
  else
    launch_step_cw<T, 32>(a, stream);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_gdr_recurrent(const GdrArgs& a, cudaStream_t stream) {
  return a.dtype ? launch_rec<__nv_bfloat16>(a, stream) : launch_rec<float>(a, stream);
}

cudaError_t launch_gdr_step(const GdrStepArgs& a, cudaStream_t stream) {
  return a.dtype ? launch_step_t<__nv_bfloat16>(a, stream) : launch_step_t<float>(a, stream);
}

}  // namespace mlstm
