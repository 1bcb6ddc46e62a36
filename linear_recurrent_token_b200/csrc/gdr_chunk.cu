// Gated delta rule in chunks of 64 tokens (formulas, precision and layouts: gdr_tile.cuh).
//
// gdr_prep_kernel computes for all chunks at once what does not depend on the state: k and q in 16-bit
// parts, R, P and the factors of each token.  gdr_walk_kernel then takes each sequence's chunks in order.
#include "gdr_walk.cuh"

namespace mlstm {
namespace gdr {
namespace {

constexpr int kPrepThreads = 256;
constexpr int kMs = kL + 1;  // row pitch of the fp32 matrices

template <int KP, int NP>
constexpr int prep_smem() {
  return keys_bytes(KP, NP) + 2 * kL * kMs * 4 + 32 * 33 * 4 + kL * 8 + kFactorBytes + 2 * kL * 4;
}

// dst (n x n, at r, c of R) = -(X + R22 b2 X), X = M21 + M21 b1 R11: joins two solved n x n diagonal blocks.
template <int N>
__device__ __forceinline__ void join_blocks(const float* M, float* R, const float* beta, float* X, int top, int t0,
                                            int nthreads) {
  const int low = top + N;
  for (int e = t0; e < N * N; e += nthreads) {
    const int t = e / N, s = e % N;
    float x = M[(low + t) * kMs + top + s];
    for (int i = s + 1; i < N; ++i) x = fmaf(M[(low + t) * kMs + top + i] * beta[top + i], R[(top + i) * kMs + top + s], x);
    X[t * 33 + s] = x;
  }
}
template <int N>
__device__ __forceinline__ void join_rows(float* R, const float* beta, const float* X, int top, int t0, int nthreads) {
  const int low = top + N;
  for (int e = t0; e < N * N; e += nthreads) {
    const int t = e / N, s = e % N;
    float x = X[t * 33 + s];
    for (int i = 0; i < t; ++i) x = fmaf(R[(low + t) * kMs + low + i] * beta[low + i], X[i * 33 + s], x);
    R[(low + t) * kMs + top + s] = -x;
  }
}

// One block for each chunk and key head; the value heads that share it follow one another.  The two
// 64 x 64 x KP products run on the tensor cores; the triangular solve is fp32: four 16 x 16 diagonal
// blocks column by column, then two joins.
template <typename T, int KP, bool P2>
__global__ void __launch_bounds__(kPrepThreads) gdr_prep_kernel(const GdrArgs a, char* keys, char* records) {
  constexpr int NP = sizeof(T) == 4 ? 2 : 1;
  extern __shared__ __align__(16) char smem[];
  char* sk = smem;  // k parts, then q parts
  char* sq = smem + keys_bytes(KP, NP) / 2;
  float* M = reinterpret_cast<float*>(smem + keys_bytes(KP, NP));
  float* R = M + kL * kMs;
  float* X = R + kL * kMs;
  double* G = reinterpret_cast<double*>(X + 32 * 33);
  float* fac = reinterpret_cast<float*>(G + kL);
  float* pmax = fac + kFactors * kL;  // [2][64]
  int n, c;
  Seq sq_;
  if (!find_chunk(a, blockIdx.x, &n, &sq_, &c)) return;
  const int hk = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const long long rec = blockIdx.x, t0 = sq_.lo + (long long)c * kL;
  const int len = (int)min((long long)kL, sq_.len - (long long)c * kL);

  {  // k, q: four threads a row
    const int row = tid >> 2, part = tid & 3;
    char* out = keys + (rec * a.HK + hk) * keys_bytes(KP, NP);
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      const GdrStride st = which ? a.sq : a.sk;
      const T* src = (const T*)(which ? a.q : a.k) + sq_.b * st.b + hk * st.h + (t0 + row) * st.t;
      float x[KP / 32][8], m = 0.f;
#pragma unroll
      for (int j = 0; j < KP / 32; ++j) {
        const int col = (j * 4 + part) * 8;
        load8<T>(src + col, row < len && col < a.K, x[j]);
#pragma unroll
        for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(x[j][e]));
      }
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
      const Scale sc = scale_of(m);
      if (part == 0) fac[(which ? kQInv : kKInv) * kL + row] = sc.inv;
#pragma unroll
      for (int j = 0; j < KP / 32; ++j) {
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) split(x[j][2 * e] * sc.mul, x[j][2 * e + 1] * sc.mul, hi[e], lo[e]);
        const int at = (which ? keys_bytes(KP, NP) / 2 : 0) + piece_at<KP>(row, (j * 4 + part) * 8);
        const uint4 h4 = make_uint4(hi[0], hi[1], hi[2], hi[3]), l4 = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        *reinterpret_cast<uint4*>(smem + at) = h4;
        *reinterpret_cast<uint4*>(out + at) = h4;
        if constexpr (NP == 2) {
          *reinterpret_cast<uint4*>(smem + at + kL * KP * 2) = l4;
          *reinterpret_cast<uint4*>(out + at + kL * KP * 2) = l4;
        }
      }
    }
  }
  __syncthreads();

  // k k^T and q k^T: a warp has 16 rows and 32 columns
  const int r0 = (warp & 3) * 16, c0 = (warp >> 2) * 32;
  const bool lower = c0 <= r0 + 15;
  float kk_[4][4], qk[4][4];
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) kk_[j][e] = qk[j][e] = 0.f;
  if (lower) {
#pragma unroll
    for (int s = 0; s < KP / 16; ++s) {
      const int at = piece_at<KP>(r0 + bt_row(lane), s * 16 + bt_col(lane));  // an A operand's rows
      uint32_t k4[4], q4[4], kl[4], ql[4];
      ldsm4(k4, smem_u32(sk) + at);
      ldsm4(q4, smem_u32(sq) + at);
      if constexpr (NP == 2) {
        ldsm4(kl, smem_u32(sk) + kL * KP * 2 + at);
        ldsm4(ql, smem_u32(sq) + kL * KP * 2 + at);
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int bt = piece_at<KP>(c0 + j * 16 + b_row(lane), s * 16 + b_col(lane));
        uint32_t b[4];
        ldsm4(b, smem_u32(sk) + bt);
        if constexpr (NP == 2) {
          uint32_t bl[4];
          ldsm4(bl, smem_u32(sk) + kL * KP * 2 + bt);
          mma(kk_[2 * j], kl, b[0], b[1]), mma(kk_[2 * j + 1], kl, b[2], b[3]);
          mma(kk_[2 * j], k4, bl[0], bl[1]), mma(kk_[2 * j + 1], k4, bl[2], bl[3]);
          mma(qk[2 * j], ql, b[0], b[1]), mma(qk[2 * j + 1], ql, b[2], b[3]);
          mma(qk[2 * j], q4, bl[0], bl[1]), mma(qk[2 * j + 1], q4, bl[2], bl[3]);
        }
        mma(kk_[2 * j], k4, b[0], b[1]), mma(kk_[2 * j + 1], k4, b[2], b[3]);
        mma(qk[2 * j], q4, b[0], b[1]), mma(qk[2 * j + 1], q4, b[2], b[3]);
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int t = r0 + (lane >> 2) + (e >> 1) * 8, s = c0 + j * 8 + (lane & 3) * 2 + (e & 1);
        kk_[j][e] = kk_[j][e] * fac[kKInv * kL + t] * fac[kKInv * kL + s];
        qk[j][e] = qk[j][e] * fac[kQInv * kL + t] * fac[kKInv * kL + s];
      }
  }

  for (int h = hk * (a.H / a.HK); h < (hk + 1) * (a.H / a.HK); ++h) {
    char* out = records + (rec * a.H + h) * record_bytes(P2);
    if (warp == 0) {  // cumulative log decays, two tokens a lane, in 64 bits
      const float* g = a.g + sq_.b * a.sg.b + h * a.sg.h;
      const float* be = a.beta + sq_.b * a.sb.b + h * a.sb.h;
      const int t = 2 * lane;
      const double2 sum = cumulative(g, a.sg.t, t0, len, lane);
      const double last = __shfl_sync(0xffffffffu, sum.y, 31);
      G[t] = sum.x, G[t + 1] = sum.y;
      fac[kGam * kL + t] = expf((float)sum.x), fac[kGam * kL + t + 1] = expf((float)sum.y);
      fac[kW * kL + t] = expf((float)(last - sum.x)), fac[kW * kL + t + 1] = expf((float)(last - sum.y));
      fac[kBeta * kL + t] = t < len ? be[(t0 + t) * a.sb.t] : 0.f;
      fac[kBeta * kL + t + 1] = t + 1 < len ? be[(t0 + t + 1) * a.sb.t] : 0.f;
    }
    __syncthreads();
    float p[4][4], big[2] = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int t = r0 + (lane >> 2) + (e >> 1) * 8, s = c0 + j * 8 + (lane & 3) * 2 + (e & 1);
        const float D = s <= t ? expf((float)(G[t] - G[s])) : 0.f;
        p[j][e] = s <= t ? qk[j][e] * D : 0.f;
        big[e >> 1] = fmaxf(big[e >> 1], fabsf(p[j][e]));
        const float m = s < t ? kk_[j][e] * D : 0.f;
        M[t * kMs + s] = m;
        R[t * kMs + s] = 0.f;
      }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      big[i] = fmaxf(big[i], __shfl_xor_sync(0xffffffffu, big[i], 1));
      big[i] = fmaxf(big[i], __shfl_xor_sync(0xffffffffu, big[i], 2));
      if ((lane & 3) == 0) pmax[(warp >> 2) * kL + r0 + (lane >> 2) + i * 8] = big[i];
    }
    __syncthreads();
    // P, rows scaled; blocks above the diagonal are never read
    if (lower) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int t = r0 + (lane >> 2) + i * 8;
        const Scale sc = scale_of(fmaxf(pmax[t], pmax[kL + t]));
        if (c0 == 0 && (lane & 3) == 0) fac[kPInv * kL + t] = sc.inv;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t hi, lo;
          split(p[j][2 * i] * sc.mul, p[j][2 * i + 1] * sc.mul, hi, lo);
          char* at = out + 2 * kTile + piece_at<kL>(t, c0 + j * 8) + (lane & 3) * 4;
          *reinterpret_cast<uint32_t*>(at) = hi;
          if constexpr (P2) *reinterpret_cast<uint32_t*>(at + kTile) = lo;
        }
      }
    }
    // R: the 16 x 16 diagonal blocks, a thread a column
    const float* beta = fac + kBeta * kL;
    if (tid < kL) {
      const int top = tid & ~15, s = tid & 15;
      float y[16];  // beta_i R[i][s]
#pragma unroll
      for (int t = 0; t < 16; ++t) {
        float x = t > s ? M[(top + t) * kMs + top + s] : 0.f;
#pragma unroll
        for (int i = 0; i < t; ++i) x = fmaf(M[(top + t) * kMs + top + i], y[i], x);
        x = t > s ? -x : 0.f;
        R[(top + t) * kMs + top + s] = x;
        y[t] = beta[top + t] * x;
      }
    }
    __syncthreads();
    {
      const int pair = tid >> 7, t1 = tid & 127;
      join_blocks<16>(M, R, beta, X + pair * 16 * 33, pair * 32, t1, 128);
      __syncthreads();
      join_rows<16>(R, beta, X + pair * 16 * 33, pair * 32, t1, 128);
      __syncthreads();
      join_blocks<32>(M, R, beta, X, 0, tid, kPrepThreads);
      __syncthreads();
      join_rows<32>(R, beta, X, 0, tid, kPrepThreads);
      __syncthreads();
    }
    {  // R, rows scaled: four threads a row, 16 columns each
      const int row = tid >> 2, part = tid & 3;
      float x[16], m = 0.f;
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        x[e] = R[row * kMs + part * 16 + e];
        m = fmaxf(m, fabsf(x[e]));
      }
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
      const Scale sc = scale_of(m);
      if (part == 0) fac[kRInv * kL + row] = sc.inv;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) split(x[i * 8 + 2 * e] * sc.mul, x[i * 8 + 2 * e + 1] * sc.mul, hi[e], lo[e]);
        const int at = piece_at<kL>(row, part * 16 + i * 8);
        *reinterpret_cast<uint4*>(out + at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4*>(out + kTile + at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
      }
    }
    __syncthreads();
    float* fout = reinterpret_cast<float*>(out + (P2 ? 4 : 3) * kTile);
    for (int e = tid; e < kFactors * kL; e += kPrepThreads) fout[e] = fac[e];
    __syncthreads();  // fac, M, R belong to the next head
  }
}

}  // namespace

template <typename T, int KP, bool P2>
cudaError_t launch_prep(const GdrArgs& a, char* keys, char* records, cudaStream_t stream) {
  constexpr int smem = prep_smem<KP, sizeof(T) == 4 ? 2 : 1>();
  const auto kernel = gdr_prep_kernel<T, KP, P2>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  kernel<<<dim3((unsigned)record_count(a), a.HK), kPrepThreads, smem, stream>>>(a, keys, records);
  return cudaGetLastError();
}
template cudaError_t launch_prep<float, 64, true>(const GdrArgs&, char*, char*, cudaStream_t);
template cudaError_t launch_prep<float, 128, true>(const GdrArgs&, char*, char*, cudaStream_t);
template cudaError_t launch_prep<__nv_bfloat16, 64, true>(const GdrArgs&, char*, char*, cudaStream_t);
template cudaError_t launch_prep<__nv_bfloat16, 128, true>(const GdrArgs&, char*, char*, cudaStream_t);

namespace {

template <typename T, int KP>
cudaError_t chunk(const GdrArgs& a, void* ws, cudaStream_t stream) {
  constexpr bool P2 = sizeof(T) == 4;
  char* keys = (char*)ws;
  char* records = keys + record_count(a) * a.HK * keys_bytes(KP, sizeof(T) == 4 ? 2 : 1);
  cudaError_t e = launch_prep<T, KP, P2>(a, keys, records, stream);
  return e != cudaSuccess ? e : launch_walk<T, KP, false>(a, keys, records, Kept{}, stream);
}

}  // namespace
}  // namespace gdr

bool gdr_chunk_supported(int K) { return K <= 128; }

size_t gdr_chunk_workspace_bytes(const GdrArgs& a) {
  const int np = a.dtype ? 1 : 2, KP = a.K <= 64 ? 64 : 128;
  return (size_t)gdr::record_count(a) *
         ((size_t)a.HK * gdr::keys_bytes(KP, np) + (size_t)a.H * gdr::record_bytes(a.dtype == 0));
}

cudaError_t launch_gdr_chunk(const GdrArgs& a, void* ws, cudaStream_t stream) {
  if (a.dtype)
    return a.K <= 64 ? gdr::chunk<__nv_bfloat16, 64>(a, ws, stream) : gdr::chunk<__nv_bfloat16, 128>(a, ws, stream);
  return a.K <= 64 ? gdr::chunk<float, 64>(a, ws, stream) : gdr::chunk<float, 128>(a, ws, stream);
}

}  // namespace mlstm
