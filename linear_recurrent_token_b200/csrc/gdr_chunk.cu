// Gated delta rule in chunks of 64 tokens (formulas, precision and layouts: gdr_tile.cuh).
//
// gdr_prep_kernel computes for all chunks at once what does not depend on the state: k and q in 16-bit
// parts, R, P and the factors of each token.  gdr_walk_kernel or gdr_tc_kernel then takes each sequence's
// chunks in order.
#include "gdr_walk.cuh"
#include "sm100.cuh"

namespace mlstm {
namespace gdr {
namespace {

constexpr int kPrepThreads = 256;
constexpr int kMs = kL + 4;  // row pitch of the fp32 matrices: a fragment's lanes meet no bank conflicts

template <int KP, int NP>
constexpr int prep_smem() {
  constexpr int matrices = (2 * kL + 32) * kMs * 4;  // in the place of k and q
  return (keys_bytes(KP, NP) > matrices ? keys_bytes(KP, NP) : matrices) + kFactorBytes + 2 * kL * 4;
}

__device__ __forceinline__ float2 times2(float2 x, float f) {
  float2 y;
  asm("{.reg .b64 p, q, r;\n mov.b64 p, {%2, %3};\n mov.b64 q, {%4, %4};\n mul.rn.f32x2 r, p, q;\n mov.b64 {%0, %1}, r;}"
      : "=f"(y.x), "=f"(y.y)
      : "f"(x.x), "f"(x.y), "f"(f));
  return y;
}

// c += (A diag(b)) B for a 16 x 8 tile of c, k = 8 STEPS: fp32 matrices in shared memory (pitch kMs) as two
// tf32 parts each, whose exponent is fp32's: no scaling.  Only steps from .. upto - 1 hold anything.
template <int STEPS>
__device__ __forceinline__ void product_tf32(float (&c)[4], const float* A, const float* b, const float* B, int from, int upto,
                                             int lane) {
  const int g = lane >> 2, q = lane & 3;
  float hl[4] = {0.f, 0.f, 0.f, 0.f}, lh[4] = {0.f, 0.f, 0.f, 0.f};  // sums of their own: shorter chains
#pragma unroll
  for (int k = 0; k < STEPS; ++k) {
    if (k < from || k >= upto) continue;
    const int i = k * 8 + q;
    const float b0 = b[i], b1 = b[i + 4];
    uint32_t ah[4], al[4], bh[2], bl[2];
    split_tf32(A[g * kMs + i] * b0, ah[0], al[0]);
    split_tf32(A[(g + 8) * kMs + i] * b0, ah[1], al[1]);
    split_tf32(A[g * kMs + i + 4] * b1, ah[2], al[2]);
    split_tf32(A[(g + 8) * kMs + i + 4] * b1, ah[3], al[3]);
    split_tf32(B[i * kMs + g], bh[0], bl[0]);
    split_tf32(B[(i + 4) * kMs + g], bh[1], bl[1]);
    mma_tf32(lh, al, bh);
    mma_tf32(hl, ah, bl);
    mma_tf32(c, ah, bh);
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) c[e] += hl[e] + lh[e];
}

// Joins the solved N x N diagonal blocks at `top` and top + N: with 1 the upper and 2 the lower block,
//     X = M21 + M21 b1 R11,   R21 = -(X + R22 b2 X).
// One warp a 16 x 8 tile (mt, nt); X has N rows of its own, and `meet` waits for the warps of the same nt.
template <int N, typename Meet>
__device__ __forceinline__ void join(const float* M, float* R, float* X, const float* beta, int top, int mt, int nt, int lane,
                                     Meet meet) {
  const int low = top + N, r = mt * 16 + (lane >> 2), cc = nt * 8 + 2 * (lane & 3);
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const float* from = half ? X : M + low * kMs + top;
    float c[4] = {from[r * kMs + cc], from[r * kMs + cc + 1], from[(r + 8) * kMs + cc], from[(r + 8) * kMs + cc + 1]};
    if (half)
      product_tf32<N / 8>(c, R + (low + mt * 16) * kMs + low, beta + low, X + nt * 8, 0, 2 * (mt + 1), lane);
    else
      product_tf32<N / 8>(c, M + (low + mt * 16) * kMs + top, beta + top, R + top * kMs + top + nt * 8, nt, N / 8, lane);
    float* to = half ? R + low * kMs + top : X;
    const float sign = half ? -1.f : 1.f;
    to[r * kMs + cc] = sign * c[0], to[r * kMs + cc + 1] = sign * c[1];
    to[(r + 8) * kMs + cc] = sign * c[2], to[(r + 8) * kMs + cc + 1] = sign * c[3];
    if (!half) meet();
  }
}

// One block for each chunk and key head; the value heads that share it follow one another.  The two
// 64 x 64 x KP products run on the tensor cores; of the triangular solve, four 16 x 16 diagonal blocks go
// row by row in fp32 and two rounds of joins on the tensor cores again.  4096 chunks of 128 keys and one value
// head (8 x 16 heads x 2048 bf16): 110 us for 378 MB, 3.4 TB/s; its phases' barriers and the issue slots (half
// of them taken) bound it.  With one value head to a key head 64 registers do, and four blocks share an SM
// (three: 129 us); with more the products stay in registers for the next head, and three do.
template <typename T, int KP, bool P2, bool ONE>
__global__ void __launch_bounds__(kPrepThreads, ONE && sizeof(T) == 2 ? 4 : 3) gdr_prep_kernel(const GdrArgs a, char* keys, char* records) {
  constexpr int NP = sizeof(T) == 4 ? 2 : 1;
  extern __shared__ __align__(16) char smem[];
  char* sk = smem;  // k parts, then q parts
  char* sq = smem + keys_bytes(KP, NP) / 2;
  float* M = reinterpret_cast<float*>(smem);  // once the products with k and q are in registers
  float* R = M + kL * kMs;
  float* X = R + kL * kMs;  // [32]
  float* fac = reinterpret_cast<float*>(smem + prep_smem<KP, NP>()) - (kFactors + 2) * kL;
  float* pmax = fac + kFactors * kL;  // [2][64]
  float2* G = reinterpret_cast<float2*>(fac + kG * kL);
  int n, c;
  Seq sq_;
  if (!find_chunk(a, blockIdx.x, &n, &sq_, &c)) return;
  const int hk = blockIdx.y, group = ONE ? 1 : a.H / a.HK, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const long long rec = blockIdx.x, t0 = sq_.lo + (long long)c * kL;
  const int len = (int)min((long long)kL, sq_.len - (long long)c * kL);

  // A head's gates, two tokens a lane of warp 4: what it reads, well ahead, and their sums, in 64 bits.
  float gate[2], write[2];
  auto load_gates = [&](int h) {
    const float* g = a.g + sq_.b * a.sg.b + h * a.sg.h;
    const float* be = a.beta + sq_.b * a.sb.b + h * a.sb.h;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int t = 2 * lane + e;
      gate[e] = t < len ? g[(t0 + t) * a.sg.t] : 0.f;
      write[e] = t < len ? be[(t0 + t) * a.sb.t] : 0.f;
    }
  };
  auto gates = [&] {
    const int t = 2 * lane;
    const double2 sum = cumulative(gate[0], gate[1], lane);
    const double last = __shfl_sync(0xffffffffu, sum.y, 31);
    G[t] = two_parts(sum.x * kPerLn2), G[t + 1] = two_parts(sum.y * kPerLn2);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const double x = e ? sum.y : sum.x;
      const float gam = expf((float)x), w = expf((float)(last - x));
      fac[kGam * kL + t + e] = gam, fac[kW * kL + t + e] = w;
      fac[kGK * kL + t + e] = gam * fac[kKInv * kL + t + e], fac[kGQ * kL + t + e] = gam * fac[kQInv * kL + t + e];
      fac[kWK * kL + t + e] = w * fac[kKInv * kL + t + e];
      fac[kBeta * kL + t + e] = write[e];
    }
  };
  if (warp == 4) load_gates(hk * group);

  {  // k, q: four threads a row
    const int row = tid >> 2, part = tid & 3;
    char* out = keys + (rec * a.HK + hk) * keys_bytes(KP, NP);
    auto source = [&](int which) {
      const GdrStride st = which ? a.sq : a.sk;
      return (const T*)(which ? a.q : a.k) + sq_.b * st.b + hk * st.h + (t0 + row) * st.t;
    };
    auto scale_row = [&](int which, float m) {
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
      const Scale sc = scale_of(m);
      if (part == 0) fac[(which ? kQInv : kKInv) * kL + row] = sc.inv;
      return sc.mul;
    };
    auto put = [&](int which, int j, int plane, const uint32_t (&w)[4]) {
      const int at = (which ? keys_bytes(KP, NP) / 2 : 0) + plane * kL * KP * 2 + piece_at<KP>(row, (j * 4 + part) * 8);
      const uint4 v = make_uint4(w[0], w[1], w[2], w[3]);
      *reinterpret_cast<uint4*>(smem + at) = v;
      *reinterpret_cast<uint4*>(out + at) = v;
    };
    if constexpr (NP == 1) {  // one part; all loads before the first use, magnitudes compared as integers
      uint4 bits[2][KP / 32];
#pragma unroll
      for (int which = 0; which < 2; ++which)
#pragma unroll
        for (int j = 0; j < KP / 32; ++j) {
          const int col = (j * 4 + part) * 8;
          bits[which][j] = row < len && col < a.K ? *reinterpret_cast<const uint4*>(source(which) + col) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
      for (int which = 0; which < 2; ++which) {
        uint32_t m2 = 0;
#pragma unroll
        for (int j = 0; j < KP / 32; ++j) {
          const uint4 u = bits[which][j];
          m2 = __vmaxu2(__vmaxu2(m2, __vmaxu2(u.x & 0x7fff7fffu, u.y & 0x7fff7fffu)),
                        __vmaxu2(u.z & 0x7fff7fffu, u.w & 0x7fff7fffu));
        }
        const float mul = scale_row(which, __uint_as_float(max(m2 & 0xffff0000u, m2 << 16)));
#pragma unroll
        for (int j = 0; j < KP / 32; ++j) {
          const uint32_t u[4] = {bits[which][j].x, bits[which][j].y, bits[which][j].z, bits[which][j].w};
          uint32_t hi[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 f = times2(unpack_bf16(u[e]), mul);
            hi[e] = pack(f.x, f.y);
          }
          put(which, j, 0, hi);
        }
      }
    } else {
#pragma unroll
      for (int which = 0; which < 2; ++which) {
        float x[KP / 32][8], m = 0.f;
#pragma unroll
        for (int j = 0; j < KP / 32; ++j) {
          const int col = (j * 4 + part) * 8;
          load8(source(which) + col, row < len && col < a.K, x[j]);
#pragma unroll
          for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(x[j][e]));
        }
        const float mul = scale_row(which, m);
#pragma unroll
        for (int j = 0; j < KP / 32; ++j) {
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) split(x[j][2 * e] * mul, x[j][2 * e + 1] * mul, hi[e], lo[e]);
          put(which, j, 0, hi);
          put(which, j, 1, lo);
        }
      }
    }
  }
  __syncthreads();

  // k k^T and q k^T: a warp has 16 rows and 32 columns; one that has none below the diagonal takes the gates
  const int r0 = (warp & 3) * 16, c0 = (warp >> 2) * 32;
  const bool upper = warp == 4 || warp == 5;  // its products lie above the diagonal
  float kk_[4][4], qk[4][4];
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) kk_[j][e] = qk[j][e] = 0.f;
  if (!upper) {
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
  } else if (warp == 4) {
    gates();
  }
  __syncthreads();

  for (int h = hk * group; h < (hk + 1) * group; ++h) {
    char* out = records + (rec * a.H + h) * record_bytes(P2);
    float* fout = reinterpret_cast<float*>(out + (P2 ? 4 : 3) * kTile);
    // P, rows scaled, and M, of which blocks above the diagonal are never read
    float p[4][4], big[2] = {0.f, 0.f};
    zero(p);
    if (!upper) {
      const int t = r0 + (lane >> 2);
      const float2 Gt[2] = {G[t], G[t + 8]};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int cj = c0 + j * 8, s = cj + (lane & 3) * 2;
        if (cj > r0 + 15) continue;
        const float4 Gs = *reinterpret_cast<const float4*>(G + s);
        float mm[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float D = decay_between(Gt[e >> 1], e & 1 ? make_float2(Gs.z, Gs.w) : make_float2(Gs.x, Gs.y));
          p[j][e] = qk[j][e] * D, mm[e] = kk_[j][e] * D;
          if (cj + 7 >= r0) {  // (a tile on the diagonal; decays that run backward may be infinite)
            const int back = s + (e & 1) - t - (e >> 1) * 8;
            p[j][e] = back <= 0 ? p[j][e] : 0.f, mm[e] = back < 0 ? mm[e] : 0.f;
          }
          big[e >> 1] = fmaxf(big[e >> 1], fabsf(p[j][e]));
        }
        *reinterpret_cast<float2*>(M + t * kMs + s) = make_float2(mm[0], mm[1]);
        *reinterpret_cast<float2*>(M + (t + 8) * kMs + s) = make_float2(mm[2], mm[3]);
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      big[i] = fmaxf(big[i], __shfl_xor_sync(0xffffffffu, big[i], 1));
      big[i] = fmaxf(big[i], __shfl_xor_sync(0xffffffffu, big[i], 2));
      if ((lane & 3) == 0) pmax[(warp >> 2) * kL + r0 + (lane >> 2) + i * 8] = big[i];
    }
    __syncthreads();
    const float* beta = fac + kBeta * kL;
    if (upper) {  // R: two 16 x 16 diagonal blocks a warp, a column a lane, then their join
      if (warp == 4 && !ONE && h + 1 < (hk + 1) * group) load_gates(h + 1);
      const int pair = warp - 4, top = pair * 32 + (lane & 16), s = lane & 15;
      float y[16];  // beta_i R[i][s]
#pragma unroll
      for (int t = 0; t < 16; ++t) {
        float m[16], x[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < t; i += 4) {
          const float4 v = *reinterpret_cast<const float4*>(M + (top + t) * kMs + top + i);
          m[i] = v.x, m[i + 1] = v.y, m[i + 2] = v.z, m[i + 3] = v.w;
        }
#pragma unroll
        for (int i = 0; i < t; ++i) x[i & 3] = fmaf(m[i], y[i], x[i & 3]);
        const float r = t > s ? -(M[(top + t) * kMs + top + s] + ((x[0] + x[1]) + (x[2] + x[3]))) : 0.f;
        R[(top + t) * kMs + top + s] = r;
        y[t] = beta[top + t] * r;
        if (lane >= 16) R[(pair * 32 + t) * kMs + pair * 32 + lane] = 0.f;  // the second join reads these too
      }
      __syncwarp();
      join<16>(M, R, X + pair * 16 * kMs, beta, pair * 32, 0, 0, lane, [] { __syncwarp(); });
      join<16>(M, R, X + pair * 16 * kMs, beta, pair * 32, 0, 1, lane, [] { __syncwarp(); });
    } else {  // P, and the factors but R's
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int t = r0 + (lane >> 2) + i * 8;
        const Scale sc = scale_of(fmaxf(pmax[t], pmax[kL + t]));
        if (c0 == 0 && (lane & 3) == 0) fout[kPInv * kL + t] = sc.inv;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t hi, lo;
          split(p[j][2 * i] * sc.mul, p[j][2 * i + 1] * sc.mul, hi, lo);
          char* at = out + 2 * kTile + piece_at<kL>(t, c0 + j * 8) + (lane & 3) * 4;
          *reinterpret_cast<uint32_t*>(at) = hi;
          if constexpr (P2) *reinterpret_cast<uint32_t*>(at + kTile) = lo;
        }
      }
      for (int e = warp < 4 ? tid : tid - 64; e < kFactors * kL; e += 192)
        if (e / kL != kRInv && e / kL != kPInv) fout[e] = fac[e];
    }
    __syncthreads();
    join<32>(M, R, X, beta, 0, warp >> 2, warp & 3, lane, [&] { sm100::named_bar(3 + (warp & 3), 64); });
    __syncthreads();
    {  // R, rows scaled: four threads a row, 16 columns each, zeros above the diagonal's block
      const int row = tid >> 2, part = tid & 3;
      const bool below = part * 16 <= row;
      float x[16], m = 0.f;
#pragma unroll
      for (int e = 0; e < 16; e += 4) {
        const float4 v = below ? *reinterpret_cast<const float4*>(R + row * kMs + part * 16 + e)
                               : make_float4(0.f, 0.f, 0.f, 0.f);
        x[e] = v.x, x[e + 1] = v.y, x[e + 2] = v.z, x[e + 3] = v.w;
        m = fmaxf(fmaxf(fmaxf(m, fabsf(v.x)), fmaxf(fabsf(v.y), fabsf(v.z))), fabsf(v.w));
      }
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
      const Scale sc = scale_of(m);
      if (part == 0) fout[kRInv * kL + row] = sc.inv;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) split(x[i * 8 + 2 * e] * sc.mul, x[i * 8 + 2 * e + 1] * sc.mul, hi[e], lo[e]);
        const int at = piece_at<kL>(row, part * 16 + i * 8);
        *reinterpret_cast<uint4*>(out + at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4*>(out + kTile + at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        if (row < 32 && part >= 2) {  // P's upper quarter
          *reinterpret_cast<uint4*>(out + 2 * kTile + at) = make_uint4(0, 0, 0, 0);
          if constexpr (P2) *reinterpret_cast<uint4*>(out + 3 * kTile + at) = make_uint4(0, 0, 0, 0);
        }
      }
    }
    if (!ONE && h + 1 < (hk + 1) * group) {  // fac, M, R belong to the next head
      __syncthreads();
      if (warp == 4) gates();
      __syncthreads();
    }
  }
}

}  // namespace

template <typename T, int KP, bool P2>
cudaError_t launch_prep(const GdrArgs& a, char* keys, char* records, cudaStream_t stream) {
  constexpr int smem = prep_smem<KP, sizeof(T) == 4 ? 2 : 1>();
  const auto kernel = a.H == a.HK ? gdr_prep_kernel<T, KP, P2, true> : gdr_prep_kernel<T, KP, P2, false>;
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
cudaError_t chunk(const GdrArgs& a, char* ws, cudaStream_t stream) {
  constexpr bool P2 = sizeof(T) == 4;
  char* keys = ws + kGdrHeader;
  char* records = keys + record_count(a) * a.HK * keys_bytes(KP, sizeof(T) == 4 ? 2 : 1);
  cudaError_t e = launch_prep<T, KP, P2>(a, keys, records, stream);
  if (e != cudaSuccess) return e;
  if constexpr (sizeof(T) == 2)
    if (gdr_tc_pass(a)) return launch_tc_walk<KP>(a, keys, records, (unsigned int*)ws, stream);
  return launch_walk<T, KP, false>(a, keys, records, Kept{}, stream);
}

}  // namespace
}  // namespace gdr

bool gdr_chunk_supported(int K) { return K <= 128; }

// bf16 inputs: whichever pass takes less (walk_cost).
bool gdr_tc_pass(const GdrArgs& a) {
  if (!a.dtype) return false;
  const int tn = a.K <= 64 ? gdr::tiles_a_block<__nv_bfloat16, 64, false>(a) : gdr::tiles_a_block<__nv_bfloat16, 128, false>(a);
  return gdr::walk_cost(a, 0) < gdr::walk_cost(a, tn);
}

size_t gdr_chunk_workspace_bytes(const GdrArgs& a) {
  const int np = a.dtype ? 1 : 2, KP = a.K <= 64 ? 64 : 128;
  return kGdrHeader + (size_t)gdr::record_count(a) *
                          ((size_t)a.HK * gdr::keys_bytes(KP, np) + (size_t)a.H * gdr::record_bytes(a.dtype == 0));
}

cudaError_t launch_gdr_chunk(const GdrArgs& a, void* workspace, cudaStream_t stream) {
  char* ws = (char*)workspace;
  if (a.dtype)
    return a.K <= 64 ? gdr::chunk<__nv_bfloat16, 64>(a, ws, stream) : gdr::chunk<__nv_bfloat16, 128>(a, ws, stream);
  return a.K <= 64 ? gdr::chunk<float, 64>(a, ws, stream) : gdr::chunk<float, 128>(a, ws, stream);
}

}  // namespace mlstm
