// Building blocks of the gated delta rule's chunk kernels (gdr_chunk.cu, gdr_bwd.cu).
//
// Inside a chunk of 64 tokens, with G_t the cumulative log decay, gam_t = e^{G_t}, w_t = e^{G_63 - G_t}
// and D[t,s] = e^{G_t - G_s} (s <= t), S the state at its start:
//     M[t,s] = (k_t . k_s) D[t,s]  (s < t)        P[t,s] = (q_t . k_s) D[t,s]  (s <= t)
//     Z  = V - gam (K S)                          what is left of v if only S were read
//     Z' = (I + M beta)^{-1} Z = Z + R (beta Z)   v_t - r_t, token by token
//     U  = beta Z'     O = gam (Q S) + P U        S <- gam_63 S + (w K)^T U
// R = (I + M beta)^{-1} M, negated, is strictly lower triangular and holds no beta of its own row or
// column, so the gradients use it transposed and a token with beta = 0 divides by nothing:
//     dU = P^T dO + w (K dS)      dY = dU + R^T (beta dU)      dV = beta dY      dbeta = dY . Z'
//     dS <- gam_63 dS + Q^T (gam dO) - K^T (gam dV)
//     dg_t = sum over tau >= t of (dO . O - dV . V)_tau + <dS, S> at the chunk's end
//
// Precision.  The products run on the tensor cores with 16-bit operands and fp32 sums, and states and
// gate gradients are to be as exact as fp32 gives them.  So an fp32 operand is split into two fp16
// parts (22 bits), a bf16 input fits one part, and a product of two split operands takes three matrix
// products (the fourth is below 2^-22).  fp16's short exponent is met by powers of two: every row of
// k, q, R and P and every warp's tile of the state and of the values is scaled so that its largest
// value lies in [2^14, 2^15), which keeps 22 bits of values down to 2^-17 of it and 11 down to 2^-28.
//
// Layout.  A warp owns 16 value columns with the state transposed, S^T [16 x K], in registers as the
// accumulator of m16n8k16; an accumulator is in the right place to be the next product's A operand,
// so Z, U and S pass from product to product without leaving the registers.  k, q, R, P are B
// operands read by ldmatrix from shared memory.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"
#include "kernels.h"

namespace mlstm {
namespace gdr {

constexpr int kL = 64;  // tokens of a chunk

// ---------------------------------------------------------------- a chunk's records in the workspace
// For each chunk and key head: k and q as [64][KP] fp16, KP = 64 or 128 (zeros behind K and behind the
// sequence's end), NP parts each.  For each chunk and value head: R (hi, lo) and P (hi, lo where P2) as
// [64][64] fp16, then the per-token factors.  The 16-byte pieces of a row of these tiles are permuted
// by the row, so that a record is copied as it is and ldmatrix meets no bank conflicts.
enum { kGam = 0, kW, kBeta, kKInv, kQInv, kRInv, kPInv, kFactors };
constexpr int kTile = kL * kL * 2;
constexpr int kFactorBytes = kFactors * kL * 4;
__host__ __device__ constexpr int keys_bytes(int KP, int np) { return 2 * np * kL * KP * 2; }
__host__ __device__ constexpr int record_bytes(bool p2) { return (p2 ? 4 : 3) * kTile + kFactorBytes; }
// byte offset of the 16-byte piece that holds (row, col) of a tile with W columns
template <int W>
__device__ __forceinline__ int piece_at(int row, int col) {
  return row * W * 2 + (((col >> 3) ^ (row & 7)) << 4);
}

// ------------------------------------------------------------------------------------- sequences
struct Seq {
  long long b, lo, len;  // batch row, first token, tokens
  long long slot;        // record of its first chunk
};
// Offsets come from the device and are bounded here to the tokens that there are.  Packed sequence n
// takes records from lo / 64 + n on: they are disjoint and end below T / 64 + N.
__device__ __forceinline__ Seq sequence(const GdrArgs& a, int n) {
  Seq s;
  if (a.packed) {
    s.b = 0;
    s.lo = min(max((long long)a.offsets[n], 0LL), (long long)a.T);
    s.len = min(max((long long)a.offsets[n + 1], s.lo), (long long)a.T) - s.lo;
    s.slot = s.lo / kL + n;
  } else {
    s.b = n;
    s.lo = 0;
    s.len = a.T;
    s.slot = (long long)n * ((a.T + kL - 1) / kL);
  }
  return s;
}
inline long long record_count(const GdrArgs& a) {
  return a.packed ? (long long)a.T / kL + a.N : (long long)a.N * ((a.T + kL - 1) / kL);
}
// The sequence and chunk of a record; false where the record belongs to none.
__device__ __forceinline__ bool find_chunk(const GdrArgs& a, long long rec, int* n, Seq* s, int* c) {
  if (!a.packed) {
    const long long per = (a.T + kL - 1) / kL;
    *n = (int)(rec / per);
  } else {
    int lo = 0, hi = a.N - 1;  // the last sequence whose records begin at or before rec
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      const long long first = min(max((long long)a.offsets[mid], 0LL), (long long)a.T) / kL + mid;
      if (first <= rec)
        lo = mid;
      else
        hi = mid - 1;
    }
    *n = lo;
  }
  *s = sequence(a, *n);
  const long long chunk = rec - s->slot;
  *c = (int)chunk;
  return chunk >= 0 && chunk * kL < s->len;
}

// e^g as a sum's term: a decay below e^-10000 (and -infinity) is as good as a full reset, and sums of
// 64 such terms keep every smaller one exactly in 64 bits.  NaN stays NaN.
__device__ __forceinline__ double log_decay(float g) { return g < -1e4f ? -1e4 : (double)g; }

// A sum in 64 bits as two fp32 parts, and the decay e^(a - b) between two of them: the difference keeps
// fp32's relative accuracy however large the sums are.
__device__ __forceinline__ float2 two_parts(double x) {
  const float hi = (float)x;
  return make_float2(hi, (float)(x - hi));
}
__device__ __forceinline__ float decay_between(float2 a, float2 b) { return expf((a.x - b.x) + (a.y - b.y)); }

// Cumulative log decays of the chunk that begins at token t0: lane has those of tokens 2 lane (x) and
// 2 lane + 1 (y); no decay from `len` on.
__device__ __forceinline__ double2 cumulative(const float* g, long long st, long long t0, int len, int lane) {
  const int t = 2 * lane;
  const double x0 = t < len ? log_decay(g[(t0 + t) * st]) : 0.0, x1 = t + 1 < len ? log_decay(g[(t0 + t + 1) * st]) : 0.0;
  double sum = x0 + x1;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const double y = __shfl_up_sync(0xffffffffu, sum, d);
    if (lane >= d) sum += y;
  }
  return make_double2(sum - x1, sum);
}

// ------------------------------------------------------------------------------------ small pieces
__device__ __forceinline__ uint32_t smem_u32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool in) {
  const int n = in ? 16 : 0;  // the rest of the 16 bytes is filled with zeros
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void cp_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}
__device__ __forceinline__ void stsm4t(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(a), "r"(b), "r"(c),
               "r"(d)
               : "memory");
}
// c += a b, fp16 operands
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// c += a b, tf32 operands
__device__ __forceinline__ void mma_tf32(float (&c)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}
// x in two tf32 parts (22 bits)
__device__ __forceinline__ void split_tf32(float x, uint32_t& hi, uint32_t& lo) {
  asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(hi) : "f"(x));
  const float rest = x - __uint_as_float(hi);
  asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(lo) : "f"(rest));
}

// Lane addresses of ldmatrix.x4 on a tile whose rows are `row`-indexed from r0 and columns from c0:
// plain: two B tiles (n = 16 rows, k = 16 columns); transposed: two B tiles (k = 16 rows, n = 16 columns).
__device__ __forceinline__ int b_row(int lane) { return (lane >> 4) * 8 + (lane & 7); }
__device__ __forceinline__ int b_col(int lane) { return ((lane >> 3) & 1) * 8; }
__device__ __forceinline__ int bt_row(int lane) { return ((lane >> 3) & 1) * 8 + (lane & 7); }
__device__ __forceinline__ int bt_col(int lane) { return (lane >> 4) * 8; }
// transposed A operand or accumulator tile: rows are k (16), columns are m (16)
__device__ __forceinline__ int at_row(int lane) { return (lane >> 4) * 8 + (lane & 7); }
__device__ __forceinline__ int at_col(int lane) { return ((lane >> 3) & 1) * 8; }

// The power of two that takes a largest magnitude m to [2^14, 2^15), and its inverse.
struct Scale {
  float mul, inv;
};
__device__ __forceinline__ Scale scale_of(float m) {
  const uint32_t e = min(max(__float_as_uint(m) >> 23, 20u), 254u);
  return Scale{__uint_as_float((268u - e) << 23), __uint_as_float((e - 14u) << 23)};
}
__device__ __forceinline__ float warp_max(float m) {  // of magnitudes
  return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));
}

__device__ __forceinline__ uint32_t pack(float x, float y) {
  const __half2 h = __floats2half2_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack(uint32_t u) { return __half22float2(*reinterpret_cast<const __half2*>(&u)); }
__device__ __forceinline__ float2 unpack_bf16(uint32_t u) {
  return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}
__device__ __forceinline__ uint32_t pack_bf16(float x, float y) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// 8 consecutive elements as fp32, zeros where !in
template <typename T>
__device__ __forceinline__ void load8(const T* p, bool in, float (&x)[8]) {
  if (!in) {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = 0.f;
  } else if constexpr (sizeof(T) == 2) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 f = unpack_bf16(u[e]);
      x[2 * e] = f.x, x[2 * e + 1] = f.y;
    }
  } else {
    const float4 u = *reinterpret_cast<const float4*>(p), v = *reinterpret_cast<const float4*>(p + 4);
    x[0] = u.x, x[1] = u.y, x[2] = u.z, x[3] = u.w, x[4] = v.x, x[5] = v.y, x[6] = v.z, x[7] = v.w;
  }
}

// x, y (already scaled) as two fp16 parts
__device__ __forceinline__ void split(float x, float y, uint32_t& hi, uint32_t& lo) {
  hi = pack(x, y);
  const float2 b = unpack(hi);
  lo = pack(x - b.x, y - b.y);
}
// Two neighbouring accumulator tiles (16 columns) times f as an A operand in two parts.
__device__ __forceinline__ void split_a(const float (&c0)[4], const float (&c1)[4], float f, uint32_t (&hi)[4],
                                        uint32_t (&lo)[4]) {
  split(c0[0] * f, c0[1] * f, hi[0], lo[0]);
  split(c0[2] * f, c0[3] * f, hi[1], lo[1]);
  split(c1[0] * f, c1[1] * f, hi[2], lo[2]);
  split(c1[2] * f, c1[3] * f, hi[3], lo[3]);
}
template <int N>
__device__ __forceinline__ float tile_max(const float (&c)[N][4]) {
  float m = 0.f;
#pragma unroll
  for (int j = 0; j < N; ++j) m = fmaxf(m, fmaxf(fmaxf(fabsf(c[j][0]), fabsf(c[j][1])), fmaxf(fabsf(c[j][2]), fabsf(c[j][3]))));
  return warp_max(m);
}

// acc[j] (j = tokens 8j ..) += A [16 x 16] B, B = columns 16 kk .. of the rows of a [64][KP] tile: one k
// step of A times the tile's transpose.  NP: parts of B (a plane further on).  lo parts first: they are
// small, and so is what the tensor cores' sums cut off below them.
template <int KP, int NP, bool LO_A>
__device__ __forceinline__ void rows_step(float (&acc)[8][4], const uint32_t (&hi)[4], const uint32_t (&lo)[4],
                                          uint32_t tile, int kk, int lane) {
  const uint32_t at = tile + piece_at<KP>(b_row(lane), kk * 16 + b_col(lane));
  uint32_t b[4][4];
#pragma unroll
  for (int j = 0; j < 4; ++j) ldsm4(b[j], at + j * 16 * KP * 2);
  if constexpr (LO_A) {
#pragma unroll
    for (int j = 0; j < 4; ++j) mma(acc[2 * j], lo, b[j][0], b[j][1]), mma(acc[2 * j + 1], lo, b[j][2], b[j][3]);
  }
  if constexpr (NP == 2) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t l[4];
      ldsm4(l, at + kL * KP * 2 + j * 16 * KP * 2);
      mma(acc[2 * j], hi, l[0], l[1]), mma(acc[2 * j + 1], hi, l[2], l[3]);
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) mma(acc[2 * j], hi, b[j][0], b[j][1]), mma(acc[2 * j + 1], hi, b[j][2], b[j][3]);
}

// S = keep S + f A B, A [16 x 64] in two parts, B = a [64][KP] tile: the state's update.  Each product is
// summed from zero and added in fp32: the tensor cores' sums never run over the state's own bits.
template <int KP, int NP>
__device__ __forceinline__ void state_add(float (&S)[KP / 8][4], float keep, const uint32_t (&hi)[4][4],
                                          const uint32_t (&lo)[4][4], float f, uint32_t tile, int lane) {
#pragma unroll
  for (int j = 0; j < KP / 8; j += 4) {
    float d[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) d[i][e] = 0.f;
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
      const uint32_t at = tile + kk * 16 * KP * 2;
      uint32_t b[4], c[4];
      const int at0 = piece_at<KP>(bt_row(lane), j * 8 + bt_col(lane));
      const int at1 = piece_at<KP>(bt_row(lane), j * 8 + 16 + bt_col(lane));
      ldsm4t(b, at + at0);
      ldsm4t(c, at + at1);
      mma(d[0], lo[kk], b[0], b[1]), mma(d[1], lo[kk], b[2], b[3]);
      mma(d[2], lo[kk], c[0], c[1]), mma(d[3], lo[kk], c[2], c[3]);
      if constexpr (NP == 2) {
        uint32_t l[4], m[4];
        ldsm4t(l, at + kL * KP * 2 + at0);
        ldsm4t(m, at + kL * KP * 2 + at1);
        mma(d[0], hi[kk], l[0], l[1]), mma(d[1], hi[kk], l[2], l[3]);
        mma(d[2], hi[kk], m[0], m[1]), mma(d[3], hi[kk], m[2], m[3]);
      }
      mma(d[0], hi[kk], b[0], b[1]), mma(d[1], hi[kk], b[2], b[3]);
      mma(d[2], hi[kk], c[0], c[1]), mma(d[3], hi[kk], c[2], c[3]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) S[j + i][e] = fmaf(keep, S[j + i][e], f * d[i][e]);
  }
}

// acc[j] += sum over k of A[., k] X[t, k] (TRANS: X[k, t]) for a swizzled lower triangular 64 x 64 X:
// plain, columns k <= t count; transposed, rows k >= t.  NA, NX: parts of A and of X.
template <bool TRANS, int NA, int NX>
__device__ __forceinline__ void triangle(float (&acc)[8][4], const uint32_t (&hi)[4][4], const uint32_t (&lo)[4][4],
                                         uint32_t tile, int lane) {
#pragma unroll
  for (int kk = 0; kk < 4; ++kk) {
#pragma unroll
    for (int jj = TRANS ? 0 : kk; jj < (TRANS ? kk + 1 : 4); ++jj) {  // tokens 16 jj .. + 15 of the result
      const int row = TRANS ? kk * 16 + bt_row(lane) : jj * 16 + b_row(lane);
      const int col = TRANS ? jj * 16 + bt_col(lane) : kk * 16 + b_col(lane);
      const uint32_t at = tile + piece_at<kL>(row, col);
      uint32_t b[4];
      if constexpr (TRANS)
        ldsm4t(b, at);
      else
        ldsm4(b, at);
      if constexpr (NA == 2) mma(acc[2 * jj], lo[kk], b[0], b[1]), mma(acc[2 * jj + 1], lo[kk], b[2], b[3]);
      if constexpr (NX == 2) {
        uint32_t l[4];
        if constexpr (TRANS)
          ldsm4t(l, at + kTile);
        else
          ldsm4(l, at + kTile);
        mma(acc[2 * jj], hi[kk], l[0], l[1]), mma(acc[2 * jj + 1], hi[kk], l[2], l[3]);
      }
      mma(acc[2 * jj], hi[kk], b[0], b[1]), mma(acc[2 * jj + 1], hi[kk], b[2], b[3]);
    }
  }
}

// acc (16 columns x 64 tokens) times f[token] of a factor row
__device__ __forceinline__ float2 factor(const float* f, int j, int lane) {
  return *reinterpret_cast<const float2*>(f + 8 * j + 2 * (lane & 3));
}

// Sum over the warp's 16 columns of a tile, per token: v[2j + e] holds this lane's share of token
// 8j + 2 (lane & 3) + e; lane (lane >> 2) = j of the result has the sums of tokens 8j + 2 (lane & 3) + {0, 1}.
__device__ __forceinline__ float2 column_sum(float (&v)[16], int lane) {
#pragma unroll
  for (int half = 8; half > 1; half /= 2) {
    // lanes with this bit of j set keep the upper half of the tokens
    const int bit = half * 2;  // 16, 8, 4: lane bits 4, 3, 2 are bits 2, 1, 0 of lane >> 2
    const bool up = lane & bit;
#pragma unroll
    for (int i = 0; i < half; ++i) {
      const float mine = up ? v[i + half] : v[i], theirs = up ? v[i] : v[i + half];
      v[i] = mine + __shfl_xor_sync(0xffffffffu, theirs, bit);
    }
  }
  return make_float2(v[0], v[1]);
}

}  // namespace gdr
}  // namespace mlstm
