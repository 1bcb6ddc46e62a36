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
// Layout.  Four warps own 16 value columns: each has a quarter of the keys of the transposed state
// S^T [16 x K] in registers, as accumulators of m16n8k16, and a quarter of the chunk's tokens of Z, U and O.
// An accumulator is in the right place to be the next product's A operand; the four exchange these
// operands through shared memory, each quarter with its own power of two, and every product of a quarter
// is summed from zero and scaled on its way into an fp32 sum.  k, q, R and P are B operands, read by
// ldmatrix.  (One warp with all keys and tokens of its columns was measured first: it needs no
// exchange, but 255 registers, and with one or two warps to a scheduler the products waited for the
// splitting between them.)
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"
#include "kernels.h"

namespace mlstm {
namespace gdr {

constexpr int kL = 64;       // tokens of a chunk
constexpr int kQuarter = 4;  // warps of a tile of 16 value columns

// ---------------------------------------------------------------- a chunk's records in the workspace
// For each chunk and key head: k and q as [64][KP] fp16, KP = 64 or 128 (zeros behind K and behind the
// sequence's end), NP parts each.  For each chunk and value head: R (hi, lo) and P (hi, lo where P2) as
// [64][64] fp16, then the per-token factors.  The 16-byte pieces of a row of these tiles are permuted
// by the row, so that a record is copied as it is and ldmatrix meets no bank conflicts.
// kGK = gam / k's scale and so on: what the passes over the chunks multiply by; the rest is for the others.
enum { kGK = 0, kGQ, kWK, kBeta, kRInv, kPInv, kGam, kW, kKInv, kQInv, kG, kFactors = kG + 2 };  // kG: G / ln 2 in two parts
constexpr int kTile = kL * kL * 2;
constexpr int kFactorBytes = kFactors * kL * 4;
__host__ __device__ constexpr int keys_bytes(int KP, int np) { return 2 * np * kL * KP * 2; }
__host__ __device__ constexpr int record_bytes(bool p2) { return (p2 ? 4 : 3) * kTile + kFactorBytes; }
// Byte offset of the 16-byte piece that holds (row, col) of a tile with W columns: blocks of 64 columns (128
// bytes a row, ROWS rows), as the tensor cores' 128-byte swizzle has it.
template <int W, int ROWS = kL>
__device__ __forceinline__ int piece_at(int row, int col) {
  return (W > 64 ? (col >> 6) * (ROWS * 128) : 0) + row * 128 + ((((col >> 3) ^ row) & 7) << 4);
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

// A sum in 64 bits (in units of ln 2) as two fp32 parts, and the decay 2^(a - b) between two: the difference keeps
// fp32's relative accuracy however large the sums are.
constexpr double kPerLn2 = 1.4426950408889634;
__device__ __forceinline__ float2 two_parts(double x) {
  const float hi = (float)x;
  return make_float2(hi, (float)(x - hi));
}
__device__ __forceinline__ float decay_between(float2 a, float2 b) { return exp2f((a.x - b.x) + (a.y - b.y)); }

// Cumulative log decays of a chunk: lane has those of tokens 2 lane (x) and 2 lane + 1 (y), and brings theirs
// (0 where there is no token).
__device__ __forceinline__ double2 cumulative(float g0, float g1, int lane) {
  const double x0 = log_decay(g0), x1 = log_decay(g1);
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
template <int N>
__device__ __forceinline__ void cp_wait() {  // all but the last N groups have come
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// the four warps of tile `tile` of the block (barrier 0 is the block's)
__device__ __forceinline__ void tile_barrier(int tile) {
  asm volatile("bar.sync %0, %1;" ::"r"(tile + 1), "n"(32 * kQuarter) : "memory");
}

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

// c = a b
__device__ __forceinline__ void mma_new(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
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
// 8 consecutive elements, zeros where !in
__device__ __forceinline__ void load8(const float* p, bool in, float (&x)[8]) {
  const float4 none = make_float4(0.f, 0.f, 0.f, 0.f);
  const float4 u = in ? *reinterpret_cast<const float4*>(p) : none, v = in ? *reinterpret_cast<const float4*>(p + 4) : none;
  x[0] = u.x, x[1] = u.y, x[2] = u.z, x[3] = u.w, x[4] = v.x, x[5] = v.y, x[6] = v.z, x[7] = v.w;
}

// x, y (already scaled) as two fp16 parts
__device__ __forceinline__ void split(float x, float y, uint32_t& hi, uint32_t& lo) {
  hi = pack(x, y);
  const float2 b = unpack(hi);
  lo = pack(x - b.x, y - b.y);
}
// Two neighbouring accumulator tiles (16 columns) times f as an A operand in two parts.
__device__ __forceinline__ void split_a(const float (&c0)[4], const float (&c1)[4], float f, uint4& hi, uint4& lo) {
  split(c0[0] * f, c0[1] * f, hi.x, lo.x);
  split(c0[2] * f, c0[3] * f, hi.y, lo.y);
  split(c1[0] * f, c1[1] * f, hi.z, lo.z);
  split(c1[2] * f, c1[3] * f, hi.w, lo.w);
}
// The power of two of a warp's accumulator tiles, as scale_of, from their largest finite magnitude.  What is not
// finite spoils its own column (a row of the operand); were it the largest, the tile's other columns would be
// scaled to nothing.  A lane's two columns, the rows r and r + 8, are compared as integers one exponent up: those
// that hold an infinity (or nothing but NaN) wrap below zero and are left out, at one addition each.  (A second
// look at the values where the largest is infinite: 16 heads of 128 x 128, 8192 tokens 220 -> 232 us; this: 219.)
template <int N>
__device__ __forceinline__ Scale tile_scale(const float (&c)[N][4]) {
  float m[2];
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    m[r] = fmaxf(fabsf(c[0][2 * r]), fabsf(c[0][2 * r + 1]));
#pragma unroll
    for (int j = 1; j < N; ++j) m[r] = fmaxf(m[r], fmaxf(fabsf(c[j][2 * r]), fabsf(c[j][2 * r + 1])));
  }
  constexpr int up = 1 << 23;
  const int top = max((int)(__float_as_uint(m[0]) + up), (int)(__float_as_uint(m[1]) + up));
  const int e = max(__reduce_max_sync(0xffffffffu, top) >> 23, 21);  // biased exponent + 1, at most 255
  return Scale{__uint_as_float((uint32_t)(269 - e) << 23), __uint_as_float((uint32_t)(e - 15) << 23)};
}

// One k step of a product of a quarter: acc (two or more tiles of 8 columns) += A B, or = A B where FRESH,
// for NA parts of A and NB of B, the planes of B `plane` bytes apart.  lo parts first: they are small, and
// so is what the tensor cores' sums cut off below them.  load(tile pair, plane) gives the B fragments.
template <bool FRESH, int NT, int NA, int NB, class Load>
__device__ __forceinline__ void step(float (&acc)[NT][4], const uint4& ah, const uint4& al, Load load) {
  const uint32_t hi[4] = {ah.x, ah.y, ah.z, ah.w}, lo[4] = {al.x, al.y, al.z, al.w};
#pragma unroll
  for (int j = 0; j < NT; j += 2) {
    uint32_t b[4];
    load(b, j, 0);
    bool fresh = FRESH;
    auto add = [&](const uint32_t (&a)[4], const uint32_t (&f)[4]) {
      if (fresh)
        mma_new(acc[j], a, f[0], f[1]), mma_new(acc[j + 1], a, f[2], f[3]);
      else
        mma(acc[j], a, f[0], f[1]), mma(acc[j + 1], a, f[2], f[3]);
      fresh = false;
    };
    if constexpr (NA == 2) add(lo, b);
    if constexpr (NB == 2) {
      uint32_t l[4];
      load(l, j, 1);
      add(hi, l);
    }
    add(hi, b);
  }
}
template <int NT>
__device__ __forceinline__ void zero(float (&acc)[NT][4]) {
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[j][e] = 0.f;
}
template <int NT>
__device__ __forceinline__ void add_scaled(float (&sum)[NT][4], const float (&x)[NT][4], float f) {
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) sum[j][e] = fmaf(x[j][e], f, sum[j][e]);
}

// Factors of the tokens t0 + 8j + 2 (lane & 3) + {0, 1}
__device__ __forceinline__ float2 factor(const float* f, int t0, int j, int lane) {
  return *reinterpret_cast<const float2*>(f + t0 + 8 * j + 2 * (lane & 3));
}

// Sum over the 16 columns of a quarter's two tiles, per token: v[2j + e] is this lane's share of token
// 8j + 2 (lane & 3) + e.  Lanes 16 j + (lane & 3) have the sums of tile j's tokens.
__device__ __forceinline__ float2 column_sum(const float (&v)[4], int lane) {
  const bool up = lane & 16;
  float x = (up ? v[2] : v[0]) + __shfl_xor_sync(0xffffffffu, up ? v[0] : v[2], 16);
  float y = (up ? v[3] : v[1]) + __shfl_xor_sync(0xffffffffu, up ? v[1] : v[3], 16);
#pragma unroll
  for (int d = 8; d > 2; d /= 2) {
    x += __shfl_xor_sync(0xffffffffu, x, d);
    y += __shfl_xor_sync(0xffffffffu, y, d);
  }
  return make_float2(x, y);
}

}  // namespace gdr
}  // namespace mlstm
