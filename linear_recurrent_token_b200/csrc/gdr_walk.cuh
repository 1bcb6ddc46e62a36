// The pass over a sequence's chunks: forward for outputs and states, or again for the gradients, which
// keep what they need of it.
#pragma once

#include "gdr_tile.cuh"

namespace mlstm {
namespace gdr {

// What the gradients keep of the forward pass, by record of a chunk and value head (states: one more
// a sequence, the final one) and by tile of 16 value columns.  Operands are stored in the order of the
// fragments, 512 bytes a warp and step.
struct Kept {
  uint4* S;       // S^T at the chunk's start: [state][tile][2 parts][KP / 16][32]
  float* S_inv;   // the parts' scale: [state][tile]
  float4* Z;      // Z': [record][tile][8][32]
  uint4* U;       // U^T: [record][tile][NK parts][4][32]
  float* U_inv;   // [record][tile]
  float* dots;    // dO . O, then dO . O - dV . V, over the tile's columns: [record][tile][64]
  // of the pass backward
  uint4* D;       // dS^T at the chunk's end: [record][tile][NK parts][KP / 16][32]
  float* D_inv;   // [record][tile]
  uint4* dV;      // dV^T: [record][tile][NK parts][4][32]
  float* dV_inv;  // [record][tile]
  float* dbeta;   // dY . Z' over the tile's columns: [record][tile][64]
  float* ends;    // <dS, S> at the chunk's end over the tile's columns: [record][tile]
};
// Parts of an operand that only products rounded to the output's type read: one for bf16 (11 bits).
template <typename T>
constexpr int kept_parts() { return sizeof(T) == 4 ? 2 : 1; }

// Four fragment registers of each of `steps` steps as they lie in a warp.
__device__ __forceinline__ void keep(uint4* at, int step, int lane, const uint32_t (&r)[4]) {
  at[step * 32 + lane] = make_uint4(r[0], r[1], r[2], r[3]);
}

template <typename T, int KP, bool P2>
cudaError_t launch_prep(const GdrArgs& a, char* keys, char* records, cudaStream_t stream);

// bytes of shared memory of one stage: k, q, the columns of v (and dO), the record
template <typename T, int KP, int W, bool GRAD>
struct WalkStage {
  static constexpr int NP = sizeof(T) == 4 ? 2 : 1;
  static constexpr bool P2 = sizeof(T) == 4 || GRAD;
  static constexpr int row = 16 * W * (int)sizeof(T) + 16;  // odd multiples of 16 bytes: no bank conflicts
  static constexpr int q = keys_bytes(KP, NP) / 2;
  static constexpr int v = keys_bytes(KP, NP);
  static constexpr int dout = v + kL * row;
  static constexpr int record = dout + (GRAD ? kL * row : 0);
  static constexpr int factors = record + (P2 ? 4 : 3) * kTile;
  static constexpr int bytes = record + record_bytes(P2);
  static constexpr int stages = 2 * bytes <= 227 * 1024 ? 2 : 1;
};

// Copies one chunk into a stage: every thread a share, 16 bytes at a time.
template <typename T, int KP, int W, bool GRAD>
__device__ __forceinline__ void fetch_chunk(const GdrArgs& a, const Seq& s, long long rec, int h, int c, int col0,
                                            const char* keys, const char* records, uint32_t stage) {
  using L = WalkStage<T, KP, W, GRAD>;
  const int tid = threadIdx.x;
  constexpr int threads = 32 * W;
  const char* k = keys + (rec * a.HK + h / (a.H / a.HK)) * keys_bytes(KP, L::NP);
  for (int i = tid; i < keys_bytes(KP, L::NP) / 16; i += threads) cp_async16(stage + i * 16, k + i * 16, true);
  const char* r = records + (rec * a.H + h) * record_bytes(L::P2);
  for (int i = tid; i < record_bytes(L::P2) / 16; i += threads) cp_async16(stage + L::record + i * 16, r + i * 16, true);
  constexpr int per = 16 / sizeof(T), pieces = 16 * W / per;  // of a row
  const long long t0 = (long long)c * kL;
  const T* v = (const T*)a.v + s.b * a.sv.b + h * a.sv.h;
  const T* d = GRAD ? (const T*)a.dout + s.b * a.so.b + h * a.so.h : nullptr;
  for (int i = tid; i < kL * pieces; i += threads) {
    const int row = i / pieces, col = i % pieces * per;
    const bool in = t0 + row < s.len && col0 + col < a.V;
    const long long t = in ? s.lo + t0 + row : 0;
    cp_async16(stage + L::v + row * L::row + col * (int)sizeof(T), in ? v + t * a.sv.t + col0 + col : v, in);
    if (GRAD) cp_async16(stage + L::dout + row * L::row + col * (int)sizeof(T), in ? d + t * a.so.t + col0 + col : d, in);
  }
  cp_commit();
}

// The warp's 16 columns x 64 tokens of a tile [64][16 W] in shared memory, as an accumulator.
template <typename T, int ROW>
__device__ __forceinline__ void read_columns(float (&x)[8][4], const char* tile, uint32_t tile_u, int lane) {
  if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int jj = 0; jj < 4; ++jj) {
      uint32_t r[4];
      ldsm4t(r, tile_u + (jj * 16 + at_row(lane)) * ROW + at_col(lane) * 2);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = unpack_bf16(r[i]);
        x[2 * jj + (i >> 1)][(i & 1) * 2] = f.x;
        x[2 * jj + (i >> 1)][(i & 1) * 2 + 1] = f.y;
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        x[j][e] = *reinterpret_cast<const float*>(tile + (8 * j + 2 * (lane & 3) + (e & 1)) * ROW +
                                                  ((lane >> 2) + (e >> 1) * 8) * 4);
  }
}

// The inverse, and from there to memory: out points at column col0 of token 0 of the chunk.  The
// warp's own columns of the tile are free when it calls.
template <typename T, int ROW>
__device__ __forceinline__ void write_columns(const float (&x)[8][4], char* tile, uint32_t tile_u, T* out, long long st,
                                              int len, int cols, int lane) {
  if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int jj = 0; jj < 4; ++jj)
      stsm4t(tile_u + (jj * 16 + at_row(lane)) * ROW + at_col(lane) * 2, pack_bf16(x[2 * jj][0], x[2 * jj][1]),
             pack_bf16(x[2 * jj][2], x[2 * jj][3]), pack_bf16(x[2 * jj + 1][0], x[2 * jj + 1][1]),
             pack_bf16(x[2 * jj + 1][2], x[2 * jj + 1][3]));
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        *reinterpret_cast<float*>(tile + (8 * j + 2 * (lane & 3) + (e & 1)) * ROW + ((lane >> 2) + (e >> 1) * 8) * 4) =
            x[j][e];
  }
  __syncwarp();
  constexpr int per = 16 / sizeof(T), pieces = 16 / per;
#pragma unroll
  for (int i = 0; i < kL * pieces / 32; ++i) {
    const int row = (i * 32 + lane) / pieces, col = (i * 32 + lane) % pieces * per;
    if (row < len && col < cols)
      *reinterpret_cast<uint4*>(out + row * st + col) = *reinterpret_cast<const uint4*>(tile + row * ROW + col * sizeof(T));
  }
}

// A block takes 16 W value columns of one value head of one sequence.
template <typename T, int KP, int W, bool GRAD>
__global__ void __launch_bounds__(32 * W) gdr_walk_kernel(const GdrArgs a, const char* keys, const char* records,
                                                          const Kept kept) {
  using L = WalkStage<T, KP, W, GRAD>;
  constexpr int NP = L::NP;
  constexpr bool FINE = L::P2;  // the output in fp32 accuracy: two parts of S, U and P under it
  extern __shared__ __align__(128) char smem[];
  const int n = blockIdx.z, h = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tile = blockIdx.x * W + warp, tiles = (a.V + 15) / 16, col0 = blockIdx.x * 16 * W;
  const int v0 = tile * 16, cols = min(16, a.V - v0);  // this warp's columns; <= 0 behind the last one
  const Seq s = sequence(a, n);
  const int chunks = (int)((s.len + kL - 1) / kL);
  const size_t state = ((size_t)n * a.H + h) * a.K * a.V;
  const int ra = lane >> 2, ca = 2 * (lane & 3);  // row and first column of this lane in an accumulator

  float S[KP / 8][4];
#pragma unroll
  for (int j = 0; j < KP / 8; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int col = ra + (e >> 1) * 8, key = 8 * j + ca + (e & 1);
      S[j][e] = a.S0 && col < cols && key < a.K ? a.S0[state + (size_t)key * a.V + v0 + col] : 0.f;
    }

  auto keep_state = [&](long long at, const Scale& sc) {  // at: the state's number
    if constexpr (GRAD) {
      if (tile >= tiles) return;
      const size_t base = ((size_t)at * a.H + h) * tiles + tile;
      if (lane == 0) kept.S_inv[base] = sc.inv;
#pragma unroll
      for (int kk = 0; kk < KP / 16; ++kk) {
        uint32_t hi[4], lo[4];
        split_a(S[2 * kk], S[2 * kk + 1], sc.mul, hi, lo);
        keep(kept.S + base * 2 * (KP / 16) * 32, kk, lane, hi);
        keep(kept.S + (base * 2 + 1) * (KP / 16) * 32, kk, lane, lo);
      }
    }
  };

  const uint32_t smem_base = smem_u32(smem);
  if (chunks > 0) fetch_chunk<T, KP, W, GRAD>(a, s, s.slot, h, 0, col0, keys, records, smem_base);
  for (int c = 0; c < chunks; ++c) {
    const long long rec = s.slot + c;
    char* st = smem + (L::stages == 2 ? (c & 1) * L::bytes : 0);
    const uint32_t su = smem_u32(st);
    cp_wait_all();
    __syncthreads();  // the chunk has come, and nobody reads the one before any more
    if (L::stages == 2 && c + 1 < chunks)
      fetch_chunk<T, KP, W, GRAD>(a, s, rec + 1, h, c + 1, col0, keys, records, smem_base + ((c + 1) & 1) * L::bytes);
    const float* fac = reinterpret_cast<const float*>(st + L::factors);

    // X = (K S)^T and (Q S)^T
    const Scale ss = scale_of(tile_max<KP / 8>(S));
    keep_state(rec + n, ss);
    float x[8][4], o[8][4];
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) x[j][e] = o[j][e] = 0.f;
#pragma unroll
    for (int kk = 0; kk < KP / 16; ++kk) {
      uint32_t hi[4], lo[4];
      split_a(S[2 * kk], S[2 * kk + 1], ss.mul, hi, lo);
      rows_step<KP, NP, true>(x, hi, lo, su, kk, lane);
      rows_step<KP, NP, FINE>(o, hi, lo, su + L::q, kk, lane);
    }
    // Z, then Z' = Z + R (beta Z)
    float z[8][4];
    char* vt = st + L::v + warp * 16 * (int)sizeof(T);
    const uint32_t vu = su + L::v + warp * 16 * (int)sizeof(T);
    read_columns<T, L::row>(z, vt, vu, lane);
    float zb[8][4];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float2 gam = factor(fac + kGam * kL, j, lane), ki = factor(fac + kKInv * kL, j, lane);
      const float2 be = factor(fac + kBeta * kL, j, lane), qi = factor(fac + kQInv * kL, j, lane);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float g = e & 1 ? gam.y : gam.x;
        z[j][e] = fmaf(-g, x[j][e] * ss.inv * (e & 1 ? ki.y : ki.x), z[j][e]);
        o[j][e] = g * (o[j][e] * ss.inv * (e & 1 ? qi.y : qi.x));
        zb[j][e] = (e & 1 ? be.y : be.x) * z[j][e];
        x[j][e] = 0.f;
      }
    }
    uint32_t hi[4][4], lo[4][4];
    const Scale sz = scale_of(tile_max<8>(zb));
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) split_a(zb[2 * kk], zb[2 * kk + 1], sz.mul, hi[kk], lo[kk]);
    triangle<false, 2, 2>(x, hi, lo, su + L::record, lane);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float2 ri = factor(fac + kRInv * kL, j, lane), be = factor(fac + kBeta * kL, j, lane);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        z[j][e] = fmaf(x[j][e] * sz.inv, e & 1 ? ri.y : ri.x, z[j][e]);
        zb[j][e] = (e & 1 ? be.y : be.x) * z[j][e];  // U
        x[j][e] = 0.f;
      }
    }
    if constexpr (GRAD) {
      if (tile < tiles) {
        float4* at = kept.Z + (((size_t)rec * a.H + h) * tiles + tile) * 8 * 32 + lane;
#pragma unroll
        for (int j = 0; j < 8; ++j) at[j * 32] = make_float4(z[j][0], z[j][1], z[j][2], z[j][3]);
      }
    }
    // O = gam (Q S) + P U
    const Scale su_ = scale_of(tile_max<8>(zb));
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) split_a(zb[2 * kk], zb[2 * kk + 1], su_.mul, hi[kk], lo[kk]);
    if constexpr (GRAD) {
      if (tile < tiles) {
        const size_t base = ((size_t)rec * a.H + h) * tiles + tile;
        if (lane == 0) kept.U_inv[base] = su_.inv;
        constexpr int NK = kept_parts<T>();
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          keep(kept.U + base * NK * 128, kk, lane, hi[kk]);
          if (NK == 2) keep(kept.U + (base * NK + 1) * 128, kk, lane, lo[kk]);
        }
      }
    }
    triangle<false, FINE ? 2 : 1, FINE ? 2 : 1>(x, hi, lo, su + L::record + 2 * kTile, lane);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float2 pi = factor(fac + kPInv * kL, j, lane);
#pragma unroll
      for (int e = 0; e < 4; ++e) o[j][e] = fmaf(x[j][e] * su_.inv, e & 1 ? pi.y : pi.x, o[j][e]);
    }
    const int len = (int)min((long long)kL, s.len - (long long)c * kL);
    if constexpr (GRAD) {
      float d[8][4], dot[16];
      read_columns<T, L::row>(d, st + L::dout + warp * 16 * (int)sizeof(T), su + L::dout + warp * 16 * (int)sizeof(T), lane);
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e) dot[2 * j + e] = d[j][e] * o[j][e] + d[j][e + 2] * o[j][e + 2];
      const float2 sum = column_sum(dot, lane);
      if (tile < tiles)
        *reinterpret_cast<float2*>(kept.dots + (((size_t)rec * a.H + h) * tiles + tile) * kL + 8 * ra + ca) = sum;
    } else {
      T* out = (T*)a.o + s.b * a.so.b + h * a.so.h + (s.lo + (long long)c * kL) * a.so.t + v0;
      write_columns<T, L::row>(o, vt, vu, out, a.so.t, len, cols, lane);
    }
    // S <- gam_63 S + (w K)^T U
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float2 w = factor(fac + kW * kL, j, lane), ki = factor(fac + kKInv * kL, j, lane);
#pragma unroll
      for (int e = 0; e < 4; ++e) zb[j][e] *= e & 1 ? w.y * ki.y : w.x * ki.x;
    }
    const Scale sw = scale_of(tile_max<8>(zb));
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) split_a(zb[2 * kk], zb[2 * kk + 1], sw.mul, hi[kk], lo[kk]);
    state_add<KP, NP>(S, fac[kGam * kL + kL - 1], hi, lo, sw.inv, su, lane);
    if (L::stages == 1 && c + 1 < chunks) {
      __syncthreads();
      fetch_chunk<T, KP, W, GRAD>(a, s, rec + 1, h, c + 1, col0, keys, records, smem_base);
    }
  }
  if constexpr (GRAD) keep_state(s.slot + chunks + n, scale_of(tile_max<KP / 8>(S)));
  if (a.S_out) {
#pragma unroll
    for (int j = 0; j < KP / 8; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int col = ra + (e >> 1) * 8, key = 8 * j + ca + (e & 1);
        if (col < cols && key < a.K) a.S_out[state + (size_t)key * a.V + v0 + col] = S[j][e];
      }
  }
}

template <typename T, int KP, int W, bool GRAD>
cudaError_t launch_walk_w(const GdrArgs& a, const char* keys, const char* records, const Kept& kept, cudaStream_t stream) {
  using L = WalkStage<T, KP, W, GRAD>;
  const auto kernel = gdr_walk_kernel<T, KP, W, GRAD>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, L::stages * L::bytes);
  if (e != cudaSuccess) return e;
  kernel<<<dim3((a.V + 16 * W - 1) / (16 * W), a.H, a.N), 32 * W, L::stages * L::bytes, stream>>>(a, keys, records, kept);
  return cudaGetLastError();
}

// Warps (tiles of 16 columns) a block: more blocks while there are fewer than the SMs.
inline int walk_warps(const GdrArgs& a) {
  const long long heads = (long long)a.N * a.H;
  if (a.V > 64 && heads * ((a.V + 127) / 128) >= 120) return 8;
  if (a.V > 32 && heads * ((a.V + 63) / 64) >= 100) return 4;
  return 2;
}

template <typename T, int KP, bool GRAD>
cudaError_t launch_walk(const GdrArgs& a, const char* keys, const char* records, const Kept& kept, cudaStream_t stream) {
  switch (walk_warps(a)) {
    case 8: return launch_walk_w<T, KP, 8, GRAD>(a, keys, records, kept, stream);
    case 4: return launch_walk_w<T, KP, 4, GRAD>(a, keys, records, kept, stream);
    default: return launch_walk_w<T, KP, 2, GRAD>(a, keys, records, kept, stream);
  }
}

}  // namespace gdr
}  // namespace mlstm
