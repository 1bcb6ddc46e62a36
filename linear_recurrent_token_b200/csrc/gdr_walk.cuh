// The pass over a sequence's chunks: forward for outputs and states, or again for the gradients, which
// keep what they need of it.
#pragma once
#include <algorithm>

#include "gdr_tile.cuh"

namespace mlstm {
namespace gdr {

// What the gradients keep of the two passes, by record of a chunk and value head (states: one more a
// sequence, the final one) and by tile of 16 value columns.  Operands are fp16 tiles [16 values][tokens or
// keys] with the pieces of a row permuted as in the other records, a tile's parts one behind the other;
// each quarter of the tokens or keys has its scale.  NK: parts of an operand that only products rounded to
// the output's type read, one (11 bits) for bf16, two for fp32.  With one part dq and dk of bf16 inputs lie
// 0.00168 and 0.00169 (relative, root of the mean square) from 64 bits, 0.00166 where only the result is
// rounded; two would double what is kept, and of 128 keys only one block of columns would fit an SM.
struct Kept {
  char* S;        // S at the chunk's start: [state][tile][2 parts][16][KP]
  float* S_inv;   // [state][tile][4]
  float* Z;       // Z': [record][tile][16][64]
  char* U;        // [record][tile][NK][16][64]
  float* U_inv;   // [record][tile][4]
  float* dots;    // dO . O, then dO . O - dV . V, over the tile's columns: [record][tile][64]
  // of the pass backward
  char* D;        // dS at the chunk's end: [record][tile][NK][16][KP]
  float* D_inv;   // [record][tile][4]
  char* dV;       // [record][tile][NK][16][64]
  float* dV_inv;  // [record][tile][4]
  char* dO;       // [record][tile][NK][16][64]
  float* dO_inv;  // [record][tile][4]
  float* dbeta;   // dY . Z' over the tile's columns: [record][tile][64]
  float* ends;    // <dS, S> at the chunk's end over the tile's columns and a quarter of the keys: [record][tile][4]
};
template <typename T>
constexpr int kept_parts() { return sizeof(T) == 4 ? 2 : 1; }

template <int KP>
cudaError_t launch_tc_walk(const GdrArgs& a, const char* keys, const char* records, unsigned int* err, cudaStream_t stream);
template <typename T, int KP, bool P2>
cudaError_t launch_prep(const GdrArgs& a, char* keys, char* records, cudaStream_t stream);

// Blocks on an SM: two, where their shared memory lets them.
template <typename T, int KP, int TN>
constexpr int kWalkBlocks = sizeof(T) == 2 && KP == 64 && TN <= 2 ? 2 : 1;

// Shared memory of a pass with TN tiles a block: one or two chunks' k, q, columns of v (and dO) and factors,
// one or two chunks' R and P, and the tiles' operands in exchange.
template <typename T, int KP, int TN, bool GRAD>
struct Stage {
  static constexpr int NP = sizeof(T) == 4 ? 2 : 1;
  static constexpr bool P2 = sizeof(T) == 4 || GRAD;
  static constexpr int row = 16 * TN * (int)sizeof(T) + 16;  // odd multiples of 16 bytes: no bank conflicts
  static constexpr int q = keys_bytes(KP, NP) / 2;
  static constexpr int v = keys_bytes(KP, NP);
  static constexpr int dout = v + kL * row;
  static constexpr int factors = dout + (GRAD ? kL * row : 0);
  static constexpr int chunk = factors + kFactorBytes;
  static constexpr int matrices = record_bytes(P2) - kFactorBytes;
  // operands in exchange, 512 bytes a k step and part
  static constexpr int fs = 0;                                 // the state, two parts
  static constexpr int fu = fs + KP / 16 * 1024;               // U (backward: dO), NU parts
  static constexpr int nu = P2 ? 2 : 1;
  static constexpr int fw = fu + 4 * nu * 512;                 // w U (backward: gam dV), two parts
  static constexpr int fz = fw + 4096;                         // beta Z (backward: gam dO), two parts
  static constexpr int inv = fz + 4096;                        // scales: [5][4]
  static constexpr int tile = inv + 5 * kQuarter * 4 + 48;     // a multiple of 128
  static constexpr int least = chunk + matrices + TN * tile;
  static constexpr int chunks = least + chunk <= 227 * 1024 ? 2 : 1;
  static constexpr bool ahead = least + chunk + matrices <= 227 * 1024 / kWalkBlocks<T, KP, TN> - 1024;  // R and P twice
  static constexpr int bytes = least + (chunks - 1) * chunk + (ahead ? matrices : 0);
  // where chunk c and its R and P lie
  __host__ __device__ static constexpr int at(int c) { return chunks == 2 ? (c & 1) * chunk : 0; }
  __host__ __device__ static constexpr int mats(int c) { return chunks * chunk + (ahead ? (c & 1) * matrices : 0); }
  static constexpr int tiles = chunks * chunk + (ahead ? 2 : 1) * matrices;
  static_assert(tile % 128 == 0, "operands keep their alignment");
  static_assert(bytes <= 227 * 1024, "a block's shared memory");
};

// Warps that only copy.  With one or two tiles a block a scheduler has one or two warps that compute, and
// copies of theirs (some 30 instructions a thread and chunk) would lengthen the chain; with four, registers
// leave no room for more warps and the others hide them.  16 heads of 128 x 128, 8192 tokens, TN = 1: 283 us
// without them, 266 with, 219 with R and P a chunk ahead as well.
template <int TN>
constexpr int kCopyWarps = TN == 1 ? 4 : TN == 2 ? 2 : 0;
template <int TN>
constexpr int kWalkThreads = 32 * (kQuarter * TN + kCopyWarps<TN>);
template <int TN>
constexpr int kCopyThreads = kCopyWarps<TN> ? 32 * kCopyWarps<TN> : kWalkThreads<TN>;
template <int TN>
__device__ __forceinline__ int copy_thread() { return kCopyWarps<TN> ? threadIdx.x - 32 * kQuarter * TN : threadIdx.x; }

// Copies the k, q, v, dO and factors of one chunk: every copying thread a share, 16 bytes at a time.
template <typename T, int KP, int TN, bool GRAD>
__device__ __forceinline__ void fetch_chunk(const GdrArgs& a, const Seq& s, long long rec, int h, int c, int col0,
                                            const char* keys, const char* records, uint32_t to) {
  using L = Stage<T, KP, TN, GRAD>;
  const int tid = copy_thread<TN>();
  constexpr int threads = kCopyThreads<TN>;
  const char* k = keys + (rec * a.HK + h / (a.H / a.HK)) * keys_bytes(KP, L::NP);
  for (int i = tid; i < keys_bytes(KP, L::NP) / 16; i += threads) cp_async16(to + i * 16, k + i * 16, true);
  const char* f = records + (rec * a.H + h) * record_bytes(L::P2) + L::matrices;
  for (int i = tid; i < kFactorBytes / 16; i += threads) cp_async16(to + L::factors + i * 16, f + i * 16, true);
  constexpr int per = 16 / sizeof(T), pieces = 16 * TN / per;  // of a row
  const long long t0 = (long long)c * kL;
  const T* v = (const T*)a.v + s.b * a.sv.b + h * a.sv.h;
  const T* d = GRAD ? (const T*)a.dout + s.b * a.so.b + h * a.so.h : nullptr;
  for (int i = tid; i < kL * pieces; i += threads) {
    const int row = i / pieces, col = i % pieces * per;
    const bool in = t0 + row < s.len && col0 + col < a.V;
    const long long t = in ? s.lo + t0 + row : 0;
    cp_async16(to + L::v + row * L::row + col * (int)sizeof(T), in ? v + t * a.sv.t + col0 + col : v, in);
    if (GRAD) cp_async16(to + L::dout + row * L::row + col * (int)sizeof(T), in ? d + t * a.so.t + col0 + col : d, in);
  }
}
// and its R and P
template <bool P2, int TN>
__device__ __forceinline__ void fetch_matrices(const GdrArgs& a, long long rec, int h, const char* records, uint32_t to) {
  const char* r = records + (rec * a.H + h) * record_bytes(P2);
  for (int i = copy_thread<TN>(); i < (record_bytes(P2) - kFactorBytes) / 16; i += kCopyThreads<TN>)
    cp_async16(to + i * 16, r + i * 16, true);
}
// A chunk with all that is copied ahead of it.
template <typename T, int KP, int TN, bool GRAD>
__device__ __forceinline__ void fetch_all(const GdrArgs& a, const Seq& s, int c, int h, int col0, const char* keys,
                                          const char* records, uint32_t smem) {
  using L = Stage<T, KP, TN, GRAD>;
  fetch_chunk<T, KP, TN, GRAD>(a, s, s.slot + c, h, c, col0, keys, records, smem + L::at(c));
  if (L::ahead) fetch_matrices<L::P2, TN>(a, s.slot + c, h, records, smem + L::mats(c));
  cp_commit();
}
// The copying warps' part of a pass, forward or from the last chunk on: the same barriers as the others'.
template <typename T, int KP, int TN, bool GRAD, bool BACK>
__device__ __forceinline__ void copy_ahead(const GdrArgs& a, const Seq& s, int chunks, int h, int col0, const char* keys,
                                           const char* records, uint32_t smem) {
  using L = Stage<T, KP, TN, GRAD>;
  auto fetch = [&](int i) {
    if (i < chunks) fetch_all<T, KP, TN, GRAD>(a, s, BACK ? chunks - 1 - i : i, h, col0, keys, records, smem);
  };
  fetch(0);
  for (int i = 0; i < chunks; ++i) {
    const int c = BACK ? chunks - 1 - i : i;
    cp_wait<0>();
    __syncthreads();
    if (!L::ahead) {  // (the next chunk's copies would hold these up)
      fetch_matrices<L::P2, TN>(a, s.slot + c, h, records, smem + L::mats(c));
      cp_commit();
      cp_wait<0>();
      __syncthreads();
    }
    if (L::chunks == 1 && i + 1 < chunks) __syncthreads();
    fetch(i + 1);
  }
}

// A quarter's 16 columns x 16 tokens of a tile [64][16 TN] in shared memory, as accumulator tiles.
template <typename T, int ROW>
__device__ __forceinline__ void read_columns(float (&x)[2][4], const char* at, int lane) {
  if constexpr (sizeof(T) == 2) {
    uint32_t r[4];
    ldsm4t(r, smem_u32(at) + at_row(lane) * ROW + at_col(lane) * 2);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = unpack_bf16(r[i]);
      x[i >> 1][(i & 1) * 2] = f.x;
      x[i >> 1][(i & 1) * 2 + 1] = f.y;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        x[j][e] = *reinterpret_cast<const float*>(at + (8 * j + 2 * (lane & 3) + (e & 1)) * ROW +
                                                  ((lane >> 2) + (e >> 1) * 8) * 4);
  }
}
// The inverse, in the place of what the warp alone has read, and from there to memory: out points at the
// quarter's first token, of which len are inside, and at the tile's first column, of which cols are.
template <typename T, int ROW>
__device__ __forceinline__ void write_columns(const float (&x)[2][4], char* at, T* out, long long st, int len, int cols,
                                              int lane) {
  __syncwarp();
  if constexpr (sizeof(T) == 2) {
    stsm4t(smem_u32(at) + at_row(lane) * ROW + at_col(lane) * 2, pack_bf16(x[0][0], x[0][1]), pack_bf16(x[0][2], x[0][3]),
           pack_bf16(x[1][0], x[1][1]), pack_bf16(x[1][2], x[1][3]));
  } else {
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        *reinterpret_cast<float*>(at + (8 * j + 2 * (lane & 3) + (e & 1)) * ROW + ((lane >> 2) + (e >> 1) * 8) * 4) = x[j][e];
  }
  __syncwarp();
  constexpr int per = 16 / sizeof(T), pieces = 16 / per;
#pragma unroll
  for (int i = 0; i < 16 * pieces / 32; ++i) {
    const int row = (i * 32 + lane) / pieces, col = (i * 32 + lane) % pieces * per;
    if (row < len && col < cols)
      *reinterpret_cast<uint4*>(out + row * st + col) = *reinterpret_cast<const uint4*>(at + row * ROW + col * sizeof(T));
  }
}

// Two accumulator tiles' operand (rows = values, 16 columns from c0) in a kept tile with COLS columns.
template <int COLS>
__device__ __forceinline__ void keep16(char* tile, int c0, const uint4& f, int lane) {
  const int row = lane >> 2, col = c0 + 2 * (lane & 3);
  char* at = tile + piece_at<COLS, 16>(row, col) + (col & 7) * 2;  // rows r and r + 8 share their permutation
  char* bt = tile + piece_at<COLS, 16>(row, col + 8) + (col & 7) * 2;
  *reinterpret_cast<uint32_t*>(at) = f.x;
  *reinterpret_cast<uint32_t*>(at + 8 * 128) = f.y;
  *reinterpret_cast<uint32_t*>(bt) = f.z;
  *reinterpret_cast<uint32_t*>(bt + 8 * 128) = f.w;
}
template <int COLS>
__device__ __forceinline__ uint4 kept16(const char* tile, int c0, int lane) {
  const int row = lane >> 2, col = c0 + 2 * (lane & 3);
  const char* at = tile + piece_at<COLS, 16>(row, col) + (col & 7) * 2;
  const char* bt = tile + piece_at<COLS, 16>(row, col + 8) + (col & 7) * 2;
  return make_uint4(*reinterpret_cast<const uint32_t*>(at), *reinterpret_cast<const uint32_t*>(at + 8 * 128),
                    *reinterpret_cast<const uint32_t*>(bt), *reinterpret_cast<const uint32_t*>(bt + 8 * 128));
}
// The quarter w of a token operand: its parts and its scale.
template <int NK>
__device__ __forceinline__ void keep_tokens(char* tiles, float* inv, size_t tile, const float (&x)[2][4], const Scale& sc, int w,
                                            int lane) {
  uint4 hi, lo;
  split_a(x[0], x[1], sc.mul, hi, lo);
  char* at = tiles + tile * NK * 16 * kL * 2;
  keep16<kL>(at, w * 16, hi, lane);
  if (NK == 2) keep16<kL>(at + 16 * kL * 2, w * 16, lo, lane);
  if (lane == 0) inv[tile * kQuarter + w] = sc.inv;
}

// A quarter of an operand into exchange: its k steps (STEPS of them) in two parts, or one, with its scale.
template <int STEPS, int PARTS>
__device__ __forceinline__ void give(const float (&x)[2 * STEPS][4], const Scale& sc, char* to, float* inv, int w, int lane) {
#pragma unroll
  for (int i = 0; i < STEPS; ++i) {
    uint4 hi, lo;
    split_a(x[2 * i], x[2 * i + 1], sc.mul, hi, lo);
    uint4* at = reinterpret_cast<uint4*>(to) + (w * STEPS + i) * PARTS * 32 + lane;
    at[0] = hi;
    if (PARTS == 2) at[32] = lo;
  }
  if (lane == 0) inv[w] = sc.inv;
}
template <int PARTS>
__device__ __forceinline__ void take(const char* from, int k, int lane, uint4& hi, uint4& lo) {
  const uint4* at = reinterpret_cast<const uint4*>(from) + k * PARTS * 32 + lane;
  hi = at[0];
  lo = PARTS == 2 ? at[32] : make_uint4(0u, 0u, 0u, 0u);
}

// x [16 columns x the quarter's 16 tokens] = F B, F the exchanged state [16 x KP], B = the tokens' rows of the
// [64][KP] tile k; where TWO, y = F times those of q, which shares F's fragments (one part of F unless LO2).
template <int KP, int NP, bool TWO, bool LO2>
__device__ __forceinline__ void by_keys(float (&x)[2][4], float (&y)[2][4], const char* f, const float* inv, uint32_t k,
                                        uint32_t q, int w, int lane) {
  constexpr int KS = KP / 16 / kQuarter;
  zero(x);
  if constexpr (TWO) zero(y);
#pragma unroll
  for (int b = 0; b < kQuarter; ++b) {
    float tx[2][4], ty[2][4];
#pragma unroll
    for (int i = 0; i < KS; ++i) {
      uint4 hi, lo;
      take<2>(f, b * KS + i, lane, hi, lo);
      const int at = piece_at<KP>(w * 16 + b_row(lane), (b * KS + i) * 16 + b_col(lane));
      auto from_k = [&](uint32_t (&r)[4], int, int plane) { ldsm4(r, k + at + plane * kL * KP * 2); };
      auto from_q = [&](uint32_t (&r)[4], int, int plane) { ldsm4(r, q + at + plane * kL * KP * 2); };
      if (i == 0) {
        step<true, 2, 2, NP>(tx, hi, lo, from_k);
        if constexpr (TWO) step<true, 2, LO2 ? 2 : 1, NP>(ty, hi, lo, from_q);
      } else {
        step<false, 2, 2, NP>(tx, hi, lo, from_k);
        if constexpr (TWO) step<false, 2, LO2 ? 2 : 1, NP>(ty, hi, lo, from_q);
      }
    }
    add_scaled(x, tx, inv[b]);
    if constexpr (TWO) add_scaled(y, ty, inv[b]);
  }
}

// sum [16 columns x the quarter's tokens] = F X^T for a lower triangular [64][64] X, F over its columns up to
// the quarter; TRANS: F X, over its rows from the quarter on.
template <bool TRANS, int NA, int NX>
__device__ __forceinline__ void by_tokens(float (&x)[2][4], const char* f, const float* inv, uint32_t tile, int w, int lane) {
  zero(x);
#pragma unroll
  for (int b = 0; b < kQuarter; ++b) {
    if (TRANS ? b < w : b > w) continue;
    float t[2][4];
    uint4 hi, lo;
    take<NA>(f, b, lane, hi, lo);
    const int at = TRANS ? piece_at<kL>(b * 16 + bt_row(lane), w * 16 + bt_col(lane))
                         : piece_at<kL>(w * 16 + b_row(lane), b * 16 + b_col(lane));
    step<true, 2, NA, NX>(t, hi, lo, [&](uint32_t (&r)[4], int, int plane) {
      if constexpr (TRANS)
        ldsm4t(r, tile + at + plane * kTile);
      else
        ldsm4(r, tile + at + plane * kTile);
    });
    add_scaled(x, t, inv[b]);
  }
}

// S [16 columns x the quarter's keys] = keep S + F B, F over the 64 tokens, B a [64][KP] tile.
template <int KP, int NP>
__device__ __forceinline__ void to_state(float (&S)[KP / 32][4], float keep, const char* f, const float* inv, uint32_t tile,
                                         int w, int lane) {
#pragma unroll
  for (int j = 0; j < KP / 32; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) S[j][e] *= keep;
#pragma unroll
  for (int b = 0; b < kQuarter; ++b) {
    float d[KP / 32][4];
    uint4 hi, lo;
    take<2>(f, b, lane, hi, lo);
    step<true, KP / 32, 2, NP>(d, hi, lo, [&](uint32_t (&r)[4], int j, int plane) {
      ldsm4t(r, tile + piece_at<KP>(b * 16 + bt_row(lane), w * (KP / 4) + j * 8 + bt_col(lane)) + plane * kL * KP * 2);
    });
    add_scaled(S, d, inv[b]);
  }
}

// A block takes 16 TN value columns of one value head of one sequence.  What bounds it is a chunk's chain (three
// exchanges and five products, one after the other): 16 heads of 128 x 128, 8192 bf16 tokens, TN = 1: 220 us,
// 1.7 us or 3250 cycles a chunk, of which K S and Q S 1000, R and its operands 850, P U 600, the state 450, its
// parts 230.  64 heads, 2048 tokens, TN = 4 for the gradients: 217 us, issue slots 42 % taken, tensor pipes 33 %.
template <typename T, int KP, int TN, bool GRAD>
__global__ void __launch_bounds__(kWalkThreads<TN>, kWalkBlocks<T, KP, TN>) gdr_walk_kernel(const GdrArgs a, const char* keys,
                                                                      const char* records, const Kept kept) {
  using L = Stage<T, KP, TN, GRAD>;
  constexpr int NP = L::NP, NK = kept_parts<T>(), KS = KP / 64;
  // The output in fp32 accuracy: two parts of S, U and P under it.  A bf16 output takes one, 11 bits under the 8 that
  // it keeps: 0.00168 from 64 bits (relative, root of the mean square) instead of 0.00166, for 220 us instead of 244
  // (16 heads of 128 x 128, 8192 tokens; 32 heads, 2048 tokens 85/94; 64 of 64 x 64 73/88).
  constexpr bool FINE = L::P2;
  extern __shared__ __align__(128) char smem[];
  const int n = blockIdx.z, h = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // the quarters' shares of the triangular products differ: over the tiles, each scheduler gets all of them
  const int local = warp / kQuarter, w = (warp + local) % kQuarter, tile = blockIdx.x * TN + local, tiles = (a.V + 15) / 16;
  const int col0 = blockIdx.x * 16 * TN, v0 = tile * 16, cols = min(16, a.V - v0);  // cols <= 0 behind the last
  const bool live = tile < tiles;
  const Seq s = sequence(a, n);
  const int chunks = (int)((s.len + kL - 1) / kL);
  const size_t state = ((size_t)n * a.H + h) * a.K * a.V;
  const int ra = lane >> 2, ca = 2 * (lane & 3);  // row and first column of this lane in an accumulator
  char* ex = smem + L::tiles + local * L::tile;
  float* inv = reinterpret_cast<float*>(ex + L::inv);

  constexpr bool copies = kCopyWarps<TN> == 0;  // the warps that compute copy as well
  if (!copies && warp >= kQuarter * TN) {
    copy_ahead<T, KP, TN, GRAD, false>(a, s, chunks, h, col0, keys, records, smem_u32(smem));
    return;
  }

  float S[2 * KS][4];  // keys w KP / 4 ..
#pragma unroll
  for (int j = 0; j < 2 * KS; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int col = ra + (e >> 1) * 8, key = w * (KP / 4) + 8 * j + ca + (e & 1);
      S[j][e] = a.S0 && col < cols && key < a.K ? a.S0[state + (size_t)key * a.V + v0 + col] : 0.f;
    }
  auto keep_state = [&](long long number, const Scale& sc) {
    if constexpr (GRAD) {
      if (!live) return;
      const size_t base = ((size_t)number * a.H + h) * tiles + tile;
      if (lane == 0) kept.S_inv[base * kQuarter + w] = sc.inv;
#pragma unroll
      for (int i = 0; i < KS; ++i) {
        uint4 hi, lo;
        split_a(S[2 * i], S[2 * i + 1], sc.mul, hi, lo);
        char* at = kept.S + base * 2 * 16 * KP * 2;
        keep16<KP>(at, (w * KS + i) * 16, hi, lane);
        keep16<KP>(at + 16 * KP * 2, (w * KS + i) * 16, lo, lane);
      }
    }
  };

  if (copies && chunks > 0) fetch_all<T, KP, TN, GRAD>(a, s, 0, h, col0, keys, records, smem_u32(smem));
  for (int c = 0; c < chunks; ++c) {
    const long long rec = s.slot + c;
    const size_t base = ((size_t)rec * a.H + h) * tiles + tile;
    char *st = smem + L::at(c), *mats = smem + L::mats(c);
    const float* fac = reinterpret_cast<const float*>(st + L::factors);
    {
      const Scale sc = tile_scale(S);
      give<KS, 2>(S, sc, ex + L::fs, inv, w, lane);
      keep_state(rec + n, sc);
    }
    if (copies) cp_wait<0>();
    __syncthreads();  // the chunk has come, the states are in exchange, and nobody is in the chunk before
    if (copies && !L::ahead) {
      fetch_matrices<L::P2, TN>(a, rec, h, records, smem_u32(mats));
      cp_commit();
    }
    if (copies && L::chunks == 2) {
      if (c + 1 < chunks)
        fetch_all<T, KP, TN, GRAD>(a, s, c + 1, h, col0, keys, records, smem_u32(smem));
      else
        cp_commit();
    }
    // Z = V - gam (K S), O = gam (Q S)
    float x[2][4], o[2][4], z[2][4], u[2][4];
    by_keys<KP, NP, true, FINE>(x, o, ex + L::fs, inv, smem_u32(st), smem_u32(st) + L::q, w, lane);
    char* vt = st + L::v + w * 16 * L::row + local * 16 * (int)sizeof(T);
    read_columns<T, L::row>(z, vt, lane);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float2 gk = factor(fac + kGK * kL, w * 16, j, lane), gq = factor(fac + kGQ * kL, w * 16, j, lane);
      const float2 be = factor(fac + kBeta * kL, w * 16, j, lane);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        z[j][e] = fmaf(e & 1 ? -gk.y : -gk.x, x[j][e], z[j][e]);
        o[j][e] *= e & 1 ? gq.y : gq.x;
        u[j][e] = (e & 1 ? be.y : be.x) * z[j][e];
      }
    }
    give<1, 2>(u, tile_scale(u), ex + L::fz, inv + kQuarter, w, lane);
    if (copies && !L::ahead) cp_wait<L::chunks == 2 ? 1 : 0>();
    if (L::ahead)
      tile_barrier(local);  // beta Z is in exchange
    else
      __syncthreads();  // and R and P have come
    // Z' = Z + R (beta Z), U = beta Z'
    by_tokens<false, 2, 2>(x, ex + L::fz, inv + kQuarter, smem_u32(mats), w, lane);
    float uw[2][4];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float2 ri = factor(fac + kRInv * kL, w * 16, j, lane), be = factor(fac + kBeta * kL, w * 16, j, lane);
      const float2 wk = factor(fac + kWK * kL, w * 16, j, lane);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        z[j][e] = fmaf(x[j][e], e & 1 ? ri.y : ri.x, z[j][e]);
        u[j][e] = (e & 1 ? be.y : be.x) * z[j][e];
        uw[j][e] = (e & 1 ? wk.y : wk.x) * u[j][e];
      }
    }
    {
      const Scale sc = tile_scale(u);
      give<1, L::nu>(u, sc, ex + L::fu, inv + 2 * kQuarter, w, lane);
      if constexpr (GRAD) {
        if (live) {
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int r = 0; r < 2; ++r)
              *reinterpret_cast<float2*>(kept.Z + (base * 16 + ra + 8 * r) * kL + w * 16 + 8 * j + ca) =
                  make_float2(z[j][2 * r], z[j][2 * r + 1]);
          keep_tokens<NK>(kept.U, kept.U_inv, base, u, sc, w, lane);
        }
      }
    }
    give<1, 2>(uw, tile_scale(uw), ex + L::fw, inv + 3 * kQuarter, w, lane);
    tile_barrier(local);  // U and w U are in exchange
    // O += P U
    by_tokens<false, L::nu, L::nu>(x, ex + L::fu, inv + 2 * kQuarter, smem_u32(mats) + 2 * kTile, w, lane);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float2 pi = factor(fac + kPInv * kL, w * 16, j, lane);
#pragma unroll
      for (int e = 0; e < 4; ++e) o[j][e] = fmaf(x[j][e], e & 1 ? pi.y : pi.x, o[j][e]);
    }
    if constexpr (GRAD) {
      float d[2][4], dot[4];
      read_columns<T, L::row>(d, st + L::dout + w * 16 * L::row + local * 16 * (int)sizeof(T), lane);
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e) dot[2 * j + e] = d[j][e] * o[j][e] + d[j][e + 2] * o[j][e + 2];
      const float2 sum = column_sum(dot, lane);
      if (live && (lane & 12) == 0)
        *reinterpret_cast<float2*>(kept.dots + base * kL + w * 16 + (lane >> 4) * 8 + ca) = sum;
    } else {
      const long long t0 = (long long)c * kL + w * 16;
      T* out = (T*)a.o + s.b * a.so.b + h * a.so.h + (s.lo + t0) * a.so.t + v0;
      write_columns<T, L::row>(o, vt, out, a.so.t, (int)max(0LL, min(16LL, s.len - t0)), cols, lane);
    }
    // S <- gam_63 S + (w K)^T U
    to_state<KP, NP>(S, fac[kGam * kL + kL - 1], ex + L::fw, inv + 3 * kQuarter, smem_u32(st), w, lane);
    if (L::chunks == 1 && c + 1 < chunks) {
      __syncthreads();
      if (copies) fetch_all<T, KP, TN, GRAD>(a, s, c + 1, h, col0, keys, records, smem_u32(smem));
    }
  }
  if constexpr (GRAD) keep_state(s.slot + chunks + n, tile_scale(S));
  if (a.S_out) {
#pragma unroll
    for (int j = 0; j < 2 * KS; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int col = ra + (e >> 1) * 8, key = w * (KP / 4) + 8 * j + ca + (e & 1);
        if (col < cols && key < a.K) a.S_out[state + (size_t)key * a.V + v0 + col] = S[j][e];
      }
  }
}

// What a pass over 32 chunks would take with blocks of 16 TN columns (TN = 0: the tcgen05 pass, 128 columns), in
// us.  A block's chunks are one chain, longer the more columns it has; blocks beyond the 148 SMs make a
// further round of it.  Where two blocks fit an SM they share each other's waits.  Sequences of one length go
// round in whole rounds; packed ones are uneven (their lengths are not known on the host): shorter ones
// make room, so count half of them, and no fewer than the longest one's chain.
// The chains are fitted to what was measured; us with the preparation, 2048 tokens, TN = 1 / 2 / 4 / tcgen05:
//   128 x 128, 16 heads 84/109/184/186, 32: 153/124/199/202, 64: 290/231/224/229, 80: 358/325/398/243,
//   128: 510/446/437/284, 256: 990/789/850/545;   128 x 256, 32 heads 262/204/199/206, 48: 384/300/371/224
//   64 x 64, 16 heads 73/95/145/173, 64: 127/143/179/207, 128: 237/212/221/253, 256: 458/410/428/483
//   64 x 128, 32 heads 106/110/156/175, 64: 193/167/178/197, 80: 273/253/311/208, 128: 373/319/341/240
//   64 x 128 packed, 13 uneven sequences of 6007 tokens, 4 heads 77/94/105/120, 8: 101/114/114/123, 16: 163/170/176/161
//   gradients 128 x 128, 16 heads 294/370/596, 64: 1100/848/797, 96: 1629/1249/1433, 128: 1965/1652/1560;
//   64 x 64, 64 heads 422/437/558, 128: 819/858/724
// fp32 inputs go by the same chains, which choose the faster of TN = 1 / 2 in all of these: 128 x 128, 16 heads
// 117/174, 32: 231/196, 64: 439/373, 128: 782/727; 64 x 64, 32 heads 103/136, 64: 189/169, 128: 367/326;
// gradients 128 x 128, 16 heads 382/547, 32: 741/650, 128: 2548/2481; 64 x 64, 32 heads 319/385, 64: 622/497
inline double walk_cost(const GdrArgs& a, int TN) {
  const bool narrow = a.dtype == 1 && a.K <= 64, two = narrow && (TN == 1 || TN == 2);
  const int columns = TN ? 16 * TN : 128;
  const long long blocks = (long long)a.N * a.H * ((a.V + columns - 1) / columns);
  const double chain = TN == 0 ? (narrow ? 170 : 172) : TN == 1 ? (narrow ? 66 : 68) : TN == 2 ? (narrow ? 98 : 95) : narrow ? 158 : 168;
  const double pair = two ? (TN == 1 ? 98 : 155) : 2 * chain;  // two blocks on one SM
  if (a.packed) return std::max(chain, 0.5 * blocks / 148 * pair / 2);
  const long long rounds = (blocks + 147) / 148;
  return rounds / 2 * pair + rounds % 2 * chain;
}

// The tiles a block, by that cost.  fp32 inputs: at most two; their second parts fill the registers.  With narrow
// bf16 keys two tiles and two blocks an SM always do better than four and one (above); for the gradients
// two do not leave an SM room for a second block: one or four.
template <typename T, int KP, bool GRAD>
constexpr bool kWalkOf(int TN) {
  const bool narrow = sizeof(T) == 2 && KP == 64;
  return TN == 1 || (TN == 2 && !(GRAD && narrow)) || (TN == 4 && sizeof(T) == 2 && (GRAD || !narrow));
}
template <typename T, int KP, bool GRAD>
int tiles_a_block(const GdrArgs& a) {
  int best = 1;
  for (int TN = 2; TN <= 4; TN *= 2)
    if (kWalkOf<T, KP, GRAD>(TN) && walk_cost(a, TN) < walk_cost(a, best)) best = TN;
  return best;
}

template <typename T, int KP, int TN, bool GRAD>
cudaError_t launch_walk_tn(const GdrArgs& a, const char* keys, const char* records, const Kept& kept, cudaStream_t stream) {
  constexpr int smem = Stage<T, KP, TN, GRAD>::bytes;
  const auto kernel = gdr_walk_kernel<T, KP, TN, GRAD>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const int tiles = (a.V + 15) / 16;
  kernel<<<dim3((tiles + TN - 1) / TN, a.H, a.N), kWalkThreads<TN>, smem, stream>>>(a, keys, records, kept);
  return cudaGetLastError();
}

template <typename T, int KP, bool GRAD>
cudaError_t launch_walk(const GdrArgs& a, const char* keys, const char* records, const Kept& kept, cudaStream_t stream) {
  const int tn = tiles_a_block<T, KP, GRAD>(a);
  if constexpr (kWalkOf<T, KP, GRAD>(4))
    if (tn == 4) return launch_walk_tn<T, KP, 4, GRAD>(a, keys, records, kept, stream);
  if constexpr (kWalkOf<T, KP, GRAD>(2))
    if (tn == 2) return launch_walk_tn<T, KP, 2, GRAD>(a, keys, records, kept, stream);
  return launch_walk_tn<T, KP, 1, GRAD>(a, keys, records, kept, stream);
}

}  // namespace gdr
}  // namespace mlstm
