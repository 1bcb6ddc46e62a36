// The forward pass over a sequence's chunks on tcgen05 (formulas, precision and records: gdr_tile.cuh; the
// same pass on warp-level products, for fp32 inputs and for few heads: gdr_walk.cuh).
//
// One block takes up to 128 value columns of one value head of one sequence.  Tensor memory has a lane for
// each value column: the state's, Z's and U's 16-bit parts are A operands there, k, q, R and P are B
// operands in shared memory, and every product has M = 128.  The state itself stays in the registers of
// eight warps (a lane is a column, two warps share its keys); each chunk's update is summed from zero in
// tensor memory and added in fp32.  A chunk is one chain:
//     S in parts -> K S, Q S -> Z -> R (beta Z) -> Z', U -> (w K)^T U -> S
// with the copies of the next chunk, Q S and P U beside it; the output is written while the update runs.  It is bound by that chain: the
// four products take about 1600 cycles of it for 128 keys and columns, the rest is what the eight warps do
// between them.
#include "gdr_walk.cuh"
#include "sm100.cuh"

namespace mlstm {
namespace gdr {
namespace {

using sm100::elect_one;
using sm100::mbar_arrive;
using sm100::mbar_arrive_expect_tx;
using sm100::mbar_init;
using sm100::mbar_test_wait;
using sm100::mbar_wait;
using sm100::mma_bf16_ts;
using sm100::mma_commit;
using sm100::named_bar;
using sm100::smem_desc_sw128;
using sm100::tc_fence_after;
using sm100::tc_fence_before;
using sm100::tmem_ld32;
using sm100::tmem_st16;
using sm100::tmem_wait_ld;
using sm100::tmem_wait_st;

constexpr int kTcThreads = 320;  // warps: producer, products, eight of the values
constexpr long long kTcWait = 4000000000LL;  // SM cycles (~2 s)
// tensor memory columns: the state's parts; Z's, then w U's; U's; K S, then R (beta Z), then P U; Q S; the update
constexpr uint32_t kTmS = 0, kTmZ = 128, kTmU = 192, kTmX = 256, kTmO = 320, kTmD = 384, kTmCols = 512;

// kind::f16 with fp16 A (K-major, in tensor memory) and B, fp32 sums, M = 128
__host__ __device__ constexpr uint32_t idesc_f16(int N, int b_mn) {
  return (1u << 4) | ((uint32_t)b_mn << 16) | ((uint32_t)(N >> 3) << 17) | ((128u >> 4) << 24);
}

struct TcBars {
  uint64_t full[2], empty[2], s_ready, x_full, z_ready, r_full, u_ready, o_full, d_full, drain;
};

template <int KP, bool GRAD>
struct TcStage {
  static constexpr int q = keys_bytes(KP, 1) / 2;
  static constexpr int record = keys_bytes(KP, 1);
  static constexpr int p = record + 2 * kTile;
  static constexpr int factors = record + record_bytes(GRAD) - kFactorBytes;
  static constexpr int v = record + record_bytes(GRAD);  // [64][128]
  static constexpr int dout = v + kL * 256;
  static constexpr int bytes = dout + (GRAD ? kL * 256 : 0);
  // behind two stages: maxima in exchange [4][2 halves][128]
  static constexpr int ex = 2 * bytes;
  static constexpr int bars = ex + 4 * 2 * 128 * 4;
  static constexpr int total = bars + (int)sizeof(TcBars) + 1024;  // and the slack of aligning the base to 1 KB
  static_assert(bytes % 1024 == 0 && total <= 227 * 1024, "a block's shared memory");
};

// (a wait that took longer than the limit counts as run out even when the phase completed meanwhile)
__device__ __noinline__ bool tc_wait_slow(uint64_t* bar, uint32_t parity, volatile int* failed, long long limit) {
  const long long t0 = clock64();
  const bool ok = !*failed && mbar_wait(bar, parity, limit) && clock64() - t0 <= limit;
  if (!ok) *failed = 1;
  return __all_sync(0xffffffffu, ok);
}

__device__ __forceinline__ float max16(float m) {  // over the 16 lanes of a tile
#pragma unroll
  for (int d = 8; d > 0; d /= 2) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
  return m;
}

// 32 values times f as two parts: 16 words each.
__device__ __forceinline__ void split32(const float* x, float f, float (&hi)[16], float (&lo)[16]) {
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    uint32_t h, l;
    split(x[2 * j] * f, x[2 * j + 1] * f, h, l);
    hi[j] = __uint_as_float(h), lo[j] = __uint_as_float(l);
  }
}
// 32 columns from c0 of row r of a kept tile
template <int COLS>
__device__ __forceinline__ void keep_row(char* tile, int r, int c0, const float (&w)[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    *reinterpret_cast<float4*>(tile + piece_at<COLS, 16>(r, c0 + 8 * i)) =
        make_float4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
}

template <int KP, bool GRAD>
__global__ void __launch_bounds__(kTcThreads, 1) gdr_tc_kernel(const GdrArgs a, const char* keys, const char* records,
                                                               const Kept kept, unsigned int* err, long long limit) {
  using L = TcStage<KP, GRAD>;
  constexpr int KH = KP / 2;
  extern __shared__ uint8_t raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  float* ex = reinterpret_cast<float*>(sm + L::ex);
  TcBars& bars = *reinterpret_cast<TcBars*>(sm + L::bars);
  __shared__ uint32_t tmem_base;
  __shared__ volatile int failed;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int n = blockIdx.z, h = blockIdx.y, v0 = blockIdx.x * 128;
  const Seq s = sequence(a, n);
  const int chunks = (int)((s.len + kL - 1) / kL);
  if (tid == 0) {
    for (int b = 0; b < 2; ++b) {
      mbar_init(&bars.full[b], 1);
      mbar_init(&bars.empty[b], 9);  // the last product's commit and eight value warps
    }
    mbar_init(&bars.s_ready, 8), mbar_init(&bars.z_ready, 8), mbar_init(&bars.u_ready, 8);
    mbar_init(&bars.x_full, 1), mbar_init(&bars.r_full, 1), mbar_init(&bars.d_full, 1), mbar_init(&bars.o_full, 1);
    mbar_init(&bars.drain, 1);
    failed = 0;
    sm100::fence_mbar_init();
  }
  if (warp == 0) sm100::tmem_alloc(&tmem_base, kTmCols);
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = tmem_base;
  const long long wlim = limit > 0 ? limit : kTcWait;  // (the drain below keeps the default)
  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    return __all_sync(0xffffffffu, mbar_test_wait(bar, parity)) || tc_wait_slow(bar, parity, &failed, wlim);
  };
  int issued = 0;

  if (warp == 0) {
    // ------------------------------------------------------------------------------------ producer
    const char* kq = keys + (s.slot * a.HK + h / (a.H / a.HK)) * keys_bytes(KP, 1);
    const char* rec = records + (s.slot * a.H + h) * record_bytes(GRAD);
    const int width = min(128, a.V - v0) * 2;  // bytes of a row of v: a multiple of 16
    const __nv_bfloat16* v = (const __nv_bfloat16*)a.v + s.b * a.sv.b + h * a.sv.h + s.lo * a.sv.t + v0;
    const __nv_bfloat16* d = GRAD ? (const __nv_bfloat16*)a.dout + s.b * a.so.b + h * a.so.h + s.lo * a.so.t + v0 : nullptr;
    for (int c = 0; c < chunks; ++c) {
      const int b = c & 1, rows = (int)min((long long)kL, s.len - (long long)c * kL);
      if (!wait(&bars.empty[b], ((c >> 1) & 1) ^ 1)) break;
      uint8_t* st = sm + b * L::bytes;
      if (lane == 0) {
        mbar_arrive_expect_tx(&bars.full[b], keys_bytes(KP, 1) + record_bytes(GRAD) + (GRAD ? 2 : 1) * rows * width);
        sm100::bulk_load(st, kq + (long long)c * a.HK * keys_bytes(KP, 1), keys_bytes(KP, 1), &bars.full[b]);
        sm100::bulk_load(st + L::record, rec + (long long)c * a.H * record_bytes(GRAD), record_bytes(GRAD), &bars.full[b]);
      }
      __syncwarp();
      for (int t = lane; t < rows; t += 32) {
        const long long at = (long long)c * kL + t;
        sm100::bulk_load(st + L::v + t * 256, v + at * a.sv.t, width, &bars.full[b]);
        if (GRAD) sm100::bulk_load(st + L::dout + t * 256, d + at * a.so.t, width, &bars.full[b]);
      }
      issued = c + 1;
      __syncwarp();
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------------------------ products
    bool ok = true;
    // D (+)= A B over the 16-column steps of the state, A's part at column `at`, B's keys at `bd`
    auto by_state = [&](uint32_t d, uint32_t at, uint64_t bd, uint32_t more) {
#pragma unroll 1
      for (int k = 0; k < KP / 16; ++k) {
        mma_bf16_ts(d, at + 8 * k, bd + (uint64_t)((k >> 2) * 512 + (k & 3) * 2), idesc_f16(64, 0), more);
        more = 1u;
      }
    };
    // the same over the tokens of a lower triangular B: the k step of tokens 16 kk .. reaches rows from 16 kk on
    auto by_tokens_of = [&](uint32_t d, uint32_t at, uint64_t bd, uint32_t more) {
#pragma unroll 1
      for (int kk = 0; kk < 4; ++kk) {
        mma_bf16_ts(d + 16 * kk, at + 8 * kk, bd + (uint64_t)(kk * 130), idesc_f16(64, 0) - ((uint32_t)(2 * kk) << 17), more);
        more = 1u;
      }
    };
    for (int c = 0; c < chunks; ++c) {
      const int b = c & 1;
      const uint32_t st = smem_u32(sm) + b * L::bytes;
      ok = wait(&bars.full[b], (c >> 1) & 1) && wait(&bars.s_ready, c & 1);
      if (!ok) break;
      tc_fence_after();
      if (elect_one()) {  // lo parts first: they are small, and so is what the sums cut off below them
        const uint64_t kd = smem_desc_sw128(st, 16, 1024), qd = smem_desc_sw128(st + L::q, 16, 1024);
        by_state(tm + kTmX, tm + kTmS + KP / 2, kd, 0u);
        by_state(tm + kTmX, tm + kTmS, kd, 1u);
        mma_commit(&bars.x_full);
        if (GRAD) by_state(tm + kTmO, tm + kTmS + KP / 2, qd, 0u);
        by_state(tm + kTmO, tm + kTmS, qd, GRAD ? 1u : 0u);
      }
      __syncwarp();
      ok = wait(&bars.z_ready, c & 1);
      if (!ok) break;
      tc_fence_after();
      if (elect_one()) {
        const uint64_t rd = smem_desc_sw128(st + L::record, 16, 1024);
        by_tokens_of(tm + kTmX, tm + kTmZ + 32, rd, 0u);
        by_tokens_of(tm + kTmX, tm + kTmZ, rd + (kTile >> 4), 1u);
        by_tokens_of(tm + kTmX, tm + kTmZ, rd, 1u);
        mma_commit(&bars.r_full);
      }
      __syncwarp();
      ok = wait(&bars.u_ready, c & 1);
      if (!ok) break;
      tc_fence_after();
      if (elect_one()) {
        const uint64_t kmn = smem_desc_sw128(st, 8192, 1024), pd = smem_desc_sw128(st + L::p, 16, 1024);
        if (GRAD) {
          by_tokens_of(tm + kTmX, tm + kTmU + 32, pd, 0u);
          by_tokens_of(tm + kTmX, tm + kTmU, pd + (kTile >> 4), 1u);
        }
        by_tokens_of(tm + kTmX, tm + kTmU, pd, GRAD ? 1u : 0u);
        mma_commit(&bars.o_full);
#pragma unroll 1
        for (int i = 0; i < 8; ++i)  // w U's second part, then its first
          mma_bf16_ts(tm + kTmD, tm + kTmZ + (i < 4 ? 32 : 0) + 8 * (i & 3), kmn + (uint64_t)((i & 3) * 128), idesc_f16(KP, 1),
                      i > 0 ? 1u : 0u);
        mma_commit(&bars.d_full);
        mma_commit(&bars.empty[b]);
      }
      __syncwarp();
    }
    if (elect_one()) mma_commit(&bars.drain);
    __syncwarp();
  } else {
    // -------------------------------------------------------------------------------------- values
    // A failed wait does not end the loop: the two warps of a column still meet at their barriers.
    const int q4 = warp & 3, half = warp >= 6, col = 32 * q4 + lane, v = v0 + col;
    const bool live = v < a.V;
    const uint32_t ln = tm + ((uint32_t)(32 * q4) << 16);
    const size_t state = ((size_t)n * a.H + h) * a.K * a.V + v;
    const int tiles = (a.V + 15) / 16, tile = v >> 4, tr = v & 15;
    const bool tile_live = tile < tiles;
    const int t0 = 32 * half;
    float S[KH];
#pragma unroll
    for (int j = 0; j < KH; ++j)
      S[j] = a.S0 && live && half * KH + j < a.K ? a.S0[state + (size_t)(half * KH + j) * a.V] : 0.f;
    // the larger of the two warps' maxima of a column (of a tile for the gradients, whose products sum over columns)
    auto agree = [&](int which, float m) {
      if (GRAD) m = max16(m);
      ex[(which * 2 + half) * 128 + col] = m;
      return m;
    };
    auto other = [&](int which) { return ex[(which * 2 + 1 - half) * 128 + col]; };
    auto keep_state = [&](long long number, const Scale& sc, int blk, const float (&hi)[16], const float (&lo)[16]) {
      if (!GRAD || !tile_live) return;
      const size_t base = ((size_t)number * a.H + h) * tiles + tile;
      char* at = kept.S + base * 2 * 16 * KP * 2;
      keep_row<KP>(at, tr, half * KH + 32 * blk, hi);
      keep_row<KP>(at + 16 * KP * 2, tr, half * KH + 32 * blk, lo);
      if (tr == 0 && half == 0 && blk == 0)
        *reinterpret_cast<float4*>(kept.S_inv + base * kQuarter) = make_float4(sc.inv, sc.inv, sc.inv, sc.inv);
    };
    auto state_scale = [&] {
      float m = 0.f;
#pragma unroll
      for (int j = 0; j < KH; ++j) m = fmaxf(m, fabsf(S[j]));
      m = agree(0, m);
      named_bar(1 + q4, 64);
      return scale_of(fmaxf(m, other(0)));
    };
    for (int c = 0; c < chunks; ++c) {
      const int b = c & 1, len = (int)min((long long)kL, s.len - (long long)c * kL);
      const long long rec = s.slot + c;
      const size_t base = ((size_t)rec * a.H + h) * tiles + tile;
      const uint8_t* st = sm + b * L::bytes;
      const float* fac = reinterpret_cast<const float*>(st + L::factors);
      const Scale ss = state_scale();  // (both warps have the update before: its columns may be written again)
#pragma unroll
      for (int blk = 0; blk < KH / 32; ++blk) {
        float hi[16], lo[16];
        split32(S + 32 * blk, ss.mul, hi, lo);
        tmem_st16(ln + kTmS + half * (KH / 2) + 16 * blk, hi);
        tmem_st16(ln + kTmS + KP / 2 + half * (KH / 2) + 16 * blk, lo);
        keep_state(rec + n, ss, blk, hi, lo);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.s_ready);

      // Z = V - gam (K S)
      wait(&bars.full[b], (c >> 1) & 1);
      wait(&bars.x_full, c & 1);
      tc_fence_after();
      float z[32], m = 0.f;
      tmem_ld32(ln + kTmX + t0, z);
      tmem_wait_ld();
      const __nv_bfloat16* vt = reinterpret_cast<const __nv_bfloat16*>(st + L::v) + col;
#pragma unroll
      for (int j = 0; j < 32; j += 4) {
        const float4 gk = *reinterpret_cast<const float4*>(fac + kGK * kL + t0 + j);
        const float4 be = *reinterpret_cast<const float4*>(fac + kBeta * kL + t0 + j);
        const float g4[4] = {gk.x, gk.y, gk.z, gk.w}, b4[4] = {be.x, be.y, be.z, be.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float x = live && t0 + j + e < len ? __bfloat162float(vt[(t0 + j + e) * 128]) : 0.f;
          z[j + e] = fmaf(-g4[e] * ss.inv, z[j + e], x);
          m = fmaxf(m, fabsf(b4[e] * z[j + e]));
        }
      }
      m = agree(1, m);
      named_bar(1 + q4, 64);
      const Scale sz = scale_of(fmaxf(m, other(1)));
      {
        float x[32], hi[16], lo[16];
#pragma unroll
        for (int j = 0; j < 32; ++j) x[j] = fac[kBeta * kL + t0 + j] * z[j];
        split32(x, sz.mul, hi, lo);
        tmem_st16(ln + kTmZ + 16 * half, hi);
        tmem_st16(ln + kTmZ + 32 + 16 * half, lo);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.z_ready);

      // Z' = Z + R (beta Z), U = beta Z', w U
      wait(&bars.r_full, c & 1);
      tc_fence_after();
      float u[32], mu = 0.f, mw = 0.f;
      tmem_ld32(ln + kTmX + t0, u);
      tmem_wait_ld();
#pragma unroll
      for (int j = 0; j < 32; j += 4) {
        const float4 ri = *reinterpret_cast<const float4*>(fac + kRInv * kL + t0 + j);
        const float4 be = *reinterpret_cast<const float4*>(fac + kBeta * kL + t0 + j);
        const float4 wk = *reinterpret_cast<const float4*>(fac + kWK * kL + t0 + j);
        const float r4[4] = {ri.x, ri.y, ri.z, ri.w}, b4[4] = {be.x, be.y, be.z, be.w}, w4[4] = {wk.x, wk.y, wk.z, wk.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          z[j + e] = fmaf(u[j + e] * sz.inv, r4[e], z[j + e]);
          u[j + e] = b4[e] * z[j + e];
          mu = fmaxf(mu, fabsf(u[j + e]));
          mw = fmaxf(mw, fabsf(w4[e] * u[j + e]));
        }
      }
      if (GRAD && tile_live) {
        float4* at = reinterpret_cast<float4*>(kept.Z + (base * 16 + tr) * kL + t0);
#pragma unroll
        for (int j = 0; j < 8; ++j) at[j] = make_float4(z[4 * j], z[4 * j + 1], z[4 * j + 2], z[4 * j + 3]);
      }
      mu = agree(2, mu);
      mw = agree(3, mw);
      named_bar(1 + q4, 64);
      const Scale su = scale_of(fmaxf(mu, other(2))), sw = scale_of(fmaxf(mw, other(3)));
      {
        float hi[16], lo[16];
        split32(u, su.mul, hi, lo);
        tmem_st16(ln + kTmU + 16 * half, hi);
        if (GRAD) tmem_st16(ln + kTmU + 32 + 16 * half, lo);
        if (GRAD && tile_live) {
          keep_row<kL>(kept.U + base * 16 * kL * 2, tr, t0, hi);
          if (tr == 0 && half == 0)
            *reinterpret_cast<float4*>(kept.U_inv + base * kQuarter) = make_float4(su.inv, su.inv, su.inv, su.inv);
        }
#pragma unroll
        for (int j = 0; j < 32; ++j) u[j] *= fac[kWK * kL + t0 + j];
        split32(u, sw.mul, hi, lo);
        tmem_st16(ln + kTmZ + 16 * half, hi);
        tmem_st16(ln + kTmZ + 32 + 16 * half, lo);
      }
      const float keep = fac[kGam * kL + kL - 1];
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.u_ready);

      // O = gam (Q S) + P U, while the update runs
      wait(&bars.o_full, c & 1);
      tc_fence_after();
      tmem_ld32(ln + kTmO + t0, z);
      tmem_ld32(ln + kTmX + t0, u);
      tmem_wait_ld();
#pragma unroll
      for (int j = 0; j < 32; j += 4) {
        const float4 gq = *reinterpret_cast<const float4*>(fac + kGQ * kL + t0 + j);
        const float4 pi = *reinterpret_cast<const float4*>(fac + kPInv * kL + t0 + j);
        const float g4[4] = {gq.x, gq.y, gq.z, gq.w}, p4[4] = {pi.x, pi.y, pi.z, pi.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) u[j + e] = fmaf(g4[e] * ss.inv, z[j + e], p4[e] * su.inv * u[j + e]);
      }
      if constexpr (GRAD) {  // dO . O over the 16 columns of a tile: lane l of 16 ends with tokens 2 l, 2 l + 1
        const __nv_bfloat16* dt = reinterpret_cast<const __nv_bfloat16*>(st + L::dout) + col;
#pragma unroll
        for (int j = 0; j < 32; ++j) u[j] = live && t0 + j < len ? u[j] * __bfloat162float(dt[(t0 + j) * 128]) : 0.f;
#pragma unroll
        for (int w = 16; w > 1; w /= 2) {
          const bool up = lane & (w / 2);
#pragma unroll
          for (int i = 0; i < w; ++i) {
            const float mine = up ? u[i + w] : u[i], theirs = up ? u[i] : u[i + w];
            u[i] = mine + __shfl_xor_sync(0xffffffffu, theirs, w / 2);
          }
        }
        if (tile_live)
          *reinterpret_cast<float2*>(kept.dots + base * kL + t0 + 2 * (lane & 15)) = make_float2(u[0], u[1]);
      } else if (live) {
        __nv_bfloat16* out = (__nv_bfloat16*)a.o + s.b * a.so.b + h * a.so.h + (s.lo + (long long)c * kL + t0) * a.so.t + v;
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (t0 + j < len) out[j * a.so.t] = __float2bfloat16_rn(u[j]);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.empty[b]);

      // S <- gam_63 S + (w K)^T U
      wait(&bars.d_full, c & 1);
      tc_fence_after();
#pragma unroll
      for (int blk = 0; blk < KH / 32; ++blk) {
        float d[32];
        tmem_ld32(ln + kTmD + half * KH + 32 * blk, d);
        tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < 32; ++j) S[32 * blk + j] = fmaf(keep, S[32 * blk + j], sw.inv * d[j]);
      }
    }
    if constexpr (GRAD) {
      const Scale ss = state_scale();
#pragma unroll
      for (int blk = 0; blk < KH / 32; ++blk) {
        float hi[16], lo[16];
        split32(S + 32 * blk, ss.mul, hi, lo);
        keep_state(s.slot + chunks + n, ss, blk, hi, lo);
      }
    }
    if (a.S_out && live)
#pragma unroll
      for (int j = 0; j < KH; ++j)
        if (half * KH + j < a.K) a.S_out[state + (size_t)(half * KH + j) * a.V] = S[j];
  }

  // drain before tensor memory is freed: every product issued has completed and every copy has landed (the
  // loops above may have stopped early after a wait that ran out)
  tc_fence_before();
  __syncthreads();
  if (tid == 0) {
    bool ok = mbar_wait(&bars.drain, 0, kTcWait);
    for (int b = 0; b < 2; ++b)
      if (issued > b) {
        const int last = b + 2 * ((issued - 1 - b) / 2);
        ok = mbar_wait(&bars.full[b], (last >> 1) & 1, kTcWait) && ok;
      }
    if (!ok) failed = 1;
    if (failed) atomicOr(err, 1u);
  }
  __syncthreads();
  tc_fence_after();
  if (warp == 0) sm100::tmem_dealloc(tm, kTmCols);
}

}  // namespace

template <int KP, bool GRAD>
cudaError_t launch_tc_walk(const GdrArgs& a, const char* keys, const char* records, const Kept& kept, unsigned int* err,
                           cudaStream_t stream) {
  constexpr int smem = TcStage<KP, GRAD>::total;
  const auto kernel = gdr_tc_kernel<KP, GRAD>;
  cudaError_t e = cudaMemsetAsync(err, 0, 64, stream);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  kernel<<<dim3((a.V + 127) / 128, a.H, a.N), kTcThreads, smem, stream>>>(a, keys, records, kept, err, a.wait);
  return cudaGetLastError();
}
template cudaError_t launch_tc_walk<64, false>(const GdrArgs&, const char*, const char*, const Kept&, unsigned int*, cudaStream_t);
template cudaError_t launch_tc_walk<128, false>(const GdrArgs&, const char*, const char*, const Kept&, unsigned int*, cudaStream_t);
template cudaError_t launch_tc_walk<64, true>(const GdrArgs&, const char*, const char*, const Kept&, unsigned int*, cudaStream_t);
template cudaError_t launch_tc_walk<128, true>(const GdrArgs&, const char*, const char*, const Kept&, unsigned int*, cudaStream_t);

}  // namespace gdr
}  // namespace mlstm
