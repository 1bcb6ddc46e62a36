// The forward pass over a sequence's chunks on tcgen05 (formulas, precision and records: gdr_tile.cuh; the
// same pass on warp-level products, for fp32 inputs and for few heads: gdr_walk.cuh).
//
// One block takes up to 128 value columns of one value head of one sequence.  Tensor memory has a lane for
// each value column: the state's, Z's and U's 16-bit parts are A operands there, k, q, R and P are B
// operands in shared memory, and every product has M = 128.  The state itself stays in the registers of
// eight warps (a lane is a column, two warps share its keys and tokens); each chunk's update is summed
// from zero in tensor memory and added in fp32.  A chunk is one chain:
//     S in parts -> K S, Q S -> Z -> R (beta Z) -> Z', U -> (w K)^T U -> S
// with the copies of the next chunk, Q S and P U beside it; a chunk's output is written beside the next one's
// K S.  That chain bounds it: 128 heads of 128 x 128, 2048 tokens, 172 us, 5.4 us or 9200 cycles a chunk; the four
// products take about 1700 of them, the rest is what the eight warps do in between (sixteen warps, four to
// a scheduler, took 10700: the chain waits for latencies, not for issue slots).
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

template <int KP>
struct TcStage {
  static constexpr int q = keys_bytes(KP, 1) / 2;
  static constexpr int record = keys_bytes(KP, 1);
  static constexpr int p = record + 2 * kTile;
  static constexpr int factors = record + record_bytes(false) - kFactorBytes;
  static constexpr int v = record + record_bytes(false);  // [64][128]
  static constexpr int bytes = v + kL * 256;
  // behind two stages: the output on its way to memory [64 tokens][136], the maxima in exchange [4][2][128]
  static constexpr int out = 2 * bytes;
  static constexpr int ex = out + kL * 272;
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

// 2 N values times f as two parts: N words each.
template <int N>
__device__ __forceinline__ void split_words(const float* x, float f, float (&hi)[N], float (&lo)[N]) {
#pragma unroll
  for (int j = 0; j < N; ++j) {
    uint32_t h, l;
    split(x[2 * j] * f, x[2 * j + 1] * f, h, l);
    hi[j] = __uint_as_float(h), lo[j] = __uint_as_float(l);
  }
}
template <int KP>
__global__ void __launch_bounds__(kTcThreads, 1) gdr_tc_kernel(const GdrArgs a, const char* keys, const char* records,
                                                               unsigned int* err, long long limit) {
  using L = TcStage<KP>;
  constexpr int KH = KP / 2, TH = kL / 2;  // keys and tokens of a value warp
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
    const char* rec = records + (s.slot * a.H + h) * record_bytes(false);
    const int width = min(128, a.V - v0) * 2;  // bytes of a row of v: a multiple of 16
    const __nv_bfloat16* v = (const __nv_bfloat16*)a.v + s.b * a.sv.b + h * a.sv.h + s.lo * a.sv.t + v0;
    for (int c = 0; c < chunks; ++c) {
      const int b = c & 1, rows = (int)min((long long)kL, s.len - (long long)c * kL);
      if (!wait(&bars.empty[b], ((c >> 1) & 1) ^ 1)) break;
      uint8_t* st = sm + b * L::bytes;
      if (lane == 0) {
        mbar_arrive_expect_tx(&bars.full[b], keys_bytes(KP, 1) + record_bytes(false) + rows * width);
        sm100::bulk_load(st, kq + (long long)c * a.HK * keys_bytes(KP, 1), keys_bytes(KP, 1), &bars.full[b]);
        sm100::bulk_load(st + L::record, rec + (long long)c * a.H * record_bytes(false), record_bytes(false), &bars.full[b]);
      }
      __syncwarp();
      for (int t = lane; t < rows; t += 32) {
        const long long at = (long long)c * kL + t;
        sm100::bulk_load(st + L::v + t * 256, v + at * a.sv.t, width, &bars.full[b]);
      }
      issued = c + 1;
      __syncwarp();
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------------------------ products
    bool ok = true;
    // D (+)= A B over the 16-column steps of the state, A's part at column `at`, B's keys at `bd`
    auto by_state = [&](uint32_t d, uint32_t at, uint64_t bd, bool more) {
#pragma unroll
      for (int k = 0; k < KP / 16; ++k)
        mma_bf16_ts(d, at + 8 * k, bd + (uint64_t)((k >> 2) * 512 + (k & 3) * 2), idesc_f16(64, 0), more || k > 0 ? 1u : 0u);
    };
    // the same over the tokens of R or P
    auto by_tokens_of = [&](uint32_t d, uint32_t at, uint64_t bd, bool more) {
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
        mma_bf16_ts(d, at + 8 * kk, bd + (uint64_t)(kk * 2), idesc_f16(64, 0), more || kk > 0 ? 1u : 0u);
    };
    for (int c = 0; c < chunks; ++c) {
      const int b = c & 1;
      const uint32_t st = smem_u32(sm) + b * L::bytes;
      ok = wait(&bars.full[b], (c >> 1) & 1) && wait(&bars.s_ready, c & 1);
      if (!ok) break;
      tc_fence_after();
      if (elect_one()) {  // lo parts first: they are small, and so is what the sums cut off below them
        const uint64_t kd = smem_desc_sw128(st, 16, 1024), qd = smem_desc_sw128(st + L::q, 16, 1024);
        by_state(tm + kTmX, tm + kTmS + KP / 2, kd, false);
        by_state(tm + kTmX, tm + kTmS, kd, true);
        mma_commit(&bars.x_full);
        by_state(tm + kTmO, tm + kTmS, qd, false);  // one part, as of P and U: 11 bits for an output of 8 (two: 175 -> 189 us)
      }
      __syncwarp();
      ok = wait(&bars.z_ready, c & 1);
      if (!ok) break;
      tc_fence_after();
      if (elect_one()) {
        const uint64_t rd = smem_desc_sw128(st + L::record, 16, 1024);
        by_tokens_of(tm + kTmX, tm + kTmZ + 32, rd, false);
        by_tokens_of(tm + kTmX, tm + kTmZ, rd + (kTile >> 4), true);
        by_tokens_of(tm + kTmX, tm + kTmZ, rd, true);
        mma_commit(&bars.r_full);
      }
      __syncwarp();
      ok = wait(&bars.u_ready, c & 1);
      if (!ok) break;
      tc_fence_after();
      if (elect_one()) {
        const uint64_t kmn = smem_desc_sw128(st, 8192, 1024), pd = smem_desc_sw128(st + L::p, 16, 1024);
        by_tokens_of(tm + kTmX, tm + kTmU, pd, false);
        mma_commit(&bars.o_full);
#pragma unroll
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
    const int t0 = TH * half, k0 = KH * half;
    float S[KH];
#pragma unroll
    for (int j = 0; j < KH; ++j) S[j] = a.S0 && live && k0 + j < a.K ? a.S0[state + (size_t)(k0 + j) * a.V] : 0.f;
    // The larger of the two warps' maxima of a column: each gives its own, they meet, and each takes both.
    auto give_max = [&](int which, float m) { ex[(which * 2 + half) * 128 + col] = m; };
    auto meet = [&] { named_bar(1 + q4, 64); };
    auto take_max = [&](int which) { return fmaxf(ex[which * 256 + col], ex[which * 256 + 128 + col]); };
    auto max4 = [](float m, const float* x) {
      return fmaxf(fmaxf(m, fmaxf(fabsf(x[0]), fabsf(x[1]))), fmaxf(fabsf(x[2]), fabsf(x[3])));
    };
    auto state_scale = [&] {
      float m = 0.f;
#pragma unroll
      for (int j = 0; j < KH; j += 4) m = max4(m, S + j);
      give_max(0, m);
      meet();
      return scale_of(take_max(0));
    };
    // The output of a chunk, two tokens a word, leaves by way of shared memory: rows of this warp's 32 columns.
    uint32_t y[TH / 2];
    char* mine = reinterpret_cast<char*>(sm + L::out) + t0 * 272 + q4 * 64;
    auto write_out = [&](int c) {
#pragma unroll
      for (int j = 0; j < TH / 2; ++j) {
        *reinterpret_cast<uint16_t*>(mine + 2 * j * 272 + lane * 2) = (uint16_t)y[j];
        *reinterpret_cast<uint16_t*>(mine + (2 * j + 1) * 272 + lane * 2) = (uint16_t)(y[j] >> 16);
      }
      __syncwarp();
      const int len = (int)min((long long)kL, s.len - (long long)c * kL), piece = lane & 3, first = v0 + 32 * q4 + 8 * piece;
      __nv_bfloat16* o = (__nv_bfloat16*)a.o + s.b * a.so.b + h * a.so.h + (s.lo + (long long)c * kL + t0) * a.so.t + first;
#pragma unroll
      for (int i = 0; i < TH / 8; ++i) {
        const int t = i * 8 + (lane >> 2);
        if (first < a.V && t0 + t < len)
          *reinterpret_cast<uint4*>(o + t * a.so.t) = *reinterpret_cast<const uint4*>(mine + t * 272 + piece * 16);
      }
      __syncwarp();
    };
    auto at4 = [](const float* f, int t) { return *reinterpret_cast<const float4*>(f + t); };
    for (int c = 0; c < chunks; ++c) {
      const int b = c & 1, len = (int)min((long long)kL, s.len - (long long)c * kL);
      const uint8_t* st = sm + b * L::bytes;
      const float* fac = reinterpret_cast<const float*>(st + L::factors) + t0;
      const Scale ss = state_scale();  // (both warps have the update before: its columns may be written again)
#pragma unroll
      for (int i = 0; i < KH; i += 32) {
        float hi[16], lo[16];
        split_words(S + i, ss.mul, hi, lo);
        tmem_st16(ln + kTmS + (k0 + i) / 2, hi);
        tmem_st16(ln + kTmS + KP / 2 + (k0 + i) / 2, lo);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.s_ready);
      if (c > 0) write_out(c - 1);  // beside K S

      // Z = V - gam (K S)
      wait(&bars.full[b], (c >> 1) & 1);
      float z[TH], u[TH], m = 0.f;
      {
        const __nv_bfloat16* vt = reinterpret_cast<const __nv_bfloat16*>(st + L::v) + t0 * 128 + col;
        if (len == kL && v0 + 128 <= a.V) {
#pragma unroll
          for (int j = 0; j < TH; ++j) u[j] = __bfloat162float(vt[j * 128]);
        } else {
#pragma unroll
          for (int j = 0; j < TH; ++j) u[j] = live && t0 + j < len ? __bfloat162float(vt[j * 128]) : 0.f;
        }
      }
      wait(&bars.x_full, c & 1);
      tc_fence_after();
      tmem_ld32(ln + kTmX + t0, z);
      tmem_wait_ld();
#pragma unroll
      for (int j = 0; j < TH; j += 4) {
        const float4 gk = at4(fac + kGK * kL, j), be = at4(fac + kBeta * kL, j);
        z[j] = fmaf(-gk.x * ss.inv, z[j], u[j]), z[j + 1] = fmaf(-gk.y * ss.inv, z[j + 1], u[j + 1]);
        z[j + 2] = fmaf(-gk.z * ss.inv, z[j + 2], u[j + 2]), z[j + 3] = fmaf(-gk.w * ss.inv, z[j + 3], u[j + 3]);
        u[j] = be.x * z[j], u[j + 1] = be.y * z[j + 1], u[j + 2] = be.z * z[j + 2], u[j + 3] = be.w * z[j + 3];
        m = max4(m, u + j);
      }
      give_max(1, m);
      meet();
      const Scale sz = scale_of(take_max(1));
      {
        float hi[TH / 2], lo[TH / 2];
        split_words(u, sz.mul, hi, lo);
        tmem_st16(ln + kTmZ + t0 / 2, hi);
        tmem_st16(ln + kTmZ + 32 + t0 / 2, lo);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.z_ready);

      // Z' = Z + R (beta Z), U = beta Z', w U
      wait(&bars.r_full, c & 1);
      tc_fence_after();
      float mu = 0.f, mw = 0.f;
      tmem_ld32(ln + kTmX + t0, u);
      tmem_wait_ld();
#pragma unroll
      for (int j = 0; j < TH; j += 4) {
        const float4 ri = at4(fac + kRInv * kL, j), be = at4(fac + kBeta * kL, j), wk = at4(fac + kWK * kL, j);
        z[j] = fmaf(u[j], ri.x * sz.inv, z[j]), z[j + 1] = fmaf(u[j + 1], ri.y * sz.inv, z[j + 1]);
        z[j + 2] = fmaf(u[j + 2], ri.z * sz.inv, z[j + 2]), z[j + 3] = fmaf(u[j + 3], ri.w * sz.inv, z[j + 3]);
        u[j] = be.x * z[j], u[j + 1] = be.y * z[j + 1], u[j + 2] = be.z * z[j + 2], u[j + 3] = be.w * z[j + 3];
        z[j] = wk.x * u[j], z[j + 1] = wk.y * u[j + 1], z[j + 2] = wk.z * u[j + 2], z[j + 3] = wk.w * u[j + 3];
        mu = max4(mu, u + j);
        mw = max4(mw, z + j);
      }
      give_max(2, mu);
      give_max(3, mw);
      meet();
      const Scale su = scale_of(take_max(2)), sw = scale_of(take_max(3));
      {
        float hi[TH / 2], lo[TH / 2];
        split_words(u, su.mul, hi, lo);
        tmem_st16(ln + kTmU + t0 / 2, hi);
        split_words(z, sw.mul, hi, lo);
        tmem_st16(ln + kTmZ + t0 / 2, hi);
        tmem_st16(ln + kTmZ + 32 + t0 / 2, lo);
      }
      const float keep = fac[kGam * kL + kL - 1 - t0];
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
      for (int j = 0; j < TH; j += 4) {
        const float4 gq = at4(fac + kGQ * kL, j), pi = at4(fac + kPInv * kL, j);
        u[j] = fmaf(gq.x * ss.inv, z[j], pi.x * su.inv * u[j]);
        u[j + 1] = fmaf(gq.y * ss.inv, z[j + 1], pi.y * su.inv * u[j + 1]);
        u[j + 2] = fmaf(gq.z * ss.inv, z[j + 2], pi.z * su.inv * u[j + 2]);
        u[j + 3] = fmaf(gq.w * ss.inv, z[j + 3], pi.w * su.inv * u[j + 3]);
      }
#pragma unroll
      for (int j = 0; j < TH / 2; ++j) y[j] = pack_bf16(u[2 * j], u[2 * j + 1]);
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.empty[b]);

      // S <- gam_63 S + (w K)^T U
      wait(&bars.d_full, c & 1);
      tc_fence_after();
#pragma unroll
      for (int i = 0; i < KH; i += 32) {
        float d[32];
        tmem_ld32(ln + kTmD + k0 + i, d);
        tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < 32; ++j) S[i + j] = fmaf(keep, S[i + j], sw.inv * d[j]);
      }
    }
    if (chunks > 0) write_out(chunks - 1);
    if (a.S_out && live)
#pragma unroll
      for (int j = 0; j < KH; ++j)
        if (k0 + j < a.K) a.S_out[state + (size_t)(k0 + j) * a.V] = S[j];
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

template <int KP>
cudaError_t launch_tc_walk(const GdrArgs& a, const char* keys, const char* records, unsigned int* err, cudaStream_t stream) {
  constexpr int smem = TcStage<KP>::total;
  const auto kernel = gdr_tc_kernel<KP>;
  cudaError_t e = cudaMemsetAsync(err, 0, 64, stream);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  kernel<<<dim3((a.V + 127) / 128, a.H, a.N), kTcThreads, smem, stream>>>(a, keys, records, err, a.wait);
  return cudaGetLastError();
}
template cudaError_t launch_tc_walk<64>(const GdrArgs&, const char*, const char*, unsigned int*, cudaStream_t);
template cudaError_t launch_tc_walk<128>(const GdrArgs&, const char*, const char*, unsigned int*, cudaStream_t);

}  // namespace gdr
}  // namespace mlstm
