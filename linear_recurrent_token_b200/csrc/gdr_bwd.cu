// Gradients of the gated delta rule (formulas, precision and layouts: gdr_tile.cuh).
//
// Four kernels: what does not depend on the state (gdr_prep_kernel), the forward pass again, which keeps
// the states (gdr_walk_kernel with GRAD), the pass backward over the chunks with dS in registers, which
// gives dV and everything that needs fp32 accuracy (gdr_back_kernel), and for all chunks at once the
// gradients of q and k and of the gates (gdr_grad_kernel):
//     dQ = gam (dO S^T) + (dP o D) K            dP = dO U^T (lower)   dW = dV U^T (strictly lower)
//     dK = -gam (dV S^T) + w (U dS^T) + (dP o D)^T Q - (dW o D) K - (dW o D)^T K
// with S at the chunk's start and dS at its end.
#include "gdr_walk.cuh"

namespace mlstm {
namespace gdr {
namespace {

// A block takes 16 TN value columns of one value head of one sequence, chunks from the last to the first.
template <typename T, int KP, int TN>
__global__ void __launch_bounds__(32 * kQuarter * TN) gdr_back_kernel(const GdrArgs a, const char* keys,
                                                                      const char* records, const Kept kept) {
  using L = Stage<T, KP, TN, true>;
  constexpr int NP = L::NP, NK = kept_parts<T>(), KS = KP / 64, threads = 32 * kQuarter * TN;
  // In exchange: dS, then beta dU in its place; dO by P's scale; gam dV; gam dO.
  constexpr int fy = L::fs;
  extern __shared__ __align__(128) char smem[];
  const int n = blockIdx.z, h = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int local = warp / kQuarter, w = warp % kQuarter, tile = blockIdx.x * TN + local, tiles = (a.V + 15) / 16;
  const int col0 = blockIdx.x * 16 * TN, v0 = tile * 16, cols = min(16, a.V - v0);
  const bool live = tile < tiles;
  const Seq s = sequence(a, n);
  const int chunks = (int)((s.len + kL - 1) / kL);
  const size_t state = ((size_t)n * a.H + h) * a.K * a.V;
  const int ra = lane >> 2, ca = 2 * (lane & 3);
  char* mats = smem + L::chunks * L::chunk;
  char* ex = mats + L::matrices + local * L::tile;
  float* inv = reinterpret_cast<float*>(ex + L::inv);

  float D[2 * KS][4];
#pragma unroll
  for (int j = 0; j < 2 * KS; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int col = ra + (e >> 1) * 8, key = w * (KP / 4) + 8 * j + ca + (e & 1);
      D[j][e] = a.dS && col < cols && key < a.K ? a.dS[state + (size_t)key * a.V + v0 + col] : 0.f;
    }
  auto slot = [&](int c) { return smem + (L::chunks == 2 ? (c & 1) * L::chunk : 0); };
  if (chunks > 0) {
    fetch_chunk<T, KP, TN, true>(a, s, s.slot + chunks - 1, h, chunks - 1, col0, keys, records, smem_u32(slot(chunks - 1)));
    cp_commit();
  }
  for (int c = chunks - 1; c >= 0; --c) {
    const long long rec = s.slot + c;
    const size_t base = ((size_t)rec * a.H + h) * tiles + tile;
    char* st = slot(c);
    const float* fac = reinterpret_cast<const float*>(st + L::factors);
    {
      const Scale sc = scale_of(tile_max(D));
      give<KS, 2>(D, sc, ex + L::fs, inv, w, lane);
      if (live) {  // dS for the gradients of k, and <dS, S> with the state that the forward pass left here
        const size_t after = ((size_t)(rec + n + 1) * a.H + h) * tiles + tile;
        float end = 0.f;
#pragma unroll
        for (int i = 0; i < KS; ++i) {
          uint4 hi, lo;
          split_a(D[2 * i], D[2 * i + 1], sc.mul, hi, lo);
          kept.D[(base * NK * (KP / 16) + w * KS + i) * 32 + lane] = hi;
          if (NK == 2) kept.D[((base * NK + 1) * (KP / 16) + w * KS + i) * 32 + lane] = lo;
          const uint4 sh = kept.S[(after * 2 * (KP / 16) + w * KS + i) * 32 + lane];
          const uint4 sl = kept.S[((after * 2 + 1) * (KP / 16) + w * KS + i) * 32 + lane];
          const uint32_t h4[4] = {sh.x, sh.y, sh.z, sh.w}, l4[4] = {sl.x, sl.y, sl.z, sl.w};
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const float2 f = unpack(h4[r]), g = unpack(l4[r]);
            end = fmaf(D[2 * i + (r >> 1)][(r & 1) * 2], f.x + g.x, end);
            end = fmaf(D[2 * i + (r >> 1)][(r & 1) * 2 + 1], f.y + g.y, end);
          }
        }
#pragma unroll
        for (int d = 16; d > 0; d /= 2) end += __shfl_xor_sync(0xffffffffu, end, d);
        if (lane == 0) {
          kept.D_inv[base * kQuarter + w] = sc.inv;
          kept.ends[base * kQuarter + w] = end * kept.S_inv[after * kQuarter + w];
        }
      }
    }
    cp_wait<0>();
    __syncthreads();  // the chunk has come, dS is in exchange, and nobody is in the chunk behind
    fetch_matrices<true, threads>(a, rec, h, records, smem_u32(mats));
    cp_commit();
    if (L::chunks == 2) {
      if (c > 0) fetch_chunk<T, KP, TN, true>(a, s, rec - 1, h, c - 1, col0, keys, records, smem_u32(slot(c - 1)));
      cp_commit();
    }
    // this quarter's share of dO by P's scale, and gam dO
    float x[2][4], y[2][4];
    {
      float d[2][4];
      read_columns<T, L::row>(d, st + L::dout + w * 16 * L::row + local * 16 * (int)sizeof(T), lane);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float2 pi = factor(fac + kPInv * kL, w * 16, j, lane), gq = factor(fac + kGQ * kL, w * 16, j, lane);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[j][e] = d[j][e] * (e & 1 ? pi.y : pi.x);
          y[j][e] = d[j][e] * (e & 1 ? gq.y : gq.x);
        }
      }
      give<1, NP>(x, scale_of(tile_max(x)), ex + L::fu, inv + 2 * kQuarter, w, lane);
      give<1, 2>(y, scale_of(tile_max(y)), ex + L::fz, inv + 4 * kQuarter, w, lane);
    }
    // dU = w (K dS) + P^T dO
    by_keys<KP, NP, false, false>(x, y, ex + L::fs, inv, smem_u32(st), 0u, w, lane);
    float4 z0 = make_float4(0.f, 0.f, 0.f, 0.f), z1 = z0;
    if (live) z0 = kept.Z[(base * 8 + 2 * w) * 32 + lane], z1 = kept.Z[(base * 8 + 2 * w + 1) * 32 + lane];
    cp_wait<L::chunks == 2 ? 1 : 0>();
    __syncthreads();  // R and P have come, dO is in exchange, dS has been read
    by_tokens<true, NP, 2>(y, ex + L::fu, inv + 2 * kQuarter, smem_u32(mats) + 2 * kTile, w, lane);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float2 wk = factor(fac + kWK * kL, w * 16, j, lane), be = factor(fac + kBeta * kL, w * 16, j, lane);
      const float2 ri = factor(fac + kRInv * kL, w * 16, j, lane);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[j][e] = fmaf(x[j][e], e & 1 ? wk.y : wk.x, y[j][e]);
        y[j][e] = x[j][e] * (e & 1 ? be.y * ri.y : be.x * ri.x);
      }
    }
    give<1, 2>(y, scale_of(tile_max(y)), ex + fy, inv + kQuarter, w, lane);
    tile_barrier(local);  // beta dU is in exchange
    // dY = dU + R^T (beta dU), dV = beta dY
    by_tokens<true, 2, 2>(y, ex + fy, inv + kQuarter, smem_u32(mats), w, lane);
    char* vt = st + L::v + w * 16 * L::row + local * 16 * (int)sizeof(T);
    {
      float dot[4], v[2][4];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float2 be = factor(fac + kBeta * kL, w * 16, j, lane), gk = factor(fac + kGK * kL, w * 16, j, lane);
        const float4 z = j ? z1 : z0;
#pragma unroll
        for (int e = 0; e < 4; ++e) x[j][e] += y[j][e];
        dot[2 * j] = x[j][0] * z.x + x[j][2] * z.z;
        dot[2 * j + 1] = x[j][1] * z.y + x[j][3] * z.w;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[j][e] *= e & 1 ? be.y : be.x;
          y[j][e] = x[j][e] * (e & 1 ? -gk.y : -gk.x);
        }
      }
      give<1, 2>(y, scale_of(tile_max(y)), ex + L::fw, inv + 3 * kQuarter, w, lane);
      const float2 db = column_sum(dot, lane);
      read_columns<T, L::row>(v, vt, lane);
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e) dot[2 * j + e] = x[j][e] * v[j][e] + x[j][e + 2] * v[j][e + 2];
      const float2 dv = column_sum(dot, lane);
      if (live) {
        const size_t at = base * kL + w * 16 + (lane >> 4) * 8 + ca;
        if ((lane & 12) == 0) {
          *reinterpret_cast<float2*>(kept.dbeta + at) = db;
          const float2 was = *reinterpret_cast<const float2*>(kept.dots + at);
          *reinterpret_cast<float2*>(kept.dots + at) = make_float2(was.x - dv.x, was.y - dv.y);
        }
        const Scale sc = scale_of(tile_max(x));
        uint4 hi, lo;
        split_a(x[0], x[1], sc.mul, hi, lo);
        if (lane == 0) kept.dV_inv[base * kQuarter + w] = sc.inv;
        kept.dV[(base * NK * 4 + w) * 32 + lane] = hi;
        if (NK == 2) kept.dV[((base * NK + 1) * 4 + w) * 32 + lane] = lo;
      }
    }
    tile_barrier(local);  // gam dV is in exchange
    const long long t0 = (long long)c * kL + w * 16;
    T* out = (T*)a.dv + s.b * a.sdv.b + h * a.sdv.h + (s.lo + t0) * a.sdv.t + v0;
    write_columns<T, L::row>(x, vt, out, a.sdv.t, (int)max(0LL, min(16LL, s.len - t0)), cols, lane);
    // dS <- gam_63 dS + Q^T (gam dO) - K^T (gam dV)
    to_state<KP, NP>(D, fac[kGam * kL + kL - 1], ex + L::fz, inv + 4 * kQuarter, smem_u32(st) + L::q, w, lane);
    to_state<KP, NP>(D, 1.f, ex + L::fw, inv + 3 * kQuarter, smem_u32(st), w, lane);
    if (L::chunks == 1 && c > 0) {
      __syncthreads();
      fetch_chunk<T, KP, TN, true>(a, s, rec - 1, h, c - 1, col0, keys, records, smem_u32(smem));
      cp_commit();
    }
  }
  if (a.dS0) {
#pragma unroll
    for (int j = 0; j < 2 * KS; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int col = ra + (e >> 1) * 8, key = w * (KP / 4) + 8 * j + ca + (e & 1);
        if (col < cols && key < a.K) a.dS0[state + (size_t)key * a.V + v0 + col] = D[j][e];
      }
  }
}

// ---------------------------------------------------------------------------------------------
constexpr int kGradThreads = 256;
constexpr int kVB = 64;  // value columns at a time: four kept tiles

template <typename T, int KP>
struct GradStage {
  static constexpr int NP = sizeof(T) == 4 ? 2 : 1;
  // behind k and q: dO [64][64], then as [value][token or key]: dV, U, S, dS
  static constexpr int dout = keys_bytes(KP, NP);
  static constexpr int dv = dout + NP * kTile;
  static constexpr int u = dv + NP * kTile;
  static constexpr int s = u + NP * kTile;
  static constexpr int ds = s + NP * kVB * KP * 2;
  // after the value columns, in their place: dP o D by k's and q's scales, dW o D by k's, rows and columns
  static constexpr int mat = dout;
  static constexpr int mats_end = mat + 4 * NP * kTile;
  static constexpr int cols_end = ds + NP * kVB * KP * 2;
  static constexpr int small = cols_end > mats_end ? cols_end : mats_end;
  // G in two parts, factors, dO's scales, maxima of the matrices
  static constexpr int bytes = small + kL * 8 + kFactorBytes + kL * 4 + 8 * 4 * 4;
};

// A kept operand's tiles first .. first + 3 as [64 values][COLS] fp16 with one scale, which it returns.
template <int COLS, int NP, int NK>
__device__ __forceinline__ float load_kept(const uint4* at, const float* inv, size_t base, int first, int tiles, char* out) {
  float big = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (first + i < tiles) {
      const float4 f = *reinterpret_cast<const float4*>(inv + (base + first + i) * kQuarter);
      big = fmaxf(big, fmaxf(fmaxf(f.x, f.y), fmaxf(f.z, f.w)));
    }
  constexpr int steps = COLS / 16;
  for (int e = threadIdx.x; e < 4 * NP * steps * 32; e += kGradThreads) {
    const int lane = e & 31, kk = (e >> 5) % steps, part = (e >> 5) / steps % NP, i = (e >> 5) / (steps * NP);
    uint4 x = make_uint4(0u, 0u, 0u, 0u);
    if (first + i < tiles) {
      x = at[(((base + first + i) * NK + part) * steps + kk) * 32 + lane];
      // a power of two, at most 1
      const __half2 f = __float2half2_rn(inv[(base + first + i) * kQuarter + kk / (steps / kQuarter)] / big);
      __half2* p = reinterpret_cast<__half2*>(&x);
#pragma unroll
      for (int j = 0; j < 4; ++j) p[j] = __hmul2(p[j], f);
    }
    const int row = i * 16 + (lane >> 2), col = kk * 16 + 2 * (lane & 3);
    char* o = out + part * kVB * COLS * 2;
    *reinterpret_cast<uint32_t*>(o + piece_at<COLS>(row, col) + (col & 7) * 2) = x.x;
    *reinterpret_cast<uint32_t*>(o + piece_at<COLS>(row + 8, col) + (col & 7) * 2) = x.y;
    *reinterpret_cast<uint32_t*>(o + piece_at<COLS>(row, col + 8) + (col & 7) * 2) = x.z;
    *reinterpret_cast<uint32_t*>(o + piece_at<COLS>(row + 8, col + 8) + (col & 7) * 2) = x.w;
  }
  return big;
}

// A fragments (16 rows from r0, 16 columns of k step kk): of a tile [row][k], or of a tile [k][row].
template <int COLS, bool TRANS>
__device__ __forceinline__ void a_frag(uint32_t (&f)[4], uint32_t tile, int r0, int kk, int lane) {
  if constexpr (TRANS)
    ldsm4t(f, tile + piece_at<COLS>(kk * 16 + at_row(lane), r0 + at_col(lane)));
  else
    ldsm4(f, tile + piece_at<COLS>(r0 + bt_row(lane), kk * 16 + bt_col(lane)));
}

// acc[j] += A B over k steps lo .. hi - 1: B a tile [k][n] with COLS columns, n from c0.  Two parts each
// where NP is 2 (planes pa and pb bytes further on).
template <int ACOLS, bool TRANS, int COLS, int NP, int NT>
__device__ __forceinline__ void gemm(float (&acc)[NT][4], uint32_t at, int pa, int r0, uint32_t bt, int pb, int c0, int lo,
                                     int hi, int lane) {
#pragma unroll
  for (int kk = 0; kk < 4; ++kk) {
    if (kk < lo || kk >= hi) continue;
    uint32_t f[4], g[4];
    a_frag<ACOLS, TRANS>(f, at, r0, kk, lane);
    if constexpr (NP == 2) a_frag<ACOLS, TRANS>(g, at + pa, r0, kk, lane);
#pragma unroll
    for (int j = 0; j < NT; j += 2) {
      const int off = piece_at<COLS>(kk * 16 + bt_row(lane), c0 + j * 8 + bt_col(lane));
      uint32_t b[4];
      ldsm4t(b, bt + off);
      if constexpr (NP == 2) {
        uint32_t l[4];
        ldsm4t(l, bt + pb + off);
        mma(acc[j], g, b[0], b[1]), mma(acc[j + 1], g, b[2], b[3]);
        mma(acc[j], f, l[0], l[1]), mma(acc[j + 1], f, l[2], l[3]);
      }
      mma(acc[j], f, b[0], b[1]), mma(acc[j + 1], f, b[2], b[3]);
    }
  }
}
// sum += acc times a factor of the row (the lane's rows r and r + 8)
template <int NT>
__device__ __forceinline__ void add_rows(float (&sum)[NT][4], const float (&acc)[NT][4], float f0, float f1) {
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) sum[j][e] = fmaf(acc[j][e], e < 2 ? f0 : f1, sum[j][e]);
}

__device__ __forceinline__ float ends(const Kept& kept, size_t tile) {
  const float4 e = *reinterpret_cast<const float4*>(kept.ends + tile * kQuarter);
  return (e.x + e.y) + (e.z + e.w);
}

// One block for each chunk and key head; the value heads that share it follow one another and their
// shares add up in registers.  A warp has 16 tokens and half of the keys (or of the other token).
template <typename T, int KP>
__global__ void __launch_bounds__(kGradThreads) gdr_grad_kernel(const GdrArgs a, const char* keys, const char* records,
                                                                const Kept kept) {
  using L = GradStage<T, KP>;
  constexpr int NP = L::NP, NK = kept_parts<T>(), NT = KP / 16;
  extern __shared__ __align__(128) char smem[];
  float2* G = reinterpret_cast<float2*>(smem + L::small);
  float* fac = reinterpret_cast<float*>(G + kL);
  float* oinv = fac + kFactors * kL;
  float* most = oinv + kL;  // [8 warps][4]
  int n, c;
  Seq s;
  if (!find_chunk(a, blockIdx.x, &n, &s, &c)) return;
  const int hk = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, tiles = (a.V + 15) / 16;
  const long long rec = blockIdx.x, t0 = s.lo + (long long)c * kL;
  const int len = (int)min((long long)kL, s.len - (long long)c * kL);
  const uint32_t su = smem_u32(smem);
  const int r0 = (warp & 3) * 16, half = warp >> 2, k0 = half * (KP / 2), c0 = half * 32;
  const int ra = r0 + (lane >> 2), ca = 2 * (lane & 3);

  const char* kq = keys + (rec * a.HK + hk) * keys_bytes(KP, NP);
  for (int i = tid; i < keys_bytes(KP, NP) / 16; i += kGradThreads) cp_async16(su + i * 16, kq + i * 16, true);
  cp_commit();

  float dq[NT][4], dk[NT][4];
  zero(dq), zero(dk);
  for (int h = hk * (a.H / a.HK); h < (hk + 1) * (a.H / a.HK); ++h) {
    const size_t base = ((size_t)rec * a.H + h) * tiles, sbase = ((size_t)(rec + n) * a.H + h) * tiles;
    const float* fin = reinterpret_cast<const float*>(records + (rec * a.H + h) * record_bytes(true) + 4 * kTile);
    for (int e = tid; e < kFactors * kL; e += kGradThreads) fac[e] = fin[e];
    if (warp == 0) {
      const double2 g = cumulative(a.g + s.b * a.sg.b + h * a.sg.h, a.sg.t, t0, len, lane);
      G[2 * lane] = two_parts(g.x), G[2 * lane + 1] = two_parts(g.y);
      // dg: what follows in the chunk, and the state's share at its end; dbeta
      float x[2] = {0.f, 0.f}, b[2] = {0.f, 0.f}, end = 0.f;
      for (int i = 0; i < tiles; ++i) {
        const float2 d = *reinterpret_cast<const float2*>(kept.dots + (base + i) * kL + 2 * lane);
        const float2 e = *reinterpret_cast<const float2*>(kept.dbeta + (base + i) * kL + 2 * lane);
        x[0] += d.x, x[1] += d.y, b[0] += e.x, b[1] += e.y, end += ends(kept, base + i);
      }
      double sum = (double)x[0] + x[1];
#pragma unroll
      for (int d = 1; d < 32; d *= 2) {
        const double y = __shfl_down_sync(0xffffffffu, sum, d);
        if (lane + d < 32) sum += y;
      }
      const size_t out = ((size_t)s.b * a.H + h) * a.T + t0 + 2 * lane;
      if (2 * lane < len) a.dg[out] = (float)(sum + end), a.dbeta[out] = b[0];
      if (2 * lane + 1 < len) a.dg[out + 1] = (float)(sum - x[0] + end), a.dbeta[out + 1] = b[1];
    }
    float dP[4][4], dW[4][4];
    zero(dP), zero(dW);
    for (int vb = 0; vb < a.V; vb += kVB) {
      if (vb > 0) __syncthreads();  // the columns before are read
      const float uinv = load_kept<kL, NP, NK>(kept.U, kept.U_inv, base, vb / 16, tiles, smem + L::u);
      const float vinv = load_kept<kL, NP, NK>(kept.dV, kept.dV_inv, base, vb / 16, tiles, smem + L::dv);
      const float sinv = load_kept<KP, NP, 2>(kept.S, kept.S_inv, sbase, vb / 16, tiles, smem + L::s);
      const float dinv = load_kept<KP, NP, NK>(kept.D, kept.D_inv, base, vb / 16, tiles, smem + L::ds);
      {  // dO, rows scaled: four threads a row
        const int row = tid >> 2, part = tid & 3;
        const T* src = (const T*)a.dout + s.b * a.so.b + h * a.so.h + (t0 + row) * a.so.t + vb;
        float x[2][8], m = 0.f;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int col = part * 16 + i * 8;
          load8<T>(src + col, row < len && vb + col < a.V, x[i]);
#pragma unroll
          for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(x[i][e]));
        }
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
        const Scale sc = scale_of(m);
        if (part == 0) oinv[row] = sc.inv;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) split(x[i][2 * e] * sc.mul, x[i][2 * e + 1] * sc.mul, hi[e], lo[e]);
          char* at = smem + L::dout + piece_at<kVB>(row, part * 16 + i * 8);
          *reinterpret_cast<uint4*>(at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          if (NP == 2) *reinterpret_cast<uint4*>(at + kTile) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
      }
      cp_wait<0>();
      __syncthreads();
      const float o0 = oinv[ra], o1 = oinv[ra + 8];
      float acc[NT][4];
      zero(acc);  // gam (dO S^T)
      gemm<kVB, false, KP, NP, NT>(acc, su + L::dout, kTile, r0, su + L::s, kVB * KP * 2, k0, 0, 4, lane);
      add_rows(dq, acc, fac[kGam * kL + ra] * (o0 * sinv), fac[kGam * kL + ra + 8] * (o1 * sinv));
      zero(acc);  // -gam (dV S^T)
      gemm<kL, true, KP, NP, NT>(acc, su + L::dv, kTile, r0, su + L::s, kVB * KP * 2, k0, 0, 4, lane);
      add_rows(dk, acc, -fac[kGam * kL + ra] * (vinv * sinv), -fac[kGam * kL + ra + 8] * (vinv * sinv));
      zero(acc);  // w (U dS^T)
      gemm<kL, true, KP, NP, NT>(acc, su + L::u, kTile, r0, su + L::ds, kVB * KP * 2, k0, 0, 4, lane);
      add_rows(dk, acc, fac[kW * kL + ra] * (uinv * dinv), fac[kW * kL + ra + 8] * (uinv * dinv));
      float p4[4][4];
      zero(p4);
      gemm<kVB, false, kL, NP, 4>(p4, su + L::dout, kTile, r0, su + L::u, kTile, c0, 0, 4, lane);
      add_rows(dP, p4, o0 * uinv, o1 * uinv);
      zero(p4);
      gemm<kL, true, kL, NP, 4>(p4, su + L::dv, kTile, r0, su + L::u, kTile, c0, 0, 4, lane);
      add_rows(dW, p4, vinv * uinv, vinv * uinv);
    }
    // (dP o D), (dW o D) with the scales of the rows that they meet, one power of two a matrix
    float big[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int t = ra + (e >> 1) * 8, q = c0 + j * 8 + ca + (e & 1);
        const float D = q <= t ? decay_between(G[t], G[q]) : 0.f;
        dP[j][e] = q <= t ? dP[j][e] * D : 0.f;
        dW[j][e] = q < t ? dW[j][e] * D : 0.f;
        big[0] = fmaxf(big[0], fabsf(dP[j][e] * fac[kKInv * kL + q]));
        big[1] = fmaxf(big[1], fabsf(dP[j][e] * fac[kQInv * kL + t]));
        big[2] = fmaxf(big[2], fabsf(dW[j][e] * fac[kKInv * kL + q]));
        big[3] = fmaxf(big[3], fabsf(dW[j][e] * fac[kKInv * kL + t]));
      }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      big[i] = warp_max(big[i]);
      if (lane == 0) most[warp * 4 + i] = big[i];
    }
    __syncthreads();  // the columns are read; the matrices take their place
    Scale sc[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float m = 0.f;
#pragma unroll
      for (int w = 0; w < 8; ++w) m = fmaxf(m, most[w * 4 + i]);
      sc[i] = scale_of(m);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int t = ra + r * 8, q = c0 + j * 8 + ca;
        const float2 ki = *reinterpret_cast<const float2*>(fac + kKInv * kL + q);
        const float kt = fac[kKInv * kL + t], qt = fac[kQInv * kL + t];
        const float x = dP[j][2 * r], y = dP[j][2 * r + 1], z = dW[j][2 * r], w = dW[j][2 * r + 1];
        const float v[4][2] = {{x * ki.x, y * ki.y}, {x * qt, y * qt}, {z * ki.x, w * ki.y}, {z * kt, w * kt}};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t hi, lo;
          split(v[i][0] * sc[i].mul, v[i][1] * sc[i].mul, hi, lo);
          char* at = smem + L::mat + i * NP * kTile + piece_at<kL>(t, q) + (q & 7) * 2;
          *reinterpret_cast<uint32_t*>(at) = hi;
          if (NP == 2) *reinterpret_cast<uint32_t*>(at + kTile) = lo;
        }
      }
    __syncthreads();
    const int mt = warp & 3;
    const uint32_t mat = su + L::mat, ku = su, qu = su + keys_bytes(KP, NP) / 2;
    constexpr int pk = kL * KP * 2;
    float acc[NT][4];
    zero(acc);
    gemm<kL, false, KP, NP, NT>(acc, mat, kTile, r0, ku, pk, k0, 0, mt + 1, lane);
    add_rows(dq, acc, sc[0].inv, sc[0].inv);
    zero(acc);
    gemm<kL, true, KP, NP, NT>(acc, mat + NP * kTile, kTile, r0, qu, pk, k0, mt, 4, lane);
    add_rows(dk, acc, sc[1].inv, sc[1].inv);
    zero(acc);
    gemm<kL, false, KP, NP, NT>(acc, mat + 2 * NP * kTile, kTile, r0, ku, pk, k0, 0, mt + 1, lane);
    add_rows(dk, acc, -sc[2].inv, -sc[2].inv);
    zero(acc);
    gemm<kL, true, KP, NP, NT>(acc, mat + 3 * NP * kTile, kTile, r0, ku, pk, k0, mt, 4, lane);
    add_rows(dk, acc, -sc[3].inv, -sc[3].inv);
    __syncthreads();  // factors and matrices belong to the next head
  }
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    const GdrStride st = which ? a.sdk : a.sdq;
    T* out = (T*)(which ? a.dk : a.dq) + s.b * st.b + hk * st.h + t0 * st.t;
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int t = ra + r * 8, key = k0 + j * 8 + ca;
        if (t >= len || key >= a.K) continue;
        const float x = which ? dk[j][2 * r] : dq[j][2 * r], y = which ? dk[j][2 * r + 1] : dq[j][2 * r + 1];
        if constexpr (sizeof(T) == 2)
          *reinterpret_cast<uint32_t*>(out + t * st.t + key) = pack_bf16(x, y);
        else
          *reinterpret_cast<float2*>(out + t * st.t + key) = make_float2(x, y);
      }
  }
}

// The workspace: keys and records, then what Kept lists.
struct BwdLayout {
  size_t records, S, S_inv, Z, U, U_inv, dots, D, D_inv, dV, dV_inv, dbeta, ends, total;
};
BwdLayout bwd_layout(const GdrArgs& a) {
  const int np = a.dtype ? 1 : 2, KP = a.K <= 64 ? 64 : 128;
  const size_t nrec = (size_t)record_count(a), tiles = (a.V + 15) / 16;
  const size_t rt = nrec * a.H * tiles, st = (nrec + a.N) * a.H * tiles, key_step = (size_t)(KP / 16) * 512;
  BwdLayout l;
  size_t at = nrec * a.HK * keys_bytes(KP, np);
  auto take = [&](size_t n) {
    const size_t here = at;
    at += (n + 255) & ~(size_t)255;
    return here;
  };
  l.records = take(nrec * a.H * record_bytes(true));
  l.S = take(st * 2 * key_step);
  l.S_inv = take(st * 16);
  l.Z = take(rt * 4096);
  l.U = take(rt * np * 2048);
  l.U_inv = take(rt * 16);
  l.dots = take(rt * 256);
  l.D = take(rt * np * key_step);
  l.D_inv = take(rt * 16);
  l.dV = take(rt * np * 2048);
  l.dV_inv = take(rt * 16);
  l.dbeta = take(rt * 256);
  l.ends = take(rt * 16);
  l.total = at;
  return l;
}

template <typename T, int KP, int TN>
cudaError_t launch_back(const GdrArgs& a, const char* keys, const char* records, const Kept& kept, cudaStream_t stream) {
  constexpr int smem = Stage<T, KP, TN, true>::bytes;
  const auto kernel = gdr_back_kernel<T, KP, TN>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const int tiles = (a.V + 15) / 16;
  kernel<<<dim3((tiles + TN - 1) / TN, a.H, a.N), 32 * kQuarter * TN, smem, stream>>>(a, keys, records, kept);
  return cudaGetLastError();
}

template <typename T, int KP>
cudaError_t backward(const GdrArgs& a, char* ws, cudaStream_t stream) {
  const BwdLayout l = bwd_layout(a);
  char* records = ws + l.records;
  Kept k;
  k.S = (uint4*)(ws + l.S), k.S_inv = (float*)(ws + l.S_inv), k.Z = (float4*)(ws + l.Z);
  k.U = (uint4*)(ws + l.U), k.U_inv = (float*)(ws + l.U_inv), k.dots = (float*)(ws + l.dots);
  k.D = (uint4*)(ws + l.D), k.D_inv = (float*)(ws + l.D_inv), k.dV = (uint4*)(ws + l.dV);
  k.dV_inv = (float*)(ws + l.dV_inv), k.dbeta = (float*)(ws + l.dbeta), k.ends = (float*)(ws + l.ends);
  cudaError_t e = launch_prep<T, KP, true>(a, ws, records, stream);
  if (e != cudaSuccess) return e;
  e = launch_walk<T, KP, true>(a, ws, records, k, stream);
  if (e != cudaSuccess) return e;
  const int tn = tiles_a_block<T>(a);
  if constexpr (sizeof(T) == 2)
    if (tn == 4) e = launch_back<T, KP, 4>(a, ws, records, k, stream);
  if (tn != 4) e = tn == 2 ? launch_back<T, KP, 2>(a, ws, records, k, stream) : launch_back<T, KP, 1>(a, ws, records, k, stream);
  if (e != cudaSuccess) return e;
  const auto kernel = gdr_grad_kernel<T, KP>;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, GradStage<T, KP>::bytes);
  if (e != cudaSuccess) return e;
  kernel<<<dim3((unsigned)record_count(a), a.HK), kGradThreads, GradStage<T, KP>::bytes, stream>>>(a, ws, records, k);
  return cudaGetLastError();
}

}  // namespace
}  // namespace gdr

size_t gdr_bwd_workspace_bytes(const GdrArgs& a) { return gdr::bwd_layout(a).total; }

cudaError_t launch_gdr_bwd(const GdrArgs& a, void* ws, cudaStream_t stream) {
  char* w = (char*)ws;
  if (a.dtype)
    return a.K <= 64 ? gdr::backward<__nv_bfloat16, 64>(a, w, stream) : gdr::backward<__nv_bfloat16, 128>(a, w, stream);
  return a.K <= 64 ? gdr::backward<float, 64>(a, w, stream) : gdr::backward<float, 128>(a, w, stream);
}

}  // namespace mlstm
