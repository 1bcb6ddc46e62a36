// Gradients of the gated delta rule (formulas, precision and layouts: gdr_tile.cuh).
//
// Five kernels: what does not depend on the state (gdr_prep_kernel), the forward pass again, which keeps
// the states (gdr_walk_kernel with GRAD), the pass backward over the chunks with dS in registers, which
// gives dV and everything that needs fp32 accuracy (gdr_back_kernel), and for all chunks at once the
// gradients of q and k (gdr_grad_kernel) and of the gates (gdr_gates_kernel):
//     dQ = gam (dO S^T) + (dP o D) K            dP = dO U^T (lower)   dW = dV U^T (strictly lower)
//     dK = -gam (dV S^T) + w (U dS^T) + (dP o D)^T Q - (dW o D) K - (dW o D)^T K
// with S at the chunk's start and dS at its end.
#include "gdr_walk.cuh"

namespace mlstm {
namespace gdr {
namespace {

// A block takes 16 TN value columns of one value head of one sequence, chunks from the last to the first: a
// chain as the forward pass's, with six products.  64 heads of 128 x 128, 2048 bf16 tokens, TN = 4: 300 us, 9.4 us
// a chunk, issue slots 40 % taken, tensor pipes 23 %.
template <typename T, int KP, int TN>
__global__ void __launch_bounds__(kWalkThreads<TN>, kWalkBlocks<T, KP, TN>) gdr_back_kernel(const GdrArgs a, const char* keys,
                                                                      const char* records, const Kept kept) {
  using L = Stage<T, KP, TN, true>;
  constexpr int NP = L::NP, NK = kept_parts<T>(), KS = KP / 64;
  // In exchange: dS, then beta dU in its place; dO by P's scale; gam dV; gam dO.
  constexpr int fy = L::fs;
  extern __shared__ __align__(128) char smem[];
  const int n = blockIdx.z, h = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int local = warp / kQuarter, w = (warp + local) % kQuarter, tile = blockIdx.x * TN + local, tiles = (a.V + 15) / 16;
  const int col0 = blockIdx.x * 16 * TN, v0 = tile * 16, cols = min(16, a.V - v0);
  const bool live = tile < tiles;
  const Seq s = sequence(a, n);
  const int chunks = (int)((s.len + kL - 1) / kL);
  const size_t state = ((size_t)n * a.H + h) * a.K * a.V;
  const int ra = lane >> 2, ca = 2 * (lane & 3);
  char* ex = smem + L::tiles + local * L::tile;
  float* inv = reinterpret_cast<float*>(ex + L::inv);

  constexpr bool copies = kCopyWarps<TN> == 0;
  if (!copies && warp >= kQuarter * TN) {
    copy_ahead<T, KP, TN, true, true>(a, s, chunks, h, col0, keys, records, smem_u32(smem));
    return;
  }

  float D[2 * KS][4];
#pragma unroll
  for (int j = 0; j < 2 * KS; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int col = ra + (e >> 1) * 8, key = w * (KP / 4) + 8 * j + ca + (e & 1);
      D[j][e] = a.dS && col < cols && key < a.K ? a.dS[state + (size_t)key * a.V + v0 + col] : 0.f;
    }
  if (copies && chunks > 0) fetch_all<T, KP, TN, true>(a, s, chunks - 1, h, col0, keys, records, smem_u32(smem));
  for (int c = chunks - 1; c >= 0; --c) {
    const long long rec = s.slot + c;
    const size_t base = ((size_t)rec * a.H + h) * tiles + tile;
    char *st = smem + L::at(c), *mats = smem + L::mats(c);
    const float* fac = reinterpret_cast<const float*>(st + L::factors);
    {
      const Scale sc = tile_scale(D);
      give<KS, 2>(D, sc, ex + L::fs, inv, w, lane);
      if (live) {  // dS for the gradients of k, and <dS, S> with the state that the forward pass left here
        const size_t after = ((size_t)(rec + n + 1) * a.H + h) * tiles + tile;
        float end = 0.f;
#pragma unroll
        for (int i = 0; i < KS; ++i) {
          uint4 hi, lo;
          split_a(D[2 * i], D[2 * i + 1], sc.mul, hi, lo);
          char* at = kept.D + base * NK * 16 * KP * 2;
          keep16<KP>(at, (w * KS + i) * 16, hi, lane);
          if (NK == 2) keep16<KP>(at + 16 * KP * 2, (w * KS + i) * 16, lo, lane);
          const char* state_at = kept.S + after * 2 * 16 * KP * 2;
          const uint4 sh = kept16<KP>(state_at, (w * KS + i) * 16, lane);
          const uint4 sl = kept16<KP>(state_at + 16 * KP * 2, (w * KS + i) * 16, lane);
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
    if (copies) cp_wait<0>();
    __syncthreads();  // the chunk has come, dS is in exchange, and nobody is in the chunk behind
    if (copies && !L::ahead) {
      fetch_matrices<true, TN>(a, rec, h, records, smem_u32(mats));
      cp_commit();
    }
    if (copies && L::chunks == 2) {
      if (c > 0)
        fetch_all<T, KP, TN, true>(a, s, c - 1, h, col0, keys, records, smem_u32(smem));
      else
        cp_commit();
    }
    // this quarter's share of dO by P's scale, and gam dO
    float x[2][4], y[2][4];
    {
      float d[2][4];
      read_columns<T, L::row>(d, st + L::dout + w * 16 * L::row + local * 16 * (int)sizeof(T), lane);
      if (live) keep_tokens<NK>(kept.dO, kept.dO_inv, base, d, tile_scale(d), w, lane);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float2 pi = factor(fac + kPInv * kL, w * 16, j, lane), gq = factor(fac + kGQ * kL, w * 16, j, lane);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[j][e] = d[j][e] * (e & 1 ? pi.y : pi.x);
          y[j][e] = d[j][e] * (e & 1 ? gq.y : gq.x);
        }
      }
      give<1, NP>(x, tile_scale(x), ex + L::fu, inv + 2 * kQuarter, w, lane);
      give<1, 2>(y, tile_scale(y), ex + L::fz, inv + 4 * kQuarter, w, lane);
    }
    // dU = w (K dS) + P^T dO
    by_keys<KP, NP, false, false>(x, y, ex + L::fs, inv, smem_u32(st), 0u, w, lane);
    float2 zp[2][2];  // Z' of this quarter: [tile of 8 tokens][row r or r + 8]
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int r = 0; r < 2; ++r)
        zp[j][r] = live ? *reinterpret_cast<const float2*>(kept.Z + (base * 16 + ra + 8 * r) * kL + w * 16 + 8 * j + ca)
                        : make_float2(0.f, 0.f);
    if (copies && !L::ahead) cp_wait<L::chunks == 2 ? 1 : 0>();
    if (L::ahead)
      tile_barrier(local);  // dO is in exchange, dS has been read
    else
      __syncthreads();  // and R and P have come
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
    give<1, 2>(y, tile_scale(y), ex + fy, inv + kQuarter, w, lane);
    tile_barrier(local);  // beta dU is in exchange
    // dY = dU + R^T (beta dU), dV = beta dY
    by_tokens<true, 2, 2>(y, ex + fy, inv + kQuarter, smem_u32(mats), w, lane);
    char* vt = st + L::v + w * 16 * L::row + local * 16 * (int)sizeof(T);
    {
      float dot[4], v[2][4];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float2 be = factor(fac + kBeta * kL, w * 16, j, lane), gk = factor(fac + kGK * kL, w * 16, j, lane);
#pragma unroll
        for (int e = 0; e < 4; ++e) x[j][e] += y[j][e];
        dot[2 * j] = x[j][0] * zp[j][0].x + x[j][2] * zp[j][1].x;
        dot[2 * j + 1] = x[j][1] * zp[j][0].y + x[j][3] * zp[j][1].y;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[j][e] *= e & 1 ? be.y : be.x;
          y[j][e] = x[j][e] * (e & 1 ? -gk.y : -gk.x);
        }
      }
      give<1, 2>(y, tile_scale(y), ex + L::fw, inv + 3 * kQuarter, w, lane);
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
        keep_tokens<NK>(kept.dV, kept.dV_inv, base, x, tile_scale(x), w, lane);
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
      if (copies) fetch_all<T, KP, TN, true>(a, s, c - 1, h, col0, keys, records, smem_u32(smem));
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
constexpr int kGradThreads = 512;
constexpr int kVB = 64;  // value columns at a time: four kept tiles

template <typename T, int KP>
struct GradStage {
  static constexpr int NP = sizeof(T) == 4 ? 2 : 1;
  // behind k and q, once or twice, as [value][token or key]: dO, dV, U, S, dS
  static constexpr int cols = keys_bytes(KP, NP);
  static constexpr int dout = 0;
  static constexpr int dv = dout + NP * kTile;
  static constexpr int u = dv + NP * kTile;
  static constexpr int s = u + NP * kTile;
  static constexpr int ds = s + NP * kVB * KP * 2;
  // dP o D by k's and q's scales and dW o D by k's, rows and columns, take the place of a head's last columns
  static constexpr int mats = 4 * NP * kTile;
  static constexpr int block = ds + NP * kVB * KP * 2 > mats ? ds + NP * kVB * KP * 2 : mats;
  // factors and the operands' scales [5][4 tiles][4], twice; the matrices' largest values [4][4 warps][64], then
  // their scales [4][64] in the place of the first warp's
  static constexpr int small = 2 * kFactorBytes + 2 * 5 * 16 * 4 + 4 * 4 * kL * 4;
  static constexpr int blocks = cols + 2 * block + small <= 227 * 1024 ? 2 : 1;
  static constexpr int bytes = cols + blocks * block + small;
  static_assert(bytes <= 227 * 1024, "a block's shared memory");
};

// acc[j] += A B (or = A B where FRESH) over one k step: A fragments (16 rows from r0) of a tile [k][row] (K_ROWS)
// or [row][k] with AC columns, B of a tile [k][n] with BC columns from c0.  Two parts each where NP is 2 (planes
// pa and pb bytes further on).
template <bool FRESH, bool K_ROWS, int AC, int BC, int NP, int NT>
__device__ __forceinline__ void grad_step(float (&acc)[NT][4], uint32_t at, int pa, int r0, uint32_t bt, int pb, int c0, int kk,
                                          int lane) {
  uint4 a[2];
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    uint32_t r[4];
    if constexpr (K_ROWS)
      ldsm4t(r, at + p * pa + piece_at<AC>(kk * 16 + at_row(lane), r0 + at_col(lane)));
    else
      ldsm4(r, at + p * pa + piece_at<AC>(r0 + bt_row(lane), kk * 16 + bt_col(lane)));
    a[p] = make_uint4(r[0], r[1], r[2], r[3]);
  }
  step<FRESH, NT, NP, NP>(acc, a[0], a[NP - 1], [&](uint32_t (&r)[4], int j, int plane) {
    ldsm4t(r, bt + plane * pb + piece_at<BC>(kk * 16 + bt_row(lane), c0 + j * 8 + bt_col(lane)));
  });
}
template <int N>
struct Columns {
  static constexpr int value = N;
};
// sum += acc times a factor of the row (the lane's rows r and r + 8)
template <int NT>
__device__ __forceinline__ void add_rows(float (&sum)[NT][4], const float (&acc)[NT][4], float f0, float f1) {
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) sum[j][e] = fmaf(acc[j][e], e < 2 ? f0 : f1, sum[j][e]);
}

// One block for each chunk and key head; the value heads that share it follow one another and their
// shares add up in registers.  Warp (t, n) of 4 x 4 has 16 tokens and a quarter of the keys (or of the other
// token).  The kept operands come 64 value columns at a time, the next ones while these are in work.
// 2048 chunks of 128 x 128: 177 us.  What bounds it is reading the operands' fragments, and the barriers of a block
// that has its SM alone.  (Blocks that stay and fetch the next chunk meanwhile took 7 us more: registers ran out.)
template <typename T, int KP>
__global__ void __launch_bounds__(kGradThreads) gdr_grad_kernel(const GdrArgs a, const char* keys, const char* records,
                                                                const Kept kept) {
  using L = GradStage<T, KP>;
  constexpr int NP = L::NP, NK = kept_parts<T>(), NT = KP / 32;
  extern __shared__ __align__(128) char smem[];
  float* const factors = reinterpret_cast<float*>(smem + L::cols + L::blocks * L::block);  // [2][kFactors][64]
  float* const scales = factors + 2 * kFactors * kL;                                       // [2][operand][tile][quarter]
  float* const most = scales + 2 * 5 * 16;  // [matrix][warp][64], then [matrix][64]
  int n, c;
  Seq s;
  if (!find_chunk(a, blockIdx.x, &n, &s, &c)) return;
  const int hk = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, tiles = (a.V + 15) / 16;
  const long long rec = blockIdx.x, t0 = s.lo + (long long)c * kL;
  const int len = (int)min((long long)kL, s.len - (long long)c * kL);
  const uint32_t su = smem_u32(smem);
  const int mt = warp & 3, nq = warp >> 2, r0 = mt * 16, k0 = nq * (KP / 4), c0 = nq * 16;
  const int ra = r0 + (lane >> 2), ca = 2 * (lane & 3);
  const int group = a.H / a.HK, parts = (tiles + 3) / 4, total = group * parts;

  const char* kq = keys + (rec * a.HK + hk) * keys_bytes(KP, NP);
  for (int i = tid; i < keys_bytes(KP, NP) / 16; i += kGradThreads) cp_async16(su + i * 16, kq + i * 16, true);

  // the columns of step i: value head hk group + i / parts, tiles 4 (i % parts) ..
  auto fetch = [&](int i) {
    const int h = hk * group + i / parts, first = i % parts * 4;
    const size_t base = ((size_t)rec * a.H + h) * tiles + first, sbase = ((size_t)(rec + n) * a.H + h) * tiles + first;
    const uint32_t to = su + L::cols + (L::blocks == 2 ? (i & 1) * L::block : 0);
    const int live = min(4, tiles - first);
    // PARTS: parts in memory, of which NP are read
    auto operand = [&](const char* from, size_t at, int PARTS, int at_smem, int cols) {
      const int per = 16 * cols * 2 / 16;  // pieces of a tile's part, 128 to a block of 64 columns
      for (int e = tid; e < 4 * NP * per; e += kGradThreads) {
        const int x = e % per, part = e / per % NP, tile = e / (per * NP);
        const bool in = tile < live;
        cp_async16(to + at_smem + part * kVB * cols * 2 + (x / 128 * kVB + tile * 16) * 128 + x % 128 * 16,
                   from + ((at + (in ? tile : 0)) * PARTS + part) * 16 * cols * 2 + x * 16, in);
      }
    };
    operand(kept.dO, base, NK, L::dout, kL);
    operand(kept.dV, base, NK, L::dv, kL);
    operand(kept.U, base, NK, L::u, kL);
    operand(kept.S, sbase, 2, L::s, KP);
    operand(kept.D, base, NK, L::ds, KP);
    if (tid < 5 * 4) {  // the scales, a tile's four a thread
      const float* invs[5] = {kept.dO_inv, kept.dV_inv, kept.U_inv, kept.S_inv, kept.D_inv};
      const int of = tid >> 2, tile = tid & 3;
      const bool in = tile < live;
      cp_async16(smem_u32(scales + ((i & 1) * 5 + of) * 16 + tile * 4),
                 invs[of] + ((of == 3 ? sbase : base) + (in ? tile : 0)) * kQuarter, in);
    }
    if (i % parts == 0) {
      const char* fin = records + (rec * a.H + h) * record_bytes(true) + 4 * kTile;
      const uint32_t to_fac = smem_u32(factors + (i / parts & 1) * kFactors * kL);
      for (int e = tid; e < kFactorBytes / 16; e += kGradThreads) cp_async16(to_fac + e * 16, fin + e * 16, true);
    }
    cp_commit();
  };

  float dq[NT][4], dk[NT][4], dP[2][4], dW[2][4];
  zero(dq), zero(dk);
  fetch(0);
  for (int i = 0; i < total; ++i) {
    const int part = i % parts;
    cp_wait<0>();
    __syncthreads();  // these columns have come; the ones before, and a head's matrices and factors, are done with
    if (L::blocks == 2 && i + 1 < total) fetch(i + 1);
    const float* fac = factors + (i / parts & 1) * kFactors * kL;
    if (part == 0) zero(dP), zero(dW);
    const uint32_t st = su + L::cols + (L::blocks == 2 ? (i & 1) * L::block : 0);
    constexpr int ps = kVB * KP * 2;
    const float* sc = scales + (i & 1) * 5 * 16;
    const float *so = sc, *sv = sc + 16, *su_ = sc + 32, *ss = sc + 48, *sd = sc + 64;
    // Every tile of 16 columns is a product from zero, scaled on its way into the fp32 sum: the scales of dO, S and
    // the others may lie any powers apart from tile to tile.  (Fragments that were scaled to share one sum took
    // 171 us and lost what lay 2^-25 below the largest product of two scales.)  f0, f1: further factors of the
    // rows.  Two tiles in flight with 128 keys, which have twice the sums (four: spills, 192 us; one: 182).
    auto over_values = [&](auto& sum, auto bc, int A, const float* fa, int B, int pb, int c0, const float* fb, float f0,
                           float f1) {
#pragma unroll(KP == 128 ? 2 : 4)
      for (int kk = 0; kk < 4; ++kk) {
        float acc[sizeof(sum) / sizeof(sum[0])][4];
        grad_step<true, true, kL, decltype(bc)::value, NP>(acc, st + A, kTile, r0, st + B, pb, c0, kk, lane);
        const float f = fminf(fa[kk * 4 + mt] * fb[kk * 4 + nq], 0x1p127f);  // (a zero times infinity is none)
        add_rows(sum, acc, f * f0, f * f1);
      }
    };
    const Columns<KP> by_key;
    const Columns<kL> by_token;
    const float g0 = fac[kGam * kL + ra], g1 = fac[kGam * kL + ra + 8];
    over_values(dq, by_key, L::dout, so, L::s, ps, k0, ss, g0, g1);                                     // gam (dO S^T)
    over_values(dk, by_key, L::dv, sv, L::s, ps, k0, ss, -g0, -g1);                                     // -gam (dV S^T)
    over_values(dk, by_key, L::u, su_, L::ds, ps, k0, sd, fac[kW * kL + ra], fac[kW * kL + ra + 8]);  // w (U dS^T)
    if (c0 <= r0) {  // the other token's quarter is not behind this one
      over_values(dP, by_token, L::dout, so, L::u, kTile, c0, su_, 1.f, 1.f);
      over_values(dW, by_token, L::dv, sv, L::u, kTile, c0, su_, 1.f, 1.f);
    }
    if (part == parts - 1) {
      // (dP o D), (dW o D) with the scales of the rows that they meet; each row of the four products has a power of
      // two of its own: 0, 2 are read by rows (tokens), 1, 3 by columns
      float row[2][2] = {{0.f, 0.f}, {0.f, 0.f}}, column[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
      const float2* G = reinterpret_cast<const float2*>(fac + kG * kL);
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int t = ra + (e >> 1) * 8, q = c0 + j * 8 + ca + (e & 1), at = 2 * j + (e & 1);
          const float D = q <= t ? decay_between(G[t], G[q]) : 0.f;
          dP[j][e] = q <= t ? dP[j][e] * D : 0.f;
          dW[j][e] = q < t ? dW[j][e] * D : 0.f;
          row[0][e >> 1] = fmaxf(row[0][e >> 1], fabsf(dP[j][e] * fac[kKInv * kL + q]));
          column[0][at] = fmaxf(column[0][at], fabsf(dP[j][e] * fac[kQInv * kL + t]));
          row[1][e >> 1] = fmaxf(row[1][e >> 1], fabsf(dW[j][e] * fac[kKInv * kL + q]));
          column[1][at] = fmaxf(column[1][at], fabsf(dW[j][e] * fac[kKInv * kL + t]));
        }
#pragma unroll
      for (int m = 0; m < 2; ++m) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          for (int d = 1; d < 4; d *= 2) row[m][x] = fmaxf(row[m][x], __shfl_xor_sync(0xffffffffu, row[m][x], d));
          if ((lane & 3) == 0) most[(2 * m * 4 + nq) * kL + ra + 8 * x] = row[m][x];
        }
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          for (int d = 4; d < 32; d *= 2) column[m][x] = fmaxf(column[m][x], __shfl_xor_sync(0xffffffffu, column[m][x], d));
          if (lane < 4) most[((2 * m + 1) * 4 + mt) * kL + c0 + (x >> 1) * 8 + ca + (x & 1)] = column[m][x];
        }
      }
      __syncthreads();  // the columns are read; the matrices take their place
      if (tid < 4 * kL) {
        float* at = most + (tid / kL * 4) * kL + tid % kL;
        *at = scale_of(fmaxf(fmaxf(at[0], at[kL]), fmaxf(at[2 * kL], at[3 * kL]))).inv;
      }
      __syncthreads();
      // the inverses, and the powers themselves
      auto inv = [&](int m, int x) { return most[m * 4 * kL + x]; };
      auto mul = [&](int m, int x) { return __uint_as_float((254u << 23) - __float_as_uint(inv(m, x))); };
      char* mats = smem + (st - su);
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int t = ra + r * 8;
        const float kt = fac[kKInv * kL + t], qt = fac[kQInv * kL + t], m0 = mul(0, t), m2 = mul(2, t);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int q = c0 + j * 8 + ca;
          const float2 ki = *reinterpret_cast<const float2*>(fac + kKInv * kL + q);
          const float x = dP[j][2 * r], y = dP[j][2 * r + 1], z = dW[j][2 * r], w = dW[j][2 * r + 1];
          const float v[4][2] = {{x * ki.x * m0, y * ki.y * m0},
                                 {x * qt * mul(1, q), y * qt * mul(1, q + 1)},
                                 {z * ki.x * m2, w * ki.y * m2},
                                 {z * kt * mul(3, q), w * kt * mul(3, q + 1)}};
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            uint32_t hi, lo;
            split(v[m][0], v[m][1], hi, lo);
            char* at = mats + m * NP * kTile + piece_at<kL>(t, q) + (q & 7) * 2;
            *reinterpret_cast<uint32_t*>(at) = hi;
            if (NP == 2) *reinterpret_cast<uint32_t*>(at + kTile) = lo;
          }
        }
      }
      __syncthreads();
      const uint32_t ku = su, qu = su + keys_bytes(KP, NP) / 2;
      constexpr int pk = kL * KP * 2, mat = NP * kTile;
      float acc[NT][4];
      zero(acc);
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
        if (kk <= mt) grad_step<false, false, kL, KP, NP>(acc, st, kTile, r0, ku, pk, k0, kk, lane);
      add_rows(dq, acc, inv(0, ra), inv(0, ra + 8));
      zero(acc);
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
        if (kk >= mt) grad_step<false, true, kL, KP, NP>(acc, st + mat, kTile, r0, qu, pk, k0, kk, lane);
      add_rows(dk, acc, inv(1, ra), inv(1, ra + 8));
      zero(acc);
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
        if (kk <= mt) grad_step<false, false, kL, KP, NP>(acc, st + 2 * mat, kTile, r0, ku, pk, k0, kk, lane);
      add_rows(dk, acc, -inv(2, ra), -inv(2, ra + 8));
      zero(acc);
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
        if (kk >= mt) grad_step<false, true, kL, KP, NP>(acc, st + 3 * mat, kTile, r0, ku, pk, k0, kk, lane);
      add_rows(dk, acc, -inv(3, ra), -inv(3, ra + 8));
    }
    if (L::blocks == 1 && i + 1 < total) {
      __syncthreads();
      fetch(i + 1);
    }
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

// dg: what follows a token in its chunk, and the state's share at the chunk's end; dbeta.  One warp a chunk
// and value head, two tokens a lane; sums over the tiles in order.  6 us for 2048 chunks.
__global__ void __launch_bounds__(128) gdr_gates_kernel(const GdrArgs a, long long records, const Kept kept) {
  const long long item = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31, tiles = (a.V + 15) / 16;
  if (item >= records * a.H) return;
  const long long rec = item / a.H;
  const int h = (int)(item % a.H);
  int n, c;
  Seq s;
  if (!find_chunk(a, rec, &n, &s, &c)) return;
  const size_t base = (size_t)item * tiles;
  float x[2] = {0.f, 0.f}, b[2] = {0.f, 0.f}, end = 0.f;
#pragma unroll 4
  for (int i = 0; i < tiles; ++i) {
    const float2 d = *reinterpret_cast<const float2*>(kept.dots + (base + i) * kL + 2 * lane);
    const float2 e = *reinterpret_cast<const float2*>(kept.dbeta + (base + i) * kL + 2 * lane);
    const float4 f = *reinterpret_cast<const float4*>(kept.ends + (base + i) * kQuarter);
    x[0] += d.x, x[1] += d.y, b[0] += e.x, b[1] += e.y, end += (f.x + f.y) + (f.z + f.w);
  }
  double sum = (double)x[0] + x[1];
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const double y = __shfl_down_sync(0xffffffffu, sum, d);
    if (lane + d < 32) sum += y;
  }
  const int len = (int)min((long long)kL, s.len - (long long)c * kL);
  const size_t out = ((size_t)s.b * a.H + h) * a.T + s.lo + (long long)c * kL + 2 * lane;
  if (2 * lane < len) a.dg[out] = (float)(sum + end), a.dbeta[out] = b[0];
  if (2 * lane + 1 < len) a.dg[out + 1] = (float)(sum - x[0] + end), a.dbeta[out + 1] = b[1];
}

// The workspace: keys and records, then what Kept lists.
struct BwdLayout {
  size_t records, S, S_inv, Z, U, U_inv, dots, D, D_inv, dV, dV_inv, dO, dO_inv, dbeta, ends, total;
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
  l.dO = take(rt * np * 2048);
  l.dO_inv = take(rt * 16);
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
  kernel<<<dim3((tiles + TN - 1) / TN, a.H, a.N), kWalkThreads<TN>, smem, stream>>>(a, keys, records, kept);
  return cudaGetLastError();
}

template <typename T, int KP>
cudaError_t backward(const GdrArgs& a, char* ws, cudaStream_t stream) {
  const BwdLayout l = bwd_layout(a);
  char *keys = ws, *records = ws + l.records;
  Kept k;
  k.S = ws + l.S, k.S_inv = (float*)(ws + l.S_inv), k.Z = (float*)(ws + l.Z);
  k.U = ws + l.U, k.U_inv = (float*)(ws + l.U_inv), k.dots = (float*)(ws + l.dots);
  k.D = ws + l.D, k.D_inv = (float*)(ws + l.D_inv), k.dV = ws + l.dV;
  k.dV_inv = (float*)(ws + l.dV_inv), k.dO = ws + l.dO, k.dO_inv = (float*)(ws + l.dO_inv);
  k.dbeta = (float*)(ws + l.dbeta), k.ends = (float*)(ws + l.ends);
  cudaError_t e = launch_prep<T, KP, true>(a, keys, records, stream);
  if (e != cudaSuccess) return e;
  e = launch_walk<T, KP, true>(a, keys, records, k, stream);
  if (e != cudaSuccess) return e;
  const int tn = tiles_a_block<T, KP, true>(a);
  if (tn == 1) e = launch_back<T, KP, 1>(a, keys, records, k, stream);
  if constexpr (kWalkOf<T, KP, true>(2))
    if (tn == 2) e = launch_back<T, KP, 2>(a, keys, records, k, stream);
  if constexpr (kWalkOf<T, KP, true>(4))
    if (tn == 4) e = launch_back<T, KP, 4>(a, keys, records, k, stream);
  if (e != cudaSuccess) return e;
  const auto kernel = gdr_grad_kernel<T, KP>;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, GradStage<T, KP>::bytes);
  if (e != cudaSuccess) return e;
  kernel<<<dim3((unsigned)record_count(a), a.HK), kGradThreads, GradStage<T, KP>::bytes, stream>>>(a, keys, records, k);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const long long items = record_count(a) * a.H;
  gdr_gates_kernel<<<(unsigned)((items + 3) / 4), 128, 0, stream>>>(a, record_count(a), k);
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
