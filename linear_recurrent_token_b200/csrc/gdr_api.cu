// C entry points of the gated delta rule and of the root-mean-square norm (declared in
// include/mlstm.h): host-side validation, workspace layout and kernel dispatch.  No entry point
// allocates, frees or synchronises.
#include "host_check.h"
#include "kernels.h"
#include "mlstm.h"

namespace {

using namespace mlstm;

GdrStride to_stride(mlstm_gdr_stride_t s) { return GdrStride{s.b, s.h, s.t}; }

// elements from the first to behind the last one of [B, H, T, D]; 0 for an empty tensor
size_t span(mlstm_gdr_stride_t s, long long B, long long H, long long T, long long D) {
  if (B == 0 || H == 0 || T == 0) return 0;
  return (size_t)((B - 1) * s.b + (H - 1) * s.h + (T - 1) * s.t + D);
}

// strides are in range (no index of [B, H, T] leaves 2^50) and keep `unit` elements' alignment;
// that of an axis with one element is never used
bool strides_ok(mlstm_gdr_stride_t s, long long B, long long H, long long T, int unit) {
  const long long st[] = {s.b, s.h, s.t}, n[] = {B, H, T};
  for (int i = 0; i < 3; ++i)
    if (n[i] > 1 && (st[i] < 0 || st[i] > (1LL << 50) / (n[i] - 1) || st[i] % unit)) return false;
  return true;
}

// distinct elements of [B, H, T, D] lie apart: by ascending stride, each axis steps over those below
bool apart(mlstm_gdr_stride_t s, long long B, long long H, long long T, long long D) {
  if (B == 0 || H == 0 || T == 0) return true;
  long long st[3] = {s.b, s.h, s.t}, n[3] = {B, H, T};
  for (int i = 0; i < 3; ++i)
    for (int j = i + 1; j < 3; ++j)
      if (st[j] < st[i] || (st[j] == st[i] && n[j] < n[i])) {
        const long long a = st[i], b = n[i];
        st[i] = st[j], n[i] = n[j], st[j] = a, n[j] = b;
      }
  long long reach = D;  // elements that the axes so far take up
  for (int i = 0; i < 3; ++i) {
    if (n[i] <= 1) continue;
    if (st[i] < reach) return false;
    reach += (n[i] - 1) * st[i];
  }
  return true;
}

struct GdrShape {
  int es, unit;  // bytes of an element, elements in 16 bytes
  long long N;
  bool any;  // there are tokens
  bool chunk;
};

bool sizes_ok(int B, int HK, int H, int K, int V) {
  if (B < 0 || HK < 0 || H < 0 || K < 8 || K % 8 || K > 256 || V < 8 || V % 8 || V > (1 << 20)) return false;
  if ((HK == 0) != (H == 0) || (HK > 0 && H % HK)) return false;
  return B <= 65535 && H <= 65535;
}

mlstm_status_t check_gdr(const mlstm_gdr_params_t* p, bool backward, GdrShape* s) {
  if (!p) return MLSTM_ERR_NULL;
  if (p->dtype != MLSTM_F32 && p->dtype != MLSTM_BF16) return MLSTM_ERR_DTYPE;
  if (!sizes_ok(p->B, p->HK, p->H, p->K, p->V) || p->T < 0 || p->T > (1 << 30)) return MLSTM_ERR_SHAPE;
  if (p->num_seqs < 0 || p->num_seqs > 65535 || (p->num_seqs > 0 && p->B != 1)) return MLSTM_ERR_SHAPE;
  if (p->mode != MLSTM_GDR_AUTO && p->mode != MLSTM_GDR_RECURRENT && p->mode != MLSTM_GDR_CHUNK) return MLSTM_ERR_SHAPE;
  s->es = p->dtype == MLSTM_BF16 ? 2 : 4;
  s->unit = 16 / s->es;
  s->N = p->num_seqs > 0 ? p->num_seqs : p->B;
  s->any = p->B > 0 && p->H > 0 && p->T > 0;
  if ((long long)p->B * p->T > (1LL << 36)) return MLSTM_ERR_SHAPE;  // chunks are counted in 32 bits
  s->chunk = false;
  if (backward || p->mode == MLSTM_GDR_CHUNK) {
    if (!gdr_chunk_supported(p->K)) return MLSTM_ERR_SHAPE;
    s->chunk = true;
  } else if (p->mode == MLSTM_GDR_AUTO) {
    s->chunk = gdr_chunk_supported(p->K) && p->T >= kGdrChunkFrom && p->T >= (long long)kGdrChunkAverage * p->num_seqs;
  }
  if (!strides_ok(p->q, p->B, p->HK, p->T, s->unit) || !strides_ok(p->k, p->B, p->HK, p->T, s->unit) ||
      !strides_ok(p->v, p->B, p->H, p->T, s->unit) || !strides_ok(p->o, p->B, p->H, p->T, s->unit) ||
      !strides_ok(p->g, p->B, p->H, p->T, 1) || !strides_ok(p->beta, p->B, p->H, p->T, 1))
    return MLSTM_ERR_SHAPE;
  return MLSTM_OK;
}

GdrArgs gdr_args(const mlstm_gdr_params_t* p, const GdrShape& s) {
  GdrArgs a = {};
  a.N = (int)s.N, a.HK = p->HK, a.H = p->H, a.T = p->T, a.K = p->K, a.V = p->V;
  a.dtype = p->dtype == MLSTM_BF16 ? 1 : 0;
  a.packed = p->num_seqs > 0 ? 1 : 0;
  a.wait = p->wait_limit_cycles > 0 ? p->wait_limit_cycles : 0;
  a.sq = to_stride(p->q), a.sk = to_stride(p->k), a.sv = to_stride(p->v);
  a.sg = to_stride(p->g), a.sb = to_stride(p->beta), a.so = to_stride(p->o);
  return a;
}

mlstm_status_t done(cudaError_t e) { return e == cudaSuccess ? MLSTM_OK : MLSTM_ERR_CUDA; }

// outs against ins and against one another; exact: an output may equal this input's address
struct Out {
  Range r;
  const void* same;
};
bool clash(const Range* ins, int ni, const Out* outs, int no) {
  for (int i = 0; i < no; ++i) {
    for (int j = 0; j < ni; ++j)
      if (overlaps(outs[i].r, ins[j]) && !(outs[i].same && outs[i].same == ins[j].p && outs[i].r.p == ins[j].p))
        return true;
    for (int j = 0; j < i; ++j)
      if (overlaps(outs[i].r, outs[j].r)) return true;
  }
  return false;
}

}  // namespace

extern "C" {

size_t mlstm_gdr_fwd_workspace_size(const mlstm_gdr_params_t* p) {
  GdrShape s;
  if (check_gdr(p, false, &s) != MLSTM_OK || !s.chunk || !s.any) return 0;
  return gdr_chunk_workspace_bytes(gdr_args(p, s));
}

mlstm_status_t mlstm_gdr_fwd(const mlstm_gdr_params_t* p, const void* q, const void* k, const void* v, const float* g,
                             const float* beta, const float* S0, const int* seq_offsets, void* o, float* S_out,
                             void* workspace, size_t workspace_bytes, mlstm_stream_t stream) {
  GdrShape s;
  mlstm_status_t st = check_gdr(p, false, &s);
  if (st != MLSTM_OK) return st;
  if (!apart(p->o, p->B, p->H, p->T, p->V)) return MLSTM_ERR_SHAPE;
  if (s.any && (!q || !k || !v || !g || !beta || !o)) return MLSTM_ERR_NULL;
  if (p->num_seqs > 0 && !seq_offsets) return MLSTM_ERR_NULL;
  const void* all[] = {q, k, v, S0, o, S_out, workspace};
  for (const void* x : all)
    if (x && misaligned(x)) return MLSTM_ERR_ALIGN;
  const void* words[] = {g, beta, seq_offsets};
  for (const void* x : words)
    if ((uintptr_t)x & 3) return MLSTM_ERR_ALIGN;
  const size_t need = mlstm_gdr_fwd_workspace_size(p), bS = (size_t)s.N * p->H * p->K * p->V * 4;
  const Range ins[] = {{q, span(p->q, p->B, p->HK, p->T, p->K) * s.es}, {k, span(p->k, p->B, p->HK, p->T, p->K) * s.es},
                       {v, span(p->v, p->B, p->H, p->T, p->V) * s.es},  {g, span(p->g, p->B, p->H, p->T, 1) * 4},
                       {beta, span(p->beta, p->B, p->H, p->T, 1) * 4},  {S0, bS},
                       {seq_offsets, p->num_seqs > 0 ? (size_t)(p->num_seqs + 1) * 4 : 0}};
  const Out outs[] = {{{o, span(p->o, p->B, p->H, p->T, p->V) * s.es}, nullptr}, {{S_out, bS}, S0}, {{workspace, need}, nullptr}};
  if (clash(ins, 7, outs, 3)) return MLSTM_ERR_ALIAS;
  if (need > 0 && (!workspace || workspace_bytes < need)) return MLSTM_ERR_WORKSPACE;
  if (s.N == 0 || p->H == 0) return MLSTM_OK;
  if (!s.any) {  // no tokens: the final states are the initial ones
    if (!S_out || S_out == S0) return MLSTM_OK;
    return done(S0 ? cudaMemcpyAsync(S_out, S0, bS, cudaMemcpyDeviceToDevice, (cudaStream_t)stream)
                   : cudaMemsetAsync(S_out, 0, bS, (cudaStream_t)stream));
  }
  GdrArgs a = gdr_args(p, s);
  a.q = q, a.k = k, a.v = v, a.g = g, a.beta = beta, a.S0 = S0, a.o = o, a.S_out = S_out;
  a.offsets = seq_offsets;
  return done(s.chunk ? launch_gdr_chunk(a, workspace, (cudaStream_t)stream)
                      : launch_gdr_recurrent(a, (cudaStream_t)stream));
}

mlstm_status_t mlstm_gdr_step(const mlstm_gdr_step_params_t* p, const void* q, const void* k, const void* v,
                              const float* g, const float* beta, const int* slots, float* S, void* o,
                              mlstm_stream_t stream) {
  if (!p) return MLSTM_ERR_NULL;
  if (p->dtype != MLSTM_F32 && p->dtype != MLSTM_BF16) return MLSTM_ERR_DTYPE;
  if (!sizes_ok(p->B, p->HK, p->H, p->K, p->V) || p->pool < 0) return MLSTM_ERR_SHAPE;
  if (!slots && p->pool < p->B) return MLSTM_ERR_SHAPE;
  const int es = p->dtype == MLSTM_BF16 ? 2 : 4;
  const int unit = 16 / es;
  if (!strides_ok(p->q, p->B, p->HK, 1, unit) || !strides_ok(p->k, p->B, p->HK, 1, unit) ||
      !strides_ok(p->v, p->B, p->H, 1, unit) || !strides_ok(p->o, p->B, p->H, 1, unit) ||
      !strides_ok(p->g, p->B, p->H, 1, 1) || !strides_ok(p->beta, p->B, p->H, 1, 1))
    return MLSTM_ERR_SHAPE;
  if (!apart(p->o, p->B, p->H, 1, p->V)) return MLSTM_ERR_SHAPE;
  if (p->B == 0 || p->H == 0) return MLSTM_OK;
  if (!q || !k || !v || !g || !beta || !o || (!S && p->pool > 0)) return MLSTM_ERR_NULL;
  const void* wide[] = {q, k, v, S, o};
  for (const void* x : wide)
    if (x && misaligned(x)) return MLSTM_ERR_ALIGN;
  const void* words[] = {g, beta, slots};
  for (const void* x : words)
    if ((uintptr_t)x & 3) return MLSTM_ERR_ALIGN;
  const Range ins[] = {{q, span(p->q, p->B, p->HK, 1, p->K) * es}, {k, span(p->k, p->B, p->HK, 1, p->K) * es},
                       {v, span(p->v, p->B, p->H, 1, p->V) * es},  {g, span(p->g, p->B, p->H, 1, 1) * 4},
                       {beta, span(p->beta, p->B, p->H, 1, 1) * 4}, {slots, slots ? (size_t)p->B * 4 : 0}};
  const Out outs[] = {{{o, span(p->o, p->B, p->H, 1, p->V) * es}, nullptr},
                      {{S, (size_t)p->pool * p->H * p->K * p->V * 4}, nullptr}};
  if (clash(ins, 6, outs, 2)) return MLSTM_ERR_ALIAS;
  GdrStepArgs a = {};
  a.B = p->B, a.HK = p->HK, a.H = p->H, a.K = p->K, a.V = p->V, a.pool = p->pool;
  a.dtype = p->dtype == MLSTM_BF16 ? 1 : 0;
  a.q = q, a.k = k, a.v = v, a.g = g, a.beta = beta, a.slots = slots, a.S = S, a.o = o;
  a.sq = to_stride(p->q), a.sk = to_stride(p->k), a.sv = to_stride(p->v);
  a.sg = to_stride(p->g), a.sb = to_stride(p->beta), a.so = to_stride(p->o);
  return done(launch_gdr_step(a, (cudaStream_t)stream));
}

size_t mlstm_gdr_bwd_workspace_size(const mlstm_gdr_params_t* p) {
  GdrShape s;
  if (check_gdr(p, true, &s) != MLSTM_OK || !s.any) return 0;
  return gdr_bwd_workspace_bytes(gdr_args(p, s));
}

mlstm_status_t mlstm_gdr_bwd(const mlstm_gdr_params_t* p, const void* q, const void* k, const void* v, const float* g,
                             const float* beta, const float* S0, const int* seq_offsets, const void* dout,
                             const float* dS, mlstm_gdr_stride_t s_dq, mlstm_gdr_stride_t s_dk,
                             mlstm_gdr_stride_t s_dv, void* dq, void* dk, void* dv, float* dg, float* dbeta,
                             float* dS0, void* workspace, size_t workspace_bytes, mlstm_stream_t stream) {
  GdrShape s;
  mlstm_status_t st = check_gdr(p, true, &s);
  if (st != MLSTM_OK) return st;
  if (!strides_ok(s_dq, p->B, p->HK, p->T, s.unit) || !strides_ok(s_dk, p->B, p->HK, p->T, s.unit) ||
      !strides_ok(s_dv, p->B, p->H, p->T, s.unit) || !apart(s_dq, p->B, p->HK, p->T, p->K) ||
      !apart(s_dk, p->B, p->HK, p->T, p->K) || !apart(s_dv, p->B, p->H, p->T, p->V))
    return MLSTM_ERR_SHAPE;
  if (s.any && (!q || !k || !v || !g || !beta || !dout || !dq || !dk || !dv || !dg || !dbeta)) return MLSTM_ERR_NULL;
  if (p->num_seqs > 0 && !seq_offsets) return MLSTM_ERR_NULL;
  const void* all[] = {q, k, v, S0, dout, dS, dq, dk, dv, dS0, workspace};
  for (const void* x : all)
    if (x && misaligned(x)) return MLSTM_ERR_ALIGN;
  const void* words[] = {g, beta, seq_offsets, dg, dbeta};
  for (const void* x : words)
    if ((uintptr_t)x & 3) return MLSTM_ERR_ALIGN;
  const size_t need = mlstm_gdr_bwd_workspace_size(p), bS = (size_t)s.N * p->H * p->K * p->V * 4;
  const size_t gates = (size_t)p->B * p->H * p->T * 4;
  const Range ins[] = {{q, span(p->q, p->B, p->HK, p->T, p->K) * s.es}, {k, span(p->k, p->B, p->HK, p->T, p->K) * s.es},
                       {v, span(p->v, p->B, p->H, p->T, p->V) * s.es},  {g, span(p->g, p->B, p->H, p->T, 1) * 4},
                       {beta, span(p->beta, p->B, p->H, p->T, 1) * 4},  {S0, bS},
                       {seq_offsets, p->num_seqs > 0 ? (size_t)(p->num_seqs + 1) * 4 : 0},
                       {dout, span(p->o, p->B, p->H, p->T, p->V) * s.es}, {dS, bS}};
  const Out outs[] = {{{dq, span(s_dq, p->B, p->HK, p->T, p->K) * s.es}, nullptr},
                      {{dk, span(s_dk, p->B, p->HK, p->T, p->K) * s.es}, nullptr},
                      {{dv, span(s_dv, p->B, p->H, p->T, p->V) * s.es}, nullptr},
                      {{dg, gates}, nullptr}, {{dbeta, gates}, nullptr}, {{dS0, bS}, nullptr},
                      {{workspace, need}, nullptr}};
  if (clash(ins, 9, outs, 7)) return MLSTM_ERR_ALIAS;
  if (need > 0 && (!workspace || workspace_bytes < need)) return MLSTM_ERR_WORKSPACE;
  if (s.N == 0 || p->H == 0) return MLSTM_OK;
  if (!s.any) {  // no tokens: the initial states are the final ones
    if (!dS0) return MLSTM_OK;
    return done(dS ? cudaMemcpyAsync(dS0, dS, bS, cudaMemcpyDeviceToDevice, (cudaStream_t)stream)
                   : cudaMemsetAsync(dS0, 0, bS, (cudaStream_t)stream));
  }
  GdrArgs a = gdr_args(p, s);
  a.q = q, a.k = k, a.v = v, a.g = g, a.beta = beta, a.S0 = S0, a.dout = dout, a.dS = dS;
  a.offsets = seq_offsets;
  a.sdq = to_stride(s_dq), a.sdk = to_stride(s_dk), a.sdv = to_stride(s_dv);
  a.dq = dq, a.dk = dk, a.dv = dv, a.dg = dg, a.dbeta = dbeta, a.dS0 = dS0;
  return done(launch_gdr_bwd(a, workspace, (cudaStream_t)stream));
}

mlstm_status_t mlstm_gdr_status(const mlstm_gdr_params_t* p, const void* workspace, mlstm_stream_t stream) {
  GdrShape s;
  mlstm_status_t st = check_gdr(p, false, &s);
  if (st != MLSTM_OK) return st;
  const bool waits = s.chunk && s.any && gdr_tc_pass(gdr_args(p, s));
  if (waits && !workspace) return MLSTM_ERR_NULL;
  if (cudaStreamSynchronize((cudaStream_t)stream) != cudaSuccess) return MLSTM_ERR_CUDA;
  if (!waits) return MLSTM_OK;
  unsigned int word = 0;
  if (cudaMemcpy(&word, workspace, sizeof(word), cudaMemcpyDeviceToHost) != cudaSuccess) return MLSTM_ERR_CUDA;
  return word == 0 ? MLSTM_OK : MLSTM_ERR_TIMEOUT;
}

static mlstm_status_t check_rms(const mlstm_rms_params_t* p, bool backward, int* group) {
  if (!p) return MLSTM_ERR_NULL;
  if (p->dtype != MLSTM_F32 && p->dtype != MLSTM_BF16) return MLSTM_ERR_DTYPE;
  if (p->rows < 0 || p->rows > (1LL << 31) - 1 || !rms_norm_supported(p->D) || !(p->eps >= 0.f)) return MLSTM_ERR_SHAPE;
  *group = p->D;
  if (backward) return MLSTM_OK;
  if (p->quant != MLSTM_RMS_NONE && p->quant != MLSTM_RMS_E4M3 && p->quant != MLSTM_RMS_INT8) return MLSTM_ERR_DTYPE;
  if (p->quant != MLSTM_RMS_NONE) {
    if (p->group != 0 && p->group != 128) return MLSTM_ERR_SHAPE;
    if (p->group == 128 && p->D > 128) *group = 128;
  }
  return MLSTM_OK;
}

mlstm_status_t mlstm_rms_norm(const mlstm_rms_params_t* p, const void* x, const void* residual, const float* weight,
                              void* r_out, void* y, float* scales, mlstm_stream_t stream) {
  int group;
  mlstm_status_t st = check_rms(p, false, &group);
  if (st != MLSTM_OK) return st;
  if (p->rows == 0) return MLSTM_OK;
  const bool quant = p->quant != MLSTM_RMS_NONE;
  if (!residual) r_out = nullptr;
  if (!quant) scales = nullptr;
  if (!x || !y || (residual && !r_out) || (quant && !scales)) return MLSTM_ERR_NULL;
  const void* all[] = {x, residual, weight, r_out, y, scales};
  for (const void* ptr : all)
    if (ptr && misaligned(ptr)) return MLSTM_ERR_ALIGN;
  const size_t n = (size_t)p->rows * p->D, es = p->dtype == MLSTM_BF16 ? 2 : 4;
  const size_t ng = (size_t)p->rows * ((p->D + group - 1) / group);
  const Range rx{x, n * es}, rr{residual, n * es}, rw{weight, (size_t)p->D * 4};
  const Range ro{r_out, n * es}, ry{y, quant ? n : n * es}, rs{scales, ng * 4};
  if ((overlaps(ro, rx) && r_out != x) || (overlaps(ro, rr) && r_out != residual) || overlaps(ro, rw)) return MLSTM_ERR_ALIAS;
  const Range rest[] = {rx, rr, rw, ro};
  for (const Range& i : rest)
    if (overlaps(ry, i) || overlaps(rs, i)) return MLSTM_ERR_ALIAS;
  if (overlaps(ry, rs)) return MLSTM_ERR_ALIAS;
  RmsArgs a = {};
  a.rows = p->rows, a.D = p->D, a.dtype = p->dtype == MLSTM_BF16 ? 1 : 0, a.kind = p->quant, a.group = group;
  a.eps = p->eps, a.x = x, a.res = residual, a.weight = weight, a.r_out = r_out, a.y = y, a.scales = scales;
  return done(launch_rms_norm(a, (cudaStream_t)stream));
}

size_t mlstm_rms_norm_bwd_workspace_size(const mlstm_rms_params_t* p) {
  int group;
  if (check_rms(p, true, &group) != MLSTM_OK || p->rows == 0) return 0;
  return rms_norm_bwd_workspace_bytes(p->rows, p->D);
}

mlstm_status_t mlstm_rms_norm_bwd(const mlstm_rms_params_t* p, const void* dy, const void* r, const float* weight,
                                  const void* dresidual, void* dx, float* dweight, void* workspace,
                                  size_t workspace_bytes, mlstm_stream_t stream) {
  int group;
  mlstm_status_t st = check_rms(p, true, &group);
  if (st != MLSTM_OK) return st;
  if (p->rows > 0 && (!dy || !r || !dx)) return MLSTM_ERR_NULL;
  const void* all[] = {dy, r, weight, dresidual, dx, dweight, workspace};
  for (const void* ptr : all)
    if (ptr && misaligned(ptr)) return MLSTM_ERR_ALIGN;
  const size_t n = (size_t)p->rows * p->D * (p->dtype == MLSTM_BF16 ? 2 : 4);
  const size_t need = dweight ? mlstm_rms_norm_bwd_workspace_size(p) : 0;
  const Range rd{dy, n}, rr{r, n}, rw{weight, (size_t)p->D * 4}, rres{dresidual, n};
  const Range rx{dx, n}, rdw{dweight, (size_t)p->D * 4}, rws{workspace, need};
  if ((overlaps(rx, rd) && dx != dy) || (overlaps(rx, rres) && dx != dresidual) || overlaps(rx, rr) || overlaps(rx, rw))
    return MLSTM_ERR_ALIAS;
  const Range rest[] = {rd, rr, rw, rres, rx};
  for (const Range& i : rest)
    if (overlaps(rdw, i) || overlaps(rws, i)) return MLSTM_ERR_ALIAS;
  if (overlaps(rdw, rws)) return MLSTM_ERR_ALIAS;
  if (need > 0 && (!workspace || workspace_bytes < need)) return MLSTM_ERR_WORKSPACE;
  if (p->rows == 0)
    return dweight ? done(cudaMemsetAsync(dweight, 0, (size_t)p->D * 4, (cudaStream_t)stream)) : MLSTM_OK;
  RmsArgs a = {};
  a.rows = p->rows, a.D = p->D, a.dtype = p->dtype == MLSTM_BF16 ? 1 : 0, a.group = group, a.eps = p->eps;
  a.dy = dy, a.x = r, a.weight = weight, a.res = dresidual, a.y = dx, a.dweight = dweight, a.part = (float*)workspace;
  return done(launch_rms_norm_bwd(a, (cudaStream_t)stream));
}

}  // extern "C"
