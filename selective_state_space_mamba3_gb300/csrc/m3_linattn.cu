// C ABI of the linear-attention operators: host-side validation and dispatch.
// Every check runs before anything is enqueued.
#include <cmath>

#include "linattn.cuh"

namespace m3 {
namespace {

constexpr int64_t kMaxRows = (int64_t)1 << 31;  // row numbers are 32-bit in offsets and tile copies
constexpr int64_t kMaxStride = (int64_t)1 << 38;  // elements; tile copies take byte strides below 2^40

bool aligned_to(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
int cuda_status(cudaError_t e) { return e == cudaSuccess ? M3_OK : M3_ERR_CUDA; }

// A required pointer: non-NULL, aligned to `n` bytes.
int need(const void* p, size_t n) {
  if (!p) return M3_ERR_INVALID_ARGUMENT;
  return aligned_to(p, n) ? M3_OK : M3_ERR_UNALIGNED;
}
int optional(const void* p, size_t n) { return !p || aligned_to(p, n) ? M3_OK : M3_ERR_UNALIGNED; }

#define M3_TRY(x)                       \
  do {                                  \
    const int try_st_ = (x);            \
    if (try_st_ != M3_OK) return try_st_; \
  } while (0)

bool dtype_ok(int d) { return d == M3_DTYPE_FP32 || d == M3_DTYPE_BF16; }
size_t elem(int d) { return d == M3_DTYPE_FP32 ? 4 : 2; }

// Row stride: 0 means dense, otherwise at least the row's width.
int stride(int64_t given, int64_t width, int64_t* out) {
  if (given < 0 || given > kMaxStride || (given > 0 && given < width)) return M3_ERR_INVALID_ARGUMENT;
  *out = given ? given : width;
  return M3_OK;
}

int resolve_rope(const m3_qk_norm_rope_config* c, bool backward, RopeArgs* a) {
  if (!c) return M3_ERR_INVALID_ARGUMENT;
  const int64_t D = c->head_dim, A = c->num_rope_angles;
  if (c->rows < 0 || c->rows >= kMaxRows || c->num_q_heads < 0 || c->num_k_heads < 0 ||
      c->num_q_heads + c->num_k_heads == 0 || c->num_q_heads > 65535 || c->num_k_heads > 65535)
    return M3_ERR_INVALID_ARGUMENT;
  if (D < 1 || D > 256 || A < 0 || 2 * A > D) return M3_ERR_INVALID_ARGUMENT;
  if (A > 0 && (c->max_positions < 1 || c->max_positions >= kMaxRows)) return M3_ERR_INVALID_ARGUMENT;
  if (!std::isfinite(c->epsilon) || !(c->epsilon > 0.f) || !dtype_ok(c->dtype))
    return M3_ERR_INVALID_ARGUMENT;
  *a = RopeArgs{};
  a->rows = c->rows;
  a->D = (int)D; a->A = (int)A; a->max_pos = (int)(A ? c->max_positions : 0);
  a->eps = c->epsilon; a->dtype = c->dtype;
  const int64_t heads[2] = {c->num_q_heads, c->num_k_heads};
  const int64_t in[2] = {c->q_stride, c->k_stride}, out[2] = {c->q_out_stride, c->k_out_stride};
  for (int i = 0; i < 2; ++i) {
    a->side[i].heads = (int)heads[i];
    M3_TRY(stride(in[i], heads[i] * D, &a->side[i].xs));
    int64_t o;
    M3_TRY(stride(out[i], heads[i] * D, &o));
    // the adjoint's output gradients have the outputs' strides, its input gradients are dense
    a->side[i].ys = backward ? heads[i] * D : o;
    a->side[i].dys = backward ? o : 0;
  }
  return M3_OK;
}

int check_rope(const m3_qk_norm_rope_config* c, RopeArgs* a, const void* const* x,
               const float* const* w, const float* cos_t, const float* sin_t, const int32_t* pos,
               const void* const* dy, void* const* y) {
  const size_t es = elem(a->dtype);
  for (int i = 0; i < 2; ++i) {
    RopeSide& s = a->side[i];
    M3_TRY(optional(w[i], 16));
    s.w = w[i];
    if (!s.heads || !a->rows) continue;
    M3_TRY(need(x[i], es));
    M3_TRY(need(y[i], es));
    if (dy) M3_TRY(need(dy[i], es));
    s.x = x[i]; s.y = y[i]; s.dy = dy ? dy[i] : nullptr;
  }
  M3_TRY(a->A ? need(cos_t, 16) : optional(cos_t, 16));
  M3_TRY(a->A ? need(sin_t, 16) : optional(sin_t, 16));
  M3_TRY(optional(pos, 4));
  if (a->A && !pos && c->rows > c->max_positions) return M3_ERR_INVALID_ARGUMENT;
  a->cos_table = cos_t; a->sin_table = sin_t; a->positions = pos;
  return M3_OK;
}

// Shape of a linear-attention call. `rep` is the heads of a group.
struct La {
  int B, H, G, rep, P, N, dtype;
  int64_t L, rows, num_slots, qs, ks, vs, os;
  float scale;
};

int resolve_la(const m3_linear_attention_config* c, La* g) {
  if (!c) return M3_ERR_INVALID_ARGUMENT;
  const int64_t G = c->num_groups == 0 ? c->num_heads : c->num_groups;
  if (c->batch_size < 1 || c->sequence_length < 1 || c->num_heads < 1 || c->num_groups < 0 ||
      c->num_heads % G != 0 || c->num_heads > 65535 || c->batch_size > 65535 * 256ll ||
      c->batch_size * c->num_heads > (1 << 22))
    return M3_ERR_INVALID_ARGUMENT;
  if (c->head_dim < 1 || c->head_dim > 128 || c->state_size < 1 || c->state_size > 128)
    return M3_ERR_INVALID_ARGUMENT;
  if (c->sequence_length >= kMaxRows || c->total_rows < 0 || c->total_rows >= kMaxRows ||
      c->num_slots < 0 || c->num_slots >= kMaxRows)
    return M3_ERR_INVALID_ARGUMENT;
  if (!std::isfinite(c->scale) || !dtype_ok(c->dtype)) return M3_ERR_INVALID_ARGUMENT;
  g->B = (int)c->batch_size; g->H = (int)c->num_heads; g->G = (int)G; g->rep = (int)(c->num_heads / G);
  g->P = (int)c->head_dim; g->N = (int)c->state_size; g->dtype = c->dtype;
  g->L = c->sequence_length; g->rows = c->total_rows; g->num_slots = c->num_slots;
  g->scale = c->scale;
  M3_TRY(stride(c->q_stride, G * c->state_size, &g->qs));
  M3_TRY(stride(c->k_stride, G * c->state_size, &g->ks));
  M3_TRY(stride(c->v_stride, c->num_heads * c->head_dim, &g->vs));
  M3_TRY(stride(c->out_stride, c->num_heads * c->head_dim, &g->os));
  return M3_OK;
}

// Without offsets the rows are B whole sequences of L tokens.
int check_rows(const La& g, const int32_t* offsets) {
  if (offsets) return optional(offsets, 4);
  return g.rows == (int64_t)g.B * g.L ? M3_OK : M3_ERR_INVALID_ARGUMENT;
}

// Segments a sequence is cut into: the number with the shortest pass, counted in
// 128-token chunks walked one after another. That is the bfloat16 kernel's chunk; the
// float32 one walks 112 tokens, so that a segment of one such chunk takes it two walks
// and one of four chunks five, and bfloat16 calls that tile copies do not take run on
// it with half the places counted here: their cuts are not the best ones (4 x 2001
// float32 tokens of one head: 16 segments, 31 walks a sequence, 18 uncut). The kernels have a block for every 64 output columns,
// and the SMs hold two (bfloat16) or one (float32) each. A cut call walks every
// segment twice, the first time (states alone) in about half the time, and starts
// two more kernels, about two chunks' time. Of numbers within 5 % of each other the
// smallest moves the fewest states; segments of fewer than four chunks, whose states
// are as large as their rows, are for calls that leave SMs without a block.
void choose_segments(const La& g, bool backward, int* nseg, int64_t* seg_len) {
  const int tp = (g.P + 63) / 64, tn = (g.N + 63) / 64;
  const int64_t blocks = (int64_t)g.B * g.H * (backward ? 2 * tn + tp : tp);
  const int64_t slots = g.dtype == M3_DTYPE_BF16 ? 304 : 152;
  const int64_t chunks = (g.L + kLaChunk - 1) / kLaChunk;
  double best = 0;
  for (int64_t n = 1; n <= 64 && n <= chunks; ++n) {
    const int64_t per = (chunks + n - 1) / n, segs = (chunks + per - 1) / per;
    if (segs > 1 && per < 4 && blocks * segs > slots) continue;
    const double turns = (double)((blocks * segs + slots - 1) / slots) * per;
    const double cost = segs > 1 ? 1.5 * turns + 2 : turns;
    if (n == 1 || cost < 0.95 * best) {
      best = cost;
      *nseg = (int)segs;
      *seg_len = per * kLaChunk;
    }
  }
}

constexpr size_t kStatusBytes = 256;
size_t round256(size_t n) { return (n + 255) / 256 * 256; }

// Workspace: the status word, the segments' states, the per-head partial
// gradients of shared queries and keys (backward).
struct LaWork {
  size_t entry, part_q, part_k, total;
  int nseg;
  int64_t seg_len;
};
LaWork la_work(const La& g, bool backward) {
  LaWork w{};
  const int nrole = backward ? 3 : 1;
  choose_segments(g, backward, &w.nseg, &w.seg_len);
  size_t o = kStatusBytes;
  w.entry = o;
  if (w.nseg > 1) o += round256((size_t)nrole * w.nseg * g.B * g.H * g.N * g.P * 4);
  w.part_q = w.part_k = o;
  if (backward && g.rep > 1) {
    const size_t one = round256((size_t)g.rows * g.H * g.N * 4);
    o += one;
    w.part_k = o;
    o += one;
  }
  w.total = o;
  return w;
}

LaArgs base_args(const La& g, const LaWork& w, int nrole, const float* ld, const int32_t* offsets,
                 void* ws) {
  LaArgs a{};
  a.nrole = nrole;
  LaCall& c = a.call;
  c.B = g.B; c.H = g.H; c.dtype = g.dtype; c.L = g.L; c.rows = g.rows;
  c.log_decay = ld; c.offsets = offsets;
  c.nseg = w.nseg; c.seg_len = w.seg_len;
  c.entry = w.nseg > 1 ? (float*)((char*)ws + w.entry) : nullptr;
  c.status = (uint32_t*)ws;
  a.entry_role = (int64_t)w.nseg * g.B * g.H * g.N * g.P;
  return a;
}

// One pass of every role.
cudaError_t launch_pass(const LaArgs& a, LaPass pass, cudaStream_t s) {
  // A few tokens (never cut into segments) go one by one: up to kLaShort where the
  // float32 kernel would take them; up to eight, and to the work that costs what the
  // bfloat16 kernel's one chunk does (7 us; 0.56 us for a million of B H L P N), where
  // that one would. Their outputs have one rounding only.
  const bool tiles = la_mma_supported(a);
  const double work = (double)a.call.B * a.call.H * a.call.L * a.role[0].P * a.role[0].N;
  const bool few = tiles ? a.call.L <= 8 && work <= 8e6 : a.call.L <= kLaShort;
  auto* const launch = few ? launch_la_short : tiles ? launch_la_mma : launch_la_split;
  for (int i = 0; i < a.nrole; ++i) {
    LaCall c = a.call;
    c.role = a.role[i];
    if (c.entry) c.entry += i * a.entry_role;
    c.clear = i == 0 && (pass == kLaSummary || c.nseg == 1);
    c.beside = i > 0;
    const cudaError_t e = launch(c, pass, s);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

int run_la(const LaArgs& a, cudaStream_t s) {
  if (a.call.nseg > 1) {
    M3_TRY(cuda_status(launch_pass(a, kLaSummary, s)));
    M3_TRY(cuda_status(launch_la_prefix(a, s)));
  }
  return cuda_status(launch_pass(a, kLaMain, s));
}

int check_workspace(const void* ws, size_t bytes, size_t want) {
  if (!ws || bytes < want) return M3_ERR_WORKSPACE;
  return aligned_to(ws, 16) ? M3_OK : M3_ERR_UNALIGNED;
}

}  // namespace
}  // namespace m3

using namespace m3;

extern "C" {

int m3_qk_norm_rope(const m3_qk_norm_rope_config* cfg, const void* q, const void* k,
                    const float* q_weight, const float* k_weight, const float* cos_table,
                    const float* sin_table, const int32_t* positions, void* q_out, void* k_out,
                    m3_stream_t stream) {
  NvtxRange nvtx_range("m3_qk_norm_rope");
  RopeArgs a;
  M3_TRY(resolve_rope(cfg, false, &a));
  const void* x[2] = {q, k};
  const float* w[2] = {q_weight, k_weight};
  void* y[2] = {q_out, k_out};
  M3_TRY(check_rope(cfg, &a, x, w, cos_table, sin_table, positions, nullptr, y));
  if (a.rows == 0) return M3_OK;
  return cuda_status(launch_qk_norm_rope(a, (cudaStream_t)stream));
}

int m3_qk_norm_rope_backward_workspace(const m3_qk_norm_rope_config* cfg, size_t* bytes) {
  RopeArgs a;
  if (!bytes) return M3_ERR_INVALID_ARGUMENT;
  M3_TRY(resolve_rope(cfg, true, &a));
  *bytes = qk_norm_rope_backward_bytes(a);
  return M3_OK;
}

int m3_qk_norm_rope_backward(const m3_qk_norm_rope_config* cfg, const void* q, const void* k,
                             const float* q_weight, const float* k_weight,
                             const float* cos_table, const float* sin_table,
                             const int32_t* positions, const void* grad_q_out,
                             const void* grad_k_out, void* grad_q, void* grad_k,
                             float* grad_q_weight, float* grad_k_weight, void* workspace,
                             size_t workspace_bytes, m3_stream_t stream) {
  NvtxRange nvtx_range("m3_qk_norm_rope_backward");
  RopeArgs a;
  M3_TRY(resolve_rope(cfg, true, &a));
  const void *x[2] = {q, k}, *dy[2] = {grad_q_out, grad_k_out};
  const float* w[2] = {q_weight, k_weight};
  void* y[2] = {grad_q, grad_k};
  M3_TRY(check_rope(cfg, &a, x, w, cos_table, sin_table, positions, dy, y));
  M3_TRY(optional(grad_q_weight, 16));
  M3_TRY(optional(grad_k_weight, 16));
  a.gw[0] = grad_q_weight; a.gw[1] = grad_k_weight;
  if (a.gw[0] || a.gw[1]) {
    M3_TRY(check_workspace(workspace, workspace_bytes, qk_norm_rope_backward_bytes(a)));
    a.partial = (float*)workspace;
  }
  if (a.rows == 0) {
    for (float* gw : a.gw)
      if (gw && cudaMemsetAsync(gw, 0, a.D * sizeof(float), (cudaStream_t)stream) != cudaSuccess)
        return M3_ERR_CUDA;
    return M3_OK;
  }
  return cuda_status(launch_qk_norm_rope_backward(a, (cudaStream_t)stream));
}

int m3_linear_attention_forward_workspace(const m3_linear_attention_config* cfg, size_t* bytes) {
  La g;
  if (!bytes) return M3_ERR_INVALID_ARGUMENT;
  M3_TRY(resolve_la(cfg, &g));
  *bytes = la_work(g, false).total;
  return M3_OK;
}

int m3_linear_attention_forward(const m3_linear_attention_config* cfg, const void* q,
                                const void* k, const void* v, const float* log_decay,
                                const int32_t* offsets, const float* initial_state, void* out,
                                float* final_state, void* workspace, size_t workspace_bytes,
                                m3_stream_t stream) {
  NvtxRange nvtx_range("m3_linear_attention_forward");
  La g;
  M3_TRY(resolve_la(cfg, &g));
  M3_TRY(check_rows(g, offsets));
  const size_t es = elem(g.dtype);
  if (g.rows > 0) {
    for (const void* p : {q, k, v, (const void*)out}) M3_TRY(need(p, es));
  }
  M3_TRY(need(log_decay, 4));
  M3_TRY(optional(initial_state, 16));
  M3_TRY(optional(final_state, 16));
  const LaWork w = la_work(g, false);
  M3_TRY(check_workspace(workspace, workspace_bytes, w.total));
  LaArgs a = base_args(g, w, 1, log_decay, offsets, workspace);
  LaRole& r = a.role[0];
  r.q = q; r.k = k; r.v = v; r.out = out;
  r.qs = g.qs; r.ks = g.ks; r.vs = g.vs; r.os = g.os;
  r.q_rep = r.k_rep = g.rep; r.v_rep = r.out_rep = 1;
  r.N = g.N; r.P = g.P;
  r.intra = r.inter = g.scale; r.kv = 1.f;
  r.init = initial_state; r.fin = final_state;
  r.sp = g.N; r.sn = 1;
  return run_la(a, (cudaStream_t)stream);
}

int m3_linear_attention_step(const m3_linear_attention_config* cfg, const void* q, const void* k,
                             const void* v, const float* log_decay, const int32_t* slots,
                             float* state, void* out, m3_stream_t stream) {
  NvtxRange nvtx_range("m3_linear_attention_step");
  La g;
  M3_TRY(resolve_la(cfg, &g));
  if (g.L != 1 || g.rows != g.B) return M3_ERR_INVALID_ARGUMENT;
  if (slots ? g.num_slots < 1 : (g.num_slots != 0 && g.num_slots < g.B)) return M3_ERR_INVALID_ARGUMENT;
  const size_t es = elem(g.dtype);
  for (const void* p : {q, k, v, (const void*)out}) M3_TRY(need(p, es));
  M3_TRY(need(log_decay, 4));
  M3_TRY(need(state, 16));
  M3_TRY(optional(slots, 4));
  LaStepArgs a{};
  a.q = q; a.k = k; a.v = v; a.out = out; a.state = state;
  a.log_decay = log_decay; a.slots = slots;
  a.qs = g.qs; a.ks = g.ks; a.vs = g.vs; a.os = g.os;
  a.B = g.B; a.H = g.H; a.rep = g.rep; a.P = g.P; a.N = g.N; a.dtype = g.dtype;
  a.num_slots = slots ? g.num_slots : g.B;
  a.scale = g.scale;
  return cuda_status(launch_la_step(a, (cudaStream_t)stream));
}

int m3_linear_attention_backward_workspace(const m3_linear_attention_config* cfg, size_t* bytes) {
  La g;
  if (!bytes) return M3_ERR_INVALID_ARGUMENT;
  M3_TRY(resolve_la(cfg, &g));
  *bytes = la_work(g, true).total;
  return M3_OK;
}

int m3_linear_attention_backward(const m3_linear_attention_config* cfg, const void* grad_out,
                                 const void* q, const void* k, const void* v,
                                 const float* log_decay, const int32_t* offsets,
                                 const float* initial_state, const float* grad_final_state,
                                 void* grad_q, void* grad_k, void* grad_v,
                                 float* grad_initial_state, void* workspace,
                                 size_t workspace_bytes, m3_stream_t stream) {
  NvtxRange nvtx_range("m3_linear_attention_backward");
  La g;
  M3_TRY(resolve_la(cfg, &g));
  M3_TRY(check_rows(g, offsets));
  const size_t es = elem(g.dtype);
  if (g.rows > 0) {
    for (const void* p : {grad_out, q, k, v, (const void*)grad_q, (const void*)grad_k,
                          (const void*)grad_v})
      M3_TRY(need(p, es));
  }
  M3_TRY(need(log_decay, 4));
  M3_TRY(optional(initial_state, 16));
  M3_TRY(optional(grad_final_state, 16));
  M3_TRY(optional(grad_initial_state, 16));
  const LaWork w = la_work(g, true);
  M3_TRY(check_workspace(workspace, workspace_bytes, w.total));
  LaArgs a = base_args(g, w, 3, log_decay, offsets, workspace);
  float* part_q = (float*)((char*)workspace + w.part_q);
  float* part_k = (float*)((char*)workspace + w.part_k);
  const int64_t hn = (int64_t)g.H * g.N, hp = (int64_t)g.H * g.P;
  const bool shared = g.rep > 1;
  // dq: the recurrence over (do, v, k), walking up, on the transposed state
  LaRole& rq = a.role[0];
  rq.q = grad_out; rq.qs = g.os; rq.q_rep = 1;
  rq.k = v; rq.ks = g.vs; rq.k_rep = 1;
  rq.v = k; rq.vs = g.ks; rq.v_rep = g.rep;
  rq.out = shared ? (void*)part_q : grad_q; rq.os = hn; rq.out_rep = g.rep;
  rq.N = g.P; rq.P = g.N;
  rq.intra = rq.inter = g.scale; rq.kv = 1.f;
  rq.init = initial_state; rq.sp = 1; rq.sn = g.N;
  // dk: over (v, do, q), walking down
  LaRole& rk = a.role[1];
  rk.q = v; rk.qs = g.vs; rk.q_rep = 1;
  rk.k = grad_out; rk.ks = g.os; rk.k_rep = 1;
  rk.v = q; rk.vs = g.qs; rk.v_rep = g.rep;
  rk.out = shared ? (void*)part_k : grad_k; rk.os = hn; rk.out_rep = g.rep;
  rk.N = g.P; rk.P = g.N;
  rk.reverse = 1; rk.shift = 1;
  rk.intra = g.scale; rk.inter = 1.f; rk.kv = g.scale;
  rk.init = grad_final_state; rk.sp = 1; rk.sn = g.N;
  // dv: over (k, q, do), walking down; its last state is that of the first token
  LaRole& rv = a.role[2];
  rv.q = k; rv.qs = g.ks; rv.q_rep = g.rep;
  rv.k = q; rv.ks = g.qs; rv.k_rep = g.rep;
  rv.v = grad_out; rv.vs = g.os; rv.v_rep = 1;
  rv.out = grad_v; rv.os = hp; rv.out_rep = 1;
  rv.N = g.N; rv.P = g.P;
  rv.reverse = 1; rv.shift = 1; rv.fin_shift = 1;
  rv.intra = g.scale; rv.inter = 1.f; rv.kv = g.scale;
  rv.init = grad_final_state; rv.sp = g.N; rv.sn = 1;
  rv.fin = grad_initial_state;
  cudaStream_t s = (cudaStream_t)stream;
  M3_TRY(run_la(a, s));
  if (!shared) return M3_OK;
  M3_TRY(cuda_status(launch_la_group_sum(a.call, part_q, grad_q, g.G, g.rep, g.N, s)));
  return cuda_status(launch_la_group_sum(a.call, part_k, grad_k, g.G, g.rep, g.N, s));
}

}  // extern "C"
