// C ABI of the operators around the mixer: argument checks and launches of the norms, the
// embedding and the AdamW step.  Declarations and documentation: include/prism.h.
#include <math.h>

#include <algorithm>
#include <new>

#include "adamw.cuh"
#include "embed.cuh"
#include "rowops.cuh"

namespace prism {
int device_setup(int** status_out);
int gated_norm_bwd_blocks(long long rows, int d);
int block_norm_blocks(long long rows, int D, bool bwd, int x_bytes, int bytes);
cudaError_t launch_gated_norm_fwd(const GatedNormParams& p, int d, int gate, int dtype, cudaStream_t stream);
cudaError_t launch_gated_norm_bwd(const GatedNormParams& p, int d, int gate, int dtype, cudaStream_t stream);
cudaError_t launch_block_norm(const BlockNormParams& p, bool bwd, int x_dtype, int dtype, cudaStream_t stream);
cudaError_t launch_embed_fwd(const EmbedParams& p, int ids_bits, int table_dtype, int dtype, cudaStream_t stream);
cudaError_t launch_embed_bwd(const EmbedParams& p, int ids_bits, int dtype, cudaStream_t stream);
void set_portable_clusters(bool on);
cudaError_t launch_adamw(const AdamTensor* tensors, int count, unsigned blocks, const AdamParams& a, int p_dtype,
                         int g_dtype, int bits, cudaStream_t stream);
}  // namespace prism

namespace {

bool dtype_ok(int dtype) { return dtype == PRISM_BF16 || dtype == PRISM_FP32; }
size_t elem(int dtype) { return dtype == PRISM_FP32 ? 4 : 2; }
cudaStream_t cuda_stream(prism_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }
int launched(cudaError_t err) { return err == cudaSuccess ? PRISM_OK : PRISM_ERR_CUDA; }
size_t round256(size_t x) { return (x + 255) & ~(size_t)255; }
bool eps_ok(float eps) { return eps > 0.f && isfinite(eps); }

// One buffer of a call.  An output may be exactly the input `may` (rewritten in place: the
// kernels read an element before the thread that read it writes it); any other overlap of an
// output with another buffer is an error.
struct Buffer {
  const void* p;
  size_t bytes;
  bool out = false;
  const void* may = nullptr;
};

template <int N>
int check_buffers(const Buffer (&b)[N]) {
  for (int i = 0; i < N; ++i)
    if (b[i].p && (reinterpret_cast<uintptr_t>(b[i].p) & 15u)) return PRISM_ERR_UNSUPPORTED;
  for (int i = 0; i < N; ++i) {
    if (!b[i].out || !b[i].p) continue;
    const uintptr_t x = reinterpret_cast<uintptr_t>(b[i].p);
    for (int j = 0; j < N; ++j) {
      if (j == i || !b[j].p) continue;
      const uintptr_t y = reinterpret_cast<uintptr_t>(b[j].p);
      if (!b[j].out && b[i].p == b[j].p && b[i].may == b[j].p && b[j].bytes == b[i].bytes) continue;
      if (x < y + b[j].bytes && y < x + b[i].bytes) return PRISM_ERR_INVALID_ARG;
    }
  }
  return PRISM_OK;
}

int check_tokens(int B, int T, int width) {
  if (B < 1 || T < 1 || width < 1) return PRISM_ERR_INVALID_ARG;
  if ((double)B * T * width > 9.0e15) return PRISM_ERR_UNSUPPORTED;
  return PRISM_OK;
}

int check_gated(int B, int T, int H, int d, long long gate_stride, bool gated, float eps, int act, int dtype) {
  if (H < 1 || d < 1 || !dtype_ok(dtype) || !eps_ok(eps)) return PRISM_ERR_INVALID_ARG;
  if (act != PRISM_ACT_SILU && act != PRISM_ACT_SIGMOID) return PRISM_ERR_INVALID_ARG;
  if ((double)H * d > 2.0e9) return PRISM_ERR_UNSUPPORTED;
  const int rc = check_tokens(B, T, H * d);
  if (rc != PRISM_OK) return rc;
  if (d != 16 && d != 32 && d != 64 && d != 128) return PRISM_ERR_UNSUPPORTED;
  if (gated) {
    if (gate_stride < (long long)H * d) return PRISM_ERR_INVALID_ARG;
    if (gate_stride * (long long)elem(dtype) % 16 != 0) return PRISM_ERR_UNSUPPORTED;
    if ((double)B * T * gate_stride > 9.0e15) return PRISM_ERR_UNSUPPORTED;
  }
  return PRISM_OK;
}

int gate_kind(const void* gate, int act) { return !gate ? 0 : act == PRISM_ACT_SILU ? 1 : 2; }

int check_block(int B, int T, int D, float res_scale, float eps, int x_dtype, int dtype) {
  if (!dtype_ok(x_dtype) || !dtype_ok(dtype) || !eps_ok(eps) || !isfinite(res_scale)) return PRISM_ERR_INVALID_ARG;
  const int rc = check_tokens(B, T, D);
  if (rc != PRISM_OK) return rc;
  if (D > PRISM_MAX_WIDTH || (x_dtype == PRISM_BF16 && dtype == PRISM_FP32)) return PRISM_ERR_UNSUPPORTED;
  if (D > 256 && (double)B * T > 2.0e9) return PRISM_ERR_UNSUPPORTED;  // the kernels number such rows in 32 bits
  return PRISM_OK;
}

int check_embed(int B, int T, int V, int D, float scale, int ids_bits) {
  if (V < 1 || (ids_bits != 32 && ids_bits != 64) || !isfinite(scale)) return PRISM_ERR_INVALID_ARG;
  const int rc = check_tokens(B, T, D);
  if (rc != PRISM_OK) return rc;
  if (D > PRISM_MAX_WIDTH || (long long)B * T > 0x7fffffffll || V > (1 << 30)) return PRISM_ERR_UNSUPPORTED;
  return PRISM_OK;
}

}  // namespace

extern "C" {

int prism_gated_norm_fwd(const void* o, const void* gate, const float* weight, const int32_t* lengths, int B, int T,
                         int H, int d, long long gate_stride, float eps, int act, int dtype, void* y,
                         prism_stream_t stream) {
  int rc = check_gated(B, T, H, d, gate_stride, gate != nullptr, eps, act, dtype);
  if (rc != PRISM_OK) return rc;
  if (!o || !weight || !y) return PRISM_ERR_INVALID_ARG;
  const size_t toks = (size_t)B * T, bytes = toks * H * d * elem(dtype);
  const Buffer bufs[] = {{o, bytes}, {gate, ((toks - 1) * gate_stride + (size_t)H * d) * elem(dtype)},
                         {weight, (size_t)d * 4}, {lengths, (size_t)B * 4}, {y, bytes, true, o}};
  rc = check_buffers(bufs);
  if (rc != PRISM_OK) return rc;
  int* status = nullptr;
  rc = prism::device_setup(&status);
  if (rc != PRISM_OK) return rc;
  const prism::GatedNormParams p{o, gate, weight, nullptr, lengths, y, nullptr, nullptr, nullptr, (long long)toks * H,
                                 gate_stride, prism::FastDiv(T), prism::FastDiv(H), eps,
                                 lengths || (gate && gate_stride != (long long)H * d)};
  return launched(prism::launch_gated_norm_fwd(p, d, gate_kind(gate, act), dtype, cuda_stream(stream)));
}

size_t prism_gated_norm_bwd_workspace_size(int B, int T, int H, int d) {
  if (check_gated(B, T, H, d, 0, false, 1.f, PRISM_ACT_SILU, PRISM_BF16) != PRISM_OK) return 0;
  return round256((size_t)prism::gated_norm_bwd_blocks((long long)B * T * H, d) * d * 4);
}

int prism_gated_norm_bwd(const void* o, const void* gate, const float* weight, const void* dy, const int32_t* lengths,
                         int B, int T, int H, int d, long long gate_stride, float eps, int act, int dtype, void* d_o,
                         void* d_gate, float* d_weight, void* workspace, size_t workspace_bytes,
                         prism_stream_t stream) {
  int rc = check_gated(B, T, H, d, gate_stride, gate != nullptr, eps, act, dtype);
  if (rc != PRISM_OK) return rc;
  if (!o || !weight || !dy || !d_o || !d_weight || (gate && !d_gate)) return PRISM_ERR_INVALID_ARG;
  if (!gate) d_gate = nullptr;
  const size_t need = prism_gated_norm_bwd_workspace_size(B, T, H, d);
  if (!workspace || workspace_bytes < need) return PRISM_ERR_WORKSPACE;
  const size_t toks = (size_t)B * T, bytes = toks * H * d * elem(dtype);
  const Buffer bufs[] = {{o, bytes}, {gate, ((toks - 1) * gate_stride + (size_t)H * d) * elem(dtype)},
                         {weight, (size_t)d * 4}, {dy, bytes}, {lengths, (size_t)B * 4}, {d_o, bytes, true, dy},
                         {d_gate, bytes, true}, {d_weight, (size_t)d * 4, true}, {workspace, need, true}};
  rc = check_buffers(bufs);
  if (rc != PRISM_OK) return rc;
  int* status = nullptr;
  rc = prism::device_setup(&status);
  if (rc != PRISM_OK) return rc;
  const prism::GatedNormParams p{o, gate, weight, dy, lengths, d_o, d_gate, static_cast<float*>(workspace),
                                 d_weight, (long long)toks * H, gate_stride, prism::FastDiv(T), prism::FastDiv(H), eps,
                                 lengths || (gate && gate_stride != (long long)H * d)};
  return launched(prism::launch_gated_norm_bwd(p, d, gate_kind(gate, act), dtype, cuda_stream(stream)));
}

int prism_block_norm_fwd(const void* x, const void* y, const float* post_weight, const float* scale,
                         const float* weight, const int32_t* lengths, int B, int T, int D, float res_scale, float eps,
                         int x_dtype, int dtype, void* x_out, void* h, prism_stream_t stream) {
  int rc = check_block(B, T, D, res_scale, eps, x_dtype, dtype);
  if (rc != PRISM_OK) return rc;
  if (!x || !weight || !h || (y && !x_out) || (!y && (post_weight || scale))) return PRISM_ERR_INVALID_ARG;
  if (!y) x_out = nullptr;
  const size_t n = (size_t)B * T * D, vec = (size_t)D * 4;
  const Buffer bufs[] = {{x, n * elem(x_dtype)}, {y, n * elem(dtype)}, {post_weight, vec}, {scale, vec}, {weight, vec},
                         {lengths, (size_t)B * 4}, {x_out, n * elem(x_dtype), true, x}, {h, n * elem(dtype), true}};
  rc = check_buffers(bufs);
  if (rc != PRISM_OK) return rc;
  int* status = nullptr;
  rc = prism::device_setup(&status);
  if (rc != PRISM_OK) return rc;
  const prism::BlockNormParams p{x, y, post_weight, scale, weight, nullptr, nullptr, lengths, x_out, h, nullptr,
                                 {nullptr, nullptr, nullptr}, (long long)B * T, prism::FastDiv(T), D, 0, 0, res_scale, eps, 1.f / D};
  return launched(prism::launch_block_norm(p, false, x_dtype, dtype, cuda_stream(stream)));
}

size_t prism_block_norm_bwd_workspace_size(int B, int T, int D) {
  if (check_block(B, T, D, 1.f, 1.f, PRISM_BF16, PRISM_BF16) != PRISM_OK) return 0;
  int blocks = 0;  // the most of all types
  for (int x_bytes = 2; x_bytes <= 4; x_bytes += 2)
    for (int bytes = 2; bytes <= x_bytes; bytes += 2)
      blocks = std::max(blocks, prism::block_norm_blocks((long long)B * T, D, true, x_bytes, bytes));
  return round256((size_t)blocks * 3 * D * 4);
}

int prism_block_norm_bwd(const void* x_out, const void* y, const float* post_weight, const float* scale,
                         const float* weight, const void* dh, const void* dx_out, const int32_t* lengths, int B,
                         int T, int D, float res_scale, float eps, int x_dtype, int dtype, void* dx, void* dy,
                         float* d_weight, float* d_post_weight, float* d_scale, void* workspace,
                         size_t workspace_bytes, prism_stream_t stream) {
  int rc = check_block(B, T, D, res_scale, eps, x_dtype, dtype);
  if (rc != PRISM_OK) return rc;
  if (!x_out || !weight || !dh || !dx || !d_weight) return PRISM_ERR_INVALID_ARG;
  if (!y && (post_weight || scale || dy)) return PRISM_ERR_INVALID_ARG;
  if ((y && !dy) || (post_weight && !d_post_weight) || (scale && !d_scale)) return PRISM_ERR_INVALID_ARG;
  const size_t need = prism_block_norm_bwd_workspace_size(B, T, D);
  if (!workspace || workspace_bytes < need) return PRISM_ERR_WORKSPACE;
  const size_t n = (size_t)B * T * D, vec = (size_t)D * 4, nx = n * elem(x_dtype), na = n * elem(dtype);
  const Buffer bufs[] = {{x_out, nx}, {y, na}, {post_weight, vec}, {scale, vec}, {weight, vec}, {dh, na},
                         {dx_out, nx}, {lengths, (size_t)B * 4}, {dx, nx, true, dx_out}, {dy, na, true},
                         {d_weight, vec, true}, {post_weight ? d_post_weight : nullptr, vec, true},
                         {scale ? d_scale : nullptr, vec, true}, {workspace, need, true}};
  rc = check_buffers(bufs);
  if (rc != PRISM_OK) return rc;
  int* status = nullptr;
  rc = prism::device_setup(&status);
  if (rc != PRISM_OK) return rc;
  const prism::BlockNormParams p{x_out, y, post_weight, scale, weight, dh, dx_out, lengths, dx, dy,
                                 static_cast<float*>(workspace),
                                 {d_weight, post_weight ? d_post_weight : d_scale, d_scale}, (long long)B * T, prism::FastDiv(T), D, 0, 0, res_scale, eps, 1.f / D};
  return launched(prism::launch_block_norm(p, true, x_dtype, dtype, cuda_stream(stream)));
}

int prism_embed_fwd(const void* ids, const void* table, const int32_t* lengths, int B, int T, int V, int D,
                    float scale, int ids_bits, int table_dtype, int dtype, void* out, prism_stream_t stream) {
  int rc = check_embed(B, T, V, D, scale, ids_bits);
  if (rc != PRISM_OK) return rc;
  if (!ids || !table || !out || !dtype_ok(table_dtype) || !dtype_ok(dtype)) return PRISM_ERR_INVALID_ARG;
  if (table_dtype == PRISM_BF16 && dtype == PRISM_FP32) return PRISM_ERR_UNSUPPORTED;
  const size_t n = (size_t)B * T;
  const Buffer bufs[] = {{ids, n * (ids_bits / 8)}, {table, (size_t)V * D * elem(table_dtype)},
                         {lengths, (size_t)B * 4}, {out, n * D * elem(dtype), true}};
  rc = check_buffers(bufs);
  if (rc != PRISM_OK) return rc;
  prism::EmbedParams p{};
  rc = prism::device_setup(&p.status);
  if (rc != PRISM_OK) return rc;
  p.ids = ids;
  p.table = table;
  p.lengths = lengths;
  p.out = out;
  p.N = (long long)n;
  p.T = prism::FastDiv(T);
  p.V = V;
  p.D = D;
  p.scale = scale;
  return launched(prism::launch_embed_fwd(p, ids_bits, table_dtype, dtype, cuda_stream(stream)));
}

size_t prism_embed_bwd_workspace_size(int B, int T, int V, int D) {
  if (check_embed(B, T, V, D, 1.f, 32) != PRISM_OK) return 0;
  return prism::EmbedPlan((long long)B * T, V, D).bytes;
}

int prism_embed_bwd(const void* ids, const void* d_out, const int32_t* lengths, int B, int T, int V, int D,
                    float scale, int ids_bits, int dtype, int accumulate, float* d_table, void* workspace,
                    size_t workspace_bytes, prism_stream_t stream) {
  int rc = check_embed(B, T, V, D, scale, ids_bits);
  if (rc != PRISM_OK) return rc;
  if (!ids || !d_out || !d_table || !dtype_ok(dtype)) return PRISM_ERR_INVALID_ARG;
  const size_t n = (size_t)B * T;
  const prism::EmbedPlan plan((long long)n, V, D);
  if (!workspace || workspace_bytes < plan.bytes) return PRISM_ERR_WORKSPACE;
  const Buffer bufs[] = {{ids, n * (ids_bits / 8)}, {d_out, n * D * elem(dtype)}, {lengths, (size_t)B * 4},
                         {d_table, (size_t)V * D * 4, true}, {workspace, plan.bytes, true}};
  rc = check_buffers(bufs);
  if (rc != PRISM_OK) return rc;
  prism::EmbedParams p{};
  rc = prism::device_setup(&p.status);
  if (rc != PRISM_OK) return rc;
  char* ws = static_cast<char*>(workspace);
  p.ids = ids;
  p.d_out = d_out;
  p.lengths = lengths;
  p.d_table = d_table;
  for (int i = 0; i < 2; ++i) p.pairs[i] = reinterpret_cast<uint2*>(ws + plan.off_pairs[i]);
  p.hist = reinterpret_cast<int*>(ws + plan.off_hist);
  p.totals = reinterpret_cast<int*>(ws + plan.off_totals);
  p.present = accumulate ? nullptr : reinterpret_cast<uint32_t*>(ws + plan.off_present);
  p.part = reinterpret_cast<float*>(ws + plan.off_part);
  p.N = (long long)n;
  p.T = prism::FastDiv(T);
  p.V = V;
  p.D = D;
  p.accumulate = accumulate != 0;
  p.scale = scale;
  return launched(prism::launch_embed_bwd(p, ids_bits, dtype, cuda_stream(stream)));
}

void prism_set_portable_clusters(int on) { prism::set_portable_clusters(on != 0); }

int prism_adamw_step(const prism_adamw_tensor* tensors, int count, int step, const int32_t* step_dev, double lr,
                     const float* lr_dev, double beta1, double beta2, double eps, const float* grad_scale, int p_dtype,
                     int g_dtype, int state_bits, prism_stream_t stream) {
  if (count < 0 || (count > 0 && !tensors) || !dtype_ok(p_dtype) || !dtype_ok(g_dtype)) return PRISM_ERR_INVALID_ARG;
  if (state_bits != 8 && state_bits != 32) return PRISM_ERR_INVALID_ARG;
  if (!(beta1 >= 0.0 && beta1 < 1.0 && beta2 >= 0.0 && beta2 < 1.0) || !(eps >= 0.0) || !isfinite(eps) ||
      !isfinite(lr) || (!step_dev && step < 1))
    return PRISM_ERR_INVALID_ARG;
  struct Range {
    uintptr_t lo, hi;
    bool out;
  };
  Range* ranges = count > 0 ? new (std::nothrow) Range[(size_t)count * 7 + 3] : nullptr;
  prism::AdamTensor* list = count > 0 ? new (std::nothrow) prism::AdamTensor[count] : nullptr;
  int rc = count > 0 && (!ranges || !list) ? PRISM_ERR_INVALID_ARG : PRISM_OK;
  int nr = 0, used = 0;
  if (rc == PRISM_OK && count > 0) {
    const void* scalars[] = {grad_scale, step_dev, lr_dev};
    for (const void* s : scalars) {
      if (!s) continue;
      const uintptr_t lo = reinterpret_cast<uintptr_t>(s);
      if (lo & 3u) rc = PRISM_ERR_UNSUPPORTED;
      ranges[nr++] = Range{lo, lo + 4, false};
    }
  }
  for (int i = 0; i < count && rc == PRISM_OK; ++i) {
    const prism_adamw_tensor& t = tensors[i];
    if (t.n < 0 || !isfinite(t.weight_decay)) rc = PRISM_ERR_INVALID_ARG;
    if (rc != PRISM_OK || t.n == 0) continue;
    if (!t.param || !t.grad || !t.exp_avg || !t.exp_avg_sq) rc = PRISM_ERR_INVALID_ARG;
    if (state_bits == 8 && (!t.exp_avg_scale || !t.exp_avg_sq_scale)) rc = PRISM_ERR_INVALID_ARG;
    if (t.copy && p_dtype != PRISM_FP32) rc = PRISM_ERR_INVALID_ARG;
    if (rc != PRISM_OK) break;
    if (t.n > (1ll << 42)) rc = PRISM_ERR_UNSUPPORTED;  // a tensor's blocks fit one grid
    const size_t n = (size_t)t.n, blocks = (n + prism::kAdamBlock - 1) / prism::kAdamBlock;
    const Buffer bufs[] = {{t.param, n * elem(p_dtype), true}, {t.grad, n * elem(g_dtype)},
                           {t.exp_avg, n * (state_bits / 8), true}, {t.exp_avg_sq, n * (state_bits / 8), true},
                           {state_bits == 8 ? t.exp_avg_scale : nullptr, blocks * 4, true},
                           {state_bits == 8 ? t.exp_avg_sq_scale : nullptr, blocks * 4, true}, {t.copy, n * 2, true}};
    for (const Buffer& b : bufs) {
      if (!b.p) continue;
      const uintptr_t lo = reinterpret_cast<uintptr_t>(b.p);
      // scales are read and written one by one, everything else in 16-byte pieces
      if (lo & (b.p == t.exp_avg_scale || b.p == t.exp_avg_sq_scale ? 3u : 15u)) rc = PRISM_ERR_UNSUPPORTED;
      ranges[nr++] = Range{lo, lo + b.bytes, b.out};
    }
    list[used++] = prism::AdamTensor{t.param, t.grad, t.exp_avg, t.exp_avg_sq, t.exp_avg_scale, t.exp_avg_sq_scale,
                                     t.copy, t.n, (float)t.weight_decay, 0};
  }
  if (rc == PRISM_OK) {
    // what is written may overlap nothing else of the call
    std::sort(ranges, ranges + nr, [](const Range& a, const Range& b) { return a.lo < b.lo; });
    uintptr_t any = 0, written = 0;
    for (int i = 0; i < nr; ++i) {
      if (ranges[i].lo < written || (ranges[i].out && ranges[i].lo < any)) rc = PRISM_ERR_INVALID_ARG;
      any = std::max(any, ranges[i].hi);
      if (ranges[i].out) written = std::max(written, ranges[i].hi);
    }
  }
  delete[] ranges;
  int* status = nullptr;
  if (rc == PRISM_OK) rc = prism::device_setup(&status);
  if (rc == PRISM_OK && used > 0) {
    prism::AdamParams a{};
    a.grad_scale = grad_scale;
    a.step_dev = step_dev;
    a.lr_dev = lr_dev;
    a.lr64 = lr;
    a.beta1 = beta1;
    a.beta2 = beta2;
    a.step = step;
    a.lr = (float)lr;
    if (!step_dev) {
      a.lr_c1 = (float)(lr / (1.0 - pow(beta1, (double)step)));
      a.rsqrt_c2 = (float)(1.0 / sqrt(1.0 - pow(beta2, (double)step)));
    }
    a.b1 = (float)beta1;
    a.r1 = (float)(1.0 - beta1);
    a.b2 = (float)beta2;
    a.r2 = (float)(1.0 - beta2);
    a.eps = (float)eps;
    long long elements = 0;
    for (int i = 0; i < used; ++i) elements += list[i].n;
    a.chunk = prism::adam_chunk(elements, state_bits);
    // as many tensors per launch as the parameters and the grid hold
    int first = 0;
    long long blocks = 0;
    for (int i = 0; i <= used && rc == PRISM_OK; ++i) {
      const long long more = i < used ? (list[i].n + a.chunk - 1) / a.chunk : 0;
      if (i == used || i - first == prism::kAdamMostTensors || (i > first && blocks + more > 0x7fffffffll)) {
        rc = launched(prism::launch_adamw(list + first, i - first, (unsigned)blocks, a, p_dtype, g_dtype, state_bits,
                                          cuda_stream(stream)));
        first = i;
        blocks = 0;
      }
      if (i < used) {
        list[i].first_block = (unsigned)blocks;
        blocks += more;
      }
    }
  }
  delete[] list;
  return rc;
}

int prism_dl_pointers(int fields, const prism_dl_field* spec, int n, void* const* objects,
                      prism_dl_from_object from_object, int device, prism_dl_tensor* views, void* out, size_t stride,
                      size_t count_offset) {
  int at = 0;
  for (int f = 0; f < fields; ++f) {
    if (spec[f].type_code == 0) continue;
    for (int i = 0; i < n; ++i, ++at) {
      prism_dl_tensor other;
      prism_dl_tensor& v = f == 0 ? views[i] : other;
      if (from_object(objects[at], &v) != 0) return at;
      if (v.device_type != 2 || v.device_id != device || v.type_code != spec[f].type_code ||
          v.type_bits != spec[f].type_bits || v.type_lanes != 1)
        return at;
      long long elements = 1;
      for (int d = 0; d < v.ndim; ++d) elements *= v.shape[d];
      long long step = 1;  // dense, as far as it matters: the stride of a dimension of one element does not
      for (int d = v.ndim - 1; d >= 0 && v.strides && elements > 0; --d) {
        if (v.shape[d] != 1 && v.strides[d] != step) return at;
        step *= v.shape[d];
      }
      char* row = static_cast<char*>(out) + i * stride;
      if (f == 0) {
        *reinterpret_cast<long long*>(row + count_offset) = elements;
      } else if (spec[f].block > 0) {
        const long long of = *reinterpret_cast<const long long*>(row + count_offset);
        if (elements != (of + spec[f].block - 1) / spec[f].block) return at;
      } else {
        if (v.ndim != views[i].ndim) return at;
        for (int d = 0; d < v.ndim; ++d)
          if (v.shape[d] != views[i].shape[d]) return at;
      }
      *reinterpret_cast<void**>(row + 8 * f) = static_cast<char*>(v.data) + v.byte_offset;
    }
  }
  return -1;
}

}  // extern "C"
