// C ABI of the operators of a decoder layer beside its products, and of its last step (declared
// in include/gemm.h): gemm_run_gated, gemm_run_gated_grad, gemm_norm_rotary,
// gemm_norm_rotary_grad, gemm_sample.  Argument validation, workspace and launches; the kernels
// are in gated_kernel.cu, heads_kernel.cuh and sample_kernel.cu.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <cstring>
#include <initializer_list>

#include "checks.h"
#include "context.h"
#include "gemm.h"
#include "operators.h"
#include "umma.cuh"

using namespace gb300;

namespace {

bool valid_gate(int a) { return a >= GEMM_GATE_SILU && a <= GEMM_GATE_RELU; }

// The sizes and types that both calls of the gated block share.
gemm_status_t check_gated(int64_t M, int64_t N, int64_t K, int dtype, int activation) {
  if (M < 0 || N < 0 || K < 0 || !valid_gate(activation) || !valid_dtype(dtype)) return GEMM_ERR_INVALID_ARG;
  if (dtype == GEMM_F32 || is_fp8(dtype)) return GEMM_ERR_UNSUPPORTED;
  if (M > INT32_MAX - 512 || N > INT32_MAX - 512 || K > INT32_MAX - 512) return GEMM_ERR_UNSUPPORTED;
  if (K % 8) return GEMM_ERR_UNSUPPORTED;
  // (tiles are counted in 32 bits)
  if (2 * ceil_div(M, 256) * ceil_div(N, 128) > INT32_MAX ||
      2 * (2 * ceil_div(N, 256) + ceil_div(M, 256)) * ceil_div(K, 256) > INT32_MAX)
    return GEMM_ERR_UNSUPPORTED;
  return GEMM_OK;
}

// Memory of a call; NULL: none.
struct Span {
  const void* p;
  int64_t bytes;
};
bool meet(const Span& a, const Span& b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return a.p && b.p && x < y + (uint64_t)b.bytes && y < x + (uint64_t)a.bytes;
}
// Whether an output lies in an input or in another output.
bool outputs_overlap(std::initializer_list<Span> outs, std::initializer_list<Span> ins) {
  for (const Span* o = outs.begin(); o != outs.end(); ++o) {
    for (const Span& i : ins)
      if (meet(*o, i)) return true;
    for (const Span* q = outs.begin(); q != o; ++q)
      if (meet(*o, *q)) return true;
  }
  return false;
}

gemm_status_t zero(gemm_ctx* h, void* p, int64_t values, cudaStream_t stream) {
  if (!p || values == 0) return GEMM_OK;
  return launched(h, cudaMemsetAsync(p, 0, (size_t)values * 2, stream));
}

// What all of the block's products take from the handle.
GatedParams gated_params(gemm_ctx* h, int activation) {
  GatedParams p;
  std::memset(&p, 0, sizeof(p));
  p.group_m = 16;
  p.slices = 1;
  p.act = activation;
  p.status = h->d_status;
  p.wait_limit_ns = h->wait_limit_ns;
  p.test_stall = h->test_stall;
  return p;
}

GatedProduct product_of(int64_t M, int64_t N, int64_t K, int64_t cols) {
  GatedProduct d;
  d.M = (int32_t)M;
  d.N = (int32_t)N;
  d.num_m = (int32_t)ceil_div(M, 256);
  d.num_n = (int32_t)ceil_div(N, cols);
  d.tiles = d.num_m * d.num_n;
  d.k_blocks = (int32_t)ceil_div(K, kBlockK);
  return d;
}

// Strides of a tensor of heads in elements.
struct Strides {
  int64_t token, head;
};

// The sizes, types and tables of normed and rotated heads; GEMM_OK with *work false: nothing to
// turn (no tokens, no heads or no values).
gemm_status_t check_heads(int64_t tokens, int64_t heads, int64_t dim, int dtype, const gemm_head_norm_t* n,
                          const gemm_rotary_t* r, bool* work) {
  *work = false;
  if (tokens < 0 || heads < 0 || dim < 0 || !valid_dtype(dtype) || !valid_dtype(n->weight_dtype))
    return GEMM_ERR_INVALID_ARG;
  if (n->query_heads < 0 || n->query_heads > heads || !(n->eps >= 0.0f)) return GEMM_ERR_INVALID_ARG;
  if (is_fp8(dtype) || is_fp8(n->weight_dtype)) return GEMM_ERR_UNSUPPORTED;
  if (!aligned(n->query_weight, (uint64_t)elem_size(n->weight_dtype)) ||
      !aligned(n->key_weight, (uint64_t)elem_size(n->weight_dtype)))
    return GEMM_ERR_UNSUPPORTED;
  if (dim > kMaxHeadDim) return GEMM_ERR_UNSUPPORTED;
  if (tokens == 0 || heads == 0 || dim == 0) return GEMM_OK;
  if (r->axes < 1 || r->axes > 8 || r->rot_dim < 2 || r->rot_dim % 2 || r->rot_dim > dim ||
      r->num_positions < 1 || (r->pairs != GEMM_PAIRS_HALF && r->pairs != GEMM_PAIRS_NEIGHBOURS) || r->inverse != 0)
    return GEMM_ERR_INVALID_ARG;
  if (!r->cos || !r->sin || !r->positions) return GEMM_ERR_INVALID_ARG;
  if (r->pair_axis)
    for (int i = 0; i < r->rot_dim / 2; ++i)
      if (r->pair_axis[i] >= r->axes) return GEMM_ERR_INVALID_ARG;
  if (tokens > INT32_MAX || heads > INT32_MAX || tokens > INT32_MAX / heads) return GEMM_ERR_UNSUPPORTED;
  if (!aligned(r->cos, 4) || !aligned(r->sin, 4) || !aligned(r->positions, 4)) return GEMM_ERR_UNSUPPORTED;
  *work = true;
  return GEMM_OK;
}

bool differ(const Strides& a, const Strides& b, int64_t tokens, int64_t heads) {
  return (tokens > 1 && a.token != b.token) || (heads > 1 && a.head != b.head);
}

// A result's strides: none negative, no two heads in one place.
bool good_result(const Strides& s, int64_t tokens, int64_t heads, int64_t dim) {
  return !overlap(tokens, s.token, heads, s.head, dim);
}

struct Tensor {
  const void* p;
  Strides s;
};

Vectors memory_of(const Tensor& t, int64_t tokens, int64_t heads, int64_t dim, int dtype) {
  const int64_t size = elem_size(dtype);
  return {(Vectors::wide) reinterpret_cast<uintptr_t>(t.p), tokens, (Vectors::wide)t.s.token * size, heads,
          (Vectors::wide)t.s.head * size, (Vectors::wide)dim * size};
}
// Whether `out` lies in the norms' weights, the tables or the positions.
bool meets_tables(const Vectors& out, int64_t tokens, int64_t dim, const gemm_head_norm_t* n, const gemm_rotary_t* r) {
  const Vectors::wide table = (Vectors::wide)r->num_positions * (r->rot_dim / 2) * 4, w = dim * elem_size(n->weight_dtype);
  const struct {
    const void* p;
    Vectors::wide bytes;
  } all[] = {{r->cos, table}, {r->sin, table}, {r->positions, (Vectors::wide)r->axes * tokens * 4},
             {n->query_weight, w}, {n->key_weight, w}};
  for (const auto& t : all)
    if (t.p && share_memory(out, {(Vectors::wide) reinterpret_cast<uintptr_t>(t.p), 1, 0, 1, 0, t.bytes})) return true;
  return false;
}

// Elements per access (16 bytes' worth, 4 or 1) that all of the tensors allow: bases, strides, the
// pairs' halves or ends and the heads' ends.
int heads_vector(std::initializer_list<Tensor> tensors, int64_t tokens, int64_t heads, int64_t dim,
                 int dtype, const gemm_rotary_t* r) {
  const int64_t pairs = r->pairs == GEMM_PAIRS_NEIGHBOURS ? r->rot_dim : r->rot_dim / 2;
  for (int v : {16 / (int)elem_size(dtype), 4}) {
    bool ok = pairs % v == 0 && (dim - r->rot_dim) % v == 0;
    for (const Tensor& t : tensors)
      ok = ok && aligned(t.p, (uint64_t)(v * elem_size(dtype))) && (tokens == 1 || t.s.token % v == 0) &&
           (heads == 1 || t.s.head % v == 0);
    if (ok) return v;
  }
  return 1;
}

HeadsParams heads_params(gemm_ctx* h, int64_t tokens, int64_t heads, int64_t dim, const gemm_head_norm_t* n,
                         const gemm_rotary_t* r) {
  HeadsParams p;
  std::memset(&p, 0, sizeof(p));
  p.tokens = tokens;
  p.heads = (int32_t)heads;
  p.query_heads = n->query_heads;
  p.dim = (int32_t)dim;
  p.half = r->rot_dim / 2;
  p.query_weight = n->query_weight;
  p.key_weight = n->key_weight;
  p.weight_elem = n->weight_dtype;
  p.eps = n->eps;
  p.inv_dim = 1.0f / (float)dim;
  p.cos = r->cos;
  p.sin = r->sin;
  p.positions = r->positions;
  p.num_positions = r->num_positions;
  p.status = h->d_status;
  if (r->pair_axis) std::memcpy(p.pair_axis, r->pair_axis, (size_t)p.half);
  return p;
}

}  // namespace

extern "C" {

gemm_status_t gemm_run_gated(gemm_handle_t h, const void* X, const void* gate_weight,
                             const void* up_weight, void* H, int64_t M, int64_t N, int64_t K,
                             gemm_dtype_t dtype, const gemm_gated_t* gated, gemm_stream_t stream_) {
  if (!h || !gated) return GEMM_ERR_INVALID_ARG;
  const gemm_status_t sizes = check_gated(M, N, K, dtype, gated->activation);
  if (sizes != GEMM_OK) return sizes;
  void* gate = gated->gate;
  void* up = gated->up;
  if (!gate != !up) return GEMM_ERR_INVALID_ARG;
  if (M == 0 || N == 0) return GEMM_OK;
  if (!H || (K > 0 && (!X || !gate_weight || !up_weight))) return GEMM_ERR_INVALID_ARG;
  const int64_t hidden = 2 * M * N, weights = 2 * N * K;
  if (outputs_overlap({{H, hidden}, {gate, hidden}, {up, hidden}},
                      {{X, 2 * M * K}, {gate_weight, weights}, {up_weight, weights}}))
    return GEMM_ERR_INVALID_ARG;
  if (!aligned(X, 16) || !aligned(gate_weight, 16) || !aligned(up_weight, 16) || !aligned(H, 2) ||
      !aligned(gate, 2) || !aligned(up, 2))
    return GEMM_ERR_UNSUPPORTED;
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  if (K == 0) {  // act(0) * 0
    for (void* out : {H, gate, up})
      if (const gemm_status_t st = zero(h, out, M * N, stream); st != GEMM_OK) return st;
    return GEMM_OK;
  }

  if (M <= kGatedFewRows) {
    GatedFewParams f;
    std::memset(&f, 0, sizeof(f));
    const GatedFewSplit split = gated_few_split(M, N, K, h->sms);
    f.tile_rows = split.tile_rows;
    f.splits = split.splits;
    f.x_rows = (int32_t)(ceil_div(M, 16) * 16);
    f.tiles = (int32_t)ceil_div(N, f.tile_rows);
    f.ctas = f.splits > 1 ? f.tiles * f.splits : std::min(f.tiles, h->sms);
    f.k_blocks = (int32_t)ceil_div(K, kBlockK);
    f.h = H;
    f.gate = gate;
    f.up = up;
    f.M = (int32_t)M;
    f.N = (int32_t)N;
    f.act = gated->activation;
    f.idesc = idesc_f16_kmajor(128, (uint32_t)f.x_rows, dtype == GEMM_BF16);
    f.status = h->d_status;
    f.wait_limit_ns = h->wait_limit_ns;
    f.test_stall = h->test_stall;
    GatedFewMaps maps;
    if (!make_map(h, gate_weight, N, K, dtype, f.tile_rows, &maps.gate) ||
        !make_map(h, up_weight, N, K, dtype, f.tile_rows, &maps.up) ||
        !make_map(h, X, M, K, dtype, f.x_rows, &maps.x))
      return GEMM_ERR_CUDA;
    return launched(h, launch_gated_few(dtype, maps, f, stream));
  }

  GatedParams p = gated_params(h, gated->activation);
  p.product[0] = product_of(M, N, K, 128);
  p.slices = gated_slices(p.product[0], p.product[0].k_blocks, 2, 0, h->sms);
  p.units = p.product[0].tiles * p.slices;
  if (p.slices > 1) {
    p.partial_pitch = (int32_t)(ceil_div(N, 4) * 4);
    const gemm_status_t st = ensure_scratch(h, (size_t)p.slices * 2 * M * p.partial_pitch * sizeof(float), 0);
    if (st != GEMM_OK) return st;
    p.partial = static_cast<float*>(h->op.ptr);
  }
  p.out[0] = H;
  p.out[1] = gate;
  p.out[2] = up;
  p.outs = gate ? 3 : 1;
  p.tma_store = N % 8 == 0 && aligned(H, 16) && aligned(gate, 16) && aligned(up, 16);
  GatedMaps maps;
  std::memset(&maps, 0, sizeof(maps));
  if (!make_map(h, X, M, K, dtype, 128, &maps.a[0]) ||
      !make_map(h, gate_weight, N, K, dtype, 128, &maps.b[0]) ||
      !make_map(h, up_weight, N, K, dtype, 128, &maps.b[1]))
    return GEMM_ERR_CUDA;
  for (int o = 0; p.tma_store && o < p.outs; ++o)
    if (!make_map(h, p.out[o], M, N, dtype, 32, &maps.out[o])) return GEMM_ERR_CUDA;
  const gemm_status_t done = launched(h, launch_gated(false, dtype, maps, p, h->sms, stream));
  return done != GEMM_OK || p.slices == 1 ? done : launched(h, launch_gated_join(false, dtype, p, stream));
}

gemm_status_t gemm_run_gated_grad(gemm_handle_t h, const void* X, const void* gate_weight,
                                  const void* up_weight, int64_t M, int64_t N, int64_t K,
                                  gemm_dtype_t dtype, const gemm_gated_grad_t* g,
                                  gemm_stream_t stream_) {
  if (!h || !g) return GEMM_ERR_INVALID_ARG;
  const gemm_status_t sizes = check_gated(M, N, K, dtype, g->activation);
  if (sizes != GEMM_OK) return sizes;
  void* dX = g->dX;
  void* dWg = g->d_gate_weight;
  void* dWu = g->d_up_weight;
  if (!dWg != !dWu) return GEMM_ERR_INVALID_ARG;
  const int64_t hidden = 2 * M * N, weights = 2 * N * K;
  if (outputs_overlap({{dX, 2 * M * K}, {dWg, weights}, {dWu, weights}},
                      {{X, 2 * M * K}, {gate_weight, weights}, {up_weight, weights}, {g->gate, hidden},
                       {g->up, hidden}, {g->dH, hidden}}))
    return GEMM_ERR_INVALID_ARG;
  if (K == 0 || (!dX && !dWg)) return GEMM_OK;
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  if (!aligned(X, 16) || !aligned(gate_weight, 16) || !aligned(up_weight, 16) || !aligned(dX, 16) ||
      !aligned(dWg, 16) || !aligned(dWu, 16) || !aligned(g->gate, 2) || !aligned(g->up, 2) ||
      !aligned(g->dH, 2))
    return GEMM_ERR_UNSUPPORTED;
  if (M == 0 || N == 0) {  // sums of nothing
    gemm_status_t st = zero(h, dX, M * K, stream);
    if (st == GEMM_OK) st = zero(h, dWg, N * K, stream);
    if (st == GEMM_OK) st = zero(h, dWu, N * K, stream);
    return st;
  }
  if (!g->gate || !g->up || !g->dH || (dWg && !X) || (dX && (!gate_weight || !up_weight)))
    return GEMM_ERR_INVALID_ARG;

  GatedRankParams r;
  std::memset(&r, 0, sizeof(r));
  const bool few = dWg && M <= kGatedRankRows;
  if (few) {
    r.x = X;
    r.dh = g->dH;
    r.gate = g->gate;
    r.up = g->up;
    r.d_gate_weight = dWg;
    r.d_up_weight = dWu;
    r.M = (int32_t)M;
    r.N = N;
    r.K = K;
    r.act = g->activation;
    if (!dX) return launched(h, launch_gated_rank(dtype, r, h->sms, stream));
    dWg = dWu = nullptr;
  }

  // dG and dU: rows that TMA can address
  const int64_t pitch = ceil_div(N, 8) * 8;
  const size_t bytes = round_up((size_t)M * pitch * 2);
  GatedParams p = gated_params(h, g->activation);
  if (dX) p.product[0] = product_of(M, K, N, 256);
  if (dWg) p.product[1] = product_of(N, K, M, 256);
  // (as if the weights' gradients were asked for, so that dX is the same bits without them)
  const GatedProduct weights_of = product_of(N, K, M, 256);
  const int64_t sums = 2 * (int64_t)p.product[0].k_blocks;
  const int64_t others = M <= kGatedRankRows ? 0 : 2 * (int64_t)weights_of.tiles * (weights_of.k_blocks + 10);
  p.slices = gated_slices(p.product[0], sums, 1, others, h->sms);
  p.partial_pitch = (int32_t)K;
  const size_t partial = p.slices > 1 ? (size_t)p.slices * M * K * sizeof(float) : 0;
  // fp16: what belongs to the scales, and a copy by columns beside the one by rows
  const bool scaled = dtype == GEMM_F16;
  const int copies = scaled && dX && dWg ? 2 : 1;
  const int64_t first_column = ceil_div(M, 4) * 4, lines = first_column + 2 * N;
  const size_t ranges = scaled ? (size_t)(lines + ceil_div(N, 256)) * sizeof(float) : 0;
  const gemm_status_t st =
      ensure_scratch(h, 2 * copies * bytes + round_up(partial) + ranges, scaled ? (size_t)lines : 0);
  if (st != GEMM_OK) return st;
  char* scratch = static_cast<char*>(h->op.ptr);
  p.partial = reinterpret_cast<float*>(scratch + 2 * copies * bytes);
  GatedSlopeParams s;
  std::memset(&s, 0, sizeof(s));
  s.dh = g->dH;
  s.gate = g->gate;
  s.up = g->up;
  s.dgate = scratch;
  s.dup = scratch + bytes;
  s.dgate_by_column = scratch + 2 * (copies - 1) * bytes;
  s.dup_by_column = scratch + (2 * copies - 1) * bytes;
  if (scaled) {
    s.range.most = static_cast<uint32_t*>(h->op_ctr.ptr);
    s.range.back = reinterpret_cast<float*>(scratch + 2 * copies * bytes + round_up(partial));
    s.range.copied = reinterpret_cast<uint32_t*>(s.range.back + lines);
    s.range.first_column = first_column;
    s.range.rows = dX != nullptr;
    s.range.columns = dWg != nullptr;
    p.range = s.range;
  }
  s.M = M;
  s.N = (int32_t)N;
  s.pitch = (int32_t)pitch;
  s.act = g->activation;
  s.vec = N % 8 == 0 && aligned(g->dH, 16) && aligned(g->gate, 16) && aligned(g->up, 16);

  GatedMaps maps;
  std::memset(&maps, 0, sizeof(maps));
  if (dX && (!make_map(h, s.dgate, M, pitch, dtype, 128, &maps.a[0]) ||
             !make_map(h, s.dup, M, pitch, dtype, 128, &maps.a[1]) ||
             !make_map(h, gate_weight, N, K, dtype, 64, &maps.b[0]) ||
             !make_map(h, up_weight, N, K, dtype, 64, &maps.b[1]) ||
             !make_map(h, dX, M, K, dtype, 32, &maps.out[0])))
    return GEMM_ERR_CUDA;
  if (dWg && (!make_map(h, s.dgate, M, pitch, dtype, 64, &maps.across[0]) ||
              !make_map(h, s.dup, M, pitch, dtype, 64, &maps.across[1]) ||
              (scaled && (!make_map(h, s.dgate_by_column, M, pitch, dtype, 64, &maps.scaled[0]) ||
                          !make_map(h, s.dup_by_column, M, pitch, dtype, 64, &maps.scaled[1]))) ||
              !make_map(h, X, M, K, dtype, 64, &maps.x) ||
              !make_map(h, dWg, N, K, dtype, 32, &maps.out[1]) ||
              !make_map(h, dWu, N, K, dtype, 32, &maps.out[2])))
    return GEMM_ERR_CUDA;
  p.out[0] = dX;
  p.out[1] = dWg;
  p.out[2] = dWu;
  p.tma_store = 1;
  p.units = p.product[0].tiles * p.slices + 2 * p.product[1].tiles;
  p.first = sums / p.slices >= p.product[1].k_blocks ? 0 : 1;

  gemm_status_t done = few ? launched(h, launch_gated_rank(dtype, r, h->sms, stream)) : GEMM_OK;
  if (done == GEMM_OK) done = launched(h, launch_gated_slope(dtype, s, h->sms, stream));
  if (done != GEMM_OK) return done;
  done = launched(h, launch_gated(true, dtype, maps, p, h->sms, stream));
  // (what the products would have left zero)
  if (done != GEMM_OK && scaled) cudaMemsetAsync(s.range.most, 0, (size_t)lines * sizeof(uint32_t), stream);
  if (done == GEMM_OK && p.slices > 1) done = launched(h, launch_gated_join(true, dtype, p, stream));
  return done;
}

gemm_status_t gemm_norm_rotary(gemm_handle_t h, const void* x, void* y, int64_t tokens, int64_t heads,
                               int64_t dim, int64_t x_token_stride, int64_t x_head_stride,
                               int64_t y_token_stride, int64_t y_head_stride, gemm_dtype_t dtype,
                               const gemm_head_norm_t* norm, const gemm_rotary_t* r,
                               gemm_stream_t stream_) {
  if (!h || !norm || !r) return GEMM_ERR_INVALID_ARG;
  const Strides sx{x_token_stride, x_head_stride}, sy{y_token_stride, y_head_stride};
  if (sx.token < 0 || sx.head < 0 || sy.token < 0 || sy.head < 0) return GEMM_ERR_INVALID_ARG;
  bool work;
  const gemm_status_t st = check_heads(tokens, heads, dim, dtype, norm, r, &work);
  if (st != GEMM_OK || !work) return st;
  if (!x || !y || (x == y && differ(sx, sy, tokens, heads))) return GEMM_ERR_INVALID_ARG;
  if (!good_result(sy, tokens, heads, dim)) return GEMM_ERR_INVALID_ARG;
  const Vectors mx = memory_of({x, sx}, tokens, heads, dim, dtype), my = memory_of({y, sy}, tokens, heads, dim, dtype);
  if ((x != y && share_memory(my, mx)) || meets_tables(my, tokens, dim, norm, r)) return GEMM_ERR_INVALID_ARG;
  if (!aligned(x, (uint64_t)elem_size(dtype)) || !aligned(y, (uint64_t)elem_size(dtype)))
    return GEMM_ERR_UNSUPPORTED;
  HeadsParams p = heads_params(h, tokens, heads, dim, norm, r);
  p.x = x;
  p.y = y;
  p.x_token = sx.token, p.x_head = sx.head;
  p.y_token = sy.token, p.y_head = sy.head;
  const int vec = heads_vector({{x, sx}, {y, sy}}, tokens, heads, dim, dtype, r);
  return launched(h, launch_heads(p, dtype, r->pairs == GEMM_PAIRS_NEIGHBOURS, vec, h->sms,
                                  reinterpret_cast<cudaStream_t>(stream_)));
}

gemm_status_t gemm_norm_rotary_grad(gemm_handle_t h, const void* x, const void* dy, void* dx, int64_t tokens,
                                    int64_t heads, int64_t dim, int64_t x_token_stride,
                                    int64_t x_head_stride, int64_t dy_token_stride,
                                    int64_t dy_head_stride, int64_t dx_token_stride,
                                    int64_t dx_head_stride, gemm_dtype_t dtype,
                                    const gemm_head_norm_t* norm, const gemm_rotary_t* r,
                                    float* d_query_weight, float* d_key_weight, gemm_stream_t stream_) {
  if (!h || !norm || !r) return GEMM_ERR_INVALID_ARG;
  const Strides sx{x_token_stride, x_head_stride}, sg{dy_token_stride, dy_head_stride},
      sd{dx_token_stride, dx_head_stride};
  if (sx.token < 0 || sx.head < 0 || sg.token < 0 || sg.head < 0 || sd.token < 0 || sd.head < 0)
    return GEMM_ERR_INVALID_ARG;
  if (d_query_weight && d_query_weight == d_key_weight) return GEMM_ERR_INVALID_ARG;
  if (!aligned(d_query_weight, 4) || !aligned(d_key_weight, 4)) return GEMM_ERR_UNSUPPORTED;
  bool work;
  gemm_status_t st = check_heads(tokens, heads, dim, dtype, norm, r, &work);
  if (st != GEMM_OK) return st;
  if (meet({d_query_weight, 4 * dim}, {d_key_weight, 4 * dim})) return GEMM_ERR_INVALID_ARG;
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  if (!work) {  // sums of nothing
    for (float* w : {d_query_weight, d_key_weight})
      if (w && dim > 0 && st == GEMM_OK)
        st = launched(h, cudaMemsetAsync(w, 0, (size_t)dim * sizeof(float), stream));
    return st;
  }
  if (!x || !dy || !dx || (dy == dx && differ(sg, sd, tokens, heads)) || x == dx) return GEMM_ERR_INVALID_ARG;
  if (!good_result(sd, tokens, heads, dim)) return GEMM_ERR_INVALID_ARG;
  const Vectors mx = memory_of({x, sx}, tokens, heads, dim, dtype), mg = memory_of({dy, sg}, tokens, heads, dim, dtype),
                md = memory_of({dx, sd}, tokens, heads, dim, dtype);
  if (share_memory(md, mx) || (dy != dx && share_memory(md, mg)) || meets_tables(md, tokens, dim, norm, r))
    return GEMM_ERR_INVALID_ARG;
  for (const float* w : {d_query_weight, d_key_weight}) {
    const Vectors m = {(Vectors::wide) reinterpret_cast<uintptr_t>(w), 1, 0, 1, 0, (Vectors::wide)dim * 4};
    if (w && (share_memory(m, mx) || share_memory(m, mg) || share_memory(m, md) || meets_tables(m, tokens, dim, norm, r)))
      return GEMM_ERR_INVALID_ARG;
  }
  for (const void* q : {x, dy, static_cast<const void*>(dx)})
    if (!aligned(q, (uint64_t)elem_size(dtype))) return GEMM_ERR_UNSUPPORTED;
  HeadsParams p = heads_params(h, tokens, heads, dim, norm, r);
  p.x = x;
  p.dy = dy;
  p.y = dx;
  p.x_token = sx.token, p.x_head = sx.head;
  p.dy_token = sg.token, p.dy_head = sg.head;
  p.y_token = sd.token, p.y_head = sd.head;
  if (d_query_weight || d_key_weight) {
    st = ensure_scratch(h, (size_t)heads_back_ctas(h->sms) * dim * sizeof(float), 0);
    if (st != GEMM_OK) return st;
    p.partial = static_cast<float*>(h->op.ptr);
    p.d_query_weight = d_query_weight;
    p.d_key_weight = d_key_weight;
  }
  const int vec = heads_vector({{x, sx}, {dy, sg}, {dx, sd}}, tokens, heads, dim, dtype, r);
  return launched(h, launch_heads_back(p, dtype, r->pairs == GEMM_PAIRS_NEIGHBOURS, vec, h->sms, stream));
}

gemm_status_t gemm_sample(gemm_handle_t h, const void* logits, int32_t* tokens, int64_t rows, int64_t vocab,
                          int64_t logits_stride, gemm_dtype_t dtype, const gemm_sampling_t* s,
                          gemm_stream_t stream_) {
  if (!h || !s) return GEMM_ERR_INVALID_ARG;
  if (rows < 0 || vocab < 0 || logits_stride < vocab || !valid_dtype(dtype)) return GEMM_ERR_INVALID_ARG;
  if (is_fp8(dtype)) return GEMM_ERR_UNSUPPORTED;
  if (rows == 0) return GEMM_OK;
  if (vocab == 0 || !logits || !tokens || !s->random) return GEMM_ERR_INVALID_ARG;
  if (vocab > kMaxSampleVocab || rows > (int64_t(1) << 24)) return GEMM_ERR_UNSUPPORTED;
  if (!aligned(logits, (uint64_t)elem_size(dtype)) || !aligned(tokens, 4) || !aligned(s->random, 4) ||
      !aligned(s->temperature, 4) || !aligned(s->top_k, 4) || !aligned(s->top_p, 4) ||
      !aligned(s->min_p, 4) || !aligned(s->probs, 4))
    return GEMM_ERR_UNSUPPORTED;
  const int64_t vec = 4 * rows;
  if (outputs_overlap({{tokens, vec}, {s->probs, vec}},
                      {{logits, ((rows - 1) * logits_stride + vocab) * elem_size(dtype)}, {s->random, vec},
                       {s->temperature, vec}, {s->top_k, vec}, {s->top_p, vec}, {s->min_p, vec}}))
    return GEMM_ERR_INVALID_ARG;
  SampleParams p;
  std::memset(&p, 0, sizeof(p));
  p.logits = logits;
  p.stride = logits_stride;
  p.rows = (int32_t)rows;
  p.vocab = (int32_t)vocab;
  p.temperature = s->temperature;
  p.top_k = s->top_k;
  p.top_p = s->top_p;
  p.min_p = s->min_p;
  p.random = s->random;
  p.tokens = tokens;
  p.probs = s->probs;
  return launched(h, launch_sample(p, dtype, h->sms, reinterpret_cast<cudaStream_t>(stream_)));
}

gemm_status_t gemm_sample_packed(const gemm_sample_call_t* c) {
  if (!c) return GEMM_ERR_INVALID_ARG;
  return gemm_sample(c->h, c->logits, c->tokens, c->rows, c->vocab, c->logits_stride,
                     static_cast<gemm_dtype_t>(c->dtype), &c->sampling, c->stream);
}

gemm_status_t gemm_norm_rotary_packed(const gemm_norm_rotary_call_t* c) {
  if (!c) return GEMM_ERR_INVALID_ARG;
  gemm_rotary_t r = c->rotary;
  if (c->axes_follow) r.pair_axis = reinterpret_cast<const uint8_t*>(c + 1);
  return gemm_norm_rotary(c->h, c->x, c->y, c->tokens, c->heads, c->dim, c->x_token_stride,
                          c->x_head_stride, c->y_token_stride, c->y_head_stride,
                          static_cast<gemm_dtype_t>(c->dtype), &c->norm, &r, c->stream);
}

gemm_status_t gemm_norm_rotary_grad_packed(const gemm_norm_rotary_grad_call_t* c) {
  if (!c) return GEMM_ERR_INVALID_ARG;
  gemm_rotary_t r = c->rotary;
  if (c->axes_follow) r.pair_axis = reinterpret_cast<const uint8_t*>(c + 1);
  return gemm_norm_rotary_grad(c->h, c->x, c->dy, c->dx, c->tokens, c->heads, c->dim,
                               c->x_token_stride, c->x_head_stride, c->dy_token_stride,
                               c->dy_head_stride, c->dx_token_stride, c->dx_head_stride,
                               static_cast<gemm_dtype_t>(c->dtype), &c->norm, &r, c->d_query_weight,
                               c->d_key_weight, c->stream);
}

gemm_status_t gemm_run_gated_packed(const gemm_gated_call_t* c) {
  if (!c) return GEMM_ERR_INVALID_ARG;
  return gemm_run_gated(c->h, c->X, c->gate_weight, c->up_weight, c->H, c->M, c->N, c->K,
                        static_cast<gemm_dtype_t>(c->dtype), &c->gated, c->stream);
}

gemm_status_t gemm_run_gated_grad_packed(const gemm_gated_grad_call_t* c) {
  if (!c) return GEMM_ERR_INVALID_ARG;
  return gemm_run_gated_grad(c->h, c->X, c->gate_weight, c->up_weight, c->M, c->N, c->K,
                             static_cast<gemm_dtype_t>(c->dtype), &c->grad, c->stream);
}

}  // extern "C"
