// C ABI of the operators around the projections (declared in include/gemm.h):
// gemm_run_adapters, gemm_rotary and gemm_adjust_logits.  Argument validation,
// workspace and launches; the kernels are in adapters_few_kernel.cu, adapters_kernel.cu (and
// gemm_kernel.cuh, ADAPT), rotary_kernel.cu and logits_kernel.cu.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <cstring>
#include <utility>

#include "context.h"
#include "gemm.h"
#include "operators.h"
#include "umma.cuh"

using namespace gb300;

namespace {

bool valid_dtype(int d) { return d >= GEMM_F16 && d <= GEMM_E5M2; }
bool is_fp8(int d) { return d == GEMM_E4M3 || d == GEMM_E5M2; }
int64_t elem_size(int d) { return d == GEMM_F32 ? 4 : 2; }
bool aligned(const void* p, uint64_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
size_t round_up(size_t n) { return (n + 255) & ~(size_t)255; }

// The handle's scratch for these operators, grown on demand; its counters are zero between
// calls.
gemm_status_t ensure_scratch(gemm_ctx* h, size_t bytes, size_t counters) {
  const gemm_status_t st = h->op.grow(bytes, false);
  return st != GEMM_OK ? st : h->op_ctr.grow(counters * sizeof(uint32_t), true);
}

// What the shared product of a call takes in place of gemm_run's choices.  Binary32 results:
// accumulation chains of K 256.  The tensor cores' error grows with a chain's length; at the
// default K 4096 it was 1.2e-6 of the result (relative Frobenius), where sums in binary32 have
// 2.4e-7.  16-bit results round by 1000 times that.  For few rows, the rows of Down that are
// streamed beside the product and the pitch of its result.
constexpr int kShortChain = 4;  // K blocks
struct ProductRules {
  gemm_ctx* h;
  ProductRules(gemm_ctx* h_, bool f32) : h(h_) {
    h->short_chains = f32 ? kShortChain : 0;
  }
  ~ProductRules() { h->short_chains = 0, h->beside_rows = 0, h->c_pitch = 0; }
};

bool nothing_forced(const gemm_ctx* h) {
  const gemm_config_t& f = h->forced;
  return !f.variant && !f.block_n && !f.splits && !f.stages && !f.epilogue && !f.swap_ab &&
         !f.max_ctas;
}

// Whether the kernels for few rows serve the call, or 256 x 256 tiles with the adapters' term
// in their last MMAs.  The first cost about the same however the rows are mixed, but their
// binary32 product goes through memory; the second's cost grows with the adapters that a
// tile's rows name, which the host does not see.  Up to 512 rows the first (256 x 4096 x
// 4096, 8 adapters of rank 16, us: 20 against 28 for the tiles; 256 x 8192 x 8192 39 and 48;
// 512 x 4096 x 4096, 16 of rank 64, mixed 36 and 52), except more than 128 rows and a small
// pool beside a product whose tiles occupy more than half of the CTA pairs without K slices
// (256 x 10240 x 8192, 2 of rank 64 56 and 46, 4 of rank 128 59 and 51, 8 of rank 16 48 and
// 48; 512 x 10240 x 8192, 8 of rank 64 97 and 78; 256 x 14336 x 4096, 8 of rank 16 37 and
// 33).  Up to 2048 rows the first for a large pool (1024 x 8192 x 8192, 64 of rank 16, mixed
// 126 and 214, sorted 112 and 119; 64 of rank 64 221 and 336, 183 and 145; 1024 x 2048 x
// 2048, 64 of rank 16 25 and 66, 25 and 27), and for a small one the second (24 of rank 64
// 175 and 186, 172 and 119).
bool takes_few_rows(const gemm_ctx* h, int64_t M, int64_t N, const gemm_adapters_t* ad) {
  if (M > kFewRows) return M <= kFewRowsLargePool && ad->count > kLargePool;
  const bool wide = M > kAdapterRows && 4 * ceil_div(M, 256) * ceil_div(N, 256) > h->sms;
  return !(wide && nothing_forced(h) && ad->count <= 8 && ad->count * ad->rank <= 512);
}

// Whether two of n1 x n2 vectors of `dim` elements, s1 and s2 elements apart, share an element
// (n1 and n2 at least 1).
bool overlap(int64_t n1, int64_t s1, int64_t n2, int64_t s2, int64_t dim) {
  if (n1 == 1) std::swap(n1, n2), std::swap(s1, s2);  // (of a single one the stride does not count)
  if (n2 == 1) return n1 > 1 && s1 < dim;
  if (s1 > s2) std::swap(n1, n2), std::swap(s1, s2);
  if (s1 < dim) return true;
  // j steps of s2 against the nearest numbers of steps of s1, as far as those reach
  using wide = __int128;
  const wide reach = (wide)(n1 - 1) * s1 + dim;
  for (int64_t j = 1; j < n2 && (wide)j * s2 < reach; ++j) {
    const wide at = (wide)j * s2, past = at % s1;
    if (past < dim || (at / s1 + 1 < n1 && s1 - past < dim)) return true;
  }
  return false;
}

gemm_status_t launched(gemm_ctx* h, cudaError_t e) {
  h->last_cuda = e;
  if (e == cudaSuccess) return GEMM_OK;
  cudaGetLastError();
  return GEMM_ERR_CUDA;
}

}  // namespace

extern "C" {

gemm_status_t gemm_run_adapters(gemm_handle_t h, const void* X, const void* W, void* Y, int64_t M,
                                int64_t N, int64_t K, gemm_dtype_t dtype_in,
                                gemm_dtype_t dtype_out, const gemm_adapters_t* ad,
                                const int32_t* row_adapter, gemm_stream_t stream_) {
  if (!h || !ad) return GEMM_ERR_INVALID_ARG;
  if (M < 0 || N < 0 || K < 0 || ad->count < 0 || ad->rank < 1) return GEMM_ERR_INVALID_ARG;
  if (!valid_dtype(dtype_in) || !valid_dtype(dtype_out)) return GEMM_ERR_INVALID_ARG;
  if (dtype_in == GEMM_F32 || is_fp8(dtype_in) || is_fp8(dtype_out)) return GEMM_ERR_UNSUPPORTED;
  if (ad->rank % 8 || ad->rank > kMaxRank) return GEMM_ERR_UNSUPPORTED;
  if (M == 0 || N == 0) return GEMM_OK;
  if (!row_adapter || !Y || (K > 0 && (!X || !W))) return GEMM_ERR_INVALID_ARG;
  if (ad->count > 0 && K > 0 && (!ad->down || !ad->up)) return GEMM_ERR_INVALID_ARG;
  if (M > INT32_MAX - 2 * kAdapterRows || N > INT32_MAX || K > INT32_MAX)
    return GEMM_ERR_UNSUPPORTED;
  if (!aligned(row_adapter, 4) || !aligned(Y, (uint64_t)elem_size(dtype_out))) return GEMM_ERR_UNSUPPORTED;
  if (K == 0 || ad->count == 0)  // nothing to add: the product itself
    return gemm_run(h, X, W, Y, M, N, K, dtype_in, dtype_out, stream_);
  if (K % 8 || !aligned(X, 16) || !aligned(W, 16) || !aligned(ad->down, 16) ||
      !aligned(ad->up, 16) || !aligned(ad->scale, 4))
    return GEMM_ERR_UNSUPPORTED;
  if ((int64_t)ad->count * ad->rank > INT32_MAX || (int64_t)ad->count * N > INT32_MAX - 256)
    return GEMM_ERR_UNSUPPORTED;
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);

  const ProductRules rules(h, dtype_out == GEMM_F32);
  if (takes_few_rows(h, M, N, ad)) {
    AdapterFewParams f;
    std::memset(&f, 0, sizeof(f));
    f.slices = few_slices((int32_t)M, (int32_t)K, ad->rank, ad->count, h->sms);
    // The binary32 product lies in Y where Y can hold it, else in the scratch: rows of
    // 16-byte multiples, which TMA writes and few_up reads 16 bytes at a time (148 x 9302 x
    // 2056, rank 128, binary32: 41 us against 52.5).
    const bool base_in_y = dtype_out == GEMM_F32 && (N % 4 == 0 || !nothing_forced(h));
    f.base_pitch = base_in_y || !nothing_forced(h) ? N : ceil_div(N, 4) * 4;
    const size_t base_bytes = base_in_y ? 0 : round_up((size_t)M * f.base_pitch * sizeof(float));
    const size_t part_bytes = round_up((size_t)M * f.slices * ad->rank * sizeof(float));
    gemm_status_t st = ensure_scratch(
        h, base_bytes + part_bytes + (size_t)M * sizeof(FewGroup), 2);
    if (st != GEMM_OK) return st;
    char* scratch = static_cast<char*>(h->op.ptr);
    void* base = base_in_y ? Y : scratch;
    h->beside_rows = few_down_rows((int32_t)M, ad->rank, ad->count);
    if (f.base_pitch != N) h->c_pitch = f.base_pitch;
    st = gemm_run(h, X, W, base, M, N, K, dtype_in, GEMM_F32, stream_);
    if (st != GEMM_OK) return st;
    f.X = X;
    f.down = ad->down;
    f.up = ad->up;
    f.scale = ad->scale;
    f.row_adapter = row_adapter;
    f.M = (int32_t)M;
    f.N = (int32_t)N;
    f.K = (int32_t)K;
    f.rank = ad->rank;
    f.count = ad->count;
    f.vec_store = aligned(Y, 16) && N % 8 == 0;
    f.vec_base = aligned(base, 16) && f.base_pitch % 4 == 0;
    f.partial = reinterpret_cast<float*>(scratch + base_bytes);
    f.groups = reinterpret_cast<FewGroup*>(scratch + base_bytes + part_bytes);
    f.counts = static_cast<uint32_t*>(h->op_ctr.ptr);
    f.base = static_cast<const float*>(base);
    f.Y = Y;
    f.status = h->d_status;
    return launched(h, launch_adapter_few(f, dtype_in, dtype_out, h->sms, stream));
  }

  // Many rows: u of every row and the tiles' adapters first, then the product with the
  // adapters' term appended to its tiles.
  AdapterParams p;
  std::memset(&p, 0, sizeof(p));
  p.scale = ad->scale;
  p.row_adapter = row_adapter;
  p.M = (int32_t)M;
  p.N = (int32_t)N;
  p.K = (int32_t)K;
  p.rank = ad->rank;
  p.count = ad->count;
  p.tiles = (int32_t)ceil_div(M, kAdapterRows);
  p.k_blocks = (int32_t)ceil_div(K, kBlockK);
  // As many CTAs per row tile as two on every SM allow (a cluster), each at least four K
  // blocks of one group of adapters.
  const int64_t groups = ceil_div(std::min<int64_t>(kAdapterRows, ad->count), kAdapterCols / p.rank);
  p.max_splits = (int32_t)std::max<int64_t>(1, p.k_blocks / 4);
  p.ctas = 1;
  while (p.ctas < 8 && (int64_t)2 * p.ctas * p.tiles <= 2 * h->sms && p.ctas < groups * p.max_splits)
    p.ctas *= 2;
  p.idesc = idesc_f16_kmajor(kAdapterRows, 0, dtype_in == GEMM_BF16);
  p.status = h->d_status;
  p.wait_limit_ns = h->wait_limit_ns;
  p.test_stall = h->test_stall;
  p.f32_out = dtype_out == GEMM_F32;
  p.parts = u_parts(dtype_in == GEMM_BF16, dtype_out == GEMM_F32);
  const bool windows = dtype_in == GEMM_F16;
  const int64_t pairs = ceil_div(p.tiles, 2);
  const int64_t u_cols = (windows ? 2 : 1) * p.parts * kBlockK * ceil_div(p.rank, kBlockK);
  const size_t u_bytes = round_up((size_t)M * u_cols * 2);
  const size_t scale_bytes = round_up((size_t)M * sizeof(float));
  const size_t pair_bytes = round_up((size_t)pairs * sizeof(AdapterTile));
  const size_t low_bytes = windows ? round_up((size_t)p.tiles * kAdaptCtas * sizeof(uint32_t)) : 0;
  gemm_status_t st = ensure_scratch(
      h, u_bytes + 2 * scale_bytes + pair_bytes + low_bytes + (size_t)M * p.rank * sizeof(float), 0);
  if (st != GEMM_OK) return st;
  char* scratch = static_cast<char*>(h->op.ptr);
  p.U = scratch;
  p.row_scale = reinterpret_cast<float*>(scratch + u_bytes);
  p.row_scale_low = reinterpret_cast<float*>(scratch + u_bytes + scale_bytes);
  p.pairs = reinterpret_cast<AdapterTile*>(scratch + u_bytes + 2 * scale_bytes);
  p.low = windows ? reinterpret_cast<uint32_t*>(scratch + u_bytes + 2 * scale_bytes + pair_bytes) : nullptr;
  p.u = reinterpret_cast<float*>(scratch + u_bytes + 2 * scale_bytes + pair_bytes + low_bytes);

  CUtensorMap tmX, tmDown;
  AdaptParams<true> g;
  if (!make_map(h, X, M, K, dtype_in, kAdapterRows, &tmX) ||
      !make_map(h, ad->down, (int64_t)ad->count * p.rank, K, dtype_in, p.rank, &tmDown) ||
      !make_map(h, p.U, M, u_cols, dtype_in, kBlockM, &g.tmU) ||
      !make_map(h, ad->up, (int64_t)ad->count * N, p.rank, dtype_in, 128, &g.tmUp) ||
      !make_map(h, ad->up, (int64_t)ad->count * N, p.rank, dtype_in, 64, &g.tmUpHalf))
    return GEMM_ERR_CUDA;
  g.tiles = p.pairs;
  g.row_scale = p.row_scale;
  g.row_scale_low = p.row_scale_low;
  g.low = p.low;
  g.low_tiles = p.tiles;
  g.low_ctas = p.ctas;
  g.u = p.u;
  g.up = ad->up;
  g.row_adapter = row_adapter;
  g.bf16 = dtype_in == GEMM_BF16;
  g.rank = p.rank;
  g.parts = p.parts;
  // (the product's configuration is settled before anything is queued)
  return run_adapted(h, X, W, Y, M, N, K, dtype_in, dtype_out, g,
                     [&] { return launch_adapter_down(tmX, tmDown, p, dtype_in, stream); }, stream_);
}

gemm_status_t gemm_rotary(gemm_handle_t h, const void* x, void* y, int64_t tokens, int64_t heads,
                          int64_t dim, int64_t x_token_stride, int64_t x_head_stride,
                          int64_t y_token_stride, int64_t y_head_stride, gemm_dtype_t dtype,
                          const gemm_rotary_t* r, gemm_stream_t stream_) {
  if (!h || !r) return GEMM_ERR_INVALID_ARG;
  if (tokens < 0 || heads < 0 || dim < 0 || x_token_stride < 0 || x_head_stride < 0 ||
      y_token_stride < 0 || y_head_stride < 0)
    return GEMM_ERR_INVALID_ARG;
  if (!valid_dtype(dtype)) return GEMM_ERR_INVALID_ARG;
  if (is_fp8(dtype)) return GEMM_ERR_UNSUPPORTED;
  if (tokens == 0 || heads == 0 || dim == 0) return GEMM_OK;
  if (r->axes < 1 || r->axes > 8 || r->rot_dim < 2 || r->rot_dim % 2 || r->rot_dim > dim ||
      r->rot_dim > 2 * kMaxPairs || r->num_positions < 1 ||
      (r->pairs != GEMM_PAIRS_HALF && r->pairs != GEMM_PAIRS_NEIGHBOURS) ||
      (r->inverse != 0 && r->inverse != 1))
    return GEMM_ERR_INVALID_ARG;
  if (!x || !y || !r->cos || !r->sin || !r->positions) return GEMM_ERR_INVALID_ARG;
  // in place with other strides, where there are two tokens or heads for them to set apart
  if (x == y && ((tokens > 1 && x_token_stride != y_token_stride) ||
                 (heads > 1 && x_head_stride != y_head_stride)))
    return GEMM_ERR_INVALID_ARG;
  const int half = r->rot_dim / 2;
  if (r->pair_axis)
    for (int i = 0; i < half; ++i)
      if (r->pair_axis[i] >= r->axes) return GEMM_ERR_INVALID_ARG;
  const int64_t esz = elem_size(dtype);
  if (tokens > INT32_MAX || heads > INT32_MAX || dim > INT32_MAX || tokens > INT32_MAX / heads)
    return GEMM_ERR_UNSUPPORTED;
  if (!aligned(x, (uint64_t)esz) || !aligned(y, (uint64_t)esz) || !aligned(r->cos, 4) ||
      !aligned(r->sin, 4) || !aligned(r->positions, 4))
    return GEMM_ERR_UNSUPPORTED;

  if (overlap(tokens, y_token_stride, heads, y_head_stride, dim)) return GEMM_ERR_INVALID_ARG;

  RotaryParams p;
  std::memset(&p, 0, sizeof(p));
  p.x = x;
  p.y = y;
  p.x_token = x_token_stride;
  p.x_head = x_head_stride;
  p.y_token = y_token_stride;
  p.y_head = y_head_stride;
  p.tokens = (int32_t)tokens;
  p.heads = (int32_t)heads;
  p.dim = (int32_t)dim;
  p.half = half;
  p.inverse = r->inverse;
  p.cos = r->cos;
  p.sin = r->sin;
  p.positions = r->positions;
  p.num_positions = r->num_positions;
  p.status = h->d_status;
  if (r->pair_axis) std::memcpy(p.pair_axis, r->pair_axis, (size_t)half);
  // Vectors of 16 bytes: every head starts on a boundary, and the halves (or the pairs'
  // end) and the head's end fall on one.
  const bool neigh = r->pairs == GEMM_PAIRS_NEIGHBOURS;
  const int64_t v = rotary_vector(dtype);
  const bool vec = aligned(x, 16) && aligned(y, 16) && half % 4 == 0 &&
                   (x_token_stride | x_head_stride | y_token_stride | y_head_stride) % v == 0 &&
                   (neigh ? 2 * half : half) % v == 0 && (dim - 2 * half) % v == 0;
  return launched(h, launch_rotary(p, dtype, neigh, vec, h->sms, reinterpret_cast<cudaStream_t>(stream_)));
}

gemm_status_t gemm_adjust_logits(gemm_handle_t h, const void* logits, void* out, int64_t rows,
                                 int64_t vocab, int64_t logits_stride, int64_t out_stride,
                                 gemm_dtype_t dtype_in, gemm_dtype_t dtype_out,
                                 const gemm_logits_t* a, gemm_stream_t stream_) {
  if (!h || !a) return GEMM_ERR_INVALID_ARG;
  if (rows < 0 || vocab < 0 || logits_stride < vocab || out_stride < vocab) return GEMM_ERR_INVALID_ARG;
  if (!valid_dtype(dtype_in) || !valid_dtype(dtype_out)) return GEMM_ERR_INVALID_ARG;
  if (is_fp8(dtype_in) || is_fp8(dtype_out)) return GEMM_ERR_UNSUPPORTED;
  if (rows == 0 || vocab == 0) return GEMM_OK;
  if (!logits || !out) return GEMM_ERR_INVALID_ARG;
  if (a->tokens && !a->token_start) return GEMM_ERR_INVALID_ARG;
  if (a->bias_tokens && (!a->bias_values || !a->bias_start)) return GEMM_ERR_INVALID_ARG;
  if (a->mask && (a->mask_stride < (vocab + 31) / 32 || a->mask_count < 1 ||
                  (!a->mask_row && a->mask_count < rows)))
    return GEMM_ERR_INVALID_ARG;
  if (logits == out && (dtype_in != dtype_out || logits_stride != out_stride)) return GEMM_ERR_INVALID_ARG;
  if (vocab > (int64_t(1) << 30) || rows > (int64_t(1) << 24)) return GEMM_ERR_UNSUPPORTED;
  if (rows * (vocab / 8192 + 2) > INT32_MAX) return GEMM_ERR_UNSUPPORTED;  // the grid
  if (!aligned(logits, (uint64_t)elem_size(dtype_in)) || !aligned(out, (uint64_t)elem_size(dtype_out)) ||
      !aligned(a->tokens, 4) || !aligned(a->token_start, 8) || !aligned(a->prompt_len, 4) ||
      !aligned(a->repetition, 4) || !aligned(a->frequency, 4) || !aligned(a->presence, 4) ||
      !aligned(a->bias_tokens, 4) || !aligned(a->bias_values, 4) || !aligned(a->bias_start, 8) ||
      !aligned(a->mask, 4) || !aligned(a->mask_row, 4))
    return GEMM_ERR_UNSUPPORTED;
  LogitsParams p;
  std::memset(&p, 0, sizeof(p));
  p.in = logits;
  p.out = out;
  p.in_stride = logits_stride;
  p.out_stride = out_stride;
  p.rows = (int32_t)rows;
  p.vocab = (int32_t)vocab;
  p.tokens = a->tokens;
  p.token_start = a->token_start;
  p.prompt_len = a->prompt_len;
  p.repetition = a->repetition;
  p.frequency = a->frequency;
  p.presence = a->presence;
  p.bias_tokens = a->bias_tokens;
  p.bias_values = a->bias_values;
  p.bias_start = a->bias_start;
  p.mask = a->mask;
  p.mask_stride = a->mask_stride;
  p.mask_count = a->mask_count;
  p.mask_row = a->mask_row;
  p.status = h->d_status;
  return launched(h, launch_logits(p, dtype_in, dtype_out, h->sms, reinterpret_cast<cudaStream_t>(stream_)));
}

gemm_status_t gemm_run_adapters_packed(const gemm_adapters_call_t* c) {
  if (!c) return GEMM_ERR_INVALID_ARG;
  return gemm_run_adapters(c->h, c->X, c->W, c->Y, c->M, c->N, c->K,
                           static_cast<gemm_dtype_t>(c->dtype_in),
                           static_cast<gemm_dtype_t>(c->dtype_out), &c->adapters, c->row_adapter,
                           c->stream);
}

gemm_status_t gemm_rotary_packed(const gemm_rotary_call_t* c) {
  if (!c) return GEMM_ERR_INVALID_ARG;
  gemm_rotary_t r = c->rotary;
  if (c->axes_follow) r.pair_axis = reinterpret_cast<const uint8_t*>(c + 1);
  return gemm_rotary(c->h, c->x, c->y, c->tokens, c->heads, c->dim, c->x_token_stride,
                     c->x_head_stride, c->y_token_stride, c->y_head_stride,
                     static_cast<gemm_dtype_t>(c->dtype), &r, c->stream);
}

gemm_status_t gemm_adjust_logits_packed(const gemm_logits_call_t* c) {
  if (!c) return GEMM_ERR_INVALID_ARG;
  return gemm_adjust_logits(c->h, c->logits, c->out, c->rows, c->vocab, c->logits_stride,
                            c->out_stride, static_cast<gemm_dtype_t>(c->dtype_in),
                            static_cast<gemm_dtype_t>(c->dtype_out), &c->adjust, c->stream);
}

}  // extern "C"
