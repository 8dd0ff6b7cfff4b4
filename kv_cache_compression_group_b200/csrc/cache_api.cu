// Host side of the paged cache's C ABI: argument checks and launches.
#include <cmath>

#include "jolt.h"
#include "common.cuh"
#include "host.cuh"
#include "cache.cuh"
#include "cache_launch.cuh"

using namespace jolt;

namespace {

constexpr int MOST = 1 << 30;   // rows or sequences of a batch, tokens of a sequence

bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

jolt_status cache_args(const jolt_cache* c, const jolt_cache_batch* b, CacheArgs* ca, BatchArgs* ba) {
  if (!c || !b) return fail(JOLT_ERR_INVALID_ARG, "null cache or batch");
  if (c->head_dim != 64 && c->head_dim != 128)
    return fail(JOLT_ERR_UNSUPPORTED_SHAPE, "cache head_dim %d not in {64, 128}", c->head_dim);
  if (c->n_heads < 1 || c->n_heads > 65535) return fail(JOLT_ERR_INVALID_ARG, "n_heads %d", c->n_heads);
  if (c->page_size < 16 || c->page_size > 4096 || (c->page_size & (c->page_size - 1)))
    return fail(JOLT_ERR_UNSUPPORTED_SHAPE, "page_size %d is not a power of two in [16, 4096]", c->page_size);
  if (c->n_pages < 1) return fail(JOLT_ERR_INVALID_ARG, "n_pages %d", c->n_pages);
  if ((long long)c->n_pages * c->page_size * c->n_heads >= 1LL << 31)
    return fail(JOLT_ERR_UNSUPPORTED_SHAPE, "a pool of %d pages has 2^31 rows or more", c->n_pages);
  for (int bits : {c->bits_k, c->bits_v})
    if (bits != 2 && bits != 4 && bits != 8)
      return fail(JOLT_ERR_UNSUPPORTED_SHAPE, "cache bits %d not in {2, 4, 8}", bits);
  if (!c->k_codes_dev || !c->k_scales_dev || !c->v_codes_dev || !c->v_scales_dev)
    return fail(JOLT_ERR_INVALID_ARG, "null cache pool");
  if (!aligned16(c->k_codes_dev) || !aligned16(c->k_scales_dev) || !aligned16(c->v_codes_dev) ||
      !aligned16(c->v_scales_dev))
    return fail(JOLT_ERR_INVALID_ARG, "cache pools must be 16-byte aligned");
  if (b->n_seqs < 0 || b->max_pages < 0 || b->max_new < 0 || b->n_rows < 0)
    return fail(JOLT_ERR_INVALID_ARG, "negative batch size");
  // a block's or a warp's first row, and the step behind the last sequence, stay ints
  if (b->n_seqs > MOST || b->n_rows > MOST)
    return fail(JOLT_ERR_UNSUPPORTED_SHAPE, "a batch of %d sequences and %d rows; at most 2^30", b->n_seqs, b->n_rows);
  // a sequence's length rounded up to whole units of tokens stays an int
  if ((long long)b->max_pages * c->page_size > MOST)
    return fail(JOLT_ERR_UNSUPPORTED_SHAPE, "%d pages of %d tokens hold more than 2^30", b->max_pages, c->page_size);
  if (b->n_seqs > 0 && (!b->page_table_dev || !b->lens_dev || !b->starts_dev || !b->status_dev))
    return fail(JOLT_ERR_INVALID_ARG, "null batch array");
  ca->codes[0] = (unsigned char*)c->k_codes_dev;
  ca->codes[1] = (unsigned char*)c->v_codes_dev;
  ca->scales[0] = (__half2*)c->k_scales_dev;
  ca->scales[1] = (__half2*)c->v_scales_dev;
  ca->bits[0] = c->bits_k;
  ca->bits[1] = c->bits_v;
  ca->H = c->n_heads;
  ca->D = c->head_dim;
  ca->n_pages = c->n_pages;
  ca->page_shift = 0;
  while ((1 << ca->page_shift) < c->page_size) ++ca->page_shift;
  ba->table = b->page_table_dev;
  ba->lens = b->lens_dev;
  ba->starts = b->starts_dev;
  ba->B = b->n_seqs;
  ba->max_pages = b->max_pages;
  ba->max_new = b->max_new;
  ba->rows = b->n_rows;
  ba->status = b->status_dev;
  return JOLT_OK;
}

template <typename T>
RowsArgs<T> rows_args(T* k, T* v, int64_t kr, int64_t kh, int64_t vr, int64_t vh) {
  const int64_t per = 16 / sizeof(T);
  RowsArgs<T> x{};
  x.x[0] = k;
  x.x[1] = v;
  x.row[0] = kr;
  x.row[1] = vr;
  x.head[0] = kh;
  x.head[1] = vh;
  x.vec[0] = aligned16(k) && kr % per == 0 && kh % per == 0;
  x.vec[1] = aligned16(v) && vr % per == 0 && vh % per == 0;
  return x;
}

// rows of a warp: enough that what is found once per warp is spread over several, few enough that
// every SM has its warps
template <typename T>
dim3 rows_grid(const CacheArgs& c, const BatchArgs& a, RowsArgs<T>* x) {
  const long long groups = ceil_div(c.H, 512 / c.D), fit = (long long)a.rows * groups * 2 / (148 * 48);
  x->per_warp = (int)(fit < 1 ? 1 : fit > 8 ? 8 : fit);
  return dim3((unsigned)ceil_div(a.rows, ROW_WARPS * x->per_warp), (unsigned)groups, 2);
}

template <typename T>
jolt_status launch_write(const CacheArgs& c, const BatchArgs& a, RowsArgs<const T> x, cudaStream_t st) {
  const dim3 grid = rows_grid(c, a, &x);
  if (c.D == 64) CUDA_TRY(launch_after(cache_write_kernel<T, 64>, grid, ROW_WARPS * 32, 0, st, c, a, x));
  else CUDA_TRY(launch_after(cache_write_kernel<T, 128>, grid, ROW_WARPS * 32, 0, st, c, a, x));
  return JOLT_OK;
}

template <typename T>
jolt_status launch_read(const CacheArgs& c, const BatchArgs& a, RowsArgs<T> x, cudaStream_t st) {
  const dim3 grid = rows_grid(c, a, &x);
  if (c.D == 64) CUDA_TRY(launch_after(cache_read_kernel<T, 64>, grid, ROW_WARPS * 32, 0, st, c, a, x));
  else CUDA_TRY(launch_after(cache_read_kernel<T, 128>, grid, ROW_WARPS * 32, 0, st, c, a, x));
  return JOLT_OK;
}

struct Scratch {
  size_t notes, pieces, total;
};
Scratch attend_scratch(const CacheArgs& c, const BatchArgs& a, int nq) {
  const long long rows = (long long)a.max_new * (nq / c.H);
  const size_t blocks = scratch_blocks(rows), tile = scratch_rows(rows);
  Scratch s;
  Bump m;
  s.notes = m.take(sizeof(int4) * blocks);
  s.pieces = m.take(sizeof(float) * 2 * blocks * tile * (c.D + 4));
  s.total = m.off;
  return s;
}

template <int D>
jolt_status launch_cache_attend(const CacheAttendArgs& A, cudaStream_t st) {
  const long long rows = (long long)A.a.max_new * A.G;
  if (rows <= FEW_ROWS) return launch_few_rows<D>(A, st);
  return launch_many_rows<D>(A, rows > 128, st);
}

}  // namespace

extern "C" {

jolt_status jolt_cache_write(const jolt_cache* cache, const jolt_cache_batch* batch, const void* k_dev,
                             const void* v_dev, int32_t dtype, int64_t k_row_stride, int64_t k_head_stride,
                             int64_t v_row_stride, int64_t v_head_stride, void* stream) {
  CacheArgs c;
  BatchArgs a;
  JTRY(cache_args(cache, batch, &c, &a));
  if (dtype != JOLT_BF16 && dtype != JOLT_F32 && dtype != JOLT_F16) return fail(JOLT_ERR_INVALID_ARG, "dtype %d", dtype);
  if (a.B == 0 || a.rows == 0) return JOLT_OK;
  if (!k_dev || !v_dev) return fail(JOLT_ERR_INVALID_ARG, "null rows");
  cudaStream_t st = (cudaStream_t)stream;
  ProfScope ps("cache_write", st, a.rows);
  if (dtype == JOLT_BF16)
    return launch_write(c, a, rows_args((const bf16*)k_dev, (const bf16*)v_dev, k_row_stride, k_head_stride,
                                        v_row_stride, v_head_stride), st);
  if (dtype == JOLT_F16)
    return launch_write(c, a, rows_args((const __half*)k_dev, (const __half*)v_dev, k_row_stride, k_head_stride,
                                        v_row_stride, v_head_stride), st);
  return launch_write(c, a, rows_args((const float*)k_dev, (const float*)v_dev, k_row_stride, k_head_stride,
                                      v_row_stride, v_head_stride), st);
}

jolt_status jolt_cache_read(const jolt_cache* cache, const jolt_cache_batch* batch, int32_t dtype, void* k_out_dev,
                            void* v_out_dev, int64_t k_row_stride, int64_t k_head_stride, int64_t v_row_stride,
                            int64_t v_head_stride, void* stream) {
  CacheArgs c;
  BatchArgs a;
  JTRY(cache_args(cache, batch, &c, &a));
  if (dtype != JOLT_BF16 && dtype != JOLT_F32 && dtype != JOLT_F16) return fail(JOLT_ERR_INVALID_ARG, "dtype %d", dtype);
  if (a.B == 0 || a.rows == 0) return JOLT_OK;
  if (!k_out_dev || !v_out_dev) return fail(JOLT_ERR_INVALID_ARG, "null rows");
  cudaStream_t st = (cudaStream_t)stream;
  ProfScope ps("cache_read", st, a.rows);
  if (dtype == JOLT_BF16)
    return launch_read(c, a, rows_args((bf16*)k_out_dev, (bf16*)v_out_dev, k_row_stride, k_head_stride, v_row_stride,
                                       v_head_stride), st);
  if (dtype == JOLT_F16)
    return launch_read(c, a, rows_args((__half*)k_out_dev, (__half*)v_out_dev, k_row_stride, k_head_stride,
                                       v_row_stride, v_head_stride), st);
  return launch_read(c, a, rows_args((float*)k_out_dev, (float*)v_out_dev, k_row_stride, k_head_stride, v_row_stride,
                                     v_head_stride), st);
}

jolt_status jolt_cache_attend_scratch_size(const jolt_cache* cache, const jolt_cache_batch* batch, int32_t n_q_heads,
                                           size_t* bytes) {
  CacheArgs c;
  BatchArgs a;
  JTRY(cache_args(cache, batch, &c, &a));
  if (!bytes || n_q_heads < 1 || n_q_heads % c.H) return fail(JOLT_ERR_INVALID_ARG, "n_q_heads %d", n_q_heads);
  if ((long long)a.max_new * (n_q_heads / c.H) > (1 << 30))
    return fail(JOLT_ERR_UNSUPPORTED_SHAPE, "%d new rows of %d query heads", a.max_new, n_q_heads);
  *bytes = attend_scratch(c, a, n_q_heads).total;
  return JOLT_OK;
}

jolt_status jolt_cache_attend(const jolt_cache* cache, const jolt_cache_batch* batch,
                              const jolt_cache_attend_options* opts, const void* q_dev, int32_t dtype,
                              int32_t n_q_heads, int64_t q_row_stride, int64_t q_head_stride, void* out_dev,
                              int64_t out_row_stride, int64_t out_head_stride, void* scratch_dev,
                              size_t scratch_bytes, void* stream) {
  CacheAttendArgs A;
  JTRY(cache_args(cache, batch, &A.c, &A.a));
  if (!opts) return fail(JOLT_ERR_INVALID_ARG, "null options");
  if (dtype != JOLT_BF16 && dtype != JOLT_F16) return fail(JOLT_ERR_INVALID_ARG, "dtype %d of the queries", dtype);
  size_t need = 0;
  JTRY(jolt_cache_attend_scratch_size(cache, batch, n_q_heads, &need));
  if (!(opts->scale >= 0.f) || !(opts->softcap >= 0.f) || std::isinf(opts->scale) || std::isinf(opts->softcap))
    return fail(JOLT_ERR_INVALID_ARG, "scale %g, softcap %g", opts->scale, opts->softcap);
  if (opts->softcap > 0.f && (opts->softcap < 1e-6f || opts->softcap > 1e30f))
    return fail(JOLT_ERR_INVALID_ARG, "softcap %g not in [1e-6, 1e30]", opts->softcap);
  if (opts->window < 0) return fail(JOLT_ERR_INVALID_ARG, "window %d", opts->window);
  if (opts->mask_dev && (opts->mask_words < 1 || opts->mask_words < ceil_div(A.a.max_new, 32)))
    return fail(JOLT_ERR_INVALID_ARG, "mask_words %d for %d new rows", opts->mask_words, A.a.max_new);
  if ((opts->prefix_out_dev == nullptr) != (opts->prefix_lse_dev == nullptr))
    return fail(JOLT_ERR_INVALID_ARG, "give both or neither of prefix_out, prefix_lse");
  if (A.a.B == 0 || A.a.rows == 0 || A.a.max_new == 0) return JOLT_OK;
  if (!q_dev || !out_dev || !scratch_dev) return fail(JOLT_ERR_INVALID_ARG, "null pointer");
  if (scratch_bytes < need)
    return fail(JOLT_ERR_WORKSPACE_TOO_SMALL, "cache attend scratch %zu bytes, need %zu", scratch_bytes, need);
  if (reinterpret_cast<uintptr_t>(scratch_dev) % 256) return fail(JOLT_ERR_INVALID_ARG, "scratch not 256-byte aligned");
  A.nq = n_q_heads;
  A.G = n_q_heads / A.c.H;
  A.scale = opts->scale > 0.f ? opts->scale : (float)(1.0 / sqrt((double)A.c.D));
  A.cap = opts->softcap;
  A.cap_inv = opts->softcap == 0.f ? 0.f : 1.f / opts->softcap;
  A.window = opts->window;
  A.words = opts->mask_words;
  A.slopes = opts->slopes_dev;
  A.positions = opts->positions_dev;
  A.mask = opts->mask_dev;
  A.prefix_out = opts->prefix_out_dev;
  A.prefix_lse = opts->prefix_lse_dev;
  const Scratch at = attend_scratch(A.c, A.a, n_q_heads);
  A.notes = reinterpret_cast<int4*>((unsigned char*)scratch_dev + at.notes);
  A.pieces = reinterpret_cast<float*>((unsigned char*)scratch_dev + at.pieces);
  A.q = q_dev;
  A.q_f16 = dtype == JOLT_F16;
  A.q_row = q_row_stride;
  A.q_head = q_head_stride;
  A.o_vec = aligned16(out_dev) && out_row_stride % 8 == 0 && out_head_stride % 8 == 0;
  A.q_vec = aligned16(q_dev) && q_row_stride % 8 == 0 && q_head_stride % 8 == 0;
  A.out = out_dev;
  A.o_row = out_row_stride;
  A.o_head = out_head_stride;
  cudaStream_t st = (cudaStream_t)stream;
  ProfScope ps("cache_attend", st, A.a.rows);
  return A.c.D == 64 ? launch_cache_attend<64>(A, st) : launch_cache_attend<128>(A, st);
}

jolt_status jolt_cache_check(const uint32_t* status_dev, void* stream) {
  if (!status_dev) return fail(JOLT_ERR_INVALID_ARG, "null status word");
  uint32_t h = 0;
  cudaStream_t st = (cudaStream_t)stream;
  CUDA_TRY(cudaMemcpyAsync(&h, status_dev, sizeof h, cudaMemcpyDeviceToHost, st));
  CUDA_TRY(cudaStreamSynchronize(st));
  if (h & DEV_ERR_TIMEOUT) return fail(JOLT_ERR_TIMEOUT, "a bounded device-side wait gave up");
  if (h & DEV_ERR_BATCH) return fail(JOLT_ERR_INVALID_ARG, "a batch named rows, lengths or pages that do not exist");
  if (h & DEV_ERR_NONFINITE) return fail(JOLT_ERR_NUMERIC, "NaN or values beyond fp16 among the rows written");
  if (h) return fail(JOLT_ERR_CUDA, "unexpected device status %u", h);
  return JOLT_OK;
}

}  // extern "C"
