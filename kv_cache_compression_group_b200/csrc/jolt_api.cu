// Host side of the JoLT C ABI: argument checks, workspace plan and launch sequences.
#include <cusolverDn.h>

#include <cstdarg>
#include <mutex>
#include <cstdio>
#include <cstring>
#include <string>
#include <vector>

#include "jolt.h"
#include "common.cuh"
#include "host.cuh"
#include "gemm.cuh"
#include "kernels.cuh"
#include "misc.cuh"
#include "umma.cuh"
#include "eig_cluster.cuh"
#include "eig_large.cuh"
#include "chol.cuh"
#include "table_tc.cuh"
#include "attend.cuh"

using namespace jolt;

namespace {

#define SOLVER_TRY(x)                                                               \
  do {                                                                              \
    cusolverStatus_t s_ = (x);                                                      \
    if (s_ != CUSOLVER_STATUS_SUCCESS) return fail(JOLT_ERR_CUDA, "%s: cusolver status %d", #x, (int)s_); \
  } while (0)
// ------------------------------------------------------------------------------------------
// cuSOLVER handle (one per thread and device)
// ------------------------------------------------------------------------------------------
struct Solver {
  cusolverDnHandle_t h = nullptr;
  cusolverDnParams_t params = nullptr;
  int device = -1;
  std::vector<char> host_ws;
};
thread_local Solver g_solver[2];   // [0]: the caller's stream, [1]: the auxiliary stream

jolt_status solver_get(cudaStream_t st, Solver** out, int idx = 0) {
  int dev = 0;
  CUDA_TRY(cudaGetDevice(&dev));
  Solver& sv = g_solver[idx];
  if (sv.h == nullptr || sv.device != dev) {
    if (sv.h) {
      cusolverDnDestroyParams(sv.params);
      cusolverDnDestroy(sv.h);
    }
    SOLVER_TRY(cusolverDnCreate(&sv.h));
    SOLVER_TRY(cusolverDnCreateParams(&sv.params));
    sv.device = dev;
  }
  SOLVER_TRY(cusolverDnSetStream(sv.h, st));
  *out = &sv;
  return JOLT_OK;
}

// An auxiliary stream (one per host thread and device) on which the feature factor runs
// concurrently with the token factor; fork / join through events on the caller's stream,
// so the pair is legal inside stream capture.
struct Aux {
  cudaStream_t st = nullptr;
  cudaEvent_t fork = nullptr, join = nullptr;
  int device = -1;
};
thread_local Aux g_aux;

jolt_status aux_get(Aux** out) {
  int dev = 0;
  CUDA_TRY(cudaGetDevice(&dev));
  if (g_aux.st == nullptr || g_aux.device != dev) {
    CUDA_TRY(cudaStreamCreateWithFlags(&g_aux.st, cudaStreamNonBlocking));
    CUDA_TRY(cudaEventCreateWithFlags(&g_aux.fork, cudaEventDisableTiming));
    CUDA_TRY(cudaEventCreateWithFlags(&g_aux.join, cudaEventDisableTiming));
    g_aux.device = dev;
  }
  *out = &g_aux;
  return JOLT_OK;
}

// ------------------------------------------------------------------------------------------
// plan: derived sizes and workspace layout
// ------------------------------------------------------------------------------------------
// Cholesky QR runs its Gram and its triangular product on the tensor cores for block widths
// of at least QR_TC_MINK columns; a Gram partial sums QR_TC_CHUNK rows in fp32
constexpr int QR_TC_MINK = 64;
constexpr int QR_TC_CHUNK = 4096;

struct Plan {
  int nL, H, T, D, Lg, S, G, NU, M, dtype;
  Cands cd;
  int nC, rTmax, rDmax, ldU, ldW, ldC, method, q, k, kp;
  int u0;                 // global index of this cache's first unit (RNG streams)
  bool m_side;            // exact token factor through the M x M Gram (T > M)
  int gd_split;           // split-K of the feature Gram
  int gt_split;           // split-K of the token Gram
  size_t solver_dev;      // cuSOLVER device workspace (token factor)
  size_t fsolver_dev;     // cuSOLVER device workspace (feature factor, on the auxiliary stream)
  size_t solver_host;
  // workspace offsets (bytes)
  size_t o_signkey, o_sign, o_ctmp;
  size_t o_status, o_gd_part, o_gd, o_evals, o_Wf, o_Ws, o_Uf, o_Us, o_core, o_zc, o_ptmp, o_P, o_partial,
      o_table, o_bytes, o_choice, o_lambda, o_hdr, o_umap, o_info, o_solver, o_fsolver, o_finfo, o_fevals, o_eigvec, o_eigscr,
      o_feigvec, o_feigscr;
  int eig_n;              // order of the token-side eigen problems solved by the own solver (0: none)
  // token factor scratch (all units)
  size_t o_gt32, o_gt, o_vsel, o_lam, o_omega, o_Y, o_Zm, o_h, o_l, o_gpart, o_G, o_Lr;
  // FlashJoLT on the tensor cores: the T x k bases only as bf16 hi + lo pairs (two pairs,
  // alternating) and the split of the M-side basis
  size_t o_h2, o_l2, o_mh, o_ml;
  size_t o_wth, o_wtl, o_winv, o_vh, o_vl;   // tensor-core Cholesky QR: W^T = L^-T split, fp64 scratch; V split
  int qr_split_max;       // split-K of the Cholesky-QR Grams
  size_t ws_total;
  int tiles;
  size_t blob_max;
  // decompress workspace
  size_t d_U, d_W, d_C, d_ptmp, d_P, d_umap, dws_total;
};

int max_in(const int32_t* v, int n) {
  int m = 0;
  for (int i = 0; i < n; ++i) m = v[i] > m ? v[i] : m;
  return m;
}

jolt_status check_list(const int32_t* v, int n, int lo, int hi, const char* name) {
  if (n < 1 || n > JOLT_MAX_CANDIDATES) return fail(JOLT_ERR_INVALID_ARG, "%s: count %d not in [1, 8]", name, n);
  for (int i = 0; i < n; ++i) {
    if (v[i] < lo || v[i] > hi) return fail(JOLT_ERR_INVALID_ARG, "%s[%d] = %d not in [%d, %d]", name, i, v[i], lo, hi);
    if (i && v[i] <= v[i - 1]) return fail(JOLT_ERR_INVALID_ARG, "%s must be strictly ascending", name);
  }
  return JOLT_OK;
}

jolt_status make_plan(const jolt_shape* sh, const jolt_options* op, Plan* p) {
  if (!sh || !op) return fail(JOLT_ERR_INVALID_ARG, "null shape or options");
  if (sh->dtype != JOLT_BF16 && sh->dtype != JOLT_F32) return fail(JOLT_ERR_INVALID_ARG, "dtype %d", sh->dtype);
  if (sh->n_layers < 1 || sh->n_heads < 1 || sh->n_tokens < 1 || sh->layers_per_group < 1)
    return fail(JOLT_ERR_INVALID_ARG, "non-positive dimension");
  const int D = sh->head_dim;
  if (D != 16 && D != 32 && D != 64 && D != 128)
    return fail(JOLT_ERR_UNSUPPORTED_SHAPE, "head_dim %d not in {16, 32, 64, 128}", D);
  if (sh->n_layers % sh->layers_per_group)
    return fail(JOLT_ERR_UNSUPPORTED_SHAPE, "n_layers %% layers_per_group != 0");
  if (sh->n_tokens % 16) return fail(JOLT_ERR_UNSUPPORTED_SHAPE, "n_tokens %d not a multiple of 16", sh->n_tokens);
  p->nL = sh->n_layers;
  p->H = sh->n_heads;
  p->T = sh->n_tokens;
  p->D = D;
  p->Lg = sh->layers_per_group;
  p->S = p->Lg * p->H;
  p->G = p->nL / p->Lg;
  p->NU = 2 * p->G;
  p->M = p->S * D;
  p->dtype = sh->dtype;
  if ((long long)p->S * p->T * D >= (1LL << 40)) return fail(JOLT_ERR_UNSUPPORTED_SHAPE, "unit too large");
  if (op->method != JOLT_EXACT && op->method != JOLT_RANDOMIZED)
    return fail(JOLT_ERR_INVALID_ARG, "method %d", op->method);
  const int rcap = p->T < p->M ? p->T : p->M;
  JTRY(check_list(op->token_ranks, op->n_token_ranks, 1, rcap, "token_ranks"));
  JTRY(check_list(op->feature_ranks, op->n_feature_ranks, 1, D, "feature_ranks"));
  JTRY(check_list(op->bits, op->n_bits, 0, 8, "bits"));
  p->cd.nT = op->n_token_ranks;
  p->cd.nD = op->n_feature_ranks;
  p->cd.nB = op->n_bits;
  for (int i = 0; i < MAXC; ++i) {
    p->cd.rT[i] = i < op->n_token_ranks ? op->token_ranks[i] : 0;
    p->cd.rD[i] = i < op->n_feature_ranks ? op->feature_ranks[i] : 0;
    p->cd.bits[i] = i < op->n_bits ? op->bits[i] : 0;
  }
  p->nC = p->cd.nT * p->cd.nD * p->cd.nB;
  p->rTmax = max_in(op->token_ranks, op->n_token_ranks);
  p->rDmax = max_in(op->feature_ranks, op->n_feature_ranks);
  if (p->rTmax % 8 || p->rDmax % 8)
    return fail(JOLT_ERR_UNSUPPORTED_SHAPE, "largest token / feature rank must be a multiple of 8");
  p->ldU = p->rTmax;
  p->ldW = p->rDmax;
  p->ldC = p->rDmax;
  p->method = op->method;
  if (op->unit_offset < 0 || op->unit_offset > (1 << 24)) return fail(JOLT_ERR_INVALID_ARG, "unit_offset %d", op->unit_offset);
  p->u0 = op->unit_offset;
  p->q = op->power_iters;
  p->k = 0;
  p->kp = 0;
  if (op->method == JOLT_RANDOMIZED) {
    if (op->oversample < 0 || op->power_iters < 0 || op->power_iters > 16)
      return fail(JOLT_ERR_INVALID_ARG, "oversample / power_iters out of range");
    p->k = p->rTmax + op->oversample;
    if (p->k > rcap) return fail(JOLT_ERR_UNSUPPORTED_SHAPE, "sketch width %d exceeds min(T, M) = %d", p->k, rcap);
    p->kp = (int)round_up(p->k, 8);
  }
  p->m_side = p->T > p->M;
  p->tiles = (int)ceil_div(p->T, TROWS);

  // split-K of the Grams (fixed: results do not depend on the device)
  long long rows = (long long)p->S * p->T;
  p->gd_split = (int)ceil_div(rows, 1024);
  if (p->gd_split > 64) p->gd_split = 64;
  p->gt_split = p->m_side ? (int)ceil_div(p->T, 4096) : (p->S < 16 ? p->S : 16);
  if (p->gt_split > 64) p->gt_split = 64;

  const int NU = p->NU, T = p->T, S = p->S, M = p->M;
  // Cholesky-QR Grams: split-K partials in fp32, summed in fp64
  {
    long long mrows = op->method == JOLT_RANDOMIZED ? (M > T ? M : T) : (p->m_side ? T : 0);
    const int kq = op->method == JOLT_RANDOMIZED ? (int)round_up(p->rTmax + op->oversample, 8) : p->rTmax;
    if (kq >= QR_TC_MINK) {
      // tensor-core Grams: split-K chunks of QR_TC_CHUNK rows; the Rayleigh-Ritz Gram (M rows,
      // chunks of 256) shares the buffer
      long long need = ceil_div(mrows, QR_TC_CHUNK);
      if (op->method == JOLT_RANDOMIZED && ceil_div(M, 256) > need) need = ceil_div(M, 256);
      p->qr_split_max = mrows > 0 ? (int)need : 1;
    } else {
      p->qr_split_max = mrows > 0 ? (int)ceil_div(mrows, 256) : 1;
    }
  }
  // cuSOLVER device workspace: with a device present the batched eigen solver is asked for
  // its exact need; without one (size queries on a host) a bound is used.
  {
    long long ntok = op->method == JOLT_EXACT ? (p->m_side ? M : T) : p->k;
    p->solver_dev = 0;
    p->fsolver_dev = 0;
    p->solver_host = 0;
    int ndev = 0;
    bool queried = false;
    if (cudaGetDeviceCount(&ndev) == cudaSuccess && ndev > 0) {
      Solver* s = nullptr;
      if (solver_get(0, &s) == JOLT_OK) {
        queried = true;
        for (long long n : {(long long)D, ntok}) {
          size_t dv = 0, hv = 0;
          if (cusolverDnXsyevBatched_bufferSize(s->h, s->params, CUSOLVER_EIG_MODE_VECTOR, CUBLAS_FILL_MODE_LOWER, n,
                                                CUDA_R_64F, nullptr, n, CUDA_R_64F, nullptr, CUDA_R_64F, &dv, &hv,
                                                NU) != CUSOLVER_STATUS_SUCCESS) {
            queried = false;
            break;
          }
          if (n == D) p->fsolver_dev = dv;
          if (n == ntok) p->solver_dev = dv > p->solver_dev ? dv : p->solver_dev;
          p->solver_host = hv > p->solver_host ? hv : p->solver_host;
        }
      }
    }
    cudaGetLastError();
    if (!queried) {
      p->solver_dev = (size_t)NU * (size_t)(8 * (1 + 6 * ntok + 2 * ntok * ntok) * 8) + (16 << 20);
      p->fsolver_dev = (size_t)NU * (size_t)(8 * (1 + 6 * (long long)D + 2 * (long long)D * D) * 8) + (16 << 20);
    }
  }

  Bump b;
  p->o_status = b.take(256);
  p->o_signkey = b.take((size_t)NU * p->rTmax * 8);   // token-factor column signs: keys, signs
  p->o_sign = b.take((size_t)NU * p->rTmax * 4);
  p->o_gd_part = b.take((size_t)NU * p->gd_split * D * D * 4);
  p->o_gd = b.take((size_t)NU * D * D * 8);
  {
    long long ntok = op->method == JOLT_EXACT ? (p->m_side ? M : T) : p->kp;
    long long nev = (long long)NU * (D > ntok ? D : ntok);
    p->o_evals = b.take((size_t)nev * 8 + 256);
  }
  p->o_Wf = b.take((size_t)NU * D * p->ldW * 4);
  p->o_Ws = b.take((size_t)NU * D * p->ldW * 2);
  p->o_Uf = b.take((size_t)NU * T * p->ldU * 4);
  p->o_Us = b.take((size_t)NU * T * p->ldU * 2);
  p->o_core = b.take((size_t)NU * S * p->rTmax * p->ldC * 2);
  p->o_zc = b.take((size_t)NU * S * T * p->ldW * 2);
  p->o_ctmp = b.take((size_t)NU * S * p->rTmax * p->ldW * 2);   // the core before its permutation
  p->o_ptmp = b.take((size_t)NU * S * p->rTmax * D * 4);
  p->o_P = b.take((size_t)NU * p->cd.nD * S * p->rTmax * D * 2);
  p->o_partial = b.take((size_t)NU * S * p->tiles * p->nC * 8);
  p->o_table = b.take((size_t)NU * p->nC * 8);
  p->o_bytes = b.take((size_t)NU * p->nC * 8);
  p->o_choice = b.take((size_t)NU * 4);
  p->o_lambda = b.take(8);
  p->o_hdr = b.take(64);
  p->o_umap = b.take((size_t)NU * S * 4 + 64);
  p->o_info = b.take((size_t)NU * 4 + 64);
  p->o_solver = b.take(p->solver_dev + 256);
  p->o_fsolver = b.take(p->fsolver_dev + 256);
  p->o_finfo = b.take((size_t)NU * 4 + 64);
  p->o_fevals = b.take((size_t)NU * D * 8 + 256);
  // token factor scratch
  p->o_gt32 = p->o_gt = p->o_vsel = p->o_lam = p->o_omega = 0;
  p->o_Y = p->o_Zm = p->o_h = p->o_l = p->o_gpart = p->o_G = p->o_eigvec = p->o_eigscr = 0;
  p->o_h2 = p->o_l2 = p->o_mh = p->o_ml = 0;
  const int kq = op->method == JOLT_RANDOMIZED ? p->kp : p->ldU;   // width of the QR'ed blocks
  if (op->method == JOLT_EXACT) {
    long long n = p->m_side ? M : T;
    p->o_gt32 = b.take((size_t)NU * n * n * 4);
    p->o_gt = b.take((size_t)NU * n * n * 8);
    p->o_lam = b.take((size_t)NU * p->rTmax * 8 + 256);
    if (p->m_side) {
      // split copies of V (M rows) for the back-projection and of U (T rows) for its QR
      p->o_vsel = b.take((size_t)NU * M * p->ldU * 4);
      p->o_h = b.take((size_t)NU * (M > T ? M : T) * p->ldU * 2);
      p->o_l = b.take((size_t)NU * (M > T ? M : T) * p->ldU * 2);
    }
  } else {
    const int kp = p->kp;
    long long big = M > T ? M : T;
    const bool pairs = sh->dtype == JOLT_BF16 && D % 64 == 0 && T % 64 == 0 && kp >= QR_TC_MINK;
    p->o_omega = b.take((size_t)NU * M * kp * 2);
    if (!pairs) p->o_Y = b.take((size_t)NU * T * kp * 4);
    p->o_Zm = b.take((size_t)NU * M * kp * 4);
    p->o_h = b.take((size_t)NU * big * kp * 2);
    p->o_l = b.take((size_t)NU * big * kp * 2);
    if (pairs) {
      p->o_h2 = b.take((size_t)NU * T * kp * 2);
      p->o_l2 = b.take((size_t)NU * T * kp * 2);
      p->o_mh = b.take((size_t)NU * M * kp * 2);
      p->o_ml = b.take((size_t)NU * M * kp * 2);
    }
    p->o_vsel = b.take((size_t)NU * kp * p->ldU * 4);
  }
  // the own eigen solver (order <= 256): the feature factor (n = D, auxiliary stream) and the
  // token-side problem (Rayleigh-Ritz, n = k; exact route, n = T or M) have separate buffers
  p->o_feigvec = b.take((size_t)NU * D * D * 8);
  p->o_feigscr = b.take((size_t)NU * eigc::scratch_doubles(D) * 8);
  {
    // order <= 256: the cluster solver in shared memory; <= 1024: the global-memory solver
    const long long ntok = op->method == JOLT_EXACT ? (p->m_side ? M : T) : p->k;
    p->eig_n = (ntok >= 2 && ntok <= eigl::MAXN) ? (int)ntok : 0;
    if (p->eig_n) {
      const size_t scr = ntok <= eigc::MAXN ? eigc::scratch_doubles((int)ntok) : eigl::scratch_doubles((int)ntok);
      p->o_eigvec = b.take((size_t)NU * ntok * ntok * 8);
      p->o_eigscr = b.take((size_t)NU * scr * 8);
    }
  }
  p->o_Lr = p->o_wth = p->o_wtl = p->o_winv = p->o_vh = p->o_vl = 0;
  if (op->method == JOLT_RANDOMIZED || p->m_side) {
    p->o_gpart = b.take((size_t)NU * p->qr_split_max * kq * kq * 4);
    p->o_G = b.take((size_t)NU * kq * kq * 8);
    // L as fp32 row-major, or (k <= 256) the transposed inverse of L at the padded width
    p->o_Lr = b.take((size_t)NU * round_up(kq, 32) * round_up(kq, 32) * 4);
    if (kq >= QR_TC_MINK) {
      const size_t kq32 = round_up(kq, 32);
      p->o_wth = b.take((size_t)NU * kq32 * kq32 * 2);
      p->o_wtl = b.take((size_t)NU * kq32 * kq32 * 2);
      p->o_winv = b.take((size_t)NU * kq32 * kq32 * 8);
      if (op->method == JOLT_RANDOMIZED) {
        p->o_vh = b.take((size_t)NU * kq * p->ldU * 2);
        p->o_vl = b.take((size_t)NU * kq * p->ldU * 2);
      }
    }
  }
  p->ws_total = b.off;

  // largest possible blob
  unsigned long long mx = 0;
  for (int i = 0; i < p->cd.nT; ++i)
    for (int j = 0; j < p->cd.nD; ++j)
      for (int l = 0; l < p->cd.nB; ++l) {
        unsigned long long v = unit_payload_bytes(T, D, S, p->cd.rT[i], p->cd.rD[j], p->cd.bits[l]);
        mx = v > mx ? v : mx;
      }
  p->blob_max = 64 + 64 * (size_t)NU + (size_t)NU * mx;

  Bump d;
  d.take(256);
  p->d_U = d.take((size_t)NU * T * p->ldU * 2);
  p->d_W = d.take((size_t)NU * D * p->ldW * 2);
  p->d_C = d.take((size_t)NU * S * p->rTmax * p->ldC * 2);
  p->d_ptmp = d.take((size_t)NU * S * p->rTmax * D * 4);
  p->d_P = d.take((size_t)NU * S * p->rTmax * D * 2);
  p->d_umap = d.take((size_t)NU * S * 4 + 64);
  p->dws_total = d.off;
  return JOLT_OK;
}

// ------------------------------------------------------------------------------------------
// GEMM dispatch on operand element types (0 bf16, 1 fp32, 2 fp64)
// ------------------------------------------------------------------------------------------
jolt_status gemm(const GemmParams& p, int ta, int tb, cudaStream_t st) {
  cudaError_t e;
  const bool dacc = p.c_type == 2;
  if (p.sym && !(ta == 1 && tb == 1 && !dacc)) return fail(JOLT_ERR_INVALID_ARG, "symmetric GEMM needs fp32 operands");
  if (ta == 0 && tb == 0) e = launch_gemm_bf16(p, st);
  else if (ta == 1 && tb == 1 && p.c_type != 2) e = launch_sgemm(p, st);
#define GEMM_CASE(A, B, TA, TB)                                                              \
  else if (ta == A && tb == B) e = dacc ? launch_gemm_simt<TA, TB, double>(p, st)           \
                                        : launch_gemm_simt<TA, TB, float>(p, st);
  GEMM_CASE(1, 1, float, float)
  GEMM_CASE(1, 0, float, bf16)
  GEMM_CASE(0, 1, bf16, float)
  GEMM_CASE(1, 2, float, double)
  GEMM_CASE(2, 1, double, float)
  GEMM_CASE(2, 2, double, double)
#undef GEMM_CASE
  else return fail(JOLT_ERR_INVALID_ARG, "gemm type combination %d/%d", ta, tb);
  if (e != cudaSuccess) return fail(JOLT_ERR_CUDA, "gemm launch: %s", cudaGetErrorString(e));
  return JOLT_OK;
}

int ilog2(int v) {
  int s = 0;
  while ((1 << s) < v) ++s;
  return s;
}

unsigned grid1d(long long n, int threads = 256) {
  long long g = ceil_div(n, threads);
  if (g > 148 * 32) g = 148 * 32;
  if (g < 1) g = 1;
  return (unsigned)g;
}

struct Ctx {
  const Plan& p;
  unsigned char* ws;
  cudaStream_t st;
  const void* k;
  const void* v;
  uint64_t seed;
  int side = 0;   // 1: the feature factor on the auxiliary stream (own eigen-solver workspace)
  template <typename T>
  T* at(size_t off) const { return reinterpret_cast<T*>(ws + off); }
  uint32_t* status() const { return at<uint32_t>(p.o_status); }
  // the tile counter of the tensor-core GEMMs launched on this context's stream (bytes 64.. of
  // the 256-byte status block; one per stream, since the two streams' GEMMs may overlap)
  int* sched() const { return at<int>(p.o_status) + 16 + 8 * side; }
  CacheView view() const {
    CacheView c;
    c.k = k;
    c.v = v;
    c.dtype = p.dtype;
    c.n_layers = p.nL;
    c.H = p.H;
    c.T = p.T;
    c.D = p.D;
    c.Lg = p.Lg;
    c.S = p.S;
    c.u0 = p.u0;
    c.unit_elems = (long long)p.S * p.T * p.D;
    return c;
  }
};

// X_(T) as operand: (row t, col (s,d))  -> offset s*T*D + t*D + d
GemmOperand xt_rowmajor(const Ctx& c, const void* x) {
  GemmOperand o;
  o.ptr = x;
  o.kmajor = true;       // as A (T x M): contiguous along the M index inside a slice
  o.ld = c.p.D;
  o.kshift = ilog2(c.p.D);
  o.skblk = (long long)c.p.T * c.p.D;
  return o;
}

// ------------------------------------------------------------------------------------------
// symmetric eigen solve (cuSOLVER, fp64), one matrix at a time
// ------------------------------------------------------------------------------------------
// the solver's device workspace must fit the plan's bound; host workspace grows on demand
jolt_status solver_ws(const Ctx& c, Solver* s, size_t dv, size_t hv, void** host) {
  const size_t cap = c.side ? c.p.fsolver_dev : c.p.solver_dev;
  if (dv > cap) return fail(JOLT_ERR_WORKSPACE_TOO_SMALL, "cuSOLVER needs %zu device bytes, plan holds %zu", dv, cap);
  if (s->host_ws.size() < hv) s->host_ws.resize(hv);
  *host = hv ? s->host_ws.data() : nullptr;
  return JOLT_OK;
}

// batched: nbatch matrices of n x n stored back to back (lda = n), eigenvalues n per matrix
jolt_status sym_eig_batched(const Ctx& c, double* A, int64_t n, double* w, int64_t nbatch) {
  ProfScope ps("sym_eig", c.st, nbatch);
  Solver* s = nullptr;
  JTRY(solver_get(c.st, &s, c.side));
  void* dws = c.at<void>(c.side ? c.p.o_fsolver : c.p.o_solver);
  int* info = c.at<int>(c.side ? c.p.o_finfo : c.p.o_info);
  size_t dv = 0, hv = 0;
  SOLVER_TRY(cusolverDnXsyevBatched_bufferSize(s->h, s->params, CUSOLVER_EIG_MODE_VECTOR, CUBLAS_FILL_MODE_LOWER, n,
                                               CUDA_R_64F, A, n, CUDA_R_64F, w, CUDA_R_64F, &dv, &hv, nbatch));
  void* host = nullptr;
  JTRY(solver_ws(c, s, dv, hv, &host));
  count_launch(), sanitize_sym_batched_kernel<<<(unsigned)nbatch, 1024, 0, c.st>>>(A, (int)n, n, n * n, c.status());
  CUDA_TRY(cudaGetLastError());
  SOLVER_TRY(cusolverDnXsyevBatched(s->h, s->params, CUSOLVER_EIG_MODE_VECTOR, CUBLAS_FILL_MODE_LOWER, n, CUDA_R_64F,
                                    A, n, CUDA_R_64F, w, CUDA_R_64F, dws, dv, host, hv, info, nbatch));
  count_launch(), info_check_kernel<<<(unsigned)ceil_div(nbatch, 32), 32, 0, c.st>>>(info, (int)nbatch, c.status(),
                                                                                   DEV_ERR_FACTOR);
  CUDA_TRY(cudaGetLastError());
  return JOLT_OK;
}

// Leading r eigenvectors (descending, sign-fixed) of nbatch symmetric n x n matrices S (fp64,
// lda = n, stride n*n; overwritten by the solver), through cuSOLVER's batched eigen solver.
jolt_status sym_eig_top(const Ctx& c, double* S, int n, int nbatch, int r, float* out_f32, bf16* out_bf16,
                        long long ldo, long long sout, double* out_vals) {
  double* w = c.at<double>(c.side ? c.p.o_fevals : c.p.o_evals);
  const bool own = c.side ? (n == c.p.D && n >= 2 && n <= eigc::MAXN) : (c.p.eig_n != 0 && n == c.p.eig_n);
  if (own && n > eigc::MAXN) {
    // the global-memory solver (csrc/eig_large.cuh)
    ProfScope ps("sym_eig", c.st, nbatch);
    double* V = c.at<double>(c.p.o_eigvec);
    double* scr = c.at<double>(c.p.o_eigscr);
    count_launch(), sanitize_sym_batched_kernel<<<(unsigned)nbatch, 1024, 0, c.st>>>(S, n, n, (long long)n * n,
                                                                                      c.status());
    count_launch(), symmetrize_lower_kernel<<<dim3(64, (unsigned)nbatch), 256, 0, c.st>>>(S, n, (long long)n * n);
    CUDA_TRY(cudaGetLastError());
    CUDA_TRY(cudaFuncSetAttribute(tridiag_gm_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)eigl::TRI_SMEM));
    {
      ProfScope ps1("eig_tridiag", c.st, nbatch);
      count_launch(), tridiag_gm_kernel<<<(unsigned)(nbatch * eigl::CL), eigl::TRI_THREADS, eigl::TRI_SMEM, c.st>>>(
          S, n, (long long)n * n, scr);
      CUDA_TRY(cudaGetLastError());
    }
    {
      ProfScope ps2("eig_tridiag_solve", c.st, nbatch);
      count_launch(), tri_eig_kernel<<<dim3((unsigned)ceil_div(n, eigl::EV_PER_CTA), (unsigned)nbatch),
                                       eigl::THREADS, 0, c.st>>>(n, w, n, V, scr);
      CUDA_TRY(cudaGetLastError());
      count_launch(), tight_mgs_kernel<<<(unsigned)nbatch, 32, 0, c.st>>>(n, w, n, V);
      CUDA_TRY(cudaGetLastError());
    }
    const size_t wsm = wy_apply_smem(n);
    CUDA_TRY(cudaFuncSetAttribute(wy_apply_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)wsm));
    {
      ProfScope ps3("eig_backtransform", c.st, nbatch);
      count_launch(), wy_tfactor_kernel<<<dim3((unsigned)wy_blocks(n), (unsigned)nbatch), eigl::WY_THREADS, 0,
                                          c.st>>>(n, scr);
      CUDA_TRY(cudaGetLastError());
      count_launch(), wy_apply_kernel<<<dim3((unsigned)ceil_div(n, eigl::WY_COLS), (unsigned)nbatch),
                                        eigl::WY_THREADS, wsm, c.st>>>(n, V, scr);
      CUDA_TRY(cudaGetLastError());
    }
    count_launch(), eig_select_kernel<<<dim3(r, nbatch), 256, 0, c.st>>>(w, V, n, 1, n, n, (long long)n * n, r,
                                                                         out_f32, out_bf16, ldo, sout, out_vals);
    CUDA_TRY(cudaGetLastError());
    return JOLT_OK;
  }
  if (own) {
    // one 8-CTA cluster per matrix (csrc/eig_cluster.cuh)
    ProfScope ps(c.side ? "feature_eig" : "sym_eig", c.st, nbatch);
    double* V = c.at<double>(c.side ? c.p.o_feigvec : c.p.o_eigvec);
    double* scr = c.at<double>(c.side ? c.p.o_feigscr : c.p.o_eigscr);
    // a non-finite matrix becomes the identity (and raises the status), as before cuSOLVER
    count_launch(), sanitize_sym_batched_kernel<<<(unsigned)nbatch, 1024, 0, c.st>>>(S, n, n, (long long)n * n,
                                                                                      c.status());
    CUDA_TRY(cudaGetLastError());
    const size_t sm = eigc::smem_bytes();
    CUDA_TRY(cudaFuncSetAttribute(sym_eig_cluster_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sm));
    count_launch(), sym_eig_cluster_kernel<<<(unsigned)(nbatch * eigc::CL), eigc::THREADS, sm, c.st>>>(
        S, n, (long long)n * n, w, n, V, scr, c.status());
    CUDA_TRY(cudaGetLastError());
    count_launch(), eig_select_kernel<<<dim3(r, nbatch), 256, 0, c.st>>>(w, V, n, 1, n, n, (long long)n * n, r,
                                                                         out_f32, out_bf16, ldo, sout, out_vals);
    CUDA_TRY(cudaGetLastError());
    return JOLT_OK;
  }
  JTRY(sym_eig_batched(c, S, n, w, nbatch));
  count_launch(), eig_select_kernel<<<dim3(r, nbatch), 256, 0, c.st>>>(w, S, n, n, 1, n, (long long)n * n, r, out_f32,
                                                                       out_bf16, ldo, sout, out_vals);
  CUDA_TRY(cudaGetLastError());
  return JOLT_OK;
}

// Cholesky QR of every unit's m x k block Y (fp32, row pitch ld, unit stride m*ld), in
// place: G = Y^T Y (fp32 partial sums of <= 256 terms, added in fp64), G = L L^T (cuSOLVER's
// batched Cholesky, fp64), Q = Y L^{-T} (blocked row-panel solve).  `passes` = 2 gives
// CholeskyQR2.

jolt_status cholqr_tc(const Ctx& c, float* Y, long long m, int k, int ld, int passes);

jolt_status cholqr_batched(const Ctx& c, float* Y, long long m, int k, int ld, int passes) {
  const Plan& p = c.p;
  if (p.o_wth) {
    if (ld % 8) return fail(JOLT_ERR_INVALID_ARG, "token factor pitch %d not a multiple of 8", ld);
    return cholqr_tc(c, Y, m, k, ld, passes);
  }
  // block widths below the tensor-core width (k < 64): fp32 Gram, own factor and inverse product
  ProfScope ps("cholesky_qr", c.st, p.NU);
  float* gpart = c.at<float>(p.o_gpart);
  double* G = c.at<double>(p.o_G);
  // split-K chunk: 256 rows, halved (down to 64) while fewer than two CTAs per SM would run
  // and the partial buffer (qr_split_max splits) still holds the splits
  int kchunk = 256;
  {
    const long long nt = ceil_div(k, sgemm_detail::BM), tiles = nt * (nt + 1) / 2;
    while (kchunk > 64 && (long long)p.NU * tiles * ceil_div(m, kchunk) < 2 * 148 &&
           ceil_div(m, kchunk / 2) <= p.qr_split_max)
      kchunk /= 2;
  }
  const int ns = (int)ceil_div(m, kchunk);
  const int gld = ld;
  if (k > 1024) return fail(JOLT_ERR_UNSUPPORTED_SHAPE, "Cholesky QR of more than 1024 columns");
  for (int pass = 0; pass < passes; ++pass) {
    const long long n = (long long)k * gld;
    {
    ProfScope ps1("qr_gram", c.st, p.NU);
    GemmParams g;
    g.M = k;
    g.N = k;
    g.K = (int)m;
    g.batch = p.NU;
    g.A.ptr = Y;
    g.A.kmajor = false;
    g.A.ld = ld;
    g.A.sbatch = m * ld;
    g.B = g.A;
    g.C = gpart;
    g.ldc = gld;
    g.sbatchC = (long long)ns * k * gld;
    g.ssplitC = (long long)k * gld;
    g.splits = ns;
    g.kchunk = kchunk;
    g.c_type = 0;
    g.sym = true;
    JTRY(gemm(g, 1, 1, c.st));
    count_launch(), reduce_splits_sym_kernel<float><<<grid1d((long long)p.NU * k * k), 256, 0, c.st>>>(
        gpart, G, p.NU, ns, k, gld, sgemm_detail::BM);
    }
    float* Lr = c.at<float>(p.o_Lr);
    const int nbk = (int)ceil_div(k, CF_NB);
    if (k <= CF_MAXK && ld % 4 == 0) {
      // own factor, block-column inverse and inverse product (chol.cuh; 16-byte row loads)
      const int kq32 = (int)round_up(k, 32);
      float* WT = Lr;
      const long long sW = (long long)kq32 * kq32;
      {
        ProfScope ps2("qr_factor", c.st, p.NU);
        CUDA_TRY(cudaFuncSetAttribute(chol_factor_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      (int)chol_factor_smem()));
        count_launch(), chol_factor_kernel<<<p.NU, CF_FT, chol_factor_smem(), c.st>>>(G, k, gld, n, c.status());
        CUDA_TRY(cudaGetLastError());
        CUDA_TRY(cudaFuncSetAttribute(tri_inv_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      (int)tri_inv_smem()));
        count_launch(), tri_inv_kernel<<<dim3(nbk, p.NU), CF_THREADS, tri_inv_smem(), c.st>>>(G, k, gld, n, WT, kq32,
                                                                                               sW);
        CUDA_TRY(cudaGetLastError());
      }
      ProfScope ps3("qr_trsm", c.st, p.NU);
      const size_t sm = trsm_inv_smem(kq32);
      CUDA_TRY(cudaFuncSetAttribute(trsm_inv_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sm));
      count_launch(), trsm_inv_kernel<<<dim3((unsigned)ceil_div(m, TI_RB), p.NU), CF_THREADS, sm, c.st>>>(
          Y, m, k, ld, m * ld, WT, kq32, sW);
      CUDA_TRY(cudaGetLastError());
      continue;
    }
    return fail(JOLT_ERR_UNSUPPORTED_SHAPE, "Cholesky QR of %d columns below the tensor-core width", k);
  }
  return JOLT_OK;
}

// C = (X-product with an fp32 operand F).  For a bf16 cache F is split as hi + lo bf16
// (hi + lo = F to 2^-17) and the two tensor-core products are summed; for an fp32 cache
// the product runs in fp32 directly.
jolt_status gemm_xf(const Ctx& c, GemmParams g, bool f_is_A, const float* F, long long nF) {
  ProfScope ps("sketch_product", c.st, c.p.NU);
  const bool xbf = c.p.dtype == JOLT_BF16;
  if (!xbf) {
    if (f_is_A) g.A.ptr = F;
    else g.B.ptr = F;
    return gemm(g, 1, 1, c.st);
  }
  bf16* hi = c.at<bf16>(c.p.o_h);
  bf16* lo = c.at<bf16>(c.p.o_l);
  count_launch(), split_bf16_kernel<<<grid1d(nF), 256, 0, c.st>>>(F, hi, lo, nF);
  CUDA_TRY(cudaGetLastError());
  GemmParams g1 = g, g2 = g;
  if (f_is_A) {
    g1.A.ptr = hi;
    g2.A.ptr = lo;
  } else {
    g1.B.ptr = hi;
    g2.B.ptr = lo;
  }
  g1.beta = 0.f;
  g2.beta = 1.f;
  JTRY(gemm(g1, 0, 0, c.st));
  JTRY(gemm(g2, 0, 0, c.st));
  return JOLT_OK;
}

int xtype(const Ctx& c) { return c.p.dtype == JOLT_BF16 ? 0 : 1; }

// the X-products of the sketch run on the tcgen05 kernel when the cache is bf16 and a
// 64-wide feature box stays inside one slice
bool umma_ok(const Plan& p) { return p.dtype == JOLT_BF16 && p.D % 64 == 0 && p.T % 64 == 0; }

// tensor maps of the K and V caches as slices (X_(T) modes) or as rows (X_(D) modes)
jolt_status cache_maps(const Ctx& c, bool rows, CUtensorMap* mk, CUtensorMap* mv) {
  const Plan& p = c.p;
  const bool ok = rows ? (map_cache_rows(mk, c.k, p.nL, p.H, p.T, p.D) && map_cache_rows(mv, c.v, p.nL, p.H, p.T, p.D))
                       : (map_cache_xt(mk, c.k, p.nL, p.H, p.T, p.D) && map_cache_xt(mv, c.v, p.nL, p.H, p.T, p.D));
  if (!ok) return fail(JOLT_ERR_CUDA, "tensor map of the cache refused");
  return JOLT_OK;
}

jolt_status umma_run(const Ctx& c, const UmmaMaps& m, UmmaArgs a, int nb) {
  a.sched = c.sched();
  cudaError_t e = launch_umma(m, a, nb, c.st);
  if (e != cudaSuccess) return fail(JOLT_ERR_CUDA, "tensor-core GEMM: %s", cudaGetErrorString(e));
  return JOLT_OK;
}

// Cholesky QR on the tensor cores (block widths >= QR_TC_MINK), in place on every unit's
// m x k block Y (fp32, pitch ld, unit stride m * ld; columns k..ld zero):
//   Y = Yh + Yl (bf16 hi + lo, Y - Yh - Yl = O(2^-17 |Y|));
//   G = Yh^T Yh + Yh^T Yl + Yl^T Yh on tcgen05 (upper tiles only, split-K partials of
//       QR_TC_CHUNK rows in fp32, summed in fp64) -- the dropped Yl^T Yl is O(2^-18 |Y|^2);
//   G = L L^T in fp64 (own kernel for k <= 256, else the batched LAPACK-style Cholesky) and
//   W = L^{-1} block column by block column in fp64 (tri_inv_kernel / tri_inv_large_kernel);
//   Q = Y W^T = Yh (Wh + Wl)^T + Yl Wh^T on tcgen05, the K range of each output tile cut at
//       the diagonal (W^T is upper triangular).
// `passes` = 2 gives CholeskyQR2.
// One pass on a block given as its bf16 hi + lo split (yh, yl; columns k..ld zero): the Gram,
// the factor and its inverse, and Q, written either as fp32 (outY) or as a bf16 pair (oh, ol,
// all ld columns; the columns k..ld come out zero).
jolt_status qr_pass_tc(const Ctx& c, const bf16* yh, const bf16* yl, long long m, int k, int ld, float* outY,
                       bf16* oh, bf16* ol) {
  const Plan& p = c.p;
  float* gpart = c.at<float>(p.o_gpart);
  double* G = c.at<double>(p.o_G);
  float* WT = c.at<float>(p.o_Lr);
  bf16* wth = c.at<bf16>(p.o_wth);
  bf16* wtl = c.at<bf16>(p.o_wtl);
  const int gld = ld, kq32 = (int)round_up(k, 32), nbk = (int)ceil_div(k, 32);
  const long long sG = (long long)k * gld, sW = (long long)kq32 * kq32;
  const int ns = (int)ceil_div(m, QR_TC_CHUNK);
  if (ns > p.qr_split_max) return fail(JOLT_ERR_WORKSPACE_TOO_SMALL, "Gram partial slots");
  UmmaMaps my, mw;
  if (!map_dense(&my.a0, yh, ld, m, p.NU) || !map_dense(&my.a1, yl, ld, m, p.NU) ||
      !map_dense(&mw.b0, wth, kq32, kq32, p.NU) || !map_dense(&mw.b1, wtl, kq32, kq32, p.NU))
    return fail(JOLT_ERR_CUDA, "tensor map of the Cholesky QR operands refused");
  // rows k..kq32 of W^T are never written: zeroed (they meet zero columns of Y)
  CUDA_TRY(cudaMemsetAsync(WT, 0, (size_t)p.NU * sW * 4, c.st));
  {
    ProfScope ps1("qr_gram", c.st, p.NU);
    UmmaArgs g;
    g.M = g.N = k;
    g.K = (int)m;
    g.batch = p.NU;
    g.splits = ns;
    g.kchunk = QR_TC_CHUNK;
    g.A.mode = UM_DENSE_MN;
    g.B.mode = UM_DENSE_MN;
    g.tri = 1;
    g.bn = 128;
    g.C = gpart;
    g.ldc = gld;
    g.sC = (long long)ns * k * gld;
    g.ssplit = (long long)k * gld;
    g.status = c.status();
    UmmaMaps m3;   // Yh^T Yh + Yh^T Yl + Yl^T Yh in one pass
    m3.a0 = my.a0;
    m3.a1 = my.a1;
    m3.b0 = my.a0;
    m3.b1 = my.a1;
    JTRY(umma_run(c, m3, g, 3));
    count_launch(), reduce_upper_sym_kernel<<<grid1d((long long)p.NU * k * k), 256, 0, c.st>>>(gpart, G, p.NU,
                                                                                                ns, k, gld);
    CUDA_TRY(cudaGetLastError());
  }
  {
    ProfScope ps2("qr_factor", c.st, p.NU);
    if (k <= CF_MAXK && gld % 4 == 0) {
      CUDA_TRY(cudaFuncSetAttribute(chol_factor_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    (int)chol_factor_smem()));
      count_launch(), chol_factor_kernel<<<p.NU, CF_FT, chol_factor_smem(), c.st>>>(G, k, gld, sG, c.status());
      CUDA_TRY(cudaGetLastError());
      CUDA_TRY(cudaFuncSetAttribute(tri_inv_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    (int)tri_inv_smem()));
      count_launch(), tri_inv_kernel<<<dim3(nbk, p.NU), CF_THREADS, tri_inv_smem(), c.st>>>(G, k, gld, sG, WT, kq32,
                                                                                             sW);
      CUDA_TRY(cudaGetLastError());
    } else {
      // 256 < k <= 1024: the cluster Cholesky (chol.cuh), then the block-column inverse
      count_launch(), sanitize_sym_batched_kernel<<<p.NU, 1024, 0, c.st>>>(G, k, gld, sG, c.status());
      {
        ProfScope ps4("chol_steps", c.st, p.NU);
        for (int J = 0; J < nbk; ++J) {
          count_launch(), chol_step_diag_kernel<<<p.NU, 32, 0, c.st>>>(G, k, gld, sG, J, c.status());
          const int below = nbk - J - 1;
          if (below > 0) {
            count_launch(), chol_step_panel_kernel<<<dim3(below, p.NU), CF_THREADS, 0, c.st>>>(G, k, gld, sG, J);
            count_launch(), chol_step_update_kernel<<<dim3(below * (below + 1) / 2, p.NU), CF_THREADS, 0, c.st>>>(
                G, k, gld, sG, J);
          }
        }
        CUDA_TRY(cudaGetLastError());
      }
      ProfScope ps5("tri_inv_large", c.st, p.NU);
      CUDA_TRY(cudaFuncSetAttribute(tri_inv_large_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    (int)tri_inv_large_smem()));
      count_launch(), tri_inv_large_kernel<<<dim3(nbk, p.NU), CF_THREADS * TI_G, tri_inv_large_smem(), c.st>>>(
          G, k, gld, sG, c.at<double>(p.o_winv), kq32, WT, kq32, sW);
      CUDA_TRY(cudaGetLastError());
    }
  }
  {
    ProfScope ps3("qr_trsm", c.st, p.NU);
    const long long nW = (long long)p.NU * sW;
    count_launch(), split_bf16_kernel<<<grid1d(nW), 256, 0, c.st>>>(WT, wth, wtl, nW);
    CUDA_TRY(cudaGetLastError());
    UmmaArgs q;
    q.M = (int)m;
    q.N = k;
    q.K = k;
    q.batch = p.NU;
    q.A.mode = UM_DENSE_K;
    q.B.mode = UM_DENSE_MN;
    q.tri = 2;
    q.bn = 128;
    if (outY) {
      q.C = outY;
    } else {
      q.N = ld;   // the pair gets every column (k..ld from zero rows of W^T)
      q.C = oh;
      q.C2 = ol;
      q.c_split = 1;
    }
    q.ldc = ld;
    q.sC = m * ld;
    q.status = c.status();
    UmmaMaps m3;   // Yh Wh^T + Yh Wl^T + Yl Wh^T in one pass
    m3.a0 = my.a0;
    m3.a1 = my.a1;
    m3.b0 = mw.b0;
    m3.b1 = mw.b1;
    JTRY(umma_run(c, m3, q, 3));
  }
  return JOLT_OK;
}

jolt_status cholqr_tc(const Ctx& c, float* Y, long long m, int k, int ld, int passes) {
  const Plan& p = c.p;
  ProfScope ps("cholesky_qr", c.st, p.NU);
  if (k > 1024) return fail(JOLT_ERR_UNSUPPORTED_SHAPE, "Cholesky QR of more than 1024 columns");
  if (ld % 8) return fail(JOLT_ERR_UNSUPPORTED_SHAPE, "Cholesky QR pitch %d not a multiple of 8", ld);
  bf16* yh = c.at<bf16>(p.o_h);
  bf16* yl = c.at<bf16>(p.o_l);
  const long long nY = (long long)p.NU * m * ld;
  for (int pass = 0; pass < passes; ++pass) {
    count_launch(), split_bf16_cols_kernel<<<grid1d(nY), 256, 0, c.st>>>(Y, yh, yl, nY, ld, k);
    CUDA_TRY(cudaGetLastError());
    JTRY(qr_pass_tc(c, yh, yl, m, k, ld, Y, nullptr, nullptr));
  }
  return JOLT_OK;
}

// Cholesky QR of a block held as bf16 pairs: pass i reads pair *cur and writes the other pair,
// so *cur names the pair holding Q afterwards.
jolt_status cholqr_tc_pairs(const Ctx& c, bf16* const* ph, bf16* const* pl, int* cur, long long m, int k, int ld,
                            int passes) {
  const Plan& p = c.p;
  ProfScope ps("cholesky_qr", c.st, p.NU);
  if (k > 1024) return fail(JOLT_ERR_UNSUPPORTED_SHAPE, "Cholesky QR of more than 1024 columns");
  if (ld % 8) return fail(JOLT_ERR_UNSUPPORTED_SHAPE, "Cholesky QR pitch %d not a multiple of 8", ld);
  for (int pass = 0; pass < passes; ++pass) {
    const int i = *cur, o = i ^ 1;
    JTRY(qr_pass_tc(c, ph[i], pl[i], m, k, ld, nullptr, ph[o], pl[o]));
    *cur = o;
  }
  return JOLT_OK;
}

// z_side = false: out (T x N per unit) = X_(T) F, F = M x kp ; z_side = true: out (M x N) =
// X_(T)^T F, F = T x kp, with F = f0 (+ f1, bf16 operands).  out is fp32, or with out2 the
// result as a bf16 hi (out) + lo (out2) pair; pitch kp.
jolt_status umma_x(const Ctx& c, bool z_side, const bf16* f0, const bf16* f1, int N, void* out, void* out2) {
  const Plan& p = c.p;
  ProfScope ps("sketch_product", c.st, p.NU);
  cudaError_t e = umma_x_product(c.k, c.v, p.nL, p.H, p.T, p.D, p.S, p.NU, z_side, f0, f1, p.kp, N, out, p.kp,
                                 c.status(), c.sched(), c.st, out2);
  if (e != cudaSuccess) return fail(JOLT_ERR_CUDA, "tensor-core X-product: %s", cudaGetErrorString(e));
  return JOLT_OK;
}

// the same with F given as bf16 (F16, one operand) or fp32 (F32, split into hi + lo into
// (hi, lo), which must hold NU x rows(F) x kp); fp32 output with N = k
jolt_status umma_product(const Ctx& c, bool z_side, const bf16* F16, const float* F32, float* out, bf16* hi = nullptr,
                         bf16* lo = nullptr) {
  const Plan& p = c.p;
  const bf16* f0 = F16;
  const bf16* f1 = nullptr;
  if (F32) {
    if (!hi) {
      hi = c.at<bf16>(p.o_h);
      lo = c.at<bf16>(p.o_l);
    }
    const long long nF = (long long)p.NU * (z_side ? p.T : p.M) * p.kp;
    count_launch(), split_bf16_kernel<<<grid1d(nF), 256, 0, c.st>>>(F32, hi, lo, nF);
    CUDA_TRY(cudaGetLastError());
    f0 = hi;
    f1 = lo;
  }
  return umma_x(c, z_side, f0, f1, p.k, out, nullptr);
}

// the cache of every unit as a batched operand: X_(T) (T x M, rows t, columns (l,h,d))
GemmOperand xt_units(const Ctx& c) {
  GemmOperand o = xt_rowmajor(c, c.k);
  o.ptr_odd = c.v;
  o.sbatch = (long long)c.p.S * c.p.T * c.p.D;
  return o;
}
// X_(T)^T (M x T): contiguous along (l,h,d) inside a slice, t stride D
GemmOperand xtT_units(const Ctx& c) {
  GemmOperand o;
  o.ptr = c.k;
  o.ptr_odd = c.v;
  o.sbatch = (long long)c.p.S * c.p.T * c.p.D;
  o.kmajor = false;
  o.ld = c.p.D;
  o.xshift = ilog2(c.p.D);
  o.sxblk = (long long)c.p.T * c.p.D;
  return o;
}

// ------------------------------------------------------------------------------------------
// stage 1a: feature factor W of every unit
// ------------------------------------------------------------------------------------------
jolt_status run_feature_factor(const Ctx& c, float* Wf, long long ldWf, bf16* Ws) {
  const Plan& p = c.p;
  ProfScope ps("feature_factor", c.st, p.NU);
  const int D = p.D;
  float* part = c.at<float>(p.o_gd_part);
  const long long rows = (long long)p.S * p.T;
  if (umma_ok(p)) {
    // G_D partial sums on the tensor cores: A = B = X_(D) (one shared tile per K block)
    UmmaMaps m;
    JTRY(cache_maps(c, true, &m.a0, &m.a1));
    m.b0 = m.a0;
    m.b1 = m.a1;
    UmmaArgs a;
    a.M = a.N = D;
    a.K = (int)rows;
    a.batch = p.NU;
    a.splits = p.gd_split;
    a.kchunk = (int)round_up(ceil_div(rows, p.gd_split), 64);
    a.A.mode = UM_ROW_MN;
    a.A.rows = rows;
    a.B = a.A;
    a.b_is_a = true;
    a.C = part;
    a.ldc = D;
    a.sC = (long long)p.gd_split * D * D;
    a.ssplit = (long long)D * D;
    a.status = c.status();
    JTRY(umma_run(c, m, a, 1));
  } else {
    const int kchunk = (int)round_up(ceil_div(rows, p.gd_split), 32);
    GemmParams g;
    g.M = D;
    g.N = D;
    g.K = (int)rows;
    g.batch = p.NU;
    g.A.ptr = c.k;
    g.A.ptr_odd = c.v;
    g.A.kmajor = false;
    g.A.ld = D;
    g.A.sbatch = rows * D;
    g.B = g.A;
    g.C = part;
    g.ldc = D;
    g.sbatchC = (long long)p.gd_split * D * D;
    g.ssplitC = (long long)D * D;
    g.splits = p.gd_split;
    g.kchunk = kchunk;
    g.c_type = 0;
    JTRY(gemm(g, xtype(c), xtype(c), c.st));
  }
  double* G = c.at<double>(p.o_gd);
  count_launch(), reduce_splits_kernel<float><<<grid1d((long long)p.NU * D * D), 256, 0, c.st>>>(
      part, G, p.NU, p.gd_split, (long long)D * D);
  count_launch(), gram_diag_check_kernel<<<p.NU, 128, 0, c.st>>>(G, D, p.NU, c.status());
  CUDA_TRY(cudaGetLastError());
  return sym_eig_top(c, G, D, p.NU, p.rDmax, Wf, Ws, ldWf, (long long)D * ldWf, nullptr);
}

// ------------------------------------------------------------------------------------------
// stage 1b: token factor U of every unit
// ------------------------------------------------------------------------------------------
jolt_status run_token_exact(const Ctx& c, float* Uf, long long ldUf) {
  const Plan& p = c.p;
  ProfScope ps("token_factor_exact", c.st, p.NU);
  const int T = p.T, M = p.M;
  const long long n = p.m_side ? M : T;
  float* G32 = c.at<float>(p.o_gt32);
  double* G = c.at<double>(p.o_gt);
  {
    GemmParams g;
    g.batch = p.NU;
    g.C = G32;
    g.ldc = n;
    g.sbatchC = n * n;
    g.c_type = 0;
    if (!p.m_side) {
      g.M = T;   // G_T = X_(T) X_(T)^T
      g.N = T;
      g.K = M;
      g.A = xt_units(c);
      g.B = g.A;
    } else {
      g.M = M;   // G_M = X_(T)^T X_(T)
      g.N = M;
      g.K = T;
      g.A = xtT_units(c);
      g.B = g.A;
    }
    if (umma_ok(p)) {
      UmmaMaps m;
      JTRY(cache_maps(c, false, &m.a0, &m.a1));
      m.b0 = m.a0;
      m.b1 = m.a1;
      UmmaArgs a;
      a.M = a.N = (int)n;
      a.K = p.m_side ? T : M;
      a.batch = p.NU;
      a.A.mode = p.m_side ? UM_XT_MN : UM_XT_K;
      a.A.S = p.S;
      a.A.d_shift = ilog2(p.D);
      a.B = a.A;
      a.C = G32;
      a.ldc = n;
      a.sC = n * n;
      a.status = c.status();
      JTRY(umma_run(c, m, a, 1));
    } else {
      JTRY(gemm(g, xtype(c), xtype(c), c.st));
    }
  }
  count_launch(), f32_to_f64_kernel<<<grid1d((long long)p.NU * n * n), 256, 0, c.st>>>(G32, G, (long long)p.NU * n * n);
  CUDA_TRY(cudaGetLastError());
  if (!p.m_side) return sym_eig_top(c, G, (int)n, p.NU, p.rTmax, Uf, nullptr, ldUf, (long long)T * ldUf, nullptr);
  // T > M: U = X_(T) V Lambda^{-1/2}, then CholeskyQR2 re-orthonormalisation
  float* V = c.at<float>(p.o_vsel);
  double* lam = c.at<double>(p.o_lam);
  JTRY(sym_eig_top(c, G, (int)n, p.NU, p.rTmax, V, nullptr, p.ldU, (long long)M * p.ldU, lam));
  count_launch(), scale_cols_kernel<<<grid1d((long long)p.NU * M * p.rTmax), 256, 0, c.st>>>(
      V, lam, M, p.rTmax, p.ldU, (long long)M * p.ldU, p.rTmax, p.NU, c.status());
  CUDA_TRY(cudaGetLastError());
  GemmParams y;
  y.M = T;
  y.N = p.rTmax;
  y.K = M;
  y.batch = p.NU;
  y.A = xt_units(c);
  y.B.kmajor = false;
  y.B.ld = p.ldU;
  y.B.sbatch = (long long)M * p.ldU;
  y.C = Uf;
  y.ldc = ldUf;
  y.sbatchC = (long long)T * ldUf;
  y.c_type = 0;
  if (umma_ok(p)) {
    bf16* hi = c.at<bf16>(p.o_h);
    bf16* lo = c.at<bf16>(p.o_l);
    const long long nF = (long long)p.NU * M * p.ldU;
    count_launch(), split_bf16_kernel<<<grid1d(nF), 256, 0, c.st>>>(V, hi, lo, nF);
    CUDA_TRY(cudaGetLastError());
    cudaError_t e = umma_x_product(c.k, c.v, p.nL, p.H, T, p.D, p.S, p.NU, false, hi, lo, p.ldU, p.rTmax, Uf, ldUf,
                                   c.status(), c.sched(), c.st);
    if (e != cudaSuccess) return fail(JOLT_ERR_CUDA, "tensor-core X-product: %s", cudaGetErrorString(e));
  } else {
    JTRY(gemm_xf(c, y, false, V, (long long)p.NU * M * p.ldU));
  }
  JTRY(cholqr_batched(c, Uf, T, p.rTmax, (int)ldUf, 2));
  return JOLT_OK;
}

// FlashJoLT: randomized subspace iteration (sketch, orthonormalise after every product),
// then the Rayleigh-Ritz step.  B B^T with B = Q^T X_(T) is Z^T Z for Z = X_(T)^T Q.
jolt_status run_token_randomized(const Ctx& c, float* Uf, long long ldUf) {
  const Plan& p = c.p;
  ProfScope ps("token_factor_randomized", c.st, p.NU);
  const int T = p.T, M = p.M, k = p.k, kp = p.kp, NU = p.NU;
  bf16* Om = c.at<bf16>(p.o_omega);
  float* Y = c.at<float>(p.o_Y);
  float* Z = c.at<float>(p.o_Zm);
  if (p.o_Y) CUDA_TRY(cudaMemsetAsync(Y, 0, (size_t)NU * T * kp * 4, c.st));   // no fp32 Y with the pairs
  CUDA_TRY(cudaMemsetAsync(Z, 0, (size_t)NU * M * kp * 4, c.st));
  count_launch(), omega_kernel<<<grid1d((long long)NU * M * kp), 256, 0, c.st>>>(Om, M, k, kp, (long long)M * kp,
                                                                                  c.seed, p.u0, NU);
  CUDA_TRY(cudaGetLastError());
  // products with X_(T) (Y side, T x k) and X_(T)^T (Z side, M x k)
  GemmParams gy;
  gy.M = T;
  gy.N = k;
  gy.K = M;
  gy.batch = NU;
  gy.A = xt_units(c);
  gy.B.kmajor = false;
  gy.B.ld = kp;
  gy.C = Y;
  gy.ldc = kp;
  gy.sbatchC = (long long)T * kp;
  gy.c_type = 0;
  GemmParams gz = gy;
  gz.M = M;
  gz.K = T;
  gz.A = xtT_units(c);
  gz.C = Z;
  gz.sbatchC = (long long)M * kp;
  const bool tc = umma_ok(p);
  // the pairs path: every T x k basis as bf16 hi + lo, in pair 0 or 1 (cur names Q's)
  const bool pairs = tc && p.o_h2;
  bf16* ph[2] = {c.at<bf16>(p.o_h), pairs ? c.at<bf16>(p.o_h2) : nullptr};
  bf16* pl[2] = {c.at<bf16>(p.o_l), pairs ? c.at<bf16>(p.o_l2) : nullptr};
  int cur = 0;
  if (pairs) {
    JTRY(umma_x(c, false, Om, nullptr, kp, ph[0], pl[0]));   // Y = X_(T) Omega, all kp columns
  } else if (tc) {
    JTRY(umma_product(c, false, Om, nullptr, Y));   // Y = X_(T) Omega
  } else {
    ProfScope ps0("sketch_product", c.st, NU);
    GemmParams g0 = gy;  // Y = X_(T) Omega
    g0.B.ptr = Om;
    g0.B.sbatch = (long long)M * kp;
    JTRY(gemm(g0, xtype(c), 0, c.st));
  }
  gy.B.sbatch = (long long)M * kp;   // Y = X_(T) Qz : B = Qz (M x k)
  gz.B.sbatch = (long long)T * kp;   // Z = X_(T)^T Q : B = Q (T x k)
  auto z_of = [&](const float* Q) -> jolt_status {  // Z = X_(T)^T Q
    return tc ? umma_product(c, true, nullptr, Q, Z) : gemm_xf(c, gz, false, Q, (long long)NU * T * kp);
  };
  auto y_of = [&](const float* Qz) -> jolt_status {  // Y = X_(T) Qz
    return tc ? umma_product(c, false, nullptr, Qz, Y) : gemm_xf(c, gy, false, Qz, (long long)NU * M * kp);
  };
  if (pairs) {
    bf16* mh = c.at<bf16>(p.o_mh);
    bf16* ml = c.at<bf16>(p.o_ml);
    JTRY(cholqr_tc_pairs(c, ph, pl, &cur, T, k, kp, p.q == 0 ? 2 : 1));
    for (int it = 0; it < p.q; ++it) {
      JTRY(umma_x(c, true, ph[cur], pl[cur], k, Z, nullptr));    // Z = X_(T)^T Q
      JTRY(cholqr_batched(c, Z, M, k, kp, 1));   // its scratch pair may overwrite Q: used above
      const long long nZ = (long long)NU * M * kp;
      count_launch(), split_bf16_kernel<<<grid1d(nZ), 256, 0, c.st>>>(Z, mh, ml, nZ);
      CUDA_TRY(cudaGetLastError());
      cur = 0;
      JTRY(umma_x(c, false, mh, ml, kp, ph[0], pl[0]));   // Y = X_(T) Qz
      JTRY(cholqr_tc_pairs(c, ph, pl, &cur, T, k, kp, it + 1 == p.q ? 2 : 1));
    }
    JTRY(umma_x(c, true, ph[cur], pl[cur], k, Z, nullptr));   // Rayleigh-Ritz: Z = X_(T)^T Q
  } else {
    JTRY(cholqr_batched(c, Y, T, k, kp, p.q == 0 ? 2 : 1));
    for (int it = 0; it < p.q; ++it) {
      JTRY(z_of(Y));
      JTRY(cholqr_batched(c, Z, M, k, kp, 1));
      JTRY(y_of(Z));
      JTRY(cholqr_batched(c, Y, T, k, kp, it + 1 == p.q ? 2 : 1));
    }
    // Rayleigh-Ritz: S = Z^T Z with Z = X_(T)^T Q  (k x k per unit)
    JTRY(z_of(Y));
  }
  float* gpart = c.at<float>(p.o_gpart);
  double* S = c.at<double>(p.o_G);
  const int ns = (int)ceil_div(M, 256);
  {
    ProfScope ps1("ritz_gram", c.st, NU);
    GemmParams g;
    g.M = k;
    g.N = k;
    g.K = M;
    g.batch = NU;
    g.A.ptr = Z;
    g.A.kmajor = false;
    g.A.ld = kp;
    g.A.sbatch = (long long)M * kp;
    g.B = g.A;
    g.C = gpart;
    g.ldc = k;
    g.sbatchC = (long long)ns * k * k;
    g.ssplitC = (long long)k * k;
    g.splits = ns;
    g.kchunk = 256;
    g.c_type = 0;
    g.sym = true;
    JTRY(gemm(g, 1, 1, c.st));
    count_launch(), reduce_splits_sym_kernel<float><<<grid1d((long long)NU * k * k), 256, 0, c.st>>>(
        gpart, S, NU, ns, k, k, sgemm_detail::BM);
    CUDA_TRY(cudaGetLastError());
  }
  float* V = c.at<float>(p.o_vsel);
  CUDA_TRY(cudaMemsetAsync(V, 0, (size_t)NU * kp * p.ldU * 4, c.st));   // rows k..kp stay zero
  JTRY(sym_eig_top(c, S, k, NU, p.rTmax, V, nullptr, p.ldU, (long long)kp * p.ldU, nullptr));
  // U = Q V
  ProfScope ps2("ritz_vectors", c.st, NU);
  if (p.o_vh) {
    // on the tensor cores: Q = Qh + Ql, V = Vh + Vl (bf16 hi + lo); U = Qh (Vh + Vl) + Ql Vh
    bf16* qh = ph[cur];
    bf16* ql = pl[cur];
    bf16* vh = c.at<bf16>(p.o_vh);
    bf16* vl = c.at<bf16>(p.o_vl);
    const long long nQ = (long long)NU * T * kp, nV = (long long)NU * kp * p.ldU;
    if (!pairs) count_launch(), split_bf16_cols_kernel<<<grid1d(nQ), 256, 0, c.st>>>(Y, qh, ql, nQ, kp, k);
    count_launch(), split_bf16_kernel<<<grid1d(nV), 256, 0, c.st>>>(V, vh, vl, nV);
    CUDA_TRY(cudaGetLastError());
    UmmaMaps mq, mv;
    if (!map_dense(&mq.a0, qh, kp, T, NU) || !map_dense(&mq.a1, ql, kp, T, NU) ||
        !map_dense(&mv.b0, vh, p.ldU, kp, NU) || !map_dense(&mv.b1, vl, p.ldU, kp, NU))
      return fail(JOLT_ERR_CUDA, "tensor map of the Ritz vectors refused");
    UmmaArgs a;
    a.M = T;
    a.N = p.rTmax;
    a.K = kp;
    a.batch = NU;
    a.A.mode = UM_DENSE_K;
    a.B.mode = UM_DENSE_MN;
    a.C = Uf;
    a.ldc = ldUf;
    a.sC = (long long)T * ldUf;
    a.status = c.status();
    UmmaMaps m3;   // Qh Vh + Qh Vl + Ql Vh in one pass
    m3.a0 = mq.a0;
    m3.a1 = mq.a1;
    m3.b0 = mv.b0;
    m3.b1 = mv.b1;
    JTRY(umma_run(c, m3, a, 3));
    return JOLT_OK;
  }
  GemmParams uq;
  uq.M = T;
  uq.N = p.rTmax;
  uq.K = k;
  uq.batch = NU;
  uq.A.ptr = Y;
  uq.A.kmajor = true;
  uq.A.ld = kp;
  uq.A.sbatch = (long long)T * kp;
  uq.B.ptr = V;
  uq.B.kmajor = false;
  uq.B.ld = p.ldU;
  uq.B.sbatch = (long long)kp * p.ldU;
  uq.C = Uf;
  uq.ldc = ldUf;
  uq.sbatchC = (long long)T * ldUf;
  uq.c_type = 0;
  JTRY(gemm(uq, 1, 1, c.st));
  return JOLT_OK;
}

jolt_status run_factor(const Ctx& c, float* Uf, long long ldUf, float* Wf, long long ldWf, bf16* Us, bf16* Ws) {
  const Plan& p = c.p;
  CUDA_TRY(cudaMemsetAsync(c.status(), 0, 4, c.st));
  // the feature factor (its Gram and a small eigen solve) runs on the auxiliary stream while
  // the token factor runs on the caller's; the two share only the status word (atomic OR)
  Aux* ax = nullptr;
  JTRY(aux_get(&ax));
  CUDA_TRY(cudaEventRecord(ax->fork, c.st));
  CUDA_TRY(cudaStreamWaitEvent(ax->st, ax->fork, 0));
  Ctx cf = c;
  cf.st = ax->st;
  cf.side = 1;
  JTRY(run_feature_factor(cf, Wf, ldWf, Ws));
  CUDA_TRY(cudaEventRecord(ax->join, ax->st));
  if (p.method == JOLT_EXACT) JTRY(run_token_exact(c, Uf, ldUf));
  else JTRY(run_token_randomized(c, Uf, ldUf));
  CUDA_TRY(cudaStreamWaitEvent(c.st, ax->join, 0));
  // sign convention of the token factor columns (the randomized and back-projected routes
  // need it; for the eigenvector route it is already in place) and the bf16 copy
  {
    ProfScope ps("sign_fix", c.st, p.NU);
    unsigned long long* keys = c.at<unsigned long long>(p.o_signkey);
    float* signs = c.at<float>(p.o_sign);
    const long long sU = (long long)p.T * ldUf;
    CUDA_TRY(cudaMemsetAsync(keys, 0, (size_t)p.NU * p.rTmax * 8, c.st));
    count_launch(), sign_key_kernel<<<dim3((unsigned)ceil_div(p.T, SK_ROWS), p.NU), 256, 0, c.st>>>(
        Uf, ldUf, sU, p.T, p.rTmax, keys);
    count_launch(), sign_of_kernel<<<p.NU, 1024, 0, c.st>>>(Uf, ldUf, sU, p.rTmax, keys, signs);
    count_launch(), sign_apply_kernel<<<grid1d((long long)p.NU * p.T * (p.rTmax / 4)), 256, 0, c.st>>>(
        Uf, ldUf, sU, p.T, p.rTmax, signs, Us, ldUf, sU, p.NU);
    CUDA_TRY(cudaGetLastError());
  }
  return JOLT_OK;
}

// ------------------------------------------------------------------------------------------
// stage 2: stored core, rotated reconstruction operators and the distortion table
// ------------------------------------------------------------------------------------------
jolt_status run_core(const Ctx& c, const bf16* Us, long long ldU, const bf16* Ws, long long ldW, bf16* core) {
  const Plan& p = c.p;
  ProfScope ps("core", c.st, p.NU);
  const int T = p.T, D = p.D, S = p.S;
  bf16* Zc = c.at<bf16>(p.o_zc);
  if (umma_ok(p)) {
    // Z_u = bf16(X_u W_u) token-major, Z[u][t][s * ldW + c]: one launch per unit, its slices as
    // the batch (A = the unit's cache slices [S][T][D], K-major; B = W_u, MN-major)
    const long long zld = (long long)S * p.ldW;
    for (int u = 0; u < p.NU; ++u) {
      const bf16* base = reinterpret_cast<const bf16*>((u & 1) ? c.v : c.k) + (long long)(u >> 1) * S * T * D;
      UmmaMaps m;
      if (!map_dense(&m.a0, base, D, T, S) || !map_dense(&m.b0, Ws + (long long)u * D * ldW, ldW, D, 1))
        return fail(JOLT_ERR_CUDA, "tensor map of X / W refused");
      m.a1 = m.a0;
      m.b1 = m.b0;
      UmmaArgs a;
      a.M = T;
      a.N = p.rDmax;
      a.K = D;
      a.batch = S;
      a.A.mode = UM_DENSE_K;
      a.B.mode = UM_DENSE_MN;
      a.B.ediv = S;   // every slice uses the unit's W
      a.C = Zc + (long long)u * T * zld;
      a.c_bf16 = 1;
      a.ldc = zld;
      a.sC = p.ldW;
      a.status = c.status();
      JTRY(umma_run(c, m, a, 1));
    }
    // C_u = bf16(U_u^T Z_u) (rTmax x S ldW per unit; N tiles of 256), then into the stored
    // layout [u][s][rTmax][ldC]
    bf16* Ct = c.at<bf16>(p.o_ctmp);
    UmmaMaps m2;
    if (!map_dense(&m2.a0, Us, ldU, T, p.NU) || !map_dense(&m2.b0, Zc, zld, T, p.NU))
      return fail(JOLT_ERR_CUDA, "tensor map of U / Z refused");
    m2.a1 = m2.a0;
    m2.b1 = m2.b0;
    UmmaArgs a2;
    a2.M = p.rTmax;
    a2.N = (int)zld;
    a2.K = T;
    a2.batch = p.NU;
    a2.A.mode = UM_DENSE_MN;
    a2.B.mode = UM_DENSE_MN;
    a2.C = Ct;
    a2.c_bf16 = 1;
    a2.ldc = zld;
    a2.sC = (long long)p.rTmax * zld;
    a2.status = c.status();
    JTRY(umma_run(c, m2, a2, 1));
    const long long n = (long long)p.NU * S * p.rTmax * p.ldC;
    count_launch(), core_permute_kernel<<<grid1d(n), 256, 0, c.st>>>(Ct, core, p.NU, S, p.rTmax, p.ldW, p.ldC);
    CUDA_TRY(cudaGetLastError());
    return JOLT_OK;
  }
  // Z = bf16(X_(D) W_s)   ((S T) x rDmax per unit)
  GemmParams z;
  z.M = S * T;
  z.N = p.rDmax;
  z.K = D;
  z.batch = p.NU;
  z.A.ptr = c.k;
  z.A.ptr_odd = c.v;
  z.A.kmajor = true;
  z.A.ld = D;
  z.A.sbatch = (long long)S * T * D;
  z.B.ptr = Ws;
  z.B.kmajor = false;
  z.B.ld = ldW;
  z.B.sbatch = (long long)D * ldW;
  z.C = Zc;
  z.ldc = p.ldW;
  z.sbatchC = (long long)S * T * p.ldW;
  z.c_type = 1;
  JTRY(gemm(z, xtype(c), 0, c.st));
  // C_s = bf16(U_s^T Z_s) per (unit, slice)  (rTmax x rDmax)
  GemmParams cc;
  cc.M = p.rTmax;
  cc.N = p.rDmax;
  cc.K = T;
  cc.batch = p.NU * S;
  cc.A.ptr = Us;
  cc.A.kmajor = false;
  cc.A.ld = ldU;
  cc.A.sbatch = (long long)T * ldU;
  cc.A.bdiv = S;
  cc.B.ptr = Zc;
  cc.B.kmajor = false;
  cc.B.ld = p.ldW;
  cc.B.sbatch = (long long)T * p.ldW;
  cc.C = core;
  cc.ldc = p.ldC;
  cc.sbatchC = (long long)p.rTmax * p.ldC;
  cc.c_type = 1;
  JTRY(gemm(cc, 0, 0, c.st));
  return JOLT_OK;
}


// P'(r_D) for one unit: bf16(rotate(C_s[:, :rT, :r_D] W_s[:, :r_D]^T)), rows rT of every slice
// out layout [S][rTslice][D] (rows >= rT of a slice are not written meaningfully)
template <int D>
jolt_status launch_pmat(const Ctx& c, const bf16* core, long long ldC, long long sC, int rT, int rD, const bf16* Ws,
                        long long ldW, long long sW, int nb, const int* umap, bf16* out, long long sOut) {
  count_launch(), pmat_exact_kernel<D><<<dim3((unsigned)ceil_div(rT, PX_ROWS), (unsigned)nb), 256, 0, c.st>>>(
      core, ldC, sC, rT, rD, Ws, ldW, sW, c.p.S, umap, c.seed, out, sOut);
  CUDA_TRY(cudaGetLastError());
  return JOLT_OK;
}

// P'(r_D) of the rT leading token ranks of nb batch entries (slices; entry b of unit umap[b / S]):
// bf16(rotate(C_b[:rT, :r_D] W[:, :r_D]^T)) in fp64 (pmat_exact_kernel); out entry stride sOut
jolt_status pmat_run(const Ctx& c, const bf16* core, long long ldC, long long sC, int rT, const bf16* Ws, long long ldW,
                     long long sW, int rD, int nb, const int* umap, bf16* out, long long sOut) {
  switch (c.p.D) {
    case 16: return launch_pmat<16>(c, core, ldC, sC, rT, rD, Ws, ldW, sW, nb, umap, out, sOut);
    case 32: return launch_pmat<32>(c, core, ldC, sC, rT, rD, Ws, ldW, sW, nb, umap, out, sOut);
    case 64: return launch_pmat<64>(c, core, ldC, sC, rT, rD, Ws, ldW, sW, nb, umap, out, sOut);
    default: return launch_pmat<128>(c, core, ldC, sC, rT, rD, Ws, ldW, sW, nb, umap, out, sOut);
  }
}

// one unit's operator (the decoder): S slices of core_u (slice stride rT * ldC), W of unit u
jolt_status pmat_unit(const Ctx& c, int u, const bf16* core_u, long long ldC, int rT, int rTslice, const bf16* Ws_u,
                      long long ldW, int rD, float* /*ptmp*/, bf16* out, const int* umap) {
  const Plan& p = c.p;
  return pmat_run(c, core_u, ldC, (long long)rT * ldC, rT, Ws_u, ldW, 0, rD, p.S, umap + u, out,
                  (long long)rTslice * p.D);
}

// P'(r_D) of every unit; out layout [unit][S][rTslice][D] (unit stride S*rTslice*D)
jolt_status pmat_all(const Ctx& c, const bf16* core, long long ldC, int rT, int rTslice, const bf16* Ws, long long ldW,
                     int rD, float* /*ptmp*/, bf16* out, const int* umap) {
  const Plan& p = c.p;
  return pmat_run(c, core, ldC, (long long)rT * ldC, rT, Ws, ldW, (long long)p.D * ldW, rD, p.NU * p.S, umap, out,
                  (long long)rTslice * p.D);
}

jolt_status fill_umap(const Ctx& c, int* umap, int n) {
  count_launch(), iota_kernel<<<(unsigned)ceil_div(n, 128), 128, 0, c.st>>>(umap, n, c.p.u0);
  CUDA_TRY(cudaGetLastError());
  return JOLT_OK;
}

template <int D, typename TX, typename BITS>
jolt_status launch_table_B(const Ctx& c, const TableArgs& a) {
  size_t sm = table_smem<D>();
  CUDA_TRY(cudaFuncSetAttribute(table_kernel<D, TX, BITS>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sm));
  count_launch(), table_kernel<D, TX, BITS><<<dim3(c.p.tiles, c.p.S, c.p.NU), table_threads<D>(), sm, c.st>>>(a);
  CUDA_TRY(cudaGetLastError());
  return JOLT_OK;
}

// the default bit-width set {0,1,2,3,4,8} has its own instantiation (constants folded)
template <int D, typename TX>
jolt_status launch_table_T(const Ctx& c, const TableArgs& a) {
  const Cands& cd = c.p.cd;
  const bool dflt = cd.nB == 6 && cd.bits[0] == 0 && cd.bits[1] == 1 && cd.bits[2] == 2 && cd.bits[3] == 3 &&
                    cd.bits[4] == 4 && cd.bits[5] == 8;
  return dflt ? launch_table_B<D, TX, DefaultBits>(c, a) : launch_table_B<D, TX, void>(c, a);
}

template <int D>
jolt_status launch_table_D(const Ctx& c, const TableArgs& a) {
  return c.p.dtype == JOLT_BF16 ? launch_table_T<D, bf16>(c, a) : launch_table_T<D, float>(c, a);
}

// the tensor-core table kernel takes D = 128 with at most 4 token-rank cuts, each a multiple
// of 16 (one K step of the MMA never straddles two cuts), and a U pitch of 16-byte rows
bool table_tc_ok(const Plan& p, long long ldU) {
  if (p.D != ttc::DIM || p.cd.nT > ttc::MAXT || ldU % 8) return false;
  for (int i = 0; i < p.cd.nT; ++i)
    if (p.cd.rT[i] % 16) return false;
  return true;
}

template <typename TX, typename BITS>
jolt_status launch_table_tc_B(const Ctx& c, const CUtensorMap& mu, const CUtensorMap& mp, const TableTcArgs& a) {
  CUDA_TRY(cudaFuncSetAttribute(table_tc_kernel<TX, BITS>, cudaFuncAttributeMaxDynamicSharedMemorySize, ttc::SMEM));
  count_launch(), table_tc_kernel<TX, BITS><<<dim3((unsigned)(a.tiles * c.p.S), c.p.NU), ttc::THREADS, ttc::SMEM, c.st>>>(mu, mp, a);
  CUDA_TRY(cudaGetLastError());
  return JOLT_OK;
}

jolt_status launch_table_tc(const Ctx& c, const bf16* Us, long long ldU, const bf16* P, const TableTcArgs& a) {
  const Plan& p = c.p;
  CUtensorMap mu, mp;
  if (!map_dense(&mu, Us, ldU, p.T, p.NU) || !map_dense(&mp, P, p.D, p.rTmax, (long long)p.cd.nD * p.NU * p.S))
    return fail(JOLT_ERR_CUDA, "tensor map of the table operands refused");
  const Cands& cd = p.cd;
  const bool dflt = cd.nB == 6 && cd.bits[0] == 0 && cd.bits[1] == 1 && cd.bits[2] == 2 && cd.bits[3] == 3 &&
                    cd.bits[4] == 4 && cd.bits[5] == 8;
  if (p.dtype == JOLT_BF16)
    return dflt ? launch_table_tc_B<bf16, DefaultBits>(c, mu, mp, a) : launch_table_tc_B<bf16, void>(c, mu, mp, a);
  return dflt ? launch_table_tc_B<float, DefaultBits>(c, mu, mp, a) : launch_table_tc_B<float, void>(c, mu, mp, a);
}

jolt_status run_table(const Ctx& c, const bf16* Us, long long ldU, const bf16* Ws, long long ldW, bf16* core,
                      double* table) {
  const Plan& p = c.p;
  JTRY(run_core(c, Us, ldU, Ws, ldW, core));
  bf16* P = c.at<bf16>(p.o_P);
  int* umap = c.at<int>(p.o_umap);
  JTRY(fill_umap(c, umap, p.NU));
  const long long sP_unit = (long long)p.S * p.rTmax * p.D;
  const long long sP_rd = p.NU * sP_unit;
  {
    ProfScope ps("recon_operator", c.st, p.NU);
    for (int iD = 0; iD < p.cd.nD; ++iD)
      JTRY(pmat_all(c, core, p.ldC, p.rTmax, p.rTmax, Ws, ldW, p.cd.rD[iD], c.at<float>(p.o_ptmp), P + iD * sP_rd,
                    umap));
  }
  TableArgs a;
  a.cv = c.view();
  a.U = Us;
  a.ldU = ldU;
  a.sU = (long long)p.T * ldU;
  a.P = P;
  a.sP_unit = sP_unit;
  a.sP_rd = sP_rd;
  a.rTmax = p.rTmax;
  a.cand = p.cd;
  a.seed = c.seed;
  a.partial = c.at<double>(p.o_partial);
  a.tiles = p.tiles;
  int tiles = p.tiles;
  if (table_tc_ok(p, ldU)) {
    ProfScope ps("table_kernel", c.st, p.NU);
    TableTcArgs t;
    t.cv = a.cv;
    t.rTmax = p.rTmax;
    t.cand = p.cd;
    t.seed = c.seed;
    t.partial = a.partial;
    t.tiles = tiles = (int)ceil_div(p.T, ttc::ROWS);
    t.status = c.status();
    JTRY(launch_table_tc(c, Us, ldU, P, t));
  } else {
    ProfScope ps("table_kernel", c.st, p.NU);
    switch (p.D) {
      case 16: JTRY(launch_table_D<16>(c, a)); break;
      case 32: JTRY(launch_table_D<32>(c, a)); break;
      case 64: JTRY(launch_table_D<64>(c, a)); break;
      default: JTRY(launch_table_D<128>(c, a)); break;
    }
  }
  count_launch(), table_reduce_kernel<<<(unsigned)((long long)p.NU * p.nC), 256, 0, c.st>>>(
      a.partial, table, p.NU, p.S, tiles, p.cd.nT, p.cd.nD, p.cd.nB);
  CUDA_TRY(cudaGetLastError());
  return JOLT_OK;
}

// ------------------------------------------------------------------------------------------
// stage 4: encode
// ------------------------------------------------------------------------------------------
template <int D, typename TX>
jolt_status launch_encode_T(const Ctx& c, const EncodeArgs& a) {
  size_t sm = table_smem<D>();
  CUDA_TRY(cudaFuncSetAttribute(encode_kernel<D, TX>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sm));
  count_launch(), encode_kernel<D, TX><<<dim3(c.p.tiles, c.p.S, c.p.NU), TTHREADS, sm, c.st>>>(a);
  CUDA_TRY(cudaGetLastError());
  return JOLT_OK;
}
template <int D>
jolt_status launch_encode_D(const Ctx& c, const EncodeArgs& a) {
  return c.p.dtype == JOLT_BF16 ? launch_encode_T<D, bf16>(c, a) : launch_encode_T<D, float>(c, a);
}

BlobHeader header_proto(const Plan& p, uint64_t seed) {
  BlobHeader h;
  memset(&h, 0, sizeof h);
  h.magic = kMagic;
  h.version = kVersion;
  h.n_units = (uint32_t)p.NU;
  h.status = 0;
  h.n_layers = p.nL;
  h.n_heads = p.H;
  h.n_tokens = p.T;
  h.head_dim = p.D;
  h.layers_per_group = p.Lg;
  h.dtype = p.dtype;
  h.block = 16;
  h.unit_offset = p.u0;
  h.seed = seed;
  return h;
}

jolt_status run_allocate(const Ctx& c, const double* table, unsigned long long budget_payload, unsigned char* blob,
                         size_t blob_cap, const int32_t* forced_choice) {
  const Plan& p = c.p;
  ProfScope ps("allocate", c.st, 1);
  unsigned long long* B = c.at<unsigned long long>(p.o_bytes);
  count_launch(), bytes_table_kernel<<<(unsigned)ceil_div((long long)p.NU * p.nC, 128), 128, 0, c.st>>>(B, p.NU, p.T, p.D, p.S, p.cd);
  CUDA_TRY(cudaGetLastError());
  AllocArgs a;
  memset(&a, 0, sizeof a);
  a.D = table;
  a.B = B;
  a.nunits = p.NU;
  a.nc = p.nC;
  a.budget = forced_choice ? ~0ull : budget_payload;
  a.choice = c.at<int>(p.o_choice);
  a.lambda = c.at<double>(p.o_lambda);
  a.status = c.status();
  a.blob = blob;
  a.blob_cap = blob_cap;
  a.header_bytes = 64ull + 64ull * p.NU;
  a.T = p.T;
  a.D_ = p.D;
  a.S = p.S;
  a.cd = p.cd;
  a.hdr = header_proto(p, c.seed);
  size_t sm = (size_t)((p.NU * 4 + 15) / 16) * 16 + (size_t)p.NU * 8;
  a.forced = forced_choice;  // caller's choices (jolt_encode): same header filling, no search
  count_launch(), allocate_kernel<<<1, 512, sm, c.st>>>(a);
  CUDA_TRY(cudaGetLastError());
  return JOLT_OK;
}

jolt_status run_encode(const Ctx& c, const bf16* Us, long long ldU, const bf16* Ws, long long ldW, const bf16* core,
                       unsigned char* blob) {
  const Plan& p = c.p;
  EncodeArgs a;
  a.cv = c.view();
  a.U = Us;
  a.ldU = ldU;
  a.sU = (long long)p.T * ldU;
  a.P = c.at<bf16>(p.o_P);
  a.sP_unit = (long long)p.S * p.rTmax * p.D;
  a.sP_rd = p.NU * a.sP_unit;
  a.rTmax = p.rTmax;
  a.cand = p.cd;
  a.seed = c.seed;
  a.blob = blob;
  ProfScope ps("encode", c.st, p.NU);
  if (table_tc_ok(p, ldU)) {
    // the tensor-core encoder (every candidate token rank a multiple of 16, D = 128)
    CUtensorMap mu, mp;
    if (!map_dense(&mu, Us, ldU, p.T, p.NU) || !map_dense(&mp, a.P, p.D, p.rTmax, (long long)p.cd.nD * p.NU * p.S))
      return fail(JOLT_ERR_CUDA, "tensor map of the encoder operands refused");
    EncodeTcArgs e;
    e.cv = a.cv;
    e.rTmax = p.rTmax;
    e.cand = p.cd;
    e.seed = c.seed;
    e.blob = blob;
    e.status = c.status();
    const dim3 grid((unsigned)(ceil_div(p.T, ttc::ROWS) * p.S), p.NU);   // slices fastest
    if (p.dtype == JOLT_BF16) {
      CUDA_TRY(cudaFuncSetAttribute(encode_tc_kernel<bf16>, cudaFuncAttributeMaxDynamicSharedMemorySize, ttc::SMEM));
      count_launch(), encode_tc_kernel<bf16><<<grid, etc::THREADS, ttc::SMEM, c.st>>>(mu, mp, e);
    } else {
      CUDA_TRY(cudaFuncSetAttribute(encode_tc_kernel<float>, cudaFuncAttributeMaxDynamicSharedMemorySize, ttc::SMEM));
      count_launch(), encode_tc_kernel<float><<<grid, etc::THREADS, ttc::SMEM, c.st>>>(mu, mp, e);
    }
    CUDA_TRY(cudaGetLastError());
  } else {
    switch (p.D) {
      case 16: JTRY(launch_encode_D<16>(c, a)); break;
      case 32: JTRY(launch_encode_D<32>(c, a)); break;
      case 64: JTRY(launch_encode_D<64>(c, a)); break;
      default: JTRY(launch_encode_D<128>(c, a)); break;
    }
  }
  count_launch(), copy_factors_kernel<<<dim3(64, p.NU), 256, 0, c.st>>>(blob, Us, ldU, (long long)p.T * ldU, Ws, ldW,
                                                         (long long)p.D * ldW, core, p.ldC, (long long)p.rTmax * p.ldC,
                                                         (long long)p.S * p.rTmax * p.ldC, p.T, p.D, p.S);
  CUDA_TRY(cudaGetLastError());
  return JOLT_OK;
}

jolt_status check_ws(const Plan& p, void* ws, size_t ws_bytes) {
  if (!ws) return fail(JOLT_ERR_INVALID_ARG, "null workspace");
  if (ws_bytes < p.ws_total)
    return fail(JOLT_ERR_WORKSPACE_TOO_SMALL, "workspace %zu bytes, need %zu", ws_bytes, p.ws_total);
  if (reinterpret_cast<uintptr_t>(ws) % 256) return fail(JOLT_ERR_INVALID_ARG, "workspace not 256-byte aligned");
  return JOLT_OK;
}

jolt_status check_inputs(const Plan& p, const void* k, const void* v) {
  if (!k || !v) return fail(JOLT_ERR_INVALID_ARG, "null cache pointer");
  if (reinterpret_cast<uintptr_t>(k) % 16 || reinterpret_cast<uintptr_t>(v) % 16)
    return fail(JOLT_ERR_INVALID_ARG, "cache pointers must be 16-byte aligned");
  (void)p;
  return JOLT_OK;
}

jolt_status check_aligned(const void* q, const char* name) {
  if (!q) return fail(JOLT_ERR_INVALID_ARG, "null %s", name);
  if (reinterpret_cast<uintptr_t>(q) % 16) return fail(JOLT_ERR_INVALID_ARG, "%s must be 16-byte aligned", name);
  return JOLT_OK;
}

}  // namespace

// ==========================================================================================
// C ABI
// ==========================================================================================
extern "C" {

const char* jolt_version(void) { return "jolt-b200 1.0 (sm_100a)"; }

const char* jolt_last_error(void) { return g_err.c_str(); }

uint64_t jolt_launch_count(void) { return launch_counter().load(); }

jolt_status jolt_profile_begin(void) {
  for (auto& r : g_prof.recs) {
    g_prof.pool.push_back(r.a);
    g_prof.pool.push_back(r.b);
  }
  g_prof.recs.clear();
  g_prof.on = true;
  return JOLT_OK;
}

jolt_status jolt_profile_end(char* buf, size_t cap) {
  g_prof.on = false;
  std::vector<std::string> names;
  std::vector<double> ms;
  std::vector<long long> cnt, units;
  for (auto& r : g_prof.recs) {
    CUDA_TRY(cudaEventSynchronize(r.b));
    float t = 0.f;
    CUDA_TRY(cudaEventElapsedTime(&t, r.a, r.b));
    size_t i = 0;
    while (i < names.size() && names[i] != r.name) ++i;
    if (i == names.size()) {
      names.push_back(r.name);
      ms.push_back(0.0);
      cnt.push_back(0);
      units.push_back(0);
    }
    ms[i] += t;
    cnt[i] += 1;
    units[i] += r.units;
  }
  std::string out;
  char line[256];
  for (size_t i = 0; i < names.size(); ++i) {
    snprintf(line, sizeof line, "%s %.6f %lld %lld\n", names[i].c_str(), ms[i], cnt[i], units[i]);
    out += line;
  }
  if (buf && cap) {
    size_t n = out.size() < cap - 1 ? out.size() : cap - 1;
    memcpy(buf, out.data(), n);
    buf[n] = 0;
  }
  return JOLT_OK;
}

jolt_status jolt_fp32_rate_probe(int32_t packed, int32_t iters, float* sink_dev, uint64_t* fma_ops, void* stream) {
  if (!sink_dev || !fma_ops || iters < 1) return fail(JOLT_ERR_INVALID_ARG, "null sink / ops or iters < 1");
  int dev = 0, sms = 0;
  CUDA_TRY(cudaGetDevice(&dev));
  CUDA_TRY(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev));
  const unsigned blocks = (unsigned)sms * 8u;
  count_launch(), fma_probe_kernel<<<blocks, 256, 0, (cudaStream_t)stream>>>(sink_dev, iters, packed ? 1 : 0,
                                                                              0.99993896484375f, 6.103515625e-05f);
  CUDA_TRY(cudaGetLastError());
  *fma_ops = (uint64_t)blocks * 256ull * (uint64_t)iters * (uint64_t)FP32_CHAINS * (packed ? 2ull : 1ull);
  return JOLT_OK;
}

jolt_status jolt_wait_selftest(int32_t arrive, uint32_t limit_us, uint32_t* status_dev, void* stream) {
  if (!status_dev) return fail(JOLT_ERR_INVALID_ARG, "null status word");
  if (limit_us < 1 || limit_us > 5000000u) return fail(JOLT_ERR_INVALID_ARG, "limit_us %u not in [1, 5e6]", limit_us);
  cudaStream_t st = (cudaStream_t)stream;
  CUDA_TRY(cudaMemsetAsync(status_dev, 0, 4, st));
  count_launch(), umma::wait_selftest_kernel<<<1, 32, 0, st>>>(arrive ? 1 : 0, (uint64_t)limit_us * 1000ull,
                                                                 status_dev);
  CUDA_TRY(cudaGetLastError());
  uint32_t h = 0;
  CUDA_TRY(cudaMemcpyAsync(&h, status_dev, 4, cudaMemcpyDeviceToHost, st));
  CUDA_TRY(cudaStreamSynchronize(st));
  if (h & DEV_ERR_TIMEOUT) return fail(JOLT_ERR_TIMEOUT, "bounded device wait gave up after %u us", limit_us);
  if (h) return fail(JOLT_ERR_CUDA, "unexpected device status %u", h);
  return JOLT_OK;
}

jolt_status jolt_workspace_size(const jolt_shape* shape, const jolt_options* opts, size_t* ws_bytes,
                                size_t* blob_bytes, size_t* dws_bytes) {
  Plan p;
  JTRY(make_plan(shape, opts, &p));
  if (ws_bytes) *ws_bytes = p.ws_total;
  if (blob_bytes) *blob_bytes = p.blob_max;
  if (dws_bytes) *dws_bytes = p.dws_total;
  return JOLT_OK;
}

jolt_status jolt_counts(const jolt_shape* shape, const jolt_options* opts, int32_t* n_units, int32_t* n_choices) {
  Plan p;
  JTRY(make_plan(shape, opts, &p));
  if (n_units) *n_units = p.NU;
  if (n_choices) *n_choices = p.nC;
  return JOLT_OK;
}

jolt_status jolt_choice_bytes(const jolt_shape* shape, const jolt_options* opts, uint64_t* bytes_host) {
  Plan p;
  JTRY(make_plan(shape, opts, &p));
  if (!bytes_host) return fail(JOLT_ERR_INVALID_ARG, "null output");
  for (int c = 0; c < p.nC; ++c) {
    int ib = c % p.cd.nB, iD = (c / p.cd.nB) % p.cd.nD, iT = c / (p.cd.nB * p.cd.nD);
    bytes_host[c] = unit_payload_bytes(p.T, p.D, p.S, p.cd.rT[iT], p.cd.rD[iD], p.cd.bits[ib]);
  }
  return JOLT_OK;
}

jolt_status jolt_factor(const jolt_shape* shape, const void* k_dev, const void* v_dev, const jolt_options* opts,
                        uint64_t seed, float* u_dev, int64_t ld_u, float* w_dev, int64_t ld_w, void* ws_dev,
                        size_t ws_bytes, void* stream) {
  Plan p;
  JTRY(make_plan(shape, opts, &p));
  JTRY(check_ws(p, ws_dev, ws_bytes));
  JTRY(check_inputs(p, k_dev, v_dev));
  if (!u_dev || !w_dev || ld_u < p.rTmax || ld_w < p.rDmax) return fail(JOLT_ERR_INVALID_ARG, "factor outputs");
  if (ld_u % 8) return fail(JOLT_ERR_INVALID_ARG, "ld_u %lld not a multiple of 8", (long long)ld_u);
  Ctx c{p, (unsigned char*)ws_dev, (cudaStream_t)stream, k_dev, v_dev, seed};
  return run_factor(c, u_dev, ld_u, w_dev, ld_w, nullptr, nullptr);
}

jolt_status jolt_table(const jolt_shape* shape, const void* k_dev, const void* v_dev, const jolt_options* opts,
                       uint64_t seed, const void* u_bf16_dev, int64_t ld_u, const void* w_bf16_dev, int64_t ld_w,
                       void* core_dev, double* table_dev, void* ws_dev, size_t ws_bytes, void* stream) {
  Plan p;
  JTRY(make_plan(shape, opts, &p));
  JTRY(check_ws(p, ws_dev, ws_bytes));
  JTRY(check_inputs(p, k_dev, v_dev));
  JTRY(check_aligned(u_bf16_dev, "u_bf16"));
  JTRY(check_aligned(w_bf16_dev, "w_bf16"));
  JTRY(check_aligned(core_dev, "core"));
  JTRY(check_aligned(table_dev, "table"));
  if (ld_u < p.rTmax || ld_w < p.rDmax || ld_u % 8 || ld_w % 8)
    return fail(JOLT_ERR_INVALID_ARG, "ld_u / ld_w must cover the largest rank and be multiples of 8");
  Ctx c{p, (unsigned char*)ws_dev, (cudaStream_t)stream, k_dev, v_dev, seed};
  CUDA_TRY(cudaMemsetAsync(c.status(), 0, 4, c.st));
  return run_table(c, (const bf16*)u_bf16_dev, ld_u, (const bf16*)w_bf16_dev, ld_w, (bf16*)core_dev, table_dev);
}

jolt_status jolt_recon_operator(const jolt_shape* shape, const jolt_options* opts, uint64_t seed,
                                const void* core_dev, const void* w_bf16_dev, int64_t ld_w, void* p_dev, void* ws_dev,
                                size_t ws_bytes, void* stream) {
  Plan p;
  JTRY(make_plan(shape, opts, &p));
  JTRY(check_ws(p, ws_dev, ws_bytes));
  JTRY(check_aligned(core_dev, "core"));
  JTRY(check_aligned(w_bf16_dev, "w_bf16"));
  JTRY(check_aligned(p_dev, "p"));
  if (ld_w < p.rDmax || ld_w % 8) return fail(JOLT_ERR_INVALID_ARG, "ld_w must cover the largest rank, multiple of 8");
  Ctx c{p, (unsigned char*)ws_dev, (cudaStream_t)stream, nullptr, nullptr, seed};
  int* umap = c.at<int>(p.o_umap);
  JTRY(fill_umap(c, umap, p.NU));
  const long long sP_rd = (long long)p.NU * p.S * p.rTmax * p.D;
  const bf16* core = (const bf16*)core_dev;
  const bf16* Ws = (const bf16*)w_bf16_dev;
  bf16* P = (bf16*)p_dev;
  ProfScope ps("recon_operator", c.st, p.NU);
  for (int iD = 0; iD < p.cd.nD; ++iD)
    JTRY(pmat_all(c, core, p.ldC, p.rTmax, p.rTmax, Ws, ld_w, p.cd.rD[iD], c.at<float>(p.o_ptmp), P + iD * sP_rd,
                  umap));
  return JOLT_OK;
}

jolt_status jolt_allocate(const double* dist_dev, const uint64_t* bytes_dev, int32_t n_units, int32_t n_choices,
                          uint64_t budget_bytes, int32_t* choice_dev, double* lambda_dev, uint32_t* status_dev,
                          void* stream) {
  if (!dist_dev || !bytes_dev || !choice_dev || !lambda_dev || !status_dev || n_units < 1 || n_choices < 1)
    return fail(JOLT_ERR_INVALID_ARG, "jolt_allocate arguments");
  cudaStream_t st = (cudaStream_t)stream;
  CUDA_TRY(cudaMemsetAsync(status_dev, 0, 4, st));
  AllocArgs a;
  memset(&a, 0, sizeof a);
  a.D = dist_dev;
  a.B = (const unsigned long long*)bytes_dev;
  a.nunits = n_units;
  a.nc = n_choices;
  a.budget = budget_bytes;
  a.choice = choice_dev;
  a.lambda = lambda_dev;
  a.status = status_dev;
  size_t sm = (size_t)((n_units * 4 + 15) / 16) * 16 + (size_t)n_units * 8;
  count_launch(), allocate_kernel<<<1, 512, sm, st>>>(a);
  CUDA_TRY(cudaGetLastError());
  return JOLT_OK;
}

jolt_status jolt_encode(const jolt_shape* shape, const void* k_dev, const void* v_dev, const jolt_options* opts,
                        uint64_t seed, const void* u_bf16_dev, int64_t ld_u, const void* w_bf16_dev, int64_t ld_w,
                        const void* core_dev, const int32_t* choice_dev, const double* dist_dev, void* blob_dev,
                        size_t blob_cap, void* ws_dev, size_t ws_bytes, void* stream) {
  Plan p;
  JTRY(make_plan(shape, opts, &p));
  JTRY(check_ws(p, ws_dev, ws_bytes));
  JTRY(check_inputs(p, k_dev, v_dev));
  JTRY(check_aligned(u_bf16_dev, "u_bf16"));
  JTRY(check_aligned(w_bf16_dev, "w_bf16"));
  JTRY(check_aligned(core_dev, "core"));
  JTRY(check_aligned(blob_dev, "blob"));
  if (!choice_dev || !dist_dev) return fail(JOLT_ERR_INVALID_ARG, "null pointer");
  if (ld_u < p.rTmax || ld_w < p.rDmax || ld_u % 8 || ld_w % 8)
    return fail(JOLT_ERR_INVALID_ARG, "ld_u / ld_w must cover the largest rank and be multiples of 8");
  Ctx c{p, (unsigned char*)ws_dev, (cudaStream_t)stream, k_dev, v_dev, seed};
  CUDA_TRY(cudaMemsetAsync(c.status(), 0, 4, c.st));
  // P' of every feature rank from the given core (the encoder's reconstruction operators)
  bf16* P = c.at<bf16>(p.o_P);
  int* umap = c.at<int>(p.o_umap);
  JTRY(fill_umap(c, umap, p.NU));
  const long long sP_rd = (long long)p.NU * p.S * p.rTmax * p.D;
  const bf16* core = (const bf16*)core_dev;
  const bf16* Ws = (const bf16*)w_bf16_dev;
  for (int iD = 0; iD < p.cd.nD; ++iD)
    JTRY(pmat_all(c, core, p.ldC, p.rTmax, p.rTmax, Ws, ld_w, p.cd.rD[iD], c.at<float>(p.o_ptmp), P + iD * sP_rd,
                  umap));
  JTRY(run_allocate(c, dist_dev, 0, (unsigned char*)blob_dev, blob_cap, choice_dev));
  return run_encode(c, (const bf16*)u_bf16_dev, ld_u, Ws, ld_w, core, (unsigned char*)blob_dev);
}

// the compress stages of one call, enqueued on c.st
jolt_status compress_body(const Ctx& c, uint64_t budget_bytes, unsigned long long hdr, void* blob_dev,
                          size_t blob_cap) {
  const Plan& p = c.p;
  float* Uf = c.at<float>(p.o_Uf);
  float* Wf = c.at<float>(p.o_Wf);
  bf16* Us = c.at<bf16>(p.o_Us);
  bf16* Ws = c.at<bf16>(p.o_Ws);
  JTRY(run_factor(c, Uf, p.ldU, Wf, p.ldW, Us, Ws));
  bf16* core = c.at<bf16>(p.o_core);
  double* table = c.at<double>(p.o_table);
  JTRY(run_table(c, Us, p.ldU, Ws, p.ldW, core, table));
  JTRY(run_allocate(c, table, budget_bytes - hdr, (unsigned char*)blob_dev, blob_cap, nullptr));
  JTRY(run_encode(c, Us, p.ldU, Ws, p.ldW, core, (unsigned char*)blob_dev));
  // device-side errors of the factor stage are folded into the header status
  count_launch(), fold_status_kernel<<<1, 1, 0, c.st>>>(c.status(), (unsigned char*)blob_dev);
  CUDA_TRY(cudaGetLastError());
  return JOLT_OK;
}

// ------------------------------------------------------------------------------------------
// CUDA graphs of whole compress calls.  A call whose arguments (shape, options, every
// pointer and size, budget, seed, device) equal those of an earlier call of this thread
// replays that call's graph: the same kernels on the same buffers, launched with one
// cudaGraphLaunch instead of ~2000 stream launches (most of them inside cuSOLVER's batched
// eigen solver and Cholesky).  The graph is captured on a private stream and launched on
// the caller's; a call that cannot be captured runs directly.
// ------------------------------------------------------------------------------------------
struct GraphKey {
  jolt_shape sh;
  jolt_options op;
  const void *k, *v;
  uint64_t budget, seed;
  void* blob;
  size_t cap;
  void* ws;
  size_t ws_bytes;
  int device;
};
struct GraphEntry {
  GraphKey key;
  cudaGraphExec_t exec = nullptr;
  unsigned long long launches = 0;
  unsigned long long last = 0;
  bool failed = false;    // capture not possible for these arguments: run directly
};
constexpr size_t kMaxGraphs = 8;
struct GraphCache {
  std::vector<GraphEntry> e;
  unsigned long long tick = 0;
  cudaStream_t cap_stream = nullptr;
  int cap_device = -1;
  bool on = true;
  ~GraphCache() {
    for (auto& g : e)
      if (g.exec) cudaGraphExecDestroy(g.exec);
  }
};
thread_local GraphCache g_graphs;

void graph_insert(GraphCache& gc, const GraphEntry& ent) {
  if (gc.e.size() >= kMaxGraphs) {
    size_t lru = 0;
    for (size_t i = 1; i < gc.e.size(); ++i)
      if (gc.e[i].last < gc.e[lru].last) lru = i;
    if (gc.e[lru].exec) cudaGraphExecDestroy(gc.e[lru].exec);
    gc.e.erase(gc.e.begin() + lru);
  }
  gc.e.push_back(ent);
}

// first call with a key: runs directly (so every lazily created library resource exists);
// second call: captured and launched; later calls: replayed
jolt_status compress_graph(const Ctx& c, const GraphKey& key, uint64_t budget_bytes, unsigned long long hdr,
                           void* blob_dev, size_t blob_cap) {
  GraphCache& gc = g_graphs;
  ++gc.tick;
  GraphEntry* hit = nullptr;
  for (auto& g : gc.e)
    if (memcmp(&g.key, &key, sizeof key) == 0) hit = &g;
  if (!hit) {
    GraphEntry ent;
    ent.key = key;
    ent.last = gc.tick;
    graph_insert(gc, ent);
    return compress_body(c, budget_bytes, hdr, blob_dev, blob_cap);
  }
  hit->last = gc.tick;
  if (hit->failed) return compress_body(c, budget_bytes, hdr, blob_dev, blob_cap);
  if (hit->exec) {
    CUDA_TRY(cudaGraphLaunch(hit->exec, c.st));
    launch_counter().fetch_add(hit->launches, std::memory_order_relaxed);
    return JOLT_OK;
  }
  if (gc.cap_stream == nullptr || gc.cap_device != key.device) {
    CUDA_TRY(cudaStreamCreateWithFlags(&gc.cap_stream, cudaStreamNonBlocking));
    gc.cap_device = key.device;
  }
  // resources the body creates on first use exist already (the first call ran directly);
  // capture the body on the private stream; the graph is launched on the caller's stream,
  // which orders it after the caller's earlier work
  Ctx cc = c;
  cc.st = gc.cap_stream;
  unsigned long long counted = 0;
  cudaGraph_t graph = nullptr;
  jolt_status st = JOLT_OK;
  bool ok = false;
  if (cudaStreamBeginCapture(gc.cap_stream, cudaStreamCaptureModeThreadLocal) == cudaSuccess) {
    capture_counter() = &counted;
    st = compress_body(cc, budget_bytes, hdr, blob_dev, blob_cap);
    capture_counter() = nullptr;
    const cudaError_t e = cudaStreamEndCapture(gc.cap_stream, &graph);
    ok = st == JOLT_OK && e == cudaSuccess && graph && cudaGraphInstantiateWithFlags(&hit->exec, graph, 0) == cudaSuccess;
    if (graph) cudaGraphDestroy(graph);
  }
  cudaGetLastError();   // a refused capture leaves no sticky error
  if (!ok) {
    hit->failed = true;
    hit->exec = nullptr;
    return compress_body(c, budget_bytes, hdr, blob_dev, blob_cap);
  }
  hit->launches = counted;
  CUDA_TRY(cudaGraphLaunch(hit->exec, c.st));
  launch_counter().fetch_add(hit->launches, std::memory_order_relaxed);
  return JOLT_OK;
}

jolt_status jolt_compress(const jolt_shape* shape, const void* k_dev, const void* v_dev, const jolt_options* opts,
                          uint64_t budget_bytes, uint64_t seed, void* blob_dev, size_t blob_cap, void* ws_dev,
                          size_t ws_bytes, void* stream) {
  Plan p;
  JTRY(make_plan(shape, opts, &p));
  JTRY(check_ws(p, ws_dev, ws_bytes));
  JTRY(check_inputs(p, k_dev, v_dev));
  if (!blob_dev) return fail(JOLT_ERR_INVALID_ARG, "null blob");
  if (reinterpret_cast<uintptr_t>(blob_dev) % 16) return fail(JOLT_ERR_INVALID_ARG, "blob not 16-byte aligned");
  if (blob_cap < budget_bytes && blob_cap < p.blob_max)
    return fail(JOLT_ERR_OUTPUT_TOO_SMALL, "blob capacity %zu below budget %llu", blob_cap,
                (unsigned long long)budget_bytes);
  const unsigned long long hdr = 64ull + 64ull * p.NU;
  if (budget_bytes < hdr) return fail(JOLT_ERR_BUDGET_INFEASIBLE, "budget below the headers (%llu bytes)", hdr);
  Ctx c{p, (unsigned char*)ws_dev, (cudaStream_t)stream, k_dev, v_dev, seed};
  cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
  CUDA_TRY(cudaStreamIsCapturing(c.st, &cs));
  if (!g_graphs.on || g_prof.on || cs != cudaStreamCaptureStatusNone)
    return compress_body(c, budget_bytes, hdr, blob_dev, blob_cap);
  GraphKey key;
  memset(&key, 0, sizeof key);
  key.sh = *shape;
  key.op = *opts;
  key.k = k_dev;
  key.v = v_dev;
  key.budget = budget_bytes;
  key.seed = seed;
  key.blob = blob_dev;
  key.cap = blob_cap;
  key.ws = ws_dev;
  key.ws_bytes = ws_bytes;
  CUDA_TRY(cudaGetDevice(&key.device));
  return compress_graph(c, key, budget_bytes, hdr, blob_dev, blob_cap);
}

void jolt_set_graphs(int32_t enable) {
  g_graphs.on = enable != 0;
  if (!g_graphs.on) {
    for (auto& g : g_graphs.e)
      if (g.exec) cudaGraphExecDestroy(g.exec);
    g_graphs.e.clear();
  }
}

jolt_status jolt_release(void) {
  jolt_status ret = JOLT_OK;
  for (auto& g : g_graphs.e)
    if (g.exec) cudaGraphExecDestroy(g.exec);
  g_graphs.e.clear();
  if (g_graphs.cap_stream && cudaStreamDestroy(g_graphs.cap_stream) != cudaSuccess) ret = JOLT_ERR_CUDA;
  g_graphs.cap_stream = nullptr;
  g_graphs.cap_device = -1;
  if (g_aux.st) {
    if (cudaStreamDestroy(g_aux.st) != cudaSuccess) ret = JOLT_ERR_CUDA;
    cudaEventDestroy(g_aux.fork);
    cudaEventDestroy(g_aux.join);
  }
  g_aux = Aux();
  for (auto& sv : g_solver) {
    if (sv.h) {
      cusolverDnDestroyParams(sv.params);
      cusolverDnDestroy(sv.h);
    }
    sv = Solver();
  }
  for (auto& r : g_prof.recs) {
    cudaEventDestroy(r.a);
    cudaEventDestroy(r.b);
  }
  for (auto e : g_prof.pool) cudaEventDestroy(e);
  g_prof.recs.clear();
  g_prof.pool.clear();
  g_prof.on = false;
  cudaGetLastError();
  if (ret != JOLT_OK) return fail(ret, "a stream of this thread could not be destroyed");
  return JOLT_OK;
}

jolt_status jolt_read_header(const void* blob_dev, jolt_shape* shape_out, uint64_t* total_bytes,
                             jolt_unit_record* records, int32_t cap, void* stream) {
  if (!blob_dev) return fail(JOLT_ERR_INVALID_ARG, "null blob");
  cudaStream_t st = (cudaStream_t)stream;
  BlobHeader h;
  CUDA_TRY(cudaMemcpyAsync(&h, blob_dev, sizeof h, cudaMemcpyDeviceToHost, st));
  CUDA_TRY(cudaStreamSynchronize(st));
  if (h.magic != kMagic || h.version != kVersion || h.n_units == 0 || h.n_units > 1u << 20)
    return fail(JOLT_ERR_BAD_BLOB, "bad blob header");
  if (shape_out) {
    shape_out->n_layers = h.n_layers;
    shape_out->n_heads = h.n_heads;
    shape_out->n_tokens = h.n_tokens;
    shape_out->head_dim = h.head_dim;
    shape_out->layers_per_group = h.layers_per_group;
    shape_out->dtype = h.dtype;
  }
  if (total_bytes) *total_bytes = h.total_bytes;
  if (records && cap > 0) {
    int n = (int)h.n_units < cap ? (int)h.n_units : cap;
    CUDA_TRY(cudaMemcpyAsync(records, (const char*)blob_dev + sizeof(BlobHeader), n * sizeof(UnitHeader),
                             cudaMemcpyDeviceToHost, st));
    CUDA_TRY(cudaStreamSynchronize(st));
  }
  if (h.status & DEV_ERR_TIMEOUT) return fail(JOLT_ERR_TIMEOUT, "a bounded device-side wait gave up");
  if (h.status & DEV_ERR_INFEASIBLE) return fail(JOLT_ERR_BUDGET_INFEASIBLE, "budget infeasible (device)");
  if (h.status & (DEV_ERR_NONFINITE | DEV_ERR_FACTOR))
    return fail(JOLT_ERR_NUMERIC, "non-finite input or factorisation breakdown (status %u)", h.status);
  if (h.status & DEV_ERR_CAPACITY) return fail(JOLT_ERR_OUTPUT_TOO_SMALL, "blob capacity below payload");
  if (h.status) return fail(JOLT_ERR_BAD_BLOB, "blob status %u", h.status);
  return JOLT_OK;
}

}  // extern "C"

namespace {
// The decoder's preparation of a blob (shared by jolt_decompress and the decode-side
// attention): read and validate the headers (synchronises once), plan a workspace for the
// stored ranks, copy every unit's U, W and core to aligned buffers, and form its rotated
// operator P' from the stored core and feature factor.
struct Prepared {
  BlobHeader h;
  jolt_shape sh;
  std::vector<jolt_unit_record> rec;
  Plan p;
};

jolt_status decode_prepare(const void* blob_dev, void* ws_dev, size_t ws_bytes, cudaStream_t st, Prepared* out,
                           bool compute) {
  Prepared& pr = *out;
  uint64_t total = 0;
  CUDA_TRY(cudaMemcpyAsync(&pr.h, blob_dev, sizeof pr.h, cudaMemcpyDeviceToHost, st));
  CUDA_TRY(cudaStreamSynchronize(st));
  const BlobHeader& h = pr.h;
  if (h.magic != kMagic || h.version != kVersion || h.n_units == 0 || h.n_units > 4096)
    return fail(JOLT_ERR_BAD_BLOB, "bad blob header");
  pr.rec.resize(h.n_units);
  JTRY(jolt_read_header(blob_dev, &pr.sh, &total, pr.rec.data(), (int32_t)h.n_units, st));
  // a plan for this shape with candidate sets made of the ranks actually stored
  jolt_options op;
  memset(&op, 0, sizeof op);
  int rTm = 8, rDm = 8;
  for (auto& r : pr.rec) {
    if (r.r_T < 1 || r.r_T > pr.sh.n_tokens || r.r_D < 1 || r.r_D > pr.sh.head_dim || r.bits < 0 || r.bits > 8)
      return fail(JOLT_ERR_BAD_BLOB, "unit record out of range");
    if (r.off_U + 2ull * pr.sh.n_tokens * r.r_T > total) return fail(JOLT_ERR_BAD_BLOB, "unit record offsets");
    rTm = r.r_T > rTm ? r.r_T : rTm;
    rDm = r.r_D > rDm ? r.r_D : rDm;
  }
  op.n_token_ranks = 1;
  op.token_ranks[0] = (int)round_up(rTm, 8) > pr.sh.n_tokens ? rTm : (int)round_up(rTm, 8);
  op.n_feature_ranks = 1;
  op.feature_ranks[0] = (int)round_up(rDm, 8) > pr.sh.head_dim ? rDm : (int)round_up(rDm, 8);
  op.n_bits = 1;
  op.method = JOLT_EXACT;
  op.unit_offset = h.unit_offset;
  JTRY(make_plan(&pr.sh, &op, &pr.p));
  const Plan& p = pr.p;
  if (ws_bytes < p.dws_total)
    return fail(JOLT_ERR_WORKSPACE_TOO_SMALL, "decompress workspace %zu bytes, need %zu", ws_bytes, p.dws_total);
  if (!compute) return JOLT_OK;
  Ctx c{p, (unsigned char*)ws_dev, st, nullptr, nullptr, h.seed};
  bf16* Ucp = c.at<bf16>(p.d_U);
  bf16* Wcp = c.at<bf16>(p.d_W);
  bf16* Ccp = c.at<bf16>(p.d_C);
  bf16* P = c.at<bf16>(p.d_P);
  int* umap = c.at<int>(p.d_umap);
  JTRY(fill_umap(c, umap, p.NU));
  const unsigned char* blob = (const unsigned char*)blob_dev;
  const long long sP_unit = (long long)p.S * p.rTmax * p.D;
  for (int u = 0; u < p.NU; ++u) {
    const jolt_unit_record& r = pr.rec[u];
    bf16* Uu = Ucp + (size_t)u * p.T * p.ldU;
    bf16* Wu = Wcp + (size_t)u * p.D * p.ldW;
    bf16* Cu = Ccp + (size_t)u * p.S * p.rTmax * p.ldC;
    count_launch(), copy2d_kernel<<<grid1d((long long)p.T * p.ldU), 256, 0, st>>>((const bf16*)(blob + r.off_U), p.T,
                                                                                r.r_T, Uu, p.ldU);
    count_launch(), copy2d_kernel<<<grid1d((long long)p.D * p.ldW), 256, 0, st>>>((const bf16*)(blob + r.off_W), p.D,
                                                                                r.r_D, Wu, p.ldW);
    count_launch(), copy2d_kernel<<<grid1d((long long)p.S * r.r_T * p.ldC), 256, 0, st>>>(
        (const bf16*)(blob + r.off_C), (long long)p.S * r.r_T, r.r_D, Cu, p.ldC);
    CUDA_TRY(cudaGetLastError());
    JTRY(pmat_unit(c, u, Cu, p.ldC, r.r_T, p.rTmax, Wu, p.ldW, r.r_D, nullptr, P + u * sP_unit, umap));
  }
  return JOLT_OK;
}
}  // namespace

extern "C" {

jolt_status jolt_decompress(const void* blob_dev, int32_t out_dtype, void* k_out_dev, void* v_out_dev, void* ws_dev,
                            size_t ws_bytes, void* stream) {
  if (out_dtype != JOLT_BF16 && out_dtype != JOLT_F32) return fail(JOLT_ERR_INVALID_ARG, "out_dtype %d", out_dtype);
  if (!k_out_dev || !v_out_dev || !ws_dev) return fail(JOLT_ERR_INVALID_ARG, "null pointer");
  cudaStream_t st = (cudaStream_t)stream;
  Prepared pr;
  JTRY(decode_prepare(blob_dev, ws_dev, ws_bytes, st, &pr, true));
  const Plan& p = pr.p;
  const BlobHeader& h = pr.h;
  Ctx c{p, (unsigned char*)ws_dev, st, nullptr, nullptr, h.seed};
  bf16* Ucp = c.at<bf16>(p.d_U);
  bf16* P = c.at<bf16>(p.d_P);
  const unsigned char* blob = (const unsigned char*)blob_dev;
  const long long sP_unit = (long long)p.S * p.rTmax * p.D;
  DecodeArgs a;
  a.blob = blob;
  a.U = Ucp;
  a.ldU = p.ldU;
  a.sU = (long long)p.T * p.ldU;
  a.P = P;
  a.sP_unit = sP_unit;
  a.rTmax = p.rTmax;
  a.T = p.T;
  a.S = p.S;
  a.Lg = p.Lg;
  a.u0 = p.u0;
  a.seed = h.seed;
  a.k_out = k_out_dev;
  a.v_out = v_out_dev;
  a.out_f32 = out_dtype == JOLT_F32;
  dim3 grid(p.tiles, p.S, p.NU);
  ProfScope ps("decode_kernel", st, p.NU);
  switch (p.D) {
#define DEC_CASE(DD)                                                                                     \
  case DD: {                                                                                             \
    CUDA_TRY(cudaFuncSetAttribute(decode_kernel<DD>, cudaFuncAttributeMaxDynamicSharedMemorySize,        \
                                  (int)decode_smem<DD>()));                                              \
    count_launch(), decode_kernel<DD><<<grid, TTHREADS, decode_smem<DD>(), st>>>(a);                                     \
    break;                                                                                               \
  }
    DEC_CASE(16)
    DEC_CASE(32)
    DEC_CASE(64)
    DEC_CASE(128)
#undef DEC_CASE
    default: return fail(JOLT_ERR_BAD_BLOB, "head_dim");
  }
  CUDA_TRY(cudaGetLastError());
  return JOLT_OK;
}

}  // extern "C"

namespace {
// token chunks per KV head for the decode-side attention: about two CTAs per SM in all,
// at least 64 tokens per chunk, at most 64 chunks
int attend_chunks(int T, int H) {
  long long n = ceil_div(2 * 148, H);
  n = n < 1 ? 1 : (n > 64 ? 64 : n);
  const long long byT = ceil_div(T, att::TT);
  return (int)(n < byT ? n : byT);
}
size_t attend_scratch(int T, int H, int D, int rTmax, int nq) {
  const int G = nq / H;
  return sizeof(float) * ((size_t)nq * D + (size_t)nq * rTmax +
                          (size_t)H * attend_chunks(T, H) * G * (2 + (size_t)rTmax + D)) + 256;
}

template <int D>
jolt_status launch_attend(const AttendArgs& a, cudaStream_t st) {
  count_launch(), attend_query_kernel<D><<<a.nq, att::THREADS, 0, st>>>(a);
  CUDA_TRY(cudaGetLastError());
  const size_t sm = attend_chunk_smem(D, a.rTmax, a.G);
  CUDA_TRY(cudaFuncSetAttribute(attend_chunk_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sm));
  count_launch(), attend_chunk_kernel<D><<<dim3(a.nch, a.H), att::THREADS, sm, st>>>(a);
  CUDA_TRY(cudaGetLastError());
  count_launch(), attend_combine_kernel<D><<<a.nq, att::THREADS, 0, st>>>(a);
  CUDA_TRY(cudaGetLastError());
  return JOLT_OK;
}

jolt_status attend_with(const void* blob_dev, const void* ws_dev, size_t ws_bytes, int32_t layer, const float* q_dev,
                        int32_t n_q_heads, float* out_dev, float* lse_dev, void* scratch_dev, size_t scratch_bytes,
                        void* stream) {
  if (!blob_dev || !ws_dev || !q_dev || !out_dev || !scratch_dev) return fail(JOLT_ERR_INVALID_ARG, "null pointer");
  cudaStream_t st = (cudaStream_t)stream;
  Prepared pr;
  JTRY(decode_prepare(blob_dev, const_cast<void*>(ws_dev), ws_bytes, st, &pr, false));
  const Plan& p = pr.p;
  if (layer < 0 || layer >= p.nL) return fail(JOLT_ERR_INVALID_ARG, "layer %d not in [0, %d)", layer, p.nL);
  if (n_q_heads < p.H || n_q_heads % p.H || n_q_heads / p.H > att::MAXG)
    return fail(JOLT_ERR_INVALID_ARG, "n_q_heads %d: a multiple of the %d KV heads, at most %d per KV head",
                n_q_heads, p.H, att::MAXG);
  if (p.rTmax > att::MAXR) return fail(JOLT_ERR_UNSUPPORTED_SHAPE, "stored token rank above %d", att::MAXR);
  if (p.D < 16) return fail(JOLT_ERR_UNSUPPORTED_SHAPE, "head_dim");
  const size_t need = attend_scratch(p.T, p.H, p.D, p.rTmax, n_q_heads);
  if (scratch_bytes < need) return fail(JOLT_ERR_WORKSPACE_TOO_SMALL, "attend scratch %zu bytes, need %zu",
                                        scratch_bytes, need);
  Ctx c{p, (unsigned char*)const_cast<void*>(ws_dev), st, nullptr, nullptr, pr.h.seed};
  AttendArgs a;
  a.blob = (const unsigned char*)blob_dev;
  a.U = c.at<bf16>(p.d_U);
  a.ldU = p.ldU;
  a.sU = (long long)p.T * p.ldU;
  a.P = c.at<bf16>(p.d_P);
  a.sP_unit = (long long)p.S * p.rTmax * p.D;
  a.rTmax = p.rTmax;
  a.T = p.T;
  a.S = p.S;
  a.H = p.H;
  a.D = p.D;
  a.Lg = p.Lg;
  a.u0 = p.u0;
  a.seed = pr.h.seed;
  a.layer = layer;
  a.nq = n_q_heads;
  a.G = n_q_heads / p.H;
  a.q = q_dev;
  float* sc = (float*)(((uintptr_t)scratch_dev + 255) & ~(uintptr_t)255);
  a.qrot = sc;
  a.a = a.qrot + (size_t)n_q_heads * p.D;
  a.part = a.a + (size_t)n_q_heads * p.rTmax;
  a.nch = attend_chunks(p.T, p.H);
  a.out = out_dev;
  a.lse = lse_dev;
  ProfScope ps("attend", st, 1);
  switch (p.D) {
    case 16: return launch_attend<16>(a, st);
    case 32: return launch_attend<32>(a, st);
    case 64: return launch_attend<64>(a, st);
    default: return launch_attend<128>(a, st);
  }
}
}  // namespace

extern "C" {

jolt_status jolt_attend_prepare(const void* blob_dev, void* ws_dev, size_t ws_bytes, void* stream) {
  if (!blob_dev || !ws_dev) return fail(JOLT_ERR_INVALID_ARG, "null pointer");
  Prepared pr;
  return decode_prepare(blob_dev, ws_dev, ws_bytes, (cudaStream_t)stream, &pr, true);
}

jolt_status jolt_attend_scratch_size(const jolt_shape* shape, int32_t max_token_rank, int32_t n_q_heads,
                                     size_t* bytes) {
  if (!shape || !bytes || n_q_heads < 1 || max_token_rank < 1) return fail(JOLT_ERR_INVALID_ARG, "attend sizes");
  if (shape->n_heads < 1 || n_q_heads % shape->n_heads) return fail(JOLT_ERR_INVALID_ARG, "n_q_heads % n_heads");
  const int rT = (int)round_up(max_token_rank, 8);
  *bytes = attend_scratch(shape->n_tokens, shape->n_heads, shape->head_dim, rT, n_q_heads);
  return JOLT_OK;
}

jolt_status jolt_attend(const void* blob_dev, const void* ws_dev, size_t ws_bytes, int32_t layer, const float* q_dev,
                        int32_t n_q_heads, float* out_dev, void* scratch_dev, size_t scratch_bytes, void* stream) {
  return attend_with(blob_dev, ws_dev, ws_bytes, layer, q_dev, n_q_heads, out_dev, nullptr, scratch_dev, scratch_bytes,
                     stream);
}

jolt_status jolt_attend_state(const void* blob_dev, const void* ws_dev, size_t ws_bytes, int32_t layer,
                              const float* q_dev, int32_t n_q_heads, float* out_dev, float* lse_dev,
                              void* scratch_dev, size_t scratch_bytes, void* stream) {
  if (!lse_dev) return fail(JOLT_ERR_INVALID_ARG, "null pointer");
  return attend_with(blob_dev, ws_dev, ws_bytes, layer, q_dev, n_q_heads, out_dev, lse_dev, scratch_dev, scratch_bytes,
                     stream);
}

jolt_status jolt_quant_baseline(const jolt_shape* shape, const void* k_dev, const void* v_dev, int32_t bits,
                                void* codes_dev, void* scales_dev, double* sq_dev, void* ws_dev, size_t ws_bytes,
                                void* stream) {
  if (!shape || !k_dev || !v_dev || !sq_dev || !ws_dev) return fail(JOLT_ERR_INVALID_ARG, "null pointer");
  if (bits < 1 || bits > 8) return fail(JOLT_ERR_INVALID_ARG, "bits %d not in [1, 8]", bits);
  if ((codes_dev == nullptr) != (scales_dev == nullptr)) return fail(JOLT_ERR_INVALID_ARG, "give both or neither output");
  if (shape->dtype != JOLT_BF16 && shape->dtype != JOLT_F32) return fail(JOLT_ERR_INVALID_ARG, "dtype");
  if (shape->n_layers < 1 || shape->layers_per_group < 1 || shape->n_layers % shape->layers_per_group ||
      shape->head_dim % 16 || shape->n_heads < 1 || shape->n_tokens < 1)
    return fail(JOLT_ERR_UNSUPPORTED_SHAPE, "shape");
  const int G = shape->n_layers / shape->layers_per_group, NU = 2 * G, nblk = 148;
  if (ws_bytes < (size_t)NU * nblk * 16) return fail(JOLT_ERR_WORKSPACE_TOO_SMALL, "baseline workspace");
  if (((uintptr_t)codes_dev % 16) || ((uintptr_t)scales_dev % 4)) return fail(JOLT_ERR_INVALID_ARG, "alignment");
  CacheView cv;
  cv.k = k_dev;
  cv.v = v_dev;
  cv.dtype = shape->dtype;
  cv.n_layers = shape->n_layers;
  cv.H = shape->n_heads;
  cv.T = shape->n_tokens;
  cv.D = shape->head_dim;
  cv.Lg = shape->layers_per_group;
  cv.S = cv.Lg * cv.H;
  cv.u0 = 0;
  cv.unit_elems = (long long)cv.S * cv.T * cv.D;
  cudaStream_t st = (cudaStream_t)stream;
  double* part = (double*)ws_dev;
  ProfScope ps("quant_baseline", st, NU);
  if (shape->dtype == JOLT_BF16)
    count_launch(), quant_baseline_kernel<bf16><<<dim3(nblk, NU), 256, 0, st>>>(
        cv, bits, (unsigned char*)codes_dev, (__half2*)scales_dev, part, nblk);
  else
    count_launch(), quant_baseline_kernel<float><<<dim3(nblk, NU), 256, 0, st>>>(
        cv, bits, (unsigned char*)codes_dev, (__half2*)scales_dev, part, nblk);
  CUDA_TRY(cudaGetLastError());
  count_launch(), frob_final_kernel<<<(unsigned)ceil_div(2 * NU, 128), 128, 0, st>>>(part, NU, nblk, sq_dev);
  CUDA_TRY(cudaGetLastError());
  return JOLT_OK;
}

jolt_status jolt_frobenius(const jolt_shape* shape, const void* k_dev, const void* v_dev, const void* ky_dev,
                           const void* vy_dev, int32_t ydtype, double* sq_dev, void* ws_dev, size_t ws_bytes,
                           void* stream) {
  if (!shape || !k_dev || !v_dev || !sq_dev || !ws_dev) return fail(JOLT_ERR_INVALID_ARG, "null pointer");
  if ((ky_dev == nullptr) != (vy_dev == nullptr)) return fail(JOLT_ERR_INVALID_ARG, "give both or neither of ky, vy");
  if (shape->n_layers < 1 || shape->layers_per_group < 1 || shape->n_layers % shape->layers_per_group)
    return fail(JOLT_ERR_INVALID_ARG, "shape");
  const int G = shape->n_layers / shape->layers_per_group, NU = 2 * G, nblk = 64;
  if (ws_bytes < (size_t)NU * nblk * 16) return fail(JOLT_ERR_WORKSPACE_TOO_SMALL, "frobenius workspace");
  const long long n = (long long)shape->layers_per_group * shape->n_heads * shape->n_tokens * shape->head_dim;
  cudaStream_t st = (cudaStream_t)stream;
  double* part = (double*)ws_dev;
  for (int kv = 0; kv < 2; ++kv) {
    const void* X = kv ? v_dev : k_dev;
    const void* Y = kv ? vy_dev : ky_dev;
    dim3 grid(nblk, G);
    if (shape->dtype == JOLT_BF16) {
      if (ydtype == JOLT_F32)
        count_launch(), frob_partial_kernel<bf16, float><<<grid, 256, 0, st>>>((const bf16*)X, (const float*)Y, n, kv, part, nblk);
      else
        count_launch(), frob_partial_kernel<bf16, bf16><<<grid, 256, 0, st>>>((const bf16*)X, (const bf16*)Y, n, kv, part, nblk);
    } else {
      if (ydtype == JOLT_F32)
        count_launch(), frob_partial_kernel<float, float><<<grid, 256, 0, st>>>((const float*)X, (const float*)Y, n, kv, part, nblk);
      else
        count_launch(), frob_partial_kernel<float, bf16><<<grid, 256, 0, st>>>((const float*)X, (const bf16*)Y, n, kv, part, nblk);
    }
    CUDA_TRY(cudaGetLastError());
  }
  count_launch(), frob_final_kernel<<<(unsigned)ceil_div(2 * NU, 128), 128, 0, st>>>(part, NU, nblk, sq_dev);
  CUDA_TRY(cudaGetLastError());
  return JOLT_OK;
}

// ------------------------------------------------------------------------------------------
// Allocation-free variant of jolt_frobenius.  Its per-block partial sums live in a file-scope
// device array instead of a caller-provided workspace, for callers that cannot allocate
// device memory themselves: for instance a host program whose device memory is entirely
// owned by another allocator, or one that must not call the CUDA allocator at all on its
// path.  The array is part of this library's image: every device that loads the library
// holds it until the process exits.
// ------------------------------------------------------------------------------------------
}  // extern "C"

namespace {
constexpr int kNoAllocBlocks = 64;                       // partial-sum blocks per unit
constexpr int kNoAllocMaxUnits = 64;                     // 2 * n_layers / layers_per_group
constexpr int kNoAllocSlots = kNoAllocMaxUnits * kNoAllocBlocks * 2;
static __device__ __align__(256) double g_frob_scratch[kNoAllocSlots];  // 64 KiB

// device address of g_frob_scratch, looked up once per device with that device current
struct NoAllocScratch {
  std::mutex mu;
  double* ptr[64] = {};
};
NoAllocScratch& noalloc_scratch() {
  static NoAllocScratch s;
  return s;
}
}  // namespace

extern "C" jolt_status jolt_frobenius_noalloc(const jolt_shape* shape, const void* k_dev, const void* v_dev,
                                              const void* ky_dev, const void* vy_dev, int32_t ydtype,
                                              double* sq_dev, void* stream) {
  if (!shape || !k_dev || !v_dev || !sq_dev) return fail(JOLT_ERR_INVALID_ARG, "null pointer");
  if ((ky_dev == nullptr) != (vy_dev == nullptr)) return fail(JOLT_ERR_INVALID_ARG, "give both or neither of ky, vy");
  if (shape->n_layers < 1 || shape->layers_per_group < 1 || shape->n_layers % shape->layers_per_group)
    return fail(JOLT_ERR_INVALID_ARG, "shape");
  const int G = shape->n_layers / shape->layers_per_group, NU = 2 * G;
  if (NU > kNoAllocMaxUnits)
    return fail(JOLT_ERR_WORKSPACE_TOO_SMALL, "jolt_frobenius_noalloc handles at most %d units (got %d); use jolt_frobenius",
                kNoAllocMaxUnits, NU);
  int dev = 0;
  CUDA_TRY(cudaGetDevice(&dev));
  if (dev < 0 || dev >= 64) return fail(JOLT_ERR_INVALID_ARG, "device ordinal %d out of range", dev);
  double* part = nullptr;
  {
    NoAllocScratch& sc = noalloc_scratch();
    std::lock_guard<std::mutex> lk(sc.mu);
    if (!sc.ptr[dev]) {
      void* p = nullptr;
      CUDA_TRY(cudaGetSymbolAddress(&p, g_frob_scratch));
      sc.ptr[dev] = static_cast<double*>(p);
    }
    part = sc.ptr[dev];
  }
  const long long n = (long long)shape->layers_per_group * shape->n_heads * shape->n_tokens * shape->head_dim;
  cudaStream_t st = (cudaStream_t)stream;
  // every partial slot read below is written first by the same call: nothing to clear
  for (int kv = 0; kv < 2; ++kv) {
    const void* X = kv ? v_dev : k_dev;
    const void* Y = kv ? vy_dev : ky_dev;
    dim3 grid(kNoAllocBlocks, G);
    if (shape->dtype == JOLT_BF16) {
      if (ydtype == JOLT_F32)
        count_launch(), frob_partial_kernel<bf16, float><<<grid, 256, 0, st>>>((const bf16*)X, (const float*)Y, n, kv,
                                                                               part, kNoAllocBlocks);
      else
        count_launch(), frob_partial_kernel<bf16, bf16><<<grid, 256, 0, st>>>((const bf16*)X, (const bf16*)Y, n, kv,
                                                                              part, kNoAllocBlocks);
    } else {
      if (ydtype == JOLT_F32)
        count_launch(), frob_partial_kernel<float, float><<<grid, 256, 0, st>>>((const float*)X, (const float*)Y, n,
                                                                                kv, part, kNoAllocBlocks);
      else
        count_launch(), frob_partial_kernel<float, bf16><<<grid, 256, 0, st>>>((const float*)X, (const bf16*)Y, n, kv,
                                                                               part, kNoAllocBlocks);
    }
    CUDA_TRY(cudaGetLastError());
  }
  count_launch(), frob_final_kernel<<<(unsigned)ceil_div(2 * NU, 128), 128, 0, st>>>(part, NU, kNoAllocBlocks, sq_dev);
  CUDA_TRY(cudaGetLastError());
  return JOLT_OK;
}
