/*
 * Host-side argument checks of the bf16 product, its gradients, the combine's
 * gradient and the low-rank adapters, for a build of the library's host code
 * with AddressSanitizer and UndefinedBehaviorSanitizer (run on the CPU by
 * tests/test_operators_sanitizers_more.py).  Every call here is rejected, or
 * is a no-op, before any HIP call.  It exits 0 when every status matches; a
 * sanitizer finding aborts it.
 */
#include <stdio.h>
#include <string.h>

#include "moesq.h"

static int failures = 0;

static void expect(const char *what, moesq_status_t got, moesq_status_t want) {
  const char *detail = moesq_last_error();
  if (got != want) {
    printf("FAIL %s: status %d, expected %d (%s)\n", what, (int)got, (int)want, detail);
    ++failures;
  } else if (want != MOESQ_OK && (!detail || !detail[0])) {
    printf("FAIL %s: error without a detail string\n", what);
    ++failures;
  }
}

#define P(x) ((void *)(uintptr_t)(x))

int main(void) {
  int32_t *ip = (int32_t *)P(0x10);
  uint16_t *x = (uint16_t *)P(0x10), *w = (uint16_t *)P(0x20), *y = (uint16_t *)P(0x30), *z = (uint16_t *)P(0x40);
  uint16_t *odd = (uint16_t *)P(0x18);
  float *fp = (float *)P(0x50);
  const int32_t low = INT32_MIN, top = INT32_MAX, most = MOESQ_GEMM_MAX_DIM;

  /* the product */
#define GEMM(what, want, x, perm, T, k, off, M, w, E, N, K, epi, y, z) \
  expect("gemm " what, moesq_gemm(x, perm, T, k, off, M, w, E, N, K, epi, y, z, NULL), want)
  GEMM("M=0", MOESQ_OK, NULL, NULL, 0, 0, NULL, 0, NULL, 1, 64, 64, 0, NULL, NULL);
  GEMM("epilogue", MOESQ_ERR_ARG, x, NULL, 0, 0, NULL, 4, w, 1, 64, 64, top, y, NULL);
  GEMM("epilogue lowest", MOESQ_ERR_ARG, x, NULL, 0, 0, NULL, 4, w, 1, 64, 64, low, y, NULL);
  GEMM("flat without perm", MOESQ_ERR_ARG, x, NULL, 0, 0, ip, 4, w, 2, 64, 64, MOESQ_OUT_FLAT, y, NULL);
  GEMM("z without SwiGLU", MOESQ_ERR_ARG, x, NULL, 0, 0, NULL, 4, w, 1, 64, 64, MOESQ_EPI_NONE, y, z);
  GEMM("z with flat", MOESQ_ERR_ARG, x, ip, 4, 1, ip, 4, w, 2, 64, 64, MOESQ_EPI_SWIGLU | MOESQ_OUT_FLAT, y, z);
  GEMM("SwiGLU N % 16", MOESQ_ERR_SHAPE, x, NULL, 0, 0, NULL, 4, w, 1, 24, 64, MOESQ_EPI_SWIGLU, y, NULL);
  GEMM("gather T*k overflow", MOESQ_ERR_SHAPE, x, ip, top, top, ip, 1, w, 2, 64, 64, 0, y, NULL);
  GEMM("gather k=0", MOESQ_ERR_SHAPE, x, ip, 4, 0, ip, 0, w, 2, 64, 64, 0, y, NULL);
  GEMM("gather T<0", MOESQ_ERR_SHAPE, x, ip, low, 1, ip, 4, w, 2, 64, 64, 0, y, NULL);
  GEMM("gather M != T*k", MOESQ_ERR_SHAPE, x, ip, 4, 2, ip, 4, w, 2, 64, 64, 0, y, NULL);
  GEMM("gather without offsets", MOESQ_ERR_NULL, x, ip, 4, 1, NULL, 4, w, 1, 64, 64, 0, y, NULL);
  GEMM("gathered tokens past 4 GiB", MOESQ_ERR_SHAPE, x, ip, 1 << 20, 1, ip, 1 << 20, w, 2, 64, 2048, 0, y, NULL);
  GEMM("NULL x", MOESQ_ERR_NULL, NULL, NULL, 0, 0, NULL, 4, w, 1, 64, 64, 0, y, NULL);
  GEMM("NULL w", MOESQ_ERR_NULL, x, NULL, 0, 0, NULL, 4, NULL, 1, 64, 64, 0, y, NULL);
  GEMM("NULL y", MOESQ_ERR_NULL, x, NULL, 0, 0, NULL, 4, w, 1, 64, 64, 0, NULL, NULL);
  GEMM("x misaligned", MOESQ_ERR_ARG, odd, NULL, 0, 0, NULL, 4, w, 1, 64, 64, 0, y, NULL);
  GEMM("z misaligned", MOESQ_ERR_ARG, x, NULL, 0, 0, NULL, 4, w, 1, 64, 64, MOESQ_EPI_SWIGLU, y, odd);

  /* the sizes, alike in all three */
#define SIZES(what, want, off, M, E, N, K)                                                                     \
  do {                                                                                                         \
    GEMM(what, want, x, NULL, 0, 0, off, M, w, E, N, K, 0, y, NULL);                                           \
    expect("gemm_dx " what, moesq_gemm_dx(x, off, M, w, E, N, K, NULL, y, NULL), want);                        \
    expect("gemm_dw " what, moesq_gemm_dw(x, w, NULL, 0, 0, off, M, E, N, K, MOESQ_F32, 0, fp, NULL, 0, NULL), want); \
  } while (0)
  SIZES("E=0", MOESQ_ERR_SHAPE, ip, 4, 0, 64, 64);
  SIZES("E lowest", MOESQ_ERR_SHAPE, ip, 4, low, 64, 64);
  SIZES("E past its limit", MOESQ_ERR_SHAPE, ip, 4, MOESQ_MAX_EXPERTS + 1, 64, 64);
  SIZES("N=0", MOESQ_ERR_SHAPE, ip, 4, 2, 0, 64);
  SIZES("N % 8", MOESQ_ERR_SHAPE, ip, 4, 2, 60, 64);
  SIZES("N lowest", MOESQ_ERR_SHAPE, ip, 4, 2, low, 64);
  SIZES("N past its limit", MOESQ_ERR_SHAPE, ip, 4, 2, most + 8, 64);
  SIZES("K=0", MOESQ_ERR_SHAPE, ip, 4, 2, 64, 0);
  SIZES("K % 8", MOESQ_ERR_SHAPE, ip, 4, 2, 64, 4);
  SIZES("K lowest", MOESQ_ERR_SHAPE, ip, 4, 2, 64, low);
  SIZES("K past its limit", MOESQ_ERR_SHAPE, ip, 4, 2, 64, most + 8);
  SIZES("an expert past 4 GiB", MOESQ_ERR_SHAPE, ip, 4, 2, most, 2048);
  SIZES("an expert far past it", MOESQ_ERR_SHAPE, ip, 4, 2, most, most);
  SIZES("M<0", MOESQ_ERR_SHAPE, ip, low, 2, 64, 64);
  SIZES("M past its limit", MOESQ_ERR_SHAPE, ip, top, 2, 64, 64);
  SIZES("experts without offsets", MOESQ_ERR_NULL, NULL, 4, 2, 64, 64);

  /* its gradients */
  expect("gemm_dx M=0", moesq_gemm_dx(NULL, NULL, 0, NULL, 1, 64, 64, NULL, NULL, NULL), MOESQ_OK);
  expect("gemm_dx NULL dy", moesq_gemm_dx(NULL, NULL, 4, w, 1, 64, 64, NULL, y, NULL), MOESQ_ERR_NULL);
  expect("gemm_dx NULL w", moesq_gemm_dx(x, NULL, 4, NULL, 1, 64, 64, NULL, y, NULL), MOESQ_ERR_NULL);
  expect("gemm_dx NULL dx", moesq_gemm_dx(x, NULL, 4, w, 1, 64, 64, NULL, NULL, NULL), MOESQ_ERR_NULL);
  expect("gemm_dx z misaligned", moesq_gemm_dx(x, NULL, 4, w, 1, 64, 64, odd, y, NULL), MOESQ_ERR_ARG);
#define DW(what, want, dy, x, perm, T, k, off, M, E, dtype, acc, dw) \
  expect("gemm_dw " what, moesq_gemm_dw(dy, x, perm, T, k, off, M, E, 64, 64, dtype, acc, dw, NULL, 0, NULL), want)
  DW("dtype", MOESQ_ERR_ARG, x, w, NULL, 0, 0, NULL, 4, 1, top, 0, fp);
  DW("dtype lowest", MOESQ_ERR_ARG, x, w, NULL, 0, 0, NULL, 4, 1, low, 0, fp);
  DW("accumulate", MOESQ_ERR_ARG, x, w, NULL, 0, 0, NULL, 4, 1, MOESQ_F32, 2, fp);
  DW("accumulate in bf16", MOESQ_ERR_ARG, x, w, NULL, 0, 0, NULL, 4, 1, MOESQ_BF16, 1, fp);
  DW("gather M != T*k", MOESQ_ERR_SHAPE, x, w, ip, top, top, ip, 4, 2, MOESQ_F32, 0, fp);
  DW("gather k lowest", MOESQ_ERR_SHAPE, x, w, ip, 4, low, ip, 4, 2, MOESQ_F32, 0, fp);
  DW("gather without offsets", MOESQ_ERR_NULL, x, w, ip, 4, 1, NULL, 4, 1, MOESQ_F32, 0, fp);
  DW("NULL dw", MOESQ_ERR_NULL, x, w, NULL, 0, 0, NULL, 0, 1, MOESQ_F32, 0, NULL);
  DW("NULL dy", MOESQ_ERR_NULL, NULL, w, NULL, 0, 0, NULL, 4, 1, MOESQ_F32, 0, fp);
  DW("dw misaligned", MOESQ_ERR_ARG, x, w, NULL, 0, 0, NULL, 4, 1, MOESQ_F32, 0, odd);

  expect("gemm_dw workspace misaligned",
         moesq_gemm_dw(x, w, NULL, 0, 0, NULL, 8192, 1, 64, 64, MOESQ_F32, 0, fp, P(0x104), 1 << 30, NULL), MOESQ_ERR_ARG);
  expect("gemm_dw workspace too small",
         moesq_gemm_dw(x, w, NULL, 0, 0, NULL, 8192, 1, 64, 64, MOESQ_F32, 0, fp, P(0x100), 16, NULL), MOESQ_ERR_WORKSPACE);
  if (!moesq_gemm_dw_workspace_bytes(8192, 1, 64, 64) || moesq_gemm_dw_workspace_bytes(8192, 1, 64, 60) ||
      moesq_gemm_dw_workspace_bytes(low, 1, 64, 64) || moesq_gemm_dw_workspace_bytes(0, 1, 64, 64) ||
      moesq_gemm_dw_workspace_bytes(1 << 30, MOESQ_MAX_EXPERTS, 8, most))
    printf("FAIL gemm_dw workspace sizes\n"), ++failures;

  /* the combine's gradient */
#define COMBINE(what, want, d, y, inv, w, T, k, N, dy, dw) \
  expect("unpermute_backward " what, moesq_unpermute_backward(d, y, inv, w, T, k, N, dy, dw, NULL), want)
  COMBINE("T=0", MOESQ_OK, NULL, NULL, NULL, NULL, 0, 8, 64, NULL, NULL);
  COMBINE("T lowest", MOESQ_ERR_SHAPE, x, y, ip, fp, low, 8, 64, z, fp);
  COMBINE("k=0", MOESQ_ERR_SHAPE, x, y, ip, fp, 4, 0, 64, z, fp);
  COMBINE("T*k past its limit", MOESQ_ERR_SHAPE, x, y, ip, fp, top, top, 64, z, fp);
  COMBINE("N=0", MOESQ_ERR_SHAPE, x, y, ip, fp, 4, 2, 0, z, fp);
  COMBINE("N % 8", MOESQ_ERR_SHAPE, x, y, ip, fp, 4, 2, 12, z, fp);
  COMBINE("nothing wanted", MOESQ_ERR_NULL, x, y, ip, fp, 4, 2, 64, NULL, NULL);
  COMBINE("NULL dout", MOESQ_ERR_NULL, NULL, y, ip, fp, 4, 2, 64, z, fp);
  COMBINE("NULL inv_perm", MOESQ_ERR_NULL, x, y, NULL, fp, 4, 2, 64, z, fp);
  COMBINE("dy without weights", MOESQ_ERR_NULL, x, y, ip, NULL, 4, 2, 64, z, NULL);
  COMBINE("dw without y", MOESQ_ERR_NULL, x, NULL, ip, fp, 4, 2, 64, NULL, fp);
  COMBINE("dy misaligned", MOESQ_ERR_ARG, x, y, ip, fp, 4, 2, 64, odd, fp);
  COMBINE("dy is dout", MOESQ_ERR_ARG, x, y, ip, fp, 4, 2, 64, x, fp);

  /* adapters: each field at its limits and far outside them */
  const moesq_lora_t good = {w, y, fp, 4, 16, 1, 64, 64};
#define LORA(what, want, T, epi, change)                                                             \
  do {                                                                                               \
    moesq_lora_t l = good;                                                                           \
    change;                                                                                          \
    expect("lora " what, moesq_lora(x, ip, T, &l, NULL, epi, z, P(0x100), 0, NULL), want);           \
    if (want == MOESQ_ERR_SHAPE && (epi) == MOESQ_EPI_NONE && moesq_lora_workspace_bytes(T, &l)) {   \
      printf("FAIL lora " what ": a workspace for refused sizes\n");                                 \
      ++failures;                                                                                    \
    }                                                                                                \
  } while (0)
  LORA("T=0", MOESQ_OK, 0, 0, (void)l);
  LORA("T lowest", MOESQ_ERR_SHAPE, low, 0, (void)l);
  LORA("T past its limit", MOESQ_ERR_SHAPE, top, 0, (void)l);
  LORA("workspace", MOESQ_ERR_WORKSPACE, 4, 0, (void)l);
  LORA("epilogue", MOESQ_ERR_ARG, 4, top, (void)l);
  LORA("flat", MOESQ_ERR_ARG, 4, MOESQ_OUT_FLAT, (void)l);
  LORA("adapters=0", MOESQ_ERR_SHAPE, 4, 0, l.adapters = 0);
  LORA("adapters lowest", MOESQ_ERR_SHAPE, 4, 0, l.adapters = low);
  LORA("rank=0", MOESQ_ERR_SHAPE, 4, 0, l.rank = 0);
  LORA("rank % 8", MOESQ_ERR_SHAPE, 4, 0, l.rank = 12);
  LORA("rank past its limit", MOESQ_ERR_SHAPE, 4, 0, l.rank = MOESQ_LORA_MAX_RANK + 8);
  LORA("slices=0", MOESQ_ERR_SHAPE, 4, 0, l.slices = 0);
  LORA("slices top", MOESQ_ERR_SHAPE, 4, 0, l.slices = top);
  LORA("N % (8 * slices)", MOESQ_ERR_SHAPE, 4, 0, (l.slices = 3, l.N = 64));
  LORA("N lowest", MOESQ_ERR_SHAPE, 4, 0, l.N = low);
  LORA("N past its limit", MOESQ_ERR_SHAPE, 4, 0, l.N = most + 8);
  LORA("K=0", MOESQ_ERR_SHAPE, 4, 0, l.K = 0);
  LORA("K past its limit", MOESQ_ERR_SHAPE, 4, 0, l.K = most + 8);
  LORA("sums past their limit", MOESQ_ERR_SHAPE, 1 << 26, 0, (l.slices = 4, l.rank = 256));
  LORA("SwiGLU N % 16", MOESQ_ERR_SHAPE, 4, MOESQ_EPI_SWIGLU, l.N = 24);
  LORA("SwiGLU of three slices", MOESQ_ERR_SHAPE, 4, MOESQ_EPI_SWIGLU, (l.slices = 3, l.N = 96));
  LORA("NULL a", MOESQ_ERR_NULL, 4, 0, l.a = NULL);
  LORA("NULL b", MOESQ_ERR_NULL, 4, 0, l.b = NULL);
  LORA("NULL scale", MOESQ_ERR_NULL, 4, 0, l.scale = NULL);
  LORA("b misaligned", MOESQ_ERR_ARG, 4, 0, l.b = odd);
  expect("lora NULL descriptor", moesq_lora(x, ip, 4, NULL, NULL, 0, z, P(0x100), 1 << 20, NULL), MOESQ_ERR_NULL);
  expect("lora NULL x", moesq_lora(NULL, ip, 4, &good, NULL, 0, z, P(0x100), 1 << 20, NULL), MOESQ_ERR_NULL);
  expect("lora NULL ids", moesq_lora(x, NULL, 4, &good, NULL, 0, z, P(0x100), 1 << 20, NULL), MOESQ_ERR_NULL);
  expect("lora NULL y", moesq_lora(x, ip, 4, &good, NULL, 0, NULL, P(0x100), 1 << 20, NULL), MOESQ_ERR_NULL);
  expect("lora SwiGLU in place", moesq_lora(x, ip, 4, &good, z, MOESQ_EPI_SWIGLU, z, P(0x100), 1 << 20, NULL), MOESQ_ERR_ARG);
  expect("lora workspace misaligned", moesq_lora(x, ip, 4, &good, NULL, 0, z, P(0x104), 1 << 20, NULL), MOESQ_ERR_ARG);
  expect("lora NULL workspace", moesq_lora(x, ip, 4, &good, NULL, 0, z, NULL, 1 << 20, NULL), MOESQ_ERR_WORKSPACE);
  if (moesq_lora_workspace_bytes(4, NULL)) printf("FAIL workspace of no descriptor\n"), ++failures;

  printf("ok: %d failure(s)\n", failures);
  return failures != 0;
}
