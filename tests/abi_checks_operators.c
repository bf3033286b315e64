/*
 * Host-side argument checks of the router, the RMS norm and the entry points
 * on microscaled rows, for a build of the library's host code with
 * AddressSanitizer and UndefinedBehaviorSanitizer (run on the CPU by
 * tests/test_operators_sanitizers.py).  Every call here is rejected, or is a
 * no-op, before any HIP call.  It exits 0 when every status matches; a
 * sanitizer finding aborts it.
 */
#include <math.h>
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
  uint16_t *hp = (uint16_t *)P(0x10);
  uint8_t *bp = (uint8_t *)P(0x10);
  float *fp = (float *)P(0x10);
  const int32_t low = INT32_MIN, top = INT32_MAX;

  /* the router: each field at its limits and far outside them */
  const moesq_gate_t good = {2, MOESQ_SCORE_SOFTMAX, 1, 1, MOESQ_GROUP_MAX, 1, 1.0f};
#define GATE(what, want, T, E, change)                                                          \
  do {                                                                                          \
    moesq_gate_t g = good;                                                                      \
    change;                                                                                     \
    expect("gate " what, moesq_gate_topk(fp, MOESQ_F32, T, E, fp, &g, ip, ip, fp, NULL), want); \
  } while (0)
  expect("gate NULL descriptor", moesq_gate_topk(fp, 0, 4, 8, NULL, NULL, NULL, ip, fp, NULL), MOESQ_ERR_NULL);
  expect("gate NULL logits", moesq_gate_topk(NULL, 0, 4, 8, NULL, &good, NULL, ip, fp, NULL), MOESQ_ERR_NULL);
  expect("gate NULL ids", moesq_gate_topk(fp, 0, 4, 8, NULL, &good, NULL, NULL, fp, NULL), MOESQ_ERR_NULL);
  expect("gate NULL weights", moesq_gate_topk(fp, 0, 4, 8, NULL, &good, NULL, ip, NULL, NULL), MOESQ_ERR_NULL);
  expect("gate dtype", moesq_gate_topk(fp, top, 4, 8, NULL, &good, NULL, ip, fp, NULL), MOESQ_ERR_ARG);
  expect("gate logits misaligned", moesq_gate_topk(P(0x12), 0, 4, 8, NULL, &good, NULL, ip, fp, NULL),
         MOESQ_ERR_ARG);
  expect("gate T=0", moesq_gate_topk(NULL, 0, 0, 8, NULL, &good, NULL, NULL, NULL, NULL), MOESQ_OK);
  GATE("E=0", MOESQ_ERR_SHAPE, 4, 0, (void)g);
  GATE("E lowest", MOESQ_ERR_SHAPE, 4, low, (void)g);
  GATE("E past its limit", MOESQ_ERR_SHAPE, 4, MOESQ_MAX_EXPERTS + 1, (void)g);
  GATE("T<0", MOESQ_ERR_SHAPE, low, 8, (void)g);
  GATE("T*k overflow", MOESQ_ERR_SHAPE, top, 8, (void)g);
  GATE("k=0", MOESQ_ERR_SHAPE, 4, 8, g.k = 0);
  GATE("k lowest", MOESQ_ERR_SHAPE, 4, 8, g.k = low);
  GATE("k>E", MOESQ_ERR_SHAPE, 4, 8, g.k = 9);
  GATE("k past its limit", MOESQ_ERR_SHAPE, 4, 512, g.k = MOESQ_GATE_MAX_TOPK + 1);
  GATE("n_group=0", MOESQ_ERR_SHAPE, 4, 8, g.n_group = 0);
  GATE("n_group=-1", MOESQ_ERR_SHAPE, 4, 8, g.n_group = -1);
  GATE("n_group lowest", MOESQ_ERR_SHAPE, 4, 8, g.n_group = low);
  GATE("n_group past its limit", MOESQ_ERR_SHAPE, 4, 130, g.n_group = 65);
  GATE("n_group does not divide E", MOESQ_ERR_SHAPE, 4, 8, g.n_group = 3);
  GATE("topk_group=0", MOESQ_ERR_SHAPE, 4, 8, (g.n_group = 4, g.topk_group = 0));
  GATE("topk_group top", MOESQ_ERR_SHAPE, 4, 8, (g.n_group = 4, g.topk_group = top));
  GATE("k past the kept groups", MOESQ_ERR_SHAPE, 4, 8, (g.n_group = 4, g.k = 3));
  GATE("score", MOESQ_ERR_ARG, 4, 8, g.score = top);
  GATE("group_score", MOESQ_ERR_ARG, 4, 8, (g.n_group = 2, g.group_score = low));
  GATE("renormalize", MOESQ_ERR_ARG, 4, 8, g.renormalize = -1);
  GATE("scale NaN", MOESQ_ERR_ARG, 4, 8, g.scale = NAN);
  GATE("scale infinite", MOESQ_ERR_ARG, 4, 8, g.scale = -INFINITY);

  /* the norm */
#define NORM(what, want, x, res, w, T, K, eps, ro, y, rows, c, s, g) \
  expect("rmsnorm " what, moesq_rmsnorm(x, res, w, T, K, eps, ro, y, rows, c, s, g, NULL), want)
  uint16_t *h2 = (uint16_t *)P(0x20), *h3 = (uint16_t *)P(0x30), *h4 = (uint16_t *)P(0x40);
  NORM("T<0", MOESQ_ERR_SHAPE, hp, NULL, hp, low, 64, 0.0, NULL, h2, 0, NULL, NULL, NULL);
  NORM("K=0", MOESQ_ERR_SHAPE, hp, NULL, hp, 4, 0, 0.0, NULL, h2, 0, NULL, NULL, NULL);
  NORM("K lowest", MOESQ_ERR_SHAPE, hp, NULL, hp, 4, low, 0.0, NULL, h2, 0, NULL, NULL, NULL);
  NORM("K%8", MOESQ_ERR_SHAPE, hp, NULL, hp, 4, top, 0.0, NULL, h2, 0, NULL, NULL, NULL);
  NORM("K%32 with rows", MOESQ_ERR_SHAPE, hp, NULL, hp, 4, 40, 0.0, NULL, h2, 2, bp, bp, NULL);
  NORM("rows_format", MOESQ_ERR_ARG, hp, NULL, hp, 4, 64, 0.0, NULL, h2, 4, bp, bp, fp);
  NORM("rows_format lowest", MOESQ_ERR_ARG, hp, NULL, hp, 4, 64, 0.0, NULL, h2, low, bp, bp, fp);
  NORM("eps NaN", MOESQ_ERR_ARG, hp, NULL, hp, 4, 64, NAN, NULL, h2, 0, NULL, NULL, NULL);
  NORM("eps infinite", MOESQ_ERR_ARG, hp, NULL, hp, 4, 64, INFINITY, NULL, h2, 0, NULL, NULL, NULL);
  NORM("eps<0", MOESQ_ERR_ARG, hp, NULL, hp, 4, 64, -1.0, NULL, h2, 0, NULL, NULL, NULL);
  NORM("x NULL", MOESQ_ERR_NULL, NULL, NULL, hp, 4, 64, 0.0, NULL, h2, 0, NULL, NULL, NULL);
  NORM("weight NULL", MOESQ_ERR_NULL, hp, NULL, NULL, 4, 64, 0.0, NULL, h2, 0, NULL, NULL, NULL);
  NORM("residual alone", MOESQ_ERR_NULL, hp, h2, hp, 4, 64, 0.0, NULL, h3, 0, NULL, NULL, NULL);
  NORM("residual_out alone", MOESQ_ERR_NULL, hp, NULL, hp, 4, 64, 0.0, h2, h3, 0, NULL, NULL, NULL);
  NORM("nothing asked for", MOESQ_ERR_NULL, hp, NULL, hp, 4, 64, 0.0, NULL, NULL, 0, NULL, NULL, NULL);
  NORM("codes NULL", MOESQ_ERR_NULL, hp, NULL, hp, 4, 64, 0.0, NULL, h2, 1, NULL, bp, NULL);
  NORM("row_scale NULL", MOESQ_ERR_NULL, hp, NULL, hp, 4, 64, 0.0, NULL, h2, 3, bp, bp, NULL);
  NORM("y over x with a residual", MOESQ_ERR_ARG, hp, h2, h4, 4, 64, 0.0, h3, hp, 0, NULL, NULL, NULL);
  NORM("y over residual_out", MOESQ_ERR_ARG, hp, h2, h4, 4, 64, 0.0, h3, h3, 0, NULL, NULL, NULL);
  NORM("misaligned", MOESQ_ERR_ARG, (uint16_t *)P(0x18), NULL, hp, 4, 64, 0.0, NULL, h2, 0, NULL, NULL, NULL);
  NORM("codes misaligned", MOESQ_ERR_ARG, hp, NULL, hp, 4, 64, 0.0, NULL, h2, 1, (uint8_t *)P(0x11), bp, NULL);
  NORM("T=0", MOESQ_OK, NULL, NULL, NULL, 0, 64, 0.0, NULL, NULL, 0, NULL, NULL, NULL);

  /* microscaled rows */
  expect("mx_quantize rows<0", moesq_mx_quantize(fp, 0, low, 64, 1, bp, bp, NULL), MOESQ_ERR_SHAPE);
  expect("mx_quantize K lowest", moesq_mx_quantize(fp, 0, 4, low, 1, bp, bp, NULL), MOESQ_ERR_SHAPE);
  expect("mx_quantize K%32", moesq_mx_quantize(fp, 0, 4, top, 1, bp, bp, NULL), MOESQ_ERR_SHAPE);
  expect("mx_quantize dtype", moesq_mx_quantize(fp, -1, 4, 64, 1, bp, bp, NULL), MOESQ_ERR_ARG);
  expect("mx_quantize format", moesq_mx_quantize(fp, 0, 4, 64, 3, bp, bp, NULL), MOESQ_ERR_ARG);
  expect("mx_quantize NULL", moesq_mx_quantize(fp, 0, 4, 64, 1, NULL, bp, NULL), MOESQ_ERR_NULL);
  expect("mx_quantize misaligned", moesq_mx_quantize(P(0x14), 0, 4, 64, 1, bp, bp, NULL), MOESQ_ERR_ARG);
  expect("mx_quantize no rows", moesq_mx_quantize(NULL, 0, 0, 64, 1, NULL, NULL, NULL), MOESQ_OK);
#define ROWS(name, rows, K, format) moesq_mx_t name = {bp, bp, rows, K, format}
  ROWS(x4, 4, 128, 2);
  ROWS(bad_k, 4, 48, 1);
  ROWS(low_k, 4, low, 1);
  ROWS(low_rows, low, 128, 1);
  ROWS(nvfp4, 4, 128, 3);
  ROWS(none, 0, 128, 1);
  moesq_mx_t no_scales = {bp, NULL, 4, 128, 1};
  expect("mx_decode NULL descriptor", moesq_mx_decode(NULL, hp, NULL), MOESQ_ERR_NULL);
  expect("mx_decode K", moesq_mx_decode(&bad_k, hp, NULL), MOESQ_ERR_SHAPE);
  expect("mx_decode K lowest", moesq_mx_decode(&low_k, hp, NULL), MOESQ_ERR_SHAPE);
  expect("mx_decode rows lowest", moesq_mx_decode(&low_rows, hp, NULL), MOESQ_ERR_SHAPE);
  expect("mx_decode format", moesq_mx_decode(&nvfp4, hp, NULL), MOESQ_ERR_ARG);
  expect("mx_decode NULL scales", moesq_mx_decode(&no_scales, hp, NULL), MOESQ_ERR_NULL);
  expect("mx_decode misaligned", moesq_mx_decode(&x4, (uint16_t *)P(0x18), NULL), MOESQ_ERR_ARG);
  expect("mx_decode no rows", moesq_mx_decode(&none, NULL, NULL), MOESQ_OK);

  /* the product */
#define GEMM(what, want, x, perm, T, k, off, M, w, E, epi, y) \
  expect("mx_gemm " what, moesq_mx_gemm(x, perm, T, k, off, M, w, E, epi, y, NULL), want)
  ROWS(w8, 8 * 64, 128, 1);
  ROWS(w_none, 0, 128, 1);
  ROWS(w_low, low, 128, 1);
  ROWS(w_odd, 8 * 64 + 1, 128, 1);
  ROWS(w_n24, 8 * 24, 128, 1);
  ROWS(w_n48, 8 * 48, 128, 1);
  ROWS(w_wide, 8 << 16, 1 << 17, 1);
  ROWS(x_wide, 4, 1 << 17, 1);
  ROWS(x_many, 1 << 20, 8192, 2);
  ROWS(w_8192, 8 * 64, 8192, 1);
  ROWS(x_top, top, 32, 1);
  ROWS(w_k32, 8 * 64, 32, 1);
  GEMM("x NULL", MOESQ_ERR_NULL, NULL, NULL, 0, 1, ip, 4, &w8, 8, 0, hp);
  GEMM("w NULL", MOESQ_ERR_NULL, &x4, NULL, 0, 1, ip, 4, NULL, 8, 0, hp);
  GEMM("x format", MOESQ_ERR_ARG, &nvfp4, NULL, 0, 1, ip, 4, &w8, 8, 0, hp);
  GEMM("w format", MOESQ_ERR_ARG, &x4, NULL, 0, 1, ip, 4, &x4, 8, 0, hp);
  GEMM("epilogue", MOESQ_ERR_ARG, &x4, NULL, 0, 1, ip, 4, &w8, 8, low, hp);
  GEMM("flat without perm", MOESQ_ERR_ARG, &x4, NULL, 0, 1, ip, 4, &w8, 8, MOESQ_OUT_FLAT, hp);
  GEMM("E=0", MOESQ_ERR_SHAPE, &x4, NULL, 0, 1, ip, 4, &w8, 0, 0, hp);
  GEMM("E lowest", MOESQ_ERR_SHAPE, &x4, NULL, 0, 1, ip, 4, &w8, low, 0, hp);
  GEMM("E past its limit", MOESQ_ERR_SHAPE, &x4, NULL, 0, 1, ip, 4, &w8, MOESQ_MAX_EXPERTS + 1, 0, hp);
  GEMM("no weight rows", MOESQ_ERR_SHAPE, &x4, NULL, 0, 1, ip, 4, &w_none, 8, 0, hp);
  GEMM("weight rows lowest", MOESQ_ERR_SHAPE, &x4, NULL, 0, 1, ip, 4, &w_low, 8, 0, hp);
  GEMM("weight rows not E*N", MOESQ_ERR_SHAPE, &x4, NULL, 0, 1, ip, 4, &w_odd, 8, 0, hp);
  GEMM("N%16", MOESQ_ERR_SHAPE, &x4, NULL, 0, 1, ip, 4, &w_n24, 8, 0, hp);
  GEMM("SwiGLU N%32", MOESQ_ERR_SHAPE, &x4, NULL, 0, 1, ip, 4, &w_n48, 8, MOESQ_EPI_SWIGLU, hp);
  GEMM("K differs", MOESQ_ERR_SHAPE, &x4, NULL, 0, 1, ip, 4, &w_k32, 8, 0, hp);
  GEMM("M lowest", MOESQ_ERR_SHAPE, &x4, NULL, 0, 1, ip, low, &w8, 8, 0, hp);
  GEMM("M past its limit", MOESQ_ERR_SHAPE, &x_top, NULL, 0, 1, ip, top, &w_k32, 8, 0, hp);
  GEMM("x rows", MOESQ_ERR_SHAPE, &x4, NULL, 0, 1, ip, 5, &w8, 8, 0, hp);
  GEMM("T*k", MOESQ_ERR_SHAPE, &x4, ip, 4, 2, ip, 7, &w8, 8, 0, hp);
  GEMM("T*k overflow", MOESQ_ERR_SHAPE, &x4, ip, top, top, ip, 1, &w8, 8, 0, hp);
  GEMM("k=0", MOESQ_ERR_SHAPE, &x4, ip, 4, 0, ip, 0, &w8, 8, 0, hp);
  GEMM("perm without offsets", MOESQ_ERR_NULL, &x4, ip, 4, 1, NULL, 4, &w8, 8, 0, hp);
  GEMM("experts without offsets", MOESQ_ERR_NULL, &x4, NULL, 0, 1, NULL, 4, &w8, 8, 0, hp);
  GEMM("expert of 4 GiB", MOESQ_ERR_SHAPE, &x_wide, NULL, 0, 1, ip, 4, &w_wide, 8, 0, hp);
  GEMM("activations of 4 GiB", MOESQ_ERR_SHAPE, &x_many, NULL, 0, 1, ip, 1 << 20, &w_8192, 8, 0, hp);
  GEMM("y NULL", MOESQ_ERR_NULL, &x4, NULL, 0, 1, ip, 4, &w8, 8, 0, NULL);
  GEMM("y misaligned", MOESQ_ERR_ARG, &x4, NULL, 0, 1, ip, 4, &w8, 8, 0, (uint16_t *)P(0x18));
  GEMM("no rows", MOESQ_OK, &none, NULL, 0, 1, ip, 0, &w8, 8, 0, NULL);

  printf("%s: %d failure(s)\n", failures ? "FAILED" : "ok", failures);
  return failures ? 1 : 0;
}
