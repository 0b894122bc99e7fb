/* Host checks of the 4-bit and expert calls: invalid, extreme and empty arguments.  Every call here is refused or has
 * nothing to do before anything is enqueued, so no GPU is needed. */
#include "lora_batch.h"

#include <limits.h>
#include <stdio.h>
#include <string.h>

static int failures;

#define CHECK(cond)                                                     \
  do {                                                                  \
    if (!(cond)) {                                                      \
      fprintf(stderr, "%s:%d: %s\n", __FILE__, __LINE__, #cond);        \
      failures++;                                                       \
    }                                                                   \
  } while (0)
#define REFUSED(call) CHECK((call) != LORA_OK)

static char mem[1 << 14] __attribute__((aligned(256)));

static lora_quant quant(void* codes, void* scales, int ld, int lds) {
  lora_quant q;
  memset(&q, 0, sizeof q);
  q.codes = (unsigned char*)codes;
  q.scales = (unsigned char*)scales;
  q.ld = ld;
  q.lds = lds;
  return q;
}

static const int kExtreme[] = {INT_MIN, INT_MIN + 1, -8, -1, 0, 1, 7, 8, 255, 256, 257, 1 << 20, 1 << 30, INT_MAX - 255, INT_MAX - 7, INT_MAX};
#define N ((int)(sizeof kExtreme / sizeof *kExtreme))

int main(void) {
  void* p = mem;
  const lora_quant none = quant(0, 0, 0, 0);
  const int big_ld = INT_MAX - 127, big_lds = INT_MAX - 7;
  const lora_quant wide = quant(p, p, big_ld, big_lds);
  lora_segments seg;
  memset(&seg, 0, sizeof seg);

  /* sizes of every magnitude, with null pointers: refused, or nothing to do, without an overflow */
  for (int a = 0; a < N; a++)
    for (int b = 0; b < N; b++) {
      const int r = kExtreme[a], c = kExtreme[b];
      (void)lora_base_product_mx_workspace_bytes(r, c, 8);
      (void)lora_base_product_mx_workspace_bytes(8, r, c);
      (void)lora_base_product_mx_workspace_bytes(c, 4096, r);
      for (int type = -1; type < 4; type++) {
        const int none_to_do = type >= 0 && type <= 1 && r == 0 && c >= 0;
        CHECK(none_to_do || lora_quant_rows_mx(type, 0, c, r, c, none, 0) != LORA_OK);
        CHECK(none_to_do || lora_dequant_rows_mx(type, none, r, c, 0, c, 0) != LORA_OK);
        REFUSED(lora_quant_weight_mx(type, 0, c, r == 0 ? 8 : r, c, type & 1, none, 0));
        for (int e = 0; e < N; e += 3) {
          const int n = kExtreme[e];
          for (int bits = 3; bits < 10; bits++) {
            if (r == 0 || n == 0 || n < 0) continue;
            REFUSED(lora_base_product_mx(type, bits, none, r, c, none, n, 0, n, 0, 0, 0, 0));
            REFUSED(lora_base_product_mx(type, bits, wide, r < 0 ? r : -1, c, wide, n, p, n, 1, p, (size_t)-1, 0));
            REFUSED(lora_expert_product_mx(type, bits, none, r, c, none, n, 8, seg, 0, 8, 0, 0));
            REFUSED(lora_expert_product_mx(type, bits, none, r, c, none, 4, n, seg, 0, n, 1, 0));
          }
          if (r > 0) {
            REFUSED(lora_expert_gather(type, 0, c, r, n, 8, 0, 0, c, 0));
            REFUSED(lora_expert_gather_backward(type, 0, c, r, n, 8, 0, 0, c, 0, 0));
            REFUSED(lora_expert_combine(type, 0, c, r, n, 8, 0, 0, 0, c, 0, 0));
            REFUSED(lora_expert_combine_backward(type, 0, c, 0, c, r, n, 8, 0, 0, 0, c, 0, 0));
            REFUSED(lora_expert_segments(0, r, n, c, seg, 0, 0, 0, 0));
          }
        }
      }
    }

  /* the choice of kernel and its tiles for rows and outputs of every magnitude: a workspace of no bytes is refused last */
  for (int a = 0; a < N; a++)
    for (int b = 0; b < N; b++)
      for (int bits = 4; bits <= 8; bits += 4)
        for (int type = 0; type < 2; type++) {
          const int n = kExtreme[b];
          if (kExtreme[a] == 0) continue;
          REFUSED(lora_base_product_mx(type, bits, wide, kExtreme[a], 8, wide, n, p, n, 0, p, 0, 0));
          REFUSED(lora_base_product_mx(type, bits, wide, kExtreme[a], INT_MAX - 255, wide, n, p, n, 1, p, 0, 0));
        }

  printf("mx checks: %s\n", failures ? "FAILED" : "ok");
  return failures != 0;
}
