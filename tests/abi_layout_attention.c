/* Prints the size and field offsets of the attention calls' structs
 * (include/fp4.h), one "struct.field offset" per line. */
#include <stddef.h>
#include <stdio.h>

#include "fp4.h"

#define F(S, f) printf(#S "." #f " %zu\n", offsetof(S, f))

int main(void) {
  printf("fp4_heads.__size__ %zu\n", sizeof(fp4_heads));
  F(fp4_heads, x);
  F(fp4_heads, token_stride);
  F(fp4_heads, head_stride);
  F(fp4_heads, heads);
  printf("fp4_qk_norm.__size__ %zu\n", sizeof(fp4_qk_norm));
  F(fp4_qk_norm, q_weight);
  F(fp4_qk_norm, k_weight);
  F(fp4_qk_norm, weight_f32);
  F(fp4_qk_norm, eps);
  F(fp4_qk_norm, table);
  F(fp4_qk_norm, table_rows);
  F(fp4_qk_norm, rotary_dim);
  F(fp4_qk_norm, interleaved);
  printf("fp4_kv_cache.__size__ %zu\n", sizeof(fp4_kv_cache));
  F(fp4_kv_cache, format);
  F(fp4_kv_cache, heads);
  F(fp4_kv_cache, head_dim);
  F(fp4_kv_cache, page_size);
  F(fp4_kv_cache, pages);
  F(fp4_kv_cache, k_codes);
  F(fp4_kv_cache, k_scales);
  F(fp4_kv_cache, v_codes);
  F(fp4_kv_cache, v_scales);
  F(fp4_kv_cache, page_stride);
  F(fp4_kv_cache, head_stride);
  F(fp4_kv_cache, token_stride);
  F(fp4_kv_cache, scale_page_stride);
  F(fp4_kv_cache, scale_head_stride);
  F(fp4_kv_cache, scale_block_stride);
  F(fp4_kv_cache, amax);
  F(fp4_kv_cache, target);
  return 0;
}
