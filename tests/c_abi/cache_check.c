/* As abi_check.c, for the paged cache and the attention over it: compiled as C99 against include/fa.h by
 * tests/test_c_abi_cache.py.  Every call here is answered by an argument check, before any CUDA call. */
#include <stdio.h>
#include <string.h>

#include "fa.h"

static int failures = 0;
#define CHECK(cond)                                                   \
  do {                                                                \
    if (!(cond)) {                                                    \
      printf("failed: %s (line %d)\n", #cond, __LINE__);              \
      ++failures;                                                     \
    }                                                                 \
  } while (0)

int main(void) {
  void* fake = (void*)(size_t)0x10000;   /* 256-byte aligned, never dereferenced */
  const int32_t* ints = (const int32_t*)fake;
  fa_cache c;
  fa_cache_append_args ap;
  fa_cache_read_args rd;
  fa_cache_keep_args kp;
  fa_fwd_tree_args tr;

  memset(&c, 0, sizeof c);
  c.k = c.v = fake;
  c.page_table = ints;
  c.pages = 8; c.Hk = 2; c.page_size = 16; c.d = 64; c.dtype = FA_BF16;
  c.B = 2; c.max_pages = 4; c.table_stride = 4;

  memset(&ap, 0, sizeof ap);
  ap.cache = c;
  ap.k_new = ap.v_new = fake;
  ap.k_token_stride = ap.v_token_stride = 128; ap.k_head_stride = ap.v_head_stride = 64;
  ap.cu_new = ap.lens = ints;
  ap.total = 4; ap.dtype = FA_FP16;                      /* not the cache's type */
  CHECK(fa_cache_append(&ap) == FA_ERR_UNSUPPORTED);
  ap.dtype = FA_BF16; ap.k_token_stride = 100;
  CHECK(fa_cache_append(&ap) == FA_ERR_INVALID_ARG);
  ap.k_token_stride = 128; ap.total = 0;
  CHECK(fa_cache_append(&ap) == FA_OK);
  CHECK(fa_cache_append(NULL) == FA_ERR_INVALID_ARG);

  memset(&rd, 0, sizeof rd);
  rd.cache = c;
  rd.cache.dtype = FA_E4M3;                              /* without scales */
  rd.lens = ints; rd.k_out = rd.v_out = fake; rd.N = 16; rd.dtype = FA_BF16;
  CHECK(fa_cache_read(&rd) == FA_ERR_INVALID_ARG);
  rd.cache.dtype = FA_BF16; rd.N = 0;
  CHECK(fa_cache_read(&rd) == FA_OK);
  CHECK(fa_cache_read(NULL) == FA_ERR_INVALID_ARG);

  memset(&kp, 0, sizeof kp);
  kp.cache = c;
  kp.cache.page_size = 24;
  kp.lens = kp.kept = kp.counts = ints; kp.width = 2;
  CHECK(fa_cache_keep(&kp) == FA_ERR_UNSUPPORTED);
  kp.cache.page_size = 16; kp.width = 0;
  CHECK(fa_cache_keep(&kp) == FA_OK);
  CHECK(fa_cache_keep(NULL) == FA_ERR_INVALID_ARG);

  memset(&tr, 0, sizeof tr);
  tr.cache = c;
  tr.q = tr.o = fake; tr.lse = (float*)fake;
  tr.q_token_stride = tr.o_token_stride = 256; tr.q_head_stride = tr.o_head_stride = 64;
  tr.cu_new = tr.lens = ints;
  tr.total = 4; tr.Hq = 4; tr.max_new = 2; tr.dtype = FA_BF16; tr.scale = 0.125f;
  tr.workspace = fake;
  tr.workspace_bytes = fa_fwd_tree_workspace_bytes(4, 4, 2, 64) - 1;
  CHECK(fa_fwd_tree(&tr) == FA_ERR_WORKSPACE);
  tr.Hq = 3;
  CHECK(fa_fwd_tree(&tr) == FA_ERR_INVALID_ARG);
  tr.Hq = 4; tr.tree_mask = (const uint64_t*)fake; tr.mask_words = 1; tr.max_new = 65;
  CHECK(fa_fwd_tree(&tr) == FA_ERR_INVALID_ARG);
  tr.tree_mask = NULL; tr.total = 0;
  CHECK(fa_fwd_tree(&tr) == FA_OK);
  CHECK(fa_fwd_tree(NULL) == FA_ERR_INVALID_ARG);
  CHECK(fa_fwd_tree_workspace_bytes(1, 8, 3, 64) == 0);

  if (failures == 0) printf("c abi ok\n");
  return failures;
}
