// Allocation-failure injection for the block manager's calls on drafted tokens
// (built and run by test_block_manager_tree_failures.py): the driver of
// bm_alloc_fail.cpp over reserve and commit.
#define main bm_alloc_fail_main
#include "bm_alloc_fail.cpp"
#undef main

int main() {
  pa_bm *bm = pa_bm_create_with_host(kBlocks, kHost, kB);
  if (!bm) return 1;
  std::vector<int32_t> prompt(22);
  for (int i = 0; i < (int)prompt.size(); ++i) prompt[i] = 1000 + i;
  int cached = 0;
  bool ok = pa_bm_add_seq_tokens(bm, 0, prompt.data(), 22, &cached) == PA_OK && pa_bm_fork(bm, 0, 1) == PA_OK &&
            pa_bm_add_seq(bm, 2, 0) == PA_OK && pa_bm_fork(bm, 0, 3) == PA_OK;
  const int32_t ids[4] = {1, 0, 2, 3};
  const int32_t tokens[64] = {7, 8, 9};
  int64_t slots[256], cow[8], slot = 0;
  const long long OOM = PA_ERR_OOM;
  // growing, shrinking and copying on write; then the accepted tokens, blocks filled and registered among them
  const int32_t counts[7][4] = {{3, 5, 9, 1}, {30, 1, 40, 0}, {1, 1, 1, 1}, {0, 0, 0, 0}, {17, 9, 12, 2}, {50, 0, 9, 3}, {8, 8, 8, 8}};
  for (int i = 0; i < 7 && ok; ++i) {
    ok = inject("reserve", bm, [&] { return (long long)pa_bm_reserve_batch(bm, ids, counts[i], 4, slots, cow); }, OOM);
    int32_t kept[4];
    for (int k = 0; k < 4; ++k) kept[k] = (counts[i][k] + 1) / 2;
    ok = ok && inject("commit", bm,
                      [&] { return (long long)pa_bm_commit_batch(bm, ids, kept, i % 2 ? nullptr : tokens, 4); }, OOM);
    ok = ok && inject("append", bm, [&] { return (long long)pa_bm_append(bm, 2, &slot, cow); }, OOM);
  }
  ok = ok && inject("fork", bm, [&] { return (long long)pa_bm_fork(bm, 2, 5); }, OOM);
  ok = ok && inject("wasted_slots", bm, [&] { return (long long)pa_bm_wasted_slots(bm); }, -1);
  for (int q : {0, 1, 2, 3, 5})
    if (ok) ok = pa_bm_free_seq(bm, q) == PA_OK;
  if (ok && pa_bm_num_free(bm) != kBlocks) {
    std::printf("blocks lost: %d free of %d\n", pa_bm_num_free(bm), kBlocks);
    ok = false;
  }
  pa_bm_destroy(bm);
  if (!ok) return 1;
  std::printf("ok %d\n", failures);
  return 0;
}
