// Extents, workspaces and launch shapes of the adapters at the ends of what the C ABI takes (host code only).
#include <stdio.h>
#include <stdlib.h>

#include "mx_launch.hpp"

#define CHECK(cond)                                                   \
  do {                                                                \
    if (!(cond)) {                                                    \
      fprintf(stderr, "line %d: %s\n", __LINE__, #cond);              \
      exit(1);                                                        \
    }                                                                 \
  } while (0)

int main() {
  using namespace mxfp8;
  const int64_t rows[] = {1, 2, 31, 512, 513, 4096, 1 << 20, kMaxAdapterRows}, ranks[] = {8, 16, 24, 64, 136, kMaxRank};
  const int64_t widths[] = {32, 128, 3584, 1 << 20, (int64_t(1) << 30) - 128}, adapters[] = {1, 2, 300, 1 << 20, 1 << 30};
  for (int64_t M : rows)
    for (int64_t rank : ranks)
      for (int64_t C : widths) {
        CHECK(adapter_packed_bytes(M, rank) >= M * rank * 6);
        if (C % 128 == 0) CHECK(adapter_project_workspace(M, C, rank) >= 0);
        for (int64_t n : adapters) {
          CHECK(adapter_grad_groups(M, C, rank, n) >= n);
          const int64_t work = adapter_grad_workspace(M, C, rank, n);
          CHECK(work >= 0 && work <= (int64_t(256) << 20) + 512 * n * 4);
        }
      }
  printf("all checks passed\n");
  return 0;
}
