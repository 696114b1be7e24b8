// Host program for the tests: the form that a product of moe_int8_product takes
// (mixture_experts_ffn_14_b200/csrc/int8_plan.cuh). Reads lines "R K N n_experts x_dtype with_up",
// writes "tile_rows split workspace_bytes" for each.
#include <cstdio>

#include "int8_plan.cuh"

int main() {
  long long R, K, N;
  int n, x, dual;
  while (std::scanf("%lld %lld %lld %d %d %d", &R, &K, &N, &n, &x, &dual) == 6) {
    const moe::i8::Layout L = moe::i8::plan(R, K, N, n, static_cast<moe_dtype_t>(x), dual != 0);
    std::printf("%d %d %zu\n", L.tile_rows, L.split, L.total);
  }
  return 0;
}
