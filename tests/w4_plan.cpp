// Prints the plan of 4-bit products: a line of numbers per line of
// "rows experts k_in n_out group f32" (experts 0: one weight, no ids).
#include <cstdio>

#include "mlora_w4_plan.h"

int main() {
  int rows, experts, k, n, group, f32;
  while (std::scanf("%d %d %d %d %d %d", &rows, &experts, &k, &n, &group, &f32) == 6) {
    mlora_w4_route r{};
    r.n_experts = experts > 0 ? experts : 1;
    r.k_in = k;
    r.n_out = n;
    r.group = group;
    const int sg = group < 128 ? 128 / group : 1;
    const int32_t some = 0;
    const mlora::W4Rows w = {experts > 0 ? &some : nullptr, rows, r.n_experts};
    const mlora::W4Plan p = mlora::plan_w4(&r, w, f32 != 0, sg);
    const int chunks = (k + 127) / 128, most = mlora::panel_chunks(f32 != 0, p.mb, sg);
    std::printf("%d %d %d %d %d %d %d %d %d %d %d\n", p.stream, p.by_row, p.places, p.mb, p.tiles,
                p.waves, p.k_waves, p.splits, p.per_slice, p.slices, chunks > most);
  }
  return 0;
}
