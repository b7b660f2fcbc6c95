// Prints the softmax loss's plans of the sizes on standard input: "rows vocab dim narrow dtype" a line.
#include <cinttypes>
#include <cstdio>

#include "loss_plan.hpp"

int main() {
  long long n, v, k;
  int narrow, dtype;
  while (std::scanf("%lld %lld %lld %d %d", &n, &v, &k, &narrow, &dtype) == 5) {
    const tbe::LossForwardPlan f = tbe::plan_loss_forward(n, v, k, narrow, dtype);
    const tbe::LossBackwardPlan b = tbe::plan_loss_backward(n, v, k, narrow, dtype);
    std::printf("%d %d %" PRId64 " %" PRId64 " %" PRId64 " %d %" PRId64 " %" PRId64 " %" PRId64 " %d %" PRId64 " %" PRId64
                " %d %" PRId64 " %" PRId64 " %" PRId64 " %" PRId64 " %" PRId64 " %" PRId64 " %d\n",
                f.tile, f.narrow, f.tiles, f.run, f.segments, b.tile, b.piece, b.pieces, b.width, b.x.tile, b.x.splits,
                b.x.each, b.w.tile, b.w.splits, b.w.each, b.nx.splits, b.nx.run, b.nw.splits, b.nw.run,
                tbe::narrow_rows(k, dtype) ? 1 : 0);
  }
}
