// Prints the plan that the feed-forward block's host side makes: for each group of arguments
// "tokens hidden inner odd" one line of name=value pairs.  odd: rows start between 16-byte
// boundaries.  Host code only: no pointer is followed.
#include <stdio.h>
#include <stdlib.h>

#include "ffn_internal.h"

int main(int argc, char** argv) {
  for (int i = 1; i + 3 < argc; i += 4) {
    const int64_t T = atoll(argv[i]), H = atoll(argv[i + 1]), F = atoll(argv[i + 2]);
    const char* at = (const char*)0x1000000 + (atoi(argv[i + 3]) ? 2 : 0);
    const zero_ffn_t f = {T, H, F, at, H, at, H, at, H, at, F, ZERO_BF16, ZERO_ACT_SILU};
    zero_ffn_grads_t g = {};
    g.dy = at;
    g.lddy = H;
    const zk::FfnPlan p = zk::ffn_plan(&f, nullptr), q = zk::ffn_plan(&f, &g);
    printf("few=%d low=%d sets_in=%d sets_out=%d pack=%d small_in=%d small_out=%d "
           "small_back1=%d small_back2=%d split_in=%d split_y=%d split_dh=%d split_dw1=%d "
           "split_dx=%d split_dw2=%d\n",
           p.few, p.low, p.few_sets_in, p.few_sets_out, q.pack_x || q.pack_down, p.small_in,
           p.small_out, q.small_back1, q.small_back2, p.split_in, p.split_y, q.split_dh,
           q.split_dw1, q.split_dx, q.split_dw2);
  }
  return 0;
}
