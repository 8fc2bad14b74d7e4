"""The hand-over of the second tile's maxima and sums in the attention over a paged cache (csrc/handover.h), compiled for
the host.  The giver may hand over twice before the taker has looked once: every state of the two that can come
about is gone through, and the taker's wait has to end where its hand-over is there, and only there."""
import os

from test_handover import CSRC, run_on_host

DRIVER = r"""
#include <cstdio>
#include "handover.h"

// A parity wait ends once the phase with that parity is complete: the barrier's current phase has the other one.
struct Barrier {
  int phase = 0;
  void complete() { ++phase; }
  bool over(int parity) const { return (phase & 1) != parity; }
};

// `given` and `taken` hand-overs through n buffers, the giver `lead` ahead at most; barriers of them: 0 or a fault.
int look(int n, int barriers, int lead, bool say) {
  for (int given = 0; given <= 40; ++given)
    for (int taken = given > lead ? given - lead : 0; taken <= given; ++taken) {
      Barrier b[4];
      for (int k = 0; k < given; ++k) b[fbd::handover::buffer_of(k, barriers)].complete();
      if (b[fbd::handover::buffer_of(taken, barriers)].over(fbd::handover::parity_of(taken, barriers)) != (given > taken)) {
        if (say) std::printf("%d buffers, %d given, %d taken\n", n, given, taken);
        return 1;
      }
      for (int k = taken; k < given; ++k)  // none of those under way lies in another's buffer
        for (int j = taken; j < k; ++j)
          if (fbd::handover::buffer_of(k, n) == fbd::handover::buffer_of(j, n)) return 1;
    }
  return 0;
}

int main() {
  if (look(2, 2, 2, true)) return 1;                      // the kernel's
  if (!look(2, 1, 2, false)) return std::printf("one barrier for two buffers holds?\n"), 1;
  for (int n = 1; n <= 4; ++n)
    if (look(n, n, n, true)) return 1;
  return 0;
}
"""


def test_a_taker_sees_each_of_two_hand_overs(tmp_path):
    run_on_host(tmp_path, DRIVER)


def test_the_kernel_has_a_barrier_for_each_buffer():
    """Both places of the kernel take buffer, barrier and parity of the same hand-over from there."""
    with open(os.path.join(CSRC, "tc_paged.cu")) as f:
        text = f.read()
    assert "handover::buffer_of(shared, 2)" in text and "handover::parity_of(shared, 2)" in text
    assert "mbar_arrive(x_full)" not in text and "wait(x_full" not in text
