"""What the adapters' kernels decide in plain arithmetic, compiled for the host
and run on the CPU."""
import random

from test_expert_products_host import run

SHARES = r"""
#include <cstdio>
#include "lora_common.cuh"
using namespace situ::lora;
int main() {
  // tiles and chunks planned for, SMs, tiles that are left
  long tiles, chunks, sms, left;
  while (scanf("%ld %ld %ld %ld", &tiles, &chunks, &sms, &left) == 4) {
    const Shares s(tiles, chunks, sms);
    const long T = left * chunks, G = sharers(T, s.ctas, s.least);
    long most = 0, wrong = 0, next = 0;
    for (long c = 0; c < G; ++c) {          // ranges follow each other and cover everything
      wrong += first_item(c, T, G) != next;
      next = first_item(c + 1, T, G);
    }
    wrong += next != T;
    for (long t = 0; t < left; ++t) {
      const long a = cta_of(t * chunks, T, G), b = cta_of(t * chunks + chunks - 1, T, G);
      if (b - a + 1 > most) most = b - a + 1;
      for (long i = t * chunks; i < (t + 1) * chunks; i += chunks > 1 ? chunks - 1 : 1) {
        const long c = cta_of(i, T, G);
        wrong += c < 0 || c >= G || first_item(c, T, G) > i || first_item(c + 1, T, G) <= i;
      }
    }
    printf("%ld %ld %ld\n", most, s.most, wrong);
  }
}
"""


def test_a_tile_comes_in_no_more_parts_than_there_is_room_for(tmp_path):
    rng = random.Random(2)
    cases = [(4, 9, 152, left) for left in range(5)] + [(1, 1, 152, 1), (1, 2, 152, 1), (64, 56, 152, 64), (1, 16384, 152, 1)]
    for _ in range(1500):
        tiles, chunks = int(2 ** rng.uniform(0, 8)), int(2 ** rng.uniform(0, 7))
        cases.append((tiles, chunks, rng.choice([1, 8, 148, 152]), rng.randint(0, tiles)))
    lines = run(tmp_path, SHARES, "".join("%d %d %d %d\n" % c for c in cases)).splitlines()
    assert len(lines) == len(cases)
    for case, line in zip(cases, lines):
        most, room, wrong = map(int, line.split())
        assert most <= room and wrong == 0, case
