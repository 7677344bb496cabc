// Prints whether the scan takes each ticket read from the input ("ticket
// tiles" a line) for a tile, the test that both of its kernels make.
#include <cstdint>
#include <cstdio>

#include "kda_layer.h"

int main() {
  unsigned long ticket;
  int tiles;
  while (std::scanf("%lu %d", &ticket, &tiles) == 2) std::printf("%d\n", kda::is_tile(uint32_t(ticket), tiles) ? 1 : 0);
  return 0;
}
