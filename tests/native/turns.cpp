// Prints turn_fraction of every frequency given (hexadecimal floating point), one
// a line.  Compiled by tests/test_turns.py with the host compiler.
#include <cinttypes>
#include <cstdio>
#include <cstdlib>

#include "turns.h"

int main(int argc, char** argv) {
  for (int i = 1; i < argc; ++i) std::printf("%" PRIu64 "\n", loong::turn_fraction(std::strtod(argv[i], nullptr)));
  return 0;
}
