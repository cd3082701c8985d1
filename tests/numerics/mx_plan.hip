// Prints the form that the library chooses for MXFP4 products: argv holds any number
// of M,N,K; a line of tile_shape quantises_inside for each.
#include <cstdio>

#include "sq_mx.hpp"

int main(int argc, char **argv) {
  for (int i = 1; i < argc; ++i) {
    long M, N, K;
    if (sscanf(argv[i], "%ld,%ld,%ld", &M, &N, &K) != 3) return 1;
    printf("%d %d\n", sq::mx_choice(M, N, K), sq::mx_rows_inside(M, N, K));
  }
  return 0;
}
