// Prints the launch shape that the library chooses for adapter calls: argv holds
// any number of M,N,K,n_req,rank,n_nseg (equal N-segments); a line of
// one_launch rows_per_tile by_row run_blocks splits for each.
#include <cstdio>

#include "sq_rows.hpp"

int main(int argc, char **argv) {
  for (int i = 1; i < argc; ++i) {
    long M, N, K;
    int n_req, rank, n_nseg;
    if (sscanf(argv[i], "%ld,%ld,%ld,%d,%d,%d", &M, &N, &K, &n_req, &rank, &n_nseg) != 6) return 1;
    sq::AdapterProblem p{};
    p.M = M;
    p.N = N;
    p.K = K;
    p.n_req = n_req;
    p.rank = rank;
    p.ns.n = n_nseg;
    for (int s = 0; s < n_nseg; ++s) p.ns.end16[s] = (uint16_t)(N / 16 * (s + 1) / n_nseg);
    sq::adapter_plan(p);
    printf("%d %d %d %d %d\n", p.one, 16 * (p.one ? 1 : p.expand_mt), p.by_row, p.run_tiles,
           p.splits);
  }
  return 0;
}
