// Prints, for n vocab cols per line of standard input, the rows that are filled beside the sort and a piece's positions.
#include <cstdio>

#include "train_embed_plan.h"

int main() {
  long long n, vocab, cols;
  while (std::scanf("%lld %lld %lld", &n, &vocab, &cols) == 3)
    std::printf("%lld %d\n", demo::filled_rows(n, vocab, cols), demo::embed_piece(n, cols));
  return 0;
}
