// How the gradient of a token table is cut (train_embedding.cu): host arithmetic alone.
#pragma once

namespace demo {

// Bytes of the gradient that are filled while n tokens are sorted, about as many as take as long; the rest is left to
// the sums' kernel, which asks of a few rows at a time whether a token is there.  4096 tokens into 32128 x 768: 25.7 us
// with 48 MB filled beside the sort, 34.6 with none, 30.8 with all 99 MB; 65536 into 50304 x 768 72 us with 142 MB, 80
// with 48.  Narrow rows make that question dear: 16384 into 500000 x 64 38 us with all filled, 44 with half.
constexpr long long fill_bytes(long long n, long long cols) { return ((44ll << 20) + 1536 * n) * (cols < 128 ? 2 : 1); }

// Rows that are filled so, the table's first ones.  Those behind them are zeroed a few at a time (4, 8, 16 or 32), as one
// run of 16-byte accesses where the rows lie end to end: a multiple of four rows keeps every run on that boundary whatever
// the width.  3000 positions into 900000 x 33 32 us, 35 from a row that leaves no run there; 4096 into 100000 x 250 37 and
// 41; into 32128 x 765, whose runs are long either way, 32 and 32.
constexpr long long filled_rows(long long n, long long vocab, long long cols) {
  const long long rows = ((fill_bytes(n, cols) / 4 + cols - 1) / cols + 3) / 4 * 4;
  return rows < vocab ? rows : vocab;
}

// Sorted positions of a piece (one warp's work on 256 columns): 32, or fewer where those would leave an SM fewer
// than three warps.  Sums and join, bfloat16 dy, us with 8 / 16 / 32 positions: 16384 x 2048 48 / 43 / 39, 4096 x
// 768 10.3 / 10.8 / 11.7, 128 x 768 7.2 / 9.2 / 12.7; three tokens, 16384 x 32, 19 / 15 / 14.
// (152 SMs, whatever the device has: the workspace's size is asked for without one, and the sums' order is the same on all.)
constexpr int embed_piece(long long n, long long cols) {
  const long long slabs = (cols + 255) / 256;
  int piece = 32;
  while (piece > 8 && (n + piece - 1) / piece * slabs < 152 * 3) piece /= 2;
  return piece;
}

}  // namespace demo
