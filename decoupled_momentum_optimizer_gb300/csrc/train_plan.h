// How a product of quantized matrices runs on a device (train_matmul.cu): host arithmetic alone.
#pragma once

#include <algorithm>

namespace demo {

constexpr int kBlock = 128;  // elements that share a scale
constexpr int kBM = 128, kBN = 224;  // rows of a CTA's tile, most columns
constexpr int kChain = 4;            // blocks of 128 that one half of tensor memory sums
constexpr int kMaxSplit = 8;         // parts of k: the portable cluster size
constexpr int kMaxStages = 8, kPairStages = 5;
constexpr int kRingBytesSingle = 3 * (kBM + kBN) * kBlock;  // a single CTA's stages

// Clusters of 1 .. kMaxSplit single CTAs, and pairs (entry 0), that a device runs at one time: a
// cluster stays within a group of SMs, so these are fewer than the SMs divided by the size, and differ
// from one device to another.
struct Clusters {
  int of[kMaxSplit + 1];
};

// CTAs that share a tile's rows (1 or 2), the tile's width, the parts k is cut into, the stages, the grid
// (0: the device has no place for the kernel); and the tensor maps' boxes (rows of codes, blocks of
// scales).
struct MatmulPlan {
  int group, bn, split, stages, rows_a, rows_b, chain;
  unsigned int grid;
};

// Few tiles (128 x 224 ones that would leave half of the SMs idle, or m that fills no pair): one CTA
// per tile, with k cut into parts where that pays.  Otherwise pairs.  Either way the cheapest width
// (and number of parts) in cycles.
//
// A pair: a block costs max(2 bn, 256 + bn) (the tensor cores, or what a CTA reads at 64 bytes a
// cycle), a tile about 2500 more.
//
// A single CTA: a block costs what the CTA reads, the tensor core, or a stage's round trip of about
// 2200 shared by the stages, whichever is longest (at 1400, 8 x 2048 x 8192 was cut into too few parts
// and took 13.8 us of 9.1; at 3200, 200 x 2048 x 8192 took 13.7 of 12.2).  Joining parts costs about
// 10000 and the reading of a tile of sums.  A tile that is not cut is staged, where eight rows' 16-byte
// stores of bn bytes apart meet in the same banks, 8 ways at widths of whole 128s, 4 of 64s, 2 of 32s:
// 2 bn cycles for each way (32 x 1024 x 128 at widths 64, 96 .. 224: 3.75, 3.80, 4.76, 4.11, 4.65,
// 4.45 us).  Stores in another order for each row have no conflicts, but the exchange of registers
// before them cost every width 0.6 to 1 us: it is code that runs once.
//
// Without place for a single CTA the plan's grid is 0; without place for a pair everything goes to
// single CTAs.
inline MatmulPlan plan_matmul(const Clusters& clusters, long long m, long long n, int kb) {
  const int sms = clusters.of[1];
  const auto tiles = [&](int rows, int bn) { return ((m + rows - 1) / rows) * ((n + bn - 1) / bn); };
  MatmulPlan plan = {};
  plan.split = 1;
  if (sms < 1) return plan;
  plan.group = m <= kBM || 2 * tiles(kBM, kBN) <= sms || clusters.of[0] < 1 ? 1 : 2;
  int rows_a = kBM;
  const auto stages_of = [&](int bn) {
    const int fit = kRingBytesSingle / ((rows_a + bn) * kBlock);
    return fit < kMaxStages ? fit : kMaxStages;
  };
  double best = 0;
  const auto offer = [&](int bn, int split, double cost, long long grid) {
    if (best == 0 || cost < best) {
      best = cost;
      plan.bn = bn;
      plan.split = split;
      plan.grid = static_cast<unsigned>(grid);
    }
  };
  if (plan.group == 1) {
    const int chains = (kb + kChain - 1) / kChain;
    const double rows = m < kBM ? m : kBM;
    rows_a = m < kBM ? static_cast<int>(m + 7) / 8 * 8 : kBM;
    for (int bn = kBN; bn >= 64; bn -= 32) {
      const long long t = tiles(kBM, bn);
      for (int split = 1; split <= kMaxSplit && (split == 1 || (split <= chains && t <= clusters.of[split])); ++split) {
        const double rounds = static_cast<double>((t + clusters.of[split] - 1) / clusters.of[split]);
        const double ways = bn % 128 == 0 ? 8 : bn % 64 == 0 ? 4 : 2;
        const double end = split > 1 ? 10000 + rows * bn / 8 : 500 + 2 * bn * ways;
        const int bytes = (rows_a + bn) * kBlock;
        const double block = std::max({bytes / 64.0, 2.0 * bn, 2200.0 / stages_of(bn)});
        offer(bn, split, rounds * (((kb + split - 1) / split) * block + end), t * split);
      }
    }
  } else {
    const long long pairs = clusters.of[0];
    for (int bn = kBN; bn >= 96; bn -= 32) {
      const long long t = tiles(2 * kBM, bn), rounds = (t + pairs - 1) / pairs;
      offer(bn, 1, static_cast<double>(rounds) * (2500.0 + static_cast<double>(kb) * (256 + bn)),
            2 * (t < pairs ? t : pairs));
    }
  }
  plan.rows_a = rows_a;
  plan.stages = plan.group == 1 ? stages_of(plan.bn) : kPairStages;
  plan.rows_b = plan.bn / plan.group;
  plan.chain = kChain;
  return plan;
}

}  // namespace demo
