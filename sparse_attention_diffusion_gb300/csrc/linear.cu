// bf16 matrix product with its epilogue: which kernel a problem takes, and the CTA-pair kernel without adapters.
#include "linear_pair.cuh"

namespace mcs {

// Which kernel and tile a problem takes: the smallest estimated time, in SM
// clocks, with constants from measured sweeps. A 64-column step of a tile costs
// its MMAs (8,192 FLOP per clock and SM), its loads (62 bytes per clock and SM out
// of L2) or a ring turn's latency (300), whichever is longest; a pair's tile is
// never shorter than its epilogue; tiles run in waves over the SMs (or pairs);
// reading every operand once from HBM (23 bytes per clock and SM) bounds
// everything; then come the start, the way out of the last tile (20 to 35 clocks a
// column or token) and the exchange between K slices.
LinearPlan plan_linear_tc(const LinearParams& p, int num_sms) {
  const int nk = (p.K + 63) / 64;
  const long long rows = p.heads > 0 ? p.N : p.M, sections = p.heads > 0 ? p.B : 1;
  const double hbm = 2.0 * (double(p.M) * p.K + double(p.O) * p.K + double(p.M) * p.O * (p.residual ? 2 : 1)) /
                     (23.0 * num_sms);
  auto larger = [](double a, double b) { return a > b ? a : b; };
  // the longer of two overlapping times, which slow each other down a little
  auto overlap = [](double a, double b) { return a > b ? a + 0.25 * b : b + 0.25 * a; };
  double best = 1e300;
  int pair_bn = 256;
  const long long row_tiles = (rows + 255) / 256 * sections;
  for (int widest = 256, last = 0; widest >= 32; widest -= 32) {
    const int cols = (p.O + widest - 1) / widest;
    const int bn = ((p.O + cols - 1) / cols + 31) / 32 * 32;  // equal column tiles, in steps of 32
    if (bn == last) continue;
    last = bn;
    const long long tiles = row_tiles * ((p.O + bn - 1) / bn), slots = num_sms / 2;
    const double step = larger(300, larger(2.0 * bn, (16384 + 64.0 * bn) / 62));
    const double tile = larger(nk * step, 850 + 14.0 * bn);  // its products, or its way out when K is short
    const double cost = overlap(double((tiles + slots - 1) / slots) * tile, hbm) + 6200 + 28 * bn;
    if (cost < best) best = cost, pair_bn = bn;
  }
  FewPlan few{};
  const long long otiles = (p.O + 127) / 128;
  for (int widest = 256, last = 0; widest >= 16 && rows <= 4096; widest -= widest > 64 ? 32 : 16) {
    const long long tt = (rows + widest - 1) / widest;
    const int bn = int((rows + tt - 1) / tt + 15) / 16 * 16;  // equal token tiles, in steps of 16
    if (bn == last) continue;
    last = bn;
    const long long tiles = otiles * sections * ((rows + bn - 1) / bn);
    const double step = larger(300, larger(2.0 * bn, (16384 + 128.0 * bn) / 62));
    for (int splits = 1; splits <= 8 && splits <= nk; ++splits) {
      const int steps = (nk + splits - 1) / splits;
      if (!few_fits(bn, steps)) continue;
      const int slots = few_slots(splits, num_sms);
      if (splits > 4 && tiles * splits > 64) break;  // clusters of more than four start late on a busy GPU
      // each CTA's way out is exposed once a wave, unless two CTAs share an SM
      const double waves = double((tiles * splits + slots - 1) / slots);
      const double out = splits > 1 ? 3500 + 20 * bn : 35 * bn;
      const double cost = overlap(waves * steps * step, hbm) + 6000 +
                          out * (few_two_per_sm(bn, steps) ? 1.0 : waves);
      if (cost < best) {
        best = cost;
        few.bn = bn;
        few.splits = splits;
      }
    }
  }
  if (few.bn > 0) return {MCS_LINEAR_FEW, few.bn, few.splits, acc_count((nk + few.splits - 1) / few.splits)};
  return {MCS_LINEAR_PAIRS, pair_bn, 1, acc_count(nk)};
}

cudaError_t linear_tc(const LinearParams& p, int num_sms, cudaStream_t s) {
  const LinearPlan plan = plan_linear_tc(p, num_sms);
  return plan.kernel == MCS_LINEAR_FEW ? linear_few(p, {plan.tile, plan.slices}, num_sms, s)
                                       : launch_pair<kNoAdapters>(p, plan.tile, nullptr, num_sms, s);
}

}  // namespace mcs
