// CTAs and stages of norm_quant_stream_kernel, from sizes alone (host only).
#pragma once

#include <algorithm>
#include <cstdint>

namespace qbsa {

constexpr int kNormMaxStages = 4;
constexpr int kNormRingBytes = 216 * 1024;  // of an SM's shared memory for rings, over its resident CTAs
constexpr int kSmSharedBytes = 228 * 1024;  // an SM's shared memory in all
constexpr int kCtaSharedBytes = 1024;       // the system's share of a CTA's

struct StreamPlan {
  int per_sm;  // resident CTAs
  int stages;  // rows in flight per CTA; below 2 there is no room to stream, and the rest has no meaning
  int64_t smem;  // dynamic shared memory of a CTA
};

// resident: threads of an SM by the kernel's registers; stage: bytes of a row in flight; staged: of the
// rows that go out through shared memory; fixed: the kernel's static shared memory.
// Rings share kNormRingBytes.  What an SM has beyond it holds the fixed and system shares of few CTAs only,
// so the grid is cut to the CTAs that fit: those that do not would run after the others, each with as many
// rows (f32 with a residual, 65536 x 1536: 9 CTAs 274 us, the 8 that fit 209; bf16, 65536 x 1360: 223 and 166).
inline StreamPlan plan_stream(int resident, int threads, int64_t stage, int64_t staged, int64_t fixed) {
  StreamPlan p = {std::max(1, std::min(32, resident / threads)), 0, 0};
  while (p.per_sm > 1 && (2 * stage + staged) * p.per_sm > kNormRingBytes) --p.per_sm;
  p.stages = static_cast<int>(std::min<int64_t>(kNormMaxStages, (kNormRingBytes / p.per_sm - staged) / stage));
  if (p.stages < 2) return p;
  p.smem = p.stages * stage + staged;
  const int64_t cta = (p.smem + fixed + kCtaSharedBytes + 127) / 128 * 128;
  p.per_sm = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(p.per_sm, kSmSharedBytes / cta)));
  return p;
}

}  // namespace qbsa
