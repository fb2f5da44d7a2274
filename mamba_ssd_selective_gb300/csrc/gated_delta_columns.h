// TMEM columns of the gated delta rule's chain kernels (512 per block), apart from the
// kernels so that a host test can hold them against the order of the kernels' reads and writes.
#pragma once

namespace ssd {
namespace delta {

// The forward chain, 64 tokens each: Q S0^T | K S0^T from one product, w | M w from the next, which may
// begin while K S0^T is still read, so that no two of them share columns; the state in float32; operands.
namespace col {
constexpr int kQS = 0, kKS = 64, kW = 128, kMW = 192, kS = 256, kOp = 384;
static_assert(kKS == kQS + 64 && kMW == kW + 64, "each pair is one product's result");
}  // namespace col

// The reverse chain: X = E K^T, D (first dY^T (M T), then dR), the state's cotangent in float32, operands, and dY's
// operands, plain and times s exp(c).
namespace rev_col {
constexpr int kX = 0, kD = 64, kE = 128, kOp = 256, kY = 384, kYe = 448;
}  // namespace rev_col

}  // namespace delta
}  // namespace ssd
