// What the kernels of a mixture of experts are planned for.  Plain C++: host only.
#pragma once

#include <algorithm>
#include <cmath>
#include <cstdint>

namespace gptq {

struct ExpertLoad {
    double experts;  // distinct experts that the tokens choose between them, as expected
    int rows;        // tokens that share one of them
};

// A token's top_k experts are distinct and taken to be any top_k with equal
// chance, so all tokens miss an expert with probability (1 - top_k/E)^T.  The
// quotient is a whole number up to rounding for one token (one) and for
// top_k = E (all tokens), hence the slack before it is rounded up.
inline ExpertLoad expert_load(int64_t tokens, int n_experts, int top_k) {
    const double experts = n_experts * (1.0 - std::pow(1.0 - (double)top_k / n_experts, (double)tokens));
    const double rows = std::ceil((double)(tokens * top_k) / experts * (1.0 - 1e-9));
    return {experts, (int)std::min((double)tokens, rows)};
}

}  // namespace gptq
