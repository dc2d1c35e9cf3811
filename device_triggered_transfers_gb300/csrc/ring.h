// How a row kernel of the norm shares an SM out: CTAs, and the stages that each one's rows come through.
#pragma once

#include <algorithm>
#include <cstdint>

namespace dtt {
namespace ring {

constexpr uint32_t kThreads = 512;          // of a row, at most
constexpr uint32_t kStages = 8;             // of a CTA, at most
constexpr uint32_t kSmem = 200 * 1024;      // stages of all CTAs of an SM
constexpr uint32_t kSmSmem = 228 * 1024;    // all shared memory of an SM
constexpr uint32_t kReserved = 1024;        // of it, each CTA's beside what its kernel asks for

struct Plan {
    uint32_t nch, threads, ctas, stages, smem;       // ctas: of an SM; 0: no ring for these rows
};

// Chunks (vec): one a thread up to `one` columns, two up to 512 threads, then four.  Elements: 8 a thread up to
// `one` columns, then 16.  Rows of one warp are left to the other forms.  threads: of an SM with one, two
// and four chunks (what the registers allow), in as many CTAs, fewer where three stages each would not
// fit, but `least` all the same where two would; then as many stages as fit, but no more than `stages`
// where an SM has four CTAs or more.  stage: bytes of one; own: of the kernel's shared memory beside the stages.
// Measured: the forward pass of 20000 x 5001 (f32) takes 279 us with one CTA of five stages, 211 with two of two;
// the backward pass of 4000 x 4096 (f32) 49 us with one, 53 with two.
// two: columns of at most two chunks a thread.
inline Plan plan(uint32_t cols, bool vec, uint64_t stage, uint32_t own, uint32_t one, const uint32_t (&threads)[3], uint32_t least,
                 uint32_t stages, uint32_t two = 16 * kThreads) {
    Plan g{};
    if (2 * stage > kSmem) return g;
    const uint32_t bytes = (uint32_t)stage;
    uint32_t i = 0;
    for (; i < (vec ? 3 : 2); ++i) {
        g.nch = 1u << i;
        g.threads = ((cols + 8 * g.nch - 1) / (8 * g.nch) + 31) / 32 * 32;
        if (g.threads <= kThreads && cols <= (i == 0 ? one : i == 1 ? two : ~0u)) break;
    }
    if (g.threads < 64 || g.threads > kThreads) return {};
    auto fit = [&](uint32_t ctas, uint32_t n) {
        return ctas * n * bytes <= kSmem && ctas * (n * bytes + own + kReserved) <= kSmSmem;
    };
    g.ctas = std::min(std::max(threads[i] / g.threads, 1u), 16u);
    while (g.ctas > 1 && !fit(g.ctas, 3) && !(g.ctas <= least && fit(g.ctas, 2))) --g.ctas;
    g.stages = g.ctas >= 4 ? stages : kStages;
    while (g.stages > 2 && !fit(g.ctas, g.stages)) --g.stages;
    g.smem = g.stages * bytes;
    return g;
}

}  // namespace ring
}  // namespace dtt
