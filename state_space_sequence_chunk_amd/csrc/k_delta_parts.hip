// Gated delta rule, plans shared by the host and the kernels, and the sums of dk and dq over the parts of
// a group's heads, in their order.
#include <algorithm>

#include "delta.h"

namespace ssd {

__global__ __launch_bounds__(256) void delta_parts_kernel(const float* __restrict__ dkp,
                                                          const float* __restrict__ dqp,
                                                          float* __restrict__ dk, float* __restrict__ dq,
                                                          size_t n4, int parts) {
    const size_t at = (size_t)blockIdx.x * 256 + threadIdx.x;
    if (at >= n4) return;
    f32x4 x = ld4(dkp + at * 4), y = ld4(dqp + at * 4);
    for (int p = 1; p < parts; ++p) {
        x += ld4(dkp + (p * n4 + at) * 4);
        y += ld4(dqp + (p * n4 + at) * 4);
    }
    *(f32x4*)(dk + at * 4) = x;
    *(f32x4*)(dq + at * 4) = y;
}

// Computing waves of a walk's workgroup, each with 16 rows of the state: four, or fewer where the workgroups
// still find a compute unit each. The waves of a workgroup read the same tiles from LDS, which holds
// four of them up.
int delta_waves(long heads, int rows) {
    const long slices = heads * (rows / 16);
    int nw = std::min(4, rows / 16);
    while (nw > 1 && slices / (nw / 2) <= 256) nw /= 2;
    return nw;
}

// Segments cost a first walk of P + S rows instead of none and a carry, and let the walk for y run side by
// side. Both plans are timed by the workgroups that the walks launch: 256 are walked at once (a second one on
// a compute unit takes about as long again), a chunk after another. The times of a chunk, in microseconds, are
// lines through those measured at dstate 16 to 256, headdim 16, 64 and 128, 2 to 96 heads, 2048 to 16384 tokens,
// both types and every count of segments (6% off on average, the calls' times and prep's included). At those 810
// shapes the plan taken is 2% slower on average than the best one (24% at worst) and takes 0.61 of one
// segment's time (1.09 at worst). 65536 tokens of 8 heads 64 x 128, bf16: 496 us in one and 307 in 7 segments;
// 16384 tokens of 48 heads 16 x 256: 924 us in one and 1076 in 3 segments.
DeltaSegs delta_segments(int in_dtype, const Dims& d) {
    const bool narrow = in_dtype == kBF16;
    const long nC = (d.seqlen + kDeltaC - 1) / kDeltaC, heads = (long)d.batch * d.nheads;
    const int P = d.headdim, S = d.dstate;
    const double first = narrow ? 0.42 + 0.005 * S : 1.4 + 0.02 * S, out = narrow ? 0.94 + 0.007 * S : 1.85 + 0.049 * S;
    // microseconds a chunk for `rows` rows in all, nw waves a workgroup
    auto chunk_time = [&](double one, long rows, int nw) {
        const long wgs = rows / (16 * nw);
        return one * (1 + (narrow ? 0.11 : 0.04) * (nw - 1)) * ((wgs + 255) / 256 + (narrow ? 0.0013 : 0.002) * S * wgs / 256);
    };
    DeltaSegs best = {1, kDeltaNoSegments};
    double least = 0.93 * nC * chunk_time(out, heads * P, delta_waves(heads, P));
    for (long n = 3; n <= 16 && n * 8 <= nC; ++n) {
        const long chunks = (nC + n - 1) / n, nseg = (nC + chunks - 1) / chunks;
        const double t = chunks * (chunk_time(first, heads * ((nseg - 1) * P + (nseg - 2) * S), delta_waves(heads * (nseg - 1), delta_first_rows(d))) +
                                   chunk_time(out, heads * nseg * P, delta_waves(heads * nseg, P))) +
                         6 + 0.02 * S * nseg;
        if (t < least) {
            least = t;
            best = {(int)nseg, (int)chunks};
        }
    }
    return best;
}

// The largest divisor of the group's heads that leaves two rounds of eight waves a compute unit.
int delta_prep_heads(const Dims& d) {
    const int nC = (d.seqlen + kDeltaC - 1) / kDeltaC, hpg = d.nheads / d.ngroups;
    int hb = 1;
    for (int n = 1; n <= hpg; ++n)
        if (hpg % n == 0 && (long)d.batch * nC * d.ngroups * (hpg / n) >= 4096) hb = n;
    return hb;
}

// As many parts as give four workgroups a compute unit, at most one for every head.
int delta_bwd_parts(const Dims& d) {
    const long base = (long)d.batch * ((d.seqlen + kDeltaC - 1) / kDeltaC) * d.ngroups;
    const long want = base > 0 ? (1024 + base - 1) / base : 1;
    return (int)std::max(1L, std::min((long)(d.nheads / d.ngroups), want));
}

hipError_t launch_delta_grads(int in_dtype, const DeltaArgs& a, const Dims& d, hipStream_t stream) {
    const hipError_t e = in_dtype == kBF16 ? launch_delta_grads_bf16(a, d, stream) : launch_delta_grads_f32(a, d, stream);
    const int parts = delta_bwd_parts(d);
    if (e != hipSuccess || parts == 1) return e;
    const size_t n4 = (size_t)d.batch * d.seqlen * d.ngroups * d.dstate / 4;
    delta_parts_kernel<<<dim3((unsigned)((n4 + 255) / 256)), 256, 0, stream>>>(a.dkp, a.dqp, a.dk, a.dq, n4, parts);
    return hipGetLastError();
}

}  // namespace ssd
