// Gated delta rule, token by token: the decode step, and the forward pass of short sequences.
//
//     a = exp(g),  u = beta (v - a H k),  H <- a H + u k^T,  y = scale H q
// Both products with the old state are taken at once, H k and H q, with k . q beside them:
//     y = scale (a (H q) + u (k . q)).
//
// gfx950 mapping, as the framework's other decode step: the state is read and written once (8
// bytes an element against 6 flops a token), so one token costs a round trip to memory. A
// thread owns 4 consecutive columns of up to ROWS rows and keeps them for all tokens; the S/4
// threads of a row are neighbours in one wave and sum by a butterfly. One token for 96 sequences of 32
// heads of 128 x 128: 0.40 GB in 71 us, 5.6 TB/s; for 2 of 80 heads of 64 x 128 (10 MB): 5.0 us.
#include <algorithm>
#include <type_traits>

#include "delta.h"

namespace ssd {

constexpr int kStepThreads = 256;

template <typename T> __device__ __forceinline__ f32x4 load4(const T* p);
template <> __device__ __forceinline__ f32x4 load4<float>(const float* p) { return *(const f32x4*)p; }
template <> __device__ __forceinline__ f32x4 load4<bf16>(const bf16* p) {
    const bf16x4 v = *(const bf16x4*)p;
    return f32x4{(float)v[0], (float)v[1], (float)v[2], (float)v[3]};
}
__device__ __forceinline__ float dot4(const f32x4& a, const f32x4& b) {
    return a[0] * b[0] + a[1] * b[1] + a[2] * b[2] + a[3] * b[3];
}

template <typename T, typename TO, int S, int ROWS>
__global__ __launch_bounds__(kStepThreads) void delta_recurrent_kernel(
    const T* __restrict__ v, const float* __restrict__ gl, const T* __restrict__ beta,
    const T* __restrict__ k, const T* __restrict__ q, const float* h0, float* out_state,
    TO* __restrict__ y, float scale, int L, int H, int P, int ngroups, int vpw) {
    constexpr int RL = S / 4;  // lanes a row
    const int per_bh = P * RL / vpw;
    const int bh = blockIdx.x / per_bh, v0 = (blockIdx.x % per_bh) * vpw;
    const int b = bh / H, h = bh % H, grp = h / (H / ngroups);
    const int sc = (threadIdx.x % RL) * 4;
    const size_t at = (size_t)bh * P * S;

    // vpw is a multiple of 64: a wave is wholly inside or outside the slice for a given j
    f32x4 st[ROWS];
#pragma unroll
    for (int j = 0; j < ROWS; ++j) {
        const int e = threadIdx.x + kStepThreads * j;
        st[j] = h0 && e < vpw ? *(const f32x4*)(h0 + at + (size_t)(v0 + e) * 4) : kZero4;
    }
    for (int t = 0; t < L; ++t) {
        const size_t tok = (size_t)b * L + t;
        const f32x4 kv = load4(k + (tok * ngroups + grp) * S + sc), qv = load4(q + (tok * ngroups + grp) * S + sc);
        const float a = exp2_fast(gl[tok * H + h] * kLog2e), bt = to_f32(beta[tok * H + h]);
        float kq = dot4(kv, qv);
#pragma unroll
        for (int off = RL / 2; off > 0; off >>= 1) kq += __shfl_xor(kq, off, RL);
#pragma unroll
        for (int j = 0; j < ROWS; ++j) {
            const int e = threadIdx.x + kStepThreads * j;
            if (e < vpw) {
                const int p = (v0 + e) / RL;
                const size_t vat = (tok * H + h) * P + p;
                const float x = to_f32(v[vat]);
                float hk = dot4(st[j], kv), hq = dot4(st[j], qv);
#pragma unroll
                for (int off = RL / 2; off > 0; off >>= 1) {
                    hk += __shfl_xor(hk, off, RL);
                    hq += __shfl_xor(hq, off, RL);
                }
                const float u = bt * (x - a * hk);
                st[j] = st[j] * a + kv * u;
                if (threadIdx.x % RL == 0) y[vat] = from_f32<TO>(scale * (a * hq + u * kq));
            }
        }
    }
    if (out_state) {
#pragma unroll
        for (int j = 0; j < ROWS; ++j) {
            const int e = threadIdx.x + kStepThreads * j;
            if (e < vpw) *(f32x4*)(out_state + at + (size_t)(v0 + e) * 4) = st[j];
        }
    }
}

namespace {
template <typename T, typename TO>
hipError_t recurrent(const DeltaArgs& a, const Dims& d, hipStream_t stream) {
    const int vecs = d.headdim * d.dstate / 4;  // per (batch, head)
    // two rows a thread unless that leaves fewer workgroups than compute units
    const int rows = (long)d.batch * d.nheads * vecs / (2 * kStepThreads) >= 256 ? 2 : 1;
    const int vpw = std::min(vecs, rows * kStepThreads);
    const unsigned blocks = (unsigned)((long)d.batch * d.nheads * (vecs / vpw));
    auto go = [&](auto s, auto r) {
        delta_recurrent_kernel<T, TO, decltype(s)::value, decltype(r)::value><<<dim3(blocks), kStepThreads, 0, stream>>>(
            (const T*)a.v, a.g, (const T*)a.beta, (const T*)a.k, (const T*)a.q, a.h0, a.final_state,
            (TO*)a.y, a.scale, d.seqlen, d.nheads, d.headdim, d.ngroups, vpw);
        return hipGetLastError();
    };
    auto by_rows = [&](auto s) {
        return rows == 2 ? go(s, std::integral_constant<int, 2>{}) : go(s, std::integral_constant<int, 1>{});
    };
    switch (d.dstate) {
        case 16: return by_rows(std::integral_constant<int, 16>{});
        case 32: return by_rows(std::integral_constant<int, 32>{});
        case 64: return by_rows(std::integral_constant<int, 64>{});
        case 128: return by_rows(std::integral_constant<int, 128>{});
        case 256: return by_rows(std::integral_constant<int, 256>{});
    }
    return hipErrorInvalidValue;
}
}  // namespace

hipError_t launch_delta_recurrent(int in_dtype, int out_dtype, const DeltaArgs& a, const Dims& d,
                                  hipStream_t stream) {
    if (in_dtype == kBF16)
        return out_dtype == kBF16 ? recurrent<bf16, bf16>(a, d, stream) : recurrent<bf16, float>(a, d, stream);
    return recurrent<float, float>(a, d, stream);
}

// The loop's time is its steps', one behind the other: 0.5 us and 0.53 for a million elements of the states. A
// chunk takes its launches and its way through both kernels whatever its tokens, and then its matrices and
// states. Lines through calls of 8 to 48 tokens with 2 states to 96 sequences of 32 heads, 16 x 16 to 128 x 256, both types, through
// the binding: the choice is 0.7% slower there than the better of both on average (33% at worst). 16 tokens in bf16
// token by token and by chunks: 160 states of 64 x 128 19 and 21 us, 96 sequences of 32 heads of 128 x 256
// 948 and 353.
bool delta_recurrent_preferred(int in_dtype, const Dims& d) {
    const double heads = (double)d.batch * d.nheads, million = heads * d.headdim * d.dstate * 1e-6;
    const double chunk = in_dtype == kBF16 ? 18 + 0.008 * heads + 2.5 * million
                                           : 20 + 0.1 * d.dstate + 0.02 * heads + 5.5 * million;
    return d.seqlen <= kDeltaC && d.seqlen * (0.5 + 0.53 * million) <= chunk;
}

}  // namespace ssd
