// Gated delta rule, what a chunk needs before the states walk: its decays, M and the inverse
// T of the unit lower triangular I + A (delta.h has the formulas).
//
// A wave takes one (batch, chunk, group) and a run of the group's heads, alone: no barrier. The
// products k_i . k_j and q_i . k_j do not depend on the head and stay in registers, the ten 16x16
// tiles on and below the diagonal each.
//
// Decays. The exponents are summed in 64 bits and kept as two floats, so that G_i - G_j of
// neighbours keeps its digits however far the chunk has decayed, a decay of minus infinity included
// (held at 2^-1024, which is 0 in fp32).
//
// The inverse, in fp32: the four diagonal blocks by forward substitution, a lane a column of a
// block (no powers of A, whose entries can grow to binomials); then from the diagonal outwards
//     T_ij^T = -T_jj^T sum_{j < k <= i} A_kj^T T_ik^T
// on the fp32 matrix cores. In step s of a 16x16x4 product slot group g carries row 4 g + s, which is
// register s of an accumulator tile: tiles of A, of T^T and the partial sums are operands as they
// stand. T^T in accumulators is T as the walk's operand.
//
// Bound by the matrices' way to memory, 24 KiB a head (backward 36): at 32768 tokens of 80 heads
// 1.0 GB in 215 us, 4.8 TB/s (644 us with a workgroup a chunk, its waves waiting at barriers); backward at
// 16384 tokens of 48 heads 0.47 GB in 100 to 108 us.
#include <type_traits>

#include "delta.h"

namespace ssd {

constexpr int kBlockLd = 20, kBlockStride = 16 * kBlockLd + 4;  // 16x16 blocks in LDS, four at a time

// acc += X^T Y for tiles X (rows k, columns: rows of the result) and Y (rows k, columns).
__device__ __forceinline__ void mm16(f32x4& acc, const f32x4& x, const f32x4& y) {
#pragma unroll
    for (int s = 0; s < 4; ++s) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(x[s], y[s], acc, 0, 0, 0);
}
__device__ __forceinline__ void wave_lds_fence() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

template <typename T, int S, bool BWD>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(2, 2))) void delta_prep_kernel(
    const T* __restrict__ k, const T* __restrict__ q, const T* __restrict__ beta,
    const float* __restrict__ gl, float* __restrict__ scal, char* __restrict__ matT,
    char* __restrict__ matM, char* __restrict__ matTt, int L, int H, int ngroups, int nC, int hb, long tasks) {
    __shared__ __align__(16) float blocks[4][4 * kBlockStride], tok[4][3][kDeltaC];
    constexpr int KN = S < 32 ? 16 : 32, NK = S < 32 ? 1 : S / 32;
    const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), c = lane & 15, g = lane >> 4;
    const int hpg = H / ngroups, nhb = hpg / hb;
    long id = (long)xcd_remap(blockIdx.x, gridDim.x) * 4 + wv;
    if (id >= tasks) return;
    const int hblk = (int)(id % nhb);
    id /= nhb;
    const int grp = (int)(id % ngroups);
    id /= ngroups;
    const int ch = (int)(id % nC), b = (int)(id / nC);
    const int t0 = ch * kDeltaC, valid = min(kDeltaC, L - t0);
    const size_t ld = (size_t)ngroups * S;
    const T* kc = k + ((size_t)b * L + t0) * ld + (size_t)grp * S;
    const T* qc = q + ((size_t)b * L + t0) * ld + (size_t)grp * S;
    float* blk = blocks[wv];
    float *ghi = tok[wv][0], *glo = tok[wv][1], *bts = tok[wv][2];

    // kk[i][j]: rows i, columns j. qk: backward the same; forward rows j, columns i.
    f32x4 kk[4][4], qk[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j <= i; ++j) kk[i][j] = qk[i][j] = kZero4;
#pragma unroll
    for (int s = 0; s < NK; ++s) {
        Frag<T> kf[4], qf[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            kf[t] = row_frag_in<KN>(kc + 32 * s, ld, 16 * t + c, valid, g);
            qf[t] = row_frag_in<KN>(qc + 32 * s, ld, 16 * t + c, valid, g);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j <= i; ++j) {
                mma(kk[i][j], kf[i], kf[j]);
                if (BWD) mma(qk[i][j], qf[i], kf[j]);
                else mma(qk[i][j], kf[j], qf[i]);
            }
    }

    for (int hh = 0; hh < hb; ++hh) {
        const int h = grp * hpg + hblk * hb + hh;
        const size_t bhc = ((size_t)b * H + h) * nC + ch;
        char *mT = matT + bhc * kDeltaMatBytes, *mM = matM + bhc * kDeltaMatBytes;
        {
            double x = 0.0;
            float bt = 0.f;
            if (lane < valid) {
                const size_t at = ((size_t)b * L + t0 + lane) * H + h;
                x = (double)gl[at] * 1.4426950408889634;
                x = x < -1024.0 ? -1024.0 : x;
                bt = to_f32(beta[at]);
            }
#pragma unroll
            for (int off = 1; off < 64; off <<= 1) {
                const double y = __shfl_up(x, off);
                if (lane >= off) x += y;
            }
            const double last = __shfl(x, 63);
            const float hi = (float)x;
            ghi[lane] = hi;
            glo[lane] = (float)(x - (double)hi);
            bts[lane] = bt;
            float* sc = scal + bhc * kDeltaScal;
            sc[lane] = exp2_fast(hi);
            sc[kDeltaC + lane] = exp2_fast((float)(last - x));
            sc[2 * kDeltaC + lane] = bt;
            if (BWD) ((double*)(sc + 3 * kDeltaC))[lane] = x;
        }
        wave_lds_fence();
        // A in rows i (diagonal blocks to LDS), M in its own order
        float ch4[4], cl4[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            ch4[t] = ghi[16 * t + c];
            cl4[t] = glo[16 * t + c];
        }
        f32x4 A[4][4], M[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const f32x4 rh = ld4(ghi + 16 * i + 4 * g), rl = ld4(glo + 16 * i + 4 * g), rb = ld4(bts + 16 * i + 4 * g);
#pragma unroll
            for (int j = 0; j <= i; ++j)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float dec = exp2_fast((rh[r] - ch4[j]) + (rl[r] - cl4[j]));
                    const bool below = j < i || c < 4 * g + r;
                    A[i][j][r] = below ? rb[r] * dec * kk[i][j][r] : 0.f;
                    if (BWD) M[i][j][r] = j < i || c <= 4 * g + r ? dec * qk[i][j][r] : 0.f;
                }
            // M and its rows j: this row tile against the column tiles i' >= i
            if (!BWD) {
#pragma unroll
                for (int i2 = i; i2 < 4; ++i2)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const float dec = exp2_fast((ch4[i2] - rh[r]) + (cl4[i2] - rl[r]));
                        M[i2][i][r] = i < i2 || 4 * g + r <= c ? dec * qk[i2][i][r] : 0.f;
                    }
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) blk[i * kBlockStride + (4 * g + r) * kBlockLd + c] = A[i][i][r];
        }
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                if (!BWD && 2 * x <= t)
                    store_tile(mM, lower_tile(t, x), lane, make_wide<T>(M[t][2 * x], 2 * x + 1 <= t ? M[t][2 * x + 1 <= t ? 2 * x + 1 : 0] : kZero4));
                if (BWD && 2 * x + 1 >= t)
                    store_tile(mM, upper_tile(t, x), lane, make_wide<T>(2 * x >= t ? M[2 * x >= t ? 2 * x : 3][t] : kZero4, M[2 * x + 1][t]));
            }
        wave_lds_fence();
        // diagonal blocks: slot group g solves block g, lane c its column c
        {
            const float* Ad = blk + g * kBlockStride;
            float t[16];
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                float s = r == c ? 1.f : 0.f;
#pragma unroll
                for (int j4 = 0; j4 < (r + 3) / 4; ++j4) {
                    const f32x4 a = ld4(Ad + r * kBlockLd + 4 * j4);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (4 * j4 + e < r) s -= a[e] * t[4 * j4 + e];
                }
                t[r] = s;
            }
            wave_lds_fence();
#pragma unroll
            for (int r = 0; r < 16; ++r) blk[g * kBlockStride + r * kBlockLd + c] = t[r];
        }
        wave_lds_fence();
        f32x4 Tt[4][4], Td[4];  // T^T: rows j, columns i; the diagonal blocks of T
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            Tt[i][i] = ld4(blk + i * kBlockStride + c * kBlockLd + 4 * g);
#pragma unroll
            for (int r = 0; r < 4; ++r) Td[i][r] = blk[i * kBlockStride + (4 * g + r) * kBlockLd + c];
        }
#pragma unroll
        for (int d = 1; d < 4; ++d)
#pragma unroll
            for (int j = 0; j + d < 4; ++j) {
                const int i = j + d;
                f32x4 p = kZero4;
#pragma unroll
                for (int x = j + 1; x <= i; ++x) mm16(p, A[x][j], Tt[i][x]);
                f32x4 o = kZero4;
                mm16(o, Td[j], p);
                Tt[i][j] = -o;
            }
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int t = 0; t < 4; ++t)
                if (2 * x <= t)
                    store_tile(mT, lower_tile(t, x), lane, make_wide<T>(Tt[t][2 * x], 2 * x + 1 <= t ? Tt[t][2 * x + 1 <= t ? 2 * x + 1 : 0] : kZero4));
        if constexpr (BWD) {
            // the same tiles turned over: rows i, columns j
            wave_lds_fence();
#pragma unroll
            for (int i = 1; i < 4; ++i) {
#pragma unroll
                for (int j = 0; j < i; ++j) *(f32x4*)(blk + j * kBlockStride + c * kBlockLd + 4 * g) = Tt[i][j];
                wave_lds_fence();
#pragma unroll
                for (int j = 0; j < i; ++j)
#pragma unroll
                    for (int r = 0; r < 4; ++r) Tt[i][j][r] = blk[j * kBlockStride + (4 * g + r) * kBlockLd + c];
                wave_lds_fence();
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) Tt[i][i] = Td[i];
            char* mTt = matTt + bhc * kDeltaMatBytes;
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int t = 0; t < 4; ++t)
                    if (2 * x + 1 >= t)
                        store_tile(mTt, upper_tile(t, x), lane, make_wide<T>(2 * x >= t ? Tt[2 * x >= t ? 2 * x : 3][t] : kZero4, Tt[2 * x + 1][t]));
        }
        wave_lds_fence();
    }
}

template <typename T, bool BWD>
static hipError_t prep_by_s(const DeltaArgs& a, const Dims& d, hipStream_t stream) {
    const int nC = (d.seqlen + kDeltaC - 1) / kDeltaC, hpg = d.nheads / d.ngroups, hb = delta_prep_heads(d);
    const long tasks = (long)d.batch * nC * d.ngroups * (hpg / hb);
    auto go = [&](auto s) {
        delta_prep_kernel<T, decltype(s)::value, BWD><<<dim3((unsigned)((tasks + 3) / 4)), 256, 0, stream>>>(
            (const T*)a.k, (const T*)a.q, (const T*)a.beta, a.g, a.scal, a.matT, a.matM, a.matTt,
            d.seqlen, d.nheads, d.ngroups, nC, hb, tasks);
        return hipGetLastError();
    };
    switch (d.dstate) {
        case 16: return go(std::integral_constant<int, 16>{});
        case 32: return go(std::integral_constant<int, 32>{});
        case 64: return go(std::integral_constant<int, 64>{});
        case 128: return go(std::integral_constant<int, 128>{});
        case 256: return go(std::integral_constant<int, 256>{});
    }
    return hipErrorInvalidValue;
}

hipError_t launch_delta_prep(int in_dtype, bool backward, const DeltaArgs& a, const Dims& d,
                             hipStream_t stream) {
    if (in_dtype == kBF16)
        return backward ? prep_by_s<bf16, true>(a, d, stream) : prep_by_s<bf16, false>(a, d, stream);
    return backward ? prep_by_s<float, true>(a, d, stream) : prep_by_s<float, false>(a, d, stream);
}

}  // namespace ssd
