// Gated delta rule, the gradients of each chunk once both walks have passed (delta.h): with H
// the state entering the chunk, E the gradient at its end, U and N of the walks, Z = scale dY,
//     dM = lower(Z U^T),  dA = -strictly lower(N U^T),  W = dM o D,  B = dA o beta_i D
//     dQ = e^G o (Z H) + W K
//     dK = (e^{G_C - G} o U) E - (beta e^G o N) H + W^T Q + (B + B^T) K
//     dbeta_i = N_i . V_i - e^{G_i} (N H)_i . k_i + sum_j dA_ij D_ij k_i . k_j
//     dg_t = e^{G_C} <H, E> + sum_{j < t} s_j + sum_{i >= t} (r_i + x_i)
// where s_j = e^{G_C - G_j} (U E)_j . k_j, r_i = e^{G_i} ((Z H)_i . q_i - beta_i (N H)_i . k_i),
// X = dA o A + dM o M off its diagonal and x_i its row sum less its column sum: both sums are
// of the same fp32 values, so that the pairs on one side of t cancel to fp32 rounding.
//
// One workgroup takes one (batch, chunk, group) and a part of the group's heads, which it adds
// up in registers; wave w owns the 16 tokens of tile w and all of S. K and Q stay in LDS for all
// heads. What the walks left (planes of H, E and of the transposed U, N, Z) comes straight from
// memory into one region of LDS: first Z and U, then N for Z, then H, then E, up to 64 of the P rows
// at a time (everything is a sum over P). The bound is that traffic, 4 (2 S + 3 * 64) P bytes a head,
// and the waits for it: a workgroup's next piece has no room while the last one is read, so that only the
// other workgroup of the compute unit (two fit at dstate 128) keeps memory busy. 16384 tokens of 48 heads of
// 64 x 128 in bf16: 1.4 GB in 433 to 504 us (2801 read from memory where used, 1300 through LDS, 724 with
// loads beside products, 665 with products in groups of tiles, 509 with 16 bytes of a lane in scratch memory).
#pragma once

#include "delta_walk.h"

namespace ssd {

// Sum over the 16 lanes of a row, or over the four slot groups of a column.
__device__ __forceinline__ float sum16(float v) {  // rotations within the row of 16 lanes
    v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x128, 0xf, 0xf, true));
    v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x124, 0xf, 0xf, true));
    v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x122, 0xf, 0xf, true));
    v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x121, 0xf, 0xf, true));
    return v;
}
__device__ __forceinline__ float sum_groups(float v) {
    v += __shfl_xor(v, 16);
    return v + __shfl_xor(v, 32);
}

// Planes (store_planes) of PB rows of N values in LDS, read by columns: a Wide fragment whose lane
// holds a column of tile t and, in slot v of group g, one of the rows 32 x .. 32 x + 31 (slot_row; 16
// rows: the upper slots are zero). STATE: the column is state column 16 t + c, and bf16's
// transposing reads meet no bank conflict; else (U, N, Z: columns are tokens) it is token 16 t + c,
// whose place kmap has moved, with two-way conflicts.
template <typename T, int PB, int N, bool STATE> struct Planes;
template <int PB, int N, bool STATE> struct Planes<bf16, PB, N, STATE> {
    static constexpr int RB = N < 32 ? 32 : 64, PLANE = PB * N * 2, BYTES = 2 * PLANE, BLOCK = PB * RB;
    uint32_t at[2][2];
    static __device__ __forceinline__ int slot_row(int g, int v) { return PB >= 32 ? 8 * g + v : 4 * g + v; }
    __device__ __forceinline__ explicit Planes(int lane) {
        const int s = lane & 15, g = lane >> 4, q = s & 3;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int o = 0; o < 2; ++o) {
                const int r = (PB >= 32 ? 8 * g + 4 * h : 4 * g) + (s >> 2);
                at[h][o] = N < 32 ? r * RB + 8 * q
                           : STATE ? r * RB + (((2 * o + (q >> 1)) ^ plane_swz(r)) << 4) + 8 * (q & 1)
                                   : r * RB + ((q ^ plane_swz(r)) << 4) + 8 * o;
                opaque(at[h][o]);
            }
    }
    // rows p0 .. p0 + PB of planes of P rows
    static __device__ __forceinline__ void stage(char* t, const char* src, int P, int p0, int wave, int lane) {
        const BufRsrc r = make_rsrc(src, (uint32_t)(P * N * 4));
        uint32_t l16 = (uint32_t)(lane * 16);
        opaque(l16);
#pragma unroll
        for (int k = 0; k < (BYTES / 1024 + 3) / 4; ++k) {
            const int u = k * 4 + wave;
            if (BYTES / 1024 % 4 == 0 || u < BYTES / 1024) {
                // (a block of less than 1 KiB is that of all P rows)
                const int n = u * 1024, from = BLOCK % 1024 == 0 ? n / BLOCK * (P * RB) + p0 * RB + n % BLOCK : n;
                __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)(t + u * 1024), 16,
                                                         l16 + (uint32_t)from, 0, 0, 0);
            }
        }
    }
    static __device__ __forceinline__ bf16x4 tr(const char* p) {
        return __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf16x4*)(__attribute__((address_space(3))) char*)p);
    }
    // tile 2 * pair + o
    __device__ __forceinline__ Wide<bf16> cols(const char* t, int x, int pair, int o) const {
        Wide<bf16> w;
        const char* p = t + pair * BLOCK + 32 * x * RB;
        const bf16x4 z = {0, 0, 0, 0};
        w.hi = __builtin_shufflevector(tr(p + at[0][o]), PB >= 32 ? tr(p + at[1][o]) : z, 0, 1, 2, 3, 4, 5, 6, 7);
        p += PLANE;
        w.lo = __builtin_shufflevector(tr(p + at[0][o]), PB >= 32 ? tr(p + at[1][o]) : z, 0, 1, 2, 3, 4, 5, 6, 7);
        return w;
    }
    static __device__ __forceinline__ float value(const Wide<bf16>& w, int v) { return (float)w.hi[v] + (float)w.lo[v]; }
};
template <int PB, int N, bool STATE> struct Planes<float, PB, N, STATE> {
    static constexpr int RB = 64, PLANE = PB * N * 4, BYTES = PLANE, BLOCK = PB * RB;
    uint32_t at;
    static __device__ __forceinline__ int slot_row(int g, int v) { return g + 4 * v; }
    __device__ __forceinline__ explicit Planes(int lane) {
        at = (lane >> 4) * RB + 4 * (lane & 15);
        opaque(at);
    }
    static __device__ __forceinline__ void stage(char* t, const char* src, int P, int p0, int wave, int lane) {
        const BufRsrc r = make_rsrc(src, (uint32_t)(P * N * 4));
        uint32_t l16 = (uint32_t)(lane * 16);
        opaque(l16);
#pragma unroll
        for (int k = 0; k < (BYTES / 1024 + 3) / 4; ++k) {
            const int u = k * 4 + wave;
            if (BYTES / 1024 % 4 == 0 || u < BYTES / 1024) {
                // (a block of less than 1 KiB is that of all P rows)
                const int n = u * 1024, from = BLOCK % 1024 == 0 ? n / BLOCK * (P * RB) + p0 * RB + n % BLOCK : n;
                __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)(t + u * 1024), 16,
                                                         l16 + (uint32_t)from, 0, 0, 0);
            }
        }
    }
    __device__ __forceinline__ Wide<float> cols(const char* t, int x, int pair, int o) const {
        Wide<float> w;
        const char* p = t + (2 * pair + o) * BLOCK + 32 * x * RB + at;
#pragma unroll
        for (int v = 0; v < 8; ++v) w.v[v] = PB >= 32 || v < 4 ? *(const float*)(p + 4 * v * RB) : 0.f;
        return w;
    }
    static __device__ __forceinline__ float value(const Wide<float>& w, int v) { return w.v[v]; }
};

template <typename T, int S, int P> struct GradsCfg {
    static constexpr int PB = P < 64 ? P : 64;  // rows of the state at a time
    using ST = Planes<T, PB, S, true>;
    using TT = Planes<T, PB, kDeltaC, false>;
    static constexpr int KB = kDeltaC * S * (int)sizeof(T), REGION = 2 * TT::BYTES > ST::BYTES ? 2 * TT::BYTES : ST::BYTES;
    static constexpr int SMALL = 5888;
    // K and Q are read from memory where they do not fit beside the region
    static constexpr bool KQ = 2 * KB + REGION + SMALL <= 163840;
    static constexpr int LDS = (KQ ? 2 * KB : 0) + REGION;
    // Two workgroups a compute unit, each with half the registers, where K and Q are in LDS too. Where they are
    // not (fp32, dstate 256) their fragments are formed from memory and half the registers would put 750 to 980
    // values in scratch memory: the backward pass of 2 x 4096 tokens of 24 heads takes 3632 us so and 3088 with
    // one workgroup at headdim 32, 3914 and 3333 at 64.
    static constexpr bool PAIR = KQ && P <= 64 && 2 * (LDS + SMALL) <= 163840;
};

template <typename T, int S, int P>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(GradsCfg<T, S, P>::PAIR ? 2 : 1, 2))) void delta_grads_kernel(
    const T* __restrict__ k, const T* __restrict__ q, const T* __restrict__ v,
    const float* __restrict__ scal, const char* __restrict__ Hc, const char* __restrict__ Ec,
    const char* __restrict__ Ut, const char* __restrict__ Nt, const char* __restrict__ Zt,
    float* __restrict__ dg, float* __restrict__ dbeta, float* __restrict__ dk, float* __restrict__ dq,
    int L, int H, int ngroups, int nC, int parts) {
    using Cfg = GradsCfg<T, S, P>;
    using ST = typename Cfg::ST;
    using TT = typename Cfg::TT;
    constexpr int KN = S < 32 ? 16 : 32, NK = S < 32 ? 1 : S / 32, NT = S / 16, PB = Cfg::PB;
    constexpr int NP = PB < 32 ? 1 : PB / 32, NB = P / PB;
    constexpr int TG = NT < 4 ? NT : 4, TH = NT < 2 ? NT : 2;  // tiles whose products run side by side
    __shared__ __align__(1024) char kq[Cfg::KQ ? 2 * Cfg::KB : 16];
    __shared__ __align__(1024) char region[Cfg::REGION];
    __shared__ __align__(1024) float sc[512];  // the head's scalars: kDeltaScal of them
    const double* Gs = (const double*)(sc + 3 * kDeltaC);
    __shared__ __align__(16) float rxs[2][2][kDeltaC], sss[2][kDeltaC], cxs[2][4][kDeltaC], edges[2][4];  // (two heads)
    const int tid = threadIdx.x, lane0 = tid & 63;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int hpg = H / ngroups;
    int id = xcd_remap(blockIdx.x, gridDim.x);
    const int part = id % parts;
    id /= parts;
    const int grp = id % ngroups;
    id /= ngroups;
    const int ch = id % nC, b = id / nC, B = gridDim.x / parts / ngroups / nC;
    const int t0 = ch * kDeltaC, valid = min(kDeltaC, L - t0);
    const size_t ld = (size_t)ngroups * S, ldv = (size_t)H * P;
    const T* kc = k + ((size_t)b * L + t0) * ld + (size_t)grp * S;
    const T* qc = q + ((size_t)b * L + t0) * ld + (size_t)grp * S;
    const Tile<T, S> ad(lane0);

    if constexpr (Cfg::KQ) {
        const uint32_t bytes = (uint32_t)(((valid - 1) * ld + S) * sizeof(T));
        Tile<T, S>::template stage<4>(kq, make_rsrc(kc, bytes), (uint32_t)(ld * sizeof(T)), w, lane0);
        Tile<T, S>::template stage<4>(kq + Cfg::KB, make_rsrc(qc, bytes), (uint32_t)(ld * sizeof(T)), w, lane0);
    }
    // the state's rows, PB at a time
    auto each_block = [](auto&& f) {
        f(std::integral_constant<int, 0>{});
        if constexpr (NB > 1) f(std::integral_constant<int, 1>{});
    };
    static_assert(NB <= 2, "at most 128 rows");
    // The lane's number is asked for anew in each phase: what is formed from it is formed where it is
    // used, and held neither through all heads nor in scratch memory, whose loads would wait for those
    // to LDS before them.
    auto lane_now = [] {
        int x;
        asm volatile("v_mbcnt_lo_u32_b32 %0, -1, 0\n\tv_mbcnt_hi_u32_b32 %0, -1, %0" : "=v"(x));
        return x;
    };
    auto here = [](int x) {
        asm volatile("" : "+v"(x));
        return x;
    };
    // Sums that only the head's end reads are formed where they stand (the compiler would hold their terms
    // until then, in scratch memory).
    auto now = [](float& x) { asm volatile("" : "+v"(x)); };
    f32x4 aq[NT], ak[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) aq[t] = ak[t] = kZero4;

    // the head's scalars, Z and U
    auto first = [&](int h) {
        const size_t at = ((size_t)b * H + h) * nC + ch, rows = at * (size_t)(4 * kDeltaC * P);
        const int lane = lane_now();
        stage_flat<kDeltaScal * 4, 4>((char*)sc, scal + at * kDeltaScal, w, lane);
        TT::stage(region, Zt + rows, P, 0, w, lane);
        TT::stage(region + TT::BYTES, Ut + rows, P, 0, w, lane);
    };
    const int h_lo = grp * hpg + hpg * part / parts, h_hi = grp * hpg + hpg * (part + 1) / parts;
    for (int h = h_lo; h < h_hi; ++h) {
        const int lane = lane_now(), c = lane & 15, g = lane >> 4, own = 16 * w + c;
        const TT tp(lane);
        // fragments of K (0) and Q (1)
        auto rows_of = [&](int m, int t, int x) {
            if constexpr (Cfg::KQ) return ad.rows(kq + m * Cfg::KB, t, x);
            else return row_frag_in<KN>((m ? qc : kc) + 32 * x, ld, 16 * t + here(c), valid, g);
        };
        auto cols_of = [&](int m, int t, int x) {
            if constexpr (Cfg::KQ) return ad.plain_cols(kq + m * Cfg::KB, t, x);
            else return col_frag_in((m ? qc : kc) + 16 * t + here(c), ld, 32 * x, valid, g);
        };
        auto acc_of = [&](int m, int t) {  // this wave's rows, as an accumulator holds them
            if constexpr (Cfg::KQ) {
                return ad.acc(kq + m * Cfg::KB, t, 16 * w);
            } else {
                f32x4 f;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int i = 16 * w + 4 * here(g) + r;
                    f[r] = i < valid ? to_f32((m ? qc : kc)[(size_t)i * ld + 16 * t + c]) : 0.f;
                }
                return f;
            }
        };
        const size_t bhc = ((size_t)b * H + h) * nC + ch;
        float (&rx)[2][kDeltaC] = rxs[h & 1], (&ss)[kDeltaC] = sss[h & 1], (&cx)[4][kDeltaC] = cxs[h & 1], (&edge)[4] = edges[h & 1];
        const char* Hh = Hc + bhc * (size_t)(4 * P * S);
        const char* Eh = Ec + bhc * (size_t)(4 * P * S);
        const size_t rows = bhc * (size_t)(4 * kDeltaC * P);
        const T* vc = v + ((size_t)b * L + t0) * ldv + (size_t)h * P;
        // pairs inside the chunk. Lower: rows j of tile t <= w, columns i of this wave's tile
        // (W and B as operands with rows i). Upper: rows i of tile t >= w, columns j of this
        // wave's tile (W^T and B^T as operands with rows j).
        float nv = 0.f;  // N_i . V_i of row `own`
        Wide<T> zf[NB][NP], uf[NB][NP], nf[NB][NP];
        float xrow = 0.f, bsum = 0.f;
        {
            f32x4 ml[4], al[4], mu[4], au[4];
#pragma unroll
            for (int t = 0; t < 4; ++t) ml[t] = al[t] = mu[t] = au[t] = kZero4;
            const char *zt = region, *ut = region + TT::BYTES;
            auto own_cols = [&](const char* m, int x) { return w & 1 ? tp.cols(m, x, w >> 1, 1) : tp.cols(m, x, w >> 1, 0); };
            each_block([&](auto pb_c) {
                constexpr int pb = decltype(pb_c)::value, p0 = pb * PB;
                if (pb == 0) {
                    if (h == h_lo) first(h);
                } else {
                    TT::stage(region, Zt + rows, P, p0, w, lane);
                    TT::stage(region + TT::BYTES, Ut + rows, P, p0, w, lane);
                }
                // this wave's rows of V
                Frag<T> vf[NP];
#pragma unroll
                for (int x = 0; x < NP; ++x) {
                    const T* vr = vc + (size_t)(own < valid ? own : 0) * ldv + p0 + 32 * x;
                    if constexpr (sizeof(T) == 2 && PB >= 32) {
                        vf[x].v = *(const bf16x8*)(vr + 8 * g);
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; ++e) vf[x].v[e] = PB >= 32 || e < 4 ? vr[TT::slot_row(g, e)] : (T)0.f;
                    }
                }
                staged_barrier<0>();
#pragma unroll
                for (int x = 0; x < NP; ++x) {
                    zf[pb][x] = own_cols(zt, x);
                    uf[pb][x] = own_cols(ut, x);
                }
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                    for (int x = 0; x < NP; ++x) {
                        if (t <= w) mma(ml[t], tp.cols(ut, x, t >> 1, t & 1), zf[pb][x]);
                        if (t >= w) mma(mu[t], tp.cols(zt, x, t >> 1, t & 1), uf[pb][x]);
                    }
                }
                lds_barrier();
                TT::stage(region, Nt + rows, P, p0, w, lane);
                staged_barrier<0>();
#pragma unroll
                for (int x = 0; x < NP; ++x) {
                    nf[pb][x] = own_cols(zt, x);
#pragma unroll
                    for (int e = 0; e < (PB >= 32 ? 8 : 4); ++e)
                        nv += own < valid ? TT::value(nf[pb][x], e) * to_f32(vf[x].v[e]) : 0.f;
                }
                now(nv);
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                    for (int x = 0; x < NP; ++x) {
                        if (t <= w) mma(al[t], tp.cols(ut, x, t >> 1, t & 1), nf[pb][x]);
                        if (t >= w) mma(au[t], tp.cols(zt, x, t >> 1, t & 1), uf[pb][x]);
                    }
                }
                lds_barrier();
            });
            // the first rows of H come in beside the products with K and Q
            ST::stage(region, Hh, P, 0, w, lane);

            const double go = Gs[own];
            const float bo = sc[2 * kDeltaC + own];
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                __builtin_amdgcn_sched_barrier(0);
                f32x4 xc = kZero4;
                if (t <= w) {
                    f32x4 kk = kZero4, qk = kZero4;
#pragma unroll
                    for (int s = 0; s < NK; ++s) {
                        const Frag<T> kt = rows_of(0, t, s);
                        mma(kk, kt, rows_of(0, w, s));
                        mma(qk, kt, rows_of(1, w, s));
                    }
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int j = 16 * t + 4 * g + r;
                        const float dec = exp2_fast((float)(go - Gs[j]));
                        const float m = j <= own ? ml[t][r] * dec : 0.f;
                        const float a = j < own ? -al[t][r] * dec : 0.f;
                        ml[t][r] = m;
                        al[t][r] = a * bo;
                        const float akk = j < own ? a * kk[r] : 0.f;
                        const float x = j < own ? m * qk[r] + akk * bo : 0.f;
                        bsum += akk;
                        xrow += x;
                        xc[r] = x;
                    }
                }
#pragma unroll
                for (int r = 0; r < 4; ++r) xc[r] = sum16(xc[r]);
                if (c == 0) *(f32x4*)&cx[w][16 * t + 4 * g] = xc;
                if (t >= w) {
                    const f32x4 bi = ld4(sc + 2 * kDeltaC + 16 * t + 4 * g);
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int i = 16 * t + 4 * g + r;
                        const float dec = exp2_fast((float)(Gs[i] - go));
                        mu[t][r] = i >= own ? mu[t][r] * dec : 0.f;
                        au[t][r] = i > own ? -au[t][r] * dec * bi[r] : 0.f;
                    }
                }
            }
            xrow = sum_groups(xrow);
            bsum = sum_groups(bsum);
            now(xrow);
            now(bsum);
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const Wide<T> lw = make_wide<T>(ml[2 * s], ml[2 * s + 1]), uw = make_wide<T>(mu[2 * s], mu[2 * s + 1]);
                // B and B^T meet the same rows of K: their sum is one operand
                const Wide<T> bw = make_wide<T>(al[2 * s] + au[2 * s], al[2 * s + 1] + au[2 * s + 1]);
#pragma unroll
                for (int t4 = 0; t4 < NT; t4 += TG) {
                    __builtin_amdgcn_sched_barrier(0);
                    Frag<T> kf[TG], qf[TG];
#pragma unroll
                    for (int t = 0; t < TG; ++t) {
                        kf[t] = cols_of(0, t4 + t, s);
                        qf[t] = cols_of(1, t4 + t, s);
                    }
#pragma unroll
                    for (int part = 0; part < Parts<T>::IW; ++part) {
#pragma unroll
                        for (int t = 0; t < TG; ++t) mma_part(ak[t4 + t], bw, kf[t], part);
                        if (2 * s <= w) {
#pragma unroll
                            for (int t = 0; t < TG; ++t) mma_part(aq[t4 + t], lw, kf[t], part);
                        }
                        if (2 * s + 1 >= w) {
#pragma unroll
                            for (int t = 0; t < TG; ++t) mma_part(ak[t4 + t], uw, qf[t], part);
                        }
                    }
                }
            }
        }

        __builtin_amdgcn_sched_barrier(0);
        // products with the states
        const ST sp(lane_now());
        f32x4 r_i = kZero4, nk = kZero4, s_j = kZero4;  // rows 16 w + 4 g + r
        float e2 = 0.f;                                 // <H, E>
        const float ec = sc[kDeltaC - 1];
        const f32x4 eg = ld4(sc + 16 * w + 4 * g), er = ld4(sc + kDeltaC + 16 * w + 4 * g),
                    bt = ld4(sc + 2 * kDeltaC + 16 * w + 4 * g);
        each_block([&](auto pb_c) {
            constexpr int pb = decltype(pb_c)::value;
            if (pb) ST::stage(region, Hh, P, pb * PB, w, lane);
            staged_barrier<0>();
#pragma unroll
            for (int t2 = 0; t2 < NT; t2 += TH) {
                __builtin_amdgcn_sched_barrier(0);
                f32x4 zh[TH], nh[TH];
                Wide<T> o[TH][NP];
#pragma unroll
                for (int t = 0; t < TH; ++t) {
                    zh[t] = nh[t] = kZero4;
#pragma unroll
                    for (int x = 0; x < NP; ++x) o[t][x] = sp.cols(region, x, (t2 + t) >> 1, (t2 + t) & 1);
                }
#pragma unroll
                for (int x = 0; x < NP; ++x)
#pragma unroll
                    for (int part = 0; part < Parts<T>::WW; ++part)
#pragma unroll
                        for (int t = 0; t < TH; ++t) {
                            mma_part(zh[t], zf[pb][x], o[t][x], part);
                            mma_part(nh[t], nf[pb][x], o[t][x], part);
                        }
#pragma unroll
                for (int t = 0; t < TH; ++t) {
                    zh[t] *= eg;
                    nh[t] *= eg;
                    r_i += zh[t] * acc_of(1, t2 + t);
                    nk += nh[t] * acc_of(0, t2 + t);
                    aq[t2 + t] += zh[t];
                    ak[t2 + t] -= bt * nh[t];
                }
            }
            // <H, E>: this thread's pieces of H wait in registers for E's, which lie alike
            constexpr int LINE = ST::PLANE / 4096 > 0 ? ST::PLANE / 4096 : 1, NPL = sizeof(T) == 2 ? 2 : 1;
            Vec16 hv[LINE][NPL];
            const int l16 = (w * 64 + lane) * 16;
#pragma unroll
            for (int x = 0; x < LINE; ++x)
#pragma unroll
                for (int pl = 0; pl < NPL; ++pl)
                    hv[x][pl] = *(const Vec16*)(region + pl * ST::PLANE + (l16 + 4096 * x < ST::PLANE ? l16 + 4096 * x : 0));
            lds_barrier();
            ST::stage(region, Eh, P, pb * PB, w, lane);
            staged_barrier<0>();
#pragma unroll
            for (int x = 0; x < LINE; ++x) {
                const int n = l16 + 4096 * x;
                if (n < ST::PLANE) {
                    if constexpr (sizeof(T) == 2) {
                        const bf16x8 eh = *(const bf16x8*)(region + n), el = *(const bf16x8*)(region + ST::PLANE + n);
                        const bf16x8 hh = __builtin_bit_cast(bf16x8, hv[x][0]), hl = __builtin_bit_cast(bf16x8, hv[x][1]);
#pragma unroll
                        for (int e = 0; e < 8; ++e) e2 += ((float)hh[e] + (float)hl[e]) * ((float)eh[e] + (float)el[e]);
                    } else {
                        const f32x4 e = *(const f32x4*)(region + n), a = __builtin_bit_cast(f32x4, hv[x][0]);
                        e2 += a[0] * e[0] + a[1] * e[1] + a[2] * e[2] + a[3] * e[3];
                    }
                }
            }
            now(e2);
#pragma unroll
            for (int t4 = 0; t4 < NT; t4 += TH) {
                __builtin_amdgcn_sched_barrier(0);
                f32x4 ue[TH];
                Wide<T> o[TH][NP];
#pragma unroll
                for (int t = 0; t < TH; ++t) {
                    ue[t] = kZero4;
#pragma unroll
                    for (int x = 0; x < NP; ++x) o[t][x] = sp.cols(region, x, (t4 + t) >> 1, (t4 + t) & 1);
                }
#pragma unroll
                for (int x = 0; x < NP; ++x)
#pragma unroll
                    for (int part = 0; part < Parts<T>::WW; ++part)
#pragma unroll
                        for (int t = 0; t < TH; ++t) mma_part(ue[t], uf[pb][x], o[t][x], part);
#pragma unroll
                for (int t = 0; t < TH; ++t) {
                    ue[t] *= er;
                    s_j += ue[t] * acc_of(0, t4 + t);
                    ak[t4 + t] += ue[t];
                }
            }
            lds_barrier();
        });
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            r_i[r] = sum16(r_i[r]);
            nk[r] = sum16(nk[r]);
            s_j[r] = sum16(s_j[r]);
        }
        nv = sum_groups(nv);
        e2 = sum_groups(sum16(e2));
        // per-token scalars
        const int le = lane_now(), ce = le & 15, ge = le >> 4, i0 = 16 * w + 4 * ge, oe = 16 * w + ce;
        if (le == 0) edge[w] = e2;
        if (ce == 0) {
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int i = i0 + r;
                rx[0][i] = r_i[r] - bt[r] * nk[r];
                ss[i] = s_j[r];
            }
        }
        {
            // nk of row `own` is register c % 4 of slot group c / 4
            const int from = (ce >> 2) * 16;
            const float n0 = __shfl(nk[0], from), n1 = __shfl(nk[1], from), n2 = __shfl(nk[2], from), n3 = __shfl(nk[3], from);
            const float no = (ce & 3) == 0 ? n0 : (ce & 3) == 1 ? n1 : (ce & 3) == 2 ? n2 : n3;
            if (ge == 0 && oe < valid) dbeta[((size_t)b * L + t0 + oe) * H + h] = nv - no + bsum;
        }
        if (ge == 0) rx[1][oe] = xrow;
        lds_barrier();
        if (w == (h & 3)) {  // the others go on: the next head has arrays of its own
            float after = rx[0][le] + rx[1][le], before = ss[le];
#pragma unroll
            for (int x = 0; x < 4; ++x) after -= cx[x][le];
#pragma unroll
            for (int off = 1; off < 64; off <<= 1) {
                const float x = __shfl_up(before, off), y = __shfl_down(after, off);
                if (le >= off) before += x;
                if (le + off < 64) after += y;
            }
            const float ed = (edge[0] + edge[1] + edge[2] + edge[3]) * ec;
            const float prev = __shfl_up(before, 1);
            if (le < valid) dg[((size_t)b * L + t0 + le) * H + h] = ed + (le ? prev : 0.f) + after;
        }
        if (h + 1 < h_hi) first(h + 1);
    }
    const int lane = lane_now(), c = lane & 15, g = lane >> 4;
    const size_t base = ((size_t)part * B + b) * L;  // row 0 of this part and batch row
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int i = 16 * w + 4 * g + r;
            if (i < valid) {
                const size_t at = (base + t0 + i) * ld + (size_t)grp * S + 16 * t + c;
                dq[at] = aq[t][r];
                dk[at] = ak[t][r];
            }
        }
}

template <typename T, int S> hipError_t delta_grads(const DeltaArgs& a, const Dims& d, hipStream_t stream) {
    const int nC = (d.seqlen + kDeltaC - 1) / kDeltaC, parts = delta_bwd_parts(d);
    const unsigned blocks = (unsigned)((long)d.batch * nC * d.ngroups * parts);
    auto go = [&](auto p) {
        delta_grads_kernel<T, S, decltype(p)::value><<<dim3(blocks), 256, 0, stream>>>(
            (const T*)a.k, (const T*)a.q, (const T*)a.v, a.scal, a.Hc, a.Ec, a.Ut, a.Nt, a.Zt, a.dg, a.dbeta,
            parts > 1 ? a.dkp : a.dk, parts > 1 ? a.dqp : a.dq, d.seqlen, d.nheads, d.ngroups, nC, parts);
        return hipGetLastError();
    };
    switch (d.headdim) {
        case 16: return go(std::integral_constant<int, 16>{});
        case 32: return go(std::integral_constant<int, 32>{});
        case 64: return go(std::integral_constant<int, 64>{});
        case 128: return go(std::integral_constant<int, 128>{});
    }
    return hipErrorInvalidValue;
}

template <typename T> hipError_t delta_grads_by_s(const DeltaArgs& a, const Dims& d, hipStream_t stream) {
    switch (d.dstate) {
        case 16: return delta_grads<T, 16>(a, d, stream);
        case 32: return delta_grads<T, 32>(a, d, stream);
        case 64: return delta_grads<T, 64>(a, d, stream);
        case 128: return delta_grads<T, 128>(a, d, stream);
        case 256: return delta_grads<T, 256>(a, d, stream);
    }
    return hipErrorInvalidValue;
}

}  // namespace ssd
