// Gated delta rule, the walks over the chunks (delta.h has the formulas).
//
// The rows of the state are independent of each other: a wave owns 16 of the P rows, keeps
// H^T [S, 16] in accumulators from the first chunk to the last, and goes through
//     R = K H^T,  U = T (beta o (V - e^G o R)),  Y = scale (e^G o Q H^T + M U),
//     H^T <- e^{G_C} H^T + K^T (e^{G_C - G} o U)
// for each, every accumulator being the next product's operand as it stands (delta.h). Up to
// four waves share a chunk's rows and matrices in LDS; four more have the next chunk's brought there
// meanwhile, so the walk holds one barrier a chunk.
//
// Bound by one wave's way through a chunk: 132 matrix instructions, some 420 others and the LDS reads
// between them, 1.9 us at dstate 128 in bf16 (a workgroup of four such waves a compute unit, each on its
// own SIMD). 32768 tokens of 80 heads of 64 x 128 in two sequences took 5819 us with rows and matrices read
// from memory where they were used, 951 with them in LDS a chunk ahead, 791 with tiles read 16 bytes at a
// time, 691 with a wave that only loads, and takes 576 with four of them and the products interleaved (665 in a
// process's first calls).
// What the backward pass keeps is bound by memory: at 16384 tokens of 48 heads in four sequences the walk
// that stores H and U takes 193 us and the reverse walk 335 us, at about 4.4 TB/s.
#pragma once

#include <algorithm>
#include <type_traits>

#include "delta.h"

namespace ssd {

// Waves of a walk's workgroup that only bring rows and matrices to LDS.
constexpr int kDeltaLoaders = 4;

// What a walk leaves: y (and the final state), the planes for the backward pass, its own gradients, or
// only the state at the end of a segment.
enum DeltaKind { kDeltaOut = 0, kDeltaSave = 1, kDeltaReverse = 2, kDeltaSegment = 3 };

// LDS of one chunk: K rows, Q rows, the workgroup's columns of V (reverse: dY), the two matrices
// and the scalars. Two sets where they fit. Where they do not, the matrices are read from memory by the
// computing waves, and V too where that is not enough (dstate 256); K and Q alone too large for two sets:
// one set (fp32).
template <typename T, int S, int NW, int KIND>
struct DeltaCfg {
    static constexpr int LDS = 163840;
    using TV = std::conditional_t<KIND == kDeltaReverse, float, T>;
    static constexpr int KB = kDeltaC * S * (int)sizeof(T), QB = KIND == kDeltaSave || KIND == kDeltaSegment ? 0 : KB,
                         VB = kDeltaC * 16 * NW * (int)sizeof(TV);
    static constexpr int MB = QB == 0 ? (int)kDeltaMatBytes : 2 * (int)kDeltaMatBytes, SB = 1024;
    static constexpr bool TWO = 2 * (KB + QB + SB) <= LDS;
    static constexpr int SETS = TWO ? 2 : 1;
    static constexpr bool MAT = SETS * (KB + QB + VB + MB + SB) <= LDS;
    static constexpr bool VL = MAT || SETS * (KB + QB + VB + SB) <= LDS;
    static constexpr int QO = KB, SO = QO + QB, VO = SO + SB, MO = VO + (VL ? VB : 0), SET = MO + (MAT ? MB : 0);
    static_assert(SETS * SET <= LDS, "a chunk's rows fit LDS");
};

// A chunk's 64 rows of N values (K, Q, a workgroup's columns of V or dY) in LDS: blocks of 64 bytes
// of columns, each with its 64 rows one behind the other, so that a lane's place is one register and
// the tile, block and row block are constants beside it. The 16-byte piece c of row r sits at
// c ^ f(r): what lanes read together then lies on distinct banks, but where a comment says otherwise.
//   rows  A fragment of rows 16 t + c. bf16: columns 32 x + 8 g + v, one 16-byte read; fp32: columns
//         32 x + kmap.
//   cols  A fragment of columns, rows 32 x + kmap: the columns are those that the state's tile t
//         holds (state_col below).
//   acc   rows r0 + 4 g + 0..3 of columns 16 t + c, as an accumulator holds them.
// Offsets are made opaque: the compiler would form one for every read, or hold them all.
template <typename T, int N> struct Tile;
__device__ __forceinline__ void opaque(uint32_t& v) { asm volatile("" : "+v"(v)); }
template <int N> struct Tile<bf16, N> {
    static constexpr int BYTES = kDeltaC * N * 2, UNITS = BYTES / 1024, RB = N < 32 ? 32 : 64, ROWS = 1024 / RB;
    uint32_t row, col, nat[2];
    static __device__ __forceinline__ int f(int r) { return N < 32 ? 0 : 2 * ((r >> 2) & 1) + ((r >> 3) & 1); }
    __device__ __forceinline__ explicit Tile(int lane) {
        const int c = lane & 15, g = lane >> 4, q = c & 3, r = 4 * g + (c >> 2);
        row = N < 32 ? c * RB + 8 * g : c * RB + ((g ^ f(c)) << 4);
        col = N < 32 ? r * RB + 8 * q : r * RB + ((q ^ f(r)) << 4);
        opaque(row);
        opaque(col);
#pragma unroll
        for (int o = 0; o < 2; ++o) {
            nat[o] = N < 32 ? r * RB + 8 * q : r * RB + (((2 * o + (q >> 1)) ^ f(r)) << 4) + 8 * (q & 1);
            opaque(nat[o]);
        }
    }
    // `src`: row 0, `stride` bytes a row; rows outside the descriptor become zero
    template <int NW> static __device__ __forceinline__ void stage(char* t, BufRsrc src, uint32_t stride, int wave, int lane) {
        // (a load covers 16 or 32 rows: the swizzle is the lane's own)
        const int r0 = lane / (RB / 16), c = (lane % (RB / 16)) ^ f(r0);
        uint32_t at = (uint32_t)r0 * stride + (uint32_t)(c * 16);
        opaque(at);
#pragma unroll
        for (int k = 0; k < (UNITS + NW - 1) / NW; ++k) {
            const int u = k * NW + wave;
            if (UNITS % NW == 0 || u < UNITS) {
                const int r = ROWS * (u % (kDeltaC / ROWS)), x = u / (kDeltaC / ROWS);
                __builtin_amdgcn_raw_ptr_buffer_load_lds(src, (__attribute__((address_space(3))) void*)(t + u * 1024), 16,
                                                         at + ((uint32_t)r * stride + (uint32_t)(x * RB)), 0, 0, 0);
            }
        }
    }
    static __device__ __forceinline__ bf16x4 tr(const char* p) {
        return __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf16x4*)(__attribute__((address_space(3))) char*)p);
    }
    __device__ __forceinline__ Frag<bf16> rows(const char* tile, int t, int x) const {
        Frag<bf16> v;
        const char* p = tile + x * (kDeltaC * RB) + 16 * t * RB + row;
        if constexpr (N < 32) {
            const bf16x4 a = *(const bf16x4*)p, z = {0, 0, 0, 0};
            v.v = __builtin_shufflevector(a, z, 0, 1, 2, 3, 4, 5, 6, 7);
        } else {
            v.v = *(const bf16x8*)p;
        }
        return v;
    }
    // (two-way conflicts: of each piece a tile takes one half)
    __device__ __forceinline__ Frag<bf16> cols(const char* tile, int t, int x) const {
        const char* p = tile + (t >> 1) * (kDeltaC * RB) + 8 * (t & 1) + 32 * x * RB + col;
        Frag<bf16> v;
        v.v = __builtin_shufflevector(tr(p), tr(p + 16 * RB), 0, 1, 2, 3, 4, 5, 6, 7);
        return v;
    }
    __device__ __forceinline__ bf16x4 nat4(const char* tile, int t, int r0) const {
        return tr(tile + (t >> 1) * (kDeltaC * RB) + r0 * RB + nat[t & 1]);
    }
    // as cols, of columns 16 t + c
    __device__ __forceinline__ Frag<bf16> plain_cols(const char* tile, int t, int x) const {
        Frag<bf16> v;
        v.v = __builtin_shufflevector(nat4(tile, t, 32 * x), nat4(tile, t, 32 * x + 16), 0, 1, 2, 3, 4, 5, 6, 7);
        return v;
    }
    __device__ __forceinline__ f32x4 acc(const char* tile, int t, int r0) const {
        const bf16x4 v = (t & 1) ? tr(tile + (t >> 1) * (kDeltaC * RB) + r0 * RB + nat[1])
                                 : tr(tile + (t >> 1) * (kDeltaC * RB) + r0 * RB + nat[0]);
        return f32x4{(float)v[0], (float)v[1], (float)v[2], (float)v[3]};
    }
};
template <int N> struct Tile<float, N> {
    static constexpr int BYTES = kDeltaC * N * 4, UNITS = BYTES / 1024, RB = 64;
    uint32_t row, col;
    static __device__ __forceinline__ int f(int r) { return (r >> 2) & 3; }
    __device__ __forceinline__ explicit Tile(int lane) {
        const int c = lane & 15, g = lane >> 4;
        row = c * RB + ((g ^ f(c)) << 4);
        col = 4 * g * RB + (((c >> 2) ^ g) << 4) + 4 * (c & 3);  // (four-way conflicts)
        opaque(row);
        opaque(col);
    }
    template <int NW> static __device__ __forceinline__ void stage(char* t, BufRsrc src, uint32_t stride, int wave, int lane) {
        uint32_t at = (uint32_t)(lane >> 2) * stride + (uint32_t)(((lane & 3) ^ f(lane >> 2)) * 16);
        opaque(at);
#pragma unroll
        for (int k = 0; k < (UNITS + NW - 1) / NW; ++k) {
            const int u = k * NW + wave;
            if (UNITS % NW == 0 || u < UNITS)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(src, (__attribute__((address_space(3))) void*)(t + u * 1024), 16,
                                                         at + ((uint32_t)(16 * (u & 3)) * stride + (uint32_t)((u >> 2) * RB)), 0, 0, 0);
        }
    }
    __device__ __forceinline__ Frag<float> rows(const char* tile, int t, int x) const {
        Frag<float> v;
        const char* p = tile + 2 * x * (kDeltaC * RB) + 16 * t * RB + row;
        const f32x4 a = *(const f32x4*)p, b = N > 16 ? *(const f32x4*)(p + kDeltaC * RB) : kZero4;
        v.v = __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
        return v;
    }
    __device__ __forceinline__ Frag<float> cols(const char* tile, int t, int x) const {
        Frag<float> v;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            v.v[e] = *(const float*)(tile + t * (kDeltaC * RB) + (32 * x + (e & 3) + 16 * (e >> 2)) * RB + col);
        return v;
    }
    __device__ __forceinline__ Frag<float> plain_cols(const char* tile, int t, int x) const { return cols(tile, t, x); }
    __device__ __forceinline__ f32x4 acc(const char* tile, int t, int r0) const {
        f32x4 v;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = *(const float*)(tile + t * (kDeltaC * RB) + (r0 + e) * RB + col);
        return v;
    }
};

// First of the four consecutive state columns that tile t of H^T holds in slot group g. For bf16 a
// pair of tiles holds eight consecutive columns a group: what a row fragment reads at once.
template <typename T, int S> __device__ __forceinline__ int state_col(int t, int g) {
    return sizeof(T) == 2 && S >= 32 ? 32 * (t >> 1) + 8 * g + 4 * (t & 1) : 16 * t + 4 * g;
}

// `bytes` bytes as they lie (a multiple of 16; the rest of the last 1 KiB becomes zero).
template <int BYTES, int NW>
__device__ __forceinline__ void stage_flat(char* dst, const void* src, int wave, int lane) {
    const BufRsrc r = make_rsrc(src, BYTES);
    constexpr int UNITS = (BYTES + 1023) / 1024;
    uint32_t at = (uint32_t)(lane * 16);
    opaque(at);
#pragma unroll
    for (int k = 0; k < (UNITS + NW - 1) / NW; ++k) {
        const int u = k * NW + wave;
        if (UNITS % NW == 0 || u < UNITS)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)(dst + u * 1024), 16,
                                                     at + (uint32_t)(u * 1024), 0, 0, 0);
    }
}

// What this wave has sent to memory and asked for before its last N stores has arrived, then the
// workgroup's barrier.
template <int N> __device__ __forceinline__ void staged_barrier() {
    static_assert(N <= 63, "vmcnt has six bits");
    __builtin_amdgcn_s_waitcnt(0x0f70 | (N & 15) | ((N >> 4) << 14));
    lds_barrier();
}

__device__ __forceinline__ void buf_store(float v, BufRsrc r, uint32_t off, float) { buf_store_f32(v, r, off, 0); }
__device__ __forceinline__ void buf_store(float v, BufRsrc r, uint32_t off, bf16) {
    __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, (bf16)v), r, off, 0, 0);
}

// acc[t] += rows 16 t + c of a tile, step x, times b.
template <typename T, int N>
__device__ __forceinline__ void rows_times(f32x4 (&acc)[4], const Tile<T, N>& ad, const char* tile, int x, const Wide<T>& b) {
    Frag<T> f[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) f[t] = ad.rows(tile, t, x);
#pragma unroll
    for (int part = 0; part < Parts<T>::IW; ++part)
#pragma unroll
        for (int t = 0; t < 4; ++t) mma_part(acc[t], f[t], b, part);
}
// acc += a stored triangular matrix (UPPER: a transposed one) times b.
template <typename T, bool UPPER, typename Load>
__device__ __forceinline__ void tri_times(f32x4 (&acc)[4], Load&& load, const Wide<T> (&b)[2]) {
    Wide<T> m[kDeltaTiles];
#pragma unroll
    for (int t = 0; t < kDeltaTiles; ++t) m[t] = load(t);
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int part = 0; part < Parts<T>::WW; ++part)
#pragma unroll
            for (int t = 0; t < 4; ++t)
                if (UPPER ? x >= t / 2 : x <= t / 2) mma_part(acc[t], m[UPPER ? upper_tile(t, x) : lower_tile(t, x)], b[x], part);
}
// acc[t] += (columns of the state's tile t)^T times b, over the 64 rows; four tiles at a time.
template <typename T, int N, int NT>
__device__ __forceinline__ void cols_times(f32x4 (&acc)[NT], const Tile<T, N>& ad, const char* tile, const Wide<T> (&b)[2]) {
    constexpr int AT = NT < 4 ? NT : 4;
#pragma unroll
    for (int t0 = 0; t0 < NT; t0 += AT)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            Frag<T> f[AT];
#pragma unroll
            for (int t = 0; t < AT; ++t) f[t] = ad.cols(tile, t0 + t, x);
#pragma unroll
            for (int part = 0; part < Parts<T>::IW; ++part)
#pragma unroll
                for (int t = 0; t < AT; ++t) mma_part(acc[t0 + t], f[t], b[x], part);
        }
}

// The chunks in order (the n-th is at(n)): the last waves of the workgroup only send for their rows
// and matrices, the others compute. A wave that did both stood still while its loads were taken up,
// one every 30 cycles, a quarter of its time (and the compiler lets a transposing read wait for every
// load to LDS that the wave has under way).
template <int SETS, typename At, typename Stage, typename Step>
__device__ __forceinline__ void walk_chunks(bool loader, int nC, At&& at, Stage&& stage, Step&& step) {
    using Zero = std::integral_constant<int, 0>;
    using One = std::integral_constant<int, 1>;
    if constexpr (SETS == 2) {
        if (loader) {
            stage(Zero(), at(0));
            staged_barrier<0>();
            for (int n = 0; n < nC; n += 2) {
                if (n + 1 < nC) stage(One(), at(n + 1));
                staged_barrier<0>();
                if (n + 1 < nC) {
                    if (n + 2 < nC) stage(Zero(), at(n + 2));
                    staged_barrier<0>();
                }
            }
        } else {
            lds_barrier();
            for (int n = 0; n < nC; n += 2) {
                step(Zero(), at(n));
                lds_barrier();
                if (n + 1 < nC) {
                    step(One(), at(n + 1));
                    lds_barrier();
                }
            }
        }
    } else {
        for (int n = 0; n < nC; ++n) {
            if (loader) {
                stage(Zero(), at(n));
                staged_barrier<0>();
            } else {
                lds_barrier();
                step(Zero(), at(n));
            }
            lds_barrier();
        }
    }
}

// Segments. With few rows to walk, the sequence is cut into nseg runs of seg_chunks chunks. The map over
// a segment is linear in the entering state, H -> H F + E: a first walk (kDeltaSegment) takes, beside the
// P rows from a state of zero (segment 0: from h0), S more rows from the identity with V = 0, which end
// as F; delta_segments_kernel carries the states through; then all segments are walked for y at once.
// `starts` [B, H, nseg, P, S] are the states entering the segments (0 for the first, which is h0's).
template <typename T, int S, int NW, typename TO, int KIND>
__global__ __launch_bounds__(64 * (NW + kDeltaLoaders)) __attribute__((amdgpu_waves_per_eu(1, 2))) void delta_walk_kernel(
    const T* __restrict__ k, const T* __restrict__ q, const T* __restrict__ v,
    const float* __restrict__ h0, const float* __restrict__ scal, const char* __restrict__ matT,
    const char* __restrict__ matM, TO* __restrict__ y, float* __restrict__ final_state,
    char* __restrict__ Hc, char* __restrict__ Ut, const float* __restrict__ starts,
    float* __restrict__ ends, float scale, int L, int H, int P, int ngroups, int nC, int nseg,
    int seg_chunks) {
    constexpr bool SAVE = KIND == kDeltaSave, OUT = KIND == kDeltaOut, SEG = KIND == kDeltaSegment;
    using Cfg = DeltaCfg<T, S, NW, KIND>;
    constexpr int NK = S < 32 ? 1 : S / 32, NT = S / 16;
    using KT = Tile<T, S>;
    using VT = Tile<typename Cfg::TV, 16 * NW>;
    __shared__ __align__(1024) char set0[Cfg::SET];
    __shared__ __align__(1024) char set1[Cfg::SETS == 2 ? Cfg::SET : 16];
    const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int id = xcd_remap(blockIdx.x, gridDim.x);
    const int rows = SEG ? P + S : P, npb = rows / (16 * NW);  // rows, and workgroups, a head and segment
    const int bh = id / npb / nseg, seg = id / npb % nseg, b = bh / H, h = bh % H, grp = h / (H / ngroups);
    const int p0 = (id % npb) * (16 * NW), p = p0 + 16 * wave + c;
    const bool unit = SEG && p0 >= P;  // the rows from the identity
    if (unit && seg == 0) return;
    const int c_lo = seg * seg_chunks, c_n = min(seg_chunks, nC - c_lo);
    const size_t ld = (size_t)ngroups * S, ldv = (size_t)H * P;

    const KT ad(lane);
    const VT vd(lane);
    auto stage = [&](auto set, int ch) {
        char* s = decltype(set)::value ? set1 : set0;
        const int t0 = ch * kDeltaC, valid = min(kDeltaC, L - t0);
        const uint32_t bytes = (uint32_t)(((valid - 1) * ld + S) * sizeof(T));
        const size_t row = ((size_t)b * L + t0) * ld + (size_t)grp * S, bhc = (size_t)bh * nC + ch;
        KT::template stage<kDeltaLoaders>(s, make_rsrc(k + row, bytes), (uint32_t)(ld * sizeof(T)), wave - NW, lane);
        if constexpr (OUT)
            KT::template stage<kDeltaLoaders>(s + Cfg::QO, make_rsrc(q + row, bytes), (uint32_t)(ld * sizeof(T)), wave - NW, lane);
        if constexpr (Cfg::VL) {
            if (!unit) VT::template stage<kDeltaLoaders>(s + Cfg::VO,
                                   make_rsrc(v + ((size_t)b * L + t0) * ldv + (size_t)h * P + p0,
                                             (uint32_t)(((valid - 1) * ldv + 16 * NW) * sizeof(T))),
                                   (uint32_t)(ldv * sizeof(T)), wave - NW, lane);
        }
        if constexpr (Cfg::MAT) {
            stage_flat<(int)kDeltaMatBytes, kDeltaLoaders>(s + Cfg::MO, matT + bhc * kDeltaMatBytes, wave - NW, lane);
            if constexpr (OUT)
                stage_flat<(int)kDeltaMatBytes, kDeltaLoaders>(s + Cfg::MO + kDeltaMatBytes, matM + bhc * kDeltaMatBytes, wave - NW, lane);
        }
        stage_flat<3 * kDeltaC * 4, kDeltaLoaders>(s + Cfg::SO, scal + bhc * kDeltaScal, wave - NW, lane);
    };

    f32x4 hs[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const int col = state_col<T, S>(t, g);
        hs[t] = kZero4;
        if (SEG && seg > 0) {
#pragma unroll
            for (int r = 0; r < 4; ++r) hs[t][r] = unit && col + r == p - P ? 1.f : 0.f;
        } else if (wave < NW && (seg > 0 || h0)) {
            hs[t] = ld4((seg > 0 ? starts + ((size_t)bh * nseg + seg) * P * S : h0 + (size_t)bh * P * S) + (size_t)p * S + col);
        }
    }

    auto step = [&](auto set, int ch) {
        const char* s = decltype(set)::value ? set1 : set0;
        const int t0 = ch * kDeltaC, valid = min(kDeltaC, L - t0);
        const size_t bhc = (size_t)bh * nC + ch;
        const char* mT = Cfg::MAT ? s + Cfg::MO : matT + bhc * kDeltaMatBytes;
        const char* mM = Cfg::MAT ? s + Cfg::MO + kDeltaMatBytes : matM + bhc * kDeltaMatBytes;
        const float* sc = (const float*)(s + Cfg::SO);
        Wide<T> tT[kDeltaTiles], tM[kDeltaTiles];
        if constexpr (!Cfg::MAT) {
#pragma unroll
            for (int t = 0; t < kDeltaTiles; ++t) {
                tT[t] = load_tile(mT, t, lane, T());
                if constexpr (OUT) tM[t] = load_tile(mM, t, lane, T());
            }
        }
        auto tile_of = [&](const char* m, const Wide<T>* held, int t) {
            if constexpr (Cfg::MAT) return load_tile(m, t, lane, T());
            else return held[t];
        };

        const char* sq = s + Cfg::QO;
        f32x4 vv[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            if (unit) {
                vv[t] = kZero4;
            } else if constexpr (Cfg::VL) {
                vv[t] = vd.acc(s + Cfg::VO, wave, 16 * t);
            } else {
                const T* vc = v + ((size_t)b * L + t0) * ldv + (size_t)h * P + p;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int i = 16 * t + 4 * g + j;
                    const float x = to_f32(vc[(size_t)(i < valid ? i : 0) * ldv]);
                    vv[t][j] = i < valid ? x : 0.f;
                }
            }
        }
        Wide<T> hw[NK];
#pragma unroll
        for (int x = 0; x < NK; ++x) hw[x] = make_wide<T>(hs[2 * x], NT > 1 ? hs[2 * x + 1 < NT ? 2 * x + 1 : 0] : kZero4);
        if constexpr (SAVE) {  // the state entering the chunk
#pragma unroll
            for (int x = 0; x < NK; ++x) store_planes<S>(Hc + bhc * (size_t)(4 * P * S), P, p, x, g, hw[x]);
        }
        f32x4 n[4], ya[4], eg[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            n[t] = ya[t] = kZero4;
            eg[t] = ld4(sc + 16 * t + 4 * g);
        }
#pragma unroll
        for (int x = 0; x < NK; ++x) rows_times(n, ad, s, x, hw[x]);
        if constexpr (OUT) {
#pragma unroll
            for (int x = 0; x < NK; ++x) {
                rows_times(ya, ad, sq, x, hw[x]);
                if (x == 0) {  // beside the products
#pragma unroll
                    for (int t = 0; t < 4; ++t)
                        n[t] = ld4(sc + 2 * kDeltaC + 16 * t + 4 * g) * (vv[t] - eg[t] * n[t]);
                }
            }
        } else {
#pragma unroll
            for (int t = 0; t < 4; ++t)
                n[t] = ld4(sc + 2 * kDeltaC + 16 * t + 4 * g) * (vv[t] - eg[t] * n[t]);
        }
        const Wide<T> nw[2] = {make_wide<T>(n[0], n[1]), make_wide<T>(n[2], n[3])};
        f32x4 u[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) u[t] = kZero4;
        tri_times<T, false>(u, [&](int t) { return tile_of(mT, tT, t); }, nw);
        f32x4 ue[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) ue[t] = u[t] * ld4(sc + kDeltaC + 16 * t + 4 * g);
        const float ec = sc[kDeltaC - 1];
        if constexpr (SAVE) {
            const Wide<T> uw[2] = {make_wide<T>(u[0], u[1]), make_wide<T>(u[2], u[3])};
#pragma unroll
            for (int x = 0; x < 2; ++x) store_planes<kDeltaC>(Ut + bhc * (size_t)(4 * kDeltaC * P), P, p, x, g, uw[x]);
        } else if constexpr (OUT) {
            const Wide<T> uw[2] = {make_wide<T>(u[0], u[1]), make_wide<T>(u[2], u[3])};
            // rows behind the last token lie outside the descriptor: their stores are dropped
            const BufRsrc ry = make_rsrc(y + ((size_t)b * L + t0) * ldv + (size_t)h * P + p0,
                                         (uint32_t)(((valid - 1) * ldv + 16 * NW) * sizeof(TO)));
#pragma unroll
            for (int t = 0; t < 4; ++t) ya[t] *= eg[t];
            tri_times<T, false>(ya, [&](int t) { return tile_of(mM, tM, t); }, uw);
#pragma unroll
            for (int t = 0; t < 4; ++t) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    buf_store(scale * ya[t][j], ry,
                              (uint32_t)((16 * t + 4 * g + j) * ldv * sizeof(TO) + (16 * wave + c) * sizeof(TO)), TO());
            }
        }
        const Wide<T> uw[2] = {make_wide<T>(ue[0], ue[1]), make_wide<T>(ue[2], ue[3])};
#pragma unroll
        for (int t = 0; t < NT; ++t) hs[t] *= ec;
        cols_times(hs, ad, s, uw);
    };

    walk_chunks<Cfg::SETS>(wave >= NW, c_n, [&](int n) { return c_lo + n; }, stage, step);
    if (wave >= NW) return;
    float* end = OUT ? (final_state && seg == nseg - 1 ? final_state + (size_t)bh * P * S : nullptr)
                 : SEG ? ends + ((size_t)bh * nseg + seg) * rows * S : nullptr;
    if (end) {
#pragma unroll
        for (int t = 0; t < NT; ++t) *(f32x4*)(end + (size_t)p * S + state_col<T, S>(t, g)) = hs[t];
    }
}

// The states entering the segments: a workgroup takes 16 rows of one head from segment to segment, a wave
// two of the tiles of H^T <- F^T H^T + E^T, in fp32 products whose operands are accumulators as they stand
// (through LDS from wave to wave); F of the next segment is on its way meanwhile.
template <int S>
__global__ __launch_bounds__(S < 32 ? 64 : 2 * S) void delta_segments_kernel(const float* __restrict__ ends,
                                                                             float* __restrict__ starts, int P, int nseg) {
    constexpr int NT = S / 16, PER = NT < 2 ? NT : 2;
    __shared__ __align__(16) float hx[2][NT][64][4];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, c = lane & 15, g = lane >> 4;
    const int bh = blockIdx.x / (P / 16), p = blockIdx.x % (P / 16) * 16 + c;
    const size_t rows = P + S;
    float f[NT][4][PER];
    auto load = [&](int k) {
        const float* F = ends + (((size_t)bh * (nseg - 1) + k) * rows + P) * S;
#pragma unroll
        for (int x = 0; x < NT; ++x)
#pragma unroll
            for (int s = 0; s < 4; ++s)
#pragma unroll
                for (int t = 0; t < PER; ++t) f[x][s][t] = F[(size_t)(16 * x + 4 * g + s) * S + 16 * (PER * w + t) + c];
    };
    if (nseg > 2) load(1);
    for (int k = 0; k + 1 < nseg; ++k) {
        const float* end = ends + ((size_t)bh * (nseg - 1) + k) * rows * S;
        f32x4 o[PER];
#pragma unroll
        for (int t = 0; t < PER; ++t) o[t] = ld4(end + (size_t)p * S + 16 * (PER * w + t) + 4 * g);
        if (k > 0) {
#pragma unroll
            for (int x = 0; x < NT; ++x) {
                const f32x4 h = ld4(&hx[k & 1][x][lane][0]);
#pragma unroll
                for (int s = 0; s < 4; ++s)
#pragma unroll
                    for (int t = 0; t < PER; ++t) o[t] = __builtin_amdgcn_mfma_f32_16x16x4f32(f[x][s][t], h[s], o[t], 0, 0, 0);
            }
            if (k + 2 < nseg) load(k + 1);
        }
#pragma unroll
        for (int t = 0; t < PER; ++t) {
            *(f32x4*)&hx[(k + 1) & 1][PER * w + t][lane][0] = o[t];
            *(f32x4*)(starts + (((size_t)bh * nseg + k + 1) * P + p) * S + 16 * (PER * w + t) + 4 * g) = o[t];
        }
        lds_barrier();
    }
}

// The walk of the gradient, from the last chunk to the first: with E the gradient arriving at
// the chunk's end (dH1) and Z = scale dY,
//     dU = M^T Z + e^{G_C - G} o (K E^T),   N = T^T dU   (N: dL/d of what T multiplies)
//     dV = beta o N,   E <- e^{G_C} E + (e^G o Z)^T Q - (beta e^G o N)^T K
template <typename T, int S, int NW>
__global__ __launch_bounds__(64 * (NW + kDeltaLoaders)) __attribute__((amdgpu_waves_per_eu(1, 2))) void delta_reverse_kernel(
    const T* __restrict__ k, const T* __restrict__ q, const float* __restrict__ dy,
    const float* __restrict__ dfinal, const float* __restrict__ scal,
    const char* __restrict__ matTt, const char* __restrict__ matMt, float* __restrict__ dv,
    float* __restrict__ dh0, char* __restrict__ Ec, char* __restrict__ Nt, char* __restrict__ Zt,
    float scale, int L, int H, int P, int ngroups, int nC) {
    using Cfg = DeltaCfg<T, S, NW, kDeltaReverse>;
    constexpr int NK = S < 32 ? 1 : S / 32, NT = S / 16;
    using KT = Tile<T, S>;
    using VT = Tile<typename Cfg::TV, 16 * NW>;
    __shared__ __align__(1024) char set0[Cfg::SET];
    __shared__ __align__(1024) char set1[Cfg::SETS == 2 ? Cfg::SET : 16];
    const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int id = xcd_remap(blockIdx.x, gridDim.x);
    const int npb = P / (16 * NW);
    const int bh = id / npb, b = bh / H, h = bh % H, grp = h / (H / ngroups);
    const int p0 = (id % npb) * (16 * NW), p = p0 + 16 * wave + c;
    const size_t ld = (size_t)ngroups * S, ldv = (size_t)H * P;

    const KT ad(lane);
    const VT vd(lane);
    auto stage = [&](auto set, int ch) {
        char* s = decltype(set)::value ? set1 : set0;
        const int t0 = ch * kDeltaC, valid = min(kDeltaC, L - t0);
        const uint32_t bytes = (uint32_t)(((valid - 1) * ld + S) * sizeof(T));
        const size_t row = ((size_t)b * L + t0) * ld + (size_t)grp * S, bhc = (size_t)bh * nC + ch;
        KT::template stage<kDeltaLoaders>(s, make_rsrc(k + row, bytes), (uint32_t)(ld * sizeof(T)), wave - NW, lane);
        KT::template stage<kDeltaLoaders>(s + Cfg::QO, make_rsrc(q + row, bytes), (uint32_t)(ld * sizeof(T)), wave - NW, lane);
        if constexpr (Cfg::VL)
            VT::template stage<kDeltaLoaders>(s + Cfg::VO,
                                   make_rsrc(dy + ((size_t)b * L + t0) * ldv + (size_t)h * P + p0,
                                             (uint32_t)(((valid - 1) * ldv + 16 * NW) * 4)),
                                   (uint32_t)(ldv * 4), wave - NW, lane);
        if constexpr (Cfg::MAT) {
            stage_flat<(int)kDeltaMatBytes, kDeltaLoaders>(s + Cfg::MO, matTt + bhc * kDeltaMatBytes, wave - NW, lane);
            stage_flat<(int)kDeltaMatBytes, kDeltaLoaders>(s + Cfg::MO + kDeltaMatBytes, matMt + bhc * kDeltaMatBytes, wave - NW, lane);
        }
        stage_flat<3 * kDeltaC * 4, kDeltaLoaders>(s + Cfg::SO, scal + bhc * kDeltaScal, wave - NW, lane);
    };

    f32x4 es[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) es[t] = dfinal && wave < NW ? ld4(dfinal + ((size_t)bh * P + p) * S + state_col<T, S>(t, g)) : kZero4;

    auto step = [&](auto set, int ch) {
        const char* s = decltype(set)::value ? set1 : set0;
        const int t0 = ch * kDeltaC, valid = min(kDeltaC, L - t0);
        const size_t bhc = (size_t)bh * nC + ch;
        const char* mT = Cfg::MAT ? s + Cfg::MO : matTt + bhc * kDeltaMatBytes;
        const char* mM = Cfg::MAT ? s + Cfg::MO + kDeltaMatBytes : matMt + bhc * kDeltaMatBytes;
        const float* sc = (const float*)(s + Cfg::SO);
        Wide<T> tT[kDeltaTiles], tM[kDeltaTiles];
        if constexpr (!Cfg::MAT) {
#pragma unroll
            for (int t = 0; t < kDeltaTiles; ++t) {
                tM[t] = load_tile(mM, t, lane, T());
                tT[t] = load_tile(mT, t, lane, T());
            }
        }
        auto tile_of = [&](const char* m, const Wide<T>* held, int t) {
            if constexpr (Cfg::MAT) return load_tile(m, t, lane, T());
            else return held[t];
        };
        f32x4 z[4], du[4];
        {
            Wide<T> ew[NK];
#pragma unroll
            for (int x = 0; x < NK; ++x) {  // the gradient at the chunk's end
                ew[x] = make_wide<T>(es[2 * x], NT > 1 ? es[2 * x + 1 < NT ? 2 * x + 1 : 0] : kZero4);
                store_planes<S>(Ec + bhc * (size_t)(4 * P * S), P, p, x, g, ew[x]);
            }
#pragma unroll
            for (int t = 0; t < 4; ++t) du[t] = kZero4;
#pragma unroll
            for (int x = 0; x < NK; ++x) rows_times(du, ad, s, x, ew[x]);
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                du[t] *= ld4(sc + kDeltaC + 16 * t + 4 * g);
                if constexpr (Cfg::VL) {
                    z[t] = scale * vd.acc(s + Cfg::VO, wave, 16 * t);
                } else {
                    const float* zc = dy + ((size_t)b * L + t0) * ldv + (size_t)h * P + p;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int i = 16 * t + 4 * g + j;
                        const float x = zc[(size_t)(i < valid ? i : 0) * ldv];
                        z[t][j] = i < valid ? scale * x : 0.f;
                    }
                }
            }
        }
        {
            const Wide<T> zw[2] = {make_wide<T>(z[0], z[1]), make_wide<T>(z[2], z[3])};
#pragma unroll
            for (int x = 0; x < 2; ++x) store_planes<kDeltaC>(Zt + bhc * (size_t)(4 * kDeltaC * P), P, p, x, g, zw[x]);
            tri_times<T, true>(du, [&](int t) { return tile_of(mM, tM, t); }, zw);
        }
        f32x4 n[4];
        {
            const Wide<T> dw[2] = {make_wide<T>(du[0], du[1]), make_wide<T>(du[2], du[3])};
#pragma unroll
            for (int t = 0; t < 4; ++t) n[t] = kZero4;
            tri_times<T, true>(n, [&](int t) { return tile_of(mT, tT, t); }, dw);
        }
        {
            const Wide<T> nw[2] = {make_wide<T>(n[0], n[1]), make_wide<T>(n[2], n[3])};
#pragma unroll
            for (int x = 0; x < 2; ++x) store_planes<kDeltaC>(Nt + bhc * (size_t)(4 * kDeltaC * P), P, p, x, g, nw[x]);
        }
        const BufRsrc rv = make_rsrc(dv + ((size_t)b * L + t0) * ldv + (size_t)h * P + p0,
                                     (uint32_t)(((valid - 1) * ldv + 16 * NW) * 4));
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const f32x4 eg = ld4(sc + 16 * t + 4 * g), bt = ld4(sc + 2 * kDeltaC + 16 * t + 4 * g);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int i = 16 * t + 4 * g + j;
                const float x = bt[j] * n[t][j];
                buf_store_f32(x, rv, (uint32_t)(i * ldv * 4 + (16 * wave + c) * 4), 0);
                n[t][j] = -eg[j] * x;
                z[t][j] *= eg[j];
            }
        }
        const Wide<T> zw[2] = {make_wide<T>(z[0], z[1]), make_wide<T>(z[2], z[3])};
        const Wide<T> nw[2] = {make_wide<T>(n[0], n[1]), make_wide<T>(n[2], n[3])};
        const float ec = sc[kDeltaC - 1];
#pragma unroll
        for (int t = 0; t < NT; ++t) es[t] *= ec;
        cols_times(es, ad, s + Cfg::QO, zw);
        cols_times(es, ad, s, nw);
    };
    walk_chunks<Cfg::SETS>(wave >= NW, nC, [&](int n) { return nC - 1 - n; }, stage, step);
    if (wave >= NW) return;
    if (dh0) {
#pragma unroll
        for (int t = 0; t < NT; ++t) *(f32x4*)(dh0 + ((size_t)bh * P + p) * S + state_col<T, S>(t, g)) = es[t];
    }
}

namespace {
template <typename F> hipError_t by_dstate(int S, F&& f) {
    switch (S) {
        case 16: return f(std::integral_constant<int, 16>{});
        case 32: return f(std::integral_constant<int, 32>{});
        case 64: return f(std::integral_constant<int, 64>{});
        case 128: return f(std::integral_constant<int, 128>{});
        case 256: return f(std::integral_constant<int, 256>{});
    }
    return hipErrorInvalidValue;
}
// f(the waves that walk `rows` rows of each of `heads` heads and segments)
template <typename F> hipError_t by_waves(long heads, int rows, F&& f) {
    const int nw = delta_waves(heads, rows);
    if (nw == 1) return f(std::integral_constant<int, 1>{});
    if (nw == 2) return f(std::integral_constant<int, 2>{});
    return f(std::integral_constant<int, 4>{});
}

// nseg segments (1: none) of seg_chunks chunks; with segments, what comes before the walk for y.
template <typename T, typename TO, int KIND>
hipError_t walk(const DeltaArgs& a, const Dims& d, const DeltaSegs& sg, hipStream_t stream) {
    const int nC = (d.seqlen + kDeltaC - 1) / kDeltaC, segs = KIND == kDeltaSegment ? sg.nseg - 1 : sg.nseg;
    const int least = KIND == kDeltaSegment ? delta_first_rows(d) : d.headdim;
    return by_dstate(d.dstate, [&](auto s) {
        return by_waves((long)d.batch * d.nheads * segs, least, [&](auto nw) {
            constexpr int NW = decltype(nw)::value;
            const int rows = KIND == kDeltaSegment ? d.headdim + d.dstate : d.headdim;
            const unsigned blocks = (unsigned)((long)d.batch * d.nheads * segs * (rows / (16 * NW)));
            delta_walk_kernel<T, decltype(s)::value, NW, TO, KIND><<<dim3(blocks), 64 * (NW + kDeltaLoaders), 0, stream>>>(
                (const T*)a.k, (const T*)a.q, (const T*)a.v, a.h0, a.scal, a.matT, a.matM, (TO*)a.y,
                a.final_state, a.Hc, a.Ut, a.seg_starts, a.seg_ends, a.scale, d.seqlen, d.nheads, d.headdim,
                d.ngroups, nC, segs, sg.chunks);
            return hipGetLastError();
        });
    });
}

template <typename T, typename TO>
hipError_t walk_out(const DeltaArgs& a, const Dims& d, hipStream_t stream) {
    const DeltaSegs sg = delta_segments(sizeof(T) == 2 ? kBF16 : kF32, d);
    if (sg.nseg > 1) {
        hipError_t e = walk<T, float, kDeltaSegment>(a, d, sg, stream);
        if (e != hipSuccess) return e;
        e = by_dstate(d.dstate, [&](auto s) {
            delta_segments_kernel<decltype(s)::value><<<dim3((unsigned)((long)d.batch * d.nheads * (d.headdim / 16))), decltype(s)::value < 32 ? 64 : 2 * decltype(s)::value, 0, stream>>>(
                a.seg_ends, a.seg_starts, d.headdim, sg.nseg);
            return hipGetLastError();
        });
        if (e != hipSuccess) return e;
    }
    return walk<T, TO, kDeltaOut>(a, d, sg, stream);
}

template <typename T> hipError_t reverse(const DeltaArgs& a, const Dims& d, hipStream_t stream) {
    const int nC = (d.seqlen + kDeltaC - 1) / kDeltaC;
    return by_dstate(d.dstate, [&](auto s) {
        return by_waves((long)d.batch * d.nheads, d.headdim, [&](auto nw) {
            constexpr int NW = decltype(nw)::value;
            const unsigned blocks = (unsigned)((long)d.batch * d.nheads * (d.headdim / (16 * NW)));
            delta_reverse_kernel<T, decltype(s)::value, NW><<<dim3(blocks), 64 * (NW + kDeltaLoaders), 0, stream>>>(
                (const T*)a.k, (const T*)a.q, a.dy, a.dfinal, a.scal, a.matTt, a.matM, a.dv, a.dh0,
                a.Ec, a.Nt, a.Zt, a.scale, d.seqlen, d.nheads, d.headdim, d.ngroups, nC);
            return hipGetLastError();
        });
    });
}
}  // namespace

}  // namespace ssd
