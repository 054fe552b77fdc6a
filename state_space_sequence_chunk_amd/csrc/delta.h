// Gated delta rule: operand types and tile layout shared by its chunked kernels.
//
// Per batch row and head, on the state H [P, S] (P = headdim, S = dstate):
//     a_t = exp(g_t),  u_t = beta_t (v_t - a_t H_{t-1} k_t),
//     H_t = a_t H_{t-1} + u_t k_t^T,   y_t = scale H_t q_t.
// A chunk of C = 64 tokens entered by H0, with G the inclusive sum of g in the chunk and
// D_ij = exp(G_i - G_j), is the matrix form of the same recurrence:
//     A = strictly lower part of beta_i D_ij (k_i . k_j),   T = (I + A)^-1 (unit lower)
//     M = lower part of D_ij (q_i . k_j)
//     U = T (beta o (V - e^G o K H0^T)),   Y = scale (e^G o Q H0^T + M U)
//     H1 = e^{G_C} H0 + (e^{G_C - G} o U)^T K
// Tokens behind the last one enter as g = beta = 0 and k = q = v = 0, which leaves U = 0.
//
// Operands. k, q and v enter the matrix cores in the inputs' type. What is computed in fp32
// (states, U, T, M, gradients) enters as a Wide operand: for bf16 inputs a bf16 high part
// and a bf16 remainder (16 significant bits, relative error 2^-17), for fp32 inputs the
// fp32 value itself. A product of two Wide operands drops low x low (at most 2^-16 of it).
// One bf16 operand alone would err by 2^-8 in every step of the walk; the fp32 matrix
// instructions hold all 24 bits and run at an eighth of bf16's rate (154 against 1178 TFLOP/s
// at 8192^3): against 64 bits, y of bf16 inputs is 3e-6 to 7e-6 off (norms), that of fp32 inputs
// 2e-7 to 4e-7.
//
// Fragments. In a K = 32 step lane l holds row (A) or column (B) l & 15 and, in slot v of
// slot group g = l >> 4, the contraction index kmap(g, v) = 4 g + (v & 3) + 16 (v >> 2).
// Two accumulator tiles one above the other (rows 4 g + r and 16 + 4 g + r of column
// l & 15) are then, as they stand, the B operand of the next product, and the tiles of a
// transposed product its A operand: no value moves between lanes on the way.
#pragma once

#include "bwd_mfma.h"
#include "ssd_device.h"
#include "ssd_launch.h"

namespace ssd {

constexpr int kDeltaC = kDeltaChunk;  // tokens a chunk

template <typename T> struct Wide;
template <> struct Wide<bf16> { bf16x8 hi, lo; };
template <> struct Wide<float> { f32x8 v; };

template <typename T> __device__ __forceinline__ Wide<T> make_wide(const f32x4& a, const f32x4& b);
template <> __device__ __forceinline__ Wide<bf16> make_wide<bf16>(const f32x4& a, const f32x4& b) {
    Wide<bf16> w;
    split8(a, b, w.hi, w.lo);
    return w;
}
template <> __device__ __forceinline__ Wide<float> make_wide<float>(const f32x4& a, const f32x4& b) {
    Wide<float> w;
#pragma unroll
    for (int v = 0; v < 4; ++v) {
        w.v[v] = a[v];
        w.v[v + 4] = b[v];
    }
    return w;
}

// Products of two Wide operands.
__device__ __forceinline__ void mma(f32x4& acc, const Wide<bf16>& a, const Wide<bf16>& b) {
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.lo, b.hi, acc, 0, 0, 0);
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.hi, b.lo, acc, 0, 0, 0);
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.hi, b.hi, acc, 0, 0, 0);
}
__device__ __forceinline__ void mma(f32x4& acc, const Wide<float>& a, const Wide<float>& b) {
#pragma unroll
    for (int v = 0; v < 8; ++v) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(a.v[v], b.v[v], acc, 0, 0, 0);
}

// These, and products with an input's fragment, one matrix instruction at a time, `part` of Parts: a chain
// of instructions on one accumulator runs at half their rate, so loops over several accumulators go through
// the parts outside.
template <typename T> struct Parts { static constexpr int IW = 2, WW = 3; };
template <> struct Parts<float> { static constexpr int IW = 8, WW = 8; };
__device__ __forceinline__ void mma_part(f32x4& acc, const Frag<bf16>& a, const Wide<bf16>& b, int part) {
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v, part == 0 ? b.lo : b.hi, acc, 0, 0, 0);
}
__device__ __forceinline__ void mma_part(f32x4& acc, const Wide<bf16>& a, const Frag<bf16>& b, int part) {
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(part == 0 ? a.lo : a.hi, b.v, acc, 0, 0, 0);
}
__device__ __forceinline__ void mma_part(f32x4& acc, const Wide<bf16>& a, const Wide<bf16>& b, int part) {
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(part == 0 ? a.lo : a.hi, part == 1 ? b.lo : b.hi, acc, 0, 0, 0);
}
__device__ __forceinline__ void mma_part(f32x4& acc, const Frag<float>& a, const Wide<float>& b, int part) {
    acc = __builtin_amdgcn_mfma_f32_16x16x4f32(a.v[part], b.v[part], acc, 0, 0, 0);
}
__device__ __forceinline__ void mma_part(f32x4& acc, const Wide<float>& a, const Frag<float>& b, int part) {
    acc = __builtin_amdgcn_mfma_f32_16x16x4f32(a.v[part], b.v[part], acc, 0, 0, 0);
}
__device__ __forceinline__ void mma_part(f32x4& acc, const Wide<float>& a, const Wide<float>& b, int part) {
    acc = __builtin_amdgcn_mfma_f32_16x16x4f32(a.v[part], b.v[part], acc, 0, 0, 0);
}

// Fragment of a row: slots kmap(g, v) of `row`, which points at the K step's first value.
// N: valid values from there (16 leaves the upper half of the slots zero).
template <int N> __device__ __forceinline__ Frag<bf16> row_frag(const bf16* row, int g) {
    Frag<bf16> f;
    const bf16x4 a = *(const bf16x4*)(row + 4 * g);
    const bf16x4 b = N > 16 ? *(const bf16x4*)(row + 16 + 4 * g) : bf16x4{0, 0, 0, 0};
    f.v = __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
    return f;
}
template <int N> __device__ __forceinline__ Frag<float> row_frag(const float* row, int g) {
    Frag<float> f;
    const f32x4 a = *(const f32x4*)(row + 4 * g);
    const f32x4 b = N > 16 ? *(const f32x4*)(row + 16 + 4 * g) : f32x4{0, 0, 0, 0};
    f.v = __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
    return f;
}
template <typename T> __device__ __forceinline__ Frag<T> zero_frag() {
    Frag<T> f;
#pragma unroll
    for (int v = 0; v < 8; ++v) f.v[v] = (T)0.f;
    return f;
}
// The same with rows at or past `valid` zero (valid >= 1).
template <int N, typename T>
__device__ __forceinline__ Frag<T> row_frag_in(const T* base, size_t ld, int row, int valid, int g) {
    const Frag<T> f = row_frag<N>(base + (size_t)(row < valid ? row : 0) * ld, g);
    return row < valid ? f : zero_frag<T>();
}
// Fragment of a column: slots kmap(g, v) are rows r0 + kmap(g, v), of which those at or past
// `valid` are zero.
template <typename T>
__device__ __forceinline__ Frag<T> col_frag_in(const T* col, size_t ld, int r0, int valid, int g) {
    Frag<T> f;
#pragma unroll
    for (int v = 0; v < 8; ++v) {
        const int r = r0 + 4 * g + (v & 3) + 16 * (v >> 2);
        const bool in = r < valid;
        const T x = col[(size_t)(in ? r : 0) * ld];
        f.v[v] = in ? x : (T)0.f;
    }
    return f;
}
// T and M (and their transposes) lie in memory as Wide A-operand fragments of the 16-row by
// 32-column tiles that hold a value: two planes of 64 lanes x 16 bytes a tile (bf16: high
// parts, remainders; fp32: slots 0-3, slots 4-7). Lower tiles are (0,0) (1,0) (2,0) (2,1)
// (3,0) (3,1); upper ones (transposes) (0,0) (0,1) (1,0) (1,1) (2,1) (3,1).
__host__ __device__ constexpr int lower_tile(int ti, int kk) { return ti < 2 ? ti : 2 * ti - 2 + kk; }
__host__ __device__ constexpr int upper_tile(int ti, int kk) { return ti < 2 ? 2 * ti + kk : ti + 2; }

__device__ __forceinline__ Wide<bf16> load_tile(const char* mat, int tile, int lane, bf16) {
    const char* p = mat + tile * kDeltaTileBytes + lane * 16;
    Wide<bf16> w;
    w.hi = *(const bf16x8*)p;
    w.lo = *(const bf16x8*)(p + 1024);
    return w;
}
__device__ __forceinline__ Wide<float> load_tile(const char* mat, int tile, int lane, float) {
    const char* p = mat + tile * kDeltaTileBytes + lane * 16;
    const f32x4 a = *(const f32x4*)p, b = *(const f32x4*)(p + 1024);
    Wide<float> w;
    w.v = __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
    return w;
}
__device__ __forceinline__ void store_tile(char* mat, int tile, int lane, const Wide<bf16>& w) {
    char* p = mat + tile * kDeltaTileBytes + lane * 16;
    *(bf16x8*)p = w.hi;
    *(bf16x8*)(p + 1024) = w.lo;
}
__device__ __forceinline__ void store_tile(char* mat, int tile, int lane, const Wide<float>& w) {
    char* p = mat + tile * kDeltaTileBytes + lane * 16;
    *(f32x4*)p = __builtin_shufflevector(w.v, w.v, 0, 1, 2, 3);
    *(f32x4*)(p + 1024) = __builtin_shufflevector(w.v, w.v, 4, 5, 6, 7);
}

// What the backward pass keeps of a chunk (rows p of N values) lies in memory as the blocks of 64
// bytes of columns that the gradients' kernel holds in LDS: for bf16 inputs the blocks of the bf16
// high parts and then those of the remainders, for fp32 those of the values. Stores a Wide fragment,
// step x of row p: a wave writes 1 KiB as it lies. The pieces of row p are swizzled by plane_swz.
__device__ __forceinline__ int plane_swz(int p) { return 2 * ((p >> 3) & 1) + ((p >> 2) & 1); }
template <int N> __device__ __forceinline__ void store_planes(char* planes, int rows, int p, int x, int g, const Wide<bf16>& w) {
    if constexpr (N >= 32) {
        char* at = planes + (size_t)x * rows * 64 + p * 64 + ((g ^ plane_swz(p)) << 4);
        *(bf16x8*)at = w.hi;
        *(bf16x8*)(at + (size_t)rows * N * 2) = w.lo;
    } else {
        char* at = planes + p * 32 + 8 * g;
        *(bf16x4*)at = __builtin_shufflevector(w.hi, w.hi, 0, 1, 2, 3);
        *(bf16x4*)(at + rows * 32) = __builtin_shufflevector(w.lo, w.lo, 0, 1, 2, 3);
    }
}
template <int N> __device__ __forceinline__ void store_planes(char* planes, int rows, int p, int x, int g, const Wide<float>& w) {
    char* at = planes + (size_t)(2 * x) * rows * 64 + p * 64 + 16 * g;
    *(f32x4*)at = __builtin_shufflevector(w.v, w.v, 0, 1, 2, 3);
    if (N > 16) *(f32x4*)(at + (size_t)rows * 64) = __builtin_shufflevector(w.v, w.v, 4, 5, 6, 7);
}

__device__ __forceinline__ f32x4 ld4(const float* p) { return *(const f32x4*)p; }
constexpr f32x4 kZero4 = {0.f, 0.f, 0.f, 0.f};

}  // namespace ssd
