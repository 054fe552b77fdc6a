// Internal launch interface between the C ABI (ssd_api.cpp) and the kernels.
// Sizes are already validated by the caller; these functions only pick the template
// instance, size the grid and enqueue on `stream`.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ssd {

enum { kF32 = 0, kBF16 = 1 };

struct Dims {
    int batch, seqlen, nheads, headdim, dstate, ngroups, chunk;
    // chunks of the sequence; the last one holds seqlen - (nchunks - 1) * chunk tokens
    int nchunks() const { return (seqlen + chunk - 1) / chunk; }
};

hipError_t launch_cumsum(int in_dtype, const void* dt, const float* A, float* G, float* dt_t,
                         const Dims& d, hipStream_t stream);

hipError_t launch_chunk_state(int in_dtype, const void* x, const void* Bm, const float* A,
                              const float* dt_t, float* dstate_chunks, const Dims& d,
                              hipStream_t stream);

hipError_t launch_state_carry(int states_dtype, const float* dstate_chunks, const float* G,
                              const float* h0, void* states, float* final_state, const Dims& d,
                              hipStream_t stream);

// Single-pass state kernel, the alternative to chunk_state + state_carry: one workgroup
// per (batch, head, slice of headdim rows) walks the whole sequence with the running state
// in registers. Built for bf16 inputs, headdim 64 or 128, dstate 64, 128 or 256, and a
// sequence of whole chunks (seqlen a positive multiple of the chunk length).
bool state_scan_supported(int in_dtype, const Dims& d);
// Whether the forward pass takes the single-pass kernel for this shape (measured faster).
bool state_scan_preferred(int in_dtype, const Dims& d);
hipError_t launch_state_scan(int states_dtype, const void* x, const void* Bm, const float* A,
                             const float* dt_t, const float* h0, void* states,
                             float* final_state, const Dims& d, hipStream_t stream);

// Segmented state pass (bf16 inputs, bf16 chunk states): workgroups walk runs of
// `chunks` consecutive chunks for blocks of `heads` heads from a zero state (segment 0 from
// h0), recording each chunk's state relative to its segment's start; a small sequential
// kernel carries the states entering each segment and gives the final state. The output
// kernel then adds 2^{dec_in} * seg_in to each recorded state (segments >= 1).
struct SegPlan {
    int heads, chunks, nseg;
};
// Below this log2 decay from a segment's start the factor 2^{D_c} is exactly 0 in fp32
// (even as a denormal), so adding the decayed entering state changes nothing and the
// kernels that form S_c = L_c + 2^{D_c} S_in skip it (and do not read S_in).
constexpr float kSegCut = -160.f;
struct SegBuffers {
    float* seg_end;   // [B, H, nseg, P, S] each segment's end state from its own start
    void* seg_in;     // [B, H, nseg, P, S] bf16 state entering each segment (>= 1)
    float* dec_in;    // [B, H, nC] log2 decay from the segment's start to each chunk's start
    float* dec_seg;   // [B, H, nseg] each segment's total log2 decay
};
bool state_seg_plan(int in_dtype, int states_dtype, const Dims& d, SegPlan* plan);
size_t state_seg_ws_bytes(const Dims& d, const SegPlan& plan);
SegBuffers state_seg_buffers(void* workspace, const Dims& d, const SegPlan& plan);
hipError_t launch_state_seg(const void* x, const void* Bm, const float* A, const float* G,
                            const float* dt_t, const float* h0, void* states,
                            float* final_state, const SegPlan& plan, const SegBuffers& sb,
                            const Dims& d, hipStream_t stream);
// Segment-relative chunk states -> true chunk-initial states, in place (after the carry),
// with the arithmetic of launch_chunk_out_seg's completion (the same bits).
hipError_t launch_seg_correct(void* states, const SegPlan& plan, const SegBuffers& sb,
                              const Dims& d, hipStream_t stream);

// final_state = h0 (zeros when h0 is NULL): the state after an empty sequence.
hipError_t launch_state_init(const float* h0, float* final_state, const Dims& d,
                             hipStream_t stream);

// One recurrent step on a carried fp32 state (in place), y for that token.
hipError_t launch_decode(int in_dtype, const void* x, const void* dt, const float* A,
                         const void* Bm, const void* Cm, const float* D, float* state, float* y,
                         const Dims& d, hipStream_t stream);

// Backward pass: every buffer below is the caller's (the workspace carved up on the host).
struct BwdWorkspace {
    float *G, *dt_t;      // [B, H, L] cumulative decay and dt (fp32)
    float *Hc, *R;        // [B, H, nC, P, S] chunk-initial states; increments, then the
                          // gradient arriving at each chunk's end
    float* fin;           // [B, H, P, S] forward final state
    float *v, *q, *dyx;   // [B, H, L] per-token scalars
    float *dA_bh, *dD_bh; // [B, H]
    float *dBh, *dCh;     // [B, L, H, S] per-head dB, dC (when heads share a group)
    float* anc;           // [B, H, nC, P*S/256] partial sums of <R_c, state after chunk c>
};
struct BwdLaunch {
    const void *x, *dt, *B, *C;
    const float *A, *D, *h0, *dy, *dfinal;
    float *dx, *ddt, *dA, *dB, *dC, *dD, *dh0;
    BwdWorkspace ws;
};
hipError_t launch_backward(int in_dtype, const BwdLaunch& k, const Dims& d, hipStream_t stream);
// Chunk length at which the backward pass runs its matrix-core kernels for this shape (0:
// none; the token walks then run at the caller's chunk length).
int bwd_mfma_chunk(int in_dtype, int P, int S);
// Partial dB, dC rows the backward pass writes per (token, group) before summing them (1:
// it writes dB and dC directly); d.chunk is the backward's chunk length.
int bwd_partials_per_group(int in_dtype, const Dims& d);

// chunk_out's launch plan for a shape: heads per workgroup, shared interaction tiles, the
// matrix-core flops the launch executes and its LDS bytes per workgroup (host-only; SEGC:
// the instance over segment-relative states). False where no instance exists.
struct OutPlan {
    int heads_per_wg;
    bool shared;
    double mfma_flops, lds_bytes;
};
bool chunk_out_plan(int in_dtype, int states_dtype, bool segc, const Dims& d, OutPlan* plan);
hipError_t launch_chunk_out(int in_dtype, int states_dtype, int out_dtype, const void* x,
                            const void* Bm, const void* Cm, const float* G, const float* dt_t,
                            const void* states, const float* D, void* y, const Dims& d,
                            hipStream_t stream);

// The output kernel over segment-relative chunk states (bf16 inputs and states): each
// chunk's state is taken as states[c] + 2^{dec_in[c]} seg_in[c / seg_chunks] for chunks
// past the first segment.
hipError_t launch_chunk_out_seg(int out_dtype, const void* x, const void* Bm, const void* Cm,
                                const float* G, const float* dt_t, const void* states,
                                const void* seg_in, const float* dec_in, int seg_chunks,
                                const float* D, void* y, const Dims& d, hipStream_t stream);

// Gated delta rule (delta.h). The chunked kernels work on chunks of kDeltaChunk tokens; every
// buffer is the caller's. `scal` holds, per (batch, head, chunk), kDeltaChunk values each of
// e^{G_i}, e^{G_C - G_i} and beta_i and, in the backward pass, G_i log2(e) in 64 bits (kDeltaScal
// floats in all); the matrices are the tile stores of delta.h.
constexpr int kDeltaChunk = 64, kDeltaScal = 5 * kDeltaChunk, kDeltaTiles = 6;
constexpr size_t kDeltaTileBytes = 2048, kDeltaMatBytes = kDeltaTiles * kDeltaTileBytes;  // a stored triangular matrix
struct DeltaArgs {
    const void *v, *beta, *k, *q;
    const float *g, *h0;
    float scale;
    // forward outputs
    void* y;
    float* final_state;
    // backward inputs and outputs
    const float *dy, *dfinal;
    float *dv, *dg, *dbeta, *dk, *dq, *dh0;
    // workspace
    float* scal;         // [B, H, nC, kDeltaScal]
    char *matT, *matM;   // [B, H, nC] tiles of T and M (backward: M^T)
    char* matTt;         // backward: tiles of T^T
    float *seg_ends, *seg_starts;  // forward by segments: [B, H, nseg - 1, P + S, S] and [B, H, nseg, P, S]
    char *Hc, *Ec;       // backward: [B, H, nC] planes [P, S]: states entering, gradients at the end of, each chunk
    char *Ut, *Nt, *Zt;  // backward: [B, H, nC] planes [P, 64]: U, N and scale dY, transposed
    float *dkp, *dqp;    // backward: [parts, B, L, G, S] partial sums over a group's heads
};
// The forward walk's segments of `chunks` chunks (nseg 1: the sequence in one).
struct DeltaSegs {
    int nseg, chunks;
};
constexpr int kDeltaNoSegments = 1 << 30;  // chunks of the one segment
DeltaSegs delta_segments(int in_dtype, const Dims& d);
// Computing waves of a walk's workgroup, for `rows` rows of each of `heads` heads (all batch rows and segments).
int delta_waves(long heads, int rows);
// Rows of the state whose count the first walk's workgroups divide into (they hold rows of both kinds).
inline int delta_first_rows(const Dims& d) { return d.headdim < d.dstate ? d.headdim : d.dstate; }
// Heads of a group that a wave prepares one after another.
int delta_prep_heads(const Dims& d);
// Heads of a group are summed by this many workgroups a chunk in the backward pass.
int delta_bwd_parts(const Dims& d);
// One token at a time, the state in registers; final_state may be h0 itself.
hipError_t launch_delta_recurrent(int in_dtype, int out_dtype, const DeltaArgs& a, const Dims& d,
                                  hipStream_t stream);
// Whether the forward pass takes the token loop for this shape (measured faster).
bool delta_recurrent_preferred(int in_dtype, const Dims& d);
hipError_t launch_delta_prep(int in_dtype, bool backward, const DeltaArgs& a, const Dims& d,
                             hipStream_t stream);
// save: record Hc and U for the backward pass instead of y and the final state.
hipError_t launch_delta_walk_bf16(int out_dtype, bool save, const DeltaArgs& a, const Dims& d, hipStream_t stream);
hipError_t launch_delta_walk_f32(bool save, const DeltaArgs& a, const Dims& d, hipStream_t stream);
hipError_t launch_delta_reverse_bf16(const DeltaArgs& a, const Dims& d, hipStream_t stream);
hipError_t launch_delta_reverse_f32(const DeltaArgs& a, const Dims& d, hipStream_t stream);
hipError_t launch_delta_grads_bf16(const DeltaArgs& a, const Dims& d, hipStream_t stream);
hipError_t launch_delta_grads_f32(const DeltaArgs& a, const Dims& d, hipStream_t stream);
hipError_t launch_delta_grads(int in_dtype, const DeltaArgs& a, const Dims& d, hipStream_t stream);

// Group norm with an activation (k_norm.hip).
enum { kActNone = 0, kActSilu = 1, kActGatePre = 2, kActGatePost = 3 };
struct NormArgs {
    long tokens;
    int channels, groups, x_dtype, z_dtype, out_dtype, act, center;
    float eps;
    const void *x, *z;
    const float *weight, *bias, *dy;
    void* out;
    float *dx, *dz, *dweight, *dbias;
    float *dwp, *dbp;  // workspace: group_norm_rows() rows of `channels` each
};
hipError_t launch_group_norm(const NormArgs& a, hipStream_t stream);
int group_norm_rows(long tokens, int channels, int groups);
hipError_t launch_group_norm_backward(const NormArgs& a, hipStream_t stream);
hipError_t launch_norm_params_zero(const NormArgs& a, hipStream_t stream);

}  // namespace ssd
