// seq_scan.hpp -- the selective scan's shared parts: parameters, tiles and the
// scan of one state's affine maps over the lanes of a row.
//
// For each channel and state,  h_t = a_t h_{t-1} + b_t  with a_t = exp(dt_t A)
// and b_t = dt_t u_t B_t, is the forward affine recurrence of this library; a
// wave scans it as the other kernels do.  A row of 16 lanes (one DPP row) owns
// a channel and a tile of 16 K steps, K consecutive steps a lane (K = 8, fewer
// for short rows):
//   * each lane folds its K maps serially into one; the product of its a's is
//     exp(A sum dt), one exponential;
//   * four DPP row shifts scan the 16 lane maps;
//   * the tile's incoming state is a carry per (channel, state) kept in LDS;
//   * each lane then applies its maps again from the state that enters it.
// A wave holds 4 channels, so even one sequence of a thousand channels gives
// every SIMD work, and a row of any length walks its tiles.
#pragma once

#include "seq.hpp"

namespace rlca {
namespace seq {

constexpr int kScanLanes = 16;  // lanes of a row
constexpr int kScanWaves = 4;   // waves of a workgroup
constexpr int kScanThreads = kScanWaves * kWave;
constexpr int kScanRows = kScanThreads / kScanLanes;  // channels of a workgroup
constexpr int kScanStates = 8;  // states whose B and C are staged in LDS together

// Steps of a lane, K, and of a tile.  A lane's cost for a tile and state is
// about 13 instructions for the scan over lanes and 7 a step (forward), so long
// rows take the most steps; rows that fill little of their last tile take
// fewer (steps_of).
constexpr int tile_of(int K) { return kScanLanes * K; }

// States of a workgroup's LDS arrays: whole pairs, since the kernels take two
// states at a time.
__host__ __device__ constexpr int padded_states(int S) { return (S + 1) & ~1; }

struct ScanParams {
    const void *u, *delta, *B, *C, *z, *grad_y;
    const float *A, *D, *delta_bias;
    const float *state, *grad_final;
    const uint8_t *flags;
    const int32_t *lengths;
    void *y;
    float *final_state;
    float *checkpoints;  // [num_seqs * channels][tiles][states]: states entering each tile
    void *grad_u, *grad_delta, *grad_z;
    float *grad_state;
    float *bc_partials;  // [num_seqs][groups][blocks of a group][2][states][tiles * tile_of(K)]
    float *row_partials; // [num_seqs][channels][states + 2]: grad_A, grad_D, grad_delta_bias
    int64_t u_n, u_d, delta_n, delta_d, z_n, z_d, g_n, g_d;
    int64_t B_n, B_g, B_s, C_n, C_g, C_s;
    uint32_t num_seqs, channels, groups, per_group, states;
    uint32_t blocks_per_group;  // workgroups that share a group's channels
    int32_t T, tiles;
    int32_t softplus, after_done;
};

// Where a lane works: its sequence, group and channel (clamped to the group's
// last one; `live` says whether it is the lane's own), its lane in the row and
// the row in the workgroup, which holds `rows` channels.
struct ScanLane {
    uint32_t n, g, d, row;
    int lane, local;
    bool live;
};

__device__ __forceinline__ ScanLane scan_lane(const ScanParams &p, int local, uint32_t rows) {
    ScanLane l;
    const uint32_t b = blockIdx.x;
    const uint32_t ng = b / p.blocks_per_group;
    l.n = ng / p.groups;
    l.g = ng - l.n * p.groups;
    l.lane = threadIdx.x & (kScanLanes - 1);
    l.local = local;
    const uint32_t c = (b - ng * p.blocks_per_group) * rows + local;
    l.live = c < p.per_group;
    l.d = l.g * p.per_group + (l.live ? c : p.per_group - 1);
    l.row = l.n * p.channels + l.d;
    return l;
}

// One map: a later run's (a, h) after an earlier run's (pa, ph).  CUT: the
// runs may hold episode starts, where a is 0 and whatever lies before, a NaN
// or infinity too, must not pass, so the product is selected away (as in
// apply_map and compose of scan_core.hpp).  Otherwise a plain fused step, which
// is enough for rows with starts too while all values are tame (below): 0
// times a finite number is 0.  For finite values both give the same bits.
template <bool CUT>
__device__ __forceinline__ float step_map(float a, float b, float h) {
    if constexpr (CUT) return a == 0.f ? b : fmaf(a, h, b);
    return fmaf(a, h, b);
}

template <bool CUT>
__device__ __forceinline__ float product(float a, float b) {
    if constexpr (CUT) return a == 0.f ? 0.f : a * b;
    return a * b;
}

// Inclusive scan of the row's 16 lane maps of two states, towards higher lanes
// (row_shr) or, REVERSE, towards lower ones (row_shl).  Lanes whose source
// lies outside the row keep their map.
//
// Without cuts a step is two instructions a state, an FMA and a product that
// fetch their operand from the other lane themselves; the compiler would move
// it to a register first, and fill that register before (8 instructions).  The
// two states take turns, so that two instructions always lie between a write
// and the lane-crossing read of it, as the hardware requires.
template <bool CUT, bool REVERSE>
__device__ __forceinline__ void row_scan(float (&a)[2], float (&h)[2]) {
    if constexpr (CUT) {
        constexpr int kShift = REVERSE ? 0x100 : 0x110;
        const auto step = [&](auto ctrl) {
            constexpr int kCtrl = decltype(ctrl)::value;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float ph = dpp_move<kCtrl, 0xf>(h[j], 0.f);
                const float pa = dpp_move<kCtrl, 0xf>(a[j], 1.f);
                h[j] = step_map<CUT>(a[j], h[j], ph);
                a[j] = product<CUT>(a[j], pa);
            }
        };
        step(std::integral_constant<int, kShift + 1>{});
        step(std::integral_constant<int, kShift + 2>{});
        step(std::integral_constant<int, kShift + 4>{});
        step(std::integral_constant<int, kShift + 8>{});
    } else {
#define RLCA_STEP(SHIFT)                                                   \
    "v_fmac_f32_dpp %1, %1, %0 " SHIFT " row_mask:0xf bank_mask:0xf\n\t"   \
    "v_fmac_f32_dpp %3, %3, %2 " SHIFT " row_mask:0xf bank_mask:0xf\n\t"   \
    "v_mul_f32_dpp %0, %0, %0 " SHIFT " row_mask:0xf bank_mask:0xf\n\t"    \
    "v_mul_f32_dpp %2, %2, %2 " SHIFT " row_mask:0xf bank_mask:0xf\n\t"
        if constexpr (REVERSE)
            asm("s_nop 1\n\t" RLCA_STEP("row_shl:1") RLCA_STEP("row_shl:2")
                    RLCA_STEP("row_shl:4") RLCA_STEP("row_shl:8")
                : "+v"(a[0]), "+v"(h[0]), "+v"(a[1]), "+v"(h[1]));
        else
            asm("s_nop 1\n\t" RLCA_STEP("row_shr:1") RLCA_STEP("row_shr:2")
                    RLCA_STEP("row_shr:4") RLCA_STEP("row_shr:8")
                : "+v"(a[0]), "+v"(h[0]), "+v"(a[1]), "+v"(h[1]));
#undef RLCA_STEP
    }
}

// The neighbouring lane's value in scan order; the row's first lane gets `x0`.
template <bool REVERSE>
__device__ __forceinline__ float row_shift(float x, float x0) {
    return dpp_move<(REVERSE ? 0x101 : 0x111), 0xf>(x, x0);
}

// The value of the row's last lane in scan order, in all its lanes.
template <bool REVERSE>
__device__ __forceinline__ float row_last(float x) {
    return dpp_move<(REVERSE ? 0x150 : 0x15f), 0xf>(x, x);
}

// Waves run their LDS accesses in order, so lanes of one wave hand values to
// each other without a barrier; this keeps the compiler's order too.
__device__ __forceinline__ void wave_order() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
}

// A tile of one state's B or C in LDS, fp32: a lane's steps in blocks of up to
// four, each lane's next to its neighbours', so that the 16-byte reads of 16
// lanes cover all banks once.
template <int N>
using Floats = float __attribute__((ext_vector_type(N)));
typedef Floats<4> float4v;

template <int K>
struct TileRow {
    static constexpr int kBlock = K < 4 ? K : 4;
    Floats<kBlock> block[K / kBlock][kScanLanes];
};

template <int K>
__device__ __forceinline__ void read_tile(const TileRow<K> &r, int lane, float (&v)[K]) {
    constexpr int N = TileRow<K>::kBlock;
#pragma unroll
    for (int i = 0; i < K / N; ++i) {
        const Floats<N> x = r.block[i][lane];
#pragma unroll
        for (int k = 0; k < N; ++k) v[i * N + k] = x[k];
    }
}

template <typename E, int K>
__device__ __forceinline__ void stage(TileRow<K> &to, const Steps<K, E> &from, int lane) {
    constexpr int N = TileRow<K>::kBlock;
    float v[K];
    from.widen(v);
#pragma unroll
    for (int i = 0; i < K / N; ++i) {
        Floats<N> x;
#pragma unroll
        for (int k = 0; k < N; ++k) x[k] = v[i * N + k];
        to.block[i][lane] = x;
    }
}

// K steps of a lane from step t: dt and dt u from raw = delta and u (0 past
// `end`, where a step then changes nothing; raw becomes dt before softplus).
// Where an episode starts within the row's steps a_t has to be 0 whatever the
// step's dt is, a NaN too: cut, which is added to a's exponent, is -infinity
// there (else 0) and dt is 0.
template <bool FLAGS, int K>
__device__ __forceinline__ void make_steps(const ScanParams &p, const uint8_t *flags, float bias,
                                           int t, int end, int row_steps, const float (&u)[K],
                                           float (&raw)[K], float (&dt)[K], float (&dtu)[K],
                                           float (&cut)[K]) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
        raw[k] += bias;
        dt[k] = p.softplus != 0 ? softplus(raw[k]) : raw[k];
        dtu[k] = dt[k] * u[k];
        if constexpr (FLAGS) cut[k] = 0.f;
    }
    if (t + K > end)  // few lanes
#pragma unroll
        for (int k = 0; k < K; ++k) {
            dt[k] = t + k < end ? dt[k] : 0.f;
            dtu[k] = t + k < end ? dtu[k] : 0.f;
        }
    if constexpr (FLAGS) {
        uint32_t starts = start_bits<K>(flags, t, p.T, p.after_done);
        if (t + K > row_steps) starts &= t < row_steps ? (1u << (row_steps - t)) - 1 : 0u;
        if (starts != 0)
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (starts >> k & 1) {
                    cut[k] = -INFINITY;
                    dt[k] = 0.f;
                }
    }
}

// The product of a lane's a's for one state: exp(A sum dt), or 0 where an
// episode starts in the lane, whatever the steps before the start hold.
template <bool FLAGS>
__device__ __forceinline__ float lane_product(float dt_sum, bool starts, float A2) {
    const float a = exp2_fast(dt_sum * A2);
    return FLAGS && starts ? 0.f : a;
}

// a_k of a lane's steps for one state, A2 = A log2(e).
template <bool FLAGS>
__device__ __forceinline__ float decay(float dt, float cut, float A2) {
    return exp2_fast(FLAGS ? fmaf(dt, A2, cut) : dt * A2);
}

// Tame values: too small for any state, gradient or product of the scans to
// overflow within a tile.  With a in [0, 1] (dt >= 0 and A <= 0), dt u, B, C and
// gy below 2^40 and entering values below 2^100, sums over a tile's steps stay
// below 2^101.  A NaN is not tame.
constexpr float kTameStep = 0x1p40f, kTameState = 0x1p100f;
__device__ __forceinline__ bool tame(float x, float limit) { return fabsf(x) < limit; }

template <int K, typename E>
__device__ __forceinline__ bool all_tame(const Steps<K, E> &s) {
    float v[K];
    s.widen(v);
    bool ok = true;
#pragma unroll
    for (int k = 0; k < K; ++k) ok &= tame(v[k], kTameStep);
    return ok;
}

// Whether a lane's steps are: dt not negative, dt and dt u small.
template <int K>
__device__ __forceinline__ bool steps_tame(const float (&dt)[K], const float (&dtu)[K]) {
    bool ok = true;
#pragma unroll
    for (int k = 0; k < K; ++k)
        ok &= dt[k] >= 0.f && tame(dt[k], kTameStep) && tame(dtu[k], kTameStep);
    return ok;
}

__device__ __forceinline__ bool whole_wave(bool x) {
    return __builtin_amdgcn_ballot_w64(!x) == 0;
}

int steps_of(int64_t T);
ScanParams scan_params(const rlca_scan_call &c, int rows);
rlca_status check_scan(const rlca_scan_call &c, bool backward, Arrays *a);

}  // namespace seq
}  // namespace rlca
