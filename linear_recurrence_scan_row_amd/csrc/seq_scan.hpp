// seq_scan.hpp -- the selective scan's shared parts: parameters, tiles and the
// scan of one state's affine maps over the lanes of a row.
//
// For each channel and state,  h_t = a_t h_{t-1} + b_t  with a_t = exp(dt_t A)
// and b_t = dt_t u_t B_t, is the forward affine recurrence of this library; a
// wave scans it as the other kernels do.  A row of L = 16, 4 or 1 lanes owns a
// channel and a tile of 8 L steps, 8 consecutive steps a lane:
//   * each lane folds its 8 maps serially into one; the product of its a's is
//     exp(A sum dt), one exponential;
//   * lane-crossing moves scan the L lane maps (four DPP row shifts for 16);
//   * the tile's incoming state is a carry per (channel, state) kept in LDS;
//   * each lane then applies its maps again from the state that enters it.
// A lane alone (L = 1) applies them once, from the carry.  Where a tile's states
// may grow, so that the product of its a's leaves float32's range, the lanes apply
// their steps one after the other instead.  Fewer lanes a row
// waste less of a short row and cost less a step, but make fewer waves:
// lanes_of weighs the two.  A row of any length walks its tiles.
#pragma once

#include "seq.hpp"

namespace rlca {
namespace seq {

constexpr int kScanK = 8;      // steps of a lane
constexpr int kScanWaves = 4;  // waves of a workgroup
constexpr int kScanThreads = kScanWaves * kWave;

// Steps of a tile, channels of a workgroup, and states whose B and C are staged
// in LDS together, by the lanes of a row.
constexpr int tile_of(int L) { return kScanK * L; }
constexpr int rows_of(int L) { return kScanThreads / L; }
constexpr int states_of(int L) { return L == 16 ? 8 : 16; }

// States of a workgroup's LDS arrays: whole pairs, since the kernels take two
// states at a time.  A row's values are `pitch` apart from the next row's, so
// that the rows of a wave fall into different banks.
__host__ __device__ constexpr int padded_states(int S) { return (S + 1) & ~1; }
__host__ __device__ constexpr int pitch_of(int S, int L) {
    return padded_states(S) + (L == 16 ? 0 : 2);
}

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
    float *bc_partials;  // [num_seqs][groups][blocks of a group][2][states][tiles * tile_of(L)]
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

template <int L>
__device__ __forceinline__ ScanLane scan_lane(const ScanParams &p, uint32_t thread, int local,
                                              uint32_t rows) {
    ScanLane l;
    const uint32_t b = blockIdx.x;
    const uint32_t ng = b / p.blocks_per_group;
    l.n = ng / p.groups;
    l.g = ng - l.n * p.groups;
    l.lane = thread & (L - 1);
    l.local = local;
    const uint32_t c = (b - ng * p.blocks_per_group) * rows + local;
    l.live = c < p.per_group;
    l.d = l.g * p.per_group + (l.live ? c : p.per_group - 1);
    l.row = l.n * p.channels + l.d;
    return l;
}

// How a wave computes a tile's states:
//   * plain: fused steps and the lane scan;
//   * with cuts: the same, with every start selected (rows with episode starts
//     whose values are not all tame);
//   * serially, where states may grow (A above 0, or steps below 0 without
//     softplus).  The product of a tile's a's may be infinite there while the states
//     are not: from a state of 0 the lane scan would give inf * 0.  So no a is formed
//     or multiplied with another: lane after lane applies its steps to the state that
//     the lane before hands on, one state at a time.  Taken where a row's a's may
//     multiply to more than 2^kMostGrowth in a tile; below that the products overflow
//     nothing that the states themselves do not nearly overflow.  Forward and backward
//     2350 us where the decaying model takes 710 (8x2048 channels of 2048 steps, 16
//     states), 530 against 415 for 4096x256 channels of 5 steps; states that grow a
//     little 730 and 530.
constexpr float kMostGrowth = 16.f;

// x, without the compiler's knowledge that it is: what is formed from it is formed
// where it stands, not ahead of the loops around it, where it would hold registers.
template <typename X>
__device__ __forceinline__ X here(X x) {
    asm volatile("" : "+v"(x));
    return x;
}

// The kernel's arguments (one structure), read anew: nothing of theirs is shared with
// code that has read them before.
template <typename Params>
__device__ __forceinline__ Params arguments_again() {
    typedef const __attribute__((address_space(4))) Params *Arguments;
    Arguments p = (Arguments)__builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(p));
    Params q;
    __builtin_memcpy(&q, p, sizeof q);
    return q;
}

// One map: a later run's (a, h) after an earlier run's (pa, ph).  CUT: the
// runs may hold episode starts, where whatever lies before, a NaN or infinity too,
// must not pass, so the product is selected away.  A start's a is -0; an a that has
// underflowed is 0 and starts nothing: 0 times a NaN stays one.  Otherwise a plain
// fused step, which is enough for rows with starts too while all values are tame
// (below): 0 times a finite number is 0.  For finite values both give the same bits.
__device__ __forceinline__ bool is_cut(float a) { return as_bits(a) == as_bits(-0.f); }

template <bool CUT>
__device__ __forceinline__ float step_map(float a, float b, float h) {
    if constexpr (CUT) return is_cut(a) ? b : fmaf(a, h, b);
    return fmaf(a, h, b);
}

// What passes of a state or gradient, and the product of two runs' a's.
template <bool CUT>
__device__ __forceinline__ float pass(float a, float h) {
    if constexpr (CUT) return is_cut(a) ? 0.f : a * h;
    return a * h;
}

template <bool CUT>
__device__ __forceinline__ float product(float a, float pa) {
    if constexpr (CUT) return is_cut(a) || is_cut(pa) ? -0.f : a * pa;
    return a * pa;
}

// The lane-crossing moves of a row: STEP lanes on in scan order (REVERSE: towards
// lower lanes), its last lane to all.
template <int L, bool REVERSE, int STEP>
constexpr int shift_ctrl() {
    if constexpr (L == 16) return (REVERSE ? 0x100 : 0x110) + STEP;  // row_shl, row_shr
    // quad_perm: lane i takes lane i - STEP (i + STEP), itself where there is none
    int c = 0;
    for (int i = 0; i < 4; ++i) {
        const int from = REVERSE ? i + STEP : i - STEP;
        c |= (from < 0 || from > 3 ? i : from) << (2 * i);
    }
    return c;
}

// Inclusive scan of the row's lane maps of two states, towards higher lanes or,
// REVERSE, towards lower ones.  Lanes whose source lies outside the row keep
// their map.
//
// For 16 lanes without cuts a step is two instructions a state, an FMA and a
// product that fetch their operand from the other lane themselves; the
// compiler would move it to a register first, and fill that register before (8
// instructions).  The two states take turns, so that two instructions always
// lie between a write and the lane-crossing read of it, as the hardware
// requires.
template <bool CUT, bool REVERSE, int L>
__device__ __forceinline__ void row_scan(float (&a)[2], float (&h)[2], int lane) {
    if constexpr (L == 4) {
        const auto step = [&](auto by) {
            constexpr int kStep = decltype(by)::value;
            constexpr int kCtrl = shift_ctrl<4, REVERSE, kStep>();
            const bool has = REVERSE ? lane + kStep < 4 : lane >= kStep;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float ph = dpp_move<kCtrl, 0xf>(h[j], h[j]);
                const float pa = dpp_move<kCtrl, 0xf>(a[j], a[j]);
                h[j] = has ? step_map<CUT>(a[j], h[j], ph) : h[j];
                a[j] = has ? product<CUT>(a[j], pa) : a[j];
            }
        };
        step(std::integral_constant<int, 1>{});
        step(std::integral_constant<int, 2>{});
    } else if constexpr (CUT) {
        const auto step = [&](auto by) {
            constexpr int kCtrl = shift_ctrl<16, REVERSE, decltype(by)::value>();
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float ph = dpp_move<kCtrl, 0xf>(h[j], 0.f);
                const float pa = dpp_move<kCtrl, 0xf>(a[j], 1.f);
                h[j] = step_map<CUT>(a[j], h[j], ph);
                a[j] = product<CUT>(a[j], pa);
            }
        };
        step(std::integral_constant<int, 1>{});
        step(std::integral_constant<int, 2>{});
        step(std::integral_constant<int, 4>{});
        step(std::integral_constant<int, 8>{});
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
template <bool REVERSE, int L>
__device__ __forceinline__ float row_shift(float x, float x0, int lane) {
    if constexpr (L == 16) return dpp_move<shift_ctrl<16, REVERSE, 1>(), 0xf>(x, x0);
    const float y = dpp_move<shift_ctrl<4, REVERSE, 1>(), 0xf>(x, x);
    return lane == (REVERSE ? L - 1 : 0) ? x0 : y;
}

// The value of the row's last lane in scan order, in all its lanes.
template <bool REVERSE, int L>
__device__ __forceinline__ float row_last(float x) {
    if constexpr (L == 16) return dpp_move<(REVERSE ? 0x150 : 0x15f), 0xf>(x, x);
    return dpp_move<(REVERSE ? 0x00 : 0xff), 0xf>(x, x);
}

__device__ __forceinline__ bool whole_wave(bool x) {
    return __builtin_amdgcn_ballot_w64(!x) == 0;
}

// Whether `x`, uniform in a wave, is true in all the workgroup's waves.
template <int WAVES>
__device__ __forceinline__ bool all_waves(bool x, uint32_t (&of_waves)[WAVES], int wave,
                                          int in_wave) {
    if (in_wave == 0) of_waves[wave] = x ? 1u : 0u;
    __syncthreads();
    uint32_t all = 1u;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) all &= of_waves[w];
    return __builtin_amdgcn_readfirstlane(all) != 0u;
}

// Waves run their LDS accesses in order, so lanes of one wave hand values to
// each other without a barrier; this keeps the compiler's order too.
__device__ __forceinline__ void wave_order() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
}

// A tile of one state's B or C in LDS, fp32: a lane's steps as two blocks of
// four, each lane's next to its neighbours', so that the 16-byte reads of 16
// lanes cover all banks once.
typedef float float4v __attribute__((ext_vector_type(4)));
template <int L>
struct TileRow {
    float4v half[2][L];
};

template <int L>
__device__ __forceinline__ void read_tile(const TileRow<L> &r, int lane, float (&v)[kScanK]) {
    const float4v x = r.half[0][lane], y = r.half[1][lane];
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = x[k], v[4 + k] = y[k];
}

template <typename E, int L>
__device__ __forceinline__ void stage(TileRow<L> &to, const Steps<kScanK, E> &from, int lane) {
    float v[kScanK];
    from.widen(v);
    float4v x, y;
#pragma unroll
    for (int k = 0; k < 4; ++k) x[k] = v[k], y[k] = v[4 + k];
    to.half[0][lane] = x;
    to.half[1][lane] = y;
}

// What a thread stages: 8 steps of one state, of B in the first kWaves waves and
// of C in the next.
template <int L, int THREADS>
struct Stager {
    static constexpr int kWaves = states_of(L) * L > kWave ? states_of(L) * L / kWave : 1;
    int c, s, lane;
    bool active;
    __device__ __forceinline__ Stager(int lane_of_row, int wave, int in_wave)
        : c(wave / kWaves % 2), s(wave % kWaves * (kWave / L) + in_wave / L),
          lane(lane_of_row),
          active((2 * kWaves * kWave >= THREADS || wave < 2 * kWaves) &&
                 (L > 1 || s < states_of(L))) {}
};

// The largest A log2(e) and -A log2(e) of a wave, at least 0: what a step's a can be,
// 2^(dt up) for a step above 0 and 2^(-dt down) for one below.  A NaN is left out: it
// does not overflow.
struct Growth {
    float up = 0.f, down = 0.f;
    __device__ __forceinline__ void add(float A2) {
        up = fmaxf(up, A2);
        down = fmaxf(down, -A2);
    }
    __device__ __forceinline__ void meet() {  // the wave's lanes
#pragma unroll
        for (int m = 1; m < kWave; m <<= 1) {
            up = fmaxf(up, __shfl_xor(up, m));
            down = fmaxf(down, __shfl_xor(down, m));
        }
        up = from_bits<float>(__builtin_amdgcn_readfirstlane(as_bits(up)));
        down = from_bits<float>(__builtin_amdgcn_readfirstlane(as_bits(down)));
    }
    // Whether the a's of a row may multiply to more than 2^kMostGrowth in a tile:
    // whether some lane's steps reach an Lth of that exponent.
    template <int L>
    __device__ __forceinline__ bool too_much(const float (&dt)[kScanK]) const {
        float on = 0.f, back = 0.f;
#pragma unroll
        for (int k = 0; k < kScanK; ++k) on += fmaxf(dt[k], 0.f), back += fmaxf(-dt[k], 0.f);
        // 0 times infinity is no growth
        const float most = (up > 0.f ? on * up : 0.f) + (back > 0.f ? back * down : 0.f);
        return !whole_wave(most < kMostGrowth / L);
    }
};

// Serial steps: a_k h for a step of size dt, A2 = A log2(e); nothing passes a start, where
// cut is not 0.
template <bool FLAGS>
__device__ __forceinline__ float serial_pass(float dt, float cut, float A2, float h) {
    const float r = times_exp2(h, dt * A2);
    return FLAGS && cut != 0.f ? 0.f : r;
}

// Serial steps: the state that enters each lane, from the one that enters the row: h =
// a_k h + b_k over each lane's steps in turn.  After i turns lane i holds its own.
template <bool FLAGS, int L>
__device__ __forceinline__ float serial_enter(const float (&dt)[kScanK],
                                              const float (&cut)[kScanK],
                                              const float (&b)[kScanK], float A2, float enter,
                                              int lane) {
    float in = enter;
    if constexpr (L > 1)
#pragma unroll 1
        for (int i = 1; i < L; ++i) {
            float h = in;
#pragma unroll
            for (int k = 0; k < kScanK; ++k) h = serial_pass<FLAGS>(dt[k], cut[k], A2, h) + b[k];
            in = row_shift<false, L>(h, enter, lane);
        }
    return in;
}

// The same for gradients, from the last lane and step to the first: r = a_k (c_k + r).
template <bool FLAGS, int L>
__device__ __forceinline__ float serial_enter_back(const float (&dt)[kScanK],
                                                   const float (&cut)[kScanK],
                                                   const float (&c)[kScanK], float A2,
                                                   float right, int lane) {
    float in = right;
    if constexpr (L > 1)
#pragma unroll 1
        for (int i = 1; i < L; ++i) {
            float r = in;
#pragma unroll
            for (int k = kScanK - 1; k >= 0; --k)
                r = serial_pass<FLAGS>(dt[k], cut[k], A2, c[k] + r);
            in = row_shift<true, L>(r, right, lane);
        }
    return in;
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

// The product of a lane's a's for one state: exp(A sum dt), or a start's 0 (-0 with
// CUT) where an episode starts in the lane, whatever the steps before the start hold.
template <bool FLAGS, bool CUT>
__device__ __forceinline__ float lane_product(float dt_sum, bool starts, float A2) {
    const float a = exp2_fast(dt_sum * A2);
    return FLAGS && starts ? (CUT ? -0.f : 0.f) : a;
}

// a_k of a lane's steps for one state, A2 = A log2(e); at a start 0, or -0 with CUT
// (cut's sign).
template <bool FLAGS, bool CUT>
__device__ __forceinline__ float decay(float dt, float cut, float A2) {
    const float a = exp2_fast(FLAGS ? fmaf(dt, A2, cut) : dt * A2);
    return CUT ? from_bits<float>(as_bits(a) | (as_bits(cut) & (int)0x80000000)) : a;
}

// Tame values: too small for any state, gradient or product of the scans to
// overflow within a tile.  With products of a's up to 2^kMostGrowth, dt u, B, C and
// gy below 2^40 and entering values below 2^100, sums over a tile's steps stay
// below 2^117.  A NaN is not tame.
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

// Whether a lane's steps are: dt and dt u small.
template <int K>
__device__ __forceinline__ bool steps_tame(const float (&dt)[K], const float (&dtu)[K]) {
    bool ok = true;
#pragma unroll
    for (int k = 0; k < K; ++k)
        ok &= tame(dt[k], kTameStep) && tame(dtu[k], kTameStep);
    return ok;
}

int lanes_of(const rlca_scan_call &c);
ScanParams scan_params(const rlca_scan_call &c, int rows);
rlca_status check_scan(const rlca_scan_call &c, bool backward, Arrays *a);

}  // namespace seq
}  // namespace rlca
