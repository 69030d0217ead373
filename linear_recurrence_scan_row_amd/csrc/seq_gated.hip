// seq_gated.hip -- the gated linear recurrence over rows of T steps, its gradients,
// and its single step:
//   r = sigmoid(decay_gate + decay_bias),  i = sigmoid(input_gate + input_bias),
//   L = scale softplus(decay) r,  a = exp(-L),
//   h_t = a_t h_{t-1} + sqrt(1 - a_t^2) i_t x_t.
//
// The affine recurrence of this library, one state a channel.  A row of 64, 16, 4 or
// 1 lanes owns a channel and a tile of 8 steps a lane: each lane folds its 8 maps
// into one, lane-crossing moves scan the maps, and each lane applies its own steps
// again from the state that enters it.  A wave owns 1, 4, 16 or 64 neighbouring
// channels and walks tiles and then sequences, the next tile's loads issued before
// this one is computed.  Where there are few rows, the waves of a workgroup share a
// row, tile after tile, and hand their maps to each other through LDS; where there are
// very few, a row is cut into chunks: one launch leaves each chunk's map, the second
// starts each chunk from the maps before it.
//
// Bound by memory: three or four values are read for each that is computed, beside 5
// transcendental instructions and about 26 others a step forward (5 and 67 backward),
// whose issue takes as long as the bytes where values have 16 bits.  Measured: 8x2048
// channels of 2048 steps bf16 forward 54 us and gradients 99 (5.0 and 4.7 TB/s), each
// alone, 62 and 87 (4.3 and 5.4) in turn, where the gradients find the forward call's
// inputs in the last-level cache;
// 4096x64 of 128 steps fp32 with flags 112 and 179 (4.8 and 5.3); one row set of 512x65535
// bf16 58 (4.6); a step of 512x8192 bf16 13 to 14 (5.1 to 4.6); a large copy reaches
// 5.05 TB/s.
#include "seq_scan.hpp"

namespace rlca {
namespace seq {

constexpr int kGateK = 8;        // steps of a lane
constexpr int kGateThreads = 256;
constexpr int kGateWaves = kGateThreads / kWave;
constexpr int gate_tile(int L) { return kGateK * L; }

struct GateParams {
    const void *x, *input_gate, *decay_gate, *grad_out;
    const float *decay, *input_bias, *decay_bias;
    const float *state, *grad_final;
    const uint8_t *flags;
    const int32_t *lengths;
    void *out;
    float *final_state;
    float *checkpoints;  // [num_seqs][channels][tiles]: states entering each tile
    void *grad_x, *grad_input, *grad_decay;
    float *grad_state;
    float *maps;      // [num_seqs][chunks][2][channels]: each chunk's map
    float *partials;  // [walkers * WAVES][3][channels]: sums for decay, decay_bias, input_bias
    int64_t x_n, x_d, ig_n, ig_d, dg_n, dg_d, g_n, g_d;
    uint32_t channels;
    uint32_t groups;      // waves that share a sequence's channels
    uint32_t walkers;     // waves (or workgroups) that share a group's sequences and chunks
    uint32_t units;       // num_seqs * chunks
    uint32_t chunks, chunk_tiles;
    int32_t T, tiles;
    int32_t after_done;
    float scale;
    FastDiv by_chunks;
};

// --------------------------------------------------------------- the arithmetic
// scale softplus(decay), and what a step's L = slow r may be at most: below, L a^2
// and its like are 0 where a is, not infinity times 0.
__device__ __forceinline__ float slow_of(float scale, float decay) {
    const float s = scale * softplus(decay);
    return s > 1e30f ? 1e30f : s;  // a NaN stays one
}

// A step's a = exp(-L) and 1 - a^2 = (1 - a)(1 + a).  Near L = 0 the difference 1 - a
// would lose digits, so up to 1/2 it is L times the polynomial that interpolates
// (1 - exp(-L)) / L there at 6 Chebyshev points (error 2.6e-9, with its coefficients in
// float32), and a is 1 minus it; from there on a is the exponential, and the difference
// of at least 0.39 loses none.  SLOW: no L of the wave's channels is above 1/8, where 4
// points do (error 3.1e-8).
constexpr float kSlow = 0.125f;
template <bool SLOW>
__device__ __forceinline__ void decay_of(float L, float &a, float &rest) {
    float d;
    if constexpr (SLOW) {
        d = fmaf(L, -0.039641775f, 0.16650987f);
        d = fmaf(L, d, -0.4999961f);
        d = fmaf(L, d, 1.f);
    } else {
        d = fmaf(L, -0.0011234042f, 0.0081896136f);
        d = fmaf(L, d, -0.041630073f);
        d = fmaf(L, d, 0.16666242f);
        d = fmaf(L, d, -0.49999982f);
        d = fmaf(L, d, 1.f);
    }
    d *= L;
    a = 1.f - d;
    if constexpr (!SLOW) {
        const float e = exp2_fast(-L * kLog2e);
        a = L > 0.5f ? e : a;
        d = L > 0.5f ? 1.f - e : d;
    }
    rest = fmaf(d, a, d);
}

// Inclusive scan of the lane maps of a row of L lanes, towards higher lanes or,
// REVERSE, towards lower ones; lanes whose source is outside the row keep theirs.
// CUT as for step_map: an episode start's a is -0.  A product of decays that has
// underflowed is 0, and makes NaN of an infinity that passes; nothing hides either.
//
// Without cuts a step of 16 lanes is two instructions, an FMA and a product that fetch
// their operand from the other lane themselves, and a wait: the hardware wants two
// instructions between a write and the lane-crossing read of it.
#define RLCA_GATE_STEP(MOVE, ROWS)                                    \
    "v_fmac_f32_dpp %1, %1, %0 " MOVE " row_mask:" ROWS " bank_mask:0xf\n\t" \
    "v_mul_f32_dpp %0, %0, %0 " MOVE " row_mask:" ROWS " bank_mask:0xf\n\t"  \
    "s_nop 1\n\t"

template <bool CUT, bool REVERSE, int L>
__device__ __forceinline__ void lanes_scan(float &a, float &h, int lane) {
    if constexpr (L == 4) {
        const auto step = [&](auto by) {
            constexpr int kStep = decltype(by)::value;
            constexpr int kCtrl = shift_ctrl<4, REVERSE, kStep>();
            const bool has = REVERSE ? lane + kStep < 4 : lane >= kStep;
            const float ph = dpp_move<kCtrl, 0xf>(h, h), pa = dpp_move<kCtrl, 0xf>(a, a);
            h = has ? step_map<CUT>(a, h, ph) : h;
            a = has ? product<CUT>(a, pa) : a;
        };
        step(std::integral_constant<int, 1>{});
        step(std::integral_constant<int, 2>{});
    } else if constexpr (L >= 16) {
        const auto step = [&](auto ctrl, auto rows) {
            constexpr int kCtrl = decltype(ctrl)::value, kRows = decltype(rows)::value;
            const float ph = dpp_move<kCtrl, kRows>(h, 0.f), pa = dpp_move<kCtrl, kRows>(a, 1.f);
            h = step_map<CUT>(a, h, ph);
            a = product<CUT>(a, pa);
        };
        if constexpr (CUT) {
            const std::integral_constant<int, 0xf> all;
            step(std::integral_constant<int, shift_ctrl<16, REVERSE, 1>()>{}, all);
            step(std::integral_constant<int, shift_ctrl<16, REVERSE, 2>()>{}, all);
            step(std::integral_constant<int, shift_ctrl<16, REVERSE, 4>()>{}, all);
            step(std::integral_constant<int, shift_ctrl<16, REVERSE, 8>()>{}, all);
        } else if constexpr (REVERSE) {
            asm("s_nop 1\n\t" RLCA_GATE_STEP("row_shl:1", "0xf") RLCA_GATE_STEP("row_shl:2", "0xf")
                    RLCA_GATE_STEP("row_shl:4", "0xf") RLCA_GATE_STEP("row_shl:8", "0xf")
                : "+v"(a), "+v"(h));
        } else {
            asm("s_nop 1\n\t" RLCA_GATE_STEP("row_shr:1", "0xf") RLCA_GATE_STEP("row_shr:2", "0xf")
                    RLCA_GATE_STEP("row_shr:4", "0xf") RLCA_GATE_STEP("row_shr:8", "0xf")
                : "+v"(a), "+v"(h));
        }
        if constexpr (L == 64 && !REVERSE) {
            // the runs of 16 lanes: the last lane of the first and third to the next run,
            // then the last lane of the second to both others
            if constexpr (CUT) {
                step(std::integral_constant<int, 0x142>{}, std::integral_constant<int, 0xa>{});
                step(std::integral_constant<int, 0x143>{}, std::integral_constant<int, 0xc>{});
            } else {
                asm("s_nop 1\n\t" RLCA_GATE_STEP("row_bcast:15", "0xa")
                        RLCA_GATE_STEP("row_bcast:31", "0xc")
                    : "+v"(a), "+v"(h));
            }
        } else if constexpr (L == 64) {
            // the maps of the runs after each run, from the first lanes of those
            float na = read_lane(a, 48), nh = read_lane(h, 48);
            const int run = lane / 16;
            float ra = run == 2 ? na : 1.f, rh = run == 2 ? nh : 0.f;
#pragma unroll
            for (int at = 2; at > 0; --at) {
                const float pa = read_lane(a, 16 * at), ph = read_lane(h, 16 * at);
                nh = step_map<CUT>(pa, ph, nh);
                na = product<CUT>(pa, na);
                ra = run == at - 1 ? na : ra;
                rh = run == at - 1 ? nh : rh;
            }
            h = step_map<CUT>(a, h, rh);
            a = product<CUT>(a, ra);
        }
    }
}
#undef RLCA_GATE_STEP

// The value of the row's last lane in scan order, in all its lanes.
template <bool REVERSE, int L>
__device__ __forceinline__ float last_lane(float x) {
    if constexpr (L == 64) return read_lane(x, REVERSE ? 0 : 63);
    if constexpr (L == 1) return x;
    return row_last<REVERSE, L>(x);
}

// The lane's scanned map applied to what enters the row, moved on by one lane: what
// enters each lane.
template <bool REVERSE, int L>
__device__ __forceinline__ float next_lane(float after, float enter, int lane) {
    if constexpr (L == 64) return dpp_move<(REVERSE ? 0x130 : 0x138), 0xf>(after, enter);
    if constexpr (L == 1) return enter;
    return row_shift<REVERSE, L>(after, enter, lane);
}

// What enters a wave's tile, from the maps of the WAVES waves whose tiles lie side by
// side (REVERSE: from the last to the first), and what leaves them all.  The slots of
// LDS alternate, so one barrier a tile is enough.
template <bool CUT, bool REVERSE, int WAVES>
__device__ __forceinline__ float enter_wave(float a, float h, float (&lds)[2][WAVES][2], int &parity,
                                            int wave, float &carry) {
    if (threadIdx.x % kWave == 0) lds[parity][wave][0] = a, lds[parity][wave][1] = h;
    __syncthreads();
    float x = carry, enter = carry;
#pragma unroll
    for (int i = 0; i < WAVES; ++i) {
        const int w = REVERSE ? WAVES - 1 - i : i;
        if (w == wave) enter = x;
        x = step_map<CUT>(lds[parity][w][0], lds[parity][w][1], x);
    }
    parity ^= 1;
    carry = x;
    return enter;
}

// ------------------------------------------------------------------- the walk
// Where a workgroup (or a wave, where they work apart) stands: a unit, which is a
// sequence's chunk, and a tile of it, or as many tiles side by side as waves share it.
struct Place {
    uint32_t unit, n, chunk;
    int tile, end;  // end: the sequence's steps that count
    __device__ __forceinline__ void set_unit(const GateParams &p, uint32_t u) {
        unit = u;
        if (u >= p.units) return;
        n = p.chunks == 1 ? u : p.by_chunks.div(u);
        chunk = u - n * p.chunks;
        end = row_end(p.lengths, n, p.T);
    }
    __device__ __forceinline__ int first(const GateParams &p) const {
        return (int)(chunk * p.chunk_tiles);
    }
    // the last tile of the unit, of those that begin a step of the walk
    __device__ __forceinline__ int last(const GateParams &p, int waves) const {
        const int past = (int)((chunk + 1) * p.chunk_tiles);
        const int tiles = (past < p.tiles ? past : p.tiles) - first(p);
        return first(p) + (tiles - 1) / waves * waves;
    }
};

// The wave's channels: lane `lane` of the row of channel d.
struct GateLane {
    uint32_t d;
    int lane;
    bool live, slow_only;  // slow_only: all the wave's channels decay slowly
    float slow;            // scale softplus(decay)
    float input2, decay2;  // -log2(e) times the biases
    template <int L>
    __device__ __forceinline__ static GateLane of(const GateParams &p, uint32_t group) {
        GateLane l;
        const int in_wave = threadIdx.x % kWave;
        l.lane = in_wave & (L - 1);
        const uint32_t d = group * (kWave / L) + in_wave / L;
        l.live = d < p.channels;
        l.d = l.live ? d : p.channels - 1;
        l.slow = slow_of(p.scale, p.decay[l.d]);
        l.slow_only = whole_wave(l.slow <= kSlow);
        l.input2 = p.input_bias == nullptr ? 0.f : -kLog2e * p.input_bias[l.d];
        l.decay2 = p.decay_bias == nullptr ? 0.f : -kLog2e * p.decay_bias[l.d];
        return l;
    }
};

// A lane's episode starts in its steps from t on, as bits; none from `end` on.
__device__ __forceinline__ uint32_t gate_starts(const GateParams &p, uint32_t n, int t, int end) {
    if (t >= end) return 0;
    uint32_t s = start_bits<kGateK>(p.flags + (int64_t)n * p.T, t, p.T, p.after_done);
    if (t + kGateK > end) s &= (1u << (end - t)) - 1;
    return s;
}

// sigmoid(x + bias), shift = -log2(e) bias.
__device__ __forceinline__ float gate_of(float x, float shift) {
    return __builtin_amdgcn_rcpf(1.f + exp2_fast(fmaf(x, -kLog2e, shift)));
}

// A lane's 8 steps: the gates, and a and 1 - a^2 of the recurrence's maps.
struct GateSteps {
    float r[kGateK], a[kGateK], rest[kGateK];
    template <typename E>
    __device__ __forceinline__ void decays(const GateLane &l, const Steps<kGateK, E> &dgs) {
        dgs.widen(r);
#pragma unroll
        for (int k = 0; k < kGateK; ++k) r[k] = gate_of(r[k], l.decay2);
        if (l.slow_only) {
#pragma unroll
            for (int k = 0; k < kGateK; ++k) decay_of<true>(l.slow * r[k], a[k], rest[k]);
        } else {
#pragma unroll
            for (int k = 0; k < kGateK; ++k) decay_of<false>(l.slow * r[k], a[k], rest[k]);
        }
    }
};

template <typename E>
__device__ __forceinline__ void input_gates(const GateLane &l, const Steps<kGateK, E> &igs,
                                            float (&i)[kGateK]) {
    igs.widen(i);
#pragma unroll
    for (int k = 0; k < kGateK; ++k) i[k] = gate_of(i[k], l.input2);
}

// The state that enters a chunk: the row's state through the maps of the chunks
// before it.  (REVERSE: the gradient that enters from the chunks after it.)
template <bool REVERSE>
__device__ __forceinline__ float enter_chunk(const GateParams &p, uint32_t n, uint32_t chunk,
                                             uint32_t d, float x) {
    const float *m = p.maps + (int64_t)n * p.chunks * 2 * p.channels + d;
    const int count = REVERSE ? (int)(p.chunks - 1 - chunk) : (int)chunk;
#pragma unroll 4
    for (int j = 0; j < count; ++j) {
        const int64_t c = REVERSE ? (int64_t)p.chunks - 1 - j : j;
        const float *at = m + c * 2 * p.channels;
        x = step_map<true>(at[0], at[p.channels], x);
    }
    return x;
}

// Whether the step after a sequence's last one starts an episode: no state leaves it.
template <bool FLAGS>
__device__ __forceinline__ bool ends_over(const GateParams &p, uint32_t n, int end) {
    return FLAGS && p.after_done && end > 0 && p.flags[(int64_t)n * p.T + end - 1] != 0;
}

constexpr int threads_of(int waves) { return waves > 1 ? waves * kWave : kGateThreads; }

// Which of the launch's units of work a wave is: waves that work apart, or a workgroup.
template <int WAVES>
__device__ __forceinline__ uint32_t gate_worker(int &wave) {
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    wave = WAVES > 1 ? w : 0;
    return WAVES > 1 ? blockIdx.x : blockIdx.x * kGateWaves + w;
}

// ------------------------------------------------------------------- forward
// MAPS: leave each chunk's map only.
template <typename E, bool FLAGS, int L, int WAVES, bool MAPS>
__global__ __launch_bounds__(threads_of(WAVES)) void gated_rows(GateParams p) {
    constexpr int K = kGateK, kTile = gate_tile(L);
    __shared__ float lds[2][WAVES][2];
    int wave, parity = 0;
    const uint32_t worker = gate_worker<WAVES>(wave);
    const uint32_t walker = worker / p.groups, group = worker - walker * p.groups;
    if (walker >= p.walkers) return;
    const GateLane l = GateLane::of<L>(p, group);
    const int own = wave * kTile + l.lane * K;

    struct Loads {
        Steps<K, E> x, ig, dg;
    } next;
    const auto load = [&](const Place &at) {
        const int t = at.tile * kTile + own, left = at.end - t;
        next.x.load(static_cast<const E *>(p.x) + at.n * p.x_n + l.d * p.x_d + t, left);
        next.ig.load(static_cast<const E *>(p.input_gate) + at.n * p.ig_n + l.d * p.ig_d + t, left);
        next.dg.load(static_cast<const E *>(p.decay_gate) + at.n * p.dg_n + l.d * p.dg_d + t, left);
    };
    // The last chunk's map is not needed.
    const auto next_unit = [&](Place &at, uint32_t u) {
        at.set_unit(p, u);
        while (MAPS && at.unit < p.units && at.chunk + 1 == p.chunks)
            at.set_unit(p, at.unit + p.walkers);
    };
    Place at;
    next_unit(at, walker);
    if (at.unit >= p.units) return;
    at.tile = at.first(p);
    load(at);
    float carry = 0.f, map = 1.f;
    bool fresh = true;
    while (true) {
        const int64_t row = (int64_t)at.n * p.channels + l.d;
        const int t0 = at.tile * kTile + wave * kTile, t = at.tile * kTile + own;
        if (fresh) {
            if constexpr (MAPS) {
                carry = 0.f;
                map = 1.f;
            } else {
                carry = p.state == nullptr ? 0.f : p.state[row];
                if (p.chunks > 1) carry = enter_chunk<false>(p, at.n, at.chunk, l.d, carry);
            }
        }
        const Loads now = next;
        uint32_t starts = 0;
        if constexpr (FLAGS) starts = gate_starts(p, at.n, t, at.end);
        // the place after this one, and its loads
        Place ahead = at;
        const bool last = at.tile == at.last(p, WAVES);
        if (last) {
            next_unit(ahead, ahead.unit + p.walkers);
            ahead.tile = ahead.unit < p.units ? ahead.first(p) : 0;
        } else {
            ahead.tile += WAVES;
        }
        if (ahead.unit < p.units) load(ahead);

        GateSteps s;
        float x[K], i[K], b[K];
        s.decays(l, now.dg);
        now.x.widen(x);
        input_gates(l, now.ig, i);
#pragma unroll
        for (int k = 0; k < K; ++k) b[k] = __builtin_amdgcn_sqrtf(s.rest[k]) * (i[k] * x[k]);
        const bool partial = t0 + kTile > at.end;
        if (partial)
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (t + k >= at.end) s.a[k] = 1.f, b[k] = 0.f;
        float a = s.a[0], fold = b[0];
#pragma unroll
        for (int k = 1; k < K; ++k) {
            if (FLAGS && (starts >> k & 1)) fold = 0.f;
            fold = fmaf(s.a[k], fold, b[k]);
            a *= s.a[k];
        }
        if (FLAGS && starts != 0) a = -0.f;
        lanes_scan<FLAGS, false, L>(a, fold, l.lane);
        float enter = carry;
        if constexpr (WAVES > 1)
            enter = enter_wave<FLAGS, false, WAVES>(last_lane<false, L>(a), last_lane<false, L>(fold),
                                                    lds, parity, wave, carry);
        if (!MAPS && p.checkpoints != nullptr && l.live && l.lane == 0 &&
            (WAVES == 1 || at.tile + wave < p.tiles))
            p.checkpoints[row * p.tiles + at.tile + wave] = enter;
        const float after = step_map<FLAGS>(a, fold, enter);
        float h = next_lane<false, L>(after, enter, l.lane);
        if constexpr (WAVES == 1) carry = last_lane<false, L>(after);
        if constexpr (MAPS) {
            map = product<FLAGS>(last_lane<false, L>(a), map);
            if (last && l.live && l.lane == 0) {
                float *m = p.maps + ((int64_t)at.n * p.chunks + at.chunk) * 2 * p.channels + l.d;
                m[0] = map;
                m[p.channels] = carry;
            }
        } else {
            float out[K];
#pragma unroll
            for (int k = 0; k < K; ++k) {
                if (FLAGS && (starts >> k & 1)) h = 0.f;
                h = fmaf(s.a[k], h, b[k]);
                out[k] = h;
            }
            if (partial)
#pragma unroll
                for (int k = 0; k < K; ++k)
                    if (t + k >= at.end) out[k] = 0.f;
            if (l.live) store_steps<K>(static_cast<E *>(p.out) + row * p.T + t, p.T - t, out);
            if (last && at.chunk + 1 == p.chunks && p.final_state != nullptr && l.live &&
                l.lane == 0 && wave == 0)
                p.final_state[row] = ends_over<FLAGS>(p, at.n, at.end) ? 0.f : carry;
        }
        if (ahead.unit >= p.units) return;
        fresh = last;
        at = ahead;
    }
}

// ------------------------------------------------------------------- backward
// With lambda_t = grad_t + a_{t+1} lambda_{t+1} the gradient of h_t, beta = sqrt(1 - a^2)
// and inv = 1 / beta:
//   grad_x = lambda beta i,   grad_input_gate = grad_x x (1 - i),
//   e = dL/d(log decay's rate) = lambda L a (a inv i x - h_{t-1}),
//   grad_decay_gate = e (1 - r),  grad_decay = sum e sigmoid(decay) / softplus(decay).
// The states are computed again, from the state that entered the tile.  What passes a
// step to the left is a_t lambda_t, so a lane's map is r -> a_k (grad_k + r) over its
// steps from the last.
template <typename E, bool FLAGS, int L, int WAVES, bool MAPS>
__global__ __launch_bounds__(threads_of(WAVES), sizeof(E) == 2 ? 4 : 3) void gated_rows_backward(GateParams p) {
    constexpr int K = kGateK, kTile = gate_tile(L);
    __shared__ float lds[2][WAVES][2];
    int wave, parity = 0;
    const uint32_t worker = gate_worker<WAVES>(wave);
    const uint32_t walker = worker / p.groups, group = worker - walker * p.groups;
    if (walker >= p.walkers) return;
    const GateLane l = GateLane::of<L>(p, group);
    const int own = wave * kTile + l.lane * K;

    struct Loads {
        Steps<K, E> x, ig, dg, g;
        float enter;
    } next;
    const auto load = [&](const Place &at) {
        const int t = at.tile * kTile + own, left = at.end - t;
        // formed here each time: kept, the rows' addresses would take registers from a wave
        const uint32_t d = here(l.d);
        next.dg.load(static_cast<const E *>(p.decay_gate) + at.n * p.dg_n + d * p.dg_d + t, left);
        next.g.load(static_cast<const E *>(p.grad_out) + at.n * p.g_n + d * p.g_d + t, left);
        if constexpr (!MAPS) {
            next.x.load(static_cast<const E *>(p.x) + at.n * p.x_n + d * p.x_d + t, left);
            next.ig.load(static_cast<const E *>(p.input_gate) + at.n * p.ig_n + d * p.ig_d + t,
                         left);
            next.enter = 0.f;
            if (WAVES == 1 || at.tile + wave < p.tiles)
                next.enter = p.checkpoints[((int64_t)at.n * p.channels + l.d) * p.tiles + at.tile +
                                           wave];
        }
    };
    // The first chunk's map is not needed.
    const auto next_unit = [&](Place &at, uint32_t u) {
        at.set_unit(p, u);
        while (MAPS && at.unit < p.units && at.chunk == 0) at.set_unit(p, at.unit + p.walkers);
    };
    float sum_decay = 0.f, sum_rate = 0.f, sum_input = 0.f;
    Place at;
    next_unit(at, walker);
    if (MAPS && at.unit >= p.units) return;
    if (at.unit < p.units) {
        at.tile = at.last(p, WAVES);
        load(at);
    }
    float carry = 0.f, map = 1.f;
    bool fresh = true;
    while (at.unit < p.units) {
        const int64_t row = (int64_t)at.n * p.channels + l.d;
        const int t0 = at.tile * kTile + wave * kTile, t = at.tile * kTile + own;
        if (fresh) {
            carry = 0.f;
            map = 1.f;
            if constexpr (!MAPS) {
                if (p.grad_final != nullptr && !ends_over<FLAGS>(p, at.n, at.end))
                    carry = p.grad_final[row];
                if (p.chunks > 1) carry = enter_chunk<true>(p, at.n, at.chunk, l.d, carry);
            }
        }
        const Loads now = next;
        uint32_t starts = 0;
        if constexpr (FLAGS) starts = gate_starts(p, at.n, t, at.end);
        Place ahead = at;
        const bool last = at.tile == at.first(p);
        if (last) {
            next_unit(ahead, ahead.unit + p.walkers);
            ahead.tile = ahead.unit < p.units ? ahead.last(p, WAVES) : 0;
        } else {
            ahead.tile -= WAVES;
        }
        if (ahead.unit < p.units) load(ahead);

        float g[K];
        now.g.widen(g);
        GateSteps s;
        s.decays(l, now.dg);
        const bool partial = t0 + kTile > at.end;
        if (partial)
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (t + k >= at.end) s.a[k] = 1.f;
        float whole = s.a[0];
#pragma unroll
        for (int k = 1; k < K; ++k) whole *= s.a[k];
        if (FLAGS && starts != 0) whole = -0.f;
        float a = whole, back = 0.f;
#pragma unroll
        for (int k = K - 1; k >= 0; --k) {
            back = s.a[k] * (g[k] + back);
            if (FLAGS && (starts >> k & 1)) back = 0.f;
        }
        lanes_scan<FLAGS, true, L>(a, back, l.lane);
        float right = carry;
        if constexpr (WAVES > 1)
            right = enter_wave<FLAGS, true, WAVES>(last_lane<true, L>(a), last_lane<true, L>(back),
                                                   lds, parity, wave, carry);
        const float after = step_map<FLAGS>(a, back, right);
        float pass = next_lane<true, L>(after, right, l.lane);
        if constexpr (WAVES == 1) carry = last_lane<true, L>(after);
        if constexpr (MAPS) {
            map = product<FLAGS>(last_lane<true, L>(a), map);
            if (last && l.live && l.lane == 0) {
                float *m = p.maps + ((int64_t)at.n * p.chunks + at.chunk) * 2 * p.channels + l.d;
                m[0] = map;
                m[p.channels] = carry;
            }
        } else {
            // lambda's factors in grad_x, and grad_x's in grad_input_gate; the input
            float beta_i[K], rest_x[K], in[K], q[K];
            {
                float x[K], i[K];
                now.x.widen(x);
                input_gates(l, now.ig, i);
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    const float rest = s.rest[k];
                    const float inv = __builtin_amdgcn_rsqf(rest < 1.2e-38f ? 1.2e-38f : rest);
                    beta_i[k] = rest * inv * i[k];
                    if (partial && t + k >= at.end) beta_i[k] = 0.f;
                    in[k] = beta_i[k] * x[k];
                    q[k] = s.a[k] * inv * (i[k] * x[k]);
                    rest_x[k] = x[k] * (1.f - i[k]);
                }
            }
            float fold = 0.f;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                if (FLAGS && (starts >> k & 1)) fold = 0.f;
                fold = fmaf(s.a[k], fold, in[k]);
            }
            a = whole;
            lanes_scan<FLAGS, false, L>(a, fold, l.lane);
            float h = next_lane<false, L>(step_map<FLAGS>(a, fold, now.enter), now.enter, l.lane);
#pragma unroll
            for (int k = 0; k < K; ++k) {
                if (FLAGS && (starts >> k & 1)) h = 0.f;
                q[k] -= h;
                h = fmaf(s.a[k], h, in[k]);
            }
            float gx[K], gi[K], gr[K];
#pragma unroll
            for (int k = K - 1; k >= 0; --k) {
                const float lambda = g[k] + pass;
                pass = s.a[k] * lambda;
                const float e = pass * (l.slow * s.r[k]) * q[k];
                if (FLAGS && (starts >> k & 1)) pass = 0.f;
                gx[k] = lambda * beta_i[k];
                gi[k] = gx[k] * rest_x[k];
                gr[k] = e * (1.f - s.r[k]);
                if (partial && t + k >= at.end) {
                    gx[k] = gi[k] = gr[k] = 0.f;
                } else {
                    sum_decay += e;
                    sum_rate += gr[k];
                    sum_input += gi[k];
                }
            }
            if (l.live) {
                store_steps<K>(static_cast<E *>(p.grad_x) + row * p.T + t, p.T - t, gx);
                store_steps<K>(static_cast<E *>(p.grad_input) + row * p.T + t, p.T - t, gi);
                store_steps<K>(static_cast<E *>(p.grad_decay) + row * p.T + t, p.T - t, gr);
            }
            if (last && at.chunk == 0 && p.grad_state != nullptr && l.live && l.lane == 0 &&
                wave == 0)
                p.grad_state[row] = carry;
        }
        fresh = last;
        at = ahead;
    }
    if constexpr (!MAPS) {
#pragma unroll
        for (int m = 1; m < L; m <<= 1) {
            sum_decay += __shfl_xor(sum_decay, m);
            sum_rate += __shfl_xor(sum_rate, m);
            sum_input += __shfl_xor(sum_input, m);
        }
        if (l.live && l.lane == 0) {
            float *to = p.partials + ((int64_t)walker * WAVES + wave) * 3 * p.channels + l.d;
            to[0] = sum_decay;
            to[p.channels] = sum_rate;
            to[2 * (int64_t)p.channels] = sum_input;
        }
    }
}

// The walkers' sums in order: a workgroup takes 64 of the 3 * channels columns, its
// 16 waves every 16th walker each.
struct GateSums {
    const float *partials, *decay;
    float *grad_decay, *grad_rate, *grad_input;
    uint32_t walkers, channels;
};
constexpr int kGateSumWaves = 16;

__global__ __launch_bounds__(kGateSumWaves *kWave) void gated_sums(GateSums p) {
    __shared__ float sums[kGateSumWaves][kWave];
    const uint32_t wave = threadIdx.x / kWave, lane = threadIdx.x % kWave;
    const uint64_t columns = 3 * (uint64_t)p.channels, c = (uint64_t)blockIdx.x * kWave + lane;
    float sum = 0.f;
    if (c < columns)
#pragma unroll 8
        for (uint32_t w = wave; w < p.walkers; w += kGateSumWaves) sum += p.partials[w * columns + c];
    sums[wave][lane] = sum;
    __syncthreads();
    if (wave != 0 || c >= columns) return;
    for (int w = 1; w < kGateSumWaves; ++w) sum += sums[w][lane];
    if (c < p.channels) {
        // dL/d(decay): the rate's derivative over the rate, 1 where both underflow
        const float x = p.decay[c];
        p.grad_decay[c] = sum * (x < -16.f ? 1.f : sigmoid(x) / softplus(x));
    } else if (c < 2 * (uint64_t)p.channels) {
        if (p.grad_rate != nullptr) p.grad_rate[c - p.channels] = sum;
    } else if (p.grad_input != nullptr) {
        p.grad_input[c - 2 * (uint64_t)p.channels] = sum;
    }
}

// ------------------------------------------------------------------ single steps
struct GateStepParams {
    const void *x, *input_gate, *decay_gate;
    const float *decay, *input_bias, *decay_bias;
    float *state;
    const int32_t *slots;
    const uint8_t *starts;
    void *out;
    int64_t x_n, ig_n, dg_n, places;
    uint32_t num_seqs, channels;
    float scale;
};

constexpr int kGateStepThreads = 256;

__device__ __forceinline__ int64_t gate_place(const GateStepParams &p, uint32_t n) {
    if (n >= p.num_seqs) return -1;
    if (p.slots == nullptr) return n;
    const int64_t s = p.slots[n];
    return s >= 0 && s < p.places ? s : -1;
}

// A thread takes a channel of the sequences blockIdx.y, blockIdx.y + gridDim.y, ..., the
// next one's loads issued before one is computed.  (Four channels a thread: 512x8192
// bf16 14.2 us against 13.2, 64x4096 3.7 against 3.3.)
template <typename E>
__global__ __launch_bounds__(kGateStepThreads) void gated_step(GateStepParams p) {
    const uint32_t d = blockIdx.x * blockDim.x + threadIdx.x;
    if (d >= p.channels) return;
    struct Loads {
        int64_t place;
        E x, ig, dg;
        float h;
    } next;
    const auto load = [&](uint32_t n) {
        next.place = gate_place(p, n);
        if (next.place < 0) return;
        next.x = static_cast<const E *>(p.x)[n * p.x_n + d];
        next.ig = static_cast<const E *>(p.input_gate)[n * p.ig_n + d];
        next.dg = static_cast<const E *>(p.decay_gate)[n * p.dg_n + d];
        next.h = p.starts != nullptr && p.starts[n] != 0 ? 0.f
                                                         : p.state[next.place * p.channels + d];
    };
    load(blockIdx.y);
    const float slow = slow_of(p.scale, p.decay[d]);
    const float input2 = p.input_bias == nullptr ? 0.f : -kLog2e * p.input_bias[d];
    const float decay2 = p.decay_bias == nullptr ? 0.f : -kLog2e * p.decay_bias[d];
    for (uint32_t n = blockIdx.y; n < p.num_seqs; n += gridDim.y) {
        const Loads now = next;
        if (n + gridDim.y < p.num_seqs) load(n + gridDim.y);
        float out = 0.f;
        if (now.place >= 0) {
            float a, rest;
            decay_of<false>(slow * gate_of((float)now.dg, decay2), a, rest);
            const float in = __builtin_amdgcn_sqrtf(rest) * (gate_of((float)now.ig, input2) * (float)now.x);
            out = fmaf(a, now.h, in);
            p.state[now.place * p.channels + d] = out;
        }
        static_cast<E *>(p.out)[(int64_t)n * p.channels + d] = (E)out;
    }
}

// ------------------------------------------------------------------- host side
// How a call is launched.  Rows of up to 8 steps take a lane, up to 32 four, others 16,
// or a whole wave where its wider tiles waste less than a fifth more lanes at the row's
// end (8x2048 channels of 2048 steps, bf16, each call alone in a row: forward 54 us
// against 58, gradients 99 against 131; 32x1024 of 600 steps the other way 55 against 37
// and 86 against 69), or where waves are few, up to kFewWaves of 16-lane rows.  From kFewRows rows down the
// kShared waves of a workgroup share a row (512 rows of 65535 steps: 71 us against 198
// apart and 114 in chunks; 4096 rows of 8191 steps 74 against 56 apart); from
// kFewestRows down rows are cut into chunks of at least kFewestTiles tiles, at most
// kMostChunks (64 rows of 131072 steps 48 us against 60 shared, 96 of 65536 33 and 33,
// 128 36 against 33).
constexpr int64_t kFewWaves = 2048;
constexpr int64_t kFewRows = 2048;
constexpr int64_t kFewestRows = 96;
constexpr int64_t kFewestTiles = 4;
constexpr int64_t kMostChunks = 64;
constexpr int kShared = 8;

// Waves that a launch wants: 4 on each of the 1024 SIMDs, or the 3 that the registers of
// the backward kernel leave where values are float32.
constexpr int64_t kSimds = 1024;
static int64_t gate_wanted(const rlca_gated_call &c, bool backward) {
    return (backward && c.dtype == RLCA_F32 ? 3 : 4) * kSimds;
}

struct GatePlan {
    int L, waves;
    int64_t tiles, groups, chunks, chunk_tiles, units, walkers;
};

static GatePlan gate_plan(const rlca_gated_call &c, bool backward) {
    GatePlan g = {};
    const int64_t wanted = gate_wanted(c, backward);
    const int64_t rows = c.num_seqs * c.channels;
    const auto per_wave = [&](int lanes) { return kWave / lanes; };
    const auto groups = [&](int lanes) {
        return (c.channels + per_wave(lanes) - 1) / per_wave(lanes);
    };
    g.L = c.T <= gate_tile(1) ? 1 : c.T <= gate_tile(4) ? 4 : 16;
    g.waves = 1;
    const bool few = groups(16) * c.num_seqs <= kFewWaves;
    const bool chunked = few && rows <= kFewestRows && c.T >= 2 * kFewestTiles * gate_tile(16);
    const auto padded = [&](int lanes) {
        return (c.T + gate_tile(lanes) - 1) / gate_tile(lanes) * gate_tile(lanes);
    };
    if (g.L == 16 && !chunked &&
        ((few && c.T > gate_tile(16)) || 5 * padded(64) <= 6 * padded(16))) {
        g.L = 64;
        if (rows <= kFewRows && c.T > kShared / 2 * gate_tile(64)) g.waves = kShared;
    }
    g.tiles = (c.T + gate_tile(g.L) - 1) / gate_tile(g.L);
    g.groups = groups(g.L);
    g.chunks = 1;
    if (chunked && rows > 0) {
        int64_t want = 4 * kSimds / (g.groups * c.num_seqs);
        if (want > g.tiles / kFewestTiles) want = g.tiles / kFewestTiles;
        if (want > kMostChunks) want = kMostChunks;
        g.chunks = want;
    }
    g.chunk_tiles = (g.tiles + g.chunks - 1) / g.chunks;
    if (g.chunk_tiles > 0) g.chunks = (g.tiles + g.chunk_tiles - 1) / g.chunk_tiles;
    g.units = c.num_seqs * g.chunks;
    g.walkers = g.groups == 0 ? 0 : (wanted / g.waves + g.groups - 1) / g.groups;
    if (g.walkers > g.units) g.walkers = g.units;
    if (g.walkers > 0) {  // as many units for each, as far as possible
        const int64_t rounds = (g.units + g.walkers - 1) / g.walkers;
        g.walkers = (g.units + rounds - 1) / rounds;
    }
    return g;
}

static GateParams gate_params(const rlca_gated_call &c, const GatePlan &g) {
    GateParams p = {};
    p.x = c.x, p.input_gate = c.input_gate, p.decay_gate = c.decay_gate;
    p.grad_out = c.grad_out;
    p.decay = c.decay, p.input_bias = c.input_bias, p.decay_bias = c.decay_bias;
    p.state = c.state, p.grad_final = c.grad_final_state;
    p.flags = c.flags, p.lengths = c.lengths;
    p.out = c.out, p.final_state = c.final_state, p.checkpoints = c.checkpoints;
    p.grad_x = c.grad_x, p.grad_input = c.grad_input_gate, p.grad_decay = c.grad_decay_gate;
    p.grad_state = c.grad_state;
    p.x_n = c.x_stride_seq, p.x_d = c.x_stride_channel;
    p.ig_n = c.input_stride_seq, p.ig_d = c.input_stride_channel;
    p.dg_n = c.decay_stride_seq, p.dg_d = c.decay_stride_channel;
    p.g_n = c.grad_stride_seq, p.g_d = c.grad_stride_channel;
    p.channels = (uint32_t)c.channels;
    p.groups = (uint32_t)g.groups;
    p.walkers = (uint32_t)g.walkers;
    p.units = (uint32_t)g.units;
    p.chunks = (uint32_t)g.chunks;
    p.chunk_tiles = (uint32_t)g.chunk_tiles;
    p.T = (int32_t)c.T;
    p.tiles = (int32_t)g.tiles;
    p.after_done = c.convention == RLCA_RESET_AFTER_DONE;
    p.scale = (float)c.scale;
    p.by_chunks = fast_div((uint32_t)g.chunks);
    return p;
}

template <typename E, int L, int WAVES, bool MAPS>
static const void *gate_kernel(bool backward, bool flags) {
    if (backward)
        return flags ? (const void *)gated_rows_backward<E, true, L, WAVES, MAPS>
                     : (const void *)gated_rows_backward<E, false, L, WAVES, MAPS>;
    return flags ? (const void *)gated_rows<E, true, L, WAVES, MAPS>
                 : (const void *)gated_rows<E, false, L, WAVES, MAPS>;
}

// Chunks exist for rows of 16 lanes only.
template <typename E>
static const void *gate_kernel(bool backward, bool flags, const GatePlan &g, bool maps) {
    return maps          ? gate_kernel<E, 16, 1, true>(backward, flags)
           : g.waves > 1 ? gate_kernel<E, 64, kShared, false>(backward, flags)
           : g.L == 64   ? gate_kernel<E, 64, 1, false>(backward, flags)
           : g.L == 16   ? gate_kernel<E, 16, 1, false>(backward, flags)
           : g.L == 4    ? gate_kernel<E, 4, 1, false>(backward, flags)
                         : gate_kernel<E, 1, 1, false>(backward, flags);
}

static rlca_status gate_launch(const rlca_gated_call &c, const GatePlan &g, GateParams &p,
                               bool backward, bool maps, hipStream_t stream) {
    const bool flags = c.flags != nullptr;
    const void *kernel = c.dtype == RLCA_F32    ? gate_kernel<float>(backward, flags, g, maps)
                         : c.dtype == RLCA_BF16 ? gate_kernel<__bf16>(backward, flags, g, maps)
                                                : gate_kernel<_Float16>(backward, flags, g, maps);
    const uint64_t workers = (uint64_t)g.groups * g.walkers;
    const uint64_t blocks = g.waves > 1 ? workers : (workers + kGateWaves - 1) / kGateWaves;
    return launch(kernel, dim3((uint32_t)blocks), threads_of(g.waves), 0, p, stream);
}

// The walkers' sums.
static size_t gate_partials_bytes(const rlca_gated_call &c, const GatePlan &g) {
    return (size_t)g.walkers * g.waves * 3 * c.channels * sizeof(float);
}

static size_t gate_maps_bytes(const rlca_gated_call &c, const GatePlan &g) {
    return g.chunks > 1 ? (size_t)c.num_seqs * g.chunks * 2 * c.channels * sizeof(float) : 0;
}

static size_t gate_checkpoints_bytes(const rlca_gated_call &c, const GatePlan &g) {
    return (size_t)c.num_seqs * c.channels * g.tiles * sizeof(float);
}

// The launch's threads stay below 2^32, and so do the units.
static bool gate_sizes_ok(const rlca_gated_call &c) {
    return sizes_ok(c.num_seqs, c.channels, c.T) && c.channels < (int64_t)1 << 25;
}

static bool gate_values_ok(int dtype, double scale) {
    // scale > 0 in float32, so that the decay's gradient has a rate to be relative to
    return element_bytes(dtype) != 0 && scale >= 1e-30 && scale <= 1e30;
}

static rlca_status check_gated(const rlca_gated_call &c, bool backward, Arrays &a) {
    if (!gate_sizes_ok(c)) return RLCA_ERR_INVALID_SIZE;
    if (!gate_values_ok(c.dtype, c.scale) ||
        (c.convention != RLCA_RESET_ON_START && c.convention != RLCA_RESET_AFTER_DONE))
        return RLCA_ERR_INVALID_VALUE;
    const int64_t N = c.num_seqs, D = c.channels, T = c.T;
    const size_t e = element_bytes(c.dtype);
    const int64_t params = N == 0 ? 0 : D;
    a.in(c.x, e, true, {{N, c.x_stride_seq}, {D, c.x_stride_channel}, {T, 1}});
    a.in(c.input_gate, e, true, {{N, c.input_stride_seq}, {D, c.input_stride_channel}, {T, 1}});
    a.in(c.decay_gate, e, true, {{N, c.decay_stride_seq}, {D, c.decay_stride_channel}, {T, 1}});
    a.in(c.decay, 4, true, {{backward ? D : params, 1}});
    a.in(c.input_bias, 4, false, {{params, 1}});
    a.in(c.decay_bias, 4, false, {{params, 1}});
    a.in(c.state, 4, false, {{N, D}, {D, 1}});
    a.in(c.flags, 1, false, {{N, T}, {T, 1}});
    a.in(c.lengths, 4, false, {{N, 1}});
    return RLCA_OK;
}

// What the walks' sums become; with no walkers the gradients of empty sums, 0.
static rlca_status launch_gate_sums(const rlca_gated_call &c, const float *partials,
                                    uint32_t walkers, hipStream_t stream) {
    GateSums p = {};
    p.partials = partials;
    p.decay = c.decay;
    p.grad_decay = c.grad_decay;
    p.grad_rate = c.grad_decay_bias;
    p.grad_input = c.grad_input_bias;
    p.walkers = walkers;
    p.channels = (uint32_t)c.channels;
    const uint64_t columns = 3 * (uint64_t)c.channels;
    return launch((const void *)gated_sums, dim3((uint32_t)((columns + kWave - 1) / kWave)),
                  kGateSumWaves * kWave, 0, p, stream);
}

// T = 0: the state goes on as it is (to: final_state or grad_state).
struct CopyParams {
    const float *from;
    float *to;
    uint64_t count;
};

__global__ __launch_bounds__(256) void gated_copy_state(CopyParams p) {
    for (uint64_t i = blockIdx.x * 256ull + threadIdx.x; i < p.count; i += gridDim.x * 256ull)
        p.to[i] = p.from == nullptr ? 0.f : p.from[i];
}

static rlca_status copy_state(const float *from, float *to, int64_t count, hipStream_t stream) {
    if (to == nullptr || count == 0) return RLCA_OK;
    CopyParams p = {from, to, (uint64_t)count};
    const int64_t blocks = (count + 255) / 256;
    return launch((const void *)gated_copy_state, dim3((uint32_t)(blocks < 4096 ? blocks : 4096)), 256, 0,
                  p, stream);
}

}  // namespace seq
}  // namespace rlca

using namespace rlca::seq;

extern "C" {

size_t rlca_gated_recurrence_checkpoints_size(const rlca_gated_call *call) {
    if (call == nullptr || !gate_sizes_ok(*call)) return 0;
    return gate_checkpoints_bytes(*call, gate_plan(*call, false));
}

size_t rlca_gated_recurrence_workspace_size(const rlca_gated_call *call) {
    if (call == nullptr || !gate_sizes_ok(*call)) return 0;
    return gate_maps_bytes(*call, gate_plan(*call, false));
}

size_t rlca_gated_recurrence_backward_workspace_size(const rlca_gated_call *call) {
    if (call == nullptr || !gate_sizes_ok(*call)) return 0;
    const GatePlan g = gate_plan(*call, true);
    return gate_maps_bytes(*call, g) + gate_partials_bytes(*call, g);
}

rlca_status rlca_gated_recurrence(const rlca_gated_call *call, void *workspace,
                                  size_t workspace_bytes, hipStream_t stream) {
    if (call == nullptr) return RLCA_ERR_NULL_POINTER;
    const rlca_gated_call &c = *call;
    Arrays a;
    rlca_status st = check_gated(c, false, a);
    if (st != RLCA_OK) return st;
    const GatePlan g = gate_plan(c, false);
    const int64_t N = c.num_seqs, D = c.channels, T = c.T;
    const size_t need = gate_maps_bytes(c, g);
    a.out(c.out, element_bytes(c.dtype), true, {{N, D * T}, {D, T}, {T, 1}});
    a.out(c.final_state, 4, false, {{N, D}, {D, 1}});
    a.out(c.checkpoints, 4, false, {{(int64_t)(gate_checkpoints_bytes(c, g) / 4), 1}});
    a.out(workspace, 4, need != 0, {{(int64_t)(need / 4), 1}});
    if ((st = a.status()) != RLCA_OK) return st;
    if (workspace_bytes < need) return RLCA_ERR_INVALID_SIZE;
    if (N * D == 0) return RLCA_OK;
    if (T == 0) return copy_state(c.state, c.final_state, N * D, stream);
    GateParams p = gate_params(c, g);
    p.maps = static_cast<float *>(workspace);
    if (g.chunks > 1 && (st = gate_launch(c, g, p, false, true, stream)) != RLCA_OK) return st;
    return gate_launch(c, g, p, false, false, stream);
}

rlca_status rlca_gated_recurrence_backward(const rlca_gated_call *call, void *workspace,
                                           size_t workspace_bytes, hipStream_t stream) {
    if (call == nullptr) return RLCA_ERR_NULL_POINTER;
    const rlca_gated_call &c = *call;
    Arrays a;
    rlca_status st = check_gated(c, true, a);
    if (st != RLCA_OK) return st;
    const GatePlan g = gate_plan(c, true);
    const int64_t N = c.num_seqs, D = c.channels, T = c.T;
    const size_t e = element_bytes(c.dtype), maps = gate_maps_bytes(c, g);
    const size_t need = maps + gate_partials_bytes(c, g);
    a.in(c.grad_out, e, true, {{N, c.grad_stride_seq}, {D, c.grad_stride_channel}, {T, 1}});
    a.in(c.grad_final_state, 4, false, {{N, D}, {D, 1}});
    a.in(c.checkpoints, 4, true, {{(int64_t)(gate_checkpoints_bytes(c, g) / 4), 1}});
    a.out(c.grad_x, e, true, {{N, D * T}, {D, T}, {T, 1}});
    a.out(c.grad_input_gate, e, true, {{N, D * T}, {D, T}, {T, 1}});
    a.out(c.grad_decay_gate, e, true, {{N, D * T}, {D, T}, {T, 1}});
    a.out(c.grad_decay, 4, true, {{D, 1}});
    a.out(c.grad_input_bias, 4, false, {{D, 1}});
    a.out(c.grad_decay_bias, 4, false, {{D, 1}});
    a.out(c.grad_state, 4, false, {{N, D}, {D, 1}});
    a.out(workspace, 4, need != 0, {{(int64_t)(need / 4), 1}});
    if ((st = a.status()) != RLCA_OK) return st;
    if (workspace_bytes < need) return RLCA_ERR_INVALID_SIZE;
    if (D == 0) return RLCA_OK;
    GateParams p = gate_params(c, g);
    p.maps = static_cast<float *>(workspace);
    p.partials = p.maps + maps / sizeof(float);
    uint32_t walkers = 0;
    if (N > 0 && T == 0) {
        if ((st = copy_state(c.grad_final_state, c.grad_state, N * D, stream)) != RLCA_OK) return st;
    } else if (N > 0) {
        walkers = p.walkers * (uint32_t)g.waves;
        if (g.chunks > 1 && (st = gate_launch(c, g, p, true, true, stream)) != RLCA_OK) return st;
        if ((st = gate_launch(c, g, p, true, false, stream)) != RLCA_OK) return st;
    }
    return launch_gate_sums(c, p.partials, walkers, stream);
}

rlca_status rlca_gated_step(const rlca_gated_step_call *call, hipStream_t stream) {
    if (call == nullptr) return RLCA_ERR_NULL_POINTER;
    const rlca_gated_step_call &c = *call;
    const int64_t N = c.num_seqs, D = c.channels;
    if (!sizes_ok(N, D, 1) || c.places < 0 || c.places > INT32_MAX ||
        (c.slots == nullptr && c.places < N))
        return RLCA_ERR_INVALID_SIZE;
    if (!gate_values_ok(c.dtype, c.scale)) return RLCA_ERR_INVALID_VALUE;
    const size_t e = element_bytes(c.dtype);
    const int64_t params = N == 0 ? 0 : D;
    Arrays a;
    a.in(c.x, e, true, {{N, c.x_stride_seq}, {D, 1}});
    a.in(c.input_gate, e, true, {{N, c.input_stride_seq}, {D, 1}});
    a.in(c.decay_gate, e, true, {{N, c.decay_stride_seq}, {D, 1}});
    a.in(c.decay, 4, true, {{params, 1}});
    a.in(c.input_bias, 4, false, {{params, 1}});
    a.in(c.decay_bias, 4, false, {{params, 1}});
    a.in(c.slots, 4, false, {{N, 1}});
    a.in(c.starts, 1, false, {{N, 1}});
    a.out(c.state, 4, N != 0, {{c.places, D}, {D, 1}});
    a.out(c.out, e, true, {{N, D}, {D, 1}});
    const rlca_status st = a.status();
    if (st != RLCA_OK || N * D == 0) return st;
    GateStepParams p = {};
    p.x = c.x, p.input_gate = c.input_gate, p.decay_gate = c.decay_gate;
    p.decay = c.decay, p.input_bias = c.input_bias, p.decay_bias = c.decay_bias;
    p.state = c.state;
    p.slots = c.slots;
    p.starts = c.starts;
    p.out = c.out;
    p.x_n = c.x_stride_seq, p.ig_n = c.input_stride_seq, p.dg_n = c.decay_stride_seq;
    p.places = c.places;
    p.num_seqs = (uint32_t)N;
    p.channels = (uint32_t)D;
    p.scale = (float)c.scale;
    const uint32_t threads = (uint32_t)D;
    const uint32_t size =
        threads >= (uint32_t)kGateStepThreads ? kGateStepThreads : (threads + 63) / 64 * 64;
    const uint32_t across = (threads + size - 1) / size;
    const uint32_t most = (2048 + across - 1) / across;  // enough to fill the chip
    const int64_t all = N < 32768 ? N : 32768;
    const void *kernel = c.dtype == RLCA_F32    ? (const void *)gated_step<float>
                         : c.dtype == RLCA_BF16 ? (const void *)gated_step<__bf16>
                                                : (const void *)gated_step<_Float16>;
    return launch(kernel, dim3(across, all < most ? (uint32_t)all : most), size, 0, p, stream);
}

}  // extern "C"
