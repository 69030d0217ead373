// seq_scan.hip -- the selective scan over rows of T steps, forward:
//   h_t = exp(dt_t A) h_{t-1} + dt_t u_t B_t,   y_t = (C_t . h_t + D u_t) silu(z_t).
// How a wave scans a state is told in seq_scan.hpp.
//
// Bound by the vector units: each (step, state) takes one exponential and the
// products of the fold, of the second pass over the maps and of y, against
// one or two stored values per step.  A workgroup's channels share the tile's B
// and C, staged in LDS in fp32 and read there 16 bytes a lane.
//
// A (step, state) takes 10.1 vector instructions (85 M wave instructions for
// 8x2048 channels of 2048 steps and 16 states) of at least 6, one of which, the
// exponential, issues at a quarter of the rate.  Measured there, bf16 with a
// gate: 169 us (hundreds of calls in a row; 185 to 200 in the first tens after
// idle, at a lower clock), the vector units busy 93% of it at 2.4 GHz; the bytes
// alone would take 60.
#include "seq_scan.hpp"

namespace rlca {
namespace seq {

// B and C are staged in two buffers: the next stage's rows are loaded while one
// is computed, and one barrier a stage suffices.
//
// SPLIT waves share the channels of one: each takes every SPLIT-th pair of states
// over all the steps, and prepares and finishes 8 / SPLIT of a lane's steps.
// They meet in LDS twice a tile, in dt and dt u before and in y's partial sums
// after (split_of below says when that pays).
//
// There are two bodies: GROW false for workgroups whose states all decay, which leaves
// with false, nothing written, where one may grow; GROW true has the serial steps too.
// They share neither addresses nor arguments in registers.  (A mere choice in one
// walk costs every decaying model 2 to 12%; the check costs rows of one tile up to 4%
// and longer ones nothing.)  Steps without softplus take the second alone, 4 to 7%
// slower than the first would be.
template <typename E, bool FLAGS, int SPLIT, int L, bool GROW, int SETS, int VALUES, int WAVES,
          int OUTS>
__device__ __forceinline__ bool scan_rows(const ScanParams &p, uint32_t thread,
                                          char *lds_bytes, TileRow<L> (&tiles)[2][2][states_of(L)],
                                          float (&steps)[SETS][VALUES][kWave],
                                          float (&sums)[WAVES][OUTS][kWave],
                                          uint32_t (&steady_waves)[kScanWaves],
                                          uint32_t (&stage_tame)[2][kScanWaves]) {
    constexpr int K = kScanK, kRows = rows_of(L) / SPLIT;
    constexpr int kTile = tile_of(L), kStates = states_of(L), kOwn = K / SPLIT;
    const int wave = __builtin_amdgcn_readfirstlane(thread / kWave);
    const int in_wave = thread % kWave;
    const int set = wave / SPLIT, part = wave % SPLIT;
    const ScanLane l = scan_lane<L>(p, thread, set * (kWave / L) + in_wave / L, kRows);
    const int S = (int)p.states, padded = padded_states(S), pitch = pitch_of(S, L);
    // [rows][pitch]: the states entering the tile, and A log2(e)
    float *carry = reinterpret_cast<float *>(lds_bytes) + l.local * pitch;
    float *A2 = carry + kRows * pitch;
    // a wave initialises and hands on the states that it computes
    const auto mine = [&](int s) { return SPLIT == 1 || (s / 2) % SPLIT == part; };
    const int end = row_end(p.lengths, l.n, p.T);
    const int own = l.lane * K + part * kOwn;  // the lane's own steps in a tile
    const uint8_t *flags = FLAGS ? p.flags + (int64_t)l.n * p.T : nullptr;
    const float bias = p.delta_bias == nullptr ? 0.f : p.delta_bias[l.d];
    const float skip = p.D == nullptr ? 0.f : p.D[l.d];
    const Stager<L, kScanThreads> st(l.lane, wave, in_wave);
    const int64_t stage_stride = st.c ? p.C_s : p.B_s;
    const E *stage_row = (st.c ? static_cast<const E *>(p.C) + l.n * p.C_n + l.g * p.C_g
                               : static_cast<const E *>(p.B) + l.n * p.B_n + l.g * p.B_g) +
                         st.s * stage_stride + st.lane * K;
    // The lane's steps of the tile at t0, in an input or y; where registers are
    // short the address is formed there and then.
    constexpr bool kLate = GROW || (FLAGS && L == 1);
    const auto in_row = [&](const void *x, int64_t by_n, int64_t by_d, int t0) {
        if constexpr (kLate)
            return static_cast<const E *>(x) + (l.n * by_n + t0) + (here(l.d) * by_d + here(own));
        return static_cast<const E *>(x) + l.n * by_n + l.d * by_d + own + t0;
    };
    const auto out_row = [&](void *out, int t0) {
        if constexpr (kLate)
            return static_cast<E *>(out) + t0 + ((int64_t)here(l.row) * p.T + here(own));
        return static_cast<E *>(out) + (int64_t)l.row * p.T + own + t0;
    };
    // Past the row's steps y is 0.
    const int live_tiles = (end + kTile - 1) / kTile;

    Steps<K, E> next_stage;
    Steps<kOwn, E> next_u, next_delta;
    const auto load_stage = [&](int t0, int s0) {
        if (st.active)
            next_stage.load(stage_row + s0 * stage_stride + t0,
                            s0 + st.s < S ? end - t0 - st.lane * K : 0);
    };
    const auto load_tile = [&](int t0) {
        next_u.load(in_row(p.u, p.u_n, p.u_d, t0), end - t0 - own);
        next_delta.load(in_row(p.delta, p.delta_n, p.delta_d, t0), end - t0 - own);
    };
    int buffer = 0;
    load_stage(0, 0);
    load_tile(0);

    bool tame_A = true;
    Growth growth;
    for (int s = l.lane; s < padded; s += L)
        if (mine(s)) {
            const float x = s >= S ? 0.f : p.A[(int64_t)l.d * S + s] * kLog2e;
            carry[s] = p.state == nullptr || s >= S ? 0.f : p.state[(int64_t)l.row * S + s];
            A2[s] = x;
            growth.add(x);
            if constexpr (FLAGS) tame_A &= tame(x, kTameStep);
        }
    if constexpr (GROW) {
        growth.meet();
    } else {
        // no a above 1 in any tile
        const bool steady = whole_wave(growth.up == 0.f);
        if (!all_waves(steady, steady_waves, wave, in_wave)) return false;
    }

    for (int tile = 0; tile < live_tiles; ++tile) {
        const int t0 = tile * kTile;
        if (p.checkpoints != nullptr && l.live)
            for (int s = l.lane; s < S; s += L)
                if (mine(s)) p.checkpoints[((int64_t)l.row * p.tiles + tile) * S + s] = carry[s];
        bool all_ok = tame_A;  // of the lane's values in this tile: tame
        if constexpr (FLAGS)
            for (int s = l.lane; s < padded; s += L)
                if (mine(s)) all_ok &= tame(carry[s], kTameState);
        float skipped[kOwn], dt[K], dtu[K], cut[K], y[K] = {};
        Steps<kOwn, E> z;
        if (p.z != nullptr) z.load(in_row(p.z, p.z_n, p.z_d, t0), end - t0 - own);
        {
            float u[kOwn], raw[kOwn], own_dt[kOwn], own_dtu[kOwn], own_cut[kOwn];
            next_u.widen(u);
            next_delta.widen(raw);
            make_steps<FLAGS>(p, flags, bias, t0 + own, end, end, u, raw, own_dt, own_dtu, own_cut);
            if (tile + 1 < live_tiles) load_tile(t0 + kTile);
#pragma unroll
            for (int k = 0; k < kOwn; ++k) {
                if constexpr (SPLIT > 1) {
                    steps[set][part * kOwn + k][in_wave] = own_dt[k];
                    steps[set][K + part * kOwn + k][in_wave] = own_dtu[k];
                    if constexpr (FLAGS)
                        steps[set][2 * K + part * kOwn + k][in_wave] = own_cut[k];
                } else {
                    dt[k] = own_dt[k];
                    dtu[k] = own_dtu[k];
                    if constexpr (FLAGS) cut[k] = own_cut[k];
                }
                skipped[k] = skip * u[k];
                if constexpr (SPLIT == 1) y[k] = skipped[k];
            }
        }
        float dt_sum = 0.f;
        bool starts = false, serial = false;
        for (int s0 = 0; s0 < S; s0 += kStates) {
            if (st.active) stage(tiles[buffer][st.c][st.s], next_stage, st.lane);
            if constexpr (FLAGS) {
                const bool ok = whole_wave(!st.active || all_tame(next_stage));
                if (in_wave == 0) stage_tame[buffer][wave] = ok ? 1u : 0u;
            }
            if (s0 + kStates < S)
                load_stage(t0, s0 + kStates);
            else if (tile + 1 < live_tiles)
                load_stage(t0 + kTile, 0);
            __syncthreads();
            if (s0 == 0) {
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    if constexpr (SPLIT > 1) {
                        dt[k] = steps[set][k][in_wave];
                        dtu[k] = steps[set][K + k][in_wave];
                        if constexpr (FLAGS) cut[k] = steps[set][2 * K + k][in_wave];
                    }
                    dt_sum += dt[k];
                    if constexpr (FLAGS) starts |= cut[k] != 0.f;
                }
                if constexpr (FLAGS) all_ok = whole_wave(all_ok && steps_tame(dt, dtu));
                if constexpr (GROW) serial = growth.too_much<L>(dt);
            }
            const TileRow<L> *B_tile = tiles[buffer][0], *C_tile = tiles[buffer][1];
            const int count = S - s0 < kStates ? S - s0 : kStates;
            const auto scan_states = [&](auto careful, int most) {
                constexpr bool CUT = decltype(careful)::value;
                for (int i = 2 * part; i < most; i += 2 * SPLIT) {
                    float a[2][K], b[2][K], h[2], prod[2], enter[2];
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const float a2 = A2[s0 + i + j];
                        enter[j] = carry[s0 + i + j];
                        read_tile(B_tile[i + j], l.lane, b[j]);
#pragma unroll
                        for (int k = 0; k < K; ++k) {
                            a[j][k] = decay<FLAGS, CUT>(dt[k], cut[k], a2);
                            b[j][k] *= dtu[k];
                            if constexpr (L > 1)
                                h[j] = k == 0 ? b[j][0] : step_map<CUT>(a[j][k], b[j][k], h[j]);
                        }
                        if constexpr (L > 1) prod[j] = lane_product<FLAGS, CUT>(dt_sum, starts, a2);
                    }
                    if constexpr (L > 1) row_scan<CUT, false, L>(prod, h, l.lane);
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        if constexpr (L > 1) {
                            const float after = step_map<CUT>(prod[j], h[j], enter[j]);
                            carry[s0 + i + j] = row_last<false, L>(after);
                            h[j] = row_shift<false, L>(after, enter[j], l.lane);
                        } else {
                            h[j] = enter[j];
                        }
                        float c[K];
                        read_tile(C_tile[i + j], l.lane, c);
#pragma unroll
                        for (int k = 0; k < K; ++k) {
                            h[j] = step_map<CUT>(a[j][k], b[j][k], h[j]);
                            y[k] = fmaf(c[k], h[j], y[k]);
                        }
                        if constexpr (L == 1) carry[s0 + i + j] = h[j];
                    }
                }
            };
            const auto scan_serially = [&](int most) {
#pragma unroll 1
                for (int i = 0; i < most; ++i) {
                    if (!mine(s0 + i)) continue;
                    const int at = s0 + i;
                    const float a2 = A2[at];
                    float v[K];
                    read_tile(B_tile[i], l.lane, v);
#pragma unroll
                    for (int k = 0; k < K; ++k) v[k] *= dtu[k];
                    float h = serial_enter<FLAGS, L>(dt, cut, v, a2, carry[at], l.lane);
                    float c[K];
                    read_tile(C_tile[i], l.lane, c);
#pragma unroll
                    for (int k = 0; k < K; ++k) {
                        h = serial_pass<FLAGS>(dt[k], cut[k], a2, h) + v[k];
                        y[k] = fmaf(c[k], h, y[k]);
                    }
                    if constexpr (L > 1)
                        carry[at] = row_last<false, L>(h);
                    else
                        carry[at] = h;
                }
            };
            bool plain = true;
            if constexpr (FLAGS) {
                uint32_t staged = 1u;
#pragma unroll
                for (int w = 0; w < kScanWaves; ++w) staged &= stage_tame[buffer][w];
                plain = all_ok && __builtin_amdgcn_readfirstlane(staged) != 0u;
            }
            if constexpr (GROW) {  // loops in turn: fewer registers than a choice
                plain = plain && !serial;
                scan_serially(plain ? 0 : count);
                scan_states(std::false_type{}, plain ? count : 0);
            } else if (!FLAGS || plain) {
                scan_states(std::false_type{}, count);
            } else if constexpr (FLAGS) {
                scan_states(std::true_type{}, count);
            }
            buffer ^= 1;
        }
        wave_order();
        float out[kOwn];
        if constexpr (SPLIT > 1) {
#pragma unroll
            for (int k = 0; k < K; ++k) sums[wave][k][in_wave] = y[k];
            __syncthreads();
#pragma unroll
            for (int k = 0; k < kOwn; ++k) {
                out[k] = skipped[k];
#pragma unroll
                for (int q = 0; q < SPLIT; ++q)
                    out[k] += sums[set * SPLIT + q][part * kOwn + k][in_wave];
            }
        } else {
#pragma unroll
            for (int k = 0; k < kOwn; ++k) out[k] = y[k];
        }
        const int t = t0 + own;
        if (l.live && t < p.T) {
            if (p.z != nullptr) {
                float gate[kOwn];
                z.widen(gate);
#pragma unroll
                for (int k = 0; k < kOwn; ++k) out[k] *= silu(gate[k]);
            }
            if (t + kOwn > end)  // few lanes
#pragma unroll
                for (int k = 0; k < kOwn; ++k) out[k] = t + k < end ? out[k] : 0.f;
            store_steps<kOwn>(out_row(p.y, t0), p.T - t, out);
        }
    }
    if (!l.live) return true;
    for (int t0 = live_tiles * kTile; t0 + own < p.T; t0 += kTile) {
        const float zeros[kOwn] = {};
        store_steps<kOwn>(out_row(p.y, t0), p.T - t0 - own, zeros);
    }
    if (p.final_state != nullptr) {
        const bool over = FLAGS && p.after_done != 0 && end > 0 && flags[end - 1] != 0;
        for (int s = l.lane; s < S; s += L)
            if (mine(s)) p.final_state[(int64_t)l.row * S + s] = over ? 0.f : carry[s];
    }
    return true;
}

// GIVEN: steps without softplus, which may be below 0.
template <typename E, bool FLAGS, int SPLIT, int L, bool GIVEN>
__global__ __launch_bounds__(kScanThreads, sizeof(E) == 2 && !FLAGS ? 4 : 3) void selective_scan(
    ScanParams p) {
    extern __shared__ __attribute__((aligned(16))) char lds_bytes[];
    __shared__ TileRow<L> tiles[2][2][states_of(L)];  // [buffer][B, C][state]
    __shared__ float steps[kScanWaves / SPLIT][SPLIT > 1 ? (FLAGS ? 3 : 2) * kScanK : 1][kWave];
    __shared__ float sums[SPLIT > 1 ? kScanWaves : 1][SPLIT > 1 ? kScanK : 1][kWave];
    __shared__ uint32_t steady_waves[kScanWaves];
    __shared__ uint32_t stage_tame[2][kScanWaves];  // [buffer]: whether what a wave staged is
    if constexpr (GIVEN)
        scan_rows<E, FLAGS, SPLIT, L, true>(p, threadIdx.x, lds_bytes, tiles, steps, sums,
                                            steady_waves, stage_tame);
    else if (!scan_rows<E, FLAGS, SPLIT, L, false>(p, threadIdx.x, lds_bytes, tiles, steps, sums,
                                                   steady_waves, stage_tame))
        scan_rows<E, FLAGS, SPLIT, L, true>(arguments_again<ScanParams>(), here(threadIdx.x),
                                            lds_bytes, tiles, steps, sums, steady_waves,
                                            stage_tame);
}

// ------------------------------------------------------------------- host side
// Lanes of a row: the cheapest of 16, 4 and 1 by the waves and the tiles of
// each, a tile weighed by what it took beside 16 lanes' (1.1 for 4 lanes and
// 16 states, 1.4 where more states leave fewer workgroups a CU, 1.85 for a lane
// alone and 0.6 for its start), where fewer waves than SIMDs count as many.  LDS
// limits the states of the two.  Forward and backward in us with 16, 4 and 1 (256
// channels, bf16 and a gate, 16 states): 4096 rows of 3 steps 2759, 746 and
// 407; 2048 of 32 1359, 381 and 550; 1024 of 64 711, 371 and 572; 512 of 130 693,
// 469 and 628; 256 of 260 530, 428 and 586; 128 of 520 437, 423 and 1004; 512
// of 64 with 64 states 1175 and 806; forward alone 16 rows of 30 (4096
// channels) 45, 18 and 24.
int lanes_of(const rlca_scan_call &c) {
    const int64_t per_group = c.groups == 0 ? 0 : c.channels / c.groups;
    int best = 16;
    double least = INFINITY;
    for (int L = 16; L >= 1; L /= 4) {
        if ((L == 4 && c.states > 64) || (L == 1 && c.states > 16)) continue;
        const int64_t blocks = (per_group + rows_of(L) - 1) / rows_of(L) * c.groups;
        const double waves = (double)c.num_seqs * blocks * kScanWaves;
        const int64_t tiles = (c.T + tile_of(L) - 1) / tile_of(L);
        const double wave = L == 16  ? 1.0 * tiles
                            : L == 4 ? (c.states > 16 ? 1.4 : 1.1) * tiles
                                     : 0.6 + 1.85 * tiles;
        const double cost = wave * (waves < 1024 ? 1024 : waves);
        if (cost < least) least = cost, best = L;
    }
    return best;
}

ScanParams scan_params(const rlca_scan_call &c, int rows) {
    ScanParams p = {};
    p.u = c.u;
    p.delta = c.delta;
    p.B = c.B;
    p.C = c.C;
    p.z = c.z;
    p.grad_y = c.grad_y;
    p.A = c.A;
    p.D = c.D;
    p.delta_bias = c.delta_bias;
    p.state = c.state;
    p.grad_final = c.grad_final_state;
    p.flags = c.flags;
    p.lengths = c.lengths;
    p.y = c.y;
    p.final_state = c.final_state;
    p.checkpoints = c.checkpoints;
    p.grad_u = c.grad_u;
    p.grad_delta = c.grad_delta;
    p.grad_z = c.grad_z;
    p.grad_state = c.grad_state;
    p.u_n = c.u_stride_seq, p.u_d = c.u_stride_channel;
    p.delta_n = c.delta_stride_seq, p.delta_d = c.delta_stride_channel;
    p.z_n = c.z_stride_seq, p.z_d = c.z_stride_channel;
    p.g_n = c.grad_stride_seq, p.g_d = c.grad_stride_channel;
    p.B_n = c.B_stride_seq, p.B_g = c.B_stride_group, p.B_s = c.B_stride_state;
    p.C_n = c.C_stride_seq, p.C_g = c.C_stride_group, p.C_s = c.C_stride_state;
    p.num_seqs = (uint32_t)c.num_seqs;
    p.channels = (uint32_t)c.channels;
    p.groups = (uint32_t)c.groups;
    p.per_group = p.channels / p.groups;
    p.states = (uint32_t)c.states;
    p.blocks_per_group = (p.per_group + rows - 1) / rows;
    p.T = (int32_t)c.T;
    const int tile = tile_of(lanes_of(c));
    p.tiles = (p.T + tile - 1) / tile;
    p.softplus = c.softplus;
    p.after_done = c.convention == RLCA_RESET_AFTER_DONE;
    return p;
}

// Waves that share four channels (rows of 16 lanes): enough that the launch
// gives the 1024 SIMDs several waves each, as long as every wave has a pair of
// states.  In us with 1, 2 and 4 (bf16, a gate, 16 states; by the waves at one each):
//   4096 steps   128 waves 143, 97, 62; 384 141, 98, 74; 1024 151, 127, 113
//   2048 steps   1280 95, 78, 75; 1536 95, 79, 83; 1792 99, 98, 95; 2048 101, 99, 106;
//                2560 133, 126, 133; 2816 134, 141, 144; 4096 167, 180, 202
//   1024 steps   3328 84, 80, 85; 4096 87, 93, 104
//   300 steps    1024 17.2, 15.5, 15.6; 2048 22.5, 22.4, 25.4; 4096 36, 38, 45
//   1024 steps and 64 states   1024 111, 92, 85; 2048 156, 150, 153
// The crossings lie near 1500 and between 2560 and 3328 waves, where the sides differ
// by 6% at most; they depend on neither the steps nor the states by more than that.
constexpr int kFewestRows = 4;

static int split_of(const rlca_scan_call &c) {
    const int64_t waves = c.num_seqs * c.channels / 4;
    const int pairs = padded_states(c.states) / 2;
    return waves <= 1536 && pairs >= 4 ? 4 : waves <= 3000 && pairs >= 2 ? 2 : 1;
}

template <typename E, int SPLIT, int L>
static const void *scan_kernel(const rlca_scan_call &c) {
    const bool flags = c.flags != nullptr, given = c.softplus == 0;
    return flags ? (given ? (const void *)selective_scan<E, true, SPLIT, L, true>
                          : (const void *)selective_scan<E, true, SPLIT, L, false>)
                 : (given ? (const void *)selective_scan<E, false, SPLIT, L, true>
                          : (const void *)selective_scan<E, false, SPLIT, L, false>);
}

template <typename E>
static const void *scan_kernel(const rlca_scan_call &c, int split, int lanes) {
    return lanes == 1   ? scan_kernel<E, 1, 1>(c)
           : lanes == 4 ? scan_kernel<E, 1, 4>(c)
           : split == 4 ? scan_kernel<E, 4, 16>(c)
           : split == 2 ? scan_kernel<E, 2, 16>(c)
                        : scan_kernel<E, 1, 16>(c);
}

static int64_t checkpoint_values(const rlca_scan_call &c) {
    const int tile = tile_of(lanes_of(c));
    return c.num_seqs * c.channels * ((c.T + tile - 1) / tile) * c.states;
}

rlca_status check_scan(const rlca_scan_call &c, bool backward, Arrays *a) {
    const int64_t N = c.num_seqs, D = c.channels, T = c.T, S = c.states, G = c.groups;
    if (!sizes_ok(N, D, T)) return RLCA_ERR_INVALID_SIZE;
    const size_t e = element_bytes(c.dtype);
    if (e == 0 || S < 1 || S > RLCA_MAX_STATES || G < 1 || D % G != 0 ||
        (c.convention != RLCA_RESET_ON_START && c.convention != RLCA_RESET_AFTER_DONE))
        return RLCA_ERR_INVALID_VALUE;
    if (T != 0 && N * D > INT64_MAX / 8 / S / T) return RLCA_ERR_INVALID_SIZE;
    // a launch holds less than 2^32 threads
    const int64_t blocks = D == 0 ? 0 : N * G * ((D / G + kFewestRows - 1) / kFewestRows);
    if (blocks >= ((int64_t)1 << 32) / kScanThreads) return RLCA_ERR_INVALID_SIZE;
    const int64_t params = N == 0 ? 0 : D, rows = D == 0 ? 0 : N;
    const Dim dense[] = {{N, D * T}, {D, T}, {T, 1}};
    const Dim state[] = {{N * D, S}, {S, 1}};
    const Dim b[] = {{rows, c.B_stride_seq}, {G, c.B_stride_group}, {S, c.B_stride_state}, {T, 1}};
    const Dim cc[] = {{rows, c.C_stride_seq}, {G, c.C_stride_group}, {S, c.C_stride_state}, {T, 1}};
    a->in(c.u, e, true, {{N, c.u_stride_seq}, {D, c.u_stride_channel}, {T, 1}});
    a->in(c.delta, e, true, {{N, c.delta_stride_seq}, {D, c.delta_stride_channel}, {T, 1}});
    a->in(c.z, e, false, {{N, c.z_stride_seq}, {D, c.z_stride_channel}, {T, 1}});
    a->in(c.A, 4, true, {{params, S}, {S, 1}});
    a->in(c.B, e, true, b);
    a->in(c.C, e, true, cc);
    a->in(c.D, 4, false, {{params, 1}});
    a->in(c.delta_bias, 4, false, {{params, 1}});
    a->in(c.flags, 1, false, {{N * T, 1}});
    a->in(c.lengths, 4, false, {{N, 1}});
    const Dim checkpoints[] = {{checkpoint_values(c), 1}};
    if (!backward) {
        a->in(c.state, 4, false, state);
        a->out(c.y, e, true, dense);
        a->out(c.final_state, 4, false, state);
        a->out(c.checkpoints, 4, false, checkpoints);
    } else {
        a->in(c.checkpoints, 4, true, checkpoints);
        a->in(c.grad_y, e, true, {{N, c.grad_stride_seq}, {D, c.grad_stride_channel}, {T, 1}});
        a->in(c.grad_final_state, 4, false, state);
        const Dim bc[] = {{rows * G * S, T}, {T, 1}};
        a->out(c.grad_u, e, true, dense);
        a->out(c.grad_delta, e, true, dense);
        a->out(c.grad_A, 4, true, {{D, S}, {S, 1}});
        a->out(c.grad_B, e, true, bc);
        a->out(c.grad_C, e, true, bc);
        a->out(c.grad_D, 4, false, {{D, 1}});
        a->out(c.grad_delta_bias, 4, false, {{D, 1}});
        if (c.z != nullptr) a->out(c.grad_z, e, true, dense);
        a->out(c.grad_state, 4, false, state);
    }
    return RLCA_OK;
}

}  // namespace seq
}  // namespace rlca

using namespace rlca::seq;

extern "C" {

size_t rlca_selective_scan_checkpoints_size(const rlca_scan_call *call) {
    Arrays a;
    if (call == nullptr || check_scan(*call, false, &a) != RLCA_OK) return 0;
    return (size_t)checkpoint_values(*call) * 4;
}

rlca_status rlca_selective_scan(const rlca_scan_call *call, hipStream_t stream) {
    if (call == nullptr) return RLCA_ERR_NULL_POINTER;
    const rlca_scan_call &c = *call;
    Arrays a;
    rlca_status st = check_scan(c, false, &a);
    if (st == RLCA_OK) st = a.status();
    if (st != RLCA_OK) return st;
    if (c.num_seqs * c.channels == 0 || (c.T == 0 && c.final_state == nullptr)) return RLCA_OK;
    const int lanes = lanes_of(c), split = lanes == 16 ? split_of(c) : 1;
    const int rows = rows_of(lanes) / split;
    ScanParams p = scan_params(c, rows);
    const void *kernel = c.dtype == RLCA_F32    ? scan_kernel<float>(c, split, lanes)
                         : c.dtype == RLCA_BF16 ? scan_kernel<__bf16>(c, split, lanes)
                                                : scan_kernel<_Float16>(c, split, lanes);
    return launch(kernel, dim3(p.num_seqs * p.groups * p.blocks_per_group), kScanThreads,
                  2 * rows * pitch_of(c.states, lanes) * 4, p, stream);
}

}  // extern "C"
