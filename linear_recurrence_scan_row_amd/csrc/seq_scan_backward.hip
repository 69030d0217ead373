// seq_scan_backward.hip -- the gradients of the selective scan.  With
// gy_t = grad_y_t silu(z_t), and for each channel and state
//   g_t = C_t gy_t + a_{t+1} g_{t+1}             (dL/dh_t, from the last step back)
//   w_t = a_t h_{t-1}
//   grad_C_t = sum_d gy_t h_t                    grad_B_t = sum_d g_t dt_t u_t
//   grad_dt_t = sum_s g_t w_t A + u_t sum_s g_t B_t
//   grad_u_t = dt_t sum_s g_t B_t + D gy_t       grad_A = sum_t g_t w_t dt_t
// A workgroup walks its channels' tiles from the last to the first.  The
// state that enters a tile comes from the forward call's checkpoints, the
// tile's states from one forward scan, and g from one reverse scan whose carry
// r = a_t g_t passes to the tile before.
//
// grad_B and grad_C sum over the channels of a group.  Within a wave the rows
// hold channels of the same steps: 16 values (8 steps of each gradient) meet in
// 12 lane-half swaps and 12 additions, after which each 16 lanes hold four of
// them, summed over rows of 16 lanes (sum_rows goes on for fewer).  The waves' sums
// meet in LDS, the workgroups' in a workspace that bc_sums adds in order.
//
// A (step, state) takes 28.4 vector instructions, of about 22 in the formulas
// above and the sums.  Measured for 8x2048 channels of 2048 steps and 16 states,
// bf16 with a gate: 479 us (hundreds of calls in a row), the vector units busy 90%
// of it at 2.4 GHz (298 MB read and 471 written, 268 of them partial sums, would
// take 161), and 54 for bc_sums (5.0 TB/s).
#include "seq_scan.hpp"

namespace rlca {
namespace seq {

__device__ __forceinline__ void swap_add(float &x, float y, bool halves) {
    const uint32_t a = __builtin_bit_cast(uint32_t, x), b = __builtin_bit_cast(uint32_t, y);
    // x's upper 32 lanes (odd rows) change places with y's lower (even) ones
    const auto r = halves ? __builtin_amdgcn_permlane32_swap(a, b, false, false)
                          : __builtin_amdgcn_permlane16_swap(a, b, false, false);
    x = __builtin_bit_cast(float, (uint32_t)r[0]) + __builtin_bit_cast(float, (uint32_t)r[1]);
}

// The sums over a wave's rows of 16 values a lane (8 steps of grad_B, then of
// grad_C).  Halves of the wave, then its rows of 16 lanes, swap half of what
// they hold: a lane of 16 keeps the four values from 4 (lane / 16) on.  Rows of
// fewer lanes go on within the 16: a lane keeps value lane / 4 (of its place in
// the row, L = 4), or all four lanes of a quad do (L = 1).
template <int L>
using RowSums = typename std::conditional<L == 16, float4v, float>::type;

template <int L>
__device__ __forceinline__ RowSums<L> sum_rows(float (&v)[16], int in_wave) {
#pragma unroll
    for (int i = 0; i < 8; ++i) swap_add(v[i], v[8 + i], true);
#pragma unroll
    for (int i = 0; i < 4; ++i) swap_add(v[i], v[4 + i], false);
    if constexpr (L == 16) {
        float4v r;
#pragma unroll
        for (int i = 0; i < 4; ++i) r[i] = v[i];
        return r;
    } else {
        // lanes 8 apart: those with bit 3 keep the upper two values
        const bool up8 = (in_wave & 8) != 0, up4 = (in_wave & 4) != 0;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float keep = up8 ? v[2 + i] : v[i], give = up8 ? v[i] : v[2 + i];
            v[i] = keep + dpp_move<0x128, 0xf>(give, 0.f);  // row_ror:8
        }
        // lanes 4 apart: quads 0 and 2 take from the quad above, 1 and 3 from below
        const float keep = up4 ? v[1] : v[0], give = up4 ? v[0] : v[1];
        const float above = dpp_move<0x12c, 0xf>(give, 0.f);  // row_ror:12
        const float below = dpp_move<0x124, 0xf>(give, 0.f);  // row_ror:4
        float r = keep + (up4 ? below : above);
        if constexpr (L == 1) {  // and the quad's four lanes
            r += dpp_move<0xb1, 0xf>(r, 0.f);  // quad_perm 1, 0, 3, 2
            r += dpp_move<0x4e, 0xf>(r, 0.f);  // quad_perm 2, 3, 0, 1
        }
        return r;
    }
}

// Sums over a row's lanes of two values, complete in its last lane.
template <int L>
__device__ __forceinline__ void row_sum(float (&x)[2]) {
    if constexpr (L == 16) {
        // the two take turns, and one idle instruction keeps the required two
        // between a write and the lane-crossing read of it; one more at the end
        // does so for whatever reads the sums next, which the compiler does not know
#define RLCA_STEP(SHIFT)                                                  \
    "v_add_f32_dpp %0, %0, %0 " SHIFT " row_mask:0xf bank_mask:0xf\n\t"   \
    "v_add_f32_dpp %1, %1, %1 " SHIFT " row_mask:0xf bank_mask:0xf\n\t"   \
    "s_nop 0\n\t"
        asm("s_nop 1\n\t" RLCA_STEP("row_shr:1") RLCA_STEP("row_shr:2") RLCA_STEP("row_shr:4")
                RLCA_STEP("row_shr:8") "s_nop 0"
            : "+v"(x[0]), "+v"(x[1]));
#undef RLCA_STEP
    } else if constexpr (L == 4) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            x[j] += dpp_move<0xb1, 0xf>(x[j], 0.f);
            x[j] += dpp_move<0x4e, 0xf>(x[j], 0.f);
        }
    }
}

// A workgroup holds four sets of 64 / L channels, SPLIT waves to each.  Waves of
// one set take every SPLIT-th pair of states, and prepare and finish 8 / SPLIT
// of a lane's steps, as in the forward scan.
//
// Two bodies, as the forward scan's kernel has.
template <typename E, bool FLAGS, bool GATE, int SPLIT, int L, bool GROW, int WAVES, int SETS,
          int BEFORE, int PARTS, int AFTER>
__device__ __forceinline__ bool scan_rows_back(const ScanParams &p, uint32_t thread,
                                               char *lds_bytes,
                                               TileRow<L> (&tiles)[2][2][states_of(L)],
                                               RowSums<L> (&bc)[kScanWaves][states_of(L)][kWave],
                                               float (&before)[SETS][BEFORE][kWave],
                                               float (&after)[PARTS][AFTER][kWave],
                                               uint32_t (&steady_waves)[WAVES],
                                               uint32_t (&stage_tame)[2][WAVES]) {
    constexpr int K = kScanK, kSets = kScanWaves, kRows = rows_of(L), kStates = states_of(L);
    constexpr int kTile = tile_of(L), kOwn = K / SPLIT, kThreads = kScanThreads * SPLIT;
    const int wave = __builtin_amdgcn_readfirstlane(thread / kWave);
    const int in_wave = thread % kWave;
    const int set = wave / SPLIT, part = wave % SPLIT;
    const ScanLane l = scan_lane<L>(p, thread, set * (kWave / L) + in_wave / L, kRows);
    const int S = (int)p.states, padded = padded_states(S), pitch = pitch_of(S, L);
    // [rows][pitch]: A, the gradient a_t g_t entering the tile from its right,
    // the states entering it from its left, and the sums of grad_A
    float *A = reinterpret_cast<float *>(lds_bytes) + l.local * pitch;
    float *carry = A + kRows * pitch;
    float *enter_states = carry + kRows * pitch;
    float *grad_A = enter_states + kRows * pitch;
    const auto mine = [&](int s) { return SPLIT == 1 || (s / 2) % SPLIT == part; };
    const int row_steps = row_end(p.lengths, l.n, p.T);
    const int end = l.live ? row_steps : 0;  // a clamped row computes on zeros
    const uint8_t *flags = FLAGS ? p.flags + (int64_t)l.n * p.T : nullptr;
    const bool over = FLAGS && p.after_done != 0 && end > 0 && flags[end - 1] != 0;
    const int own = l.lane * K + part * kOwn;  // the lane's own steps in a tile
    // The lane's steps of the tile at t0, in an input or a gradient; where registers are
    // short the address is formed there and then.
    constexpr bool kLate = GROW || (GATE && (FLAGS || (L == 4 && sizeof(E) == 4)));
    constexpr bool kLateOut = kLate || (GATE && L == 4);
    const auto in_row = [&](const void *x, int64_t by_n, int64_t by_d, int t0) {
        if constexpr (kLate)
            return static_cast<const E *>(x) + (l.n * by_n + t0) + (here(l.d) * by_d + here(own));
        return static_cast<const E *>(x) + l.n * by_n + l.d * by_d + own + t0;
    };
    const auto out_row = [&](void *out, int t0) {
        if constexpr (kLateOut)
            return static_cast<E *>(out) + t0 + ((int64_t)here(l.row) * p.T + here(own));
        return static_cast<E *>(out) + (int64_t)l.row * p.T + own + t0;
    };
    const float bias = p.delta_bias == nullptr ? 0.f : p.delta_bias[l.d];
    const float skip = p.D == nullptr ? 0.f : p.D[l.d];
    float *partials = p.bc_partials + (int64_t)blockIdx.x * 2 * S * p.tiles * kTile;
    float totals[2] = {0.f, 0.f};  // of grad_D and grad_delta_bias

    const Stager<L, kThreads> st(l.lane, wave, in_wave);
    const int64_t stage_stride = st.c ? p.C_s : p.B_s;
    const E *stage_row = (st.c ? static_cast<const E *>(p.C) + l.n * p.C_n + l.g * p.C_g
                               : static_cast<const E *>(p.B) + l.n * p.B_n + l.g * p.B_g) +
                         st.s * stage_stride + st.lane * K;
    const int live_tiles = (row_steps + kTile - 1) / kTile;
    Steps<K, E> next_stage;
    Steps<kOwn, E> u, delta, go, z, next_u, next_delta, next_go, next_z;
    const auto load_stage = [&](int t0, int s0) {
        if (st.active)
            next_stage.load(stage_row + s0 * stage_stride + t0,
                            s0 + st.s < S ? row_steps - t0 - st.lane * K : 0);
    };
    const auto load_tile = [&](int t0) {
        next_u.load(in_row(p.u, p.u_n, p.u_d, t0), end - t0 - own);
        next_delta.load(in_row(p.delta, p.delta_n, p.delta_d, t0), end - t0 - own);
        next_go.load(in_row(p.grad_y, p.g_n, p.g_d, t0), end - t0 - own);
        if constexpr (GATE) next_z.load(in_row(p.z, p.z_n, p.z_d, t0), end - t0 - own);
    };

    // Each tile's rows are loaded a tile ahead, where registers allow it.
    constexpr bool kAhead = !GATE || ((sizeof(E) == 2 || SPLIT > 1) && !FLAGS);
    // With both episodes and a gate they are loaded again at a tile's end instead
    // of kept over its states.
    constexpr bool kReload = FLAGS && GATE;
    int buffer = 0;
    if (live_tiles > 0) {  // an empty row has no last tile
        load_stage((live_tiles - 1) * kTile, 0);
        if constexpr (kAhead) load_tile((live_tiles - 1) * kTile);
    }

    bool tame_A = true;
    Growth growth;
    for (int s = l.lane; s < padded; s += L)
        if (mine(s)) {
            const float x = s >= S ? 0.f : p.A[(int64_t)l.d * S + s];
            A[s] = x;
            growth.add(x * kLog2e);
            if constexpr (FLAGS) tame_A &= tame(x, kTameStep);
            carry[s] = p.grad_final == nullptr || over || !l.live || s >= S
                           ? 0.f
                           : p.grad_final[(int64_t)l.row * S + s];
            grad_A[s] = 0.f;
        }
    if constexpr (GROW) {
        growth.meet();
    } else {
        // no a above 1 in any tile
        const bool steady = whole_wave(growth.up == 0.f);
        if (!all_waves(steady, steady_waves, wave, in_wave)) return false;
    }
    // tiles past the row's steps are zeros, and their sums are not read
    for (int t0 = live_tiles * kTile; l.live && t0 + own < p.T; t0 += kTile) {
        const float zeros[kOwn] = {};
        const int n = p.T - t0 - own;
        store_steps<kOwn>(out_row(p.grad_u, t0), n, zeros);
        store_steps<kOwn>(out_row(p.grad_delta, t0), n, zeros);
        if constexpr (GATE) store_steps<kOwn>(out_row(p.grad_z, t0), n, zeros);
    }


    for (int tile = live_tiles - 1; tile >= 0; --tile) {
        const int t0 = tile * kTile;
        bool all_ok = tame_A;  // of the lane's values in this tile: tame
        if constexpr (!kAhead) load_tile(t0);
        u = next_u;
        delta = next_delta;
        go = next_go;
        if constexpr (GATE) z = next_z;
        {
            const float *from = p.checkpoints + ((int64_t)l.row * p.tiles + tile) * S;
            for (int s = l.lane; s < padded; s += L)
                if (mine(s)) {
                    const float x = l.live && s < S ? from[s] : 0.f;
                    enter_states[s] = x;
                    if constexpr (FLAGS)
                        all_ok &= tame(x, kTameState) && tame(carry[s], kTameState);
                }
        }
        if (kAhead && tile > 0) load_tile(t0 - kTile);
        float dt[K], dtu[K], cut[K], gy[K];
        float y[K] = {}, grad_dt[K] = {}, gB[K] = {};
        {
            float v[kOwn], raw[kOwn], own_dt[kOwn], own_dtu[kOwn], own_cut[kOwn], own_gy[kOwn];
            u.widen(v);
            delta.widen(raw);
            make_steps<FLAGS>(p, flags, bias, t0 + own, end, row_steps, v, raw, own_dt, own_dtu,
                              own_cut);
            go.widen(own_gy);
            if constexpr (GATE) {
                z.widen(v);
#pragma unroll
                for (int k = 0; k < kOwn; ++k) own_gy[k] *= silu(v[k]);  // 0 past the end
            }
#pragma unroll
            for (int k = 0; k < kOwn; ++k) {
                if constexpr (SPLIT > 1) {
                    const int at = part * kOwn + k;
                    before[set][at][in_wave] = own_dt[k];
                    before[set][K + at][in_wave] = own_dtu[k];
                    before[set][2 * K + at][in_wave] = own_gy[k];
                    if constexpr (FLAGS) before[set][3 * K + at][in_wave] = own_cut[k];
                } else {
                    dt[k] = own_dt[k];
                    dtu[k] = own_dtu[k];
                    gy[k] = own_gy[k];
                    if constexpr (FLAGS) cut[k] = own_cut[k];
                }
            }
        }
        float dt_sum = 0.f;
        bool starts = false, serial = false;
        for (int s0 = 0; s0 < S; s0 += kStates) {
            const int count = S - s0 < kStates ? S - s0 : kStates;
            if (st.active) stage(tiles[buffer][st.c][st.s], next_stage, st.lane);
            if constexpr (FLAGS) {
                const bool ok = whole_wave(!st.active || all_tame(next_stage));
                if (in_wave == 0) stage_tame[buffer][wave] = ok ? 1u : 0u;
            }
            if (s0 + kStates < S)
                load_stage(t0, s0 + kStates);
            else if (tile > 0)
                load_stage(t0 - kTile, 0);
            __syncthreads();
            if (s0 == 0) {
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    if constexpr (SPLIT > 1) {
                        dt[k] = before[set][k][in_wave];
                        dtu[k] = before[set][K + k][in_wave];
                        gy[k] = before[set][2 * K + k][in_wave];
                        if constexpr (FLAGS) cut[k] = before[set][3 * K + k][in_wave];
                    }
                    dt_sum += dt[k];
                    if constexpr (FLAGS) starts |= cut[k] != 0.f;
                }
                if constexpr (FLAGS) {
                    all_ok &= steps_tame(dt, dtu);
#pragma unroll
                    for (int k = 0; k < K; ++k) all_ok &= tame(gy[k], kTameStep);
                    all_ok = whole_wave(all_ok);
                }
                if constexpr (GROW) serial = growth.too_much<L>(dt);
            }
            const TileRow<L> *B_tile = tiles[buffer][0], *C_tile = tiles[buffer][1];
            const auto scan_states = [&](auto careful, int most) {
                constexpr bool CUT = decltype(careful)::value;
                for (int i = 2 * part; i < most; i += 2 * SPLIT) {
                    float a[2][K], w[2][K], g[2], prod[2], dA[2];
                    float h[2], prefix[2], enter[2];
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const float a2 = A[s0 + i + j] * kLog2e;
                        enter[j] = enter_states[s0 + i + j];
                        float b[K];
                        if constexpr (L > 1) read_tile(B_tile[i + j], l.lane, b);
#pragma unroll
                        for (int k = 0; k < K; ++k) {
                            a[j][k] = decay<FLAGS, CUT>(dt[k], cut[k], a2);
                            if constexpr (L > 1) {
                                const float x = b[k] * dtu[k];
                                h[j] = k == 0 ? x : step_map<CUT>(a[j][k], x, h[j]);
                            }
                        }
                        if constexpr (L > 1)
                            prefix[j] = prod[j] = lane_product<FLAGS, CUT>(dt_sum, starts, a2);
                    }
                    if constexpr (L > 1) row_scan<CUT, false, L>(prefix, h, l.lane);
                    float v[2][16], r[2], c[2][K];
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        if constexpr (L > 1)
                            h[j] = row_shift<false, L>(step_map<CUT>(prefix[j], h[j], enter[j]),
                                                       enter[j], l.lane);
                        else
                            h[j] = enter[j];
                        float b[K];
                        read_tile(B_tile[i + j], l.lane, b);
                        read_tile(C_tile[i + j], l.lane, c[j]);
#pragma unroll
                        for (int k = 0; k < K; ++k) {
                            w[j][k] = pass<CUT>(a[j][k], h[j]);
                            h[j] = fmaf(b[k], dtu[k], w[j][k]);
                            v[j][8 + k] = gy[k] * h[j];
                            if constexpr (GATE) y[k] = fmaf(c[j][k], h[j], y[k]);
                            c[j][k] *= gy[k];  // what y's gradient adds to g
                        }
                        if constexpr (L > 1) {
                            g[j] = c[j][K - 1];
#pragma unroll
                            for (int k = K - 2; k >= 0; --k)
                                g[j] = step_map<CUT>(a[j][k + 1], c[j][k], g[j]);
                            r[j] = pass<CUT>(a[j][0], g[j]);
                        }
                    }
                    if constexpr (L > 1) row_scan<CUT, true, L>(prod, r, l.lane);
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const float right = carry[s0 + i + j], A_s = A[s0 + i + j];
                        if constexpr (L > 1) {
                            r[j] = step_map<CUT>(prod[j], r[j], right);
                            carry[s0 + i + j] = row_last<true, L>(r[j]);
                            // a g of the step after the lane's
                            g[j] = row_shift<true, L>(r[j], right, l.lane);
                        } else {
                            g[j] = right;
                        }
                        float b[K];
                        read_tile(B_tile[i + j], l.lane, b);
                        dA[j] = 0.f;
#pragma unroll
                        for (int k = K - 1; k >= 0; --k) {
                            g[j] = k == K - 1 ? c[j][k] + g[j]
                                              : step_map<CUT>(a[j][k + 1], c[j][k], g[j]);
                            v[j][k] = g[j] * dtu[k];
                            gB[k] = fmaf(g[j], b[k], gB[k]);
                            const float q = g[j] * w[j][k];
                            dA[j] = fmaf(q, dt[k], dA[j]);  // at a start w is 0, and dt put to 0
                            grad_dt[k] = fmaf(q, A_s, grad_dt[k]);
                        }
                        if constexpr (L == 1) carry[s0 + i + j] = pass<CUT>(a[j][0], g[j]);
                        bc[set][i + j][in_wave] = sum_rows<L>(v[j], in_wave);
                    }
                    row_sum<L>(dA);
#pragma unroll
                    for (int j = 0; j < 2; ++j)  // all lanes of the row write the same value
                        grad_A[s0 + i + j] += L == 16 ? row_last<false, L>(dA[j]) : dA[j];
                }
            };
            const auto scan_serially = [&](int most) {
#pragma unroll 1
                for (int i = 0; i < most; ++i) {
                    if (!mine(s0 + i)) continue;
                    const int at = s0 + i;
                    const float A_s = A[at], a2 = A_s * kLog2e;
                    float b[K], c[K], w[K], v[16];
                    read_tile(B_tile[i], l.lane, b);
#pragma unroll
                    for (int k = 0; k < K; ++k) b[k] *= dtu[k];
                    float h = serial_enter<FLAGS, L>(dt, cut, b, a2, enter_states[at], l.lane);
                    read_tile(C_tile[i], l.lane, c);
#pragma unroll
                    for (int k = 0; k < K; ++k) {
                        w[k] = serial_pass<FLAGS>(dt[k], cut[k], a2, h);
                        h = b[k] + w[k];
                        v[8 + k] = gy[k] * h;
                        if constexpr (GATE) y[k] = fmaf(c[k], h, y[k]);
                        c[k] *= gy[k];
                    }
                    float g = serial_enter_back<FLAGS, L>(dt, cut, c, a2, carry[at], l.lane);
                    float dA[2] = {0.f, 0.f};
                    read_tile(B_tile[i], l.lane, b);
#pragma unroll
                    for (int k = K - 1; k >= 0; --k) {
                        g += c[k];
                        v[k] = g * dtu[k];
                        gB[k] = fmaf(g, b[k], gB[k]);
                        const float q = g * w[k];
                        dA[0] = fmaf(q, dt[k], dA[0]);
                        grad_dt[k] = fmaf(q, A_s, grad_dt[k]);
                        g = serial_pass<FLAGS>(dt[k], cut[k], a2, g);
                    }
                    bc[set][i][in_wave] = sum_rows<L>(v, in_wave);
                    if constexpr (L > 1)
                        carry[at] = row_last<true, L>(g);
                    else
                        carry[at] = g;
                    row_sum<L>(dA);
                    grad_A[at] += L == 16 ? row_last<false, L>(dA[0]) : dA[0];
                }
            };
            bool plain = true;
            if constexpr (FLAGS) {
                uint32_t staged = 1u;
#pragma unroll
                for (int w = 0; w < kThreads / kWave; ++w) staged &= stage_tame[buffer][w];
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
            if constexpr (SPLIT > 1) {
                if (s0 + kStates >= S) {  // the tile's last stage
#pragma unroll
                    for (int k = 0; k < K; ++k) {
                        after[wave][k][in_wave] = gB[k];
                        after[wave][K + k][in_wave] = grad_dt[k];
                        if constexpr (GATE) after[wave][2 * K + k][in_wave] = y[k];
                    }
                }
            }
            __syncthreads();
            if constexpr (L == 16) {
                // lane x of a wave holds, for state i, half a lane's steps of
                // grad_B (rows 0 and 1) or grad_C (rows 2 and 3)
                for (int j = thread; j < count * kWave; j += kThreads) {
                    const int i = j / kWave, x = j % kWave, q = x / 16;
                    float4v sum = bc[0][i][x];
#pragma unroll
                    for (int m = 1; m < kSets; ++m) sum += bc[m][i][x];
                    float *to = partials + ((int64_t)(q >> 1) * S + s0 + i) * p.tiles * kTile + t0 +
                                (x % 16) * K + (q & 1) * 4;
                    *reinterpret_cast<float4v *>(to) = sum;
                }
            } else {
                // lane x holds value x / 4 of its place in the row (L = 4), or
                // of the row (L = 1)
                for (int j = thread; j < count * 2 * kTile; j += kThreads) {
                    const int i = j / (2 * kTile), which = j / kTile % 2, t = j % kTile;
                    const int x = (which * 8 + t % K) * 4 + t / K;
                    float sum = bc[0][i][x];
#pragma unroll
                    for (int m = 1; m < kSets; ++m) sum += bc[m][i][x];
                    partials[((int64_t)which * S + s0 + i) * p.tiles * kTile + t0 + t] = sum;
                }
            }
        }
        wave_order();
        float sum_gB[kOwn], sum_dt[kOwn], sum_y[kOwn];
#pragma unroll
        for (int k = 0; k < kOwn; ++k) {
            if constexpr (SPLIT > 1) {
                sum_gB[k] = sum_dt[k] = sum_y[k] = 0.f;
                const int at = part * kOwn + k;
#pragma unroll
                for (int q = 0; q < SPLIT; ++q) {
                    sum_gB[k] += after[set * SPLIT + q][at][in_wave];
                    sum_dt[k] += after[set * SPLIT + q][K + at][in_wave];
                    if constexpr (GATE) sum_y[k] += after[set * SPLIT + q][2 * K + at][in_wave];
                }
            } else {
                sum_gB[k] = gB[k];
                sum_dt[k] = grad_dt[k];
                sum_y[k] = y[k];
            }
        }
        const int t = t0 + own;
        if (l.live && t < p.T) {
            float own_u[kOwn], raw[kOwn], out_u[kOwn], out_delta[kOwn], own_gy[kOwn];
            if constexpr (kReload) {
                load_tile(t0);
                u = next_u;
                delta = next_delta;
                go = next_go;
                z = next_z;
            }
            u.widen(own_u);
            delta.widen(raw);
            go.widen(own_gy);
            if constexpr (GATE) {
                float own_z[kOwn], out_z[kOwn];
                z.widen(own_z);
#pragma unroll
                for (int k = 0; k < kOwn; ++k) {
                    const float sig = sigmoid(own_z[k]);
                    const float y0 = fmaf(skip, own_u[k], sum_y[k]);
                    out_z[k] = own_gy[k] * y0 * silu_slope(own_z[k], sig);
                    own_gy[k] = SPLIT == 1 ? gy[k] : own_gy[k] * (own_z[k] * sig);
                }
                if (t + kOwn > end)  // few lanes
#pragma unroll
                    for (int k = 0; k < kOwn; ++k) out_z[k] = t + k < end ? out_z[k] : 0.f;
                store_steps<kOwn>(out_row(p.grad_z, t0), p.T - t, out_z);
            }
#pragma unroll
            for (int k = 0; k < kOwn; ++k) {
                raw[k] += bias;
                // dt of this step; dt[] holds it, but for an episode's first
                // step, and at a place that depends on the part with several
                float step;
                if (SPLIT == 1 && (!FLAGS || cut[k] == 0.f))
                    step = dt[k];
                else
                    step = p.softplus != 0 ? softplus(raw[k]) : raw[k];
                out_u[k] = fmaf(step, sum_gB[k], skip * own_gy[k]);
                out_delta[k] = fmaf(own_u[k], sum_gB[k], sum_dt[k]);
                if (p.softplus != 0) out_delta[k] *= sigmoid(raw[k]);
            }
            if (t + kOwn > end)  // few lanes
#pragma unroll
                for (int k = 0; k < kOwn; ++k) {
                    const bool in = t + k < end;
                    out_u[k] = in ? out_u[k] : 0.f;
                    out_delta[k] = in ? out_delta[k] : 0.f;
                    own_gy[k] = in ? own_gy[k] : 0.f;
                }
#pragma unroll
            for (int k = 0; k < kOwn; ++k) {
                totals[0] = fmaf(own_gy[k], own_u[k], totals[0]);
                totals[1] += out_delta[k];
            }
            store_steps<kOwn>(out_row(p.grad_u, t0), p.T - t, out_u);
            store_steps<kOwn>(out_row(p.grad_delta, t0), p.T - t, out_delta);
        }
    }
    row_sum<L>(totals);
    if constexpr (SPLIT > 1) {  // the parts' totals, in order
        __syncthreads();
        if (l.lane == L - 1)
#pragma unroll
            for (int q = 0; q < 2; ++q) after[wave][q][in_wave] = totals[q];
        __syncthreads();
        if (l.lane == L - 1)
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                totals[q] = 0.f;
#pragma unroll
                for (int m = 0; m < SPLIT; ++m) totals[q] += after[set * SPLIT + m][q][in_wave];
            }
    }
    if (!l.live) return true;
    float *out = p.row_partials + (int64_t)l.row * (S + 2);
    for (int s = l.lane; s < S; s += L)
        if (mine(s)) {
            out[s] = grad_A[s];
            if (p.grad_state != nullptr) p.grad_state[(int64_t)l.row * S + s] = carry[s];
        }
    if (part == 0 && l.lane == L - 1) {
        out[S] = totals[0];
        out[S + 1] = totals[1];
    }
    return true;
}

// GIVEN: steps without softplus, which may be below 0.
template <typename E, bool FLAGS, bool GATE, int SPLIT, int L, bool GIVEN>
__global__ __launch_bounds__(kScanThreads *SPLIT, 2) void selective_scan_backward(ScanParams p) {
    extern __shared__ __attribute__((aligned(16))) char lds_bytes[];
    constexpr int kWaves = kScanWaves * SPLIT;
    constexpr int kBefore = FLAGS ? 4 : 3, kAfter = GATE ? 3 : 2;  // values a step that waves share
    __shared__ TileRow<L> tiles[2][2][states_of(L)];  // [buffer][B, C][state]
    __shared__ RowSums<L> bc[kScanWaves][states_of(L)][kWave];
    __shared__ float before[SPLIT > 1 ? kScanWaves : 1][SPLIT > 1 ? kBefore * kScanK : 1][kWave];
    __shared__ float after[SPLIT > 1 ? kWaves : 1][SPLIT > 1 ? kAfter * kScanK : 1][kWave];
    __shared__ uint32_t steady_waves[kWaves];
    __shared__ uint32_t stage_tame[2][kWaves];  // [buffer]: whether what a wave staged is
    if constexpr (GIVEN)
        scan_rows_back<E, FLAGS, GATE, SPLIT, L, true>(p, threadIdx.x, lds_bytes, tiles, bc, before,
                                                       after, steady_waves, stage_tame);
    else if (!scan_rows_back<E, FLAGS, GATE, SPLIT, L, false>(
                 p, threadIdx.x, lds_bytes, tiles, bc, before, after, steady_waves, stage_tame))
        scan_rows_back<E, FLAGS, GATE, SPLIT, L, true>(
            arguments_again<ScanParams>(), here(threadIdx.x), lds_bytes, tiles, bc, before, after,
            steady_waves, stage_tame);
}

// grad_B and grad_C: the sum of a group's workgroups, in order, 4 steps a lane.
// 2^lane_bits lanes share a row (a sequence, group and state of one of the
// two), so that short rows fill a workgroup too.
struct BcSums {
    const float *partials;
    void *grad_B, *grad_C;
    const int32_t *lengths;
    uint32_t blocks, states, groups, rows;  // rows: num_seqs * groups * 2 * states
    uint32_t lane_bits;
    int32_t T, padded;  // padded: whole tiles
};

template <typename E>
__global__ __launch_bounds__(kScanThreads) void bc_sums(BcSums p) {
    const uint32_t lanes = 1u << p.lane_bits, rows = kScanThreads >> p.lane_bits;
    const int lane = (int)(threadIdx.x & (lanes - 1));
    for (uint64_t r64 = (uint64_t)blockIdx.x * rows + (threadIdx.x >> p.lane_bits); r64 < p.rows;
         r64 += (uint64_t)gridDim.x * rows) {
        const uint32_t r = (uint32_t)r64;
        const uint32_t ng = r / (2 * p.states), which = r / p.states & 1, s = r % p.states;
        const int end = row_end(p.lengths, ng / p.groups, p.T);
        const int64_t step = (int64_t)2 * p.states * p.padded;
        const float *from = p.partials + (int64_t)ng * p.blocks * step +
                            ((int64_t)which * p.states + s) * p.padded;
        E *to = static_cast<E *>(which == 0 ? p.grad_B : p.grad_C) +
                ((int64_t)ng * p.states + s) * p.T;
        for (int t = ((int)(blockIdx.y << p.lane_bits) + lane) * 4; t < p.T;
             t += (int)(gridDim.y << p.lane_bits) * 4) {
            float4v sum = {};
            if (t < end)  // beyond, nothing was written
#pragma unroll 4
                for (uint32_t b = 0; b < p.blocks; ++b)
                    sum += *reinterpret_cast<const float4v *>(from + b * step + t);
            float v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] = t + k < end ? sum[k] : 0.f;
            store_steps<4>(to + t, p.T - t, v);
        }
    }
}

// grad_A, grad_D and grad_delta_bias: the sums over sequences, in fp64.  A
// workgroup takes kSumValues neighbouring values; its lanes of one value take
// every so many sequences and meet in LDS in a fixed tree.  Many sequences are
// first summed in ranges (blockIdx.y) into `ranges`, and those by a second launch.
constexpr int kSumValues = 16, kSumThreads = 1024, kSumRange = 256;
constexpr uint32_t kMostRanges = 1u << 15;

template <typename In>
__global__ __launch_bounds__(kSumThreads) void row_sums(const In *partials, uint32_t parts,
                                                        uint32_t channels, uint32_t states,
                                                        uint32_t range, double *ranges,
                                                        float *grad_A, float *grad_D,
                                                        float *grad_bias) {
    __shared__ double sums[kSumThreads];
    const int64_t width = states + 2, count = (int64_t)channels * width;
    const uint32_t lanes = blockDim.x / kSumValues;  // a power of two
    const uint32_t lane = threadIdx.x / kSumValues;
    const uint64_t begin = (uint64_t)blockIdx.y * range;
    const uint32_t end = begin + range < parts ? (uint32_t)(begin + range) : parts;
    for (int64_t i0 = (int64_t)blockIdx.x * kSumValues; i0 < count;
         i0 += (int64_t)gridDim.x * kSumValues) {
        const int64_t i = i0 + threadIdx.x % kSumValues;
        double sum = 0.0;
        if (i < count)
#pragma unroll 4
            for (uint64_t n = begin + lane; n < end; n += lanes)
                sum += (double)partials[n * count + i];
        sums[threadIdx.x] = sum;
        for (uint32_t m = lanes / 2; m > 0; m /= 2) {
            __syncthreads();
            if (lane < m) sums[threadIdx.x] += sums[threadIdx.x + m * kSumValues];
        }
        if (lane == 0 && i < count) {
            const double total = sums[threadIdx.x];
            const int64_t d = i / width;
            const int s = (int)(i - d * width);
            if (ranges != nullptr) {
                ranges[blockIdx.y * count + i] = total;
            } else if (s < (int)states) {
                grad_A[d * states + s] = (float)total;
            } else if (s == (int)states) {
                if (grad_D != nullptr) grad_D[d] = (float)total;
            } else if (grad_bias != nullptr) {
                grad_bias[d] = (float)total;
            }
        }
        __syncthreads();
    }
}

// The workspace, in floats: the partial sums of grad_B and grad_C, those of
// each sequence's rows, and (fp64) those of ranges of sequences.
struct Workspace {
    size_t bc, rows, ranges;
    size_t total() const { return bc + rows + ranges; }
};

// How many sequences a range holds, and how many ranges (0: too few to need them).
struct Ranges {
    uint32_t size, count;
};

static Ranges ranges_of(int64_t num_seqs) {
    if (num_seqs <= 2 * kSumRange) return {(uint32_t)num_seqs, 0};
    int64_t size = kSumRange;
    while ((num_seqs + size - 1) / size > kMostRanges) size *= 2;
    return {(uint32_t)size, (uint32_t)((num_seqs + size - 1) / size)};
}

// Waves that share four channels: two where one would leave the SIMDs a single
// wave each (with one and two, forward and backward, 16 states, bf16: 1024
// channels of 4096 steps 405 and 375 us, 4096 of 4096 502 and 480, 2048 of 2048 223
// and 208, 4x1024 of 2048 244 and 230; 5120 354 and 414, 8192 430 and 492).  Above 64 states two would need over 160 KB of LDS.
static int split_of(const rlca_scan_call &c) {
    return c.num_seqs * c.channels <= 4096 && c.states > 2 && c.states <= 64 ? 2 : 1;
}

static Workspace workspace_of(const rlca_scan_call &c) {
    const int lanes = lanes_of(c), tile = tile_of(lanes);
    const int64_t padded = (c.T + tile - 1) / tile * tile;
    const int64_t per_group = c.groups == 0 ? 0 : c.channels / c.groups;
    const int64_t blocks = c.num_seqs * c.groups * ((per_group + rows_of(lanes) - 1) / rows_of(lanes));
    return {(size_t)(blocks * 2 * c.states * padded),
            (size_t)((c.num_seqs * c.channels * (c.states + 2) + 3) / 4 * 4),
            (size_t)(2 * ranges_of(c.num_seqs).count * c.channels * (c.states + 2))};
}

template <typename E, int SPLIT, int L, bool GIVEN>
static const void *backward_kernel(const rlca_scan_call &c) {
    const bool flags = c.flags != nullptr, gate = c.z != nullptr;
    return flags ? (gate ? (const void *)selective_scan_backward<E, true, true, SPLIT, L, GIVEN>
                         : (const void *)selective_scan_backward<E, true, false, SPLIT, L, GIVEN>)
                 : (gate ? (const void *)selective_scan_backward<E, false, true, SPLIT, L, GIVEN>
                         : (const void *)selective_scan_backward<E, false, false, SPLIT, L, GIVEN>);
}

template <typename E, int SPLIT, int L>
static const void *backward_kernel(const rlca_scan_call &c) {
    return c.softplus == 0 ? backward_kernel<E, SPLIT, L, true>(c)
                           : backward_kernel<E, SPLIT, L, false>(c);
}

template <typename E>
static const void *backward_kernel(const rlca_scan_call &c, int split, int lanes) {
    return lanes == 1   ? backward_kernel<E, 1, 1>(c)
           : lanes == 4 ? backward_kernel<E, 1, 4>(c)
           : split == 2 ? backward_kernel<E, 2, 16>(c)
                        : backward_kernel<E, 1, 16>(c);
}

}  // namespace seq
}  // namespace rlca

using namespace rlca::seq;

extern "C" {

size_t rlca_selective_scan_backward_workspace_size(const rlca_scan_call *call) {
    Arrays a;
    if (call == nullptr || check_scan(*call, true, &a) != RLCA_OK) return 0;
    const Workspace w = workspace_of(*call);
    return w.total() * 4;
}

rlca_status rlca_selective_scan_backward(const rlca_scan_call *call, void *workspace,
                                         size_t workspace_bytes, hipStream_t stream) {
    if (call == nullptr) return RLCA_ERR_NULL_POINTER;
    const rlca_scan_call &c = *call;
    Arrays a;
    rlca_status st = check_scan(c, true, &a);
    if (st != RLCA_OK) return st;
    const Workspace w = workspace_of(c);
    a.out(workspace, 16, true, {{(int64_t)((w.total() + 3) / 4), 1}});
    st = a.status();
    if (st != RLCA_OK) return st;
    if (workspace_bytes < w.total() * 4) return RLCA_ERR_INVALID_SIZE;
    if (c.channels == 0) return RLCA_OK;
    const int lanes = lanes_of(c), split = lanes == 16 ? split_of(c) : 1;
    ScanParams p = scan_params(c, rows_of(lanes));
    p.bc_partials = static_cast<float *>(workspace);
    p.row_partials = p.bc_partials + w.bc;
    if (c.num_seqs != 0) {
        const void *kernel = c.dtype == RLCA_F32    ? backward_kernel<float>(c, split, lanes)
                             : c.dtype == RLCA_BF16 ? backward_kernel<__bf16>(c, split, lanes)
                                                    : backward_kernel<_Float16>(c, split, lanes);
        st = launch(kernel, dim3(p.num_seqs * p.groups * p.blocks_per_group),
                    kScanThreads * split, 4 * rows_of(lanes) * pitch_of(c.states, lanes) * 4, p,
                    stream);
        if (st != RLCA_OK) return st;
        if (p.T != 0) {
            BcSums b = {};
            b.partials = p.bc_partials;
            b.grad_B = c.grad_B;
            b.grad_C = c.grad_C;
            b.lengths = c.lengths;
            b.blocks = p.blocks_per_group;
            b.states = p.states;
            b.groups = p.groups;
            b.rows = p.num_seqs * p.groups * 2 * p.states;
            b.T = p.T;
            b.padded = p.tiles * tile_of(lanes);
            while ((4 << b.lane_bits) < p.T && (1 << b.lane_bits) < kScanThreads) ++b.lane_bits;
            const uint32_t across = (p.T + (4 << b.lane_bits) - 1) / (4 << b.lane_bits);
            const uint32_t at_once = kScanThreads >> b.lane_bits;
            const uint32_t down = (b.rows + at_once - 1) / at_once;
            const void *sums = c.dtype == RLCA_F32    ? (const void *)bc_sums<float>
                               : c.dtype == RLCA_BF16 ? (const void *)bc_sums<__bf16>
                                                      : (const void *)bc_sums<_Float16>;
            st = launch(sums, dim3(down < (1u << 18) ? down : 1u << 18, across < 64 ? across : 64),
                        kScanThreads, 0, b, stream);
            if (st != RLCA_OK) return st;
        }
    }
    const Ranges ranges = ranges_of(c.num_seqs);
    const uint64_t groups = ((uint64_t)p.channels * (p.states + 2) + kSumValues - 1) / kSumValues;
    const uint32_t across = (uint32_t)(groups < (1u << 20) ? groups : 1u << 20);
    double *range_sums = reinterpret_cast<double *>(p.row_partials + w.rows);
    for (int pass = ranges.count == 0 ? 1 : 0; pass < 2; ++pass) {
        // pass 0: rows into ranges; pass 1: ranges, or rows if few, into the gradients
        const bool into_ranges = pass == 0, of_rows = into_ranges || ranges.count == 0;
        const void *in = of_rows ? (const void *)p.row_partials : (const void *)range_sums;
        uint32_t parts = of_rows ? p.num_seqs : ranges.count;
        uint32_t range = into_ranges ? ranges.size : parts;
        double *out = into_ranges ? range_sums : nullptr;
        float *gA = c.grad_A, *gD = c.grad_D, *gb = c.grad_delta_bias;
        void *args[] = {&in, &parts, &p.channels, &p.states, &range, &out, &gA, &gD, &gb};
        uint32_t threads = rlca::kWave;
        while (threads < (uint32_t)kSumThreads && threads / kSumValues < range) threads *= 2;
        const hipError_t e = hipLaunchKernel(
            of_rows ? (const void *)row_sums<float> : (const void *)row_sums<double>,
            dim3(across, into_ranges ? ranges.count : 1), dim3(threads), args, 0, stream);
        if (e != hipSuccess) return RLCA_ERR_HIP;
    }
    return RLCA_OK;
}

}  // extern "C"
