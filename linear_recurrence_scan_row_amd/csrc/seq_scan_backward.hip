// seq_scan_backward.hip -- the gradients of the selective scan.  With
// gy_t = grad_y_t silu(z_t), and for each channel and state
//   g_t = C_t gy_t + a_{t+1} g_{t+1}             (dL/dh_t, from the last step back)
//   w_t = a_t h_{t-1}
//   grad_C_t = sum_d gy_t h_t                    grad_B_t = sum_d g_t dt_t u_t
//   grad_dt_t = sum_s g_t w_t A + u_t sum_s g_t B_t
//   grad_u_t = dt_t sum_s g_t B_t + D gy_t       grad_A = sum_t g_t w_t dt_t
// A workgroup walks its 16 channels' tiles from the last to the first.  The
// state that enters a tile comes from the forward call's checkpoints, the
// tile's states from one forward scan, and g from one reverse scan whose carry
// r = a_t g_t passes to the tile before.
//
// grad_B and grad_C sum over the channels of a group.  Within a wave the four
// rows hold four channels of the same steps: 16 values (8 steps of each
// gradient) meet in 12 lane-half swaps and 12 additions, after which each row
// holds the sums of four of them.  The waves' sums meet in LDS, the
// workgroups' in a workspace that bc_sums adds in order.
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

// v[0..15] of four rows -> row q's lanes hold the sums over rows of v[4q .. 4q+3].
__device__ __forceinline__ float4v sum_rows(float (&v)[16]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) swap_add(v[i], v[8 + i], true);
#pragma unroll
    for (int i = 0; i < 4; ++i) swap_add(v[i], v[4 + i], false);
    float4v r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = v[i];
    return r;
}

// Sum over a row's 16 lanes, complete in lane 15.
__device__ __forceinline__ float row_sum(float x) {
    x += dpp_move<0x111, 0xf>(x, 0.f);
    x += dpp_move<0x112, 0xf>(x, 0.f);
    x += dpp_move<0x114, 0xf>(x, 0.f);
    x += dpp_move<0x118, 0xf>(x, 0.f);
    return x;
}

template <typename E, bool FLAGS>
__global__ __launch_bounds__(kScanThreads) void selective_scan_backward(ScanParams p) {
    extern __shared__ __attribute__((aligned(16))) char lds_bytes[];
    __shared__ TileRow B_tile[kScanStates], C_tile[kScanStates];
    __shared__ float4v bc[kScanWaves][kScanStates][kWave];
    const ScanLane l = scan_lane(p);
    const int S = (int)p.states;
    // [rows][S]: A, the gradient a_t g_t entering the tile from its right, and
    // the sums of grad_A
    float *A = reinterpret_cast<float *>(lds_bytes) + l.local * S;
    float *carry = A + kScanRows * S;
    float *grad_A = carry + kScanRows * S;
    const int row_steps = row_end(p.lengths, l.n, p.T);
    const int end = l.live ? row_steps : 0;  // a clamped row computes on zeros
    const uint8_t *flags = FLAGS ? p.flags + (int64_t)l.n * p.T : nullptr;
    const bool over = FLAGS && p.after_done != 0 && end > 0 && flags[end - 1] != 0;
    for (int s = l.lane; s < S; s += kScanLanes) {
        A[s] = p.A[(int64_t)l.d * S + s];
        carry[s] = p.grad_final == nullptr || over || !l.live
                       ? 0.f
                       : p.grad_final[(int64_t)l.row * S + s];
        grad_A[s] = 0.f;
    }
    const E *u_row = static_cast<const E *>(p.u) + l.n * p.u_n + l.d * p.u_d;
    const E *delta_row = static_cast<const E *>(p.delta) + l.n * p.delta_n + l.d * p.delta_d;
    const E *g_row = static_cast<const E *>(p.grad_y) + l.n * p.g_n + l.d * p.g_d;
    const E *z_row =
        p.z == nullptr ? nullptr : static_cast<const E *>(p.z) + l.n * p.z_n + l.d * p.z_d;
    const E *B = static_cast<const E *>(p.B) + l.n * p.B_n + l.g * p.B_g;
    const E *C = static_cast<const E *>(p.C) + l.n * p.C_n + l.g * p.C_g;
    const float bias = p.delta_bias == nullptr ? 0.f : p.delta_bias[l.d];
    const float skip = p.D == nullptr ? 0.f : p.D[l.d];
    const int64_t out_row = (int64_t)l.row * p.T;
    const int wave = threadIdx.x / kWave;
    float *partials = p.bc_partials + (int64_t)blockIdx.x * 2 * S * p.tiles * kScanTile;
    float grad_D = 0.f, grad_bias = 0.f;

    for (int tile = p.tiles - 1; tile >= 0; --tile) {
        const int t0 = tile * kScanTile, t = t0 + l.lane * kScanK;
        float dt[kScanK], raw[kScanK], u[kScanK], dtu[kScanK], cut[kScanK], gy[kScanK], y[kScanK];
        load_inputs<E, FLAGS>(p, u_row, delta_row, flags, bias, t, end, row_steps, dt, raw, u,
                              dtu, cut);
        load_steps<kScanK>(g_row + t, end - t, gy);
        if (z_row != nullptr) {
            float z[kScanK];
            load_steps<kScanK>(z_row + t, end - t, z);
#pragma unroll
            for (int k = 0; k < kScanK; ++k) gy[k] = t + k < end ? gy[k] * silu(z[k]) : 0.f;
        }
        float grad_dt[kScanK], gB[kScanK], dt_sum = 0.f;
        bool starts = false;
#pragma unroll
        for (int k = 0; k < kScanK; ++k) {
            dt_sum += dt[k];
            if constexpr (FLAGS) starts |= cut[k] != 0.f;
            y[k] = skip * u[k];
            grad_dt[k] = gB[k] = 0.f;
        }
        const float *enter_row = p.checkpoints + ((int64_t)l.row * p.tiles + tile) * S;
        for (int s0 = 0; s0 < S; s0 += kScanStates) {
            const int count = S - s0 < kScanStates ? S - s0 : kScanStates;
            __syncthreads();  // the tiles and sums before are used up
            stage_rows(B_tile, B, p.B_s, s0, count, t0, row_steps);
            stage_rows(C_tile, C, p.C_s, s0, count, t0, row_steps);
            __syncthreads();
            for (int i = 0; i < count; ++i) {
                const float A_s = A[s0 + i], a2 = A_s * kLog2e;
                const float enter = l.live ? enter_row[s0 + i] : 0.f;
                float a[kScanK], b[kScanK], c[kScanK], w[kScanK], v[16];
                read_tile(B_tile[i], l.lane, b);
                read_tile(C_tile[i], l.lane, c);
                float h = 0.f;
#pragma unroll
                for (int k = 0; k < kScanK; ++k) {
                    a[k] = decay<FLAGS>(dt[k], cut[k], a2);
                    h = step_map<FLAGS>(a[k], b[k] * dtu[k], h);
                }
                const float prod = lane_product<FLAGS>(dt_sum, starts, a2);
                float prefix = prod;
                row_scan<FLAGS, false>(prefix, h);
                h = row_shift<false>(step_map<FLAGS>(prefix, h, enter), enter);
#pragma unroll
                for (int k = 0; k < kScanK; ++k) {
                    w[k] = product<FLAGS>(a[k], h);
                    h = fmaf(b[k], dtu[k], w[k]);
                    v[8 + k] = gy[k] * h;
                    y[k] = fmaf(c[k], h, y[k]);
                    c[k] *= gy[k];  // what y's gradient adds to g
                }
                float g = c[kScanK - 1];
#pragma unroll
                for (int k = kScanK - 2; k >= 0; --k) g = step_map<FLAGS>(a[k + 1], c[k], g);
                float r = product<FLAGS>(a[0], g), suffix = prod;
                row_scan<FLAGS, true>(suffix, r);
                const float right = carry[s0 + i];
                r = step_map<FLAGS>(suffix, r, right);
                if (l.lane == 0) carry[s0 + i] = r;
                g = row_shift<true>(r, right);  // a_{t+8} g_{t+8}
                float dA = 0.f;
#pragma unroll
                for (int k = kScanK - 1; k >= 0; --k) {
                    g = k == kScanK - 1 ? c[k] + g : step_map<FLAGS>(a[k + 1], c[k], g);
                    v[k] = g * dtu[k];
                    gB[k] = fmaf(g, b[k], gB[k]);
                    const float q = g * w[k];
                    dA = fmaf(q, dt[k], dA);  // at a start w is 0, and dt put to 0
                    grad_dt[k] = fmaf(q, A_s, grad_dt[k]);
                }
                bc[wave][i][threadIdx.x & (kWave - 1)] = sum_rows(v);
                dA = row_sum(dA);
                if (l.lane == kScanLanes - 1) grad_A[s0 + i] += dA;
            }
            __syncthreads();
            // lane x of a wave holds, for state i, four steps of grad_B (rows 0
            // and 1) or grad_C (rows 2 and 3)
            for (int j = threadIdx.x; j < count * kWave; j += kScanThreads) {
                const int i = j / kWave, x = j % kWave, q = x / kScanLanes;
                float4v sum = bc[0][i][x];
#pragma unroll
                for (int m = 1; m < kScanWaves; ++m) sum += bc[m][i][x];
                float *to = partials + ((int64_t)(q >> 1) * S + s0 + i) * p.tiles * kScanTile + t0 +
                            (x % kScanLanes) * kScanK + (q & 1) * 4;
                *reinterpret_cast<float4v *>(to) = sum;
            }
        }
        wave_order();
        if (l.live && t < p.T) {
            float gz[kScanK], gu[kScanK];
            if (z_row != nullptr) {
                float z[kScanK], go[kScanK];
                load_steps<kScanK>(z_row + t, end - t, z);
                load_steps<kScanK>(g_row + t, end - t, go);
#pragma unroll
                for (int k = 0; k < kScanK; ++k)
                    gz[k] = t + k < end ? go[k] * y[k] * silu_slope(z[k], sigmoid(z[k])) : 0.f;
                store_steps<kScanK>(static_cast<E *>(p.grad_z) + out_row + t, p.T - t, gz);
            }
#pragma unroll
            for (int k = 0; k < kScanK; ++k) {
                const bool in = t + k < end;
                // an episode's first step has its dt put to 0 for a alone
                const float step = !FLAGS || cut[k] == 0.f ? dt[k]
                                   : p.softplus != 0       ? softplus(raw[k])
                                                           : raw[k];
                gu[k] = in ? fmaf(step, gB[k], skip * gy[k]) : 0.f;
                float gd = fmaf(u[k], gB[k], grad_dt[k]);
                if (p.softplus != 0) gd *= sigmoid(raw[k]);
                grad_dt[k] = in ? gd : 0.f;
                grad_D += in ? gy[k] * u[k] : 0.f;
                grad_bias += grad_dt[k];
            }
            store_steps<kScanK>(static_cast<E *>(p.grad_u) + out_row + t, p.T - t, gu);
            store_steps<kScanK>(static_cast<E *>(p.grad_delta) + out_row + t, p.T - t, grad_dt);
        }
    }
    grad_D = row_sum(grad_D);
    grad_bias = row_sum(grad_bias);
    if (!l.live) return;
    float *out = p.row_partials + (int64_t)l.row * (S + 2);
    for (int s = l.lane; s < S; s += kScanLanes) {
        out[s] = grad_A[s];
        if (p.grad_state != nullptr) p.grad_state[(int64_t)l.row * S + s] = carry[s];
    }
    if (l.lane == kScanLanes - 1) {
        out[S] = grad_D;
        out[S + 1] = grad_bias;
    }
}

// grad_B and grad_C: the sum of a group's workgroups, in order, 4 steps a lane.
struct BcSums {
    const float *partials;
    void *grad_B, *grad_C;
    const int32_t *lengths;
    uint32_t blocks, states, groups, rows;  // rows: num_seqs * groups * 2 * states
    int32_t T, padded;                      // padded: tiles * kScanTile
};

template <typename E>
__global__ __launch_bounds__(kScanThreads) void bc_sums(BcSums p) {
    for (uint32_t r = blockIdx.x; r < p.rows; r += gridDim.x) {
        const uint32_t ng = r / (2 * p.states), which = r / p.states & 1, s = r % p.states;
        const int end = row_end(p.lengths, ng / p.groups, p.T);
        const int64_t step = (int64_t)2 * p.states * p.padded;
        const float *from = p.partials + (int64_t)ng * p.blocks * step +
                            ((int64_t)which * p.states + s) * p.padded;
        E *to = static_cast<E *>(which == 0 ? p.grad_B : p.grad_C) +
                ((int64_t)ng * p.states + s) * p.T;
        for (int t = (int)(blockIdx.y * kScanThreads + threadIdx.x) * 4; t < p.T;
             t += (int)(gridDim.y * kScanThreads * 4)) {
            float4v sum = *reinterpret_cast<const float4v *>(from + t);
            for (uint32_t b = 1; b < p.blocks; ++b)
                sum += *reinterpret_cast<const float4v *>(from + b * step + t);
            float v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] = t + k < end ? sum[k] : 0.f;
            store_steps<4>(to + t, p.T - t, v);
        }
    }
}

// grad_A, grad_D and grad_delta_bias: the sum over sequences, in fp64; a wave
// takes 64 neighbouring values.
__global__ __launch_bounds__(kWave) void row_sums(const float *partials, uint32_t num_seqs,
                                                  uint32_t channels, uint32_t states,
                                                  float *grad_A, float *grad_D,
                                                  float *grad_bias) {
    const int64_t width = states + 2, count = (int64_t)channels * width;
    for (int64_t i = (int64_t)blockIdx.x * kWave + threadIdx.x; i < count;
         i += (int64_t)gridDim.x * kWave) {
        double sum = 0.0;
        for (uint32_t n = 0; n < num_seqs; ++n) sum += (double)partials[n * count + i];
        const int64_t d = i / width;
        const int s = (int)(i - d * width);
        if (s < (int)states)
            grad_A[d * states + s] = (float)sum;
        else if (s == (int)states) {
            if (grad_D != nullptr) grad_D[d] = (float)sum;
        } else if (grad_bias != nullptr) {
            grad_bias[d] = (float)sum;
        }
    }
}

struct Workspace {
    size_t bc, rows;  // floats
};

static Workspace workspace_of(const rlca_scan_call &c) {
    const int64_t tiles = (c.T + kScanTile - 1) / kScanTile;
    const int64_t per_group = c.groups == 0 ? 0 : c.channels / c.groups;
    const int64_t blocks = c.num_seqs * c.groups * ((per_group + kScanRows - 1) / kScanRows);
    return {(size_t)(blocks * 2 * c.states * tiles * kScanTile),
            (size_t)(c.num_seqs * c.channels * (c.states + 2))};
}

}  // namespace seq
}  // namespace rlca

using namespace rlca::seq;

extern "C" {

size_t rlca_selective_scan_backward_workspace_size(const rlca_scan_call *call) {
    Arrays a;
    if (call == nullptr || check_scan(*call, true, &a) != RLCA_OK) return 0;
    const Workspace w = workspace_of(*call);
    return (w.bc + w.rows) * 4;
}

rlca_status rlca_selective_scan_backward(const rlca_scan_call *call, void *workspace,
                                         size_t workspace_bytes, hipStream_t stream) {
    if (call == nullptr) return RLCA_ERR_NULL_POINTER;
    const rlca_scan_call &c = *call;
    Arrays a;
    rlca_status st = check_scan(c, true, &a);
    if (st != RLCA_OK) return st;
    const Workspace w = workspace_of(c);
    a.out(workspace, 16, true, {{(int64_t)((w.bc + w.rows + 3) / 4), 1}});
    st = a.status();
    if (st != RLCA_OK) return st;
    if (workspace_bytes < (w.bc + w.rows) * 4) return RLCA_ERR_INVALID_SIZE;
    if (c.channels == 0) return RLCA_OK;
    ScanParams p = scan_params(c);
    p.bc_partials = static_cast<float *>(workspace);
    p.row_partials = p.bc_partials + w.bc;
    const bool flags = c.flags != nullptr;
    if (c.num_seqs != 0) {
        const void *kernel =
            c.dtype == RLCA_F32    ? (flags ? (const void *)selective_scan_backward<float, true>
                                            : (const void *)selective_scan_backward<float, false>)
            : c.dtype == RLCA_BF16 ? (flags ? (const void *)selective_scan_backward<__bf16, true>
                                            : (const void *)selective_scan_backward<__bf16, false>)
                                   : (flags
                                          ? (const void *)selective_scan_backward<_Float16, true>
                                          : (const void *)selective_scan_backward<_Float16, false>);
        st = launch(kernel, dim3(p.num_seqs * p.groups * p.blocks_per_group), kScanThreads,
                    3 * kScanRows * p.states * 4, p, stream);
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
            b.padded = p.tiles * kScanTile;
            const uint32_t across = (p.T + kScanThreads * 4 - 1) / (kScanThreads * 4);
            const void *sums = c.dtype == RLCA_F32    ? (const void *)bc_sums<float>
                               : c.dtype == RLCA_BF16 ? (const void *)bc_sums<__bf16>
                                                      : (const void *)bc_sums<_Float16>;
            st = launch(sums, dim3(b.rows < (1u << 18) ? b.rows : 1u << 18, across < 64 ? across : 64),
                        kScanThreads, 0, b, stream);
            if (st != RLCA_OK) return st;
        }
    }
    const float *partials = p.row_partials;
    uint32_t num_seqs = p.num_seqs, channels = p.channels, states = p.states;
    float *gA = c.grad_A, *gD = c.grad_D, *gb = c.grad_delta_bias;
    void *args[] = {&partials, &num_seqs, &channels, &states, &gA, &gD, &gb};
    const uint64_t waves = ((uint64_t)channels * (states + 2) + rlca::kWave - 1) / rlca::kWave;
    const hipError_t e =
        hipLaunchKernel((const void *)row_sums, dim3(waves < (1u << 20) ? waves : 1u << 20),
                        dim3(rlca::kWave), args, 0, stream);
    return e == hipSuccess ? RLCA_OK : RLCA_ERR_HIP;
}

}  // extern "C"
