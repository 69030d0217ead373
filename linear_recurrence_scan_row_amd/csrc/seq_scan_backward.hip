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

// Sums over a row's 16 lanes of two values, complete in lane 15.
__device__ __forceinline__ void row_sum(float (&x)[2]) {
    // the two take turns, and one idle instruction keeps the required two
    // between a write and the lane-crossing read of it
#define RLCA_STEP(SHIFT)                                                  \
    "v_add_f32_dpp %0, %0, %0 " SHIFT " row_mask:0xf bank_mask:0xf\n\t"   \
    "v_add_f32_dpp %1, %1, %1 " SHIFT " row_mask:0xf bank_mask:0xf\n\t"   \
    "s_nop 0\n\t"
    asm("s_nop 1\n\t" RLCA_STEP("row_shr:1") RLCA_STEP("row_shr:2") RLCA_STEP("row_shr:4")
            RLCA_STEP("row_shr:8")
        : "+v"(x[0]), "+v"(x[1]));
#undef RLCA_STEP
}

template <typename E, bool FLAGS>
__global__ __launch_bounds__(kScanThreads) void selective_scan_backward(ScanParams p) {
    extern __shared__ __attribute__((aligned(16))) char lds_bytes[];
    __shared__ TileRow B_tile[kScanStates], C_tile[kScanStates];
    __shared__ float4v bc[kScanWaves][kScanStates][kWave];
    const ScanLane l = scan_lane(p);
    const int S = (int)p.states, padded = padded_states(S);
    // [rows][padded]: A, the gradient a_t g_t entering the tile from its right, and
    // the sums of grad_A
    float *A = reinterpret_cast<float *>(lds_bytes) + l.local * padded;
    float *carry = A + kScanRows * padded;
    float *grad_A = carry + kScanRows * padded;
    const int row_steps = row_end(p.lengths, l.n, p.T);
    const int end = l.live ? row_steps : 0;  // a clamped row computes on zeros
    const uint8_t *flags = FLAGS ? p.flags + (int64_t)l.n * p.T : nullptr;
    const bool over = FLAGS && p.after_done != 0 && end > 0 && flags[end - 1] != 0;
    for (int s = l.lane; s < padded; s += kScanLanes) {
        A[s] = s >= S ? 0.f : p.A[(int64_t)l.d * S + s];
        carry[s] = p.grad_final == nullptr || over || !l.live || s >= S
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
            stage_rows(B_tile, B, p.B_s, s0, S, t0, row_steps);
            stage_rows(C_tile, C, p.C_s, s0, S, t0, row_steps);
            __syncthreads();
            for (int i = 0; i < count; i += 2) {
                float a[2][kScanK], w[2][kScanK], g[2], prod[2], dA[2];
                float h[2], prefix[2], enter[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float a2 = A[s0 + i + j] * kLog2e;
                    enter[j] = l.live && s0 + i + j < S ? enter_row[s0 + i + j] : 0.f;
                    float b[kScanK];
                    read_tile(B_tile[i + j], l.lane, b);
#pragma unroll
                    for (int k = 0; k < kScanK; ++k) {
                        a[j][k] = decay<FLAGS>(dt[k], cut[k], a2);
                        const float x = b[k] * dtu[k];
                        h[j] = k == 0 ? x : step_map<FLAGS>(a[j][k], x, h[j]);
                    }
                    prefix[j] = prod[j] = lane_product<FLAGS>(dt_sum, starts, a2);
                }
                row_scan<FLAGS, false>(prefix, h);
                float v[2][16], r[2], c[2][kScanK];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    h[j] = row_shift<false>(step_map<FLAGS>(prefix[j], h[j], enter[j]), enter[j]);
                    float b[kScanK];
                    read_tile(B_tile[i + j], l.lane, b);
                    read_tile(C_tile[i + j], l.lane, c[j]);
#pragma unroll
                    for (int k = 0; k < kScanK; ++k) {
                        w[j][k] = product<FLAGS>(a[j][k], h[j]);
                        h[j] = fmaf(b[k], dtu[k], w[j][k]);
                        v[j][8 + k] = gy[k] * h[j];
                        y[k] = fmaf(c[j][k], h[j], y[k]);
                        c[j][k] *= gy[k];  // what y's gradient adds to g
                    }
                    g[j] = c[j][kScanK - 1];
#pragma unroll
                    for (int k = kScanK - 2; k >= 0; --k)
                        g[j] = step_map<FLAGS>(a[j][k + 1], c[j][k], g[j]);
                    r[j] = product<FLAGS>(a[j][0], g[j]);
                }
                row_scan<FLAGS, true>(prod, r);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float right = carry[s0 + i + j], A_s = A[s0 + i + j];
                    r[j] = step_map<FLAGS>(prod[j], r[j], right);
                    carry[s0 + i + j] = row_last<true>(r[j]);
                    g[j] = row_shift<true>(r[j], right);  // a_{t+8} g_{t+8}
                    float b[kScanK];
                    read_tile(B_tile[i + j], l.lane, b);
                    dA[j] = 0.f;
#pragma unroll
                    for (int k = kScanK - 1; k >= 0; --k) {
                        g[j] = k == kScanK - 1 ? c[j][k] + g[j]
                                               : step_map<FLAGS>(a[j][k + 1], c[j][k], g[j]);
                        v[j][k] = g[j] * dtu[k];
                        gB[k] = fmaf(g[j], b[k], gB[k]);
                        const float q = g[j] * w[j][k];
                        dA[j] = fmaf(q, dt[k], dA[j]);  // at a start w is 0, and dt put to 0
                        grad_dt[k] = fmaf(q, A_s, grad_dt[k]);
                    }
                    bc[wave][i + j][threadIdx.x & (kWave - 1)] = sum_rows(v[j]);
                }
                row_sum(dA);
                if (l.lane == kScanLanes - 1)
#pragma unroll
                    for (int j = 0; j < 2; ++j) grad_A[s0 + i + j] += dA[j];
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
    float totals[2] = {grad_D, grad_bias};
    row_sum(totals);
    if (!l.live) return;
    float *out = p.row_partials + (int64_t)l.row * (S + 2);
    for (int s = l.lane; s < S; s += kScanLanes) {
        out[s] = grad_A[s];
        if (p.grad_state != nullptr) p.grad_state[(int64_t)l.row * S + s] = carry[s];
    }
    if (l.lane == kScanLanes - 1) {
        out[S] = totals[0];
        out[S + 1] = totals[1];
    }
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
    int32_t T, padded;  // padded: tiles * kScanTile
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
            float4v sum = *reinterpret_cast<const float4v *>(from + t);
#pragma unroll 4
            for (uint32_t b = 1; b < p.blocks; ++b)
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
// every so many sequences and meet in LDS in a fixed tree.
constexpr int kSumValues = 16, kSumThreads = 1024;

__global__ __launch_bounds__(kSumThreads) void row_sums(const float *partials, uint32_t num_seqs,
                                                        uint32_t channels, uint32_t states,
                                                        float *grad_A, float *grad_D,
                                                        float *grad_bias) {
    __shared__ double sums[kSumThreads];
    const int64_t width = states + 2, count = (int64_t)channels * width;
    const uint32_t lanes = blockDim.x / kSumValues;  // a power of two
    const uint32_t lane = threadIdx.x / kSumValues;
    for (int64_t i0 = (int64_t)blockIdx.x * kSumValues; i0 < count;
         i0 += (int64_t)gridDim.x * kSumValues) {
        const int64_t i = i0 + threadIdx.x % kSumValues;
        double sum = 0.0;
        if (i < count)
#pragma unroll 8
            for (uint32_t n = lane; n < num_seqs; n += lanes) sum += (double)partials[n * count + i];
        sums[threadIdx.x] = sum;
        for (uint32_t m = lanes / 2; m > 0; m /= 2) {
            __syncthreads();
            if (lane < m) sums[threadIdx.x] += sums[threadIdx.x + m * kSumValues];
        }
        if (lane == 0 && i < count) {
            const float total = (float)sums[threadIdx.x];
            const int64_t d = i / width;
            const int s = (int)(i - d * width);
            if (s < (int)states)
                grad_A[d * states + s] = total;
            else if (s == (int)states) {
                if (grad_D != nullptr) grad_D[d] = total;
            } else if (grad_bias != nullptr) {
                grad_bias[d] = total;
            }
        }
        __syncthreads();
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
                    3 * kScanRows * padded_states(c.states) * 4, p, stream);
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
    const float *partials = p.row_partials;
    uint32_t num_seqs = p.num_seqs, channels = p.channels, states = p.states;
    float *gA = c.grad_A, *gD = c.grad_D, *gb = c.grad_delta_bias;
    void *args[] = {&partials, &num_seqs, &channels, &states, &gA, &gD, &gb};
    const uint64_t groups = ((uint64_t)channels * (states + 2) + kSumValues - 1) / kSumValues;
    uint32_t threads = 64;
    while (threads < (uint32_t)kSumThreads && threads / kSumValues < num_seqs) threads *= 2;
    const hipError_t e =
        hipLaunchKernel((const void *)row_sums, dim3(groups < (1u << 20) ? groups : 1u << 20),
                        dim3(threads), args, 0, stream);
    return e == hipSuccess ? RLCA_OK : RLCA_ERR_HIP;
}

}  // extern "C"
