// seq_step.hip -- one step of the causal convolution and of the selective scan
// for each sequence of a batch, the states updated in place.
//
// Both are bound by the states' traffic: each is read and written once, and a
// step's few products cost nothing beside that.  With one sequence the time is
// a launch and one chain of dependent loads.
#include "seq.hpp"

namespace rlca {
namespace seq {

constexpr int kStepThreads = 256;

// Sequence n's place in the pool, or -1 for an empty seat.
__device__ __forceinline__ int64_t place_of(const int32_t *slots, uint32_t n, int64_t places) {
    if (slots == nullptr) return n;
    const int64_t s = slots[n];
    return s >= 0 && s < places ? s : -1;
}

// ------------------------------------------------------------ the convolution
struct ConvStepParams {
    const void *x;
    const float *weight, *bias;
    void *state;
    const int32_t *slots;
    const uint8_t *starts;
    void *out;
    int64_t x_n, places;
    uint32_t num_seqs, channels, blocks;  // blocks: of VEC channels, in a sequence
    int32_t silu;
    FastDiv by_blocks;
};

// A thread takes VEC neighbouring channels: their states are VEC (W-1)
// consecutive values, read and written in VEC-wide pieces.
template <typename E, int W, int VEC>
__global__ __launch_bounds__(kStepThreads) void causal_conv_step(ConvStepParams p) {
    const uint32_t i = blockIdx.x * kStepThreads + threadIdx.x;
    if (i >= p.num_seqs * p.blocks) return;
    const uint32_t n = p.by_blocks.div(i), d = (i - n * p.blocks) * VEC;
    const int left = (int)(p.channels - d);  // VEC or more: whole blocks
    const int64_t place = place_of(p.slots, n, p.places);
    E *out = static_cast<E *>(p.out) + (int64_t)n * p.channels + d;
    float o[VEC] = {};
    if (place >= 0) {
        E *state = static_cast<E *>(p.state) + (place * p.channels + d) * (W - 1);
        float v[W - 1][VEC], x[VEC], w[W][VEC], bias[VEC] = {};
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
            load_steps<VEC>(state + j * VEC, left * (W - 1) - j * VEC, v[j]);
        load_steps<VEC>(static_cast<const E *>(p.x) + n * p.x_n + d, left, x);
#pragma unroll
        for (int j = 0; j < W; ++j)
            load_steps<VEC>(p.weight + (int64_t)d * W + j * VEC, left * W - j * VEC, w[j]);
        if (p.bias != nullptr) load_steps<VEC>(p.bias + d, left, bias);
        if (p.starts != nullptr && p.starts[n] != 0)
#pragma unroll
            for (int j = 0; j < W - 1; ++j)
#pragma unroll
                for (int c = 0; c < VEC; ++c) v[j][c] = 0.f;
        float next[W - 1][VEC];
#pragma unroll
        for (int c = 0; c < VEC; ++c) {
            float pre = bias[c];
#pragma unroll
            for (int k = 0; k < W; ++k) {
                // element k of channel c in a run of rows of W - 1 (state) or W (weight)
                const int e = c * (W - 1) + k, q = c * W + k;
                const float tap = k == W - 1 ? x[c] : v[e / VEC][e % VEC];
                pre = fmaf(w[q / VEC][q % VEC], tap, pre);
                if (k > 0) next[(e - 1) / VEC][(e - 1) % VEC] = tap;
            }
            o[c] = p.silu != 0 ? silu(pre) : pre;
        }
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
            store_steps<VEC>(state + j * VEC, left * (W - 1) - j * VEC, next[j]);
    }
    store_steps<VEC>(out, left, o);
}

// ------------------------------------------------------------------- the scan
struct ScanStepParams {
    const void *u, *delta, *B, *C, *z;
    const float *A, *D, *delta_bias;
    float *state;
    const int32_t *slots;
    const uint8_t *starts;
    void *y;
    int64_t u_n, delta_n, z_n, B_n, B_g, C_n, C_g, places;
    uint32_t rows, channels, states;
    uint32_t lane_bits;  // log2 of the lanes of a channel
    int32_t softplus;
    FastDiv by_channels, by_group;
};

// One channel of a lane: where its values are, and those that every lane of
// the channel needs.
template <typename E>
struct StepRow {
    bool in, live;  // a row of the call; one with a place in the pool
    uint32_t row, d;
    float u, raw, z;
    float *state;
    const E *B, *C;
    bool fresh;
    __device__ __forceinline__ void load(const ScanStepParams &p, uint64_t row64) {
        in = row64 < p.rows;
        live = false;
        if (!in) return;
        row = (uint32_t)row64;
        const uint32_t n = p.by_channels.div(row);
        d = row - n * p.channels;
        const uint32_t g = p.by_group.div(d);
        const int64_t place = place_of(p.slots, n, p.places);
        live = place >= 0;
        if (!live) return;
        fresh = p.starts != nullptr && p.starts[n] != 0;
        state = p.state + (place * p.channels + d) * (int)p.states;
        B = static_cast<const E *>(p.B) + n * p.B_n + g * p.B_g;
        C = static_cast<const E *>(p.C) + n * p.C_n + g * p.C_g;
        u = (float)static_cast<const E *>(p.u)[n * p.u_n + d];
        raw = (float)static_cast<const E *>(p.delta)[n * p.delta_n + d];
        z = p.z == nullptr ? 0.f : (float)static_cast<const E *>(p.z)[n * p.z_n + d];
    }
};

// 2^lane_bits lanes share a channel, each owning 4 consecutive states (with at
// most 128 states, up to 32 lanes); y's sum meets in a butterfly over them.
// ROWS channels of a lane are loaded together, which keeps enough bytes in
// flight.  Lanes of a channel share every branch.
template <typename E, int ROWS>
__global__ __launch_bounds__(kStepThreads) void selective_step(ScanStepParams p) {
    const uint32_t lanes = 1u << p.lane_bits;
    const uint32_t rows_per_block = kStepThreads >> p.lane_bits;
    const int S = (int)p.states, s = (int)(threadIdx.x & (lanes - 1)) * 4;
    for (uint64_t row0 = (uint64_t)blockIdx.x * rows_per_block * ROWS + (threadIdx.x >> p.lane_bits);
         row0 < p.rows; row0 += (uint64_t)gridDim.x * rows_per_block * ROWS) {
        StepRow<E> r[ROWS];
        float h[ROWS][4];
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            r[i].load(p, row0 + i * rows_per_block);
            if (r[i].live) load_steps<4>(r[i].state + s, S - s, h[i]);
        }
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            if (!r[i].in) continue;
            float y = 0.f;
            if (r[i].live) {
                float a[4], b[4], c[4], dt = r[i].raw;
                load_steps<4>(p.A + (int64_t)r[i].d * S + s, S - s, a);
                load_steps<4>(r[i].B + s, S - s, b);
                load_steps<4>(r[i].C + s, S - s, c);
                if (p.delta_bias != nullptr) dt += p.delta_bias[r[i].d];
                if (p.softplus != 0) dt = softplus(dt);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float old = r[i].fresh ? 0.f : h[i][k];
                    h[i][k] = fmaf(exp2_fast(dt * a[k] * kLog2e), old, dt * r[i].u * b[k]);
                    if (s + k < S) y = fmaf(c[k], h[i][k], y);
                }
                store_steps<4>(r[i].state + s, S - s, h[i]);
            }
            for (uint32_t m = 1; m < lanes; m <<= 1) y += __shfl_xor(y, (int)m);
            if (s != 0) continue;
            if (r[i].live) {
                if (p.D != nullptr) y = fmaf(p.D[r[i].d], r[i].u, y);
                if (p.z != nullptr) y *= silu(r[i].z);
            }
            static_cast<E *>(p.y)[r[i].row] = (E)y;
        }
    }
}

// ------------------------------------------------------------------- host side
// Channels of a thread of the convolution's step, where that leaves
// kWideThreads threads or more (one wave for each SIMD): the states' 6 bytes a
// channel then move 16 at a time (512x8192 bf16: 21 us against 33; 1x2048 fp32
// 3.7 against 3.0).
constexpr int kWideChannels = 8;
constexpr int64_t kWideThreads = 1 << 16;

// Threads of the scan's step from which a lane takes two channels (512x4096, 16
// states, bf16: 70 us against 73 with one; 1x2048 3.7 against 4.9).
constexpr uint64_t kTwoRowsThreads = 1 << 20;

template <typename E>
static const void *step_kernel(int rows) {
    return rows == 2 ? (const void *)selective_step<E, 2> : (const void *)selective_step<E, 1>;
}

static rlca_status check_step(int64_t num_seqs, int64_t channels, int64_t places,
                              const int32_t *slots) {
    if (!sizes_ok(num_seqs, channels, 1) || places < 0 || places > INT32_MAX ||
        (slots == nullptr && places < num_seqs))
        return RLCA_ERR_INVALID_SIZE;
    return RLCA_OK;
}

template <typename E, int VEC>
static const void *conv_step_kernel(int width) {
    return width == 2   ? (const void *)causal_conv_step<E, 2, VEC>
           : width == 3 ? (const void *)causal_conv_step<E, 3, VEC>
                        : (const void *)causal_conv_step<E, 4, VEC>;
}

template <typename E>
static const void *conv_step_kernel(int width, bool wide) {
    return wide ? conv_step_kernel<E, kWideChannels>(width) : conv_step_kernel<E, 1>(width);
}

}  // namespace seq
}  // namespace rlca

using namespace rlca::seq;

extern "C" {

rlca_status rlca_causal_conv_step(const rlca_conv_step_call *call, hipStream_t stream) {
    if (call == nullptr) return RLCA_ERR_NULL_POINTER;
    const rlca_conv_step_call &c = *call;
    const int64_t N = c.num_seqs, D = c.channels, W = c.width;
    rlca_status st = check_step(N, D, c.places, c.slots);
    if (st != RLCA_OK) return st;
    const size_t e = element_bytes(c.dtype);
    if (e == 0 || W < 2 || W > 4) return RLCA_ERR_INVALID_VALUE;
    Arrays a;
    a.in(c.x, e, true, {{N, c.x_stride_seq}, {D, 1}});
    a.in(c.weight, 4, true, {{N == 0 ? 0 : D, W}, {W, 1}});
    a.in(c.bias, 4, false, {{N == 0 ? 0 : D, 1}});
    a.in(c.slots, 4, false, {{N, 1}});
    a.in(c.starts, 1, false, {{N, 1}});
    a.out(c.state, e, N != 0, {{c.places, D * (W - 1)}, {D * (W - 1), 1}});
    a.out(c.out, e, true, {{N, D}, {D, 1}});
    st = a.status();
    if (st != RLCA_OK || N * D == 0) return st;
    ConvStepParams p = {};
    p.x = c.x;
    p.weight = c.weight;
    p.bias = c.bias;
    p.state = c.state;
    p.slots = c.slots;
    p.starts = c.starts;
    p.out = c.out;
    p.x_n = c.x_stride_seq;
    p.places = c.places;
    const bool wide = N * ((D + kWideChannels - 1) / kWideChannels) >= kWideThreads;
    const int64_t vec = wide ? kWideChannels : 1;
    p.num_seqs = (uint32_t)N;
    p.channels = (uint32_t)D;
    p.blocks = (uint32_t)((D + vec - 1) / vec);
    p.silu = c.silu;
    p.by_blocks = fast_div(p.blocks);
    const void *kernel = c.dtype == RLCA_F32    ? conv_step_kernel<float>(c.width, wide)
                         : c.dtype == RLCA_BF16 ? conv_step_kernel<__bf16>(c.width, wide)
                                                : conv_step_kernel<_Float16>(c.width, wide);
    return launch(kernel, dim3((p.num_seqs * p.blocks + kStepThreads - 1) / kStepThreads),
                  kStepThreads, 0, p, stream);
}

rlca_status rlca_selective_step(const rlca_scan_step_call *call, hipStream_t stream) {
    if (call == nullptr) return RLCA_ERR_NULL_POINTER;
    const rlca_scan_step_call &c = *call;
    const int64_t N = c.num_seqs, D = c.channels, S = c.states, G = c.groups;
    rlca_status st = check_step(N, D, c.places, c.slots);
    if (st != RLCA_OK) return st;
    const size_t e = element_bytes(c.dtype);
    if (e == 0 || S < 1 || S > RLCA_MAX_STATES || G < 1 || D % G != 0)
        return RLCA_ERR_INVALID_VALUE;
    const int64_t params = N == 0 ? 0 : D;
    Arrays a;
    a.in(c.u, e, true, {{N, c.u_stride_seq}, {D, 1}});
    a.in(c.delta, e, true, {{N, c.delta_stride_seq}, {D, 1}});
    a.in(c.z, e, false, {{N, c.z_stride_seq}, {D, 1}});
    a.in(c.A, 4, true, {{params, S}, {S, 1}});
    a.in(c.B, e, D != 0, {{N, c.B_stride_seq}, {G, c.B_stride_group}, {S, 1}});
    a.in(c.C, e, D != 0, {{N, c.C_stride_seq}, {G, c.C_stride_group}, {S, 1}});
    a.in(c.D, 4, false, {{params, 1}});
    a.in(c.delta_bias, 4, false, {{params, 1}});
    a.in(c.slots, 4, false, {{N, 1}});
    a.in(c.starts, 1, false, {{N, 1}});
    a.out(c.state, 4, N != 0, {{c.places, D * S}, {D * S, 1}});
    a.out(c.y, e, true, {{N, D}, {D, 1}});
    st = a.status();
    if (st != RLCA_OK || N * D == 0) return st;
    ScanStepParams p = {};
    p.u = c.u;
    p.delta = c.delta;
    p.B = c.B;
    p.C = c.C;
    p.z = c.z;
    p.A = c.A;
    p.D = c.D;
    p.delta_bias = c.delta_bias;
    p.state = c.state;
    p.slots = c.slots;
    p.starts = c.starts;
    p.y = c.y;
    p.u_n = c.u_stride_seq;
    p.delta_n = c.delta_stride_seq;
    p.z_n = c.z_stride_seq;
    p.B_n = c.B_stride_seq;
    p.B_g = c.B_stride_group;
    p.C_n = c.C_stride_seq;
    p.C_g = c.C_stride_group;
    p.places = c.places;
    p.rows = (uint32_t)(N * D);
    p.channels = (uint32_t)D;
    p.states = (uint32_t)S;
    p.softplus = c.softplus;
    p.by_channels = fast_div(p.channels);
    p.by_group = fast_div((uint32_t)(D / G));
    while ((4 << p.lane_bits) < S) ++p.lane_bits;  // at most 32 lanes (128 states)
    const uint32_t rows_per_block = kStepThreads >> p.lane_bits;
    const int rows_per_lane = (uint64_t)p.rows << p.lane_bits >= kTwoRowsThreads ? 2 : 1;
    const void *kernel = c.dtype == RLCA_F32    ? step_kernel<float>(rows_per_lane)
                         : c.dtype == RLCA_BF16 ? step_kernel<__bf16>(rows_per_lane)
                                                : step_kernel<_Float16>(rows_per_lane);
    const uint64_t blocks =
        ((uint64_t)p.rows + rows_per_block * rows_per_lane - 1) / (rows_per_block * rows_per_lane);
    return launch(kernel, dim3((uint32_t)(blocks < (1u << 22) ? blocks : 1u << 22)), kStepThreads,
                  0, p, stream);
}

}  // extern "C"
