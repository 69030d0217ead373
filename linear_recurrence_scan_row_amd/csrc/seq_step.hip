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
    uint32_t rows, channels;
    int32_t silu;
    FastDiv by_channels;
};

template <typename E, int W>
__global__ __launch_bounds__(kStepThreads) void causal_conv_step(ConvStepParams p) {
    const uint32_t row = blockIdx.x * kStepThreads + threadIdx.x;
    if (row >= p.rows) return;
    const uint32_t n = p.by_channels.div(row), d = row - n * p.channels;
    const int64_t place = place_of(p.slots, n, p.places);
    E *out = static_cast<E *>(p.out) + row;
    if (place < 0) {
        *out = (E)0.f;
        return;
    }
    E *state = static_cast<E *>(p.state) + (place * p.channels + d) * (W - 1);
    const bool fresh = p.starts != nullptr && p.starts[n] != 0;
    float v[W];
#pragma unroll
    for (int i = 0; i < W - 1; ++i) v[i] = fresh ? 0.f : (float)state[i];
    v[W - 1] = (float)static_cast<const E *>(p.x)[n * p.x_n + d];
    float pre = p.bias == nullptr ? 0.f : p.bias[d];
#pragma unroll
    for (int i = 0; i < W; ++i) pre = fmaf(p.weight[(int64_t)d * W + i], v[i], pre);
#pragma unroll
    for (int i = 0; i < W - 1; ++i) state[i] = (E)v[i + 1];
    *out = (E)(p.silu != 0 ? silu(pre) : pre);
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

// 2^lane_bits lanes share a channel, each owning 4 consecutive states at a
// time; y's sum meets in a butterfly over them.
template <typename E>
__global__ __launch_bounds__(kStepThreads) void selective_step(ScanStepParams p) {
    const uint32_t lanes = 1u << p.lane_bits, lane = threadIdx.x & (lanes - 1);
    const uint32_t rows_per_block = kStepThreads >> p.lane_bits;
    const int S = (int)p.states;
    // whole channels share every branch below
    for (uint64_t row64 = (uint64_t)blockIdx.x * rows_per_block + (threadIdx.x >> p.lane_bits);
         row64 < p.rows; row64 += (uint64_t)gridDim.x * rows_per_block) {
        const uint32_t row = (uint32_t)row64;
        const uint32_t n = p.by_channels.div(row), d = row - n * p.channels;
        const int64_t place = place_of(p.slots, n, p.places);
        E *y = static_cast<E *>(p.y) + row;
        if (place < 0) {
            if (lane == 0) *y = (E)0.f;
            continue;
        }
        const uint32_t g = p.by_group.div(d);
        const bool fresh = p.starts != nullptr && p.starts[n] != 0;
        const float u = (float)static_cast<const E *>(p.u)[n * p.u_n + d];
        float dt = (float)static_cast<const E *>(p.delta)[n * p.delta_n + d];
        if (p.delta_bias != nullptr) dt += p.delta_bias[d];
        if (p.softplus != 0) dt = softplus(dt);
        float *state = p.state + (place * p.channels + d) * S;
        const float *A = p.A + (int64_t)d * S;
        const E *B = static_cast<const E *>(p.B) + n * p.B_n + g * p.B_g;
        const E *C = static_cast<const E *>(p.C) + n * p.C_n + g * p.C_g;
        float sum = 0.f;
        for (int s = (int)lane * 4; s < S; s += (int)lanes * 4) {
            float h[4], a[4], b[4], c[4];
            load_steps<4>(state + s, S - s, h);
            load_steps<4>(A + s, S - s, a);
            load_steps<4>(B + s, S - s, b);
            load_steps<4>(C + s, S - s, c);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float old = fresh ? 0.f : h[k];
                h[k] = fmaf(exp2_fast(dt * a[k] * kLog2e), old, dt * u * b[k]);
                if (s + k < S) sum = fmaf(c[k], h[k], sum);
            }
            store_steps<4>(state + s, S - s, h);
        }
        for (uint32_t m = 1; m < lanes; m <<= 1) sum += __shfl_xor(sum, (int)m);
        if (lane != 0) continue;
        if (p.D != nullptr) sum = fmaf(p.D[d], u, sum);
        if (p.z != nullptr) sum *= silu((float)static_cast<const E *>(p.z)[n * p.z_n + d]);
        *y = (E)sum;
    }
}

// ------------------------------------------------------------------- host side
static rlca_status check_step(int64_t num_seqs, int64_t channels, int64_t places,
                              const int32_t *slots) {
    if (!sizes_ok(num_seqs, channels, 1) || places < 0 || places > INT32_MAX ||
        (slots == nullptr && places < num_seqs))
        return RLCA_ERR_INVALID_SIZE;
    return RLCA_OK;
}

template <typename E>
static const void *conv_step_kernel(int width) {
    return width == 2   ? (const void *)causal_conv_step<E, 2>
           : width == 3 ? (const void *)causal_conv_step<E, 3>
                        : (const void *)causal_conv_step<E, 4>;
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
    p.rows = (uint32_t)(N * D);
    p.channels = (uint32_t)D;
    p.silu = c.silu;
    p.by_channels = fast_div(p.channels);
    const void *kernel = c.dtype == RLCA_F32    ? conv_step_kernel<float>(c.width)
                         : c.dtype == RLCA_BF16 ? conv_step_kernel<__bf16>(c.width)
                                                : conv_step_kernel<_Float16>(c.width);
    return launch(kernel, dim3((p.rows + kStepThreads - 1) / kStepThreads), kStepThreads, 0, p,
                  stream);
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
    const void *kernel = c.dtype == RLCA_F32    ? (const void *)selective_step<float>
                         : c.dtype == RLCA_BF16 ? (const void *)selective_step<__bf16>
                                                : (const void *)selective_step<_Float16>;
    const uint64_t blocks = ((uint64_t)p.rows + rows_per_block - 1) / rows_per_block;
    return launch(kernel, dim3((uint32_t)(blocks < (1u << 22) ? blocks : 1u << 22)), kStepThreads,
                  0, p, stream);
}

}  // extern "C"
