// seq_step.hip -- one step of the causal convolution and of the selective scan
// for each sequence of a batch, the states updated in place.
//
// Both are bound by the states' traffic: each is read and written once, and a
// step's few products cost nothing beside that.  With one sequence the time is
// a launch and one chain of dependent loads.  Measured: convolution 512x8192
// bf16 16 us (4.2 TB/s), scan 512x4096 with 16 states 66 us with the states
// from HBM (4.3 TB/s) and 49 when half of them lie in the last-level cache; one
// sequence of 2048 channels 2.6 and 3.5 us.
#include "seq.hpp"

namespace rlca {
namespace seq {

constexpr int kStepThreads = 256;

// In both kernels blockIdx.x walks a sequence's channels and y the sequences, so
// a slot is the same for a whole workgroup, and a thread takes its channels of
// several sequences: their parameters are read once.

// Sequence n's place in the pool, or -1 for an empty seat or none.
__device__ __forceinline__ int64_t place_of(const int32_t *slots, uint32_t n, uint32_t num_seqs,
                                            int64_t places) {
    if (n >= num_seqs) return -1;
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
    uint32_t num_seqs, channels;
    int32_t silu;
};

// What a thread loads of one sequence.
template <typename E, int W, int VEC>
struct ConvStepLoads {
    int64_t place;
    Steps<VEC, E> state[W - 1], x;
    __device__ __forceinline__ void load(const ConvStepParams &p, uint32_t n, uint32_t d, int left) {
        place = place_of(p.slots, n, p.num_seqs, p.places);
        if (place < 0) return;
        const E *from = static_cast<const E *>(p.state) + (place * p.channels + d) * (W - 1);
        const bool fresh = p.starts != nullptr && p.starts[n] != 0;
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
            state[j].load(from + j * VEC, fresh ? 0 : left * (W - 1) - j * VEC);
        x.load(static_cast<const E *>(p.x) + n * p.x_n + d, left);
    }
};

// A thread takes VEC neighbouring channels: their states are VEC (W-1)
// consecutive values, read and written in VEC-wide pieces.
template <typename E, int W, int VEC>
__global__ __launch_bounds__(kStepThreads) void causal_conv_step(ConvStepParams p) {
    const uint32_t d = (blockIdx.x * blockDim.x + threadIdx.x) * VEC;
    if (d >= p.channels) return;
    // the thread's channels: times the taps, the channels left would pass 32 bits
    const int left = p.channels - d < (uint32_t)VEC ? (int)(p.channels - d) : VEC;
    ConvStepLoads<E, W, VEC> next;
    next.load(p, blockIdx.y, d, left);
    float w[W][VEC], bias[VEC] = {};
#pragma unroll
    for (int j = 0; j < W; ++j)
        load_steps<VEC>(p.weight + (int64_t)d * W + j * VEC, left * W - j * VEC, w[j]);
    if (p.bias != nullptr) load_steps<VEC>(p.bias + d, left, bias);
    for (uint32_t n = blockIdx.y; n < p.num_seqs; n += gridDim.y) {
        const ConvStepLoads<E, W, VEC> now = next;
        if (n + gridDim.y < p.num_seqs) next.load(p, n + gridDim.y, d, left);
        float out[VEC] = {};
        if (now.place >= 0) {
            float old[W - 1][VEC], x[VEC], shifted[W - 1][VEC];
#pragma unroll
            for (int j = 0; j < W - 1; ++j) now.state[j].widen(old[j]);
            now.x.widen(x);
#pragma unroll
            for (int c = 0; c < VEC; ++c) {
                float pre = bias[c];
#pragma unroll
                for (int k = 0; k < W; ++k) {
                    // element k of channel c in runs of W - 1 (state) or W (weight)
                    const int e = c * (W - 1) + k, q = c * W + k;
                    const float tap = k == W - 1 ? x[c] : old[e / VEC][e % VEC];
                    pre = fmaf(w[q / VEC][q % VEC], tap, pre);
                    if (k > 0) shifted[(e - 1) / VEC][(e - 1) % VEC] = tap;
                }
                out[c] = p.silu != 0 ? silu(pre) : pre;
            }
            E *to = static_cast<E *>(p.state) + (now.place * p.channels + d) * (W - 1);
#pragma unroll
            for (int j = 0; j < W - 1; ++j)
                store_steps<VEC>(to + j * VEC, left * (W - 1) - j * VEC, shifted[j]);
        }
        store_steps<VEC>(static_cast<E *>(p.out) + (int64_t)n * p.channels + d, left, out);
    }
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
    uint32_t num_seqs, channels, states;
    uint32_t lane_bits;  // log2 of the lanes of a channel
    int32_t softplus;
    FastDiv by_group;
};

// What a lane loads of one sequence.
template <typename E>
struct StepLoads {
    int64_t place;
    Steps<4, float> h;
    Steps<4, E> b, c;
    E u, raw, z;
    __device__ __forceinline__ void load(const ScanStepParams &p, uint32_t n, uint32_t d,
                                         uint32_t g, int s, int S) {
        place = place_of(p.slots, n, p.num_seqs, p.places);
        if (place < 0) return;
        const bool fresh = p.starts != nullptr && p.starts[n] != 0;
        h.load(p.state + (place * p.channels + d) * S + s, fresh ? 0 : S - s);
        u = static_cast<const E *>(p.u)[n * p.u_n + d];
        raw = static_cast<const E *>(p.delta)[n * p.delta_n + d];
        if (p.z != nullptr) z = static_cast<const E *>(p.z)[n * p.z_n + d];
        b.load(static_cast<const E *>(p.B) + n * p.B_n + g * p.B_g + s, S - s);
        c.load(static_cast<const E *>(p.C) + n * p.C_n + g * p.C_g + s, S - s);
    }
};

// 2^lane_bits lanes share a channel, each owning 4 consecutive states (with at
// most 128 states, up to 32 lanes); y's sum meets in a butterfly over them.  A
// workgroup walks the sequences blockIdx.y, blockIdx.y + gridDim.y, ... and
// loads one while it computes the one before, so the parameters are read once
// and the chain from a slot to its state is hidden.
template <typename E>
__global__ __launch_bounds__(kStepThreads, 8) void selective_step(ScanStepParams p) {
    const uint32_t lanes = 1u << p.lane_bits;
    const uint32_t d = (blockIdx.x * kStepThreads + threadIdx.x) >> p.lane_bits;
    if (d >= p.channels) return;  // a channel's lanes leave together
    const int S = (int)p.states, s = (int)(threadIdx.x & (lanes - 1)) * 4;
    const uint32_t g = p.by_group.div(d);
    StepLoads<E> next;
    next.load(p, blockIdx.y, d, g, s, S);
    float a[4];
    load_steps<4>(p.A + (int64_t)d * S + s, S - s, a);
    const float bias = p.delta_bias == nullptr ? 0.f : p.delta_bias[d];
    const float skip = p.D == nullptr ? 0.f : p.D[d];
    for (uint32_t n = blockIdx.y; n < p.num_seqs; n += gridDim.y) {
        const StepLoads<E> now = next;
        if (n + gridDim.y < p.num_seqs) next.load(p, n + gridDim.y, d, g, s, S);
        float y = 0.f;
        if (now.place >= 0) {
            const float u = (float)now.u;
            float dt = (float)now.raw + bias, h[4], in[4], out[4];
            if (p.softplus != 0) dt = softplus(dt);
            now.h.widen(h);
            now.b.widen(in);
            now.c.widen(out);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float x = dt * a[k] * kLog2e, b = dt * u * in[k];
                // a growth beyond float32's range leaves a state of 0 at 0
                h[k] = x < 100.f ? fmaf(exp2_fast(x), h[k], b) : times_exp2(h[k], x) + b;
                if (s + k < S) y = fmaf(out[k], h[k], y);
            }
            store_steps<4>(p.state + (now.place * p.channels + d) * S + s, S - s, h);
        }
        for (uint32_t m = 1; m < lanes; m <<= 1) y += __shfl_xor(y, (int)m);
        if (s != 0) continue;
        if (now.place >= 0) {
            y = fmaf(skip, (float)now.u, y);
            if (p.z != nullptr) y *= silu((float)now.z);
        }
        static_cast<E *>(p.y)[(int64_t)n * p.channels + d] = (E)y;
    }
}

// ------------------------------------------------------------------- host side
// Workgroups of a launch, as far as there are sequences: what the chip holds at
// once.  The scan's step, 512x4096, 16 states, bf16, states from HBM: 130, 90,
// 67, 66 and 73 us with 512, 1024, 2048, 4096 and a workgroup for each sequence.
constexpr uint32_t kStepBlocks = 2048;

// The convolution's step: eight channels a thread, with a quarter of the
// workgroups, from kWideThreads such threads on; the states' 6 bytes a channel
// then move 16 at a time.  512x8192 bf16: 15.8 us against 17.9 with one channel,
// 512x4096 10.7 against 10.4; 256x4096 fp32 12.3 against 8.8.
constexpr int kWideChannels = 8;
constexpr int64_t kWideThreads = 1 << 18;
constexpr uint32_t kWideBlocks = 512;
constexpr uint32_t kStepGroups = 1u << 15;  // workgroups in y at most

template <typename E, int VEC>
static const void *conv_step_kernel(int width) {
    return width == 2   ? (const void *)causal_conv_step<E, 2, VEC>
           : width == 3 ? (const void *)causal_conv_step<E, 3, VEC>
                        : (const void *)causal_conv_step<E, 4, VEC>;
}

template <typename E>
static const void *conv_step_kernel(int width, int vec) {
    return vec == 1 ? conv_step_kernel<E, 1>(width) : conv_step_kernel<E, kWideChannels>(width);
}

// Workgroups in y: enough to fill the chip, each then walks several sequences.
static uint32_t step_groups(int64_t num_seqs, uint32_t across, uint32_t blocks) {
    const uint32_t most = (blocks + across - 1) / across;
    const uint32_t all = (uint32_t)(num_seqs < kStepGroups ? num_seqs : kStepGroups);
    return all < most ? all : most;
}

static rlca_status check_step(int64_t num_seqs, int64_t channels, int64_t places,
                              const int32_t *slots) {
    if (!sizes_ok(num_seqs, channels, 1) || places < 0 || places > INT32_MAX ||
        (slots == nullptr && places < num_seqs))
        return RLCA_ERR_INVALID_SIZE;
    return RLCA_OK;
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
    p.num_seqs = (uint32_t)N;
    p.channels = (uint32_t)D;
    p.silu = c.silu;
    const int vec = N * ((D + kWideChannels - 1) / kWideChannels) >= kWideThreads ? kWideChannels : 1;
    const uint32_t threads = (uint32_t)((D + vec - 1) / vec);
    const uint32_t size = threads >= (uint32_t)kStepThreads ? kStepThreads : (threads + 63) / 64 * 64;
    const uint32_t across = (threads + size - 1) / size;
    const void *kernel = c.dtype == RLCA_F32    ? conv_step_kernel<float>(c.width, vec)
                         : c.dtype == RLCA_BF16 ? conv_step_kernel<__bf16>(c.width, vec)
                                                : conv_step_kernel<_Float16>(c.width, vec);
    return launch(kernel, dim3(across, step_groups(N, across, vec == 1 ? kStepBlocks : kWideBlocks)),
                  size, 0, p, stream);
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
    if (D * S >= (int64_t)1 << 32) return RLCA_ERR_INVALID_SIZE;  // the launch's threads
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
    p.num_seqs = (uint32_t)N;
    p.channels = (uint32_t)D;
    p.states = (uint32_t)S;
    p.softplus = c.softplus;
    p.by_group = fast_div((uint32_t)(D / G));
    while ((4 << p.lane_bits) < S) ++p.lane_bits;  // at most 32 lanes (128 states)
    const uint64_t threads = (uint64_t)D << p.lane_bits;
    const uint32_t across = (uint32_t)((threads + kStepThreads - 1) / kStepThreads);
    const void *kernel = c.dtype == RLCA_F32    ? (const void *)selective_step<float>
                         : c.dtype == RLCA_BF16 ? (const void *)selective_step<__bf16>
                                                : (const void *)selective_step<_Float16>;
    return launch(kernel, dim3(across, step_groups(N, across, kStepBlocks)), kStepThreads, 0, p, stream);
}

}  // extern "C"
