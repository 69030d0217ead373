// seq_conv.hip -- the short causal convolution over rows of T steps, forward
// and backward:  pre_t = bias + sum_j weight[W-1-j] x_{t-j},  out = silu(pre).
//
// Bound by memory: W products and one exponential per step against two
// (forward) or three (backward) arrays of steps moved once.  A lane owns K = 8
// consecutive steps: their inputs are one or two 16-byte loads, and the W-1
// inputs before them (and, backward, the steps after them, whose pre is formed
// again here) are loads of lines that the neighbouring lanes read as well, so
// lanes need nothing from each other and HBM delivers each line once.
#include "seq.hpp"

namespace rlca {
namespace seq {

constexpr int kConvThreads = 256;
constexpr int kConvK = 8;
constexpr int kBack = 4;   // steps loaded before the block: W - 1 <= 3 are used
constexpr int kAhead = 4;  // backward: steps loaded after it
// at most so many workgroups in each grid dimension; they walk further ones
constexpr uint32_t kConvMaxRowBlocks = 1u << 22, kConvMaxTiles = 1u << 15;

struct ConvParams {
    const void *x, *grad_out;
    const float *weight, *bias;
    const void *state, *grad_final;
    const uint8_t *flags;
    const int32_t *lengths;
    void *out, *final_state;
    void *grad_x, *grad_state;
    float *partials;  // [channels][num_seqs * tiles][W + 1]
    int64_t x_n, x_d, g_n, g_d;
    uint32_t rows, channels;
    int32_t T;
    uint32_t lane_bits;  // log2 of the lanes of a row
    uint32_t row_blocks, tiles;
    int32_t silu, after_done;
    FastDiv by_channels;
};

// Where a lane's block lies, and what its row's end and episode starts say of
// it.
struct ConvLane {
    uint32_t row, n, d;
    int t0, end;
};

__device__ __forceinline__ ConvLane conv_lane(const ConvParams &p, uint32_t row_block,
                                              uint32_t tile) {
    const uint32_t rows_per_block = kConvThreads >> p.lane_bits;
    ConvLane l;
    l.row = row_block * rows_per_block + (threadIdx.x >> p.lane_bits);
    const uint32_t block = (tile << p.lane_bits) + (threadIdx.x & ((1u << p.lane_bits) - 1));
    l.n = p.by_channels.div(l.row);
    l.d = l.row - l.n * p.channels;
    l.t0 = (int)(block * kConvK);
    l.end = 0;
    if (l.row < p.rows) l.end = row_end(p.lengths, l.n, p.T);
    return l;
}

// Which taps stay within their step's episode.  `starts` bit i: an episode
// starts at step t0 - 2 + i.  Tap j of step k reads across a start if one lies
// in steps k-j+1 .. k; within[j - 1] has bit k + 2 set where none does.
template <int W>
struct Episodes {
    uint32_t within[W - 1];
    __device__ __forceinline__ explicit Episodes(uint32_t starts) {
        uint32_t across = starts;
#pragma unroll
        for (int j = 1; j < W; ++j) {
            within[j - 1] = ~across;
            across |= starts << j;
        }
    }
    // x where the tap stays within, else 0 (whatever x is)
    __device__ __forceinline__ float keep(float x, int k, int j) const {
        const int mask = (int)(within[j - 1] << (29 - k)) >> 31;
        return from_bits<float>(as_bits(x) & mask);
    }
};

// A tap's input: the value j steps before step k, or 0 across a start.
template <int W, bool FLAGS, int N>
__device__ __forceinline__ float tap(const float (&x)[N], const Episodes<W> &e, int k, int j) {
    const float v = x[kBack + k - j];
    if (!FLAGS || j == 0) return v;
    return e.keep(v, k, j);
}

// The state's input at time -1-q (q = 0 the newest), 0 without a state.
template <int W, typename E>
__device__ __forceinline__ float state_at(const void *state, uint32_t row, int q) {
    return state == nullptr ? 0.f
                            : (float)static_cast<const E *>(state)[(int64_t)row * (W - 1) + W - 2 - q];
}

// Whether the input at time p is still seen by the step after the row's last:
// no episode starts after p up to and including that step.
__device__ __forceinline__ bool reaches_end(const uint8_t *flags, int p, int end, int T,
                                            int after_done) {
    if (after_done != 0 && end > 0 && flags[end - 1] != 0) return false;
    for (int t = p + 1 > 0 ? p + 1 : 0; t < end; ++t)
        if (is_start(flags, t, T, after_done)) return false;
    return true;
}

template <typename E, int W, bool FLAGS>
__global__ __launch_bounds__(kConvThreads) void causal_conv(ConvParams p) {
    for (uint32_t rb = blockIdx.x; rb < p.row_blocks; rb += gridDim.x)
        for (uint32_t tile = blockIdx.y; tile < p.tiles; tile += gridDim.y) {
            const ConvLane l = conv_lane(p, rb, tile);
            if (l.row >= p.rows) continue;
            const E *x = static_cast<const E *>(p.x) + l.n * p.x_n + l.d * p.x_d;
            const uint8_t *flags = FLAGS ? p.flags + (int64_t)l.n * p.T : nullptr;
            if (l.t0 < p.T) {
                float v[kBack + kConvK], o[kConvK] = {};
                const int n = l.end - l.t0;
                if (n > 0) {
                    float back[kBack], cur[kConvK];
                    load_steps<kConvK>(x + l.t0, n, cur);
                    load_steps_before<kBack>(x + l.t0, l.t0, back);
                    if (l.t0 == 0)
#pragma unroll
                        for (int q = 0; q < W - 1; ++q)
                            back[kBack - 1 - q] = state_at<W, E>(p.state, l.row, q);
                    uint32_t starts = 0;
                    if constexpr (FLAGS)
                        starts = start_bits<8>(flags, l.t0 - 2, p.T, p.after_done) |
                                 start_bits<2>(flags, l.t0 + 6, p.T, p.after_done) << 8;
                    const Episodes<W> episodes(starts);
#pragma unroll
                    for (int k = 0; k < kBack; ++k) v[k] = back[k];
#pragma unroll
                    for (int k = 0; k < kConvK; ++k) v[kBack + k] = cur[k];
                    float w[W];
#pragma unroll
                    for (int j = 0; j < W; ++j) w[j] = p.weight[(int64_t)l.d * W + j];
                    const float bias = p.bias == nullptr ? 0.f : p.bias[l.d];
#pragma unroll
                    for (int k = 0; k < kConvK; ++k) {
                        float pre = bias;
#pragma unroll
                        for (int j = 0; j < W; ++j)
                            pre = fmaf(w[W - 1 - j], tap<W, FLAGS>(v, episodes, k, j), pre);
                        pre = p.silu != 0 ? silu(pre) : pre;
                        o[k] = k < n ? pre : 0.f;
                    }
                }
                store_steps<kConvK>(static_cast<E *>(p.out) + (int64_t)l.row * p.T + l.t0,
                                    p.T - l.t0, o);
            }
            if (p.final_state != nullptr && l.t0 == 0) {
                E *f = static_cast<E *>(p.final_state) + (int64_t)l.row * (W - 1);
                for (int i = 0; i < W - 1; ++i) {
                    const int at = l.end - (W - 1) + i;
                    float y = at >= 0 ? (float)x[at] : state_at<W, E>(p.state, l.row, -1 - at);
                    if (FLAGS && !reaches_end(flags, at, l.end, p.T, p.after_done)) y = 0.f;
                    f[i] = (E)y;
                }
            }
        }
}

// Backward:  dpre_t = grad_out_t silu'(pre_t),
//   grad_x_t = sum_j weight[W-1-j] dpre_{t+j}   (taps within t's episode),
//   grad_weight[k] = sum dpre_t x_{t-(W-1)+k},  grad_bias = sum dpre_t.
// A lane forms pre for its 8 steps and the W-1 after them.  Its sums for the
// weights meet the other lanes' of its row (at most one wave) and are written
// as one partial per row and tile; conv_weight_sums adds those in order.
template <typename E, int W, bool FLAGS>
__global__ __launch_bounds__(kConvThreads) void causal_conv_backward(ConvParams p) {
    constexpr int kSteps = kConvK + W - 1;  // pre of these
    for (uint32_t rb = blockIdx.x; rb < p.row_blocks; rb += gridDim.x)
        for (uint32_t tile = blockIdx.y; tile < p.tiles; tile += gridDim.y) {
            const ConvLane l = conv_lane(p, rb, tile);
            float dw[W] = {}, db = 0.f;
            if (l.row < p.rows && l.t0 < p.T) {
                const E *x = static_cast<const E *>(p.x) + l.n * p.x_n + l.d * p.x_d;
                const E *g = static_cast<const E *>(p.grad_out) + l.n * p.g_n + l.d * p.g_d;
                const uint8_t *flags = FLAGS ? p.flags + (int64_t)l.n * p.T : nullptr;
                const int n = l.end - l.t0;
                float dx[kConvK] = {};
                if (n > 0) {
                    float w[W];
#pragma unroll
                    for (int j = 0; j < W; ++j) w[j] = p.weight[(int64_t)l.d * W + j];
                    const float bias = p.bias == nullptr ? 0.f : p.bias[l.d];
                    float v[kBack + kConvK + kAhead], go[kConvK + kAhead];
                    {
                        float back[kBack], cur[kConvK], ahead[kAhead];
                        float gcur[kConvK], gahead[kAhead];
                        load_steps<kConvK>(x + l.t0, n, cur);
                        load_steps<kConvK>(g + l.t0, n, gcur);
                        load_steps_before<kBack>(x + l.t0, l.t0, back);
                        load_steps<kAhead>(x + l.t0 + kConvK, n - kConvK, ahead);
                        load_steps<kAhead>(g + l.t0 + kConvK, n - kConvK, gahead);
                        if (l.t0 == 0)
#pragma unroll
                            for (int q = 0; q < W - 1; ++q)
                                back[kBack - 1 - q] = state_at<W, E>(p.state, l.row, q);
#pragma unroll
                        for (int k = 0; k < kBack; ++k) v[k] = back[k];
#pragma unroll
                        for (int k = 0; k < kConvK; ++k) v[kBack + k] = cur[k], go[k] = gcur[k];
#pragma unroll
                        for (int k = 0; k < kAhead; ++k)
                            v[kBack + kConvK + k] = ahead[k], go[kConvK + k] = gahead[k];
                    }
                    uint32_t starts = 0;  // bit i: step t0 - 2 + i
                    if constexpr (FLAGS)
                        starts = start_bits<8>(flags, l.t0 - 2, p.T, p.after_done) |
                                 start_bits<5>(flags, l.t0 + 6, p.T, p.after_done) << 8;
                    const Episodes<W> episodes(starts);
                    float dpre[kSteps];
#pragma unroll
                    for (int k = 0; k < kSteps; ++k) {
                        float pre = bias;
#pragma unroll
                        for (int j = 0; j < W; ++j)
                            pre = fmaf(w[W - 1 - j], tap<W, FLAGS>(v, episodes, k, j), pre);
                        const float slope = p.silu != 0 ? silu_slope(pre, sigmoid(pre)) : 1.f;
                        dpre[k] = k < n ? go[k] * slope : 0.f;
                    }
#pragma unroll
                    for (int k = 0; k < kConvK; ++k) {
                        float s = 0.f;
#pragma unroll
                        for (int j = 0; j < W; ++j) {
                            // step k is tap j of step k + j
                            const float g = FLAGS && j > 0 ? episodes.keep(dpre[k + j], k + j, j)
                                                           : dpre[k + j];
                            s = fmaf(w[W - 1 - j], g, s);
                        }
                        dx[k] = k < n ? s : 0.f;
                        db += dpre[k];
#pragma unroll
                        for (int j = 0; j < W; ++j)
                            dw[W - 1 - j] = fmaf(dpre[k], tap<W, FLAGS>(v, episodes, k, j),
                                                 dw[W - 1 - j]);
                    }
                    if (p.grad_state != nullptr && l.t0 == 0) {
                        E *gs = static_cast<E *>(p.grad_state) + (int64_t)l.row * (W - 1);
#pragma unroll
                        for (int q = 0; q < W - 1; ++q) {  // the input at time q - (W-1)
                            float s = 0.f;
#pragma unroll
                            for (int t = 0; t <= q; ++t) {  // tap t + (W-1) - q of step t
                                const bool cut = FLAGS && (starts & (((1u << (t + 1)) - 1) << 2)) != 0;
                                s = fmaf(w[q - t], cut ? 0.f : dpre[t], s);
                            }
                            const int i = q - l.end;  // its place in the final state
                            if (p.grad_final != nullptr && i >= 0 &&
                                !(FLAGS && !reaches_end(flags, q - (W - 1), l.end, p.T,
                                                        p.after_done)))
                                s += (float)static_cast<const E *>(
                                    p.grad_final)[(int64_t)l.row * (W - 1) + i];
                            gs[q] = (E)s;
                        }
                    }
                    if (p.grad_final != nullptr && n - kConvK < W - 1) {
                        const E *gf =
                            static_cast<const E *>(p.grad_final) + (int64_t)l.row * (W - 1);
#pragma unroll
                        for (int k = 0; k < kConvK; ++k) {
                            const int i = l.t0 + k - (l.end - (W - 1));
                            if (i < 0 || i >= W - 1) continue;
                            if (FLAGS &&
                                !reaches_end(flags, l.t0 + k, l.end, p.T, p.after_done))
                                continue;
                            dx[k] += (float)gf[i];
                        }
                    }
                }
                store_steps<kConvK>(static_cast<E *>(p.grad_x) + (int64_t)l.row * p.T + l.t0,
                                    p.T - l.t0, dx);
            }
            if (l.row < p.rows && l.t0 == 0 && l.end == 0 && p.grad_state != nullptr)
                for (int q = 0; q < W - 1; ++q) {  // an empty row hands its state on
                    const int64_t at = (int64_t)l.row * (W - 1) + q;
                    static_cast<E *>(p.grad_state)[at] =
                        p.grad_final == nullptr ? (E)0.f : static_cast<const E *>(p.grad_final)[at];
                }
            // the row's lanes, in a fixed tree
            for (uint32_t m = 1; m < (1u << p.lane_bits); m <<= 1) {
#pragma unroll
                for (int j = 0; j < W; ++j) dw[j] += __shfl_xor(dw[j], (int)m);
                db += __shfl_xor(db, (int)m);
            }
            if (l.row < p.rows && (threadIdx.x & ((1u << p.lane_bits) - 1)) == 0) {
                const uint64_t per_channel = (uint64_t)(p.rows / p.channels) * p.tiles;
                float *o = p.partials +
                           (l.d * per_channel + (uint64_t)l.n * p.tiles + tile) * (W + 1);
#pragma unroll
                for (int j = 0; j < W; ++j) o[j] = dw[j];
                o[W] = db;
            }
        }
}

// A workgroup per channel adds its partials in fp64, its waves' sums in order.
constexpr int kSumThreads = 1024;

template <int W>
__global__ __launch_bounds__(kSumThreads) void conv_weight_sums(const float *partials,
                                                                uint64_t per_channel,
                                                                uint32_t channels,
                                                                float *grad_weight,
                                                                float *grad_bias) {
    __shared__ double sums[kSumThreads / kWave][W + 1];
    for (uint32_t d = blockIdx.x; d < channels; d += gridDim.x) {
        const float *in = partials + d * per_channel * (W + 1);
        double s[W + 1] = {};
#pragma unroll 4
        for (uint64_t i = threadIdx.x; i < per_channel; i += blockDim.x)
#pragma unroll
            for (int j = 0; j <= W; ++j) s[j] += (double)in[i * (W + 1) + j];
#pragma unroll
        for (int m = 1; m < kWave; m <<= 1)
#pragma unroll
            for (int j = 0; j <= W; ++j) s[j] += __shfl_xor(s[j], m);
        if (threadIdx.x % kWave == 0)
#pragma unroll
            for (int j = 0; j <= W; ++j) sums[threadIdx.x / kWave][j] = s[j];
        __syncthreads();
        const uint32_t j = threadIdx.x;
        if (j <= W) {
            double total = 0.0;
            for (uint32_t w = 0; w < blockDim.x / kWave; ++w) total += sums[w][j];
            if (j < W)
                grad_weight[(int64_t)d * W + j] = (float)total;
            else if (grad_bias != nullptr)
                grad_bias[d] = (float)total;
        }
        __syncthreads();
    }
}

// ------------------------------------------------------------------- host side
// Lanes of a row, a power of two up to `most`: the most whose idle lanes past
// the row's end stay below a quarter, so that a row's loads are long runs.
static uint32_t lane_bits_for(int64_t T, uint32_t most) {
    const int64_t blocks = T <= 0 ? 1 : (T + kConvK - 1) / kConvK;
    uint32_t bits = 0;
    while ((1ll << bits) < blocks && bits < most) ++bits;
    for (uint32_t b = bits; b >= 3; --b) {
        const int64_t lanes = (blocks + (1ll << b) - 1) >> b << b;
        if (4 * lanes <= 5 * blocks) return b;
    }
    return bits;
}

static uint32_t tiles_of(int64_t T, uint32_t bits) {
    const int64_t blocks = T <= 0 ? 1 : (T + kConvK - 1) / kConvK;
    return (uint32_t)((blocks + (1ll << bits) - 1) >> bits);
}

static ConvParams conv_params(const rlca_conv_call &c, uint32_t most_bits) {
    ConvParams p = {};
    p.x = c.x;
    p.grad_out = c.grad_out;
    p.weight = c.weight;
    p.bias = c.bias;
    p.state = c.state;
    p.grad_final = c.grad_final_state;
    p.flags = c.flags;
    p.lengths = c.lengths;
    p.out = c.out;
    p.final_state = c.final_state;
    p.grad_x = c.grad_x;
    p.grad_state = c.grad_state;
    p.x_n = c.x_stride_seq;
    p.x_d = c.x_stride_channel;
    p.g_n = c.grad_stride_seq;
    p.g_d = c.grad_stride_channel;
    p.rows = (uint32_t)(c.num_seqs * c.channels);
    p.channels = (uint32_t)c.channels;
    p.T = (int32_t)c.T;
    p.lane_bits = lane_bits_for(c.T, most_bits);
    const uint32_t rows_per_block = kConvThreads >> p.lane_bits;
    p.row_blocks = (uint32_t)(((uint64_t)p.rows + rows_per_block - 1) / rows_per_block);
    p.tiles = tiles_of(c.T, p.lane_bits);
    p.silu = c.silu;
    p.after_done = c.convention == RLCA_RESET_AFTER_DONE;
    p.by_channels = fast_div(p.channels);
    return p;
}

static dim3 conv_grid(const ConvParams &p) {
    return dim3(p.row_blocks < kConvMaxRowBlocks ? p.row_blocks : kConvMaxRowBlocks,
                p.tiles < kConvMaxTiles ? p.tiles : kConvMaxTiles);
}

static rlca_status check_conv(const rlca_conv_call &c, bool backward, Arrays *a) {
    if (!sizes_ok(c.num_seqs, c.channels, c.T)) return RLCA_ERR_INVALID_SIZE;
    const size_t e = element_bytes(c.dtype);
    if (e == 0 || c.width < 2 || c.width > 4 ||
        (c.convention != RLCA_RESET_ON_START && c.convention != RLCA_RESET_AFTER_DONE))
        return RLCA_ERR_INVALID_VALUE;
    const int64_t N = c.num_seqs, D = c.channels, T = c.T, W = c.width;
    const Dim dense[] = {{N, D * T}, {D, T}, {T, 1}};
    const Dim state[] = {{N * D, W - 1}, {W - 1, 1}};
    a->in(c.x, e, true, {{N, c.x_stride_seq}, {D, c.x_stride_channel}, {T, 1}});
    a->in(c.weight, 4, true, {{N == 0 ? 0 : D, W}, {W, 1}});
    a->in(c.bias, 4, false, {{N == 0 ? 0 : D, 1}});
    a->in(c.state, e, false, state);
    a->in(c.flags, 1, false, {{N * T, 1}});
    a->in(c.lengths, 4, false, {{N, 1}});
    if (!backward) {
        a->out(c.out, e, true, dense);
        a->out(c.final_state, e, false, state);
    } else {
        a->in(c.grad_out, e, true,
              {{N, c.grad_stride_seq}, {D, c.grad_stride_channel}, {T, 1}});
        a->in(c.grad_final_state, e, false, state);
        a->out(c.grad_x, e, true, dense);
        a->out(c.grad_weight, 4, true, {{D, W}, {W, 1}});
        a->out(c.grad_bias, 4, false, {{D, 1}});
        a->out(c.grad_state, e, false, state);
    }
    return RLCA_OK;
}

template <typename E, int W>
static const void *conv_kernel(bool flags, bool backward) {
    if (backward)
        return flags ? (const void *)causal_conv_backward<E, W, true>
                     : (const void *)causal_conv_backward<E, W, false>;
    return flags ? (const void *)causal_conv<E, W, true> : (const void *)causal_conv<E, W, false>;
}

template <typename E>
static const void *conv_kernel(int width, bool flags, bool backward) {
    return width == 2   ? conv_kernel<E, 2>(flags, backward)
           : width == 3 ? conv_kernel<E, 3>(flags, backward)
                        : conv_kernel<E, 4>(flags, backward);
}

static const void *conv_kernel(const rlca_conv_call &c, bool backward) {
    const bool flags = c.flags != nullptr;
    return c.dtype == RLCA_F32    ? conv_kernel<float>(c.width, flags, backward)
           : c.dtype == RLCA_BF16 ? conv_kernel<__bf16>(c.width, flags, backward)
                                  : conv_kernel<_Float16>(c.width, flags, backward);
}

constexpr uint32_t kForwardLaneBits = 8, kBackwardLaneBits = 6;

}  // namespace seq
}  // namespace rlca

using namespace rlca::seq;

extern "C" {

rlca_status rlca_causal_conv(const rlca_conv_call *call, hipStream_t stream) {
    if (call == nullptr) return RLCA_ERR_NULL_POINTER;
    Arrays a;
    rlca_status st = check_conv(*call, false, &a);
    if (st == RLCA_OK) st = a.status();
    if (st != RLCA_OK) return st;
    if (call->num_seqs * call->channels == 0 || (call->T == 0 && call->final_state == nullptr))
        return RLCA_OK;
    ConvParams p = conv_params(*call, kForwardLaneBits);
    return launch(conv_kernel(*call, false), conv_grid(p), kConvThreads, 0, p, stream);
}

static size_t conv_partials(const rlca_conv_call &c) {
    return (size_t)c.num_seqs * c.channels *
           tiles_of(c.T, lane_bits_for(c.T, kBackwardLaneBits)) * (c.width + 1) * 4;
}

size_t rlca_causal_conv_backward_workspace_size(const rlca_conv_call *call) {
    Arrays a;
    if (call == nullptr || check_conv(*call, true, &a) != RLCA_OK) return 0;
    return conv_partials(*call);
}

rlca_status rlca_causal_conv_backward(const rlca_conv_call *call, void *workspace,
                                      size_t workspace_bytes, hipStream_t stream) {
    if (call == nullptr) return RLCA_ERR_NULL_POINTER;
    Arrays a;
    rlca_status st = check_conv(*call, true, &a);
    if (st != RLCA_OK) return st;
    const size_t need = conv_partials(*call);
    a.out(workspace, 4, true, {{(int64_t)(need / 4), 1}});
    st = a.status();
    if (st != RLCA_OK) return st;
    if (workspace_bytes < need) return RLCA_ERR_INVALID_SIZE;
    if (call->channels == 0) return RLCA_OK;
    const uint32_t tiles = tiles_of(call->T, lane_bits_for(call->T, kBackwardLaneBits));
    if (call->num_seqs != 0) {
        ConvParams p = conv_params(*call, kBackwardLaneBits);
        p.partials = static_cast<float *>(workspace);
        st = launch(conv_kernel(*call, true), conv_grid(p), kConvThreads, 0, p, stream);
        if (st != RLCA_OK) return st;
    }
    const float *partials = static_cast<const float *>(workspace);
    uint64_t per_channel = (uint64_t)call->num_seqs * tiles;
    uint32_t channels = (uint32_t)call->channels;
    float *gw = call->grad_weight, *gb = call->grad_bias;
    void *args[] = {&partials, &per_channel, &channels, &gw, &gb};
    const void *kernel = call->width == 2   ? (const void *)conv_weight_sums<2>
                         : call->width == 3 ? (const void *)conv_weight_sums<3>
                                            : (const void *)conv_weight_sums<4>;
    uint32_t threads = rlca::kWave;
    while (threads < (uint32_t)kSumThreads && threads < per_channel) threads *= 2;
    const hipError_t e = hipLaunchKernel(
        kernel, dim3(channels < (1u << 20) ? channels : 1u << 20), dim3(threads), args, 0, stream);
    return e == hipSuccess ? RLCA_OK : RLCA_ERR_HIP;
}

}  // extern "C"
