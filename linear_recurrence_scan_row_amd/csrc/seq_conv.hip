// seq_conv.hip -- the short causal convolution over rows of T steps, forward
// and backward:  pre_t = bias + sum_j weight[W-1-j] x_{t-j},  out = silu(pre).
//
// Bound by memory: W products and one exponential per step against two
// (forward) or three (backward) arrays of steps moved once.  A lane owns K = 8
// consecutive steps: their inputs are one or two 16-byte loads, and the W-1
// inputs before them (and, backward, the steps after them, whose pre is formed
// again here) are loads of lines that the neighbouring lanes read as well, so
// lanes need nothing from each other and HBM delivers each line once.
//
// Next to the memory's time stand a step's vector instructions: 20 forward, 36
// with episode starts, 86 backward with them.  So a workgroup keeps its channels
// and walks tiles of several rows: weights and addresses are formed once, one item is loaded while the one before is
// computed, and the weights' gradients leave the registers once at the end.
//
// Measured, hundreds of calls in a row: forward 1x4096x8191 bf16 29 us (4.8 TB/s);
// 4096x64x128 fp32 with episode starts 57 us forward (4.8 TB/s), 102 backward
// (4.1 TB/s; the vector units are busy 74% of it) and 5 for the weights' sums.
#include "seq.hpp"

namespace rlca {
namespace seq {

constexpr int kConvThreads = 256;
constexpr int kConvK = 8;
constexpr int kBack = 4;   // steps loaded before the block: W - 1 <= 3 are used
constexpr int kAhead = 4;  // backward: steps loaded after it

struct ConvParams {
    const void *x, *grad_out;
    const float *weight, *bias;
    const void *state, *grad_final;
    const uint8_t *flags;
    const int32_t *lengths;
    void *out, *final_state;
    void *grad_x, *grad_state;
    float *partials;  // [channels][gridDim.y][W + 1]
    int64_t x_n, x_d, g_n, g_d;
    uint32_t num_seqs, channels, tiles;
    uint32_t lane_bits;  // log2 of the lanes of a row
    int32_t T;
    int32_t silu, after_done;
};

// The tiles of all rows in order, every gridDim.y-th from blockIdx.y on.
struct ConvItem {
    uint32_t n, tile, step_n, step_tile;
    __device__ __forceinline__ explicit ConvItem(const ConvParams &p)
        : n(blockIdx.y / p.tiles), tile(blockIdx.y % p.tiles), step_n(gridDim.y / p.tiles),
          step_tile(gridDim.y % p.tiles) {}
    __device__ __forceinline__ void advance(const ConvParams &p) {
        n += step_n;
        tile += step_tile;
        if (tile >= p.tiles) tile -= p.tiles, ++n;
    }
};

// What a lane loads for a block of steps: the block, the steps before it (the
// state's at the row's start) and, backward, the steps after it and the
// output's gradient; and the flags that say where episodes start.
template <typename E, int W, bool FLAGS, bool BACKWARD>
struct ConvLoads {
    int t0, end;
    uint32_t n;
    Steps<kConvK, E> x, g;
    Steps<kBack, E> back;
    Steps<kAhead, E> after, g_after;
    FlagWindow flags, more_flags;

    __device__ __forceinline__ void load(const ConvParams &p, const ConvItem &item, uint32_t d,
                                         uint32_t lane) {
        n = item.n;
        end = row_end(p.lengths, n, p.T);
        t0 = (int)(((item.tile << p.lane_bits) + lane) * kConvK);
        if (t0 >= end) return;
        const E *row = static_cast<const E *>(p.x) + n * p.x_n + d * p.x_d + t0;
        x.load(row, end - t0);
        if (t0 > 0) {
            back.load(row - kBack, kBack);
        } else {
            back.b = {};
            if (p.state != nullptr) {
                const E *s = static_cast<const E *>(p.state) +
                             ((int64_t)n * p.channels + d) * (W - 1);
#pragma unroll
                for (int i = 0; i < W - 1; ++i) back.b[kBack - (W - 1) + i] = s[i];
            }
        }
        if constexpr (BACKWARD) {
            const E *grad = static_cast<const E *>(p.grad_out) + n * p.g_n + d * p.g_d + t0;
            g.load(grad, end - t0);
            if (end - t0 > kConvK) {
                after.load(row + kConvK, end - t0 - kConvK);
                g_after.load(grad + kConvK, end - t0 - kConvK);
            } else {  // a row's last lane, in nearly every wave: no step by step
                after.b = {};
                g_after.b = {};
            }
        }
        if constexpr (FLAGS) {
            const uint8_t *f = p.flags + (int64_t)n * p.T;
            flags.load(f, t0 - 2 - p.after_done, p.T);
            more_flags.load(f, t0 + 6 - p.after_done, p.T);
        }
    }
    // bit i: an episode starts at step t0 - 2 + i
    __device__ __forceinline__ uint32_t starts() const {
        if constexpr (!FLAGS) return 0u;
        return flags.template bits<8>() | more_flags.template bits<5>() << 8;
    }
};

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
__device__ __forceinline__ float state_at(const void *state, int64_t row, int q) {
    return state == nullptr ? 0.f : (float)static_cast<const E *>(state)[row * (W - 1) + W - 2 - q];
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
    constexpr int K = kConvK;
    const uint32_t lane = threadIdx.x & ((1u << p.lane_bits) - 1);
    const uint32_t d = (blockIdx.x * blockDim.x + threadIdx.x) >> p.lane_bits;
    if (d >= p.channels) return;
    ConvItem item(p);
    ConvLoads<E, W, FLAGS, false> next;
    next.load(p, item, d, lane);  // gridDim.y is at most the number of items
    float w[W];
#pragma unroll
    for (int j = 0; j < W; ++j) w[j] = p.weight[(int64_t)d * W + j];
    const float bias = p.bias == nullptr ? 0.f : p.bias[d];
    bool more = true;
    while (more) {
        const ConvLoads<E, W, FLAGS, false> now = next;
        item.advance(p);
        more = item.n < p.num_seqs;
        if (more) next.load(p, item, d, lane);
        const int64_t row = (int64_t)now.n * p.channels + d;
        const int n = now.end - now.t0;
        float o[K] = {};
        if (n > 0) {
            float v[kBack + K], back[kBack], cur[K];
            now.back.widen(back);
            now.x.widen(cur);
#pragma unroll
            for (int k = 0; k < kBack; ++k) v[k] = back[k];
#pragma unroll
            for (int k = 0; k < K; ++k) v[kBack + k] = cur[k];
            const Episodes<W> episodes(now.starts());
#pragma unroll
            for (int k = 0; k < K; ++k) {
                float pre = bias;
#pragma unroll
                for (int j = 0; j < W; ++j)
                    pre = fmaf(w[W - 1 - j], tap<W, FLAGS>(v, episodes, k, j), pre);
                o[k] = p.silu != 0 ? silu(pre) : pre;
            }
            if (n < K)
#pragma unroll
                for (int k = 0; k < K; ++k) o[k] = k < n ? o[k] : 0.f;
        }
        if (now.t0 < p.T)
            store_steps<K>(static_cast<E *>(p.out) + row * p.T + now.t0, p.T - now.t0, o);
        if (p.final_state != nullptr && now.t0 == 0) {
            const E *x = static_cast<const E *>(p.x) + now.n * p.x_n + d * p.x_d;
            const uint8_t *flags = FLAGS ? p.flags + (int64_t)now.n * p.T : nullptr;
            E *f = static_cast<E *>(p.final_state) + row * (W - 1);
            for (int i = 0; i < W - 1; ++i) {
                const int at = now.end - (W - 1) + i;
                float y = at >= 0 ? (float)x[at] : state_at<W, E>(p.state, row, -1 - at);
                if (FLAGS && !reaches_end(flags, at, now.end, p.T, p.after_done)) y = 0.f;
                f[i] = (E)y;
            }
        }
    }
}

// Backward:  dpre_t = grad_out_t silu'(pre_t),
//   grad_x_t = sum_j weight[W-1-j] dpre_{t+j}   (taps within t's episode),
//   grad_weight[k] = sum dpre_t x_{t-(W-1)+k},  grad_bias = sum dpre_t.
// A lane forms pre for its K steps and the W-1 after them.  Its sums for the
// weights meet the other lanes' of its row (at most one wave) at the end and
// are written as one partial per workgroup; conv_weight_sums adds those in
// order.
template <typename E, int W, bool FLAGS>
__global__ __launch_bounds__(kConvThreads) void causal_conv_backward(ConvParams p) {
    constexpr int K = kConvK, kSteps = K + W - 1;  // pre of these
    const uint32_t lane = threadIdx.x & ((1u << p.lane_bits) - 1);
    const uint32_t d = (blockIdx.x * blockDim.x + threadIdx.x) >> p.lane_bits;
    if (d >= p.channels) return;  // a row's lanes leave together
    ConvItem item(p);
    ConvLoads<E, W, FLAGS, true> next;
    next.load(p, item, d, lane);  // gridDim.y is at most the number of items
    float w[W], dw[W] = {}, db = 0.f;
#pragma unroll
    for (int j = 0; j < W; ++j) w[j] = p.weight[(int64_t)d * W + j];
    const float bias = p.bias == nullptr ? 0.f : p.bias[d];
    bool more = true;
    while (more) {
        const ConvLoads<E, W, FLAGS, true> now = next;
        item.advance(p);
        more = item.n < p.num_seqs;
        if (more) next.load(p, item, d, lane);
        const int64_t row = (int64_t)now.n * p.channels + d;
        const int t0 = now.t0, end = now.end, n = end - t0;
        const uint8_t *flags = FLAGS ? p.flags + (int64_t)now.n * p.T : nullptr;
        float dx[K] = {};
        if (n > 0) {
            float v[kBack + K + kAhead], go[K + kAhead];
            {
                float back[kBack], cur[K], after[kAhead], g[K], g_after[kAhead];
                now.back.widen(back);
                now.x.widen(cur);
                now.after.widen(after);
                now.g.widen(g);
                now.g_after.widen(g_after);
#pragma unroll
                for (int k = 0; k < kBack; ++k) v[k] = back[k];
#pragma unroll
                for (int k = 0; k < K; ++k) v[kBack + k] = cur[k], go[k] = g[k];
#pragma unroll
                for (int k = 0; k < kAhead; ++k) v[kBack + K + k] = after[k], go[K + k] = g_after[k];
            }
            const uint32_t starts = now.starts();
            const Episodes<W> episodes(starts);
            float dpre[kSteps];
#pragma unroll
            for (int k = 0; k < kSteps; ++k) {
                float pre = bias;
#pragma unroll
                for (int j = 0; j < W; ++j)
                    pre = fmaf(w[W - 1 - j], tap<W, FLAGS>(v, episodes, k, j), pre);
                dpre[k] = p.silu != 0 ? go[k] * silu_slope(pre, sigmoid(pre)) : go[k];
            }
            if (n < kSteps)  // past the end go is 0, but a slope may be anything
#pragma unroll
                for (int k = 0; k < kSteps; ++k) dpre[k] = k < n ? dpre[k] : 0.f;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                float s = 0.f;
#pragma unroll
                for (int j = 0; j < W; ++j) {
                    // step k is tap j of step k + j
                    const float g =
                        FLAGS && j > 0 ? episodes.keep(dpre[k + j], k + j, j) : dpre[k + j];
                    s = fmaf(w[W - 1 - j], g, s);
                }
                dx[k] = s;
                db += dpre[k];
#pragma unroll
                for (int j = 0; j < W; ++j)
                    dw[W - 1 - j] = fmaf(dpre[k], tap<W, FLAGS>(v, episodes, k, j), dw[W - 1 - j]);
            }
            if (n < K)
#pragma unroll
                for (int k = 0; k < K; ++k) dx[k] = k < n ? dx[k] : 0.f;
            if (p.grad_state != nullptr && t0 == 0) {
                E *gs = static_cast<E *>(p.grad_state) + row * (W - 1);
#pragma unroll
                for (int q = 0; q < W - 1; ++q) {  // the input at time q - (W-1)
                    float s = 0.f;
#pragma unroll
                    for (int t = 0; t <= q; ++t) {  // tap t + (W-1) - q of step t
                        const bool cut = FLAGS && (starts & (((1u << (t + 1)) - 1) << 2)) != 0;
                        s = fmaf(w[q - t], cut ? 0.f : dpre[t], s);
                    }
                    const int i = q - end;  // its place in the final state
                    if (p.grad_final != nullptr && i >= 0 &&
                        !(FLAGS && !reaches_end(flags, q - (W - 1), end, p.T, p.after_done)))
                        s += (float)static_cast<const E *>(p.grad_final)[row * (W - 1) + i];
                    gs[q] = (E)s;
                }
            }
            if (p.grad_final != nullptr && n - K < W - 1) {
                const E *gf = static_cast<const E *>(p.grad_final) + row * (W - 1);
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    const int i = t0 + k - (end - (W - 1));
                    if (i < 0 || i >= W - 1) continue;
                    if (FLAGS && !reaches_end(flags, t0 + k, end, p.T, p.after_done)) continue;
                    dx[k] += (float)gf[i];
                }
            }
        } else if (t0 == 0 && p.grad_state != nullptr) {  // an empty row hands its state on
            for (int q = 0; q < W - 1; ++q) {
                const int64_t at = row * (W - 1) + q;
                static_cast<E *>(p.grad_state)[at] =
                    p.grad_final == nullptr ? (E)0.f : static_cast<const E *>(p.grad_final)[at];
            }
        }
        if (t0 < p.T)
            store_steps<K>(static_cast<E *>(p.grad_x) + row * p.T + t0, p.T - t0, dx);
    }
    // the row's lanes, in a fixed tree
    for (uint32_t m = 1; m < (1u << p.lane_bits); m <<= 1) {
#pragma unroll
        for (int j = 0; j < W; ++j) dw[j] += __shfl_xor(dw[j], (int)m);
        db += __shfl_xor(db, (int)m);
    }
    if (lane == 0) {
        float *o = p.partials + ((int64_t)d * gridDim.y + blockIdx.y) * (W + 1);
#pragma unroll
        for (int j = 0; j < W; ++j) o[j] = dw[j];
        o[W] = db;
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

struct ConvShape {
    uint32_t lane_bits, tiles, threads;
    dim3 grid;
    // a launch's threads in x (2^24 channels of long rows do not fit one)
    bool fits() const { return (uint64_t)grid.x * threads < (1ull << 32); }
};

// A workgroup of at most 256 threads takes whole channels; about `blocks` of them
// walk the rows' tiles, with one number of turns for all.
static ConvShape conv_shape(const rlca_conv_call &c, uint32_t most_bits, uint32_t blocks) {
    ConvShape s = {};
    s.lane_bits = lane_bits_for(c.T, most_bits);
    const int64_t row_blocks = c.T <= 0 ? 1 : (c.T + kConvK - 1) / kConvK;
    s.tiles = (uint32_t)((row_blocks + (1ll << s.lane_bits) - 1) >> s.lane_bits);
    const uint64_t lanes = (uint64_t)c.channels << s.lane_bits;
    s.threads = lanes >= (uint64_t)kConvThreads ? kConvThreads
                : lanes == 0                    ? 64
                                                : (uint32_t)(lanes + 63) / 64 * 64;
    const uint64_t across = (lanes + s.threads - 1) / s.threads;
    const uint64_t items = (uint64_t)c.num_seqs * s.tiles;
    uint64_t most = across == 0 ? 1 : (blocks + across - 1) / across;  // 0: no channels
    if (most > 65535) most = 65535;
    const uint64_t turns = (items + most - 1) / most;
    s.grid = dim3((uint32_t)across, turns == 0 ? 0u : (uint32_t)((items + turns - 1) / turns));
    return s;
}

static ConvParams conv_params(const rlca_conv_call &c, const ConvShape &s) {
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
    p.num_seqs = (uint32_t)c.num_seqs;
    p.channels = (uint32_t)c.channels;
    p.tiles = s.tiles;
    p.T = (int32_t)c.T;
    p.lane_bits = s.lane_bits;
    p.silu = c.silu;
    p.after_done = c.convention == RLCA_RESET_AFTER_DONE;
    return p;
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

// Lanes of a row and workgroups of the two launches.  Forward and backward,
// fp32 with episode starts, 4096x64x128: 171, 166, 155, 151 and 156 us with
// 1024 / 640, 2048 / 1280, 4096 / 2560, 8192 / 5120 workgroups and one for every
// tile; bf16, 4x2048x2048: 42, 41, 44, 42 and 43.
static ConvShape forward_shape(const rlca_conv_call &c) { return conv_shape(c, 8, 8192); }
static ConvShape backward_shape(const rlca_conv_call &c) { return conv_shape(c, 6, 5120); }

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
    const ConvShape shape = forward_shape(*call);
    if (!shape.fits()) return RLCA_ERR_INVALID_SIZE;
    ConvParams p = conv_params(*call, shape);
    return launch(conv_kernel(*call, false), shape.grid, shape.threads, 0, p, stream);
}

static size_t conv_partials(const rlca_conv_call &c) {
    return (size_t)c.channels * backward_shape(c).grid.y * (c.width + 1) * 4;
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
    const ConvShape shape = backward_shape(*call);
    if (!shape.fits()) return RLCA_ERR_INVALID_SIZE;
    if (call->num_seqs != 0) {
        ConvParams p = conv_params(*call, shape);
        p.partials = static_cast<float *>(workspace);
        st = launch(conv_kernel(*call, true), shape.grid, shape.threads, 0, p, stream);
        if (st != RLCA_OK) return st;
    }
    const float *partials = static_cast<const float *>(workspace);
    uint64_t per_channel = call->num_seqs == 0 ? 0 : shape.grid.y;
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
