// norm.hip -- the root-mean-square norm over the channels of each step, with the
// residual's addition before it, its output in the storage type or in 8 bits with
// a scale a step, and its gradients:
//   s = x + residual,  r = 1 / sqrt(mean s^2 + eps),  y = s r weight;
//   grad_s = r (g w - s r mean(g w s r)) + grad_sum,  grad_weight = sum of g s r.
//
// Bound by memory: each value is read once and written once, so what a step's sums
// are formed of stays in registers until they are known.  Time is contiguous in the
// rows and the sums run over channels: a workgroup takes a few steps of a
// sequence, a thread 16 bytes of a channel's steps in `R` channels; where there are
// more channels than that, the rest are read again (from the caches).  Dense rows of
// channels (T = 1) take a wave or a workgroup a row.
//
// Measured, where a large copy reaches 5.05 TB/s: 8x2048 channels of 2048 steps bf16 with
// residual 43 us and gradients 62, each alone in a row, where part of the arrays stays in
// the last-level cache, 63 and 71 in turn (4.3 and 5.0 TB/s; the gradients read 286 MB for
// the 201 of the inputs, since not all of both arrays stays in registers); prompts of
// 6x1536x2049 fp16 to 8 bits, of different lengths, 37 to 47 (rows that begin at any 2
// bytes, and fewer tiles than compute units); 4096x64 of 128 steps fp32 107 (5.0).  Dense
// rows: one of 4096 channels 3.8; 16384 of 2048, bf16 with residual, 43 and 71 + 8, alone.
#include "seq.hpp"

namespace rlca {
namespace norm {

using seq::FastDiv;
using seq::Steps;

struct NormParams {
    const void *x, *residual, *grad_out, *grad_sum;
    const float *weight;
    const int32_t *lengths;
    void *out, *sum, *grad_x;
    uint8_t *out8;
    float *scale;
    float *partials;  // [workgroups or waves][channels]: sums for grad_weight
    int64_t x_n, x_d, r_n, r_d, g_n, g_d, s_n, s_d;
    uint32_t channels;
    int32_t T;
    uint32_t tiles;       // of a sequence
    uint32_t work;        // tiles, or rows, of the call
    float eps, per_channel;  // 1 / channels
    FastDiv by_tiles;
};

// x, without the compiler's knowledge that it is: addresses formed from it are formed
// where they stand, not kept in registers from an earlier pass over the channels.
__device__ __forceinline__ uint32_t here(uint32_t x) {
    asm volatile("" : "+v"(x));
    return x;
}

// The same for a block: what was widened for the sums is widened again, not kept.
template <int K, typename E>
__device__ __forceinline__ void here(Steps<K, E> &b) {
    typedef uint32_t words __attribute__((ext_vector_type(sizeof(b.b) / 4)));
    words w = __builtin_bit_cast(words, b.b);
    asm volatile("" : "+v"(w));
    b.b = __builtin_bit_cast(decltype(b.b), w);
}

// Squares of values from 2^50 on may overflow a sum of float32, so where a thread's
// sum reaches 2^100 the workgroup forms its sums again, from values times 2^-80 in the
// steps whose sums do.  (fp16 values end at 2^16.)  `factor` is 2^-80 or 1; r below
// includes it.
constexpr float kMuch = 0x1p100f, kDown = 0x1p-80f;
template <typename E>
constexpr bool overflows() {
    return !std::is_same<E, _Float16>::value;
}

constexpr int kBatch = 2;  // channels whose loads are issued together
template <int N>
using Count = std::integral_constant<int, N>;

constexpr float kMostE4m3 = 448.f, kLeastScale = 0x1p-120f;

// The largest magnitude, a NaN above all: float32 bits without the sign, as integers.
__device__ __forceinline__ uint32_t magnitude(float x) {
    return __builtin_bit_cast(uint32_t, x) & 0x7fffffffu;
}
__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) { return a > b ? a : b; }

// r / factor, from the sum of squares of values times factor; and a step's scale.
__device__ __forceinline__ float rsqrt_of(const NormParams &p, float sum, float factor) {
    return __builtin_amdgcn_rsqf(fmaf(sum, p.per_channel, p.eps * factor * factor));
}
__device__ __forceinline__ float scale_of(uint32_t most, float r) {
    const float s = __builtin_bit_cast(float, most) * r / kMostE4m3;
    return s < kLeastScale ? kLeastScale : s;  // a NaN stays one
}
// What s and the weight are multiplied by for the 8-bit value: 448 / max|s weight|, since
// r is in both (each rounding left out is a value less that falls on the other side of
// a border); NaN where the scale is.  Where all products are 0 anything finite will do.
__device__ __forceinline__ float gain_of(uint32_t most, float factor, float r, float scale) {
    const float g = kMostE4m3 / __builtin_bit_cast(float, most) * factor;
    return scale != scale ? scale : most == 0 ? r : g;
}
// Whether a step's 8-bit values have to be formed from y itself, with passes of their own:
// near the least scale, and where s weight is so small that its largest is no normal
// number or 448 / it too large a one, or that all of them have underflowed and r is
// large enough to bring them back (eps below 2^-36).
__device__ __forceinline__ bool small_values(uint32_t most, float factor, float r, float scale) {
    const uint32_t least = __builtin_bit_cast(uint32_t, kMostE4m3 * 0x1p-126f);
    return most == 0 ? r > 0x1p18f : scale < 0x1p-100f || (factor == 1.f && most < least);
}

// K values in e4m3, rounded to nearest even.  Those of one step are at most 448 up to
// the rounding of their products, which rounds to 448.
template <int K>
__device__ __forceinline__ void store_e4m3(uint8_t *to, int n, const float (&v)[K]) {
    static_assert(K % 4 == 0, "whole words");
    uint32_t w[K / 4];
#pragma unroll
    for (int j = 0; j < K / 4; ++j) {
        int q = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * j], v[4 * j + 1], 0, false);
        q = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * j + 2], v[4 * j + 3], q, true);
        w[j] = (uint32_t)q;
    }
    if (n >= K) {
        __builtin_memcpy(to, w, K);
    } else {
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (k < n) to[k] = (uint8_t)(w[k / 4] >> (8 * (k % 4)));
    }
}

template <int K, typename E>
__device__ __forceinline__ void clear(Steps<K, E> &b) {
#pragma unroll
    for (int k = 0; k < K; ++k) b.b[k] = (E)0.f;
}

// x + residual as it is stored.
template <int K, typename E>
__device__ __forceinline__ void add_residual(Steps<K, E> &b, const Steps<K, E> &r) {
#pragma unroll
    for (int k = 0; k < K; ++k) b.b[k] = (E)((float)b.b[k] + (float)r.b[k]);
}

template <int K, typename E>
__device__ __forceinline__ void store_block(E *p, int n, const Steps<K, E> &b) {
    if (n >= K) {
        __builtin_memcpy(p, &b.b, sizeof b.b);
    } else {
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (k < n) p[k] = b.b[k];
    }
}

// ------------------------------------------------------------- rows over time
// The tile of workgroup i of n: workgroups go to the 8 XCDs in turn, and tiles side by
// side share cache lines where a row is not aligned or a tile is narrower than a line,
// so each XCD gets a run of tiles.
__device__ __forceinline__ uint32_t near(uint32_t i, uint32_t n) {
    const uint32_t run = n / 8;
    return i < 8 * run ? i % 8 * run + i / 8 : i;
}

// Where a workgroup works: LT threads side by side take VEC = 16 / sizeof(E) steps
// each, and THREADS / LT channels at a time.
template <typename E, int THREADS, int LT>
struct Tile {
    static constexpr int VEC = 16 / sizeof(E), STEPS = LT * VEC, ACROSS = THREADS / LT,
                         WAVES = THREADS / kWave;
    uint32_t n, first;  // the sequence and the thread's first channel
    int column, t, left, room;  // first step in the tile, in the row; steps that count, that exist
    __device__ __forceinline__ void set(const NormParams &p, uint32_t i) {
        const uint32_t tile = near(i, p.work);
        n = p.by_tiles.div(tile);
        column = (int)(threadIdx.x % LT) * VEC;
        t = (int)(tile - n * p.tiles) * STEPS + column;
        first = here(threadIdx.x / LT);
        left = seq::row_end(p.lengths, n, p.T) - t;
        room = p.T - t;
    }
};

// Sums over the channels of a tile's steps: s over a wave's lanes of one column, then
// over the waves through LDS.
template <int VEC, int LT>
__device__ __forceinline__ void wave_sums(float (&s)[VEC]) {
#pragma unroll
    for (int m = LT; m < kWave; m <<= 1)
#pragma unroll
        for (int k = 0; k < VEC; ++k) s[k] += __shfl_xor(s[k], m);
}

template <int VEC, int LT>
__device__ __forceinline__ void wave_most(uint32_t (&s)[VEC]) {
#pragma unroll
    for (int m = LT; m < kWave; m <<= 1)
#pragma unroll
        for (int k = 0; k < VEC; ++k) s[k] = larger(s[k], (uint32_t)__shfl_xor((int)s[k], m));
}

// Any lane of the workgroup: one word a wave in LDS, written before a barrier.
__device__ __forceinline__ void tell(uint32_t *words, bool x) {
    const bool any = __builtin_amdgcn_ballot_w64(x) != 0;
    if (threadIdx.x % kWave == 0) words[threadIdx.x / kWave] = any ? 1u : 0u;
}
template <int WAVES>
__device__ __forceinline__ bool told(const uint32_t *words) {
    uint32_t any = 0;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) any |= words[w];
    return __builtin_amdgcn_readfirstlane(any) != 0;
}

template <typename E, int THREADS, int LT, int R, bool Q8>
__global__ __launch_bounds__(THREADS) void rms_norm_rows(NormParams p) {
    typedef Tile<E, THREADS, LT> Mine;
    constexpr int VEC = Mine::VEC, ACROSS = Mine::ACROSS, WAVES = Mine::WAVES;
    __shared__ __attribute__((aligned(16))) float sums[WAVES][Mine::STEPS];
    __shared__ __attribute__((aligned(16))) uint32_t mosts[Q8 ? WAVES : 1][Mine::STEPS];
    __shared__ uint32_t large[WAVES];
    __shared__ float factors[Q8 ? Mine::STEPS : 1];  // of the steps, where told(large)
    Mine at;
    at.set(p, blockIdx.x);
    const E *x = static_cast<const E *>(p.x) + at.n * p.x_n;
    const E *res =
        p.residual == nullptr ? nullptr : static_cast<const E *>(p.residual) + at.n * p.r_n;
    const int64_t out_row = (int64_t)at.n * p.channels * p.T;
    E *sum_out = static_cast<E *>(p.sum) + out_row;
    const auto to = [&](uint32_t d) { return out_row + (int64_t)d * p.T + at.t; };

    // kBatch channels' steps, every load issued before the first value is used; their
    // sums are stored the first time
    const auto fetch_batch = [&](uint32_t d, auto *b, auto count, bool store) {
        constexpr int N = decltype(count)::value;
#pragma unroll
        for (int u = 0; u < N; ++u)
            if (d + u * ACROSS < p.channels)
                b[u].load(x + ((d + u * ACROSS) * p.x_d + at.t), at.left);
            else
                clear(b[u]);
        if (res == nullptr) return;
        Steps<VEC, E> r[N];
#pragma unroll
        for (int u = 0; u < N; ++u)
            if (d + u * ACROSS < p.channels)
                r[u].load(res + ((d + u * ACROSS) * p.r_d + at.t), at.left);
#pragma unroll
        for (int u = 0; u < N; ++u)
            if (d + u * ACROSS < p.channels) {
                add_residual(b[u], r[u]);
                if (store)
                    store_block(sum_out + ((int64_t)(d + u * ACROSS) * p.T + at.t), at.room, b[u]);
            }
    };
    const auto weight = [&](uint32_t d) { return p.weight == nullptr ? 1.f : p.weight[d]; };

    Steps<VEC, E> kept[R];
    float s[VEC] = {};
    uint32_t most[VEC] = {};
    float factor[VEC];
#pragma unroll
    for (int k = 0; k < VEC; ++k) factor[k] = 1.f;
    const auto add = [&](const Steps<VEC, E> &b, uint32_t d, bool scaled) {
        float v[VEC];
        b.widen(v);
        const float w = Q8 ? weight(d) : 0.f;
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
            if (scaled) v[k] *= factor[k];
            s[k] = fmaf(v[k], v[k], s[k]);
            if constexpr (Q8) most[k] = larger(most[k], magnitude(v[k] * w));
        }
    };
#pragma unroll
    for (int j = 0; j < R; j += kBatch)
        fetch_batch(at.first + j * ACROSS, kept + j, Count<kBatch>{}, true);
    const uint32_t wave = threadIdx.x / kWave;
    const auto meet = [&] {
        wave_sums<VEC, LT>(s);
        if constexpr (Q8) wave_most<VEC, LT>(most);
        if (threadIdx.x % kWave < LT)
#pragma unroll
            for (int k = 0; k < VEC; ++k) {
                sums[wave][at.column + k] = s[k];
                if constexpr (Q8) mosts[wave][at.column + k] = most[k];
            }
    };
    const auto all = [&] {
#pragma unroll
        for (int k = 0; k < VEC; ++k) s[k] = 0.f, most[k] = 0;
#pragma unroll 2
        for (int w = 0; w < WAVES; ++w)
#pragma unroll
            for (int k = 0; k < VEC; ++k) {
                s[k] += sums[w][at.column + k];
                if constexpr (Q8) most[k] = larger(most[k], mosts[w][at.column + k]);
            }
    };
#pragma unroll
    for (int j = 0; j < R; ++j) {
        const uint32_t d = at.first + j * ACROSS;
        if (d < p.channels) add(kept[j], d, false);
    }
    for (uint32_t d = at.first + R * ACROSS; d < p.channels; d += kBatch * ACROSS) {
        Steps<VEC, E> b[kBatch];
        fetch_batch(d, b, Count<kBatch>{}, true);
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
            if (d + u * ACROSS < p.channels) add(b[u], d + u * ACROSS, false);
    }
    if constexpr (overflows<E>()) {
        bool much = false;
#pragma unroll
        for (int k = 0; k < VEC; ++k) much |= s[k] >= kMuch;
        tell(large, much);
    }
    meet();
    __syncthreads();
    all();
    at.first = here(at.first);
    if (overflows<E>() && told<WAVES>(large)) {
        __syncthreads();
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
            factor[k] = s[k] >= kMuch ? kDown : 1.f;
            if (Q8 && threadIdx.x < LT) factors[at.column + k] = factor[k];
            s[k] = 0.f, most[k] = 0;
        }
        // read again, so that this costs the usual case no registers
#pragma unroll 1
        for (uint32_t d = at.first; d < p.channels; d += ACROSS) {
            Steps<VEC, E> b[1];
            fetch_batch(d, b, Count<1>{}, false);
            add(b[0], d, true);
        }
        meet();
        __syncthreads();
        all();
    }
    float r[VEC], scale[VEC];
    bool small = false;
#pragma unroll
    for (int k = 0; k < VEC; ++k) {
        const float root = rsqrt_of(p, s[k], factor[k]);
        r[k] = factor[k] * root;
        if constexpr (Q8) {
            // `most` has the factor too
            scale[k] = scale_of(most[k], root);
            small |= small_values(most[k], factor[k], r[k], scale[k]);
            r[k] = gain_of(most[k], factor[k], r[k], scale[k]);
        }
    }
    const auto store_scales = [&] {
        if (threadIdx.x < LT)
#pragma unroll
            for (int k = 0; k < VEC; ++k)
                if (k < at.room)
                    p.scale[(int64_t)at.n * p.T + at.t + k] = k < at.left ? scale[k] : 0.f;
    };
    if constexpr (Q8) {
        store_scales();
        // every wave has all columns, so all of the workgroup's agree
        if (__builtin_amdgcn_ballot_w64(small) != 0) {
            // the steps that need it: their largest |y|, and y / scale; the others as
            // below.  All is formed anew, so that this costs the usual case no registers.
            at.first = here(at.first);
            at.t = (int)here((uint32_t)at.t);
            all();
            const bool down = overflows<E>() && told<WAVES>(large);
            float by[VEC];
#pragma unroll
            for (int k = 0; k < VEC; ++k) {
                const float f = down ? factors[at.column + k] : 1.f, root = rsqrt_of(p, s[k], f);
                scale[k] = scale_of(most[k], root);
                by[k] = 1.f;
                if (small_values(most[k], f, f * root, scale[k])) {
                    r[k] = f * root;
                    by[k] = 0.f;
                    most[k] = 0;
                }
            }
            const auto value = [&](const Steps<VEC, E> &b, uint32_t d, float(&v)[VEC]) {
                b.widen(v);
                const float w = weight(d);
#pragma unroll
                for (int k = 0; k < VEC; ++k) v[k] = v[k] * r[k] * w;
            };
#pragma unroll 1
            for (uint32_t d = at.first; d < p.channels; d += ACROSS) {
                Steps<VEC, E> b[1];
                float v[VEC];
                fetch_batch(d, b, Count<1>{}, false);
                value(b[0], d, v);
#pragma unroll
                for (int k = 0; k < VEC; ++k)
                    if (by[k] == 0.f) most[k] = larger(most[k], magnitude(v[k]));
            }
            wave_most<VEC, LT>(most);
            __syncthreads();  // the sums have been read
            if (threadIdx.x % kWave < LT)
#pragma unroll
                for (int k = 0; k < VEC; ++k) mosts[wave][at.column + k] = most[k];
            __syncthreads();
#pragma unroll
            for (int k = 0; k < VEC; ++k)
                if (by[k] == 0.f) {
                    for (int w = 0; w < WAVES; ++w)
                        most[k] = larger(most[k], mosts[w][at.column + k]);
                    scale[k] = scale_of(most[k], 1.f);
                    by[k] = 1.f / scale[k];
                }
            store_scales();
#pragma unroll 1
            for (uint32_t d = at.first; d < p.channels; d += ACROSS) {
                Steps<VEC, E> b[1];
                float v[VEC];
                fetch_batch(d, b, Count<1>{}, false);
                value(b[0], d, v);
#pragma unroll
                for (int k = 0; k < VEC; ++k) v[k] = k < at.left ? v[k] * by[k] : 0.f;
                store_e4m3<VEC>(p.out8 + to(d), at.room, v);
            }
            return;
        }
    }
    at.first = here(at.first);
    at.t = (int)here((uint32_t)at.t);
#pragma unroll
    for (int j = 0; j < R; ++j) here(kept[j]);
    const auto finish = [&](const Steps<VEC, E> &b, uint32_t d) {
        float v[VEC];
        b.widen(v);
        const float w = weight(d);
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
            v[k] = v[k] * r[k] * w;
            if (k >= at.left) v[k] = 0.f;
        }
        if constexpr (Q8)
            store_e4m3<VEC>(p.out8 + to(d), at.room, v);
        else
            seq::store_steps<VEC>(static_cast<E *>(p.out) + to(d), at.room, v);
    };
#pragma unroll
    for (int j = 0; j < R; ++j) {
        const uint32_t d = at.first + j * ACROSS;
        if (d < p.channels) finish(kept[j], d);
    }
    for (uint32_t d = at.first + R * ACROSS; d < p.channels; d += kBatch * ACROSS) {
        Steps<VEC, E> b[kBatch];
        fetch_batch(d, b, Count<kBatch>{}, false);
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
            if (d + u * ACROSS < p.channels) finish(b[u], d + u * ACROSS);
    }
}

// The gradients: a workgroup walks tiles and keeps its channels' sums for
// grad_weight, in registers for the channels that it keeps, in its own part of the
// partial sums for the others.
template <typename E, int THREADS, int LT, int R>
__global__ __launch_bounds__(THREADS) void rms_norm_rows_backward(NormParams p) {
    typedef Tile<E, THREADS, LT> Mine;
    constexpr int VEC = Mine::VEC, ACROSS = Mine::ACROSS, WAVES = Mine::WAVES;
    static_assert(R % kBatch == 0, "whole batches");
    __shared__ __attribute__((aligned(16))) float sums[2][WAVES][Mine::STEPS];
    __shared__ uint32_t large[WAVES];
    const auto weight = [&](uint32_t d) { return p.weight == nullptr ? 1.f : p.weight[d]; };
    float *partial = p.partials + (int64_t)blockIdx.x * p.channels;
    constexpr int kKept = R > 0 ? R : 1;
    float grad_weight[kKept] = {};
    bool begun = false;
    for (uint32_t tile = blockIdx.x; tile < p.work; tile += gridDim.x) {
        Mine at;
        at.set(p, tile);
        const E *x = static_cast<const E *>(p.x) + at.n * p.x_n + at.t;
        const E *go = static_cast<const E *>(p.grad_out) + at.n * p.g_n + at.t;
        const E *gs = p.grad_sum == nullptr
                          ? nullptr
                          : static_cast<const E *>(p.grad_sum) + at.n * p.s_n + at.t;
        E *to = static_cast<E *>(p.grad_x) + (int64_t)at.n * p.channels * p.T + at.t;
        Steps<VEC, E> xs[kKept], gos[kKept];
        float s[VEC] = {}, c[VEC] = {}, factor[VEC];
#pragma unroll
        for (int k = 0; k < VEC; ++k) factor[k] = 1.f;
        const auto add = [&](const Steps<VEC, E> &xb, const Steps<VEC, E> &gb, uint32_t d,
                             bool scaled) {
            float v[VEC], g[VEC];
            xb.widen(v);
            gb.widen(g);
            const float w = weight(d);
#pragma unroll
            for (int k = 0; k < VEC; ++k) {
                if (scaled) v[k] *= factor[k];
                s[k] = fmaf(v[k], v[k], s[k]);
                c[k] = fmaf(v[k], g[k] * w, c[k]);
            }
        };
        const auto fetch_batch = [&](uint32_t d, auto &xb, auto &gb) {
            constexpr int N = sizeof(xb) / sizeof(xb[0]);
#pragma unroll
            for (int u = 0; u < N; ++u) {
                const uint32_t e = d + u * ACROSS;
                if (e < p.channels) {
                    xb[u].load(x + e * p.x_d, at.left);
                    gb[u].load(go + e * p.g_d, at.left);
                } else {
                    clear(xb[u]);
                    clear(gb[u]);
                }
            }
        };
        const auto fetch_more = [&](uint32_t d, auto &more) {
            constexpr int N = sizeof(more) / sizeof(more[0]);
#pragma unroll
            for (int u = 0; u < N; ++u)
                if (gs != nullptr && d + u * ACROSS < p.channels)
                    more[u].load(gs + (d + u * ACROSS) * p.s_d, at.left);
                else
                    clear(more[u]);
        };
        if constexpr (R > 0) fetch_batch(at.first, xs, gos);
        const uint32_t wave = threadIdx.x / kWave;
        const auto meet = [&] {
            wave_sums<VEC, LT>(s);
            wave_sums<VEC, LT>(c);
            if (threadIdx.x % kWave < LT)
#pragma unroll
                for (int k = 0; k < VEC; ++k) {
                    sums[0][wave][at.column + k] = s[k];
                    sums[1][wave][at.column + k] = c[k];
                }
        };
        const auto all = [&] {
#pragma unroll
            for (int k = 0; k < VEC; ++k) s[k] = c[k] = 0.f;
#pragma unroll 2
            for (int w = 0; w < WAVES; ++w)
#pragma unroll
                for (int k = 0; k < VEC; ++k) {
                    s[k] += sums[0][w][at.column + k];
                    c[k] += sums[1][w][at.column + k];
                }
        };
#pragma unroll
        for (int j = 0; j < R; ++j) {
            const uint32_t d = at.first + j * ACROSS;
            if (d < p.channels) add(xs[j], gos[j], d, false);
        }
        for (uint32_t d = at.first + R * ACROSS; d < p.channels; d += kBatch * ACROSS) {
            Steps<VEC, E> xb[kBatch], gb[kBatch];
            fetch_batch(d, xb, gb);
#pragma unroll
            for (int u = 0; u < kBatch; ++u)
                if (d + u * ACROSS < p.channels) add(xb[u], gb[u], d + u * ACROSS, false);
        }
        __syncthreads();  // the sums of the tile before have been read
        if constexpr (overflows<E>()) {
            bool much = false;
#pragma unroll
            for (int k = 0; k < VEC; ++k) much |= s[k] >= kMuch;
            tell(large, much);
        }
        meet();
        __syncthreads();
        all();
        at.first = here(at.first);
        if (overflows<E>() && told<WAVES>(large)) {
            __syncthreads();
#pragma unroll
            for (int k = 0; k < VEC; ++k) {
                factor[k] = s[k] >= kMuch ? kDown : 1.f;
                s[k] = c[k] = 0.f;
            }
            // read again, so that this costs the usual case no registers
#pragma unroll 1
            for (uint32_t d = at.first; d < p.channels; d += ACROSS) {
                Steps<VEC, E> xb, gb;
                xb.load(x + d * p.x_d, at.left);
                gb.load(go + d * p.g_d, at.left);
                add(xb, gb, d, true);
            }
            meet();
            __syncthreads();
            all();
        }
        float r[VEC];
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
            const float root = rsqrt_of(p, s[k], factor[k]);
            r[k] = factor[k] * root;
            c[k] = c[k] * root * p.per_channel;  // mean(g w s r)
        }
        at.first = here(at.first);
#pragma unroll
        for (int j = 0; j < R; ++j) here(xs[j]), here(gos[j]);
        const auto finish = [&](const Steps<VEC, E> &xb, const Steps<VEC, E> &gb,
                                const Steps<VEC, E> &mb, uint32_t d) {
            float v[VEC], g[VEC], more[VEC], total = 0.f;
            xb.widen(v);
            gb.widen(g);
            mb.widen(more);
            const float w = weight(d);
#pragma unroll
            for (int k = 0; k < VEC; ++k) {
                const float xh = v[k] * r[k];
                const bool counts = k < at.left;
                total += counts ? g[k] * xh : 0.f;
                v[k] = counts ? fmaf(r[k], fmaf(g[k], w, -xh * c[k]), more[k]) : 0.f;
            }
            seq::store_steps<VEC>(to + (int64_t)d * p.T, at.room, v);
            return total;
        };
#pragma unroll
        for (int j = 0; j < R; j += kBatch) {
            Steps<VEC, E> more[kBatch];
            fetch_more(at.first + j * ACROSS, more);
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                const uint32_t d = at.first + (j + u) * ACROSS;
                if (d < p.channels) grad_weight[j + u] += finish(xs[j + u], gos[j + u], more[u], d);
            }
        }
        for (uint32_t d = at.first + R * ACROSS; d < p.channels; d += kBatch * ACROSS) {
            Steps<VEC, E> xb[kBatch], gb[kBatch], more[kBatch];
            fetch_batch(d, xb, gb);
            fetch_more(d, more);
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                const uint32_t e = d + u * ACROSS;
                if (e >= p.channels) continue;
                float total = finish(xb[u], gb[u], more[u], e);
#pragma unroll
                for (int m = 1; m < LT; m <<= 1) total += __shfl_xor(total, m);
                if (threadIdx.x % LT == 0) partial[e] = begun ? partial[e] + total : total;
            }
        }
        begun = true;
    }
#pragma unroll
    for (int j = 0; j < R; ++j) {
        const uint32_t d = threadIdx.x / LT + j * ACROSS;
        float total = grad_weight[j];
#pragma unroll
        for (int m = 1; m < LT; m <<= 1) total += __shfl_xor(total, m);
        if (threadIdx.x % LT == 0 && d < p.channels) partial[d] = total;
    }
}

// ------------------------------------------------------------- rows of channels
// WAVES waves of a workgroup take a row: thread i the blocks i, i + 64 WAVES, ... of
// VEC channels.
constexpr int kRowThreads = 256;

template <int WAVES>
__device__ __forceinline__ void row_sums(float &a, float &b, uint32_t &most, float (&lds)[2][4],
                                         uint32_t (&lds_most)[4]) {
#pragma unroll
    for (int m = 1; m < kWave; m <<= 1) {
        a += __shfl_xor(a, m);
        b += __shfl_xor(b, m);
        most = larger(most, (uint32_t)__shfl_xor((int)most, m));
    }
    if constexpr (WAVES > 1) {
        const uint32_t wave = threadIdx.x / kWave;
        __syncthreads();  // what stood there has been read
        if (threadIdx.x % kWave == 0) lds[0][wave] = a, lds[1][wave] = b, lds_most[wave] = most;
        __syncthreads();
        a = b = 0.f;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) {
            a += lds[0][w];
            b += lds[1][w];
            most = larger(most, lds_most[w]);
        }
    }
}

template <typename E, int WAVES, int R, bool Q8>
__global__ __launch_bounds__(kRowThreads) void rms_norm_dense(NormParams p) {
    constexpr int VEC = 16 / sizeof(E), ROWS = kRowThreads / kWave / WAVES;
    constexpr uint32_t ACROSS = WAVES * kWave;
    __shared__ float lds[2][4];
    __shared__ uint32_t lds_most[4];
    const uint32_t n = blockIdx.x * ROWS + threadIdx.x / ACROSS;
    if (n >= p.work) return;  // whole waves, and whole workgroups where waves meet
    const bool counts = seq::row_end(p.lengths, n, 1) > 0;
    const int D = counts ? (int)p.channels : 0;
    const E *x = static_cast<const E *>(p.x) + n * p.x_n;
    const E *res =
        p.residual == nullptr ? nullptr : static_cast<const E *>(p.residual) + n * p.r_n;
    const int64_t to = (int64_t)n * p.channels;
    const uint32_t blocks = (p.channels + VEC - 1) / VEC, first = threadIdx.x % ACROSS;
    const auto fetch = [&](uint32_t i, Steps<VEC, E> &b, bool store) {
        b.load(x + (int64_t)i * VEC, D - (int)i * VEC);
        if (res != nullptr) {
            Steps<VEC, E> r;
            r.load(res + (int64_t)i * VEC, D - (int)i * VEC);
            add_residual(b, r);
            if (store)
                store_block(static_cast<E *>(p.sum) + to + (int64_t)i * VEC,
                            (int)p.channels - (int)i * VEC, b);
        }
    };
    const auto weights = [&](uint32_t i, float(&w)[VEC]) {
        if (p.weight != nullptr) {
            seq::load_steps<VEC>(p.weight + (int64_t)i * VEC, (int)p.channels - (int)i * VEC, w);
        } else {
#pragma unroll
            for (int k = 0; k < VEC; ++k) w[k] = 1.f;
        }
    };
    Steps<VEC, E> kept[R];
    float s = 0.f, unused = 0.f;
    uint32_t most = 0;
    const auto add = [&](const Steps<VEC, E> &b, uint32_t i, float factor) {
        float v[VEC], w[VEC];
        b.widen(v);
        if constexpr (Q8) weights(i, w);
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
            v[k] *= factor;
            s = fmaf(v[k], v[k], s);
            if constexpr (Q8) most = larger(most, magnitude(v[k] * w[k]));
        }
    };
#pragma unroll
    for (int j = 0; j < R; ++j)
        if (first + j * ACROSS < blocks) fetch(first + j * ACROSS, kept[j], true);
#pragma unroll
    for (int j = 0; j < R; ++j)
        if (first + j * ACROSS < blocks) add(kept[j], first + j * ACROSS, 1.f);
    for (uint32_t i = first + R * ACROSS; i < blocks; i += ACROSS) {
        Steps<VEC, E> b;
        fetch(i, b, true);
        add(b, i, 1.f);
    }
    row_sums<WAVES>(s, unused, most, lds, lds_most);
    float factor = 1.f;
    if (overflows<E>() && s >= kMuch) {  // the same in all of a row's threads
        factor = kDown;
        s = 0.f;
        most = 0;
#pragma unroll
        for (int j = 0; j < R; ++j)
            if (first + j * ACROSS < blocks) add(kept[j], first + j * ACROSS, factor);
        for (uint32_t i = first + R * ACROSS; i < blocks; i += ACROSS) {
            Steps<VEC, E> b;
            fetch(i, b, false);
            add(b, i, factor);
        }
        row_sums<WAVES>(s, unused, most, lds, lds_most);
    }
    const float root = rsqrt_of(p, s, factor);
    float r = factor * root;
    if constexpr (Q8) {
        float scale = scale_of(most, root);
        if (small_values(most, factor, r, scale)) {  // the same in all of a row's threads
            const auto value = [&](uint32_t i, float(&v)[VEC]) {
                Steps<VEC, E> b;
                float w[VEC];
                fetch(i, b, false);
                b.widen(v);
                weights(i, w);
#pragma unroll
                for (int k = 0; k < VEC; ++k) v[k] = v[k] * r * w[k];
            };
            most = 0;
#pragma unroll 1
            for (uint32_t i = first; i < blocks; i += ACROSS) {
                float v[VEC];
                value(i, v);
#pragma unroll
                for (int k = 0; k < VEC; ++k) most = larger(most, magnitude(v[k]));
            }
            row_sums<WAVES>(s, unused, most, lds, lds_most);
            scale = scale_of(most, 1.f);
            const float by = 1.f / scale;
            if (first == 0) p.scale[n] = counts ? scale : 0.f;
#pragma unroll 1
            for (uint32_t i = first; i < blocks; i += ACROSS) {
                float v[VEC];
                value(i, v);
#pragma unroll
                for (int k = 0; k < VEC; ++k) v[k] = counts ? v[k] * by : 0.f;
                store_e4m3<VEC>(p.out8 + to + (int64_t)i * VEC, (int)p.channels - (int)i * VEC, v);
            }
            return;
        }
        if (first == 0) p.scale[n] = counts ? scale : 0.f;
        r = gain_of(most, factor, r, scale);
    }
    const auto finish = [&](const Steps<VEC, E> &b, uint32_t i) {
        float v[VEC], w[VEC];
        b.widen(v);
        weights(i, w);
#pragma unroll
        for (int k = 0; k < VEC; ++k) v[k] = counts ? v[k] * r * w[k] : 0.f;
        const int room = (int)p.channels - (int)i * VEC;
        if constexpr (Q8)
            store_e4m3<VEC>(p.out8 + to + (int64_t)i * VEC, room, v);
        else
            seq::store_steps<VEC>(static_cast<E *>(p.out) + to + (int64_t)i * VEC, room, v);
    };
#pragma unroll
    for (int j = 0; j < R; ++j)
        if (first + j * ACROSS < blocks) finish(kept[j], first + j * ACROSS);
    for (uint32_t i = first + R * ACROSS; i < blocks; i += ACROSS) {
        Steps<VEC, E> b;
        fetch(i, b, false);
        finish(b, i);
    }
}

// The gradients: a wave, or a workgroup, walks rows.
template <typename E, int WAVES, int R>
__global__ __launch_bounds__(kRowThreads) void rms_norm_dense_backward(NormParams p) {
    constexpr int VEC = 16 / sizeof(E), ROWS = kRowThreads / kWave / WAVES;
    constexpr uint32_t ACROSS = WAVES * kWave;
    __shared__ float lds[2][4];
    __shared__ uint32_t lds_most[4];
    const uint32_t walker = blockIdx.x * ROWS + threadIdx.x / ACROSS, walkers = gridDim.x * ROWS;
    const uint32_t blocks = (p.channels + VEC - 1) / VEC, first = threadIdx.x % ACROSS;
    float *partial = p.partials + (int64_t)walker * p.channels;
    float grad_weight[R][VEC] = {};
    const auto weights = [&](uint32_t i, float(&w)[VEC]) {
        if (p.weight != nullptr) {
            seq::load_steps<VEC>(p.weight + (int64_t)i * VEC, (int)p.channels - (int)i * VEC, w);
        } else {
#pragma unroll
            for (int k = 0; k < VEC; ++k) w[k] = 1.f;
        }
    };
    bool begun = false;
    for (uint32_t n = walker; n < p.work; n += walkers) {
        const bool counts = seq::row_end(p.lengths, n, 1) > 0;
        const int D = counts ? (int)p.channels : 0;
        const E *x = static_cast<const E *>(p.x) + n * p.x_n;
        const E *go = static_cast<const E *>(p.grad_out) + n * p.g_n;
        const E *gs =
            p.grad_sum == nullptr ? nullptr : static_cast<const E *>(p.grad_sum) + n * p.s_n;
        E *to = static_cast<E *>(p.grad_x) + (int64_t)n * p.channels;
        Steps<VEC, E> xs[R], gos[R];
        float s = 0.f, c = 0.f;
        uint32_t unused = 0;
        const auto fetch = [&](uint32_t i, Steps<VEC, E> &xb, Steps<VEC, E> &gb) {
            xb.load(x + (int64_t)i * VEC, D - (int)i * VEC);
            gb.load(go + (int64_t)i * VEC, D - (int)i * VEC);
        };
        const auto add = [&](const Steps<VEC, E> &xb, const Steps<VEC, E> &gb, uint32_t i,
                             float factor) {
            float v[VEC], g[VEC], w[VEC];
            xb.widen(v);
            gb.widen(g);
            weights(i, w);
#pragma unroll
            for (int k = 0; k < VEC; ++k) {
                v[k] *= factor;
                s = fmaf(v[k], v[k], s);
                c = fmaf(v[k], g[k] * w[k], c);
            }
        };
        const auto all_channels = [&](float factor) {
#pragma unroll
            for (int j = 0; j < R; ++j)
                if (first + j * ACROSS < blocks) add(xs[j], gos[j], first + j * ACROSS, factor);
            for (uint32_t i = first + R * ACROSS; i < blocks; i += ACROSS) {
                Steps<VEC, E> xb, gb;
                fetch(i, xb, gb);
                add(xb, gb, i, factor);
            }
            row_sums<WAVES>(s, c, unused, lds, lds_most);
        };
#pragma unroll
        for (int j = 0; j < R; ++j)
            if (first + j * ACROSS < blocks) fetch(first + j * ACROSS, xs[j], gos[j]);
        all_channels(1.f);
        float factor = 1.f;
        if (overflows<E>() && s >= kMuch) {
            factor = kDown;
            s = c = 0.f;
            all_channels(factor);
        }
        const float root = rsqrt_of(p, s, factor), r = factor * root;
        c = c * root * p.per_channel;
        const auto finish = [&](const Steps<VEC, E> &xb, const Steps<VEC, E> &gb, uint32_t i,
                                float(&total)[VEC]) {
            float v[VEC], g[VEC], w[VEC], more[VEC] = {};
            xb.widen(v);
            gb.widen(g);
            weights(i, w);
            if (gs != nullptr)
                seq::load_steps<VEC>(gs + (int64_t)i * VEC, D - (int)i * VEC, more);
#pragma unroll
            for (int k = 0; k < VEC; ++k) {
                const float xh = v[k] * r;
                total[k] += counts ? g[k] * xh : 0.f;
                v[k] = counts ? fmaf(r, fmaf(g[k], w[k], -xh * c), more[k]) : 0.f;
            }
            seq::store_steps<VEC>(to + (int64_t)i * VEC, (int)p.channels - (int)i * VEC, v);
        };
#pragma unroll
        for (int j = 0; j < R; ++j)
            if (first + j * ACROSS < blocks)
                finish(xs[j], gos[j], first + j * ACROSS, grad_weight[j]);
        for (uint32_t i = first + R * ACROSS; i < blocks; i += ACROSS) {
            Steps<VEC, E> xb, gb;
            fetch(i, xb, gb);
            float total[VEC] = {};
            const int room = (int)p.channels - (int)i * VEC;
            if (begun) seq::load_steps<VEC>(partial + (int64_t)i * VEC, room, total);
            finish(xb, gb, i, total);
            seq::store_steps<VEC>(partial + (int64_t)i * VEC, room, total);
        }
        begun = true;
    }
#pragma unroll
    for (int j = 0; j < R; ++j)
        if (first + j * ACROSS < blocks) {
            const int64_t d = (int64_t)(first + j * ACROSS) * VEC;
            seq::store_steps<VEC>(partial + d, (int)(p.channels - d), grad_weight[j]);
        }
}

// The walkers' sums in order: a workgroup takes 64 channels (and, of more than 2^26, more
// of them: a launch holds fewer than 2^32 threads), its 16 waves every 16th walker each.
struct SumParams {
    const float *partials;
    float *out;
    uint32_t walkers, channels;
};
constexpr int kSumWaves = 16;
constexpr uint32_t kSumGroups = 1u << 20;

__global__ __launch_bounds__(kSumWaves *kWave) void rms_norm_sums(SumParams p) {
    __shared__ float sums[kSumWaves][kWave];
    const uint32_t wave = threadIdx.x / kWave, lane = threadIdx.x % kWave;
    for (uint32_t first = blockIdx.x * kWave; first < p.channels; first += gridDim.x * kWave) {
        const uint32_t d = first + lane;
        float sum = 0.f;
        if (d < p.channels)
#pragma unroll 8
            for (uint32_t w = wave; w < p.walkers; w += kSumWaves)
                sum += p.partials[(int64_t)w * p.channels + d];
        __syncthreads();  // the channels before have been read
        sums[wave][lane] = sum;
        __syncthreads();
        if (wave == 0 && d < p.channels) {
            for (int w = 1; w < kSumWaves; ++w) sum += sums[w][lane];
            p.out[d] = sum;
        }
    }
}

// With no channels: the scales.
struct EmptyParams {
    float *scale;
    uint64_t count;
};

__global__ __launch_bounds__(256) void rms_norm_empty(EmptyParams p) {
    for (uint64_t i = blockIdx.x * 256ull + threadIdx.x; i < p.count; i += gridDim.x * 256ull)
        p.scale[i] = 0.f;
}

// ------------------------------------------------------------------- host side
// How a call is launched.
struct Shape {
    bool dense;
    int threads, lanes;  // time rows: THREADS and LT
    int waves;           // dense rows: WAVES
    int64_t tiles, work, groups;
};

constexpr int64_t kBackwardGroups = 512;  // workgroups that walk in the backward call
constexpr int64_t kCompute = 256;         // compute units

static Shape shape_of(const rlca_norm_call &c, bool backward) {
    Shape s = {};
    const int64_t N = c.num_seqs, D = c.channels, T = c.T;
    const int vec = (int)(16 / seq::element_bytes(c.dtype));
    const auto row = [&](const void *p, int64_t stride) {
        return p == nullptr || stride == 1 || D <= 1;
    };
    s.dense = T == 1 && row(c.x, c.x_stride_channel) &&
              (backward ? row(c.grad_out, c.grad_stride_channel) &&
                              row(c.grad_sum, c.grad_sum_stride_channel)
                        : row(c.residual, c.residual_stride_channel));
    if (s.dense) {
        // a wave a row where it holds the row and there are rows enough for the chip, or
        // one block a lane is all of it (2048 channels, bf16: one row 4.4 us against 3.9
        // with four waves, 64 rows 5.1 against 3.4, 2048 rows 8.8 against 9.4)
        s.waves = D <= kWave * vec || (D <= 4 * kWave * vec && N >= 1024) ? 1 : 4;
        s.work = N;
        const int64_t rows = 4 / s.waves;
        s.groups = (N + rows - 1) / rows;
        if (backward && s.groups > kBackwardGroups) s.groups = kBackwardGroups;
        return s;
    }
    const auto tiles = [&](int lanes) { return (T + lanes * vec - 1) / (lanes * vec); };
    // 128 bytes of a channel's steps side by side, a whole cache line (64 bytes: 78 us
    // against 58 forward and 101 against 80 backward for 8x2048 channels of 2048 steps,
    // bf16 with residual).  64 with more channels than registers hold then (4096 of 1024
    // steps: 70 against 94, and 99 against 115), or where even those make no more
    // workgroups than there are compute units, one on each: 1x2048 channels of 8192 steps,
    // 256 of them, 27.0 against 29.7, and of 8256, with two more, 38.0 against 29.4; with
    // gradients 35.6 against 41.5 and 50.8 against 39.8.  (So it is wherever rows begin:
    // 8191 steps 54.0 against 58.8, 6x1536 of 2049, 390 workgroups, 38.2 against 30.2.)
    // 16 where tiles are fewest (2048 of 512 steps: 10.8 against 13.5 and 20; not for 64 of
    // 1024: 6.5 against 4.6).
    const bool few = N * tiles(4) <= kCompute;
    s.lanes = D <= 512 ? 8 : N * tiles(4) < 64 ? 1 : D <= 2048 && !few ? 8 : 4;
    s.threads = s.lanes != 8 || D > 512 ? 1024 : D > 128 ? 512 : 256;
    s.tiles = tiles(s.lanes);
    s.work = N * s.tiles;
    s.groups = backward && s.work > kBackwardGroups ? kBackwardGroups : s.work;
    return s;
}

template <typename E, bool Q8>
static const void *forward_kernel(const Shape &s) {
    if (s.dense)
        return s.waves == 1 ? (const void *)rms_norm_dense<E, 1, 4, Q8>
                            : (const void *)rms_norm_dense<E, 4, 4, Q8>;
    return s.threads == 256 ? (const void *)rms_norm_rows<E, 256, 8, 4, Q8>
           : s.threads == 512 ? (const void *)rms_norm_rows<E, 512, 8, 8, Q8>
           : s.lanes == 8     ? (const void *)rms_norm_rows<E, 1024, 8, Q8 ? 12 : 16, Q8>
           : s.lanes == 4     ? (const void *)rms_norm_rows<E, 1024, 4, Q8 ? 12 : 16, Q8>
                              : (const void *)rms_norm_rows<E, 1024, 1, 4, Q8>;
}

// Both arrays of the backward call do not fit the registers from 1024 channels on, of
// which 1024 threads take all; as many blocks are kept as fit (8x2048 channels of 2048
// steps, bf16, alone in a row: 2 blocks a thread 67 us, 6 62).
template <typename E>
static const void *backward_kernel(const Shape &s) {
    if (s.dense)
        return s.waves == 1 ? (const void *)rms_norm_dense_backward<E, 1, 4>
                            : (const void *)rms_norm_dense_backward<E, 4, 4>;
    return s.threads == 256 ? (const void *)rms_norm_rows_backward<E, 256, 8, 4>
           : s.threads == 512 ? (const void *)rms_norm_rows_backward<E, 512, 8, 8>
           : s.lanes == 8     ? (const void *)rms_norm_rows_backward<E, 1024, 8, 6>
           : s.lanes == 4     ? (const void *)rms_norm_rows_backward<E, 1024, 4, 6>
                              : (const void *)rms_norm_rows_backward<E, 1024, 1, 2>;
}

// Workgroups are numbered in 32 bits, and their threads too.
static bool sizes_fit(const rlca_norm_call &c, bool backward) {
    if (!seq::sizes_ok(c.num_seqs, c.channels, c.T) || seq::element_bytes(c.dtype) == 0) return false;
    const Shape s = shape_of(c, backward);
    const int64_t threads = s.dense ? kRowThreads : s.threads;
    return s.work < (int64_t)1 << 31 && s.groups * threads < (int64_t)1 << 32;
}

static size_t workspace_bytes_of(const rlca_norm_call &c) {
    const Shape s = shape_of(c, true);
    const int64_t walkers = s.dense ? s.groups * (4 / s.waves) : s.groups;
    return (size_t)walkers * c.channels * sizeof(float);
}

static NormParams params_of(const rlca_norm_call &c, const Shape &s) {
    NormParams p = {};
    p.x = c.x, p.residual = c.residual, p.grad_out = c.grad_out, p.grad_sum = c.grad_sum;
    p.weight = c.weight;
    p.lengths = c.lengths;
    p.out = c.out, p.sum = c.sum, p.grad_x = c.grad_x;
    p.out8 = c.out8, p.scale = c.scale;
    p.x_n = c.x_stride_seq, p.x_d = c.x_stride_channel;
    p.r_n = c.residual_stride_seq, p.r_d = c.residual_stride_channel;
    p.g_n = c.grad_stride_seq, p.g_d = c.grad_stride_channel;
    p.s_n = c.grad_sum_stride_seq, p.s_d = c.grad_sum_stride_channel;
    p.channels = (uint32_t)c.channels;
    p.T = (int32_t)c.T;
    p.tiles = (uint32_t)(s.dense ? 1 : s.tiles);
    p.work = (uint32_t)s.work;
    p.eps = (float)c.eps;
    p.per_channel = (float)(1.0 / (double)c.channels);
    p.by_tiles = seq::fast_div(p.tiles);
    return p;
}

static rlca_status check_norm(const rlca_norm_call &c, bool backward, seq::Arrays &a) {
    if (!seq::sizes_ok(c.num_seqs, c.channels, c.T)) return RLCA_ERR_INVALID_SIZE;
    const size_t e = seq::element_bytes(c.dtype);
    if (e == 0 || !(c.eps >= 1e-30 && c.eps <= 1e30)) return RLCA_ERR_INVALID_VALUE;
    if (!sizes_fit(c, backward)) return RLCA_ERR_INVALID_SIZE;
    const int64_t N = c.num_seqs, D = c.channels, T = c.T;
    a.in(c.x, e, true, {{N, c.x_stride_seq}, {D, c.x_stride_channel}, {T, 1}});
    a.in(c.weight, 4, false, {{N * T == 0 ? 0 : D, 1}});
    a.in(c.lengths, 4, false, {{N, 1}});
    return RLCA_OK;
}

}  // namespace norm
}  // namespace rlca

using namespace rlca::norm;
using rlca::kWave;
using rlca::seq::Arrays;
using rlca::seq::element_bytes;
using rlca::seq::launch;

extern "C" {

size_t rlca_rms_norm_backward_workspace_size(const rlca_norm_call *call) {
    if (call == nullptr || !sizes_fit(*call, true)) return 0;
    return workspace_bytes_of(*call);
}

rlca_status rlca_rms_norm(const rlca_norm_call *call, hipStream_t stream) {
    if (call == nullptr) return RLCA_ERR_NULL_POINTER;
    const rlca_norm_call &c = *call;
    Arrays a;
    rlca_status st = check_norm(c, false, a);
    if (st != RLCA_OK) return st;
    const int64_t N = c.num_seqs, D = c.channels, T = c.T;
    const size_t e = element_bytes(c.dtype);
    if (N * D != 0 && T != 0 && (c.out == nullptr) == (c.out8 == nullptr))
        return c.out == nullptr ? RLCA_ERR_NULL_POINTER : RLCA_ERR_INVALID_VALUE;
    a.in(c.residual, e, false,
         {{N, c.residual_stride_seq}, {D, c.residual_stride_channel}, {T, 1}});
    a.out(c.out, e, false, {{N, D * T}, {D, T}, {T, 1}});
    a.out(c.out8, 1, false, {{N, D * T}, {D, T}, {T, 1}});
    a.out(c.scale, 4, c.out8 != nullptr, {{N, T}, {T, 1}});
    a.out(c.sum, e, c.residual != nullptr, {{N, D * T}, {D, T}, {T, 1}});
    if ((st = a.status()) != RLCA_OK || N == 0 || T == 0) return st;
    if (D == 0) {
        if (c.scale == nullptr || c.out != nullptr) return RLCA_OK;
        EmptyParams p = {c.scale, (uint64_t)N * T};
        const uint64_t blocks = (p.count + 255) / 256;
        return launch((const void *)rms_norm_empty, dim3((uint32_t)(blocks < 4096 ? blocks : 4096)),
                      256, 0, p, stream);
    }
    const Shape s = shape_of(c, false);
    NormParams p = params_of(c, s);
    const bool q8 = c.out8 != nullptr;
    const void *kernel =
        c.dtype == RLCA_F32    ? (q8 ? forward_kernel<float, true>(s) : forward_kernel<float, false>(s))
        : c.dtype == RLCA_BF16 ? (q8 ? forward_kernel<__bf16, true>(s)
                                     : forward_kernel<__bf16, false>(s))
                               : (q8 ? forward_kernel<_Float16, true>(s)
                                     : forward_kernel<_Float16, false>(s));
    return launch(kernel, dim3((uint32_t)s.groups), s.dense ? kRowThreads : s.threads, 0, p, stream);
}

rlca_status rlca_rms_norm_backward(const rlca_norm_call *call, void *workspace,
                                   size_t workspace_bytes, hipStream_t stream) {
    if (call == nullptr) return RLCA_ERR_NULL_POINTER;
    const rlca_norm_call &c = *call;
    Arrays a;
    rlca_status st = check_norm(c, true, a);
    if (st != RLCA_OK) return st;
    const int64_t N = c.num_seqs, D = c.channels, T = c.T;
    const size_t e = element_bytes(c.dtype), need = workspace_bytes_of(c);
    a.in(c.grad_out, e, true, {{N, c.grad_stride_seq}, {D, c.grad_stride_channel}, {T, 1}});
    a.in(c.grad_sum, e, false,
         {{N, c.grad_sum_stride_seq}, {D, c.grad_sum_stride_channel}, {T, 1}});
    a.out(c.grad_x, e, true, {{N, D * T}, {D, T}, {T, 1}});
    a.out(c.grad_weight, 4, false, {{D, 1}});
    a.out(workspace, 4, need != 0, {{(int64_t)(need / 4), 1}});
    if ((st = a.status()) != RLCA_OK) return st;
    if (workspace_bytes < need) return RLCA_ERR_INVALID_SIZE;
    if (D == 0) return RLCA_OK;
    uint32_t walkers = 0;
    if (N * T != 0) {
        const Shape s = shape_of(c, true);
        NormParams p = params_of(c, s);
        p.partials = static_cast<float *>(workspace);
        walkers = (uint32_t)(s.dense ? s.groups * (4 / s.waves) : s.groups);
        const void *kernel = c.dtype == RLCA_F32    ? backward_kernel<float>(s)
                             : c.dtype == RLCA_BF16 ? backward_kernel<__bf16>(s)
                                                    : backward_kernel<_Float16>(s);
        st = launch(kernel, dim3((uint32_t)s.groups), s.dense ? kRowThreads : s.threads, 0, p,
                    stream);
        if (st != RLCA_OK) return st;
    }
    if (c.grad_weight == nullptr) return RLCA_OK;
    SumParams sum = {static_cast<const float *>(workspace), c.grad_weight, walkers, (uint32_t)D};
    const uint32_t groups = (uint32_t)((D + kWave - 1) / kWave);
    return launch((const void *)rms_norm_sums, dim3(groups < kSumGroups ? groups : kSumGroups),
                  kSumWaves * kWave, 0, sum, stream);
}

}  // extern "C"
