// seq.hpp -- what the sequence-model kernels share (seq_conv.hip, seq_scan.hip,
// seq_scan_backward.hip, seq_step.hip): access to rows of stored steps, the
// activations, episode starts, and the host's argument checks.
#pragma once

#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <type_traits>

#include "rlca.h"
#include "scan_core.hpp"

namespace rlca {
namespace seq {

// ----------------------------------------------------------------- device side
// K consecutive steps from p, of which the first n exist (n may be <= 0 or
// above K); the others read as 0 and are not accessed.  Rows may start at any
// element: gfx950 loads and stores 16 bytes at any address, so a whole block
// is one access whatever T is, and only a row's last block goes step by step.
template <int K, typename E>
__device__ __forceinline__ void load_steps(const E *p, int n, float (&v)[K]) {
    typedef E block __attribute__((ext_vector_type(K)));
    if (n >= K) {
        block b;
        __builtin_memcpy(&b, p, sizeof b);
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] = (float)b[k];
    } else {
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] = k < n ? (float)p[k] : 0.f;
    }
}

// As load_steps, in the storage type: loads that are issued long before their
// use keep 16-bit steps in half the registers.
template <int K, typename E>
struct Steps {
    typedef E block __attribute__((ext_vector_type(K)));
    block b;
    __device__ __forceinline__ void load(const E *p, int n) {
        if (n >= K) {
            __builtin_memcpy(&b, p, sizeof b);
        } else {
#pragma unroll
            for (int k = 0; k < K; ++k) b[k] = k < n ? p[k] : (E)0.f;
        }
    }
    __device__ __forceinline__ void widen(float (&v)[K]) const {
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] = (float)b[k];
    }
};

// One rounding, to nearest even, from fp32 to the storage type.
template <int K, typename E>
__device__ __forceinline__ void store_steps(E *p, int n, const float (&v)[K]) {
    typedef E block __attribute__((ext_vector_type(K)));
    if (n >= K) {
        block b;
#pragma unroll
        for (int k = 0; k < K; ++k) b[k] = (E)v[k];
        __builtin_memcpy(p, &b, sizeof b);
    } else {
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (k < n) p[k] = (E)v[k];
    }
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLog2eLow = 1.925963033500913e-08f;  // log2(e) - (float)log2(e)

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// h 2^x, where 2^x alone may leave float32's range: 0 stays 0, and what is in
// range comes out.  2^x is split at x's whole part, towards 0, so that the
// product with the rest (in [1, 2) for a growth, (1/2, 1] for a decay) rounds
// as h 2^x does.  Beyond 2^300 every h but 0 is infinite, and below 2^-300 0.
__device__ __forceinline__ float times_exp2(float h, float x) {
    x = x > 300.f ? 300.f : x < -300.f ? -300.f : x;  // a NaN stays one
    const float whole = truncf(x);
    return ldexpf(h * exp2_fast(x - whole), (int)whole);
}

// 1 / (1 + exp(-x)); 0 and 1 at the infinities.
__device__ __forceinline__ float sigmoid(float x) {
    return __builtin_amdgcn_rcpf(1.f + exp2_fast(-x * kLog2e));
}

// silu(x) = x sigmoid(x) and its derivative sig (1 + x (1 - sig)).
__device__ __forceinline__ float silu(float x) { return x * sigmoid(x); }
__device__ __forceinline__ float silu_slope(float x, float sig) {
    return sig * (1.f + x * (1.f - sig));
}

// softplus(x) = log(1 + e^x) = max(x, 0) + log1p(e), e = exp(-|x|) in (0, 1].
// A step size of 1e-3 is log1p(1e-3), where log(1 + e) alone would keep four
// digits: with w the rounded 1 + e, log1p(e) = log(w) + (e - (w - 1)) / w, and
// the 1 / w is left out, since what it scales is at most half a step of w.  e's
// exponent is formed with the low part of log2(e), so that its error does not
// grow with |x|.  Relative error at most 6 x 2^-24.  -|x| ends at -200, where e
// is 0: a step masked by -infinity or the lowest value has size 0, not NaN.
__device__ __forceinline__ float softplus(float x) {
    const float y = fmaxf(-fabsf(x), -200.f);
    const float t = y * kLog2e;
    const float low = fmaf(y, kLog2e, -t) + y * kLog2eLow;
    const float e = exp2_fast(t) * fmaf(low, 0.6931471805599453f, 1.f);
    const float w = 1.f + e;
    const float l = fmaf(__builtin_amdgcn_logf(w), 0.6931471805599453f, e - (w - 1.f));
    return (x < 0.f ? 0.f : x) + l;  // a NaN stays one
}

// Eight flags of a row of T from step `first` on, which may begin before the
// row or end past it (those count as 0).  One load, moved inside the row where
// necessary and its bits moved back; bits() is apart from load() so that the
// load can be issued long before its use.
struct FlagWindow {
    uint64_t w;
    int d;
    __device__ __forceinline__ void load(const uint8_t *flags, int first, int T) {
        if (T >= 8) {
            const int at = first < 0 ? 0 : first > T - 8 ? T - 8 : first;
            d = at - first;
            __builtin_memcpy(&w, flags + at, 8);
        } else {
            w = 0;
            d = 0;
            for (int k = 0; k < 8; ++k)
                if (first + k >= 0 && first + k < T) w |= (uint64_t)flags[first + k] << (8 * k);
        }
    }
    // Bit k: the flag at first + k is set (k < K).
    template <int K>
    __device__ __forceinline__ uint32_t bits() const {
        // nonzero bytes -> their top bit -> one bit each, in order
        uint64_t x = w | ((w & 0x7f7f7f7f7f7f7f7full) + 0x7f7f7f7f7f7f7f7full);
        x = (x >> 7) & 0x0101010101010101ull;
        const uint32_t found = (uint32_t)((x * 0x0102040810204080ull) >> 56);
        const uint32_t at = d >= 8 || d <= -8 ? 0u : d >= 0 ? found << d : found >> -d;
        return at & ((1u << K) - 1);
    }
};

// Bit k of the result: an episode starts at step t0 + k (k < K <= 8), from a
// row of T flags.  AFTER_DONE: a flag at t - 1 makes t a start.
template <int K>
__device__ __forceinline__ uint32_t start_bits(const uint8_t *flags, int t0, int T, int after_done) {
    FlagWindow f;
    f.load(flags, t0 - after_done, T);
    return f.bits<K>();
}

__device__ __forceinline__ bool is_start(const uint8_t *flags, int t, int T, int after_done) {
    const int f = t - after_done;
    return f >= 0 && f < T && flags[f] != 0;
}

// Number of a row's steps that count.
__device__ __forceinline__ int row_end(const int32_t *lengths, uint32_t n, int T) {
    if (lengths == nullptr) return T;
    const int l = lengths[n];
    return l < 0 ? 0 : l > T ? T : l;
}

// ------------------------------------------------------------------- host side
// n / d for n < 2^31: a multiplication by the rounded-up reciprocal and a
// shift.  With 2^s >= d and m = ceil(2^(31+s) / d) < 2^32, m exceeds
// 2^(31+s) / d by less than 1, so n m / 2^(31+s) exceeds n / d by less than
// 2^31 / 2^(31+s) <= 1 / d: the quotient is exact.
struct FastDiv {
    uint32_t m, shift;
    __device__ __forceinline__ uint32_t div(uint32_t n) const {
        return (uint32_t)(((uint64_t)n * m) >> shift);
    }
};

inline FastDiv fast_div(uint32_t d) {
    uint32_t s = 0;
    while (((uint64_t)1 << s) < d) ++s;
    return FastDiv{(uint32_t)((((uint64_t)1 << (31 + s)) + d - 1) / d), 31 + s};
}

inline size_t element_bytes(int dtype) {
    return dtype == RLCA_F32 ? 4 : dtype == RLCA_BF16 || dtype == RLCA_F16 ? 2 : 0;
}

// The byte range that a strided array of up to four dimensions covers.
// Dimensions of size 0 cover nothing.  false: a negative stride, or a range
// that does not fit 62 bits.
struct Dim {
    int64_t size, stride;
};

inline bool covered(const Dim *dims, int n, size_t elem, size_t *bytes) {
    unsigned __int128 last = 0;
    *bytes = 0;
    for (int i = 0; i < n; ++i) {
        if (dims[i].size == 0) return true;
        if (dims[i].size < 0 || (dims[i].stride < 0 && dims[i].size > 1)) return false;
        if (dims[i].size > 1)
            last += (unsigned __int128)(dims[i].size - 1) * (uint64_t)dims[i].stride;
        if (last >= ((unsigned __int128)1 << 59)) return false;
    }
    *bytes = ((size_t)last + 1) * elem;
    return true;
}

// Collects a call's arrays and checks them together: required pointers,
// alignment, and that no output overlaps an input or another output.  The
// first error of each kind is kept, and status() returns them in the order
// in which the other entry points check.
class Arrays {
  public:
    void in(const void *p, size_t elem, bool required, const Dim *dims, int n) {
        add(p, elem, required, dims, n, false);
    }
    void out(const void *p, size_t elem, bool required, const Dim *dims, int n) {
        add(p, elem, required, dims, n, true);
    }
    template <int N>
    void in(const void *p, size_t elem, bool required, const Dim (&dims)[N]) {
        add(p, elem, required, dims, N, false);
    }
    template <int N>
    void out(const void *p, size_t elem, bool required, const Dim (&dims)[N]) {
        add(p, elem, required, dims, N, true);
    }
    rlca_status status() const {
        if (bad_size_) return RLCA_ERR_INVALID_SIZE;
        if (null_) return RLCA_ERR_NULL_POINTER;
        if (misaligned_) return RLCA_ERR_MISALIGNED;
        for (int i = 0; i < count_; ++i)
            for (int j = 0; j < count_; ++j) {
                if (i == j || !spans_[i].written || (spans_[j].written && j < i)) continue;
                const uintptr_t a = spans_[i].p, b = spans_[j].p;
                if (a < b + spans_[j].bytes && b < a + spans_[i].bytes) return RLCA_ERR_ALIASING;
            }
        return RLCA_OK;
    }

  private:
    struct Span {
        uintptr_t p;
        size_t bytes;
        bool written;
    };
    void add(const void *p, size_t elem, bool required, const Dim *dims, int n, bool written) {
        size_t bytes;
        if (!covered(dims, n, elem, &bytes)) {
            bad_size_ = true;
            return;
        }
        if (bytes == 0) return;
        if (p == nullptr) {
            if (required) null_ = true;
            return;
        }
        if ((uintptr_t)p % elem != 0) misaligned_ = true;
        spans_[count_++] = {(uintptr_t)p, bytes, written};
    }
    Span spans_[32];
    int count_ = 0;
    bool bad_size_ = false, null_ = false, misaligned_ = false;
};

// Sizes that every call of this kind checks: false for an invalid one.
inline bool sizes_ok(int64_t num_seqs, int64_t channels, int64_t T) {
    return num_seqs >= 0 && channels >= 0 && T >= 0 && T <= RLCA_MAX_T &&
           num_seqs < ((int64_t)1 << 31) && channels < ((int64_t)1 << 31) &&
           num_seqs * channels < ((int64_t)1 << 31);
}

template <typename Params>
inline rlca_status launch(const void *kernel, dim3 grid, uint32_t threads, size_t lds,
                          Params &params, hipStream_t stream) {
    void *args[] = {&params};
    const hipError_t e = hipLaunchKernel(kernel, grid, dim3(threads), args, lds, stream);
    return e == hipSuccess ? RLCA_OK : RLCA_ERR_HIP;
}

}  // namespace seq
}  // namespace rlca
