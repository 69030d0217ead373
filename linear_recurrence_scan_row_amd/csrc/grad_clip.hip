// grad_clip.hip -- the global norm of many gradient tensors, and the gradients
// scaled to at most max_norm.
//
// Bound by memory: every element is read for the norm, and read and written
// again for the scaling, which cannot begin before the last element was seen.
// The scaling goes through the list from its end: what the norm read last, up
// to 256 MB, still lies in the last-level cache.  Measured: 60 bf16 tensors of
// 400 M elements 164 us for the norm (4.9 TB/s) and 288 for the scaling (5.6
// TB/s); 26 fp32 tensors of 400 K elements 6.5 and 4.4 us.
// The tensors' addresses travel as kernel arguments, so nothing is copied to the
// device; one launch takes up to kMaxTensors tensors as a list of chunks of
// kChunk elements, so many small tensors fill the chip like one large one.
#include <algorithm>

#include "kernels.hpp"
#include "seq.hpp"

namespace rlca {
namespace clip {

constexpr int kThreads = 256;
constexpr int kPerThread = 16;
constexpr int kChunk = kThreads * kPerThread;
constexpr int kMaxTensors = 96;  // 32 bytes each, of 4 KB kernel arguments
constexpr uint32_t kClipGrid = 2048;

// The workspace: ticket counters, one partial sum per workgroup, then the
// running total of the launches before and the scale.
struct Head {
    double total;
    double scale;
};
constexpr size_t kHeadAt = kTicketBytes + kClipGrid * sizeof(double);
static_assert(kHeadAt + 128 == RLCA_CLIP_WORKSPACE_BYTES, "the header's workspace size");

struct Tensor {
    const void *data;
    void *out;
    uint64_t count;
    uint32_t first_chunk;
    int32_t dtype;
};

struct Launch {
    Tensor tensors[kMaxTensors];
    uint32_t num_tensors, chunks;
    double *partials;
    Head *head;
    double *norm;
    double max_norm, eps;
    int32_t first, last;  // of the launches of one call
};

// The tensor that holds a chunk: the last one whose first chunk is not after it.
__device__ __forceinline__ uint32_t tensor_of(const Launch &l, uint32_t chunk) {
    uint32_t lo = 0, hi = l.num_tensors;
    while (hi - lo > 1) {
        const uint32_t mid = (lo + hi) / 2;
        if (l.tensors[mid].first_chunk <= chunk)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

// A thread's elements of a chunk: kBlocks blocks of 16 bytes, a workgroup's
// next to each other.
template <typename E>
struct Blocks {
    static constexpr int kElems = 16 / sizeof(E);
    static constexpr int kBlocks = kPerThread / kElems;
};

template <typename E, typename F>
__device__ __forceinline__ void for_blocks(const Tensor &t, uint32_t chunk, F f) {
    constexpr int K = Blocks<E>::kElems, N = Blocks<E>::kBlocks;
    const uint64_t begin = (uint64_t)chunk * kChunk;
    const int64_t left = (int64_t)(t.count - begin);
    float v[N][K];
#pragma unroll
    for (int b = 0; b < N; ++b) {
        const int at = (b * kThreads + (int)threadIdx.x) * K;
        const int64_t n = left - at;
        seq::load_steps<K>(static_cast<const E *>(t.data) + begin + at, n < K ? (int)(n < 0 ? 0 : n) : K,
                           v[b]);
    }
#pragma unroll
    for (int b = 0; b < N; ++b) {
        const int at = (b * kThreads + (int)threadIdx.x) * K;
        const int64_t n = left - at;
        f(v[b], begin + at, n < K ? (int)(n < 0 ? 0 : n) : K);
    }
}

// Squares and sums in fp64: a float32 square overflows from 1.8e19 on and is
// 0 below 1e-23, and fp64 sums of 10^9 terms keep ten digits.
template <typename E>
__device__ __forceinline__ double chunk_square_sum(const Tensor &t, uint32_t chunk) {
    double sum = 0.0;
    for_blocks<E>(t, chunk, [&](const float(&v)[Blocks<E>::kElems], uint64_t, int) {
#pragma unroll
        for (int k = 0; k < Blocks<E>::kElems; ++k) sum = fma((double)v[k], (double)v[k], sum);
    });
    return sum;
}

__global__ __launch_bounds__(kThreads) void grad_norm(Launch l) {
    double sum = 0.0;
    for (uint32_t c = blockIdx.x; c < l.chunks; c += gridDim.x) {
        const Tensor &t = l.tensors[tensor_of(l, c)];
        const uint32_t chunk = c - t.first_chunk;
        sum += t.dtype == RLCA_F32    ? chunk_square_sum<float>(t, chunk)
               : t.dtype == RLCA_BF16 ? chunk_square_sum<__bf16>(t, chunk)
                                      : chunk_square_sum<_Float16>(t, chunk);
    }
    double unused = 0.0;
    workgroup_sum2<kThreads / kWave>(sum, unused);
    Head *head = l.head;
    double *norm = l.norm;
    const double max_norm = l.max_norm, eps = l.eps;
    const bool first = l.first != 0, last = l.last != 0;
    finish_in_last_workgroup<kThreads, 1>(l.partials, sum, 0.0, [=](double s, double) {
        const double total = first ? s : load_coherent(&head->total) + s;
        store_coherent(&head->total, total);
        if (!last) return;
        const double n = sqrt(total), scale = max_norm / (n + eps);
        norm[0] = n;
        // a NaN stays one
        store_coherent(&head->scale, n == 0.0 || scale >= 1.0 ? 1.0 : scale);
    });
}

// A value times the scale, which is rounded to fp32 once.  Where fp32 would hold it
// with fewer digits, or as 0 (a norm of 1e38 and more times max_norm: large gradients
// that come out in range all the same), the product is taken in fp64.
struct Scale {
    double exact;
    float rounded;
    __device__ __forceinline__ explicit Scale(double s) : exact(s), rounded((float)s) {}
    __device__ __forceinline__ bool wide() const { return exact > 0.0 && exact < 0x1p-126; }
};

template <typename E>
__device__ __forceinline__ void scale_chunk(const Tensor &t, uint32_t chunk, const Scale &scale) {
    for_blocks<E>(t, chunk, [&](float(&v)[Blocks<E>::kElems], uint64_t at, int n) {
        if (scale.wide())
#pragma unroll
            for (int k = 0; k < Blocks<E>::kElems; ++k) v[k] = (float)((double)v[k] * scale.exact);
        else
#pragma unroll
            for (int k = 0; k < Blocks<E>::kElems; ++k) v[k] *= scale.rounded;
        seq::store_steps<Blocks<E>::kElems>(static_cast<E *>(t.out) + at, n, v);
    });
}

__global__ __launch_bounds__(kThreads) void grad_scale(Launch l) {
    const Scale scale(load_coherent(&l.head->scale));
    for (uint32_t i = blockIdx.x; i < l.chunks; i += gridDim.x) {
        const uint32_t c = l.chunks - 1 - i;
        const Tensor &t = l.tensors[tensor_of(l, c)];
        if (scale.rounded == 1.f && t.out == t.data) continue;  // nothing changes
        const uint32_t chunk = c - t.first_chunk;
        if (t.dtype == RLCA_F32)
            scale_chunk<float>(t, chunk, scale);
        else if (t.dtype == RLCA_BF16)
            scale_chunk<__bf16>(t, chunk, scale);
        else
            scale_chunk<_Float16>(t, chunk, scale);
    }
}

// ------------------------------------------------------------------- host side
struct Range {
    uintptr_t begin, end;
    uint32_t id;  // of the call's ranges, for an order among equal addresses
    bool written;
    bool operator<(const Range &o) const {
        return begin != o.begin ? begin < o.begin : id < o.id;
    }
};

// The call's ranges in order of their addresses, kAtOnce at a time: the smallest of
// those after the last batch's, kept in a heap on the stack (each batch goes over all
// ranges again, and the host allocates nothing).
class Ordered {
  public:
    // Whether the sweep so far has met an overlap of a written range.
    bool overlap() const { return overlap_; }
    // Offers one of the call's ranges to the batch.
    void offer(const Range &r) {
        if (started_ && !(last_ < r)) return;
        if (count_ < kAtOnce) {
            batch_[count_++] = r;
            if (count_ == kAtOnce) std::make_heap(batch_, batch_ + kAtOnce);
        } else if (r < batch_[0]) {
            std::pop_heap(batch_, batch_ + kAtOnce);
            batch_[kAtOnce - 1] = r;
            std::push_heap(batch_, batch_ + kAtOnce);
        }
    }
    // Sweeps the batch; false: it was the last.
    bool sweep() {
        std::sort(batch_, batch_ + count_);
        for (size_t i = 0; i < count_; ++i) {
            const Range &r = batch_[i];
            if (r.begin < (r.written ? any_ : written_)) overlap_ = true;
            any_ = std::max(any_, r.end);
            if (r.written) written_ = std::max(written_, r.end);
        }
        const bool more = count_ == kAtOnce;
        if (more) last_ = batch_[kAtOnce - 1];
        started_ = true;
        count_ = 0;
        return more;
    }

  private:
    static constexpr size_t kAtOnce = 2048;  // 48 KB
    Range batch_[kAtOnce];
    size_t count_ = 0;
    Range last_ = {};
    bool started_ = false, overlap_ = false;
    uintptr_t any_ = 0, written_ = 0;  // the ends of the ranges so far
};

static rlca_status check_tensors(const rlca_grad_tensor *tensors, int64_t n, bool scaled,
                                 double *norm, void *workspace) {
    for (int64_t i = 0; i < n; ++i) {
        const rlca_grad_tensor &t = tensors[i];
        const size_t e = seq::element_bytes(t.dtype);
        if (t.count < 0 || t.count >= (int64_t)1 << 43) return RLCA_ERR_INVALID_SIZE;
        if (e == 0) return RLCA_ERR_INVALID_VALUE;
        if (t.count == 0) continue;
        if (t.data == nullptr || (scaled && t.out == nullptr)) return RLCA_ERR_NULL_POINTER;
        if ((uintptr_t)t.data % e != 0 || (scaled && (uintptr_t)t.out % e != 0))
            return RLCA_ERR_MISALIGNED;
    }
    // no written range may overlap another range
    Ordered ranges;
    const uint32_t ends = 2 * (uint32_t)n;
    do {
        for (int64_t i = 0; i < n; ++i) {
            const rlca_grad_tensor &t = tensors[i];
            if (t.count == 0) continue;
            const size_t bytes = (size_t)t.count * seq::element_bytes(t.dtype);
            const uintptr_t data = (uintptr_t)t.data, out = (uintptr_t)t.out;
            ranges.offer({data, data + bytes, 2 * (uint32_t)i, scaled && out == data});
            if (scaled && out != data)
                ranges.offer({out, out + bytes, 2 * (uint32_t)i + 1, true});
        }
        ranges.offer({(uintptr_t)norm, (uintptr_t)norm + 8, ends, true});
        ranges.offer({(uintptr_t)workspace, (uintptr_t)workspace + RLCA_CLIP_WORKSPACE_BYTES,
                      ends + 1, true});
    } while (ranges.sweep() && !ranges.overlap());
    return ranges.overlap() ? RLCA_ERR_ALIASING : RLCA_OK;
}

// Fills `l` with a launch's worth of the tensors in [*begin, *end), from the
// front or the back, and takes them out of that range; empty tensors are
// dropped.  (A tensor has fewer than 2^43 elements, 2^31 chunks.)
static void fill(Launch *l, const rlca_grad_tensor *tensors, int64_t *begin, int64_t *end,
                 bool from_back) {
    int64_t first = *begin, last = *end;  // the launch's tensors
    uint32_t count = 0;
    uint64_t chunks = 0;
    for (int64_t left = *end - *begin; left > 0; --left) {
        const int64_t i = from_back ? *end - 1 : *begin;
        const uint64_t c = ((uint64_t)tensors[i].count + kChunk - 1) / kChunk;
        if (c != 0 && (count == (uint32_t)kMaxTensors || (count != 0 && chunks + c > 1ull << 31)))
            break;
        if (from_back)
            --*end;
        else
            ++*begin;
        if (c != 0) ++count;
        chunks += c;
    }
    if (from_back)
        first = *end;
    else
        last = *begin;
    l->num_tensors = 0;
    l->chunks = 0;
    for (int64_t i = first; i < last; ++i) {
        const rlca_grad_tensor &t = tensors[i];
        if (t.count == 0) continue;
        l->tensors[l->num_tensors++] = {t.data, t.out, (uint64_t)t.count, l->chunks, t.dtype};
        l->chunks += (uint32_t)(((uint64_t)t.count + kChunk - 1) / kChunk);
    }
}

}  // namespace clip
}  // namespace rlca

using rlca::kTicketBytes;
using namespace rlca::clip;

extern "C" rlca_status rlca_clip_grad_norm(const rlca_grad_tensor *tensors, int64_t num_tensors,
                                           double max_norm, double eps, double *norm,
                                           void *workspace, size_t workspace_bytes,
                                           hipStream_t stream) {
    if (num_tensors < 0 || num_tensors > (1 << 24)) return RLCA_ERR_INVALID_SIZE;
    if (!(max_norm >= 0.0) || !(eps >= 0.0 && isfinite(eps))) return RLCA_ERR_INVALID_VALUE;
    if ((tensors == nullptr && num_tensors != 0) || norm == nullptr || workspace == nullptr)
        return RLCA_ERR_NULL_POINTER;
    if ((uintptr_t)norm % 8 != 0 || (uintptr_t)workspace % 8 != 0) return RLCA_ERR_MISALIGNED;
    if (workspace_bytes < RLCA_CLIP_WORKSPACE_BYTES) return RLCA_ERR_INVALID_SIZE;
    const bool scaled = !isinf(max_norm);
    rlca_status st = check_tensors(tensors, num_tensors, scaled, norm, workspace);
    if (st != RLCA_OK) return st;
    char *ws = static_cast<char *>(workspace);
    Launch l;
    l.partials = reinterpret_cast<double *>(ws + kTicketBytes);
    l.head = reinterpret_cast<Head *>(ws + kHeadAt);
    l.norm = norm;
    l.max_norm = max_norm;
    l.eps = eps;
    for (int pass = 0; pass < (scaled ? 2 : 1); ++pass) {
        int64_t begin = 0, end = num_tensors;
        l.first = 1;
        do {
            fill(&l, tensors, &begin, &end, pass == 1);
            l.last = begin == end;
            if (l.chunks != 0 || pass == 0) {
                const uint32_t grid = l.chunks < 1 ? 1 : l.chunks < kClipGrid ? l.chunks : kClipGrid;
                st = rlca::seq::launch(
                    pass == 0 ? (const void *)grad_norm : (const void *)grad_scale, dim3(grid),
                    kThreads, 0, l, stream);
                if (st != RLCA_OK) return st;
            }
            l.first = 0;
        } while (begin < end);
    }
    return RLCA_OK;
}
