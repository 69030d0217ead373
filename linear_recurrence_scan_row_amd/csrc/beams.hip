// beams.hip -- a beam search's selection over beams and vocabulary, and the
// reordering of the states that the beams keep in pools.
//
// Selection: total = score_b + (logit_bv - log sum_v exp(logit_bv)), the best `picks`
// of beams * vocab.  Bound by reading the logits once, beside the exponentials.  A
// workgroup takes a chunk of a beam's vocabulary in registers, and leaves the sum of
// its exponentials and its best logits: the K-th largest of the threads' own largest
// logits is a bound that at least K logits reach, and few more than K do, so only
// those are ranked.  A second launch forms the beams' sums and takes the best of the
// chunks' best, in float64.  A thread's exponentials and their sum, of up to 24, are
// float32: at most 2e-6 off, relative, in all 24 roundings' worst case, and about 1e-8
// over a beam's threads, so only beams whose totals lie that close can change places.
// (Exponentials in float64: 64 searches of 8 beams and 100003 tokens, bf16, 55 us for 29.)
//
// Reordering: bound by the states that have to move.  A parent's first child keeps its
// place, so only further children's states are copied, to the places of beams without
// children, which nothing reads: no order of copies matters.  Measured: 32 searches of 8
// beams with 18 pools 56 us (306 MB, 5.4 TB/s; the same places in every call, so part of
// it comes from the last-level cache); one with 2 pools 3.6.
#include "seq.hpp"

namespace rlca {
namespace beams {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;
constexpr int kVec = 8;          // neighbouring logits of a thread
constexpr int kRanked = kThreads;  // logits that are ranked, one a thread
constexpr int kHeld = 80;          // threads whose logits are looked through for those
constexpr float kNear = 0x1p22f;   // logits whose products with log2(e) are rounded by <= 1/4

struct Best {
    float logit;
    int32_t token;  // -1: none
};

// What a chunk leaves: its largest logit, and the sum of exp(logit - largest).
struct ChunkSum {
    double sum;
    float most;
    float unused;
};

struct SelectParams {
    const void *logits;
    const float *scores;
    const uint8_t *finished;
    float *out_scores;
    int32_t *out_tokens, *out_parents;
    ChunkSum *sums;  // [searches][beams][chunks]
    Best *best;      // [searches][beams][chunks][picks]
    int64_t by_search, by_beam;
    uint32_t searches, beams, vocab, picks, chunks;
    int32_t pad_token;
    seq::FastDiv by_chunks, by_beams, by_each, by_vocab;  // each: chunks * picks
};

// A beam whose logits count: not finished, and of a finite score.
__device__ __forceinline__ bool reads_logits(const SelectParams &p, uint32_t row) {
    return fabsf(p.scores[row]) < INFINITY && (p.finished == nullptr || p.finished[row] == 0);
}

// Order of float32 values as integers.
__device__ __forceinline__ uint32_t order_of(float x) {
    const uint32_t u = __builtin_bit_cast(uint32_t, x);
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t order) {
    const uint32_t u = order & 0x80000000u ? order ^ 0x80000000u : ~order;
    return __builtin_bit_cast(float, u);
}

// The order of candidates of one beam: by logit, and the lower token of equal ones
// first (-0 equals 0).  No two are alike; 0 is none.
__device__ __forceinline__ uint64_t key_of(float logit, uint32_t token) {
    return (uint64_t)order_of(logit + 0.f) << 32 | (uint32_t)~token;
}

__device__ __forceinline__ uint64_t wave_most(uint64_t x) {
#pragma unroll
    for (int m = 1; m < kWave; m <<= 1) {
        const uint64_t y = (uint64_t)(uint32_t)__shfl_xor((int)(x >> 32), m) << 32 |
                           (uint32_t)__shfl_xor((int)x, m);
        x = y > x ? y : x;
    }
    return x;
}

// A bound that at least K of the workgroup's kThreads values reach, and few more: the
// K-th largest without its last LEFT bits, bit by bit, four values a lane of one wave.
template <int LEFT>
__device__ __forceinline__ uint32_t kth_largest(const uint32_t *values, uint32_t K) {
    uint32_t v[kThreads / kWave];
#pragma unroll
    for (int j = 0; j < kThreads / kWave; ++j) v[j] = values[j * kWave + threadIdx.x % kWave];
    uint32_t bound = 0;
    for (int bit = 31; bit >= LEFT; --bit) {
        const uint32_t trial = bound | 1u << bit;
        uint32_t count = 0;
#pragma unroll
        for (int j = 0; j < kThreads / kWave; ++j)
            count += __builtin_popcountll(__builtin_amdgcn_ballot_w64(v[j] >= trial));
        if (count >= K) bound = trial;
        if (count == K) break;
    }
    return bound;
}

// BLOCKS blocks of kVec logits a thread.
template <typename E, int BLOCKS>
__global__ __launch_bounds__(kThreads) void beam_chunks(SelectParams p) {
    constexpr int kOwn = kVec * BLOCKS;
    __shared__ uint32_t most_of[kThreads];
    __shared__ double sums[kWaves];
    __shared__ float mosts[kWaves];
    __shared__ uint64_t ranked[kRanked];
    // the logits of threads that reach the bound, and whose they are
    __shared__ __attribute__((aligned(16))) float held[kHeld][kOwn];
    __shared__ uint32_t holders[kHeld];
    __shared__ uint32_t count, hits, bound;
    constexpr uint32_t kChunk = kThreads * kOwn;
    const uint32_t row = p.by_chunks.div(blockIdx.x), chunk = blockIdx.x - row * p.chunks;
    if (!reads_logits(p, row)) return;
    const uint32_t search = p.by_beams.div(row), beam = row - search * p.beams;
    const uint32_t tid = threadIdx.x, wave = tid / kWave;
    const uint32_t first = chunk * kChunk + tid * kVec;
    const E *logits = static_cast<const E *>(p.logits) + search * p.by_search + beam * p.by_beam;
    if (tid == 0) count = hits = 0;
    // element e of thread t's
    const auto token_of = [&](uint32_t t, uint32_t e) {
        return chunk * kChunk + t * kVec + e / kVec * (kThreads * kVec) + e % kVec;
    };

    float x[BLOCKS][kVec];
#pragma unroll
    for (int j = 0; j < BLOCKS; ++j) {
        const uint32_t t = first + j * (kThreads * kVec);
        const int n = t >= p.vocab ? 0 : p.vocab - t < (uint32_t)kVec ? (int)(p.vocab - t) : kVec;
        seq::load_steps<kVec>(logits + t, n, x[j]);
        if (n < kVec)
#pragma unroll
            for (int k = 0; k < kVec; ++k)
                if (k >= n) x[j][k] = -INFINITY;
    }
    // the thread's largest, and its sum of exponentials from there (a NaN or +infinity
    // makes that sum NaN): 2^(x log2(e) - from), where `low`, what the product for `from`
    // was rounded by, is put right in the sum.  `low` grows with the largest, and is at most
    // 1/4 up to 2^22; further out, where 2^low would leave float32's range, and for
    // infinities, the difference is formed first, an instruction more a logit.
    float most = -INFINITY;
#pragma unroll
    for (int j = 0; j < BLOCKS; ++j)
#pragma unroll
        for (int k = 0; k < kVec; ++k) most = fmaxf(most, x[j][k]);
    const float top = fmaxf(fminf(most, kNear), -kNear);
    const float from = top * seq::kLog2e, low = fmaf(top, seq::kLog2e, -from);
    float sum = 0.f;
    if (most == top) {
#pragma unroll
        for (int j = 0; j < BLOCKS; ++j)
#pragma unroll
            for (int k = 0; k < kVec; ++k)
                sum += seq::exp2_fast(fmaf(x[j][k], seq::kLog2e, -from));
        sum *= seq::exp2_fast(-low);
    } else {
        const float base = most == -INFINITY ? 0.f : most;
#pragma unroll
        for (int j = 0; j < BLOCKS; ++j)
#pragma unroll
            for (int k = 0; k < kVec; ++k) sum += seq::exp2_fast((x[j][k] - base) * seq::kLog2e);
    }
    most_of[tid] = order_of(most);
    float all = most;
#pragma unroll
    for (int m = 1; m < kWave; m <<= 1) all = fmaxf(all, __shfl_xor(all, m));
    if (tid % kWave == 0) mosts[wave] = all;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWaves; ++w) all = fmaxf(all, mosts[w]);
    if (wave == 0) {
        const uint32_t b = kth_largest<16>(most_of, p.picks);
        if (tid == 0) bound = b;
    }
    // the threads' sums from the chunk's largest, in float64
    double total = sum;
    if (most > -INFINITY && sum == sum) total *= (double)seq::exp2_fast((most - all) * seq::kLog2e);
#pragma unroll
    for (int m = 1; m < kWave; m <<= 1) total += __shfl_xor(total, m);
    if (tid % kWave == 0) sums[wave] = total;
    __syncthreads();
    const int64_t out = ((int64_t)row * p.chunks + chunk);
    if (tid == 0) {
        total = 0.0;
        for (int w = 0; w < kWaves; ++w) total += sums[w];
        p.sums[out] = ChunkSum{total, all, 0.f};
    }
    // What reaches the bound; never -infinity, whose totals the second launch knows.  The
    // threads that hold such logits show them to all the others.
    const float least =
        bound <= order_of(-INFINITY) ? -INFINITY : value_of(bound);
    if (most >= least && most > -INFINITY) {
        const uint32_t at = atomicAdd(&hits, 1u);
        if (at < kHeld) {
            holders[at] = tid;
#pragma unroll
            for (int j = 0; j < BLOCKS; ++j)
#pragma unroll
                for (int k = 0; k < kVec; ++k) held[at][j * kVec + k] = x[j][k];
        }
    }
    __syncthreads();
    Best *best = p.best + out * p.picks;
    const uint32_t holding = hits;
    if (holding <= kHeld) {
        for (uint32_t i = tid; i < holding * kOwn; i += kThreads) {
            const float v = held[i / kOwn][i % kOwn];
            if (v >= least && v > -INFINITY) {
                const uint32_t at = atomicAdd(&count, 1u);
                if (at < kRanked) ranked[at] = key_of(v, token_of(holders[i / kOwn], i % kOwn));
            }
        }
        __syncthreads();
        const uint32_t found = count;
        if (found <= kRanked) {
            // a key's rank is how many are larger
            if (tid < found) {
                const uint64_t mine = ranked[tid];
                uint32_t rank = 0;
                for (uint32_t i = 0; i < found; ++i) rank += ranked[i] > mine ? 1u : 0u;
                if (rank < p.picks)
                    best[rank] = Best{value_of((uint32_t)(mine >> 32)), (int32_t)~(uint32_t)mine};
            }
            if (tid >= found && tid < p.picks) best[tid] = Best{0.f, -1};
            return;
        }
    }
    // Many equal logits: one after the other, the largest key below the last one.
    uint64_t last = ~0ull;
    for (uint32_t i = 0; i < p.picks; ++i) {
        uint64_t mine = 0;
#pragma unroll
        for (int j = 0; j < BLOCKS; ++j)
#pragma unroll
            for (int k = 0; k < kVec; ++k) {
                const uint64_t key = key_of(x[j][k], token_of(tid, j * kVec + k));
                if (x[j][k] > -INFINITY && key < last && key > mine) mine = key;
            }
        mine = wave_most(mine);
        __syncthreads();  // the round before has read
        if (tid % kWave == 0) ranked[wave] = mine;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kWaves; ++w) mine = ranked[w] > mine ? ranked[w] : mine;
        last = mine;
        if (tid == 0)
            best[i] = mine == 0 ? Best{0.f, -1}
                                : Best{value_of((uint32_t)(mine >> 32)), (int32_t)~(uint32_t)mine};
    }
}

// A candidate of a search: its total's order (a NaN above all, 0 for none), its place
// among beams * vocab, and its logit's order (0 where the beam's logits do not count).
// Totals that float64 does not tell apart (about a score of -1e30, say) are ordered by
// beam, those of one beam by logit, as the chunks' lists are, then by token: which
// logits reach the lists depends on the chunks' size, so no other order of one beam's
// would be the same for every launch.
struct Candidate {
    uint64_t order;
    uint32_t index, logit;
    __device__ __forceinline__ bool before(const Candidate &c, seq::FastDiv by_vocab) const {
        if (order != c.order) return order > c.order;
        return logit != c.logit && by_vocab.div(index) == by_vocab.div(c.index)
                   ? logit > c.logit
                   : index < c.index;
    }
};

__device__ __forceinline__ uint64_t order_of(double x) {
    if (x != x) return ~0ull;
    const uint64_t u = __builtin_bit_cast(uint64_t, x + 0.0);
    return u ^ ((uint64_t)((int64_t)u >> 63) | 0x8000000000000000ull);
}
__device__ __forceinline__ double double_of(uint64_t order) {
    if (order == ~0ull) return (double)NAN;
    return __builtin_bit_cast(double, order >> 63 ? order ^ 0x8000000000000000ull : ~order);
}

__device__ __forceinline__ Candidate wave_first(Candidate c, seq::FastDiv by_vocab) {
#pragma unroll
    for (int m = 1; m < kWave; m <<= 1) {
        Candidate d;
        d.order = (uint64_t)(uint32_t)__shfl_xor((int)(c.order >> 32), m) << 32 |
                  (uint32_t)__shfl_xor((int)c.order, m);
        d.index = (uint32_t)__shfl_xor((int)c.index, m);
        d.logit = (uint32_t)__shfl_xor((int)c.logit, m);
        if (d.before(c, by_vocab)) c = d;
    }
    return c;
}

constexpr uint32_t kCandidates = 2048;  // of a search, in LDS

enum Kind : uint32_t { kNone, kLogits, kFinished, kNan };

// One workgroup a search.
__global__ __launch_bounds__(kThreads) void beam_merge(SelectParams p) {
    // of a beam: score - log sum exp(logit - most), and most; a finished one's score
    __shared__ double offset[RLCA_MAX_BEAMS], largest[RLCA_MAX_BEAMS];
    __shared__ uint32_t kinds[RLCA_MAX_BEAMS];
    __shared__ Candidate firsts[kWaves];
    __shared__ uint32_t chosen[RLCA_MAX_BEAMS];
    __shared__ uint64_t orders[kCandidates], ranked[kRanked];
    __shared__ uint32_t most_of[kThreads], ranked_index[kRanked], ranked_logit[kRanked];
    __shared__ uint32_t indexes[kCandidates], logits[kCandidates], bound, reached;
    const uint32_t search = blockIdx.x, tid = threadIdx.x, wave = tid / kWave, lane = tid % kWave;
    // 16 lanes a beam
    for (uint32_t b = tid / 16; b < p.beams; b += kThreads / 16) {
        const uint32_t part = tid % 16;
        const uint32_t row = search * p.beams + b;
        const float score = p.scores[row];
        const bool finished = p.finished != nullptr && p.finished[row] != 0;
        uint32_t kind = finished              ? kFinished
                        : score == -INFINITY  ? kNone
                        : score < INFINITY    ? kLogits
                                              : kNan;
        double off = score < INFINITY ? (double)score : (double)NAN, top = 0.0;
        if (kind == kLogits) {
            const ChunkSum *sums = p.sums + (int64_t)row * p.chunks;
            float most = -INFINITY;
            for (uint32_t c = part; c < p.chunks; c += 16) most = fmaxf(most, sums[c].most);
#pragma unroll
            for (int m = 1; m < 16; m <<= 1) most = fmaxf(most, __shfl_xor(most, m));
            double sum = 0.0;
            for (uint32_t c = part; c < p.chunks; c += 16) {
                const ChunkSum s = sums[c];
                // a chunk of -infinity alone has sum 0; a NaN stays one
                sum += s.most == -INFINITY ? s.sum : s.sum * exp((double)s.most - (double)most);
            }
#pragma unroll
            for (int m = 1; m < 16; m <<= 1) sum += __shfl_xor(sum, m);
            if (sum != sum)
                kind = kNan;
            else if (sum == 0.0)
                kind = kNone;
            else
                off = (double)score - log(sum), top = most;
        }
        if (part == 0) {
            offset[b] = off;
            largest[b] = top;
            kinds[b] = kind;
        }
    }
    __syncthreads();
    // Candidate i of the search's beams * chunks * picks, or none.
    const uint32_t each = p.chunks * p.picks, count = p.beams * each;
    const Best *best = p.best + (int64_t)search * count;
    const auto candidate = [&](uint32_t i) {
        const uint32_t b = p.by_each.div(i), of_beam = i - b * each, kind = kinds[b];
        Candidate c = {0, b * p.vocab, 0};
        if (kind == kLogits) {
            const Best x = best[i];
            if (x.token >= 0) {
                c.order = order_of(offset[b] + ((double)x.logit - largest[b]));
                c.index += (uint32_t)x.token;
                c.logit = order_of(x.logit);
            }
        } else if (kind == kFinished && of_beam == 0 && !(offset[b] == -INFINITY)) {
            c.order = order_of(offset[b]);
            c.index += (uint32_t)p.pad_token;
        } else if (kind == kNan && of_beam < p.picks && of_beam < p.vocab) {
            c.order = ~0ull;
            c.index += of_beam;
        }
        return c;
    };
    // They are formed once, as long as they fit in LDS; a thread's are every kThreads-th.
    const bool fits = count <= kCandidates;
    if (tid == 0) reached = 0;
    if (fits)
        for (uint32_t i = tid; i < count; i += kThreads) {
            const Candidate c = candidate(i);
            orders[i] = c.order;
            indexes[i] = c.index;
            logits[i] = c.logit;
        }
    const auto at = [&](uint32_t i) {
        return fits ? Candidate{orders[i], indexes[i], logits[i]} : candidate(i);
    };
    const auto choose = [&](const Candidate &c, uint32_t n) {
        const uint32_t b = p.by_vocab.div(c.index);
        const int64_t to = (int64_t)search * p.picks + n;
        p.out_scores[to] = (float)double_of(c.order);
        p.out_tokens[to] = (int32_t)(c.index - b * p.vocab);
        p.out_parents[to] = (int32_t)b;
        chosen[n] = c.index;
    };
    // Those that reach a bound which at least `picks` do, ranked among each other.
    uint32_t highest = 0;
    for (uint32_t i = tid; i < count; i += kThreads) {
        const uint32_t high = (uint32_t)(at(i).order >> 32);
        highest = high > highest ? high : highest;
    }
    most_of[tid] = highest;
    __syncthreads();
    if (wave == 0) {
        const uint32_t b = kth_largest<8>(most_of, p.picks);
        if (tid == 0) bound = b;
    }
    __syncthreads();
    for (uint32_t i = tid; i < count; i += kThreads) {
        const Candidate c = at(i);
        if (c.order != 0 && (uint32_t)(c.order >> 32) >= bound) {
            const uint32_t to = atomicAdd(&reached, 1u);
            if (to < kRanked)
                ranked[to] = c.order, ranked_index[to] = c.index, ranked_logit[to] = c.logit;
        }
    }
    __syncthreads();
    uint32_t n = reached;
    if (n <= kRanked) {
        if (tid < n) {
            const auto one = [&](uint32_t i) {
                return Candidate{ranked[i], ranked_index[i], ranked_logit[i]};
            };
            const Candidate mine = one(tid);
            uint32_t rank = 0;
            bool by_logit = false;  // equal totals of unequal logits: hardly ever
            for (uint32_t i = 0; i < n; ++i) {
                const Candidate c = one(i);
                const bool equal = c.order == mine.order;
                rank += c.order > mine.order || (equal && c.index < mine.index) ? 1u : 0u;
                by_logit |= equal && c.logit != mine.logit;
            }
            if (by_logit) {
                rank = 0;
                for (uint32_t i = 0; i < n; ++i)
                    rank += one(i).before(mine, p.by_vocab) ? 1u : 0u;
            }
            if (rank < p.picks) choose(mine, rank);
        }
        n = n < p.picks ? n : p.picks;
        __syncthreads();
    } else {
        // many equal ones: one after the other, the thread's first after the last one
        const auto next_after = [&](const Candidate &last, bool any) {
            Candidate found = {0, ~0u, 0};
            for (uint32_t i = tid; i < count; i += kThreads) {
                const Candidate c = at(i);
                if (c.order != 0 && (any || last.before(c, p.by_vocab)) &&
                    c.before(found, p.by_vocab))
                    found = c;
            }
            return found;
        };
        Candidate mine = next_after(Candidate{0, 0, 0}, true);
        for (n = 0; n < p.picks; ++n) {
            Candidate first = wave_first(mine, p.by_vocab);
            if (lane == 0) firsts[wave] = first;
            __syncthreads();
#pragma unroll
            for (int w = 0; w < kWaves; ++w)
                if (firsts[w].before(first, p.by_vocab)) first = firsts[w];
            __syncthreads();
            if (first.order == 0) break;  // the same in all threads
            if (tid == 0) choose(first, n);
            if (mine.index == first.index && mine.order == first.order)
                mine = next_after(first, false);
        }
    }
    // All others have a total of -infinity: the lowest of them.
    if (tid == 0)
        for (uint32_t index = 0, taken = n; n < p.picks; ++index) {
            bool used = false;
            for (uint32_t i = 0; i < taken; ++i) used |= chosen[i] == index;
            if (used) continue;
            const uint32_t b = index / p.vocab;
            const int64_t to = (int64_t)search * p.picks + n++;
            p.out_scores[to] = -INFINITY;
            p.out_tokens[to] = (int32_t)(index - b * p.vocab);
            p.out_parents[to] = (int32_t)b;
        }
}

// ------------------------------------------------------------------ reordering
constexpr int kMaxPools = 96;  // of a launch: 24 bytes each of its arguments
constexpr int kPiece = 16;     // bytes of a thread's access

struct Pool {
    char *data;
    int64_t place_bytes;
    uint64_t first_tile;
};

struct ReorderParams {
    Pool pools[kMaxPools];
    const int32_t *slots, *parents;
    int32_t *new_slots;
    int64_t places;
    uint32_t num_pools, searches, beams;
};

// A workgroup copies a tile of 4 KB of a place, 16 bytes a thread, for every copy of its
// searches.  (Tiles of 16 KB: 32 searches of 8 beams with 18 pools 80 us against 67, 4
// searches with 12 pools 18 against 5.)
constexpr int64_t kTile = (int64_t)kThreads * kPiece;

__global__ __launch_bounds__(kThreads) void beam_reorder(ReorderParams p) {
    __shared__ int32_t free_slots[RLCA_MAX_BEAMS], from[RLCA_MAX_BEAMS], to[RLCA_MAX_BEAMS];
    __shared__ uint32_t copies;
    const uint32_t tid = threadIdx.x, lane = tid % kWave;
    uint32_t pool = 0, past = p.num_pools;  // the last pool whose first tile is not after ours
    while (past - pool > 1) {
        const uint32_t mid = (pool + past) / 2;
        if (p.pools[mid].first_tile <= blockIdx.x)
            pool = mid;
        else
            past = mid;
    }
    char *data = p.num_pools == 0 ? nullptr : p.pools[pool].data;
    const int64_t place = p.num_pools == 0 ? 0 : p.pools[pool].place_bytes;
    const int64_t at =
        p.num_pools == 0 ? 0 : (int64_t)(blockIdx.x - p.pools[pool].first_tile) * kTile;
    for (uint32_t search = blockIdx.y; search < p.searches; search += gridDim.y) {
        __syncthreads();  // the copies of the search before have been read
        if (tid < kWave) {
            const bool beam = lane < p.beams;
            const int64_t row = (int64_t)search * p.beams + lane;
            const int32_t slot = beam ? p.slots[row] : -1;
            const int32_t parent = beam ? p.parents[row] : -1;
            const bool valid = beam && parent >= 0 && parent < (int32_t)p.beams;
            bool first = valid, childless = beam;
            for (uint32_t j = 0; j < p.beams; ++j) {
                const int32_t other = __builtin_amdgcn_readlane(parent, (int)j);
                if (j < lane && other == parent) first = false;
                if (other == (int32_t)lane) childless = false;
            }
            const uint64_t below = (1ull << lane) - 1;
            const uint64_t without = __builtin_amdgcn_ballot_w64(childless);
            const uint64_t moved = __builtin_amdgcn_ballot_w64(beam && !first);
            if (childless) free_slots[__builtin_popcountll(without & below)] = slot;
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            const int32_t source = __shfl(slot, valid ? parent : 0);
            const int32_t target =
                first ? source : beam ? free_slots[__builtin_popcountll(moved & below)] : -1;
            if (beam && blockIdx.x == 0) p.new_slots[row] = target;
            const bool copy = valid && !first && source >= 0 && source < p.places &&
                              target >= 0 && target < p.places && source != target;
            const uint64_t all = __builtin_amdgcn_ballot_w64(copy);
            if (copy) {
                const int i = __builtin_popcountll(all & below);
                from[i] = source;
                to[i] = target;
            }
            if (lane == 0) copies = (uint32_t)__builtin_popcountll(all);
        }
        __syncthreads();
        const uint32_t count = copies;
        const int64_t mine = at + (int64_t)tid * kPiece;
        for (uint32_t c = 0; c < count; ++c) {
            const char *source = data + from[c] * place + mine;
            char *target = data + to[c] * place + mine;
            if (mine + kPiece <= place) {
                typedef uint32_t piece __attribute__((ext_vector_type(4)));
                piece v;
                __builtin_memcpy(&v, source, kPiece);
                __builtin_memcpy(target, &v, kPiece);
            } else {
                // a place's last bytes
                for (int64_t i = mine; i < place; ++i) target[i - mine] = source[i - mine];
            }
        }
    }
}

// ------------------------------------------------------------------- host side
// Blocks of kVec logits a thread: chunks of 2048 logits where 6144 would make too few
// workgroups for the chip (4 beams of 32000 tokens, fp32: 9.7 us against 10.8; 32 of
// 50000, bf16: 14.8 against 12.3; 512 of 100003: 39 us, 42 with 4096 or 8192).
static int blocks_of(const rlca_beam_call &c) {
    const int64_t rows = c.num_searches * c.beams;
    return rows * ((c.vocab + 6143) / 6144) < 128 ? 1 : 3;
}

static int64_t chunks_of(const rlca_beam_call &c) {
    const int64_t chunk = (int64_t)kThreads * kVec * blocks_of(c);
    return (c.vocab + chunk - 1) / chunk;
}

static bool sizes_fit(const rlca_beam_call &c) {
    return c.num_searches >= 0 && c.num_searches < (int64_t)1 << 24 && c.beams >= 1 &&
           c.beams <= RLCA_MAX_BEAMS && c.vocab >= 1 && c.vocab < (int64_t)1 << 31 &&
           c.beams * c.vocab < (int64_t)1 << 31 && c.picks >= 1 && c.picks <= RLCA_MAX_BEAMS &&
           c.picks <= c.beams * c.vocab &&
           // the launch's threads
           c.num_searches * c.beams * chunks_of(c) < (int64_t)1 << 24;
}

static size_t workspace_of(const rlca_beam_call &c) {
    const size_t chunks = (size_t)c.num_searches * c.beams * chunks_of(c);
    return chunks * (sizeof(ChunkSum) + c.picks * sizeof(Best));
}

template <typename E>
static const void *chunks_kernel(int blocks) {
    return blocks == 1 ? (const void *)beam_chunks<E, 1> : (const void *)beam_chunks<E, 3>;
}

}  // namespace beams
}  // namespace rlca

using namespace rlca::beams;
using rlca::seq::Arrays;
using rlca::seq::element_bytes;
using rlca::seq::fast_div;
using rlca::seq::launch;

extern "C" {

size_t rlca_beam_select_workspace_size(const rlca_beam_call *call) {
    if (call == nullptr || !sizes_fit(*call)) return 0;
    return workspace_of(*call);
}

rlca_status rlca_beam_select(const rlca_beam_call *call, void *workspace, size_t workspace_bytes,
                             hipStream_t stream) {
    if (call == nullptr) return RLCA_ERR_NULL_POINTER;
    const rlca_beam_call &c = *call;
    if (!sizes_fit(c)) return RLCA_ERR_INVALID_SIZE;
    const size_t e = element_bytes(c.dtype);
    if (e == 0 || (c.finished != nullptr && (c.pad_token < 0 || c.pad_token >= c.vocab)))
        return RLCA_ERR_INVALID_VALUE;
    const int64_t N = c.num_searches, K = c.beams, V = c.vocab, P = c.picks;
    const size_t need = workspace_of(c);
    Arrays a;
    a.in(c.logits, e, true, {{N, c.logits_stride_search}, {K, c.logits_stride_beam}, {V, 1}});
    a.in(c.scores, 4, true, {{N, K}, {K, 1}});
    a.in(c.finished, 1, false, {{N, K}, {K, 1}});
    a.out(c.out_scores, 4, true, {{N, P}, {P, 1}});
    a.out(c.out_tokens, 4, true, {{N, P}, {P, 1}});
    a.out(c.out_parents, 4, true, {{N, P}, {P, 1}});
    a.out(workspace, 8, need != 0, {{(int64_t)(need / 8), 1}});
    rlca_status st = a.status();
    if (st != RLCA_OK) return st;
    if (workspace_bytes < need) return RLCA_ERR_INVALID_SIZE;
    if (N == 0) return RLCA_OK;
    SelectParams p = {};
    p.logits = c.logits;
    p.scores = c.scores;
    p.finished = c.finished;
    p.out_scores = c.out_scores;
    p.out_tokens = c.out_tokens;
    p.out_parents = c.out_parents;
    p.by_search = c.logits_stride_search;
    p.by_beam = c.logits_stride_beam;
    p.searches = (uint32_t)N;
    p.beams = (uint32_t)K;
    p.vocab = (uint32_t)V;
    p.picks = (uint32_t)P;
    p.chunks = (uint32_t)chunks_of(c);
    p.pad_token = c.pad_token;
    p.by_chunks = fast_div(p.chunks);
    p.by_beams = fast_div(p.beams);
    p.by_each = fast_div(p.chunks * p.picks);
    p.by_vocab = fast_div(p.vocab);
    const uint32_t groups = p.searches * p.beams * p.chunks;
    p.sums = static_cast<ChunkSum *>(workspace);
    p.best = reinterpret_cast<Best *>(p.sums + groups);
    const int blocks = blocks_of(c);
    const void *kernel = c.dtype == RLCA_F32    ? chunks_kernel<float>(blocks)
                         : c.dtype == RLCA_BF16 ? chunks_kernel<__bf16>(blocks)
                                                : chunks_kernel<_Float16>(blocks);
    if ((st = launch(kernel, dim3(groups), kThreads, 0, p, stream)) != RLCA_OK) return st;
    return launch((const void *)beam_merge, dim3(p.searches), kThreads, 0, p, stream);
}

rlca_status rlca_beam_reorder(const rlca_state_pool *pools, int64_t num_pools,
                              int64_t num_searches, int64_t beams, int64_t places,
                              const int32_t *slots, const int32_t *parents, int32_t *new_slots,
                              hipStream_t stream) {
    const int64_t N = num_searches, K = beams;
    if (num_pools < 0 || N < 0 || N >= (int64_t)1 << 31 || K < 1 || K > RLCA_MAX_BEAMS ||
        places < 0 || places > INT32_MAX || N * K >= (int64_t)1 << 31)
        return RLCA_ERR_INVALID_SIZE;
    if (pools == nullptr && num_pools > 0) return RLCA_ERR_NULL_POINTER;
    Arrays a;
    a.in(slots, 4, true, {{N, K}, {K, 1}});
    a.in(parents, 4, true, {{N, K}, {K, 1}});
    a.out(new_slots, 4, true, {{N, K}, {K, 1}});
    rlca_status st = a.status();
    if (st != RLCA_OK) return st;
    const auto bytes_of = [&](const rlca_state_pool &p, size_t *bytes) {
        return p.place_bytes >= 0 &&
               rlca::seq::covered((const rlca::seq::Dim[]){{places, p.place_bytes}, {p.place_bytes, 1}},
                                  2, 1, bytes);
    };
    for (int64_t i = 0; i < num_pools; ++i) {
        size_t bytes, other;
        if (!bytes_of(pools[i], &bytes)) return RLCA_ERR_INVALID_SIZE;
        // the workgroups of a launch
        if (pools[i].place_bytes > (int64_t)1 << 35) return RLCA_ERR_INVALID_SIZE;
        if (bytes == 0 || N == 0) continue;
        if (pools[i].data == nullptr) return RLCA_ERR_NULL_POINTER;
        const uintptr_t at = (uintptr_t)pools[i].data;
        const auto meets = [&](const void *p, size_t n) {
            return at < (uintptr_t)p + n && (uintptr_t)p < at + bytes;
        };
        const size_t words = (size_t)(N * K) * 4;
        if (meets(slots, words) || meets(parents, words) || meets(new_slots, words))
            return RLCA_ERR_ALIASING;
        for (int64_t j = 0; j < i; ++j)
            if (bytes_of(pools[j], &other) && other != 0 && meets(pools[j].data, other))
                return RLCA_ERR_ALIASING;
    }
    if (N == 0) return RLCA_OK;
    ReorderParams p;
    p.slots = slots;
    p.parents = parents;
    p.new_slots = new_slots;
    p.places = places;
    p.searches = (uint32_t)N;
    p.beams = (uint32_t)K;
    int64_t i = 0;
    do {  // the first launch writes new_slots, with no pools too
        int64_t blocks = 0;
        p.num_pools = 0;
        for (; i < num_pools && p.num_pools < kMaxPools; ++i) {
            const int64_t more = (pools[i].place_bytes + kTile - 1) / kTile;
            if (more == 0 || places == 0) continue;
            if (blocks + more > (int64_t)1 << 23) break;
            p.pools[p.num_pools++] =
                Pool{static_cast<char *>(pools[i].data), pools[i].place_bytes, (uint64_t)blocks};
            blocks += more;
        }
        const dim3 grid((uint32_t)(blocks < 1 ? 1 : blocks), (uint32_t)(N < 65535 ? N : 65535));
        st = launch((const void *)beam_reorder, grid, kThreads, 0, p, stream);
        if (st != RLCA_OK) return st;
    } while (i < num_pools);
    return RLCA_OK;
}

}  // extern "C"
