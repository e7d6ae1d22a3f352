// kv4_evict.hip -- the tokens of a sequence with the largest weight, its first and its last
// ones, moved in their order to other pages of the 4-bit cache, kv head by kv head.
//
// Choosing: a workgroup to a (sequence, kv head), or several where these are few and histories
// long.  Weights become integers of the same order; three passes over them, 11, 11 and 10
// bits each, find the smallest one that is kept and how many of its equals are; a last pass
// over the tokens in order gives each kept one its place.  Moving: a workgroup to a page of the result, which gathers its 64 tokens
// (records as kv4.h lays them out) and writes them once.
//
// What bounds it: latency in the choice, of loads, LDS counts and barriers (16 sequences of
// 2176 tokens, 8 heads: 12 to 14 us; one of 131072, 5 heads: 240 us by one workgroup each, 38 by 16 in
// four launches of 7 to 12), HBM in the move of many tokens (13000 of 8 heads of 128, 34 MB with
// the weights: 10 us).
#include <algorithm>

#include "kv4.h"

namespace bitnet {

namespace {

constexpr int kChooseThreads = 1024;
constexpr int kChooseWaves = kChooseThreads / 64;
constexpr int kBatch = 4;
constexpr int kMoveThreads = 256;

// Integers in the order of the weights; a NaN counts as -infinity, -0 as 0.
__device__ __forceinline__ uint32_t order_of(float w) {
    if (w != w) w = -INFINITY;
    const uint32_t u = __float_as_uint(w + 0.0f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Sum over the workgroup of one int each, to every thread; `slot` is not used by the last call.
__device__ __forceinline__ int block_sum(int v, int *slot) {
    v = wave_sum_i32(v);
    if ((threadIdx.x & 63) == 0) slot[threadIdx.x >> 6] = v;
    __syncthreads();
    int t = 0;
    for (int w = 0; w < kChooseWaves; ++w) t += slot[w];
    __syncthreads();
    return t;
}

// Two of them at once, or four.
template <bool FOUR>
__device__ __forceinline__ int4 block_sum4(int4 v, int4 *slot) {
    v.x = wave_sum_i32(v.x);
    v.y = wave_sum_i32(v.y);
    if constexpr (FOUR) {
        v.z = wave_sum_i32(v.z);
        v.w = wave_sum_i32(v.w);
    }
    if ((threadIdx.x & 63) == 0) slot[threadIdx.x >> 6] = v;
    __syncthreads();
    int4 t = make_int4(0, 0, 0, 0);
    for (int w = 0; w < kChooseWaves; ++w)
        t = make_int4(t.x + slot[w].x, t.y + slot[w].y, t.z + slot[w].z, t.w + slot[w].w);
    __syncthreads();
    return t;
}

// Inclusive sum over the lanes of a wave.
__device__ __forceinline__ uint32_t wave_scan(uint32_t v) {
    const int lane = threadIdx.x & 63;
    for (int d = 1; d < 64; d *= 2) {
        const uint32_t o = __shfl_up(v, d);
        if (lane >= d) v += o;
    }
    return v;
}

// A (sequence, kv head) and how many of its tokens are kept; every thread of a workgroup has it.
struct Unit {
    int64_t seq, row;   // row: of the index
    int head, held;
    int there, kept, quota;   // tokens whose page is there; of them kept; of those by their weight
    __device__ bool choose() const { return kept < there && quota > 0; }
    __device__ bool spared(const EvictArgs &a, int t) const { return t < a.sinks || t >= held - a.recent; }
    __device__ int page_of(const EvictArgs &a, int t) const {   // or -1
        const int id = a.table[seq * a.max_pages + t / kPage];
        return id >= 0 && id < a.n_pages ? id : -1;
    }
    __device__ float4 weights4(const EvictArgs &a, int id, int t0) const {   // of tokens t0 .. t0 + 3
        return *reinterpret_cast<const float4 *>(a.weights + ((int64_t)id * a.kv_heads + head) * kPage + t0 % kPage);
    }
};
__device__ __forceinline__ Unit unit_at(const EvictArgs &a, int64_t unit) {   // without its counts
    Unit u;
    u.seq = unit / a.kv_heads;
    u.row = unit;
    u.head = (int)(unit - u.seq * a.kv_heads);
    u.held = min(max(a.kv_len[u.seq], 0), (int)(a.max_pages * kPage));
    return u;
}
__device__ __forceinline__ void set_counts(const EvictArgs &a, Unit &u, int there, int quota) {
    u.there = there;
    u.kept = min(there, a.keep);
    u.quota = quota;
}
// The counts of a unit.  With BEFORE also of the tokens before `from` those whose page is
// there, and of these the ones kept in any case.
template <bool BEFORE>
__device__ __forceinline__ int2 count_unit(const EvictArgs &a, Unit &u, int from, int4 *slot) {
    int4 mine = make_int4(0, 0, 0, 0);
    for (int t0 = threadIdx.x * kPage; t0 < u.held; t0 += kChooseThreads * kPage)
        if (u.page_of(a, t0) >= 0) {
            // of [t0, t1): [0, sinks) and [held - recent, held) may meet
            auto safe = [&](int t1) {
                const int low = min(max(a.sinks - t0, 0), t1 - t0);
                const int high = min(max(t1 - max(u.held - a.recent, t0), 0), t1 - t0);
                return min(low + high, t1 - t0);
            };
            const int t1 = min(u.held, t0 + kPage);
            mine.x += t1 - t0;
            mine.y += safe(t1);
            if constexpr (BEFORE) {
                const int cut = min(max(from, t0), t1);
                mine.z += cut - t0;
                mine.w += safe(cut);
            }
        }
    const int4 all = block_sum4<BEFORE>(mine, slot);
    set_counts(a, u, all.x, min(all.x, a.keep) - all.y);   // not negative: sinks + recent <= keep
    return make_int2(all.z, all.w);
}

// The search for the smallest order that is kept: its upper bits so far, and how many of the
// tokens that share them are kept.
struct Search {
    uint32_t least;
    int ties;
};
constexpr int kPasses = 3;
__device__ __forceinline__ int shift_of(int pass) { return pass == 0 ? 21 : pass == 1 ? 10 : 0; }
__device__ __forceinline__ int width_of(int pass) { return pass < 2 ? 11 : 10; }

// Counts four tokens t0 on by the next bits of their order.
__device__ __forceinline__ void count_four(const EvictArgs &a, const Unit &u, int pass, const Search &f, int id, int t0,
                                           int to, const float4 &w, int *bins) {
    const int shift = shift_of(pass), width = width_of(pass);
    const float v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if (id < 0 || t0 + e >= to || u.spared(a, t0 + e)) continue;
        const uint32_t o = order_of(v[e]);
        if (pass > 0 && (o ^ f.least) >> (shift + width)) continue;   // other upper bits
        atomicAdd(&bins[o >> shift & ((1 << width) - 1)], 1);
    }
}
// Four tokens to a thread, kBatch times, are loaded before any is looked at.
struct Batch {
    int id[kBatch];
    float4 w[kBatch];
};
__device__ __forceinline__ void load_batch(Batch &b, const EvictArgs &a, const Unit &u, int base, int to) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
        const int t0 = base + 4 * kChooseThreads * i;
        b.id[i] = t0 < to ? u.page_of(a, t0) : -1;
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) b.w[i] = u.weights4(a, max(b.id[i], 0), base + 4 * kChooseThreads * i);
}
// Counts the tokens of [from, to) (from a multiple of four); `b`: the first of each thread.
__device__ __forceinline__ void count_bins(const EvictArgs &a, const Unit &u, int pass, const Search &f, int from,
                                           int to, int *bins, Batch b) {
    for (int i = threadIdx.x; i < kBins; i += kChooseThreads) bins[i] = 0;
    __syncthreads();
    for (int base = from + 4 * (int)threadIdx.x; base < to;) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) count_four(a, u, pass, f, b.id[i], base + 4 * kChooseThreads * i, to, b.w[i], bins);
        base += 4 * kChooseThreads * kBatch;
        if (base < to) load_batch(b, a, u, base, to);
    }
    __syncthreads();
}
// One step of the search; c1, c0: what bins 2047 - 2 i and 2046 - 2 i of thread i count.
__device__ __forceinline__ void pick(Search &f, int pass, int c1, int c0, uint32_t *scan, int *found) {
    const int wave = threadIdx.x >> 6, b1 = kBins - 1 - 2 * (int)threadIdx.x;
    uint32_t up = wave_scan((uint32_t)(c1 + c0));
    if ((threadIdx.x & 63) == 63) scan[wave] = up;
    __syncthreads();
    for (int w = 0; w < wave; ++w) up += scan[w];
    const int before = (int)up - c1 - c0;   // in the bins above this thread's
    if (before < f.ties && before + c1 >= f.ties) {
        found[0] = b1;
        found[1] = f.ties - before;
    } else if (before + c1 < f.ties && before + c1 + c0 >= f.ties) {
        found[0] = b1 - 1;
        found[1] = f.ties - before - c1;
    }
    __syncthreads();
    f.least |= (uint32_t)found[0] << shift_of(pass);
    f.ties = found[1];
    __syncthreads();
}

// Which of four tokens t0 on are kept whatever comes before them, and which if they are among
// the first ties: bits.
__device__ __forceinline__ void kinds_of(const EvictArgs &a, const Unit &u, const Search &f, int id, int t0, int to,
                                         const float4 &w4, uint32_t &sure, uint32_t &tie) {
    sure = tie = 0;
    if (id < 0) return;
    const float w[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if (t0 + e >= to) continue;
        const uint32_t o = order_of(w[e]);
        if (u.kept == u.there || u.spared(a, t0 + e) || (u.choose() && o > f.least)) sure |= 1u << e;
        else if (u.choose() && o == f.least) tie |= 1u << e;
    }
}
// A thread's page and weights of a turn of placing, and its next page.
struct Turn {
    int id, id1;
    float4 w4;
};
__device__ __forceinline__ Turn first_turn(const EvictArgs &a, const Unit &u, int from, int to) {
    auto entry = [&](int t0) { return t0 < to ? u.page_of(a, t0) : -1; };
    Turn t{entry(from + 4 * (int)threadIdx.x), entry(from + 4 * ((int)threadIdx.x + kChooseThreads)), {}};
    t.w4 = u.weights4(a, max(t.id, 0), from + 4 * threadIdx.x);
    return t;
}
// Gives the kept tokens of [from, to) their places, in order, behind those before them.
__device__ __forceinline__ void place_tokens(const EvictArgs &a, const Unit &u, const Search &f, int from, int to,
                                             int sure_before, int ties_before, uint32_t *scan, const Turn &first) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    int32_t *index = a.index + u.row * a.keep;
    auto entry = [&](int t0) { return t0 < to ? u.page_of(a, t0) : -1; };
    int id = first.id, id1 = first.id1;
    float4 w4 = first.w4;
    for (int base = from; base < to; base += 4 * kChooseThreads) {
        const int t0 = base + 4 * tid, id2 = entry(t0 + 8 * kChooseThreads);
        const float4 next = u.weights4(a, max(id1, 0), t0 + 4 * kChooseThreads);
        uint32_t sure, tie;
        kinds_of(a, u, f, id, t0, to, w4, sure, tie);
        const uint32_t counts = (uint32_t)__popc(sure) << 16 | (uint32_t)__popc(tie);
        const uint32_t up = wave_scan(counts);
        if (lane == 63) scan[wave] = up;
        __syncthreads();
        uint32_t off = up - counts, all = 0;   // 4096 of each at most
        for (int w = 0; w < kChooseWaves; ++w) {
            if (w < wave) off += scan[w];
            all += scan[w];
        }
        int s = sure_before + (int)(off >> 16), t = ties_before + (int)(off & 0xffffu);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const bool is_tie = tie >> e & 1, in = (sure >> e & 1) || (is_tie && t < f.ties);
            const int at = s + min(t, f.ties);
            // (always a place of the index, unless another stream writes the weights during the call:
            // then a search may end without a result and `at` be anything, below 0 too)
            if (in && (uint32_t)at < (uint32_t)u.kept) index[at] = t0 + e;
            s += sure >> e & 1;
            t += is_tie;
        }
        sure_before += (int)(all >> 16);
        ties_before += (int)(all & 0xffffu);
        id = id1;
        id1 = id2;
        w4 = next;
        __syncthreads();
    }
}

// The whole choice by one workgroup.
__global__ __launch_bounds__(kChooseThreads) void evict_choose_kernel(const EvictArgs a, int64_t units) {
    __shared__ int bins[kBins], found[2];
    __shared__ int4 slot[kChooseWaves];
    __shared__ uint32_t scan[kChooseWaves];
    for (int64_t unit = blockIdx.x; unit < units; unit += gridDim.x) {
        Unit u = unit_at(a, unit);
        // four tokens to a thread are looked at again and again without being loaded again
        const bool few = u.held <= 4 * kChooseThreads;
        const int id = few && 4 * (int)threadIdx.x < u.held ? u.page_of(a, 4 * threadIdx.x) : -1;
        const float4 w4 = u.weights4(a, max(id, 0), 4 * threadIdx.x);
        count_unit<false>(a, u, 0, slot);
        if (u.head == 0 && threadIdx.x == 0) a.new_len[u.seq] = u.kept;
        Search f{0, u.quota};
        if (u.choose())
            for (int pass = 0; pass < kPasses; ++pass) {
                if (few) {
                    for (int i = threadIdx.x; i < kBins; i += kChooseThreads) bins[i] = 0;
                    __syncthreads();
                    count_four(a, u, pass, f, id, 4 * threadIdx.x, u.held, w4, bins);
                    __syncthreads();
                } else {
                    Batch b;
                    load_batch(b, a, u, 4 * threadIdx.x, u.held);
                    count_bins(a, u, pass, f, 0, u.held, bins, b);
                }
                const int b1 = kBins - 1 - 2 * (int)threadIdx.x;
                pick(f, pass, bins[b1], bins[b1 - 1], scan, found);
            }
        place_tokens(a, u, f, 0, u.held, 0, 0, scan, few ? Turn{id, -1, w4} : first_turn(a, u, 0, u.held));
        for (int i = u.kept + threadIdx.x; i < a.keep; i += kChooseThreads) a.index[u.row * a.keep + i] = -1;
    }
}

// The choice of a long history by `slices` workgroups, a launch for each step: 0 to 2 count
// a slice's bins, 3 gives its tokens their places.  A step first finishes the pass before it
// from the counts of all slices, which also say how many of the slices before its own are kept:
// its weights are on their way meanwhile.  a.search [3][unit]: what the passes 0 and 1 found, each
// in a place of its own since other slices still read the last one's, and the unit's counts;
// a.slices [unit][slice]: tokens before the slice that are known to be kept (x; y is not used).
template <int STEP>
__global__ __launch_bounds__(kChooseThreads) void evict_step_kernel(const EvictArgs a, int slices) {
    __shared__ int bins[kBins], found[2], tied;
    __shared__ int4 slot[kChooseWaves];
    __shared__ uint32_t scan[kChooseWaves];
    const int64_t unit = blockIdx.x / slices, units = gridDim.x / slices;
    const int slice = (int)(blockIdx.x - unit * slices), tid = threadIdx.x;
    Unit u = unit_at(a, unit);
    const EvictSlice part = evict_slice(u.held, slices, slice);
    const int from = part.from, to = part.to;
    Batch b;
    Turn first;
    if constexpr (STEP < kPasses) load_batch(b, a, u, from + 4 * tid, to);
    else first = first_turn(a, u, from, to);
    int *const counts = a.counts + unit * slices * kBins;   // [pass][unit][slice][bin]
    const int64_t pass_size = units * slices * kBins;
    int2 &known = a.slices[unit * slices + slice];
    int sure_before, ties_before = 0;
    if constexpr (STEP == 0) {
        const int2 before = count_unit<true>(a, u, from, slot);
        sure_before = u.kept == u.there ? before.x : before.y;
        if (slice == 0 && tid == 0) a.search[2 * units + unit] = make_int2(u.there, u.quota);
    } else {
        const int2 c = a.search[2 * units + unit];
        set_counts(a, u, c.x, c.y);
        sure_before = known.x;
    }
    Search f{0, u.quota};
    if (STEP > 0 && u.choose()) {
        if (STEP > 1) {
            const int2 last = a.search[(STEP - 2) * units + unit];
            f = Search{(uint32_t)last.x, last.y};
        }
        const int *of_pass = counts + (STEP - 1) * pass_size + kBins - 2 - 2 * tid;
        int c1 = 0, c0 = 0, p1 = 0, p0 = 0;   // p: in the slices before
#pragma unroll 8
        for (int s = 0; s < slices; ++s) {
            const int2 c = *reinterpret_cast<const int2 *>(of_pass + s * kBins);
            c0 += c.x;
            c1 += c.y;
            p0 += s < slice ? c.x : 0;
            p1 += s < slice ? c.y : 0;
        }
        pick(f, STEP - 1, c1, c0, scan, found);
        const int bin = (int)(f.least >> shift_of(STEP - 1)) & ((1 << width_of(STEP - 1)) - 1);
        const int b1 = kBins - 1 - 2 * tid;
        if (bin == b1) tied = p1;
        if (bin == b1 - 1) tied = p0;
        sure_before += block_sum((b1 > bin ? p1 : 0) + (b1 - 1 > bin ? p0 : 0), reinterpret_cast<int *>(slot));
        ties_before = tied;
        if (STEP < kPasses && slice == 0 && tid == 0) a.search[(STEP - 1) * units + unit] = make_int2((int)f.least, f.ties);
    }
    if constexpr (STEP < kPasses) {
        if (tid == 0) known.x = sure_before;
        if (u.choose()) {
            count_bins(a, u, STEP, f, from, to, bins, b);
            for (int i = tid; i < kBins; i += kChooseThreads)
                counts[STEP * pass_size + slice * kBins + i] = bins[i];
        }
    } else {
        place_tokens(a, u, f, from, to, sure_before, ties_before, scan, first);
        for (int i = u.kept + slice * kChooseThreads + tid; i < a.keep; i += slices * kChooseThreads)
            a.index[u.row * a.keep + i] = -1;
        if (u.head == 0 && slice == 0 && tid == 0) a.new_len[u.seq] = u.kept;
    }
}

template <int D>
__global__ __launch_bounds__(kMoveThreads) void evict_move_kernel(const EvictArgs a, int pages, int64_t units) {
    using L = Kv4Page<D>;
    constexpr int NG = L::kGroups;
    __shared__ int64_t from[kPage];   // records of the 64 tokens, in front of which lies their place
    __shared__ int at[kPage];
    for (int64_t unit = blockIdx.x; unit < units; unit += gridDim.x) {
        const int64_t u = unit / a.kv_heads, seq = u / pages;
        const int head = (int)(unit - u * a.kv_heads), page = (int)(u - seq * pages);
        const int n = min(a.new_len[seq] - page * kPage, kPage);   // tokens of this page
        if (n <= 0) continue;   // the whole workgroup
        const int id = a.new_table[seq * a.new_pages + page];
        if (id < 0 || id >= a.n_pages) continue;
        const int64_t rec_at = ((int64_t)id * a.kv_heads + head);
        if (threadIdx.x < kPage) {
            // tokens behind the last one stand in for it, and are not written
            const int t = min(max(a.index[(seq * a.kv_heads + head) * a.keep + page * kPage + min((int)threadIdx.x, n - 1)], 0),
                              (int)(a.max_pages * kPage) - 1);
            const int src = a.table[seq * a.max_pages + t / kPage];
            const int64_t rec = (int64_t)(src >= 0 && src < a.n_pages ? src : id) * a.kv_heads + head;
            from[threadIdx.x] = rec;
            at[threadIdx.x] = t % kPage;
            if ((int)threadIdx.x < n) a.weights[rec_at * kPage + threadIdx.x] = a.weights[rec * kPage + t % kPage];
        }
        __syncthreads();
        uint8_t *out = a.cache + rec_at * L::kBytes;
        // key codes: 16 bytes at a time
        for (int i = threadIdx.x; i < n * (L::kRow / 16); i += kMoveThreads) {
            const int t = i / (L::kRow / 16), p = i % (L::kRow / 16);
            reinterpret_cast<uint4 *>(out + t * L::kRow)[p] =
                reinterpret_cast<const uint4 *>(a.cache + from[t] * L::kBytes + at[t] * L::kRow)[p];
        }
        for (int i = threadIdx.x; i < n * NG; i += kMoveThreads) {
            const int t = i / NG, g = i % NG;
            reinterpret_cast<uint32_t *>(out + L::kKeyPairs)[i] = reinterpret_cast<const uint32_t *>(
                a.cache + from[t] * L::kBytes + L::kKeyPairs)[at[t] * NG + g];
        }
        // value codes: a halfword of each of four tokens; then their pairs, a step or a middle
        for (int i = threadIdx.x; i < 16 * 16 * NG + 16 * NG * 2; i += kMoveThreads) {
            const bool codes = i < 16 * 16 * NG;
            const int k = codes ? i : i - 16 * 16 * NG, per = codes ? 16 * NG : 2 * NG;
            const int block = k / per, line = k % per;   // line: (lane, group), or (group, kind)
            const int part = codes ? L::kValues : L::kValuePairs;
            if (4 * block >= n) continue;
            uint16_t h[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int t = 4 * block + e;
                h[e] = reinterpret_cast<const uint16_t *>(a.cache + from[t] * L::kBytes + part)
                    [((at[t] >> 2) * per + line) * 4 + (at[t] & 3)];
            }
            uint16_t *o = reinterpret_cast<uint16_t *>(out + part) + (block * per + line) * 4;
            if (4 * block + 4 <= n) {
                *reinterpret_cast<uint2 *>(o) = make_uint2(h[0] | (uint32_t)h[1] << 16, h[2] | (uint32_t)h[3] << 16);
            } else {
#pragma unroll
                for (int e = 0; e < 3; ++e)
                    if (4 * block + e < n) o[e] = h[e];
            }
        }
        __syncthreads();   // `from` and `at` are used again
    }
}

}  // namespace

hipError_t launch_kv4_evict(const EvictArgs &a, const EvictPlan &p, int dim, hipStream_t st) {
    constexpr int64_t kMost = 1 << 21;   // workgroups; more units take turns
    const int64_t heads = a.n_seqs * a.kv_heads;
    if (p.slices == 1) {
        hipLaunchKernelGGL(evict_choose_kernel, dim3((unsigned)std::min(heads, kMost)), dim3(kChooseThreads), 0, st, a,
                           heads);
    } else {
        const dim3 g((unsigned)(heads * p.slices)), t(kChooseThreads);
        hipLaunchKernelGGL((evict_step_kernel<0>), g, t, 0, st, a, p.slices);
        hipLaunchKernelGGL((evict_step_kernel<1>), g, t, 0, st, a, p.slices);
        hipLaunchKernelGGL((evict_step_kernel<2>), g, t, 0, st, a, p.slices);
        hipLaunchKernelGGL((evict_step_kernel<3>), g, t, 0, st, a, p.slices);
    }
    const int pages = (a.keep + kPage - 1) / kPage;
    const int64_t units = heads * pages;
    const dim3 g((unsigned)std::min(units, kMost)), t(kMoveThreads);
    if (dim == 64) hipLaunchKernelGGL((evict_move_kernel<64>), g, t, 0, st, a, pages, units);
    else if (dim == 128) hipLaunchKernelGGL((evict_move_kernel<128>), g, t, 0, st, a, pages, units);
    else hipLaunchKernelGGL((evict_move_kernel<256>), g, t, 0, st, a, pages, units);
    return hipGetLastError();
}

}  // namespace bitnet
