// kv4_evict.hip -- the tokens of a sequence with the largest weight, its first and its last
// ones, moved in their order to other pages of the 4-bit cache, kv head by kv head.
//
// Choosing: a workgroup to a (sequence, kv head).  Weights become integers of the same
// order; three passes over them, 11, 11 and 10 bits each, find the smallest one that is
// kept and how many of its equals are; a last pass over the tokens in order gives each kept
// one its place.  Moving: a workgroup to a page of the result, which gathers its 64 tokens
// (records as kv4.h lays them out) and writes them once.
#include <algorithm>

#include "kv4.h"

namespace bitnet {

namespace {

constexpr int kChooseThreads = 1024;
constexpr int kChooseWaves = kChooseThreads / 64;
constexpr int kBins = 2048;
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

// Inclusive sum over the lanes of a wave.
__device__ __forceinline__ uint32_t wave_scan(uint32_t v) {
    const int lane = threadIdx.x & 63;
    for (int d = 1; d < 64; d *= 2) {
        const uint32_t o = __shfl_up(v, d);
        if (lane >= d) v += o;
    }
    return v;
}

__global__ __launch_bounds__(kChooseThreads) void evict_choose_kernel(const EvictArgs a, int64_t units) {
    __shared__ int bins[kBins], slot[kChooseWaves];
    __shared__ uint32_t scan[2][kChooseWaves];
    __shared__ int found[2];   // the bin that the last kept one is in, and how many of it are kept
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    for (int64_t unit = blockIdx.x; unit < units; unit += gridDim.x) {
        const int64_t seq = unit / a.kv_heads;
        const int head = (int)(unit - seq * a.kv_heads);
        const int held = min(max(a.kv_len[seq], 0), (int)(a.max_pages * kPage));
        const int pages = (held + kPage - 1) / kPage;
        const int32_t *table = a.table + seq * a.max_pages;
        auto page_of = [&](int p) {
            const int id = table[p];
            return id >= 0 && id < a.n_pages ? id : -1;
        };
        auto weights4 = [&](int id, int t0) {   // of tokens t0 .. t0 + 3
            return *reinterpret_cast<const float4 *>(a.weights + ((int64_t)id * a.kv_heads + head) * kPage + t0 % kPage);
        };
        // tokens that are there, and those of them that are spared
        auto spared = [&](int t) { return t < a.sinks || t >= held - a.recent; };
        int mine = 0, safe = 0;
        for (int p = tid; p < pages; p += kChooseThreads)
            if (page_of(p) >= 0) {
                const int t0 = p * kPage, t1 = min(held, t0 + kPage);
                mine += t1 - t0;
                // [0, sinks) and [held - recent, held) may meet
                const int low = min(max(a.sinks - t0, 0), t1 - t0);
                const int high = min(max(t1 - max(held - a.recent, t0), 0), t1 - t0);
                safe += min(low + high, t1 - t0);
            }
        const int there = block_sum(mine, slot);
        const int safe_all = block_sum(safe, slot);
        const int kept = min(there, a.keep), quota = kept - safe_all;   // quota >= 0: sinks + recent <= keep
        if (head == 0 && tid == 0) a.new_len[seq] = kept;
        // ---- the smallest order that is kept, bit by bit from the top
        uint32_t least = 0;   // its upper bits so far
        int ties = quota;     // how many of those that share them are kept
        const bool choose = kept < there && quota > 0;
        if (choose) {
            int shift = 21;
            for (int pass = 0; pass < 3; ++pass) {
                const int width = pass < 2 ? 11 : 10, next = pass == 0 ? 10 : 0;
                for (int i = tid; i < kBins; i += kChooseThreads) bins[i] = 0;
                __syncthreads();
                // four tokens to a thread, kBatch times: first all loads, then the counts
                for (int base = 4 * tid; base < held; base += 4 * kChooseThreads * kBatch) {
                    int id[kBatch];
                    float4 w[kBatch];
#pragma unroll
                    for (int i = 0; i < kBatch; ++i) {
                        const int t0 = base + 4 * kChooseThreads * i;
                        id[i] = t0 < held ? page_of(t0 / kPage) : -1;
                    }
#pragma unroll
                    for (int i = 0; i < kBatch; ++i)
                        w[i] = weights4(max(id[i], 0), base + 4 * kChooseThreads * i);
#pragma unroll
                    for (int i = 0; i < kBatch; ++i) {
                        const int t0 = base + 4 * kChooseThreads * i;
                        const float v[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            if (id[i] < 0 || t0 + e >= held || spared(t0 + e)) continue;
                            const uint32_t o = order_of(v[e]);
                            if (pass > 0 && (o ^ least) >> (shift + width)) continue;   // other upper bits
                            atomicAdd(&bins[o >> shift & ((1 << width) - 1)], 1);
                        }
                    }
                }
                __syncthreads();
                // from the top: thread i has bins 2047 - 2 i and 2046 - 2 i
                const int b1 = kBins - 1 - 2 * tid, c1 = bins[b1], c0 = bins[b1 - 1];
                uint32_t up = wave_scan((uint32_t)(c1 + c0));
                if (lane == 63) scan[0][wave] = up;
                __syncthreads();
                for (int w = 0; w < wave; ++w) up += scan[0][w];
                const int before = (int)up - c1 - c0;   // in the bins above this thread's
                if (before < ties && before + c1 >= ties) {
                    found[0] = b1;
                    found[1] = ties - before;
                } else if (before + c1 < ties && before + c1 + c0 >= ties) {
                    found[0] = b1 - 1;
                    found[1] = ties - before - c1;
                }
                __syncthreads();
                least |= (uint32_t)found[0] << shift;
                ties = found[1];
                __syncthreads();
                shift = next;
            }
        }
        // ---- places, in the order of the tokens: four tokens to a thread
        int32_t *index = a.index + (seq * a.kv_heads + head) * a.keep;
        int sure_before = 0, ties_before = 0;
        auto entry = [&](int t0) { return t0 < held ? page_of(t0 / kPage) : -1; };
        int id = entry(4 * tid), id1 = entry(4 * (tid + kChooseThreads));   // of this turn and the next
        float4 w4 = weights4(max(id, 0), 4 * tid);
        for (int base = 0; base < held; base += 4 * kChooseThreads) {
            const int t0 = base + 4 * tid;
            const int id2 = entry(t0 + 8 * kChooseThreads);
            const float4 next = weights4(max(id1, 0), t0 + 4 * kChooseThreads);
            uint32_t sure = 0, tie = 0;   // bits of the four tokens
            if (id >= 0) {
                const float w[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (t0 + e >= held) continue;
                    const uint32_t o = order_of(w[e]);
                    if (kept == there || spared(t0 + e) || (choose && o > least)) sure |= 1u << e;
                    else if (choose && o == least) tie |= 1u << e;
                }
            }
            const uint32_t counts = (uint32_t)__popc(sure) << 16 | (uint32_t)__popc(tie);
            const uint32_t up = wave_scan(counts);
            if (lane == 63) scan[1][wave] = up;
            __syncthreads();
            uint32_t off = up - counts, all = 0;   // 4096 of each at most
            for (int w = 0; w < kChooseWaves; ++w) {
                if (w < wave) off += scan[1][w];
                all += scan[1][w];
            }
            int s = sure_before + (int)(off >> 16), t = ties_before + (int)(off & 0xffffu);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const bool is_tie = tie >> e & 1, in = (sure >> e & 1) || (is_tie && t < ties);
                const int to = s + min(t, ties);
                if (in && to < kept) index[to] = t0 + e;   // (always, unless the weights change meanwhile)
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
        for (int i = kept + tid; i < a.keep; i += kChooseThreads) index[i] = -1;
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

hipError_t launch_kv4_evict(const EvictArgs &a, int dim, hipStream_t st) {
    constexpr int64_t kMost = 1 << 21;   // workgroups; more units take turns
    const int64_t heads = a.n_seqs * a.kv_heads;
    hipLaunchKernelGGL(evict_choose_kernel, dim3((unsigned)std::min(heads, kMost)), dim3(kChooseThreads), 0, st, a,
                       heads);
    const int pages = (a.keep + kPage - 1) / kPage;
    const int64_t units = heads * pages;
    const dim3 g((unsigned)std::min(units, kMost)), t(kMoveThreads);
    if (dim == 64) hipLaunchKernelGGL((evict_move_kernel<64>), g, t, 0, st, a, pages, units);
    else if (dim == 128) hipLaunchKernelGGL((evict_move_kernel<128>), g, t, 0, st, a, pages, units);
    else hipLaunchKernelGGL((evict_move_kernel<256>), g, t, 0, st, a, pages, units);
    return hipGetLastError();
}

}  // namespace bitnet
