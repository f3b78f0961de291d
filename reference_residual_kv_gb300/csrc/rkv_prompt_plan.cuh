// rkv_prompt_plan.cuh -- how the rows of packed prompts, or of pieces behind cached text, are dealt
// out to the CTAs of the prompt attention (rkv_prompt_attention.cu).
//
// An item is a tile of up to `tile_tokens` tokens of one sequence for one KV head, and a range of its key
// tiles; its cost is their number.  One CTA reads the lengths and writes the items
//   by cost, the largest first, KV heads innermost: the last ones to start are short;
//   by sequence and KV head, each from its last tile to its first, where K and V are more than
//   stays in L2 and a KV head would otherwise have few CTAs at a time: those that read the same K and V
//   run together;
//   where there are few, the largest ones, as many as are whole rounds of all CTAs (or a round less), as
//   they are, the others cut into parts of L key tiles each: the rounds and L for which the time, taken
//   as (all costs) / CTAs + what the last round of parts leaves idle, is least.  Parts of full length come
//   by their place in the text, so that those that read the same K and V run together.  2048 rows of 32
//   heads behind 129024 keys (256 items of equal cost) take 1790 key tiles' time to a CTA so, 2040 whole.
// Sums of parts are joined in the order of the keys whatever CTA had them: the same lengths give
// the same bits.
#pragma once

#include "rkv_prompt.cuh"

namespace rkv {

struct PromptItem {
    int q_row, tokens;      // first row (token) of the item and its tokens
    int k_row;              // packed: row of K and V that holds key 0; else the sequence
    int first;              // the key that the first token sees last
    int kt0, kt1;           // key tiles
    int slot;               // partial of this part for KV head 0; below 0: the item is whole (-1 - its
                            // sequence's items, where items go by sequence)
    int seq;                // index of its sequence's first item, where items go by sequence
};
static_assert(sizeof(PromptItem) == 32, "two 16-byte loads");
struct PromptJoin { int q_row, tokens, slot, parts; };
struct PromptHead {
    int items;              // for each KV head
    int by_seq;             // items of a sequence in a row for each KV head (else KV heads innermost)
    int next;               // the item to take next
    int joins, slots;
    int pad[3];
};

constexpr int kPromptCtas = 152;
constexpr int kPromptSlots = 4 * kPromptCtas;        // partials at most
// K and V that stay in L2 beside what else is read
constexpr long long kInL2 = 80LL << 20;
constexpr int kItemCost = 2, kPartCost = 4;      // of an item or a part beside its keys, in key tiles of 128
constexpr int kFewItems = 512, kFewRounds = 8;       // parts are considered up to here

constexpr int kPlanBeside = 256;               // sequences whose items k_dense_rows works out

struct PlanArgs {
    const int32_t *start;                      // packed prompts
    const int32_t *len, *n_new;                // pieces: [S], n rows each at most
    int S, rows, n, T;
    int N, tile_tokens, tok, key_bytes, max_slots, max_items, max_joins, ctas;
    PromptHead *head;
    PromptItem *items;
    PromptJoin *joins;
    int32_t *status;
};

struct PromptText { int q_row, n, before, k_row; };      // q_row < 0: packed rows that do not ascend
__device__ __forceinline__ PromptText text_of(const PlanArgs &a, int s)
{
    if (a.start) {
        const int b = __ldg(a.start + s), e = __ldg(a.start + s + 1);
        if (b < 0 || e < b || e > a.rows) {
            set_status(a.status, RKV_ERR_INDEX);
            return PromptText{-1, 0, 0, 0};
        }
        return PromptText{b, e - b, 0, b};
    }
    const int before = __ldg(a.len + s), n = a.n_new ? __ldg(a.n_new + s) : a.n;
    if (before < 0 || n < 0 || n > a.n || before > a.T - n) {
        set_status(a.status, RKV_ERR_INDEX);
        return PromptText{0, 0, 0, 0};
    }
    return PromptText{s * a.n, n, before, s};
}

constexpr int kCands = 32;
constexpr int kFull = 256, kBuckets = 2 * kFull;     // parts of full length by their place, others by cost

template <int THREADS>
struct PlanShared {
    int warps[32], first_tile[THREADS + 1], bucket[kBuckets], cost[kFewItems], sorted[kFewItems], rank[kFewItems];
    PromptText texts[THREADS];
    long long sum_cost, sum_keys;
    float best[kCands];
    int sum_tiles, max_cost, part_len, whole, slots, n_items, n_joins, wrong;
};

template <int THREADS>
__device__ __forceinline__ int plan_scan(int v, int *warps, int &total)      // exclusive
{
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int x = lane_scan(v);
    __syncthreads();
    if (lane == 31) warps[w] = x;
    __syncthreads();
    if (w == 0) warps[lane] = lane_scan(lane < THREADS / 32 ? warps[lane] : 0);
    __syncthreads();
    total = warps[THREADS / 32 - 1];
    return x - v + (w ? warps[w - 1] : 0);
}

// All THREADS threads of one CTA.
template <int THREADS>
__device__ __forceinline__ void prompt_plan(const PlanArgs &a, PlanShared<THREADS> &z)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) {
        z.sum_cost = z.sum_keys = 0;
        z.sum_tiles = z.max_cost = z.part_len = z.whole = z.slots = z.n_items = z.n_joins = z.wrong = 0;
    }
    for (int i = tid; i < kBuckets; i += THREADS) z.bucket[i] = 0;
    __syncthreads();

    // Calls f(x, text, tile, cost, tiles of that text, the text's first x) for every tile x, THREADS texts at a
    // time; fewer texts are read once
    bool have = false;
    int have_total = 0;
    auto each = [&](auto f) {
        int before = 0;
        for (int s0 = 0; s0 < a.S; s0 += THREADS) {
            int total = have_total;
            if (!have) {
                const int s = s0 + tid;
                PromptText t{0, 0, 0, 0};
                if (s < a.S) t = text_of(a, s);
                if (t.q_row < 0) z.wrong = 1;
                const int tiles = (t.n + a.tile_tokens - 1) / a.tile_tokens;
                const int at = plan_scan<THREADS>(tiles, z.warps, total);
                z.texts[tid] = t;
                z.first_tile[tid] = at;
                if (tid == 0) z.first_tile[THREADS] = total;
                __syncthreads();
                if (a.S <= THREADS) {
                    have = true;
                    have_total = total;
                }
            }
            for (int x = tid; x < total; x += THREADS) {
                int lo = 0, hi = min(THREADS, a.S - s0);   // the last text that begins at or before x
                while (hi - lo > 1) {
                    const int mid = (lo + hi) >> 1;
                    if (z.first_tile[mid] <= x) lo = mid;
                    else hi = mid;
                }
                const PromptText &w = z.texts[lo];
                const int tile = x - z.first_tile[lo], last = min(w.n, (tile + 1) * a.tile_tokens);
                f(before + x, w, tile, (w.before + last + a.tok - 1) / a.tok, z.first_tile[lo + 1] - z.first_tile[lo],
                  before + z.first_tile[lo]);
            }
            before += total;
            if (!have) __syncthreads();
        }
    };
    {
        long long cost = 0, keys = 0;
        int n = 0, most = 0;
        each([&](int x, const PromptText &w, int tile, int c, int, int) {
            cost += c;
            ++n;
            most = max(most, c);
            if (tile == 0) keys += w.before + w.n;
            if (x < kFewItems) z.cost[x] = c;
        });
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            cost += __shfl_xor_sync(0xffffffffu, cost, o);
            keys += __shfl_xor_sync(0xffffffffu, keys, o);
        }
        n = __reduce_add_sync(0xffffffffu, n);
        most = __reduce_max_sync(0xffffffffu, most);
        if (lane == 0) {
            atomicAdd((unsigned long long *)&z.sum_cost, (unsigned long long)cost);
            atomicAdd((unsigned long long *)&z.sum_keys, (unsigned long long)keys);
            atomicAdd(&z.sum_tiles, n);
            atomicMax(&z.max_cost, most);
        }
        __syncthreads();
    }
    // Packed rows that do not ascend may be more than the workspace is for: nothing attends
    if (z.wrong || z.sum_tiles == 0) {
        if (tid == 0) *a.head = PromptHead{0, 0, a.ctas, 0, 0, {0, 0, 0}};
        return;
    }
    const int E = z.sum_tiles, N = a.N;
    // parts of a cost: the last one is longer by up to a quarter than the others, or shorter
    auto parts_of = [](int c, int L) { return c <= L + L / 4 ? 1 : (c - L / 4 + L - 1) / L; };
    const bool few = E <= kFewItems && (long long)E * N < kFewRounds * kPromptCtas && a.max_slots > 0 && z.max_cost < 65536;
    if (few) {
        // by cost, equal ones as they come: the same for the same lengths
        for (int x = tid; x < E; x += THREADS) {
            const int c = z.cost[x];
            int r = 0;
            for (int y = 0; y < E; ++y) r += z.cost[y] > c || (z.cost[y] == c && y < x);
            z.rank[x] = r;
            z.sorted[r] = c;
        }
        __syncthreads();
        // a candidate to a warp: rounds of whole items, and L = the largest other item / k
        const int rounds = E * N / kPromptCtas;
        auto whole_of = [&](int i) { return min(E, max(0, rounds - (i >= kCands / 2 && rounds > 0)) * kPromptCtas / N); };
        auto len_of = [&](int i) {
            const int w = whole_of(i), k = rounds > 0 ? i % (kCands / 2) + 1 : i + 1;
            return w < E ? (z.sorted[w] + k - 1) / k : 1;
        };
        for (int i = warp; i < kCands; i += THREADS / 32) {
            const int w = whole_of(i), L = len_of(i);
            const uint32_t inv = 0xffffffffu / (uint32_t)max(L, 2) + 1u;     // quotients of numbers below 2^16 by a multiplication
            int n = 0, cut = 0;
            for (int x = w + lane; x < E; x += 32) {
                const int c = z.sorted[x];
                const int k = c <= L + L / 4 ? 1 : (L < 2 ? c : (int)__umulhi((uint32_t)(c - L / 4 + L - 1), inv));
                n += k;
                cut += k > 1 ? k : 0;
            }
            n = __reduce_add_sync(0xffffffffu, n) * N;
            cut = __reduce_add_sync(0xffffffffu, cut) * N;
            const float unit = 128.0f / a.tok, more = cut ? kPartCost * unit : kItemCost * unit;
            const float all = (float)z.sum_cost * N + kItemCost * unit * (w * N + n - cut) + kPartCost * unit * cut;
            const float t = all / kPromptCtas + (ceilf((float)n / kPromptCtas) - (float)n / kPromptCtas) * (L + more);
            if (lane == 0) z.best[i] = cut > a.max_slots || (cut && L < 4 * unit) ? INFINITY : t;
        }
        __syncthreads();
        if (tid < 32) {
            float t = z.best[tid];
            int best = tid;
#pragma unroll
            for (int o = 16; o; o >>= 1) {
                const float y = __shfl_xor_sync(0xffffffffu, t, o);
                const int b = __shfl_xor_sync(0xffffffffu, best, o);
                if (y < t || (y == t && b < best)) { t = y; best = b; }
            }
            if (tid == 0) {
                z.whole = whole_of(best);
                z.part_len = len_of(best);
            }
        }
        __syncthreads();
    } else {
        if (tid == 0) z.part_len = z.max_cost;
        __syncthreads();
    }
    const int L = z.part_len, whole = z.whole;
    const bool by_seq = !few && z.sum_keys * a.key_bytes > kInL2 && 4LL * a.S * N > kPromptCtas;
    if (by_seq) {
        each([&](int, const PromptText &w, int tile, int c, int tiles, int seq) {
            if (seq + tiles > a.max_items) return;         // lengths that changed under the call
            a.items[seq + tiles - 1 - tile] = PromptItem{w.q_row + tile * a.tile_tokens, min(a.tile_tokens, w.n - tile * a.tile_tokens),
                                                         w.k_row, w.before + tile * a.tile_tokens, 0, c, -1 - tiles, seq};
        });
        if (tid == 0) z.n_items = E;
    } else {
        // parts of full length by their place, others by their cost
        auto bucket_of = [&](int part, int c) {
            return few && c >= L ? min(part, kFull - 1) : kFull + (kFull - 1) - (int)((long long)min(c, L) * (kFull - 1) / L);
        };
        auto parts_here = [&](int x, int c) { return few ? (z.rank[min(x, kFewItems - 1)] < whole ? 0 : parts_of(c, L)) : 1; };
        each([&](int x, const PromptText &, int, int c, int, int) {
            const int parts = parts_here(x, c);
            for (int i = 0; i < parts; ++i) atomicAdd(&z.bucket[bucket_of(i, i + 1 < parts ? L : c - i * L)], 1);
        });
        __syncthreads();
        // exclusive sums over the buckets, kBuckets / THREADS (or one) to a thread
        constexpr int kOwn = (kBuckets + THREADS - 1) / THREADS;
        int own[kOwn], sum = 0, total;
#pragma unroll
        for (int i = 0; i < kOwn; ++i) {
            const int at = tid * kOwn + i;
            own[i] = sum;
            if (at < kBuckets) sum += z.bucket[at];
        }
        const int at0 = whole + plan_scan<THREADS>(sum, z.warps, total);
#pragma unroll
        for (int i = 0; i < kOwn; ++i)
            if (tid * kOwn + i < kBuckets) z.bucket[tid * kOwn + i] = at0 + own[i];
        if (tid == 0) z.n_items = whole + total;
        __syncthreads();
        each([&](int x, const PromptText &w, int tile, int c, int, int) {
            const int parts = parts_here(x, c);
            const int q_row = w.q_row + tile * a.tile_tokens, tokens = min(a.tile_tokens, w.n - tile * a.tile_tokens);
            const int first = w.before + tile * a.tile_tokens;
            if (parts == 0 && z.rank[x] < a.max_items) a.items[z.rank[x]] = PromptItem{q_row, tokens, w.k_row, first, 0, c, -1, 0};
            int slot = -1;
            if (parts > 1) {
                const int j = atomicAdd(&z.n_joins, 1);
                slot = atomicAdd(&z.slots, parts * N);
                if (j >= a.max_joins || slot + parts * N > a.max_slots) return;
                a.joins[j] = PromptJoin{q_row, tokens, slot, parts};
            }
            for (int i = 0; i < parts; ++i) {
                const int to = i + 1 < parts ? (i + 1) * L : c;
                const int at = atomicAdd(&z.bucket[bucket_of(i, to - i * L)], 1);
                if (at >= a.max_items) return;
                a.items[at] = PromptItem{q_row, tokens, w.k_row, first, i * L, to, parts > 1 ? slot + i * N : -1, 0};
            }
        });
    }
    __syncthreads();
    if (tid == 0)
        *a.head = PromptHead{min(z.n_items, a.max_items), by_seq, a.ctas, min(z.n_joins, a.max_joins), z.slots, {0, 0, 0}};
}

}  // namespace rkv
