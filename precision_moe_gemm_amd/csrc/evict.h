// evict.h -- which cached tokens a sequence keeps when it passes its budget,
// and moves of cached tokens within their sequence (the cache of page
// "Qwen3.8-2.4T-A95B-NVFP4").
//
// A KV head of a sequence keeps the `keep` tokens with the largest keys: those
// that are kept anyway first (the first and the most recent positions), then by
// weight, and of equal ones the one at the lowest place.  Nothing is sorted:
// three counts of 11, 11 and 10 bits of the key give the smallest key that
// stays, and one pass in the tokens' order gives the gaps among the first
// `keep` places and, as many, the kept tokens behind them.  The i-th of these
// goes to the i-th gap: rows that stay where they are cost nothing, and no
// move's source is another's destination.
//
// Counting is bound by its steps and not by bytes: 64 sequences of 8 KV heads
// and 2064 tokens take 12.2 us (8.5 MB, 1.7 us at the rate of a copy), 16 of up to
// 16000 tokens 18.3: two dependent reads, six passes over keys in shared memory
// and their barriers.
#pragma once
#include "attn.h"

namespace nvfp4 {

struct SelectArgs {
    AttnArgs a;                // kv_lens, table, pages
    const float* weights;      // [kv_heads, tokens], row stride ld_w
    int64_t ld_w;
    const int32_t* positions;  // the same of the tokens' positions; null: their places
    int64_t ld_pos;
    const int32_t* next;       // [seqs] the position after the newest (with positions)
    int keep, sinks, recent;
    int32_t* moves;            // [seqs, kv_heads, cap, 2]
    int cap;
    int32_t* lens;             // [seqs]
    // longer rows: [list, pages * page] keys, and those with the last one's first bits (a share's at its tokens)
    uint32_t* keys;
    uint32_t* some;
    uint32_t* counts;             // [list, share, 2048]
    uint32_t* coarse;             // [list, share, 64]
    struct SelectShare* share;    // [list, share]
    struct SelectFound* found;    // [list]
    int shares, span;             // tokens of a share: a multiple of four
};

// Order of a weight among unsigned numbers: a NaN like -inf, -0 like 0.
NVFP4_DEV uint32_t select_order(float w)
{
    uint32_t u = __float_as_uint(w);
    u = w != w ? 0xFF800000u : (u == 0x80000000u ? 0u : u);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// One sequence and KV head.
struct SelectList {
    const int32_t* table;
    int b, h, tokens;
    int64_t after;  // the position behind the newest
    bool cut;       // the length was out of range
};

NVFP4_DEV SelectList select_list(const SelectArgs& s, int list)
{
    SelectList l;
    l.b = list / s.a.kv_heads;
    l.h = list - l.b * s.a.kv_heads;
    l.table = s.a.table + l.b * s.a.ld_table;
    const int given = s.a.kv_lens[l.b];
    const int64_t most = (int64_t)s.a.pages * s.a.page;
    l.tokens = given < 0 ? 0 : (given > most ? (int)most : given);
    l.cut = l.tokens != given;
    l.after = s.positions ? (int64_t)s.next[l.b] : (int64_t)l.tokens;
    return l;
}

// Keys of the list's tokens t0 + i * step, i < N, below `end`: put(token, key).  The loads of all of them are under
// way together (a chain of two each: 16 x 16000 tokens one by one took 23 us).  A token in a page that is none
// of the cache's is the first to go.
template <int N, class Put>
NVFP4_DEV void select_keys(const SelectArgs& s, const SelectList& l, int t0, int step, int end, Put put)
{
    int page[N], place[N];
#pragma unroll
    for (int i = 0; i < N; i++) {
        const int t = t0 + i * step < end ? t0 + i * step : end - 1;
        const int p = attn_page(s.a, t);
        place[i] = t - p * s.a.page;
        page[i] = l.table[p];
    }
    float w[N];
    int pos[N];
    bool bad = false;
#pragma unroll
    for (int i = 0; i < N; i++) {
        const bool ok = page[i] >= 0 && page[i] < s.a.num_pages;
        bad |= !ok;
        const int64_t slot = (int64_t)(ok ? page[i] : 0) * s.a.page + place[i];
        w[i] = s.weights[l.h * s.ld_w + slot];
        pos[i] = s.positions ? s.positions[l.h * s.ld_pos + slot] : t0 + i * step;
        place[i] = ok;
    }
#pragma unroll
    for (int i = 0; i < N; i++) {
        const uint32_t key = pos[i] < s.sinks || pos[i] >= l.after - s.recent ? 0xFFFFFFFFu : select_order(w[i]);
        if (t0 + i * step < end)
            put(t0 + i * step, place[i] ? key : 0u);
    }
    if (bad)
        raise_error(NVFP4_ERR_RANGE);
}

// The sum of the lanes up to this one.
template <int CTRL, int ROWS>
NVFP4_DEV int add_dpp(int v)
{
    return v + __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xF, true);
}
NVFP4_DEV int wave_sum_below(int v)
{
    v = add_dpp<0x111, 0xF>(v);  // row_shr:1
    v = add_dpp<0x112, 0xF>(v);  // row_shr:2
    v = add_dpp<0x114, 0xF>(v);  // row_shr:4
    v = add_dpp<0x118, 0xF>(v);  // row_shr:8
    v = add_dpp<0x142, 0xA>(v);  // row_bcast:15
    return add_dpp<0x143, 0xC>(v);  // row_bcast:31
}
NVFP4_DEV int wave_sum(int v) { return __builtin_amdgcn_readlane(wave_sum_below(v), 63); }

// f(t, four keys) for every t0 + i * step below `end`; eight loads are under way together.
template <class F>
NVFP4_DEV void select_each(const uint32_t* keys, int t0, int step, int end, F f)
{
    constexpr int N = 8;
    for (; t0 < end; t0 += N * step) {
        u32x4 k[N];
#pragma unroll
        for (int i = 0; i < N; i++)
            if (t0 + i * step < end)
                k[i] = *(const u32x4*)(keys + t0 + i * step);  // (their space is a multiple of four)
#pragma unroll
        for (int i = 0; i < N; i++)
            if (t0 + i * step < end)
                f(t0 + i * step, k[i]);
    }
}

// What the waves of a workgroup tell each other.
template <int WAVES>
struct SelectShared {
    int wave[WAVES][4];
    int digit, need;
};

// The bin, from the top, in which the need-th key lies, and the how-manieth of the bin it is.  c: the counts of
// bins top, top - 1, ... (BINS per thread, thread 0 from the highest on).
template <int THREADS, int BINS>
NVFP4_DEV void select_digit(const int (&c)[BINS], SelectShared<THREADS / 64>& sh, int* digit, int* need)
{
    const int tid = threadIdx.x, wave = tid >> 6, top = BINS * (THREADS - tid) - 1;
    int mine = 0;
#pragma unroll
    for (int i = 0; i < BINS; i++)
        mine += c[i];
    const int sum = wave_sum_below(mine);
    if ((tid & 63) == 63)
        sh.wave[wave][0] = sum;
    __syncthreads();
    int before = sum - mine;
#pragma unroll
    for (int i = 0; i < THREADS / 64; i++)
        before += i < wave ? sh.wave[i][0] : 0;
    if (before < *need && *need <= before + mine) {
        int at = 0;
#pragma unroll
        for (int j = 0; j + 1 < BINS; j++)
            if (at == j && *need > before + c[j]) {
                before += c[j];
                at = j + 1;
            }
        sh.digit = top - at;
        sh.need = *need - before;
    }
    __syncthreads();
    *digit = sh.digit;
    *need = sh.need;
}

// Tokens among keys[a, b) (a and the runs multiples of four), each wave a run of them: larger and equal keys than
// `last` before this wave's run and in all, and the same below `keep`.
struct SelectCount {
    int t0, t1;                        // this wave's run
    int gt, eq;                        // before it
    int all_gt, all_eq, low_gt, low_eq;
};

template <int THREADS>
NVFP4_DEV SelectCount select_count(const uint32_t* keys, int a, int b, uint32_t last, int keep,
                                   SelectShared<THREADS / 64>& sh)
{
    const int lane = threadIdx.x & 63, wave = uniform((int)(threadIdx.x >> 6));
    const int per = (b - a + 4 * THREADS - 1) / (4 * THREADS) * 256;
    SelectCount c{};
    c.t0 = a + wave * per;
    c.t1 = c.t0 + per < b ? c.t0 + per : b;
    int gt = 0, eq = 0, gt_low = 0, eq_low = 0;
    for (int u = c.t0; u < c.t1; u += 1 << 14) {
        const int u1 = u + (1 << 14) < c.t1 ? u + (1 << 14) : c.t1;
        int all = 0, low = 0;  // larger ones, and equal ones times 2^16
        select_each(keys, u + 4 * lane, 256, u1, [&](int t, u32x4 k) {
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const int x = t + i < u1 ? (k[i] > last ? 1 : (k[i] == last ? 0x10000 : 0)) : 0;
                all += x;
                low += t + i < keep ? x : 0;
            }
        });
        all = wave_sum(all);
        low = wave_sum(low);
        gt += all & 0xFFFF;
        eq += all >> 16;
        gt_low += low & 0xFFFF;
        eq_low += low >> 16;
    }
    if (lane == 0) {
        sh.wave[wave][0] = gt;
        sh.wave[wave][1] = eq;
        sh.wave[wave][2] = gt_low;
        sh.wave[wave][3] = eq_low;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < THREADS / 64; i++) {
        c.gt += i < wave ? sh.wave[i][0] : 0;
        c.eq += i < wave ? sh.wave[i][1] : 0;
        c.all_gt += sh.wave[i][0];
        c.all_eq += sh.wave[i][1];
        c.low_gt += sh.wave[i][2];
        c.low_eq += sh.wave[i][3];
    }
    return c;
}

// The moves of this wave's run of tokens: the gaps below `keep`, and the kept tokens behind.  need: how many of
// the keys equal to `last` stay; stay: how many tokens below `keep` do.  (gt and eq count from token 0 on.)
NVFP4_DEV void select_moves(const SelectArgs& s, int32_t* moves, const uint32_t* keys, const SelectCount& c,
                            uint32_t last, int need, int stay)
{
    constexpr int N = 8;
    const int lane = threadIdx.x & 63;
    int gt = c.gt, eq = c.eq;
    for (int u = c.t0; u < c.t1; u += 256 * N) {
        u32x4 k[N];
#pragma unroll
        for (int j = 0; j < N; j++) {
            k[j] = (u32x4){0, 0, 0, 0};
            if (u + 256 * j + 4 * lane < c.t1)
                k[j] = *(const u32x4*)(keys + u + 256 * j + 4 * lane);
        }
#pragma unroll
        for (int j = 0; j < N; j++) {  // gt, eq: before these 256
            if (u + 256 * j >= c.t1)
                break;
            const int t = u + 256 * j + 4 * lane;
            int mine = 0;
#pragma unroll
            for (int i = 0; i < 4; i++)
                mine += t + i < c.t1 ? (k[j][i] > last ? 1 : (k[j][i] == last ? 0x10000 : 0)) : 0;
            const int sum = wave_sum_below(mine), whole = __builtin_amdgcn_readlane(sum, 63);
            int g = gt + ((sum - mine) & 0xFFFF), e = eq + ((sum - mine) >> 16);
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const bool in = t + i < c.t1, equal = in && k[j][i] == last;
                const int rank = g + (e < need ? e : need);  // kept tokens before t + i
                const bool keep = in && (k[j][i] > last || (equal && e < need));
                if (in && t + i < s.keep && !keep && t + i - rank < s.cap)
                    moves[2 * (t + i - rank) + 1] = t + i;
                if (keep && t + i >= s.keep && rank - stay < s.cap)
                    moves[2 * (rank - stay)] = t + i;
                g += in && k[j][i] > last;
                e += equal;
            }
            gt += whole & 0xFFFF;
            eq += whole >> 16;
        }
    }
}

// A workgroup a sequence and KV head (blockIdx.x: sequence * kv_heads + head),
// for rows of the table of up to HELD tokens: its keys are in shared memory, 16
// KB with 256 threads (several workgroups a CU) or 128 KB with 1024.
template <int THREADS, int HELD>
__global__ void __launch_bounds__(THREADS)
select_kernel(SelectArgs s)
{
    constexpr int kBins = 2048 / THREADS;
    __shared__ __attribute__((aligned(16))) uint32_t keys[HELD];
    __shared__ uint32_t hist[2048];
    __shared__ SelectShared<THREADS / 64> sh;
    const int tid = threadIdx.x;
    const SelectList l = select_list(s, blockIdx.x);
    const int L = l.tokens;
    if (tid == 0 && l.h == 0) {
        s.lens[l.b] = L < s.keep ? L : s.keep;
        if (l.cut)
            raise_error(NVFP4_ERR_RANGE);
    }
    int32_t* moves = s.moves + (int64_t)blockIdx.x * s.cap * 2;
    int count = 0;  // moves
    if (L > s.keep) {
        for (int t = tid; t < L; t += 8 * THREADS)
            select_keys<8>(s, l, t, THREADS, L, [&](int i, uint32_t k) { keys[i] = k; });
        // ---- the smallest key that stays, and how many of its equals do
        uint32_t last = 0;
        int need = s.keep;
#pragma unroll
        for (int pass = 0; pass < 3; pass++) {
            const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0), bits = pass == 2 ? 10 : 11;
#pragma unroll
            for (int i = 0; i < kBins; i++)
                hist[i * THREADS + tid] = 0;
            __syncthreads();
            select_each(keys, 4 * tid, 4 * THREADS, L, [&](int t, u32x4 k) {
#pragma unroll
                for (int i = 0; i < 4; i++)
                    if (t + i < L && (pass == 0 || (k[i] >> (shift + bits)) == last))
                        atomicAdd(&hist[(k[i] >> shift) & ((1u << bits) - 1)], 1u);
            });
            __syncthreads();
            int c[kBins], digit;
#pragma unroll
            for (int i = 0; i < kBins; i++)
                c[i] = hist[2047 - kBins * tid - i];
            select_digit<THREADS>(c, sh, &digit, &need);
            last = last << bits | (uint32_t)digit;
        }
        const SelectCount c = select_count<THREADS>(keys, 0, L, last, s.keep, sh);
        const int stay = c.low_gt + (c.low_eq < need ? c.low_eq : need);  // kept tokens below `keep`
        count = s.keep - stay;
        select_moves(s, moves, keys, c, last, need, stay);
    }
    for (int i = count + tid; i < s.cap; i += THREADS)
        moves[2 * i] = moves[2 * i + 1] = -1;
}

// ---- longer rows: shares of a list's tokens by workgroups of their own (one workgroup reads what others wrote
// at 50 GB/s: five passes over 131072 keys took it 107 us), in four launches.  16384 of 131072 tokens, 4 KV heads:
// 4.8 + 6.5 + 7.6 + 6.0 us, each little more than a launch and its chain of reads (342 by one workgroup a head with
// sums across workgroups in between).  blockIdx.x: list, blockIdx.y: share.
constexpr int kSelectThreads = 512;
constexpr int kSelectSpan = 4096;   // tokens of a share, at least
constexpr int kSelectShares = 256;  // shares of a list, at most
constexpr int kSelectHeld = 32768;  // keys that fit the shared memory

// What a share tells: keys with larger first 11 bits than the last one that stays, in all and below `keep`; the
// number with the same; of these the larger and equal ones.
struct SelectShare {
    int gt, gt_low, some;
    int gt2, gt2_low, eq2, eq2_low, pad;
};
struct SelectFound {
    uint32_t last;
    int need;
};

NVFP4_DEV int64_t select_places(const SelectArgs& s) { return (int64_t)s.a.pages * s.a.page; }

// 1: the keys, and how often each value of their first 6 and 11 bits comes.
__global__ void __launch_bounds__(kSelectThreads)
select_keys_kernel(SelectArgs s)
{
    __shared__ uint32_t hist[2048];
    const SelectList l = select_list(s, blockIdx.x);
    if (l.tokens <= s.keep)
        return;
    const int tid = threadIdx.x;
#pragma unroll
    for (int i = 0; i < 4; i++)
        hist[i * kSelectThreads + tid] = 0;
    __syncthreads();
    uint32_t* keys = s.keys + blockIdx.x * select_places(s);
    const int a = blockIdx.y * s.span, b = l.tokens - a < s.span ? l.tokens : a + s.span;
    for (int t = a + tid; t < b; t += 8 * kSelectThreads)
        select_keys<8>(s, l, t, kSelectThreads, b, [&](int i, uint32_t k) {
            keys[i] = k;
            atomicAdd(&hist[k >> 21], 1u);
        });
    __syncthreads();
    const int64_t share = (int64_t)blockIdx.x * s.shares + blockIdx.y;
    u32x4 c;
#pragma unroll
    for (int i = 0; i < 4; i++)
        c[i] = hist[4 * tid + i];
    *(u32x4*)(s.counts + share * 2048 + 4 * tid) = c;
    // eight threads hold the 32 bins of one coarse value
    int sum = c.x + c.y + c.z + c.w;
    sum += __shfl_xor(sum, 1, 64);
    sum += __shfl_xor(sum, 2, 64);
    sum += __shfl_xor(sum, 4, 64);
    if ((tid & 7) == 0)
        s.coarse[share * 64 + (tid >> 3)] = sum;
}

// 2: the first 11 bits of the last key that stays (every share finds them by itself), and the share's keys with
// these bits: the other bits, bit 31 for tokens below `keep`.
__global__ void __launch_bounds__(kSelectThreads)
select_some_kernel(SelectArgs s)
{
    __shared__ int part[kSelectThreads];
    __shared__ int found[2], some, wave_gt[kSelectThreads / 64][2];
    const SelectList l = select_list(s, blockIdx.x);
    if (l.tokens <= s.keep)
        return;
    const int tid = threadIdx.x, lane = tid & 63;
    const int64_t share = (int64_t)blockIdx.x * s.shares + blockIdx.y, list = (int64_t)blockIdx.x * s.shares;
    int digit = 0, need = s.keep;
    // the coarse value among 64, then the fine one among its 32: counts are added by shares, then by threads
#pragma unroll
    for (int level = 0; level < 2; level++) {
        const int bins = level == 0 ? 64 : 32, bin = tid % bins;
        int c = 0;
        for (int j = tid / bins; j < s.shares; j += kSelectThreads / bins)
            c += level == 0 ? s.coarse[(list + j) * 64 + bin] : s.counts[(list + j) * 2048 + 32 * digit + bin];
        part[tid] = c;
        __syncthreads();
        if (tid < 64) {
            // lane i: bin bins - 1 - i
            int n = 0;
#pragma unroll
            for (int j = 0; j < kSelectThreads; j += bins)
                n += tid < bins ? part[j + bins - 1 - tid] : 0;
            const int before = wave_sum_below(n) - n;
            if (before < need && need <= before + n) {
                found[0] = bins - 1 - tid;
                found[1] = need - before;
            }
        }
        __syncthreads();
        digit = 32 * digit + found[0];
        need = found[1];
        if (tid == 0)
            some = 0;
        __syncthreads();
    }
    const uint32_t first = digit;
    const int a = blockIdx.y * s.span, b = l.tokens - a < s.span ? l.tokens : a + s.span;
    const uint32_t* keys = s.keys + blockIdx.x * select_places(s);
    uint32_t* out = s.some + blockIdx.x * select_places(s) + a;
    int gt = 0, low = 0;
    select_each(keys, a + 4 * tid, 4 * kSelectThreads, b, [&](int t, u32x4 k) {
        int mine = 0;
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const bool in = t + i < b, more = in && (k[i] >> 21) > first;
            gt += more;
            low += more && t + i < s.keep;
            mine += in && (k[i] >> 21) == first;
        }
        if (mine > 0) {
            int at = atomicAdd(&some, mine);
#pragma unroll
            for (int i = 0; i < 4; i++)
                if (t + i < b && (k[i] >> 21) == first)
                    out[at++] = (k[i] & 0x1FFFFFu) | (t + i < s.keep ? 0x80000000u : 0u);
        }
    });
    gt = wave_sum(gt);
    low = wave_sum(low);
    if (lane == 0) {
        wave_gt[tid >> 6][0] = gt;
        wave_gt[tid >> 6][1] = low;
    }
    __syncthreads();
    if (tid == 0) {
        gt = low = 0;
#pragma unroll
        for (int i = 0; i < kSelectThreads / 64; i++) {
            gt += wave_gt[i][0];
            low += wave_gt[i][1];
        }
        SelectShare* r = s.share + share;
        r->gt = gt;
        r->gt_low = low;
        r->some = some;
        if (blockIdx.y == 0)
            s.found[blockIdx.x] = SelectFound{first << 21, need};
    }
}

// 3: the last key that stays, and how many of its equals do, from the keys that were collected; a workgroup a
// list, a wave a share at a time.
__global__ void __launch_bounds__(1024)
select_last_kernel(SelectArgs s)
{
    __shared__ uint32_t held[kSelectHeld];
    __shared__ uint32_t hist[2048];
    __shared__ int start[kSelectShares + 1];
    __shared__ SelectShared<16> sh;
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    const SelectList l = select_list(s, blockIdx.x);
    if (tid == 0 && l.h == 0) {
        s.lens[l.b] = l.tokens < s.keep ? l.tokens : s.keep;
        if (l.cut)
            raise_error(NVFP4_ERR_RANGE);
    }
    if (l.tokens <= s.keep)
        return;
    SelectShare* share = s.share + (int64_t)blockIdx.x * s.shares;
    const uint32_t* some = s.some + blockIdx.x * select_places(s);
    // where the keys of each share begin, one after the other
    if (tid < 64) {
        int sum = 0;
        for (int j = 0; j < s.shares; j += 64) {
            const int n = j + lane < s.shares && (j + lane) * (int64_t)s.span < l.tokens ? share[j + lane].some : 0;
            const int to = sum + wave_sum_below(n);
            if (j + lane < s.shares)
                start[j + lane + 1] = to;
            sum = __builtin_amdgcn_readlane(to, 63);
        }
        if (lane == 0)
            start[0] = 0;
    }
    __syncthreads();
    const bool fits = start[s.shares] <= kSelectHeld;
    // f(key) for the wave's lanes' keys of share j
    auto each = [&](int j, auto f) {
        const int n = start[j + 1] - start[j];
        const uint32_t* src = some + (int64_t)j * s.span;
        if (fits) {
            for (int i = lane; i < n; i += 64)
                f(held[start[j] + i]);
        } else {
            for (int i = lane; i < n; i += 64)
                f(src[i]);
        }
    };
    if (fits)
        for (int j = wave; j < s.shares; j += 16) {
            const int n = start[j + 1] - start[j];
#pragma unroll 4
            for (int i = lane; i < n; i += 64)
                held[start[j] + i] = some[(int64_t)j * s.span + i];
        }
    SelectFound r = s.found[blockIdx.x];
    uint32_t last = 0;  // its bits below the first 11
#pragma unroll
    for (int pass = 1; pass < 3; pass++) {
        const int shift = pass == 1 ? 10 : 0, bits = pass == 1 ? 11 : 10;
        hist[tid] = hist[tid + 1024] = 0;
        __syncthreads();
        for (int j = wave; j < s.shares; j += 16)
            each(j, [&](uint32_t k) {
                k &= 0x1FFFFFu;
                if (pass == 1 || (k >> 10) == last)
                    atomicAdd(&hist[(k >> shift) & ((1u << bits) - 1)], 1u);
            });
        __syncthreads();
        const int c[2] = {(int)hist[2047 - 2 * tid], (int)hist[2046 - 2 * tid]};
        int digit;
        select_digit<1024>(c, sh, &digit, &r.need);
        last = last << bits | (uint32_t)digit;
    }
    if (tid == 0)
        s.found[blockIdx.x] = SelectFound{r.last | last, r.need};
    for (int j = wave; j < s.shares; j += 16) {
        int gt = 0, eq = 0, gt_low = 0, eq_low = 0;
        each(j, [&](uint32_t k) {
            const bool low = k >> 31, more = (k & 0x1FFFFFu) > last, same = (k & 0x1FFFFFu) == last;
            gt += more;
            eq += same;
            gt_low += more && low;
            eq_low += same && low;
        });
        gt = wave_sum(gt);
        eq = wave_sum(eq);
        gt_low = wave_sum(gt_low);
        eq_low = wave_sum(eq_low);
        if (lane == 0) {
            share[j].gt2 = gt;
            share[j].eq2 = eq;
            share[j].gt2_low = gt_low;
            share[j].eq2_low = eq_low;
        }
    }
}

// 4: the moves of a share's tokens.
__global__ void __launch_bounds__(kSelectThreads)
select_moves_kernel(SelectArgs s)
{
    __shared__ SelectShared<kSelectThreads / 64> sh;
    const int tid = threadIdx.x, lane = tid & 63;
    const SelectList l = select_list(s, blockIdx.x);
    int32_t* moves = s.moves + (int64_t)blockIdx.x * s.cap * 2;
    int count = 0;
    if (l.tokens > s.keep) {
        const SelectFound r = s.found[blockIdx.x];
        // what the shares have, before this one and below `keep` (every wave by itself)
        int gt = 0, eq = 0, gt_low = 0, eq_low = 0;
        for (int j = lane; j < s.shares && j * (int64_t)s.span < l.tokens; j += 64) {
            const SelectShare x = s.share[(int64_t)blockIdx.x * s.shares + j];
            gt += j < (int)blockIdx.y ? x.gt + x.gt2 : 0;
            eq += j < (int)blockIdx.y ? x.eq2 : 0;
            gt_low += x.gt_low + x.gt2_low;
            eq_low += x.eq2_low;
        }
        gt = wave_sum(gt);
        eq = wave_sum(eq);
        gt_low = wave_sum(gt_low);
        eq_low = wave_sum(eq_low);
        const int stay = gt_low + (eq_low < r.need ? eq_low : r.need);
        count = s.keep - stay;
        const int a = blockIdx.y * s.span, b = l.tokens - a < s.span ? l.tokens : a + s.span;
        if (a < b) {
            const uint32_t* keys = s.keys + blockIdx.x * select_places(s);
            SelectCount c = select_count<kSelectThreads>(keys, a, b, r.last, s.keep, sh);
            c.gt += gt;
            c.eq += eq;
            select_moves(s, moves, keys, c, r.last, r.need, stay);
        }
    }
    for (int i = count + blockIdx.y * kSelectThreads + tid; i < s.cap; i += gridDim.y * kSelectThreads)
        moves[2 * i] = moves[2 * i + 1] = -1;
}

// ---------------------------------------------------------------------------
// Moves.  A cached token of one KV head is cut into units: 16 bytes of codes
// each, then its scales, its weight and its position.  A move's rows lie
// anywhere: of D = 256 two runs of 128 bytes, two of 16 and two of 4, so that the
// lines touched are about twice the bytes moved.
// ---------------------------------------------------------------------------
struct MoveArgs {
    AttnArgs a;           // table, pages, kv_heads
    uint8_t* codes[2];    // K, V (one where both lie in the same memory: tensors = 1)
    uint8_t* scales[2];
    int tensors;
    int dim;
    int scale_unit;       // bytes: 16, 8, 4 or 2
    int code_units, scale_units, units;  // of one tensor, of one tensor, in all
    float* weights;       // or null
    int64_t ld_w;
    int32_t* positions;   // or null
    int64_t ld_pos;
    const int32_t* moves;  // [seqs, lists, cap, 2] (source, destination)
    int lists, cap;
};

typedef u32x4 u32x4_a4 __attribute__((aligned(4)));
typedef u32x2 u32x2_a4 __attribute__((aligned(4)));

// The address of unit u of a token's row of KV head h (row: token * kv_heads + h), and its bytes.
NVFP4_DEV uint8_t* move_at(const MoveArgs& m, int u, int64_t token, int h, int* bytes)
{
    const int64_t row = token * m.a.kv_heads + h;
    if (u < m.tensors * m.code_units) {
        const int which = u >= m.code_units;
        *bytes = 16;
        return (which ? m.codes[1] : m.codes[0]) + row * (m.dim / 2) + (u - which * m.code_units) * 16;
    }
    u -= m.tensors * m.code_units;
    if (u < m.tensors * m.scale_units) {
        const int which = u >= m.scale_units;
        *bytes = m.scale_unit;
        return (which ? m.scales[1] : m.scales[0]) + row * (m.dim / 16) + (u - which * m.scale_units) * m.scale_unit;
    }
    u -= m.tensors * m.scale_units;
    *bytes = 4;
    return u == 0 && m.weights ? (uint8_t*)(m.weights + h * m.ld_w + token) : (uint8_t*)(m.positions + h * m.ld_pos + token);
}

NVFP4_DEV u32x4 move_load(const uint8_t* p, int bytes)
{
    u32x4 v = (u32x4){0, 0, 0, 0};
    if (bytes == 16) {
        v = *(const u32x4_a4*)p;
    } else if (bytes == 8) {
        const u32x2 w = *(const u32x2_a4*)p;
        v.x = w.x;
        v.y = w.y;
    } else if (bytes == 4) {
        v.x = *(const uint32_t*)p;
    } else {
        v.x = *(const uint16_t*)p;
    }
    return v;
}

NVFP4_DEV void move_store(uint8_t* p, int bytes, u32x4 v)
{
    if (bytes == 16)
        *(u32x4_a4*)p = v;
    else if (bytes == 8)
        *(u32x2_a4*)p = (u32x2){v.x, v.y};
    else if (bytes == 4)
        *(uint32_t*)p = v.x;
    else
        *(uint16_t*)p = (uint16_t)v.x;
}

// Move i of a list: the cache tokens that it reads and writes; false: none, or not in the sequence's pages.
NVFP4_DEV bool move_of(const MoveArgs& m, int b, int h, int i, int64_t* from, int64_t* to)
{
    const int32_t* e = m.moves + (((int64_t)b * m.lists + (m.lists > 1 ? h : 0)) * m.cap + i) * 2;
    const int src = e[0], dst = e[1];
    if (src < 0)
        return false;
    const int64_t most = (int64_t)m.a.pages * m.a.page;
    bool ok = src < most && dst >= 0 && dst < most;
    if (ok) {
        const int32_t* table = m.a.table + b * m.a.ld_table;
        const int i0 = attn_page(m.a, src), i1 = attn_page(m.a, dst);
        const int p0 = table[i0], p1 = table[i1];
        ok = p0 >= 0 && p0 < m.a.num_pages && p1 >= 0 && p1 < m.a.num_pages;
        *from = (int64_t)p0 * m.a.page + (src - i0 * m.a.page);
        *to = (int64_t)p1 * m.a.page + (dst - i1 * m.a.page);
    }
    if (!ok)
        raise_error(NVFP4_ERR_RANGE);
    return ok;
}

// Short lists: a token that one move writes may be another's source, and is
// read first.  All moves of a unit are in one wave (64 moves, ROUNDS times; or
// 64 / side of them, side by side with other units), which stores when its last
// load is back.  Loads do not depend on whether there is a move, so that no
// branch parts them.  32 lists of 6 moves for 8 KV heads of 128: 4.4 us, the
// launch and three dependent reads.  blockIdx.x: sequence * kv_heads + head,
// blockIdx.y: a share of the units.
constexpr int kMoveTogether = 256;
template <int ROUNDS>
__global__ void __launch_bounds__(256)
move_together_kernel(MoveArgs m, int side)
{
    const int b = blockIdx.x / m.a.kv_heads, h = blockIdx.x - b * m.a.kv_heads, lane = threadIdx.x & 63;
    const int wave = blockIdx.y * 4 + (int)(threadIdx.x >> 6), waves = gridDim.y * 4;
    const int i0 = lane / side, u0 = lane % side;  // neighbouring lanes: neighbouring units of one token
    int64_t from[ROUNDS], to[ROUNDS];
    bool ok[ROUNDS];
#pragma unroll
    for (int r = 0; r < ROUNDS; r++) {
        const int i = i0 + r * 64;
        ok[r] = i < m.cap && move_of(m, b, h, i, &from[r], &to[r]);
        from[r] = ok[r] ? from[r] : 0;
        to[r] = ok[r] ? to[r] : 0;
    }
    for (int u = wave * side + u0; u < m.units; u += waves * side) {
        u32x4 v[ROUNDS];
        int bytes;
#pragma unroll
        for (int r = 0; r < ROUNDS; r++) {
            const uint8_t* p = move_at(m, u, from[r], h, &bytes);
            v[r] = move_load(p, bytes);
        }
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int r = 0; r < ROUNDS; r++)
            if (ok[r])
                move_store(move_at(m, u, to[r], h, &bytes), bytes, v[r]);
    }
}

// Long lists, whose sources nobody writes: `lanes` lanes a move.  14336 moves of 4
// KV heads of 256: 17.9 us, 34 MB read and written (1.9 TB/s; about 60 MB in
// lines).  Four moves of a thread under way at once: no gain (300 moves of 64
// sequences 66 us for 60).  blockIdx.x: sequence * kv_heads + head, blockIdx.y: a
// share of the moves.
__global__ void __launch_bounds__(256)
move_apart_kernel(MoveArgs m, int lanes)
{
    const int b = blockIdx.x / m.a.kv_heads, h = blockIdx.x - b * m.a.kv_heads;
    const int per = 256 / lanes, u0 = threadIdx.x % lanes;
    for (int i = blockIdx.y * per + (int)threadIdx.x / lanes; i < m.cap; i += gridDim.y * per) {
        int64_t from, to;
        if (!move_of(m, b, h, i, &from, &to))
            continue;
        for (int u = u0; u < m.units; u += lanes) {
            int bytes;
            const uint8_t* p = move_at(m, u, from, h, &bytes);
            const u32x4 v = move_load(p, bytes);
            move_store(move_at(m, u, to, h, &bytes), bytes, v);
        }
    }
}

}  // namespace nvfp4
