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
};

// Order of a weight among unsigned numbers: a NaN like -inf, -0 like 0.
NVFP4_DEV uint32_t select_order(float w)
{
    uint32_t u = __float_as_uint(w);
    u = w != w ? 0xFF800000u : (u == 0x80000000u ? 0u : u);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// The key of token t of a sequence and KV head; after: the position behind the newest.  A token in a page
// that is none of the cache's is the first to go.
NVFP4_DEV uint32_t select_key(const SelectArgs& s, const int32_t* table, int h, int t, int64_t after)
{
    const int i = attn_page(s.a, t), page = table[i];
    if (page < 0 || page >= s.a.num_pages) {
        raise_error(NVFP4_ERR_RANGE);
        return 0;
    }
    const int64_t slot = (int64_t)page * s.a.page + (t - i * s.a.page);
    const int64_t pos = s.positions ? s.positions[h * s.ld_pos + slot] : t;
    const uint32_t key = select_order(s.weights[h * s.ld_w + slot]);
    return pos < s.sinks || pos >= after - s.recent ? 0xFFFFFFFFu : key;
}

constexpr int kSelectThreads = 1024;

// A workgroup a sequence and KV head (blockIdx.x: sequence * kv_heads + head),
// which holds the first HELD keys in shared memory and reads the others again.
template <int HELD>
__global__ void __launch_bounds__(kSelectThreads)
select_kernel(SelectArgs s)
{
    __shared__ uint32_t keys[HELD];
    __shared__ uint32_t hist[2048];
    __shared__ int wave_sum[16][4];
    __shared__ int found[2];
    const int b = blockIdx.x / s.a.kv_heads, h = blockIdx.x - b * s.a.kv_heads, tid = threadIdx.x, lane = tid & 63;
    const int wave = uniform(tid >> 6);
    const int32_t* table = s.a.table + b * s.a.ld_table;
    const int given = s.a.kv_lens[b];
    const int64_t most = (int64_t)s.a.pages * s.a.page;
    const int L = given < 0 ? 0 : (given > most ? (int)most : given);
    if (tid == 0 && h == 0) {
        s.lens[b] = L < s.keep ? L : s.keep;
        if (L != given)
            raise_error(NVFP4_ERR_RANGE);
    }
    int32_t* moves = s.moves + ((int64_t)b * s.a.kv_heads + h) * s.cap * 2;
    int count = 0;  // moves
    if (L > s.keep) {
        const int64_t after = s.positions ? (int64_t)s.next[b] : (int64_t)L;
        auto key = [&](int t) { return t < HELD ? keys[t] : select_key(s, table, h, t, after); };
        for (int t = tid; t < L && t < HELD; t += kSelectThreads)
            keys[t] = select_key(s, table, h, t, after);
        // ---- the smallest key that stays, and how many of its equals do
        uint32_t prefix = 0;
        int need = s.keep;
#pragma unroll
        for (int pass = 0; pass < 3; pass++) {
            const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0), bits = pass == 2 ? 10 : 11;
            hist[tid] = hist[tid + 1024] = 0;
            __syncthreads();
            for (int t = tid; t < L; t += kSelectThreads) {
                const uint32_t k = key(t);
                if (pass == 0 || (k >> (shift + bits)) == prefix)
                    atomicAdd(&hist[(k >> shift) & ((1u << bits) - 1)], 1u);
            }
            __syncthreads();
            // sums from the top: this thread's bins are top and top - 1
            const int top = 2047 - 2 * tid;
            const int c0 = hist[top], c1 = hist[top - 1];
            int sum = c0 + c1;
#pragma unroll
            for (int off = 1; off < 64; off <<= 1) {
                const int x = __shfl_up(sum, off, 64);
                sum += lane >= off ? x : 0;
            }
            if (lane == 63)
                wave_sum[wave][0] = sum;
            __syncthreads();
            int before = sum - c0 - c1;
            for (int i = 0; i < wave; i++)
                before += wave_sum[i][0];
            if (before < need && need <= before + c0 + c1) {
                const bool first = need <= before + c0;
                found[0] = first ? top : top - 1;
                found[1] = need - before - (first ? 0 : c0);
            }
            __syncthreads();
            prefix = prefix << bits | (uint32_t)found[0];
            need = found[1];
        }
        // ---- each wave a run of tokens: larger and equal keys, in all and below `keep`
        const int per = ((L + 1023) / 1024) * 64;
        const int t0 = wave * per, t1 = t0 + per < L ? t0 + per : L;
        int gt = 0, eq = 0, gt_low = 0, eq_low = 0;
        for (int t = t0; t < t1; t += 64) {
            const uint32_t k = t + lane < t1 ? key(t + lane) : 0;
            const uint64_t in = __ballot(t + lane < t1), low = __ballot(t + lane < s.keep);
            const uint64_t g = __ballot(k > prefix) & in, e = __ballot(k == prefix) & in;
            gt += __builtin_popcountll(g);
            eq += __builtin_popcountll(e);
            gt_low += __builtin_popcountll(g & low);
            eq_low += __builtin_popcountll(e & low);
        }
        if (lane == 0) {
            wave_sum[wave][0] = gt;
            wave_sum[wave][1] = eq;
            wave_sum[wave][2] = gt_low;
            wave_sum[wave][3] = eq_low;
        }
        __syncthreads();
        gt = eq = gt_low = eq_low = 0;
        for (int i = 0; i < 16; i++) {
            gt += i < wave ? wave_sum[i][0] : 0;
            eq += i < wave ? wave_sum[i][1] : 0;
            gt_low += wave_sum[i][2];
            eq_low += wave_sum[i][3];
        }
        const int stay = gt_low + (eq_low < need ? eq_low : need);  // kept tokens below `keep`
        count = s.keep - stay;
        int kept = gt + (eq < need ? eq : need);  // before t
        for (int t = t0; t < t1; t += 64) {
            const int me = t + lane;
            const uint32_t k = me < t1 ? key(me) : 0;
            const uint64_t lower = (1ull << lane) - 1;
            const uint64_t e = __ballot(me < t1 && k == prefix);
            const bool mine = me < t1 && (k > prefix || (k == prefix && eq + __builtin_popcountll(e & lower) < need));
            const uint64_t all = __ballot(mine);
            const int rank = kept + __builtin_popcountll(all & lower);
            if (me < t1 && me < s.keep && !mine && me - rank < s.cap)
                moves[2 * (me - rank) + 1] = me;
            if (mine && me >= s.keep && rank - stay < s.cap)
                moves[2 * (rank - stay)] = me;
            eq += __builtin_popcountll(e);
            kept += __builtin_popcountll(all);
        }
    }
    for (int i = count + tid; i < s.cap; i += kSelectThreads)
        moves[2 * i] = moves[2 * i + 1] = -1;
}

// ---------------------------------------------------------------------------
// Moves.  A cached token of one KV head is cut into units: 16 bytes of codes
// each, then its scales, its weight and its position.
// ---------------------------------------------------------------------------
struct MoveArgs {
    AttnArgs a;           // table, pages, kv_heads
    uint8_t* codes[2];    // K, V
    uint8_t* scales[2];
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
    if (u < 2 * m.code_units) {
        const int which = u >= m.code_units;
        *bytes = 16;
        return (which ? m.codes[1] : m.codes[0]) + row * (m.dim / 2) + (u - which * m.code_units) * 16;
    }
    u -= 2 * m.code_units;
    if (u < 2 * m.scale_units) {
        const int which = u >= m.scale_units;
        *bytes = m.scale_unit;
        return (which ? m.scales[1] : m.scales[0]) + row * (m.dim / 16) + (u - which * m.scale_units) * m.scale_unit;
    }
    u -= 2 * m.scale_units;
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
// branch parts them.  blockIdx.x: sequence * kv_heads + head, blockIdx.y: a share
// of the units.
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

// Long lists, whose sources nobody writes: `lanes` lanes a move.  blockIdx.x:
// sequence * kv_heads + head, blockIdx.y: a share of the moves.
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
