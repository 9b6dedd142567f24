// weigh.h -- the attention weight that each cached token receives (the cache
// of page "Qwen3.8-2.4T-A95B-NVFP4"), for caches whose length is bounded by
// giving up the tokens that received least.
//
//   w'[h, t] = w[h, t] + sum over query rows r and heads j of KV head h of
//              exp(scale q[r, j] . k[t, h] - lse[r, j])
//
// with lse from the attention over the same tokens, so that a weight is one
// pass over K alone: no maximum, no rescaling, and tokens do not depend on
// each other.  Every (token, KV head) is summed by one wave (or, split over
// its rows, by a fixed number of them in a fixed order): results do not depend
// on the order of the waves.  A weight is held to [0, 1], which the clamp of
// the exponential's result gives for nothing; the clamp also makes a NaN a
// zero.  A row whose lse is not finite adds nothing, and a row of q with a NaN
// or an infinity has no finite one: its scores are NaN or infinite throughout.
// (Under a finite lse from elsewhere an infinite score is 0 or 1; a test for it
// would read all of q once more.)
//
// S = Q K^T with a token per column: a lane holds the scores of one token for
// several rows, and the sum over the rows stays within the lane until the last
// step.
#pragma once
#include "attn.h"

namespace nvfp4 {

struct WeighArgs {
    AttnArgs a;
    const float* lse;     // [n, heads]
    const float* before;  // [kv_heads, tokens], row stride ld_before; null: zeros
    int64_t ld_before;
    float* after;         // the same shape (may be before itself)
    int64_t ld_after;
    float* partial;       // tile kernel: sums of blocks whose rows are split
};

// 2^x in [0, 1], 0 for a NaN.
NVFP4_DEV float weigh_exp(float x) { return __builtin_amdgcn_fmed3f(__builtin_amdgcn_exp2f(x), 0.0f, 1.0f); }

// -lse / ln 2; a row without a finite lse: -inf, so that its weights are 0 or NaN.
NVFP4_DEV float weigh_shift(float lse)
{
    return __builtin_fabsf(lse) <= 3.402823466e38f ? lse * -1.4426950408889634f : -__builtin_inff();
}

// The shifts of the 16 rows 8 i + .. + 4 of a tile, from shared memory.  (The compiler would have reads of it wait
// for all copies in flight, which go to other arrays, so they and their wait are written out.)
NVFP4_DEV void weigh_shifts(const float* src, float4_t (&z)[4])
{
    const uint32_t at = (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) float*)src;
    asm volatile(
        "ds_read_b128 %0, %4\n\t"
        "ds_read_b128 %1, %4 offset:32\n\t"
        "ds_read_b128 %2, %4 offset:64\n\t"
        "ds_read_b128 %3, %4 offset:96\n\t"
        "s_waitcnt lgkmcnt(0)"
        : "=&v"(z[0]), "=&v"(z[1]), "=&v"(z[2]), "=&v"(z[3])
        : "v"(at)
        : "memory");
}

// The first token whose weight a call writes: in place, the first in the first
// row's window (entries of pages that lie wholly before it may hold anything,
// another sequence's page as well), and none of a sequence without rows.  Steps
// and blocks begin before it, at whole multiples of their tokens; what they
// store does not.
NVFP4_DEV int weigh_first(const WeighArgs& w, const AttnSeq& s)
{
    int lo, hi;
    attn_limits(w.a, s, 0, &lo, &hi);
    return w.before != w.after ? 0 : (s.nq > 0 ? lo : s.kv);
}

// The steps or blocks of `each` tokens that hold the tokens from `first` on.
NVFP4_DEV int weigh_units(int first, int kv, int each)
{
    return first < kv ? (kv + each - 1) / each - first / each : 0;
}

// Adds x to what token t of a sequence and KV head had (from `fresh` on: nothing).
NVFP4_DEV void weigh_put(const WeighArgs& w, const int32_t* table_row, int h, int t, int fresh, float x)
{
    const int i = attn_page(w.a, t), page = table_row[i];
    if (page < 0 || page >= w.a.num_pages) {
        raise_error(NVFP4_ERR_RANGE);
        return;
    }
    const int64_t slot = (int64_t)page * w.a.page + (t - i * w.a.page);
    if (w.before && t < fresh)
        x += w.before[h * w.ld_before + slot];
    w.after[h * w.ld_after + slot] = x;
}

// ---------------------------------------------------------------------------
// Few query rows per sequence: the time is K's way from HBM.  The steps of 32
// tokens of all sequences are cut into equal shares, as in the attention's row
// kernel; a wave takes a run of them for one KV head.  K comes by direct copies
// into two buffers, one of them under way while the other is used.  The sums
// of up to kWeighRun tokens stay in shared memory and go to the weights in
// runs of neighbours.
//
// 64 single tokens on 64-16384 tokens, 32/8 heads of 128: 42 us for 117 MB (2.8
// TB/s; 23.5 us at the rate of a copy): the decode of K and the exponentials of
// tiles that four rows fill of 16 (the vector unit works 64% of the cycles, the
// matrix unit 8%).  64 rows of 16 x 8000 tokens, 4 heads of 64, 128, 256: 25, 31
// and 55 us, 4.6, 8.4 and 16 at that rate: about eight steps a wave, whose waits
// (43, 43 and 54% of the waves' cycles) one workgroup a CU does not cover (vector
// unit 50, 50, 39%, matrix unit 7, 12, 14%).
// One sequence of 700 tokens: 8.8 us of dependent reads (lengths, page, K, the
// weights before).
// ---------------------------------------------------------------------------
constexpr int kWeighRun = 512;

// Workgroups of eight waves on a CU.  Two, where the registers of four waves on a SIMD hold the queries (64
// sequences of 4000 tokens, 16 rows: 43.3 us; one: 52.3; three shares a CU for two places: 45.6).  One with more rows
// (40 rows, 16 sequences of 8000: 50.2; two: 60.2) and with D = 256 (one sequence of 262144: 41.3; two: 49.2).
template <int D, int NT>
constexpr int weigh_rows_per_cu() { return D <= 128 && NT <= 2 ? 2 : 1; }

template <int D, int NT>
struct WeighRows {
    AttnWave<D, NT> x;  // the queries and the copies
    float c[NT][4], z[NT][4];  // of rows 4 g + i of the tile: score's factor, -lse / ln 2
    int start[NT][4], end[NT][4];

    NVFP4_DEV void open(const WeighArgs& w, const AttnSeq& s, int h, int row0)
    {
        x.open(w.a, s, h, row0);
#pragma unroll
        for (int t = 0; t < NT; t++) {
            const int r = row0 + 16 * t + lane_n();
            const int i = r / w.a.group, head = h * w.a.group + r - i * w.a.group;
            float shift = -__builtin_inff();
            if (i < s.nq)
                shift = weigh_shift(w.lse[(int64_t)(s.q0 + i) * (w.a.kv_heads * w.a.group) + head]);
            const float f = __builtin_fminf(__builtin_ldexpf(x.c1[t], x.k[t]), 3.402823466e38f);
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const int from = 4 * lane_g() + j;
                c[t][j] = __shfl(f, from, 64);
                z[t][j] = __shfl(shift, from, 64);
                start[t][j] = __shfl(x.start[t], from, 64);
                end[t][j] = __shfl(x.end[t], from, 64);
            }
        }
    }

    // the sums over the rows of one step (tokens t0 .. t0 + 32): lane group g < 2 holds token 16 g + 4 (n % 4) + n / 4
    NVFP4_DEV float step(const float4_t (&sc)[NT][2], int t0, bool inside) const
    {
        float sum[2];
#pragma unroll
        for (int half = 0; half < 2; half++) {
            const int tok = t0 + 16 * half + 4 * (lane_n() & 3) + (lane_n() >> 2);
            float p[NT][4];
#pragma unroll
            for (int t = 0; t < NT; t++)
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    p[t][j] = weigh_exp(__builtin_fmaf(sc[t][half][j], c[t][j], z[t][j]));
                    if (!inside)
                        p[t][j] = tok >= start[t][j] && tok < end[t][j] ? p[t][j] : 0.0f;
                }
            sum[half] = 0.0f;
#pragma unroll
            for (int t = 0; t < NT; t++)
                sum[half] += (p[t][0] + p[t][1]) + (p[t][2] + p[t][3]);
            sum[half] += __shfl_xor(sum[half], 16, 64);
            sum[half] += __shfl_xor(sum[half], 32, 64);
        }
        return lane_g() & 1 ? sum[1] : sum[0];
    }

    // adds the weights of tokens [t0, t1) (t0 a multiple of 32) to sums[]; [lo, hi): the tokens that every row sees
    NVFP4_DEV void walk(const WeighArgs& w, const int32_t* table_row, int h, int t0, int t1, int lo, int hi,
                        uint8_t* buf0, uint8_t* buf1, float* sums) const
    {
        if (t0 >= t1)
            return;
        AttnPages pages;
        pages.row = table_row;
        pages.last = attn_page(w.a, t1 - 1);
        pages.needed = pages.last + 1;  // (a bad entry is reported where its tokens are stored)
        pages.idx = attn_page(w.a, t0);
        pages.off = t0 - pages.idx * w.a.page;
        pages.fill(w.a, pages.idx);
        int64_t row[2];
        bool ok[2];
        auto request = [&](uint8_t* buf) {
            x.rows(w.a, pages, row, ok, h);
            x.request(w.a.k_packed, w.a.k_scales, row, buf);
        };
        const int place = 16 * (lane_g() & 1) + 4 * (lane_n() & 3) + (lane_n() >> 2);
        auto use = [&](uint8_t* buf, int t) {
            float4_t sc[NT][2];
            wait_copies<AttnWave<D, NT>::kCopies>();
            x.template scores<true>(buf, sc);
            request(buf);
            const float v = step(sc, t, t >= lo && t + kAttnStep <= hi);
            if (lane_g() < 2)
                sums[t - t0 + place] += v;
        };
        request(buf0);
        request(buf1);
        // (no branch in the loop: with one the compiler waits for both copies before it reads the first)
        int t = t0;
        for (; t + kAttnStep < t1; t += 2 * kAttnStep) {
            use(buf0, t);
            use(buf1, t + kAttnStep);
        }
        if (t < t1)
            use(buf0, t);
        wait_vm<0>();
    }
};

template <int D, int NT>
__global__ void __launch_bounds__(512, (2 * weigh_rows_per_cu<D, NT>()))
weigh_rows_kernel(WeighArgs w)
{
    constexpr int kWaves = 8;
    __shared__ __attribute__((aligned(16))) uint8_t buf0[kWaves * attn_stage<D>()];
    __shared__ __attribute__((aligned(16))) uint8_t buf1[kWaves * attn_stage<D>()];
    __shared__ float run[kWaves][kWeighRun];
    const AttnArgs& a = w.a;
    const int wave = uniform((int)(threadIdx.x >> 6));
    const int hl = a.head_lanes, tls = kWaves / hl;
    // (head blocks of one share on one XCD, as in attn_rows_kernel)
    const int blocks = a.kv_heads / hl;
    const int hb = blockIdx.x / 8 % blocks, share = blockIdx.x / (8 * blocks) * 8 + blockIdx.x % 8;
    const int h = hb * hl + wave % hl, tl = wave / hl;
    AttnSeq own{0, 0, 0, false};
    auto count = [&](int b) {
        own = attn_seq(a, b);
        return AttnCount{1, weigh_units(weigh_first(w, own), own.kv, kAttnStep), own.down};
    };
    const AttnScan scan = attn_scan(a.seqs, count);
    const int64_t total = scan.units;
    const int shares = attn_shares(a, scan.units);
    if (share >= shares)
        return;
    int u = (int)(share * total / shares);
    const int u1 = (int)((share + 1) * total / shares);
    AttnFound f = attn_find(scan, a.seqs, u, count);
    float* sums = run[wave];
    while (u < u1) {
        const AttnSeq s = attn_seq_uniform(a, own, f.seq);
        const int lowest = weigh_first(w, s), first = lowest & ~(kAttnStep - 1);
        const int units = weigh_units(lowest, s.kv, kAttnStep);
        if (f.at >= units) {
            f.seq++;
            f.at = 0;
            continue;
        }
        const int n = units - f.at < u1 - u ? units - f.at : u1 - u;
        // this wave's tokens
        const int per = (n + tls - 1) / tls * kAttnStep, t0 = first + f.at * kAttnStep;
        int from = t0 + tl * per, to = from + per;
        to = to < t0 + n * kAttnStep ? to : t0 + n * kAttnStep;
        to = to < s.kv ? to : s.kv;
        const int32_t* row = a.table + f.seq * a.ld_table;
        const int rows = s.nq * a.group, fresh = s.kv - s.nq;
        WeighRows<D, NT> x;
        int open = -1;
        for (; from < to; from += kWeighRun) {
            const int end = to - from < kWeighRun ? to : from + kWeighRun;
            for (int i = threadIdx.x & 63; i < kWeighRun; i += 64)
                sums[i] = 0.0f;
            for (int r = 0; r < rows; r += 16 * NT) {
                int lo0, hi0, lo1, hi1;  // tokens of the tile's first and last row
                const int last = (r + 16 * NT - 1) / a.group;
                attn_limits(a, s, r / a.group, &lo0, &hi0);
                attn_limits(a, s, last < s.nq ? last : s.nq - 1, &lo1, &hi1);
                int b = lo0 & ~(kAttnStep - 1);
                b = b > from ? b : from;
                const int e = end < hi1 ? end : hi1;
                if (b >= e)
                    continue;
                if (open != r)
                    x.open(w, s, h, open = r);
                x.walk(w, row, h, b, e, lo1, hi0, buf0 + wave * attn_stage<D>(), buf1 + wave * attn_stage<D>(),
                       sums + (b - from));
            }
            wait_lgkm0();
            for (int t = from + (int)(threadIdx.x & 63); t < end; t += 64)
                if (t >= lowest)
                    weigh_put(w, row, h, t, fresh, sums[t - from]);
            wait_lgkm0();
        }
        u += n;
        f.at += n;
    }
}

// ---------------------------------------------------------------------------
// Many query rows per sequence: the time is the product and the exponentials.
// A wave takes 32 tokens of one KV head, a workgroup the block of tokens of its
// waves, and walks the rows in tiles of 32.  K is decoded to bf16 once (six
// significant bits: exact) and stays in registers; q goes to the products as
// it is, copied into shared memory three tiles ahead, so that no element is
// converted in the loop.  Blocks and parts of their rows are jobs of about
// equal size; where rows are split, a second launch adds the parts in their
// order.
//
// v_mfma_f32_32x32x16_bf16 (A: row l % 32, B: column l % 32, both elements
// 8 (l / 32) .. + 8 of the contraction; output: column l % 32, rows
// 8 (i / 4) + 4 (l / 32) + i % 4).  The contraction's order is free: lane half
// e takes elements [e D / 2, + D / 2).
//
// An element costs a multiply-add, an exponential (10 cycles of a wave) and an
// addition on the vector unit and D / 512 cycles on the matrix unit.  A wave issues
// a vector instruction about every seven cycles and no more, so up to D = 128
// there are four waves on a SIMD, each with its products and then its
// exponentials.  With D = 256, whose K alone takes 64 registers, there are two,
// and a tile's exponentials stand between the products of the next.
//
// A prompt of 4096, 32/8 heads of 128: 102 us and 5.4 for the joining launch, 0.68
// PFLOP/s.  The matrix unit works 36% of the cycles and the vector unit 57%, in all
// 94%: hardly any of either runs beside the other (the waves of a workgroup pass
// the barrier of each 32 rows together).  Graphs of both launches replayed, 123 us
// so: with 64 tokens a wave 147
// (two waves on a SIMD, products and exponentials in turn), 129 (exponentials
// between the products), 127 (those and one tile ahead); three waves of 32 tokens
// 118-125 (registers spill; D = 256 143 for 109); tokens as rows of the product
// 327 (the sums then cross lanes, registers spill).
// ---------------------------------------------------------------------------
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));

template <int D>
constexpr bool weigh_turns() { return D == 256; }
template <int D>
constexpr int weigh_waves() { return D == 256 ? 4 : 8; }
template <int D>
constexpr int weigh_block() { return 32 * weigh_waves<D>(); }  // tokens of a workgroup
constexpr int kWeighRows = 1024;    // rows whose shifts are in shared memory at a time (a multiple of 128)
constexpr int kWeighWorkers = 512;  // workgroups, two per CU
constexpr int kWeighJobs = 1024;    // parts of split blocks, at most

// The blocks of tokens of a sequence.
template <int D>
NVFP4_DEV AttnCount weigh_count(const WeighArgs& w, const AttnSeq& s)
{
    AttnCount c;
    c.tiles = w.a.kv_heads;
    c.units = weigh_units(weigh_first(w, s), s.kv, weigh_block<D>());
    c.down = s.down;
    return c;
}

// Parts that each block's rows are split into (units: blocks of all sequences and KV heads).
NVFP4_DEV int weigh_splits(int units)
{
    const int s = units > 0 ? kWeighJobs / units : 1;
    return s < 1 ? 1 : (s < 16 ? s : 16);
}

// Rows [r0, r1) of a sequence (a row: query token * group + head) that see a token of [t0, t1).
NVFP4_DEV void weigh_span(const AttnArgs& a, const AttnSeq& s, int t0, int t1, int* r0, int* r1)
{
    int i0 = 0, i1 = s.nq;
    if (a.causal) {
        const int base = s.kv - s.nq;  // the first row's position
        i0 = t0 - base > 0 ? t0 - base : 0;
        if (a.window > 0) {
            const int64_t e = (int64_t)t1 - base + a.window - 1;
            i1 = e < i1 ? (e > 0 ? (int)e : 0) : i1;
        }
    }
    *r0 = i0 < i1 ? i0 * a.group : 0;
    *r1 = i0 < i1 ? i1 * a.group : 0;
}

template <int D>
__global__ void __launch_bounds__((64 * weigh_waves<D>()), (weigh_turns<D>() ? 2 : 4))
weigh_tile_kernel(WeighArgs w)
{
    constexpr int BT = weigh_block<D>(), NT = 64 * weigh_waves<D>(), N = D / 16, C = D / 8;  // C: chunks of a q row
    // (separate arrays, picked at compile time, so that reads of one do not wait for the copies into another)
    __shared__ __attribute__((aligned(16))) u32x4 q0[32 * C], q1[32 * C], q2[32 * C], q3[32 * C];
    __shared__ __attribute__((aligned(16))) float shift[kWeighRows];
    __shared__ __attribute__((aligned(16))) int limit[kWeighRows];  // a row sees the tokens below
    const AttnArgs& a = w.a;
    const int tid = threadIdx.x, lane = tid & 63, col = lane & 31, e = lane >> 5;
    const int wave = uniform(tid >> 6);
    AttnSeq own{0, 0, 0, false};
    auto count = [&](int b) ATTN_INLINE {
        own = attn_seq(a, b);
        return weigh_count<D>(w, own);
    };
    const AttnScan scan = attn_scan(a.seqs, count);
    const int splits = weigh_splits(scan.units);
    const int64_t jobs = (int64_t)scan.units * splits;
    // (a score is s c, with s the sum over codes * scales: K's global is in c)
    const double cd = a.scale_log2 * (double)*a.k_global;
    const float c = (float)(cd < 3e38 ? cd : 3e38);
    // Jobs in rounds of one per workgroup, every other round backwards: in a
    // causal sequence the first blocks have the most rows.
    for (int round = 0;; round++) {
        const int place = round & 1 ? (kWeighWorkers / 8 - 1 - (int)blockIdx.x / 8) * 8 + (int)blockIdx.x % 8 : (int)blockIdx.x;
        const int64_t job = (int64_t)round * kWeighWorkers + place;
        if ((int64_t)round * kWeighWorkers >= jobs)
            break;
        if (job >= jobs)
            continue;
        // (split and block before the KV head: neighbouring workgroups share rows of q)
        const int unit_head = (int)(job / splits);
        const AttnFound f = attn_find(scan, a.seqs, unit_head, count);
        const AttnSeq s = attn_seq_uniform(a, own, f.seq);
        const int64_t in_seq = job - (int64_t)f.before.units * splits;
        const int h = (int)(in_seq % a.kv_heads);
        const int split = (int)(in_seq / a.kv_heads % splits), block = (int)(in_seq / a.kv_heads / splits);
        const int lowest = weigh_first(w, s), t0 = (lowest / BT + block) * BT;
        const int32_t* table = a.table + f.seq * a.ld_table;
        int r0, r1;
        weigh_span(a, s, t0, t0 + BT < s.kv ? t0 + BT : s.kv, &r0, &r1);
        // this part's rows, whole tiles of 32
        if (splits > 1) {
            const int tiles = (r1 - r0 + 31) / 32, per = (tiles + splits - 1) / splits * 32;
            const int base = r0;
            r0 = base + split * per < r1 ? base + split * per : r1;
            r1 = r1 - r0 < per ? r1 : r0 + per;
        }
        // ---- K of this wave's tokens
        const int tw = t0 + wave * 32, token = tw + col;
        bf16x8_t k[N];
        {
            const int i = attn_page(a, token < s.kv ? token : s.kv - 1);
            const int page = table[i];
            const bool ok = token < s.kv && page >= 0 && page < a.num_pages;
            const int64_t row = ok ? ((int64_t)page * a.page + (token - i * a.page)) * a.kv_heads + h : h;
            uint32_t kc[D / 16], ks[D / 128 > 0 ? D / 128 : 1];
            load_bytes<D / 4>(a.k_packed + row * (D / 2) + e * (D / 4), kc);
            load_bytes<(D / 32 > 4 ? 4 : D / 32)>(a.k_scales + row * (D / 16) + e * (D / 32), ks);
            if constexpr (D == 256)
                load_bytes<4>(a.k_scales + row * (D / 16) + e * (D / 32) + 4, ks + 1);
            for_range<0, N>([&](auto ji) ATTN_INLINE {
                constexpr int j = decltype(ji)::value;
                const float sc = e4m3_decode(ks[j / 8] >> (8 * (j / 2 % 4)) & 0x7F);
                u32x4 v;
                for_range<0, 4>([&](auto ii) ATTN_INLINE {
                    constexpr int i = decltype(ii)::value;
                    const float2_t y = __builtin_bit_cast(float2_t, FP4_TO_F32X2(kc[j], i));
                    v[i] = pack_bf16x2(y.x * sc, y.y * sc);
                });
                k[j] = __builtin_bit_cast(bf16x8_t, v);
            });
        }
        float sum = 0.0f;
        // Copies of a tile: chunk ch of row rr goes to slot ch ^ swizzle of its row.  The tiles are copied in
        // order, so that a row's query token and head advance by 32 / group and 32 % group.
        constexpr int NJ = 32 * C > NT ? 32 * C / NT : 1;
        const bool copies = 32 * C >= NT || wave * 64 < 32 * C;
        const uint16_t* next[NJ];
        int hh[NJ];
        int next_row = r0;
        auto chunk = [&](int j) ATTN_INLINE {
            const int rr = (j * NT + tid) / C, ch = (j * NT + tid) % C;
            return 8 * (ch ^ (C >= 16 ? rr & 15 : (rr >> 1) & 7));
        };
        auto row_at = [&](int row) ATTN_INLINE {
            const int i = row / a.group;
            return a.q + (int64_t)(s.q0 + i) * a.ld_q + (int64_t)(h * a.group + row - i * a.group) * D;
        };
        const int step_q = 32 / a.group, step_h = 32 - step_q * a.group;
        const int64_t step = step_q * a.ld_q + step_h * D, wrap = a.ld_q - a.group * D;
#pragma unroll
        for (int j = 0; j < NJ; j++) {
            const int row = r0 + (j * NT + tid) / C;
            next[j] = row_at(row < r1 ? row : (r1 > 0 ? r1 - 1 : 0)) + chunk(j);
            hh[j] = row % a.group;
        }
        auto copy = [&](auto buf) ATTN_INLINE {
            constexpr int B = decltype(buf)::value;
            const bool whole = next_row + 32 <= r1;  // (past the end the copies go on, so that their number is known)
            if (copies) {
#pragma unroll
                for (int j = 0; j < NJ; j++) {
                    const uint16_t* src = next[j];
                    if (!whole && next_row + (j * NT + tid) / C >= r1)  // past the end: the last row again
                        src = row_at(r1 - 1) + chunk(j);
                    u32x4* const dst = B == 0 ? q0 : (B == 1 ? q1 : (B == 2 ? q2 : q3));
                    __builtin_amdgcn_global_load_lds((const void*)src, (attn_lds_t)(dst + j * NT + wave * 64), 16, 0, 0);
                    next[j] += step;
                    if (step_h != 0) {
                        hh[j] += step_h;
                        const bool over = hh[j] >= a.group;
                        hh[j] -= over ? a.group : 0;
                        next[j] += over ? wrap : 0;
                    }
                }
            }
            next_row += 32;
        };
        int first_q = r0 / a.group, first_h = r0 - first_q * a.group;  // query token and head of the first row weighed next
        float16_t s0, s1;
        // One turn: the products of tile r (in buffer B) into `to`, and the weights of the tile before, whose
        // products are in `from` (between the products, where both are asked for).
        auto turn = [&](int r, int seg, auto buf, auto has_old, auto has_new, float16_t& from, float16_t& to) ATTN_INLINE {
            constexpr int B = decltype(buf)::value, per = 16 / N;
            const int old = r - 32;
            float4_t z[4];
            bool inside = true;
            if constexpr (has_old) {
                weigh_shifts(shift + (old - seg) + 4 * e, z);
                // what the tile's first and last row see (rows behind the last one have no weight)
                const int base = s.kv - s.nq, lo = base + first_q + 1, hi = base + first_q + (first_h + 31) / a.group + 1;
                inside = tw + 32 <= s.kv && (!a.causal || (tw + 32 <= lo && (a.window <= 0 || tw >= hi - a.window)));
                first_q += step_q;
                first_h += step_h;
                if (first_h >= a.group) {
                    first_h -= a.group;
                    first_q++;
                }
            }
            if constexpr (has_new)
                copy(std::integral_constant<int, (B + 3) % 4>{});
            bf16x8_t f[N];
            auto read = [&](auto ji) ATTN_INLINE {
                constexpr int j = decltype(ji)::value;
                const u32x4* const src = B == 0 ? q0 : (B == 1 ? q1 : (B == 2 ? q2 : q3));
                f[j] = __builtin_bit_cast(bf16x8_t,
                                          src[col * C + ((e * N + j) ^ (C >= 16 ? col & 15 : (col >> 1) & 7))]);
            };
            auto multiply = [&](auto ji) ATTN_INLINE {
                constexpr int j = decltype(ji)::value;
                if constexpr (j + 1 < N)
                    read(std::integral_constant<int, j + 1>{});
                to = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f[j], k[j], to, 0, 0, 0);
            };
            if constexpr (has_new) {
#pragma unroll
                for (int i = 0; i < 16; i++)
                    to[i] = 0.0f;
                read(std::integral_constant<int, 0>{});
            }
            if (inside) {
                for_range<0, N>([&](auto ji) ATTN_INLINE {
                    constexpr int j = decltype(ji)::value;
                    if constexpr (has_new)
                        multiply(ji);
                    if constexpr (has_old)
#pragma unroll
                        for (int i = j * per; i < (j + 1) * per; i++)
                            sum += weigh_exp(__builtin_fmaf(from[i], c, z[i >> 2][i & 3]));
                });
            } else {
                if constexpr (has_new)
                    for_range<0, N>(multiply);
                if constexpr (has_old) {
#pragma unroll
                    for (int i = 0; i < 16; i++) {
                        const int below = limit[old - seg + 8 * (i >> 2) + 4 * e + (i & 3)];
                        const bool seen = token < below && (a.window <= 0 || token >= below - a.window);
                        const float x = weigh_exp(__builtin_fmaf(from[i], c, z[i >> 2][i & 3]));
                        sum += seen ? x : 0.0f;
                    }
                }
            }
        };
        constexpr std::integral_constant<int, 0> zero{};
        constexpr std::integral_constant<int, 1> one{};
        constexpr std::integral_constant<int, 2> two{};
        constexpr std::integral_constant<int, 3> three{};
        constexpr std::true_type yes{};
        constexpr std::false_type no{};
        // the next tile is here (of three on their way), and nobody reads the buffer of the last one any more
        auto arrive = [&]() ATTN_INLINE {
            wait_copies<2 * NJ>();
            lds_barrier();
        };
        lds_barrier();  // nobody reads the last job's tiles any more
        if (r0 < r1) {
            copy(zero);
            copy(one);
            copy(two);
        }
        for (int seg = r0; seg < r1; seg += kWeighRows) {
            const int end = r1 - seg < kWeighRows ? r1 : seg + kWeighRows;
            lds_barrier();  // nobody reads the last rows' shifts any more
            for (int x = tid; x < ((end - seg + 31) & ~31); x += NT) {
                const int r = seg + x, i = r / a.group, head = h * a.group + r - i * a.group;
                shift[x] = r < end ? weigh_shift(w.lse[(int64_t)(s.q0 + i) * (a.kv_heads * a.group) + head])
                                   : -__builtin_inff();
                const int to = s.kv - s.nq + i + 1;
                limit[x] = !a.causal || to > s.kv ? s.kv : (to > 0 ? to : 0);
            }
            const int tiles = (end - seg + 31) / 32;
            // f(first row, buffer, parity) for tiles x0, x0 + 1, ... of the segment
            auto each = [&](int x, auto f) ATTN_INLINE {
                for (; x + 4 <= tiles; x += 4) {
                    f(seg + 32 * x, one, one);
                    f(seg + 32 * x + 32, two, zero);
                    f(seg + 32 * x + 64, three, one);
                    f(seg + 32 * x + 96, zero, zero);
                }
                if (x < tiles)
                    f(seg + 32 * x, one, one);
                if (x + 1 < tiles)
                    f(seg + 32 * x + 32, two, zero);
                if (x + 2 < tiles)
                    f(seg + 32 * x + 64, three, one);
            };
            arrive();
            if constexpr (weigh_turns<D>()) {
                turn(seg, seg, zero, no, yes, s1, s0);
                each(1, [&](int r, auto buf, auto odd) ATTN_INLINE {
                    arrive();
                    if constexpr (odd)
                        turn(r, seg, buf, yes, yes, s0, s1);
                    else
                        turn(r, seg, buf, yes, yes, s1, s0);
                });
                if (tiles & 1)
                    turn(seg + 32 * tiles, seg, zero, yes, no, s0, s1);
                else
                    turn(seg + 32 * tiles, seg, zero, yes, no, s1, s0);
            } else {
                turn(seg, seg, zero, no, yes, s0, s0);
                turn(seg + 32, seg, zero, yes, no, s0, s0);
                each(1, [&](int r, auto buf, auto) ATTN_INLINE {
                    arrive();
                    turn(r, seg, buf, no, yes, s0, s0);
                    turn(r + 32, seg, buf, yes, no, s0, s0);
                });
            }
        }
        wait_vm<0>();
        sum += __shfl_xor(sum, 32, 64);
        if (e == 0 && token >= lowest && token < s.kv) {
            if (splits > 1) {
                // [sequence's units in a row: block, head][split][token of the block]
                const int64_t unit = f.before.units + (int64_t)block * a.kv_heads + h;
                w.partial[(unit * splits + split) * BT + (token - t0)] = sum;
            } else {
                weigh_put(w, table, h, token, s.kv - s.nq, sum);
            }
        }
    }
}

// Adds the parts of split blocks, in order; a workgroup a block and KV head at a time.
template <int D>
__global__ void __launch_bounds__(weigh_block<D>())
weigh_join_kernel(WeighArgs w)
{
    constexpr int BT = weigh_block<D>();
    const AttnArgs& a = w.a;
    AttnSeq own{0, 0, 0, false};
    auto count = [&](int b) {
        own = attn_seq(a, b);
        return weigh_count<D>(w, own);
    };
    const AttnScan scan = attn_scan(a.seqs, count);
    const int splits = weigh_splits(scan.units);
    if (splits == 1)
        return;
    for (int unit = blockIdx.x; unit < scan.units; unit += gridDim.x) {
        const AttnFound f = attn_find(scan, a.seqs, unit, count);
        const AttnSeq s = attn_seq_uniform(a, own, f.seq);
        const int lowest = weigh_first(w, s);
        const int h = f.at % a.kv_heads, t = (lowest / BT + f.at / a.kv_heads) * BT + (int)threadIdx.x;
        if (t < lowest || t >= s.kv)
            continue;
        float sum = 0.0f;
        for (int i = 0; i < splits; i++)
            sum += w.partial[((int64_t)unit * splits + i) * BT + threadIdx.x];
        weigh_put(w, a.table + f.seq * a.ld_table, h, t, s.kv - s.nq, sum);
    }
}

}  // namespace nvfp4
