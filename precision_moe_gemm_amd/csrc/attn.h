// attn.h -- attention over the paged NVFP4 KV cache (page
// "Qwen3.8-2.4T-A95B-NVFP4": K and V stored at about 4 bits, read back by
// every later token).
//
//   s[r, t] = scale * q[r] . k[t],  p = softmax over the tokens r may see,
//   o[r] = sum_t p[r, t] v[t],      lse[r] = log sum_t exp(s[r, t])
//
// One pass over the tokens: a running maximum m and sum l per row r (fp32),
// o rescaled when m grows.  Scores are kept in units of log 2.
//
// Operands.  An NVFP4 value without its tensor global is code * scale with
// 2 + 4 significant bits between 2^-10 and 2688: exact in f16, so K and V are
// decoded to f16 without rounding and the globals applied in fp32 afterwards
// (K's to the scores, V's to the output).  q (bf16) is scaled per row by a
// power of two to a largest magnitude in [1, 2) and held in f16: exact for
// every element down to 2^-16 of the row's largest, and off by at most 2^-25
// of that below.  p is rounded to f16 for the second product (off by at
// most 2^-11 of it), l sums the unrounded p.
//
// Both products are written transposed, S^T = K Q^T and O^T = V^T P^T, with
// v_mfma_f32_16x16x32_f16 (A: row l % 16, B: column l % 16, both elements
// 8 (l / 16) .. + 8 of the contraction; output: column l % 16, rows
// 4 (l / 16) .. + 4 for lane l).  A lane then holds the scores of one query
// row for 4 + 4 tokens of two 16-token tiles, which is its share of the
// second product's B operand as it stands: p never leaves its registers.
// The order of the contraction elements is free as long as both operands
// agree on it, and so is the order of a tile's rows: with n = l % 16 and
// g = l / 16, the first product gives lane group g the elements [g D / 4,
// + D / 4), one contiguous piece of a K row, and row n is token
// 4 (n % 4) + n / 4; so output row 4g + i is token 4i + g, and the second
// product gives group g tokens 4i + g of both tiles; its output row m of MFMA
// dd is element m D / 16 + dd, so a lane needs a contiguous piece of a V row.
#pragma once
#include <type_traits>

#include "common.h"
#include "gemm.h"

namespace nvfp4 {

struct AttnArgs {
    const uint16_t* q;       // [n, heads, D], token stride ld_q
    int64_t ld_q;
    const uint8_t* k_packed;
    const uint8_t* k_scales;
    const uint8_t* v_packed;
    const uint8_t* v_scales;
    const float* k_global;
    const float* v_global;
    const int32_t* cu_q;     // [seqs + 1], or null: one query token per sequence
    const int32_t* kv_lens;  // [seqs]
    const int32_t* table;    // [seqs, pages], row stride ld_table
    int64_t ld_table;
    int64_t num_pages;       // pages in the cache
    int64_t n;               // rows of q
    int seqs, pages, page;   // page: tokens of a page (a multiple of 16)
    int page_shift;          // t / page = (t / 8) * page_mul >> (32 + page_shift)
    uint32_t page_mul;
    int kv_heads, group;     // group: query heads per KV head
    double scale_log2;       // scale * log2(e)
    int causal, window;
    const uint32_t* mask;    // trees of drafts: bit j % 32 of word j / 32 of a query row: it sees draft j
    int64_t ld_mask;         // words
    int mask_words;
    uint16_t* out;           // [n, heads, D], token stride ld_out
    int64_t ld_out;
    float* lse;              // [n, heads] or null
    int head_lanes;          // KV heads a workgroup holds side by side (1, 2 or 4)
    int workers;             // shares that the tokens are cut into (at most)
    int whole;               // a workgroup takes a whole tile of rows instead of a share
    struct AttnTile* tiles;  // tiles of rows, as the joining launch needs them
    float* partial;          // what shares leave of tiles that they hold a part of
};

// Waves of a row workgroup: 8, or 4 where their joining space would pass the
// shared memory.
template <int D, int NT>
constexpr int attn_waves() { return D * NT <= 256 ? 8 : 4; }
typedef __attribute__((address_space(3))) void* attn_lds_t;
constexpr int kAttnStep = 32;            // tokens of one step
constexpr float kAttnLow = -3.402823466e38f;  // running maximum of a row that has seen nothing
constexpr float kAttnLazy = 8.0f;        // growth of the maximum (log 2) that is let pass
constexpr float kAttnLift = 7.0f;        // p is held times 2^7, at most 2^15 (f16 holds 65504)

// Far scores.  Scores are s * c1 with a factor c1 per row, and weights
// 2^(s c1 + lift) come from one fused multiply-add, whose exact product exceeds
// the rounded one that the maximum was taken from by up to half a step of it,
// as the lift is off by half a step: together with the 2^15 that a weight may
// be, at most 2^15.5 while the maximum stays within 2^22, but past f16's
// largest value from 2^24 on.  A row whose maximum leaves that range therefore
// keeps its scores in units of 2^k (c1 and m times 2^-k, m back inside).  What
// lies 32 units below the maximum counts for nothing, so this is as if a score
// were off by up to 32 2^k, 2^-16 of the largest: past 2^22, fp32 holds its own
// sum of D products to D 2^-24 of that.

// c1 and k of a row whose q was divided by 2^e, in 64 bits, as the factors alone
// may pass fp32's range.  c1 stays above zero (-inf times it stays -inf) and
// below 2^100 (|s| is below 2^21).
NVFP4_DEV float attn_factor(double scale_log2, float k_global, int e, int* k)
{
    const double x = __builtin_ldexp(scale_log2 * k_global, e);
    const int over = __builtin_amdgcn_frexp_exp(x) - 100;
    *k = over > 0 ? over : 0;
    return x < 1e-37 ? 1e-37f : (float)__builtin_ldexp(x, -*k);
}

// The running maximum m of a row becomes `now`: what l and o are multiplied by.
NVFP4_DEV float attn_grow(float now, float* m, float* c1, int* k)
{
    float f = __builtin_amdgcn_exp2f(*m - now);
    const bool far = (__builtin_fabsf(now) > 4194304.0f || *k > 0) && now > kAttnLow;
    if (__any(far)) {
        f = __builtin_amdgcn_exp2f(__builtin_ldexpf(*m - now, *k));
        // (a maximum near zero under a factor past 2^100: later scores must not overflow)
        int over = now != 0.0f ? __builtin_amdgcn_frexp_expf(now) - 22 : -1000;
        const int most = __builtin_amdgcn_frexp_expf(*c1) - 100;
        over = (over > most ? over : most) + *k;
        const int by = far ? *k - (over > 0 ? over : 0) : 0;
        now = __builtin_ldexpf(now, by);
        *c1 = __builtin_ldexpf(*c1, by);
        *k -= by;
    }
    *m = now;
    return f;
}

// The maximum itself, at most fp32's largest value.
NVFP4_DEV float attn_whole(float m, int k)
{
    return __builtin_fminf(__builtin_fmaxf(__builtin_ldexpf(m, k), kAttnLow), -kAttnLow);
}

// One sequence as the kernels see it: bad lengths are cut to what exists and
// raise NVFP4_ERR_RANGE.  down: its end lies before its start.
struct AttnSeq {
    int q0, nq, kv;
    bool down;
};

// The page of token t >= 0 of a sequence.
NVFP4_DEV int attn_page(const AttnArgs& a, int t)
{
    return (int)(__umulhi((uint32_t)t >> 3, a.page_mul) >> a.page_shift);
}

// The value of a variable that is the same in all lanes, held in a scalar
// register: addresses and branches that depend on it are then scalar too.
NVFP4_DEV int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

NVFP4_DEV AttnSeq attn_seq(const AttnArgs& a, int b)
{
    AttnSeq s;
    bool bad = false;
    if (a.cu_q) {
        const int lo = a.cu_q[b], hi = a.cu_q[b + 1];
        const int n = (int)a.n;
        s.q0 = lo < 0 ? 0 : (lo > n ? n : lo);
        const int e = hi < s.q0 ? s.q0 : (hi > n ? n : hi);
        s.nq = e - s.q0;
        bad = s.q0 != lo || e != hi;
        s.down = hi < lo;
    } else {
        s.q0 = b;
        s.nq = 1;
        s.down = false;
    }
    const int kv = a.kv_lens[b];
    const int64_t most = (int64_t)a.pages * a.page;
    s.kv = kv < 0 ? 0 : ((int64_t)kv > most ? (int)most : kv);
    if (bad || s.kv != kv)
        raise_error(NVFP4_ERR_RANGE);
    return s;
}

// Tokens [start, end) that query token i of a sequence sees.
NVFP4_DEV void attn_limits(const AttnArgs& a, const AttnSeq& s, int i, int* start, int* end)
{
    int e = s.kv, b = 0;
    if (a.causal) {
        const int pos = s.kv - s.nq + i;  // its own position
        e = pos + 1 < s.kv ? pos + 1 : s.kv;
        // (pos may be far below zero: pos - window could wrap)
        if (a.window > 0 && pos >= a.window)
            b = pos - a.window + 1;
    }
    *end = e < 0 ? 0 : e;
    *start = b;
}

// ---- trees of drafts (TREE): the m query tokens of a sequence are its last m
// tokens, as otherwise.  Each sees every token before them, [0, base), and of
// the m themselves those of its mask; with a window, the last `window` of what
// it sees.

NVFP4_DEV int attn_tree_base(const AttnSeq& s) { return s.kv > s.nq ? s.kv - s.nq : 0; }

// Drafts past the mask's words are seen by no row.
NVFP4_DEV void attn_tree_check(const AttnArgs& a, const AttnSeq& s)
{
    if (s.nq > 32 * (int64_t)a.mask_words)
        raise_error(NVFP4_ERR_RANGE);
}

// The mask of 32 tokens of which the first is draft j0 (tokens before the
// drafts are seen), for the query token in row `row` of q.
NVFP4_DEV uint32_t attn_tree_bits(const AttnArgs& a, int row, int j0)
{
    if (j0 <= -32)
        return ~0u;
    const uint32_t* m = a.mask + row * a.ld_mask;
    const int w = j0 >> 5, sh = j0 & 31;  // (j0 < 0: word -1 is all ones)
    const uint32_t lo = w < 0 ? ~0u : (w < a.mask_words ? m[w] : 0u);
    const uint32_t hi = w + 1 < a.mask_words ? m[w + 1] : 0u;
    return (uint32_t)((((uint64_t)hi << 32) | lo) >> sh);
}

// The first token that query token i (row `row` of q) sees under the window.
NVFP4_DEV int attn_tree_start(const AttnArgs& a, const AttnSeq& s, int i)
{
    if (a.window <= 0)
        return 0;
    const uint32_t* m = a.mask + (int64_t)(s.q0 + i) * a.ld_mask;
    const int base = s.kv - s.nq;  // (below zero: the first drafts are not cached)
    const int first = base < 0 ? -base : 0;
    int left = a.window;
    const int words = (s.nq + 31) / 32 < a.mask_words ? (s.nq + 31) / 32 : a.mask_words;
    for (int w = words - 1; w >= 0 && 32 * w + 31 >= first; w--) {
        uint32_t bits = m[w];
        if (32 * w + 32 > s.nq)
            bits &= ~0u >> (32 * w + 32 - s.nq);
        if (32 * w < first)
            bits &= ~0u << (first - 32 * w);
        const int c = __builtin_popcount(bits);
        if (c >= left) {
            while (--left > 0)
                bits &= ~(0x80000000u >> __builtin_clz(bits));
            return base + 32 * w + 31 - __builtin_clz(bits);
        }
        left -= c;
    }
    return base > left ? base - left : 0;
}

// The tokens [lo0, hi0) of the first and [lo1, hi1) of the last of the query
// tokens i0 .. i1.  TREE: every row sees tokens of [lo0, hi1) only, and all of
// [lo1, hi0).
template <bool TREE>
NVFP4_DEV void attn_span(const AttnArgs& a, const AttnSeq& s, int i0, int i1, int* lo0, int* hi0, int* lo1, int* hi1)
{
    if constexpr (TREE) {
        const int base = attn_tree_base(s);
        *lo0 = *lo1 = 0;
        if (a.window > 0) {
            // (a row of no draft sees `window` tokens before them, a row of all of them fewer by their number)
            const int from = base - a.window, most = from + s.nq;
            *lo0 = from > 0 ? from : 0;
            *lo1 = most < 0 ? 0 : (most < base ? most : base);
        }
        *hi0 = base;
        *hi1 = s.kv;
    } else {
        attn_limits(a, s, i0, lo0, hi0);
        attn_limits(a, s, i1, lo1, hi1);
    }
}

// Sequence b, uniform.  own: lane l's sequence l, where there are at most 64.
NVFP4_DEV AttnSeq attn_seq_uniform(const AttnArgs& a, const AttnSeq& own, int b)
{
    if (a.seqs <= 64)
        return AttnSeq{__builtin_amdgcn_readlane(own.q0, b), __builtin_amdgcn_readlane(own.nq, b),
                       __builtin_amdgcn_readlane(own.kv, b), false};
    const AttnSeq s = attn_seq(a, b);
    return AttnSeq{uniform(s.q0), uniform(s.nq), uniform(s.kv), s.down};
}

// Work of a row kernel is counted in units: sequence b has `tiles` tiles of
// rows and `units` steps of tokens for each of them (at least one, so that
// rows that see nothing are written too).  The host refuses launches whose
// units could pass 31 bits.
struct AttnCount {
    int tiles, units;
    bool down;
};

// Every wave scans all sequences by itself: lane l sums the run of
// sequences [l per, + per).  Offsets that go down anywhere (rows would then
// belong to several sequences, and their number would have no bound) leave
// no work at all.
struct AttnScan {
    AttnCount before;  // tiles and units before this lane's run
    int mine;          // units of the run
    int tiles, units;  // of all sequences
};

template <class Count>
NVFP4_DEV AttnScan attn_scan(int seqs, Count count)
{
    const int lane = threadIdx.x & 63;
    const int per = (seqs + 63) >> 6;
    const int b0 = lane * per, b1 = b0 + per < seqs ? b0 + per : seqs;
    int tiles = 0, units = 0;
    bool down = false;
    for (int b = b0; b < b1; b++) {
        const AttnCount c = count(b);
        down |= c.down;
        tiles += c.tiles;
        units += c.tiles * c.units;
    }
    int ut = tiles, uu = units;  // inclusive sums over the lanes
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const int x = __shfl_up(ut, off, 64), y = __shfl_up(uu, off, 64);
        ut += lane >= off ? x : 0;
        uu += lane >= off ? y : 0;
    }
    AttnScan s;
    s.before.tiles = ut - tiles;
    s.before.units = uu - units;
    s.mine = units;
    const bool none = __any(down);
    s.tiles = none ? 0 : __builtin_amdgcn_readlane(ut, 63);
    s.units = none ? 0 : __builtin_amdgcn_readlane(uu, 63);
    return s;
}

// The sequence that holds unit u (u < s.units), the unit's number in it and
// the tiles and units before it: all uniform.
struct AttnFound {
    int seq, at;
    AttnCount before;
};

template <class Count>
NVFP4_DEV AttnFound attn_find(const AttnScan& s, int seqs, int u, Count count)
{
    const int per = (seqs + 63) >> 6;
    const uint64_t hit = __ballot(u >= s.before.units && u - s.before.units < s.mine);
    const int l = __builtin_ctzll(hit);
    AttnFound f;
    f.seq = l * per;
    f.before.tiles = __builtin_amdgcn_readlane(s.before.tiles, l);
    f.before.units = __builtin_amdgcn_readlane(s.before.units, l);
    f.at = u - f.before.units;
    if (per == 1)
        return f;
    for (;;) {
        const AttnCount c = count(f.seq);
        const int tiles = uniform(c.tiles), units = uniform(c.tiles * c.units);
        if (f.at < units)
            return f;
        f.at -= units;
        f.before.tiles += tiles;
        f.before.units += units;
        f.seq++;
    }
}

NVFP4_DEV float4_t mfma16(half8_t a, half8_t b, float4_t c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

// Two f16 scales from E4M3 bytes (low seven bits; a valid scale has no
// sign): the bits as f16 are the value times 2^-8, subnormals included, and
// the codes are converted times 2^8.  No byte gives an infinity or NaN.
NVFP4_DEV half2_t scale_pair(uint32_t lo, uint32_t hi)
{
    return __builtin_bit_cast(half2_t, ((lo & 0x7Fu) << 7) | ((hi & 0x7Fu) << 23));
}

#define FP4_TO_F16X2_256(src, sel) __builtin_amdgcn_cvt_scalef32_pk_f16_fp4((src), 256.0f, (sel))

// Eight codes of one row (a dword) under one block scale.
NVFP4_DEV half8_t decode_row8(uint32_t w, half2_t s)
{
    const half2_t a = FP4_TO_F16X2_256(w, 0) * s, b = FP4_TO_F16X2_256(w, 1) * s;
    const half2_t c = FP4_TO_F16X2_256(w, 2) * s, d = FP4_TO_F16X2_256(w, 3) * s;
    return (half8_t){a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}

// Wait until at most N copies are in flight, with the reads of the older ones
// to follow.  The compiler would have such a read wait for every copy (it
// takes them for flat accesses, which may finish out of order) if it had not
// seen this wait take effect, which an instruction behind it ensures.
template <int N>
NVFP4_DEV void wait_copies()
{
    wait_vm<N>();
    asm volatile("s_nop 0" ::: "memory");
}

// A wave's lanes: query column n, lane group g.
NVFP4_DEV int lane_n() { return threadIdx.x & 15; }
NVFP4_DEV int lane_g() { return (threadIdx.x >> 4) & 3; }

// A wave's copy of 32 tokens of K or V in shared memory: codes [32][D / 2],
// then scales [32][D / 16].  It is filled by direct copies of 16 bytes per
// lane (4 for scales below 16 bytes a row) in which neighbouring lanes take
// neighbouring bytes of a row: read straight into registers, the operands
// need 20 loads of 1 to 16 bytes per lane whose neighbours lie in different
// rows, and ran at 3.3 TB/s where the wide copies of the same bytes reach 5.0
// (32 query heads, 8 KV heads of 128).  Chunk c (16 bytes) of row r lies in
// slot c ^ attn_swz(r) of the row, which spreads the 16 rows of a K read over
// the banks.
template <int D>
constexpr int attn_stage() { return 16 * D + (D == 256 ? 1024 : 256); }

template <int D>
NVFP4_DEV int attn_swz(int r)
{
    return D == 64 ? 0 : (D == 128 ? (r >> 2) & 3 : (r >> 1) & 7);
}

// The pages of a wave's token range: lane l holds the entry of page
// first + l of the sequence (-1: not a page of the cache).  (idx, off): the
// page and the place in it of the next 16 tokens to be read.
struct AttnPages {
    const int32_t* row;
    int first, last;
    int needed;  // first page with a token that some row sees (a page before it may be gone)
    int idx, off;
    int entry;
    NVFP4_DEV void fill(const AttnArgs& a, int i0)
    {
        first = i0;
        int i = i0 + (int)(threadIdx.x & 63);
        i = i < last ? i : last;
        const int e = row[i];
        const bool ok = e >= 0 && e < a.num_pages;
        if (!ok && i >= needed)
            raise_error(NVFP4_ERR_RANGE);
        entry = ok ? e : -1;
    }
    NVFP4_DEV int get(const AttnArgs& a)
    {
        const int i = idx < last ? idx : last;  // past the end: any page, masked
        if (i - first >= 64)
            fill(a, i);
        return __builtin_amdgcn_readlane(entry, i - first);
    }
    NVFP4_DEV void next(const AttnArgs& a)
    {
        off += 16;
        const bool over = off == a.page;
        off = over ? 0 : off;
        idx += over;
    }
};

// A wave's walk over the tokens of one KV head for 16 NT query rows.
template <int D, int NT, bool TREE = false>
struct AttnWave {
    half8_t q[NT][D / 32];
    float4_t o[NT][D / 16];
    float m[NT], l[NT], c1[NT];
    int k[NT];  // m, c1 and the scores are in units of 2^k
    int start[NT], end[NT];
    int token[TREE ? NT : 1], base;  // TREE: the rows' query tokens (rows of q and of the mask); the first draft
    // the lane's part of the copies: its place in 16 tokens' codes (of the even and the odd copies of a
    // half) and its row among the 32 tokens' scales
    uint32_t co[2], so;

    // rows row0 .. row0 + 16 NT of sequence s: row r is query token r / group, head r % group of KV head h
    NVFP4_DEV void open(const AttnArgs& a, const AttnSeq& s, int h, int row0)
    {
        const float kg = *a.k_global;
        const uint32_t lane = threadIdx.x & 63, stride = a.kv_heads;
        base = s.kv - s.nq;
        const uint32_t r = (lane / (D / 32)) & 15, c = lane % (D / 32);
        co[0] = r * stride * (D / 2) + 16 * (c ^ attn_swz<D>(r));
        co[1] = D == 256 ? (r + 8) * stride * (D / 2) + 16 * (c ^ attn_swz<D>(r + 8)) : co[0];
        so = D == 128 ? ((lane >> 1) & 15) * stride * (D / 16) + 4 * (lane & 1) : (lane & 15) * stride * (D / 16);
#pragma unroll
        for (int t = 0; t < NT; t++) {
            const int r = row0 + 16 * t + lane_n();
            const int i = r / a.group, hh = r - i * a.group;
            const bool in = i < s.nq;
            start[t] = end[t] = 0;
            u32x4 w[D / 32];
            uint32_t am = 0;
            if constexpr (TREE) {
                token[t] = s.q0 + (in ? i : 0);
                if (in) {
                    start[t] = attn_tree_start(a, s, i);
                    end[t] = s.kv;
                }
            } else if (in) {
                attn_limits(a, s, i, &start[t], &end[t]);
            }
            const uint16_t* src = a.q + (int64_t)(s.q0 + (in ? i : 0)) * a.ld_q + (int64_t)(h * a.group + hh) * D +
                                  lane_g() * (D / 4);
#pragma unroll
            for (int c = 0; c < D / 32; c++) {
                w[c] = (u32x4){0, 0, 0, 0};
                if (in)
                    w[c] = *(const u32x4*)(src + 8 * c);
                am = umax_u32(am, absmax_bits8(w[c]));
            }
            am = umax_u32(am, (uint32_t)__shfl_xor((int)am, 16, 64));
            am = umax_u32(am, (uint32_t)__shfl_xor((int)am, 32, 64));
            // the row's largest magnitude is f * 2^e, f in [1, 2)
            const float top = __uint_as_float(am << 16);
            const int e = am ? __builtin_amdgcn_frexp_expf(top) - 1 : 0;
            c1[t] = attn_factor(a.scale_log2, kg, e, &k[t]);
#pragma unroll
            for (int c = 0; c < D / 32; c++)
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    q[t][c][2 * j] = (_Float16)__builtin_ldexpf(bf16_lo(w[c][j]), -e);
                    q[t][c][2 * j + 1] = (_Float16)__builtin_ldexpf(bf16_hi(w[c][j]), -e);
                }
            m[t] = kAttnLow;
            l[t] = 0.0f;
#pragma unroll
            for (int dd = 0; dd < D / 16; dd++)
                o[t][dd] = (float4_t){0, 0, 0, 0};
        }
    }

    // Copies of one step of K (or V).
    static constexpr int kCopies = D == 64 ? 2 : (D == 128 ? 3 : 5);

    // request the 32 tokens of K (or V) whose halves begin at cache rows row[]
    NVFP4_DEV void request(const uint8_t* packed, const uint8_t* scales, const int64_t (&row)[2], uint8_t* dst) const
    {
        const int lane = threadIdx.x & 63;
        wait_lgkm0();  // the reads of dst's last step are done
        const int64_t apart = row[1] - row[0];
        if constexpr (D == 64) {
            __builtin_amdgcn_global_load_lds((const void*)(packed + (row[0] + (lane < 32 ? 0 : apart)) * (D / 2) + co[0]),
                                             (attn_lds_t)dst, 16, 0, 0);
        } else {
#pragma unroll
            for (int i = 0; i < D / 64; i++)
                __builtin_amdgcn_global_load_lds(
                    (const void*)(packed + row[i / (D / 128)] * (D / 2) + co[D == 256 ? i & 1 : 0]),
                    (attn_lds_t)(dst + i * 1024), 16, 0, 0);
        }
        // D = 128: two lanes per row; else one (lanes 32 .. 63 copy the same again, behind)
        const bool second = D == 128 ? lane >= 32 : (lane & 16) != 0;
        const uint8_t* src = scales + (row[0] + (second ? apart : 0)) * (D / 16) + so;
        if constexpr (D == 256)
            __builtin_amdgcn_global_load_lds((const void*)src, (attn_lds_t)(dst + 16 * D), 16, 0, 0);
        else
            __builtin_amdgcn_global_load_lds((const void*)src, (attn_lds_t)(dst + 16 * D), 4, 0, 0);
    }

    // S^T of one step: tokens t0 .. t0 + 32 from a finished copy of K (SWAP: S, the rows of q as rows and the
    // tokens as columns)
    template <bool SWAP = false>
    NVFP4_DEV void scores(const uint8_t* src, float4_t (&s)[NT][2]) const
    {
        const int n = lane_n(), g = lane_g();
        const int kt = 4 * (n & 3) + (n >> 2);  // row n of a K tile
        uint32_t kc[2][D / 32], ks[2];
#pragma unroll
        for (int half = 0; half < 2; half++) {
            const int k = (16 * half + kt) * (D / 2);
            if constexpr (D == 64) {
                const u32x2 w = *(const u32x2*)(src + (k + 8 * g));
                kc[half][0] = w.x;
                kc[half][1] = w.y;
            } else {
#pragma unroll
                for (int c = 0; c < D / 128; c++) {
                    const u32x4 w = *(const u32x4*)(src + (k + 16 * ((g * (D / 128) + c) ^ attn_swz<D>(kt))));
#pragma unroll
                    for (int i = 0; i < 4; i++)
                        kc[half][4 * c + i] = w[i];
                }
            }
            const int b = 16 * D + (16 * half + kt) * (D / 16) + g * (D / 64);
            if constexpr (D == 64)
                ks[half] = src[b];
            else if constexpr (D == 128)
                ks[half] = *(const uint16_t*)(src + b);
            else
                ks[half] = *(const uint32_t*)(src + b);
        }
#pragma unroll
        for (int half = 0; half < 2; half++) {
#pragma unroll
            for (int t = 0; t < NT; t++)
                s[t][half] = (float4_t){0, 0, 0, 0};
#pragma unroll
            for (int c = 0; c < D / 32; c++) {
                const uint32_t b = ks[half] >> (8 * (c >> 1));
                const half8_t k = decode_row8(kc[half][c], scale_pair(b, b));
#pragma unroll
                for (int t = 0; t < NT; t++)
                    s[t][half] = SWAP ? mfma16(q[t][c], k, s[t][half]) : mfma16(k, q[t][c], s[t][half]);
            }
        }
    }

    // P^T of one step; ok: which halves lie in a page of the cache
    NVFP4_DEV void weights(const AttnArgs& a, float4_t (&s)[NT][2], half8_t (&p)[NT], int t0, bool inside,
                           const bool (&ok)[2])
    {
#pragma unroll
        for (int t = 0; t < NT; t++) {
            if (!inside) {
                uint32_t bits = 0;
                if constexpr (TREE)
                    bits = attn_tree_bits(a, token[t], t0 - base) >> lane_g();
#pragma unroll
                for (int half = 0; half < 2; half++)
#pragma unroll
                    for (int i = 0; i < 4; i++) {
                        const int tok = t0 + 16 * half + 4 * i + lane_g();
                        const bool seen = ok[half] && tok >= start[t] && tok < end[t] &&
                                          (!TREE || (bits >> (16 * half + 4 * i) & 1));
                        s[t][half][i] = seen ? s[t][half][i] : -__builtin_inff();
                    }
            }
            float top = s[t][0][0];
#pragma unroll
            for (int i = 1; i < 8; i++)
                top = __builtin_fmaxf(top, s[t][i >> 2][i & 3]);
            top *= c1[t];
            if (__any(top > m[t] + kAttnLazy)) {
                top = __builtin_fmaxf(top, __shfl_xor(top, 16, 64));
                top = __builtin_fmaxf(top, __shfl_xor(top, 32, 64));
                const float f = attn_grow(__builtin_fmaxf(m[t], top), &m[t], &c1[t], &k[t]);
                l[t] *= f;
#pragma unroll
                for (int dd = 0; dd < D / 16; dd++)
                    o[t][dd] *= f;
            }
            const float lift = kAttnLift - m[t];
            float e[8];
#pragma unroll
            for (int i = 0; i < 8; i++)
                e[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[t][i >> 2][i & 3], c1[t], lift));
            l[t] += ((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7]));
#pragma unroll
            for (int i = 0; i < 8; i++)
                p[t][i] = (_Float16)e[i];
        }
    }

    // O^T += V^T P^T of one step from a finished copy of V
    NVFP4_DEV void values(const uint8_t* src, const half8_t (&p)[NT])
    {
        const int n = lane_n(), g = lane_g();
        uint32_t vc[8][D > 128 ? D / 128 : 1], vs[8];
#pragma unroll
        for (int half = 0; half < 2; half++)
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const int r = 4 * j + g;
                const int v = (16 * half + r) * (D / 2);
                if constexpr (D == 64) {
                    vc[4 * half + j][0] = *(const uint16_t*)(src + (v + 2 * n));
                } else if constexpr (D == 128) {
                    vc[4 * half + j][0] = *(const uint32_t*)(src + (v + 16 * ((n >> 2) ^ attn_swz<D>(r)) + 4 * (n & 3)));
                } else {
                    const u32x2 w = *(const u32x2*)(src + (v + 16 * ((n >> 1) ^ attn_swz<D>(r)) + 8 * (n & 1)));
                    vc[4 * half + j][0] = w.x;
                    vc[4 * half + j][1] = w.y;
                }
                vs[4 * half + j] = src[16 * D + (16 * half + r) * (D / 16) + n * D / 256];
            }
        half2_t sc[4];
#pragma unroll
        for (int j = 0; j < 4; j++)
            sc[j] = scale_pair(vs[2 * j], vs[2 * j + 1]);
        // token pairs side by side: byte i of even / odd holds elements 2i / 2i + 1 of both tokens
#pragma unroll
        for (int w = 0; w < (D > 128 ? D / 128 : 1); w++) {
            uint32_t even[4], odd[4];
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const uint32_t x = vc[2 * j][w], y = vc[2 * j + 1][w];
                even[j] = (x & 0x0F0F0F0Fu) | ((y << 4) & 0xF0F0F0F0u);
                odd[j] = ((x >> 4) & 0x0F0F0F0Fu) | (y & 0xF0F0F0F0u);
            }
            // (the byte selector of the conversion is an immediate)
#define ATTN_PV(I)                                                                                           \
    if constexpr (8 * (D > 128 ? D / 128 : 1) > 0 && 2 * (I) < D / 16) {                                     \
        half8_t ve, vo;                                                                                      \
        _Pragma("unroll") for (int j = 0; j < 4; j++)                                                       \
        {                                                                                                    \
            const half2_t x = FP4_TO_F16X2_256(even[j], I) * sc[j], y = FP4_TO_F16X2_256(odd[j], I) * sc[j]; \
            ve[2 * j] = x.x;                                                                                 \
            ve[2 * j + 1] = x.y;                                                                             \
            vo[2 * j] = y.x;                                                                                 \
            vo[2 * j + 1] = y.y;                                                                             \
        }                                                                                                    \
        _Pragma("unroll") for (int t = 0; t < NT; t++)                                                      \
        {                                                                                                    \
            o[t][8 * w + 2 * (I)] = mfma16(ve, p[t], o[t][8 * w + 2 * (I)]);                                 \
            o[t][8 * w + 2 * (I) + 1] = mfma16(vo, p[t], o[t][8 * w + 2 * (I) + 1]);                         \
        }                                                                                                    \
    }
            ATTN_PV(0)
            ATTN_PV(1)
            ATTN_PV(2)
            ATTN_PV(3)
#undef ATTN_PV
        }
    }

    // the cache rows of the next 32 tokens' halves; ok: which lie in a page of the cache
    NVFP4_DEV void rows(const AttnArgs& a, AttnPages& pages, int64_t (&row)[2], bool (&ok)[2], int h) const
    {
#pragma unroll
        for (int half = 0; half < 2; half++) {
            const int page = pages.get(a);
            ok[half] = page >= 0;
            row[half] = ((int64_t)(page < 0 ? 0 : page) * a.page + pages.off) * a.kv_heads + h;
            pages.next(a);
        }
    }

    // tokens [t0, t1) (t0 a multiple of 32); any: the first token that some
    // row sees; [lo, hi): the tokens that every row sees.  The next step's K is
    // requested as soon as this step's is in registers, and V likewise, so
    // that one of them is always under way.  Past the end the requests go to
    // the last page again (lines that are near) and the copy is not used.
    NVFP4_DEV void walk(const AttnArgs& a, const int32_t* table_row, int h, int t0, int t1, int any, int lo, int hi,
                        uint8_t* bufk, uint8_t* bufv)
    {
        if (t0 >= t1)
            return;
        AttnPages pages;
        pages.row = table_row;
        pages.last = (t1 - 1) / a.page;
        pages.needed = any / a.page;
        pages.idx = t0 / a.page;
        pages.off = t0 - pages.idx * a.page;
        pages.fill(a, pages.idx);
        int64_t row[2];
        bool ok[2], next[2];
        rows(a, pages, row, ok, h);
        request(a.k_packed, a.k_scales, row, bufk);
        request(a.v_packed, a.v_scales, row, bufv);
        for (int t = t0; t < t1; t += kAttnStep) {
            float4_t s[NT][2];
            half8_t p[NT];
            wait_copies<kCopies>();
            scores(bufk, s);
            rows(a, pages, row, next, h);
            request(a.k_packed, a.k_scales, row, bufk);
            weights(a, s, p, t, ok[0] && ok[1] && t >= lo && t + kAttnStep <= hi, ok);
            wait_copies<kCopies>();
            values(bufv, p);
            request(a.v_packed, a.v_scales, row, bufv);
            ok[0] = next[0];
            ok[1] = next[1];
        }
        wait_vm<0>();
    }

    // the sums of the lane groups, the maxima in units of 1
    NVFP4_DEV void close()
    {
#pragma unroll
        for (int t = 0; t < NT; t++) {
            m[t] = attn_whole(m[t], k[t]);
            l[t] += __shfl_xor(l[t], 16, 64);
            l[t] += __shfl_xor(l[t], 32, 64);
        }
    }
};

// Joins the waves that walked different tokens for the same head: wave w
// holds head lane w % hl and token lane w / hl.  buf: D / 4 + 2 floats x 64
// lanes x NT per writing wave, half the waves at most.  Afterwards token lane
// 0 holds the whole.
template <int D, int NT, bool TREE>
NVFP4_DEV void attn_join(AttnWave<D, NT, TREE>& w, int hl, int wave, float* buf)
{
    constexpr int kRow = D / 4 + 2;
    const int tl = wave / hl, lane = threadIdx.x & 63;
    for (int s = attn_waves<D, NT>() / hl / 2; s > 0; s >>= 1) {
        __syncthreads();
        if (tl >= s && tl < 2 * s) {
            float* b = buf + (wave - s * hl) * (kRow * NT * 64) + lane;
#pragma unroll
            for (int t = 0; t < NT; t++) {
                b[(t * kRow) * 64] = w.m[t];
                b[(t * kRow + 1) * 64] = w.l[t];
#pragma unroll
                for (int i = 0; i < D / 4; i++)
                    b[(t * kRow + 2 + i) * 64] = w.o[t][i >> 2][i & 3];
            }
        }
        __syncthreads();
        if (tl < s) {
            const float* b = buf + wave * (kRow * NT * 64) + lane;
#pragma unroll
            for (int t = 0; t < NT; t++) {
                const float om = b[(t * kRow) * 64], m = __builtin_fmaxf(w.m[t], om);
                const float f = __builtin_amdgcn_exp2f(w.m[t] - m), g = __builtin_amdgcn_exp2f(om - m);
                w.m[t] = m;
                w.l[t] = w.l[t] * f + b[(t * kRow + 1) * 64] * g;
#pragma unroll
                for (int i = 0; i < D / 4; i++)
                    w.o[t][i >> 2][i & 3] = w.o[t][i >> 2][i & 3] * f + b[(t * kRow + 2 + i) * 64] * g;
            }
        }
    }
}

// Rows of a finished wave: o V-global / l as bf16, and lse.
template <int D, int NT, bool TREE>
NVFP4_DEV void attn_finish(const AttnArgs& a, const AttnWave<D, NT, TREE>& w, const AttnSeq& s, int h, int row0)
{
    const float vg = *a.v_global;
#pragma unroll
    for (int t = 0; t < NT; t++) {
        const int r = row0 + 16 * t + lane_n();
        const int i = r / a.group, hh = r - i * a.group;
        if (i >= s.nq)
            continue;
        const int head = h * a.group + hh;
        const int64_t token = s.q0 + i;
        const float f = w.l[t] != 0.0f ? vg / w.l[t] : 0.0f;  // a row that sees nothing: zeros
        uint16_t* dst = a.out + token * a.ld_out + (int64_t)head * D + 4 * lane_g() * (D / 16);
#pragma unroll
        for (int k = 0; k < 4; k++)
#pragma unroll
            for (int dd = 0; dd < D / 16; dd += 4)
                *(u32x2*)(dst + k * (D / 16) + dd) =
                    (u32x2){pack_bf16x2(w.o[t][dd][k] * f, w.o[t][dd + 1][k] * f),
                            pack_bf16x2(w.o[t][dd + 2][k] * f, w.o[t][dd + 3][k] * f)};
        if (a.lse && lane_g() == 0)
            a.lse[token * (a.kv_heads * a.group) + head] =
                w.l[t] != 0.0f ? (w.m[t] - kAttnLift + __builtin_amdgcn_logf(w.l[t])) * 0.69314718056f
                               : -__builtin_inff();
    }
}

// Floats that one wave leaves of a part of its tokens: m, l and o of its 64
// lanes, 16 NT query rows.
template <int D, int NT>
constexpr int attn_part() { return (D / 4 + 2) * NT * 64; }

// Rows of 16 that a part keeps: value e of row n and lane group g is at
// (4 e + g) rows + n (0: m, 1: l, 2 + i: o).
NVFP4_DEV int attn_part_rows(int left) { return left < 0 ? 0 : (left < 16 ? left : 16); }

// The shares: the units of all sequences in a row, cut into equal runs of at
// least kAttnLeast units.  Share w holds units [w T / W, (w + 1) T / W).
constexpr int kAttnLeast = 4;
NVFP4_DEV int attn_shares(const AttnArgs& a, int total)
{
    const int most = (total + kAttnLeast - 1) / kAttnLeast;
    return most < a.workers ? most : a.workers;
}

template <int D, int NT, bool TREE>
NVFP4_DEV AttnCount attn_count(const AttnArgs& a, const AttnSeq& s)
{
    int lo0, hi0, lo1, hi1;
    attn_span<TREE>(a, s, 0, s.nq > 0 ? s.nq - 1 : 0, &lo0, &hi0, &lo1, &hi1);
    const int t0 = lo0 & ~(kAttnStep - 1);
    AttnCount c;
    c.tiles = (s.nq * a.group + 16 * NT - 1) / (16 * NT);
    c.units = hi1 > t0 ? (hi1 - t0 + kAttnStep - 1) / kAttnStep : 1;
    c.down = s.down;
    return c;
}

// A tile of rows as the row kernel leaves it to the joining one: the first of
// the `parts` shares that hold its tokens, and its rows.  Entry 0 of the list
// holds the number of tiles in `parts`, entry 1 + i tile i.
struct AttnTile {
    int first, parts, q0, nq, row0, pad[3];
};

// Few query rows per sequence (decode, drafts): the time is the K and V
// bytes' way from HBM.  The tokens of all sequences are cut into equal shares,
// one per resident workgroup, so that long and short sequences load the chip
// alike; a share that holds a whole tile of rows writes its output, one that
// holds a part leaves (m, l, o) for attn_combine_kernel, in slot 1 if it holds
// the tile's first unit, else in slot 0 (a share has at most one of each).
// A workgroup holds head_lanes KV heads side by side, which lie next to each
// other in memory, and (waves / head_lanes) runs of the tokens.
template <int D, int NT, bool TREE>
__global__ void __launch_bounds__((64 * attn_waves<D, NT>()), (D * NT <= 64 ? 4 : (D * NT <= 256 ? 2 : 1)))
attn_rows_kernel(AttnArgs a)
{
    // the waves' copies of K and V; between walks the space of joined waves
    constexpr int kWaves = attn_waves<D, NT>(), kStages = kWaves * attn_stage<D>();
    constexpr int kJoin = kWaves / 2 * attn_part<D, NT>() * 4;
    __shared__ __attribute__((aligned(16))) uint8_t bufk[kStages > kJoin ? kStages : kJoin];
    __shared__ __attribute__((aligned(16))) uint8_t bufv[kStages];
    const int wave = uniform((int)(threadIdx.x >> 6));
    const int hl = a.head_lanes, tls = kWaves / hl;
    // workgroups go to the 8 XCDs in turn: the head blocks of one share go to
    // the same one, whose L2 then holds the lines that they share
    const int blocks = a.kv_heads / hl;
    const int hb = blockIdx.x / 8 % blocks, w = blockIdx.x / (8 * blocks) * 8 + blockIdx.x % 8;
    const int h = hb * hl + wave % hl, tl = wave / hl;
    AttnSeq own{0, 0, 0, false};
    auto count = [&](int b) {
        own = attn_seq(a, b);
        AttnCount c = attn_count<D, NT, TREE>(a, own);
        c.units = a.whole ? 1 : c.units;  // whole tiles: w counts tiles
        return c;
    };
    const AttnScan scan = attn_scan(a.seqs, count);
    const int64_t total = scan.units, shares = a.whole ? scan.units : attn_shares(a, scan.units);
    if (!a.whole && w == 0 && hb == 0 && threadIdx.x == 0)
        a.tiles[0].parts = scan.tiles;
    if (w >= shares)
        return;
    int u = (int)(w * total / shares);
    const int u1 = (int)((w + 1) * total / shares);
    AttnFound f = attn_find(scan, a.seqs, u, count);
    while (u < u1) {
        const AttnSeq s = attn_seq_uniform(a, own, f.seq);
        AttnCount c = attn_count<D, NT, TREE>(a, s);
        const int units = c.units;
        c.units = a.whole ? 1 : c.units;
        if (f.at >= c.tiles * c.units) {
            f.before.tiles += c.tiles;
            f.before.units += c.tiles * c.units;
            f.seq++;
            f.at = 0;
            continue;
        }
        const int tile = f.at / c.units, first = f.at - tile * c.units;
        const int n = a.whole ? units : (units - first < u1 - u ? units - first : u1 - u);
        const int row0 = tile * 16 * NT;
        if (!a.whole && first == 0 && hb == 0 && threadIdx.x == 0) {
            const int64_t end = u + units;  // the share of the tile's last unit
            a.tiles[1 + f.before.tiles + tile] = AttnTile{w, (int)((end * shares - 1) / total) - w + 1, s.q0, s.nq, row0};
        }
        int any, none, lo0, hi0, lo1, hi1;  // tokens of the sequence's, the tile's first and last row
        const int last = (row0 + 16 * NT - 1) / a.group;
        attn_span<TREE>(a, s, row0 / a.group, last < s.nq ? last : s.nq - 1, &lo0, &hi0, &lo1, &hi1);
        if constexpr (TREE) {
            any = lo0;
            attn_tree_check(a, s);
        } else {
            attn_limits(a, s, 0, &any, &none);
        }
        AttnWave<D, NT, TREE> x;
        x.open(a, s, h, row0);
        const int t0 = (any & ~(kAttnStep - 1)) + first * kAttnStep;
        const int share = (n + tls - 1) / tls * kAttnStep;
        int from = t0 + tl * share, to = from + share;
        to = to < t0 + n * kAttnStep ? to : t0 + n * kAttnStep;
        to = to < hi1 ? to : hi1;
        from = from > (lo0 & ~(kAttnStep - 1)) ? from : lo0 & ~(kAttnStep - 1);
        x.walk(a, a.table + f.seq * a.ld_table, h, from, to, lo0, lo1, hi0,
               bufk + wave * attn_stage<D>(), bufv + wave * attn_stage<D>());
        x.close();
        if (tls > 1) {
            attn_join(x, hl, wave, (float*)bufk);
            __syncthreads();
        }
        if (tl == 0) {
            if (n == units) {
                attn_finish(a, x, s, h, row0);
            } else {
                const int slot = first == 0;
                float* dst = a.partial + (((int64_t)w * blocks + hb) * 2 + slot) * hl * attn_part<D, NT>() +
                             (wave % hl) * attn_part<D, NT>();
#pragma unroll
                for (int t = 0; t < NT; t++) {
                    const int rows = attn_part_rows(s.nq * a.group - row0 - 16 * t);
                    float* p = dst + t * (D / 4 + 2) * 64 + lane_g() * rows + lane_n();
                    if (lane_n() < rows) {
                        p[0] = x.m[t];
                        p[4 * rows] = x.l[t];
#pragma unroll
                        for (int i = 0; i < D / 4; i++)
                            p[(2 + i) * 4 * rows] = x.o[t][i >> 2][i & 3];
                    }
                }
            }
        }
        u += a.whole ? 1 : n;
        f.at += a.whole ? 1 : n;
    }
}

// Joins what the shares left of one tile of rows (blockIdx.x) for one KV head
// (blockIdx.y), 16 of its rows (blockIdx.z % NT), in the order of the tokens,
// with the running maximum and sum of the walk.  A wave holds a piece of 4
// output elements per lane; `pieces` waves of a workgroup take different
// pieces, the others different runs of the parts, joined through shared
// memory.  What it takes is the latency of three dependent reads and the launch.
template <int D, int NT>
__global__ void __launch_bounds__(1024)
attn_combine_kernel(AttnArgs a, int pieces)
{
    __shared__ float4_t sum[16][64];
    __shared__ float2_t red[16][64];
    const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
    const int wave = uniform((int)(threadIdx.x >> 6)), waves = blockDim.x >> 6;
    // (both read before the first test, so that their latencies overlap)
    const int tiles = a.tiles[0].parts;
    const AttnTile tile = a.tiles[1 + blockIdx.x];
    const float vg = *a.v_global;
    const int parts = uniform(tile.parts), w0 = uniform(tile.first);
    if ((int)blockIdx.x >= tiles || parts == 1)
        return;  // no such tile, or one share held the whole of it
    const int hl = a.head_lanes, blocks = a.kv_heads / hl;
    const int h = blockIdx.y, hb = h / hl;
    // part p: the share w0 + p, slot 1 of the first, slot 0 of the others
    auto part = [&](int p) {
        return a.partial + (((int64_t)(w0 + p) * blocks + hb) * 2 + (p == 0)) * hl * attn_part<D, NT>() +
               (h - hb * hl) * attn_part<D, NT>();
    };
    const int runs = waves / pieces, pw = wave / pieces;
    const int run = (parts + runs - 1) / runs, p0 = pw * run, p1 = p0 + run < parts ? p0 + run : parts;
    const int t = blockIdx.z % NT;
    const int rows = attn_part_rows(tile.nq * a.group - tile.row0 - 16 * t);
    if (rows == 0)
        return;
    const bool in = n < rows;
    const int off = t * (D / 4 + 2) * 64 + g * rows + (in ? n : 0);
    const int r = tile.row0 + 16 * t + n;
    const int i = r / a.group, head = h * a.group + r - i * a.group;
    const int64_t token = tile.q0 + i;
    const int c = blockIdx.z / NT * pieces + wave % pieces;
    const int k = c / (D / 64), dd = 4 * (c - k * (D / 64));
    float m = kAttnLow, l = 0.0f;
    float4_t o = (float4_t){0, 0, 0, 0};
    auto join = [&](float om, float ol, float4_t oo) {
        const float now = __builtin_fmaxf(m, om);
        const float f = __builtin_amdgcn_exp2f(m - now), q = __builtin_amdgcn_exp2f(om - now);
        l = l * f + ol * q;
        o = o * f + oo * q;
        m = now;
    };
#pragma unroll 4
    for (int p = p0; p < p1; p++) {
        const float* src = part(p) + off;
        float4_t oo;
#pragma unroll
        for (int j = 0; j < 4; j++)
            oo[j] = src[(2 + 4 * (dd + j) + k) * 4 * rows];
        join(src[0], src[4 * rows], oo);
    }
    if (runs > 1) {
        sum[wave][lane] = o;
        red[wave][lane] = (float2_t){m, l};
        __syncthreads();
        for (int q = 1; q < runs && pw == 0; q++) {
            const float2_t ml = red[wave + q * pieces][lane];
            join(ml.x, ml.y, sum[wave + q * pieces][lane]);
        }
    }
    if (pw != 0 || !in)
        return;
    const float scale = l != 0.0f ? vg / l : 0.0f;
    *(u32x2*)(a.out + token * a.ld_out + (int64_t)head * D + (4 * g + k) * (D / 16) + dd) =
        (u32x2){pack_bf16x2(o[0] * scale, o[1] * scale), pack_bf16x2(o[2] * scale, o[3] * scale)};
    if (a.lse && c == 0 && g == 0)
        a.lse[token * (a.kv_heads * a.group) + head] =
            l != 0.0f ? (m - kAttnLift + __builtin_amdgcn_logf(l)) * 0.69314718056f : -__builtin_inff();
}

// ---------------------------------------------------------------------------
// Many query rows per sequence (chunks, prompts): the time is the two
// products.  A workgroup of NW waves takes a tile of 32 NW query rows of one
// sequence and KV head, each wave 32 of them, and walks the tokens in blocks
// of 64.  A block of K and V is decoded to f16 once for all waves, into one of
// two buffers in shared memory while the other is multiplied: decoding it in
// every wave took 680 VALU cycles a wave for 512 cycles of products (D = 128).
//
// v_mfma_f32_32x32x16_f16 (A: row l % 32, B: column l % 32, both elements
// 8 (l / 32) .. + 8 of the contraction; output: column l % 32, rows
// 8 (i / 4) + 4 (l / 32) + i % 4 for register i of lane l), transposed as in
// the row kernel: S^T = K Q^T, O^T = V^T P^T, and eight registers of S^T are
// a lane's share of P^T for 16 tokens.  They are tokens 4 e .. 4 e + 3 and
// 8 + 4 e .. + 3 of the 16 (e = l / 32), so V^T rows are kept with their tokens
// in that order: token t of 16 at place t % 4 + 4 (t / 8) + 8 (t / 4 % 2).
// ---------------------------------------------------------------------------
constexpr int kTileTok = 64;

// TREE: the work of each of a sequence's tiles, in blocks of tokens, and the shares that the work of all tiles is
// cut into.  Starting and ending a tile counts as kTileStart blocks, which come first, so that shares of many
// short tiles take no longer than those of a long one (32 trees of 26-63 drafts on 300-16000 tokens, replayed: 213 us
// with two, 201 with four, 200 with eight; 4 trees of 60 on 2000 tokens, 4 KV heads of 256: 58, 57, 59; one of 60 on
// 3000, 8 heads of 128: 36, 36, 38).  Before waves without rows were left out a split of each tile's blocks into as
// many parts as fill the chip took 421 us for the first, equal pieces of tiles 251 and these shares 220.
constexpr int kTileStart = 4;
NVFP4_DEV int attn_tile_units(const AttnArgs& a, const AttnSeq& s)
{
    const int base = attn_tree_base(s), b0 = a.window > 0 && base > a.window ? (base - a.window) / kTileTok : 0;
    return (s.kv + kTileTok - 1) / kTileTok - b0 + kTileStart;
}

NVFP4_DEV int attn_tile_shares(const AttnArgs& a, int total)
{
    const int most = (total + kTileStart) / (kTileStart + 1);
    return most < a.workers ? most : a.workers;
}

// Place (in 16-byte chunks) of chunk c of row r in the f16 tiles, rows of C
// chunks: the XOR spreads both the operand reads (32 consecutive rows, one
// chunk) and the writes over the banks.
template <int C>
NVFP4_DEV int tile_chunk(int r, int c)
{
    return r * C + (c ^ (C >= 16 ? r & 15 : ((r >> 1) ^ (r >> 4)) & 7));
}

// (a kernel's pieces: a call would put the registers that they share in memory)
#define ATTN_INLINE __attribute__((always_inline))

// f(integral_constant<int, B>), ..., f(integral_constant<int, E - 1>)
template <int B, int E, class F>
NVFP4_DEV void for_range(F f)
{
    if constexpr (B < E) {
        f(std::integral_constant<int, B>{});
        for_range<B + 1, E>(f);
    }
}

NVFP4_DEV float16_t mfma32(half8_t a, half8_t b, float16_t c)
{
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}

// What one of 256 threads holds of a block on its way: kK elements of one
// token of K, and kV elements of four tokens of V.
template <int D>
struct TileRaw {
    static constexpr int kK = kTileTok * D / 256, kV = kK / 4;
    static constexpr int kUnits = kK / 8;  // pieces of decoding of K (8 elements each) and of V (2 of each token)
    uint32_t kc[kK / 8];
    uint32_t ks;
    uint32_t vc[4][kV > 8 ? kV / 8 : 1];
    uint32_t vs[4];
    bool ok;  // K's page is one of the cache
};

// N bytes (1, 2, 4, 8, 16 or 32) from src into dwords.
template <int N>
NVFP4_DEV void load_bytes(const uint8_t* src, uint32_t* w)
{
    if constexpr (N == 1) {
        w[0] = *src;
    } else if constexpr (N == 2) {
        w[0] = *(const uint16_t*)src;
    } else if constexpr (N == 4) {
        w[0] = *(const uint32_t*)src;
    } else if constexpr (N == 8) {
        const u32x2 v = *(const u32x2*)src;
        w[0] = v.x;
        w[1] = v.y;
    } else {
#pragma unroll
        for (int i = 0; i < N / 16; i++) {
            const u32x4 v = ((const u32x4*)src)[i];
#pragma unroll
            for (int j = 0; j < 4; j++)
                w[4 * i + j] = v[j];
        }
    }
}

// Byte I of an interleaved dword (two tokens' codes of one element) under the two tokens' scales.
template <int I>
NVFP4_DEV uint32_t decode_pair(uint32_t w, half2_t s)
{
    return __builtin_bit_cast(uint32_t, FP4_TO_F16X2_256(w, I) * s);
}

// o *= f for accumulators that fill the accumulation registers (D = 256: 128 of
// a wave's 512 registers).  Written as a plain product under the rare branch
// that grows the maximum, it made the compiler move all 128 to the other half
// of the register file and back in every block (128 moves of 4 cycles against
// 2062 of products); the constraints keep them where the products want them.
// The compiler does not see these moves, so the waits that a product (16
// passes) asks for before its result is read, and a move before its result is
// an operand, are written out.
template <int N>
NVFP4_DEV void scale_acc(float16_t (&o)[N], float f)
{
    asm volatile("s_nop 15\n\ts_nop 7" ::: "memory");
#pragma unroll
    for (int d = 0; d < N; d++)
#pragma unroll
        for (int i = 0; i < 16; i++) {
            float x;
            asm volatile("v_accvgpr_read_b32 %0, %1" : "=v"(x) : "a"(o[d][i]));
            x *= f;
            float y;
            asm volatile("v_accvgpr_write_b32 %0, %1\n\ts_nop 1" : "=a"(y) : "v"(x));
            o[d][i] = y;
        }
}

template <int D, int NW, bool TREE>
__global__ void __launch_bounds__((64 * NW), (D == 256 ? 1 : 2))
attn_tile_kernel(AttnArgs a)
{
    constexpr int NT = 64 * NW, ROWS = 32 * NW;
    constexpr int KC = D / 8;  // chunks of a K row
    typedef TileRaw<D> Raw;
    // Eight waves: two on each SIMD, in two groups that take turns.  While one
    // group multiplies S^T (and decodes), the other weighs P and multiplies
    // O^T, half a block behind; waves that all waited at one barrier a block
    // stood in the same phase and hardly overlapped the matrix unit with the
    // rest.  The first group decodes K and the second V: what either writes is
    // then read by both a barrier later and no longer by anybody when it is
    // written again.  Four waves decode both.
    constexpr bool kTurns = NW == 8;
    // (separate arrays, picked at compile time, so that the compiler may move
    // the reads of one buffer past the writes of the other)
    __shared__ __attribute__((aligned(16))) u32x4 lk0[kTileTok * KC], lk1[kTileTok * KC];
    __shared__ __attribute__((aligned(16))) u32x4 lv0[D * 8], lv1[D * 8];
    __shared__ __attribute__((aligned(16))) int lok[2][4];  // which 16 tokens lie in a page of the cache
    // ---- the tile: heavy ones first (causal tiles grow towards the end).  TREE: a share of the blocks of all
    // tiles, as in the row kernel: the tiles are few and their contexts unlike
    const int h = blockIdx.x % a.kv_heads;
    const int split = TREE ? 0 : blockIdx.y;
    AttnSeq own{0, 0, 0, false};
    auto count = [&](int b) ATTN_INLINE {
        own = attn_seq(a, b);
        return AttnCount{(own.nq * a.group + ROWS - 1) / ROWS, TREE ? attn_tile_units(a, own) : 1, own.down};
    };
    const AttnScan scan = attn_scan(a.seqs, count);
    const int slot = blockIdx.x / a.kv_heads;
    if ((TREE || gridDim.y > 1) && blockIdx.x == 0 && split == 0 && threadIdx.x == 0)
        a.tiles[0].parts = TREE ? scan.tiles : scan.units;
    const int total = scan.units, shares = TREE ? attn_tile_shares(a, total) : 1;
    if (slot >= (TREE ? shares : total))
        return;
    int unit = TREE ? uniform((int)((int64_t)slot * total / shares)) : total - 1 - slot;
    const int unit_end = TREE ? uniform((int)((int64_t)(slot + 1) * total / shares)) : unit + 1;
    AttnFound f = attn_find(scan, a.seqs, unit, count);
    do {
    // (TREE: what depends on the lane is computed again for every tile; kept over all of them it took 200
    // registers more than there are)
    int tid = threadIdx.x;
    if constexpr (TREE)
        asm volatile("" : "+v"(tid));
    const int lane = tid & 63, col = lane & 31, e = lane >> 5;
    const int wave = uniform(tid >> 6);
    AttnSeq s;
    if constexpr (TREE) {
        s = attn_seq(a, f.seq);
        s = AttnSeq{uniform(s.q0), uniform(s.nq), uniform(s.kv), false};
    } else {
        s = attn_seq_uniform(a, own, f.seq);
    }
    const int units = TREE ? uniform(attn_tile_units(a, s)) : 1;
    const int tile = TREE ? uniform(f.at / units) : f.at;
    if (TREE && tile * ROWS >= s.nq * a.group) {
        f.before.tiles += tile;
        f.seq++;
        f.at = 0;
        continue;
    }
    const int row0 = tile * ROWS;
    int lo0, hi0, lo1, hi1;  // tokens of the tile's first and last row
    const int last = (row0 + ROWS - 1) / a.group;
    attn_span<TREE>(a, s, row0 / a.group, last < s.nq ? last : s.nq - 1, &lo0, &hi0, &lo1, &hi1);
    const int tile_no = TREE ? f.before.tiles + tile : unit;
    // ---- this split's blocks [b0, b1) of the tile's
    int b0 = lo0 / kTileTok, b1 = hi1 > lo0 ? (hi1 + kTileTok - 1) / kTileTok : b0;
    const int first = TREE ? f.at - tile * units : 0;  // the share's part of the tile's work
    const int part = TREE && units - first > unit_end - unit ? unit_end - unit : units - first;
    if constexpr (TREE) {
        attn_tree_check(a, s);
        const int from = first - kTileStart, to = from + part;
        b1 = b0 + (to > 0 ? to : 0);
        b0 += from > 0 ? from : 0;
        // (`parts` is the last share here: no division where registers are scarce)
        if (h == 0 && tid == 0) {
            int* const t = &a.tiles[1 + tile_no].first;
            if (first == 0) {
                t[0] = slot;
                t[2] = s.q0;
                t[3] = s.nq;
                t[4] = row0;
            }
            if (first + part == units)
                t[1] = slot;
        }
        lds_barrier();  // nobody reads the last tile's blocks any more
    } else if (gridDim.y > 1) {
        const int n = b1 - b0, per = (n + (int)gridDim.y - 1) / (int)gridDim.y;
        const int base = b0;
        b0 = base + split * per < b1 ? base + split * per : b1;
        b1 = b0 + per < b1 ? b0 + per : b1;
    }
    // ---- queries: lane's row (column of the products) and its limits
    const int r = row0 + 32 * wave + col;
    const int qi = r / a.group, hh = r - qi * a.group;
    const bool in = qi < s.nq;
    int start = 0, end = 0;
    if constexpr (TREE) {
        if (in) {
            start = attn_tree_start(a, s, qi);
            end = s.kv;
        }
    } else if (in) {
        attn_limits(a, s, qi, &start, &end);
    }
    // (D = 256: converted behind the first requests of K and V, 2218 against 2257 us for 2048 rows on 30720
    // tokens; at D = 128 registers then spill and 4096 rows take 167 instead of 150)
    u32x4 qw[D / 16];
    {
        const uint16_t* src = a.q + (int64_t)(s.q0 + (in ? qi : 0)) * a.ld_q + (int64_t)(h * a.group + hh) * D + 8 * e;
#pragma unroll
        for (int c = 0; c < D / 16; c++) {
            qw[c] = (u32x4){0, 0, 0, 0};
            if (in)
                qw[c] = *(const u32x4*)(src + 16 * c);
        }
    }
    half8_t q[D / 16];
    float c1;
    // m, c1 and the scores are in units of 2^k.  It is read where the maximum grows only, and kept in shared
    // memory where a register more spills (D = 128, eight waves: 4096 rows 155 us, 152 so)
    __shared__ int row_k[D < 256 ? ROWS : 1];
    int one_k;
    int* const k2 = D < 256 ? row_k + 32 * wave + col : &one_k;
    *k2 = 0;
    auto convert = [&]() ATTN_INLINE {
        uint32_t am = 0;
#pragma unroll
        for (int c = 0; c < D / 16; c++)
            am = umax_u32(am, absmax_bits8(qw[c]));
        am = umax_u32(am, (uint32_t)__shfl_xor((int)am, 32, 64));
        const int ex = am ? __builtin_amdgcn_frexp_expf(__uint_as_float(am << 16)) - 1 : 0;
        c1 = attn_factor(a.scale_log2, *a.k_global, ex, k2);
#pragma unroll
        for (int c = 0; c < D / 16; c++)
#pragma unroll
            for (int j = 0; j < 4; j++) {
                q[c][2 * j] = (_Float16)__builtin_ldexpf(bf16_lo(qw[c][j]), -ex);
                q[c][2 * j + 1] = (_Float16)__builtin_ldexpf(bf16_hi(qw[c][j]), -ex);
            }
    };
    if constexpr (D < 256)
        convert();
    // ---- staging: the thread's elements of K (token kt, elements kd .. + kK)
    // and of V (tokens 4 vt .. + 4, elements vd .. + kV)
    const int32_t* table = a.table + f.seq * a.ld_table;
    const int first_page = attn_page(a, lo0), last_page = attn_page(a, hi1 > 0 ? hi1 - 1 : 0);
    const uint32_t crow = a.kv_heads * (D / 2), srow = a.kv_heads * (D / 16);
    const int job = tid & 255;
    // (D = 256: K elements kd .. + 32 and 128 + kd .. + 32, whose places in shared memory spread over the banks)
    const int kt = job / (D / Raw::kK), kd = job % (D / Raw::kK) * (D < 256 ? Raw::kK : 32);
    const int vt = job / (D / Raw::kV), vd = job % (D / Raw::kV) * Raw::kV;
    const uint8_t* const k_codes = a.k_packed + h * (D / 2) + kd / 2;
    const uint8_t* const k_scales = a.k_scales + h * (D / 16) + kd / 16;
    const uint8_t* const v_codes = a.v_packed + h * (D / 2) + vd / 2;
    const uint8_t* const v_scales = a.v_scales + h * (D / 16) + vd / 16;
    Raw raw;
    int kp = 0, vp = 0;  // the pages of the next block's tokens
    bool bad = false;
    // the entry of the page of token t (past the end: the last page, masked)
    auto entry = [&](int t) ATTN_INLINE {
        const int i = attn_page(a, t);
        return table[i < last_page ? i : last_page];
    };
    auto pages_k = [&](int blk) ATTN_INLINE { kp = entry(blk * kTileTok + kt); };
    auto pages_v = [&](int blk) ATTN_INLINE { vp = entry(blk * kTileTok + 4 * vt); };
    // the first row of token t in the cache; a page that is none of the cache's: page 0
    auto row_of = [&](int page, int t, bool* ok) ATTN_INLINE {
        const int i = attn_page(a, t);
        *ok = page >= 0 && page < a.num_pages;
        // (a page with no token that a row sees may hold anything)
        bad |= !*ok && t < hi1 && i >= first_page;
        return (uint32_t)(*ok ? page : 0) * (uint32_t)a.page + (uint32_t)(t - i * a.page);
    };
    auto load_k = [&](int blk) ATTN_INLINE {
        const uint64_t k = row_of(kp, blk * kTileTok + kt, &raw.ok);
        if constexpr (D < 256) {
            load_bytes<Raw::kK / 2>(k_codes + k * crow, raw.kc);
            load_bytes<(Raw::kK > 16 ? Raw::kK / 16 : 1)>(k_scales + k * srow, &raw.ks);
        } else {
            uint32_t hi;
            load_bytes<16>(k_codes + k * crow, raw.kc);
            load_bytes<16>(k_codes + k * crow + 64, raw.kc + 4);
            load_bytes<2>(k_scales + k * srow, &raw.ks);
            load_bytes<2>(k_scales + k * srow + 8, &hi);
            raw.ks |= hi << 16;
        }
    };
    auto load_v = [&](int blk) ATTN_INLINE {
        bool ok;
        const uint64_t v = row_of(vp, blk * kTileTok + 4 * vt, &ok);
#pragma unroll
        for (int i = 0; i < 4; i++) {
            load_bytes<Raw::kV / 2>(v_codes + (v + i) * crow, raw.vc[i]);
            raw.vs[i] = v_scales[(v + i) * srow];
        }
    };
    // V's codes with two tokens side by side: byte i of even / odd: elements 2i / 2i + 1
    uint32_t even[2][Raw::kV > 8 ? Raw::kV / 8 : 1], odd[2][Raw::kV > 8 ? Raw::kV / 8 : 1];
    half2_t vsc[2];
    auto interleave = [&]() ATTN_INLINE {
#pragma unroll
        for (int i = 0; i < 2; i++) {
#pragma unroll
            for (int w = 0; w < (Raw::kV > 8 ? Raw::kV / 8 : 1); w++) {
                const uint32_t x = raw.vc[2 * i][w], y = raw.vc[2 * i + 1][w];
                even[i][w] = (x & 0x0F0F0F0Fu) | ((y << 4) & 0xF0F0F0F0u);
                odd[i][w] = ((x >> 4) & 0x0F0F0F0Fu) | (y & 0xF0F0F0F0u);
            }
            vsc[i] = scale_pair(raw.vs[2 * i], raw.vs[2 * i + 1]);
        }
    };
    // tokens 4 vt .. + 4 of the block: 8 bytes at place 8 (vt % 2) + 4 (vt / 2 % 2) of their 16
    const int vchunk = 2 * (vt >> 2) + (vt & 1), vpart = (vt >> 1) & 1;
    // piece U of decoding the block in raw into buffer B
    auto decode_k = [&](auto buf, auto unit) ATTN_INLINE {
        constexpr int B = decltype(buf)::value, U = decltype(unit)::value;
        const uint32_t b = raw.ks >> (8 * (U >> 1));
        (B ? lk1 : lk0)[tile_chunk<KC>(kt, kd / 8 + (D < 256 ? U : U % 4 + U / 4 * 16))] =
            __builtin_bit_cast(u32x4, decode_row8(raw.kc[U], scale_pair(b, b)));
        if (U == 0 && kd == 0 && (kt & 15) == 0)
            lok[B][kt >> 4] = raw.ok;
    };
    auto decode_v = [&](auto buf, auto unit) ATTN_INLINE {
        constexpr int B = decltype(buf)::value, U = decltype(unit)::value, W = U / 4, I = U % 4;
        u32x2* dst = (u32x2*)(B ? lv1 : lv0) + vpart;
        dst[2 * tile_chunk<8>(vd + 2 * U, vchunk)] =
            (u32x2){decode_pair<I>(even[0][W], vsc[0]), decode_pair<I>(even[1][W], vsc[1])};
        dst[2 * tile_chunk<8>(vd + 2 * U + 1, vchunk)] =
            (u32x2){decode_pair<I>(odd[0][W], vsc[0]), decode_pair<I>(odd[1][W], vsc[1])};
    };

    float16_t o[D / 32];
#pragma unroll
    for (int d = 0; d < D / 32; d++)
#pragma unroll
        for (int i = 0; i < 16; i++)
            o[d][i] = 0.0f;
    float m = kAttnLow, l = 0.0f;
    float16_t sc[2];
    u32x4 ok;  // which 16 tokens of the block lie in a page of the cache
    // S^T of block blk, and between its products the decoding of the next one
    // (what of it is this wave's) and the requests for the one after.  Past the
    // end these go to the last page again and are not used.
    auto multiply = [&](int blk, auto buf, auto has_k, auto has_v) ATTN_INLINE {
        constexpr int B = decltype(buf)::value, kAhead = 2, N = D / 16;
        // the group that feeds the matrix unit goes first (measured 4% at D = 128; the other way round 1%)
        if constexpr (kTurns)
            __builtin_amdgcn_s_setprio(1);
        const std::integral_constant<int, 1 - B> other{};
        ok = *(const u32x4*)lok[B];
        if constexpr (has_v)
            interleave();
#pragma unroll
        for (int p = 0; p < 2; p++)
#pragma unroll
            for (int i = 0; i < 16; i++)
                sc[p][i] = 0.0f;
        // (operands are read two product steps ahead)
        half8_t f[N][2];
        auto read = [&](auto ci) ATTN_INLINE {
            constexpr int c = decltype(ci)::value;
#pragma unroll
            for (int p = 0; p < 2; p++)
                f[c][p] = __builtin_bit_cast(half8_t, (B ? lk1 : lk0)[tile_chunk<KC>(32 * p + col, 2 * c + e)]);
        };
        for_range<0, kAhead>(read);
        for_range<0, N>([&](auto ci) ATTN_INLINE {
            constexpr int c = decltype(ci)::value, per = N / Raw::kUnits;  // (2)
            if constexpr (c + kAhead < N)
                read(std::integral_constant<int, c + kAhead>{});
#pragma unroll
            for (int p = 0; p < 2; p++)
                sc[p] = mfma32(f[c][p], q[c], sc[p]);
            if constexpr (has_k && c % per == 0)
                decode_k(other, std::integral_constant<int, c / per>{});
            if constexpr (has_v && c % per == per - 1)
                decode_v(other, std::integral_constant<int, c / per>{});
        });
        if constexpr (has_k) {
            load_k(blk + 2);
            pages_k(blk + 3);
        }
        if constexpr (has_v) {
            load_v(blk + 2);
            pages_v(blk + 3);
        }
    };
    // P^T of block blk, and O^T += V^T P^T
    auto accumulate = [&](int blk, auto buf) ATTN_INLINE {
        constexpr int B = decltype(buf)::value, N = D / 32, kAhead = 4;
        if constexpr (kTurns)
            __builtin_amdgcn_s_setprio(0);
        const int t0 = blk * kTileTok;
        if (!(t0 >= lo1 && t0 + kTileTok <= hi0 && (ok.x & ok.y & ok.z & ok.w) != 0)) {
#pragma unroll
            for (int p = 0; p < 2; p++) {
                uint32_t bits = 0;
                if constexpr (TREE)
                    bits = attn_tree_bits(a, s.q0 + (in ? qi : 0), t0 + 32 * p - (s.kv - s.nq)) >> (4 * e);
#pragma unroll
                for (int i = 0; i < 16; i++) {
                    const int tok = t0 + 32 * p + 8 * (i >> 2) + 4 * e + (i & 3);
                    const bool seen = tok >= start && tok < end && ok[2 * p + (i >> 3)] != 0 &&
                                      (!TREE || (bits >> (8 * (i >> 2) + (i & 3)) & 1));
                    sc[p][i] = seen ? sc[p][i] : -__builtin_inff();
                }
            }
        }
        float top = sc[0][0];
#pragma unroll
        for (int i = 1; i < 32; i++)
            top = __builtin_fmaxf(top, sc[i >> 4][i & 15]);
        top *= c1;
        if (__any(top > m + kAttnLazy)) {
            top = __builtin_fmaxf(top, __shfl_xor(top, 32, 64));
            const float g = attn_grow(__builtin_fmaxf(m, top), &m, &c1, k2);
            l *= g;
            if constexpr (D < 256) {
#pragma unroll
                for (int d = 0; d < D / 32; d++)
                    o[d] *= g;
            } else {
                scale_acc(o, g);
            }
        }
        const float lift = kAttnLift - m;
        half8_t pt[4];
        auto weigh = [&](int k) ATTN_INLINE {
            float x[8];
#pragma unroll
            for (int i = 0; i < 8; i++)
                x[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[k >> 1][8 * (k & 1) + i], c1, lift));
            l += ((x[0] + x[1]) + (x[2] + x[3])) + ((x[4] + x[5]) + (x[6] + x[7]));
#pragma unroll
            for (int i = 0; i < 8; i++)
                pt[k][i] = (_Float16)x[i];
        };
        // each 16 tokens are weighed between the products of the 16 before;
        // operands are read four products ahead
        half8_t f[4 * N];
        auto read = [&](auto xi) ATTN_INLINE {
            constexpr int x = decltype(xi)::value;
            f[x] = __builtin_bit_cast(half8_t, (B ? lv1 : lv0)[tile_chunk<8>(32 * (x % N) + col, 2 * (x / N) + e)]);
        };
        for_range<0, kAhead>(read);
        weigh(0);
        for_range<0, 4 * N>([&](auto xi) ATTN_INLINE {
            constexpr int x = decltype(xi)::value, k = x / N, d = x % N;
            if constexpr (d == 0 && k < 3)
                weigh(k + 1);
            if constexpr (x + kAhead < 4 * N)
                read(std::integral_constant<int, x + kAhead>{});
            o[d] = mfma32(f[x], pt[k], o[d]);
        });
    };
    constexpr std::integral_constant<int, 0> zero{};
    constexpr std::integral_constant<int, 1> one{};
    auto prepare = [&](auto has_k, auto has_v) ATTN_INLINE {
        if constexpr (has_k) {
            pages_k(b0);
            load_k(b0);
            pages_k(b0 + 1);
        }
        if constexpr (has_v) {
            pages_v(b0);
            load_v(b0);
            pages_v(b0 + 1);
        }
        if constexpr (D == 256)
            convert();
        if constexpr (has_k) {
            for_range<0, Raw::kUnits>([&](auto u) ATTN_INLINE { decode_k(zero, u); });
            load_k(b0 + 1);
            pages_k(b0 + 2);
        }
        if constexpr (has_v) {
            interleave();
            for_range<0, Raw::kUnits>([&](auto u) ATTN_INLINE { decode_v(zero, u); });
            load_v(b0 + 1);
            pages_v(b0 + 2);
        }
    };
    constexpr std::true_type yes{};
    constexpr std::false_type no{};
    // TREE: waves without a row (a tree's tiles are often partly filled) only decode
    const bool idle = TREE && row0 + 32 * wave >= s.nq * a.group;
    if (b0 < b1) {
        if (TREE && idle && (!kTurns || wave >= NW / 2)) {
            auto turn = [&](int blk, auto buf) ATTN_INLINE {
                constexpr std::integral_constant<int, 1 - decltype(buf)::value> other{};
                lds_barrier();
                interleave();
                for_range<0, Raw::kUnits>([&](auto u) ATTN_INLINE {
                    if constexpr (!kTurns)
                        decode_k(other, u);
                    decode_v(other, u);
                });
                if constexpr (!kTurns) {
                    load_k(blk + 2);
                    pages_k(blk + 3);
                }
                load_v(blk + 2);
                pages_v(blk + 3);
                if constexpr (kTurns)
                    lds_barrier();
            };
            if constexpr (kTurns) {
                prepare(no, yes);
                lds_barrier();
            } else {
                prepare(yes, yes);
            }
            for (int blk = b0; blk < b1; blk += 2) {
                turn(blk, zero);
                if (blk + 1 < b1)
                    turn(blk + 1, one);
            }
        } else if constexpr (!kTurns) {
            prepare(yes, yes);
            auto turn = [&](int blk, auto buf) ATTN_INLINE {
                lds_barrier();  // the block is written, and nobody reads the other buffer any more
                multiply(blk, buf, yes, yes);
                accumulate(blk, buf);
            };
            for (int blk = b0; blk < b1; blk += 2) {
                turn(blk, zero);
                if (blk + 1 < b1)
                    turn(blk + 1, one);
            }
        } else if (wave < NW / 2) {
            prepare(yes, no);
            lds_barrier();
            auto turn = [&](int blk, auto buf) ATTN_INLINE {
                multiply(blk, buf, yes, no);
                lds_barrier();
                accumulate(blk, buf);
                lds_barrier();
            };
            for (int blk = b0; blk < b1; blk += 2) {
                turn(blk, zero);
                if (blk + 1 < b1)
                    turn(blk + 1, one);
            }
        } else {
            prepare(no, yes);
            lds_barrier();
            auto turn = [&](int blk, auto buf) ATTN_INLINE {
                lds_barrier();  // half a block behind
                multiply(blk, buf, no, yes);
                lds_barrier();
                accumulate(blk, buf);
            };
            for (int blk = b0; blk < b1; blk += 2) {
                turn(blk, zero);
                if (blk + 1 < b1)
                    turn(blk + 1, one);
            }
        }
    }
    if (bad)
        raise_error(NVFP4_ERR_RANGE);
    m = attn_whole(m, *k2);
    l += __shfl_xor(l, 32, 64);
    const int head = h * a.group + hh;
    const int64_t token = s.q0 + qi;
    if (TREE ? part < units : gridDim.y > 1) {
        // (m, l, o) of this split: [tile][kv head][split][row][D + 4]; TREE: [share][kv head][slot], slot 1 for the
        // tile's first share
        if (!TREE && split == 0 && h == 0 && tid == 0)
            a.tiles[1 + tile_no] = AttnTile{0, (int)gridDim.y, s.q0, s.nq, row0};
        if (in) {
            const int64_t at = TREE ? ((int64_t)slot * a.kv_heads + h) * 2 + (first == 0)
                                    : ((int64_t)tile_no * a.kv_heads + h) * gridDim.y + split;
            float* dst = a.partial + (at * ROWS + 32 * wave + col) * (D + 4);
            if (e == 0) {
                dst[D] = m;
                dst[D + 1] = l;
            }
#pragma unroll
            for (int d = 0; d < D / 32; d++)
#pragma unroll
                for (int i = 0; i < 4; i++)
                    *(float4_t*)(dst + 32 * d + 8 * i + 4 * e) =
                        (float4_t){o[d][4 * i], o[d][4 * i + 1], o[d][4 * i + 2], o[d][4 * i + 3]};
        }
    } else if (in) {
        const float g = l != 0.0f ? *a.v_global / l : 0.0f;
        uint16_t* dst = a.out + token * a.ld_out + (int64_t)head * D + 4 * e;
#pragma unroll
        for (int d = 0; d < D / 32; d++)
#pragma unroll
            for (int i = 0; i < 4; i++)
                *(u32x2*)(dst + 32 * d + 8 * i) = (u32x2){pack_bf16x2(o[d][4 * i] * g, o[d][4 * i + 1] * g),
                                                          pack_bf16x2(o[d][4 * i + 2] * g, o[d][4 * i + 3] * g)};
        if (a.lse && e == 0)
            a.lse[token * (a.kv_heads * a.group) + head] =
                l != 0.0f ? (m - kAttnLift + __builtin_amdgcn_logf(l)) * 0.69314718056f : -__builtin_inff();
    }
    unit += part;
    f.at += part;
    } while (TREE && unit < unit_end);
}

// Joins the splits (TREE: the shares) of a tile of ROWS rows (blockIdx.x) and KV
// head (blockIdx.y): a wave a row at a time.
template <int D, int ROWS, bool TREE>
__global__ void __launch_bounds__(256)
attn_tile_combine_kernel(AttnArgs a)
{
    const int lane = threadIdx.x & 63, wave = uniform((int)(threadIdx.x >> 6));
    const int tiles = a.tiles[0].parts;
    const AttnTile tile = a.tiles[1 + blockIdx.x];
    const float vg = *a.v_global;
    const int first = uniform(tile.first), parts = uniform(tile.parts) - (TREE ? first - 1 : 0);
    if ((int)blockIdx.x >= tiles || (TREE && parts == 1))
        return;
    const int h = blockIdx.y;
    constexpr int V = D / 64;  // elements per lane
    for (int row = blockIdx.z * 4 + wave; row < ROWS; row += gridDim.z * 4) {
        const int r = tile.row0 + row, i = r / a.group, head = h * a.group + r - i * a.group;
        if (i >= tile.nq)
            break;
        // (TREE: slot 1 of the tile's first share, slot 0 of the others)
        const int64_t at = TREE ? ((int64_t)first * a.kv_heads + h) * 2 : ((int64_t)blockIdx.x * a.kv_heads + h) * parts;
        const float* src = a.partial + (at * ROWS + row) * (D + 4);
        const int64_t step = (int64_t)(TREE ? 2 * a.kv_heads : 1) * ROWS * (D + 4);
        float m = kAttnLow, l = 0.0f, o[V];
#pragma unroll
        for (int j = 0; j < V; j++)
            o[j] = 0.0f;
#pragma unroll 4
        for (int p = 0; p < parts; p++) {
            const float* x = src + p * step + (TREE && p == 0 ? ROWS * (D + 4) : 0);
            const float om = x[D], ol = x[D + 1], now = __builtin_fmaxf(m, om);
            const float f = __builtin_amdgcn_exp2f(m - now), g = __builtin_amdgcn_exp2f(om - now);
            l = l * f + ol * g;
#pragma unroll
            for (int j = 0; j < V; j++)
                o[j] = o[j] * f + x[lane * V + j] * g;
            m = now;
        }
        const int64_t token = tile.q0 + i;
        const float scale = l != 0.0f ? vg / l : 0.0f;
        uint16_t* dst = a.out + token * a.ld_out + (int64_t)head * D + lane * V;
        if constexpr (V == 1)
            *dst = f32_to_bf16(o[0] * scale);
        else
#pragma unroll
            for (int j = 0; j < V; j += 2)
                *(uint32_t*)(dst + j) = pack_bf16x2(o[j] * scale, o[j + 1] * scale);
        if (a.lse && lane == 0)
            a.lse[token * (a.kv_heads * a.group) + head] =
                l != 0.0f ? (m - kAttnLift + __builtin_amdgcn_logf(l)) * 0.69314718056f : -__builtin_inff();
    }
}

}  // namespace nvfp4
