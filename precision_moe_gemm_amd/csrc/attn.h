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
// of that below.  p is rounded to f16 for the second product (half a step is
// 2^-12 of it), l sums the unrounded p.
//
// Both products are written transposed, S^T = K Q^T and O^T = V^T P^T, with
// v_mfma_f32_16x16x32_f16 (A: row l % 16, B: column l % 16, both elements
// 8 (l / 16) .. + 8 of the contraction; output: column l % 16, rows
// 4 (l / 16) .. + 4 for lane l).  A lane then holds the scores of one query
// row for 4 + 4 tokens of two 16-token tiles, which is its share of the
// second product's B operand as it stands: p never leaves its registers.
// The order of the contraction elements is free as long as both operands
// agree on it: the first product gives lane group g = l / 16 the elements
// [g D / 4, + D / 4), one contiguous piece of a K row; the second gives it
// tokens 4g .. 4g + 3 of both tiles, and output row m of its MFMA dd is
// element m D / 16 + dd, so a lane reads a contiguous piece of a V row too.
// Neither operand passes through shared memory.
#pragma once
#include "common.h"

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
    int kv_heads, group;     // group: query heads per KV head
    float scale_log2;        // scale * log2(e)
    int causal, window;
    uint16_t* out;           // [n, heads, D], token stride ld_out
    int64_t ld_out;
    float* lse;              // [n, heads] or null
    int head_lanes;          // KV heads a workgroup holds side by side (1, 2 or 4)
    int workers;             // shares that the tokens are cut into (at most)
    float* partial;          // what shares leave of sequences that they hold a part of
};

constexpr int kAttnThreads = 256;
constexpr int kAttnStep = 32;            // tokens of one step
constexpr float kAttnLow = -1e30f;       // running maximum of a row that has seen nothing
constexpr float kAttnLazy = 8.0f;        // growth of the maximum (log 2) that is let pass
constexpr float kAttnLift = 7.0f;        // p is held times 2^7, at most 2^15 (f16 holds 65504)

// One sequence as the kernels see it: bad lengths are cut to what exists and
// raise NVFP4_ERR_RANGE.
struct AttnSeq {
    int q0, nq, kv;
};

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
    } else {
        s.q0 = b;
        s.nq = 1;
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
        if (a.window > 0)
            b = pos - a.window + 1;
    }
    *end = e < 0 ? 0 : e;
    *start = b < 0 ? 0 : b;
}

// Work of a row kernel is counted in units: sequence b has tiles(b) tiles of
// rows and units(b) steps of tokens for each of them (at least one, so that
// rows that see nothing are written too).  The sequence that holds unit x (or
// tile x, by_tile), the number of that unit (tile) in the sequence, the units
// before the sequence and the units of all sequences.  All threads of the
// workgroup call it; every thread sums a contiguous run of sequences.
struct AttnCount {
    int64_t tiles, units;
};
struct AttnFound {
    int64_t local, before, total, all_tiles;
    int seq;
};

constexpr int kAttnFoundLds = 2 * 16 + 3;

template <class Count>
NVFP4_DEV AttnFound attn_locate(int seqs, int64_t x, bool by_tile, int64_t* lds, Count count)
{
    const int nt = blockDim.x, waves = nt >> 6, wave = threadIdx.x >> 6;
    const int per = (seqs + nt - 1) / nt;
    const int b0 = threadIdx.x * per, b1 = b0 + per < seqs ? b0 + per : seqs;
    AttnCount mine = {0, 0};
    for (int b = b0; b < b1; b++) {
        const AttnCount c = count(b);
        mine.tiles += c.tiles;
        mine.units += c.tiles * c.units;
    }
    AttnCount up = mine;  // inclusive sums over the wave's lanes
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const int64_t a = __shfl_up(up.tiles, off, 64), u = __shfl_up(up.units, off, 64);
        const bool in = (int)(threadIdx.x & 63) >= off;
        up.tiles += in ? a : 0;
        up.units += in ? u : 0;
    }
    if ((threadIdx.x & 63) == 63) {
        lds[2 * wave] = up.tiles;
        lds[2 * wave + 1] = up.units;
    }
    __syncthreads();
    AttnCount before = {0, 0}, total = {0, 0};
    for (int w = 0; w < waves; w++) {
        before.tiles += w < wave ? lds[2 * w] : 0;
        before.units += w < wave ? lds[2 * w + 1] : 0;
        total.tiles += lds[2 * w];
        total.units += lds[2 * w + 1];
    }
    before.tiles += up.tiles - mine.tiles;
    before.units += up.units - mine.units;
    int64_t rest = x - (by_tile ? before.tiles : before.units);
    if (rest >= 0 && rest < (by_tile ? mine.tiles : mine.units)) {
        int b = b0;
        for (; b < b1; b++) {
            const AttnCount c = count(b);
            const int64_t size = by_tile ? c.tiles : c.tiles * c.units;
            if (rest < size)
                break;
            rest -= size;
            before.units += c.tiles * c.units;
        }
        lds[32] = rest;
        lds[33] = before.units;
        lds[34] = b;
    }
    __syncthreads();
    AttnFound f;
    f.local = lds[32];
    f.before = lds[33];
    f.total = total.units;
    f.all_tiles = total.tiles;
    f.seq = (int)lds[34];
    return f;
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

// A wave's lanes: query column n, lane group g.
NVFP4_DEV int lane_n() { return threadIdx.x & 15; }
NVFP4_DEV int lane_g() { return (threadIdx.x >> 4) & 3; }

// What a lane holds of one step's 32 tokens of K and V, as read.
template <int D>
struct AttnRaw {
    uint32_t kc[2][D / 32];                  // K codes: token n of each 16, elements [g D / 4, + D / 4)
    uint32_t ks[2];                          // their scale bytes (D / 64)
    uint32_t vc[8][D > 128 ? D / 128 : 1];   // V codes: tokens 4g + j of each 16, elements [n D / 16, + D / 16)
    uint32_t vs[8];                          // their scale byte
};

// The pages of a wave's token range: lane l holds the entry of page
// first + l of the sequence (-1: not a page of the cache).
struct AttnPages {
    const int32_t* row;
    int first, last;
    int needed;  // first page with a token that some row sees (a page before it may be gone)
    int entry;
    NVFP4_DEV void fill(const AttnArgs& a, int idx)
    {
        first = idx;
        int i = idx + (int)(threadIdx.x & 63);
        i = i < last ? i : last;
        const int e = row[i];
        const bool ok = e >= 0 && e < a.num_pages;
        if (!ok && i >= needed)
            raise_error(NVFP4_ERR_RANGE);
        entry = ok ? e : -1;
    }
    NVFP4_DEV int get(const AttnArgs& a, int idx)
    {
        if (idx - first >= 64)
            fill(a, idx);
        return __builtin_amdgcn_readlane(entry, idx - first);
    }
};

// A wave's walk over the tokens of one KV head for 16 NT query rows.
template <int D, int NT>
struct AttnWave {
    half8_t q[NT][D / 32];
    float4_t o[NT][D / 16];
    float m[NT], l[NT], c1[NT];
    int start[NT], end[NT];

    // rows row0 .. row0 + 16 NT of sequence s: row r is query token r / group, head r % group of KV head h
    NVFP4_DEV void open(const AttnArgs& a, const AttnSeq& s, int h, int row0)
    {
        const float kg = *a.k_global;
#pragma unroll
        for (int t = 0; t < NT; t++) {
            const int r = row0 + 16 * t + lane_n();
            const int i = r / a.group, hh = r - i * a.group;
            const bool in = i < s.nq;
            start[t] = end[t] = 0;
            u32x4 w[D / 32];
            uint32_t am = 0;
            if (in)
                attn_limits(a, s, i, &start[t], &end[t]);
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
            // (kept above zero: -inf times it stays -inf)
            c1[t] = __builtin_fmaxf(__builtin_ldexpf(a.scale_log2 * kg, e), 1e-37f);
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

    // the 16 tokens of half `half` of a step: they lie in one page.  The first
    // token's row is the same for all lanes, so it goes into the scalar base
    // of the loads and the lane's part is 32 bits.
    NVFP4_DEV void load_half(const AttnArgs& a, AttnRaw<D>& raw, int half, int h, int64_t tok) const
    {
        const int64_t row = tok * a.kv_heads + h;  // the first token's cache row
        const uint32_t stride = a.kv_heads;
        const uint8_t* kc = a.k_packed + row * (D / 2) + (uint32_t)(lane_n() * stride * (D / 2) + lane_g() * (D / 8));
        const uint8_t* ks = a.k_scales + row * (D / 16) + (uint32_t)(lane_n() * stride * (D / 16) + lane_g() * (D / 64));
        if constexpr (D == 64) {
            const u32x2 w = *(const u32x2*)kc;
            raw.kc[half][0] = w.x;
            raw.kc[half][1] = w.y;
            raw.ks[half] = *ks;
        } else {
#pragma unroll
            for (int c = 0; c < D / 128; c++) {
                const u32x4 w = ((const u32x4*)kc)[c];
#pragma unroll
                for (int i = 0; i < 4; i++)
                    raw.kc[half][4 * c + i] = w[i];
            }
            if constexpr (D == 128)
                raw.ks[half] = *(const uint16_t*)ks;
            else
                raw.ks[half] = *(const uint32_t*)ks;
        }
        const uint32_t vo = 4 * lane_g() * stride * (D / 2) + lane_n() * (D / 32);
        const uint32_t so = 4 * lane_g() * stride * (D / 16) + lane_n() * D / 256;
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const uint8_t* p = a.v_packed + (row + j * (int64_t)stride) * (D / 2) + vo;
            if constexpr (D == 64) {
                raw.vc[4 * half + j][0] = *(const uint16_t*)p;
            } else if constexpr (D == 128) {
                raw.vc[4 * half + j][0] = *(const uint32_t*)p;
            } else {
                const u32x2 w = *(const u32x2*)p;
                raw.vc[4 * half + j][0] = w.x;
                raw.vc[4 * half + j][1] = w.y;
            }
            raw.vs[4 * half + j] = a.v_scales[(row + j * (int64_t)stride) * (D / 16) + so];
        }
    }

    // one step: tokens t0 .. t0 + 32; ok: which halves lie in a page of the cache
    NVFP4_DEV void step(const AttnRaw<D>& raw, int t0, bool inside, const bool (&ok)[2])
    {
        float4_t s[NT][2];
#pragma unroll
        for (int half = 0; half < 2; half++) {
#pragma unroll
            for (int t = 0; t < NT; t++)
                s[t][half] = (float4_t){0, 0, 0, 0};
#pragma unroll
            for (int c = 0; c < D / 32; c++) {
                const uint32_t b = raw.ks[half] >> (8 * (c >> 1));
                const half8_t k = decode_row8(raw.kc[half][c], scale_pair(b, b));
#pragma unroll
                for (int t = 0; t < NT; t++)
                    s[t][half] = mfma16(k, q[t][c], s[t][half]);
            }
        }
        half8_t p[NT];
#pragma unroll
        for (int t = 0; t < NT; t++) {
            if (!inside) {
#pragma unroll
                for (int half = 0; half < 2; half++)
#pragma unroll
                    for (int i = 0; i < 4; i++) {
                        const int tok = t0 + 16 * half + 4 * lane_g() + i;
                        const bool seen = ok[half] && tok >= start[t] && tok < end[t];
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
                const float now = __builtin_fmaxf(m[t], top);
                const float f = __builtin_amdgcn_exp2f(m[t] - now);
                m[t] = now;
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
        half2_t sc[4];
#pragma unroll
        for (int j = 0; j < 4; j++)
            sc[j] = scale_pair(raw.vs[2 * j], raw.vs[2 * j + 1]);
        // token pairs side by side: byte i of even / odd holds elements 2i / 2i + 1 of both tokens
#pragma unroll
        for (int w = 0; w < (D > 128 ? D / 128 : 1); w++) {
            uint32_t even[4], odd[4];
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const uint32_t x = raw.vc[2 * j][w], y = raw.vc[2 * j + 1][w];
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

    // the step at token t0 + 32 k of a walk (the last one again past the end)
    NVFP4_DEV void load(const AttnArgs& a, AttnPages& pages, AttnRaw<D>& raw, bool (&ok)[2], int h, int t) const
    {
#pragma unroll
        for (int half = 0; half < 2; half++) {
            int i = (t + 16 * half) / a.page;
            const int off = t + 16 * half - i * a.page;
            i = i < pages.last ? i : pages.last;  // past the end: any page, masked
            const int page = pages.get(a, i);
            ok[half] = page >= 0;
            load_half(a, raw, half, h, (int64_t)(page < 0 ? 0 : page) * a.page + off);
        }
    }

    // tokens [t0, t1) (t0 a multiple of 32); any: the first token that some
    // row sees; [lo, hi): the tokens that every row sees.  Each step's data is
    // requested while the step before it is computed; the requests are
    // unconditional (past the end the last step's, which is in the cache), so
    // that the compiler can count them and wait for the older step only.
    NVFP4_DEV void walk(const AttnArgs& a, const int32_t* table_row, int h, int t0, int t1, int any, int lo, int hi)
    {
        if (t0 >= t1)
            return;
        AttnPages pages;
        pages.row = table_row;
        pages.last = (t1 - 1) / a.page;
        pages.needed = any / a.page;
        pages.fill(a, t0 / a.page);
        const int end = t0 + (t1 - t0 - 1) / kAttnStep * kAttnStep;  // the last step
        AttnRaw<D> x, y;
        bool okx[2], oky[2];
        load(a, pages, x, okx, h, t0);
        for (int t = t0; t <= end; t += 2 * kAttnStep) {
            const int u = t + kAttnStep, v = u + kAttnStep;
            load(a, pages, y, oky, h, u < end ? u : end);
            step(x, t, okx[0] && okx[1] && t >= lo && u <= hi, okx);
            load(a, pages, x, okx, h, v < end ? v : end);
            if (u <= end)
                step(y, u, oky[0] && oky[1] && u >= lo && v <= hi, oky);
        }
    }

    // the sums of the lane groups
    NVFP4_DEV void close()
    {
#pragma unroll
        for (int t = 0; t < NT; t++) {
            l[t] += __shfl_xor(l[t], 16, 64);
            l[t] += __shfl_xor(l[t], 32, 64);
        }
    }
};

// Joins the waves that walked different tokens for the same head: wave w
// holds head lane w % hl and token lane w / hl.  buf: D / 4 + 2 floats x 64
// lanes x NT per writing wave, two of them at most.  Afterwards token lane 0
// holds the whole.
template <int D, int NT>
NVFP4_DEV void attn_join(AttnWave<D, NT>& w, int hl, int wave, float* buf)
{
    constexpr int kRow = D / 4 + 2;
    const int tl = wave / hl, lane = threadIdx.x & 63;
    for (int s = (kAttnThreads / 64) / hl / 2; s > 0; s >>= 1) {
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
template <int D, int NT>
NVFP4_DEV void attn_finish(const AttnArgs& a, const AttnWave<D, NT>& w, const AttnSeq& s, int h, int row0)
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
        const float f = w.l[t] > 0.0f ? vg / w.l[t] : 0.0f;  // a row that sees nothing: zeros
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
                w.l[t] > 0.0f ? (w.m[t] - kAttnLift + __builtin_amdgcn_logf(w.l[t])) * 0.69314718056f
                              : -__builtin_inff();
    }
}

// Floats that one wave leaves of a part of its tokens: m, l and o of its 64
// lanes, 16 NT query rows.
template <int D, int NT>
constexpr int attn_part() { return (D / 4 + 2) * NT * 64; }

// The shares: the units of all sequences in a row, cut into equal runs, at
// least `least` units each.  Share w holds units [w T / W, (w + 1) T / W).
NVFP4_DEV int64_t attn_shares(const AttnArgs& a, int64_t total, int least)
{
    const int64_t most = (total + least - 1) / least;
    return most < a.workers ? most : a.workers;
}

template <int D, int NT>
NVFP4_DEV AttnCount attn_count(const AttnArgs& a, int b)
{
    const AttnSeq s = attn_seq(a, b);
    int lo0, hi0, lo1, hi1;
    attn_limits(a, s, 0, &lo0, &hi0);
    attn_limits(a, s, s.nq > 0 ? s.nq - 1 : 0, &lo1, &hi1);
    const int t0 = lo0 & ~(kAttnStep - 1);
    AttnCount c;
    c.tiles = ((int64_t)s.nq * a.group + 16 * NT - 1) / (16 * NT);
    c.units = hi1 > t0 ? (hi1 - t0 + kAttnStep - 1) / kAttnStep : 1;
    return c;
}

// Few query rows per sequence (decode, drafts): the time is the K and V
// bytes' way from HBM.  The tokens of all sequences are cut into equal shares,
// one per resident workgroup, so that long and short sequences load the chip
// alike; a share that holds a whole tile of rows writes its output, one that
// holds a part leaves (m, l, o) for attn_combine_kernel, in slot 1 if it holds
// the tile's first unit, else in slot 0 (a share has at most one of each).
// A workgroup holds head_lanes KV heads side by side, which lie next to each
// other in memory, and (waves / head_lanes) runs of the tokens.
template <int D, int NT>
__global__ void __launch_bounds__(kAttnThreads, D * NT <= 64 ? 4 : (D * NT <= 128 ? 3 : (D * NT <= 256 ? 2 : 1)))
attn_rows_kernel(AttnArgs a)
{
    __shared__ int64_t found[kAttnFoundLds];
    __shared__ float buf[2 * attn_part<D, NT>()];
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int hl = a.head_lanes, tls = (kAttnThreads / 64) / hl;
    // workgroups go to the 8 XCDs in turn: the head blocks of one share go to
    // the same one, whose L2 then holds the lines that they share
    const int blocks = a.kv_heads / hl;
    const int hb = blockIdx.x / 8 % blocks, w = blockIdx.x / (8 * blocks) * 8 + blockIdx.x % 8;
    const int h = hb * hl + wave % hl, tl = wave / hl;
    auto count = [&](int b) { return attn_count<D, NT>(a, b); };
    // (the total first: the share's bounds need it)
    AttnFound f = attn_locate(a.seqs, 0, false, found, count);
    const int64_t shares = attn_shares(a, f.total, 4);
    if (w >= shares)
        return;
    int64_t u = w * f.total / shares;
    const int64_t u1 = (w + 1) * f.total / shares;
    __syncthreads();
    f = attn_locate(a.seqs, u, false, found, count);
    int b = __builtin_amdgcn_readfirstlane(f.seq);
    int64_t at = f.local;  // the unit's number in the sequence
    while (u < u1) {
        const AttnSeq s = attn_seq(a, b);
        const AttnCount c = count(b);
        if (at >= c.tiles * c.units) {
            b++;
            at = 0;
            continue;
        }
        const int tile = __builtin_amdgcn_readfirstlane((int)(at / c.units));
        const int first = __builtin_amdgcn_readfirstlane((int)(at - tile * c.units));
        const int units = (int)c.units;
        const int n = __builtin_amdgcn_readfirstlane(units - first < u1 - u ? units - first : (int)(u1 - u));
        const int row0 = tile * 16 * NT;
        int any, none, lo0, hi0, lo1, hi1;  // tokens of the sequence's, the tile's first and last row
        const int last = (row0 + 16 * NT - 1) / a.group;
        attn_limits(a, s, 0, &any, &none);
        attn_limits(a, s, row0 / a.group, &lo0, &hi0);
        attn_limits(a, s, last < s.nq ? last : s.nq - 1, &lo1, &hi1);
        AttnWave<D, NT> x;
        x.open(a, s, h, row0);
        const int t0 = (any & ~(kAttnStep - 1)) + first * kAttnStep;
        const int share = (n + tls - 1) / tls * kAttnStep;
        int from = t0 + tl * share, to = from + share;
        to = to < t0 + n * kAttnStep ? to : t0 + n * kAttnStep;
        to = to < hi1 ? to : hi1;
        from = from > (lo0 & ~(kAttnStep - 1)) ? from : lo0 & ~(kAttnStep - 1);
        x.walk(a, a.table + b * a.ld_table, h, from, to, lo0, lo1, hi0);
        x.close();
        attn_join<D, NT>(x, hl, wave, buf);
        if (tl == 0) {
            if (n == units) {
                attn_finish<D, NT>(a, x, s, h, row0);
            } else {
                const int slot = first == 0;
                float* dst = a.partial + (((int64_t)w * blocks + hb) * 2 + slot) * hl * attn_part<D, NT>() +
                             (wave % hl) * attn_part<D, NT>() + (threadIdx.x & 63);
#pragma unroll
                for (int t = 0; t < NT; t++) {
                    dst[(t * (D / 4 + 2)) * 64] = x.m[t];
                    dst[(t * (D / 4 + 2) + 1) * 64] = x.l[t];
#pragma unroll
                    for (int i = 0; i < D / 4; i++)
                        dst[(t * (D / 4 + 2) + 2 + i) * 64] = x.o[t][i >> 2][i & 3];
                }
            }
        }
        u += n;
        at += n;
    }
}

// Joins what the shares left of one tile of rows (blockIdx.x) for one KV head
// (blockIdx.y), in the order of the tokens: the weights exp2(m - max) of all
// parts first, then the weighted sums of o, each wave a run of the parts.
// blockIdx.z: pieces of 4 output elements per lane.
constexpr int kAttnParts = 512;  // shares of one tile, at most
template <int D, int NT>
__global__ void __launch_bounds__(1024)
attn_combine_kernel(AttnArgs a)
{
    __shared__ int64_t found[kAttnFoundLds];
    __shared__ float weight[kAttnParts][16];
    __shared__ float red[16][2][16];
    __shared__ float4_t sum[16][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
    auto count = [&](int b) { return attn_count<D, NT>(a, b); };
    const AttnFound f = attn_locate(a.seqs, blockIdx.x, true, found, count);
    if ((int64_t)blockIdx.x >= f.all_tiles)
        return;
    const int b = f.seq;
    const int64_t units = count(b).units;
    const int64_t shares = attn_shares(a, f.total, 4);
    const int64_t u0 = f.before + f.local * units;
    const int w0 = (int)(((u0 + 1) * shares - 1) / f.total), w1 = (int)(((u0 + units) * shares - 1) / f.total);
    if (w0 == w1)
        return;  // one share held the whole tile
    const int parts = w1 - w0 + 1;
    const int hl = a.head_lanes, blocks = a.kv_heads / hl;
    const int h = blockIdx.y, hb = h / hl;
    const AttnSeq s = attn_seq(a, b);
    const int row0 = (int)f.local * 16 * NT;
    const float vg = *a.v_global;
    // part p: the share w0 + p, slot 1 of the first, slot 0 of the others
    auto part = [&](int p) {
        return a.partial + (((int64_t)(w0 + p) * blocks + hb) * 2 + (p == 0)) * hl * attn_part<D, NT>() +
               (h - hb * hl) * attn_part<D, NT>();
    };
#pragma unroll 1
    for (int t = 0; t < NT; t++) {
        const int n = lane & 15;
        float m = kAttnLow;
        for (int p = wave * 4 + (lane >> 4); p < parts; p += waves * 4)
            m = __builtin_fmaxf(m, part(p)[t * (D / 4 + 2) * 64 + n]);
        m = __builtin_fmaxf(m, __shfl_xor(m, 16, 64));
        m = __builtin_fmaxf(m, __shfl_xor(m, 32, 64));
        __syncthreads();
        if (lane < 16)
            red[wave][0][n] = m;
        __syncthreads();
        for (int i = 0; i < waves; i++)
            m = __builtin_fmaxf(m, red[i][0][n]);
        float l = 0.0f;
        for (int p = wave * 4 + (lane >> 4); p < parts; p += waves * 4) {
            const float* src = part(p) + t * (D / 4 + 2) * 64 + n;
            const float g = __builtin_amdgcn_exp2f(src[0] - m);
            weight[p][n] = g;
            l += src[64] * g;
        }
        l += __shfl_xor(l, 16, 64);
        l += __shfl_xor(l, 32, 64);
        if (lane < 16)
            red[wave][1][n] = l;
        __syncthreads();
        l = 0.0f;
        for (int i = 0; i < waves; i++)
            l += red[i][1][n];
        const int r = row0 + 16 * t + n;
        const int i = r / a.group, head = h * a.group + r - i * a.group;
        const int64_t token = s.q0 + i;
        const float scale = l > 0.0f ? vg / l : 0.0f;
        if (i < s.nq && a.lse && blockIdx.z == 0 && threadIdx.x < 16)
            a.lse[token * (a.kv_heads * a.group) + head] =
                l > 0.0f ? (m - kAttnLift + __builtin_amdgcn_logf(l)) * 0.69314718056f : -__builtin_inff();
        const int run = (parts + waves - 1) / waves, p1 = (wave + 1) * run < parts ? (wave + 1) * run : parts;
        for (int c = blockIdx.z; c < D / 16; c += gridDim.z) {
            const int k = c / (D / 64), dd = 4 * (c - k * (D / 64));
            float4_t o = (float4_t){0, 0, 0, 0};
#pragma unroll 4
            for (int p = wave * run; p < p1; p++) {
                const float* src = part(p) + (t * (D / 4 + 2) + 2 + 4 * dd + k) * 64 + lane;
                const float g = weight[p][n];
#pragma unroll
                for (int j = 0; j < 4; j++)
                    o[j] = __builtin_fmaf(src[4 * j * 64], g, o[j]);
            }
            __syncthreads();  // the last piece's reads of sum are done
            sum[wave][lane] = o;
            __syncthreads();
            if (wave == 0 && i < s.nq) {
                for (int q = 1; q < waves; q++)
                    o += sum[q][lane];
                *(u32x2*)(a.out + token * a.ld_out + (int64_t)head * D + (4 * (lane >> 4) + k) * (D / 16) + dd) =
                    (u32x2){pack_bf16x2(o[0] * scale, o[1] * scale), pack_bf16x2(o[2] * scale, o[3] * scale)};
            }
        }
        __syncthreads();  // weight and red are written again
    }
}

}  // namespace nvfp4
