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

// The sequence that holds item x when sequence b has count(b) items, the
// item's number in it and the number of all items.  All threads of a
// workgroup of kAttnThreads call it; every thread sums a contiguous share of
// the sequences.
struct AttnFound {
    int64_t total, local;
    int seq;
};

template <class Count>
NVFP4_DEV AttnFound attn_locate(int seqs, int64_t x, int64_t* lds, Count count)
{
    const int per = (seqs + kAttnThreads - 1) / kAttnThreads;
    const int b0 = threadIdx.x * per, b1 = b0 + per < seqs ? b0 + per : seqs;
    int64_t mine = 0;
    for (int b = b0; b < b1; b++)
        mine += count(b);
    int64_t up = mine;  // inclusive sum over the wave's lanes
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const int64_t o = __shfl_up(up, off, 64);
        up += (int)(threadIdx.x & 63) >= off ? o : 0;
    }
    __syncthreads();
    if ((threadIdx.x & 63) == 63)
        lds[threadIdx.x >> 6] = up;
    __syncthreads();
    int64_t before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < kAttnThreads / 64; w++) {
        before += w < (int)(threadIdx.x >> 6) ? lds[w] : 0;
        total += lds[w];
    }
    before += up - mine;
    if (x >= before && x < before + mine) {
        int64_t rest = x - before;
        int b = b0;
        for (; b < b1 - 1; b++) {
            const int64_t c = count(b);
            if (rest < c)
                break;
            rest -= c;
        }
        lds[4] = rest;
        lds[5] = b;
    }
    __syncthreads();
    AttnFound f;
    f.total = total;
    f.local = lds[4];
    f.seq = (int)lds[5];
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

    // the 16 tokens of half `half` of a step: they lie in one page
    NVFP4_DEV void load_half(const AttnArgs& a, AttnRaw<D>& raw, int half, int h, int64_t tok)
    {
        const int64_t row = tok * a.kv_heads + h;  // the first token's cache row
        const int stride = a.kv_heads;
        const uint8_t* kc = a.k_packed + row * (D / 2) + (lane_n() * stride) * (D / 2) + lane_g() * (D / 8);
        const uint8_t* ks = a.k_scales + row * (D / 16) + (lane_n() * stride) * (D / 16) + lane_g() * (D / 64);
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
        const uint8_t* vc = a.v_packed + row * (D / 2) + (4 * lane_g() * stride) * (D / 2) + lane_n() * (D / 32);
        const uint8_t* vs = a.v_scales + row * (D / 16) + (4 * lane_g() * stride) * (D / 16) + lane_n() * D / 256;
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const uint8_t* p = vc + j * stride * (D / 2);
            if constexpr (D == 64) {
                raw.vc[4 * half + j][0] = *(const uint16_t*)p;
            } else if constexpr (D == 128) {
                raw.vc[4 * half + j][0] = *(const uint32_t*)p;
            } else {
                const u32x2 w = *(const u32x2*)p;
                raw.vc[4 * half + j][0] = w.x;
                raw.vc[4 * half + j][1] = w.y;
            }
            raw.vs[4 * half + j] = vs[j * stride * (D / 16)];
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

    // tokens [t0, t1) (t0 a multiple of 32); any: the first token that some
    // row sees; [lo, hi): the tokens that every row sees
    NVFP4_DEV void walk(const AttnArgs& a, const int32_t* table_row, int h, int t0, int t1, int any, int lo, int hi)
    {
        if (t0 >= t1)
            return;
        AttnPages pages;
        pages.row = table_row;
        pages.last = (t1 - 1) / a.page;
        pages.needed = any / a.page;
        int idx = t0 / a.page, off = t0 - idx * a.page;
        pages.fill(a, idx);
        for (int t = t0; t < t1; t += kAttnStep) {
            AttnRaw<D> raw;
            bool ok[2];
#pragma unroll
            for (int half = 0; half < 2; half++) {
                const int i = idx < pages.last ? idx : pages.last;  // past the end: any page, masked
                const int page = pages.get(a, i);
                ok[half] = page >= 0;
                load_half(a, raw, half, h, (int64_t)(page < 0 ? 0 : page) * a.page + off);
                off += 16;
                if (off == a.page) {
                    off = 0;
                    idx++;
                }
            }
            step(raw, t, ok[0] && ok[1] && t >= lo && t + kAttnStep <= hi, ok);
        }
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

// One workgroup: 16 NT query rows of one sequence for head_lanes KV heads
// (blockIdx.y), each wave one of the heads and a share of the tokens.
template <int D, int NT>
__global__ void __launch_bounds__(kAttnThreads)
attn_rows_kernel(AttnArgs a)
{
    __shared__ int64_t found[6];
    __shared__ float buf[2 * (D / 4 + 2) * NT * 64];
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int hl = a.head_lanes, tls = (kAttnThreads / 64) / hl;
    const int h = blockIdx.y * hl + wave % hl, tl = wave / hl;
    const AttnFound f = attn_locate(a.seqs, blockIdx.x, found, [&](int b) {
        const AttnSeq s = attn_seq(a, b);
        return ((int64_t)s.nq * a.group + 16 * NT - 1) / (16 * NT);
    });
    if (blockIdx.x >= f.total)
        return;
    const int b = __builtin_amdgcn_readfirstlane(f.seq);
    const int row0 = __builtin_amdgcn_readfirstlane((int)f.local) * (16 * NT);
    const AttnSeq s = attn_seq(a, b);
    int lo0, hi0, lo1, hi1;  // tokens of the first and of the last row
    const int last = (row0 + 16 * NT - 1) / a.group;
    attn_limits(a, s, row0 / a.group, &lo0, &hi0);
    attn_limits(a, s, last < s.nq ? last : s.nq - 1, &lo1, &hi1);
    AttnWave<D, NT> w;
    w.open(a, s, h, row0);
    const int t0 = lo0 & ~(kAttnStep - 1);
    const int steps = hi1 > t0 ? (hi1 - t0 + kAttnStep - 1) / kAttnStep : 0;
    const int share = (steps + tls - 1) / tls * kAttnStep;
    const int from = t0 + tl * share, to = from + share < hi1 ? from + share : hi1;
    w.walk(a, a.table + b * a.ld_table, h, from, to, lo0, lo1, hi0);
    attn_join<D, NT>(w, hl, wave, buf);
    if (tl == 0)
        attn_finish<D, NT>(a, w, s, h, row0);
}

}  // namespace nvfp4
