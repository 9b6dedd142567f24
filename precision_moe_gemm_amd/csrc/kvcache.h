// kvcache.h -- writing the paged NVFP4 KV cache (page
// "Qwen3.8-2.4T-A95B-NVFP4": K and V stored at about 4 bits): q and k rotated
// by position, k and v quantized and stored in the slots of their tokens.
//
// Rotation of a pair (a, b) with the cosine c and sine s of its angle:
//   a' = bf16(a * c - b * s),  b' = bf16(b * c + a * s)
// in fp32, every step rounded (no fused multiply-add).  The rotated k goes
// through bf16 as the k of a separate rotation would, so the cache bytes are
// those of nvfp4_kv_quant on the rotated k.
#pragma once
#include "common.h"

namespace nvfp4 {

struct AppendArgs {
    const uint16_t* x[3];      // q, k, v rows [n, heads * D]; q may be null
    int64_t ld[3];             // token strides in elements
    int heads[3];
    uint16_t* q_out;           // rotated q
    int64_t ld_qout;
    uint32_t* packed[2];       // k, v caches
    uint8_t* scales[2];
    const float* global[2];
    const int64_t* slots;      // [n]
    const int32_t* positions;  // [n]; null without rotation
    const float* cos_sin;      // [max_pos, rot]: rot / 2 cosines, then rot / 2 sines
    int64_t max_pos, tokens;   // table rows; cache tokens
    int64_t n;
    int cpr;                   // 8-element chunks per row (D / 8)
    int rot;                   // rotated elements of a row
    int interleaved;           // pairs (2i, 2i + 1) instead of (i, i + rot / 2)
};

// A row of D elements is cut into D / 16 units of two 8-element chunks:
// rotated halves (chunks c and c + rot / 16 hold the first and the second
// elements of eight pairs), then the rest in two halves likewise.  One thread
// holds the same unit of many rows of one token, so it reads its 8 cosines
// and 8 sines once, and q may be rotated in place.  D and rot are multiples
// of 32: units 2j and 2j + 1 then hold the two halves of the same NVFP4
// blocks, and two neighbouring lanes share the block maxima.
// blockIdx.y walks tokens, blockIdx.x a token's rows (q, then k, then v).
__global__ void __launch_bounds__(256)
kv_append_kernel(AppendArgs a)
{
    const int units = a.cpr >> 1;
    const int per = 256 / units;  // rows per trip
    const int r0 = threadIdx.x / units, u = threadIdx.x - r0 * units;
    const int half = a.rot >> 1, uh = half >> 3;  // rotated units
    const int rows = a.heads[0] + a.heads[1] + a.heads[2];
    const bool turn = u < uh;
    const int ca = turn ? u : uh + u;             // the unit's chunks
    const int cb = turn ? u + uh : units + u;
    for (int64_t t = blockIdx.y; t < a.n; t += gridDim.y) {
        const int64_t slot = a.slots[t];
        // a negative slot stores nothing: a padding token
        bool keep = slot >= 0 && slot < a.tokens;
        bool ok = true;
        float4_t co[2], si[2];
        if (a.rot > 0) {
            const int32_t pos = a.positions[t];
            ok = pos >= 0 && pos < a.max_pos;
            if (turn) {
                const float* cs = a.cos_sin + (int64_t)(ok ? pos : 0) * a.rot;
                // interleaved: pairs [4c, 4c + 4) of each chunk; else pairs [8u, 8u + 8)
                const int p0 = a.interleaved ? 4 * ca : 8 * u, p1 = a.interleaved ? 4 * cb : 8 * u + 4;
                co[0] = *(const float4_t*)(cs + p0);
                co[1] = *(const float4_t*)(cs + p1);
                si[0] = *(const float4_t*)(cs + half + p0);
                si[1] = *(const float4_t*)(cs + half + p1);
            }
        }
        keep = keep && ok;
        if (blockIdx.x == 0 && threadIdx.x == 0 && (slot >= a.tokens || (!ok && slot >= 0)))
            raise_error(NVFP4_ERR_RANGE);
        // (every lane of a wave runs every trip: the block maxima cross lanes)
        const int step = gridDim.x * per;
        for (int base = blockIdx.x * per; base < rows; base += step) {
            const int r = base + r0;
            const int which = r < a.heads[0] ? 0 : (r < a.heads[0] + a.heads[1] ? 1 : 2);
            const int head = r - (which == 0 ? 0 : (which == 1 ? a.heads[0] : a.heads[0] + a.heads[1]));
            const bool in = r0 < per && r < rows && (which == 0 || keep);
            u32x4 x = (u32x4){0, 0, 0, 0}, y = x;
            if (in && ok) {
                const u32x4* row = (const u32x4*)(a.x[which] + t * a.ld[which]) + (int64_t)head * a.cpr;
                x = row[ca];
                y = row[cb];
                if (turn && which != 2) {
#pragma unroll
                    for (int i = 0; i < 4; i++) {
                        if (a.interleaved) {
                            const float a0 = bf16_lo(x[i]), b0 = bf16_hi(x[i]), a1 = bf16_lo(y[i]), b1 = bf16_hi(y[i]);
                            x[i] = pack_bf16x2(a0 * co[0][i] - b0 * si[0][i], b0 * co[0][i] + a0 * si[0][i]);
                            y[i] = pack_bf16x2(a1 * co[1][i] - b1 * si[1][i], b1 * co[1][i] + a1 * si[1][i]);
                        } else {
                            const float a0 = bf16_lo(x[i]), a1 = bf16_hi(x[i]), b0 = bf16_lo(y[i]), b1 = bf16_hi(y[i]);
                            const int q = i >> 1, e = (i & 1) * 2;
                            x[i] = pack_bf16x2(a0 * co[q][e] - b0 * si[q][e], a1 * co[q][e + 1] - b1 * si[q][e + 1]);
                            y[i] = pack_bf16x2(b0 * co[q][e] + a0 * si[q][e], b1 * co[q][e + 1] + a1 * si[q][e + 1]);
                        }
                    }
                }
            }
            if (in && which == 0) {
                u32x4* o = (u32x4*)(a.q_out + t * a.ld_qout) + (int64_t)head * a.cpr;
                o[ca] = x;
                o[cb] = y;
            }
            uint32_t ax = absmax_bits8(x), ay = absmax_bits8(y);
            ax = umax_u32(ax, swz_xor<1>(ax));
            ay = umax_u32(ay, swz_xor<1>(ay));
            if (in && which != 0) {
                const float G = *a.global[which - 1], six_g = 6.0f * G;
                const int64_t o = (slot * a.heads[which] + head) * a.cpr;
                uint32_t* packed = a.packed[which - 1] + o;
                uint8_t* scales = a.scales[which - 1] + (o >> 1);
                uint32_t sx, sy;
                const float rx = block_scale(ax, G, six_g, &sx), ry = block_scale(ay, G, six_g, &sy);
                packed[ca] = encode_half(x, rx);
                packed[cb] = encode_half(y, ry);
                if ((u & 1) == 0) {
                    scales[ca >> 1] = (uint8_t)sx;
                    scales[cb >> 1] = (uint8_t)sy;
                }
            }
        }
    }
}

}  // namespace nvfp4
