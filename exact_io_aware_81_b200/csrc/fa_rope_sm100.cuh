// fa_rope_sm100.cuh -- rotary positions with several axes, and the rotated keys' way into a
// paged KV cache.
//
// A token t has one position per axis (time, height, width, ...); frequency f belongs to one
// axis and turns one pair (x, y) of a head's elements by the angle
//     a = positions[axis_f][t] * inv_freq[f]:   (x cos a - y sin a,  x sin a + y cos a).
// The pairs are (f, f + F) or, interleaved, (2f, 2f + 1); elements past 2F (partial rotary)
// are copied.  The inverse rotation (-a) is the transpose, i.e. the gradient.
//
// Rounding.  The angle of a far position needs more than 24 bits: a is formed in 64 bits, in
// turns, reduced to [-1/2, 1/2] exactly there, and only then rounded to 32 bits for
// sincospif.  The rotation runs in 32 bits and is rounded once, to the output's type.
//
// Bound: HBM (every element is read once and written once, about 3 flops per element).  A CTA
// takes `tokens` tokens (few tokens: a share of one token's rows): its threads compute the
// tokens' sines and cosines once, into shared memory, then go over the rows, 2 x 16 bytes per
// thread, the angles read back as needed, so few registers are held and many warps keep loads
// in flight.  (16384 tokens of 32 + 8 heads, d = 128, bf16: 55.7 us = 6.0 TB/s, 0.92 of a plain
// copy; a warp per token with the angles in registers, 105 of them, ran at 4.8 TB/s.  12187 packed
// tokens into pages: k and v alone 18.8 us as bf16 and 14.4 as E4M3, 0.81 and 0.79 of the copy rate;
// with rotated k and q 54.2 and 58.8, 0.84 and 0.71.)
//
// PAGES: k and v rows go to row p % page_size of page block_table[b][p / page_size], p the
// token's position in its sequence's cache, as bf16 or (FP8) as E4M3 bytes of the scaled value.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "fa.h"
#include "fa_common.cuh"

namespace fa {

struct RopeParams {
    const void *q, *k, *v;   // (T, Hq | Hkv, d), heads contiguous, token strides below
    void *q_out, *k_out;
    long long q_s, k_s, v_s, qo_s, ko_s;  // token strides in elements
    const int *positions;    // (A, T)
    const float *inv_freq;   // (F)
    const int *axes;         // (F), or null: all axis 0
    int T, Hq, Hkv, F, A;
    int interleaved, inverse;
    int split;               // shares of a CTA's rows, over as many CTAs (the any-F kernel: warps per token)
    int tokens;              // tokens of a CTA
    // pages only
    void *kpages, *vpages;   // (num_pages, Hkv, page_size, d)
    const float *k_scale, *v_scale;
    const int *block_table;  // (B, max_pages)
    const int *cu_seqlens;   // (B + 1)
    const int *seqlens;      // (B): lengths that include these tokens
    const int *status;       // (1) or null: not FA_OK, the lengths do not include them and nothing is written
    int B, num_pages, page_size, max_pages;
};

namespace rope {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kTokens = 4;      // most tokens of a CTA
constexpr long long kPadding = -2;  // place of a token behind the last sequence

template <typename T>
struct Vec {
    static constexpr int N = 16 / sizeof(T);
};

__device__ __forceinline__ void unpack(const uint4 &x, float (&f)[8], __nv_bfloat16)
{
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void unpack(const uint4 &x, float (&f)[4], float)
{
    f[0] = __uint_as_float(x.x);
    f[1] = __uint_as_float(x.y);
    f[2] = __uint_as_float(x.z);
    f[3] = __uint_as_float(x.w);
}
__device__ __forceinline__ uint4 pack(const float (&f)[8], __nv_bfloat16)
{
    return make_uint4(ptx::pack_bf16x2(f[0], f[1]), ptx::pack_bf16x2(f[2], f[3]), ptx::pack_bf16x2(f[4], f[5]),
                      ptx::pack_bf16x2(f[6], f[7]));
}
__device__ __forceinline__ uint4 pack(const float (&f)[4], float)
{
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
}

// A scale as the two factors that values are multiplied by: `inv`, its reciprocal rounded to 24
// bits, and `pre`, a power of two, other than 1 where 1 / scale is no normal number (below 2^-128
// it would be infinite, and a zero NaN).  Both are always applied: a branch around the first took
// 47 registers instead of 32, and the append of a prompt batch 22.6 us instead of 18.4.
struct Scaling {
    float pre, inv;
};
__device__ __forceinline__ Scaling scaling(float scale)
{
    const float a = fabsf(scale);
    const float pre = a < 0x1p-126f ? 0x1p64f : a > 0x1p126f ? 0x1p-64f : 1.f;
    return {pre, __frcp_rn(scale * pre)};
}

// Eight values times 1 / scale as E4M3 bytes, round to nearest even, saturated to +-448 (a NaN
// stays one).  The reciprocal, rounded once per row to 32 bits, instead of a division per value:
// the quotient is then off by at most 1.5 steps of 32 bits before it is rounded to 4 bits, and 16
// divisions per thread and row made the append of a prompt batch 15% slower.
__device__ __forceinline__ uint2 pack_e4m3(const float (&f)[8], const Scaling &s)
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = __nv_cvt_float2_to_fp8x2(make_float2(f[2 * i] * s.pre * s.inv, f[2 * i + 1] * s.pre * s.inv), __NV_SATFINITE,
                                        __NV_E4M3);
    return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

// cos and sin of pos * inv_freq (see the text above).
__device__ __forceinline__ void angle(int pos, float inv_freq, int inverse, float &c, float &s)
{
    constexpr double kInvTwoPi = 0.15915494309189533577;
    double turns = (double)pos * (double)inv_freq * kInvTwoPi;
    turns -= rint(turns);
    sincospif((float)(2.0 * turns), &s, &c);
    if (inverse) s = -s;
}

// Axis of frequency f; one outside [0, A) is reported and read as axis 0.
__device__ __forceinline__ int axis_of(const RopeParams &p, int f)
{
    if (!p.axes) return 0;
    const int a = read_at(p.axes, f, p.F);
    if (a >= 0 && a < p.A) return a;
    raise_error(kErrAxisRange);
    return 0;
}

// Sequence of packed token t: the number of cu_seqlens[1 .. B] that are <= t (B: the token
// lies behind the last sequence).  Whole warp; each step narrows the range 32 times.
__device__ __forceinline__ int sequence_of(const int *cu, int B, int t)
{
    const int lane = threadIdx.x & 31;
    int lo = 0, n = B;  // the count lies in [lo, lo + n]
    while (n > 0) {
        const int step = (n + 31) / 32;
        const int i = lo + (lane + 1) * step;  // entries up to i are <= t?
        const bool le = (lane + 1) * step <= n && read_at(cu, i, B + 1) <= t;
        const int c = __popc(__ballot_sync(0xffffffffu, le));
        lo += c * step;
        n = min(step - 1, n - c * step);
    }
    return lo;
}

// Did the reservation that the tokens need not take place?  Their positions are then those of
// finished tokens, perhaps in shared pages.
__device__ __forceinline__ bool refused(const RopeParams &p) { return p.status && *p.status != FA_OK; }

// Where token t's k and v go: row = page * Hkv * page_size + the row in the page, or -1 (and
// an error recorded) when the lengths or the block table do not hold the token.  False for a
// token behind the last sequence, of which nothing is written.  Whole warp.
__device__ __forceinline__ bool page_row_of(const RopeParams &p, int t, long long &row)
{
    row = -1;
    const int b = sequence_of(p.cu_seqlens, p.B, t);
    if (b >= p.B) return false;
    const int c0 = read_at(p.cu_seqlens, b, p.B + 1), n = read_at(p.cu_seqlens, b + 1, p.B + 1) - c0;
    const long long pos = (long long)read_at(p.seqlens, b, p.B) - n + (t - c0);
    unsigned int err = 0;
    if (t < c0 || t - c0 >= n || pos < 0 || pos >= (long long)p.page_size * p.max_pages) {
        err = kErrCuSeqlens;
    } else {
        const int pg = read_at(p.block_table, (long long)b * p.max_pages + pos / p.page_size, (long long)p.B * p.max_pages);
        if (pg < 0 || pg >= p.num_pages) err = kErrPageRange;
        else row = (long long)pg * p.Hkv * p.page_size + pos % p.page_size;
    }
    if (err && (threadIdx.x & 31) == 0) raise_error(err);
    return true;
}

// cos and sin of frequency f of token t.
__device__ __forceinline__ void angle_of(const RopeParams &p, int f, int t, float &c, float &s)
{
    angle(read_at(p.positions, (long long)axis_of(p, f) * p.T + t, (long long)p.A * p.T), read_at(p.inv_freq, f, p.F),
          p.inverse, c, s);
}

// Does row h of token t lie in a (T, H, D) tensor with token stride s (q, k, v and the outputs)?
template <int D>
__device__ __forceinline__ bool row_ok(const RopeParams &p, long long s, int H, long long t, int h)
{
    return in_bounds(t * s + (long long)h * D, (p.T - 1) * s + (long long)H * D - (D - 1));
}

// The same for row r of the rows of token t that are read: those of q, then of k, then of v.
template <int D>
__device__ __forceinline__ bool source_ok(const RopeParams &p, long long t, int r)
{
    return r < p.Hq           ? row_ok<D>(p, p.q_s, p.Hq, t, r)
           : r < p.Hq + p.Hkv ? row_ok<D>(p, p.k_s, p.Hkv, t, r - p.Hq)
                              : row_ok<D>(p, p.v_s, p.Hkv, t, r - p.Hq - p.Hkv);
}

// And of the rows that are written to the outputs.
template <int D>
__device__ __forceinline__ bool output_ok(const RopeParams &p, long long t, int r)
{
    return r < p.Hq ? row_ok<D>(p, p.qo_s, p.Hq, t, r) : row_ok<D>(p, p.ko_s, p.Hkv, t, r - p.Hq);
}

}  // namespace rope

// D: head dim.  T: element type of q, k, v.  PAGES: k and v go to the pages (FP8: as E4M3
// bytes) instead of k_out.  ROT: rotate q and k (else k and v are only stored).  For frequency
// counts with which every 16-byte chunk is rotated as a whole or not at all: F a multiple of a
// chunk's elements, or of half of them when interleaved.
template <int D, typename T, bool PAGES, bool FP8, bool ROT>
__global__ void __launch_bounds__(rope::kThreads) fa_rope_kernel(const RopeParams p)
{
    using namespace rope;
    constexpr int V = Vec<T>::N;           // elements per 16-byte chunk
    constexpr int CH = D / V;              // chunks per row
    constexpr int LANES = CH / 2;          // threads per row, two chunks each
    constexpr int STEP = kThreads / LANES; // rows the CTA takes at a time
    constexpr int QV = V / 4;              // float4s of V angles
    constexpr int kUnroll = FP8 ? 1 : 3;   // rows in flight per thread (registers against warps)
    static_assert(!FP8 || V == 8, "FP8 pages are written from bf16 rows");
    // cos and sin of frequency lc * V + 4 q + e of token t at [t][q][lc].e: the threads of a row
    // read consecutive 16-byte words
    __shared__ float4 cos_t[ROT ? kTokens : 1][QV][LANES], sin_t[ROT ? kTokens : 1][QV][LANES];
    __shared__ long long page_rows[kTokens];

    if (PAGES && refused(p)) return;
    const int tid = threadIdx.x;
    const int part = blockIdx.x % p.split;
    const int t0 = (int)(blockIdx.x / p.split) * p.tokens;
    const int nt = min(p.tokens, p.T - t0);
    const int n_rows = p.Hq + p.Hkv + (PAGES ? p.Hkv : 0);
    const int lc = tid % LANES;

    // Chunks of this thread in every row, and whether each is rotated.
    const int FC = p.F / V;  // half-split: chunks of x elements
    int ca = 2 * lc, cb = 2 * lc + 1;
    bool rot_a = false, rot_b = false;
    if (ROT && !p.interleaved) {
        // chunk c < FC pairs with c + FC; from 2 FC on elements are copied
        if (lc < FC) {
            ca = lc;
            cb = lc + FC;
            rot_a = rot_b = true;
        }
    } else if (ROT) {
        rot_a = (ca + 1) * V <= 2 * p.F;
        rot_b = (cb + 1) * V <= 2 * p.F;
    }

    // Where the tokens' k and v go: a warp per token.
    if (PAGES) {
        for (int i = tid >> 5; i < nt; i += kThreads / 32) {
            long long row;
            const bool real = page_row_of(p, t0 + i, row);
            if ((tid & 31) == 0) page_rows[i] = real ? row : kPadding;
        }
    }
    if (ROT) {
        float *ct = reinterpret_cast<float *>(cos_t), *st = reinterpret_cast<float *>(sin_t);
        for (int i = tid; i < nt * p.F; i += kThreads) {
            const int t = i / p.F, f = i - t * p.F;
            float c, sn;
            angle_of(p, f, t0 + t, c, sn);
            const int l = f / V, e = f % V;
            const int at = ((t * QV + e / 4) * LANES + l) * 4 + e % 4;
            ct[at] = c;
            st[at] = sn;
        }
    }
    __syncthreads();

    // Rows part * STEP + tid / LANES, ... of the CTA's tokens, token by token.
    int tok = 0, row = part * STEP + tid / LANES;
    const int hop = p.split * STEP;
    auto settle = [&]() {
        while (row >= n_rows && tok < nt) {
            row -= n_rows;
            ++tok;
        }
    };
    settle();
    while (tok < nt) {
        uint4 xa[kUnroll], xb[kUnroll];
        int toks[kUnroll], rows[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            toks[u] = tok;
            rows[u] = row;
            if (tok < nt) {
                const long long t = t0 + tok;
                const T *src = row < p.Hq           ? static_cast<const T *>(p.q) + t * p.q_s + (long long)row * D
                               : row < p.Hq + p.Hkv ? static_cast<const T *>(p.k) + t * p.k_s + (long long)(row - p.Hq) * D
                                                    : static_cast<const T *>(p.v) + t * p.v_s +
                                                          (long long)(row - p.Hq - p.Hkv) * D;
                if (source_ok<D>(p, t, row)) {
                    xa[u] = *reinterpret_cast<const uint4 *>(src + ca * V);
                    xb[u] = *reinterpret_cast<const uint4 *>(src + cb * V);
                }
            }
            row += hop;
            settle();
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            if (toks[u] >= nt) continue;
            const long long t = t0 + toks[u];
            const int r = rows[u];
            const bool is_q = r < p.Hq, is_k = !is_q && r < p.Hq + p.Hkv;
            const long long place = PAGES ? page_rows[toks[u]] : 0;
            if (PAGES && place == kPadding) continue;  // behind the last sequence: nothing is written
            float a[V], b[V];
            const bool turn = ROT && (is_q || is_k) && (rot_a || rot_b);
            if (turn || FP8) {
                unpack(xa[u], a, T());
                unpack(xb[u], b, T());
            }
            if (turn) {
                float cs[V], sn[V];
#pragma unroll
                for (int q = 0; q < QV; ++q) {
                    const float4 c = cos_t[toks[u]][q][lc], d = sin_t[toks[u]][q][lc];
                    cs[4 * q] = c.x, cs[4 * q + 1] = c.y, cs[4 * q + 2] = c.z, cs[4 * q + 3] = c.w;
                    sn[4 * q] = d.x, sn[4 * q + 1] = d.y, sn[4 * q + 2] = d.z, sn[4 * q + 3] = d.w;
                }
                if (!p.interleaved) {
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const float x = a[i], y = b[i];
                        a[i] = x * cs[i] - y * sn[i];
                        b[i] = x * sn[i] + y * cs[i];
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < V / 2; ++i) {
                        const float x = a[2 * i], y = a[2 * i + 1];
                        if (rot_a) {
                            a[2 * i] = x * cs[i] - y * sn[i];
                            a[2 * i + 1] = x * sn[i] + y * cs[i];
                        }
                        const float z = b[2 * i], w = b[2 * i + 1];
                        if (rot_b) {
                            b[2 * i] = z * cs[V / 2 + i] - w * sn[V / 2 + i];
                            b[2 * i + 1] = z * sn[V / 2 + i] + w * cs[V / 2 + i];
                        }
                    }
                }
                if (rot_a) xa[u] = pack(a, T());
                if (rot_b) xb[u] = pack(b, T());
            }
            if (is_q || (is_k && !PAGES)) {
                T *dst = is_q ? static_cast<T *>(p.q_out) + t * p.qo_s + (long long)r * D
                              : static_cast<T *>(p.k_out) + t * p.ko_s + (long long)(r - p.Hq) * D;
                if (!output_ok<D>(p, t, r)) continue;
                *reinterpret_cast<uint4 *>(dst + ca * V) = xa[u];
                *reinterpret_cast<uint4 *>(dst + cb * V) = xb[u];
            } else if (PAGES && place >= 0) {
                const int h = is_k ? r - p.Hq : r - p.Hq - p.Hkv;
                const long long at = (place + (long long)h * p.page_size) * D;
                void *pool = is_k ? p.kpages : p.vpages;
                if (!in_bounds(at + D - 1, (long long)p.num_pages * p.Hkv * p.page_size * D)) continue;
                if constexpr (FP8) {
                    const Scaling sc = scaling(read_at(is_k ? p.k_scale : p.v_scale, h, p.Hkv));
                    uint8_t *dst = static_cast<uint8_t *>(pool) + at;
                    *reinterpret_cast<uint2 *>(dst + ca * V) = pack_e4m3(a, sc);
                    *reinterpret_cast<uint2 *>(dst + cb * V) = pack_e4m3(b, sc);
                } else {
                    T *dst = static_cast<T *>(pool) + at;
                    *reinterpret_cast<uint4 *>(dst + ca * V) = xa[u];
                    *reinterpret_cast<uint4 *>(dst + cb * V) = xb[u];
                }
            }
        }
    }
}

// Any F: one lane per pair of one row, element by element; the copied elements follow.  Only
// frequency counts that do not fill whole chunks come here: bound by their 2- and 4-byte accesses
// (16384 tokens of 32 + 8 heads, 13 frequencies, bf16: 157 us, where 64 take 55).
template <int D, typename T, bool PAGES, bool FP8>
__global__ void __launch_bounds__(32 * rope::kWarps) fa_rope_any_kernel(const RopeParams p)
{
    using namespace rope;
    if (PAGES && refused(p)) return;
    const int lane = threadIdx.x & 31;
    const int warp = blockIdx.x * kWarps + (threadIdx.x >> 5);
    const int n_rows = p.Hq + p.Hkv + (PAGES ? p.Hkv : 0);
    for (long long item = warp; item < (long long)p.T * p.split; item += (long long)gridDim.x * kWarps) {
        const int t = (int)(item / p.split);
        const int part = (int)(item - (long long)t * p.split);
        long long page_row = -1;
        if (PAGES && !page_row_of(p, t, page_row)) continue;  // behind the last sequence
        // D / 2 element pairs per row: F turned ones, then the copied elements two by two
        for (int f = lane; f < D / 2; f += 32) {
            float c = 1.f, s = 0.f;
            const bool turned = f < p.F;
            int i0 = 2 * f, i1 = 2 * f + 1;
            if (turned) {
                angle_of(p, f, t, c, s);
                if (!p.interleaved) {
                    i0 = f;
                    i1 = f + p.F;
                }
            }
            for (int r = part; r < n_rows; r += p.split) {
                const bool is_q = r < p.Hq, is_k = !is_q && r < p.Hq + p.Hkv;
                const int h = is_q ? r : is_k ? r - p.Hq : r - p.Hq - p.Hkv;
                const T *src = is_q   ? static_cast<const T *>(p.q) + t * p.q_s
                               : is_k ? static_cast<const T *>(p.k) + t * p.k_s
                                      : static_cast<const T *>(p.v) + t * p.v_s;
                if (!source_ok<D>(p, t, r)) continue;
                T x = src[(long long)h * D + i0], y = src[(long long)h * D + i1];
                float fx = (float)x, fy = (float)y;
                if (turned && (is_q || is_k)) {
                    const float u = fx * c - fy * s, w = fx * s + fy * c;
                    fx = u;
                    fy = w;
                    x = (T)u;
                    y = (T)w;
                }
                if (is_q || (is_k && !PAGES)) {
                    T *dst = is_q ? static_cast<T *>(p.q_out) + t * p.qo_s : static_cast<T *>(p.k_out) + t * p.ko_s;
                    if (!output_ok<D>(p, t, r)) continue;
                    dst[(long long)h * D + i0] = x;
                    dst[(long long)h * D + i1] = y;
                } else if (PAGES && page_row >= 0) {
                    const long long at = (page_row + (long long)h * p.page_size) * D;
                    if (!in_bounds(at + D - 1, (long long)p.num_pages * p.Hkv * p.page_size * D)) continue;
                    void *pool = is_k ? p.kpages : p.vpages;
                    if (FP8) {
                        const Scaling sc = scaling(read_at(is_k ? p.k_scale : p.v_scale, h, p.Hkv));
                        uint8_t *dst = static_cast<uint8_t *>(pool) + at;
                        dst[i0] = __nv_cvt_float_to_fp8(fx * sc.pre * sc.inv, __NV_SATFINITE, __NV_E4M3);
                        dst[i1] = __nv_cvt_float_to_fp8(fy * sc.pre * sc.inv, __NV_SATFINITE, __NV_E4M3);
                    } else {
                        static_cast<T *>(pool)[at + i0] = x;
                        static_cast<T *>(pool)[at + i1] = y;
                    }
                }
            }
        }
    }
}

}  // namespace fa
