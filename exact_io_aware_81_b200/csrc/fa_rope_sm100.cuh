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
// Bound: HBM (every element is read once and written once, about 3 flops per element).  One
// warp takes one token (or, with few tokens, a share of one token's rows): a lane owns the
// same two 16-byte chunks of every row, so its sines and cosines are computed once per token
// and stay in registers over all heads of q and k.  kRowUnroll rows per lane are loaded before
// the first is used, to keep enough bytes in flight.
//
// PAGES: k and v rows go to row p % page_size of page block_table[b][p / page_size], p the
// token's position in its sequence's cache, as bf16 or (FP8) as E4M3 bytes of value / scale.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp8.h>

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
    int split;               // warps per token
    // pages only
    void *kpages, *vpages;   // (num_pages, Hkv, page_size, d)
    const float *k_scale, *v_scale;
    const int *block_table;  // (B, max_pages)
    const int *cu_seqlens;   // (B + 1)
    const int *seqlens;      // (B): lengths that include these tokens
    int B, num_pages, page_size, max_pages;
};

namespace rope {

constexpr int kWarps = 8;       // warps per CTA
constexpr int kRowUnroll = 4;   // rows in flight per lane

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

// Eight values / scale as E4M3 bytes, round to nearest even, saturated to +-448 (a NaN stays
// one).  The division is the correctly rounded one, so the byte depends on the value alone.
__device__ __forceinline__ uint2 pack_e4m3(const float (&f)[8], float scale)
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = __nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(f[2 * i], scale), __fdiv_rn(f[2 * i + 1], scale)),
                                        __NV_SATFINITE, __NV_E4M3);
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
    const int a = p.axes[f];
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
        const bool le = (lane + 1) * step <= n && cu[i] <= t;
        const int c = __popc(__ballot_sync(0xffffffffu, le));
        lo += c * step;
        n = min(step - 1, n - c * step);
    }
    return lo;
}

// Where token t's k and v go: row = page * Hkv * page_size + the row in the page, or -1 (and
// an error recorded) when the lengths or the block table do not hold the token.  False for a
// token behind the last sequence, of which nothing is written.  Whole warp.
__device__ __forceinline__ bool page_row_of(const RopeParams &p, int t, long long &row)
{
    row = -1;
    const int b = sequence_of(p.cu_seqlens, p.B, t);
    if (b >= p.B) return false;
    const int c0 = p.cu_seqlens[b], n = p.cu_seqlens[b + 1] - c0;
    const long long pos = (long long)p.seqlens[b] - n + (t - c0);
    unsigned int err = 0;
    if (t < c0 || t - c0 >= n || pos < 0 || pos >= (long long)p.page_size * p.max_pages) {
        err = kErrCuSeqlens;
    } else {
        const int pg = p.block_table[(long long)b * p.max_pages + pos / p.page_size];
        if (pg < 0 || pg >= p.num_pages) err = kErrPageRange;
        else row = (long long)pg * p.Hkv * p.page_size + pos % p.page_size;
    }
    if (err && (threadIdx.x & 31) == 0) raise_error(err);
    return true;
}

}  // namespace rope

// D: head dim.  T: element type of q, k, v.  PAGES: k and v go to the pages (FP8: as E4M3
// bytes) instead of k_out.  ROT: rotate q and k (else k and v are only stored).  VEC: every
// 16-byte chunk is rotated by whole chunks of pairs (F a multiple of the chunk's elements,
// or of half of them when interleaved) or not at all; otherwise pairs are taken one by one.
template <int D, typename T, bool PAGES, bool FP8, bool ROT, bool VEC>
__global__ void __launch_bounds__(32 * rope::kWarps) fa_rope_kernel(const RopeParams p)
{
    using namespace rope;
    constexpr int V = Vec<T>::N;           // elements per 16-byte chunk
    constexpr int CH = D / V;              // chunks per row
    constexpr int LANES = CH / 2;          // lanes per row, two chunks each
    constexpr int ROWS = 32 / LANES;       // rows a warp takes at a time
    static_assert(LANES <= 32 && 32 % LANES == 0, "row layout");
    static_assert(!FP8 || V == 8, "FP8 pages are written from bf16 rows");

    const int lane = threadIdx.x & 31;
    const int warp = blockIdx.x * kWarps + (threadIdx.x >> 5);
    const int n_warps = gridDim.x * kWarps;
    const int lr = lane / LANES, lc = lane % LANES;

    // This lane's two chunks, and the frequency of each of its pairs (the same for every token).
    const int FC = p.F / V;  // half-split: chunks of x elements
    int ca, cb;
    bool rot_a = false, rot_b = false;
    if (ROT && VEC && !p.interleaved) {
        if (lc < FC) {
            ca = lc;
            cb = lc + FC;
            rot_a = rot_b = true;
        } else {
            ca = 2 * lc;  // 2 FC + 2 (lc - FC)
            cb = ca + 1;
        }
    } else {
        ca = 2 * lc;
        cb = ca + 1;
        rot_a = ROT && VEC && (ca + 1) * V <= 2 * p.F;
        rot_b = ROT && VEC && (cb + 1) * V <= 2 * p.F;
    }
    const int f0 = lc * V;  // first of the V frequencies of the two chunks
    const int n_rows = p.Hq + p.Hkv + (PAGES ? p.Hkv : 0);

    for (long long item = warp; item < (long long)p.T * p.split; item += n_warps) {
        const int t = (int)(item / p.split);
        const int part = (int)(item - (long long)t * p.split);

        long long page_row = -1;
        if (PAGES && !page_row_of(p, t, page_row)) continue;  // behind the last sequence

        float cs[V], sn[V];
        if (ROT && VEC) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const bool used = p.interleaved ? (i < V / 2 ? rot_a : rot_b) : rot_a;
                cs[i] = 1.f;
                sn[i] = 0.f;
                if (used) {
                    const int f = f0 + i;
                    angle(p.positions[(long long)axis_of(p, f) * p.T + t], p.inv_freq[f], p.inverse, cs[i], sn[i]);
                }
            }
        }

        // rows of this warp: ROWS at a time, kRowUnroll times
        for (int r0 = part * ROWS; r0 < n_rows; r0 += p.split * ROWS * kRowUnroll) {
            uint4 xa[kRowUnroll], xb[kRowUnroll];
            const T *src[kRowUnroll];
#pragma unroll
            for (int u = 0; u < kRowUnroll; ++u) {
                const int r = r0 + u * p.split * ROWS + lr;
                src[u] = nullptr;
                if (r < p.Hq) src[u] = static_cast<const T *>(p.q) + t * p.q_s + (long long)r * D;
                else if (r < p.Hq + p.Hkv) src[u] = static_cast<const T *>(p.k) + t * p.k_s + (long long)(r - p.Hq) * D;
                else if (r < n_rows) src[u] = static_cast<const T *>(p.v) + t * p.v_s + (long long)(r - p.Hq - p.Hkv) * D;
                if (src[u]) {
                    xa[u] = *reinterpret_cast<const uint4 *>(src[u] + ca * V);
                    xb[u] = *reinterpret_cast<const uint4 *>(src[u] + cb * V);
                }
            }
#pragma unroll
            for (int u = 0; u < kRowUnroll; ++u) {
                const int r = r0 + u * p.split * ROWS + lr;
                const bool is_q = r < p.Hq, is_k = !is_q && r < p.Hq + p.Hkv;
                const bool turn = ROT && VEC && (is_q || is_k);
                float a[V], b[V];
                if (turn || FP8) {
                    unpack(xa[u], a, T());
                    unpack(xb[u], b, T());
                }
                if (turn) {
                    if (!p.interleaved) {
                        if (rot_a) {
#pragma unroll
                            for (int i = 0; i < V; ++i) {
                                const float x = a[i], y = b[i];
                                a[i] = x * cs[i] - y * sn[i];
                                b[i] = x * sn[i] + y * cs[i];
                            }
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < V / 2; ++i) {
                            if (rot_a) {
                                const float x = a[2 * i], y = a[2 * i + 1];
                                a[2 * i] = x * cs[i] - y * sn[i];
                                a[2 * i + 1] = x * sn[i] + y * cs[i];
                            }
                            if (rot_b) {
                                const float x = b[2 * i], y = b[2 * i + 1];
                                b[2 * i] = x * cs[V / 2 + i] - y * sn[V / 2 + i];
                                b[2 * i + 1] = x * sn[V / 2 + i] + y * cs[V / 2 + i];
                            }
                        }
                    }
                    if (rot_a) xa[u] = pack(a, T());
                    if (rot_b) xb[u] = pack(b, T());
                }
                if (is_q || (is_k && !PAGES)) {
                    T *dst = is_q ? static_cast<T *>(p.q_out) + t * p.qo_s + (long long)r * D
                                  : static_cast<T *>(p.k_out) + t * p.ko_s + (long long)(r - p.Hq) * D;
                    *reinterpret_cast<uint4 *>(dst + ca * V) = xa[u];
                    *reinterpret_cast<uint4 *>(dst + cb * V) = xb[u];
                } else if (PAGES && r < n_rows && page_row >= 0) {
                    const int h = is_k ? r - p.Hq : r - p.Hq - p.Hkv;
                    const long long at = (page_row + (long long)h * p.page_size) * D;
                    void *pool = is_k ? p.kpages : p.vpages;
                    if (!in_bounds(at + D - 1, (long long)p.num_pages * p.Hkv * p.page_size * D)) continue;
                    if (FP8) {
                        const float scale = is_k ? p.k_scale[h] : p.v_scale[h];
                        uint8_t *dst = static_cast<uint8_t *>(pool) + at;
                        if constexpr (V == 8) {
                            *reinterpret_cast<uint2 *>(dst + ca * V) = pack_e4m3(a, scale);
                            *reinterpret_cast<uint2 *>(dst + cb * V) = pack_e4m3(b, scale);
                        }
                    } else {
                        T *dst = static_cast<T *>(pool) + at;
                        *reinterpret_cast<uint4 *>(dst + ca * V) = xa[u];
                        *reinterpret_cast<uint4 *>(dst + cb * V) = xb[u];
                    }
                }
            }
        }
    }
}

// Any F: one lane per pair of one row, element by element; the copied elements follow.  Only
// frequency counts that do not fill whole chunks come here.
template <int D, typename T, bool PAGES, bool FP8>
__global__ void __launch_bounds__(32 * rope::kWarps) fa_rope_any_kernel(const RopeParams p)
{
    using namespace rope;
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
                angle(p.positions[(long long)axis_of(p, f) * p.T + t], p.inv_freq[f], p.inverse, c, s);
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
                    dst[(long long)h * D + i0] = x;
                    dst[(long long)h * D + i1] = y;
                } else if (PAGES && page_row >= 0) {
                    const long long at = (page_row + (long long)h * p.page_size) * D;
                    if (!in_bounds(at + D - 1, (long long)p.num_pages * p.Hkv * p.page_size * D)) continue;
                    void *pool = is_k ? p.kpages : p.vpages;
                    if (FP8) {
                        const float scale = is_k ? p.k_scale[h] : p.v_scale[h];
                        uint8_t *dst = static_cast<uint8_t *>(pool) + at;
                        dst[i0] = __nv_cvt_float_to_fp8(__fdiv_rn(fx, scale), __NV_SATFINITE, __NV_E4M3);
                        dst[i1] = __nv_cvt_float_to_fp8(__fdiv_rn(fy, scale), __NV_SATFINITE, __NV_E4M3);
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
