// fa_api.cu -- the C ABI of libfa.so (declared in include/fa.h): argument validation,
// TMA tensor-map encoding, kernel launches on the caller's stream, and the device error
// word.  The library owns no device memory on the compute path; the caller passes every
// buffer, including the decode workspace.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <mutex>

#include "fa.h"
#include "fa_common.cuh"
#include "fa_decode_sm100.cuh"
#include "fa_pages_sm100.cuh"
#include "fa_prefill_sm100.cuh"
#include "fa_rope_sm100.cuh"
#include "fa_varlen_sm100.cuh"

namespace {

constexpr int kVersion = 10000;  // 1.0.0
constexpr unsigned long long kDefaultWaitLimitNs = 2000000000ull;

thread_local char g_msg[512] = "";
unsigned long long g_wait_limit_ns = kDefaultWaitLimitNs;

int fail(int status, const char *fmt, ...)
{
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_msg, sizeof g_msg, fmt, ap);
    va_end(ap);
    return status;
}

int ok()
{
    g_msg[0] = '\0';
    return FA_OK;
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// ------------------------------------------------------------ device facts, cached

struct DeviceInfo {
    bool valid = false;
    bool sm100 = false;
    int num_sms = 0;
    bool prefill_attr_set[2][2][2][2][2] = {};
    bool decode_attr_set[2][4][2][2] = {};
    bool varlen_attr_set[2][2][2][2][2] = {};
};
constexpr int kMaxDevices = 64;
DeviceInfo g_dev[kMaxDevices];
std::mutex g_dev_mu;

int current_device(int *dev, DeviceInfo **info)
{
    cudaError_t e = cudaGetDevice(dev);
    if (e != cudaSuccess) return fail(FA_ERR_CUDA, "cudaGetDevice: %s", cudaGetErrorString(e));
    if (*dev < 0 || *dev >= kMaxDevices) return fail(FA_ERR_UNSUPPORTED, "device index %d", *dev);
    std::lock_guard<std::mutex> lk(g_dev_mu);
    DeviceInfo &d = g_dev[*dev];
    if (!d.valid) {
        int major = 0, minor = 0, sms = 0;
        cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, *dev);
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, *dev);
        e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, *dev);
        if (e != cudaSuccess) return fail(FA_ERR_CUDA, "cudaDeviceGetAttribute: %s", cudaGetErrorString(e));
        d.sm100 = (major == 10 && minor == 0);
        d.num_sms = sms;
        d.valid = true;
    }
    *info = &d;
    if (!d.sm100) return fail(FA_ERR_UNSUPPORTED, "libfa.so is built for sm_100a (B200) only");
    return FA_OK;
}

// -------------------------------------------------------------- TMA descriptors

typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                  const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                  const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn get_encode_fn()
{
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(p);
    });
    return fn;
}

// Encoded maps are cached on the host, keyed by every argument of the encode call (data
// type, rank, base address, sizes, strides, box): a map is a pure function of these, so a
// hit returns exactly what re-encoding would.  Repeated calls on the same buffers (a
// serving loop, a benchmark) then skip the driver's encode, about a microsecond per map.
struct MapKey {
    int dtype, rank;
    const void *base;
    cuuint64_t dims[4], strides[3];
    cuuint32_t box[4];
};
constexpr int kMapCacheSize = 64;
struct MapCache {
    uint64_t hash[kMapCacheSize] = {};  // of the keys: one word to look at per entry
    MapKey key[kMapCacheSize];
    CUtensorMap map[kMapCacheSize];
    bool used[kMapCacheSize] = {};
    int next = 0;
};
MapCache g_maps;
std::mutex g_maps_mu;

uint64_t hash_key(const MapKey &k)
{
    static_assert(sizeof(MapKey) % 8 == 0, "hashed by words");
    uint64_t w[sizeof(MapKey) / 8], h = 0;
    memcpy(w, &k, sizeof k);
    for (uint64_t x : w) {
        h = (h ^ x) * 0x9E3779B97F4A7C15ull;
        h ^= h >> 29;
    }
    return h;
}

int encode_map_cached(CUtensorMap *m, CUtensorMapDataType dtype, int rank, const void *base,
                      const cuuint64_t *dims, const cuuint64_t *strides, const cuuint32_t *box)
{
    MapKey k;
    memset(&k, 0, sizeof k);  // padding too: keys are compared bytewise
    k.dtype = (int)dtype;
    k.rank = rank;
    k.base = base;
    for (int i = 0; i < rank; ++i) {
        k.dims[i] = dims[i];
        k.box[i] = box[i];
        if (i + 1 < rank) k.strides[i] = strides[i];
    }
    const uint64_t hash = hash_key(k);
    {
        std::lock_guard<std::mutex> lk(g_maps_mu);
        for (int i = 0; i < kMapCacheSize; ++i)
            if (g_maps.hash[i] == hash && g_maps.used[i] && memcmp(&g_maps.key[i], &k, sizeof k) == 0) {
                *m = g_maps.map[i];
                return FA_OK;
            }
    }
    EncodeTiledFn fn = get_encode_fn();
    if (!fn) return fail(FA_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    CUresult r = fn(m, dtype, (cuuint32_t)rank, const_cast<void *>(base), dims, strides, box, estr,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(FA_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", (int)r);
    std::lock_guard<std::mutex> lk(g_maps_mu);
    const int slot = g_maps.next;
    g_maps.next = (slot + 1) % kMapCacheSize;
    g_maps.hash[slot] = hash;
    g_maps.key[slot] = k;
    g_maps.map[slot] = *m;
    g_maps.used[slot] = true;
    return FA_OK;
}

// A (D, rows, planes) bf16 tensor with boxes of `box_rows` rows x 64 columns, 128-byte
// swizzle.
int encode_rows_map(CUtensorMap *m, const void *base, int D, long long rows, long long planes,
                    unsigned box_rows = 128, bool fp8 = false)
{
    // one box row is 128 bytes: 64 bf16 or 128 FP8 (byte) elements
    const cuuint64_t eb = fp8 ? 1 : 2;
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)rows, (cuuint64_t)planes};
    const cuuint64_t strides[2] = {(cuuint64_t)D * eb, (cuuint64_t)rows * D * eb};
    const cuuint32_t box[3] = {(cuuint32_t)(128 / eb), box_rows, 1};
    return encode_map_cached(m, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, base,
                             dims, strides, box);
}

// A prefill operand as a 4-D (d, rows, heads, batch) tensor with boxes of `box_rows` rows x
// 128 bytes of one head (64 bf16 or 128 E4M3 columns), 128-byte swizzle.  The memory layout
// is (batch, heads, rows, d), or (batch, rows, heads, d) when `bshd`: only the strides differ.
int encode_heads_map(CUtensorMap *m, const void *base, int D, int rows, int heads, int batch, bool bshd,
                     unsigned box_rows = 128, bool fp8 = false)
{
    const cuuint64_t eb = fp8 ? 1 : 2;
    const cuuint64_t row = (cuuint64_t)D * eb, plane = (cuuint64_t)rows * heads * row;
    const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)rows, (cuuint64_t)heads, (cuuint64_t)batch};
    const cuuint64_t strides[3] = {bshd ? heads * row : row, bshd ? row : rows * row, plane};
    const cuuint32_t box[4] = {(cuuint32_t)(128 / eb), box_rows, 1, 1};
    return encode_map_cached(m, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, base,
                             dims, strides, box);
}

// ------------------------------------------------------------------- prefill

int validate_fwd(const void *q, const void *k, const void *v, const void *o, const float *lse,
                 int B, int Hq, int Hkv, int Nq, int Nk, int d, float scale, int causal,
                 int o_dtype)
{
    if (!q || !k || !v || !o || !lse) return fail(FA_ERR_INVALID, "null pointer argument");
    if (B <= 0 || Hq <= 0 || Hkv <= 0 || Nq <= 0 || Nk <= 0 || d <= 0)
        return fail(FA_ERR_INVALID, "sizes must be positive (B=%d Hq=%d Hkv=%d Nq=%d Nk=%d d=%d)",
                    B, Hq, Hkv, Nq, Nk, d);
    if (Hq % Hkv != 0) return fail(FA_ERR_INVALID, "Hq (%d) must be a multiple of Hkv (%d)", Hq, Hkv);
    if (causal && Nq > Nk) return fail(FA_ERR_INVALID, "causal attention needs Nq <= Nk (%d > %d)", Nq, Nk);
    if (!(scale > 0.f) || !std::isfinite(scale)) return fail(FA_ERR_INVALID, "scale must be finite and > 0");
    if (o_dtype != FA_BF16 && o_dtype != FA_F32) return fail(FA_ERR_INVALID, "unknown output dtype %d", o_dtype);
    if (d != 64 && d != 128) return fail(FA_ERR_UNSUPPORTED, "head dim %d (supported: 64, 128)", d);
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o))
        return fail(FA_ERR_UNSUPPORTED, "q, k, v and o must be 16-byte aligned");
    if ((long long)B * Hq > 0x7fffffffLL || (long long)B * Hkv * Nk > 0x7fffffffLL * 64LL)
        return fail(FA_ERR_UNSUPPORTED, "problem too large");
    return FA_OK;
}

template <int D, bool F32, bool SPLIT, bool WINDOW, bool FP8 = false>
int launch_prefill(const fa::PrefillParams &p, DeviceInfo *info, cudaStream_t st)
{
    using C = fa::prefill::Cfg<D, FP8>;
    static_assert(C::kSmemBytes <= 227 * 1024, "prefill shared memory");
    auto kern = fa::fa_prefill_kernel<D, F32, SPLIT, WINDOW, FP8>;
    {
        std::lock_guard<std::mutex> lk(g_dev_mu);
        bool &set = info->prefill_attr_set[D == 128][F32][SPLIT][WINDOW][FP8];
        if (!set) {
            cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 C::kSmemBytes);
            if (e != cudaSuccess)
                return fail(FA_ERR_CUDA, "cudaFuncSetAttribute: %s", cudaGetErrorString(e));
            set = true;
        }
    }
    const int grid = p.n_slots < info->num_sms ? p.n_slots : info->num_sms;
    kern<<<grid, fa::prefill::kThreads, C::kSmemBytes, st>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return fail(FA_ERR_CUDA, "prefill launch: %s", cudaGetErrorString(e));
    return FA_OK;
}

// Kernel variant for one head dim, output type and input type: P handed over in halves for
// head-pair tiling, and the sliding-window variant only when a window is set.
template <int D, bool F32, bool FP8 = false>
int launch_prefill_variant(const fa::PrefillParams &p, DeviceInfo *info, cudaStream_t st)
{
    const bool win = p.window > 0;
    if (p.head_pair)
        return win ? launch_prefill<D, F32, true, true, FP8>(p, info, st)
                   : launch_prefill<D, F32, true, false, FP8>(p, info, st);
    return win ? launch_prefill<D, F32, false, true, FP8>(p, info, st)
               : launch_prefill<D, F32, false, false, FP8>(p, info, st);
}

// FP8 inputs: E4M3 Q, K, V with per-head scales (q_scale, k_scale, v_scale non-null).
struct Fp8Scales {
    const float *q, *k, *v;
};

int fwd_impl(const void *q, const void *k, const void *v, void *o, float *lse, int B, int Hq,
             int Hkv, int Nq, int Nk, int d, float scale, int causal, int window, int o_dtype,
             bool bshd, void *stream, int selftest_timeout, const Fp8Scales *fp8 = nullptr,
             bool debug_bounds_selftest = false)
{
    int rc = validate_fwd(q, k, v, o, lse, B, Hq, Hkv, Nq, Nk, d, scale, causal, o_dtype);
    if (rc != FA_OK) return rc;
    if (window < 0) return fail(FA_ERR_INVALID, "window must be >= 0 (got %d)", window);
    if (window > 0 && !causal) return fail(FA_ERR_INVALID, "a sliding window needs causal attention");
    if (fp8 && (!fp8->q || !fp8->k || !fp8->v)) return fail(FA_ERR_INVALID, "null scale pointer");
    if (fp8 && d != 128) return fail(FA_ERR_UNSUPPORTED, "FP8 prefill needs d = 128 (got %d)", d);
    int dev;
    DeviceInfo *info;
    if ((rc = current_device(&dev, &info)) != FA_OK) return rc;

    fa::PrefillParams p;
    memset(&p, 0, sizeof p);
    const bool f8 = fp8 != nullptr;
    if ((rc = encode_heads_map(&p.tm_q, q, d, Nq, Hq, B, bshd, 128, f8)) != FA_OK) return rc;
    if ((rc = encode_heads_map(&p.tm_k, k, d, Nk, Hkv, B, bshd, 128, f8)) != FA_OK) return rc;
    if ((rc = encode_heads_map(&p.tm_v, v, d, Nk, Hkv, B, bshd, 128, f8)) != FA_OK) return rc;
    // bf16 O leaves through TMA stores of one warp's 32 rows
    if (o_dtype == FA_BF16 && (rc = encode_heads_map(&p.tm_o, o, d, Nq, Hq, B, bshd, 32)) != FA_OK) return rc;
    if (f8) {
        p.q_scale = fp8->q;
        p.k_scale = fp8->k;
        p.v_scale = fp8->v;
    }
    p.o = o;
    p.o_sb = (long long)Hq * Nq * d;
    p.o_sh = bshd ? d : (long long)Nq * d;
    p.o_sn = bshd ? (long long)Hq * d : d;
    p.lse = lse;
    p.B = B;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.Nq = Nq;
    p.Nk = Nk;
    p.R = Hq / Hkv;
    p.causal = causal ? 1 : 0;
    p.window = window < Nk ? window : 0;  // a window of Nk or more keys is plain causal
    p.head_pair = (p.R % 2 == 0) ? 1 : 0;
    const int tiles = (Nq + 127) / 128;
    long long head_slots;
    if (p.head_pair) {
        p.T = tiles;
        head_slots = (long long)B * Hkv * (p.R / 2);
    } else {
        p.T = (tiles + 1) / 2;
        head_slots = (long long)B * Hq;
    }
    p.P = p.causal ? (p.T + 1) / 2 : p.T;
    const long long slots = head_slots * p.P;
    if (slots > 0x3fffffffLL) return fail(FA_ERR_UNSUPPORTED, "problem too large");
    p.n_slots = (int)slots;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.wait_limit_ns = g_wait_limit_ns;
    p.selftest_no_s_signal = selftest_timeout;
    // the debug build's bounds self-test moves every LSE index past the end of its buffer
    p.debug_lse_offset = debug_bounds_selftest ? (long long)B * Hq * Nq : 0;

    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool f32 = o_dtype == FA_F32;
    if (f8)
        rc = f32 ? launch_prefill_variant<128, true, true>(p, info, st)
                 : launch_prefill_variant<128, false, true>(p, info, st);
    else if (d == 128)
        rc = f32 ? launch_prefill_variant<128, true>(p, info, st) : launch_prefill_variant<128, false>(p, info, st);
    else
        rc = f32 ? launch_prefill_variant<64, true>(p, info, st) : launch_prefill_variant<64, false>(p, info, st);
    if (rc != FA_OK) return rc;
    return ok();
}

// -------------------------------------------------------------------- decode

long long decode_splits(int Nmax) { return (Nmax + fa::decode::kChunk - 1) / fa::decode::kChunk; }

// Rows per TMA box of the decode kernels: the 64-row stages of the bf16 kernel and the
// 64-key blocks of the FP8 one.
int decode_block_keys(int, bool fp8) { return fp8 ? fa::decode::kSK : fa::decode::kSub; }

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

size_t decode_ws_bytes(int B, int Hq, int Nmax, int d)
{
    if (B <= 0 || Hq <= 0 || Nmax <= 0 || d <= 0) return 0;
    const size_t S = (size_t)decode_splits(Nmax);
    return align256((size_t)B * Hq * S * d * sizeof(float)) + align256((size_t)B * Hq * S * sizeof(float));
}

// Persistent split kernel, 3 CTAs per SM (at most one per candidate work item): the bf16
// kernel, or the FP8 one (head dim 128).
template <int D, int RG, bool PAGED, bool FP8>
int launch_split(fa::DecodeParams p, DeviceInfo *info, cudaStream_t st)
{
    static_assert(!FP8 || D == 128, "FP8 caches: head dim 128");
    constexpr int smem = FP8 ? fa::decode::WorkerCfg<RG>::kSmemBytes : fa::decode::SplitCfg<D, RG>::kSmemBytes;
    static_assert(smem * fa::decode::kCtasPerSm <= 227 * 1024, "decode CTAs per SM do not fit");
    void (*kern)(fa::DecodeParams);
    if constexpr (FP8) kern = fa::fa_decode_fp8_kernel<RG, PAGED>;
    else kern = fa::fa_decode_split_kernel<D, RG, PAGED>;
    {
        std::lock_guard<std::mutex> lk(g_dev_mu);
        bool &set = info->decode_attr_set[D == 128][RG == 8 ? 3 : RG == 4 ? 2 : RG == 2 ? 1 : 0][PAGED][FP8];
        if (!set) {
            cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
            if (e != cudaSuccess)
                return fail(FA_ERR_CUDA, "cudaFuncSetAttribute: %s", cudaGetErrorString(e));
            set = true;
        }
    }
    p.n_hg = p.Hq / RG;
    p.n_items = p.S_max * p.B * p.n_hg;
    const int max_ctas = fa::decode::kCtasPerSm * info->num_sms;
    const int grid = p.n_items < max_ctas ? p.n_items : max_ctas;
    kern<<<grid, fa::decode::kThreads, smem, st>>>(p);
    return FA_OK;
}

template <int D, bool PAGED = false, bool FP8 = false>
int launch_split_rg(const fa::DecodeParams &p, int rg, DeviceInfo *info, cudaStream_t st)
{
    switch (rg) {
    case 8: return launch_split<D, 8, PAGED, FP8>(p, info, st);
    case 4: return launch_split<D, 4, PAGED, FP8>(p, info, st);
    case 2: return launch_split<D, 2, PAGED, FP8>(p, info, st);
    default: return launch_split<D, 1, PAGED, FP8>(p, info, st);
    }
}

// The merge kernel is launched as a programmatic dependent of the split kernel, so its
// launch overlaps the split kernel's tail; griddepcontrol.wait inside it orders the reads.
template <int D>
cudaError_t launch_merge(const fa::DecodeParams &p, cudaStream_t st)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.B * p.Hq));
    cfg.blockDim = dim3(32 * fa::kMergeWarps);
    cfg.dynamicSmemBytes = 0;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, fa::fa_decode_merge_kernel<D>, p);
}

}  // namespace

namespace {

// The caches of a decode call beyond the contiguous bf16 layout of fa_decode.
struct CacheDesc {
    const void *k, *v;                // contiguous caches (B, Hkv, Nmax, d) or page pools
    bool fp8;                         // E4M3 bytes with per-head scales
    const float *k_scale, *v_scale;   // (Hkv) each, FP8 only
    bool paged;
    const int *block_table;           // (B, max_pages), paged only
    int num_pages, page_size, max_pages;
};

// Validation and launch shared by every decode entry point.  Nmax is the contiguous cache
// length (ignored when paged: page_size * max_pages).
int decode_general(const void *q, const CacheDesc &c, const int *seqlens, void *o, float *lse,
                   int B, int Hq, int Hkv, int Nmax, int d, float scale, void *workspace,
                   size_t workspace_bytes, void *stream, int o_dtype = FA_BF16, int selftest = 0)
{
    if (o_dtype != FA_BF16 && o_dtype != FA_F32) return fail(FA_ERR_INVALID, "unknown output dtype %d", o_dtype);
    if (!q || !c.k || !c.v || !seqlens || !o) return fail(FA_ERR_INVALID, "null pointer argument");
    if (c.fp8 && (!c.k_scale || !c.v_scale)) return fail(FA_ERR_INVALID, "null scale pointer");
    if (c.paged && !c.block_table) return fail(FA_ERR_INVALID, "null block table");
    if (B <= 0 || Hq <= 0 || Hkv <= 0 || d <= 0)
        return fail(FA_ERR_INVALID, "sizes must be positive (B=%d Hq=%d Hkv=%d d=%d)", B, Hq, Hkv, d);
    if (c.paged) {
        if (c.num_pages <= 0 || c.page_size <= 0 || c.max_pages <= 0)
            return fail(FA_ERR_INVALID, "page sizes must be positive (num_pages=%d page_size=%d max_pages=%d)",
                        c.num_pages, c.page_size, c.max_pages);
    } else if (Nmax <= 0) {
        return fail(FA_ERR_INVALID, "Nmax must be positive (%d)", Nmax);
    }
    if (Hq % Hkv != 0) return fail(FA_ERR_INVALID, "Hq (%d) must be a multiple of Hkv (%d)", Hq, Hkv);
    if (!(scale > 0.f) || !std::isfinite(scale)) return fail(FA_ERR_INVALID, "scale must be finite and > 0");
    if (d != 64 && d != 128) return fail(FA_ERR_UNSUPPORTED, "head dim %d (supported: 64, 128)", d);
    if (c.fp8 && d != 128) return fail(FA_ERR_UNSUPPORTED, "FP8 caches need d = 128 (got %d)", d);
    if (c.paged && c.page_size % 16 != 0)
        return fail(FA_ERR_UNSUPPORTED, "page_size %d is not a multiple of 16", c.page_size);
    if (!aligned16(q) || !aligned16(c.k) || !aligned16(c.v) || !aligned16(o))
        return fail(FA_ERR_UNSUPPORTED, "q, the caches and o must be 16-byte aligned");
    const long long nmax = c.paged ? (long long)c.page_size * c.max_pages : Nmax;
    const long long planes = c.paged ? (long long)c.num_pages * Hkv : (long long)B * Hkv;
    if (B > 65535 || nmax > 0x7fffffffLL || planes > 0x7fffffffLL)
        return fail(FA_ERR_UNSUPPORTED, "problem too large");
    Nmax = (int)nmax;
    const size_t need = decode_ws_bytes(B, Hq, Nmax, d);
    if (!workspace || workspace_bytes < need)
        return fail(FA_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need, workspace_bytes);
    if (!aligned16(workspace)) return fail(FA_ERR_WORKSPACE, "workspace must be 16-byte aligned");
    int dev, rc;
    DeviceInfo *info;
    if ((rc = current_device(&dev, &info)) != FA_OK) return rc;

    const int R = Hq / Hkv;
    const int rg = (R % 8 == 0) ? 8 : (R % 4 == 0) ? 4 : (R % 2 == 0) ? 2 : 1;
    if (Hq / rg > 65535) return fail(FA_ERR_UNSUPPORTED, "too many head groups");

    fa::DecodeParams p;
    memset(&p, 0, sizeof p);
    p.q = static_cast<const __nv_bfloat16 *>(q);
    if (c.paged) {
        // rows per copy: the largest power of two that divides page_size, at most one block
        p.box_rows = c.page_size & -c.page_size;
        if (p.box_rows > decode_block_keys(d, c.fp8)) p.box_rows = decode_block_keys(d, c.fp8);
        p.block_table = c.block_table;
        p.page_size = c.page_size;
        p.max_pages = c.max_pages;
        p.num_pages = c.num_pages;
    } else {
        p.box_rows = decode_block_keys(d, c.fp8);
    }
    const long long map_rows = c.paged ? c.page_size : Nmax;
    if ((rc = encode_rows_map(&p.tm_k, c.k, d, map_rows, planes, p.box_rows, c.fp8)) != FA_OK) return rc;
    if ((rc = encode_rows_map(&p.tm_v, c.v, d, map_rows, planes, p.box_rows, c.fp8)) != FA_OK) return rc;
    p.k_scale = c.k_scale;
    p.v_scale = c.v_scale;
    p.seqlens = seqlens;
    p.S_max = (int)decode_splits(Nmax);
    p.part_o = static_cast<float *>(workspace);
    p.part_lse = reinterpret_cast<float *>(static_cast<char *>(workspace) +
                                           align256((size_t)B * Hq * p.S_max * d * sizeof(float)));
    if (o_dtype == FA_F32) p.o_f32 = static_cast<float *>(o);
    else p.o = static_cast<__nv_bfloat16 *>(o);
    p.lse = lse;
    p.B = B;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.Nmax = Nmax;
    p.R = R;
    p.scale_log2 = scale * 1.4426950408889634f;

    cudaStream_t st = static_cast<cudaStream_t>(stream);
    p.wait_limit_ns = g_wait_limit_ns;
    p.selftest_no_full = selftest;
    if (c.fp8)
        rc = c.paged ? launch_split_rg<128, true, true>(p, rg, info, st) : launch_split_rg<128, false, true>(p, rg, info, st);
    else if (c.paged)
        rc = (d == 128) ? launch_split_rg<128, true>(p, rg, info, st) : launch_split_rg<64, true>(p, rg, info, st);
    else
        rc = (d == 128) ? launch_split_rg<128, false>(p, rg, info, st) : launch_split_rg<64, false>(p, rg, info, st);
    if (rc != FA_OK) return rc;
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return fail(FA_ERR_CUDA, "decode split launch: %s", cudaGetErrorString(e));
    e = (d == 128) ? launch_merge<128>(p, st) : launch_merge<64>(p, st);
    if (e != cudaSuccess) return fail(FA_ERR_CUDA, "decode merge launch: %s", cudaGetErrorString(e));
    return ok();
}

}  // namespace

// ------------------------------------------------- attention over packed sequences

namespace {

constexpr int kVarlenHeadBytes = 256;
int check_workspace(const void *ws, size_t have, size_t need)
{
    if (!ws || have < need) return fail(FA_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need, have);
    if (!aligned16(ws)) return fail(FA_ERR_WORKSPACE, "workspace must be 16-byte aligned");
    return FA_OK;
}

// Query heads of one K/V head that share a tile: the largest divisor of R up to 32 (so that a
// job holds at least 8 tokens).
int varlen_pack(int R)
{
    for (int p = R < 32 ? R : 32; p > 1; --p)
        if (R % p == 0) return p;
    return 1;
}

int varlen_max_jobs(int B, int Tq, int pack) { return Tq / (2 * (128 / pack)) + B; }

size_t varlen_ws_bytes(int B, int Tq, int Hq, int Hkv)
{
    if (B <= 0 || Tq <= 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0) return 0;
    return kVarlenHeadBytes + (size_t)varlen_max_jobs(B, Tq, varlen_pack(Hq / Hkv)) * 32;
}

// The attention kernel is a programmatic dependent of the plan kernel: its set-up runs while
// the plan is made.
template <int D, bool F32, bool WINDOW, bool PAGED, bool SHORT>
int launch_varlen(const fa::VarlenParams &p, int grid, DeviceInfo *info, cudaStream_t st)
{
    using C = fa::varlen::Cfg<D, SHORT>;
    static_assert(C::kSmemBytes <= 227 * 1024, "packed attention shared memory");
    auto kern = fa::fa_varlen_kernel<D, F32, WINDOW, PAGED, SHORT>;
    {
        std::lock_guard<std::mutex> lk(g_dev_mu);
        bool &set = info->varlen_attr_set[D == 128][F32][WINDOW][PAGED][SHORT];
        if (!set) {
            cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
            if (e != cudaSuccess) return fail(FA_ERR_CUDA, "cudaFuncSetAttribute: %s", cudaGetErrorString(e));
            set = true;
        }
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(fa::varlen::kAttnThreads);
    cfg.dynamicSmemBytes = C::kSmemBytes;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.plan ? 1 : 0;  // (without a plan kernel before it, it depends on what came before)
    cudaError_t e = cudaLaunchKernelEx(&cfg, kern, p);
    if (e != cudaSuccess) return fail(FA_ERR_CUDA, "packed attention launch: %s", cudaGetErrorString(e));
    return FA_OK;
}

template <int D, bool F32, bool PAGED>
int launch_varlen_sized(const fa::VarlenParams &p, bool few, int grid, DeviceInfo *info, cudaStream_t st)
{
    if (few)
        return p.window > 0 ? launch_varlen<D, F32, true, PAGED, true>(p, grid, info, st)
                            : launch_varlen<D, F32, false, PAGED, true>(p, grid, info, st);
    return p.window > 0 ? launch_varlen<D, F32, true, PAGED, false>(p, grid, info, st)
                        : launch_varlen<D, F32, false, PAGED, false>(p, grid, info, st);
}

template <bool PAGED>
int launch_varlen_variant(const fa::VarlenParams &p, int d, bool f32, bool few, int grid, DeviceInfo *info,
                          cudaStream_t st)
{
    if (d == 128)
        return f32 ? launch_varlen_sized<128, true, PAGED>(p, few, grid, info, st)
                   : launch_varlen_sized<128, false, PAGED>(p, few, grid, info, st);
    return f32 ? launch_varlen_sized<64, true, PAGED>(p, few, grid, info, st)
               : launch_varlen_sized<64, false, PAGED>(p, few, grid, info, st);
}

// The same rows as a (d, heads, tokens, 1) map with boxes of `pack` heads of `tokens` tokens:
// the tile's rows are then token by token, head by head.
int encode_token_map(CUtensorMap *m, const void *base, int D, long long rows, int heads, long long stride, int pack,
                     int tokens)
{
    const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)rows, 1};
    const cuuint64_t strides[3] = {(cuuint64_t)D * 2, (cuuint64_t)stride * 2, (cuuint64_t)stride * 2};
    const cuuint32_t box[4] = {64, (cuuint32_t)pack, (cuuint32_t)tokens, 1};
    return encode_map_cached(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, base, dims, strides, box);
}

// Packed rows (T, heads, d), tokens `stride` elements apart, as the 4-D (d, rows, heads, 1)
// map of the prefill kernel.
int encode_packed_map(CUtensorMap *m, const void *base, int D, long long rows, int heads, long long stride)
{
    const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)rows, (cuuint64_t)heads, 1};
    const cuuint64_t strides[3] = {(cuuint64_t)stride * 2, (cuuint64_t)D * 2, (cuuint64_t)stride * 2};
    const cuuint32_t box[4] = {64, 128, 1, 1};
    return encode_map_cached(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, base, dims, strides, box);
}

// The keys of a packed call: packed tensors, or pages.
struct VarlenKeys {
    const void *k, *v;
    const int *cu_k;
    int Tk;
    long long k_stride, v_stride;
    bool paged;
    const int *block_table, *seqlens;
    int num_pages, page_size, max_pages;
};

bool token_stride_ok(long long stride, int heads, int d) { return stride >= (long long)heads * d && stride % 8 == 0; }

int varlen_general(const void *q, const VarlenKeys &c, const int *cu_q, void *o, float *lse, int B, int Tq, int Hq,
                   int Hkv, int d, long long q_stride, float scale, int causal, int window, int o_dtype,
                   void *workspace, size_t workspace_bytes, void *stream)
{
    if (!q || !o || !lse || !cu_q) return fail(FA_ERR_INVALID, "null pointer argument");
    if (c.paged ? (!c.k || !c.v || !c.block_table || !c.seqlens) : (!c.cu_k || (c.Tk > 0 && (!c.k || !c.v))))
        return fail(FA_ERR_INVALID, "null pointer argument");
    if (B <= 0 || Tq <= 0 || Hq <= 0 || Hkv <= 0 || d <= 0 || c.Tk < 0)
        return fail(FA_ERR_INVALID, "sizes must be positive (B=%d Tq=%d Tk=%d Hq=%d Hkv=%d d=%d)", B, Tq, c.Tk, Hq, Hkv, d);
    if (c.paged && (c.num_pages <= 0 || c.page_size <= 0 || c.max_pages <= 0))
        return fail(FA_ERR_INVALID, "page sizes must be positive (num_pages=%d page_size=%d max_pages=%d)", c.num_pages,
                    c.page_size, c.max_pages);
    if (Hq % Hkv != 0) return fail(FA_ERR_INVALID, "Hq (%d) must be a multiple of Hkv (%d)", Hq, Hkv);
    if (!(scale > 0.f) || !std::isfinite(scale)) return fail(FA_ERR_INVALID, "scale must be finite and > 0");
    if (o_dtype != FA_BF16 && o_dtype != FA_F32) return fail(FA_ERR_INVALID, "unknown output dtype %d", o_dtype);
    if (window < 0) return fail(FA_ERR_INVALID, "window must be >= 0 (got %d)", window);
    if (window > 0 && !causal) return fail(FA_ERR_INVALID, "a sliding window needs causal attention");
    if (d != 64 && d != 128) return fail(FA_ERR_UNSUPPORTED, "head dim %d (supported: 64, 128)", d);
    if (!token_stride_ok(q_stride, Hq, d) ||
        (!c.paged && c.Tk > 0 && (!token_stride_ok(c.k_stride, Hkv, d) || !token_stride_ok(c.v_stride, Hkv, d))))
        return fail(FA_ERR_UNSUPPORTED, "a token stride must hold the heads and be a multiple of 16 bytes");
    if (c.paged && c.page_size % 16 != 0)
        return fail(FA_ERR_UNSUPPORTED, "page_size %d is not a multiple of 16", c.page_size);
    if (!aligned16(q) || !aligned16(c.k) || !aligned16(c.v) || !aligned16(o))
        return fail(FA_ERR_UNSUPPORTED, "q, k, v and o must be 16-byte aligned");
    if (B > fa::varlen::kMaxSeqs) return fail(FA_ERR_UNSUPPORTED, "at most %d sequences in one call (%d)", fa::varlen::kMaxSeqs, B);
    const long long keys = c.paged ? (long long)c.page_size * c.max_pages : c.Tk;
    const int R = Hq / Hkv;
    const int pack = varlen_pack(R), slots = Hq / pack;
    const long long units = ((long long)Tq / (2 * (128 / pack)) + B) * slots;
    if (Tq >= (1 << 26) || keys >= (1 << 30) || units > 0x3fffffffLL ||
        (c.paged && (long long)c.num_pages * Hkv > 0x3fffffffLL))
        return fail(FA_ERR_UNSUPPORTED, "problem too large");
    int rc;
    if ((rc = check_workspace(workspace, workspace_bytes, varlen_ws_bytes(B, Tq, Hq, Hkv))) != FA_OK) return rc;
    int dev;
    DeviceInfo *info;
    if ((rc = current_device(&dev, &info)) != FA_OK) return rc;

    fa::VarlenParams p;
    memset(&p, 0, sizeof p);
    if ((rc = encode_token_map(&p.tm_q, q, d, Tq, Hq, q_stride, pack, 128 / pack)) != FA_OK) return rc;
    if (c.paged) {
        p.box_rows = c.page_size & -c.page_size;
        if (p.box_rows > 128) p.box_rows = 128;
        const long long planes = (long long)c.num_pages * Hkv;
        if ((rc = encode_rows_map(&p.tm_k, c.k, d, c.page_size, planes, p.box_rows)) != FA_OK) return rc;
        if ((rc = encode_rows_map(&p.tm_v, c.v, d, c.page_size, planes, p.box_rows)) != FA_OK) return rc;
        p.block_table = c.block_table;
        p.page_size = c.page_size;
        p.max_pages = c.max_pages;
        p.num_pages = c.num_pages;
    } else {
        // without a single key every tile is masked and its values cleared: any memory does
        const bool none = c.Tk == 0;
        if ((rc = encode_packed_map(&p.tm_k, none ? q : c.k, d, none ? Tq : c.Tk, Hkv, none ? q_stride : c.k_stride)) != FA_OK ||
            (rc = encode_packed_map(&p.tm_v, none ? q : c.v, d, none ? Tq : c.Tk, Hkv, none ? q_stride : c.v_stride)) != FA_OK)
            return rc;
    }
    if (o_dtype == FA_BF16 && 32 % pack == 0 &&
        (rc = encode_token_map(&p.tm_o, o, d, Tq, Hq, (long long)Hq * d, pack, 32 / pack)) != FA_OK)
        return rc;
    p.o = o;
    p.lse = lse;
    p.B = B;
    p.Tq = Tq;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.R = R;
    p.causal = causal ? 1 : 0;
    p.window = window < keys ? window : 0;  // a window of every key is plain causal
    p.pack = pack;
    p.tile_tokens = 128 / pack;
    p.slots = slots;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.wait_limit_ns = g_wait_limit_ns;
    p.plan_head = static_cast<int *>(workspace);
    int4 *plan = reinterpret_cast<int4 *>(static_cast<char *>(workspace) + kVarlenHeadBytes);

    fa::VarlenPlanParams &m = p.jobs;
    m.cu_q = cu_q;
    m.cu_k = c.cu_k;
    m.seqlens = c.paged ? c.seqlens : nullptr;
    m.plan = plan;
    m.head = p.plan_head;
    m.B = B;
    m.Tq = Tq;
    m.Tk = (int)keys;
    m.rows = 2 * p.tile_tokens;
    m.causal = p.causal;
    m.window = p.window;
    // SHORT is for a few tokens against many keys: tiles without a partner, units that are few and
    // long.  The lengths are known on the device only, so the rule looks at what the host has: the
    // tokens, the keys that k, or the pool and the table, can hold (a server's hold more than its
    // sequences have), both on average, and how many units a CTA gets at most.  Measured on B200
    // (32 + 8 heads, d = 128, pages of 64; us with SHORT / LONG): 12 chunks of 1 to 512 tokens over
    // contexts of up to 8192 131 / 187, 24 such 124 / 158; single tokens on contexts of 4096 111 /
    // 118 (37 of them) and 322 / 341 (111), of 1024 45 / 45 and 115 / 112, of 256 26 / 25 and 67 /
    // 56; 512 prompts of 64 tokens with no context 211 / 157.  With many units there is little to
    // gain, and up to a third to lose where the contexts are short: from five a CTA on it is LONG.
    // (Calls of one wave run SHORT, without a plan, whatever this says.)
    const long long pool_keys = c.paged ? (long long)c.page_size * c.num_pages : keys;
    const long long all_keys = c.paged && pool_keys > keys * B ? keys * B : pool_keys;
    m.max_jobs = varlen_max_jobs(B, Tq, pack);
    const long long bound = (long long)m.max_jobs * slots;
    const bool few = (long long)Tq <= 4LL * B * p.tile_tokens && all_keys >= 1024LL * B &&
                     bound <= 5LL * info->num_sms;
    m.twins = few ? 1 : 0;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool wave = bound <= info->num_sms;  // no more units than CTAs: no order to plan
    const int grid = wave ? (int)bound : info->num_sms;
    if (!wave) {
        p.plan = plan;
        fa::fa_varlen_plan_kernel<<<1, fa::varlen::kThreads, 0, st>>>(m);
        cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return fail(FA_ERR_CUDA, "plan launch: %s", cudaGetErrorString(e));
    }
    const bool f32 = o_dtype == FA_F32;
    rc = c.paged ? launch_varlen_variant<true>(p, d, f32, few || wave, grid, info, st)
                 : launch_varlen_variant<false>(p, d, f32, few || wave, grid, info, st);
    if (rc != FA_OK) return rc;
    return ok();
}

}  // namespace

// ---------------------------------------------- rotary positions and cache filling

namespace {

// Where fa_cache_append and fa_rope_append write.
struct PageDest {
    void *k, *v;
    const float *k_scale, *v_scale;
    const int *block_table, *cu_seqlens, *seqlens, *status;
    int B, num_pages, page_size, max_pages;
};

bool stride_ok(long long stride, int heads, int d, int elem)
{
    return heads == 0 || (stride >= (long long)heads * d && (stride * elem) % 16 == 0);
}

template <int D, typename T, bool PAGES, bool FP8>
void launch_rope(fa::RopeParams &p, bool rot, bool vec, int num_sms, cudaStream_t st)
{
    using namespace fa::rope;
    const int rows = p.Hq + p.Hkv + (PAGES ? p.Hkv : 0);
    if (rot && !vec) {
        // a warp per token, or per share of a token's rows while warps are few
        p.split = num_sms * 32 / p.T;
        p.split = p.split < 1 ? 1 : p.split > rows ? rows : p.split;
        const long long ctas = ((long long)p.T * p.split + kWarps - 1) / kWarps;
        const int grid = ctas < num_sms * 8 ? (int)ctas : num_sms * 8;
        fa::fa_rope_any_kernel<D, T, PAGES, FP8><<<grid, kThreads, 0, st>>>(p);
        return;
    }
    // Tokens per CTA: one while that leaves SMs idle, kTokens from two rounds of CTAs on; with
    // fewer tokens than SMs a token's rows are shared out, at least one step of rows to a CTA.
    const int step = kThreads / (D * (int)sizeof(T) / 32);
    p.tokens = p.T >= num_sms * 2 * kTokens ? kTokens : 1;
    const int groups = (p.T + p.tokens - 1) / p.tokens;
    const int most = (p.tokens * rows + step - 1) / step;
    p.split = num_sms / groups;
    p.split = p.split < 1 ? 1 : p.split > most ? most : p.split;
    const long long grid = (long long)groups * p.split;
    if constexpr (PAGES) {
        if (!rot) {
            fa::fa_rope_kernel<D, T, PAGES, FP8, false><<<(unsigned)grid, kThreads, 0, st>>>(p);
            return;
        }
    }
    fa::fa_rope_kernel<D, T, PAGES, FP8, true><<<(unsigned)grid, kThreads, 0, st>>>(p);
}

// Validation and launch shared by fa_rope (pages null), fa_rope_append and fa_cache_append
// (inv_freq null: nothing is rotated).
int rope_general(fa::RopeParams &p, const PageDest *pages, int d, int dtype, void *stream)
{
    const bool rot = p.inv_freq != nullptr;
    if (dtype != FA_BF16 && dtype != FA_F32) return fail(FA_ERR_INVALID, "unknown dtype %d", dtype);
    if (p.T <= 0 || p.Hq < 0 || p.Hkv < 0 || p.Hq + p.Hkv <= 0 || d <= 0)
        return fail(FA_ERR_INVALID, "sizes must be positive (T=%d Hq=%d Hkv=%d d=%d)", p.T, p.Hq, p.Hkv, d);
    if ((p.Hq && (!p.q || !p.q_out)) || (p.Hkv && !p.k) || (!pages && p.Hkv && !p.k_out) || (pages && !p.v))
        return fail(FA_ERR_INVALID, "null pointer argument");
    if (rot && !p.positions) return fail(FA_ERR_INVALID, "null positions");
    if (rot && (p.F <= 0 || p.F > d / 2)) return fail(FA_ERR_INVALID, "F (%d) must lie in [1, d / 2]", p.F);
    if (rot && p.A <= 0) return fail(FA_ERR_INVALID, "A (%d) must be positive", p.A);
    if (d != 64 && d != 128) return fail(FA_ERR_UNSUPPORTED, "head dim %d (supported: 64, 128)", d);
    const int es = dtype == FA_F32 ? 4 : 2;
    if (!stride_ok(p.q_s, p.Hq, d, es) || !stride_ok(p.qo_s, p.Hq, d, es) || !stride_ok(p.k_s, p.Hkv, d, es) ||
        (!pages && !stride_ok(p.ko_s, p.Hkv, d, es)) || (pages && !stride_ok(p.v_s, p.Hkv, d, es)))
        return fail(FA_ERR_UNSUPPORTED, "a token stride must hold the heads and be a multiple of 16 bytes");
    if (!aligned16(p.q) || !aligned16(p.q_out) || !aligned16(p.k) || !aligned16(p.k_out) || !aligned16(p.v))
        return fail(FA_ERR_UNSUPPORTED, "q, k, v and the outputs must be 16-byte aligned");
    bool fp8 = false;
    if (pages) {
        if (!pages->k || !pages->v || !pages->block_table || !pages->cu_seqlens || !pages->seqlens)
            return fail(FA_ERR_INVALID, "null pointer argument");
        if ((pages->k_scale == nullptr) != (pages->v_scale == nullptr))
            return fail(FA_ERR_INVALID, "give both FP8 scale pointers or neither");
        if (p.Hkv <= 0 || pages->B <= 0 || pages->num_pages <= 0 || pages->page_size <= 0 || pages->max_pages <= 0)
            return fail(FA_ERR_INVALID, "sizes must be positive (Hkv=%d B=%d num_pages=%d page_size=%d max_pages=%d)",
                        p.Hkv, pages->B, pages->num_pages, pages->page_size, pages->max_pages);
        fp8 = pages->k_scale != nullptr;
        if (fp8 && d != 128) return fail(FA_ERR_UNSUPPORTED, "FP8 caches need d = 128 (got %d)", d);
        if (pages->page_size % 16 != 0)
            return fail(FA_ERR_UNSUPPORTED, "page_size %d is not a multiple of 16", pages->page_size);
        if (!aligned16(pages->k) || !aligned16(pages->v))
            return fail(FA_ERR_UNSUPPORTED, "the page pools must be 16-byte aligned");
        p.kpages = pages->k;
        p.vpages = pages->v;
        p.k_scale = pages->k_scale;
        p.v_scale = pages->v_scale;
        p.block_table = pages->block_table;
        p.cu_seqlens = pages->cu_seqlens;
        p.seqlens = pages->seqlens;
        p.status = pages->status;
        p.B = pages->B;
        p.num_pages = pages->num_pages;
        p.page_size = pages->page_size;
        p.max_pages = pages->max_pages;
    }
    int dev, rc;
    DeviceInfo *info;
    if ((rc = current_device(&dev, &info)) != FA_OK) return rc;

    const int per = 16 / es;  // elements per 16-byte chunk
    const bool vec = p.interleaved ? (2 * p.F) % per == 0 : p.F % per == 0;

    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (pages) {
        if (fp8) launch_rope<128, __nv_bfloat16, true, true>(p, rot, vec, info->num_sms, st);
        else if (d == 128) launch_rope<128, __nv_bfloat16, true, false>(p, rot, vec, info->num_sms, st);
        else launch_rope<64, __nv_bfloat16, true, false>(p, rot, vec, info->num_sms, st);
    } else if (dtype == FA_F32) {
        if (d == 128) launch_rope<128, float, false, false>(p, true, vec, info->num_sms, st);
        else launch_rope<64, float, false, false>(p, true, vec, info->num_sms, st);
    } else {
        if (d == 128) launch_rope<128, __nv_bfloat16, false, false>(p, true, vec, info->num_sms, st);
        else launch_rope<64, __nv_bfloat16, false, false>(p, true, vec, info->num_sms, st);
    }
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return fail(FA_ERR_CUDA, "rope launch: %s", cudaGetErrorString(e));
    return ok();
}

}  // namespace

// ------------------------------------------------------------------ page management

namespace {

int make_tables(fa::PageTables *t, int *block_table, int *seqlens, int *refcount, int S, int max_pages,
                int num_pages, int page_size, DeviceInfo **info)
{
    if (!block_table || !seqlens || !refcount) return fail(FA_ERR_INVALID, "null pointer argument");
    if (S <= 0 || max_pages <= 0 || num_pages <= 0 || page_size <= 0)
        return fail(FA_ERR_INVALID, "sizes must be positive (S=%d max_pages=%d num_pages=%d page_size=%d)", S,
                    max_pages, num_pages, page_size);
    if (page_size % 16 != 0) return fail(FA_ERR_UNSUPPORTED, "page_size %d is not a multiple of 16", page_size);
    if ((long long)page_size * max_pages > 0x7fffffffLL - page_size || num_pages >= (1 << 21) - 1 || S > (1 << 20))
        return fail(FA_ERR_UNSUPPORTED, "problem too large");
    *t = fa::PageTables{block_table, seqlens, refcount, S, max_pages, num_pages, page_size};
    int dev;
    return current_device(&dev, info);
}

size_t reserve_ws_bytes(int S, int num_pages)
{
    if (S <= 0 || num_pages <= 0) return 0;
    return align256((size_t)S * 4) + align256((size_t)num_pages * 4);
}

size_t compact_ws_bytes(int num_pages)
{
    if (num_pages <= 0) return 0;
    return 256 + 2 * align256((size_t)num_pages * 4);
}

int launched(const char *what)
{
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return fail(FA_ERR_CUDA, "%s launch: %s", what, cudaGetErrorString(e));
    return ok();
}

// What fa_get_error returns for the bits of the error word: one status a call, in this order.
struct ErrorStatus {
    unsigned int bits;
    int status;
};
constexpr ErrorStatus kErrorStatuses[] = {
    {fa::kErrTimeout, FA_ERR_TIMEOUT},
    {fa::kErrSeqlenRange | fa::kErrPageRange | fa::kErrSlot | fa::kErrCuSeqlens | fa::kErrAxisRange, FA_ERR_DEVICE_ARG},
    {fa::kErrNoPages, FA_ERR_NO_PAGES},
    {fa::kErrDebugBounds, FA_ERR_DEBUG_CHECK},
};

struct ErrorMessage {
    unsigned int bit;
    const char *text;
};
constexpr ErrorMessage kErrorMessages[] = {
    {fa::kErrTimeout, "a kernel pipeline wait exceeded its time limit"},
    {fa::kErrSeqlenRange, "seqlens held a value outside [0, Nmax]"},
    {fa::kErrPageRange, "the block table or a copy list held a page outside [0, num_pages)"},
    {fa::kErrSlot, "page management: a slot, length or refcount was not usable"},
    {fa::kErrCuSeqlens, "cu_seqlens does not ascend within [0, T], or disagrees with seqlens"},
    {fa::kErrAxisRange, "axes held a value outside [0, A)"},
    {fa::kErrNoPages, "the pool has fewer free pages than fa_pages_reserve needs; nothing was changed"},
    {fa::kErrDebugBounds, "a kernel's global-memory index failed its bounds check (access skipped)"},
};

}  // namespace

extern "C" {

int fa_fwd(const void *q, const void *k, const void *v, void *o, float *lse, int B, int Hq,
           int Hkv, int Nq, int Nk, int d, float scale, int causal, void *stream)
{
    return fwd_impl(q, k, v, o, lse, B, Hq, Hkv, Nq, Nk, d, scale, causal, 0, FA_BF16, false, stream, 0);
}

int fa_fwd_ex(const void *q, const void *k, const void *v, void *o, float *lse, int B, int Hq,
              int Hkv, int Nq, int Nk, int d, float scale, int causal, int o_dtype, void *stream)
{
    return fwd_impl(q, k, v, o, lse, B, Hq, Hkv, Nq, Nk, d, scale, causal, 0, o_dtype, false, stream, 0);
}

int fa_fwd_window(const void *q, const void *k, const void *v, void *o, float *lse, int B,
                  int Hq, int Hkv, int Nq, int Nk, int d, float scale, int window, int o_dtype,
                  void *stream)
{
    if (window <= 0) return fail(FA_ERR_INVALID, "window must be >= 1 (got %d)", window);
    return fwd_impl(q, k, v, o, lse, B, Hq, Hkv, Nq, Nk, d, scale, 1, window, o_dtype, false, stream, 0);
}

int fa_fwd_bshd(const void *q, const void *k, const void *v, void *o, float *lse, int B, int Hq,
                int Hkv, int Nq, int Nk, int d, float scale, int causal, int window, int o_dtype,
                void *stream)
{
    return fwd_impl(q, k, v, o, lse, B, Hq, Hkv, Nq, Nk, d, scale, causal, window, o_dtype, true, stream, 0);
}

int fa_fwd_fp8(const void *q, const void *k, const void *v, const float *q_scale, const float *k_scale,
               const float *v_scale, void *o, float *lse, int B, int Hq, int Hkv, int Nq, int Nk, int d,
               float scale, int causal, int window, int o_dtype, void *stream)
{
    if (window > 0 && !causal) return fail(FA_ERR_INVALID, "a sliding window needs causal attention");
    const Fp8Scales sc{q_scale, k_scale, v_scale};
    return fwd_impl(q, k, v, o, lse, B, Hq, Hkv, Nq, Nk, d, scale, causal, window, o_dtype, false, stream, 0, &sc);
}

int fa_fwd_selftest_timeout(const void *q, const void *k, const void *v, void *o, float *lse,
                            int B, int Hq, int Hkv, int Nq, int Nk, int d, float scale,
                            int causal, void *stream)
{
    return fwd_impl(q, k, v, o, lse, B, Hq, Hkv, Nq, Nk, d, scale, causal, 0, FA_BF16, false, stream, 1);
}

size_t fa_decode_workspace_size(int B, int Hq, int Nmax, int d) { return decode_ws_bytes(B, Hq, Nmax, d); }

int fa_decode(const void *q, const void *kcache, const void *vcache, const int *seqlens, void *o,
              float *lse, int B, int Hq, int Hkv, int Nmax, int d, float scale, void *workspace,
              size_t workspace_bytes, void *stream)
{
    const CacheDesc c{kcache, vcache, false, nullptr, nullptr, false, nullptr, 0, 0, 0};
    return decode_general(q, c, seqlens, o, lse, B, Hq, Hkv, Nmax, d, scale, workspace, workspace_bytes, stream);
}


int fa_decode_paged(const void *q, const void *kpages, const void *vpages, const int *block_table,
                    const int *seqlens, void *o, float *lse, int B, int Hq, int Hkv, int num_pages,
                    int page_size, int max_pages, int d, float scale, void *workspace,
                    size_t workspace_bytes, void *stream)
{
    const CacheDesc c{kpages, vpages, false, nullptr, nullptr, true, block_table, num_pages, page_size, max_pages};
    return decode_general(q, c, seqlens, o, lse, B, Hq, Hkv, 0, d, scale, workspace, workspace_bytes, stream);
}

int fa_decode_ex(const void *q, const void *kcache, const void *vcache, const int *seqlens, void *o,
                 float *lse, int B, int Hq, int Hkv, int Nmax, int d, float scale, int o_dtype,
                 void *workspace, size_t workspace_bytes, void *stream)
{
    const CacheDesc c{kcache, vcache, false, nullptr, nullptr, false, nullptr, 0, 0, 0};
    return decode_general(q, c, seqlens, o, lse, B, Hq, Hkv, Nmax, d, scale, workspace, workspace_bytes,
                          stream, o_dtype);
}

int fa_decode_selftest_timeout(const void *q, const void *kcache, const void *vcache, const float *k_scale,
                               const float *v_scale, const int *seqlens, void *o, float *lse, int B, int Hq,
                               int Hkv, int Nmax, int d, float scale, void *workspace, size_t workspace_bytes,
                               void *stream)
{
    if ((k_scale == nullptr) != (v_scale == nullptr))
        return fail(FA_ERR_INVALID, "give both FP8 scale pointers or neither");
    const bool fp8 = k_scale != nullptr;
    const CacheDesc c{kcache, vcache, fp8, k_scale, v_scale, false, nullptr, 0, 0, 0};
    return decode_general(q, c, seqlens, o, lse, B, Hq, Hkv, Nmax, d, scale, workspace, workspace_bytes,
                          stream, FA_BF16, 1);
}

int fa_merge_lse(const float *o_parts, const float *lse_parts, int P, int rows, int d, void *o,
                 float *lse, int o_dtype, void *stream)
{
    if (!o_parts || !lse_parts || !o) return fail(FA_ERR_INVALID, "null pointer argument");
    if (P <= 0 || rows <= 0 || d <= 0) return fail(FA_ERR_INVALID, "sizes must be positive (P=%d rows=%d d=%d)", P, rows, d);
    if (o_dtype != FA_BF16 && o_dtype != FA_F32) return fail(FA_ERR_INVALID, "unknown output dtype %d", o_dtype);
    if (d != 64 && d != 128) return fail(FA_ERR_UNSUPPORTED, "head dim %d (supported: 64, 128)", d);
    if ((long long)P * rows * d > 0x7fffffffffffLL) return fail(FA_ERR_UNSUPPORTED, "problem too large");
    int dev, rc;
    DeviceInfo *info;
    if ((rc = current_device(&dev, &info)) != FA_OK) return rc;
    fa::MergeLseParams m;
    m.o_parts = o_parts;
    m.lse_parts = lse_parts;
    m.o = o_dtype == FA_BF16 ? static_cast<__nv_bfloat16 *>(o) : nullptr;
    m.o_f32 = o_dtype == FA_F32 ? static_cast<float *>(o) : nullptr;
    m.lse = lse;
    m.P = P;
    m.rows = rows;
    const unsigned grid = (unsigned)((rows + fa::kMergeLseWarps - 1) / fa::kMergeLseWarps);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (d == 128) fa::fa_merge_lse_kernel<128><<<grid, 32 * fa::kMergeLseWarps, 0, st>>>(m);
    else fa::fa_merge_lse_kernel<64><<<grid, 32 * fa::kMergeLseWarps, 0, st>>>(m);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return fail(FA_ERR_CUDA, "merge launch: %s", cudaGetErrorString(e));
    return ok();
}

int fa_decode_fp8(const void *q, const void *kcache, const void *vcache, const float *k_scale,
                  const float *v_scale, const int *seqlens, void *o, float *lse, int B, int Hq,
                  int Hkv, int Nmax, int d, float scale, void *workspace, size_t workspace_bytes,
                  void *stream)
{
    const CacheDesc c{kcache, vcache, true, k_scale, v_scale, false, nullptr, 0, 0, 0};
    return decode_general(q, c, seqlens, o, lse, B, Hq, Hkv, Nmax, d, scale, workspace, workspace_bytes, stream);
}

int fa_decode_paged_fp8(const void *q, const void *kpages, const void *vpages, const float *k_scale,
                        const float *v_scale, const int *block_table, const int *seqlens, void *o,
                        float *lse, int B, int Hq, int Hkv, int num_pages, int page_size,
                        int max_pages, int d, float scale, void *workspace, size_t workspace_bytes,
                        void *stream)
{
    const CacheDesc c{kpages, vpages, true, k_scale, v_scale, true, block_table, num_pages, page_size, max_pages};
    return decode_general(q, c, seqlens, o, lse, B, Hq, Hkv, 0, d, scale, workspace, workspace_bytes, stream);
}

// ------------------------------------------------------------ allocation-free decode
//
// For callers that cannot allocate device memory (see fa_decode_noalloc in fa.h): the
// split-KV partials live in this fixed array instead of a caller workspace.  In host code
// `g_noalloc_scratch` only names a host-side stand-in; its device address is looked up
// with cudaGetSymbolAddress, with the device current, and that address is what the kernels
// get.  The lookup is done on a device's first call and again whenever the device's
// context has changed since (a cudaDeviceReset unloads the module and the array with it).
static __device__ __align__(256) unsigned char g_noalloc_scratch[FA_NOALLOC_SCRATCH_BYTES];

namespace {

typedef CUresult (*CtxGetCurrentFn)(CUcontext *);
typedef CUresult (*CtxGetIdFn)(CUcontext, unsigned long long *);

// Unique id of the calling thread's current context (0 if it cannot be read).
unsigned long long current_context_id()
{
    static CtxGetCurrentFn get_current = nullptr;
    static CtxGetIdFn get_id = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuCtxGetCurrent", &p, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            get_current = reinterpret_cast<CtxGetCurrentFn>(p);
        if (cudaGetDriverEntryPoint("cuCtxGetId", &p, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            get_id = reinterpret_cast<CtxGetIdFn>(p);
    });
    CUcontext ctx = nullptr;
    unsigned long long id = 0;
    if (!get_current || !get_id || get_current(&ctx) != CUDA_SUCCESS || !ctx || get_id(ctx, &id) != CUDA_SUCCESS)
        return 0;
    return id;
}

struct NoallocScratch {
    void *ptr = nullptr;
    unsigned long long ctx_id = 0;
};
NoallocScratch g_noalloc[kMaxDevices];
std::mutex g_noalloc_mu;

// Device address of the scratch array on the current device, in its current context.
int noalloc_scratch(int dev, void **out)
{
    const unsigned long long ctx = current_context_id();
    std::lock_guard<std::mutex> lk(g_noalloc_mu);
    NoallocScratch &c = g_noalloc[dev];
    if (!c.ptr || ctx == 0 || ctx != c.ctx_id) {
        void *p = nullptr;
        cudaError_t e = cudaGetSymbolAddress(&p, g_noalloc_scratch);
        if (e != cudaSuccess || !p)
            return fail(FA_ERR_CUDA, "cudaGetSymbolAddress of the decode scratch: %s",
                        cudaGetErrorString(e));
        c.ptr = p;
        c.ctx_id = ctx;
    }
    *out = c.ptr;
    return FA_OK;
}

}  // namespace

int fa_decode_noalloc(const void *q, const void *kcache, const void *vcache, const int *seqlens,
                      void *o, float *lse, int B, int Hq, int Hkv, int Nmax, int d, float scale,
                      void *stream)
{
    // the partials must fit the fixed scratch; every other check is fa_decode's
    if (B > 0 && Hq > 0 && Nmax > 0 && d > 0) {
        const size_t need = decode_ws_bytes(B, Hq, Nmax, d);
        if (need > (size_t)FA_NOALLOC_SCRATCH_BYTES)
            return fail(FA_ERR_WORKSPACE,
                        "this decode needs %zu bytes of scratch; fa_decode_noalloc has %u bytes "
                        "(use fa_decode with a workspace for larger problems)",
                        need, (unsigned)FA_NOALLOC_SCRATCH_BYTES);
    }
    if (!q || !kcache || !vcache || !seqlens || !o) return fail(FA_ERR_INVALID, "null pointer argument");
    int dev, rc;
    DeviceInfo *info;
    if ((rc = current_device(&dev, &info)) != FA_OK) return rc;
    void *scratch = nullptr;
    if ((rc = noalloc_scratch(dev, &scratch)) != FA_OK) return rc;
    const CacheDesc c{kcache, vcache, false, nullptr, nullptr, false, nullptr, 0, 0, 0};
    return decode_general(q, c, seqlens, o, lse, B, Hq, Hkv, Nmax, d, scale, scratch,
                          (size_t)FA_NOALLOC_SCRATCH_BYTES, stream);
}

// ---------------------------------------------- rotary positions and cache filling

size_t fa_fwd_varlen_workspace_size(int B, int Tq, int Hq, int Hkv) { return varlen_ws_bytes(B, Tq, Hq, Hkv); }

int fa_fwd_varlen(const void *q, const void *k, const void *v, void *o, float *lse, const int *cu_q, const int *cu_k,
                  int B, int Tq, int Tk, int Hq, int Hkv, int d, long long q_stride, long long k_stride,
                  long long v_stride, float scale, int causal, int window, int o_dtype, void *workspace,
                  size_t workspace_bytes, void *stream)
{
    const VarlenKeys c{k, v, cu_k, Tk, k_stride, v_stride, false, nullptr, nullptr, 0, 0, 0};
    return varlen_general(q, c, cu_q, o, lse, B, Tq, Hq, Hkv, d, q_stride, scale, causal, window, o_dtype, workspace,
                          workspace_bytes, stream);
}

int fa_fwd_varlen_paged(const void *q, const void *kpages, const void *vpages, const int *block_table,
                        const int *cu_q, const int *seqlens, void *o, float *lse, int B, int Tq, int Hq, int Hkv,
                        int num_pages, int page_size, int max_pages, int d, long long q_stride, float scale,
                        int causal, int window, int o_dtype, void *workspace, size_t workspace_bytes, void *stream)
{
    const VarlenKeys c{kpages, vpages, nullptr, 0, 0, 0, true, block_table, seqlens, num_pages, page_size, max_pages};
    return varlen_general(q, c, cu_q, o, lse, B, Tq, Hq, Hkv, d, q_stride, scale, causal, window, o_dtype, workspace,
                          workspace_bytes, stream);
}

int fa_rope(const void *q, const void *k, void *q_out, void *k_out, const int *positions, const float *inv_freq,
            const int *axes, int T, int Hq, int Hkv, int d, int F, int A, long long q_stride, long long k_stride,
            long long q_out_stride, long long k_out_stride, int dtype, int interleaved, int inverse, void *stream)
{
    if (!inv_freq) return fail(FA_ERR_INVALID, "null pointer argument");
    fa::RopeParams p;
    memset(&p, 0, sizeof p);
    p.q = q, p.k = k, p.q_out = q_out, p.k_out = k_out;
    p.q_s = q_stride, p.k_s = k_stride, p.qo_s = q_out_stride, p.ko_s = k_out_stride;
    p.positions = positions, p.inv_freq = inv_freq, p.axes = axes;
    p.T = T, p.Hq = Hq, p.Hkv = Hkv, p.F = F, p.A = A;
    p.interleaved = interleaved ? 1 : 0;
    p.inverse = inverse ? 1 : 0;
    return rope_general(p, nullptr, d, dtype, stream);
}

int fa_rope_append_ex(const void *q, const void *k, const void *v, void *q_out, const int *positions,
                      const float *inv_freq, const int *axes, void *kpages, void *vpages, const float *k_scale,
                      const float *v_scale, const int *block_table, const int *cu_seqlens, const int *seqlens,
                      const int *status, int T, int B, int Hq, int Hkv, int num_pages, int page_size, int max_pages,
                      int d, int F, int A, long long q_stride, long long k_stride, long long v_stride,
                      long long q_out_stride, int interleaved, void *stream)
{
    if (!inv_freq) return fail(FA_ERR_INVALID, "null pointer argument");
    fa::RopeParams p;
    memset(&p, 0, sizeof p);
    p.q = q, p.k = k, p.v = v, p.q_out = q_out;
    p.q_s = q_stride, p.k_s = k_stride, p.v_s = v_stride, p.qo_s = q_out_stride;
    p.positions = positions, p.inv_freq = inv_freq, p.axes = axes;
    p.T = T, p.Hq = Hq, p.Hkv = Hkv, p.F = F, p.A = A;
    p.interleaved = interleaved ? 1 : 0;
    const PageDest dest{kpages, vpages, k_scale, v_scale, block_table, cu_seqlens, seqlens, status, B, num_pages,
                        page_size, max_pages};
    return rope_general(p, &dest, d, FA_BF16, stream);
}

int fa_rope_append(const void *q, const void *k, const void *v, void *q_out, const int *positions,
                   const float *inv_freq, const int *axes, void *kpages, void *vpages, const float *k_scale,
                   const float *v_scale, const int *block_table, const int *cu_seqlens, const int *seqlens, int T,
                   int B, int Hq, int Hkv, int num_pages, int page_size, int max_pages, int d, int F, int A,
                   long long q_stride, long long k_stride, long long v_stride, long long q_out_stride,
                   int interleaved, void *stream)
{
    return fa_rope_append_ex(q, k, v, q_out, positions, inv_freq, axes, kpages, vpages, k_scale, v_scale, block_table,
                             cu_seqlens, seqlens, nullptr, T, B, Hq, Hkv, num_pages, page_size, max_pages, d, F, A,
                             q_stride, k_stride, v_stride, q_out_stride, interleaved, stream);
}

int fa_cache_append_ex(const void *k, const void *v, void *kpages, void *vpages, const float *k_scale,
                       const float *v_scale, const int *block_table, const int *cu_seqlens, const int *seqlens,
                       const int *status, int T, int B, int Hkv, int num_pages, int page_size, int max_pages, int d,
                       long long k_stride, long long v_stride, void *stream)
{
    fa::RopeParams p;
    memset(&p, 0, sizeof p);
    p.k = k, p.v = v, p.k_s = k_stride, p.v_s = v_stride;
    p.T = T, p.Hkv = Hkv;
    const PageDest dest{kpages, vpages, k_scale, v_scale, block_table, cu_seqlens, seqlens, status, B, num_pages,
                        page_size, max_pages};
    return rope_general(p, &dest, d, FA_BF16, stream);
}

int fa_cache_append(const void *k, const void *v, void *kpages, void *vpages, const float *k_scale,
                    const float *v_scale, const int *block_table, const int *cu_seqlens, const int *seqlens, int T,
                    int B, int Hkv, int num_pages, int page_size, int max_pages, int d, long long k_stride,
                    long long v_stride, void *stream)
{
    return fa_cache_append_ex(k, v, kpages, vpages, k_scale, v_scale, block_table, cu_seqlens, seqlens, nullptr, T, B,
                              Hkv, num_pages, page_size, max_pages, d, k_stride, v_stride, stream);
}

// ------------------------------------------------------------------ page management

int fa_pages_fork(int *block_table, int *seqlens, int *refcount, const int *src, const int *dst, const int *lengths,
                  int n, int S, int max_pages, int num_pages, int page_size, void *stream)
{
    if (!src || !dst) return fail(FA_ERR_INVALID, "null pointer argument");
    if (n <= 0) return fail(FA_ERR_INVALID, "n must be positive (%d)", n);
    if (n > 65535) return fail(FA_ERR_UNSUPPORTED, "at most 65535 pairs in one call (%d)", n);
    fa::ForkParams p;
    DeviceInfo *info;
    const int rc = make_tables(&p.t, block_table, seqlens, refcount, S, max_pages, num_pages, page_size, &info);
    if (rc != FA_OK) return rc;
    p.src = src, p.dst = dst, p.lengths = lengths, p.n = n;
    fa::fa_pages_fork_kernel<<<n, fa::pages::kSlotThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
    return launched("fork");
}

int fa_pages_free(int *block_table, int *seqlens, int *refcount, const int *slots, const int *keep, int n, int S,
                  int max_pages, int num_pages, int page_size, void *stream)
{
    if (!slots) return fail(FA_ERR_INVALID, "null pointer argument");
    if (n <= 0) return fail(FA_ERR_INVALID, "n must be positive (%d)", n);
    if (n > 65535) return fail(FA_ERR_UNSUPPORTED, "at most 65535 slots in one call (%d)", n);
    fa::FreeParams p;
    DeviceInfo *info;
    const int rc = make_tables(&p.t, block_table, seqlens, refcount, S, max_pages, num_pages, page_size, &info);
    if (rc != FA_OK) return rc;
    p.slots = slots, p.keep = keep, p.n = n;
    fa::fa_pages_free_kernel<<<n, fa::pages::kSlotThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
    return launched("free");
}

size_t fa_pages_reserve_workspace_size(int S, int num_pages) { return reserve_ws_bytes(S, num_pages); }

int fa_pages_reserve_ex(int *block_table, int *seqlens, int *refcount, const int *add, int *copies, int *status, int S,
                        int max_pages, int num_pages, int page_size, void *workspace, size_t workspace_bytes,
                        void *stream)
{
    if (!add || !copies) return fail(FA_ERR_INVALID, "null pointer argument");
    fa::ReserveParams p;
    DeviceInfo *info;
    int rc = make_tables(&p.t, block_table, seqlens, refcount, S, max_pages, num_pages, page_size, &info);
    if (rc != FA_OK) return rc;
    if ((rc = check_workspace(workspace, workspace_bytes, reserve_ws_bytes(S, num_pages))) != FA_OK) return rc;
    p.add = add, p.copies = copies, p.status = status;
    p.first = static_cast<int *>(workspace);
    p.free_ids = reinterpret_cast<int *>(static_cast<char *>(workspace) + align256((size_t)S * 4));
    fa::fa_pages_reserve_kernel<<<1, fa::pages::kPlanThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
    return launched("reserve");
}

int fa_pages_reserve(int *block_table, int *seqlens, int *refcount, const int *add, int *copies, int S, int max_pages,
                     int num_pages, int page_size, void *workspace, size_t workspace_bytes, void *stream)
{
    return fa_pages_reserve_ex(block_table, seqlens, refcount, add, copies, nullptr, S, max_pages, num_pages, page_size,
                               workspace, workspace_bytes, stream);
}

size_t fa_pages_compact_workspace_size(int num_pages) { return compact_ws_bytes(num_pages); }

int fa_pages_compact(int *block_table, int *seqlens, int *refcount, int *copies, int S, int max_pages, int num_pages,
                     int page_size, void *workspace, size_t workspace_bytes, void *stream)
{
    if (!copies && num_pages > 1) return fail(FA_ERR_INVALID, "null pointer argument");
    fa::CompactParams p;
    DeviceInfo *info;
    int rc = make_tables(&p.t, block_table, seqlens, refcount, S, max_pages, num_pages, page_size, &info);
    if (rc != FA_OK) return rc;
    if ((rc = check_workspace(workspace, workspace_bytes, compact_ws_bytes(num_pages))) != FA_OK) return rc;
    p.copies = copies;
    p.n_live = static_cast<int *>(workspace);
    p.rank = reinterpret_cast<int *>(static_cast<char *>(workspace) + 256);
    p.holes = reinterpret_cast<int *>(static_cast<char *>(workspace) + 256 + align256((size_t)num_pages * 4));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    fa::fa_pages_compact_kernel<<<1, fa::pages::kPlanThreads, 0, st>>>(p);
    if ((rc = launched("compact")) != FA_OK) return rc;
    fa::fa_pages_remap_kernel<<<S, fa::pages::kSlotThreads, 0, st>>>(p);
    return launched("compact");
}

int fa_pages_copy(void *kpages, void *vpages, const int *copies, int n, int num_pages, long long page_bytes,
                  void *stream)
{
    if (!kpages || !copies) return fail(FA_ERR_INVALID, "null pointer argument");
    if (n < 0 || num_pages <= 0 || page_bytes <= 0)
        return fail(FA_ERR_INVALID, "sizes must be positive (n=%d num_pages=%d page_bytes=%lld)", n, num_pages, page_bytes);
    if (page_bytes % 16 != 0 || page_bytes > (1LL << 44) / num_pages)
        return fail(FA_ERR_UNSUPPORTED, "a page of %lld bytes is not a multiple of 16, or the pool is too large", page_bytes);
    if (!aligned16(kpages) || !aligned16(vpages))
        return fail(FA_ERR_UNSUPPORTED, "the page pools must be 16-byte aligned");
    int dev, rc;
    DeviceInfo *info;
    if ((rc = current_device(&dev, &info)) != FA_OK) return rc;
    if (n == 0) return ok();
    fa::PageCopyParams p;
    p.k = static_cast<uint4 *>(kpages);
    p.v = static_cast<uint4 *>(vpages);
    p.copies = copies;
    p.n = n;
    p.num_pages = num_pages;
    p.page_vecs = page_bytes / 16;
    p.pieces = (int)((page_bytes + fa::pages::kPieceBytes - 1) / fa::pages::kPieceBytes);
    const long long items = (long long)n * p.pieces * (vpages ? 2 : 1);
    const int max_ctas = info->num_sms * 8;
    fa::fa_pages_copy_kernel<<<(int)(items < max_ctas ? items : max_ctas), fa::pages::kCopyThreads, 0,
                               static_cast<cudaStream_t>(stream)>>>(p);
    return launched("page copy");
}

int fa_get_error(void *stream)
{
    cudaError_t e = cudaStreamSynchronize(static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return fail(FA_ERR_CUDA, "stream synchronize: %s", cudaGetErrorString(e));
    unsigned int word = 0;
    e = cudaMemcpyFromSymbol(&word, fa::g_error_word, sizeof word);
    if (e != cudaSuccess) return fail(FA_ERR_CUDA, "reading the error word: %s", cudaGetErrorString(e));
    for (const ErrorStatus &s : kErrorStatuses) {
        if (!(word & s.bits)) continue;
        cudaStream_t st = static_cast<cudaStream_t>(stream);
        fa::fa_clear_errors_kernel<<<1, 1, 0, st>>>(s.bits & word);
        e = cudaGetLastError();
        if (e == cudaSuccess) e = cudaStreamSynchronize(st);
        if (e != cudaSuccess) return fail(FA_ERR_CUDA, "clearing the error word: %s", cudaGetErrorString(e));
        for (const ErrorMessage &m : kErrorMessages)
            if (word & s.bits & m.bit) return fail(s.status, "%s", m.text);
    }
    return ok();
}

void fa_set_wait_limit_ns(unsigned long long ns) { g_wait_limit_ns = ns ? ns : kDefaultWaitLimitNs; }

const char *fa_status_str(int status)
{
    switch (status) {
    case FA_OK: return "FA_OK";
    case FA_ERR_INVALID: return "FA_ERR_INVALID";
    case FA_ERR_UNSUPPORTED: return "FA_ERR_UNSUPPORTED";
    case FA_ERR_WORKSPACE: return "FA_ERR_WORKSPACE";
    case FA_ERR_CUDA: return "FA_ERR_CUDA";
    case FA_ERR_TIMEOUT: return "FA_ERR_TIMEOUT";
    case FA_ERR_DEVICE_ARG: return "FA_ERR_DEVICE_ARG";
    case FA_ERR_DEBUG_CHECK: return "FA_ERR_DEBUG_CHECK";
    case FA_ERR_NO_PAGES: return "FA_ERR_NO_PAGES";
    default: return "FA_ERR_UNKNOWN";
    }
}

const char *fa_last_error_message(void) { return g_msg; }

int fa_version(void) { return kVersion; }

int fa_build_flags(void) { return fa::kDebugChecks ? 1 : 0; }

int fa_debug_selftest_bounds(const void *q, const void *k, const void *v, void *o, float *lse, int B, int Hq,
                             int Hkv, int Nq, int Nk, int d, float scale, int causal, void *stream)
{
    if (!fa::kDebugChecks)
        return fail(FA_ERR_UNSUPPORTED, "bounds checks are compiled only into the debug build (libfa_debug.so)");
    return fwd_impl(q, k, v, o, lse, B, Hq, Hkv, Nq, Nk, d, scale, causal, 0, FA_BF16, false, stream, 0, nullptr,
                    true);
}

}  // extern "C"
