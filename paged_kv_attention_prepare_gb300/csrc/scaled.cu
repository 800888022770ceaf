// Writing and reading back pools with a scale per (block, kv head).
//
// "How vLLM Works Internally", section "FP8 KV Cache" (the cache may hold
// FP8 values), with scales that follow the data: a pool holds E4M3 codes, and
// each (block, kv head) of it one power of two 2^e as the byte e + 127, so the
// cached value is code * 2^e.  "Inside vLLM: Following One Request", the write
// op; "Building the Batch", section "Reading and writing the KV cache".
//
// Why powers of two: dividing by the scale is exact, so a code is one
// rounding away from its source; and when a block's exponent grows, because
// a later token is larger, code * 2^(old - new) is exact too unless it falls
// under E4M3's normal range, so the earlier tokens lose nothing else.
#include <cuda_fp8.h>

#include "pa_internal.cuh"

namespace pa {

namespace {

constexpr int kPage = 16;
constexpr int kScaledThreads = 256;
constexpr int kScaledWarps = kScaledThreads / 32;
constexpr int kScaledMaxReqs = 50000;   // the prefix over requests is kept in shared memory

// ---------------------------------------------------------------------------
// Write
// ---------------------------------------------------------------------------

// 16-bit elements: the first magnitude (bits without the sign) that is not
// finite, and a magnitude's float value.
template <typename T> struct Mag;
template <> struct Mag<__nv_bfloat16> {
    static constexpr uint32_t kInf2 = 0x7f807f80u;
    __device__ __forceinline__ static float value(uint32_t m) { return __uint_as_float(m << 16); }
};
template <> struct Mag<__half> {
    static constexpr uint32_t kInf2 = 0x7c007c00u;
    __device__ __forceinline__ static float value(uint32_t m) {
        return __half2float(__ushort_as_half((unsigned short)m));
    }
};

// The smallest e in [kScaleMinExp, kScaleMaxExp] with amax <= 448 * 2^e, the
// largest one where none is.  amax = 1.f * 2^x with 448 = 1.75 * 2^8.
__device__ __forceinline__ int scale_exponent(float amax) {
    const uint32_t b = __float_as_uint(amax);
    const int x = (int)(b >> 23) - 127;
    const int e = (b & 0x7fffffu) <= 0x600000u ? x - 8 : x - 7;
    return min(max(e, kScaleMinExp), kScaleMaxExp);
}

// Eight 16-bit elements to E4M3 codes of element * mul (mul a power of two,
// the product exact), to nearest, ties to even, saturating at +-448 (NaN
// stays NaN).
template <typename T>
__device__ __forceinline__ uint2 quantize8_pow2(const uint4 src, float mul) {
    const uint32_t w[4] = {src.x, src.y, src.z, src.w};
    uint32_t out[2] = {0u, 0u};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        float a, b;
        Elt<T>::unpack2(w[e], a, b);
        const uint32_t q =
            __nv_cvt_float2_to_fp8x2(make_float2(a * mul, b * mul), __NV_SATFINITE, __NV_E4M3);
        out[e >> 1] |= (q & 0xffffu) << (16 * (e & 1));
    }
    return make_uint2(out[0], out[1]);
}

// Two E4M3 codes (the low half of w) as floats, exactly.
__device__ __forceinline__ float2 e4m3x2_value(uint32_t w) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w & 0xffffu), __NV_E4M3);
    return __half22float2(__half2(h));
}

// Eight codes re-coded for a scale 2^-log2(mul) times larger.
__device__ __forceinline__ uint2 recode8(const uint2 c, float mul) {
    const uint32_t w[2] = {c.x, c.y};
    uint32_t out[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const float2 a = e4m3x2_value(w[e]), b = e4m3x2_value(w[e] >> 16);
        const uint32_t qa = __nv_cvt_float2_to_fp8x2(make_float2(a.x * mul, a.y * mul),
                                                     __NV_SATFINITE, __NV_E4M3);
        const uint32_t qb = __nv_cvt_float2_to_fp8x2(make_float2(b.x * mul, b.y * mul),
                                                     __NV_SATFINITE, __NV_E4M3);
        out[e] = (qa & 0xffffu) | (qb << 16);
    }
    return make_uint2(out[0], out[1]);
}

// One warp per (block that the step writes, K or V, kv head): its new rows (1
// to 16 of D elements, all loaded before anything depends on them), their
// largest finite magnitude by an integer maximum of the 16-bit patterns, the
// exponent, the codes.  Only a block that already held tokens reads its own
// exponent, and only one whose exponent grows reads and re-codes its earlier
// rows.  Every CTA scans the requests for the blocks each writes (as the
// index build scans them), so a warp finds its block by a binary search and no
// list is stored; consecutive warps take the kv heads of one block, whose
// rows lie side by side.  Three round trips to memory (lengths; rows and block
// id; the old scale) bound small steps, one wave of four CTAs per SM the large
// ones (64 registers hold a block's 16 rows): 256 single tokens at 8 x 128 in
// 8 us, a 5000-token chunk beside 200 in 14 us (as graph replays, which take
// 4 us empty; three, five or six CTAs per SM 15 us, more waves 14-16).
template <typename T, int D>
__global__ void __launch_bounds__(kScaledThreads, 4) cache_write_scaled_kernel(const ScaledWriteArgs a) {
    constexpr int kLanes = D / 8;            // lanes that share a row, 8 elements each
    constexpr int kRows = 32 / kLanes;       // rows a warp takes at a time
    constexpr int kIters = kPage / kRows;
    extern __shared__ int32_t s_first[];     // [R + 1]: blocks written by earlier requests
    __shared__ int32_t s_scan[33];
    const int tid = threadIdx.x, lane = tid & 31;
    const int R = a.R;
    auto blocks_of = [&](int r, bool report) -> int {
        const int q0 = a.qsl[r], q1 = a.qsl[r + 1], L = a.seq_lens[r];
        const int n = q1 - q0;
        if (q0 < 0 || q1 > a.T || n < 0 || L < n) {
            if (report) flag(a.status, PA_CHECK_SEQ_LEN);
            return 0;
        }
        return n > 0 ? (L - 1) / kPage - (L - n) / kPage + 1 : 0;
    };
    const int per = (R + kScaledThreads - 1) / kScaledThreads;
    const int r0 = min(R, tid * per), r1 = min(R, r0 + per);
    int local = 0;
    for (int r = r0; r < r1; ++r) local += blocks_of(r, blockIdx.x == 0);
    int total = 0;
    int run = block_exclusive_scan(local, s_scan, total);
    for (int r = r0; r < r1; ++r) {
        s_first[r] = run;
        run += per == 1 ? local : blocks_of(r, false);
    }
    __syncthreads();

    const long long tasks = (long long)total * 2 * a.Hkv;
    const int col = lane % kLanes, row_l = lane / kLanes;
    for (long long task = (long long)blockIdx.x * kScaledWarps + (tid >> 5); task < tasks;
         task += (long long)gridDim.x * kScaledWarps) {
        const int u = (int)(task / (2 * a.Hkv)), rest = (int)(task - (long long)u * (2 * a.Hkv));
        const int kv = rest >= a.Hkv, h = kv ? rest - a.Hkv : rest;
        int lo = 0, hi = R - 1;              // the last request with s_first[r] <= u
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (s_first[mid] <= u) lo = mid;
            else hi = mid - 1;
        }
        // Starts that go back and forth can add up past 32 bits, and the search
        // then end anywhere: nothing but a block of this request goes on.
        const int j = u - s_first[lo];
        if (j < 0 || j >= blocks_of(lo, false)) continue;
        const int q0 = a.qsl[lo], L = a.seq_lens[lo], p0 = L - (a.qsl[lo + 1] - q0);
        const int logical = p0 / kPage + j;
        const int first = max(p0, logical * kPage);              // first new position here
        const int cnt = min(L, logical * kPage + kPage) - first; // new rows here
        const int off = first - logical * kPage;                 // slots held by earlier tokens
        if (logical >= a.MB) {
            if (lane == 0) flag(a.status, PA_CHECK_LOGICAL_BLOCK);
            continue;
        }
        const int blk = a.bt[(long long)lo * a.MB + logical];
        const T *src = static_cast<const T *>(kv ? a.value : a.key) +
                       (long long)(q0 + first - p0) * a.stride + h * D + col * 8;
        uint4 x[kIters];
#pragma unroll
        for (int i = 0; i < kIters; ++i) {
            const int row = i * kRows + row_l;
            x[i] = make_uint4(0u, 0u, 0u, 0u);
            if (row < cnt) x[i] = __ldg(reinterpret_cast<const uint4 *>(src + row * a.stride));
        }
        if (blk < 0 || blk >= a.NB) {
            if (lane == 0) flag(a.status, PA_CHECK_BLOCK_ID);
            continue;
        }
        uint8_t *scale = (kv ? a.v_scales : a.k_scales) + (long long)blk * a.Hkv + h;
        const int old = off > 0 ? (int)*scale : 0;
        uint32_t mx = 0;
#pragma unroll
        for (int i = 0; i < kIters; ++i) {
            const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t m = w[e] & 0x7fff7fffu;
                mx = __vmaxu2(mx, m & ~__vcmpgeu2(m, Mag<T>::kInf2));
            }
        }
        mx = __reduce_max_sync(0xffffffffu, max(mx & 0xffffu, mx >> 16));
        int e = scale_exponent(Mag<T>::value(mx));
        uint8_t *dst = (kv ? a.vc : a.kc) + ((long long)blk * kPage * a.Hkv + h) * D + col * 8;
        const int pitch = a.Hkv * D;         // bytes from one slot to the next
        if (off > 0) {
            const int e_old = clamp_scale(old) - kScaleBias;
            if (e > e_old) {
                const float mul = pow2f(e_old - e);
                for (int row = row_l; row < off; row += kRows) {
                    uint2 *c = reinterpret_cast<uint2 *>(dst + (long long)row * pitch);
                    *c = recode8(*c, mul);
                }
            } else {
                e = e_old;
            }
        }
        const float mul = pow2f(-e);
#pragma unroll
        for (int i = 0; i < kIters; ++i) {
            const int row = i * kRows + row_l;
            if (row < cnt)
                *reinterpret_cast<uint2 *>(dst + (long long)(off + row) * pitch) =
                    quantize8_pow2<T>(x[i], mul);
        }
        if (lane == 0) *scale = (uint8_t)(e + kScaleBias);
    }
}

// ---------------------------------------------------------------------------
// Read
// ---------------------------------------------------------------------------

// One warp per run of consecutive rows of the output: its lanes find the rows'
// requests (a search 32 probes wide in row_start_loc, then one step per row)
// and slots side by side, then walk the rows' 8-element units 32 at a time, K
// and V together.  HBM-bound: 3 bytes an element from FP8 pools, two of them
// written.  Two units of each in flight and six CTAs per SM, written with the
// streaming hint: 262,664 rows of 8 x 128 in 266 us (6.07 TB/s, 89% of the copy
// rate; four units and four CTAs 270, without the hint 273-276).
constexpr int kReadRows = 8;    // rows a warp takes at a time, at most
constexpr int kReadUnroll = 2;  // units of K and of V in flight per lane
constexpr int kReadCtasPerSm = 6;

// kPool 0: 16-bit pools (a copy); 1: E4M3 pools with one scale each; 2: E4M3
// pools with a scale per (block, kv head).  A unit is 8 elements.
template <typename T, int kPool>
__global__ void __launch_bounds__(kScaledThreads, kReadCtasPerSm) cache_read_kernel(const CacheReadArgs a) {
    using Src = typename std::conditional<kPool == 0, uint4, uint2>::type;
    const int lane = threadIdx.x & 31;
    const float ks = kPool == 1 && a.k_scale ? *a.k_scale : 1.f;
    const float vs = kPool == 1 && a.v_scale ? *a.v_scale : 1.f;
    const int R = a.R, nu = a.row / 8;
    const Src *kc = static_cast<const Src *>(a.kc), *vc = static_cast<const Src *>(a.vc);
    uint4 *ko = static_cast<uint4 *>(a.key_out), *vo = static_cast<uint4 *>(a.value_out);
    const int rows_in = a.row_starts[R];     // rows asked for
    if (blockIdx.x == 0 && threadIdx.x == 0 && (rows_in > a.N || rows_in < 0))
        flag(a.status, PA_CHECK_TOKEN_COUNT);
    const int rows_all = min(rows_in, a.N);
    const int per = a.rows_per_warp;
    const long long step = (long long)gridDim.x * kScaledWarps * per;
    for (long long t0 = ((long long)blockIdx.x * kScaledWarps + (threadIdx.x >> 5)) * per;
         t0 < rows_all; t0 += step) {
        const int rows = (int)min((long long)per, rows_all - t0);
        // The last request with row_starts[r] <= t0: 32 probes at a time.
        int lo = 0, n = R;                   // among requests lo .. lo + n - 1
        while (n > 1) {
            const int w = (n + 31) / 32;
            const int i = lo + lane * w;
            const unsigned below =
                __ballot_sync(0xffffffffu, lane * w < n && a.row_starts[min(i, R)] <= t0);
            const int k = below ? 31 - __clz(below) : 0;
            n = min(w, n - k * w);
            lo += k * w;
        }
        // Lane i: row t0 + i's request, position and slot.
        int slot = -1, blk = 0;
        if (lane < rows) {
            const int t = (int)t0 + lane;
            int r = lo, end = R - 1;
            if (r < end && a.row_starts[r + 1] <= t) {
                ++r;
                while (r < end) {
                    const int mid = (r + end + 1) >> 1;
                    if (a.row_starts[mid] <= t) r = mid;
                    else end = mid - 1;
                }
            }
            const int i = t - a.row_starts[r];
            const long long pos = (long long)a.first_pos[r] + i;
            if (i < 0 || pos < 0) {
                flag(a.status, PA_CHECK_SEQ_LEN);
            } else if (pos / a.bs >= a.MB) {
                flag(a.status, PA_CHECK_LOGICAL_BLOCK);
            } else {
                blk = a.bt[(long long)r * a.MB + pos / a.bs];
                if (blk < 0 || blk >= a.NB) {
                    flag(a.status, PA_CHECK_BLOCK_ID);
                    blk = 0;
                } else {
                    slot = blk * a.bs + (int)(pos % a.bs);
                }
            }
        }
        // The rows' units one after another, 32 lanes wide.
        int row = 0, u = lane;               // this lane's next unit: of row `row`
        while (u >= nu) {
            u -= nu;
            ++row;
        }
        const int units = rows * nu;
        for (int i0 = 0; i0 < units; i0 += 32 * kReadUnroll) {
            Src k[kReadUnroll], v[kReadUnroll];
            float kf[kReadUnroll], vf[kReadUnroll];
            long long to[kReadUnroll];       // unit of the output, -1: none
#pragma unroll
            for (int j = 0; j < kReadUnroll; ++j) {
                const int s = __shfl_sync(0xffffffffu, slot, row & (kReadRows - 1));
                const int b = __shfl_sync(0xffffffffu, blk, row & (kReadRows - 1));
                const bool have = i0 + 32 * j + lane < units && s >= 0;
                to[j] = have ? (t0 + row) * nu + u : -1;
                if (have) {
                    const long long from = (long long)s * nu + u;
                    k[j] = __ldg(kc + from);
                    v[j] = __ldg(vc + from);
                    if constexpr (kPool == 2) {
                        const long long g = (long long)b * a.Hkv + (u >> a.head_shift);
                        kf[j] = scale_value(__ldg(a.k_scales + g));
                        vf[j] = scale_value(__ldg(a.v_scales + g));
                    } else {
                        kf[j] = ks;
                        vf[j] = vs;
                    }
                }
                u += 32;
                while (u >= nu) {
                    u -= nu;
                    ++row;
                }
            }
#pragma unroll
            for (int j = 0; j < kReadUnroll; ++j) {
                if (to[j] < 0) continue;
                if constexpr (kPool == 0) {
                    __stcs(ko + to[j], k[j]);
                    __stcs(vo + to[j], v[j]);
                } else {
                    __stcs(ko + to[j], dequantize8<T>(k[j], kf[j]));
                    __stcs(vo + to[j], dequantize8<T>(v[j], vf[j]));
                }
            }
        }
    }
}

// Copy-on-write of blocks takes their scales along: Hkv bytes of each pool's
// table per pair.
__global__ void __launch_bounds__(kScaledThreads)
copy_scales_kernel(uint8_t *__restrict__ ks, uint8_t *__restrict__ vs, int32_t Hkv, int32_t NB,
                   const int32_t *__restrict__ src, const int32_t *__restrict__ dst, int64_t n) {
    const int64_t stride = (int64_t)gridDim.x * blockDim.x;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += stride) {
        const int64_t pair = i / Hkv, h = i % Hkv;
        const int32_t s = src[pair], d = dst[pair];
        if (s < 0 || s >= NB || d < 0 || d >= NB) continue;   // the block copy flags it
        ks[(int64_t)d * Hkv + h] = ks[(int64_t)s * Hkv + h];
        vs[(int64_t)d * Hkv + h] = vs[(int64_t)s * Hkv + h];
    }
}

template <typename T>
pa_status launch_read(const CacheReadArgs &a, int pool, int blocks, cudaStream_t stream) {
    if (pool == 0) cache_read_kernel<T, 0><<<blocks, kScaledThreads, 0, stream>>>(a);
    else if (pool == 1) cache_read_kernel<T, 1><<<blocks, kScaledThreads, 0, stream>>>(a);
    else cache_read_kernel<T, 2><<<blocks, kScaledThreads, 0, stream>>>(a);
    PA_TRY_CUDA(cudaGetLastError());
    note_launch();
    return PA_OK;
}

}  // namespace

pa_status launch_cache_write_scaled(ScaledWriteArgs a, int32_t D, pa_dtype dtype,
                                    cudaStream_t stream) {
    if (a.T == 0 || a.R == 0) return PA_OK;
    if (a.R > kScaledMaxReqs) return PA_ERR_UNSUPPORTED;
    a.status = status_word();
    if (!a.status) return PA_ERR_CUDA;
    const size_t smem = ((size_t)a.R + 1) * sizeof(int32_t);
    auto kernel = dtype == PA_BF16 ? (D == 128 ? cache_write_scaled_kernel<__nv_bfloat16, 128>
                                               : cache_write_scaled_kernel<__nv_bfloat16, 64>)
                                   : (D == 128 ? cache_write_scaled_kernel<__half, 128>
                                               : cache_write_scaled_kernel<__half, 64>);
    if (smem > 48 * 1024)
        PA_TRY_CUDA(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)smem));
    // A request of n tokens writes at most (n + 14) / 16 + 1 blocks, and n.
    const long long units =
        min((long long)a.T, ((long long)a.T + 14LL * a.R) / kPage + a.R);
    long long blocks = (units * 2 * a.Hkv + kScaledWarps - 1) / kScaledWarps;
    const long long cap = 4LL * num_sms();   // one wave
    if (blocks > cap) blocks = cap;
    kernel<<<(int)blocks, kScaledThreads, smem, stream>>>(a);
    PA_TRY_CUDA(cudaGetLastError());
    note_launch();
    return PA_OK;
}

pa_status launch_cache_read(CacheReadArgs a, int pool, pa_dtype dtype, cudaStream_t stream) {
    if (a.N == 0 || a.R == 0) return PA_OK;
    a.status = status_word();
    if (!a.status) return PA_ERR_CUDA;
    // Few rows: fewer a warp, down to one, until they fill the GPU once.
    const long long cap = (long long)kReadCtasPerSm * num_sms();
    a.rows_per_warp = kReadRows;
    while (a.rows_per_warp > 1 && (long long)a.N < cap * kScaledWarps * a.rows_per_warp) a.rows_per_warp /= 2;
    const int per_block = a.rows_per_warp * kScaledWarps;
    long long blocks = ((long long)a.N + per_block - 1) / per_block;
    if (blocks > cap) blocks = cap;
    return dtype == PA_BF16 ? launch_read<__nv_bfloat16>(a, pool, (int)blocks, stream)
                            : launch_read<__half>(a, pool, (int)blocks, stream);
}

pa_status launch_copy_scales(uint8_t *k_scales, uint8_t *v_scales, int32_t Hkv, int32_t NB,
                             const int32_t *src, const int32_t *dst, int32_t n,
                             cudaStream_t stream) {
    if (n == 0) return PA_OK;
    const int64_t items = (int64_t)n * Hkv;
    int64_t blocks = (items + kScaledThreads - 1) / kScaledThreads;
    const int64_t cap = 8LL * num_sms();
    if (blocks > cap) blocks = cap;
    copy_scales_kernel<<<(int)blocks, kScaledThreads, 0, stream>>>(k_scales, v_scales, Hkv, NB, src,
                                                                   dst, items);
    PA_TRY_CUDA(cudaGetLastError());
    note_launch();
    return PA_OK;
}

}  // namespace pa
