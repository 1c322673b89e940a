// bd_fp8.hip -- 8-bit floating point (FP8) base weights and tokens: quantisation,
// dequantisation, the RMS norm that leaves its output in both forms a layer's products read,
// and the base products Y = X Wq^T.
//
// Codes are OCP e4m3 (sign, 4 exponent bits of bias 7, 3 mantissa bits; largest 448), one
// byte per element, row-major.  A weight has one fp32 scale per block of 128 x 128,
// [ceil(rows / 128)][ceil(cols / 128)]; tokens have one power of two 2^E per 128 columns of
// a row, the byte E + 127 (255: NaN), in rows of 4 ceil(cols / 512) bytes with zeros past the last block, so that the scales
// of any 512 columns are one aligned dword.
#include "bd_fp8.h"
#include "bd_fp8_plan.h"
#include "bd_tiles.h"

#include <type_traits>

namespace bd {
namespace {

typedef float f32x2 __attribute__((ext_vector_type(2)));
// 16 bytes at any element of y
typedef u32x4 u32x4_a2 __attribute__((aligned(2)));
typedef u32x4 u32x4_a4 __attribute__((aligned(4)));

// Eight consecutive columns as fp32.
__device__ __forceinline__ void load8(const uint16_t* p, float* f) {
    const u32x4 v = *(const u32x4*)p;
    f[0] = bf16_lo(v.x), f[1] = bf16_hi(v.x), f[2] = bf16_lo(v.y), f[3] = bf16_hi(v.y);
    f[4] = bf16_lo(v.z), f[5] = bf16_hi(v.z), f[6] = bf16_lo(v.w), f[7] = bf16_hi(v.w);
}
__device__ __forceinline__ void load4(const float* p, float* f) {
    const f32x4 a = *(const f32x4*)p;
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = a[i];
}
__device__ __forceinline__ void load8(const float* p, float* f) {
    load4(p, f);
    load4(p + 4, f + 4);
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {  // v_cvt_pk_bf16_f32: nearest even
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2){a, b}, bf16x2));
}
// Stores past the caches' usual ways: outputs of a whole matrix, read much later (bf16: 4096 x
// 14336 quantised with its values 63.1 -> 56.6 us, dequantised 31.8 -> 27.7)
__device__ __forceinline__ void store8_far(uint16_t* p, const float* f) {
    __builtin_nontemporal_store(
        u32x4{pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7])}, (u32x4*)p);
}
// (fp32: four values a lane, so that 16 lanes store whole lines; two such pieces a lane, half
// lines each, took 87 us for 4096 x 14336 against 58 with plain stores and 41 in this form)
__device__ __forceinline__ void store4_far(float* p, const float* f) {
    __builtin_nontemporal_store(f32x4{f[0], f[1], f[2], f[3]}, (f32x4*)p);
}
// The residual stream, which the layer's next norm reads: bf16 past the caches (512 x 4096 6.5
// -> 5.5 us, 8192 x 8192 108 -> 104), fp32, in half lines, plainly (91 against 103 us for 8192 x 4096).
__device__ __forceinline__ void store8_keep(uint16_t* p, const float* f) { store8_far(p, f); }
__device__ __forceinline__ void store8_keep(float* p, const float* f) {
    *(f32x4*)p = f32x4{f[0], f[1], f[2], f[3]};
    *(f32x4*)(p + 4) = f32x4{f[4], f[5], f[6], f[7]};
}

// What four (eight) codes stand for.
__device__ __forceinline__ void widen4(uint32_t c, float scale, float* f) {
    const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)c, false), b = __builtin_amdgcn_cvt_pk_f32_fp8((int)c, true);
    f[0] = a.x * scale, f[1] = a.y * scale, f[2] = b.x * scale, f[3] = b.y * scale;
}
__device__ __forceinline__ void widen8(u32x2 c, float scale, float* f) {
    widen4(c.x, scale, f);
    widen4(c.y, scale, f + 4);
}

// The largest over the 16 lanes that share a block of 128 columns.
__device__ __forceinline__ uint32_t max16(uint32_t a) {
#pragma unroll
    for (int d = 1; d < 16; d *= 2) a = umax(a, (uint32_t)__shfl_xor((int)a, d));
    return a;
}

constexpr int kQuantThreads = 256;

}  // namespace

// Tokens: E = the least with max |x| <= 448 2^E, codes = e4m3(x 2^-E), both exact but for the
// codes' one rounding.  16 lanes per block of 128 columns, 8 columns a lane; unit q is block
// q % nb of row q / nb, so that short rows leave no lane idle.  Bound by HBM (3 bytes an element
// of bf16): 512 x 14336 in 6.9 us (22 MB), 8192 x 5120 in 27.4 (4.6 TB/s), one row in 2.9, the
// launch.  One unit a lane and no more: two or four held at once took 0.4 to 1.5 us longer on up
// to 64 tokens and gained nothing on 8192.  The codes stay in the caches for the products.
template <typename XT>
__global__ void __launch_bounds__(kQuantThreads)
k_fp8_tokens(const XT* __restrict__ x, int64_t units, uint32_t nb, int64_t cols, uint8_t* __restrict__ codes,
             uint8_t* __restrict__ scales) {
    const int l = threadIdx.x & 15;
    const uint32_t ld = (nb + 3) / 4 * 4;
    for (int64_t q = (int64_t)blockIdx.x * (kQuantThreads / 16) + (threadIdx.x >> 4); q < units;
         q += (int64_t)gridDim.x * (kQuantThreads / 16)) {
        const int64_t row = units < ((int64_t)1 << 32) ? (int64_t)((uint32_t)q / nb) : q / nb;
        const uint32_t b = (uint32_t)(q - row * nb);
        const int64_t col = 128 * (int64_t)b + 8 * l;
        float f[8] = {};
        if (col < cols) load8(x + row * cols + col, f);
        const uint32_t byte = fp8_scale_byte(max16(amax8(f)), 0u);
        // the last block's lanes also write the zeros up to the stride
        if (l == 0) scales[row * ld + b] = (uint8_t)byte;
        else if (b == nb - 1 && b + l < ld) scales[row * ld + b + l] = 0;
        if (col < cols)
            *(u32x2*)(codes + row * cols + col) = byte == 255u ? u32x2{0u, 0u} : codes8(f, fp8_inverse(byte));
    }
}

// Weights: one thread block per block of 128 x 128, which it holds in registers between its
// maximum and its codes (16 lanes a row, 8 rows a thread; a lane takes 8 columns of bf16, or 4
// of fp32 and 4 that are 64 on, so that lanes next to each other read and write whole lines).
// `values` (may be null, may be w itself: a thread reads its columns before it writes them)
// receives what the codes stand for.  Bound by HBM: 4096 x 14336 of bf16 with its values in 56
// us (294 MB, 5.2 TB/s), of fp32 in 99 (528 MB).  A block per 128 x 512, 1024 threads, was slower.
template <typename WT>
__global__ void __launch_bounds__(256)
k_fp8_weights(const WT* w, int64_t rows, int64_t cols, uint32_t nb, uint8_t* __restrict__ codes,
              float* __restrict__ scales, WT* values) {
    constexpr bool F = sizeof(WT) == 4;
    __shared__ uint32_t red[4];
    const int64_t br = blockIdx.x / nb;
    const uint32_t bc = blockIdx.x - (uint32_t)br * nb;
    const int64_t col = 128 * (int64_t)bc + (F ? 4 : 8) * (threadIdx.x & 15);
    const int64_t row0 = 128 * br + (threadIdx.x >> 4);
    const bool on = col < cols, on2 = F && col + 64 < cols;
    float f[8][8] = {};
    uint32_t a = 0u;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const WT* const p = w + (row0 + 16 * k) * cols + col;
        if (!on || row0 + 16 * k >= rows) continue;
        if constexpr (F) {
            load4(p, f[k]);
            if (on2) load4(p + 64, f[k] + 4);
        } else {
            load8(p, f[k]);
        }
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) a = umax(a, amax8(f[k]));
    a = max16(a);
    a = umax(a, (uint32_t)__shfl_xor((int)a, 16));
    a = umax(a, (uint32_t)__shfl_xor((int)a, 32));
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = a;
    __syncthreads();
    a = umax(umax(red[0], red[1]), umax(red[2], red[3]));
    const uint32_t byte = fp8_scale_byte(a, 1u);
    const float scale = byte == 255u ? __uint_as_float(0x7FC00000u) : fp8_scale(byte);
    if (threadIdx.x == 0) scales[br * nb + bc] = scale;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const int64_t row = row0 + 16 * k;
        if (!on || row >= rows) continue;
        const int64_t at = row * cols + col;
        const u32x2 c = byte == 255u ? u32x2{0u, 0u} : codes8(f[k], fp8_inverse(byte));
        float v[8];
        if (values) widen8(c, scale, v);
        if constexpr (F) {
            __builtin_nontemporal_store(c.x, (uint32_t*)(codes + at));
            if (on2) __builtin_nontemporal_store(c.y, (uint32_t*)(codes + at + 64));
            if (values) {
                store4_far(values + at, v);
                if (on2) store4_far(values + at + 64, v + 4);
            }
        } else {
            __builtin_nontemporal_store(c, (u32x2*)(codes + at));
            if (values) store8_far(values + at, v);
        }
    }
}

// out = code * scale, one rounding to fp32 (and one more to bf16): 8 columns of bf16, or 4 of
// fp32, a thread and turn (16 bytes of output).  Bound by HBM: 17408 x 5120 to bf16 in 45 us
// (267 MB, 5.9 TB/s), 4096 x 14336 to fp32 in 41 (294 MB), 1024 x 4096 to fp32 in 4.7 (21 MB).
template <typename OT>
__global__ void __launch_bounds__(kQuantThreads)
k_fp8_dequantize(const uint8_t* __restrict__ codes, const float* __restrict__ scales, int64_t chunks,
                 uint32_t per_row, uint32_t nb, OT* __restrict__ out) {
    constexpr bool F = sizeof(OT) == 4;
    for (int64_t q = (int64_t)blockIdx.x * kQuantThreads + threadIdx.x; q < chunks;
         q += (int64_t)gridDim.x * kQuantThreads) {
        const int64_t row = chunks < ((int64_t)1 << 32) ? (int64_t)((uint32_t)q / per_row) : q / per_row;
        const uint32_t c = (uint32_t)(q - row * per_row);
        const float scale = scales[(row >> 7) * nb + (c >> (F ? 5 : 4))];
        float f[8];
        if constexpr (F) {
            widen4(*(const uint32_t*)(codes + 4 * q), scale, f);
            store4_far(out + 4 * q, f);
        } else {
            widen8(*(const u32x2*)(codes + 8 * q), scale, f);
            store8_far(out + 8 * q, f);
        }
    }
}

// RMS norm of h + r (or of h): one thread block per row, 8 columns a thread and turn, the row
// in registers between its sum of squares and its output (V turns).  The sum s is rounded to
// h's type first and the norm is that of the stored value, so that the call equals an
// addition and a norm one after the other; x = s rsqrt(mean s^2 + eps) g in fp32, rounded to
// bf16 once; the codes are those of the rounded x (k_fp8_tokens).  A thread reads its columns of
// h and r before it writes them, so that h_out may be either.  Rows whose squares leave fp32's
// range (beyond 1e-15 or 1e19) are scaled by a power of two first.  Bound by HBM, one pass: 8192 x
// 5120 of bf16 with an fp32 residual in 81 us (462 MB, 5.7 TB/s); one row of 4096 in 3.1 us,
// where the sum across the block's waves is what there is to wait for.
template <typename HT, int V>
__global__ void __launch_bounds__(1024)
k_rmsnorm_fp8(const HT* h, const void* r, int r_bf16, const void* __restrict__ g, int g_bf16,
              int d, float eps, HT* h_out, uint16_t* __restrict__ x, uint8_t* __restrict__ codes,
              uint8_t* __restrict__ scales) {
    __shared__ float red[16];
    const int nt = (int)blockDim.x, tid = (int)threadIdx.x;
    const int64_t row = (int64_t)blockIdx.x * d;
    float f[V][8];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int col = 8 * (v * nt + tid);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[v][i] = 0.f;
        if (col < d) load8(h + row + col, f[v]);
    }
    if (r) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int col = 8 * (v * nt + tid);
            if (col >= d) continue;
            float a[8];
            if (r_bf16) load8((const uint16_t*)r + row + col, a);
            else load8((const float*)r + row + col, a);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                f[v][i] += a[i];
                if constexpr (sizeof(HT) == 2) f[v][i] = (float)(__bf16)f[v][i];
            }
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int col = 8 * (v * nt + tid);
            if (col < d) store8_keep(h_out + row + col, f[v]);
        }
    }
    auto squares = [&]() {  // of the row, the same in every thread
        float sum = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int i = 0; i < 8; ++i) sum += f[v][i] * f[v][i];
#pragma unroll
        for (int m = 1; m < 64; m *= 2) sum += __shfl_xor(sum, m);
        if ((tid & 63) == 0) red[tid >> 6] = sum;
        __syncthreads();
        sum = red[0];
        for (int w = 1; w < nt / 64; ++w) sum += red[w];
        return sum;
    };
    const float sum = squares();
    float ms = sum / (float)d + eps;
    // Squares that left fp32's range (a sum under 2^-100 may lack those under 2^-126): the row
    // again in units of 2^k, k the exponent of its largest magnitude or of sqrt(eps).  (uniform)
    if (sum < 0x1p-100f || !(sum < INFINITY) || !(ms < INFINITY)) {
        uint32_t a = 0u;
#pragma unroll
        for (int v = 0; v < V; ++v) a = umax(a, amax8(f[v]));
#pragma unroll
        for (int m = 1; m < 64; m *= 2) a = umax(a, (uint32_t)__shfl_xor((int)a, m));
        __syncthreads();
        if ((tid & 63) == 0) red[tid >> 6] = __uint_as_float(a);
        __syncthreads();
        for (int w = 0; w < nt / 64; ++w) a = umax(a, __float_as_uint(red[w]));
        if ((a | __float_as_uint(eps)) != 0u && a < 0x7F800000u) {  // (0 / 0, Inf and NaN stay what they are)
            int e = -2 * 149, k = e;
            if (a != 0u) (void)frexpf(__uint_as_float(a), &k);
            if (eps != 0.f) (void)frexpf(eps, &e);
            e = (e + 1) >> 1;
            k = e > k ? e : k;
#pragma unroll
            for (int v = 0; v < V; ++v)
#pragma unroll
                for (int i = 0; i < 8; ++i) f[v][i] = ldexpf(f[v][i], -k);
            __syncthreads();
            ms = squares() / (float)d + ldexpf(eps, -2 * k);
        }
    }
    const float rstd = rsqrtf(ms);
    const int nb = (d + 127) / 128, ld = (d + 511) / 512 * 4;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int col = 8 * (v * nt + tid);
        float o[8] = {};
        if (col < d) {
            float w[8];
            if (g_bf16) load8((const uint16_t*)g + col, w);
            else load8((const float*)g + col, w);
            uint32_t p[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                p[i] = pack_bf16(f[v][2 * i] * rstd * w[2 * i], f[v][2 * i + 1] * rstd * w[2 * i + 1]);
                o[2 * i] = bf16_lo(p[i]), o[2 * i + 1] = bf16_hi(p[i]);
            }
            *(u32x4*)(x + row + col) = u32x4{p[0], p[1], p[2], p[3]};
        }
        // (nt is a multiple of 64: the 16 lanes of a block of 128 columns are in one wave)
        const uint32_t byte = fp8_scale_byte(max16(amax8(o)), 0u);
        const int b = (v * nt + tid) >> 4;
        if ((tid & 15) == 0 && b < ld) scales[(int64_t)blockIdx.x * ld + b] = b < nb ? (uint8_t)byte : 0;
        if (col < d) *(u32x2*)(codes + row + col) = byte == 255u ? u32x2{0u, 0u} : codes8(o, fp8_inverse(byte));
    }
}

namespace {

unsigned grid_of(int64_t n, int per) {
    const int64_t b = (n + per - 1) / per;
    return (unsigned)(b < 65536 ? b : 65536);
}

}  // namespace

hipError_t launch_fp8_tokens(const void* x, int dtype, int64_t rows, int64_t cols, uint8_t* codes,
                             uint8_t* scales, hipStream_t s) {
    if (rows == 0) return hipSuccess;
    const uint32_t nb = (uint32_t)((cols + 127) / 128);
    const int64_t units = rows * nb;
    const dim3 grid(grid_of(units, kQuantThreads / 16)), block(kQuantThreads);
    if (dtype == BD_BF16)
        k_fp8_tokens<uint16_t><<<grid, block, 0, s>>>((const uint16_t*)x, units, nb, cols, codes, scales);
    else
        k_fp8_tokens<float><<<grid, block, 0, s>>>((const float*)x, units, nb, cols, codes, scales);
    return hipGetLastError();
}

hipError_t launch_fp8_weights(const void* w, int dtype, int64_t rows, int64_t cols, uint8_t* codes,
                              float* scales, void* values, hipStream_t s) {
    if (rows == 0) return hipSuccess;
    const uint32_t nb = (uint32_t)((cols + 127) / 128);
    const dim3 grid((unsigned)((rows + 127) / 128 * nb)), block(256);
    if (dtype == BD_BF16)
        k_fp8_weights<uint16_t><<<grid, block, 0, s>>>((const uint16_t*)w, rows, cols, nb, codes, scales,
                                                       (uint16_t*)values);
    else
        k_fp8_weights<float><<<grid, block, 0, s>>>((const float*)w, rows, cols, nb, codes, scales,
                                                    (float*)values);
    return hipGetLastError();
}

hipError_t launch_fp8_dequantize(const uint8_t* codes, const float* scales, int64_t rows, int64_t cols,
                                 void* out, int odtype, hipStream_t s) {
    if (rows == 0) return hipSuccess;
    const uint32_t nb = (uint32_t)((cols + 127) / 128), per_row = (uint32_t)(cols / (odtype == BD_BF16 ? 8 : 4));
    const int64_t chunks = rows * per_row;
    const dim3 grid(grid_of(chunks, kQuantThreads)), block(kQuantThreads);
    if (odtype == BD_BF16)
        k_fp8_dequantize<uint16_t><<<grid, block, 0, s>>>(codes, scales, chunks, per_row, nb, (uint16_t*)out);
    else
        k_fp8_dequantize<float><<<grid, block, 0, s>>>(codes, scales, chunks, per_row, nb, (float*)out);
    return hipGetLastError();
}

hipError_t launch_rmsnorm_fp8(const void* h, int hdtype, const void* r, int rdtype, const void* g, int gdtype,
                              int64_t T, int64_t d, float eps, void* h_out, uint16_t* x, uint8_t* codes,
                              uint8_t* scales, hipStream_t s) {
    if (T == 0) return hipSuccess;
    const int64_t chunks = d / 8;
    const int V = chunks <= 1024 ? 1 : chunks <= 2048 ? 2 : 4;
    const int nt = (int)((chunks + V - 1) / V + 63) / 64 * 64;
    const dim3 grid((unsigned)T), block((unsigned)nt);
    const int rb = rdtype == BD_BF16, gb = gdtype == BD_BF16;
    auto go = [&](auto ht, auto vc) {
        using HT = decltype(ht);
        k_rmsnorm_fp8<HT, decltype(vc)::value><<<grid, block, 0, s>>>(
            (const HT*)h, r, rb, g, gb, (int)d, eps, (HT*)h_out, x, codes, scales);
    };
    auto by_v = [&](auto ht) {
        if (V == 1) go(ht, std::integral_constant<int, 1>());
        else if (V == 2) go(ht, std::integral_constant<int, 2>());
        else go(ht, std::integral_constant<int, 4>());
    };
    if (hdtype == BD_BF16) by_v(uint16_t());
    else by_v(float());
    return hipGetLastError();
}

// ------------------------------------------------------------------ base products

// The product for batches of at most 16 NT tokens: one thread block per 16 rows, wave w on
// columns 512 w .. 512 w + 511 and every 4096 after them, a unit's loads all at once, the
// eight partial tiles summed in LDS in wave order.  There is nothing to reuse at so few tokens:
// every byte of Wq goes from memory to the registers of the one wave that multiplies it, and
// the time is the latency of one such round beside the bytes' (1 token on 4096 + 1024 + 1024
// rows of 4096: 9.4 us for 25 MB, 5.2 at the rate of a large copy).
template <int NT>
__global__ void __launch_bounds__(64 * kRowsWaves)
k_fp8_rows(const uint8_t* __restrict__ x, const uint8_t* __restrict__ xs, const GemmMats gm, int T, int K,
           int y_bf16) {
    __shared__ f32x4 red[NT][kRowsWaves][64];
    const int lane = threadIdx.x & 63;
    const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int m = lane & 15, g = lane >> 4;
    const int nb = (K + 127) / 128, nu = (K + 511) / 512;
    BD_MAT_OF(mt, gm, (int)blockIdx.x);
    const int N = mt.N, r0 = 16 * ((int)blockIdx.x - mt.rt0);
    const __amdgpu_buffer_rsrc_t wr = make_rsrc_u32(mt.w, (uint32_t)N * (uint32_t)K);
    const __amdgpu_buffer_rsrc_t xr = make_rsrc_u32(x, (uint32_t)T * (uint32_t)K);
    const __amdgpu_buffer_rsrc_t er = make_rsrc_u32(xs, (uint32_t)(T * nu) * 4u);
    const scales_ptr ws = (scales_ptr)(uintptr_t)mt.s + (int64_t)(r0 / 128) * nb;
    f32x4 acc[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[j] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int u = wv; u < nu; u += kRowsWaves) {
        u32x4 W[4][2], X[NT][4][2];
        float sw[4];
        uint32_t xe[NT];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int col = 512 * u + 128 * q + 32 * g;
            const uint32_t ow = col < K && r0 + m < N ? (uint32_t)(r0 + m) * (uint32_t)K + (uint32_t)col : kOOB;
            W[q][0] = buf_load16(wr, ow), W[q][1] = buf_load16(wr, add_sat(ow, 16));
            const int b = 4 * u + q;
            sw[q] = ws[b < nb ? b : nb - 1];
        }
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const int t = 16 * j + m;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int col = 512 * u + 128 * q + 32 * g;  // (K is a multiple of 64: all 32 columns, or none)
                const uint32_t ox = col < K && t < T ? (uint32_t)t * (uint32_t)K + (uint32_t)col : kOOB;
                X[j][q][0] = buf_load16(xr, ox), X[j][q][1] = buf_load16(xr, add_sat(ox, 16));
            }
            xe[j] = buf_load4(er, t < T ? 4u * (uint32_t)(t * nu + u) : kOOB);
        }
        __builtin_amdgcn_sched_barrier(0);  // (every load before the first product)
        auto block = [&](auto qc) {
            constexpr int q = decltype(qc)::value;
            const Wide w = widen32(W[q][0], W[q][1]);
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const f32x4 p = mfma128(w, widen32(X[j][q][0], X[j][q][1]));
                const float f = product_scale<q>(sw[q], xe[j]);
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[j][e] = 4 * u + q < nb ? __builtin_fmaf(p[e], f, acc[j][e]) : acc[j][e];
            }
        };
        block(std::integral_constant<int, 0>());
        block(std::integral_constant<int, 1>());
        block(std::integral_constant<int, 2>());
        block(std::integral_constant<int, 3>());
    }
#pragma unroll
    for (int j = 0; j < NT; ++j) red[j][wv][lane] = acc[j];
    __syncthreads();
#pragma unroll
    for (int i = threadIdx.x; i < NT * 256; i += 64 * kRowsWaves) {
        const int t = i >> 4, r = i & 15;  // token, row
        if (t >= T || r0 + r >= N) continue;
        const int l = (t & 15) + 16 * (r >> 2);
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < kRowsWaves; ++w) v += ((const float*)&red[t >> 4][w][l])[r & 3];
        const int64_t at = (int64_t)t * N + r0 + r;
        if (y_bf16) ((uint16_t*)mt.y)[at] = f32_to_bf16(v);
        else mt.y[at] = v;
    }
}

// The product for larger batches: block tiles of BR rows of Wq x BT tokens, NWR x NWT waves,
// each a block of RI x TJ tiles of 16 x 16, a product of 128 columns at a time as four
// v_mfma_f32_16x16x32_bf16 on the codes widened to bf16 (mfma128: why not the FP8 instructions).
// A product's sums p are without scales; sw 2^E, the weight's scale (one per wave and 128
// columns: a wave's rows lie in one block of 128 rows) times the lane's token's, enters as
// acc = p (sw 2^E) + acc, the fma of a group of tiles issued one group later, when the matrix
// unit has left its result.
// K advances one block of 128 columns per stage (128 bytes of a row) through a ring of NS LDS
// stages filled by buffer loads that write LDS directly; 16-byte chunks are swizzled in their
// row so that 16 rows read at one chunk hit all banks.  A wave holds its tokens' operands of a
// stage in bf16 and reads its W rows 16 at a time, one row ahead of the products.  Behind the
// last read of a stage stands its one barrier: it frees the stage's slot, whose copies of stage
// s + NS go out from there on, and shows stage s + 1, whose token codes are read then and
// widened into the places of the operands that the products leave.
// Token scales come 512 columns (one dword a token) at a time into a ring of two slots.
// S > 1: K part sp covers columns [sp kps, (sp + 1) kps) (kps a multiple of 512) and writes
// its partial tile to part.
// H: y in bf16.  Row m of a pair of 16-row tiles is then row 8 (m / 4) + m % 4 (+ 4 for the
// second) of their 32, so that a lane ends up with 8 consecutive rows of its token and stores
// them as 16 bytes; the swizzle of W's chunks takes the bits by which 16 such rows differ.
//
// Large batches: the matrix unit at the bf16 rate and the vector instructions beside it.  On a
// wave's 64 x 64 a stage is 64 products (16 cycles each) and 232 vector instructions (4 each),
// 128 of them widen; the same mix run from registers alone, without LDS, reached 1600 TFLOP/s, a
// library's bf16 product 1391 to 1458.  8192 tokens on 14336 x 4096, fp32 out: 830 to 875 us,
// 1100 to 1160 TFLOP/s; 780 where the copies bring nothing from memory, 720 with the codes taken
// as they are (no widening).  Less ordering between the instructions or chains of one tile: within
// 2%; 128 x 128 on four waves, two blocks a CU: 960.  Wave tiles of 128 x 64 leave no registers for
// the widened operands.
// Middling batches: 1144 tokens on 5120 x 17408, 240 tiles of 256 x 192 in two K parts on 256
// CUs, 183 us (1110 TFLOP/s; as many of 128 x 192 over all of K 192, 160 of them without
// widening): 6 tiles of 192 tokens cover 1144 where 9 of 128 or 5 of 256 would leave a second
// round or a fifth of the work empty (128 x 256 221 us).
// Few tokens: the bytes of Wq.
template <int BR, int BT, int NS, int NWR, int NWT, bool H>
__global__ void __launch_bounds__(64 * NWR * NWT)
k_fp8_gemm(const uint8_t* __restrict__ x, const uint8_t* __restrict__ xsc, const GemmMats gm, int T, int K,
           int ntt, int S, int kps, int GR, int tiles) {
    constexpr int NW = NWR * NWT, RI = BR / NWR / 16, TJ = BT / NWT / 16, M = RI * TJ;
    constexpr int G = TJ % 2 == 0 ? 2 : TJ, NG = TJ / G;  // tiles of a group, groups of a row
    constexpr int kStage = (BR + BT) * 128, kSSlot = (BT < 64 ? 64 : BT) * 4;
    constexpr int kWInst = BR / 8 / NW, kXInst = BT / 8 / NW, kD = kWInst + kXInst;
    constexpr int kSI = (BT + 63) / 64;  // copies of a period's scales, a wave each (in turn)
    // copy c of a stage goes out with product at(c) behind the barrier that frees its slot; kPre
    // of them with the row of products there, the others with the next stage's
    constexpr auto at = [](int c) { return kD <= M ? c : c * M / kD; };
    constexpr int kPre = [] {
        int n = 0;
        for (int c = 0; c < kD; ++c) n += (kD <= M ? c : c * M / kD) < TJ ? 1 : 0;
        return n;
    }();
    constexpr int kStores = H ? M / 2 : M;
    static_assert(BR % (8 * NW) == 0 && BT % (8 * NW) == 0, "whole copy instructions per wave");
    static_assert(BR % (16 * NWR) == 0 && BT % (16 * NWT) == 0 && RI % 2 == 0 && G <= 3, "whole tiles");
    static_assert(128 % (BR / NWR) == 0, "a wave's rows share one scale");
    static_assert(NS >= 2 && NS <= 5, "a period's scales land before they are read");
    static_assert(kSI <= NW, "a wave copies one piece of the scales");
    static_assert((NS - 2) * kD + kPre + kStores < 64, "a count that s_waitcnt takes");
    extern __shared__ __attribute__((aligned(16))) char smem[];
    char* const sring = smem + NS * kStage;
    const int nb = (K + 127) / 128;
    const uint32_t ld = 4u * (uint32_t)((K + 511) / 512);
    const int lane = threadIdx.x & 63;
    const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wr = wv / NWT, wt = wv % NWT;
    const int m = lane & 15, g = lane >> 4;
    const __amdgpu_buffer_rsrc_t xss = make_rsrc_u32(xsc, (uint32_t)T * ld);

    // The tile whose copies go out.
    MatId mt;
    int r0, t0, sp, kcols, nk, nbl;
    scales_ptr wsc;
    uint32_t wsrc[kWInst], xsrc[kXInst], ssrc;
    // loader: instruction i of an operand fills rows 8 i .. 8 i + 7; lane l lands on row
    // 8 i + l / 8, slot l % 8, i.e. takes the chunk whose swizzled slot that is
    auto swz = [](int r) { return (r >> 1) & 7; };
    auto swzw = [&](int r) { return H ? ((r >> 1) & 1) | ((r >> 2) & 6) : swz(r); };
    const int si = wv % kSI;  // (a wave without scales of its own repeats another's)
    auto take = [&](int block) {  // false: no tile there
        const TileId tid = tile_id(block, tiles, gm.rt_begin[gm.n], ntt, S, GR);
        if (tid.rt >= gm.rt_begin[gm.n]) return false;  // uniform
        BD_MAT_OF(mm, gm, tid.rt);
        mt = mm;
        sp = tid.sp;
        r0 = (tid.rt - mt.rt0) * BR, t0 = tid.tt * BT;
        const int kbeg = sp * kps;
        kcols = K - kbeg < kps ? K - kbeg : kps;  // columns of this part
        nk = (kcols + 127) / 128;
        // this wave's weight scales, from the part's first column on, and the last of all
        const int first = (r0 + wr * (BR / NWR)) / 128 * nb + kbeg / 128;
        wsc = (scales_ptr)(uintptr_t)mt.s + first;
        nbl = (mt.N + 127) / 128 * nb - 1 - first;
#pragma unroll
        for (int j = 0; j < kWInst; ++j) {
            const int r = (wv * kWInst + j) * 8 + lane / 8;
            wsrc[j] = r0 + r < mt.N ? (uint32_t)(r0 + r) * (uint32_t)K + (uint32_t)(kbeg + 16 * ((lane & 7) ^ swzw(r))) : kOOB;
        }
#pragma unroll
        for (int j = 0; j < kXInst; ++j) {
            const int r = (wv * kXInst + j) * 8 + lane / 8;
            xsrc[j] = t0 + r < T ? (uint32_t)(t0 + r) * (uint32_t)K + (uint32_t)(kbeg + 16 * ((lane & 7) ^ swz(r))) : kOOB;
        }
        ssrc = 64 * si + lane < BT && t0 + 64 * si + lane < T
                   ? (uint32_t)(t0 + 64 * si + lane) * ld + (uint32_t)(kbeg / 128)
                   : kOOB;
        return true;
    };
    // Copy c of stage s's kD, into its ring slot, and of period p's scales (columns 512 p ..
    // + 511), into slot p % 2.  A part's last stage may have 64 columns: the lanes of the upper
    // four chunks are then out of bounds (they bring zeros), as all are behind it.
    const uint32_t up = (lane & 4) ? kOOB : 0u;  // slots 4..7: upper chunks where the swizzle's bit 2 is 0
    auto copy = [&](int s, int slot, int c) {
        char* base = smem + slot * kStage;
        const int left = kcols - 128 * s, adv = left > 0 ? 128 * s : 0;  // (uniform)
        const uint32_t half = left == 64 ? ~0u : 0u;
        if (c < kWInst) {
            const int i = wv * kWInst + c;
            const uint32_t cut = (((H ? i >> 1 : i) & 1) ? up ^ kOOB : up) & half;
            copy16_to_lds(make_rsrc_u32(mt.w, left > 0 ? (uint32_t)mt.N * (uint32_t)K : 0u), base + i * 1024, wsrc[c < kWInst ? c : 0] | cut, adv);
        } else {
            const int i = wv * kXInst + c - kWInst;
            const uint32_t cut = ((i & 1) ? up ^ kOOB : up) & half;
            copy16_to_lds(make_rsrc_u32(x, left > 0 ? (uint32_t)T * (uint32_t)K : 0u), base + BR * 128 + i * 1024, xsrc[c < kWInst ? 0 : c - kWInst] | cut, adv);
        }
    };
    auto copy_scales = [&](int p) {
        copy4_to_lds(xss, sring + (p & 1) * kSSlot + si * 256, add_sat(ssrc, 512 * p < kcols ? 4u * (uint32_t)p : kOOB));
    };
    // The first period's scales, NS - 1 stages and the copies of stage NS - 1 that the loop
    // would have sent with the last row of products before it.
    auto prologue = [&]() {
        copy_scales(0);
#pragma unroll
        for (int t = 0; t < NS - 1; ++t)
#pragma unroll
            for (int c = 0; c < kD; ++c) copy(t, t, c);
#pragma unroll
        for (int c = 0; c < kD; ++c)
            if (at(c) < TJ) copy(NS - 1, NS - 1, c);
    };

    // Lane m + 16 g takes a row's chunks g and g + 4, at off and off ^ 64, of both operands
    // (which columns a lane multiplies is free as long as both agree).  A 16-byte read serves
    // lanes of several g at a time: chunks 2 g and 2 g + 1 met 2-way bank conflicts in every
    // read (8 cycles a read against 4).
    const int off = m * 128 + 16 * (g ^ swz(m));
    const int mw = H ? 8 * (m >> 2) + (m & 3) : m;
    const int offw[2] = {mw * 128 + 16 * (g ^ swzw(mw)), H ? (mw + 4) * 128 + 16 * (g ^ swzw(mw + 4)) : off};
    f32x4 acc[RI][TJ];
    u32x4 A[2], Bv[TJ][2];  // codes: of the next 16 rows; of the next stage's tokens
    Wide AW, XW[TJ];        // ... and in bf16: of these rows, of this stage's tokens
    uint32_t xe[TJ];
    f32x4 P[2][G];
    float sw[4], f[TJ], fl[G];  // a period's weight scales; this stage's; those of the last group before it
    auto read_a = [&](int slot, int i) {
        const char* p = smem + slot * kStage + (wr * (BR / NWR) + (H ? i / 2 * 32 : 16 * i)) * 128;
        const int o = offw[i & 1];
        A[0] = *(const u32x4*)(p + o), A[1] = *(const u32x4*)(p + (o ^ 64));
    };
    auto read_b = [&](int slot, int j) {
        const char* p = smem + slot * kStage + (BR + wt * (BT / NWT) + 16 * j) * 128;
        Bv[j][0] = *(const u32x4*)(p + off), Bv[j][1] = *(const u32x4*)(p + (off ^ 64));
    };
    auto read_e = [&](int p, int j) {
        xe[j] = *(const uint32_t*)(sring + (p & 1) * kSSlot + (wt * (BT / NWT) + 16 * j + m) * 4);
    };
    auto read_sw = [&](int p) {
#pragma unroll
        for (int q = 0; q < 4; ++q) sw[q] = wsc[4 * p + q < nbl ? 4 * p + q : nbl];
    };
    // Columns 32 q .. of the operands (of the order in which the products take them)
    auto widen_a = [&](int q) {
        AW.q[q] = (q & 1) ? widen_bf16(A[q / 2].z, A[q / 2].w) : widen_bf16(A[q / 2].x, A[q / 2].y);
    };
    auto widen_x = [&](int j, int q) {
        XW[j].q[q] = (q & 1) ? widen_bf16(Bv[j][q / 2].z, Bv[j][q / 2].w) : widen_bf16(Bv[j][q / 2].x, Bv[j][q / 2].y);
    };
    // Stage s in slot `slot` (s % 4 == J), stage s + 1 in slot `next`.  A row of 16 goes through
    // the wave's tokens in groups of G tiles, each four products of 32 columns for the group's
    // tiles in turn.  Between them stand, a step at a time, what later ones need: the reads, the
    // copies, the widening of the next row's and the next group's operands into the registers
    // that the products leave, and the scaled sums of the group before.
    auto stage = [&](int s, int slot, int next, auto jc) {
        constexpr int J = decltype(jc)::value;
        const int prev = slot == 0 ? NS - 1 : slot - 1;  // the slot that stage s - 1 left
#pragma unroll
        for (int i = 0; i < RI; ++i) {
            if (i == RI - 1) {
                // the wave's reads of this stage are done; its copies of stage s + 1 have landed
                wait_vmcnt_lgkm<(NS - 2) * kD>();
                __builtin_amdgcn_s_barrier();
                if constexpr (J == 0) copy_scales(s / 4 + 1);
            }
#pragma unroll
            for (int gj = 0; gj < NG; ++gj) {
                const int pp = (i * NG + gj) & 1;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                    for (int h = 0; h < G; ++h) {
                        const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
                        P[pp][h] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(AW.q[q], XW[gj * G + h].q[q],
                                                                           q == 0 ? zero : P[pp][h], 0, 0, 0);
                    }
                    __builtin_amdgcn_sched_barrier(0);
                    if (q == 0) {
                        if (gj == 0) read_a(i == RI - 1 ? next : slot, (i + 1) % RI);
                        if (i == RI - 1) {
#pragma unroll
                            for (int h = 0; h < G; ++h) {
                                read_b(next, gj * G + h);
                                if constexpr (J == 3) read_e(s / 4 + 1, gj * G + h);
                            }
                        }
                    }
#pragma unroll
                    for (int h = 0; h < G; ++h) {
                        const int j = gj * G + h, n = i * TJ + j, k = i == RI - 1 ? j : n + TJ;  // this product, from the barrier on
                        if (q == (h == 0 ? 1 : 3)) {
#pragma unroll
                            for (int c = 0; c < kD; ++c)
                                if (at(c) == k) {
                                    if (i == RI - 1) copy(s + NS, slot, c);
                                    else copy(s - 1 + NS, prev, c);
                                }
                        }
                        // the group before: i * NG + gj - 1, at first the last of stage s - 1
                        if (q == 1 + h) {
                            const int o = (n + M - G) % M;
                            const float sc = i + gj == 0 ? fl[h] : f[o % TJ];
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                acc[o / TJ][o % TJ][e] = __builtin_fmaf(P[pp ^ 1][h][e], sc, acc[o / TJ][o % TJ][e]);
                        }
                        // the next group's tokens: in the first row this stage's, behind the last
                        // row's last group the next stage's
                        if (i == 0 && gj + 1 < NG) widen_x(j + G, q);
                        if (i == RI - 1 && gj == NG - 1 && NG > 1) widen_x(h, q);
                    }
                    if (gj == NG - 1 && NG > 1) widen_a(q);
                    if (NG == 1 && q == 3) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            widen_a(k);
#pragma unroll
                            for (int h = 0; h < G; ++h)
                                if (i == RI - 1) widen_x(h, k);
                        }
                    }
                    if (i + gj == 0 && q == 3) {
#pragma unroll
                        for (int j = 0; j < TJ; ++j) f[j] = product_scale<J>(sw[J], xe[j]);
                    }
                }
            }
        }
#pragma unroll
        for (int h = 0; h < G; ++h) fl[h] = f[TJ - G + h];
        if constexpr (J == 3) read_sw(s / 4 + 1);
    };
    // The finished tile at rows o0, tokens u0 of y [T][N]: lane m + 16 g holds token m of each
    // product's tile, rows 4 g .. 4 g + 3 (H: 8 g .. 8 g + 7 of a pair), one 16-byte piece.
    // Where rows are whole pieces (vec) exactly kStores stores, those outside y dropped by its
    // num_records; else pieces go where they fall, those across a row's end in their elements.
    auto store = [&](auto* y, int N, int o0, int u0, bool vec) {
        using YT = std::remove_reference_t<decltype(*y)>;
        constexpr int kStep = H ? 2 : 1, kE = 4 * kStep;
        YT* const yt = y + (int64_t)u0 * N;
        const uint32_t bytes = (uint32_t)(T - u0 < BT ? T - u0 : BT) * (uint32_t)N * (uint32_t)sizeof(YT);
        const __amdgpu_buffer_rsrc_t yr = make_rsrc_u32(yt, bytes);
#pragma unroll
        for (int j = 0; j < TJ; ++j) {
            const int t = wt * (BT / NWT) + 16 * j + m;
#pragma unroll
            for (int i = 0; i < RI; i += kStep) {
                const int o = o0 + wr * (BR / NWR) + 16 * i + kE * g;
                u32x4 v;
                if constexpr (H)
                    v = u32x4{pack_bf16(acc[i][j][0], acc[i][j][1]), pack_bf16(acc[i][j][2], acc[i][j][3]),
                              pack_bf16(acc[i + 1][j][0], acc[i + 1][j][1]),
                              pack_bf16(acc[i + 1][j][2], acc[i + 1][j][3])};
                else
                    v = __builtin_bit_cast(u32x4, acc[i][j]);
                if (vec) {
                    const uint32_t at = o < N && u0 + t < T ? ((uint32_t)t * (uint32_t)N + (uint32_t)o) * (uint32_t)sizeof(YT) : bytes;
                    __builtin_amdgcn_raw_buffer_store_b128(v, yr, (int)at, 0, 0);
                } else if (u0 + t < T) {
                    YT* const p = yt + (int64_t)t * N + o;
                    if (o + kE <= N) {
                        *(std::conditional_t<H, u32x4_a2, u32x4_a4>*)p = v;
                    } else {
#pragma unroll
                        for (int e = 0; e < kE - 1; ++e)
                            if (o + e < N) {
                                if constexpr (H) p[e] = (uint16_t)(v[e / 2] >> (16 * (e & 1)));
                                else p[e] = __uint_as_float(v[e]);
                            }
                    }
                }
            }
        }
    };

    int block = (int)blockIdx.x;
    while (block < tiles && !take(block)) block += (int)gridDim.x;
    if (block >= tiles) return;  // uniform
    prologue();
    wait_vmcnt<(NS - 2) * kD + kPre>();
    for (;;) {
        __builtin_amdgcn_s_barrier();
        read_sw(0);
#pragma unroll
        for (int j = 0; j < TJ; ++j) {
            read_b(0, j);
            read_e(0, j);
        }
        read_a(0, 0);
#pragma unroll
        for (int i = 0; i < RI; ++i)
#pragma unroll
            for (int j = 0; j < TJ; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int h = 0; h < G; ++h) P[1][h] = f32x4{0.f, 0.f, 0.f, 0.f}, fl[h] = 0.f;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            widen_a(q);
#pragma unroll
            for (int h = 0; h < G; ++h) widen_x(h, q);
        }
        int slot = 0;
        auto one = [&](int s, auto jc) {
            const int next = slot == NS - 1 ? 0 : slot + 1;
            stage(s, slot, next, jc);
            slot = next;
        };
        for (int s = 0; s < nk; s += 4) {  // (uniform branches)
            one(s, std::integral_constant<int, 0>());
            if (s + 1 < nk) one(s + 1, std::integral_constant<int, 1>());
            if (s + 2 < nk) one(s + 2, std::integral_constant<int, 2>());
            if (s + 3 < nk) one(s + 3, std::integral_constant<int, 3>());
        }
#pragma unroll
        for (int h = 0; h < G; ++h)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                acc[RI - 1][TJ - G + h][e] = __builtin_fmaf(P[1][h][e], fl[h], acc[RI - 1][TJ - G + h][e]);
        // The next tile's first copies go out before this tile's stores (the empty copies past
        // the end have landed, and every wave has read what it will).
        const MatId done = mt;
        const int o0 = r0, u0 = t0, part = sp;
        const bool vec = (done.N & (H ? 7 : 3)) == 0;  // (uniform) y's rows are 16-byte aligned
        do block += (int)gridDim.x;
        while (block < tiles && !take(block));
        const bool more = block < tiles;
        wait_vmcnt_lgkm<0>();
        if (more) {
            __builtin_amdgcn_s_barrier();
            prologue();
        }
        if constexpr (H) store((uint16_t*)done.y, done.N, o0, u0, vec);
        else store(S > 1 ? done.part + (int64_t)part * T * done.N : done.y, done.N, o0, u0, vec);
        if (!more) break;
        if (vec) wait_vmcnt<(NS - 2) * kD + kPre + kStores>();
        else wait_vmcnt<(NS - 2) * kD + kPre>();
    }
}

namespace {

// One launch of a tile: S K parts of kps columns (S == 1: all of K, straight into y).
struct Fp8Launch {
    const uint8_t *x, *xscales;
    int64_t T, d_in;
    const GemmMatArg* mats;
    const float* const* wscales;
    int n, S;
    int64_t kps;
    float* const* parts;
    bool bf16;
    hipStream_t s;
};

// Row tiles an XCD takes together: 8 from 8 token tiles on (its 32 blocks then share 8 + 4
// operand tiles: 8192 x 8192 at 8192 tokens, fp32 out, 966 to 995 us against 1005 with 4 and 1087
// with 1; 14336 x 4096 872 to 876, 869 and 897), else 1.
inline int fp8_row_group(int ntt) { return ntt >= 8 ? 8 : 1; }

template <int BR, int BT, int NS, int NWR, int NWT>
hipError_t launch_gemm(const Fp8Launch& l) {
    int rt = 0;
    const GemmMats gm = gemm_mats(l.mats, l.wscales, l.n, BR, l.parts, &rt);
    const int ntt = (int)((l.T + BT - 1) / BT), GR = fp8_row_group(ntt);
    const unsigned blocks = tile_grid(rt, ntt, l.S);
    constexpr int lds = NS * (BR + BT) * 128 + 2 * (BT < 64 ? 64 : BT) * 4;
    // as many blocks as the chip holds at a time, each taking every so many-th tile (a multiple
    // of 8 apart: all on its XCD)
    constexpr int kByLds = 160 * 1024 / lds, kByWaves = (BR / NWR * (BT / NWT) <= 2048 ? 16 : 8) / (NWR * NWT);
    constexpr unsigned kHold = 256 * (kByLds < kByWaves ? kByLds : kByWaves);
    const dim3 grid(blocks < kHold ? blocks : kHold), block(64 * NWR * NWT);
    if (l.bf16 && l.S == 1)
        k_fp8_gemm<BR, BT, NS, NWR, NWT, true><<<grid, block, lds, l.s>>>(
            l.x, l.xscales, gm, (int)l.T, (int)l.d_in, ntt, 1, (int)l.kps, GR, (int)blocks);
    else
        k_fp8_gemm<BR, BT, NS, NWR, NWT, false><<<grid, block, lds, l.s>>>(
            l.x, l.xscales, gm, (int)l.T, (int)l.d_in, ntt, l.S, (int)l.kps, GR, (int)blocks);
    return hipGetLastError();
}

}  // namespace

bool fp8_product_supported(int64_t T, int64_t d_in, int64_t d_out) {
    // (each size first: their products then stay inside 64 bits; 32-bit offsets, also those
    // of a tile's rows past the last, and of 256 tokens' outputs)
    return d_in % 64 == 0 && d_in <= ((int64_t)1 << 22) && d_out < ((int64_t)1 << 22) &&
           T < ((int64_t)1 << 20) && T * d_in < ((int64_t)1 << 31) && d_out * d_in < ((int64_t)1 << 31);
}

size_t fp8_product_bytes(int64_t T, int64_t d_in, const int64_t* d_outs, int n) {
    const Fp8Plan pl = plan_fp8(T, d_in, d_outs, n, true);
    if (pl.S == 1) return 0;
    size_t b = 0;
    for (int i = 0; i < n; ++i) b += align_up((size_t)pl.S * T * d_outs[i] * 4);
    return b;
}

hipError_t launch_fp8_product(const uint8_t* x, const uint8_t* xscales, int64_t T, int64_t d_in,
                              const GemmMatArg* mats, const float* const* wscales, int n, int ydtype,
                              char* ws, hipStream_t s) {
    if (n < 1 || n > kMaxMats) return hipErrorInvalidValue;
    if (T == 0) return hipSuccess;
    int64_t d_outs[kMaxMats], nmax = 0;
    for (int i = 0; i < n; ++i) {
        d_outs[i] = mats[i].d_out;
        nmax = d_outs[i] > nmax ? d_outs[i] : nmax;
    }
    const Fp8Plan pl = plan_fp8(T, d_in, d_outs, n, ws != nullptr);
    float* parts[kMaxMats] = {};
    size_t off = 0;
    for (int i = 0; i < n && pl.S > 1; ++i) {
        parts[i] = (float*)(ws + off);
        off += align_up((size_t)pl.S * T * d_outs[i] * 4);
    }
    const Fp8Launch l = {x, xscales, T, d_in, mats, wscales, n, pl.S, pl.kps,
                         pl.S > 1 ? parts : nullptr, ydtype == BD_BF16, s};
    hipError_t e;
    int rt = 0;
    switch (pl.tile) {
        case kRows: {
            const GemmMats gm = gemm_mats(mats, wscales, n, 16, l.parts, &rt);
            auto go = [&](auto nt) {
                k_fp8_rows<decltype(nt)::value><<<dim3((unsigned)rt), dim3(64 * kRowsWaves), 0, s>>>(
                    x, xscales, gm, (int)T, (int)d_in, l.bf16);
            };
            if (T <= 16) go(std::integral_constant<int, 1>());
            else if (T <= 32) go(std::integral_constant<int, 2>());
            else go(std::integral_constant<int, 4>());
            e = hipGetLastError();
            break;
        }
        case k256x192: e = launch_gemm<256, 192, 2, 2, 4>(l); break;
        case k256x128: e = launch_gemm<256, 128, 3, 4, 2>(l); break;
        case k128x256: e = launch_gemm<128, 256, 3, 2, 4>(l); break;
        case k128x192: e = launch_gemm<128, 192, 3, 2, 4>(l); break;
        case k128x128: e = launch_gemm<128, 128, 3, 2, 4>(l); break;
        case k64x128: e = launch_gemm<64, 128, 4, 2, 4>(l); break;
        case k128x64: e = launch_gemm<128, 64, 4, 4, 2>(l); break;
        case k64x64: e = launch_gemm<64, 64, 4, 2, 2>(l); break;
        case k128x32: e = launch_gemm<128, 32, 4, 4, 1>(l); break;
        default: e = launch_gemm<64, 32, 3, 2, 1>(l); break;
    }
    if (e != hipSuccess || pl.S == 1) return e;
    return launch_sum_parts(gemm_mats(mats, wscales, n, 16, parts, &rt), T, nmax, pl.S, ydtype, s);
}

}  // namespace bd
