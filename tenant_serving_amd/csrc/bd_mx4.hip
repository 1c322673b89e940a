// bd_mx4.hip -- microscaled 4-bit (MX4) base weights and tokens: quantisation,
// dequantisation and the base products Y = X Wq^T.
//
// A block of 32 consecutive columns of a row shares one power-of-two scale 2^E (the byte
// E + 127; 255 stands for NaN); its elements are e2m1 codes (0, .5, 1, 1.5, 2, 3, 4, 6
// and a sign), two per byte, the lower column in the low nibble.  Codes are row-major
// [rows][cols / 2]; a row of scales is padded with zeros to 16 ceil(cols / 512) bytes, so
// that the scales of any 512 columns are one aligned 16-byte piece.
#include "bd_internal.h"

namespace bd {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr uint32_t kOOB = 0x80000000u;  // buffer offset past num_records: the load returns 0

__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const void* base, uint64_t bytes) {
    const int nrec = bytes > 0x7FFFFFFFull ? 0x7FFFFFFF : (int)bytes;
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, nrec, 0x00020000);
}
__device__ __forceinline__ u32x4 buf_load16(__amdgpu_buffer_rsrc_t r, uint32_t off) {
    return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, (int)off, 0, 0));
}
__device__ __forceinline__ uint32_t buf_load1(__amdgpu_buffer_rsrc_t r, uint32_t off) {
    return (uint32_t)(uint8_t)__builtin_amdgcn_raw_buffer_load_b8(r, (int)off, 0, 0);
}

__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

// The scale byte of a block whose largest magnitude has the fp32 bits `a`: with a in
// [2^e, 2^(e+1)), E = e - 2 (the block's maximum lands on 4..8, saturating above 6),
// never under -127: byte = max(biased exponent - 2, 0).  A NaN or Inf in the block: 255.
__device__ __forceinline__ uint32_t mx4_scale_byte(uint32_t a) {
    const uint32_t eb = a >> 23;
    return eb == 255u ? 255u : eb > 2u ? eb - 2u : 0u;
}
// A scale byte as the fp32 operand of the conversions, which read only its exponent
// field (0: 2^-127, 255: NaN).
__device__ __forceinline__ float mx4_scale(uint32_t byte) { return __uint_as_float(byte << 23); }

// Eight codes (one dword, low nibble first) as four bf16 pairs, each code times the
// scale: exact (2 significant bits), Inf where the product leaves the range of bf16.
__device__ __forceinline__ u32x4 widen_mx4(uint32_t c, float scale) {
    u32x4 v;
    v.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 0));
    v.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 1));
    v.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 2));
    v.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 3));
    return v;
}

// Eight consecutive columns of a row, as loaded.
template <typename WT>
struct Cols8;
template <>
struct Cols8<uint16_t> {
    u32x4 v;
    __device__ __forceinline__ void load(const uint16_t* p) { v = *(const u32x4*)p; }
    __device__ __forceinline__ uint32_t amax() const {  // fp32 bits of the largest magnitude
        uint32_t m = 0u;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            m = umax(m, umax((v[i] << 16) & 0x7FFF0000u, v[i] & 0x7FFF0000u));
        return m;
    }
    __device__ __forceinline__ uint32_t codes(float scale) const {  // nearest even, saturating
        // (through scalars: this compiler's bit cast of a vector element reads element 0)
        const uint32_t p0 = v.x, p1 = v.y, p2 = v.z, p3 = v.w;
        uint32_t c = 0u;
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2, p0), scale, 0);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2, p1), scale, 1);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2, p2), scale, 2);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2, p3), scale, 3);
        return c;
    }
};
template <>
struct Cols8<float> {
    f32x4 a, b;
    __device__ __forceinline__ void load(const float* p) {
        a = *(const f32x4*)p;
        b = *(const f32x4*)(p + 4);
    }
    __device__ __forceinline__ uint32_t amax() const {
        uint32_t m = 0u;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            m = umax(m, umax(__float_as_uint(a[i]) & 0x7FFFFFFFu, __float_as_uint(b[i]) & 0x7FFFFFFFu));
        return m;
    }
    __device__ __forceinline__ uint32_t codes(float scale) const {
        uint32_t c = 0u;
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, a[0], a[1], scale, 0);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, a[2], a[3], scale, 1);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, b[0], b[1], scale, 2);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, b[2], b[3], scale, 3);
        return c;
    }
};
__device__ __forceinline__ void store_values(uint16_t* p, uint32_t c, float scale) {
    *(u32x4*)p = widen_mx4(c, scale);
}
__device__ __forceinline__ void store_values(float* p, uint32_t c, float scale) {
    const f32x2 v0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, scale, 0);
    const f32x2 v1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, scale, 1);
    const f32x2 v2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, scale, 2);
    const f32x2 v3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, scale, 3);
    *(f32x4*)p = f32x4{v0.x, v0.y, v1.x, v1.y};
    *(f32x4*)(p + 4) = f32x4{v2.x, v2.y, v3.x, v3.y};
}

constexpr int kQuantWaves = 4;

}  // namespace

// One wave per 512-column segment of a row: a lane holds 8 consecutive columns, four
// lanes one block.  `values` (may be null, may be w itself: a lane reads its columns
// before it writes them) receives what the codes stand for.
template <typename WT>
__global__ void __launch_bounds__(64 * kQuantWaves)
k_mx4_quantize(const WT* w, int64_t rows, int64_t cols, int64_t nseg, uint8_t* __restrict__ codes,
               uint8_t* __restrict__ scales, WT* values) {
    const int lane = threadIdx.x & 63;
    const int64_t total = rows * nseg;
    for (int64_t q = (int64_t)blockIdx.x * kQuantWaves + (threadIdx.x >> 6); q < total;
         q += (int64_t)gridDim.x * kQuantWaves) {
        const int64_t o = q / nseg, seg = q - o * nseg;
        const int64_t col = 512 * seg + 8 * lane;
        const bool in = col < cols;  // (cols % 32 == 0: a block's four lanes agree)
        Cols8<WT> v;
        uint32_t a = 0u;
        if (in) {
            v.load(w + o * cols + col);
            a = v.amax();
        }
        a = umax(a, (uint32_t)__shfl_xor((int)a, 1));
        a = umax(a, (uint32_t)__shfl_xor((int)a, 2));
        const uint32_t byte = mx4_scale_byte(a);
        if ((lane & 3) == 0) scales[(o * nseg + seg) * 16 + (lane >> 2)] = (uint8_t)byte;
        if (in) {
            const uint32_t c = byte == 255u ? 0u : v.codes(mx4_scale(byte));
            *(uint32_t*)(codes + (o * cols + col) / 2) = c;
            if (values) store_values(values + o * cols + col, c, mx4_scale(byte));
        }
    }
}

template <typename OT>
__global__ void __launch_bounds__(64 * kQuantWaves)
k_mx4_dequantize(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                 int64_t rows, int64_t cols, int64_t nseg, OT* __restrict__ out) {
    const int lane = threadIdx.x & 63;
    const int64_t total = rows * nseg;
    for (int64_t q = (int64_t)blockIdx.x * kQuantWaves + (threadIdx.x >> 6); q < total;
         q += (int64_t)gridDim.x * kQuantWaves) {
        const int64_t o = q / nseg, seg = q - o * nseg;
        const int64_t col = 512 * seg + 8 * lane;
        if (col >= cols) continue;
        const uint32_t c = *(const uint32_t*)(codes + (o * cols + col) / 2);
        store_values(out + o * cols + col, c, mx4_scale(scales[(o * nseg + seg) * 16 + (lane >> 2)]));
    }
}

// The product, one wave per 16 rows of Wq x 16 tokens, operands straight from memory.
// bf16 tokens (X4 = false): the codes are widened to bf16 (exact) and a lane's block of
// 32 columns feeds four v_mfma_f32_16x16x32_bf16, step j taking columns 8 j .. 8 j + 7 of
// every block.  MX4 tokens: one block-scaled 16x16x128 product per 128 columns.
template <bool X4>
__global__ void __launch_bounds__(64)
k_mx4_product(const void* __restrict__ x, const uint8_t* __restrict__ xs, const GemmMats gm, int T,
              int K) {
    const int lane = threadIdx.x;
    const int m = lane & 15, g = lane >> 4;
    const int rtg = (int)blockIdx.x;
    int mi = 0;
#pragma unroll
    for (int j = 1; j < kMaxMats; ++j) mi += (j < gm.n && rtg >= gm.rt_begin[j]) ? 1 : 0;
    const int N = gm.N[mi];
    const int r0 = 16 * (rtg - gm.rt_begin[mi]), t0 = 16 * (int)blockIdx.y;
    const uint32_t ld = 16u * (uint32_t)((K + 511) / 512);
    const __amdgpu_buffer_rsrc_t wr = make_rsrc(gm.w[mi], (uint64_t)N * K / 2);
    const __amdgpu_buffer_rsrc_t sr = make_rsrc(gm.s[mi], (uint64_t)N * ld);
    const __amdgpu_buffer_rsrc_t xr = make_rsrc(x, X4 ? (uint64_t)T * K / 2 : (uint64_t)T * K * 2);
    const __amdgpu_buffer_rsrc_t er = make_rsrc(xs, X4 ? (uint64_t)T * ld : 0);
    const bool okw = r0 + m < N, okx = t0 + m < T;
    const uint32_t wo = (uint32_t)(r0 + m) * (uint32_t)(K / 2), so = (uint32_t)(r0 + m) * ld;
    const uint32_t xo = (uint32_t)(t0 + m) * (uint32_t)(X4 ? K / 2 : 2 * K), eo = (uint32_t)(t0 + m) * ld;
    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
    for (int b = g; b - g < K / 32; b += 4) {  // this lane's block of 32 columns
        const bool ok = b < K / 32;
        const u32x4 c = buf_load16(wr, ok && okw ? wo + 16u * b : kOOB);
        const uint32_t s = buf_load1(sr, ok && okw ? so + b : kOOB);
        if constexpr (X4) {
            const u32x4 d = buf_load16(xr, ok && okx ? xo + 16u * b : kOOB);
            const uint32_t e = buf_load1(er, ok && okx ? eo + b : kOOB);
            const i32x8 a8 = {(int)c.x, (int)c.y, (int)c.z, (int)c.w, 0, 0, 0, 0};
            const i32x8 b8 = {(int)d.x, (int)d.y, (int)d.z, (int)d.w, 0, 0, 0, 0};
            acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a8, b8, acc, 4, 4, 0, (int)s, 0, (int)e);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const u32x4 d = buf_load16(xr, ok && okx ? xo + 64u * b + 16u * j : kOOB);
                acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                    __builtin_bit_cast(bf16x8, widen_mx4(c[j], mx4_scale(s))),
                    __builtin_bit_cast(bf16x8, d), acc, 0, 0, 0);
            }
        }
    }
    // D lane layout (16 x 16): column m (token), element e row 4 g + e
    if (!okx) return;
    float* const y = gm.y[mi] + (int64_t)(t0 + m) * N;
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (r0 + 4 * g + e < N) y[r0 + 4 * g + e] = acc[e];
}

namespace {

unsigned quant_blocks(int64_t rows, int64_t nseg) {
    const int64_t b = (rows * nseg + kQuantWaves - 1) / kQuantWaves;
    return (unsigned)(b < 65536 ? b : 65536);
}

}  // namespace

hipError_t launch_mx4_quantize(const void* w, int dtype, int64_t rows, int64_t cols, uint8_t* codes,
                               uint8_t* scales, void* values, hipStream_t s) {
    if (rows == 0) return hipSuccess;
    const int64_t nseg = (cols + 511) / 512;
    const dim3 grid(quant_blocks(rows, nseg)), block(64 * kQuantWaves);
    if (dtype == BD_BF16)
        k_mx4_quantize<uint16_t><<<grid, block, 0, s>>>((const uint16_t*)w, rows, cols, nseg, codes,
                                                        scales, (uint16_t*)values);
    else
        k_mx4_quantize<float><<<grid, block, 0, s>>>((const float*)w, rows, cols, nseg, codes,
                                                     scales, (float*)values);
    return hipGetLastError();
}

hipError_t launch_mx4_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows,
                                 int64_t cols, void* out, int odtype, hipStream_t s) {
    if (rows == 0) return hipSuccess;
    const int64_t nseg = (cols + 511) / 512;
    const dim3 grid(quant_blocks(rows, nseg)), block(64 * kQuantWaves);
    if (odtype == BD_BF16)
        k_mx4_dequantize<uint16_t><<<grid, block, 0, s>>>(codes, scales, rows, cols, nseg, (uint16_t*)out);
    else
        k_mx4_dequantize<float><<<grid, block, 0, s>>>(codes, scales, rows, cols, nseg, (float*)out);
    return hipGetLastError();
}

bool mx4_product_supported(bool x4, int64_t T, int64_t d_in, int64_t d_out) {
    return d_in % 64 == 0 && T * d_in * (x4 ? 1 : 4) < ((int64_t)1 << 32) &&
           d_out * d_in < ((int64_t)1 << 32) && d_out < ((int64_t)1 << 30) && T < ((int64_t)1 << 20);
}

size_t mx4_product_bytes(bool x4, int64_t T, int64_t d_in, const int64_t* d_outs, int n) {
    (void)x4, (void)T, (void)d_in, (void)d_outs, (void)n;
    return 0;
}

hipError_t launch_mx4_product(const void* x, const uint8_t* xscales, int64_t T, int64_t d_in,
                              const GemmMatArg* mats, const uint8_t* const* wscales, int n, char* ws,
                              hipStream_t s) {
    (void)ws;
    if (n < 1 || n > kMaxMats) return hipErrorInvalidValue;
    if (T == 0) return hipSuccess;
    GemmMats gm = {};
    gm.n = n;
    int rt = 0;
    for (int i = 0; i < n; ++i) {
        gm.w[i] = (const uint16_t*)mats[i].w;
        gm.s[i] = (const float*)wscales[i];
        gm.y[i] = mats[i].y;
        gm.N[i] = (int)mats[i].d_out;
        gm.rt_begin[i] = rt;
        rt += (int)((mats[i].d_out + 15) / 16);
    }
    for (int i = n; i <= kMaxMats; ++i) gm.rt_begin[i] = rt;
    const dim3 grid((unsigned)rt, (unsigned)((T + 15) / 16));
    if (xscales) k_mx4_product<true><<<grid, dim3(64), 0, s>>>(x, xscales, gm, (int)T, (int)d_in);
    else k_mx4_product<false><<<grid, dim3(64), 0, s>>>(x, nullptr, gm, (int)T, (int)d_in);
    return hipGetLastError();
}

}  // namespace bd
