// bd_mx4.hip -- microscaled 4-bit (MX4) base weights and tokens: quantisation,
// dequantisation and the base products Y = X Wq^T.
//
// A block of 32 consecutive columns of a row shares one power-of-two scale 2^E (the byte
// E + 127; 255 stands for NaN); its elements are e2m1 codes (0, .5, 1, 1.5, 2, 3, 4, 6
// and a sign), two per byte, the lower column in the low nibble.  Codes are row-major
// [rows][cols / 2]; a row of scales is padded with zeros to 16 ceil(cols / 512) bytes, so
// that the scales of any 512 columns are one aligned 16-byte piece.
#include "bd_tiles.h"

#include <type_traits>

namespace bd {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

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

// One wave's MI x NJ tiles of 32 rows x 32 tokens into y[T][N], rows from o0, tokens from
// t0.  The tokens are the products' first operand: in the D lane layout (32 x 32) a lane's
// column m32 is a row of W, its register 4 b + e token 8 b + 4 h + e, so a store writes whole
// 128-byte lines of y.
template <int MI, int NJ>
__device__ __forceinline__ void store_tile(const f32x16 (&acc)[MI][NJ], float* y, int N, int T,
                                           int o0, int t0, int m32, int h) {
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
#pragma unroll
        for (int b = 0; b < 4; ++b) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int t = t0 + 32 * j + 8 * b + 4 * h + e;
#pragma unroll
                for (int i = 0; i < MI; ++i) {
                    const int o = o0 + 32 * i + m32;
                    if (t < T && o < N) y[(int64_t)t * N + o] = acc[i][j][4 * b + e];
                }
            }
        }
    }
}

}  // namespace

// One wave per 512-column segment of a row: a lane holds 8 consecutive columns, four
// lanes one block.  `values` (may be null, may be w itself: a lane reads its columns
// before it writes them) receives what the codes stand for.  Bound by HBM: 4096 x 14336 with
// the values 41.6 us from bf16 (6.4 TB/s), 91.9 from fp32 (5.5).  Rows that leave lanes of
// their last segment without columns cost those lanes: at the same number of elements 52 us
// in rows of 512 columns, 63 of 576, 184 of 64 (weights have thousands of columns).
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

// The product for batches of at most 16 tokens on matrices of few rows and at most 4096
// columns, where a launch's latency is all that counts: one block per 16 rows, wave w on
// columns 512 w .. 512 w + 511, every load issued at once, the eight partial tiles summed in
// LDS in wave order.  bf16 tokens: a lane's block of 32 columns, widened to bf16 (exact),
// feeds four v_mfma_f32_16x16x32_bf16, step j taking columns 8 j .. 8 j + 7 of every block.
// MX4 tokens: one block-scaled 16x16x128 product per 128 columns.
// Every block reads all tokens, so the tiles below win from some rows on.  Against them
// (graph replays, us, 4096 columns): bf16, 6144 rows: 6.3 / 8.9 at 1 token, 8.9 / 9.3 at 8,
// 10.2 / 9.4 at 12; 4096 rows: 7.0 / 8.9 at 16; 14336 rows: 11.1 / 10.6 at 1.  MX4, 6144 rows:
// 5.7 / 7.5 at 1, 8.0 / 8.2 at 16; 14336 rows: 11.0 / 9.1 at 8.
constexpr int kRowsWaves = 8, kRowsK = 512 * kRowsWaves;
inline bool rows_fit(bool x4, int64_t T, int64_t d_in, int64_t row_tiles) {
    return T <= 16 && d_in <= kRowsK && row_tiles * (x4 ? 12 : T + 8) <= 6144;
}
template <bool X4>
__global__ void __launch_bounds__(64 * kRowsWaves)
k_mx4_rows(const void* __restrict__ x, const uint8_t* __restrict__ xs, const GemmMats gm, int T,
           int K) {
    __shared__ f32x4 red[kRowsWaves][64];
    const int lane = threadIdx.x & 63;
    const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int m = lane & 15, g = lane >> 4;
    const uint32_t rowb = (uint32_t)(K / 2), ld = 16u * (uint32_t)((K + 511) / 512);
    BD_MAT_OF(mt, gm, (int)blockIdx.x);
    const int N = mt.N, r0 = 16 * ((int)blockIdx.x - mt.rt0);
    const __amdgpu_buffer_rsrc_t wr = make_rsrc(mt.w, (uint64_t)N * rowb);
    const __amdgpu_buffer_rsrc_t sr = make_rsrc(mt.s, (uint64_t)N * ld);
    const __amdgpu_buffer_rsrc_t xr = make_rsrc(x, X4 ? (uint64_t)T * rowb : (uint64_t)T * K * 2);
    const __amdgpu_buffer_rsrc_t er = make_rsrc(xs, X4 ? (uint64_t)T * ld : 0);
    const int b0 = 16 * wv + g;  // this lane's blocks of 32 columns: b0 + 4 s
    const uint32_t row = (uint32_t)(r0 + m);
    u32x4 C[4], Xv[X4 ? 4 : 16];
    uint32_t xe[4];
#pragma unroll
    for (int s = 0; s < 4; ++s)
        C[s] = buf_load16(wr, r0 + m < N && b0 + 4 * s < K / 32 ? row * rowb + 16u * (uint32_t)(b0 + 4 * s) : kOOB);
    // the 16 scale bytes of the row's 512 columns
    const u32x4 E = buf_load16(sr, r0 + m < N && 512 * wv < K ? row * ld + 16u * (uint32_t)wv : kOOB);
#pragma unroll
    for (int s = 0; s < 4; ++s) {  // token m's same blocks
        const bool ok = m < T && b0 + 4 * s < K / 32;
        if constexpr (X4) {
            Xv[s] = buf_load16(xr, ok ? (uint32_t)m * rowb + 16u * (uint32_t)(b0 + 4 * s) : kOOB);
            xe[s] = buf_load1(er, ok ? (uint32_t)m * ld + (uint32_t)(b0 + 4 * s) : kOOB);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                Xv[4 * s + j] = buf_load16(
                    xr, ok ? (uint32_t)m * (uint32_t)(2 * K) + 64u * (uint32_t)(b0 + 4 * s) + 16u * j : kOOB);
        }
    }
    __builtin_amdgcn_sched_barrier(0);  // (else products start between the loads, to save registers)
    f32x4 acc[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
    for (int s = 0; s < 4; ++s) {
        const uint32_t es = s == 0 ? E.x : s == 1 ? E.y : s == 2 ? E.z : E.w;
        const uint32_t byte = (es >> (8 * g)) & 255u;
        if constexpr (X4) {
            const i32x8 a8 = {(int)C[s].x, (int)C[s].y, (int)C[s].z, (int)C[s].w, 0, 0, 0, 0};
            const i32x8 b8 = {(int)Xv[s].x, (int)Xv[s].y, (int)Xv[s].z, (int)Xv[s].w, 0, 0, 0, 0};
            acc[s & 1] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a8, b8, acc[s & 1], 4, 4, 0, (int)byte, 0,
                                                                          (int)xe[s]);
        } else {
            const float f = mx4_scale(byte);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t d = j == 0 ? C[s].x : j == 1 ? C[s].y : j == 2 ? C[s].z : C[s].w;
                acc[j & 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                    __builtin_bit_cast(bf16x8, widen_mx4(d, f)), __builtin_bit_cast(bf16x8, Xv[4 * s + j]),
                    acc[j & 1], 0, 0, 0);
            }
        }
    }
    red[wv][lane] = acc[0] + acc[1];
    __syncthreads();
    const int t = threadIdx.x >> 4, r = threadIdx.x & 15;  // token, row
    if (t >= T || r0 + r >= N) return;
    const int l = t + 16 * (r >> 2);  // D lane layout: column t, element r % 4
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kRowsWaves; ++w) v += ((const float*)&red[w][l])[r & 3];
    mt.y[(int64_t)t * N + r0 + r] = v;
}

// The product on MX4 tokens for batches of many tokens: block tiles of BR rows of Wq x BT
// tokens, NWR x NWT waves, each a block of MI x NJ tiles of the block-scaled
// v_mfma_scale_f32_32x32x64_f8f6f4.  K advances KC columns per stage (KC / 2 bytes of codes
// per row) through a ring of NS LDS stages filled by buffer loads that write LDS directly;
// the 16-byte chunks (one block of 32 columns each) are swizzled within their row so that
// 16 consecutive rows read at one chunk hit 16 distinct bank groups.  Lane half h takes
// chunks kSteps h + kk of a row in the stage's steps kk, so that one small read of scales per
// row serves the stage, step kk its byte kk.  The scales come 512 columns (16 bytes a row,
// one period of P stages) at a time into a ring of two slots.
// S > 1: K part sp covers columns [sp kps, (sp + 1) kps) (kps a multiple of 512) and
// writes its partial tile to part.
template <int BR, int BT, int KC, int NS, int NWR, int NWT>
__global__ void __launch_bounds__(64 * NWR * NWT)
k_mx4_gemm4(const uint8_t* __restrict__ x, const uint8_t* __restrict__ xsc, const GemmMats gm,
            int T, int K, int ntt, int S, int kps, int GR) {
    constexpr int NW = NWR * NWT;
    constexpr int MI = BR / NWR / 32, NJ = BT / NWT / 32;
    constexpr int kRowB = KC / 2, kC = KC / 32, kSteps = kC / 2, P = 512 / KC;
    constexpr int kRpI = 64 / kC;  // rows of one copy instruction
    constexpr int kRows = BR + BT, kStageBytes = kRows * kRowB, kSRows = (kRows + 63) / 64 * 64;
    constexpr int kWInst = BR / kRpI / NW, kXInst = BT / kRpI / NW, kD = kWInst + kXInst;
    constexpr int kSInst = (kSRows / 64 + NW - 1) / NW;  // scale copies per wave and period
    static_assert(KC == 128 || KC == 256, "4 or 8 chunks per row");
    static_assert(BR % (kRpI * NW) == 0 && BT % (kRpI * NW) == 0 && BR % 64 == 0,
                  "whole copy instructions per wave");
    static_assert(MI >= 1 && NJ >= 1 && BR % (32 * NWR) == 0 && BT % (32 * NWT) == 0, "32 x 32 tiles");
    static_assert(NS >= 3, "a stage's copies go out between the products of an earlier one");
    extern __shared__ __attribute__((aligned(16))) char smem[];
    char* const sring = smem + NS * kStageBytes;
    const TileId tid = tile_id(gm.rt_begin[gm.n], ntt, S, GR);
    const int sp = tid.sp, rtg = tid.rt, tt = tid.tt;
    if (rtg >= gm.rt_begin[gm.n]) return;  // uniform
    BD_MAT_OF(mt, gm, rtg);
    const int N = mt.N;
    float* const y = S > 1 ? mt.part + (int64_t)sp * T * N : mt.y;
    const int r0 = (rtg - mt.rt0) * BR, t0 = tt * BT;
    const int kbeg = sp * kps;
    const int kcols = K - kbeg < kps ? K - kbeg : kps;  // columns of this part
    const int nk = (kcols + KC - 1) / KC;
    const uint32_t rowb = (uint32_t)(K / 2), ld = 16u * (uint32_t)((K + 511) / 512);

    const int lane = threadIdx.x & 63;
    const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wr = wv / NWT, wt = wv % NWT;
    const __amdgpu_buffer_rsrc_t wrs = make_rsrc(mt.w, (uint64_t)N * rowb);
    const __amdgpu_buffer_rsrc_t wss = make_rsrc(mt.s, (uint64_t)N * ld);
    const __amdgpu_buffer_rsrc_t xrs = make_rsrc(x, (uint64_t)T * rowb);
    const __amdgpu_buffer_rsrc_t xss = make_rsrc(xsc, (uint64_t)T * ld);

    // loader: instruction i of an operand fills kRpI rows; lane l lands on row kRpI i + l / kC,
    // slot l % kC, i.e. takes the chunk whose swizzled slot that is
    auto swz = [](int r) { return (r / (16 / kC)) % kC; };
    uint32_t wsrc[kWInst], xsrc[kXInst];
#pragma unroll
    for (int j = 0; j < kWInst; ++j) {
        const int r = (wv * kWInst + j) * kRpI + lane / kC;
        const int c = (lane % kC) ^ swz(r);
        wsrc[j] = r0 + r < N ? (uint32_t)(r0 + r) * rowb + (uint32_t)(kbeg / 2 + 16 * c) : kOOB;
    }
#pragma unroll
    for (int j = 0; j < kXInst; ++j) {
        const int r = (wv * kXInst + j) * kRpI + lane / kC;
        const int c = (lane % kC) ^ swz(r);
        xsrc[j] = t0 + r < T ? (uint32_t)(t0 + r) * rowb + (uint32_t)(kbeg / 2 + 16 * c) : kOOB;
    }
    // scale copies: instruction i fills rows 64 i .. 64 i + 63 (W rows, then tokens)
    uint32_t ssrc[kSInst];
    int sdst[kSInst];
    bool sw[kSInst];
#pragma unroll
    for (int j = 0; j < kSInst; ++j) {
        const int i = (wv + j * NW) % (kSRows / 64);  // (a wave without its own repeats another's)
        sdst[j] = i * 1024;
        sw[j] = 64 * i < BR;
        const int r = 64 * i + lane;
        ssrc[j] = sw[j] ? (r0 + r < N ? (uint32_t)(r0 + r) * ld + (uint32_t)(kbeg / 32) : kOOB)
                        : (r < kRows && t0 + r - BR < T ? (uint32_t)(t0 + r - BR) * ld + (uint32_t)(kbeg / 32) : kOOB);
    }
    // Copy c of stage s's kD, into ring slot s % NS (zeros past the part's columns), and of
    // period p's scales (columns 512 p .. + 511), into slot p % 2.
    auto copy = [&](int s, int c) {
        char* base = smem + (s % NS) * kStageBytes;
        const int left = kcols - KC * s;  // columns from this stage on (uniform)
        const int i = c < kWInst ? wv * kWInst + c : wv * kXInst + c - kWInst;
        const int ch = (lane % kC) ^ swz(i * kRpI + lane / kC);
        const uint32_t add = 32 * ch < left ? (uint32_t)(kRowB * s) : kOOB;
        if (c < kWInst) copy16_to_lds(wrs, base + i * 1024, add_sat(wsrc[c < kWInst ? c : 0], add));
        else copy16_to_lds(xrs, base + BR * kRowB + i * 1024, add_sat(xsrc[c < kWInst ? 0 : c - kWInst], add));
    };
    auto copy_scales = [&](int p, int c) {
        char* base = sring + (p & 1) * kSRows * 16;
        const uint32_t off = add_sat(ssrc[c], 512 * p < kcols ? 16u * (uint32_t)p : kOOB);
        if (sw[c]) copy16_to_lds(wss, base + sdst[c], off);  // (uniform)
        else copy16_to_lds(xss, base + sdst[c], off);
    };

    f32x16 acc[MI][NJ];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.f;

    // The prologue: the first period's scales and the copies of NS - 1 stages.
#pragma unroll
    for (int c = 0; c < kSInst; ++c) copy_scales(0, c);
#pragma unroll
    for (int t = 0; t < NS - 1; ++t)
#pragma unroll
        for (int c = 0; c < kD; ++c) copy(t, c);

    const int m32 = lane & 31, h = lane >> 5;
    int sa[2][MI], sb[2][NJ];          // a stage's scales, by its parity
    u32x4 A[2][MI], Bv[2][NJ];         // a step's operands, by its parity (kSteps is even)
    // operand r of step kk of stage s (chunk kSteps h + kk of 32 rows): MI of W, then NJ tokens'
    auto read = [&](int s, auto kc, int r) {
        constexpr int kk = decltype(kc)::value;
        const char* base = smem + (s % NS) * kStageBytes + m32 * kRowB + 16 * ((kSteps * h + kk) ^ swz(m32));
        if (r < MI) A[kk & 1][r < MI ? r : 0] = *(const u32x4*)(base + (wr * (BR / NWR) + 32 * r) * kRowB);
        else Bv[kk & 1][r < MI ? 0 : r - MI] = *(const u32x4*)(base + (BR + wt * (BT / NWT) + 32 * (r - MI)) * kRowB);
    };
    auto read_scales = [&](int s, auto jc) {  // s % P == J
        constexpr int J = decltype(jc)::value % P, O = J & 1;
        using ST = std::conditional_t<kSteps == 4, int, uint16_t>;
        const char* sc = sring + ((s / P) & 1) * kSRows * 16 + J * kC + kSteps * h + 16 * m32;
#pragma unroll
        for (int i = 0; i < MI; ++i) sa[O][i] = (int)*(const ST*)(sc + (wr * (BR / NWR) + 32 * i) * 16);
#pragma unroll
        for (int j = 0; j < NJ; ++j) sb[O][j] = (int)*(const ST*)(sc + (BR + wt * (BT / NWT) + 32 * j) * 16);
    };
    // Step kk's products; between them the reads of the next step (sn, nc)'s operands and stage
    // s's share of copies: stage s sends out the copies of stage s + NS - 1, and a period's
    // first stage before them the scales of the next period, spread evenly over its products.
    // (All at once, copies or reads hold up every wave's products while the address unit or
    // the LDS takes them in turn: 256 columns of a 256 x 256 block took 3600 cycles with the
    // copies behind the barrier, 3250 with the reads alone in bursts, and take 2740 to 2850
    // like this, of which the products alone take 2300.)
    auto products = [&](int s, auto kc, auto jc, int sn, auto nc) {
        constexpr int kk = decltype(kc)::value, J = decltype(jc)::value, O = J & 1;
        constexpr int kS = J == 0 ? kSInst : 0, kTot = kS + kD, M = kSteps * MI * NJ;
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < MI; ++i) {
            const u32x4 v = A[kk & 1][i];
            const i32x8 a8 = {(int)v.x, (int)v.y, (int)v.z, (int)v.w, 0, 0, 0, 0};
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                const int ql = i * NJ + j, q = kk * MI * NJ + ql;  // this product of the step, of the stage
#pragma unroll
                for (int r = 0; r < MI + NJ; ++r)
                    if (r * MI * NJ / (MI + NJ) == ql) read(sn, nc, r);
#pragma unroll
                for (int c = 0; c < kTot; ++c) {
                    if (c * M / kTot != q) continue;
                    if (c < kS) copy_scales(s / P + 1, c < kS ? c : 0);
                    else copy(s + NS - 1, c - kS);
                }
                __builtin_amdgcn_sched_barrier(0);
                const u32x4 w = Bv[kk & 1][j];
                const i32x8 b8 = {(int)w.x, (int)w.y, (int)w.z, (int)w.w, 0, 0, 0, 0};
                acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(b8, a8, acc[i][j], 4, 4, kk, sb[O][j],
                                                                            kk, sa[O][i]);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    };
    using C0 = std::integral_constant<int, 0>;
    using C1 = std::integral_constant<int, 1>;
    using C2 = std::integral_constant<int, 2>;
    using C3 = std::integral_constant<int, 3>;
    // A stage's first operands are read behind the last products of the stage before: at
    // that point every wave holds the last operands of its stage, so the barrier frees its
    // slot and, after the wait, shows stage s + 1.
    auto stage = [&](int s, auto jc) {  // s % P == J
        constexpr int J = decltype(jc)::value;
        products(s, C0(), jc, s, C1());
        if constexpr (kSteps == 4) {
            products(s, C1(), jc, s, C2());
            products(s, C2(), jc, s, C3());
        }
        // in flight beyond what stage s + 1 needs: this stage's copies so far and those of the
        // NS - 3 stages before it, except scales that stage s + 1 starts on
        constexpr auto pending = [] {
            int n = 0;
            for (int d = 0; d <= NS - 3; ++d) {
                const int j = (J - d + 4 * P) % P, kS = j == 0 ? kSInst : 0, M = kSteps * MI * NJ;
                int sent = kS + kD;
                if (d == 0) {  // the last step's copies are still to come
                    sent = 0;
                    for (int c = 0; c < kS + kD; ++c) sent += c * M / (kS + kD) < M - MI * NJ ? 1 : 0;
                }
                if (J == P - 1 && d == P - 1) return n + sent - kS;
                n += sent;
            }
            return n;
        }();
        wait_vmcnt_lgkm<pending>();
        __builtin_amdgcn_s_barrier();
        read_scales(s + 1, std::integral_constant<int, J + 1>());
        products(s, std::integral_constant<int, kSteps - 1>(), jc, s + 1, C0());
    };
    wait_vmcnt<(NS - 2) * kD>();
    __builtin_amdgcn_s_barrier();
    read_scales(0, C0());
#pragma unroll
    for (int r = 0; r < MI + NJ; ++r) read(0, C0(), r);
    for (int s = 0; s < nk; s += P) {  // (uniform branches)
        stage(s, C0());
        if (s + 1 < nk) stage(s + 1, C1());
        if constexpr (P == 4) {
            if (s + 2 < nk) stage(s + 2, C2());
            if (s + 3 < nk) stage(s + 3, C3());
        }
    }
    wait_vmcnt<0>();  // the empty copies past the end have landed
    store_tile<MI, NJ>(acc, y, N, T, r0 + wr * (BR / NWR), t0 + wt * (BT / NWT), m32, h);
}

// The product on bf16 tokens for batches of many tokens: the tiles of k_mx4_gemm4 on
// v_mfma_f32_32x32x16_bf16, with the weights kept as codes in LDS and widened to bf16
// (exact) as a wave reads its operand.  K advances 64 columns per stage; the tokens come
// one stage (128 bytes a row) at a time into a ring of NSX slots, the codes WC columns at
// a time (WC / 2 bytes a row) into a ring of NSW slots, the scales 512 columns at a time
// into two slots.  Lane half h takes block h (32 columns) of a stage: 16 bytes of codes and
// one scale per row serve its four steps, step kk columns 8 kk .. 8 kk + 7 of the block.
// WHOLE: a stage's operands are all read during the stage before (their registers are few for
// tiles of 32 and 64 tokens), so that no product waits for the LDS: 28672 x 4096 at 16 tokens
// 18.8 -> 16.7 us, at 128 tokens 38 -> 36, 4096 x 4096 at 64 tokens 11.2 -> 10.5 (the 128 x 128
// tile, whose larger ring then leaves two blocks to a CU no more slack, 188 -> 196 us on
// 5120 x 17408 at 1144 tokens, stays with the step before).
template <int BR, int BT, int WC, int NSX, int NSW, int NWR, int NWT, bool WHOLE>
__global__ void __launch_bounds__(64 * NWR * NWT)
k_mx4_gemm16(const uint16_t* __restrict__ x, const GemmMats gm, int T, int K, int ntt, int S,
             int kps, int GR) {
    constexpr int NW = NWR * NWT;
    constexpr int MI = BR / NWR / 32, NJ = BT / NWT / 32;
    constexpr int kWRow = WC / 2, kWC = WC / 32;  // bytes and chunks of a row of codes
    constexpr int kSpW = WC / 64;                 // stages per slot of codes
    constexpr int kXSlot = BT * 128, kWSlot = BR * kWRow, kSSlot = BR * 16;
    constexpr int kXInst = BT / 8 / NW, kWInst = kWSlot / 1024 / NW;
    constexpr int kSInst = (BR / 64 + NW - 1) / NW;
    static_assert(BT % (8 * NW) == 0 && kWSlot % (1024 * NW) == 0 && BR % 64 == 0,
                  "whole copy instructions per wave");
    static_assert(MI >= 1 && NJ >= 1 && BR % (32 * NWR) == 0 && BT % (32 * NWT) == 0, "32 x 32 tiles");
    static_assert(NSX >= 3 && (NSW - 1) * kSpW >= NSX - (WHOLE ? 0 : 1) && NSX <= 7 && 8 % kSpW == 0,
                  "a stage's copies go out between the products of an earlier one, its codes and "
                  "scales no later than its tokens");
    extern __shared__ __attribute__((aligned(16))) char smem[];
    char* const wring = smem + NSX * kXSlot;
    char* const sring = wring + NSW * kWSlot;
    const TileId tid = tile_id(gm.rt_begin[gm.n], ntt, S, GR);
    const int sp = tid.sp, rtg = tid.rt, tt = tid.tt;
    if (rtg >= gm.rt_begin[gm.n]) return;  // uniform
    BD_MAT_OF(mt, gm, rtg);
    const int N = mt.N;
    float* const y = S > 1 ? mt.part + (int64_t)sp * T * N : mt.y;
    const int r0 = (rtg - mt.rt0) * BR, t0 = tt * BT;
    const int kbeg = sp * kps;
    const int kcols = K - kbeg < kps ? K - kbeg : kps;  // columns of this part
    const int nk = kcols / 64;
    const uint32_t rowb = (uint32_t)(K / 2), ld = 16u * (uint32_t)((K + 511) / 512);

    const int lane = threadIdx.x & 63;
    const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wr = wv / NWT, wt = wv % NWT;
    const __amdgpu_buffer_rsrc_t wrs = make_rsrc(mt.w, (uint64_t)N * rowb);
    const __amdgpu_buffer_rsrc_t wss = make_rsrc(mt.s, (uint64_t)N * ld);
    const __amdgpu_buffer_rsrc_t xrs = make_rsrc(x, (uint64_t)T * K * 2);

    // loaders: every lane takes the 16-byte chunk whose swizzled slot is its own
    uint32_t wsrc[kWInst], xsrc[kXInst], ssrc[kSInst];
    int sdst[kSInst];
#pragma unroll
    for (int j = 0; j < kXInst; ++j) {
        const int r = (wv * kXInst + j) * 8 + lane / 8;
        const int c = (lane % 8) ^ ((r / 2) % 8);
        xsrc[j] = t0 + r < T ? (uint32_t)(((int64_t)(t0 + r) * K + kbeg + 8 * c) * 2) : kOOB;
    }
    auto wchunk = [&](int r) { return (lane % kWC) ^ ((r / (16 / kWC)) % kWC); };
#pragma unroll
    for (int j = 0; j < kWInst; ++j) {
        const int r = (wv * kWInst + j) * (64 / kWC) + lane / kWC;
        wsrc[j] = r0 + r < N ? (uint32_t)(r0 + r) * rowb + (uint32_t)(kbeg / 2 + 16 * wchunk(r)) : kOOB;
    }
#pragma unroll
    for (int j = 0; j < kSInst; ++j) {
        const int i = (wv + j * NW) % (BR / 64);  // (a wave without its own repeats another's)
        sdst[j] = i * 1024;
        const int r = 64 * i + lane;
        ssrc[j] = r0 + r < N ? (uint32_t)(r0 + r) * ld + (uint32_t)(kbeg / 32) : kOOB;
    }
    // Copy c of the tokens of stage s (zeros past the part's columns), of the codes of columns
    // WC u .. WC u + WC - 1, and of the scales of columns 512 p .. 512 p + 511.
    auto copy_x = [&](int s, int c) {
        copy16_to_lds(xrs, smem + (s % NSX) * kXSlot + (wv * kXInst + c) * 1024,
                      add_sat(xsrc[c], s < nk ? 128u * (uint32_t)s : kOOB));
    };
    auto copy_w = [&](int u, int c) {
        const int r = (wv * kWInst + c) * (64 / kWC) + lane / kWC;
        copy16_to_lds(wrs, wring + (u % NSW) * kWSlot + (wv * kWInst + c) * 1024,
                      add_sat(wsrc[c], 32 * wchunk(r) < kcols - WC * u ? (uint32_t)(kWRow * u) : kOOB));
    };
    auto copy_s = [&](int p, int c) {
        copy16_to_lds(wss, sring + (p & 1) * kSSlot + sdst[c],
                      add_sat(ssrc[c], 512 * p < kcols ? 16u * (uint32_t)p : kOOB));
    };

    f32x16 acc[MI][NJ];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.f;

    const int m32 = lane & 31, h = lane >> 5;
    if constexpr (WHOLE) {
        // The prologue issues in the loop's order, as if by stages -8 .. -1.
#pragma unroll
        for (int t = -8; t < 0; ++t) {
            if (t == -8)
#pragma unroll
                for (int c = 0; c < kSInst; ++c) copy_s(0, c);
            if (t % kSpW == 0 && t / kSpW + NSW - 1 >= 0)
#pragma unroll
                for (int c = 0; c < kWInst; ++c) copy_w(t / kSpW + NSW - 1, c);
            if (t + NSX >= 0)
#pragma unroll
                for (int c = 0; c < kXInst; ++c) copy_x(t + NSX, c);
        }
        u32x4 C[2][MI], Bv[2][4][NJ];  // a stage's codes and tokens, by its parity
        float f[2][MI];
        constexpr int kReads = MI + 4 * NJ;
        auto read = [&](int s, auto jc, int r) {  // read r of stage s (s % 8 == J): codes, then tokens
            constexpr int J = decltype(jc)::value % 8, O = J & 1;
            if (r < MI) {
                const int row = wr * (BR / NWR) + 32 * r + m32;
                C[O][r < MI ? r : 0] =
                    *(const u32x4*)(wring + ((s / kSpW) % NSW) * kWSlot + row * kWRow +
                                    16 * ((2 * (J % kSpW) + h) ^ ((m32 / (16 / kWC)) % kWC)));
                f[O][r < MI ? r : 0] =
                    mx4_scale(*(const uint8_t*)(sring + ((s >> 3) & 1) * kSSlot + 2 * J + h + 16 * row));
            } else {
                const int kk = r < MI ? 0 : (r - MI) / NJ, j = r < MI ? 0 : (r - MI) % NJ;
                Bv[O][kk][j] = *(const u32x4*)(smem + (s % NSX) * kXSlot + (wt * (BT / NWT) + 32 * j + m32) * 128 +
                                               16 * ((4 * h + kk) ^ ((m32 / 2) % 8)));
            }
        };
        // in flight behind stage s's tokens, seen from the stage J at whose start they are
        // needed: what the d = 1 .. n stages before it issued
        constexpr auto issued = [](int J, int n) {
            int k = 0;
            for (int d = 1; d <= n; ++d) {
                const int j = (J - d + 16) % 8;
                k += kXInst + (j % kSpW == 0 ? kWInst : 0) + (j == 0 ? kSInst : 0);
            }
            return k;
        };
        auto stage = [&](int s, auto jc) {  // s % 8 == J
            constexpr int J = decltype(jc)::value, O = J & 1;
            constexpr int kS = J == 0 ? kSInst : 0, kW = J % kSpW == 0 ? kWInst : 0;
            constexpr int kTot = kS + kW + kXInst, M = 4 * MI * NJ;
            wait_vmcnt_lgkm<issued(J, NSX - 2)>();  // (and the wave holds stage s: its slot is free)
            __builtin_amdgcn_s_barrier();
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
#pragma unroll
                for (int i = 0; i < MI; ++i) {
                    const u32x4 A =
                        widen_mx4(kk == 0 ? C[O][i].x : kk == 1 ? C[O][i].y : kk == 2 ? C[O][i].z : C[O][i].w, f[O][i]);
#pragma unroll
                    for (int j = 0; j < NJ; ++j) {
                        const int q = (kk * MI + i) * NJ + j;
#pragma unroll
                        for (int r = 0; r < kReads; ++r)
                            if (r * M / kReads == q) read(s + 1, std::integral_constant<int, J + 1>(), r);
#pragma unroll
                        for (int c = 0; c < kTot; ++c) {
                            if (c * M / kTot != q) continue;
                            if (c < kS) copy_s(s / 8 + 1, c < kS ? c : 0);
                            else if (c < kS + kW) copy_w(s / kSpW + NSW - 1, c < kS + kW ? c - kS : 0);
                            else copy_x(s + NSX, c - kS - kW);
                        }
                        __builtin_amdgcn_sched_barrier(0);
                        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                            __builtin_bit_cast(bf16x8, Bv[O][kk][j]), __builtin_bit_cast(bf16x8, A), acc[i][j], 0, 0, 0);
                        if (j + 1 < NJ) __builtin_amdgcn_sched_barrier(0);
                    }
                }
            }
            __builtin_amdgcn_sched_barrier(0);
        };
        wait_vmcnt<issued(0, NSX - 1)>();
        __builtin_amdgcn_s_barrier();
#pragma unroll
        for (int r = 0; r < kReads; ++r) read(0, std::integral_constant<int, 0>(), r);
        for (int s = 0; s < nk; s += 8) {  // (uniform branches)
            stage(s, std::integral_constant<int, 0>());
            if (s + 1 < nk) stage(s + 1, std::integral_constant<int, 1>());
            if (s + 2 < nk) stage(s + 2, std::integral_constant<int, 2>());
            if (s + 3 < nk) stage(s + 3, std::integral_constant<int, 3>());
            if (s + 4 < nk) stage(s + 4, std::integral_constant<int, 4>());
            if (s + 5 < nk) stage(s + 5, std::integral_constant<int, 5>());
            if (s + 6 < nk) stage(s + 6, std::integral_constant<int, 6>());
            if (s + 7 < nk) stage(s + 7, std::integral_constant<int, 7>());
        }
    } else {
        // The prologue: the first period's scales, NSW - 1 slots of codes, NSX - 1 stages of tokens.
#pragma unroll
        for (int c = 0; c < kSInst; ++c) copy_s(0, c);
#pragma unroll
        for (int u = 0; u < NSW - 1; ++u)
#pragma unroll
            for (int c = 0; c < kWInst; ++c) copy_w(u, c);
#pragma unroll
        for (int t = 0; t < NSX - 1; ++t)
#pragma unroll
            for (int c = 0; c < kXInst; ++c) copy_x(t, c);

        u32x4 C[2][MI];  // a stage's codes and scales, by its parity
        float f[2][MI];
        u32x4 Bv[2][NJ];  // a step's tokens, by its parity
        auto read_x = [&](int s, auto kc, int j) {  // step kk of stage s: chunk 4 h + kk of token tile j
            constexpr int kk = decltype(kc)::value;
            Bv[kk & 1][j] = *(const u32x4*)(smem + (s % NSX) * kXSlot + (wt * (BT / NWT) + 32 * j + m32) * 128 +
                                            16 * ((4 * h + kk) ^ ((m32 / 2) % 8)));
        };
        auto read_w = [&](int s, auto jc) {  // s % 8 == J: block 2 (J % kSpW) + h of the wave's rows
            constexpr int J = decltype(jc)::value % 8, O = J & 1;
            const char* wt_base = wring + ((s / kSpW) % NSW) * kWSlot + wr * (BR / NWR) * kWRow + m32 * kWRow +
                                  16 * ((2 * (J % kSpW) + h) ^ ((m32 / (16 / kWC)) % kWC));
            const char* sc = sring + ((s >> 3) & 1) * kSSlot + 2 * J + h + 16 * (wr * (BR / NWR) + m32);
#pragma unroll
            for (int i = 0; i < MI; ++i) {
                C[O][i] = *(const u32x4*)(wt_base + 32 * kWRow * i);
                f[O][i] = mx4_scale(*(const uint8_t*)(sc + 512 * i));
            }
        };
        // Step kk's products; between them the reads of the next step (sn, nc)'s tokens and stage
        // s's share of copies, as in k_mx4_gemm4: stage s sends out the tokens of stage
        // s + NSX - 1 and before them, in a slot's first stage, the codes NSW - 1 slots on and,
        // in a period's first, the next period's scales.
        auto products = [&](int s, auto kc, auto jc, int sn, auto nc) {
            constexpr int kk = decltype(kc)::value, J = decltype(jc)::value, O = J & 1;
            constexpr int kS = J == 0 ? kSInst : 0, kW = J % kSpW == 0 ? kWInst : 0;
            constexpr int kTot = kS + kW + kXInst, M = 4 * MI * NJ;
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int i = 0; i < MI; ++i) {
                const u32x4 A =
                    widen_mx4(kk == 0 ? C[O][i].x : kk == 1 ? C[O][i].y : kk == 2 ? C[O][i].z : C[O][i].w, f[O][i]);
#pragma unroll
                for (int j = 0; j < NJ; ++j) {
                    const int ql = i * NJ + j, q = kk * MI * NJ + ql;  // this product of the step, of the stage
#pragma unroll
                    for (int r = 0; r < NJ; ++r)
                        if (r * MI == ql) read_x(sn, nc, r);
#pragma unroll
                    for (int c = 0; c < kTot; ++c) {
                        if (c * M / kTot != q) continue;
                        if (c < kS) copy_s(s / 8 + 1, c < kS ? c : 0);
                        else if (c < kS + kW) copy_w(s / kSpW + NSW - 1, c < kS + kW ? c - kS : 0);
                        else copy_x(s + NSX - 1, c - kS - kW);
                    }
                    __builtin_amdgcn_sched_barrier(0);
                    acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                        __builtin_bit_cast(bf16x8, Bv[kk & 1][j]), __builtin_bit_cast(bf16x8, A), acc[i][j], 0, 0, 0);
                    if (j + 1 < NJ) __builtin_amdgcn_sched_barrier(0);
                }
            }
            __builtin_amdgcn_sched_barrier(0);
        };
        using C0 = std::integral_constant<int, 0>;
        using C1 = std::integral_constant<int, 1>;
        using C2 = std::integral_constant<int, 2>;
        using C3 = std::integral_constant<int, 3>;
        auto stage = [&](int s, auto jc) {  // s % 8 == J
            constexpr int J = decltype(jc)::value;
            products(s, C0(), jc, s, C1());
            products(s, C1(), jc, s, C2());
            products(s, C2(), jc, s, C3());
            // in flight beyond what stage s + 1 needs: this stage's copies so far and those of the
            // NSX - 3 stages before it (its codes and scales went out no later than its tokens)
            constexpr auto pending = [] {
                int n = 0;
                for (int d = 0; d <= NSX - 3; ++d) {
                    const int j = (J - d + 8) % 8, M = 4 * MI * NJ;
                    const int kTot = (j == 0 ? kSInst : 0) + (j % kSpW == 0 ? kWInst : 0) + kXInst;
                    int sent = kTot;
                    if (d == 0) {  // the last step's copies are still to come
                        sent = 0;
                        for (int c = 0; c < kTot; ++c) sent += c * M / kTot < M - MI * NJ ? 1 : 0;
                    }
                    n += sent;
                }
                return n;
            }();
            wait_vmcnt_lgkm<pending>();
            __builtin_amdgcn_s_barrier();
            read_w(s + 1, std::integral_constant<int, J + 1>());
            products(s, C3(), jc, s + 1, C0());
        };
        wait_vmcnt<(NSX - 2) * kXInst>();
        __builtin_amdgcn_s_barrier();
        read_w(0, C0());
#pragma unroll
        for (int j = 0; j < NJ; ++j) read_x(0, C0(), j);
        for (int s = 0; s < nk; s += 8) {  // (uniform branches)
            stage(s, std::integral_constant<int, 0>());
            if (s + 1 < nk) stage(s + 1, std::integral_constant<int, 1>());
            if (s + 2 < nk) stage(s + 2, std::integral_constant<int, 2>());
            if (s + 3 < nk) stage(s + 3, std::integral_constant<int, 3>());
            if (s + 4 < nk) stage(s + 4, std::integral_constant<int, 4>());
            if (s + 5 < nk) stage(s + 5, std::integral_constant<int, 5>());
            if (s + 6 < nk) stage(s + 6, std::integral_constant<int, 6>());
            if (s + 7 < nk) stage(s + 7, std::integral_constant<int, 7>());
        }
    }
    wait_vmcnt<0>();  // the empty copies past the end have landed
    store_tile<MI, NJ>(acc, y, N, T, r0 + wr * (BR / NWR), t0 + wt * (BT / NWT), m32, h);
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
    // (each size first: their products then stay inside 64 bits)
    return d_in % 64 == 0 && d_in < ((int64_t)1 << 30) && d_out < ((int64_t)1 << 30) &&
           T < ((int64_t)1 << 20) && T * d_in * (x4 ? 1 : 4) < ((int64_t)1 << 32) &&
           d_out * d_in < ((int64_t)1 << 32);
}

namespace {

// One launch of a tile: S K parts of kps columns (S == 1: all of K, straight into y).
struct Mx4Launch {
    const void* x;
    const uint8_t* xscales;
    int64_t T, d_in;
    const GemmMatArg* mats;
    const uint8_t* const* wscales;
    int n, S;
    int64_t kps;
    float* const* parts;
    hipStream_t s;
};

template <int BR, int BT, int KC, int NS, int NWR, int NWT>
hipError_t launch_gemm4(const Mx4Launch& l) {
    int rt = 0;
    const GemmMats gm = gemm_mats(l.mats, l.wscales, l.n, BR, l.parts, &rt);
    const int ntt = (int)((l.T + BT - 1) / BT), GR = row_group(ntt);
    const unsigned blocks = tile_grid(rt, ntt, l.S);
    constexpr int lds = (BR + BT) * NS * (KC / 2) + (BR + BT + 63) / 64 * 64 * 32;
    k_mx4_gemm4<BR, BT, KC, NS, NWR, NWT><<<dim3(blocks), dim3(64 * NWR * NWT), lds, l.s>>>(
        (const uint8_t*)l.x, l.xscales, gm, (int)l.T, (int)l.d_in, ntt, l.S, (int)l.kps, GR);
    return hipGetLastError();
}

template <int BR, int BT, int WC, int NSX, int NSW, int NWR, int NWT, bool WHOLE>
hipError_t launch_gemm16(const Mx4Launch& l) {
    int rt = 0;
    const GemmMats gm = gemm_mats(l.mats, l.wscales, l.n, BR, l.parts, &rt);
    const int ntt = (int)((l.T + BT - 1) / BT), GR = row_group(ntt);
    const unsigned blocks = tile_grid(rt, ntt, l.S);
    constexpr int lds = NSX * BT * 128 + NSW * BR * (WC / 2) + 2 * BR * 16;
    k_mx4_gemm16<BR, BT, WC, NSX, NSW, NWR, NWT, WHOLE><<<dim3(blocks), dim3(64 * NWR * NWT), lds, l.s>>>(
        (const uint16_t*)l.x, gm, (int)l.T, (int)l.d_in, ntt, l.S, (int)l.kps, GR);
    return hipGetLastError();
}

hipError_t launch_rows(const Mx4Launch& l) {
    int rt = 0;
    const GemmMats gm = gemm_mats(l.mats, l.wscales, l.n, 16, nullptr, &rt);
    const dim3 grid((unsigned)rt), block(64 * kRowsWaves);
    if (l.xscales) k_mx4_rows<true><<<grid, block, 0, l.s>>>(l.x, l.xscales, gm, (int)l.T, (int)l.d_in);
    else k_mx4_rows<false><<<grid, block, 0, l.s>>>(l.x, nullptr, gm, (int)l.T, (int)l.d_in);
    return hipGetLastError();
}

// y (fp32, or bf16 rounded once) = the sum of the S partial products, in part order (grid.y:
// the matrix).
__device__ __forceinline__ void put4(float* y, int64_t i, f32x4 v) { ((f32x4*)y)[i] = v; }
__device__ __forceinline__ void put4(uint16_t* y, int64_t i, f32x4 v) {
    ((uint2*)y)[i] = make_uint2((uint32_t)f32_to_bf16(v[0]) | (uint32_t)f32_to_bf16(v[1]) << 16,
                                (uint32_t)f32_to_bf16(v[2]) | (uint32_t)f32_to_bf16(v[3]) << 16);
}
__device__ __forceinline__ void put1(float* y, int64_t i, float v) { y[i] = v; }
__device__ __forceinline__ void put1(uint16_t* y, int64_t i, float v) { y[i] = f32_to_bf16(v); }

template <typename YT>
__global__ void __launch_bounds__(256)
k_sum_parts(const GemmMats gm, int T, int S) {
    typedef f32x4 f32x4_a4 __attribute__((aligned(4)));  // (a part starts at any float)
    const int mi = (int)blockIdx.y;
    const int64_t n = (int64_t)T * gm.N[mi];
    const float* part = gm.part[mi];
    YT* y = (YT*)gm.y[mi];
    const int64_t i0 = (int64_t)blockIdx.x * 256 + threadIdx.x, step = (int64_t)gridDim.x * 256;
    for (int64_t i = i0; i < n / 4; i += step) {
        f32x4 v = ((const f32x4*)part)[i];
        for (int q = 1; q < S; ++q) v += ((const f32x4_a4*)(part + q * n))[i];
        put4(y, i, v);
    }
    if (const int64_t i = n / 4 * 4 + i0; i < n) {
        float v = part[i];
        for (int q = 1; q < S; ++q) v += part[q * n + i];
        put1(y, i, v);
    }
}

// Tile and K split by a model of their time (us), fitted to measurements of the tiles and
// splits at 17..8192 tokens on 700 x 1088 to 34816 x 5120 (graph replays on one MI355X):
//   a + max(ceil(blocks / (256 occ)) b, ceil(blocks / 256) c) n + (S > 1: 2 + bytes / 3.5 TB/s)
// with n the 256-column steps of a block's K part, occ the blocks a CU holds, a the fixed
// cost, b one block's time per step, c a CU's per block and step.  Against every tile and
// split on matrices and batches that the fit did not see (seven matrices, 24 to 6000 tokens),
// the choice is 1.2% (MX4 tokens) and 1.9% (bf16) off the best on average, 18% and 16% at the
// worst; always the largest tile, with its best split, is 42% and 57% off on average, always
// the smallest 25% and 26%.  At 1, 8 and 16 tokens, where rows_fit and the model share the
// choice: 4.9% and 2.2%, 27% (16 tokens on 10240 x 8192) and 21% (8 tokens on 6912 x 2560,
// where the row kernel would win) at the worst.
struct TileCost {
    int tile, br, bt, occ;
    double a, b, c;
};
enum { kRows, k256x256, k128x256, k128x128, k128x64, k128x32, k64x64, k64x32 };
constexpr TileCost kCost4[] = {{k256x256, 256, 256, 1, 7.7, 0.0, 1.60},
                               {k128x256, 128, 256, 1, 4.9, 0.0, 1.09},
                               {k128x128, 128, 128, 1, 5.1, 0.0, 0.655},
                               {k128x64, 128, 64, 2, 5.0, 0.135, 0.418},
                               {k64x64, 64, 64, 3, 4.4, 0.30, 0.279}};
constexpr TileCost kCost16[] = {{k256x256, 256, 256, 1, 7.7, 0.0, 4.54},
                                {k128x128, 128, 128, 2, 7.5, 1.70, 1.57},
                                {k128x64, 128, 64, 2, 5.85, 1.05, 0.937},
                                {k128x32, 128, 32, 3, 5.5, 0.60, 0.56},
                                {k64x32, 64, 32, 3, 5.2, 0.59, 0.353}};
struct Mx4Plan {
    int tile, S;
    int64_t kps;
};
Mx4Plan plan_mx4(bool x4, int64_t T, int64_t d_in, const int64_t* d_outs, int n, bool split_ok) {
    Mx4Plan pl = {kRows, 1, d_in};
    int64_t N = 0, tiles = 0;
    for (int i = 0; i < n; ++i) {
        N += d_outs[i];
        tiles += (d_outs[i] + 15) / 16;
    }
    if (rows_fit(x4, T, d_in, tiles)) return pl;
    double best = 1e30;
    for (int k = 0; k < 5; ++k) {
        const TileCost& t = x4 ? kCost4[k] : kCost16[k];
        int64_t rt = 0;
        for (int i = 0; i < n; ++i) rt += (d_outs[i] + t.br - 1) / t.br;
        for (int S = 1; S <= (split_ok ? 8 : 1); S *= 2) {
            if (S > 1 && d_in < 1024 * S) break;  // parts of 1024 columns or more
            const int64_t kps = S > 1 ? (d_in + 512 * S - 1) / (512 * S) * 512 : d_in;
            const int64_t parts = (d_in + kps - 1) / kps;
            const int64_t blocks = rt * ((T + t.bt - 1) / t.bt) * parts;
            const double one = t.b * (double)((blocks + 256 * t.occ - 1) / (256 * t.occ));
            const double cu = t.c * (double)((blocks + 255) / 256);
            double us = t.a + (one > cu ? one : cu) * (double)kps / 256;
            if (parts > 1) us += 2.0 + (double)(T * N * (4 * parts + 4)) / 3.5e6;
            if (us < best) {
                best = us;
                pl = {t.tile, (int)parts, kps};
            }
        }
    }
    return pl;
}

}  // namespace

hipError_t launch_sum_parts(const GemmMats& gm, int64_t T, int64_t nmax, int S, int ydtype, hipStream_t s) {
    const int64_t nb = (T * nmax / 4 + 255) / 256;
    const dim3 grid((unsigned)(nb < 1 ? 1 : nb < 2048 ? nb : 2048), (unsigned)gm.n), block(256);
    if (ydtype == BD_BF16) k_sum_parts<uint16_t><<<grid, block, 0, s>>>(gm, (int)T, S);
    else k_sum_parts<float><<<grid, block, 0, s>>>(gm, (int)T, S);
    return hipGetLastError();
}

size_t mx4_product_bytes(bool x4, int64_t T, int64_t d_in, const int64_t* d_outs, int n) {
    const Mx4Plan pl = plan_mx4(x4, T, d_in, d_outs, n, true);
    if (pl.S == 1) return 0;
    size_t b = 0;
    for (int i = 0; i < n; ++i) b += align_up((size_t)pl.S * T * d_outs[i] * 4);
    return b;
}

hipError_t launch_mx4_product(const void* x, const uint8_t* xscales, int64_t T, int64_t d_in,
                              const GemmMatArg* mats, const uint8_t* const* wscales, int n, char* ws,
                              hipStream_t s) {
    if (n < 1 || n > kMaxMats) return hipErrorInvalidValue;
    if (T == 0) return hipSuccess;
    int64_t d_outs[kMaxMats], nmax = 0;
    for (int i = 0; i < n; ++i) {
        d_outs[i] = mats[i].d_out;
        nmax = d_outs[i] > nmax ? d_outs[i] : nmax;
    }
    const Mx4Plan pl = plan_mx4(xscales != nullptr, T, d_in, d_outs, n, ws != nullptr);
    float* parts[kMaxMats] = {};
    size_t off = 0;
    for (int i = 0; i < n && pl.S > 1; ++i) {
        parts[i] = (float*)(ws + off);
        off += align_up((size_t)pl.S * T * d_outs[i] * 4);
    }
    const Mx4Launch l = {x, xscales, T, d_in, mats, wscales, n, pl.S, pl.kps, pl.S > 1 ? parts : nullptr, s};
    hipError_t e;
    if (pl.tile == kRows) {
        e = launch_rows(l);
    } else if (xscales) {
        switch (pl.tile) {
            case k256x256: e = launch_gemm4<256, 256, 128, 4, 4, 2>(l); break;
            case k128x256: e = launch_gemm4<128, 256, 128, 4, 2, 4>(l); break;
            case k128x128: e = launch_gemm4<128, 128, 256, 4, 2, 2>(l); break;
            case k128x64: e = launch_gemm4<128, 64, 256, 3, 4, 1>(l); break;
            default: e = launch_gemm4<64, 64, 256, 3, 2, 2>(l); break;
        }
    } else {
        switch (pl.tile) {
            case k256x256: e = launch_gemm16<256, 256, 128, 3, 3, 4, 2, false>(l); break;
            case k128x128: e = launch_gemm16<128, 128, 128, 3, 2, 2, 2, false>(l); break;
            case k128x64: e = launch_gemm16<128, 64, 256, 4, 2, 2, 2, true>(l); break;
            case k128x32: e = launch_gemm16<128, 32, 256, 4, 2, 4, 1, true>(l); break;
            default: e = launch_gemm16<64, 32, 256, 4, 2, 2, 1, true>(l); break;
        }
    }
    if (e != hipSuccess || pl.S == 1) return e;
    int rt = 0;
    return launch_sum_parts(gemm_mats(mats, wscales, n, 16, parts, &rt), T, nmax, pl.S, BD_F32, s);
}

}  // namespace bd
