// block.hpp -- launchers of the feed-forward block's operators (declared for
// block_api.cpp, which validates) and the device helpers they share.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gemm_block.h"
#include "gemm_core.hpp"

namespace mg {

// ---- host side ---------------------------------------------------------------

// Failure reporting and plan facts of gemm_api.cpp.
gemm_status api_fail(gemm_status s, const char *fmt, ...);
gemm_status api_ok();
struct PlanInfo {
    bool mxf4_tn;   // F4_E2M1, A RowMajor, B ColumnMajor, C RowMajor
    int act;
};
bool plan_info(gemm_plan_t p, PlanInfo *out);
gemm_status plan_on_device(gemm_plan_t p);   // its device is the current one; its first run binds it

// A matrix and where its codes and scales along the columns (rc, rs) and along
// the rows (cc, cs) go, one pair of which may be null. A second matrix (null:
// none) of the same type shares the launch; both have cc then.
struct Mx4Quant {
    const void *x;
    int64_t rows, cols, ld;
    uint8_t *rc, *rs, *cc, *cs;
};
hipError_t launch_mx4_quantize(int type, const Mx4Quant &a, const Mx4Quant *b, hipStream_t st);
hipError_t launch_mx4_dequantize(const uint8_t *codes, const uint8_t *scales, int64_t rows,
                                 int64_t k, void *out, int type, int64_t ld, hipStream_t st);
// The product of few rows of x; they are quantised on the way where xc is
// NULL (mx4_in_kernel), else given as codes and scales. More rows are the tile
// GEMM's. Whole calls with the quantiser, inputs in turn: 64 rows of 8192 x 8192
// 14.6 us here, 24.3 with the tile GEMM; of N = 28672, K = 8192 33 rows 46.0 and
// 49.0, 64 rows, where the two meet, 50.1 and 49.5.
constexpr int64_t MX4_FEW = 64, MX4_FEW_K = 1 << 26;   // rows; K that its 32-bit offsets reach in 32 rows
inline bool mx4_is_few(int64_t M, int64_t K) { return M <= MX4_FEW && K <= MX4_FEW_K; }
// Every workgroup quantises x again, which at 16 rows costs more than a launch
// (N = 28672, K = 8192: 53 us against 27). At eight it costs less where W is short
// (2048 x 2048 4.6 us against 7.8, 8192 x 8192 10.7 against 11.4) and more where
// many workgroups do it (N = 28672, K = 8192: 32.4 against 29.2); a rule on N too
// would save that.
inline bool mx4_in_kernel(int64_t M, int64_t K) { return M <= 8 && K <= MX4_FEW_K; }
hipError_t launch_mx4_few(const void *x, int type, int64_t ldx, const uint8_t *xc, const uint8_t *xs,
                          const uint8_t *wc, const uint8_t *ws, const void *bias, void *y, int64_t M,
                          int64_t N, int64_t K, int act, hipStream_t st);

struct MoeArgs {
    int64_t H, I, ldx, ldo;
    int T, E, k, renorm;
    const void *x, *router, *up, *down;
    const uint8_t *up_s, *down_s, *mask;
    void *out;
    int32_t *ids;
    float *probs;
    char *ws;
};
struct MoeLayout {
    // byte offsets into the workspace (the state words come first)
    int64_t columns, logits, ids, probs, slots, active, h, peak, y, total;
    int64_t ip;   // padded row length of h, in elements
};
int64_t moe_state_bytes(int64_t H);
MoeLayout moe_layout(int64_t H, int64_t I, int E, int k, int T, bool wide_h);   // wide_h: fp16
hipError_t launch_moe(int type, int weight_type, const MoeArgs &a, hipStream_t st);

hipError_t launch_norm_forward(const gemm_norm_args &a, hipStream_t st);
// How the backward pass cuts its rows: chunks of a group that are summed by
// one workgroup, or whole groups together.
struct NormCut {
    int64_t parts;            // workgroups = rows of the partial column sums
    int64_t rows_per_part;    // rows of a part (the last of a group may have fewer)
    int64_t chunks;           // parts per group; 1: a part holds whole groups
    int64_t groups_per_part;  // used where chunks == 1
    int64_t rows_per_group;
};
NormCut norm_cut(int64_t rows, int64_t cols, int64_t gate_rows);
hipError_t launch_norm_backward(const gemm_norm_backward_args &a, hipStream_t st);

// ---- device side ---------------------------------------------------------------

typedef __attribute__((ext_vector_type(2))) float f32x2;

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(_Float16 v) { return (float)v; }
__device__ __forceinline__ float to_f(__bf16 v) { return (float)v; }
template <class T> __device__ __forceinline__ T from_f(float v) { return (T)v; }

// 16 bytes at an address that is only element-aligned (global memory takes
// dwordx4 accesses at any alignment on this target).
typedef u32x4 u32x4_any __attribute__((aligned(2)));

// Eight consecutive elements, of which the first n exist (the others read as
// zero and are not touched).
template <class T> struct Vec8 {
    static constexpr int W = (int)sizeof(T) * 8 / 16;   // 16-byte words
    u32x4 w[W];
    __device__ __forceinline__ void load(const T *p, int64_t n) {
        if (n >= 8) {
            const u32x4_any *q = reinterpret_cast<const u32x4_any *>(p);
#pragma unroll
            for (int i = 0; i < W; ++i) w[i] = q[i];
        } else {
            T t[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) t[i] = i < n ? p[i] : (T)0.0f;
            __builtin_memcpy(w, t, sizeof(w));
        }
    }
    __device__ __forceinline__ void store(T *p, int64_t n) const {
        if (n >= 8) {
            u32x4_any *q = reinterpret_cast<u32x4_any *>(p);
#pragma unroll
            for (int i = 0; i < W; ++i) q[i] = w[i];
        } else {
            T t[8];
            __builtin_memcpy(t, w, sizeof(w));
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < n) p[i] = t[i];
        }
    }
    __device__ __forceinline__ void get(float *f) const {
        T t[8];
        __builtin_memcpy(t, w, sizeof(w));
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = to_f(t[i]);
    }
    __device__ __forceinline__ void set(const float *f) {
        T t[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) t[i] = from_f<T>(f[i]);
        __builtin_memcpy(w, t, sizeof(w));
    }
};

// A lane's eight elements from element c on of a row of H (c a multiple of
// eight): fetch_row asks for them, row_values gives them as fp32, zeros past the
// end. Where the row ends inside them its last eight are read and moved into
// place when they are used: loads of single elements would each be waited for.
// EVEN: H is a multiple of eight.
template <bool EVEN, class T>
__device__ __forceinline__ void fetch_row(Vec8<T> &x, const T *row, int64_t c, int64_t H) {
    if (H >= 8) {
        x.load(row + min(c, H - 8), 8);
    } else if constexpr (!EVEN) {
        T t[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) t[j] = j + H >= 8 ? row[j + H - 8] : (T)0.0f;
        __builtin_memcpy(x.w, t, sizeof(x.w));
    }
}
template <bool EVEN, class T>
__device__ __forceinline__ void row_values(const Vec8<T> &x, float *f, int64_t c, int64_t H) {
    x.get(f);
    const int n = (int)max((int64_t)0, min(c + 8 - H, (int64_t)8));   // elements past the end
    if constexpr (EVEN) {
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = n == 0 ? f[j] : 0.0f;
    } else if (n > 0) {
#pragma unroll
        for (int o = 8; o > 0; o >>= 1)
            if (n & o)
#pragma unroll
                for (int j = 0; j < 8; ++j) f[j] = j + o < 8 ? f[j + o] : 0.0f;
    }
}

// The largest of a value over the four lanes 4 i .. 4 i + 3, in each of them.
__device__ __forceinline__ uint32_t max_of_four(uint32_t v) {
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, true));   // lane ^ 1
    return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, true));   // lane ^ 2
}

// ---- MXFP4 blocks --------------------------------------------------------------

// E8M0 byte of a block whose largest magnitude has these fp32 bits (sign
// cleared; NaN and infinity compare above every number).
__device__ __forceinline__ uint32_t mx4_scale_byte(uint32_t amax) {
    if (amax >= 0x7F800000u) return 255u;
    const uint32_t e = amax >> 23;   // biased exponent: floor(log2) + 127, 0 below 2^-126
    return amax == 0u ? 127u : (e > 2u ? e - 2u : 0u);
}
// 2^(127 - byte), what brings the block's values below 8: exact in fp32 for
// every byte of a finite block (0..252); 0 for byte 255.
__device__ __forceinline__ float mx4_unscale(uint32_t byte) {
    return byte == 255u ? 0.0f : __builtin_bit_cast(float, (254u - byte) << 23);
}
// 2^(byte - 127) as fp32: a subnormal for byte 0, NaN for 255.
__device__ __forceinline__ float mx4_scale_value(uint32_t byte) {
    uint32_t b = byte << 23;
    b = byte == 0u ? 0x00400000u : b;
    return __builtin_bit_cast(float, byte == 255u ? 0x7FC00000u : b);
}
// Eight values (unscaled, below 8 in magnitude, or any where the factor is 0)
// to eight codes: v_cvt_scalef32_pk_fp4_f32 rounds to nearest even on the
// e2m1 grid and saturates at 6.
__device__ __forceinline__ uint32_t mx4_pack8(const float *v, float unscale) {
    float t[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = unscale == 0.0f ? 0.0f : v[i] * unscale;
    uint32_t r = 0;
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, t[0], t[1], 1.0f, 0);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, t[2], t[3], 1.0f, 1);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, t[4], t[5], 1.0f, 2);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, t[6], t[7], 1.0f, 3);
    return r;
}
__device__ __forceinline__ uint32_t abs_bits(float v) {
    return __builtin_bit_cast(uint32_t, v) & 0x7FFFFFFFu;
}

__host__ __device__ constexpr int64_t mx4_kp(int64_t k) { return (k + 255) / 256 * 256; }

}  // namespace mg
