// kernels_norm.hip -- the norms before and after a block, fused with its gate
// and residual scale, and their gradients.
#include "block.hpp"

namespace mg {

namespace {

// Sum over the lanes of a wave, in every lane.
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
    return v;
}

// Sums of N values over the WPR waves that share a row. The slots alternate
// between calls (`turn`), so one barrier per call is enough: a slot is written
// again only after the barrier of the call between. The barrier waits for the
// LDS alone, so that the next row's loads stay in flight.
template <int WPR, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float (*slot)[N][WPR], int &turn) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
    if constexpr (WPR > 1) {
        const int wave = threadIdx.x >> 6;
        if ((threadIdx.x & 63) == 0)
#pragma unroll
            for (int i = 0; i < N; ++i) slot[turn][i][wave] = v[i];
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
#pragma unroll
        for (int i = 0; i < N; ++i) {
            v[i] = 0.0f;
#pragma unroll
            for (int w = 0; w < WPR; ++w) v[i] += slot[turn][i][w];
        }
        turn ^= 1;
    }
}

// A gate's value and the slope of it, to a few steps of fp32 at any v: from
// exp(-|v|), since act (1 - act) loses the slope of a gate that is nearly open
// (all of it from v = 17 on), and the fast exp loses a step with each unit of v.
__device__ __forceinline__ float sigmoid(float v) {
    const float e = expf(-__builtin_fabsf(v));
    return (v < 0.0f ? e : 1.0f) / (1.0f + e);
}
__device__ __forceinline__ float sigmoid_slope(float v) {
    const float e = expf(-__builtin_fabsf(v));
    return e / ((1.0f + e) * (1.0f + e));
}

// A thread's eight columns of a row. EVEN: the row's length is a multiple of
// eight, so they all exist or none does. Else the thread that the row ends in
// asks for the row's last eight elements and moves them into place when it
// uses them: loads of single elements would each be waited for.
template <bool EVEN, class T>
__device__ __forceinline__ void fetch(Vec8<T> &x, const T *row, int64_t c, int64_t H) {
    if (EVEN || H >= 8) {
        if (c < H) x.load(row + (EVEN ? c : min(c, H - 8)), 8);
    } else if (c < H) {
        T t[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) t[j] = j + H >= 8 ? row[j + H - 8] : (T)0.0f;
        __builtin_memcpy(x.w, t, sizeof(x.w));
    }
}
template <bool EVEN, class T>
__device__ __forceinline__ void unpack(const Vec8<T> &x, float *f, int64_t c, int64_t H) {
    x.get(f);
    if constexpr (!EVEN)
        if (c < H && c + 8 > H) {
            const int n = (int)(c + 8 - H);
#pragma unroll
            for (int o = 4; o > 0; o >>= 1)
                if (n & o)
#pragma unroll
                    for (int j = 0; j < 8; ++j) f[j] = j + o < 8 ? f[j + o] : 0.0f;
        }
}
template <bool EVEN, class T>
__device__ __forceinline__ void put(const float *f, T *row, int64_t c, int64_t H) {
    if (c >= H) return;
    Vec8<T> x;
    x.set(f);
    x.store(row + c, EVEN ? 8 : H - c);
}

// ---- forward --------------------------------------------------------------------
//
//   y = b rstd(b) w_post,  out = residual + scale act(gate) y,
//   next = out rstd(out) w_next
// Bound by memory: two reads and two writes of [rows][cols]. WPR waves hold a
// row in registers from its first load to its last store (VPT groups of eight
// elements a thread); a workgroup walks over rows, holds the vectors, and asks
// for the next row before it sums this one.
template <class T, int WPR, int VPT, bool EVEN>
__global__ __launch_bounds__(WPR == 1 ? 256 : WPR * 64) void norm_forward_kernel(gemm_norm_args a) {
    constexpr int RPB = WPR == 1 ? 4 : 1, NT = WPR * 64;
    __shared__ float slot[2][1][WPR];
    int turn = 0;
    const int t = WPR == 1 ? (threadIdx.x & 63) : threadIdx.x;
    const int64_t H = a.cols;
    const uint32_t per = a.gate ? (uint32_t)a.rows / (uint32_t)a.gate_rows : 1u;
    const float inv = 1.0f / (float)H;
    int64_t row = (int64_t)blockIdx.x * RPB + (WPR == 1 ? threadIdx.x >> 6 : 0);
    if (row >= a.rows) return;   // whole waves; no barrier where a row is one wave's
    Vec8<T> res[VPT] = {}, blk[VPT] = {}, gat[VPT] = {}, wn[VPT] = {};   // the row asked for; w_next
    float q[VPT][8];                                                     // w_post * scale
    const auto ask = [&](int64_t r) {
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int64_t c = ((int64_t)v * NT + t) * 8;
            fetch<EVEN>(res[v], static_cast<const T *>(a.residual) + r * a.ld_residual, c, H);
            if (a.block) fetch<EVEN>(blk[v], static_cast<const T *>(a.block) + r * a.ld_block, c, H);
            if (a.gate) fetch<EVEN>(gat[v], static_cast<const T *>(a.gate) + (int64_t)((uint32_t)r / per) * a.ld_gate,
                                    c, H);
        }
    };
    ask(row);
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        const int64_t c = ((int64_t)v * NT + t) * 8;
        Vec8<T> wp = {}, sc = {};
        if (a.w_post) fetch<EVEN>(wp, static_cast<const T *>(a.w_post), c, H);
        if (a.scale) fetch<EVEN>(sc, static_cast<const T *>(a.scale), c, H);
        if (a.w_next) fetch<EVEN>(wn[v], static_cast<const T *>(a.w_next), c, H);
        float f[8];
        unpack<EVEN>(wp, q[v], c, H);
        unpack<EVEN>(sc, f, c, H);
#pragma unroll
        for (int j = 0; j < 8; ++j) q[v][j] = (a.w_post ? q[v][j] : 1.0f) * (a.scale ? f[j] : 1.0f);
    }
    for (; row < a.rows; row += (int64_t)gridDim.x * RPB) {
        float r[VPT][8], b[VPT][8], f[8];
        Vec8<T> gate[VPT];
        const int64_t next_row = row + (int64_t)gridDim.x * RPB;
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            unpack<EVEN>(res[v], r[v], ((int64_t)v * NT + t) * 8, H);
            unpack<EVEN>(blk[v], b[v], ((int64_t)v * NT + t) * 8, H);
            gate[v] = gat[v];
        }
        if (next_row < a.rows) ask(next_row);
        if (a.block) {
            float rb = 1.0f;
            if (a.w_post) {
                float s[1] = {0.0f};
#pragma unroll
                for (int v = 0; v < VPT; ++v)
#pragma unroll
                    for (int j = 0; j < 8; ++j) s[0] += b[v][j] * b[v][j];
                row_sums<WPR>(s, slot, turn);
                rb = rsqrtf(s[0] * inv + a.eps);
                if (a.rstd_post && t == 0) a.rstd_post[row] = rb;
            }
            T *out = static_cast<T *>(a.out) + row * a.ld_out;
#pragma unroll
            for (int v = 0; v < VPT; ++v) {
#pragma unroll
                for (int j = 0; j < 8; ++j) b[v][j] *= rb * q[v][j];
                if (a.gate) {
                    unpack<EVEN>(gate[v], f, ((int64_t)v * NT + t) * 8, H);
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        b[v][j] *= a.gate_act == GEMM_EPI_SIGMOID ? sigmoid(f[j]) : f[j];
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) r[v][j] += b[v][j];
                put<EVEN>(r[v], out, ((int64_t)v * NT + t) * 8, H);
                // the next norm reads what is stored, as the backward pass does
#pragma unroll
                for (int j = 0; j < 8; ++j) r[v][j] = to_f(from_f<T>(r[v][j]));
            }
        }
        if (!a.w_next) continue;
        float s[1] = {0.0f};
#pragma unroll
        for (int v = 0; v < VPT; ++v)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                s[0] += ((int64_t)v * NT + t) * 8 + j < H ? r[v][j] * r[v][j] : 0.0f;
        row_sums<WPR>(s, slot, turn);
        const float rr = rsqrtf(s[0] * inv + a.eps);
        if (a.rstd_next && t == 0) a.rstd_next[row] = rr;
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            unpack<EVEN>(wn[v], f, ((int64_t)v * NT + t) * 8, H);
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] *= r[v][j] * rr;
            put<EVEN>(f, static_cast<T *>(a.next) + row * a.ld_next, ((int64_t)v * NT + t) * 8, H);
        }
    }
}

// ---- backward --------------------------------------------------------------------
//
// With xn = out rstd_next, xb = block rstd_post, act the gate's value:
//   g  = d_next w_next,  d = d_out + rstd_next (g - xn mean(g xn))  (d_residual)
//   q  = scale act w_post,  d_block = rstd_post (d q - xb mean(d q xb))
// The second mean follows from sums that do not wait for the first,
//   sum(d q xb) = sum((d_out + rstd_next g) q xb) - rstd_next mean(g xn) sum(xn q xb),
// so a row costs one barrier. All column sums but d_w_next = sum(d_next xn)
// are multiples of B = sum(d xb) over a group's rows, where act is constant:
//   d_gate = scale w_post act' B,  A = sum over groups of act B,
//   d_w_post = scale A,  d_scale = w_post A,
// so a row adds to two registers a column. Bound by memory: four reads and two
// writes of [rows][cols]. A workgroup walks the rows of its part with a fixed
// set of columns per thread and asks for the next row before it sums this one;
// the parts' sums are added by norm_columns_kernel in part order, so no result
// depends on the order of execution.
struct ColumnSums {
    float *part;        // [parts][3][cols]: d_w_post, d_scale, d_w_next
    float *gate_part;   // [parts][cols], where a group is cut into chunks
    NormCut cut;
};

template <class T, int WPR, int VPT, bool EVEN>
__global__ __launch_bounds__(WPR * 64) void norm_backward_kernel(gemm_norm_backward_args a,
                                                                 ColumnSums cs) {
    constexpr int NT = WPR * 64;
    // A thread of one column group holds w_post, scale and the gate, one of two
    // has no registers for them and reads them again (from the L2) where a
    // group ends: held, 32 spills made 4096 x 8192 bf16 take 113 us against 88.
    constexpr bool HOLD = VPT == 1;
    __shared__ float slot[2][3][WPR];
    int turn = 0;
    const int t = threadIdx.x;
    const int64_t H = a.cols, part = blockIdx.x;
    const NormCut cut = cs.cut;
    int64_t row, end;
    if (cut.chunks > 1) {
        const int64_t group = (uint32_t)part / (uint32_t)cut.chunks, chunk = part - group * cut.chunks;
        row = group * cut.rows_per_group + chunk * cut.rows_per_part;
        end = min(row + cut.rows_per_part, (group + 1) * cut.rows_per_group);
    } else {
        row = part * cut.groups_per_part * cut.rows_per_group;
        end = min(row + cut.groups_per_part * cut.rows_per_group, a.rows);
    }
    const float inv = 1.0f / (float)H;
    const bool sig = a.gate_act == GEMM_EPI_SIGMOID;
    float A[VPT][8] = {}, B[VPT][8] = {}, N[VPT][8] = {}, q[VPT][8];
    Vec8<T> xo[VPT] = {}, xd[VPT] = {}, xr[VPT] = {}, xk[VPT] = {}, xg[VPT] = {};   // the row asked for
    Vec8<T> wn[VPT] = {};
    Vec8<T> wp = {}, sc = {}, cg = {};   // with HOLD; cg: the gate of the group at hand
    float rr = 0.0f, rb = 1.0f;
    int64_t group = (uint32_t)row / (uint32_t)cut.rows_per_group, group_end = (group + 1) * cut.rows_per_group;
    const auto ask_gate = [&](int64_t gr) {
#pragma unroll
        for (int v = 0; v < VPT; ++v)
            fetch<EVEN>(xg[v], static_cast<const T *>(a.gate) + gr * a.ld_gate, ((int64_t)v * NT + t) * 8, H);
    };
    const auto ask = [&](int64_t r) {
        if (a.w_next) rr = a.rstd_next[r];
        if (a.w_post) rb = a.rstd_post[r];
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int64_t c = ((int64_t)v * NT + t) * 8;
            if (a.d_out) fetch<EVEN>(xo[v], static_cast<const T *>(a.d_out) + r * a.ld_d_out, c, H);
            if (a.d_next) {
                fetch<EVEN>(xd[v], static_cast<const T *>(a.d_next) + r * a.ld_d_next, c, H);
                fetch<EVEN>(xr[v], static_cast<const T *>(a.out) + r * a.ld_out, c, H);
            }
            if (a.block) fetch<EVEN>(xk[v], static_cast<const T *>(a.block) + r * a.ld_block, c, H);
        }
    };
    const auto ask_vectors = [&](int v, Vec8<T> &p, Vec8<T> &e) {
        const int64_t c = ((int64_t)v * NT + t) * 8;
        if (a.w_post) fetch<EVEN>(p, static_cast<const T *>(a.w_post), c, H);
        if (a.scale) fetch<EVEN>(e, static_cast<const T *>(a.scale), c, H);
    };
    // w_post, scale (1 where there is none) of a thread's columns
    const auto vectors = [&](int v, float *p, float *e) {
        const int64_t c = ((int64_t)v * NT + t) * 8;
        if constexpr (HOLD) {
            unpack<EVEN>(wp, p, c, H);
            unpack<EVEN>(sc, e, c, H);
        } else {
            Vec8<T> x = {}, y = {};
            ask_vectors(v, x, y);
            unpack<EVEN>(x, p, c, H);
            unpack<EVEN>(y, e, c, H);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            p[j] = a.w_post ? p[j] : 1.0f;
            e[j] = a.scale ? e[j] : 1.0f;
        }
    };
    const auto new_group = [&]() {
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            float e[8];
            vectors(v, q[v], e);
#pragma unroll
            for (int j = 0; j < 8; ++j) q[v][j] *= e[j];
            if (a.gate) {
                unpack<EVEN>(xg[v], e, ((int64_t)v * NT + t) * 8, H);
                if constexpr (HOLD) cg = xg[v];
#pragma unroll
                for (int j = 0; j < 8; ++j) q[v][j] *= sig ? sigmoid(e[j]) : e[j];
            }
        }
    };
    // A += act B, and d_gate = scale w_post act' B to `to`
    const auto end_group = [&](T *to, float *to_part) {
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int64_t c = ((int64_t)v * NT + t) * 8;
            float f[8], p[8], e[8];
            if (!a.gate) {
#pragma unroll
                for (int j = 0; j < 8; ++j) A[v][j] += B[v][j];
            } else {
                Vec8<T> x = cg;
                if constexpr (!HOLD) fetch<EVEN>(x, static_cast<const T *>(a.gate) + group * a.ld_gate, c, H);
                unpack<EVEN>(x, f, c, H);
                vectors(v, p, e);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float act = sig ? sigmoid(f[j]) : f[j];
                    A[v][j] += act * B[v][j];
                    f[j] = e[j] * p[j] * (sig ? sigmoid_slope(f[j]) : 1.0f) * B[v][j];
                }
                if (to) put<EVEN>(f, to, c, H);
                if (to_part) put<EVEN>(f, to_part, c, H);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) B[v][j] = 0.0f;
        }
    };
    if (a.gate) ask_gate(group);
    if constexpr (HOLD) ask_vectors(0, wp, sc);
    ask(row);
#pragma unroll
    for (int v = 0; v < VPT; ++v)
        if (a.w_next) fetch<EVEN>(wn[v], static_cast<const T *>(a.w_next), ((int64_t)v * NT + t) * 8, H);
    new_group();
    while (true) {
        float d[VPT][8], xn[VPT][8], xb[VPT][8];
        float s[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            float g[8], w[8];
            const int64_t c = ((int64_t)v * NT + t) * 8;
            unpack<EVEN>(xo[v], d[v], c, H);
            unpack<EVEN>(xd[v], g, c, H);
            unpack<EVEN>(xr[v], xn[v], c, H);
            unpack<EVEN>(xk[v], xb[v], c, H);
            unpack<EVEN>(wn[v], w, c, H);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                xn[v][j] *= rr;
                xb[v][j] *= rb;
                N[v][j] += g[j] * xn[v][j];
                g[j] *= w[j];
                s[0] += g[j] * xn[v][j];
                d[v][j] += rr * g[j];
                const float qx = q[v][j] * xb[v][j];
                s[1] += d[v][j] * qx;
                s[2] += xn[v][j] * qx;
            }
        }
        const float rn = rr, rp = rb;
        const bool more = row + 1 < end, last = row + 1 == group_end;
        if (more) {
            ask(row + 1);
            if (a.gate && last) ask_gate(group + 1);
        }
        row_sums<WPR>(s, slot, turn);
        const float m = a.d_next ? rn * (s[0] * inv) : 0.0f;
        const float mb = a.w_post ? (s[1] - m * s[2]) * inv : 0.0f;
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int64_t c = ((int64_t)v * NT + t) * 8;
            float f[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                d[v][j] -= m * xn[v][j];
                B[v][j] += d[v][j] * xb[v][j];
                f[j] = rp * (d[v][j] * q[v][j] - xb[v][j] * mb);
            }
            put<EVEN>(d[v], static_cast<T *>(a.d_residual) + row * a.ld_d_residual, c, H);
            if (a.block) put<EVEN>(f, static_cast<T *>(a.d_block) + row * a.ld_d_block, c, H);
        }
        if (!more) break;
        ++row;
        if (last) {
            end_group(a.d_gate ? static_cast<T *>(a.d_gate) + group * H : nullptr, nullptr);
            ++group;
            group_end += cut.rows_per_group;
            if (a.gate) new_group();
        }
    }
    end_group(a.d_gate && cut.chunks == 1 ? static_cast<T *>(a.d_gate) + group * H : nullptr,
              a.d_gate && cut.chunks > 1 ? cs.gate_part + part * H : nullptr);
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        const int64_t c = ((int64_t)v * NT + t) * 8;
        float *to = cs.part + part * 3 * H;
        float p[8], e[8];
        vectors(v, p, e);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            e[j] *= A[v][j];
            p[j] *= A[v][j];
        }
        if (a.d_w_post) put<EVEN>(e, to, c, H);
        if (a.d_scale) put<EVEN>(p, to + H, c, H);
        if (a.d_w_next) put<EVEN>(N[v], to + 2 * H, c, H);
    }
}

// The same for rows too long for registers: sixteen waves read a row twice,
// for its sums and (from the L2) for its results, one column group after the
// other, and keep B and N in LDS and A in the part's row of the partial sums,
// each thread its own columns. (In registers they spill: 219 us for 1024 x
// 16384 bf16, against 72 here.)
template <class T, bool EVEN>
__global__ __launch_bounds__(1024) void norm_backward_long_kernel(gemm_norm_backward_args a, ColumnSums cs) {
    constexpr int WPR = 16, NT = 1024, VPT = GEMM_NORM_MAX_COLS / (NT * 8);
    __shared__ float slot[2][3][WPR];
    __shared__ float B[VPT * 8][NT], N[VPT * 8][NT];
    int turn = 0;
    const int t = threadIdx.x;
    const int64_t H = a.cols, part = blockIdx.x;
    const NormCut cut = cs.cut;
    const bool sig = a.gate_act == GEMM_EPI_SIGMOID;
    const float inv = 1.0f / (float)H;
    int64_t row, end;
    if (cut.chunks > 1) {
        const int64_t group = (uint32_t)part / (uint32_t)cut.chunks, chunk = part - group * cut.chunks;
        row = group * cut.rows_per_group + chunk * cut.rows_per_part;
        end = min(row + cut.rows_per_part, (group + 1) * cut.rows_per_group);
    } else {
        row = part * cut.groups_per_part * cut.rows_per_group;
        end = min(row + cut.groups_per_part * cut.rows_per_group, a.rows);
    }
    int64_t group = (uint32_t)row / (uint32_t)cut.rows_per_group, group_end = (group + 1) * cut.rows_per_group;
    float *const sums = cs.part + part * 3 * H;
    for (int v = 0; v < VPT; ++v) {
        const float zero[8] = {};
        put<EVEN>(zero, sums, ((int64_t)v * NT + t) * 8, H);
#pragma unroll
        for (int j = 0; j < 8; ++j) B[v * 8 + j][t] = N[v * 8 + j][t] = 0.0f;
    }
    const auto get = [&](const void *p, int64_t ld, int64_t r, int v, float *f, float none) {
        const int64_t c = ((int64_t)v * NT + t) * 8;
        Vec8<T> x = {};
        if (p) fetch<EVEN>(x, static_cast<const T *>(p) + r * ld, c, H);
        unpack<EVEN>(x, f, c, H);
        if (!p)
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = none;
    };
    const auto gate_of = [&](int v, float *act) {
        get(a.gate, a.ld_gate, group, v, act, 1.0f);
        if (a.gate && sig)
#pragma unroll
            for (int j = 0; j < 8; ++j) act[j] = sigmoid(act[j]);
    };
    // xn, xb, d_out + rstd_next g, q of a column group, and d_next (g before w_next)
    const auto values = [&](int v, float rr, float rb, float *xn, float *xb, float *d, float *q, float *dn) {
        float f[8];
        get(a.d_out, a.ld_d_out, row, v, d, 0.0f);
        get(a.d_next, a.ld_d_next, row, v, dn, 0.0f);
        get(a.d_next ? a.out : nullptr, a.ld_out, row, v, xn, 0.0f);
        get(a.block, a.ld_block, row, v, xb, 0.0f);
        gate_of(v, q);
        get(a.w_next, 0, 0, v, f, 0.0f);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            xn[j] *= rr;
            xb[j] *= rb;
            d[j] += rr * dn[j] * f[j];
        }
        get(a.w_post, 0, 0, v, f, 1.0f);
#pragma unroll
        for (int j = 0; j < 8; ++j) q[j] *= f[j];
        get(a.scale, 0, 0, v, f, 1.0f);
#pragma unroll
        for (int j = 0; j < 8; ++j) q[j] *= f[j];
    };
    const auto end_group = [&](T *to, float *to_part) {
#pragma unroll 1
        for (int v = 0; v < VPT; ++v) {
            const int64_t c = ((int64_t)v * NT + t) * 8;
            float gate[8], act[8], p[8], e[8];
            get(a.gate, a.ld_gate, group, v, gate, 1.0f);
            gate_of(v, act);
            get(a.w_post, 0, 0, v, p, 1.0f);
            get(a.scale, 0, 0, v, e, 1.0f);
            float A[8];
            Vec8<float> x = {};
            fetch<EVEN>(x, (const float *)sums, c, H);
            unpack<EVEN>(x, A, c, H);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float sum = B[v * 8 + j][t];
                A[j] += act[j] * sum;
                e[j] *= p[j] * (sig ? sigmoid_slope(gate[j]) : 1.0f) * sum;
                B[v * 8 + j][t] = 0.0f;
            }
            put<EVEN>(A, sums, c, H);
            if (to) put<EVEN>(e, to, c, H);
            if (to_part) put<EVEN>(e, to_part, c, H);
        }
    };
    for (; row < end; ++row) {
        const float rr = a.w_next ? a.rstd_next[row] : 0.0f, rb = a.w_post ? a.rstd_post[row] : 1.0f;
        float s[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll 1
        for (int v = 0; v < VPT; ++v) {
            float xn[8], xb[8], d[8], q[8], dn[8], w[8];
            values(v, rr, rb, xn, xb, d, q, dn);
            get(a.w_next, 0, 0, v, w, 0.0f);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                N[v * 8 + j][t] += dn[j] * xn[j];
                s[0] += dn[j] * w[j] * xn[j];
                s[1] += d[j] * q[j] * xb[j];
                s[2] += xn[j] * q[j] * xb[j];
            }
        }
        row_sums<WPR>(s, slot, turn);
        const float m = a.d_next ? rr * (s[0] * inv) : 0.0f;
        const float mb = a.w_post ? (s[1] - m * s[2]) * inv : 0.0f;
#pragma unroll 1
        for (int v = 0; v < VPT; ++v) {
            const int64_t c = ((int64_t)v * NT + t) * 8;
            float xn[8], xb[8], d[8], q[8], dn[8];
            values(v, rr, rb, xn, xb, d, q, dn);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                d[j] -= m * xn[j];
                B[v * 8 + j][t] += d[j] * xb[j];
                q[j] = rb * (d[j] * q[j] - xb[j] * mb);
            }
            put<EVEN>(d, static_cast<T *>(a.d_residual) + row * a.ld_d_residual, c, H);
            if (a.block) put<EVEN>(q, static_cast<T *>(a.d_block) + row * a.ld_d_block, c, H);
        }
        if (row + 1 == group_end || row + 1 == end) {
            end_group(a.d_gate && cut.chunks == 1 ? static_cast<T *>(a.d_gate) + group * H : nullptr,
                      a.d_gate && cut.chunks > 1 ? cs.gate_part + part * H : nullptr);
            ++group;
            group_end += cut.rows_per_group;
        }
    }
#pragma unroll 1
    for (int v = 0; v < VPT; ++v) {
        const int64_t c = ((int64_t)v * NT + t) * 8;
        float p[8], e[8], A[8];
        get(a.w_post, 0, 0, v, p, 1.0f);
        get(a.scale, 0, 0, v, e, 1.0f);
        Vec8<float> x = {};
        fetch<EVEN>(x, (const float *)sums, c, H);
        unpack<EVEN>(x, A, c, H);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            p[j] *= A[j];
            e[j] *= A[j];
            A[j] = N[v * 8 + j][t];
        }
        if (a.d_w_post) put<EVEN>(e, sums, c, H);
        if (a.d_scale) put<EVEN>(p, sums + H, c, H);
        if (a.d_w_next) put<EVEN>(A, sums + 2 * H, c, H);
    }
}

// out[c] = sum over n rows, `stride` apart, of the column partials, in row
// order within each of 16 interleaved strands and then in strand order. One
// workgroup per 64 columns of one output vector, four columns a thread.
template <class T>
__global__ __launch_bounds__(256) void norm_columns_kernel(gemm_norm_backward_args a, ColumnSums cs) {
    __shared__ float sum[16][64];
    const int64_t H = a.cols, blocks = (H + 63) / 64, job = blockIdx.x / blocks;
    const int lane = threadIdx.x & 15, strand = threadIdx.x >> 4;
    const int64_t c = (blockIdx.x - job * blocks) * 64 + lane * 4;
    const float *src;
    int64_t n, stride;
    T *dst;
    if (job < 3) {
        dst = static_cast<T *>(job == 0 ? a.d_w_post : job == 1 ? a.d_scale : a.d_w_next);
        if (!dst) return;
        src = cs.part + job * H;
        n = cs.cut.parts;
        stride = 3 * H;
    } else {
        dst = static_cast<T *>(a.d_gate) + (job - 3) * H;
        src = cs.gate_part + (job - 3) * cs.cut.chunks * H;
        n = cs.cut.chunks;
        stride = H;
    }
    f32x4 s{0, 0, 0, 0};
    if (c + 4 <= H) {
        typedef f32x4 f32x4_any __attribute__((aligned(4)));
#pragma unroll 8
        for (int64_t i = strand; i < n; i += 16)
            s += *reinterpret_cast<const f32x4_any *>(src + i * stride + c);
    } else if (c < H) {
        for (int64_t i = strand; i < n; i += 16)
            for (int j = 0; j < 4; ++j)
                if (c + j < H) s[j] += src[i * stride + c + j];
    }
    *reinterpret_cast<f32x4 *>(&sum[strand][lane * 4]) = s;
    __syncthreads();
    const int64_t col = (blockIdx.x - job * blocks) * 64 + threadIdx.x;
    if (threadIdx.x < 64 && col < H) {
        float v = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) v += sum[i][threadIdx.x];
        dst[col] = from_f<T>(v);
    }
}

template <class T, bool EVEN>
void forward(const gemm_norm_args &a, hipStream_t st) {
    // A workgroup walks over rows where there are more than per_cu workgroups of
    // rows a CU, one to two and a half times what the registers let it hold at once
    // (two of the four with 8192 columns). One row a workgroup: 82 us against 51 for
    // 4096 x 8192 bf16.
    const auto grid = [&](int rpb, int per_cu) {
        const int64_t wgs = (a.rows + rpb - 1) / rpb;
        return (unsigned)(wgs < 256 * per_cu ? wgs : 256 * per_cu);
    };
    if (a.cols <= 512) norm_forward_kernel<T, 1, 1, EVEN><<<grid(4, 8), 256, 0, st>>>(a);
    else if (a.cols <= 1024) norm_forward_kernel<T, 1, 2, EVEN><<<grid(4, 4), 256, 0, st>>>(a);
    else if (a.cols <= 2048) norm_forward_kernel<T, 4, 1, EVEN><<<grid(1, 8), 256, 0, st>>>(a);
    else if (a.cols <= 4096) norm_forward_kernel<T, 4, 2, EVEN><<<grid(1, 8), 256, 0, st>>>(a);
    else if (a.cols <= 8192) norm_forward_kernel<T, 8, 2, EVEN><<<grid(1, 4), 512, 0, st>>>(a);
    else norm_forward_kernel<T, 16, 2, EVEN><<<grid(1, 1), 1024, 0, st>>>(a);
}

template <class T, bool EVEN>
void backward_rows(const gemm_norm_backward_args &a, const ColumnSums &cs, hipStream_t st) {
    const unsigned parts = (unsigned)cs.cut.parts;
    if (a.cols <= 512) norm_backward_kernel<T, 1, 1, EVEN><<<parts, 64, 0, st>>>(a, cs);
    else if (a.cols <= 1024) norm_backward_kernel<T, 2, 1, EVEN><<<parts, 128, 0, st>>>(a, cs);
    else if (a.cols <= 2048) norm_backward_kernel<T, 4, 1, EVEN><<<parts, 256, 0, st>>>(a, cs);
    else if (a.cols <= 4096) norm_backward_kernel<T, 4, 2, EVEN><<<parts, 256, 0, st>>>(a, cs);
    else if (a.cols <= 8192) norm_backward_kernel<T, 8, 2, EVEN><<<parts, 512, 0, st>>>(a, cs);
    else norm_backward_long_kernel<T, EVEN><<<parts, 1024, 0, st>>>(a, cs);
}

template <class T>
hipError_t backward(const gemm_norm_backward_args &a, hipStream_t st) {
    ColumnSums cs;
    cs.cut = norm_cut(a.rows, a.cols, a.gate ? a.gate_rows : 1);
    cs.part = static_cast<float *>(a.workspace);
    cs.gate_part = cs.part + cs.cut.parts * 3 * a.cols;
    if (cs.cut.parts > 0) {
        if (a.cols % 8 == 0) backward_rows<T, true>(a, cs, st);
        else backward_rows<T, false>(a, cs, st);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    const int64_t gates = a.d_gate && cs.cut.chunks != 1 ? a.gate_rows : 0;
    if (!a.d_w_post && !a.d_scale && !a.d_w_next && gates == 0) return hipSuccess;
    const int64_t grid = (3 + gates) * ((a.cols + 63) / 64);
    norm_columns_kernel<T><<<(unsigned)grid, 256, 0, st>>>(a, cs);
    return hipGetLastError();
}

}  // namespace

NormCut norm_cut(int64_t rows, int64_t cols, int64_t gate_rows) {
    NormCut c;
    c.rows_per_group = rows > 0 ? rows / (gate_rows > 0 ? gate_rows : 1) : 0;
    if (rows == 0) {
        c.parts = 0;
        c.rows_per_part = 0;
        c.chunks = 0;   // every sum is over nothing
        c.groups_per_part = 1;
        return c;
    }
    // 16 or fewer waves a CU, which the loads ahead keep busy: twice the parts
    // write twice the partial sums and took 51 + 11 us against 42 + 5 (rows and
    // columns kernel, 4096 x 4096 bf16), 50 + 7 against 40 + 5 (8192 x 2048), but
    // 22 + 5 against 26 + 4 (8192 x 1024, two waves a part).
    const int64_t most = cols > 2048 ? 256 : cols > 1024 ? 512 : 1024;
    int64_t R = (rows + most - 1) / most;
    if (R < 2) R = 2;
    if (c.rows_per_group > R) {
        c.rows_per_part = R;
        c.chunks = (c.rows_per_group + R - 1) / R;
        c.groups_per_part = 1;
        c.parts = gate_rows * c.chunks;
    } else {
        c.chunks = 1;
        c.groups_per_part = R / c.rows_per_group;
        c.rows_per_part = c.groups_per_part * c.rows_per_group;
        c.parts = (gate_rows + c.groups_per_part - 1) / c.groups_per_part;
    }
    return c;
}

hipError_t launch_norm_forward(const gemm_norm_args &a, hipStream_t st) {
    const bool even = a.cols % 8 == 0;
    if (a.type == GEMM_F32) even ? forward<float, true>(a, st) : forward<float, false>(a, st);
    else if (a.type == GEMM_F16) even ? forward<_Float16, true>(a, st) : forward<_Float16, false>(a, st);
    else even ? forward<__bf16, true>(a, st) : forward<__bf16, false>(a, st);
    return hipGetLastError();
}

hipError_t launch_norm_backward(const gemm_norm_backward_args &a, hipStream_t st) {
    if (a.type == GEMM_F32) return backward<float>(a, st);
    if (a.type == GEMM_F16) return backward<_Float16>(a, st);
    return backward<__bf16>(a, st);
}

}  // namespace mg
