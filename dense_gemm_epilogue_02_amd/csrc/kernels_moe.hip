// kernels_moe.hip -- a mixture-of-experts layer for a few tokens.
//
// Bound by the one read of every chosen expert's weights. Three launches:
// the router (logits, the choice, the experts' token lists), the gate and up
// products with their activation, and the down product with the weighted sum
// over a token's experts.
#include "block.hpp"

namespace mg {

namespace {

constexpr int RT = 4;   // tokens per router workgroup, one wave each for the choice

// The workspace's state words.
enum { ST_CHUNK = 0, ST_DONE = GEMM_MOE_MAX_TOKENS / RT };
static_assert((ST_DONE + 1) * 4 <= GEMM_MOE_STATE_BYTES, "state words");

struct Active {
    int expert, first, count, pad;   // its slots are slots[first .. first + count)
};

struct Ws {
    unsigned *state;
    double *logits;   // [T][E]
    int *ids;         // [T][k]
    float *probs;     // [T][k]
    int *pos;         // [T][k]: the slot's place in `slots`, -1 for masked tokens
    int *slots;       // token * k + choice, ordered by expert
    int *n_active;    // then the list
    Active *active;
    char *h;          // [T * k][ip] activations, by place
    int64_t ip;
};

__host__ __device__ inline Ws moe_ws(char *p, const MoeLayout &l) {
    Ws w;
    w.state = reinterpret_cast<unsigned *>(p);
    w.logits = reinterpret_cast<double *>(p + l.logits);
    w.ids = reinterpret_cast<int *>(p + l.ids);
    w.probs = reinterpret_cast<float *>(p + l.probs);
    w.pos = reinterpret_cast<int *>(p + l.pos);
    w.slots = reinterpret_cast<int *>(p + l.slots);
    w.n_active = reinterpret_cast<int *>(p + l.active);
    w.active = reinterpret_cast<Active *>(p + l.active + 16);
    w.h = p + l.h;
    w.ip = l.ip;
    return w;
}

// True in the workgroup that arrives last of n; its reads then see what the
// others wrote. The counter is left zero. Nobody waits.
__device__ __forceinline__ bool last_of(unsigned *counter, unsigned n, int *flag) {
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) {
        const unsigned old =
            __hip_atomic_fetch_add(counter, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT);
        *flag = old == n - 1;
        if (old == n - 1)
            __hip_atomic_store(counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    __syncthreads();
    const bool last = *flag != 0;
    __syncthreads();
    if (last) __threadfence();
    return last;
}

__device__ __forceinline__ double shfl_xor_d(double v, int o) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __shfl_xor((int)(uint32_t)b, o), hi = __shfl_xor((int)(b >> 32), o);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ int64_t shfl_xor_l(int64_t v, int o) {
    const uint32_t lo = __shfl_xor((int)(uint32_t)v, o), hi = __shfl_xor((int)(v >> 32), o);
    return (int64_t)((uint64_t)hi << 32 | lo);
}

// An integer that orders like the number; NaN below every number, both zeros alike.
__device__ __forceinline__ int64_t order_key(double v) {
    if (v != v) return INT64_MIN;
    const int64_t b = __builtin_bit_cast(int64_t, v + 0.0);
    return b < 0 ? (b ^ INT64_MAX) : b;
}

// ---- router ---------------------------------------------------------------------
//
// l[t][e] = sum_h x[t][h] router[e][h] in 64 bits: products of 16-bit values
// are exact there and the sum's order no longer decides between experts that
// are close. A wave takes one expert and RT tokens; the workgroup that
// completes a chunk of tokens chooses for it (a wave per token), and the one
// that completes the last chunk builds the experts' lists.
template <class T>
__global__ __launch_bounds__(256) void moe_router_kernel(MoeArgs a, MoeLayout lay) {
    __shared__ int flag;
    __shared__ int count[GEMM_MOE_MAX_EXPERTS], first[GEMM_MOE_MAX_EXPERTS];
    const Ws w = moe_ws(a.ws, lay);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int e = blockIdx.x * 4 + wave, t0 = blockIdx.y * RT;
    if (e < a.E) {
        double acc[RT] = {};
        const T *rp = static_cast<const T *>(a.router) + (int64_t)e * a.H;
        for (int64_t h = lane * 8; h < a.H; h += 512) {
            float f[8], g[8];
            Vec8<T> v;
            v.load(rp + h, a.H - h);
            v.get(f);
#pragma unroll
            for (int i = 0; i < RT; ++i) {
                const int t = min(t0 + i, a.T - 1);
                v.load(static_cast<const T *>(a.x) + t * a.ldx + h, a.H - h);
                v.get(g);
#pragma unroll
                for (int j = 0; j < 8; ++j) acc[i] = __builtin_fma((double)f[j], (double)g[j], acc[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < RT; ++i) {
#pragma unroll
            for (int o = 32; o > 0; o >>= 1) acc[i] += shfl_xor_d(acc[i], o);
            if (lane == 0 && t0 + i < a.T) w.logits[(int64_t)(t0 + i) * a.E + e] = acc[i];
        }
    }
    if (!last_of(w.state + ST_CHUNK + blockIdx.y, gridDim.x, &flag)) return;

    constexpr int PER = GEMM_MOE_MAX_EXPERTS / 64;
    const int t = t0 + wave;
    if (t < a.T) {
        const bool live = !a.mask || a.mask[t] != 0;
        double l[PER];
        int64_t key[PER];
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int x = i * 64 + lane;
            l[i] = x < a.E ? w.logits[(int64_t)t * a.E + x] : 0.0;
            key[i] = x < a.E ? order_key(l[i]) : INT64_MIN;
        }
        unsigned taken = 0;   // bit i: expert i * 64 + lane is chosen already
        double top = 0.0, mine = 0.0;   // the largest l; the choice of rank `lane`
        int id = -1;
        for (int j = 0; j < a.k; ++j) {
            int64_t best = INT64_MIN;
            int at = INT32_MAX;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int x = i * 64 + lane;
                if (x < a.E && !(taken >> i & 1) && (at == INT32_MAX || key[i] > best)) {
                    best = key[i];
                    at = x;
                }
            }
#pragma unroll
            for (int o = 32; o > 0; o >>= 1) {
                const int64_t ob = shfl_xor_l(best, o);
                const int oa = __shfl_xor(at, o);
                if (oa != INT32_MAX && (at == INT32_MAX || ob > best || (ob == best && oa < at))) {
                    best = ob;
                    at = oa;
                }
            }
            double v = 0.0;
#pragma unroll
            for (int i = 0; i < PER; ++i) v = (at >> 6) == i ? l[i] : v;
            const uint64_t vb = __builtin_bit_cast(uint64_t, v);
            const uint32_t lo = __shfl((int)(uint32_t)vb, at & 63), hi = __shfl((int)(vb >> 32), at & 63);
            v = __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
            if (lane == (at & 63)) taken |= 1u << (at >> 6);
            if (j == 0) top = v;
            if (lane == j) {
                mine = v;
                id = at;
            }
        }
        const double p = lane < a.k ? exp(mine - top) : 0.0;
        double sum = p;
        if (!a.renorm) {
            sum = 0.0;
#pragma unroll
            for (int i = 0; i < PER; ++i)
                if (i * 64 + lane < a.E) sum += exp(l[i] - top);
        }
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) sum += shfl_xor_d(sum, o);
        if (lane < a.k) {
            const int i = t * a.k + lane;
            const int out_id = live ? id : -1;
            const float out_p = live ? (float)(p / sum) : 0.0f;
            w.ids[i] = out_id;
            w.probs[i] = out_p;
            if (a.ids) a.ids[i] = out_id;
            if (a.probs) a.probs[i] = out_p;
        }
    }
    if (!last_of(w.state + ST_DONE, gridDim.y, &flag)) return;

    // Lists: an expert's slots stand together. The order within an expert is
    // that of the atomics and changes no result: a slot's products do not
    // depend on its place.
    for (int i = threadIdx.x; i < a.E; i += 256) count[i] = 0;
    __syncthreads();
    const int n = a.T * a.k;
    for (int i = threadIdx.x; i < n; i += 256)
        if (w.ids[i] >= 0) atomicAdd(&count[w.ids[i]], 1);
    __syncthreads();
    if (wave == 0) {
        int base = 0, actives = 0;
        for (int b = 0; b < a.E; b += 64) {
            const int x = b + lane, c = x < a.E ? count[x] : 0;
            int run = c, act = c > 0;
#pragma unroll
            for (int o = 1; o < 64; o <<= 1) {
                const int r = __shfl_up(run, o), q = __shfl_up(act, o);
                if (lane >= o) {
                    run += r;
                    act += q;
                }
            }
            if (x < a.E) first[x] = base + run - c;
            if (c > 0) w.active[actives + act - 1] = Active{x, base + run - c, c, 0};
            base += __shfl(run, 63);
            actives += __shfl(act, 63);
        }
        if (lane == 0) *w.n_active = actives;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += 256) {
        const int id = w.ids[i];
        int at = -1;
        if (id >= 0) {
            at = atomicAdd(&first[id], 1);
            w.slots[at] = i;
        }
        w.pos[i] = at;
    }
}

// ---- the products ------------------------------------------------------------------
//
// v_mfma 16x16x32 with 16 weight rows as operand A and 16 tokens as operand B:
// a lane (r, g) supplies 8 k of weight row r and of token r, and ends with four
// consecutive rows of one token. Weights go from memory straight to operand
// registers: a lane group takes consecutive k of a unit (64 k of 16-bit
// weights, 256 k of MXFP4 ones: a 128-byte line per row), the same ones for
// both operands, so the order of k inside a unit is free.
template <class T> __device__ __forceinline__ f32x4 mma16(u32x4 a, u32x4 b, f32x4 c);
template <> __device__ __forceinline__ f32x4 mma16<__bf16>(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}
template <> __device__ __forceinline__ f32x4 mma16<_Float16>(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                  __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// Rows of 16-bit weights.
template <class T> struct Rows16 {
    static constexpr int UK = 64, NF = 2, LK = 16;   // k per unit; fragments; k per lane and unit
    const T *p;
    u32x4 f[NF];
    __device__ __forceinline__ void at(const void *base, const uint8_t *, int64_t row, int64_t K) {
        p = static_cast<const T *>(base) + row * K;
    }
    // n: how many of the lane's k exist (anything >= LK: all)
    __device__ __forceinline__ void load(int64_t u, int g, int64_t n) {
        const T *q = p + u * UK + g * LK;
        Vec8<T> v;
#pragma unroll
        for (int j = 0; j < NF; ++j) {
            v.load(q + 8 * j, n - 8 * j);
            f[j] = v.w[0];
        }
    }
    __device__ __forceinline__ void load_full(int64_t u, int g) {
        const u32x4_any *q = reinterpret_cast<const u32x4_any *>(p + u * UK + g * LK);
#pragma unroll
        for (int j = 0; j < NF; ++j) f[j] = q[j];
    }
    __device__ __forceinline__ u32x4 frag(int j) const { return f[j]; }
};

// Rows of MXFP4 weights (their padding holds zeros, so no load is cut). An
// element times its block's scale is exact in bf16.
struct Rows4 {
    static constexpr int UK = 256, NF = 8, LK = 64;
    const uint8_t *p, *s;
    u32x4 c[2];
    uint32_t sc;
    __device__ __forceinline__ void at(const void *base, const uint8_t *scales, int64_t row,
                                       int64_t K) {
        const int64_t kp = mx4_kp(K);
        p = static_cast<const uint8_t *>(base) + row * (kp / 2);
        s = scales + row * (kp / 32);
    }
    __device__ __forceinline__ void load_full(int64_t u, int g) {
        const u32x4 *q = reinterpret_cast<const u32x4 *>(p + u * 128 + g * 32);
        c[0] = q[0];
        c[1] = q[1];
        sc = *reinterpret_cast<const uint16_t *>(s + u * 8 + g * 2);
    }
    __device__ __forceinline__ void load(int64_t u, int g, int64_t) { load_full(u, g); }
    __device__ __forceinline__ u32x4 frag(int j) const {
        typedef __attribute__((ext_vector_type(2))) __bf16 b2;
        const uint32_t q = c[j >> 2][j & 3];
        const float s = mx4_scale_value(j < 4 ? (sc & 255u) : (sc >> 8));
        const b2 x = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, s, 0),
                 y = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, s, 1),
                 z = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, s, 2),
                 v = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, s, 3);
        return u32x4{__builtin_bit_cast(uint32_t, x), __builtin_bit_cast(uint32_t, y),
                     __builtin_bit_cast(uint32_t, z), __builtin_bit_cast(uint32_t, v)};
    }
};

// acc[mt][m] += 16 rows of each of NM weight matrices times MT x 16 tokens, over
// the units first, first + step, ... of K.
template <class T, class R, int MT, int NM>
__device__ __forceinline__ void multiply(R *w, const T *const *xp, int64_t K, int first, int step,
                                         int g, f32x4 (*acc)[NM]) {
    const int64_t full = K / R::UK, units = (K + R::UK - 1) / R::UK;
    int64_t u = first;
#pragma unroll 2
    for (; u < full; u += step) {
#pragma unroll
        for (int m = 0; m < NM; ++m) w[m].load_full(u, g);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            const u32x4_any *q =
                reinterpret_cast<const u32x4_any *>(xp[mt] + u * R::UK + g * R::LK);
#pragma unroll
            for (int j = 0; j < R::NF; ++j) {
                const u32x4 b = q[j];
#pragma unroll
                for (int m = 0; m < NM; ++m) acc[mt][m] = mma16<T>(w[m].frag(j), b, acc[mt][m]);
            }
        }
    }
    if (u < units) {   // the unit that K ends in
        const int64_t k = u * R::UK + g * R::LK;
#pragma unroll
        for (int m = 0; m < NM; ++m) w[m].load(u, g, K - k);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
            for (int j = 0; j < R::NF; ++j) {
                Vec8<T> v;
                v.load(xp[mt] + (k < K ? k : 0) + 8 * j, K - k - 8 * j);
#pragma unroll
                for (int m = 0; m < NM; ++m)
                    acc[mt][m] = mma16<T>(w[m].frag(j), v.w[0], acc[mt][m]);
            }
        }
    }
}

// h = silu(g) u for 16 rows of the gate and of the up matrix and every token of
// one expert: a workgroup per (active expert, 16 rows), its waves share K.
constexpr int UP_W = 4;
template <class T, class R, int MT>
__device__ __forceinline__ void up_body(const MoeArgs &a, const Ws &w, const Active &x, int64_t i0,
                                        int mt0, float (*part)[GEMM_MOE_MAX_TOKENS][33]) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15, g = lane >> 4;
    R wt[2];
    const int64_t row = min(i0 + r, a.I - 1);
    wt[0].at(a.up, a.up_s, (int64_t)x.expert * 2 * a.I + row, a.H);
    wt[1].at(a.up, a.up_s, (int64_t)x.expert * 2 * a.I + a.I + row, a.H);
    const T *xp[MT];
    f32x4 acc[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        const int s = w.slots[x.first + min((mt0 + mt) * 16 + r, x.count - 1)];
        xp[mt] = static_cast<const T *>(a.x) + (int64_t)(s / a.k) * a.ldx;
        acc[mt][0] = acc[mt][1] = f32x4{0, 0, 0, 0};
    }
    multiply<T, R, MT, 2>(wt, xp, a.H, wave, UP_W, g, acc);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i) part[wave][mt * 16 + r][m * 16 + g * 4 + i] = acc[mt][m][i];
    __syncthreads();
    T *h = reinterpret_cast<T *>(w.h);
    for (int i = threadIdx.x; i < MT * 256; i += UP_W * 64) {
        const int n = i & 15, tok = i >> 4, p = mt0 * 16 + tok;
        if (p >= x.count || i0 + n >= w.ip) continue;
        float gate = 0.0f, up = 0.0f;
#pragma unroll
        for (int v = 0; v < UP_W; ++v) {
            gate += part[v][tok][n];
            up += part[v][tok][16 + n];
        }
        const float y = i0 + n < a.I ? gate / (1.0f + __expf(-gate)) * up : 0.0f;
        h[(int64_t)(x.first + p) * w.ip + i0 + n] = from_f<T>(y);
    }
}

template <class T, class R>
__global__ __launch_bounds__(UP_W * 64) void moe_up_kernel(MoeArgs a, MoeLayout lay, int blocks) {
    __shared__ float part[UP_W][GEMM_MOE_MAX_TOKENS][33];
    const Ws w = moe_ws(a.ws, lay);
    const int at = blockIdx.x / blocks;
    if (at >= *w.n_active) return;
    const Active x = w.active[at];
    const int64_t i0 = (int64_t)(blockIdx.x - at * blocks) * 16;
    if (x.count <= 16) up_body<T, R, 1>(a, w, x, i0, 0, part);
    else if (x.count <= 32) up_body<T, R, 2>(a, w, x, i0, 0, part);
    else up_body<T, R, 4>(a, w, x, i0, 0, part);
}

// out[t] = sum over the token's experts of p down[e] h: a workgroup per 16
// rows of out's columns, a wave per active expert (per share of its K, where
// there are fewer experts than waves). Every slot's product stands in LDS once
// per share; the sum over shares and experts is in a fixed order.
constexpr int DOWN_W = 8;
template <class T, class R, int MT>
__device__ __forceinline__ void down_body(const MoeArgs &a, const Ws &w, const Active &x, int64_t n0,
                                          int share, int shares, float (*y)[16]) {
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    R wt[1];
    wt[0].at(a.down, a.down_s, (int64_t)x.expert * a.H + min(n0 + r, a.H - 1), a.I);
    const T *xp[MT];
    f32x4 acc[MT][1];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        xp[mt] = reinterpret_cast<const T *>(w.h) +
                 (int64_t)(x.first + min(mt * 16 + r, x.count - 1)) * w.ip;
        acc[mt][0] = f32x4{0, 0, 0, 0};
    }
    multiply<T, R, MT, 1>(wt, xp, a.I, share, shares, g, acc);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
        if (mt * 16 + r < x.count)
            *reinterpret_cast<f32x4 *>(&y[x.first + mt * 16 + r][g * 4]) = acc[mt][0];
}

template <class T, class R>
__global__ __launch_bounds__(DOWN_W * 64) void moe_down_kernel(MoeArgs a, MoeLayout lay) {
    extern __shared__ __align__(16) float y_lds[];
    float(*y)[16] = reinterpret_cast<float(*)[16]>(y_lds);
    const Ws w = moe_ws(a.ws, lay);
    const int wave = threadIdx.x >> 6, n_active = *w.n_active, slots = a.T * a.k;
    const int64_t n0 = (int64_t)blockIdx.x * 16;
    const int shares = n_active > 0 ? max(1, DOWN_W / n_active) : 1;
    for (int i = wave; i < n_active * shares; i += DOWN_W) {
        const int share = i / n_active;
        const Active x = w.active[i - share * n_active];
        float(*ys)[16] = y + share * slots;
        if (x.count <= 16) down_body<T, R, 1>(a, w, x, n0, share, shares, ys);
        else if (x.count <= 32) down_body<T, R, 2>(a, w, x, n0, share, shares, ys);
        else down_body<T, R, 4>(a, w, x, n0, share, shares, ys);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < a.T * 16; i += DOWN_W * 64) {
        const int n = i & 15, t = i >> 4;
        if (n0 + n >= a.H) continue;
        float v = 0.0f;
        for (int j = 0; j < a.k; ++j) {
            const int p = w.pos[t * a.k + j];
            if (p < 0) continue;
            float d = 0.0f;
            for (int s = 0; s < shares; ++s) d += y[s * slots + p][n];
            v += w.probs[t * a.k + j] * d;
        }
        static_cast<T *>(a.out)[t * a.ldo + n0 + n] = from_f<T>(v);
    }
}

template <class T, class R>
hipError_t run(const MoeArgs &a, hipStream_t st) {
    const MoeLayout lay = moe_layout(a.H, a.I, a.E, a.k, a.T);
    const dim3 rg((a.E + 3) / 4, (a.T + RT - 1) / RT);
    moe_router_kernel<T><<<rg, 256, 0, st>>>(a, lay);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int most = a.T * a.k < a.E ? a.T * a.k : a.E;
    const int64_t blocks = (lay.ip + 15) / 16;
    if (blocks * most > 0x7FFFFFFF) return hipErrorInvalidConfiguration;
    if (blocks > 0)
        moe_up_kernel<T, R><<<(unsigned)(blocks * most), UP_W * 64, 0, st>>>(a, lay, (int)blocks);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (a.H == 0) return hipSuccess;
    // active experts >= k wherever a token is routed, so shares <= max(1, W / k)
    const int shares = a.k < DOWN_W ? DOWN_W / a.k : 1;
    const size_t lds = (size_t)shares * a.T * a.k * 16 * sizeof(float);
    moe_down_kernel<T, R><<<(unsigned)((a.H + 15) / 16), DOWN_W * 64, lds, st>>>(a, lay);
    return hipGetLastError();
}

}  // namespace

MoeLayout moe_layout(int64_t H, int64_t I, int E, int k, int T) {
    MoeLayout l;
    int64_t at = GEMM_MOE_STATE_BYTES;
    const auto take = [&](int64_t bytes) {
        const int64_t p = at;
        at += (bytes + 15) / 16 * 16;
        return p;
    };
    const int64_t n = (int64_t)T * k;
    l.ip = (I + 7) / 8 * 8;
    l.logits = take((int64_t)T * E * 8);
    l.ids = take(n * 4);
    l.probs = take(n * 4);
    l.pos = take(n * 4);
    l.slots = take(n * 4);
    l.active = take(16 + (int64_t)(n < E ? n : E) * 16);
    l.h = take(n * l.ip * 2);
    l.total = at;
    return l;
}

hipError_t launch_moe(int type, int weight_type, const MoeArgs &a, hipStream_t st) {
    if (weight_type == GEMM_F4_E2M1) return run<__bf16, Rows4>(a, st);
    if (type == GEMM_F16) return run<_Float16, Rows16<_Float16>>(a, st);
    return run<__bf16, Rows16<__bf16>>(a, st);
}

}  // namespace mg
