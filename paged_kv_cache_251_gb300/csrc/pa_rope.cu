// Rotary positions, alone and fused with the KV append.
//
// y_a = m (x_a cos t - x_b sin t), y_b = m (x_b cos t + x_a sin t) with
// t = position * freq_i.  The angle is kept as a fraction of a turn in 64-bit
// fixed point: freq_i / 2 pi is a 0.64 fraction, formed from the caller's double
// with 1 / 2 pi in two doubles (one alone is off by 2^-54 relative: 2^-25 turn at
// position 2^31), and position times it wraps modulo one turn exactly.  No 64-bit
// floating arithmetic runs per position.  The fraction is off by 2^-64 turn a
// position (two roundings), its top 32 bits by 2^-33: within 2^-31 turn at every
// position.  They go to sincospif as a signed fraction in [-1/2, 1/2) turn, with
// one fp32 rounding.
//
// The rows are read once and written once: HBM-bound, or launch-bound for a
// decode step.  A CTA takes `tok` tokens.  It first forms their rot / 2
// (cos, sin) pairs once, in shared memory (every head of a token shares them).
// Its threads are x lanes by y rows: lane x of a row holds E elements of both
// halves (or E adjacent ones, interleaved), or E of the elements past rot.  They
// walk the CTA's rows (every token's q, k and v rows in order) y at a time,
// kRopeUnroll rows' loads before the first is used.
//
// Measured: 16384 tokens of 40 + 40 heads of 128, fp16, adjacent pairs: 153 us,
// 6.6 TB/s of the bytes read and written (a plain copy of them takes 148 us).  Small
// CTAs do best (128 threads, about 128 rows; 256 threads and 8 tokens: 172 us), as
// do streaming stores (-10 us) and three rows in flight (four: +1 us, six: +7).
// 512 tokens of 32 + 8 heads, bf16: 11 us.  A decode step's call is bound by its
// launch.
#include <cuda_runtime.h>

#include "pa_device.cuh"
#include "pa_host.h"
#include "pa_internal.h"
#include "pa_rope.h"

namespace pa {

namespace {

constexpr int kRopeThreads = 128;
constexpr int kRopeMaxTok = 8;

__device__ inline float load_f(const float *p) { return *p; }
__device__ inline float load_f(const __half *p) { return __half2float(*p); }
__device__ inline float load_f(const __nv_bfloat16 *p) { return __bfloat162float(*p); }
__device__ inline void store_f(float *p, float v) { *p = v; }
__device__ inline void store_f(__half *p, float v) { *p = __float2half_rn(v); }
__device__ inline void store_f(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }

// E consecutive elements of T: one 16-byte access when E fills it, else one
// element (E == 1).
template <typename T, int E> struct Vec {
    uint4 r;
    __device__ inline void load(const T *p) { r = *reinterpret_cast<const uint4 *>(p); }
    // (not read again soon, for the most part: the lines may leave the cache first)
    __device__ inline void store(T *p) const { __stcs(reinterpret_cast<uint4 *>(p), r); }
    __device__ inline void get(float *f) const { Elt<T>::unpack(r, f); }
    __device__ inline void set(const float *f) {
        T *t = reinterpret_cast<T *>(&r);
#pragma unroll
        for (int i = 0; i < E; ++i)
            store_f(t + i, f[i]);
    }
};
template <typename T> struct Vec<T, 1> {
    T r;
    __device__ inline void load(const T *p) { r = *p; }
    __device__ inline void store(T *p) const { *p = r; }
    __device__ inline void get(float *f) const { f[0] = load_f(&r); }
    __device__ inline void set(const float *f) { store_f(&r, f[0]); }
};

// Lanes of a row: the pair lanes, then the lanes that copy the elements past
// rot.  Half layout: a pair lane holds elements [E x, E x + E) of both halves.
// Interleaved: E / 2 adjacent pairs (one pair when E == 1), in `P` elements.
template <int E, bool Inter> struct RopeUnit {
    static constexpr int kPairs = Inter ? (E == 1 ? 1 : E / 2) : E;  // pairs of a pair lane
};

constexpr int kRopeUnroll = 3;

// A lane's share of a row, loaded; its rotation or copy, stored.
template <typename T, int E, bool Inter> struct RowUnit {
    Vec<T, E> a, b;  // b: half layout, the second half's elements; interleaved with E == 1, the odd element
    __device__ inline void load(const T *src, int x, int half, bool pair, int copy_at) {
        if (!pair) {
            a.load(src + copy_at);
        } else if constexpr (!Inter) {
            a.load(src + x * E);
            b.load(src + half + x * E);
        } else if constexpr (E == 1) {
            a.load(src + 2 * x);
            b.load(src + 2 * x + 1);
        } else {
            a.load(src + x * E);
        }
    }
    __device__ inline void store(T *dst, int x, int half, bool pair, int copy_at) const {
        if (!pair) {
            a.store(dst + copy_at);
        } else if constexpr (!Inter) {
            a.store(dst + x * E);
            b.store(dst + half + x * E);
        } else if constexpr (E == 1) {
            a.store(dst + 2 * x);
            b.store(dst + 2 * x + 1);
        } else {
            a.store(dst + x * E);
        }
    }
    // trig: (cos, sin) of the unit's pairs
    __device__ inline void rotate(const float2 *trig) {
        constexpr int P = RopeUnit<E, Inter>::kPairs;
        if constexpr (!Inter || E == 1) {
            float fa[E], fb[E], ya[E], yb[E];
            a.get(fa);
            b.get(fb);
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const float2 cs = trig[i];
                ya[i] = fa[i] * cs.x - fb[i] * cs.y;
                yb[i] = fb[i] * cs.x + fa[i] * cs.y;
            }
            a.set(ya);
            b.set(yb);
        } else {
            float f[E], y[E];
            a.get(f);
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const float2 cs = trig[i];
                y[2 * i] = f[2 * i] * cs.x - f[2 * i + 1] * cs.y;
                y[2 * i + 1] = f[2 * i + 1] * cs.x + f[2 * i] * cs.y;
            }
            a.set(y);
        }
    }
};

template <typename T, int E, bool Inter>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeParams p) {
    constexpr int P = RopeUnit<E, Inter>::kPairs;
    pdl_launch_dependents();
    extern __shared__ __align__(16) float2 trig[];  // [tok][rot / 2]
    __shared__ long long place[kRopeMaxTok];        // cache element of a token's first kv head; -1: not appended
    pdl_wait();
    const int half = p.rot / 2;
    const long long tok0 = static_cast<long long>(blockIdx.x) * p.tok;
    const int ntok = static_cast<int>(min(static_cast<long long>(p.tok), p.num_tokens - tok0));
    // thread: pair j of every groups-th token (its frequency is turned into a
    // fraction once: 64-bit floating operations are scarce here)
    const int groups = kRopeThreads / half, j = threadIdx.x % half;
    if (static_cast<int>(threadIdx.x) < groups * half) {
        // a fraction of a turn per position, in units of 2^-64 turn: the product with 1 / 2 pi,
        // its whole turns taken off (exactly), and what its rounding and the constant's left
        constexpr double kTurn = 0.15915494309189535, kTurnRest = -9.839338337591243e-18, kUnits = 18446744073709551616.0;
        const double freq = p.freqs[j], turns = freq * kTurn;
        const double rest = fma(freq, kTurnRest, fma(freq, kTurn, -turns));
        const unsigned long long frac = static_cast<unsigned long long>(__double2ll_rn((turns - rint(turns)) * kUnits)) +
                                        static_cast<unsigned long long>(__double2ll_rn(rest * kUnits));
        for (int t = threadIdx.x / half; t < ntok; t += groups) {
            const long long pos = static_cast<long long>(p.positions[tok0 + t]) * p.direction;
            const unsigned long long angle = frac * static_cast<unsigned long long>(pos);
            float sn, cs;
            sincospif(static_cast<float>(static_cast<int>((angle + 0x80000000ull) >> 32)) * 4.656612873077393e-10f,
                      &sn, &cs);
            trig[t * half + j] = make_float2(cs * p.mscale, sn * p.mscale);
        }
    }
    const long long step = static_cast<long long>(p.block_size) * p.head_dim;  // kv head to kv head
    if (p.num_kv_heads && threadIdx.x < ntok) {
        const long long slot = p.slots[tok0 + threadIdx.x];
        long long at = -1;
        if (slot >= static_cast<long long>(p.num_blocks) * p.block_size) {
            if (p.err)
                atomicOr(p.err, PA_DEVERR_BAD_SLOT);
        } else if (slot >= 0) {
            const long long phys = slot / p.block_size;
            at = phys * p.num_kv_heads * step + (slot - phys * p.block_size) * p.head_dim;
        }
        place[threadIdx.x] = at;
    }
    __syncthreads();
    const int pair_lanes = half / P;
    const int lanes = pair_lanes + (p.head_dim - p.rot) / E;  // lanes of a row
    const int rows_at_once = kRopeThreads / lanes;
    const int y = threadIdx.x / lanes;
    const int x = threadIdx.x - y * lanes;
    if (y >= rows_at_once)
        return;
    const bool pair = x < pair_lanes;
    const int copy_at = pair ? 0 : p.rot + (x - pair_lanes) * E;
    const int per_tok = p.num_heads + 2 * p.num_kv_heads;  // rows of a token: q, k, v
    // the thread's next row: r of token t
    int t = 0, r = y;
    while (r >= per_tok && t < ntok)
        r -= per_tok, ++t;
    while (t < ntok) {
        RowUnit<T, E, Inter> unit[kRopeUnroll];
        T *dst[kRopeUnroll];
        int turn[kRopeUnroll];  // token to rotate by, -1: a copy
#pragma unroll
        for (int u = 0; u < kRopeUnroll; ++u) {
            dst[u] = nullptr;
            turn[u] = -1;
            if (t < ntok) {
                const long long tok = tok0 + t;
                const T *src;
                if (r < p.num_heads) {
                    src = static_cast<const T *>(p.q) + tok * p.q_stride + r * p.head_dim;
                    dst[u] = static_cast<T *>(p.q_out) + tok * p.q_out_stride + r * p.head_dim;
                    turn[u] = t;
                } else {
                    const bool is_v = r >= p.num_heads + p.num_kv_heads;
                    const int h = r - p.num_heads - (is_v ? p.num_kv_heads : 0);
                    src = (is_v ? static_cast<const T *>(p.v) + tok * p.v_stride
                                : static_cast<const T *>(p.k) + tok * p.k_stride) +
                          h * p.head_dim;
                    const long long at = place[t];
                    if (at >= 0)
                        dst[u] = static_cast<T *>(is_v ? p.v_cache : p.k_cache) + at + h * step;
                    turn[u] = is_v ? -1 : t;
                }
                if (dst[u])
                    unit[u].load(src, x, half, pair, copy_at);
                r += rows_at_once;
                while (r >= per_tok && t < ntok)
                    r -= per_tok, ++t;
            }
        }
#pragma unroll
        for (int u = 0; u < kRopeUnroll; ++u) {
            if (dst[u]) {
                if (pair && turn[u] >= 0)
                    unit[u].rotate(trig + turn[u] * half + x * P);
                unit[u].store(dst[u], x, half, pair, copy_at);
            }
        }
    }
}

template <typename T, int E> const void *rope_fn(bool inter) {
    return inter ? reinterpret_cast<const void *>(&rope_kernel<T, E, true>)
                 : reinterpret_cast<const void *>(&rope_kernel<T, E, false>);
}

}  // namespace

cudaError_t launch_rope(RopeParams p, int dtype, int interleaved, int num_sms, cudaStream_t stream) {
    const int elt = elt_bytes(dtype), E = 16 / elt;
    const auto wide = [&](const void *ptr, long long stride) { return aligned16(ptr) && stride % E == 0; };
    // 16-byte accesses need every row and both halves of a row on a 16-byte
    // boundary; anything else goes element by element
    const bool vec = (interleaved ? p.rot % E == 0 : (p.rot / 2) % E == 0) && wide(p.q, p.q_stride) &&
                     wide(p.q_out, p.q_out_stride) &&
                     (p.num_kv_heads == 0 || (wide(p.k, p.k_stride) && wide(p.v, p.v_stride)));
    const void *fn;
    if (dtype == PA_F32)
        fn = vec ? rope_fn<float, 4>(interleaved) : rope_fn<float, 1>(interleaved);
    else if (dtype == PA_F16)
        fn = vec ? rope_fn<__half, 8>(interleaved) : rope_fn<__half, 1>(interleaved);
    else
        fn = vec ? rope_fn<__nv_bfloat16, 8>(interleaved) : rope_fn<__nv_bfloat16, 1>(interleaved);
    // tokens per CTA: enough CTAs for every SM first, then about 128 rows a CTA (16384
    // tokens of 120 rows each: 160 us with one a CTA, 164 us with two; 65536 tokens of 6
    // rows: 54 us with eight, 80 us with two)
    long long tok = p.num_tokens / (8LL * num_sms);
    tok = tok < 1 ? 1 : (tok > kRopeMaxTok ? kRopeMaxTok : tok);
    const long long few = 128 / (p.num_heads + 2 * p.num_kv_heads);
    tok = tok > few ? (few < 1 ? 1 : few) : tok;
    p.tok = static_cast<int>(tok);
    const long long grid = (p.num_tokens + tok - 1) / tok;
    void *args[] = {&p};
    return launch_dependent(fn, dim3(static_cast<unsigned>(grid)), dim3(kRopeThreads), args,
                            static_cast<size_t>(p.tok) * (p.rot / 2) * sizeof(float2), stream);
}

}  // namespace pa
