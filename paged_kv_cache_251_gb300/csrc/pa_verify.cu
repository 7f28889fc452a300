// Verification of drafted tokens: which of a sequence's drafted tokens are kept,
// and the token after them, from given random numbers, so that what is kept is
// distributed as if the target had drawn every token itself.
//
// At a node of the tree with target p and draft q, after r of its children were
// rejected, the next token's weights are w_r = max(0, p - a_r q) over S_r = sum w_r,
// with a_0 = 0, S_0 = 1: rejecting a child drawn from q leaves max(0, w_r / S_r - q),
// which is max(0, p - (a_r + S_r) q) / S_r, so a_(r+1) = a_r + S_r.  A child x is
// accepted when u S_r q(x) < w_r(x).  Without q (the drafted tokens were chosen, not
// drawn) w_r is p without the rejected tokens, and x is accepted when u S_r < p(x).
// The walk goes over the drafted tokens in order (parents come before children).
// Where it ends, the next token is the first whose running sum of w exceeds u S.
//
// A drawn token must not hang on how a sum was rounded, so weights are summed to
// about 46 bits: p - q as fp32 value and error, lanes' sums as pairs of floats (their
// roundings kept), everything past a lane in 64-bit fixed point (2^-54, in smaller
// units again where that comes to less than 2^-20, in larger ones where a row that is not
// normalised comes to 16 or more), the walk's own numbers again as pairs of floats.  fp64
// arithmetic would be the limit here.
//
// A sequence is a cluster of CTAs, each taking a share of the vocabulary, a warp a
// contiguous slice of it.  The first CTA gathers what the walk needs (every drafted
// token's p, q and u) and hands it to the others, so all walk alike on the same
// bits.  Only a rejection with q, and the end, read a row; the slice of the warp whose
// sum holds the token is read once more, shared by its CTA's warps, to find it.
//
// Measured (fp32, with q, on the GPU): 256 chains over 128000 entries 46 us, 5.7 TB/s of the
// two rows each (without q 27, a row each); 64 chains 15 us (floor 9.7: the gather, two
// cluster barriers and the search are 6); one chain over 32000 entries 7 us, all latency.
// 32 trees of 24 drafted tokens over 50257 entries, bf16: 19 us (without q 11); a
// rejection's sum costs 3 to 4 us (two thirds arithmetic and its barriers).  Loads held a
// step ahead (64 chains 19 us) and twice the loads at once (19 us: one CTA an SM) were slower.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include "pa_device.cuh"
#include "pa_f32x2.cuh"
#include "pa_host.h"
#include "pa_internal.h"
#include "pa_verify.h"

namespace cg = cooperative_groups;

namespace pa {

namespace {

constexpr int kVerifyThreads = 512;
constexpr int kVerifyWarps = kVerifyThreads / 32;
constexpr int kVerifyMaxCluster = 8;
constexpr int kFixedBits = 54;
// Sums below 2^-20 are taken again in smaller units.
constexpr unsigned long long kSmallSum = 1ull << 34;
// From 2^58 units (16) on they are taken again in units 2^12 times larger.  Every lane's, warp's and
// CTA's sum counts about this much at most, so none wraps, and a total below it has not been cut.
constexpr unsigned long long kLargeSum = 1ull << 58;
constexpr int kLargeStep = 12;
constexpr int kLeastBits = kFixedBits - 10 * kLargeStep;  // sums up to 2^124

// A number as two floats, hi + lo with |lo| <= ulp(hi) / 2: about 48 bits.  (One thread's fp64
// instructions took longer than a pass over a row.)
struct Pair {
    float hi, lo;
};
__device__ inline Pair quick_sum(float a, float b) {  // |a| >= |b|
    const float s = __fadd_rn(a, b);
    return {s, __fsub_rn(b, __fsub_rn(s, a))};
}
__device__ inline Pair two_sum(float a, float b) {
    const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
    return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}
__device__ inline Pair add(Pair a, Pair b) {
    const Pair s = two_sum(a.hi, b.hi);
    return quick_sum(s.hi, __fadd_rn(s.lo, __fadd_rn(a.lo, b.lo)));
}
__device__ inline Pair mul(Pair a, float b) {
    const float h = __fmul_rn(a.hi, b);
    return quick_sum(h, __fmaf_rn(a.lo, b, __fmaf_rn(a.hi, b, -h)));
}
__device__ inline Pair negative(Pair a) { return {-a.hi, -a.lo}; }
__device__ inline bool less(Pair a, Pair b) {
    const Pair d = add(a, negative(b));
    return d.hi < 0;
}
// x / 2^bits, rounded down to 48 bits.
__device__ inline Pair pair_of(unsigned long long x, int bits) {
    if (x == 0)
        return {0.f, 0.f};
    const int lead = __clzll(x);
    x <<= lead;  // the top 48 bits as two of 24
    const float hi = static_cast<float>(static_cast<uint32_t>(x >> 40));
    const float lo = static_cast<float>(static_cast<uint32_t>(x >> 16) & 0xffffffu);
    const int e = 40 - lead - bits;
    return quick_sum(ldexpf(hi, e), ldexpf(lo, e - 24));
}

struct VerifyShared {
    // of every drafted token: p, q and u, and the token (its bits; -1: not a token); its parent,
    // twice, plus 1 if it is accepted where it is the first of its node's to be tried
    float4 given[kVerifyMaxDraft + 1];
    int parent2[kVerifyMaxDraft];
    int drafts;
    // of every CTA (0 beyond the last); two passes' (a slow CTA may still read the last)
    __align__(16) unsigned long long total[2][kVerifyMaxCluster];
    unsigned long long warp_sum[kVerifyWarps], part_sum[kVerifyWarps];
    // the walk
    Pair a, s;
    int node, next, n, ngone, need;
    bool summed;  // total[] holds the sum of the present weights
    int path[kVerifyMaxDraft], gone[kVerifyMaxDraft];
};

__device__ inline void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ inline void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

enum { kWalkDone = 0, kWalkSum = 1, kWalkEnd = 2 };

// The walk up to a sum that it needs (kWalkSum: of a rejection's weights, kWalkEnd:
// of the weights it ends with) or to its end (kWalkDone).
template <bool HasQ> __device__ int walk(VerifyShared *sh) {
    int node = sh->node, n = sh->n;
    Pair a = sh->a, s = sh->s;
    int ngone = sh->ngone;
    bool summed = sh->summed;
    bool tried = HasQ ? a.hi != 0 : ngone != 0;  // a child of the node was rejected
    int need = -1;
    int i = sh->next;
    for (; i < sh->drafts; ++i) {
        const int parent2 = sh->parent2[i];
        if (parent2 >> 1 != node)
            continue;
        const float4 given = sh->given[i];
        const int tok = __float_as_int(given.w);
        if (tok < 0)
            continue;
        const float p = given.x, q = given.y, u = given.z;
        bool ok = parent2 & 1;
        if (HasQ) {
            if (tried) {
                const Pair w = add(Pair{p, 0.f}, negative(mul(a, q)));
                ok = w.hi > 0 && less(mul(mul(s, u), q), w);
            }
        } else {
            bool again = false;
            if (tried) {
                for (int g = 0; g < ngone; ++g)
                    again |= sh->gone[g] == tok;
                ok = !again && less(mul(s, u), Pair{p, 0.f});
            }
            if (!ok && !again) {
                sh->gone[ngone++] = tok;
                s = add(s, Pair{p > 0 ? -p : 0.f, 0.f});
                summed = false;
            }
        }
        tried = !ok;
        if (ok) {
            sh->path[n++] = i;
            node = i;
            a = Pair{0.f, 0.f};
            s = Pair{1.f, 0.f};
            ngone = 0;
            summed = false;
        } else if (HasQ) {
            a = add(a, s);
            summed = false;
            need = kWalkSum;
            ++i;
            break;
        }
    }
    if (need < 0)
        need = summed ? kWalkDone : kWalkEnd;
    sh->next = i;
    sh->node = node;
    sh->n = n;
    sh->a = a;
    sh->s = s;
    sh->ngone = ngone;
    sh->summed = summed;
    return need;
}

// max(0, p - a q) as value and error; a in two floats.  An entry whose p or q is
// NaN has no weight.
struct Weight {
    float d, e;
};
template <bool Unit> __device__ inline Weight weight(float p, float q, float ah, float al) {
    if (Unit) {  // a = 1
        const float d = __fsub_rn(p, q);
        const float e = __fsub_rn(__fsub_rn(p, d), q);
        return d > 0 ? Weight{d, e} : Weight{0.f, 0.f};
    }
    const float h = __fmul_rn(ah, q);
    const float l = __fmaf_rn(al, q, __fmaf_rn(ah, q, -h));
    const float d = __fsub_rn(p, h);
    const float e = __fsub_rn(__fsub_rn(__fsub_rn(p, d), h), l);
    return __fadd_rn(d, e) > 0 ? Weight{d, e} : Weight{0.f, 0.f};
}

// x >= 0 in units of 2^-bits, rounded down; 2^63 or more where it is not below that (NaN and
// infinities among it).  (Integer arithmetic: fp64 conversions are slow.)
__device__ inline unsigned long long fixed(float x, int bits) {
    const uint32_t b = __float_as_uint(x);
    const int e = static_cast<int>(b >> 23) & 0xff;
    const unsigned long long m = (b & 0x7fffffu) | (e ? 0x800000u : 0u);
    const int left = bits - 150 + (e ? e : 1);  // x = m 2^(e - 150)
    return left >= 0 ? m << (left > 40 ? 40 : left) : m >> (left < -63 ? 63 : -left);
}
__device__ inline unsigned long long fixed(float hi, float lo, int bits) {
    const unsigned long long a = fixed(hi, bits), b = fixed(fabsf(lo), bits);
    return lo < 0 ? (a > b ? a - b : 0) : a + b;
}
// Of a lane's sum; kLargeSum where hi is not below that (or, in units that no such sum asks for, 2^-126).
__device__ inline unsigned long long fixed_sum(float hi, float lo, int bits) {
    return static_cast<int>(__float_as_uint(hi) >> 23) < max(127 + 58 - bits, 1) ? fixed(hi, lo, bits) : kLargeSum;
}

__device__ inline float to_f(float x) { return x; }
__device__ inline float to_f(__half x) { return __half2float(x); }
__device__ inline float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }

// E consecutive entries of a row from `at` (a multiple of E below `end`), zeros
// from `end` on.
template <typename T, int E> struct Entries {
    float f[E];
    __device__ inline void load(const T *row, int at, int end) {
        if constexpr (E == 1) {
            f[0] = at < end ? to_f(row[at]) : 0.f;
        } else {
            uint4 r = make_uint4(0, 0, 0, 0);
            if (at < end)  // (rows of this form are whole vectors)
                r = *reinterpret_cast<const uint4 *>(row + at);
            Elt<T>::unpack(r, f);
        }
    }
};

__device__ inline unsigned long long warp_add(unsigned long long x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

enum { kRowP = 0, kRowUnit = 1, kRowScaled = 2 };  // p; p - q; p - a q

template <typename T, int E, int Mode>
__device__ inline Weight entry(const float *p, const float *q, int k, float ah, float al) {
    if (Mode == kRowP)
        return p[k] > 0 ? Weight{p[k], 0.f} : Weight{0.f, 0.f};
    return weight<Mode == kRowUnit>(p[k], q[k], ah, al);
}

// Entries of gone[] in a warp's next `n` vectors lose their weight.
template <typename T, int E>
__device__ inline void leave_out(Entries<T, E> *p, int n, int base, int lane, const int *gone, int ngone) {
    for (int g = 0; g < ngone; ++g) {
        const int x = gone[g] - base;
        if (x < 0 || x >= n * 32 * E)  // the same for the whole warp
            continue;
#pragma unroll
        for (int j = 0; j < n; ++j)
#pragma unroll
            for (int k = 0; k < E; ++k)
                if (x == (j * 32 + lane) * E + k)
                    p[j].f[k] = 0.f;
    }
}

// Sum of the weights of [lo, hi) in units of 2^-bits (every lane gets it), entries in
// gone[] left out (Mode kRowP only); a lane's counts kLargeSum at most.
template <typename T, int E, int Mode>
__device__ unsigned long long slice_sum(const T *prow, const T *qrow, int lo, int hi, float ah, float al,
                                        const int *gone, int ngone, int bits, int lane) {
    constexpr int kFlight = 16 / E;  // loads in flight of each row
    F2 h2 = f2(0.f, 0.f), l2 = h2;  // of even and odd entries
    for (int base = lo; base < hi; base += 32 * E * kFlight) {
        Entries<T, E> p[kFlight], q[kFlight];
#pragma unroll
        for (int j = 0; j < kFlight; ++j) {
            const int at = base + (j * 32 + lane) * E;
            p[j].load(prow, at, hi);
            if (Mode != kRowP)
                q[j].load(qrow, at, hi);
        }
        if (Mode == kRowP)
            leave_out<T, E>(p, kFlight, base, lane, gone, ngone);
#pragma unroll
        for (int k = 0; k < kFlight * E; k += 2) {
            F2 d, e = f2(0.f, 0.f);
            const float px = p[k / E].f[k % E], py = p[(k + 1) / E].f[(k + 1) % E];
            const float qx = Mode == kRowP ? 0.f : q[k / E].f[k % E], qy = Mode == kRowP ? 0.f : q[(k + 1) / E].f[(k + 1) % E];
            if (Mode == kRowP) {
                d = f2(fmaxf(px, 0.f), fmaxf(py, 0.f));
            } else if (Mode == kRowUnit) {  // max(p, q) - q; a NaN of q as a large number
                const F2 b = f2(fminf(qx, 1e30f), fminf(qy, 1e30f));
                const F2 a = f2(fmaxf(px, fminf(qx, 1e30f)), fmaxf(py, fminf(qy, 1e30f)));
                d = f2_sub(a, b);
                e = f2_sub(f2_sub(a, d), b);
            } else {
                const Weight x = weight<false>(px, qx, ah, al), y = weight<false>(py, qy, ah, al);
                d = f2(x.d, y.d);
                e = f2(x.e, y.e);
            }
            // h + d as value and error
            const F2 s = f2_add(h2, d), b = f2_sub(s, h2);
            const F2 err = f2_add(f2_sub(h2, f2_sub(s, b)), f2_sub(d, b));
            h2 = s;
            l2 = f2_add(l2, Mode == kRowP ? err : f2_add(err, e));
        }
    }
    const float2 hs = f2_get(h2), ls = f2_get(l2);
    const Pair sum = two_sum(hs.x, hs.y);
    const float h = sum.hi, l = __fadd_rn(sum.lo, __fadd_rn(ls.x, ls.y));
    return warp_add(fixed_sum(h, l, bits));
}

// The first entry of [lo, hi) whose running sum exceeds t, entries in gone[] left
// out; the last with any weight where rounding leaves none (-1: no weight at all).
template <typename T, int E, int Mode>
__device__ int slice_find(const T *prow, const T *qrow, int lo, int hi, float ah, float al, const int *gone, int ngone,
                          unsigned long long t, int bits, int lane) {
    unsigned long long before = 0;
    int last = -1;
    for (int base = lo; base < hi; base += 32 * E) {
        const int at = base + lane * E;
        Entries<T, E> p, q;
        p.load(prow, at, hi);
        if (Mode != kRowP)
            q.load(qrow, at, hi);
        if (Mode == kRowP)
            leave_out<T, E>(&p, 1, base, lane, gone, ngone);
        unsigned long long w[E], sum = 0;
#pragma unroll
        for (int k = 0; k < E; ++k) {
            const Weight we = entry<T, E, Mode>(p.f, q.f, k, ah, al);
            w[k] = fixed(we.d, we.e, bits);
            if (we.d > 0)
                last = at + k;
            sum += w[k];
        }
        unsigned long long incl = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned long long y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o)
                incl += y;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, before + incl > t);
        if (hit) {
            const int who = __ffs(hit) - 1;
            int x = -1;
            if (lane == who) {
                unsigned long long run = before + incl - sum;
#pragma unroll
                for (int k = 0; k < E; ++k) {
                    run += w[k];
                    if (x < 0 && run > t)
                        x = at + k;
                }
            }
            return __shfl_sync(0xffffffffu, x, who);
        }
        before += __shfl_sync(0xffffffffu, incl, 31);
    }
    return __reduce_max_sync(0xffffffffu, last);
}

template <typename T, int E, bool HasQ>
__global__ void __launch_bounds__(kVerifyThreads) verify_kernel(const VerifyParams p) {
    __shared__ VerifyShared shared;
    VerifyShared *sh = &shared;
    pdl_launch_dependents();
    pdl_wait();
    cg::cluster_group cluster = cg::this_cluster();
    const int ranks = p.cluster, rank = ranks > 1 ? static_cast<int>(cluster.block_rank()) : 0;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const long long s = blockIdx.x / ranks;
    const int T1 = p.num_draft, V = p.vocab;
    const T *target = static_cast<const T *>(p.target) + s * (T1 + 1) * p.target_stride;
    const T *draft = static_cast<const T *>(p.draft) + (HasQ ? s * T1 * p.draft_stride : 0);

    // what the walk needs, gathered once for all CTAs (every one walks on the same bits):
    // thread i drafted token i, and one more the last random number
    static_assert(kVerifyMaxDraft < kVerifyThreads, "a thread a drafted token, and one more");
    if (ranks > 1)
        cluster_arrive();
    int drafts = T1, parent = -1, tok = -1;
    float u = 0.f, pv = 0.f, qv = 0.f;
    bool fine = false;
    const int i = tid;
    if (rank == 0 && i <= T1) {
        uint32_t bad = 0;
        u = p.uniforms[s * (T1 + 1) + i];
        if (p.draft_lens) {
            drafts = p.draft_lens[s];
            if (drafts < 0 || drafts > T1) {
                bad = PA_DEVERR_BAD_LEN;
                drafts = drafts < 0 ? 0 : T1;
            }
        }
        if (i < T1) {
            tok = p.draft_tokens[s * T1 + i];
            parent = p.parents ? p.parents[s * T1 + i] : i - 1;
            if (parent < 0)
                parent = -1;
            if (i >= drafts) {
                tok = -1;
            } else if (tok < 0 || tok >= V || parent >= i) {
                bad |= PA_DEVERR_BAD_INDEX;
                tok = -1;
            } else {
                pv = to_f(target[static_cast<long long>(parent + 1) * p.target_stride + tok]);
                if (HasQ)
                    qv = to_f(draft[static_cast<long long>(parent + 1) * p.draft_stride + tok]);
                // u q < p without rounding: the product as value and error
                const float h = HasQ ? __fmul_rn(u, qv) : u;
                fine = h < pv || (HasQ && h == pv && __fmaf_rn(u, qv, -h) < 0);
            }
        }
        if (bad && p.err)
            atomicOr(p.err, bad);
    }
    if (ranks > 1)
        cluster_wait();  // every CTA of the cluster has started
    if (rank == 0 && i <= T1) {
        for (int r = 0; r < ranks; ++r) {
            VerifyShared *to = ranks > 1 ? cluster.map_shared_rank(sh, r) : sh;
            to->given[i] = make_float4(pv, qv, u, __int_as_float(tok));
            if (i < T1)
                to->parent2[i] = parent * 2 + fine;
            else
                to->drafts = drafts;
        }
    }
    if (tid < 2 * kVerifyMaxCluster)
        (&sh->total[0][0])[tid] = 0;  // (before any CTA's first sums: the barrier below)
    if (tid == 0) {
        sh->a = Pair{0.f, 0.f};
        sh->s = Pair{1.f, 0.f};
        sh->node = -1;
        sh->next = sh->n = sh->ngone = 0;
        sh->summed = false;
    }
    if (ranks > 1)
        cluster.sync();
    else
        __syncthreads();

    const int lo = static_cast<int>(min(static_cast<long long>(rank * kVerifyWarps + warp) * p.slice,
                                        static_cast<long long>(V)));
    const int hi = V - lo < p.slice ? V : lo + p.slice;
    const T *prow, *qrow;
    float ah, al;
    int mode, parity = 0;
    unsigned long long total = 0;
    int bits = kFixedBits;  // more where the sum is small, less where it is large
    for (bool again = false, rescaled = false;;) {
        if (tid == 0 && !again && !rescaled)
            sh->need = walk<HasQ>(sh);
        __syncthreads();
        const int need = sh->need;
        if (need != kWalkDone) {
            if (!rescaled)
                bits = kFixedBits;
            const int node = sh->node;
            prow = target + static_cast<long long>(node + 1) * p.target_stride;
            ah = sh->a.hi;
            al = sh->a.lo;
            mode = !HasQ || ah == 0 ? kRowP : (ah == 1 && al == 0 ? kRowUnit : kRowScaled);
            qrow = mode == kRowP ? nullptr : draft + static_cast<long long>(node + 1) * p.draft_stride;
            unsigned long long sum;
            if (mode == kRowP)
                sum = slice_sum<T, E, kRowP>(prow, qrow, lo, hi, ah, al, sh->gone, sh->ngone, bits, lane);
            else if (mode == kRowUnit)
                sum = slice_sum<T, E, kRowUnit>(prow, qrow, lo, hi, ah, al, sh->gone, sh->ngone, bits, lane);
            else
                sum = slice_sum<T, E, kRowScaled>(prow, qrow, lo, hi, ah, al, sh->gone, sh->ngone, bits, lane);
            if (lane == 0)
                sh->warp_sum[warp] = sum;
            __syncthreads();
            if (warp == 0) {
                const unsigned long long of_warp = lane < kVerifyWarps ? sh->warp_sum[lane] : 0ull;
                const unsigned long long mine = min(warp_add(min(of_warp, kLargeSum)), kLargeSum);
                if (lane < ranks) {
                    VerifyShared *to = ranks > 1 ? cluster.map_shared_rank(sh, lane) : sh;
                    to->total[parity][rank] = mine;
                }
            }
            if (ranks > 1)
                cluster.sync();
            else
                __syncthreads();
            total = 0;
#pragma unroll
            for (int r = 0; r < kVerifyMaxCluster; r += 2) {
                const ulonglong2 x = *reinterpret_cast<const ulonglong2 *>(&sh->total[parity][r]);
                total += x.x + x.y;
            }
            parity ^= 1;
            rescaled = false;
            if (total - kSmallSum >= kLargeSum - kSmallSum) {  // below kSmallSum, or kLargeSum and more
                const bool large = total >= kLargeSum;
                rescaled = large ? bits > kLeastBits : bits < kFixedBits + 150;  // (fp32 ends at 2^-149)
                if (rescaled) {
                    bits += large ? -kLargeStep : (total ? 20 : 50);
                    continue;
                }
            }
            if (tid == 0) {
                sh->s = pair_of(total, bits);
                sh->summed = true;
            }
        }
        again = false;
        if (need == kWalkSum)
            continue;
        // nothing is left of p (p and q alike, up to rounding, or every token rejected): p itself
        if (total == 0 && (sh->a.hi != 0 || sh->ngone != 0)) {
            __syncthreads();
            if (tid == 0) {
                sh->a = Pair{0.f, 0.f};
                sh->ngone = 0;
                sh->need = kWalkEnd;
            }
            again = true;
            continue;
        }
        break;
    }

    const int n = sh->n;
    if (rank == 0) {
        if (i <= T1) {
            const int at = i < n ? sh->path[i] : -1;
            if (i < T1)
                p.accepted[s * T1 + i] = at;
            if (i != n || total == 0)
                p.tokens[s * (T1 + 1) + i] = i < n ? __float_as_int(sh->given[at].w) : -1;
        }
        if (tid == 0)
            p.accept_lens[s] = n;
    }
    if (total == 0)
        return;
    // t = floor(u total): u as a fraction of 64 bits
    u = sh->given[T1].z;
    unsigned long long t = u >= 1.f ? total - 1 : (u > 0.f ? __umul64hi(total, fixed(u, 64)) : 0ull);
    int owner = 0;
    parity ^= 1;
    // (bounded: sums of infinite entries are cut)
    while (owner < ranks - 1 && t >= sh->total[parity][owner])
        t -= sh->total[parity][owner++];
    if (rank != owner)
        return;
    int w = 0;
    while (w < kVerifyWarps - 1 && t >= sh->warp_sum[w])
        t -= sh->warp_sum[w++];
    // the slice of warp w that holds it, shared by all warps, then the part that does
    const int begin = (rank * kVerifyWarps + w) * p.slice, end = min(begin + p.slice, V);
    // (a few vectors a lane: its warp alone is faster.  fp32, shared and not: slices of 256
    // entries 7.5 and 7.0 us, of 416 10.0 and 9.1, of 1024 8.3 and 8.6, of 2016 15.2 and 18.9,
    // of 8000 46 and 90)
    const bool shared_out = p.slice > 4 * 32 * E;
    const int part = shared_out ? (p.slice / kVerifyWarps + 31) / 32 * 32 : p.slice;
    const int plo = shared_out ? min(begin + warp * part, end) : begin, phi = min(plo + part, end);
    const int *gone = sh->gone;
    const int ngone = sh->ngone;
    int which = 0;
    if (shared_out) {
        unsigned long long sum;
        if (mode == kRowP)
            sum = slice_sum<T, E, kRowP>(prow, qrow, plo, phi, ah, al, gone, ngone, bits, lane);
        else if (mode == kRowUnit)
            sum = slice_sum<T, E, kRowUnit>(prow, qrow, plo, phi, ah, al, gone, ngone, bits, lane);
        else
            sum = slice_sum<T, E, kRowScaled>(prow, qrow, plo, phi, ah, al, gone, ngone, bits, lane);
        if (lane == 0)
            sh->part_sum[warp] = sum;
        __syncthreads();
        int last = 0;
        which = -1;
        for (int k = 0; k < kVerifyWarps && which < 0; ++k) {
            const unsigned long long x = sh->part_sum[k];
            if (x)
                last = k;
            if (t < x)
                which = k;
            else
                t -= x;
        }
        if (which < 0) {  // the parts' sums are rounded apart from the slice's
            which = last;
            t = ~0ull;
        }
    }
    if (warp != which)
        return;
    int found;
    if (mode == kRowP)
        found = slice_find<T, E, kRowP>(prow, qrow, plo, phi, ah, al, gone, ngone, t, bits, lane);
    else if (mode == kRowUnit)
        found = slice_find<T, E, kRowUnit>(prow, qrow, plo, phi, ah, al, gone, ngone, t, bits, lane);
    else
        found = slice_find<T, E, kRowScaled>(prow, qrow, plo, phi, ah, al, gone, ngone, t, bits, lane);
    if (lane == 0)
        p.tokens[s * (T1 + 1) + n] = found;
}

template <typename T> const void *verify_fn(bool vec, bool has_q) {
    constexpr int E = 16 / sizeof(T);
    if (vec)
        return has_q ? reinterpret_cast<const void *>(&verify_kernel<T, E, true>)
                     : reinterpret_cast<const void *>(&verify_kernel<T, E, false>);
    return has_q ? reinterpret_cast<const void *>(&verify_kernel<T, 1, true>)
                 : reinterpret_cast<const void *>(&verify_kernel<T, 1, false>);
}

}  // namespace

cudaError_t launch_verify(VerifyParams p, int dtype, int num_sms, cudaStream_t stream) {
    const int e = 16 / elt_bytes(dtype);
    // (whole vectors of 16 bytes; else entry by entry: 32 trees over 50257 bf16 entries 18 us,
    // over 50256 16)
    const bool vec = p.vocab % e == 0 && p.target_stride % e == 0 && p.draft_stride % e == 0 && aligned16(p.target) &&
                     aligned16(p.draft);
    const void *fn = dtype == PA_F32   ? verify_fn<float>(vec, p.draft != nullptr)
                     : dtype == PA_F16 ? verify_fn<__half>(vec, p.draft != nullptr)
                                       : verify_fn<__nv_bfloat16>(vec, p.draft != nullptr);
    // As many CTAs as are resident at once (two an SM), while each has eight entries a thread:
    // 8 and 4 CTAs for a chain of 128000 entries 8.3 and 9.3 us, for 32 chains of 50256 9.2 and
    // 10.6, for one of 32000 7.0 and 6.8; 4 and 1 for one of 8000 5.7 and 5.2, for 32 of 8000 8.0
    // and 6.6.  More than are resident: 64 chains of 128000 24 us instead of 15.
    int cluster = 1;
    while (cluster < kVerifyMaxCluster && static_cast<long long>(p.num_seqs) * cluster * 2 <= 2LL * num_sms &&
           p.vocab / (cluster * 2) >= 8 * kVerifyThreads)
        cluster *= 2;
    p.cluster = cluster;
    const int warps = cluster * kVerifyWarps;
    p.slice = ((p.vocab + warps - 1) / warps + 31) / 32 * 32;
    // (the grid's first dimension holds 2^31 - 1 CTAs: the caller bounds num_seqs)
    void *args[] = {&p};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(p.num_seqs) * cluster);
    cfg.blockDim = dim3(kVerifyThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelExC(&cfg, fn, args);
}

}  // namespace pa
