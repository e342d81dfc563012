// The distillation loss against a teacher's top logits: loss, gradient, backward pass.
//
// With z' = z/tau, lse the log-sum-exp of a row's z' and rest the one over the tokens
// outside the teacher's list, the loss is
//   sum_j p_j log p_j - sum_j p_j (z'_j - lse)  [+ p_rest (log p_rest - (rest - lse))]
// and its gradient by z, times tau, with M = sum_j p_j + p_rest:
//   M q_v - p_v on the list, softmax_rest(z')_v * (M q_rest - p_rest) outside it,
// q_rest = exp(rest - lse), p_rest = 0 without a rest entry. M is 1 unless the list's own mass is above
// 1 (top values rounded to 16 bits beside the log-sum-exp of the unrounded ones): p_rest is 0 there.
// Summing the rest apart (rather than as 1 minus the list) keeps its precision when the list holds
// nearly all the mass.
//
// What has to move: each logit in once and, with the gradient, out once; the lists are small. The
// one pass keeps a row on chip (k_distill_row), so nothing is read twice. What bounds it is the
// chain of a row, copy, maximum, sum, the blocks' exchange, gradient, of which three run in turn on
// an SM, at 60% of the issue slots and 68% of DRAM's rate (the loss alone 53 and 54%). Measured (CUDA
// events), loss with gradient: 8192 x 32000 bfloat16, K = 64, 192 us (5.5 TB/s); 8192 x 131072, K = 100,
// with the rest entry, 845 us (5.1 TB/s); 4096 x 50257 float32, K = 20, 327 us (5.0 TB/s). The loss
// alone: 125, 542 and 216 us (3.8 - 4.2 TB/s). Backward from saved statistics: 174, 692 and 254 us
// (6.0 - 6.5 TB/s).
#include <algorithm>

#include "ob_student.cuh"
#include "ob_student.h"
#include "ob_tma.cuh"

namespace ob {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// A row's teacher entries in shared memory: Kp (K rounded up to 4) of each.
struct Teacher {
    int* token;     // its token (-1: padding)
    int* first;     // the token, or -1 where an earlier entry has it
    float* t;       // its value
    float* total;   // p summed over the entries of one token
    float* z;       // the student's logit there
};

constexpr int kTeacherWords = 5;

__host__ __device__ __forceinline__ int padded(int K) { return (K + 3) / 4 * 4; }

__device__ __forceinline__ Teacher teacher_at(void* base, int K)
{
    int* b = static_cast<int*>(base);
    const int Kp = padded(K);
    float* f = reinterpret_cast<float*>(b + 2 * Kp);
    return Teacher{b, b + Kp, f, f + Kp, f + 2 * Kp};
}

// What a row's list comes to.
struct List {
    float self, mass;           // sums of p log p, p
    float rest, slack;          // p_rest, and how much of it the roundings of mass may have made
    float m, s;                 // its student logits' sum of exponentials, as below
};

// What the list warp tells the others of a row.
struct RowInfo {
    List list;
    float w, next_w;            // this row's weight and the next one's
};

__device__ __forceinline__ float warp_sum(float v)
{
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

__device__ __forceinline__ float warp_max(float v)
{
    for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

__device__ __forceinline__ float top_at(const DistillArgs& a, int64_t o)
{
    if (a.top_dtype == OB_F32) return static_cast<const float*>(a.top)[o];
    if (a.top_dtype == OB_F16) return to_f32(static_cast<const __half*>(a.top)[o]);
    return to_f32(static_cast<const __nv_bfloat16*>(a.top)[o]);
}

__device__ __forceinline__ int token_at(const DistillArgs& a, int64_t o)
{
    const int64_t k = a.index_bits == 64 ? static_cast<const int64_t*>(a.index)[o]
                                         : (int64_t)static_cast<const int32_t*>(a.index)[o];
    return k >= 0 && k < a.V ? (int)k : -1;
}

// ---- sums of exponentials ------------------------------------------------------------------------
//
// (m, s) stands for s * 2^c(m), c(m) = m*k2 rounded to float32 and k2 = log2(e)/tau: s is the sum over
// some logits z of 2^(z*k2 - c), each exponent formed by one multiply-add, so that the rounding of c
// (of the order of 1e-6) is the same in every term and in what is made of s later, and drops out.
//
// That rounding grows with m and would overflow the terms themselves (a row at -1e30 or at the type's
// lowest value). From |m*k2| = kHuge on c(m) is m*k2 itself: any two float32 values of which one is
// that large are at least 64 apart in z*k2, so the terms are 1 where z = m and nothing to float32
// elsewhere, which a power of two in place of k2 makes exactly.

constexpr float kHuge = 1073741824.0f;      // 2^30

// The exponent of a logit z <= m is z*k - c.
struct Scale {
    float k, c;
};

__device__ __forceinline__ Scale scale_of(float m, float k2)
{
    const float c = m * k2;
    if (fabsf(c) < kHuge) return Scale{k2, c};
    if (isinf(m)) return Scale{k2, fmaxf(m, 0.0f)};
    // k*|m| in [2^30, 2^31)
    const unsigned e = __float_as_uint(m) >> 23 & 255u;
    const float k = __uint_as_float(min(284u - e, 254u) << 23);
    return Scale{k, k * m};
}

// 2^(c(a) - c(b)) for a <= b.
__device__ __forceinline__ float between(float a, float b, float k2)
{
    const float ca = a * k2, cb = b * k2, f = fast_exp2(ca - cb);
    return a == b ? 1.0f : fmaxf(fabsf(ca), fabsf(cb)) < kHuge ? f : 0.0f;
}

__device__ __forceinline__ float2 join(float2 a, float2 b, float k2)
{
    const float m = fmaxf(a.x, b.x);
    return make_float2(m, a.y * between(a.x, m, k2) + b.y * between(b.x, m, k2));
}

// (m, s) of every lane joined, in every lane. An empty one is (-infinity, 0); a sum of NaN stays.
__device__ __forceinline__ float2 warp_join(float m, float s, float k2)
{
    const float top = warp_max(m);
    return make_float2(top, warp_sum(s * between(m, top, k2)));
}

// log(s * 2^c(m)) - m/tau: what the rounding of c makes of log(s).
__device__ __forceinline__ float log_over(float2 a, float k2)
{
    const float c = a.x * k2, off = fabsf(c) < kHuge ? kLn2 * fmaf(-a.x, k2, c) : 0.0f;
    return a.y == 0.0f ? -INFINITY : logf(a.y) + off;
}

// Entry j of row n's list into shared memory.
template <typename IO>
__device__ __forceinline__ void put_entry(const DistillArgs& a, int64_t n, const IO* z, const Teacher& t, int j)
{
    const int k = j < a.K ? token_at(a, n * a.K + j) : -1;
    t.token[j] = k;
    t.t[j] = k < 0 ? -INFINITY : top_at(a, n * a.K + j);
    t.z[j] = k < 0 ? -INFINITY : to_f32(z[k]);
}

// First and total from the entries in shared memory, and their sums, by one warp. A token listed more
// than once counts once, with the sum of its entries: `seen`, kSeenWords words of shared memory,
// has a bit for each of 2,048 classes of tokens, and only entries that find theirs taken are
// compared with the others.
constexpr int kSeenWords = 64;

__device__ List prepare_list(const DistillArgs& a, float top_lse, const Teacher& t, unsigned* seen)
{
    const int lane = threadIdx.x & 31, K = a.K;
    const float k2 = a.inv_tau * kLog2e;
    float top = -INFINITY, m = -INFINITY, off, lse;      // log p = (t - off)/tau - lse
    for (int w = lane; w < kSeenWords; w += 32) seen[w] = 0u;
    for (int j = lane; j < K; j += 32) {
        top = fmaxf(top, t.t[j]);
        m = fmaxf(m, t.z[j]);
    }
    __syncwarp();
    m = warp_max(m);
    if (a.top_lse) {
        off = 0.0f;
        lse = top_lse;
    } else {
        // relative to the largest, so that neither the size of the values nor 1/tau costs precision or overflows
        off = warp_max(top);
        float sum = 0.0f;
        for (int j = lane; j < K; j += 32) sum += t.t[j] == -INFINITY ? 0.0f : expf((t.t[j] - off) * a.inv_tau);
        lse = logf(warp_sum(sum));
    }
    List l{0.0f, 0.0f, 0.0f, 0.0f, m, 0.0f};
    for (int j0 = 0; j0 < K; j0 += 32) {
        const int j = j0 + lane, k = j < K ? t.token[j] : -1;
        bool taken = false;
        if (j < K) {
            const float lp = fmaf(t.t[j] - off, a.inv_tau, -lse), p = t.t[j] == -INFINITY ? 0.0f : expf(lp);
            l.mass += p;
            if (!(p == 0.0f)) l.self += p * lp;
            t.total[j] = p;
            t.first[j] = k;
            const unsigned h = (unsigned)k * 2654435761u >> 21;
            if (k >= 0) taken = atomicOr(&seen[h >> 5], 1u << (h & 31u)) >> (h & 31u) & 1u;
        }
        __syncwarp();
        for (unsigned todo = __ballot_sync(0xffffffffu, taken); todo; todo &= todo - 1) {
            const int key = __shfl_sync(0xffffffffu, k, __ffs(todo) - 1);
            float total = 0.0f;
            int first = -1;
            for (int q0 = 0; q0 <= j0; q0 += 32) {
                const int q = q0 + lane;
                const bool same = q < K && t.token[q] == key;
                if (same) {
                    total += t.total[q];
                    t.total[q] = 0.0f;
                    t.first[q] = -1;
                }
                const unsigned who = __ballot_sync(0xffffffffu, same);
                if (first < 0 && who) first = q0 + __ffs(who) - 1;
            }
            total = warp_sum(total);
            __syncwarp();
            if (lane == 0) {
                t.total[first] = total;
                t.first[first] = key;
            }
            __syncwarp();
        }
    }
    const Scale c = scale_of(m, k2);
    for (int j = lane; j < K; j += 32)
        if (t.first[j] >= 0) l.s += fast_exp2(fmaf(t.z[j], c.k, -c.c));
    l.s = warp_sum(l.s);
    l.self = warp_sum(l.self);
    l.mass = warp_sum(l.mass);
    if (a.top_lse) {
        l.rest = fmaxf(0.0f, 1.0f - l.mass);
        // an entry that counts has top/tau near lse: two roundings of the one, one of the other, one of their
        // difference, the exponential's 4; and the sum's
        l.slack = 0x1p-24f * (4.0f * fabsf(lse) + (float)K / 32.0f + 16.0f);
    }
    return l;
}

// p_rest. Where the student has no mass outside the list (its logits there are masked, by -infinity or a
// value so far below the largest that float32 has no ratio for it) any of it makes the loss huge or
// infinite, so there what rounding may have left does not count.
__device__ __forceinline__ float rest_mass(const List& l, float2 rest, float2 all, float k2)
{
    return l.rest <= l.slack && between(rest.x, all.x, k2) == 0.0f ? 0.0f : l.rest;
}

// The same for a whole block: warp 0 prepares the list of row n (z: the whole row) and tells the
// others. Ends with the block's barrier.
template <typename IO>
__device__ __forceinline__ List read_list(const DistillArgs& a, int64_t n, const IO* z, const Teacher& t, unsigned* seen,
                                          List* shared)
{
    for (int j = threadIdx.x; j < padded(a.K); j += kThreads) put_entry(a, n, z, t, j);
    __syncthreads();
    if (threadIdx.x < 32) {
        const List l = prepare_list(a, a.top_lse ? a.top_lse[n] : 0.0f, t, seen);
        if (threadIdx.x == 0) *shared = l;
    }
    __syncthreads();
    return *shared;
}

// What a row's gradient is made of: M q = 2^(z*k2 - c(top)) * inv on the list, and (M q_rest - p_rest) times
// the softmax of the rest, 2^(z*k2 - c(rest)) * coef, outside it; top and rest are the largest logits.
// inv is 0 for a row without a loss.
struct RowGrad {
    float top, inv, rest, coef;
};

__device__ __forceinline__ RowGrad row_grad(const DistillArgs& a, const List& l, float2 rest, float2 all, float k2)
{
    const float prest = rest_mass(l, rest, all, k2);
    RowGrad g;
    g.top = all.x;
    g.inv = __fdividef(a.top_lse && prest == 0.0f ? l.mass : 1.0f, all.y);     // mass + prest
    g.rest = rest.x;
    g.coef = rest.y == 0.0f ? 0.0f : between(rest.x, all.x, k2) * g.inv - __fdividef(prest, rest.y);
    return g;
}

// The row's loss; one warp calls it.
__device__ __forceinline__ float row_loss(const DistillArgs& a, const Teacher& t, const List& l, float2 rest,
                                          float2 all, float k2)
{
    // sum p log q = sum p (z - m)/tau - mass * log(sum over all)
    const float over = log_over(all, k2);
    float cross = 0.0f;
    for (int j = threadIdx.x & 31; j < a.K; j += 32)
        if (t.first[j] >= 0 && !(t.total[j] == 0.0f)) cross += t.total[j] * (t.z[j] - all.x);
    cross = warp_sum(cross) * a.inv_tau;
    float loss = l.self;
    if (!(l.mass == 0.0f)) loss -= cross - l.mass * over;
    const float prest = rest_mass(l, rest, all, k2);
    if (prest > 0.0f) {
        const float lrest = rest.y == 0.0f ? -INFINITY : (rest.x - all.x) * a.inv_tau + log_over(rest, k2);
        loss += prest * (logf(prest) - (lrest - over));
    }
    return loss;
}

// ---- vectors of 16 bytes ---------------------------------------------------------------------------

template <typename IO>
struct Vec {
    static constexpr int kN = 16 / sizeof(IO);
    alignas(16) IO v[kN];
};

template <typename IO>
__device__ __forceinline__ Vec<IO> load_vec(const void* p)
{
    Vec<IO> r;
    const uint4 w = *static_cast<const uint4*>(p);
    memcpy(&r, &w, 16);
    return r;
}

template <typename IO>
__device__ __forceinline__ void store_vec(void* p, const Vec<IO>& v)
{
    uint4 w;
    memcpy(&w, &v, 16);
    *static_cast<uint4*>(p) = w;
}

// Two elements of a vector in float32, and back.
template <typename IO>
__device__ __forceinline__ float2 two(const Vec<IO>& v, int e)
{
    unsigned w;
    memcpy(&w, &v.v[e], 4);
    return unpack_pair(w, IO{});
}

template <>
__device__ __forceinline__ float2 two<float>(const Vec<float>& v, int e) { return make_float2(v.v[e], v.v[e + 1]); }

template <typename IO>
__device__ __forceinline__ void set_two(Vec<IO>& v, int e, float2 f)
{
    const unsigned w = pack_pair(f, IO{});
    memcpy(&v.v[e], &w, 4);
}

template <>
__device__ __forceinline__ void set_two<float>(Vec<float>& v, int e, float2 f)
{
    v.v[e] = f.x;
    v.v[e + 1] = f.y;
}

// A running maximum over vectors, in the storage type.
template <typename IO>
struct VecMax;

template <>
struct VecMax<float> {
    float m = -INFINITY;
    __device__ __forceinline__ void add(const Vec<float>& v)
    {
        m = fmaxf(m, fmaxf(fmaxf(v.v[0], v.v[1]), fmaxf(v.v[2], v.v[3])));
    }
    __device__ __forceinline__ float get() const { return m; }
};

template <>
struct VecMax<__half> {
    __half2 m = __float2half2_rn(-INFINITY);
    __device__ __forceinline__ void add(const Vec<__half>& v)
    {
        __half2 p[4];
        memcpy(p, &v, 16);
        m = __hmax2(m, __hmax2(__hmax2(p[0], p[1]), __hmax2(p[2], p[3])));
    }
    __device__ __forceinline__ float get() const { return fmaxf(__low2float(m), __high2float(m)); }
};

template <>
struct VecMax<__nv_bfloat16> {
    __nv_bfloat162 m = __float2bfloat162_rn(-INFINITY);
    __device__ __forceinline__ void add(const Vec<__nv_bfloat16>& v)
    {
        __nv_bfloat162 p[4];
        memcpy(p, &v, 16);
        m = __hmax2(m, __hmax2(__hmax2(p[0], p[1]), __hmax2(p[2], p[3])));
    }
    __device__ __forceinline__ float get() const { return fmaxf(__low2float(m), __high2float(m)); }
};

// (m, s) of the vectors from, from + step, ... below end of a buffer in shared memory: a first
// pass for the thread's maximum, a second for its sum.
template <typename IO>
__device__ __forceinline__ float2 sum_vectors(const IO* buf, int from, int step, int end, float k2)
{
    constexpr int E = Vec<IO>::kN;
    VecMax<IO> top;
#pragma unroll 4
    for (int k = from; k < end; k += step) top.add(load_vec<IO>(buf + k * E));
    const float m = top.get();
    const Scale c = scale_of(m, k2);
    const float2 kk = hold(c.k), cc = both(-c.c);
    float2 s0 = both(0.0f), s1 = both(0.0f);
#pragma unroll 4
    for (int k = from; k < end; k += step) {
        const Vec<IO> v = load_vec<IO>(buf + k * E);
#pragma unroll
        for (int e = 0; e < E; e += 4) {
            const float2 p = fma2(two(v, e), kk, cc), q = fma2(two(v, e + 2), kk, cc);
            s0 = add2(s0, make_float2(fast_exp2(p.x), fast_exp2(p.y)));
            s1 = add2(s1, make_float2(fast_exp2(q.x), fast_exp2(q.y)));
        }
    }
    s0 = add2(s0, s1);
    return make_float2(m, s0.x + s0.y);
}

// coef * 2^(z kk - c) of a vector.
template <typename IO>
__device__ __forceinline__ void grad_vector(Vec<IO>& v, float2 kk, float2 minus_c, float2 coef)
{
#pragma unroll
    for (int e = 0; e < Vec<IO>::kN; e += 2) {
        const float2 p = fma2(two(v, e), kk, minus_c);
        set_two(v, e, mul2(coef, make_float2(fast_exp2(p.x), fast_exp2(p.y))));
    }
}

__device__ __forceinline__ uint32_t phase_of(const void* p, int elem)
{
    return (uint32_t)(reinterpret_cast<uintptr_t>(p) % 16) / elem;
}

// A store of 4 bytes into the same place of another block's shared memory.
__device__ __forceinline__ void store_remote(uint32_t local, uint32_t rank, float v)
{
    asm volatile(
        "{\n\t.reg .b32 a;\n\t"
        "mapa.shared::cluster.u32 a, %0, %1;\n\t"
        "st.shared::cluster.f32 [a], %2;\n\t}" ::"r"(local),
        "r"(rank), "f"(v)
        : "memory");
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// Orders this thread's accesses to shared memory before later copies into it.
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// One arrival at the barrier of another block of the cluster (or this one), after which what this
// thread has written to that block is visible to those who wait there.
__device__ __forceinline__ void arrive_remote(uint32_t local, uint32_t rank)
{
    asm volatile(
        "{\n\t.reg .b32 a;\n\t"
        "mapa.shared::cluster.u32 a, %0, %1;\n\t"
        "mbarrier.arrive.release.cluster.shared::cluster.b64 _, [a];\n\t}" ::"r"(local),
        "r"(rank)
        : "memory");
}

// 1 once any wait of these kernels has run out (read and cleared by distill_status).
__device__ unsigned wait_status;

__device__ __forceinline__ void note_timeout() { atomicMax(&wait_status, kStatusWaitTimeout); }

// Waits (bounded) for the arrivals of other blocks.
__device__ __forceinline__ bool wait_cluster(uint32_t bar, uint32_t parity, uint64_t limit_ns)
{
    const uint64_t t0 = global_ns();
    for (uint32_t spins = 0; spins < (1u << 30); ++spins) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(bar), "r"(parity)
            : "memory");
        if (ok) return true;
        if (global_ns() - t0 > limit_ns) return false;
    }
    return false;
}

// A barrier of the warps that have the logits, without the list warp.
__device__ __forceinline__ void data_barrier() { asm volatile("bar.sync 1, %0;" ::"n"(kThreads) : "memory"); }

// ---- one pass: a row on chip -------------------------------------------------------------------------
//
// A cluster of `blocks` blocks takes row after row, each block a slice of `slice` tokens, and each of
// its eight data warps a segment of `per` 16-byte vectors of that, which only this warp loads, sums
// and turns into gradients: as soon as it is done with its segment of a row (loss alone: as soon as it
// is summed) it starts the copy of the next row's, so that copies run on under the rest. A ninth warp
// prepares the list of the next row meanwhile. The row lies in shared memory at the phase of 16
// bytes that it has in global memory, -infinity in what is left of the first and last vector. The
// list's tokens are taken out before the rest is summed; the blocks' sums go to every block of the
// cluster, whose barriers in shared memory they arrive at. The logits are read once.
//
// Waits that run out. A block waits longer for the others' sums than they can wait for their copies,
// so a copy that is late, or never lands, reaches the others as a sum (of NaN) and not as silence. A
// warp whose copy has not landed starts no other, one that has waited for the cluster in vain exchanges
// nothing more (its barriers' phases would no longer be the rows'): all its later rows are NaN.
// The late block still writes to the others, so a warp that gave up does not end, and with
// it its block's shared memory does not go, before every other warp of the cluster has ended or
// given up as well; a block whose exchanges were all answered is written to no more.
// kLate, for tests of that: the waits for the cluster end after kLateLimitNs, and the blocks of
// rank 1 sleep for much longer before their first exchange.
constexpr uint64_t kLateLimitNs = 2000000, kLateNs = 20 * kLateLimitNs;

template <typename IO, bool kGrad, bool kLate>
__global__ void __launch_bounds__(kThreads + 32, 3) k_distill_row(DistillArgs a, int blocks, int slice, int per)
{
    constexpr int E = Vec<IO>::kN;
    extern __shared__ __align__(16) unsigned char dyn[];
    __shared__ RowInfo info[2];
    __shared__ unsigned seen[kSeenWords];
    // each warp's sum, rows by turns, and each block's, by turns over the rows that have any (one that
    // has none is not waited for, so a block might run two rows ahead there)
    __shared__ float2 part[2][kWarps], parts[2][8];
    __shared__ __align__(8) uint64_t bars[kWarps], joins[2];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t step = gridDim.x / blocks;
    const int rank = (int)(blockIdx.x % blocks);
    const int64_t v0 = (int64_t)rank * slice;
    const int len = v0 >= a.V ? 0 : (int)(a.V - v0 < slice ? a.V - v0 : slice);
    IO* buf = reinterpret_cast<IO*>(dyn);
    unsigned char* lists = dyn + (size_t)kWarps * per * 16;
    const float k2 = a.inv_tau * kLog2e;

    auto row_of = [&](int64_t n) { return static_cast<const IO*>(a.logits) + n * a.zs; };
    auto weight_of = [&](int64_t n) { return n < a.N && a.weight ? a.weight[n] : 1.0f; };
    auto list_of = [&](int turn) {
        return teacher_at(lists + (size_t)turn * padded(a.K) * kTeacherWords * 4, a.K);
    };
    int64_t n = blockIdx.x / blocks;
    if (tid == 0) {
        for (int q = 0; q < 2; ++q) mbar_init(smem_u32(&joins[q]), (uint32_t)blocks);
        for (int q = 0; q < kWarps; ++q) mbar_init(smem_u32(&bars[q]), 1);
        mbar_init_fence();
    }
    __syncthreads();
    if (blocks > 1) {
        cluster_arrive();      // every block is running, its barriers made, before another reaches into it
        cluster_wait();
    }

    if (warp == kWarps) {
        // the first kAhead entries a lane of the next row's list are on their way while this row's are
        // prepared: first their tokens and values, then the student's logits there
        constexpr int kAhead = 4;
        int token[kAhead];
        float top[kAhead], logit[kAhead], lse = 0.0f;
        auto fetch = [&](int64_t n) {
#pragma unroll
            for (int q = 0; q < kAhead; ++q) {
                const int j = lane + 32 * q;
                token[q] = j < a.K ? token_at(a, n * a.K + j) : -1;
                top[q] = j < a.K ? top_at(a, n * a.K + j) : 0.0f;
            }
            if (a.top_lse) lse = a.top_lse[n];
        };
        auto gather = [&](int64_t n) {
            const IO* z = row_of(n);
#pragma unroll
            for (int q = 0; q < kAhead; ++q) {
                logit[q] = token[q] < 0 ? -INFINITY : to_f32(z[token[q]]);
            }
        };
        float w = weight_of(n);
        fetch(n);
        gather(n);
        for (int turn = 0; n < a.N; n += step, turn ^= 1) {
            const bool more = n + step < a.N;
            const float next_w = weight_of(n + step), this_lse = lse;
            const Teacher t = list_of(turn);
#pragma unroll
            for (int q = 0; q < kAhead; ++q) {
                const int j = lane + 32 * q;
                if (j >= padded(a.K)) continue;
                t.token[j] = token[q];
                t.t[j] = token[q] < 0 ? -INFINITY : top[q];
                t.z[j] = logit[q];
            }
            for (int j = lane + 32 * kAhead; j < padded(a.K); j += 32) put_entry(a, n, row_of(n), t, j);
            if (more) fetch(n + step);
            __syncwarp();
            const List list = prepare_list(a, this_lse, t, seen);
            if (more) gather(n + step);
            if (lane == 0) info[turn] = RowInfo{list, w, next_w};
            w = next_w;
            __syncthreads();
        }
        return;
    }

    const uint32_t bar = smem_u32(&bars[warp]);
    const int s0 = warp * per;
    // this warp's segment: vectors [s0, s1) of the slice as it lies in 16 bytes, [lo, hi) of them whole
    auto segment = [&](int phase, int& s1, int& lo, int& hi) {
        const int nvec = len ? (phase + len + E - 1) / E : 0;
        s1 = max(s0, min(s0 + per, nvec));
        lo = max(s0, phase ? 1 : 0);
        hi = max(lo, min(s1, (phase + len) / E));
    };
    auto begin = [&](int64_t n) {
        const IO* z = row_of(n) + v0;
        const int phase = (int)phase_of(z, sizeof(IO));
        int s1, lo, hi;
        segment(phase, s1, lo, hi);
        if (lane == 0) {
            const uint32_t bytes = (uint32_t)(hi - lo) * 16;
            mbar_arrive_expect(bar, bytes);
            if (bytes) bulk_load(smem_u32(buf + lo * E), z - phase + lo * E, bytes, bar);
        }
        // the ends that no 16-byte copy covers
        if (lane < E) {
            if (phase && s0 == 0 && s1 > 0)
                buf[lane] = lane >= phase && lane - phase < len ? z[lane - phase] : from_f32<IO>(-INFINITY);
            const int last = (phase + len) / E, at = last * E + lane - phase;
            if ((phase + len) % E && last >= s0 && last < s1 && !(phase && last == 0))
                buf[last * E + lane] = at < len ? z[at] : from_f32<IO>(-INFINITY);
        }
    };
    if (!(weight_of(n) == 0.0f)) begin(n);
    uint32_t parity = 0, met = 0;
    bool copied = true, joined = true;      // whether no wait of this warp has run out
    for (int turn = 0; n < a.N; n += step, turn ^= 1) {
        __syncthreads();                    // the list of this row is ready
        const Teacher t = list_of(turn);
        const RowInfo& row = info[turn];
        const List list = row.list;
        const float w = row.w;
        const bool live = !(w == 0.0f) && (a.top_lse || !(list.mass == 0.0f));
        bool next = n + step < a.N && !(row.next_w == 0.0f);        // whether there is a row to copy
        const IO* z = row_of(n) + v0;
        IO* d = kGrad ? static_cast<IO*>(a.dlogits) + n * a.ds + v0 : nullptr;
        const int phase = (int)phase_of(z, sizeof(IO));
        int s1, lo, hi;
        segment(phase, s1, lo, hi);
        // the list's tokens in this warp's segment
        auto mine = [&](int j, int& at) {
            const int64_t k = (int64_t)t.first[j] - v0;
            at = (int)k;
            return t.first[j] >= 0 && k >= 0 && k < len && phase + k >= s0 * E && phase + k < s1 * E;
        };
        if (!(w == 0.0f) && copied) {
            copied = __all_sync(0xffffffffu, mbar_wait(bar, parity) || mbar_wait(bar, parity));
            parity ^= 1;
            if (!copied) note_timeout();
        }
        next = next && copied;
        RowGrad g{0.0f, 0.0f, 0.0f, 0.0f};
        float2 rest = make_float2(-INFINITY, 0.0f), all = rest;
        if (live) {
            __syncwarp();
            for (int j = lane; j < a.K; j += 32) {
                int at;
                if (mine(j, at)) buf[phase + at] = from_f32<IO>(-INFINITY);
            }
            __syncwarp();
            rest = sum_vectors<IO>(buf, s0 + lane, 32, s1, k2);
            rest = warp_join(rest.x, rest.y, k2);
            if (!copied) rest.y = __int_as_float(0x7fc00000);
            if (lane == 0) part[turn][warp] = rest;
            if (!kGrad && next) {
                fence_async();
                __syncwarp();
                begin(n + step);
            }
            data_barrier();
            rest = lane < kWarps ? part[turn][lane] : make_float2(-INFINITY, 0.0f);
            rest = warp_join(rest.x, rest.y, k2);
            if (blocks > 1 && joined) {
                const int slot = met & 1;
                if (kLate && met == 0 && rank == 1) {
                    const uint64_t t0 = global_ns();
                    for (int k = 0; k < 1000000 && global_ns() - t0 < kLateNs; ++k) __nanosleep(1000);
                }
                if (warp == 0 && lane < blocks) {
                    store_remote(smem_u32(&parts[slot][rank].x), (uint32_t)lane, rest.x);
                    store_remote(smem_u32(&parts[slot][rank].y), (uint32_t)lane, rest.y);
                    arrive_remote(smem_u32(&joins[slot]), (uint32_t)lane);
                }
                constexpr uint64_t limit = kLate ? kLateLimitNs : 3 * kWaitLimitNs;
                joined = __all_sync(0xffffffffu, wait_cluster(smem_u32(&joins[slot]), met >> 1 & 1, limit));
                if (!joined) note_timeout();
                ++met;
                rest = lane < blocks ? parts[slot][lane] : make_float2(-INFINITY, 0.0f);
                rest = warp_join(rest.x, rest.y, k2);
            }
            if (!joined) rest.y = __int_as_float(0x7fc00000);
            all = join(rest, make_float2(list.m, list.s), k2);
            g = row_grad(a, list, rest, all, k2);
        }
        if (kGrad) {
            const float f = w * a.inv_tau, coef = f * g.coef;
            const Scale c = scale_of(g.rest, k2);
            auto grad = [&](int at) {
                return live ? from_f32<IO>(coef * fast_exp2(fmaf(to_f32(buf[phase + at]), c.k, -c.c))) : from_f32<IO>(0.0f);
            };
            if (phase_of(d, sizeof(IO)) == (uint32_t)phase) {
                const float2 kk = hold(c.k), mc = hold(-c.c), cc = hold(coef);
                IO* o = d - phase;
                if (live) {
#pragma unroll 4
                    for (int k = lo + lane; k < hi; k += 32) {
                        Vec<IO> v = load_vec<IO>(buf + k * E);
                        grad_vector(v, kk, mc, cc);
                        store_vec(o + k * E, v);
                    }
                } else {
                    Vec<IO> v;
#pragma unroll
                    for (int e = 0; e < E; ++e) v.v[e] = from_f32<IO>(0.0f);
                    for (int k = lo + lane; k < hi; k += 32) store_vec(o + k * E, v);
                }
                // what is left of the segment's first and last vector
                if (lane < E) {
                    if (phase && s0 == 0 && lane >= phase && lane - phase < len) d[lane - phase] = grad(lane - phase);
                    const int last = (phase + len) / E, at = last * E + lane - phase;
                    if ((phase + len) % E && last >= s0 && last < s1 && !(phase && last == 0) && at < len) d[at] = grad(at);
                }
            } else {
                // rows of logits and gradient that lie differently in 16 bytes: element by element
                for (int k = max(s0 * E - phase, 0) + lane; k < min(s1 * E - phase, len); k += 32) d[k] = grad(k);
            }
            if (next) {
                fence_async();
                __syncwarp();
                begin(n + step);
            }
            __syncwarp();
            if (live) {
                const Scale top = scale_of(g.top, k2);
                for (int j = lane; j < a.K; j += 32) {
                    int at;
                    if (mine(j, at)) d[at] = from_f32<IO>(f * (fast_exp2(fmaf(t.z[j], top.k, -top.c)) * g.inv - t.total[j]));
                }
            }
        } else if (!live && next) {
            fence_async();
            __syncwarp();
            begin(n + step);
        }
        if (rank == 0 && warp == 0) {
            const float loss = live ? w * row_loss(a, t, list, rest, all, k2) : 0.0f;
            if (lane == 0) {
                a.loss[n] = loss;
                if (a.stats) *reinterpret_cast<float4*>(a.stats + 4 * n) = make_float4(g.top, g.inv, g.rest, g.coef);
            }
        }
    }
    if (!joined) {
        __syncwarp();
        cluster_arrive();
        cluster_wait();        // for the warps that have not ended; each of their waits is bounded
    }
}

// ---- rows longer than a cluster holds ----------------------------------------------------------------

// One block per row; pieces of the row pass through shared memory, where the list's tokens are
// taken out before the rest is summed.
constexpr int kPieceBytes = 32768;

template <typename IO>
__global__ void __launch_bounds__(kThreads) k_distill_long(DistillArgs a)
{
    constexpr int E = Vec<IO>::kN, kPiece = kPieceBytes / (int)sizeof(IO);
    extern __shared__ __align__(16) unsigned char dyn[];
    __shared__ List list;
    __shared__ unsigned seen[kSeenWords];
    __shared__ float2 part[kWarps];
    IO* piece = reinterpret_cast<IO*>(dyn);
    const Teacher t = teacher_at(dyn + kPieceBytes, a.K);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t n = blockIdx.x;
    const float w = a.weight ? a.weight[n] : 1.0f;
    const float k2 = a.inv_tau * kLog2e;
    const IO* z = static_cast<const IO*>(a.logits) + n * a.zs;
    List l{};
    if (w != 0.0f) l = read_list(a, n, z, t, seen, &list);
    if (w == 0.0f || (!a.top_lse && l.mass == 0.0f)) {
        if (tid == 0) {
            a.loss[n] = 0.0f;
            if (a.stats) *reinterpret_cast<float4*>(a.stats + 4 * n) = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        }
        return;
    }
    float2 rest = make_float2(-INFINITY, 0.0f);
    for (int64_t v0 = 0; v0 < a.V; v0 += kPiece) {
        const int len = (int)(a.V - v0 < kPiece ? a.V - v0 : kPiece), nvec = (len + E - 1) / E;
        for (int v = tid; v < nvec * E; v += kThreads) piece[v] = v < len ? z[v0 + v] : from_f32<IO>(-INFINITY);
        __syncthreads();
        for (int j = tid; j < a.K; j += kThreads) {
            const int64_t k = t.first[j] - v0;
            if (t.first[j] >= 0 && k >= 0 && k < len) piece[k] = from_f32<IO>(-INFINITY);
        }
        __syncthreads();
        rest = join(rest, sum_vectors<IO>(piece, tid, kThreads, nvec, k2), k2);
        __syncthreads();
    }
    rest = warp_join(rest.x, rest.y, k2);
    if (lane == 0) part[warp] = rest;
    __syncthreads();
    rest = lane < kWarps ? part[lane] : make_float2(-INFINITY, 0.0f);
    rest = warp_join(rest.x, rest.y, k2);
    if (warp == 0) {
        const float2 all = join(rest, make_float2(l.m, l.s), k2);
        const float loss = row_loss(a, t, l, rest, all, k2);
        const RowGrad g = row_grad(a, l, rest, all, k2);
        if (lane == 0) {
            a.loss[n] = w * loss;
            if (a.stats) *reinterpret_cast<float4*>(a.stats + 4 * n) = make_float4(g.top, g.inv, g.rest, g.coef);
        }
    }
}

// ---- gradient from saved statistics ------------------------------------------------------------------
//
// Element by element but for the list, whose tokens are written once more at the end. A block has
// 32 KB of a row; its first warp prepares the list while the others go ahead.

constexpr int kGradSlice = 32768;    // bytes of logits a block

template <typename IO>
__global__ void __launch_bounds__(kThreads) k_distill_grad(DistillArgs a, int blocks)
{
    constexpr int E = 16 / (int)sizeof(IO), kSlice = kGradSlice / (int)sizeof(IO), kVecs = 2;
    extern __shared__ __align__(16) unsigned char dyn[];
    __shared__ unsigned seen[kSeenWords];
    const Teacher t = teacher_at(dyn, a.K);
    const int64_t n = blockIdx.x / blocks, v0 = (blockIdx.x - n * blocks) * (int64_t)kSlice;
    const int len = (int)(a.V - v0 < kSlice ? a.V - v0 : kSlice), tid = threadIdx.x;
    const IO* z = static_cast<const IO*>(a.logits) + n * a.zs + v0;
    IO* d = static_cast<IO*>(a.dlogits) + n * a.ds + v0;
    const float4 st = *reinterpret_cast<const float4*>(a.stats + 4 * n);
    const float w = (a.weight ? a.weight[n] : 1.0f) * (a.dloss ? a.dloss[n] : 1.0f) * a.inv_tau;
    const float k2 = a.inv_tau * kLog2e, coef = w * st.w;
    const Scale c = scale_of(st.z, k2);
    const bool live = !(w == 0.0f) && !(st.y == 0.0f);
    const int phase = (int)phase_of(z, sizeof(IO));
    const bool aligned = phase_of(d, sizeof(IO)) == (uint32_t)phase;
    const int head = aligned ? min(len, (E - phase) % E) : len, nvec = (len - head) / E;
    const float2 kk = both(c.k), mc = both(-c.c), cc = both(coef);
    auto grad = [&](IO v) { return live ? from_f32<IO>(coef * fast_exp2(fmaf(to_f32(v), c.k, -c.c))) : from_f32<IO>(0.0f); };

    if (live) {
        // the student's logits on the list, before anything is written: dlogits may be logits
        for (int j = tid; j < padded(a.K); j += kThreads) put_entry(a, n, z - v0, t, j);
        __syncthreads();
        if (tid < 32) prepare_list(a, a.top_lse ? a.top_lse[n] : 0.0f, t, seen);
    }
    for (int k = tid; k < nvec; k += kThreads * kVecs) {
        Vec<IO> v[kVecs];
#pragma unroll
        for (int q = 0; q < kVecs; ++q)
            if (k + q * kThreads < nvec) v[q] = load_vec<IO>(z + head + (k + q * kThreads) * E);
#pragma unroll
        for (int q = 0; q < kVecs; ++q) {
            if (k + q * kThreads >= nvec) continue;
            if (live) {
                grad_vector(v[q], kk, mc, cc);
            } else {
#pragma unroll
                for (int e = 0; e < E; ++e) v[q].v[e] = from_f32<IO>(0.0f);
            }
            store_vec(d + head + (k + q * kThreads) * E, v[q]);
        }
    }
    for (int k = tid; k < head; k += kThreads) d[k] = grad(z[k]);
    for (int k = head + nvec * E + tid; k < len; k += kThreads) d[k] = grad(z[k]);
    if (!live) return;
    __syncthreads();
    const Scale top = scale_of(st.x, k2);
    for (int j = tid; j < a.K; j += kThreads) {
        const int64_t k = t.first[j] - v0;
        if (t.first[j] >= 0 && k >= 0 && k < len) d[k] = from_f32<IO>(w * (fast_exp2(fmaf(t.z[j], top.k, -top.c)) * st.y - t.total[j]));
    }
}

// How a row is shared out: the fewest blocks whose slices are at most kSliceWant bytes, so that three
// of them fit an SM and one row's copy overlaps another's arithmetic and stores (8192 x 32000
// bfloat16: 192 us with slices of 64 KB, 270 us with 32 KB; 8192 x 131072: 848 and 1,332 us); more
// while the launch would leave SMs without a block (4 x 32000 float32: 7.8 us with eight blocks a row,
// 9.0 us with two); larger slices when eight blocks are not enough.
constexpr int kSliceWant = 65536 + 1024, kSliceMost = 188416;
constexpr size_t kSmemMost = 231424;    // of a block, beside its static part

struct Plan {
    int blocks, slice;    // slice in tokens; blocks 0: longer than a cluster holds
};

Plan plan_for(int64_t N, int64_t V, int elem, int sms)
{
    const int64_t bytes = V * elem;
    int64_t c = 1;
    while (c < 8 && (bytes + c - 1) / c > kSliceWant) c *= 2;
    if ((bytes + c - 1) / c > kSliceMost) return Plan{0, 0};
    while (c < 8 && N * c < sms && bytes / c > 8192) c *= 2;
    const int64_t unit = 16 / elem, per = (V + c - 1) / c;
    return Plan{(int)c, (int)((per + unit - 1) / unit * unit)};
}

}  // namespace

size_t distill_workspace_bytes(int64_t N, int64_t V, int dtype)
{
    return plan_for(N, V, dtype == OB_F32 ? 4 : 2, 152).blocks ? 0 : (size_t)N * 4 * sizeof(float);
}

// How many clusters of a kernel fit the device: asked again only when something it depends on is
// another than at this thread's last call (the query takes several microseconds).
struct Resident {
    int device = -1, blocks = 0, clusters = 0;
    size_t smem = 0;
};

template <typename IO, bool kGrad, bool kLate = false>
static cudaError_t run_row(const DistillArgs& a, const Plan& p, const DeviceFacts& dev, cudaStream_t s)
{
    constexpr int E = Vec<IO>::kN;
    constexpr auto kernel = k_distill_row<IO, kGrad, kLate>;
    const int per = (p.slice / E + 1 + kWarps - 1) / kWarps;
    const size_t smem = (size_t)kWarps * per * 16 + (size_t)2 * padded(a.K) * kTeacherWords * 4;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(a.N * p.blocks));
    cfg.blockDim = dim3(kThreads + 32);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)p.blocks;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return with_opt_in<kernel>(dev.device, kSmemMost, [&] {
        // one wave: a cluster takes row after row
        if (a.N * p.blocks > dev.sms) {
            static thread_local Resident r;
            if (r.device != dev.device || r.blocks != p.blocks || r.smem != smem) {
                int n = 0;
                const cudaError_t e = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg);
                if (e != cudaSuccess) return e;
                r.device = dev.device, r.blocks = p.blocks, r.smem = smem, r.clusters = std::max(n, 1);
            }
            cfg.gridDim = dim3((unsigned)(std::min<int64_t>(a.N, r.clusters) * p.blocks));
        }
        const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, a, p.blocks, p.slice, per);
        return e != cudaSuccess ? e : cudaGetLastError();
    });
}

cudaError_t launch_distill(const DistillArgs& a, void* ws, cudaStream_t s)
{
    DeviceFacts dev;
    const cudaError_t e = current_device(&dev);
    if (e != cudaSuccess) return e;
    return by_dtype(a.dtype, [&](auto io) {
        using IO = decltype(io);
        const Plan p = plan_for(a.N, a.V, (int)sizeof(IO), dev.sms);
        if (p.blocks) return a.dlogits ? run_row<IO, true>(a, p, dev, s) : run_row<IO, false>(a, p, dev, s);
        DistillArgs b = a;
        if (!b.stats && b.dlogits) b.stats = static_cast<float*>(ws);
        const size_t smem = kPieceBytes + (size_t)padded(a.K) * kTeacherWords * 4;
        const cudaError_t e = with_opt_in<k_distill_long<IO>>(dev.device, kSmemMost, [&] {
            k_distill_long<IO><<<(unsigned)b.N, kThreads, smem, s>>>(b);
            return cudaGetLastError();
        });
        return e != cudaSuccess || !b.dlogits ? e : launch_distill_bwd(b, s);
    });
}

cudaError_t launch_distill_late(const DistillArgs& a, cudaStream_t s)
{
    DeviceFacts dev;
    const cudaError_t e = current_device(&dev);
    if (e != cudaSuccess) return e;
    const Plan p = plan_for(a.N, a.V, sizeof(float), dev.sms);
    return p.blocks > 1 ? run_row<float, true, true>(a, p, dev, s) : cudaErrorInvalidValue;
}

cudaError_t distill_status(unsigned* status, cudaStream_t s) { return take_status(wait_status, status, s); }

cudaError_t launch_distill_bwd(const DistillArgs& a, cudaStream_t s)
{
    return by_dtype(a.dtype, [&](auto io) {
        using IO = decltype(io);
        const int64_t blocks = (a.V * (int64_t)sizeof(IO) + kGradSlice - 1) / kGradSlice;
        if (a.N * blocks >= (int64_t{1} << 31)) return cudaErrorInvalidConfiguration;
        k_distill_grad<IO><<<(unsigned)(a.N * blocks), kThreads, (size_t)padded(a.K) * kTeacherWords * 4, s>>>(a, (int)blocks);
        return cudaGetLastError();
    });
}

}  // namespace ob
