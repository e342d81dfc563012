// The gated scan's element arithmetic, packed loads and the look-back along a chain of tiles.
#pragma once

#include "ob_student.cuh"
#include "ob_student.h"
#include "ob_tma.cuh"

namespace ob {

__device__ __forceinline__ float fast_rcp(float v)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

__device__ __forceinline__ float fast_sqrt(float v)
{
    float r;
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// ---- the gates ------------------------------------------------------------------------------------
//
// w = decay*s(r), a = exp(-w), b = sqrt(1 - a^2). For small w, 1 - a^2 = 2w*P(w) with
// P(w) = (1 - exp(-2w))/(2w) keeps the precision that a near 1 has rounded away, and as
// (2 decay)*(s(r)*P) its root does not vanish where w underflows. P is a polynomial in
// l = -w log2(e), the argument of ex2: the degree-5 interpolation at the Chebyshev points of
// 0 <= w <= 1/4 (within 1.5e-9). For larger w, 1 - a^2 itself is within a few roundings. Both are
// carried divided by 2 decay and times 2^64 through the root, so that the fast root, which flushes
// subnormal arguments, meets none.

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kTwo32 = 4294967296.0f, kTwoM32 = 1.0f / 4294967296.0f;
constexpr float kSmallW = 0.25f;

// The packed constants of the gates.
struct Held {
    float2 p[6], half_log2e, two_m32;
};

__device__ __forceinline__ Held held()
{
    constexpr double t = 4294967296.0;
    Held c;
    c.p[0] = hold((float)(t * 0.9999999987426018));
    c.p[1] = hold((float)(t * 0.99999963754846));
    c.p[2] = hold((float)(t * 0.6666496747460877));
    c.p[3] = hold((float)(t * 0.33304058265219977));
    c.p[4] = hold((float)(t * 0.1310338180861702));
    c.p[5] = hold((float)(t * 0.03594893499156057));
    c.half_log2e = hold(-0.5f * kLog2e);
    c.two_m32 = hold(kTwoM32);
    return c;
}

// Constants of a pair of channels (or of one channel, twice).
struct Rate {
    float2 minus;    // -decay * 2^-32
    float2 small;    // 2^32 s(r) below which w is small
    float2 inv;      // 2^64/(2*decay)
    float2 minus_inv;
    float2 root;     // sqrt(2*decay) * 2^-32
};

__device__ __forceinline__ Rate rate(float2 d)
{
    Rate k;
    k.minus = mul2(d, both(-kTwoM32));
    const float2 r = make_float2(fast_rcp(d.x), fast_rcp(d.y));
    k.small = mul2(r, both(kSmallW * kTwo32));
    k.inv = mul2(r, both(0.5f * kTwo32 * kTwo32));
    k.minus_inv = mul2(r, both(-0.5f * kTwo32 * kTwo32));
    // through 2^32 d: the fast root would flush a subnormal decay
    const float2 s = mul2(d, both(kTwo32));
    k.root = mul2(make_float2(fast_sqrt(s.x), fast_sqrt(s.y)), both(1.4142135623730951f / 65536.0f * kTwoM32));
    return k;
}

struct Gates {
    float2 a, s32, si, b;   // a, 2^32 s(r), s(i), sqrt(1 - a^2)
};

// 2^32/(1 + exp(-v)) as 1/(2^-32 + (2^-32 n) n), n = exp(-v/2): nothing overflows before the result is
// below the smallest subnormal number, so a shut gate keeps its precision. The argument of ex2 has
// a rounding error of |v| units of 2^-24, which drowns in a 16-bit input's own; for float32
// inputs (kExact) it is found exactly and n corrected by it.
template <bool kExact>
__device__ __forceinline__ float2 logistic32(float2 v, const Held& c)
{
    const float2 m = mul2(v, c.half_log2e);
    float2 n = make_float2(fast_exp2(m.x), fast_exp2(m.y));
    if constexpr (kExact) {
        constexpr float hi = -0.5f * kLog2e;
        constexpr float lo = (float)(-0.72134752044448170367996234050095 - (double)hi);
        float2 e = fma2(v, c.half_log2e, make_float2(-m.x, -m.y));
        e = fma2(v, both(lo), e);
        e = make_float2(fminf(e.x, 1.0f), fminf(e.y, 1.0f));     // NaN, from an infinite v, becomes 1
        // a factor that is finite and not 0, so that an overflown n stays infinite (of either sign: it is squared)
        n = mul2(n, fma2(e, both(0.6931471805599453f), both(1.0f)));
    }
    const float2 d = fma2(mul2(n, c.two_m32), n, c.two_m32);
    return make_float2(fast_rcp(d.x), fast_rcp(d.y));
}

// r = -infinity makes an element that changes nothing: a = 1, b = 0. a is expf of -w and not the
// cheaper ex2: near 1 that has a one-sided error of some 1e-8, of the other sign than expf's, and
// memories of thousands of tokens add the two up to some 1e-5 of states and gradients, apart from
// what other float32 implementations of the formula have there.
template <bool kExact>
__device__ __forceinline__ Gates gates(float2 r, float2 i, const Rate& k, const Held& c)
{
    Gates g;
    g.s32 = logistic32<kExact>(r, c);
    g.si = mul2(logistic32<kExact>(i, c), c.two_m32);
    const float2 v = mul2(k.minus, g.s32);  // -w
    g.a = make_float2(expf(v.x), expf(v.y));
    float2 p = fma2(v, c.p[5], c.p[4]);     // 2^32 * P
    p = fma2(v, p, c.p[3]);
    p = fma2(v, p, c.p[2]);
    p = fma2(v, p, c.p[1]);
    p = fma2(v, p, c.p[0]);
    p = mul2(g.s32, p);
    const float2 large = fma2(mul2(g.a, g.a), k.minus_inv, k.inv);
    const float2 arg = make_float2(g.s32.x < k.small.x ? p.x : large.x, g.s32.y < k.small.y ? p.y : large.y);
    g.b = mul2(make_float2(fast_sqrt(arg.x), fast_sqrt(arg.y)), k.root);
    return g;
}

// The decay over steps with a reset among them, which drops whatever state came before, even an
// infinite one or a NaN. Decays and their products are never -0, and one that is small enough to have become +0
// is no reset: an infinite state or a NaN goes on through it.
constexpr float kResetDecay = -0.0f;
__device__ __forceinline__ bool is_reset(float a) { return __float_as_uint(a) == 0x80000000u; }

// ---- a lane's elements ----------------------------------------------------------------------------
//
// A lane has one word per row and tensor: two adjacent 16-bit channels, or one channel. With one
// channel a pair is two steps.

template <typename IO, int V>
__device__ __forceinline__ float2 unpack(unsigned w)
{
    static_assert(V == 2 && sizeof(IO) == 2, "two 16-bit channels");
    return unpack_pair(w, IO{});
}

template <typename IO>
__device__ __forceinline__ float unpack_one(unsigned w)
{
    IO v;
    memcpy(&v, &w, sizeof(IO));
    return to_f32(v);
}

template <typename IO>
__device__ __forceinline__ unsigned pack_one(float v)
{
    const IO o = from_f32<IO>(v);
    unsigned w = 0u;
    memcpy(&w, &o, sizeof(IO));
    return w;
}

// The pair `m` of a lane's rows, row j's word being at p[j*32].
template <typename IO, int V>
__device__ __forceinline__ float2 pair_at(const unsigned* p, int m)
{
    if constexpr (V == 2) return unpack<IO, V>(p[m * 32]);
    else return make_float2(unpack_one<IO>(p[2 * m * 32]), unpack_one<IO>(p[(2 * m + 1) * 32]));
}

// Moves a pointer on by one addition: left to itself the compiler forms each row's address of an
// unrolled loop anew, with several operations (the backward pass of 16 x 4096 x 4096 bfloat16 took
// 1,029 us so and 937 with this).
template <typename T>
__device__ __forceinline__ void advance(T*& p, int64_t bytes)
{
    p = reinterpret_cast<T*>(reinterpret_cast<char*>(p) + bytes);
    asm volatile("" : "+l"(p));
}

template <typename T>
__device__ __forceinline__ void advance(const T*& p, int64_t bytes)
{
    p = reinterpret_cast<const T*>(reinterpret_cast<const char*>(p) + bytes);
    asm volatile("" : "+l"(p));
}

template <typename IO>
__device__ __forceinline__ void store_two(IO* p, float2 v)
{
    *reinterpret_cast<unsigned*>(p) = pack_pair(v, IO{});
}

// ---- look-back ------------------------------------------------------------------------------------
//
// A chain is one row's block of 32*V channels; its tiles are its chunks of time, in the order
// in which the state passes. Tiles are numbered chunk by chunk over all chains and taken in
// that order from a counter, so a tile only ever waits for tiles already taken (the single-pass
// scan with decoupled look-back, D. Merrill and M. Garland, 2016). A tile publishes
// what it makes of any state (A, H: h -> A*h + H), then the state it ends with. State and
// flag travel in one 16-byte word, written and read whole, so no fence orders them. Since the
// state a tile hands on is by definition A*carry + H (H alone where A marks a reset), joined by the
// same operations here and in the tile's own block, it does not matter how many tiles back a final
// state is found: the same bits, for states that are not finite too.

constexpr unsigned kPartial = 1u, kFinal = 2u;
constexpr int kWindow = 32;             // tiles looked at before waiting for the oldest of them
constexpr size_t kScanHeader = 256;     // workspace: status word, tile counter, then the slots

struct alignas(16) Slot {
    float a, h;
    unsigned flag, unused;
};

__device__ __forceinline__ Slot read_slot(const Slot* p)
{
    uint64_t lo, hi;
    asm volatile(
        "{\n\t.reg .b128 t;\n\t"
        "ld.relaxed.gpu.global.b128 t, [%2];\n\t"
        "mov.b128 {%0, %1}, t;\n\t}"
        : "=l"(lo), "=l"(hi)
        : "l"(p)
        : "memory");
    return Slot{__uint_as_float((unsigned)lo), __uint_as_float((unsigned)(lo >> 32)), (unsigned)hi, 0u};
}

__device__ __forceinline__ void write_slot(Slot* p, float a, float h, unsigned flag)
{
    const uint64_t lo = (uint64_t)__float_as_uint(a) | (uint64_t)__float_as_uint(h) << 32;
    asm volatile(
        "{\n\t.reg .b128 t;\n\t"
        "mov.b128 t, {%1, %2};\n\t"
        "st.relaxed.gpu.global.b128 [%0], t;\n\t}" ::"l"(p),
        "l"(lo), "l"((uint64_t)flag)
        : "memory");
}

// 1 once any wait of the scans has run out (read and cleared by scan_status).
static __device__ unsigned scan_wait_status;

// Waits (bounded) until the slot holds at least `flag`. A wait that runs out sets the workspace's
// status word and the one above and stands in a final NaN.
__device__ __forceinline__ Slot await_slot(const Slot* p, unsigned flag, unsigned* status, uint64_t limit_ns = kWaitLimitNs)
{
    Slot s = read_slot(p);
    if (s.flag >= flag) return s;
    const uint64_t t0 = global_ns();
    for (uint32_t spins = 0; spins < (1u << 30); ++spins) {
        s = read_slot(p);
        if (s.flag >= flag) return s;
        if (global_ns() - t0 > limit_ns) break;
    }
    atomicMax(status, kStatusWaitTimeout);
    atomicMax(&scan_wait_status, kStatusWaitTimeout);
    return Slot{0.0f, __int_as_float(0x7fc00000), kFinal, 0u};
}

// The state that reaches tile `pos` of a chain (pos >= 1 tiles before it; the slots of the tile
// before are at `prev`, those of earlier ones `stride` slots lower each). All kWarps warps of the
// block call it; lane l has channels l*V .. l*V+V-1. win: [kWindow][32*V] in shared memory; an
// entry's A is -1 where it is final.
template <int V, int kWarps, bool kReset>
__device__ void look_back(const Slot* prev, int64_t stride, int pos, float2* win, float carry[V], unsigned* status)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int rows = 0;
    for (int base = 0; base < kWindow; base += kWarps) {
        const int back = base + warp;
        if (back < pos) {
            const unsigned need = back == kWindow - 1 ? kFinal : kPartial;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const Slot s = await_slot(prev - back * stride + lane * V + v, need, status);
                win[back * 32 * V + lane * V + v] = make_float2(s.flag == kFinal ? -1.0f : s.a, s.h);
            }
        }
        __syncthreads();
        rows = base + kWarps < pos ? base + kWarps : pos;
        int found = 1;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            int f = 0;
            for (int k = base; k < rows; ++k) f |= win[k * 32 * V + lane * V + v].x < 0.0f;
            found &= f;
        }
        if (__syncthreads_and(found)) break;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const float2* w = win + lane * V + v;
        int k = 0;
        while (k < rows - 1 && !(w[k * 32 * V].x < 0.0f)) ++k;     // a NaN is no final entry
        float c = w[k * 32 * V].y;
        for (--k; k >= 0; --k) {
            const float2 e = w[k * 32 * V];
            c = kReset && is_reset(e.x) ? e.y : fmaf(e.x, c, e.y);
        }
        carry[v] = c;
    }
}

}  // namespace ob
