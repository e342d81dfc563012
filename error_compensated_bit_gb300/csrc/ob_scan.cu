// The gated scan: forward, backward and single-token kernels.
//
//   a_t = exp(-decay*s(r_t));  h_t = a_t*h_{t-1} + sqrt(1 - a_t^2)*s(i_t)*x_t
//
// What has to move per element of e bytes: forward x, r, i in and y out, 4e; backward x, r, i, dy in
// and dx, dr, di out, 7e (and in training 4/64 bytes of saved states, written and read). Both
// are one pass: the scan over time is split into tiles whose maps h -> A*h + H are joined within a
// block through shared memory and along time by look-back (ob_scan.cuh), each element being gated
// once and kept in registers until the state that reaches its tile is known.
//
// What bounds them now is the latency of the instructions, with too few warps to hide it: a pair of
// 16-bit elements takes 87 instructions forward and 179 backward (ncu, 8 x 2048 x 2048 bfloat16), and
// with 16 warps an SM (128 registers a thread) 53 and 60% of the issue slots and 38% of DRAM's rate are
// used; a warp mostly waits for a fixed latency or for the arithmetic pipes. Hence the packed arithmetic
// and everything else here that saves instructions. Measured on bfloat16 without resets (CUDA events,
// launches back to back):
//   forward   8 x 2048 x 2048    83 us, 3.2 TB/s;   16 x 4096 x 4096   505 us, 4.3 TB/s
//   backward  8 x 2048 x 2048   162 us, 2.9 TB/s;   16 x 4096 x 4096   937 us, 4.0 TB/s
// The smaller case has 256 chains for 304 blocks.
#include <algorithm>
#include <type_traits>

#include "ob_internal.h"
#include "ob_scan.cuh"

namespace ob {
namespace {

constexpr int kChunk = OB_SCAN_CHUNK;

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Shape of a scan kernel: V channels a lane, L steps a warp, kWarps warps along time; blocks are
// persistent, kBlocks on an SM, and copy the next tile into shared memory while they work on
// one. Each warp copies just the rows that it will read itself.
constexpr int kWarps = 8, kThreads = 32 * kWarps, kBlocks = 2;

template <int V, int L>
struct Tile {
    static constexpr int kCols = 32 * V, kSteps = L * kWarps, kPairs = L * V / 2;
};

// How the tiles are shared out. A block takes items of `run` consecutive tiles of one chain; within an
// item the state passes in the block, from item to item by look-back.
struct Grid {
    int nchains, ncols, nchunks, run, nitems;
    FastDiv by_chains, by_cols;
};

__device__ __forceinline__ int divide(int n, const FastDiv& f)
{
    if (f.d == 1) return n;
    const uint32_t t = __umulhi((uint32_t)n, f.m);
    return (int)((t + (((uint32_t)n - t) >> 1)) >> (f.l - 1));
}

// Where a tile is.
struct Place {
    int item, chunk;          // chunk counts along the direction of the scan
    int b, col;               // row, this lane's first channel
};

template <int V>
__device__ __forceinline__ Place place_of(int item, const Grid& g)
{
    Place q;
    const int part = divide(item, g.by_chains), chain = item - part * g.nchains, row = divide(chain, g.by_cols);
    q.item = item;
    q.chunk = part * g.run;
    q.b = row;
    q.col = (chain - row * g.ncols) * 32 * V + (threadIdx.x & 31) * V;
    return q;
}

// Whether a tile is its item's last.
__device__ __forceinline__ bool ends(const Place& q, const Grid& g)
{
    return q.chunk + 1 == g.nchunks || q.chunk + 1 == (divide(q.item, g.by_chains) + 1) * g.run;
}

// The L reset flags from step t0 on, as bits.
template <int L>
__device__ __forceinline__ unsigned reset_bits(const uint8_t* reset, int b, int T, int t0)
{
    const int lane = threadIdx.x & 31;
    const bool f = lane < L && t0 + lane < T && reset[(int64_t)b * T + t0 + lane];
    return __ballot_sync(0xffffffffu, f);
}

__device__ __forceinline__ void copy4(uint32_t dst, const void* src)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

__device__ __forceinline__ void copy16(uint32_t dst, const void* src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// How a lane's words come into shared memory: 16 bytes at a time (a row's 128 bytes by eight
// lanes) where every row starts on 16 bytes and x, r and i have the same strides (their offsets are
// then computed once), else word by word; a single 16-bit channel, narrower than any
// asynchronous copy, through a register. 16 x 4096 x 4096 bfloat16 forward, backward: 505, 937 us
// wide; 723, 1,061 us by words (the same tensors 4 bytes on); 949, 1,507 us by single channels (2
// bytes on: odd numbers of channels, odd addresses).
enum Copy { kWide, kWord, kPlain };

// What the copies of a tile's tensors have in common.
struct Rows {
    int b, t0, rows, row, c;     // row of the batch; first step, steps there are; this lane's first row, channel
    bool here;
};

template <typename IO, int V, int L, Copy kCopy>
__device__ __forceinline__ Rows rows_of(int b, int t0, int col, const ScanArgs& p)
{
    const int lane = threadIdx.x & 31;
    Rows x;
    x.b = b;
    x.t0 = t0;
    x.rows = max(0, min(L, (int)p.T - t0));
    x.row = kCopy == kWide ? lane >> 3 : 0;
    x.c = kCopy == kWide ? col - lane * V + (lane & 7) * (16 / (int)sizeof(IO)) : col;
    x.here = x.c < (int)p.D;
    return x;
}

__device__ __forceinline__ int64_t offset_in(const ob_view& t, const Rows& x)
{
    return x.b * t.batch + (x.t0 + x.row) * t.time + x.c;
}

// Starts the copy of this warp's L rows of a tensor, [L][32] words at dst; rows that are not there
// become `none`, words of channels that are not there are left as they are.
template <typename IO, int V, int L, Copy kCopy>
__device__ __forceinline__ void stage(unsigned* dst, const ob_view& t, const Rows& x, int64_t offset, unsigned none)
{
    const int lane = threadIdx.x & 31;
    const int rows = t.ptr ? x.rows : 0;
    const IO* p = static_cast<const IO*>(t.ptr) + offset;
    if (x.here) {
        if constexpr (kCopy == kWide) {
            const uint32_t s = smem_u32(dst) + lane * 16;
            const int64_t step = 4 * t.time * (int64_t)sizeof(IO);
            if (rows == L) {
#pragma unroll
                for (int j = 0; j < L; j += 4, advance(p, step)) copy16(s + j * 128, p);
            } else {
                for (int j = x.row; j < rows; j += 4, advance(p, step)) copy16(s + (j - x.row) * 128, p);
            }
        } else if constexpr (kCopy == kWord) {
            const uint32_t s = smem_u32(dst + lane);
            const int64_t step = t.time * (int64_t)sizeof(IO);
            if (rows == L) {
#pragma unroll
                for (int j = 0; j < L; ++j, advance(p, step)) copy4(s + j * 128, p);
            } else {
                for (int j = 0; j < rows; ++j, advance(p, step)) copy4(s + j * 128, p);
            }
        }
    }
    if (rows < L) {
        for (int j = rows; j < L; ++j) dst[j * 32 + lane] = none;
    }
}

// For kPlain, the same through registers: the loads now, their place in shared memory (put_rows) when
// the tile before is done with, so that nothing waits for them.
template <typename IO, int L>
__device__ __forceinline__ void load_rows(unsigned (&w)[L], const ob_view& t, const Rows& x, unsigned none)
{
    const int rows = t.ptr && x.here ? x.rows : 0;
    const IO* p = static_cast<const IO*>(t.ptr) + offset_in(t, x);
    const int64_t step = t.time * (int64_t)sizeof(IO);
#pragma unroll
    for (int j = 0; j < L; ++j, advance(p, step)) {
        w[j] = none;
        if (j < rows) w[j] = __ldg(reinterpret_cast<const unsigned short*>(p));
    }
}

template <int L>
__device__ __forceinline__ void put_rows(unsigned* dst, const unsigned (&w)[L])
{
#pragma unroll
    for (int j = 0; j < L; ++j) dst[j * 32 + (threadIdx.x & 31)] = w[j];
}

// Takes the next item's number. Items taken in the order of their numbers never wait for one that
// no running block has.
__device__ __forceinline__ int next_item(unsigned* counter, int nitems, bool chained, int& plain)
{
    if (chained) return (int)min(atomicAdd(counter, 1u), (unsigned)nitems);
    const int t = plain;
    plain = t + (int)gridDim.x < nitems ? t + (int)gridDim.x : nitems;
    return t;
}

// h along a lane's L steps: u_t becomes h_t, or h_{t-1} with kBefore (after a reset 0). kResets
// says whether there is a reset among the steps; without one a step is one multiply-add.
template <int V, int L, bool kBefore, bool kResets>
__device__ __forceinline__ void run_states(const float2* a, float2* u, float2& h, unsigned resets)
{
    if constexpr (V == 2) {
#pragma unroll
        for (int j = 0; j < L; ++j) {
            if (kResets && (resets >> j & 1u)) h = both(0.0f);
            const float2 n = fma2(a[j], h, u[j]);
            u[j] = kBefore ? h : n;
            h = n;
        }
    } else {
#pragma unroll
        for (int m = 0; m < L / 2; ++m) {
            if (kResets && (resets >> (2 * m) & 1u)) h.x = 0.0f;
            const float n0 = fmaf(a[m].x, h.x, u[m].x);
            const float h1 = kResets && (resets >> (2 * m + 1) & 1u) ? 0.0f : n0;
            const float n1 = fmaf(a[m].y, h1, u[m].y);
            u[m] = kBefore ? make_float2(h.x, h1) : make_float2(n0, n1);
            h.x = n1;
        }
    }
}

// The state after a lane's L steps from h.
template <int V, int L, bool kResets>
__device__ __forceinline__ float2 end_state(const float2* a, const float2* u, float2 h, unsigned resets)
{
    if constexpr (V == 2) {
#pragma unroll
        for (int j = 0; j < L; ++j) {
            if (kResets && (resets >> j & 1u)) h = both(0.0f);
            h = fma2(a[j], h, u[j]);
        }
    } else {
#pragma unroll
        for (int m = 0; m < L / 2; ++m) {
            if (kResets && (resets >> (2 * m) & 1u)) h.x = 0.0f;
            h.x = fmaf(a[m].x, h.x, u[m].x);
            if (kResets && (resets >> (2 * m + 1) & 1u)) h.x = 0.0f;
            h.x = fmaf(a[m].y, h.x, u[m].y);
        }
    }
    return h;
}

// The flow a_t*g_t of the gradient out of a lane's L steps, backwards, from none.
template <typename IO, int V, int L, bool kResets>
__device__ __forceinline__ float2 end_flow(const float2* a, const unsigned* wd, unsigned resets)
{
    float2 f = both(0.0f);
#pragma unroll
    for (int m = L * V / 2 - 1; m >= 0; --m) {
        const float2 dy = pair_at<IO, V>(wd, m);
        if constexpr (V == 2) {
            f = mul2(a[m], add2(f, dy));
            if (kResets && (resets >> m & 1u)) f = both(0.0f);
        } else {
            f.x = a[m].y * (f.x + dy.y);
            if (kResets && (resets >> (2 * m + 1) & 1u)) f.x = 0.0f;
            f.x = a[m].x * (f.x + dy.x);
            if (kResets && (resets >> (2 * m) & 1u)) f.x = 0.0f;
        }
    }
    return f;
}

// The product of a lane's L decays (kResetDecay with a reset among them, which all channels of a row share).
template <int V, int L>
__device__ __forceinline__ float2 product(const float2* a, unsigned resets)
{
    float2 A = both(1.0f);
#pragma unroll
    for (int m = 0; m < L * V / 2; ++m) A = mul2(A, a[m]);
    if (V == 1) A.x *= A.y;
    return resets ? both(kResetDecay) : A;
}

// The decay over two stretches of steps. A reset in either wins, even over the NaN that a NaN gate makes.
__device__ __forceinline__ float2 both_decays(float2 a, float2 b, bool can_reset)
{
    const float2 p = mul2(a, b);
    if (!can_reset) return p;
    const bool r = is_reset(a.x) || is_reset(b.x);
    return make_float2(r ? kResetDecay : p.x, r ? kResetDecay : p.y);
}

// a*h + u, without a*h where a reset is among the steps of a.
__device__ __forceinline__ float2 join(float2 a, float2 h, float2 u, bool can_reset)
{
    const float2 n = fma2(a, h, u);
    if (!can_reset) return n;
    const bool r = is_reset(a.x);
    return make_float2(r ? u.x : n.x, r ? u.y : n.y);
}

// The state that reaches an item, where it is known at once: the initial one for a chain's first, or
// what the item before has published as final.
template <int V>
__device__ __forceinline__ bool arriving(const Slot* before, bool first, const float* initial, bool here, float carry[V])
{
    bool known = true;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        carry[v] = 0.0f;
        if (!first) {
            const Slot s = read_slot(before + (threadIdx.x & 31) * V + v);
            carry[v] = s.h;
            known = known && s.flag == kFinal;
        } else if (here && initial) {
            carry[v] = initial[v];
        }
    }
    return known;
}

template <int V>
__device__ __forceinline__ void publish(Slot* mine, float2 a, float2 h, unsigned flag)
{
    const int lane = threadIdx.x & 31;
    write_slot(mine + lane * V, a.x, h.x, flag);
    if (V == 2) write_slot(mine + lane * V + 1, a.y, h.y, flag);
}

template <int V>
__device__ __forceinline__ void put(float* o, float2 v)
{
    o[0] = v.x;
    if (V == 2) o[1] = v.y;
}

// The decays of a tile's channels, and (backwards) the states saved before it; fetched while the
// tile before is worked on.
template <int V>
__device__ __forceinline__ float2 decay_at(const ScanArgs& p, const Place& q, const Grid& g)
{
    if (q.item >= g.nitems || q.col >= (int)p.D) return both(1.0f);
    return make_float2(p.decay[q.col], p.decay[q.col + V - 1]);
}

template <int V>
__device__ __forceinline__ float2 state_at(const ScanArgs& p, const Place& q, const Grid& g)
{
    if (q.item >= g.nitems || q.col >= (int)p.D) return both(0.0f);
    const float* s = p.states + ((int64_t)q.b * g.nchunks + (g.nchunks - 1 - q.chunk)) * p.D + q.col;
    return make_float2(s[0], s[V - 1]);
}

// kReset: there are reset flags. Without, what follows from them is left out (backward, 16 x 4096 x
// 4096 bfloat16 937 us where the kernel with them takes 1,016).
template <typename IO, int V, int L, Copy kCopy, bool kReset>
__global__ void __launch_bounds__(kThreads, kBlocks) k_scan_fwd(ScanArgs p, Grid g)
{
    using S = Tile<V, L>;
    constexpr bool kExact = sizeof(IO) == 4;
    constexpr int kWords = 3 * L * 32;                    // of a warp's rows
    extern __shared__ __align__(16) unsigned words[];     // [2][kWarps][3][L][32]
    // what each warp makes of a state; two sets by turns, so that one barrier a tile is enough
    __shared__ float2 sa[2][kWarps][32], sh[2][kWarps][32], sc[2][32];
    __shared__ int taken[2];
    const int lane = threadIdx.x & 31, warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
    unsigned* header = static_cast<unsigned*>(p.ws);
    const bool chained = g.nchunks > g.run;
    constexpr bool can_reset = kReset;
    Slot* slots = reinterpret_cast<Slot*>(static_cast<char*>(p.ws) + kScanHeader);
    const int64_t stride = (int64_t)g.nchains * S::kCols;
    unsigned none_r = pack_one<IO>(-INFINITY);
    if (V == 2) none_r |= none_r << 16;
    const int64_t saved = (p.T + kChunk - 1) / kChunk;

    unsigned pending[kCopy == kPlain ? 3 : 1][L];
    auto begin = [&](const Place& q, int buf) {
        if (q.item < g.nitems) {
            const Rows x = rows_of<IO, V, L, kCopy>(q.b, q.chunk * S::kSteps + warp * L, q.col, p);
            if constexpr (kCopy == kPlain) {
                load_rows<IO, L>(pending[0], p.r, x, none_r);
                load_rows<IO, L>(pending[1], p.i, x, 0u);
                load_rows<IO, L>(pending[2], p.x, x, 0u);
            } else {
                unsigned* w = words + (buf * kWarps + warp) * kWords;
                const int64_t at = offset_in(p.x, x);
                stage<IO, V, L, kCopy>(w, p.r, x, kCopy == kWide ? at : offset_in(p.r, x), none_r);
                stage<IO, V, L, kCopy>(w + L * 32, p.i, x, kCopy == kWide ? at : offset_in(p.i, x), 0u);
                stage<IO, V, L, kCopy>(w + 2 * L * 32, p.x, x, at, 0u);
            }
        }
        cp_async_commit();
    };
    auto settle = [&](const Place& q, int buf) {
        if constexpr (kCopy == kPlain) {
            unsigned* w = words + (buf * kWarps + warp) * kWords;
            if (q.item < g.nitems) {
#pragma unroll
                for (int k = 0; k < 3; ++k) put_rows(w + k * L * 32, pending[k]);
            }
        }
    };

    int plain = (int)blockIdx.x;
    if (threadIdx.x == 0) {
        if (!chained && blockIdx.x == 0) header[0] = 0u;
        taken[0] = next_item(header + 1, g.nitems, chained, plain);
    }
    __syncthreads();
    const Held held_ = held();
    Place q = place_of<V>(taken[0], g);
    begin(q, 0);
    settle(q, 0);
    float2 d = decay_at<V>(p, q, g);
    for (int turn = 0; q.item < g.nitems; turn ^= 1) {
        // the item after this one: its number is ready one barrier later, its copies start then
        const bool last = ends(q, g), first = q.chunk == divide(q.item, g.by_chains) * g.run;
        if (last && threadIdx.x == 0) taken[turn ^ 1] = next_item(header + 1, g.nitems, chained, plain);
        Slot* mine = slots + (int64_t)q.item * S::kCols;
        const bool here = q.col < (int)p.D;
        const int t0 = q.chunk * S::kSteps + warp * L;
        const unsigned resets = kReset ? reset_bits<L>(p.reset, q.b, (int)p.T, t0) : 0u;
        float carry[V];
        bool known = true;
        if (first)
            known = arriving<V>(mine - stride, q.chunk == 0, p.h0 ? p.h0 + (int64_t)q.b * p.D + q.col : nullptr, here, carry);
        const Rate k = rate(d);
        cp_async_wait<0>();
        __syncwarp();

        const unsigned* w = words + (turn * kWarps + warp) * kWords + lane;
        float2 a[S::kPairs], u[S::kPairs];
#pragma unroll
        for (int m = 0; m < S::kPairs; ++m) {
            const Gates e = gates<kExact>(pair_at<IO, V>(w, m), pair_at<IO, V>(w + L * 32, m), k, held_);
            a[m] = e.a;
            u[m] = mul2(mul2(e.b, e.si), pair_at<IO, V>(w + 2 * L * 32, m));
        }
        sa[turn][warp][lane] = product<V, L>(a, resets);
        sh[turn][warp][lane] = resets ? end_state<V, L, true>(a, u, both(0.0f), resets)
                                      : end_state<V, L, false>(a, u, both(0.0f), 0u);
        const bool all_known = __syncthreads_and(known);
        Place next = q;
        if (last) next = place_of<V>(taken[turn ^ 1], g);
        else next.chunk += 1;

        const bool more = q.chunk + 1 < g.nchunks;
        float2 tA, tH;      // the tile as one step
        if (warp == 0 || !all_known) {
            tA = sa[turn][0][lane];
            tH = sh[turn][0][lane];
#pragma unroll
            for (int e = 1; e < kWarps; ++e) {
                const float2 aw = sa[turn][e][lane];
                tH = join(aw, tH, sh[turn][e][lane], can_reset);
                tA = both_decays(tA, aw, can_reset);
            }
        }
        // what the next tile of the chain waits for goes out before the copies of this block's next start
        // (65536 x 768 float32 217 instead of 231 us); with two channels a lane the orders are within 2% of
        // each other (16 x 4096 x 4096 bfloat16 forward 495 so and 505, backward 947 and 937 us)
        constexpr bool kEarly = V == 1;
        float2 h;
        auto hand_on = [&] {
            h = first ? make_float2(carry[0], V == 2 ? carry[V - 1] : 0.0f) : sc[turn][lane];
            if (warp != 0) return;
            const float2 end = join(tA, h, tH, can_reset);
            sc[turn ^ 1][lane] = end;
            if (last && more) publish<V>(mine, both(0.0f), end, kFinal);
            if (!more && here && p.h_last) put<V>(p.h_last + (int64_t)q.b * p.D + q.col, end);
        };
        // an item of one tile can say what it makes of a state before it knows its own
        const bool partial = !all_known && last && more && warp == 0;
        if (kEarly && all_known) hand_on();
        if (kEarly && partial) publish<V>(mine, tA, tH, kPartial);
        begin(next, turn ^ 1);
        d = decay_at<V>(p, next, g);
        if (!all_known) {
            if (!kEarly && partial) publish<V>(mine, tA, tH, kPartial);
            // every warp has read its words of this tile: their place serves the look-back
            static_assert(kWarps * kWords * 4 >= kWindow * S::kCols * 8, "room for the look-back");
            float2* win = reinterpret_cast<float2*>(words + turn * kWarps * kWords);
            look_back<V, kWarps, kReset>(mine - stride, stride, divide(q.item, g.by_chains), win, carry, header);
        }
        if (!kEarly || !all_known) hand_on();
#pragma unroll
        for (int e = 0; e < kWarps - 1; ++e)
            if (e < warp) h = join(sa[turn][e][lane], h, sh[turn][e][lane], can_reset);
        if (here && t0 < (int)p.T) {
            if (p.states && t0 % kChunk == 0) put<V>(p.states + ((int64_t)q.b * saved + t0 / kChunk) * p.D + q.col, h);
            if (resets) run_states<V, L, false, true>(a, u, h, resets);
            else run_states<V, L, false, false>(a, u, h, 0u);
            IO* y = static_cast<IO*>(p.y) + ((int64_t)q.b * p.T + t0) * p.D + q.col;
            const int rows = min(L, (int)p.T - t0);
            const int64_t row_bytes = p.D * (int64_t)sizeof(IO);
            auto store = [&](auto whole) {
#pragma unroll
                for (int j = 0; j < L; ++j, advance(y, row_bytes)) {
                    if (whole.value || j < rows) {
                        if constexpr (V == 2) store_two<IO>(y, u[j]);
                        else *y = from_f32<IO>(j & 1 ? u[j / 2].y : u[j / 2].x);
                    }
                }
            };
            if (rows == L) store(std::true_type{});
            else store(std::false_type{});
        }
        settle(next, turn ^ 1);
        q = next;
    }
    cp_async_wait<0>();
}

// A tile is one saved chunk: h is rebuilt from its saved state, and the flow a_t*g_t of the
// gradient back in time is the scan, over the chunks from the last to the first. Rebuilding h
// costs one multiply-add an element; reading y instead would add 2 to the 14 bytes an element
// of a 16-bit pass and round every state to 16 bits. ddecay's sums leave as one row a tile.
template <typename IO, int V, int L, Copy kCopy, bool kReset>
__global__ void __launch_bounds__(kThreads, kBlocks) k_scan_bwd(ScanArgs p, float* part, Grid g)
{
    using S = Tile<V, L>;
    static_assert(S::kSteps == kChunk, "a tile is a saved chunk");
    constexpr bool kExact = sizeof(IO) == 4;
    constexpr int kWords = 4 * L * 32;
    extern __shared__ __align__(16) unsigned words[];     // [2][kWarps][4][L][32]
    __shared__ float2 sa[2][kWarps][32], sh[2][kWarps][32], sf[2][kWarps][32], ss[2][kWarps][32], sc[2][32];
    __shared__ float2 win[kWindow * S::kCols];
    __shared__ int taken[2];
    const int lane = threadIdx.x & 31, warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
    unsigned* header = static_cast<unsigned*>(p.ws);
    const bool chained = g.nchunks > g.run;
    constexpr bool can_reset = kReset;
    Slot* slots = reinterpret_cast<Slot*>(static_cast<char*>(p.ws) + kScanHeader);
    const int64_t stride = (int64_t)g.nchains * S::kCols;
    unsigned none_r = pack_one<IO>(-INFINITY);
    if (V == 2) none_r |= none_r << 16;

    unsigned pending[kCopy == kPlain ? 4 : 1][L];
    auto begin = [&](const Place& q, int buf) {
        if (q.item < g.nitems) {
            const Rows x = rows_of<IO, V, L, kCopy>(q.b, (g.nchunks - 1 - q.chunk) * kChunk + warp * L, q.col, p);
            if constexpr (kCopy == kPlain) {
                load_rows<IO, L>(pending[0], p.r, x, none_r);
                load_rows<IO, L>(pending[1], p.i, x, 0u);
                load_rows<IO, L>(pending[2], p.x, x, 0u);
                load_rows<IO, L>(pending[3], p.dy, x, 0u);
            } else {
                unsigned* w = words + (buf * kWarps + warp) * kWords;
                const int64_t at = offset_in(p.x, x);
                stage<IO, V, L, kCopy>(w, p.r, x, kCopy == kWide ? at : offset_in(p.r, x), none_r);
                stage<IO, V, L, kCopy>(w + L * 32, p.i, x, kCopy == kWide ? at : offset_in(p.i, x), 0u);
                stage<IO, V, L, kCopy>(w + 2 * L * 32, p.x, x, at, 0u);
                stage<IO, V, L, kCopy>(w + 3 * L * 32, p.dy, x, offset_in(p.dy, x), 0u);
            }
        }
        cp_async_commit();
    };
    auto settle = [&](const Place& q, int buf) {
        if constexpr (kCopy == kPlain) {
            unsigned* w = words + (buf * kWarps + warp) * kWords;
            if (q.item < g.nitems) {
#pragma unroll
                for (int k = 0; k < 4; ++k) put_rows(w + k * L * 32, pending[k]);
            }
        }
    };
    // a tile's part of ddecay, joined once a barrier has passed
    int64_t sum_at = -1;
    auto sum_part = [&](int turn) {
        if (warp != kWarps - 1 || sum_at < 0) return;
        float2 s = ss[turn][0][lane];
#pragma unroll
        for (int e = 1; e < kWarps; ++e) s = add2(s, ss[turn][e][lane]);
        put<V>(part + sum_at, s);
    };

    int plain = (int)blockIdx.x, turn = 0;
    if (threadIdx.x == 0) {
        if (!chained && blockIdx.x == 0) header[0] = 0u;
        taken[0] = next_item(header + 1, g.nitems, chained, plain);
    }
    __syncthreads();
    const Held held_ = held();
    Place q = place_of<V>(taken[0], g);
    begin(q, 0);
    settle(q, 0);
    float2 d = decay_at<V>(p, q, g), h = state_at<V>(p, q, g);
    for (; q.item < g.nitems; turn ^= 1) {
        const bool last = ends(q, g), first = q.chunk == divide(q.item, g.by_chains) * g.run;
        if (last && threadIdx.x == 0) taken[turn ^ 1] = next_item(header + 1, g.nitems, chained, plain);
        Slot* mine = slots + (int64_t)q.item * S::kCols;
        const bool here = q.col < (int)p.D;
        const int c = g.nchunks - 1 - q.chunk, t0 = c * kChunk + warp * L;
        const int64_t at = ((int64_t)q.b * g.nchunks + c) * p.D + q.col;
        const unsigned resets = kReset ? reset_bits<L>(p.reset, q.b, (int)p.T, t0) : 0u;
        float carry[V];
        bool known = true;
        if (first)
            known = arriving<V>(mine - stride, q.chunk == 0, p.dh_last ? p.dh_last + (int64_t)q.b * p.D + q.col : nullptr, here, carry);
        const Rate k = rate(d);
        cp_async_wait<0>();
        __syncwarp();

        const unsigned* w = words + (turn * kWarps + warp) * kWords + lane;
        const unsigned *wx = w + 2 * L * 32, *wd = w + 3 * L * 32;
        float2 a[S::kPairs], u[S::kPairs], s32[S::kPairs], si[S::kPairs], b[S::kPairs];
#pragma unroll
        for (int m = 0; m < S::kPairs; ++m) {
            const Gates e = gates<kExact>(pair_at<IO, V>(w, m), pair_at<IO, V>(w + L * 32, m), k, held_);
            a[m] = e.a, s32[m] = e.s32, si[m] = e.si, b[m] = e.b;
            u[m] = mul2(mul2(e.b, e.si), pair_at<IO, V>(wx, m));
            // one pair after the other: more of them under way at a time spill (16 x 4096 x 4096 bfloat16
            // with resets 1,016 instead of 1,195 us, without 937 instead of 943)
            if (V == 2) asm volatile("" : "+f"(a[m].x), "+f"(a[m].y), "+f"(u[m].x), "+f"(u[m].y));
        }
        sh[turn][warp][lane] = resets ? end_state<V, L, true>(a, u, both(0.0f), resets)
                                      : end_state<V, L, false>(a, u, both(0.0f), 0u);
        sf[turn][warp][lane] = resets ? end_flow<IO, V, L, true>(a, wd, resets) : end_flow<IO, V, L, false>(a, wd, 0u);
        sa[turn][warp][lane] = product<V, L>(a, resets);
        const bool all_known = __syncthreads_and(known);
        Place next = q;
        if (last) next = place_of<V>(taken[turn ^ 1], g);
        else next.chunk += 1;

        const bool more = q.chunk + 1 < g.nchunks;
        float2 tA, tF;
        if (warp == 0 || !all_known) {
            tA = sa[turn][kWarps - 1][lane];
            tF = sf[turn][kWarps - 1][lane];
#pragma unroll
            for (int e = kWarps - 2; e >= 0; --e) {
                const float2 aw = sa[turn][e][lane];
                tF = join(aw, tF, sf[turn][e][lane], can_reset);
                tA = both_decays(tA, aw, can_reset);
            }
        }
        constexpr bool kEarly = V == 1;      // as in the forward pass
        float2 f;
        auto hand_on = [&] {
            f = first ? make_float2(carry[0], V == 2 ? carry[V - 1] : 0.0f) : sc[turn][lane];
            if (warp != 0) return;
            const float2 end = join(tA, f, tF, can_reset);
            sc[turn ^ 1][lane] = end;
            if (last && more) publish<V>(mine, both(0.0f), end, kFinal);
            if (!more && here && p.dh0) put<V>(p.dh0 + (int64_t)q.b * p.D + q.col, end);
        };
        const bool partial = !all_known && last && more && warp == 0;
        if (kEarly && all_known) hand_on();
        if (kEarly && partial) publish<V>(mine, tA, tF, kPartial);
        begin(next, turn ^ 1);
        const float2 next_d = decay_at<V>(p, next, g), next_h = state_at<V>(p, next, g);
        sum_part(turn ^ 1);
        if (!all_known) {
            if (!kEarly && partial) publish<V>(mine, tA, tF, kPartial);
            look_back<V, kWarps, kReset>(mine - stride, stride, divide(q.item, g.by_chains), win, carry, header);
        }
        if (!kEarly || !all_known) hand_on();
#pragma unroll
        for (int e = 0; e < kWarps - 1; ++e)
            if (e < warp) h = join(sa[turn][e][lane], h, sh[turn][e][lane], can_reset);
#pragma unroll
        for (int e = kWarps - 1; e > 0; --e)
            if (e > warp) f = join(sa[turn][e][lane], f, sf[turn][e][lane], can_reset);
        if (resets) run_states<V, L, true, true>(a, u, h, resets);
        else run_states<V, L, true, false>(a, u, h, 0u);

        // from the last step to the first: g = dy + flow, and every gradient from it
        float2 sum = both(0.0f);
        // dr's factor 2^-32 goes with 1 - s(r): decays below 2^-94 would lose bits to it
        const float2 minus_d = make_float2(-d.x, -d.y), one = hold(1.0f), minus_one = hold(-1.0f),
                     minus_m32 = hold(-kTwoM32), m32 = hold(kTwoM32), minus_m64 = hold(-kTwoM32 * kTwoM32);
        const int64_t o = ((int64_t)q.b * p.T + t0) * p.D + q.col;
        const int rows = here ? max(0, min(L, (int)p.T - t0)) : 0;
        const int64_t back = -p.D * (int64_t)sizeof(IO);
        auto gradients = [&](auto with_resets, auto whole) {
            IO *dx = static_cast<IO*>(p.dx) + o + (L - 1) * p.D, *dr = static_cast<IO*>(p.dr) + o + (L - 1) * p.D,
               *di = static_cast<IO*>(p.di) + o + (L - 1) * p.D;
#pragma unroll
            for (int m = S::kPairs - 1; m >= 0; --m) {
                const float2 dy = pair_at<IO, V>(wd, m), x = pair_at<IO, V>(wx, m);
                float2 gt, keep = a[m];
                if constexpr (V == 2) {
                    gt = add2(dy, f);
                    f = mul2(keep, gt);
                    if (with_resets.value && (resets >> m & 1u)) keep = u[m] = f = both(0.0f);
                } else {
                    gt.y = dy.y + f.x;
                    f.x = keep.y * gt.y;
                    if (with_resets.value && (resets >> (2 * m + 1) & 1u)) keep.y = u[m].y = f.x = 0.0f;
                    gt.x = dy.x + f.x;
                    f.x = keep.x * gt.x;
                    if (with_resets.value && (resets >> (2 * m) & 1u)) keep.x = u[m].x = f.x = 0.0f;
                }
                // the slope a^2/b of b by log a is taken as 0 where b is
                const float2 xs = mul2(x, si[m]), ax = mul2(mul2(a[m], a[m]), xs);
                const float2 rb = make_float2(b[m].x > 0.0f ? fast_rcp(b[m].x) : 0.0f, b[m].y > 0.0f ? fast_rcp(b[m].y) : 0.0f);
                const float2 inner = fma2(mul2(ax, rb), minus_one, mul2(keep, u[m]));
                const float2 dlog = mul2(mul2(gt, inner), s32[m]);        // times 2^32 s(r)
                const float2 gb = mul2(gt, b[m]);
                const float2 one_i = fma2(si[m], minus_one, one), one_r = fma2(s32[m], minus_m64, m32);
                const float2 ox = mul2(gb, si[m]), oi = mul2(mul2(gb, xs), one_i), orr = mul2(mul2(dlog, minus_d), one_r);
                sum = fma2(dlog, minus_m32, sum);
                if constexpr (V == 2) {
                    if (whole.value || m < rows) {
                        store_two<IO>(dx, ox);
                        store_two<IO>(dr, orr);
                        store_two<IO>(di, oi);
                    }
                    advance(dx, back), advance(dr, back), advance(di, back);
                } else {
                    if (whole.value || 2 * m + 1 < rows) {
                        *dx = from_f32<IO>(ox.y);
                        *dr = from_f32<IO>(orr.y);
                        *di = from_f32<IO>(oi.y);
                    }
                    advance(dx, back), advance(dr, back), advance(di, back);
                    if (whole.value || 2 * m < rows) {
                        *dx = from_f32<IO>(ox.x);
                        *dr = from_f32<IO>(orr.x);
                        *di = from_f32<IO>(oi.x);
                    }
                    advance(dx, back), advance(dr, back), advance(di, back);
                }
            }
        };
        if ((kReset && resets) || rows < L) gradients(std::integral_constant<bool, kReset>{}, std::false_type{});
        else gradients(std::false_type{}, std::true_type{});
        if (V == 1) sum.x += sum.y;
        ss[turn][warp][lane] = sum;
        sum_at = here ? at : -1;
        settle(next, turn ^ 1);
        q = next;
        d = next_d;
        h = next_h;
    }
    cp_async_wait<0>();
    __syncthreads();
    sum_part(turn ^ 1);
}

// Column sums of part [rows][D], kSumRows rows to a block: out [ceil(rows/kSumRows)][D], in a
// fixed order (32 columns a block, 8 groups of rows, joined in shared memory).
constexpr int kSumRows = 256;

__global__ void __launch_bounds__(256) k_column_sums(const float* part, int64_t rows, int64_t D, float* out)
{
    __shared__ float s[8][32];
    const int lane = threadIdx.x & 31, group = threadIdx.x >> 5;
    const int64_t d = (int64_t)blockIdx.x * 32 + lane, r0 = (int64_t)blockIdx.y * kSumRows;
    float v = 0.0f;
    if (d < D) {
#pragma unroll 8
        for (int64_t k = r0 + group; k < r0 + kSumRows; k += 8)
            if (k < rows) v += part[k * D + d];
    }
    s[group][lane] = v;
    __syncthreads();
    if (group == 0 && d < D) {
#pragma unroll
        for (int g = 1; g < 8; ++g) v += s[g][lane];
        out[(int64_t)blockIdx.y * D + d] = v;
    }
}

// One token for B sequences; two channels a thread where V is 2 (an even number of channels). One
// sequence of 2,048 channels takes 2.0 us in a graph, an empty launch 1.8; 512 of 4,096, 33.6 MB,
// 8.0 us, from the L2 in part.
template <typename IO, int V>
__global__ void __launch_bounds__(128) k_scan_step(ScanStepArgs p, int64_t ncols)
{
    const int64_t id = (int64_t)blockIdx.x * 128 + threadIdx.x;
    if (id >= p.B * ncols) return;
    const int64_t b = id / ncols, d = (id - b * ncols) * V, o = b * p.D + d;
    auto load = [&](const void* t, int64_t stride) {
        const IO* q = static_cast<const IO*>(t) + b * stride + d;
        return make_float2(to_f32(q[0]), to_f32(q[V - 1]));
    };
    const Gates g = gates<sizeof(IO) == 4>(load(p.r, p.rs), load(p.i, p.is), rate(make_float2(p.decay[d], p.decay[d + V - 1])), held());
    const bool reset = p.reset && p.reset[b];
    const float2 h = reset ? both(0.0f) : make_float2(p.h[o], p.h[o + V - 1]);
    const float2 n = fma2(g.a, h, mul2(mul2(g.b, g.si), load(p.x, p.xs)));
    IO* y = static_cast<IO*>(p.y) + o;
    p.h[o] = n.x;
    y[0] = from_f32<IO>(n.x);
    if (V == 2) {
        p.h[o + 1] = n.y;
        y[1] = from_f32<IO>(n.y);
    }
}

__global__ void __launch_bounds__(256) k_clear(uint4* p, int64_t n)
{
    for (int64_t k = (int64_t)blockIdx.x * 256 + threadIdx.x; k < n; k += (int64_t)gridDim.x * 256)
        p[k] = make_uint4(0u, 0u, 0u, 0u);
}

// A look-back's wait for a slot that nothing publishes, for tests.
__global__ void k_scan_wait(unsigned* header, uint64_t limit_ns)
{
    const Slot* slot = reinterpret_cast<const Slot*>(reinterpret_cast<char*>(header) + kScanHeader / 2);
    await_slot(slot, kPartial, header, limit_ns);
}

// Bytes of slots for `steps`-step tiles, one tile an item: channels rounded up to the widest tile.
size_t slot_bytes(int64_t B, int64_t T, int64_t D, int steps)
{
    const int64_t nchunks = ceil_div(T, steps);
    return nchunks > 1 ? (size_t)(B * ceil_div(D, 64) * 64 * nchunks) * sizeof(Slot) : 0;
}

// Whether every row of every tensor starts on `bytes` bytes and holds a whole number of them.
bool rows_on(const ScanArgs& a, const void* const* outs, int nouts, int elem, int bytes)
{
    const int per = bytes / elem;
    if (a.D % per) return false;
    const ob_view* in[4] = {&a.x, &a.r, &a.i, &a.dy};
    for (const ob_view* v : in) {
        if (!v->ptr) continue;
        if (reinterpret_cast<uintptr_t>(v->ptr) % bytes) return false;
        if ((a.B > 1 && v->batch % per) || (a.T > 1 && v->time % per)) return false;
    }
    for (int k = 0; k < nouts; ++k)
        if (reinterpret_cast<uintptr_t>(outs[k]) % bytes) return false;
    return true;
}

// Whether x, r and i have the same strides (along axes that have any length).
bool alike(const ScanArgs& a)
{
    return (a.B == 1 || (a.x.batch == a.r.batch && a.x.batch == a.i.batch)) &&
           (a.T == 1 || (a.x.time == a.r.time && a.x.time == a.i.time));
}

// One wave of persistent blocks. Where there are at least as many chains as blocks, a block takes up to
// 8 consecutive tiles of a chain (at least 6 items a block are left, for balance): 16 x 4096 x 4096
// bfloat16 forward, backward 505, 937 us instead of 540, 1,027 us with one tile each; 64 x 512 x 4096
// 270, 510 instead of 276, 539 us. With nearly as many, each block takes a whole chain and none waits:
// B x 2048 x D bfloat16 with 256 chains for 304 blocks 83, 163 us instead of 92, 178, with 288 (4,096
// steps) 159, 307 instead of 188, 351; with 240 83, 163 instead of 89, 171, with 224 82, 162 instead of 86, 162,
// with 208 82, 163 instead of 82, 156: below about 0.72 of the blocks' number the idle ones outweigh it, and 0.8
// is a little above that. With fewer, an item would keep its successor's block waiting, so each is one
// tile.
template <int V, int L, auto kKernel, typename... A>
cudaError_t launch_tiles(const ScanArgs& a, int tensors, cudaStream_t s, A... more)
{
    using S = Tile<V, L>;
    const int64_t ncols = ceil_div(a.D, S::kCols), nchains = a.B * ncols, nchunks = ceil_div(a.T, S::kSteps);
    DeviceFacts dev;
    cudaError_t e = current_device(&dev);
    if (e != cudaSuccess) return e;
    const int64_t blocks = (int64_t)dev.sms * kBlocks;
    int64_t run = 1;
    if (nchains >= blocks) run = std::min<int64_t>(8, std::max<int64_t>(1, nchains * nchunks / (blocks * 6)));
    else if (nchains * 5 >= blocks * 4) run = nchunks;
    Grid g{};
    g.nchains = (int)nchains, g.ncols = (int)ncols, g.nchunks = (int)nchunks, g.run = (int)run;
    g.nitems = (int)(nchains * ceil_div(nchunks, run));
    g.by_chains = make_fastdiv((uint32_t)nchains);
    g.by_cols = make_fastdiv((uint32_t)ncols);
    if (nchunks > run) {
        const int64_t n = (int64_t)kScanHeader / 16 + (int64_t)g.nitems * S::kCols;
        k_clear<<<(unsigned)std::min<int64_t>(ceil_div(n, 256), dev.sms * 8), 256, 0, s>>>(static_cast<uint4*>(a.ws), n);
        e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    const size_t smem = (size_t)2 * kWarps * tensors * L * 32 * 4;
    return with_opt_in<kKernel>(dev.device, smem, [&] {
        kKernel<<<(unsigned)std::min<int64_t>(g.nitems, blocks), kThreads, smem, s>>>(a, more..., g);
        return cudaGetLastError();
    });
}

template <typename IO, int V, Copy kCopy>
cudaError_t run_fwd(const ScanArgs& a, cudaStream_t s)
{
    return a.reset ? launch_tiles<V, 16, k_scan_fwd<IO, V, 16, kCopy, true>>(a, 3, s)
                   : launch_tiles<V, 16, k_scan_fwd<IO, V, 16, kCopy, false>>(a, 3, s);
}

template <typename IO, int V, Copy kCopy>
cudaError_t run_bwd(const ScanArgs& a, cudaStream_t s)
{
    constexpr int L = kChunk / kWarps;
    const int64_t nchunks = ceil_div(a.T, kChunk);
    float* part = reinterpret_cast<float*>(static_cast<char*>(a.ws) + kScanHeader + slot_bytes(a.B, a.T, a.D, kChunk));
    cudaError_t e = a.reset ? launch_tiles<V, L, k_scan_bwd<IO, V, L, kCopy, true>>(a, 4, s, part)
                            : launch_tiles<V, L, k_scan_bwd<IO, V, L, kCopy, false>>(a, 4, s, part);
    int64_t rows = a.B * nchunks;
    while (e == cudaSuccess) {
        const int64_t blocks = ceil_div(rows, kSumRows);
        float* out = blocks == 1 ? a.ddecay : part + rows * a.D;
        // at most 65535 blocks along y: 16.7 M rows in one go
        for (int64_t y = 0; y < blocks && e == cudaSuccess; y += 65535) {
            const int64_t n = std::min<int64_t>(65535, blocks - y);
            k_column_sums<<<dim3((unsigned)ceil_div(a.D, 32), (unsigned)n), 256, 0, s>>>(
                part + y * kSumRows * a.D, rows - y * kSumRows, a.D, out + y * a.D);
            e = cudaGetLastError();
        }
        if (blocks == 1) break;
        part += rows * a.D;
        rows = blocks;
    }
    return e;
}

}  // namespace

size_t scan_workspace_bytes(int64_t B, int64_t T, int64_t D, int, int backward)
{
    if (B == 0 || T == 0 || D == 0) return kScanHeader;
    size_t bytes = kScanHeader + slot_bytes(B, T, D, kChunk);
    if (backward) {
        int64_t rows = B * ceil_div(T, kChunk), all = rows;
        while (rows > 1) {
            rows = ceil_div(rows, kSumRows);
            all += rows;
        }
        bytes += (size_t)all * D * sizeof(float);
    }
    return bytes;
}

cudaError_t launch_scan_fwd(const ScanArgs& a, cudaStream_t s)
{
    return by_dtype(a.dtype, [&](auto io) {
        using IO = decltype(io);
        const void* outs[1] = {a.y};
        const bool wide = rows_on(a, outs, 1, sizeof(IO), 16) && alike(a);
        if constexpr (sizeof(IO) == 4) {
            return wide ? run_fwd<IO, 1, kWide>(a, s) : run_fwd<IO, 1, kWord>(a, s);
        } else {
            return wide ? run_fwd<IO, 2, kWide>(a, s)
                   : rows_on(a, outs, 1, sizeof(IO), 4) ? run_fwd<IO, 2, kWord>(a, s)
                                                        : run_fwd<IO, 1, kPlain>(a, s);
        }
    });
}

cudaError_t launch_scan_bwd(const ScanArgs& a, cudaStream_t s)
{
    return by_dtype(a.dtype, [&](auto io) {
        using IO = decltype(io);
        const void* outs[3] = {a.dx, a.dr, a.di};
        const bool wide = rows_on(a, outs, 3, sizeof(IO), 16) && alike(a);
        if constexpr (sizeof(IO) == 4) {
            return wide ? run_bwd<IO, 1, kWide>(a, s) : run_bwd<IO, 1, kWord>(a, s);
        } else {
            return wide ? run_bwd<IO, 2, kWide>(a, s)
                   : rows_on(a, outs, 3, sizeof(IO), 4) ? run_bwd<IO, 2, kWord>(a, s)
                                                        : run_bwd<IO, 1, kPlain>(a, s);
        }
    });
}

cudaError_t launch_scan_step(const ScanStepArgs& a, cudaStream_t s)
{
    return by_dtype(a.dtype, [&](auto io) {
        using IO = decltype(io);
        if (a.D % 2 == 0)
            k_scan_step<IO, 2><<<(unsigned)ceil_div(a.B * a.D / 2, 128), 128, 0, s>>>(a, a.D / 2);
        else
            k_scan_step<IO, 1><<<(unsigned)ceil_div(a.B * a.D, 128), 128, 0, s>>>(a, a.D);
        return cudaGetLastError();
    });
}

cudaError_t launch_scan_wait(void* ws, uint64_t limit_ns, cudaStream_t s)
{
    cudaError_t e = cudaMemsetAsync(ws, 0, kScanHeader, s);
    if (e != cudaSuccess) return e;
    k_scan_wait<<<1, 32, 0, s>>>(static_cast<unsigned*>(ws), limit_ns);
    return cudaGetLastError();
}

cudaError_t scan_status(unsigned* status, cudaStream_t s) { return take_status(scan_wait_status, status, s); }

}  // namespace ob
