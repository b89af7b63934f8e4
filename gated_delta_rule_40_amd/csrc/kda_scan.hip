// kda_scan.hip -- the gated linear recurrence h_t = exp(g_t) h_{t-1} + x_t per
// channel over packed sequences, its decode step and its gradients.
//
// With a_t = exp(g_t), a run of tokens maps the state that enters it to the
// state that leaves it by h -> A h + B, A the product of its a_t and B its end
// state from zero, and two runs in a row map by (A2 A1, A2 B1 + B2).  The packed
// tokens are cut into tiles of 128, whatever the sequences; a sequence's start
// drops what entered (A = RESET) and takes the initial state into B.  One
// workgroup of eight waves reads a tile of 128 tokens x 64 V channels once, 16
// tokens a wave, keeps it in registers, publishes its (A, B), obtains the state
// that enters it from the tiles before it, and writes its outputs: every input
// is read once and every output written once, which is all the traffic there
// has to be (8 bytes an element with bf16 x), and HBM's rate is the bound.
//
// The state that enters a tile is found in one pass by looking back (the method
// of D. Merrill and M. Garland, 2016, in another form): it is joined from the runs
// of the tiles before it in its block of 16, 32 or 64 tiles (for V = 4, 2, 1), all
// read side by side, and the state that enters the block, which is passed from
// block to block.  Which runs are joined, and in which order, depends on the tile
// alone, not on what is ready first, so that results are the same bits on every
// call.  A published run is one 64-bit word a channel, written and polled with
// relaxed device-scope atomics: the word is its own flag (all ones: not there yet), so no fence is
// needed between data and flag.  Tiles of a channel block are handed out in
// order by a counter, so a tile waits only for workgroups that are already
// running, and these wait for earlier ones in turn: every wait ends.
//
// The gradients run the same scheme from the end to the start,
//     dh_t = dout_t + e,  e <- a_t dh_t,
// with the state entering each tile taken from the forward pass's checkpoints.
//
// Measured on one MI355X (a large copy reaches 4.9-5.4 TB/s there): 2^20 tokens
// x 1,024 channels in bf16 1.57 ms (5.5 TB/s of the 8 bytes an element; counters
// show 3 % more read and 10 % more written: 71 MB of published words, and 138 MB
// that are most likely the 6 registers a lane which V = 4 keeps in scratch, as
// the gradients at V = 2 do with 7 or 8), forward and backward of 65,536 x 4,096
// 1.07 ms (5.5 TB/s of 22 bytes an element).  Short
// batches are bound by the chain of waits: 4,096 x 1,024 takes 13 us in the
// kernel, of which the counter's answer is 2, the reads 2, the gates and runs 2,
// passing the state on 3 and the writes 2.
#include "kda_device.hpp"
#include "kda_layer.hpp"
#include "kda_seq.hpp"

namespace kda {

constexpr int TILE = 128;             // tokens of a tile, and between checkpoints
constexpr int WAVES = 8;              // waves of a workgroup
constexpr int L = TILE / WAVES;       // tokens of a wave
constexpr int NTH = WAVES * 64;
constexpr int GATHER = 8;             // published runs a thread joins
constexpr float RESET = -1.f;         // an A that drops what enters (products of exp() are never negative)
constexpr uint64_t NOT_YET = ~(uint64_t)0;
constexpr int TICKET_STRIDE = 32;     // columns' counters lie in cache lines of their own

// ---------------------------------------------------------------- published runs
struct Chain {
    uint32_t *ticket;                 // [column of channels][TICKET_STRIDE], from ~0
    uint64_t *tile, *block;           // [index][D]: tiles' runs, states that enter blocks
    int32_t ntiles;
    int64_t D;
    int32_t width;                    // channels of a column
};

struct Run {
    float A, B;
};

// first, then second
__device__ __forceinline__ Run join(const Run &first, const Run &second)
{
    if (second.A == RESET) return second;
    return {first.A == RESET ? RESET : first.A * second.A, second.A * first.B + second.B};
}
__device__ __forceinline__ float apply(const Run &r, float h) { return r.A == RESET ? r.B : r.A * h + r.B; }

__device__ __forceinline__ uint64_t pack(const Run &r)
{
    const uint64_t w = (uint64_t)__float_as_uint(r.A) | ((uint64_t)__float_as_uint(r.B) << 32);
    return w == NOT_YET ? 0x7fc000007fc00000ull : w;   // two NaNs stay two NaNs
}
__device__ __forceinline__ Run unpack(uint64_t w)
{
    return {__uint_as_float((uint32_t)w), __uint_as_float((uint32_t)(w >> 32))};
}
__device__ __forceinline__ uint64_t peek(const uint64_t *p)
{
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void publish(uint64_t *p, const Run &r)
{
    __hip_atomic_store(p, pack(r), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// the m <= GATHER runs p[0], p[D], ... joined in order; all are asked for before any is waited for
__device__ __forceinline__ Run gather(const uint64_t *p, int64_t D, int m)
{
    uint64_t w[GATHER];
#pragma unroll
    for (int i = 0; i < GATHER; ++i) w[i] = i < m ? peek(p + i * D) : 0;
    Run r = {1.f, 0.f};
#pragma unroll
    for (int i = 0; i < GATHER; ++i) {
        if (i < m) {
            while (w[i] == NOT_YET) w[i] = peek(p + i * D);
            r = i == 0 ? unpack(w[i]) : join(r, unpack(w[i]));
        }
    }
    return r;
}

// Roles of a workgroup's threads in passing a state on: CB threads each, one a
// channel.  Each role joins GATHER of the tiles of the block before this one.
template <int CB> struct Roles {
    static constexpr int N = NTH / CB;
    static constexpr int BLOCK = N * GATHER;   // tiles of a block
};

// The value that enters tile k (counted in the direction of the walk) for
// every channel of the workgroup, in `enter`; publishes the tile's own run.
// `runs` holds the waves' runs in the order of the walk.  `fresh`: nothing
// enters (the tile begins at a boundary, or is the first); `resets`: it has a
// boundary, which holds for every fresh tile but the first, so that every
// block's last tile publishes on one of the two ways.  Begins after a barrier
// and ends with one.
template <int CB, int V>
__device__ __forceinline__ void pass_on(const Chain &ch, int k, int64_t c0, bool fresh, bool resets,
                                        const Run (*runs)[CB], Run (*parts)[CB], float *enter)
{
    constexpr int N = Roles<CB>::N, BLOCK = Roles<CB>::BLOCK;
    const int c = threadIdx.x % CB, role = threadIdx.x / CB;
    const bool in = c / V * V < ch.width && c0 + c / V * V < ch.D;
    const int place = k % BLOCK, block = k / BLOCK;   // the tile's place in its block
    const bool last = place == BLOCK - 1;
    const int64_t ci = min(c0 + c / V * V, ch.D - V) + c % V;
    Run own = {1.f, 0.f};
    uint64_t before = 0;
    if (role == 0 && in) {
        own = runs[0][c];
#pragma unroll
        for (int w = 1; w < WAVES; ++w) own = join(own, runs[w][c]);
        if (!last) publish(ch.tile + k * ch.D + ci, own);
        else if (resets) publish(ch.block + (block + 1) * ch.D + ci, {RESET, own.B});   // whatever enters
    }
    if (!fresh) {
        if (role == 0 && in && block > 0) before = peek(ch.block + block * ch.D + ci);
        const int m = min(place - role * GATHER, GATHER);
        if (role < N && in && m > 0)
            parts[role][c] = gather(ch.tile + (int64_t)(k - place + role * GATHER) * ch.D + ci, ch.D, m);
        __syncthreads();
        if (role == 0 && in) {
            // nothing enters the first block: its first run drops what would
            while (before == NOT_YET) before = peek(ch.block + block * ch.D + ci);
            float h = unpack(before).B;
#pragma unroll
            for (int r = 0; r < N; ++r)
                if (place > r * GATHER) h = apply(parts[r][c], h);
            enter[c] = h;
            if (!resets && last) publish(ch.block + (block + 1) * ch.D + ci, {RESET, apply(own, h)});
        }
    }
    __syncthreads();
}

// ---------------------------------------------------------------- tokens in registers
// V consecutive channels of a row.  In memory they need the alignment of one:
// rows of a channel count that V does not divide begin anywhere, and the last
// lane's channels overlap its neighbour's (both compute the same).
template <typename T, int V> struct Vec {
    typedef T raw __attribute__((ext_vector_type(V)));
    typedef raw mem __attribute__((aligned(sizeof(T))));
};
template <typename T> struct Vec<T, 1> {
    typedef T raw, mem;
};
template <typename T, int V> __device__ __forceinline__ typename Vec<T, V>::raw read_once(const T *p)
{
    return __builtin_nontemporal_load(reinterpret_cast<const typename Vec<T, V>::mem *>(p));
}
template <typename T, int V> __device__ __forceinline__ void write_once(T *p, const typename Vec<T, V>::raw &v)
{
    __builtin_nontemporal_store(v, reinterpret_cast<typename Vec<T, V>::mem *>(p));
}

template <typename R> __device__ __forceinline__ float elem(const R &r, int j) { return to_f(r[j]); }
template <> __device__ __forceinline__ float elem<float>(const float &r, int) { return r; }
template <> __device__ __forceinline__ float elem<bf16_t>(const bf16_t &r, int) { return to_f(r); }
template <typename R, typename T> __device__ __forceinline__ void put(R &r, int j, T v) { r[j] = v; }
template <> __device__ __forceinline__ void put<float, float>(float &r, int, float v) { r = v; }
template <> __device__ __forceinline__ void put<bf16_t, bf16_t>(bf16_t &r, int, bf16_t v) { r = v; }

// exp(g) within about one unit in the last place: the product with log2(e) is
// carried in two parts, since its rounding alone would be |g| units, and slow
// gates let errors of one sign add up over a thousand tokens.
__device__ __forceinline__ float gate(float g)
{
    const float L2E = 1.44269502f, L2E_LO = 1.92596299e-8f, LN2 = 0.693147182f;
    const float t = g * L2E;
    const float lo = __builtin_fmaf(g, L2E_LO, __builtin_fmaf(g, L2E, -t));
    const float e = __builtin_amdgcn_exp2f(t);
    // (positive and finite: elsewhere e is right by itself, and the parts need not
    // be numbers: t is infinite from g = -2.4e38 on, which a mask may hold)
    return __builtin_amdgcn_classf(e, 0x180) ? __builtin_fmaf(e, lo * LN2, e) : e;
}

// A wave's rows: scalar addresses, and a lane's place in a row of its own.
// Rows past the last token stand for the last one.
template <int V> struct Rows {
    int64_t first, D;
    int32_t last;
    int32_t lane;
    __device__ __forceinline__ Rows(const Seqs &sq, int32_t t0, int64_t D_, int64_t c0, int32_t lane_) : D(D_) {
        const int32_t t = min(t0, sq.T - 1);
        first = t * D + c0;
        last = sq.T - 1 - t;
        lane = lane_;
    }
    template <typename T> __device__ __forceinline__ typename Vec<T, V>::raw at(const T *p, int i) const {
        return read_once<T, V>(p + first + min(i, last) * D + lane);
    }
};

// The compiler keeps a value that it could unpack again: this makes it forget
// how `r` was unpacked, so that only the packed form stays in registers.
template <typename R> __device__ __forceinline__ void repack(R &r) { asm volatile("" : "+v"(r)); }

// Boundaries of sequences at a wave's tokens: bit i stands for token t0 + i,
// i = 0 .. L; lane i holds the number of the sequence that owns the token
// (outside [0, N): none).  `end` is the first token of no sequence.
struct Edges {
    uint32_t mask;
    int32_t end, own;
    __device__ __forceinline__ int32_t owner(int i, int32_t N) const {
        const int32_t n = __builtin_amdgcn_readlane(own, i);
        return n < N ? n : -1;
    }
};

__device__ __forceinline__ Edges edges(const SeqWindow &sq, int32_t t0, int32_t end)
{
    const int32_t i = threadIdx.x & 63;
    if (sq.below(t0 + L + 1) == 64) {   // more entries than are held: each lane looks for its own
        const int32_t own = i <= L ? sq.sq.first_at_or_after(t0 + i + 1) - 1 : -1;
        return {(uint32_t)__ballot(own >= 0 && sq.sq.at(own) == t0 + i), end, own};
    }
    int32_t n = sq.first_at_or_after(t0);
    Edges e = {0, end, n - 1};
    for (; n <= sq.sq.N; ++n) {
        const int32_t p = sq.at(n);
        if (p > t0 + L || p < t0) break;
        e.mask |= 1u << (p - t0);
        e.own += i >= p - t0;
    }
    return e;
}

// whether a sequence's boundary lies at a token of [t, t + len), and whether at t
__device__ __forceinline__ void boundary_in(const SeqWindow &sq, int32_t t, int len, bool *any, bool *at_first)
{
    const int32_t n = sq.first_at_or_after(t);
    const int64_t p = n <= sq.sq.N ? sq.at(n) : INT64_MAX;
    *any = p < (int64_t)t + len;
    *at_first = p == t;
}

// ---------------------------------------------------------------- forward
template <typename T, int V>
__global__ __launch_bounds__(NTH) __attribute__((amdgpu_waves_per_eu(4)))   // two workgroups per CU
void kda_scan_kernel(const T *x, const float *g, const float *init, Seqs sq, int64_t D, int32_t cols,
                     uint32_t work, T *out, float *fin, float *chk, Chain ch)
{
    constexpr int CB = 64 * V;
    typedef typename Vec<T, V>::raw XR;
    typedef typename Vec<float, V>::raw GR;
    __shared__ Run runs[WAVES][CB];
    __shared__ Run parts[Roles<CB>::N][CB];
    __shared__ float enter[CB];
    __shared__ uint32_t s_tile;

    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int col = blockIdx.x % cols;
    if (blockIdx.x >= work) return copy_empty(sq, blockIdx.x - work, D, init, fin);
    const int32_t tend = sq.at(sq.N);
    SeqWindow win(sq);
    int k = 0;
    if (ch.ntiles > 1) {
        if (threadIdx.x == 0) s_tile = atomicAdd(ch.ticket + col * TICKET_STRIDE, 1u) + 1u;
        __syncthreads();
        k = __builtin_amdgcn_readfirstlane((int)s_tile);
    }
    const int64_t c0 = (int64_t)col * ch.width, c = min(c0 + lane * V, D - V);
    const bool in = lane * V < ch.width && c0 + lane * V < D;
    XR xr[L];
    GR gr[L];
    const int32_t t0 = k * TILE + w * L;
    {
        const Rows<V> rows(sq, t0, D, c0, (int32_t)(c - c0));
#pragma unroll
        for (int i = 0; i < L; ++i) {
            xr[i] = rows.at(x, i);
            gr[i] = rows.at(g, i);
        }
    }
    win.locate(k * TILE);
    const Edges e = edges(win, t0, tend);
    const uint32_t starts = e.mask & ((1u << L) - 1);
    bool fresh, resets;
    boundary_in(win, k * TILE, TILE, &resets, &fresh);
    fresh = fresh || k == 0;
    // what a token leaves: its output, and the final state of a sequence that ends with it
    auto leave = [&](int i, const float (&h)[V]) {
        if (t0 + i >= e.end) return;
        if (out && in) {
            XR o;
            for (int j = 0; j < V; ++j) put(o, j, from_f<T>(h[j]));
            write_once<T, V>(out + (int64_t)(t0 + i) * D + c, o);
        }
        if (fin && (e.mask >> (i + 1) & 1)) {
            const int64_t n = e.owner(i, sq.N);
            if (n >= 0 && in)
                for (int j = 0; j < V; ++j) fin[n * D + c + j] = h[j];
        }
    };

    // the wave's run; after its first start the states are known, and leave at once
    float a[L][V];
    {
        float A[V], B[V];
#pragma unroll
        for (int j = 0; j < V; ++j) A[j] = 1.f, B[j] = 0.f;
        bool known = false;
#pragma unroll
        for (int i = 0; i < L; ++i) {
            if (starts >> i & 1) {
                known = true;
                const int64_t n = init ? e.owner(i, sq.N) : -1;
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    A[j] = RESET;
                    B[j] = (n >= 0 && in) ? init[n * D + c + j] : 0.f;
                }
            }
#pragma unroll
            for (int j = 0; j < V; ++j) {
                a[i][j] = gate(elem(gr[i], j));
                if (!known) A[j] *= a[i][j];
                B[j] = a[i][j] * B[j] + elem(xr[i], j);
            }
            if (known) leave(i, B);
        }
#pragma unroll
        for (int j = 0; j < V; ++j) runs[w][lane * V + j] = {A[j], B[j]};
#pragma unroll
        for (int i = 0; i < L; ++i) repack(xr[i]);
    }
    __syncthreads();
    if (ch.ntiles > 1) {
        pass_on<CB, V>(ch, k, c0, fresh, resets, runs, parts, enter);
        if (chk && w == 0 && in && !fresh)
            for (int j = 0; j < V; ++j) chk[k * D + c + j] = enter[lane * V + j];
    }
    // the tokens before the wave's first start
    if (starts & 1) return;
    float h[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        h[j] = fresh ? 0.f : enter[lane * V + j];
        for (int v = 0; v < w; ++v) h[j] = apply(runs[v][lane * V + j], h[j]);
    }
    if (e.mask == 0 && t0 + L <= e.end) {
        if (!out) return;
#pragma unroll
        for (int i = 0; i < L; ++i) {
            XR o;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                h[j] = a[i][j] * h[j] + elem(xr[i], j);
                put(o, j, from_f<T>(h[j]));
            }
            if (in) write_once<T, V>(out + (int64_t)(t0 + i) * D + c, o);
        }
    } else {
#pragma unroll
        for (int i = 0; i < L; ++i) {
            if (starts & ((2u << i) - 1)) break;
#pragma unroll
            for (int j = 0; j < V; ++j) h[j] = a[i][j] * h[j] + elem(xr[i], j);
            leave(i, h);
        }
    }
}

// ---------------------------------------------------------------- gradients
template <typename T, int V>
__global__ __launch_bounds__(NTH) __attribute__((amdgpu_waves_per_eu(4)))   // two workgroups per CU
void kda_scan_bwd_kernel(const T *x, const float *g, const float *init, Seqs sq, int64_t D, int32_t cols,
                         uint32_t work, const T *dout, const float *dfin, const float *chk, T *dx, float *dg,
                         float *dinit, Chain ch)
{
    constexpr int CB = 64 * V;
    typedef typename Vec<T, V>::raw XR;
    typedef typename Vec<float, V>::raw GR;
    __shared__ Run fwd[WAVES][CB];      // forward runs of the waves, first to last
    __shared__ Run back[WAVES][CB];     // backward runs of the waves, last to first
    __shared__ Run parts[Roles<CB>::N][CB];
    __shared__ float enter[CB];
    __shared__ uint32_t s_tile;

    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int col = blockIdx.x % cols;
    if (blockIdx.x >= work) return copy_empty(sq, blockIdx.x - work, D, dfin, dinit);
    const int32_t tend = sq.at(sq.N);
    SeqWindow win(sq);
    int kb = 0;                         // the tile's number from the end
    if (ch.ntiles > 1) {
        if (threadIdx.x == 0) s_tile = atomicAdd(ch.ticket + col * TICKET_STRIDE, 1u) + 1u;
        __syncthreads();
        kb = __builtin_amdgcn_readfirstlane((int)s_tile);
    }
    const int64_t c0 = (int64_t)col * ch.width, c = min(c0 + lane * V, D - V);
    const bool in = lane * V < ch.width && c0 + lane * V < D;
    XR xr[L], dr[L];
    GR gr[L];
    const int k = ch.ntiles - 1 - kb;
    const int32_t t0 = k * TILE + w * L;
    {
        const Rows<V> rows(sq, t0, D, c0, (int32_t)(c - c0));
#pragma unroll
        for (int i = 0; i < L; ++i) {
            gr[i] = rows.at(g, i);
            xr[i] = rows.at(x, i);
            dr[i] = rows.at(dout, i);
        }
    }
    float a[L][V];
    float h[V];
#pragma unroll
    for (int j = 0; j < V; ++j) h[j] = (in && k > 0) ? chk[k * D + c + j] : 0.f;
    win.locate(k * TILE);
    const Edges e = edges(win, t0, tend);
    const uint32_t starts = e.mask & ((1u << L) - 1);
    bool fresh, resets, unused;         // boundaries behind a token of the tile
    boundary_in(win, k * TILE + 1, TILE, &resets, &unused);
    boundary_in(win, (k + 1) * TILE, 1, &fresh, &unused);
    resets = resets || fresh;           // (so it is, unless cu_seqlens breaks its rules)
    fresh = fresh || kb == 0;
    {
        float A[V], B[V], E[V], Ae[V];
#pragma unroll
        for (int j = 0; j < V; ++j) A[j] = 1.f, B[j] = 0.f, E[j] = 0.f;
#pragma unroll
        for (int i = 0; i < L; ++i) {
            if (starts >> i & 1) {
                const int64_t n = init ? e.owner(i, sq.N) : -1;
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    A[j] = RESET;
                    B[j] = (n >= 0 && in) ? init[n * D + c + j] : 0.f;
                }
            }
#pragma unroll
            for (int j = 0; j < V; ++j) {
                a[i][j] = gate(elem(gr[i], j));
                if (!(starts & ((2u << i) - 1))) A[j] *= a[i][j];
                B[j] = a[i][j] * B[j] + elem(xr[i], j);
            }
        }
#pragma unroll
        for (int j = 0; j < V; ++j) {
            fwd[w][lane * V + j] = {A[j], B[j]};
            Ae[j] = 1.f;
        }
#pragma unroll
        for (int i = L - 1; i >= 0; --i) {
            if (e.mask >> (i + 1) & 1) {   // the gradient of the final state enters here
                const int64_t n = dfin ? e.owner(i, sq.N) : -1;
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    Ae[j] = RESET;
                    E[j] = (n >= 0 && in) ? dfin[n * D + c + j] : 0.f;
                }
            }
#pragma unroll
            for (int j = 0; j < V; ++j) {
                if (!(e.mask >> (i + 1))) Ae[j] *= a[i][j];
                E[j] = a[i][j] * (elem(dr[i], j) + E[j]);
            }
        }
#pragma unroll
        for (int j = 0; j < V; ++j) back[WAVES - 1 - w][lane * V + j] = {Ae[j], E[j]};
    }
    const uint32_t ends = e.mask >> 1;
    __syncthreads();
    if (ch.ntiles > 1) pass_on<CB, V>(ch, kb, c0, fresh, resets, back, parts, enter);

    // the states again, forward: p_t = a_t h_{t-1}
    float p[L][V], E[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        for (int v = 0; v < w; ++v) h[j] = apply(fwd[v][lane * V + j], h[j]);
        E[j] = fresh ? 0.f : enter[lane * V + j];
        for (int v = 0; v < WAVES - 1 - w; ++v) E[j] = apply(back[v][lane * V + j], E[j]);
    }
#pragma unroll
    for (int i = 0; i < L; ++i) {
        if (starts >> i & 1) {
            const int64_t n = init ? e.owner(i, sq.N) : -1;
#pragma unroll
            for (int j = 0; j < V; ++j) h[j] = (n >= 0 && in) ? init[n * D + c + j] : 0.f;
        }
#pragma unroll
        for (int j = 0; j < V; ++j) {
            p[i][j] = a[i][j] * h[j];
            h[j] = p[i][j] + elem(xr[i], j);
        }
    }
#pragma unroll
    for (int i = L - 1; i >= 0; --i) {
        if (ends >> i & 1) {
            const int64_t n = dfin ? e.owner(i, sq.N) : -1;
#pragma unroll
            for (int j = 0; j < V; ++j) E[j] = (n >= 0 && in) ? dfin[n * D + c + j] : 0.f;
        }
        XR ox;
        GR og;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float dh = elem(dr[i], j) + E[j];
            put(ox, j, from_f<T>(dh));
            put(og, j, dh * p[i][j]);
            E[j] = a[i][j] * dh;
        }
        if (in && t0 + i < e.end) {
            const int64_t at = (int64_t)(t0 + i) * D + c;
            write_once<T, V>(dx + at, ox);
            write_once<float, V>(dg + at, og);
        }
        if (dinit && t0 + i < e.end && (starts >> i & 1)) {
            const int64_t n = e.owner(i, sq.N);
            if (n >= 0 && in)
                for (int j = 0; j < V; ++j) dinit[n * D + c + j] = E[j];
        }
    }
}

// ---------------------------------------------------------------- decode
template <typename T>
__global__ void kda_scan_step_kernel(const T *x, const float *g, float *state, int64_t n, T *out)
{
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (int64_t)gridDim.x * blockDim.x) {
        const float h = gate(g[i]) * state[i] + to_f(x[i]);
        state[i] = h;
        out[i] = from_f<T>(h);
    }
}

// marks every published word and counter as not there yet (a kernel: a memset
// node of a captured graph is not relied on)
__global__ void kda_scan_fill_kernel(uint64_t *p, int64_t n)
{
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (int64_t)gridDim.x * blockDim.x)
        p[i] = NOT_YET;
}

// ---------------------------------------------------------------- host
inline int32_t tiles_of(int32_t T) { return T > 0 ? (int32_t)(((int64_t)T + TILE - 1) / TILE) : 1; }

// Words of a chain: counters of the columns (of 32 channels at least), then the tiles'
// runs and the states that enter blocks (of 16 tiles at least).  A single tile
// needs none.
struct ChainLayout {
    size_t tile, block, words;
};
inline ChainLayout chain_layout(int32_t T, int32_t D)
{
    const size_t nt = tiles_of(T), d = D;
    ChainLayout l = {};
    if (nt <= 1) return l;
    l.tile = (d + 31) / 32 * (TICKET_STRIDE / 2);
    l.block = l.tile + nt * d;
    l.words = l.block + (nt / Roles<256>::BLOCK + 1) * d;
    return l;
}
inline Chain chain_at(uint64_t *p, int32_t T, int32_t D)
{
    const ChainLayout l = chain_layout(T, D);
    return {reinterpret_cast<uint32_t *>(p), p + l.tile, p + l.block, tiles_of(T), (int64_t)D, 0};
}

inline hipError_t fill_chain(uint64_t *p, size_t words, hipStream_t s)
{
    if (words == 0) return hipSuccess;
    const size_t blocks = (words + 255) / 256;
    hipLaunchKernelGGL(kda_scan_fill_kernel, dim3((unsigned)(blocks < 4096 ? blocks : 4096)), dim3(256), 0, s, p,
                       (int64_t)words);
    return hipGetLastError();
}

template <typename T, int V>
hipError_t run_scan(const void *x, const float *g, const float *init, const Seqs &sq, int32_t D, void *out, float *fin,
                    float *chk, Chain ch, hipStream_t s)
{
    ch.width = kda_column_width(D, V);
    const int32_t cols = (D - 1) / ch.width + 1;
    const int64_t work = sq.T > 0 ? (int64_t)cols * ch.ntiles : 0, groups = work + empty_groups(sq.N, init, fin);
    if (groups > 0)
        hipLaunchKernelGGL((kda_scan_kernel<T, V>), dim3((unsigned)groups), dim3(NTH), 0, s, (const T *)x, g, init, sq,
                           (int64_t)D, cols, (uint32_t)work, (T *)out, fin, chk, ch);
    return hipGetLastError();
}

// One channel a lane: for rows of up to 64 (300,000 x 64 in bf16: 68 us, 135 with
// idle lanes of two), and where two would leave at most one workgroup for every
// CU, so that there are twice as many (graph replays, bf16: 4,096 x 1,024 13.6 us,
// 14.1 with two, with the gradients 30.8, 34.0; fp32: 14.5, 15.5 and 33.8, 40.8;
// beyond, fp32 10,007 x 1,000: 41.5 us, 37.2 with two).
inline bool one_channel(const Chain &ch)
{
    return ch.D <= 64 || ch.ntiles * ((ch.D + 127) / 128) <= 256;
}

template <typename T>
hipError_t scan(const void *x, const float *g, const float *init, const Seqs &sq, int32_t D, void *out, float *fin,
                float *chk, const Chain &ch, hipStream_t s)
{
    // Four channels a lane for bf16 where that leaves two workgroups for every
    // CU and few lanes idle (2^20 x 1,024: 1.57 ms, 1.68 with two; 65,536 x 4,096:
    // 389 us both; 4,096 x 1,024 with its 128 workgroups: 22 us, 16 with two).  In
    // between, two can be better: 32,768 x 1,024 takes 77 us, 66 with two.  fp32
    // tokens of four would not fit the registers.
    const int64_t wide = ((int64_t)D + 255) / 256;
    if (sizeof(T) == 2 && ch.ntiles * wide >= 512 && 4 * (int64_t)D >= 3 * 256 * wide)
        return run_scan<T, sizeof(T) == 2 ? 4 : 2>(x, g, init, sq, D, out, fin, chk, ch, s);
    return one_channel(ch) ? run_scan<T, 1>(x, g, init, sq, D, out, fin, chk, ch, s)
                           : run_scan<T, 2>(x, g, init, sq, D, out, fin, chk, ch, s);
}

template <typename T, int V>
hipError_t run_scan_backward(const void *x, const float *g, const float *init, const Seqs &sq, int32_t D,
                             const void *dout, const float *dfin, const float *chk, void *dx, float *dg, float *dinit,
                             Chain ch, hipStream_t s)
{
    ch.width = kda_column_width(D, V);
    const int32_t cols = (D - 1) / ch.width + 1;
    const int64_t work = sq.T > 0 ? (int64_t)cols * ch.ntiles : 0, groups = work + empty_groups(sq.N, dfin, dinit);
    if (groups > 0)
        hipLaunchKernelGGL((kda_scan_bwd_kernel<T, V>), dim3((unsigned)groups), dim3(NTH), 0, s, (const T *)x, g, init,
                           sq, (int64_t)D, cols, (uint32_t)work, (const T *)dout, dfin, chk, (T *)dx, dg, dinit, ch);
    return hipGetLastError();
}

template <typename T>
hipError_t scan_backward(const void *x, const float *g, const float *init, const Seqs &sq, int32_t D, const void *dout,
                         const float *dfin, const float *chk, void *dx, float *dg, float *dinit, const Chain &ch,
                         hipStream_t s)
{
    return one_channel(ch) ? run_scan_backward<T, 1>(x, g, init, sq, D, dout, dfin, chk, dx, dg, dinit, ch, s)
                           : run_scan_backward<T, 2>(x, g, init, sq, D, dout, dfin, chk, dx, dg, dinit, ch, s);
}

}  // namespace kda

using namespace kda;

// (by the widest grid there can be for these sizes, of columns of 64)
bool kda_scan_fits(int32_t N, int32_t T, int32_t D)
{
    return kda_grid_ok((int64_t)tiles_of(T) * (((int64_t)D + 63) / 64) + N / EMPTY_SEQS + 1, NTH);
}

size_t kda_scan_ws_bytes(int32_t T, int32_t D) { return chain_layout(T, D).words * sizeof(uint64_t); }

hipError_t kda_launch_scan(bool bf16, const void *x, const float *g, const float *init, const int32_t *cu, int32_t N,
                           int32_t T, int32_t D, void *out, float *fin, float *chk, void *ws, hipStream_t s)
{
    const Seqs sq{cu, N, T};
    const Chain ch = chain_at((uint64_t *)ws, T, D);
    if (hipError_t e = fill_chain((uint64_t *)ws, chain_layout(T, D).words, s)) return e;
    return bf16 ? scan<bf16_t>(x, g, init, sq, D, out, fin, chk, ch, s)
                : scan<float>(x, g, init, sq, D, out, fin, chk, ch, s);
}

hipError_t kda_launch_scan_step(bool bf16, const void *x, const float *g, float *state, int64_t n, void *out,
                                hipStream_t s)
{
    const int64_t want = (n + 255) / 256;
    const unsigned blocks = (unsigned)(want < 65536 ? want : 65536);
    if (bf16)
        hipLaunchKernelGGL(kda_scan_step_kernel<bf16_t>, dim3(blocks), dim3(256), 0, s, (const bf16_t *)x, g, state, n,
                           (bf16_t *)out);
    else
        hipLaunchKernelGGL(kda_scan_step_kernel<float>, dim3(blocks), dim3(256), 0, s, (const float *)x, g, state, n,
                           (float *)out);
    return hipGetLastError();
}

// Without checkpoints: a second chain and the checkpoints of a forward pass of our own.
size_t kda_scan_bwd_ws_bytes(int32_t T, int32_t D, bool has_checkpoints)
{
    const size_t words = chain_layout(T, D).words;
    if (words == 0 || has_checkpoints) return words * sizeof(uint64_t);
    return 2 * words * sizeof(uint64_t) + (size_t)tiles_of(T) * D * sizeof(float);
}

hipError_t kda_launch_scan_backward(bool bf16, const void *x, const float *g, const float *init, const int32_t *cu,
                                    int32_t N, int32_t T, int32_t D, const void *dout, const float *dfinal,
                                    const float *checkpoints, void *dx, float *dg, float *dinit, void *ws,
                                    hipStream_t s)
{
    const Seqs sq{cu, N, T};
    const size_t words = chain_layout(T, D).words;
    uint64_t *w = (uint64_t *)ws;
    const bool states = words > 0 && !checkpoints;
    if (hipError_t e = fill_chain(w, states ? 2 * words : words, s)) return e;
    if (states) {
        float *chk = reinterpret_cast<float *>(w + 2 * words);
        const Chain ch = chain_at(w + words, T, D);
        if (hipError_t e = bf16 ? scan<bf16_t>(x, g, init, sq, D, nullptr, nullptr, chk, ch, s)
                                : scan<float>(x, g, init, sq, D, nullptr, nullptr, chk, ch, s))
            return e;
        checkpoints = chk;
    }
    const Chain ch = chain_at(w, T, D);
    return bf16 ? scan_backward<bf16_t>(x, g, init, sq, D, dout, dfinal, checkpoints, dx, dg, dinit, ch, s)
                : scan_backward<float>(x, g, init, sq, D, dout, dfinal, checkpoints, dx, dg, dinit, ch, s);
}
