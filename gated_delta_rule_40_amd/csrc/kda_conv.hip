// kda_conv.hip -- short causal convolution over the tokens of packed
// sequences, per channel, with an optional SiLU; its decode step and gradients.
//
//     pre_t = bias + sum_{j < W} w_j x_{t - (W - 1) + j},  out_t = silu(pre_t)
//     dpre_t = dout_t silu'(pre_t),  dx_t = sum_k w_{W-1-k} dpre_{t + k}
//     dw_j = sum_t dpre_t x_{t - (W - 1) + j},  dbias = sum_t dpre_t
//
// One wave walks a strip of tokens of 64 V channels (V consecutive channels a
// lane), the last W - 1 inputs and the weights in registers: every input is read
// once (and W - 1 rows of it at a strip's edge once more, mostly from cache) and
// every output written once, so HBM's rate is the bound.  Rows are read a batch
// ahead of their use.
//
// Measured on one MI355X (a large copy reaches 4.9-5.4 TB/s there), width 4 with
// SiLU, bf16: 65,536 x 4,096 196 us (5.5 TB/s), its backward for 131,072 x 2,048
// 326 us (4.9 TB/s; 32 vector instructions an element take two thirds of that),
// 512 single tokens x 12,288 19.5 us (5.2 TB/s).
//
// A sequence's initial state is read by the wave whose strip holds the
// sequence's first token and by no other: that wave also computes the first
// W - 1 tokens where they lie beyond its strip, and writes the final state, so
// that the state may be updated in place.
#include "kda_colsum.hpp"
#include "kda_device.hpp"
#include "kda_layer.hpp"
#include "kda_seq.hpp"

#include <type_traits>

namespace kda {

struct ConvArgs {
    const float *w, *bias;   // [D][W], [D] or null
    int64_t D;
    bool silu;
};

// V consecutive channels of a row, as held and as they lie in memory
template <typename T, int V> struct Row {
    typedef T raw __attribute__((ext_vector_type(V)));
    typedef raw mem __attribute__((aligned(sizeof(T))));
    __device__ static __forceinline__ float at(const raw &r, int j) { return to_f(r[j]); }
    __device__ static __forceinline__ void set(raw &r, int j, float v) { r[j] = from_f<T>(v); }
};
template <typename T> struct Row<T, 1> {
    typedef T raw, mem;
    __device__ static __forceinline__ float at(const raw &r, int) { return to_f(r); }
    __device__ static __forceinline__ void set(raw &r, int, float v) { r = from_f<T>(v); }
};
template <typename T, int V> __device__ __forceinline__ typename Row<T, V>::raw load_row(const T *p)
{
    return *reinterpret_cast<const typename Row<T, V>::mem *>(p);
}
template <typename T, int V> __device__ __forceinline__ void store_row(T *p, const typename Row<T, V>::raw &r)
{
    *reinterpret_cast<typename Row<T, V>::mem *>(p) = r;
}
// outputs are not read here again: past the caches
template <typename T, int V> __device__ __forceinline__ void write_once(T *p, const typename Row<T, V>::raw &r)
{
    __builtin_nontemporal_store(r, reinterpret_cast<typename Row<T, V>::mem *>(p));
}

// 1 / (1 + exp(-p)): exp within |p| + 2 units in the last place, the quotient
// one more.  Where exp overflows the quotient is 0, the limit.
__device__ __forceinline__ float sigmoid_f(float p) { return __builtin_amdgcn_rcpf(1.f + __expf(-p)); }
__device__ __forceinline__ float silu_f(float p) { return p * sigmoid_f(p); }
__device__ __forceinline__ float dsilu_f(float p)
{
    const float s = sigmoid_f(p);
    return s * (1.f + p * (1.f - s));
}

template <int W, int V> struct Weights {
    float w[W][V], b[V];
    __device__ __forceinline__ void load(const ConvArgs &a, int64_t c) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            b[v] = a.bias ? a.bias[c + v] : 0.f;
#pragma unroll
            for (int j = 0; j < W; ++j) w[j][v] = a.w[(c + v) * W + j];
        }
    }
};

// The row that lies k tokens before token t of a sequence whose first token is
// s: an input, or a row of its initial state (null: zeros).
template <typename T, int W, int V>
__device__ __forceinline__ typename Row<T, V>::raw row_before(const T *x, const T *init, const ConvArgs &a, int64_t c,
                                                              int32_t n, int32_t s, int32_t t, int k)
{
    const int32_t p = t - s - k;
    if (p >= 0) return load_row<T, V>(x + (int64_t)(t - k) * a.D + c);
    if (init) return load_row<T, V>(init + ((int64_t)n * (W - 1) + W - 1 + p) * a.D + c);
    return typename Row<T, V>::raw{};
}

// ---------------------------------------------------------------- forward
template <typename T, int W, int V, bool SILU>
__global__ __launch_bounds__(256)
void kda_conv_kernel(const T *x, const T *init, ConvArgs a, Seqs sq, int32_t strip, int32_t nstrips, int32_t cols,
                     int32_t width, uint32_t work, T *out, T *fin)
{
    typedef typename Row<T, V>::raw R;
    constexpr int BATCH = 4;
    if (blockIdx.x >= work) return copy_empty(sq, blockIdx.x - work, (W - 1) * a.D, init, fin);
    const int32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int32_t k = (int32_t)(blockIdx.x / cols) * 4 + wave;
    // A lane past its column or the last channel repeats the column's last lane.
    const int64_t c0 = (int64_t)(blockIdx.x % cols) * width;
    const int64_t c = min(c0 + (int64_t)min((int32_t)(threadIdx.x & 63) * V, width - V), a.D - V);
    if (k >= nstrips) return;
    SeqWindow win(sq);
    const int32_t t0 = k * strip, t1 = (int32_t)min((int64_t)t0 + strip, (int64_t)sq.T);
    const int32_t tend = sq.at(sq.N);
    Weights<W, V> wt;
    wt.load(a, c);
    win.locate(t0);

    if (t0 < tend) {
        int32_t n = win.owner(t0);
        if (n < 0) return;                     // (cu_seqlens against its rules)
        // (held to what a valid cu_seqlens gives: s <= t0 < next)
        int32_t s = min(win.at(n), t0), next = max(win.at(n + 1), t0 + 1), t = t0;
        // tokens that belong to the wave of their sequence's start
        if (s < t0 && t0 - s < W - 1) t = min(s + W - 1, next);
        const int32_t stop = min(t1, tend);
        float before[W - 1][V];                // the last W - 1 inputs, unpacked once
        auto enter = [&]() {
#pragma unroll
            for (int j = 0; j < W - 1; ++j) {
                const R r = row_before<T, W, V>(x, init, a, c, n, s, t, W - 1 - j);
#pragma unroll
                for (int v = 0; v < V; ++v) before[j][v] = Row<T, V>::at(r, v);
            }
        };
        // The sequence's last token is done: the window is its final state.  (Not
        // where that takes the initial state's place: the wave of the sequence's
        // start may still have to read it.)
        auto leave = [&]() {
            if (!fin || fin == init) return;
#pragma unroll
            for (int j = 0; j < W - 1; ++j) {
                R r;
#pragma unroll
                for (int v = 0; v < V; ++v) Row<T, V>::set(r, v, before[j][v]);
                store_row<T, V>(fin + ((int64_t)n * (W - 1) + j) * a.D + c, r);
            }
        };
        auto advance = [&]() {                 // to the sequence that begins at token t
            win.advance(t, n, next);
            s = t;
        };
        auto token = [&](const R &r) {
            R o;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float in = Row<T, V>::at(r, v);
                float p = wt.b[v] + wt.w[W - 1][v] * in;
#pragma unroll
                for (int j = 0; j < W - 1; ++j) p += wt.w[j][v] * before[j][v];
                Row<T, V>::set(o, v, SILU ? silu_f(p) : p);
#pragma unroll
                for (int j = 0; j + 1 < W - 1; ++j) before[j][v] = before[j + 1][v];
                before[W - 2][v] = in;
            }
            write_once<T, V>(out + (int64_t)t * a.D + c, o);
            ++t;
        };
        auto read = [&](R (&rows)[BATCH], int32_t from) {
#pragma unroll
            for (int i = 0; i < BATCH; ++i) rows[i] = load_row<T, V>(x + (int64_t)min(from + i, stop - 1) * a.D + c);
        };
        if (t < stop) {
            if (t == next) advance();
            R rows[BATCH], ahead[BATCH];
            read(rows, t);
            enter();
            while (t < stop) {
                read(ahead, t + BATCH);
                if (stop - t >= BATCH && next >= t + BATCH) {
#pragma unroll
                    for (int i = 0; i < BATCH; ++i) token(rows[i]);
                    if (t == next) {
                        leave();
                        if (t < stop) {
                            advance();
                            enter();
                        }
                    }
                } else {
                    const int32_t m = min(stop - t, BATCH);
#pragma unroll
                    for (int i = 0; i < BATCH; ++i) {
                        if (i < m) {
                            token(rows[i]);
                            if (t == next) {
                                leave();
                                if (t < stop) {
                                    advance();
                                    enter();
                                }
                            }
                        }
                    }
                }
#pragma unroll
                for (int i = 0; i < BATCH; ++i) rows[i] = ahead[i];
            }
        }
        // the first W - 1 tokens of the last sequence that begins here, beyond the strip
        if (s >= t0 && t > s && t >= t1) {
            const int32_t most = min(min(s + W - 1, next), tend);
            while (t < most) {
                token(load_row<T, V>(x + (int64_t)t * a.D + c));
                if (t == next) leave();
            }
        }
    }
    // Final states in the initial states' place, of the sequences that begin here:
    // the walk has read those by now.
    if (fin && fin == init)
        for (int32_t t = t0; t < min(t1, tend);) {
            const int32_t s = win.sq.at(min(win.first_at_or_after(t), sq.N)), n = win.owner(s);
            if (s < t || s >= min(t1, tend) || n < 0) break;
            const int32_t e = max(win.at(n + 1), s + 1);
            R r[W - 1];
#pragma unroll
            for (int j = 0; j < W - 1; ++j) r[j] = row_before<T, W, V>(x, init, a, c, n, s, e, W - 1 - j);
#pragma unroll
            for (int j = 0; j < W - 1; ++j) store_row<T, V>(fin + ((int64_t)n * (W - 1) + j) * a.D + c, r[j]);
            t = e;
        }
}

// ---------------------------------------------------------------- decode
// A thread takes PER sequences of its channels with one reading of the weights,
// all their rows read before any is used.
template <typename T, int W, int V, int PER>
__global__ __launch_bounds__(256) void kda_conv_step_kernel(const T *x, T *state, ConvArgs a, int32_t N, int32_t cols,
                                                            T *out)
{
    typedef typename Row<T, V>::raw R;
    const int64_t c = ((int64_t)(blockIdx.x % cols) * blockDim.x + threadIdx.x) * V;
    if (c >= a.D) return;
    const int64_t n0 = (int64_t)(blockIdx.x / cols) * PER;
    R r[PER][W];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int64_t n = min(n0 + i, (int64_t)N - 1);
#pragma unroll
        for (int j = 0; j < W - 1; ++j) r[i][j] = load_row<T, V>(state + (n * (W - 1) + j) * a.D + c);
        r[i][W - 1] = load_row<T, V>(x + n * a.D + c);
    }
    Weights<W, V> wt;
    wt.load(a, c);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int64_t n = n0 + i;
        if (n >= N) break;
        R o;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float p = wt.b[v];
#pragma unroll
            for (int j = 0; j < W; ++j) p += wt.w[j][v] * Row<T, V>::at(r[i][j], v);
            Row<T, V>::set(o, v, a.silu ? silu_f(p) : p);
        }
#pragma unroll
        for (int j = 0; j < W - 1; ++j) store_row<T, V>(state + (n * (W - 1) + j) * a.D + c, r[i][j + 1]);
        store_row<T, V>(out + n * a.D + c, o);
    }
}

// ---------------------------------------------------------------- gradients
// The walk keeps the W - 1 newest places' dx unfinished in `acc` (the place of
// token t takes from dpre_t .. dpre_{t + W - 1}); at a sequence's start they
// stand for its initial state's rows, at its end the final state's gradient
// joins them.  A strip's wave finishes the places of its tokens, and of the
// initial states of the sequences that begin in it, by walking W - 1 tokens
// beyond the strip; only its own tokens count for dw and dbias.
template <typename T, int W, int V, bool SILU>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(3)))
void kda_conv_bwd_kernel(const T *x, const T *init, ConvArgs a, Seqs sq, int32_t strip, int32_t nstrips, int32_t cols,
                         uint32_t work, const T *dout, const T *dfin, T *dx, T *dinit, float *partial)
{
    typedef typename Row<T, V>::raw R;
    constexpr int BATCH = 4;
    if (blockIdx.x >= work) return copy_empty(sq, blockIdx.x - work, (W - 1) * a.D, dfin, dinit);
    __shared__ float sums[4][W + 1][64 * V];
    const int32_t lane = threadIdx.x & 63;
    const int32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int32_t part = blockIdx.x / cols, k = part * 4 + wave;
    const int64_t c0 = (int64_t)(blockIdx.x % cols) * 64 * V, c = min(c0 + lane * V, a.D - V);
    float dw[W][V] = {}, db[V] = {};
    if (k < nstrips) {
        SeqWindow win(sq);
        const int32_t t0 = (int32_t)min((int64_t)k * strip, (int64_t)sq.T);
        const int32_t t1 = (int32_t)min((int64_t)t0 + strip, (int64_t)sq.T), tend = sq.at(sq.N);
        win.locate(t0);
        auto put_dinit = [&](int32_t n, int j, const float (&v)[V]) {
            R r;
#pragma unroll
            for (int i = 0; i < V; ++i) Row<T, V>::set(r, i, v[i]);
            store_row<T, V>(dinit + ((int64_t)n * (W - 1) + j) * a.D + c, r);
        };
        auto get_dfin = [&](int32_t n, int j) {
            return dfin ? load_row<T, V>(dfin + ((int64_t)n * (W - 1) + j) * a.D + c) : R{};
        };
        int32_t n = t0 < min(tend, t1) ? win.owner(t0) : -1;
        if (n >= 0) {
            Weights<W, V> wt;
            wt.load(a, c);
            // (held to what a valid cu_seqlens gives: s <= t0 < next)
            int32_t s = min(win.at(n), t0), next = max(win.at(n + 1), t0 + 1), t = t0;
            float before[W - 1][V];   // the last W - 1 inputs, unpacked once
            float acc[W - 1][V] = {};
            auto enter = [&]() {
#pragma unroll
                for (int j = 0; j < W - 1; ++j) {
                    const R r = row_before<T, W, V>(x, init, a, c, n, s, t, W - 1 - j);
#pragma unroll
                    for (int v = 0; v < V; ++v) before[j][v] = Row<T, V>::at(r, v);
                }
            };
            // place p of the sequence (p < 0: of its initial state) is finished
            auto finish = [&](int32_t p, const float (&v)[V]) {
                if (p >= 0) {
                    if (s + p < t0 || s + p >= t1) return;
                    R r;
#pragma unroll
                    for (int i = 0; i < V; ++i) Row<T, V>::set(r, i, v[i]);
                    write_once<T, V>(dx + (int64_t)(s + p) * a.D + c, r);
                } else if (dinit && s >= t0 && s < t1) {
                    put_dinit(n, p + W - 1, v);
                }
            };
            const int32_t stop = (int32_t)min((int64_t)t1 + W - 1, (int64_t)tend);
            auto token = [&](const R &r, const R &d) {
                float done[V], in[W][V], g[V];
#pragma unroll
                for (int v = 0; v < V; ++v) {
#pragma unroll
                    for (int j = 0; j < W - 1; ++j) in[j][v] = before[j][v];
                    in[W - 1][v] = Row<T, V>::at(r, v);
                    g[v] = Row<T, V>::at(d, v);
                    if (SILU) {
                        float p = wt.b[v];
#pragma unroll
                        for (int j = 0; j < W; ++j) p += wt.w[j][v] * in[j][v];
                        g[v] *= dsilu_f(p);
                    }
                }
                if (t < t1) {   // one branch for all channels
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        db[v] += g[v];
#pragma unroll
                        for (int j = 0; j < W; ++j) dw[j][v] += g[v] * in[j][v];
                    }
                }
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    done[v] = acc[0][v] + g[v] * wt.w[0][v];
#pragma unroll
                    for (int j = 0; j + 1 < W - 1; ++j) acc[j][v] = acc[j + 1][v] + g[v] * wt.w[j + 1][v];
                    acc[W - 2][v] = g[v] * wt.w[W - 1][v];
                }
                finish(t - s - (W - 1), done);
#pragma unroll
                for (int v = 0; v < V; ++v) {
#pragma unroll
                    for (int j = 0; j + 1 < W - 1; ++j) before[j][v] = before[j + 1][v];
                    before[W - 2][v] = in[W - 1][v];
                }
                ++t;
            };
            // the sequence ends before token t: its unfinished places, then the next sequence
            auto leave = [&]() {
#pragma unroll
                for (int j = 0; j < W - 1; ++j) {
                    const R f = get_dfin(n, j);
#pragma unroll
                    for (int v = 0; v < V; ++v) acc[j][v] += Row<T, V>::at(f, v);
                    finish(t - s - (W - 1) + j, acc[j]);
#pragma unroll
                    for (int v = 0; v < V; ++v) acc[j][v] = 0.f;
                }
                if (t < stop) win.advance(t, n, next);
                s = t;
            };
            R xr[BATCH], dr[BATCH], xa[BATCH], da[BATCH];
            auto read = [&](R (&xs)[BATCH], R (&ds)[BATCH], int32_t from) {
#pragma unroll
                for (int i = 0; i < BATCH; ++i) {
                    const int64_t at = (int64_t)min(from + i, stop - 1) * a.D + c;
                    xs[i] = load_row<T, V>(x + at);
                    ds[i] = load_row<T, V>(dout + at);
                }
            };
            read(xr, dr, t);
            enter();
            bool over = false;
            while (t < stop && !over) {
                read(xa, da, t + BATCH);
                const int32_t m = min(stop - t, BATCH);
#pragma unroll
                for (int i = 0; i < BATCH; ++i) {
                    if (i < m && !over) {
                        token(xr[i], dr[i]);
                        if (t == next) {
                            leave();
                            over = t >= t1 || t >= stop;   // nothing of ours is unfinished
                            if (!over) enter();
                        }
                    }
                }
#pragma unroll
                for (int i = 0; i < BATCH; ++i) xr[i] = xa[i], dr[i] = da[i];
            }
        }
    }
    // the four waves' sums, in order, as the workgroup's part
    // (a lane whose channels overlap its neighbour's writes the same values
    // there; those of the workgroup before are that one's)
    const int place = (int)(c - c0);
#pragma unroll
    for (int v = 0; v < V; ++v) {
        if (place + v < 0) continue;
        sums[wave][W][place + v] = db[v];
#pragma unroll
        for (int j = 0; j < W; ++j) sums[wave][j][place + v] = dw[j][v];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < (W + 1) * 64 * V; i += 256) {
        const int j = i / (64 * V), cc = i % (64 * V);
        const float total = ((sums[0][j][cc] + sums[1][j][cc]) + sums[2][j][cc]) + sums[3][j][cc];
        if (c0 + cc < a.D) partial[((int64_t)part * (W + 1) + j) * a.D + c0 + cc] = total;
    }
}

// dw[c][j] and dbias[c] from the workgroups' parts [n][W + 1][D]
template <int W>
__global__ __launch_bounds__(COLSUM_THREADS) void kda_conv_sums_kernel(const float *src, int32_t n, int64_t D,
                                                                       float *dw, float *dbias)
{
    const int64_t i = (int64_t)blockIdx.x * COLSUM_COLS + threadIdx.x % COLSUM_COLS;
    const float s = column_sum(src, n, (W + 1) * D, i);
    if (threadIdx.x >= COLSUM_COLS || i >= (W + 1) * D) return;
    const int64_t j = i / D, c = i % D;
    if (j < W) dw[c * W + j] = s;
    else if (dbias) dbias[c] = s;
}

// ---------------------------------------------------------------- host
inline int64_t up(int64_t n, int64_t per) { return (n + per - 1) / per; }

// The backward's strips: as long as three workgroups for every CU allow (what
// its registers let be resident at once; longer strips also read fewer rows
// twice and leave fewer partial sums: 131,072 x 2,048 with the forward 555 us,
// 575 with 1,024 workgroups, 588 with 2,048), and 16 tokens at least.
constexpr int32_t BWD_GROUPS = 768;
constexpr int BWD_V = 4;   // channels a lane (the sums and unfinished places of eight would not fit the registers)

// Rows too short for BWD_V channels a lane (most lanes would be idle) take one
// (200,000 x 64 with the forward: 51 us, 74 with four; x 192: 128, 105).
inline bool bwd_wide(int64_t D) { return D >= 128; }
inline int64_t bwd_cols(int64_t D) { return up(D, bwd_wide(D) ? 64 * BWD_V : 64); }
inline int32_t bwd_strip(int32_t T, int64_t D)
{
    const int64_t parts = up(BWD_GROUPS, bwd_cols(D)), len = up(T, parts * 4);
    return (int32_t)(len < 16 ? 16 : len);
}
inline int32_t bwd_parts(int32_t T, int64_t D) { return (int32_t)(T > 0 ? up(up(T, bwd_strip(T, D)), 4) : 1); }
inline int32_t bwd_walks(int32_t N, int32_t T, int64_t D) { return N > 0 ? bwd_parts(T, D) : 0; }

// Short strips: the waves that begin and end spread reads and writes evenly
// (65,536 x 4,096, V = 4: 8 tokens 222 us, 12 199, 16 196, 24 203, 64 207;
// 8,192 x 2,048: 14.4, 14.2, 13.0, 13.9).
constexpr int32_t STRIP = 16;

// workgroups of a prefill's walk, at V channels a lane
inline int64_t conv_walks(int32_t T, int64_t D, int V)
{
    return up(up(T, STRIP), 4) * up(D, kda_column_width((int32_t)D, V));
}

template <typename T, int W, int V>
hipError_t run_conv(const void *x, const ConvArgs &a, const void *init, const Seqs &sq, void *out, void *fin,
                    hipStream_t s)
{
    const int32_t cw = kda_column_width((int32_t)a.D, V);
    const int64_t cols = up(a.D, cw);
    const int32_t strip = STRIP;
    const int32_t nstrips = (int32_t)up(sq.T, strip);
    const int64_t work = conv_walks(sq.T, a.D, V), groups = work + empty_groups(sq.N, init, fin);
    if (groups == 0) return hipSuccess;
    if (a.silu)
        hipLaunchKernelGGL((kda_conv_kernel<T, W, V, true>), dim3((unsigned)groups), dim3(256), 0, s, (const T *)x,
                           (const T *)init, a, sq, strip, nstrips, (int32_t)cols, cw, (uint32_t)work, (T *)out,
                           (T *)fin);
    else
        hipLaunchKernelGGL((kda_conv_kernel<T, W, V, false>), dim3((unsigned)groups), dim3(256), 0, s, (const T *)x,
                           (const T *)init, a, sq, strip, nstrips, (int32_t)cols, cw, (uint32_t)work, (T *)out,
                           (T *)fin);
    return hipGetLastError();
}

// Four sequences to a reading of the weights where there are many, by the
// workgroups of one each (replays, bf16; 1,024: 512 x 4,096 10.7 us, 15.0 with one
// sequence; 384: 192 x 4,096 6.9, 8.2 and 64 x 12,288 7.1, 8.3; 288: 48 x 12,288
// 6.8, 8.0; 256: 128 x 4,096 6.7, 6.3; 48: 8 x 12,288 6.3, 5.5).
inline bool step_many(int32_t N, int64_t cols) { return N * cols >= 384; }

template <typename T, int W, int V>
hipError_t run_conv_step(const void *x, const ConvArgs &a, void *state, int32_t N, void *out, hipStream_t s)
{
    const int64_t cols = up(a.D, 256 * V);
    if (step_many(N, cols))
        hipLaunchKernelGGL((kda_conv_step_kernel<T, W, V, 4>), dim3((unsigned)(cols * up(N, 4))), dim3(256), 0, s,
                           (const T *)x, (T *)state, a, N, (int32_t)cols, (T *)out);
    else
        hipLaunchKernelGGL((kda_conv_step_kernel<T, W, V, 1>), dim3((unsigned)(cols * N)), dim3(256), 0, s,
                           (const T *)x, (T *)state, a, N, (int32_t)cols, (T *)out);
    return hipGetLastError();
}

template <typename T, int W, int V>
hipError_t run_conv_backward(const void *x, const ConvArgs &a, const void *init, const Seqs &sq, const void *dout,
                             const void *dfin, void *dx, float *dw, float *dbias, void *dinit, void *ws,
                             hipStream_t s)
{
    const int32_t strip = bwd_strip(sq.T, a.D), parts = bwd_walks(sq.N, sq.T, a.D);
    const int64_t cols = bwd_cols(a.D), work = parts * cols, groups = work + empty_groups(sq.N, dfin, dinit);
    const int32_t nstrips = (int32_t)up(sq.T, strip);
    if (groups > 0 && a.silu)
        hipLaunchKernelGGL((kda_conv_bwd_kernel<T, W, V, true>), dim3((unsigned)groups), dim3(256), 0, s, (const T *)x,
                           (const T *)init, a, sq, strip, nstrips, (int32_t)cols, (uint32_t)work, (const T *)dout,
                           (const T *)dfin, (T *)dx, (T *)dinit, (float *)ws);
    else if (groups > 0)
        hipLaunchKernelGGL((kda_conv_bwd_kernel<T, W, V, false>), dim3((unsigned)groups), dim3(256), 0, s, (const T *)x,
                           (const T *)init, a, sq, strip, nstrips, (int32_t)cols, (uint32_t)work, (const T *)dout,
                           (const T *)dfin, (T *)dx, (T *)dinit, (float *)ws);
    hipLaunchKernelGGL(kda_conv_sums_kernel<W>, dim3((unsigned)up((W + 1) * a.D, COLSUM_COLS)),
                       dim3(COLSUM_THREADS), 0, s,
                       (const float *)ws, parts, a.D, dw, dbias);
    return hipGetLastError();
}

// calls f with the width and the piece as compile-time numbers
template <int V, typename F> hipError_t with_width(int32_t width, F f)
{
    switch (width) {
    case 2: return f(std::integral_constant<int, 2>(), std::integral_constant<int, V>());
    case 3: return f(std::integral_constant<int, 3>(), std::integral_constant<int, V>());
    default: return f(std::integral_constant<int, 4>(), std::integral_constant<int, V>());
    }
}

// Channels a lane: four (65,536 x 4,096 in bf16: 196 us, 203 with two, 206 with
// eight; 16,384 x 4,096: 44, 47, 54), or fewer where many lanes would be idle
// (200,000 x 320: 51 us, 45 with two; x 300: bf16 55, 59, fp32 134, 119; 200,000 x
// 64: 26, 16 with one).
inline int conv_lane(int64_t D)
{
    if (D <= 64) return 1;
    const bool idle = D > 256 && 4 * D <= 3 * 256 * up(D, 256);
    return D <= 128 || idle ? 2 : 4;
}

template <typename T>
hipError_t conv(const void *x, const ConvArgs &a, const void *init, const Seqs &sq, int32_t width, void *out, void *fin,
                hipStream_t s)
{
    auto f = [&](auto w, auto v) { return run_conv<T, w(), v()>(x, a, init, sq, out, fin, s); };
    const int lane = conv_lane(a.D);
    return lane == 1 ? with_width<1>(width, f) : lane == 2 ? with_width<2>(width, f) : with_width<4>(width, f);
}

// Channels a thread of the token call: 16 bytes, where rows are made of them.
template <typename T> constexpr int step_lane(int64_t D) { return D % (16 / sizeof(T)) == 0 ? 16 / sizeof(T) : 1; }

template <typename T>
hipError_t conv_step(const void *x, const ConvArgs &a, void *state, int32_t N, int32_t width, void *out, hipStream_t s)
{
    auto f = [&](auto w, auto v) { return run_conv_step<T, w(), v()>(x, a, state, N, out, s); };
    return step_lane<T>(a.D) > 1 ? with_width<16 / sizeof(T)>(width, f) : with_width<1>(width, f);
}

template <typename T>
hipError_t conv_backward(const void *x, const ConvArgs &a, const void *init, const Seqs &sq, int32_t width,
                         const void *dout, const void *dfin, void *dx, float *dw, float *dbias, void *dinit, void *ws,
                         hipStream_t s)
{
    auto f = [&](auto w, auto v) {
        return run_conv_backward<T, w(), v()>(x, a, init, sq, dout, dfin, dx, dw, dbias, dinit, ws, s);
    };
    return bwd_wide(a.D) ? with_width<BWD_V>(width, f) : with_width<1>(width, f);
}

}  // namespace kda

using namespace kda;

bool kda_conv_fits(int32_t N, int32_t T, int32_t D, const void *init, const void *fin)
{
    return kda_grid_ok(conv_walks(T, D, conv_lane(D)) + empty_groups(N, init, fin), 256);
}

bool kda_conv_step_fits(bool bf16, int32_t N, int32_t D)
{
    const int64_t cols = up(D, 256 * (bf16 ? step_lane<bf16_t>(D) : step_lane<float>(D)));
    return kda_grid_ok(step_many(N, cols) ? cols * up(N, 4) : cols * N, 256);
}

bool kda_conv_backward_fits(int32_t N, int32_t T, int32_t D, int32_t width, const void *dfinal, const void *dinit)
{
    return kda_grid_ok(bwd_walks(N, T, D) * bwd_cols(D) + empty_groups(N, dfinal, dinit), 256) &&
           kda_grid_ok(up((width + 1) * (int64_t)D, COLSUM_COLS), COLSUM_THREADS);
}

hipError_t kda_launch_conv(bool bf16, const void *x, const float *w, const float *bias, const void *init,
                           const int32_t *cu, int32_t N, int32_t T, int32_t D, int32_t width, bool silu, void *out,
                           void *fin, hipStream_t s)
{
    const ConvArgs a{w, bias, D, silu};
    const Seqs sq{cu, N, T};
    return bf16 ? conv<bf16_t>(x, a, init, sq, width, out, fin, s) : conv<float>(x, a, init, sq, width, out, fin, s);
}

hipError_t kda_launch_conv_step(bool bf16, const void *x, const float *w, const float *bias, void *state, int32_t N,
                                int32_t D, int32_t width, bool silu, void *out, hipStream_t s)
{
    const ConvArgs a{w, bias, D, silu};
    return bf16 ? conv_step<bf16_t>(x, a, state, N, width, out, s) : conv_step<float>(x, a, state, N, width, out, s);
}

size_t kda_conv_bwd_ws_bytes(int32_t T, int32_t D, int32_t width, bool)
{
    return (size_t)bwd_parts(T, D) * (width + 1) * D * sizeof(float);
}

hipError_t kda_launch_conv_backward(bool bf16, const void *x, const float *w, const float *bias, const void *init,
                                    const int32_t *cu, int32_t N, int32_t T, int32_t D, int32_t width, bool silu,
                                    const void *dout, const void *dfinal, void *dx, float *dw, float *dbias,
                                    void *dinit, void *ws, hipStream_t s)
{
    const ConvArgs a{w, bias, D, silu};
    const Seqs sq{cu, N, T};
    return bf16 ? conv_backward<bf16_t>(x, a, init, sq, width, dout, dfinal, dx, dw, dbias, dinit, ws, s)
                : conv_backward<float>(x, a, init, sq, width, dout, dfinal, dx, dw, dbias, dinit, ws, s);
}
